// paged_copy.cu — pages copied in every layer's cache, as a list on the device
// asks for.
//
// A (page, layer) is one run of 16-byte pieces over its arrays (K, V, scales,
// block scales); a tile of it is kVecs pieces a thread, all loaded before the
// first is stored.  The number of pairs is known on the device only, so the
// grid is fixed and strides over the tiles.  HBM bound: every byte is read and
// written once (1,200 pages of 128 KB in 3 layers: 145 us, 944 MB, 6.5 TB/s; 40
// pages of 8.3 KB in 24 layers: 7 us).
#include "paged_pages.cuh"

namespace flamia {

namespace {

constexpr int kThreads = 256, kVecs = 8, kTile = kThreads * kVecs;

__global__ void __launch_bounds__(kThreads) paged_copy_kernel(const __grid_constant__ CopyParams p) {
  const int n = __ldg(p.n_copies);
  if (n < 0 || n > p.max_copies) {
    report(&p.hdr->base, FLAMIA_ERR_INVALID_ARG, 0x750);
    return;
  }
  const int page_vecs = 2 * (p.kv_vecs + p.scale_vecs + p.block_vecs), tiles = (page_vecs + kTile - 1) / kTile;
  const int64_t units = (int64_t)n * p.layers * tiles;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int64_t rest = unit / tiles;
    const int tile = (int)(unit - rest * tiles), pair = (int)(rest / p.layers), l = (int)(rest - (int64_t)pair * p.layers);
    const int from = __ldg(p.copies + 2 * (int64_t)pair), to = __ldg(p.copies + 2 * (int64_t)pair + 1);
    if ((unsigned)from >= (unsigned)p.n_pages || (unsigned)to >= (unsigned)p.n_pages) {
      report(&p.hdr->base, FLAMIA_ERR_BAD_PAGE, 0x751);
      continue;
    }
    const CopyLayer& c = p.layer[l];
    uint4 x[kVecs];
    uint8_t* dst[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      int v = tile * kTile + i * kThreads + threadIdx.x, a = 0, size = p.kv_vecs;
      dst[i] = nullptr;
      if (v >= page_vecs) continue;
      if (v >= 2 * p.kv_vecs) {
        v -= 2 * p.kv_vecs, a = 2, size = p.scale_vecs;
        if (v >= 2 * p.scale_vecs) v -= 2 * p.scale_vecs, a = 4, size = p.block_vecs;
      }
      if (v >= size) v -= size, ++a;
      const int64_t s = a < 2 ? p.src_stride[l] : (int64_t)size * 16, d = a < 2 ? p.dst_stride[l] : (int64_t)size * 16;
      x[i] = *reinterpret_cast<const uint4*>(c.src[a] + from * s + (int64_t)v * 16);
      dst[i] = c.dst[a] + to * d + (int64_t)v * 16;
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (dst[i]) *reinterpret_cast<uint4*>(dst[i]) = x[i];
  }
}

}  // namespace

cudaError_t launch_paged_copy(const CopyParams& p, int sms, cudaStream_t st) {
  paged_copy_kernel<<<sms * 8, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace flamia
