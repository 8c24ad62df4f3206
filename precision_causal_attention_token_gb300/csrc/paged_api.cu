// paged_api.cu — the C ABI of serving from a paged cache (include/flamia.h):
// host-side validation, workspace layout, TMA descriptors and launches.
#include <cmath>
#include <cudaTypedefs.h>

#include "kernels.h"
#include "paged_pages.cuh"

using namespace flamia;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool dev16(const void* p) { return p && aligned(p, 16); }
bool dev4(const void* p) { return p && aligned(p, 4); }

int max_q_of(const flamia_paged_t* p) { return p->max_q ? p->max_q : p->T; }

// Up to 32 query rows of a key/value head: the decode kernel, whose MMAs have
// 8, 16 or 32 columns for them and which is bound by the cache's bytes.  More
// rows: 256-row tiles on the tensor cores.
int path_of(const flamia_paged_t* p) {
  const int64_t rows = (int64_t)max_q_of(p) * (p->H / p->Hkv);
  return rows <= 8 ? kPathDecode8 : rows <= 16 ? kPathDecode16 : rows <= 32 ? kPathDecode32 : kPathChunk;
}

flamia_status_t validate(const flamia_paged_t* p) {
  if (!p) return FLAMIA_ERR_INVALID_ARG;
  if (p->n_req < 1 || p->T < 1 || p->H < 1 || p->Hkv < 1 || p->max_q < 0 || p->max_q > p->T || p->n_pages < 1 ||
      p->max_pages < 1 || p->H % p->Hkv != 0 || !dev4(p->cu_q) || !dev4(p->kv_len) || !dev4(p->block_table))
    return FLAMIA_ERR_INVALID_ARG;
  if (p->d != 64 && p->d != 128) return FLAMIA_ERR_UNSUPPORTED;
  if (p->page_size != 16 && p->page_size != 32 && p->page_size != 64 && p->page_size != 128) return FLAMIA_ERR_UNSUPPORTED;
  if (p->cache_dtype != FLAMIA_BF16 && p->cache_dtype != FLAMIA_E4M3 && p->cache_dtype != FLAMIA_E2M1) return FLAMIA_ERR_UNSUPPORTED;
  if (p->in_dtype != FLAMIA_BF16 && p->in_dtype != FLAMIA_F32) return FLAMIA_ERR_UNSUPPORTED;
  if (p->n_req > kMaxReq || p->T > (1 << 30) || p->H / p->Hkv > kChunkRows / 2) return FLAMIA_ERR_UNSUPPORTED;
  if ((int64_t)p->T * p->H * p->d >= (int64_t)1 << 40) return FLAMIA_ERR_UNSUPPORTED;
  if ((int64_t)p->n_pages * p->page_size > INT32_MAX || (int64_t)p->max_pages * p->page_size > (1 << 30) ||
      (int64_t)p->n_req * p->max_pages > INT32_MAX)
    return FLAMIA_ERR_UNSUPPORTED;
  if (path_of(p) == kPathChunk && (int64_t)p->max_pages * p->page_size > kMaxChunkKeys) return FLAMIA_ERR_UNSUPPORTED;
  if (!(p->softmax_scale >= 0.f) || std::isinf(p->softmax_scale)) return FLAMIA_ERR_INVALID_ARG;
  const int64_t kv_el = p->in_dtype == FLAMIA_BF16 ? 8 : 4;  // elements of 16 bytes
  if (p->q_stride && (p->q_stride < (int64_t)p->H * p->d || p->q_stride % 8)) return FLAMIA_ERR_INVALID_ARG;
  if (p->kv_stride && (p->kv_stride < (int64_t)p->Hkv * p->d || p->kv_stride % kv_el)) return FLAMIA_ERR_INVALID_ARG;
  return FLAMIA_OK;
}

PagedLayout layout(const flamia_paged_t& p) {
  PagedLayout L{};
  L.path = path_of(&p);
  const size_t dec = 2 * (size_t)kMaxWorkers * (L.path == kPathDecode8 ? 8 : L.path == kPathDecode32 ? 32 : 16);
  const size_t chunk = L.path == kPathChunk ? 2 * (size_t)kMaxChunkWorkers * kChunkRows : 0;
  auto a256 = [](size_t x) { return (x + 255) & ~size_t(255); };
  size_t o = 0;
  L.header = o; o = a256(o + sizeof(PagedHeader));
  L.reqs = o; o = a256(o + sizeof(ReqRec) * 2 * p.n_req);
  L.workers = o; o = a256(o + sizeof(WorkerRec) * (kMaxWorkers + kMaxChunkWorkers));
  L.part_ml = o; o = a256(o + sizeof(float2) * dec);
  L.part_o = o; o = a256(o + sizeof(float) * dec * p.d);
  L.chunk_ml = o; o = a256(o + sizeof(float2) * chunk);
  L.chunk_o = o; o = a256(o + sizeof(float) * chunk * p.d);
  L.total = o;
  return L;
}

flamia_status_t fill(const flamia_paged_t* p, void* ws, size_t ws_bytes, PagedParams* a) {
  flamia_status_t s = validate(p);
  if (s != FLAMIA_OK) return s;
  const PagedLayout L = layout(*p);
  if (!dev16(ws)) return FLAMIA_ERR_INVALID_ARG;
  if (ws_bytes < L.total) return FLAMIA_ERR_WORKSPACE_TOO_SMALL;
  *a = PagedParams{};
  a->n_req = p->n_req;
  a->T = p->T;
  a->max_q = max_q_of(p);
  a->H = p->H;
  a->Hkv = p->Hkv;
  a->G = p->H / p->Hkv;
  a->page_size = p->page_size;
  a->page_shift = p->page_size == 16 ? 4 : p->page_size == 32 ? 5 : p->page_size == 64 ? 6 : 7;
  a->n_pages = p->n_pages;
  a->max_pages = p->max_pages;
  a->causal = p->causal != 0;
  a->path = L.path;
  const int sms = sm_count();
  const int w0 = paged_decode_workers(sms);
  a->W_max[0] = w0 < kMaxWorkers ? w0 : kMaxWorkers;
  a->W_max[1] = sms < kMaxChunkWorkers ? sms : kMaxChunkWorkers;
  // which requests the decode kernel takes: all of a call with few rows each;
  // in a call with chunks those of up to 8 rows (16 where a token alone has more than 8)
  a->small_rows = L.path == kPathDecode8 ? 8 : L.path == kPathDecode16 ? 16 : L.path == kPathDecode32 ? 32
                  : a->G <= 8 ? 8 : a->G <= 16 ? 16 : 0;
  a->half_toks = kChunkRows / 2 / a->G;
  {
    // tiles of a head, of one request and of all, times the longest there can be
    const double keys = (double)p->max_pages * p->page_size, half = a->half_toks;
    const double chunk_tile = keys / kChunkBlk + kChunkTileCost + 1, decode_tile = keys / kDecodeBlk + kDecodeTileCost + 1;
    a->count_places = (a->max_q / (2 * half) + 1) * chunk_tile > (double)kMaxHeadPlaces ||
                      (p->T / (2 * half) + p->n_req) * chunk_tile * p->Hkv > (double)kMaxPlaces ||
                      p->n_req * decode_tile * p->Hkv > (double)kMaxPlaces;
  }
  const float scale = p->softmax_scale > 0.f ? p->softmax_scale : 1.0f / std::sqrt((float)p->d);
  a->c_log2 = scale * 1.44269504088896341f;
  // what the plan's records depend on (FNV-1a)
  uint64_t sig = 0xcbf29ce484222325ull;
  for (int x : {p->n_req, p->T, a->max_q, p->H, p->Hkv, p->d, p->page_size, p->n_pages, p->max_pages, a->causal, a->path,
                a->W_max[0], a->W_max[1]})
    sig = (sig ^ (uint32_t)x) * 0x100000001b3ull;
  a->signature = sig;
  a->cu_q = p->cu_q;
  a->kv_len = p->kv_len;
  a->block_table = p->block_table;
  a->q_stride = p->q_stride ? p->q_stride : (int64_t)p->H * p->d;
  a->kv_stride = p->kv_stride ? p->kv_stride : (int64_t)p->Hkv * p->d;
  uint8_t* b = static_cast<uint8_t*>(ws);
  a->hdr = reinterpret_cast<PagedHeader*>(b + L.header);
  a->reqs = reinterpret_cast<ReqRec*>(b + L.reqs);
  a->workers = reinterpret_cast<WorkerRec*>(b + L.workers);
  a->part_ml = reinterpret_cast<float2*>(b + L.part_ml);
  a->part_o = reinterpret_cast<float*>(b + L.part_o);
  a->chunk_ml = reinterpret_cast<float2*>(b + L.chunk_ml);
  a->chunk_o = reinterpret_cast<float*>(b + L.chunk_o);
  return FLAMIA_OK;
}

int cache_of(const flamia_paged_t* p) {
  return p->cache_dtype == FLAMIA_BF16 ? kCacheBF16 : p->cache_dtype == FLAMIA_E4M3 ? kCacheE4M3 : kCacheE2M1;
}

flamia_status_t fill_cache(const flamia_paged_t* p, const flamia_cache_t* c, PagedParams* a) {
  if (!c || !dev16(c->k) || !dev16(c->v)) return FLAMIA_ERR_INVALID_ARG;
  const int cache = cache_of(p);
  if (cache != kCacheBF16 ? !dev16(c->k_scales) || !dev16(c->v_scales) : c->k_scales || c->v_scales) return FLAMIA_ERR_INVALID_ARG;
  if (cache == kCacheE2M1 && (!dev16(c->k_blocks) || !dev16(c->v_blocks))) return FLAMIA_ERR_INVALID_ARG;
  const int64_t page = (int64_t)p->Hkv * p->page_size * p->d, per_16 = cache == kCacheBF16 ? 8 : cache == kCacheE4M3 ? 16 : 32;
  if (c->page_stride && (c->page_stride < page || c->page_stride % per_16)) return FLAMIA_ERR_INVALID_ARG;
  a->page_bytes = (c->page_stride ? c->page_stride : page) / per_16 * 16;
  a->k = static_cast<uint8_t*>(c->k);
  a->v = static_cast<uint8_t*>(c->v);
  a->k_scales = static_cast<uint8_t*>(c->k_scales);
  a->v_scales = static_cast<uint8_t*>(c->v_scales);
  if (cache == kCacheE2M1) {
    a->k_blocks = static_cast<uint8_t*>(c->k_blocks);
    a->v_blocks = static_cast<uint8_t*>(c->v_blocks);
  }
  return FLAMIA_OK;
}

PagesLayout pages_layout(const flamia_paged_t& p) {
  PagesLayout L{};
  auto a256 = [](size_t x) { return (x + 255) & ~size_t(255); };
  const size_t table = sizeof(int32_t) * (size_t)p.n_req * p.max_pages;
  L.header = 0;
  L.pages = sizeof(PagesHeader);
  size_t o = a256(L.pages + sizeof(PageRec) * (size_t)p.n_pages);
  L.staged = o; o = a256(o + table);
  L.freed = o; o = a256(o + table);
  L.counts = o; o = a256(o + sizeof(int4) * p.n_req);
  L.total = o;
  return L;
}

flamia_status_t fill_pages(const flamia_paged_t* p, void* pages_ws, size_t bytes, PagesParams* a) {
  flamia_status_t s = validate(p);
  if (s != FLAMIA_OK) return s;
  const PagesLayout L = pages_layout(*p);
  if (!dev16(pages_ws)) return FLAMIA_ERR_INVALID_ARG;
  if (bytes < L.total) return FLAMIA_ERR_WORKSPACE_TOO_SMALL;
  *a = PagesParams{};
  a->n_req = p->n_req;
  a->T = p->T;
  a->max_q = max_q_of(p);
  a->page_size = p->page_size;
  a->page_shift = p->page_size == 16 ? 4 : p->page_size == 32 ? 5 : p->page_size == 64 ? 6 : 7;
  a->n_pages = p->n_pages;
  a->max_pages = p->max_pages;
  a->cu_q = p->cu_q;
  a->kv_len = p->kv_len;
  a->block_table = p->block_table;
  uint8_t* b = static_cast<uint8_t*>(pages_ws);
  a->hdr = reinterpret_cast<PagesHeader*>(b + L.header);
  a->pages = reinterpret_cast<PageRec*>(b + L.pages);
  a->staged = reinterpret_cast<int32_t*>(b + L.staged);
  a->freed = reinterpret_cast<int32_t*>(b + L.freed);
  a->counts = reinterpret_cast<int4*>(b + L.counts);
  a->bits = reinterpret_cast<uint32_t*>(b + L.pages);
  a->rank = reinterpret_cast<int32_t*>(b + L.pages + 4 * (size_t)p->n_pages);
  return FLAMIA_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }
  return fn;
}

// bf16 map, 128B swizzle, out-of-range elements read as zero.
template <int N>
bool bf16_map(CUtensorMap* m, const void* ptr, const cuuint64_t (&dims)[N], const cuuint64_t (&strides)[N - 1],
              const cuuint32_t (&box)[N]) {
  auto fn = encode_fn();
  cuuint32_t estr[N];
  for (auto& e : estr) e = 1;
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, N, const_cast<void*>(ptr), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Over the queries [T][H][d]: box = half a tile's tokens x the heads of one
// key/value head x 64 channels (128 bytes).
bool make_q_map(CUtensorMap* m, const PagedParams& a, int d) {
  return bf16_map<3>(m, a.q, {(cuuint64_t)d, (cuuint64_t)a.H, (cuuint64_t)a.T}, {(cuuint64_t)d * 2, (cuuint64_t)a.q_stride * 2},
                     {64, (cuuint32_t)a.G, (cuuint32_t)a.half_toks});
}
// Over bf16 pages [n_pages][Hkv][page_size][d]: box = one page and head, 64 channels.
bool make_pages_map(CUtensorMap* m, const void* ptr, const PagedParams& a, int d) {
  return bf16_map<4>(m, ptr, {(cuuint64_t)d, (cuuint64_t)a.page_size, (cuuint64_t)a.Hkv, (cuuint64_t)a.n_pages},
                     {(cuuint64_t)d * 2, (cuuint64_t)a.page_size * d * 2, (cuuint64_t)a.page_bytes},
                     {64, (cuuint32_t)a.page_size, 1, 1});
}

flamia_status_t of(cudaError_t e) { return e == cudaSuccess ? FLAMIA_OK : FLAMIA_ERR_CUDA; }

}  // namespace

extern "C" {

size_t flamia_paged_workspace_size(const flamia_paged_t* p) { return validate(p) == FLAMIA_OK ? layout(*p).total : 0; }

flamia_status_t flamia_paged_plan(const flamia_paged_t* p, int32_t* slot_map, const int32_t* old_len, int32_t* free_pages,
                                  const int32_t* n_free, int32_t* n_free_out, void* ws, size_t ws_bytes,
                                  cudaStream_t stream) {
  PagedParams a;
  flamia_status_t s = fill(p, ws, ws_bytes, &a);
  if (s != FLAMIA_OK) return s;
  const bool manage = old_len || free_pages || n_free || n_free_out;
  if (manage && (!dev4(old_len) || !dev4(free_pages) || !dev4(n_free) || !dev4(n_free_out))) return FLAMIA_ERR_INVALID_ARG;
  if (!aligned(slot_map, 4)) return FLAMIA_ERR_INVALID_ARG;
  a.slot_map = slot_map;
  a.old_len = old_len;
  a.free_pages = free_pages;
  a.n_free = n_free;
  // every CTA of the launch reads *n_free: a result for the same word goes
  // through the workspace
  const bool same = manage && n_free == n_free_out;
  a.n_free_out = same ? &a.hdr->n_free_new : n_free_out;
  cudaError_t e = launch_paged_plan(a, stream);
  if (e == cudaSuccess && same) e = cudaMemcpyAsync(n_free_out, a.n_free_out, sizeof(int32_t), cudaMemcpyDeviceToDevice, stream);
  return of(e);
}

size_t flamia_paged_pages_workspace_size(const flamia_paged_t* p) {
  return validate(p) == FLAMIA_OK ? pages_layout(*p).total : 0;
}

flamia_status_t flamia_paged_plan_shared(const flamia_paged_t* p, int32_t* slot_map, const int32_t* src,
                                         const int32_t* old_len, int32_t* refs, int32_t* free_pages, const int32_t* n_free,
                                         int32_t* n_free_out, int32_t* copies, int32_t* n_copies, void* pages_ws,
                                         size_t pages_ws_bytes, void* ws, size_t ws_bytes, cudaStream_t stream) {
  PagedParams a;
  PagesParams b;
  flamia_status_t s = fill(p, ws, ws_bytes, &a);
  if (s != FLAMIA_OK) return s;
  if ((s = fill_pages(p, pages_ws, pages_ws_bytes, &b)) != FLAMIA_OK) return s;
  if (a.count_places) return FLAMIA_ERR_UNSUPPORTED;  // the plan could refuse the step once its pages have moved
  if (!dev4(old_len) || !dev4(refs) || !dev4(free_pages) || !dev4(n_free) || !dev4(n_free_out) || !dev4(copies) ||
      !dev4(n_copies) || !aligned(src, 4) || !aligned(slot_map, 4))
    return FLAMIA_ERR_INVALID_ARG;
  b.src = src;
  b.old_len = old_len;
  b.refs = refs;
  b.free_pages = free_pages;
  b.n_free = n_free;
  b.n_free_out = n_free_out;
  b.copies = copies;
  b.n_copies = n_copies;
  b.dbg_withhold = debug_withhold() ? kShareBarriers : 0;
  a.slot_map = slot_map;
  a.before = &b.hdr->fail;
  const cudaError_t e = launch_paged_share(b, sm_count(), stream);
  return of(e != cudaSuccess ? e : launch_paged_plan(a, stream));
}

flamia_status_t flamia_paged_compact(const flamia_paged_t* p, const int32_t* len, int32_t* refs, int32_t* free_pages,
                                     const int32_t* n_free, int32_t* copies, int32_t* n_copies, void* pages_ws,
                                     size_t pages_ws_bytes, cudaStream_t stream) {
  PagesParams b;
  flamia_status_t s = fill_pages(p, pages_ws, pages_ws_bytes, &b);
  if (s != FLAMIA_OK) return s;
  if (!dev4(len) || !aligned(refs, 4) || !dev4(free_pages) || !dev4(n_free) || !copies || !aligned(copies, 8) || !dev4(n_copies))
    return FLAMIA_ERR_INVALID_ARG;
  b.old_len = len;
  b.refs = refs;
  b.free_pages = free_pages;
  b.n_free = n_free;
  b.copies = copies;
  b.n_copies = n_copies;
  b.dbg_withhold = debug_withhold() ? kCompactBarriers : 0;
  return of(launch_paged_compact(b, sm_count(), stream));
}

flamia_status_t flamia_paged_copy(const flamia_paged_t* p, int32_t n_layers, const flamia_cache_t* src,
                                  const flamia_cache_t* dst, const int32_t* copies, int32_t max_copies,
                                  const int32_t* n_copies, void* pages_ws, size_t pages_ws_bytes, cudaStream_t stream) {
  PagesParams b;
  flamia_status_t s = fill_pages(p, pages_ws, pages_ws_bytes, &b);
  if (s != FLAMIA_OK) return s;
  if (n_layers < 1 || !src || !dst || !dev4(copies) || max_copies < 0 || !dev4(n_copies)) return FLAMIA_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n_layers; ++i) {  // all of them before the first launch
    PagedParams c;
    if ((s = fill_cache(p, src + i, &c)) != FLAMIA_OK || (s = fill_cache(p, dst + i, &c)) != FLAMIA_OK) return s;
  }
  const int kind = cache_of(p);
  const int64_t rows = (int64_t)p->Hkv * p->page_size, kv = rows * p->d;
  if (kv / 8 > (1 << 28)) return FLAMIA_ERR_UNSUPPORTED;  // 16-byte pieces of a page count in 32 bits
  for (int32_t l0 = 0; l0 < n_layers; l0 += kCopyLayers) {
    CopyParams a{};
    a.layers = n_layers - l0 < kCopyLayers ? n_layers - l0 : kCopyLayers;
    for (int i = 0; i < a.layers; ++i) {
      PagedParams from{}, to{};
      fill_cache(p, src + l0 + i, &from);
      fill_cache(p, dst + l0 + i, &to);
      CopyLayer& c = a.layer[i];
      const uint8_t* f[6] = {from.k, from.v, from.k_scales, from.v_scales, from.k_blocks, from.v_blocks};
      uint8_t* t[6] = {to.k, to.v, to.k_scales, to.v_scales, to.k_blocks, to.v_blocks};
      for (int j = 0; j < 6; ++j) {
        c.src[j] = f[j];
        c.dst[j] = t[j];
      }
      a.src_stride[i] = from.page_bytes;
      a.dst_stride[i] = to.page_bytes;
    }
    a.n_pages = p->n_pages;
    a.kv_vecs = (int)(kv / (kind == kCacheBF16 ? 8 : kind == kCacheE4M3 ? 16 : 32));
    a.scale_vecs = kind == kCacheBF16 ? 0 : (int)(rows / 16);
    a.block_vecs = kind == kCacheE2M1 ? (int)(kv / 256) : 0;
    a.copies = copies;
    a.n_copies = n_copies;
    a.max_copies = max_copies;
    a.hdr = b.hdr;
    const cudaError_t e = launch_paged_copy(a, sm_count(), stream);
    if (e != cudaSuccess) return of(e);
  }
  return FLAMIA_OK;
}

flamia_status_t flamia_paged_append(const flamia_paged_t* p, const void* k, const void* v, const int32_t* slot_map,
                                    const flamia_cache_t* cache, void* ws, size_t ws_bytes, cudaStream_t stream) {
  PagedParams a;
  flamia_status_t s = fill(p, ws, ws_bytes, &a);
  if (s != FLAMIA_OK) return s;
  if ((s = fill_cache(p, cache, &a)) != FLAMIA_OK) return s;
  if (!dev16(k) || !dev16(v) || !dev4(slot_map)) return FLAMIA_ERR_INVALID_ARG;
  a.k_new = k;
  a.v_new = v;
  a.slots = slot_map;
  return of(launch_paged_append(a, p->d, cache_of(p), p->in_dtype == FLAMIA_BF16, sm_count(), stream));
}

flamia_status_t flamia_paged_fwd(const flamia_paged_t* p, const void* q, const flamia_cache_t* cache, void* O, float* lse,
                                 void* ws, size_t ws_bytes, cudaStream_t stream) {
  PagedParams a;
  flamia_status_t s = fill(p, ws, ws_bytes, &a);
  if (s != FLAMIA_OK) return s;
  if ((s = fill_cache(p, cache, &a)) != FLAMIA_OK) return s;
  if (!dev16(q) || !dev16(O) || !aligned(lse, 4)) return FLAMIA_ERR_INVALID_ARG;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.O = static_cast<__nv_bfloat16*>(O);
  a.lse = lse;
  const int kind = cache_of(p);
  if (a.small_rows) {
    const cudaError_t e = kind == kCacheE2M1 ? launch_paged_decode4(a, p->d, stream) : launch_paged_decode(a, p->d, kind, stream);
    if (e != cudaSuccess || a.path != kPathChunk) return of(e);
  }
  CUtensorMap mq{}, mk{}, mv{};
  if (!make_q_map(&mq, a, p->d) || (kind == kCacheBF16 && (!make_pages_map(&mk, a.k, a, p->d) || !make_pages_map(&mv, a.v, a, p->d))))
    return FLAMIA_ERR_CUDA;
  return of(launch_paged_chunk(a, p->d, kind, mq, mk, mv, stream));
}

}  // extern "C"
