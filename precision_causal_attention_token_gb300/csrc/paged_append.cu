// paged_append.cu — a step's K and V rows into their cache slots.
//
// A row (token, key/value head) is read by a group of lanes, 16 bytes a lane,
// and written as one contiguous run of its page: rounded to bf16, as E4M3
// codes with the row's own no-clamp exponent, whose maximum the group forms by
// shuffles, or as E2M1 codes with an E4M3 scale for each 16 channels (the
// maximum of two or four lanes) under the row's exponent.  Every byte is read and written once; HBM bound at large sizes, a
// launch's latency at small ones: 46 us for 46,806 tokens of 8 heads x 128 from
// bf16 to E4M3 (289 MB, 6.3 TB/s), 2.6 us for 65.  A CTA takes a few consecutive tokens and
// heads at a time, so that what it reads is contiguous (tokens of all heads)
// and so is what it writes (a head's tokens: with a token's rows in a row
// instead, the stores came in 128-byte pieces and the same call took 83 us); a
// thread keeps kHeads rows in flight.
#include "paged.cuh"

namespace flamia {

namespace {

constexpr int kThreads = 256, kHeads = 4;

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The smallest integer e with amax <= 2688 2^e (2688 = 6 * 448 = 1.3125 * 2^11, the
// largest E2M1 value times the largest block scale), at least -127; 0 for 0.
__device__ __forceinline__ int e2m1_row_exp(float amax) {
  const uint32_t b = __float_as_uint(amax);
  if (b == 0u) return 0;
  const int E = (int)(b >> 23);
  return E == 0 ? -127 : max(-127, (b & 0x7FFFFFu) <= 0x280000u ? E - 138 : E - 137);
}
// The smallest E4M3 value with 6 s >= bm (0 <= bm <= 2688), as its code and value.
// RNE of bm / 6 is that value or the one below; 6 s is exact in fp32.
__device__ __forceinline__ uint32_t e2m1_block_scale(float bm, float& s) {
  uint32_t c = pack_e4m3x2(bm * (1.f / 6.f), 0.f) & 0xFFu;
  s = unpack_e4m3x2((uint16_t)c).x;
  if (6.f * s < bm) s = unpack_e4m3x2((uint16_t)++c).x;
  return c;
}
// Eight of a bf16 row's elements (or four of an fp32 one's) over their block
// scale, rounded to E2M1.  The codes are those of the exact quotient.  fp32: a
// rounded quotient never reaches a border between two codes that the exact one
// misses (a border has at most 3 significant bits, the scale 4).  bf16: times
// the rounded reciprocal, and the product rounded to 16 significant bits.
// Quotients of an 8-bit by a 4-bit number lie on a border or 2^-9 of it away,
// and the product is off by less than 2^-22, so the second rounding puts the
// first kind on the border and moves no other over it.  (The division took 4
// times the instructions.)
template <bool BF16, int N>
__device__ __forceinline__ uint32_t e2m1_codes(const float (&y)[N], float s) {
  uint32_t c = 0;
  if (s == 0.f) return c;
  const float r = 1.f / s;
#pragma unroll
  for (int k = 0; k < N; k += 2) {
    float q[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if constexpr (BF16) q[e] = __uint_as_float((__float_as_uint(y[k + e] * r) + 0x80u) & 0xFFFFFF00u);
      else q[e] = __fdiv_rn(y[k + e], s);
    }
    c |= pack_e2m1x2(q[0], q[1]) << (4 * k);
  }
  return c;
}

template <int D, int CACHE, bool BF16>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const PagedParams p, int tiles, int head_groups) {
  constexpr int kEl = BF16 ? 8 : 4;         // elements a lane holds
  constexpr int kLanes = D / kEl;           // lanes of a row (8, 16 or 32)
  constexpr int kToks = kThreads / kLanes;  // tokens of a tile
  constexpr bool E4M3 = CACHE == kCacheE4M3, E2M1 = CACHE == kCacheE2M1;
  [[maybe_unused]] constexpr int kBlkLanes = 16 / kEl;  // lanes of 16 channels
  const int sub = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  if (!planned(p)) return;
  const int rows = p.hdr->rows;
  const int64_t n_slots = (int64_t)p.n_pages << p.page_shift;
  // units: (token tile, K or V, head group)
  for (int unit = blockIdx.x; unit < tiles * 2 * head_groups; unit += gridDim.x) {
    const int rest = unit / head_groups, h0 = (unit - rest * head_groups) * kHeads;
    const bool is_v = rest & 1;
    const int t = (rest >> 1) * kToks + group;
    const bool in = t < p.T;  // whole groups of lanes
    int64_t slot = in ? __ldg(p.slots + t) : -1;
    uint4 x[kHeads];
    const uint8_t* src = static_cast<const uint8_t*>(is_v ? p.v_new : p.k_new) +
                         ((int64_t)t * p.kv_stride + (int64_t)h0 * D + sub * kEl) * (BF16 ? 2 : 4);
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
      x[u] = make_uint4(0, 0, 0, 0);
      if (in && h0 + u < p.Hkv) x[u] = __ldg(reinterpret_cast<const uint4*>(src + u * D * (BF16 ? 2 : 4)));
    }
    if (t >= rows) slot = -1;  // behind the last request
    if (slot >= n_slots || slot < -1) {
      report(&p.hdr->base, FLAMIA_ERR_BAD_PAGE, 0x711);
      slot = -1;
    }
    const int64_t page = slot >> p.page_shift;
    const int at = (int)(slot & (p.page_size - 1));
    uint8_t* pool = (is_v ? p.v : p.k) + page * p.page_bytes;
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
      const bool write = slot >= 0 && h0 + u < p.Hkv;
      const int64_t in_page = (int64_t)(h0 + u) * p.page_size + at;
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      float f[kEl];
#pragma unroll
      for (int e = 0; e < kEl; ++e)
        f[e] = BF16 ? __uint_as_float((e & 1) ? (w[e / 2] & 0xFFFF0000u) : (w[e / 2] << 16)) : __uint_as_float(w[e & 3]);
      if constexpr (E4M3 || E2M1) {
        // The row's largest magnitude: magnitudes order like their bits,
        // infinities and NaN last.  bf16 in pairs, until the end.
        uint32_t top = w[0] & (BF16 ? 0x7FFF7FFFu : 0x7FFFFFFFu);
#pragma unroll
        for (int k = 1; k < 4; ++k)
          top = BF16 ? max_u16x2(top, w[k] & 0x7FFF7FFFu) : max(top, w[k] & 0x7FFFFFFFu);
        [[maybe_unused]] uint32_t top_blk = top;  // of this lane's 16 channels
#pragma unroll
        for (int s = 1; s < kLanes; s <<= 1) {
          const uint32_t o = __shfl_xor_sync(0xffffffffu, top, s);
          top = BF16 ? max_u16x2(top, o) : max(top, o);
          if (2 * s == kBlkLanes) top_blk = top;
        }
        if (BF16) {
          top = max(top & 0xFFFF0000u, top << 16);
          top_blk = max(top_blk & 0xFFFF0000u, top_blk << 16);
        }
        const bool finite = top < 0x7F800000u;
        const int e = !finite ? 0 : E2M1 ? e2m1_row_exp(__uint_as_float(top)) : noclamp_exp_clamped(__uint_as_float(top));
        const float inv = exp2i(max(-e, -126));  // 2^-e; e = 127 does not occur
        if constexpr (E2M1) {
          float y[kEl], s;
#pragma unroll
          for (int k = 0; k < kEl; k += 2) f2_unpack(f2_mul(f2_pack(f[k], f[k + 1]), f2_pack(inv, inv)), y[k], y[k + 1]);
          uint32_t blk = finite ? e2m1_block_scale(__uint_as_float(top_blk) * inv, s) : 0u;
          const uint32_t c = finite ? e2m1_codes<BF16>(y, s) : 0u;
          if (write) {
            uint8_t* dst = pool + in_page * (D / 2) + sub * (kEl / 2);
            if constexpr (kEl == 8) *reinterpret_cast<uint32_t*>(dst) = c;
            else *reinterpret_cast<uint16_t*>(dst) = (uint16_t)c;
            const int64_t row = page * p.Hkv * p.page_size + in_page;
            if (sub % kBlkLanes == 0) (is_v ? p.v_blocks : p.k_blocks)[row * (D / 16) + sub / kBlkLanes] = (uint8_t)blk;
            if (sub == 0) (is_v ? p.v_scales : p.k_scales)[row] = (uint8_t)(finite ? e + 127 : 255);
          }
        } else {
          uint32_t c[kEl / 4];
#pragma unroll
          for (int k = 0; k < kEl / 4; ++k) {
            float y[4];
            f2_unpack(f2_mul(f2_pack(f[4 * k], f[4 * k + 1]), f2_pack(inv, inv)), y[0], y[1]);
            f2_unpack(f2_mul(f2_pack(f[4 * k + 2], f[4 * k + 3]), f2_pack(inv, inv)), y[2], y[3]);
            c[k] = finite ? pack_e4m3x4(y[0], y[1], y[2], y[3]) : 0x7F7F7F7Fu;
          }
          if (write) {
            uint8_t* dst = pool + in_page * D + sub * kEl;
            if constexpr (kEl == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(c[0], c[kEl / 4 - 1]);
            else *reinterpret_cast<uint32_t*>(dst) = c[0];
            if (sub == 0)
              (is_v ? p.v_scales : p.k_scales)[page * p.Hkv * p.page_size + in_page] = (uint8_t)(finite ? e + 127 : 255);
          }
        }
      } else if (write) {
        uint8_t* dst = pool + (in_page * D + sub * kEl) * 2;
        if constexpr (BF16) *reinterpret_cast<uint4*>(dst) = x[u];
        else *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
      }
    }
  }
}

template <int D, int CACHE, bool BF16>
cudaError_t launch(const PagedParams& p, int sms, cudaStream_t st) {
  constexpr int kToks = kThreads / (D / (BF16 ? 8 : 4));
  const int tiles = (p.T + kToks - 1) / kToks, groups = (p.Hkv + kHeads - 1) / kHeads;
  const int64_t units = (int64_t)tiles * 2 * groups, most = (int64_t)sms * 16;
  if (units > (1 << 30)) return cudaErrorInvalidValue;
  paged_append_kernel<D, CACHE, BF16><<<(int)(units < most ? units : most), kThreads, 0, st>>>(p, tiles, groups);
  return cudaGetLastError();
}
template <int D>
cudaError_t launch_d(const PagedParams& p, int cache, bool bf16, int sms, cudaStream_t st) {
  if (cache == kCacheE2M1) return bf16 ? launch<D, kCacheE2M1, true>(p, sms, st) : launch<D, kCacheE2M1, false>(p, sms, st);
  if (cache == kCacheE4M3) return bf16 ? launch<D, kCacheE4M3, true>(p, sms, st) : launch<D, kCacheE4M3, false>(p, sms, st);
  return bf16 ? launch<D, kCacheBF16, true>(p, sms, st) : launch<D, kCacheBF16, false>(p, sms, st);
}

}  // namespace

cudaError_t launch_paged_append(const PagedParams& p, int d, int cache, bool in_bf16, int sms, cudaStream_t st) {
  return d == 128 ? launch_d<128>(p, cache, in_bf16, sms, st) : launch_d<64>(p, cache, in_bf16, sms, st);
}

}  // namespace flamia
