// paged_append.cu — a step's K and V rows into their cache slots.
//
// A row (token, key/value head) is read by a group of lanes, 16 bytes a lane,
// and written as one contiguous run of its page: rounded to bf16, as E4M3
// codes with the row's own no-clamp exponent, whose maximum the group forms by
// shuffles, or as E2M1 codes with an E4M3 scale for each 16 channels under the
// row's exponent (32 bytes a lane).  Every byte is read and written once; HBM
// bound at large sizes, a launch's latency at small ones: 46 us for 46,806
// tokens of 8 heads x 128 from bf16 to E4M3 (289 MB, 6.3 TB/s), 2.6 us for 65;
// to E2M1 35 us for 40,900 tokens (221 MB, 6.4 TB/s; from fp32 5.8), 17 us for
// 17,900 (5.6), 4.6 us for 67, and there the instructions count almost as much
// (71% of the issue slots; with a division an element and 16 bytes a lane it
// took 73 us for 40,900).  A CTA takes a few consecutive tokens and
// heads at a time, so that what it reads is contiguous (tokens of all heads)
// and so is what it writes (a head's tokens: with a token's rows in a row
// instead, the stores came in 128-byte pieces and the same call took 83 us); a
// thread keeps kHeads rows in flight.
#include "paged.cuh"

namespace flamia {

namespace {

constexpr int kThreads = 256, kHeads = 4;

// The smallest integer e with amax <= 2688 2^e (2688 = 6 * 448 = 1.3125 * 2^11, the
// largest E2M1 value times the largest block scale), at least -127; 0 for 0.
__device__ __forceinline__ int e2m1_row_exp(float amax) {
  const uint32_t b = __float_as_uint(amax);
  // a mantissa above that of 1.3125 (0x280000) carries into the exponent
  const int e = max(-127, (int)((b + 0x57FFFFu) >> 23) - 138);
  return b == 0u ? 0 : e;
}
// The smallest E4M3 value s with 6 s >= bm (0 <= bm <= 2688), as its code; 6 s is
// exact in fp32.  Up from a little above bm / 6 to three bits behind the first,
// and one back where that was too far; with subnormal values, from the nearest.
__device__ __forceinline__ uint32_t e2m1_block_scale(float bm, float& s) {
  if (bm >= 0.095f) {  // 6 * 2^-6 and a little
    uint32_t b = (__float_as_uint(bm * 0.16666675f) + 0xFFFFFu) & 0xFFF00000u;  // (1 + 2^-21) / 6
    if (6.f * __uint_as_float(b - 0x100000u) >= bm) b -= 0x100000u;
    s = __uint_as_float(b);
    return (b >> 20) - (120u << 3);
  }
  uint32_t c = pack_e4m3x2(bm * (1.f / 6.f), 0.f) & 0xFFu;
  s = unpack_e4m3x2((uint16_t)c).x;
  if (6.f * s < bm) s = unpack_e4m3x2((uint16_t)++c).x;
  return c;
}
// The E2M1 codes of a lane's elements f times inv over their block scale s: those
// of the exact quotients.  A border between two codes has at most 3 significant
// bits and the scale 4, so an element on a border has at most 7.
// bf16 (8 elements): times a reciprocal, which is off by less than 2^-21, and
// rounded to multiples of 2^-11 by adding 4096.  An 8-bit element that is not on
// a border lies at least 2^-8 of it, so 2^-10, away: the rounding puts the
// others on it and moves none over it.
// fp32 (4 elements): the correctly rounded quotient, which reaches no border that
// the exact one misses; from the correctly rounded reciprocal by one step on the
// quotient's remainder (Markstein, Computation of elementary functions on the IBM
// RISC System/6000 processor, 1990).
template <bool BF16>
__device__ __forceinline__ float e2m1_reciprocal(float s) {
  float r;
  if constexpr (BF16) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  else r = __frcp_rn(s);
  return s == 0.f ? 0.f : r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t e2m1_codes(const float* f, float inv, float s, float r) {
  uint32_t c;
  if constexpr (BF16) {
    const uint64_t inv2 = f2_pack(inv, inv), r2 = f2_pack(r, r), up = f2_pack(4096.f, 4096.f), down = f2_pack(-4096.f, -4096.f);
    float q[8];
#pragma unroll
    for (int k = 0; k < 8; k += 2) f2_unpack(f2_add(f2_fma(f2_mul(f2_pack(f[k], f[k + 1]), inv2), r2, up), down), q[k], q[k + 1]);
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(c) : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  } else {
    const uint64_t r2 = f2_pack(r, r), s2 = f2_pack(-s, -s), inv2 = f2_pack(inv, inv);
    float q[4];
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      const uint64_t y = f2_mul(f2_pack(f[k], f[k + 1]), inv2), q0 = f2_mul(y, r2);
      f2_unpack(f2_fma(f2_fma(q0, s2, y), r2, q0), q[k], q[k + 1]);
    }
    uint16_t h;
    asm("{\n\t.reg .b8 a, b;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "mov.b16 %0, {a, b};\n\t}"
        : "=h"(h) : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]));
    c = h;
  }
  return c;
}

// How a tile's rows are dealt.  E2M1: 32 bytes of a row a lane, so that a bf16
// lane has a block of 16 channels to itself and what is done once a lane and
// row (exponents, scales, addresses) counts half (18,000 tokens 24 -> 17 us).
template <int D, int CACHE, bool BF16>
struct AppendTile {
  static constexpr int kVec = CACHE == kCacheE2M1 ? 2 : 1;  // 16-byte loads of a lane
  static constexpr int kEl = kVec * (BF16 ? 8 : 4);         // elements a lane holds
  static constexpr int kLanes = D / kEl;                    // lanes of a row (4 to 32)
  static constexpr int kToks = kThreads / kLanes;           // tokens of a tile
};

template <int D, int CACHE, bool BF16>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const PagedParams p, int tiles, int head_groups) {
  constexpr bool E4M3 = CACHE == kCacheE4M3, E2M1 = CACHE == kCacheE2M1;
  using Tile = AppendTile<D, CACHE, BF16>;
  constexpr int kVec = Tile::kVec, kEl = Tile::kEl, kLanes = Tile::kLanes, kToks = Tile::kToks;
  [[maybe_unused]] constexpr int kBlkLanes = kEl >= 16 ? 1 : 16 / kEl;  // lanes of 16 channels
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
    uint4 x[kHeads][kVec];
    const uint8_t* src = static_cast<const uint8_t*>(is_v ? p.v_new : p.k_new) +
                         ((int64_t)t * p.kv_stride + (int64_t)h0 * D + sub * kEl) * (BF16 ? 2 : 4);
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
#pragma unroll
      for (int k = 0; k < kVec; ++k) {
        x[u][k] = make_uint4(0, 0, 0, 0);
        if (in && h0 + u < p.Hkv) x[u][k] = __ldg(reinterpret_cast<const uint4*>(src + u * D * (BF16 ? 2 : 4)) + k);
      }
    }
    if (t >= rows) slot = -1;  // behind the last request
    if (slot >= n_slots || slot < -1) {
      report(&p.hdr->base, FLAMIA_ERR_BAD_PAGE, 0x711);
      slot = -1;
    }
    const int64_t page = slot >> p.page_shift;
    const int at = (int)(slot & (p.page_size - 1));
    uint8_t* pool = (is_v ? p.v : p.k) + page * p.page_bytes;
    // E2M1: this lane's places in the row of head h0; a head further is a page's length on
    [[maybe_unused]] const int64_t row0 = E2M1 ? page * p.Hkv * p.page_size + (int64_t)h0 * p.page_size + at : 0;
    [[maybe_unused]] uint8_t* codes4 = pool + ((int64_t)h0 * p.page_size + at) * (D / 2) + sub * (kEl / 2);
    [[maybe_unused]] uint8_t* blocks4 = (is_v ? p.v_blocks : p.k_blocks) + row0 * (D / 16) + sub / kBlkLanes;
    [[maybe_unused]] uint8_t* scales4 = (is_v ? p.v_scales : p.k_scales) + row0;
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
      const bool write = slot >= 0 && h0 + u < p.Hkv;
      const int64_t in_page = (int64_t)(h0 + u) * p.page_size + at;
      uint32_t w[4 * kVec];
#pragma unroll
      for (int k = 0; k < kVec; ++k) w[4 * k] = x[u][k].x, w[4 * k + 1] = x[u][k].y, w[4 * k + 2] = x[u][k].z, w[4 * k + 3] = x[u][k].w;
      float f[kEl];
#pragma unroll
      for (int e = 0; e < kEl; ++e)
        f[e] = BF16 ? __uint_as_float((e & 1) ? (w[e / 2] & 0xFFFF0000u) : (w[e / 2] << 16)) : __uint_as_float(w[BF16 ? 0 : e]);
      if constexpr (E4M3 || E2M1) {
        // The row's largest magnitude: magnitudes order like their bits,
        // infinities and NaN last.  bf16 in pairs, until the end.
        uint32_t top = w[0] & (BF16 ? 0x7FFF7FFFu : 0x7FFFFFFFu);
#pragma unroll
        for (int k = 1; k < 4 * kVec; ++k)
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
        const float inv = E2M1 ? exp2i(-e) : exp2i(max(-e, -126));  // 2^-e; e = 127 does not occur (E2M1: nor does 118)
        if constexpr (E2M1) {
          float s;
          // (a block so far below its row that the product underflows still has the smallest scale)
          const float bm = __uint_as_float(top_blk);
          uint32_t blk = e2m1_block_scale(fmaxf(bm * inv, fminf(bm, 1.17549435e-38f)), s);
          const float r = e2m1_reciprocal<BF16>(s);
          uint32_t c0 = e2m1_codes<BF16>(f, inv, s, r), c1 = e2m1_codes<BF16>(f + kEl / 2, inv, s, r);
          if (!finite) blk = c0 = c1 = 0u;
          if (write) {
            if constexpr (BF16) *reinterpret_cast<uint2*>(codes4) = make_uint2(c0, c1);
            else *reinterpret_cast<uint32_t*>(codes4) = c0 | c1 << 16;
            if (sub % kBlkLanes == 0) *blocks4 = (uint8_t)blk;
            if (sub == 0) *scales4 = (uint8_t)(finite ? e + 127 : 255);
          }
          codes4 += p.page_size * (D / 2);
          blocks4 += p.page_size * (D / 16);
          scales4 += p.page_size;
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
        if constexpr (BF16) *reinterpret_cast<uint4*>(dst) = x[u][0];
        else *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
      }
    }
  }
}

template <int D, int CACHE, bool BF16>
cudaError_t launch(const PagedParams& p, int sms, cudaStream_t st) {
  constexpr int kToks = AppendTile<D, CACHE, BF16>::kToks;
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
