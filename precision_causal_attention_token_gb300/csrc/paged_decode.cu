// paged_decode.cu — attention of few query rows over a paged cache: one token
// per request, or a few drafted ones (up to 16 rows of a key/value head).
//
// Every cached byte is used by all rows of its head at once and needed once,
// so the kernel is bound by HBM and its work is to keep loads in flight.  A
// warp takes its own chunks of 4 KB of K and of V and runs them with no
// barrier: fragments go from global memory straight to registers, 16 bytes a
// lane, in whole 64- and 128-byte segments.  The products are m16n8k16 MMAs
// in which the keys (S^T = K Q^T) and then the channels (O^T = V^T P^T) fill
// the 16 rows and the query rows the 8 columns, so few rows waste little; a
// dot product may take its channels in any order, so lane (g, t) simply holds
// 16 contiguous bytes of key g, and V^T's channels are dealt the same way.
// P^T leaves the first product with keys in rows and is turned for the second
// by movmatrix.  The weights enter as two bf16 terms (hi + lo: 16 bits), which
// is free here and leaves the output's own rounding as the only one that
// counts.  The next chunk's K is requested as soon as this one's scores are
// formed, its V as soon as P V is: about 6 KB in flight per warp.
//
// E4M3: K's codes become f16 (exact) and the queries f16 with a power-of-two
// row scale (bf16's 8 significant bits fit; the scale puts the row's largest
// element at 2^13, so what f16 cannot hold lies 2^-37 below it); the key's
// scale multiplies its scores.  V's codes become bf16 (exact), the key's
// scale multiplies its weights, whose range bf16 keeps.
//
// The softmax reference of a column moves only when a score passes it by 2^8,
// so most chunks need no shuffles; sums and accumulators are fp32.
#include <climits>

#include "paged.cuh"

namespace flamia {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
// CTAs of an SM: 4 x 128 threads x 128 registers fill its register file
// (16 rows: 168 registers, 3 CTAs).
constexpr int ctas_of(int nt) { return nt == 1 ? 4 : 3; }

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8x8 of 16-bit values across the warp: lane (g, t) holds row g, columns 2t, 2t + 1.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
// Cache bytes are read once: past L1.
__device__ __forceinline__ uint4 ld16(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld8(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

template <int D, bool FP8, int NT>
struct Decode {
  static constexpr int kRowB = D * (FP8 ? 1 : 2);   // bytes of a cached row
  static constexpr int kChunk = 4096 / kRowB;       // keys a warp takes at a time
  static constexpr int kSub = kChunk / 16;          // m16 key tiles of a chunk
  static constexpr int kKJ = kRowB / 64;            // 16-byte loads of a K row, 4 lanes side by side
  static constexpr int kVW = kRowB / 32;            // 32-bit words of a V row per lane, 8 lanes side by side
  static constexpr int kMT = D / 16;                // m16 channel tiles
  static constexpr int kQ = 8 * NT;                 // query rows
};

template <int D, bool FP8, int NT>
struct DecodeSmem {
  float o[kWarps][8 * NT][D + 4];
  float m[kWarps][8 * NT], l[kWarps][8 * NT];
  int last;
};

template <int D, bool FP8, int NT>
__global__ void __launch_bounds__(kThreads, ctas_of(NT)) paged_decode_kernel(const PagedParams p) {
  using C = Decode<D, FP8, NT>;
  __shared__ DecodeSmem<D, FP8, NT> sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  PagedHeader* hdr = p.hdr;
  if (!hdr->ok) return;
  const int W = hdr->workers, w = blockIdx.x;
  if (w >= W) return;
  const int64_t cost = hdr->cost;
  const WorkerRec rec = p.workers[w];
  int left = rec.n, r = rec.r, h = rec.h, blk = rec.blk;

  while (left > 0) {
    const ReqRec rq = p.reqs[r];
    if (rq.per_head == 0) {  // no new tokens
      ++r;
      continue;
    }
    const int nb = min(left, rq.per_head - blk);
    const int kbeg = blk * kDecodeBlk, kend = min(rq.kv_len, (blk + nb) * kDecodeBlk);
    const int rows = rq.q_len * p.G;
    // ------------------------------------------------ queries (B operand) and column limits
    uint32_t qf[NT][D / 16][2];
    float cq[NT][2];  // score factor of columns 2t, 2t + 1
    int vis[NT][2];   // keys that they see
    int vis_min = kend;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = 8 * nt + g;
      const int tok = row / p.G, hq = h * p.G + (row - tok * p.G);
      const __nv_bfloat16* src = p.q + (int64_t)(rq.q0 + tok) * p.q_stride + (int64_t)hq * D;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        // K step ks of lane t: channels d .. d + 3, as the K loads deal them
        const int d = FP8 ? (ks >> 2) * 64 + t * 16 + (ks & 3) * 4 : (ks >> 1) * 32 + t * 8 + (ks & 1) * 4;
        uint2 x = make_uint2(0, 0);
        if (row < rows) x = __ldg(reinterpret_cast<const uint2*>(src + d));
        qf[nt][ks][0] = x.x;
        qf[nt][ks][1] = x.y;
      }
      float scale = p.c_log2;  // of row g
      if constexpr (FP8) {
        uint32_t top = 0;  // largest magnitude's bits
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            top = max(top, max(qf[nt][ks][i] & 0x7FFFu, (qf[nt][ks][i] >> 16) & 0x7FFFu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // exponent field E: the row's largest element is below 2^(E - 126);
        // times 2^(139 - E) it is below 2^13 (E clamped: the factor and its inverse stay normal)
        const int E = min(max((int)(top >> 7), 13), 254);
        const float up = exp2i(139 - E);
        scale *= exp2i(E - 139);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const __half2 v = __floats2half2_rn(bf16_lo(qf[nt][ks][i]) * up, bf16_hi(qf[nt][ks][i]) * up);
            qf[nt][ks][i] = *reinterpret_cast<const uint32_t*>(&v);
          }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        cq[nt][e] = __shfl_sync(0xffffffffu, scale, 4 * (2 * t + e));
        const int c = 8 * nt + 2 * t + e;
        const int n = visible_keys(p.causal, rq.q_len, rq.kv_len, c / p.G);
        vis[nt][e] = c < rows ? n : kend;  // columns past the rows hold zeros
        vis_min = min(vis_min, vis[nt][e]);
      }
    }
    vis_min = __reduce_min_sync(0xffffffffu, vis_min);

    // ------------------------------------------------ this warp's chunks
    const int n_it = (kend - kbeg - warp * C::kChunk + kWarps * C::kChunk - 1) / (kWarps * C::kChunk);
    const int32_t* table = p.block_table + (int64_t)r * p.max_pages;
    auto key_of = [&](int it) { return kbeg + (it * kWarps + warp) * C::kChunk; };
    // page ids: lane i of a group holds the page of key tile i % kSub of chunk it0 + i / kSub
    constexpr int kGroup = 32 / C::kSub;
    auto page_group = [&](int it0) {
      const int key = key_of(it0 + lane / C::kSub) + 16 * (lane % C::kSub);
      int id = key < kend ? __ldg(table + (key >> p.page_shift)) : 0;
      if ((unsigned)id >= (unsigned)p.n_pages) {
        report(&hdr->base, FLAMIA_ERR_BAD_PAGE, 0x721);
        id = 0;
      }
      return id;
    };
    uint32_t kr[C::kSub][2][C::kKJ][4];
    uint32_t vr[C::kSub][4][C::kVW];
    uint32_t sc_k = 0, sc_v = 0;  // scale bytes: lane i (< 16) K's of key i, lane 16 + i V's, a byte per key tile
    auto load_k = [&](int it, int pg) {
      const int key0 = key_of(it);
#pragma unroll
      for (int s = 0; s < C::kSub; ++s) {
        const int id = __shfl_sync(0xffffffffu, pg, (it % kGroup) * C::kSub + s);
        const int key = key0 + 16 * s;
        const int64_t in_page = (int64_t)h * p.page_size + (key & (p.page_size - 1));
        const uint8_t* base = p.k + id * p.page_bytes + in_page * C::kRowB + t * 16;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const bool in = key + 8 * half + g < kend;
#pragma unroll
          for (int j = 0; j < C::kKJ; ++j) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (in) x = ld16(base + (8 * half + g) * C::kRowB + 64 * j);
            kr[s][half][j][0] = x.x;
            kr[s][half][j][1] = x.y;
            kr[s][half][j][2] = x.z;
            kr[s][half][j][3] = x.w;
          }
        }
        if constexpr (FP8) {
          const int64_t at = (int64_t)id * p.Hkv * p.page_size + in_page + (lane & 15);
          uint32_t b = 127;
          if (key + (lane & 15) < kend) b = __ldg((lane < 16 ? p.k_scales : p.v_scales) + at);
          sc_k = s ? sc_k | (b << (8 * s)) : b;
        }
      }
    };
    auto load_v = [&](int it, int pg) {
      const int key0 = key_of(it);
#pragma unroll
      for (int s = 0; s < C::kSub; ++s) {
        const int id = __shfl_sync(0xffffffffu, pg, (it % kGroup) * C::kSub + s);
        const int key = key0 + 16 * s;
        const int64_t in_page = (int64_t)h * p.page_size + (key & (p.page_size - 1));
        const uint8_t* base = p.v + id * p.page_bytes + in_page * C::kRowB;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int kk = 2 * t + (i & 1) + 8 * (i >> 1);
          const bool in = key + kk < kend;
          if constexpr (C::kVW == 2) {
            uint2 x = make_uint2(0, 0);
            if (in) x = ld8(base + kk * C::kRowB + g * 8);
            vr[s][i][0] = x.x;
            vr[s][i][1] = x.y;
          } else {
#pragma unroll
            for (int j = 0; j < C::kVW / 4; ++j) {
              uint4 x = make_uint4(0, 0, 0, 0);
              if (in) x = ld16(base + kk * C::kRowB + 128 * j + g * 16);
              vr[s][i][4 * j] = x.x;
              vr[s][i][4 * j + 1] = x.y;
              vr[s][i][4 * j + 2] = x.z;
              vr[s][i][4 * j + 3] = x.w;
            }
          }
        }
      }
    };

    float o[C::kMT][NT][4];
    float m[NT][2], l[NT][2];
    // bf16: an infinity in V times the lower term, or times the weight 0 of a
    // row that may not see it, gives a NaN that the formula does not have.  So
    // a warp that ends with a NaN takes its keys once more, carefully.
    bool careful = false;
  again:
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < C::kMT; ++i) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
    }
    int pg = 0, pg_next = 0;
    if (n_it > 0) {
      pg = page_group(0);
      load_k(0, pg);
      load_v(0, pg);
      if (n_it > kGroup) pg_next = page_group(kGroup);
    }
    for (int it = 0; it < n_it; ++it) {
      const int key0 = key_of(it);
      // ---------------------------------------------- S^T = K Q^T
      float s[C::kSub][NT][4];
#pragma unroll
      for (int i = 0; i < C::kSub; ++i) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[i][nt][0] = s[i][nt][1] = s[i][nt][2] = s[i][nt][3] = 0.f;
#pragma unroll
        for (int j = 0; j < C::kKJ; ++j) {
          if constexpr (FP8) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const uint32_t x = kr[i][0][j][u], y = kr[i][1][j][u];
              const uint32_t a0 = e4m3x2_to_f16x2(x & 0xFFFFu), a2 = e4m3x2_to_f16x2(x >> 16);
              const uint32_t a1 = e4m3x2_to_f16x2(y & 0xFFFFu), a3 = e4m3x2_to_f16x2(y >> 16);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_f16(s[i][nt], a0, a1, a2, a3, qf[nt][4 * j + u][0], qf[nt][4 * j + u][1]);
            }
          } else {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_bf16(s[i][nt], kr[i][0][j][2 * u], kr[i][1][j][2 * u], kr[i][0][j][2 * u + 1], kr[i][1][j][2 * u + 1],
                         qf[nt][2 * j + u][0], qf[nt][2 * j + u][1]);
          }
        }
      }
      sc_v = sc_k;  // this chunk's scale bytes; load_k takes the next one's
      int pg_now = pg;
      if (it + 1 < n_it) {
        if ((it + 1) % kGroup == 0) {
          pg_now = pg_next;
          if (it + 1 + kGroup < n_it) pg_next = page_group(it + 1 + kGroup);
        }
        load_k(it + 1, pg_now);
      }
      // ---------------------------------------------- scores, reference, weights
      float top[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) top[nt][0] = top[nt][1] = -INFINITY;
#pragma unroll
      for (int i = 0; i < C::kSub; ++i) {
        float f0 = 1.f, f1 = 1.f;
        if constexpr (FP8) {
          f0 = ue8m0((__shfl_sync(0xffffffffu, sc_v, g) >> (8 * i)) & 0xFFu);
          f1 = ue8m0((__shfl_sync(0xffffffffu, sc_v, 8 + g) >> (8 * i)) & 0xFFu);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            s[i][nt][e] *= FP8 ? cq[nt][e] * f0 : cq[nt][e];
            s[i][nt][2 + e] *= FP8 ? cq[nt][e] * f1 : cq[nt][e];
          }
        }
      }
      if (key0 + C::kChunk > vis_min) {
#pragma unroll
        for (int i = 0; i < C::kSub; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int key = key0 + 16 * i + g, lim = min(vis[nt][e], kend);
              if (key >= lim) s[i][nt][e] = -INFINITY;
              if (key + 8 >= lim) s[i][nt][2 + e] = -INFINITY;
            }
      }
      bool up = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int i = 0; i < C::kSub; ++i) top[nt][e] = fmax3(top[nt][e], s[i][nt][e], s[i][nt][2 + e]);
          up |= top[nt][e] > m[nt][e] + 8.f;
        }
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = top[nt][e];
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            x = fmaxf(x, m[nt][e]);
            const float a = x == m[nt][e] ? 1.f : ex2_approx(m[nt][e] - x);  // 0 from an empty reference
            m[nt][e] = x;
            l[nt][e] *= a;
#pragma unroll
            for (int i = 0; i < C::kMT; ++i) {
              o[i][nt][e] *= a;
              o[i][nt][2 + e] *= a;
            }
          }
      }
      uint32_t hi[C::kSub][NT][2], lo[C::kSub][NT][2];  // P^T as B operand
#pragma unroll
      for (int i = 0; i < C::kSub; ++i) {
        float f[2] = {1.f, 1.f};
        if constexpr (FP8) {
          f[0] = ue8m0((__shfl_sync(0xffffffffu, sc_v, 16 + g) >> (8 * i)) & 0xFFu);
          f[1] = ue8m0((__shfl_sync(0xffffffffu, sc_v, 24 + g) >> (8 * i)) & 0xFFu);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float y[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              y[e] = ex2_approx(s[i][nt][2 * k + e] - (m[nt][e] == -INFINITY ? 0.f : m[nt][e]));
              l[nt][e] += y[e];
              // a NaN scale stays with the rows that see the key
              if constexpr (FP8) y[e] = s[i][nt][2 * k + e] == -INFINITY ? 0.f : y[e] * f[k];
            }
            const uint32_t a = pack_bf16x2(y[0], y[1]);
            hi[i][nt][k] = transpose8(a);
            lo[i][nt][k] = transpose8(pack_bf16x2(y[0] - bf16_lo(a), y[1] - bf16_hi(a)));
          }
      }
      // ---------------------------------------------- O^T += V^T P^T
      // tok >= 0 (careful): only the columns of token tok, over the keys that
      // it sees, and the lower terms over finite values
      auto add_pv = [&](int tok) {
        const int lim = tok < 0 ? INT_MAX : visible_keys(p.causal, rq.q_len, rq.kv_len, tok) - key0;
#pragma unroll
        for (int i = 0; i < C::kSub; ++i) {
#pragma unroll
          for (int mt = 0; mt < C::kMT; ++mt) {
            uint32_t a[4];
            if constexpr (FP8) {
              // channels 2 mt, 2 mt + 1 of the lane's run: bytes of one word
              const int wd = mt >> 1, b = 2 * (mt & 1);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t sel = (uint32_t)(b + (k & 1)) * 0x0011u + (uint32_t)(4 + b + (k & 1)) * 0x1100u;
                const uint32_t x = prmt(vr[i][(k >> 1) * 2][wd], vr[i][(k >> 1) * 2 + 1][wd], sel);
                a[k] = bf16x2_mul(e4m3_hi_to_bf16x2(x), 0x7B807B80u);
              }
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int kk = 16 * i + 2 * t + 8 * (k >> 1);
                const uint32_t x = kk < lim ? vr[i][(k >> 1) * 2][mt] : 0u, y = kk + 1 < lim ? vr[i][(k >> 1) * 2 + 1][mt] : 0u;
                a[k] = prmt(x, y, (k & 1) ? 0x7632u : 0x5410u);
              }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float c[4] = {o[mt][nt][0], o[mt][nt][1], o[mt][nt][2], o[mt][nt][3]};
              mma_bf16(c, a[0], a[1], a[2], a[3], hi[i][nt][0], hi[i][nt][1]);
              uint32_t f[4] = {a[0], a[1], a[2], a[3]};
              if (!FP8 && tok >= 0) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  if ((f[k] & 0x7F80u) == 0x7F80u) f[k] &= 0xFFFF0000u;
                  if ((f[k] & 0x7F800000u) == 0x7F800000u) f[k] &= 0xFFFFu;
                }
              }
              mma_bf16(c, f[0], f[1], f[2], f[3], lo[i][nt][0], lo[i][nt][1]);
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (tok < 0 || (8 * nt + 2 * t + e) / p.G == tok) {
                  o[mt][nt][e] = c[e];
                  o[mt][nt][2 + e] = c[2 + e];
                }
            }
          }
        }
      };
      if (FP8 || !careful) {
        add_pv(-1);
      } else {
#pragma unroll 1
        for (int tok = 0; tok < rq.q_len; ++tok) add_pv(tok);
      }
      pg = pg_now;
      if (it + 1 < n_it) load_v(it + 1, pg);
    }

    float sum = 0.f;  // NaN where one of them is, and for infinities of both signs
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < C::kMT; ++i) sum += (o[i][nt][0] + o[i][nt][1]) + (o[i][nt][2] + o[i][nt][3]);
    if (!FP8 && !careful && __any_sync(0xffffffffu, sum != sum)) {
      careful = true;
      goto again;
    }

    // ------------------------------------------------ join the warps
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[nt][e];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        const int c = 8 * nt + 2 * t + e;
        if (g == 0) {
          sm.m[warp][c] = m[nt][e];
          sm.l[warp][c] = x;
        }
#pragma unroll
        for (int i = 0; i < C::kMT; i += 2) {
          // two channel tiles: four channels in a row
          const int d = C::kVW == 8 ? (i / 4) * 64 + g * 8 + (i % 4) * 2 : (D / 8) * g + 2 * i;
          *reinterpret_cast<float4*>(&sm.o[warp][c][d]) =
              make_float4(o[i][nt][e], o[i][nt][2 + e], o[i + 1][nt][e], o[i + 1][nt][2 + e]);
        }
      }
    __syncthreads();
    const bool whole = nb == rq.per_head;
    constexpr int kSpan = kThreads / C::kQ;      // threads of a query row (16 or 8)
    constexpr int kPer = D / kSpan;              // channels of a thread
    const int row = tid / kSpan, d0 = (tid % kSpan) * kPer;
    float M = sm.m[0][row];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) M = fmaxf(M, sm.m[i][row]);
    float L = 0.f, acc[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const float a = sm.m[i][row] == M ? 1.f : ex2_approx(sm.m[i][row] - M);
      L += a * sm.l[i][row];
#pragma unroll
      for (int k = 0; k < kPer; k += 4) {
        const float4 x = *reinterpret_cast<const float4*>(&sm.o[i][row][d0 + k]);
        acc[k] += a * x.x;
        acc[k + 1] += a * x.y;
        acc[k + 2] += a * x.z;
        acc[k + 3] += a * x.w;
      }
    }
    bool write = whole;
    if (!whole) {
      const int64_t tile0 = rq.base + (int64_t)h * rq.per_head;
      const int w0 = worker_of(tile0, cost, W), n = worker_of(tile0 + rq.per_head - 1, cost, W) - w0 + 1;
      const int slot = blk == 0 ? 2 * w + 1 : 2 * w;
      float* po = p.part_o + ((int64_t)slot * C::kQ + row) * D + d0;
#pragma unroll
      for (int k = 0; k < kPer; k += 4)
        __stcg(reinterpret_cast<float4*>(po + k), make_float4(acc[k], acc[k + 1], acc[k + 2], acc[k + 3]));
      if (d0 == 0) __stcg(p.part_ml + (int64_t)slot * C::kQ + row, make_float2(M, L));
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const bool last = atomicAdd(&hdr->count[w0], 1u) == (unsigned)(n - 1);
        if (last) hdr->count[w0] = 0;
        sm.last = last;
      }
      __syncthreads();
      write = sm.last;
      if (write) {
        __threadfence();
        auto slot_of = [&](int i) { return (int64_t)(i == 0 ? 2 * w0 + 1 : 2 * (w0 + i)); };
        M = -INFINITY;
        for (int i = 0; i < n; ++i) M = fmaxf(M, __ldcg(p.part_ml + slot_of(i) * C::kQ + row).x);
        L = 0.f;
#pragma unroll
        for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
          const float2 ml = __ldcg(p.part_ml + slot_of(i) * C::kQ + row);
          const float a = ml.x == M ? 1.f : ex2_approx(ml.x - M);
          L += a * ml.y;
          const float* src = p.part_o + (slot_of(i) * C::kQ + row) * D + d0;
#pragma unroll
          for (int k = 0; k < kPer; k += 4) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(src + k));
            acc[k] += a * x.x;
            acc[k + 1] += a * x.y;
            acc[k + 2] += a * x.z;
            acc[k + 3] += a * x.w;
          }
        }
      }
    }
    if (write && row < rows) {
      const int tok = row / p.G, hq = h * p.G + (row - tok * p.G);
      const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);  // a NaN sum stays
      uint32_t out[kPer / 2];
#pragma unroll
      for (int k = 0; k < kPer; k += 2) out[k / 2] = pack_bf16x2(acc[k] * inv, acc[k + 1] * inv);
      __nv_bfloat16* dst = p.O + ((int64_t)(rq.q0 + tok) * p.H + hq) * D + d0;
      if constexpr (kPer % 8 == 0) {
#pragma unroll
        for (int k = 0; k < kPer / 8; ++k)
          *reinterpret_cast<uint4*>(dst + 8 * k) = make_uint4(out[4 * k], out[4 * k + 1], out[4 * k + 2], out[4 * k + 3]);
      } else {
        *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
      }
      if (d0 == 0 && p.lse) p.lse[(int64_t)hq * p.T + rq.q0 + tok] = (M + lg2_f(L)) * 0.69314718055994531f;
    }
    __syncthreads();  // the join buffers are free
    left -= nb;
    blk = 0;
    if (++h == p.Hkv) {
      h = 0;
      ++r;
    }
  }
}

template <int D, bool FP8, int NT>
cudaError_t launch(const PagedParams& p, cudaStream_t st) {
  paged_decode_kernel<D, FP8, NT><<<p.W_max, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}
template <int D, bool FP8>
cudaError_t launch_n(const PagedParams& p, cudaStream_t st) {
  return p.path == kPathDecode8 ? launch<D, FP8, 1>(p, st) : launch<D, FP8, 2>(p, st);
}

}  // namespace

int paged_decode_workers(int sms, int path) { return sms * ctas_of(path == kPathDecode8 ? 1 : 2); }

cudaError_t launch_paged_decode(const PagedParams& p, int d, bool e4m3, cudaStream_t st) {
  if (d == 128) return e4m3 ? launch_n<128, true>(p, st) : launch_n<128, false>(p, st);
  return e4m3 ? launch_n<64, true>(p, st) : launch_n<64, false>(p, st);
}

}  // namespace flamia
