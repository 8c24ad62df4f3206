// paged_decode.cu — attention of few query rows over a paged cache: one token
// per request, or a few drafted ones (up to 32 rows of a key/value head).
//
// Every cached byte is used by all rows of its head at once and needed once,
// so the kernel is bound by HBM and its work is to keep loads in flight.  A
// warp takes its own chunks of 4 KB of K and of V and runs them with no
// block barrier: asynchronous copies in whole 512-byte pieces bring them to a
// shared-memory ring of its own, two chunks deep (12 to 16 KB in flight per
// warp and no registers held), from where the fragments are read without a
// bank conflict.  The products are
// m16n8k16 MMAs in which the keys (S^T = K Q^T) and then the channels
// (O^T = V^T P^T) fill the 16 rows and the query rows the 8 columns, so few
// rows waste little; a dot product may take its channels in any order, so lane
// (g, t) simply holds 16 contiguous bytes of key g, and V^T's channels are
// dealt the same way.  P^T leaves the first product with keys in rows and is
// turned for the second by movmatrix.
//
// bf16: the weights enter as two bf16 terms (hi + lo: 16 bits), which leaves
// the output's own rounding as the only one that counts.
// E4M3: codes become f16 (exact, one instruction for two).  The queries are
// f16 with a power-of-two row scale (bf16's 8 significant bits fit; the scale
// puts the row's largest element at 2^13, so what f16 cannot hold lies 2^-37
// below it); the key's scale, less 2^12, multiplies its scores, which so stay
// below 2^128 for keys up to 2^119 at any query.  The weights are f16
// (2^-11 relative), times 2^(e - E + 7) with e the key's V exponent and E the
// largest seen so far: at most 2^15; E's rise rescales the accumulators.  E
// counts keys that a row may not see, that have no weight in it or that hold
// zeros, and what lies far below it leaves f16's range.  So a warp whose keys'
// exponents turn out to lie more than 12 apart (a weight of 2^-9 of the
// reference still has all its bits then, and none is off by more than 2^-20 of
// it) takes its keys once more, with V as bf16 (code times scale is exact) and
// the weights as two bf16 terms (16 requests of 8,000 tokens whose warps all
// do: 57 -> 68 us at 4 rows, 85 -> 116 at 32; more where the first pass is
// nearly done when it finds out).
//
// Measured (152 SMs, H = 32, Hkv = 8, d = 128): one request of 65,522 bf16
// tokens 57 us (268 MB; 46 us at the last SM's last load, then the join), 64
// requests in E4M3 108 to 114 us (578 MB, 5.2 TB/s; the SMs' loops end between 73 and
// 105 us, the same SMs first every time), 6 short requests 7.7 us, 16 requests of 2 to 8
// drafted tokens in E4M3 62 us.  Up to 16 rows HBM bounds it; with 32 the
// latency of one warp's 1,100 instructions a chunk does, at eight warps an SM
// (two warps a chunk, 16 rows each, sixteen an SM: 71 us; the conversions double).
//
// The softmax reference of a column moves only when a score passes it by 2^8,
// so most chunks need no shuffles; sums and accumulators are fp32.
#include <climits>
#include <type_traits>

#include "paged.cuh"

namespace flamia {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kUnit = 4096;  // bytes of a chunk's K (or V)
constexpr int kSpread = 12;  // binades between V rows that f16 weights serve
constexpr int kRingB = kWarps * 4 * kUnit;  // two chunks a warp
// 2 CTAs of an SM (3: 59 against 57 us on 65,522 tokens; more partials to join)
constexpr int kCtas = 2;

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
// 16 bytes to shared memory; of them the first `n` are read, the rest is zero.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, uint32_t n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
// Four E4M3 codes -> two f16 pairs, exact.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}" : "=r"(lo), "=r"(hi) : "r"(w));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
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
  // 32 rows: the queries' fragments stay in shared memory, the registers hold
  // the 128 accumulators
  static constexpr bool kQShared = NT == 4;
  // Which 16-byte pieces of a row trade places (xor), so that the eight lanes
  // of a shared-memory phase read eight different 16-byte columns of the
  // banks' 128 bytes.  K: rows g, g + 1, four pieces side by side; V: rows 2t
  // (or 2t + 1) for t = 0..3, pieces g, g + 1.  Rows of 64 bytes: two to a
  // 128-byte line, so the line counts in place of the row.
  __host__ __device__ static constexpr int swap(bool v, int r) {
    if (kRowB == 64) return v ? ((r >> 1) & 3) : 0;
    return v ? (r & 6) : (r & 1) << 2;
  }
};

// Dynamic shared memory: the warps' rings and, after a tile's last key, the
// join's buffers in the same place; then the E4M3 scale bytes and, for 32
// rows, the queries.
template <int D, int NT>
struct Join {
  float o[kWarps][8 * NT][D + 4];
  float m[kWarps][8 * NT], l[kWarps][8 * NT];
};
struct Scales {
  uint8_t b[kWarps][2][2][64];  // [warp][chunk mod 2][K, V][key]
};
template <int D>
struct Queries {
  uint2 q[4][D / 16][32];  // [8 rows][K step][lane]
  float scale[32];
};
template <int D, int NT>
constexpr size_t ring_bytes() {
  return sizeof(Join<D, NT>) > kRingB ? (sizeof(Join<D, NT>) + 15) / 16 * 16 : kRingB;
}

template <int D, bool FP8, int NT>
__global__ void __launch_bounds__(kThreads, kCtas) paged_decode_kernel(const PagedParams p) {
  using C = Decode<D, FP8, NT>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int sm_last;
  Join<D, NT>& sm = *reinterpret_cast<Join<D, NT>*>(smem);
  Scales& scl = *reinterpret_cast<Scales*>(smem + ring_bytes<D, NT>());
  [[maybe_unused]] Queries<D>& qsm = *reinterpret_cast<Queries<D>*>(smem + ring_bytes<D, NT>() + sizeof(Scales));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  PagedHeader* hdr = p.hdr;
  // the chunk kernel, where one follows, works on other rows: its CTAs come in
  // as this kernel's leave
  asm volatile("griddepcontrol.launch_dependents;");
  const int w = blockIdx.x;
  const WorkerRec rec = p.workers[w];  // on its way while the signature is
  if (!planned(p)) return;
  int left = rec.n, at = rec.at, h = rec.h, pos = rec.pos;
  if (left == 0) return;
  ReqRec rq = rec.q;

  while (true) {
    // the worker's part of this tile: blocks [blk, blk + nb) behind the tile's own cost
    const int take = min(left, rq.per_head - pos), blk = max(0, pos - kDecodeTileCost);
    const int blocks = rq.per_head - kDecodeTileCost, nb = max(0, pos + take - kDecodeTileCost) - blk;
    const int r = rq.r;
    const int kbeg = blk * kDecodeBlk, kend = min(rq.kv_len, (blk + nb) * kDecodeBlk);
   if (nb > 0) {
    const int rows = rq.q_len * p.G;
    // ------------------------------------------------ queries (B operand) and column limits
    // fragments of rows 8 nt .. 8 nt + 7, and the score factor of row g of them
    auto load_q = [&](int nt, uint32_t (&f)[D / 16][2]) {
      const int row = 8 * nt + g;
      const int tok = row / p.G, hq = h * p.G + (row - tok * p.G);
      const __nv_bfloat16* src = p.q + (int64_t)(rq.q0 + tok) * p.q_stride + (int64_t)hq * D;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        // K step ks of lane t: channels d .. d + 3, as the K loads deal them
        const int d = FP8 ? (ks >> 2) * 64 + t * 16 + (ks & 3) * 4 : (ks >> 1) * 32 + t * 8 + (ks & 1) * 4;
        uint2 x = make_uint2(0, 0);
        if (row < rows) x = __ldg(reinterpret_cast<const uint2*>(src + d));
        f[ks][0] = x.x;
        f[ks][1] = x.y;
      }
      float scale = p.c_log2;
      if constexpr (FP8) {
        uint32_t top = 0;  // largest magnitude's bits
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int i = 0; i < 2; ++i) top = max(top, max(f[ks][i] & 0x7FFFu, (f[ks][i] >> 16) & 0x7FFFu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // exponent field E: the row's largest element is below 2^(E - 126);
        // times 2^(139 - E) it is below 2^13 (E clamped: the factor and its inverse stay normal)
        const int E = min(max((int)(top >> 7), 13), 254);
        const float up = exp2i(139 - E);
        // with the 2^12 that the keys' scales lack; above 0: a masked -inf stays one
        scale = fminf(fmaxf(scale * exp2i(E - 127), 1.17549435e-38f), 3.4e38f);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int i = 0; i < 2; ++i) f[ks][i] = pack_f16x2(bf16_lo(f[ks][i]) * up, bf16_hi(f[ks][i]) * up);
      }
      return scale;
    };
    [[maybe_unused]] uint32_t qf[C::kQShared ? 1 : NT][D / 16][2];
    float cq[NT][2];  // score factor of columns 2t, 2t + 1
    int vis[NT][2];   // keys that they see
    int vis_min = kend;
    if constexpr (C::kQShared) {  // a warp each
      static_assert(kWarps == NT || !C::kQShared, "a warp for every eight rows");
      uint32_t f[D / 16][2];
      const float scale = load_q(warp, f);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) qsm.q[warp][ks][lane] = make_uint2(f[ks][0], f[ks][1]);
      if (t == 0) qsm.scale[8 * warp + g] = scale;
      __syncthreads();
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float scale = 0.f;
      if constexpr (!C::kQShared) scale = load_q(nt, qf[nt]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        cq[nt][e] = C::kQShared ? qsm.scale[8 * nt + 2 * t + e] : __shfl_sync(0xffffffffu, scale, 4 * (2 * t + e));
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
    const uint32_t ring = smem_u32(smem) + warp * 4 * kUnit;  // K, V of even chunks, K, V of odd ones
    const uint32_t scales = smem_u32(scl.b[warp]);
    // Request a chunk's K (or V) and its scale bytes: one group of copies
    // each.  A copy instruction takes 512 contiguous bytes: with K in the
    // fragments' own order (64-byte pieces of eight rows) the decode of 65,522
    // tokens took 74 us in place of 59.
    // 16-byte piece c of row r lies at r * kRowB + 16 * (c ^ swap(r)): the reads
    // below then meet no bank twice.
    auto request = [&](int it, int pg, auto is_v) {
      constexpr bool kV = decltype(is_v)::value;
      constexpr int kPieces = C::kRowB / 16, kRowsAt = 32 / kPieces;  // of a row; rows of an instruction
      const int key0 = key_of(it);
      const int row = lane / kPieces, piece = lane % kPieces;
      const uint32_t dst = ring + (2 * (it & 1) + kV) * kUnit;
#pragma unroll
      for (int s = 0; s < C::kSub; ++s) {
        const int id = __shfl_sync(0xffffffffu, pg, (it % kGroup) * C::kSub + s);
        const int key = key0 + 16 * s;
        const int64_t in_page = (int64_t)h * p.page_size + (key & (p.page_size - 1));
        const uint8_t* src = (kV ? p.v : p.k) + id * p.page_bytes + in_page * C::kRowB + lane * 16;
#pragma unroll
        for (int i = 0; i < 16 / kRowsAt; ++i) {
          const int rr = i * kRowsAt + row;
          copy16(dst + (16 * s + rr) * C::kRowB + ((piece ^ C::swap(kV, rr)) << 4), src + i * 512, key + rr < kend ? 16 : 0);
        }
        if constexpr (FP8) {
          // 16 bytes of one page; zero for keys from kend on, whose slots hold
          // what an earlier owner left: the reference below is a maximum
          if (lane == s)
            copy16(scales + ((it & 1) * 2 + kV) * 64 + 16 * s, (kV ? p.v_scales : p.k_scales) + (int64_t)id * p.Hkv * p.page_size + in_page,
                   min(max(kend - key, 0), 16));
        }
      }
      copy_commit();
    };
    using K_ = std::integral_constant<bool, false>;
    using V_ = std::integral_constant<bool, true>;

    float o[C::kMT][NT][4];
    float m[NT][2], l[NT][2];
    // bf16: an infinity in V times the lower term, or times the weight 0 of a
    // row that may not see it, gives a NaN that the formula does not have.  So
    // a warp that ends with a NaN takes its keys once more, carefully; E4M3: one
    // that meets V exponents more than kSpread apart.
    // A loop of its own: in one with the usual pass, the 32-row kernel spilled
    // (drafts 63 -> 72 us).
    [[maybe_unused]] int e_ref = 0;  // E + 127: the largest V scale byte so far
   auto pass = [&](auto careful_) {  // true: to be done carefully
    constexpr bool careful = decltype(careful_)::value;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < C::kMT; ++i) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
    }
    e_ref = FP8 && careful ? 134 : 0;  // 134: no factor
    [[maybe_unused]] int e_low = 255;  // the smallest that this lane has read
    int pg = 0, pg_next = 0;
    if (n_it > 0) {
      pg = page_group(0);
      request(0, pg, K_{});
      request(0, pg, V_{});
      if (n_it > 1) {
        request(1, pg, K_{});
        request(1, pg, V_{});
      } else {
        copy_commit();
        copy_commit();
      }
      if (n_it > kGroup) pg_next = page_group(kGroup);
    }
    for (int it = 0; it < n_it; ++it) {
      const int key0 = key_of(it);
      const uint32_t kb = ring + 2 * (it & 1) * kUnit, vb = kb + kUnit;
      // the page ids of chunk it + 2
      if ((it + 2) % kGroup == 0) {
        pg = pg_next;
        if (it + 2 + kGroup < n_it) pg_next = page_group(it + 2 + kGroup);
      }
      // ---------------------------------------------- S^T = K Q^T
      copy_wait<3>();
      __syncwarp();  // the bytes are other lanes' copies
      float s[C::kSub][NT][4];
#pragma unroll
      for (int i = 0; i < C::kSub; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[i][nt][0] = s[i][nt][1] = s[i][nt][2] = s[i][nt][3] = 0.f;
      // the queries' fragments of a K step serve all key tiles
      constexpr int kU = FP8 ? 4 : 2;  // K steps of a 64-byte piece
#pragma unroll
      for (int j = 0; j < C::kKJ; ++j) {
        uint32_t x[C::kSub][4], y[C::kSub][4];
#pragma unroll
        for (int i = 0; i < C::kSub; ++i) {
          const uint32_t a = kb + (16 * i + g) * C::kRowB + (((4 * j + t) ^ C::swap(false, g)) << 4);  // g and g + 8 alike
          const uint4 u0 = lds16(a), u1 = lds16(a + 8 * C::kRowB);
          x[i][0] = u0.x, x[i][1] = u0.y, x[i][2] = u0.z, x[i][3] = u0.w;
          y[i][0] = u1.x, y[i][1] = u1.y, y[i][2] = u1.z, y[i][3] = u1.w;
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          uint32_t b[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if constexpr (C::kQShared) {
              const uint2 q = qsm.q[nt][kU * j + u][lane];
              b[nt][0] = q.x;
              b[nt][1] = q.y;
            } else {
              b[nt][0] = qf[nt][kU * j + u][0];
              b[nt][1] = qf[nt][kU * j + u][1];
            }
          }
#pragma unroll
          for (int i = 0; i < C::kSub; ++i) {
            if constexpr (FP8) {
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_f16(x[i][u], a0, a2);
              e4m3x4_to_f16(y[i][u], a1, a3);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_f16(s[i][nt], a0, a1, a2, a3, b[nt][0], b[nt][1]);
            } else {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_bf16(s[i][nt], x[i][2 * u], y[i][2 * u], x[i][2 * u + 1], y[i][2 * u + 1], b[nt][0], b[nt][1]);
            }
          }
        }
      }
      if constexpr (FP8) {
        const uint8_t* sk = scl.b[warp][it & 1][0];
#pragma unroll
        for (int i = 0; i < C::kSub; ++i) {
          const float f0 = ue8m0(sk[16 * i + g]) * 0x1p-12f, f1 = ue8m0(sk[16 * i + 8 + g]) * 0x1p-12f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              s[i][nt][e] *= f0;
              s[i][nt][2 + e] *= f1;
            }
        }
      }
      __syncwarp();  // every lane has read K: its place is free
      if (it + 2 < n_it) request(it + 2, pg, K_{});
      else copy_commit();
      // ---------------------------------------------- scores, reference, weights
      float top[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) top[nt][0] = top[nt][1] = -INFINITY;
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
          top[nt][e] *= cq[nt][e];  // the factor is positive
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
      // ---------------------------------------------- weights: P^T as B operand
      uint32_t hi[C::kSub][NT][2];
      [[maybe_unused]] uint32_t lo[FP8 ? 1 : C::kSub][NT][2];
      copy_wait<3>();  // this chunk's V
      __syncwarp();
      bool nan_key = false;
      if constexpr (FP8) {
        const uint8_t* sv = scl.b[warp][it & 1][1];
        int e_top = 0;
#pragma unroll
        for (int i = 0; i < C::kSub; ++i) {
          const int b = sv[16 * i + (lane & 15)];
          e_top = max(e_top, b == 255 ? 0 : b);
          if (key0 + 16 * i + (lane & 15) < kend) e_low = min(e_low, b);
          nan_key |= b == 255;
        }
        nan_key = __any_sync(0xffffffffu, nan_key);
        if (!careful &&
            __any_sync(0xffffffffu, e_top > e_ref || e_low < e_ref - kSpread)) {
          e_top = __reduce_max_sync(0xffffffffu, max(e_top, e_ref));
          if (e_top - __reduce_min_sync(0xffffffffu, e_low) > kSpread) {
            copy_wait<0>();  // the ring's copies in flight
            __syncwarp();
            return true;
          }
          const float a = e_top - e_ref < 127 ? exp2i(e_ref - e_top) : 0.f;
          e_ref = e_top;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < C::kMT; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[i][nt][e] *= a;
        }
      }
      float neg[NT][2];  // minus the references
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) neg[nt][e] = m[nt][e] == -INFINITY ? 0.f : -m[nt][e];
      // keep: a NaN scale's key stays with the rows that see it (0 x NaN)
      auto weights = [&](auto keep) {
#pragma unroll
        for (int i = 0; i < C::kSub; ++i) {
          [[maybe_unused]] float f[2];
          if constexpr (FP8) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int b = scl.b[warp][it & 1][1][16 * i + 8 * k + g];
              f[k] = __uint_as_float(max(b - e_ref + 134, 0) << 23);
              if (decltype(keep)::value && b == 255) f[k] = __uint_as_float(0x7FC00000u);
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float y[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                y[e] = ex2_approx(__fmaf_rn(s[i][nt][2 * k + e], cq[nt][e], neg[nt][e]));
                l[nt][e] += y[e];
                if constexpr (FP8) y[e] = decltype(keep)::value && s[i][nt][2 * k + e] == -INFINITY ? 0.f : y[e] * f[k];
              }
              if constexpr (FP8) {
                hi[i][nt][k] = transpose8(pack_f16x2(y[0], y[1]));
              } else {
                const uint32_t a = pack_bf16x2(y[0], y[1]);
                hi[i][nt][k] = transpose8(a);
                lo[i][nt][k] = transpose8(pack_bf16x2(y[0] - bf16_lo(a), y[1] - bf16_hi(a)));
              }
            }
        }
      };
      if (FP8 && nan_key) {
        // its codes may be NaN too: the NaN comes with the weight, and rows that
        // do not see it have the weight 0 (0 x NaN)
        for (int key = 0; key < C::kChunk; ++key)
          if (scl.b[warp][it & 1][1][key] == 255 && lane < C::kRowB / 4)
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(vb + key * C::kRowB + lane * 4), "r"(0) : "memory");
        __syncwarp();
      }
      // E4M3, careful: V as bf16 values, two bf16 terms a weight; eight rows of
      // one key tile at a time, so that it needs no registers beside the usual
      // pass's (all rows at once spilled 500 bytes of the 32-row kernel)
      auto add_careful = [&] {
        const uint8_t* sv = scl.b[warp][it & 1][1];
#pragma unroll
        for (int i = 0; i < C::kSub; ++i) {
          // 2^120 times the scales of keys 2t, 2t + 1 (then 2t + 8, 2t + 9) in two
          // factors, as bf16 pairs
          uint32_t f[2][2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t b0 = min((int)sv[16 * i + 8 * k + 2 * t], 254), b1 = min((int)sv[16 * i + 8 * k + 2 * t + 1], 254);
            f[k][0] = ((min(b0, 134u) + 120u) << 7) | ((min(b1, 134u) + 120u) << 23);
            f[k][1] = ((max(b0, 134u) - 7u) << 7) | ((max(b1, 134u) - 7u) << 23);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            uint32_t ph[2], pl[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float y[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float x = s[i][nt][2 * k + e];
                y[e] = ex2_approx(__fmaf_rn(x, cq[nt][e], neg[nt][e]));
                l[nt][e] += y[e];
                if (sv[16 * i + 8 * k + g] == 255 && x != -INFINITY) y[e] = __uint_as_float(0x7FC00000u);
              }
              const uint32_t a = pack_bf16x2(y[0], y[1]);
              ph[k] = transpose8(a);
              pl[k] = transpose8(pack_bf16x2(y[0] - bf16_lo(a), y[1] - bf16_hi(a)));
            }
#pragma unroll
            for (int x = 0; x < C::kVW; ++x) {
              uint32_t w[4];  // channels 4x .. 4x + 3 of four keys
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int rk = 2 * t + (k & 1) + 8 * (k >> 1);
                const uint32_t piece = C::kVW == 2 ? g >> 1 : g, in = C::kVW == 2 ? (g & 1) * 8 + 4 * x : 4 * x;
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[k])
                             : "r"(vb + (16 * i + rk) * C::kRowB + ((piece ^ C::swap(true, rk)) << 4) + in) : "memory");
              }
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                uint32_t a[4];  // channels 4x + 2 half, + 1: keys 2t, 2t + 1; the same of 2t + 8, 2t + 9
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const uint32_t two = prmt(w[k & 2], w[(k & 2) + 1], 0x5410u + 0x2222u * half) >> (8 * (k & 1)) & 0x00FF00FFu;
                  a[k] = bf16x2_mul(bf16x2_mul(e4m3_to_bf16x2(two), f[k >> 1][0]), f[k >> 1][1]);
                }
                mma_bf16(o[2 * x + half][nt], a[0], a[1], a[2], a[3], ph[0], ph[1]);
                mma_bf16(o[2 * x + half][nt], a[0], a[1], a[2], a[3], pl[0], pl[1]);
              }
            }
          }
        }
      };
      if constexpr (FP8 && careful) {
        add_careful();
      } else if (FP8 && nan_key) {
        weights(std::true_type{});
      } else {
        weights(std::false_type{});
      }
      // ---------------------------------------------- O^T += V^T P^T
      // tok >= 0 (careful): only the columns of token tok, over the keys that
      // it sees, and the lower terms over finite values
      auto add_pv = [&](int tok) {
        const int lim = tok < 0 ? INT_MAX : visible_keys(p.causal, rq.q_len, rq.kv_len, tok) - key0;
#pragma unroll
        for (int i = 0; i < C::kSub; ++i) {
          // four channel tiles (E4M3: 16 bytes of a row are eight) at a time
          constexpr int kW = C::kVW == 2 ? 2 : 4;  // words a load gives
#pragma unroll
          for (int j = 0; j < C::kVW / kW; ++j) {
            uint32_t w[4][kW];  // [key][word]
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int rk = 2 * t + (k & 1) + 8 * (k >> 1);
              const uint32_t at = vb + (16 * i + rk) * C::kRowB;
              if constexpr (kW == 2) {
                const uint2 x = lds8(at + ((((g >> 1) ^ C::swap(true, rk)) << 4) | (g & 1) << 3));
                w[k][0] = x.x;
                w[k][1] = x.y;
              } else {
                const uint4 x = lds16(at + (((8 * j + g) ^ C::swap(true, rk)) << 4));
                w[k][0] = x.x;
                w[k][1] = x.y;
                w[k][kW - 2] = x.z;
                w[k][kW - 1] = x.w;
              }
              if (!FP8 && 16 * i + 2 * t + (k & 1) + 8 * (k >> 1) >= lim)
#pragma unroll
                for (int x = 0; x < kW; ++x) w[k][x] = 0u;
            }
            if constexpr (FP8) {
#pragma unroll
              for (int x = 0; x < kW; ++x) {
                // codes of two keys side by side before they are converted: half
                // the permutations of doing it after
                uint32_t a01[4], a23[4];  // channels 4x .. 4x + 3: keys 2t, 2t + 1 and 2t + 8, 2t + 9
                e4m3x4_to_f16(prmt(w[0][x], w[1][x], 0x5140u), a01[0], a01[1]);
                e4m3x4_to_f16(prmt(w[0][x], w[1][x], 0x7362u), a01[2], a01[3]);
                e4m3x4_to_f16(prmt(w[2][x], w[3][x], 0x5140u), a23[0], a23[1]);
                e4m3x4_to_f16(prmt(w[2][x], w[3][x], 0x7362u), a23[2], a23[3]);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt)
                    mma_f16(o[2 * x + half][nt], a01[2 * half], a01[2 * half + 1], a23[2 * half], a23[2 * half + 1], hi[i][nt][0], hi[i][nt][1]);
                }
              }
            } else {
#pragma unroll
              for (int x = 0; x < kW; ++x) {
                const int mt = 4 * j + x;
                uint32_t a[4] = {prmt(w[0][x], w[1][x], 0x5410u), prmt(w[0][x], w[1][x], 0x7632u),
                                 prmt(w[2][x], w[3][x], 0x5410u), prmt(w[2][x], w[3][x], 0x7632u)};
                float c[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                  for (int e = 0; e < 4; ++e) c[nt][e] = o[mt][nt][e];
                  mma_bf16(c[nt], a[0], a[1], a[2], a[3], hi[i][nt][0], hi[i][nt][1]);
                }
                if (tok >= 0) {
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    if ((a[k] & 0x7F80u) == 0x7F80u) a[k] &= 0xFFFF0000u;
                    if ((a[k] & 0x7F800000u) == 0x7F800000u) a[k] &= 0xFFFFu;
                  }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  mma_bf16(c[nt], a[0], a[1], a[2], a[3], lo[i][nt][0], lo[i][nt][1]);
#pragma unroll
                  for (int e = 0; e < 2; ++e)
                    if (tok < 0 || (8 * nt + 2 * t + e) / p.G == tok) {
                      o[mt][nt][e] = c[nt][e];
                      o[mt][nt][2 + e] = c[nt][2 + e];
                    }
                }
              }
            }
          }
        }
      };
      if constexpr (!careful) {
        add_pv(-1);
      } else if constexpr (!FP8) {
#pragma unroll 1
        for (int tok = 0; tok < rq.q_len; ++tok) add_pv(tok);
      }
      __syncwarp();  // every lane has read V
      if (it + 2 < n_it) request(it + 2, pg, V_{});
      else copy_commit();
    }

    if (FP8 || careful) return false;
    float sum = 0.f;  // NaN where one of them is, and for infinities of both signs
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < C::kMT; ++i) sum += (o[i][nt][0] + o[i][nt][1]) + (o[i][nt][2] + o[i][nt][3]);
    return (bool)__any_sync(0xffffffffu, sum != sum);
   };
    if (pass(std::false_type{})) pass(std::true_type{});

    // ------------------------------------------------ join the warps
    if constexpr (FP8) {  // the accumulators hold 2^(134 - e_ref) times the sum; in two normal factors
      const float f0 = exp2i((e_ref - 134) / 2), f1 = exp2i(e_ref - 134 - (e_ref - 134) / 2);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < C::kMT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][nt][e] = o[i][nt][e] * f0 * f1;
    }
    __syncthreads();  // every warp is done with its ring
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
    const bool whole = nb == blocks;
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
      const int64_t cost = hdr->cost[0], tile0 = rq.base + (int64_t)h * rq.per_head;
      const int W = hdr->workers[0];
      const int w0 = worker_of(tile0 + kDecodeTileCost, cost, W), n = worker_of(tile0 + rq.per_head - 1, cost, W) - w0 + 1;
      const int slot = blk == 0 ? 2 * w + 1 : 2 * w;
      float* po = p.part_o + ((int64_t)slot * C::kQ + row) * D + d0;
#pragma unroll
      for (int k = 0; k < kPer; k += 4)
        __stcg(reinterpret_cast<float4*>(po + k), make_float4(acc[k], acc[k + 1], acc[k + 2], acc[k + 3]));
      if (d0 == 0) __stcg(p.part_ml + (int64_t)slot * C::kQ + row, make_float2(M, L));
      __syncthreads();
      if (tid == 0) {
        __threadfence();  // after the barrier: for the whole CTA
        const bool last = atomicAdd(&hdr->count[w0], 1u) == (unsigned)(n - 1);
        if (last) hdr->count[w0] = 0;
        sm_last = last;
      }
      __syncthreads();
      write = sm_last;
      if (write) {
        // A row's threads form the partials' weights together, then add up
        // their channels, eight partials in flight (one after the other, 57 of
        // them took 20 us).
        __threadfence();
        auto slot_of = [&](int i) { return (int64_t)(i == 0 ? 2 * w0 + 1 : 2 * (w0 + i)); };
        float* wt = reinterpret_cast<float*>(smem);  // [n][kQ]; the join's buffers are free
        const int me = tid % kSpan;
        constexpr int kOwn = 4;  // a thread's first partials are read once
        float2 own[kOwn];
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
          const int i = me + j * kSpan;
          own[j] = i < n ? __ldcg(p.part_ml + slot_of(i) * C::kQ + row) : make_float2(-INFINITY, 0.f);
        }
        M = -INFINITY;
#pragma unroll
        for (int j = 0; j < kOwn; ++j) M = fmaxf(M, own[j].x);
        for (int i = me + kOwn * kSpan; i < n; i += kSpan) M = fmaxf(M, __ldcg(p.part_ml + slot_of(i) * C::kQ + row).x);
#pragma unroll
        for (int k = kSpan / 2; k; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
        L = 0.f;
        auto weigh = [&](int i, float2 x) {
          const float a = x.x == M ? 1.f : ex2_approx(x.x - M);
          L += a * x.y;
          wt[i * C::kQ + row] = a;
        };
#pragma unroll
        for (int j = 0; j < kOwn; ++j)
          if (me + j * kSpan < n) weigh(me + j * kSpan, own[j]);
        for (int i = me + kOwn * kSpan; i < n; i += kSpan) weigh(i, __ldcg(p.part_ml + slot_of(i) * C::kQ + row));
#pragma unroll
        for (int k = kSpan / 2; k; k >>= 1) L += __shfl_xor_sync(0xffffffffu, L, k);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
#pragma unroll (kPer <= 16 ? 8 : 2)
        for (int i = 0; i < n; ++i) {
          const float a = wt[i * C::kQ + row];
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
   }
    left -= take;
    if (left == 0) break;
    pos = 0;
    if (++h == p.Hkv) {
      h = 0;
      rq = p.reqs[++at];
    }
  }
}

template <int D, bool FP8, int NT>
cudaError_t launch(const PagedParams& p, cudaStream_t st) {
  constexpr size_t smem = ring_bytes<D, NT>() + sizeof(Scales) + (NT == 4 ? sizeof(Queries<D>) : 0);
  static_assert(sizeof(float) * kMaxWorkers * 8 * NT <= ring_bytes<D, NT>(), "the weights lie in the rings' place");
  static bool attr_set[64] = {};  // per device: raised once
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(paged_decode_kernel<D, FP8, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  paged_decode_kernel<D, FP8, NT><<<p.W_max[0], kThreads, smem, st>>>(p);
  return cudaGetLastError();
}
template <int D, bool FP8>
cudaError_t launch_n(const PagedParams& p, cudaStream_t st) {
  return p.small_rows == 8 ? launch<D, FP8, 1>(p, st) : p.small_rows == 16 ? launch<D, FP8, 2>(p, st) : launch<D, FP8, 4>(p, st);
}

}  // namespace

int paged_decode_workers(int sms) { return sms * kCtas; }

cudaError_t launch_paged_decode(const PagedParams& p, int d, bool e4m3, cudaStream_t st) {
  if (d == 128) return e4m3 ? launch_n<128, true>(p, st) : launch_n<128, false>(p, st);
  return e4m3 ? launch_n<64, true>(p, st) : launch_n<64, false>(p, st);
}

}  // namespace flamia
