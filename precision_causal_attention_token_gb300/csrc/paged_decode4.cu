// paged_decode4.cu — attention of few query rows over a paged cache of four
// bits (E2M1 codes, an E4M3 scale for each 16 channels, a power of two a row).
//
// The products and the join are those of paged_decode.cu: S^T = K Q^T and O^T =
// V^T P^T as m16n8k16 MMAs in f16, a warp on its own chunks of keys.  A byte
// holds two values here, so the kernel is bound by the instructions that turn
// codes into operands as much as by HBM (281,000 keys of 8 heads: 328 MB, 49 us
// of HBM; 0.57 of E4M3's bytes).  For a pair of values these are one conversion and one
// multiplication by the block scale, both exact in f16 (1 + 1 mantissa bits
// times 1 + 3, up to 6 * 448).  A chunk's copies are asynchronous 16-byte
// copies, 512 contiguous bytes an instruction, into a ring of the warp's own
// (boxes by TMA, a lane each, took 415 instructions a key tile against 390 then: their
// operands are per warp, so the lanes' boxes are issued one after the other).  Slots behind a
// request's last token hold what an earlier owner left: V's block scales there
// are replaced by zeros (codes are always finite).
// In V two keys' codes are interleaved by nibbles before they are converted,
// so that a conversion gives the pair that the MMA's fragment holds.
//
// Scales of queries and keys, f16 weights relative to the largest exponent of
// V and the careful second pass (bf16 values, two bf16 terms a weight) where
// exponents lie more than kSpread apart: as for E4M3, see paged_decode.cu.  V near the
// largest numbers: bf16 values of 2^128 (an append may round the largest row up to
// there) would be infinite, and NaN times the weight 0 of a row that does not see them,
// and sums of such values would overflow although their mean does not.  Once a warp has met an
// exponent byte of kWideByte (V of 2^66 and more), its sums, and in the careful pass V, are
// 2^-kWideShift times themselves, with the reference kWideShift higher: 32,000 of
// the largest rows add up.
//
// Measured (152 SMs, H = 32, Hkv = 8, d = 128): 64 requests, 281,000 tokens, 80 us
// (4.1 TB/s, 61% of the copy rate; the E4M3 kernel 109 us for 1.76 times the
// bytes; its own code with E2M1 operands took 104); one request of 65,522 tokens
// 28 us; 32 requests of 2 to 4 drafted tokens 70 us (205 MB), 16 of 2 to 8 (32 rows) 68 (96 MB).
// Of a long tile's 113,000 cycles of loop, the loads alone take 95,000 and the
// instructions alone 97,000; 6 us go by before a CTA's first chunk is there and
// 3 to 4 with each tile's join.  With d = 64: 55 us for 166 MB.
#include <type_traits>

#include "paged_decode.cuh"

namespace flamia {

namespace {

__device__ __forceinline__ uint32_t lds4(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds2(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds1(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float f16_lo(uint32_t v) { return __half2float(__ushort_as_half((unsigned short)(v & 0xFFFFu))); }
__device__ __forceinline__ float f16_hi(uint32_t v) { return __half2float(__ushort_as_half((unsigned short)(v >> 16))); }

constexpr int kWideByte = 192, kWideShift = 24;
constexpr int kCareful = 134, kCarefulWide = 512;  // e_ref of the careful pass: no factor, 2^-kWideShift in V

template <int D, int NT>
struct Cfg {
  // Up to 8 rows a thread needs 168 registers: twelve warps an SM (eight: 87
  // against 85 us on the batch of 64, 64.6 against 60.6 at d = 64).
  static constexpr int kWarps = NT == 1 ? 6 : 4, kThreads = 32 * kWarps, kCtas = 2;
  static constexpr int kRowB = D / 2;               // bytes of a row's codes
  static constexpr int kChunk = NT != 2 && D == 128 ? 32 : 64;  // keys a warp takes at a time (32: registers)
  static constexpr int kSub = kChunk / 16, kUnit = kChunk * kRowB;
  static constexpr int kStages = kUnit == 4096 || NT == 1 ? 2 : 3;  // chunks of a warp's ring
  // The next tile's first chunks come in while this one is joined; 32 rows have
  // neither the registers (drafts of 2 to 8 tokens: 69 -> 89 us) nor the memory.
  static constexpr bool kEarly = NT < 4;
  static constexpr int kMT = D / 16;                // m16 channel tiles
  static constexpr int kBl = D / 16;                // block scales of a row
  static constexpr bool kQShared = NT == 4;
  static_assert(kSub * kBl <= 32, "a 16-byte piece of block scales a lane");
  // A row's 16-byte piece c lies at c ^ swap(r).  K: eight lanes read two whole rows; V: rows 0, 2, 4, 6 of
  // eight keys, half a row of each, find eight different 16-byte columns (rows of
  // 32 bytes: two meet).
  __host__ __device__ static constexpr int swap(int r) { return D == 128 ? (r >> 1) & 3 : (r >> 2) & 1; }
};

template <int D, int NT>
struct Ring {  // per warp
  uint8_t codes[Cfg<D, NT>::kStages][2][Cfg<D, NT>::kUnit];  // [K, V]
};
template <int D, int NT>
struct __align__(16) Small {
  uint8_t blocks[Cfg<D, NT>::kWarps][Cfg<D, NT>::kStages][2][Cfg<D, NT>::kChunk * (D / 16)];
  uint8_t scales[Cfg<D, NT>::kWarps][Cfg<D, NT>::kStages][2][Cfg<D, NT>::kChunk];
  uint2 q[NT == 4 ? 4 : 1][NT == 4 ? D / 16 : 1][32];  // 32 rows: the queries' fragments
  float scale[32];
  int last;
};
// Shared memory: the rings, the join's buffers or the partials' weights (behind
// the rings where the next chunks come in meanwhile, else in their place), the rest.
template <int D, int NT>
constexpr size_t join_at() { return Cfg<D, NT>::kEarly ? sizeof(Ring<D, NT>) * Cfg<D, NT>::kWarps : 0; }
template <int D, int NT>
constexpr size_t small_at() {
  constexpr size_t j = (sizeof(Join<D, NT, Cfg<D, NT>::kWarps>) + 15) / 16 * 16, w = sizeof(float) * kMaxWorkers * 8 * NT;
  constexpr size_t end = join_at<D, NT>() + (j > w ? j : w), ring = sizeof(Ring<D, NT>) * Cfg<D, NT>::kWarps;
  return end > ring ? end : ring;
}

template <int D, int NT>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, Cfg<D, NT>::kCtas)
    paged_decode4_kernel(const PagedParams p) {
  using C = Cfg<D, NT>;
  constexpr int kWarps = C::kWarps, kSub = C::kSub, kS = C::kStages, kBl = C::kBl;
  extern __shared__ __align__(16) uint8_t smem[];
  Join<D, NT, kWarps>& sm = *reinterpret_cast<Join<D, NT, kWarps>*>(smem + join_at<D, NT>());
  Small<D, NT>& sml = *reinterpret_cast<Small<D, NT>*>(smem + small_at<D, NT>());
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

  // This lane's part of a chunk's requests: every 32nd piece of the codes, a
  // piece of one key tile's block scales, and (the first of its pieces) the
  // tile's scales.
  constexpr int kUnit = C::kUnit, kBlkB = C::kChunk * kBl;
  const uint32_t ring = smem_u32(smem) + warp * (uint32_t)sizeof(Ring<D, NT>);
  const uint32_t blocks_at = smem_u32(sml.blocks[warp]), scales_at = smem_u32(sml.scales[warp]);
  constexpr int kPieces = C::kRowB / 16, kRowsAt = 32 / kPieces;  // pieces of a row; rows of an instruction
  const uint32_t codes_at = ring + (lane / kPieces) * C::kRowB + ((lane % kPieces ^ C::swap(lane / kPieces)) << 4);
  const int piece = lane % kBl, piece_tile = lane / kBl;
  const uint32_t page_rows = (uint32_t)p.Hkv * p.page_size;

  // ------------------------------------------------ the worker's tiles
  // Its part of the present one: blocks [blk, blk + nb) behind the tile's own cost.
  int take = 0, blk = 0, nb = 0, kbeg = 0, kend = 0, n_it = 0;
  auto advance = [&] {  // to the next tile with blocks for it; false: none
    do {
      left -= take;
      if (left == 0) return false;
      if (take) {
        pos = 0;
        if (++h == p.Hkv) {
          h = 0;
          rq = p.reqs[++at];
        }
      }
      take = min(left, rq.per_head - pos);
      blk = max(0, pos - kDecodeTileCost);
      nb = max(0, pos + take - kDecodeTileCost) - blk;
    } while (nb == 0);
    kbeg = blk * kDecodeBlk;
    kend = min(rq.kv_len, (blk + nb) * kDecodeBlk);
    // this warp's chunks
    n_it = (kend - kbeg - warp * C::kChunk + kWarps * C::kChunk - 1) / (kWarps * C::kChunk);
    return true;
  };
  auto key_of = [&](int it) { return kbeg + (it * kWarps + warp) * C::kChunk; };
  // Where the tiles of kGroup chunks lie: lane i of a group holds key tile i %
  // kSub of chunk it0 + i / kSub, as its codes' offset in the pool and its row
  // among all (page, head, token) rows.
  constexpr int kGroup = 32 / kSub;
  auto page_group = [&](int it0) {
    const int key = key_of(it0 + lane / kSub) + 16 * (lane % kSub);
    int id = key < kend ? __ldg(p.block_table + (int64_t)rq.r * p.max_pages + (key >> p.page_shift)) : 0;
    if ((unsigned)id >= (unsigned)p.n_pages) {
      report(&hdr->base, FLAMIA_ERR_BAD_PAGE, 0x721);
      id = 0;
    }
    return id;
  };
  int64_t at_code = 0, at_row = 0;
  auto place_group = [&](int it0, int id) {
    const int in_page = (key_of(it0 + lane / kSub) + 16 * (lane % kSub)) & (p.page_size - 1);
    const int64_t head_row = (int64_t)h * p.page_size + in_page;
    at_code = id * p.page_bytes + head_row * C::kRowB;
    at_row = (int64_t)id * page_rows + head_row;
  };
  const uint8_t* const k_src = p.k + lane * 16;
  const uint8_t* const v_src = p.v + lane * 16;
  auto request = [&](int it, int st) {
    const int from = (it % kGroup) * kSub;
#pragma unroll
    for (int i = 0; i < kSub; ++i) {
      const int64_t off = __shfl_sync(0xffffffffu, at_code, from + i);
      const uint32_t dst = codes_at + 2 * st * kUnit + 16 * i * C::kRowB;
#pragma unroll
      for (int r = 0; r < 16; r += kRowsAt) {  // rows of this lane: the same place in the swizzle
        copy16(dst + r * C::kRowB, k_src + off + r * C::kRowB, 16);
        copy16(dst + kUnit + r * C::kRowB, v_src + off + r * C::kRowB, 16);
      }
    }
    const int64_t row = __shfl_sync(0xffffffffu, at_row, from + piece_tile % kSub);
    if (kSub * kBl == 32 || lane < kSub * kBl) {
      const uint32_t dst = blocks_at + 2 * st * kBlkB + lane * 16;
      copy16(dst, p.k_blocks + row * kBl + piece * 16, 16);
      copy16(dst + kBlkB, p.v_blocks + row * kBl + piece * 16, 16);
      if (piece == 0) {
        const uint32_t to = scales_at + 2 * st * C::kChunk + piece_tile * 16;
        copy16(to, p.k_scales + row, 16);
        copy16(to + C::kChunk, p.v_scales + row, 16);
      }
    }
  };
  int id_next = 0;
  auto begin = [&] {  // the first chunks; a group of copies each
    if (n_it > 0) place_group(0, page_group(0));
#pragma unroll
    for (int s = 0; s < kS; ++s) {
      if (s < n_it) request(s, s);  // kS <= kGroup
      copy_commit();
    }
    if (n_it > kGroup) id_next = page_group(kGroup);
  };
  // The tile's queries as they are: K step ks of lane t holds channels t D / 4 +
  // 4 ks .. + 3 of a row, as the K loads deal them.  32 rows: eight a warp.
  uint32_t qf[C::kQShared ? 1 : NT][D / 16][2];
  auto ask_q = [&] {
#pragma unroll
    for (int nt = 0; nt < (C::kQShared ? 1 : NT); ++nt) {
      const int row = 8 * (C::kQShared ? warp : nt) + g;
      const int tok = row / p.G, hq = h * p.G + (row - tok * p.G);
      const __nv_bfloat16* src = p.q + (int64_t)(rq.q0 + tok) * p.q_stride + (int64_t)hq * D + t * (D / 4);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint2 x = make_uint2(0, 0);
        if (row < rq.q_len * p.G) x = __ldg(reinterpret_cast<const uint2*>(src + ks * 4));
        qf[nt][ks][0] = x.x;
        qf[nt][ks][1] = x.y;
      }
    }
  };

  if (!advance()) return;
  ask_q();
  begin();
  while (true) {
    const int rows = rq.q_len * p.G;
    // ------------------------------------------------ queries (B operand) and column limits
    auto scaled_q = [&](uint32_t (&f)[D / 16][2]) {  // as f16; returns the rows' score factor
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
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int i = 0; i < 2; ++i) f[ks][i] = pack_f16x2(bf16_lo(f[ks][i]) * up, bf16_hi(f[ks][i]) * up);
      // with the 2^12 that the keys' scales lack; above 0: a masked -inf stays one
      return fminf(fmaxf(p.c_log2 * exp2i(E - 127), 1.17549435e-38f), 3.4e38f);
    };
    float cq[NT][2];  // score factor of columns 2t, 2t + 1
    int vis[NT][2];   // keys that they see
    int vis_min = kend;
    if constexpr (C::kQShared) {  // a warp each
      static_assert(kWarps == NT || !C::kQShared, "a warp for every eight rows");
      const float scale = scaled_q(qf[0]);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) sml.q[warp][ks][lane] = make_uint2(qf[0][ks][0], qf[0][ks][1]);
      if (t == 0) sml.scale[8 * warp + g] = scale;
      __syncthreads();
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float scale = 0.f;
      if constexpr (!C::kQShared) scale = scaled_q(qf[nt]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        cq[nt][e] = C::kQShared ? sml.scale[8 * nt + 2 * t + e] : __shfl_sync(0xffffffffu, scale, 4 * (2 * t + e));
        const int c = 8 * nt + 2 * t + e;
        const int n = visible_keys(p.causal, rq.q_len, rq.kv_len, c / p.G);
        vis[nt][e] = c < rows ? n : kend;  // columns past the rows hold zeros
        vis_min = min(vis_min, vis[nt][e]);
      }
    }
    vis_min = __reduce_min_sync(0xffffffffu, vis_min);

    float o[C::kMT][NT][4];
    float m[NT][2], l[NT][2];
    int e_ref = 0;  // E + 127: the largest V scale byte so far
    // One pass over the warp's keys; true: to be done once more, carefully.  The
    // first chunks have been requested.
    auto pass = [&](auto careful_) {
      constexpr bool careful = decltype(careful_)::value;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int i = 0; i < C::kMT; ++i) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
      }
      e_ref = careful ? kCareful : 0;
      int e_low = 255;            // the smallest that this lane has read
      int st = 0;
      for (int it = 0; it < n_it; ++it) {
        const int key0 = key_of(it);
        const uint32_t kb = ring + 2 * st * kUnit, vb = kb + kUnit;
        const uint32_t bk = blocks_at + 2 * st * kBlkB, bv = bk + kBlkB, sk = scales_at + 2 * st * C::kChunk, sv = sk + C::kChunk;
        // the places of chunk it + kS
        if ((it + kS) % kGroup == 0) {
          place_group(it + kS, id_next);
          if (it + kS + kGroup < n_it) id_next = page_group(it + kS + kGroup);
        }
        copy_wait<kS - 1>();
        __syncwarp();  // the bytes are other lanes' copies
        if (key0 + C::kChunk > kend) {
          // Slots behind the last token hold what an earlier owner left: V's block
          // scales become 0 (0 x NaN is NaN), its exponents the last token's.
          const uint32_t last = lds1(sv + kend - 1 - key0);
          for (int key = kend - key0 + lane; key < C::kChunk; key += 32) {
            asm volatile("st.shared.u8 [%0], %1;" ::"r"(sv + key), "r"(last) : "memory");
#pragma unroll
            for (int k = 0; k < kBl; k += 4) asm volatile("st.shared.b32 [%0], %1;" ::"r"(bv + key * kBl + k), "r"(0) : "memory");
          }
          __syncwarp();
        }
        // ---------------------------------------------- what this chunk's exponents ask for
        // V: a new largest, one too far below it, NaN; K: 0 to 12 and NaN take more than a shift
        bool odd_k = false, nan_key = false;
        int e_top = 0;
        bool rare = false;
#pragma unroll
        for (int i = 0; i < C::kChunk / 32; ++i) {
          const int ek = lds1(sk + 32 * i + lane), ev = lds1(sv + 32 * i + lane);
          odd_k |= (unsigned)(ek - 13) > 241u;  // of a slot behind the last token: masked below, either way
          e_top = max(e_top, ev == 255 ? 0 : ev);
          e_low = min(e_low, ev);
          nan_key |= ev == 255;
          rare |= ev > e_ref;
        }
        rare |= odd_k || e_low < e_ref - kSpread;
        if (careful) rare = true;
        if (__any_sync(0xffffffffu, rare)) {
          odd_k = __any_sync(0xffffffffu, odd_k);
          nan_key = __any_sync(0xffffffffu, nan_key);
          if constexpr (!careful) {
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
          } else if (e_ref == kCareful && __any_sync(0xffffffffu, e_top >= kWideByte)) {
            e_ref = kCarefulWide;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < C::kMT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][nt][e] *= exp2i(-kWideShift);
          }
          if (nan_key) {
            // its block scales may be NaN too: the NaN comes with the weight, and
            // rows that do not see it have the weight 0 (0 x NaN)
            for (int key = 0; key < C::kChunk; ++key)
              if (lds1(sv + key) == 255 && lane < kBl)
                asm volatile("st.shared.u8 [%0], %1;" ::"r"(bv + key * kBl + lane), "r"(0) : "memory");
            __syncwarp();
          }
        } else {
          odd_k = nan_key = false;
        }
        // ---------------------------------------------- S^T = K Q^T
        float s[kSub][NT][4];
#pragma unroll
        for (int i = 0; i < kSub; ++i) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) s[i][nt][0] = s[i][nt][1] = s[i][nt][2] = s[i][nt][3] = 0.f;
          uint32_t x[D / 32], y[D / 32];  // of keys g, g + 8: channels t D / 4 ..
          uint32_t fx[2], fy[2];          // the block scales of these, as pairs of one value
          const uint32_t a = kb + (16 * i + g) * C::kRowB, b = bk + (16 * i + g) * kBl;
          if constexpr (D == 128) {
            const uint4 u0 = lds16(a + ((t ^ C::swap(g)) << 4)), u1 = lds16(a + 8 * C::kRowB + ((t ^ C::swap(g + 8)) << 4));
            x[0] = u0.x, x[1] = u0.y, x[2] = u0.z, x[3] = u0.w;
            y[0] = u1.x, y[1] = u1.y, y[2] = u1.z, y[3] = u1.w;
            const uint32_t s0 = e4m3x2_to_f16(lds2(b + 2 * t)), s1 = e4m3x2_to_f16(lds2(b + 8 * kBl + 2 * t));
            fx[0] = prmt(s0, 0u, 0x1010u), fx[1] = prmt(s0, 0u, 0x3232u);
            fy[0] = prmt(s1, 0u, 0x1010u), fy[1] = prmt(s1, 0u, 0x3232u);
          } else {
            const uint2 u0 = lds8(a + (((t >> 1) ^ C::swap(g)) << 4) + (t & 1) * 8);
            const uint2 u1 = lds8(a + 8 * C::kRowB + (((t >> 1) ^ C::swap(g + 8)) << 4) + (t & 1) * 8);
            x[0] = u0.x, x[1] = u0.y;
            y[0] = u1.x, y[1] = u1.y;
            fx[0] = fx[1] = e4m3x2_to_f16(lds1(b + t) * 0x0101u);
            fy[0] = fy[1] = e4m3x2_to_f16(lds1(b + 8 * kBl + t) * 0x0101u);
          }
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {  // a word: K steps 2k, 2k + 1
            uint32_t hx[4], hy[4];
            e2m1x8_to_f16(x[k], hx);
            e2m1x8_to_f16(y[k], hy);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              hx[e] = f16x2_mul(hx[e], fx[k / 2]);
              hy[e] = f16x2_mul(hy[e], fy[k / 2]);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                uint2 q;
                if constexpr (C::kQShared) q = sml.q[nt][2 * k + u][lane];
                else q = make_uint2(qf[nt][2 * k + u][0], qf[nt][2 * k + u][1]);
                mma_f16(s[i][nt], hx[2 * u], hy[2 * u], hx[2 * u + 1], hy[2 * u + 1], q.x, q.y);
              }
          }
        }
        // the rows' scales, less 2^12
#pragma unroll
        for (int i = 0; i < kSub; ++i) {
          const uint32_t b0 = lds1(sk + 16 * i + g), b1 = lds1(sk + 16 * i + 8 + g);
          float f0 = __uint_as_float(b0 * 0x800000u - 12u * 0x800000u), f1 = __uint_as_float(b1 * 0x800000u - 12u * 0x800000u);
          if (odd_k) f0 = ue8m0(b0) * 0x1p-12f, f1 = ue8m0(b1) * 0x1p-12f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              s[i][nt][e] *= f0;
              s[i][nt][2 + e] *= f1;
            }
        }
        // ---------------------------------------------- scores, reference
        if (key0 + C::kChunk > vis_min) {
#pragma unroll
          for (int i = 0; i < kSub; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int key = key0 + 16 * i + g, lim = min(vis[nt][e], kend);
                if (key >= lim) s[i][nt][e] = -INFINITY;
                if (key + 8 >= lim) s[i][nt][2 + e] = -INFINITY;
              }
        }
        float top[NT][2];
        bool up = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            top[nt][e] = fmaxf(s[0][nt][e], s[0][nt][2 + e]);
#pragma unroll
            for (int i = 1; i < kSub; ++i) top[nt][e] = fmax3(top[nt][e], s[i][nt][e], s[i][nt][2 + e]);
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
        float neg[NT][2];  // minus the references
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) neg[nt][e] = m[nt][e] == -INFINITY ? 0.f : -m[nt][e];
        // ---------------------------------------------- O^T += V^T P^T
        // One key tile's V: use(mt, a0 .. a3) with channels 2 mt and 2 mt + 1 of this
        // lane's D / 8 as f16 pairs of keys 2t, 2t + 1 (a0, a1) and 2t + 8, 2t + 9
        // (a2, a3), block scales in.
        auto v_tiles = [&](int i, auto use) {
          uint32_t wd[4][D / 64], f[2];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int rk = 2 * t + (k & 1) + 8 * (k >> 1);
            const uint32_t a = vb + (16 * i + rk) * C::kRowB;
            if constexpr (D == 128) {
              const uint2 x = lds8(a + (((g >> 1) ^ C::swap(rk)) << 4) + (g & 1) * 8);
              wd[k][0] = x.x;
              wd[k][1] = x.y;
            } else {
              wd[k][0] = lds4(a + (((g >> 2) ^ C::swap(rk)) << 4) + (g & 3) * 4);
            }
          }
          const uint32_t b = bv + (16 * i + 2 * t) * kBl + (D == 128 ? g : g >> 1);
#pragma unroll
          for (int k = 0; k < 2; ++k) f[k] = e4m3x2_to_f16(lds1(b + 8 * k * kBl) | lds1(b + (8 * k + 1) * kBl) << 8);
#pragma unroll
          for (int x = 0; x < D / 64; ++x) {
            uint32_t hv[4][4];  // even channels of keys 2t, 2t + 1; odd ones; the same of 2t + 8, 2t + 9
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t w0 = wd[2 * k][x], w1 = wd[2 * k + 1][x];
              e2m1x8_to_f16((w0 & 0x0F0F0F0Fu) | ((w1 << 4) & 0xF0F0F0F0u), hv[2 * k]);
              e2m1x8_to_f16(((w0 >> 4) & 0x0F0F0F0Fu) | (w1 & 0xF0F0F0F0u), hv[2 * k + 1]);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
              use(4 * x + q, f16x2_mul(hv[0][q], f[0]), f16x2_mul(hv[1][q], f[0]), f16x2_mul(hv[2][q], f[1]), f16x2_mul(hv[3][q], f[1]));
          }
        };
        if constexpr (!careful) {
          const uint32_t f_ref = (uint32_t)(134 - e_ref) << 23;
          auto add = [&](auto keep) {  // keep: a NaN scale's key stays with the rows that see it
#pragma unroll
            for (int i = 0; i < kSub; ++i) {
              uint32_t hi[NT][2];
              float f[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int b = lds1(sv + 16 * i + 8 * k + g);
                f[k] = __uint_as_float((uint32_t)b * 0x800000u + f_ref);  // b >= e_ref - kSpread
                if (decltype(keep)::value && b == 255) f[k] = __uint_as_float(0x7FC00000u);
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  float y[2];
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    const float x = s[i][nt][2 * k + e];
                    y[e] = ex2_approx(__fmaf_rn(x, cq[nt][e], neg[nt][e]));
                    l[nt][e] += y[e];
                    y[e] = decltype(keep)::value && x == -INFINITY ? 0.f : y[e] * f[k];
                  }
                  hi[nt][k] = transpose8(pack_f16x2(y[0], y[1]));
                }
              v_tiles(i, [&](int mt, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16(o[mt][nt], a0, a1, a2, a3, hi[nt][0], hi[nt][1]);
              });
            }
          };
          if (nan_key) add(std::true_type{});
          else add(std::false_type{});
        } else {
          // V as bf16 values (six significant bits: exact), two bf16 terms a weight
          const float v_unit = e_ref == kCareful ? 1.f : exp2i(-kWideShift);
#pragma unroll 1
          for (int i = 0; i < kSub; ++i) {
            float fv[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) fv[k] = ue8m0(min(lds1(sv + 16 * i + 2 * t + (k & 1) + 8 * (k >> 1)), 254u)) * v_unit;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint32_t ph[2], pl[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const bool nan_row = lds1(sv + 16 * i + 8 * k + g) == 255;
                float y[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  float x = s[0][nt][2 * k + e];
#pragma unroll
                  for (int j = 1; j < kSub; ++j)
                    if (j == i) x = s[j][nt][2 * k + e];
                  y[e] = ex2_approx(__fmaf_rn(x, cq[nt][e], neg[nt][e]));
                  l[nt][e] += y[e];
                  if (nan_row && x != -INFINITY) y[e] = __uint_as_float(0x7FC00000u);
                }
                const uint32_t a = pack_bf16x2(y[0], y[1]);
                ph[k] = transpose8(a);
                pl[k] = transpose8(pack_bf16x2(y[0] - bf16_lo(a), y[1] - bf16_hi(a)));
              }
              v_tiles(i, [&](int mt, uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3) {
                const uint32_t hv[4] = {v0, v1, v2, v3};
                uint32_t a[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  a[k] = pack_bf16x2(f16_lo(hv[k]) * fv[2 * (k >> 1)], f16_hi(hv[k]) * fv[2 * (k >> 1) + 1]);
                mma_bf16(o[mt][nt], a[0], a[1], a[2], a[3], ph[0], ph[1]);
                mma_bf16(o[mt][nt], a[0], a[1], a[2], a[3], pl[0], pl[1]);
              });
            }
          }
        }
        __syncwarp();  // every lane has read the chunk: its place is free
        if (it + kS < n_it) request(it + kS, st);
        copy_commit();
        st = st + 1 == kS ? 0 : st + 1;
      }
      return false;
    };
    if (pass(std::false_type{})) {
      begin();
      pass(std::true_type{});
    }

    // ------------------------------------------------ join the warps
    {  // the accumulators hold 2^(134 - e_ref) times the sum; in two normal factors
      const int shift = e_ref >= kWideByte ? kWideShift : 0, x = e_ref == kCarefulWide ? 0 : e_ref - 134 - shift;
      const float f0 = exp2i(x / 2), f1 = exp2i(x - x / 2), unit = exp2i(-shift);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          m[nt][e] += (float)shift;
          l[nt][e] *= unit;
        }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < C::kMT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][nt][e] = o[i][nt][e] * f0 * f1;
    }
    // (the next tile's first chunks come in meanwhile)
    const ReqRec jq = rq;
    const int jh = h, jblk = blk, jnb = nb;
    const bool more = advance();
    if (C::kEarly && more) {
      ask_q();
      begin();
    }
    join_tile<D, NT, kWarps, false>(p, jq, jh, w, jblk, jnb, jq.per_head - kDecodeTileCost, o, m, l, sm, sml.last,
                                    reinterpret_cast<float*>(&sm));
    if (!more) break;
    if (!C::kEarly) {
      ask_q();
      begin();
    }
  }
}

template <int D, int NT>
cudaError_t launch(const PagedParams& p, cudaStream_t st) {
  using C = Cfg<D, NT>;
  constexpr size_t smem = small_at<D, NT>() + sizeof(Small<D, NT>);
  static_assert(C::kCtas * (smem + 1024) <= 233472, "shared memory of an SM");
  static bool attr_set[64] = {};  // per device: raised once
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(paged_decode4_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  paged_decode4_kernel<D, NT><<<p.W_max[0], C::kThreads, smem, st>>>(p);
  return cudaGetLastError();
}
template <int D>
cudaError_t launch_n(const PagedParams& p, cudaStream_t st) {
  return p.small_rows == 8 ? launch<D, 1>(p, st) : p.small_rows == 16 ? launch<D, 2>(p, st) : launch<D, 4>(p, st);
}

}  // namespace

cudaError_t launch_paged_decode4(const PagedParams& p, int d, cudaStream_t st) {
  return d == 128 ? launch_n<128>(p, st) : launch_n<64>(p, st);
}

}  // namespace flamia
