// paged_chunk.cu — attention of a chunk of new tokens over a paged cache on
// the tensor cores: S = Q K^T and O += P V as tcgen05 kind::f16 MMAs in bf16
// with fp32 accumulators in tensor memory.
//
// A CTA works on tiles of up to 256 query rows (two halves of up to 128, a
// TMEM lane a row, each of whole tokens) against 128-key blocks of one key/value head: the rows are the
// tokens of the chunk times the G = H / Hkv heads that share that head, so a
// K/V block is fetched once for all of them.  Per block and half the tensor
// cores need 2 x 128 x 128 x d multiply-adds, the softmax 128 x 128
// exponentials; the halves alternate, so one half's products run under the
// other half's softmax.  Warp roles (512 threads, one CTA per SM):
//   warps 0-3, 4-7  softmax of half 0 and 1: a thread owns a row.  It reads
//              the row's 128 scores from tensor memory, masks, moves its
//              reference when a score passes it by 2^8 (then it rescales the
//              row's accumulator), and writes the weights back as bf16 over
//              the scores, from where the P V product reads them as its A
//              operand: P never touches shared memory.
//   warps 8-11 loaders.  E4M3: each block's codes from the raw ring into bf16
//              tiles, times the row's scale (exact).  Both: zeros in rows past
//              the request's last key, where pages hold what an earlier owner
//              left: 0 x NaN is NaN.  For the same reason they take infinities
//              and NaN out of V in the blocks that some row sees in part, and
//              leave word of the first such key, so that the rows that do see
//              it get them back.
//   warp 12    producer: the block's pages, one copy per page and 64 channels
//              (bf16, TMA into the swizzled tile) or one per page (E4M3 codes
//              and scale bytes, into the raw ring).
//   warp 13    MMA issuer.
//   warp 14    scheduler: the worker's tiles (the plan's split).
//   warp 15    the queries of each half, as soon as its last scores of the
//              tile before are formed: one box of G heads x tokens for 64
//              channels, whose rows come in the tile's order whatever G is.
// The row's weights are rounded to bf16 once (2^-8 relative); sums use the
// unrounded ones.
//
// Measured (152 SMs, H = 32, Hkv = 8, d = 128): 2,048 new tokens over 32,768 in
// bf16 720 us (1,575 TFLOP/s; 808 back to back under the power limit), in E4M3
// 850; four times 4,096 from nothing (16 heads each) 231 us in bf16, 294 in
// E4M3.  bf16 is bound by the tensor cores, and by 3 to 4 us between one tile's last
// product and the next one's first; E4M3 by shared memory, which conversion and
// the MMAs' operands share: a step's operands take 1,536 of its 2,048 tensor
// cycles, codes and converted tiles 1,024 more.
#include <climits>

#include "paged.cuh"

namespace flamia {

namespace {

constexpr int kThreads = 512;
constexpr uint32_t kRegSoftmax = 192, kRegLoad = 80, kRegCtl = 48;
static_assert(256 * kRegSoftmax + 128 * kRegLoad + 128 * kRegCtl <= kThreads * 128, "register split");
constexpr int kWarpProd = 12, kWarpMma = 13, kWarpSched = 14, kWarpQ = 15;
constexpr int kFragRing = 2;  // odd_key's eight slots go by it
constexpr int kFragConsumers = 8 + 4 + 3;  // warps that read a fragment
constexpr uint32_t kColS = 0, kColO = 256;     // half h: + 128 h

// One worker's share of one tile.
struct Frag {
  int r, h, tile, kb0;       // first key block
  int n0, n1;                // blocks of each half
  int load;                  // blocks fetched: the larger
  int q0, q_len, kv_len, tok0, toks;
  int whole, starts, w0, parts;  // parts: workers that share the tile
  int end;
};

template <int D, bool FP8>
struct Cfg {
  static constexpr int kTileB = 128 * D * 2;        // bytes of a bf16 tile of 128 rows
  static constexpr int kStages = FP8 ? 3 : 4;       // K/V tiles
  static constexpr int kRaw = FP8 ? 3 : 0;          // raw E4M3 tiles
  static constexpr int kRawB = 128 * D;
};

template <int D, bool FP8>
struct __align__(1024) Tiles {
  uint8_t q[2][Cfg<D, FP8>::kTileB];  // [half][d / 64][128 rows][128 bytes]
  uint8_t kv[Cfg<D, FP8>::kStages][Cfg<D, FP8>::kTileB];
  uint8_t raw[FP8 ? Cfg<D, FP8>::kRaw : 1][FP8 ? Cfg<D, FP8>::kRawB : 1024];
  uint8_t out[8][2048];  // softmax warps: 32 rows x 32 channels of O on their way out
};

struct Ctl {
  uint8_t scales[4][128];  // raw ring: scale bytes
  uint64_t q_full[2], q_empty[2], kv_full[5], kv_empty[5], raw_full[4], raw_empty[4];
  uint64_t s_full[2], p_full[2], o_full[2], fix[5], wg[2];
  uint64_t f_full[kFragRing], f_empty[kFragRing];
  Frag frag[kFragRing];
  int last[2];
  int odd_key[8];  // per fragment (mod 8): the first key whose V was taken out for not being finite
  uint32_t tmem_base;
  int abort_flag;
};

template <int D, bool FP8>
constexpr size_t smem_bytes() { return sizeof(Tiles<D, FP8>) + sizeof(Ctl) + 1024; }

// D[tmem] (+)= A[smem] * B[smem], bf16, fp32 accumulate.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// A from tensor memory: row m at lane m, two bf16 a column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// S[half] = Q[half] K^T: both K-major, 128-byte swizzled rows of 64 channels.
template <int D>
__device__ __forceinline__ void issue_s(uint32_t d, const uint8_t* q, const uint8_t* k) {
  const uint32_t qa = smem_u32(q), ka = smem_u32(k);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = (kk / 4) * 128 * 128 + (kk % 4) * 32;
    mma_ss(d, smem_desc(qa + off, 16, 1024, kSwz128), smem_desc(ka + off, 16, 1024, kSwz128), bf16_idesc(128, 128, 0, 0), kk > 0);
  }
}
// O[half] += P[half] V: P in tensor memory, V's rows are keys (MN-major B):
// 64 channels a 128-byte row, the next 64 channels 16 KB on (leading
// offset), the next 8 keys 1 KB on (stride offset).
template <int D>
__device__ __forceinline__ void issue_pv(uint32_t d, uint32_t pcol, const uint8_t* v, bool acc) {
  const uint32_t va = smem_u32(v);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    mma_ts(d, pcol + 8 * kk, smem_desc(va + kk * 16 * 128, 128 * 128, 1024, kSwz128), bf16_idesc(128, D, 0, 1), acc || kk > 0);
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads, 1)
    paged_chunk_kernel(const PagedParams p, const __grid_constant__ CUtensorMap map_q,
                       const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  using C = Cfg<D, FP8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_base_1k(smem_raw);
  Tiles<D, FP8>& tl = *reinterpret_cast<Tiles<D, FP8>*>(base);
  Ctl& c = *reinterpret_cast<Ctl*>(base + sizeof(Tiles<D, FP8>));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  WsHeader* hdr = &p.hdr->base;
  volatile int* abort_flag = &c.abort_flag;
  // Launched while the decode kernel of the same call may still run (other
  // rows, other partials): what follows on the stream waits for this grid, so
  // this grid ends after that one.
  auto wait_for_decode = [] { asm volatile("griddepcontrol.wait;" ::: "memory"); };
  const WorkerRec* rec_at = p.workers + kMaxWorkers + blockIdx.x;
  const int places = rec_at->n;  // on its way while the signature is
  if (!planned(p) || places == 0) {
    wait_for_decode();
    return;
  }

  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&c.q_full[s], 1);
      mbar_init(&c.q_empty[s], 1);
    }
    for (int s = 0; s < 5; ++s) {
      mbar_init(&c.kv_full[s], FP8 ? 128 : 1);
      mbar_init(&c.kv_empty[s], FP8 ? 1 : 1 + 4);  // the MMA issuer; bf16: also the loader warps
      mbar_init(&c.fix[s], 128);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&c.raw_full[s], 1);
      mbar_init(&c.raw_empty[s], 128);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&c.s_full[s], 1);
      mbar_init(&c.p_full[s], 128);
      mbar_init(&c.o_full[s], 1);
      mbar_init(&c.wg[s], 128);
    }
    for (int s = 0; s < 8; ++s) c.odd_key[s] = INT_MAX;
    for (int s = 0; s < kFragRing; ++s) {
      mbar_init(&c.f_full[s], 1);
      mbar_init(&c.f_empty[s], kFragConsumers);
    }
    c.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) tmem_alloc(&c.tmem_base, 512);
  if (warp == kWarpQ && lane == 0) prefetch_tensormap(&map_q);
  if (!FP8 && warp == kWarpProd && lane == 0) {
    prefetch_tensormap(&map_k);
    prefetch_tensormap(&map_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = c.tmem_base;
  // Keys from here on are not seen by every row of the tile: V's tiles from
  // this one's block on go through the loaders.
  auto seen_by_all = [&](const Frag& f) { return min(f.kv_len, visible_keys(p.causal, f.q_len, f.kv_len, f.tok0)); };
  // a warp's next fragment (lane 0 frees the slot once all lanes have read it)
  auto next_frag = [&](uint32_t n, Frag& f, bool& ok, uint32_t where) {
    const int s = n % kFragRing;
    if (!(ok = mbar_wait_warp(&c.f_full[s], (n / kFragRing) & 1, abort_flag, hdr, where))) return false;
    f = c.frag[s];
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.f_empty[s]);
    return !f.end;
  };

  if (warp >= 12) {
    setmaxnreg_dec<kRegCtl>();
    if (warp == kWarpSched && lane == 0) {
      // ------------------------------------------------------------ scheduler
      const WorkerRec rec = *rec_at;
      ReqRec rq = rec.q;
      int left = rec.n, at = rec.at, h = rec.h, tile = rec.tile, pos = rec.pos, off = rec.tile_off;
      bool ok = true;
      uint32_t n = 0;
      while (true) {
        const int s = n % kFragRing;
        if (!(ok = mbar_wait(&c.f_empty[s], ((n / kFragRing) & 1) ^ 1, abort_flag, hdr, 0x801))) break;
        Frag& f = c.frag[s];
        const int tok0 = tile * 2 * p.half_toks, toks = min(2 * p.half_toks, rq.q_len - tok0);
        int nb[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int last = min(toks, (hf + 1) * p.half_toks) - 1;  // last token of the half
          nb[hf] = hf * p.half_toks < toks
                       ? (visible_keys(p.causal, rq.q_len, rq.kv_len, tok0 + last) + kChunkBlk - 1) / kChunkBlk : 0;
        }
        // the worker's part: blocks [blk, blk + nblk) behind the tile's own cost
        const int all = max(1, max(nb[0], nb[1])), take = min(left, kChunkTileCost + all - pos);
        const int blk = max(0, pos - kChunkTileCost), nblk = max(0, pos + take - kChunkTileCost) - blk;
        f.r = rq.r;
        f.h = h;
        f.tile = tile;
        f.kb0 = blk;
        f.n0 = max(0, min(nb[0], blk + nblk) - blk);
        f.n1 = max(0, min(nb[1], blk + nblk) - blk);
        f.load = max(f.n0, f.n1);
        f.q0 = rq.q0;
        f.q_len = rq.q_len;
        f.kv_len = rq.kv_len;
        f.tok0 = tok0;
        f.toks = toks;
        f.whole = nblk == all;
        f.starts = blk == 0;
        f.w0 = f.parts = 0;
        if (!f.whole) {
          const int64_t cost = p.hdr->cost[1], x = rq.base + (int64_t)h * rq.per_head + off + kChunkTileCost;
          const int W = p.hdr->workers[1];
          f.w0 = worker_of(x, cost, W);
          f.parts = worker_of(x + all - 1, cost, W) - f.w0 + 1;
        }
        f.end = 0;
        if (nblk > 0) {
          mbar_arrive(&c.f_full[s]);
          ++n;
        }
        left -= take;
        if (left == 0) break;
        pos = 0;
        off += kChunkTileCost + all;
        if (++tile == rq.tiles) {
          tile = off = 0;
          if (++h == p.Hkv) {
            h = 0;
            rq = p.reqs[p.n_req + ++at];
          }
        }
      }
      if (ok) {  // no more
        const int s = n % kFragRing;
        if (mbar_wait(&c.f_empty[s], ((n / kFragRing) & 1) ^ 1, abort_flag, hdr, 0x815)) {
          c.frag[s].end = 1;
          mbar_arrive(&c.f_full[s]);
        }
      }
    } else if (warp == kWarpProd) {
      // ------------------------------------------------------------ producer
      uint32_t it = 0;
      bool ok = true;
      Frag f;
      for (uint32_t n = 0; ok && next_frag(n, f, ok, 0x802); ++n) {
        const int ps = p.page_size, per = kChunkBlk >> p.page_shift;  // pages of a block (<= 8)
        const int32_t* table = p.block_table + (int64_t)f.r * p.max_pages;
        const int pages = (f.kv_len + ps - 1) >> p.page_shift;
        auto page_at = [&](int blk) {
          const int k = blk * per + lane;
          int id = lane < per && k < pages ? __ldg(table + k) : 0;
          if ((unsigned)id >= (unsigned)p.n_pages) {
            report(hdr, FLAMIA_ERR_BAD_PAGE, 0x822);
            id = 0;
          }
          return id;
        };
        int id = f.load ? page_at(f.kb0) : 0;
        for (int b = 0; ok && b < f.load; ++b) {
          const int blk = f.kb0 + b;
          const int id_next = b + 1 < f.load ? page_at(blk + 1) : 0;
          const int np = min(per, pages - blk * per);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++it) {
            if constexpr (FP8) {
              const int s = it % C::kRaw;
              if (!(ok = mbar_wait_warp(&c.raw_empty[s], ((it / C::kRaw) & 1) ^ 1, abort_flag, hdr, 0x803))) break;
              if (lane == 0) mbar_arrive_expect_tx(&c.raw_full[s], np * ps * (D + 1));
              __syncwarp();
              if (lane < np) {
                bulk_load(tl.raw[s] + lane * ps * D, (kv ? p.v : p.k) + id * p.page_bytes + (int64_t)f.h * ps * D, ps * D,
                          &c.raw_full[s]);
                bulk_load(c.scales[s] + lane * ps, (kv ? p.v_scales : p.k_scales) + ((int64_t)id * p.Hkv + f.h) * ps, ps,
                          &c.raw_full[s]);
              }
            } else {
              const int s = it % C::kStages;
              if (!(ok = mbar_wait_warp(&c.kv_empty[s], ((it / C::kStages) & 1) ^ 1, abort_flag, hdr, 0x804))) break;
              if (lane == 0) mbar_arrive_expect_tx(&c.kv_full[s], np * ps * D * 2);
              __syncwarp();
              if (lane < np) {
#pragma unroll
                for (int j = 0; j < D / 64; ++j)
                  tma_load_4d(tl.kv[s] + j * 128 * 128 + lane * ps * 128, kv ? &map_v : &map_k, &c.kv_full[s], 64 * j, 0, f.h,
                              id);
              }
            }
          }
          id = id_next;
        }
      }
    } else if (warp == kWarpQ) {
      // ------------------------------------------------------------ queries
      uint32_t uses[2] = {0, 0};
      bool ok = true;
      Frag f;
      for (uint32_t n = 0; ok && next_frag(n, f, ok, 0x816); ++n) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          if (!ok || (hf ? f.n1 : f.n0) == 0) continue;
          ok = mbar_wait_warp(&c.q_empty[hf], (uses[hf] & 1) ^ 1, abort_flag, hdr, 0x80b);
          if (!ok) continue;
          ++uses[hf];
          if (lane == 0) {  // a half's whole box: rows past the tile's last are not its own and not written
            mbar_arrive_expect_tx(&c.q_full[hf], p.half_toks * p.G * D * 2);
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
              tma_load_3d(tl.q[hf] + j * 128 * 128, &map_q, &c.q_full[hf], 64 * j, f.h * p.G, f.q0 + f.tok0 + hf * p.half_toks);
          }
          __syncwarp();
        }
      }
    } else if (warp == kWarpMma) {
      // ------------------------------------------------------------ MMA issuer
      uint32_t it = 0, pc[2] = {0, 0}, qc[2] = {0, 0}, fixed = 0;  // fixed: phase bits of fix[]
      bool ok = true;
      const uint32_t elected = elect_one();
      Frag f;
      for (uint32_t n = 0; ok && next_frag(n, f, ok, 0x805); ++n) {
        const int nh[2] = {f.n0, f.n1};
        const int all_see = seen_by_all(f);
        // one thread waits and issues; the warp stays together at the fragment's end
        if (elected) {
          do {
            auto full = [&](uint32_t i) {
              return mbar_wait(&c.kv_full[i % C::kStages], (i / C::kStages) & 1, abort_flag, hdr, 0x807);
            };
            if (f.load) {
              if (!(ok = full(it))) break;
#pragma unroll
              for (int hf = 0; hf < 2; ++hf)
                if (ok && nh[hf]) {
                  ok = mbar_wait(&c.q_full[hf], qc[hf] & 1, abort_flag, hdr, 0x806);
                  if (!ok) continue;
                  ++qc[hf];
                  tc_fence_after();
                  issue_s<D>(tb + kColS + 128 * hf, tl.q[hf], tl.kv[it % C::kStages]);
                  tc_commit(&c.s_full[hf]);
                  if (nh[hf] == 1) tc_commit(&c.q_empty[hf]);
                }
              if (!ok) break;
              tc_commit(&c.kv_empty[it % C::kStages]);
            }
            for (int b = 0; ok && b < f.load; ++b) {
              const uint32_t vi = it + 2 * b + 1, ki = vi + 1;
              const uint8_t* vt = tl.kv[vi % C::kStages];
              const uint8_t* kt = tl.kv[ki % C::kStages];
              const bool more = b + 1 < f.load;
              if (!(ok = full(vi))) break;
              if (!FP8 && (f.kb0 + b + 1) * kChunkBlk > all_see) {
                const uint32_t s = vi % C::kStages;
                if (!(ok = mbar_wait(&c.fix[s], (fixed >> s) & 1, abort_flag, hdr, 0x808))) break;
                fixed ^= 1u << s;
              }
              bool k_in = false;
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                if (ok && b < nh[hf]) {
                  ok = mbar_wait(&c.p_full[hf], pc[hf] & 1, abort_flag, hdr, 0x809);
                  if (!ok) continue;
                  ++pc[hf];
                  tc_fence_after();
                  issue_pv<D>(tb + kColO + 128 * hf, tb + kColS + 128 * hf, vt, b > 0);
                  if (b + 1 == nh[hf]) tc_commit(&c.o_full[hf]);
                }
                if (ok && b + 1 < nh[hf]) {
                  if (!k_in) {
                    ok = full(ki);
                    if (!ok) continue;
                    k_in = true;
                    tc_fence_after();
                  }
                  issue_s<D>(tb + kColS + 128 * hf, tl.q[hf], kt);
                  tc_commit(&c.s_full[hf]);
                  // the queries are free once the last block's scores are formed
                  if (b + 2 == nh[hf]) tc_commit(&c.q_empty[hf]);
                }
              }
              if (!ok) break;
              tc_commit(&c.kv_empty[vi % C::kStages]);
              if (more) tc_commit(&c.kv_empty[ki % C::kStages]);
            }
            if (!ok) break;
            it += 2 * f.load;
          } while (false);
        }
        ok = __all_sync(0xffffffffu, ok);
      }
    }
  } else if (warp >= 8) {
    setmaxnreg_dec<kRegLoad>();
    // -------------------------------------------------------------- loaders
    const int lt = tid - 256;
    uint32_t it = 0;
    bool ok = true;
    Frag f;
    for (uint32_t n = 0; ok && next_frag(n, f, ok, 0x80a); ++n) {
      // Clear the slot of the fragment four on.  Its last user, four back, is
      // done: this fragment is published once every softmax warp has taken the
      // one two back (the fragment ring), having finished the one before.  And
      // no loader warp is at the one four on before this one has gone on.
      if (lt == 0) c.odd_key[(n + 4) % 8] = INT_MAX;
      int* odd_key = &c.odd_key[n % 8];
      if constexpr (FP8) {
        for (int b = 0; ok && b < 2 * f.load; ++b, ++it) {
          const int rs = it % C::kRaw, s = it % C::kStages;
          const int keys = f.kv_len - (f.kb0 + b / 2) * kChunkBlk;  // rows from here on are cleared
          if (!(ok = mbar_wait_warp(&c.raw_full[rs], (it / C::kRaw) & 1, abort_flag, hdr, 0x80c))) break;
          if (!(ok = mbar_wait_warp(&c.kv_empty[s], ((it / C::kStages) & 1) ^ 1, abort_flag, hdr, 0x80d))) break;
          // A thread takes the same 16 channels of every kStep-th row: its place
          // in the swizzle (row mod 8) stays.  The upper 64 channels' lanes
          // write their two 16-byte chunks in the other order: the two
          // 64-channel columns share their banks.
          constexpr int kRawCh = D / 16, kStep = 128 / kRawCh, kBatch = kRawCh;
          const int ch = lt % kRawCh, row0 = lt / kRawCh;
          const int flip = (ch >> 2) & 1;
          const uint8_t* src = tl.raw[rs] + row0 * D + ch * 16;
          uint8_t* dst = tl.kv[s] + (ch / 4) * 128 * 128 + row0 * 128;
          const uint32_t at0 = (((2 * ch) & 7) ^ (row0 & 7)) << 4, at1 = at0 ^ 16;
          auto convert = [](const uint4& x, uint32_t f, uint32_t (&y)[8]) {
            const uint32_t wd[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              y[2 * k] = bf16x2_mul(e4m3_to_bf16x2(prmt(wd[k], 0u, 0x4140u)), f);
              y[2 * k + 1] = bf16x2_mul(e4m3_to_bf16x2(prmt(wd[k], 0u, 0x4342u)), f);
            }
          };
          auto put = [&](int i, const uint32_t (&y)[8]) {
            const uint4 lo = make_uint4(y[0], y[1], y[2], y[3]), hi = make_uint4(y[4], y[5], y[6], y[7]);
            uint8_t* d = dst + i * kStep * 128;
            *reinterpret_cast<uint4*>(d + (flip ? at1 : at0)) = flip ? hi : lo;
            *reinterpret_cast<uint4*>(d + (flip ? at0 : at1)) = flip ? lo : hi;
          };
          uint32_t sb[kRawCh];
          bool plain = keys >= kChunkBlk;
#pragma unroll
          for (int i = 0; i < kRawCh; ++i) {
            sb[i] = c.scales[rs][row0 + i * kStep];
            plain = plain && sb[i] <= 134u;
          }
          if (__all_sync(0xffffffffu, plain)) {
#pragma unroll
            for (int i0 = 0; i0 < kRawCh; i0 += kBatch) {
              uint4 x[kBatch];
#pragma unroll
              for (int i = 0; i < kBatch; ++i) x[i] = *reinterpret_cast<const uint4*>(src + (i0 + i) * kStep * D);
#pragma unroll
              for (int i = 0; i < kBatch; ++i) {
                uint32_t y[8];
                // 2^120 undoes the conversion's bias: (byte + 120) << 7 in both halves
                convert(x[i], sb[i0 + i] * 0x00800080u + 120u * 0x00800080u, y);
                put(i0 + i, y);
              }
            }
          } else {
#pragma unroll 1
            for (int i = 0; i < kRawCh; ++i) {
              const int row = row0 + i * kStep;
              const uint32_t sc = c.scales[rs][row];
              uint32_t y[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) y[k] = 0u;
              if (row < keys) {
                if (sc != 255u) {  // a scale above 2^7: in two factors
                  convert(*reinterpret_cast<const uint4*>(src + i * kStep * D), min(sc, 134u) * 0x00800080u + 120u * 0x00800080u, y);
                  const uint32_t f2 = ((max(sc, 134u) - 134u + 127u) << 7) * 0x10001u;
#pragma unroll
                  for (int k = 0; k < 8; ++k) y[k] = bf16x2_mul(y[k], f2);
                } else if (b & 1) {
                  atomicMin(odd_key, (f.kb0 + b / 2) * kChunkBlk + row);
                } else {
#pragma unroll
                  for (int k = 0; k < 8; ++k) y[k] = 0x7FC07FC0u;
                }
              }
              put(i, y);
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(&c.kv_full[s]);
          mbar_arrive(&c.raw_empty[rs]);
        }
      } else {
        // The loaders go through every tile, so that their waits never fall a
        // ring's turn behind (a parity wait would then pass or stay wrongly):
        // a stage is filled anew only when they have passed it too.
        const int all_see = seen_by_all(f);
        for (int i2 = 0; i2 < 2 * f.load; ++i2, ++it) {
          const int s = it % C::kStages, key0 = (f.kb0 + i2 / 2) * kChunkBlk, keys = f.kv_len - key0;
          if (!(ok = mbar_wait_warp(&c.kv_full[s], (it / C::kStages) & 1, abort_flag, hdr, 0x80e))) break;
          if (!(i2 & 1) || key0 + kChunkBlk <= all_see) {  // K, or V that every row sees
            if (lane == 0) mbar_arrive(&c.kv_empty[s]);
            continue;
          }
#pragma unroll 4
          for (int i = lt; i < 128 * (D / 8); i += 128) {
            const int row = i / (D / 8), ch = i % (D / 8);
            uint4* at = reinterpret_cast<uint4*>(tl.kv[s] + (ch / 8) * 128 * 128 + sw128_off(row, ch % 8));
            if (row >= keys) {
              *at = make_uint4(0, 0, 0, 0);
            } else {
              uint4 x = *at;
              uint32_t* wd = &x.x;
              // an exponent field of ones carries into the sign's place
              uint32_t odd = 0;
#pragma unroll
              for (int k = 0; k < 4; ++k) odd |= ((wd[k] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
              if (odd) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  if ((wd[k] & 0x7F80u) == 0x7F80u) wd[k] &= 0xFFFF0000u;
                  if ((wd[k] & 0x7F800000u) == 0x7F800000u) wd[k] &= 0xFFFFu;
                }
                *at = x;
                atomicMin(odd_key, key0 + row);
              }
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(&c.fix[s]);
          __syncwarp();
          if (lane == 0) mbar_arrive(&c.kv_empty[s]);
        }
      }
    }
  } else {
    setmaxnreg_inc<kRegSoftmax>();
    // -------------------------------------------------------------- softmax
    const int hf = warp >> 2, row = tid & 127;
    const uint32_t ts = taddr(tb, (warp & 3) * 32, kColS + 128 * hf), to = taddr(tb, (warp & 3) * 32, kColO + 128 * hf);
    uint32_t sc = 0, oc = 0, wgc = 0;
    bool ok = true;
    Frag f;
    for (uint32_t n = 0; ok && next_frag(n, f, ok, 0x810); ++n) {
      const int R = 128 * hf + row;
      if (hf * p.half_toks >= f.toks) continue;  // the half is empty
      const int n_blk = hf ? f.n1 : f.n0;
      const int tok = hf * p.half_toks + row / p.G, hq = f.h * p.G + row % p.G;
      const bool row_ok = row < p.half_toks * p.G && tok < f.toks;
      const int vis = row_ok ? min(f.kv_len, visible_keys(p.causal, f.q_len, f.kv_len, f.tok0 + tok)) : f.kv_len;
      const int vis_min = __reduce_min_sync(0xffffffffu, vis);
      float m = -INFINITY, l = 0.f;
      for (int b = 0; ok && b < n_blk; ++b, ++sc) {
        if (!(ok = mbar_wait_warp(&c.s_full[hf], sc & 1, abort_flag, hdr, 0x811))) break;
        tc_fence_after();
        const int key0 = (f.kb0 + b) * kChunkBlk, nv = vis - key0;
        const bool masked = key0 + kChunkBlk > vis_min;
        if (FP8 && masked) {
          // through tensor memory, a quarter at a time: a fourth of the code.
          // The E4M3 kernel's roles fill the instruction cache (4 x 4,096: 312
          // against 298 us); bf16 is better off in registers.
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            uint32_t x[32];
            tmem_ld32(ts + 32 * q, x);
            tmem_ld_wait_regs(x);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (32 * q + j >= nv) x[j] = 0xFF800000u;
            tmem_st32(ts + 32 * q, x);
          }
          tmem_st_wait();
        }
        uint32_t s0[32], s1[32], s2[32], s3[32];
        tmem_ld32(ts, s0);
        tmem_ld32(ts + 32, s1);
        tmem_ld32(ts + 64, s2);
        tmem_ld32(ts + 96, s3);
        tmem_ld_wait_regs(s0, s1);
        tmem_ld_wait_regs(s2, s3);
        if (!FP8 && masked) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            if (j >= nv) s0[j] = 0xFF800000u;
            if (32 + j >= nv) s1[j] = 0xFF800000u;
            if (64 + j >= nv) s2[j] = 0xFF800000u;
            if (96 + j >= nv) s3[j] = 0xFF800000u;
          }
        }
        float t0 = -INFINITY, t1 = -INFINITY, t2 = -INFINITY, t3 = -INFINITY;
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          t0 = fmax3(t0, __uint_as_float(s0[j]), __uint_as_float(s0[j + 1]));
          t1 = fmax3(t1, __uint_as_float(s1[j]), __uint_as_float(s1[j + 1]));
          t2 = fmax3(t2, __uint_as_float(s2[j]), __uint_as_float(s2[j + 1]));
          t3 = fmax3(t3, __uint_as_float(s3[j]), __uint_as_float(s3[j + 1]));
        }
        const float top = fmaxf(fmax3(t0, t1, t2), t3) * p.c_log2;
        const bool up = top > m + 8.f;
        if (__any_sync(0xffffffffu, up)) {
          const float a = up ? ex2_approx(m - top) : 1.f;  // 0 from an empty reference
          if (up) m = top;
          l *= a;
          if (b > 0) {  // s_full follows this half's previous P V
            // 16 columns at a time: the 128 scores stay in registers meanwhile
            // (32 at a time spill, and the whole kernel takes twice as long)
#pragma unroll 1
            for (int j = 0; j < D / 16; ++j) {
              uint32_t o[16];
              tmem_ld16(to + 16 * j, o);
              tmem_ld_wait_regs(o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
              tmem_st16(to + 16 * j, o);
            }
          }
        }
        const float mref = m == -INFINITY ? 0.f : m;
        const uint64_t c2 = f2_pack(p.c_log2, p.c_log2), m2 = f2_pack(-mref, -mref);
        uint64_t sum0 = 0, sum1 = 0;
        auto weights = [&](uint32_t (&x)[32], uint32_t* out) {
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            float a0, a1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), c2, m2), a0, a1);
            a0 = ex2_approx(a0);
            a1 = ex2_approx(a1);
            if (j & 2) sum1 = f2_add(sum1, f2_pack(a0, a1));
            else sum0 = f2_add(sum0, f2_pack(a0, a1));
            out[j / 2] = pack_bf16x2(a0, a1);
          }
        };
        uint32_t w0[32];
        weights(s0, w0);
        weights(s1, w0 + 16);
        tmem_st32(ts, w0);
        uint32_t w1[32];
        weights(s2, w1);
        weights(s3, w1 + 16);
        tmem_st32(ts + 32, w1);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&c.p_full[hf]);
        float u0, u1, u2, u3;
        f2_unpack(sum0, u0, u1);
        f2_unpack(sum1, u2, u3);
        l += (u0 + u1) + (u2 + u3);
      }
      if (!ok) break;
      // ------------------------------------------------------------ the rows' results
      // 32 channels at a time: out of tensor memory, then to the workspace or
      // through a small shared-memory square to O in 64-byte pieces (a row's
      // 16 bytes a store, 128 rows side by side, took 3 us a tile)
      if (n_blk) {
        if (!(ok = mbar_wait_warp(&c.o_full[hf], oc & 1, abort_flag, hdr, 0x812))) break;
        ++oc;
        tc_fence_after();
      }
      // infinities and NaN that the loaders took out of V: a weight is above 0
      const int odd = f.load ? *reinterpret_cast<volatile int*>(&c.odd_key[n % 8]) : INT_MAX;
      const int odd_end = min(vis, (f.kb0 + n_blk) * kChunkBlk);
      auto piece = [&](int j, float (&v)[32]) {
        if (n_blk) {
          uint32_t o[32];
          tmem_ld32(to + 32 * j, o);
          tmem_ld_wait_regs(o);
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(o[k]);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = 0.f;
        }
        if (odd < odd_end) {
          if constexpr (FP8) {  // a whole row
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(0x7FC00000u);
          } else {
#pragma unroll 1
            for (int key = odd; key < odd_end; ++key) {
              const int id = __ldg(p.block_table + (int64_t)f.r * p.max_pages + (key >> p.page_shift));
              if ((unsigned)id >= (unsigned)p.n_pages) continue;
              const uint4* src = reinterpret_cast<const uint4*>(p.v + id * p.page_bytes +
                                                                (((int64_t)f.h * p.page_size + (key & (p.page_size - 1))) * D + 32 * j) * 2);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint4 x = __ldg(src + k);
                const uint32_t wd[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if ((wd[e] & 0x7F80u) == 0x7F80u) v[8 * k + 2 * e] += bf16_lo(wd[e]);
                  if ((wd[e] & 0x7F800000u) == 0x7F800000u) v[8 * k + 2 * e + 1] += bf16_hi(wd[e]);
                }
              }
            }
          }
        }
      };
      const int64_t t_row = f.q0 + f.tok0 + tok, my_out = row_ok ? (t_row * p.H + hq) * D : -1;
      uint8_t* sq = tl.out[warp];
      int64_t out_at[4];  // of the rows that this lane stores a piece of
#pragma unroll
      for (int i = 0; i < 4; ++i) out_at[i] = __shfl_sync(0xffffffffu, my_out, 8 * i + (lane >> 2));
      // row r of the square: 16-byte piece k at (k ^ (r / 2) % 4)
      auto emit = [&](int j, const float (&v)[32], float inv) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<uint4*>(sq + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)) =
              make_uint4(pack_bf16x2(v[8 * k] * inv, v[8 * k + 1] * inv), pack_bf16x2(v[8 * k + 2] * inv, v[8 * k + 3] * inv),
                         pack_bf16x2(v[8 * k + 4] * inv, v[8 * k + 5] * inv), pack_bf16x2(v[8 * k + 6] * inv, v[8 * k + 7] * inv));
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 8 * i + (lane >> 2), k = lane & 3;
          const uint4 x = *reinterpret_cast<const uint4*>(sq + r * 64 + ((k ^ ((r >> 1) & 3)) << 4));
          if (out_at[i] >= 0) *reinterpret_cast<uint4*>(p.O + out_at[i] + 32 * j + 8 * k) = x;
        }
        __syncwarp();
      };
      auto inverse = [](float x) { return x > 0.f ? 1.f / x : (x == 0.f ? 0.f : x); };  // a NaN sum stays
      const int64_t slot = f.starts ? 2 * (int)blockIdx.x + 1 : 2 * (int)blockIdx.x;
      const float inv_l = inverse(l);
#pragma unroll 1  // unrolled, the code outgrows the instruction cache (E4M3 4 x 4,096: 310 -> 367 us)
      for (int j = 0; j < D / 32; ++j) {
        float v[32];
        piece(j, v);
        if (f.whole) {
          emit(j, v, inv_l);
        } else if (row_ok) {
          float4* po = reinterpret_cast<float4*>(p.chunk_o) + (slot * (D / 4) + 8 * j) * kChunkRows + R;
#pragma unroll
          for (int k = 0; k < 8; ++k) __stcg(po + k * kChunkRows, make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]));
        }
      }
      tc_fence_before();
      if (f.whole) {
        if (row_ok && p.lse) p.lse[(int64_t)hq * p.T + t_row] = (m + lg2_f(l)) * 0.69314718055994531f;
        continue;
      }
      if (row_ok) __stcg(p.chunk_ml + slot * kChunkRows + R, make_float2(m, l));
      mbar_arrive(&c.wg[hf]);
      if (!(ok = mbar_wait_warp(&c.wg[hf], wgc & 1, abort_flag, hdr, 0x813))) break;
      ++wgc;
      unsigned int* ctr = &p.hdr->count_chunk[2 * f.w0 + hf];
      if (row == 0) {
        __threadfence();  // after the barrier: for the whole half
        const bool last = atomicAdd(ctr, 1u) == (unsigned)(f.parts - 1);
        if (last) *ctr = 0;
        __threadfence();
        c.last[hf] = last;
      }
      mbar_arrive(&c.wg[hf]);
      if (!(ok = mbar_wait_warp(&c.wg[hf], wgc & 1, abort_flag, hdr, 0x814))) break;
      ++wgc;
      if (*reinterpret_cast<volatile int*>(&c.last[hf]) == 0) continue;
      // the last of the tile's workers adds the partials up, in worker order
      auto slot_of = [&](int i) { return (int64_t)(i == 0 ? 2 * f.w0 + 1 : 2 * (f.w0 + i)); };
      const float2* ml = p.chunk_ml + R;
      m = -INFINITY;
      l = 0.f;
      if (row_ok) {
#pragma unroll 8
        for (int i = 0; i < f.parts; ++i) m = fmaxf(m, __ldcg(ml + slot_of(i) * kChunkRows).x);
#pragma unroll 8
        for (int i = 0; i < f.parts; ++i) {
          const float2 x = __ldcg(ml + slot_of(i) * kChunkRows);
          l += (x.x == m ? 1.f : ex2_approx(x.x - m)) * x.y;
        }
      }
      const float inv = inverse(l);
#pragma unroll 1
      for (int j = 0; j < D / 32; ++j) {
        float v[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = 0.f;
        if (row_ok) {
#pragma unroll 2
          for (int i = 0; i < f.parts; ++i) {
            const float x = __ldcg(ml + slot_of(i) * kChunkRows).x, a = x == m ? 1.f : ex2_approx(x - m);
            const float4* src = reinterpret_cast<const float4*>(p.chunk_o) + (slot_of(i) * (D / 4) + 8 * j) * kChunkRows + R;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float4 y = __ldcg(src + k * kChunkRows);
              v[4 * k] += a * y.x;
              v[4 * k + 1] += a * y.y;
              v[4 * k + 2] += a * y.z;
              v[4 * k + 3] += a * y.w;
            }
          }
        }
        emit(j, v, inv);
      }
      if (row_ok && p.lse) p.lse[(int64_t)hq * p.T + t_row] = (m + lg2_f(l)) * 0.69314718055994531f;
    }
  }
  __syncwarp();  // single-thread roles rejoin their warp
  tc_fence_before();
  __syncthreads();
  drain_after_abort(abort_flag);
  if (warp == kWarpMma) tmem_dealloc(tb, 512);
  wait_for_decode();
}

template <int D, bool FP8>
cudaError_t launch(const PagedParams& p, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t st) {
  constexpr size_t smem = smem_bytes<D, FP8>();
  static_assert(smem <= 232448, "shared memory");
  using T = Tiles<D, FP8>;
  static_assert(offsetof(T, kv) % 1024 == 0 && offsetof(T, raw) % 1024 == 0 && offsetof(T, out) % 1024 == 0, "tile alignment");
  static bool attr_set[64] = {};  // per device: raised once
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(paged_chunk_kernel<D, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.W_max[1]);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = p.small_rows ? 1 : 0;  // a decode kernel came before
  return cudaLaunchKernelEx(&cfg, paged_chunk_kernel<D, FP8>, p, mq, mk, mv);
}

}  // namespace

cudaError_t launch_paged_chunk(const PagedParams& p, int d, bool e4m3, const CUtensorMap& mq, const CUtensorMap& mk,
                               const CUtensorMap& mv, cudaStream_t st) {
  if (d == 128) return e4m3 ? launch<128, true>(p, mq, mk, mv, st) : launch<128, false>(p, mq, mk, mv, st);
  return e4m3 ? launch<64, true>(p, mq, mk, mv, st) : launch<64, false>(p, mq, mk, mv, st);
}

}  // namespace flamia
