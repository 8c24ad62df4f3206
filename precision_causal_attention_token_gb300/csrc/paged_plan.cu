// paged_plan.cu — one serving step's pages, slots and attention work split,
// built on the GPU from the request lengths in one launch.
//
// Three prefix sums over the requests (pages taken, pages given back, blocks
// of attention work) fix everything else, and they are small, so every CTA
// forms the first two in its own shared memory and nothing is passed between
// CTAs: page k of the step is the k-th from the end of the free stack, which
// is a page the step gives back or a word of free_pages, so each thread can
// tell any new token's page by itself, before the table entry is written.
// CTA 0 forms the work split; the others share the table entries and slots.
// The launch moves a few bytes per request and token and is bound by its
// chain of dependent steps (loads, scan, search, store), not by bandwidth:
// 6.4 us for 64 requests of one new token each, 13.5 us for 1,094 requests with
// 105,413 (CTA 0's split; the searches by warps instead of threads took 26 us).
#include "paged.cuh"

namespace flamia {

namespace {

constexpr int kPlanThreads = 512;

__device__ __forceinline__ int pages_of(int len, int shift) { return (len + (1 << shift) - 1) >> shift; }

// Exclusive scan of one 64-bit value per thread; *total: the sum.
__device__ int64_t block_scan(int64_t v, int64_t* sm, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, s);
    if (lane >= s) x += y;
  }
  if (lane == 31) sm[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int64_t w = lane < kPlanThreads / 32 ? sm[lane] : 0;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, w, s);
      if (lane >= s) w += y;
    }
    sm[lane] = w;
  }
  __syncthreads();
  *total = sm[31];
  const int64_t before = warp ? sm[warp - 1] : 0;
  __syncthreads();
  return before + x - v;
}

// The request r with pre[r] <= i < pre[r + 1] (pre[0] = 0 <= i < pre[n]).
template <typename I>
__device__ __forceinline__ int find(const I* pre, int n, int64_t i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= i) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Quotient of non-negative numbers: in 32 bits where they fit (a 64-bit
// division is a hundred instructions).
__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// The line of a request with new tokens.
__device__ __forceinline__ int line_of(const PagedParams& p, int q_len) { return (int64_t)q_len * p.G > p.small_rows; }
__device__ __forceinline__ int tiles_of(const PagedParams& p, int q_len) {
  return line_of(p, q_len) ? (q_len + 2 * p.half_toks - 1) / (2 * p.half_toks) : q_len > 0;
}
// Places of one tile.
__device__ __forceinline__ int tile_places(const PagedParams& p, int line, int q_len, int kv_len, int tile) {
  if (!line) return kDecodeTileCost + max(1, (kv_len + kDecodeBlk - 1) / kDecodeBlk);
  const int last = min(q_len, (tile + 1) * 2 * p.half_toks) - 1;
  return kChunkTileCost + max(1, (visible_keys(p.causal, q_len, kv_len, last) + kChunkBlk - 1) / kChunkBlk);
}

// Whether the step passes the limits of places, with a request's tiles all
// taken as its longest (the last): every CTA of the launch finds the same,
// before any page moves.
__device__ bool too_large(const PagedParams& p, const int32_t* cu, int r0, int r1, int64_t* sm) {
  int64_t mine[2] = {0, 0}, all[2];
  int big = 0;
  for (int r = r0; r < r1; ++r) {
    const int ql = cu[r + 1] - cu[r], line = line_of(p, ql), nt = tiles_of(p, ql);
    if (nt == 0) continue;
    const int64_t head = (int64_t)nt * tile_places(p, line, ql, p.kv_len[r], nt - 1);
    big |= head > kMaxHeadPlaces;
    mine[line] += min(min(head, kMaxHeadPlaces) * p.Hkv, kMaxPlaces + 1);  // below 2^62; n_req of them below 2^52
  }
  block_scan(mine[0], sm, &all[0]);
  block_scan(mine[1], sm, &all[1]);
  return __syncthreads_or(big) || all[0] > kMaxPlaces || all[1] > kMaxPlaces;
}

__device__ void no_work(const PagedParams& p) {
  for (int w = threadIdx.x; w < kMaxWorkers + kMaxChunkWorkers; w += kPlanThreads) p.workers[w] = WorkerRec{};
}

// The work split (one CTA): the requests of each line with their places, and
// where each worker starts.  smem: per [n] places of a head, pre [n + 2] first
// places, rid [n + 2] the requests; line 0 from entry 0, line 1 behind it,
// each with an end entry.
__device__ void split_work(const PagedParams& p, const int32_t* cu, int64_t* per, int64_t* pre, int32_t* rid, int64_t* sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = p.n_req;
  constexpr int kSerial = 4;  // tiles that a thread adds up alone; longer chunks take a warp
  __shared__ int n_long;
  if (tid == 0) n_long = 0;
  __syncthreads();
  for (int r = tid; r < n; r += kPlanThreads) {
    const int ql = cu[r + 1] - cu[r], kv = p.kv_len[r], nt = tiles_of(p, ql), line = line_of(p, ql);
    int64_t sum = 0;
    if (nt <= kSerial) {
      for (int i = 0; i < nt; ++i) sum += tile_places(p, line, ql, kv, i);
      per[r] = sum;
    } else {
      rid[atomicAdd(&n_long, 1)] = r;
    }
  }
  __syncthreads();
  for (int k = warp; k < n_long; k += kPlanThreads / 32) {
    const int r = rid[k], ql = cu[r + 1] - cu[r], kv = p.kv_len[r], nt = tiles_of(p, ql);
    int64_t sum = 0;
    for (int i = lane; i < nt; i += 32) sum += tile_places(p, 1, ql, kv, i);
#pragma unroll
    for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
    if (lane == 0) per[r] = sum;
  }
  __syncthreads();
  const int seg = (n + kPlanThreads - 1) / kPlanThreads, r0 = min(n, tid * seg), r1 = min(n, r0 + seg);
  int64_t cnt = 0, mine[2] = {0, 0}, cost[2], all;
  for (int r = r0; r < r1; ++r) {
    const int ql = cu[r + 1] - cu[r];
    if (ql == 0) continue;
    const int line = line_of(p, ql);
    cnt += line ? (int64_t)1 << 32 : 1;
    mine[line] += per[r] * p.Hkv;
  }
  const int64_t at = block_scan(cnt, sm, &all);
  const int n0 = (int)(all & 0xFFFFFFFF), n1 = (int)(all >> 32);
  int64_t place[2] = {block_scan(mine[0], sm, &cost[0]), block_scan(mine[1], sm, &cost[1])};
  int idx[2] = {(int)(at & 0xFFFFFFFF), (int)(at >> 32)};
  for (int r = r0; r < r1; ++r) {
    const int ql = cu[r + 1] - cu[r];
    if (ql == 0) continue;
    const int line = line_of(p, ql);
    ReqRec q;
    q.r = r;
    q.q0 = cu[r];
    q.q_len = ql;
    q.kv_len = p.kv_len[r];
    q.base = place[line];
    q.per_head = (int)per[r];
    q.tiles = tiles_of(p, ql);
    p.reqs[(int64_t)line * n + idx[line]] = q;
    const int e = line * (n0 + 1) + idx[line];
    pre[e] = place[line];
    rid[e] = r;
    place[line] += per[r] * p.Hkv;
    ++idx[line];
  }
  if (tid == 0) {
    pre[n0] = cost[0];
    pre[n0 + 1 + n1] = cost[1];
  }
  __syncthreads();
  for (int line = 0; line < 2; ++line) {
    const int64_t* lp = pre + line * (n0 + 1);
    const int32_t* lr = rid + line * (n0 + 1);
    const int nl = line ? n1 : n0;
    const int64_t c = cost[line];
    // Fewer workers than fit the GPU where a share would be too small to pay
    // for joining its partial results.
    const int64_t share = line ? kChunkTileCost + 2 : kDecodeTileCost + 3;
    const int W = (int)max((int64_t)(c > 0), min((int64_t)p.W_max[line], quot(c, share)));
    if (tid == 0) {
      p.hdr->cost[line] = c;
      p.hdr->workers[line] = W;
    }
    WorkerRec* out = p.workers + (line ? kMaxWorkers : 0);
    auto start_of = [&](int w, int64_t& y) {  // the worker's request and its place there
      WorkerRec rec{};
      const int64_t x0 = quot(c * w, W), x1 = quot(c * (w + 1), W);
      const int i = find(lp, nl, x0), r = lr[i];
      rec.q.r = r;
      rec.q.q0 = cu[r];
      rec.q.q_len = cu[r + 1] - cu[r];
      rec.q.kv_len = p.kv_len[r];
      rec.q.base = lp[i];
      rec.q.per_head = (int)per[r];
      rec.q.tiles = tiles_of(p, rec.q.q_len);
      rec.at = i;
      rec.n = (int)(x1 - x0);
      y = x0 - lp[i];
      rec.h = (int)quot(y, rec.q.per_head);
      y -= (int64_t)rec.h * rec.q.per_head;
      return rec;
    };
    for (int w = tid; w < p.W_max[line]; w += kPlanThreads) {
      WorkerRec rec{};
      if (w < W) {
        int64_t y;
        rec = start_of(w, y);
        rec.pos = (int)y;  // of the head, which is a tile in line 0
      }
      out[w] = rec;
    }
    if (!line) continue;
    // line 1: the tile that holds the place, 32 tiles at a time
    __syncthreads();
    for (int w = warp; w < W; w += kPlanThreads / 32) {
      const int ql = out[w].q.q_len, kv = out[w].q.kv_len, nt = out[w].q.tiles, z = out[w].pos;
      if (nt == 1) continue;
      int off = 0;
      for (int t0 = 0; t0 < nt; t0 += 32) {
        const int nb = t0 + lane < nt ? tile_places(p, 1, ql, kv, t0 + lane) : 0;
        int incl = nb;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, incl, s);
          if (lane >= s) incl += o;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, off + incl > z);
        if (hit) {
          if (lane == __ffs(hit) - 1) {
            out[w].tile = t0 + lane;
            out[w].tile_off = off + incl - nb;
            out[w].pos = z - (off + incl - nb);
          }
          break;
        }
        off += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
  }
}

// smem: cu [n + 1], then CTA 0: per [n], pre [n + 2], rid [n + 2]; the others:
// taken [n + 1], given [n + 1]
constexpr size_t plan_smem(int n) { return (size_t)(n + 2) * 24; }

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PagedParams p) {
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ int64_t sm[32];
  const int n = p.n_req, tid = threadIdx.x, sh = p.page_shift;
  int64_t* per = reinterpret_cast<int64_t*>(raw);
  int64_t* pre = per + n;
  int32_t* rid = reinterpret_cast<int32_t*>(pre + n + 2);
  int32_t* cu = rid + n + 2;
  int32_t* taken = reinterpret_cast<int32_t*>(raw);
  int32_t* given = taken + n + 1;
  const bool manage = p.old_len != nullptr;
  const bool first = blockIdx.x == 0;

  if (first) {
    if (tid == 0) {
      p.hdr->base.status = 0;
      p.hdr->base.status_where = 0;
      p.hdr->signature = p.signature;
    }
    for (int i = tid; i < kMaxWorkers; i += kPlanThreads) p.hdr->count[i] = 0;
    for (int i = tid; i < 2 * kMaxChunkWorkers; i += kPlanThreads) p.hdr->count_chunk[i] = 0;
  }
  // lengths in, checked
  int bad = 0;
  for (int i = tid; i <= n; i += kPlanThreads) cu[i] = p.cu_q[i];
  __syncthreads();
  const int seg = (n + kPlanThreads - 1) / kPlanThreads, r0 = min(n, tid * seg), r1 = min(n, r0 + seg);
  if (tid == 0 && (cu[0] != 0 || cu[n] < 0 || cu[n] > p.T)) bad = 1;
  const int cap = p.max_pages << sh;
  int64_t mine = 0;
  for (int r = r0; r < r1; ++r) {
    const int ql = cu[r + 1] - cu[r], kv = p.kv_len[r], old = manage ? p.old_len[r] : 0;
    if (cu[r + 1] < cu[r] || cu[r] < 0 || ql > p.max_q || kv < 0 || kv > cap || old < 0 || old > cap) {
      bad = 1;
    } else if (manage) {
      const int d = pages_of(kv, sh) - pages_of(old, sh);
      mine += d > 0 ? (int64_t)d << 32 : (int64_t)-d;
    }
  }
  bad = __syncthreads_or(bad);
  uint32_t why = bad ? FLAMIA_ERR_BAD_SEQLENS : FLAMIA_OK;
  int n_free = 0, n_taken = 0, n_given = 0;
  if (manage && !bad) {
    n_free = *p.n_free;
    int64_t sum;
    int64_t at = block_scan(mine, sm, &sum);
    n_taken = (int)(sum >> 32);
    n_given = (int)(sum & 0xFFFFFFFF);
    for (int r = r0; !first && r < r1; ++r) {
      taken[r] = (int)(at >> 32);
      given[r] = (int)(at & 0xFFFFFFFF);
      const int d = pages_of(p.kv_len[r], sh) - pages_of(p.old_len[r], sh);
      at += d > 0 ? (int64_t)d << 32 : (int64_t)-d;
    }
    if (!first && tid == 0) {
      taken[n] = n_taken;
      given[n] = n_given;
    }
    if (n_free < 0 || n_free > p.n_pages || (int64_t)n_free + n_given > p.n_pages) why = FLAMIA_ERR_BAD_PAGE;
    else if (n_taken > n_free + n_given) why = FLAMIA_ERR_NO_PAGES;
  }
  if (p.count_places && !why && too_large(p, cu, r0, r1, sm)) why = FLAMIA_ERR_UNSUPPORTED;
  __syncthreads();
  const int top = n_free + n_given;
  if (first) {
    if (tid == 0) {
      if (manage) *p.n_free_out = why ? *p.n_free : top - n_taken;
      if (why) report(&p.hdr->base, why, 0x700);
      p.hdr->rows = why ? 0 : cu[n];
    }
    if (!why) {
      split_work(p, cu, per, pre, rid, sm);
    } else {  // no worker has work
      no_work(p);
    }
    return;
  }
  const int i0 = ((int)blockIdx.x - 1) * kPlanThreads + tid, step = ((int)gridDim.x - 1) * kPlanThreads;
  if (why) {
    if (p.slot_map)
      for (int t = i0; t < p.T; t += step) p.slot_map[t] = -1;
    return;
  }
  // page k counted from the bottom of the stack S
  auto given_page = [&](int j) {
    const int r = find(given, n, j);
    return p.block_table[(int64_t)r * p.max_pages + pages_of(p.kv_len[r], sh) + (j - given[r])];
  };
  auto stack_at = [&](int k) { return k < n_free ? p.free_pages[k] : given_page(k - n_free); };
  if (manage) {
    for (int i = i0; i < n_taken; i += step) {
      const int r = find(taken, n, i);
      p.block_table[(int64_t)r * p.max_pages + pages_of(p.old_len[r], sh) + (i - taken[r])] = stack_at(top - 1 - i);
    }
    for (int j = i0; j < n_given - n_taken; j += step) p.free_pages[n_free + j] = given_page(j);
  }
  if (!p.slot_map) return;
  for (int t = i0; t < p.T; t += step) {
    int slot = -1;
    if (t < cu[n]) {
      const int r = find(cu, n, t);
      const int pos = p.kv_len[r] - (cu[r + 1] - t);
      if (pos >= 0) {
        const int k = pos >> sh, had = manage ? pages_of(p.old_len[r], sh) : 0;
        const int page = manage && k >= had ? stack_at(top - 1 - (taken[r] + k - had))
                                            : p.block_table[(int64_t)r * p.max_pages + k];
        // -2: the append kernel reports it (a report from here could come
        // before CTA 0 clears the status word)
        slot = (unsigned)page < (unsigned)p.n_pages ? (page << sh) + (pos & (p.page_size - 1)) : -2;
      }
    }
    p.slot_map[t] = slot;
  }
}

}  // namespace

cudaError_t launch_paged_plan(const PagedParams& p, cudaStream_t st) {
  const size_t smem = plan_smem(p.n_req);
  static bool attr_set[64] = {};  // per device: raised once
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)plan_smem(kMaxReq));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  int helpers = 0;
  if (p.slot_map || p.old_len) {
    helpers = (p.T + kPlanThreads - 1) / kPlanThreads;
    if (p.old_len && helpers < (p.n_req + 31) / 32) helpers = (p.n_req + 31) / 32;
    helpers = helpers < 1 ? 1 : helpers > 151 ? 151 : helpers;
  }
  paged_plan_kernel<<<1 + helpers, kPlanThreads, smem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace flamia
