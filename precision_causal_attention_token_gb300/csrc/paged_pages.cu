// paged_pages.cu — pages that requests share: a step's forks, releases, copies
// on write and new pages (paged_share_kernel), and the compaction of the pool.
//
// Share.  Each page has a count of the table entries (and other holders) that
// hold it.  What a step does follows from the counts as they are once every
// row has been re-pointed: a page whose count has become 0 is free; a request
// that writes into a page with other holders takes a copy of it, but the
// first of them keeps it where all its holders write.  So the counts come
// first, then what hangs on them, then the writes, with a barrier over the
// grid between the three; nothing is written but scratch before the step is
// known to fit.
//   1  per row: +1 for each page taken over from another row (a row's first
//      continuation inherits its entries and costs nothing), -1 for each
//      entry that no row continues; the requests that write into a page
//   2  per row: the pages it was the first to let go of whose count is 0, in
//      table order; whether its partly filled page is copied
//   3  prefix sums over the rows (every CTA forms them alone); tables, counts,
//      stack and the list of copies
// Rows that neither move nor shrink cost no reads of their table.  The data
// are a few words a page, so the launch is bound by its chain of dependent
// steps: 14 us for 64 beams of 16 prompts, 28 us for 800 requests that hold
// 270,000 entries (its own lengths and sources 2 us, the three parts 4 to 5 us
// each where a row has 1,000 entries, a barrier 1.5 us).
//
// Compact.  The pages in use that lie behind the first U ids (U: how many
// there are) move to the free ids before, k-th to k-th: ranks are population
// counts over a bitmap of the free pages.  15 us for 64 requests of 1,100 pages,
// 28 us for 700 with 145,000 of 290,000 in use; four parts of dependent reads,
// three barriers.
#include <climits>

#include "paged_pages.cuh"

namespace flamia {

namespace {

constexpr int kThreads = kPagesThreads;
constexpr int kSpinLimit = 1 << 23;  // polls of 32 ns or more each, but for the first

__device__ __forceinline__ int pages_of(int len, int shift) { return (len + (1 << shift) - 1) >> shift; }

// All CTAs of the launch (they are resident together); `nth` counts a launch's
// barriers from 1.  False, for the whole CTA, where the wait ran out.  A CTA whose
// wait has run out closes the barrier, unless it is complete by then: so either
// every CTA passes it or none does, those that come later included, and what stands
// behind a launch's last barrier happens whole or not at all.
constexpr uint32_t kClosed = 1u << 31;
__device__ bool grid_barrier(const PagesParams& p, uint32_t nth) {
  __shared__ int sm_ok;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    if (!(nth == (uint32_t)p.dbg_withhold && blockIdx.x == 0)) atomicAdd(&p.hdr->arrived, 1u);
    const uint32_t all = nth * gridDim.x;
    int left = kSpinLimit;
    uint32_t seen;
    while (true) {
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(&p.hdr->arrived) : "memory");
      if (seen >= all || --left == 0) break;  // closed: above all counts
      if (left < kSpinLimit - 100) __nanosleep(32);
    }
    while (seen < all) {
      const uint32_t was = atomicCAS(&p.hdr->arrived, seen, seen | kClosed);
      seen = was == seen ? seen | kClosed : was;
    }
    sm_ok = seen < kClosed;
    if (!sm_ok) {  // no page moves, and what follows on the stream has nothing to do
      report(&p.hdr->base, FLAMIA_ERR_TIMEOUT, 0x740);
      p.hdr->fail = FLAMIA_ERR_TIMEOUT;
      if (p.n_free_out) *p.n_free_out = *p.n_free;
      *p.n_copies = 0;
    }
    __threadfence();
  }
  __syncthreads();
  return sm_ok != 0;
}

// Exclusive scan over the CTA's threads; *total: the sum.
template <typename I>
__device__ I block_scan(I v, I* sm, I* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  I x = v;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const I y = __shfl_up_sync(0xffffffffu, x, s);
    if (lane >= s) x += y;
  }
  if (lane == 31) sm[warp] = x;
  __syncthreads();
  if (warp == 0) {
    I w = lane < kThreads / 32 ? sm[lane] : 0;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const I y = __shfl_up_sync(0xffffffffu, w, s);
      if (lane >= s) w += y;
    }
    sm[lane] = w;
  }
  __syncthreads();
  *total = sm[31];
  const I before = warp ? sm[warp - 1] : 0;
  __syncthreads();
  return before + x - v;
}

// What row r of the step is.
struct Row {
  int src, keep, need, write_at;  // write_at: index of the partly filled page it writes into, -1: none
};
__device__ __forceinline__ Row row_of(const PagesParams& p, int r) {
  const int q = p.cu_q[r + 1] - p.cu_q[r], kv = p.kv_len[r], kept = max(0, kv - q);
  Row x;
  x.src = p.src ? p.src[r] : r;
  x.keep = x.src < 0 ? 0 : min(pages_of(p.old_len[x.src], p.page_shift), pages_of(kept, p.page_shift));
  x.need = pages_of(kv, p.page_shift);
  const int at = kept >> p.page_shift;
  x.write_at = q > 0 && (kept & (p.page_size - 1)) && kept < kv && at < x.keep ? at : -1;
  return x;
}
// One of the CTA's own rows (every gridDim.x-th), read once.
struct __align__(16) OwnRow {
  Row row;
  int lost, held;  // the entries that it lets go of: [lost, held)
  int copy, pad;
};

// smem: heir [n], taken [n], given [n + 1], copied [n] and, on a 16-byte border, the CTA's own rows
constexpr size_t share_smem(int n, int ctas) {
  return ((size_t)(4 * n + 1) * 4 + 15) / 16 * 16 + sizeof(OwnRow) * (size_t)((n + ctas - 1) / ctas);
}

__global__ void __launch_bounds__(kThreads, 1) paged_share_kernel(const PagesParams p) {
  extern __shared__ __align__(16) int32_t smi[];
  __shared__ int64_t sm[32];
  __shared__ int sm32[32];
  const int n = p.n_req, mp = p.max_pages, tid = threadIdx.x, sh = p.page_shift;
  int32_t* heir = smi;  // the first row that continues a row; INT_MAX: none
  int32_t* taken = heir + n;
  int32_t* given = taken + n;
  int32_t* copied = given + n + 1;
  OwnRow* own = reinterpret_cast<OwnRow*>(smi + (4 * n + 1 + 3) / 4 * 4);
  const int n_own = (n - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
  const bool first = blockIdx.x == 0;
  // the plan that follows reads its lengths meanwhile and waits for this grid's end
  asm volatile("griddepcontrol.launch_dependents;");

  auto give_up = [&](uint32_t why) {  // no page has moved
    if (first && tid == 0) {
      report(&p.hdr->base, why, 0x741);
      p.hdr->fail = why;
      *p.n_free_out = *p.n_free;
      *p.n_copies = 0;
    }
  };
  // ------------------------------------------------ lengths in, checked; by every CTA alike
  for (int r = tid; r < n; r += kThreads) heir[r] = INT_MAX;
  __syncthreads();
  int bad = 0;
  const int cap = mp << sh;
  if (tid == 0 && (p.cu_q[0] != 0 || p.cu_q[n] < 0 || p.cu_q[n] > p.T)) bad = 1;
  for (int r = tid; r < n; r += kThreads) {
    const int c0 = p.cu_q[r], c1 = p.cu_q[r + 1], kv = p.kv_len[r], old = p.old_len[r], s = p.src ? p.src[r] : r;
    if (c0 < 0 || c1 < c0 || c1 - c0 > p.max_q || kv < 0 || kv > cap || old < 0 || old > cap || s < -1 || s >= n) bad = 1;
    else if (s >= 0) atomicMin(&heir[s], r);
  }
  if (__syncthreads_or(bad)) return give_up(FLAMIA_ERR_BAD_SEQLENS);
  const int n_free = *p.n_free;
  if (n_free < 0 || n_free > p.n_pages) return give_up(FLAMIA_ERR_BAD_PAGE);

  auto page_ok = [&](int id) {
    if ((unsigned)id < (unsigned)p.n_pages) return true;
    atomicOr(&p.hdr->bad, 1u);
    return false;
  };
  for (int j = tid; j < n_own; j += kThreads) {
    const int r = blockIdx.x + j * gridDim.x, h = heir[r];
    OwnRow x;
    x.row = row_of(p, r);
    x.held = pages_of(p.old_len[r], sh);
    x.lost = h == INT_MAX ? 0 : min(x.held, h == r ? x.row.keep : row_of(p, h).keep);
    x.copy = x.pad = 0;
    own[j] = x;
  }
  __syncthreads();
  // ------------------------------------------------ 1: holders gained and lost
  unsigned long long most = 0;  // pages that these rows take at most
  for (int j = 0; j < n_own; ++j) {
    const int r = blockIdx.x + j * gridDim.x;
    const OwnRow& x = own[j];
    const Row& row = x.row;
    most += max(0, row.need - row.keep) + (row.write_at >= 0);
    if (row.src >= 0 && (row.src != r || heir[r] != r)) {
      const int32_t* from = p.block_table + (int64_t)row.src * mp;
      const bool more = heir[row.src] != r;
#pragma unroll 4
      for (int k = tid; k < row.keep; k += kThreads) {
        const int id = from[k];
        if (row.src != r) p.staged[(int64_t)r * mp + k] = id;
        if (page_ok(id) && more) atomicAdd(&p.pages[id].delta, 1);
      }
    }
    if (tid == 0 && row.write_at >= 0) {
      const int id = p.block_table[(int64_t)row.src * mp + row.write_at];
      if (page_ok(id)) {
        atomicAdd(&p.pages[id].writers, 1);
        atomicMax(&p.pages[id].writer, n - r);
      }
    }
#pragma unroll 4
    for (int k = x.lost + tid; k < x.held; k += kThreads) {
      const int id = p.block_table[(int64_t)r * mp + k];
      if (page_ok(id)) {
        atomicAdd(&p.pages[id].delta, -1);
        atomicMax(&p.pages[id].first, INT_MAX - (r * mp + k));
      }
    }
  }
  if (tid == 0 && most) atomicAdd(&p.hdr->most, most);
  if (!grid_barrier(p, 1)) return;
  // ------------------------------------------------ 2: pages without a holder, pages to copy
  if (__ldcg(&p.hdr->bad)) return give_up(FLAMIA_ERR_BAD_PAGE);
  auto rec_of = [&](int id) {
    const int4 v = __ldcg(reinterpret_cast<const int4*>(p.pages + id));
    return PageRec{v.x, v.y, v.z, v.w};
  };
  uint32_t wrong = 0;  // counts that do not cover the tables' entries, free pages outside the pool
  // (how many the step takes is known behind the next barrier)
  const int64_t may_take = min((int64_t)__ldcg(&p.hdr->most), (int64_t)n_free);
  for (int64_t i = (int64_t)blockIdx.x * kThreads + tid; i < may_take; i += (int64_t)gridDim.x * kThreads)
    wrong |= (unsigned)p.free_pages[n_free - 1 - i] >= (unsigned)p.n_pages;
  for (int j = tid; j < n_own; j += kThreads) {
    const Row row = own[j].row;
    if (row.write_at < 0) continue;
    const int r = blockIdx.x + j * gridDim.x, id = p.block_table[(int64_t)row.src * mp + row.write_at];
    const PageRec rec = rec_of(id);
    const int total = p.refs[id] + rec.delta;
    wrong |= total < rec.writers;
    own[j].copy = !(total == rec.writers && rec.writer == n - r);
  }
  __syncthreads();
  for (int j = 0; j < n_own; ++j) {
    const int r = blockIdx.x + j * gridDim.x, x = own[j].lost, y = own[j].held;
    int out = 0;
    constexpr int kPer = 4;  // entries of a thread at a time, in table order
    for (int k0 = x; k0 < y; k0 += kPer * kThreads) {
      int id[kPer], mine = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int k = k0 + kPer * tid + i;
        id[i] = k < y ? p.block_table[(int64_t)r * mp + k] : -1;
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (id[i] < 0) continue;
        const PageRec rec = rec_of(id[i]);
        const int total = p.refs[id[i]] + rec.delta;
        wrong |= total < 0;
        if (total != 0 || rec.first != INT_MAX - (r * mp + k0 + kPer * tid + i)) id[i] = -1;
        mine += id[i] >= 0;
      }
      int all;
      int at = out + block_scan(mine, sm32, &all);
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (id[i] >= 0) p.freed[(int64_t)r * mp + at++] = id[i];
      out += all;
    }
    if (tid == 0) p.counts[r] = make_int4(max(0, own[j].row.need - own[j].row.keep) + own[j].copy, out, own[j].copy, 0);
  }
  if (wrong) atomicOr(&p.hdr->wrong, 1u);
  if (!grid_barrier(p, 2)) return;
  // ------------------------------------------------ 3: where each row's pages come from and go to
  if (__ldcg(&p.hdr->bad) || __ldcg(&p.hdr->wrong)) return give_up(FLAMIA_ERR_BAD_PAGE);
  const int seg = (n + kThreads - 1) / kThreads, r0 = min(n, tid * seg), r1 = min(n, r0 + seg);
  int64_t mine = 0, sum, at;
  int mine_c = 0, n_copied;
  for (int r = r0; r < r1; ++r) {
    const int4 c = __ldcg(p.counts + r);
    mine += ((int64_t)c.x << 32) + c.y;
    mine_c += c.z;
  }
  at = block_scan(mine, sm, &sum);
  int at_c = block_scan(mine_c, sm32, &n_copied);
  for (int r = r0; r < r1; ++r) {
    const int4 c = __ldcg(p.counts + r);
    taken[r] = (int)(at >> 32);
    given[r] = (int)(at & 0xFFFFFFFF);
    copied[r] = at_c;
    at += ((int64_t)c.x << 32) + c.y;
    at_c += c.z;
  }
  const int64_t n_taken = sum >> 32, n_given = sum & 0xFFFFFFFF;
  if (tid == 0) given[n] = (int)n_given;
  __syncthreads();
  if (n_free + n_given > p.n_pages) return give_up(FLAMIA_ERR_BAD_PAGE);
  // (a sum of more than 2^31 entries passes the sign)
  if (n_taken < 0 || n_taken > n_free + n_given) return give_up(FLAMIA_ERR_NO_PAGES);
  const int top = n_free + (int)n_given;
  auto given_page = [&](int j) {  // the j-th page that the step frees
    int lo = 0, hi = n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (given[mid] <= j) lo = mid; else hi = mid - 1;
    }
    return __ldcg(p.freed + (int64_t)lo * mp + (j - given[lo]));
  };
  auto fresh = [&](int i) {  // the i-th page that the step takes
    const int k = top - 1 - i;
    return k < n_free ? p.free_pages[k] : given_page(k - n_free);
  };
  for (int j = 0; j < n_own; ++j) {
    const int r = blockIdx.x + j * gridDim.x;
    int32_t* table = p.block_table + (int64_t)r * mp;
    const Row row = own[j].row;
    const int copy = own[j].copy;
    if (own[j].lost < own[j].held) {  // from the row's table as it was
#pragma unroll 4
      for (int k = own[j].lost + tid; k < own[j].held; k += kThreads) atomicAdd(p.refs + table[k], -1);
      __syncthreads();
    }
    const bool moved = row.src >= 0 && row.src != r, more = row.src >= 0 && heir[row.src] != r;
    if (moved || more || copy) {
#pragma unroll 4
      for (int k = tid; k < row.keep; k += kThreads) {
        const bool mine = copy && k == row.write_at;
        if (!moved && !more && !mine) continue;
        int id = moved ? p.staged[(int64_t)r * mp + k] : table[k];
        if (more) atomicAdd(p.refs + id, 1);
        if (mine) {
          const int to = fresh(taken[r]);
          p.copies[2 * (int64_t)copied[r]] = id;
          p.copies[2 * (int64_t)copied[r] + 1] = to;
          atomicAdd(p.refs + id, -1);
          atomicAdd(p.refs + to, 1);
          id = to;
        }
        if (moved || mine) table[k] = id;
      }
    }
    for (int k = row.keep + tid; k < row.need; k += kThreads) {
      const int id = fresh(taken[r] + copy + k - row.keep);
      table[k] = id;
      atomicAdd(p.refs + id, 1);
    }
  }
  for (int64_t j = (int64_t)blockIdx.x * kThreads + tid; j < n_given - n_taken; j += (int64_t)gridDim.x * kThreads)
    p.free_pages[n_free + j] = given_page((int)j);
  if (first && tid == 0) {
    *p.n_free_out = (int)(top - n_taken);
    *p.n_copies = n_copied;
  }
}

__global__ void __launch_bounds__(kThreads, 1) paged_compact_kernel(const PagesParams p) {
  __shared__ int sm32[32];
  const int n = p.n_req, mp = p.max_pages, tid = threadIdx.x, sh = p.page_shift;
  const bool first = blockIdx.x == 0;
  const int64_t i0 = (int64_t)blockIdx.x * kThreads + tid, step = (int64_t)gridDim.x * kThreads;
  auto give_up = [&](uint32_t why) {
    if (first && tid == 0) {
      report(&p.hdr->base, why, 0x742);
      *p.n_copies = 0;
    }
  };
  int bad = 0;
  const int cap = mp << sh;
  for (int r = tid; r < n; r += kThreads) bad |= p.old_len[r] < 0 || p.old_len[r] > cap;
  // pages of the CTA's own rows (every gridDim.x-th) and of those before each
  extern __shared__ __align__(16) int64_t before_own[];
  const int n_own = (n - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
  for (int j = tid; j < n_own; j += kThreads) before_own[j + 1] = pages_of(max(0, p.old_len[blockIdx.x + j * gridDim.x]), sh);
  if (tid == 0) before_own[0] = 0;
  __syncthreads();
  if (tid == 0)
    for (int j = 0; j < n_own; ++j) before_own[j + 1] += before_own[j];
  // use(entry) for all table entries of these rows, several on their way at a time
  auto entries = [&](auto use) {
    const int64_t all = before_own[n_own];
#pragma unroll 4
    for (int64_t i = tid; i < all; i += kThreads) {
      int lo = 0, hi = n_own - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (before_own[mid] <= i) lo = mid; else hi = mid - 1;
      }
      use(p.block_table + (int64_t)(blockIdx.x + lo * gridDim.x) * mp + (i - before_own[lo]));
    }
  };
  if (__syncthreads_or(bad)) return give_up(FLAMIA_ERR_BAD_SEQLENS);
  const int n_free = *p.n_free;
  if (n_free < 0 || n_free > p.n_pages) return give_up(FLAMIA_ERR_BAD_PAGE);
  const int used = p.n_pages - n_free;  // U
  // ------------------------------------------------ the free pages, each once
#pragma unroll 4
  for (int64_t i = i0; i < n_free; i += step) {
    const int id = p.free_pages[i];
    if ((unsigned)id < (unsigned)p.n_pages) atomicOr(&p.bits[id >> 5], 1u << (id & 31));
    else atomicOr(&p.hdr->bad, 1u);
  }
  if (!grid_barrier(p, 1)) return;
  // ------------------------------------------------ counts; the tables hold no free page
  const int words = (p.n_pages + 31) >> 5, per = (words + gridDim.x - 1) / gridDim.x;
  const int w0 = min(words, (int)blockIdx.x * per), w1 = min(words, w0 + per);
  int mine = 0, all;
  for (int w = w0 + tid; w < w1; w += kThreads) mine += __popc(__ldcg(p.bits + w));
  block_scan(mine, sm32, &all);
  if (tid == 0) p.hdr->count[blockIdx.x] = all;
  int held_free = 0;
  entries([&](const int32_t* at) {
    const int id = *at;
    held_free |= (unsigned)id >= (unsigned)p.n_pages || (__ldcg(p.bits + (id >> 5)) >> (id & 31) & 1u);
  });
  if (held_free) atomicOr(&p.hdr->bad, 1u);
  if (!grid_barrier(p, 2)) return;
  if (__ldcg(&p.hdr->bad)) return give_up(FLAMIA_ERR_BAD_PAGE);
  // ------------------------------------------------ ranks: F(x) = free pages before x
  // before: F of this CTA's first word; below: F(U)
  const int uw = used >> 5, last = uw / max(per, 1);  // U's word and the CTA whose part it is in (or behind all)
  int v = 0, b = 0, c = 0;
  if (tid < gridDim.x) {
    c = (int)__ldcg(&p.hdr->count[tid]);
    if (tid < blockIdx.x) b = c;
    if (tid < last) v = c;
  }
  for (int w = last * per + tid; w <= uw && w < words; w += kThreads) {
    const uint32_t x = __ldcg(p.bits + w);
    v += __popc(w < uw ? x : x & ((1u << (used & 31)) - 1u));
  }
  int before, below, distinct;
  block_scan(c, sm32, &distinct);
  if (distinct != n_free) return give_up(FLAMIA_ERR_BAD_PAGE);  // a page twice on the stack
  block_scan(b, sm32, &before);
  block_scan(v, sm32, &below);
  __shared__ int f_word[kThreads];  // F of a word's first page
  for (int k0 = w0; k0 < w1; k0 += kThreads) {
    const int w = k0 + tid;
    int total;
    f_word[tid] = before + block_scan(w < w1 ? __popc(__ldcg(p.bits + w)) : 0, sm32, &total);
    before += total;
    __syncthreads();
    const int ids = min(32 * min(w1 - k0, kThreads), p.n_pages - 32 * k0);
#pragma unroll 4
    for (int i = tid; i < ids; i += kThreads) {  // a word a warp
      const uint32_t x = __ldcg(p.bits + k0 + (i >> 5));
      const int id = 32 * k0 + i, f = f_word[i >> 5] + __popc(x & ((1u << (i & 31)) - 1u));
      if (x >> (i & 31) & 1u) {
        if (id < used) p.copies[2 * (int64_t)f + 1] = id;
      } else if (id >= used) {
        const int k = (id - used) - (f - below);
        p.copies[2 * (int64_t)k] = id;
        p.rank[id] = k;
      }
    }
    __syncthreads();
  }
  if (!grid_barrier(p, 3)) return;
  // ------------------------------------------------ stack, tables and counts
  if (first && tid == 0) *p.n_copies = below;
  for (int64_t i = i0; i < n_free; i += step) p.free_pages[i] = p.n_pages - 1 - (int)i;
  entries([&](int32_t* at) {
    const int id = *at;
    if (id >= used) *at = __ldcg(p.copies + 2 * (int64_t)__ldcg(p.rank + id) + 1);
  });
  if (p.refs) {
    for (int64_t k = i0; k < below; k += step) {
      const int2 c = __ldcg(reinterpret_cast<const int2*>(p.copies) + k);
      p.refs[c.y] = p.refs[c.x];
      p.refs[c.x] = 0;
    }
  }
}

template <typename K>
cudaError_t launch(K kernel, const PagesParams& p, int ctas, size_t smem, cudaStream_t st) {
  cudaLaunchAttribute together{};
  together.id = cudaLaunchAttributeCooperative;
  together.val.cooperative = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &together;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_paged_share(const PagesParams& p, int sms, cudaStream_t st) {
  int ctas = sms < kMaxPagesCtas ? sms : kMaxPagesCtas;
  if (p.n_req < ctas) ctas = p.n_req;
  const size_t smem = share_smem(p.n_req, ctas);
  static bool attr_set[64] = {};  // per device: raised once
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(paged_share_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)share_smem(kMaxReq, 128));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  e = cudaMemsetAsync(p.hdr, 0, sizeof(PagesHeader) + sizeof(PageRec) * (size_t)p.n_pages, st);
  if (e != cudaSuccess) return e;
  return launch(paged_share_kernel, p, ctas, smem, st);
}

cudaError_t launch_paged_compact(const PagesParams& p, int sms, cudaStream_t st) {
  const size_t words = ((size_t)p.n_pages + 31) / 32;
  cudaError_t e = cudaMemsetAsync(p.hdr, 0, sizeof(PagesHeader) + 4 * words, st);
  if (e != cudaSuccess) return e;
  int64_t ctas = p.n_pages / kThreads + 1;
  if (ctas < p.n_req) ctas = p.n_req;
  if (ctas > sms) ctas = sms;
  if (ctas > kMaxPagesCtas) ctas = kMaxPagesCtas;
  return launch(paged_compact_kernel, p, (int)ctas, sizeof(int64_t) * (size_t)((p.n_req + ctas - 1) / ctas + 1), st);
}

}  // namespace flamia
