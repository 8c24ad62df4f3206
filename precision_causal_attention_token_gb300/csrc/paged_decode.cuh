// paged_decode.cuh — what the decode kernels share (paged_decode.cu: bf16 and
// E4M3 caches, paged_decode4.cu: E2M1): the small MMAs, and the join of a
// tile's warps and of its workers.
#pragma once
#include "paged.cuh"

namespace flamia {

constexpr int kSpread = 12;  // binades between V rows that f16 weights serve

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

// The warps' results of a tile, in shared memory.
template <int D, int NT, int kWarps>
struct Join {
  float o[kWarps][8 * NT][D + 4];
  float m[kWarps][8 * NT], l[kWarps][8 * NT];
};

// After a tile's last key: the warps' accumulators (o: channel tiles in rows,
// query rows in columns; kWide: a lane's channels in two runs of eight) are
// added up, and the tile's result goes to O and lse, or, where the tile is
// shared, to the workspace, from where the last of its workers adds the
// partials up in worker order.  `sm` and `wt_buf` (the partials' weights) may lie
// in the place of the warps' rings only if no copy into these is in flight: a kernel
// that asks for its next tile's chunks before the join has them elsewhere.
template <int D, int NT, int kWarps, bool kWide>
__device__ __forceinline__ void join_tile(const PagedParams& p, const ReqRec& rq, int h, int w, int blk, int nb, int blocks,
                                          const float (&o)[D / 16][NT][4], const float (&m)[NT][2], const float (&l)[NT][2],
                                          Join<D, NT, kWarps>& sm, int& sm_last, float* wt_buf) {
  constexpr int kMT = D / 16, kQ = 8 * NT;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int rows = rq.q_len * p.G;
  PagedHeader* hdr = p.hdr;
  __syncthreads();  // every warp is done with its ring's chunks of this tile
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
      for (int i = 0; i < kMT; i += 2) {
        // two channel tiles: four channels in a row
        const int d = kWide ? (i / 4) * 64 + g * 8 + (i % 4) * 2 : (D / 8) * g + 2 * i;
        *reinterpret_cast<float4*>(&sm.o[warp][c][d]) =
            make_float4(o[i][nt][e], o[i][nt][2 + e], o[i + 1][nt][e], o[i + 1][nt][2 + e]);
      }
    }
  __syncthreads();
  const bool whole = nb == blocks;
  constexpr int kRowThreads = 128;             // the first four warps add up the rows
  constexpr int kSpan = kRowThreads / kQ;      // threads of a query row (16, 8 or 4)
  constexpr int kPer = D / kSpan;              // channels of a thread
  const int row = tid / kSpan, d0 = (tid % kSpan) * kPer;
  const bool mine = kWarps == 4 || tid < kRowThreads;
  float M = -INFINITY, L = 0.f, acc[kPer];
  if (mine) {
    M = sm.m[0][row];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) M = fmaxf(M, sm.m[i][row]);
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
  }
  bool write = whole;
  if (!whole) {
    const int64_t cost = hdr->cost[0], tile0 = rq.base + (int64_t)h * rq.per_head;
    const int W = hdr->workers[0];
    const int w0 = worker_of(tile0 + kDecodeTileCost, cost, W), n = worker_of(tile0 + rq.per_head - 1, cost, W) - w0 + 1;
    const int slot = blk == 0 ? 2 * w + 1 : 2 * w;
    float* po = p.part_o + ((int64_t)slot * kQ + row) * D + d0;
    if (mine) {
#pragma unroll
      for (int k = 0; k < kPer; k += 4)
        __stcg(reinterpret_cast<float4*>(po + k), make_float4(acc[k], acc[k + 1], acc[k + 2], acc[k + 3]));
    }
    if (mine && d0 == 0) __stcg(p.part_ml + (int64_t)slot * kQ + row, make_float2(M, L));
    __syncthreads();
    if (tid == 0) {
      __threadfence();  // after the barrier: for the whole CTA
      const bool last = atomicAdd(&hdr->count[w0], 1u) == (unsigned)(n - 1);
      if (last) hdr->count[w0] = 0;
      sm_last = last;
    }
    __syncthreads();
    write = sm_last;
    if (write && mine) {
      // A row's threads form the partials' weights together, then add up
      // their channels, eight partials in flight (one after the other, 57 of
      // them took 20 us).
      __threadfence();
      auto slot_of = [&](int i) { return (int64_t)(i == 0 ? 2 * w0 + 1 : 2 * (w0 + i)); };
      float* wt = wt_buf;  // [n][kQ]; the join's buffers are free
      const int me = tid % kSpan;
      constexpr int kOwn = 4;  // a thread's first partials are read once
      float2 own[kOwn];
#pragma unroll
      for (int j = 0; j < kOwn; ++j) {
        const int i = me + j * kSpan;
        own[j] = i < n ? __ldcg(p.part_ml + slot_of(i) * kQ + row) : make_float2(-INFINITY, 0.f);
      }
      M = -INFINITY;
#pragma unroll
      for (int j = 0; j < kOwn; ++j) M = fmaxf(M, own[j].x);
      for (int i = me + kOwn * kSpan; i < n; i += kSpan) M = fmaxf(M, __ldcg(p.part_ml + slot_of(i) * kQ + row).x);
#pragma unroll
      for (int k = kSpan / 2; k; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
      L = 0.f;
      auto weigh = [&](int i, float2 x) {
        const float a = x.x == M ? 1.f : ex2_approx(x.x - M);
        L += a * x.y;
        wt[i * kQ + row] = a;
      };
#pragma unroll
      for (int j = 0; j < kOwn; ++j)
        if (me + j * kSpan < n) weigh(me + j * kSpan, own[j]);
      for (int i = me + kOwn * kSpan; i < n; i += kSpan) weigh(i, __ldcg(p.part_ml + slot_of(i) * kQ + row));
#pragma unroll
      for (int k = kSpan / 2; k; k >>= 1) L += __shfl_xor_sync(0xffffffffu, L, k);
      __syncwarp();
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
#pragma unroll (kPer <= 16 ? 8 : 2)
      for (int i = 0; i < n; ++i) {
        const float a = wt[i * kQ + row];
        const float* src = p.part_o + (slot_of(i) * kQ + row) * D + d0;
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
  if (write && mine && row < rows) {
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

}  // namespace flamia
