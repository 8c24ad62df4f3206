// paged.cuh — what the paged-cache kernels share: parameters, workspace
// layout, the split of the attention's work, fp8 -> 16-bit conversions.
#pragma once
#include "common.cuh"

namespace flamia {

// ---------------------------------------------------------------------------
// The split of the attention's work.  A tile is up to `rows` query rows (token
// major, the G = H/Hkv query heads of a key/value head side by side) of one
// request and one key/value head; its keys are visited in blocks of `blk`.
// All blocks of all tiles in the order (request, head, tile, block) form a
// line, on which every tile also takes kTileCost places before its first
// block for what a tile costs beside them, and worker w (a CTA) takes the
// places [floor(cost w / W), floor(cost (w + 1) / W)).  So the work is even
// whatever the lengths, a long context is split over as many SMs as there
// are, and a worker leaves at most two unfinished tiles, whose partial results
// (fp32) go to its two slots of the workspace: slot 2w for a tile that an
// earlier worker began, 2w + 1 for one that it begins itself.  The last worker
// of a tile to finish adds the partials up in worker order, so the result does
// not depend on who is last.
//
// Requests with few rows (one new token, a few drafted ones) are served by
// the decode kernel, the others by the chunk kernel: two lines.
// ---------------------------------------------------------------------------
// What the cache holds.
enum { kCacheBF16 = 0, kCacheE4M3 = 1, kCacheE2M1 = 2 };
enum { kPathDecode8 = 0, kPathDecode16 = 1, kPathDecode32 = 2, kPathChunk = 3 };
constexpr int kDecodeBlk = 64, kChunkBlk = 128, kChunkRows = 256;
// What a tile costs beside its blocks, in blocks: its queries, first loads and
// result (decode: 5 us of about 1 us a block)
constexpr int kDecodeTileCost = 5, kChunkTileCost = 2;
constexpr int kMaxWorkers = 512, kMaxChunkWorkers = 160;
constexpr int kMaxReq = 8192;
// Keys of a request in a call with chunks: 2^18 blocks of a tile at 1.2 to 4 us
// each stay below the limit of the chunk kernel's waits, whose longest is for
// a tile's end.
constexpr int kMaxChunkKeys = 1 << 25;
// Places of a head's tiles of one request and of a line, at most: positions
// within a head's tiles and a worker's share (kMaxPlaces over 128 or more
// workers) are 32-bit.
constexpr int64_t kMaxHeadPlaces = INT32_MAX, kMaxPlaces = (int64_t)1 << 38;

struct PagedHeader {
  WsHeader base;       // status words first, as flamia_get_device_status reads them
  int64_t cost[2];     // places of each line (0: decode, 1: chunk)
  int32_t workers[2];  // W of each line
  int32_t rows;        // cu_q[n_req], 0 after an inconsistent plan
  int32_t n_free_new;  // for a plan whose n_free and n_free_out are one word
  int32_t pad[2];
  uint64_t signature;  // of the problem that was planned
  int32_t pad2[4];
  unsigned int count[kMaxWorkers];              // decode: partials written, per tile (by its first worker)
  unsigned int count_chunk[2 * kMaxChunkWorkers];  // chunk: also by half
};

// A request of one line.
struct __align__(16) ReqRec {
  int32_t r, q0, q_len, kv_len;
  int64_t base;      // its first place
  int32_t per_head;  // places of one head's tiles
  int32_t tiles;     // of a head
};
// Where a worker starts: everything that its first tile needs, in one read.
struct __align__(16) WorkerRec {
  ReqRec q;
  int32_t at;        // the request's index in the line's list
  int32_t h, tile;
  int32_t pos;       // place within the tile
  int32_t n;         // the worker's places (0: none)
  int32_t tile_off;  // places of the head's earlier tiles
  int32_t pad[2];
};
static_assert(sizeof(ReqRec) == 32 && sizeof(WorkerRec) == 64, "read in 16-byte pieces");

struct PagedLayout {
  size_t header, reqs, workers, part_ml, part_o, chunk_ml, chunk_o, total;
  int path;
};

struct PagedParams {
  uint64_t signature;  // of what the plan depends on
  int n_req, T, max_q, H, Hkv, G, page_size, page_shift, n_pages, max_pages, causal, path;
  int W_max[2];   // workers at most, of each line
  int small_rows; // requests of up to so many rows go to the decode kernel (8, 16, 32; 0: none)
  int half_toks;  // tokens of a tile's half (chunk kernel): 128 / G
  int count_places;  // sizes at which the plan may pass the limits of places
  float c_log2;   // softmax_scale * log2(e)
  const int32_t* cu_q;
  const int32_t* kv_len;
  int32_t* block_table;
  int64_t q_stride, kv_stride;  // elements
  PagedHeader* hdr;
  ReqRec* reqs;        // [2][n_req]
  WorkerRec* workers;  // [kMaxWorkers], [kMaxChunkWorkers]
  float2* part_ml;     // decode: [2 W][rows] (reference, sum)
  float* part_o;       // [2 W][rows][d]
  float2* chunk_ml;    // chunk: [2 W][256]
  float* chunk_o;      // [2 W][d / 4][256][4]
  // plan
  int32_t* slot_map;
  const int32_t* old_len;
  int32_t* free_pages;
  const int32_t* n_free;
  int32_t* n_free_out;
  const uint32_t* before;  // status of the page management that ran before in the same call (NULL: none)
  // append, forward
  const void* k_new;
  const void* v_new;
  const int32_t* slots;
  const __nv_bfloat16* q;
  uint8_t* k;
  uint8_t* v;
  uint8_t* k_scales;
  uint8_t* v_scales;
  uint8_t* k_blocks;  // E2M1: block scales
  uint8_t* v_blocks;
  int64_t page_bytes;  // between pages of k (and of v)
  __nv_bfloat16* O;
  float* lse;
};

cudaError_t launch_paged_plan(const PagedParams& p, cudaStream_t st);
cudaError_t launch_paged_append(const PagedParams& p, int d, int cache, bool in_bf16, int sms, cudaStream_t st);
cudaError_t launch_paged_decode(const PagedParams& p, int d, int cache, cudaStream_t st);
cudaError_t launch_paged_decode4(const PagedParams& p, int d, cudaStream_t st);
cudaError_t launch_paged_chunk(const PagedParams& p, int d, int cache, const CUtensorMap& mq, const CUtensorMap& mk,
                               const CUtensorMap& mv, cudaStream_t st);
// Workers of a launch on a GPU with `sms` SMs: what the kernel keeps resident.
int paged_decode_workers(int sms);

// Keys that the rows of tokens [.., tok] of a request see (tok: its last token).
__host__ __device__ __forceinline__ int visible_keys(int causal, int q_len, int kv_len, int tok) {
  if (!causal) return kv_len;
  const int n = kv_len - q_len + tok + 1;
  return n < 0 ? 0 : n;
}

// Whether the workspace holds a plan of this problem: a launch on any other
// (never planned, or planned for other sizes) reads nothing more and reports.
__device__ __forceinline__ bool planned(const PagedParams& p) {
  if (p.hdr->signature == p.signature) return true;
  report(&p.hdr->base, FLAMIA_ERR_INVALID_ARG, 0x730);
  return false;
}

// Worker that owns block x of a line of `cost` blocks split over W.
__device__ __forceinline__ int worker_of(int64_t x, int64_t cost, int W) { return (int)(((x + 1) * W - 1) / cost); }

// 2^(b - 127) for a UE8M0 byte: b = 0 is subnormal, 255 is NaN.
__device__ __forceinline__ float ue8m0(uint32_t b) {
  return __uint_as_float(b == 0u ? 0x00400000u : b == 255u ? 0x7FC00000u : b << 23);
}

// Two E4M3 codes in bits 0-7 and 16-23 of `t` (the other bits zero) -> bf16x2
// values times 2^-120: exponent and mantissa move to bits 4-10 of their half,
// the low end of bf16's exponent field, where they keep their meaning,
// subnormal codes included, with the bias 127 in place of 7; the sign moves
// from bit 7 to bit 15 (16 * 128 + 240 * 128 = 2^15).  The caller multiplies by
// 2^120 times the row's scale, which is exact for every code.  Multiply-adds,
// because logic runs at half their rate (shift and mask: 876 us against 854 for
// 2,048 tokens over 32,768).
__device__ __forceinline__ uint32_t e4m3_to_bf16x2(uint32_t t) { return t * 16u + (t & 0x00800080u) * 240u; }
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Infinities become bf16's largest numbers: E4M3 rows hold values of 2^128 (255 *
// 2^120, bf16's largest number, rounds to 256 * 2^120), and 0 x inf is NaN.
__device__ __forceinline__ uint32_t bf16x2_finite(uint32_t a) {
  uint32_t r;
  asm("min.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(0x7F7F7F7Fu));
  return r;
}
// Two fp32 -> bf16x2 (RNE), `lo` in the low half.
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// Two fp32 -> f16x2 (RNE), `lo` in the low half.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Eight E2M1 codes -> four f16 pairs, exact: pair b from byte b, its low nibble in the low half.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}
// Two E4M3 codes in bits 0-15 -> f16 pair, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The larger of each half.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

// Instruction descriptor, kind::f16 (bf16 x bf16 -> fp32): c_format (4-5) 1 =
// F32, a_format (7-9) and b_format (10-12) 1 = BF16, a_major (15), b_major
// (16), N >> 3 in 17-22, M >> 4 in 24-28.
__host__ __device__ constexpr uint32_t bf16_idesc(uint32_t M, uint32_t N, uint32_t a_mn, uint32_t b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn << 15) | (b_mn << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// The same for f16 operands (format 0).
__host__ __device__ constexpr uint32_t f16_idesc(uint32_t M, uint32_t N, uint32_t a_mn, uint32_t b_mn) {
  return (1u << 4) | (a_mn << 15) | (b_mn << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

__device__ __forceinline__ float lg2_f(float x) { return __log2f(x); }

}  // namespace flamia
