// paged_pages.cuh — pages that several requests share: parameters and the
// workspace of the page operators (paged_pages.cu, paged_copy.cu).
#pragma once
#include "paged.cuh"

namespace flamia {

constexpr int kPagesThreads = 512, kMaxPagesCtas = 160;
constexpr int kShareBarriers = 2, kCompactBarriers = 3;  // of a launch
constexpr int kCopyLayers = 32;  // of a launch: its parameters stay below 4 KB

struct PagesHeader {
  WsHeader base;         // status words first, as flamia_get_device_status reads them
  uint32_t fail;         // why the step moved no page: flamia_paged_plan_shared's plan reads it
  uint32_t bad;          // found by some CTA before anything is written
  uint32_t arrived;      // CTAs at the grid's barriers, all of the launch together; its top bit: a wait ran out
  uint32_t wrong;        // found between the barriers; apart from `bad`, which a slow CTA may
                         // still have to read at one barrier while a fast one is at the next
  unsigned long long most;  // pages that the step takes at most
  uint32_t pad[10];
  uint32_t count[kMaxPagesCtas];  // compact: free pages in each CTA's part
};

// What a step does to one page; zero at the launch's start.
struct __align__(16) PageRec {
  int32_t delta;   // holders gained less those lost, copies aside
  int32_t first;   // INT_MAX less the first entry (row * max_pages + index) that lets go of it; 0: none
  int32_t writers; // requests whose new tokens go into it
  int32_t writer;  // n_req less the first of them; 0: none
};
static_assert(sizeof(PageRec) == 16, "one sector for two");

struct PagesLayout {
  size_t header, pages, staged, freed, counts, total;
};

struct PagesParams {
  int n_req, T, max_q, page_size, page_shift, n_pages, max_pages;
  const int32_t* cu_q;
  const int32_t* kv_len;
  int32_t* block_table;
  const int32_t* src;      // may be NULL: every request continues itself
  const int32_t* old_len;
  int32_t* refs;
  int32_t* free_pages;
  const int32_t* n_free;
  int32_t* n_free_out;
  int32_t* copies;         // [.][2]
  int32_t* n_copies;
  PagesHeader* hdr;
  PageRec* pages;          // [n_pages]
  int32_t* staged;         // [n_req][max_pages] pages that a row takes over from another's
  int32_t* freed;          // [n_req][max_pages] pages without a holder, by the row that let go of them first
  int4* counts;            // [n_req] pages that the row takes, its freed ones, whether its partly filled one is copied
  int dbg_withhold;        // test hook: the barrier, from 1, at which one CTA's arrival is withheld
  // compact, in the place of `pages`
  uint32_t* bits;          // free pages
  int32_t* rank;           // [n_pages] of the pages that move
};

struct CopyLayer {
  const uint8_t* src[6];  // k, v, their scales, their block scales
  uint8_t* dst[6];
};
struct CopyParams {
  CopyLayer layer[kCopyLayers];
  int64_t src_stride[kCopyLayers], dst_stride[kCopyLayers];  // bytes between pages of k and of v
  int layers, n_pages;
  int kv_vecs, scale_vecs, block_vecs;  // of a page of each array, 16 bytes each
  const int32_t* copies;
  const int32_t* n_copies;
  int max_copies;
  PagesHeader* hdr;
};

cudaError_t launch_paged_share(const PagesParams& p, int sms, cudaStream_t st);
cudaError_t launch_paged_compact(const PagesParams& p, int sms, cudaStream_t st);
cudaError_t launch_paged_copy(const CopyParams& p, int sms, cudaStream_t st);

}  // namespace flamia
