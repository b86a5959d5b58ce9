// Host-visible pieces of the paged key/value cache: the batch and cache as
// the kernels see them, and the launchers. Contract: include/fa2.h.
#pragma once
#include "fa2_launch.h"

namespace fa2 {

// A batch of sequences whose keys and values lie in pages. Sequence b has
// `length` positions, the last `n` of which are the batch's tokens [t0, t0 + n).
struct PagedBatch {
  const int* table;        // [B][max_pages], rows table_stride apart: page of each page-size run of positions
  const int* lengths;      // [B]
  const int* starts;       // [B + 1], or NULL: every sequence has T / B tokens
  long long table_stride;
  int T, B, heads;         // heads: key heads
  int pages, max_pages;
  int page_shift;          // log2 of the page size
  int each;                // T / B
  int capacity;            // max_pages * page size, at most 2^30
};

struct PagedStrides {  // of a cache, in elements
  long long page, head, slot;
};

constexpr bool paged_head_dim_ok(int d) { return d == 32 || d == 64 || d == 96 || d == 128; }
constexpr int kMaxPageShift = 8;  // page sizes 16 .. 256

// ------------------------------------------------------------- attention
struct PagedAttnParams : PagedBatch {
  const void* q;
  long long q_token, q_head;  // strides
  void* o;                    // [T][Hq][D]
  float* lse;                 // [T][Hq]
  int group;                  // query heads per key head
  int causal;
  int rows_from, rows_to;     // this kernel's sequences: rows_from <= n * group <= rows_to
  float scale_log2;
  int* status;
  unsigned long long watchdog_ns;
  unsigned long long epoch;
  int test_withhold;
  float* ws_o;
  float* ws_stats;
  unsigned long long* ws_flags;
};

// At most 16 query rows per key head at a time (fa2_paged_rows.cu).
constexpr int kPagedRows = 16;
constexpr int kPagedRowsKeys = 128;
constexpr int kPagedRowsMaxCtas = 256;
constexpr size_t paged_rows_workspace_bytes(int grid, int d) {  // ws_o [grid][16][D], ws_stats [grid][3][16], flags
  return (static_cast<size_t>(grid) * kPagedRows * (d + 3) * sizeof(float) + 255) / 256 * 256 +
         (static_cast<size_t>(grid) * 8 + 255) / 256 * 256;
}
// k, v: maps (D, slot, head, page) with boxes of 64 elements x 16 slots.
cudaError_t launch_paged_rows(int D, bool bf16, const CUtensorMap& k, const CUtensorMap& v, const PagedAttnParams& p,
                              int grid, cudaStream_t stream);

// More rows (fa2_paged_kernel.cuh, instantiated in fa2_paged_d{32,64,96,128}.cu).
// q: map (D, head, token) with boxes of 64 elements x group heads x sub-tile
// tokens; k, v: as above with boxes of min(page size, 128) slots.
struct PagedTileParams : PagedAttnParams {
  int sub_tokens;   // tokens of a sub-tile: 128 / group
  int page_rows;    // positions of a page in one K/V tile: min(page size, 128)
  int wide;         // head dimension above 64
  unsigned long long* ws_spread;  // [2][grid][kPagedMostParts]: which parts of its unit a CTA may read
};
// Parts that a unit is cut into at most.
constexpr int kPagedMostParts = 32;
constexpr size_t paged_spread_bytes(int grid) { return static_cast<size_t>(grid) * 2 * kPagedMostParts * 8; }
template <int D, bool kBf16>
cudaError_t launch_paged_tiles(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                               const PagedTileParams& p, int grid, cudaStream_t stream);

// ------------------------------------------------------------ key weights
struct PagedWeighParams : PagedBatch {
  const float* lse;           // [T][Hq]
  const float* in;            // [pages][heads][page size], or NULL: zeros
  float* out;
  int group, causal;
  float scale_log2;
  // a block of query rows: tokens, heads of the group, blocks that a group takes, columns of its product
  int block_tokens, block_heads, head_blocks, columns;
  int page_rows;              // as in PagedTileParams
  int* status;
  unsigned long long watchdog_ns;
  int test_withhold;
  unsigned long long epoch;
  float* ws_sums;             // [grid][256]
  unsigned long long* ws_flags;  // [grid]
};
constexpr size_t paged_weigh_workspace_bytes(int grid) { return static_cast<size_t>(grid) * (2 * kKeys * sizeof(float) + 8); }
// q: map (D, head, token) with boxes of 64 elements x block heads x block tokens; k: as for launch_paged_tiles.
cudaError_t launch_paged_weigh(int D, bool bf16, const CUtensorMap& q, const CUtensorMap& k, const PagedWeighParams& p,
                               int grid, cudaStream_t stream);

// --------------------------------------------------------- append, evict
struct PagedAppendParams : PagedBatch {
  const void* k;
  const void* v;
  long long k_token, k_head, v_token, v_head;
  void* kc;
  void* vc;
  PagedStrides ks, vs;
  float* weights;             // [pages][heads][page size], or NULL
};
cudaError_t launch_paged_append(int D, const PagedAppendParams& p, int sms, cudaStream_t stream);

struct PagedEvictParams : PagedBatch {
  void* kc;
  void* vc;
  PagedStrides ks, vs;
  float* weights;
  const int* new_table;       // [B][new_max_pages]
  long long new_stride;
  int new_max_pages;
  int keep, recent;
  int* new_lengths;           // [B]
  int* kept;                  // [B][heads][keep]
};
cudaError_t launch_paged_evict(int D, const PagedEvictParams& p, int sms, cudaStream_t stream);

}  // namespace fa2
