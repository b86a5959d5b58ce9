// C ABI of the paged key/value cache: argument checks, tensor maps, the choice
// of the kernels and their launch. Declarations and the contract: include/fa2.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "fa2.h"
#include "fa2_paged.h"

namespace fa2 {
namespace {

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_tiled() {
  static std::once_flag once;
  static EncodeFn fn = nullptr;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(f);
  });
  return fn;
}

// Sizes and strides as the caller gave them.
struct Sizes {
  int T, B, Hkv, D, pages, page_size, max_pages, dtype;
};

constexpr long long kReach = 1ll << 44;  // no view reaches further, in elements

// A view's strides (elements): of dimensions longer than 1 multiples of 8, at least `least`, and in reach.
bool strides_ok(const long long* stride, const long long* size, int dims, long long least) {
  long long reach = 0;
  for (int i = 0; i < dims; ++i) {
    if (size[i] <= 1) continue;
    if (stride[i] < least || stride[i] % 8 != 0 || stride[i] > kReach) return false;
    const long double far = static_cast<long double>(size[i] - 1) * stride[i];
    if (far > kReach) return false;
    reach += (size[i] - 1) * stride[i];
    if (reach > kReach) return false;
  }
  return true;
}

// What a tensor map takes besides: positive strides below 2^40 bytes.
bool map_strides_ok(const long long* stride, const long long* size, int dims) {
  for (int i = 0; i < dims; ++i)
    if (size[i] > 1 && stride[i] >= 1ll << 39) return false;
  return strides_ok(stride, size, dims, 8);
}
bool cache_strides_ok(const PagedStrides& c, const Sizes& z) {
  const long long stride[3] = {c.page, c.head, c.slot}, size[3] = {z.pages, z.Hkv, z.page_size};
  return map_strides_ok(stride, size, 3);
}


// Bytes from a cache's first element to its last.
size_t cache_reach(const PagedStrides& c, const Sizes& z) {
  const long long last = (z.pages - 1) * c.page * (z.pages > 1) + (z.Hkv - 1) * c.head * (z.Hkv > 1) +
                         (z.page_size - 1) * c.slot + z.D;
  return static_cast<size_t>(last) * 2;
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

int check_sizes(const Sizes& z) {
  if (z.T < 0 || z.B < 0 || z.Hkv < 0 || z.pages < 0 || z.max_pages < 0) return FA2_ERR_INVALID_ARG;
  if (!paged_head_dim_ok(z.D)) return FA2_ERR_UNSUPPORTED;
  if (z.dtype != FA2_F16 && z.dtype != FA2_BF16) return FA2_ERR_UNSUPPORTED;
  if (z.page_size < 16 || z.page_size > (1 << kMaxPageShift) || (z.page_size & (z.page_size - 1)))
    return FA2_ERR_UNSUPPORTED;
  // 2^30: a position, token, row or sequence index plus a tile or a warp's step stays inside 32 bits
  if (static_cast<int64_t>(z.max_pages) * z.page_size > (1 << 30) || z.T > (1 << 30) || z.B > (1 << 30))
    return FA2_ERR_INVALID_ARG;
  // 2^24: the rows of up to 128 tokens (a block of key weights) are counted in 32 bits over all heads
  if (static_cast<int64_t>(z.B) * z.Hkv > INT32_MAX || z.Hkv > (1 << 24)) return FA2_ERR_INVALID_ARG;
  return FA2_OK;
}

// The batch as the kernels see it. Without starts every sequence has T / B tokens.
int fill_batch(PagedBatch& p, const Sizes& z, const int* table, const int* lengths, const int* starts,
               long long table_stride) {
  if (!table || !lengths) return FA2_ERR_INVALID_ARG;
  if (!aligned(table, 4) || !aligned(lengths, 4) || !aligned(starts, 4)) return FA2_ERR_ALIGN;
  if (z.B > 1 && (table_stride < 0 || table_stride > kReach)) return FA2_ERR_INVALID_ARG;
  if (!starts && z.T % z.B != 0) return FA2_ERR_INVALID_ARG;
  p.table = table;
  p.lengths = lengths;
  p.starts = starts;
  p.table_stride = z.B > 1 ? table_stride : 0;
  p.T = z.T;
  p.B = z.B;
  p.heads = z.Hkv;
  p.pages = z.pages;
  p.max_pages = z.max_pages;
  p.page_shift = 0;
  while ((1 << p.page_shift) < z.page_size) ++p.page_shift;
  p.each = starts ? 0 : z.T / z.B;
  p.capacity = z.max_pages * z.page_size;
  return FA2_OK;
}

// (D, slot, head, page) of a cache, boxes of 64 elements x `rows` slots, 128-byte swizzled; columns past D and
// pages past the last read as zeros.
bool encode_cache_map(CUtensorMap* m, const void* ptr, const PagedStrides& c, const Sizes& z, unsigned rows) {
  const EncodeFn enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)z.D, (cuuint64_t)z.page_size, (cuuint64_t)z.Hkv, (cuuint64_t)z.pages};
  const cuuint64_t one = (cuuint64_t)z.D * 2;  // stands in for the stride of a dimension of length 1
  const cuuint64_t strides[3] = {(cuuint64_t)c.slot * 2, z.Hkv > 1 ? (cuuint64_t)c.head * 2 : one,
                                 z.pages > 1 ? (cuuint64_t)c.page * 2 : one};
  const cuuint32_t box[4] = {64, rows, 1, 1}, step[4] = {1, 1, 1, 1};
  return enc(m, z.dtype == FA2_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
             const_cast<void*>(ptr), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// (D, head, token) of the queries, boxes of 64 elements x `heads` heads x `tokens` tokens.
bool encode_query_map(CUtensorMap* m, const void* ptr, long long token, long long head, int T, int Hq, int D, int dtype,
                      unsigned heads, unsigned tokens) {
  const EncodeFn enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)T}, one = (cuuint64_t)D * 2;
  const cuuint64_t strides[2] = {Hq > 1 ? (cuuint64_t)head * 2 : one, T > 1 ? (cuuint64_t)token * 2 : one};
  const cuuint32_t box[3] = {64, heads, tokens}, step[3] = {1, 1, 1};
  return enc(m, dtype == FA2_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
             const_cast<void*>(ptr), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether any output meets any of the other ranges (inputs, or a later output); empty ranges meet nothing.
struct Range {
  const void* at;
  size_t bytes;
};
bool any_overlap(const Range* outs, int n_out, const Range* ins, int n_in) {
  for (int a = 0; a < n_out; ++a) {
    if (!outs[a].at || !outs[a].bytes) continue;
    for (int b = 0; b < n_in; ++b)
      if (ins[b].at && ins[b].bytes && ranges_overlap(outs[a].at, outs[a].bytes, ins[b].at, ins[b].bytes)) return true;
    for (int b = a + 1; b < n_out; ++b)
      if (outs[b].at && outs[b].bytes && ranges_overlap(outs[a].at, outs[a].bytes, outs[b].at, outs[b].bytes)) return true;
  }
  return false;
}

size_t tokens_reach(int T, long long token, int heads, long long head, int D) {
  return static_cast<size_t>((T - 1) * token * (T > 1) + (heads - 1) * head * (heads > 1) + D) * 2;
}

// The rows kernel's partial results, then the tiles kernel's, then its flags for units that all of their CTAs join.
size_t rows_workspace(int sms, int D) { return paged_rows_workspace_bytes(std::min(sms, kPagedRowsMaxCtas), D); }
size_t fwd_workspace_bytes(int sms, int D) {
  return rows_workspace(sms, D) + stream_k_workspace_bytes(sms, D) + paged_spread_bytes(sms);
}

using TilesFn = cudaError_t (*)(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const PagedTileParams&, int,
                                cudaStream_t);
TilesFn pick_tiles(int d, bool bf) {
  switch (d) {
    case 32: return bf ? launch_paged_tiles<32, true> : launch_paged_tiles<32, false>;
    case 64: return bf ? launch_paged_tiles<64, true> : launch_paged_tiles<64, false>;
    case 96: return bf ? launch_paged_tiles<96, true> : launch_paged_tiles<96, false>;
    default: return bf ? launch_paged_tiles<128, true> : launch_paged_tiles<128, false>;
  }
}

int cuda_result(cudaError_t e) { return e == cudaSuccess ? FA2_OK : record_cuda_error(e); }

}  // namespace
}  // namespace fa2

using namespace fa2;

extern "C" int fa2_paged_append(const void* K, const void* V, void* k_cache, void* v_cache, float* weights,
                                const int* block_table, const int* key_lengths, const int* query_starts,
                                const long long* strides, int T, int B, int Hkv, int D, int pages, int page_size,
                                int max_pages, int dtype, struct CUstream_st* stream) {
  const Sizes z = {T, B, Hkv, D, pages, page_size, max_pages, dtype};
  int rc = check_sizes(z);
  if (rc != FA2_OK) return rc;
  if (T == 0 || B == 0 || Hkv == 0 || pages == 0 || max_pages == 0) return FA2_OK;
  if (!K || !V || !k_cache || !v_cache || !strides) return FA2_ERR_INVALID_ARG;
  PagedAppendParams p = {};
  rc = fill_batch(p, z, block_table, key_lengths, query_starts, strides[10]);
  if (rc != FA2_OK) return rc;
  p.k = K;
  p.v = V;
  p.k_token = strides[0];
  p.k_head = strides[1];
  p.v_token = strides[2];
  p.v_head = strides[3];
  p.kc = k_cache;
  p.vc = v_cache;
  p.ks = PagedStrides{strides[4], strides[5], strides[6]};
  p.vs = PagedStrides{strides[7], strides[8], strides[9]};
  p.weights = weights;
  const long long tokens[2] = {T, Hkv};
  if (!strides_ok(strides, tokens, 2, 0) || !strides_ok(strides + 2, tokens, 2, 0) || !cache_strides_ok(p.ks, z) ||
      !cache_strides_ok(p.vs, z))
    return FA2_ERR_INVALID_ARG;
  if (!aligned(K, 16) || !aligned(V, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(weights, 4))
    return FA2_ERR_ALIGN;
  const size_t starts_bytes = static_cast<size_t>(B + 1) * 4;
  const Range ins[5] = {{K, tokens_reach(T, p.k_token, Hkv, p.k_head, D)}, {V, tokens_reach(T, p.v_token, Hkv, p.v_head, D)},
                        {block_table, static_cast<size_t>((B - 1) * p.table_stride + max_pages) * 4},
                        {key_lengths, static_cast<size_t>(B) * 4}, {query_starts, starts_bytes}};
  const Range outs[3] = {{k_cache, cache_reach(p.ks, z)}, {v_cache, cache_reach(p.vs, z)},
                         {weights, static_cast<size_t>(pages) * Hkv * page_size * 4}};
  for (const Range& o : outs)  // the two caches may interleave
    if (any_overlap(&o, 1, ins, 5)) return FA2_ERR_INVALID_ARG;
  if (any_overlap(outs + 2, 1, outs, 2)) return FA2_ERR_INVALID_ARG;
  int sms = 0;
  int* status = nullptr;
  rc = current_device_facts(&sms, &status);
  if (rc != FA2_OK) return rc;
  return cuda_result(launch_paged_append(D, p, sms, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" int fa2_paged_fwd_workspace_bytes(int D, size_t* bytes) {
  if (!bytes) return FA2_ERR_INVALID_ARG;
  if (!paged_head_dim_ok(D)) return FA2_ERR_UNSUPPORTED;
  int sms = 0;
  int* status = nullptr;
  const int rc = current_device_facts(&sms, &status);
  if (rc != FA2_OK) return rc;
  *bytes = fwd_workspace_bytes(sms, D);
  return FA2_OK;
}

extern "C" int fa2_paged_fwd(const void* Q, const void* k_cache, const void* v_cache, void* O, float* LSE,
                             const int* block_table, const int* key_lengths, const int* query_starts,
                             const long long* strides, int T, int B, int Hq, int Hkv, int D, int pages, int page_size,
                             int max_pages, int max_query_length, float scale, int is_causal, int dtype,
                             void* workspace, size_t workspace_bytes, struct CUstream_st* stream) {
  const Sizes z = {T, B, Hkv, D, pages, page_size, max_pages, dtype};
  int rc = check_sizes(z);
  if (rc != FA2_OK) return rc;
  if (Hq < 0 || max_query_length < 0) return FA2_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA2_ERR_INVALID_ARG;
  if (T == 0 || B == 0 || Hq == 0) return FA2_OK;
  if (Hkv == 0 || Hq % Hkv != 0) return FA2_ERR_INVALID_ARG;
  const int group = Hq / Hkv;
  if (static_cast<int64_t>(T) * group > (1 << 30)) return FA2_ERR_INVALID_ARG;
  if (pages == 0 || max_pages == 0) return FA2_ERR_INVALID_ARG;
  if (!Q || !k_cache || !v_cache || !O || !LSE || !strides || !workspace) return FA2_ERR_INVALID_ARG;
  PagedTileParams p = {};
  rc = fill_batch(p, z, block_table, key_lengths, query_starts, strides[8]);
  if (rc != FA2_OK) return rc;
  const PagedStrides ks = {strides[2], strides[3], strides[4]}, vs = {strides[5], strides[6], strides[7]};
  const long long tokens[2] = {T, Hq};
  if (!map_strides_ok(strides, tokens, 2) || !cache_strides_ok(ks, z) || !cache_strides_ok(vs, z))
    return FA2_ERR_INVALID_ARG;
  if (!aligned(Q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(O, 16) || !aligned(LSE, 4) ||
      !aligned(workspace, 16))
    return FA2_ERR_ALIGN;
  const size_t rows = static_cast<size_t>(T) * Hq;
  const Range outs[3] = {{O, rows * D * 2}, {LSE, rows * 4}, {workspace, workspace_bytes}};
  const Range ins[6] = {{Q, tokens_reach(T, strides[0], Hq, strides[1], D)}, {k_cache, cache_reach(ks, z)},
                        {v_cache, cache_reach(vs, z)}, {key_lengths, static_cast<size_t>(B) * 4},
                        {query_starts, static_cast<size_t>(B + 1) * 4},
                        {block_table, static_cast<size_t>((B - 1) * p.table_stride + max_pages) * 4}};
  if (any_overlap(outs, 3, ins, 6)) return FA2_ERR_INVALID_ARG;
  int sms = 0;
  int* status = nullptr;
  rc = current_device_facts(&sms, &status);
  if (rc != FA2_OK) return rc;
  if (workspace_bytes < fwd_workspace_bytes(sms, D)) return FA2_ERR_INVALID_ARG;
  p.q = Q;
  p.q_token = strides[0];
  p.q_head = strides[1];
  p.o = O;
  p.lse = LSE;
  p.group = group;
  p.causal = is_causal != 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.status = status;
  p.watchdog_ns = watchdog_limit_ns();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // Sequences of at most 16 rows per key head run on the rows kernel, those of
  // more on the tensor cores (unless a token alone has more rows than a
  // sub-tile); each kernel passes over the other's. Only the device knows the
  // sequences' tokens, so both are launched unless the sizes rule one out.
  //
  // The rows kernel takes them all (in blocks of 16 rows) where there are few
  // blocks (us, rows kernel / tensor cores, over 300, 1000, 4000 and 16,000
  // positions; D = 128, 16 blocks: 11.2 / 10.2, 14.3 / 15.5, 15.3 / 18.4, 25.9 / 26.6;
  // 32 blocks: 12.3 / 10.4, 14.4 / 15.5, 19.9 / 18.6, 39.6 / 26.7; D = 64, 24 blocks:
  // 9.3 / 9.5, 10.8 / 14.6, 13.8 / 16.2, 25.6 / 22.4; 48 blocks: 10.0 / 9.4, 11.8 / 14.5,
  // 17.2 / 16.2, 40.2 / 22.3). Of the positions the host knows the table's width alone.
  const int longest = query_starts ? std::min(T, max_query_length) : p.each;
  const int64_t most = static_cast<int64_t>(longest) * group;
  const int64_t blocks = std::min(static_cast<int64_t>(B) * ((most + kPagedRows - 1) / kPagedRows),
                                  static_cast<int64_t>(T) * group / kPagedRows + B) * Hkv;
  const bool tiles = most > kPagedRows && group <= kRows && blocks > (D > 64 ? 16 : 24);
  // A sequence of so few tokens would leave the others more than `longest` each.
  const int few = kPagedRows / group;
  const bool none_short = group > kPagedRows || (longest > few && static_cast<int64_t>(B) * longest - T < longest - few);
  const bool rows_too = !tiles || !none_short;
  p.test_withhold = take_test_withhold();
  char* const ws = static_cast<char*>(workspace);
  const bool bf = dtype == FA2_BF16;
  if (rows_too) {
    CUtensorMap mk, mv;
    if (!encode_cache_map(&mk, k_cache, ks, z, 16u) || !encode_cache_map(&mv, v_cache, vs, z, 16u))
      return record_cuda_error(cudaErrorInvalidValue);
    const int grid = std::min(sms, kPagedRowsMaxCtas);
    p.rows_from = 1;
    p.rows_to = tiles ? kPagedRows : INT_MAX;
    p.ws_o = reinterpret_cast<float*>(ws);
    p.ws_stats = p.ws_o + static_cast<size_t>(grid) * kPagedRows * D;
    p.ws_flags = reinterpret_cast<unsigned long long*>(ws + rows_workspace(sms, D) -
                                                       (static_cast<size_t>(grid) * 8 + 255) / 256 * 256);
    p.epoch = next_launch_epoch();
    const cudaError_t e = launch_paged_rows(D, bf, mk, mv, p, grid, s);
    if (e != cudaSuccess) return record_cuda_error(e);
  }
  if (!tiles) return FA2_OK;
  CUtensorMap mq, mk, mv;
  p.sub_tokens = kRows / group;
  p.page_rows = std::min(page_size, kKeys);
  p.wide = D > 64;
  if (!encode_query_map(&mq, Q, p.q_token, p.q_head, T, Hq, D, dtype, group, p.sub_tokens) ||
      !encode_cache_map(&mk, k_cache, ks, z, p.page_rows) || !encode_cache_map(&mv, v_cache, vs, z, p.page_rows))
    return record_cuda_error(cudaErrorInvalidValue);
  p.rows_from = rows_too ? kPagedRows + 1 : 1;
  p.rows_to = INT_MAX;
  const size_t slots = static_cast<size_t>(sms) * kSubTiles;
  p.ws_o = reinterpret_cast<float*>(ws + rows_workspace(sms, D));
  p.ws_stats = p.ws_o + slots * D * 128;
  p.ws_flags = reinterpret_cast<unsigned long long*>(
      ws + rows_workspace(sms, D) + (slots * (static_cast<size_t>(D) * 128 + 3 * 128) * sizeof(float) + 255) / 256 * 256);
  p.ws_spread = reinterpret_cast<unsigned long long*>(ws + rows_workspace(sms, D) + stream_k_workspace_bytes(sms, D));
  p.epoch = next_launch_epoch();
  return cuda_result(pick_tiles(D, bf)(mq, mk, mv, p, sms, s));
}

extern "C" int fa2_paged_key_weights_workspace_bytes(size_t* bytes) {
  if (!bytes) return FA2_ERR_INVALID_ARG;
  int sms = 0;
  int* status = nullptr;
  const int rc = current_device_facts(&sms, &status);
  if (rc != FA2_OK) return rc;
  *bytes = paged_weigh_workspace_bytes(sms);
  return FA2_OK;
}

extern "C" int fa2_paged_key_weights(const void* Q, const float* LSE, const void* k_cache, const float* weights,
                                     float* out, const int* block_table, const int* key_lengths,
                                     const int* query_starts, const long long* strides, int T, int B, int Hq, int Hkv,
                                     int D, int pages, int page_size, int max_pages, int max_query_length, float scale,
                                     int is_causal, int dtype, void* workspace, size_t workspace_bytes,
                                     struct CUstream_st* stream) {
  const Sizes z = {T, B, Hkv, D, pages, page_size, max_pages, dtype};
  int rc = check_sizes(z);
  if (rc != FA2_OK) return rc;
  if (Hq < 0 || max_query_length < 0) return FA2_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA2_ERR_INVALID_ARG;
  if (B == 0 || Hkv == 0 || pages == 0 || max_pages == 0) return FA2_OK;
  if (Hq % Hkv != 0 || (Hq == 0 && T > 0)) return FA2_ERR_INVALID_ARG;
  const int group = Hq / Hkv;
  if (static_cast<int64_t>(T) * group > (1 << 30)) return FA2_ERR_INVALID_ARG;
  if ((T > 0 && (!Q || !LSE)) || !k_cache || !out || !strides || !workspace) return FA2_ERR_INVALID_ARG;
  PagedWeighParams p = {};
  rc = fill_batch(p, z, block_table, key_lengths, query_starts, strides[5]);
  if (rc != FA2_OK) return rc;
  const PagedStrides ks = {strides[2], strides[3], strides[4]};
  const long long tokens[2] = {T, Hq};
  if (!map_strides_ok(strides, tokens, 2) || !cache_strides_ok(ks, z)) return FA2_ERR_INVALID_ARG;
  if (!aligned(Q, 16) || !aligned(k_cache, 16) || !aligned(LSE, 4) || !aligned(weights, 4) || !aligned(out, 4) ||
      !aligned(workspace, 16))
    return FA2_ERR_ALIGN;
  const size_t pool = static_cast<size_t>(pages) * Hkv * page_size * 4;
  const Range outs[2] = {{out, pool}, {workspace, workspace_bytes}};
  const Range ins[7] = {{T > 0 ? Q : nullptr, T > 0 ? tokens_reach(T, strides[0], Hq, strides[1], D) : 0},
                        {k_cache, cache_reach(ks, z)}, {LSE, static_cast<size_t>(T) * Hq * 4},
                        {key_lengths, static_cast<size_t>(B) * 4}, {query_starts, static_cast<size_t>(B + 1) * 4},
                        {block_table, static_cast<size_t>((B - 1) * p.table_stride + max_pages) * 4},
                        {weights == out ? nullptr : weights, pool}};
  if (any_overlap(outs, 2, ins, 7)) return FA2_ERR_INVALID_ARG;
  int sms = 0;
  int* status = nullptr;
  rc = current_device_facts(&sms, &status);
  if (rc != FA2_OK) return rc;
  if (workspace_bytes < paged_weigh_workspace_bytes(sms)) return FA2_ERR_INVALID_ARG;
  p.lse = LSE;
  p.in = weights;
  p.out = out;
  p.group = group;
  p.causal = is_causal != 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.block_heads = std::max(1, std::min(group, kRows));
  p.head_blocks = (group + kRows - 1) / kRows;
  // No larger blocks than the sequences fill: a block is loaded and multiplied whole.
  const int most = query_starts ? std::min(T, max_query_length) : p.each;
  p.block_tokens = std::max(1, std::min(kRows / p.block_heads, most));
  p.columns = (p.block_tokens * p.block_heads + 15) / 16 * 16;
  p.page_rows = std::min(page_size, kKeys);
  p.status = status;
  p.watchdog_ns = watchdog_limit_ns();
  CUtensorMap mq, mk;
  if (!encode_cache_map(&mk, k_cache, ks, z, p.page_rows)) return record_cuda_error(cudaErrorInvalidValue);
  if (T == 0) mq = mk;  // not read
  else if (!encode_query_map(&mq, Q, strides[0], strides[1], T, Hq, D, dtype, p.block_heads, p.block_tokens))
    return record_cuda_error(cudaErrorInvalidValue);
  p.test_withhold = take_test_withhold();
  p.ws_sums = static_cast<float*>(workspace);
  p.ws_flags = reinterpret_cast<unsigned long long*>(p.ws_sums + static_cast<size_t>(sms) * 2 * kKeys);
  p.epoch = next_launch_epoch();
  return cuda_result(launch_paged_weigh(D, dtype == FA2_BF16, mq, mk, p, sms, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" int fa2_paged_evict(void* k_cache, void* v_cache, float* weights, const int* block_table,
                               const int* key_lengths, const int* new_table, int* new_lengths, int* kept,
                               const long long* strides, int B, int Hkv, int D, int pages, int page_size,
                               int max_pages, int new_max_pages, int keep, int recent, int dtype,
                               struct CUstream_st* stream) {
  const Sizes z = {0, B, Hkv, D, pages, page_size, max_pages, dtype};
  int rc = check_sizes(z);
  if (rc != FA2_OK) return rc;
  if (keep < 0 || recent < 0 || recent > keep || new_max_pages < 0) return FA2_ERR_INVALID_ARG;
  if (static_cast<int64_t>(new_max_pages) * page_size < keep) return FA2_ERR_INVALID_ARG;
  if (keep > (1 << 30)) return FA2_ERR_INVALID_ARG;  // as positions: an index plus a block's step stays inside 32 bits
  if (static_cast<int64_t>(B) * Hkv * std::max(keep, 1) > (1ll << 40)) return FA2_ERR_INVALID_ARG;
  if (B == 0) return FA2_OK;
  if (Hkv == 0 || pages == 0 || max_pages == 0) return FA2_ERR_INVALID_ARG;
  if (!k_cache || !v_cache || !weights || !new_lengths || !strides || (keep > 0 && (!kept || !new_table)))
    return FA2_ERR_INVALID_ARG;
  PagedEvictParams p = {};
  rc = fill_batch(p, z, block_table, key_lengths, nullptr, strides[6]);
  if (rc != FA2_OK) return rc;
  p.ks = PagedStrides{strides[0], strides[1], strides[2]};
  p.vs = PagedStrides{strides[3], strides[4], strides[5]};
  if (!cache_strides_ok(p.ks, z) || !cache_strides_ok(p.vs, z)) return FA2_ERR_INVALID_ARG;
  if (B > 1 && (strides[7] < 0 || strides[7] > kReach)) return FA2_ERR_INVALID_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(weights, 4) || !aligned(new_table, 4) ||
      !aligned(new_lengths, 4) || !aligned(kept, 4))
    return FA2_ERR_ALIGN;
  p.new_stride = B > 1 ? strides[7] : 0;
  const size_t old_bytes = static_cast<size_t>((B - 1) * p.table_stride + max_pages) * 4;
  const size_t new_bytes = static_cast<size_t>((B - 1) * p.new_stride + new_max_pages) * 4;
  const Range outs[2] = {{new_lengths, static_cast<size_t>(B) * 4}, {kept, static_cast<size_t>(B) * Hkv * keep * 4}};
  const Range ins[6] = {{k_cache, cache_reach(p.ks, z)}, {v_cache, cache_reach(p.vs, z)},
                        {weights, static_cast<size_t>(pages) * Hkv * page_size * 4}, {block_table, old_bytes},
                        {new_table, new_bytes}, {key_lengths, static_cast<size_t>(B) * 4}};
  if (any_overlap(outs, 2, ins, 6)) return FA2_ERR_INVALID_ARG;
  // the caches (which may interleave) and the weights are written too
  for (int i = 0; i < 3; ++i)
    if (any_overlap(ins + i, 1, ins + std::max(i + 1, 2), 6 - std::max(i + 1, 2))) return FA2_ERR_INVALID_ARG;
  // pages are written while others are read
  if (keep > 0 && new_table == block_table) return FA2_ERR_INVALID_ARG;
  int sms = 0;
  int* status = nullptr;
  rc = current_device_facts(&sms, &status);
  if (rc != FA2_OK) return rc;
  p.kc = k_cache;
  p.vc = v_cache;
  p.weights = weights;
  p.new_table = new_table;
  p.new_max_pages = new_max_pages;
  p.keep = keep;
  p.recent = recent;
  p.new_lengths = new_lengths;
  p.kept = kept;
  return cuda_result(launch_paged_evict(D, p, sms, reinterpret_cast<cudaStream_t>(stream)));
}
