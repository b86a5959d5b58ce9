// C ABI of cross attention: argument checks, tensor maps, the choice of the
// schedule and the launch. Declarations and the contract: include/fa2.h.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "fa2.h"
#include "fa2_cross.h"
#include "fa2_cross_schedule.h"

namespace fa2 {
namespace {

constexpr bool cross_head_dim_ok(int d) { return d == 32 || d == 64 || d == 96 || d == 128; }

// LSE of rows that have no key at all.
__global__ void fa2_cross_fill_lse(float* lse, long long n) {
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += stride)
    lse[i] = CUDART_INF_F;
}

using CrossFn = cudaError_t (*)(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                const CrossParams&, int, cudaStream_t);

CrossFn pick_cross(int d, bool bf) {
  switch (d) {
    case 32: return bf ? launch_cross_fwd<32, true> : launch_cross_fwd<32, false>;
    case 64: return bf ? launch_cross_fwd<64, true> : launch_cross_fwd<64, false>;
    case 96: return bf ? launch_cross_fwd<96, true> : launch_cross_fwd<96, false>;
    default: return bf ? launch_cross_fwd<128, true> : launch_cross_fwd<128, false>;
  }
}

// What a unit counts in the equal shares besides its tiles: the tensor cores
// idle while its last P.V drains and its rows go out. Without it the CTAs with
// the short units of a padded batch came last (us, by the cost 0, 2, 3, 4, 6:
// 4 x 16 heads of 2048 rows over 2048, 4096, 6144 and 8192 keys, D = 128: 220,
// 203, 208, 202, 204; 8 x 8 heads of 1024 rows over 256, 512 .. 2048 keys: D =
// 128 55.6, 43.9, 44.3, 45.7, 45.8, D = 64 41.9, 35.4, 35.2, 35.6, 39.7; 32 x
// 8 heads of 128 rows over 128, 256 .. 4096 keys, D = 64 59.7, 40.3, 38.5,
// 39.0, 39.4). Units of one length keep equal tiles: there every CTA has about
// as many segments as any other (8 heads of 4096 rows x 8192 keys, D = 128:
// 90.6 with cost 0, 94.5 with 4).
constexpr int unit_cost(int D, bool lengths) { return !lengths ? 0 : D <= 64 ? 3 : 4; }

// Whether the few-keys kernel beats the tcgen05 one. Measured (us, few-keys
// against tcgen05): 32 heads of 4096 rows, D = 64, 16 keys 8.7 / 20.6, 77 keys
// 16.5 / 21.3, 128 keys 19.2 / 19.1; D = 128, 16 keys 14.6 / 26.7, 96 keys
// 27.1 / 27.4, 128 keys 34.8 / 25.9 (its products run at the rate of
// mma.sync); 32 heads of 17 rows, one wave whatever the keys: D = 64, 128
// keys 3.9 / 5.6, D = 128, 128 keys 5.5 / 7.0.
bool few_keys_pay(int D, int Nk, int64_t units, int sms) {
  if (Nk > kFewKeys) return false;
  return D <= 64 || Nk <= 96 || units <= 2ll * sms;
}

// The larger of the two kernels' partial results.
size_t workspace_bytes_for(int sms, int D) {
  return std::max(stream_k_workspace_bytes(sms, D), few_rows_workspace_bytes(sms, D));
}

}  // namespace
}  // namespace fa2

using namespace fa2;

extern "C" int fa2_cross_fwd_workspace_bytes(int D, size_t* bytes) {
  if (!bytes) return FA2_ERR_INVALID_ARG;
  if (!cross_head_dim_ok(D)) return FA2_ERR_UNSUPPORTED;
  int sms = 0;
  int* status = nullptr;
  const int rc = current_device_facts(&sms, &status);
  if (rc != FA2_OK) return rc;
  *bytes = workspace_bytes_for(sms, D);
  return FA2_OK;
}

extern "C" int fa2_cross_fwd(const void* Q, const void* K, const void* V, void* O, float* LSE, const int* key_lengths,
                             int B, int Hq, int Hkv, int Nq, int Nk, int D, float scale, int dtype, void* workspace,
                             size_t workspace_bytes, struct CUstream_st* stream) {
  if (B < 0 || Hq < 0 || Hkv < 0 || Nq < 0 || Nk < 0) return FA2_ERR_INVALID_ARG;
  if (!cross_head_dim_ok(D)) return FA2_ERR_UNSUPPORTED;
  if (dtype != FA2_F16 && dtype != FA2_BF16) return FA2_ERR_UNSUPPORTED;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA2_ERR_INVALID_ARG;
  if (B == 0 || Hq == 0 || Nq == 0) return FA2_OK;
  if (Hkv == 0 || Hq % Hkv != 0) return FA2_ERR_INVALID_ARG;
  if (!Q || !O || !LSE || (Nk > 0 && (!K || !V))) return FA2_ERR_INVALID_ARG;
  const int64_t bh = static_cast<int64_t>(B) * Hkv;
  const int64_t rows = static_cast<int64_t>(Hq / Hkv) * Nq;  // query rows per key head
  const int64_t n_qt = (rows + kSubTiles * kRows - 1) / (kSubTiles * kRows);
  // 2^30: a row index plus a unit's 256 rows stays inside 32 bits
  if (rows > (1 << 30) || Nk > (1 << 30) || bh > INT32_MAX || bh * n_qt > INT32_MAX) return FA2_ERR_INVALID_ARG;
  const uintptr_t mis = reinterpret_cast<uintptr_t>(Q) | reinterpret_cast<uintptr_t>(K) |
                        reinterpret_cast<uintptr_t>(V) | reinterpret_cast<uintptr_t>(O) |
                        reinterpret_cast<uintptr_t>(LSE) | reinterpret_cast<uintptr_t>(workspace);
  if ((mis & 15u) || (reinterpret_cast<uintptr_t>(key_lengths) & 3u)) return FA2_ERR_ALIGN;
  const size_t qb = static_cast<size_t>(bh) * rows * D * 2, kb = static_cast<size_t>(bh) * Nk * D * 2;
  const size_t lb = static_cast<size_t>(bh) * rows * 4, nb = key_lengths ? static_cast<size_t>(B) * 4 : 0;
  const void* ins[4] = {Q, K, V, key_lengths};
  const size_t in_bytes[4] = {qb, kb, kb, nb};
  const void* outs[3] = {O, LSE, workspace};
  const size_t out_bytes[3] = {qb, lb, workspace ? workspace_bytes : 0};
  for (int a = 0; a < 3; ++a) {
    if (!out_bytes[a]) continue;
    for (int b = 0; b < 4; ++b)
      if (in_bytes[b] && ranges_overlap(outs[a], out_bytes[a], ins[b], in_bytes[b])) return FA2_ERR_INVALID_ARG;
    for (int b = a + 1; b < 3; ++b)
      if (out_bytes[b] && ranges_overlap(outs[a], out_bytes[a], outs[b], out_bytes[b])) return FA2_ERR_INVALID_ARG;
  }
  int sms = 0;
  int* status = nullptr;
  const int rc = current_device_facts(&sms, &status);
  if (rc != FA2_OK) return rc;
  if (workspace && workspace_bytes < workspace_bytes_for(sms, D)) return FA2_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);

  if (Nk == 0) {
    cudaError_t e = cudaMemsetAsync(O, 0, qb, s);
    if (e != cudaSuccess) return record_cuda_error(e);
    const long long n = bh * rows;
    fa2_cross_fill_lse<<<static_cast<int>(std::min<long long>((n + 255) / 256, 8ll * sms)), 256, 0, s>>>(LSE, n);
    e = cudaGetLastError();
    return e == cudaSuccess ? FA2_OK : record_cuda_error(e);
  }

  CrossRowsParams p = {};
  p.o = O;
  p.lse = LSE;
  p.status = status;
  p.watchdog_ns = watchdog_limit_ns();
  p.N = (int)rows;
  p.BH = (int)bh;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.Nk = Nk;
  p.B = B;
  p.heads = Hkv;
  p.key_lengths = key_lengths;
  char* const ws = static_cast<char*>(workspace);
  // At most 16 rows (what its products hold): the rows kernel. Measured (us,
  // rows kernel / tcgen05; the latter takes as long for 17 rows as for 16): 16
  // rows, D = 64: 8 heads of 300 keys 8.4 / 8.2, 1500 9.5 / 14.2, 16,384 15.4 /
  // 26.4; 48 heads 8.5 / 8.1, 11.7 / 15.0, 39.1 / 42.6; 512 heads of 300 keys
  // 21.1 / 24.6, 4096 89.7 / 96.2. D = 128: 8 heads of 300 keys 10.2 / 9.4, 1500
  // 12.1 / 18.1, 16,384 20.9 / 39.6; 48 heads 10.9 / 9.6, 16.6 / 18.4, 69.6 /
  // 73.3; 512 heads of 300 keys 27.9 / 29.7, 4096 172 / 172. One row is up to 20 %
  // faster than 16 on the rows kernel, the same on the other. Over at most 128
  // keys the few-keys kernel would be as fast or faster, which this rule leaves
  // aside (us, rows / few keys, 1 row): D = 64, 8 heads of 77 keys 4.6 / 4.2, 512
  // heads of 32 keys 9.0 / 4.0, 128 keys 10.2 / 8.4; D = 128, 8 heads of 128 keys
  // 5.1 / 5.5, 512 heads of 32 keys 10.2 / 6.6, 128 keys 13.3 / 13.1.
  if (workspace && rows <= kFewRows) {
    const int grid = static_cast<int>(
        std::min<long long>(std::min(sms, kFewRowsMaxCtas), bh * ((static_cast<long long>(Nk) + kFewRowsKeys - 1) / kFewRowsKeys)));
    CUtensorMap mk, mv;
    if (!encode_tile_map(&mk, K, (int)bh, Nk, D, dtype, 16u) || !encode_tile_map(&mv, V, (int)bh, Nk, D, dtype, 16u))
      return record_cuda_error(cudaErrorInvalidValue);
    p.q = Q;
    p.test_withhold = take_test_withhold();
    p.ws_o = reinterpret_cast<float*>(ws);
    p.ws_stats = p.ws_o + static_cast<size_t>(grid) * kFewRows * D;
    p.ws_flags = reinterpret_cast<unsigned long long*>(ws + few_rows_workspace_bytes(grid, D) - static_cast<size_t>(grid) * 8);
    p.epoch = next_launch_epoch();
    const cudaError_t e = launch_cross_rows(D, dtype == FA2_BF16, mk, mv, p, grid, s);
    return e == cudaSuccess ? FA2_OK : record_cuda_error(e);
  }

  const int64_t short_tiles = (rows + kFewKeysRows - 1) / kFewKeysRows;
  if (few_keys_pay(D, Nk, bh * short_tiles, sms) && bh * short_tiles <= INT32_MAX) {
    CrossShortParams sp = {};
    static_cast<CrossParams&>(sp) = p;
    sp.n_qt = (int)short_tiles;
    sp.num_units = (int)(bh * short_tiles);
    sp.q = Q;
    sp.k = K;
    sp.v = V;
    const cudaError_t e = launch_cross_short(D, dtype == FA2_BF16, sp, sms, s);
    return e == cudaSuccess ? FA2_OK : record_cuda_error(e);
  }

  CUtensorMap mq, mk, mv, mo;
  if (!encode_tile_map(&mq, Q, (int)bh, (int)rows, D, dtype, 128u) || !encode_tile_map(&mk, K, (int)bh, Nk, D, dtype, 128u) ||
      !encode_tile_map(&mv, V, (int)bh, Nk, D, dtype, 128u) || !encode_tile_map(&mo, O, (int)bh, (int)rows, D, dtype, 128u))
    return record_cuda_error(cudaErrorInvalidValue);
  p.test_withhold = take_test_withhold();
  p.n_qt = (int)n_qt;
  p.num_units = (int)(bh * n_qt);
  p.nkv_full = (Nk + kKeys - 1) / kKeys;
  p.key_split = split_keys(D, rows, p.nkv_full);
  int grid = workspace ? cross_share_ctas(D, p.key_split, p.num_units, p.nkv_full, key_lengths && B > 1, sms) : 0;
  if (grid > 0) {
    p.stream_k = 1;
    p.unit_cost = unit_cost(D, key_lengths != nullptr);
    const size_t slots = static_cast<size_t>(sms) * kSubTiles;
    p.ws_o = reinterpret_cast<float*>(ws);
    p.ws_stats = p.ws_o + slots * D * 128;
    p.ws_flags = reinterpret_cast<unsigned long long*>(
        ws + (slots * (static_cast<size_t>(D) * 128 + 3 * 128) * sizeof(float) + 255) / 256 * 256);
    p.epoch = next_launch_epoch();
  } else {
    grid = std::min(p.num_units, sms);
  }
  const cudaError_t e = pick_cross(D, dtype == FA2_BF16)(mq, mk, mv, mo, p, grid, s);
  return e == cudaSuccess ? FA2_OK : record_cuda_error(e);
}
