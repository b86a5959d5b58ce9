// C ABI of the cross-attention backward: argument checks, the workspace
// layout, tensor maps, the launches, and the kernels before and after the
// main one (fa2_bwd_kernel.cuh).
// Declarations and the contract: include/fa2.h.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
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

constexpr int kEndThreads = 256;
constexpr int kStatRows = kRangeRows;  // query rows a block takes at a time (divides a step's rows)
constexpr int kZeroRows = 128;  // dK, dV rows a block writes zeros to at a time

size_t round_up_256(size_t x) { return (x + 255) / 256 * 256; }

// dQ accumulator | -LSE*log2(e) | Delta | partial dV, dK of cut units | flags
struct CrossBwdWorkspace {
  size_t dq_bytes, stat_bytes, part_bytes, flag_bytes, total;
};

CrossBwdWorkspace cross_bwd_layout(int64_t bh, int64_t rows, int D) {
  const int64_t sr = bwd_step_rows(D), npad = (rows + sr - 1) / sr * sr;
  CrossBwdWorkspace w;
  w.dq_bytes = round_up_256(static_cast<size_t>(bh) * rows * D * sizeof(float));
  w.stat_bytes = round_up_256(static_cast<size_t>(bh) * npad * sizeof(float));
  w.part_bytes = round_up_256(static_cast<size_t>(kBwdMaxCtas) * 2 * D * 128 * sizeof(float));
  w.flag_bytes = round_up_256(static_cast<size_t>(kBwdMaxCtas) * sizeof(unsigned long long));
  w.total = w.dq_bytes + 2 * w.stat_bytes + w.part_bytes + w.flag_bytes;
  return w;
}

__device__ __forceinline__ uint32_t pack_two(float lo, float hi, bool bf16) {
  if (bf16) {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ float2 unpack_two(uint32_t w, bool bf16) {
  if (bf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

__device__ __forceinline__ float dot8(const uint4& x, const uint4& y, bool bf16) {
  const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack_two(a[i], bf16), g = unpack_two(b[i], bf16);
    s = fmaf(f.x, g.x, fmaf(f.y, g.y, s));
  }
  return s;
}

// x - v, element by element in 32 bits, in products with y.
__device__ __forceinline__ float dot8_diff(const uint4& x, const uint4& v, const uint4& y, bool bf16) {
  const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {v.x, v.y, v.z, v.w}, c[4] = {y.x, y.y, y.z, y.w};
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack_two(a[i], bf16), g = unpack_two(b[i], bf16), h = unpack_two(c[i], bf16);
    s = fmaf(f.x - g.x, h.x, fmaf(f.y - g.y, h.y, s));
  }
  return s;
}

// Before the main kernel. Per row of the padded [B*Hkv, Npad] grid: Delta_i =
// <dO_i, O_i> and -LSE_i * log2(e) (rows >= N: 0 and -inf, so that P is 0
// there), and the row of the fp32 dQ accumulator zeroed, where there is one.
// In a batch entry with one key, Delta_i = <dO_i, O_i - V_0>, and the main
// kernel takes V_0 as 0: dP - Delta is then what it was without the rounding
// of two sums that cancel. With the forward's own O, which is V_0 there, it is
// exactly 0; with the O and LSE of a larger softmax that the key is a part of,
// it is that part's.
// Zeros also for what no unit writes: dK and dV of tiles wholly behind their
// keys, and without an accumulator dQ of batch entries without keys. And the
// flags of the partial results taken back, so that a replay of a captured
// call, which carries the same tag, does not find them set. In fp16 also what
// a unit's scale is taken from (cross_unit_shift), into `range`.
// A block takes 64 rows of a head at a time, D/8 threads of 16 bytes per row
// in groups of a power of two, all loads of a pass before its sums.
template <int D, bool kBf16>
__global__ void __launch_bounds__(kEndThreads) fa2_cross_bwd_prologue(const uint4* __restrict__ O,
                                                                      const uint4* __restrict__ dO,
                                                                      const uint4* __restrict__ V,
                                                                      const float* __restrict__ LSE, float* neg_lse2,
                                                                      float* delta, uint4* dk, uint4* dv,
                                                                      float2* range, const CrossBwdParams p) {
  constexpr int kPer = D / 8;
  constexpr int kLanes = kPer <= 4 ? 4 : (kPer <= 8 ? 8 : 16);
  constexpr int kPasses = kStatRows * kLanes / kEndThreads;
  static_assert(kStatRows * kLanes % kEndThreads == 0, "passes");
  const int part = threadIdx.x % kLanes;
  const int tiles = p.Npad / kStatRows;
  const long long items = static_cast<long long>(p.BH) * tiles;
  const uint4 z = make_uint4(0u, 0u, 0u, 0u);
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int bh = static_cast<int>(it / tiles);
    const int r0 = static_cast<int>(it - static_cast<long long>(bh) * tiles) * kStatRows + threadIdx.x / kLanes;
    const size_t head = static_cast<size_t>(bh) * p.N;
    const bool one_key = cross_keys(p, bh / p.heads) == 1;
    uint4 x[kPasses], g[kPasses];
#pragma unroll
    for (int s = 0; s < kPasses; ++s) {
      const int r = r0 + s * (kEndThreads / kLanes);
      x[s] = g[s] = z;
      if (r < p.N && part < kPer) {
        x[s] = O[(head + r) * kPer + part];
        g[s] = dO[(head + r) * kPer + part];
      }
    }
    const uint4 v0 = one_key && part < kPer ? V[static_cast<size_t>(bh) * p.Nk * kPer + part] : z;
    [[maybe_unused]] __half2 most_do = __half2half2(__ushort_as_half(0));
    [[maybe_unused]] float most_delta = 0.f;
#pragma unroll
    for (int s = 0; s < kPasses; ++s) {
      const int r = r0 + s * (kEndThreads / kLanes);
      if (p.dq_acc && r < p.N && part < kPer) {
        uint4* to = reinterpret_cast<uint4*>(p.dq_acc) + ((head + r) * kPer + part) * 2;
        to[0] = z;
        to[1] = z;
      }
      float d = one_key ? dot8_diff(x[s], v0, g[s], kBf16) : dot8(x[s], g[s], kBf16);
#pragma unroll
      for (int off = kLanes / 2; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off, kLanes);
      if constexpr (!kBf16) {
        const uint32_t w[4] = {g[s].x, g[s].y, g[s].z, g[s].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) most_do = __hmax2(most_do, __habs2(*reinterpret_cast<const __half2*>(&w[i])));
        if (r < p.N) most_delta = fmaxf(most_delta, fabsf(d));
      }
      if (part == 0) {
        const size_t at = static_cast<size_t>(bh) * p.Npad + r;
        delta[at] = r < p.N ? d : 0.f;
        neg_lse2[at] = r < p.N ? -(LSE[head + r] * 1.4426950408889634f) : -CUDART_INF_F;
      }
    }
    if constexpr (!kBf16) {
      __shared__ uint2 warps[kEndThreads / 32];
      const float m = fmaxf(__low2float(most_do), __high2float(most_do));
      const uint2 mine = make_uint2(__reduce_max_sync(0xffffffffu, __float_as_uint(m)),
                                    __reduce_max_sync(0xffffffffu, __float_as_uint(most_delta)));
      if (threadIdx.x % 32 == 0) warps[threadIdx.x / 32] = mine;
      __syncthreads();
      if (threadIdx.x == 0) {
        uint2 all = mine;
#pragma unroll
        for (int w = 1; w < kEndThreads / 32; ++w) all = make_uint2(max(all.x, warps[w].x), max(all.y, warps[w].y));
        range[it] = make_float2(__uint_as_float(all.x), __uint_as_float(all.y));
      }
      __syncthreads();
    }
  }
  if (p.ws_flags && blockIdx.x == 0 && threadIdx.x < kBwdMaxCtas) p.ws_flags[threadIdx.x] = 0ull;
  if (!p.key_lengths) return;
  // pieces of kZeroRows rows of a head, dealt to the blocks in turn
  const int pieces = (p.Nk + kZeroRows - 1) / kZeroRows;
  const long long all = static_cast<long long>(p.BH) * pieces;
  for (long long i = blockIdx.x; i < all; i += gridDim.x) {
    const int h = static_cast<int>(i / pieces), piece = static_cast<int>(i - static_cast<long long>(h) * pieces);
    const int n_keys = cross_keys(p, h / p.heads);
    const int from = (n_keys + kKeys - 1) / kKeys * kKeys;
    const int a = max(piece * kZeroRows, from), b = min((piece + 1) * kZeroRows, p.Nk);
    const long long base = static_cast<long long>(h) * p.Nk;
    for (long long e = (base + a) * kPer + threadIdx.x; e < (base + b) * kPer; e += blockDim.x) {
      dk[e] = z;
      dv[e] = z;
    }
    if (p.dq_out && n_keys == 0 && piece == 0) {
      uint4* q = static_cast<uint4*>(p.dq_out) + static_cast<size_t>(h) * p.N * kPer;
      for (long long e = threadIdx.x; e < static_cast<long long>(p.N) * kPer; e += blockDim.x) q[e] = z;
    }
  }
}

// After the main kernel: dQ = dtype(scale * accumulator), 8 elements per thread.
template <bool kBf16>
__global__ void __launch_bounds__(kEndThreads) fa2_cross_bwd_finish(const float4* __restrict__ acc, uint4* __restrict__ dq,
                                                                    long long n8, float scale) {
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < n8; i += stride) {
    const float4 x = acc[2 * i], y = acc[2 * i + 1];
    dq[i] = make_uint4(pack_two(x.x * scale, x.y * scale, kBf16), pack_two(x.z * scale, x.w * scale, kBf16),
                       pack_two(y.x * scale, y.y * scale, kBf16), pack_two(y.z * scale, y.w * scale, kBf16));
  }
}

template <int D>
cudaError_t launch_prologue(bool bf, const void* O, const void* dO, const void* V, const float* LSE, float* neg_lse2,
                            float* delta, void* dK, void* dV, float2* range, const CrossBwdParams& p, int sms,
                            cudaStream_t s) {
  const long long items = static_cast<long long>(p.BH) * (p.Npad / kStatRows);
  const int grid = static_cast<int>(std::min<long long>(items, 8ll * sms));
  auto kern = bf ? fa2_cross_bwd_prologue<D, true> : fa2_cross_bwd_prologue<D, false>;
  kern<<<grid, kEndThreads, 0, s>>>(static_cast<const uint4*>(O), static_cast<const uint4*>(dO),
                                    static_cast<const uint4*>(V), LSE, neg_lse2, delta, static_cast<uint4*>(dK),
                                    static_cast<uint4*>(dV), range, p);
  return cudaGetLastError();
}

using CrossBwdFn = cudaError_t (*)(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                   const CUtensorMap&, const CrossBwdParams&, int, cudaStream_t);

CrossBwdFn pick_cross_bwd(int d, bool bf) {
  switch (d) {
    case 32: return bf ? launch_cross_bwd<32, true> : launch_cross_bwd<32, false>;
    case 64: return bf ? launch_cross_bwd<64, true> : launch_cross_bwd<64, false>;
    case 96: return bf ? launch_cross_bwd<96, true> : launch_cross_bwd<96, false>;
    default: return bf ? launch_cross_bwd<128, true> : launch_cross_bwd<128, false>;
  }
}

}  // namespace
}  // namespace fa2

using namespace fa2;

namespace {

int check_sizes(int B, int Hq, int Hkv, int Nq, int Nk, int D) {
  if (B < 0 || Hq < 0 || Hkv < 0 || Nq < 0 || Nk < 0) return FA2_ERR_INVALID_ARG;
  if (!bwd_head_dim_ok(D)) return FA2_ERR_UNSUPPORTED;
  if (B > 0 && Hq > 0 && (Hkv == 0 || Hq % Hkv != 0)) return FA2_ERR_INVALID_ARG;
  if (static_cast<int64_t>(B) * std::max(Hq, Hkv) > INT32_MAX) return FA2_ERR_INVALID_ARG;
  const int64_t rows = Hkv > 0 ? static_cast<int64_t>(Hq / Hkv) * Nq : 0;
  if (rows > (1 << 30) || Nk > (1 << 30)) return FA2_ERR_INVALID_ARG;
  return FA2_OK;
}

}  // namespace

extern "C" int fa2_cross_bwd_workspace_bytes(int B, int Hq, int Hkv, int Nq, int Nk, int D, size_t* bytes) {
  if (!bytes) return FA2_ERR_INVALID_ARG;
  const int rc = check_sizes(B, Hq, Hkv, Nq, Nk, D);
  if (rc != FA2_OK) return rc;
  const int64_t rows = Hkv > 0 ? static_cast<int64_t>(Hq / Hkv) * Nq : 0;
  *bytes = cross_bwd_layout(static_cast<int64_t>(B) * Hkv, rows, D).total;
  return FA2_OK;
}

extern "C" int fa2_cross_bwd(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                             const float* LSE, void* dQ, void* dK, void* dV, const int* key_lengths, int B, int Hq,
                             int Hkv, int Nq, int Nk, int D, float scale, int dtype, void* workspace,
                             size_t workspace_bytes, struct CUstream_st* stream) {
  int rc = check_sizes(B, Hq, Hkv, Nq, Nk, D);
  if (rc != FA2_OK) return rc;
  if (dtype != FA2_F16 && dtype != FA2_BF16) return FA2_ERR_UNSUPPORTED;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA2_ERR_INVALID_ARG;
  const bool has_q = B > 0 && Hq > 0 && Nq > 0, has_k = B > 0 && Hkv > 0 && Nk > 0;
  if (!has_q && !has_k) return FA2_OK;
  if ((has_q && (!Q || !O || !dO || !LSE || !dQ)) || (has_k && (!K || !V || !dK || !dV))) return FA2_ERR_INVALID_ARG;
  const uintptr_t mis = reinterpret_cast<uintptr_t>(Q) | reinterpret_cast<uintptr_t>(K) |
                        reinterpret_cast<uintptr_t>(V) | reinterpret_cast<uintptr_t>(O) |
                        reinterpret_cast<uintptr_t>(dO) | reinterpret_cast<uintptr_t>(LSE) |
                        reinterpret_cast<uintptr_t>(dQ) | reinterpret_cast<uintptr_t>(dK) |
                        reinterpret_cast<uintptr_t>(dV);
  if ((mis & 15u) || (reinterpret_cast<uintptr_t>(key_lengths) & 3u)) return FA2_ERR_ALIGN;
  const int64_t bh = static_cast<int64_t>(B) * Hkv;
  const int64_t rows = Hkv > 0 ? static_cast<int64_t>(Hq / Hkv) * Nq : 0;
  const int sr = bwd_step_rows(D);
  const int64_t npad = (rows + sr - 1) / sr * sr, nkv = (static_cast<int64_t>(Nk) + kBwdKeys - 1) / kBwdKeys;
  if (bh * nkv > INT32_MAX) return FA2_ERR_INVALID_ARG;
  const bool work = has_q && has_k;
  const CrossBwdWorkspace wl = cross_bwd_layout(bh, rows, D);
  if (work) {
    if (!workspace || workspace_bytes < wl.total) return FA2_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return FA2_ERR_ALIGN;
  }
  const size_t qb = static_cast<size_t>(bh) * rows * D * 2, kb = static_cast<size_t>(bh) * Nk * D * 2;
  const size_t lb = static_cast<size_t>(bh) * rows * 4;
  const void* ins[7] = {Q, K, V, O, dO, LSE, key_lengths};
  const size_t in_bytes[7] = {qb, kb, kb, qb, qb, lb, key_lengths ? static_cast<size_t>(B) * 4 : 0};
  const void* outs[4] = {dQ, dK, dV, workspace};
  const size_t out_bytes[4] = {qb, kb, kb, work ? workspace_bytes : 0};
  for (int a = 0; a < 4; ++a) {
    if (!out_bytes[a]) continue;
    for (int b = 0; b < 7; ++b)
      if (in_bytes[b] && ranges_overlap(outs[a], out_bytes[a], ins[b], in_bytes[b])) return FA2_ERR_INVALID_ARG;
    for (int b = a + 1; b < 4; ++b)
      if (out_bytes[b] && ranges_overlap(outs[a], out_bytes[a], outs[b], out_bytes[b])) return FA2_ERR_INVALID_ARG;
  }
  int sms = 0;
  int* status = nullptr;
  if ((rc = current_device_facts(&sms, &status)) != FA2_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (!work) {  // no query or no key: every gradient there is is zero
    if (has_q) e = cudaMemsetAsync(dQ, 0, qb, s);
    if (has_k) e = cudaMemsetAsync(dK, 0, kb, s);
    if (has_k && e == cudaSuccess) e = cudaMemsetAsync(dV, 0, kb, s);
    return e == cudaSuccess ? FA2_OK : record_cuda_error(e);
  }

  char* ws = static_cast<char*>(workspace);
  float* dq_acc = reinterpret_cast<float*>(ws);
  float* neg_lse2 = reinterpret_cast<float*>(ws + wl.dq_bytes);
  float* delta = reinterpret_cast<float*>(ws + wl.dq_bytes + wl.stat_bytes);
  CUtensorMap mk, mv, mq, mdo, mdq;
  const int n = (int)rows, ibh = (int)bh;
  if (!encode_tile_map(&mk, K, ibh, Nk, D, dtype, kBwdKeys) || !encode_tile_map(&mv, V, ibh, Nk, D, dtype, kBwdKeys) ||
      !encode_tile_map(&mq, Q, ibh, n, D, dtype, static_cast<unsigned>(sr)) ||
      !encode_tile_map(&mdo, dO, ibh, n, D, dtype, static_cast<unsigned>(sr)) ||
      !(D <= 64 ? encode_f32_cols_map_sw128(&mdq, dq_acc, ibh, n, D, 128) : encode_f32_rows_map(&mdq, dq_acc, ibh, n, D, 32)))
    return record_cuda_error(cudaErrorInvalidValue);
  const bool bf = dtype == FA2_BF16;
  CrossBwdParams p = {};
  p.dk = dK;
  p.dv = dV;
  p.dq_acc = dq_acc;
  p.neg_lse2 = neg_lse2;
  p.delta = delta;
  p.status = status;
  p.watchdog_ns = watchdog_limit_ns();
  p.N = n;
  p.Npad = (int)npad;
  p.BH = ibh;
  p.nkv = (int)nkv;
  p.nq = (int)(npad / sr);
  p.num_units = (int)(bh * nkv);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.scale = scale;
  p.Nk = Nk;
  p.B = B;
  p.heads = Hkv;
  p.key_lengths = key_lengths;
  p.test_withhold = take_test_withhold();
  const int shares = cross_bwd_share_ctas(D, p.num_units, p.nq, key_lengths && nkv > 1 && B > 1, bh * rows * D * 8,
                                          std::min(sms, kBwdMaxCtas));
  int grid = std::min(p.num_units, sms);
  if (shares > 0) {
    p.stream_k = 1;
    grid = shares;
    p.ws_part = reinterpret_cast<float*>(ws + wl.dq_bytes + 2 * wl.stat_bytes);
    p.ws_flags = reinterpret_cast<unsigned long long*>(ws + wl.dq_bytes + 2 * wl.stat_bytes + wl.part_bytes);
    p.epoch = next_launch_epoch();
  }
  // fp16's maxima, one float2 per 64 rows, lie where nothing is written before
  // the main kernel has ended: in dQ, or, where that kernel writes dQ itself, in
  // the accumulator that it then has no use for (both hold at least 64 bytes per row).
  float2* range = static_cast<float2*>(dQ);
  if (Nk <= kBwdKeys) {
    range = reinterpret_cast<float2*>(dq_acc);
    p.dq_out = dQ;
    p.dq_acc = nullptr;
  }
  p.range = range;
  switch (D) {
    case 32: e = launch_prologue<32>(bf, O, dO, V, LSE, neg_lse2, delta, dK, dV, range, p, sms, s); break;
    case 64: e = launch_prologue<64>(bf, O, dO, V, LSE, neg_lse2, delta, dK, dV, range, p, sms, s); break;
    case 96: e = launch_prologue<96>(bf, O, dO, V, LSE, neg_lse2, delta, dK, dV, range, p, sms, s); break;
    default: e = launch_prologue<128>(bf, O, dO, V, LSE, neg_lse2, delta, dK, dV, range, p, sms, s); break;
  }
  if (e != cudaSuccess) return record_cuda_error(e);
  e = pick_cross_bwd(D, bf)(mk, mv, mq, mdo, mdq, p, grid, s);
  if (e != cudaSuccess) return record_cuda_error(e);

  if (p.dq_out) return FA2_OK;
  const long long n8 = bh * rows * (D / 8);
  const int blocks = static_cast<int>(std::max<long long>(1, std::min<long long>((n8 + kEndThreads - 1) / kEndThreads, 8ll * sms)));
  auto finish = bf ? fa2_cross_bwd_finish<true> : fa2_cross_bwd_finish<false>;
  finish<<<blocks, kEndThreads, 0, s>>>(reinterpret_cast<const float4*>(dq_acc), static_cast<uint4*>(dQ), n8, scale);
  e = cudaGetLastError();
  return e == cudaSuccess ? FA2_OK : record_cuda_error(e);
}
