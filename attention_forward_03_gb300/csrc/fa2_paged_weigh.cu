// What every cached key weighs in the softmax rows of a batch's new tokens:
//   out_j = in_j + sum over the rows i that see j of exp(scale <q_i, k_j> - LSE_i)
// for each key head, over the query heads of its group.
//
// A key's sum is one thread block's (fixed order, no atomics): a block takes
// 128 positions of one key head, each of its 8 warps 16 of them in registers as
// the B operand of mma.m16n8k16, and walks the query rows 16 at a time.
#include <cuda_runtime.h>

#include "fa2_paged.cuh"
#include "mma_sync.cuh"

namespace fa2 {
namespace {

constexpr int kWeighKeys = 128;

template <int D, bool kBf16>
__global__ void __launch_bounds__(256) fa2_paged_weigh_kernel(const PagedWeighParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c2 = 2 * (lane & 3);
  const int b = blockIdx.x / p.heads, head = blockIdx.x - b * p.heads;
  const PagedSeq s = paged_seq(p, b);
  for (int tile = blockIdx.y;; tile += gridDim.y) {
    const int key0 = tile * kWeighKeys + warp * 16;
    if (tile * kWeighKeys >= s.length) break;
    if (key0 >= s.length) continue;
    const int page = paged_entry(p, b, key0);
    if (!page_ok(p, page)) continue;
    const int slot0 = key0 & ((1 << p.page_shift) - 1);
    const uint16_t* k = static_cast<const uint16_t*>(p.k) + page * p.ks.page + head * p.ks.head + slot0 * p.ks.slot;
    uint32_t kf[D / 16][4];  // keys g and g + 8: columns (c2, c2 + 8)
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        kf[kk][i] = __ldg(reinterpret_cast<const uint32_t*>(k + (g + 8 * (i >> 1)) * p.ks.slot + kk * 16 + c2 + 8 * (i & 1)));
    float sum[4] = {0.f, 0.f, 0.f, 0.f};  // keys c2, c2 + 1, c2 + 8, c2 + 9
    const int rows = s.n * p.group;
    const int first = s.length - s.n;  // position of token 0
    const int from = p.causal ? max(key0 - first, 0) * p.group : 0;  // the first row that sees a key
    for (int r0 = from; r0 < rows; r0 += 16) {
      float sc[2][4] = {};
      uint32_t qf[D / 16][4];
      float neg[2];
      int seen[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = r0 + g + 8 * h, rr = min(r, rows - 1), token = rr / p.group, j = rr - token * p.group;
        const uint16_t* q = static_cast<const uint16_t*>(p.q) + (s.t0 + token) * p.q_token + (head * p.group + j) * p.q_head + c2;
        neg[h] = __ldg(p.lse + (static_cast<long long>(s.t0 + token) * p.heads + head) * p.group + j) * -1.4426950408889634f;
        seen[h] = r >= rows ? 0 : p.causal ? min(first + token + 1, s.length) : s.length;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
          for (int i = 0; i < 2; ++i) qf[kk][h + 2 * i] = __ldg(reinterpret_cast<const uint32_t*>(q + kk * 16 + 8 * i));
      }
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        mma_16816<kBf16>(sc[0], qf[kk], kf[kk][0], kf[kk][1]);
        mma_16816<kBf16>(sc[1], qf[kk], kf[kk][2], kf[kk][3]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = key0 + c2 + (j & 1) + 8 * (j >> 1);
          const float w = ex2_approx(fmaf(sc[j >> 1][2 * h + (j & 1)], p.scale_log2, neg[h]));
          sum[j] += key < seen[h] ? w : 0.f;
        }
    }
#pragma unroll
    for (int off = 4; off < 32; off <<= 1)
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], off);
    const long long at = ((static_cast<long long>(page) * p.heads + head) << p.page_shift) + slot0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int key = c2 + (j & 1) + 8 * (j >> 1);
      if (g == 0 && key0 + key < s.length) p.out[at + key] = (p.in ? p.in[at + key] : 0.f) + sum[j];
    }
  }
}

template <int D, bool kBf16>
cudaError_t launch(const PagedWeighParams& p, int sms, cudaStream_t s) {
  const int tiles = (p.capacity + kWeighKeys - 1) / kWeighKeys;
  const dim3 grid(p.B * p.heads, tiles < 512 ? tiles : 512);
  fa2_paged_weigh_kernel<D, kBf16><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_weigh(int D, bool bf, const PagedWeighParams& p, int sms, cudaStream_t s) {
  switch (D) {
    case 32: return bf ? launch<32, true>(p, sms, s) : launch<32, false>(p, sms, s);
    case 64: return bf ? launch<64, true>(p, sms, s) : launch<64, false>(p, sms, s);
    case 96: return bf ? launch<96, true>(p, sms, s) : launch<96, false>(p, sms, s);
    default: return bf ? launch<128, true>(p, sms, s) : launch<128, false>(p, sms, s);
  }
}

}  // namespace fa2
