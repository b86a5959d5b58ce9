// Cross attention over few keys (at most 128: a caption, a handful of
// conditioning vectors) of more query rows than fa2_cross_rows.cu takes.
//
// What bounds it: the bytes of Q and O. A row's scores against all keys fit a
// warp's registers, so there is one pass, no running maximum and nothing to
// rescale; K and V of a head stay in shared memory while its rows stream by.
// On the tcgen05 kernel such a unit is one tile long and spends its time on
// hand-offs between its roles (4096 rows x 77 keys, 32 heads of 64: 21 us);
// here a warp takes 16 rows from load to store by itself, with mma.m16n8k16.
//
// Layout. Neither product needs its columns in order, so both are permuted to
// give every thread 16-byte pieces:
//   S = Q K^T: the head dimension is a sum; the 16 columns of a K-step pair
//     are dealt so that thread t of a row (lane % 4) holds elements 8 t .. 8 t
//     + 7 of 32: Q comes straight from global memory and K from shared memory
//     in 16-byte loads, with no shuffle in between. K rows are 64 bytes apart
//     modulo 128, so that the two rows a quarter warp reads share no bank.
//   O = P V: column n of the n-tile j of a group of 32 stands for element 8 (n
//     / 2) + 2 j + n % 2, by V's 4-byte words being stored in that order; the
//     accumulators then hold 8 consecutive elements of a row per thread, and O
//     goes out in 16-byte stores.
// Keys behind a batch entry's count are zeros in shared memory (never read)
// and -inf as scores.
#include <cuda_runtime.h>

#include <algorithm>

#include "fa2_cross.cuh"
#include "mma_sync.cuh"

namespace fa2 {
namespace {

constexpr int kShortThreads = 128;
// CTAs per SM to compile for: what the registers of Q, S and O (and some 30
// more) leave room for.
constexpr int short_ctas(int d, int steps) {
  const int regs = d / 4 + 8 * steps + d / 2 + 28;
  return regs <= 80 ? 6 : regs <= 100 ? 5 : regs <= 128 ? 4 : regs <= 168 ? 3 : 2;
}
static_assert(kShortThreads / 32 * 16 == kFewKeysRows, "a warp takes 16 rows of a unit");

template <int D, int kSteps>
struct ShortLayout {
  static constexpr int kKRow = D * 2 + (D * 2 % 128 == 0 ? 64 : 0);  // 64 modulo 128
  static constexpr int kVRow = D * 2 + 16;                           // an odd number of 16-byte chunks
  static constexpr int kV = kSteps * 16 * kKRow;
  static constexpr int kSmemBytes = kV + kSteps * 16 * kVRow;
  static_assert(kKRow % 128 == 64 && kVRow % 32 == 16, "bank layout");
};

// kSteps: 16-key steps, ceil(Nk / 16). Every step is computed whatever a batch
// entry's count is (its missing keys are zeros), so there are no branches.
template <int D, bool kBf16, int kSteps>
__global__ void __launch_bounds__(kShortThreads, short_ctas(D, kSteps)) fa2_cross_short_kernel(const CrossShortParams p) {
  using L = ShortLayout<D, kSteps>;
  constexpr int kGroups = D / 32;
  extern __shared__ __align__(16) uint8_t smem[];
  const uint32_t sm = smem_addr(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const float c = p.scale_log2;

  // this CTA's units (64 rows of a head), a run of consecutive ones
  const int u0 = static_cast<int>(static_cast<long long>(p.num_units) * blockIdx.x / gridDim.x);
  const int u1 = static_cast<int>(static_cast<long long>(p.num_units) * (blockIdx.x + 1) / gridDim.x);
  // Q of this warp's rows g and g + 8 of a unit: elements 32 i + 8 t ..
  auto load_q = [&](int u, uint4 (&q)[kGroups][2]) {
    const int bh = u / p.n_qt, row0 = (u - bh * p.n_qt) * kFewKeysRows + warp * 16 + g;
#pragma unroll
    for (int i = 0; i < kGroups; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = row0 + 8 * h;
        q[i][h] = row < p.N ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                                  (static_cast<size_t>(bh) * p.N + row) * D + 32 * i + 8 * t))
                            : make_uint4(0u, 0u, 0u, 0u);
      }
  };
  uint4 q[kGroups][2];
  if (u0 < u1) load_q(u0, q);
  int held = -1, n_keys = 0;
  for (int u = u0; u < u1; ++u) {
    const int bh = u / p.n_qt;
    if (bh != held) {
      if (held >= 0) __syncthreads();  // every warp is done with the head before
      held = bh;
      n_keys = cross_keys(p, bh / p.heads);
      for (int e = threadIdx.x; e < kSteps * 16 * (D / 8); e += kShortThreads) {
        const int key = e / (D / 8), ch = e - key * (D / 8);
        uint4 kk = make_uint4(0u, 0u, 0u, 0u), vv = kk;
        if (key < n_keys) {
          const size_t at = (static_cast<size_t>(bh) * p.Nk + key) * D + ch * 8;
          kk = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.k) + at));
          vv = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.v) + at));
        }
        *reinterpret_cast<uint4*>(smem + key * L::kKRow + ch * 16) = kk;
        // word j of the chunk (elements 8 (ch % 4) + 2 j) to place 4 j + ch % 4 of its group's 16 words
        uint32_t* v = reinterpret_cast<uint32_t*>(smem + L::kV + key * L::kVRow + (ch >> 2) * 64) + (ch & 3);
        v[0] = vv.x;
        v[4] = vv.y;
        v[8] = vv.z;
        v[12] = vv.w;
      }
      __syncthreads();
    }
    // S: 16 rows x 8 keys per tile
    float s[2 * kSteps][4];
#pragma unroll
    for (int nt = 0; nt < 2 * kSteps; ++nt) {
      s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        const uint4 b = *reinterpret_cast<const uint4*>(smem + (nt * 8 + g) * L::kKRow + i * 64 + t * 16);
        const uint32_t a0[4] = {q[i][0].x, q[i][1].x, q[i][0].y, q[i][1].y};
        const uint32_t a1[4] = {q[i][0].z, q[i][1].z, q[i][0].w, q[i][1].w};
        mma_16816<kBf16>(s[nt], a0, b.x, b.y);
        mma_16816<kBf16>(s[nt], a1, b.z, b.w);
      }
    }
    if (u + 1 < u1) load_q(u + 1, q);  // under way during the rest of this unit
    // rows g (h = 0) and g + 8 (h = 1): maximum, weights and their sum. The
    // base is the maximum itself, so the largest weight is exactly 1 and the
    // others' roundings, of either sign, are all that O differs by.
    float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f}, nb[2];
#pragma unroll
    for (int nt = 0; nt < 2 * kSteps; ++nt) {
      if (nt * 8 + 8 > n_keys) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (nt * 8 + 2 * t + e >= n_keys) s[nt][e] = s[nt][2 + e] = -CUDART_INF_F;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) m[h] = fmax3(m[h], s[nt][2 * h], s[nt][2 * h + 1]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      m[h] = fmaxf(m[h], __shfl_xor_sync(0xffffffffu, m[h], 1));
      m[h] = fmaxf(m[h], __shfl_xor_sync(0xffffffffu, m[h], 2)) * c;
      nb[h] = m[h] == -CUDART_INF_F ? 0.f : -m[h];
    }
    float o[D / 8][4];
#pragma unroll
    for (int d = 0; d < D / 8; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      uint32_t a[4];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x0, x1;
          ffma2_bcast(x0, x1, s[2 * k + j][2 * h], s[2 * k + j][2 * h + 1], c, nb[h]);
          const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
          l[h] += p0 + p1;
          a[2 * j + h] = pack2(p0, p1, kBf16);
        }
      // V of 16 keys: matrices (keys 0-7, 8-15) x (words 4 j .. 4 j + 3) of a group, two tiles j at a time
      const uint32_t at = sm + static_cast<uint32_t>(L::kV + (k * 16 + (lane & 15)) * L::kVRow + (lane >> 4) * 16);
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        uint32_t b[4];
        ldmatrix_x4_trans(b, at + d * 32);
        mma_16816<kBf16>(o[2 * d], a, b[0], b[1]);
        mma_16816<kBf16>(o[2 * d + 1], a, b[2], b[3]);
      }
    }
    const int row0 = (u - bh * p.n_qt) * kFewKeysRows + warp * 16 + g;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int off = 1; off < 4; off <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], off);
      const int row = row0 + 8 * h;
      if (row >= p.N) continue;
      const float inv = l[h] > 0.f ? __frcp_rn(l[h]) : 0.f;
      const size_t at = static_cast<size_t>(bh) * p.N + row;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = pack2(o[4 * i + j][2 * h] * inv, o[4 * i + j][2 * h + 1] * inv, kBf16);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + at * D + 32 * i + 8 * t) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if (t == 0) p.lse[at] = l[h] != 0.f ? (m[h] + __log2f(l[h])) * 0.69314718055994530942f : CUDART_INF_F;
    }
  }
}

template <int D, int kSteps>
cudaError_t launch_steps(const CrossShortParams& p, bool bf, int sms, cudaStream_t stream) {
  auto kern = bf ? fa2_cross_short_kernel<D, true, kSteps> : fa2_cross_short_kernel<D, false, kSteps>;
  constexpr int smem = ShortLayout<D, kSteps>::kSmemBytes;
  // Once per device: the shared-memory opt-in and how many CTAs an SM holds.
  static PerDeviceOnce prepared[2];
  static int ctas[2][kMaxDevices];
  int dev = 0, per_sm = 1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = once_per_device(prepared[bf], [&]() {
    cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (r == cudaSuccess) r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kShortThreads, smem);
    if (r == cudaSuccess && dev < kMaxDevices) ctas[bf][dev] = per_sm;
    return r;
  });
  if (e != cudaSuccess) return e;
  if (dev < kMaxDevices) per_sm = ctas[bf][dev];
  const long long grid = std::min<long long>(p.num_units, static_cast<long long>(std::max(per_sm, 1)) * sms);
  kern<<<static_cast<int>(grid), kShortThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_short(const CrossShortParams& p, bool bf, int sms, cudaStream_t s) {
  switch ((p.Nk + 15) / 16) {
    case 1: return launch_steps<D, 1>(p, bf, sms, s);
    case 2: return launch_steps<D, 2>(p, bf, sms, s);
    case 3: return launch_steps<D, 3>(p, bf, sms, s);
    case 4: return launch_steps<D, 4>(p, bf, sms, s);
    case 5: return launch_steps<D, 5>(p, bf, sms, s);
    case 6: return launch_steps<D, 6>(p, bf, sms, s);
    case 7: return launch_steps<D, 7>(p, bf, sms, s);
    default: return launch_steps<D, 8>(p, bf, sms, s);
  }
}

}  // namespace

cudaError_t launch_cross_short(int D, bool bf, const CrossShortParams& p, int sms, cudaStream_t s) {
  switch (D) {
    case 32: return launch_short<32>(p, bf, sms, s);
    case 64: return launch_short<64>(p, bf, sms, s);
    case 96: return launch_short<96>(p, bf, sms, s);
    default: return launch_short<128>(p, bf, sms, s);
  }
}

}  // namespace fa2
