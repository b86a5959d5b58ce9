// RMS norm of every query and key head with the position rotation in the same
// pass, and its gradient. Declarations and the contract: include/fa2.h.
//
// Mathematics, for one head row x of D elements at position pos:
//   r = 1 / sqrt(mean(x^2) + eps),  y = x * r * gain
//   pairs (a, b) of the first `rot` elements: (a cos - b sin, b cos + a sin)
//   with (a, b) = (y_i, y_{i + rot/2}), or (y_2i, y_2i+1) when interleaved
// and backward, for an upstream gradient g of the rotated row:
//   h = R^T g (the rotation by the opposite angle),  n = x * r
//   d gain += h * n,   dx = r * (h gain - n * mean(h gain n))
// The backward recomputes r from x, which it has to read anyway, so the
// forward keeps no statistics.
//
// What bounds it: bytes. One pass reads x and writes y (backward: reads x
// and g, writes dx) and does ~10 operations per element. So a thread holds
// 16 elements of a row (two 16-byte loads); D/16 threads make a row, and for
// the half-split rotation a thread's two chunks are the two halves of its
// pairs, so the rotation needs no exchange between threads and the norm only
// a shuffle over the row's threads. Neighbouring row groups take neighbouring
// tokens of one head: with outputs in [B, H, N, D] their writes are
// contiguous, and each row read out of a packed projection is D contiguous
// elements. A thread walks several heads of its token, so that the token's
// cos and sin (32 bits each, as many bytes as the row itself) are read once
// for all of them.
//
// Sums, r and gain gradients are held in 32 bits. The 16-bit results are
// rounded once, after the rotation.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "fa2.h"
#include "fa2_launch.h"

namespace fa2 {
namespace {

constexpr int kThreadsNr = 256;
// Heads of one token per thread at most (see heads_per_item).
constexpr int kMaxHeads = 8;

// One of the two tensors (queries or keys) of a call. Strides in elements.
struct NormRopeSide {
  const uint16_t* x;
  const uint16_t* g;   // backward: upstream gradient
  uint16_t* y;         // forward: rotated rows; backward: dx
  const void* gain;    // NULL: ones
  long long xb, xh, xn, gb, gh, gn, yb, yh, yn;
  int heads;
  int slices;          // ceil(heads / heads per item)
};

struct NormRopeParams {
  NormRopeSide side[2];
  const float* cos;    // [table_rows, rot/2]; NULL: no rotation
  const float* sin;
  const void* positions;
  long long pb, pn;    // strides of positions
  int positions_64;
  int gain_f32;
  int table_rows;
  int rot;
  int D;
  int N;
  long long tokens;    // B * N
  int heads_per_item;
  float eps;
  // backward
  float* partials;     // [grid][D] gain-gradient sums of each block
  int q_blocks;        // blocks [0, q_blocks) take the queries, the rest the keys
};

__device__ __forceinline__ void unpack2(uint32_t w, float& lo, float& hi, bool bf16) {
  if (bf16) {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xffff0000u);
  } else {
    const __half2 h = *reinterpret_cast<const __half2*>(&w);
    lo = __low2float(h);
    hi = __high2float(h);
  }
}

__device__ __forceinline__ uint32_t pack_2(float lo, float hi, bool bf16) {
  if (bf16) {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ void unpack8(const uint4& u, float* f, bool bf16) {
  unpack2(u.x, f[0], f[1], bf16);
  unpack2(u.y, f[2], f[3], bf16);
  unpack2(u.z, f[4], f[5], bf16);
  unpack2(u.w, f[6], f[7], bf16);
}

__device__ __forceinline__ uint4 pack8(const float* f, bool bf16) {
  return make_uint4(pack_2(f[0], f[1], bf16), pack_2(f[2], f[3], bf16), pack_2(f[4], f[5], bf16),
                    pack_2(f[6], f[7], bf16));
}

__device__ __forceinline__ float gain_at(const NormRopeParams& p, const void* gain, int i, bool bf16) {
  if (!gain) return 1.f;
  if (p.gain_f32) return static_cast<const float*>(gain)[i];
  const uint16_t u = static_cast<const uint16_t*>(gain)[i];
  return bf16 ? __uint_as_float(static_cast<uint32_t>(u) << 16) : __half2float(__ushort_as_half(u));
}

// The element offsets of the two 8-element chunks of chunk pair i (0 <= i <
// D/16). Half-split rotation: pair i of the first rot/16 holds elements
// 8i.. and their partners rot/2 + 8i..; the rest of the row follows in order.
// Otherwise the chunks are 8i and D/2 + 8i (contiguous over the row's threads).
template <bool kInter>
__device__ __forceinline__ void chunk_offsets(int i, int rot, int D, int& a, int& b) {
  if (!kInter && rot > 0) {
    if (i < rot / 16) {
      a = 8 * i;
      b = rot / 2 + 8 * i;
    } else {
      a = rot + 16 * (i - rot / 16);
      b = a + 8;
    }
  } else {
    a = 8 * i;
    b = D / 2 + 8 * i;
  }
}

// cos and sin of the 8 pairs of a chunk pair. `ok` false (a position outside
// the tables): NaN, so that the row's rotated elements show it.
template <bool kInter>
__device__ __forceinline__ void load_angles(const NormRopeParams& p, long long pos, bool ok, int a, int b, float* cs,
                                            float* sn) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    // half-split: pairs a..a+7; interleaved: 4 pairs of each chunk
    const int e = kInter ? (h ? b : a) : a;  // first element
    const int at = kInter ? e / 2 : e + 4 * h;
    if (e >= p.rot) continue;  // not rotated
    float4 c = make_float4(CUDART_NAN_F, CUDART_NAN_F, CUDART_NAN_F, CUDART_NAN_F), s = c;
    if (ok) {
      const size_t o = static_cast<size_t>(pos) * (p.rot / 2) + at;
      c = __ldg(reinterpret_cast<const float4*>(p.cos + o));
      s = __ldg(reinterpret_cast<const float4*>(p.sin + o));
    }
    cs[4 * h] = c.x; cs[4 * h + 1] = c.y; cs[4 * h + 2] = c.z; cs[4 * h + 3] = c.w;
    sn[4 * h] = s.x; sn[4 * h + 1] = s.y; sn[4 * h + 2] = s.z; sn[4 * h + 3] = s.w;
  }
}

// Rotates the 16 elements of a chunk pair (f[0..7] at offset a, f[8..15] at
// b) by the angles, or back (kBack).
template <bool kInter, bool kBack>
__device__ __forceinline__ void rotate16(float* f, const float* cs, const float* sn, int a, int b, int rot) {
  if (kInter) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if ((h ? b : a) >= rot) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float c = cs[4 * h + i], s = kBack ? -sn[4 * h + i] : sn[4 * h + i];
        const float x = f[8 * h + 2 * i], y = f[8 * h + 2 * i + 1];
        f[8 * h + 2 * i] = x * c - y * s;
        f[8 * h + 2 * i + 1] = y * c + x * s;
      }
    }
  } else if (a < rot) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = cs[i], s = kBack ? -sn[i] : sn[i];
      const float x = f[i], y = f[8 + i];
      f[i] = x * c - y * s;
      f[8 + i] = y * c + x * s;
    }
  }
}

__device__ __forceinline__ long long position_of(const NormRopeParams& p, long long b, int n) {
  if (!p.positions) return n;
  const long long o = b * p.pb + n * p.pn;
  return p.positions_64 ? static_cast<const long long*>(p.positions)[o] : static_cast<const int*>(p.positions)[o];
}

// A row's threads: kLanes of a warp (6 of 8 at D = 96), each with kPairs
// chunk pairs. An item is one token and one slice of heads.
template <int kLanes, int kPairs, bool kBf16, bool kInter>
__global__ void __launch_bounds__(kThreadsNr) fa2_norm_rope_fwd_kernel(const __grid_constant__ NormRopeParams p) {
  const int lane = threadIdx.x % kLanes;
  const long long q_items = p.tokens * p.side[0].slices;
  const long long items = q_items + p.tokens * p.side[1].slices;
  const int per = p.D / 16;
  long long item = (static_cast<long long>(blockIdx.x) * kThreadsNr + threadIdx.x) / kLanes;
  const bool live = item < items && lane < per;
  if (item >= items) item = items - 1;  // whole warps take part in the shuffles
  const bool is_k = item >= q_items;
  if (is_k) item -= q_items;
  const NormRopeSide& sd = p.side[is_k ? 1 : 0];
  const long long slice = item / p.tokens, t = item - slice * p.tokens;
  const long long b = t / p.N;
  const int n = static_cast<int>(t - b * p.N);
  const int h0 = static_cast<int>(slice) * p.heads_per_item, h1 = min(h0 + p.heads_per_item, sd.heads);

  int oa[kPairs], ob[kPairs];
  float cs[kPairs][8], sn[kPairs][8], w[kPairs][16];
  const long long pos = p.rot ? position_of(p, b, n) : 0;
  const bool pos_ok = pos >= 0 && pos < p.table_rows;
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
    const int i = min(lane, per - 1) + kLanes * j;
    chunk_offsets<kInter>(i, p.rot, p.D, oa[j], ob[j]);
    load_angles<kInter>(p, pos, pos_ok, oa[j], ob[j], cs[j], sn[j]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[j][e] = gain_at(p, sd.gain, oa[j] + e, kBf16);
      w[j][8 + e] = gain_at(p, sd.gain, ob[j] + e, kBf16);
    }
  }
  const uint16_t* x = sd.x + b * sd.xb + n * sd.xn;
  uint16_t* y = sd.y + b * sd.yb + n * sd.yn;
  const float inv_d = 1.f / static_cast<float>(p.D);
  // every lane of the warp runs the same number of rounds (the shuffles)
  constexpr int kUnroll = kPairs == 1 ? 4 : 2;
  for (int hb = 0; hb < p.heads_per_item; hb += kUnroll) {
    uint4 u[kUnroll][kPairs][2];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int h = h0 + hb + k;
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        u[k][j][0] = u[k][j][1] = make_uint4(0u, 0u, 0u, 0u);
        if (live && h < h1) {
          u[k][j][0] = *reinterpret_cast<const uint4*>(x + h * sd.xh + oa[j]);
          u[k][j][1] = *reinterpret_cast<const uint4*>(x + h * sd.xh + ob[j]);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int h = h0 + hb + k;
      float f[kPairs][16], ss = 0.f;
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        unpack8(u[k][j][0], f[j], kBf16);
        unpack8(u[k][j][1], f[j] + 8, kBf16);
#pragma unroll
        for (int e = 0; e < 16; ++e) ss = fmaf(f[j][e], f[j][e], ss);
      }
#pragma unroll
      for (int off = kLanes / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off, kLanes);
      const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
#pragma unroll
        for (int e = 0; e < 16; ++e) f[j][e] = f[j][e] * r * w[j][e];
        rotate16<kInter, false>(f[j], cs[j], sn[j], oa[j], ob[j], p.rot);
        if (live && h < h1) {
          *reinterpret_cast<uint4*>(y + h * sd.yh + oa[j]) = pack8(f[j], kBf16);
          *reinterpret_cast<uint4*>(y + h * sd.yh + ob[j]) = pack8(f[j] + 8, kBf16);
        }
      }
    }
  }
}

// Backward. Blocks [0, q_blocks) walk the query items, the others the key
// items; each block leaves its sum of the gain gradient in its row of
// `partials`, which fa2_norm_rope_gain_kernel adds up in a fixed order.
template <int kLanes, int kPairs, bool kBf16, bool kInter>
__global__ void __launch_bounds__(kThreadsNr) fa2_norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int kRows = kThreadsNr / kLanes;  // row groups of a block
  __shared__ float sums[kThreadsNr / 32][kLanes * kPairs * 16];
  const int lane = threadIdx.x % kLanes;
  const bool is_k = static_cast<int>(blockIdx.x) >= p.q_blocks;
  const NormRopeSide& sd = p.side[is_k ? 1 : 0];
  const long long first = is_k ? blockIdx.x - p.q_blocks : blockIdx.x;
  const long long blocks = is_k ? gridDim.x - p.q_blocks : p.q_blocks;
  const long long items = p.tokens * sd.slices;
  const int per = p.D / 16;
  const float inv_d = 1.f / static_cast<float>(p.D);

  int oa[kPairs], ob[kPairs];
  float w[kPairs][16], dw[kPairs][16];
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
    chunk_offsets<kInter>(min(lane, per - 1) + kLanes * j, p.rot, p.D, oa[j], ob[j]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[j][e] = gain_at(p, sd.gain, oa[j] + e, kBf16);
      w[j][8 + e] = gain_at(p, sd.gain, ob[j] + e, kBf16);
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) dw[j][e] = 0.f;
  }

  for (long long base = first * kRows; base < items; base += blocks * kRows) {
    long long item = base + threadIdx.x / kLanes;
    const bool live = item < items && lane < per;
    if (item >= items) item = items - 1;
    const long long slice = item / p.tokens, t = item - slice * p.tokens;
    const long long b = t / p.N;
    const int n = static_cast<int>(t - b * p.N);
    const int h0 = static_cast<int>(slice) * p.heads_per_item, h1 = min(h0 + p.heads_per_item, sd.heads);
    const long long pos = p.rot ? position_of(p, b, n) : 0;
    const bool pos_ok = pos >= 0 && pos < p.table_rows;
    float cs[kPairs][8], sn[kPairs][8];
#pragma unroll
    for (int j = 0; j < kPairs; ++j) load_angles<kInter>(p, pos, pos_ok, oa[j], ob[j], cs[j], sn[j]);
    const uint16_t* x = sd.x + b * sd.xb + n * sd.xn;
    const uint16_t* g = sd.g + b * sd.gb + n * sd.gn;
    uint16_t* y = sd.y + b * sd.yb + n * sd.yn;
    constexpr int kUnroll = kPairs == 1 ? 2 : 1;
    for (int hb = 0; hb < p.heads_per_item; hb += kUnroll) {
      uint4 u[kUnroll][kPairs][2], v[kUnroll][kPairs][2];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int h = h0 + hb + k;
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          u[k][j][0] = u[k][j][1] = v[k][j][0] = v[k][j][1] = make_uint4(0u, 0u, 0u, 0u);
          if (live && h < h1) {
            u[k][j][0] = *reinterpret_cast<const uint4*>(x + h * sd.xh + oa[j]);
            u[k][j][1] = *reinterpret_cast<const uint4*>(x + h * sd.xh + ob[j]);
            v[k][j][0] = *reinterpret_cast<const uint4*>(g + h * sd.gh + oa[j]);
            v[k][j][1] = *reinterpret_cast<const uint4*>(g + h * sd.gh + ob[j]);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int h = h0 + hb + k;
        const bool row = live && h < h1;
        float f[kPairs][16], hg[kPairs][16], ss = 0.f, dot = 0.f;
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          unpack8(u[k][j][0], f[j], kBf16);
          unpack8(u[k][j][1], f[j] + 8, kBf16);
          unpack8(v[k][j][0], hg[j], kBf16);
          unpack8(v[k][j][1], hg[j] + 8, kBf16);
          rotate16<kInter, true>(hg[j], cs[j], sn[j], oa[j], ob[j], p.rot);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            ss = fmaf(f[j][e], f[j][e], ss);
            dot = fmaf(hg[j][e] * w[j][e], f[j][e], dot);
          }
        }
        if (!row) ss = dot = 0.f;
#pragma unroll
        for (int off = kLanes / 2; off > 0; off >>= 1) {
          ss += __shfl_xor_sync(0xffffffffu, ss, off, kLanes);
          dot += __shfl_xor_sync(0xffffffffu, dot, off, kLanes);
        }
        const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
        const float m = dot * r * inv_d;  // mean(h gain n)
        if (row) {
#pragma unroll
          for (int j = 0; j < kPairs; ++j) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float nx = f[j][e] * r;
              dw[j][e] = fmaf(hg[j][e], nx, dw[j][e]);
              f[j][e] = r * (hg[j][e] * w[j][e] - nx * m);
            }
            *reinterpret_cast<uint4*>(y + h * sd.yh + oa[j]) = pack8(f[j], kBf16);
            *reinterpret_cast<uint4*>(y + h * sd.yh + ob[j]) = pack8(f[j] + 8, kBf16);
          }
        }
      }
    }
  }
  if (!sd.gain) return;  // block-uniform
  // the block's sum: over the row groups of each warp by shuffles, then over
  // the warps through shared memory
  const int warp = threadIdx.x / 32;
#pragma unroll
  for (int j = 0; j < kPairs; ++j)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float s = dw[j][e];
#pragma unroll
      for (int off = 16; off >= kLanes; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      if (threadIdx.x % 32 < kLanes) sums[warp][(j * 16 + e) * kLanes + lane] = s;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < kLanes * kPairs * 16; i += kThreadsNr) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kThreadsNr / 32; ++k) s += sums[k][i];
    const int l = i % kLanes, e = (i / kLanes) % 16, j = i / kLanes / 16;
    if (l >= per) continue;
    int a, b;
    chunk_offsets<kInter>(l + kLanes * j, p.rot, p.D, a, b);
    p.partials[static_cast<size_t>(blockIdx.x) * p.D + (e < 8 ? a + e : b + e - 8)] = s;
  }
}

// d gain = the sum of the blocks' partials, in block order for each of 8
// interleaved runs, then over the runs: the same order on every launch. One
// block per 32 elements and side.
__global__ void __launch_bounds__(kThreadsNr) fa2_norm_rope_gain_kernel(const float* __restrict__ partials, void* dq_gain,
                                                                        void* dk_gain, int q_blocks, int blocks, int D,
                                                                        int gain_f32, int bf16) {
  __shared__ float part[kThreadsNr / 32][32];
  const bool is_k = blockIdx.y != 0;
  void* out = is_k ? dk_gain : dq_gain;
  if (!out) return;
  const int lane = threadIdx.x % 32, run = threadIdx.x / 32;
  const int i = blockIdx.x * 32 + lane;
  float s = 0.f;
  for (int b = (is_k ? q_blocks : 0) + run; b < (is_k ? blocks : q_blocks); b += kThreadsNr / 32)
    s += partials[static_cast<size_t>(b) * D + i];
  part[run][lane] = s;
  __syncthreads();
  if (run != 0) return;
  for (int k = 1; k < kThreadsNr / 32; ++k) s += part[k][lane];
  if (gain_f32)
    static_cast<float*>(out)[i] = s;
  else if (bf16)
    static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(s);
  else
    static_cast<__half*>(out)[i] = __float2half_rn(s);
}

template <bool kBwd, int kLanes, int kPairs>
const void* pick_variant(bool bf16, bool inter) {
  if constexpr (kBwd) {
    if (bf16)
      return inter ? (const void*)fa2_norm_rope_bwd_kernel<kLanes, kPairs, true, true>
                   : (const void*)fa2_norm_rope_bwd_kernel<kLanes, kPairs, true, false>;
    return inter ? (const void*)fa2_norm_rope_bwd_kernel<kLanes, kPairs, false, true>
                 : (const void*)fa2_norm_rope_bwd_kernel<kLanes, kPairs, false, false>;
  } else {
    if (bf16)
      return inter ? (const void*)fa2_norm_rope_fwd_kernel<kLanes, kPairs, true, true>
                   : (const void*)fa2_norm_rope_fwd_kernel<kLanes, kPairs, true, false>;
    return inter ? (const void*)fa2_norm_rope_fwd_kernel<kLanes, kPairs, false, true>
                 : (const void*)fa2_norm_rope_fwd_kernel<kLanes, kPairs, false, false>;
  }
}

int lanes_for(int D) { return D <= 32 ? 2 : D <= 64 ? 4 : D <= 128 ? 8 : D <= 256 ? 16 : 32; }

template <bool kBwd>
const void* pick_kernel(int D, bool bf16, bool inter) {
  switch (D) {
    case 32: return pick_variant<kBwd, 2, 1>(bf16, inter);
    case 64: return pick_variant<kBwd, 4, 1>(bf16, inter);
    case 96:
    case 128: return pick_variant<kBwd, 8, 1>(bf16, inter);
    case 256: return pick_variant<kBwd, 16, 1>(bf16, inter);
    case 512: return pick_variant<kBwd, 32, 1>(bf16, inter);
    default: return pick_variant<kBwd, 32, 2>(bf16, inter);
  }
}

// A [B, H, N, D] view: base address, strides in elements (head dim contiguous).
struct View {
  const void* p;
  long long b, h, n;
  int B, H, N, D;
  bool empty() const { return B == 0 || H == 0 || N == 0; }
  long long span() const {  // elements from the first to one past the last
    return empty() ? 0 : (B - 1) * b + (H - 1) * h + (N - 1) * n + D;
  }
  bool same(const View& o) const {
    return p == o.p && (B < 2 || b == o.b) && (H < 2 || h == o.h) && (N < 2 || n == o.n) && H == o.H;
  }
};

bool aligned(const View& v) {
  return !(reinterpret_cast<uintptr_t>(v.p) & 15u) && (v.B < 2 || v.b % 8 == 0) && (v.H < 2 || v.h % 8 == 0) &&
         (v.N < 2 || v.n % 8 == 0);
}

// No two rows of the view share an element: with the dimensions sorted by
// stride, each stride reaches past everything the smaller ones span.
bool no_self_overlap(const View& v) {
  long long s[3] = {v.b, v.h, v.n};
  int d[3] = {v.B, v.H, v.N}, order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int i, int j) { return s[i] < s[j]; });
  long long reach = v.D;
  for (int i : order) {
    if (d[i] < 2) continue;
    if (s[i] < reach) return false;
    reach += (d[i] - 1) * s[i];
  }
  return true;
}

// No element in common: disjoint address ranges, or two views that interleave
// batch by batch or token by token (heads of one packed projection): equal
// batch and token strides, and both views' parts inside one batch's (token's)
// stretch without meeting.
bool disjoint(const View& a, const View& b) {
  if (a.empty() || b.empty()) return true;
  if (!ranges_overlap(a.p, a.span() * 2, b.p, b.span() * 2)) return true;
  const long long off = (static_cast<const char*>(b.p) - static_cast<const char*>(a.p)) / 2;
  if ((reinterpret_cast<uintptr_t>(a.p) ^ reinterpret_cast<uintptr_t>(b.p)) & 1u) return false;
  if ((a.B > 1 && a.b != b.b) || (a.N > 1 && a.n != b.n)) return false;
  // batch by batch: each view's heads and tokens inside one batch stride
  const long long ba = (a.H - 1) * a.h + (a.N - 1) * a.n + a.D, bb = (b.H - 1) * b.h + (b.N - 1) * b.n + b.D;
  if (off >= 0 ? (off >= ba && off + bb <= a.b) : (-off >= bb && -off + ba <= a.b)) return true;
  // token by token
  const long long wa = (a.H - 1) * a.h + a.D, wb = (b.H - 1) * b.h + b.D;  // one token's stretch of each
  if (off >= 0 ? off < wa : -off < wb) return false;
  const long long stretch = off >= 0 ? off + wb : -off + wa;  // one token's stretch of both
  long long reach = stretch;
  const bool n_first = a.N > 1 && (a.B < 2 || a.n <= a.b);
  for (int i = 0; i < 2; ++i) {
    const bool tok = (i == 0) == n_first;
    const int d = tok ? a.N : a.B;
    const long long s = tok ? a.n : a.b;
    if (d < 2) continue;
    if (s < reach) return false;
    reach += (d - 1) * s;
  }
  return true;
}

struct NormRopeArgs {
  View x[2], g[2], y[2];
  const void* gain[2];
  NormRopeParams p;
  int B;
  bool bf16, inter;
};

// Heads of one token per thread. More heads re-use the token's angles, fewer
// give a small call more threads: halved from kMaxHeads until the items fill
// two blocks per SM.
int heads_per_item(long long tokens, int hq, int hk, int D, int sms) {
  int hp = kMaxHeads;
  const long long rows = kThreadsNr / lanes_for(D);
  while (hp > 1) {
    const long long items = tokens * ((hq + hp - 1) / hp + (hk + hp - 1) / hp);
    if (items >= 2ll * sms * rows) break;
    hp /= 2;
  }
  return hp;
}

// What forward and backward check alike.
int check_common(NormRopeArgs& a, const void* q, const void* k, const void* cos, const void* sin, int B, int Hq,
                 int Hkv, int N, int D, int rot, int table_rows, float eps, int dtype) {
  if (B < 0 || Hq < 0 || Hkv < 0 || N < 0 || rot < 0 || table_rows < 0) return FA2_ERR_INVALID_ARG;
  if (!fwd_head_dim_ok(D)) return FA2_ERR_UNSUPPORTED;
  if (dtype != FA2_F16 && dtype != FA2_BF16) return FA2_ERR_UNSUPPORTED;
  if (!std::isfinite(eps) || eps < 0.f) return FA2_ERR_INVALID_ARG;
  if (rot > D) return FA2_ERR_INVALID_ARG;
  if (rot % 16 != 0) return FA2_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(Hq) + Hkv > INT32_MAX) return FA2_ERR_INVALID_ARG;
  if (B == 0 || N == 0 || (Hq == 0 && Hkv == 0)) return FA2_OK;
  if ((Hq > 0 && !q) || (Hkv > 0 && !k)) return FA2_ERR_INVALID_ARG;
  if (rot > 0 && (!cos || !sin)) return FA2_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(cos) | reinterpret_cast<uintptr_t>(sin)) & 15u) return FA2_ERR_ALIGN;
  if (static_cast<int64_t>(B) * N > INT32_MAX) return FA2_ERR_INVALID_ARG;
  a.B = B;
  return FA2_OK;
}

View view_of(const void* p, const long long* s, int B, int H, int N, int D) {
  if (s) return View{p, s[0], s[1], s[2], B, H, N, D};
  return View{p, static_cast<long long>(H) * N * D, static_cast<long long>(N) * D, D, B, H, N, D};
}

int check_views(const NormRopeArgs& a, bool backward) {
  for (int i = 0; i < 2; ++i) {
    const View* vs[3] = {&a.x[i], &a.y[i], &a.g[i]};
    for (int j = 0; j < (backward ? 3 : 2); ++j) {
      const View& v = *vs[j];
      if (v.empty()) continue;
      if (!v.p) return FA2_ERR_INVALID_ARG;
      if (v.b < 0 || v.h < 0 || v.n < 0) return FA2_ERR_INVALID_ARG;
      // every offset stays far inside 63 bits
      if (v.b > (1ll << 40) || v.h > (1ll << 40) || v.n > (1ll << 40)) return FA2_ERR_INVALID_ARG;
      if (!aligned(v)) return FA2_ERR_ALIGN;
    }
    if (!a.y[i].empty() && !no_self_overlap(a.y[i])) return FA2_ERR_INVALID_ARG;
  }
  // An output may be exactly one of its own side's inputs (each row is read
  // before it is written, by the same threads); otherwise it meets nothing.
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j) {
      if (!(i == j && a.y[i].same(a.x[j])) && !disjoint(a.y[i], a.x[j])) return FA2_ERR_INVALID_ARG;
      if (backward && !(i == j && a.y[i].same(a.g[j])) && !disjoint(a.y[i], a.g[j])) return FA2_ERR_INVALID_ARG;
    }
  if (!disjoint(a.y[0], a.y[1])) return FA2_ERR_INVALID_ARG;
  return FA2_OK;
}

// The outputs against the plain arrays a call reads.
int check_arrays(const NormRopeArgs& a, const float* cos, const float* sin, const void* positions, int rot,
                 int table_rows, int gain_f32, int positions_64, long long pb, long long pn, int N, int D) {
  const size_t table = static_cast<size_t>(table_rows) * (rot / 2) * 4, gain = static_cast<size_t>(D) * (gain_f32 ? 4 : 2);
  if (positions && (pb < 0 || pn < 0 || pb > (1ll << 40) || pn > (1ll << 40))) return FA2_ERR_INVALID_ARG;
  const size_t at = static_cast<size_t>((a.B - 1) * pb + (N - 1) * pn + 1) * (positions_64 ? 8 : 4);
  for (const View& y : a.y) {
    if (y.empty()) continue;
    const size_t n = static_cast<size_t>(y.span()) * 2;
    if (rot && (ranges_overlap(y.p, n, cos, table) || ranges_overlap(y.p, n, sin, table))) return FA2_ERR_INVALID_ARG;
    if (positions && ranges_overlap(y.p, n, positions, at)) return FA2_ERR_INVALID_ARG;
    for (const void* w : a.gain)
      if (w && ranges_overlap(y.p, n, w, gain)) return FA2_ERR_INVALID_ARG;
  }
  return FA2_OK;
}

void fill_params(NormRopeArgs& a, const float* cos, const float* sin, const void* positions, int Hq, int Hkv, int N,
                 int D, int rot, int table_rows, float eps, int gain_f32, int positions_64, long long pb, long long pn,
                 int sms) {
  NormRopeParams& p = a.p;
  p = {};
  const int heads[2] = {Hq, Hkv};
  p.tokens = static_cast<long long>(a.B) * N;
  p.heads_per_item = heads_per_item(p.tokens, Hq, Hkv, D, sms);
  for (int i = 0; i < 2; ++i) {
    NormRopeSide& s = p.side[i];
    s.x = static_cast<const uint16_t*>(a.x[i].p);
    s.g = static_cast<const uint16_t*>(a.g[i].p);
    s.y = static_cast<uint16_t*>(const_cast<void*>(a.y[i].p));
    s.gain = a.gain[i];
    s.xb = a.x[i].b; s.xh = a.x[i].h; s.xn = a.x[i].n;
    s.gb = a.g[i].b; s.gh = a.g[i].h; s.gn = a.g[i].n;
    s.yb = a.y[i].b; s.yh = a.y[i].h; s.yn = a.y[i].n;
    s.heads = heads[i];
    s.slices = (heads[i] + p.heads_per_item - 1) / p.heads_per_item;
  }
  p.cos = cos;
  p.sin = sin;
  p.positions = positions;
  p.pb = pb;
  p.pn = pn;
  p.positions_64 = positions_64;
  p.gain_f32 = gain_f32;
  p.table_rows = table_rows;
  p.rot = rot;
  p.D = D;
  p.N = N;
  p.eps = eps;
}

// Blocks of the backward at most: 8 per SM of a 160-SM device, so that the
// workspace's size needs no device.
constexpr int kMaxGainBlocks = 1280;

int launch_kernel(const void* kern, int grid, NormRopeParams& p, cudaStream_t s) {
  void* args[1] = {&p};
  const cudaError_t e = cudaLaunchKernel(kern, dim3(grid), dim3(kThreadsNr), args, 0, s);
  return e == cudaSuccess ? FA2_OK : record_cuda_error(e);
}

}  // namespace
}  // namespace fa2

using namespace fa2;

extern "C" int fa2_qk_norm_rope_fwd(const void* q, const void* k, const void* q_gain, const void* k_gain,
                                    const float* cos, const float* sin, const void* positions, void* q_out,
                                    void* k_out, const long long* strides, int B, int Hq, int Hkv, int N, int D,
                                    int rot, int table_rows, float eps, int interleaved, int gain_f32,
                                    int positions_64, int dtype, struct CUstream_st* stream) {
  NormRopeArgs a = {};
  int rc = check_common(a, q, k, cos, sin, B, Hq, Hkv, N, D, rot, table_rows, eps, dtype);
  if (rc != FA2_OK || B == 0 || N == 0 || (Hq == 0 && Hkv == 0)) return rc;
  if (rot > 0 && !positions && table_rows < N) return FA2_ERR_INVALID_ARG;
  a.x[0] = view_of(q, strides, B, Hq, N, D);
  a.x[1] = view_of(k, strides ? strides + 3 : nullptr, B, Hkv, N, D);
  a.y[0] = view_of(q_out, strides ? strides + 6 : nullptr, B, Hq, N, D);
  a.y[1] = view_of(k_out, strides ? strides + 9 : nullptr, B, Hkv, N, D);
  a.gain[0] = q_gain;
  a.gain[1] = k_gain;
  const long long pb = strides ? strides[12] : N, pn = strides ? strides[13] : 1;
  if ((rc = check_views(a, false)) != FA2_OK) return rc;
  if ((rc = check_arrays(a, cos, sin, positions, rot, table_rows, gain_f32, positions_64, pb, pn, N, D)) != FA2_OK)
    return rc;
  int sms = 0;
  int* status = nullptr;
  if ((rc = current_device_facts(&sms, &status)) != FA2_OK) return rc;
  fill_params(a, cos, sin, positions, Hq, Hkv, N, D, rot, table_rows, eps, gain_f32, positions_64, pb, pn, sms);
  const long long items = a.p.tokens * (a.p.side[0].slices + a.p.side[1].slices);
  const long long rows = kThreadsNr / lanes_for(D);
  const long long grid = (items + rows - 1) / rows;
  if (grid > INT32_MAX) return FA2_ERR_INVALID_ARG;
  return launch_kernel(pick_kernel<false>(D, dtype == FA2_BF16, interleaved != 0), static_cast<int>(grid), a.p,
                       reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int fa2_qk_norm_rope_bwd_workspace_bytes(int D, size_t* bytes) {
  if (!bytes) return FA2_ERR_INVALID_ARG;
  if (!fwd_head_dim_ok(D)) return FA2_ERR_UNSUPPORTED;
  *bytes = static_cast<size_t>(kMaxGainBlocks) * D * sizeof(float);
  return FA2_OK;
}

extern "C" int fa2_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q, const void* k,
                                    const void* q_gain, const void* k_gain, const float* cos, const float* sin,
                                    const void* positions, void* dq, void* dk, void* dq_gain, void* dk_gain,
                                    const long long* strides, int B, int Hq, int Hkv, int N, int D, int rot,
                                    int table_rows, float eps, int interleaved, int gain_f32, int positions_64,
                                    int dtype, void* workspace, size_t workspace_bytes, struct CUstream_st* stream) {
  NormRopeArgs a = {};
  int rc = check_common(a, q, k, cos, sin, B, Hq, Hkv, N, D, rot, table_rows, eps, dtype);
  if (rc != FA2_OK) return rc;
  const size_t gbytes = static_cast<size_t>(D) * (gain_f32 ? 4 : 2);
  // a gain's gradient is written exactly where there is a gain
  if (!q_gain != !dq_gain || !k_gain != !dk_gain) return FA2_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (B == 0 || N == 0 || (Hq == 0 && Hkv == 0)) {  // a sum over nothing
    for (void* w : {dq_gain, dk_gain})
      if (w) {
        const cudaError_t e = cudaMemsetAsync(w, 0, gbytes, s);
        if (e != cudaSuccess) return record_cuda_error(e);
      }
    return FA2_OK;
  }
  if (rot > 0 && !positions && table_rows < N) return FA2_ERR_INVALID_ARG;
  a.g[0] = view_of(dq_out, strides, B, Hq, N, D);
  a.g[1] = view_of(dk_out, strides ? strides + 3 : nullptr, B, Hkv, N, D);
  a.x[0] = view_of(q, strides ? strides + 6 : nullptr, B, Hq, N, D);
  a.x[1] = view_of(k, strides ? strides + 9 : nullptr, B, Hkv, N, D);
  a.y[0] = view_of(dq, strides ? strides + 12 : nullptr, B, Hq, N, D);
  a.y[1] = view_of(dk, strides ? strides + 15 : nullptr, B, Hkv, N, D);
  a.gain[0] = q_gain;
  a.gain[1] = k_gain;
  const long long pb = strides ? strides[18] : N, pn = strides ? strides[19] : 1;
  if ((rc = check_views(a, true)) != FA2_OK) return rc;
  if ((rc = check_arrays(a, cos, sin, positions, rot, table_rows, gain_f32, positions_64, pb, pn, N, D)) != FA2_OK)
    return rc;
  const bool gains = q_gain || k_gain;
  if (gains) {
    if (!workspace) return FA2_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(workspace) & 15u) return FA2_ERR_ALIGN;
    if (workspace_bytes < static_cast<size_t>(kMaxGainBlocks) * D * sizeof(float)) return FA2_ERR_INVALID_ARG;
    for (int i = 0; i < 2; ++i)
      for (const View* v : {&a.x[i], &a.g[i], &a.y[i]})
        if (!v->empty()) {
          const size_t n = static_cast<size_t>(v->span()) * 2;
          if (ranges_overlap(workspace, workspace_bytes, v->p, n)) return FA2_ERR_INVALID_ARG;
          for (void* w : {dq_gain, dk_gain})
            if (w && ranges_overlap(w, gbytes, v->p, n)) return FA2_ERR_INVALID_ARG;
        }
    for (void* w : {dq_gain, dk_gain})
      if (w && (ranges_overlap(w, gbytes, workspace, workspace_bytes) ||
                (q_gain && ranges_overlap(w, gbytes, q_gain, gbytes)) ||
                (k_gain && ranges_overlap(w, gbytes, k_gain, gbytes))))
        return FA2_ERR_INVALID_ARG;
    if (dq_gain && dk_gain && ranges_overlap(dq_gain, gbytes, dk_gain, gbytes)) return FA2_ERR_INVALID_ARG;
  }
  int sms = 0;
  int* status = nullptr;
  if ((rc = current_device_facts(&sms, &status)) != FA2_OK) return rc;
  fill_params(a, cos, sin, positions, Hq, Hkv, N, D, rot, table_rows, eps, gain_f32, positions_64, pb, pn, sms);
  a.p.partials = static_cast<float*>(workspace);
  // Blocks: as many as the items need, at most 4 per SM (each leaves one row
  // of partial sums), dealt to queries and keys by their shares of the work.
  const long long rows = kThreadsNr / lanes_for(D);
  auto need = [&](int i) { return (a.p.tokens * a.p.side[i].slices + rows - 1) / rows; };
  const long long cap = std::min<long long>(4ll * sms, kMaxGainBlocks);
  long long nq = need(0), nk = need(1);
  if (nq + nk > cap) {
    const long long all = nq + nk;
    nk = nk ? std::max<long long>(1, cap * nk / all) : 0;
    nq = nq ? std::max<long long>(1, cap - nk) : 0;
  }
  a.p.q_blocks = static_cast<int>(nq);
  const int grid = static_cast<int>(nq + nk);
  if ((rc = launch_kernel(pick_kernel<true>(D, dtype == FA2_BF16, interleaved != 0), grid, a.p, s)) != FA2_OK)
    return rc;
  if (gains) {
    fa2_norm_rope_gain_kernel<<<dim3(D / 32, 2), kThreadsNr, 0, s>>>(a.p.partials, dq_gain, dk_gain, a.p.q_blocks,
                                                                      grid, D, gain_f32, dtype == FA2_BF16);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return record_cuda_error(e);
  }
  return FA2_OK;
}
