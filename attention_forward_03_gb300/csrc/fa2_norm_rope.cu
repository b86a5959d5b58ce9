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
// Bytes in flight: rows come through shared memory by cp.async, 16 bytes at a
// time, and every thread reads back only what it copied itself, so there is
// no barrier and the depth costs no registers. The forward requests all rows
// of its item at once, the backward runs four rows ahead across its items.
// (Rows loaded into registers, four at a time: 37.7 us forward and 55.3 us
// backward on the shapes below, at a quarter of the warps and 45 to 57 % of
// the memory's rate.) Products run two at a time (f32x2).
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
constexpr int kMaxHeads = 8;  // a power of two

// One of the two tensors (queries or keys) of a call. Strides in elements.
struct NormRopeSide {
  const uint16_t* x;
  const uint16_t* g;   // backward: upstream gradient
  uint16_t* y;         // forward: rotated rows; backward: dx
  const void* gain;    // NULL: ones
  long long xb, xh, xn, gb, gh, gn, yb, yh, yn;
  int heads;
  int per_item;        // heads per item, a power of two
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
  int heads_per_item;  // the larger of the two sides'
  float eps;
  // backward
  float* partials;     // [grid][D] gain-gradient sums of each block
  int q_blocks;        // blocks [0, q_blocks) take the queries, the rest the keys
};

// Two fp32 values in one 64-bit register pair.
using F2 = unsigned long long;
__device__ __forceinline__ F2 pair(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void halves(F2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 swapped(F2 v) {
  float a, b;
  halves(v, a, b);
  return pair(b, a);
}
__device__ __forceinline__ float sum2(F2 v) {
  float a, b;
  halves(v, a, b);
  return a + b;
}

__device__ __forceinline__ F2 unpack2(uint32_t w, bool bf16) {
  if (bf16) return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pair(f.x, f.y);
}

__device__ __forceinline__ uint32_t pack2h(F2 v, bool bf16) {
  float lo, hi;
  halves(v, lo, hi);
  if (bf16) {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ void unpack8(const uint4& u, F2* f, bool bf16) {
  f[0] = unpack2(u.x, bf16);
  f[1] = unpack2(u.y, bf16);
  f[2] = unpack2(u.z, bf16);
  f[3] = unpack2(u.w, bf16);
}

__device__ __forceinline__ uint4 pack8(const F2* f, bool bf16) {
  return make_uint4(pack2h(f[0], bf16), pack2h(f[1], bf16), pack2h(f[2], bf16), pack2h(f[3], bf16));
}

__device__ __forceinline__ void copy_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// Gains of the 8 elements from i on (i a multiple of 8).
__device__ __forceinline__ void load_gains(const NormRopeParams& p, const void* gain, int i, float* w, bool bf16) {
  if (!gain) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.f;
  } else if (p.gain_f32) {
    const float4* g = reinterpret_cast<const float4*>(static_cast<const float*>(gain) + i);
    const float4 u = __ldg(g), v = __ldg(g + 1);
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    w[4] = v.x; w[5] = v.y; w[6] = v.z; w[7] = v.w;
  } else {
    F2 f[4];
    unpack8(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(gain) + i)), f, bf16);
#pragma unroll
    for (int e = 0; e < 4; ++e) halves(f[e], w[2 * e], w[2 * e + 1]);
  }
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

// What a pair of elements of chunk h (0: a, 1: b) is multiplied with in a
// rotation by the angle (cs, sn): out = own * cos + partner * sin_signed,
// where the partner is the same place of the other chunk (half-split) or the
// pair's other element (interleaved). i: the pair of registers, 0..3.
template <bool kInter>
__device__ __forceinline__ void angle_factors(const float* cs, const float* sn, int h, int i, float& c0, float& c1,
                                              float& s0, float& s1) {
  if (kInter) {
    c0 = c1 = cs[4 * h + i];
    s0 = -sn[4 * h + i];
    s1 = sn[4 * h + i];
  } else {
    c0 = cs[2 * i];
    c1 = cs[2 * i + 1];
    s0 = h ? sn[2 * i] : -sn[2 * i];
    s1 = h ? sn[2 * i + 1] : -sn[2 * i + 1];
  }
}

__device__ __forceinline__ long long position_of(const NormRopeParams& p, long long b, int n) {
  if (!p.positions) return n;
  const long long o = b * p.pb + n * p.pn;
  return p.positions_64 ? static_cast<const long long*>(p.positions)[o] : static_cast<const int*>(p.positions)[o];
}

// Rows a thread of the forward has under way at most (its item's heads).
template <int kPairs>
constexpr int kFwdDepth = kMaxHeads / kPairs;
// ... and of the backward (x and g of each).
template <int kPairs>
constexpr int kBwdDepth = 4 / kPairs;

// The token, the first head and the number of heads of an item. Items of one
// slice of heads are neighbouring tokens.
struct Item {
  int b, n, h0, heads;
};
__device__ __forceinline__ Item item_at(const NormRopeParams& p, const NormRopeSide& sd, unsigned item) {
  const unsigned tokens = static_cast<unsigned>(p.tokens), slice = item / tokens, t = item - slice * tokens;
  Item it;
  it.b = static_cast<int>(t / static_cast<unsigned>(p.N));
  it.n = static_cast<int>(t - static_cast<unsigned>(it.b) * p.N);
  it.h0 = static_cast<int>(slice) * sd.per_item;
  it.heads = min(sd.per_item, sd.heads - it.h0);
  return it;
}

// A row's threads: kLanes of a warp (6 of 8 at D = 96), each with kPairs
// chunk pairs. An item is one token and one slice of heads.
template <int kLanes, int kPairs, bool kBf16, bool kInter>
__global__ void __launch_bounds__(kThreadsNr) fa2_norm_rope_fwd_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int kDepth = kFwdDepth<kPairs>;
  extern __shared__ __align__(16) uint4 rows[];  // [depth][pairs][2][threads]
  const int lane = threadIdx.x % kLanes;
  const int per = p.D / 16;
  const unsigned q_items = static_cast<unsigned>(p.tokens * p.side[0].slices);
  const unsigned items = q_items + static_cast<unsigned>(p.tokens * p.side[1].slices);
  unsigned item = blockIdx.x * (kThreadsNr / kLanes) + threadIdx.x / kLanes;
  const bool live = item < items && lane < per;
  if (item >= items) item = items - 1;  // whole warps take part in the shuffles
  const bool is_k = item >= q_items;
  if (is_k) item -= q_items;
  const NormRopeSide& sd = p.side[is_k ? 1 : 0];
  const Item it = item_at(p, sd, item);
  const uint16_t* x = sd.x + it.b * sd.xb + it.n * sd.xn + it.h0 * sd.xh;
  uint16_t* y = sd.y + it.b * sd.yb + it.n * sd.yn + it.h0 * sd.yh;
  const int heads = live ? it.heads : 0;

  int oa[kPairs], ob[kPairs];
#pragma unroll
  for (int j = 0; j < kPairs; ++j) chunk_offsets<kInter>(min(lane, per - 1) + kLanes * j, p.rot, p.D, oa[j], ob[j]);
  uint4* const mine = rows + threadIdx.x;
  const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
  // two groups of copies, so that the first half's arithmetic overlaps the second half's arrival
#pragma unroll
  for (int k = 0; k < kDepth; ++k) {
    if (k < heads) {
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        copy_16(to + ((k * kPairs + j) * 2) * kThreadsNr * 16, x + k * sd.xh + oa[j]);
        copy_16(to + ((k * kPairs + j) * 2 + 1) * kThreadsNr * 16, x + k * sd.xh + ob[j]);
      }
    }
    if (k == kDepth / 2 - 1 || k == kDepth - 1) copies_commit();
  }

  // out = r * (x * own + partner * other), gain and angle in one factor each
  F2 own[kPairs][8], other[kPairs][8];
  bool rot_a[kPairs], rot_b[kPairs];
  {
    const long long pos = p.rot ? position_of(p, it.b, it.n) : 0;
    const bool pos_ok = pos >= 0 && pos < p.table_rows;
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      float cs[8], sn[8], w[16];
      load_angles<kInter>(p, pos, pos_ok, oa[j], ob[j], cs, sn);
      load_gains(p, sd.gain, oa[j], w, kBf16);
      load_gains(p, sd.gain, ob[j], w + 8, kBf16);
      rot_a[j] = oa[j] < p.rot;
      rot_b[j] = kInter ? ob[j] < p.rot : rot_a[j];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float* wo = w + 8 * h + 2 * i;                              // own gains
          const float* wp = kInter ? wo : w + 8 * (1 - h) + 2 * i;          // the partners'
          own[j][4 * h + i] = pair(wo[0], wo[1]);
          other[j][4 * h + i] = pair(0.f, 0.f);
          if (h ? rot_b[j] : rot_a[j]) {
            float c0, c1, s0, s1;
            angle_factors<kInter>(cs, sn, h, i, c0, c1, s0, s1);
            own[j][4 * h + i] = pair(wo[0] * c0, wo[1] * c1);
            other[j][4 * h + i] = kInter ? pair(wp[1] * s0, wp[0] * s1) : pair(wp[0] * s0, wp[1] * s1);
          }
        }
    }
  }
  const float inv_d = 1.f / static_cast<float>(p.D);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if (half == 0) copies_wait<1>();
    else copies_wait<0>();
#pragma unroll 2
    for (int k = half * (kDepth / 2); k < (half + 1) * (kDepth / 2); ++k) {
      if (k >= p.heads_per_item) break;  // the same for every thread: whole warps take part in the shuffles
      F2 f[kPairs][8], ss2 = pair(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
        unpack8(k < heads ? mine[((k * kPairs + j) * 2) * kThreadsNr] : z, f[j], kBf16);
        unpack8(k < heads ? mine[((k * kPairs + j) * 2 + 1) * kThreadsNr] : z, f[j] + 4, kBf16);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss2 = fma2(f[j][e], f[j][e], ss2);
      }
      float ss = sum2(ss2);
#pragma unroll
      for (int off = kLanes / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off, kLanes);
      const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
      const F2 r2 = pair(r, r);
      if (k < heads) {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          F2 o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            f[j][e] = mul2(f[j][e], r2);
            o[e] = mul2(f[j][e], own[j][e]);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e < 4 ? rot_a[j] : rot_b[j])
              o[e] = fma2(kInter ? swapped(f[j][e]) : f[j][e ^ 4], other[j][e], o[e]);
          *reinterpret_cast<uint4*>(y + k * sd.yh + oa[j]) = pack8(o, kBf16);
          *reinterpret_cast<uint4*>(y + k * sd.yh + ob[j]) = pack8(o + 4, kBf16);
        }
      }
    }
  }
}

// Backward. Blocks [0, q_blocks) walk the query items, the others the key
// items; each block leaves its sum of the gain gradient in its row of
// `partials`, which fa2_norm_rope_gain_kernel adds up in a fixed order.
template <int kLanes, int kPairs, bool kBf16, bool kInter>
__global__ void __launch_bounds__(kThreadsNr, kPairs == 1 ? 2 : 1)
    fa2_norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int kRows = kThreadsNr / kLanes;  // row groups of a block
  constexpr int kDepth = kBwdDepth<kPairs>;
  extern __shared__ __align__(16) uint4 rows[];  // [depth][pairs][x a, x b, g a, g b][threads]
  __shared__ float sums[kThreadsNr / 32][kLanes * kPairs * 16];
  const int lane = threadIdx.x % kLanes;
  const bool is_k = static_cast<int>(blockIdx.x) >= p.q_blocks;
  const NormRopeSide& sd = p.side[is_k ? 1 : 0];
  const unsigned first = is_k ? blockIdx.x - p.q_blocks : blockIdx.x;
  const unsigned blocks = is_k ? gridDim.x - p.q_blocks : p.q_blocks;
  const unsigned items = static_cast<unsigned>(p.tokens * sd.slices);
  const int per = p.D / 16;
  const float inv_d = 1.f / static_cast<float>(p.D);

  int oa[kPairs], ob[kPairs];
  F2 w[kPairs][8], dw[kPairs][8];
  bool rot_a[kPairs], rot_b[kPairs];
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
    chunk_offsets<kInter>(min(lane, per - 1) + kLanes * j, p.rot, p.D, oa[j], ob[j]);
    rot_a[j] = oa[j] < p.rot;
    rot_b[j] = kInter ? ob[j] < p.rot : rot_a[j];
    float g[16];
    load_gains(p, sd.gain, oa[j], g, kBf16);
    load_gains(p, sd.gain, ob[j], g + 8, kBf16);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[j][e] = pair(g[2 * e], g[2 * e + 1]);
      dw[j][e] = pair(0.f, 0.f);
    }
  }

  // The rows of this thread, one after the other: row u is head u % per_item
  // of its item u / per_item; the same count for every thread of the block. Rows past the items, or past an item's heads, are
  // walked without data.
  const unsigned steps = items > first * kRows ? (items - first * kRows + blocks * kRows - 1) / (blocks * kRows) : 0;
  const unsigned total = steps * sd.per_item;
  uint4* const mine = rows + threadIdx.x;
  const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
  const unsigned my_first = first * kRows + threadIdx.x / kLanes, my_stride = blocks * kRows;
  int ahead_heads = 0;  // heads of the item being requested
  int ahead_head = 0;   // its next head
  const uint16_t *ahead_x = nullptr, *ahead_g = nullptr;  // and that head's rows
  unsigned ahead_item = my_first, requested = 0;
  uint32_t ahead_at = to;  // ring slot
  auto request = [&]() {
    if (requested < total) {
      if (ahead_head == 0) {
        const bool live = ahead_item < items && lane < per;
        const Item it = item_at(p, sd, live ? ahead_item : 0u);
        ahead_heads = live ? it.heads : 0;
        ahead_x = sd.x + it.b * sd.xb + it.n * sd.xn + it.h0 * sd.xh;
        ahead_g = sd.g + it.b * sd.gb + it.n * sd.gn + it.h0 * sd.gh;
      }
      if (ahead_head < ahead_heads) {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          copy_16(ahead_at + (j * 4) * kThreadsNr * 16, ahead_x + oa[j]);
          copy_16(ahead_at + (j * 4 + 1) * kThreadsNr * 16, ahead_x + ob[j]);
          copy_16(ahead_at + (j * 4 + 2) * kThreadsNr * 16, ahead_g + oa[j]);
          copy_16(ahead_at + (j * 4 + 3) * kThreadsNr * 16, ahead_g + ob[j]);
        }
      }
      ++requested;
      ahead_x += sd.xh;
      ahead_g += sd.gh;
      ahead_at += kPairs * 4 * kThreadsNr * 16;
      if (ahead_at == to + kDepth * (kPairs * 4 * kThreadsNr * 16)) ahead_at = to;
      if (++ahead_head == sd.per_item) {
        ahead_head = 0;
        ahead_item += my_stride;
      }
    }
    copies_commit();
  };
#pragma unroll
  for (int i = 0; i < kDepth; ++i) request();

  unsigned slot = 0;
  unsigned item = my_first;
  for (unsigned step = 0; step < steps; ++step, item += my_stride) {
    const bool live = item < items && lane < per;
    const Item it = item_at(p, sd, live ? item : 0u);
    const long long pos = p.rot ? position_of(p, it.b, it.n) : 0;
    const bool pos_ok = pos >= 0 && pos < p.table_rows;
    float cs[kPairs][8], sn[kPairs][8];
#pragma unroll
    for (int j = 0; j < kPairs; ++j) load_angles<kInter>(p, pos, pos_ok, oa[j], ob[j], cs[j], sn[j]);
    uint16_t* y = sd.y + it.b * sd.yb + it.n * sd.yn + it.h0 * sd.yh;
    for (int k = 0; k < sd.per_item; ++k, y += sd.yh) {
      const bool row = live && k < it.heads;
      copies_wait<kDepth - 1>();
      F2 x[kPairs][8], h[kPairs][8], ss2 = pair(0.f, 0.f), dot2 = ss2;
      const uint4* at = mine + slot * (kPairs * 4 * kThreadsNr);
      slot = (slot + 1) % kDepth;
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        F2 g[8];
        unpack8(at[(j * 4) * kThreadsNr], x[j], kBf16);
        unpack8(at[(j * 4 + 1) * kThreadsNr], x[j] + 4, kBf16);
        unpack8(at[(j * 4 + 2) * kThreadsNr], g, kBf16);
        unpack8(at[(j * 4 + 3) * kThreadsNr], g + 4, kBf16);
        // h = R^T g: the rotation by the opposite angle
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          h[j][e] = g[e];
          if (e < 4 ? rot_a[j] : rot_b[j]) {
            float c0, c1, s0, s1;
            angle_factors<kInter>(cs[j], sn[j], e >> 2, e & 3, c0, c1, s0, s1);
            h[j][e] = fma2(kInter ? swapped(g[e]) : g[e ^ 4], pair(-s0, -s1), mul2(g[e], pair(c0, c1)));
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ss2 = fma2(x[j][e], x[j][e], ss2);
          dot2 = fma2(mul2(h[j][e], w[j][e]), x[j][e], dot2);
        }
      }
      // this thread has read its row: the slot takes the row kDepth further on
      request();
      float ss = row ? sum2(ss2) : 0.f, dot = row ? sum2(dot2) : 0.f;
#pragma unroll
      for (int off = kLanes / 2; off > 0; off >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, off, kLanes);
        dot += __shfl_xor_sync(0xffffffffu, dot, off, kLanes);
      }
      const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
      const float m = -dot * r * inv_d;  // -mean(h gain n)
      if (row) {
        const F2 r2 = pair(r, r), m2 = pair(m, m);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          F2 o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const F2 n = mul2(x[j][e], r2);
            dw[j][e] = fma2(h[j][e], n, dw[j][e]);
            o[e] = mul2(r2, fma2(n, m2, mul2(h[j][e], w[j][e])));
          }
          *reinterpret_cast<uint4*>(y + oa[j]) = pack8(o, kBf16);
          *reinterpret_cast<uint4*>(y + ob[j]) = pack8(o + 4, kBf16);
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
      float lo, hi;
      halves(dw[j][e / 2], lo, hi);
      float s = e & 1 ? hi : lo;
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

// d gain = the sum of the blocks' partials: 32 interleaved runs of blocks, each
// in block order, then the runs in theirs, the same order on every launch. One
// block per 32 elements and side. Launched as a programmatic dependent of the
// backward, which never triggers it: its blocks may start when the last of the
// backward's has exited, so that only the launch itself overlaps, and wait
// here until the partials are visible.
constexpr int kGainRuns = 32;
__global__ void __launch_bounds__(32 * kGainRuns) fa2_norm_rope_gain_kernel(const float* partials, void* dq_gain,
                                                                            void* dk_gain, int q_blocks, int blocks,
                                                                            int D, int gain_f32, int bf16) {
  __shared__ float part[kGainRuns][33];
  const bool is_k = blockIdx.y != 0;
  void* out = is_k ? dk_gain : dq_gain;
  if (!out) return;
  const int lane = threadIdx.x % 32, run = threadIdx.x / 32;
  const int i = blockIdx.x * 32 + lane;
  cudaGridDependencySynchronize();
  const int end = is_k ? blocks : q_blocks;
  float s = 0.f;
#pragma unroll 10
  for (int b = (is_k ? q_blocks : 0) + run; b < end; b += kGainRuns) s += partials[static_cast<size_t>(b) * D + i];
  part[run][lane] = s;
  __syncthreads();
  if (run != 0) return;
  s = 0.f;
#pragma unroll
  for (int k = 0; k < kGainRuns; ++k) s += part[k][lane];
  if (gain_f32)
    static_cast<float*>(out)[i] = s;
  else if (bf16)
    static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(s);
  else
    static_cast<__half*>(out)[i] = __float2half_rn(s);
}

// A kernel and its one-time set-up on each device.
struct Picked {
  const void* kern;
  PerDeviceOnce* prepared;
};

template <bool kBwd, int kLanes, int kPairs, bool kBf16, bool kInter>
Picked picked() {
  static PerDeviceOnce prepared;
  if constexpr (kBwd) return {(const void*)fa2_norm_rope_bwd_kernel<kLanes, kPairs, kBf16, kInter>, &prepared};
  else return {(const void*)fa2_norm_rope_fwd_kernel<kLanes, kPairs, kBf16, kInter>, &prepared};
}

template <bool kBwd, int kLanes, int kPairs>
Picked pick_variant(bool bf16, bool inter) {
  if (bf16) return inter ? picked<kBwd, kLanes, kPairs, true, true>() : picked<kBwd, kLanes, kPairs, true, false>();
  return inter ? picked<kBwd, kLanes, kPairs, false, true>() : picked<kBwd, kLanes, kPairs, false, false>();
}

int lanes_for(int D) { return D <= 32 ? 2 : D <= 64 ? 4 : D <= 128 ? 8 : D <= 256 ? 16 : 32; }

template <bool kBwd>
Picked pick_kernel(int D, bool bf16, bool inter) {
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
  int hp = D == 1024 ? kMaxHeads / 2 : kMaxHeads;
  const long long rows = kThreadsNr / lanes_for(D);
  while (hp > 1) {
    const long long items = tokens * ((hq + hp - 1) / hp + (hk + hp - 1) / hp);
    if (items >= 2ll * sms * rows) break;
    hp /= 2;
  }
  return hp;
}

// What forward and backward check alike.
int check_common(NormRopeArgs& a, const void* q, const void* k, const void* q_gain, const void* k_gain, const void* cos,
                 const void* sin, const void* positions, int B, int Hq, int Hkv, int N, int D, int rot, int table_rows,
                 float eps, int positions_64, int dtype) {
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
  if ((reinterpret_cast<uintptr_t>(cos) | reinterpret_cast<uintptr_t>(sin) | reinterpret_cast<uintptr_t>(q_gain) |
       reinterpret_cast<uintptr_t>(k_gain)) & 15u)
    return FA2_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(positions) & (positions_64 ? 7u : 3u)) return FA2_ERR_ALIGN;
  if (static_cast<int64_t>(B) * N > INT32_MAX) return FA2_ERR_INVALID_ARG;
  a.B = B;
  return FA2_OK;
}

View view_of(const void* p, const long long* s, int B, int H, int N, int D) {
  if (s) return View{p, s[0], s[1], s[2], B, H, N, D};
  return View{p, static_cast<long long>(H) * N * D, static_cast<long long>(N) * D, D, B, H, N, D};
}

// A dimension reaches at most 2^44 elements, so every offset stays far inside 63 bits.
bool reach_ok(long long stride, int size) { return stride >= 0 && (size < 2 || stride <= (1ll << 44) / (size - 1)); }

int check_views(const NormRopeArgs& a, bool backward) {
  for (int i = 0; i < 2; ++i) {
    const View* vs[3] = {&a.x[i], &a.y[i], &a.g[i]};
    for (int j = 0; j < (backward ? 3 : 2); ++j) {
      const View& v = *vs[j];
      if (v.empty()) continue;
      if (!v.p) return FA2_ERR_INVALID_ARG;
      if (!reach_ok(v.b, v.B) || !reach_ok(v.h, v.H) || !reach_ok(v.n, v.N)) return FA2_ERR_INVALID_ARG;
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

// What a call writes besides its views (the gains' gradients and the scratch
// of the backward): address and bytes, NULL where absent.
struct Written {
  const void* p;
  size_t n;
};

// Everything written against the plain arrays a call reads: the tables, the
// positions, the gains.
int check_arrays(const NormRopeArgs& a, const float* cos, const float* sin, const void* positions, int rot,
                 int table_rows, int gain_f32, int positions_64, long long pb, long long pn, int N, int D,
                 const Written (&more)[3]) {
  const size_t table = static_cast<size_t>(table_rows) * (rot / 2) * 4, gain = static_cast<size_t>(D) * (gain_f32 ? 4 : 2);
  if (positions && (!reach_ok(pb, a.B) || !reach_ok(pn, N))) return FA2_ERR_INVALID_ARG;
  const size_t at = positions ? static_cast<size_t>((a.B - 1) * pb + (N - 1) * pn + 1) * (positions_64 ? 8 : 4) : 0;
  auto meets_an_array = [&](const void* p, size_t n) {
    if (!p || !n) return false;
    if (rot && (ranges_overlap(p, n, cos, table) || ranges_overlap(p, n, sin, table))) return true;
    if (positions && ranges_overlap(p, n, positions, at)) return true;
    for (const void* w : a.gain)
      if (w && ranges_overlap(p, n, w, gain)) return true;
    return false;
  };
  for (const View& y : a.y)
    if (!y.empty() && meets_an_array(y.p, static_cast<size_t>(y.span()) * 2)) return FA2_ERR_INVALID_ARG;
  for (const Written& w : more)
    if (meets_an_array(w.p, w.n)) return FA2_ERR_INVALID_ARG;
  return FA2_OK;
}

void fill_params(NormRopeArgs& a, const float* cos, const float* sin, const void* positions, int Hq, int Hkv, int N,
                 int D, int rot, int table_rows, float eps, int gain_f32, int positions_64, long long pb, long long pn,
                 int sms) {
  NormRopeParams& p = a.p;
  p = {};
  const int heads[2] = {Hq, Hkv};
  p.tokens = static_cast<long long>(a.B) * N;
  const int hp = heads_per_item(p.tokens, Hq, Hkv, D, sms);
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
    s.per_item = hp;
    while (s.per_item / 2 >= std::max(heads[i], 1)) s.per_item /= 2;
    s.slices = (heads[i] + s.per_item - 1) / s.per_item;
    p.heads_per_item = std::max(p.heads_per_item, s.per_item);
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

// Blocks of the backward at most, so that the workspace's size needs no device.
constexpr int kMaxGainBlocks = 1280;

// Shared memory of a block: the rows its threads have under way.
constexpr int kRowStageBytes = kMaxHeads * 2 * kThreadsNr * 16;
static_assert(kRowStageBytes == 4 * 4 * kThreadsNr * 16, "forward and backward take the same");

int launch_kernel(const void* kern, PerDeviceOnce& prepared, int grid, NormRopeParams& p, cudaStream_t s) {
  cudaError_t e = once_per_device(prepared, [&]() {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowStageBytes);
  });
  if (e != cudaSuccess) return record_cuda_error(e);
  void* args[1] = {&p};
  e = cudaLaunchKernel(kern, dim3(grid), dim3(kThreadsNr), args, kRowStageBytes, s);
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
  int rc = check_common(a, q, k, q_gain, k_gain, cos, sin, positions, B, Hq, Hkv, N, D, rot, table_rows, eps,
                        positions_64, dtype);
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
  if ((rc = check_arrays(a, cos, sin, positions, rot, table_rows, gain_f32, positions_64, pb, pn, N, D, {})) != FA2_OK)
    return rc;
  int sms = 0;
  int* status = nullptr;
  if ((rc = current_device_facts(&sms, &status)) != FA2_OK) return rc;
  fill_params(a, cos, sin, positions, Hq, Hkv, N, D, rot, table_rows, eps, gain_f32, positions_64, pb, pn, sms);
  const long long items = a.p.tokens * (a.p.side[0].slices + a.p.side[1].slices);
  const long long rows = kThreadsNr / lanes_for(D);
  const long long grid = (items + rows - 1) / rows;
  if (items > INT32_MAX) return FA2_ERR_INVALID_ARG;  // the kernels count items in 32 bits
  const Picked kern = pick_kernel<false>(D, dtype == FA2_BF16, interleaved != 0);
  return launch_kernel(kern.kern, *kern.prepared, static_cast<int>(grid), a.p, reinterpret_cast<cudaStream_t>(stream));
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
  int rc = check_common(a, q, k, q_gain, k_gain, cos, sin, positions, B, Hq, Hkv, N, D, rot, table_rows, eps,
                        positions_64, dtype);
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
  const Written more[3] = {{dq_gain, gbytes}, {dk_gain, gbytes}, {q_gain || k_gain ? workspace : nullptr, workspace_bytes}};
  if ((rc = check_arrays(a, cos, sin, positions, rot, table_rows, gain_f32, positions_64, pb, pn, N, D, more)) != FA2_OK)
    return rc;
  const bool gains = q_gain || k_gain;
  if ((reinterpret_cast<uintptr_t>(dq_gain) | reinterpret_cast<uintptr_t>(dk_gain)) & 15u) return FA2_ERR_ALIGN;
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
      if (w && ranges_overlap(w, gbytes, workspace, workspace_bytes)) return FA2_ERR_INVALID_ARG;
    if (dq_gain && dk_gain && ranges_overlap(dq_gain, gbytes, dk_gain, gbytes)) return FA2_ERR_INVALID_ARG;
  }
  int sms = 0;
  int* status = nullptr;
  if ((rc = current_device_facts(&sms, &status)) != FA2_OK) return rc;
  fill_params(a, cos, sin, positions, Hq, Hkv, N, D, rot, table_rows, eps, gain_f32, positions_64, pb, pn, sms);
  a.p.partials = static_cast<float*>(workspace);
  // Blocks: as many as the items need, at most 2 per SM (what an SM holds;
  // each leaves one row of partial sums), dealt to queries and keys by their
  // shares of the work.
  const long long rows = kThreadsNr / lanes_for(D);
  auto need = [&](int i) { return (a.p.tokens * a.p.side[i].slices + rows - 1) / rows; };
  const long long cap = std::min<long long>(2ll * sms, kMaxGainBlocks);
  long long nq = need(0), nk = need(1);
  if (std::max(nq, nk) * rows > INT32_MAX) return FA2_ERR_INVALID_ARG;  // the kernels count items in 32 bits
  if (nq + nk > cap) {
    const long long all = nq + nk;
    nk = nk ? std::max<long long>(1, cap * nk / all) : 0;
    nq = nq ? std::max<long long>(1, cap - nk) : 0;
  }
  a.p.q_blocks = static_cast<int>(nq);
  const int grid = static_cast<int>(nq + nk);
  const Picked kern = pick_kernel<true>(D, dtype == FA2_BF16, interleaved != 0);
  if ((rc = launch_kernel(kern.kern, *kern.prepared, grid, a.p, s)) != FA2_OK) return rc;
  if (gains) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(D / 32, 2);
    cfg.blockDim = dim3(32 * kGainRuns);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fa2_norm_rope_gain_kernel, static_cast<const float*>(a.p.partials),
                                             dq_gain, dk_gain, a.p.q_blocks, grid, D, gain_f32,
                                             static_cast<int>(dtype == FA2_BF16));
    if (e != cudaSuccess) return record_cuda_error(e);
  }
  return FA2_OK;
}
