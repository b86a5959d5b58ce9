// The work-unit walks of cross attention on the forward and backward kernels
// (fa2_kernel.cuh, fa2_bwd_kernel.cuh): as next_segment in fa2_fwd_common.cuh
// and bwd_next_segment, with the number of K/V tiles depending on the batch
// entry's key count, which only the device knows.
//
// In the forward a batch entry without keys counts as one tile of masked
// keys: its rows then run the ordinary path and come out as O = 0, LSE = +inf.
//
// The counts are read again at every step of a walk. Should they change while
// a kernel runs (another stream writes them), a walk still ends at the last
// batch entry and touches nothing behind the tensors.
#pragma once
#include "fa2_cross.h"
#include "fa2_fwd_common.cuh"

namespace fa2 {

struct CrossSegment : Segment {
  int n_keys;  // keys of the unit's batch entry
};

// Where this CTA's stream-K share begins, found once per CTA.
struct CrossStart {
  long long total;    // steps of the whole call
  long long b_start;  // first step of batch entry b
  int b;              // batch entry that holds the share's first step
  int shares;         // CTAs with a share: min(grid, total)
  int head, tile;     // the unit with the first step: key head, query tile (forward) or K/V tile (backward)
  int from;           // steps of that unit before it
};

// Where a walk stands. It steps from unit to unit without a division and reads
// a batch entry's key count once: every role of a CTA repeats it for every
// unit, and the instructions of 64-bit divisions, fetched anew each time, and
// the read were part of what a unit costs besides its tiles (16 key heads of
// 8192 rows over up to 8192 keys, D = 128: 218 us with them, 203 without).
struct CrossCursor {
  int round;
  int b, head, tile;
  int from;    // steps of the unit already walked (by this CTA or those before it)
  int n_keys;  // of batch entry b
  long long step, end;
};

__device__ __forceinline__ int cross_tiles(int n_keys) { return max(1, (n_keys + kKeys - 1) / kKeys); }

__device__ __forceinline__ long long cross_batch_steps(const CrossParams& p, int b) {
  return static_cast<long long>(p.heads) * p.n_qt * (cross_tiles(cross_keys(p, b)) + p.unit_cost);
}

__device__ __forceinline__ long long cross_share_begin(const CrossStart& st, int c) {
  return c >= st.shares ? st.total : st.total * c / st.shares;
}

// By one whole warp: the total, then the batch entry of this CTA's first step
// (32 entries at a time: a shuffle scan of their steps). `steps(b)` are the
// steps of batch entry b, the same for all entries when `uniform`.
template <typename F>
__device__ __forceinline__ CrossStart cross_find_start(int B, bool uniform, F&& steps) {
  CrossStart st;
  const int lane = threadIdx.x & 31;
  if (uniform) {
    const long long per = steps(0);
    st.total = per * B;
    st.shares = static_cast<int>(min(static_cast<long long>(gridDim.x), st.total));
    st.b = static_cast<int>(min(cross_share_begin(st, blockIdx.x) / per, static_cast<long long>(B - 1)));
    st.b_start = per * st.b;
    return st;
  }
  long long sum = 0;
  for (int b = lane; b < B; b += 32) sum += steps(b);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  st.total = sum;
  st.shares = static_cast<int>(min(static_cast<long long>(gridDim.x), st.total));
  st.b = 0;
  st.b_start = 0;
  const long long want = cross_share_begin(st, blockIdx.x);
  long long before = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int b = b0 + lane;
    const long long mine = b < B ? steps(b) : 0;
    long long upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += v;
    }
    const unsigned past = __ballot_sync(0xffffffffu, b < B && before + upto > want);
    if (past) {
      const int l = __ffs(past) - 1;
      st.b = b0 + l;
      st.b_start = before + __shfl_sync(0xffffffffu, upto - mine, l);
      break;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return st;
}

// The forward's start; the round schedule needs none.
__device__ __forceinline__ CrossStart cross_fwd_start(const CrossParams& p) {
  if (!p.stream_k) return CrossStart{};
  CrossStart st = cross_find_start(p.B, !p.key_lengths, [&](int b) { return cross_batch_steps(p, b); });
  const int per_unit = cross_tiles(cross_keys(p, st.b)) + p.unit_cost;
  const long long r = cross_share_begin(st, blockIdx.x) - st.b_start;
  const long long unit = r / per_unit;
  st.from = static_cast<int>(r % per_unit);
  st.head = static_cast<int>(min(unit / p.n_qt, p.heads - 1ll));  // (should the counts have changed meanwhile)
  st.tile = static_cast<int>(unit % p.n_qt);
  return st;
}

template <typename P>
__device__ __forceinline__ CrossCursor cross_first_cursor(const P& p, const CrossStart& st) {
  CrossCursor c;
  c.round = 0;
  c.b = st.b;
  c.head = st.head;
  c.tile = st.tile;
  c.from = st.from;
  c.n_keys = cross_keys(p, st.b);
  c.step = p.stream_k ? cross_share_begin(st, blockIdx.x) : 0;
  c.end = p.stream_k ? cross_share_begin(st, blockIdx.x + 1) : 0;
  return c;
}

// To the next unit; a key head has `tiles` of them. Past the last one the walk ends.
template <typename P>
__device__ __forceinline__ void cross_next_unit(CrossCursor& c, int tiles, const P& p) {
  c.from = 0;
  if (++c.tile < tiles) return;
  c.tile = 0;
  if (++c.head < p.heads) return;
  c.head = 0;
  if (++c.b < p.B) c.n_keys = cross_keys(p, c.b);
  else c.step = c.end;
}

// Next segment of this CTA. Every role walks the same sequence.
__device__ __forceinline__ bool cross_next_segment(CrossCursor& c, CrossSegment& s, const CrossParams& p) {
  if (!p.stream_k) {
    const int u = c.round++ * gridDim.x + blockIdx.x;
    if (u >= p.num_units || u < 0) return false;
    s.bh = u / p.n_qt;
    s.q0 = (u - s.bh * p.n_qt) * kSubTiles * kRows;
    s.n_keys = p.key_lengths ? cross_keys(p, s.bh / p.heads) : p.Nk;
    s.nkv = cross_tiles(s.n_keys);
    s.kv_begin = 0;
    s.kv_end = s.nkv;
    s.unit_end = 0;
    return true;
  }
  // The steps of a unit: p.unit_cost that stand for no tile, then its
  // tiles. A share that ends among the first has no tile of the unit; the next
  // share then holds all of them.
  while (c.step < c.end) {
    s.n_keys = c.n_keys;
    s.nkv = cross_tiles(c.n_keys);
    s.bh = c.b * p.heads + c.head;
    s.q0 = c.tile * kSubTiles * kRows;
    const int per_unit = s.nkv + p.unit_cost, from = min(c.from, per_unit);
    const int to = static_cast<int>(min(static_cast<long long>(per_unit), from + (c.end - c.step)));
    s.unit_end = c.step - from + per_unit;
    s.kv_begin = max(from - p.unit_cost, 0);
    s.kv_end = max(to - p.unit_cost, 0);
    c.step += to - from;
    cross_next_unit(c, p.n_qt, p);  // a unit that the share's end cuts is its last
    if (s.kv_end > s.kv_begin) return true;
  }
  return false;
}

// The backward's walk: units are (key head, K/V tile), each with the nq query
// steps of the head's rows. Tiles wholly behind the keys are no units (the
// prologue writes their dK and dV, zeros).
struct CrossBwdSegment {
  int bh, kv;
  int i_begin, i_end;
  int n_keys;
  long long unit_end;  // stream-K: global step one past the unit's last step
};

__device__ __forceinline__ int cross_bwd_tiles(int n_keys) { return (n_keys + kKeys - 1) / kKeys; }

__device__ __forceinline__ long long cross_bwd_batch_steps(const CrossBwdParams& p, int b) {
  return static_cast<long long>(p.heads) * cross_bwd_tiles(cross_keys(p, b)) * p.nq;
}

__device__ __forceinline__ CrossStart cross_bwd_start(const CrossBwdParams& p) {
  if (!p.stream_k) return CrossStart{};
  CrossStart st = cross_find_start(p.B, !p.key_lengths, [&](int b) { return cross_bwd_batch_steps(p, b); });
  const int tiles = max(cross_bwd_tiles(cross_keys(p, st.b)), 1);  // 0: no batch entry has keys
  const long long r = cross_share_begin(st, blockIdx.x) - st.b_start;
  const long long unit = r / p.nq;
  st.from = static_cast<int>(r % p.nq);
  st.head = static_cast<int>(min(unit / tiles, p.heads - 1ll));
  st.tile = static_cast<int>(unit % tiles);
  return st;
}

__device__ __forceinline__ bool cross_bwd_next_segment(CrossCursor& c, CrossBwdSegment& s, const CrossBwdParams& p) {
  if (!p.stream_k) {
    for (;;) {
      const int u = c.round++ * gridDim.x + blockIdx.x;
      if (u >= p.num_units || u < 0) return false;
      s.bh = u / p.nkv;
      s.kv = u - s.bh * p.nkv;
      s.n_keys = cross_keys(p, s.bh / p.heads);
      if (s.kv < cross_bwd_tiles(s.n_keys)) break;
    }
    s.i_begin = 0;
    s.i_end = p.nq;
    s.unit_end = 0;
    return true;
  }
  while (c.step < c.end) {
    const int tiles = cross_bwd_tiles(c.n_keys);
    s.n_keys = c.n_keys;
    s.bh = c.b * p.heads + c.head;
    s.kv = c.tile;
    s.i_begin = c.from;
    s.i_end = static_cast<int>(min(static_cast<long long>(p.nq), c.from + (c.end - c.step)));
    s.unit_end = c.step - c.from + p.nq;
    const bool any = c.tile < tiles;  // not in a batch entry without keys
    if (any) c.step += s.i_end - s.i_begin;
    cross_next_unit(c, tiles, p);
    if (any) return true;
  }
  return false;
}

// fp16 in the backward. P and dS = P (dP - Delta) are rounded to 16 bits for
// their products, and with P around 1 / Nk they soon lie among the subnormals,
// below 2^-14, where a step is 2^-24 whatever the value: dO of 1e-3 and 8192
// keys left 0.6 % of dQ and dK wrong, dO of 1e-4 5 %. So a unit (a K/V tile)
// takes both 2^e times as large, by e in the exponent, and its fp32 sums 2^-e
// times (exact). e is the largest, up to 14, that dS is sure to have room for:
// |P| <= 1, |dP - Delta| <= D max |dO_id| max |V_jd| + max |Delta_i| over the
// head's query rows and the tile's keys, and 2^e times that is at most 2^15,
// half of what fp16 holds. (With normally distributed dO and V it is 2^7 times
// the usual dP, so dS keeps its 11 bits to P = 2^-21.) A NaN is none of the
// maxima; an infinity makes e 0.
// The maxima of dO and Delta come from the prologue, which reads both anyway,
// V's from the tile in shared memory. Measured (us, unscaled / scaled): 64
// heads of 1000 rows over up to 1500 keys, D = 64, 72.0 / 75.3; 8 heads of 4096
// rows x 8192 keys, D = 128, 313 / 325; 32 heads of 4096 rows x 77 keys, D = 64,
// 36.9 / 37.1; 1024 heads of 128 rows x 257 keys, D = 64, 114 / 124 (units of
// one step, where what a unit's start adds shows most). With one scale for a
// head, V read by the prologue too: a second kernel that shifts -LSE * log2(e)
// by e, 82.0 for the first of these; a cluster of blocks per head in the
// prologue, 79.2 for the first and 172 for the last.
__device__ __forceinline__ int cross_unit_shift(float bound) {
  const float room = 32768.f / bound;  // 2 at least: an exponent of at least 1
  return room >= 2.f ? min(static_cast<int>(__float_as_uint(room) >> 23) - 127, 14) : 0;
}

// Two fp32 values (their bits) times s.
__device__ __forceinline__ void cross_scale2(uint32_t& a, uint32_t& b, float s) {
  asm("{\n"
      ".reg .b64 X, S;\n"
      "mov.b64 X, {%0, %1};\n"
      "mov.b64 S, {%2, %2};\n"
      "mul.rn.f32x2 X, X, S;\n"
      "mov.b64 {%0, %1}, X;\n"
      "}\n"
      : "+r"(a), "+r"(b)
      : "f"(s));
}

// The largest absolute value in a thread's share of its row of the V tile (8 or
// 4 of the row's 16-byte chunks, in an order that spreads the rows of a quarter
// warp over the banks).
template <int kPanels>
__device__ __forceinline__ float cross_row_max(const uint8_t* tile, int row, int half) {
  __half2 m = __half2half2(__ushort_as_half(0));
#pragma unroll
  for (int i = 0; i < 4 * kPanels; ++i) {
    const int at = kPanels == 2 ? half * kPanelBytes + row * 128 + ((i ^ (row & 7)) << 4)
                                : row * 128 + (((4 * half + i) ^ (row & 7)) << 4);
    const uint4 u = *reinterpret_cast<const uint4*>(tile + at);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) m = __hmax2(m, __habs2(*reinterpret_cast<const __half2*>(&w[k])));
  }
  return fmaxf(__low2float(m), __high2float(m));
}

// A K or V tile's rows [valid, 16-row boundary) in shared memory, zeroed by
// one thread: what lies behind a batch entry's keys can be anything, and a
// product of a zero weight with a NaN is a NaN. The products that contract
// over keys stop at that boundary (cross_key_steps), so at most 16 rows of
// each 64-column panel are written. Full 128-byte rows: the swizzle moves
// bytes only within a row.
__device__ __forceinline__ int cross_key_steps(int valid) { return min(max((valid + 15) / 16, 1), kKeys / 16); }

__device__ __forceinline__ void cross_zero_rows(uint32_t tile, int panels, int valid) {
  const int end = cross_key_steps(valid) * 16;
  for (int r = max(valid, 0); r < end; ++r)
    for (int pn = 0; pn < panels; ++pn)
#pragma unroll
      for (int ch = 0; ch < 8; ++ch)
        st_shared_v4(tile + static_cast<uint32_t>(pn * kPanelBytes + r * 128 + ch * 16), 0u, 0u, 0u, 0u);
  fence_proxy_async_shared();
}

}  // namespace fa2
