// What every cached key weighs in the softmax rows of a batch's new tokens:
//   out_j = in_j + sum over the rows i that see j of exp(scale <q_i, k_j> - LSE_i)
// for each key head, over the query heads of its group.
//
// The products are taken the other way round from attention, S^T = K Q^T: 128
// positions are the lanes of tensor memory and the query rows its columns. So a
// thread holds one key, its sum needs no other thread, and nothing goes back to
// the tensor cores. A key's sum is one CTA's, in a fixed order.
//
// What bounds it: with single tokens the bytes of K (each tile of 128
// positions meets a handful of rows); with a chunk of tokens the exponentials,
// one per product of a row and a key, as many cycles as the products take at
// D = 128 (16,384 of either kind's 128 x 128 step: 512 cycles of a special
// function unit, 512 of the tensor core).
//
// One CTA per SM. Work: units (a sequence's tile of 128 positions, of one key
// head) in the order (sequence, key head, tile), each with as many steps as
// there are blocks of query rows that see a key of it; every CTA takes the units
// that begin in its equal share of all steps.
//   warps 0-7   two warpgroups that take the steps in turn: thread = key
//   warps 8, 9  one thread each issues the products of one warpgroup's steps
//   warp  10    loads: K tiles (one box per page) and blocks of query rows, in
//               rings of their own
// A block of query rows is up to 128 / group tokens with all heads of the
// group (of more than 128 heads: one token, 128 heads). Where all rows of a
// sequence fit into one block it stays for all tiles of a key head. Four S^T
// buffers of 128 columns in tensor memory, two per warpgroup. The rows' LSE are
// laid out once per warp and step in shared memory, as factors of the
// exponent. A unit's sum of the warpgroup that did not take its last step goes
// through shared memory to the other, which writes.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "fa2_paged_walk.cuh"

namespace fa2 {
namespace {

enum : int {
  kSiteWeighKEmpty = 61,
  kSiteWeighQEmpty = 62,
  kSiteWeighKFull = 63,
  kSiteWeighQFull = 64,
  kSiteWeighSFree = 65,
  kSiteWeighSFull = 66,
  kSiteWeighPart = 67,
  kSiteWeighTaken = 68,
  kSiteWeighDrain = 69,
};

// Steps of a unit besides those of its blocks: loads that wait, the sum's way out.
constexpr int kWeighUnitCost = 1;

// Blocks of one key head's query rows, tiles and steps of a sequence.
struct WeighSeq {
  PagedSeq s;
  int tiles;   // units per key head
  int blocks;  // blocks of query rows
};

__device__ __forceinline__ WeighSeq weigh_seq(const PagedWeighParams& p, int b) {
  WeighSeq w;
  w.s = paged_seq(p, b);
  w.blocks = (w.s.n + p.block_tokens - 1) / p.block_tokens * p.head_blocks;
  // without new tokens the weights stay: nothing to do in place
  w.tiles = w.blocks == 0 && p.in == p.out ? 0 : (w.s.length + kKeys - 1) / kKeys;
  return w;
}

// The first block with a row that sees a position of the tile: that of the
// token that stands at the tile's first position.
__device__ __forceinline__ int first_block(const PagedWeighParams& p, const WeighSeq& w, int tile) {
  return p.causal ? max(tile * kKeys - (w.s.length - w.s.n), 0) / p.block_tokens * p.head_blocks : 0;
}

// Steps of the first m tiles of a key head.
__device__ __forceinline__ long long weigh_before(const PagedWeighParams& p, const WeighSeq& w, int m) {
  long long steps = static_cast<long long>(m) * (w.blocks + kWeighUnitCost);
  if (p.causal && w.blocks) {
    const int c = w.s.length - w.s.n, j0 = c > 0 ? (c + kKeys - 1) / kKeys : 0;
    if (m > j0)
      steps -= p.head_blocks * floor_sum(static_cast<unsigned>(m - j0), static_cast<unsigned>(p.block_tokens), kKeys,
                                         static_cast<unsigned>(j0 * kKeys - c));
  }
  return steps;
}

// The first unit that begins in this CTA's share, and the shares' ends.
struct WeighStart {
  long long step, end;
  int b, head, tile;
};

__device__ __forceinline__ WeighStart weigh_start(const PagedWeighParams& p) {
  WeighStart st = {};
  const int lane = threadIdx.x & 31;
  long long sum = 0;
  for (int b = lane; b < p.B; b += 32) {
    const WeighSeq w = weigh_seq(p, b);
    sum += p.heads * weigh_before(p, w, w.tiles);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  const long long want = sum * blockIdx.x / gridDim.x;
  st.end = sum * (blockIdx.x + 1) / gridDim.x;
  st.step = st.end;  // none
  if (want >= st.end) return st;
  long long before = 0;
  st.b = -1;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    long long mine = 0;
    if (b < p.B) {
      const WeighSeq w = weigh_seq(p, b);
      mine = p.heads * weigh_before(p, w, w.tiles);
    }
    long long upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += v;
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + upto > want);
    if (past) {
      const int l = __ffs(past) - 1;
      st.b = b0 + l;
      before += __shfl_sync(0xffffffffu, upto - mine, l);
      break;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  if (st.b < 0) return st;
  const WeighSeq w = weigh_seq(p, st.b);
  if (w.tiles == 0) return st;  // only should the tables have changed meanwhile
  const long long per_head = weigh_before(p, w, w.tiles);
  const long long r0 = want - before;
  st.head = static_cast<int>(min(r0 / per_head, p.heads - 1ll));
  const long long r = r0 - st.head * per_head;
  // the last tile that begins at or before step r, 32 candidates at a time
  int lo = 0, hi = w.tiles;
  while (hi - lo > 1) {
    const int by = (hi - lo + 31) / 32, m = lo + (lane + 1) * by;
    const bool ok = m < hi && weigh_before(p, w, m) <= r;
    lo += __popc(__ballot_sync(0xffffffffu, ok)) * by;
    hi = min(hi, lo + by);
  }
  long long at = weigh_before(p, w, lo);
  if (at < r) at = weigh_before(p, w, ++lo);  // it began in an earlier share
  st.tile = lo;
  st.step = want - r + at;
  return st;  // (tile == tiles: the walk goes on to the next key head)
}

struct WeighCursor {
  WeighSeq w;
  int b, head, tile;
  long long step, end;
};

struct WeighUnit {
  int b, head, tile;
  int first, blocks;  // blocks of query rows [first, blocks)
  bool new_rows;      // of another sequence or key head than the unit before
  PagedSeq s;
};

__device__ __forceinline__ WeighCursor weigh_cursor(const PagedWeighParams& p, const WeighStart& st) {
  WeighCursor c;
  c.b = st.b;
  c.head = st.head;
  c.tile = st.tile;
  c.step = st.step;
  c.end = st.end;
  if (c.step < c.end) c.w = weigh_seq(p, c.b);
  return c;
}

// Next unit of this CTA; every role walks the same sequence.
__device__ __forceinline__ bool weigh_next(WeighCursor& c, WeighUnit& u, bool first_unit, const PagedWeighParams& p) {
  if (c.step >= c.end) return false;
  u.new_rows = first_unit;
  if (c.tile >= c.w.tiles) {
    u.new_rows = true;
    c.tile = 0;
    if (++c.head >= p.heads) {
      c.head = 0;
      do {
        if (++c.b >= p.B) {
          c.step = c.end;
          return false;
        }
        c.w = weigh_seq(p, c.b);
      } while (c.w.tiles == 0);
    }
  }
  u.b = c.b;
  u.head = c.head;
  u.tile = c.tile;
  u.s = c.w.s;
  u.blocks = c.w.blocks;
  u.first = min(first_block(p, c.w, c.tile), u.blocks);
  c.step += u.blocks - u.first + kWeighUnitCost;
  ++c.tile;
  return true;
}

template <int D>
struct WeighLayout {
  static constexpr int kPanels = (D + 63) / 64;
  static constexpr int kTileBytes = kPanels * kPanelBytes;
  static constexpr int kSmallRows = 32;  // blocks of at most so many rows: more room for K
  static constexpr int kSmallBytes = kPanels * kSmallRows * 128;
  // stages of K and Q, with blocks of up to 128 rows and with small ones
  static constexpr int kK = kPanels == 2 ? 4 : 8, kQ = kPanels == 2 ? 2 : 4;
  static constexpr int kKSmall = kPanels == 2 ? 6 : 12, kQSmall = kPanels == 2 ? 3 : 6;
  static constexpr int kMostK = kKSmall, kMostQ = kQ > kQSmall ? kQ : kQSmall;
  static constexpr int kWide = kK * kTileBytes + kQ * kTileBytes;
  static constexpr int kNarrow = kKSmall * kTileBytes + kQSmall * kSmallBytes;
  static constexpr int kLseOffset = kWide > kNarrow ? kWide : kNarrow;  // [8 warps][128] floats
  static constexpr int kPartOffset = kLseOffset + 8 * 128 * 4;          // [2][128] floats
  static constexpr int kBarOffset = kPartOffset + 2 * 128 * 4;
  // k_full, k_empty [K], q_full, q_empty [Q], s_full[4], s_free[4], part[2], taken[2], drain[2]
  static constexpr int kNumBars = 2 * kMostK + 2 * kMostQ + 14;
  static constexpr int kMiscOffset = kBarOffset + kNumBars * 8;
  static constexpr int kStartOffset = kMiscOffset + 16;
  static constexpr int kSmemBytes = kStartOffset + static_cast<int>(sizeof(WeighStart)) + 1024;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
  static_assert(kStartOffset % alignof(WeighStart) == 0, "alignment");
};

template <int D, bool kBf16>
__global__ void __launch_bounds__(kThreads, 1)
    fa2_paged_weigh_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const PagedWeighParams p) {
  using L = WeighLayout<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const bool small = p.columns <= L::kSmallRows;
  const int k_stages = small ? L::kKSmall : L::kK, q_stages = small ? L::kQSmall : L::kQ;
  const uint32_t q_panel = small ? L::kSmallRows * 128 : kPanelBytes;
  const uint32_t q_slot = L::kPanels * q_panel;
  const uint32_t sK = base, sQ = base + static_cast<uint32_t>(k_stages * L::kTileBytes);
  const uint32_t bars = base + L::kBarOffset;
  auto bar_k_full = [&](int s) { return bars + 8u * s; };
  auto bar_k_empty = [&](int s) { return bars + 8u * (L::kMostK + s); };
  auto bar_q_full = [&](int s) { return bars + 8u * (2 * L::kMostK + s); };
  auto bar_q_empty = [&](int s) { return bars + 8u * (2 * L::kMostK + L::kMostQ + s); };
  const uint32_t rest = bars + 8u * (2 * L::kMostK + 2 * L::kMostQ);
  const uint32_t bar_s_full0 = rest, bar_s_free0 = rest + 32;  // [buffer]
  const uint32_t bar_part0 = rest + 64, bar_taken0 = rest + 80, bar_drain0 = rest + 96;  // [warpgroup]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOffset);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOffset + 4);
  WeighStart* const start = reinterpret_cast<WeighStart*>(smem + L::kStartOffset);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == 0) {
    const WeighStart st = weigh_start(p);
    if (lane == 0) *start = st;
  }
  if (threadIdx.x == 32) {
    for (int s = 0; s < L::kMostK; ++s) {
      mbar_init(bar_k_full(s), 1);
      mbar_init(bar_k_empty(s), 2);  // both issuers pass every tile and block
    }
    for (int s = 0; s < L::kMostQ; ++s) {
      mbar_init(bar_q_full(s), 1);
      mbar_init(bar_q_empty(s), 2);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar_s_full0 + 8 * i, 1);
      mbar_init(bar_s_free0 + 8 * i, 128);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_part0 + 8 * i, 128);
      mbar_init(bar_taken0 + 8 * i, 128);
      mbar_init(bar_drain0 + 8 * i, 1);
    }
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  Watchdog wd;
  wd.status = p.status;
  wd.abort_flag = abort_flag;
  wd.limit_ns = p.watchdog_ns;
  WeighCursor cur = weigh_cursor(p, *start);
  WeighUnit u;
  bool ok = true, first_unit = true;

  // Whether a unit's block q needs its rows loaded: where one block is all, it
  // stays for the tiles that follow.
  auto loads_rows = [](const WeighUnit& u) { return u.blocks > 1 || u.new_rows; };

  if (warp == kLoadWarp) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_map(&tmQ);
      tma_prefetch_map(&tmK);
    }
    const uint64_t again = l2_policy_evict_last(), once = l2_policy_evict_first();
    const uint32_t page_bytes = static_cast<uint32_t>(p.page_rows * 128 * L::kPanels);
    const uint32_t q_bytes = static_cast<uint32_t>(p.block_tokens * p.block_heads * 128 * L::kPanels);
    const int in_page = (1 << p.page_shift) - 1;
    int ks = 0, qs = 0;
    uint32_t k_ph = 0, q_ph = 0;
    uint32_t k_used = 0, q_used = 0;  // loads so far
    for (; ok && weigh_next(cur, u, first_unit, p); first_unit = false) {
      if (u.first == u.blocks) continue;
      // this lane's page of the tile
      const int pos = u.tile * kKeys + lane * p.page_rows;
      const bool mine = lane * p.page_rows < kKeys && pos < u.s.length;
      const int page = mine ? paged_entry(p, u.b, pos) : 0;
      bool free = lane != 0 || wait_bounded(bar_k_empty(ks), k_ph ^ 1u, wd, kSiteWeighKEmpty, true, kNapNs);
      ok = __all_sync(0xffffffffu, free);
      if (!ok) break;
      const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, mine));
      if (!(p.test_withhold && k_used == 0)) {  // test hook: the first tile never arrives
        if (lane == 0) mbar_arrive_expect_tx(bar_k_full(ks), boxes * page_bytes);
        __syncwarp();
        if (mine)
          for (int pn = 0; pn < L::kPanels; ++pn)
            tma_load_4d_hint(sK + static_cast<uint32_t>(ks * L::kTileBytes + pn * kPanelBytes + lane * p.page_rows * 128),
                             &tmK, bar_k_full(ks), pn * 64, pos & in_page, u.head, page_ok(p, page) ? page : p.pages, once);
      }
      ++k_used;
      if (++ks == k_stages) {
        ks = 0;
        k_ph ^= 1u;
      }
      if (!loads_rows(u)) continue;
      for (int q = u.first; q < u.blocks && ok; ++q) {
        free = lane != 0 || wait_bounded(bar_q_empty(qs), q_ph ^ 1u, wd, kSiteWeighQEmpty, true, kNapNs);
        ok = __all_sync(0xffffffffu, free);
        if (!ok) break;
        if (lane == 0) {
          const int token = q / p.head_blocks, part = q - token * p.head_blocks;
          mbar_arrive_expect_tx(bar_q_full(qs), q_bytes);
          for (int pn = 0; pn < L::kPanels; ++pn)
            tma_load_3d_hint(sQ + qs * q_slot + pn * q_panel, &tmQ, bar_q_full(qs), pn * 64,
                             u.head * p.group + part * p.block_heads, u.s.t0 + token * p.block_tokens, again);
        }
        ++q_used;
        if (++qs == q_stages) {
          qs = 0;
          q_ph ^= 1u;
        }
      }
    }
    // Drain: every copy issued must have landed before the CTA may exit.
    if (lane == 0) {
      for (int i = 0; i < k_stages && k_used > 0; ++i, --k_used) {  // backwards from the latest
        if (--ks < 0) {
          ks = k_stages - 1;
          k_ph ^= 1u;
        }
        wait_bounded(bar_k_full(ks), k_ph, wd, kSiteWeighDrain, false, kNapNs);
      }
      for (int i = 0; i < q_stages && q_used > 0; ++i, --q_used) {
        if (--qs < 0) {
          qs = q_stages - 1;
          q_ph ^= 1u;
        }
        wait_bounded(bar_q_full(qs), q_ph, wd, kSiteWeighDrain, false, kNapNs);
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
    // --------------------------------------------------------- MMA issuers
    if (lane == 0) {
      const int me = warp - kMmaWarp;
      const uint32_t idesc = make_idesc_f16(kBf16, p.columns, false);
      constexpr uint32_t kHi = desc_hi_sw128(1024);
      int ks = 0, qs = -1;  // qs: the block's slot; -1 none yet
      uint32_t k_ph = 0, q_ph = 1;
      uint32_t free_ph[2] = {1u, 1u};  // of this warpgroup's two buffers: nothing to wait for at first
      uint32_t step = 0;
      bool held = false;  // a block that stays
      for (; ok && weigh_next(cur, u, first_unit, p); first_unit = false) {
        if (u.first == u.blocks) continue;
        ok = wait_bounded(bar_k_full(ks), k_ph, wd, kSiteWeighKFull, true, kNapNs);
        if (!ok) break;
        for (int q = u.first; q < u.blocks; ++q, ++step) {
          if (loads_rows(u)) {
            if (held) {  // the block before is not needed any more
              mma_commit(bar_q_empty(qs));
              held = false;
            }
            if (++qs == q_stages || qs == 0) {
              qs = 0;
              q_ph ^= 1u;
            }
            ok = wait_bounded(bar_q_full(qs), q_ph, wd, kSiteWeighQFull, true, kNapNs);
            if (!ok) break;
          }
          if ((step & 1u) == static_cast<uint32_t>(me)) {
            const int half = (step >> 1) & 1;
            const int buf = me + 2 * half;
            ok = wait_bounded(bar_s_free0 + 8 * buf, free_ph[half], wd, kSiteWeighSFree, true, kNapNs);
            if (!ok) break;
            free_ph[half] ^= 1u;
            tc_fence_after_sync();
            const uint32_t ka = desc_lo_sw128(sK, 16) + static_cast<uint32_t>(ks * (L::kTileBytes >> 4));
            const uint32_t qa = desc_lo_sw128(sQ, 16) + ((static_cast<uint32_t>(qs) * q_slot) >> 4);
            const uint32_t dt = tmem + static_cast<uint32_t>(buf * 128);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t k_off = static_cast<uint32_t>(((kk >> 2) * kPanelBytes + (kk & 3) * 32) >> 4);
              const uint32_t q_off = ((kk >> 2) * q_panel + (kk & 3) * 32) >> 4;
              mma_ss_w(dt, ka + k_off, kHi, qa + q_off, kHi, idesc, kk > 0 ? 1u : 0u);
            }
            mma_commit(bar_s_full0 + 8 * buf);
          }
          if (u.blocks > 1) mma_commit(bar_q_empty(qs));
          else held = true;
        }
        if (!ok) break;
        mma_commit(bar_k_empty(ks));
        if (++ks == k_stages) {
          ks = 0;
          k_ph ^= 1u;
        }
      }
      // Drain: all issued tensor-core work completes before TMEM is released.
      mma_commit(bar_drain0 + 8 * me);
      wait_bounded(bar_drain0 + 8 * me, 0u, wd, kSiteWeighDrain, false, kNapNs);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------ exponentials: thread = key
    const int me = warp >> 2, key_lane = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    float* const lse = reinterpret_cast<float*>(smem + L::kLseOffset) + warp * 128;
    float* const part = reinterpret_cast<float*>(smem + L::kPartOffset);
    const float c = p.scale_log2;
    uint32_t full_ph[2] = {0u, 0u}, step = 0;
    uint32_t part_ph = 0, taken_ph = 1;  // of the other's sums; of this one's being read
    // this lane's four columns: where their LSE lie, from the block's first token and head on
    int at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = 4 * lane + i, token = col / p.block_heads;
      at[i] = token * p.heads * p.group + (col - token * p.block_heads);
    }
    for (; ok && weigh_next(cur, u, first_unit, p); first_unit = false) {
      const int key = u.tile * kKeys + key_lane;
      const int steps = u.blocks - u.first;
      // who writes the unit: the warpgroup of its last step
      const bool writes = steps > 0 ? ((step + steps - 1) & 1u) == static_cast<uint32_t>(me) : me == 0;
      long long to = -1;
      float old = 0.f;
      if (writes && key < u.s.length) {
        const int page = paged_entry(p, u.b, key);
        if (page_ok(p, page)) {
          to = ((static_cast<long long>(page) * p.heads + u.head) << p.page_shift) + (key & ((1 << p.page_shift) - 1));
          if (p.in) old = p.in[to];
        }
      }
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int q = u.first; q < u.blocks; ++q, ++step) {
        if ((step & 1u) != static_cast<uint32_t>(me)) continue;
        const int block = q / p.head_blocks, hb = q - block * p.head_blocks, token0 = block * p.block_tokens;
        const int valid = p.head_blocks > 1 ? min(p.block_heads, p.group - hb * p.block_heads)
                                            : min(p.block_tokens, u.s.n - token0) * p.group;
        // the columns that see this key: [lo, valid)
        const int lo = p.causal ? min(max(key - (u.s.length - u.s.n) - token0, 0), p.block_tokens) * p.block_heads : 0;
        const float* from = p.lse + (static_cast<long long>(u.s.t0 + token0) * p.heads + u.head) * p.group + hb * p.block_heads;
        float neg[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) neg[i] = 4 * lane + i < valid ? __ldg(from + at[i]) * -1.4426950408889634f : 0.f;
        __syncwarp();  // the step before has been read
        *reinterpret_cast<float4*>(lse + 4 * lane) = make_float4(neg[0], neg[1], neg[2], neg[3]);
        __syncwarp();
        const int half = (step >> 1) & 1, buf = me + 2 * half;
        bool got = wait_bounded(bar_s_full0 + 8 * buf, full_ph[half], wd, kSiteWeighSFull);
        got = __all_sync(0xffffffffu, got);
        if (!got) { ok = false; break; }
        full_ph[half] ^= 1u;
        tc_fence_after_sync();
        const bool masked = __any_sync(0xffffffffu, lo > 0) || (valid & 31);
        const uint32_t tS = tmem + lane_off + static_cast<uint32_t>(buf * 128);
#pragma unroll 1
        for (int c0 = 0; c0 < valid; c0 += 32) {
          uint32_t sr[32];
          tmem_ld32x32_wait(tS + c0, sr);
          const float4* l4 = reinterpret_cast<const float4*>(lse + c0);
          if (masked) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 l = l4[i];
              const float x[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int col = c0 + 4 * i + j;
                const float w = ex2_approx(fmaf(__uint_as_float(sr[4 * i + j]), c, x[j]));
                acc[j] += col >= lo && col < valid ? w : 0.f;
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 l = l4[i];
              float x0, x1, x2, x3;
              ffma2(x0, x1, __uint_as_float(sr[4 * i]), __uint_as_float(sr[4 * i + 1]), c, l.x, l.y);
              ffma2(x2, x3, __uint_as_float(sr[4 * i + 2]), __uint_as_float(sr[4 * i + 3]), c, l.z, l.w);
              fadd2_acc(acc[4 * (i & 1)], acc[4 * (i & 1) + 1], ex2_approx(x0), ex2_approx(x1));
              fadd2_acc(acc[4 * (i & 1) + 2], acc[4 * (i & 1) + 3], ex2_approx(x2), ex2_approx(x3));
            }
          }
        }
        tc_fence_before_sync();
        mbar_arrive(bar_s_free0 + 8 * buf);
      }
      if (!ok) break;
      float sum = ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
      if (steps > 1) {
        if (!writes) {
          bool got = wait_bounded(bar_taken0 + 8 * me, taken_ph, wd, kSiteWeighTaken);
          got = __all_sync(0xffffffffu, got);
          if (!got) break;
          taken_ph ^= 1u;
          part[me * 128 + key_lane] = sum;
          mbar_arrive(bar_part0 + 8 * me);
          continue;
        }
        bool got = wait_bounded(bar_part0 + 8 * (me ^ 1), part_ph, wd, kSiteWeighPart);
        got = __all_sync(0xffffffffu, got);
        if (!got) break;
        part_ph ^= 1u;
        sum += part[(me ^ 1) * 128 + key_lane];
        mbar_arrive(bar_taken0 + 8 * (me ^ 1));
      }
      if (to >= 0) p.out[to] = old + sum;
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, bool kBf16>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& k, const PagedWeighParams& p, int grid, cudaStream_t s) {
  auto kern = fa2_paged_weigh_kernel<D, kBf16>;
  constexpr int smem = WeighLayout<D>::kSmemBytes;
  static PerDeviceOnce prepared;
  const cudaError_t e = once_per_device(
      prepared, [&]() { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
  if (e != cudaSuccess) return e;
  kern<<<grid, kThreads, smem, s>>>(q, k, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_weigh(int D, bool bf, const CUtensorMap& q, const CUtensorMap& k, const PagedWeighParams& p,
                               int grid, cudaStream_t s) {
  switch (D) {
    case 32: return bf ? launch<32, true>(q, k, p, grid, s) : launch<32, false>(q, k, p, grid, s);
    case 64: return bf ? launch<64, true>(q, k, p, grid, s) : launch<64, false>(q, k, p, grid, s);
    case 96: return bf ? launch<96, true>(q, k, p, grid, s) : launch<96, false>(q, k, p, grid, s);
    default: return bf ? launch<128, true>(q, k, p, grid, s) : launch<128, false>(q, k, p, grid, s);
  }
}

}  // namespace fa2
