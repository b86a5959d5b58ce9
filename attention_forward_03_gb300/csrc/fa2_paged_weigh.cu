// What every cached key weighs in the softmax rows of a batch's new tokens:
//   out_j = in_j + sum over the rows i that see j of exp(scale <q_i, k_j> - LSE_i)
// for each key head, over the query heads of its group.
//
// The products are taken the other way round from attention, S^T = K Q^T: 128
// positions are the lanes of tensor memory and the query rows its columns. So a
// thread holds one key, its sum needs no other thread, and nothing goes back to
// the tensor cores. A key's sum has a fixed order.
//
// What bounds it: with single tokens the bytes of K (each tile of 128
// positions meets a handful of rows); with a chunk of tokens the products and
// the exponentials, one for each product of a row and a key.
//
// One CTA per SM. Work: units (a sequence's 256 positions, two tiles, of one
// key head) in the order (sequence, key head, unit), each with as many steps as
// there are blocks of query rows that see a key of it. Every CTA takes an equal
// share of all steps; a unit that is cut between CTAs is finished by the one
// that holds its first block, which adds the sums that the following CTAs left
// in the workspace (they did so at the start of their shares, long before).
//   warps 0-7     two warpgroups, which take the steps in turn: thread = key of
//                 either tile
//   warps 8, 9    one thread each issues the products of one tile
//   warps 10, 11  load one tile's K each (one box per page, a page number per
//                 lane, read a unit ahead); warp 10 the blocks of query rows too
// A block of query rows is up to 128 / group tokens with all heads of the
// group (of more than 128 heads: one token, 128 heads). Where all rows of a
// sequence fit into one block it stays for all units of a key head. Each
// warpgroup has a buffer of 128 columns per tile in tensor memory. The rows'
// LSE are laid out once per warp and block in shared memory, as factors of the
// exponent; a thread reads them once for its two keys (a warpgroup per tile,
// with twice the reads and what a step takes besides its exponentials not
// overlapped with another's: 1.45 us a step; so 0.85).
// Measured, 8 key heads of 128 with 4 query heads each: single tokens of 64
// sequences of up to 4096 positions 51 us (floor 41.5, the bytes of K); 512
// tokens over 8192 positions 37 us (floor 16.9). Of these a CTA has no scores for
// 7 (its share 3, the first instructions 1, the first loads and product 3), then
// 26.5 steps of 256 keys x 128 rows, two in 1.55 to 1.7 us, 22 in all; 1 goes
// where the unit changes, 2 into sums that are left to others or joined; and the
// last CTA ends 2.5 after the mean (time stamps in every warpgroup). Of a step
// the exponentials take 0.54, the rows' factors out of shared memory 0.27 (0.54, and
// 41 us in all, with one tile after the other, whose buffers are filled again
// earlier), the products 0.56.
// A unit's sums of the warpgroup that did not take its last step go through
// shared memory to the other, which writes.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <type_traits>

#include "fa2_paged_walk.cuh"

namespace fa2 {
namespace {

__device__ __forceinline__ void tmem_ld32x8_wait(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}

// 32 columns from each of two places, and the wait for them.
__device__ __forceinline__ void tmem_ld32x32_two_wait(uint32_t from0, uint32_t from1, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%64];\n"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%65];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7]), "=&r"(r[8]), "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]), "=&r"(r[12]), "=&r"(r[13]), "=&r"(r[14]), "=&r"(r[15]), "=&r"(r[16]), "=&r"(r[17]), "=&r"(r[18]), "=&r"(r[19]), "=&r"(r[20]), "=&r"(r[21]), "=&r"(r[22]), "=&r"(r[23]), "=&r"(r[24]), "=&r"(r[25]), "=&r"(r[26]), "=&r"(r[27]), "=&r"(r[28]), "=&r"(r[29]), "=&r"(r[30]), "=&r"(r[31]), "=&r"(r[32]), "=&r"(r[33]), "=&r"(r[34]), "=&r"(r[35]), "=&r"(r[36]), "=&r"(r[37]), "=&r"(r[38]), "=&r"(r[39]), "=&r"(r[40]), "=&r"(r[41]), "=&r"(r[42]), "=&r"(r[43]), "=&r"(r[44]), "=&r"(r[45]), "=&r"(r[46]), "=&r"(r[47]), "=&r"(r[48]), "=&r"(r[49]), "=&r"(r[50]), "=&r"(r[51]), "=&r"(r[52]), "=&r"(r[53]), "=&r"(r[54]), "=&r"(r[55]), "=&r"(r[56]), "=&r"(r[57]), "=&r"(r[58]), "=&r"(r[59]), "=&r"(r[60]), "=&r"(r[61]), "=&r"(r[62]), "=&r"(r[63])
      : "r"(from0), "r"(from1)
      : "memory");
}

enum : int {
  kSiteWeighKEmpty = 61,
  kSiteWeighQEmpty = 62,
  kSiteWeighKFull = 63,
  kSiteWeighQFull = 64,
  kSiteWeighSFree = 65,
  kSiteWeighSFull = 66,
  kSiteWeighPart = 67,
  kSiteWeighTaken = 68,
  kSiteWeighFlag = 69,
  kSiteWeighDrain = 70,
};

constexpr int kUnitKeys = 2 * kKeys;

// Units and blocks of query rows of one key head of a sequence.
struct WeighSeq {
  PagedSeq s;
  int units, blocks;
};

__device__ __forceinline__ WeighSeq weigh_seq(const PagedWeighParams& p, int b) {
  WeighSeq w;
  w.s = paged_seq(p, b);
  w.blocks = (w.s.n + p.block_tokens - 1) / p.block_tokens * p.head_blocks;
  // without new tokens the weights stay: nothing to do in place
  w.units = w.blocks == 0 && p.in == p.out ? 0 : (w.s.length + kUnitKeys - 1) / kUnitKeys;
  return w;
}

// The first block with a row that sees a position of the unit: that of the
// token that stands at the unit's first position.
__device__ __forceinline__ int first_block(const PagedWeighParams& p, const WeighSeq& w, int unit) {
  const int token = unit * kUnitKeys - (w.s.length - w.s.n);
  return p.causal && w.blocks && token > 0 ? token / p.block_tokens * p.head_blocks : 0;
}

// What the steps of a unit with tokens of its own count more: blocks that some
// rows see and others do not, about half a step each (without it the CTAs with
// a chunk's last units came 6 us after the others' 33).
__device__ __forceinline__ int own_cost(const PagedWeighParams& p, const WeighSeq& w) {
  return p.causal ? min(w.blocks, kUnitKeys / p.block_tokens * p.head_blocks) / 2 : 0;
}

// Steps of a unit besides those of its blocks: loads that wait, the sum's way
// out; of a key head's first one also the rows' (without it the CTA with a
// batch's shortest sequences, single tokens over up to 256 positions, came
// last: 51 us, the others 38 to 44).
__device__ __forceinline__ int unit_cost(const PagedWeighParams& p, const WeighSeq& w, int unit) {
  return (unit == 0 ? 2 : 1) + ((unit + 1) * kUnitKeys > w.s.length - w.s.n ? own_cost(p, w) : 0);
}

// Steps of the first m units of a key head.
__device__ __forceinline__ long long weigh_before(const PagedWeighParams& p, const WeighSeq& w, int m) {
  long long steps = static_cast<long long>(m) * (w.blocks + 1) + (m > 0 ? 1 : 0);
  if (p.causal && w.blocks) {
    const int c = w.s.length - w.s.n, j0 = c > 0 ? (c + kUnitKeys - 1) / kUnitKeys : 0;
    const int j1 = c > 0 ? c / kUnitKeys : 0;  // the first unit with tokens of its own
    if (m > j1) steps += static_cast<long long>(m - j1) * own_cost(p, w);
    if (m > j0)
      steps -= p.head_blocks * floor_sum(static_cast<unsigned>(m - j0), static_cast<unsigned>(p.block_tokens), kUnitKeys,
                                         static_cast<unsigned>(j0 * kUnitKeys - c));
  }
  return steps;
}

// This CTA's share [begin, end) of all steps, and where it begins.
struct WeighStart {
  long long total, begin, end;
  int shares;
  int b, head, unit;
  int from;  // steps of that unit before the share
};

__device__ __forceinline__ long long weigh_share_begin(const WeighStart& st, int c) {
  return c >= st.shares ? st.total : quotient(st.total * c, st.shares);
}

// By one whole warp.
__device__ __forceinline__ WeighStart weigh_start(const PagedWeighParams& p) {
  WeighStart st = {};
  const int lane = threadIdx.x & 31;
  auto steps = [&](int b) {
    const WeighSeq w = weigh_seq(p, b);
    return p.heads * weigh_before(p, w, w.units);
  };
  const long long first = lane < p.B ? steps(lane) : 0;
  long long sum = first;
  for (int b = lane + 32; b < p.B; b += 32) sum += steps(b);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  st.total = sum;
  st.shares = static_cast<int>(min(static_cast<long long>(gridDim.x), sum));
  if (static_cast<int>(blockIdx.x) >= st.shares) return st;
  st.begin = weigh_share_begin(st, blockIdx.x);
  st.end = weigh_share_begin(st, blockIdx.x + 1);
  long long before, mine;
  st.b = find_entry(p.B, st.begin, first, steps, &before, &mine);
  const WeighSeq w = weigh_seq(p, st.b);
  if (w.units == 0 || mine == 0) {  // only should the tables have changed meanwhile
    st.end = st.begin;
    return st;
  }
  const long long per_head = quotient(mine, p.heads);
  long long r = st.begin - before;
  st.head = static_cast<int>(min(quotient(r, per_head), p.heads - 1ll));
  r -= st.head * per_head;
  // the last unit that begins at or before step r, 32 candidates at a time
  int lo = 0, hi = w.units;
  long long at = 0;  // steps before unit lo
  while (hi - lo > 1) {
    const int by = (hi - lo + 31) / 32, m = lo + (lane + 1) * by;
    const long long s = m < hi ? weigh_before(p, w, m) : LLONG_MAX;
    const int n = __popc(__ballot_sync(0xffffffffu, s <= r));
    if (n > 0) at = __shfl_sync(0xffffffffu, s, n - 1);
    lo += n * by;
    hi = min(hi, lo + by);
  }
  st.unit = lo;
  st.from = static_cast<int>(r - at);
  return st;
}

struct WeighCursor {
  WeighSeq w;
  int b, head, unit, from;
  bool new_rows;
  long long step, end;
};

struct WeighSegment {
  int b, head, unit;
  int begin, end;      // blocks of query rows of this segment
  int first, blocks;   // of the whole unit: [first, blocks)
  bool new_rows;       // of another sequence or key head than the segment before
  PagedSeq s;
};

__device__ __forceinline__ WeighCursor weigh_cursor(const PagedWeighParams& p, const WeighStart& st) {
  WeighCursor c;
  c.b = st.b;
  c.head = st.head;
  c.unit = st.unit;
  c.from = st.from;
  c.new_rows = true;
  c.step = st.begin;
  c.end = st.end;
  c.w = weigh_seq(p, st.b);
  return c;
}

// Next segment of this CTA; every role walks the same sequence. Of a unit
// without blocks whoever has its last step has all.
__device__ __forceinline__ bool weigh_next(WeighCursor& c, WeighSegment& u, const PagedWeighParams& p) {
  while (c.step < c.end) {
    u.b = c.b;
    u.head = c.head;
    u.unit = c.unit;
    u.s = c.w.s;
    u.blocks = c.w.blocks;
    u.first = min(first_block(p, c.w, c.unit), u.blocks);
    const int cost = unit_cost(p, c.w, c.unit), per_unit = u.blocks - u.first + cost, from = min(c.from, per_unit);
    const int to = static_cast<int>(min(static_cast<long long>(per_unit), from + (c.end - c.step)));
    u.begin = u.first + max(from - cost, 0);
    u.end = u.first + max(to - cost, 0);
    c.step += to - from;
    c.from = 0;
    const bool any = u.end > u.begin || (u.first == u.blocks && to == per_unit);
    if (any) {
      u.new_rows = c.new_rows;
      c.new_rows = false;
    }
    if (++c.unit >= c.w.units) {
      c.unit = 0;
      c.new_rows = true;
      if (++c.head >= p.heads) {
        c.head = 0;
        do {
          if (++c.b >= p.B) {
            c.step = c.end;
            break;
          }
          c.w = weigh_seq(p, c.b);
        } while (c.w.units == 0);
      }
    }
    if (any) return true;
  }
  return false;
}

template <int D>
struct WeighLayout {
  static constexpr int kPanels = (D + 63) / 64;
  static constexpr int kTileBytes = kPanels * kPanelBytes;
  static constexpr int kSmallRows = 32;  // blocks of at most so many rows: more room for K
  static constexpr int kSmallBytes = kPanels * kSmallRows * 128;
  // stages of each tile's K and of Q, with blocks of up to 128 rows and with small ones
  static constexpr int kK = kPanels == 2 ? 2 : 4, kQ = kPanels == 2 ? 2 : 4;
  static constexpr int kKSmall = kPanels == 2 ? 3 : 6, kQSmall = kPanels == 2 ? 2 : 4;
  static constexpr int kMostK = kKSmall, kMostQ = kQ > kQSmall ? kQ : kQSmall;
  static constexpr int kWide = 2 * kK * kTileBytes + kQ * kTileBytes;
  static constexpr int kNarrow = 2 * kKSmall * kTileBytes + kQSmall * kSmallBytes;
  static constexpr int kLseOffset = kWide > kNarrow ? kWide : kNarrow;  // [8 warps][128] floats
  static constexpr int kPartOffset = kLseOffset + 8 * 128 * 4;          // [2 warpgroups][128] pairs of floats
  static constexpr int kBarOffset = kPartOffset + 2 * 128 * 8;
  // k_full, k_empty [tile][K], q_full, q_empty [Q], s_full, s_free [warpgroup][tile], part, taken, flag [warpgroup], drain[2]
  static constexpr int kNumBars = 4 * kMostK + 2 * kMostQ + 16;
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
  // K: [tile][stage], then Q
  const uint32_t sK = base, sQ = base + static_cast<uint32_t>(2 * k_stages * L::kTileBytes);
  const uint32_t bars = base + L::kBarOffset;
  auto bar_k_full = [&](int t, int s) { return bars + 8u * (t * L::kMostK + s); };
  auto bar_k_empty = [&](int t, int s) { return bars + 8u * ((2 + t) * L::kMostK + s); };
  auto bar_q_full = [&](int s) { return bars + 8u * (4 * L::kMostK + s); };
  auto bar_q_empty = [&](int s) { return bars + 8u * (4 * L::kMostK + L::kMostQ + s); };
  const uint32_t rest = bars + 8u * (4 * L::kMostK + 2 * L::kMostQ);
  const uint32_t bar_s_full0 = rest, bar_s_free0 = rest + 32;      // [warpgroup][tile]
  // [warpgroup]: its sums of a unit are in shared memory; those have been read; steps of
  // joining a cut unit
  const uint32_t bar_part0 = rest + 64, bar_taken0 = rest + 80, bar_flag0 = rest + 96;
  const uint32_t bar_drain0 = rest + 112;                          // [issuer]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOffset);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOffset + 4);
  WeighStart* const start = reinterpret_cast<WeighStart*>(smem + L::kStartOffset);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == 0) {
    const WeighStart st = weigh_start(p);
    if (lane == 0) *start = st;
  }
  if (threadIdx.x == 32) {
    for (int t = 0; t < 2; ++t)
      for (int s = 0; s < L::kMostK; ++s) {
        mbar_init(bar_k_full(t, s), 1);
        mbar_init(bar_k_empty(t, s), 1);
      }
    for (int s = 0; s < L::kMostQ; ++s) {
      mbar_init(bar_q_full(s), 1);
      mbar_init(bar_q_empty(s), 2);  // both issuers pass every block
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar_s_full0 + 8 * i, 1);
      mbar_init(bar_s_free0 + 8 * i, 128);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_part0 + 8 * i, 128);
      mbar_init(bar_taken0 + 8 * i, 128);
      mbar_init(bar_flag0 + 8 * i, 128);
      mbar_init(bar_drain0 + 8 * i, 1);
    }
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == kLoadWarp * 32) {
    tma_prefetch_map(&tmQ);
    tma_prefetch_map(&tmK);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  Watchdog wd;
  wd.status = p.status;
  wd.abort_flag = abort_flag;
  wd.limit_ns = p.watchdog_ns;
  // Whether the segment's rows are loaded: where one block is all, it stays for
  // the units that follow.
  auto loads_rows = [](const WeighSegment& u) { return u.blocks > 1 || u.new_rows; };
  // Whether the unit's tile t has a position.
  auto has_tile = [](const WeighSegment& u, int t) { return u.unit * kUnitKeys + t * kKeys < u.s.length; };

  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kControlRegs));
    if (warp >= kLoadWarp) {
      // --------------------------------------------- loads of tile t (and Q)
      const int t = warp - kLoadWarp;
      const uint64_t again = l2_policy_evict_last(), once = l2_policy_evict_first();
      const uint32_t page_bytes = static_cast<uint32_t>(p.page_rows * 128 * L::kPanels);
      const uint32_t q_bytes = static_cast<uint32_t>(p.block_tokens * p.block_heads * 128 * L::kPanels);
      const int in_page = (1 << p.page_shift) - 1;
      int ks = 0, qs = 0;
      uint32_t k_ph = 0, q_ph = 0;
      uint32_t k_used = 0, q_used = 0;  // loads so far
      // this lane's page of the tile
      auto position = [&](const WeighSegment& u) { return u.unit * kUnitKeys + t * kKeys + lane * p.page_rows; };
      auto mine = [&](const WeighSegment& u) { return lane * p.page_rows < kKeys && position(u) < u.s.length; };
      WeighCursor cur = weigh_cursor(p, *start);
      WeighSegment u, ahead;
      bool ok = true, more = weigh_next(cur, ahead, p);
      int next = more && mine(ahead) ? paged_entry(p, ahead.b, position(ahead)) : 0;
      while (more && ok) {
        u = ahead;
        const int page = next;
        more = weigh_next(cur, ahead, p);
        if (more && mine(ahead)) next = paged_entry(p, ahead.b, position(ahead));
        if (u.begin == u.end) continue;
        if (has_tile(u, t)) {
          const bool free = lane != 0 || wait_bounded(bar_k_empty(t, ks), k_ph ^ 1u, wd, kSiteWeighKEmpty, true, kNapNs);
          ok = __all_sync(0xffffffffu, free);
          if (!ok) break;
          const bool load = mine(u);
          const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, load));
          const uint32_t full = bar_k_full(t, ks);
          if (!(p.test_withhold && t == 0 && k_used == 0)) {  // test hook: the first tile never arrives
            if (lane == 0) mbar_arrive_expect_tx(full, boxes * page_bytes);
            __syncwarp();
            if (load) {
              const uint32_t dst = sK + static_cast<uint32_t>((t * k_stages + ks) * L::kTileBytes + lane * p.page_rows * 128);
              for (int pn = 0; pn < L::kPanels; ++pn)
                tma_load_4d_hint(dst + static_cast<uint32_t>(pn * kPanelBytes), &tmK, full, pn * 64,
                                 position(u) & in_page, u.head, page_ok(p, page) ? page : p.pages, once);
            }
          }
          ++k_used;
          if (++ks == k_stages) {
            ks = 0;
            k_ph ^= 1u;
          }
        }
        if (t == 1 || !loads_rows(u)) continue;
        for (int q = u.begin; q < u.end; ++q) {
          const bool free = lane != 0 || wait_bounded(bar_q_empty(qs), q_ph ^ 1u, wd, kSiteWeighQEmpty, true, kNapNs);
          ok = __all_sync(0xffffffffu, free);
          if (!ok) break;
          if (lane == 0) {
            int token = q, part = 0;
            if (p.head_blocks > 1) {
              token = q / p.head_blocks;
              part = q - token * p.head_blocks;
            }
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
          wait_bounded(bar_k_full(t, ks), k_ph, wd, kSiteWeighDrain, false, kNapNs);
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
    } else {
      // ------------------------------------------------- MMA issuer of a tile
      if (lane == 0) {
        const int t = warp - kMmaWarp;
        const uint32_t idesc = make_idesc_f16(kBf16, p.columns, false);
        constexpr uint32_t kHi = desc_hi_sw128(1024);
        int ks = 0, qs = -1;  // qs: the block's slot; -1 none yet
        uint32_t k_ph = 0, q_ph = 1;
        uint32_t step = 0, free_bits = 3u;  // [warpgroup]: parity of its next s_free phase; nothing to wait for at first
        bool held = false;  // a block that stays
        WeighCursor cur = weigh_cursor(p, *start);
        WeighSegment u;
        bool ok = true;
        while (ok && weigh_next(cur, u, p)) {
          if (u.begin == u.end) continue;
          const bool live = has_tile(u, t), loads = loads_rows(u);
          if (live) ok = wait_bounded(bar_k_full(t, ks), k_ph, wd, kSiteWeighKFull, true, kNapNs);
          if (!ok) break;
          const uint32_t ka = desc_lo_sw128(sK, 16) + static_cast<uint32_t>((t * k_stages + ks) * (L::kTileBytes >> 4));
          for (int q = u.begin; q < u.end; ++q) {
            if (loads) {
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
            const uint32_t wg = step++ & 1u;  // whose step
            if (live) {
              // The warpgroup's step before with this tile has been read. (Tiles have barriers
              // of their own: a barrier's phase is known by its parity alone, so whoever waits
              // must wait for every phase, and not all units have the second tile.)
              const uint32_t buf = 2 * wg + t;
              ok = wait_bounded(bar_s_free0 + 8 * buf, (free_bits >> wg) & 1u, wd, kSiteWeighSFree, true, kNapNs);
              if (!ok) break;
              free_bits ^= 1u << wg;
              tc_fence_after_sync();
              const uint32_t qa = desc_lo_sw128(sQ, 16) + ((static_cast<uint32_t>(qs) * q_slot) >> 4);
              const uint32_t dt = tmem + buf * 128;
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
          if (!live) continue;
          mma_commit(bar_k_empty(t, ks));
          if (++ks == k_stages) {
            ks = 0;
            k_ph ^= 1u;
          }
        }
        // Drain: all issued tensor-core work completes before TMEM is released.
        mma_commit(bar_drain0 + 8 * t);
        wait_bounded(bar_drain0 + 8 * t, 0u, wd, kSiteWeighDrain, false, kNapNs);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---------------------- exponentials: thread = a key of either tile
    const uint32_t wg = warp >> 2;
    const int key_lane = (warp & 3) * 32 + lane;
    const uint32_t tS = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + wg * 256;
    const uint32_t bar_full = bar_s_full0 + 16 * wg, bar_free = bar_s_free0 + 16 * wg, bar_flag = bar_flag0 + 8 * wg;
    float* const lse = reinterpret_cast<float*>(smem + L::kLseOffset) + warp * 128;
    const float4* const l4 = reinterpret_cast<const float4*>(lse);
    float2* const part = reinterpret_cast<float2*>(smem + L::kPartOffset) + key_lane;  // [warpgroup][128]
    const float c = p.scale_log2;
    uint32_t step = 0, full_ph[2] = {0u, 0u}, part_ph = 0, taken_ph = 1, flag_ph = 0;
    // this lane's four columns: where their LSE lie, from the block's first token and head on
    int at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = 4 * lane + i, token = col / p.block_heads;
      at[i] = token * p.heads * p.group + (col - token * p.block_heads);
    }
    // a block's first token, its rows (columns of the product), and their LSE (used a step
    // later: nothing is done with them here that would wait for them)
    auto read_block = [&](const WeighSegment& u, int q, int& token0, int& valid, float (&row_lse)[4]) {
      int hb = 0;
      if (p.head_blocks > 1) {  // blocks of one token
        token0 = q / p.head_blocks;
        hb = q - token0 * p.head_blocks;
        valid = min(p.block_heads, p.group - hb * p.block_heads);
      } else {
        token0 = q * p.block_tokens;
        valid = min(p.block_tokens, u.s.n - token0) * p.group;
      }
      const float* from = p.lse + (static_cast<long long>(u.s.t0 + token0) * p.heads + u.head) * p.group + hb * p.block_heads;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * lane + i < valid) row_lse[i] = __ldg(from + at[i]);
    };
    // this thread's page of a segment's tile
    auto entry = [&](const WeighSegment& u, int t) {
      const int key = u.unit * kUnitKeys + t * kKeys + key_lane;
      return key < u.s.length ? paged_entry(p, u.b, key) : -1;
    };
    // Of the warpgroup's threads. All of its warps wait: a share can meet twice (a cut
    // unit's tail, then the next unit's head), and the arrivals of a warp that went on
    // would stand for those of one that has yet to store its sums.
    auto meet = [&]() {
      mbar_arrive(bar_flag);
      const bool met = wait_bounded(bar_flag, flag_ph, wd, kSiteWeighPart);
      flag_ph ^= 1u;
      return __all_sync(0xffffffffu, met) != 0;
    };
    WeighCursor cur = weigh_cursor(p, *start);
    WeighSegment u;
    bool ok = true;
    int laid_b = -1, laid_head = -1;  // whose only block's factors are laid out
    while (ok && weigh_next(cur, u, p)) {
      const long long unit_end = cur.step;  // one past the unit's last step here, or where the share ends
      const int steps = u.end - u.begin;
      // who finishes the segment: the warpgroup of its last step
      const bool finishes = steps > 0 ? ((step + steps - 1) & 1u) == wg : wg == 0;
      int q = u.begin + static_cast<int>((step ^ wg) & 1u);
      step += steps;
      if (q >= u.end && !finishes) continue;
      const int key = u.unit * kUnitKeys + key_lane;
      const bool two = has_tile(u, 1);
      const bool owner = u.begin == u.first;  // of the unit's first block
      int page0 = -1, page1 = -1;             // asked for now, used at the end
      if (finishes && owner) {
        page0 = entry(u, 0);
        page1 = entry(u, 1);
      }
      float acc0[4] = {0.f, 0.f, 0.f, 0.f}, acc1[4] = {0.f, 0.f, 0.f, 0.f};
      float row_lse[4] = {0.f, 0.f, 0.f, 0.f};
      const bool laid = u.blocks == 1 && laid_b == u.b && laid_head == u.head;
      int token0 = 0, valid = u.s.n * p.group;  // (of the only block, when it is laid out)
      if (q < u.end && !laid) read_block(u, q, token0, valid, row_lse);
      for (; q < u.end; q += 2) {
        // the columns that see this thread's keys: [lo0, now) and [lo1, now)
        const int now = valid, behind = key - (u.s.length - u.s.n) - token0;
        const int lo0 = p.causal ? min(max(behind, 0), p.block_tokens) * p.block_heads : 0;
        const int lo1 = p.causal ? min(max(behind + kKeys, 0), p.block_tokens) * p.block_heads : 0;
        if (!laid) {
          constexpr float kLog2e = 1.4426950408889634f;
          __syncwarp();  // the block before has been read
          *reinterpret_cast<float4*>(lse + 4 * lane) =
              make_float4(-kLog2e * row_lse[0], -kLog2e * row_lse[1], -kLog2e * row_lse[2], -kLog2e * row_lse[3]);
          __syncwarp();
          if (q + 2 < u.end) read_block(u, q + 2, token0, valid, row_lse);
        }
        auto filled = [&](int t) {  // the step's S^T of tile t is there
          bool got = wait_bounded(bar_full + 8 * t, full_ph[t], wd, kSiteWeighSFull);
          got = __all_sync(0xffffffffu, got);
          full_ph[t] ^= 1u;
          tc_fence_after_sync();
          return got;
        };
        if (!filled(0)) { ok = false; break; }
        if (now > 16) {
          if (two && !filled(1)) { ok = false; break; }
          // 32 columns of both tiles at a time. `masked`: a warp asks which of a tile's
          // columns its keys are seen from, and only where some are and some are not it
          // asks each. (Where the second tile has no position its columns are anything:
          // not written.)
          auto chunk = [&](int c0, auto masked) {
            uint32_t sr[64];
            tmem_ld32x32_two_wait(tS + c0, tS + 128 + c0, sr);
            if (c0 + 32 >= now) {
              tc_fence_before_sync();
              mbar_arrive(bar_free);  // S^T is in registers: the buffers may be filled again
              if (two) mbar_arrive(bar_free + 8);
            }
            auto add = [&](int t, int lo, float(&acc)[4], auto each) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 l = l4[c0 / 4 + i];
                const uint32_t* const x = sr + 32 * t + 4 * i;
                float w[4];
                ffma2(w[0], w[1], __uint_as_float(x[0]), __uint_as_float(x[1]), c, l.x, l.y);
                ffma2(w[2], w[3], __uint_as_float(x[2]), __uint_as_float(x[3]), c, l.z, l.w);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  w[j] = ex2_approx(w[j]);
                  if constexpr (each.value) {
                    const int col = c0 + 4 * i + j;
                    if (col < lo || col >= now) w[j] = 0.f;
                  }
                }
                fadd2_acc(acc[0], acc[1], w[0], w[1]);
                fadd2_acc(acc[2], acc[3], w[2], w[3]);
              }
            };
            if constexpr (!masked.value) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {  // both tiles with one read of the factors
                const float4 l = l4[c0 / 4 + i];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                  float(&acc)[4] = t == 0 ? acc0 : acc1;
                  const uint32_t* const x = sr + 32 * t + 4 * i;
                  float x0, x1, x2, x3;
                  ffma2(x0, x1, __uint_as_float(x[0]), __uint_as_float(x[1]), c, l.x, l.y);
                  ffma2(x2, x3, __uint_as_float(x[2]), __uint_as_float(x[3]), c, l.z, l.w);
                  fadd2_acc(acc[0], acc[1], ex2_approx(x0), ex2_approx(x1));
                  fadd2_acc(acc[2], acc[3], ex2_approx(x2), ex2_approx(x3));
                }
              }
            } else {
              const bool whole = c0 + 32 <= now;
              if (whole && __all_sync(0xffffffffu, lo0 <= c0)) add(0, lo0, acc0, std::false_type{});
              else if (__any_sync(0xffffffffu, lo0 < c0 + 32)) add(0, lo0, acc0, std::true_type{});
              if (whole && __all_sync(0xffffffffu, lo1 <= c0)) add(1, lo1, acc1, std::false_type{});
              else if (__any_sync(0xffffffffu, lo1 < c0 + 32)) add(1, lo1, acc1, std::true_type{});
            }
          };
          if (now == 128 && !__any_sync(0xffffffffu, lo1 > 0)) {
#pragma unroll
            for (int c0 = 0; c0 < 128; c0 += 32) chunk(c0, std::false_type{});
          } else {
#pragma unroll 1
            for (int c0 = 0; c0 < now; c0 += 32) chunk(c0, std::true_type{});
          }
        } else {
          // eight columns at a time: single tokens' blocks have few. One tile after the
          // other, the second one's product under way meanwhile.
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t == 1) {
              if (!two) break;
              if (!filled(1)) { ok = false; break; }
            }
            const int lo = t == 0 ? lo0 : lo1;
            float(&acc)[4] = t == 0 ? acc0 : acc1;
#pragma unroll 1
            for (int c0 = 0; c0 < now; c0 += 8) {
              uint32_t sr[8];
              tmem_ld32x8_wait(tS + 128 * t + c0, sr);
              if (c0 + 8 >= now) {
                tc_fence_before_sync();
                mbar_arrive(bar_free + 8 * t);
              }
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float4 l = l4[c0 / 4 + i];
                const float x[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const int col = c0 + 4 * i + j;
                  const float w = ex2_approx(fmaf(__uint_as_float(sr[4 * i + j]), c, x[j]));
                  acc[j] += col >= lo && col < now ? w : 0.f;
                }
              }
            }
          }
          if (!ok) break;
        }
      }
      if (!ok) break;
      laid_b = u.b;  // (asked only where one block is all)
      laid_head = u.head;
      float sum0 = (acc0[0] + acc0[1]) + (acc0[2] + acc0[3]), sum1 = (acc1[0] + acc1[1]) + (acc1[2] + acc1[3]);
      if (steps > 1) {  // the other warpgroup had steps too
        if (!finishes) {
          bool got = wait_bounded(bar_taken0 + 8 * wg, taken_ph, wd, kSiteWeighTaken);
          got = __all_sync(0xffffffffu, got);
          if (!got) break;
          taken_ph ^= 1u;
          part[wg * 128] = make_float2(sum0, sum1);
          mbar_arrive(bar_part0 + 8 * wg);
          continue;
        }
        const uint32_t other = wg ^ 1u;
        bool got = wait_bounded(bar_part0 + 8 * other, part_ph, wd, kSiteWeighPart);
        got = __all_sync(0xffffffffu, got);
        if (!got) break;
        part_ph ^= 1u;
        const float2 theirs = part[other * 128];
        sum0 += theirs.x;
        sum1 += theirs.y;
        mbar_arrive(bar_taken0 + 8 * other);
      }
      if (!owner) {
        // not the unit's first blocks: the sums to their holder
        float* const ws = p.ws_sums + static_cast<size_t>(blockIdx.x) * kUnitKeys + key_lane;
        __stcg(ws, sum0);
        __stcg(ws + kKeys, sum1);
        __threadfence();
        if (!meet()) break;
        if (key_lane == 0) store_release(p.ws_flags + blockIdx.x, p.epoch);
        continue;
      }
      if (u.end < u.blocks) {  // others hold the rest: this is the share's last segment
        const long long rest_end = unit_end + (u.blocks - u.end);
        int last = blockIdx.x;
        while (last + 1 < start->shares && weigh_share_begin(*start, last + 1) < rest_end) ++last;
        bool fine = true;
        for (int cb = blockIdx.x + 1 + lane; cb <= last && fine; cb += 32)
          fine = wait_flag(p.ws_flags + cb, p.epoch, wd, kSiteWeighFlag);
        fine = __all_sync(0xffffffffu, fine);
        if (!fine) break;
        __syncwarp();  // what one lane acquired is visible to all
        for (int cb = blockIdx.x + 1; cb <= last; ++cb) {
          const float* ws = p.ws_sums + static_cast<size_t>(cb) * kUnitKeys + key_lane;
          sum0 += __ldcg(ws);
          sum1 += __ldcg(ws + kKeys);
        }
        // every thread has seen the flags: taken back, so that a replay of a captured
        // launch, which carries the same tag, does not find them
        if (!meet()) break;
        for (int cb = blockIdx.x + 1 + key_lane; cb <= last; cb += 128) p.ws_flags[cb] = 0ull;
      }
      auto place = [&](int page, int k) {
        return ((static_cast<long long>(page) * p.heads + u.head) << p.page_shift) + (k & ((1 << p.page_shift) - 1));
      };
      const bool there0 = page_ok(p, page0), there1 = page_ok(p, page1);
      const long long to0 = place(page0, key), to1 = place(page1, key + kKeys);
      const float old0 = there0 && p.in ? p.in[to0] : 0.f, old1 = there1 && p.in ? p.in[to1] : 0.f;
      if (there0) p.out[to0] = old0 + sum0;
      if (there1) p.out[to1] = old1 + sum1;
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// A unit's holder waits for other CTAs: all are resident, or the launch fails.
template <int D, bool kBf16>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& k, const PagedWeighParams& p, int grid, cudaStream_t s) {
  auto kern = fa2_paged_weigh_kernel<D, kBf16>;
  constexpr int smem = WeighLayout<D>::kSmemBytes;
  static PerDeviceOnce prepared;
  const cudaError_t e = once_per_device(prepared, [&]() -> cudaError_t {
    cudaFuncAttributes fa;
    cudaError_t r = cudaFuncGetAttributes(&fa, kern);
    if (r != cudaSuccess) return r;
    // The in-kernel register split assumes exactly kLaunchRegs per thread at launch.
    if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, q, k, p);
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
