// The work-unit walk of attention over a paged cache on the tensor cores
// (fa2_paged_kernel.cuh): as the one of cross attention in fa2_cross.cuh, with
// units whose number of K/V tiles depends on the sequence and, under the causal
// mask, on the unit's last token.
#pragma once
#include <climits>

#include "fa2_paged.cuh"

namespace fa2 {

// A sub-tile is 128 rows (tokens of one sequence, query heads of one key head), a unit two of them.

// The sum of floor((a i + b) / m) over i < n, for n, m > 0 and a, b >= 0: whole
// parts out, then the lattice points under the line counted the other way
// round, as in Euclid's algorithm. a n + b stays below 2^31.
__device__ __forceinline__ long long floor_sum(unsigned n, unsigned m, unsigned a, unsigned b) {
  long long sum = 0;
  for (;;) {
    if (a >= m) {
      sum += static_cast<long long>(n) * (n - 1) / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      sum += static_cast<long long>(n) * (b / m);
      b %= m;
    }
    const unsigned y = a * n + b;
    if (y < m) return sum;
    n = y / m;
    b = y % m;
    const unsigned t = m;
    m = a;
    a = t;
  }
}

// The same with m = 128. Steps of a power of two below it (those of 1, 2, 4, ..
// query heads to a key head) need no division: every CTA takes this sum several
// times before its first load.
__device__ __forceinline__ long long floor_sum128(unsigned n, unsigned a, unsigned b) {
  if ((a & 127u) == 0) {
    // whole parts alone
    return static_cast<long long>(n) * (n - 1) / 2 * (a >> 7) + static_cast<long long>(n) * (b >> 7);
  }
  if (a < 128u && (a & (a - 1u)) == 0) {
    // floor((a i + b) / 128) = floor((i + b / a) / k), k = 128 / a: sums of floor(i / k) from 0
    const int shift = 7 - (31 - __clz(a));  // log2 k
    auto upto = [&](unsigned x) {
      const long long t = x >> shift;
      return (t * (t - 1) / 2 << shift) + t * (x - (static_cast<unsigned>(t) << shift));
    };
    const unsigned from = b >> (7 - shift);
    return upto(from + n) - upto(from);
  }
  return floor_sum(n, 128u, a, b);
}

struct PagedUnits {  // of one sequence
  PagedSeq s;
  int units;  // per key head; 0: none of this kernel's
};

__device__ __forceinline__ int key_tiles(int keys) { return max(1, (keys + kKeys - 1) / kKeys); }

__device__ __forceinline__ PagedUnits paged_units(const PagedTileParams& p, int b) {
  PagedUnits u;
  u.s = paged_seq(p, b);
  const int rows = u.s.n * p.group, per = 2 * p.sub_tokens;
  u.units = rows >= p.rows_from && rows <= p.rows_to ? (u.s.n + per - 1) / per : 0;
  return u;
}

// Positions that token i of the sequence sees.
__device__ __forceinline__ int paged_seen(const PagedTileParams& p, const PagedSeq& s, int i) {
  return p.causal ? min(max(s.length - s.n + i + 1, 0), s.length) : s.length;
}

// What a unit counts in the equal shares besides its tiles: the tensor cores
// idle while its last P.V drains and its rows go out. (Four prompts of 4096, us:
// 1 233, 2 226, 3 220, 4 222, 6 225; a chunk and a mixed batch within 2 of each other.)
constexpr int kPagedUnitCost = 3;

// Positions that a unit's last token sees, which no other one of it exceeds.
__device__ __forceinline__ int unit_keys(const PagedTileParams& p, const PagedSeq& s, int unit) {
  return paged_seen(p, s, min((unit + 1) * 2 * p.sub_tokens, s.n) - 1);
}

// Steps of the first m of a sequence's units of one key head.
__device__ __forceinline__ long long steps_before(const PagedTileParams& p, const PagedUnits& u, int m) {
  long long tiles = 0;
  if (!p.causal) {
    tiles = static_cast<long long>(m) * key_tiles(u.s.length);
  } else {
    const int per = 2 * p.sub_tokens, c = u.s.length - u.s.n;
    int full = min(m, u.units - 1);
    if (m == u.units) tiles += key_tiles(u.s.length);  // the last unit sees every position
    // units of tokens before the first position: one masked tile
    const int none = c < 0 ? min(full, -c / per) : 0;
    tiles += none;
    full -= none;
    if (full > 0)
      tiles += floor_sum128(static_cast<unsigned>(full), static_cast<unsigned>(per),
                            static_cast<unsigned>(c + (none + 1) * per + kKeys - 1));
  }
  return tiles + static_cast<long long>(m) * kPagedUnitCost;
}

// a / b for b > 0; in 32 bits where that is enough (most calls; a 64-bit division
// is a routine of its own, fetched by every CTA).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return (a | b) >> 32 ? a / b : static_cast<long long>(static_cast<unsigned>(a) / static_cast<unsigned>(b));
}

// Where this CTA's share begins, found once per CTA.
struct PagedStart {
  long long total;       // steps of the whole call
  long long begin, end;  // this CTA's share of them
  int shares;            // CTAs with a share
  int parts, part;       // where every unit is `parts` CTAs': which part this one's is (0: equal shares)
  bool whole;            // equal shares of units that are not cut: those that begin in the share
  int b, head, unit;
  int from;         // steps of that unit before the share
};

__device__ __forceinline__ long long paged_share_begin(const PagedStart& st, int c) {
  return c >= st.shares ? st.total : quotient(st.total * c, st.shares);
}

// Which batch entry holds step `want`, by one whole warp: `steps(b)` are the
// steps of entry b; *before: those of the entries before it, *mine: its own.
// `first`: steps(lane), which the caller has taken already.
template <typename F>
__device__ __forceinline__ int find_entry(int B, long long want, long long first, F&& steps, long long* before,
                                          long long* mine) {
  const int lane = threadIdx.x & 31;
  long long sum = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    const long long here = b0 == 0 ? first : (b0 + lane < B ? steps(b0 + lane) : 0);
    long long upto = here;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += v;
    }
    const unsigned past = __ballot_sync(0xffffffffu, sum + upto > want);
    if (past) {
      const int l = __ffs(past) - 1;
      *before = sum + __shfl_sync(0xffffffffu, upto - here, l);
      *mine = __shfl_sync(0xffffffffu, here, l);
      return b0 + l;
    }
    sum += __shfl_sync(0xffffffffu, upto, 31);
  }
  *before = *mine = 0;
  return 0;  // only should the tables have changed meanwhile
}

// A unit in so many parts or more is joined by all of its CTAs, 16 rows of a
// sub-tile at a time (8 of 16 parts or more); below, by its first part's.
constexpr int kPagedSpreadParts = 6;
constexpr float kSpreadCut = 4.f, kSpreadPart = 0.3f;
static_assert(kPagedMostParts == 32, "a number of parts per lane");

// Whether and how to cut units when there are fewer than CTAs, all of about
// `most` tiles: into how many parts each, or 0 for equal shares over all CTAs. In
// tiles: a cut costs the way through memory, every part that the unit's first
// holder adds to its own another, and shares that do not end where units do
// make a CTA work on parts of two. The warp's lanes take a number of parts each.
// Units that all of their CTAs join cost less, and each part 0.3. Fitted to sweeps
// of 16 to 512 tokens of 2 and 8 key heads over 1000 to 32,000 positions; D = 128,
// 8 key heads of 8192 positions: 16 tokens 42.4 us in equal shares, 33.6 joined by
// the first part's CTA, 20 by all; 64 tokens 50.0, 40.8, 26; 512 tokens (64 units)
// 58.8 in equal shares and 66 in two parts, for which the rule takes the former.
__device__ __forceinline__ int cut_parts(const PagedTileParams& p, long long tiles, int units, int most) {
  const int lane = threadIdx.x & 31;
  const float cut = 8.f, cut_equal = 5.f, join = p.wide ? 1.6f : 1.f;
  const int parts = lane + 1;
  float cost = 3e38f;
  if (parts * units <= static_cast<int>(gridDim.x) && parts <= most) {
    cost = static_cast<float>((most + parts - 1) / parts);
    if (parts >= kPagedSpreadParts)
      cost += kSpreadCut + kSpreadPart * static_cast<float>(parts) + (parts < 16 ? static_cast<float>((8 + parts - 1) / parts) : 0.f);
    else if (parts > 1) cost += cut + join * static_cast<float>(parts - 1);
  }
  float best = cost;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) best = fminf(best, __shfl_xor_sync(0xffffffffu, best, off));
  const float shares = static_cast<float>(gridDim.x);
  const float equal = static_cast<float>(tiles) / shares + cut_equal + join * ceilf(shares / static_cast<float>(units));
  const int n = __ffs(__ballot_sync(0xffffffffu, cost == best));  // the fewest parts
  return best < 3e38f && best <= equal ? n : 0;
}

// By one whole warp.
__device__ __forceinline__ PagedStart paged_start(const PagedTileParams& p) {
  PagedStart st = {};
  const int lane = threadIdx.x & 31;
  int units = 0, most = 0;  // of all sequences; the most tiles that a unit has
  auto steps = [&](int b) {
    const PagedUnits u = paged_units(p, b);
    if (!u.units) return 0ll;
    units += u.units;
    most = max(most, key_tiles(u.s.length));
    return p.heads * steps_before(p, u, u.units);
  };
  const long long first = lane < p.B ? steps(lane) : 0;
  const int first_units = units;
  long long sum = first;
  for (int b = lane + 32; b < p.B; b += 32) sum += steps(b);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, off);
    units += __shfl_xor_sync(0xffffffffu, units, off);
    most = max(most, __shfl_xor_sync(0xffffffffu, most, off));
  }
  st.total = sum;
  st.shares = static_cast<int>(min(static_cast<long long>(gridDim.x), sum));
  if (static_cast<int>(blockIdx.x) >= st.shares) return st;
  const long long all = static_cast<long long>(units) * p.heads, tiles = sum - all * kPagedUnitCost;
  // fewer units than CTAs, and all about as long as the longest
  const bool alike = 10 * tiles >= 9 * all * most;
  if (all < gridDim.x && alike) st.parts = cut_parts(p, tiles, static_cast<int>(all), most);
  // Units are not cut where what the CTA with the most of them has to do beyond an
  // equal share (of units of very different lengths: one of the longest) costs less
  // than the cuts: in tiles, a cut and a join, and about one more for every unit of a
  // share. Fitted to 160 to 800 units (us whole / cut at 1.3 and at 5.3 units to a
  // CTA). D = 128, all of 8 tiles: 40.2 / 39.1 and 113 / 123, of 16: 65.6 / 56.9 and
  // 196 / 186, of up to 8: 29.9 / 28.9 and 83 / 97, of up to 16: 44.8 / 41.4 and 130 /
  // 130. D = 64: 30.4 / 27.3 and 81 / 85, 49.4 / 41.3 and 139 / 131, 25.2 / 22.7 and
  // 64 / 68, 34.5 / 29.3 and 98 / 93.
  if (!st.parts) {
    const float mean = static_cast<float>(sum) / static_cast<float>(all), each = static_cast<float>(all) / static_cast<float>(gridDim.x);
    st.whole = alike ? (ceilf(each) - each) * mean <= each + (p.wide ? 6.f : 5.f)
                     : static_cast<float>(most + kPagedUnitCost) <= each + (p.wide ? 12.f : 7.f);
  }
  if (st.parts) {
    // this CTA's unit, counted over the sequences
    const int index = blockIdx.x / st.parts;
    st.part = blockIdx.x - index * st.parts;
    st.shares = static_cast<int>(all) * st.parts;
    if (static_cast<int>(blockIdx.x) >= st.shares) return st;
    long long before, mine;
    st.b = find_entry(p.B, index, static_cast<long long>(first_units) * p.heads,
                      [&](int b) { return static_cast<long long>(paged_units(p, b).units) * p.heads; }, &before, &mine);
    const PagedUnits u = paged_units(p, st.b);
    if (u.units == 0 || mine == 0) return st;  // only should the tables have changed meanwhile
    const int r = index - static_cast<int>(before);
    st.head = min(r / u.units, p.heads - 1);
    st.unit = min(r - st.head * u.units, u.units - 1);
    // No more parts than tiles, so that every part has one. Steps are counted from the
    // unit's first; those that stand for no tile are left out.
    const int its = key_tiles(unit_keys(p, u.s, st.unit));
    st.parts = min(st.parts, its);
    if (st.part >= st.parts) return st;
    st.from = kPagedUnitCost + its * st.part / st.parts;
    st.begin = st.from;
    st.end = kPagedUnitCost + its * (st.part + 1) / st.parts;
    return st;
  }
  st.begin = paged_share_begin(st, blockIdx.x);
  st.end = paged_share_begin(st, blockIdx.x + 1);
  long long before, mine;
  st.b = find_entry(p.B, st.begin, first, steps, &before, &mine);
  const PagedUnits u = paged_units(p, st.b);
  if (u.units == 0 || mine == 0) {  // only should the tables have changed meanwhile
    st.end = st.begin;
    return st;
  }
  const long long per_head = quotient(mine, p.heads);
  long long r = st.begin - before;
  st.head = static_cast<int>(min(quotient(r, per_head), p.heads - 1ll));
  r -= st.head * per_head;
  // the last unit that starts at or before step r, 32 candidates at a time
  int lo = 0, hi = u.units;
  long long at = 0;  // steps before unit lo
  while (hi - lo > 1) {
    const int by = (hi - lo + 31) / 32, m = lo + (lane + 1) * by;
    const long long s = m < hi ? steps_before(p, u, m) : LLONG_MAX;
    const int n = __popc(__ballot_sync(0xffffffffu, s <= r));
    if (n > 0) at = __shfl_sync(0xffffffffu, s, n - 1);
    lo += n * by;
    hi = min(hi, lo + by);
  }
  st.unit = lo;
  st.from = static_cast<int>(r - at);
  return st;
}

struct PagedSegment {
  int b, head;
  int token, t0, n, length;  // the unit's first token in the sequence; the sequence
  int keys;                  // positions that the unit's tokens see at most
  int kv_begin, kv_end;      // K/V tiles of this segment
  int nkv;                   // of the whole unit
  long long unit_end;        // step one past the unit's last
};

struct PagedCursor {
  PagedUnits u;
  int b, head, unit, from;
  bool whole;
  long long step, end;
};

__device__ __forceinline__ PagedCursor paged_first(const PagedTileParams& p, const PagedStart& st) {
  PagedCursor c;
  c.b = st.b;
  c.head = st.head;
  c.unit = st.unit;
  c.from = st.from;
  c.whole = st.whole;
  c.step = st.begin;
  c.end = st.end;
  c.u = paged_units(p, st.b);
  return c;
}

// Next segment of this CTA. Every role walks the same sequence. A share that
// ends among the steps of a unit that stand for no tile has no tile of it; the
// next share then holds all of them.
__device__ __forceinline__ bool paged_next(PagedCursor& c, PagedSegment& s, const PagedTileParams& p) {
  while (c.step < c.end) {
    s.b = c.b;
    s.head = c.head;
    s.token = c.unit * 2 * p.sub_tokens;
    s.t0 = c.u.s.t0;
    s.n = c.u.s.n;
    s.length = c.u.s.length;
    s.keys = unit_keys(p, c.u.s, c.unit);
    s.nkv = key_tiles(s.keys);
    const int per_unit = s.nkv + kPagedUnitCost, from = min(c.from, per_unit);
    const int to = c.whole ? per_unit : static_cast<int>(min(static_cast<long long>(per_unit), from + (c.end - c.step)));
    const bool mine = !c.whole || from == 0;  // else it began in an earlier share, whose it is
    s.unit_end = c.step - from + per_unit;
    s.kv_begin = max(from - kPagedUnitCost, 0);
    s.kv_end = max(to - kPagedUnitCost, 0);
    c.step += to - from;
    c.from = 0;
    if (++c.unit >= c.u.units) {
      c.unit = 0;
      if (++c.head >= p.heads) {
        c.head = 0;
        do {
          if (++c.b >= p.B) {
            c.step = c.end;
            break;
          }
          c.u = paged_units(p, c.b);
        } while (c.u.units == 0);
      }
    }
    if (mine && s.kv_end > s.kv_begin) return true;
  }
  return false;
}

}  // namespace fa2
