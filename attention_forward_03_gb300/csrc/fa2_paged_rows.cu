// Attention of a batch's new tokens over a paged cache, 16 query rows of a key
// head at a time: a decoding step's single tokens with their grouped heads.
//
// What bounds it: the bytes of K and V, each read once for a handful of rows
// (at 16 rows and D = 128, 32 operations per byte). So, as in fa2_cross_rows.cu,
// the work is cut evenly over all SMs along the keys, and K and V stream
// through shared memory by TMA.
//
// Split: a unit is 16 query rows (token, head of the group) of one key head of
// one sequence; tiles of 128 positions, in the order (sequence, key head, row
// block, tile), are dealt to the CTAs (one per SM) in equal shares whatever the
// sequences' lengths are. A unit that is cut between CTAs is finished by the
// one that holds its first tile, with the (m, l) merge of the online softmax
// over the fp32 partial results that the following CTAs left in the workspace.
//
// A tile: each of the CTA's 8 warps takes 16 of its positions, which lie in one
// page (page sizes are multiples of 16), for all rows and works on its own. It
// has a ring of 16-position pieces of K and V that its first lane fills by TMA,
// a barrier of its own for each, and no other warp to wait for until the unit's
// end. The page numbers of its pieces of 32 tiles are read at once, one per lane
// (one per piece, a piece ahead, and the loads waited for it: 95 us below, 89 so).
// S comes from mma.m16n8k16 (rows x keys, Q in registers for the
// whole unit), the weights stay in registers in the layout that the second
// product's A operand has, O (rows x D) accumulates in fp32 registers. The
// exponent base of a row lags its maximum by up to 2^8, as in the other
// kernels, so O is rescaled rarely. At the unit's end the warps' O, m and l are
// merged through shared memory.
//
// Measured: single tokens of 64 sequences of up to 4096 positions, 8 key heads of
// 128 with 4 query heads each, 88 to 91 us, 6.1 TB/s (90 % of the measured copy;
// floor 80.5), for pages of 16 as for those of 256: equal shares end up to a fifth
// apart, some SMs' loads are served slower. 4 sequences of up to 1000 positions,
// 12 heads of 64: 10 us, latency (start, two or three tiles, join). Whole units
// instead of cut ones, where each SM would have one: 12.5 against 10.6 us and 12.1
// against 9.0.
//
// Positions that a row does not see have their scores set to -inf; V behind the
// sequence's positions is set to zero in registers, so what lies there is never
// used. The scores of positions whose page number is not one are NaN.
#include <cuda_runtime.h>

#include <climits>

#include "fa2_paged_walk.cuh"
#include "mma_sync.cuh"

namespace fa2 {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kPiece = 16;  // keys per warp and tile
static_assert(kRowWarps * kPiece == kPagedRowsKeys, "a tile's keys");
enum : int { kSitePagedFlag = 51, kSitePagedPiece = 52 };

template <int D>
struct RowsLayout {
  static constexpr int kPanels = (D + 63) / 64;
  static constexpr int kPanelBytes16 = kPiece * 128;          // 16 keys x 64 elements, 128-byte swizzled
  static constexpr int kHalfBytes = kPanels * kPanelBytes16;  // K or V of a piece
  static constexpr int kPieceBytes = 2 * kHalfBytes;
  static constexpr int kStages = kPanels == 2 ? 3 : 6;        // per warp: 24 KB
  // O of four warps, 8 rows at a time; rows 8 floats longer than D, so that
  // the 8 rows a warp writes at once meet in no bank
  static constexpr int kRowFloats = D + 8;
  static constexpr int kBufFloats = 8 * kRowFloats;
  static constexpr int kMerge = kRowWarps * kStages * kPieceBytes;
  static constexpr int kStats = kMerge + 4 * kBufFloats * 4;            // [warps][3][16]
  static constexpr int kBars = kStats + kRowWarps * 3 * kPagedRows * 4;   // [warps][stages]
  static constexpr int kAbort = kBars + kRowWarps * kStages * 8;
  static constexpr int kNoPage = kAbort + 16;                           // [warps][stages] int: the piece has no page
  static constexpr int kSmemBytes = kNoPage + kRowWarps * kStages * 4 + 1024;  // + slack for 1 KB alignment
  static_assert(kSmemBytes <= 232448, "shared memory budget");
  // what joining the partial results of up to kPagedRowsMaxCtas CTAs takes fits the ring
  static_assert((kPagedRows * D + 3 * kPagedRows + (kPagedRowsMaxCtas + 3) * kPagedRows) * 4 + 2 * kPagedRows * D * 4 + 16 * kRowThreads <= kMerge,
                "joining in the ring");
  static_assert(kBars % 8 == 0, "alignment");
};

__device__ __forceinline__ int row_tiles(int n_keys) { return max(1, (n_keys + kPagedRowsKeys - 1) / kPagedRowsKeys); }

// What a unit counts in the equal shares besides its tiles: the warps' merge.
constexpr int kRowsUnitCost = 2;

// A position in the sequence of tiles, and its step: a unit has kRowsUnitCost
// steps that stand for no tile before those of its tiles.
struct TileCursor {
  int b, head, block, tile;
  int tiles, blocks;  // of every unit of the sequence, of every key head
  int keys;           // positions that the unit's last row sees (no row sees more)
  PagedSeq s;
  long long step;
  __device__ __forceinline__ void enter(const PagedAttnParams& p) {
    s = paged_seq(p, b);
    tiles = row_tiles(s.length);
    blocks = row_blocks(p, s);
  }
  static __device__ __forceinline__ int row_blocks(const PagedAttnParams& p, const PagedSeq& s) {
    const int rows = s.n * p.group;
    return rows >= p.rows_from && rows <= p.rows_to ? (rows + kPagedRows - 1) / kPagedRows : 0;
  }
  // Positions that the sequence's token i sees.
  __device__ __forceinline__ int seen(const PagedAttnParams& p, int i) const {
    return p.causal ? min(max(s.length - s.n + i + 1, 0), s.length) : s.length;
  }
  __device__ __forceinline__ int rows(const PagedAttnParams& p) const {
    return min(kPagedRows, s.n * p.group - block * kPagedRows);
  }
  __device__ __forceinline__ void enter_block(const PagedAttnParams& p) {
    keys = seen(p, (block * kPagedRows + rows(p) - 1) / p.group);
  }
  // Row of O (token, query head) of the block's row r.
  __device__ __forceinline__ size_t out_row(const PagedAttnParams& p, int r) const {
    const int at = block * kPagedRows + r, token = at / p.group;
    return (static_cast<size_t>(s.t0 + token) * p.heads + head) * p.group + (at - token * p.group);
  }
  __device__ __forceinline__ void next(const PagedAttnParams& p) {
    ++step;
    if (++tile < tiles) return;
    tile = 0;
    step += kRowsUnitCost;
    if (++block == blocks) {
      block = 0;
      if (++head == p.heads) {
        head = 0;
        do {
          if (++b >= p.B) {
            step = LLONG_MAX;  // past the last tile
            return;
          }
          enter(p);
        } while (blocks == 0);
      }
    }
    enter_block(p);
  }
};

// Elements [4 d, 4 d + 4) of a finished row, and with d = 0 its LSE (a NaN sum
// is no row without keys: it stays).
template <int D, bool kBf16>
__device__ __forceinline__ void write_row(const PagedAttnParams& p, size_t row, int d, const float4& v, float m,
                                          float sum, float sum_o) {
  const float inv = sum > 0.f ? __frcp_rn(sum_o) : 0.f;
  reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + row * D)[d] =
      make_uint2(pack2(v.x * inv, v.y * inv, kBf16), pack2(v.z * inv, v.w * inv, kBf16));
  if (d == 0) p.lse[row] = sum != 0.f ? (m + __log2f(sum)) * 0.69314718055994530942f : CUDART_INF_F;
}

// By the whole CTA that holds the first tiles of a cut unit: its own result
// (`own`: O [16][D], then base, l and l_o, [3][16]) joined with those of the
// `others` CTAs after it, and the unit's O and LSE written. Everything is
// read in parallel: first all statistics (16 threads per row, one CTA's each),
// from which come the rows' common base, the weights and the sums, then O in
// runs of CTAs dealt to groups of threads, whose sums meet in shared memory in
// a fixed order. (One thread per element over all CTAs in turn: 4 us more at
// 8 heads of 16,384 keys.) False when a flag did not come in time.
template <int D, bool kBf16>
__device__ __forceinline__ bool join_partials(const PagedAttnParams& p, float* own, int others, const TileCursor& unit,
                                              int R, const Watchdog& wd) {
  float* const own_stats = own + kPagedRows * D;
  float* const weight = own_stats + 3 * kPagedRows;                 // [others + 1][16]
  float* const total = weight + (others + 1) * kPagedRows;          // base, l, l_o: [3][16]
  float4* const runs = reinterpret_cast<float4*>(total + 3 * kPagedRows);  // [groups][items]
  const int first = blockIdx.x + 1;
  bool ok = true;
  for (int h = threadIdx.x; h < others && ok; h += kRowThreads) {
    ok = wait_flag(p.ws_flags + first + h, p.epoch, wd, kSitePagedFlag);
    // seen: taken back, so that a replay of a captured launch, which carries
    // the same tag, does not find it set
    if (ok) p.ws_flags[first + h] = 0ull;
  }
  if (__syncthreads_or(!ok)) return false;
  {
    const int row = threadIdx.x / 16, j = threadIdx.x % 16;
    float m = -CUDART_INF_F, l = 0.f, lo = 0.f;
    if (row < R) {
      for (int h = j; h <= others; h += 16) {
        const float* at = h == 0 ? own_stats + row : p.ws_stats + static_cast<size_t>(first + h - 1) * 3 * kPagedRows + row;
        const float mh = h == 0 ? at[0] : __ldcg(at);
        weight[h * kPagedRows + row] = mh;
        m = fmaxf(m, mh);
      }
    }
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (row < R) {
      for (int h = j; h <= others; h += 16) {
        const float* at = h == 0 ? own_stats + row : p.ws_stats + static_cast<size_t>(first + h - 1) * 3 * kPagedRows + row;
        const float mh = weight[h * kPagedRows + row];
        const float e = mh == -CUDART_INF_F ? 0.f : ex2_approx(mh - m);
        weight[h * kPagedRows + row] = e;
        l = fmaf(e, h == 0 ? at[kPagedRows] : __ldcg(at + kPagedRows), l);
        lo = fmaf(e, h == 0 ? at[2 * kPagedRows] : __ldcg(at + 2 * kPagedRows), lo);
      }
    }
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) {
      l += __shfl_xor_sync(0xffffffffu, l, off);
      lo += __shfl_xor_sync(0xffffffffu, lo, off);
    }
    if (row < R && j == 0) {
      total[row] = m;
      total[kPagedRows + row] = l;
      total[2 * kPagedRows + row] = lo;
    }
  }
  __syncthreads();
  const int items = R * (D / 4);
  const int groups = max(1, kRowThreads / items);  // of CTAs, h = group, group + groups, ...
  for (int e = threadIdx.x; e < items * groups; e += kRowThreads) {
    const int group = e / items, i = e - group * items;
    const int row = i / (D / 4), d = i - row * (D / 4);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int h = group; h <= others; h += groups) {
      const float4 u = h == 0 ? *reinterpret_cast<const float4*>(own + row * D + d * 4)
                              : __ldcg(reinterpret_cast<const float4*>(
                                           p.ws_o + (static_cast<size_t>(first + h - 1) * kPagedRows + row) * D) + d);
      const float a = weight[h * kPagedRows + row];
      v.x = fmaf(a, u.x, v.x);
      v.y = fmaf(a, u.y, v.y);
      v.z = fmaf(a, u.z, v.z);
      v.w = fmaf(a, u.w, v.w);
    }
    runs[e] = v;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < items; i += kRowThreads) {
    const int row = i / (D / 4), d = i - row * (D / 4);
    float4 v = runs[i];
    for (int q = 1; q < groups; ++q) {
      const float4 u = runs[q * items + i];
      v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
    }
    write_row<D, kBf16>(p, unit.out_row(p, row), d, v, total[row], total[kPagedRows + row], total[2 * kPagedRows + row]);
  }
  return true;
}

template <int D, bool kBf16>
__global__ void __launch_bounds__(kRowThreads, 1)
    fa2_paged_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const PagedAttnParams p) {
  using L = RowsLayout<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t smem_base = (raw + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (smem_base - raw);
  float* const merge = reinterpret_cast<float*>(smem + L::kMerge);
  float* const stats = reinterpret_cast<float*>(smem + L::kStats);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem + L::kAbort);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = smem_base + static_cast<uint32_t>(warp * L::kStages * L::kPieceBytes);
  const uint32_t bars = smem_base + static_cast<uint32_t>(L::kBars + warp * L::kStages * 8);
  volatile int* const no_page = reinterpret_cast<volatile int*>(smem + L::kNoPage) + warp * L::kStages;

  // every warp finds the share and sets up its own ring
  auto steps = [&](int b) {
    const PagedSeq q = paged_seq(p, b);
    return static_cast<long long>(p.heads) * TileCursor::row_blocks(p, q) * (row_tiles(q.length) + kRowsUnitCost);
  };
  const long long first = lane < p.B ? steps(lane) : 0;
  long long total = first;
  for (int b = lane + 32; b < p.B; b += 32) total += steps(b);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
  const int shares = static_cast<int>(min(static_cast<long long>(gridDim.x), total));
  if (static_cast<int>(blockIdx.x) >= shares) return;
  auto share_begin = [&](int c) { return c >= shares ? total : quotient(total * c, shares); };
  const long long s0 = share_begin(blockIdx.x), s1 = share_begin(blockIdx.x + 1);
  long long before, mine;
  if (lane == 0) {
    for (int i = 0; i < L::kStages; ++i) mbar_init(bars + 8 * i, 1);
    mbar_init_fence();
    if (warp == 0) *abort_flag = 0;
  }
  TileCursor cur;  // the tile being computed
  cur.b = find_entry(p.B, s0, first, steps, &before, &mine);
  cur.enter(p);
  if (cur.blocks == 0) return;  // only should the tables have changed meanwhile
  {
    const long long r = s0 - before;
    const int unit = static_cast<int>(quotient(r, cur.tiles + kRowsUnitCost));
    const int at = static_cast<int>(r - static_cast<long long>(unit) * (cur.tiles + kRowsUnitCost));
    cur.head = unit / cur.blocks;
    cur.block = unit - cur.head * cur.blocks;
    cur.tile = max(at - kRowsUnitCost, 0);
    cur.step = s0 - at + kRowsUnitCost + cur.tile;
    cur.enter_block(p);
  }
  if (cur.step >= s1) return;  // a share without a tile
  const long long first_step = cur.step;
  // whether this warp's piece of a tile has a key
  auto has_keys = [&](const TileCursor& t) { return t.tile * kPagedRowsKeys + warp * kPiece < t.keys; };
  TileCursor ahead = cur;  // the tile whose piece is requested next
  // the pages of this warp's pieces of 32 tiles of a sequence, one per lane
  int pages = 0, pages_b = -1, pages_tile = 0;
  int into = 0;       // its ring slot
  int under_way = 0;  // pieces requested and not yet used
  auto find_page = [&]() {
    while (ahead.step < s1 && !has_keys(ahead)) ahead.next(p);
    if (ahead.step >= s1 || (ahead.b == pages_b && (ahead.tile & ~31) == pages_tile)) return;
    pages_b = ahead.b;
    pages_tile = ahead.tile & ~31;
    const int at = (pages_tile + lane) * kPagedRowsKeys + warp * kPiece;
    pages = at < ahead.s.length ? paged_entry(p, ahead.b, at) : -1;
  };
  const uint64_t once = l2_policy_evict_first();
  auto request = [&]() {
    if (ahead.step >= s1) return;
    const int page = __shfl_sync(0xffffffffu, pages, ahead.tile & 31);
    if (lane == 0) {
      const bool ok = page_ok(p, page);
      no_page[into] = !ok;
      if (!(p.test_withhold && ahead.step == first_step)) {  // test hook: the first tile never arrives
        const uint32_t dst = ring + static_cast<uint32_t>(into * L::kPieceBytes), bar = bars + 8 * into;
        const int slot = (ahead.tile * kPagedRowsKeys + warp * kPiece) & ((1 << p.page_shift) - 1);
        const int from = ok ? page : p.pages;  // behind the last page the copy engine reads zeros
        mbar_arrive_expect_tx(bar, L::kPieceBytes);
#pragma unroll
        for (int pn = 0; pn < L::kPanels; ++pn) {
          tma_load_4d_hint(dst + pn * L::kPanelBytes16, &tmK, bar, pn * 64, slot, ahead.head, from, once);
          tma_load_4d_hint(dst + L::kHalfBytes + pn * L::kPanelBytes16, &tmV, bar, pn * 64, slot, ahead.head, from, once);
        }
      }
    }
    if (++into == L::kStages) into = 0;
    ++under_way;
    ahead.next(p);
    find_page();
  };
  find_page();
  __syncwarp();  // the barriers are set up before lane 0 uses them, and for every lane
  for (int i = 0; i < L::kStages; ++i) request();
  __syncthreads();  // the abort flag too

  // this thread's rows in an accumulator: g and g + 8
  const int g = lane >> 2, c2 = 2 * (lane & 3);
  uint32_t qf[D / 16][4];
  int seen[2];   // positions that the rows see
  int all_seen;  // that every row sees
  auto load_q = [&](const TileCursor& t) {
    const int R = t.rows(p);
    all_seen = t.seen(p, t.block * kPagedRows / p.group);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = g + 8 * h, at = t.block * kPagedRows + min(row, R - 1), token = at / p.group;
      seen[h] = t.seen(p, token);
      const uint16_t* q = static_cast<const uint16_t*>(p.q) + (t.s.t0 + token) * p.q_token +
                          (t.head * p.group + (at - token * p.group)) * p.q_head + c2;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int i = 0; i < 2; ++i)  // a0: (g, k), a1: (g + 8, k), a2: (g, k + 8), a3: (g + 8, k + 8)
          qf[kk][h + 2 * i] = row < R ? __ldg(reinterpret_cast<const uint32_t*>(q + kk * 16 + 8 * i)) : 0u;
    }
  };
  float o[D / 8][4];
  float base[2], l[2], l_o[2];
  auto clear = [&]() {
#pragma unroll
    for (int d = 0; d < D / 8; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      base[i] = -CUDART_INF_F;
      l[i] = l_o[i] = 0.f;
    }
  };
  // ldmatrix addresses inside a piece: 16-byte chunk c of key row r lies at
  // chunk c ^ (r % 8) of its 64-column panel. K: rows 0-7 and 8-15, two
  // column halves each; V (transposed): rows 0-15 of two column halves.
  uint32_t k_off[4], v_off[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int kr = (lane & 7) + ((lane >> 4) << 3), vr = lane & 15;
    k_off[i] = static_cast<uint32_t>(kr * 128 + (((2 * i + ((lane >> 3) & 1)) ^ (lane & 7)) << 4));
    v_off[i] = static_cast<uint32_t>(L::kHalfBytes + vr * 128 + (((2 * i + (lane >> 4)) ^ (lane & 7)) << 4));
  }
  const float c = p.scale_log2;
  Watchdog wd;
  wd.status = p.status;
  wd.abort_flag = abort_flag;
  wd.limit_ns = p.watchdog_ns;

  // One piece: scores, weights and their products for this warp's 16 keys from
  // position `key` on.
  auto compute = [&](uint32_t at, int key, int length, bool lost) {
    // S: 16 rows x 16 keys (two n = 8 products), even and odd K-steps in
    // accumulators of their own
    float sc[2][2][4] = {};
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      uint32_t b[4];
      ldmatrix_x4(b, at + k_off[kk & 3] + (kk >> 2) * L::kPanelBytes16);
      mma_16816<kBf16>(sc[kk & 1][0], qf[kk], b[0], b[1]);
      mma_16816<kBf16>(sc[kk & 1][1], qf[kk], b[2], b[3]);
    }
    float x[2][4];  // [row g or g + 8][keys c2, c2 + 1, c2 + 8, c2 + 9]
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = 2 * i + (j & 1), nt = j >> 1;
        x[i][j] = sc[0][nt][e] + sc[1][nt][e];
      }
    if (lost) {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[0][j] = x[1][j] = CUDART_NAN_F;
    }
    if (key + kPiece > all_seen) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (key + c2 + (j & 1) + 8 * (j >> 1) >= seen[i]) x[i][j] = -CUDART_INF_F;
    }
    const int valid = length - key;
    const bool ragged = valid < kPiece;
    // move the bases only if some row's maximum passed its base by 2^8 (or has none yet)
    float top[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) top[i] = fmaxf(fmaxf(x[i][0], x[i][1]), fmaxf(x[i][2], x[i][3])) * c;
    if (__any_sync(0xffffffffu, top[0] > base[0] + kRescaleLog2 || top[1] > base[1] + kRescaleLog2)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
        float alpha = 1.f;
        if (top[i] > base[i] + kRescaleLog2) {
          alpha = ex2_approx(base[i] - top[i]);
          base[i] = top[i];
        }
        l[i] *= alpha;
        l_o[i] *= alpha;
#pragma unroll
        for (int d = 0; d < D / 8; ++d) {
          o[d][2 * i] *= alpha;
          o[d][2 * i + 1] *= alpha;
        }
      }
    }
    uint32_t pa[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float nb = base[i] == -CUDART_INF_F ? 0.f : -base[i];
      float pr[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        pr[j] = ex2_approx(fmaf(x[i][j], c, nb));
        l[i] += pr[j];
        l_o[i] += round16(pr[j], kBf16);  // O is normalised by the weights it is made of
      }
      pa[i] = pack2(pr[0], pr[1], kBf16);
      pa[2 + i] = pack2(pr[2], pr[3], kBf16);
    }
    // V's values of keys c2, c2 + 1 (first register of a product) and c2 + 8, c2 + 9
    uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
    if (ragged) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        keep[h] = (c2 + 8 * h < valid ? 0xffffu : 0u) | (c2 + 8 * h + 1 < valid ? 0xffff0000u : 0u);
    }
#pragma unroll
    for (int d = 0; d < D / 16; ++d) {
      uint32_t b[4];
      ldmatrix_x4_trans(b, at + v_off[d & 3] + (d >> 2) * L::kPanelBytes16);
      mma_16816<kBf16>(o[2 * d], pa, b[0] & keep[0], b[1] & keep[1]);
      mma_16816<kBf16>(o[2 * d + 1], pa, b[2] & keep[0], b[3] & keep[1]);
    }
  };

  load_q(cur);
  clear();
  bool from_start = cur.tile == 0;
  bool ok = true;
  int slot = 0;
  uint32_t phase = 0;
  while (cur.step < s1) {
    if (has_keys(cur)) {
      ok = ok && wait_bounded(bars + 8 * slot, phase, wd, kSitePagedPiece);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) {
        compute(ring + static_cast<uint32_t>(slot * L::kPieceBytes), cur.tile * kPagedRowsKeys + warp * kPiece,
                cur.s.length, no_page[slot] != 0);
        __syncwarp();  // every lane has read the piece: its slot is free
        --under_way;
        request();
        if (++slot == L::kStages) {
          slot = 0;
          phase ^= 1u;
        }
      }
    }
    const TileCursor done = cur;
    cur.next(p);
    const bool unit_end = done.tile == done.tiles - 1;
    const bool more = cur.step < s1;
    if (!unit_end && more) continue;
    // ------------------------------------------- the end of a unit (or share)
    if (more) load_q(cur);  // under way while the warps merge
    // the warps' bases and sums (each over the 4 threads of a row)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int off = 1; off < 4; off <<= 1) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
        l_o[i] += __shfl_xor_sync(0xffffffffu, l_o[i], off);
      }
      if ((lane & 3) == 0) {
        float* at = stats + warp * 3 * kPagedRows + g + 8 * i;
        at[0] = base[i];
        at[kPagedRows] = l[i];
        at[2 * kPagedRows] = l_o[i];
      }
    }
    // the holders of the unit's other tiles, if it is cut
    int last = blockIdx.x;
    if (from_start && !unit_end) {
      const long long end = done.step + done.tiles - done.tile;  // one past the unit's last tile
      while (last + 1 < shares && share_begin(last + 1) < end) ++last;
    }
    ok = !__syncthreads_or(!ok);
    if (!ok) break;
    // A cut unit's holder joins the partial results in its ring: the cut is
    // the end of the share, so nothing is under way there any more.
    const int others = last - static_cast<int>(blockIdx.x);
    float* const own = reinterpret_cast<float*>(smem);  // [16][D]
    const int R = done.rows(p);
    for (int i = 0; i < 2 && 8 * i < R; ++i) {  // rows [8 i, 8 i + 8)
      const int n_rows = min(8, R - 8 * i);
      float t = -CUDART_INF_F;
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) t = fmaxf(t, stats[w * 3 * kPagedRows + g + 8 * i]);
      const float own_base = i == 0 ? base[0] : base[1];
      const float f = own_base == -CUDART_INF_F ? 0.f : ex2_approx(own_base - t);
      // warps 4 to 7 leave their O, warps 0 to 3 add theirs; the four sums
      // meet where they are read
      float* const mine = merge + (warp & 3) * L::kBufFloats + g * L::kRowFloats + c2;
#pragma unroll
      for (int round = 0; round < 2; ++round) {
        if ((warp < 4) == (round == 1) && g < n_rows) {
#pragma unroll
          for (int d = 0; d < D / 8; ++d) {
            float2* at = reinterpret_cast<float2*>(mine + d * 8);
            float2 v = round == 0 ? make_float2(0.f, 0.f) : *at;
            v.x = fmaf(i == 0 ? o[d][0] : o[d][2], f, v.x);
            v.y = fmaf(i == 0 ? o[d][1] : o[d][3], f, v.y);
            *at = v;
          }
        }
        __syncthreads();
      }
      for (int e = threadIdx.x; e < n_rows * (D / 4); e += kRowThreads) {
        const int r8 = e / (D / 4), d = e - r8 * (D / 4), row = 8 * i + r8;
        float m = -CUDART_INF_F, sum = 0.f, sum_o = 0.f;
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) m = fmaxf(m, stats[w * 3 * kPagedRows + row]);
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) {
          const float* at = stats + w * 3 * kPagedRows + row;
          const float a = at[0] == -CUDART_INF_F ? 0.f : ex2_approx(at[0] - m);
          sum = fmaf(a, at[kPagedRows], sum);
          sum_o = fmaf(a, at[2 * kPagedRows], sum_o);
        }
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float4 u = *reinterpret_cast<const float4*>(merge + w * L::kBufFloats + r8 * L::kRowFloats + d * 4);
          v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
        }
        if (!from_start) {
          // not the unit's first tiles: leave the partial result to their holder
          float* ps = p.ws_stats + static_cast<size_t>(blockIdx.x) * 3 * kPagedRows + row;
          __stcg(reinterpret_cast<float4*>(p.ws_o + (static_cast<size_t>(blockIdx.x) * kPagedRows + row) * D) + d, v);
          if (d == 0) {
            __stcg(ps, m);
            __stcg(ps + kPagedRows, sum);
            __stcg(ps + 2 * kPagedRows, sum_o);
          }
          continue;
        }
        if (others > 0) {
          *reinterpret_cast<float4*>(own + row * D + d * 4) = v;
          if (d == 0) {
            float* at = own + kPagedRows * D + row;
            at[0] = m;
            at[kPagedRows] = sum;
            at[2 * kPagedRows] = sum_o;
          }
          continue;
        }
        write_row<D, kBf16>(p, done.out_row(p, row), d, v, m, sum, sum_o);
      }
      __syncthreads();  // the buffers are free again
    }
    if (!from_start) {
      // every thread's writes came before the barrier above: the release is cumulative over them
      if (threadIdx.x == 0) store_release(p.ws_flags + blockIdx.x, p.epoch);
    }
    if (others > 0) {
      ok = join_partials<D, kBf16>(p, own, others, done, R, wd);
      if (!ok) break;
    }
    clear();
    from_start = true;
  }
  // Only an aborted walk leaves pieces under way: they land before the CTA's
  // shared memory goes away.
  if (!ok) {
    for (; under_way > 0; --under_way) {
      wait_bounded(bars + 8 * slot, phase, wd, kSitePagedPiece, false, kNapNs);
      if (++slot == L::kStages) {
        slot = 0;
        phase ^= 1u;
      }
    }
  }
}

template <int D, bool kBf16>
cudaError_t launch_rows(const CUtensorMap& k, const CUtensorMap& v, const PagedAttnParams& p, int grid,
                        cudaStream_t stream) {
  auto kern = fa2_paged_rows_kernel<D, kBf16>;
  constexpr int smem = RowsLayout<D>::kSmemBytes;
  static PerDeviceOnce prepared;
  const cudaError_t e = once_per_device(
      prepared, [&]() { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
  if (e != cudaSuccess) return e;
  // the holder of a cut unit waits for other CTAs: all are resident, or the launch fails
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kRowThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, k, v, p);
}

}  // namespace

cudaError_t launch_paged_rows(int D, bool bf, const CUtensorMap& k, const CUtensorMap& v, const PagedAttnParams& p,
                              int grid, cudaStream_t s) {
  switch (D) {
    case 32: return bf ? launch_rows<32, true>(k, v, p, grid, s) : launch_rows<32, false>(k, v, p, grid, s);
    case 64: return bf ? launch_rows<64, true>(k, v, p, grid, s) : launch_rows<64, false>(k, v, p, grid, s);
    case 96: return bf ? launch_rows<96, true>(k, v, p, grid, s) : launch_rows<96, false>(k, v, p, grid, s);
    default: return bf ? launch_rows<128, true>(k, v, p, grid, s) : launch_rows<128, false>(k, v, p, grid, s);
  }
}

}  // namespace fa2
