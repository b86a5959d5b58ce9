// The write of a batch's new keys and values into a paged cache, and the choice
// and move of what stays in one when it is cut down.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "fa2_paged.cuh"

namespace fa2 {
namespace {

// Sequence that token t belongs to, or -1; `s` is it. By one whole warp: the
// starts ascend, and the last one at or before t is searched for among 32
// candidates at a time.
__device__ __forceinline__ int seq_of_token(const PagedBatch& p, int t, PagedSeq& s) {
  int b;
  if (!p.starts) {
    b = t / p.each;
  } else {
    const int lane = threadIdx.x & 31;
    int lo = -1, hi = p.B;  // starts[lo] <= t < starts[hi]
    while (hi - lo > 1) {
      const int by = (hi - lo + 31) / 32, m = lo + (lane + 1) * by;
      const bool before = m < hi && __ldg(p.starts + m) <= t;
      lo += __popc(__ballot_sync(0xffffffffu, before)) * by;
      hi = min(hi, lo + by);
    }
    b = lo;
  }
  if (b < 0 || b >= p.B) return -1;
  s = paged_seq(p, b);
  return t >= s.t0 && t < s.t0 + s.n ? b : -1;
}

// ------------------------------------------------------------------ append
// Bound by bytes, each read and written once. A warp takes a token: 16 bytes of
// its keys' and values' rows per lane and step, up to eight of them under way
// while the token's sequence and page are looked up. 20,480 tokens of 8 heads
// of 128: 27.7 us, 6.1 TB/s (floor 24.8); with a thread to a piece, each looking
// its token up, 46.
constexpr int kMoveThreads = 256;
constexpr int kUnder = 8;  // 16-byte pieces under way per lane

template <int D>
__global__ void __launch_bounds__(kMoveThreads) fa2_paged_append_kernel(const PagedAppendParams p) {
  constexpr int kVecs = D / 8;  // 16-byte pieces of a row
  const int lane = threadIdx.x & 31;
  const int items = p.heads * 2 * kVecs;  // of a token: [head][K, V][piece]
  const int warps = gridDim.x * (kMoveThreads / 32);
  for (int t = blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5); t < p.T; t += warps) {
    const uint16_t* const k = static_cast<const uint16_t*>(p.k) + t * p.k_token;
    const uint16_t* const v = static_cast<const uint16_t*>(p.v) + t * p.v_token;
    int page = -1, slot = 0;
    for (int i0 = 0; i0 < items; i0 += 32 * kUnder) {
      uint4 piece[kUnder];
#pragma unroll
      for (int j = 0; j < kUnder; ++j) {
        const int i = i0 + 32 * j + lane, head = i / (2 * kVecs), r = i - head * 2 * kVecs;
        if (i < items)
          piece[j] = __ldg(reinterpret_cast<const uint4*>(r < kVecs ? k + head * p.k_head : v + head * p.v_head) +
                           (r < kVecs ? r : r - kVecs));
      }
      if (i0 == 0) {
        PagedSeq s;
        const int b = seq_of_token(p, t, s);
        const int pos = b < 0 ? -1 : s.length - s.n + (t - s.t0);
        if (pos >= 0) page = paged_entry(p, b, pos);  // (of more tokens than positions the first ones have none)
        slot = pos & ((1 << p.page_shift) - 1);
      }
      if (!page_ok(p, page)) break;
#pragma unroll
      for (int j = 0; j < kUnder; ++j) {
        const int i = i0 + 32 * j + lane, head = i / (2 * kVecs), r = i - head * 2 * kVecs;
        if (i >= items) continue;
        const bool is_k = r < kVecs;
        const PagedStrides& c = is_k ? p.ks : p.vs;
        uint16_t* const to = static_cast<uint16_t*>(is_k ? p.kc : p.vc) + page * c.page + head * c.head + slot * c.slot;
        reinterpret_cast<uint4*>(to)[is_k ? r : r - kVecs] = piece[j];
      }
    }
    if (!p.weights || !page_ok(p, page)) continue;
    for (int head = lane; head < p.heads; head += 32)
      p.weights[((static_cast<long long>(page) * p.heads + head) << p.page_shift) + slot] = 0.f;
  }
}

// ------------------------------------------------------------------- evict
// Keys, values and weights of the kept positions to their new pages: bound by
// bytes. A warp takes runs of up to 32 rows: a lane looks up a row each, then
// 16 bytes per lane and step, eight of them under way. 64 heads of 2048 kept
// rows of 128: 22 us, 6.1 TB/s.
template <int D>
struct Moves {
  static constexpr int kVecs = D / 8;
  static constexpr int kRowsAtOnce = 32 / (2 * kVecs) > 0 ? 32 / (2 * kVecs) : 1;  // rows (K and V) of a step
  static constexpr int kRun = kRowsAtOnce * kUnder;                                  // rows of a run: 8, 16 or 32
  static_assert(kRun <= 32 && 2 * kVecs <= 32, "a lane per row and piece");

  // By one warp: kept rows j0, j0 + 1, .. of key head bh (counted over the sequences).
  static __device__ __forceinline__ void run(const PagedEvictParams& p, int bh, int j0) {
    const int lane = threadIdx.x & 31, in_page = (1 << p.page_shift) - 1;
    const int b = bh / p.heads, head = bh - b * p.heads;
    // this lane's piece of a step: row, cache, 16 bytes
    const int row_of = lane / (2 * kVecs), r = lane - row_of * 2 * kVecs;
    const bool is_k = r < kVecs, works = row_of < kRowsAtOnce;
    const int vec = is_k ? r : r - kVecs;
    const PagedStrides& c = is_k ? p.ks : p.vs;
    // lane l: row j0 + l; `from`: its old page or -1, `to`: its new one or -1
    int src = -1, from = -1, to = -1;
    if (lane < kRun && j0 + lane < p.keep) src = p.kept[static_cast<long long>(bh) * p.keep + j0 + lane];
    if (src >= 0) {
      from = paged_entry(p, b, src);
      to = __ldg(p.new_table + b * p.new_stride + ((j0 + lane) >> p.page_shift));
      if (!page_ok(p, from)) from = -1;
      if (!page_ok(p, to)) to = -1;
    }
    if (__all_sync(0xffffffffu, src < 0)) return;
    uint16_t* const cache = static_cast<uint16_t*>(is_k ? p.kc : p.vc) + head * c.head;
    uint4 piece[kUnder];
#pragma unroll
    for (int i = 0; i < kUnder; ++i) {
      const int row = i * kRowsAtOnce + (works ? row_of : 0);
      const int f = __shfl_sync(0xffffffffu, from, row), s = __shfl_sync(0xffffffffu, src, row);
      piece[i] = make_uint4(0u, 0u, 0u, 0u);  // of a position whose page is none
      if (works && f >= 0) piece[i] = reinterpret_cast<const uint4*>(cache + f * c.page + (s & in_page) * c.slot)[vec];
    }
    float w = 0.f;
    if (from >= 0) w = p.weights[((static_cast<long long>(from) * p.heads + head) << p.page_shift) + (src & in_page)];
#pragma unroll
    for (int i = 0; i < kUnder; ++i) {
      const int row = i * kRowsAtOnce + (works ? row_of : 0);
      const int t = __shfl_sync(0xffffffffu, to, row);
      if (works && t >= 0) reinterpret_cast<uint4*>(cache + t * c.page + ((j0 + row) & in_page) * c.slot)[vec] = piece[i];
    }
    if (to >= 0) p.weights[((static_cast<long long>(to) * p.heads + head) << p.page_shift) + ((j0 + lane) & in_page)] = w;
  }
};

// Which positions stay: of those before the last `recent` the `need` of the
// greatest weight, found by a radix selection over the weights' bits as
// unsigned integers in the same order (11, 11 and 10 bits at a time), then all
// that are above the threshold and the first of those at it, written in order.
// One block for each key head of a sequence. What bounds it is latency: the
// rounds over the positions and the three scans of the counts (64 heads of 8192
// positions: 12 us; digits of 8 bits, each position counted by itself: 4 more).
// Of more than kSelectKeys positions every pass reads the table and the weights
// again (8 key heads of one sequence cut to 2048, with the move: of 49,152 positions
// 49 us, of 65,536 126, of 131,072 239).
constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kSelectKeys = 49152;  // bits of so many positions are kept in shared memory
constexpr int kBins = 2048;         // of a digit

// NaN above +inf; zeros of both signs equal.
__device__ __forceinline__ uint32_t ordered_bits(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// `kMoves`: the block moves its key head's rows itself afterwards.
template <int D, bool kMoves>
__global__ void __launch_bounds__(kSelectThreads, 1) fa2_paged_select_kernel(const PagedEvictParams p) {
  extern __shared__ __align__(16) uint32_t bits[];
  __shared__ int hist[kBins];
  __shared__ int warp_sum[kSelectWarps];
  __shared__ int warp_above[kSelectWarps], warp_equal[kSelectWarps];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  if constexpr (!kMoves) cudaTriggerProgrammaticLaunchCompletion();  // the moving kernel may take the SMs that are free
  const int b = blockIdx.x / p.heads, head = blockIdx.x - b * p.heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int length = min(max(__ldg(p.lengths + b), 0), p.capacity);
  const int m = min(length, p.keep);
  int* const kept = p.kept + static_cast<long long>(blockIdx.x) * p.keep;
  if (head == 0 && threadIdx.x == 0) p.new_lengths[b] = m;
  for (int i = m + threadIdx.x; i < p.keep; i += kSelectThreads) kept[i] = -1;
  auto move = [&]() {
    if constexpr (kMoves) {
      __syncthreads();  // the kept positions are all written
      for (int j0 = warp * Moves<D>::kRun; j0 < m; j0 += kSelectWarps * Moves<D>::kRun) Moves<D>::run(p, blockIdx.x, j0);
    }
  };
  if (length <= p.keep) {
    for (int i = threadIdx.x; i < m; i += kSelectThreads) kept[i] = i;
    move();
    return;
  }
  const int old = length - p.recent;  // positive: recent <= keep < length
  const bool in_smem = old <= kSelectKeys;
  auto read = [&](int i) -> uint32_t {
    const int page = paged_entry(p, b, i);
    if (!page_ok(p, page)) return 0u;  // below every weight
    return ordered_bits(__ldg(p.weights + ((static_cast<long long>(page) * p.heads + head) << p.page_shift) +
                              (i & ((1 << p.page_shift) - 1))));
  };
  if (in_smem) {
    // the pages, then the weights of eight positions at once (one after another: 1.5 us
    // of latency for every 1024 positions)
    for (int i0 = threadIdx.x; i0 < old; i0 += 8 * kSelectThreads) {
      int page[8];
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) page[j] = i0 + j * kSelectThreads < old ? paged_entry(p, b, i0 + j * kSelectThreads) : -1;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (page_ok(p, page[j]))
          w[j] = __ldg(p.weights + ((static_cast<long long>(page[j]) * p.heads + head) << p.page_shift) +
                       ((i0 + j * kSelectThreads) & ((1 << p.page_shift) - 1)));
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i0 + j * kSelectThreads < old) bits[i0 + j * kSelectThreads] = page_ok(p, page[j]) ? ordered_bits(w[j]) : 0u;
    }
  }
  // four positions' keys from i, a multiple of 4, on
  auto keys4 = [&](int i) {
    if (in_smem) return *reinterpret_cast<const uint4*>(bits + i);  // (past `old`: anything)
    return make_uint4(read(i), i + 1 < old ? read(i + 1) : 0u, i + 2 < old ? read(i + 2) : 0u, i + 3 < old ? read(i + 3) : 0u);
  };
  if (threadIdx.x == 0) {
    s_prefix = 0;
    s_need = p.keep - p.recent;
  }
  __syncthreads();
  // The threshold, a digit at a time from the top: the prefix that the need-th
  // greatest has, and how many are needed among those with it.
  if (s_need > 0) {
    for (int digits = 0; digits < 3; ++digits) {
      const int shift = digits == 0 ? 21 : digits == 1 ? 10 : 0, width = digits == 2 ? 10 : 11;
      hist[threadIdx.x] = hist[threadIdx.x + kSelectThreads] = 0;
      __syncthreads();
      const uint32_t prefix = s_prefix;
      auto count = [&](uint32_t u, bool there) {
        const bool in = there && (digits == 0 || (u >> (shift + width)) == prefix);
        const int digit = (u >> shift) & ((1 << width) - 1);
        // equal weights meet in one count: a warp of them adds once
        const unsigned who = __ballot_sync(0xffffffffu, in);
        if (in) {
          int same;
          __match_all_sync(who, digit, &same);
          if (!same) atomicAdd(&hist[digit], 1);
          else if (__ffs(who) - 1 == lane) atomicAdd(&hist[digit], __popc(who));
        }
      };
      for (int i0 = 0; i0 < old; i0 += 4 * kSelectThreads) {
        const int i = i0 + 4 * static_cast<int>(threadIdx.x);
        if (i0 + 128 * warp >= old) break;  // none of the warp's
        const uint4 u = i < old ? keys4(i) : make_uint4(0u, 0u, 0u, 0u);
        count(u.x, i < old);
        count(u.y, i + 1 < old);
        count(u.z, i + 2 < old);
        count(u.w, i + 3 < old);
      }
      __syncthreads();
      // thread i: digits 2047 - 2 i and 2046 - 2 i; how many lie above
      const int bin = kBins - 1 - 2 * static_cast<int>(threadIdx.x);
      const int high = hist[bin], sum = high + hist[bin - 1];
      int upto = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += v;
      }
      if (lane == 31) warp_sum[warp] = upto;
      __syncthreads();
      int warps_before = lane < warp ? warp_sum[lane] : 0;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) warps_before += __shfl_xor_sync(0xffffffffu, warps_before, off);
      const int need = s_need, above = warps_before + upto - sum;
      __syncthreads();  // everyone has read the need
      if (above < need && need <= above + sum) {
        const bool first = above + high >= need;
        s_prefix = (prefix << width) | static_cast<uint32_t>(first ? bin : bin - 1);
        s_need = need - above - (first ? 0 : high);
      }
      __syncthreads();
    }
  }
  const uint32_t threshold = s_prefix;
  const int equal_kept = s_need;  // of the positions at the threshold
  const bool any = p.keep > p.recent;
  // Each warp a run of positions, eight neighbouring ones to a lane and step: how
  // many lie above and at the threshold (in two halves of one number), then the
  // places of those that stay.
  constexpr int kStep = 8 * 32;
  const int run = ((old + kSelectWarps - 1) / kSelectWarps + kStep - 1) / kStep * kStep;
  const int from = min(old, warp * run), to = min(old, from + run);
  auto keys8 = [&](int i, uint32_t (&u)[8]) {
    const uint4 a = i < to ? keys4(i) : make_uint4(0u, 0u, 0u, 0u), b = i + 4 < to ? keys4(i + 4) : make_uint4(0u, 0u, 0u, 0u);
    u[0] = a.x; u[1] = a.y; u[2] = a.z; u[3] = a.w;
    u[4] = b.x; u[5] = b.y; u[6] = b.z; u[7] = b.w;
  };
  // (above, at) of a lane's eight, 16 bits each: a step of a warp has 256 at most
  auto counts = [&](const uint32_t (&u)[8], int i) {
    unsigned n = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + k < to) n += (u[k] > threshold ? 1u : 0u) + (u[k] == threshold ? 0x10000u : 0u);
    return n;
  };
  int above = 0, equal = 0;
  if (any)
    for (int i0 = from; i0 < to; i0 += kStep) {
      uint32_t u[8];
      keys8(i0 + 8 * lane, u);
      const unsigned n = __reduce_add_sync(0xffffffffu, counts(u, i0 + 8 * lane));
      above += n & 0xffffu;
      equal += n >> 16;
    }
  if (lane == 0) {
    warp_above[warp] = above;
    warp_equal[warp] = equal;
  }
  __syncthreads();
  if (any && from < to) {
    int at = __reduce_add_sync(0xffffffffu, lane < warp ? warp_above[lane] : 0);
    int eq = __reduce_add_sync(0xffffffffu, lane < warp ? warp_equal[lane] : 0);
    // `at`: above the threshold so far; `eq`: at it, of which the first equal_kept stay
    for (int i0 = from; i0 < to; i0 += kStep) {
      const int i = i0 + 8 * lane;
      uint32_t u[8];
      keys8(i, u);
      const unsigned mine = counts(u, i);
      unsigned upto = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const unsigned v = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += v;
      }
      const unsigned all = __shfl_sync(0xffffffffu, upto, 31);
      int lane_at = at + static_cast<int>((upto - mine) & 0xffffu), lane_eq = eq + static_cast<int>((upto - mine) >> 16);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (i + k >= to) continue;
        const bool gt = u[k] > threshold, is = u[k] == threshold;
        const int place = lane_at + min(lane_eq, equal_kept);
        if ((gt || (is && lane_eq < equal_kept)) && place < p.keep - p.recent) kept[place] = i + k;
        lane_at += gt;
        lane_eq += is;
      }
      at += all & 0xffffu;
      eq += all >> 16;
    }
  }
  for (int i = threadIdx.x; i < p.recent; i += kSelectThreads) kept[p.keep - p.recent + i] = old + i;
  move();
}

// The moves of all key heads by as many warps as there are SMs for.
template <int D>
__global__ void __launch_bounds__(kMoveThreads) fa2_paged_move_kernel(const PagedEvictParams p) {
  cudaGridDependencySynchronize();  // what the selection wrote
  constexpr int kRun = Moves<D>::kRun;
  const int runs = (p.keep + kRun - 1) / kRun;  // of a key head of a sequence
  const long long all = static_cast<long long>(p.B) * p.heads * runs;
  const long long warps = static_cast<long long>(gridDim.x) * (kMoveThreads / 32);
  for (long long run = static_cast<long long>(blockIdx.x) * (kMoveThreads / 32) + (threadIdx.x >> 5); run < all; run += warps) {
    const int bh = static_cast<int>(run / runs);
    Moves<D>::run(p, bh, static_cast<int>(run - static_cast<long long>(bh) * runs) * kRun);
  }
}

// At most 8 blocks per SM; `dependent`: the kernel may be set up while the one before it still runs.
template <typename P, typename F>
cudaError_t launch_moves(F kern, const P& p, long long warps, int sms, bool dependent, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>((warps * 32 + kMoveThreads - 1) / kMoveThreads, 8ll * sms)));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

// Up to so many bytes of a key head the block that chose its rows moves them
// too, without a second kernel. Of 2500 positions, D = 64 and 8 key heads (us,
// one block / second kernel): 32 KB 10.6 / 11.3, 64 KB 11.2 / 11.5, 128 KB 13.3 /
// 11.6; 256 key heads: 20.0 / 21.9, 21.6 / 21.9, 26.2 / 26.2; and the host
// launches once.
constexpr long long kOwnMoveBytes = 64 << 10;

template <int D, bool kMoves>
cudaError_t launch_select(const PagedEvictParams& p, cudaStream_t s) {
  constexpr int kMost = kSelectKeys * 4;
  auto kern = fa2_paged_select_kernel<D, kMoves>;
  static PerDeviceOnce prepared;
  const cudaError_t e = once_per_device(
      prepared, [&]() { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost); });
  if (e != cudaSuccess) return e;
  kern<<<p.B * p.heads, kSelectThreads, std::min(p.capacity, kSelectKeys) * 4, s>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_evict(const PagedEvictParams& p, int sms, cudaStream_t s) {
  if (static_cast<long long>(p.keep) * D * 4 <= kOwnMoveBytes) return launch_select<D, true>(p, s);
  const cudaError_t e = launch_select<32, false>(p, s);  // the same for every head dimension
  if (e != cudaSuccess) return e;
  constexpr int rows = Moves<D>::kRun;
  return launch_moves(fa2_paged_move_kernel<D>, p, static_cast<long long>(p.B) * p.heads * ((p.keep + rows - 1) / rows), sms,
                      true, s);
}

}  // namespace

cudaError_t launch_paged_append(int D, const PagedAppendParams& p, int sms, cudaStream_t s) {
  switch (D) {
    case 32: return launch_moves(fa2_paged_append_kernel<32>, p, p.T, sms, false, s);
    case 64: return launch_moves(fa2_paged_append_kernel<64>, p, p.T, sms, false, s);
    case 96: return launch_moves(fa2_paged_append_kernel<96>, p, p.T, sms, false, s);
    default: return launch_moves(fa2_paged_append_kernel<128>, p, p.T, sms, false, s);
  }
}

cudaError_t launch_paged_evict(int D, const PagedEvictParams& p, int sms, cudaStream_t s) {
  switch (D) {
    case 32: return launch_evict<32>(p, sms, s);
    case 64: return launch_evict<64>(p, sms, s);
    case 96: return launch_evict<96>(p, sms, s);
    default: return launch_evict<128>(p, sms, s);
  }
}

}  // namespace fa2
