// The write of a batch's new keys and values into a paged cache, and the choice
// and move of what stays in one when it is cut down.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "fa2_paged.cuh"

namespace fa2 {
namespace {

// Sequence that token t belongs to, or -1; `s` is it. The starts ascend, so
// the last one at or before t is searched for.
__device__ __forceinline__ int seq_of_token(const PagedBatch& p, int t, PagedSeq& s) {
  int b;
  if (!p.starts) {
    b = t / p.each;
  } else {
    int lo = 0, hi = p.B;  // the first start past t lies in (lo, hi]
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.starts + mid) > t) hi = mid;
      else lo = mid + 1;
    }
    b = lo - 1;
  }
  if (b < 0 || b >= p.B) return -1;
  s = paged_seq(p, b);
  return t >= s.t0 && t < s.t0 + s.n ? b : -1;
}

// ------------------------------------------------------------------ append
// Bound by bytes (each read and written once); a thread moves 16 of them.
template <int D>
__global__ void __launch_bounds__(256) fa2_paged_append_kernel(const PagedAppendParams p) {
  constexpr int kVecs = D / 8;  // 16-byte pieces of a row
  const int per_token = p.heads * 2 * kVecs;
  const long long items = static_cast<long long>(p.T) * per_token;
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < items; i += stride) {
    const int t = static_cast<int>(i / per_token);
    const int r = static_cast<int>(i - static_cast<long long>(t) * per_token);
    const int vec = r % kVecs, kv = (r / kVecs) & 1, head = r / (2 * kVecs);
    PagedSeq s;
    const int b = seq_of_token(p, t, s);
    if (b < 0) continue;
    const int pos = s.length - s.n + (t - s.t0);
    if (pos < 0) continue;  // more tokens than positions
    const int page = paged_entry(p, b, pos);
    if (!page_ok(p, page)) continue;
    const int slot = pos & ((1 << p.page_shift) - 1);
    const uint16_t* from = kv ? static_cast<const uint16_t*>(p.v) + t * p.v_token + head * p.v_head
                              : static_cast<const uint16_t*>(p.k) + t * p.k_token + head * p.k_head;
    const PagedStrides& cs = kv ? p.vs : p.ks;
    uint16_t* to = static_cast<uint16_t*>(kv ? p.vc : p.kc) + page * cs.page + head * cs.head + slot * cs.slot;
    reinterpret_cast<uint4*>(to)[vec] = __ldg(reinterpret_cast<const uint4*>(from) + vec);
    if (p.weights && kv == 0 && vec == 0)
      p.weights[((static_cast<long long>(page) * p.heads + head) << p.page_shift) + slot] = 0.f;
  }
}

// ------------------------------------------------------------------- evict
// Which positions stay: of those before the last `recent` the `need` of the
// greatest weight, found by a radix selection over the weights' bits as
// unsigned integers in the same order, then all that are above the threshold
// and the first of those at it, written in order.
constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kSelectKeys = 49152;  // bits of so many positions are kept in shared memory

// NaN above +inf; zeros of both signs equal.
__device__ __forceinline__ uint32_t ordered_bits(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelectThreads, 1) fa2_paged_select_kernel(const PagedEvictParams p) {
  extern __shared__ uint32_t bits[];
  __shared__ int hist[256];
  __shared__ int warp_above[kSelectWarps], warp_equal[kSelectWarps];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int b = blockIdx.x / p.heads, head = blockIdx.x - b * p.heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int length = min(max(__ldg(p.lengths + b), 0), p.capacity);
  const int m = min(length, p.keep);
  int* const kept = p.kept + static_cast<long long>(blockIdx.x) * p.keep;
  if (head == 0 && threadIdx.x == 0) p.new_lengths[b] = m;
  for (int i = m + threadIdx.x; i < p.keep; i += kSelectThreads) kept[i] = -1;
  if (length <= p.keep) {
    for (int i = threadIdx.x; i < m; i += kSelectThreads) kept[i] = i;
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
  if (in_smem)
    for (int i = threadIdx.x; i < old; i += kSelectThreads) bits[i] = read(i);
  auto key = [&](int i) { return in_smem ? bits[i] : read(i); };
  if (threadIdx.x == 0) {
    s_prefix = 0;
    s_need = p.keep - p.recent;
  }
  __syncthreads();
  // The threshold, 8 bits at a time from the top: the prefix that the need-th
  // greatest has, and how many are needed among those with it.
  const int rounds = (old + kSelectThreads - 1) / kSelectThreads;
  if (s_need > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (threadIdx.x < 256) hist[threadIdx.x] = 0;
      __syncthreads();
      const uint32_t prefix = s_prefix;
      for (int r = 0; r < rounds; ++r) {
        const int i = r * kSelectThreads + threadIdx.x;
        const uint32_t u = i < old ? key(i) : 0u;
        const bool in = i < old && (shift == 24 || (u >> (shift + 8)) == prefix);
        const unsigned who = __ballot_sync(0xffffffffu, in);
        if (in) {
          const int digit = (u >> shift) & 255;
          const unsigned same = __match_any_sync(who, digit);
          if (__ffs(same) - 1 == lane) atomicAdd(&hist[digit], __popc(same));
        }
      }
      __syncthreads();
      if (warp == 0) {
        // lane l holds digits 255 - 8 l .. 248 - 8 l; how many lie above
        int sum = 0;
#pragma unroll
        for (int d = 0; d < 8; ++d) sum += hist[255 - 8 * lane - d];
        int upto = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, upto, off);
          if (lane >= off) upto += v;
        }
        const int need = s_need;
        __syncwarp();
        int above = upto - sum;
        if (above < need && need <= upto) {
          int d = 255 - 8 * lane;
          while (above + hist[d] < need && (d & 7)) above += hist[d--];  // at most its 8 digits
          s_prefix = (prefix << 8) | static_cast<uint32_t>(d);
          s_need = need - above;
        }
      }
      __syncthreads();
    }
  }
  const uint32_t threshold = s_prefix;
  const int equal_kept = s_need;  // of the positions at the threshold
  const bool any = p.keep > p.recent;
  // each warp a run of positions: how many above and at the threshold, then written in order
  const int run = ((old + kSelectWarps - 1) / kSelectWarps + 31) / 32 * 32;
  const int from = min(old, warp * run), to = min(old, from + run);
  int above = 0, equal = 0;
  if (any)
    for (int i0 = from; i0 < to; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t u = i < to ? key(i) : 0u;
      above += __popc(__ballot_sync(0xffffffffu, i < to && u > threshold));
      equal += __popc(__ballot_sync(0xffffffffu, i < to && u == threshold));
    }
  if (lane == 0) {
    warp_above[warp] = above;
    warp_equal[warp] = equal;
  }
  __syncthreads();
  if (any) {
    int at = 0, eq = 0;
    for (int w = 0; w < warp; ++w) {
      at += warp_above[w];
      eq += warp_equal[w];
    }
    at += min(eq, equal_kept);
    for (int i0 = from; i0 < to; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t u = i < to ? key(i) : 0u;
      const bool gt = i < to && u > threshold, is = i < to && u == threshold;
      const unsigned below = (1u << lane) - 1u;
      const unsigned eqs = __ballot_sync(0xffffffffu, is);
      const bool stays = gt || (is && eq + __popc(eqs & below) < equal_kept);
      const unsigned all = __ballot_sync(0xffffffffu, stays);
      if (stays && at + __popc(all & below) < p.keep - p.recent) kept[at + __popc(all & below)] = i;
      at += __popc(all);
      eq += __popc(eqs);
    }
  }
  for (int i = threadIdx.x; i < p.recent; i += kSelectThreads) kept[p.keep - p.recent + i] = old + i;
}

// Keys, values and weights of the kept positions to their new pages: bound by
// bytes, 16 of them per thread and step.
template <int D>
__global__ void __launch_bounds__(256) fa2_paged_move_kernel(const PagedEvictParams p) {
  constexpr int kVecs = D / 8;
  const int per_row = 2 * kVecs;
  const long long rows = static_cast<long long>(p.B) * p.heads * p.keep;
  const long long items = rows * per_row;
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  const int in_page = (1 << p.page_shift) - 1;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < items; i += stride) {
    const long long row = i / per_row;
    const int r = static_cast<int>(i - row * per_row), vec = r % kVecs, kv = r / kVecs;
    const int src = __ldg(p.kept + row);
    if (src < 0) continue;
    const int bh = static_cast<int>(row / p.keep), j = static_cast<int>(row - static_cast<long long>(bh) * p.keep);
    const int b = bh / p.heads, head = bh - b * p.heads;
    const int from = paged_entry(p, b, src), to = __ldg(p.new_table + b * p.new_stride + (j >> p.page_shift));
    if (!page_ok(p, to)) continue;
    const bool there = page_ok(p, from);
    const PagedStrides& cs = kv ? p.vs : p.ks;
    uint16_t* const c = static_cast<uint16_t*>(kv ? p.vc : p.kc) + head * cs.head;
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
    if (there) u = reinterpret_cast<const uint4*>(c + from * cs.page + (src & in_page) * cs.slot)[vec];
    reinterpret_cast<uint4*>(c + to * cs.page + (j & in_page) * cs.slot)[vec] = u;
    if (r == 0) {
      const float w = there ? p.weights[((static_cast<long long>(from) * p.heads + head) << p.page_shift) + (src & in_page)] : 0.f;
      p.weights[((static_cast<long long>(to) * p.heads + head) << p.page_shift) + (j & in_page)] = w;
    }
  }
}

template <typename P, typename F>
cudaError_t launch_flat(F kern, const P& p, long long items, int sms, cudaStream_t s) {
  const int grid = static_cast<int>(std::min<long long>((items + 255) / 256, 8ll * sms));
  kern<<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(int D, const PagedAppendParams& p, int sms, cudaStream_t s) {
  const long long items = static_cast<long long>(p.T) * p.heads * 2 * (D / 8);
  switch (D) {
    case 32: return launch_flat(fa2_paged_append_kernel<32>, p, items, sms, s);
    case 64: return launch_flat(fa2_paged_append_kernel<64>, p, items, sms, s);
    case 96: return launch_flat(fa2_paged_append_kernel<96>, p, items, sms, s);
    default: return launch_flat(fa2_paged_append_kernel<128>, p, items, sms, s);
  }
}

cudaError_t launch_paged_evict(int D, const PagedEvictParams& p, int sms, cudaStream_t s) {
  constexpr int kMost = kSelectKeys * 4;
  static PerDeviceOnce prepared;
  cudaError_t e = once_per_device(prepared, [&]() {
    return cudaFuncSetAttribute(fa2_paged_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
  });
  if (e != cudaSuccess) return e;
  const int smem = std::min(p.capacity, kSelectKeys) * 4;
  fa2_paged_select_kernel<<<p.B * p.heads, kSelectThreads, smem, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const long long items = static_cast<long long>(p.B) * p.heads * p.keep * 2 * (D / 8);
  if (items == 0) return cudaSuccess;
  switch (D) {
    case 32: return launch_flat(fa2_paged_move_kernel<32>, p, items, sms, s);
    case 64: return launch_flat(fa2_paged_move_kernel<64>, p, items, sms, s);
    case 96: return launch_flat(fa2_paged_move_kernel<96>, p, items, sms, s);
    default: return launch_flat(fa2_paged_move_kernel<128>, p, items, sms, s);
  }
}

}  // namespace fa2
