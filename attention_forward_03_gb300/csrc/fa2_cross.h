// Host-visible pieces of cross attention (queries and keys of different
// lengths, per-batch key counts, grouped heads): the parameter blocks and the
// launcher templates, instantiated in fa2_cross_d{32,64,96,128}.cu.
//
// Grouped heads need no kernel of their own: without a causal mask every
// query row is independent, so the Hq / Hkv query heads that share a key
// head, adjacent in [B, Hq, Nq, D], are the rows of one [B * Hkv, G * Nq, D]
// tensor. The kernels see B * Hkv heads of N = G * Nq query rows.
#pragma once
#include "fa2_launch.h"

namespace fa2 {

struct CrossParams : Params {  // N: query rows per key head; BH: B * Hkv
  int Nk;                      // rows of K and V per head
  int B;
  int heads;                   // Hkv
  const int* key_lengths;      // [B] keys of each batch entry (clamped to [0, Nk]), or NULL: Nk
  int unit_cost;               // what a unit counts in the equal shares besides its tiles
  int key_split;               // a unit's sub-tiles are its keys' (D <= 64, N <= 128)
};

constexpr int kRangeRows = 64;  // divides a step's rows
struct CrossBwdParams : BwdParams {  // N: query rows per key head; nkv: K/V tiles of Nk keys
  int Nk;
  int B;
  int heads;
  const int* key_lengths;
  // One K/V tile per head (Nk <= 128): a query row's dQ is complete after its
  // only step, and goes out scaled and rounded ([B*Hkv, N, D]; NULL otherwise,
  // then it is added into dq_acc).
  void* dq_out;
  // fp16: the largest |dO_id| and |Delta_i| of every kRangeRows query rows,
  // [B*Hkv][Npad / kRangeRows], from which a unit's scale is taken
  // (cross_unit_shift in fa2_cross.cuh).
  const float2* range;
};

// Keys of batch entry b.
template <typename P>
__device__ __forceinline__ int cross_keys(const P& p, int b) {
  return p.key_lengths ? min(max(__ldg(p.key_lengths + b), 0), p.Nk) : p.Nk;
}

// The forward on the tensor-core kernel of fa2_kernel.cuh.
template <int D, bool kBf16>
cudaError_t launch_cross_fwd(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& o,
                             const CrossParams& p, int grid, cudaStream_t stream);

// Few query rows per key head (fa2_cross_rows.cu): 16 at most, 128 keys per
// tile, 16 of them for each of a CTA's 8 warps.
constexpr int kFewRows = 16;
constexpr int kFewRowsKeys = 128;
constexpr int kFewRowsMaxCtas = 256;  // what a cut unit's holder has room to join
struct CrossRowsParams : CrossParams {  // ws_o: [grid][16][D], ws_stats: [grid][3][16], ws_flags: [grid]
  const void* q;
};

constexpr size_t few_rows_workspace_bytes(int grid, int d) {
  return (static_cast<size_t>(grid) * kFewRows * (d + 3) * sizeof(float) + 255) / 256 * 256 +
         static_cast<size_t>(grid) * 8;
}

// k, v: maps with boxes of 16 rows x 64 elements.
cudaError_t launch_cross_rows(int D, bool bf16, const CUtensorMap& k, const CUtensorMap& v, const CrossRowsParams& p,
                              int grid, cudaStream_t stream);

// Few keys (fa2_cross_short.cu): 128 at most, all of them in shared memory.
constexpr int kFewKeys = 128;
constexpr int kFewKeysRows = 64;  // query rows per unit
struct CrossShortParams : CrossParams {  // n_qt: units per key head; num_units: BH * n_qt
  const void* q;
  const void* k;
  const void* v;
};
cudaError_t launch_cross_short(int D, bool bf16, const CrossShortParams& p, int sms, cudaStream_t stream);

// The backward on the tensor-core kernel of fa2_bwd_kernel.cuh.
template <int D, bool kBf16>
cudaError_t launch_cross_bwd(const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& q, const CUtensorMap& dout,
                             const CUtensorMap& dq_acc, const CrossBwdParams& p, int grid, cudaStream_t stream);

}  // namespace fa2
