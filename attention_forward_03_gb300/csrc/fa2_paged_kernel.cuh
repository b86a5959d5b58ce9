// Attention of a batch's new tokens over a paged cache on the tensor cores:
// sequences with more than 16 query rows per key head (chunks of prompts, whole
// prompts). The design is that of fa2_kernel.cuh (persistent CTAs, TMA loads,
// tcgen05 products accumulating in tensor memory, one softmax warpgroup per
// 128-row sub-tile, equal shares of all K/V tiles per CTA with a merge of the
// units that are cut); what is different:
//
//   rows      a sub-tile is 128 / group tokens of one sequence with all the
//             query heads of one key head, row = token * group + head: one box
//             of the map (D, head, token) of q. K and V are read once for all
//             of them. Rows past the sequence's tokens see no key.
//   tiles     128 positions, from one box per page of the map (D, slot, head,
//             page) of the cache: the producer warp's lanes hold one page
//             number each, read a tile ahead, and each issues its page's boxes.
//             Pages past the last position are not loaded; a page number that
//             is none leaves NaN in K's rows (written by the lane) and zeros in
//             V's (out of the map).
//   mask      a row sees its token's position and the earlier ones, so units
//             have different numbers of tiles; the walk (fa2_paged_walk.cuh)
//             counts them in closed form.
//   output    through the warp's own rows of the P buffer (its own buffer where
//             P lives in tensor memory), so that a row's 256 bytes go out
//             together, 16-byte chunks by neighbouring lanes; rows of a next
//             sequence may follow, so no box of rows is stored. (Boxes of a
//             warp's 32 rows, where they are whole tokens of the sequence, made
//             no difference: 222 and 220 us for four prompts of 4096.)
//
// Measured: four prompts of 4096, 16 query heads on 4 key heads of 128, 220 us
// (1,250 TFLOP/s, 64 % of the measured peak; floor 140): a tile step takes about
// 1.3 us, bound by shared memory (K, V and P are read from it) with a ring of
// three tiles, and the power cap lowers the clock. 512 tokens over 8192
// positions, 32 query heads on 8 key heads: 58 us (floor 34), with about 5 for the
// start (search of the share, first instructions and loads) and a join of cut
// units at the end; 64 tokens 26 us, a unit's 19 CTAs joining its rows. At D = 64
// the exponentials bound it. Issuers by type where D > 64 and by sub-tile below, as
// in fa2_kernel.cuh; at D = 64 that, rows without a token unmasked and the rules for
// cutting took a mixed batch from 88 to 66 us together.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <type_traits>

#include "fa2_cross.cuh"
#include "fa2_paged_walk.cuh"

namespace fa2 {

template <int D>
struct PagedLayout {
  static constexpr int kPanels = (D + 63) / 64;
  static constexpr int kDp = kPanels * 64;
  static constexpr int kTileBytes = kPanels * kPanelBytes;
  static constexpr bool kPInTmem = kPanels == 1;
  static constexpr int kStages = kPanels == 2 ? 3 : 10;
  static constexpr int kNpv = D == 32 ? 64 : D;  // N of P.V, as in fa2_kernel.cuh
  static constexpr int kQBytes = kSubTiles * kTileBytes;
  static constexpr int kPOffset = kQBytes;  // P and the rows on their way out; with P in tensor memory those alone
  static constexpr int kPBytes = kPInTmem ? kPanelBytes : kPTileBytes;  // per sub-tile
  static constexpr int kRingOffset = kPOffset + kSubTiles * kPBytes;
  static constexpr int kBarOffset = kRingOffset + kStages * kTileBytes;
  // q_full, q_empty, ring full (K)[S], ring full (V)[S], ring empty[S], s_full[2], s_free[2], p_full[2], p_free[2],
  // o_full[2], drain[2], part[2]
  static constexpr int kNumBars = 2 + 3 * kStages + 2 * 7;
  static constexpr int kMiscOffset = kBarOffset + kNumBars * 8;
  static constexpr int kStartOffset = kMiscOffset + 16;
  static constexpr int kSmemBytes = kStartOffset + static_cast<int>(sizeof(PagedStart)) + 1024;
  static constexpr uint32_t kColO = 2 * kKeys;
  static constexpr uint32_t kColP = kColO + 2 * kDp;
  static_assert(kColO + 2 * kDp + (kPInTmem ? 2 * kKeys / 2 : 0) <= kTmemCols, "TMEM budget");
  static_assert(kSmemBytes <= 232448, "shared memory budget");
  static_assert(kStartOffset % alignof(PagedStart) == 0, "alignment");
};

template <int D, bool kBf16>
__global__ void __launch_bounds__(kThreads, 1)
    fa2_paged_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const PagedTileParams p) {
  using L = PagedLayout<D>;
  // issuers by instruction type (one thread for every S, one for every P.V) or by
  // sub-tile: as in fa2_kernel.cuh
  constexpr bool kTypeSplit = L::kPanels == 2;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t sQ = base, sP = base + L::kPOffset, sRing = base + L::kRingOffset, bars = base + L::kBarOffset;
  const uint32_t bar_q_full = bars, bar_q_empty = bars + 8;
  // K and V tiles have "full" barriers of their own in every slot, as in fa2_kernel.cuh
  auto bar_full = [&](int s, uint32_t is_v) { return bars + 16 + 8u * (is_v * L::kStages + s); };
  auto bar_empty = [&](int s) { return bars + 16 + 8u * (2 * L::kStages + s); };
  const uint32_t bar_s_full0 = bars + 16 + 24u * L::kStages;  // these: [sub-tile]
  const uint32_t bar_s_free0 = bar_s_full0 + 16;
  const uint32_t bar_p_full0 = bar_s_free0 + 16;
  const uint32_t bar_p_free0 = bar_p_full0 + 16;
  const uint32_t bar_o_full0 = bar_p_free0 + 16;
  const uint32_t bar_drain = bar_o_full0 + 16;  // [issuer]
  const uint32_t bar_part0 = bar_drain + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOffset);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOffset + 4);
  PagedStart* const start = reinterpret_cast<PagedStart*>(smem + L::kStartOffset);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (warp == 0) {
    const PagedStart st = paged_start(p);
    if (lane == 0) *start = st;
  }
  if (threadIdx.x == 32) {
    mbar_init(bar_q_full, 1);
    mbar_init(bar_q_empty, kTypeSplit ? 1 : 2);
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(bar_full(s, 0u), 1);
      mbar_init(bar_full(s, 1u), 1);
      mbar_init(bar_empty(s), kTypeSplit ? 1 : 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar_s_full0 + 8 * t, 1);
      mbar_init(bar_s_free0 + 8 * t, 4 * 32);
      mbar_init(bar_p_full0 + 8 * t, 4 * 32);
      mbar_init(bar_p_free0 + 8 * t, 1);
      mbar_init(bar_o_full0 + 8 * t, 1);
      mbar_init(bar_drain + 8 * t, 1);
      mbar_init(bar_part0 + 8 * t, 4 * 32);
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
  // Sub-tiles with tokens.
  auto live_subtiles = [&](const PagedSegment& s) { return s.token + p.sub_tokens >= s.n ? 1 : kSubTiles; };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kControlRegs));
    if (warp == kLoadWarp) {
      // ---------------------------------------------------------- producer
      // Ring order per segment [b, e): K_b, then for each j: K_{j+1}, V_j —
      // the order the MMA issuers consume and release them.
      if (lane == 0) {
        tma_prefetch_map(&tmQ);
        tma_prefetch_map(&tmK);
        tma_prefetch_map(&tmV);
      }
      const uint64_t keep = l2_policy_evict_last();          // K/V: re-read by every unit of the head
      const uint64_t stream_once = l2_policy_evict_first();  // Q: read once
      const uint32_t q_bytes = static_cast<uint32_t>(p.sub_tokens * p.group * 128 * L::kPanels);
      const uint32_t page_bytes = static_cast<uint32_t>(p.page_rows * 128 * L::kPanels);
      const int in_page = (1 << p.page_shift) - 1;
      int slot = 0;
      uint32_t ring_ph = 0, issued = 0, q_round = 0;
      uint32_t types = 0, kbits = 0, vbits = 0;  // as in fa2_kernel.cuh
      bool ok = true;
      PagedCursor cur = paged_first(p, *start);
      PagedSegment w;
      // This lane's page of tile j: pages of a tile are dealt to the lanes.
      auto position = [&](int j) { return j * kKeys + lane * p.page_rows; };
      auto has_page = [&](int j) { return lane * p.page_rows < kKeys && position(j) < w.keys; };
      auto entry = [&](int j) { return j < w.kv_end && has_page(j) ? paged_entry(p, w.b, position(j)) : -1; };
      auto load_tile = [&](const CUtensorMap* map, int j, int page, uint32_t is_v) -> bool {
        const uint32_t full = bar_full(slot, is_v);
        const uint32_t dst = sRing + static_cast<uint32_t>(slot * L::kTileBytes + lane * p.page_rows * 128);
        const bool mine = has_page(j), there = mine && page_ok(p, page), load = mine && (there || is_v);
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, load)) * page_bytes;
        const int at = position(j) & in_page, from = there ? page : p.pages;
        // every lane waits: each may go on by itself then (a box may land before lane 0
        // has announced it: the phase still lacks that arrival)
        const bool free = wait_bounded(bar_empty(slot), ring_ph ^ 1u, wd, kSiteLoadRingEmpty, true, kNapNs);
        if (!__all_sync(0xffffffffu, free)) return false;
        if (mine && !there && !is_v) {  // no such page: its scores are NaN
          for (int pn = 0; pn < L::kPanels; ++pn)
            for (int r = 0; r < p.page_rows * 8; ++r)
              st_shared_v4(dst + static_cast<uint32_t>(pn * kPanelBytes + r * 16), 0x7fff7fffu, 0x7fff7fffu,
                           0x7fff7fffu, 0x7fff7fffu);
          fence_proxy_async_shared();
        }
        __syncwarp();
        if (!(p.test_withhold && issued == 0)) {  // test hook: the first tile never arrives
          if (lane == 0) mbar_arrive_expect_tx(full, bytes);
          if (load)
            for (int pn = 0; pn < L::kPanels; ++pn)
              tma_load_4d_hint(dst + static_cast<uint32_t>(pn * kPanelBytes), map, full, pn * 64, at, w.head, from, keep);
        }
        types = (types & ~(1u << slot)) | (is_v << slot);
        if (is_v) vbits ^= 1u << slot; else kbits ^= 1u << slot;
        ++issued;
        if (++slot == L::kStages) {
          slot = 0;
          ring_ph ^= 1u;
        }
        return true;
      };
      while (ok && paged_next(cur, w, p)) {
        int now = entry(w.kv_begin), next = entry(w.kv_begin + 1);
        if (q_round > 0) {
          bool free = lane != 0 || wait_bounded(bar_q_empty, (q_round - 1) & 1u, wd, kSiteLoadQEmpty, true, kNapNs);
          ok = __all_sync(0xffffffffu, free);
          if (!ok) break;
        }
        if (lane == 0) {
          const int n_sub = live_subtiles(w);
          mbar_arrive_expect_tx(bar_q_full, n_sub * q_bytes);
          for (int t = 0; t < n_sub; ++t)
            for (int pn = 0; pn < L::kPanels; ++pn)
              tma_load_3d_hint(sQ + t * L::kTileBytes + pn * kPanelBytes, &tmQ, bar_q_full, pn * 64,
                               w.head * p.group, w.t0 + w.token + t * p.sub_tokens, stream_once);
        }
        ++q_round;
        ok = load_tile(&tmK, w.kv_begin, now, 0u);
        for (int j = w.kv_begin; j < w.kv_end && ok; ++j) {
          const int after = entry(j + 2);
          if (j + 1 < w.kv_end) ok = load_tile(&tmK, j + 1, next, 0u);
          if (ok) ok = load_tile(&tmV, j, now, 1u);
          now = next;
          next = after;
        }
      }
      // Drain: every copy issued must have landed before the CTA may exit.
      if (lane == 0) {
        const uint32_t first = issued > static_cast<uint32_t>(L::kStages) ? issued - L::kStages : 0u;
        for (uint32_t i = first; i < issued; ++i) {  // the latest tile of each slot
          const int s = static_cast<int>(i % L::kStages);
          const uint32_t is_v = (types >> s) & 1u;
          const uint32_t par = (((is_v ? vbits : kbits) >> s) & 1u) ^ 1u;
          wait_bounded(bar_full(s, is_v), par, wd, kSiteDrain, false, kNapNs);
        }
        if (q_round > 0) wait_bounded(bar_q_full, (q_round - 1) & 1u, wd, kSiteDrain, false, kNapNs);
      }
      __syncwarp();
    } else if (warp < kMmaWarp + kIssuers) {
      // ------------------------------------------------------ MMA issuers
      if (lane == 0) {
        const int me = warp - kMmaWarp;
        constexpr uint32_t idesc_s = make_idesc_f16(kBf16, kKeys, false);
        constexpr uint32_t idesc_o = make_idesc_f16(kBf16, L::kNpv, true);
        constexpr uint32_t kHi = desc_hi_sw128(1024);
        auto issue_s = [&](int t, int slot) {
          const uint32_t qa = desc_lo_sw128(sQ, 16) + static_cast<uint32_t>((t * L::kTileBytes) >> 4);
          const uint32_t ka = desc_lo_sw128(sRing, 16) + static_cast<uint32_t>(slot * (L::kTileBytes >> 4));
          const uint32_t dt = tmem + static_cast<uint32_t>(t * kKeys);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = static_cast<uint32_t>(((kk >> 2) * kPanelBytes + (kk & 3) * 32) >> 4);
            mma_ss_w(dt, qa + off, kHi, ka + off, kHi, idesc_s, kk > 0 ? 1u : 0u);
          }
        };
        // `tail`: only the tile's first `steps` ones of 16 positions, those with keys
        auto issue_pv = [&](int t, int slot, bool acc, auto tail, [[maybe_unused]] int steps) {
          const uint32_t pa = desc_lo_sw128(sP, 16) + static_cast<uint32_t>((t * L::kPBytes) >> 4);
          const uint32_t va = desc_lo_sw128(sRing, kPanelBytes) + static_cast<uint32_t>(slot * (L::kTileBytes >> 4));
          const uint32_t dt = tmem + L::kColO + static_cast<uint32_t>(t * L::kDp);
          const uint32_t pt = tmem + L::kColP + static_cast<uint32_t>(t * (kKeys / 2));
          auto one = [&](int kk) {
            const uint32_t vb = va + static_cast<uint32_t>((kk * 16 * 128) >> 4);
            const uint32_t acc_kk = (acc || kk > 0) ? 1u : 0u;
            if constexpr (L::kPInTmem) {
              mma_ts_w(dt, pt + 8u * kk, vb, kHi, idesc_o, acc_kk);
            } else {
              const uint32_t po = static_cast<uint32_t>(((kk >> 2) * kPanelBytes + (kk & 3) * 32) >> 4);
              mma_ss_w(dt, pa + po, kHi, vb, kHi, idesc_o, acc_kk);
            }
          };
          if constexpr (tail.value) {
#pragma unroll 1
            for (int kk = 0; kk < steps; ++kk) one(kk);
          } else {
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk) one(kk);
          }
        };
        auto k_index = [](int j, int b) { return j == b ? 0 : 2 * (j - b) - 1; };
        auto v_index = [](int j, int b, int e) { return j == e - 1 ? 2 * (j - b) + 1 : 2 * (j - b) + 2; };
        uint32_t bits[2] = {0u, 0u};  // [type]: parity of the next use of each slot's full barrier
        auto take = [&](uint32_t idx, uint32_t is_v) -> int {
          const int s = static_cast<int>(idx % L::kStages);
          const uint32_t par = (bits[is_v] >> s) & 1u;
          bits[is_v] ^= 1u << s;
          return wait_bounded(bar_full(s, is_v), par, wd, kSiteMmaRingFull, true, kNapNs) ? s : -1;
        };
        // The unit's last tile may be short: its rows behind the keys up to the last
        // product's 16 are zeroed, the products beyond left out.
        auto clean_v = [&](const PagedSegment& u, int j, int slot) -> int {
          const int valid = u.keys - j * kKeys;
          cross_zero_rows(sRing + static_cast<uint32_t>(slot * L::kTileBytes), L::kPanels, valid);
          return cross_key_steps(valid);
        };
        auto full_end = [](const PagedSegment& u, int e) { return e == u.nkv && u.keys < e * kKeys ? e - 1 : e; };
        uint32_t base_idx = 0;  // global load index of the current segment's first tile
        bool ok = true;
        PagedCursor cur = paged_first(p, *start);
        PagedSegment w;
        if constexpr (kTypeSplit) {
          if (me == 0) {
            uint32_t q_round = 0, s_free_ph[2] = {0u, 0u};
            bool s_out[2] = {false, false};  // an S issued whose TMEM the softmax has not released yet
            while (ok && paged_next(cur, w, p)) {
              const int b = w.kv_begin, e = w.kv_end;
              const int n_sub = live_subtiles(w);
              if (!wait_bounded(bar_q_full, q_round & 1u, wd, kSiteMmaQFull, true, kNapNs)) break;
              ++q_round;
              for (int j = b; j < e && ok; ++j) {
                const int slot_k = take(base_idx + k_index(j, b), 0u);
                if (slot_k < 0) { ok = false; break; }
                for (int t = 0; t < n_sub; ++t) {
                  if (s_out[t]) {
                    if (!wait_bounded(bar_s_free0 + 8 * t, s_free_ph[t], wd, kSiteMmaSFree, true, kNapNs)) { ok = false; break; }
                    s_free_ph[t] ^= 1u;
                  }
                  tc_fence_after_sync();
                  issue_s(t, slot_k);
                  mma_commit(bar_s_full0 + 8 * t);
                  s_out[t] = true;
                }
                if (!ok) break;
                mma_commit(bar_empty(slot_k));
                if (j == e - 1) mma_commit(bar_q_empty);
              }
              base_idx += 2u * static_cast<uint32_t>(e - b);
            }
          } else {
            uint32_t p_full_ph[2] = {0u, 0u};
            while (ok && paged_next(cur, w, p)) {
              const int b = w.kv_begin, e = w.kv_end;
              const int n_sub = live_subtiles(w);
              auto tile = [&](int j, auto tail) {
                const int slot_v = take(base_idx + v_index(j, b, e), 1u);
                if (slot_v < 0) { ok = false; return; }
                int steps = kKeys / 16;
                if constexpr (tail.value) steps = clean_v(w, j, slot_v);
                for (int t = 0; t < n_sub; ++t) {
                  if (!wait_bounded(bar_p_full0 + 8 * t, p_full_ph[t], wd, kSiteMmaPFull, true, kNapNs)) { ok = false; return; }
                  p_full_ph[t] ^= 1u;
                  tc_fence_after_sync();
                  issue_pv(t, slot_v, j > b, tail, steps);
                  mma_commit(bar_p_free0 + 8 * t);
                  if (j == e - 1) mma_commit(bar_o_full0 + 8 * t);
                }
                mma_commit(bar_empty(slot_v));
              };
              const int e_full = full_end(w, e);
              for (int j = b; j < e_full && ok; ++j) tile(j, std::false_type{});
              if (e_full < e && ok) tile(e_full, std::true_type{});
              base_idx += 2u * static_cast<uint32_t>(e - b);
            }
          }
        } else {
          // One issuer per sub-tile t = me: S_t one tile ahead of P.V_t, each S as soon as
          // its K tile has landed and the softmax has loaded the sub-tile's S before, each
          // P.V as soon as its V tile has landed and the softmax has published P_t. A
          // sub-tile without tokens: nothing but the slots' release.
          const int t = me;
          uint32_t q_round = 0, s_free_ph = 0, p_full_ph = 0;
          bool s_out = false;
          while (ok && paged_next(cur, w, p)) {
            const int b = w.kv_begin, e = w.kv_end;
            const bool live = t < live_subtiles(w);
            if (!wait_bounded(bar_q_full, q_round & 1u, wd, kSiteMmaQFull, true, kNapNs)) break;
            ++q_round;
            auto next_s = [&](int j) -> bool {
              const int slot_k = take(base_idx + k_index(j, b), 0u);
              if (slot_k < 0) return false;
              if (live) {
                if (s_out) {
                  if (!wait_bounded(bar_s_free0 + 8 * t, s_free_ph, wd, kSiteMmaSFree, true, kNapNs)) return false;
                  s_free_ph ^= 1u;
                }
                tc_fence_after_sync();
                issue_s(t, slot_k);
                mma_commit(bar_s_full0 + 8 * t);
                s_out = true;
              }
              mma_commit(bar_empty(slot_k));
              if (j + 1 == e) mma_commit(bar_q_empty);
              return true;
            };
            auto tile = [&](int j, auto tail) {
              if (j + 1 < e && !next_s(j + 1)) { ok = false; return; }
              const int slot_v = take(base_idx + v_index(j, b, e), 1u);
              if (slot_v < 0) { ok = false; return; }
              if (live) {
                int steps = kKeys / 16;
                if constexpr (tail.value) steps = clean_v(w, j, slot_v);
                if (!wait_bounded(bar_p_full0 + 8 * t, p_full_ph, wd, kSiteMmaPFull, true, kNapNs)) { ok = false; return; }
                p_full_ph ^= 1u;
                tc_fence_after_sync();
                issue_pv(t, slot_v, j > b, tail, steps);
                mma_commit(bar_p_free0 + 8 * t);
                if (j == e - 1) mma_commit(bar_o_full0 + 8 * t);
              }
              mma_commit(bar_empty(slot_v));
            };
            if (!next_s(b)) break;
            const int e_full = full_end(w, e);
            for (int j = b; j < e_full && ok; ++j) tile(j, std::false_type{});
            if (e_full < e && ok) tile(e_full, std::true_type{});
            base_idx += 2u * static_cast<uint32_t>(e - b);
          }
        }
        // Drain: all issued tensor-core work completes before TMEM is released.
        mma_commit(bar_drain + 8 * me);
        wait_bounded(bar_drain + 8 * me, 0u, wd, kSiteDrain, false, kNapNs);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ------------------------------------------------- softmax warpgroups
    const int t = warp >> 2;                 // sub-tile
    const int wr = warp & 3;
    const int rr = wr * 32 + lane;           // row within the sub-tile
    const uint32_t lane_off = static_cast<uint32_t>(wr * 32) << 16;
    const uint32_t tS = tmem + lane_off + static_cast<uint32_t>(t * kKeys);
    const uint32_t tO = tmem + lane_off + L::kColO + static_cast<uint32_t>(t * L::kDp);
    const uint32_t tP = tmem + lane_off + L::kColP + static_cast<uint32_t>(t * (kKeys / 2));
    const uint32_t bar_s = bar_s_full0 + 8 * t, bar_sf = bar_s_free0 + 8 * t, bar_p = bar_p_full0 + 8 * t;
    const uint32_t bar_pf = bar_p_free0 + 8 * t, bar_o = bar_o_full0 + 8 * t, bar_part = bar_part0 + 8 * t;
    // this thread's row in shared memory: 128 bytes per 64 keys (or columns of O), 16-byte chunks
    // placed by the 128-byte swizzle (chunk c of row r at c ^ (r % 8))
    const uint32_t p_tile = sP + static_cast<uint32_t>(t * L::kPBytes);
    const uint32_t p_row = p_tile + static_cast<uint32_t>(rr * 128);
    const uint32_t p_xor = static_cast<uint32_t>(rr & 7);
    const float c = p.scale_log2;
    const int row_token = rr / p.group, row_head = rr - row_token * p.group;
    uint32_t s_phase = 0, o_phase = 0, part_phase = 0;
    uint32_t p_count = 0;  // P tiles published so far
    bool ok = true;
    // By a warpgroup of each of the `parts` CTAs that hold a unit: every parts-th 8 or 16
    // rows of its sub-tile, from all partial results (the first holder alone, one partial
    // result after another: 23 us for 19 of them). The rows' statistics are read at once,
    // then 4 rows of two columns per thread from eight holders at a time.
    auto join_rows = [&](const PagedSegment& u, int parts, auto per) {
      constexpr int kPer = per.value;
      auto meet = [&]() {  // of the warpgroup's threads
        mbar_arrive(bar_part);
        bool met = wait_bounded(bar_part, part_phase, wd, kSitePartialFlag);
        part_phase ^= 1u;
        return __all_sync(0xffffffffu, met) != 0;
      };
      const int first = blockIdx.x - start->part;
      unsigned long long* const flags = p.ws_spread + (static_cast<size_t>(t) * gridDim.x + blockIdx.x) * kPagedMostParts;
      bool fine = lane >= parts || wait_flag(flags + lane, p.epoch, wd, kSitePartialFlag);
      fine = __all_sync(0xffffffffu, fine);
      if (!fine) return;
      __syncwarp();  // what one lane acquired is visible to all
      // seen by every thread of the warpgroup: taken back, so that a replay of a captured
      // launch, which carries the same tag, does not find them
      if (!meet()) return;
      if (rr < parts) flags[rr] = 0ull;
      // in the P buffer, which is free: [part][row] bases, l, l_o, weights, then base, l, l_o of the rows
      constexpr int kAll = kPagedMostParts * kPer;
      float* const sm = reinterpret_cast<float*>(smem + L::kPOffset + t * L::kPBytes);
      float* const total = sm + 4 * kAll;
      const int token0 = u.token + t * p.sub_tokens, rows = min(p.sub_tokens, u.n - token0) * p.group;
      const float* const po = p.ws_o + (static_cast<size_t>(first) * 2 + t) * D * 128;
      const float* const ps = p.ws_stats + (static_cast<size_t>(first) * 2 + t) * 3 * 128;
      for (int row0 = kPer * start->part; row0 < rows; row0 += kPer * parts) {
        const int row = rr % kPer;
        for (int j = rr / kPer; j < parts; j += 128 / kPer) {
          const float* const from = ps + static_cast<size_t>(j) * 2 * 3 * 128 + row0 + row;
          const float a = __ldcg(from), b = __ldcg(from + 128), d = __ldcg(from + 256);
          sm[j * kPer + row] = a;
          sm[kAll + j * kPer + row] = b;
          sm[2 * kAll + j * kPer + row] = d;
        }
        if (!meet()) return;
        float top = -CUDART_INF_F;
        for (int j = 0; j < parts; ++j) top = fmaxf(top, sm[j * kPer + row]);
        auto weight = [&](int j) {
          const float b = sm[j * kPer + row];
          return b == -CUDART_INF_F ? 0.f : ex2_approx(b - top);
        };
        for (int j = rr / kPer; j < parts; j += 128 / kPer) sm[3 * kAll + j * kPer + row] = weight(j);
        if (rr < kPer) {
          float l = 0.f, l_o = 0.f;
          for (int j = 0; j < parts; ++j) {
            const float e = weight(j);
            l = fmaf(e, sm[kAll + j * kPer + row], l);
            l_o = fmaf(e, sm[2 * kAll + j * kPer + row], l_o);
          }
          total[row] = top;
          total[kPer + row] = l;
          total[2 * kPer + row] = l_o;
        }
        if (!meet()) return;
        const int q = 4 * (rr % (kPer / 4));
        // two columns at a time, eight holders' loads of both under way
        constexpr int kStep = 512 / kPer;
        for (int col = rr / (kPer / 4); col < D; col += 2 * kStep) {
          float acc[2][4] = {};
          const bool two = col + kStep < D;
          const float* const from = po + static_cast<size_t>(col) * 128 + row0 + q;
#pragma unroll 1
          for (int j0 = 0; j0 < parts; j0 += 8) {
            float4 x[2][8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float* const at = from + static_cast<size_t>(j0 + k) * 2 * D * 128;
              x[0][k] = x[1][k] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (j0 + k < parts) x[0][k] = __ldcg(reinterpret_cast<const float4*>(at));
              if (j0 + k < parts && two) x[1][k] = __ldcg(reinterpret_cast<const float4*>(at + kStep * 128));
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              if (j0 + k >= parts) break;
              const float4 e = *reinterpret_cast<const float4*>(sm + 3 * kAll + (j0 + k) * kPer + q);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                acc[h][0] = fmaf(e.x, x[h][k].x, acc[h][0]);
                acc[h][1] = fmaf(e.y, x[h][k].y, acc[h][1]);
                acc[h][2] = fmaf(e.z, x[h][k].z, acc[h][2]);
                acc[h][3] = fmaf(e.w, x[h][k].w, acc[h][3]);
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = row0 + q + i;
            if (at >= rows) break;
            const float l = total[kPer + q + i];
            const float inv = l > 0.f ? __frcp_rn(total[2 * kPer + q + i]) : 0.f;
            const int tok = at / p.group;
            const long long to = (static_cast<long long>(u.t0 + token0 + tok) * p.heads + u.head) * p.group + (at - tok * p.group);
            uint16_t* const o = static_cast<uint16_t*>(p.o) + to * D + col;
            *o = static_cast<uint16_t>(pack2(acc[0][i] * inv, 0.f, kBf16) & 0xffffu);
            if (two) o[kStep] = static_cast<uint16_t>(pack2(acc[1][i] * inv, 0.f, kBf16) & 0xffffu);
            if (col == 0) p.lse[to] = l != 0.f ? (total[q + i] + __log2f(l)) * 0.69314718055994530942f : CUDART_INF_F;
          }
        }
        if (row0 + kPer * parts < rows && !meet()) return;  // read before the next rows' are written there
      }
    };
    PagedCursor cur = paged_first(p, *start);
    PagedSegment w;
    while (ok && paged_next(cur, w, p)) {
      if (t >= live_subtiles(w)) continue;
      const int token = w.token + t * p.sub_tokens + row_token;
      const bool live = row_token < p.sub_tokens && token < w.n;
      // this row's keys: [0, limit). A row without a token is anything and not written: it is
      // not masked, so that it does not send its warp through the masks of every tile.
      int limit = INT_MAX;
      if (live) limit = p.causal ? min(max(w.length - w.n + token + 1, 0), w.length) : w.length;
      float m_raw = -CUDART_INF_F;  // running max of the raw scores seen so far
      float base2 = -CUDART_INF_F;  // exponent base (log2 units) that l and O are relative to
      float l = 0.f, l_o = 0.f;     // sum of p; normaliser of O (see fa2_kernel.cuh)
      for (int j = w.kv_begin; j < w.kv_end; ++j) {
        bool got = wait_bounded(bar_s, s_phase, wd, kSiteSoftmaxSFull);
        got = __all_sync(0xffffffffu, got);
        if (!got) { ok = false; break; }
        s_phase ^= 1u;
        tc_fence_after_sync();
        uint32_t sr[128];
        tmem_ld32x128_wait(tS, sr);
        tc_fence_before_sync();
        mbar_arrive(bar_sf);  // S is in registers: the next scores may be computed
        float s[128];
#pragma unroll
        for (int i = 0; i < 128; ++i) s[i] = __uint_as_float(sr[i]);
        const int kv0 = j * kKeys;
        if (kv0 + kKeys > limit) {
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (kv0 + i >= limit) s[i] = -CUDART_INF_F;
        }
        float mx[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          mx[q] = fmax3(s[32 * q], s[32 * q + 1], s[32 * q + 2]);
#pragma unroll
          for (int i = 3; i < 31; i += 2) mx[q] = fmax3(mx[q], s[32 * q + i], s[32 * q + i + 1]);
          mx[q] = fmaxf(mx[q], s[32 * q + 31]);
        }
        const float m_tile = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]);
        m_raw = fmaxf(m_raw, m_tile);
        // the base moves only when the max has passed it by 2^kRescaleLog2 (or on the first key)
        const float cand = m_raw * c;
        float alpha = 1.f;
        if (live && m_raw != -CUDART_INF_F && (base2 == -CUDART_INF_F || cand - base2 > kRescaleLog2)) {
          alpha = ex2_approx(base2 - cand);
          base2 = cand;
        }
        const float nb = (base2 == -CUDART_INF_F) ? 0.f : -base2;
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        uint32_t pk[64];
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          float x0, x1;
          ffma2_bcast(x0, x1, s[2 * i], s[2 * i + 1], c, nb);
          const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
          fadd2_acc(acc[2 * (i & 3)], acc[2 * (i & 3) + 1], p0, p1);
          pk[i] = pack2(p0, p1, kBf16);
        }
        // the previous P.V is complete before its P is overwritten and O rescaled
        if (p_count > 0) {
          bool fr = wait_bounded(bar_pf, (p_count - 1) & 1u, wd, kSiteSoftmaxPFree);
          fr = __all_sync(0xffffffffu, fr);
          if (!fr) { ok = false; break; }
          tc_fence_after_sync();
        }
        if constexpr (L::kPInTmem) {
          tmem_st32x32(tP, *reinterpret_cast<const uint32_t(*)[32]>(pk));
          tmem_st32x32(tP + 32, *reinterpret_cast<const uint32_t(*)[32]>(pk + 32));
        } else {
#pragma unroll
          for (int ch = 0; ch < 16; ++ch) {
            const uint32_t addr = p_row + static_cast<uint32_t>((ch >> 3) * kPanelBytes) +
                                  ((static_cast<uint32_t>(ch & 7) ^ p_xor) << 4);
            st_shared_v4(addr, pk[4 * ch], pk[4 * ch + 1], pk[4 * ch + 2], pk[4 * ch + 3]);
          }
        }
        if (j > w.kv_begin && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
          for (int cc = 0; cc < D; cc += 32) {
            uint32_t o[32];
            tmem_ld32x32_wait(tO + cc, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st32x32(tO + cc, o);
          }
        }
        tmem_wait_st();
        if constexpr (!L::kPInTmem) fence_proxy_async_shared();
        tc_fence_before_sync();
        mbar_arrive(bar_p);
        ++p_count;
        const float lt = ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
        // the largest weight enters O's normaliser as it is rounded (fa2_kernel.cuh)
        float x0, x1;
        ffma2_bcast(x0, x1, m_tile, m_tile, c, nb);
        const float px = ex2_approx(x0), pxr = round16(px, kBf16);
        l = l * alpha + lt;
        l_o = l_o * alpha + (lt + (pxr - px));
      }
      if (!ok) break;
      // -------------------------------------------------------- epilogue
      bool got = wait_bounded(bar_o, o_phase, wd, kSiteSoftmaxOFull);
      got = __all_sync(0xffffffffu, got);
      if (!got) break;
      o_phase ^= 1u;
      tc_fence_after_sync();
      const int spread = start->parts >= kPagedSpreadParts ? start->parts : 0;
      if (w.kv_begin > 0 || spread) {
        // Not the unit's first tiles: the unnormalised partial (O, base, l, l_o) to the owner,
        // or to all that the unit is cut between.
        const size_t slot = static_cast<size_t>(blockIdx.x) * 2 + t;
        float* po = p.ws_o + slot * D * 128;
        float* ps = p.ws_stats + slot * 3 * 128;
#pragma unroll 1
        for (int cc = 0; cc < D; cc += 32) {
          uint32_t o[32];
          tmem_ld32x32_wait(tO + cc, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) __stcg(po + (cc + i) * 128 + rr, __uint_as_float(o[i]));
        }
        __stcg(ps + rr, base2);
        __stcg(ps + 128 + rr, l);
        __stcg(ps + 256 + rr, l_o);
        __threadfence();
        mbar_arrive(bar_part);
        if (rr < 32) {
          bool done = wait_bounded(bar_part, part_phase, wd, kSitePartialWrite);
          done = __all_sync(0xffffffffu, done);
          if (!done) break;
          if (spread) {
            if (lane < spread)
              store_release(p.ws_spread + (static_cast<size_t>(t) * gridDim.x + blockIdx.x - start->part + lane) * kPagedMostParts + start->part,
                            p.epoch);
          } else if (rr == 0) {
            store_release(p.ws_flags + slot, p.epoch);
          }
        }
        part_phase ^= 1u;
        tc_fence_before_sync();
        if (spread) {
          if (spread >= 16) join_rows(w, spread, std::integral_constant<int, 8>{});
          else join_rows(w, spread, std::integral_constant<int, 16>{});
          break;  // the share's only segment
        }
        continue;
      }
      // Owner (or whole unit): fold in the partials of the CTAs that took the rest of it, if any.
      float a_own = 1.f, nbase = base2;
      int first_c = blockIdx.x + 1, last_c = blockIdx.x;  // partial holders [first_c, last_c]
      if (w.kv_end < w.nkv) {
        if (start->parts) last_c += start->parts - 1 - start->part;
        else
          while (last_c + 1 < start->shares && paged_share_begin(*start, last_c + 1) < w.unit_end) ++last_c;
        bool fine = true;
        for (int cb = first_c + (rr & 31); cb <= last_c && fine; cb += 32)
          fine = wait_flag(p.ws_flags + static_cast<size_t>(cb) * 2 + t, p.epoch, wd, kSitePartialFlag);
        fine = __all_sync(0xffffffffu, fine);
        if (!fine) break;
        __syncwarp();  // what one lane acquired is visible to all
        // every thread of the warpgroup has seen the flags: taken back, so that a
        // replay of a captured launch, which carries the same tag, does not find them
        mbar_arrive(bar_part);
        if (rr < 32) {
          bool seen = wait_bounded(bar_part, part_phase, wd, kSitePartialFlag);
          seen = __all_sync(0xffffffffu, seen);
          if (!seen) break;
          for (int cb = first_c + rr; cb <= last_c; cb += 32) p.ws_flags[static_cast<size_t>(cb) * 2 + t] = 0ull;
        }
        part_phase ^= 1u;
        // their statistics, eight holders' loads under way at once (one holder after
        // another: 25 us for 18 of them); 0 for a partial that saw no key
#pragma unroll 1
        for (int c0 = first_c; c0 <= last_c; c0 += 8) {
          float bs[8], ls[8], los[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float* ps = p.ws_stats + (static_cast<size_t>(min(c0 + i, last_c)) * 2 + t) * 3 * 128 + rr;
            bs[i] = __ldcg(ps);
            ls[i] = __ldcg(ps + 128);
            los[i] = __ldcg(ps + 256);
          }
          float top = nbase;
#pragma unroll
          for (int i = 0; i < 8; ++i) top = fmaxf(top, bs[i]);
          const float scale = nbase == -CUDART_INF_F ? 0.f : ex2_approx(nbase - top);
          a_own *= base2 == -CUDART_INF_F ? 0.f : scale;
          l *= scale;
          l_o *= scale;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float a = bs[i] == -CUDART_INF_F ? 0.f : ex2_approx(bs[i] - top);
            if (c0 + i <= last_c) {
              l = fmaf(a, ls[i], l);
              l_o = fmaf(a, los[i], l_o);
            }
          }
          nbase = top;
        }
        base2 = nbase;
      }
      const float inv = l > 0.f ? __frcp_rn(l_o) : 0.f;
      // 32 columns of the finished rows into the staged tile
      auto stage = [&](int cc, const float (&of)[32]) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t pk[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) pk[i] = pack2(of[8 * q + 2 * i] * inv, of[8 * q + 2 * i + 1] * inv, kBf16);
          const int c8 = cc / 8 + q;
          st_shared_v4(p_row + static_cast<uint32_t>((c8 >> 3) * kPanelBytes) + ((static_cast<uint32_t>(c8 & 7) ^ p_xor) << 4),
                       pk[0], pk[1], pk[2], pk[3]);
        }
      };
      if (last_c < first_c) {
        if constexpr (D == 128) {
          uint32_t o[128];
          tmem_ld32x128_wait(tO, o);
#pragma unroll
          for (int cc = 0; cc < D; cc += 32) stage(cc, *reinterpret_cast<const float(*)[32]>(o + cc));
        } else {
#pragma unroll
          for (int cc = 0; cc < D; cc += 32) {
            uint32_t o[32];
            tmem_ld32x32_wait(tO + cc, o);
            stage(cc, *reinterpret_cast<const float(*)[32]>(o));
          }
        }
      } else {
        // Partial results, 32 columns of one at a time, the next ones under way meanwhile
        // (each waited for by itself: 8 us for one partial result at D = 128).
        float part[32], part_base;
        auto fetch = [&](int cc, int cb) {
          const float* po = p.ws_o + ((static_cast<size_t>(cb) * 2 + t) * D + cc) * 128 + rr;
          part_base = __ldcg(p.ws_stats + (static_cast<size_t>(cb) * 2 + t) * 3 * 128 + rr);
#pragma unroll
          for (int i = 0; i < 32; ++i) part[i] = __ldcg(po + i * 128);
        };
        fetch(0, first_c);
#pragma unroll 1
        for (int cc = 0; cc < D; cc += 32) {
          uint32_t o[32];
          tmem_ld32x32_wait(tO + cc, o);
          float of[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) of[i] = __uint_as_float(o[i]) * a_own;
#pragma unroll 1
          for (int cb = first_c; cb <= last_c; ++cb) {
            const float a = part_base == -CUDART_INF_F ? 0.f : ex2_approx(part_base - nbase);
            float now[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) now[i] = part[i];
            const bool more = cb < last_c;
            if (more || cc + 32 < D) fetch(more ? cc : cc + 32, more ? cb + 1 : first_c);
#pragma unroll
            for (int i = 0; i < 32; ++i) of[i] = fmaf(a, now[i], of[i]);
          }
          stage(cc, of);
        }
      }
      // O_t is read out; the next segment's first P.V may overwrite it once this
      // warpgroup publishes that segment's first P (ordered by bar_p).
      tc_fence_before_sync();
      const long long out_row =
          live ? (static_cast<long long>(w.t0 + token) * p.heads + w.head) * p.group + row_head : -1ll;
      // whole rows at a time: 16-byte chunks of a row by neighbouring lanes
      __syncwarp();
      constexpr int kChunks = D / 8;
#pragma unroll 4
      for (int i = 0; i < kChunks; ++i) {
        const int at = i * 32 + lane, r = at / kChunks, ch = at - r * kChunks;
        const long long to = __shfl_sync(0xffffffffu, out_row, r);
        const uint8_t* from = smem + L::kPOffset + t * L::kPBytes + (ch >> 3) * kPanelBytes + (wr * 32 + r) * 128 +
                              (((ch & 7) ^ (r & 7)) << 4);
        if (to >= 0) reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + to * D)[ch] = *reinterpret_cast<const uint4*>(from);
      }
      __syncwarp();  // read before the next segment's P is written there
      if (live) p.lse[out_row] = l != 0.f ? (base2 + __log2f(l)) * 0.69314718055994530942f : CUDART_INF_F;  // NaN stays
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
cudaError_t launch_paged_tiles(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                               const PagedTileParams& p, int grid, cudaStream_t stream) {
  auto kern = fa2_paged_kernel<D, kBf16>;
  constexpr int smem = PagedLayout<D>::kSmemBytes;
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
  // the holder of a cut unit waits for other CTAs: all are resident, or the launch fails
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, q, k, v, p);
}

}  // namespace fa2
