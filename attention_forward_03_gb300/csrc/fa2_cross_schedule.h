// How cross attention deals its work units to the SMs: host arithmetic alone
// (no CUDA in it, so that it can be checked without a device).
#pragma once

namespace fa2 {

// What cutting units costs, in steps of the busiest SM: cutting them at all
// (the flags, the way through memory), every result that a unit's first holder
// joins to its own, and shares that do not end where units do (then a CTA
// works on parts of two units).
struct CutCosts {
  double cut, join, uneven;
};

// Fewer units than SMs: how many CTAs share their steps equally, or 0 for
// whole units. The first holder of a unit joins the other holders' results one
// after another, so more CTAs are not always faster. Tried are whole parts per
// unit and all SMs. With key counts on the device (`lengths`) the longest unit
// is taken to have `unit_steps` steps and the mean 0.6 of them, as with evenly
// spread counts; shares then end where they may, and every second one in a
// unit of its own.
inline int cross_cut_ctas(long long units, long long unit_steps, bool lengths, int sms, const CutCosts& c) {
  double best = 0.95 * static_cast<double>(unit_steps);
  int ctas = 0;
  const auto consider = [&](long long n, long long joins, double uneven) {
    const double share = lengths ? 0.6 * static_cast<double>(units * unit_steps) / static_cast<double>(n)
                                 : static_cast<double>((units * unit_steps + n - 1) / n);
    const double cost = share + c.cut + c.join * static_cast<double>(joins) + uneven;
    if (cost < best) {
      best = cost;
      ctas = static_cast<int>(n);
    }
  };
  for (long long parts = 2; parts <= unit_steps && parts * units <= sms; ++parts)
    consider(parts * units, lengths ? parts : parts - 1, lengths ? 0.5 * c.uneven : 0.0);
  if (units * unit_steps > sms) consider(sms, (sms + units - 1) / units, lengths ? 0.5 * c.uneven : c.uneven);
  return ctas;
}

// Whether a unit's two sub-tiles take its key tiles in turn (fa2_kernel.cuh):
// with at most 128 rows per key head there is no second sub-tile of rows, and
// from 5 key tiles on the overlap is worth the joining of the two (us, with /
// without, 1024 such heads, D = 64: 300 keys 46.4 / 42.5, 512 keys 43.1 /
// 43.9, 768 keys 54.0 / 59.0, 4096 keys 177 / 238; 8 heads, in the best number
// of parts, 4068 keys 16.3 / 18.3). Above D = 64 the tensor cores have more to
// do and the gain is below a tenth (1 head per SM, 16384 keys, D = 128: 114 /
// 131; 256 heads of 4096 keys 91.5 / 94.7), the loss at 257 keys as large.
inline bool split_keys(int D, long long rows, long long nkv) { return D <= 64 && rows <= 128 && nkv > 4; }

// How many CTAs share the K/V-tile steps equally, with a merge of the units
// that they cut, or 0 for whole units in rounds.
//
// At least one unit per SM: equal shares when that saves the busiest SM 5 %
// with what the cuts cost, in steps 5, 7 above D = 64, 12 with split keys.
// With key counts on the device the host cannot know the units; then from as
// many tiles on as measured to pay on evenly spread counts (us, whole / equal;
// 192 and 1024 units): D = 64, 256 rows: 4 tiles 17.8 / 18.8 and 53.2 / 58.6, 6
// tiles 22.3 / 21.1 and 67.0 / 65.8, 32 tiles 63.3 / 44.1 and 211 / 167; D =
// 128, 128 rows: 8 tiles 23.9 / 24.0 and 76.0 / 86.7, 12 tiles 31.8 / 28.0 and
// 100 / 99.2; split keys: 16 tiles 26.8 / 27.2 and 77.8 / 104, 32 tiles 42.3 /
// 38.5 and 130 / 143.
//
// Fewer: cross_cut_ctas, in steps of about 1 us, 0.65 us with split keys.
// Measured (us, by the parts per unit; 1: not cut, * the choice), 128 rows: D =
// 64, 8 heads: 500 keys 1* 9.4, 2 11.4; 1000 keys 1* 11.4, 2 12.5, 4 12.8; 1508
// keys 1 13.9, 2 13.7, 3* 14.5, 4 13.3, 12 20.9; 2000 keys 1 16.4, 4* 13.9, 5
// 14.2; 4068 keys 1 27.0, 4* 16.9, 5 16.4, 8 18.2, 19 26.0; 16,356 keys 1 89.8, 8
// 26.3, 10* 26.6, 19 29.3; 32 heads of 16,356 keys 4* 35.6, all SMs 40.0; 96
// heads of 256 rows over up to 4096 keys 1 44.5, all SMs* 30.2. D = 128, 8
// heads: 500 keys 1* 10.9, 2 13.5; 1000 keys 1* 14.5, 4 15.8; 1508 keys 1* 18.6,
// 2 17.4, 4 16.7, 12 29.8; 2000 keys 1 22.2, 4* 17.5, 5 18.5; 4068 keys 1 37.7, 4*
// 21.3, 8 24.8, 19 36.8; 16,356 keys 1 129, 8 38.3, 10* 40.2, 16 38.9. Around 12
// tiles the costs miss the best by a tenth, at D = 64 on the cut side and at D =
// 128 on the other.
inline int cross_share_ctas(int D, bool split, long long units, long long nkv, bool lengths, int sms) {
  if (units < sms) {
    const CutCosts c = split ? CutCosts{4.6, 1.3, 12.0} : D <= 64 ? CutCosts{5.8, 0.6, 3.0} : CutCosts{5.0, 1.25, 4.0};
    return cross_cut_ctas(units, nkv, lengths, sms, c);
  }
  const double per_sm = static_cast<double>(units) / sms;
  if (lengths) return static_cast<double>(nkv) >= (split ? 16.0 + 5.0 * per_sm : D <= 64 ? 6.0 : 12.0) ? sms : 0;
  const double rounds = static_cast<double>((units + sms - 1) / sms) * static_cast<double>(nkv);
  const double balanced = per_sm * static_cast<double>(nkv) + (split ? 12.0 : D <= 64 ? 5.0 : 7.0);
  return balanced < 0.95 * rounds ? sms : 0;
}

// How many CTAs share all query steps equally, with a merge of the units that
// they cut, or 0 for whole units in rounds.
//
// At least one unit per SM: when that saves the busiest SM at least 5 %, with
// 2 steps for a cut unit's partial results. With key counts on the device and
// more than one key tile per head always, as the shares follow the counts (us,
// equal shares / whole units: 64 heads of 1024 rows over up to 1500 keys, D =
// 64 73.5 / 98.8, D = 128 115 / 156; 64 rows 28.7 / 35.6; but 1024 heads over
// up to 100 keys, one tile each, 256 rows 75.4 / 68.4). In rounds the key
// tiles of a head run at the same time and share its Q, dO and dQ; where those
// are more than the L2 cache holds, equal shares have to save a quarter (256
// heads of 2048 rows x 257 keys, D = 128: 545 us equal, 418 whole; D = 64 266
// and 250).
//
// Fewer: cross_cut_ctas. Measured (us, by the parts per unit; 1: not cut, *
// the choice): 8 heads over 77 keys, D = 64: 256 rows 1* 10.7, 2 12.7; 1024
// rows 1 21.3, 4* 16.3, 12 18.7; 4096 rows 1 62.5, 8* 24.5, 19 26.9; 16,384
// rows 1 231, 8 51.7, 16* 41.8, 19 42.8. D = 128: 256 rows 1* 14.8, 4 18.9;
// 1024 rows 1 29.8, 4* 22.7, 12 33.3; 4096 rows 1 93.3, 6 38.1, 8* 37.6, 19
// 43.4; 16,384 rows 1 348, 12 74.7, 16* 63.2, 19 70.1.
inline int cross_bwd_share_ctas(int D, long long units, long long nq, bool lengths, long long q_bytes, int sms) {
  if (units >= sms) {
    constexpr long long kSplitCostSteps = 2;
    const long long rounds = (units + sms - 1) / sms * nq;
    constexpr long long kL2Bytes = 128ll << 20;
    const int most = q_bytes > kL2Bytes ? 75 : 95;  // percent of the rounds
    return lengths || 100 * ((units * nq + sms - 1) / sms + kSplitCostSteps) < most * rounds ? sms : 0;
  }
  return cross_cut_ctas(units, nq, lengths, sms, D <= 64 ? CutCosts{1.5, 0.6, 2.0} : CutCosts{2.3, 1.0, 10.0});
}

}  // namespace fa2
