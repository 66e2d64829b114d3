// ss_ffn_plan.h -- which kernels a problem of the feed-forward block gets: the
// family of each product, the tile, the cluster. Plain C++, so that it can be
// looked at over all sizes without a GPU.
//
// A product is N rows of output (tokens, or rows of a weight gradient) by M
// columns, K = 64 kb. The two families' times are estimated in microseconds
// with constants fitted on one GB300 to 110 problem sizes (T 65 to 16000, D 64
// to 4096, F 64 to 12288), every product in every form. At the fit, what the
// estimates picked took 2.4% longer than the best form on average; the low bits
// of G and U and the tiles of 192 columns came after it, and fp32 or accumulated
// weight gradients were not in it.
#pragma once

#include <stdint.h>

#include <algorithm>

#ifdef __CUDACC__
#define SS_PLAN_FN __host__ __device__ __forceinline__
#else
#define SS_PLAN_FN inline
#endif

namespace ss {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
// 256 x 256 tiles
inline int64_t pair_units(int64_t rows, int64_t cols) { return cdiv(rows, 256) * cdiv(cols, 256); }

// ------------------------------------------------------------- CTA pairs

// A CTA pair's time per k-block of a tile of 256 columns; launch, first loads,
// the last tile's epilogue and the exit together.
constexpr float kPairUsPerKb = 0.35f, kPairUsFixed = 5.7f;
// out_us: what the outputs of the epilogue cost beyond one bf16 value (gate/up
// and dA: two to four values read or written for each sum).
inline float pair_us(int64_t units, int64_t kb, float out_us, int num_sms) {
  const int64_t pairs = num_sms / 2, waves = (units + pairs - 1) / pairs;
  return kPairUsFixed + out_us + kPairUsPerKb * static_cast<float>(waves * kb);
}

// gate/up and dA also have tiles of 192 columns, for sizes whose last round of
// pairs they fill better: a k-block of theirs takes 0.87 of the time for 0.75 of
// the products. Gate/up and down of T 1003, D 1096, F 2952: 33.8 us against 35.8
// (2 rounds either way); backward of T 3001, D 1352, F 3640: 167.7 against 170.4.
// cols: of the product (gate/up: both matrices).
struct PairPlan {
  int bn;
  float us;
};
inline PairPlan pair_plan(int64_t rows, int64_t cols, int64_t kb, float out_us, int num_sms) {
  auto at = [&](int bn, float cost) {
    const int64_t units = cdiv(rows, 256) * cdiv(cols, bn);
    return PairPlan{bn, kPairUsFixed + cost * (pair_us(units, kb, out_us, num_sms) - kPairUsFixed)};
  };
  const PairPlan whole = at(256, 1.f), narrow = at(192, 0.87f);
  return narrow.us < whole.us ? narrow : whole;
}

// ------------------------------------- dX and the three dW in one launch
//
// Units of two lengths, each handed to the pair that is free first (the lowest
// of several), the longer ones first: units that run at the same time are
// neighbours, which share operands in L2, and the pairs finish within about one
// short unit of each other. Walked round-robin instead, T 8192, D 2048, F 5504
// loses 7%, and the backward of T 512, D 4096, F 12288 (2304 units of 8 k-blocks,
// 32 of 384) takes 273 us for 228.
// That order has a closed form, so neither a list nor a limit on the units is
// needed:
//   1. the long units in turn to all pairs; the first `ahead` = n_long % pairs
//      pairs have one more than the others;
//   2. while those are busy with it, `rounds` = ceil(kb_long / kb_short) short
//      units to each of the others, in turn;
//   3. the remaining short units in turn to all pairs.
struct UnitDeal {
  int n_long, n_short;
  int first_long, first_short;  // indices of the first unit of each
  int rounds;
};
// units 0 .. n_a - 1 of kb_a k-blocks and the n_b after them of kb_b
inline UnitDeal deal_units(int n_a, int64_t kb_a, int n_b, int64_t kb_b) {
  return kb_a >= kb_b ? UnitDeal{n_a, n_b, 0, n_a, static_cast<int>(cdiv(kb_a, kb_b))}
                      : UnitDeal{n_b, n_a, n_a, 0, static_cast<int>(cdiv(kb_b, kb_a))};
}

// What one pair runs: three runs of units (the steps above), each evenly spaced.
struct PairShare {
  int n1, n2, n3;
  int at1, at2, at3;
  int step2, pairs;
  SS_PLAN_FN int count() const { return n1 + n2 + n3; }
  SS_PLAN_FN int unit(int k) const {  // the k-th
    if (k < n1) return at1 + k * pairs;
    if (k < n1 + n2) return at2 + (k - n1) * step2;
    return at3 + (k - n1 - n2) * pairs;
  }
};
// of n things in turn to `among`, how many number `me` gets
SS_PLAN_FN int turns(int n, int me, int among) { return n > me ? (n - me + among - 1) / among : 0; }
SS_PLAN_FN PairShare share_of(const UnitDeal& d, int pair, int pairs) {
  const int ahead = d.n_long % pairs, others = ahead ? pairs - ahead : 0;
  const int64_t most = static_cast<int64_t>(d.rounds) * others;
  const int early = most < d.n_short ? static_cast<int>(most) : d.n_short;
  PairShare s;
  s.pairs = pairs;
  s.n1 = turns(d.n_long, pair, pairs);
  s.at1 = d.first_long + pair;
  s.n2 = others && pair >= ahead ? turns(early, pair - ahead, others) : 0;
  s.at2 = d.first_short + pair - ahead;
  s.step2 = others;
  s.n3 = turns(d.n_short - early, pair, pairs);
  s.at3 = d.first_short + early + pair;
  return s;
}
// k-blocks of the busiest pair
inline int64_t busiest_pair(const UnitDeal& d, int64_t kb_long, int64_t kb_short, int pairs) {
  int64_t most = 0;
  for (int p = 0; p < pairs; ++p) {
    const PairShare s = share_of(d, p, pairs);
    most = std::max(most, s.n1 * kb_long + (s.n2 + s.n3) * kb_short);
  }
  return most;
}

// ------------------------------------------- single CTAs, K over a cluster

constexpr int kSplitMaxCluster = 8;

struct SplitPlan {
  int bn, cluster;
  float us;
};

// 128 x bn tiles (m_tile = 64 features of two matrices for gate/up), bn the
// narrowest that takes all tokens, up to 64, or 128; K over up to 8 CTAs.
// A CTA alone on its SM takes 0.28 to 0.59 us a k-block (16 to 128 tokens, the
// rate at which one CTA takes operands in); two on an SM share that rate and
// hide each other's gaps, so that they hardly slow one another; a third waits
// for a place. A cluster's join costs a barrier; the outputs' cost goes with the
// tokens of a tile.
inline SplitPlan split_plan(int64_t n, int64_t m, int m_tile, int64_t kb, float out_us,
                            bool wide_only, int num_sms) {
  constexpr float kFixed = 2.2f, kJoin = 0.1f, kTile = 1.15f;
  SplitPlan best{0, 0, 0.f};
  for (int bn = wide_only ? 128 : 16; bn <= 128; bn *= 2) {
    if (bn < 64 && n > bn) continue;  // narrower tiles only re-read the weights
    const float per_kb = bn == 16 ? 0.28f : bn == 32 ? 0.3f : bn == 64 ? 0.364f : 0.59f;
    const int64_t tiles = cdiv(n, bn) * cdiv(m, m_tile);
    for (int S = 1; S <= kSplitMaxCluster && (S == 1 || kb / S >= 2); S *= 2) {
      const float share = static_cast<float>(tiles * S) / num_sms;
      const float load = share <= 1.f ? 1.f : share <= 2.f ? 1.f + 0.18f * (share - 1.f) : 1.09f * share;
      const float us = kFixed + (S > 1 ? kJoin : 0.f) +
                       load * (per_kb * kb / S + (kTile + out_us) * bn / 64);
      // few tokens: the weights' bytes bound the kernel; every CTA has a place
      // from the start, so that all of K streams at once
      if (n <= 64 && S > 1 && share > 2.f) continue;
      if (best.bn == 0 || us < best.us) best = SplitPlan{bn, S, us};
    }
    if (n <= bn) break;
  }
  return best;
}

// ---------------------------------------------------------- the whole calls

// What an epilogue's further outputs cost on either family, in us (on split
// tiles, per 64 tokens): gate/up writes G, U and A, dA reads G and U and writes
// dG and dU.
constexpr float kPairUpUs = 0.6f, kPairActUs = 0.45f, kSplitUpUs = 2.9f, kSplitActUs = 2.f;

struct ForwardPlan {
  bool up_on_pairs, down_on_pairs;
  PairPlan up_pair;
  SplitPlan up, down;
};
inline ForwardPlan forward_plan(int64_t T, int64_t D, int64_t F, int num_sms) {
  ForwardPlan p;
  p.up = split_plan(T, F, 64, cdiv(D, 64), kSplitUpUs, false, num_sms);
  p.up_pair = pair_plan(T, 2 * F, cdiv(D, 64), kPairUpUs, num_sms);
  p.up_on_pairs = p.up_pair.us < p.up.us;
  p.down = split_plan(T, D, 128, cdiv(F, 64), 0.f, false, num_sms);
  p.down_on_pairs = pair_us(pair_units(T, D), cdiv(F, 64), 0.f, num_sms) < p.down.us;
  return p;
}

struct BackwardPlan {
  bool act_on_pairs, grads_together, x_on_pairs, w_on_pairs;
  PairPlan act_pair;
  SplitPlan act, x, w;
};
inline BackwardPlan backward_plan(int64_t T, int64_t D, int64_t F, int num_sms) {
  BackwardPlan p;
  p.act = split_plan(T, F, 128, cdiv(D, 64), kSplitActUs, false, num_sms);
  p.act_pair = pair_plan(T, F, cdiv(D, 64), kPairActUs, num_sms);
  p.act_on_pairs = p.act_pair.us < p.act.us;
  // dX (K = 2 F) and the three dW (K = T): each on either family, or all in
  // one launch of pairs, as long as its busiest pair
  const int64_t kx = 2 * cdiv(F, 64), kw = cdiv(T, 64);
  const int64_t ux = pair_units(T, D), uw = 3 * pair_units(F, D);
  p.x = split_plan(T, D, 128, kx, 0.f, false, num_sms);
  // three gradients of F x D, as one of 3 F rows
  p.w = split_plan(3 * cdiv(F, 128) * 128, D, 128, kw, 0.f, true, num_sms);
  const float x_us = pair_us(ux, kx, 0.f, num_sms), w_us = pair_us(uw, kw, 0.f, num_sms);
  p.x_on_pairs = x_us < p.x.us;
  p.w_on_pairs = w_us < p.w.us;
  const UnitDeal deal = deal_units(static_cast<int>(uw), kw, static_cast<int>(ux), kx);
  const int pairs = static_cast<int>(std::min<int64_t>(uw + ux, num_sms / 2));
  const float both_us =
      kPairUsFixed + kPairUsPerKb * static_cast<float>(
                                        busiest_pair(deal, std::max(kx, kw), std::min(kx, kw), pairs));
  p.grads_together = both_us <= std::min(x_us, p.x.us) + std::min(w_us, p.w.us);
  return p;
}

}  // namespace ss
