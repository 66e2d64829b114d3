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
  const int64_t share = cdiv(ux * kx + uw * kw, num_sms / 2);
  const float both_us =
      kPairUsFixed + kPairUsPerKb * static_cast<float>(std::max(share, std::max(kx, kw)));
  p.grads_together = both_us <= std::min(x_us, p.x.us) + std::min(w_us, p.w.us);
  return p;
}

}  // namespace ss
