// pa_rule.cuh -- the score rule of pa_decode_scored / pa_decode_multi_scored on
// the device: which key positions a query row sees, and what becomes of its
// scores.
//
//   t    = scale * q . K_j                          (products in fp32)
//   t    = c tanh(t / c)                            if a cap c is given
//   t    = t - slope_h |pos - j|                    if slopes are given
//   seen = max(key_start, pos - window + 1, 0) <= j <= max(pos, prefix - 1)
//
// The kernels work in base 2 (scores times log2 e).  The cap is taken as
// c tanh(x) = c - 2 c / (1 + e^(2 x)), one exponential and one reciprocal: its
// error is about c 2^-22 whatever x is (e^(2x) = inf gives c, 0 gives -c), a
// thousandth of what the hardware's tanh (2^-11 of its value) would leave on a
// cap of 50, where a score off by 0.02 is a weight off by 2 %.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "pa_internal.h"

namespace pa {

// The rule as the kernels take it (host-built by make_rule).
struct RuleParams {
  const float* slopes;        // [Hq] or null
  const int32_t* key_starts;  // [query rows] or null
  const int32_t* prefix_lens; // [num_seqs] or null
  int window;                 // 0: none
  float cap_log2;             // cap * log2 e; 0: no cap
  float scale;                // of the raw dot: scale * log2 e, or 2 log2 e * scale / cap with a cap
};

constexpr float kLog2e = 1.4426950408889634f;

inline RuleParams make_rule(const pa_score_rule& r, float scale) {
  RuleParams p;
  p.slopes = r.alibi_slopes;
  p.key_starts = r.key_starts;
  p.prefix_lens = r.prefix_lens;
  p.window = r.window;
  p.cap_log2 = r.softcap * kLog2e;
  p.scale = r.softcap > 0.f ? 2.f * kLog2e * (scale / r.softcap) : scale * kLog2e;
  return p;
}

// Positions lo .. hi that query row `row` (of sequence b, at position pos of
// its L tokens) sees; none when lo > hi.
__device__ __forceinline__ void rule_limits(const RuleParams& r, int b, int64_t row, int pos, int L,
                                            int& lo, int& hi) {
  lo = r.key_starts != nullptr ? max(0, __ldcg(r.key_starts + row)) : 0;
  if (r.window > 0) lo = max(lo, pos - r.window + 1);
  hi = pos;
  if (r.prefix_lens != nullptr) hi = max(hi, min(max(__ldcg(r.prefix_lens + b), 0), L) - 1);
}

// First and last position seen by any of the query tokens i0 .. i1 - 1 of
// sequence b (rows q0 + i, positions first_pos + i); lo > hi when none sees
// any.  Every lane of the warp gets the same answer.
__device__ __forceinline__ void rule_span(const RuleParams& r, int b, int64_t q0, int first_pos,
                                          int L, int i0, int i1, int& lo, int& hi) {
  lo = 0x7fffffff;
  hi = -1;
  for (int i = i0 + static_cast<int>(threadIdx.x & 31); i < i1; i += 32) {
    int l, h;
    rule_limits(r, b, q0 + i, first_pos + i, L, l, h);
    if (l <= h) {
      lo = min(lo, l);
      hi = max(hi, h);
    }
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
}

__device__ __forceinline__ float rule_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rule_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What a kernel instance does to the scores.  The cap is a property of the
// instance: as a run-time condition the compiler turns it into a select, and
// every score pays its exponential and reciprocal (512-token chunks without a
// cap, 332 GFLOP, on the kernel with two threads per row: 964 us, 805 us as an
// instance of its own).
enum Rule { kNoRule = 0, kRuleOpen = 1, kRuleCapped = 2 };

inline Rule rule_kind(bool has_rule, const pa_score_rule& r) {
  return !has_rule ? kNoRule : r.softcap > 0.f ? kRuleCapped : kRuleOpen;
}

// x = rule.scale * (q . K_j) capped (base 2); x itself without a cap.
template <int RULE>
__device__ __forceinline__ float rule_cap(float cap_log2, float x) {
  if constexpr (RULE == kRuleCapped)
    return fmaf(-2.f * cap_log2, rule_rcp(1.f + rule_ex2(x)), cap_log2);
  else
    return x;
}

// The score (base 2) of x = rule.scale * (q . K_j): capped, and less
// slope_log2 * away (slope_log2 = slope * log2 e, 0 without slopes).
template <int RULE>
__device__ __forceinline__ float rule_score(const RuleParams& r, float x, float slope_log2,
                                            float away) {
  return fmaf(-slope_log2, away, rule_cap<RULE>(r.cap_log2, x));
}

}  // namespace pa
