// route_scored.cu -- routing by scores: sigmoid or softmax scores, a balance
// bias on the score, groups of experts, top-k, renormalised and scaled gates;
// and the gradient of the logits through the gates.
//
//   score[e] = sigmoid(l[e])  or  softmax(l)[e]
//   key[e]   = score[e] + bias[e]
//   group score = the largest key of the group, or the sum of its two largest;
//   the top_groups best groups are kept (ties: the lower group)
//   ids = the k largest keys of the kept groups (ties: the lower expert)
//   gate[j] = scale * score[ids[j]] (/ the sum of the k scores with renorm)
//
// Scores and keys are defined in binary64: a selection is a discontinuous
// function of the keys, so two evaluations agree only if neither rounds keys
// that differ onto one value.  A binary64 score of every expert is what bounds
// that definition taken literally (Fine-grained, 65536 x 512: 504 us), so the
// keys of a token are formed in binary32 with a bound on their error, and
// binary64 decides among the few that the bound leaves open:
//   1. group scores in binary32; the kept groups are certain when the gap
//      between the last kept and the first left out exceeds the bound, else the
//      keys that count in them are taken in binary64;
//   2. tau = the k-th largest lane maximum of the kept keys, less the bound: no
//      key below it can be among the k best; the keys at or above it (k to k+4
//      of them, usually) are compacted, one a lane;
//   3. they are ranked by their binary32 keys; where two neighbours among the k
//      best are closer than the bound, by their binary64 keys, ties by expert.
// A token whose candidates stay open is decided in binary64 throughout, out of line:
//   - masks that leave less than k finite keys, and NaN;
//   - more than 32 keys within the bound of the k-th largest lane maximum: keys closer
//     together than 1e-6 (sigmoid scores all below that or saturated, logits below -14 or
//     above 16; a biased softmax over logits equal to 1e-3), or k above about 20, where
//     the k-th lane maximum lies far below the k-th key;
//   - more than 32 groups.
// A whole batch of them costs what the definition taken literally does: 65536 x 512 without
// groups takes 55 us, 240 with sigmoid logits around -14, 380 around -16 and of equal
// logits, 440 with a biased softmax equal to 1e-3, 700 with k = 24, 880 with k = 32; 750
// with 64 groups.
//
// Bound by issue: 989 warp instructions a token of 512 experts with groups, 699
// without.  65536 x 512, k 10, 4 of 8 groups: 78 us; without groups 55.
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "route_core.cuh"

namespace moe {

namespace {

constexpr int kScoredWarps = 4;

// Groups of experts: none, any, or a power of two of them whose keys are as many whole
// 16-byte pieces for every lane (E = 32 NK, E / groups a multiple of 4).
enum { kNoGroups = 0, kAnyGroups = 1, kEvenGroups = 2 };

__device__ __forceinline__ double wmax_d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
__device__ __forceinline__ double wsum_d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// Warp arg-max over (value, id), larger value first, then the lower id; lanes
// without a candidate pass id < 0.  Every lane returns the winner's id.
__device__ __forceinline__ int warp_argmax(double v, int id) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double ov = __shfl_xor_sync(kFull, v, o);
    const int oi = __shfl_xor_sync(kFull, id, o);
    if (oi >= 0 && (id < 0 || ov > v || (ov == v && oi < id))) {
      v = ov;
      id = oi;
    }
  }
  return id;
}

__device__ __forceinline__ double score_d(double l, double m, double inv_sum, bool softmax) {
  return softmax ? exp(l - m) * inv_sum : __drcp_rn(1.0 + exp(-l));
}

// One token, one warp, everything in binary64.  `key` holds E doubles of this
// warp; a key becomes NaN once its expert is excluded or taken.  Lane j < k
// returns slot j's expert and its score; false: a key was NaN or +inf.
__device__ bool scored_token_exact(const float* __restrict__ row, const float* __restrict__ bias,
                                   int E, int k, const ScoreRule& R, int lane, double* key,
                                   int& sel_e, double& sel_s) {
  const bool softmax = R.softmax != 0;
  double m = 0.0, inv_sum = 1.0;
  if (softmax) {
    m = -INFINITY;
    for (int e = lane; e < E; e += 32) m = fmax(m, (double)__ldg(row + e));
    m = wmax_d(m);
    double s = 0.0;
    for (int e = lane; e < E; e += 32) s += exp((double)__ldg(row + e) - m);
    inv_sum = 1.0 / wsum_d(s);
  }
  bool bad = false;
  for (int e = lane; e < E; e += 32) {
    double v = score_d((double)__ldg(row + e), m, inv_sum, softmax);
    if (bias != nullptr) v += (double)__ldg(bias + e);
    bad |= !(v < INFINITY);
    key[e] = v;
  }
  if (__any_sync(kFull, bad)) return false;
  __syncwarp();
  if (R.top_groups < R.groups) {
    const int G = E / R.groups;
    double gs[2];  // lane l scores groups l and l + 32
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      double a = -INFINITY, b = -INFINITY;
      const int g = lane + 32 * u;
      if (g < R.groups)
        for (int i = 0; i < G; ++i) {
          const double v = key[g * G + i];
          if (v > a) {
            b = a;
            a = v;
          } else if (v > b) {
            b = v;
          }
        }
      gs[u] = R.group_top == 2 ? a + b : a;
    }
    uint64_t kept = 0ull;
    for (int r = 0; r < R.top_groups; ++r) {
      int id = -1;
      double v = 0.0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int g = lane + 32 * u;
        if (g < R.groups && !((kept >> g) & 1ull) && (id < 0 || gs[u] > v)) {
          v = gs[u];
          id = g;
        }
      }
      kept |= 1ull << warp_argmax(v, id);
    }
    for (int e = lane; e < E; e += 32)
      if (!((kept >> (e / G)) & 1ull)) key[e] = NAN;
    __syncwarp();
  }
  sel_e = 0;
  for (int j = 0; j < k; ++j) {
    int id = -1;
    double v = 0.0;
    for (int e = lane; e < E; e += 32) {
      const double q = key[e];
      if (q == q && (id < 0 || q > v)) {
        v = q;
        id = e;
      }
    }
    const int win = warp_argmax(v, id);
    if (lane == j) sel_e = win;
    if (lane == (win & 31)) key[win] = NAN;
    __syncwarp();
  }
  sel_s = lane < k ? score_d((double)__ldg(row + sel_e), m, inv_sum, softmax) : 0.0;
  return true;
}

__device__ __forceinline__ float scored_gate(double s, int renorm, double scale) {
  if (renorm) {
    const double sum = wsum_d(s);
    s = sum > 1e-290 ? s * __drcp_rn(sum) : sum > 0.0 ? s / sum : 0.0;
  }
  return (float)(s * scale);
}

// Per-warp shared memory: two staged rows of logits (together the exact form's E
// doubles), the candidates and, where groups are scored from shared memory, the
// binary32 keys.
constexpr int kCand = 32;
struct CandArea {
  double key[kCand];  // binary64 keys, where they are needed
  float key32[kCand + 4];
  int expert[kCand];
  int slot[kCand];
};

__device__ __noinline__ bool scored_token_slow(const float* row, const float* bias, int E, int k,
                                               const ScoreRule& R, int lane, double* key,
                                               int& sel_e, double& sel_s) {
  return scored_token_exact(row, bias, E, k, R, lane, key, sel_e, sel_s);
}

// How far a binary32 key can be from its binary64 value, in steps u = 2^-24.
// Sigmoid: 2^x is off by 4 u of itself and its argument by 1.23 u |l|; the score s takes
// s (1 - s) of that (at most 1 u and 0.28 u), 1 u for the addition, 2 u for the reciprocal:
// 4.3 u, 2.6e-7.
// Softmax: 2^x is off by 4 u and its argument, d = l - m times log2 e, by 1.23 u |d|, of
// which the score p takes p and p |d| < 0.37: 4.9 u for two scores, which sum to at most 1.
// (Without a bias by 2.23 u |d|, but nothing else is: 5.7 u.)  The sum is off by 4 u, 1.23 u
// times the scores' mean |d| (at most 4.45 over 1024 scores: one ahead of equal others),
// 10 u for its additions and 3 u for the reciprocal, alike for every score of the token: two
// keys move apart by the difference of their scores, at most 1, times these 22.5 u.  27.4 u
// or 1.7e-6 in all, below the 2e-6 by which two bounds keep keys apart.
// One addition adds 1 u of the key.
// The gates of the full softmax are binary64 exponentials times a reciprocal of which 5 u
// are its additions and 1 u its rounding, and are rounded once: 16.5 u, 9.8e-7.
__device__ __forceinline__ float key_bound(float v) { return 1.0e-6f + 2.5e-7f * fabsf(v); }

// What the group scoring needs of the sizes, computed once: unit = 1 << shift lanes a
// group (a power of two) walk its n pieces (16 bytes, or single keys where groups are
// not whole pieces) from `start` on, in turns that keep the groups' lanes on different
// banks.
struct GroupPlan {
  int G = 1, shift = 0, n = 1, start = 0;
  // of this lane's group (0: none), one bit each: its columns of 32 experts where groups
  // are whole columns, else the group itself
  uint32_t bits = 0u;
  uint32_t magic = 0u;  // e / G == __umulhi(e, magic) for e < 2^16 (G > 1)
  __device__ void init(int E, int groups, int lane) {
    G = E / groups;
    if (groups > 32) return;  // (the exact form's)
    shift = 31 - __clz(32 / groups);
    n = (G & 3) == 0 ? G >> 2 : G;
    const int unit = 1 << shift, g = lane >> shift, sub = lane & (unit - 1);
    start = sub + unit * g;
    if (start >= n) start = sub + unit * (g % ((n + unit - 1) >> shift));
    if (g < groups) bits = (G & 31) == 0 ? (kFull >> (32 - (G >> 5))) << (g * (G >> 5)) : 1u << g;
    magic = G > 1 ? (uint32_t)((0x100000000ull + (uint64_t)G - 1) / (uint64_t)G) : 0u;
  }
};

// 1 / sum of the row's exponentials, summed as the exact form sums them.
__device__ __noinline__ double softmax_scale_d(const float* row, int E, double m, int lane) {
  double s = 0.0;
  for (int e = lane; e < E; e += 32) s += exp((double)row[e] - m);
  return 1.0 / wsum_d(s);
}

// f(LO) + .. + f(LO + N - 1), N a power of two, added pairwise.
template <int LO, int N, typename F>
__device__ __forceinline__ float sum_tree(const F& f) {
  if constexpr (N == 1)
    return f(LO);
  else
    return sum_tree<LO, N / 2>(f) + sum_tree<LO + N / 2, N / 2>(f);
}

// 1 / (sum of the lanes' values, each in [0, 33] and together at least 0.9), to one
// rounding.  The values are added as whole numbers of 2^-20 and, of the rest, of 2^-42:
// exact but for 32 * 2^-42, and the reduction of an integer is one instruction.
__device__ __forceinline__ float lanes_total_inverse(float v) {
  const float scaled = v * 0x1p20f;
  const uint32_t whole = __float2uint_rz(scaled);
  const uint32_t rest = __float2uint_rz((scaled - (float)whole) * 0x1p22f);
  const uint32_t hi = __reduce_add_sync(kFull, whole), lo = __reduce_add_sync(kFull, rest);
  const float a = (float)hi;
  const float b = fmaf((float)lo, 0x1p-22f, (float)(int)(hi - (uint32_t)a));  // a + b: the sum
  const float r = rcp_f(a);
  return fmaf(r, fmaf(-b, r, fmaf(-a, r, 1.0f)), r) * 0x1p20f;
}

// A softmax's powers are 2^(l log2 e - c), c = m log2 e rounded, up to this |m|.
constexpr float kShift = 32768.0f;
// 2^(m log2 e - c) - 1: what the reciprocal of their sum lacks of that of the sum of
// e^(l - m).  (|m log2 e - c| < 2^-8: the third power of its series is 2^-35.)
__device__ __forceinline__ float shift_lost(float m) {
  const float lost =
      fabsf(m) <= kShift ? 0.693147181f * fmaf(m, kLog2e, -(m * kLog2e)) : 0.0f;
  return lost * fmaf(lost, fmaf(lost, 0.166666667f, 0.5f), 1.0f);
}

// The kept groups' bits by binary64 scores, where binary32 leaves them open:
// keys below `low` are not among the ones that count in this lane's group.  (Decided by
// the exact form, one such token held its warp for some 10 us: 65536 x 512 took 90 us
// instead of 80.)
__device__ __noinline__ uint32_t open_groups(const float* row, const float* __restrict__ bias,
                                             const float* skey, const ScoreRule& R, int G,
                                             int shift, uint32_t bits, float low, double m,
                                             double inv_sum, int lane) {
  const int unit = 1 << shift, g = lane >> shift, sub = lane & (unit - 1);
  double a = -INFINITY, b = -INFINITY;
  if (g < R.groups)
    for (int e = g * G + sub; e < (g + 1) * G; e += unit)
      if (skey[e] >= low) {
        double v = score_d((double)row[e], m, inv_sum, R.softmax != 0);
        if (bias != nullptr) v += (double)__ldg(bias + e);
        b = fmax(b, fmin(a, v));
        a = fmax(a, v);
      }
  for (int o = 1; o < unit; o <<= 1) {
    const double oa = __shfl_xor_sync(kFull, a, o), ob = __shfl_xor_sync(kFull, b, o);
    b = fmax(fmin(a, oa), fmax(b, ob));
    a = fmax(a, oa);
  }
  const double score = R.group_top == 2 ? a + b : a;
  int rank = 0;
  for (int j = 0; j < R.groups; ++j) {
    const double other = __shfl_sync(kFull, score, j << shift);
    rank += (other > score || (other == score && j < g)) ? 1 : 0;
  }
  return __reduce_or_sync(kFull, rank < R.top_groups ? bits : 0u);
}

// One token, decided as described above; false: not decided.  Lane j < k returns
// slot j's expert and score.  `row` is the staged row.
template <int NK, bool SOFTMAX, bool BIAS, int GROUPED, bool FULL>
__device__ __forceinline__ bool scored_token_fast(const float* row, int E, int k,
                                                  const ScoreRule& R, const GroupPlan& L, int lane,
                                                  uint32_t vmask, const float* __restrict__ bias,
                                                  float* skey, CandArea* C, int& sel_e,
                                                  double& sel_s) {
  // without a bias the logits are in the softmax's order (but their sums are not)
  const bool raw = SOFTMAX && !BIAS && !(GROUPED && R.group_top == 2);
  auto valid = [&](int i) { return FULL || ((vmask >> i) & 1u) != 0u; };
  float key[NK];
#pragma unroll
  for (int i = 0; i < NK; ++i) key[i] = valid(i) ? row[lane + 32 * i] : -INFINITY;
  float m = 0.0f, scale = 1.0f;  // softmax: largest logit, and what 2^.. is multiplied with
  float from = 0.0f, c = 0.0f;
  auto power = [&](float l) { return ex2_f(fmaf(l - from, kLog2e, -c)); };  // e^(l - m)
  if (SOFTMAX) {
    m = key[0];
#pragma unroll
    for (int i = 1; i < NK; ++i) m = max2_nan(m, key[i]);
    if (__any_sync(kFull, m != m)) return false;
    m = code_float(__reduce_max_sync(kFull, order_code(m)));
    if (!(fabsf(m) < INFINITY)) return false;  // a row without a finite maximum
    from = m;
    if (BIAS || !R.renorm) {
      // The argument (l - m) log2 e with one rounding: less c, which is m log2 e rounded (all
      // powers and their sum are off by the same factor, see shift_lost); from 2^15 on,
      // where that would be too much, l - m is exact wherever 2^.. is not 0.  A lane's terms
      // are added pairwise: log2(NK) <= 5 roundings.  Where the sum goes into the gates, the
      // lanes' parts are added without any (for the keys alone too, 65536 x 512 took 69 us
      // instead of 66).
      const bool small = fabsf(m) <= kShift;
      from = small ? 0.0f : m;
      c = small ? m * kLog2e : 0.0f;
      float part = sum_tree<0, NK>([&](int i) { return power(key[i]); });
      if (R.renorm) {  // scales the keys alone
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(kFull, part, o);
        scale = rcp_f(part);
      } else {
        scale = lanes_total_inverse(part);
      }
    }
  }
  // the key of expert e with logit l
  auto key_of = [&](float l, int e) -> float {
    float v;
    if (SOFTMAX) {
      if (raw) return l;
      v = power(l);
      return BIAS ? fmaf(v, scale, __ldg(bias + e)) : v;
    }
    v = sigmoid_f(l);
    return BIAS ? v + __ldg(bias + e) : v;
  };
  if (!SOFTMAX || !raw) {
#pragma unroll
    for (int i = 0; i < NK; ++i)
      if (valid(i)) key[i] = key_of(key[i], lane + 32 * i);
  }
  // logits are exact; two closer than the bound are left to binary64, whose
  // exponentials could coincide
  auto bound = [&](float v) { return key_bound(raw ? fabsf(v) + fabsf(m) : v); };

  if (GROUPED) {
    const int G = L.G, unit = 1 << L.shift, g = lane >> L.shift, sub = lane & (unit - 1);
#pragma unroll
    for (int i = 0; i < NK; ++i)
      if (valid(i)) skey[lane + 32 * i] = key[i];
    __syncwarp();
    float a = -INFINITY, b = -INFINITY;  // the group's two largest keys (NaN: in a)
    auto take = [&](float v) {
      b = fmaxf(b, fminf(a, v));
      a = max2_nan(a, v);
    };
    if constexpr (GROUPED == kEvenGroups) {
      // straight-line: 79 us instead of 83 at 65536 x 512 with 8 groups, 53 instead of 57 at
      // 65536 x 128 with 4
      constexpr int kSteps = NK / 4;
      const float4* part = reinterpret_cast<const float4*>(skey + g * G) + sub;
#pragma unroll
      for (int it = 0; it < kSteps; ++it) {
        const float4 q = part[((g ^ it) & (kSteps - 1)) << L.shift];
        const float h0 = max2_nan(q.x, q.y), l0 = fminf(q.x, q.y);
        const float h1 = max2_nan(q.z, q.w), l1 = fminf(q.z, q.w);
        const float h = max2_nan(h0, h1), l = max3_nan(fminf(h0, h1), l0, l1);
        b = max3_nan(b, l, fminf(a, h));
        a = max2_nan(a, h);
      }
    } else if (g < R.groups) {
      const float* part = skey + g * G;
      const int n = L.n;
      int at = L.start;
      for (int it = sub; it < n + sub; it += unit) {
        if (at < n) {
          if ((G & 3) == 0) {
            const float4 q = reinterpret_cast<const float4*>(part)[at];
            take(q.x);
            take(q.y);
            take(q.z);
            take(q.w);
          } else {
            take(part[at]);
          }
        }
        at += unit;
        if (at >= n + sub) at = sub;
      }
    }
    if (__any_sync(kFull, !(a < INFINITY))) return false;
#pragma unroll 1
    for (int o = 1; o < unit; o <<= 1) {
      const float oa = __shfl_xor_sync(kFull, a, o), ob = __shfl_xor_sync(kFull, b, o);
      b = fmaxf(fminf(a, oa), fmaxf(b, ob));
      a = fmaxf(a, oa);
    }
    const float score = g < R.groups ? (R.group_top == 2 ? a + b : a) : -INFINITY;
    float mag = 0.0f;
    if (score > -INFINITY) mag = fmaxf(fabsf(a), R.group_top == 2 ? fabsf(b) : 0.0f);
    // the kept groups, certain if the best one left out is further off than the errors
    // of two scores (a group without a finite key scores -inf in any precision), else
    // decided by their binary64 scores
    // (maxima on order codes: the integer reduction is one instruction)
    const float big = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(mag)));
    // (ranks of the groups, each compared with all others, were no faster for 8 of them, 2 us
    // slower for 2 and 13 for 32: 65536 x 512)
    uint32_t kept = 0u, best = 0u;
    uint32_t scode = sub == 0 && g < R.groups ? order_code(score) : 0u;
    for (int r = 0; r < R.top_groups; ++r) {
      best = __reduce_max_sync(kFull, scode);
      const int who = __ffs(__ballot_sync(kFull, scode == best)) - 1;
      kept |= __shfl_sync(kFull, L.bits, who);
      if (lane == who) scode = 0u;
    }
    const uint32_t next = __reduce_max_sync(kFull, scode);
    if (!(code_float(best) - code_float(next) > 4.0f * bound(big))) {
      const float last = R.group_top == 2 ? b : a;
      const double md = (double)m;
      kept = open_groups(row, BIAS ? bias : nullptr, skey, R, G, L.shift, L.bits,
                         last - 2.0f * bound(big), md, SOFTMAX ? softmax_scale_d(row, E, md, lane) : 1.0, lane);
    }
    if ((G & 31) == 0) {  // whole columns: bit i says whether column i is kept
#pragma unroll
      for (int i = 0; i < NK; ++i) key[i] = (kept & (1u << i)) ? key[i] : -INFINITY;
    } else {
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        const uint32_t e = (uint32_t)(lane + 32 * i);
        const uint32_t q = G > 1 ? __umulhi(e, L.magic) : e;
        if (!((kept >> (q & 31u)) & 1u)) key[i] = -INFINITY;
      }
    }
  }

  // tau: the k-th largest lane maximum, on order codes whose low 5 bits are the lane
  float mm = key[0];
#pragma unroll
  for (int i = 1; i + 1 < NK; i += 2) mm = max3_nan(mm, key[i], key[i + 1]);
  mm = max2_nan(mm, key[NK - 1]);
  if (__any_sync(kFull, !(mm < INFINITY))) return false;
  uint32_t code = (order_code(mm) & ~31u) | (uint32_t)(31 - lane);
  uint32_t top = __reduce_max_sync(kFull, code);
  const float wmax = code_float(top | 31u);  // no lane's maximum is larger
#pragma unroll 2
  for (int j = 1; j < k; ++j) {
    code = code == top ? 0u : code;
    top = __reduce_max_sync(kFull, code);
  }
  if (top < 0x00800000u) return false;  // a lane without a finite key among the k
  const float tau = code_float(top & ~31u);
  if (SOFTMAX && raw && !(tau - m > -700.0f)) return false;  // scores that vanish in binary64 tie
  const float open = 2.0f * bound(fmaxf(fabsf(tau), fabsf(wmax)));
  const float thr = tau - open;
  uint32_t cm = 0u;
#pragma unroll
  for (int i = 0; i < NK; ++i) cm |= (key[i] >= thr) ? (1u << i) : 0u;
  const int total = (int)__reduce_add_sync(kFull, (unsigned)__popc(cm));
  if (total > kCand || total < k) return false;
  int base = 0;
#pragma unroll 1
  while (true) {
    const unsigned any = __ballot_sync(kFull, cm != 0u);
    if (any == 0u) break;
    if (cm != 0u) {
      C->expert[base + __popc(any & lanemask_lt())] = lane + 32 * (__ffs(cm) - 1);
      cm &= cm - 1u;
    }
    base += __popc(any);
  }
  __syncwarp();
  const int e = lane < total ? C->expert[lane] : 0;
  const float v = lane < total ? key_of(row[e], e) : -INFINITY;
  C->key32[lane] = v;
  if (lane < 4) C->key32[kCand + lane] = -INFINITY;
  __syncwarp();
  // ranked by the binary32 keys: larger ones, and whether one is no further below than
  // the bound (equal ones, the key itself among them, do not count twice)
  int n = 0, within = 0;
  const float low = v - open;
#pragma unroll 2
  for (int j = 0; j < total; j += 4) {
    const float4 q = *reinterpret_cast<const float4*>(C->key32 + j);
    n += (q.x > v) + (q.y > v) + (q.z > v) + (q.w > v);
    within += (q.x >= low) + (q.y >= low) + (q.z >= low) + (q.w >= low);
  }
  if (lane < total) C->slot[n] = lane;
  if (__any_sync(kFull, lane < total && n < k && within - n != 1)) {
    const double inv = SOFTMAX && BIAS ? softmax_scale_d(row, E, (double)m, lane) : 1.0;
    double d = 0.0;
    if (lane < total) {
      d = score_d((double)row[e], (double)m, inv, SOFTMAX);
      if (BIAS) d += (double)__ldg(bias + e);
      C->key[lane] = d;
    }
    __syncwarp();
    n = 0;
    if (lane < total)
      for (int j = 0; j < total; ++j) {
        const double o = C->key[j];
        n += (o > d || (o == d && C->expert[j] < e)) ? 1 : 0;
      }
    if (lane < total) C->slot[n] = lane;
  }
  __syncwarp();
  sel_e = 0;
  sel_s = 0.0;
  if (lane < k) {
    sel_e = C->expert[C->slot[lane]];
    sel_s = score_d((double)row[sel_e], (double)m, 1.0, SOFTMAX);
    if (SOFTMAX && !R.renorm) sel_s *= (double)scale * (1.0 + (double)shift_lost(m));
  }
  __syncwarp();
  return true;
}

// Stage a row: this lane's 16-byte pieces, or words where rows are not aligned.
__device__ __forceinline__ void stage_row(float* dst, const float* __restrict__ src, int E, int lane,
                                          bool vec) {
  if (vec) {
    for (int i = lane * 4; i < E; i += 128)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                       static_cast<uint32_t>(__cvta_generic_to_shared(dst + i))),
                   "l"(src + i)
                   : "memory");
  } else {
    for (int i = lane; i < E; i += 32)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                       static_cast<uint32_t>(__cvta_generic_to_shared(dst + i))),
                   "l"(src + i)
                   : "memory");
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}

// Floats of a staged row, and bytes of a warp's shared memory.
__host__ __device__ constexpr int row_floats(int E) { return (E + 3) / 4 * 4; }
__host__ __device__ constexpr size_t warp_bytes(int E, bool keys) {
  return sizeof(float) * (size_t)row_floats(E) * (keys ? 3 : 2) + sizeof(CandArea);
}

constexpr int scored_min_blocks(int nk) { return nk <= 8 ? 8 : nk == 16 ? 7 : 4; }

template <int NK, bool SOFTMAX, bool BIAS, int GROUPED, bool FULL>
__global__ void __launch_bounds__(kScoredWarps * 32, scored_min_blocks(NK))
    route_scored_kernel(const float* __restrict__ logits, const float* __restrict__ bias, int T,
                        int E, int k, const __grid_constant__ ScoreRule R, int vec,
                        int32_t* __restrict__ ids, float* __restrict__ gates, WsHeader* hdr) {
  extern __shared__ __align__(16) uint8_t smem[];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  uint8_t* mine = smem + (size_t)w * warp_bytes(E, GROUPED);
  CandArea* C = reinterpret_cast<CandArea*>(mine);
  float* rows = reinterpret_cast<float*>(mine + sizeof(CandArea));
  const int stride = row_floats(E);
  float* skey = rows + 2 * stride;
  uint32_t vmask = 0u;
#pragma unroll
  for (int i = 0; i < NK; ++i)
    if (lane + 32 * i < E) vmask |= 1u << i;
  const bool fast = !GROUPED || R.groups <= 32;
  GroupPlan plan;
  if (GROUPED) plan.init(E, R.groups, lane);
  const int step = gridDim.x * kScoredWarps;
  int t = blockIdx.x * kScoredWarps + w, turn = 0;
  if (t < T) stage_row(rows, logits + (size_t)t * E, E, lane, vec != 0);
  for (; t < T; t += step, turn ^= 1) {
    if (t + step < T) {
      stage_row(rows + (turn ^ 1) * stride, logits + (size_t)(t + step) * E, E, lane, vec != 0);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncwarp();
    int e = 0;
    double s = 0.0;
    bool ok = fast && scored_token_fast<NK, SOFTMAX, BIAS, GROUPED, FULL>(
                          rows + turn * stride, E, k, R, plan, lane, vmask, bias, skey, C, e, s);
    // Scores at the end of binary64's range: their quotients depend on how each was
    // rounded there, which is for the exact form to say (it divides by the row's sum).
    if (SOFTMAX && BIAS && ok && R.renorm && !__any_sync(kFull, s > 1e-280)) ok = false;
    if (!ok) {
      // the exact form's keys take both staged rows: the next one is staged again
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncwarp();
      ok = scored_token_slow(logits + (size_t)t * E, bias, E, k, R, lane,
                             reinterpret_cast<double*>(rows), e, s);
      __syncwarp();
      if (t + step < T)
        stage_row(rows + (turn ^ 1) * stride, logits + (size_t)(t + step) * E, E, lane, vec != 0);
    }
    float g = 0.0f;
    if (ok) {
      g = scored_gate(s, R.renorm, R.scale);
    } else {  // the slots stay valid: experts 0..k-1 with gates of zero
      e = lane;
      if (lane == 0) report(hdr, MOE_ERR_DEVICE_NAN, t);
    }
    if (lane < k) {
      ids[(size_t)t * k + lane] = e;
      gates[(size_t)t * k + lane] = g;
    }
    __syncwarp();
  }
}

constexpr int kBackWarps = 8;

// The sum, or largest value, over the W lanes of a token.
template <int W, typename F>
__device__ __forceinline__ F lanes_sum(F v) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
template <int W>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

// An expert that appears in several slots of a token gets the sum of their parts, in
// slot order, from its first slot (the others' expert becomes -1).
template <int W>
__device__ __forceinline__ float merge_slots(float d, int& e, int lane) {
  const unsigned same = __match_any_sync(kFull, e < 0 ? -1 - lane : (e | (lane / W) << 16));
  if (__any_sync(kFull, __popc(same) > 1)) {
    float sum = 0.0f;
    for (int j = 0; j < 32; ++j) {
      const float dj = __shfl_sync(kFull, d, j);
      if ((same >> j) & 1u) sum += dj;
    }
    d = sum;
    if (lane != __ffs(same) - 1) e = -1;
  }
  return d;
}

// The largest of row[0..E-1] over the W lanes of its token (NaN passed over).
template <int W>
__device__ __forceinline__ float row_max(const float* __restrict__ row, int E, int j, bool vec) {
  float m = -INFINITY;
  if (vec) {
    for (int i = j * 4; i < E; i += W * 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(row + i));
      m = fmaxf(m, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)));
    }
  } else {
    for (int i = j; i < E; i += W) m = fmaxf(m, __ldg(row + i));
  }
  return lanes_max<W>(m);
}

// Whether the scores of a token's chosen experts (logit l, one a lane; -INFINITY: none)
// sum to zero in binary64, formed as the route's exact form forms them.  M: the row's
// largest logit.  Called by whole warps.
template <int W>
__device__ __noinline__ bool scores_vanish(const float* __restrict__ row, int E, float M, float l,
                                           int j, bool token) {
  double s = 0.0;
  if (token)
    for (int i = j; i < E; i += W) s += exp((double)__ldg(row + i) - (double)M);
  const double inv_sum = 1.0 / lanes_sum<W>(s);
  const double mine = l > -INFINITY ? score_d((double)l, (double)M, inv_sum, true) : 0.0;
  return lanes_sum<W>(mine) == 0.0;
}

// The gradient lives on the chosen experts alone (every rule but the full softmax).
// W lanes a token, two tokens a warp where k <= 16.  The row is zeroed by wide stores
// that wait for nothing, the k values follow them (the warp's stores are ordered by
// the barrier between): store-bound, 4E bytes a token (softmax: 4E read as well, since
// only the row's largest logit tells whether the chosen scores vanish).  32768 x 256,
// k 8, over buffers larger than the L2: sigmoid 13.5 us, softmax 15.4 (13.4 without the
// row); 65536 x 512, k 10, softmax: 55 us, 4.9 TB/s.  On one buffer sigmoid takes 10.2
// us, in 36 registers instead of 32 (fewer warps to hide the loads' latency) 10.9.
template <int W, bool SOFTMAX>
__global__ void __launch_bounds__(kBackWarps * 32, 8)
    route_scored_backward_kernel(const float* __restrict__ logits, const int32_t* __restrict__ ids,
                                 const float* __restrict__ grad_gates, int T, int E, int k,
                                 const __grid_constant__ ScoreRule R,
                                 float* __restrict__ grad_logits, int vec, WsHeader* hdr) {
  constexpr int kTok = 32 / W;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, j = lane % W;
  const int step = gridDim.x * kBackWarps * kTok;
  for (int t0 = (blockIdx.x * kBackWarps + (threadIdx.x >> 5)) * kTok; t0 < T; t0 += step) {
    const int t = t0 + lane / W;
    int e = -1;
    float up = 0.0f;
    if (j < k && t < T) {
      e = __ldg(ids + (size_t)t * k + j);
      up = __ldg(grad_gates + (size_t)t * k + j);
    }
    float* out = grad_logits + (size_t)t0 * E;
    const int n = (min(T - t0, kTok)) * E;
    if ((vec & 1) != 0) {
      for (int i = lane * 4; i < n; i += 128)
        *reinterpret_cast<float4*>(out + i) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    } else {
      for (int i = lane; i < n; i += 32) out[i] = 0.0f;
    }
    if (e >= E || (e < 0 && j < k && t < T)) {
      report(hdr, MOE_ERR_DEVICE_RANGE, e);
      e = -1;
    }
    const float l = e >= 0 ? __ldg(logits + (size_t)t * E + e) : 0.0f;
    up = e >= 0 ? (float)((double)up * R.scale) : 0.0f;
    float d;
    if (SOFTMAX) {  // renormalised: the softmax of the chosen
      // A bias, or few unmasked experts, can choose scores that are all zero in binary64
      // (masks of -inf or any finite value, logits 745 below the largest): the gates are
      // zero there, whatever the logits, and there is no gradient.
      const float* row = logits + (size_t)min(t, T - 1) * E;
      const float M = row_max<W>(row, E, j, (vec & 2) != 0);
      const float c = e >= 0 ? l : -INFINITY;
      const float m = lanes_max<W>(c);
      const float x = c != -INFINITY ? expf(l - m) : 0.0f;
      const float sum = lanes_sum<W>(x);
      float p = sum != 0.0f ? x * (1.0f / sum) : 0.0f;
      const bool far = m > -INFINITY && m - M < -600.0f;
      if (__any_sync(kFull, far)) {
        const bool gone = scores_vanish<W>(row, E, M, c, j, far);
        if (far && gone) p = 0.0f;
      }
      d = p * (up - lanes_sum<W>(up * p));
    } else {
      // sigmoid(l) and 1 - sigmoid(l), both without cancellation
      const float x = expf(-fabsf(l));
      const float big = 1.0f / (1.0f + x), small = x * big;
      const float s = e >= 0 ? (l >= 0.0f ? big : small) : 0.0f, c = l >= 0.0f ? small : big;
      d = up * s;
      if (R.renorm) {
        const float sum = lanes_sum<W>(s), us = lanes_sum<W>(up * s);
        d = sum > 0.0f ? s / sum * (up - us / sum) : 0.0f;
        // scores near or below binary32's range: their quotients in binary64, as the gates'
        const bool tiny = sum < 0x1p-100f;
        if (__any_sync(kFull, tiny && e >= 0)) {
          const double sd = e >= 0 ? 1.0 / (1.0 + exp(-(double)l)) : 0.0;
          const double sumd = lanes_sum<W>(sd);
          const float q = sumd > 0.0 ? (float)(sd / sumd) : 0.0f;
          const float uq = lanes_sum<W>(up * q);
          if (tiny) d = q * (up - uq);
        }
      }
      d = e >= 0 ? d * c : 0.0f;
    }
    d = merge_slots<W>(d, e, lane);
    __syncwarp();
    if (e >= 0) grad_logits[(size_t)t * E + e] = d;
  }
}

// The full softmax without renormalisation: every logit has a gradient.  One warp per
// token; the row's exponentials stay in shared memory between the passes.
__global__ void __launch_bounds__(kBackWarps * 32)
    route_softmax_backward_kernel(const float* __restrict__ logits, const int32_t* __restrict__ ids,
                                  const float* __restrict__ grad_gates, int T, int E, int k,
                                  double scale, float* __restrict__ grad_logits, int vec,
                                  WsHeader* hdr) {
  extern __shared__ float4 sback[];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int words = (E + 3) / 4 * 4;
  float* srow = reinterpret_cast<float*>(sback) + (size_t)w * words;
  for (int t = blockIdx.x * kBackWarps + w; t < T; t += gridDim.x * kBackWarps) {
    const float* row = logits + (size_t)t * E;
    int e = -1;
    float up = 0.0f;
    if (lane < k) {
      e = __ldg(ids + (size_t)t * k + lane);
      up = (float)((double)__ldg(grad_gates + (size_t)t * k + lane) * scale);
      if ((unsigned)e >= (unsigned)E) {
        report(hdr, MOE_ERR_DEVICE_RANGE, e);
        e = -1;
      }
    }
    float m = -INFINITY;
    for (int i = lane; i < E; i += 32) {
      const float l = __ldg(row + i);
      srow[i] = l;
      m = fmaxf(m, l);
    }
    m = lanes_max<32>(m);
    // (a row whose mask leaves nothing has gates of zero: zeros here too, not NaN)
    if (m == -INFINITY) m = 0.0f;
    float sum = 0.0f;
    for (int i = lane; i < E; i += 32) {
      const float p = expf(srow[i] - m);
      srow[i] = p;
      sum += p;
    }
    __syncwarp();
    sum = lanes_sum<32>(sum);
    const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
    float d = e >= 0 ? up * (srow[e] * inv) : 0.0f;
    const float dot = lanes_sum<32>(d);  // sum of up * p over the chosen
    d = merge_slots<32>(d, e, lane);
    for (int i = lane; i < E; i += 32) srow[i] = -(srow[i] * inv) * dot;
    __syncwarp();
    if (e >= 0) srow[e] += d;
    __syncwarp();
    float* out = grad_logits + (size_t)t * E;
    if (vec) {
      for (int i = lane; i < E / 4; i += 32)
        reinterpret_cast<float4*>(out)[i] = reinterpret_cast<const float4*>(srow)[i];
    } else {
      for (int i = lane; i < E; i += 32) out[i] = srow[i];
    }
    __syncwarp();
  }
}

}  // namespace

namespace {

using ScoredKernel = void (*)(const float*, const float*, int, int, int, ScoreRule, int, int32_t*,
                              float*, WsHeader*);

template <int NK, bool SOFTMAX, bool BIAS>
ScoredKernel scored_kernel(int E, int groups) {  // 0: not scored by groups
  const bool full = E == 32 * NK;
  if (groups == 0)
    return full ? route_scored_kernel<NK, SOFTMAX, BIAS, kNoGroups, true>
                : route_scored_kernel<NK, SOFTMAX, BIAS, kNoGroups, false>;
  if constexpr (NK >= 4) {
    if (full && groups <= 32 && (groups & (groups - 1)) == 0 && (E / groups) % 4 == 0)
      return route_scored_kernel<NK, SOFTMAX, BIAS, kEvenGroups, true>;
  }
  return full ? route_scored_kernel<NK, SOFTMAX, BIAS, kAnyGroups, true>
              : route_scored_kernel<NK, SOFTMAX, BIAS, kAnyGroups, false>;
}
template <bool SOFTMAX, bool BIAS>
ScoredKernel scored_kernel(int E, int groups) {
  return E <= 64    ? scored_kernel<2, SOFTMAX, BIAS>(E, groups)
         : E <= 128 ? scored_kernel<4, SOFTMAX, BIAS>(E, groups)
         : E <= 256 ? scored_kernel<8, SOFTMAX, BIAS>(E, groups)
         : E <= 512 ? scored_kernel<16, SOFTMAX, BIAS>(E, groups)
                    : scored_kernel<32, SOFTMAX, BIAS>(E, groups);
}

}  // namespace

cudaError_t launch_route_scored(const LaunchEnv& env, const float* logits, const float* bias, int T,
                                int E, int k, const ScoreRule& rule, int32_t* ids, float* gates,
                                WsHeader* hdr) {
  const bool grouped = rule.top_groups < rule.groups;
  const int groups = grouped ? rule.groups : 0;
  const ScoredKernel kernel =
      rule.softmax ? (bias != nullptr ? scored_kernel<true, true>(E, groups)
                                      : scored_kernel<true, false>(E, groups))
                   : (bias != nullptr ? scored_kernel<false, true>(E, groups)
                                      : scored_kernel<false, false>(E, groups));
  const int vec = (E % 4) == 0 && (reinterpret_cast<uintptr_t>(logits) % 16) == 0;
  const size_t smem = kScoredWarps * warp_bytes(E, grouped);
  int per_sm = 1;
  cudaError_t err = blocks_per_sm((const void*)kernel, kScoredWarps * 32, smem, &per_sm);
  if (err != cudaSuccess) return err;
  int64_t grid = ((int64_t)T + kScoredWarps - 1) / kScoredWarps;
  if (grid > (int64_t)per_sm * env.num_sms) grid = (int64_t)per_sm * env.num_sms;
  return launch_pdl(env, kernel, dim3((unsigned)grid), dim3(kScoredWarps * 32), smem, logits, bias,
                    T, E, k, rule, vec, ids, gates, hdr);
}

cudaError_t launch_route_scored_backward(const LaunchEnv& env, const float* logits,
                                         const int32_t* ids, const float* grad_gates, int T, int E,
                                         int k, const ScoreRule& rule, float* grad_logits,
                                         WsHeader* hdr) {
  const auto wide = [&](const float* p) { return E % 4 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  const int vec = (wide(grad_logits) ? 1 : 0) | (wide(logits) ? 2 : 0);
  const bool dense = rule.softmax && !rule.renorm;
  const size_t smem = dense ? sizeof(float) * kBackWarps * (size_t)((E + 3) / 4 * 4) : 0;
  const auto chosen =
      rule.softmax
          ? (k <= 16 ? route_scored_backward_kernel<16, true> : route_scored_backward_kernel<32, true>)
          : (k <= 16 ? route_scored_backward_kernel<16, false>
                     : route_scored_backward_kernel<32, false>);
  int per_sm = 1;
  cudaError_t err = blocks_per_sm(
      dense ? (const void*)route_softmax_backward_kernel : (const void*)chosen, kBackWarps * 32, smem,
      &per_sm);
  if (err != cudaSuccess) return err;
  const int64_t tokens = kBackWarps * (!dense && k <= 16 ? 2 : 1);
  int64_t grid = ((int64_t)T + tokens - 1) / tokens;
  if (grid > (int64_t)per_sm * env.num_sms) grid = (int64_t)per_sm * env.num_sms;
  if (dense)
    return launch_pdl(env, route_softmax_backward_kernel, dim3((unsigned)grid),
                      dim3(kBackWarps * 32), smem, logits, ids, grad_gates, T, E, k, rule.scale,
                      grad_logits, vec & 1, hdr);
  return launch_pdl(env, chosen, dim3((unsigned)grid), dim3(kBackWarps * 32), 0, logits, ids,
                    grad_gates, T, E, k, rule, grad_logits, vec, hdr);
}

}  // namespace moe
