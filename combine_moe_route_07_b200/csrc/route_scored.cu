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
//      between the last kept and the first left out exceeds the bound;
//   2. tau = the k-th largest lane maximum of the kept keys, less the bound: no
//      key below it can be among the k best; the keys at or above it (k to k+4
//      of them, usually) are compacted, one a lane;
//   3. they are ranked by their binary32 keys; where two neighbours among the k
//      best are closer than the bound, by their binary64 keys, ties by expert.
// A token whose groups or candidates stay open (ties, masks that leave less
// than k finite keys, NaN, more than 32 candidates) is decided in binary64
// throughout, out of line.
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "route_core.cuh"

namespace moe {

namespace {

constexpr int kScoredWarps = 4;

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

// Per-warp shared memory: E doubles (the exact form's keys; the binary32 keys
// while groups are scored), then the candidates.
constexpr int kCand = 32;
struct CandArea {
  double key[kCand];    // binary64 keys, where they are needed
  float key32[kCand + 4];
  int expert[kCand];
  int slot[kCand];
};

__device__ __noinline__ bool scored_token_slow(const float* row, const float* bias, int E, int k,
                                               const ScoreRule& R, int lane, double* key,
                                               int& sel_e, double& sel_s) {
  return scored_token_exact(row, bias, E, k, R, lane, key, sel_e, sel_s);
}

__device__ __forceinline__ float redux_max_f(float v) { return warp_max_nan(v); }

// One token, decided as above; false: not decided.  Lane j < k returns slot j's
// expert and score.  `skey` holds E floats.
template <int NK, bool SOFTMAX, bool BIAS>
__device__ __forceinline__ bool scored_token_fast(const float* __restrict__ row, int E, int k,
                                                  const ScoreRule& R, int lane, uint32_t vmask,
                                                  const float* __restrict__ bias, float* skey,
                                                  CandArea* C, int& sel_e, double& sel_s) {
  float key[NK];
#pragma unroll
  for (int i = 0; i < NK; ++i) key[i] = ((vmask >> i) & 1u) ? __ldg(row + lane + 32 * i) : -INFINITY;
  float m = 0.0f, sum = 1.0f;
  const bool grouped = R.top_groups < R.groups;
  // without a bias the logits are in the softmax's order (but their sums are not)
  const bool raw = SOFTMAX && !BIAS && !(grouped && R.group_top == 2);
  if (SOFTMAX) {
    m = key[0];
#pragma unroll
    for (int i = 1; i < NK; ++i) m = max2_nan(m, key[i]);
    m = redux_max_f(m);
    if (!(fabsf(m) < INFINITY)) return false;  // NaN, or a row without a finite maximum
    if (!raw || !R.renorm) {
      float part = 0.0f;
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        const float p = __expf(key[i] - m);
        part += p;
        if (!raw) key[i] = p;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(kFull, part, o);
      sum = part;
    }
    if (BIAS) {
      const float inv = __fdividef(1.0f, sum);
#pragma unroll
      for (int i = 0; i < NK; ++i) key[i] = ((vmask >> i) & 1u) ? fmaf(key[i], inv, __ldg(bias + lane + 32 * i)) : -INFINITY;
    } else if (!raw) {  // (unnormalised: the scores' order and that of their sums)
#pragma unroll
      for (int i = 0; i < NK; ++i) key[i] = ((vmask >> i) & 1u) ? key[i] : -INFINITY;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const float s = __fdividef(1.0f, 1.0f + __expf(-key[i]));
      key[i] = ((vmask >> i) & 1u) ? (BIAS ? s + __ldg(bias + lane + 32 * i) : s) : -INFINITY;
    }
  }
  // How far a key can be from its binary64 value: scores are within 2^-21 of theirs
  // (the fast exponential is off by 2^-22 and its argument's rounding, which the
  // scores damp; quotient 2^-22; sum of the softmax 2^-22), one addition 2^-24 of the
  // key.  Logits are exact; two of them closer than 2^-20 of their size are left to
  // binary64, whose exponentials could coincide.
  auto bound = [&](float v) { return 1.0e-6f + 2.5e-7f * (fabsf(v) + (raw ? fabsf(m) : 0.0f)); };

#pragma unroll
  for (int i = 0; i < NK; ++i)
    if ((vmask >> i) & 1u) skey[lane + 32 * i] = key[i];
  __syncwarp();
  if (grouped) {
    // Lg lanes a group; they walk its experts in turns that keep the groups' lanes on
    // different banks, and meet in a butterfly of (largest, second largest).
    const int G = E / R.groups;
    const int Lg = 1 << (31 - __clz(32 / R.groups));
    const int g = lane / Lg, sub = lane & (Lg - 1);
    const int steps = (G + Lg - 1) / Lg;
    float a = -INFINITY, b = -INFINITY;
    bool odd = false;
    if (g < R.groups) {
      int turn = g < steps ? g : g % steps;
#pragma unroll 4
      for (int it = 0; it < steps; ++it) {
        const int at = sub + Lg * turn;
        turn = turn + 1 == steps ? 0 : turn + 1;
        if (at < G) {
          const float v = skey[g * G + at];
          odd |= !(v < INFINITY);
          b = fmaxf(b, fminf(a, v));
          a = fmaxf(a, v);
        }
      }
    }
    if (__any_sync(kFull, odd)) return false;
    for (int o = 1; o < Lg; o <<= 1) {
      const float oa = __shfl_xor_sync(kFull, a, o), ob = __shfl_xor_sync(kFull, b, o);
      b = fmaxf(fminf(a, oa), fmaxf(b, ob));
      a = fmaxf(a, oa);
    }
    float score = R.group_top == 2 ? a + b : a;
    if (g >= R.groups || sub != 0) score = -INFINITY;
    // the largest key among those that scores are made of (a group without a finite
    // key scores -inf in any precision)
    const float mag = score == -INFINITY ? 0.0f : fmaxf(fabsf(a), R.group_top == 2 ? fabsf(b) : 0.0f);
    const float big = redux_max_f(mag);
    uint32_t kept = 0u;
    float last = 0.0f;
    for (int r = 0; r < R.top_groups; ++r) {
      last = redux_max_f(score);
      const unsigned hold = __ballot_sync(kFull, score == last);
      const int who = __ffs(hold) - 1;
      kept |= 1u << (who / Lg);
      if (lane == who) score = -INFINITY;
    }
    const float next = redux_max_f(score);
    if (!(last - next > 4.0f * bound(big))) return false;
    const uint32_t magic = G > 1 ? (uint32_t)((0x100000000ull + (uint64_t)G - 1) / (uint64_t)G) : 0u;
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const uint32_t e = (uint32_t)(lane + 32 * i);
      const uint32_t q = G > 1 ? __umulhi(e, magic) : e;
      if (!((kept >> (q & 31u)) & 1u)) key[i] = -INFINITY;
    }
  }

  // tau: the k-th largest lane maximum, on order codes whose low 5 bits are the lane
  float mm = key[0];
#pragma unroll
  for (int i = 1; i + 1 < NK; i += 2) mm = max3_nan(mm, key[i], key[i + 1]);
  mm = max2_nan(mm, key[NK - 1]);
  const float wmax = redux_max_f(mm);
  if (!(wmax < INFINITY)) return false;
  uint32_t code = (order_code(mm) & ~31u) | (uint32_t)(31 - lane);
  uint32_t top = 0u;
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    top = __reduce_max_sync(kFull, code);
    code = code == top ? 0u : code;
  }
  if (top < 0x00800000u) return false;  // a lane without a finite key among the k
  const float tau = code_float(top & ~31u);
  if (raw && !(tau - m > -700.0f)) return false;  // scores that vanish in binary64 tie
  const float open = 2.0f * bound(fmaxf(fabsf(tau), BIAS ? fabsf(wmax) : 0.0f));
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
      const int e = lane + 32 * (__ffs(cm) - 1), p = base + __popc(any & lanemask_lt());
      C->expert[p] = e;
      C->key32[p] = skey[e];
      cm &= cm - 1u;
    }
    base += __popc(any);
  }
  if (lane < 4) C->key32[total + lane] = -INFINITY;  // pads the last group of four
  __syncwarp();
  // ranked by the binary32 keys (equal ones collide on a slot: a gap of zero below)
  const int e = lane < total ? C->expert[lane] : 0;
  const float v = lane < total ? C->key32[lane] : INFINITY;
  int n = 0;
#pragma unroll 2
  for (int j = 0; j < total; j += 4) {
    const float4 q = *reinterpret_cast<const float4*>(C->key32 + j);
    n += (q.x > v) + (q.y > v) + (q.z > v) + (q.w > v);
  }
  float gap = INFINITY;  // to the nearest key below; equal keys: 0
#pragma unroll 2
  for (int j = 0; j < total; j += 4) {
    const float4 q = *reinterpret_cast<const float4*>(C->key32 + j);
    gap = fminf(gap, q.x < v ? v - q.x : INFINITY);
    gap = fminf(gap, q.y < v ? v - q.y : INFINITY);
    gap = fminf(gap, q.z < v ? v - q.z : INFINITY);
    gap = fminf(gap, q.w < v ? v - q.w : INFINITY);
  }
  if (lane < total) C->slot[n] = lane;
  __syncwarp();
  const bool near = lane < total && n < k && (!(gap > open) || C->slot[n] != lane);
  if (__any_sync(kFull, near)) {
    if (SOFTMAX && BIAS) return false;  // (needs the binary64 sum too)
    double d = 0.0;
    if (lane < total) {
      d = score_d((double)__ldg(row + e), (double)m, 1.0, SOFTMAX);
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
    __syncwarp();
    if (lane < total) C->slot[n] = lane;
    __syncwarp();
  }
  sel_e = 0;
  sel_s = 0.0;
  if (lane < k) {
    sel_e = C->expert[C->slot[lane]];
    sel_s = score_d((double)__ldg(row + sel_e), (double)m, 1.0, SOFTMAX);
    if (SOFTMAX && !R.renorm) sel_s /= (double)sum;
  }
  __syncwarp();
  return true;
}

constexpr int scored_min_blocks(int nk) { return nk <= 8 ? 10 : nk == 16 ? 8 : 6; }

template <int NK, bool SOFTMAX, bool BIAS>
__global__ void __launch_bounds__(kScoredWarps * 32, scored_min_blocks(NK))
    route_scored_kernel(const float* __restrict__ logits, const float* __restrict__ bias, int T,
                        int E, int k, const __grid_constant__ ScoreRule R, int32_t* __restrict__ ids,
                        float* __restrict__ gates, WsHeader* hdr) {
  extern __shared__ double skey[];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  double* key = skey + (size_t)w * E;
  CandArea* C = reinterpret_cast<CandArea*>(skey + (size_t)kScoredWarps * E) + w;
  uint32_t vmask = 0u;
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    const int e = lane + 32 * i;
    if (e < E) vmask |= 1u << i;
  }
  const bool fast = R.groups <= 32 || R.top_groups == R.groups;
  for (int t = blockIdx.x * kScoredWarps + w; t < T; t += gridDim.x * kScoredWarps) {
    const float* row = logits + (size_t)t * E;
    int e = 0;
    double s = 0.0;
    bool ok = fast && scored_token_fast<NK, SOFTMAX, BIAS>(row, E, k, R, lane, vmask, bias,
                                                           reinterpret_cast<float*>(key), C, e, s);
    if (!ok) {
      __syncwarp();
      ok = scored_token_slow(row, bias, E, k, R, lane, key, e, s);
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

// One warp per token.  The row of grad_logits is built in shared memory and
// written once: it is zero outside the chosen experts except with the full
// softmax.  Store-bound: 4E bytes a token.
__global__ void __launch_bounds__(kBackWarps * 32)
    route_scored_backward_kernel(const float* __restrict__ logits, const int32_t* __restrict__ ids,
                                 const float* __restrict__ grad_gates, int T, int E, int k,
                                 ScoreRule R, float* __restrict__ grad_logits, int vec,
                                 WsHeader* hdr) {
  extern __shared__ float4 sback[];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int words = (E + 3) / 4 * 4;
  float* srow = reinterpret_cast<float*>(sback) + (size_t)w * words;
  const bool dense = R.softmax && !R.renorm;
  for (int t = blockIdx.x * kBackWarps + w; t < T; t += gridDim.x * kBackWarps) {
    const float* row = logits + (size_t)t * E;
    int e = -1;
    float up = 0.0f;
    if (lane < k) {
      e = __ldg(ids + (size_t)t * k + lane);
      up = (float)((double)__ldg(grad_gates + (size_t)t * k + lane) * R.scale);
      if ((unsigned)e >= (unsigned)E) {
        report(hdr, MOE_ERR_DEVICE_RANGE, e);
        e = -1;
        up = 0.0f;
      }
    }
    float d = 0.0f;    // this slot's part of the gradient at its expert
    float dot = 0.0f;  // dense: sum of up * p over the chosen
    float m = 0.0f, inv = 1.0f;
    if (R.softmax) {
      // the maximum and the sum over all experts (dense) or the chosen ones
      m = -INFINITY;
      if (dense) {
        for (int i = lane; i < E; i += 32) {
          const float l = __ldg(row + i);
          srow[i] = l;
          m = fmaxf(m, l);
        }
      } else if (e >= 0) {
        m = __ldg(row + e);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
      float sum = 0.0f;
      if (dense) {
        for (int i = lane; i < E; i += 32) {
          const float p = expf(srow[i] - m);
          srow[i] = p;
          sum += p;
        }
        __syncwarp();
      } else if (e >= 0) {
        sum = expf(__ldg(row + e) - m);
      }
      const float own = sum;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
      inv = 1.0f / sum;
      const float p = dense ? (e >= 0 ? srow[e] * inv : 0.0f) : own * inv;
      dot = up * p;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
      d = dense ? up * p : p * (up - dot);
      __syncwarp();
    } else {
      float s = 0.0f, c = 0.0f;  // sigmoid(l) and 1 - sigmoid(l), both without cancellation
      if (e >= 0) {
        const float l = __ldg(row + e);
        const float x = expf(-fabsf(l));
        const float big = 1.0f / (1.0f + x), small = x * big;
        s = l >= 0.0f ? big : small;
        c = l >= 0.0f ? small : big;
      }
      d = up;
      if (R.renorm) {
        float sum = s, us = up * s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          sum += __shfl_xor_sync(kFull, sum, o);
          us += __shfl_xor_sync(kFull, us, o);
        }
        d = sum > 0.0f ? (up - us / sum) / sum : 0.0f;
      }
      d = e >= 0 ? d * s * c : 0.0f;
    }
    // an expert that appears in several slots gets the sum of their parts, in
    // slot order, from its first slot
    const unsigned same = __match_any_sync(kFull, e);
    if (__any_sync(kFull, e >= 0 && __popc(same) > 1)) {
      float sum = 0.0f;
      for (int j = 0; j < k; ++j) {
        const float dj = __shfl_sync(kFull, d, j);
        if ((same >> j) & 1u) sum += dj;
      }
      d = sum;
      if (lane != __ffs(same) - 1) e = -1;
    }
    if (dense) {
      for (int i = lane; i < E; i += 32) srow[i] = -(srow[i] * inv) * dot;
    } else {
      for (int i = lane; i < E; i += 32) srow[i] = 0.0f;
    }
    __syncwarp();
    if (e >= 0) srow[e] += d;
    __syncwarp();
    float* out = grad_logits + (size_t)t * E;
    if (vec) {
      for (int i = lane; i < E / 4; i += 32)
        __stcs(reinterpret_cast<float4*>(out) + i, reinterpret_cast<const float4*>(srow)[i]);
    } else {
      for (int i = lane; i < E; i += 32) out[i] = srow[i];
    }
    __syncwarp();
  }
}

}  // namespace

namespace {

using ScoredKernel = void (*)(const float*, const float*, int, int, int, ScoreRule, int32_t*, float*,
                              WsHeader*);

template <int NK>
ScoredKernel scored_kernel(bool softmax, bool bias) {
  if (softmax)
    return bias ? route_scored_kernel<NK, true, true> : route_scored_kernel<NK, true, false>;
  return bias ? route_scored_kernel<NK, false, true> : route_scored_kernel<NK, false, false>;
}

}  // namespace

cudaError_t launch_route_scored(const LaunchEnv& env, const float* logits, const float* bias, int T,
                                int E, int k, const ScoreRule& rule, int32_t* ids, float* gates,
                                WsHeader* hdr) {
  const bool softmax = rule.softmax != 0, has_bias = bias != nullptr;
  const ScoredKernel kernel = E <= 64    ? scored_kernel<2>(softmax, has_bias)
                              : E <= 128 ? scored_kernel<4>(softmax, has_bias)
                              : E <= 256 ? scored_kernel<8>(softmax, has_bias)
                              : E <= 512 ? scored_kernel<16>(softmax, has_bias)
                                         : scored_kernel<32>(softmax, has_bias);
  const size_t smem = kScoredWarps * (sizeof(double) * (size_t)E + sizeof(CandArea));
  int per_sm = 1;
  cudaError_t err = blocks_per_sm((const void*)kernel, kScoredWarps * 32, smem, &per_sm);
  if (err != cudaSuccess) return err;
  int64_t grid = ((int64_t)T + kScoredWarps - 1) / kScoredWarps;
  if (grid > (int64_t)per_sm * env.num_sms) grid = (int64_t)per_sm * env.num_sms;
  return launch_pdl(env, kernel, dim3((unsigned)grid), dim3(kScoredWarps * 32), smem, logits, bias,
                    T, E, k, rule, ids, gates, hdr);
}

cudaError_t launch_route_scored_backward(const LaunchEnv& env, const float* logits,
                                         const int32_t* ids, const float* grad_gates, int T, int E,
                                         int k, const ScoreRule& rule, float* grad_logits,
                                         WsHeader* hdr) {
  const size_t smem = sizeof(float) * kBackWarps * (size_t)((E + 3) / 4 * 4);
  int per_sm = 1;
  cudaError_t err =
      blocks_per_sm((const void*)route_scored_backward_kernel, kBackWarps * 32, smem, &per_sm);
  if (err != cudaSuccess) return err;
  int64_t grid = ((int64_t)T + kBackWarps - 1) / kBackWarps;
  if (grid > (int64_t)per_sm * env.num_sms) grid = (int64_t)per_sm * env.num_sms;
  const int vec = (E % 4) == 0 && (reinterpret_cast<uintptr_t>(grad_logits) % 16) == 0;
  return launch_pdl(env, route_scored_backward_kernel, dim3((unsigned)grid), dim3(kBackWarps * 32),
                    smem, logits, ids, grad_gates, T, E, k, rule, grad_logits, vec, hdr);
}

}  // namespace moe
