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
// that differ onto one value.
#include <math.h>

#include "common.cuh"
#include "kernels.h"

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
  return softmax ? exp(l - m) * inv_sum : 1.0 / (1.0 + exp(-l));
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
    s = sum > 0.0 ? s / sum : 0.0;
  }
  return (float)(s * scale);
}

__global__ void __launch_bounds__(kScoredWarps * 32)
    route_scored_kernel(const float* __restrict__ logits, const float* __restrict__ bias, int T,
                        int E, int k, ScoreRule R, int32_t* __restrict__ ids,
                        float* __restrict__ gates, WsHeader* hdr) {
  extern __shared__ double skey[];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  double* key = skey + (size_t)w * E;
  for (int t = blockIdx.x * kScoredWarps + w; t < T; t += gridDim.x * kScoredWarps) {
    int e = 0;
    double s = 0.0;
    const bool ok = scored_token_exact(logits + (size_t)t * E, bias, E, k, R, lane, key, e, s);
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

cudaError_t launch_route_scored(const LaunchEnv& env, const float* logits, const float* bias, int T,
                                int E, int k, const ScoreRule& rule, int32_t* ids, float* gates,
                                WsHeader* hdr) {
  const size_t smem = sizeof(double) * kScoredWarps * (size_t)E;
  int per_sm = 1;
  cudaError_t err = blocks_per_sm((const void*)route_scored_kernel, kScoredWarps * 32, smem, &per_sm);
  if (err != cudaSuccess) return err;
  int64_t grid = ((int64_t)T + kScoredWarps - 1) / kScoredWarps;
  if (grid > (int64_t)per_sm * env.num_sms) grid = (int64_t)per_sm * env.num_sms;
  return launch_pdl(env, route_scored_kernel, dim3((unsigned)grid), dim3(kScoredWarps * 32), smem,
                    logits, bias, T, E, k, rule, ids, gates, hdr);
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
