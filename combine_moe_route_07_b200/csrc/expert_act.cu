// expert_act.cu -- the gradient through an expert product's activation, and
// the bias gradient.
//
//   dz[p,:] = dy[p,:] * act'(z[p,:])     (swiglu: both halves of z)
//   db_e    = sum over the rows p of expert e of dz[p,:]
//
// z is read as the forward wrote it (bf16) and dz is rounded to bf16 once, the
// operand type of the two products that read it; db sums dz before that
// rounding, in fp32.  Bound by HBM (2F + 4W bytes a row with an activation).
// Each CTA takes tiles of 64 rows of one expert and leaves their column sums in
// a scratch table; a second kernel adds an expert's tiles in a fixed order, so
// the sums do not depend on scheduling.
#include <math.h>

#include "block_scan.cuh"
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct ActParams {
  const uint16_t* dy;
  const uint16_t* z;
  uint16_t* dz;      // NULL: dz is dy itself
  float* partial;    // [tiles][W] or NULL
  int32_t* tile_of;  // with partial: first tile of each expert [E+1]
  const int32_t* counts;
  const int32_t* off;
  WsHeader* hdr;
  int64_t N, max_rows;
  int E, capacity, F, W;
};

__device__ __forceinline__ int seg_rows(const ActParams& P, int e, int* off) {
  if (P.counts == nullptr) {
    *off = 0;
    return (int)P.N;
  }
  int o = __ldg(P.off + e), r = __ldg(P.counts + e);
  if (P.capacity > 0 && r > P.capacity) r = P.capacity;
  if (r <= 0 || o < 0 || (int64_t)o + r > P.N) {
    if (r != 0 && blockIdx.x == 0) report(P.hdr, MOE_ERR_DEVICE_RANGE, e);
    r = 0;
    o = 0;
  }
  *off = o;
  return r;
}

// Slope of the activation at z (gelu: Phi(z) + z phi(z)).
template <int ACT>
__device__ __forceinline__ float slope(float z) {
  if (ACT == MOE_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
  if (ACT == MOE_ACT_GELU) {
    float e;
    const float tail = normal_tail(z, &e);
    return fmaf(z * 0.39894228f, e, z < 0.0f ? tail : 1.0f - tail);
  }
  if (ACT == MOE_ACT_SILU || ACT == MOE_ACT_SWIGLU) {
    const float s = sigmoid_f(z);
    return s * fmaf(z, 1.0f - s, 1.0f);
  }
  return 1.0f;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16lo(w[i]);
    f[2 * i + 1] = bf16hi(w[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int kUnroll = 2;  // rows of a warp whose loads are in flight together

template <int ACT>
__global__ void __launch_bounds__(kThreads, 4)
    expert_act_backward_kernel(ActParams P) {
  extern __shared__ int32_t tab[];
  __shared__ float red[kWarps][2][256];
  __shared__ int32_t warp_tot[kWarps];
  int32_t* off = tab;
  int32_t* rows = tab + P.E;
  int32_t* first = rows + P.E;
  __shared__ unsigned long long rows_sum;
  if (threadIdx.x == 0) rows_sum = 0ull;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  unsigned long long my_rows = 0ull;
  for (int e = threadIdx.x; e < P.E; e += kThreads) {
    int o;
    const int r = seg_rows(P, e, &o);
    off[e] = o;
    rows[e] = r;
    first[e] = (r + kActRows - 1) / kActRows;
    my_rows += (unsigned long long)r;
  }
  if (my_rows != 0ull) atomicAdd(&rows_sum, my_rows);
  __syncthreads();
  int tiles = block_exclusive_scan<kThreads>(first, P.E, warp_tot);
  if (threadIdx.x == 0) first[P.E] = tiles;
  __syncthreads();
  // more rows than assignments: not a layout's segments, and more tiles than the
  // scratch table holds
  if ((int64_t)rows_sum > P.max_rows) {
    if (threadIdx.x == 0 && blockIdx.x == 0) report(P.hdr, MOE_ERR_DEVICE_RANGE, P.E);
    tiles = 0;
  }
  if (P.partial != nullptr && blockIdx.x == 0)
    for (int e = threadIdx.x; e <= P.E; e += kThreads) P.tile_of[e] = tiles > 0 ? first[e] : 0;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int strips = (P.F + 255) / 256;  // 256 channels: 8 a lane
  constexpr bool gated = ACT == MOE_ACT_SWIGLU, plain = ACT == MOE_ACT_NONE;
  for (int64_t u = blockIdx.x; u < (int64_t)tiles * strips; u += gridDim.x) {
    const int tile = (int)(u / strips), strip = (int)(u - (int64_t)tile * strips);
    int lo = 0, hi = P.E;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= tile)
        lo = mid;
      else
        hi = mid;
    }
    const int r0 = (tile - first[lo]) * kActRows;
    const int n = min(kActRows, rows[lo] - r0);
    const int c = strip * 256 + lane * 8;
    float s0[8], s1[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s0[i] = s1[i] = 0.0f;
    if (c < P.F) {
      for (int r = w; r < n; r += kUnroll * kWarps) {
        uint4 dv[kUnroll], zv[kUnroll], uv[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
          if (r + k * kWarps < n) {
            const size_t p = (size_t)off[lo] + r0 + r + k * kWarps;
            dv[k] = ld16_stream(P.dy + p * P.F + c);
            if (!plain) zv[k] = ld16_stream(P.z + p * P.W + c);
            if (gated) uv[k] = ld16_stream(P.z + p * P.W + P.F + c);
          }
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
          if (r + k * kWarps < n) {
            const size_t p = (size_t)off[lo] + r0 + r + k * kWarps;
            float d[8], z[8];
            unpack8(dv[k], d);
            if (!plain) unpack8(zv[k], z);
            if (gated) {
              float up[8], g[8];
              unpack8(uv[k], up);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float s = sigmoid_f(z[i]);
                g[i] = d[i] * up[i] * (s * fmaf(z[i], 1.0f - s, 1.0f));
                up[i] = d[i] * (z[i] * s);
                s0[i] += g[i];
                s1[i] += up[i];
              }
              st16(P.dz + p * P.W + c, pack8(g));
              st16(P.dz + p * P.W + P.F + c, pack8(up));
            } else {
              if (!plain) {
#pragma unroll
                for (int i = 0; i < 8; ++i) d[i] *= slope<ACT>(z[i]);
                st16(P.dz + p * P.W + c, pack8(d));
              }
#pragma unroll
              for (int i = 0; i < 8; ++i) s0[i] += d[i];
            }
          }
        }
      }
    }
    if (P.partial != nullptr) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        red[w][0][lane * 8 + i] = s0[i];
        red[w][1][lane * 8 + i] = s1[i];
      }
      __syncthreads();
      const int ch = strip * 256 + threadIdx.x;
      if (ch < P.F) {
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
          a += red[i][0][threadIdx.x];
          b += red[i][1][threadIdx.x];
        }
        P.partial[(size_t)tile * P.W + ch] = a;
        if (gated) P.partial[(size_t)tile * P.W + P.F + ch] = b;
      }
      __syncthreads();
    }
  }
}

// grad_bias[e][c] = sum of expert e's partial sums: 8 warps take every 8th tile,
// then meet in warp order.  One CTA for 128 channels of one expert, four a lane.
__global__ void __launch_bounds__(kThreads)
    expert_bias_reduce_kernel(const float* __restrict__ partial, const int32_t* __restrict__ tile_of,
                              int W, float* __restrict__ grad_bias) {
  __shared__ float4 red[kWarps][32];
  pdl_wait();
  pdl_trigger();
  const int e = blockIdx.y, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 128 + lane * 4;
  const int lo = __ldg(tile_of + e), hi = __ldg(tile_of + e + 1);
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (c < W) {
#pragma unroll 4
    for (int i = lo + w; i < hi; i += kWarps) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(partial + (size_t)i * W + c));
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
  }
  red[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < W) {
    float4 a = red[0][lane];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) {
      const float4 v = red[i][lane];
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
    float* out = grad_bias + (size_t)e * W + c;
    out[0] = a.x;
    out[1] = a.y;
    out[2] = a.z;
    out[3] = a.w;
  }
}

}  // namespace

int64_t expert_act_tiles(int64_t assignments, int E) {
  return assignments / kActRows + (assignments < E ? assignments : E);
}

size_t expert_act_scratch_bytes(int64_t assignments, int E, int wide) {
  // the experts' first tiles, then the tiles' sums
  const int64_t tiles = expert_act_tiles(assignments, E);
  return (((size_t)E + 1) * sizeof(int32_t) + 15) / 16 * 16 + (size_t)tiles * wide * sizeof(float);
}

cudaError_t launch_expert_act_backward(const LaunchEnv& env, const ExpertMatmul& a, const void* dy,
                                       const void* z, void* dz, void* scratch, float* grad_bias) {
  ActParams P = {};
  P.dy = static_cast<const uint16_t*>(dy);
  P.z = static_cast<const uint16_t*>(z);
  P.dz = static_cast<uint16_t*>(dz);
  if (grad_bias != nullptr) {
    P.tile_of = static_cast<int32_t*>(scratch);
    P.partial = reinterpret_cast<float*>(static_cast<char*>(scratch) +
                                         (((size_t)a.E + 1) * sizeof(int32_t) + 15) / 16 * 16);
  }
  P.counts = a.counts;
  P.off = a.expert_off;
  P.hdr = a.hdr;
  P.N = a.N;
  P.max_rows = a.assignments;
  P.E = a.E;
  P.capacity = a.capacity;
  P.F = a.out_features;
  P.W = a.act == MOE_ACT_SWIGLU ? 2 * a.out_features : a.out_features;
  const size_t smem = sizeof(int32_t) * (3 * (size_t)P.E + 1);
  int per_sm = 1;
  void (*kernel)(ActParams) = expert_act_backward_kernel<MOE_ACT_NONE>;
  switch (a.act) {
    case MOE_ACT_RELU: kernel = expert_act_backward_kernel<MOE_ACT_RELU>; break;
    case MOE_ACT_GELU: kernel = expert_act_backward_kernel<MOE_ACT_GELU>; break;
    case MOE_ACT_SILU: kernel = expert_act_backward_kernel<MOE_ACT_SILU>; break;
    case MOE_ACT_SWIGLU: kernel = expert_act_backward_kernel<MOE_ACT_SWIGLU>; break;
  }
  cudaError_t err = blocks_per_sm((const void*)kernel, kThreads, smem, &per_sm);
  if (err != cudaSuccess) return err;
  const int64_t strips = (P.F + 255) / 256;
  int64_t grid = expert_act_tiles(a.assignments, a.E) * strips;
  if (grid > (int64_t)per_sm * env.num_sms) grid = (int64_t)per_sm * env.num_sms;
  if (grid < 1) grid = 1;
  err = launch_pdl(env, kernel, dim3((unsigned)grid), dim3(kThreads), smem, P);
  if (err != cudaSuccess || grad_bias == nullptr) return err;
  return launch_pdl(env, expert_bias_reduce_kernel,
                    dim3((unsigned)((P.W + 127) / 128), (unsigned)P.E), dim3(kThreads), 0,
                    (const float*)P.partial, (const int32_t*)P.tile_of, P.W, grad_bias);
}

}  // namespace moe
