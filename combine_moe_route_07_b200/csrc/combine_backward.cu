// combine_backward.cu -- gradients of the combine's operands.
//
// out[t] = sum_j gates[t,j] * y[dst_pos[t,j]] (+ shared[t] + residual[t]), so
//   grad_y[dst_pos[t,j]] = bf16(gates[t,j] * grad_out[t])
//   grad_gates[t,j]      = <grad_out[t], y[dst_pos[t,j]]>   (0 for a dropped slot)
// and the shared and residual gradients are grad_out itself.
//
// One CTA per token: its threads split the row, each holding the partial sums of
// eight slots (more slots take further passes over grad_out's row, which stays in
// the L2); the partial sums meet in a fixed order (a shuffle tree, then the warps in
// order), so results do not depend on scheduling.  No contraction to feed tensor
// cores: bound by HBM, 2H + 4Hk bytes a token.  Prefill (4096 x 4096, k 8): 571 MB in
// 98 us, 5.8 TB/s of the 6.54 TB/s of a copy.
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kMaxThreads = 512;

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

constexpr int kMaxSlots = 32;

template <int KB>
__global__ void __launch_bounds__(kMaxThreads)
    combine_backward_kernel(const void* __restrict__ grad_out, const void* __restrict__ y,
                            const int32_t* __restrict__ dst_pos, const float* __restrict__ gates,
                            int T, int H, int k, int64_t N, void* __restrict__ grad_y,
                            float* __restrict__ grad_gates, WsHeader* hdr) {
  __shared__ int32_t s_row[kMaxSlots];
  __shared__ float s_gate[kMaxSlots];
  __shared__ float s_part[kMaxThreads / 32][kMaxSlots];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int chunks = H / 8;
  for (int t = blockIdx.x; t < T; t += gridDim.x) {
    if (threadIdx.x < kMaxSlots) {
      int r = -1;
      float g = 0.0f;
      if ((int)threadIdx.x < k) {
        r = __ldg(dst_pos + (size_t)t * k + threadIdx.x);
        g = __ldg(gates + (size_t)t * k + threadIdx.x);
        if (r >= N) {
          report(hdr, MOE_ERR_DEVICE_RANGE, r);
          r = -1;
        }
      }
      s_row[threadIdx.x] = r;
      s_gate[threadIdx.x] = g;
    }
    __syncthreads();
    const char* orow = static_cast<const char*>(grad_out) + (size_t)t * H * 2;
    for (int j0 = 0; j0 < k; j0 += KB) {
      float acc[KB];
#pragma unroll
      for (int j = 0; j < KB; ++j) acc[j] = 0.0f;
      for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
        const uint4 o = ld16_stream(orow + (size_t)c * 16);
        const uint32_t ow[4] = {o.x, o.y, o.z, o.w};
        uint4 v[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j)
          if (s_row[j0 + j] >= 0)
            v[j] = ld16_stream(static_cast<const char*>(y) + (size_t)s_row[j0 + j] * H * 2 +
                               (size_t)c * 16);
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          if (s_row[j0 + j] < 0) continue;
          const uint32_t yw[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
          const float g = s_gate[j0 + j];
          uint32_t dw[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            acc[j] = fmaf(bf16lo(ow[q]), bf16lo(yw[q]), acc[j]);
            acc[j] = fmaf(bf16hi(ow[q]), bf16hi(yw[q]), acc[j]);
            dw[q] = pack_bf16x2(g * bf16lo(ow[q]), g * bf16hi(ow[q]));
          }
          st16(static_cast<char*>(grad_y) + (size_t)s_row[j0 + j] * H * 2 + (size_t)c * 16,
               make_uint4(dw[0], dw[1], dw[2], dw[3]));
        }
      }
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        float a = acc[j];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(kFull, a, o);
        if (lane == 0) s_part[w][j0 + j] = a;
      }
    }
    __syncthreads();
    if ((int)threadIdx.x < k) {
      float a = 0.0f;
      for (int i = 0; i < (int)blockDim.x / 32; ++i) a += s_part[i][threadIdx.x];
      grad_gates[(size_t)t * k + threadIdx.x] = s_row[threadIdx.x] >= 0 ? a : 0.0f;
    }
    __syncthreads();
  }
}

template <int KB>
cudaError_t launch_k(const LaunchEnv& env, const void* grad_out, const void* y,
                     const int32_t* dst_pos, const float* gates, int T, int H, int k, int64_t N,
                     void* grad_y, float* grad_gates, WsHeader* hdr) {
  // 128 threads a token, which leaves many tokens in flight; batches too small to fill
  // the SMs with those split a row over more threads (130 tokens of 7168: 12.3 us with
  // 128 threads, 8.5 with 512)
  int threads = 128;
  while (threads < kMaxThreads && threads * 8 < H &&
         (int64_t)T * threads < (int64_t)env.num_sms * 1024)
    threads *= 2;
  int per_sm = 1;
  cudaError_t err = blocks_per_sm((const void*)combine_backward_kernel<KB>, threads, 0, &per_sm);
  if (err != cudaSuccess) return err;
  int64_t grid = T;
  if (grid > (int64_t)per_sm * env.num_sms) grid = (int64_t)per_sm * env.num_sms;
  return launch_pdl(env, combine_backward_kernel<KB>, dim3((unsigned)grid), dim3(threads), 0,
                    grad_out, y, dst_pos, gates, T, H, k, N, grad_y, grad_gates, hdr);
}

}  // namespace

cudaError_t launch_combine_backward(const LaunchEnv& env, const void* grad_out, const void* y,
                                    const int32_t* dst_pos, const float* gates, int T, int H, int k,
                                    int64_t N, void* grad_y, float* grad_gates, WsHeader* hdr) {
  if (k <= 4)
    return launch_k<4>(env, grad_out, y, dst_pos, gates, T, H, k, N, grad_y, grad_gates, hdr);
  return launch_k<8>(env, grad_out, y, dst_pos, gates, T, H, k, N, grad_y, grad_gates, hdr);
}

}  // namespace moe
