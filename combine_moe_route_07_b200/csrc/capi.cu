// capi.cu -- the C ABI declared in include/moe_route07.h: host-side argument
// checks, workspace sizing, launch and status mapping.  No computation of the
// path happens here; every step runs in the kernels.
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "moe_route07.h"

namespace {

using moe::WsHeader;

constexpr size_t kHeaderBytes = sizeof(WsHeader);

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Host-side check of a shape; the limits keep every index in 32 bits.
bool shape_ok(const moe_shape_t* s) {
  if (s == nullptr) return false;
  const int64_t T = s->tokens, H = s->hidden, E = s->experts, k = s->k, R = s->ranks;
  if (T < 0 || H < 8 || (H % 8) != 0) return false;
  if ((s->flags & ~(MOE_F_RENORM | MOE_F_FP8 | MOE_F_SRC_LAYOUT)) != 0u) return false;
  if ((s->flags & MOE_F_FP8) && (H % 128) != 0) return false;
  if (E < 1 || E > 1024 || R < 1 || (E % R) != 0) return false;
  if (k < 1 || k > E || k > 32) return false;
  if (s->capacity < 0 || s->align < 1 || s->align > (1 << 20)) return false;
  if (s->capacity > 0 && s->align != 1) return false;
  if (T * k >= (int64_t(1) << 30)) return false;
  const int64_t segs = (s->flags & MOE_F_SRC_LAYOUT) ? R * E : E;  // R*E <= 2^20
  const int64_t rows = s->capacity > 0 ? segs * s->capacity : T * k + segs * (s->align - 1);
  if (rows >= (int64_t(1) << 31)) return false;
  if (T * (H / 8) >= (int64_t(1) << 31)) return false;
  return true;
}

bool src_layout(const moe_shape_t* s) { return (s->flags & MOE_F_SRC_LAYOUT) != 0u; }

int64_t rows_of(const moe_shape_t* s) {
  const int64_t segs = src_layout(s) ? int64_t(s->ranks) * s->experts : int64_t(s->experts);
  return s->capacity > 0 ? segs * s->capacity
                         : int64_t(s->tokens) * s->k + segs * (s->align - 1);
}

// Workspace: header, then two tile tables of equal size (words a multiple of
// 4); for the per-source-rank layout, header + part counts + kept prefix.
size_t ws_bytes_of(const moe_shape_t* s) {
  if (src_layout(s))
    return kHeaderBytes + (moe::layout_src_part_words(s->tokens, s->experts, s->ranks) +
                           moe::layout_src_cum_words(s->experts, s->ranks)) *
                              sizeof(int32_t);
  const size_t words = (moe::layout_table_words(s->tokens, s->experts) + 3) / 4 * 4;
  return kHeaderBytes + 2 * words * sizeof(uint32_t);
}

size_t half_words_of(size_t ws_bytes) { return ((ws_bytes - kHeaderBytes) / 8) / 4 * 4; }

moe_status_t ws_ok(const moe_shape_t* s, void* ws, size_t ws_bytes) {
  if (ws == nullptr || !aligned(ws, 16)) return MOE_ERR_WORKSPACE;
  if (ws_bytes < ws_bytes_of(s)) return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

int sm_count() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (dev >= 0 && dev < 64 && cached[dev] > 0) return cached[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
    n = 148;
  if (dev >= 0 && dev < 64) cached[dev] = n;
  return n;
}

moe::LaunchEnv env_of(moe_stream_t stream) {
  moe::LaunchEnv env;
  env.stream = reinterpret_cast<cudaStream_t>(stream);
  env.num_sms = sm_count();
  return env;
}

moe_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

}  // namespace

extern "C" {

int32_t moe_abi_version(void) { return MOE_ABI_VERSION; }

const char* moe_status_string(moe_status_t s) {
  switch (s) {
    case MOE_OK: return "ok";
    case MOE_ERR_INVALID_ARG: return "invalid argument";
    case MOE_ERR_UNSUPPORTED: return "unsupported";
    case MOE_ERR_WORKSPACE: return "workspace missing, misaligned, too small or not zeroed";
    case MOE_ERR_CUDA: return "CUDA runtime error";
    case MOE_ERR_DEVICE_RANGE: return "device: index out of range";
    case MOE_ERR_DEVICE_TIMEOUT: return "device: bounded wait gave up";
    case MOE_ERR_DEVICE_NAN: return "device: NaN routing key";
  }
  return "unknown status";
}

int64_t moe_layout_rows(const moe_shape_t* shape) {
  if (!shape_ok(shape)) return -1;
  return rows_of(shape);
}

size_t moe_workspace_bytes(const moe_shape_t* shape) {
  if (!shape_ok(shape)) return 0;
  return ws_bytes_of(shape);
}

moe_status_t moe_workspace_init(void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (ws == nullptr || !aligned(ws, 16) || ws_bytes < kHeaderBytes) return MOE_ERR_WORKSPACE;
  return from_cuda(cudaMemsetAsync(ws, 0, ws_bytes, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_route(const moe_shape_t* shape, const float* logits, const float* bias,
                       int32_t* ids, float* gates, void* ws, size_t ws_bytes,
                       moe_stream_t stream) {
  if (!shape_ok(shape)) return MOE_ERR_INVALID_ARG;
  if (shape->tokens > 0 && (logits == nullptr || ids == nullptr || gates == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(logits, 4) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(gates, 4))
    return MOE_ERR_INVALID_ARG;
  moe_status_t st = ws_ok(shape, ws, ws_bytes);
  if (st != MOE_OK) return st;
  if (shape->tokens == 0) return MOE_OK;
  return from_cuda(moe::launch_route(env_of(stream), logits, bias, shape->tokens,
                                     shape->experts, shape->k,
                                     (shape->flags & MOE_F_RENORM) ? 1 : 0, ids, gates,
                                     static_cast<WsHeader*>(ws)));
}

moe_status_t moe_route_limited(const moe_shape_t* shape, const float* logits, const float* bias,
                               int32_t max_ranks, int32_t* ids, float* gates, void* ws,
                               size_t ws_bytes, moe_stream_t stream) {
  if (!shape_ok(shape) || max_ranks < 1) return MOE_ERR_INVALID_ARG;
  const int R = shape->ranks, Er = shape->experts / shape->ranks;
  if (max_ranks < R && shape->k > (int64_t)max_ranks * Er) return MOE_ERR_INVALID_ARG;
  if (shape->tokens > 0 && (logits == nullptr || ids == nullptr || gates == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(logits, 4) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(gates, 4))
    return MOE_ERR_INVALID_ARG;
  moe_status_t st = ws_ok(shape, ws, ws_bytes);
  if (st != MOE_OK) return st;
  if (shape->tokens == 0) return MOE_OK;
  return from_cuda(moe::launch_route(env_of(stream), logits, bias, shape->tokens,
                                     shape->experts, shape->k,
                                     (shape->flags & MOE_F_RENORM) ? 1 : 0, ids, gates,
                                     static_cast<WsHeader*>(ws), nullptr, 0, R,
                                     max_ranks < R ? max_ranks : 0));
}

moe_status_t moe_layout_remote_first(const moe_shape_t* shape, const int32_t* ids,
                                     int32_t home_rank, int32_t* counts, int32_t* expert_off,
                                     int32_t* rank_off, int32_t* rank_counts, int32_t* dst_pos,
                                     int32_t* src_idx, int32_t* tile_expert, void* ws,
                                     size_t ws_bytes, moe_stream_t stream) {
  if (!shape_ok(shape) || src_layout(shape)) return MOE_ERR_INVALID_ARG;
  if (home_rank < 0 || home_rank >= shape->ranks) return MOE_ERR_INVALID_ARG;
  const int64_t N = rows_of(shape);
  if (counts == nullptr || expert_off == nullptr || rank_off == nullptr ||
      rank_counts == nullptr)
    return MOE_ERR_INVALID_ARG;
  if (shape->tokens > 0 && (ids == nullptr || dst_pos == nullptr)) return MOE_ERR_INVALID_ARG;
  if (N > 0 && src_idx == nullptr) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {ids, counts, expert_off, rank_off, rank_counts, dst_pos, src_idx,
                        tile_expert};
  for (const void* p : ptrs)
    if (!aligned(p, 4)) return MOE_ERR_INVALID_ARG;
  moe_status_t st = ws_ok(shape, ws, ws_bytes);
  if (st != MOE_OK) return st;
  WsHeader* hdr = static_cast<WsHeader*>(ws);
  uint32_t* tables = reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + kHeaderBytes);
  return from_cuda(moe::launch_layout(env_of(stream), ids, shape->tokens, shape->experts,
                                      shape->k, shape->ranks, shape->capacity, shape->align, N,
                                      tables, half_words_of(ws_bytes), hdr, counts, expert_off,
                                      rank_off, rank_counts, dst_pos, src_idx, true, home_rank,
                                      tile_expert));
}

moe_status_t moe_route_round_robin(const moe_shape_t* shape, int32_t* ids, float* gates,
                                   moe_stream_t stream) {
  if (!shape_ok(shape)) return MOE_ERR_INVALID_ARG;
  if (shape->tokens > 0 && (ids == nullptr || gates == nullptr)) return MOE_ERR_INVALID_ARG;
  if (!aligned(ids, 4) || !aligned(gates, 4)) return MOE_ERR_INVALID_ARG;
  if (shape->tokens == 0) return MOE_OK;
  return from_cuda(moe::launch_route_round_robin(env_of(stream), shape->tokens, shape->experts,
                                                 shape->k, ids, gates));
}

moe_status_t moe_bias_update(const moe_shape_t* shape, const int32_t* counts, float gamma,
                             float* bias, moe_stream_t stream) {
  if (!shape_ok(shape) || counts == nullptr || bias == nullptr) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(gamma) || gamma < 0.0f) return MOE_ERR_INVALID_ARG;
  if (!aligned(counts, 4) || !aligned(bias, 4)) return MOE_ERR_INVALID_ARG;
  return from_cuda(moe::launch_bias_update(env_of(stream), counts, shape->experts,
                                           int64_t(shape->tokens) * shape->k, gamma, bias));
}

moe_status_t moe_layout(const moe_shape_t* shape, const int32_t* ids, int32_t* counts,
                        int32_t* expert_off, int32_t* rank_off, int32_t* rank_counts,
                        int32_t* dst_pos, int32_t* src_idx, void* ws, size_t ws_bytes,
                        moe_stream_t stream) {
  if (!shape_ok(shape) || src_layout(shape)) return MOE_ERR_INVALID_ARG;
  const int64_t N = rows_of(shape);
  if (counts == nullptr || expert_off == nullptr || rank_off == nullptr ||
      rank_counts == nullptr)
    return MOE_ERR_INVALID_ARG;
  if (shape->tokens > 0 && (ids == nullptr || dst_pos == nullptr)) return MOE_ERR_INVALID_ARG;
  if (N > 0 && src_idx == nullptr) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {ids, counts, expert_off, rank_off, rank_counts, dst_pos, src_idx};
  for (const void* p : ptrs)
    if (!aligned(p, 4)) return MOE_ERR_INVALID_ARG;
  moe_status_t st = ws_ok(shape, ws, ws_bytes);
  if (st != MOE_OK) return st;
  WsHeader* hdr = static_cast<WsHeader*>(ws);
  uint32_t* tables = reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + kHeaderBytes);
  return from_cuda(moe::launch_layout(env_of(stream), ids, shape->tokens, shape->experts,
                                      shape->k, shape->ranks, shape->capacity, shape->align, N,
                                      tables, half_words_of(ws_bytes), hdr, counts, expert_off,
                                      rank_off, rank_counts, dst_pos, src_idx, true));
}

moe_status_t moe_layout_src(const moe_shape_t* shape, const int32_t* ids, int32_t* src_counts,
                            int32_t* seg_off, int32_t* pair_counts, int32_t* rank_off,
                            int32_t* rank_counts, int32_t* dst_pos, int32_t* src_idx, void* ws,
                            size_t ws_bytes, moe_stream_t stream) {
  if (!shape_ok(shape) || !src_layout(shape)) return MOE_ERR_INVALID_ARG;
  const int64_t N = rows_of(shape);
  if (src_counts == nullptr || seg_off == nullptr || pair_counts == nullptr ||
      rank_off == nullptr || rank_counts == nullptr)
    return MOE_ERR_INVALID_ARG;
  if (shape->tokens > 0 && (ids == nullptr || dst_pos == nullptr)) return MOE_ERR_INVALID_ARG;
  if (N > 0 && src_idx == nullptr) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {ids, src_counts, seg_off, pair_counts, rank_off, rank_counts, dst_pos,
                        src_idx};
  for (const void* p : ptrs)
    if (!aligned(p, 4)) return MOE_ERR_INVALID_ARG;
  moe_status_t st = ws_ok(shape, ws, ws_bytes);
  if (st != MOE_OK) return st;
  WsHeader* hdr = static_cast<WsHeader*>(ws);
  int32_t* partc = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + kHeaderBytes);
  int32_t* scratch =
      partc + moe::layout_src_part_words(shape->tokens, shape->experts, shape->ranks);
  return from_cuda(moe::launch_layout_src(env_of(stream), ids, shape->tokens, shape->experts,
                                          shape->k, shape->ranks, shape->capacity, shape->align,
                                          N, partc, scratch, hdr, src_counts, seg_off,
                                          pair_counts, rank_off, rank_counts, dst_pos,
                                          src_idx));
}

}  // extern "C"

namespace {

// The argument checks of moe_route_layout (and of the route and layout part of
// moe_route_layout_dispatch).
moe_status_t route_layout_args_ok(const moe_shape_t* shape, const float* logits, const float* bias,
                                  int32_t* ids, float* gates, int32_t* counts,
                                  int32_t* expert_off, int32_t* rank_off, int32_t* rank_counts,
                                  int32_t* dst_pos, int32_t* src_idx, void* ws, size_t ws_bytes) {
  if (!shape_ok(shape) || src_layout(shape)) return MOE_ERR_INVALID_ARG;
  const int64_t N = rows_of(shape);
  if (counts == nullptr || expert_off == nullptr || rank_off == nullptr ||
      rank_counts == nullptr)
    return MOE_ERR_INVALID_ARG;
  if (shape->tokens > 0 && (logits == nullptr || ids == nullptr || gates == nullptr ||
                            dst_pos == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (N > 0 && src_idx == nullptr) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {logits, bias, ids, gates, counts, expert_off, rank_off, rank_counts,
                        dst_pos, src_idx};
  for (const void* p : ptrs)
    if (!aligned(p, 4)) return MOE_ERR_INVALID_ARG;
  return ws_ok(shape, ws, ws_bytes);
}

}  // namespace

extern "C" {

moe_status_t moe_route_layout(const moe_shape_t* shape, const float* logits, const float* bias,
                              int32_t* ids, float* gates, int32_t* counts, int32_t* expert_off,
                              int32_t* rank_off, int32_t* rank_counts, int32_t* dst_pos,
                              int32_t* src_idx, void* ws, size_t ws_bytes, moe_stream_t stream) {
  const moe_status_t st = route_layout_args_ok(shape, logits, bias, ids, gates, counts,
                                               expert_off, rank_off, rank_counts, dst_pos,
                                               src_idx, ws, ws_bytes);
  if (st != MOE_OK) return st;
  const int64_t N = rows_of(shape);
  WsHeader* hdr = static_cast<WsHeader*>(ws);
  uint32_t* tables = reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + kHeaderBytes);
  const size_t half = half_words_of(ws_bytes);
  const moe::LaunchEnv env = env_of(stream);
  if (moe::route_layout_small_fits(shape->tokens, shape->experts, shape->k))
    return from_cuda(moe::launch_route_layout_small(
        env, logits, bias, shape->tokens, shape->experts, shape->k, shape->ranks,
        (shape->flags & MOE_F_RENORM) ? 1 : 0, shape->capacity, shape->align, N, hdr, ids, gates,
        counts, expert_off, rank_off, rank_counts, dst_pos, src_idx));
  if (shape->tokens > 0) {
    const cudaError_t err = moe::launch_route(env, logits, bias, shape->tokens, shape->experts,
                                              shape->k, (shape->flags & MOE_F_RENORM) ? 1 : 0,
                                              ids, gates, hdr, tables, half);
    if (err != cudaSuccess) return MOE_ERR_CUDA;
  }
  return from_cuda(moe::launch_layout(env, ids, shape->tokens, shape->experts, shape->k,
                                      shape->ranks, shape->capacity, shape->align, N, tables, half,
                                      hdr, counts, expert_off, rank_off, rank_counts, dst_pos,
                                      src_idx, false));
}

moe_status_t moe_route_layout_dispatch(const moe_shape_t* shape, const float* logits,
                                       const float* bias, const void* x, int32_t* ids,
                                       float* gates, int32_t* counts, int32_t* expert_off,
                                       int32_t* rank_off, int32_t* rank_counts, int32_t* dst_pos,
                                       int32_t* src_idx, void* out, float* scales, void* ws,
                                       size_t ws_bytes, moe_stream_t stream) {
  if (!shape_ok(shape) || src_layout(shape)) return MOE_ERR_INVALID_ARG;
  const bool fp8 = (shape->flags & MOE_F_FP8) != 0u;
  if (shape->tokens > 0 && (x == nullptr || out == nullptr || (fp8 && scales == nullptr)))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(scales, 4)) return MOE_ERR_INVALID_ARG;
  const int T = shape->tokens, E = shape->experts, k = shape->k, H = shape->hidden;
  if (!fp8 && T > 0 && !moe::route_layout_small_fits(T, E, k)) {
    const moe::LaunchEnv env = env_of(stream);
    if (moe::place_dispatch_fits(T, E, k, H, shape->capacity, env.num_sms)) {
      // the route kernel fills the tile table; one kernel places and streams the rows
      const moe_status_t sa = route_layout_args_ok(shape, logits, bias, ids, gates, counts,
                                                   expert_off, rank_off, rank_counts, dst_pos,
                                                   src_idx, ws, ws_bytes);
      if (sa != MOE_OK) return sa;
      WsHeader* hdr = static_cast<WsHeader*>(ws);
      uint32_t* tables = reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + kHeaderBytes);
      const size_t half = half_words_of(ws_bytes);
      const cudaError_t err =
          moe::launch_route(env, logits, bias, T, E, k, (shape->flags & MOE_F_RENORM) ? 1 : 0,
                            ids, gates, hdr, tables, half);
      if (err != cudaSuccess) return MOE_ERR_CUDA;
      return from_cuda(moe::launch_place_dispatch(
          env, ids, x, T, H, E, k, shape->ranks, shape->align, rows_of(shape), tables, half, hdr,
          counts, expert_off, rank_off, rank_counts, dst_pos, src_idx, out));
    }
  }
  moe_status_t st = moe_route_layout(shape, logits, bias, ids, gates, counts, expert_off,
                                     rank_off, rank_counts, dst_pos, src_idx, ws, ws_bytes,
                                     stream);
  if (st != MOE_OK || shape->tokens == 0) return st;
  const moe::LaunchEnv env = env_of(stream);
  WsHeader* hdr = static_cast<WsHeader*>(ws);
  const int64_t N = rows_of(shape);
  if (fp8)
    return from_cuda(moe::launch_dispatch_fp8(env, x, dst_pos, shape->tokens, shape->hidden,
                                              shape->k, N, out, scales, hdr));
  return from_cuda(moe::launch_dispatch_bf16(env, x, dst_pos, shape->tokens, shape->hidden,
                                             shape->k, N, out, hdr, true));
}

moe_status_t moe_dispatch(const moe_shape_t* shape, const void* x, const int32_t* dst_pos,
                          void* out, float* scales, void* ws, size_t ws_bytes,
                          moe_stream_t stream) {
  if (!shape_ok(shape)) return MOE_ERR_INVALID_ARG;
  const bool fp8 = (shape->flags & MOE_F_FP8) != 0u;
  if (shape->tokens > 0 && (x == nullptr || dst_pos == nullptr || out == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (fp8 && shape->tokens > 0 && scales == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(dst_pos, 4) || !aligned(scales, 4))
    return MOE_ERR_INVALID_ARG;
  moe_status_t st = ws_ok(shape, ws, ws_bytes);
  if (st != MOE_OK) return st;
  if (shape->tokens == 0) return MOE_OK;
  const moe::LaunchEnv env = env_of(stream);
  WsHeader* hdr = static_cast<WsHeader*>(ws);
  const int64_t N = rows_of(shape);
  if (fp8)
    return from_cuda(moe::launch_dispatch_fp8(env, x, dst_pos, shape->tokens, shape->hidden,
                                              shape->k, N, out, scales, hdr));
  return from_cuda(moe::launch_dispatch_bf16(env, x, dst_pos, shape->tokens, shape->hidden,
                                             shape->k, N, out, hdr));
}

moe_status_t moe_combine(const moe_shape_t* shape, const void* y, const int32_t* dst_pos,
                         const float* gates, const void* shared, const void* residual,
                         void* out, void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (!shape_ok(shape)) return MOE_ERR_INVALID_ARG;
  if (shape->tokens > 0 &&
      (y == nullptr || dst_pos == nullptr || gates == nullptr || out == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(y, 16) || !aligned(out, 16) || !aligned(shared, 16) || !aligned(residual, 16) ||
      !aligned(dst_pos, 4) || !aligned(gates, 4))
    return MOE_ERR_INVALID_ARG;
  moe_status_t st = ws_ok(shape, ws, ws_bytes);
  if (st != MOE_OK) return st;
  if (shape->tokens == 0) return MOE_OK;
  return from_cuda(moe::launch_combine(env_of(stream), y, dst_pos, gates, shared, residual,
                                       shape->tokens, shape->hidden, shape->k, rows_of(shape),
                                       out, static_cast<WsHeader*>(ws), shape->capacity > 0));
}

moe_status_t moe_combine_backward(const moe_shape_t* shape, const void* grad_out, const void* y,
                                  const int32_t* dst_pos, const float* gates, void* grad_y,
                                  float* grad_gates, void* ws, size_t ws_bytes,
                                  moe_stream_t stream) {
  if (!shape_ok(shape)) return MOE_ERR_INVALID_ARG;
  if (shape->tokens > 0 && (grad_out == nullptr || dst_pos == nullptr || gates == nullptr ||
                            grad_gates == nullptr || y == nullptr || grad_y == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(grad_out, 16) || !aligned(y, 16) || !aligned(grad_y, 16) || !aligned(dst_pos, 4) ||
      !aligned(gates, 4) || !aligned(grad_gates, 4))
    return MOE_ERR_INVALID_ARG;
  moe_status_t st = ws_ok(shape, ws, ws_bytes);
  if (st != MOE_OK) return st;
  if (shape->tokens == 0) return MOE_OK;
  return from_cuda(moe::launch_combine_backward(env_of(stream), grad_out, y, dst_pos, gates,
                                                shape->tokens, shape->hidden, shape->k,
                                                rows_of(shape), grad_y, grad_gates,
                                                static_cast<WsHeader*>(ws)));
}

}  // extern "C"

namespace {

bool rule_ok(const moe_shape_t* s, const moe_score_t* r, moe::ScoreRule* out) {
  if (r == nullptr) return false;
  if (r->func != MOE_SCORE_SOFTMAX && r->func != MOE_SCORE_SIGMOID) return false;
  if (r->groups < 1 || r->groups > 64 || (s->experts % r->groups) != 0) return false;
  const int size = s->experts / r->groups;
  if (r->top_groups < 1 || r->top_groups > r->groups) return false;
  if ((int64_t)r->top_groups * size < s->k) return false;
  if (r->group_top < 1 || r->group_top > 2 || r->group_top > size) return false;
  if (!std::isfinite(r->scale) || r->scale <= 0.0) return false;
  out->softmax = r->func == MOE_SCORE_SOFTMAX ? 1 : 0;
  out->groups = r->groups;
  out->top_groups = r->top_groups;
  out->group_top = r->group_top;
  out->renorm = (s->flags & MOE_F_RENORM) ? 1 : 0;
  out->scale = r->scale;
  return true;
}

int wide_of(int32_t out_features, int32_t act) {
  return act == MOE_ACT_SWIGLU ? 2 * out_features : out_features;
}

// The checks the experts' products share.
moe_status_t experts_ok(const moe_shape_t* s, int32_t in, int32_t out, int32_t act,
                        const int32_t* counts, const int32_t* expert_off) {
  if (!shape_ok(s) || src_layout(s)) return MOE_ERR_INVALID_ARG;
  if (in < 8 || (in % 8) != 0 || in > 65536) return MOE_ERR_INVALID_ARG;
  if (out < 8 || (out % 8) != 0 || out > 65536) return MOE_ERR_INVALID_ARG;
  if (act < MOE_ACT_NONE || act > MOE_ACT_SWIGLU) return MOE_ERR_INVALID_ARG;
  if ((counts == nullptr) != (expert_off == nullptr)) return MOE_ERR_INVALID_ARG;
  if (counts == nullptr && (s->experts != 1 || s->capacity != 0 || s->align != 1))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(counts, 4) || !aligned(expert_off, 4)) return MOE_ERR_INVALID_ARG;
  if (!moe::expert_tiles_fit(int64_t(s->tokens) * s->k, s->experts, in, wide_of(out, act)))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe::ExpertMatmul experts_of(const moe_shape_t* s, int32_t in, int32_t out, int32_t act,
                             const void* x, const void* w, const int32_t* counts,
                             const int32_t* expert_off, void* ws) {
  moe::ExpertMatmul a = {};
  a.x = x;
  a.w = w;
  a.counts = counts;
  a.expert_off = expert_off;
  a.hdr = static_cast<WsHeader*>(ws);
  a.N = rows_of(s);
  a.assignments = int64_t(s->tokens) * s->k;
  a.E = s->experts;
  a.capacity = s->capacity;
  a.in_features = in;
  a.out_features = out;
  a.act = act;
  return a;
}

}  // namespace

extern "C" {

moe_status_t moe_route_scored(const moe_shape_t* shape, const float* logits, const float* bias,
                              const moe_score_t* rule, int32_t* ids, float* gates, void* ws,
                              size_t ws_bytes, moe_stream_t stream) {
  moe::ScoreRule r;
  if (!shape_ok(shape) || !rule_ok(shape, rule, &r)) return MOE_ERR_INVALID_ARG;
  if (shape->tokens > 0 && (logits == nullptr || ids == nullptr || gates == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(logits, 4) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(gates, 4))
    return MOE_ERR_INVALID_ARG;
  moe_status_t st = ws_ok(shape, ws, ws_bytes);
  if (st != MOE_OK) return st;
  if (shape->tokens == 0) return MOE_OK;
  return from_cuda(moe::launch_route_scored(env_of(stream), logits, bias, shape->tokens,
                                            shape->experts, shape->k, r, ids, gates,
                                            static_cast<WsHeader*>(ws)));
}

moe_status_t moe_route_scored_backward(const moe_shape_t* shape, const float* logits,
                                       const moe_score_t* rule, const int32_t* ids,
                                       const float* grad_gates, float* grad_logits, void* ws,
                                       size_t ws_bytes, moe_stream_t stream) {
  moe::ScoreRule r;
  if (!shape_ok(shape) || !rule_ok(shape, rule, &r)) return MOE_ERR_INVALID_ARG;
  if (shape->tokens > 0 && (logits == nullptr || ids == nullptr || grad_gates == nullptr ||
                            grad_logits == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(logits, 4) || !aligned(ids, 4) || !aligned(grad_gates, 4) ||
      !aligned(grad_logits, 4))
    return MOE_ERR_INVALID_ARG;
  moe_status_t st = ws_ok(shape, ws, ws_bytes);
  if (st != MOE_OK) return st;
  if (shape->tokens == 0) return MOE_OK;
  return from_cuda(moe::launch_route_scored_backward(
      env_of(stream), logits, ids, grad_gates, shape->tokens, shape->experts, shape->k, r,
      grad_logits, static_cast<WsHeader*>(ws)));
}

moe_status_t moe_expert_matmul(const moe_shape_t* shape, int32_t in_features,
                               int32_t out_features, int32_t act, const void* x, const void* w,
                               const float* bias, const int32_t* counts,
                               const int32_t* expert_off, const void* residual, void* out,
                               void* pre, void* ws, size_t ws_bytes, moe_stream_t stream) {
  moe_status_t st = experts_ok(shape, in_features, out_features, act, counts, expert_off);
  if (st != MOE_OK) return st;
  if (shape->tokens > 0 && (x == nullptr || w == nullptr || out == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(pre, 16) ||
      !aligned(residual, 16) || !aligned(bias, 4))
    return MOE_ERR_INVALID_ARG;
  st = ws_ok(shape, ws, ws_bytes);
  if (st != MOE_OK) return st;
  if (shape->tokens == 0) return MOE_OK;
  moe::ExpertMatmul a = experts_of(shape, in_features, out_features, act, x, w, counts,
                                   expert_off, ws);
  a.bias = bias;
  a.residual = residual;
  a.out = out;
  a.pre = pre;
  return from_cuda(moe::launch_expert_matmul(env_of(stream), a));
}

size_t moe_expert_matmul_backward_scratch_bytes(const moe_shape_t* shape, int32_t out_features,
                                                int32_t act) {
  if (!shape_ok(shape) || src_layout(shape)) return 0;
  if (out_features < 8 || (out_features % 8) != 0 || out_features > 65536) return 0;
  if (act < MOE_ACT_NONE || act > MOE_ACT_SWIGLU) return 0;
  return moe::expert_act_scratch_bytes(int64_t(shape->tokens) * shape->k, shape->experts,
                                       wide_of(out_features, act));
}

moe_status_t moe_expert_matmul_backward(const moe_shape_t* shape, int32_t in_features,
                                        int32_t out_features, int32_t act, const void* grad_out,
                                        const void* x, const void* w, const void* pre,
                                        const int32_t* counts, const int32_t* expert_off,
                                        void* grad_pre, void* grad_x, void* grad_w,
                                        float* grad_bias, void* scratch, size_t scratch_bytes,
                                        void* ws, size_t ws_bytes, moe_stream_t stream) {
  moe_status_t st = experts_ok(shape, in_features, out_features, act, counts, expert_off);
  if (st != MOE_OK) return st;
  const bool rows = shape->tokens > 0;
  if (rows && grad_out == nullptr) return MOE_ERR_INVALID_ARG;
  if (rows && act != MOE_ACT_NONE && (pre == nullptr || grad_pre == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (rows && grad_x != nullptr && w == nullptr) return MOE_ERR_INVALID_ARG;
  if (rows && grad_w != nullptr && x == nullptr) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {grad_out, x, w, pre, grad_pre, grad_x, grad_w, scratch};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return MOE_ERR_INVALID_ARG;
  if (!aligned(grad_bias, 4)) return MOE_ERR_INVALID_ARG;
  if (grad_bias != nullptr &&
      (scratch == nullptr ||
       scratch_bytes < moe_expert_matmul_backward_scratch_bytes(shape, out_features, act)))
    return MOE_ERR_WORKSPACE;
  st = ws_ok(shape, ws, ws_bytes);
  if (st != MOE_OK) return st;
  const int wide = wide_of(out_features, act);
  if (!rows) {  // no rows: the sums over rows are zero
    const size_t cells = (size_t)shape->experts * wide;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (grad_w != nullptr &&
        cudaMemsetAsync(grad_w, 0, cells * in_features * 2, s) != cudaSuccess)
      return MOE_ERR_CUDA;
    if (grad_bias != nullptr &&
        cudaMemsetAsync(grad_bias, 0, cells * sizeof(float), s) != cudaSuccess)
      return MOE_ERR_CUDA;
    return MOE_OK;
  }
  const moe::LaunchEnv env = env_of(stream);
  const moe::ExpertMatmul a = experts_of(shape, in_features, out_features, act, x, w, counts,
                                         expert_off, ws);
  const void* dz = act == MOE_ACT_NONE ? grad_out : grad_pre;
  cudaError_t err = cudaSuccess;
  if (act != MOE_ACT_NONE || grad_bias != nullptr)
    err = moe::launch_expert_act_backward(env, a, grad_out, pre, grad_pre, scratch,
                                          grad_bias);
  if (err == cudaSuccess && grad_x != nullptr)
    err = moe::launch_expert_grad_rows(env, a, dz, grad_x);
  if (err == cudaSuccess && grad_w != nullptr)
    err = moe::launch_expert_grad_weights(env, a, dz, grad_w);
  return from_cuda(err);
}

moe_status_t moe_selftest_wait_timeout(void* ws, uint32_t timeout_us, moe_stream_t stream) {
  if (ws == nullptr || !aligned(ws, 16)) return MOE_ERR_WORKSPACE;
  if (timeout_us < 1u || timeout_us > 2000000u) return MOE_ERR_INVALID_ARG;
  return from_cuda(moe::launch_wait_timeout_selftest(env_of(stream), static_cast<WsHeader*>(ws),
                                                     uint64_t(timeout_us) * 1000u));
}

moe_status_t moe_get_device_error(void* ws, int32_t* detail, moe_stream_t stream) {
  if (ws == nullptr || !aligned(ws, 16)) return MOE_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int32_t h[2] = {0, 0};
  if (cudaMemcpyAsync(h, ws, sizeof(h), cudaMemcpyDeviceToHost, s) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return MOE_ERR_CUDA;
  if (h[0] != 0) {
    if (cudaMemsetAsync(ws, 0, sizeof(h), s) != cudaSuccess) return MOE_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return MOE_ERR_CUDA;
  }
  if (detail != nullptr) *detail = h[1];
  return static_cast<moe_status_t>(h[0]);
}

}  // extern "C"
