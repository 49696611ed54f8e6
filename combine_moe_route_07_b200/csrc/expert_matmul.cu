// expert_matmul.cu -- the experts' matrix products on the rows of a layout,
// with bias, activation and residual in the epilogue, and their gradients.
//
//   forward   z[p,:] = x[p,:] W_e^T + b_e,  y[p,:] = act(z[p,:]) + residual[p,:]
//   rows      dx[p,:] = dz[p,:] W_e
//   weights   dW_e    = sum over the rows p of expert e of dz[p,:]^T x[p,:]
//
// for the rows p that hold a token of expert e.  Products of bf16 operands are
// summed in fp32 in tensor memory (tcgen05, kind::f16); bias, activation and
// residual are applied in fp32 and the result is rounded once.
//
// The weights are the M operand (128 channels a tile) and the tokens the N
// operand: an expert's ragged number of rows then only sets N of the
// instruction (a multiple of 16, up to 256), so a decode batch with a few rows
// an expert does no padded work and streams its weights, and a row of another
// expert that a tile's copy brings along can never reach this expert's sums
// (columns of D are independent).
//
// One persistent CTA per SM: a producer thread feeds a ring of 4 stages by
// tensor-map copies (64-deep slices, 128-byte swizzle), one thread issues the
// matrix instructions, four warps drain the accumulator of the previous tile
// meanwhile (two accumulators in tensor memory).  Every wait is bounded.
#include <math.h>

#include "block_scan.cuh"
#include "common.cuh"
#include "kernels.h"
#include "umma.cuh"

namespace moe {

namespace {

constexpr int kBK = 64;       // contraction depth of a stage
constexpr int kBM = 128;      // channels of a tile
constexpr int kStages = 4;
constexpr int kStageBytes = 48 * 1024;
constexpr int kGemmThreads = 256;
constexpr int kEpiPad = 36;   // floats between staged rows: 16-byte rows on distinct banks
constexpr int kEpiBytes = 4 * 32 * kEpiPad * 4;
constexpr int kTmemCols = 512;
constexpr uint64_t kWaitNs = 2000000000ull;

enum { kFwd = 0, kRows = 1, kWeights = 2 };

struct GemmParams {
  CUtensorMap ma;  // M operand: weights [E][W][K]; weights gradient: dz [N][W]
  CUtensorMap mb;  // N operand: x or dz [N][..]
  const int32_t* counts;  // NULL: one expert holding every row
  const int32_t* off;
  const float* bias;
  const uint16_t* residual;
  uint16_t* out;
  uint16_t* pre;
  WsHeader* hdr;
  int64_t N;
  int64_t max_rows;  // T*k: rows of all segments together, at most
  int E, capacity;
  int M;       // channels of an expert (gated: of one half)
  int kdim;    // contraction length (weights gradient: per expert)
  int cols;    // weights gradient: columns of x
  int band;    // token tiles an expert walks together
  int act;
};

struct Segment {
  int off, rows;
};

// Rows of expert e; a segment outside [0, N) is reported and treated as empty.
__device__ __forceinline__ Segment segment(const GemmParams& P, int e, bool tell) {
  Segment s;
  if (P.counts == nullptr) {
    s.off = 0;
    s.rows = (int)P.N;
    return s;
  }
  s.off = __ldg(P.off + e);
  s.rows = __ldg(P.counts + e);
  if (P.capacity > 0 && s.rows > P.capacity) s.rows = P.capacity;
  if (s.rows <= 0 || s.off < 0 || (int64_t)s.off + s.rows > P.N) {
    if (tell && s.rows != 0) report(P.hdr, MOE_ERR_DEVICE_RANGE, e);
    s.off = 0;
    s.rows = 0;
  }
  return s;
}

__device__ __forceinline__ float sigmoid_f(float x) {
  return __fdividef(1.0f, 1.0f + __expf(-x));
}
__device__ __forceinline__ float act_f(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z != z ? z : fmaxf(z, 0.0f);
    case MOE_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    case MOE_ACT_SILU: return z * sigmoid_f(z);
  }
  return z;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Tile t of the forward / rows products.
struct Tile {
  int e, c, row0, rows;  // expert, channel tile, first row, rows
};

template <int MODE, bool GATED>
__global__ void __launch_bounds__(kGemmThreads, 1)
    expert_gemm_kernel(const __grid_constant__ GemmParams P) {
  constexpr int kBN = GATED ? 128 : 256;
  constexpr int kABytes = (GATED ? 2 : 1) * kBM * kBK * 2;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[kStages], empty[kStages], tfull[2], tempty[2], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ unsigned long long rows_sum;
  __shared__ int32_t warp_tot[kGemmThreads / 32];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  float* epi = reinterpret_cast<float*>(smem + kStages * kStageBytes);
  int32_t* seg_off = reinterpret_cast<int32_t*>(smem + kStages * kStageBytes + kEpiBytes);
  int32_t* seg_rows = seg_off + P.E;
  int32_t* first = seg_rows + P.E;  // forward / rows: exclusive prefix of token tiles [E+1]

  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&tfull[s], 1);
      mbar_init(&tempty[s], 4);
    }
    mbar_init(&drain, 1);
    abort_flag = 0;
    rows_sum = 0ull;
    mbar_fence_init();
    tma_prefetch_map(&P.ma);
    tma_prefetch_map(&P.mb);
  }
  if (wid == 1) tmem_alloc(&tmem_slot, kTmemCols);
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  unsigned long long my_rows = 0ull;
  for (int e = tid; e < P.E; e += kGemmThreads) {
    const Segment s = segment(P, e, blockIdx.x == 0);
    seg_off[e] = s.off;
    seg_rows[e] = s.rows;
    my_rows += (unsigned long long)s.rows;
    if (MODE != kWeights) first[e] = (s.rows + kBN - 1) / kBN;
  }
  if (my_rows != 0ull) atomicAdd(&rows_sum, my_rows);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int ctiles = (P.M + kBM - 1) / kBM;
  int total;
  if constexpr (MODE == kWeights) {
    total = P.E * ctiles * ((P.cols + kBN - 1) / kBN);
  } else {
    const int tt = block_exclusive_scan<kGemmThreads>(first, P.E, warp_tot);
    if (tid == 0) first[P.E] = tt;
    __syncthreads();
    total = tt * ctiles;
  }

  // more rows than assignments: the segments are not a layout's, nothing is done
  if ((int64_t)rows_sum > P.max_rows) {
    if (tid == 0 && blockIdx.x == 0) report(P.hdr, MOE_ERR_DEVICE_RANGE, P.E);
    total = 0;
  }

  volatile int* stop = &abort_flag;
  // Wait for a phase; false: it gave up, or another role did.
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (unsigned it = 0; it < (1u << 24); ++it) {
      if (mbar_try_wait(bar, parity)) return true;
      if ((it & 63u) == 63u && (*stop != 0 || global_ns() - t0 > kWaitNs)) break;
    }
    if (*stop == 0) report(P.hdr, MOE_ERR_DEVICE_TIMEOUT, blockIdx.x);
    *stop = 1;
    return false;
  };

  // Tile t: its expert, channel tile, rows (forward / rows) or column tile.
  auto tile_of = [&](int t) -> Tile {
    Tile r;
    if constexpr (MODE == kWeights) {
      const int nt = (P.cols + kBN - 1) / kBN;
      r.e = t / (ctiles * nt);
      const int u = t - r.e * ctiles * nt;
      r.c = u / nt;
      r.row0 = (u - r.c * nt) * kBN;  // first column
      r.rows = min(kBN, P.cols - r.row0);
    } else {
      const int u = t / ctiles;
      int lo = 0, hi = P.E;  // first[lo] <= u < first[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= u)
          lo = mid;
        else
          hi = mid;
      }
      const int nt = first[lo + 1] - first[lo];
      const int local = t - first[lo] * ctiles;
      const int b = local / (P.band * ctiles);
      const int nb = min(P.band, nt - b * P.band);
      const int v = local - b * P.band * ctiles;
      const int n = b * P.band + v % nb;
      // the rows split evenly over the expert's tiles, in multiples of 16
      const int per = ((seg_rows[lo] + nt - 1) / nt + 15) & ~15;
      r.e = lo;
      r.c = v / nb;
      r.row0 = n * per;
      r.rows = min(per, seg_rows[lo] - r.row0);
    }
    return r;
  };

  if (wid == 0) {
    // ---- producer -------------------------------------------------------------
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
        const Tile r = tile_of(t);
        const int depth = MODE == kWeights ? seg_rows[r.e] : P.kdim;
        const int row = seg_off[r.e] + (MODE == kWeights ? 0 : r.row0);
        const int nkb = (depth + kBK - 1) / kBK;
        const int boxes = (r.rows + 63) >> 6;
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const int s = it % kStages;
          if (!wait(&empty[s], ((it / kStages) & 1u) ^ 1u)) {
            ok = false;
            break;
          }
          uint8_t* a = smem + s * kStageBytes;
          uint8_t* b = a + kABytes;
          mbar_arrive_expect_tx(&full[s], (uint32_t)kABytes + (uint32_t)boxes * 8192u);
          if constexpr (MODE == kFwd) {
            tma_load_3d(a, &P.ma, kb * kBK, r.c * kBM, r.e, &full[s]);
            if constexpr (GATED) tma_load_3d(a + 16384, &P.ma, kb * kBK, P.M + r.c * kBM, r.e, &full[s]);
            for (int i = 0; i < boxes; ++i)
              tma_load_2d(b + i * 8192, &P.mb, kb * kBK, row + i * 64, &full[s]);
          } else if constexpr (MODE == kRows) {
            tma_load_3d(a, &P.ma, r.c * kBM, kb * kBK, r.e, &full[s]);
            tma_load_3d(a + 8192, &P.ma, r.c * kBM + 64, kb * kBK, r.e, &full[s]);
            for (int i = 0; i < boxes; ++i)
              tma_load_2d(b + i * 8192, &P.mb, kb * kBK, row + i * 64, &full[s]);
          } else {
            tma_load_2d(a, &P.ma, r.c * kBM, row + kb * kBK, &full[s]);
            tma_load_2d(a + 8192, &P.ma, r.c * kBM + 64, row + kb * kBK, &full[s]);
            for (int i = 0; i < boxes; ++i)
              tma_load_2d(b + i * 8192, &P.mb, r.row0 + i * 64, row + kb * kBK, &full[s]);
          }
        }
      }
      if (!ok) {  // copies in flight land before the CTA ends
        for (uint32_t j = it > kStages ? it - kStages : 0; j < it; ++j)
          mbar_wait_bounded(&full[j % kStages], (j / kStages) & 1u, kWaitNs);
      }
    }
    __syncwarp();
  } else if (wid == 1) {
    // ---- matrix instructions ----------------------------------------------------
    constexpr uint32_t a_mn = MODE == kFwd ? 0u : 1u, b_mn = MODE == kWeights ? 1u : 0u;
    uint32_t it = 0, nacc = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
      const Tile r = tile_of(t);
      const int depth = MODE == kWeights ? seg_rows[r.e] : P.kdim;
      const int nkb = (depth + kBK - 1) / kBK;
      if (nkb == 0) continue;
      const uint32_t acc = nacc & 1u;
      if (!wait(&tempty[acc], ((nacc >> 1) & 1u) ^ 1u)) break;
      tc_fence_after();
      ++nacc;
      const uint32_t d = tmem + acc * 256u;
      const uint32_t idesc = umma_idesc(kBM, (uint32_t)((r.rows + 15) & ~15), a_mn, b_mn);
      for (int kb = 0; kb < nkb; ++kb, ++it) {
        const int s = it % kStages;
        if (!wait(&full[s], (it / kStages) & 1u)) {
          ok = false;
          break;
        }
        uint8_t* a = smem + s * kStageBytes;
        uint8_t* b = a + kABytes;
        int ksteps = kBK / 16;
        if constexpr (MODE == kWeights) {
          // rows behind the expert's last one: another expert's, or never written.
          // Steps wholly behind it are skipped; in the last step they become zero
          // in both operands (zero times NaN is not zero).
          const int valid = min(kBK, depth - kb * kBK);
          ksteps = (valid + 15) >> 4;
          const int stale = ksteps * 16 - valid;
          if (stale > 0) {
            const int blocks = 2 + ((r.rows + 63) >> 6);
            for (int i = lane; i < blocks * stale * 8; i += 32) {
              const int q = i & 7, row = valid + (i >> 3) % stale, blk = (i >> 3) / stale;
              uint8_t* base = blk < 2 ? a + blk * 8192 : b + (blk - 2) * 8192;
              *reinterpret_cast<uint4*>(base + row * 128 + q * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
        }
        tc_fence_after();
        if (lane == 0) {
          const uint32_t sa = smem_addr(a), sb = smem_addr(b);
          for (int q = 0; q < ksteps; ++q) {
            const uint64_t da = a_mn ? umma_desc(sa + q * 2048, 8192, 1024)
                                     : umma_desc(sa + q * 32, 16, 1024);
            const uint64_t db = b_mn ? umma_desc(sb + q * 2048, 8192, 1024)
                                     : umma_desc(sb + q * 32, 16, 1024);
            umma_f16(d, da, db, idesc, kb > 0 || q > 0);
            if constexpr (GATED)
              umma_f16(d + 128u, umma_desc(sa + 16384 + q * 32, 16, 1024), db, idesc,
                       kb > 0 || q > 0);
          }
          umma_commit(&empty[s]);
        }
        __syncwarp();
      }
      if (ok && lane == 0) umma_commit(&tfull[acc]);
      __syncwarp();
    }
    if (*stop != 0) {
      if (lane == 0) {
        umma_commit(&drain);
        mbar_wait_bounded(&drain, 0u, kWaitNs);
      }
      __syncwarp();
    }
  } else if (wid >= 4) {
    // ---- epilogue: warp q drains rows 32q..32q+31 of the accumulator -------------
    const int q = wid - 4;
    float* buf = epi + q * 32 * kEpiPad;
    uint32_t nacc = 0;
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
      const Tile r = tile_of(t);
      const bool empty_sum = MODE == kWeights && seg_rows[r.e] == 0;
      const uint32_t acc = nacc & 1u;
      if (!empty_sum) {
        if (!wait(&tfull[acc], (nacc >> 1) & 1u)) break;
        tc_fence_after();
        ++nacc;
      }
      const uint32_t d = tmem + acc * 256u + ((uint32_t)(q * 32) << 16);
      const int ch0 = r.c * kBM + q * 32;  // this warp's first channel
      // Store a staged 32 x 32 block: rows of `dst` `stride` elements apart,
      // columns in 16-byte pieces (widths are multiples of 8), coalesced.
      auto flush = [&](uint16_t* dst, size_t stride, int nrows, int ncols, const uint16_t* add) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = i * 8 + (lane >> 2), cc = (lane & 3) * 8;
          if (rr < nrows && cc < ncols) {
            const float4 v0 = *reinterpret_cast<const float4*>(buf + rr * kEpiPad + cc);
            const float4 v1 = *reinterpret_cast<const float4*>(buf + rr * kEpiPad + cc + 4);
            float f[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
            const size_t at = (size_t)rr * stride + cc;
            if (add != nullptr) {
              const uint4 a4 = *reinterpret_cast<const uint4*>(add + at);
              const uint32_t aw[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                f[2 * u] += bf16lo(aw[u]);
                f[2 * u + 1] += bf16hi(aw[u]);
              }
            }
            st16(dst + at, make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]),
                                      pack2(f[6], f[7])));
          }
        }
        __syncwarp();
      };
      const int nchunks = (r.rows + 31) >> 5;
      if constexpr (MODE == kWeights) {
        uint16_t* dst = P.out + ((size_t)r.e * P.M + ch0) * P.cols + r.row0;
        for (int j = 0; j < nchunks; ++j) {
          uint32_t v[32];
          if (!empty_sum) {
            tmem_ld32(d + j * 32, v);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0u;
          }
          // this lane holds 32 columns of one row of dW
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<uint4*>(buf + lane * kEpiPad + i) =
                make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
          flush(dst + j * 32, (size_t)P.cols, P.M - ch0, r.rows - j * 32, nullptr);
        }
      } else {
        const int ch = ch0 + lane;
        float b0 = 0.0f, b1 = 0.0f;
        if constexpr (MODE == kFwd) {
          if (P.bias != nullptr && ch < P.M) {
            const float* bp = P.bias + (size_t)r.e * P.M * (GATED ? 2 : 1) + ch;
            b0 = __ldg(bp);
            if constexpr (GATED) b1 = __ldg(bp + P.M);
          }
        }
        const int64_t row = (int64_t)seg_off[r.e] + r.row0;
        for (int j = 0; j < nchunks; ++j) {
          uint32_t v[32];
          tmem_ld32(d + j * 32, v);
          uint32_t u[GATED ? 32 : 1];
          if constexpr (GATED) tmem_ld32(d + 128u + j * 32, reinterpret_cast<uint32_t(&)[32]>(u));
          tmem_ld_wait();
          const int64_t row_j = row + j * 32;
          const int nr = r.rows - j * 32, nc = P.M - ch0;
          // this lane holds one channel of 32 tokens: staged token-major
          if constexpr (MODE == kFwd) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + b0);
            if constexpr (GATED) {
#pragma unroll
              for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) + b1);
            }
            if (P.pre != nullptr) {
              const size_t wide = (size_t)P.M * (GATED ? 2 : 1);
#pragma unroll
              for (int i = 0; i < 32; ++i) buf[i * kEpiPad + lane] = __uint_as_float(v[i]);
              flush(P.pre + row_j * wide + ch0, wide, nr, nc, nullptr);
              if constexpr (GATED) {
#pragma unroll
                for (int i = 0; i < 32; ++i) buf[i * kEpiPad + lane] = __uint_as_float(u[i]);
                flush(P.pre + row_j * wide + P.M + ch0, wide, nr, nc, nullptr);
              }
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float z = __uint_as_float(v[i]);
              float y;
              if constexpr (GATED)
                y = z * sigmoid_f(z) * __uint_as_float(u[i]);
              else
                y = act_f(z, P.act);
              buf[i * kEpiPad + lane] = y;
            }
            flush(P.out + row_j * P.M + ch0, (size_t)P.M, nr, nc,
                  P.residual != nullptr ? P.residual + row_j * P.M + ch0 : nullptr);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) buf[i * kEpiPad + lane] = __uint_as_float(v[i]);
            flush(P.out + row_j * P.M + ch0, (size_t)P.M, nr, nc, nullptr);
          }
        }
      }
      if (!empty_sum) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[acc]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (wid == 1) tmem_free(tmem, kTmemCols);
}

// ---- tensor maps --------------------------------------------------------------

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// bf16 tensor [d2][d1][d0] (d2 = 1: a matrix), boxes of 64 x box1, 128-byte
// swizzle, zeros outside.
cudaError_t make_map(CUtensorMap* map, const void* ptr, int64_t d0, int64_t d1, int64_t d2,
                     int box1) {
  const EncodeFn fn = encode_fn();
  if (fn == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {(cuuint64_t)d0, (cuuint64_t)d1, (cuuint64_t)d2};
  const cuuint64_t strides[2] = {(cuuint64_t)d0 * 2, (cuuint64_t)d0 * (cuuint64_t)d1 * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box1, 1};
  const cuuint32_t es[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, d2 > 0 ? 3 : 2,
                        const_cast<void*>(ptr), dims, strides, box, es,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int MODE, bool GATED>
cudaError_t launch_gemm(const LaunchEnv& env, const GemmParams& P, int64_t max_tiles) {
  const size_t smem = 1024 + (size_t)kStages * kStageBytes + kEpiBytes +
                      sizeof(int32_t) * ((size_t)P.E * (MODE == kWeights ? 2 : 3) + 1);
  int per_sm = 1;
  const auto kernel = expert_gemm_kernel<MODE, GATED>;
  cudaError_t err = blocks_per_sm((const void*)kernel, kGemmThreads, smem, &per_sm);
  if (err != cudaSuccess) return err;
  const int64_t grid = max_tiles < env.num_sms ? max_tiles : env.num_sms;
  return launch_pdl(env, kernel, dim3((unsigned)(grid > 0 ? grid : 1)), dim3(kGemmThreads), smem, P);
}

// Token tiles of `bn` rows there can be at most: full ones, and a partial one
// for each expert that can hold a row.
int64_t max_token_tiles(int64_t assignments, int E, int64_t bn) {
  return assignments / bn + (assignments < E ? assignments : E);
}

}  // namespace

bool expert_tiles_fit(int64_t assignments, int E, int in, int wide) {
  const int64_t ct = (wide + kBM - 1) / kBM, it = (in + kBM - 1) / kBM;
  const int64_t tt = max_token_tiles(assignments, E, 128);
  return tt * (ct > it ? ct : it) < (int64_t(1) << 31) && (int64_t)E * ct * it < (int64_t(1) << 31);
}

cudaError_t launch_expert_matmul(const LaunchEnv& env, const ExpertMatmul& a) {
  const bool gated = a.act == MOE_ACT_SWIGLU;
  const int wide = gated ? 2 * a.out_features : a.out_features;
  GemmParams P = {};
  cudaError_t err = make_map(&P.ma, a.w, a.in_features, wide, a.E, kBM);
  if (err != cudaSuccess) return err;
  err = make_map(&P.mb, a.x, a.in_features, a.N, 0, 64);
  if (err != cudaSuccess) return err;
  P.counts = a.counts;
  P.off = a.expert_off;
  P.bias = a.bias;
  P.residual = static_cast<const uint16_t*>(a.residual);
  P.out = static_cast<uint16_t*>(a.out);
  P.pre = static_cast<uint16_t*>(a.pre);
  P.hdr = a.hdr;
  P.N = a.N;
  P.max_rows = a.assignments;
  P.E = a.E;
  P.capacity = a.capacity;
  P.M = a.out_features;
  P.kdim = a.in_features;
  P.act = a.act;
  P.band = 16;
  const int64_t ct = (P.M + kBM - 1) / kBM;
  if (gated) return launch_gemm<kFwd, true>(env, P, max_token_tiles(a.assignments, a.E, 128) * ct);
  return launch_gemm<kFwd, false>(env, P, max_token_tiles(a.assignments, a.E, 256) * ct);
}

cudaError_t launch_expert_grad_rows(const LaunchEnv& env, const ExpertMatmul& a, const void* dz,
                                    void* grad_x) {
  const int wide = a.act == MOE_ACT_SWIGLU ? 2 * a.out_features : a.out_features;
  GemmParams P = {};
  cudaError_t err = make_map(&P.ma, a.w, a.in_features, wide, a.E, kBK);
  if (err != cudaSuccess) return err;
  err = make_map(&P.mb, dz, wide, a.N, 0, 64);
  if (err != cudaSuccess) return err;
  P.counts = a.counts;
  P.off = a.expert_off;
  P.out = static_cast<uint16_t*>(grad_x);
  P.hdr = a.hdr;
  P.N = a.N;
  P.max_rows = a.assignments;
  P.E = a.E;
  P.capacity = a.capacity;
  P.M = a.in_features;
  P.kdim = wide;
  P.band = 16;
  const int64_t ct = (P.M + kBM - 1) / kBM;
  return launch_gemm<kRows, false>(env, P, max_token_tiles(a.assignments, a.E, 256) * ct);
}

cudaError_t launch_expert_grad_weights(const LaunchEnv& env, const ExpertMatmul& a, const void* dz,
                                       void* grad_w) {
  const int wide = a.act == MOE_ACT_SWIGLU ? 2 * a.out_features : a.out_features;
  GemmParams P = {};
  cudaError_t err = make_map(&P.ma, dz, wide, a.N, 0, kBK);
  if (err != cudaSuccess) return err;
  err = make_map(&P.mb, a.x, a.in_features, a.N, 0, kBK);
  if (err != cudaSuccess) return err;
  P.counts = a.counts;
  P.off = a.expert_off;
  P.out = static_cast<uint16_t*>(grad_w);
  P.hdr = a.hdr;
  P.N = a.N;
  P.max_rows = a.assignments;
  P.E = a.E;
  P.capacity = a.capacity;
  P.M = wide;
  P.cols = a.in_features;
  const int64_t tiles = (int64_t)a.E * ((wide + kBM - 1) / kBM) * ((a.in_features + 255) / 256);
  return launch_gemm<kWeights, false>(env, P, tiles);
}

}  // namespace moe
