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
// The weights are the M operand (256 channels a tile, 128 on each CTA of a
// pair) and the tokens the N operand: an expert's ragged number of rows then
// only sets N of the instruction (a multiple of 32, up to 256), so a decode
// batch with a few rows an expert does little padded work and streams its
// weights, and a row of another expert that a tile's copy brings along can
// never reach this expert's sums (columns of D are independent).
//
// Persistent pairs of CTAs (cta_group::2), one CTA per SM: in each CTA a
// producer thread feeds a ring of 6 stages of 32 KiB by tensor-map copies
// (64-deep slices, 128-byte swizzle), the even CTA's issuing thread runs the
// matrix instructions of both, and eight warps of each drain the accumulator
// of the previous tile meanwhile (two accumulators in tensor memory).  A pair
// shares its operands, so a 256 x 256 tile costs each SM 32 KiB of copies per
// 64-deep slice; one CTA alone moves 48 KiB for the same work and is bound by
// the L2 (about 10 TB/s).  Every wait is bounded.
#include <math.h>

#include "block_scan.cuh"
#include "common.cuh"
#include "kernels.h"
#include "umma.cuh"

namespace moe {

namespace {

constexpr int kBK = 64;       // contraction depth of a stage
constexpr int kBM = 128;      // rows of the M operand on each CTA of a pair
constexpr int kBN = 256;      // columns of a tile
constexpr int kBox = 32;      // token rows of one copy
constexpr int kABytes = kBM * kBK * 2;
constexpr int kStages = 6;
constexpr int kStageBytes = 32 * 1024;
constexpr int kEpiWarps = 8;
constexpr int kGemmThreads = (4 + kEpiWarps) * 32;
constexpr int kEpiBytes = kEpiWarps * 2048;  // 32 x 32 bf16 a warp
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

// gelu(z) = z * Phi(z), Phi by the rational approximation 7.1.26 of Abramowitz
// and Stegun's Handbook (erfc(x) = (a1 t + .. + a5 t^5) exp(-x^2), t = 1 / (1 +
// p x), within 1.5e-7): the tail is not a difference of near-equal numbers.
__device__ __forceinline__ float gelu_f(float z) {
  const float x = fabsf(z) * 0.70710678f;
  const float t = __fdividef(1.0f, fmaf(0.3275911f, x, 1.0f));
  float q = fmaf(1.061405429f, t, -1.453152027f);
  q = fmaf(q, t, 1.421413741f);
  q = fmaf(q, t, -0.284496736f);
  q = fmaf(q, t, 0.254829592f);
  const float tail = 0.5f * q * t * __expf(-x * x);  // Phi(-|z|)
  return z * (z < 0.0f ? tail : 1.0f - tail);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint16_t to_bf16(float v) {
  uint16_t r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(v));
  return r;
}

// Tile t of the forward / rows products.
struct Tile {
  int e, c, row0, rows;  // expert, channel tile, first row, rows
};

template <int MODE, bool GATED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
    expert_gemm_kernel(const __grid_constant__ GemmParams P) {
  constexpr int kTileM = GATED ? kBM : 2 * kBM;  // output channels of a pair's tile
  extern __shared__ uint8_t smem_raw[];
  // tempty and fixed are waited on by the even CTA only; full too, but for an odd
  // CTA's slices with stale rows.  A stage's barriers see at most one phase at a
  // time: the stage is filled again only once the instructions that read it are done.
  __shared__ uint64_t full[kStages], empty[kStages], tfull[2], tempty[2], drain;
  __shared__ uint64_t fixed[kStages];  // weights gradient: the odd CTA's stale rows are zero
  __shared__ uint64_t swap[4];      // gated: between the two warps of a channel block
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ unsigned long long rows_sum;
  __shared__ int32_t warp_tot[kGemmThreads / 32];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* epi = smem + kStages * kStageBytes;
  int32_t* seg_off = reinterpret_cast<int32_t*>(smem + kStages * kStageBytes + kEpiBytes);
  int32_t* seg_rows = seg_off + P.E;
  int32_t* first = seg_rows + P.E;  // forward / rows: exclusive prefix of token tiles [E+1]

  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&fixed[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&tfull[s], 1);
      mbar_init(&tempty[s], 2 * kEpiWarps);
    }
    for (int s = 0; s < 4; ++s) mbar_init(&swap[s], 2);
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
  cluster_sync_all();  // the other CTA's barriers are ready too
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int ctiles = (P.M + kTileM - 1) / kTileM;
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
    if (mbar_try_wait_cluster(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (unsigned it = 0; it < (1u << 24); ++it) {
      if (mbar_try_wait_cluster(bar, parity)) return true;
      if ((it & 63u) == 63u && (*stop != 0 || global_ns() - t0 > kWaitNs)) break;
    }
    if (*stop == 0) report(P.hdr, MOE_ERR_DEVICE_TIMEOUT, blockIdx.x);
    *stop = 1;
    return false;
  };

  // The same for a whole warp: one answer for all its lanes.
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(kFull, wait(bar, parity));
  };

  // Tile t: its expert, channel tile, rows (forward / rows) or columns.
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
      // the rows split evenly over the expert's tiles, in multiples of 32
      const int per = ((seg_rows[lo] + nt - 1) / nt + 31) & ~31;
      r.e = lo;
      r.c = v / nb;
      r.row0 = n * per;
      r.rows = min(per, seg_rows[lo] - r.row0);
    }
    return r;
  };
  // Rows of the last slice that belong to the expert, when fewer than its
  // 16-deep steps take in (weights gradient).
  auto stale_tail = [&](int depth, int kb) -> bool {
    return MODE == kWeights && (kb + 1) * kBK > depth && (depth & 15) != 0;
  };
  // Rows behind the expert's last one are another expert's, or never written.
  // Steps wholly behind it are skipped; in the last step they become zero in
  // both operands (zero times NaN is not zero).  One warp, on this CTA's half.
  auto zero_stale = [&](uint8_t* stage, int depth, int kb, int blocks) {
    const int valid = depth - kb * kBK, stale = 16 - (valid & 15);
    for (int i = lane; i < blocks * stale * 8; i += 32) {
      const int q = i & 7, row = valid + (i >> 3) % stale, blk = (i >> 3) / stale;
      *reinterpret_cast<uint4*>(stage + blk * 8192 + row * 128 + q * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    __syncwarp();
  };

  if (wid == 0) {
    // ---- producer -------------------------------------------------------------
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int t = pair; t < total && ok; t += pairs) {
        const Tile r = tile_of(t);
        const int depth = MODE == kWeights ? seg_rows[r.e] : P.kdim;
        const int nkb = (depth + kBK - 1) / kBK;
        const int half = ((r.rows + 31) & ~31) / 2;  // columns of D from each CTA's operand
        const int boxes = MODE == kWeights ? (half + 63) >> 6 : (half + kBox - 1) / kBox;
        const uint32_t bytes = (uint32_t)kABytes + (uint32_t)boxes * (MODE == kWeights ? 8192u : kBox * 128u);
        const int row = seg_off[r.e] + (MODE == kWeights ? 0 : r.row0 + (int)rank * half);
        const int col = r.row0 + (int)rank * half;                     // weights gradient
        const int ch = r.c * kTileM + (int)rank * (GATED ? kBM / 2 : kBM);
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const int s = it % kStages;
          if (!wait(&empty[s], ((it / kStages) & 1u) ^ 1u)) {
            ok = false;
            break;
          }
          uint8_t* a = smem + s * kStageBytes;
          uint8_t* b = a + kABytes;
          // both CTAs' copies complete on the even CTA's barrier, except that an odd CTA's
          // slice with stale rows passes through that CTA's hands first
          uint32_t bar = even_addr(&full[s]);
          const bool apart = stale_tail(depth, kb);
          if (rank == 0) {
            mbar_arrive_expect_tx(&full[s], apart ? bytes : 2u * bytes);
          } else if (apart) {
            mbar_arrive_expect_tx(&full[s], bytes);
            bar = smem_addr(&full[s]);
          }
          if constexpr (MODE == kFwd) {
            tma_load_3d(a, &P.ma, kb * kBK, ch, r.e, bar);
            if constexpr (GATED) tma_load_3d(a + kABytes / 2, &P.ma, kb * kBK, P.M + ch, r.e, bar);
            for (int i = 0; i < boxes; ++i)
              tma_load_2d(b + i * kBox * 128, &P.mb, kb * kBK, row + i * kBox, bar);
          } else if constexpr (MODE == kRows) {
            tma_load_3d(a, &P.ma, ch, kb * kBK, r.e, bar);
            tma_load_3d(a + 8192, &P.ma, ch + 64, kb * kBK, r.e, bar);
            for (int i = 0; i < boxes; ++i)
              tma_load_2d(b + i * kBox * 128, &P.mb, kb * kBK, row + i * kBox, bar);
          } else {
            tma_load_2d(a, &P.ma, ch, row + kb * kBK, bar);
            tma_load_2d(a + 8192, &P.ma, ch + 64, row + kb * kBK, bar);
            for (int i = 0; i < boxes; ++i)
              tma_load_2d(b + i * 8192, &P.mb, col + i * 64, row + kb * kBK, bar);
          }
        }
      }
      if (!ok) {  // copies in flight land before the pair ends
        if (rank == 0)
          for (uint32_t j = it > kStages ? it - kStages : 0; j < it; ++j)
            mbar_wait_bounded(&full[j % kStages], (j / kStages) & 1u, 1000000ull);
        else
          mbar_wait_bounded(&drain, 1u ^ 1u, 1000000ull);  // a pause; nothing arrives
      }
    }
    __syncwarp();
  } else if (wid == 1 && rank == 0) {
    // ---- matrix instructions ----------------------------------------------------
    constexpr uint32_t a_mn = MODE == kFwd ? 0u : 1u, b_mn = MODE == kWeights ? 1u : 0u;
    uint32_t it = 0, nacc = 0, fix_par = 0;  // bit s: parity of fixed[s]'s next phase
    bool ok = true;
    for (int t = pair; t < total && ok; t += pairs) {
      const Tile r = tile_of(t);
      const int depth = MODE == kWeights ? seg_rows[r.e] : P.kdim;
      const int nkb = (depth + kBK - 1) / kBK;
      if (nkb == 0) continue;
      const uint32_t acc = nacc & 1u;
      if (!warp_wait(&tempty[acc], ((nacc >> 1) & 1u) ^ 1u)) break;
      tc_fence_after();
      ++nacc;
      const uint32_t d = tmem + acc * 256u;
      const int n = (r.rows + 31) & ~31;
      const uint32_t idesc = umma_idesc(2 * kBM, (uint32_t)n, a_mn, b_mn);
      for (int kb = 0; kb < nkb; ++kb, ++it) {
        const int s = it % kStages;
        if (!warp_wait(&full[s], (it / kStages) & 1u)) {
          ok = false;
          break;
        }
        uint8_t* a = smem + s * kStageBytes;
        int ksteps = kBK / 16;
        if constexpr (MODE == kWeights) ksteps = (min(kBK, depth - kb * kBK) + 15) >> 4;
        if (stale_tail(depth, kb)) {
          zero_stale(a, depth, kb, 2 + ((n / 2 + 63) >> 6));
          if (!warp_wait(&fixed[s], (fix_par >> s) & 1u)) {
            ok = false;
            break;
          }
          fix_par ^= 1u << s;
        }
        tc_fence_after();
        if (lane == 0) {
          const uint32_t sa = smem_addr(a), sb = sa + kABytes;
          for (int q = 0; q < ksteps; ++q) {
            const uint64_t da = a_mn ? umma_desc(sa + q * 2048, 8192, 1024)
                                     : umma_desc(sa + q * 32, 16, 1024);
            const uint64_t db = b_mn ? umma_desc(sb + q * 2048, 8192, 1024)
                                     : umma_desc(sb + q * 32, 16, 1024);
            umma_f16(d, da, db, idesc, kb > 0 || q > 0);
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
  } else if (wid == 1 && MODE == kWeights) {
    // ---- odd CTA: its stale rows ------------------------------------------------
    uint32_t it = 0, par = 0;  // bit s: parity of full[s]'s next phase here
    for (int t = pair; t < total; t += pairs) {
      const Tile r = tile_of(t);
      const int depth = seg_rows[r.e];
      const int nkb = (depth + kBK - 1) / kBK;
      if (nkb == 0) continue;
      if (stale_tail(depth, nkb - 1)) {
        const int n = (r.rows + 31) & ~31;
        const int s = (int)((it + nkb - 1) % kStages);
        if (!warp_wait(&full[s], (par >> s) & 1u)) break;
        par ^= 1u << s;
        zero_stale(smem + s * kStageBytes, depth, nkb - 1, 2 + ((n / 2 + 63) >> 6));
        if (lane == 0) mbar_arrive_cluster(even_addr(&fixed[s]));
      }
      it += nkb;
    }
  } else if (wid >= 4) {
    // ---- epilogue ---------------------------------------------------------------
    // Warps 4..7 and 8..11: quarter q (rows 32q..32q+31) of the accumulator, in
    // turn every second block of 32 columns.  A block is staged in the warp's
    // 2 KiB as 32 rows of 64 bytes, 16-byte pieces swizzled by the row, so that
    // both the column-wise and the row-wise accesses are free of conflicts.
    const int q = wid & 3, half = (wid - 4) >> 2;
    uint8_t* buf = epi + (wid - 4) * 2048;
    uint16_t* buf16 = reinterpret_cast<uint16_t*>(buf);
    const int frow = lane >> 2, fcol = (lane & 3) * 8;
    // piece (row, lane & 3) of the staged block
    auto piece = [&](int row) {
      return reinterpret_cast<uint4*>(buf + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) << 4));
    };
    // this lane's column of a staged row
    auto cell = [&](int row) {
      return buf16 + row * 32 + (((lane >> 3) ^ ((row >> 1) & 3)) << 3) + (lane & 7);
    };
    // the first 8 * n8 staged rows -> rows of `dst`, `stride` elements apart, 64
    // bytes each (widths are multiples of 8 elements)
    auto flush = [&](uint16_t* dst, size_t stride, int nrows, int ncols, int n8) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rr = i * 8 + frow;
        if (i < n8 && rr < nrows && fcol < ncols) st16(dst + (size_t)rr * stride + fcol, *piece(rr));
      }
      __syncwarp();
    };
    uint32_t nacc = 0, nswap = 0;
    bool ok = true;
    for (int t = pair; t < total && ok; t += pairs) {
      const Tile r = tile_of(t);
      const bool empty_sum = MODE == kWeights && seg_rows[r.e] == 0;
      const uint32_t acc = nacc & 1u;
      if (!empty_sum) {
        if (!warp_wait(&tfull[acc], (nacc >> 1) & 1u)) break;
        tc_fence_after();
        ++nacc;
      }
      const uint32_t d = tmem + acc * 256u + ((uint32_t)(q * 32) << 16);
      // this warp's first channel (gated: of the half that it holds)
      const int ch0 = GATED ? r.c * kTileM + (int)rank * 64 + (q & 1) * 32
                            : r.c * kTileM + (int)rank * kBM + q * 32;
      const int nc = P.M - ch0;
      const int nchunks = (r.rows + 31) >> 5;
      if constexpr (MODE == kWeights) {
        uint16_t* dst = P.out + ((size_t)r.e * P.M + ch0) * P.cols + r.row0;
        for (int j = half; j < nchunks; j += 2) {
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
          for (int i = 0; i < 4; ++i) {
            uint32_t p[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
              p[u] = pack2(__uint_as_float(v[8 * i + 2 * u]), __uint_as_float(v[8 * i + 2 * u + 1]));
            *reinterpret_cast<uint4*>(buf + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) =
                make_uint4(p[0], p[1], p[2], p[3]);
          }
          flush(dst + j * 32, (size_t)P.cols, nc, r.rows - j * 32, 4);
        }
      } else {
        const int ch = ch0 + lane;
        const bool up_half = GATED && q >= 2;
        float b0 = 0.0f;
        if constexpr (MODE == kFwd) {
          if (P.bias != nullptr && ch < P.M)
            b0 = __ldg(P.bias + (size_t)r.e * P.M * (GATED ? 2 : 1) + (up_half ? P.M : 0) + ch);
        }
        const int64_t row = (int64_t)seg_off[r.e] + r.row0;
        for (int j = half; j < nchunks; j += 2) {
          const int64_t row_j = row + j * 32;
          const int nr = r.rows - j * 32;
          // tokens whose results this warp writes: all 32, or gated its half
          const int tok0 = up_half ? 16 : 0;
          constexpr int kTok = GATED ? 16 : 32;
          // the residual's block, on its way while the accumulator is read
          uint4 res[MODE == kFwd ? kTok / 8 : 1];
          if constexpr (MODE == kFwd) {
            if (P.residual != nullptr) {
              const uint16_t* src = P.residual + (row_j + tok0) * P.M + ch0;
#pragma unroll
              for (int i = 0; i < kTok / 8; ++i) {
                const int rr = i * 8 + frow;
                res[i] = rr + tok0 < nr && fcol < nc
                             ? *reinterpret_cast<const uint4*>(src + (size_t)rr * P.M + fcol)
                             : make_uint4(0, 0, 0, 0);
              }
            }
          }
          uint32_t v[32];
          tmem_ld32(d + j * 32, v);
          tmem_ld_wait();
          // this lane holds one channel of 32 tokens: staged token-major
          float z[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) z[i] = __uint_as_float(v[i]) + b0;
          if constexpr (MODE == kFwd) {
            if (P.pre != nullptr) {
              const size_t wide = (size_t)P.M * (GATED ? 2 : 1);
#pragma unroll
              for (int i = 0; i < 32; ++i) *cell(i) = to_bf16(z[i]);
              flush(P.pre + row_j * wide + (up_half ? P.M : 0) + ch0, wide, nr, nc, 4);
            }
          }
          if constexpr (GATED) {
            // lanes 0..63 of the accumulator are gates, 64..127 the same channels' ups.
            // The gate's warp takes tokens 0..15, the up's 16..31: each hands the other
            // its 16 values through its staging block, in fp32.
            uint64_t* bar = &swap[half * 2 + (q & 1)];
            float* mine = reinterpret_cast<float*>(buf);
            const float* theirs = reinterpret_cast<const float*>(epi + ((wid - 4) ^ 2) * 2048);
#pragma unroll
            for (int i = 0; i < 16; ++i) mine[i * 32 + lane] = up_half ? z[i] : z[16 + i];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
            if (!warp_wait(bar, nswap++ & 1u)) {
              ok = false;
              break;
            }
            float other[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) other[i] = theirs[i * 32 + lane];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
            if (!warp_wait(bar, nswap++ & 1u)) {
              ok = false;
              break;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float g = up_half ? other[i] : z[i], u = up_half ? z[16 + i] : other[i];
              z[i] = g * sigmoid_f(g) * u;
            }
          } else if constexpr (MODE == kFwd) {
            if (P.act == MOE_ACT_RELU) {
#pragma unroll
              for (int i = 0; i < 32; ++i) z[i] = z[i] < 0.0f ? 0.0f : z[i];
            } else if (P.act == MOE_ACT_GELU) {
#pragma unroll
              for (int i = 0; i < 32; ++i) z[i] = gelu_f(z[i]);
            } else if (P.act == MOE_ACT_SILU) {
#pragma unroll
              for (int i = 0; i < 32; ++i) z[i] = z[i] * sigmoid_f(z[i]);
            }
          }
          if constexpr (MODE == kFwd) {
            if (P.residual != nullptr) {
              // through the staging block to this lane's column; added in fp32
#pragma unroll
              for (int i = 0; i < kTok / 8; ++i) *piece(i * 8 + frow) = res[i];
              __syncwarp();
#pragma unroll
              for (int i = 0; i < kTok; ++i) z[i] += bf16lo(*cell(i));
            }
          }
#pragma unroll
          for (int i = 0; i < kTok; ++i) *cell(i) = to_bf16(z[i]);
          flush(P.out + (row_j + tok0) * P.M + ch0, (size_t)P.M, nr - tok0, nc, kTok / 8);
        }
      }
      if (!empty_sum) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(even_addr(&tempty[acc]));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the pair's copies, matrix instructions and arrivals are done
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
  int64_t pairs = max_tiles < env.num_sms / 2 ? max_tiles : env.num_sms / 2;
  if (pairs < 1) pairs = 1;
  return launch_pdl(env, kernel, dim3((unsigned)(2 * pairs)), dim3(kGemmThreads), smem, P);
}

// Token tiles of `bn` rows there can be at most: full ones, and a partial one
// for each expert that can hold a row.
int64_t max_token_tiles(int64_t assignments, int E, int64_t bn) {
  return assignments / bn + (assignments < E ? assignments : E);
}

}  // namespace

bool expert_tiles_fit(int64_t assignments, int E, int in, int wide) {
  const int64_t ct = (wide + kBM - 1) / kBM, it = (in + kBM - 1) / kBM;
  const int64_t tt = max_token_tiles(assignments, E, kBN);
  return tt * (ct > it ? ct : it) < (int64_t(1) << 31) && (int64_t)E * ct * it < (int64_t(1) << 31);
}

cudaError_t launch_expert_matmul(const LaunchEnv& env, const ExpertMatmul& a) {
  const bool gated = a.act == MOE_ACT_SWIGLU;
  const int wide = gated ? 2 * a.out_features : a.out_features;
  GemmParams P = {};
  cudaError_t err = make_map(&P.ma, a.w, a.in_features, wide, a.E, gated ? kBM / 2 : kBM);
  if (err != cudaSuccess) return err;
  err = make_map(&P.mb, a.x, a.in_features, a.N, 0, kBox);
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
  const int64_t tt = max_token_tiles(a.assignments, a.E, kBN);
  if (gated) return launch_gemm<kFwd, true>(env, P, tt * ((P.M + kBM - 1) / kBM));
  return launch_gemm<kFwd, false>(env, P, tt * ((P.M + 2 * kBM - 1) / (2 * kBM)));
}

cudaError_t launch_expert_grad_rows(const LaunchEnv& env, const ExpertMatmul& a, const void* dz,
                                    void* grad_x) {
  const int wide = a.act == MOE_ACT_SWIGLU ? 2 * a.out_features : a.out_features;
  GemmParams P = {};
  cudaError_t err = make_map(&P.ma, a.w, a.in_features, wide, a.E, kBK);
  if (err != cudaSuccess) return err;
  err = make_map(&P.mb, dz, wide, a.N, 0, kBox);
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
  const int64_t ct = (P.M + 2 * kBM - 1) / (2 * kBM);
  return launch_gemm<kRows, false>(env, P, max_token_tiles(a.assignments, a.E, kBN) * ct);
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
  const int64_t tiles = (int64_t)a.E * ((wide + 2 * kBM - 1) / (2 * kBM)) *
                        ((a.in_features + kBN - 1) / kBN);
  return launch_gemm<kWeights, false>(env, P, tiles);
}

}  // namespace moe
