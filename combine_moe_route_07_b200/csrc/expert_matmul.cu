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
// Persistent pairs of CTAs (cta_group::2), one CTA per SM: in each CTA two producer
// threads (one an operand) feed a ring of shared memory by tensor-map copies (64-deep
// slices, 128-byte swizzle; a slice takes the bytes its tile's rows need, so the ring
// holds six full slices of 32 KiB or eight narrow ones), one thread of the even CTA
// issues the matrix instructions of both, and eight warps of each drain the
// accumulator of the previous tile meanwhile (two accumulators in tensor memory).  A
// pair shares its operands: a 256 x 256 tile costs each SM 32 KiB of copies per
// slice, where one CTA alone would move 48 KiB for the same work.  With swiglu a
// tile is 128 channels: gates in lanes 0..63 of each CTA's accumulator, the same
// channels' ups in lanes 64..127.  Every wait is bounded.
//
// What decides, by size (one B200, short runs at 1.9 GHz; long ones are held to the
// board's 1000 W, down to 1.2 GHz, and take a fifth longer):
//   18944 rows, 4096 x 2048, one expert: 208 us, 1530 TFLOP/s; tensor pipe 90 % active
//   64 experts x 4 rows, 4096 x 2048: 172 us, 6.25 TB/s: the weights' stream
//   64 experts x 256 rows: 243 us, 1130 TFLOP/s and 5.2 TB/s: both
//   its weights gradient: 305 us, 900 TFLOP/s, 1.07 GB written at 3.5 TB/s (a plain
//     fill of as much takes 270 us)
// Most of the way there was the length of the issuing threads' loops: behind a test
// of the lane number every copy and matrix instruction sits in a loop over the lanes
// (about 100 ns each; elect.sync removes it), and one producer thread for both
// operands took 900 cycles a slice.
#include <limits.h>
#include <math.h>

#include "block_scan.cuh"
#include "common.cuh"
#include "kernels.h"
#include "umma.cuh"

namespace moe {

namespace {

constexpr int kBK = 64;       // contraction depth of a stage
constexpr int kBM = 128;      // rows of the M operand on each CTA of a pair
constexpr int kBN = 256;      // columns of one accumulator
constexpr int kABytes = kBM * kBK * 2;
constexpr int kSlots = 8;     // slices in flight, at most (a power of two)
constexpr int kEpiWarps = 8;
constexpr int kGemmThreads = (4 + kEpiWarps) * 32;
constexpr int kEpiBytes = kEpiWarps * 4096;  // two 32 x 32 bf16 blocks a warp, or one 32 x 64
constexpr int kMaxSlice = kABytes + 128 * kBK * 2;
constexpr int kTmemCols = 512;
// The longest wait: two seconds, and 20 ns for each row (the weights gradient of one
// expert is one tile's contraction over all its rows: about 6 ns a row).
constexpr uint64_t kWaitNs = 2000000000ull, kWaitRowNs = 20ull;

enum { kFwd = 0, kRows = 1, kWeights = 2 };

struct GemmParams {
  CUtensorMap ma;  // M operand: weights [E][W][K]; weights gradient: dz [N][W]
  CUtensorMap mb[3];  // N operand, x or dz [N][..], in boxes of 32, 64 and 128 rows
                      // (weights gradient: one of 64)
  CUtensorMap mo, mp;  // out and pre, in boxes of 32 x 32
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
  int adapt;   // few tiles: choose their height by the rounds they take
  int smem;    // bytes of dynamic shared memory
  int sorted;  // experts in descending order of their rows (see my_tile)
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

// gelu(z) = z * Phi(z).
__device__ __forceinline__ float gelu_f(float z) {
  float e;
  const float tail = normal_tail(z, &e);
  return z * (z < 0.0f ? tail : 1.0f - tail);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A tile: its expert, channel tile, first row (weights gradient: column) and rows;
// n columns of D.  (Tiles of up to 512 tokens over two accumulators read the
// weights once instead of twice, but leave nothing for the epilogue to overlap with:
// Prefill's first product was as fast, a dense product of 16384 rows a third slower.)
struct Tile {
  int e, seg, c, row0, rows, n;  // seg: the expert's place in the segment table
};

// Tile heights to choose from: 256 - 32 c.
constexpr int kHeights = 8;
// Time of a 64-deep slice of a tile of n rows, in cycles: the matrix instructions'
// 2 n, or what bringing its operands costs (measured: 335 ns for the narrowest, 450
// for 256 rows with weights from HBM).
__device__ __forceinline__ int slice_cost(int n) { return max(2 * n, 230 + (4 * n) / 5); }

// Token rows that copies bring for `half` (a multiple of 16, up to 128) wanted:
// one box of 32, 64 or 128, or 64 + 32.  Few large copies: with boxes of 32
// rows alone a 256-column tile ran at 1230 TFLOP/s, with one of 128 at 1340.
__device__ __forceinline__ int box_rows(int half) { return (half + 31) & ~31; }

// The part of a wait that is not over at once; false: it gave up, or another
// role of this CTA did.
__device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, int* abort_flag,
                                       uint64_t limit_ns, WsHeader* hdr) {
  volatile int* stop = abort_flag;
  uint64_t t0 = 0;
  for (unsigned it = 1; it < (1u << 24); ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0u) {
      const uint64_t now = global_ns();
      if (t0 == 0) t0 = now;
      if (*stop != 0 || now - t0 > limit_ns) break;
    }
  }
  if (*stop == 0) report(hdr, MOE_ERR_DEVICE_TIMEOUT, blockIdx.x);
  *stop = 1;
  return false;
}

template <int MODE, bool GATED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
    expert_gemm_kernel(const __grid_constant__ GemmParams P) {
  constexpr int kTileM = GATED ? kBM : 2 * kBM;  // output channels of a pair's tile
  extern __shared__ uint8_t smem_raw[];
  // full, tempty and fixed are waited on by the even CTA only.  A slot's barriers see at
  // most one phase at a time: the slot is used again only once the instructions that
  // read it are done.
  __shared__ uint64_t full[kSlots], empty[kSlots], tfull[2], tempty[2], drain;
  // weights gradient, slices with stale rows: this CTA's half has landed; both
  // CTAs' stale rows are zero
  __shared__ uint64_t landed[kSlots], fixed[kSlots];
  __shared__ uint64_t swap[4];      // gated: between the two warps of a channel block
  __shared__ int taken[2][kSlots];  // producers: bytes of the slices in flight
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ unsigned long long rows_sum;
  __shared__ int tiles_at[kHeights];
  __shared__ int32_t warp_tot[kGemmThreads / 32];
  // The segment table: offsets, rows, exclusive prefix of token tiles [E+1] (forward /
  // rows), and the experts in the table's order.  Behind it, from a 1024-byte boundary
  // on, the operand ring in whole KiB, and the staging blocks.
  int32_t* seg_off = reinterpret_cast<int32_t*>(smem_raw);
  int32_t* seg_rows = seg_off + P.E;
  int32_t* first = seg_rows + P.E;
  int32_t* expert = first + P.E + 1;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(expert + P.E) + 1023) & ~uintptr_t(1023));
  const int ring = (int)(smem_raw + P.smem - smem - kEpiBytes) & ~1023;
  uint8_t* epi = smem + ring;

  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  if (tid == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&landed[s], 1);
      mbar_init(&fixed[s], 2);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&tfull[s], 1);
      mbar_init(&tempty[s], 2 * kEpiWarps);
    }
    for (int s = 0; s < 4; ++s) mbar_init(&swap[s], 2);
    mbar_init(&drain, 1);
    abort_flag = 0;
    rows_sum = 0ull;
    for (int c = 0; c < kHeights; ++c) tiles_at[c] = 0;
    mbar_fence_init();
    tma_prefetch_map(&P.ma);
    tma_prefetch_map(&P.mb[0]);
  }
  if (wid == 1) tmem_alloc(&tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the other CTA's barriers are ready too
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  unsigned long long my_rows = 0ull;
  constexpr int kMine = (1024 + kGemmThreads - 1) / kGemmThreads;
  Segment seg[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int e = tid + i * kGemmThreads;
    if (e < P.E) {
      seg[i] = segment(P, e, blockIdx.x == 0);
      my_rows += (unsigned long long)seg[i].rows;
      if (P.sorted) first[e] = seg[i].rows;
    }
  }
  if (my_rows != 0ull) atomicAdd(&rows_sum, my_rows);
  const int ctiles = (P.M + kTileM - 1) / kTileM;
  int height = kBN;
  if (MODE != kWeights && P.adapt) {
    // Fewer full tiles than pairs: the height whose rounds take least, which hands idle
    // pairs a part.
#pragma unroll
    for (int c = 0; c < kHeights; ++c) {
      int n = 0;
#pragma unroll
      for (int i = 0; i < kMine; ++i)
        if (tid + i * kGemmThreads < P.E) n += (seg[i].rows + kBN - 32 * c - 1) / (kBN - 32 * c);
      n = (int)__reduce_add_sync(kFull, (unsigned)n);
      if (lane == 0 && n > 0) atomicAdd(&tiles_at[c], n);
    }
    __syncthreads();
    // (at most one round at the largest height: everything fits 32 bits)
    uint32_t best = 0xffffffffu;
    for (int c = 0; c < kHeights; ++c) {
      const uint32_t rounds = ((uint32_t)tiles_at[c] * ctiles + pairs - 1) / pairs;
      const uint32_t cost = rounds * slice_cost(kBN - 32 * c);
      if (cost < best) {
        best = cost;
        height = kBN - 32 * c;
      }
    }
  }
  int at[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) at[i] = tid + i * kGemmThreads;
  if (P.sorted) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int e = tid + i * kGemmThreads;
      if (e < P.E) {
        int before = 0;
        for (int j = 0; j < P.E; ++j) {
          const int rj = first[j];
          before += (rj > seg[i].rows || (rj == seg[i].rows && j < e)) ? 1 : 0;
        }
        at[i] = before;
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int e = tid + i * kGemmThreads;
    if (e < P.E) {
      seg_off[at[i]] = seg[i].off;
      seg_rows[at[i]] = seg[i].rows;
      expert[at[i]] = e;
      if (MODE != kWeights) first[at[i]] = (seg[i].rows + height - 1) / height;
    }
  }
  __syncthreads();
  const uint32_t tmem = tmem_slot;
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

  // Wait for a phase; false: it gave up, or another role did.
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (mbar_try_wait(bar, parity)) return true;
    return wait_long(bar, parity, &abort_flag, kWaitNs + kWaitRowNs * (uint64_t)P.max_rows, P.hdr);
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
      r.seg = t / (ctiles * nt);
      r.e = expert[r.seg];
      const int u = t - r.seg * ctiles * nt;
      r.c = u / nt;
      r.row0 = (u - r.c * nt) * kBN;  // first column
      r.rows = min(kBN, P.cols - r.row0);
      r.n = (r.rows + 31) & ~31;
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
      r.e = expert[lo];
      r.seg = lo;
      r.c = v / nb;
      r.row0 = n * per;
      r.rows = min(per, seg_rows[lo] - r.row0);
      r.n = (r.rows + 31) & ~31;
    }
    return r;
  };
  // The j-th tile of this pair, -1 if it has none in that round.  Tiles are dealt
  // out in rounds.  Sorted experts: every second round in reverse, so that each
  // pair gets about the same work, and half of the pairs walk their rounds
  // backwards, so that large tiles (bound by the tensor cores) and small ones
  // (bound by HBM) run side by side.
  const int rounds = (total + pairs - 1) / pairs;
  auto my_tile = [&](int j) -> int {
    int t;
    if (P.sorted) {
      const int round = pair < (pairs >> 1) ? j : rounds - 1 - j;
      t = round * pairs + ((round & 1) ? pairs - 1 - pair : pair);
    } else {
      t = j * pairs + pair;
    }
    return t < total ? t : -1;
  };

  // The ring: a slice of a tile takes the bytes it needs (the M operand's 16 KiB and
  // the rows of the N operand), behind the one before it or, where it does not fit
  // there, at the ring's start.  Every role places the slices alike.
  auto slice_bytes = [&](const Tile& r) -> int {
    return kABytes + (MODE == kWeights ? ((r.n / 2 + 63) >> 6) * 8192
                                       : box_rows(r.n / 2) * (kBK * 2));
  };
  auto place = [&](int& head, int bytes) -> int {
    if (head + bytes > ring) head = 0;
    const int at = head;
    head += bytes;
    return at;
  };
  // Rows of the last slice that belong to the expert, when fewer than its
  // 16-deep steps take in (weights gradient).
  auto stale_tail = [&](int depth, int k0) -> bool {
    return MODE == kWeights && k0 + kBK > depth && (depth & 15) != 0;
  };
  // Rows behind the expert's last one are another expert's, or never written.
  // Steps wholly behind it are skipped; in the last step they become zero in
  // both operands (zero times NaN is not zero).  One warp, on this CTA's half.
  auto zero_stale = [&](uint8_t* slice, int depth, int k0, int blocks) {
    const int valid = depth - k0, end = (valid + 15) & ~15;
    for (int row = valid + (lane >> 3); row < end; row += 4) {
      uint8_t* at = slice + row * 128 + (lane & 7) * 16;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (b < blocks) *reinterpret_cast<uint4*>(at + b * 8192) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    __syncwarp();
  };

  if (wid == 0 || wid == 2) {
    // ---- producers: warp 0 the M operand, warp 2 the N operand --------------------
    if (elect_one()) {
      uint32_t it = 0, old = 0;  // slices issued, and those known to be used up
      int head = 0, room = ring;
      int* const mine = taken[wid >> 1];
      const uint32_t even_full = even_addr(&full[0]), own_landed = smem_addr(&landed[0]);
      bool ok = true;
      for (int j = 0; j < rounds && ok; ++j) {
        const int t = my_tile(j);
        if (t < 0) continue;
        const Tile r = tile_of(t);
        const int depth = MODE == kWeights ? seg_rows[r.seg] : P.kdim;
        const int half = r.n / 2;  // columns of an accumulator from each CTA's operand
        const int bytes = slice_bytes(r);
        const int row = seg_off[r.seg] + (MODE == kWeights ? 0 : r.row0 + (int)rank * half);
        const int col = r.row0 + (int)rank * half;  // weights gradient
        const int ch = r.c * kTileM + (int)rank * (GATED ? kBM / 2 : kBM);
        const int fetched = box_rows(half);
        for (int k0 = 0; k0 < depth; k0 += kBK, ++it) {
          const uint32_t s = it % kSlots;
          int need = bytes;
          if (head + bytes > ring) {  // (as place())
            need += ring - head;
            head = 0;
          }
          // the oldest slices make room: for the bytes, and for the slot
          while (room < need || it - old == kSlots) {
            const uint32_t o = old % kSlots;
            if (!wait(&empty[o], (old / kSlots) & 1u)) {
              ok = false;
              break;
            }
            room += mine[o];
            ++old;
          }
          if (!ok) break;
          room -= need;
          mine[s] = need;
          uint8_t* a = smem + head;
          head += bytes;
          // both CTAs' copies complete on the even CTA's barrier; of slices with stale
          // rows each CTA's on its own, whose fixer passes them on
          const bool apart = stale_tail(depth, k0);
          const uint32_t bar = (apart ? own_landed : even_full) + s * 8;
          if (wid == 0) {
            if (apart)
              mbar_arrive_expect_tx(&landed[s], (uint32_t)bytes);
            else if (rank == 0)
              mbar_arrive_expect_tx(&full[s], (uint32_t)(2 * bytes));
            if constexpr (MODE == kWeights) {
              tma_load_2d(a, &P.ma, ch, row + k0, bar);
              tma_load_2d(a + 8192, &P.ma, ch + 64, row + k0, bar);
            } else if constexpr (MODE == kFwd) {
              tma_load_3d(a, &P.ma, k0, ch, r.e, bar);
              if constexpr (GATED) tma_load_3d(a + kABytes / 2, &P.ma, k0, P.M + ch, r.e, bar);
            } else {
              tma_load_3d(a, &P.ma, ch, k0, r.e, bar);
              tma_load_3d(a + 8192, &P.ma, ch + 64, k0, r.e, bar);
            }
          } else {
            uint8_t* b = a + kABytes;
            if constexpr (MODE == kWeights) {
              tma_load_2d(b, &P.mb[0], col, row + k0, bar);
              if (half > 64) tma_load_2d(b + 8192, &P.mb[0], col + 64, row + k0, bar);
            } else {
              if (fetched == 128) {
                tma_load_2d(b, &P.mb[2], k0, row, bar);
              } else if (fetched == 32) {
                tma_load_2d(b, &P.mb[0], k0, row, bar);
              } else {
                tma_load_2d(b, &P.mb[1], k0, row, bar);
                if (fetched == 96) tma_load_2d(b + 8192, &P.mb[0], k0, row + 64, bar);
              }
            }
          }
        }
      }
      if (!ok) {  // copies in flight land before the pair ends: they take microseconds
        const uint64_t t0 = global_ns();
        for (int i = 0; i < 100000 && global_ns() - t0 < 2000000ull; ++i) __nanosleep(1000);
      }
    }
    __syncwarp();
  } else if (wid == 1 && rank == 0) {
    // ---- matrix instructions: one thread of the even CTA --------------------------
    if (elect_one()) {
      constexpr uint32_t a_mn = MODE == kFwd ? 0u : 1u, b_mn = MODE == kWeights ? 1u : 0u;
      // a 16-deep step further: 32 bytes along K-major rows, 2048 over MN-major ones
      constexpr uint64_t sa16 = a_mn ? 128 : 2, sb16 = b_mn ? 128 : 2;
      const uint64_t da_ring = a_mn ? umma_desc(smem_addr(smem), 8192, 1024)
                                    : umma_desc(smem_addr(smem), 16, 1024);
      const uint64_t db_ring = b_mn ? umma_desc(smem_addr(smem) + kABytes, 8192, 1024)
                                    : umma_desc(smem_addr(smem) + kABytes, 16, 1024);
      uint32_t it = 0, nacc = 0;
      uint32_t full_par = 0, fix_par = 0;  // bit s: parity of full[s]'s, fixed[s]'s next phase
      int head = 0;
      bool ok = true;
      for (int j = 0; j < rounds && ok; ++j) {
        const int t = my_tile(j);
        if (t < 0) continue;
        const Tile r = tile_of(t);
        const int depth = MODE == kWeights ? seg_rows[r.seg] : P.kdim;
        if (depth == 0) continue;
        ok = wait(&tempty[nacc & 1u], ((nacc >> 1) & 1u) ^ 1u);
        if (!ok) break;
        tc_fence_after();
        const uint32_t idesc = umma_idesc(2 * kBM, (uint32_t)r.n, a_mn, b_mn);
        const int bytes = slice_bytes(r);
        const uint32_t d = tmem + (nacc & 1u) * 256u;
        for (int k0 = 0; k0 < depth; k0 += kBK, ++it) {
          const uint32_t s = it % kSlots;
          const int at = place(head, bytes);
          if (stale_tail(depth, k0)) {
            ok = wait(&fixed[s], (fix_par >> s) & 1u);
            fix_par ^= 1u << s;
          } else {
            ok = wait(&full[s], (full_par >> s) & 1u);
            full_par ^= 1u << s;
          }
          if (!ok) break;
          tc_fence_after();
          const uint64_t da = da_ring + (uint32_t)(at >> 4), db = db_ring + (uint32_t)(at >> 4);
          const int ksteps = MODE == kWeights ? (min(kBK, depth - k0) + 15) >> 4 : kBK / 16;
#pragma unroll
          for (int q = 0; q < kBK / 16; ++q)
            if (MODE != kWeights || q < ksteps)
              umma_f16(d, da + q * sa16, db + q * sb16, idesc, k0 > 0 || q > 0);
          umma_commit(&empty[s]);
        }
        if (!ok) break;
        umma_commit(&tfull[nacc & 1u]);
        ++nacc;
      }
      if (!ok) {  // what was issued ends before the pair does
        umma_commit(&drain);
        mbar_wait_bounded(&drain, 0u, kWaitNs);
      }
    }
    __syncwarp();
  } else if (wid == 3 && MODE == kWeights) {
    // ---- fixer: zeros for the stale rows of this CTA's half -------------------------
    uint32_t it = 0, par = 0;  // bit s: parity of landed[s]'s next phase
    int head = 0;
    for (int j = 0; j < rounds; ++j) {
      const int t = my_tile(j);
      if (t < 0) continue;
      const Tile r = tile_of(t);
      const int depth = seg_rows[r.seg];
      const int bytes = slice_bytes(r);
      for (int k0 = 0; k0 < depth; k0 += kBK, ++it) {
        const int at = place(head, bytes);
        if (!stale_tail(depth, k0)) continue;
        const uint32_t s = it % kSlots;
        if (!warp_wait(&landed[s], (par >> s) & 1u)) break;
        par ^= 1u << s;
        zero_stale(smem + at, depth, k0, bytes / 8192);
        if (lane == 0) mbar_arrive_remote(even_addr(&fixed[s]));
      }
    }
  } else if (wid >= 4) {
    // ---- epilogue ---------------------------------------------------------------
    // Warps 4..7 and 8..11: quarter q (rows 32q..32q+31) of an accumulator, in
    // turn every second block of 32 columns.  A block is staged as 32 rows of 64
    // bytes, 16-byte pieces swizzled by the row (the tensor map's 64-byte swizzle:
    // neither the column-wise nor the row-wise accesses conflict), and stored by a
    // tensor-map copy that runs while the warp goes on with its other staging
    // block.  Blocks that end inside (rows behind them belong to another expert,
    // or to nobody) are stored by the lanes.
    const int q = wid & 3, half = (wid - 4) >> 2;
    uint8_t* const blocks = epi + (wid - 4) * 4096;
    const int frow = lane >> 2, fcol = (lane & 3) * 8;
    uint32_t uses = 0;
    // A staging block.  Every use is one bulk group, empty or not: with at most one
    // group still reading, the use before last is done.
    auto open_block = [&]() -> uint8_t* {
      if (elect_one()) bulk_wait_read<1>();
      __syncwarp();
      return blocks + (uses++ & 1u) * 2048;
    };
    // piece (row, lane & 3) of a staged block
    auto piece = [&](uint8_t* buf, int row) {
      return reinterpret_cast<uint4*>(buf + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) << 4));
    };
    // Products by channel: a block of 32 channels x 32 tokens sits in fragments (see
    // tmem_ld16): value (h, j, i) of a thread, at 16h + 4j + i, is channel 16h + 8(i/2)
    // + lane/4 of token 8j + 2(lane%4) + i%2.  Four transposing block stores a block
    // bring it token-major into shared memory (one 2-byte store a value cost half as
    // much again as everything else here).
    const uint32_t t_addr =
        (uint32_t)((lane & 7) * 64 + (((lane >> 3) ^ ((lane & 7) >> 1)) << 4));
    auto load_block = [&](uint32_t addr, uint32_t(&v)[32]) {
      tmem_ld16(addr, v);
      tmem_ld16(addr + (16u << 16), v + 16);
    };
    // tokens 8j..8j+7 of z (row stride of a fragment group: 4 nj values) -> staged rows
    // 8r..8r+7
    auto stage8 = [&](uint8_t* buf, int r, const float* z, int j, int nj) {
      const float* a = z + 4 * j;
      const float* b = z + 4 * nj + 4 * j;
      stmatrix_t(smem_addr(buf) + t_addr + r * 512, pack2(a[0], a[1]), pack2(a[2], a[3]),
                 pack2(b[0], b[1]), pack2(b[2], b[3]));
    };
    // Token-major block of `box` rows at (row, ch) of a matrix `stride` wide, of which
    // `nrows` rows and `ncols` columns (a multiple of 8) are this expert's.
    auto close_tokens = [&](uint8_t* buf, const CUtensorMap* map, uint16_t* base, int64_t row,
                            int ch, int stride, int box, int nrows, int ncols) {
      if (nrows >= box) {
        fence_proxy_async_smem();
        __syncwarp();
        if (elect_one()) {
          if (ncols > 0) tma_store_2d(map, buf, ch, (int)row);
          bulk_commit();
        }
      } else {
        __syncwarp();
        uint16_t* dst = base + (size_t)row * stride + ch;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = i * 8 + frow;
          if (rr < nrows && fcol < ncols) st16(dst + (size_t)rr * stride + fcol, *piece(buf, rr));
        }
        __syncwarp();
        if (elect_one()) bulk_commit();
      }
    };
    uint32_t nacc = 0, nswap = 0;
    bool ok = true;
    for (int i = 0; i < rounds && ok; ++i) {
      const int t = my_tile(i);
      if (t < 0) continue;
      const Tile r = tile_of(t);
      const bool empty_sum = MODE == kWeights && seg_rows[r.seg] == 0;
      // this warp's first channel (gated: of the half that it holds)
      const int ch0 = GATED ? r.c * kTileM + (int)rank * 64 + (q & 1) * 32
                            : r.c * kTileM + (int)rank * kBM + q * 32;
      const int nc = P.M - ch0;
      const uint32_t acc = nacc & 1u;
      if (!empty_sum) {
        if (!warp_wait(&tfull[acc], (nacc >> 1) & 1u)) {
          ok = false;
          break;
        }
        tc_fence_after();
        ++nacc;
      }
      const uint32_t d = tmem + acc * 256u + ((uint32_t)(q * 32) << 16);
      const int row0 = r.row0, rows = r.rows;
      const int nchunks = (rows + 31) >> 5;
      if constexpr (MODE == kWeights) {
        // Warps 4..7 take columns 0..127, warps 8..11 the others, 64 at a time.  A lane
        // holds 32 columns of one row of dW; 32 rows of 128 bytes (16-byte pieces swizzled
        // by the row) are staged and stored as one box.  (Boxes of 32 x 32 held the
        // gradient of 256-row experts at 3.2 TB/s; a second staging block per warp, which
        // costs a stage of the ring, at 3.9 instead of 4.1.)
        const int col0 = half * 128, ncols = min(128, rows - col0);
        uint32_t v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0u;
        if (!empty_sum && ncols > 0) tmem_ld32(d + col0, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j * 32 < ncols) {
            uint8_t* buf = epi + (wid - 4) * 4096;
            if ((j & 1) == 0) {
              if (elect_one()) bulk_wait_read<0>();
              __syncwarp();
            }
            uint32_t w[16];
            if (!empty_sum) tmem_ld_wait(v);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              w[i] = pack2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
            if (!empty_sum && (j + 1) * 32 < ncols) tmem_ld32(d + col0 + (j + 1) * 32, v);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(buf + lane * 128 + ((((j & 1) * 4 + i) ^ (lane & 7)) << 4)) =
                  make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            if ((j & 1) != 0 || (j + 1) * 32 >= ncols) {
              fence_proxy_async_smem();
              __syncwarp();
              if (elect_one()) {
                if (nc > 0) tma_store_3d(&P.mo, buf, row0 + col0 + (j >> 1) * 64, ch0, r.e);
                bulk_commit();
              }
            }
          }
        }
      } else {
        const int64_t row = (int64_t)seg_off[r.seg] + row0;
        const bool up_half = GATED && q >= 2;
        // this thread's channels: ch0 + lane/4 + 8c
        float bias[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (MODE == kFwd && P.bias != nullptr) {
          const float* bp = P.bias + (size_t)r.e * P.M * (GATED ? 2 : 1) + (up_half ? P.M : 0) + ch0;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int ch = (lane >> 2) + 8 * c;
            if (ch < nc) bias[c] = __ldg(bp + ch);
          }
        }
        uint32_t next[32];
        if (half < nchunks) load_block(d + half * 32, next);
        for (int j = half; j < nchunks; j += 2) {
          const int64_t row_j = row + j * 32;
          const int nr = rows - j * 32;
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
          tmem_ld_wait(next);
          float z[32];
#pragma unroll
          for (int i = 0; i < 32; ++i)
            z[i] = __uint_as_float(next[i]) + bias[(i >> 4) * 2 + ((i >> 1) & 1)];
          if (j + 2 < nchunks) load_block(d + (j + 2) * 32, next);
          if constexpr (MODE == kFwd) {
            if (P.pre != nullptr) {
              const int wide = P.M * (GATED ? 2 : 1);
              uint8_t* buf = open_block();
#pragma unroll
              for (int i = 0; i < 4; ++i) stage8(buf, i, z, i, 4);
              // (a gate half's block may reach into the up half's columns: lane stores)
              const bool inside = !GATED || up_half || nc >= 32;
              close_tokens(buf, &P.mp, P.pre, row_j, (up_half ? P.M : 0) + ch0, wide,
                           inside ? 32 : INT_MAX, nr, nc);
            }
          }
          float y[kTok];  // the results: fragments of kTok / 8 token groups
          if constexpr (GATED) {
            // lanes 0..63 of the accumulator are gates, 64..127 the same channels' ups.
            // The gate's warp takes tokens 0..15, the up's 16..31: each hands the other
            // its 16 values a thread through a staging block, in fp32.
            uint64_t* bar = &swap[half * 2 + (q & 1)];
            uint8_t* buf = open_block();
            float4* mine = reinterpret_cast<float4*>(buf) + lane;
            const float4* theirs =
                reinterpret_cast<const float4*>(epi + ((wid - 4) ^ 2) * 4096 + (buf - blocks)) + lane;
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // (h, j) = (i / 2, i % 2 of the pair handed over)
              const int lo = (i >> 1) * 16 + (i & 1) * 4, hi = lo + 8;
              mine[i * 32] = up_half ? make_float4(z[lo], z[lo + 1], z[lo + 2], z[lo + 3])
                                     : make_float4(z[hi], z[hi + 1], z[hi + 2], z[hi + 3]);
            }
            __syncwarp();
            if (elect_one()) {
              bulk_commit();
              mbar_arrive(bar);
            }
            if (!warp_wait(bar, nswap++ & 1u)) {
              ok = false;
              break;
            }
            float4 other[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) other[i] = theirs[i * 32];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
            if (!warp_wait(bar, nswap++ & 1u)) {
              ok = false;
              break;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int lo = (i >> 1) * 16 + (i & 1) * 4, hi = lo + 8;
              const float o[4] = {other[i].x, other[i].y, other[i].z, other[i].w};
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const float g = up_half ? o[u] : z[lo + u], v = up_half ? z[hi + u] : o[u];
                y[i * 4 + u] = g * sigmoid_f(g) * v;
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = z[i];
            if (MODE == kFwd) {
              if (P.act == MOE_ACT_RELU) {
#pragma unroll
                for (int i = 0; i < 32; ++i) y[i] = z[i] < 0.0f ? 0.0f : z[i];
              } else if (P.act == MOE_ACT_GELU) {
#pragma unroll
                for (int i = 0; i < 32; ++i) y[i] = gelu_f(z[i]);
              } else if (P.act == MOE_ACT_SILU) {
#pragma unroll
                for (int i = 0; i < 32; ++i) y[i] = z[i] * sigmoid_f(z[i]);
              }
            }
          }
          uint8_t* buf = open_block();
          if constexpr (MODE == kFwd) {
            if (P.residual != nullptr) {
              // through the staging block into the fragments; added in fp32
#pragma unroll
              for (int i = 0; i < kTok / 8; ++i) *piece(buf, i * 8 + frow) = res[i];
              __syncwarp();
#pragma unroll
              for (int i = 0; i < kTok / 8; ++i) {
                uint32_t f[4];
                ldmatrix_t(smem_addr(buf) + t_addr + i * 512, f);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  float* at = y + (c >> 1) * (kTok / 2) + 4 * i + (c & 1) * 2;
                  at[0] += bf16lo(f[c]);
                  at[1] += bf16hi(f[c]);
                }
              }
              __syncwarp();
            }
          }
#pragma unroll
          for (int i = 0; i < kTok / 8; ++i) stage8(buf, i, y, i, kTok / 8);
          close_tokens(buf, &P.mo, P.out, row_j + tok0, ch0, P.M, kTok, nr - tok0, nc);
        }
      }
      if (!empty_sum) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(even_addr(&tempty[acc]));
      }
    }
    if (elect_one()) bulk_wait_all();
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

// bf16 tensor [d2][d1][d0] (d2 = 0: a matrix), boxes of box0 x box1 (64 wide:
// 128-byte swizzle, 32 wide: 64-byte), zeros outside.
cudaError_t make_map(CUtensorMap* map, const void* ptr, int64_t d0, int64_t d1, int64_t d2,
                     int box0, int box1) {
  const EncodeFn fn = encode_fn();
  if (fn == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {(cuuint64_t)d0, (cuuint64_t)d1, (cuuint64_t)d2};
  const cuuint64_t strides[2] = {(cuuint64_t)d0 * 2, (cuuint64_t)d0 * (cuuint64_t)d1 * 2};
  const cuuint32_t box[3] = {(cuuint32_t)box0, (cuuint32_t)box1, 1};
  const cuuint32_t es[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, d2 > 0 ? 3 : 2,
                        const_cast<void*>(ptr), dims, strides, box, es,
                        CU_TENSOR_MAP_INTERLEAVE_NONE,
                        box0 == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Token tiles of `bn` rows there can be at most: full ones, and a partial one
// for each expert that can hold a row.
int64_t max_token_tiles(int64_t assignments, int E, int64_t bn) {
  return assignments / bn + (assignments < E ? assignments : E);
}

constexpr int kSmemLimit = 227 * 1024;  // of a CTA, static and dynamic

template <int MODE, bool GATED>
cudaError_t launch_gemm(const LaunchEnv& env, GemmParams& P, int64_t max_tiles = 0) {
  constexpr int kTileM = GATED ? kBM : 2 * kBM;
  const int64_t all = env.num_sms / 2;
  if (MODE != kWeights) {
    const int64_t ct = (P.M + kTileM - 1) / kTileM;
    max_tiles = max_token_tiles(P.max_rows, P.E, kBN) * ct;
    // The tiles' height is chosen where full ones would not give every pair one: 300 rows of
    // 16384 -> 256 take 69 us instead of 78, 512 of 8192 -> 1024 38 instead of 42; near a full
    // round it can lose (64 tiles for 74 pairs, 2048 rows of 2048 -> 2048: 18.5 instead of
    // 17.7), but a limit at half a round loses as much in between.  With more
    // tiles lower ones cost more than an even last round gains, since each reads its weights:
    // 30000 rows of 2048 -> 2048 took 246 us instead of 201, 64 experts x 256 rows of 2048 ->
    // 2048 200 instead of 181.
    P.adapt = max_tiles <= all;
    if (P.adapt) max_tiles = max_token_tiles(P.max_rows, P.E, 32) * ct;
  }
  const auto kernel = expert_gemm_kernel<MODE, GATED>;
  static const int static_bytes = [&] {
    cudaFuncAttributes attr = {};
    return cudaFuncGetAttributes(&attr, (const void*)kernel) == cudaSuccess
               ? (int)attr.sharedSizeBytes
               : -1;
  }();
  if (static_bytes < 0) return cudaErrorInvalidDeviceFunction;
  // room for the table, the boundary behind it, the staging blocks and five of the
  // largest slices at E = 1024 (six up to E of about 160)
  static_assert(kSmemLimit - 1024 - (16 * 1024 + 4) - 1023 - kEpiBytes >= 5 * kMaxSlice, "five slices");
  const size_t smem = (size_t)(kSmemLimit - static_bytes);
  if (static_bytes > 1024) return cudaErrorInvalidConfiguration;
  P.smem = (int)smem;
  int per_sm = 1;
  cudaError_t err = blocks_per_sm((const void*)kernel, kGemmThreads, smem, &per_sm);
  if (err != cudaSuccess) return err;
  int64_t pairs = max_tiles < all ? max_tiles : all;
  if (pairs < 1) pairs = 1;
  return launch_pdl(env, kernel, dim3((unsigned)(2 * pairs)), dim3(kGemmThreads), smem, P);
}

void segments_of(GemmParams& P, const ExpertMatmul& a) {
  P.counts = a.counts;
  P.off = a.expert_off;
  P.hdr = a.hdr;
  P.N = a.N;
  P.max_rows = a.assignments;
  P.E = a.E;
  P.capacity = a.capacity;
  // ranking costs E^2 / 384 steps a CTA (4 us for 512 experts): where tiles are large
  // enough to differ, and few enough experts
  P.sorted = a.E > 1 && a.E <= 512 && a.assignments >= (int64_t)32 * a.E;
}

// The token operand's maps, and the tiles' shape.
cudaError_t token_operand(GemmParams& P, const ExpertMatmul& a, const void* rows, int cols) {
  for (int i = 0; i < 3; ++i) {
    const cudaError_t err = make_map(&P.mb[i], rows, cols, a.N, 0, 64, 32 << i);
    if (err != cudaSuccess) return err;
  }
  P.kdim = cols;
  // 18944 rows of 4096 -> 2048 (past the L2): 242 us with bands of 8, 251 of 16, 298 of 64, 238
  // of 1, which reads ragged experts' weights once a tile more (128 x 256 rows: 1 % slower)
  P.band = 8;
  return cudaSuccess;
}

int wide_features(const ExpertMatmul& a) {
  return a.act == MOE_ACT_SWIGLU ? 2 * a.out_features : a.out_features;
}

}  // namespace

bool expert_tiles_fit(int64_t assignments, int E, int in, int wide) {
  const int64_t ct = (wide + kBM - 1) / kBM, it = (in + kBM - 1) / kBM;
  const int64_t tt = max_token_tiles(assignments, E, 32);
  return tt * (ct > it ? ct : it) < (int64_t(1) << 31) && (int64_t)E * ct * it < (int64_t(1) << 31);
}

cudaError_t launch_expert_matmul(const LaunchEnv& env, const ExpertMatmul& a) {
  const bool gated = a.act == MOE_ACT_SWIGLU;
  const int wide = wide_features(a);
  GemmParams P = {};
  segments_of(P, a);
  cudaError_t err = make_map(&P.ma, a.w, a.in_features, wide, a.E, 64, gated ? kBM / 2 : kBM);
  if (err == cudaSuccess) err = token_operand(P, a, a.x, a.in_features);
  if (err == cudaSuccess) err = make_map(&P.mo, a.out, a.out_features, a.N, 0, 32, gated ? 16 : 32);
  if (err == cudaSuccess && a.pre != nullptr) err = make_map(&P.mp, a.pre, wide, a.N, 0, 32, 32);
  if (err != cudaSuccess) return err;
  P.bias = a.bias;
  P.residual = static_cast<const uint16_t*>(a.residual);
  P.out = static_cast<uint16_t*>(a.out);
  P.pre = static_cast<uint16_t*>(a.pre);
  P.M = a.out_features;
  P.act = a.act;
  return gated ? launch_gemm<kFwd, true>(env, P) : launch_gemm<kFwd, false>(env, P);
}

cudaError_t launch_expert_grad_rows(const LaunchEnv& env, const ExpertMatmul& a, const void* dz,
                                    void* grad_x) {
  const int wide = wide_features(a);
  GemmParams P = {};
  segments_of(P, a);
  cudaError_t err = make_map(&P.ma, a.w, a.in_features, wide, a.E, 64, kBK);
  if (err == cudaSuccess) err = token_operand(P, a, dz, wide);
  if (err == cudaSuccess) err = make_map(&P.mo, grad_x, a.in_features, a.N, 0, 32, 32);
  if (err != cudaSuccess) return err;
  P.out = static_cast<uint16_t*>(grad_x);
  P.M = a.in_features;
  return launch_gemm<kRows, false>(env, P);
}

cudaError_t launch_expert_grad_weights(const LaunchEnv& env, const ExpertMatmul& a, const void* dz,
                                       void* grad_w) {
  const int wide = wide_features(a);
  GemmParams P = {};
  segments_of(P, a);
  cudaError_t err = make_map(&P.ma, dz, wide, a.N, 0, 64, kBK);
  if (err == cudaSuccess) err = make_map(&P.mb[0], a.x, a.in_features, a.N, 0, 64, kBK);
  if (err == cudaSuccess) err = make_map(&P.mo, grad_w, a.in_features, wide, a.E, 64, 32);
  if (err != cudaSuccess) return err;
  P.out = static_cast<uint16_t*>(grad_w);
  P.M = wide;
  P.cols = a.in_features;
  const int64_t tiles = (int64_t)a.E * ((wide + 2 * kBM - 1) / (2 * kBM)) *
                        ((a.in_features + kBN - 1) / kBN);
  return launch_gemm<kWeights, false>(env, P, tiles);
}

}  // namespace moe
