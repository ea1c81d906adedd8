// Products over many ragged rows on tcgen05 tensor cores:
//
//     gated    [gate | up][i, :] = x[token(i), :] W[g(i)],  h = prob * silu(gate) * up
//     adapt    y[t, :] = x[t, :] W + u[t, :] b[ad(t)]^T          (W [K, N], b [A, N, R])
//     adaptT   the same with W given as [N, K]                   (the gradient of x)
//
// Tile: 256 rows x 256 accumulator columns on a pair of CTAs (cta_group::2),
// reduced 64 at a time through seven stage slots; CTA r owns rows 128 r .. 128 r
// + 127, whose fp32 accumulators (two buffers) sit in its tensor memory. (Or 512
// columns, four slots and one accumulator: see choose_halves.) The
// weights come by TMA. The rows of x are gathered by token with 16-byte
// cp.async, one warp per stage slot; where a CTA's rows are neighbouring tokens
// (adapt: requests one after another) they come as one TMA box instead (714
// cycles a step against 753). TMA's own gather of four rows is no way out: 75
// cycles an instruction, 2.5 times the whole product's time.
//
// gated: 128 of the accumulator's columns are gates and the other 128 the ups
// that belong to them (each CTA loads one of the two operands), so a thread of
// the epilogue finds both of its pair in its own lane, and neither is written
// unless the caller keeps them: h alone is a third of what a product of
// [M, 2F] and an activation over it would move.
//
// adapt: rows are taken in the order of their adapters, 256 at a time whatever
// the adapters' borders, so that no row of the shared product is padding. The
// low-rank part is more steps of the same reduction: for each adapter the tile
// meets, the A operand is u and the B operand b[ad], and the MMA writes only
// that adapter's accumulator lanes (disable-output-lane). Masking the output
// and not the operand keeps what another adapter's weights hold (infinities,
// NaN) out of the row: 0 * inf never happens. u is an operand of the tensor
// cores, so it comes as the sum of two values of the dtype (see LowRankForm): a
// low-rank step covers 32 ranks, their 32 hi and 32 lo parts fill the step's 64
// columns of A, and both meet the same rows of b. Two more MMAs a 32 ranks are
// hidden behind the step's copies; ranks above 32 take a step per 32.
//
// Warp roles per CTA: 0 TMA; 1 tensor-memory allocation and (even CTA) MMA
// issue; one gather warp per stage slot; eight epilogue warps an MMA. Tiles are
// statically interleaved over the clusters. Waits are bounded; when one runs
// out the kernel records PGG_ERR_TIMEOUT, drains its copies and MMAs, frees
// tensor memory and returns.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <cstring>

#include "pgg_epilogue.cuh"
#include "pgg_ops.h"
#include "pgg_ops_launch.h"
#include "pgg_ops_mma.cuh"
#include "pgg_ptx.cuh"

namespace pgg {
namespace {

constexpr int kFM = 128;   // rows per CTA (the pair's MMA M is 256)
constexpr int kFN = 256;   // MMA N
constexpr int kFK = 64;    // reduction per stage: one 128-byte row of A
constexpr int kPanel = kFK * 128;   // MN-major B panel: 64 k rows x 128 bytes (64 n)
constexpr int kABytes = kFM * 128;  // A: 128 rows x 128 bytes
constexpr int kHalfBytes = 2 * kPanel;  // B of one MMA: this CTA's 128 of the 256 columns
constexpr int kTmemCols = 512;
constexpr int kMaxStages = 7;

// H = 1: tiles of 256 accumulator columns, two accumulators. H = 2: 512 columns, one accumulator.
template <int H>
struct Cfg {
  static constexpr int kBBytes = H * kHalfBytes;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = H == 1 ? 7 : 4;
  static constexpr int kGatherWarps = kStages;
  // Eight epilogue warps an MMA: two share its lanes' quarter, each half of the columns. (A tile's
  // drain is bound by its stores, and takes 13,000 cycles with gate_up with four warps as with
  // eight; eight leave fewer columns a thread to unroll.)
  static constexpr int kEpiWarps = 8 * H;
  static constexpr int kEpiWarp0 = 2 + kGatherWarps;
  static constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
};

struct WideCtl {
  uint64_t full[kMaxStages];   // even CTA: weight bytes of both CTAs + rows gathered in both
  uint64_t empty[kMaxStages];  // each CTA: MMAs of the stage done (multicast commit)
  uint64_t tfull[2];           // each CTA: accumulator ready
  uint64_t tempty[2];          // even CTA: accumulator drained (epilogue warps x 2 CTAs)
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

template <int H>
constexpr int smem_bytes() {
  return Cfg<H>::kStages * Cfg<H>::kStageBytes + static_cast<int>(sizeof(WideCtl)) + 1024;
}
static_assert(smem_bytes<1>() <= 227 * 1024 && smem_bytes<2>() <= 227 * 1024,
              "shared memory per CTA");

__device__ __forceinline__ uint32_t cluster_id() { return blockIdx.x >> 1; }
__device__ __forceinline__ uint32_t n_clusters() { return gridDim.x >> 1; }

struct Tile {
  int64_t g, row0, n0;  // row0: this CTA's first row; n0: first output column
  int rows;             // this CTA's rows of the block (0 .. 128)
  int steps;            // reduction steps, the low-rank ones included
  int seg0;             // adapt: first adapter segment of the tile
  bool both;            // H == 2: the second MMA's columns are this tile's too
  int32_t box[2];       // adapt: first token of each CTA's rows if they are neighbours, else -1
};

template <int MODE, int H>
struct Shape {
  static constexpr int kHalfN = MODE == kGated ? 128 : 256;  // output columns of one MMA
  static constexpr int kTileN = H * kHalfN;
};

// Steps of the x W part, and per adapter segment.
__device__ __forceinline__ int main_steps(const RowsArgs& a) {
  return static_cast<int>((a.K + kFK - 1) / kFK);
}
__device__ __forceinline__ int rank_span(const RowsArgs& a) {
  return a.low_form == kLowSplit ? kFK / 2 : kFK;
}
__device__ __forceinline__ int rank_steps(const RowsArgs& a) {
  return (a.R + rank_span(a) - 1) / rank_span(a);
}

// The tiles' numbers: `full` whole ones, then (H == 2) the two halves of each of the others, so that
// a last round that would leave most pairs of CTAs idle takes half the time.
struct Schedule {
  uint32_t full, total;
};

template <int H>
__device__ __forceinline__ Schedule schedule_of(uint32_t tiles) {
  const uint32_t pairs = n_clusters(), rest = tiles % pairs;
  Schedule s;
  s.full = H == 2 && 2 * rest <= pairs ? tiles - rest : tiles;
  s.total = s.full + 2 * (tiles - s.full);
  return s;
}

template <int MODE, int H>
__device__ __forceinline__ Tile tile_of(uint32_t t, const Schedule& s, const RowsArgs& a,
                                        uint32_t rank) {
  const bool part = H == 2 && t >= s.full;
  const uint32_t f = part ? s.full + (t - s.full) / 2 : t;
  const uint32_t rb = f / static_cast<uint32_t>(a.n_blocks);
  Tile x;
  x.n0 = static_cast<int64_t>(f - rb * static_cast<uint32_t>(a.n_blocks)) * Shape<MODE, H>::kTileN;
  if (part && ((t - s.full) & 1)) x.n0 += Shape<MODE, H>::kHalfN;
  x.both = H == 2 && !part && x.n0 + Shape<MODE, H>::kHalfN < a.N;
  x.steps = main_steps(a);
  x.seg0 = 0;
  x.box[0] = x.box[1] = -1;
  int left;
  if constexpr (MODE == kGated) {
    int4 e = a.rblist[check_index(a.hdr, rb, a.max_row_blocks, 80)];
    if (!check_ok(a.hdr,
                  e.x >= 0 && e.x < a.G && e.y >= 0 && e.z >= 0 &&
                      static_cast<int64_t>(e.y) + e.z <= a.M,
                  81))
      e = make_int4(0, 0, 0, 0);
    x.g = e.x;
    x.row0 = static_cast<int64_t>(e.y) + kFM * rank;
    left = e.z - kFM * static_cast<int>(rank);
  } else {
    x.g = 0;
    x.row0 = static_cast<int64_t>(rb) * (2 * kFM) + kFM * rank;
    const int64_t l = a.M - x.row0;
    left = l > kFM ? kFM : static_cast<int>(l);
    const int2 s = a.blkseg[rb];
    x.seg0 = s.x;
    x.box[0] = a.box[2 * rb];
    x.box[1] = a.box[2 * rb + 1];
    x.steps += s.y * rank_steps(a);
  }
  x.rows = left < 0 ? 0 : (left > kFM ? kFM : left);
  return x;
}

// Segment and first rank of low-rank step e of a tile.
__device__ __forceinline__ int4 segment_of(const RowsArgs& a, const Tile& x, int e, int* r0) {
  const int rs = rank_steps(a);
  const int s = e / rs;
  *r0 = (e - s * rs) * rank_span(a);
  return a.segs[x.seg0 + s];
}

// First weight column of panel j (64 columns) of MMA h that CTA `rank` loads, as the output column
// it belongs to (gated: both CTAs' panels belong to the same outputs).
template <int MODE>
__device__ __forceinline__ int64_t panel_column(int64_t n0, int h, int j, uint32_t rank) {
  return MODE == kGated ? n0 + 128 * h + 64 * j : n0 + 256 * h + 128 * rank + 64 * j;
}

// Weight bytes that CTA `rank` loads for one main or low-rank step of a tile.
template <int MODE, int H>
__device__ __forceinline__ uint32_t w_bytes(const RowsArgs& a, const Tile& x, uint32_t rank,
                                            bool low_rank) {
  const int64_t n0 = x.n0;
  uint32_t b = 0;
#pragma unroll
  for (int h = 0; h < H; ++h) {
    if (h == 1 && !x.both) continue;
    if (MODE == kAdaptT || low_rank) {
      b += panel_column<MODE>(n0, h, 0, rank) < a.N ? static_cast<uint32_t>(kHalfBytes) : 0u;
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        b += panel_column<MODE>(n0, h, j, rank) < a.N ? static_cast<uint32_t>(kPanel) : 0u;
    }
  }
  return b;
}

template <int MODE, int H>
__device__ void w_producer(uint8_t* smem, WideCtl* ctl, const CUtensorMap* tm_w,
                           const CUtensorMap* tm_b, const CUtensorMap* tm_x, const RowsArgs& a,
                           const Schedule& sc, uint32_t rank) {
  using C = Cfg<H>;
  const uint64_t lim = a.wait_limit_ns;
  volatile int* abort = &ctl->abort;
  const bool leader = rank == 0;
  const int nks = main_steps(a);
  int stage = 0;
  uint32_t phase = 0, outstanding = 0, last_parity = 0;
  bool failed = false;
  for (uint32_t t = cluster_id(); t < sc.total && !failed; t += n_clusters()) {
    const Tile x = tile_of<MODE, H>(t, sc, a, rank);
    for (int ks = 0; ks < x.steps; ++ks) {
      const bool low = MODE != kGated && ks >= nks;
      int4 seg = make_int4(0, 0, 0, 0);
      int r0 = 0;
      if (low) seg = segment_of(a, x, ks - nks, &r0);
      if (!ptx::mbar_wait_cluster(&ctl->empty[stage], phase ^ 1u, lim, abort)) {
        failed = true;
        break;
      }
      uint8_t* sb = smem + stage * C::kStageBytes + kABytes;
      const uint32_t fb = ptx::mapa(&ctl->full[stage], 0);
      if (leader) {
        uint32_t bytes = w_bytes<MODE, H>(a, x, 0, low) + w_bytes<MODE, H>(a, x, 1, low);
        if (MODE != kGated && !low)
          bytes += (x.box[0] >= 0 ? kABytes : 0) + (x.box[1] >= 0 ? kABytes : 0);
        ptx::mbar_arrive_expect_tx(&ctl->full[stage], bytes);
      }
      if (MODE != kGated && !low && (rank ? x.box[1] : x.box[0]) >= 0)
        ptx::tma_load_2d_pair(sb - kABytes, tm_x, fb, ks * kFK, (rank ? x.box[1] : x.box[0]));
#pragma unroll
      for (int h = 0; h < H; ++h) {
        if (h == 1 && !x.both) continue;
        uint8_t* sh = sb + h * kHalfBytes;
        const int64_t nc = panel_column<MODE>(x.n0, h, 0, rank);
        if (low) {
          if (nc < a.N) ptx::tma_load_3d_pair(sh, tm_b, fb, r0, static_cast<int32_t>(nc), seg.x);
        } else if (MODE == kAdaptT) {
          if (nc < a.N)
            ptx::tma_load_3d_pair(sh, tm_w, fb, ks * kFK, static_cast<int32_t>(nc), 0);
        } else {
          // gated: the even CTA loads the gates' columns, the odd one the ups'
          const int64_t shift = MODE == kGated && rank ? a.N : 0;
          for (int j = 0; j < 2; ++j)
            if (nc + 64 * j < a.N)
              ptx::tma_load_3d_pair(sh + j * kPanel, tm_w, fb,
                                    static_cast<int32_t>(nc + 64 * j + shift), ks * kFK,
                                    static_cast<int32_t>(x.g));
        }
      }
      outstanding |= 1u << stage;
      last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
  if (failed) {
    ctl->abort = 1;
    raise_status(a.hdr, kStTimeout, 32);
  }
  if (leader) {
    int no_abort = 0;
    for (int s = 0; s < C::kStages; ++s)
      if (outstanding & (1u << s))
        ptx::mbar_wait_cluster(&ctl->full[s], (last_parity >> s) & 1u, lim, &no_abort);
  }
}

// Gather warp w fills stage slot w: the CTA's stages w, w + S, ... in the
// sequence of all steps of all its tiles. Rows lane >> 3 + 4 q, 16-byte chunk lane & 7.
template <int MODE, int H>
__device__ void x_gatherer(uint8_t* smem, WideCtl* ctl, const RowsArgs& a, const Schedule& sc,
                           uint32_t rank) {
  using C = Cfg<H>;
  const uint64_t lim = a.wait_limit_ns;
  volatile int* abort = &ctl->abort;
  const int w = (threadIdx.x >> 5) - 2;
  const int lane = threadIdx.x & 31;
  const int c = lane & 7;
  const char* xb = static_cast<const char*>(a.x);
  const uint32_t sa_slot = ptx::smem_addr(smem + w * C::kStageBytes);
  const uint32_t full = ptx::mapa(&ctl->full[w], 0);
  const int nks = main_steps(a);
  uint32_t phase = 0;
  bool failed = false;
  bool u_there = a.late == 0;
  int kb = w;  // the warp's next step, counted from the start of tile t
  // this lane's rows (lane >> 3) + 4 q of the tile: the x row's offset in
  // 16-byte units, or kNoRow past the block
  constexpr uint32_t kNoRow = 0xFFFFFFFFu;
  const uint32_t row_units = static_cast<uint32_t>(a.K / 8);
  uint32_t row16[kFM / 4];
  for (uint32_t t = cluster_id(); t < sc.total && !failed; t += n_clusters()) {
    const Tile x = tile_of<MODE, H>(t, sc, a, rank);
    if (kb < x.steps) {
      int32_t tok[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int r = lane + 32 * h;
        tok[h] = r < x.rows ? static_cast<int32_t>(check_index(
                                  a.hdr, a.rowinfo[check_index(a.hdr, x.row0 + r, a.M, 82)].token,
                                  a.batch, 83))
                            : -1;
      }
#pragma unroll
      for (int q = 0; q < kFM / 4; ++q) {
        const int rr = (lane >> 3) + 4 * q;
        const int32_t tk = __shfl_sync(0xFFFFFFFFu, tok[rr >> 5], rr & 31);
        row16[q] = tk >= 0 ? static_cast<uint32_t>(tk) * row_units : kNoRow;
      }
    }
    for (; kb < x.steps; kb += C::kStages) {
      if (!ptx::mbar_wait_cluster(&ctl->empty[w], phase ^ 1u, lim, abort)) {
        failed = true;
        break;
      }
      if (MODE != kGated && kb < nks && (rank ? x.box[1] : x.box[0]) >= 0) {
        // neighbouring rows: the weight's producer copies them as one box. This warp has written
        // nothing, so its arrival need not release anything across the cluster (which costs the
        // odd CTA's warp up to 1,500 cycles).
        if (lane == 0) ptx::mbar_arrive_remote_cta(full);
        phase ^= 1u;
        continue;
      } else if (MODE == kGated || kb < nks) {
        const int64_t k = static_cast<int64_t>(kb) * kFK + c * 8;
        const bool k_ok = k < a.K;
        const char* xk = xb + k * 2;
#pragma unroll
        for (int q = 0; q < kFM / 4; ++q) {
          const int rr = (lane >> 3) + 4 * q;
          const bool ok = k_ok && row16[q] != kNoRow;
          const void* src = ok ? static_cast<const void*>(
                                     xk + (static_cast<uint64_t>(row16[q]) << 4))
                               : static_cast<const void*>(xb);
          ptx::cp_async_16(sa_slot + rr * 128 + ((c ^ (rr & 7)) << 4), src, ok ? 16u : 0u);
        }
      } else {
        // rows of u that belong to the step's adapter; zeros elsewhere
        if (!u_there) {
          ptx::griddep_wait();
          u_there = true;
        }
        int r0;
        const int4 seg = segment_of(a, x, kb - nks, &r0);
        // chunk c: ranks 8 c, or the hi or lo parts of ranks 8 (c % 4), of the step's
        const bool split = a.low_form == kLowSplit;
        const bool in = r0 + 8 * (split ? c & 3 : c) < a.R;
        const int64_t width = split ? low_width(a.R) : a.R;
        const int64_t col = (split ? 2 * r0 : r0) + 8 * c;
        const char* ub = static_cast<const char*>(a.u);
#pragma unroll 4
        for (int q = 0; q < kFM / 4; ++q) {
          const int rr = (lane >> 3) + 4 * q;
          const int64_t row = x.row0 + rr;
          const bool ok = in && rr < x.rows && row >= seg.y && row < seg.z;
          const void* src = ok ? static_cast<const void*>(
                                     ub + ((seg.w + (row - seg.y)) * width + col) * 2)
                               : static_cast<const void*>(ub);
          ptx::cp_async_16(sa_slot + rr * 128 + ((c ^ (rr & 7)) << 4), src, ok ? 16u : 0u);
        }
      }
      ptx::cp_async_commit();
      ptx::cp_async_wait<0>();
      ptx::fence_proxy_async_smem();
      __syncwarp();
      // the even CTA's own rows go to its own MMA thread: CTA scope suffices
      if (lane == 0) {
        if (rank == 0)
          ptx::mbar_arrive(&ctl->full[w]);
        else
          ptx::mbar_arrive_remote(full);
      }
      phase ^= 1u;
    }
    kb -= x.steps;
  }
  ptx::cp_async_wait<0>();
  if (failed) {
    ctl->abort = 1;
    if (lane == 0) raise_status(a.hdr, kStTimeout, 33);
  }
}

// Lanes of the pair's 256 that lie outside rows [lo, hi) of the tile, as the eight words of a
// disable-output-lane mask.
__device__ __forceinline__ void lane_mask(int lo, int hi, uint32_t (&m)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int l = lo - 32 * i, h = hi - 32 * i;
    const uint32_t below = l <= 0 ? 0u : (l >= 32 ? 0xFFFFFFFFu : (1u << l) - 1u);
    const uint32_t upto = h <= 0 ? 0u : (h >= 32 ? 0xFFFFFFFFu : (1u << h) - 1u);
    m[i] = ~(upto & ~below);
  }
}

template <int DT, int MODE, int H>
__device__ void mma_issuer(uint8_t* smem, WideCtl* ctl, uint32_t tmem_base, const RowsArgs& a,
                           const Schedule& sc) {
  using C = Cfg<H>;
  constexpr uint32_t kFmt = DT == PGG_BF16 ? 1u : 0u;
  constexpr uint32_t idesc_k = ptx::idesc_make(kFmt, 2 * kFM, kFN);  // both operands K-major
  constexpr uint32_t idesc_mn = idesc_k | (1u << 16);                // B MN-major
  const uint64_t lim = a.wait_limit_ns;
  volatile int* abort = &ctl->abort;
  const int nks = main_steps(a);
  int stage = 0, acc = 0;
  uint32_t phase = 0, aph = 0;
  bool issued = false, failed = false;
  for (uint32_t t = cluster_id(); t < sc.total && !failed; t += n_clusters()) {
    const Tile x = tile_of<MODE, H>(t, sc, a, 0);
    if (!ptx::mbar_wait_cluster(&ctl->tempty[acc], aph ^ 1u, lim, abort)) {
      failed = true;
      break;
    }
    ptx::tc_fence_after_sync();
    for (int ks = 0; ks < x.steps; ++ks) {
      const bool low = MODE != kGated && ks >= nks;
      int4 seg = make_int4(0, 0, 0, 0);
      int r0 = 0;
      if (low) seg = segment_of(a, x, ks - nks, &r0);
      if (!ptx::mbar_wait_cluster(&ctl->full[stage], phase, lim, abort)) {
        failed = true;
        break;
      }
      ptx::tc_fence_after_sync();
      const uint32_t sa = ptx::smem_addr(smem + stage * C::kStageBytes);
      const uint64_t da = ptx::sdesc_sw128(sa);
      uint32_t m[8];
      if (low) lane_mask(static_cast<int>(seg.y - x.row0), static_cast<int>(seg.z - x.row0), m);
#pragma unroll
      for (int h = 0; h < H; ++h) {
        if (h == 1 && !x.both) continue;
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>((H == 1 ? acc : h) * kFN);
        const uint32_t sb = sa + kABytes + h * kHalfBytes;
        if (low) {
          const uint64_t db = ptx::sdesc_sw128(sb);
          const bool split = a.low_form == kLowSplit;
#pragma unroll
          for (int kk = 0; kk < kFK / 16; ++kk) {
            const int kb = split ? kk & 1 : kk;  // 16 ranks of b; kk 2 and 3 of a split are lo parts
            if (r0 + 16 * kb < a.R) {
              const uint64_t off = static_cast<uint64_t>((kk * 32) >> 4);
              const uint64_t b_off = static_cast<uint64_t>((kb * 32) >> 4);
              mma_f16_pair_lanes(d_tmem, da + off, db + b_off, idesc_k, m, 1u);
            }
          }
        } else if constexpr (MODE == kAdaptT) {
          const uint64_t db = ptx::sdesc_sw128(sb);
#pragma unroll
          for (int kk = 0; kk < kFK / 16; ++kk) {
            const uint64_t off = static_cast<uint64_t>((kk * 32) >> 4);
            ptx::mma_f16_pair(d_tmem, da + off, db + off, idesc_k, (ks > 0 || kk > 0) ? 1u : 0u);
          }
        } else {
          const uint64_t db = ptx::sdesc_sw128_mn(sb, kPanel);
#pragma unroll
          for (int kk = 0; kk < kFK / 16; ++kk) {
            const uint64_t a_off = static_cast<uint64_t>((kk * 32) >> 4);        // 16 k: 32 bytes
            const uint64_t b_off = static_cast<uint64_t>((kk * 16 * 128) >> 4);  // 16 k rows
            ptx::mma_f16_pair(d_tmem, da + a_off, db + b_off, idesc_mn,
                              (ks > 0 || kk > 0) ? 1u : 0u);
          }
        }
      }
      issued = true;
      ptx::mma_commit_pair(&ctl->empty[stage], 0x3);
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (failed) break;
    ptx::mma_commit_pair(&ctl->tfull[acc], 0x3);
    if (H == 1) acc ^= 1;
    if (acc == 0) aph ^= 1u;
  }
  if (failed) {
    ctl->abort = 1;
    raise_status(a.hdr, kStTimeout, 34);
  }
  if (issued) {
    int no_abort = 0;
    ptx::mma_commit_pair(&ctl->drain, 0x1);
    ptx::mbar_wait(&ctl->drain, 0u, lim, &no_abort);
  }
}

// Each lane's own row, 64 columns from `taddr` on, as 128 bytes of 16-bit values. (16 columns at a
// time: the epilogue's threads have 80 registers.)
template <int DT>
__device__ __forceinline__ void plain_blocks(uint32_t taddr, uint4 (&b)[8]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t v[16];
    ptx::tmem_ld_32x32b_x16(taddr + 16u * q, v);
    ptx::tmem_ld_wait();
    b[2 * q] = pack8<DT>(v);
    b[2 * q + 1] = pack8<DT>(v + 8);
  }
}

// The same of the gated product of the columns from `taddr` on and those 128 further.
template <int DT>
__device__ __forceinline__ void gated_blocks(uint32_t taddr, float p, uint4 (&b)[8]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t g[16], u[16];
    ptx::tmem_ld_32x32b_x16(taddr + 16u * q, g);
    ptx::tmem_ld_32x32b_x16(taddr + 128u + 16u * q, u);
    ptx::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i)
      u[i] = __float_as_uint(gate(__uint_as_float(g[i]), __uint_as_float(u[i]), p));
    b[2 * q] = pack8<DT>(u);
    b[2 * q + 1] = pack8<DT>(u + 8);
  }
}

// 32 lanes' rows x 64 columns of 16-bit values (b: each lane its own row's 128 bytes) to rows
// `row` (each lane's own, -1 = not written) of a row-major [*, ld] output, columns col ..
// col + 63 below `ncols`: after the transpose every warp store covers four rows' full segments.
__device__ __forceinline__ void store_rows(uint4 (&b)[8], void* out, int64_t row, int64_t ld,
                                           int64_t base, int64_t col, int64_t ncols, int lane) {
  transpose8(b, lane);
  const int bg = lane >> 3;
  const int64_t c = col + (lane & 7) * 8;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t r = __shfl_sync(0xFFFFFFFFu, row, 8 * bg + j);
    if (r >= 0 && c < ncols)
      *reinterpret_cast<uint4*>(static_cast<char*>(out) + (r * ld + base + c) * 2) = b[j];
  }
}

template <int DT, int MODE, int H>
__device__ void epilogue(WideCtl* ctl, uint32_t tmem_base, const RowsArgs& a, const Schedule& sc,
                         uint32_t rank) {
  const uint64_t lim = a.wait_limit_ns;
  volatile int* abort = &ctl->abort;
  const int lane = threadIdx.x & 31;
  const int quarter = (threadIdx.x >> 5) & 3;  // accumulator lanes (rows) 32 q .. 32 q + 31
  const int part = ((threadIdx.x >> 5) - Cfg<H>::kEpiWarp0) / 4;
  const int h = part >> 1;  // H == 2: the MMA it drains
  constexpr int kSpan = Shape<MODE, H>::kHalfN / 2;
  const int col0 = (part & 1) * kSpan;  // its columns of that MMA's outputs
  const uint32_t tempty0 = ptx::mapa(&ctl->tempty[0], 0);
  const uint32_t tempty1 = ptx::mapa(&ctl->tempty[1], 0);
  int acc = 0;
  uint32_t aph = 0;
  bool held = a.hold_release != 0;  // (test hook: the first release is withheld)
  for (uint32_t t = cluster_id(); t < sc.total; t += n_clusters()) {
    const Tile x = tile_of<MODE, H>(t, sc, a, rank);
    const int64_t n0 = x.n0 + h * Shape<MODE, H>::kHalfN;
    const int valid = x.rows - 32 * quarter;  // rows of this warp's 32 that exist
    int64_t row = -1;                         // output row of this lane
    float p = 1.0f;
    if (lane < valid) {
      row = x.row0 + 32 * quarter + lane;
      const RowInfo ri = a.rowinfo[check_index(a.hdr, row, a.M, 84)];
      if constexpr (MODE == kGated) {
        if (a.probs) p = a.probs[check_index(a.hdr, ri.rank, a.M, 85)];
      } else {
        row = check_index(a.hdr, ri.token, a.batch, 86);
      }
    }
    const bool ok = ptx::mbar_wait_cluster(&ctl->tfull[acc], aph, lim, abort);
    if (!__all_sync(0xFFFFFFFFu, ok)) {
      if (lane == 0) {
        ctl->abort = 1;
        raise_status(a.hdr, kStTimeout, 35);
      }
      break;
    }
    ptx::tc_fence_after_sync();
    const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(32 * quarter) << 16) +
                            static_cast<uint32_t>((H == 1 ? acc : h) * kFN);
#pragma unroll 1
    for (int c0 = col0; c0 < col0 + kSpan && n0 + c0 < a.N && valid > 0 && (h == 0 || x.both);
         c0 += 64) {
      uint4 b[8];
      if constexpr (MODE == kGated) {
        gated_blocks<DT>(t_lane + static_cast<uint32_t>(c0), p, b);
        store_rows(b, a.out, row, a.N, 0, n0 + c0, a.N, lane);
        if (a.gate_up) {
          plain_blocks<DT>(t_lane + static_cast<uint32_t>(c0), b);
          store_rows(b, a.gate_up, row, 2 * a.N, 0, n0 + c0, a.N, lane);
          plain_blocks<DT>(t_lane + static_cast<uint32_t>(128 + c0), b);
          store_rows(b, a.gate_up, row, 2 * a.N, a.N, n0 + c0, a.N, lane);
        }
      } else {
        plain_blocks<DT>(t_lane + static_cast<uint32_t>(c0), b);
        store_rows(b, a.out, row, a.N, 0, n0 + c0, a.N, lane);
      }
    }
    ptx::tc_fence_before_sync();
    __syncwarp();
    // tensor memory changes hands (the output goes out through global memory,
    // not to the MMA thread): CTA scope
    if (lane == 0 && !held) ptx::mbar_arrive_remote_cta(acc ? tempty1 : tempty0);
    held = false;
    if (H == 1) acc ^= 1;
    if (acc == 0) aph ^= 1u;
  }
}

template <int DT, int MODE, int H>
__global__ void __launch_bounds__(Cfg<H>::kThreads, 1)
    rows_wide_kernel(const __grid_constant__ CUtensorMap tm_w,
                     const __grid_constant__ CUtensorMap tm_b,
                     const __grid_constant__ CUtensorMap tm_x, const RowsArgs a) {
  using C = Cfg<H>;
  // late: u alone is not there yet. The gather warps wait before they read it, and the first
  // epilogue warp before it lets the next launch start.
  if (!a.late) launch_order(a.early, false);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  auto* ctl = reinterpret_cast<WideCtl*>(smem + C::kStages * C::kStageBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();

  if (routing_failed(a.hdr)) {  // the result is defined as zeros
    zero_rows16(a);
    if (a.late) ptx::griddep_wait();
    return;
  }
  const uint32_t row_blocks = MODE == kGated
                                  ? a.hdr->n_row_blocks
                                  : static_cast<uint32_t>((a.M + 2 * kFM - 1) / (2 * kFM));
  const Schedule sc = schedule_of<H>(row_blocks * static_cast<uint32_t>(a.n_blocks));

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(&ctl->full[s], 3);
      ptx::mbar_init(&ctl->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&ctl->tfull[b], 1);
      ptx::mbar_init(&ctl->tempty[b], 2 * C::kEpiWarps);
    }
    ptx::mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::tma_prefetch_desc(&tm_w);
    if (MODE != kGated) ptx::tma_prefetch_desc(&tm_b);
    if (MODE != kGated) ptx::tma_prefetch_desc(&tm_x);
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(&ctl->tmem_base, kTmemCols);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before_sync();
  __syncthreads();
  ptx::cluster_sync();
  ptx::tc_fence_after_sync();
  const uint32_t tmem_base = ctl->tmem_base;

  if (warp == 0) {
    if (lane == 0) w_producer<MODE, H>(smem, ctl, &tm_w, &tm_b, &tm_x, a, sc, rank);
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) mma_issuer<DT, MODE, H>(smem, ctl, tmem_base, a, sc);
  } else if (warp < 2 + C::kGatherWarps) {
    x_gatherer<MODE, H>(smem, ctl, a, sc, rank);
  } else if (warp >= C::kEpiWarp0) {
    if (a.late && warp == C::kEpiWarp0) launch_order(a.early, false);
    epilogue<DT, MODE, H>(ctl, tmem_base, a, sc, rank);
  }

  ptx::tc_fence_before_sync();
  __syncthreads();
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after_sync();
    ptx::tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

// Tiles of 256 or of 512 accumulator columns: the form whose busiest pair of CTAs has the fewer
// cycles. A 64-k step takes about 720 with 256 columns and 1230 with 512 (1113 where the rows come
// as boxes): the wider tile reads a quarter less per product and has eight MMAs to a wait and a
// commit. With 512 columns there is one accumulator, so nothing hides a tile's output:
// 13,000 cycles with gate_up, 7,300 for h alone, 5,200 for y. Both sides: 13,500 tokens x 8, 60
// experts, K 7168, F 2048: 4.45 ms and 4.13; 4096 x 8, 16 experts, K 2048, F 1024: 198 us and 238;
// adapters, K = N = 4096, 2048 tokens: 79 and 71 us, 8191: 203 and 206.
int choose_halves(RowsMode mode, const RowsArgs& a, int64_t row_blocks, int pairs) {
  const int64_t half_n = mode == kGated ? 128 : 256;
  const int64_t steps = (a.K + kFK - 1) / kFK;
  const int64_t drain = mode != kGated ? 5200 : a.gate_up ? 13000 : 7300;
  const int64_t step2 = mode != kGated ? 1113 : 1230;
  const int64_t n1 = row_blocks * ((a.N + half_n - 1) / half_n);
  const int64_t n2 = row_blocks * ((a.N + 2 * half_n - 1) / (2 * half_n));
  const int64_t one = (n1 + pairs - 1) / pairs * (steps * 720 > drain ? steps * 720 : drain);
  const int64_t rest = n2 % pairs;  // as halves when they are few (see schedule_of)
  const int64_t tail = rest == 0           ? 0
                       : 2 * rest <= pairs ? steps * 720 + drain
                                           : steps * step2 + drain;
  const int64_t two = n2 / pairs * (steps * step2 + drain) + tail;
  return two < one ? 2 : 1;
}

template <int DT, int H>
cudaError_t launch_t(RowsMode mode, const CUtensorMap (&tm)[3], const RowsArgs& a,
                     int64_t max_tiles, int num_sms, cudaStream_t stream) {
  using K = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const RowsArgs);
  const K kern = mode == kGated   ? K(rows_wide_kernel<DT, kGated, H>)
                 : mode == kAdapt ? K(rows_wide_kernel<DT, kAdapt, H>)
                                  : K(rows_wide_kernel<DT, kAdaptT, H>);
  static ClusterLimits limits[3];
  int clusters = 0;
  const cudaError_t err =
      clusters_that_fit(&limits[mode == kGated ? 0 : mode == kAdapt ? 1 : 2], kern,
                        Cfg<H>::kThreads, smem_bytes<H>(), 2, num_sms, &clusters);
  if (err != cudaSuccess) return err;
  const int64_t want = max_tiles < num_sms / 2 ? max_tiles : num_sms / 2;
  return launch_pdl(kern, dim3(static_cast<unsigned>(2 * (clusters < want ? clusters : want))),
                    dim3(Cfg<H>::kThreads), static_cast<size_t>(smem_bytes<H>()), stream, 2, tm[0],
                    tm[1], tm[2], a);
}

}  // namespace

// live_blocks: about how many row blocks there will be (the choice of the tile goes by it, nothing
// else).
cudaError_t launch_rows_wide(int dtype, RowsMode mode, RowsArgs a, int64_t live_blocks,
                             int num_sms, cudaStream_t stream) {
  const int64_t half_n = mode == kGated ? 128 : 256;
  const int64_t row_blocks = mode == kGated ? a.max_row_blocks : (a.M + 2 * kFM - 1) / (2 * kFM);
  const int H = choose_halves(mode, a, mode == kGated ? live_blocks : row_blocks, num_sms / 2);
  a.n_blocks = static_cast<int32_t>((a.N + H * half_n - 1) / (H * half_n));
  CUtensorMap tm[3];  // weight, b, x
  std::memset(tm, 0, sizeof(tm));
  bool ok;
  if (mode == kGated)
    ok = encode_map_3d(&tm[0], dtype, a.w, 2 * a.N, a.K, a.G, kFK);
  else if (mode == kAdapt)
    ok = encode_map_3d(&tm[0], dtype, a.w, a.N, a.K, 1, kFK);
  else
    ok = encode_map_3d(&tm[0], dtype, a.w, a.K, a.N, 1, 128);
  if (mode != kGated)
    ok = ok && encode_map_3d(&tm[1], dtype, a.b, a.R, a.N, a.G, 128) &&
         encode_map_rows(&tm[2], dtype, a.x, a.K, a.batch, kFM);
  if (!ok) return cudaErrorInvalidValue;
  const int64_t tiles = row_blocks * a.n_blocks;
  if (dtype == PGG_BF16)
    return H == 2 ? launch_t<PGG_BF16, 2>(mode, tm, a, tiles, num_sms, stream)
                  : launch_t<PGG_BF16, 1>(mode, tm, a, tiles, num_sms, stream);
  if (dtype == PGG_F16)
    return H == 2 ? launch_t<PGG_F16, 2>(mode, tm, a, tiles, num_sms, stream)
                  : launch_t<PGG_F16, 1>(mode, tm, a, tiles, num_sms, stream);
  return cudaErrorInvalidValue;
}

int rows_wide_block() { return 2 * kFM; }

}  // namespace pgg
