// Gradients of the adapters' factors on tcgen05 tensor cores:
//
//     d_a[ad] = sum over the tokens t of ad of x[t, :]^T v[t, :]       [K, R]
//     d_b[ad] = sum over the tokens t of ad of d_y[t, :]^T u[t, :]     [N, R]
//
// Both in one launch: tall, R-wide products whose reduction runs over the rows
// of one adapter, so what they cost is reading x and d_y once (R multiply-adds
// a byte). Tile: one adapter, 128 of the K (N) columns as accumulator lanes and
// 32 or 64 ranks (P of 32) as accumulator columns, fp32 in tensor memory (two
// buffers): u and v come as the sums of two values (see LowRankForm), so 32 ranks
// take 64 columns, 32 for the hi and 32 for the lo parts, which the epilogue adds.
// Both operands are MN-major. A stage is 128 rows: 128 columns of x, by TMA where
// the 128 rows are neighbouring tokens, else gathered by token with cp.async
// (one warp per stage slot), and the rows' ranks of v by TMA. v is stored so
// that an adapter's rows end on a multiple of 128 with rows of zeros, and their
// x rows read as zeros: nobody's rows, whatever they hold, take part there.
//
// A cluster of S CTAs shares a tile: each reduces its part of the adapter's
// rows, the partial sums meet through distributed shared memory, 128 / S
// columns a CTA, and are added in the order of the CTAs. Bitwise repeatable. An
// adapter without tokens gets zeros. Waits are bounded as everywhere.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <cstring>

#include "pgg_ops.h"
#include "pgg_ops_launch.h"
#include "pgg_ops_mma.cuh"
#include "pgg_ptx.cuh"

namespace pgg {
namespace {

constexpr int kM = 128;            // columns of x (d_y) per tile: accumulator lanes
constexpr int kRows = 128;         // reduction per stage
constexpr int kPanel = kRows * 128;
constexpr int kABytes = 2 * kPanel;
constexpr int kEpiWarps = 4;

// P: panels of 32 ranks a tile. One where the rank is at most 32, else two, so that x and d_y are
// not read more often than ranks beyond 64 need.
template <int P>
struct Cfg {
  static constexpr int kNR = 32 * P;       // ranks per tile
  static constexpr int kCols = 64 * P;     // accumulator columns
  static constexpr int kBBytes = P * kPanel;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = P == 1 ? 4 : 3;
  static constexpr int kRedBytes = kM * kNR * 4;
  static constexpr int kGatherWarps = 2 * kStages;  // two per stage slot
  static constexpr int kEpiWarp0 = P == 1 ? 12 : 8;  // (a multiple of four: tensor-memory lanes)
  static constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
  static constexpr int kTmemCols = 2 * kCols;
  static_assert(2 + kGatherWarps <= kEpiWarp0, "warp roles");
};
constexpr int kMaxStages = 4;

struct Ctl {
  uint64_t full[kMaxStages];   // bytes + the two gather warps' arrivals
  uint64_t empty[kMaxStages];  // MMAs of the stage done
  uint64_t tfull[2], tempty[2];
  uint64_t rfull, rempty;   // partial sums of all CTAs received here / mine read by all CTAs
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

template <int P>
constexpr int smem_bytes() {
  return Cfg<P>::kStages * Cfg<P>::kStageBytes + Cfg<P>::kRedBytes +
         static_cast<int>(sizeof(Ctl)) + 1024;
}
static_assert(smem_bytes<1>() <= 227 * 1024 && smem_bytes<2>() <= 227 * 1024,
              "shared memory per CTA");

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
  return r;
}

struct Tile {
  int which;               // 0: d_a, 1: d_b
  int ad, r0;
  int64_t c0;              // first column
  int4 range;              // {first compact row, rows, first row of v, 0}
  int s0, s1;              // this CTA's steps of 128 rows
  int steps;               // all steps of the adapter
};

// Tiles run over the adapters first, so that neighbouring clusters share the work of a large one.
template <int P>
__device__ __forceinline__ Tile tile_of(uint32_t t, const OuterArgs& a, uint32_t rank,
                                        uint32_t S) {
  Tile x;
  const uint32_t A = static_cast<uint32_t>(a.A);
  x.ad = static_cast<int>(t % A);
  uint32_t q = t / A;
  x.r0 = static_cast<int>(q % a.r_blocks) * Cfg<P>::kNR;
  q /= a.r_blocks;
  x.which = q >= static_cast<uint32_t>(a.blocks0) ? 1 : 0;
  x.c0 = static_cast<int64_t>(x.which ? q - a.blocks0 : q) * kM;
  x.range = a.range[x.ad];
  x.steps = (x.range.y + kRows - 1) / kRows;
  x.s0 = x.steps * static_cast<int>(rank) / static_cast<int>(S);
  x.s1 = x.steps * (static_cast<int>(rank) + 1) / static_cast<int>(S);
  return x;
}

// First token of the 128 rows of step s if all of them are the adapter's and neighbouring tokens.
__device__ __forceinline__ int32_t box_of(const OuterArgs& a, const Tile& x, int s) {
  if (kRows * (s + 1) > x.range.y) return -1;
  return box_of_rows(a.order, static_cast<int64_t>(x.range.x) + kRows * s, kRows);
}

template <int P>
__device__ void producer(uint8_t* smem, Ctl* ctl, const CUtensorMap* tm, const OuterArgs& a,
                         uint32_t total, uint32_t first, uint32_t step, uint32_t rank,
                         uint32_t S) {
  using C = Cfg<P>;
  const uint64_t lim = a.wait_limit_ns;
  volatile int* abort = &ctl->abort;
  int stage = 0;
  uint32_t phase = 0, outstanding = 0, last_parity = 0;
  bool failed = false;
  for (uint32_t t = first; t < total && !failed; t += step) {
    const Tile x = tile_of<P>(t, a, rank, S);
    const CUtensorMap* tm_x = tm + 2 * x.which;
    const bool second = x.c0 + 64 < a.cols[x.which];
    for (int s = x.s0; s < x.s1; ++s) {
      const int32_t box = box_of(a, x, s);
      if (!ptx::mbar_wait(&ctl->empty[stage], phase ^ 1u, lim, abort)) {
        failed = true;
        break;
      }
      uint8_t* sa = smem + stage * C::kStageBytes;
      ptx::mbar_arrive_expect_tx(&ctl->full[stage],
                                 C::kBBytes + (box >= 0 ? (second ? 2 * kPanel : kPanel) : 0));
      for (int p = 0; p < P; ++p)  // (32 ranks are 64 columns of v)
        ptx::tma_load_2d(sa + kABytes + p * kPanel, tm_x + 1, &ctl->full[stage],
                         2 * x.r0 + 64 * p, x.range.z + kRows * s);
      if (box >= 0) {
        ptx::tma_load_2d(sa, tm_x, &ctl->full[stage], static_cast<int32_t>(x.c0), box);
        if (second)
          ptx::tma_load_2d(sa + kPanel, tm_x, &ctl->full[stage], static_cast<int32_t>(x.c0 + 64),
                           box);
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
    raise_status(a.hdr, kStTimeout, 52);
  }
  int no_abort = 0;
  for (int s = 0; s < C::kStages; ++s)
    if (outstanding & (1u << s))
      ptx::mbar_wait(&ctl->full[s], (last_parity >> s) & 1u, lim, &no_abort);
}

// Gather warps 2 w and 2 w + 1 fill half of stage slot w each where its rows are not neighbours:
// row (lane >> 4) + 2 q, 16-byte chunk lane & 15 of its 256 bytes.
template <int P>
__device__ void gatherer(uint8_t* smem, Ctl* ctl, const OuterArgs& a, uint32_t total,
                         uint32_t first, uint32_t step, uint32_t rank, uint32_t S) {
  const uint64_t lim = a.wait_limit_ns;
  volatile int* abort = &ctl->abort;
  const int w = ((threadIdx.x >> 5) - 2) >> 1, half = ((threadIdx.x >> 5) - 2) & 1;
  const int lane = threadIdx.x & 31, c = lane & 15;
  const uint32_t sa = ptx::smem_addr(smem + w * Cfg<P>::kStageBytes + (c >> 3) * kPanel);
  uint32_t phase = 0;
  bool failed = false;
  int kb = w;  // the warp's next step, counted from the start of tile t
  for (uint32_t t = first; t < total && !failed; t += step) {
    const Tile x = tile_of<P>(t, a, rank, S);
    const int64_t C = a.cols[x.which];
    const char* base = static_cast<const char*>(a.left[x.which]);
    const int64_t col = x.c0 + 8 * c;
    const bool in = col < C;
    const int steps = x.s1 - x.s0;
    for (; kb < steps; kb += Cfg<P>::kStages) {
      const int s = x.s0 + kb;
      const int32_t box = box_of(a, x, s);
      int32_t tok[2];  // rows 64 half + lane + 32 h of the step; -1 past the adapter's
      if (box < 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = kRows * s + 64 * half + lane + 32 * h;
          tok[h] = row < x.range.y ? a.order[static_cast<int64_t>(x.range.x) + row].token : -1;
        }
      }
      if (!ptx::mbar_wait(&ctl->empty[w], phase ^ 1u, lim, abort)) {
        failed = true;
        break;
      }
      if (box < 0) {
#pragma unroll
        for (int q = 0; q < kRows / 4; ++q) {
          const int rq = (lane >> 4) + 2 * q, rr = 64 * half + rq;
          const int32_t tk = __shfl_sync(0xFFFFFFFFu, tok[q / 16], rq & 31);
          const bool ok = in && tk >= 0;
          const void* src = ok ? static_cast<const void*>(
                                     base + (static_cast<int64_t>(tk) * C + col) * 2)
                               : static_cast<const void*>(base);
          ptx::cp_async_16(sa + rr * 128 + (((c & 7) ^ (rr & 7)) << 4), src, ok ? 16u : 0u);
        }
        ptx::cp_async_commit();
        ptx::cp_async_wait<0>();
        ptx::fence_proxy_async_smem();
        __syncwarp();
      }
      if (lane == 0) ptx::mbar_arrive(&ctl->full[w]);
      phase ^= 1u;
    }
    kb -= steps;
  }
  ptx::cp_async_wait<0>();
  if (failed) {
    ctl->abort = 1;
    if (lane == 0) raise_status(a.hdr, kStTimeout, 53);
  }
}

template <int DT, int P>
__device__ void mma_issuer(uint8_t* smem, Ctl* ctl, uint32_t tmem_base, const OuterArgs& a,
                           uint32_t total, uint32_t first, uint32_t step, uint32_t rank,
                           uint32_t S) {
  using C = Cfg<P>;
  constexpr uint32_t idesc = ptx::idesc_make_mn(DT == PGG_BF16 ? 1u : 0u, kM, C::kCols);
  const uint64_t lim = a.wait_limit_ns;
  volatile int* abort = &ctl->abort;
  int stage = 0, acc = 0;
  uint32_t phase = 0, aph = 0;
  bool issued = false, failed = false;
  for (uint32_t t = first; t < total && !failed; t += step) {
    const Tile x = tile_of<P>(t, a, rank, S);
    if (!ptx::mbar_wait(&ctl->tempty[acc], aph ^ 1u, lim, abort)) {
      failed = true;
      break;
    }
    ptx::tc_fence_after_sync();
    const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * C::kCols);
    for (int s = x.s0; s < x.s1; ++s) {
      if (!ptx::mbar_wait(&ctl->full[stage], phase, lim, abort)) {
        failed = true;
        break;
      }
      ptx::tc_fence_after_sync();
      const uint32_t sa = ptx::smem_addr(smem + stage * C::kStageBytes);
      const uint64_t da = ptx::sdesc_sw128_mn(sa, kPanel);
      const uint64_t db = ptx::sdesc_sw128_mn(sa + kABytes, kPanel);
#pragma unroll
      for (int kk = 0; kk < kRows / 16; ++kk) {
        const uint64_t off = static_cast<uint64_t>((kk * 16 * 128) >> 4);  // 16 rows
        ptx::mma_f16(d_tmem, da + off, db + off, idesc, (s > x.s0 || kk > 0) ? 1u : 0u);
      }
      issued = true;
      ptx::mma_commit(&ctl->empty[stage]);
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (failed) break;
    ptx::mma_commit(&ctl->tfull[acc]);  // (at once when this CTA had no step)
    acc ^= 1;
    if (acc == 0) aph ^= 1u;
  }
  if (failed) {
    ctl->abort = 1;
    raise_status(a.hdr, kStTimeout, 54);
  }
  if (issued) {
    int no_abort = 0;
    ptx::mma_commit(&ctl->drain);
    ptx::mbar_wait(&ctl->drain, 0u, lim, &no_abort);
  }
}

template <int DT, int P>
__device__ void epilogue(Ctl* ctl, float* red, uint32_t tmem_base, const OuterArgs& a,
                         uint32_t total, uint32_t first, uint32_t step, uint32_t rank,
                         uint32_t S) {
  constexpr int kNR = Cfg<P>::kNR;
  const uint64_t lim = a.wait_limit_ns;
  volatile int* abort = &ctl->abort;
  const int lane = threadIdx.x & 31;
  const int quarter = (threadIdx.x >> 5) & 3;
  const int tid = 32 * quarter + lane;
  const int lanes = kM / static_cast<int>(S);  // columns that each CTA finishes
  const int shift = 31 - __clz(lanes);
  int acc = 0;
  uint32_t aph = 0, rph = 0;
  bool held = a.hold_release != 0;
  for (uint32_t t = first; t < total; t += step) {
    const Tile x = tile_of<P>(t, a, rank, S);
    const int nr = a.R - x.r0 < kNR ? a.R - x.r0 : kNR;  // (a multiple of 8)
    bool ok = ptx::mbar_wait(&ctl->tfull[acc], aph, lim, abort);
    ok = ok && ptx::mbar_wait_cluster(&ctl->rempty, rph ^ 1u, lim, abort);
    if (!__all_sync(0xFFFFFFFFu, ok)) {
      if (lane == 0) {
        ctl->abort = 1;
        raise_status(a.hdr, kStTimeout, 55);
      }
      break;
    }
    ptx::tc_fence_after_sync();
    if (x.s1 > x.s0) {  // (a CTA without a step has nothing to send, and is not read)
      const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(32 * quarter) << 16) +
                              static_cast<uint32_t>(acc * Cfg<P>::kCols);
      const int dst = tid >> shift;  // the CTA that finishes this lane's column
      float* mine = red + static_cast<int>(rank) * kNR * lanes + (tid & (lanes - 1));
      const uint32_t to = ptx::mapa(mine, static_cast<uint32_t>(dst));
#pragma unroll 1
      for (int c0 = 0; c0 < nr; c0 += 16) {
        uint32_t hi[16], lo[16];  // ranks c0 .. c0 + 15
        const uint32_t at = t_lane + static_cast<uint32_t>(c0 / 32 * 64 + c0 % 32);
        ptx::tmem_ld_32x32b_x16(at, hi);
        ptx::tmem_ld_32x32b_x16(at + 32u, lo);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i)
          st_cluster_f32(to + static_cast<uint32_t>((c0 + i) * lanes * 4),
                         __uint_as_float(hi[i]) + __uint_as_float(lo[i]));
      }
    }
    ptx::tc_fence_before_sync();
    __syncwarp();
    if (lane == 0 && !held) ptx::mbar_arrive(&ctl->tempty[acc]);
    held = false;
    if (lane < static_cast<int>(S)) ptx::mbar_arrive_remote(ptx::mapa(&ctl->rfull, lane));
    ok = ptx::mbar_wait_cluster(&ctl->rfull, rph, lim, abort);
    if (!__all_sync(0xFFFFFFFFu, ok)) {
      if (lane == 0) {
        ctl->abort = 1;
        raise_status(a.hdr, kStTimeout, 56);
      }
      break;
    }
    const int64_t C = a.cols[x.which];
    uint16_t* out = static_cast<uint16_t*>(a.out[x.which]) + static_cast<int64_t>(x.ad) * C * a.R;
    for (int i = tid; i < lanes * (nr / 8); i += 32 * kEpiWarps) {
      const int l = i & (lanes - 1), r = (i >> shift) * 8;
      const int64_t col = x.c0 + static_cast<int64_t>(rank) * lanes + l;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.0f;
      for (int c = 0; c < static_cast<int>(S); ++c) {
        // CTAs without a step (fewer steps than CTAs) have sent nothing
        if (x.steps * (c + 1) / static_cast<int>(S) == x.steps * c / static_cast<int>(S)) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += red[(c * kNR + r + j) * lanes + l];
      }
      if (col < C)
        *reinterpret_cast<uint4*>(out + col * a.R + x.r0 + r) =
            make_uint4(pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]),
                       pack2<DT>(v[6], v[7]));
    }
    __syncwarp();
    if (lane < static_cast<int>(S)) ptx::mbar_arrive_remote(ptx::mapa(&ctl->rempty, lane));
    rph ^= 1u;
    acc ^= 1;
    if (acc == 0) aph ^= 1u;
  }
}

struct OuterMaps {
  CUtensorMap m[4];  // x, v, d_y, u
};

template <int DT, int P>
__global__ void __launch_bounds__(Cfg<P>::kThreads, 1)
    rows_outer_kernel(const __grid_constant__ OuterMaps maps, const OuterArgs a) {
  using C = Cfg<P>;
  launch_order(false, a.late);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  float* red = reinterpret_cast<float*>(smem + C::kStages * C::kStageBytes);
  auto* ctl = reinterpret_cast<Ctl*>(smem + C::kStages * C::kStageBytes + C::kRedBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank(), S = cluster_size();

  if (routing_failed(a.hdr)) {  // the result is defined as zeros
    for (int w = 0; w < 2; ++w) {
      const int64_t n = static_cast<int64_t>(a.A) * a.cols[w] * a.R;
      for (int64_t q = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; q < n;
           q += static_cast<int64_t>(gridDim.x) * blockDim.x)
        static_cast<uint16_t*>(a.out[w])[q] = 0;
    }
    launch_end(a.late);
    return;
  }
  const uint32_t total =
      static_cast<uint32_t>(a.A) * a.r_blocks * static_cast<uint32_t>(a.blocks0 + a.blocks1);
  const uint32_t first = blockIdx.x / S, step = gridDim.x / S;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(&ctl->full[s], 3);
      ptx::mbar_init(&ctl->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&ctl->tfull[b], 1);
      ptx::mbar_init(&ctl->tempty[b], kEpiWarps);
    }
    ptx::mbar_init(&ctl->rfull, kEpiWarps * S);
    ptx::mbar_init(&ctl->rempty, kEpiWarps * S);
    ptx::mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0 && lane < 4) ptx::tma_prefetch_desc(&maps.m[lane]);
  if (warp == 1) {
    ptx::tmem_alloc(&ctl->tmem_base, C::kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before_sync();
  __syncthreads();
  ptx::cluster_sync();
  ptx::tc_fence_after_sync();
  const uint32_t tmem_base = ctl->tmem_base;

  if (warp == 0) {
    if (lane == 0) producer<P>(smem, ctl, maps.m, a, total, first, step, rank, S);
  } else if (warp == 1) {
    if (lane == 0) mma_issuer<DT, P>(smem, ctl, tmem_base, a, total, first, step, rank, S);
  } else if (warp < 2 + C::kGatherWarps) {
    gatherer<P>(smem, ctl, a, total, first, step, rank, S);
  } else if (warp >= C::kEpiWarp0) {
    epilogue<DT, P>(ctl, red, tmem_base, a, total, first, step, rank, S);
  }

  ptx::tc_fence_before_sync();
  __syncthreads();
  ptx::cluster_sync();  // no CTA leaves while another may still write to it
  if (warp == 1) {
    ptx::tc_fence_after_sync();
    ptx::tmem_dealloc(tmem_base, C::kTmemCols);
  }
  launch_end(a.late);
}

template <int DT, int P>
cudaError_t launch_t(const OuterMaps& maps, OuterArgs a, int num_sms, cudaStream_t stream) {
  using C = Cfg<P>;
  a.r_blocks = static_cast<uint32_t>((a.R + C::kNR - 1) / C::kNR);
  // Two CTAs a tile while there are few tiles for the SMs, so that one long adapter does not hold up
  // the rest; with many the exchange costs more than it evens out (8192 tokens, K 4096, N 2048, of
  // one adapter: 204 us alone, 190 in two; of 48: 227 alone, 264 in two).
  const int64_t all_tiles =
      static_cast<int64_t>(a.A) * a.r_blocks * (a.blocks0 + a.blocks1);
  const int S = all_tiles < 4 * num_sms ? 2 : 1;
  static ClusterLimits limits;
  const auto kern = rows_outer_kernel<DT, P>;
  int clusters = 0;
  const cudaError_t err = clusters_that_fit(&limits, kern, C::kThreads, smem_bytes<P>(), S, num_sms,
                                            &clusters);
  if (err != cudaSuccess) return err;
  if (all_tiles < clusters) clusters = static_cast<int>(all_tiles);
  return launch_pdl(kern, dim3(static_cast<unsigned>(S * clusters)), dim3(C::kThreads),
                    static_cast<size_t>(smem_bytes<P>()), stream, static_cast<unsigned>(S), maps, a);
}

}  // namespace

cudaError_t launch_rows_outer(int dtype, OuterArgs a, int num_sms, cudaStream_t stream) {
  a.blocks0 = static_cast<int32_t>((a.cols[0] + kM - 1) / kM);
  a.blocks1 = static_cast<int32_t>((a.cols[1] + kM - 1) / kM);
  OuterMaps maps;
  for (int w = 0; w < 2; ++w)
    if (!encode_map_rows(&maps.m[2 * w], dtype, a.left[w], a.cols[w], a.T, kRows) ||
        !encode_map_rows(&maps.m[2 * w + 1], dtype, a.right[w], low_width(a.R), a.right_rows, kRows))
      return cudaErrorInvalidValue;
  if (dtype == PGG_BF16)
    return a.R <= 32 ? launch_t<PGG_BF16, 1>(maps, a, num_sms, stream)
                     : launch_t<PGG_BF16, 2>(maps, a, num_sms, stream);
  return a.R <= 32 ? launch_t<PGG_F16, 1>(maps, a, num_sms, stream)
                   : launch_t<PGG_F16, 2>(maps, a, num_sms, stream);
}

}  // namespace pgg
