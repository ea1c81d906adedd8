// Products over few rows per group on tcgen05 tensor cores: what is streamed is
// the weight, so the weight is the MMA's M operand and the rows are its N.
//
//     gated    [gate | up][i, :] = x[token(i), :] W[g(i)],  h = prob * silu(gate) * up
//     shrink   u[i, :] = scale[ad] * x[token(i), :] a[ad]
//     adapt    y[t, :] = x[t, :] W + u[t, :] b[ad(t)]^T
//
// Tile: a block of at most NR rows x 128 weight columns (gated: 64 gates and
// their 64 ups) whose transposed fp32 accumulator, 128 lanes x NR columns, sits
// in tensor memory (two buffers). A cluster of S CTAs shares a tile: each
// reduces its part of K, then every CTA receives from the others, through
// distributed shared memory, the partial sums of its NR / S rows and adds them
// in the order of the CTAs: split-K without a second launch, atomics or
// workspace, bitwise repeatable. S = 1 when the tiles alone fill the GPU.
//
// A stage is 128 of k (64 for NR = 128): two 64-column panels of the weight by
// TMA (32 KB) and NR x rows, gathered by token with cp.async or, where they are
// neighbours, as TMA boxes. With NR = 16 six stages are in flight per SM, 192 KB
// of weight (adapt: four). The one thread that issues the MMAs is the limit
// otherwise: a wait, four MMAs and a commit took it 0.33 us a 64 of k, everything
// present; with eight MMAs to a wait and a commit it is 0.2.
//
// adapt with few tokens: rows stay in the caller's order, and the low-rank part
// is added in fp32 by the epilogue warps, which work it out from a row's u and
// its adapter's b (the bytes the operator needs anyway) while the weight still
// streams. A row meets no adapter but its own. The stream needs nothing from the
// launch before it (adapters_few.cu), so it starts while that one runs.
//
// Warp roles per CTA: 0 TMA, 1 tensor memory and MMA issue, one gather warp per
// stage slot, four epilogue warps. Waits are bounded as everywhere.

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

constexpr int kM = 128;            // weight columns per tile: accumulator lanes
constexpr int kFK = 64;            // reduction of one 128-byte row of x
constexpr int kEpiWarps = 4;
constexpr int kMaxSplit = 8;

template <int MODE, int NR, int PANELS>
struct Cfg {
  static constexpr int kSub = NR <= 64 ? 2 : 1;       // 64s of k per stage
  static constexpr int kPanel = kSub * kFK * 128;     // k rows x 128 bytes (64 columns)
  static constexpr int kABytes = PANELS * kPanel;
  static constexpr int kSubBytes = NR * 128;          // rows x 64 of k
  static constexpr int kBBytes = kSub * kSubBytes;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kRedBytes = NR * kM * 4;  // S slots of NR / S rows x 128 lanes
  // adapt: a block of the launch before it (the low-rank rows: 17 KB, 256 threads of 64 registers)
  // fits beside, so that the weight streams while that one runs: 48 tokens, 64 adapters, K 7168,
  // N 4096 24.4 -> 24.0 us, 32 tokens of rank 32 28.1 -> 25.9.
  static constexpr int kRoom = MODE == kAdapt ? 182 * 1024 : 226 * 1024;
  static constexpr int kFit = (kRoom - 2048 - kRedBytes) / kStageBytes;
  static constexpr int kStages = kFit < 12 ? kFit : 12;
  static constexpr int kThreads = 32 * (2 + kStages + kEpiWarps);
  static constexpr int kTmemCols = 2 * NR < 32 ? 32 : 2 * NR;
  static_assert(kSubBytes % 1024 == 0, "operand alignment");
};

template <int STAGES>
struct Ctl {
  uint64_t full[STAGES];   // weight bytes + the gather warp's arrival
  uint64_t empty[STAGES];  // MMAs of the stage done
  uint64_t tfull[2], tempty[2];
  uint64_t rfull, rempty;  // partial sums of all CTAs received here / mine read by all CTAs
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

template <int MODE, int NR, int PANELS>
constexpr int smem_bytes() {
  using C = Cfg<MODE, NR, PANELS>;
  return C::kStages * C::kStageBytes + C::kRedBytes +
         static_cast<int>(sizeof(Ctl<C::kStages>)) + 1024;
}

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
  return r;
}

struct Tile {
  int64_t g, row0, n0;  // n0: first output column (gated: of h)
  int rows, urow;
};

template <int MODE, int NR>
__device__ __forceinline__ Tile tile_of(uint32_t t, const RowsArgs& a) {
  const uint32_t rb = t / static_cast<uint32_t>(a.n_blocks);
  Tile x;
  x.n0 = static_cast<int64_t>(t - rb * static_cast<uint32_t>(a.n_blocks)) *
         (MODE == kGated ? 64 : kM);
  if constexpr (MODE == kAdapt) {
    x.g = 0;
    x.row0 = static_cast<int64_t>(rb) * NR;
    x.rows = a.M - x.row0 < NR ? static_cast<int>(a.M - x.row0) : NR;
    x.urow = 0;
  } else {
    int4 e = a.rblist[check_index(a.hdr, rb, a.max_row_blocks, 90)];
    if (!check_ok(a.hdr,
                  e.x >= 0 && e.x <= a.G && e.y >= 0 && e.z >= 0 && e.z <= NR &&
                      static_cast<int64_t>(e.y) + e.z <= a.M,
                  91))
      e = make_int4(0, 0, 0, 0);
    x.g = e.x;
    x.row0 = e.y;
    x.rows = e.z;
    x.urow = e.w;
  }
  return x;
}

// The tiles that this CTA walks, and its part of the reduction.
struct Walk {
  uint32_t first, step, total;
  int ks0, ks1;
};

// First token of the tile's rows if they are neighbours (they come as one TMA box then), else -1.
template <int MODE>
__device__ __forceinline__ int32_t box_of(const RowsArgs& a, const Tile& x) {
  if (MODE == kAdapt) return static_cast<int32_t>(x.row0);
  if (MODE == kShrink) return box_of_rows(a.rowinfo, x.row0, x.rows);
  return -1;
}

// Rows of tokens without an adapter have nothing to shrink.
template <int MODE>
__device__ __forceinline__ bool skipped(const RowsArgs& a, const Tile& x) {
  return MODE == kShrink && x.g >= a.G;
}

template <int MODE, int NR, int PANELS>
__device__ void w_producer(uint8_t* smem, Ctl<Cfg<MODE, NR, PANELS>::kStages>* ctl,
                           const CUtensorMap* tm_w, const CUtensorMap* tm_x, const RowsArgs& a,
                           const Walk& k) {
  using C = Cfg<MODE, NR, PANELS>;
  const uint64_t lim = a.wait_limit_ns;
  volatile int* abort = &ctl->abort;
  int stage = 0;
  uint32_t phase = 0, outstanding = 0, last_parity = 0;
  bool failed = false;
  for (uint32_t t = k.first; t < k.total && !failed; t += k.step) {
    const Tile x = tile_of<MODE, NR>(t, a);
    if (skipped<MODE>(a, x)) continue;
    int32_t col[2];
    bool on[2];
    for (int j = 0; j < 2; ++j) {
      col[j] = static_cast<int32_t>(MODE == kGated ? x.n0 + (j ? a.N : 0) : x.n0 + 64 * j);
      on[j] = j < PANELS && (MODE == kGated || x.n0 + 64 * j < a.N);
    }
    const int32_t box = box_of<MODE>(a, x);
    const uint32_t bytes =
        (on[0] ? C::kPanel : 0) + (on[1] ? C::kPanel : 0) + (box >= 0 ? C::kBBytes : 0);
    for (int ks = k.ks0; ks < k.ks1; ++ks) {
      if (!ptx::mbar_wait(&ctl->empty[stage], phase ^ 1u, lim, abort)) {
        failed = true;
        break;
      }
      uint8_t* sa = smem + stage * C::kStageBytes;
      ptx::mbar_arrive_expect_tx(&ctl->full[stage], bytes);
      for (int j = 0; j < C::kSub && box >= 0; ++j)
        ptx::tma_load_2d(sa + C::kABytes + j * C::kSubBytes, tm_x, &ctl->full[stage],
                         (ks * C::kSub + j) * kFK, box);
      for (int j = 0; j < PANELS; ++j)
        if (on[j])
          ptx::tma_load_3d(sa + j * C::kPanel, tm_w, &ctl->full[stage], col[j],
                           ks * C::kSub * kFK, static_cast<int32_t>(x.g));
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
    raise_status(a.hdr, kStTimeout, 42);
  }
  int no_abort = 0;
  for (int s = 0; s < C::kStages; ++s)
    if (outstanding & (1u << s)) ptx::mbar_wait(&ctl->full[s], (last_parity >> s) & 1u, lim, &no_abort);
}

// Gather warp w fills stage slot w: rows (lane >> 3) + 4 q, 16-byte chunk lane & 7.
template <int MODE, int NR, int PANELS>
__device__ void x_gatherer(uint8_t* smem, Ctl<Cfg<MODE, NR, PANELS>::kStages>* ctl, const RowsArgs& a,
                           const Walk& k) {
  using C = Cfg<MODE, NR, PANELS>;
  const uint64_t lim = a.wait_limit_ns;
  volatile int* abort = &ctl->abort;
  const int w = (threadIdx.x >> 5) - 2;
  const int lane = threadIdx.x & 31, c = lane & 7;
  const char* xb = static_cast<const char*>(a.x);
  const uint32_t sb = ptx::smem_addr(smem + w * C::kStageBytes + C::kABytes);
  const int steps = k.ks1 - k.ks0;
  constexpr uint32_t kNoRow = 0xFFFFFFFFu;
  const uint32_t row_units = static_cast<uint32_t>(a.K / 8);
  uint32_t row16[NR / 4];
  uint32_t phase = 0;
  bool failed = false;
  int kb = w;  // the warp's next step, counted from the start of tile t
  for (uint32_t t = k.first; t < k.total && !failed; t += k.step) {
    const Tile x = tile_of<MODE, NR>(t, a);
    if (skipped<MODE>(a, x)) continue;
    const int32_t box = box_of<MODE>(a, x);
    if (kb < steps && box < 0) {
#pragma unroll
      for (int q = 0; q < NR / 4; ++q) {
        const int rr = (lane >> 3) + 4 * q;
        row16[q] = kNoRow;
        if (rr < x.rows) {
          const int64_t row = check_index(a.hdr, x.row0 + rr, a.M, 92);
          row16[q] = static_cast<uint32_t>(
                         check_index(a.hdr, a.rowinfo[row].token, a.batch, 93)) *
                     row_units;
        }
      }
    }
    for (; kb < steps; kb += C::kStages) {
      if (!ptx::mbar_wait(&ctl->empty[w], phase ^ 1u, lim, abort)) {
        failed = true;
        break;
      }
      if (box < 0) {
#pragma unroll
        for (int j = 0; j < C::kSub; ++j) {
          const int64_t kk = static_cast<int64_t>((k.ks0 + kb) * C::kSub + j) * kFK + c * 8;
          const bool k_ok = kk < a.K;
          const char* xk = xb + kk * 2;
#pragma unroll
          for (int q = 0; q < NR / 4; ++q) {
            const int rr = (lane >> 3) + 4 * q;
            const bool ok = k_ok && row16[q] != kNoRow;
            const void* src = ok ? static_cast<const void*>(
                                       xk + (static_cast<uint64_t>(row16[q]) << 4))
                                 : static_cast<const void*>(xb);
            ptx::cp_async_16(sb + j * C::kSubBytes + rr * 128 + ((c ^ (rr & 7)) << 4), src,
                             ok ? 16u : 0u);
          }
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
    if (lane == 0) raise_status(a.hdr, kStTimeout, 43);
  }
}

template <int DT, int MODE, int NR, int PANELS>
__device__ void mma_issuer(uint8_t* smem, Ctl<Cfg<MODE, NR, PANELS>::kStages>* ctl, uint32_t tmem_base,
                           const RowsArgs& a, const Walk& k) {
  using C = Cfg<MODE, NR, PANELS>;
  constexpr uint32_t kFmt = DT == PGG_BF16 ? 1u : 0u;
  constexpr uint32_t idesc = ptx::idesc_make(kFmt, kM, NR) | (1u << 15);  // A MN-major
  const uint64_t lim = a.wait_limit_ns;
  volatile int* abort = &ctl->abort;
  int stage = 0, acc = 0;
  uint32_t phase = 0, aph = 0;
  bool issued = false, failed = false;
  for (uint32_t t = k.first; t < k.total && !failed; t += k.step) {
    if (skipped<MODE>(a, tile_of<MODE, NR>(t, a))) continue;
    if (!ptx::mbar_wait(&ctl->tempty[acc], aph ^ 1u, lim, abort)) {
      failed = true;
      break;
    }
    ptx::tc_fence_after_sync();
    const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * NR);
    for (int ks = k.ks0; ks < k.ks1; ++ks) {
      if (!ptx::mbar_wait(&ctl->full[stage], phase, lim, abort)) {
        failed = true;
        break;
      }
      ptx::tc_fence_after_sync();
      const uint32_t sa = ptx::smem_addr(smem + stage * C::kStageBytes);
      // with one panel the upper 64 lanes read it again (and are not looked at): the operand stays
      // inside its stage
      const uint64_t da = ptx::sdesc_sw128_mn(sa, PANELS == 1 ? 0 : C::kPanel);
      const uint64_t db = ptx::sdesc_sw128(sa + C::kABytes);
#pragma unroll
      for (int kk = 0; kk < C::kSub * kFK / 16; ++kk)
        ptx::mma_f16(d_tmem, da + static_cast<uint64_t>((kk * 16 * 128) >> 4),
                     db + static_cast<uint64_t>(((kk / 4) * C::kSubBytes + (kk % 4) * 32) >> 4),
                     idesc, (ks > k.ks0 || kk > 0) ? 1u : 0u);
      issued = true;
      ptx::mma_commit(&ctl->empty[stage]);
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (failed) break;
    ptx::mma_commit(&ctl->tfull[acc]);
    acc ^= 1;
    if (acc == 0) aph ^= 1u;
  }
  if (failed) {
    ctl->abort = 1;
    raise_status(a.hdr, kStTimeout, 44);
  }
  if (issued) {
    int no_abort = 0;
    ptx::mma_commit(&ctl->drain);
    ptx::mbar_wait(&ctl->drain, 0u, lim, &no_abort);
  }
}

// Sums of the S CTAs' partial sums for four neighbouring lanes (weight columns) of a row: red holds
// S slots of `slot` floats, rows of 128.
__device__ __forceinline__ float4 sum4(const float* red, int slot, uint32_t S, int at) {
  float4 v = *reinterpret_cast<const float4*>(red + at);
  for (uint32_t s = 1; s < S; ++s) {
    const float4 p = *reinterpret_cast<const float4*>(red + s * slot + at);
    v.x += p.x;
    v.y += p.y;
    v.z += p.z;
    v.w += p.w;
  }
  return v;
}

template <int DT>
__device__ __forceinline__ uint2 pack4(const float4& v) {
  return make_uint2(pack2<DT>(v.x, v.y), pack2<DT>(v.z, v.w));
}

// Output of tile rows j0 .. j0 + n - 1, four columns a thread (N is a multiple of 8, so all four
// are there or none is). One warp at a time would be bound by its own latency here: the rows are
// spread over all the epilogue's threads.
template <int DT, int MODE, int LR>
__device__ __forceinline__ void write_rows(const float* red, int slot, uint32_t S, const RowsArgs& a,
                                           const Tile& x, int j0, int n, bool failed,
                                           const float (&lr)[LR][4], float row_scale) {
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
  if constexpr (MODE == kGated) {
    // 16 threads a row, two rows a warp: gates in lanes 0 .. 63 of the tile, ups in 64 .. 127
    const int f4 = 4 * (lane & 15);
    const int64_t f = x.n0 + f4;
#pragma unroll 2
    for (int j = 2 * warp + (lane >> 4); j < (n + 1) / 2 * 2; j += 2 * kEpiWarps) {
      // (both rows of a pair take part in the shuffle)
      const float p = __shfl_sync(0xFFFFFFFFu, row_scale, 2 * ((j - 2 * warp) / 8) + (j & 1));
      if (j >= n || f >= a.N) continue;
      const int64_t row = x.row0 + j0 + j;
      const float4 g = sum4(red, slot, S, j * kM + f4);
      const float4 u = sum4(red, slot, S, j * kM + 64 + f4);
      const float4 h = make_float4(gate(g.x, u.x, p), gate(g.y, u.y, p), gate(g.z, u.z, p),
                                   gate(g.w, u.w, p));
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * a.N + f) = pack4<DT>(h);
      if (a.gate_up) {
        uint16_t* gu = static_cast<uint16_t*>(a.gate_up) + row * 2 * a.N + f;
        *reinterpret_cast<uint2*>(gu) = pack4<DT>(g);
        *reinterpret_cast<uint2*>(gu + a.N) = pack4<DT>(u);
      }
    }
  } else if constexpr (MODE == kShrink) {
    const int left = static_cast<int>(a.N - x.n0 < kM ? a.N - x.n0 : kM);
    const int groups = left / 4;  // of four columns
    const int64_t width = a.low_form == kLowSplit ? low_width(a.N) : a.N;
#pragma unroll 2
    for (int i = 32 * warp + lane; i < n * groups; i += 32 * kEpiWarps) {
      const int j = i / groups, c = 4 * (i - j * groups);
      float4 v = sum4(red, slot, S, j * kM + c);
      v = make_float4(v.x * row_scale, v.y * row_scale, v.z * row_scale, v.w * row_scale);
      const int64_t row = (static_cast<int64_t>(x.urow) + j0 + j) * width, r = x.n0 + c;
      if (a.low_form == kLowFloat) {
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + row + r) = v;
        continue;
      }
      uint16_t* p = static_cast<uint16_t*>(a.out) + row;
      if (a.low_form == kLowRounded) {
        *reinterpret_cast<uint2*>(p + r) = pack4<DT>(v);
        continue;
      }
      ushort4 hi, lo;
      split16<DT>(v.x, &hi.x, &lo.x);
      split16<DT>(v.y, &hi.y, &lo.y);
      split16<DT>(v.z, &hi.z, &lo.z);
      split16<DT>(v.w, &hi.w, &lo.w);
      p += r / 32 * 64 + r % 32;
      *reinterpret_cast<ushort4*>(p) = hi;
      *reinterpret_cast<ushort4*>(p + 32) = lo;
    }
  } else {
    const int64_t c = x.n0 + 4 * lane;
#pragma unroll
    for (int q = 0; q < LR; ++q) {
      const int j = warp + kEpiWarps * q;
      if (j >= n || c >= a.N) continue;
      float4 v = sum4(red, slot, S, j * kM + 4 * lane);
      v = failed ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                 : make_float4(v.x + lr[q][0], v.y + lr[q][1], v.z + lr[q][2], v.w + lr[q][3]);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + (x.row0 + j0 + j) * a.N + c) =
          pack4<DT>(v);
    }
  }
}

// Low-rank part of tile rows j0 + j, j = warp, warp + 4, ... < n: each row's u [R] against its own
// adapter's b [n][R], 8 ranks (16 bytes of b) at a time, in fp32; lane l takes columns 4 l + i.
template <int DT, int LR>
__device__ __forceinline__ void low_rank(const RowsArgs& a, const Tile& x, int j0, int n,
                                         float (&lr)[LR][4]) {
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
  // lane i loads the adapter of this warp's i-th row
  int ids = -1;
  if (lane < LR && warp + kEpiWarps * lane < n)
    ids = static_cast<int>(a.adapter[x.row0 + j0 + warp + kEpiWarps * lane]);
  const bool col = x.n0 + 4 * lane < a.N;
#pragma unroll
  for (int q0 = 0; q0 < LR; q0 += 2) {  // two rows' loads at a time: latency is what this costs
#pragma unroll
    for (int q = q0; q < q0 + 2; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) lr[q][i] = 0.0f;
    if (warp + kEpiWarps * q0 >= n) continue;
    const float* u[2];
    const char* b[2];
    bool on[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int64_t ad = __shfl_sync(0xFFFFFFFFu, ids, q0 + e);
      on[e] = ad >= 0 && ad < a.G;  // (-1 past the rows)
      u[e] = static_cast<const float*>(a.u) + (x.row0 + j0 + warp + kEpiWarps * (q0 + e)) * a.R;
      b[e] = static_cast<const char*>(a.b) + (((on[e] ? ad : 0) * a.N + x.n0 + 4 * lane) * a.R) * 2;
    }
#pragma unroll 2
    for (int r0 = 0; r0 < a.R; r0 += 8) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float4 ua = make_float4(0.0f, 0.0f, 0.0f, 0.0f), ub = ua;
        uint4 w[4];
        if (on[e]) {
          ua = __ldcg(reinterpret_cast<const float4*>(u[e] + r0));
          ub = __ldcg(reinterpret_cast<const float4*>(u[e] + r0 + 4));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[i] = make_uint4(0, 0, 0, 0);
          if (on[e] && col)
            w[i] = __ldg(reinterpret_cast<const uint4*>(b[e] + (i * a.R + r0) * 2));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float& v = lr[q0 + e][i];
          const float2 b0 = unpack2<DT>(w[i].x), b1 = unpack2<DT>(w[i].y);
          const float2 b2 = unpack2<DT>(w[i].z), b3 = unpack2<DT>(w[i].w);
          v = fmaf(ua.x, b0.x, v);
          v = fmaf(ua.y, b0.y, v);
          v = fmaf(ua.z, b1.x, v);
          v = fmaf(ua.w, b1.y, v);
          v = fmaf(ub.x, b2.x, v);
          v = fmaf(ub.y, b2.y, v);
          v = fmaf(ub.z, b3.x, v);
          v = fmaf(ub.w, b3.y, v);
        }
      }
    }
  }
}

template <int DT, int MODE, int NR, int PANELS>
__device__ void epilogue(Ctl<Cfg<MODE, NR, PANELS>::kStages>* ctl, float* red, uint32_t tmem_base,
                         const RowsArgs& a, const Walk& k, uint32_t rank, uint32_t S) {
  const uint64_t lim = a.wait_limit_ns;
  volatile int* abort = &ctl->abort;
  const int lane = threadIdx.x & 31;
  const int quarter = (threadIdx.x >> 5) & 3;
  const int shift = 31 - __clz(NR / static_cast<int>(S));
  const int per = 1 << shift;  // rows that each CTA of the cluster finishes
  const int slot = per * kM;
  int acc = 0;
  uint32_t aph = 0, rph = 0;
  bool failed_input = false;
  if constexpr (MODE == kAdapt) {
    ptx::griddep_wait();  // u and the ids' check; the weight stream is under way already
    failed_input = routing_failed(a.hdr);
  }
  bool held = a.hold_release != 0;
  for (uint32_t t = k.first; t < k.total; t += k.step) {
    const Tile x = tile_of<MODE, NR>(t, a);
    if (skipped<MODE>(a, x)) {
      // (fills of padded rows belong to adapters only)
      continue;
    }
    const int j0 = static_cast<int>(rank) * per;  // this CTA finishes rows j0 .. j0 + n - 1
    const int n = x.rows - j0 < per ? x.rows - j0 : per;
    // what the rows are scaled by is loaded ahead: lane i holds the weight of this warp's i-th row,
    // rows 2 q, 2 q + 1, 2 q + 8, 2 q + 9, ... for warp q
    float row_scale = 1.0f;
    if constexpr (MODE == kGated) {
      const int j = 2 * quarter + (lane & 1) + 8 * (lane >> 1);
      if (a.probs && j < n)
        row_scale = a.probs[check_index(
            a.hdr, a.rowinfo[check_index(a.hdr, x.row0 + j0 + j, a.M, 94)].rank, a.M, 95)];
    } else if constexpr (MODE == kShrink) {
      if (a.scale) row_scale = a.scale[x.g];
    }
    constexpr int kLR = MODE == kAdapt ? NR / kEpiWarps : 1;
    float lr[kLR][4];
    if constexpr (MODE == kAdapt) {
      if (!failed_input) low_rank<DT, kLR>(a, x, j0, n, lr);
    }
    bool ok = ptx::mbar_wait(&ctl->tfull[acc], aph, lim, abort);
    // the others have read what they got from this CTA for the tile before
    ok = ok && ptx::mbar_wait_cluster(&ctl->rempty, rph ^ 1u, lim, abort);
    if (!__all_sync(0xFFFFFFFFu, ok)) {
      if (lane == 0) {
        ctl->abort = 1;
        raise_status(a.hdr, kStTimeout, 45);
      }
      break;
    }
    ptx::tc_fence_after_sync();
    const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(32 * quarter) << 16) +
                            static_cast<uint32_t>(acc * NR);
    const uint32_t mine = 32 * quarter + lane;
    // (lanes past the rank hold nothing)
    const int cols = MODE == kShrink && x.n0 + 32 * quarter >= a.N ? 0 : x.rows;
    // (whole groups of 16 rows: what lies past the tile's rows is sent and not read)
#pragma unroll 1
    for (int c0 = 0; c0 < NR && c0 < cols; c0 += 16) {
      uint32_t v[16];
      ptx::tmem_ld_32x32b_x16(t_lane + static_cast<uint32_t>(c0), v);
      ptx::tmem_ld_wait();
      if (S == 1) {
#pragma unroll
        for (int i = 0; i < 16; ++i) red[(c0 + i) * kM + mine] = __uint_as_float(v[i]);
      } else {
        // row j goes to slot `rank` of the CTA that finishes it
        const uint32_t base = ptx::smem_addr(red + rank * slot + mine);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = c0 + i;
          st_cluster_f32(mapa_addr(base + (j & (per - 1)) * kM * 4, j >> shift),
                         __uint_as_float(v[i]));
        }
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
        raise_status(a.hdr, kStTimeout, 46);
      }
      break;
    }
    write_rows<DT, MODE, kLR>(red, slot, S, a, x, j0, n, failed_input, lr, row_scale);
    if constexpr (MODE == kShrink) {
      if (a.padded) {  // the adapter's last block: rows that fill it up
        const int end = x.rows + rows_to_fill(a, make_int4(static_cast<int>(x.g),
                                                           static_cast<int>(x.row0), x.rows,
                                                           x.urow));
        for (int j = x.rows + static_cast<int>(rank) * kEpiWarps + quarter; j < end;
             j += static_cast<int>(S) * kEpiWarps)
          for (int64_t c = x.n0 + lane; c < a.N && c < x.n0 + kM; c += 32) {
            uint16_t* p = static_cast<uint16_t*>(a.out) +
                          (static_cast<int64_t>(x.urow) + j) * low_width(a.N) + c / 32 * 64 + c % 32;
            p[0] = 0;
            p[32] = 0;
          }
      }
    }
    __syncwarp();
    if (lane < static_cast<int>(S)) ptx::mbar_arrive_remote(ptx::mapa(&ctl->rempty, lane));
    rph ^= 1u;
    acc ^= 1;
    if (acc == 0) aph ^= 1u;
  }
}

template <int DT, int MODE, int NR, int PANELS>
__global__ void __launch_bounds__(Cfg<MODE, NR, PANELS>::kThreads, 1)
    rows_skinny_kernel(const __grid_constant__ CUtensorMap tm_w,
                       const __grid_constant__ CUtensorMap tm_x, const RowsArgs a) {
  using C = Cfg<MODE, NR, PANELS>;
  if (MODE != kAdapt) launch_order(a.early, a.late);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  float* red = reinterpret_cast<float*>(smem + C::kStages * C::kStageBytes);
  auto* ctl = reinterpret_cast<Ctl<C::kStages>*>(smem + C::kStages * C::kStageBytes + C::kRedBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank(), S = cluster_size();

  if (MODE != kAdapt && routing_failed(a.hdr)) {
    if (MODE == kGated) zero_rows16(a);
    launch_end(a.late);
    return;
  }
  Walk k;
  const uint32_t row_blocks = MODE == kAdapt ? static_cast<uint32_t>((a.M + NR - 1) / NR)
                                             : a.hdr->n_row_blocks;
  k.total = row_blocks * static_cast<uint32_t>(a.n_blocks);
  k.first = blockIdx.x / S;
  k.step = gridDim.x / S;
  const int nks = static_cast<int>((a.K + C::kSub * kFK - 1) / (C::kSub * kFK));
  k.ks0 = nks * static_cast<int>(rank) / static_cast<int>(S);
  k.ks1 = nks * (static_cast<int>(rank) + 1) / static_cast<int>(S);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(&ctl->full[s], 2);
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
  if (warp == 0 && lane == 0) {
    ptx::tma_prefetch_desc(&tm_w);
    if (MODE != kGated) ptx::tma_prefetch_desc(&tm_x);
  }
  if (warp == 1) {
    ptx::tmem_alloc(&ctl->tmem_base, C::kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before_sync();
  __syncthreads();
  ptx::cluster_sync();  // the others' barriers are ready before anything arrives there
  ptx::tc_fence_after_sync();
  const uint32_t tmem_base = ctl->tmem_base;

  if (warp == 0) {
    if (lane == 0) w_producer<MODE, NR, PANELS>(smem, ctl, &tm_w, &tm_x, a, k);
  } else if (warp == 1) {
    if (lane == 0) mma_issuer<DT, MODE, NR, PANELS>(smem, ctl, tmem_base, a, k);
  } else if (warp < 2 + C::kStages) {
    x_gatherer<MODE, NR, PANELS>(smem, ctl, a, k);
  } else {
    epilogue<DT, MODE, NR, PANELS>(ctl, red, tmem_base, a, k, rank, S);
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

// CTAs per tile: the split of K that leaves the fewest steps on the critical path for about
// `tiles` tiles, counting kTileCost steps per tile for its epilogue and exchange.
int choose_split(int64_t tiles, int nks, int NR, int num_sms) {
  constexpr int kTileCost = 5;
  int best = 1;
  int64_t best_cost = 0;
  for (int s = 1; s <= kMaxSplit && s <= nks && s <= NR; s *= 2) {
    const int64_t clusters = num_sms / s;
    const int64_t waves = (tiles + clusters - 1) / clusters;
    const int64_t cost = waves * ((nks + s - 1) / s + kTileCost);
    if (s == 1 || cost < best_cost) {
      best = s;
      best_cost = cost;
    }
  }
  return best;
}

template <int DT, int MODE, int NR, int PANELS>
cudaError_t launch_t(const CUtensorMap (&tm)[2], const RowsArgs& a, int64_t tiles, int num_sms,
                     cudaStream_t stream) {
  using C = Cfg<MODE, NR, PANELS>;
  constexpr int smem = smem_bytes<MODE, NR, PANELS>();
  static_assert(smem <= 227 * 1024, "shared memory per CTA");
  auto kern = rows_skinny_kernel<DT, MODE, NR, PANELS>;
  const int nks = static_cast<int>((a.K + C::kSub * kFK - 1) / (C::kSub * kFK));
  const int S = choose_split(tiles, nks, NR, num_sms);
  static ClusterLimits limits;
  int clusters = 0;
  const cudaError_t err =
      clusters_that_fit(&limits, kern, C::kThreads, smem, S, num_sms, &clusters);
  if (err != cudaSuccess) return err;
  int64_t want = num_sms / S;
  const int64_t most = (MODE == kAdapt ? (a.M + NR - 1) / NR : a.max_row_blocks) * a.n_blocks;
  if (most < want) want = most;
  if (clusters < want) want = clusters;
  return launch_pdl(kern, dim3(static_cast<unsigned>(S * want)), dim3(C::kThreads),
                    static_cast<size_t>(smem), stream, static_cast<unsigned>(S), tm[0], tm[1], a);
}

template <int DT>
cudaError_t launch_mode(RowsMode mode, int NR, const CUtensorMap (&m)[2], const RowsArgs& a,
                        int64_t tiles, int sms, cudaStream_t st) {
  if (mode == kGated) {
    if (NR == 16) return launch_t<DT, kGated, 16, 2>(m, a, tiles, sms, st);
    if (NR == 32) return launch_t<DT, kGated, 32, 2>(m, a, tiles, sms, st);
    if (NR == 64) return launch_t<DT, kGated, 64, 2>(m, a, tiles, sms, st);
    if (NR == 128) return launch_t<DT, kGated, 128, 2>(m, a, tiles, sms, st);
  } else if (mode == kShrink) {
    // ranks up to 64 fit one panel of the factor: more stages in flight
    if (NR == 16 && a.N <= 64) return launch_t<DT, kShrink, 16, 1>(m, a, tiles, sms, st);
    if (NR == 16) return launch_t<DT, kShrink, 16, 2>(m, a, tiles, sms, st);
    if (NR == 64 && a.N <= 64) return launch_t<DT, kShrink, 64, 1>(m, a, tiles, sms, st);
    if (NR == 64) return launch_t<DT, kShrink, 64, 2>(m, a, tiles, sms, st);
  } else if (mode == kAdapt) {
    if (NR == 16) return launch_t<DT, kAdapt, 16, 2>(m, a, tiles, sms, st);
    if (NR == 32) return launch_t<DT, kAdapt, 32, 2>(m, a, tiles, sms, st);
    if (NR == 64) return launch_t<DT, kAdapt, 64, 2>(m, a, tiles, sms, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

// live_blocks: about how many row blocks there will be (the launch's shape goes by it, nothing
// else).
cudaError_t launch_rows_skinny(int dtype, RowsMode mode, int NR, RowsArgs a, int64_t live_blocks,
                               int num_sms, cudaStream_t stream) {
  const int64_t tile_n = mode == kGated ? 64 : kM;
  a.n_blocks = static_cast<int32_t>((a.N + tile_n - 1) / tile_n);
  CUtensorMap tm[2];  // weight, x
  std::memset(tm, 0, sizeof(tm));
  const int64_t cols = mode == kGated ? 2 * a.N : a.N;
  if (!encode_map_3d(&tm[0], dtype, a.w, cols, a.K, mode == kAdapt ? 1 : a.G,
                     NR <= 64 ? 2 * kFK : kFK))
    return cudaErrorInvalidValue;
  if (mode != kGated && !encode_map_rows(&tm[1], dtype, a.x, a.K, a.batch, NR))
    return cudaErrorInvalidValue;
  const int64_t tiles = live_blocks * a.n_blocks;
  if (dtype == PGG_BF16)
    return launch_mode<PGG_BF16>(mode, NR, tm, a, tiles, num_sms, stream);
  if (dtype == PGG_F16) return launch_mode<PGG_F16>(mode, NR, tm, a, tiles, num_sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pgg
