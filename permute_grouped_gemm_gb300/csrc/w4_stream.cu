// Products with 4-bit expert weights, few rows an expert: the codes are
// streamed once per block of up to 32 rows, and that stream is the bound.
//
// Tile: 128 columns of one expert (gated: 64 gates and their 64 ups) x NR rows.
// A stage is 256 of k: 128 columns x 128 bytes of codes by TMA, the rows of x,
// and the columns' scales. Eight warps take 32 columns x half of k each: codes
// are unpacked in registers, (v >> 4 j) & 0x000F000F | magic is the pair of
// numbers 2^7 + code (bf16; 2^10 + code in fp16), from which 2^7 + zero is
// subtracted exactly, and go as the A operand into mma.sync m16n8k16 with eight
// rows of x as B. (A word holds codes k .. k + 7, so such a pair is k + j, k + 4 + j;
// the warp that lays out x pairs it the same way.) A group's fp32 sum is then
// multiplied by its scale: the weights are never rounded. The warp-wide product
// is used because the operand is made in registers: for tcgen05 it would go
// through shared memory once more (5 bytes a code, where 128 a cycle serve all)
// or through tensor memory and two hand-overs a step; with eight to 32 rows the
// product itself is far from a bound.
//
// The tiles' steps of k are dealt to the CTAs in equal runs. A tile that is
// shared leaves fp32 parts in the workspace, and the CTA that comes last (a
// counter) adds them in the order of k: no CTA waits for another, and the result
// does not depend on who comes last.
//
// Warps: 0 TMA; one per stage slot for x and the scales; eight for the product.
// Waits are bounded as everywhere.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <cstring>

#include "pgg_block.h"
#include "pgg_ops_launch.h"
#include "pgg_ops_mma.cuh"
#include "pgg_ptx.cuh"

namespace pgg {
namespace {

constexpr int kTile = 128;       // columns of codes
constexpr int kStep = 256;       // of k a stage
constexpr int kMmaWarps = 8;     // 4 x 32 columns, 2 halves of a stage's k
constexpr int kCodeBytes = kTile * kStep / 2;
constexpr int kRedStride = kTile + 4;

template <int NT, int U, bool ZEROS>
struct Cfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kUnits = kStep / U;  // groups of a stage, U of k each
  static constexpr int kXBytes = kRows * kStep * 2;
  static constexpr int kScaleBytes = kUnits * kTile * 4;
  static constexpr int kStageBytes = kCodeBytes + kXBytes + kScaleBytes * (ZEROS ? 2 : 1);
  static constexpr int kRedBytes = kRows * kRedStride * 4;
  static constexpr int kFit = (225 * 1024 - kRedBytes - 1024) / kStageBytes;
  static constexpr int kStages = kFit < 7 ? kFit : 7;  // (16 warps: 128 registers a thread)
  static constexpr int kThreads = 32 * (1 + kStages + kMmaWarps);
  static constexpr int kSmem = kStages * kStageBytes + kRedBytes + 2048;
  static_assert(kStageBytes % 1024 == 0, "operand alignment");
};

struct Ctl {
  uint64_t full[8];   // codes' bytes, and x and scales written
  uint64_t empty[8];  // read by all eight warps
  int abort;
  int last;           // this CTA is the one that adds the tile's parts
};

// The steps [begin, end) of this CTA among `total`, dealt to `ctas` of them; nks steps a tile.
struct Walk {
  int64_t begin, end, total, ctas;
  int nks;
};

struct Tile {
  int64_t g, row0, n0;
  int rows;
};

template <int NR>
__device__ __forceinline__ Tile tile_of(uint32_t t, const W4Args& a) {
  const uint32_t rb = t / static_cast<uint32_t>(a.n_blocks);
  int4 e = a.rblist[check_index(a.hdr, rb, a.max_row_blocks, 170)];
  if (!check_ok(a.hdr,
                e.x >= 0 && e.x < a.G && e.y >= 0 && e.z >= 0 && e.z <= NR &&
                    static_cast<int64_t>(e.y) + e.z <= a.M,
                171))
    e = make_int4(0, 0, 0, 0);
  Tile x;
  x.n0 = static_cast<int64_t>(t - rb * static_cast<uint32_t>(a.n_blocks)) *
         (a.product == PGG_W4_GATED ? kTile / 2 : kTile);
  x.g = e.x;
  x.row0 = e.y;
  x.rows = e.z;
  return x;
}

// Column of codes of the tile's column r, or -1.
__device__ __forceinline__ int64_t column_of(const W4Args& a, const Tile& x, int r) {
  if (a.product == PGG_W4_GATED) {
    const int64_t f = x.n0 + (r & 63);
    return f < a.N ? f + (r >= 64 ? a.N : 0) : -1;
  }
  return x.n0 + r < a.N ? x.n0 + r : -1;
}

template <int NT, int U, bool ZEROS>
__device__ void code_producer(uint8_t* smem, Ctl* ctl, const CUtensorMap* tm, const W4Args& a,
                              const Walk& k) {
  using C = Cfg<NT, U, ZEROS>;
  volatile int* abort = &ctl->abort;
  int stage = 0;
  uint32_t phase = 0, outstanding = 0, last_parity = 0;
  bool failed = false;
  for (int64_t s = k.begin; s < k.end && !failed;) {
    const uint32_t t = static_cast<uint32_t>(s / k.nks);
    int ks = static_cast<int>(s - static_cast<int64_t>(t) * k.nks);
    const Tile x = tile_of<C::kRows>(t, a);
    const bool gated = a.product == PGG_W4_GATED;
    const int32_t c0 = static_cast<int32_t>(x.n0);
    const int32_t c1 = static_cast<int32_t>(x.n0 + (gated ? a.N : 64));
    const bool second = gated || x.n0 + 64 < a.N;
    for (; ks < k.nks && s < k.end; ++ks, ++s) {
      if (!ptx::mbar_wait(&ctl->empty[stage], phase ^ 1u, a.wait_limit_ns, abort)) {
        failed = true;
        break;
      }
      uint8_t* p = smem + stage * C::kStageBytes;
      ptx::mbar_arrive_expect_tx(&ctl->full[stage], second ? kCodeBytes : kCodeBytes / 2);
      ptx::tma_load_3d(p, tm, &ctl->full[stage], ks * (kStep / 4), c0, static_cast<int32_t>(x.g));
      if (second)
        ptx::tma_load_3d(p + kCodeBytes / 2, tm, &ctl->full[stage], ks * (kStep / 4), c1,
                         static_cast<int32_t>(x.g));
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
    raise_status(a.hdr, kStTimeout, 172);
  }
  // the copies in flight land before the CTA ends (the feeders arrive whatever happens)
  int no_abort = 0;
  for (int i = 0; i < C::kStages; ++i)
    if (outstanding & (1u << i))
      ptx::mbar_wait(&ctl->full[i], (last_parity >> i) & 1u, a.wait_limit_ns, &no_abort);
}

// Where the eight values of x at k = 8 v of a stage, row n, stand: in the order in which the
// product's lanes read them, 16 bytes each, mixed so that neither side meets in a bank.
template <int U>
__device__ __forceinline__ int x_place(int n, int v) {
  const int unit = v / (U / 8), rest = v % (U / 8), q = rest / (U / 32), i = rest % (U / 32);
  const int s = unit * (U / 32) + i, p = (n & 7) * 4 + q;
  return ((n >> 3) * 8 + s) * 512 + ((p ^ (s & 3) ^ ((p & 1) << 2)) << 4);
}

// (x0 x1)(x2 x3)(x4 x5)(x6 x7) -> (x0 x4)(x1 x5)(x2 x6)(x3 x7)
__device__ __forceinline__ uint4 pair_up(const uint4& x) {
  return make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632),
                    __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
}

// Feeder warp w fills stage slot w: the rows of x, a row of 512 bytes at a time, and the columns'
// scales (and zeros, as the pair that is subtracted).
template <int DT, int NT, int U, bool ZEROS>
__device__ void feeder(uint8_t* smem, Ctl* ctl, int w, const W4Args& a, const Walk& k) {
  using C = Cfg<NT, U, ZEROS>;
  volatile int* abort = &ctl->abort;
  const int lane = threadIdx.x & 31;
  uint8_t* xs = smem + w * C::kStageBytes + kCodeBytes;
  float* scales = reinterpret_cast<float*>(xs + C::kXBytes);
  uint32_t* zeros = reinterpret_cast<uint32_t*>(xs + C::kXBytes + C::kScaleBytes);
  const int64_t columns = a.product == PGG_W4_GATED ? 2 * a.N : a.N;
  uint32_t phase = 0;
  bool failed = false;
  int64_t tile = -1;
  Tile x = {};
  int64_t xrow = 0;       // lane n: offset of row n of x
  int64_t at[4] = {};     // first scale of columns lane + 32 i, or -1
  for (int64_t s = k.begin + w; s < k.end; s += C::kStages) {
    const int64_t t = s / k.nks;
    const int ks = static_cast<int>(s - t * k.nks);
    if (t != tile) {
      tile = t;
      x = tile_of<C::kRows>(static_cast<uint32_t>(t), a);
      if (lane < x.rows) {
        const int64_t row = check_index(a.hdr, x.row0 + lane, a.M, 173);
        xrow = (a.product == PGG_W4_COMBINED
                    ? row
                    : check_index(a.hdr, a.rowinfo[row].token, a.batch, 174)) *
               a.K;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t c = column_of(a, x, lane + 32 * i);
        at[i] = c < 0 ? -1 : (x.g * columns + c) * a.groups;
      }
    }
    const uint32_t k0 = static_cast<uint32_t>(ks) * kStep;
    const uint32_t K = static_cast<uint32_t>(a.K);
#pragma unroll
    for (int n0 = 0; n0 < C::kRows; n0 += 8) {
      uint4 v[8];  // (the first eight rows are loaded before the wait: they need no room yet)
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const int64_t row = __shfl_sync(0xFFFFFFFFu, xrow, n0 + n);
        v[n] = make_uint4(0, 0, 0, 0);
        if (n0 + n < x.rows && k0 + 8 * lane < K)
          v[n] = __ldg(
              reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + row + k0) + lane);
      }
      if (n0 == 0) {
        if (!failed && !ptx::mbar_wait(&ctl->empty[w], phase ^ 1u, a.wait_limit_ns, abort))
          failed = true;  // (from here on it only arrives, so that copies in flight are waited for)
        failed = __any_sync(0xFFFFFFFFu, failed);
      }
      if (failed) break;
#pragma unroll
      for (int n = 0; n < 8; ++n)
        if (n0 + n < x.rows)  // (what stands in the others reaches no row that is looked at)
          *reinterpret_cast<uint4*>(xs + x_place<U>(n0 + n, lane)) = pair_up(v[n]);
    }
    if (!failed) {
#pragma unroll
      for (int u = 0; u < C::kUnits; ++u) {
        const uint32_t kk = k0 + u * U;
        const uint32_t group = kk < K ? kk / static_cast<uint32_t>(a.group) : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float sc = 0.0f;
          uint32_t z = 8;
          if (at[i] >= 0 && kk < K) {
            if (a.scale_f32)
              sc = __ldg(static_cast<const float*>(a.scales) + at[i] + group);
            else if (DT == PGG_BF16)
              sc = __uint_as_float(static_cast<uint32_t>(__ldg(
                       static_cast<const uint16_t*>(a.scales) + at[i] + group)) << 16);
            else
              sc = __half2float(__ldg(static_cast<const __half*>(a.scales) + at[i] + group));
            if (ZEROS) z = __ldg(a.zeros + at[i] + group);
          }
          scales[u * kTile + lane + 32 * i] = sc;
          if (ZEROS) {
            const uint16_t h = DT == PGG_BF16
                                   ? __bfloat16_as_ushort(__float2bfloat16_rn(128.0f + z))
                                   : __half_as_ushort(__float2half_rn(1024.0f + z));
            zeros[u * kTile + lane + 32 * i] = h * 0x10001u;
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&ctl->full[w]);
    phase ^= 1u;
  }
  if (failed && lane == 0) {
    ctl->abort = 1;
    raise_status(a.hdr, kStTimeout, 175);
  }
}

template <int DT>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (DT == PGG_BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3},"
        " {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3},"
        " {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Codes j and 4 + j of a word, less the zero (`z` is the pair 2^7 + zero, or 2^10 + zero).
template <int DT>
__device__ __forceinline__ uint32_t unpack(uint32_t w, int j, uint32_t z) {
  const uint32_t v = ((w >> (4 * j)) & 0x000F000Fu) | (DT == PGG_BF16 ? 0x43004300u : 0x64006400u);
  uint32_t r;
  if constexpr (DT == PGG_BF16)
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(z));
  else
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(z));
  return r;
}

template <int W>
struct Words {
  uint32_t v[W];
};

template <int W>
__device__ __forceinline__ Words<W> load_words(const uint8_t* p) {
  Words<W> r;
  if constexpr (W == 4) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    r.v[0] = q.x;
    r.v[1] = q.y;
    r.v[2] = q.z;
    r.v[3] = q.w;
  } else if constexpr (W == 2) {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    r.v[0] = q.x;
    r.v[1] = q.y;
  } else {
    r.v[0] = *reinterpret_cast<const uint32_t*>(p);
  }
  return r;
}

// The tile's results from `red` [row][column].
template <int DT, int NT>
__device__ __forceinline__ void write_tile(const float* red, const W4Args& a, const Tile& x,
                                           int thread) {
  constexpr int kThr = 32 * kMmaWarps;
  const bool gated = a.product == PGG_W4_GATED;
  const int half = gated ? 32 : 64;  // pairs of a row
  for (int i = thread; i < x.rows * half; i += kThr) {
    const int j = i / half, c = 2 * (i - j * half);
    const int64_t n = x.n0 + c;
    if (n >= a.N) continue;
    const int64_t row = x.row0 + j;
    const int64_t pos = check_index(a.hdr, a.rowinfo[row].rank, a.M, 176);
    float v0 = red[j * kRedStride + c], v1 = red[j * kRedStride + c + 1];
    if (gated) {
      const float p = a.probs ? a.probs[pos] : 1.0f;
      v0 = gate(v0, red[j * kRedStride + 64 + c], p);
      v1 = gate(v1, red[j * kRedStride + 65 + c], p);
    }
    const int64_t at = (a.product == PGG_W4_COMBINED ? pos : row) * a.N + n;
    if (a.out_f32) {
      float* o = static_cast<float*>(a.out) + at;
      if (a.pairs) {
        *reinterpret_cast<float2*>(o) = make_float2(v0, v1);
      } else {
        o[0] = v0;
        if (n + 1 < a.N) o[1] = v1;
      }
    } else {
      uint16_t* o = static_cast<uint16_t*>(a.out) + at;
      const uint32_t p = pack2<DT>(v0, v1);
      if (a.pairs) {
        *reinterpret_cast<uint32_t*>(o) = p;
      } else {
        o[0] = static_cast<uint16_t>(p);
        if (n + 1 < a.N) o[1] = static_cast<uint16_t>(p >> 16);
      }
    }
  }
}

template <int DT, int NT, int U, bool ZEROS>
__device__ void multiplier(uint8_t* smem, Ctl* ctl, float* red, int w, const W4Args& a,
                           const Walk& k) {
  using C = Cfg<NT, U, ZEROS>;
  constexpr int W = U / 32;            // words of a lane and group
  constexpr int kHalf = C::kUnits / 2;  // groups of this warp and stage
  volatile int* abort = &ctl->abort;
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int col0 = 32 * (w & 3), part = w >> 2;
  // fragment row g is column perm of each eight, so that the lanes of one access to shared memory
  // (two g) lie in different halves of the swizzled 128 bytes
  const int perm = (g >> 1) + 4 * (g & 1);
  const int thread = 32 * w + lane;
  constexpr uint32_t kZero8 = DT == PGG_BF16 ? 0x43084308u : 0x64086408u;
  int stage = 0;
  uint32_t phase = 0;
  bool failed = false;
  for (int64_t s = k.begin; s < k.end;) {
    const uint32_t t = static_cast<uint32_t>(s / k.nks);
    const int ks0 = static_cast<int>(s - static_cast<int64_t>(t) * k.nks);
    const int64_t left = k.end - s;
    const int n_steps = left < k.nks - ks0 ? static_cast<int>(left) : k.nks - ks0;
    const Tile x = tile_of<C::kRows>(t, a);
    float sum[2][NT][4] = {};
    for (int i = 0; i < n_steps; ++i) {
      if (!failed && !__all_sync(0xFFFFFFFFu, ptx::mbar_wait(&ctl->full[stage], phase,
                                                             a.wait_limit_ns, abort))) {
        failed = true;
        if (lane == 0) {
          ctl->abort = 1;
          raise_status(a.hdr, kStTimeout, 177);
        }
      }
      if (failed) break;  // (the eight warps still meet at every barrier below)
      const uint8_t* codes = smem + stage * C::kStageBytes;
      const uint8_t* xs = codes + kCodeBytes;
      const float* scales = reinterpret_cast<const float*>(xs + C::kXBytes);
      const uint32_t* zeros = reinterpret_cast<const uint32_t*>(xs + C::kXBytes + C::kScaleBytes);
#pragma unroll
      for (int h = 0; h < kHalf; ++h) {
        const int u = part * kHalf + h;
        const int byte = u * (U / 2) + q * (U / 8);
        Words<W> word[2][2];
        uint32_t z[2][2];
        float sc[2][2];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int col = col0 + 16 * r + 8 * e + perm;
            word[r][e] = load_words<W>(codes + col * 128 + ((((byte >> 4) ^ perm) << 4) | (byte & 15)));
            sc[r][e] = scales[u * kTile + col];
            z[r][e] = ZEROS ? zeros[u * kTile + col] : kZero8;
          }
        float d[2][NT][4] = {};
#pragma unroll
        for (int i8 = 0; i8 < W; ++i8) {
          const int slot = u * W + i8;
          uint4 b[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n)
            b[n] = *reinterpret_cast<const uint4*>(
                xs + (n * 8 + slot) * 512 + ((lane ^ (slot & 3) ^ ((lane & 1) << 2)) << 4));
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            uint32_t p[2][4];
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int j = 0; j < 4; ++j) p[e][j] = unpack<DT>(word[r][e].v[i8], j, z[r][e]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma<DT>(d[r][n], p[0][0], p[1][0], p[0][1], p[1][1], b[n].x, b[n].y);
              mma<DT>(d[r][n], p[0][2], p[1][2], p[0][3], p[1][3], b[n].z, b[n].w);
            }
          }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            sum[r][n][0] = fmaf(sc[r][0], d[r][n][0], sum[r][n][0]);
            sum[r][n][1] = fmaf(sc[r][0], d[r][n][1], sum[r][n][1]);
            sum[r][n][2] = fmaf(sc[r][1], d[r][n][2], sum[r][n][2]);
            sum[r][n][3] = fmaf(sc[r][1], d[r][n][3], sum[r][n][3]);
          }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&ctl->empty[stage]);
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    // both halves of k into red [row][column]
    for (int turn = 0; turn < 2; ++turn) {
      if (part == turn) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float* p = red + (8 * n + 2 * q + (e & 1)) * kRedStride + col0 + 16 * r +
                         8 * (e >> 1) + perm;
              *p = turn == 0 ? sum[r][n][e] : *p + sum[r][n][e];
            }
      }
      ptx::named_bar_sync(1, 32 * kMmaWarps);
    }
    bool mine = true;
    if (n_steps < k.nks) {
      // a part of the tile: leave it, and add them all if the others are there
      const int64_t s0 = static_cast<int64_t>(t) * k.nks;
      const int64_t first = ((s0 + 1) * k.ctas - 1) / k.total;
      const int64_t last = ((s0 + k.nks) * k.ctas - 1) / k.total;
      constexpr int kPart = C::kRows * kTile;
      float* own = a.parts + (2 * static_cast<int64_t>(blockIdx.x) + (ks0 == 0 ? 1 : 0)) * kPart;
      for (int i = thread; i < x.rows * kTile; i += 32 * kMmaWarps)
        own[i] = red[(i / kTile) * kRedStride + i % kTile];
      __threadfence();
      ptx::named_bar_sync(1, 32 * kMmaWarps);
      if (thread == 0) {
        const uint32_t before = atomicAdd(a.arrived + first, 1u);
        ctl->last = before == static_cast<uint32_t>(last - first) ? 1 : 0;
      }
      ptx::named_bar_sync(1, 32 * kMmaWarps);
      mine = *const_cast<volatile int*>(&ctl->last) != 0;
      if (mine) {
        __threadfence();
        for (int i = thread; i < x.rows * kTile; i += 32 * kMmaWarps) {
          float v = 0.0f;
          for (int64_t c = first; c <= last; ++c)
            v += __ldcg(a.parts + (2 * c + (c == first ? 1 : 0)) * kPart + i);
          red[(i / kTile) * kRedStride + i % kTile] = v;
        }
        ptx::named_bar_sync(1, 32 * kMmaWarps);
      }
    }
    if (mine) write_tile<DT, NT>(red, a, x, thread);
    ptx::named_bar_sync(1, 32 * kMmaWarps);  // red is read before the next tile's sums go there
    s += n_steps;
  }
}

template <int DT, int NT, int U, bool ZEROS>
__global__ void __launch_bounds__(Cfg<NT, U, ZEROS>::kThreads, 1)
    w4_stream_kernel(const __grid_constant__ CUtensorMap tm, const W4Args a) {
  using C = Cfg<NT, U, ZEROS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  float* red = reinterpret_cast<float*>(smem + C::kStages * C::kStageBytes);
  __shared__ Ctl ctl;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(&ctl.full[s], 2);
      ptx::mbar_init(&ctl.empty[s], kMmaWarps);
    }
    ctl.abort = 0;
    ptx::fence_mbar_init();
    ptx::tma_prefetch_desc(&tm);
  }
  __syncthreads();
  ptx::griddep_wait();
  if (routing_failed(a.hdr)) {  // (combined: the sum over the rows gives the zeros)
    const int64_t n = a.product == PGG_W4_COMBINED ? 0 : a.M * a.N;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
      if (a.out_f32)
        static_cast<float*>(a.out)[i] = 0.0f;
      else
        static_cast<uint16_t*>(a.out)[i] = 0;
    }
    return;
  }
  Walk k;
  k.nks = static_cast<int>((a.K + kStep - 1) / kStep);
  k.total = static_cast<int64_t>(a.hdr->n_row_blocks) * a.n_blocks * k.nks;
  // at least two steps a CTA, so that each has some
  k.ctas = k.total < 2 * static_cast<int64_t>(gridDim.x) ? (k.total + 1) / 2 : gridDim.x;
  if (static_cast<int64_t>(blockIdx.x) >= k.ctas) return;
  k.begin = static_cast<int64_t>(blockIdx.x) * k.total / k.ctas;
  k.end = (static_cast<int64_t>(blockIdx.x) + 1) * k.total / k.ctas;
  if (warp == 0) {
    if (lane == 0) code_producer<NT, U, ZEROS>(smem, &ctl, &tm, a, k);
  } else if (warp <= C::kStages) {
    feeder<DT, NT, U, ZEROS>(smem, &ctl, warp - 1, a, k);
  } else {
    multiplier<DT, NT, U, ZEROS>(smem, &ctl, red, warp - 1 - C::kStages, a, k);
  }
}

template <int DT, int NT, int U, bool ZEROS>
cudaError_t launch_t(const CUtensorMap& tm, const W4Args& a, int num_sms, cudaStream_t stream) {
  using C = Cfg<NT, U, ZEROS>;
  static_assert(C::kSmem <= 227 * 1024 && C::kStages >= 3, "shared memory");
  auto kern = w4_stream_kernel<DT, NT, U, ZEROS>;
  static SmemLimit limit;
  const cudaError_t err = allow_smem(&limit, kern, C::kSmem);
  if (err != cudaSuccess) return err;
  return launch_pdl(kern, dim3(static_cast<unsigned>(num_sms < kW4Grid ? num_sms : kW4Grid)),
                    dim3(C::kThreads), static_cast<size_t>(C::kSmem), stream, 1, tm, a);
}

template <int DT, int NT>
cudaError_t launch_u(const CUtensorMap& tm, const W4Args& a, int num_sms, cudaStream_t stream) {
  const bool z = a.zeros != nullptr;
  if (a.group % 128 == 0)
    return z ? launch_t<DT, NT, 128, true>(tm, a, num_sms, stream)
             : launch_t<DT, NT, 128, false>(tm, a, num_sms, stream);
  if (a.group % 64 == 0)
    return z ? launch_t<DT, NT, 64, true>(tm, a, num_sms, stream)
             : launch_t<DT, NT, 64, false>(tm, a, num_sms, stream);
  return z ? launch_t<DT, NT, 32, true>(tm, a, num_sms, stream)
           : launch_t<DT, NT, 32, false>(tm, a, num_sms, stream);
}

template <int DT>
cudaError_t launch_nt(const CUtensorMap& tm, int rows, const W4Args& a, int num_sms,
                      cudaStream_t stream) {
  if (rows == 8) return launch_u<DT, 1>(tm, a, num_sms, stream);
  if (rows == 16) return launch_u<DT, 2>(tm, a, num_sms, stream);
  if (rows == 32) return launch_u<DT, 4>(tm, a, num_sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_w4_stream(int dtype, int rows_per_block, W4Args a, int num_sms,
                             cudaStream_t stream) {
  const int tile = a.product == PGG_W4_GATED ? kTile / 2 : kTile;
  a.n_blocks = static_cast<int32_t>((a.N + tile - 1) / tile);
  CUtensorMap tm;  // codes as words of 16 bits: boxes of 128 bytes x 64 columns
  std::memset(&tm, 0, sizeof(tm));
  if (!encode_map_3d(&tm, PGG_F16, a.codes, a.row_bytes / 2,
                     a.product == PGG_W4_GATED ? 2 * a.N : a.N, a.G, 64))
    return cudaErrorInvalidValue;
  if (dtype == PGG_BF16) return launch_nt<PGG_BF16>(tm, rows_per_block, a, num_sms, stream);
  if (dtype == PGG_F16) return launch_nt<PGG_F16>(tm, rows_per_block, a, num_sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pgg
