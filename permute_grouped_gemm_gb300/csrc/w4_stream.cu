// Products with 4-bit expert weights, few rows an expert: the codes are
// streamed once per block of up to 32 rows, and that stream is the bound.
//
// Tile: 128 columns of one expert (gated: 64 gates and their 64 ups) x NR rows.
// A stage is 256 of k. A warp takes 32 columns x 128 of k of it and multiplies
// with mma.sync m16n8k16 in fp16: the codes, unpacked in registers, are the A
// operand, eight rows of x the B operand. What the loop is made for is few
// instructions a code (64 experts, 512 rows, K 7168, F 2048: 227 us, with codes
// made to halves by an OR and a subtraction of halves 248; the bytes alone, copied
// and not multiplied, take some 180):
//
//   - A code needs no conversion: the four bits alone, (w & 0x000F000F), are two
//     fp16 subnormals of code 2^-24, and (w & 0x00F000F0) two of code 2^-20, so a
//     word of eight codes costs four ANDs and one shift. Products with x and
//     their fp32 sums are exact or rounded as in any fp32 sum.
//   - x is brought to fp16 by a power of two a row, so that its largest value lies
//     in [2^14, 2^15): bf16 keeps its eight bits, and what is lost is below 2^-35
//     of the row's largest value. A launch before this one does that, gathers the
//     rows, and lays them out in the order in which the products read them (a
//     pair is k + j, k + 4 + j, as in the codes' word; those that meet code 2^-20
//     divided by 16), with every group's sum of x.
//   - The zero is taken off a group's sum, zero times the sum of x, and then the
//     scale multiplies it: the weights are never rounded.
//
// The warp-wide product is used because the operand is made in registers: for
// tcgen05 it would go through shared memory once more or through tensor memory
// and two hand-overs a step; with 8 to 32 rows the product is not the bound.
//
// The tiles' steps of k are dealt to the CTAs (two an SM, so that one multiplies
// while the other ends a tile) in equal runs. A tile that is shared leaves fp32
// parts in the workspace, and the CTA that comes last (a counter) adds them in
// the order of k: no CTA waits for another, and the result does not depend on
// who comes last.
//
// Warp 0 copies, eight multiply. Waits are bounded as everywhere.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <cstring>

#include "pgg_block.h"
#include "pgg_ops_launch.h"
#include "pgg_ops_mma.cuh"
#include "pgg_ptx.cuh"
#include "pgg_vec.cuh"
#include "pgg_w4_rows.cuh"

namespace pgg {
namespace {

constexpr int kTile = 128;       // columns of codes
constexpr int kStep = 256;       // of k a stage
constexpr int kPart = 128;       // of k: what a warp takes of a stage
constexpr int kMmaWarps = 8;     // 4 x 32 columns, two parts of k
constexpr int kThreads = 32 * (1 + kMmaWarps);
constexpr int kCodeBytes = kTile * kStep / 2;
constexpr int kRedStride = kTile + 4;
constexpr int kMaxStages = 8;
constexpr int32_t kWritten = INT32_MIN;  // as a row's power of two: its results are there already

// NT: eights of rows. U: of k that share a scale (a divisor of the group).
template <int NT, int U>
struct Cfg {
  static constexpr int kCtas = NT <= 2 ? 2 : 1;  // (32 rows need the registers)
  static constexpr int kRows = 8 * NT;
  static constexpr int kUnits = kPart / U;       // groups of a part
  static constexpr int kStageUnits = kStep / U;
  // x of a stage, then its groups' sums [unit][row]
  static constexpr int kXBytes = kRows * kStep * 2 + kStageUnits * kRows * 4;
  // a column's scales of a stage (room for fp32), then its zeros
  static constexpr int kScaleBytes = kTile * kStageUnits * 4;
  static constexpr int kZeroBytes = kTile * kStageUnits;
  static constexpr int kExtraBytes = (kXBytes + kScaleBytes + kZeroBytes + 127) / 128 * 128;
  static constexpr int kRedBytes = kRows * kRedStride * 4;
  // (a block may have 227 KB, an SM 228 KB with 1 KB of each block's kept back)
  static constexpr int kRoom = kCtas == 2 ? 113 * 1024 : 227 * 1024;
  static constexpr int kFit = (kRoom - kRedBytes - 1024 - 256) / (kCodeBytes + kExtraBytes);
  static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
  // codes of all stages (in pieces of 1 KB), then what else they have, then the tile's sums
  static constexpr int kExtra = kStages * kCodeBytes;
  static constexpr int kRed = kExtra + kStages * kExtraBytes;
  static constexpr int kSmem = kRed + kRedBytes + 1024;
  static_assert(kStages >= 3, "shared memory");
};

struct Ctl {
  uint64_t full[kMaxStages];   // bytes by TMA, and the copying warp's stores
  uint64_t empty[kMaxStages];  // read by all eight warps
  int abort;
  int last;                    // this CTA is the one that adds the tile's parts
};

// The steps [begin, end) of this CTA among `total`, dealt to `ctas` of them; nks steps a tile.
struct Walk {
  int64_t begin, end, total, ctas;
  int nks;
};

struct Tile {
  int64_t g, row0, n0;
  uint32_t rb;
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
  x.rb = rb;
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

// ------------------------------------------------------------------ x

// A row of a row block: its power of two, its values in the products' order, and its groups' sums.
// 128 threads a row, eight of k a thread and turn.
template <int DT, int NT, int U>
__global__ void __launch_bounds__(128) w4_pack_kernel(const W4Args a) {
  using C = Cfg<NT, U>;
  __shared__ float s_max[4];
  ptx::griddep_wait();
  if (routing_failed(a.hdr)) return;
  const int tid = threadIdx.x;
  const int64_t nks = (a.K + kStep - 1) / kStep;
  const int64_t total = static_cast<int64_t>(a.hdr->n_row_blocks) * C::kRows;
  for (int64_t i = blockIdx.x; i < total; i += gridDim.x) {
    const int64_t rb = i / C::kRows;
    const int n = static_cast<int>(i - rb * C::kRows);
    const int4 e = a.rblist[check_index(a.hdr, rb, a.max_row_blocks, 172)];
    if (n >= e.z) continue;  // (what stands there reaches no row that is looked at)
    const int64_t row = check_index(a.hdr, static_cast<int64_t>(e.y) + n, a.M, 173);
    const int64_t xrow = a.product == PGG_W4_COMBINED
                             ? row
                             : check_index(a.hdr, a.rowinfo[row].token, a.batch, 174);
    const uint16_t* x = static_cast<const uint16_t*>(a.x) + xrow * a.K;
    float most = 0.0f, rest = 0.0f;  // rest: 0 times the values, NaN where one is not finite
    for (int64_t k = 8 * tid; k < a.K; k += 8 * 128) {
      float v[8];
      vec::load<DT, 8>(x, k, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        most = fmaxf(most, fabsf(v[j]));
        rest = fmaf(v[j], 0.0f, rest);
      }
    }
    bool infinite;
    most = row_max(most, rest, s_max, &infinite);
    int exponent = 0;  // of two: most = m 2^exponent, m in [0.5, 1)
    if (most > 0.0f) frexpf(most, &exponent);
    exponent -= 15;
    // 2^-exponent in two factors (it may lie outside fp32)
    const float by0 = ldexpf(1.0f, -(exponent / 2)), by1 = ldexpf(1.0f, -(exponent - exponent / 2));
    if (tid == 0) a.exponent[i] = infinite ? kWritten : exponent;
    if (infinite) {
      const int64_t pos = check_index(a.hdr, a.rowinfo[row].rank, a.M, 178);
      write_infinite_row<DT>(a, x, check_index(a.hdr, e.x, a.G, 179), row, pos);
    }
    char* out = static_cast<char*>(a.packed) + rb * nks * C::kXBytes;
    const int64_t end = nks * kStep;
    for (int64_t k = 8 * tid; k < end; k += 8 * 128) {
      float v[8] = {};
      if (k < a.K) vec::load<DT, 8>(x, k, v);
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = __half2float(__float2half_rn(v[j] * by0 * by1));
        sum += v[j];
      }
      // lanes of a group (U / 8 neighbours)
#pragma unroll
      for (int d = 1; d < U / 8; d *= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
      uint4 w;
      w.x = vec::pack2<PGG_F16>(v[0], v[4]);
      w.y = vec::pack2<PGG_F16>(v[1] * 0.0625f, v[5] * 0.0625f);
      w.z = vec::pack2<PGG_F16>(v[2], v[6]);
      w.w = vec::pack2<PGG_F16>(v[3] * 0.0625f, v[7] * 0.0625f);
      const int64_t ks = k / kStep;
      const int in = static_cast<int>(k - ks * kStep) / 8;  // eight of the stage
      const int unit = in / (U / 8), rest = in % (U / 8), q = rest / (U / 32);
      const int slot = unit * (U / 32) + rest % (U / 32);  // of 32 k
      char* stage = out + ks * C::kXBytes;
      *reinterpret_cast<uint4*>(stage + ((n >> 3) * 8 + slot) * 512 + (((n & 7) * 4 + q) << 4)) = w;
      if (rest == 0)
        reinterpret_cast<float*>(stage + C::kRows * kStep * 2)[unit * C::kRows + n] =
            sum * 0x1p-24f;
    }
  }
}

// ------------------------------------------------------------------ the copying warp

// B bytes (4, 8, 16 or 32) from memory into words, and from words to shared memory.
template <int B>
__device__ __forceinline__ void load_bytes(const void* p, uint32_t* w) {
  if constexpr (B == 4) {
    w[0] = __ldg(static_cast<const uint32_t*>(p));
  } else if constexpr (B == 8) {
    const uint2 v = __ldg(static_cast<const uint2*>(p));
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < B / 16; ++i) {
      const uint4 v = __ldg(static_cast<const uint4*>(p) + i);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  }
}
template <int B>
__device__ __forceinline__ void store_bytes(uint8_t* p, const uint32_t* w) {
  if constexpr (B == 4) {
    *reinterpret_cast<uint32_t*>(p) = w[0];
  } else if constexpr (B == 8) {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < B / 16; ++i)
      reinterpret_cast<uint4*>(p)[i] =
          make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
}

// Codes by TMA, x as one piece, the columns' scales and zeros as they stand in memory, through
// registers: a stage's of a column in one load where they are one aligned piece, else one by one.
template <int NT, int U>
__device__ void copier(uint8_t* smem, Ctl* ctl, const CUtensorMap* tm, const W4Args& a,
                       const Walk& k) {
  using C = Cfg<NT, U>;
  constexpr int kS = C::kStageUnits;
  volatile int* abort = &ctl->abort;
  const int lane = threadIdx.x & 31;
  const bool gated = a.product == PGG_W4_GATED;
  const int64_t columns = gated ? 2 * a.N : a.N;
  const int es = a.scale_f32 ? 4 : 2;
  const uint32_t groups = static_cast<uint32_t>(a.groups);
  const int piece = kS * es < 16 ? kS * es : 16;
  // the same of zeros, for a load of one to eight bytes
  const bool whole_z = a.group == U && groups % kS == 0 &&
                       reinterpret_cast<uintptr_t>(a.zeros) % kS == 0;
  const bool whole = a.group == U && groups % kS == 0 &&
                     reinterpret_cast<uintptr_t>(a.scales) % piece == 0;
  int stage = 0;
  uint32_t phase = 0, outstanding = 0, last_parity = 0;
  bool failed = false;
  for (int64_t s = k.begin; s < k.end && !failed;) {
    const uint32_t t = static_cast<uint32_t>(s / k.nks);
    int ks = static_cast<int>(s - static_cast<int64_t>(t) * k.nks);
    const Tile x = tile_of<C::kRows>(t, a);
    const int32_t c0 = static_cast<int32_t>(x.n0);
    const int32_t c1 = static_cast<int32_t>(x.n0 + (gated ? a.N : 64));
    const bool second = gated || x.n0 + 64 < a.N;
    const char* xp = static_cast<const char*>(a.packed) +
                     static_cast<int64_t>(x.rb) * k.nks * C::kXBytes;
    int64_t at[4];  // first scale of columns lane + 32 i (one that is not there: any)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t c = column_of(a, x, lane + 32 * i);
      at[i] = (x.g * columns + (c < 0 ? 0 : c)) * a.groups;
    }
    for (; ks < k.nks && s < k.end; ++ks, ++s) {
      const uint32_t unit = static_cast<uint32_t>(ks) * kS;
      // scales and zeros are loaded before the wait: they need no room yet
      uint32_t raw[4][kS];  // 16 bits: kS / 2 words each
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const char* src = static_cast<const char*>(a.scales) + (at[i] + unit) * es;
        if (whole && unit < groups) {  // (groups end with a stage, so all of its are there)
          if (a.scale_f32)
            load_bytes<4 * kS>(src, raw[i]);
          else
            load_bytes<2 * kS>(src, raw[i]);
        } else {
#pragma unroll
          for (int u = 0; u < kS; ++u) {
            uint32_t group = unit + u;
            if (a.group != U) group = group * U / static_cast<uint32_t>(a.group);
            const bool in = group < groups;  // (x is 0 behind, but 0 inf is not)
            if (a.scale_f32) {
              raw[i][u] = in ? __ldg(static_cast<const uint32_t*>(a.scales) + at[i] + group) : 0;
            } else {
              const uint32_t v =
                  in ? __ldg(static_cast<const uint16_t*>(a.scales) + at[i] + group) : 0;
              raw[i][u / 2] = u & 1 ? raw[i][u / 2] | v << 16 : v;
            }
          }
        }
      }
      uint64_t z[4] = {};
      if (a.zeros && unit * U < static_cast<uint64_t>(a.K)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint8_t* p = a.zeros + at[i] + unit;
          if (whole_z) {
            if constexpr (kS == 2) z[i] = __ldg(reinterpret_cast<const uint16_t*>(p));
            if constexpr (kS == 4) z[i] = __ldg(reinterpret_cast<const uint32_t*>(p));
            if constexpr (kS == 8) z[i] = __ldg(reinterpret_cast<const unsigned long long*>(p));
          } else {
#pragma unroll
            for (int u = 0; u < kS; ++u) {
              uint32_t group = unit + u;
              if (a.group != U) group = group * U / static_cast<uint32_t>(a.group);
              if (group < groups)
                z[i] |= static_cast<uint64_t>(__ldg(a.zeros + at[i] + group)) << (8 * u);
            }
          }
        }
      }
      if (!__all_sync(0xFFFFFFFFu, ptx::mbar_wait(&ctl->empty[stage], phase ^ 1u, a.wait_limit_ns,
                                                  abort))) {
        failed = true;
        break;
      }
      uint8_t* p = smem + stage * kCodeBytes;
      uint8_t* px = smem + C::kExtra + stage * C::kExtraBytes;
      uint64_t* full = &ctl->full[stage];
      if (lane == 0) {
        ptx::mbar_arrive_expect_tx(full, (second ? kCodeBytes : kCodeBytes / 2) + C::kXBytes);
        ptx::tma_load_3d(p, tm, full, ks * (kStep / 4), c0, static_cast<int32_t>(x.g));
        if (second)
          ptx::tma_load_3d(p + kCodeBytes / 2, tm, full, ks * (kStep / 4), c1,
                           static_cast<int32_t>(x.g));
        bulk_load(px, xp + static_cast<int64_t>(ks) * C::kXBytes, C::kXBytes, full);
      }
      outstanding |= 1u << stage;
      last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
      uint8_t* sc = px + C::kXBytes;
      uint8_t* zs = sc + C::kScaleBytes;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (a.scale_f32)
          store_bytes<4 * kS>(sc + (lane + 32 * i) * 4 * kS, raw[i]);
        else
          store_bytes<2 * kS>(sc + (lane + 32 * i) * 2 * kS, raw[i]);
      }
      if (a.zeros) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (kS == 2)
            reinterpret_cast<uint16_t*>(zs)[lane + 32 * i] = static_cast<uint16_t>(z[i]);
          if constexpr (kS == 4)
            reinterpret_cast<uint32_t*>(zs)[lane + 32 * i] = static_cast<uint32_t>(z[i]);
          if constexpr (kS == 8) reinterpret_cast<uint64_t*>(zs)[lane + 32 * i] = z[i];
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(full);
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
  if (failed && lane == 0) {
    ctl->abort = 1;
    raise_status(a.hdr, kStTimeout, 175);
  }
  // the copies in flight land before the CTA ends
  int no_abort = 0;
  for (int i = 0; i < C::kStages; ++i)
    if (outstanding & (1u << i))
      ptx::mbar_wait(&ctl->full[i], (last_parity >> i) & 1u, a.wait_limit_ns, &no_abort);
}

// ------------------------------------------------------------------ the multiplying warps

// d = a b, or d += a b.
template <bool FIRST>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  const float c0 = FIRST ? 0.0f : d[0], c1 = FIRST ? 0.0f : d[1], c2 = FIRST ? 0.0f : d[2],
              c3 = FIRST ? 0.0f : d[3];
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3},"
      " {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

template <int W>
struct Words {
  uint32_t v[W];
};

// W words of shared memory.
template <int W>
__device__ __forceinline__ Words<W> load_words(uint32_t addr) {
  Words<W> r;
  if constexpr (W == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.v[0]), "=r"(r.v[1]), "=r"(r.v[2]), "=r"(r.v[3])
                 : "r"(addr)
                 : "memory");
  else if constexpr (W == 2)
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                 : "=r"(r.v[0]), "=r"(r.v[1])
                 : "r"(addr)
                 : "memory");
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r.v[0]) : "r"(addr) : "memory");
  return r;
}

__device__ __forceinline__ uint32_t load_half(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t load_byte(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Results of the tile from `red` [row][column], which lack the rows' powers of two and 2^24.
template <int NT>
__device__ __forceinline__ void write_tile(const float* red, const W4Args& a, const Tile& x,
                                           int thread) {
  const bool gated = a.product == PGG_W4_GATED;
  const int half = gated ? 32 : 64;  // pairs of a row
  for (int i = thread; i < x.rows * half; i += 32 * kMmaWarps) {
    const int j = i / half, c = 2 * (i - j * half);
    const int64_t n = x.n0 + c;
    if (n >= a.N) continue;
    const int64_t row = x.row0 + j;
    const int64_t pos = check_index(a.hdr, a.rowinfo[row].rank, a.M, 176);
    const int power = a.exponent[static_cast<int64_t>(x.rb) * (8 * NT) + j], e = power + 24;
    if (power == kWritten) continue;
    const float* r = red + j * kRedStride + c;
    float v0 = ldexpf(r[0], e), v1 = ldexpf(r[1], e);
    if (gated) {
      const float p = a.probs ? a.probs[pos] : 1.0f;
      v0 = gate(v0, ldexpf(r[64], e), p);
      v1 = gate(v1, ldexpf(r[65], e), p);
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
      const uint32_t p = a.bf16 ? pack2<PGG_BF16>(v0, v1) : pack2<PGG_F16>(v0, v1);
      if (a.pairs) {
        *reinterpret_cast<uint32_t*>(o) = p;
      } else {
        o[0] = static_cast<uint16_t>(p);
        if (n + 1 < a.N) o[1] = static_cast<uint16_t>(p >> 16);
      }
    }
  }
}

template <int NT, int U>
__device__ void multiplier(uint8_t* smem, Ctl* ctl, float* red, int w, const W4Args& a,
                           const Walk& k) {
  using C = Cfg<NT, U>;
  constexpr int W = U / 32;  // words of a lane and unit
  constexpr int kThr = 32 * kMmaWarps;
  volatile int* abort = &ctl->abort;
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int col0 = 32 * (w & 3), part = w >> 2;
  // fragment row g is column perm of each eight, so that the lanes of one access to shared memory
  // (two g) lie in different halves of the swizzled 128 bytes
  const int perm = (g >> 1) + 4 * (g & 1);
  const int thread = 32 * w + lane;
  const bool f32 = a.scale_f32 != 0, zeros = a.zeros != nullptr, bf16 = a.bf16 != 0;
  const uint32_t my_codes = ptx::smem_addr(smem) + (col0 + perm) * 128;
  const uint32_t my_x = ptx::smem_addr(smem) + C::kExtra + part * 4 * 512 + lane * 16;
  const uint32_t my_sums = ptx::smem_addr(smem) + C::kExtra + C::kRows * kStep * 2 +
                           part * C::kUnits * C::kRows * 4 + q * 8;
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
      if (failed) break;  // (the warps still meet at every barrier below)
      const uint32_t codes = my_codes + stage * kCodeBytes, extra = stage * C::kExtraBytes;
      const uint32_t scales = ptx::smem_addr(smem) + C::kExtra + extra + C::kXBytes;
#pragma unroll
      for (int u = 0; u < C::kUnits; ++u) {
        const int byte = part * 64 + u * (U / 2) + q * (U / 8);
        const int in_row = (((byte >> 4) ^ perm) << 4) | (byte & 15);
        Words<W> word[2][2];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            word[r][e] = load_words<W>(codes + (16 * r + 8 * e) * 128 + in_row);
        // products that add to the same sums are at least four apart: one waits for the other
        constexpr int kSums = NT == 1 ? 2 : 1;
        float d[kSums][2][NT][4];
#pragma unroll
        for (int i8 = 0; i8 < W; ++i8) {
          Words<4> b[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n)
            b[n] = load_words<4>(my_x + extra + (n * 8 + u * W + i8) * 512);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint32_t w0 = word[r][0].v[i8] >> (8 * h), w1 = word[r][1].v[i8] >> (8 * h);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                if (i8 == 0 && h < kSums)
                  mma<true>(d[h % kSums][r][n], w0 & 0x000F000Fu, w1 & 0x000F000Fu,
                            w0 & 0x00F000F0u, w1 & 0x00F000F0u, b[n].v[2 * h], b[n].v[2 * h + 1]);
                else
                  mma<false>(d[h % kSums][r][n], w0 & 0x000F000Fu, w1 & 0x000F000Fu,
                             w0 & 0x00F000F0u, w1 & 0x00F000F0u, b[n].v[2 * h], b[n].v[2 * h + 1]);
              }
            }
        }
        if constexpr (kSums == 2) {
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) d[0][r][0][e] += d[1][r][0][e];
        }
        float sc[2][2], z[2][2];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int e = 0; e < 2; ++e) z[r][e] = -8.0f;
        const int at = (col0 + perm) * C::kStageUnits + part * C::kUnits + u;
        if (f32) {
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              sc[r][e] = __uint_as_float(
                  load_words<1>(scales + (at + (16 * r + 8 * e) * C::kStageUnits) * 4).v[0]);
        } else {
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t v = load_half(scales + (at + (16 * r + 8 * e) * C::kStageUnits) * 2);
              sc[r][e] = bf16 ? __uint_as_float(v << 16)
                              : __half2float(__ushort_as_half(static_cast<uint16_t>(v)));
            }
        }
        if (zeros) {
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e)  // (2^23 + z, without its lowest bits' exponent)
              z[r][e] = 8388608.0f -
                        __uint_as_float(0x4B000000u | load_byte(scales + C::kScaleBytes + at +
                                                                (16 * r + 8 * e) * C::kStageUnits));
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const Words<2> xs = load_words<2>(my_sums + extra + u * C::kRows * 4 + n * 32);
          const float x0 = __uint_as_float(xs.v[0]), x1 = __uint_as_float(xs.v[1]);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            sum[r][n][0] = fmaf(sc[r][0], fmaf(z[r][0], x0, d[0][r][n][0]), sum[r][n][0]);
            sum[r][n][1] = fmaf(sc[r][0], fmaf(z[r][0], x1, d[0][r][n][1]), sum[r][n][1]);
            sum[r][n][2] = fmaf(sc[r][1], fmaf(z[r][1], x0, d[0][r][n][2]), sum[r][n][2]);
            sum[r][n][3] = fmaf(sc[r][1], fmaf(z[r][1], x1, d[0][r][n][3]), sum[r][n][3]);
          }
        }
      }
      // (the stage's next bytes are the asynchronous proxy's: without the fence they have overtaken the
      // last of these loads)
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&ctl->empty[stage]);
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    // both parts of k into red [row][column], one after the other
    if (s > k.begin) ptx::named_bar_sync(1, kThr);  // (the tile before is read)
#pragma unroll
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
      ptx::named_bar_sync(1, kThr);
    }
    bool mine = true;
    if (n_steps < k.nks) {
      // a part of the tile: leave it, and add them all if the others are there
      const int64_t s0 = static_cast<int64_t>(t) * k.nks;
      const int64_t first = ((s0 + 1) * k.ctas - 1) / k.total;
      const int64_t last = ((s0 + k.nks) * k.ctas - 1) / k.total;
      constexpr int kShare = C::kRows * kTile;
      float* own = a.parts + (2 * static_cast<int64_t>(blockIdx.x) + (ks0 == 0 ? 1 : 0)) * kShare;
      for (int i = thread; i < x.rows * kTile; i += kThr)
        own[i] = red[(i / kTile) * kRedStride + i % kTile];
      __threadfence();
      ptx::named_bar_sync(1, kThr);
      if (thread == 0) {
        const uint32_t before = atomicAdd(a.arrived + first, 1u);
        ctl->last = before == static_cast<uint32_t>(last - first) ? 1 : 0;
      }
      ptx::named_bar_sync(1, kThr);
      mine = *const_cast<volatile int*>(&ctl->last) != 0;
      if (mine) {
        __threadfence();
        for (int i = thread; i < x.rows * kTile; i += kThr) {
          float v = 0.0f;
          for (int64_t c = first; c <= last; ++c)
            v += __ldcg(a.parts + (2 * c + (c == first ? 1 : 0)) * kShare + i);
          red[(i / kTile) * kRedStride + i % kTile] = v;
        }
        ptx::named_bar_sync(1, kThr);
      }
    }
    if (mine) write_tile<NT>(red, a, x, thread);
    s += n_steps;
  }
}

template <int NT, int U>
__global__ void __launch_bounds__(kThreads, Cfg<NT, U>::kCtas)
    w4_stream_kernel(const __grid_constant__ CUtensorMap tm, const W4Args a) {
  using C = Cfg<NT, U>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  float* red = reinterpret_cast<float*>(smem + C::kRed);
  __shared__ Ctl ctl;
  const int warp = threadIdx.x >> 5;
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
  if (warp == 0)
    copier<NT, U>(smem, &ctl, &tm, a, k);
  else
    multiplier<NT, U>(smem, &ctl, red, warp - 1, a, k);
}

template <int NT, int U>
cudaError_t launch_t(int dtype, const CUtensorMap& tm, const W4Args& a, int num_sms,
                     cudaStream_t stream) {
  using C = Cfg<NT, U>;
  auto kern = w4_stream_kernel<NT, U>;
  static SmemLimit limit;
  cudaError_t err = allow_smem(&limit, kern, C::kSmem);
  if (err != cudaSuccess) return err;
  int64_t blocks = a.max_row_blocks * C::kRows;
  if (blocks > num_sms * 16) blocks = num_sms * 16;
  err = launch_pdl(dtype == PGG_BF16 ? w4_pack_kernel<PGG_BF16, NT, U>
                                     : w4_pack_kernel<PGG_F16, NT, U>,
                   dim3(static_cast<unsigned>(blocks)), dim3(128), 0, stream, 1, a);
  if (err != cudaSuccess) return err;
  const int grid = num_sms * C::kCtas < kW4Grid ? num_sms * C::kCtas : kW4Grid;
  return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads),
                    static_cast<size_t>(C::kSmem), stream, 1, tm, a);
}

template <int NT>
cudaError_t launch_u(int dtype, const CUtensorMap& tm, const W4Args& a, int num_sms,
                     cudaStream_t stream) {
  if (a.group % 128 == 0) return launch_t<NT, 128>(dtype, tm, a, num_sms, stream);
  if (a.group % 64 == 0) return launch_t<NT, 64>(dtype, tm, a, num_sms, stream);
  return launch_t<NT, 32>(dtype, tm, a, num_sms, stream);
}

}  // namespace

// (groups' sums for groups of 32: the most there are)
int64_t w4_packed_bytes(int64_t row_blocks, int rows_per_block, int64_t K) {
  return row_blocks * rows_per_block * ((K + kStep - 1) / kStep) * (kStep * 2 + kStep / 32 * 4);
}

cudaError_t launch_w4_stream(int dtype, int rows_per_block, W4Args a, int num_sms,
                             cudaStream_t stream) {
  const int tile = a.product == PGG_W4_GATED ? kTile / 2 : kTile;
  a.n_blocks = static_cast<int32_t>((a.N + tile - 1) / tile);
  a.bf16 = dtype == PGG_BF16;
  CUtensorMap tm;  // codes as words of 16 bits: boxes of 128 bytes x 64 columns
  std::memset(&tm, 0, sizeof(tm));
  if (!encode_map_3d(&tm, PGG_F16, a.codes, a.row_bytes / 2,
                     a.product == PGG_W4_GATED ? 2 * a.N : a.N, a.G, 64))
    return cudaErrorInvalidValue;
  if (rows_per_block == 8) return launch_u<1>(dtype, tm, a, num_sms, stream);
  if (rows_per_block == 16) return launch_u<2>(dtype, tm, a, num_sms, stream);
  if (rows_per_block == 32) return launch_u<4>(dtype, tm, a, num_sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pgg
