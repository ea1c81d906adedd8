// Products with 4-bit expert weights, many rows an expert: the tensor cores are
// the bound (tcgen05, 128 columns x up to 160 rows a tile).
//
//     y[column, row] = sum over k of scale (code - zero) x
//
// The columns are the MMA's M operand, so a column is a lane of tensor memory: a
// thread unpacks its own column's codes, multiplies its group's scale in and
// writes them to tensor memory, from where the MMA takes them (tcgen05.st, A
// operand in tensor memory): through shared memory they would cost it as much as
// x does. The other operand is x, brought to fp16 by a power of two a row (its
// largest value in [2^14, 2^15): bf16 keeps its eight bits, what is lost is below
// 2^-39 of the row's largest) and laid out as the MMA reads it (panels of 64 k,
// 128-byte swizzle, pairs k + j, k + 4 + j as in a word of codes) by a launch
// before this one, so that it arrives in plain pieces.
//
// Brought to fp16 by a power of two a column (found by the launch before), a bf16
// scale has eight bits and code - 8 at most three, so the product is an fp16 number
// and the weight is not rounded. With zeros or other scales it is the sum of two (hi
// and what is left, 22 bits), and the MMAs run twice. Either way bits are lost that lie
// below 2^-35 of the column's largest scale. Scaling each group's fp32 sums
// instead costs more: tensor memory is read at about 20 bytes a cycle and
// quarter, so bringing back 128 x 144 sums took 880 cycles, the products of a
// group of 128 are 580 (2048 tokens, 60 experts, K 7168, F 2048: 1432 us, now 825
// to 875; with zeros 1605).
//
// An accumulator cuts off at every step what falls out of its 24 bits, which adds up
// over a long k (K 7168: 7.3e-6 of the results' size, with two-part weights 1.7e-5; fp32
// products, rounded, 1.0e-6 and 1.5e-6). The rounding of 16-bit results hides it. For fp32
// results an accumulator adds up eight groups (two-part weights: three), and the writing
// warps add these sums: 0.9e-6 (2048 tokens' down projection, K 2048, N 7168: 685 us, 655 with
// one sum; four groups 740).
//
// Tensor memory: two accumulators and three A buffers (128 of k: 64 columns; split
// two of 128). Roles: one warp copies, one issues the MMAs; eight unpack (four lane
// quarters x even and odd groups, so that the latencies of a group's waits and
// stores hide behind the other's); eight write the results (four quarters x two
// halves of the rows, up to 80 sums a thread, for which the warpgroups' registers
// are split unevenly) while the next tile's products run. Waits are bounded as
// everywhere.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
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

constexpr int kTile = 128;            // columns of codes
constexpr int kGroup = 128;           // of k: one A buffer, one stage of x
constexpr int kSlotBytes = kTile * 128;           // codes of 256 of k
constexpr int kStageBytes = kW4WideRows * kGroup * 2;  // x of 128 of k
constexpr int kSlots = 4, kStages = 4;

// Most rows of a tile, first tensor-memory column of the A buffers, columns of one.
template <bool SPLIT>
struct Cfg {
  static constexpr int kRows = SPLIT ? kW4SplitRows : kW4WideRows;
  static constexpr int kChunks = kRows / 32;  // of 16 rows, that a writing warp takes
  static constexpr int kACols = 2 * kRows;
  static constexpr int kABuf = SPLIT ? 128 : 64;
  static constexpr int kBufs = SPLIT ? 2 : 3;
  static constexpr int kChain = SPLIT ? 3 : 8;  // groups that an accumulator adds up for fp32 results
  static_assert(kACols + kBufs * kABuf <= 512 && kBufs < kStages, "tensor memory");
};
// Warpgroups: copies and MMAs; two that unpack; two that write. Registers a thread of each, which
// draw on what the block is launched with.
constexpr int kThreads = 5 * 128;
constexpr int kLaunchRegs = 96, kFewRegs = 32, kUnpackRegs = 72, kWriteRegs = 152;
static_assert(128 * kFewRegs + 256 * kUnpackRegs + 256 * kWriteRegs <= kThreads * kLaunchRegs,
              "registers");

struct Ctl {
  uint64_t cfull[kSlots], cempty[kSlots];  // codes
  // of a group: its x has arrived and its codes are in tensor memory; its MMAs are done (one barrier
  // each: what a wait and a commit cost the thread that issues, 100 cycles, is what bounds it)
  uint64_t full[kStages], done[kStages];
  uint64_t dfull[2], dempty[2];  // accumulators
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

constexpr int kSmem = kSlots * kSlotBytes + kStages * kStageBytes +
                      static_cast<int>(sizeof(Ctl)) + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory");

struct Tile {
  int64_t g, row0, n0, prow;  // prow: its first row in the packed x
  int rows, rows16;
};

__device__ __forceinline__ int64_t packed_row(const int4& e, int64_t rb) {
  return static_cast<int64_t>(e.y) + 16 * rb;  // (every block has room up to a multiple of 16)
}

__device__ __forceinline__ Tile tile_of(uint32_t t, const W4Args& a) {
  const uint32_t rb = t / static_cast<uint32_t>(a.n_blocks);
  int4 e = a.rblist[check_index(a.hdr, rb, a.max_row_blocks, 180)];
  if (!check_ok(a.hdr,
                e.x >= 0 && e.x < a.G && e.y >= 0 && e.z > 0 && e.z <= kW4WideRows &&
                    static_cast<int64_t>(e.y) + e.z <= a.M,
                181))
    e = make_int4(0, 0, 1, 0);
  Tile x;
  x.n0 = static_cast<int64_t>(t - rb * static_cast<uint32_t>(a.n_blocks)) *
         (a.product == PGG_W4_GATED ? kTile / 2 : kTile);
  x.g = e.x;
  x.row0 = e.y;
  x.prow = packed_row(e, rb);
  x.rows = e.z;
  x.rows16 = (e.z + 15) / 16 * 16;
  return x;
}

// ------------------------------------------------------------------ x

__device__ __forceinline__ float scale_at(const W4Args& a, int64_t i) {
  if (a.scale_f32) return __ldg(static_cast<const float*>(a.scales) + i);
  const uint16_t v = __ldg(static_cast<const uint16_t*>(a.scales) + i);
  return a.bf16 ? __uint_as_float(static_cast<uint32_t>(v) << 16) : __half2float(__ushort_as_half(v));
}

// A number's size, 0 where it is not finite; the largest of a word of scales.
__device__ __forceinline__ float finite(float v) { return fabsf(v) < INFINITY ? fabsf(v) : 0.0f; }
template <int DT>
__device__ __forceinline__ float largest(const W4Args& a, uint32_t w) {
  if (a.scale_f32) return finite(__uint_as_float(w));
  float lo, hi;
  vec::unpack2<DT>(w, lo, hi);
  return fmaxf(finite(lo), finite(hi));
}

// The power of two of a number that is to become m 2^e with m in [0.5, 1).
__device__ __forceinline__ int exponent_of(float most) {
  int e = 0;
  if (most > 0.0f) frexpf(most, &e);
  return e;
}

// The first `row_blocks` blocks: a row of a row block, its power of two and its values as the MMA
// reads them, 128 threads a row. The others: the columns' powers of two, eight lanes a column of an
// expert with rows: its largest scale comes to lie in [2^10, 2^11), and lower by the bits that a zero
// above 16 has over four, so that scale (code - zero) stays at 2^15 or below, in fp16's range, whose
// smallest step is then 2^-34 of that scale or less (with zeros near 255 2^-30).
template <int DT>
__global__ void __launch_bounds__(128)
    w4_pack_wide_kernel(const W4Args a, const int64_t* group_list, const int row_blocks) {
  __shared__ float s_max[4];
  ptx::griddep_wait();
  if (routing_failed(a.hdr)) return;
  const int tid = threadIdx.x;
  if (static_cast<int>(blockIdx.x) >= row_blocks) {
    const int64_t columns = a.product == PGG_W4_GATED ? 2 * a.N : a.N;
    const int64_t step = static_cast<int64_t>(gridDim.x - row_blocks) * 16;
    const int lane = tid & 7, es = a.scale_f32 ? 4 : 2;
    // a column's scales are whole words of 16 bytes
    const bool words =
        a.groups * es % 16 == 0 && reinterpret_cast<uintptr_t>(a.scales) % 16 == 0;
    const bool zero_words = a.groups % 4 == 0 && reinterpret_cast<uintptr_t>(a.zeros) % 4 == 0;
    // (whole warps walk together: the exchange below needs them)
    const int64_t end = (a.G * columns + 3) / 4 * 4;
    for (int64_t c = (static_cast<int64_t>(blockIdx.x) - row_blocks) * 16 + (tid >> 3); c < end;
         c += step) {
      float most = 0.0f;
      const bool live = c < a.G * columns && group_list[c / columns] > 0;
      if (live && words) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(a.scales) +
                                                        c * a.groups * es);
        for (int i = lane; i < a.groups * es / 16; i += 8) {
          const uint4 q = __ldg(p + i);
          most = fmaxf(fmaxf(most, largest<DT>(a, q.x)), largest<DT>(a, q.y));
          most = fmaxf(fmaxf(most, largest<DT>(a, q.z)), largest<DT>(a, q.w));
        }
      } else if (live) {
        for (int64_t i = lane; i < a.groups; i += 8)
          most = fmaxf(most, finite(scale_at(a, c * a.groups + i)));
      }
      uint32_t zero = 16;  // the column's largest, at least this
      if (live && a.zeros) {
        const uint8_t* z = a.zeros + c * a.groups;
        if (zero_words) {
          for (int i = lane; i < a.groups / 4; i += 8) {
            const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(z) + i);
            zero = max(max(max(zero, w & 255u), w >> 8 & 255u), max(w >> 16 & 255u, w >> 24));
          }
        } else {
          for (int64_t i = lane; i < a.groups; i += 8)
            zero = max(zero, static_cast<uint32_t>(__ldg(z + i)));
        }
      }
#pragma unroll
      for (int d = 1; d < 8; d *= 2) {
        most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, d));
        zero = max(zero, __shfl_xor_sync(0xFFFFFFFFu, zero, d));
      }
      if (live && lane == 0)
        a.col_exponent[c] = exponent_of(most) - 11 + (32 - __clz(static_cast<int>(zero - 1)) - 4);
    }
    return;
  }
  const int64_t width = (a.K + kGroup - 1) / kGroup * kGroup;
  const int64_t total = static_cast<int64_t>(a.hdr->n_row_blocks) * a.block_rows;
  for (int64_t i = blockIdx.x; i < total; i += row_blocks) {
    const int64_t rb = i / a.block_rows;
    const int n = static_cast<int>(i - rb * a.block_rows);
    const int4 e = a.rblist[check_index(a.hdr, rb, a.max_row_blocks, 182)];
    if (n >= e.z) continue;  // (what stands there reaches no row that is looked at)
    const int64_t row = check_index(a.hdr, static_cast<int64_t>(e.y) + n, a.M, 183);
    const int64_t xrow = a.product == PGG_W4_COMBINED
                             ? row
                             : check_index(a.hdr, a.rowinfo[row].token, a.batch, 184);
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
    const int exponent = exponent_of(most) - 15;
    const float by0 = ldexpf(1.0f, -(exponent / 2)), by1 = ldexpf(1.0f, -(exponent - exponent / 2));
    const int64_t prow = packed_row(e, rb);
    if (tid == 0) {  // what the results need to know of the row (-1: they are there already)
      const int64_t pos = check_index(a.hdr, a.rowinfo[row].rank, a.M, 189);
      const float p = a.probs ? a.probs[pos] : 1.0f;
      const int to = static_cast<int>(a.product == PGG_W4_COMBINED ? pos : row);
      a.meta[prow + n] = make_int4(infinite ? -1 : to, exponent, __float_as_int(p), 0);
    }
    if (infinite) {
      const int64_t pos = check_index(a.hdr, a.rowinfo[row].rank, a.M, 190);
      write_infinite_row<DT>(a, x, check_index(a.hdr, e.x, a.G, 191), row, pos);
    }
    char* out = static_cast<char*>(a.packed) + prow * width * 2;
    const int64_t panel = static_cast<int64_t>((e.z + 15) / 16 * 16) * 128;
    for (int64_t k = 8 * tid; k < width; k += 8 * 128) {
      float v[8] = {};
      if (k < a.K) vec::load<DT, 8>(x, k, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = v[j] * by0 * by1;
      uint4 w;
      w.x = vec::pack2<PGG_F16>(v[0], v[4]);
      w.y = vec::pack2<PGG_F16>(v[1], v[5]);
      w.z = vec::pack2<PGG_F16>(v[2], v[6]);
      w.w = vec::pack2<PGG_F16>(v[3], v[7]);
      const int chunk = static_cast<int>(k / 8) & 7;
      *reinterpret_cast<uint4*>(out + k / 64 * panel + n * 128 + ((chunk ^ (n & 7)) << 4)) = w;
    }
  }
}

// ------------------------------------------------------------------ copies

struct Walk {
  uint32_t first, step, total;
  int groups;  // of 128 of k
  int chain;   // of them, that an accumulator adds up
};

// One thread.
__device__ void copier(uint8_t* smem, Ctl* ctl, const CUtensorMap* tm, const W4Args& a,
                       const Walk& k) {
  volatile int* abort = &ctl->abort;
  const bool gated = a.product == PGG_W4_GATED;
  const int64_t width = static_cast<int64_t>(k.groups) * kGroup;
  uint8_t* xs = smem + kSlots * kSlotBytes;
  int slot = 0, stage = 0;
  uint32_t cphase = 0, xphase = 0;
  uint32_t c_out = 0, x_out = 0, c_parity = 0, x_parity = 0;
  bool failed = false;
  for (uint32_t t = k.first; t < k.total && !failed; t += k.step) {
    const Tile x = tile_of(t, a);
    const int32_t c0 = static_cast<int32_t>(x.n0);
    const int32_t c1 = static_cast<int32_t>(x.n0 + (gated ? a.N : 64));
    const bool second = gated || x.n0 + 64 < a.N;
    const uint32_t bytes = static_cast<uint32_t>(x.rows16) * kGroup * 2;
    const char* src = static_cast<const char*>(a.packed) + x.prow * width * 2;
    for (int g = 0; g < k.groups; ++g) {
      if ((g & 1) == 0) {
        if (!ptx::mbar_wait(&ctl->cempty[slot], cphase ^ 1u, a.wait_limit_ns, abort)) {
          failed = true;
          break;
        }
        uint8_t* p = smem + slot * kSlotBytes;
        ptx::mbar_arrive_expect_tx(&ctl->cfull[slot], second ? kSlotBytes : kSlotBytes / 2);
        ptx::tma_load_3d(p, tm, &ctl->cfull[slot], g * 32, c0, static_cast<int32_t>(x.g));
        if (second)
          ptx::tma_load_3d(p + kSlotBytes / 2, tm, &ctl->cfull[slot], g * 32, c1,
                           static_cast<int32_t>(x.g));
        c_out |= 1u << slot;
        c_parity = (c_parity & ~(1u << slot)) | (cphase << slot);
        if (++slot == kSlots) {
          slot = 0;
          cphase ^= 1u;
        }
      }
      if (!ptx::mbar_wait(&ctl->done[stage], xphase ^ 1u, a.wait_limit_ns, abort)) {
        failed = true;
        break;
      }
      ptx::mbar_arrive_expect_tx(&ctl->full[stage], bytes);
      bulk_load(xs + stage * kStageBytes, src + static_cast<int64_t>(g) * bytes, bytes,
                &ctl->full[stage]);
      x_out |= 1u << stage;
      x_parity = (x_parity & ~(1u << stage)) | (xphase << stage);
      if (++stage == kStages) {
        stage = 0;
        xphase ^= 1u;
      }
    }
  }
  if (failed) {
    ctl->abort = 1;
    raise_status(a.hdr, kStTimeout, 185);
  }
  int no_abort = 0;  // the copies in flight land before the CTA ends
  for (int i = 0; i < kSlots; ++i)
    if (c_out & (1u << i))
      ptx::mbar_wait(&ctl->cfull[i], (c_parity >> i) & 1u, a.wait_limit_ns, &no_abort);
  for (int i = 0; i < kStages; ++i) {
    if (!(x_out & (1u << i))) continue;
    // (unpacking warps that gave up have not arrived: their arrivals are made up for)
    for (int n = 0; ctl->abort && n < 4; ++n)
      if (!ptx::mbar_try_wait(&ctl->full[i], (x_parity >> i) & 1u)) ptx::mbar_arrive(&ctl->full[i]);
    ptx::mbar_wait(&ctl->full[i], (x_parity >> i) & 1u, a.wait_limit_ns, &no_abort);
  }
}

// ------------------------------------------------------------------ MMAs

// One lane of a converged warp.
__device__ __forceinline__ bool elected() {
  uint32_t r;
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "elect.sync _|p, 0xFFFFFFFF;\n"
      "selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(r));
  return r != 0;
}

// D[tmem] (+)= A[tmem] * B[smem]^T, fp16, fp32 accumulator.
__device__ __forceinline__ void mma_tmem(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
      "}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// One warp, of which one lane issues: the others keep it converged, so that what the MMAs take (all of
// it the same in every lane) stays in uniform registers.
template <bool SPLIT>
__device__ void issuer(uint8_t* smem, Ctl* ctl, uint32_t tmem, const W4Args& a, const Walk& k) {
  using C = Cfg<SPLIT>;
  volatile int* abort = &ctl->abort;
  uint8_t* xs = smem + kSlots * kSlotBytes;
  int stage = 0, buf = 0, acc = 0;
  uint32_t phase = 0, dphase = 0;
  bool issued = false, failed = false;
  for (uint32_t t = k.first; t < k.total && !failed; t += k.step) {
    const Tile x = tile_of(t, a);
    const uint32_t panel = static_cast<uint32_t>(x.rows16) * 128;
    const uint32_t idesc = ptx::idesc_make(0, kTile, x.rows16);
    for (int g0 = 0; g0 < k.groups && !failed; g0 += k.chain) {
      const uint32_t d = tmem + C::kRows * acc;
      if (!__all_sync(0xFFFFFFFFu, ptx::mbar_wait(&ctl->dempty[acc], dphase ^ 1u, a.wait_limit_ns,
                                                  abort))) {
        failed = true;
        break;
      }
      const int end = g0 + k.chain < k.groups ? g0 + k.chain : k.groups;
      for (int g = g0; g < end; ++g) {
        if (!__all_sync(0xFFFFFFFFu, ptx::mbar_wait(&ctl->full[stage], phase, a.wait_limit_ns,
                                                    abort))) {
          failed = true;
          break;
        }
        ptx::tc_fence_after_sync();
        const uint32_t xb = ptx::smem_addr(xs + stage * kStageBytes);
        const uint32_t ab = tmem + C::kACols + C::kABuf * buf;
        const uint64_t desc0 = ptx::sdesc_sw128(xb), desc1 = ptx::sdesc_sw128(xb + panel);
        if (elected()) {
#pragma unroll
          for (int s = 0; s < kGroup / 16; ++s) {  // of 16 k: 32 bytes of a panel's rows
            const uint64_t desc = (s < 4 ? desc0 : desc1) + 2 * (s & 3);
            mma_tmem(d, ab + 8 * s, desc, idesc, ((g - g0) | s) > 0 ? 1u : 0u);
            if (SPLIT) mma_tmem(d, ab + 64 + 8 * s, desc, idesc, 1u);
          }
          ptx::mma_commit(&ctl->done[stage]);
        }
        __syncwarp();
        issued = true;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
        buf = buf + 1 == C::kBufs ? 0 : buf + 1;
      }
      if (failed) break;
      if (elected()) ptx::mma_commit(&ctl->dfull[acc]);
      __syncwarp();
      acc ^= 1;
      if (acc == 0) dphase ^= 1u;
    }
  }
  if (failed) {
    ctl->abort = 1;
    raise_status(a.hdr, kStTimeout, 186);
  }
  if (issued) {
    int no_abort = 0;
    if (elected()) ptx::mma_commit(&ctl->drain);
    __syncwarp();
    ptx::mbar_wait(&ctl->drain, 0u, a.wait_limit_ns, &no_abort);
  }
}

// ------------------------------------------------------------------ workers

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0],"
      " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// Pairs of fp16.
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t twice(float v) {
  return __half_as_ushort(__float2half_rn(v)) * 0x10001u;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Lane l of the tile: its row of codes in shared memory. Gated: gates in the even lanes, their ups in
// the odd ones, so that neighbours hold what belongs together.
__device__ __forceinline__ int code_row(bool gated, int l) {
  return gated ? (l >> 1) + 64 * (l & 1) : l;
}

// The column of codes of lane l, or -1.
__device__ __forceinline__ int64_t column_of(const W4Args& a, const Tile& x, int l) {
  if (a.product == PGG_W4_GATED) {
    const int64_t f = x.n0 + (l >> 1);
    return f < a.N ? f + ((l & 1) ? a.N : 0) : -1;
  }
  return x.n0 + l < a.N ? x.n0 + l : -1;
}

// v 2^e, e in (-400, 250): in two factors, since 2^e may lie outside fp32.
__device__ __forceinline__ float times_power(float v, int e) {
  const int half = e >> 1, rest = e - half;
  return v * __int_as_float((max(half, -126) + 127) << 23) *
         __int_as_float((max(rest, -126) + 127) << 23);
}

// A lane's column among all experts' (one that is not there: any).
__device__ __forceinline__ int64_t column_index(const W4Args& a, const Tile& x, int l) {
  const int64_t c = column_of(a, x, l);
  return x.g * (a.product == PGG_W4_GATED ? 2 * a.N : a.N) + (c < 0 ? 0 : c);
}

// What a thread needs from memory for a group, loaded ahead: its column's scales and zeros.
template <int U>
struct Ahead {
  static constexpr int kN = kGroup / U;
  uint32_t s[kN];  // as they stand in memory: what converts them would wait for them
  uint32_t z[kN];

  __device__ __forceinline__ void load(const W4Args& a, int64_t at, int g) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      uint32_t group = g * kN + i;
      if (a.group != U) group = group * U / static_cast<uint32_t>(a.group);
      const bool in = group < static_cast<uint32_t>(a.groups);  // (x is 0 behind, but 0 inf is not)
      s[i] = 0;
      z[i] = 8;
      if (!in) continue;
      s[i] = a.scale_f32 ? __ldg(static_cast<const uint32_t*>(a.scales) + at + group)
                         : __ldg(static_cast<const uint16_t*>(a.scales) + at + group);
      if (a.zeros) z[i] = __ldg(a.zeros + at + group);
    }
  }
  __device__ __forceinline__ float scale(const W4Args& a, int i) const {
    if (a.scale_f32) return __uint_as_float(s[i]);
    return a.bf16 ? __uint_as_float(s[i] << 16)
                  : __half2float(__ushort_as_half(static_cast<uint16_t>(s[i])));
  }
};

// Groups `par`, par + 2, ... of this CTA's sequence of groups: the thread's column, 128 of k, into an
// A buffer. U: of k that share a scale.
template <int U, bool SPLIT>
__device__ void unpacker(uint8_t* smem, Ctl* ctl, uint32_t tmem, int par, const W4Args& a,
                         const Walk& k) {
  using C = Cfg<SPLIT>;
  volatile int* abort = &ctl->abort;
  const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, l = 32 * quarter + lane;
  const int row = code_row(a.product == PGG_W4_GATED, l);
  const uint32_t codes = ptx::smem_addr(smem) + row * 128;
  const uint32_t a_lanes = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + C::kACols;
  // A code becomes a half as the low bits of 2^10, or 16 times as high, which are ones there (a published
  // way: Kim et al., "Who Says Elephants Can't Run: Bringing Large Scale MoE Models into Cloud Scale
  // Production", 2022).
  uint32_t magic;  // the pair 2^10, from a register: an instruction holds one of two constants only
  asm volatile("mov.u32 %0, 0x64006400;" : "=r"(magic));
  int slot = 0;  // of codes: two groups of a tile
  uint32_t cphase = 0;
  uint32_t turn = 0;  // of all groups
  // a tile ahead: the column, and its power of two
  int64_t next = k.first < k.total ? column_index(a, tile_of(k.first, a), l) : 0;
  int next_exponent = k.first < k.total ? a.col_exponent[next] : 0;
  Ahead<U> now;
  bool loaded = false;
  for (uint32_t t = k.first; t < k.total; t += k.step) {
    const int64_t at = next * a.groups;
    const int exponent = next_exponent;
    if (!loaded) now.load(a, at, static_cast<int>((turn ^ par) & 1u));
    loaded = false;
    const bool more = t + k.step < k.total;
    if (more) {
      next = column_index(a, tile_of(t + k.step, a), l);
      next_exponent = a.col_exponent[next];
    }
    for (int g = 0; g < k.groups; ++g, ++turn) {
      const bool slot_done = (g & 1) || g + 1 == k.groups;
      const bool mine = (turn & 1) == static_cast<uint32_t>(par);
      if (!mine && !(slot_done && (g & 1) == 0)) {
        if (slot_done && ++slot == kSlots) {
          slot = 0;
          cphase ^= 1u;
        }
        continue;
      }
      bool ok = ptx::mbar_wait(&ctl->cfull[slot], cphase, a.wait_limit_ns, abort);
      if (mine && turn >= C::kBufs) {  // the buffer's last group
        const uint32_t last = turn - C::kBufs;
        ok = ok && ptx::mbar_wait(&ctl->done[last % kStages], (last / kStages) & 1u,
                                  a.wait_limit_ns, abort);
      }
      if (!__all_sync(0xFFFFFFFFu, ok)) {
        if (lane == 0) {
          ctl->abort = 1;
          raise_status(a.hdr, kStTimeout, 187);
        }
        return;
      }
      if (mine) {
        ptx::tc_fence_after_sync();
        const uint32_t a_tmem = a_lanes + C::kABuf * (turn % C::kBufs);
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // 32 of k: four words, 16 columns of tensor memory
          const int chunk = (g & 1) * 4 + i;
          const uint4 q = lds128(codes + slot * kSlotBytes + ((chunk ^ (row & 7)) << 4));
          const uint32_t w[4] = {q.x, q.y, q.z, q.w};
          const float zero = static_cast<float>(now.z[32 * i / U]);
          const uint32_t z0 = twice(1024.0f + zero), z1 = twice(-64.0f - zero);
          const float sf = times_power(now.scale(a, 32 * i / U), -exponent);
          const uint32_t s_hi = twice(sf);
          const uint32_t s_lo =
              SPLIT ? twice(sf - __half2float(__ushort_as_half(static_cast<uint16_t>(s_hi)))) : 0;
          uint32_t v[16], left[SPLIT ? 16 : 1];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t b = w[j] >> (8 * h);
              uint32_t t0, t1;  // 2^10 + code, 2^10 + 16 code
              asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(t0) : "r"(b), "r"(magic));
              asm("lop3.b32 %0, %1, 0x00F000F0, %2, 0xEA;" : "=r"(t1) : "r"(b), "r"(magic));
              t0 = sub2(t0, z0);
              t1 = fma2(t1, 0x2C002C00u, z1);  // times 2^-4, less 64 + zero: exact
              const int to = 4 * j + 2 * h;
              v[to] = mul2(t0, s_hi);
              v[to + 1] = mul2(t1, s_hi);
              if constexpr (SPLIT) {
                left[to] = fma2(t0, s_lo, fma2(t0, s_hi, v[to] ^ 0x80008000u));
                left[to + 1] = fma2(t1, s_lo, fma2(t1, s_hi, v[to + 1] ^ 0x80008000u));
              }
            }
          }
          tmem_st_x16(a_tmem + 16 * i, v);
          if constexpr (SPLIT) tmem_st_x16(a_tmem + 64 + 16 * i, left);
        }
        if (g + 2 < k.groups) {
          now.load(a, at, g + 2);
        } else if (more && k.groups > 1) {
          now.load(a, next * a.groups, g + 2 - k.groups);
          loaded = true;
        }
        ptx::tmem_st_wait();  // (so the codes have been read: TMA may write their slot)
        ptx::tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(&ctl->full[turn % kStages]);
          ptx::mbar_arrive(&ctl->cempty[slot]);
        }
      } else if (lane == 0) {
        // a slot with one group: these warps have nothing to read of it (but it has to be this use
        // of the slot that they let go)
        ptx::mbar_arrive(&ctl->cempty[slot]);
      }
      if (slot_done && ++slot == kSlots) {
        slot = 0;
        cphase ^= 1u;
      }
    }
  }
}

// 16-bit results of the thread's column: 16-row chunks half, half + 2, ... of the tile's rows.
template <bool SPLIT>
__device__ void writer(Ctl* ctl, uint32_t tmem, int half, const W4Args& a, const Walk& k) {
  using C = Cfg<SPLIT>;
  volatile int* abort = &ctl->abort;
  const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, l = 32 * quarter + lane;
  const bool gated = a.product == PGG_W4_GATED;
  const uint32_t d_tmem = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + 16 * half;
  int acc = 0;
  uint32_t dphase = 0;
  for (uint32_t t = k.first; t < k.total; t += k.step) {
    const Tile x = tile_of(t, a);
    const int exponent = a.col_exponent[column_index(a, x, l)];
    int4 m[C::kChunks];  // lane i holds what belongs to a chunk's row i
#pragma unroll
    for (int c = 0; c < C::kChunks; ++c) {
      const int j0 = 32 * c + 16 * half;
      m[c] = make_int4(0, 0, 0, 0);
      if (lane < 16 && j0 + lane < x.rows) m[c] = a.meta[x.prow + j0 + lane];
    }
    if (!__all_sync(0xFFFFFFFFu,
                    ptx::mbar_wait(&ctl->dfull[acc], dphase, a.wait_limit_ns, abort))) {
      if (lane == 0) {
        ctl->abort = 1;
        raise_status(a.hdr, kStTimeout, 188);
      }
      return;
    }
    ptx::tc_fence_after_sync();
    uint32_t sum[C::kChunks][16];
#pragma unroll
    for (int c = 0; c < C::kChunks; ++c)
      if (32 * c + 16 * half < x.rows16)
        ptx::tmem_ld_32x32b_x16(d_tmem + C::kRows * acc + 32 * c, sum[c]);
    ptx::tmem_ld_wait();
    ptx::tc_fence_before_sync();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&ctl->dempty[acc]);
    acc ^= 1;
    if (acc == 0) dphase ^= 1u;
    const int64_t f = x.n0 + (gated ? l >> 1 : l);
    const bool writes = f < a.N && (!gated || (lane & 1) == 0);
#pragma unroll
    for (int c = 0; c < C::kChunks; ++c) {
      const int left = x.rows - 32 * c - 16 * half;
      if (left <= 0) continue;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (i >= left) continue;
        float v = times_power(__uint_as_float(sum[c][i]),
                              __shfl_sync(0xFFFFFFFFu, m[c].y, i) + exponent);
        if (gated) {
          const float up = __shfl_xor_sync(0xFFFFFFFFu, v, 1);
          v = gate(v, up, __int_as_float(__shfl_sync(0xFFFFFFFFu, m[c].z, i)));
        }
        const int row = __shfl_sync(0xFFFFFFFFu, m[c].x, i);
        const int64_t to = static_cast<int64_t>(row) * a.N + f;
        if (!writes || row < 0) continue;
        if (a.bf16)
          static_cast<__nv_bfloat16*>(a.out)[to] = __float2bfloat16_rn(v);
        else
          static_cast<__half*>(a.out)[to] = __float2half_rn(v);
      }
    }
  }
}

// fp32 results (not gated) of the same: an accumulator's sums are added to those before.
template <bool SPLIT>
__device__ void writer_f32(Ctl* ctl, uint32_t tmem, int half, const W4Args& a, const Walk& k) {
  using C = Cfg<SPLIT>;
  volatile int* abort = &ctl->abort;
  const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, l = 32 * quarter + lane;
  const uint32_t d_tmem = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + 16 * half;
  int acc = 0;
  uint32_t dphase = 0;
  for (uint32_t t = k.first; t < k.total; t += k.step) {
    const Tile x = tile_of(t, a);
    float sum[C::kChunks][16];
#pragma unroll
    for (int c = 0; c < C::kChunks; ++c)
#pragma unroll
      for (int i = 0; i < 16; ++i) sum[c][i] = 0.0f;
#pragma unroll 1
    for (int g = 0; g < k.groups; g += k.chain) {
      if (!__all_sync(0xFFFFFFFFu,
                      ptx::mbar_wait(&ctl->dfull[acc], dphase, a.wait_limit_ns, abort))) {
        if (lane == 0) {
          ctl->abort = 1;
          raise_status(a.hdr, kStTimeout, 192);
        }
        return;
      }
      ptx::tc_fence_after_sync();
#pragma unroll
      for (int c = 0; c < C::kChunks; ++c) {
        if (32 * c + 16 * half >= x.rows16) continue;
        uint32_t part[16];
        ptx::tmem_ld_32x32b_x16(d_tmem + C::kRows * acc + 32 * c, part);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[c][i] += __uint_as_float(part[i]);
      }
      ptx::tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&ctl->dempty[acc]);
      acc ^= 1;
      if (acc == 0) dphase ^= 1u;
    }
    const int exponent = a.col_exponent[column_index(a, x, l)];
    const bool writes = x.n0 + l < a.N;
#pragma unroll
    for (int c = 0; c < C::kChunks; ++c) {
      const int j0 = 32 * c + 16 * half, left = x.rows - j0;
      if (left <= 0) continue;
      int4 m = make_int4(0, 0, 0, 0);  // lane i holds what belongs to row i
      if (lane < 16 && lane < left) m = a.meta[x.prow + j0 + lane];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (i >= left) continue;
        const float v = times_power(sum[c][i], __shfl_sync(0xFFFFFFFFu, m.y, i) + exponent);
        const int row = __shfl_sync(0xFFFFFFFFu, m.x, i);
        if (writes && row >= 0)
          static_cast<float*>(a.out)[static_cast<int64_t>(row) * a.N + x.n0 + l] = v;
      }
    }
  }
}

template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

template <int U, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    w4_wide_kernel(const __grid_constant__ CUtensorMap tm, const W4Args a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + kSlots * kSlotBytes + kStages * kStageBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
  k.first = blockIdx.x;
  k.step = gridDim.x;
  k.total = a.hdr->n_row_blocks * static_cast<uint32_t>(a.n_blocks);
  k.groups = static_cast<int>((a.K + kGroup - 1) / kGroup);
  k.chain = a.out_f32 ? Cfg<SPLIT>::kChain : k.groups;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      ptx::mbar_init(&ctl->cfull[i], 1);
      ptx::mbar_init(&ctl->cempty[i], 8);
    }
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&ctl->full[i], 1 + 4);
      ptx::mbar_init(&ctl->done[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&ctl->dfull[i], 1);
      ptx::mbar_init(&ctl->dempty[i], 8);
    }
    ptx::mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    ptx::fence_mbar_init();
    ptx::tma_prefetch_desc(&tm);
  }
  if (warp == 1) {
    ptx::tmem_alloc(&ctl->tmem_base, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before_sync();
  __syncthreads();
  ptx::tc_fence_after_sync();
  const uint32_t tmem = ctl->tmem_base;
  const int wg = warp >> 2;
  if (wg == 0) {
    fewer_registers<kFewRegs>();
    if (warp == 0 && lane == 0) copier(smem, ctl, &tm, a, k);
    if (warp == 1) issuer<SPLIT>(smem, ctl, __shfl_sync(0xFFFFFFFFu, tmem, 0), a, k);
  } else if (wg <= 2) {
    fewer_registers<kUnpackRegs>();
    unpacker<U, SPLIT>(smem, ctl, tmem, wg - 1, a, k);
  } else {
    more_registers<kWriteRegs>();
    if (a.out_f32)
      writer_f32<SPLIT>(ctl, tmem, wg - 3, a, k);
    else
      writer<SPLIT>(ctl, tmem, wg - 3, a, k);
  }
  ptx::tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after_sync();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <int U, bool SPLIT>
cudaError_t launch_t(const CUtensorMap& tm, const W4Args& a, int num_sms, cudaStream_t stream) {
  auto kern = w4_wide_kernel<U, SPLIT>;
  static SmemLimit limit;
  cudaError_t err = allow_smem(&limit, kern, kSmem);
  if (err != cudaSuccess) return err;
  // The warpgroups' shares are those of kLaunchRegs a thread: with fewer (flags that ask the compiler for
  // it) the writers would wait for theirs without end.
  static std::atomic<bool> enough{false};
  if (!enough.load()) {
    cudaFuncAttributes attr;
    err = cudaFuncGetAttributes(&attr, kern);
    if (err != cudaSuccess) return err;
    if (attr.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;
    enough.store(true);
  }
  return launch_pdl(kern, dim3(static_cast<unsigned>(num_sms)), dim3(kThreads),
                    static_cast<size_t>(kSmem), stream, 1, tm, a);
}

template <bool SPLIT>
cudaError_t launch_u(const CUtensorMap& tm, const W4Args& a, int num_sms, cudaStream_t stream) {
  if (a.group % 128 == 0) return launch_t<128, SPLIT>(tm, a, num_sms, stream);
  if (a.group % 64 == 0) return launch_t<64, SPLIT>(tm, a, num_sms, stream);
  return launch_t<32, SPLIT>(tm, a, num_sms, stream);
}

}  // namespace

int w4_wide_rows(int dtype, bool scale_f32, bool zeros) {
  return dtype == PGG_BF16 && !scale_f32 && !zeros ? kW4WideRows : kW4SplitRows;
}
int64_t w4_packed_wide_rows(int64_t M, int64_t row_blocks) { return M + 16 * row_blocks; }
int64_t w4_packed_wide_bytes(int64_t M, int64_t row_blocks, int64_t K) {
  return w4_packed_wide_rows(M, row_blocks) * ((K + kGroup - 1) / kGroup * kGroup) * 2;
}

cudaError_t launch_w4_wide(int dtype, W4Args a, const int64_t* group_list, int num_sms,
                           cudaStream_t stream) {
  const int tile = a.product == PGG_W4_GATED ? kTile / 2 : kTile;
  const int64_t columns = a.product == PGG_W4_GATED ? 2 * a.N : a.N;
  a.n_blocks = static_cast<int32_t>((a.N + tile - 1) / tile);
  a.bf16 = dtype == PGG_BF16;
  a.block_rows = w4_wide_rows(dtype, a.scale_f32 != 0, a.zeros != nullptr);
  CUtensorMap tm;  // codes as words of 16 bits: boxes of 128 bytes x 64 columns
  std::memset(&tm, 0, sizeof(tm));
  if (!encode_map_3d(&tm, PGG_F16, a.codes, a.row_bytes / 2, columns, a.G, 64))
    return cudaErrorInvalidValue;
  const int64_t rows = a.max_row_blocks * a.block_rows, cols = (a.G * columns + 15) / 16;
  const int row_blocks = static_cast<int>(rows < num_sms * 12 ? rows : num_sms * 12);
  const int col_blocks = static_cast<int>(cols < num_sms * 4 ? cols : num_sms * 4);
  const cudaError_t err =
      launch_pdl(dtype == PGG_BF16 ? w4_pack_wide_kernel<PGG_BF16> : w4_pack_wide_kernel<PGG_F16>,
                 dim3(static_cast<unsigned>(row_blocks + col_blocks)), dim3(128), 0, stream, 1, a,
                 group_list, row_blocks);
  if (err != cudaSuccess) return err;
  return a.block_rows == kW4WideRows ? launch_u<false>(tm, a, num_sms, stream)
                                     : launch_u<true>(tm, a, num_sms, stream);
}

}  // namespace pgg
