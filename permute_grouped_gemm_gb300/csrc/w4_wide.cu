// Products with 4-bit expert weights, many rows an expert: the tensor cores are
// the bound (tcgen05, 128 columns x up to 192 rows a tile).
//
//     D[column, row] = sum over a group of (code - zero) x,  sum += scale[column] D
//
// The columns are the MMA's M operand, so a column is a lane of tensor memory: a
// thread unpacks its own column's codes, four ANDs, a shift and four exact
// subtractions a word of eight (codes and zeros as fp16 subnormals, see
// w4_stream.cu), and writes them to tensor memory, from where the MMA takes them
// (tcgen05.st, A operand in tensor memory): through shared memory they would cost
// it as much as x does. A group's fp32 sums come back to the same thread, which
// multiplies its column's scale and adds: the weights are never rounded. x is
// brought to fp16 by a power of two a row and laid out as the MMA's other operand
// (panels of 64 k, 128-byte swizzle, pairs k + j, k + 4 + j) by a launch before
// this one, so it arrives in plain pieces.
//
// Tensor memory: two accumulators of up to 192 columns, two A buffers (128 of k:
// 64 columns). Roles: one warp copies, one issues the MMAs; eight unpack (four
// lane quarters x even and odd groups, so that the latencies of a group's waits and
// stores hide behind the other's); eight add up (four quarters x two halves of the
// rows, up to 96 sums a thread, for which the warpgroups' registers are split
// unevenly) and write the results, while the products of the next tile begin.
// Unpacking and adding up in the same warps, one after the other, took 2100
// cycles a group where this takes XX. Waits are bounded as everywhere.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <cstring>

#include "pgg_block.h"
#include "pgg_ops_launch.h"
#include "pgg_ops_mma.cuh"
#include "pgg_ptx.cuh"
#include "pgg_vec.cuh"

namespace pgg {
namespace {

constexpr int kTile = 128;            // columns of codes
constexpr int kRows = kW4WideRows;    // most rows of a tile
constexpr int kGroup = 128;           // of k: one A buffer, one stage of x
constexpr int kSlotBytes = kTile * 128;           // codes of 256 of k
constexpr int kStageBytes = kRows * kGroup * 2;   // x of 128 of k
constexpr int kSlots = 2, kStages = 4;
constexpr int kChunks = kRows / 32;   // of 16 rows, that an adding warp takes
constexpr int kACols = 2 * kRows;     // first tensor-memory column of the A buffers
// Warpgroups: copies and MMAs; two that unpack; two that add. Registers a thread of each, which
// draw on what the block is launched with.
constexpr int kThreads = 5 * 128;
constexpr int kLaunchRegs = 96, kFewRegs = 40, kUnpackRegs = 56, kAddRegs = 160;
static_assert(128 * kFewRegs + 256 * kUnpackRegs + 256 * kAddRegs <= kThreads * kLaunchRegs,
              "registers");

struct Ctl {
  uint64_t cfull[kSlots], cempty[kSlots];  // codes
  uint64_t xfull[kStages], xempty[kStages];
  uint64_t afull[2], aempty[2];  // codes of a group in tensor memory
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
                e.x >= 0 && e.x < a.G && e.y >= 0 && e.z > 0 && e.z <= kRows &&
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

__device__ __forceinline__ float block_max(float v, float* s) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  return fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
}

// A row of a row block: its power of two and its values as the MMA reads them. 128 threads a row.
template <int DT>
__global__ void __launch_bounds__(128) w4_pack_wide_kernel(const W4Args a) {
  __shared__ float s_max[4];
  ptx::griddep_wait();
  if (routing_failed(a.hdr)) return;
  const int tid = threadIdx.x;
  const int64_t width = (a.K + kGroup - 1) / kGroup * kGroup;
  const int64_t total = static_cast<int64_t>(a.hdr->n_row_blocks) * kRows;
  for (int64_t i = blockIdx.x; i < total; i += gridDim.x) {
    const int64_t rb = i / kRows;
    const int n = static_cast<int>(i - rb * kRows);
    const int4 e = a.rblist[check_index(a.hdr, rb, a.max_row_blocks, 182)];
    if (n >= e.z) continue;  // (what stands there reaches no row that is looked at)
    const int64_t row = check_index(a.hdr, static_cast<int64_t>(e.y) + n, a.M, 183);
    const int64_t xrow = a.product == PGG_W4_COMBINED
                             ? row
                             : check_index(a.hdr, a.rowinfo[row].token, a.batch, 184);
    const uint16_t* x = static_cast<const uint16_t*>(a.x) + xrow * a.K;
    float most = 0.0f;
    for (int64_t k = 8 * tid; k < a.K; k += 8 * 128) {
      float v[8];
      vec::load<DT, 8>(x, k, v);
#pragma unroll
      for (int j = 0; j < 8; ++j)  // (infinities and NaN stay what they are under any power)
        most = fmaxf(most, fabsf(v[j]) < INFINITY ? fabsf(v[j]) : 0.0f);
    }
    most = block_max(most, s_max);
    int exponent = 0;  // of two: most = m 2^exponent, m in [0.5, 1)
    if (most > 0.0f) frexpf(most, &exponent);
    exponent -= 15;
    const float by0 = ldexpf(1.0f, -(exponent / 2)), by1 = ldexpf(1.0f, -(exponent - exponent / 2));
    const int64_t prow = packed_row(e, rb);
    if (tid == 0) {  // what the results need to know of the row
      const int64_t pos = check_index(a.hdr, a.rowinfo[row].rank, a.M, 189);
      const float p = a.probs ? a.probs[pos] : 1.0f;
      a.meta[prow + n] = make_int4(static_cast<int>(a.product == PGG_W4_COMBINED ? pos : row),
                                   exponent + 24, __float_as_int(p), 0);
    }
    char* out = static_cast<char*>(a.packed) + prow * width * 2;
    const int64_t panel = static_cast<int64_t>((e.z + 15) / 16 * 16) * 128;
    for (int64_t k = 8 * tid; k < width; k += 8 * 128) {
      float v[8] = {};
      if (k < a.K) vec::load<DT, 8>(x, k, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __half2float(__float2half_rn(v[j] * by0 * by1));
      uint4 w;
      w.x = vec::pack2<PGG_F16>(v[0], v[4]);
      w.y = vec::pack2<PGG_F16>(v[1] * 0.0625f, v[5] * 0.0625f);
      w.z = vec::pack2<PGG_F16>(v[2], v[6]);
      w.w = vec::pack2<PGG_F16>(v[3] * 0.0625f, v[7] * 0.0625f);
      const int chunk = static_cast<int>(k / 8) & 7;
      *reinterpret_cast<uint4*>(out + k / 64 * panel + n * 128 + ((chunk ^ (n & 7)) << 4)) = w;
    }
  }
}

// ------------------------------------------------------------------ copies

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          ptx::smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(ptx::smem_addr(bar))
      : "memory");
}

struct Walk {
  uint32_t first, step, total;
  int groups;  // of 128 of k
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
      if (!ptx::mbar_wait(&ctl->xempty[stage], xphase ^ 1u, a.wait_limit_ns, abort)) {
        failed = true;
        break;
      }
      ptx::mbar_arrive_expect_tx(&ctl->xfull[stage], bytes);
      bulk_load(xs + stage * kStageBytes, src + static_cast<int64_t>(g) * bytes, bytes,
                &ctl->xfull[stage]);
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
  for (int i = 0; i < kStages; ++i)
    if (x_out & (1u << i))
      ptx::mbar_wait(&ctl->xfull[i], (x_parity >> i) & 1u, a.wait_limit_ns, &no_abort);
}

// ------------------------------------------------------------------ MMAs

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

// One thread. U: of k that share a scale.
template <int U>
__device__ void issuer(uint8_t* smem, Ctl* ctl, uint32_t tmem, const W4Args& a, const Walk& k) {
  volatile int* abort = &ctl->abort;
  uint8_t* xs = smem + kSlots * kSlotBytes;
  int stage = 0, buf = 0, acc = 0;
  uint32_t xphase = 0, aphase = 0, dphase = 0;
  bool issued = false, failed = false;
  for (uint32_t t = k.first; t < k.total && !failed; t += k.step) {
    const Tile x = tile_of(t, a);
    const uint32_t panel = static_cast<uint32_t>(x.rows16) * 128;
    const uint32_t idesc = ptx::idesc_make(0, kTile, x.rows16);
    for (int g = 0; g < k.groups && !failed; ++g) {
      if (!ptx::mbar_wait(&ctl->xfull[stage], xphase, a.wait_limit_ns, abort) ||
          !ptx::mbar_wait(&ctl->afull[buf], aphase, a.wait_limit_ns, abort)) {
        failed = true;
        break;
      }
      ptx::tc_fence_after_sync();
      const uint32_t xb = ptx::smem_addr(xs + stage * kStageBytes);
      for (int u = 0; u < kGroup / U; ++u) {
        if (!ptx::mbar_wait(&ctl->dempty[acc], dphase ^ 1u, a.wait_limit_ns, abort)) {
          failed = true;
          break;
        }
        ptx::tc_fence_after_sync();
#pragma unroll
        for (int kk = 0; kk < U / 16; ++kk) {
          const int s = u * (U / 16) + kk;  // of 16 k
          mma_tmem(tmem + kRows * acc, tmem + kACols + 64 * buf + 8 * s,
                   ptx::sdesc_sw128(xb + (s >> 2) * panel) +
                       static_cast<uint64_t>(((s & 3) * 32) >> 4),
                   idesc, kk > 0 ? 1u : 0u);
        }
        issued = true;
        ptx::mma_commit(&ctl->dfull[acc]);
        acc ^= 1;
        if (acc == 0) dphase ^= 1u;
      }
      if (failed) break;
      ptx::mma_commit(&ctl->aempty[buf]);
      ptx::mma_commit(&ctl->xempty[stage]);
      if (++stage == kStages) {
        stage = 0;
        xphase ^= 1u;
      }
      buf ^= 1;
      if (buf == 0) aphase ^= 1u;
    }
  }
  if (failed) {
    ctl->abort = 1;
    raise_status(a.hdr, kStTimeout, 186);
  }
  if (issued) {
    int no_abort = 0;
    ptx::mma_commit(&ctl->drain);
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

__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
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

// A scale as it stands in memory (what converts it would wait for it), and as a number.
__device__ __forceinline__ uint32_t raw_scale(const W4Args& a, int64_t i) {
  return a.scale_f32 ? __ldg(static_cast<const uint32_t*>(a.scales) + i)
                     : __ldg(static_cast<const uint16_t*>(a.scales) + i);
}
__device__ __forceinline__ float scale_of(const W4Args& a, uint32_t v) {
  if (a.scale_f32) return __uint_as_float(v);
  return a.bf16 ? __uint_as_float(v << 16)
                : __half2float(__ushort_as_half(static_cast<uint16_t>(v)));
}

// A lane's first scale in its column (a column that is not there: any scales).
__device__ __forceinline__ int64_t first_scale(const W4Args& a, const Tile& x, int l) {
  const int64_t c = column_of(a, x, l);
  return (x.g * (a.product == PGG_W4_GATED ? 2 * a.N : a.N) + (c < 0 ? 0 : c)) * a.groups;
}

template <int U>
__device__ __forceinline__ uint32_t group_of(const W4Args& a, uint32_t unit) {
  return a.group == U ? unit : unit * U / static_cast<uint32_t>(a.group);
}

// Groups `par`, par + 2, ... of this CTA's sequence of groups: the thread's column, 128 of k, into A
// buffer par.
template <int U>
__device__ void unpacker(uint8_t* smem, Ctl* ctl, uint32_t tmem, int par, const W4Args& a,
                         const Walk& k) {
  constexpr int kZeros = U < kGroup ? kGroup / U : 1;  // of a column and group
  volatile int* abort = &ctl->abort;
  const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, l = 32 * quarter + lane;
  const int row = code_row(a.product == PGG_W4_GATED, l);
  const uint32_t codes = ptx::smem_addr(smem) + row * 128;
  const uint32_t a_tmem = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + kACols + 64 * par;
  // slots of codes: one for two groups of a tile
  int slot = 0;
  uint32_t cphase = 0, aphase = 0;
  uint32_t turn = 0;  // of all groups
  for (uint32_t t = k.first; t < k.total; t += k.step) {
    const int64_t at = a.zeros ? first_scale(a, tile_of(t, a), l) : 0;
    for (int g = 0; g < k.groups; ++g, ++turn) {
      const bool slot_done = (g & 1) || g + 1 == k.groups;
      if ((turn & 1) == static_cast<uint32_t>(par)) {
        uint32_t zero[kZeros];
#pragma unroll
        for (int i = 0; i < kZeros; ++i) {
          zero[i] = 8;
          if (a.zeros) {
            const uint32_t group = group_of<U>(a, g * (kGroup / U) + i);
            zero[i] = group < static_cast<uint32_t>(a.groups) ? __ldg(a.zeros + at + group) : 0;
          }
        }
        const bool ok = ptx::mbar_wait(&ctl->cfull[slot], cphase, a.wait_limit_ns, abort) &&
                        ptx::mbar_wait(&ctl->aempty[par], aphase ^ 1u, a.wait_limit_ns, abort);
        if (!__all_sync(0xFFFFFFFFu, ok)) {
          if (lane == 0) {
            ctl->abort = 1;
            raise_status(a.hdr, kStTimeout, 187);
          }
          return;
        }
        ptx::tc_fence_after_sync();
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // 32 of k: four words, 16 columns of tensor memory
          const int chunk = (g & 1) * 4 + i;
          const uint4 q = lds128(codes + slot * kSlotBytes + ((chunk ^ (row & 7)) << 4));
          const uint32_t w[4] = {q.x, q.y, q.z, q.w};
          const uint32_t z = zero[i * 32 / U < kZeros ? i * 32 / U : 0];
          // zero 2^-24 and 2^-20
          const uint32_t z0 = __half_as_ushort(__float2half_rn(z * 0x1p-24f)) * 0x10001u;
          const uint32_t z1 = __half_as_ushort(__float2half_rn(z * 0x1p-20f)) * 0x10001u;
          uint32_t v[16];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t hi = w[j] >> 8;
            v[4 * j] = sub2(w[j] & 0x000F000Fu, z0);
            v[4 * j + 1] = sub2(w[j] & 0x00F000F0u, z1);
            v[4 * j + 2] = sub2(hi & 0x000F000Fu, z0);
            v[4 * j + 3] = sub2(hi & 0x00F000F0u, z1);
          }
          tmem_st_x16(a_tmem + 16 * i, v);
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(&ctl->afull[par]);
          ptx::mbar_arrive(&ctl->cempty[slot]);
        }
        aphase ^= 1u;
      } else if (slot_done && (g & 1) == 0) {
        // a slot with one group: the other warps have nothing to read of it (but it has to be this
        // use of the slot that they let go)
        if (!__all_sync(0xFFFFFFFFu, ptx::mbar_wait(&ctl->cfull[slot], cphase, a.wait_limit_ns,
                                                    abort))) {
          if (lane == 0) {
            ctl->abort = 1;
            raise_status(a.hdr, kStTimeout, 190);
          }
          return;
        }
        if (lane == 0) ptx::mbar_arrive(&ctl->cempty[slot]);
      }
      if (slot_done && ++slot == kSlots) {
        slot = 0;
        cphase ^= 1u;
      }
    }
  }
}

// Sums of the thread's column: 16-row chunks half, half + 2, ... of the tile's rows.
template <int U>
__device__ void adder(Ctl* ctl, uint32_t tmem, int half, const W4Args& a, const Walk& k) {
  volatile int* abort = &ctl->abort;
  const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, l = 32 * quarter + lane;
  const bool gated = a.product == PGG_W4_GATED;
  const uint32_t d_tmem = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + 16 * half;
  int acc = 0;
  uint32_t dphase = 0;
  for (uint32_t t = k.first; t < k.total; t += k.step) {
    const Tile x = tile_of(t, a);
    const int64_t at = first_scale(a, x, l);
    uint32_t s_next = raw_scale(a, at);
    float sum[kChunks][16];
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int i = 0; i < 16; ++i) sum[c][i] = 0.0f;
    const uint32_t units = k.groups * (kGroup / U);
    for (uint32_t unit = 0; unit < units; ++unit) {
      // (x is 0 behind the last group, but 0 inf is not)
      const bool in = group_of<U>(a, unit) < static_cast<uint32_t>(a.groups);
      const float s = in ? scale_of(a, s_next) : 0.0f;
      const uint32_t next = group_of<U>(a, unit + 1);
      if (next < static_cast<uint32_t>(a.groups)) s_next = raw_scale(a, at + next);
      if (!__all_sync(0xFFFFFFFFu, ptx::mbar_wait(&ctl->dfull[acc], dphase, a.wait_limit_ns,
                                                  abort))) {
        if (lane == 0) {
          ctl->abort = 1;
          raise_status(a.hdr, kStTimeout, 188);
        }
        return;
      }
      ptx::tc_fence_after_sync();
      const uint32_t d = d_tmem + kRows * acc;
#pragma unroll
      for (int c = 0; c < kChunks; c += 2) {  // rows 32 c + 16 half ..
        if (32 * c + 16 * half >= x.rows16) continue;
        uint32_t v[2][16];
        const bool two = 32 * (c + 1) + 16 * half < x.rows16;
        ptx::tmem_ld_32x32b_x16(d + 32 * c, v[0]);
        if (two) ptx::tmem_ld_32x32b_x16(d + 32 * (c + 1), v[1]);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[c][i] = fmaf(s, __uint_as_float(v[0][i]), sum[c][i]);
        if (two)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            sum[c + 1][i] = fmaf(s, __uint_as_float(v[1][i]), sum[c + 1][i]);
      }
      ptx::tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&ctl->dempty[acc]);
      acc ^= 1;
      if (acc == 0) dphase ^= 1u;
    }
    // results: this thread's column of its rows
    const int64_t f = x.n0 + (gated ? l >> 1 : l);
    const bool writes = f < a.N && (!gated || (lane & 1) == 0);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int j0 = 32 * c + 16 * half, left = x.rows - j0;
      if (left <= 0) continue;
      int4 m = make_int4(0, 0, 0, 0);  // lane i holds what belongs to the chunk's row i
      if (lane < 16 && lane < left) m = a.meta[x.prow + j0 + lane];
      // 2^e in two factors (it may lie outside fp32)
      const float by0 = ldexpf(1.0f, m.y / 2), by1 = ldexpf(1.0f, m.y - m.y / 2);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (i >= left) continue;
        float v = sum[c][i] * __shfl_sync(0xFFFFFFFFu, by0, i) * __shfl_sync(0xFFFFFFFFu, by1, i);
        if (gated) {
          const float up = __shfl_xor_sync(0xFFFFFFFFu, v, 1);
          v = gate(v, up, __int_as_float(__shfl_sync(0xFFFFFFFFu, m.z, i)));
        }
        const int64_t to = static_cast<int64_t>(__shfl_sync(0xFFFFFFFFu, m.x, i)) * a.N + f;
        if (!writes) continue;
        if (a.out_f32)
          static_cast<float*>(a.out)[to] = v;
        else if (a.bf16)
          static_cast<__nv_bfloat16*>(a.out)[to] = __float2bfloat16_rn(v);
        else
          static_cast<__half*>(a.out)[to] = __float2half_rn(v);
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

template <int U>
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
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      ptx::mbar_init(&ctl->cfull[i], 1);
      ptx::mbar_init(&ctl->cempty[i], 8);
    }
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&ctl->xfull[i], 1);
      ptx::mbar_init(&ctl->xempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&ctl->afull[i], 4);
      ptx::mbar_init(&ctl->aempty[i], 1);
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
    if (warp == 1 && lane == 0) issuer<U>(smem, ctl, tmem, a, k);
  } else if (wg <= 2) {
    fewer_registers<kUnpackRegs>();
    unpacker<U>(smem, ctl, tmem, wg - 1, a, k);
  } else {
    more_registers<kAddRegs>();
    adder<U>(ctl, tmem, wg - 3, a, k);
  }
  ptx::tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after_sync();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <int U>
cudaError_t launch_t(const CUtensorMap& tm, const W4Args& a, int num_sms, cudaStream_t stream) {
  auto kern = w4_wide_kernel<U>;
  static SmemLimit limit;
  const cudaError_t err = allow_smem(&limit, kern, kSmem);
  if (err != cudaSuccess) return err;
  return launch_pdl(kern, dim3(static_cast<unsigned>(num_sms)), dim3(kThreads),
                    static_cast<size_t>(kSmem), stream, 1, tm, a);
}

}  // namespace

int64_t w4_packed_wide_rows(int64_t M, int64_t row_blocks) { return M + 16 * row_blocks; }
int64_t w4_packed_wide_bytes(int64_t M, int64_t row_blocks, int64_t K) {
  return w4_packed_wide_rows(M, row_blocks) * ((K + kGroup - 1) / kGroup * kGroup) * 2;
}

cudaError_t launch_w4_wide(int dtype, W4Args a, int num_sms, cudaStream_t stream) {
  const int tile = a.product == PGG_W4_GATED ? kTile / 2 : kTile;
  a.n_blocks = static_cast<int32_t>((a.N + tile - 1) / tile);
  a.bf16 = dtype == PGG_BF16;
  CUtensorMap tm;  // codes as words of 16 bits: boxes of 128 bytes x 64 columns
  std::memset(&tm, 0, sizeof(tm));
  if (!encode_map_3d(&tm, PGG_F16, a.codes, a.row_bytes / 2,
                     a.product == PGG_W4_GATED ? 2 * a.N : a.N, a.G, 64))
    return cudaErrorInvalidValue;
  const int64_t rows = a.max_row_blocks * kRows;
  const int blocks = static_cast<int>(rows < num_sms * 16 ? rows : num_sms * 16);
  const cudaError_t err = launch_pdl(dtype == PGG_BF16 ? w4_pack_wide_kernel<PGG_BF16>
                                                       : w4_pack_wide_kernel<PGG_F16>,
                                     dim3(static_cast<unsigned>(blocks)), dim3(128), 0, stream, 1,
                                     a);
  if (err != cudaSuccess) return err;
  if (a.group % 128 == 0) return launch_t<128>(tm, a, num_sms, stream);
  if (a.group % 64 == 0) return launch_t<64>(tm, a, num_sms, stream);
  return launch_t<32>(tm, a, num_sms, stream);
}

}  // namespace pgg
