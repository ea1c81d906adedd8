// Products with 4-bit expert weights, few rows an expert: the codes are
// streamed once per block of up to 32 rows, and that stream is the bound.
//
// Tile: 128 columns of one expert (gated: 64 gates and their 64 ups) x NR rows.
// A stage is 512 of k (256 with 32 rows): the columns' codes by TMA, and the rows
// of x, which a launch before this one has gathered and laid out in the order in
// which the products read them. A warp takes 32 columns x 128 of k: codes are
// unpacked in registers, (v >> 4 j) & 0x000F000F | magic is the pair of numbers
// 2^7 + code (bf16; 2^10 + code in fp16), from which 2^7 + zero is subtracted
// exactly, and go as the A operand into mma.sync m16n8k16 with eight rows of x as
// B. (A word holds codes k .. k + 7, so such a pair is k + j, k + 4 + j; x is laid
// out the same way.) A group's fp32 sum is then multiplied by its scale: the
// weights are never rounded. The warp-wide product is used because the operand is
// made in registers: for tcgen05 it would go through shared memory once more (5
// bytes a code, where 128 a cycle serve all) or through tensor memory and two
// hand-overs a step; with eight to 32 rows the product itself is far from a bound.
//
// The tiles' steps of k are dealt to the CTAs in equal runs. A tile that is
// shared leaves fp32 parts in the workspace, and the CTA that comes last (a
// counter) adds them in the order of k: no CTA waits for another, and the result
// does not depend on who comes last.
//
// Warp 0 copies, the others multiply. Waits are bounded as everywhere.

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
constexpr int kPart = 128;       // of k: what a warp takes of a stage
constexpr int kPanelBytes = kTile * 128;  // codes of 256 of k
constexpr int kRedStride = kTile + 4;

// NT: eights of rows. U: of k that share a scale (a divisor of the group).
template <int NT, int U, bool ZEROS>
struct Cfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kParts = NT <= 2 ? 4 : 2;  // (more rows need more registers a warp)
  static constexpr int kStep = kParts * kPart;
  static constexpr int kMmaWarps = 4 * kParts;
  static constexpr int kUnits = kPart / U;  // scales of a column and part
  static constexpr int kCodeBytes = kParts / 2 * kPanelBytes;
  static constexpr int kXBytes = kRows * kStep * 2;
  static constexpr int kStageBytes = kCodeBytes + kXBytes;
  static constexpr int kRedFloats = kRows * kRedStride;
  static constexpr int kRedBytes = kParts / 2 * kRedFloats * 4;  // one for two parts
  static constexpr int kFit = (225 * 1024 - kRedBytes - 1024) / kStageBytes;
  static constexpr int kStages = kFit < 8 ? kFit : 8;
  static constexpr int kThreads = 32 * (1 + kMmaWarps);
  static constexpr int kSmem = kStages * kStageBytes + kRedBytes + 2048;
  static_assert(kStageBytes % 1024 == 0, "operand alignment");
};

struct Ctl {
  uint64_t full[8];   // the stage's bytes are there
  uint64_t empty[8];  // read by all warps
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

// `bytes` (a multiple of 16) from global to shared memory, both 16-byte aligned.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          ptx::smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(ptx::smem_addr(bar))
      : "memory");
}

template <int NT, int U, bool ZEROS>
__device__ void producer(uint8_t* smem, Ctl* ctl, const CUtensorMap* tm, const W4Args& a,
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
    const char* xp = static_cast<const char*>(a.packed) +
                     static_cast<int64_t>(x.rb) * k.nks * C::kXBytes;
    for (; ks < k.nks && s < k.end; ++ks, ++s) {
      if (!ptx::mbar_wait(&ctl->empty[stage], phase ^ 1u, a.wait_limit_ns, abort)) {
        failed = true;
        break;
      }
      uint8_t* p = smem + stage * C::kStageBytes;
      // (panels behind the last column or code bring nothing or zeros; x is zero there)
      ptx::mbar_arrive_expect_tx(&ctl->full[stage],
                                 (second ? C::kCodeBytes : C::kCodeBytes / 2) + C::kXBytes);
#pragma unroll
      for (int j = 0; j < C::kParts / 2; ++j) {
        const int32_t c = (ks * (C::kParts / 2) + j) * 64;
        ptx::tma_load_3d(p + j * kPanelBytes, tm, &ctl->full[stage], c, c0,
                         static_cast<int32_t>(x.g));
        if (second)
          ptx::tma_load_3d(p + j * kPanelBytes + kPanelBytes / 2, tm, &ctl->full[stage], c, c1,
                           static_cast<int32_t>(x.g));
      }
      bulk_load(p + C::kCodeBytes, xp + static_cast<int64_t>(ks) * C::kXBytes, C::kXBytes,
                &ctl->full[stage]);
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
  // the copies in flight land before the CTA ends
  int no_abort = 0;
  for (int i = 0; i < C::kStages; ++i)
    if (outstanding & (1u << i))
      ptx::mbar_wait(&ctl->full[i], (last_parity >> i) & 1u, a.wait_limit_ns, &no_abort);
}

// Where the eight values of x at k = 8 v of a stage, row n, stand: in the order in which the
// product's lanes read them, 16 bytes each.
template <int PARTS, int U>
__device__ __forceinline__ int x_place(int n, int v) {
  const int unit = v / (U / 8), rest = v % (U / 8), q = rest / (U / 32), i = rest % (U / 32);
  const int slot = unit * (U / 32) + i;  // of 32 k
  return ((n >> 3) * (4 * PARTS) + slot) * 512 + (((n & 7) * 4 + q) << 4);
}

// (x0 x1)(x2 x3)(x4 x5)(x6 x7) -> (x0 x4)(x1 x5)(x2 x6)(x3 x7)
__device__ __forceinline__ uint4 pair_up(const uint4& x) {
  return make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632),
                    __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
}

// The rows of x of every row block, gathered and in the products' order. A warp takes eight rows of
// a block and 32 of k: every 16 bytes of a lane are one of its 512 neighbouring bytes.
template <int NT, int U, bool ZEROS>
__global__ void __launch_bounds__(256) w4_pack_kernel(const W4Args a) {
  using C = Cfg<NT, U, ZEROS>;
  ptx::griddep_wait();
  if (routing_failed(a.hdr)) return;
  const int lane = threadIdx.x & 31;
  const uint32_t K = static_cast<uint32_t>(a.K);
  const uint32_t nks = (K + C::kStep - 1) / C::kStep;
  constexpr uint32_t kSlots = 4 * C::kParts * NT;  // of 512 bytes, a stage
  const uint64_t total = static_cast<uint64_t>(a.hdr->n_row_blocks) * nks * kSlots;
  const uint64_t step = static_cast<uint64_t>(gridDim.x) * 8;
  for (uint64_t i = blockIdx.x * 8ull + (threadIdx.x >> 5); i < total; i += step) {
    const uint64_t stage = i / kSlots;
    const uint32_t in_stage = static_cast<uint32_t>(i - stage * kSlots);
    const uint32_t rb = static_cast<uint32_t>(stage / nks);
    const uint32_t ks = static_cast<uint32_t>(stage - static_cast<uint64_t>(rb) * nks);
    const uint32_t slot = in_stage % (4 * C::kParts);
    const int n = 8 * static_cast<int>(in_stage / (4 * C::kParts)) + (lane >> 2);
    const int4 e = a.rblist[rb];
    if (n >= e.z) continue;  // (what stands there reaches no row that is looked at)
    // the inverse of x_place: this lane's eight values of k
    const uint32_t unit = slot / (U / 32), w = slot % (U / 32);
    const uint32_t k = ks * C::kStep + unit * U + (lane & 3) * (U / 4) + w * 8;
    const int64_t row = check_index(a.hdr, static_cast<int64_t>(e.y) + n, a.M, 173);
    const int64_t xrow = a.product == PGG_W4_COMBINED
                             ? row
                             : check_index(a.hdr, a.rowinfo[row].token, a.batch, 174);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (k < K)
      v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + xrow * a.K + k));
    *reinterpret_cast<uint4*>(static_cast<char*>(a.packed) + i * 512 + lane * 16) = pair_up(v);
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

// Codes j and 4 + j of a word, less the zero (`z` is the pair 2^7 + zero, or 2^10 + zero; `magic` the
// pair 2^7 or 2^10, from a register: an instruction holds one of the two constants only).
template <int DT>
__device__ __forceinline__ uint32_t unpack(uint32_t w, int j, uint32_t magic, uint32_t z) {
  uint32_t v, r;
  asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(v) : "r"(w >> (4 * j)), "r"(magic));
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

// A sum over the stage's parts of k, of which each two have been added already.
template <int PARTS, int STRIDE>
__device__ __forceinline__ float sum_parts(const float* p) {
  return PARTS == 4 ? p[0] + p[STRIDE] : p[0];
}

// The tile's results from `red` [row][column].
template <int DT, int NT>
__device__ __forceinline__ void write_tile(const float* red, const W4Args& a, const Tile& x,
                                           int thread) {
  using C = Cfg<NT, 128, false>;
  constexpr int kThr = C::kMmaWarps * 32;
  auto at_red = [&](int j, int c) {
    return sum_parts<C::kParts, C::kRedFloats>(red + j * kRedStride + c);
  };
  const bool gated = a.product == PGG_W4_GATED;
  const int half = gated ? 32 : 64;  // pairs of a row
  for (int i = thread; i < x.rows * half; i += kThr) {
    const int j = i / half, c = 2 * (i - j * half);
    const int64_t n = x.n0 + c;
    if (n >= a.N) continue;
    const int64_t row = x.row0 + j;
    const int64_t pos = check_index(a.hdr, a.rowinfo[row].rank, a.M, 176);
    float v0 = at_red(j, c), v1 = at_red(j, c + 1);
    if (gated) {
      const float p = a.probs ? a.probs[pos] : 1.0f;
      v0 = gate(v0, at_red(j, 64 + c), p);
      v1 = gate(v1, at_red(j, 65 + c), p);
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

// Scales (and zeros) of this lane's column for one step, a part of the k.
template <int DT, int NT, int U, bool ZEROS>
struct Scales {
  using C = Cfg<NT, U, ZEROS>;
  uint32_t s[C::kUnits];  // as they stand in memory: what converts them would wait for them
  uint32_t z[ZEROS ? C::kUnits : 1];

  // `at`: the column's first scale or -1;  unit: the first of the step's units of U
  __device__ __forceinline__ void load(const W4Args& a, int64_t at, uint32_t unit) {
#pragma unroll
    for (int u = 0; u < C::kUnits; ++u) {
      uint32_t group = unit + u;
      if (a.group != U) group = group * U / static_cast<uint32_t>(a.group);
      s[u] = 0;
      if (ZEROS) z[u] = 0;
      if (at < 0 || group >= static_cast<uint32_t>(a.groups)) continue;
      if (a.scale_f32)
        s[u] = __ldg(static_cast<const uint32_t*>(a.scales) + at + group);
      else
        s[u] = __ldg(static_cast<const uint16_t*>(a.scales) + at + group);
      if (ZEROS) z[u] = __ldg(a.zeros + at + group);
    }
  }
  __device__ __forceinline__ float scale(const W4Args& a, int u) const {
    if (a.scale_f32) return __uint_as_float(s[u]);
    if (DT == PGG_BF16) return __uint_as_float(s[u] << 16);
    return __half2float(__ushort_as_half(static_cast<uint16_t>(s[u])));
  }
};

template <int DT, int NT, int U, bool ZEROS>
__device__ void multiplier(uint8_t* smem, Ctl* ctl, float* red, int w, const W4Args& a,
                           const Walk& k) {
  using C = Cfg<NT, U, ZEROS>;
  constexpr int W = U / 32;  // words of a lane and unit
  constexpr int kThr = 32 * C::kMmaWarps;
  volatile int* abort = &ctl->abort;
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int col0 = 32 * (w & 3), part = w >> 2;
  // fragment row g is column perm of each eight, so that the lanes of one access to shared memory
  // (two g) lie in different halves of the swizzled 128 bytes
  const int perm = (g >> 1) + 4 * (g & 1);
  const int thread = 32 * w + lane;
  // bf16: 2^7 + z is 0x4300 | z, fp16: 2^10 + z is 0x6400 | z
  constexpr uint32_t kMagic = DT == PGG_BF16 ? 0x43004300u : 0x64006400u;
  const int64_t columns = a.product == PGG_W4_GATED ? 2 * a.N : a.N;
  const uint32_t my_codes =
      ptx::smem_addr(smem) + (part >> 1) * kPanelBytes + (col0 + perm) * 128;
  const uint32_t my_x = ptx::smem_addr(smem) + C::kCodeBytes + part * 4 * 512 + lane * 16;
  uint32_t magic;
  asm volatile("mov.u32 %0, %1;" : "=r"(magic) : "n"(kMagic));
  int stage = 0;
  uint32_t phase = 0;
  bool failed = false;
  for (int64_t s = k.begin; s < k.end;) {
    const uint32_t t = static_cast<uint32_t>(s / k.nks);
    const int ks0 = static_cast<int>(s - static_cast<int64_t>(t) * k.nks);
    const int64_t left = k.end - s;
    const int n_steps = left < k.nks - ks0 ? static_cast<int>(left) : k.nks - ks0;
    const Tile x = tile_of<C::kRows>(t, a);
    const int64_t column = column_of(a, x, col0 + lane);
    const int64_t at = column < 0 ? -1 : (x.g * columns + column) * a.groups;
    float sum[2][NT][4] = {};
    Scales<DT, NT, U, ZEROS> now, next;
    uint32_t unit = static_cast<uint32_t>(ks0 * C::kParts + part) * C::kUnits;
    next.load(a, at, unit);
    for (int i = 0; i < n_steps; ++i) {
      now = next;
      unit += C::kParts * C::kUnits;
      if (i + 1 < n_steps) next.load(a, at, unit);  // (a step ahead)
      if (!failed && !__all_sync(0xFFFFFFFFu, ptx::mbar_wait(&ctl->full[stage], phase,
                                                             a.wait_limit_ns, abort))) {
        failed = true;
        if (lane == 0) {
          ctl->abort = 1;
          raise_status(a.hdr, kStTimeout, 177);
        }
      }
      if (failed) break;  // (the warps still meet at every barrier below)
      const uint32_t codes = my_codes + stage * C::kStageBytes;
      const uint32_t xs = my_x + stage * C::kStageBytes;
#pragma unroll
      for (int u = 0; u < C::kUnits; ++u) {
        const int byte = (part & 1) * 64 + u * (U / 2) + q * (U / 8);
        const int in_row = (((byte >> 4) ^ perm) << 4) | (byte & 15);
        Words<W> word[2][2];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            word[r][e] = load_words<W>(codes + (16 * r + 8 * e) * 128 + in_row);
        uint32_t z[2][2];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            z[r][e] = kMagic + (ZEROS ? __shfl_sync(0xFFFFFFFFu, now.z[ZEROS ? u : 0],
                                                    16 * r + 8 * e + perm) * 0x10001u
                                      : 0x00080008u);
        float d[2][NT][4] = {};
#pragma unroll
        for (int i8 = 0; i8 < W; ++i8) {
          Words<4> b[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n)
            b[n] = load_words<4>(xs + (n * 4 * C::kParts + u * W + i8) * 512);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            uint32_t p[2][4];
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int j = 0; j < 4; ++j) p[e][j] = unpack<DT>(word[r][e].v[i8], j, magic, z[r][e]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma<DT>(d[r][n], p[0][0], p[1][0], p[0][1], p[1][1], b[n].v[0], b[n].v[1]);
              mma<DT>(d[r][n], p[0][2], p[1][2], p[0][3], p[1][3], b[n].v[2], b[n].v[3]);
            }
          }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float s0 = __shfl_sync(0xFFFFFFFFu, now.scale(a, u), 16 * r + perm);
          const float s1 = __shfl_sync(0xFFFFFFFFu, now.scale(a, u), 16 * r + 8 + perm);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            sum[r][n][0] = fmaf(s0, d[r][n][0], sum[r][n][0]);
            sum[r][n][1] = fmaf(s0, d[r][n][1], sum[r][n][1]);
            sum[r][n][2] = fmaf(s1, d[r][n][2], sum[r][n][2]);
            sum[r][n][3] = fmaf(s1, d[r][n][3], sum[r][n][3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&ctl->empty[stage]);
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    // the parts of k into red [row][column], each two one after the other
    if (s > k.begin) ptx::named_bar_sync(1, kThr);  // (the tile before is read)
#pragma unroll
    for (int turn = 0; turn < 2; ++turn) {
      if ((part & 1) == turn) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float* p = red + (part >> 1) * C::kRedFloats +
                         (8 * n + 2 * q + (e & 1)) * kRedStride + col0 + 16 * r + 8 * (e >> 1) +
                         perm;
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
        own[i] = sum_parts<C::kParts, C::kRedFloats>(red + (i / kTile) * kRedStride + i % kTile);
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
          float* p = red + (i / kTile) * kRedStride + i % kTile;
          p[0] = v;
          if (C::kParts == 4) p[C::kRedFloats] = 0.0f;
        }
        ptx::named_bar_sync(1, kThr);
      }
    }
    if (mine) write_tile<DT, NT>(red, a, x, thread);
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
      ptx::mbar_init(&ctl.full[s], 1);
      ptx::mbar_init(&ctl.empty[s], C::kMmaWarps);
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
  k.nks = static_cast<int>((a.K + C::kStep - 1) / C::kStep);
  k.total = static_cast<int64_t>(a.hdr->n_row_blocks) * a.n_blocks * k.nks;
  // at least two steps a CTA, so that each has some
  k.ctas = k.total < 2 * static_cast<int64_t>(gridDim.x) ? (k.total + 1) / 2 : gridDim.x;
  if (static_cast<int64_t>(blockIdx.x) >= k.ctas) return;
  k.begin = static_cast<int64_t>(blockIdx.x) * k.total / k.ctas;
  k.end = (static_cast<int64_t>(blockIdx.x) + 1) * k.total / k.ctas;
  if (warp == 0) {
    if (lane == 0) producer<NT, U, ZEROS>(smem, &ctl, &tm, a, k);
  } else {
    multiplier<DT, NT, U, ZEROS>(smem, &ctl, red, warp - 1, a, k);
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
  const int64_t slots = a.max_row_blocks * ((a.K + C::kStep - 1) / C::kStep) * 4 * C::kParts * NT;
  int64_t blocks = (slots + 7) / 8;
  if (blocks > num_sms * 8) blocks = num_sms * 8;
  const cudaError_t packed = launch_pdl(w4_pack_kernel<NT, U, ZEROS>,
                                        dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream,
                                        1, a);
  if (packed != cudaSuccess) return packed;
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

int64_t w4_packed_bytes(int64_t row_blocks, int rows_per_block, int64_t K) {
  const int64_t step = rows_per_block <= 16 ? 4 * kPart : 2 * kPart;
  return row_blocks * rows_per_block * ((K + step - 1) / step) * step * 2;
}

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
