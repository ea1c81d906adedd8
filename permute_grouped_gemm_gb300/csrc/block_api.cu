// C ABI of the 4-bit experts, the norms around a block and the gradients' norm
// (include/pgg.h): argument validation, workspace layouts, the choice of kernel
// and the launches.

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <initializer_list>

#include <cuda_runtime.h>

#include "pgg.h"
#include "pgg_block.h"

namespace pgg {
namespace {

constexpr int64_t kInt32Max = 2147483647;

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool known_dtype(int d) { return d == PGG_F32 || d == PGG_F16 || d == PGG_BF16; }
uintptr_t elem_size(int d) { return d == PGG_F32 ? 4 : 2; }
int status_of(cudaError_t e) { return e == cudaSuccess ? PGG_OK : PGG_ERR_CUDA; }

// ---------------------------------------------------------------- 4-bit experts

constexpr int kSimtRows = 32;
constexpr int kVariantWide = 0;    // tensor cores, row blocks of up to 160 rows (two-part weights: 128)
constexpr int kVariantStream = 1;  // tensor cores, the codes streamed for blocks of 8 to 32 rows
constexpr int kVariantSimt = 3;    // FP32 pipes: any dtype, size and alignment

// Up to this many rows per live expert the codes are streamed: 64 experts, K 7168, F 2048, gated, us
// streamed / wide: 16 rows 375 / 414, 24 rows 409 / 418, 32 rows 568 / 423; with zero points 386 / 555,
// 422 / 561 and 582 / 572; groups of 32 537 / 593, 570 / 598, 794 / 604. (The wide form reads and
// unpacks a weight once whatever the rows are; streamed blocks have at most 32 rows.) The rows are those
// of an even routing, as the host knows no other; an uneven one pays for it, since an expert's codes are
// streamed once for each of its blocks: 60 tokens on the same 8 of 256 experts 202 us, wide 120 (on 209
// experts 609 and 1265), 256 tokens 433, wide 185 (on 256 experts 894 and 1544).
constexpr double kStreamRows = 24.0;

struct W4Plan {
  int variant;
  int rows_per_block;
  int64_t max_row_blocks;
  size_t rblist, rowinfo, inv, rows, packed, exponent, col_exponent, parts, arrived, total;
};

int w4_plan(int product, int64_t M, int64_t N, int64_t K, int64_t G, int64_t L, int64_t batch,
            int64_t topK, int rowIdxType, int64_t groupSize, int dtype, W4Plan* p) {
  if (!known_dtype(dtype)) return PGG_ERR_DTYPE;
  if (product != PGG_W4_ROWS && product != PGG_W4_GATED && product != PGG_W4_COMBINED)
    return PGG_ERR_ATTR;
  if (batch <= 0 || topK <= 0 || (rowIdxType != 0 && rowIdxType != 1) || groupSize <= 0)
    return PGG_ERR_ATTR;
  if (M <= 0 || N <= 0 || K <= 0 || G <= 0) return PGG_ERR_SHAPE;
  if (M > kInt32Max || N > kInt32Max / 2 || K > kInt32Max || G > kInt32Max ||
      groupSize > kInt32Max)
    return PGG_ERR_SHAPE;
  if (L != M || batch > M || topK > M || batch * topK != M) return PGG_ERR_SHAPE;
  p->variant = kVariantSimt;
  p->rows_per_block = kSimtRows;
  if (dtype != PGG_F32 && K % 32 == 0 && groupSize % 32 == 0 && forced_variant() != kVariantSimt) {
    p->variant = kVariantStream;
    // room for an even routing's rows and what a draw adds to them in all but a few experts (their
    // rows take a second block), but an expert has at most one row of a token
    const double miss = topK >= G ? 0.0 : 1.0 - static_cast<double>(topK) / G;
    const double live = G * (1.0 - std::pow(miss, static_cast<double>(batch)));
    const double rows = M / live, most = rows + 2.8 * std::sqrt(rows);
    const double want = most < batch ? most : static_cast<double>(batch);
    p->rows_per_block = want <= 8 ? 8 : want <= 16 ? 16 : 32;
    const int forced = forced_variant();
    if (forced == kVariantWide || (forced != kVariantStream && rows > kStreamRows)) {
      p->variant = kVariantWide;
      p->rows_per_block = kW4SplitRows;  // (the smaller one, for the tables' sizes)
    }
  }
  p->max_row_blocks = (M + p->rows_per_block - 1) / p->rows_per_block + (G < M ? G : M);
  if (p->max_row_blocks * ((N + 31) / 32) > kInt32Max) return PGG_ERR_SHAPE;  // 32-bit tile numbers
  size_t used = 256;
  auto take = [&](int64_t bytes) {
    const size_t at = used;
    used = align_up(used + static_cast<size_t>(bytes), 256);
    return at;
  };
  p->rblist = take(static_cast<int64_t>(sizeof(int4)) * p->max_row_blocks);
  p->rowinfo = take(static_cast<int64_t>(sizeof(RowInfo)) * M);
  p->inv = take(4 * M);
  p->rows = take(product == PGG_W4_COMBINED ? 4 * M * N : 0);
  const bool stream = p->variant == kVariantStream, wide = p->variant == kVariantWide;
  p->packed = take(stream ? w4_packed_bytes(p->max_row_blocks, p->rows_per_block, K)
                   : wide ? w4_packed_wide_bytes(M, p->max_row_blocks, K)
                          : 0);
  p->exponent = take(stream ? p->max_row_blocks * p->rows_per_block * 4
                     : wide ? w4_packed_wide_rows(M, p->max_row_blocks) * 16
                            : 0);
  p->col_exponent = take(wide ? 4 * G * N * (product == PGG_W4_GATED ? 2 : 1) : 0);
  p->parts = take(stream ? 2ll * kW4Grid * p->rows_per_block * 128 * 4 : 0);
  p->arrived = take(stream ? kW4Grid * 4 : 0);
  p->total = used;
  return PGG_OK;
}

// ---------------------------------------------------------------- norms

bool known_norm(int k) {
  return k == PGG_NORM_NONE || k == PGG_NORM_RMS || k == PGG_NORM_LAYER;
}

// What the forward and the backward check alike.
int check_norm(const void* y, const void* gate, const void* post_weight, const void* post_bias,
               const void* pre_weight, const void* pre_bias, int64_t T, int64_t H, int dtype,
               int y_dtype, int param_dtype, int post, int pre, int gate_kind) {
  if (!known_dtype(dtype) || (y_dtype != dtype && y_dtype != PGG_F32) ||
      (param_dtype != dtype && param_dtype != PGG_F32))
    return PGG_ERR_DTYPE;
  if (!known_norm(post) || !known_norm(pre) || gate_kind < PGG_GATE_NONE ||
      gate_kind > PGG_GATE_FULL || T <= 0)
    return PGG_ERR_ATTR;
  if (H <= 0 || H > kInt32Max || T > kInt32Max) return PGG_ERR_SHAPE;
  if ((gate_kind != PGG_GATE_NONE) != (gate != nullptr)) return PGG_ERR_NULL;
  if (!y && (post != PGG_NORM_NONE || gate)) return PGG_ERR_NULL;
  if ((post == PGG_NORM_NONE && post_weight) || (pre == PGG_NORM_NONE && pre_weight) ||
      (post != PGG_NORM_LAYER && post_bias) || (pre != PGG_NORM_LAYER && pre_bias))
    return PGG_ERR_ATTR;
  const uintptr_t ps = elem_size(param_dtype);
  if (!aligned(y, elem_size(y_dtype)) || !aligned(gate, ps) || !aligned(post_weight, ps) ||
      !aligned(post_bias, ps) || !aligned(pre_weight, ps) || !aligned(pre_bias, ps))
    return PGG_ERR_ALIGN;
  return PGG_OK;
}

// How the rows of a call can be read: vectors of 16 bytes of the dtype, pairs of 16-bit elements, or
// (0) one by one. A vector of another dtype's tensor is 16-byte aligned, or to its own size.
struct Tensor {
  const void* p;
  int dtype;
};
int row_words(int64_t H, int dtype, std::initializer_list<const void*> own,
              std::initializer_list<Tensor> others) {
  for (const int words : {16, 4}) {
    const uintptr_t elems = words / elem_size(dtype);
    bool ok = elems > 1 && H % static_cast<int64_t>(elems) == 0;
    for (const void* p : own) ok = ok && aligned(p, words);
    for (const Tensor& t : others) {
      const uintptr_t bytes = elems * elem_size(t.dtype);
      ok = ok && aligned(t.p, bytes < 16 ? bytes : 16);
    }
    if (ok) return words;
  }
  return 0;
}

NormArgs norm_args(const void* x, const void* y, const void* gate, const void* post_weight,
                   const void* post_bias, const void* pre_weight, const void* pre_bias, int64_t T,
                   int64_t H, int y_dtype, int param_dtype, int post, int pre, int gate_kind,
                   float residual_scale, float weight_offset, float eps) {
  NormArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = x;
  a.y = y;
  a.gate = gate;
  a.w_post = post_weight;
  a.b_post = post_bias;
  a.w_pre = pre_weight;
  a.b_pre = pre_bias;
  a.T = T;
  a.H = H;
  a.post = post;
  a.pre = pre;
  a.gate_kind = gate_kind;
  a.y_f32 = y_dtype == PGG_F32;
  a.p_f32 = param_dtype == PGG_F32;
  a.residual_scale = residual_scale;
  a.weight_offset = weight_offset;
  a.eps = eps;
  return a;
}

// ---------------------------------------------------------------- clipping

struct ClipPlan {
  int64_t tables;
  size_t partial, total;
};

int clip_plan(int64_t count, ClipPlan* p) {
  if (count < 0) return PGG_ERR_ATTR;
  if (count > kInt32Max) return PGG_ERR_SHAPE;
  p->tables = (count + kClipTensors - 1) / kClipTensors;
  if (p->tables == 0) p->tables = 1;
  p->partial = 256;
  p->total = align_up(256 + static_cast<size_t>(p->tables) * kClipBlocks * sizeof(double), 256);
  return PGG_OK;
}

int check_clip(int64_t count, const void* const* grads, const int64_t* sizes,
               const pgg_dtype* dtypes, void* const* out, bool clip) {
  if (count > 0 && (!grads || !sizes || !dtypes || (clip && !out))) return PGG_ERR_NULL;
  int64_t chunks = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (!known_dtype(dtypes[i])) return PGG_ERR_DTYPE;
    if (sizes[i] < 0) return PGG_ERR_SHAPE;
    if (sizes[i] == 0) continue;
    if (!grads[i] || (clip && !out[i])) return PGG_ERR_NULL;
    if (!aligned(grads[i], elem_size(dtypes[i])) ||
        (clip && !aligned(out[i], elem_size(dtypes[i]))))
      return PGG_ERR_ALIGN;
    chunks += clip_chunks(sizes[i], dtypes[i]);
    if (chunks > kInt32Max) return PGG_ERR_SHAPE;  // 32-bit chunk numbers
  }
  return PGG_OK;
}

// No output may reach into another output, or into a gradient but its own (blocks of one read what
// those of the other write): the ranges in the order of their addresses.
int check_clip_ranges(int64_t count, const void* const* grads, const int64_t* sizes,
                      const pgg_dtype* dtypes, void* const* out) {
  struct Range {
    uintptr_t begin, end;
    bool written;
  };
  if (count == 0) return PGG_OK;
  Range* ranges = static_cast<Range*>(std::malloc(sizeof(Range) * 2 * static_cast<size_t>(count)));
  if (!ranges) return PGG_ERR_CUDA;
  int64_t n = 0;
  for (int64_t i = 0; i < count; ++i) {
    const uintptr_t bytes = static_cast<uintptr_t>(sizes[i]) * elem_size(dtypes[i]);
    if (bytes == 0) continue;
    const uintptr_t to = reinterpret_cast<uintptr_t>(out[i]);
    const uintptr_t from = reinterpret_cast<uintptr_t>(grads[i]);
    ranges[n++] = {to, to + bytes, true};
    if (from != to) ranges[n++] = {from, from + bytes, false};
  }
  std::sort(ranges, ranges + n, [](const Range& a, const Range& b) { return a.begin < b.begin; });
  uintptr_t written = 0, read = 0;  // ends of those before
  bool ok = true;
  for (int64_t i = 0; ok && i < n; ++i) {
    ok = ranges[i].begin >= written && !(ranges[i].written && ranges[i].begin < read);
    uintptr_t& end = ranges[i].written ? written : read;
    end = std::max(end, ranges[i].end);
  }
  std::free(ranges);
  return ok ? PGG_OK : PGG_ERR_ATTR;
}

// The tensors of one launch; returns its blocks.
int fill_table(ClipTable* t, int64_t begin, int64_t count, const void* const* grads,
               const int64_t* sizes, const pgg_dtype* dtypes, void* const* out, int num_sms) {
  int64_t left = count - begin;
  t->tensors = static_cast<int32_t>(left < kClipTensors ? left : kClipTensors);
  uint32_t chunks = 0;
  for (int i = 0; i < t->tensors; ++i) {
    t->in[i] = grads[begin + i];
    t->out[i] = out ? out[begin + i] : nullptr;
    t->n[i] = sizes[begin + i];
    t->dtype[i] = static_cast<uint8_t>(dtypes[begin + i]);
    t->first[i] = chunks;
    chunks += static_cast<uint32_t>(clip_chunks(sizes[begin + i], dtypes[begin + i]));
  }
  t->first[t->tensors] = chunks;
  int blocks = num_sms * 4 < kClipBlocks ? num_sms * 4 : kClipBlocks;
  if (chunks < static_cast<uint32_t>(blocks)) blocks = chunks > 0 ? static_cast<int>(chunks) : 1;
  return blocks;
}

int run_clip(int64_t count, const void* const* grads, const int64_t* sizes,
             const pgg_dtype* dtypes, float max_norm, float eps, float scale, void* workspace,
             size_t workspace_bytes, float* norm, void* const* out, bool clip,
             cudaStream_t stream) {
  if (!workspace || !norm) return PGG_ERR_NULL;
  ClipPlan p;
  int rc = clip_plan(count, &p);
  if (rc != PGG_OK) return rc;
  if (clip && !(max_norm >= 0.0f && eps >= 0.0f)) return PGG_ERR_ATTR;
  rc = check_clip(count, grads, sizes, dtypes, out, clip);
  if (rc != PGG_OK) return rc;
  if (!aligned(workspace, 256) || !aligned(norm, 4)) return PGG_ERR_ALIGN;
  if (workspace_bytes < p.total) return PGG_ERR_WORKSPACE;
  if (clip) {
    rc = check_clip_ranges(count, grads, sizes, dtypes, out);
    if (rc != PGG_OK) return rc;
  }
  HostEnv env;
  if (host_env(&env) != PGG_OK) return PGG_ERR_CUDA;
  WsHeader* hdr = static_cast<WsHeader*>(workspace);
  double* partial = reinterpret_cast<double*>(static_cast<char*>(workspace) + p.partial);
  ClipTable t;
  int64_t partials = 0;
  for (int64_t i = 0; i < p.tables; ++i) {
    const int blocks =
        fill_table(&t, i * kClipTensors, count, grads, sizes, dtypes, out, env.num_sms);
    rc = status_of(launch_clip_squares(t, hdr, partial + partials, blocks, stream));
    if (rc != PGG_OK) return rc;
    partials += blocks;
  }
  if (!clip) return status_of(launch_clip_norm(partial, partials, scale, norm, stream));
  for (int64_t i = p.tables - 1; i >= 0; --i) {
    const int blocks =
        fill_table(&t, i * kClipTensors, count, grads, sizes, dtypes, out, env.num_sms);
    rc = status_of(launch_clip_apply(t, partial, partials, max_norm, eps, scale, norm, blocks,
                                     stream));
    if (rc != PGG_OK) return rc;
  }
  return PGG_OK;
}

}  // namespace
}  // namespace pgg

using namespace pgg;

extern "C" {

int pgg_w4_workspace_size(pgg_w4_product product, int64_t M, int64_t N, int64_t K, int64_t G,
                          int64_t L, int64_t batch, int64_t topK, int rowIdxType,
                          int64_t groupSize, pgg_dtype dtype, size_t* workspace_bytes) {
  if (!workspace_bytes) return PGG_ERR_NULL;
  W4Plan p;
  const int rc = w4_plan(product, M, N, K, G, L, batch, topK, rowIdxType, groupSize, dtype, &p);
  if (rc != PGG_OK) return rc;
  *workspace_bytes = p.total;
  return PGG_OK;
}

int pgg_w4_execute(pgg_w4_product product, const void* x, const uint8_t* codes,
                   const void* scales, const uint8_t* zeros, const int64_t* expandedRowIdx,
                   const int64_t* groupList, const float* probs, int64_t M, int64_t N, int64_t K,
                   int64_t G, int64_t L, int64_t batch, int64_t topK, int rowIdxType,
                   int64_t groupSize, pgg_dtype dtype, pgg_dtype scale_dtype, pgg_dtype out_dtype,
                   void* workspace, size_t workspace_bytes, void* out, pgg_stream_t stream) {
  if (!x || !codes || !scales || !expandedRowIdx || !groupList || !workspace || !out)
    return PGG_ERR_NULL;
  W4Plan p;
  int rc = w4_plan(product, M, N, K, G, L, batch, topK, rowIdxType, groupSize, dtype, &p);
  if (rc != PGG_OK) return rc;
  if (probs && product != PGG_W4_GATED) return PGG_ERR_ATTR;
  if ((scale_dtype != dtype && scale_dtype != PGG_F32) ||
      (out_dtype != dtype && out_dtype != PGG_F32) ||
      (product == PGG_W4_GATED && out_dtype != dtype) ||
      (product == PGG_W4_COMBINED && out_dtype != PGG_F32))
    return PGG_ERR_DTYPE;
  if (!aligned(workspace, 256) || !aligned(expandedRowIdx, 8) || !aligned(groupList, 8) ||
      !aligned(probs, 4) || !aligned(x, elem_size(dtype)) ||
      !aligned(scales, elem_size(scale_dtype)) || !aligned(out, elem_size(out_dtype)))
    return PGG_ERR_ALIGN;
  if (workspace_bytes < p.total) return PGG_ERR_WORKSPACE;
  HostEnv env;
  if (host_env(&env) != PGG_OK) return PGG_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char* w = static_cast<char*>(workspace);
  RowsPrepArgs pr;
  pr.idx = expandedRowIdx;
  pr.groups = groupList;
  pr.hdr = reinterpret_cast<WsHeader*>(w);
  pr.rblist = reinterpret_cast<int4*>(w + p.rblist);
  pr.rowinfo = reinterpret_cast<RowInfo*>(w + p.rowinfo);
  pr.inv = reinterpret_cast<int32_t*>(w + p.inv);
  pr.M = M;
  pr.G = G;
  pr.top_k = static_cast<int32_t>(topK);
  pr.row_idx_type = rowIdxType;
  pr.rows_per_block = p.rows_per_block;
  // the tensor cores need 16-byte aligned rows; the FP32 pipes take any row blocks
  const bool tensor = p.variant != kVariantSimt && aligned(x, 16) && aligned(codes, 16);
  const bool stream_rows = tensor && p.variant == kVariantStream;
  if (tensor && !stream_rows) {
    pr.rows_per_block = w4_wide_rows(dtype, scale_dtype == PGG_F32, zeros != nullptr);
    pr.even = 1;
  }
  if (stream_rows) {
    pr.clear = reinterpret_cast<uint32_t*>(w + p.arrived);
    pr.n_clear = kW4Grid;
  }
  rc = status_of(launch_rows_prep(pr, env.num_sms, s));
  if (rc != PGG_OK) return rc;
  W4Args a;
  std::memset(&a, 0, sizeof(a));
  a.x = x;
  a.codes = codes;
  a.scales = scales;
  a.zeros = zeros;
  a.probs = probs;
  a.rblist = pr.rblist;
  a.rowinfo = pr.rowinfo;
  a.hdr = pr.hdr;
  a.out = product == PGG_W4_COMBINED ? w + p.rows : out;
  a.M = M;
  a.N = N;
  a.K = K;
  a.G = G;
  a.batch = batch;
  a.max_row_blocks = p.max_row_blocks;
  a.row_bytes = (K + 1) / 2;
  a.group = static_cast<int32_t>(groupSize);
  a.groups = static_cast<int32_t>((K + groupSize - 1) / groupSize);
  a.product = product;
  a.scale_f32 = scale_dtype == PGG_F32;
  a.out_f32 = out_dtype == PGG_F32;
  a.wait_limit_ns = env.wait_limit_ns;
  a.packed = w + p.packed;
  a.exponent = reinterpret_cast<int32_t*>(w + p.exponent);
  a.meta = reinterpret_cast<int4*>(w + p.exponent);
  a.col_exponent = reinterpret_cast<int32_t*>(w + p.col_exponent);
  if (tensor && !stream_rows) {
    rc = status_of(launch_w4_wide(dtype, a, groupList, env.num_sms, s));
  } else if (stream_rows) {
    a.parts = reinterpret_cast<float*>(w + p.parts);
    a.arrived = reinterpret_cast<uint32_t*>(w + p.arrived);
    a.pairs = N % 2 == 0 && aligned(a.out, 2 * elem_size(out_dtype));
    rc = status_of(launch_w4_stream(dtype, p.rows_per_block, a, env.num_sms, s));
  } else {
    rc = status_of(launch_w4_simt(dtype, a, env.num_sms, s));
  }
  if (rc != PGG_OK || product != PGG_W4_COMBINED) return rc;
  return status_of(launch_w4_combine(static_cast<const float*>(a.out), a.hdr, batch, topK, N,
                                     static_cast<float*>(out), env.num_sms, s));
}

int pgg_block_norm(const void* x, const void* y, const void* gate, const void* post_weight,
                   const void* post_bias, const void* pre_weight, const void* pre_bias, int64_t T,
                   int64_t H, pgg_dtype dtype, pgg_dtype y_dtype, pgg_dtype param_dtype,
                   pgg_norm post, pgg_norm pre, pgg_gate gate_kind, float residual_scale,
                   float weight_offset, float eps, void* r, void* h, pgg_stream_t stream) {
  if (!x || (!r && !h) || (h != nullptr) != (pre != PGG_NORM_NONE)) return PGG_ERR_NULL;
  const int rc = check_norm(y, gate, post_weight, post_bias, pre_weight, pre_bias, T, H, dtype,
                            y_dtype, param_dtype, post, pre, gate_kind);
  if (rc != PGG_OK) return rc;
  const uintptr_t es = elem_size(dtype);
  if (!aligned(x, es) || !aligned(r, es) || !aligned(h, es)) return PGG_ERR_ALIGN;
  HostEnv env;
  if (host_env(&env) != PGG_OK) return PGG_ERR_CUDA;
  NormArgs a = norm_args(x, y, gate, post_weight, post_bias, pre_weight, pre_bias, T, H, y_dtype,
                         param_dtype, post, pre, gate_kind, residual_scale, weight_offset, eps);
  a.r = r;
  a.h = h;
  const int words = row_words(
      H, dtype, {x, r, h},
      {{y, y_dtype}, {gate_kind == PGG_GATE_TOKEN ? nullptr : gate, param_dtype},
       {post_weight, param_dtype}, {post_bias, param_dtype}, {pre_weight, param_dtype},
       {pre_bias, param_dtype}});
  return status_of(launch_block_norm(dtype, a, words, env.num_sms,
                                     reinterpret_cast<cudaStream_t>(stream)));
}

int pgg_block_norm_grad_workspace_size(int64_t T, int64_t H, size_t* workspace_bytes) {
  if (!workspace_bytes) return PGG_ERR_NULL;
  if (T <= 0) return PGG_ERR_ATTR;
  if (H <= 0 || H > kInt32Max || T > kInt32Max) return PGG_ERR_SHAPE;
  *workspace_bytes = align_up(256 + static_cast<size_t>(norm_grad_blocks(T, H)) * 5 * 4 *
                                        static_cast<size_t>(H), 256);
  return PGG_OK;
}

int pgg_block_norm_grad(const void* d_r, const void* d_h, const void* r, const void* y,
                        const void* gate, const void* post_weight, const void* post_bias,
                        const void* pre_weight, const void* pre_bias, int64_t T, int64_t H,
                        pgg_dtype dtype, pgg_dtype y_dtype, pgg_dtype dh_dtype,
                        pgg_dtype param_dtype, pgg_norm post, pgg_norm pre, pgg_gate gate_kind,
                        float residual_scale, float weight_offset, float eps, void* workspace,
                        size_t workspace_bytes, void* d_x, void* d_y, void* d_gate,
                        float* d_post_weight, float* d_post_bias, float* d_pre_weight,
                        float* d_pre_bias, pgg_stream_t stream) {
  const bool pre_norm = pre != PGG_NORM_NONE;
  if (!workspace || !d_x || (!d_r && !d_h) || (d_h != nullptr) != pre_norm ||
      (r != nullptr) != pre_norm || (d_y != nullptr) != (y != nullptr) ||
      (d_gate != nullptr) != (gate != nullptr))
    return PGG_ERR_NULL;
  const int rc = check_norm(y, gate, post_weight, post_bias, pre_weight, pre_bias, T, H, dtype,
                            y_dtype, param_dtype, post, pre, gate_kind);
  if (rc != PGG_OK) return rc;
  if ((d_post_weight && !post_weight) || (d_post_bias && !post_bias) ||
      (d_pre_weight && !pre_weight) || (d_pre_bias && !pre_bias))
    return PGG_ERR_NULL;
  if (dh_dtype != dtype && dh_dtype != PGG_F32) return PGG_ERR_DTYPE;
  const uintptr_t es = elem_size(dtype);
  const uintptr_t gs = gate_kind == PGG_GATE_FULL ? elem_size(param_dtype) : 4;
  if (!aligned(workspace, 256) || !aligned(d_r, es) || !aligned(d_h, elem_size(dh_dtype)) ||
      !aligned(r, es) || !aligned(d_x, es) || !aligned(d_y, es) || !aligned(d_gate, gs) ||
      !aligned(d_post_weight, 4) || !aligned(d_post_bias, 4) || !aligned(d_pre_weight, 4) ||
      !aligned(d_pre_bias, 4))
    return PGG_ERR_ALIGN;
  size_t need = 0;
  const int size_rc = pgg_block_norm_grad_workspace_size(T, H, &need);
  if (size_rc != PGG_OK) return size_rc;
  if (workspace_bytes < need) return PGG_ERR_WORKSPACE;
  HostEnv env;
  if (host_env(&env) != PGG_OK) return PGG_ERR_CUDA;
  NormArgs a = norm_args(r, y, gate, post_weight, post_bias, pre_weight, pre_bias, T, H, y_dtype,
                         param_dtype, post, pre, gate_kind, residual_scale, weight_offset, eps);
  a.dh_f32 = dh_dtype == PGG_F32;
  a.d_r = d_r;
  a.d_h = d_h;
  a.r = d_x;
  a.h = d_y;
  a.d_gate = d_gate;
  a.d_cols[0] = gate_kind == PGG_GATE_CHANNEL ? static_cast<float*>(d_gate) : nullptr;
  a.d_cols[1] = d_post_weight;
  a.d_cols[2] = d_post_bias;
  a.d_cols[3] = d_pre_weight;
  a.d_cols[4] = d_pre_bias;
  a.hdr = static_cast<WsHeader*>(workspace);
  a.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + 256);
  const int words = row_words(H, dtype, {d_r, r, d_x, d_y},
                              {{y, y_dtype}, {d_h, dh_dtype},
                               {gate_kind == PGG_GATE_TOKEN ? nullptr : gate, param_dtype},
                               {gate_kind == PGG_GATE_FULL ? d_gate : nullptr, param_dtype},
                               {post_weight, param_dtype}, {post_bias, param_dtype},
                               {pre_weight, param_dtype}});
  return status_of(launch_block_norm_grad(dtype, a, words,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

int pgg_clip_workspace_size(int64_t count, size_t* workspace_bytes) {
  if (!workspace_bytes) return PGG_ERR_NULL;
  ClipPlan p;
  const int rc = clip_plan(count, &p);
  if (rc != PGG_OK) return rc;
  *workspace_bytes = p.total;
  return PGG_OK;
}

int pgg_grad_norm(int64_t count, const void* const* grads, const int64_t* sizes,
                  const pgg_dtype* dtypes, float scale, void* workspace, size_t workspace_bytes,
                  float* norm, pgg_stream_t stream) {
  return run_clip(count, grads, sizes, dtypes, 0.0f, 0.0f, scale, workspace, workspace_bytes, norm,
                  nullptr, false, reinterpret_cast<cudaStream_t>(stream));
}

int pgg_clip_grads(int64_t count, const void* const* grads, const int64_t* sizes,
                   const pgg_dtype* dtypes, float max_norm, float eps, float scale,
                   void* workspace, size_t workspace_bytes, float* norm, void* const* out,
                   pgg_stream_t stream) {
  return run_clip(count, grads, sizes, dtypes, max_norm, eps, scale, workspace, workspace_bytes,
                  norm, out, true, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
