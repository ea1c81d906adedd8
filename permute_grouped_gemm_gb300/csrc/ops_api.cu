// C ABI of the router, the gated product and the adapters (include/pgg.h):
// argument validation, workspace layouts, the choice of kernel and the launches.

#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda.h>
#include <cuda_runtime.h>

#include "pgg.h"
#include "pgg_internal.h"
#include "pgg_ops.h"

namespace pgg {
namespace {

constexpr int64_t kInt32Max = 2147483647;
constexpr int kVariantWide = 0;  // tensor cores, row blocks of up to 256 rows on CTA pairs
constexpr int kVariantSkinny = 1;  // tensor cores, few rows per block, the weight streamed
constexpr int kVariantSimt = 3;  // FP32 pipes: any dtype, size and alignment

// Gated product: up to this many rows per live expert the weights bound it and are streamed once
// per block of rows; beyond, the tensor cores do. (60 experts, K 4096, F 1024: 96 rows each take
// 185 us this way and 210 in blocks of 256 rows, 128 rows 230 and 214; 32 experts, K 7168, F 2048:
// 302 and 363, 411 and 366.)
constexpr double kSkinnyRows = 104.0;

// Adapters: whether the shared weight is streamed for blocks of 64 tokens in the caller's order,
// with the low-rank part on the FP32 pipes (its cost grows with T R), or the tokens are sorted and
// the low-rank part is more steps of the product (0.4 to 0.7 us an adapter). Both sides: K 7168,
// N 4096, R 16, 256 tokens: 4 adapters 48 us and 53, 64 adapters 52 and 109; K = N = 4096, R 32,
// 32 adapters, 256 tokens: 56 and 64; R 64, 16 adapters: 64 tokens 32 and 44, 96 tokens 51 and 45;
// K 2048, N 5120, R 64: 128 tokens 79 and 40. Beyond one block of tokens only while the tiles of 64
// tokens x 128 columns fit the SMs at once (K 2048, N 5120, R 32: 192 tokens 42 and 51, 256 67 and
// 50). Their number is written here: the plan and the workspace's size go by this rule, and no
// device is asked for them.
constexpr int64_t kSms = 152;
bool few_tokens(int64_t T, int64_t N, int64_t R) {
  if (T <= 64) return T * R <= 8192;
  return T <= 256 && R <= 32 && (T + 63) / 64 * ((N + 127) / 128) <= kSms;
}

int few_token_block(int64_t T) { return T <= 16 ? 16 : T <= 32 ? 32 : 64; }

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool known_dtype(int d) { return d == PGG_F32 || d == PGG_F16 || d == PGG_BF16; }
int64_t elem_size(int d) { return d == PGG_F32 ? 4 : 2; }
int status_of(cudaError_t e) { return e == cudaSuccess ? PGG_OK : PGG_ERR_CUDA; }

// Takes pieces of a workspace, each aligned to 256 bytes.
struct Carver {
  size_t used = 0;
  size_t take(int64_t bytes) {
    const size_t at = used;
    used = align_up(used + static_cast<size_t>(bytes), 256);
    return at;
  }
};

// ---------------------------------------------------------------- router

int check_route(int64_t batch, int64_t G, int64_t topK) {
  if (batch <= 0 || topK <= 0) return PGG_ERR_ATTR;
  if (G <= 0 || G > kMaxRouteExperts || topK > G || topK > kMaxRouteTopK) return PGG_ERR_SHAPE;
  if (batch > kInt32Max / topK) return PGG_ERR_SHAPE;
  return PGG_OK;
}

// Header, the blocks' counts, and (several blocks only) every pair's rank.
size_t route_workspace(int64_t batch, int64_t G, int64_t topK, size_t* rank) {
  int blocks, per;
  route_blocks(batch, G, topK, &blocks, &per);
  *rank = 256 + align_up(static_cast<size_t>(G) * static_cast<size_t>(blocks) * 4, 256);
  return *rank + (blocks > 1 ? align_up(static_cast<size_t>(batch * topK) * 4, 256) : 0);
}

// ---------------------------------------------------------------- gated product

struct GatedPlan {
  int variant;
  int rows_per_block;
  int64_t max_row_blocks;
  int64_t live_blocks;  // about how many row blocks an even routing gives
  size_t rblist, rowinfo, inv, total;
};

int check_gated(int64_t M, int64_t F, int64_t K, int64_t G, int64_t L, int64_t batch,
                int64_t topK, int rowIdxType, int dtype) {
  if (!known_dtype(dtype)) return PGG_ERR_DTYPE;
  if (batch <= 0 || topK <= 0 || (rowIdxType != 0 && rowIdxType != 1)) return PGG_ERR_ATTR;
  if (M <= 0 || F <= 0 || K <= 0 || G <= 0) return PGG_ERR_SHAPE;
  if (M > kInt32Max || F > kInt32Max / 2 || K > kInt32Max || G > kInt32Max) return PGG_ERR_SHAPE;
  if (L != M || batch > M || topK > M || batch * topK != M) return PGG_ERR_SHAPE;
  return PGG_OK;
}

// 16-bit rows that the tensor-memory-access unit can stream, x rows (K elements) that 32-bit
// offsets in 16-byte units can address.
bool tensor_sizes(int dtype, int64_t rows, int64_t K, int64_t N) {
  return dtype != PGG_F32 && K % 8 == 0 && N % 8 == 0 && rows * (K / 8) < 0xFFFFFFFFll;
}

int gated_plan(int64_t M, int64_t F, int64_t K, int64_t G, int64_t batch, int dtype,
               GatedPlan* p) {
  const int forced = forced_variant();
  p->variant = kVariantSimt;
  p->rows_per_block = 64;
  p->live_blocks = 0;
  if (forced != kVariantSimt && tensor_sizes(dtype, batch, K, F)) {
    const double topK = static_cast<double>(M) / static_cast<double>(batch);
    const double miss = topK >= G ? 0.0 : 1.0 - topK / static_cast<double>(G);
    const double live = G * (1.0 - std::pow(miss, static_cast<double>(batch)));
    const double rows = M / live;  // per live expert, if the routing is even
    p->variant = forced == kVariantWide || (forced != kVariantSkinny && rows > kSkinnyRows)
                     ? kVariantWide
                     : kVariantSkinny;
    p->rows_per_block = rows_wide_block();
    if (p->variant == kVariantSkinny) {
      // room for the even share and what an even draw adds to it in all but 0.3% of the experts
      // (their rows take a second block), but an expert has at most one row of a token
      const double most = rows + 2.8 * std::sqrt(rows);
      const double want = most < static_cast<double>(batch) ? most : static_cast<double>(batch);
      p->rows_per_block = want <= 16 ? 16 : want <= 32 ? 32 : want <= 64 ? 64 : 128;
    }
    p->live_blocks = static_cast<int64_t>(live * std::ceil(rows / p->rows_per_block) + 0.5);
  }
  p->max_row_blocks = (M + p->rows_per_block - 1) / p->rows_per_block + (G < M ? G : M);
  if (p->max_row_blocks * ((F + 63) / 64) > kInt32Max) return PGG_ERR_SHAPE;  // 32-bit tile numbers
  Carver c;
  c.take(sizeof(WsHeader));
  p->rblist = c.take(static_cast<int64_t>(sizeof(int4)) * p->max_row_blocks);
  p->rowinfo = c.take(static_cast<int64_t>(sizeof(RowInfo)) * M);
  p->inv = c.take(4 * M);
  p->total = c.used;
  return PGG_OK;
}

// ---------------------------------------------------------------- adapters

struct AdapterPlan {
  int variant;
  int rb;        // rows per low-rank row block
  int padded;
  int64_t max_row_blocks, rows_u;
  int blocks, tokens_per_block;
  size_t off, range, order, rblist, segs, blkseg, box, counts, u, v, total;
};

int check_adapters(int64_t T, int64_t K, int64_t N, int64_t R, int64_t A, int dtype) {
  if (!known_dtype(dtype)) return PGG_ERR_DTYPE;
  if (T <= 0) return PGG_ERR_ATTR;
  if (K <= 0 || N <= 0 || R <= 0 || A <= 0) return PGG_ERR_SHAPE;
  if (R > kMaxRank || A > kMaxAdapters) return PGG_ERR_SHAPE;
  if (T > kInt32Max / 2 || K > kInt32Max || N > kInt32Max) return PGG_ERR_SHAPE;
  return PGG_OK;
}

int adapter_plan(int64_t T, int64_t K, int64_t N, int64_t R, int64_t A, int dtype, bool grad,
                 AdapterPlan* p) {
  p->variant = kVariantSimt;
  const int forced = forced_variant();
  const int64_t groups = A + 1 < T ? A + 1 : T;
  p->rb = 64;
  if (forced != kVariantSimt && R % 8 == 0 && tensor_sizes(dtype, T, K, N) &&
      tensor_sizes(dtype, T, N, K)) {
    p->variant = !grad && (forced == kVariantSkinny || (forced != kVariantWide && few_tokens(T, N, R)))
                     ? kVariantSkinny
                     : kVariantWide;
    // low-rank rows: blocks of 16 when adapters have about that many tokens
    p->rb = !grad && T <= 16 * groups ? 16 : 64;
  }
  p->padded = 0;
  p->max_row_blocks = (T + p->rb - 1) / p->rb + groups;
  p->rows_u = grad ? T + (kRowPad - 1) * groups : T;
  const int64_t widest = N > K ? N : K;
  if (p->max_row_blocks * ((widest + 63) / 64) > kInt32Max) return PGG_ERR_SHAPE;
  adapter_blocks(T, &p->blocks, &p->tokens_per_block);
  Carver c;
  c.take(sizeof(WsHeader));
  p->off = c.take(8 * (A + 1));
  p->range = c.take(static_cast<int64_t>(sizeof(int4)) * (A + 1));
  p->order = c.take(static_cast<int64_t>(sizeof(RowInfo)) * T);
  p->rblist = c.take(static_cast<int64_t>(sizeof(int4)) * p->max_row_blocks);
  p->segs = c.take(static_cast<int64_t>(sizeof(int4)) * A);
  p->blkseg = c.take(static_cast<int64_t>(sizeof(int2)) * ((T + 255) / 256));
  p->box = c.take(8 * ((T + 255) / 256));
  p->counts = c.take(p->blocks > 8 ? 4 * (A + 1) * p->blocks : 0);
  // (16-bit: room for each of the forms, of which the split one is the largest)
  const int64_t low_bytes = dtype == PGG_F32 ? R * 4 : low_width(R) * 2;
  p->u = c.take(p->rows_u * low_bytes);
  p->v = c.take(grad ? p->rows_u * low_bytes : 0);
  p->total = c.used;
  return PGG_OK;
}

AdapterTables tables_of(const AdapterPlan& p, void* ws) {
  char* w = static_cast<char*>(ws);
  AdapterTables t;
  t.hdr = reinterpret_cast<WsHeader*>(w);
  t.off = reinterpret_cast<int64_t*>(w + p.off);
  t.range = reinterpret_cast<int4*>(w + p.range);
  t.order = reinterpret_cast<RowInfo*>(w + p.order);
  t.rblist = reinterpret_cast<int4*>(w + p.rblist);
  t.segs = reinterpret_cast<int4*>(w + p.segs);
  t.blkseg = reinterpret_cast<int2*>(w + p.blkseg);
  t.box = reinterpret_cast<int32_t*>(w + p.box);
  t.counts = reinterpret_cast<uint32_t*>(w + p.counts);
  return t;
}

int run_adapter_prep(const AdapterPlan& p, const AdapterTables& t, bool by_first,
                     const int64_t* adapter, int64_t T, int64_t A, cudaStream_t stream) {
  AdapterPrepArgs a;
  a.adapter = adapter;
  a.t = t;
  a.T = T;
  a.A = static_cast<int32_t>(A);
  a.rb = p.rb;
  a.padded = p.padded;
  a.by_first = by_first ? 1 : 0;
  a.blocks = p.blocks;
  a.tokens_per_block = p.tokens_per_block;
  return status_of(launch_adapter_prep(a, stream));
}

// u = scale * x f[adapter] for f [A, K, R], into rows of `u`, in the adapters' order.
// (early, late: see launch_order in pgg_ops_mma.cuh)
int run_shrink(const AdapterPlan& p, const AdapterTables& t, const HostEnv& env, LowRankForm form,
               bool early, bool late, const void* x, const void* f, const float* scale, void* u,
               int64_t T, int64_t K, int64_t R, int64_t A, int dtype, cudaStream_t stream) {
  RowsArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = x;
  a.w = f;
  a.scale = scale;
  a.rblist = t.rblist;
  a.rowinfo = t.order;
  a.hdr = t.hdr;
  a.out = u;
  a.M = T;
  a.N = R;
  a.K = K;
  a.G = A;
  a.batch = T;
  a.max_row_blocks = p.max_row_blocks;
  a.low_form = form;
  a.padded = p.padded;
  a.range = t.range;
  a.early = early ? 1 : 0;
  a.late = late ? 1 : 0;
  a.hold_release = env.hold_release;
  a.wait_limit_ns = env.wait_limit_ns;
  if (p.variant != kVariantSimt && aligned(x, 16) && aligned(f, 16)) {
    const int64_t live = (T + p.rb - 1) / p.rb + (A < T ? A : T) / 2;
    return status_of(launch_rows_skinny(dtype, kShrink, p.rb, a, live, env.num_sms, stream));
  }
  return status_of(launch_rows_simt(dtype, kShrink, a, env.num_sms, stream));
}

// The same for a few tokens, fp32 in the tokens' order; checks the ids too.
int run_few_shrink(const AdapterTables& t, const void* x, const void* f, const int64_t* adapter,
                   const float* scale, void* u, int64_t T, int64_t K, int64_t R, int64_t A,
                   int dtype, cudaStream_t stream) {
  RowsArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = x;
  a.w = f;
  a.adapter = adapter;
  a.scale = scale;
  a.hdr = t.hdr;
  a.out = u;
  a.M = T;
  a.N = R;
  a.K = K;
  a.G = A;
  return status_of(launch_few_shrink(dtype, a, stream));
}

// Whether the tensor cores take a projection of these tensors (the FP32 pipes do otherwise).
bool wide_takes(const AdapterPlan& p, const void* x, const void* w, const void* f, const void* y) {
  return p.variant != kVariantSimt && aligned(x, 16) && aligned(w, 16) && aligned(f, 16) &&
         aligned(y, 16);
}

// y = x W + u f[adapter]^T for W [K, N] (transposed: [N, K]) and f [A, N, R]. by_token: the
// adapter ids when u is fp32 in the tokens' order, else null.
int run_adapt(const AdapterPlan& p, const AdapterTables& t, const HostEnv& env, LowRankForm form,
              bool transposed, bool early, bool late, const int64_t* by_token, const void* x,
              const void* w, const void* u, const void* f, void* y, int64_t T, int64_t K, int64_t N,
              int64_t R, int64_t A, int dtype, cudaStream_t stream) {
  RowsArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = x;
  a.w = w;
  a.u = u;
  a.b = f;
  a.rblist = t.rblist;
  a.rowinfo = t.order;
  a.segs = t.segs;
  a.blkseg = t.blkseg;
  a.box = t.box;
  a.hdr = t.hdr;
  a.out = y;
  a.M = T;
  a.N = N;
  a.K = K;
  a.G = A;
  a.R = static_cast<int32_t>(R);
  a.low_form = form;
  a.batch = T;
  a.max_row_blocks = p.max_row_blocks;
  a.early = early ? 1 : 0;
  a.late = late ? 1 : 0;
  a.hold_release = env.hold_release;
  a.wait_limit_ns = env.wait_limit_ns;
  const RowsMode mode = transposed ? kAdaptT : kAdapt;
  if (by_token) {
    a.adapter = by_token;
    const int nr = few_token_block(T);
    return status_of(launch_rows_skinny(dtype, mode, nr, a, (T + nr - 1) / nr, env.num_sms,
                                        stream));
  }
  if (wide_takes(p, x, w, f, y))
    return status_of(launch_rows_wide(dtype, mode, a, (T + 255) / 256, env.num_sms, stream));
  return status_of(launch_rows_simt(dtype, mode, a, env.num_sms, stream));
}

}  // namespace
}  // namespace pgg

using namespace pgg;

extern "C" {

int pgg_route_workspace_size(int64_t batch, int64_t G, int64_t topK, size_t* workspace_bytes) {
  if (!workspace_bytes) return PGG_ERR_NULL;
  const int rc = check_route(batch, G, topK);
  if (rc != PGG_OK) return rc;
  size_t rank;
  *workspace_bytes = route_workspace(batch, G, topK, &rank);
  return PGG_OK;
}

int pgg_route_execute(const void* logits, const float* bias, int64_t batch, int64_t G,
                      int64_t topK, int rowIdxType, pgg_dtype dtype, pgg_score score,
                      int renormalize, float scale, void* workspace, size_t workspace_bytes,
                      float* probs, int64_t* experts, int64_t* expandedRowIdx, int64_t* groupList,
                      pgg_stream_t stream) {
  if (!logits || !workspace || !probs || !experts || !expandedRowIdx || !groupList)
    return PGG_ERR_NULL;
  if (!known_dtype(dtype)) return PGG_ERR_DTYPE;
  if (rowIdxType != 0 && rowIdxType != 1) return PGG_ERR_ATTR;
  const int kind = score & ~PGG_BIAS_ON_SCORE;
  if (kind != PGG_SCORE_SOFTMAX && kind != PGG_SCORE_SIGMOID) return PGG_ERR_ATTR;
  const int rc = check_route(batch, G, topK);
  if (rc != PGG_OK) return rc;
  if (!aligned(logits, static_cast<uintptr_t>(elem_size(dtype))) || !aligned(bias, 4) ||
      !aligned(probs, 4) || !aligned(experts, 8) || !aligned(expandedRowIdx, 8) ||
      !aligned(groupList, 8) || !aligned(workspace, 256))
    return PGG_ERR_ALIGN;
  size_t rank;
  if (workspace_bytes < route_workspace(batch, G, topK, &rank)) return PGG_ERR_WORKSPACE;
  RouteArgs a;
  a.logits = logits;
  a.bias = bias;
  a.probs = probs;
  a.experts = experts;
  a.idx = expandedRowIdx;
  a.groups = groupList;
  a.counts = reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) + 256);
  a.rank = reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) + rank);
  a.T = batch;
  a.scale = scale;
  a.G = static_cast<int32_t>(G);
  a.k = static_cast<int32_t>(topK);
  a.row_idx_type = rowIdxType;
  a.sigmoid = kind == PGG_SCORE_SIGMOID ? 1 : 0;
  a.bias_on_score = bias && (score & PGG_BIAS_ON_SCORE) ? 1 : 0;
  a.renormalize = renormalize != 0 ? 1 : 0;
  a.hdr = static_cast<WsHeader*>(workspace);
  route_blocks(batch, G, topK, &a.blocks, &a.tokens_per_block);
  return status_of(launch_route(dtype, a, reinterpret_cast<cudaStream_t>(stream)));
}

int pgg_route_grad(const float* d_probs, const void* logits, const int64_t* experts,
                   int64_t batch, int64_t G, int64_t topK, pgg_dtype dtype, pgg_score score,
                   int renormalize, float scale, void* d_logits, pgg_stream_t stream) {
  if (!d_probs || !logits || !experts || !d_logits) return PGG_ERR_NULL;
  if (!known_dtype(dtype)) return PGG_ERR_DTYPE;
  if (score != PGG_SCORE_SOFTMAX && score != PGG_SCORE_SIGMOID) return PGG_ERR_ATTR;
  const int rc = check_route(batch, G, topK);
  if (rc != PGG_OK) return rc;
  const uintptr_t es = static_cast<uintptr_t>(elem_size(dtype));
  if (!aligned(logits, es) || !aligned(d_logits, es) || !aligned(d_probs, 4) ||
      !aligned(experts, 8))
    return PGG_ERR_ALIGN;
  HostEnv env;
  if (host_env(&env) != PGG_OK) return PGG_ERR_CUDA;
  RouteGradArgs a;
  a.d_probs = d_probs;
  a.logits = logits;
  a.experts = experts;
  a.d_logits = d_logits;
  a.T = batch;
  a.scale = scale;
  a.G = static_cast<int32_t>(G);
  a.k = static_cast<int32_t>(topK);
  a.sigmoid = score == PGG_SCORE_SIGMOID ? 1 : 0;
  a.renormalize = renormalize != 0 ? 1 : 0;
  return status_of(launch_route_grad(dtype, a, env.num_sms,
                                     reinterpret_cast<cudaStream_t>(stream)));
}

int pgg_swiglu_workspace_size(int64_t M, int64_t F, int64_t K, int64_t G, int64_t L,
                              int64_t batch, int64_t topK, int rowIdxType, pgg_dtype dtype,
                              size_t* workspace_bytes) {
  if (!workspace_bytes) return PGG_ERR_NULL;
  int rc = check_gated(M, F, K, G, L, batch, topK, rowIdxType, dtype);
  if (rc != PGG_OK) return rc;
  GatedPlan p;
  rc = gated_plan(M, F, K, G, batch, dtype, &p);
  if (rc != PGG_OK) return rc;
  *workspace_bytes = p.total;
  return PGG_OK;
}

int pgg_swiglu_plan(int64_t M, int64_t F, int64_t K, int64_t G, int64_t L, int64_t batch,
                    int64_t topK, int rowIdxType, pgg_dtype dtype, pgg_plan_info* info) {
  if (!info) return PGG_ERR_NULL;
  int rc = check_gated(M, F, K, G, L, batch, topK, rowIdxType, dtype);
  if (rc != PGG_OK) return rc;
  GatedPlan p;
  rc = gated_plan(M, F, K, G, batch, dtype, &p);
  if (rc != PGG_OK) return rc;
  std::memset(info, 0, sizeof(*info));
  info->variant = p.variant;
  info->rows_per_block = p.rows_per_block;
  info->max_row_blocks = p.max_row_blocks;
  info->workspace_bytes = p.total;
  info->cta_pair = p.variant == kVariantWide ? 1 : 0;
  return PGG_OK;
}

int pgg_swiglu_execute(const void* x, const void* weight, const int64_t* expandedRowIdx,
                       const int64_t* groupList, const float* probs, int64_t M, int64_t F,
                       int64_t K, int64_t G, int64_t L, int64_t batch, int64_t topK,
                       int rowIdxType, pgg_dtype dtype, void* workspace, size_t workspace_bytes,
                       void* h, void* gate_up, pgg_stream_t stream) {
  if (!x || !weight || !expandedRowIdx || !groupList || !workspace || !h) return PGG_ERR_NULL;
  int rc = check_gated(M, F, K, G, L, batch, topK, rowIdxType, dtype);
  if (rc != PGG_OK) return rc;
  GatedPlan p;
  rc = gated_plan(M, F, K, G, batch, dtype, &p);
  if (rc != PGG_OK) return rc;
  const uintptr_t es = static_cast<uintptr_t>(elem_size(dtype));
  if (!aligned(workspace, 256) || !aligned(expandedRowIdx, 8) || !aligned(groupList, 8) ||
      !aligned(probs, 4) || !aligned(x, es) || !aligned(weight, es) || !aligned(h, es) ||
      !aligned(gate_up, es))
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
  rc = status_of(launch_rows_prep(pr, env.num_sms, s));
  if (rc != PGG_OK) return rc;
  RowsArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = x;
  a.w = weight;
  a.probs = probs;
  a.rblist = pr.rblist;
  a.rowinfo = pr.rowinfo;
  a.hdr = pr.hdr;
  a.out = h;
  a.gate_up = gate_up;
  a.M = M;
  a.N = F;
  a.K = K;
  a.G = G;
  a.batch = batch;
  a.max_row_blocks = p.max_row_blocks;
  a.hold_release = env.hold_release;
  a.wait_limit_ns = env.wait_limit_ns;
  // the tensor cores need 16-byte aligned rows; the FP32 pipes take any row blocks
  const bool rows16 = aligned(x, 16) && aligned(weight, 16) && aligned(h, 16) &&
                      aligned(gate_up, 16);
  if (p.variant == kVariantSkinny && rows16)
    return status_of(launch_rows_skinny(dtype, kGated, p.rows_per_block, a, p.live_blocks,
                                        env.num_sms, s));
  if (p.variant == kVariantWide && rows16)
    return status_of(launch_rows_wide(dtype, kGated, a, p.live_blocks, env.num_sms, s));
  return status_of(launch_rows_simt(dtype, kGated, a, env.num_sms, s));
}

int pgg_swiglu_grad_workspace_size(int64_t M, int64_t batch, int64_t topK,
                                   size_t* workspace_bytes) {
  return pgg_unpermute_grad_workspace_size(M, batch, topK, workspace_bytes);
}

int pgg_swiglu_grad(const void* d_h, const void* gate_up, const float* probs,
                    const int64_t* expandedRowIdx, int64_t M, int64_t F, int64_t batch,
                    int64_t topK, int rowIdxType, pgg_dtype dtype, void* workspace,
                    size_t workspace_bytes, void* d_gate_up, float* d_probs, void* h,
                    pgg_stream_t stream) {
  if (!d_h || !gate_up || !expandedRowIdx || !workspace || !d_gate_up) return PGG_ERR_NULL;
  if (d_probs && !probs) return PGG_ERR_NULL;
  if (!known_dtype(dtype)) return PGG_ERR_DTYPE;
  if (rowIdxType != 0 && rowIdxType != 1) return PGG_ERR_ATTR;
  size_t need = 0;
  int rc = pgg_swiglu_grad_workspace_size(M, batch, topK, &need);
  if (rc != PGG_OK) return rc;
  if (F <= 0 || F > kInt32Max / 2) return PGG_ERR_SHAPE;
  const uintptr_t es = static_cast<uintptr_t>(elem_size(dtype));
  if (!aligned(workspace, 256) || !aligned(expandedRowIdx, 8) || !aligned(probs, 4) ||
      !aligned(d_probs, 4) || !aligned(d_h, es) || !aligned(gate_up, es) ||
      !aligned(d_gate_up, es) || !aligned(h, es))
    return PGG_ERR_ALIGN;
  if (workspace_bytes < need) return PGG_ERR_WORKSPACE;
  HostEnv env;
  if (host_env(&env) != PGG_OK) return PGG_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char* w = static_cast<char*>(workspace);
  WsHeader* hdr = reinterpret_cast<WsHeader*>(w);
  rc = status_of(launch_index_prep(expandedRowIdx, M, rowIdxType,
                                   reinterpret_cast<int32_t*>(w + 256), hdr, env.num_sms, s));
  if (rc != PGG_OK) return rc;
  GatedGradArgs a;
  a.d_h = d_h;
  a.gate_up = gate_up;
  a.probs = probs;
  a.idx = expandedRowIdx;
  a.hdr = hdr;
  a.d_gate_up = d_gate_up;
  a.h = h;
  a.d_probs = d_probs;
  a.M = M;
  a.F = F;
  a.row_idx_type = rowIdxType;
  const bool vec = (F * static_cast<int64_t>(es)) % 16 == 0 && aligned(d_h, 16) &&
                   aligned(gate_up, 16) && aligned(d_gate_up, 16) && aligned(h, 16);
  return status_of(launch_gated_grad(dtype, a, vec, env.num_sms, s));
}

int pgg_adapters_workspace_size(int64_t T, int64_t K, int64_t N, int64_t R, int64_t A,
                                pgg_dtype dtype, size_t* workspace_bytes) {
  if (!workspace_bytes) return PGG_ERR_NULL;
  int rc = check_adapters(T, K, N, R, A, dtype);
  if (rc != PGG_OK) return rc;
  AdapterPlan p;
  rc = adapter_plan(T, K, N, R, A, dtype, false, &p);
  if (rc != PGG_OK) return rc;
  *workspace_bytes = p.total;
  return PGG_OK;
}

int pgg_adapters_plan(int64_t T, int64_t K, int64_t N, int64_t R, int64_t A, pgg_dtype dtype,
                      pgg_plan_info* info) {
  if (!info) return PGG_ERR_NULL;
  int rc = check_adapters(T, K, N, R, A, dtype);
  if (rc != PGG_OK) return rc;
  AdapterPlan p;
  rc = adapter_plan(T, K, N, R, A, dtype, false, &p);
  if (rc != PGG_OK) return rc;
  std::memset(info, 0, sizeof(*info));
  info->variant = p.variant;
  info->rows_per_block = p.variant == kVariantWide     ? rows_wide_block()
                         : p.variant == kVariantSkinny ? few_token_block(T)
                                                       : p.rb;
  info->max_row_blocks = p.max_row_blocks;
  info->workspace_bytes = p.total;
  info->cta_pair = p.variant == kVariantWide ? 1 : 0;
  return PGG_OK;
}

int pgg_adapters_execute(const void* x, const void* weight, const void* a, const void* b,
                         const int64_t* adapter, const float* scale, int64_t T, int64_t K,
                         int64_t N, int64_t R, int64_t A, pgg_dtype dtype, void* workspace,
                         size_t workspace_bytes, void* y, pgg_stream_t stream) {
  if (!x || !weight || !a || !b || !adapter || !workspace || !y) return PGG_ERR_NULL;
  int rc = check_adapters(T, K, N, R, A, dtype);
  if (rc != PGG_OK) return rc;
  AdapterPlan p;
  rc = adapter_plan(T, K, N, R, A, dtype, false, &p);
  if (rc != PGG_OK) return rc;
  const uintptr_t es = static_cast<uintptr_t>(elem_size(dtype));
  if (!aligned(workspace, 256) || !aligned(adapter, 8) || !aligned(scale, 4) || !aligned(x, es) ||
      !aligned(weight, es) || !aligned(a, es) || !aligned(b, es) || !aligned(y, es))
    return PGG_ERR_ALIGN;
  if (workspace_bytes < p.total) return PGG_ERR_WORKSPACE;
  HostEnv env;
  if (host_env(&env) != PGG_OK) return PGG_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const AdapterTables t = tables_of(p, workspace);
  void* u = static_cast<char*>(workspace) + p.u;
  // (the few-token form writes y eight bytes at a time)
  if (p.variant == kVariantSkinny && aligned(x, 16) && aligned(weight, 16) && aligned(a, 16) &&
      aligned(b, 16) && aligned(y, 8)) {
    rc = run_few_shrink(t, x, a, adapter, scale, u, T, K, R, A, dtype, s);
    if (rc != PGG_OK) return rc;
    return run_adapt(p, t, env, kLowFloat, false, false, false, adapter, x, weight, u, b, y, T, K, N,
                     R, A, dtype, s);
  }
  rc = run_adapter_prep(p, t, true, adapter, T, A, s);
  if (rc != PGG_OK) return rc;
  const LowRankForm form = dtype == PGG_F32                   ? kLowRounded
                           : wide_takes(p, x, weight, b, y) ? kLowSplit
                                                            : kLowFloat;
  rc = run_shrink(p, t, env, form, true, false, x, a, scale, u, T, K, R, A, dtype, s);
  if (rc != PGG_OK) return rc;
  return run_adapt(p, t, env, form, false, false, true, nullptr, x, weight, u, b, y, T, K, N, R, A,
                   dtype, s);
}

int pgg_adapters_grad_workspace_size(int64_t T, int64_t K, int64_t N, int64_t R, int64_t A,
                                     pgg_dtype dtype, size_t* workspace_bytes) {
  if (!workspace_bytes) return PGG_ERR_NULL;
  int rc = check_adapters(T, K, N, R, A, dtype);
  if (rc != PGG_OK) return rc;
  AdapterPlan p;
  rc = adapter_plan(T, K, N, R, A, dtype, true, &p);
  if (rc != PGG_OK) return rc;
  *workspace_bytes = p.total;
  return PGG_OK;
}

int pgg_adapters_grad(const void* d_y, const void* x, const void* weight, const void* a,
                      const void* b, const int64_t* adapter, const float* scale, int64_t T,
                      int64_t K, int64_t N, int64_t R, int64_t A, pgg_dtype dtype,
                      void* workspace, size_t workspace_bytes, void* d_x, void* d_a, void* d_b,
                      pgg_stream_t stream) {
  if (!d_y || !x || !weight || !a || !b || !adapter || !workspace || !d_a || !d_b)
    return PGG_ERR_NULL;
  int rc = check_adapters(T, K, N, R, A, dtype);
  if (rc != PGG_OK) return rc;
  AdapterPlan p;
  rc = adapter_plan(T, K, N, R, A, dtype, true, &p);
  if (rc != PGG_OK) return rc;
  const uintptr_t es = static_cast<uintptr_t>(elem_size(dtype));
  if (!aligned(workspace, 256) || !aligned(adapter, 8) || !aligned(scale, 4) ||
      !aligned(d_y, es) || !aligned(x, es) || !aligned(weight, es) || !aligned(a, es) ||
      !aligned(b, es) || !aligned(d_x, es) || !aligned(d_a, es) || !aligned(d_b, es))
    return PGG_ERR_ALIGN;
  if (workspace_bytes < p.total) return PGG_ERR_WORKSPACE;
  HostEnv env;
  if (host_env(&env) != PGG_OK) return PGG_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const AdapterTables t = tables_of(p, workspace);
  void* u = static_cast<char*>(workspace) + p.u;
  void* v = static_cast<char*>(workspace) + p.v;
  // on the tensor cores throughout, or, for what they cannot take, on the FP32 pipes and with the
  // weight-gradient kernels (which want the groups by id, one behind the other)
  const bool tensor = p.variant != kVariantSimt && aligned(x, 16) && aligned(d_y, 16) &&
                      aligned(a, 16) && aligned(b, 16) && aligned(d_a, 16) && aligned(d_b, 16) &&
                      (!d_x || wide_takes(p, d_y, weight, a, d_x)) &&
                      static_cast<int64_t>(A) * ((K + 127) / 128 + (N + 127) / 128) <
                          kInt32Max / 4;
  const LowRankForm form = tensor ? kLowSplit : kLowRounded;
  p.padded = tensor ? 1 : 0;
  rc = run_adapter_prep(p, t, tensor, adapter, T, A, s);
  if (rc != PGG_OK) return rc;
  // u and v need the tables alone, and the factors' gradients u and v alone: each runs beside the
  // launch before it. 8192 tokens, K 4096, N 2048, R 32: 149 us against 172 one after another.
  rc = run_shrink(p, t, env, form, tensor, false, x, a, scale, u, T, K, R, A, dtype, s);
  if (rc != PGG_OK) return rc;
  rc = run_shrink(p, t, env, form, tensor, tensor, d_y, b, scale, v, T, N, R, A, dtype, s);
  if (rc != PGG_OK) return rc;
  if (d_x) {
    rc = run_adapt(p, t, env, form, true, tensor, true, nullptr, d_y, weight, v, a, d_x, T, N, K, R,
                   A, dtype, s);
    if (rc != PGG_OK) return rc;
  }
  if (tensor) {
    OuterArgs o;
    std::memset(&o, 0, sizeof(o));
    o.left[0] = x;
    o.left[1] = d_y;
    o.right[0] = v;
    o.right[1] = u;
    o.out[0] = d_a;
    o.out[1] = d_b;
    o.range = t.range;
    o.order = t.order;
    o.hdr = t.hdr;
    o.cols[0] = K;
    o.cols[1] = N;
    o.T = T;
    o.right_rows = p.rows_u;
    o.A = static_cast<int32_t>(A);
    o.R = static_cast<int32_t>(R);
    o.late = d_x ? 1 : 0;  // (else the launch before it writes v)
    o.hold_release = env.hold_release;
    o.wait_limit_ns = env.wait_limit_ns;
    return status_of(launch_rows_outer(dtype, o, env.num_sms, s));
  }
  rc = run_dw_tables(x, v, t.off, t.order, t.hdr, T, R, K, A, T, dtype, d_a, s);
  if (rc != PGG_OK) return rc;
  return run_dw_tables(d_y, u, t.off, t.order, t.hdr, T, R, N, A, T, dtype, d_b, s);
}

}  // extern "C"
