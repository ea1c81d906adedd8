// Internal definitions of the router, gated-product and adapter operators:
// the tables their preparation kernels build in the workspace, the kernels'
// arguments, and the host helpers they share with the other entry points.
#pragma once

#include "pgg_internal.h"

namespace pgg {

// ------------------------------------------------------------ shared host helpers (pgg_api.cu)

struct HostEnv {
  int num_sms;             // of the current device
  int hold_release;        // test hook
  uint64_t wait_limit_ns;  // bound of every wait inside a kernel
};
int host_env(HostEnv* env);  // pgg_status
int forced_variant();        // test hook, -1 = automatic
// Tensor map of a row-major 16-bit [d2][d1][d0] array (d0 innermost) with boxes of 64 x box1 x 1
// elements and the 128-byte swizzle; reads outside it give zeros. False when it cannot be encoded.
bool encode_map_3d(CUtensorMap* m, int dtype, const void* base, int64_t d0, int64_t d1, int64_t d2,
                   int box1);
// The same of a row-major 16-bit [d1][d0] array with boxes of 64 x box1 elements.
bool encode_map_rows(CUtensorMap* m, int dtype, const void* base, int64_t d0, int64_t d1,
                     int box1);
// The weight-gradient kernels on tables already in memory: out[g] = sum over rows i in
// [off[g], off[g + 1]) of x[token(i)]^T dy[i], g < G. dy has `rows` rows; no group's sum reads a row
// of another's, whatever it holds (the form with TMA copies does, against zeros of x).
int run_dw_tables(const void* x, const void* dy, const int64_t* off, const RowInfo* rowinfo,
                  WsHeader* hdr, int64_t rows, int64_t N, int64_t K, int64_t G, int64_t batch,
                  int dtype, void* out, cudaStream_t stream);

// ------------------------------------------------------------ limits

constexpr int64_t kMaxRouteExperts = 1024;  // a token's logits sit in one warp's registers
constexpr int64_t kMaxRouteTopK = 32;       // one lane per choice
constexpr int64_t kMaxAdapters = 1023;      // + the group of tokens without one: one thread each
constexpr int64_t kMaxRank = 256;
constexpr int kRowPad = 128;  // rows of the factors' gradients reduced at a time

// ------------------------------------------------------------ router

struct RouteArgs {
  const void* logits;   // [T, G]
  const float* bias;    // [G] or null
  float* probs;         // [T, k]
  int64_t* experts;     // [T, k]
  int64_t* idx;         // [T * k]
  int64_t* groups;      // [G]
  uint32_t* counts;     // [G][blocks]: entries of each block per expert, then their prefix sums
  uint32_t* rank;       // [T * k] rank of a pair among its block's pairs of its expert
  WsHeader* hdr;
  int64_t T;
  float scale;
  int32_t G, k;
  int32_t row_idx_type;
  int32_t sigmoid, renormalize;
  int32_t bias_on_score;     // (with a bias) the choice goes by score + bias, not logit + bias
  int32_t blocks;            // blocks of the choice and placement launches
  int32_t tokens_per_block;  // tokens of each
};

struct RouteGradArgs {
  const float* d_probs;    // [T, k]
  const void* logits;      // [T, G]
  const int64_t* experts;  // [T, k]
  void* d_logits;          // [T, G]
  int64_t T;
  float scale;
  int32_t G, k;
  int32_t sigmoid, renormalize;
};

// counts [G][blocks] -> their exclusive prefix sums over the blocks, and the totals.
cudaError_t launch_count_scan(uint32_t* counts, int G, int blocks, int64_t* groups,
                              cudaStream_t stream);
void route_blocks(int64_t T, int64_t G, int64_t k, int* blocks, int* tokens_per_block);
cudaError_t launch_route(int dtype, const RouteArgs& a, cudaStream_t stream);
cudaError_t launch_route_scores(int dtype, const RouteArgs& a, cudaStream_t stream);  // (bias_on_score)
cudaError_t launch_route_place(const RouteArgs& a, cudaStream_t stream);
cudaError_t launch_route_grad(int dtype, const RouteGradArgs& a, int num_sms, cudaStream_t stream);

// ------------------------------------------------------------ tables of the gated product

struct RowsPrepArgs {
  const int64_t* idx;     // expandedRowIdx [M]
  const int64_t* groups;  // groupList [G]
  WsHeader* hdr;
  int4* rblist;      // {expert, first row, rows, 0}
  RowInfo* rowinfo;  // [M] {token, original position} of each expanded row
  int32_t* inv;      // [M]
  int64_t M, G;
  int32_t top_k, row_idx_type, rows_per_block;
  int32_t even = 0;  // 1: a group's rows in blocks of like size, a multiple of 16 rows
  uint32_t* clear = nullptr;  // words that the launch sets to 0
  int32_t n_clear = 0;
};
cudaError_t launch_rows_prep(const RowsPrepArgs& a, int num_sms, cudaStream_t stream);

// ------------------------------------------------------------ tables of the adapters

// Tokens are put in order of their adapter (stable; tokens without one are group A). The groups
// stand in the order of their first token (by_first), so that a batch of requests one after
// another stays as it is and its rows can be copied in boxes; or in the order of their ids (the
// weight-gradient kernels that take off[] need that). That compact order of T rows is what the
// projection walks. The low-rank factors u and v are stored in a second order, in which
// (padded = 1) every group starts at a multiple of kRowPad rows and is filled up with zero rows: the
// reduction over an adapter's rows (rows_outer.cu) reads that many at a time, and what it reads past
// them must not be another adapter's. (The rows of x and d_y that meet them there read as zeros.)
struct AdapterTables {
  WsHeader* hdr;
  int64_t* off;       // [A + 1] first row of each group in the order of u and v, groups by id
  int4* range;        // [A + 1] {first compact row, rows, first row of u, 0} by id
  RowInfo* order;     // [T] compact order: {token, adapter}
  int4* rblist;       // {adapter, first compact row, rows, first row of u}: at most rb rows each
  int4* segs;         // {adapter, first compact row, end, first row of u} of each live adapter
  int32_t* box;       // [2 ceil(T / 256)] first token of each 128 compact rows if they are neighbours
                      // in token order, else -1
  int2* blkseg;       // [ceil(T / 256)] {first segment, segments} of each 256 compact rows
  uint32_t* counts;   // [A + 1][blocks], for many tokens
};

struct AdapterPrepArgs {
  const int64_t* adapter;  // [T]
  AdapterTables t;
  int64_t T;
  int32_t A;
  int32_t rb;      // rows per entry of rblist, a divisor of kRowPad when padded
  int32_t padded, by_first;
  int32_t blocks, tokens_per_block;  // of the counting and placement launches
};
void adapter_blocks(int64_t T, int* blocks, int* tokens_per_block);
cudaError_t launch_adapter_prep(const AdapterPrepArgs& a, cudaStream_t stream);

// ------------------------------------------------------------ products over ragged rows

enum RowsMode {
  kGated = 0,    // h and gate_up from x [batch, K] and weight [G, K, 2F]
  kShrink = 1,   // u [rows, R] = scale[ad] * x a[ad], a [A, K, R]
  kAdapt = 2,    // y [T, N] = x W + u b[ad]^T, W [K, N], b [A, N, R]
  kAdaptT = 3,   // the same with W given as [N, K]: the gradient of x
};

// How the low-rank rows u and v are stored between the product that writes them and the one that
// reads them. They are sums, and the tensor cores read 16-bit operands: one rounding to 16 bits there
// would be as large as the output's own (the factors' gradients of 8192 tokens lay 1.4 times as far
// from the 64-bit values). So a 16-bit call on the tensor cores keeps each value as the sum of two
// (split16 in pgg_ops_mma.cuh) and multiplies with both: at most 2^-16 of u is lost in bf16, 2^-21
// of it or 2^-25 in fp16. It costs 1.5% at rank 32 (8191 tokens, 24 adapters, K = N = 4096: 191 -> 195
// us), 5 to 8% at ranks of 64 and more, where it takes more low-rank steps.
enum LowRankForm {
  kLowRounded = 0,  // [rows, R] of the dtype (fp32 calls; the weight-gradient kernels' operand)
  kLowSplit = 1,    // [rows, low_width(R)]: for each 32 ranks 32 hi, then 32 lo
  kLowFloat = 2,    // [rows, R] fp32, for the FP32 pipes
};
#ifdef __CUDACC__
#define PGG_HOST_DEVICE __host__ __device__
#else
#define PGG_HOST_DEVICE
#endif
PGG_HOST_DEVICE constexpr int64_t low_width(int64_t R) { return (R + 31) / 32 * 64; }

struct RowsArgs {
  const void* x;           // rows gathered by token, K elements each
  const void* w;           // kGated [G, K, 2 N]; kShrink [G, K, N]; kAdapt [K, N]; kAdaptT [N, K]
  const void* u;           // kAdapt*: low-rank rows, scale applied, stored as low_form says
  const void* b;           // kAdapt*: [A, N, R]
  const float* probs;      // kGated: [M] weight of each original position, or null
  const float* scale;      // kShrink: [A] or null
  const int4* rblist;      // row blocks (kAdapt*: of the FP32-pipe kernel only)
  const RowInfo* rowinfo;  // kGated {token, position}; else {token, adapter}
  const int4* segs;        // kAdapt*
  const int2* blkseg;      // kAdapt*
  const int4* range;       // kShrink, padded: see AdapterTables
  const int32_t* box;      // kAdapt*
  WsHeader* hdr;
  void* out;               // h [M, N], u (as low_form says), y [T, N] (rows in token order)
  void* gate_up;           // kGated: [M, 2 N] or null
  int64_t M, N, K, G, batch, max_row_blocks;
  int32_t R;
  int32_t n_blocks;
  int32_t low_form;        // LowRankForm of u: kShrink writes it, kAdapt* reads it
  int32_t padded;          // kShrink, split: fill up an adapter's rows with zeros to a multiple of kRowPad
  const int64_t* adapter;  // few tokens: [T]; u is fp32 in token order then
  int32_t early, late;     // see launch_order in pgg_ops_mma.cuh
  int32_t hold_release;
  uint64_t wait_limit_ns;
};

// Rows of zeros behind a row block of an adapter (none but behind its last).
#ifdef __CUDACC__
__device__ __forceinline__ int rows_to_fill(const RowsArgs& a, const int4& block) {
  const int4 r = a.range[block.x];
  if (block.y + block.z != r.x + r.y) return 0;
  return (r.y + kRowPad - 1) / kRowPad * kRowPad - r.y;
}
#endif

cudaError_t launch_rows_simt(int dtype, RowsMode mode, RowsArgs a, int num_sms,
                             cudaStream_t stream);

// Tensor cores, many rows per group (16-bit, every width a multiple of 8, 16-byte aligned).
cudaError_t launch_rows_wide(int dtype, RowsMode mode, RowsArgs a, int64_t live_blocks,
                             int num_sms, cudaStream_t stream);
int rows_wide_block();

// Tensor cores, at most NR rows per block (kGated 16, 32, 64, 128; kShrink 16, 64; kAdapt 16, 32, 64).
cudaError_t launch_rows_skinny(int dtype, RowsMode mode, int NR, RowsArgs a, int64_t live_blocks,
                               int num_sms, cudaStream_t stream);

// Few tokens: u [T, R] fp32 in token order (R and K multiples of 8), and the ids' check.
cudaError_t launch_few_shrink(int dtype, const RowsArgs& a, cudaStream_t stream);

// Both factors' gradients, for tables in the padded order (16-bit, u and v split, widths multiples
// of 8, 16-byte aligned): out[w] [A, cols[w], R] = sum over an adapter's rows of left[w]^T right[w].
struct OuterArgs {
  const void* left[2];   // x [T, cols[0]], d_y [T, cols[1]]: rows by token
  const void* right[2];  // v, u [right_rows, low_width(R)]: rows in the padded order
  void* out[2];
  const int4* range;     // [A + 1]
  const RowInfo* order;
  WsHeader* hdr;
  int64_t cols[2];
  int64_t T, right_rows;
  int32_t A, R;
  int32_t blocks0, blocks1;  // 128-column blocks of each (set by the launch)
  uint32_t r_blocks;
  int32_t late;            // see launch_order in pgg_ops_mma.cuh
  int32_t hold_release;
  uint64_t wait_limit_ns;
};
cudaError_t launch_rows_outer(int dtype, OuterArgs a, int num_sms, cudaStream_t stream);

// ------------------------------------------------------------ gradient of the gate

struct GatedGradArgs {
  const void* d_h;      // [M, F]
  const void* gate_up;  // [M, 2F]
  const float* probs;   // [M] by original position, or null
  const int64_t* idx;   // [M]
  WsHeader* hdr;
  void* d_gate_up;      // [M, 2F]
  void* h;              // [M, F] or null
  float* d_probs;       // [M] by original position, or null
  int64_t M, F;
  int32_t row_idx_type;
};
cudaError_t launch_gated_grad(int dtype, const GatedGradArgs& a, bool vec, int num_sms,
                              cudaStream_t stream);
cudaError_t launch_index_prep(const int64_t* idx, int64_t M, int row_idx_type, int32_t* inv,
                              WsHeader* hdr, int num_sms, cudaStream_t stream);

}  // namespace pgg
