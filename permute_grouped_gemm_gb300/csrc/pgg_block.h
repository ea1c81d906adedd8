// Internal definitions of what surrounds the experts' products in a block:
// products with 4-bit weights, the norms before and after the block, and the
// gradients' global norm.
#pragma once

#include "pgg_ops.h"

namespace pgg {

// ------------------------------------------------------------ 4-bit experts

struct W4Args {
  const void* x;         // [batch, K] by token, or (combined) [M, K] in expanded order
  const uint8_t* codes;  // [G, C, ceil(K / 2)], C = N, gated: 2 N columns
  const void* scales;    // [G, C, groups]
  const uint8_t* zeros;  // [G, C, groups] or null (8)
  const float* probs;    // gated: [M] weight of each original position, or null
  const int4* rblist;    // {expert, first row, rows, 0}
  const RowInfo* rowinfo;  // {token, original position}
  WsHeader* hdr;
  void* out;             // [M, N], expanded order; combined: fp32 [M, N] by original position
  int64_t M, N, K, G, batch, max_row_blocks;
  int64_t row_bytes;     // ceil(K / 2)
  int32_t group, groups;  // codes of a scale, scales of a row
  int32_t product;       // pgg_w4_product
  int32_t scale_f32;     // scales are fp32 (else the dtype)
  int32_t out_f32;       // out is fp32 (else the dtype)
  // of the streaming kernel
  void* packed;          // the row blocks' rows of x in the products' order
  int32_t* exponent;     // [row blocks][rows of a block] their powers of two
  int32_t* col_exponent; // (wide) [G][C] the columns' powers of two
  int32_t block_rows;    // (wide) most rows of a block (set by the launch)
  int4* meta;            // (wide) of each packed row: {output row or -1, power of two, weight, 0}
  float* parts;          // [2 kW4Grid][rows of a block][128] sums of the tiles that CTAs share
  uint32_t* arrived;     // [kW4Grid] parts of the tile that begins in a CTA; zeros at the start
  int32_t n_blocks;      // blocks of columns (set by the launch)
  int32_t bf16;          // the dtype is bf16 (set by the launch)
  int32_t pairs;         // two neighbouring outputs are one aligned word
  uint64_t wait_limit_ns;
};

constexpr int kW4Grid = 304;  // most CTAs of the streaming kernel: two an SM

int64_t w4_packed_bytes(int64_t row_blocks, int rows_per_block, int64_t K);
// 16-bit, K and group multiples of 32, x and codes 16-byte aligned; blocks of 8, 16 or 32 rows.
cudaError_t launch_w4_stream(int dtype, int rows_per_block, W4Args a, int num_sms,
                             cudaStream_t stream);

cudaError_t launch_w4_simt(int dtype, const W4Args& a, int num_sms, cudaStream_t stream);
// out[b] = sum over j of rows[b * top_k + j] in fp32, zeros when the status word is set.
cudaError_t launch_w4_combine(const float* rows, const WsHeader* hdr, int64_t batch, int64_t top_k,
                              int64_t N, float* out, int num_sms, cudaStream_t stream);

// Most rows of a block of the tensor-core kernel; where its weights are the sum of two.
constexpr int kW4WideRows = 160, kW4SplitRows = 128;
int w4_wide_rows(int dtype, bool scale_f32, bool zeros);  // which
int64_t w4_packed_wide_rows(int64_t M, int64_t row_blocks);
int64_t w4_packed_wide_bytes(int64_t M, int64_t row_blocks, int64_t K);
// The same tensors, many rows an expert: row blocks of up to w4_wide_rows rows.
cudaError_t launch_w4_wide(int dtype, W4Args a, const int64_t* group_list, int num_sms,
                           cudaStream_t stream);

// ------------------------------------------------------------ norms around a block

struct NormArgs {
  const void* x;     // [T, H]; backward: r, the forward's output, or null without a pre norm
  const void* y;     // [T, H] or null
  const void* gate;  // as gate_kind says
  const void* w_post;
  const void* b_post;
  const void* w_pre;
  const void* b_pre;
  void* r;           // forward: [T, H] or null;  backward: d_x
  void* h;           // forward: [T, H] or null;  backward: d_y or null
  // backward
  const void* d_r;   // [T, H] or null
  const void* d_h;   // [T, H] or null
  void* d_gate;      // full: [T, H] of the parameters' dtype; token: fp32 [T]; channel: fp32 [H]
  float* d_cols[5];  // fp32 [H] or null: gate (channel), w_post, b_post, w_pre, b_pre
  float* partial;    // [blocks][5][H]
  WsHeader* hdr;
  int64_t T, H;
  int32_t post, pre;       // pgg_norm
  int32_t gate_kind;       // pgg_gate
  int32_t y_f32, p_f32, dh_f32;  // fp32 (else the dtype)
  float residual_scale, weight_offset, eps;
};

// Columns' sums that a block of the backward keeps, in the order of d_cols.
enum { kColGate, kColWPost, kColBPost, kColWPre, kColBPre, kNormCols };

// Blocks whose column sums the backward keeps apart.
int64_t norm_grad_blocks(int64_t T, int64_t H);
// words: bytes of a vector of the dtype that all rows allow: 16, 4, or 0 (element by element).
cudaError_t launch_block_norm(int dtype, const NormArgs& a, int words, int num_sms,
                              cudaStream_t stream);
cudaError_t launch_block_norm_grad(int dtype, const NormArgs& a, int words, cudaStream_t stream);
// Rows of 16-byte vectors that fit a block's threads: false, and nothing launched, where they do not.
bool launch_block_norm_rows(int dtype, const NormArgs& a, int words, int num_sms,
                           cudaStream_t stream, cudaError_t* err);
bool launch_block_norm_rows_grad(int dtype, const NormArgs& a, int words, cudaStream_t stream,
                                cudaError_t* err);

// ------------------------------------------------------------ the gradients' norm

constexpr int kClipTensors = 512;    // tensors of one launch
constexpr int kClipBlocks = 1024;    // most blocks, and partial sums, of one

struct ClipTable {
  const void* in[kClipTensors];
  void* out[kClipTensors];
  int64_t n[kClipTensors];
  uint32_t first[kClipTensors + 1];  // first chunk of each; behind the last, all chunks
  uint8_t dtype[kClipTensors];
  int32_t tensors;
};

// One partial sum of squares a block into partial[0, blocks).
int64_t clip_chunks(int64_t n, int dtype);  // chunks of a tensor of n elements
cudaError_t launch_clip_squares(const ClipTable& t, WsHeader* hdr, double* partial, int blocks,
                                cudaStream_t stream);
// norm = |scale| sqrt(sum of partial), in fp32.
cudaError_t launch_clip_norm(const double* partial, int64_t count, float scale, float* norm,
                             cudaStream_t stream);
// The norm as above, and out = in * c, c = scale min(1, max_norm / (norm + eps)) (scale alone if norm
// is not finite).
cudaError_t launch_clip_apply(const ClipTable& t, const double* partial, int64_t count,
                              float max_norm, float eps, float scale, float* norm, int blocks,
                              cudaStream_t stream);

}  // namespace pgg
