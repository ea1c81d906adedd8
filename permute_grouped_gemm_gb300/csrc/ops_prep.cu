// Preparation launches of the gated product and of the adapters: the tables
// that the products walk, and the validation of what the caller gave.
//
// Gated product (rows_prep): the row blocks of every expert from groupList,
// {token, original position} of every expanded row from expandedRowIdx, and
// the checks that groupList sums to M and expandedRowIdx is a permutation.
// Few rows: one block, one launch (a bit per position finds a repetition).
// Many: two launches (the inverse is written, then compared).
//
// Adapters (adapter_prep): a stable counting sort of the tokens by adapter
// (tokens without one last), the list of live adapters, which of them each 256
// rows meet, and the row blocks of the low-rank factors. Up to kSmallTokens
// tokens one cluster of eight blocks does it, an eighth of the tokens each, with
// the counts exchanged through distributed shared memory (one block alone took
// 13 us for 8192 tokens: the matches inside 32 keys are what it waits for);
// beyond that counting, prefix sums, the lists, placement and the search for
// neighbouring rows are five launches.
//
// All of it is integer work on a few bytes per row: latency is what it costs,
// so what counts is the number of launches.

#include <cstdint>

#include "pgg_ops.h"
#include "pgg_ops_cluster.cuh"
#include "pgg_ops_launch.h"
#include "pgg_ptx.cuh"
#include "pgg_sort.cuh"

namespace pgg {
namespace {

constexpr int kSmallRows = 8192;     // gated product: one block up to here
constexpr int kSmallGroups = 4096;
constexpr int64_t kSmallTokens = 65536;  // adapters: one cluster up to here
constexpr int kCluster = 8;

__device__ __forceinline__ RowInfo row_info(int64_t p, int top_k) {
  RowInfo r;
  r.token = static_cast<int32_t>(static_cast<uint32_t>(p) / static_cast<uint32_t>(top_k));
  r.rank = static_cast<int32_t>(p);
  return r;
}

// The whole block: expert offsets and row blocks; returns whether groupList is
// right. Writes n_row_blocks (0 when it is not).
__device__ bool build_row_blocks(const RowsPrepArgs& a) {
  __shared__ uint32_t s_scan[33];
  __shared__ int s_bad;
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  // 64-bit sum of the counts beside the 32-bit scan: counts are at most M < 2^31
  // each, so a wrong list is noticed before a scan could wrap
  __shared__ unsigned long long s_sum;
  if (threadIdx.x == 0) s_sum = 0;
  __syncthreads();
  for (int64_t g = threadIdx.x; g < a.G; g += blockDim.x) {
    const int64_t c = a.groups[g];
    if (c < 0 || c > a.M)
      s_bad = 1;
    else
      atomicAdd(&s_sum, static_cast<unsigned long long>(c));
  }
  __syncthreads();
  const bool ok = !s_bad && s_sum == static_cast<unsigned long long>(a.M);
  uint32_t rows = 0, blocks = 0;
  for (int64_t g0 = 0; ok && g0 < a.G; g0 += blockDim.x) {
    const int64_t g = g0 + threadIdx.x;
    const uint32_t c = g < a.G ? static_cast<uint32_t>(a.groups[g]) : 0u;
    uint32_t rpb = static_cast<uint32_t>(a.rows_per_block);
    uint32_t nb = (c + rpb - 1) / rpb;
    if (a.even && nb > 1) {  // (never more blocks than of full size)
      rpb = ((c + nb - 1) / nb + 15) / 16 * 16;
      nb = (c + rpb - 1) / rpb;
    }
    uint32_t tot_c, tot_b;
    const uint32_t row0 = rows + block_scan_u32(c, s_scan, &tot_c);
    const uint32_t b0 = blocks + block_scan_u32(nb, s_scan, &tot_b);
    for (uint32_t j = 0; j < nb; ++j) {
      const uint32_t left = c - j * rpb;
      a.rblist[b0 + j] = make_int4(static_cast<int>(g), static_cast<int>(row0 + j * rpb),
                                   static_cast<int>(left < rpb ? left : rpb), 0);
    }
    rows += tot_c;
    blocks += tot_b;
  }
  for (int i = threadIdx.x; i < a.n_clear; i += blockDim.x) a.clear[i] = 0;
  if (threadIdx.x == 0) {
    a.hdr->n_row_blocks = blocks;
    a.hdr->sched_next = 0;
    a.hdr->timeout_site = 0;
    a.hdr->unsorted = 0;
  }
  return ok;
}

__global__ void __launch_bounds__(1024) rows_prep_small_kernel(const RowsPrepArgs a) {
  __shared__ uint32_t s_seen[kSmallRows / 32];
  __shared__ uint32_t s_status;
  ptx::griddep_wait();
  const int M = static_cast<int>(a.M);
  for (int i = threadIdx.x; i < (M + 31) / 32; i += blockDim.x) s_seen[i] = 0;
  if (threadIdx.x == 0) s_status = 0;
  const bool ok = build_row_blocks(a);  // (has barriers)
  for (int q = threadIdx.x; q < M; q += blockDim.x) {
    const int64_t v = a.idx[q];
    if (v < 0 || v >= a.M) {
      atomicCAS(&s_status, 0u, kStIndex);
      continue;
    }
    const uint32_t bit = 1u << (v & 31);
    if (atomicOr(&s_seen[v >> 5], bit) & bit) atomicCAS(&s_status, 0u, kStNotPerm);
    const int64_t row = a.row_idx_type == 0 ? q : v;
    const int64_t pos = a.row_idx_type == 0 ? v : q;
    a.rowinfo[row] = row_info(pos, a.top_k);
  }
  __syncthreads();
  if (threadIdx.x == 0) a.hdr->status = ok ? s_status : kStGroupSum;
}

// Many rows, first launch: block 0 builds the row blocks, the others the rows'
// records and the inverse index.
__global__ void __launch_bounds__(512) rows_prep_fill_kernel(const RowsPrepArgs a) {
  ptx::griddep_wait();
  if (blockIdx.x == 0) {
    const bool ok = build_row_blocks(a);
    if (threadIdx.x == 0) a.hdr->status = ok ? 0u : kStGroupSum;
    return;
  }
  const int64_t stride = static_cast<int64_t>(gridDim.x - 1) * blockDim.x;
  for (int64_t q = static_cast<int64_t>(blockIdx.x - 1) * blockDim.x + threadIdx.x; q < a.M;
       q += stride) {
    const int64_t v = a.idx[q];
    if (v < 0 || v >= a.M) {
      // the record stays readable: whoever reads it before the status is seen is in bounds
      if (a.row_idx_type == 0) a.rowinfo[q] = row_info(0, a.top_k);
      continue;
    }
    a.inv[v] = static_cast<int32_t>(q);
    const int64_t row = a.row_idx_type == 0 ? q : v;
    const int64_t pos = a.row_idx_type == 0 ? v : q;
    a.rowinfo[row] = row_info(pos, a.top_k);
  }
}

// Second launch: every entry must find itself in the inverse. (What earlier
// calls left in inv cannot pass for this call's: inv[idx[q]] was written by
// this call, by q or by another entry with the same value.)
__global__ void __launch_bounds__(512) rows_prep_check_kernel(const RowsPrepArgs a) {
  ptx::griddep_wait();
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t q = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; q < a.M;
       q += stride) {
    const int64_t v = a.idx[q];
    if (v < 0 || v >= a.M)
      atomicCAS(&a.hdr->status, 0u, kStIndex);
    else if (a.inv[v] != q)
      atomicCAS(&a.hdr->status, 0u, kStNotPerm);
  }
}

// ------------------------------------------------------------------ adapters

// Key of a token: its adapter, A without one; an id outside [-1, A) counts as none.
__device__ __forceinline__ int adapter_key(int64_t id, int A) {
  return id >= 0 && id < A ? static_cast<int>(id) : A;
}

// Block-wide, blockDim.x > A (one thread per adapter and one for the group without): the lists
// from the groups' sizes, into memory if `write`, and s_start (by id) in any case.
// Thread g holds group g's count and first token; s_work is 3 x [A + 1].
__device__ void build_adapter_lists(const AdapterPrepArgs& a, bool write, uint32_t count,
                                    uint32_t first, uint32_t* s_scan, uint32_t* s_start,
                                    uint32_t* s_work) {
  const int G = a.A + 1, g = threadIdx.x;
  const bool group = g < G;
  uint32_t *s_first = s_work, *s_by = s_work + G, *s_end = s_work + 2 * G;
  // place of the group among the groups: its id, or how many have an earlier first token (empty
  // groups last, by id)
  int place = g;
  if (a.by_first) {
    if (group) s_first[g] = count > 0 ? first : 0x80000000u + static_cast<uint32_t>(g);
    __syncthreads();
    if (group) {
      const uint32_t mine = s_first[g];
      place = 0;
      for (int i = 0; i < G; ++i) place += s_first[i] < mine ? 1 : 0;
    }
  }
  if (group) s_by[place] = static_cast<uint32_t>(g) | (count > 0 ? 0x80000000u : 0u);
  if (group) s_start[place] = count;  // (by place for now)
  __syncthreads();
  // from here on thread i stands for the group in place i
  const uint32_t id = group ? s_by[g] & 0x7FFFFFFFu : 0u;
  const uint32_t n = group ? s_start[g] : 0u;
  uint32_t total, n_seg, n_rb;
  const uint32_t start = block_scan_u32(n, s_scan, &total);
  const uint32_t ustart =
      block_scan_u32(a.padded ? (n + kRowPad - 1) / kRowPad * kRowPad : n, s_scan, &total);
  const bool live = group && n > 0 && static_cast<int>(id) < a.A;
  const uint32_t seg = block_scan_u32(live ? 1u : 0u, s_scan, &n_seg);
  const uint32_t nb = (n + a.rb - 1) / a.rb;
  const uint32_t rb0 = block_scan_u32(nb, s_scan, &n_rb);
  if (group) s_start[id] = start;
  if (write) {
    if (group) {
      a.t.off[id] = ustart;
      a.t.range[id] = make_int4(static_cast<int>(start), static_cast<int>(n),
                                static_cast<int>(ustart), 0);
      for (uint32_t j = 0; j < nb; ++j) {
        const uint32_t left = n - j * a.rb;
        a.t.rblist[rb0 + j] = make_int4(
            static_cast<int>(id), static_cast<int>(start + j * a.rb),
            static_cast<int>(left < static_cast<uint32_t>(a.rb) ? left : a.rb),
            static_cast<int>(ustart + j * a.rb));
      }
    }
    if (live) {
      a.t.segs[seg] = make_int4(static_cast<int>(id), static_cast<int>(start),
                                static_cast<int>(start + n), static_cast<int>(ustart));
      s_end[seg] = start + n;
      s_first[seg] = start;
    }
    if (g == 0) a.t.hdr->n_row_blocks = n_rb;
  }
  __syncthreads();
  if (!write) return;
  // segments that rows [256 b, 256 b + 256) meet: they are in row order
  for (int64_t b = threadIdx.x; b < (a.T + 255) / 256; b += blockDim.x) {
    const uint32_t r0 = static_cast<uint32_t>(256 * b);
    const uint32_t r1 = static_cast<uint32_t>(256 * b + 256 < a.T ? 256 * b + 256 : a.T);
    uint32_t lo = 0, hi = n_seg;  // first segment that ends past r0
    while (lo < hi) {
      const uint32_t mid = (lo + hi) >> 1;
      if (s_end[mid] > r0) hi = mid; else lo = mid + 1;
    }
    uint32_t e = lo, top = n_seg;  // first segment from there that starts at r1 or past it
    while (e < top) {
      const uint32_t mid = (e + top) >> 1;
      if (s_first[mid] >= r1) top = mid; else e = mid + 1;
    }
    a.t.blkseg[b] = make_int2(static_cast<int>(lo), static_cast<int>(e - lo));
  }
}

// Record of one sorted token.
__device__ __forceinline__ void put_token(const AdapterPrepArgs& a, int64_t token, int g,
                                          uint32_t where) {
  RowInfo r;
  r.token = static_cast<int32_t>(token);
  r.rank = g;
  a.t.order[where] = r;
}

// Warps w, w + warps, ...: whether each 128 compact rows are neighbours in token order.
__device__ __forceinline__ void find_boxes(const AdapterPrepArgs& a, int64_t w, int64_t warps) {
  const int lane = threadIdx.x & 31;
  for (int64_t b = w; b < 2 * ((a.T + 255) / 256); b += warps) {
    const int64_t r0 = 128 * b;
    const int32_t t0 = r0 < a.T ? a.t.order[r0].token : -1;
    bool same = r0 < a.T;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t r = r0 + lane + 32 * i;
      if (r < a.T) same = same && a.t.order[r].token - t0 == r - r0;
    }
    same = __all_sync(0xFFFFFFFFu, same);
    if (lane == 0) a.t.box[b] = same ? t0 : -1;
  }
}

__global__ void __launch_bounds__(1024) adapter_prep_small_kernel(const AdapterPrepArgs a) {
  // [warps][A + 1] counters, [kCluster][A + 1] counts of every block and their first tokens,
  // 4 x [A + 1], the block's keys
  extern __shared__ uint32_t s_cnt[];
  __shared__ uint32_t s_scan[33];
  __shared__ int s_bad[kCluster];
  cluster_started();
  ptx::griddep_wait();
  const int G = a.A + 1, warps = blockDim.x >> 5;
  const int C = static_cast<int>(gridDim.x), rank = static_cast<int>(blockIdx.x);  // one cluster
  uint32_t* s_all = s_cnt + warps * G;
  uint32_t* s_allf = s_all + kCluster * G;
  uint32_t* s_start = s_all + (a.by_first ? 2 : 1) * kCluster * G;  // (no s_allf otherwise)
  uint32_t* s_work = s_start + G;
  uint16_t* s_key = reinterpret_cast<uint16_t*>(s_work + 3 * G);
  const int64_t t0 = static_cast<int64_t>(rank) * a.tokens_per_block;
  const int64_t left = a.T - t0;
  const int n = left < 0 ? 0
                         : (left < a.tokens_per_block ? static_cast<int>(left)
                                                      : a.tokens_per_block);
  bool bad = false;
#pragma unroll 8
  for (int e = threadIdx.x; e < n; e += blockDim.x) {
    const int64_t id = a.adapter[t0 + e];
    bad = bad || id < -1 || id >= a.A;
    s_key[e] = static_cast<uint16_t>(adapter_key(id, a.A));
  }
  for (int i = threadIdx.x; i < G; i += blockDim.x) s_work[i] = 0xFFFFFFFFu;
  bad = __syncthreads_or(bad);
  for (int e = threadIdx.x; a.by_first && e < n; e += blockDim.x)
    if (e == 0 || s_key[e] != s_key[e - 1])  // (starts of runs are enough)
      atomicMin(&s_work[s_key[e]], static_cast<uint32_t>(t0 + e));
  const int run = ((n + warps - 1) / warps + 31) / 32 * 32;
  auto key = [&](int e) { return static_cast<int>(s_key[e]); };
  sort_count(s_cnt, G, n, run, key);
  const int g = threadIdx.x;
  // every block's counts to every block
  cluster_all_started();
  if (g < G) {
    uint32_t c = 0;
    for (int w = 0; w < warps; ++w) c += s_cnt[w * G + g];
    for (int d = 0; d < C; ++d) {
      st_cluster_u32(ptx::mapa(&s_all[rank * G + g], d), c);
      if (a.by_first) st_cluster_u32(ptx::mapa(&s_allf[rank * G + g], d), s_work[g]);
    }
  }
  if (g == 0) st_cluster_u32(ptx::mapa(&s_bad[rank], 0), bad ? 1u : 0u);
  ptx::cluster_sync();
  uint32_t c = 0, mine = 0, first = 0xFFFFFFFFu;
  if (g < G) {
    for (int d = 0; d < C; ++d) {
      if (d == rank) mine = c;
      c += s_all[d * G + g];
      if (a.by_first && s_allf[d * G + g] < first) first = s_allf[d * G + g];
    }
  }
  build_adapter_lists(a, rank == 0, c, first, s_scan, s_start, s_work);
  __syncthreads();
  sort_place(
      s_cnt, G, n, run, key, [&](int k) { return s_start[k] + mine; },
      [&](int e, uint32_t where) { put_token(a, t0 + e, key(e), where); });
  ptx::cluster_sync();  // every block's part of the order is there
  find_boxes(a, rank * warps + (threadIdx.x >> 5), static_cast<int64_t>(C) * warps);
  if (rank == 0 && threadIdx.x == 0) {
    int any = 0;
    for (int d = 0; d < C; ++d) any |= s_bad[d];
    a.t.hdr->status = any ? kStIndex : 0u;
    a.t.hdr->sched_next = 0;
    a.t.hdr->timeout_site = 0;
    a.t.hdr->unsorted = 0;
  }
}

constexpr int kSortThreads = 256;

// Many tokens, first launch: the block's count of every adapter.
__global__ void __launch_bounds__(kSortThreads) adapter_count_kernel(const AdapterPrepArgs a) {
  extern __shared__ uint32_t s_cnt[];  // [A + 1]
  ptx::griddep_wait();
  const int G = a.A + 1;
  for (int g = threadIdx.x; g < G; g += blockDim.x) s_cnt[g] = 0;
  __syncthreads();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens_per_block;
  const int64_t t1 = t0 + a.tokens_per_block < a.T ? t0 + a.tokens_per_block : a.T;
  for (int64_t t = t0 + threadIdx.x; t < t1; t += blockDim.x)
    atomicAdd(&s_cnt[adapter_key(a.adapter[t], a.A)], 1u);
  __syncthreads();
  for (int g = threadIdx.x; g < G; g += blockDim.x)
    a.t.counts[static_cast<int64_t>(g) * a.blocks + blockIdx.x] = s_cnt[g];
}

// Third launch (one block), after the prefix sums: the lists. The totals arrive in off.
__global__ void __launch_bounds__(1024) adapter_lists_kernel(const AdapterPrepArgs a) {
  extern __shared__ uint32_t s_lists[];  // 4 x [A + 1]
  __shared__ uint32_t s_scan[33];
  ptx::griddep_wait();
  const int G = a.A + 1, g = threadIdx.x;
  const uint32_t c = g < G ? static_cast<uint32_t>(a.t.off[g]) : 0u;
  // (groups by id: the first tokens would be one more launch's work)
  build_adapter_lists(a, true, c, 0, s_scan, s_lists, s_lists + G);
  if (g == 0) {
    a.t.hdr->status = 0;
    a.t.hdr->sched_next = 0;
    a.t.hdr->timeout_site = 0;
    a.t.hdr->unsorted = 0;
  }
}

// Fourth launch: placement, and the check of the ids.
__global__ void __launch_bounds__(kSortThreads) adapter_place_kernel(const AdapterPrepArgs a) {
  extern __shared__ uint32_t s_cnt[];  // [warps][A + 1]
  ptx::griddep_wait();
  const int G = a.A + 1;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens_per_block;
  const int64_t left = a.T - t0;
  const int n = left < a.tokens_per_block ? static_cast<int>(left) : a.tokens_per_block;
  constexpr int kW = kSortThreads / 32;
  const int run = ((n + kW - 1) / kW + 31) / 32 * 32;
  auto key = [&](int e) { return adapter_key(a.adapter[t0 + e], a.A); };
  for (int e = threadIdx.x; e < n; e += blockDim.x) {
    const int64_t id = a.adapter[t0 + e];
    if (id < -1 || id >= a.A) atomicCAS(&a.t.hdr->status, 0u, kStIndex);
  }
  sort_count(s_cnt, G, n, run, key);
  sort_place(
      s_cnt, G, n, run, key,
      [&](int g) {
        return static_cast<uint32_t>(a.t.range[g].x) +
               a.t.counts[static_cast<int64_t>(g) * a.blocks + blockIdx.x];
      },
      [&](int e, uint32_t where) { put_token(a, t0 + e, key(e), where); });
}

// Fifth launch.
__global__ void __launch_bounds__(kSortThreads) adapter_boxes_kernel(const AdapterPrepArgs a) {
  ptx::griddep_wait();
  const int64_t per = kSortThreads / 32;
  find_boxes(a, blockIdx.x * per + (threadIdx.x >> 5), gridDim.x * per);
}

}  // namespace

cudaError_t launch_rows_prep(const RowsPrepArgs& a, int num_sms, cudaStream_t stream) {
  if (a.M <= kSmallRows && a.G <= kSmallGroups) {
    int64_t threads = (a.M > a.G ? a.M : a.G);
    threads = (threads + 31) / 32 * 32;
    if (threads > 1024) threads = 1024;
    return launch_pdl(rows_prep_small_kernel, dim3(1), dim3(static_cast<unsigned>(threads)), 0,
                      stream, 1, a);
  }
  int64_t blocks = (a.M + 511) / 512;
  const int64_t cap = static_cast<int64_t>(num_sms) * 4;
  if (blocks > cap) blocks = cap;
  cudaError_t err = launch_pdl(rows_prep_fill_kernel, dim3(static_cast<unsigned>(blocks + 1)),
                               dim3(512), 0, stream, 1, a);
  if (err != cudaSuccess) return err;
  return launch_pdl(rows_prep_check_kernel, dim3(static_cast<unsigned>(blocks)), dim3(512), 0,
                    stream, 1, a);
}

// Blocks of the counting and placement launches, and the tokens of each; at most kCluster blocks:
// one launch, one cluster.
void adapter_blocks(int64_t T, int* blocks, int* tokens_per_block) {
  int64_t n = T <= 512 ? 1 : T <= kSmallTokens ? kCluster : 512;  // (count_scan takes up to 608)
  int64_t per = (T + n - 1) / n;
  if (n > kCluster) per = (per + kSortThreads - 1) / kSortThreads * kSortThreads;
  *tokens_per_block = static_cast<int>(per);
  *blocks = static_cast<int>(n > kCluster ? (T + per - 1) / per : n);
}

cudaError_t launch_adapter_prep(const AdapterPrepArgs& a, cudaStream_t stream) {
  const int G = a.A + 1;
  if (a.blocks <= kCluster) {
    int threads = a.tokens_per_block > G ? a.tokens_per_block : G;
    if (threads > 512) threads = G > 512 ? G : 512;
    threads = (threads + 31) / 32 * 32;
    AdapterPrepArgs q = a;
    if (G > 512) q.by_first = 0;  // (their tables would not fit beside the counters)
    const size_t smem =
        static_cast<size_t>(threads / 32 + (q.by_first ? 2 : 1) * kCluster + 4) * G * 4 +
        static_cast<size_t>(a.tokens_per_block) * 2;
    // the most of it: 1024 threads and groups (by id), and the keys of kSmallTokens / kCluster tokens
    constexpr int kMost =
        (1024 / 32 + kCluster + 4) * static_cast<int>(kMaxAdapters + 1) * 4 +
        static_cast<int>(kSmallTokens / kCluster) * 2;
    static SmemLimit limit;
    const cudaError_t err = allow_smem(&limit, adapter_prep_small_kernel, kMost);
    if (err != cudaSuccess) return err;
    return launch_pdl(adapter_prep_small_kernel, dim3(a.blocks), dim3(threads), smem, stream,
                      static_cast<unsigned>(a.blocks), q);
  }
  cudaError_t err = launch_pdl(adapter_count_kernel, dim3(a.blocks), dim3(kSortThreads),
                               static_cast<size_t>(G) * 4, stream, 1, a);
  if (err != cudaSuccess) return err;
  err = launch_count_scan(a.t.counts, G, a.blocks, a.t.off, stream);
  if (err != cudaSuccess) return err;
  AdapterPrepArgs by_id = a;
  by_id.by_first = 0;
  err = launch_pdl(adapter_lists_kernel, dim3(1), dim3(1024), static_cast<size_t>(4) * G * 4,
                   stream, 1, by_id);
  if (err != cudaSuccess) return err;
  err = launch_pdl(adapter_place_kernel, dim3(a.blocks), dim3(kSortThreads),
                   static_cast<size_t>(kSortThreads / 32) * G * 4, stream, 1, a);
  if (err != cudaSuccess) return err;
  const int64_t per = kSortThreads / 32;  // boxes of a block at a time, a warp each
  const int64_t boxes = (2 * ((a.T + 255) / 256) + per - 1) / per;
  return launch_pdl(adapter_boxes_kernel, dim3(static_cast<unsigned>(boxes < 1024 ? boxes : 1024)),
                    dim3(kSortThreads), 0, stream, 1, a);
}

}  // namespace pgg
