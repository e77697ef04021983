// Arguments and internal entry points of the decode kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace isoq {
namespace decode {

constexpr int kMaxGroup = 16;  // query heads per KV head

// What the split kernels read: one contiguous cache row per (b, kvh)
// (kSplitDense), the same under a sliding window with sink tokens
// (kSplitWindow), cache pages through a block table, also with window and
// sinks (kSplitPaged), or one prefix shared by all batch rows, the query heads
// of every batch row being the query rows of a KV head, followed by each
// row's own cache (kSplitPrefix).
enum SplitMode { kSplitDense = 0, kSplitWindow = 1, kSplitPaged = 2, kSplitPrefix = 3 };

struct SplitArgs {
  const void *q;
  const uint8_t *packed_k;
  const uint8_t *packed_v;
  const uint16_t *norms_k;
  const uint16_t *norms_v;
  const int32_t *seq_lens;
  const float *params_k;
  float *ws_acc;   // [B][Hq][n_splits][d]
  float2 *ws_ml;   // [B][Hq][n_splits] (max, sum)
  uint32_t *ws_qprep;  // [B][Hkv][decode_qprep_words(d)] prepared queries (int8 path)
  long long tmax;
  long long chunk;  // tokens per split
  int batch, hq, hkv, group, n_splits;
  float scale;
  float centroid[16];
  // The modes other than kSplitDense.  A CTA takes one group of query rows:
  // zrow_size heads of one (b, kvh), n_zrows groups for each, or (the first
  // n_zrows_p groups of kSplitPrefix) zrow_size_p of a KV head's batch x group
  // rows over the prefix.
  int n_zrows, zrow_size, n_zrows_p, zrow_size_p;
  int slot_stride, slot_off;   // partial states per query head; the first one over the own cache
  int window, n_sink;      // a decode query sees the last `window` tokens and the first n_sink
  const uint8_t *prefix_k, *prefix_v;      // kSplitPrefix: [Hkv][head_stride][d*bits/8]
  const uint16_t *prefix_nk, *prefix_nv;   // [Hkv][head_stride]
  const int32_t *prefix_len;
  long long head_stride, prefix_max, chunk_p;   // the prefix's room, most tokens and tokens per split
  int n_splits_p;
  const int32_t *block_table;  // kSplitPaged: [B][max_pages] page indices
  int page_shift, max_pages, n_pages;
  float *ws_qrot;          // rotated float32 queries [B][Hq][d] (the CUDA-core split)
  int mode;
  // One launch for everything: a cluster holds the splits of a row group, each
  // CTA prepares its own queries, and the cluster merges the partial states in
  // its shared memory, rotates back and stores (no workspace).
  bool fused, full, half_out;
  const float *params_v;
  void *out;
};

// A page index of a block table outside [0, n_pages), or a slot outside the
// pages (the device error word).
constexpr unsigned kErrBadPage = 8u;
// Block tables: a request that the table or the free list has no room for.
constexpr unsigned kErrTableFull = 16u;

// The query rows of one CTA: heads r0 .. r0 + rows - 1 of batch row `row`, or
// rows r0 .. of a KV head's batch x group over the prefix.
struct RowGroup {
  int row, r0, rows;
  bool prefix;
};

__host__ __device__ inline RowGroup row_group(const SplitArgs &a, int mode, int z) {
  RowGroup g;
  g.prefix = mode == kSplitPrefix && z < a.n_zrows_p;
  const int zz = mode == kSplitPrefix ? z - a.n_zrows_p : z;
  const int size = g.prefix ? a.zrow_size_p : a.zrow_size;
  g.row = g.prefix ? 0 : zz / a.n_zrows;
  g.r0 = (g.prefix ? z : zz % a.n_zrows) * size;
  const int left = (g.prefix ? a.batch * a.group : a.group) - g.r0;
  g.rows = left < size ? left : size;
  return g;
}

// Index [B][Hq] of row h of the group at KV head kvh, and its partial state
// in split `split`.
__host__ __device__ inline long long group_query(const SplitArgs &a, const RowGroup &g, int kvh, int h) {
  const int r = g.r0 + h;
  return g.prefix ? static_cast<long long>(r / a.group) * a.hq + kvh * a.group + r % a.group
                  : static_cast<long long>(g.row) * a.hq + kvh * a.group + r;
}

__host__ __device__ inline long long group_slot(const SplitArgs &a, const RowGroup &g, int kvh, int h, int split) {
  return group_query(a, g, kvh, h) * a.slot_stride + (g.prefix ? 0 : a.slot_off) + split;
}

// Groups of query rows in a launch (the grid's last dimension).
inline int group_count(const SplitArgs &a, int mode) {
  return (mode == kSplitPrefix ? a.n_zrows_p : 0) + a.batch * a.n_zrows;
}

// The 32-token blocks that a decode query at the end of `len` tokens sees, in
// order: blocks [0, n_sink_blocks), then from block `first` on, n_blocks in
// all.  Token j of those blocks is seen if j < len and (j < sink or j >= lo);
// every listed block holds at least one such token.
struct SeenBlocks {
  int len, sink, lo, n_sink_blocks, first, n_blocks;
};

__host__ __device__ inline SeenBlocks seen_blocks(int len, int window, int n_sink) {
  SeenBlocks s;
  s.len = len;
  s.sink = n_sink < len ? n_sink : len;
  s.lo = len > window ? len - window : 0;
  if (s.lo <= s.sink) s.lo = 0;                       // nothing between the sinks and the window
  s.n_sink_blocks = s.lo > 0 ? (s.sink >> 5) + ((s.sink & 31) != 0) : 0;
  s.first = s.lo / 32 > s.n_sink_blocks ? s.lo / 32 : s.n_sink_blocks;
  const int end = (len >> 5) + ((len & 31) != 0);
  s.n_blocks = s.n_sink_blocks + (s.lo < len && end > s.first ? end - s.first : 0);
  return s;
}

// Bit j: token 32 block + j is seen.
__host__ __device__ inline unsigned seen_mask(const SeenBlocks &s, int block) {
  const int t0 = 32 * block;
  auto below = [](int n) { return n <= 0 ? 0u : (n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u); };
  return below(s.len - t0) & (below(s.sink - t0) | ~below(s.lo - t0));
}

struct CombineArgs {
  const float *params_v;
  void *out;
  const float *ws_acc;
  const float2 *ws_ml;
  int batch, hq, group, n_splits;
};

bool i8_path_supported(int dtype, int d, int bits, const SplitArgs &a);
int run_split_i8(int d, int variant, const SplitArgs &a, cudaStream_t stream);
int run_combine(int dtype, int d, int variant, const CombineArgs &a, cudaStream_t st);

}  // namespace decode
}  // namespace isoq
