// Serving attention on the packed cache: decode under a sliding window with
// sink tokens, decode of a batch that shares a prefix, the paged cache (block
// tables, append, decode), and windowed chunked prefill.
//
// Decode runs as query preparation, split and combine, the launches of
// isoq_decode_attention: the integer tensor-core split (decode_i8.cuh) for
// float16 queries and 3-bit codes at d = 128 and 256, the CUDA-core split
// (serve_any.cuh) for everything else.  A split covers a run of the list of
// 32-token blocks that the query sees.  Measured: 32 rows x 4,112 seen tokens,
// 16 query over 8 KV heads, d = 256: 81 us; 16 rows of 8,192 to 16,384 tokens
// through pages of 64: 118 us (16 x 12,288 tokens: 100 us with a window, 113
// through pages, 94 by isoq_decode_attention).

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "tcgen05.cuh"
#include "decode.h"
#include "internal.h"

namespace isoq {
namespace decode {

#include "decode_common.cuh"
#include "decode_i8.cuh"
#include "prefill.cuh"
#include "serve_any.cuh"
#include "paged.cuh"

inline int64_t round256(int64_t n) { return (n + 255) / 256 * 256; }
inline int64_t div_up(int64_t n, int64_t m) { return (n + m - 1) / m; }

// Most 32-token blocks that a decode query sees of a row of up to `tmax`
// tokens.
inline int64_t most_blocks(int64_t tmax, int64_t window, int64_t n_sink) {
  if (window > tmax) window = tmax;
  if (n_sink > tmax) n_sink = tmax;
  const int64_t all = div_up(tmax, 32), near = div_up(window, 32) + 1, sink = div_up(n_sink, 32);
  return near < all && sink < all && near + sink < all ? near + sink : all;
}

#include "rows_tc.cuh"
#include "serve_prefix.cuh"

// ---------------------------------------------------------------------------
// Plans
// ---------------------------------------------------------------------------

// Query heads of one CTA: a KV head's group, or even shares of at most 8.
inline int row_share(int rows) { return static_cast<int>(div_up(rows, div_up(rows, 8))); }

// Tokens per split for `ctas` row groups of up to `tokens` listed tokens each:
// the chunk that minimises the wave model of decode_chunk_tokens (4 CTAs
// resident per SM, k of them moving k / (k + 0.7) of its full rate, a CTA
// costing about 160 tokens' worth of set-up and merge), over finer chunks, down
// to one round of 128 tokens (1 row x 1,028 tokens x 4 KV heads: 10.3 us at
// 128 tokens per split, 16.4 at 512).  Without a window the rows are taken to
// fill three quarters of the longest, ragged as they are (16 rows of 8,192 to
// 16,384 tokens, 8 KV heads: 121 us at 1,024 tokens per split, 134 at the 2,048
// that full rows would suggest).  `slots`: CTAs resident per SM (resident_ctas),
// but 1 at d = 512, where a second CTA adds little (16 rows x 8,192 tokens, 8
// heads, float32, 2 bits: 281 us with the chunk of 1, 302 with that of 2).
template <int64_t C>
inline void weigh_chunk(int64_t ctas, int64_t tokens, bool ragged, int64_t slots, int64_t &best_cost, int64_t &best_chunk) {
  constexpr int64_t kSms = 148, kCtaCost = 160;
  int64_t n = ctas * ((tokens + C - 1) / C);
  if (ragged && tokens > C) n = (3 * n + 3) / 4;
  const int64_t m = (n + kSms - 1) / kSms, full = slots == 4 ? m / 4 : slots == 3 ? m / 3 : slots == 2 ? m / 2 : m;
  const int64_t rest = m - full * slots, phases10 = full * (10 * slots + 7) + (rest ? 10 * rest + 7 : 0);
  const int64_t cost = phases10 * ((C < tokens ? C : tokens) + kCtaCost);
  if (best_cost < 0 || cost < best_cost) {
    best_cost = cost;
    best_chunk = C;
  }
}

// Every candidate with its divisors known to the compiler: the plan is formed
// in each call.
template <int64_t... C>
inline int64_t best_chunk_of(int64_t ctas, int64_t tokens, bool ragged, int64_t slots) {
  int64_t cost = -1, chunk = 0;
  (weigh_chunk<C>(ctas, tokens, ragged, slots, cost, chunk), ...);
  return chunk;
}

inline int64_t serve_chunk(int64_t ctas, int64_t tokens, bool ragged, int64_t slots) {
  return best_chunk_of<4096, 2560, 2048, 1536, 1280, 1024, 896, 768, 640, 512, 384, 256, 128>(ctas, tokens, ragged, slots);
}

struct DecodePlan {
  int share, groups;                 // query heads per CTA, CTAs per (b, kvh)
  int share_p, groups_p;             // the same over the prefix's rows
  int64_t chunk, chunk_p;
  int splits, splits_p;
  int64_t acc_bytes, prep_bytes;     // workspace: partial states; prepared queries
  // The prefix on tcgen05: 128-row tiles per KV head (0: the other splits);
  // at d = 256 the prepared query tiles' place in the workspace.
  int row_tiles;
  int64_t tiles_at;
  bool fused;                        // one launch of clusters, no workspace
};

// CTAs of the split that an SM holds, for `rows` query rows each: of the integer
// split 4, but 3 for 8 rows at d = 128 and 4 rows at d = 256, 2 for 8 rows there;
// of the CUDA-core one 4 at d = 128, 2 or 3 at 256, 1 or 2 at 512.  Measured
// against 4 for every integer split and every cluster, and 2 of the CUDA-core
// one at d = 256: 32 rows x 1,024 tokens, 32 query over 4 KV heads, float16, d =
// 256: 49.3 -> 36.5 us, d = 128: 30.1 -> 25.1; 16 x 512 tokens, 16 over 4,
// float32, 4 bits, d = 512: 39.0 -> 28.9; 16 x 8,192 tokens, 16 over 4, float32,
// 3 bits, d = 256: 149 -> 138; 16 x 12,288, 32 over 4, float16, d = 128: 77.2 ->
// 75.1.
template <int D, int BITS>
constexpr int any_slots(int rows) {
  return rows <= 2 ? AnyCfg<D, BITS, 2>::SLOTS : (rows <= 4 ? AnyCfg<D, BITS, 4>::SLOTS : AnyCfg<D, BITS, 8>::SLOTS);
}

template <int D>
constexpr int any_slots_b(int bits, int rows) {
  return bits == 2 ? any_slots<D, 2>(rows) : (bits == 3 ? any_slots<D, 3>(rows) : any_slots<D, 4>(rows));
}

template <int D>
constexpr int i8_slots(int rows) {
  return rows == 1   ? I8Cfg<D, 1>::MIN_BLOCKS
         : rows == 2 ? I8Cfg<D, 2>::MIN_BLOCKS
         : rows <= 4 ? I8Cfg<D, 4>::MIN_BLOCKS
                     : I8Cfg<D, 8>::MIN_BLOCKS;
}

inline int resident_ctas(bool i8, int d, int bits, int rows) {
  if (i8) return d == 128 ? i8_slots<128>(rows) : i8_slots<256>(rows);
  return d == 128 ? any_slots_b<128>(bits, rows) : (d == 256 ? any_slots_b<256>(bits, rows) : any_slots_b<512>(bits, rows));
}

// Small problems run as one launch: up to 8 splits of a row group form a
// cluster that merges its partial states itself.  Taken where 8 splits of at
// most 16 blocks cover the longest list and all CTAs are resident at once.
// 1 row, 32 query over 4 KV heads, 1,028 tokens: 12.3 us on the GPU against 10.3
// for the three launches, but 5.3 us of host time to queue it against 9.9 (and
// no workspace): with the Python call around it a step of many layers is bound
// by the queueing, 13.4 us a call against 19.2.
constexpr int kFusedSplits = kMaxClusterSplits, kFusedBlocks = 16;

// The rows of a KV head's batch x group from which on the prefix goes to the
// tcgen05 split (float16 queries, 3-bit codes).  Its time hardly depends on the
// rows of a 128-row tile, the integer split's goes with every 8.  Integer and
// tcgen05 split, 4 KV heads, us: d = 128, 8,192 tokens: 8 rows 20.5, 20.5, 16
// rows 22.6, 20.6; 65,536 tokens: 8 rows 39.0, 47.2, 16 rows 63.6, 55.4, 64
// rows 167, 58.6.  d = 256, 8,192 tokens: 16 rows 36.4, 39.0, 32 rows 43.9,
// 41.0; 65,536 tokens: 16 rows 113, 139, 32 rows 201, 142.
constexpr int prefix_tc_rows(int d) { return d == 128 ? 9 : 24; }

// prefix_max < 0: no prefix.  The list of a row is cut into the same splits
// whatever its length.
DecodePlan plan_decode(int B, int Hq, int Hkv, int64_t tmax, int64_t prefix_max, int d, int bits, int64_t window,
                       int64_t n_sink, bool i8, bool prefix_tc = false) {
  DecodePlan p{};
  const int G = Hq / Hkv;
  const int64_t rows = static_cast<int64_t>(B) * G;   // of a KV head, over the prefix
  p.share = row_share(G);
  if (prefix_max >= 0) p.share_p = row_share(static_cast<int>(rows < 8 ? rows : 8));
  const int slots = resident_ctas(i8, d, bits, !prefix_tc && p.share_p > p.share ? p.share_p : p.share);
  p.groups = static_cast<int>(div_up(G, p.share));
  const int64_t tokens = 32 * most_blocks(tmax, window, n_sink);
  if (prefix_max < 0) {
    const int64_t ctas = static_cast<int64_t>(B) * Hkv * p.groups, blocks = tokens / 32, room = slots * 148 / ctas;
    int64_t s = div_up(blocks, 4);
    if (s > kFusedSplits) s = kFusedSplits;
    if (s > room) s = room;
    if (s > 0 && div_up(blocks, s) <= kFusedBlocks) {
      p.fused = true;
      p.chunk = 32 * div_up(blocks, s);
      p.splits = static_cast<int>(div_up(tokens, p.chunk));
      return p;
    }
  }
  const int wave_slots = d == 512 ? 1 : slots;
  p.chunk = serve_chunk(static_cast<int64_t>(B) * Hkv * p.groups, tokens, window >= tmax, wave_slots);
  p.splits = static_cast<int>(div_up(tokens, p.chunk));
  int64_t prep_rows = static_cast<int64_t>(B) * p.groups;
  if (prefix_max >= 0) {
    p.groups_p = static_cast<int>(div_up(rows, p.share_p));
    const int64_t tp = 32 * div_up(prefix_max, 32);
    p.chunk_p = serve_chunk(static_cast<int64_t>(Hkv) * p.groups_p, tp > 0 ? tp : 32, false, wave_slots);
    p.splits_p = static_cast<int>(div_up(tp, p.chunk_p));
    prep_rows += p.groups_p;
    if (prefix_tc) {
      p.row_tiles = static_cast<int>(div_up(rows, kTcRows));
      // Even splits of whole tiles, as many as fill the resident CTAs (one
      // per SM) once.
      const int64_t tok = d == 128 ? kRowsTok : kTcTok, tiles = div_up(prefix_max, tok);
      const int64_t ctas = static_cast<int64_t>(p.row_tiles) * Hkv, slots = 148;
      int64_t splits = slots / ctas > 1 ? slots / ctas : 1;
      if (splits > tiles) splits = tiles;
      const int64_t per = div_up(tiles, splits > 0 ? splits : 1);
      p.chunk_p = tok * per;
      p.splits_p = per > 0 ? static_cast<int>(div_up(tiles, per)) : 0;
    }
  }
  p.acc_bytes = round256(static_cast<int64_t>(B) * Hq * (p.splits + p.splits_p) * (d + 2) * 4);
  p.prep_bytes = round256(i8 ? prep_rows * Hkv * decode_qprep_words(d) * 4 : static_cast<int64_t>(B) * Hq * d * 4);
  p.tiles_at = p.acc_bytes + p.prep_bytes;
  if (d == 256) p.prep_bytes += static_cast<int64_t>(p.row_tiles) * Hkv * TcCfg<256>::Q_TILE;
  return p;
}

// The most that any of these shapes' plans needs: which one runs also depends
// on types, bits and alignment (the tcgen05 prefix has 3 bits).
size_t most_workspace(int B, int Hq, int Hkv, int64_t tmax, int64_t prefix_max, int d, int64_t window, int64_t n_sink) {
  int64_t need = 0;
  auto weigh = [&](int bits, bool i8, bool prefix_tc) {
    const DecodePlan p = plan_decode(B, Hq, Hkv, tmax, prefix_max, d, bits, window, n_sink, i8, prefix_tc);
    need = p.acc_bytes + p.prep_bytes > need ? p.acc_bytes + p.prep_bytes : need;
  };
  for (int tc = 0; tc < (prefix_max >= 0 ? 2 : 1); ++tc) {
    weigh(3, false, tc);
    if (d != 512) weigh(3, true, tc);
  }
  if (d != 128) {   // (d = 128: as 3 bits)
    weigh(2, false, false);
    weigh(4, false, false);
  }
  return static_cast<size_t>(need);
}

// ---------------------------------------------------------------------------
// Checks and launches
// ---------------------------------------------------------------------------

int check_decode(int dtype, int B, int Hq, int Hkv, int64_t tmax, int d, int bits, int variant, int64_t window,
                 int64_t n_sink, float scale) {
  if (!supported_d(d)) return set_error(ISOQ_ERR_UNSUPPORTED, "d=%d not supported", d);
  if (!supported_bits(bits)) return set_error(ISOQ_ERR_UNSUPPORTED, "bits=%d not supported", bits);
  if (!supported_decode_variant(variant)) return set_error(ISOQ_ERR_UNSUPPORTED, "variant=%d", variant);
  if (!supported_dtype(dtype)) return set_error(ISOQ_ERR_UNSUPPORTED, "dtype=%d", dtype);
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || tmax <= 0)
    return set_error(ISOQ_ERR_INVALID_ARG, "B, Hq, Hkv and the longest row must be positive");
  if (Hq % Hkv) return set_error(ISOQ_ERR_INVALID_ARG, "Hq %% Hkv != 0");
  if (Hq / Hkv > kMaxGroup) return set_error(ISOQ_ERR_UNSUPPORTED, "Hq/Hkv > %d", kMaxGroup);
  if (tmax >= (1ll << 31) || B > 16000 || Hkv > 65535 || Hq > (1 << 24))
    return set_error(ISOQ_ERR_INVALID_ARG, "shape too large");
  if (window < 0 || n_sink < 0) return set_error(ISOQ_ERR_INVALID_ARG, "window and n_sink must not be negative");
  if (!std::isfinite(scale)) return set_error(ISOQ_ERR_INVALID_ARG, "scale is not finite");
  return ISOQ_OK;
}

int check_workspace(const void *ws, size_t bytes, size_t need) {
  if (need == 0) return ISOQ_OK;
  if (!ws) return set_error(ISOQ_ERR_INVALID_ARG, "workspace is NULL");
  if (!aligned(ws, 256)) return set_error(ISOQ_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (bytes < need) return set_error(ISOQ_ERR_INVALID_ARG, "workspace too small: %zu < %zu", bytes, need);
  return ISOQ_OK;
}

// The page size's logarithm; -1: not a power of two from 16 to 256.
int page_shift_of(int page_tokens) {
  for (int s = 4; s <= 8; ++s)
    if (page_tokens == 1 << s) return s;
  return -1;
}

inline int clamp31(int64_t n) { return n > 0x7FFFFFFF ? 0x7FFFFFFF : static_cast<int>(n); }

template <int D, bool FULL, int GP>
int run_i8_mode(const SplitArgs &a, cudaStream_t st) {
  if (a.mode == kSplitPaged) return launch_split_i8<D, FULL, GP, kSplitPaged>(a, st);
  if (a.mode == kSplitPrefix) return launch_split_i8<D, FULL, GP, kSplitPrefix>(a, st);
  return launch_split_i8<D, FULL, GP, kSplitWindow>(a, st);
}

template <int D, bool FULL>
int run_i8_rows(const SplitArgs &a, cudaStream_t st) {
  const int rows = a.mode == kSplitPrefix && a.zrow_size_p > a.zrow_size ? a.zrow_size_p : a.zrow_size;
  if (rows == 1) return run_i8_mode<D, FULL, 1>(a, st);
  if (rows == 2) return run_i8_mode<D, FULL, 2>(a, st);
  if (rows <= 4) return run_i8_mode<D, FULL, 4>(a, st);
  return run_i8_mode<D, FULL, 8>(a, st);
}

bool i8_split(int dtype, int d, int bits) { return dtype == ISOQ_F16 && bits == 3 && (d == 128 || d == 256); }

// The bulk copies of the integer split start on 16-byte boundaries: rows of
// a multiple of 8 tokens, norms aligned to 16 bytes.
bool i8_cache(const uint16_t *nk, const uint16_t *nv, int64_t room) {
  return room % 8 == 0 && aligned(nk, 16) && aligned(nv, 16);
}

// Preparation, split and combine over the partial states in `workspace`.
int run_decode(SplitArgs &a, const DecodePlan &p, int dtype, int d, int bits, int variant, bool i8, const float *params_v,
               void *out, void *workspace, cudaStream_t st) {
  variant = block_map_variant(variant);
  a.group = a.hq / a.hkv;
  a.n_splits = p.splits;
  a.n_splits_p = p.splits_p;
  a.slot_stride = p.splits + p.splits_p;
  a.slot_off = p.splits_p;
  a.chunk = p.chunk;
  a.chunk_p = p.chunk_p;
  a.fused = p.fused;
  a.full = variant == ISOQ_FULL;
  a.half_out = dtype == ISOQ_F16;
  a.params_v = params_v;
  a.out = out;
  a.zrow_size = p.share;
  a.n_zrows = p.groups;
  a.zrow_size_p = p.share_p;
  a.n_zrows_p = p.groups_p;
  if (a.mode == kSplitWindow && p.row_tiles > 0) a.zrow_size_p = a.n_zrows_p = 0;
  a.ws_acc = static_cast<float *>(workspace);
  a.ws_ml = reinterpret_cast<float2 *>(a.ws_acc + static_cast<int64_t>(a.batch) * a.hq * a.slot_stride * d);
  unsigned char *prep = static_cast<unsigned char *>(workspace) + p.acc_bytes;
  a.ws_qprep = reinterpret_cast<uint32_t *>(prep);
  a.ws_qrot = reinterpret_cast<float *>(prep);
  CodebookF32 cb;
  codebook_f32(d, bits, &cb);
  for (int j = 0; j < 16; ++j) a.centroid[j] = j < cb.levels ? cb.centroid[j] : 0.f;
  int e = ISOQ_OK;
  // The prefix on tcgen05: its query tiles first, its split last, so that it
  // runs beside the split over the rows' own caches.
  if (p.row_tiles > 0 && d != 128) e = run_prep_prefix(d, variant, a, static_cast<unsigned char *>(workspace) + p.tiles_at, p.row_tiles, st);
  if (e) return e;
  if (i8) {
    if (d == 128)
      e = variant == ISOQ_FULL ? run_i8_rows<128, true>(a, st) : run_i8_rows<128, false>(a, st);
    else
      e = variant == ISOQ_FULL ? run_i8_rows<256, true>(a, st) : run_i8_rows<256, false>(a, st);
  } else {
    if (!p.fused) e = run_prep_rotate(dtype, d, variant, a, st);
    if (e == ISOQ_OK) e = run_split_any(d, bits, a, st);
  }
  if (e == ISOQ_OK && p.row_tiles > 0)
    e = run_prefix_tc(d, variant, a, static_cast<unsigned char *>(workspace) + p.tiles_at, p.row_tiles, p.splits_p,
                      static_cast<int>(p.chunk_p), st);
  if (e || p.fused) return e;
  CombineArgs c;
  c.params_v = params_v;
  c.out = out;
  c.ws_acc = a.ws_acc;
  c.ws_ml = a.ws_ml;
  c.batch = a.batch;
  c.hq = a.hq;
  c.group = a.group;
  c.n_splits = a.slot_stride;
  return run_combine(dtype, d, variant, c, st);
}

// Whether two byte ranges share a byte.
bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + static_cast<uintptr_t>(nb) && y < x + static_cast<uintptr_t>(na);
}

}  // namespace decode
}  // namespace isoq

using namespace isoq;

extern "C" {

size_t isoq_decode_window_workspace_size(int B, int Hq, int Hkv, int64_t Tmax, int d, int64_t window, int64_t n_sink) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Tmax <= 0 || Tmax >= (1ll << 31) || !supported_d(d) || Hq % Hkv || window < 0 ||
      n_sink < 0)
    return 0;
  return decode::most_workspace(B, Hq, Hkv, Tmax, -1, d, window, n_sink);
}

size_t isoq_decode_prefix_workspace_size(int B, int Hq, int Hkv, int64_t prefix_tokens, int64_t Tmax, int d) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Tmax <= 0 || Tmax >= (1ll << 31) || prefix_tokens < 0 ||
      prefix_tokens >= (1ll << 31) || !supported_d(d) || Hq % Hkv)
    return 0;
  return decode::most_workspace(B, Hq, Hkv, Tmax, prefix_tokens, d, Tmax, 0);
}

int isoq_decode_attention_window(const void *q_dev, int dtype, const uint8_t *packed_k_dev,
                                 const uint8_t *packed_v_dev, const uint16_t *norms_k_dev,
                                 const uint16_t *norms_v_dev, const int32_t *seq_lens_dev, int B, int Hq, int Hkv,
                                 int64_t Tmax, int d, int bits, int variant, const float *params_k_dev,
                                 const float *params_v_dev, float scale, int64_t window, int64_t n_sink,
                                 void *out_dev, void *workspace_dev, size_t workspace_bytes, isoq_stream_t stream) {
  clear_error();
  int st = decode::check_decode(dtype, B, Hq, Hkv, Tmax, d, bits, variant, window, n_sink, scale);
  if (st) return st;
  if (!q_dev || !packed_k_dev || !packed_v_dev || !norms_k_dev || !norms_v_dev || !seq_lens_dev || !params_k_dev ||
      !params_v_dev || !out_dev)
    return set_error(ISOQ_ERR_INVALID_ARG, "null pointer");
  if (!decode::aligned(q_dev, 16) || !decode::aligned(packed_k_dev, 16) || !decode::aligned(packed_v_dev, 16) ||
      !decode::aligned(params_k_dev, 16) || !decode::aligned(params_v_dev, 16) || !decode::aligned(out_dev, 16) ||
      !decode::aligned(norms_k_dev, 2) || !decode::aligned(norms_v_dev, 2) || !decode::aligned(seq_lens_dev, 4))
    return set_error(ISOQ_ERR_UNSUPPORTED, "misaligned pointer");
  const bool i8 = decode::i8_split(dtype, d, bits) && decode::i8_cache(norms_k_dev, norms_v_dev, Tmax);
  const decode::DecodePlan p = decode::plan_decode(B, Hq, Hkv, Tmax, -1, d, bits, window, n_sink, i8);
  st = decode::check_workspace(workspace_dev, workspace_bytes, decode::most_workspace(B, Hq, Hkv, Tmax, -1, d, window, n_sink));
  if (st) return st;
  decode::SplitArgs a{};
  a.mode = decode::kSplitWindow;
  a.q = q_dev;
  a.packed_k = packed_k_dev;
  a.packed_v = packed_v_dev;
  a.norms_k = norms_k_dev;
  a.norms_v = norms_v_dev;
  a.seq_lens = seq_lens_dev;
  a.params_k = params_k_dev;
  a.tmax = Tmax;
  a.batch = B;
  a.hq = Hq;
  a.hkv = Hkv;
  a.scale = scale;
  a.window = decode::clamp31(window);
  a.n_sink = decode::clamp31(n_sink);
  return decode::run_decode(a, p, dtype, d, bits, variant, i8, params_v_dev,
                            out_dev, workspace_dev, reinterpret_cast<cudaStream_t>(stream));
}

int isoq_decode_attention_prefix(const void *q_dev, int dtype, const uint8_t *prefix_k_dev,
                                 const uint8_t *prefix_v_dev, const uint16_t *prefix_norms_k_dev,
                                 const uint16_t *prefix_norms_v_dev, const int32_t *prefix_len_dev,
                                 int64_t prefix_tokens, int64_t prefix_head_stride, const uint8_t *packed_k_dev,
                                 const uint8_t *packed_v_dev, const uint16_t *norms_k_dev,
                                 const uint16_t *norms_v_dev, const int32_t *seq_lens_dev, int B, int Hq, int Hkv,
                                 int64_t Tmax, int d, int bits, int variant, const float *params_k_dev,
                                 const float *params_v_dev, float scale, void *out_dev, void *workspace_dev,
                                 size_t workspace_bytes, isoq_stream_t stream) {
  clear_error();
  int st = decode::check_decode(dtype, B, Hq, Hkv, Tmax, d, bits, variant, 0, 0, scale);
  if (st) return st;
  if (prefix_tokens < 0 || prefix_tokens >= (1ll << 31))
    return set_error(ISOQ_ERR_INVALID_ARG, "prefix_tokens=%lld", static_cast<long long>(prefix_tokens));
  if (prefix_head_stride < prefix_tokens)
    return set_error(ISOQ_ERR_INVALID_ARG, "prefix_head_stride < prefix_tokens");
  if (!q_dev || !packed_k_dev || !packed_v_dev || !norms_k_dev || !norms_v_dev || !seq_lens_dev || !params_k_dev ||
      !params_v_dev || !out_dev || !prefix_len_dev ||
      (prefix_tokens > 0 && (!prefix_k_dev || !prefix_v_dev || !prefix_norms_k_dev || !prefix_norms_v_dev)))
    return set_error(ISOQ_ERR_INVALID_ARG, "null pointer");
  if (!decode::aligned(q_dev, 16) || !decode::aligned(packed_k_dev, 16) || !decode::aligned(packed_v_dev, 16) ||
      !decode::aligned(prefix_k_dev, 16) || !decode::aligned(prefix_v_dev, 16) || !decode::aligned(params_k_dev, 16) ||
      !decode::aligned(params_v_dev, 16) || !decode::aligned(out_dev, 16) || !decode::aligned(norms_k_dev, 2) ||
      !decode::aligned(norms_v_dev, 2) || !decode::aligned(prefix_norms_k_dev, 2) ||
      !decode::aligned(prefix_norms_v_dev, 2) || !decode::aligned(seq_lens_dev, 4) || !decode::aligned(prefix_len_dev, 4))
    return set_error(ISOQ_ERR_UNSUPPORTED, "misaligned pointer");
  // The tcgen05 split reads codes and norms by plain loads: any prefix does.
  const bool tc = decode::tc_prefix(dtype, d, bits) && B * static_cast<int64_t>(Hq / Hkv) >= decode::prefix_tc_rows(d) &&
                  prefix_tokens > 0;
  // The integer split rounds a copy of norms up to 8 tokens: within the room
  // of the last KV head only where the prefix's tokens are a multiple of 8.
  const bool i8 = decode::i8_split(dtype, d, bits) && decode::i8_cache(norms_k_dev, norms_v_dev, Tmax) &&
                  (tc || (decode::i8_cache(prefix_norms_k_dev, prefix_norms_v_dev, prefix_head_stride) &&
                          prefix_tokens % 8 == 0));
  const decode::DecodePlan p = decode::plan_decode(B, Hq, Hkv, Tmax, prefix_tokens, d, bits, Tmax, 0, i8, tc);
  st = decode::check_workspace(workspace_dev, workspace_bytes,
                               decode::most_workspace(B, Hq, Hkv, Tmax, prefix_tokens, d, Tmax, 0));
  if (st) return st;
  decode::SplitArgs a{};
  a.mode = tc ? decode::kSplitWindow : decode::kSplitPrefix;
  a.q = q_dev;
  a.packed_k = packed_k_dev;
  a.packed_v = packed_v_dev;
  a.norms_k = norms_k_dev;
  a.norms_v = norms_v_dev;
  a.seq_lens = seq_lens_dev;
  a.params_k = params_k_dev;
  a.tmax = Tmax;
  a.batch = B;
  a.hq = Hq;
  a.hkv = Hkv;
  a.scale = scale;
  a.window = 0x7FFFFFFF;
  a.n_sink = 0;
  a.prefix_k = prefix_k_dev;
  a.prefix_v = prefix_v_dev;
  a.prefix_nk = prefix_norms_k_dev;
  a.prefix_nv = prefix_norms_v_dev;
  a.prefix_len = prefix_len_dev;
  a.prefix_max = prefix_tokens;
  a.head_stride = prefix_head_stride;
  return decode::run_decode(a, p, dtype, d, bits, variant, i8, params_v_dev, out_dev, workspace_dev,
                            reinterpret_cast<cudaStream_t>(stream));
}

int isoq_paged_decode_attention(const void *q_dev, int dtype, const uint8_t *pages_k_dev, const uint8_t *pages_v_dev,
                                const uint16_t *norms_k_dev, const uint16_t *norms_v_dev,
                                const int32_t *block_table_dev, const int32_t *seq_lens_dev, int B, int Hq, int Hkv,
                                int n_pages, int page_tokens, int max_pages, int64_t max_len, int d, int bits,
                                int variant, const float *params_k_dev, const float *params_v_dev, float scale,
                                int64_t window, int64_t n_sink, void *out_dev, void *workspace_dev,
                                size_t workspace_bytes, isoq_stream_t stream) {
  clear_error();
  const int shift = decode::page_shift_of(page_tokens);
  if (shift < 0)
    return set_error(ISOQ_ERR_UNSUPPORTED, "page_tokens=%d (16, 32, 64, 128 or 256)", page_tokens);
  if (n_pages <= 0 || max_pages <= 0) return set_error(ISOQ_ERR_INVALID_ARG, "n_pages and max_pages must be positive");
  int st = decode::check_decode(dtype, B, Hq, Hkv, max_len, d, bits, variant, window, n_sink, scale);
  if (st) return st;
  if (max_len > static_cast<int64_t>(max_pages) * page_tokens)
    return set_error(ISOQ_ERR_INVALID_ARG, "max_len is more than the block table holds");
  if (!q_dev || !pages_k_dev || !pages_v_dev || !norms_k_dev || !norms_v_dev || !block_table_dev || !seq_lens_dev ||
      !params_k_dev || !params_v_dev || !out_dev)
    return set_error(ISOQ_ERR_INVALID_ARG, "null pointer");
  if (!decode::aligned(q_dev, 16) || !decode::aligned(pages_k_dev, 16) || !decode::aligned(pages_v_dev, 16) ||
      !decode::aligned(params_k_dev, 16) || !decode::aligned(params_v_dev, 16) || !decode::aligned(out_dev, 16) ||
      !decode::aligned(norms_k_dev, 2) || !decode::aligned(norms_v_dev, 2) || !decode::aligned(seq_lens_dev, 4) ||
      !decode::aligned(block_table_dev, 4))
    return set_error(ISOQ_ERR_UNSUPPORTED, "misaligned pointer");
  const bool i8 = decode::i8_split(dtype, d, bits) && decode::i8_cache(norms_k_dev, norms_v_dev, 8);
  const decode::DecodePlan p = decode::plan_decode(B, Hq, Hkv, max_len, -1, d, bits, window, n_sink, i8);
  st = decode::check_workspace(workspace_dev, workspace_bytes,
                               decode::most_workspace(B, Hq, Hkv, max_len, -1, d, window, n_sink));
  if (st) return st;
  decode::SplitArgs a{};
  a.mode = decode::kSplitPaged;
  a.q = q_dev;
  a.packed_k = pages_k_dev;
  a.packed_v = pages_v_dev;
  a.norms_k = norms_k_dev;
  a.norms_v = norms_v_dev;
  a.seq_lens = seq_lens_dev;
  a.params_k = params_k_dev;
  a.tmax = max_len;
  a.batch = B;
  a.hq = Hq;
  a.hkv = Hkv;
  a.scale = scale;
  a.window = decode::clamp31(window);
  a.n_sink = decode::clamp31(n_sink);
  a.block_table = block_table_dev;
  a.page_shift = shift;
  a.max_pages = max_pages;
  a.n_pages = n_pages;
  return decode::run_decode(a, p, dtype, d, bits, variant, i8, params_v_dev,
                            out_dev, workspace_dev, reinterpret_cast<cudaStream_t>(stream));
}

int isoq_prefill_attention_window(const void *q_dev, int dtype, const uint8_t *packed_k_dev,
                                  const uint8_t *packed_v_dev, const uint16_t *norms_k_dev,
                                  const uint16_t *norms_v_dev, const int32_t *seq_lens_dev, int B, int Tq, int Hq,
                                  int Hkv, int64_t Tmax, int d, int bits, int variant, const float *params_k_dev,
                                  const float *params_v_dev, float scale, int64_t window, int64_t n_sink,
                                  void *out_dev, isoq_stream_t stream) {
  clear_error();
  decode::PrefillArgs a{};
  const int st = decode::prefill_args(q_dev, dtype, packed_k_dev, packed_v_dev, norms_k_dev, norms_v_dev, seq_lens_dev,
                                      B, Tq, Hq, Hkv, Tmax, d, bits, variant, params_k_dev, params_v_dev, scale,
                                      out_dev, &a);
  if (st) return st;
  if (window < 0 || n_sink < 0) return set_error(ISOQ_ERR_INVALID_ARG, "window and n_sink must not be negative");
  if (Tq == 0) return ISOQ_OK;
  a.window = decode::clamp31(window);
  a.n_sink = decode::clamp31(n_sink);
  variant = block_map_variant(variant);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // The 128-row kernel moves rows 8 bytes at a time.
  if (d == 128 && decode::aligned(q_dev, 8) && decode::aligned(out_dev, 8)) return decode::run_window_rows(variant, a, s);
  return decode::run_prefill<decode::kPfWindow>(d, variant, a, s);
}

int isoq_build_block_tables(const int32_t *seq_lens_dev, const int32_t *new_lens_dev, const int32_t *free_pages_dev,
                            const int32_t *free_head_dev, int n_free, int B, int page_tokens, int max_pages,
                            int32_t *block_table_dev, int64_t n_slots, int64_t *slot_map_dev, int32_t *row_start_dev,
                            int32_t *total_lens_dev, int32_t *pages_used_dev, isoq_stream_t stream) {
  clear_error();
  const int shift = decode::page_shift_of(page_tokens);
  if (shift < 0)
    return set_error(ISOQ_ERR_UNSUPPORTED, "page_tokens=%d (16, 32, 64, 128 or 256)", page_tokens);
  if (B <= 0 || max_pages <= 0 || n_free < 0 || n_slots < 0)
    return set_error(ISOQ_ERR_INVALID_ARG, "B and max_pages must be positive, n_free and n_slots not negative");
  if (n_slots >= (1ll << 31)) return set_error(ISOQ_ERR_INVALID_ARG, "n_slots too large");
  if (!seq_lens_dev || !new_lens_dev || (!free_pages_dev && n_free > 0) || !block_table_dev ||
      (!slot_map_dev && n_slots > 0) || !row_start_dev || !total_lens_dev || !pages_used_dev)
    return set_error(ISOQ_ERR_INVALID_ARG, "null pointer");
  if (!decode::aligned(seq_lens_dev, 4) || !decode::aligned(new_lens_dev, 4) || !decode::aligned(free_pages_dev, 4) ||
      !decode::aligned(free_head_dev, 4) || !decode::aligned(block_table_dev, 4) || !decode::aligned(slot_map_dev, 8) ||
      !decode::aligned(row_start_dev, 4) || !decode::aligned(total_lens_dev, 4) || !decode::aligned(pages_used_dev, 4))
    return set_error(ISOQ_ERR_UNSUPPORTED, "misaligned pointer");
  // Every CTA reads the inputs while others write: no output may share memory
  // with an input or another output.
  struct { const void *p; int64_t n; } r[] = {
      {block_table_dev, 4ll * B * max_pages}, {slot_map_dev, 8 * n_slots}, {row_start_dev, 4ll * B + 4},
      {total_lens_dev, 4ll * B}, {pages_used_dev, 4}, {seq_lens_dev, 4ll * B}, {new_lens_dev, 4ll * B},
      {free_pages_dev, 4ll * n_free}, {free_head_dev, free_head_dev ? 4 : 0}};
  for (int i = 0; i < 5; ++i)
    for (int j = i + 1; j < 9; ++j)
      if (decode::overlap(r[i].p, r[i].n, r[j].p, r[j].n))
        return set_error(ISOQ_ERR_INVALID_ARG, "an output overlaps an input or another output");
  decode::TableArgs a;
  a.seq_lens = seq_lens_dev;
  a.new_lens = new_lens_dev;
  a.free_pages = free_pages_dev;
  a.free_head = free_head_dev;
  a.block_table = block_table_dev;
  a.slot_map = reinterpret_cast<long long *>(slot_map_dev);
  a.row_start = row_start_dev;
  a.total_lens = total_lens_dev;
  a.pages_used = pages_used_dev;
  a.n_slots = n_slots;
  a.batch = B;
  a.n_free = n_free;
  a.max_pages = max_pages;
  a.page_shift = shift;
  const int64_t ctas = decode::div_up(n_slots, decode::kTableTokens);
  decode::block_tables_kernel<<<static_cast<unsigned>(ctas > 1 ? ctas : 1), decode::kTableThreads, 0,
                                reinterpret_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ISOQ_OK : set_error(ISOQ_ERR_CUDA, "block tables launch: %s", cudaGetErrorString(e));
}

int isoq_paged_append(const void *k_new_dev, const void *v_new_dev, int dtype, uint8_t *pages_k_dev,
                      uint8_t *pages_v_dev, uint16_t *norms_k_dev, uint16_t *norms_v_dev, const int64_t *slot_map_dev,
                      int64_t N, int Hkv, int n_pages, int page_tokens, int d, int bits, int variant,
                      const float *params_k_dev, const float *params_v_dev, isoq_stream_t stream) {
  clear_error();
  if (!supported_d(d)) return set_error(ISOQ_ERR_UNSUPPORTED, "d=%d not supported", d);
  if (!supported_bits(bits)) return set_error(ISOQ_ERR_UNSUPPORTED, "bits=%d not supported", bits);
  if (!supported_decode_variant(variant)) return set_error(ISOQ_ERR_UNSUPPORTED, "variant=%d", variant);
  if (!supported_dtype(dtype)) return set_error(ISOQ_ERR_UNSUPPORTED, "dtype=%d", dtype);
  const int shift = decode::page_shift_of(page_tokens);
  if (shift < 0)
    return set_error(ISOQ_ERR_UNSUPPORTED, "page_tokens=%d (16, 32, 64, 128 or 256)", page_tokens);
  if (N < 0 || Hkv <= 0 || n_pages <= 0)
    return set_error(ISOQ_ERR_INVALID_ARG, "Hkv and n_pages must be positive, N >= 0");
  if (Hkv > 32767 || N >= (1ll << 31)) return set_error(ISOQ_ERR_INVALID_ARG, "shape too large");
  if (N == 0) return ISOQ_OK;
  if (!k_new_dev || !v_new_dev || !pages_k_dev || !pages_v_dev || !norms_k_dev || !norms_v_dev || !slot_map_dev ||
      !params_k_dev || !params_v_dev)
    return set_error(ISOQ_ERR_INVALID_ARG, "null pointer");
  if (!decode::aligned(k_new_dev, 16) || !decode::aligned(v_new_dev, 16) || !decode::aligned(pages_k_dev, 16) ||
      !decode::aligned(pages_v_dev, 16) || !decode::aligned(params_k_dev, 16) || !decode::aligned(params_v_dev, 16) ||
      !decode::aligned(norms_k_dev, 2) || !decode::aligned(norms_v_dev, 2) || !decode::aligned(slot_map_dev, 8))
    return set_error(ISOQ_ERR_UNSUPPORTED, "misaligned pointer");
  decode::PagedAppendArgs a{};
  a.k_new = k_new_dev;
  a.v_new = v_new_dev;
  a.pages_k = pages_k_dev;
  a.pages_v = pages_v_dev;
  a.norms_k = norms_k_dev;
  a.norms_v = norms_v_dev;
  a.slot_map = reinterpret_cast<const long long *>(slot_map_dev);
  a.params_k = params_k_dev;
  a.params_v = params_v_dev;
  a.n_tok = N;
  a.n_rows = static_cast<long long>(n_pages) << shift;
  a.hkv = Hkv;
  a.page_shift = shift;
  const int half = 1 << (bits - 1);
  isoq_make_codebook(d, bits, nullptr, a.thr64);
  for (int k = 0; k < half; ++k) a.thr[k] = static_cast<float>(a.thr64[half - 1 + k]);
  return decode::run_paged_append(dtype, d, bits, block_map_variant(variant), a, reinterpret_cast<cudaStream_t>(stream));
}

__attribute__((visibility("hidden"))) cudaError_t isoq_detail_serve_error_word(void **word) {
  return cudaGetSymbolAddress(word, decode::g_decode_error);
}

}  // extern "C"
