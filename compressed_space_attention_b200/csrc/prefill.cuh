// Causal attention of a chunk of Tq new queries over the packed cache
// (chunked prefill), on the 5th-generation tensor cores (tcgen05 + TMEM).
// Included by isoq_decode.cu and isoq_serve.cu inside namespace isoq::decode,
// after the rotation helpers.
//
// Query t of batch row b sits at position p = seq_lens[b] - Tq + t and
// attends to the cached tokens j <= p (RotaryQuant §3.4: kernel A with
// causal masking, which ends each query tile's token loop early; Figure 1's
// path with more than one query).  Everything stays in the rotated domain as
// in the decode: q~ = R_K q once per query, scores against the centroids,
// softmax, V accumulated as centroids, one inverse rotation per output row.
//
// CTA = 128 query-head rows (128 / GP positions x GP heads; heads >= G are
// dead rows), one TMEM lane each, 8 warps: warps w and w + 4 share TMEM
// sub-partition w (lanes 32 w .. + 31) and split each row's S and O columns
// in halves.  Per 64-token tile j, software-pipelined by one product:
//   the packed codes and norms of the next tiles are loaded into registers
//   one phase ahead; the CTA expands K tile j + 1's codes into float16
//   centroids alpha c_k in a 128B-swizzled tile, and their float16
//   residuals alpha c_k - fp16(alpha c_k) into a second tile (alpha is
//   searched on the host; the residuals are below 2^-15 of the centroids,
//   so hi + lo keeps them to about 2^-26), and one thread issues
//   S(j + 1) = Q~hi K~hi^T + Q~lo K~hi^T + Q~hi K~lo^T (tcgen05.mma
//   kind::f16, M = 128, N = 64; q~ split into float16 hi and lo parts, each
//   row scaled by a power of two: query_scale) into
//   the other of two TMEM S buffers, so it runs under the softmax of tile j;
//   each thread reads its half row of S(j) (tcgen05.ld), scales it by
//   s^K scale / alpha, masks it on diagonal tiles, exchanges its half-row
//   maximum with the partner warp through the consumed S buffer, writes
//   P = p s^V as float16 hi and lo parts (22 bits of each weight, s^V scaled by
//   a power of two for the whole CTA: value_scale) over that
//   S buffer in TMEM and, when its warp's maximum moved, rescales its half
//   of the O row in TMEM; the CTA expands V tile j into its own tile buffer
//   and one thread issues O += P_hi V~ + P_lo V~ (A = P from tensor memory,
//   N = d, V~ read MN-major from the token-row tile).  The next product into
//   that S buffer (QK of tile j + 2) is issued after the PV product, and the
//   tensor core runs one CTA's products in issue order.
// Both the hi/lo query and the hi/lo centroid residual are needed for the
// float16 output bar on outlier-heavy K/V: float16 centroids alone (relative
// error 1.9e-5) or float16 weights alone (2^-12) move scores or weights
// enough to shift outputs of magnitude 30-80 by several 1e-3.
// d = 128 fits two CTAs per SM (one CTA's thread work runs under the
// other's products); d = 256 one.
// The epilogue reads O from TMEM, normalises, rotates back (R_V^T) in shared
// memory and stores float16.
// Operand tiles use the canonical SW128 layouts: rows of 128 bytes (64
// float16), 16-byte chunks XOR-swizzled by (row % 8), 8-row groups 1024
// bytes apart, 64-element blocks of the row direction `blk_stride` apart.
// Every wait is bounded; on a timeout the CTA records kErrWaitTimeout, waits
// (bounded) for its outstanding products, frees its tensor memory and
// returns.
//
// Requires float16 queries (float16 tiles meet the float16 output tolerance,
// not the float32 one), 3-bit codes, d in {128, 256}, G = Hq / Hkv in
// {1, 2, 4, 8}, Tmax % 8 == 0 and 16-byte aligned code rows.

// The prefill kernel found its dynamic shared memory off a 1024-byte
// boundary (its two-CTAs-per-SM layout keeps no slack to align it) and
// returned without writing its output.
constexpr unsigned kErrSmemAlign = 4u;

struct PrefillArgs {
  const void *q;                  // [B][Tq][Hq][d]
  const uint8_t *packed_k, *packed_v;
  const uint16_t *norms_k, *norms_v;
  const int32_t *seq_lens;
  const float *params_k, *params_v;
  void *out;                      // [B][Tq][Hq][d], dtype of q
  long long tmax;
  int batch, tq, hq, hkv, group;
  float score_unit;               // scale * log2(e) / (alpha sqrt(d))
  float out_unit;                 // 1 / (alpha * d)
  uint32_t lut_lo0, lut_lo1, lut_hi0, lut_hi1;   // float16 alpha c_k, low / high bytes
  uint32_t res_lo0, res_lo1, res_hi0, res_hi1;   // float16 alpha c_k - fp16(alpha c_k), low / high bytes
  int window, n_sink;             // kPfWindow: tokens j > p - window or j < n_sink only
  // kPfPrefix: query rows prepared in the operand layout, [Hkv][row tiles] of
  // float16 hi and lo tiles and the rows' inverse scales (TcCfg::Q_TILE bytes);
  // partial states as the decode's splits write them.
  const unsigned char *q_tiles;
  const int32_t *prefix_len;
  long long head_stride;          // tokens between KV heads
  int row_tiles, chunk;           // 128-row tiles per KV head; tokens per split
  float *ws_acc;
  float2 *ws_ml;
  int slot_stride;
  float acc_unit;                 // 1 / (alpha sqrt(d))
};

// What the kernel computes: the causal chunk, the same under a sliding window
// with sinks, or partial states of a batch's queries over one shared prefix.
enum PrefillKind { kPfCausal = 0, kPfWindow = 1, kPfPrefix = 2 };

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// The scale of a query row's float16 hi and lo parts, and its inverse, which
// the row's scores take: 1 while the largest rotated component `mx` lies in
// [1/4, 2^15), else the power of two that takes it to [2^14, 2^15).  A rotated
// component can reach |q|, sqrt(d) times what float16 holds, and below 1/4 the
// lo parts lose bits to the subnormal numbers (steps of 2^-24); so hi + lo
// keeps 22 bits of every row.  (The exponent is kept from 64 on, for zeros and
// for what cancels to next to nothing.)
__device__ __forceinline__ float query_scale(float mx, float &inverse) {
  uint32_t e = __float_as_uint(mx) >> 23;
  e = e < 64u ? 64u : (e >= 125u && e < 142u ? 141u : e);
  inverse = __uint_as_float((e - 14u) << 23);
  return __uint_as_float((127u + 14u + 127u - e) << 23);
}

// The largest finite V norm (float16 bits) of tokens [a, b), over the lanes of a
// warp; 0 if there is none.  Eight loads are under way at once: the pass
// stands before a CTA's first tile.
template <int THREADS>
__device__ __forceinline__ uint32_t largest_norm(const uint16_t *norms, int a, int b, int tid) {
  uint32_t mx = 0;
  for (int t = a; t < b; t += 8 * THREADS) {
    uint32_t u[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) u[k] = b - t > k * THREADS + tid ? __ldg(norms + t + k * THREADS + tid) & 0x7FFFu : 0u;
#pragma unroll
    for (int k = 0; k < 8; ++k) mx = u[k] < 0x7C00u && u[k] > mx ? u[k] : mx;   // magnitudes order as integers
  }
  return __reduce_max_sync(0xffffffffu, mx);
}

// The scale of V's norms for the float16 hi and lo parts of the weights p s^V
// (p <= 1): the power of two that takes the largest of them (float16 bits) to
// [2^14, 2^15).  Unscaled, weights below 2^-14 lose bits and those below 2^-25
// vanish, however many there are of them; with it, that is relative to the
// largest norm.  The results are divided by it.
__device__ __forceinline__ float value_scale(uint32_t largest) {
  if (largest == 0) return 1.f;
  const uint32_t e = __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(largest)))) >> 23;
  return __uint_as_float((127u + 14u + 127u - e) << 23);
}

// Multi-row inverse rotation H_d R_SO4^T u (unnormalised) of nvec rows in
// shared memory, by the whole CTA.
template <int D, bool FULL>
__device__ void rotate_inverse_rows(float *v, int nvec, const float *params_head, int tid, int nthreads) {
  for (int idx = tid; idx < nvec * (D / 4); idx += nthreads) {
    const int g = idx / (D / 4), bi = idx % (D / 4);
    float *w = v + g * D + 4 * bi;
    const Quat u{w[0], w[1], w[2], w[3]};
    const Quat x = block_inverse(load_quat(params_head + 8 * bi), load_quat(params_head + 8 * bi + 4), u, FULL);
    w[0] = x.w;
    w[1] = x.x;
    w[2] = x.y;
    w[3] = x.z;
  }
  __syncthreads();
#pragma unroll 1
  for (int h = 1; h < D; h <<= 1) {
    for (int idx = tid; idx < nvec * (D / 2); idx += nthreads) {
      const int g = idx / (D / 2), p = idx % (D / 2);
      float *w = v + g * D;
      const int i = (p / h) * 2 * h + (p % h);
      const float x0 = w[i], x1 = w[i + h];
      w[i] = x0 + x1;
      w[i + h] = x0 - x1;
    }
    __syncthreads();
  }
}

constexpr int kTcThreads = 256;   // 8 warps: two per TMEM sub-partition, one per column half
constexpr int kTcRows = 128;      // M: query-head rows per CTA
constexpr int kTcTok = 64;        // N of QK, K of PV

template <int D>
struct TcCfg {
  static constexpr int PB = D * 3 / 8;
  static constexpr int ITEMS = kTcTok * (D / 32) / kTcThreads;   // 32-code groups per thread per tile
  static constexpr int Q_BYTES = kTcRows * D * 2;         // one of hi / lo
  static constexpr int Q_TILE = 2 * Q_BYTES + kTcRows * 4;   // prepared: hi, lo, the rows' inverse scales
  static constexpr int KV_BYTES = kTcTok * D * 2;         // one K, K-residual or V tile
  static constexpr int NORM_BYTES = 2 * kTcTok * 4;       // s^K score_unit, s^V of one tile
  static constexpr int OFF_QLO = Q_BYTES;
  static constexpr int OFF_K = 2 * Q_BYTES;
  static constexpr int OFF_KLO = OFF_K + KV_BYTES;
  static constexpr int OFF_V = OFF_KLO + KV_BYTES;
  static constexpr int OFF_NORM = OFF_V + KV_BYTES;
  static constexpr int OFF_BAR = OFF_NORM + NORM_BYTES;
  // Two CTAs per SM at d = 128 (the second CTA's softmax and expansion run
  // under the first one's products).  Their layout leaves no room to align
  // the dynamic shared memory by hand: the kernel checks that it starts on a
  // 1024-byte boundary and reports kErrSmemAlign otherwise.
  static constexpr int MIN_BLOCKS = D == 128 ? 2 : 1;
  static constexpr int SLACK = MIN_BLOCKS == 2 ? 0 : 1024;
  static constexpr int SMEM = OFF_BAR + 8 * 4 + 8 + SLACK;
  static constexpr int TMEM_COLS = D == 128 ? 256 : 512;     // S (2 x 64) + O (D), rounded to a power of 2
  static_assert(32 * D * 4 <= 2 * KV_BYTES, "prep scratch (32 rows) fits the K and K-residual tiles");
  static_assert(MIN_BLOCKS * (SMEM + 1024) <= 233472, "shared memory per SM (1 KB reserved per CTA)");
  static_assert(MIN_BLOCKS * TMEM_COLS <= 512, "tensor memory columns");
};

// Packed codes of one tile, this thread's share (ITEMS 32-code groups),
// loaded from global memory one phase before they are expanded.
template <int D>
struct TcCodes {
  uint32_t w[TcCfg<D>::ITEMS][3];
};

template <int D>
__device__ __forceinline__ void tc_fetch(TcCodes<D> &c, const uint8_t *base, int t0, int tend, int tid) {
  constexpr int GROUPS = D / 32, PB = D * 3 / 8;
#pragma unroll
  for (int k = 0; k < TcCfg<D>::ITEMS; ++k) {
    const int idx = tid + k * kTcThreads, tok = idx / GROUPS, grp = idx % GROUPS;
    if (t0 + tok < tend) {
      const uint32_t *src = reinterpret_cast<const uint32_t *>(base + static_cast<long long>(t0 + tok) * PB + 12 * grp);
      c.w[k][0] = __ldg(src);
      c.w[k][1] = __ldg(src + 1);
      c.w[k][2] = __ldg(src + 2);
    } else {
      c.w[k][0] = c.w[k][1] = c.w[k][2] = 0u;
    }
  }
}

// Fetched codes -> float16 centroids alpha c_k in the SW128 token-row tile
// (64-dim blocks kTcTok * 128 bytes apart); the same layout serves K (K-major
// B of QK) and V (MN-major B of PV).  With RES, the float16 residuals
// alpha c_k - fp16(alpha c_k) go to a second tile of the same layout.
template <int D, bool RES>
__device__ __forceinline__ void tc_expand(const TcCodes<D> &c, unsigned char *tile, unsigned char *tile_res,
                                          const PrefillArgs &a, int tid) {
  constexpr int GROUPS = D / 32, BLK = kTcTok * 128;
#pragma unroll
  for (int k = 0; k < TcCfg<D>::ITEMS; ++k) {
    const int idx = tid + k * kTcThreads, tok = idx / GROUPS, grp = idx % GROUPS;
    uint32_t s[8];
    group_sel8(c.w[k][0], c.w[k][1], c.w[k][2], s);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      uint32_t v[4], r[4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t lo = prmt(a.lut_lo0, a.lut_lo1, s[2 * m + u]);
        const uint32_t hi = prmt(a.lut_hi0, a.lut_hi1, s[2 * m + u]);
        v[2 * u] = prmt(lo, hi, 0x5140u);
        v[2 * u + 1] = prmt(lo, hi, 0x7362u);
        if constexpr (RES) {
          const uint32_t rlo = prmt(a.res_lo0, a.res_lo1, s[2 * m + u]);
          const uint32_t rhi = prmt(a.res_hi0, a.res_hi1, s[2 * m + u]);
          r[2 * u] = prmt(rlo, rhi, 0x5140u);
          r[2 * u + 1] = prmt(rlo, rhi, 0x7362u);
        }
      }
      // dims 32 grp + 8 m .. + 7, as two 8-byte stores (measured faster
      // here than one 16-byte store, despite the latter's fewer bank conflicts)
      *reinterpret_cast<uint2 *>(tile + tc_off(tok, 32 * grp + 8 * m, BLK)) = make_uint2(v[0], v[1]);
      *reinterpret_cast<uint2 *>(tile + tc_off(tok, 32 * grp + 8 * m + 4, BLK)) = make_uint2(v[2], v[3]);
      if constexpr (RES) {
        *reinterpret_cast<uint2 *>(tile_res + tc_off(tok, 32 * grp + 8 * m, BLK)) = make_uint2(r[0], r[1]);
        *reinterpret_cast<uint2 *>(tile_res + tc_off(tok, 32 * grp + 8 * m + 4, BLK)) = make_uint2(r[2], r[3]);
      }
    }
  }
}

// kPfWindow: a sliding window with sink tokens.  The query at position p sees j <= p
// with j > p - window or j < n_sink.  The CTA's tiles are the sink tiles, then
// those from the first row's window on; a tile that some row of a warp does
// not see whole is masked by column.
//
// kPfPrefix: the rows are the query heads of all batch rows (row r of a KV
// head: batch row r / G, head r mod G), rotated and split beforehand
// (prep_prefix_kernel) and fetched by two bulk copies; every row sees all of
// the CTA's tokens, a chunk of the prefix; instead of outputs the epilogue
// writes one partial state (m, l, acc) per row.  Grid (row tiles, Hkv, splits).
template <typename T, int D, bool FULL, int GP, int KIND = kPfCausal>
__global__ void __launch_bounds__(kTcThreads, TcCfg<D>::MIN_BLOCKS) prefill_tc_kernel(const PrefillArgs a) {
  using C = TcCfg<D>;
  constexpr bool WIN = KIND == kPfWindow, PREFIX = KIND == kPfPrefix;
  constexpr int BQ = kTcRows / GP;
  constexpr int QBLK = kTcRows * 128, KBLK = kTcTok * 128;
  extern __shared__ unsigned char smem_raw[];
  // Aligned by an offset from the shared array itself (not through an
  // integer cast), so the compiler keeps the shared address space.
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  if (pad > static_cast<uint32_t>(C::SLACK)) {   // uniform over the grid: nothing allocated yet
    if (threadIdx.x == 0) atomicOr(&g_decode_error, kErrSmemAlign);
    return;
  }
  unsigned char *smem = smem_raw + pad;
  unsigned char *q_hi = smem, *q_lo = smem + C::OFF_QLO;
  unsigned char *kt = smem + C::OFF_K, *klt = smem + C::OFF_KLO, *vt = smem + C::OFF_V;
  float *nrm_s = reinterpret_cast<float *>(smem + C::OFF_NORM);   // [2][kTcTok] s^K score_unit, s^V of the tile in the softmax
  uint64_t *bar_s = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);   // [2]: S buffer b's product done
  uint64_t *bar_o = bar_s + 2;                                          // PV product done
  uint64_t *bar_q = bar_o + 1;                                          // kPfPrefix: the query tiles
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar_q + 1);
  // A product wait that gave up in iteration j sets fail_s[j % 2]; it is read
  // after the iteration's last block barrier (see the loop).
  volatile uint8_t *fail_s = reinterpret_cast<volatile uint8_t *>(tmem_slot + 1);
  float *scratch = reinterpret_cast<float *>(kt);   // 32 rows x D floats over the K tiles (prep, epilogue)

  const int qt = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5;
  const int G = a.group;

  const int32_t *lens = PREFIX ? a.prefix_len : a.seq_lens + b;
  // Positions follow the length as given, also beyond the room; below 0 as 0.
  // None of them, dead rows' among them, may leave the range of an int.
  const int given = *lens < 0 ? 0 : *lens;
  const int len = given > a.tmax ? static_cast<int>(a.tmax) : given;
  const int pos_base = PREFIX ? 0 : given - a.tq;
  const int tq0 = PREFIX ? 0 : qt * BQ;
  const int p_first = PREFIX ? 0x7FFFFF00 : pos_base + tq0;   // (every token is at or before it)
  const int p_last = pos_base + (tq0 + BQ > a.tq ? a.tq : tq0 + BQ) - 1;
  int tend = p_last + 1 < len ? p_last + 1 : len;
  if (tend < 0) tend = 0;
  int n_tiles = (tend + kTcTok - 1) / kTcTok;
  int t_base = 0;   // kPfPrefix: the split's first token
  if constexpr (PREFIX) {
    const long long first = static_cast<long long>(b) * a.chunk;
    t_base = first < len ? static_cast<int>(first) : len;
    tend = len - t_base > a.chunk ? t_base + a.chunk : len;
    n_tiles = (tend - t_base + kTcTok - 1) / kTcTok;
  }
  // WIN: tiles [0, n_sink_tiles), then from win_tile on.
  int n_sink_tiles = 0, win_tile = 0, sink = 0, lo = 0;
  if constexpr (WIN) {
    sink = a.n_sink < tend ? a.n_sink : tend;
    // The first row's window begins at lo; a window of none holds no token.
    lo = a.window == 0 ? tend : (p_first >= a.window ? p_first - a.window + 1 : 0);
    if (lo > tend) lo = tend;
    if (lo > sink) {
      const int all = n_tiles;
      n_sink_tiles = (sink + kTcTok - 1) / kTcTok;
      win_tile = lo / kTcTok > n_sink_tiles ? lo / kTcTok : n_sink_tiles;
      n_tiles = n_sink_tiles + (all > win_tile ? all - win_tile : 0);
    }
  }
  auto tile_t0 = [&](int j) {
    if constexpr (WIN)
      return kTcTok * (j < n_sink_tiles ? j : j - n_sink_tiles + win_tile);
    else
      return t_base + kTcTok * j;
  };

  const long long cache0 = PREFIX ? kvh * a.head_stride : (static_cast<long long>(b) * a.hkv + kvh) * a.tmax;
  const uint8_t *kb = a.packed_k + cache0 * C::PB;
  const uint8_t *vb = a.packed_v + cache0 * C::PB;
  const uint16_t *nkb = a.norms_k + cache0;
  const uint16_t *nvb = a.norms_v + cache0;

  // Codes and norms of upcoming tiles, one phase ahead, in registers:
  // kc = the next K tile to expand, vc = the next V tile, nrm = the norm
  // (K for tid < 64, V for tid < 128) of the next tile to enter the softmax.
  TcCodes<D> kc, vc;
  uint16_t nrm = 0;
  auto fetch_norm = [&](int j) {
    const int t0 = tile_t0(j), tok = tid & (kTcTok - 1);
    nrm = (tid < 2 * kTcTok && t0 + tok < tend) ? __ldg(((tid < kTcTok) ? nkb : nvb) + t0 + tok)
                                                : static_cast<uint16_t>(0);
  };
  if (n_tiles > 0) {
    tc_fetch<D>(kc, kb, tile_t0(0), tend, tid);
    tc_fetch<D>(vc, vb, tile_t0(0), tend, tid);
    fetch_norm(0);
  }

  // One word per warp where the first V tile goes later.
  uint32_t *v_max = reinterpret_cast<uint32_t *>(vt);
  {
    // What no row sees has no part in the scale: with a gap behind the sinks,
    // tokens [0, sink) and from lo on.
    const uint32_t m0 = lo > sink ? largest_norm<kTcThreads>(nvb, 0, sink, tid) : 0u;
    const uint32_t m1 = largest_norm<kTcThreads>(nvb, lo > sink ? lo : t_base, tend, tid);
    if ((tid & 31) == 0) v_max[warp] = m0 > m1 ? m0 : m1;
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(C::TMEM_COLS));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    mbar_init(&bar_s[0], 1);
    mbar_init(&bar_s[1], 1);
    mbar_init(bar_o, 1);
    mbar_init(bar_q, 1);
    fail_s[0] = fail_s[1] = 0;
    mbar_fence_init();
  }
  // kPfPrefix: hi and lo tile, then the rows' inverse scales.
  const unsigned char *q_tile = a.q_tiles + (static_cast<long long>(kvh) * a.row_tiles + qt) * C::Q_TILE;
  if constexpr (PREFIX) {
    // The prepared query tiles; a wait that gives up counts as a product's.
    if (tid == 0) {
      mbar_arrive_expect_tx(bar_q, 2 * C::Q_BYTES);
      bulk_load(q_hi, q_tile, C::Q_BYTES, bar_q);
      bulk_load(q_lo, q_tile + C::Q_BYTES, C::Q_BYTES, bar_q);
    }
  } else {
  // ---- prep, 32 rows per pass: rotate, split into float16 hi / lo (SW128 K-major) ----
  for (int pass = 0; pass < kTcRows / 32; ++pass) {
    for (int i = tid; i < 32 * D; i += kTcThreads) {
      const int m = 32 * pass + i / D, e = i % D;
      const int tl = m / GP, h = m % GP;
      float v = 0.f;
      if (h < G && tq0 + tl < a.tq) {
        const long long row = (static_cast<long long>(b) * a.tq + tq0 + tl) * a.hq + kvh * G + h;
        v = to_f32<T>(static_cast<const T *>(a.q)[row * D + e]);
      }
      scratch[i] = v;
    }
    __syncthreads();
    rotate_forward_smem<D, FULL>(scratch, 32, a.params_k + static_cast<size_t>(kvh) * 2 * D, tid, kTcThreads, 0);
    for (int i = tid; i < 32 * (D / 8); i += kTcThreads) {
      const int r = i / (D / 8), c = i % (D / 8), m = 32 * pass + r;
      uint32_t hv[4], lv[4];
      float big = 0.f, back;   // over the row: D / 8 neighbouring lanes hold it
#pragma unroll
      for (int k = 0; k < 8; ++k) big = fmaxf(big, fabsf(scratch[r * D + 8 * c + k]));
#pragma unroll
      for (int o = D / 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
      const float sc = query_scale(big, back);
      if (c == 0) nrm_s[m] = back;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x0 = scratch[r * D + 8 * c + 2 * k] * sc, x1 = scratch[r * D + 8 * c + 2 * k + 1] * sc;
        const __half h0 = __float2half_rn(x0), h1 = __float2half_rn(x1);
        const __half l0 = __float2half_rn(x0 - __half2float(h0)), l1 = __float2half_rn(x1 - __half2float(h1));
        const __half2 hh = __halves2half2(h0, h1), ll = __halves2half2(l0, l1);
        hv[k] = *reinterpret_cast<const uint32_t *>(&hh);
        lv[k] = *reinterpret_cast<const uint32_t *>(&ll);
      }
      *reinterpret_cast<uint4 *>(q_hi + tc_off(m, 8 * c, QBLK)) = make_uint4(hv[0], hv[1], hv[2], hv[3]);
      *reinterpret_cast<uint4 *>(q_lo + tc_off(m, 8 * c, QBLK)) = make_uint4(lv[0], lv[1], lv[2], lv[3]);
    }
    __syncthreads();
  }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  uint32_t norm_max = 0;
#pragma unroll
  for (int w = 0; w < kTcThreads / 32; ++w) norm_max = v_max[w] > norm_max ? v_max[w] : norm_max;
  const float v_scale = value_scale(norm_max);
  const uint32_t tmem = *tmem_slot;
  const uint32_t t_o = tmem + 128;                           // S buffers at columns [0, 64), [64, 128); O after
  // Warp w reads TMEM lanes 32 (w % 4) .. + 31 (its sub-partition) and
  // handles column half w / 4 of those rows' S and O.
  const int sub = warp & 3, half = warp >> 2, lane = tid & 31;
  const uint32_t lane_off = static_cast<uint32_t>(32 * sub) << 16;
  const uint32_t qh_s = smem_u32(q_hi), ql_s = smem_u32(q_lo), k_s = smem_u32(kt), kl_s = smem_u32(klt),
                 v_s = smem_u32(vt);

  // Expands K tile j (codes and norms from the registers), then issues its QK
  // product into S buffer j % 2.  The caller has made sure the K tile and
  // that S buffer are free.
  auto store_norm = [&]() {
    if (tid < 2 * kTcTok) nrm_s[tid] = __half2float(__ushort_as_half(nrm)) * (tid < kTcTok ? a.score_unit : v_scale);
  };
  auto stage_qk = [&](int j) {
    tc_expand<D, true>(kc, kt, klt, a, tid);
    if (j + 1 < n_tiles) tc_fetch<D>(kc, kb, tile_t0(j + 1), tend, tid);
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0) {
      constexpr uint32_t idesc = tc_idesc(kTcRows, kTcTok, 0);
      const uint32_t t_s = tmem + (j & 1) * 64;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t ko = (ks >> 2) * KBLK + (ks & 3) * 32, qo = (ks >> 2) * QBLK + (ks & 3) * 32;
        const uint64_t bd = tc_desc(k_s + ko, 16, 1024), ad = tc_desc(qh_s + qo, 16, 1024);
        tc_mma(t_s, ad, bd, idesc, ks > 0 ? 1u : 0u);
        tc_mma(t_s, tc_desc(ql_s + qo, 16, 1024), bd, idesc, 1u);
        tc_mma(t_s, ad, tc_desc(kl_s + ko, 16, 1024), idesc, 1u);
      }
      tc_commit(&bar_s[j & 1]);
    }
  };

  const int r = 32 * sub + lane;                              // this thread's row / TMEM lane
  auto position = [&](int row) { return PREFIX ? p_first + row / GP : p_first + min(row / GP, p_last - p_first); };
  const int pr = position(r), pw_min = position(32 * sub), pw_max = position(32 * sub + 31);
  constexpr int HC = kTcTok / 2;                               // score columns per thread
  constexpr int OH = D / 2;                                    // output columns per thread
  float mx = -INFINITY;
  uint64_t l2 = f2_pack(0.f, 0.f);                             // running row sum, two partial lanes
  bool failed = false;
  int qk_issued = 0, qk_done = 0, o_issued = 0, o_done = 0;

  // The row's scores are those of its scaled query: times q_back.
  float q_back;
  if constexpr (PREFIX) {
    q_back = reinterpret_cast<const float *>(q_tile + 2 * C::Q_BYTES)[r];
    if (__syncthreads_or(!mbar_wait_bounded(bar_q, 0))) {
      failed = true;
      n_tiles = 0;
    }
  } else {
    q_back = nrm_s[r];
    __syncthreads();   // the norms go over it
  }
  const uint64_t back2 = f2_pack(q_back, q_back);
  if (n_tiles > 0) {
    store_norm();
    if (n_tiles > 1) fetch_norm(1);
    stage_qk(0);
    ++qk_issued;
  }
  for (int it = 0; it < n_tiles; ++it) {
    const int t0 = tile_t0(it);
    // QK(it) must be complete: its S buffer is read below and the K tile is
    // free.  Every thread waits on the mbarrier itself, so no block barrier
    // follows: a wait that gave up is recorded in fail_s[it % 2], which all
    // threads read after the block barrier that ends the iteration and leave
    // the loop together.  (A flag per iteration parity: the writes of
    // iteration it + 2 come after every thread has passed the barrier that
    // ends iteration it + 1, i.e. after every read of iteration it.)
    if (mbar_wait_bounded(&bar_s[it & 1], (it >> 1) & 1))
      ++qk_done;
    else
      fail_s[it & 1] = 1;
    tc_fence_after();
    // The next tile's QK runs on the tensor cores under this tile's softmax.
    // Its block barrier also publishes this tile's norms, stored after the
    // previous iteration's last barrier; the last tile needs a barrier of
    // its own for that.
    if (it + 1 < n_tiles) {
      stage_qk(it + 1);
      ++qk_issued;
    } else {
      __syncthreads();
    }

    // ---- softmax on this thread's half row of S(it) ----
    // Arithmetic on float pairs (f32x2: one instruction per two columns);
    // the norms are read as 16-byte broadcasts.
    const ulonglong2 *nk4 = reinterpret_cast<const ulonglong2 *>(nrm_s + HC * half);
    const ulonglong2 *nv4 = reinterpret_cast<const ulonglong2 *>(nrm_s + kTcTok + HC * half);
    const int c0 = t0 + HC * half;                             // token of this thread's first column
    float x[HC];
    uint32_t sraw[HC / 16][16];
#pragma unroll
    for (int c = 0; c < HC / 16; ++c) tc_ld16_nowait(tmem + (it & 1) * 64 + HC * half + lane_off + 16 * c, sraw[c]);
    tc_wait_ld();
#pragma unroll
    for (int c = 0; c < HC / 16; ++c) {
      float v[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(sraw[c][j]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const ulonglong2 n = nk4[4 * c + k];
        f2_unpack(f2_mul(f2_pack(v[4 * k], v[4 * k + 1]), n.x), x[16 * c + 4 * k], x[16 * c + 4 * k + 1]);
        f2_unpack(f2_mul(f2_pack(v[4 * k + 2], v[4 * k + 3]), n.y), x[16 * c + 4 * k + 2], x[16 * c + 4 * k + 3]);
      }
    }
    if (t0 + kTcTok - 1 > pw_min || t0 + kTcTok > tend) {   // uniform over the warp pair
#pragma unroll
      for (int j = 0; j < HC; ++j)
        if (c0 + j > pr || c0 + j >= tend) x[j] = -INFINITY;
    }
    if constexpr (WIN) {
      // Some row of the warp pair has left part of this tile behind, and the
      // tile is not all sinks.
      if (pw_max >= a.window && t0 <= pw_max - a.window && t0 + kTcTok > a.n_sink) {
        const int behind = pr >= a.window ? pr - a.window : -1;   // the row's last token behind its window
#pragma unroll
        for (int j = 0; j < HC; ++j)
          if (c0 + j <= behind && c0 + j >= a.n_sink) x[j] = -INFINITY;
      }
    }
    float tmx = -INFINITY;
#pragma unroll
    for (int j = 0; j < HC; ++j) tmx = fmaxf(tmx, x[j]);

    // PV(it - 1) must be complete before O is rescaled and the V tile
    // reused (P(it) goes to the other S buffer, which PV(it - 1) does not read).
    auto wait_pv = [&]() {
      if (o_issued > o_done) {
        if (mbar_wait_bounded(bar_o, o_done & 1))
          ++o_done;
        else
          fail_s[it & 1] = 1;
        tc_fence_after();
      }
    };
    // The row maximum over both column halves, exchanged with the partner
    // warp through the consumed S buffer: each thread leaves its value in a
    // column of its own half of S (already read) that the partner overwrites
    // with its P later, and reads the partner's from a column that it
    // overwrites itself later.  Half 0 reads S columns 0..31 and writes P
    // into 0..15 and 32..47; half 1 reads 32..63 and writes 16..31, 48..63.
    const uint32_t s_col = tmem + (it & 1) * 64 + lane_off;
    tc_st1(s_col + 16 + 16 * half, __float_as_uint(tmx));
    tc_wait_st();
    tc_fence_before();
    named_barrier(1 + sub, 64);
    tc_fence_after();
    tmx = fmaxf(tmx, __uint_as_float(tc_ld1(s_col + 16 + 16 * (half ^ 1))));
    tc_wait_ld();
    const float nm = fmaxf(mx, tmx * q_back);
    const float base = nm == -INFINITY ? 0.f : nm;
    const float f = ex2f(mx - base);                            // 0 while mx = -inf
    const bool moved = __any_sync(0xffffffffu, nm > mx);       // the same in both warps of the pair
    mx = nm;
    const uint64_t base2 = f2_pack(-base, -base);
    l2 = f2_mul(l2, f2_pack(f, f));
    // P = p s^V as float16 hi and lo parts: tokens 2i, 2i + 1 of the tile in
    // column i of the hi block (columns 0..31) and of the lo block (32..63).
    uint32_t phi[HC / 2], plo[HC / 2];
#pragma unroll
    for (int c = 0; c < HC / 8; ++c) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = 8 * c + 2 * k;
        float p0, p1;
        f2_unpack(f2_fma(f2_pack(x[j], x[j + 1]), back2, base2), p0, p1);
        const uint64_t p2 = f2_pack(ex2f(p0), ex2f(p1));
        l2 = f2_add(l2, p2);
        const ulonglong2 n = nv4[j >> 2];
        f2_unpack(f2_mul(p2, (k & 1) ? n.y : n.x), p0, p1);
        if constexpr (WIN) {   // a token that is not seen weighs nothing, whatever its norm holds
          p0 = x[j] == -INFINITY ? 0.f : p0;
          p1 = x[j + 1] == -INFINITY ? 0.f : p1;
        }
        const __half2 h = __floats2half2_rn(p0, p1);
        const float2 hf = __half22float2(h);
        phi[4 * c + k] = *reinterpret_cast<const uint32_t *>(&h);
        plo[4 * c + k] = pack_f16x2(p0 - hf.x, p1 - hf.y);
      }
    }
    tc_st16u(s_col + 16 * half, phi);
    tc_st16u(s_col + 32 + 16 * half, plo);
    tc_wait_st();
    wait_pv();

    if (moved && it > 0) {
#pragma unroll 1
      for (int c = 0; c < OH / 16; ++c) {
        float v[16];
        tc_ld16(t_o + OH * half + lane_off + 16 * c, v);
        const uint64_t f2 = f2_pack(f, f);
#pragma unroll
        for (int j = 0; j < 16; j += 2) f2_unpack(f2_mul(f2_pack(v[j], v[j + 1]), f2), v[j], v[j + 1]);
        tc_st16(t_o + OH * half + lane_off + 16 * c, v);
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
    }
    tc_expand<D, false>(vc, vt, nullptr, a, tid);
    if (it + 1 < n_tiles) tc_fetch<D>(vc, vb, tile_t0(it + 1), tend, tid);
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (fail_s[it & 1]) {   // the same value for every thread
      failed = true;
      break;
    }
    // Every thread is past the softmax of tile it: its norms can be replaced.
    if (it + 1 < n_tiles) {
      store_norm();
      if (it + 2 < n_tiles) fetch_norm(it + 2);
    }
    if (tid == 0) {
      constexpr uint32_t idesc = tc_idesc(kTcRows, D, 1);
      const uint32_t pa = tmem + (it & 1) * 64;               // P(it): hi in columns 0..31, lo in 32..63
#pragma unroll
      for (int ks = 0; ks < kTcTok / 16; ++ks) {
        const uint64_t bd = tc_desc(v_s + ks * 2048, KBLK, 1024);
        tc_mma_ts(t_o, pa + 8 * ks, bd, idesc, (it > 0 || ks > 0) ? 1u : 0u);
        tc_mma_ts(t_o, pa + 32 + 8 * ks, bd, idesc, 1u);
      }
      tc_commit(bar_o);
    }
    ++o_issued;
  }

  if (!failed && o_issued > o_done) {
    const bool ok = mbar_wait_bounded(bar_o, o_done & 1);
    if (__syncthreads_or(!ok))
      failed = true;
    else
      ++o_done;
  }
  if (failed) {
    if (tid == 0) {
      atomicOr(&g_decode_error, kErrWaitTimeout);
      for (int j = qk_done; j < qk_issued; ++j)
        if (!mbar_wait_bounded(&bar_s[j & 1], (j >> 1) & 1)) break;
      if (o_issued > o_done) mbar_wait_bounded(bar_o, o_done & 1);
    }
  } else if constexpr (PREFIX) {
    // ---- epilogue: one partial state per row ----
    tc_fence_after();
    __syncthreads();
    float *xchg = reinterpret_cast<float *>(q_hi);   // [2][kTcRows] row sums; the query tiles are free
    float l0, l1;
    f2_unpack(l2, l0, l1);
    xchg[half * kTcRows + r] = l0 + l1;
    __syncthreads();
    const int row = kTcRows * qt + r;
    const bool live = row < a.batch * a.group;
    const long long query = live ? static_cast<long long>(row / a.group) * a.hq + kvh * a.group + row % a.group : 0;
    const long long slot = query * a.slot_stride + b;
    const float unit = a.acc_unit / v_scale;
#pragma unroll 1
    for (int c = 0; c < OH / 16; ++c) {
      float v[16];
      if (n_tiles > 0) {
        tc_ld16(t_o + OH * half + lane_off + 16 * c, v);
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = 0.f;
      }
      if (live) {
        float4 *dst = reinterpret_cast<float4 *>(a.ws_acc + slot * D + OH * half + 16 * c);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          dst[j] = make_float4(v[4 * j] * unit, v[4 * j + 1] * unit, v[4 * j + 2] * unit, v[4 * j + 3] * unit);
      }
    }
    if (live && half == 0)
      a.ws_ml[slot] = make_float2(mx == -INFINITY ? -INFINITY : mx * 0.69314718055994531f, xchg[r] + xchg[kTcRows + r]);
  } else {
    // ---- epilogue, 32 rows per pass: O / l from TMEM, rotate back, store ----
    tc_fence_after();
    __syncthreads();
    float *xchg = reinterpret_cast<float *>(q_hi);   // [2][kTcRows] row sums; the query tiles are free
    float l0, l1;
    f2_unpack(l2, l0, l1);
    const float l = l0 + l1;
    xchg[half * kTcRows + r] = l;
    __syncthreads();
    const float lt = l + xchg[(half ^ 1) * kTcRows + r];
    const float inv = lt > 0.f ? a.out_unit / lt / v_scale : 0.f;
    for (int pass = 0; pass < kTcRows / 32; ++pass) {
      __syncthreads();   // scratch (over the K and V tiles) is free
      if (sub == pass) {
#pragma unroll 1
        for (int c = 0; c < OH / 16; ++c) {
          float v[16];
          if (n_tiles > 0) {
            tc_ld16(t_o + OH * half + lane_off + 16 * c, v);
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = 0.f;
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) scratch[lane * D + OH * half + 16 * c + j] = v[j] * inv;
        }
      }
      __syncthreads();
      rotate_inverse_rows<D, FULL>(scratch, 32, a.params_v + static_cast<size_t>(kvh) * 2 * D, tid, kTcThreads);
      for (int i = tid; i < 32 * D; i += kTcThreads) {
        const int m = 32 * pass + i / D, e = i % D;
        const int tl = m / GP, h = m % GP;
        if (h < G && tq0 + tl < a.tq) {
          const long long row = (static_cast<long long>(b) * a.tq + tq0 + tl) * a.hq + kvh * G + h;
          static_cast<T *>(a.out)[row * D + e] = from_f32<T>(scratch[i]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // kPfPrefix overlaps the split over the rows' own caches, launched before
  // it; the combine waits for this grid, so this grid ends after that one.
  if constexpr (PREFIX) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS));
}

template <typename T, int D, bool FULL, int GP, int KIND>
int launch_prefill_tc(const PrefillArgs &a, cudaStream_t stream) {
  using C = TcCfg<D>;
  auto kernel = prefill_tc_kernel<T, D, FULL, GP, KIND>;
  static std::atomic<unsigned long long> allowed;
  cudaError_t e = allow_smem(allowed, reinterpret_cast<const void *>(kernel), C::SMEM);
  if (e != cudaSuccess) return set_error(ISOQ_ERR_CUDA, "prefill (tcgen05): %s", cudaGetErrorString(e));
  constexpr int BQ = kTcRows / GP;
  dim3 grid((a.tq + BQ - 1) / BQ, a.hkv, a.batch);
  kernel<<<grid, kTcThreads, C::SMEM, stream>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(ISOQ_ERR_CUDA, "prefill (tcgen05) launch: %s", cudaGetErrorString(e));
  return ISOQ_OK;
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

inline uint16_t pf_half_bits(double v) {
  const __half h = __double2half(v);
  return *reinterpret_cast<const uint16_t *>(&h);
}

// alpha in [1, 2) minimising the largest relative float16 rounding error of
// alpha c_k over the unit-variance 3-bit centroids (searched once), the
// float16 tables of alpha c_k and of its residual alpha c_k - fp16(alpha c_k)
// (below 2^-15 of the centroid; subnormal float16 values where small).
struct PfTables {
  double alpha;
  uint32_t lo0, lo1, hi0, hi1;
  uint32_t rlo0, rlo1, rhi0, rhi1;
};

inline const PfTables &pf_tables() {
  static PfTables tb;
  static std::once_flag once;
  std::call_once(once, [] {
    double c[8];
    codebook_unit_f64(3, c);
    double best = 1.0, best_err = 1.0;
    const int steps = 1 << 20;
    for (int i = 0; i < steps; ++i) {
      const double al = 1.0 + static_cast<double>(i) / steps;
      double err = 0.0;
      for (int k = 4; k < 8 && err < best_err; ++k) {
        const double v = al * c[k];
        const double r = static_cast<double>(__half2float(__double2half(v)));
        err = std::fmax(err, std::fabs(r - v) / v);
      }
      if (err < best_err) {
        best_err = err;
        best = al;
      }
    }
    tb.alpha = best;
    tb.lo0 = tb.lo1 = tb.hi0 = tb.hi1 = 0;
    tb.rlo0 = tb.rlo1 = tb.rhi0 = tb.rhi1 = 0;
    for (int k = 0; k < 8; ++k) {
      const double v = best * c[k];
      const uint16_t hb = pf_half_bits(v);
      const double vh = static_cast<double>(__half2float(*reinterpret_cast<const __half *>(&hb)));
      const uint16_t rb = pf_half_bits(v - vh);
      const int sh = 8 * (k % 4);
      (k < 4 ? tb.lo0 : tb.lo1) |= static_cast<uint32_t>(hb & 0xFFu) << sh;
      (k < 4 ? tb.hi0 : tb.hi1) |= static_cast<uint32_t>(hb >> 8) << sh;
      (k < 4 ? tb.rlo0 : tb.rlo1) |= static_cast<uint32_t>(rb & 0xFFu) << sh;
      (k < 4 ? tb.rhi0 : tb.rhi1) |= static_cast<uint32_t>(rb >> 8) << sh;
    }
  });
  return tb;
}

template <typename T, int D, bool FULL, int KIND>
int run_prefill_g(const PrefillArgs &a, cudaStream_t st) {
  switch (a.group) {
    case 1: return launch_prefill_tc<T, D, FULL, 1, KIND>(a, st);
    case 2: return launch_prefill_tc<T, D, FULL, 2, KIND>(a, st);
    case 4: return launch_prefill_tc<T, D, FULL, 4, KIND>(a, st);
    default: return launch_prefill_tc<T, D, FULL, 8, KIND>(a, st);
  }
}

template <typename T, int KIND>
int run_prefill_t(int d, int variant, const PrefillArgs &a, cudaStream_t st) {
  if (d == 128)
    return variant == ISOQ_FULL ? run_prefill_g<T, 128, true, KIND>(a, st) : run_prefill_g<T, 128, false, KIND>(a, st);
  return variant == ISOQ_FULL ? run_prefill_g<T, 256, true, KIND>(a, st) : run_prefill_g<T, 256, false, KIND>(a, st);
}

// The kernel's tables and units of alpha.
inline void prefill_tables(PrefillArgs &a, int d) {
  const PfTables &tb = pf_tables();
  a.lut_lo0 = tb.lo0;
  a.lut_lo1 = tb.lo1;
  a.lut_hi0 = tb.hi0;
  a.lut_hi1 = tb.hi1;
  a.res_lo0 = tb.rlo0;
  a.res_lo1 = tb.rlo1;
  a.res_hi0 = tb.rhi0;
  a.res_hi1 = tb.rhi1;
  a.out_unit = static_cast<float>(1.0 / (tb.alpha * d));
  a.acc_unit = static_cast<float>(1.0 / (tb.alpha * std::sqrt(static_cast<double>(d))));
  a.score_unit = static_cast<float>(a.score_unit / (tb.alpha * std::sqrt(static_cast<double>(d))));
}

template <int KIND>
int run_prefill(int d, int variant, PrefillArgs a, cudaStream_t st) {
  prefill_tables(a, d);
  return run_prefill_t<__half, KIND>(d, variant, a, st);
}

// Checks the arguments of a prefill entry point and fills in the kernel's.
inline int prefill_args(const void *q_dev, int dtype, const uint8_t *packed_k_dev, const uint8_t *packed_v_dev,
                        const uint16_t *norms_k_dev, const uint16_t *norms_v_dev, const int32_t *seq_lens_dev, int B,
                        int Tq, int Hq, int Hkv, int64_t Tmax, int d, int bits, int variant,
                        const float *params_k_dev, const float *params_v_dev, float scale, void *out_dev,
                        PrefillArgs *out) {
  if (d != 128 && d != 256) return set_error(ISOQ_ERR_UNSUPPORTED, "prefill: d=%d (128 or 256)", d);
  if (bits != 3) return set_error(ISOQ_ERR_UNSUPPORTED, "prefill: bits=%d (3)", bits);
  if (!supported_decode_variant(variant)) return set_error(ISOQ_ERR_UNSUPPORTED, "variant=%d", variant);
  if (dtype != ISOQ_F16) return set_error(ISOQ_ERR_UNSUPPORTED, "prefill: dtype=%d (float16 queries)", dtype);
  if (B <= 0 || Tq < 0 || Hq <= 0 || Hkv <= 0 || Tmax <= 0)
    return set_error(ISOQ_ERR_INVALID_ARG, "B, Hq, Hkv and Tmax must be positive, Tq >= 0");
  if (Hq % Hkv) return set_error(ISOQ_ERR_INVALID_ARG, "Hq %% Hkv != 0");
  const int G = Hq / Hkv;
  if (G != 1 && G != 2 && G != 4 && G != 8)
    return set_error(ISOQ_ERR_UNSUPPORTED, "prefill: Hq/Hkv=%d (1, 2, 4 or 8)", G);
  if (Tmax >= (1ll << 31) || B > 65535 || Hkv > 65535 || Tq > (1 << 24))
    return set_error(ISOQ_ERR_INVALID_ARG, "shape too large");
  if (Tmax % 8) return set_error(ISOQ_ERR_UNSUPPORTED, "prefill: Tmax %% 8 != 0");
  if (!q_dev || !packed_k_dev || !packed_v_dev || !norms_k_dev || !norms_v_dev || !seq_lens_dev ||
      !params_k_dev || !params_v_dev || !out_dev)
    return set_error(ISOQ_ERR_INVALID_ARG, "null pointer");
  if (!aligned(packed_k_dev, 16) || !aligned(packed_v_dev, 16) ||
      !aligned(params_k_dev, 16) || !aligned(params_v_dev, 16) ||
      !aligned(q_dev, 4) || !aligned(out_dev, 4) || !aligned(norms_k_dev, 2) ||
      !aligned(norms_v_dev, 2) || !aligned(seq_lens_dev, 4))
    return set_error(ISOQ_ERR_UNSUPPORTED, "misaligned pointer");
  if (!std::isfinite(scale)) return set_error(ISOQ_ERR_INVALID_ARG, "scale is not finite");
  PrefillArgs &a = *out;
  a.q = q_dev;
  a.packed_k = packed_k_dev;
  a.packed_v = packed_v_dev;
  a.norms_k = norms_k_dev;
  a.norms_v = norms_v_dev;
  a.seq_lens = seq_lens_dev;
  a.params_k = params_k_dev;
  a.params_v = params_v_dev;
  a.out = out_dev;
  a.tmax = Tmax;
  a.batch = B;
  a.tq = Tq;
  a.hq = Hq;
  a.hkv = Hkv;
  a.group = G;
  a.score_unit = static_cast<float>(scale * 1.4426950408889634);
  return ISOQ_OK;
}
