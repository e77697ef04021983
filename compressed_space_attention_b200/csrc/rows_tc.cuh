// Attention of 128 query rows over packed K/V at d = 128, 3 bits, on the
// 5th-generation tensor cores, with the query tile in tensor memory.  Included
// by isoq_serve.cu inside namespace isoq::decode, after prefill.cuh, whose
// arguments, tables and tile layouts it shares.
//
// The mathematics is prefill.cuh's: S = Q~hi K~hi^T + Q~lo K~hi^T + Q~hi K~lo^T
// with float16 hi and lo parts of the rotated query (each row scaled by a power
// of two: query_scale) and of the centroids, x = S s^K scale, p = 2^(x - r),
// O += P_hi V~ + P_lo V~ with P = p s^V.
//
// Why the queries sit in tensor memory: with both operands in shared memory a
// 128 x 128 x 16 product reads 8 KB in its 64 cycles, all that shared memory
// delivers, and the unpacking and the softmax starve (a form with two 128-row
// tiles per CTA and the queries in shared memory took 225 to 299 us for 64
// batch rows x 8 heads behind 65,536 tokens, no faster than the two-CTA form
// of prefill.cuh).  From tensor memory a product reads 4 KB, and the 128 KB
// that two query tiles took hold second buffers of K and V.
//
// Roles (16 warps, four to a scheduler, 128 registers a thread):
//   warps 0-7   softmax: two threads per row, warp w and w + 4 on TMEM lanes
//               32 (w mod 4) .., columns 0-63 and 64-127 of the scores.  The
//               weights go over the scores (per 32 tokens 16 columns of hi
//               and 16 of lo parts).  The reference r moves only when a score
//               passes it, and then to that score + 8: p <= 1 always, and O,
//               which follows, is seldom rescaled.  s^V is scaled by a power
//               of two (value_scale), so P stays far from float16's subnormal
//               numbers for all that headroom.
//   warps 8-14  unpack: codes (fetched one tile ahead into registers) to
//               float16 centroids and residuals of K, centroids of V, and the
//               norms.
//   warp 15     issues the products: S(j + 1), PV(j).
// Tensor memory (512 columns): S (2 x 128), O, Q~hi, Q~lo.  Shared memory: two
// buffers of K (hi, lo) and V, 192 KB, and four of the norms.
//
// Bound: the tensor core, five products of 128 x 128 x 128 per 128 tokens (2.5
// times the operator's arithmetic), 57 % busy: about 4,200 cycles per 128 rows
// and tokens, of which the score products take 2,200 and the value products
// 1,350 (1,536 and 1,024 at the tensor core's rate), the softmax of a tile 3,300
// beside them.  64 batch rows x 8 heads behind 65,536 tokens, 4 KV heads: 170 us
// on the GPU, 184 a call with the own caches' split and the host's work; 2 x
// 2,048 queries, 32 over 4 heads, window 2,048: 350 us.
//
// kPfWindow: rows are positions x heads of a chunk; rotation of the queries
// before and of the output after the loop, both in the CTA.  Where the chunk
// has fewer row tiles than there are SMs, a cluster of CTAs shares the tokens
// of a row tile and merges its partial states in shared memory (256 queries,
// 32 over 4 heads, window 1,024: 39.4 us with one CTA per row tile, 30.8 with
// two).  kPfPrefix: rows are a KV head's batch x group; one partial state per
// row and split.
//
// Every wait is bounded.  A role whose wait gives up records kErrWaitTimeout
// and stops; the others' waits then run out as well, the products already
// issued are waited for (bounded), tensor memory is freed and the CTA ends.

constexpr int kRowsWarps = 16, kRowsUnpackWarps = 7;
constexpr int kRowsThreads = 32 * kRowsWarps;
constexpr int kRowsTok = 128;
static_assert(kTcRows / kRowsWarps == 8, "rows of a warp: a byte of flags each");
constexpr float kRowsHeadroom = 8.f;   // log2: how far the reference is set above the score that moves it

struct RowsCfg {
  static constexpr int D = 128, PB = 48;
  static constexpr int KV = kRowsTok * D * 2;              // one K, K-residual or V tile
  static constexpr int STAGE = 3 * KV;                     // K hi, K lo, V
  static constexpr int OFF_NORM = 2 * STAGE;               // [4][s^K unit, s^V][128] float32
  static constexpr int OFF_XCHG = OFF_NORM + 4 * 2 * kRowsTok * 4;   // [2][2][128] float32
  static constexpr int OFF_BAR = OFF_XCHG + 2 * 2 * kTcRows * 4;
  static constexpr int OFF_BACK = OFF_BAR + 24 * 8;        // [128] float32, the rows' inverse query scales
  static constexpr int SMEM = OFF_BACK + kTcRows * 4;
  static_assert(SMEM <= 232448, "shared memory of one CTA");
};

// 32 columns of this warp's TMEM lanes, not waited for; tc_ld32_done waits and
// ties the values to the wait.
__device__ __forceinline__ void tc_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

__device__ __forceinline__ void tc_ld32_done(uint32_t (&r)[32]) {
  tc_wait_ld();
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                      "+r"(r[i + 6]), "+r"(r[i + 7]));
}

__device__ __forceinline__ void tc_st8u(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Bits 0 .. n - 1.
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u); }

template <int KIND, bool FULL, bool CLUSTER = false>
__global__ void __launch_bounds__(kRowsThreads, 1) rows_tc_kernel(const PrefillArgs a) {
  using C = RowsCfg;
  constexpr bool WIN = KIND == kPfWindow;
  constexpr int KBLK = kRowsTok * 128;
  extern __shared__ unsigned char smem[];
  if (smem_u32(smem) & 1023u) {   // uniform over the grid: nothing allocated yet
    if (threadIdx.x == 0) atomicOr(&g_decode_error, kErrSmemAlign);
    return;
  }
  float *norms = reinterpret_cast<float *>(smem + C::OFF_NORM);
  float *xchg = reinterpret_cast<float *>(smem + C::OFF_XCHG);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
  float *q_back = reinterpret_cast<float *>(smem + C::OFF_BACK);
  uint64_t *k_full = bars /* [2] */, *v_full = bars + 2 /* [2] */, *k_free = bars + 4 /* [2] */,
           *v_free = bars + 6 /* [2] */, *s_full = bars + 8 /* [2] */, *p_full = bars + 10 /* [2] */,
           *n_full = bars + 12 /* [4] */, *o_done = bars + 16, *all_done = bars + 17;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 18);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ranks = CLUSTER ? static_cast<int>(cluster_size()) : 1, rank = CLUSTER ? static_cast<int>(cluster_rank()) : 0;
  const int qt = CLUSTER ? blockIdx.x / ranks : blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
  const int G = a.group;

  // ---- the CTA's rows and tokens ----
  const int32_t *lens = WIN ? a.seq_lens + b : a.prefix_len;
  // (Positions follow the length as given, also beyond the room; below 0 as 0.)
  const int given = *lens < 0 ? 0 : *lens;
  const int len = given > a.tmax ? static_cast<int>(a.tmax) : given;
  const int per_cta = kTcRows / (WIN ? G : 1);               // kPfWindow: positions of the CTA
  const int tq0 = WIN ? qt * per_cta : 0;
  const int p_first = WIN ? given - a.tq + tq0 : 0;          // position of the CTA's first row
  const int total_rows = WIN ? 0 : a.batch * G;
  int tend, t_base = 0, n_sink_tiles = 0, win_tile = 0, sink = 0, lo = 0, n_iter, j_base = 0;
  if constexpr (WIN) {
    const int p_last = tq0 + per_cta > a.tq ? given - 1 : p_first + per_cta - 1;
    tend = p_last + 1 < len ? p_last + 1 : len;
    if (tend < 0) tend = 0;
    const int all = (tend + kRowsTok - 1) / kRowsTok;
    sink = a.n_sink < tend ? a.n_sink : tend;
    lo = a.window == 0 ? tend : (p_first >= a.window ? p_first - a.window + 1 : 0);   // (no window holds no token)
    if (lo > tend) lo = tend;
    n_iter = all;
    if (lo > sink) {
      n_sink_tiles = (sink + kRowsTok - 1) / kRowsTok;
      win_tile = lo / kRowsTok > n_sink_tiles ? lo / kRowsTok : n_sink_tiles;
      n_iter = n_sink_tiles + (all > win_tile ? all - win_tile : 0);
    }
    // This CTA's share of the cluster's tiles.
    if constexpr (CLUSTER) {
      j_base = n_iter * rank / ranks;
      n_iter = n_iter * (rank + 1) / ranks - j_base;
    }
  } else {
    const long long first = static_cast<long long>(b) * a.chunk;
    t_base = first < len ? static_cast<int>(first) : len;
    tend = len - t_base > a.chunk ? t_base + a.chunk : len;
    n_iter = (tend - t_base + kRowsTok - 1) / kRowsTok;
  }
  auto tile_t0 = [&](int j) {
    if constexpr (WIN) {
      const int v = j_base + j;
      return kRowsTok * (v < n_sink_tiles ? v : v - n_sink_tiles + win_tile);
    } else {
      return t_base + kRowsTok * j;
    }
  };
  // Row i of the CTA: its query (row of q and out), or -1.
  auto query_of = [&](int i) -> long long {
    if constexpr (WIN) {
      const int t = tq0 + i / G;
      return t < a.tq ? (static_cast<long long>(b) * a.tq + t) * a.hq + kvh * G + i % G : -1;
    } else {
      const int r = kTcRows * qt + i;
      return r < total_rows ? static_cast<long long>(r / G) * a.hq + kvh * G + r % G : -1;
    }
  };
  const long long cache0 = WIN ? (static_cast<long long>(b) * a.hkv + kvh) * a.tmax : kvh * a.head_stride;

  {
    uint32_t mx = 0;
    auto among = [&](int t0, int t1) {
      const uint32_t u = largest_norm<kRowsThreads>(a.norms_v + cache0, t0, t1, tid);
      mx = u > mx ? u : mx;
    };
    if constexpr (WIN) {
      // Of the CTA's tiles (n0 of sinks, then the others) the tokens that some
      // row sees: with a gap behind the sinks, those before `sink` or from lo on.
      const int n0 = max(min(n_sink_tiles - j_base, n_iter), 0);
      const int a0 = kRowsTok * j_base, b0 = a0 + kRowsTok * n0, a1 = tile_t0(n0), b1 = min(a1 + kRowsTok * (n_iter - n0), tend);
      if (n0 > 0) {
        among(a0, min(b0, sink));
        among(max(a0, lo), min(b0, tend));
      }
      among(lo > sink ? max(a1, lo) : a1, b1);
    } else {
      among(t_base, tend);
    }
    if (lane == 0) reinterpret_cast<uint32_t *>(xchg)[warp] = mx;
  }
  if (warp == kRowsWarps - 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(k_full + t, kRowsUnpackWarps);
      mbar_init(v_full + t, kRowsUnpackWarps);
      mbar_init(k_free + t, 1);
      mbar_init(v_free + t, 1);
      mbar_init(s_full + t, 1);
      mbar_init(p_full + t, 8);
    }
    for (int t = 0; t < 4; ++t) mbar_init(n_full + t, kRowsUnpackWarps);
    mbar_init(o_done, 1);
    mbar_init(all_done, 1);
    mbar_fence_init();
  }

  // ---- queries: one warp per row, rotated in registers (lane: 4 dims), split,
  // and passed through shared memory (16-byte chunk c of a row's 256 bytes at
  // c ^ (row mod 16)) to the row's own thread, which stores them to TMEM ----
  const float inv_sqrt_d = rsqrtf(128.f);
  {
    const float *prm = a.params_k + static_cast<size_t>(kvh) * 256 + 8 * lane;
    const Quat ql = load_quat(prm), qr = load_quat(prm + 4);
    auto rotated = [&](long long row) {
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      if (row >= 0) {
        const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const __half *>(a.q) + row * 128 + 4 * lane);
        const float2 f0 = __half22float2(*reinterpret_cast<const __half2 *>(&u.x));
        const float2 f1 = __half22float2(*reinterpret_cast<const __half2 *>(&u.y));
        x[0] = f0.x;
        x[1] = f0.y;
        x[2] = f1.x;
        x[3] = f1.y;
      }
      const float y0 = x[0] + x[1], y1 = x[0] - x[1], y2 = x[2] + x[3], y3 = x[2] - x[3];
      x[0] = y0 + y2;
      x[1] = y1 + y3;
      x[2] = y0 - y2;
      x[3] = y1 - y3;
#pragma unroll
      for (int lm = 1; lm < 32; lm <<= 1) {
        const float sgn = (lane & lm) ? -1.f : 1.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = fmaf(x[e], sgn, __shfl_xor_sync(0xffffffffu, x[e], lm));
      }
      const Quat v{x[0] * inv_sqrt_d, x[1] * inv_sqrt_d, x[2] * inv_sqrt_d, x[3] * inv_sqrt_d};
      return block_forward(ql, qr, v, FULL);
    };
    auto stage = [&](int i, const Quat &y) {
      const __half2 h0 = __floats2half2_rn(y.w, y.x), h1 = __floats2half2_rn(y.y, y.z);
      const float2 f0 = __half22float2(h0), f1 = __half22float2(h1);
      unsigned char *at = smem + 256 * i + 16 * ((lane >> 1) ^ (i & 15)) + 8 * (lane & 1);
      *reinterpret_cast<uint2 *>(at) =
          make_uint2(*reinterpret_cast<const uint32_t *>(&h0), *reinterpret_cast<const uint32_t *>(&h1));
      *reinterpret_cast<uint2 *>(at + 256 * kTcRows) =
          make_uint2(pack_f16x2(y.w - f0.x, y.x - f0.y), pack_f16x2(y.y - f1.x, y.z - f1.y));
    };
    auto largest = [](const Quat &y) { return fmaxf(fmaxf(fabsf(y.w), fabsf(y.x)), fmaxf(fabsf(y.y), fabsf(y.z))); };
    // Bit k: row k of the warp has a component of 1/4 or more (or no query),
    // bit 8 + k: one of 2^15 or more.  Rows that need a scale are done again, so
    // that no maximum over the warp stands in every row's chain.
    uint32_t range = 0;
    for (int i = warp, k = 0; i < kTcRows; i += kRowsWarps, ++k) {
      const long long row = query_of(i);
      const Quat y = rotated(row);
      const float big = largest(y);
      range |= (row < 0 || big >= 0.25f ? 1u : 0u) << k | (big >= 32768.f ? 256u : 0u) << k;
      stage(i, y);
    }
    range = __reduce_or_sync(0xffffffffu, range);
    if (lane < kTcRows / kRowsWarps) q_back[warp + kRowsWarps * lane] = 1.f;
    __syncwarp();
#pragma unroll 1
    for (uint32_t redo = (~range & 255u) | range >> 8; redo; redo &= redo - 1) {
      const int i = warp + kRowsWarps * (__ffs(redo) - 1);
      const Quat y = rotated(query_of(i));
      float back;   // (not negative: the maximum is ordered as integers)
      const float sc = query_scale(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(largest(y)))), back);
      stage(i, Quat{y.w * sc, y.x * sc, y.y * sc, y.z * sc});
      if (lane == 0) q_back[i] = back;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t t_o = tmem + 256, t_q = tmem + 384;       // Q~hi 64 columns, Q~lo 64
  const uint32_t lane_off = static_cast<uint32_t>(32 * (warp & 3)) << 16;
  uint32_t norm_max = 0;
#pragma unroll
  for (int w = 0; w < kRowsWarps; ++w) {
    const uint32_t u = reinterpret_cast<const uint32_t *>(xchg)[w];
    norm_max = u > norm_max ? u : norm_max;
  }
  const float v_scale = value_scale(norm_max);
  if (warp < 8) {   // warps 0-3 the hi parts, 4-7 the lo parts
    const int i = 32 * (warp & 3) + lane, part = warp >> 2;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      uint32_t r[16];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint4 u = *reinterpret_cast<const uint4 *>(smem + 256 * (kTcRows * part + i) + 16 * ((4 * c + k) ^ (i & 15)));
        r[4 * k] = u.x;
        r[4 * k + 1] = u.y;
        r[4 * k + 2] = u.z;
        r[4 * k + 3] = u.w;
      }
      tc_st16u(t_q + 64 * part + 16 * c + lane_off, r);
    }
    tc_wait_st();
  }
  tc_fence_before();
  __syncthreads();   // Q~ is in place; the buffers are free
  tc_fence_after();
  bool ok = true;

  if (warp < 8) {
    // ================= softmax =================
    const int half = warp >> 2, i = 32 * (warp & 3) + lane;    // column half, row
    // The last token the row sees, and the last one behind its window.
    int p_row = 0x7FFFFFFF, behind = -1, n_sink = 0;
    if constexpr (WIN) {
      p_row = p_first + min(i / G, a.tq - 1 - tq0);   // (a dead row: the last one's)
      behind = p_row >= a.window ? p_row - a.window : -1;
      n_sink = a.n_sink;
    }
    const int last = p_row < tend - 1 ? p_row : tend - 1;
    const float back = q_back[i];   // the row's scores are those of its scaled query: times back
    float ref = -INFINITY;
    uint64_t la = f2_pack(0.f, 0.f), lb = la;
    auto tiles = [&](auto scaled) {
      constexpr bool SCALED = decltype(scaled)::value;
      for (int j = 0; j < n_iter; ++j) {
        // (After a wait that gave up the loop goes on without waiting, so that
        // the barriers of a pair of warps always meet.)
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(s_full + (j & 1), (j >> 1) & 1) &&
                                                 mbar_wait_bounded(n_full + (j & 3), (j >> 2) & 1));
        tc_fence_after();
        const uint32_t t_s = tmem + 128 * (j & 1) + 64 * half + lane_off;
        const int t0 = tile_t0(j) + 64 * half;
        const float *nk = norms + (j & 3) * 2 * kRowsTok + 64 * half, *nv = nk + kRowsTok;
        // Which columns the row sees, 32 at a time.
        uint32_t vis[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int cb = t0 + 32 * c;
          vis[c] = bits_below(last - cb + 1);
          if constexpr (WIN) vis[c] &= bits_below(n_sink - cb) | ~bits_below(behind - cb + 1);
        }
        const bool part = __any_sync(0xffffffffu, (vis[0] & vis[1]) != 0xFFFFFFFFu);
        uint32_t s[2][32];
        tc_ld32(t_s, s[0]);
        tc_ld32(t_s + 32, s[1]);
        tc_ld32_done(s[0]);
        tc_ld32_done(s[1]);
        // x = S s^K scale (log2 domain), in place, and the row's maximum
        float x[2][32], m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const ulonglong2 *n4 = reinterpret_cast<const ulonglong2 *>(nk + 32 * c);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const ulonglong2 n = n4[k];
            f2_unpack(f2_mul(f2_pack(__uint_as_float(s[c][4 * k]), __uint_as_float(s[c][4 * k + 1])), n.x), x[c][4 * k], x[c][4 * k + 1]);
            f2_unpack(f2_mul(f2_pack(__uint_as_float(s[c][4 * k + 2]), __uint_as_float(s[c][4 * k + 3])), n.y), x[c][4 * k + 2], x[c][4 * k + 3]);
          }
          if constexpr (SCALED) {
#pragma unroll
            for (int e = 0; e < 32; ++e) x[c][e] *= back;
          }
          if (part) {
#pragma unroll
            for (int e = 0; e < 32; ++e) x[c][e] = (vis[c] >> e) & 1u ? x[c][e] : -INFINITY;
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) m4[e & 3] = fmaxf(m4[e & 3], x[c][e]);
        }
        float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        float *xm = xchg + (j & 1) * 2 * kTcRows;
        xm[half * kTcRows + i] = mx;
        named_barrier(1 + (warp & 3), 64);
        mx = fmaxf(mx, xm[(half ^ 1) * kTcRows + i]);
        // Move the reference (both warps of the pair alike); O follows, once its
        // last product is complete.
        if (__any_sync(0xffffffffu, mx > ref)) {
          const bool move = mx > ref;
          const float nref = move ? mx + kRowsHeadroom : ref;
          const float f = move ? ex2f(ref - nref) : 1.f;      // 0 while ref = -inf
          ref = nref;
          const uint64_t f2 = f2_pack(f, f);
          la = f2_mul(la, f2);
          lb = f2_mul(lb, f2);
          if (j > 0) {
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(o_done, (j - 1) & 1));
            tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
              float v[16];
              tc_ld16(t_o + 64 * half + lane_off + 16 * k, v);
#pragma unroll
              for (int e = 0; e < 16; e += 2) f2_unpack(f2_mul(f2_pack(v[e], v[e + 1]), f2), v[e], v[e + 1]);
              tc_st16(t_o + 64 * half + lane_off + 16 * k, v);
            }
          }
        }
        const float base = ref == -INFINITY ? 0.f : ref;
        const uint64_t base2 = f2_pack(base, base);
#pragma unroll
        for (int c = 0; c < 4; ++c) {   // 16 scores: 8 columns of hi and 8 of lo parts
          const ulonglong2 *v4 = reinterpret_cast<const ulonglong2 *>(nv + 16 * c);
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const ulonglong2 w = v4[k];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int q = 16 * (c & 1) + 4 * k + 2 * e;
              float x0, x1, w0, w1, d0, d1;
              f2_unpack(f2_sub(f2_pack(x[c >> 1][q], x[c >> 1][q + 1]), base2), x0, x1);
              const uint64_t p2 = f2_pack(ex2f(x0), ex2f(x1));
              if (e) lb = f2_add(lb, p2); else la = f2_add(la, p2);
              f2_unpack(f2_mul(p2, e ? w.y : w.x), w0, w1);
              if (part) {   // a token that is not seen weighs nothing, whatever its norm holds
                w0 = (vis[c >> 1] >> q) & 1u ? w0 : 0.f;
                w1 = (vis[c >> 1] >> (q + 1)) & 1u ? w1 : 0.f;
              }
              const __half2 h = __floats2half2_rn(w0, w1);
              const float2 hf = __half22float2(h);
              hi[2 * k + e] = *reinterpret_cast<const uint32_t *>(&h);
              f2_unpack(f2_sub(f2_pack(w0, w1), f2_pack(hf.x, hf.y)), d0, d1);
              lo[2 * k + e] = pack_f16x2(d0, d1);
            }
          }
          tc_st8u(t_s + 32 * (c >> 1) + 8 * (c & 1), hi);
          tc_st8u(t_s + 32 * (c >> 1) + 16 + 8 * (c & 1), lo);
        }
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + (j & 1));
      }
    };
    // Two versions of the loop: the factor (or a branch around it) in the one
    // that hardly a call needs it in costs 1.2 % of the windowed prefill (355
    // against 351 us).
    if (__any_sync(0xffffffffu, back != 1.f))
      tiles(std::true_type{});
    else
      tiles(std::false_type{});
    // ---- the row's result ----
    if (ok && n_iter > 0) ok = __all_sync(0xffffffffu, mbar_wait_bounded(all_done, 0));
    if (!ok) atomicOr(&g_decode_error, kErrWaitTimeout);
    tc_fence_after();
    float l0, l1;
    f2_unpack(f2_add(la, lb), l0, l1);
    float l = l0 + l1;
    named_barrier(1 + (warp & 3), 64);   // both halves are past their last exchange
    xchg[half * kTcRows + i] = l;
    named_barrier(1 + (warp & 3), 64);
    l += xchg[(half ^ 1) * kTcRows + i];
    if constexpr (WIN) {
      // O into shared memory over the K and V buffers: row i, 16-byte chunk c at
      // c ^ (i mod 32) (no bank conflicts for a thread per row here, a warp per
      // row below); (r, l) beside it, over the norms
      const float inv = 1.f / v_scale;
      if (half == 0) reinterpret_cast<float2 *>(norms)[i] = make_float2(ref, l);
      float4 *dst = reinterpret_cast<float4 *>(smem) + 32 * i;
#pragma unroll 1
      for (int c = 4 * half; c < 4 * half + 4; ++c) {
        float v[16];
        if (n_iter > 0) {
          tc_ld16(t_o + lane_off + 16 * c, v);
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          dst[(4 * c + k) ^ (i & 31)] = make_float4(v[4 * k] * inv, v[4 * k + 1] * inv, v[4 * k + 2] * inv, v[4 * k + 3] * inv);
      }
    } else {
      const long long query = query_of(i);
      const long long slot = query * a.slot_stride + b;
      const float unit = a.acc_unit / v_scale;
#pragma unroll 1
      for (int c = 4 * half; c < 4 * half + 4; ++c) {
        float v[16];
        if (n_iter > 0) {
          tc_ld16(t_o + lane_off + 16 * c, v);
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = 0.f;
        }
        if (query >= 0) {
          float4 *dst = reinterpret_cast<float4 *>(a.ws_acc + slot * 128 + 16 * c);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            dst[k] = make_float4(v[4 * k] * unit, v[4 * k + 1] * unit, v[4 * k + 2] * unit, v[4 * k + 3] * unit);
        }
      }
      if (query >= 0 && half == 0)
        a.ws_ml[slot] = make_float2(ref == -INFINITY ? -INFINITY : ref * 0.69314718055994531f, l);
    }
    tc_fence_before();
  } else if (warp < 8 + kRowsUnpackWarps) {
    // ================= unpacking =================
    // A tile is 16 items of 8 tokens, item w + 7 k to warp w: token lane mod 8
    // of the item, 32-code group lane / 8 (the warp's loads cover whole lines,
    // its stores all banks).
    constexpr int NI = (16 + kRowsUnpackWarps - 1) / kRowsUnpackWarps, NT = 32 * kRowsUnpackWarps;
    const int w = warp - 8, grp = lane >> 3, te = tid - 256;
    const uint8_t *kb = a.packed_k + cache0 * C::PB + 12 * grp, *vb = a.packed_v + cache0 * C::PB + 12 * grp;
    uint32_t kw[NI][3], vw[NI][3];
    uint16_t nw[2] = {0, 0};
    auto fetch = [&](uint32_t (&d)[NI][3], const uint8_t *base, int t0) {
#pragma unroll
      for (int k = 0; k < NI; ++k) {
        const int item = w + kRowsUnpackWarps * k, tok = t0 + 8 * item + (lane & 7);
        d[k][0] = d[k][1] = d[k][2] = 0u;
        if (item < 16 && tok < tend) {
          const uint32_t *src = reinterpret_cast<const uint32_t *>(base + static_cast<long long>(tok) * C::PB);
          d[k][0] = __ldg(src);
          d[k][1] = __ldg(src + 1);
          d[k][2] = __ldg(src + 2);
        }
      }
    };
    // Norm i of a tile: of K for i < 128, then of V.
    auto fetch_norm = [&](int t0) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int i = te + NT * k, tok = t0 + (i & (kRowsTok - 1));
        nw[k] = i < 2 * kRowsTok && tok < tend ? __ldg((i < kRowsTok ? a.norms_k : a.norms_v) + cache0 + tok)
                                               : static_cast<uint16_t>(0);
      }
    };
    // One 32-code group to float16 centroids (and residuals), 16 bytes at a time.
    auto expand = [&](const uint32_t (&g)[3], unsigned char *tile, unsigned char *res, int tok) {
      uint32_t s[8];
      group_sel8(g[0], g[1], g[2], s);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        uint32_t v[4], r[4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t lo = prmt(a.lut_lo0, a.lut_lo1, s[2 * m + u]), hi = prmt(a.lut_hi0, a.lut_hi1, s[2 * m + u]);
          v[2 * u] = prmt(lo, hi, 0x5140u);
          v[2 * u + 1] = prmt(lo, hi, 0x7362u);
          if (res) {
            const uint32_t rl = prmt(a.res_lo0, a.res_lo1, s[2 * m + u]), rh = prmt(a.res_hi0, a.res_hi1, s[2 * m + u]);
            r[2 * u] = prmt(rl, rh, 0x5140u);
            r[2 * u + 1] = prmt(rl, rh, 0x7362u);
          }
        }
        const uint32_t off = tc_off(tok, 32 * grp + 8 * m, KBLK);
        *reinterpret_cast<uint4 *>(tile + off) = make_uint4(v[0], v[1], v[2], v[3]);
        if (res) *reinterpret_cast<uint4 *>(res + off) = make_uint4(r[0], r[1], r[2], r[3]);
      }
    };
    if (n_iter > 0) {
      fetch(kw, kb, tile_t0(0));
      fetch(vw, vb, tile_t0(0));
      fetch_norm(tile_t0(0));
    }
    for (int j = 0; j < n_iter; ++j) {
      const int s = j & 1;
      unsigned char *kt = smem + s * C::STAGE, *klt = kt + C::KV, *vt = klt + C::KV;
      // S(j - 2) has read the K buffer (and, issued before it, PV(j - 4) the
      // weights that softmax(j - 4) formed from these norms' buffer).
      if (j > 1) ok = __all_sync(0xffffffffu, mbar_wait_bounded(k_free + s, ((j >> 1) - 1) & 1));
      if (!ok) break;
#pragma unroll
      for (int k = 0; k < NI; ++k)
        if (w + kRowsUnpackWarps * k < 16) expand(kw[k], kt, klt, 8 * (w + kRowsUnpackWarps * k) + (lane & 7));
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int i = te + NT * k;
        if (i < 2 * kRowsTok)
          norms[(j & 3) * 2 * kRowsTok + i] = __half2float(__ushort_as_half(nw[k])) * (i < kRowsTok ? a.score_unit : v_scale);
      }
      if (j + 1 < n_iter) {
        fetch(kw, kb, tile_t0(j + 1));
        fetch_norm(tile_t0(j + 1));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(n_full + (j & 3));
        mbar_arrive(k_full + s);
      }
      if (j > 1) ok = __all_sync(0xffffffffu, mbar_wait_bounded(v_free + s, ((j >> 1) - 1) & 1));
      if (!ok) break;
#pragma unroll
      for (int k = 0; k < NI; ++k)
        if (w + kRowsUnpackWarps * k < 16) expand(vw[k], vt, nullptr, 8 * (w + kRowsUnpackWarps * k) + (lane & 7));
      if (j + 1 < n_iter) fetch(vw, vb, tile_t0(j + 1));
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(v_full + s);
    }
    if (!ok) atomicOr(&g_decode_error, kErrWaitTimeout);
  } else if (lane == 0 && n_iter > 0) {
    // ================= products =================
    const uint32_t s_s = smem_u32(smem);
    auto scores = [&](int j) {
      constexpr uint32_t idesc = tc_idesc(kTcRows, kRowsTok, 0);
      const uint32_t k_s = s_s + (j & 1) * C::STAGE, kl_s = k_s + C::KV, d = tmem + 128 * (j & 1);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const uint32_t ko = (ks >> 2) * KBLK + (ks & 3) * 32;
        const uint64_t bd = tc_desc(k_s + ko, 16, 1024);
        tc_mma_ts(d, t_q + 8 * ks, bd, idesc, ks > 0 ? 1u : 0u);
        tc_mma_ts(d, t_q + 64 + 8 * ks, bd, idesc, 1u);
        tc_mma_ts(d, t_q + 8 * ks, tc_desc(kl_s + ko, 16, 1024), idesc, 1u);
      }
      tc_commit(s_full + (j & 1));
      tc_commit(k_free + (j & 1));
    };
    ok = mbar_wait_bounded(k_full, 0);
    if (ok) {
      tc_fence_after();
      scores(0);
    }
    for (int j = 0; j < n_iter && ok; ++j) {
      if (j + 1 < n_iter) {
        // Its scores go over P(j - 1), whose product was issued before.
        ok = mbar_wait_bounded(k_full + ((j + 1) & 1), ((j + 1) >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        scores(j + 1);
      }
      ok = mbar_wait_bounded(v_full + (j & 1), (j >> 1) & 1) && mbar_wait_bounded(p_full + (j & 1), (j >> 1) & 1);
      if (!ok) break;
      tc_fence_after();
      constexpr uint32_t idesc = tc_idesc(kTcRows, 128, 1);
      const uint32_t v_s = s_s + (j & 1) * C::STAGE + 2 * C::KV, p = tmem + 128 * (j & 1);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const uint64_t bd = tc_desc(v_s + ks * 2048, KBLK, 1024);
        const uint32_t pc = p + 32 * (ks >> 1) + 8 * (ks & 1);
        tc_mma_ts(t_o, pc, bd, idesc, (j > 0 || ks > 0) ? 1u : 0u);
        tc_mma_ts(t_o, pc + 16, bd, idesc, 1u);
      }
      tc_commit(v_free + (j & 1));
      tc_commit(o_done);
    }
    // Everything issued completes before tensor memory is freed.
    tc_commit(all_done);
    if (!mbar_wait_bounded(all_done, 0)) ok = false;
    if (!ok) atomicOr(&g_decode_error, kErrWaitTimeout);
  }
  __syncthreads();

  if constexpr (WIN) {
    // ---- merge over the cluster in rank order and rotate back: one warp per
    // row (lane: 4 dims), the rows dealt out over the CTAs ----
    if constexpr (CLUSTER) cluster_sync();
    const float *prm = a.params_v + static_cast<size_t>(kvh) * 256 + 8 * lane;
    const Quat ql = load_quat(prm), qr = load_quat(prm + 4);
    for (int i = rank + ranks * warp; i < kTcRows; i += ranks * kRowsWarps) {
      const long long row = query_of(i);
      if (row < 0) continue;   // warp-uniform
      float l = 0.f;
      float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
      if constexpr (!CLUSTER) {
        l = norms[2 * i + 1];
        u = reinterpret_cast<const float4 *>(smem)[32 * i + (lane ^ (i & 31))];
      } else {
      const float2 mine = lane < ranks ? peer_load2(peer_address(norms + 2 * i, lane)) : make_float2(-INFINITY, 0.f);
      float m = mine.x;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      m = __shfl_sync(0xffffffffu, m, 0);
      const float w_mine = mine.x == -INFINITY ? 0.f : ex2f(mine.x - m);
      for (int k = 0; k < ranks; ++k) {
        const float4 v = peer_load4(peer_address(smem + 16 * (32 * i + (lane ^ (i & 31))), k));
        const float w = __shfl_sync(0xffffffffu, w_mine, k);
        l = fmaf(__shfl_sync(0xffffffffu, mine.y, k), w, l);
        u.x = fmaf(v.x, w, u.x);
        u.y = fmaf(v.y, w, u.y);
        u.z = fmaf(v.z, w, u.z);
        u.w = fmaf(v.w, w, u.w);
      }
      }
      const float inv = l > 0.f ? a.out_unit / l : 0.f;
      u = make_float4(u.x * inv, u.y * inv, u.z * inv, u.w * inv);
      const Quat r = block_inverse(ql, qr, Quat{u.x, u.y, u.z, u.w}, FULL);
      const float y0 = r.w + r.x, y1 = r.w - r.x, y2 = r.y + r.z, y3 = r.y - r.z;
      float x[4] = {y0 + y2, y1 + y3, y0 - y2, y1 - y3};
#pragma unroll
      for (int lm = 1; lm < 32; lm <<= 1) {
        const float sgn = (lane & lm) ? -1.f : 1.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = fmaf(x[e], sgn, __shfl_xor_sync(0xffffffffu, x[e], lm));
      }
      *reinterpret_cast<uint2 *>(static_cast<__half *>(a.out) + row * 128 + 4 * lane) =
          make_uint2(pack_f16x2(x[0], x[1]), pack_f16x2(x[2], x[3]));
    }
    if constexpr (CLUSTER) cluster_sync();   // no CTA ends while its shared memory is read
  } else {
    // This grid overlaps the split over the rows' own caches, launched before
    // it; the combine waits for this grid, so this grid ends after that one.
    asm volatile("griddepcontrol.wait;" ::: "memory");
  }
  if (warp == kRowsWarps - 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

// `ranks` (kPfWindow): CTAs of the cluster that shares a row tile's tokens.
template <int KIND, bool FULL>
int launch_rows_tc(const PrefillArgs &a, dim3 grid, int ranks, cudaStream_t st) {
  auto kernel = rows_tc_kernel<KIND, FULL>;
  if constexpr (KIND == kPfWindow)
    if (ranks > 1) kernel = rows_tc_kernel<KIND, FULL, true>;
  static std::atomic<unsigned long long> allowed[2];
  const cudaError_t c = allow_smem(allowed[ranks > 1], reinterpret_cast<const void *>(kernel), RowsCfg::SMEM);
  if (c != cudaSuccess) return set_error(ISOQ_ERR_CUDA, "attention (128 rows): %s", cudaGetErrorString(c));
  cudaError_t e = cudaSuccess;
  if (KIND == kPfPrefix)
    e = launch_pdl(kernel, grid, dim3(kRowsThreads), RowsCfg::SMEM, st, a);
  else if (ranks == 1)
    kernel<<<grid, kRowsThreads, RowsCfg::SMEM, st>>>(a);
  else
    e = launch_cluster(kernel, dim3(grid.x * ranks, grid.y, grid.z), dim3(kRowsThreads), RowsCfg::SMEM, st, ranks, a);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? ISOQ_OK : set_error(ISOQ_ERR_CUDA, "attention (128 rows) launch: %s", cudaGetErrorString(e));
}
