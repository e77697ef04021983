// The paged packed cache: block tables and slot maps from request lengths,
// and the append of new tokens into page slots.  Included by isoq_serve.cu
// inside namespace isoq::decode.

// ---------------------------------------------------------------------------
// Block tables and slot maps
// ---------------------------------------------------------------------------
// Request b holds L_b tokens and gets n_b more.  It holds ceil(L_b / P) pages
// and takes ceil((L_b + n_b) / P) minus that many from the free list, in
// request order; token i of its new ones goes to slot
//   page[(L_b + i) / P] P + (L_b + i) mod P.
// Two running sums over the requests (new tokens, pages taken) give every
// place; each CTA forms them itself, 1024 requests at a time in shared memory
// (8 bytes a request, from L2), and then writes its own share of the slots,
// finding a token's request by bisection, and of the table rows.  One launch,
// nothing exchanged between CTAs; at these sizes its cost is the launch and
// two or three dependent reads (on the GPU 64 requests of one token take 7 us
// with the copy of the table before it, 512 requests and 43,000 slots 8; 14
// with 2,048 slots per CTA, whose reads follow one another; a call of either
// with its host work 19).

constexpr int kTableThreads = 256;
constexpr int kTableRows = 1024;     // requests per pass
constexpr int kTableTokens = 512;    // slots per CTA, two per thread at once

struct TableArgs {
  const int32_t *seq_lens, *new_lens, *free_pages, *free_head;
  int32_t *block_table;     // [B][max_pages]
  long long *slot_map;      // [n_slots]
  int32_t *row_start;       // [B + 1]
  int32_t *total_lens;      // [B]
  int32_t *pages_used;      // [1]
  long long n_slots;
  int batch, n_free, max_pages, page_shift;
};

__global__ void __launch_bounds__(kTableThreads) block_tables_kernel(const TableArgs a) {
  constexpr int R = kTableRows / kTableThreads;   // consecutive requests per thread
  __shared__ long long start_s[kTableRows + 1];   // first new token
  __shared__ int first_s[kTableRows];             // first place in the free list, -1: the request does not fit
  __shared__ int len_s[kTableRows];
  __shared__ long long part[2][kTableThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = 1 << a.page_shift;
  // Most tokens of a request: what its table row and an int32 length hold.
  const long long room = min(static_cast<long long>(a.max_pages) << a.page_shift, 0x7FFFFFFFll);
  const long long lo = static_cast<long long>(blockIdx.x) * kTableTokens;
  const long long hi = lo + kTableTokens < a.n_slots ? lo + kTableTokens : a.n_slots;
  long long head = a.free_head ? *a.free_head : 0;
  head = head < 0 ? 0 : head;

  long long tok0 = 0, page0 = 0, used = 0;   // sums before this pass; pages taken so far
  bool full = false;
  for (int b0 = 0; b0 < a.batch; b0 += kTableRows) {
    const int nb = a.batch - b0 < kTableRows ? a.batch - b0 : kTableRows;
    __syncthreads();   // the previous pass is read
    int len[R], add[R], take[R];
    bool fits[R];
    long long st = 0, sp = 0;
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int b = R * tid + k;
      len[k] = add[k] = take[k] = 0;
      fits[k] = false;
      if (b < nb) {
        const int n = a.new_lens[b0 + b];
        len[k] = max(a.seq_lens[b0 + b], 0);
        add[k] = max(n, 0);
        fits[k] = n >= 0 && static_cast<long long>(len[k]) + n <= room;
      }
      st += add[k];
    }
    // exclusive sum of the new tokens over the threads
    long long xt = st;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, xt, o);
      if (lane >= o) xt += u;
    }
    if (lane == 31) part[0][warp] = xt;
    __syncthreads();
    long long bt = tok0, all_t = 0;
#pragma unroll
    for (int w = 0; w < kTableThreads / 32; ++w) {
      if (w < warp) bt += part[0][w];
      all_t += part[0][w];
    }
    bt += xt - st;
    // a request whose tokens the slot map does not hold takes no pages
    long long t = bt;
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int b = R * tid + k;
      if (b < nb) start_s[b] = t;
      t += add[k];
      if (t > a.n_slots && add[k] > 0) fits[k] = false;
      if (fits[k]) {
        const long long end = static_cast<long long>(len[k]) + add[k];
        take[k] = static_cast<int>(((end + P - 1) >> a.page_shift) - ((static_cast<long long>(len[k]) + P - 1) >> a.page_shift));
      }
      sp += take[k];
    }
    long long xp = sp;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, xp, o);
      if (lane >= o) xp += u;
    }
    if (lane == 31) part[1][warp] = xp;
    if (tid == 0) start_s[nb] = tok0 + all_t;
    __syncthreads();
    long long bp = page0, all_p = 0;
#pragma unroll
    for (int w = 0; w < kTableThreads / 32; ++w) {
      if (w < warp) bp += part[1][w];
      all_p += part[1][w];
    }
    bp += xp - sp;
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int b = R * tid + k;
      if (b < nb) {
        // The free list is taken in order; a request that finds it too short
        // takes nothing, and so does every later one that needs a page.
        const bool ok = fits[k] && (take[k] == 0 || head + bp + take[k] <= a.n_free);
        full |= !ok;
        first_s[b] = ok ? static_cast<int>(head + bp) * (take[k] > 0) : -1;
        len_s[b] = len[k];
        if (ok && take[k] > 0) used = bp + take[k];
        if (blockIdx.x == 0) {
          const long long s = start_s[b];
          a.row_start[b0 + b] = s < 0x7FFFFFFFll ? static_cast<int>(s) : 0x7FFFFFFF;
          a.total_lens[b0 + b] = ok ? len[k] + add[k] : len[k];
        }
      }
      bp += take[k];
    }
    __syncthreads();

    // This CTA's slots of these requests.
    const long long f0 = start_s[0] > lo ? start_s[0] : lo, f1 = start_s[nb] < hi ? start_s[nb] : hi;
#pragma unroll 2
    for (long long i = f0 + tid; i < f1; i += kTableThreads) {
      int x = 0, y = nb;   // the last request with start <= i
      while (y - x > 1) {
        const int m = (x + y) >> 1;
        if (start_s[m] <= i) x = m; else y = m;
      }
      long long slot = -1;
      if (first_s[x] >= 0) {
        const long long pos = len_s[x] + (i - start_s[x]);
        const int col = static_cast<int>(pos >> a.page_shift), have = static_cast<int>((static_cast<long long>(len_s[x]) + P - 1) >> a.page_shift);
        const long long page = col < have ? a.block_table[static_cast<long long>(b0 + x) * a.max_pages + col]
                                          : a.free_pages[first_s[x] + col - have];
        slot = (page << a.page_shift) + (pos & (P - 1));
      }
      a.slot_map[i] = slot;
    }
    // This CTA's table rows (one warp each).
    for (int b = blockIdx.x + gridDim.x * warp; b < nb; b += gridDim.x * (kTableThreads / 32)) {
      if (first_s[b] < 0) continue;
      const long long end = len_s[b] + (start_s[b + 1] - start_s[b]);
      const int have = static_cast<int>((static_cast<long long>(len_s[b]) + P - 1) >> a.page_shift);
      const int need = static_cast<int>((end + P - 1) >> a.page_shift);
      int32_t *row = a.block_table + static_cast<long long>(b0 + b) * a.max_pages;
      for (int c = have + lane; c < need; c += 32) row[c] = a.free_pages[first_s[b] + c - have];
    }
    tok0 += all_t;
    page0 += all_p;
  }
  // Slots that no token of this call has.
  for (long long i = (tok0 > lo ? tok0 : lo) + tid; i < hi; i += kTableThreads) a.slot_map[i] = -1;
  if (blockIdx.x == 0) {
    // pages taken: the largest over the threads (each saw its own requests)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const long long u = __shfl_xor_sync(0xffffffffu, used, o);
      used = u > used ? u : used;
    }
    __syncthreads();
    if (lane == 0) part[0][warp] = used;
    full = __syncthreads_or(full);
    if (tid == 0) {
      for (int w = 1; w < kTableThreads / 32; ++w) used = part[0][w] > used ? part[0][w] : used;
      *a.pages_used = static_cast<int>(used);
      a.row_start[a.batch] = tok0 < 0x7FFFFFFFll ? static_cast<int>(tok0) : 0x7FFFFFFF;
      if (full) atomicOr(&g_decode_error, kErrTableFull);
    }
  }
}

// ---------------------------------------------------------------------------
// Append into page slots
// ---------------------------------------------------------------------------
// Algorithm 1 of the compressor on the new tokens' K and V vectors, written
// to the slots of the slot map.  d / 16 lanes hold a vector, 16 consecutive
// dims each (4, 2 or 1 vectors per warp at d = 128, 256, 512): float32 norm,
// Walsh-Hadamard stages 1 .. 8 in the lane and the others by shuffles, the
// lane's four block maps with their quaternions kept in registers over the
// warp's tokens, codes #{k : y > s t_k} by bisection of the positive
// thresholds, and the packed words from at most one exchange between
// neighbour lanes.  A warp keeps one (KV head, K or V) and walks its tokens,
// the next one's loads under way while it works.
//
// The codes and norms are the float64 decisions: float32 leaves y within
// kExactBand s of its value (each of the log2 d stages and of the two
// quaternion products rounds by at most 2^-24 of a partial sum that is at
// most s, in the l2 sense: below 50 2^-24 s = 3e-6 s in all), so a
// coordinate farther than that from every threshold is decided, and the rest
// (about 2 vectors in 100 at d = 128 and 3 bits) are summed again in double
// by the vector's lanes.  The same for a norm near a float16 rounding
// boundary.
//
// Bound: issue slots (0.64 per cycle), 204 warp instructions per vector at
// d = 128 and 3 bits.  8,191 tokens x 4 KV heads, float16: 24.6 us; one warp per
// vector and token took 38.9.
constexpr float kExactBand = 4e-6f;

struct PagedAppendArgs {
  const void *k_new, *v_new;   // [N][Hkv][d]
  uint8_t *pages_k, *pages_v;
  uint16_t *norms_k, *norms_v;
  const long long *slot_map;
  const float *params_k, *params_v;
  long long n_tok, n_rows;     // N; n_pages P
  int hkv, page_shift;
  float thr[8];                // the positive thresholds, ascending, from 0
  double thr64[15];
};

// Sixteen consecutive elements as loaded, and as float32.
template <typename T>
struct Raw16 {
  uint4 u[sizeof(T)];
  __device__ __forceinline__ void load(const T *src) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)); ++i) u[i] = __ldcs(reinterpret_cast<const uint4 *>(src) + i);
  }
  __device__ __forceinline__ float get(int e) const {   // e known at compile time
    const uint32_t *w = reinterpret_cast<const uint32_t *>(u);
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
    else return __half2float(__ushort_as_half(static_cast<unsigned short>(w[e >> 1] >> (16 * (e & 1)))));
  }
};

template <typename T, int D, int BITS, bool FULL>
__global__ void __launch_bounds__(128) paged_append_kernel(const PagedAppendArgs a) {
  constexpr int LV = D / 16, VPW = 32 / LV;              // lanes per vector, vectors per warp
  constexpr int L = 1 << BITS, HP = L / 2;               // HP non-negative thresholds, 0 among them
  const int lane = threadIdx.x & 31, vl = lane % LV;     // the lane within its vector
  const int kvh = blockIdx.y >> 1;
  const bool val = blockIdx.y & 1;
  const long long step = static_cast<long long>(gridDim.x) * 4 * VPW;
  long long n = (static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5)) * VPW + lane / LV;
  const long long n_warp_end = a.n_tok;
  const T *x_base = static_cast<const T *>(val ? a.v_new : a.k_new) + static_cast<long long>(kvh) * D + 16 * vl;
  const float *prm = (val ? a.params_v : a.params_k) + static_cast<size_t>(kvh) * 2 * D;
  constexpr int PB = D * BITS / 8;

  Raw16<T> nx{};
  long long slot_nx = -1;
  if (n < n_warp_end) {
    nx.load(x_base + n * a.hkv * D);
    slot_nx = a.slot_map[n];
  }
  Quat ql[4], qr[4];
  const float inv = rsqrtf(static_cast<float>(D));
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    ql[u] = load_quat(prm + 8 * (4 * vl + u));
    qr[u] = FULL ? load_quat(prm + 8 * (4 * vl + u) + 4) : Quat{1.f, 0.f, 0.f, 0.f};
  }

  for (; __any_sync(0xffffffffu, n < n_warp_end); n += step) {
    const Raw16<T> cur = nx;
    const bool here = n < n_warp_end;
    const long long slot = here ? slot_nx : -1;
    if (n + step < n_warp_end) {
      nx.load(x_base + (n + step) * a.hkv * D);
      slot_nx = a.slot_map[n + step];
    }
    const bool write = slot >= 0 && slot < a.n_rows;
    if (slot >= a.n_rows && vl == 0) atomicOr(&g_decode_error, kErrBadPage);

    float x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = cur.get(e);
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
    for (int o = 1; o < LV; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float s = sqrtf(ss);
    // A float32 vector whose squares leave float32's range: all in double.
    bool extreme = false;
    if constexpr (sizeof(T) == 4) {
      bool some = false;
#pragma unroll
      for (int e = 0; e < 16; ++e) some |= x[e] != 0.f;
      const unsigned any = __ballot_sync(0xffffffffu, some && (ss < 1e-30f || ss > 1e30f));
      const unsigned mine = LV == 32 ? 0xFFFFFFFFu : ((1u << LV) - 1u) << (lane - vl);
      extreme = (any & mine) != 0;
    }
#pragma unroll
    for (int hs = 1; hs < 16; hs <<= 1) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if (!(e & hs)) {
          const float p = x[e], q = x[e + hs];
          x[e] = p + q;
          x[e + hs] = p - q;
        }
      }
    }
#pragma unroll
    for (int lm = 1; lm < LV; lm <<= 1) {
      const float sgn = (lane & lm) ? -1.f : 1.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = fmaf(x[e], sgn, __shfl_xor_sync(0xffffffffu, x[e], lm));
    }
    unsigned near = 0;            // bit e: coordinate e is decided in double
    uint64_t codes = 0;           // code e in bits 4 e .. + 3
    const float band = kExactBand * s;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const Quat w{x[4 * u] * inv, x[4 * u + 1] * inv, x[4 * u + 2] * inv, x[4 * u + 3] * inv};
      const Quat r = block_forward(ql[u], qr[u], w, FULL);
      const float y[4] = {r.w, r.x, r.y, r.z};
      uint32_t c4 = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // m: |y|; c: positive thresholds below it, by bisection; gap: distance
        // to the nearest threshold met, 0 among them (the nearest one is
        // always met).
        const float m = fabsf(y[e]);
        float gap = m;
        unsigned c = 0;
        if constexpr (BITS == 2) {
          const float d1 = m - a.thr[1] * s;
          c = d1 > 0.f;
          gap = fminf(gap, fabsf(d1));
        } else if constexpr (BITS == 3) {
          const float d2 = m - a.thr[2] * s;
          const bool b2 = d2 > 0.f;
          const float d1 = m - (b2 ? a.thr[3] : a.thr[1]) * s;
          c = (b2 ? 2u : 0u) + (d1 > 0.f ? 1u : 0u);
          gap = fminf(gap, fminf(fabsf(d2), fabsf(d1)));
        } else {
          const float d4 = m - a.thr[4] * s;
          const bool b4 = d4 > 0.f;
          const float d2 = m - (b4 ? a.thr[6] : a.thr[2]) * s;
          const bool b2 = d2 > 0.f;
          const float lo = b2 ? a.thr[3] : a.thr[1], hi = b2 ? a.thr[7] : a.thr[5];
          const float d1 = m - (b4 ? hi : lo) * s;
          c = (b4 ? 4u : 0u) + (b2 ? 2u : 0u) + (d1 > 0.f ? 1u : 0u);
          gap = fminf(fminf(gap, fabsf(d4)), fminf(fabsf(d2), fabsf(d1)));
        }
        c4 |= (y[e] > 0.f ? HP + c : HP - 1 - c) << (4 * e);
        if (gap < band) near |= 1u << (4 * u + e);
      }
      codes |= static_cast<uint64_t>(c4) << (16 * u);
    }
    if (extreme) near = 0xFFFFu;
    __half nrm = __float2half_rn(s);
    const bool round_near = extreme || __half_as_ushort(__float2half_rn(s * (1.f + 4e-6f))) !=
                                           __half_as_ushort(__float2half_rn(s * (1.f - 4e-6f)));
    if (!write) near = 0;
    if (__any_sync(0xffffffffu, near != 0 || (round_near && write))) {
      double sq = 0.0;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const double xe = static_cast<double>(cur.get(e));
        sq = fma(xe, xe, sq);
      }
#pragma unroll
      for (int o = 1; o < LV; o <<= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
      const double s64 = sqrt(sq);
      nrm = __double2half(s64);
      // Each vector's lanes take one of its coordinates per turn.
      while (__any_sync(0xffffffffu, near != 0)) {
        const unsigned all = __ballot_sync(0xffffffffu, near != 0);
        const unsigned mine = LV == 32 ? all : (all >> (lane - vl)) & ((1u << (LV & 31)) - 1u);
        const int fl = mine ? __ffs(mine) - 1 : 0;                    // the lane (of the vector) that holds it
        const unsigned es = __shfl_sync(0xffffffffu, near, lane - vl + fl);
        const int fe = es ? __ffs(es) - 1 : 0;
        const int i = 16 * fl + fe, bi = i >> 2, rr = i & 3;
        double h[4] = {0.0, 0.0, 0.0, 0.0};                           // the block's Walsh-Hadamard outputs
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const double xe = static_cast<double>(cur.get(e));
#pragma unroll
          for (int c = 0; c < 4; ++c) h[c] += (__popc((4 * bi + c) & (16 * vl + e)) & 1) ? -xe : xe;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int o = 1; o < LV; o <<= 1) h[c] += __shfl_xor_sync(0xffffffffu, h[c], o);
        auto mul = [](const double *p, const double *q, double *r) {
          r[0] = p[0] * q[0] - p[1] * q[1] - p[2] * q[2] - p[3] * q[3];
          r[1] = p[0] * q[1] + p[1] * q[0] + p[2] * q[3] - p[3] * q[2];
          r[2] = p[0] * q[2] - p[1] * q[3] + p[2] * q[0] + p[3] * q[1];
          r[3] = p[0] * q[3] + p[1] * q[2] - p[2] * q[1] + p[3] * q[0];
        };
        const double q4[4] = {prm[8 * bi], prm[8 * bi + 1], prm[8 * bi + 2], prm[8 * bi + 3]};
        double y4[4];
        mul(q4, h, y4);
        if (FULL) {
          const double r4[4] = {prm[8 * bi + 4], -static_cast<double>(prm[8 * bi + 5]),
                                -static_cast<double>(prm[8 * bi + 6]), -static_cast<double>(prm[8 * bi + 7])};
          double z4[4];
          mul(y4, r4, z4);
#pragma unroll
          for (int c = 0; c < 4; ++c) y4[c] = z4[c];
        }
        const double y = (rr == 0 ? y4[0] : rr == 1 ? y4[1] : rr == 2 ? y4[2] : y4[3]) / sqrt(static_cast<double>(D));
        uint64_t c = 0;
#pragma unroll 1
        for (int k = 0; k < L - 1; ++k) c += y > a.thr64[k] * s64 ? 1u : 0u;
        if (near != 0 && vl == fl) {
          codes = (codes & ~(15ull << (4 * fe))) | (c << (4 * fe));
          near &= near - 1;
        }
      }
    }

    const int mask = (1 << a.page_shift) - 1;
    const long long at = (((slot >> a.page_shift) * a.hkv + kvh) << a.page_shift) + (slot & mask);
    uint8_t *dst = (val ? a.pages_v : a.pages_k) + at * PB;
    const uint32_t c0 = static_cast<uint32_t>(codes), c1 = static_cast<uint32_t>(codes >> 32);   // codes 0..7, 8..15
    if (write && vl == 0) (val ? a.norms_v : a.norms_k)[at] = __half_as_ushort(nrm);
    if constexpr (BITS == 3) {
      // Two lanes share a 32-code group: the even one holds words 0 and 1, the
      // odd one word 2 and codes 24 .. 31, whose bit r goes to the spare bits
      // of word r.
      const bool odd = vl & 1;
      const uint32_t t0 = (c1 & 0x11111111u) << 3, t1 = (c1 & 0x22222222u) << 2, t2 = (c1 & 0x44444444u) << 1;
      const uint32_t g0 = __shfl_xor_sync(0xffffffffu, t0, 1), g1 = __shfl_xor_sync(0xffffffffu, t1, 1);
      uint32_t *g = reinterpret_cast<uint32_t *>(dst) + 3 * (vl >> 1);
      if (write) {
        if (odd) {
          g[2] = c0 | t2;
        } else {
          g[0] = c0 | g0;
          g[1] = c1 | g1;
        }
      }
    } else if constexpr (BITS == 4) {
      if (write) reinterpret_cast<uint2 *>(dst)[vl] = make_uint2(c0, c1);
    } else {
      // 4-bit fields to 2-bit ones
      auto squeeze = [](uint32_t v) {
        v = (v | (v >> 2)) & 0x0F0F0F0Fu;
        v = (v | (v >> 4)) & 0x00FF00FFu;
        return (v | (v >> 8)) & 0xFFFFu;
      };
      if (write) reinterpret_cast<uint32_t *>(dst)[vl] = squeeze(c0) | (squeeze(c1) << 16);
    }
  }
}

template <typename T, int D, int BITS>
int launch_paged_append(int variant, const PagedAppendArgs &a, cudaStream_t st) {
  // The CTAs that are resident at once (4 per SM) over all heads; a warp walks
  // the rest.
  constexpr int VPC = 4 * (512 / D);   // tokens of a CTA per turn
  const long long turns = (a.n_tok + VPC - 1) / VPC;
  long long gx = (4 * 148 + 2 * a.hkv - 1) / (2 * a.hkv);
  if (gx > turns) gx = turns;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(2 * a.hkv));
  if (variant == ISOQ_FULL)
    paged_append_kernel<T, D, BITS, true><<<grid, 128, 0, st>>>(a);
  else
    paged_append_kernel<T, D, BITS, false><<<grid, 128, 0, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ISOQ_OK : set_error(ISOQ_ERR_CUDA, "paged append launch: %s", cudaGetErrorString(e));
}

template <typename T, int D>
int run_paged_append_b(int bits, int variant, const PagedAppendArgs &a, cudaStream_t st) {
  if (bits == 2) return launch_paged_append<T, D, 2>(variant, a, st);
  if (bits == 3) return launch_paged_append<T, D, 3>(variant, a, st);
  return launch_paged_append<T, D, 4>(variant, a, st);
}

template <typename T>
int run_paged_append_d(int d, int bits, int variant, const PagedAppendArgs &a, cudaStream_t st) {
  if (d == 128) return run_paged_append_b<T, 128>(bits, variant, a, st);
  if (d == 256) return run_paged_append_b<T, 256>(bits, variant, a, st);
  return run_paged_append_b<T, 512>(bits, variant, a, st);
}

int run_paged_append(int dtype, int d, int bits, int variant, const PagedAppendArgs &a, cudaStream_t st) {
  return dtype == ISOQ_F16 ? run_paged_append_d<__half>(d, bits, variant, a, st)
                           : run_paged_append_d<float>(d, bits, variant, a, st);
}
