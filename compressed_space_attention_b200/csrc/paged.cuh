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
// two or three dependent reads.

constexpr int kTableThreads = 256;
constexpr int kTableRows = 1024;     // requests per pass
constexpr int kTableTokens = 2048;   // slots per CTA

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
        fits[k] = n >= 0 && static_cast<long long>(len[k]) + n <= static_cast<long long>(a.max_pages) << a.page_shift;
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
// to the slots of the slot map.  One warp per vector, lane j holding dims
// E j .. E j + E - 1 (E = d / 32): float32 norm by shuffles, Walsh-Hadamard
// stages in the lane and by shuffles, block maps, codes #{k : y > s t_k}.
//
// The codes and norms are the float64 decisions: float32 leaves y within
// kExactBand s of its value (each of the log2 d stages and of the two
// quaternion products rounds by at most 2^-24 of a partial sum that is at
// most s, in the l2 sense: below 50 2^-24 s = 3e-6 s in all), so a
// coordinate farther than that from every threshold is decided, and the rest
// (about 2 vectors in 100 at d = 128 and 3 bits) are summed again in double
// by the whole warp.  The same for a norm near a float16 rounding boundary.
constexpr float kExactBand = 4e-6f;

struct PagedAppendArgs {
  const void *k_new, *v_new;   // [N][Hkv][d]
  uint8_t *pages_k, *pages_v;
  uint16_t *norms_k, *norms_v;
  const long long *slot_map;
  const float *params_k, *params_v;
  long long n_vec, n_rows;     // N Hkv; n_pages P
  int hkv, page_shift;
  float thr[8];                // the positive thresholds, ascending, from 0
  double thr64[15];
};

// E consecutive elements (8 to 64 bytes, aligned to their size or 16 bytes).
template <typename T, int E>
__device__ __forceinline__ void load_elements(const T *src, float (&x)[E]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < E; e += 4) {
      const float4 u = *reinterpret_cast<const float4 *>(src + e);
      x[e] = u.x;
      x[e + 1] = u.y;
      x[e + 2] = u.z;
      x[e + 3] = u.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; e += 4) {
      const uint2 u = *reinterpret_cast<const uint2 *>(src + e);
      const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&u.x));
      const float2 q = __half22float2(*reinterpret_cast<const __half2 *>(&u.y));
      x[e] = p.x;
      x[e + 1] = p.y;
      x[e + 2] = q.x;
      x[e + 3] = q.y;
    }
  }
}

template <typename T, int D, int BITS, bool FULL>
__global__ void __launch_bounds__(128) paged_append_kernel(const PagedAppendArgs a) {
  constexpr int E = D / 32, L = 1 << BITS, HP = L / 2;   // HP positive thresholds, 0 among them
  const int lane = threadIdx.x & 31;
  const long long v = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (v >= a.n_vec) return;
  const bool val = blockIdx.y != 0;
  const long long n = v / a.hkv;
  const int kvh = static_cast<int>(v - n * a.hkv);
  const long long slot = a.slot_map[n];
  if (slot < 0) return;
  if (slot >= a.n_rows) {
    if (lane == 0) atomicOr(&g_decode_error, kErrBadPage);
    return;
  }
  const T *src = static_cast<const T *>(val ? a.v_new : a.k_new) + v * D + E * lane;
  float x[E];
  load_elements<T, E>(src, x);
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float s = sqrtf(ss);
  // A float32 vector whose squares leave float32's range: all in double.
  bool extreme = false;
  if constexpr (sizeof(T) == 4) {
    if (ss < 1e-30f || ss > 1e30f) {
      bool some = false;
#pragma unroll
      for (int e = 0; e < E; ++e) some |= x[e] != 0.f;
      extreme = __any_sync(0xffffffffu, some);
    }
  }
#pragma unroll
  for (int hs = 1; hs < E; hs <<= 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (!(e & hs)) {
        const float p = x[e], q = x[e + hs];
        x[e] = p + q;
        x[e + hs] = p - q;
      }
    }
  }
#pragma unroll
  for (int lm = 1; lm < 32; lm <<= 1) {
    const bool upper = (lane & lm) != 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float o = __shfl_xor_sync(0xffffffffu, x[e], lm);
      x[e] = upper ? o - x[e] : x[e] + o;
    }
  }
  const float inv = rsqrtf(static_cast<float>(D));
  const float *prm = (val ? a.params_v : a.params_k) + static_cast<size_t>(kvh) * 2 * D;
  unsigned code[E], near = 0;   // near: bit e, coordinate e is decided in double
#pragma unroll
  for (int u = 0; u < E / 4; ++u) {
    const int bi = (E / 4) * lane + u;
    const Quat w{x[4 * u] * inv, x[4 * u + 1] * inv, x[4 * u + 2] * inv, x[4 * u + 3] * inv};
    const Quat r = block_forward(load_quat(prm + 8 * bi), load_quat(prm + 8 * bi + 4), w, FULL);
    const float y[4] = {r.w, r.x, r.y, r.z};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float m = fabsf(y[e]);
      float gap = m;   // distance to the nearest threshold: to 0, then to the others
      unsigned c = 0;
#pragma unroll
      for (int k = 1; k < HP; ++k) {
        const float dlt = m - a.thr[k] * s;
        c += dlt > 0.f ? 1u : 0u;
        gap = fminf(gap, fabsf(dlt));
      }
      code[4 * u + e] = y[e] > 0.f ? HP + c : HP - 1 - c;
      if (gap < kExactBand * s) near |= 1u << (4 * u + e);
    }
  }
  if (extreme) near = (1u << E) - 1u;
  __half nrm = __float2half_rn(s);
  const bool round_near = __half_as_ushort(__float2half_rn(s * (1.f + 4e-6f))) != __half_as_ushort(__float2half_rn(s * (1.f - 4e-6f)));
  if (round_near || extreme || __any_sync(0xffffffffu, near != 0)) {   // warp-uniform
    double sq = 0.0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const double xe = static_cast<double>(to_f32<T>(src[e]));
      sq = fma(xe, xe, sq);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    const double s64 = sqrt(sq);
    nrm = __double2half(s64);
    for (unsigned lanes = __ballot_sync(0xffffffffu, near != 0); lanes; lanes &= lanes - 1) {
      const int fl = __ffs(lanes) - 1;
      for (unsigned es = __shfl_sync(0xffffffffu, near, fl); es; es &= es - 1) {
        const int fe = __ffs(es) - 1, i = E * fl + fe, bi = i >> 2, rr = i & 3;
        // the four Walsh-Hadamard outputs of block bi
        double h[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const double xe = static_cast<double>(to_f32<T>(src[e]));
#pragma unroll
          for (int c = 0; c < 4; ++c) h[c] += (__popc((4 * bi + c) & (E * lane + e)) & 1) ? -xe : xe;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) h[c] += __shfl_xor_sync(0xffffffffu, h[c], o);
        auto mul = [](const double *p, const double *q, double *r) {
          r[0] = p[0] * q[0] - p[1] * q[1] - p[2] * q[2] - p[3] * q[3];
          r[1] = p[0] * q[1] + p[1] * q[0] + p[2] * q[3] - p[3] * q[2];
          r[2] = p[0] * q[2] - p[1] * q[3] + p[2] * q[0] + p[3] * q[1];
          r[3] = p[0] * q[3] + p[1] * q[2] - p[2] * q[1] + p[3] * q[0];
        };
        const double ql[4] = {prm[8 * bi], prm[8 * bi + 1], prm[8 * bi + 2], prm[8 * bi + 3]};
        double y4[4];
        mul(ql, h, y4);
        if (FULL) {
          const double qr[4] = {prm[8 * bi + 4], -static_cast<double>(prm[8 * bi + 5]),
                                -static_cast<double>(prm[8 * bi + 6]), -static_cast<double>(prm[8 * bi + 7])};
          double z4[4];
          mul(y4, qr, z4);
#pragma unroll
          for (int c = 0; c < 4; ++c) y4[c] = z4[c];
        }
        const double y = (rr == 0 ? y4[0] : rr == 1 ? y4[1] : rr == 2 ? y4[2] : y4[3]) / sqrt(static_cast<double>(D));
        unsigned c = 0;
#pragma unroll
        for (int k = 0; k < L - 1; ++k) c += y > a.thr64[k] * s64 ? 1u : 0u;
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (lane == fl && e == fe) code[e] = c;
      }
    }
  }

  const int mask = (1 << a.page_shift) - 1;
  const long long at = (((slot >> a.page_shift) * a.hkv + kvh) << a.page_shift) + (slot & mask);
  constexpr int PB = D * BITS / 8;
  uint8_t *dst = (val ? a.pages_v : a.pages_k) + at * PB;
  if (lane == 0) (val ? a.norms_v : a.norms_k)[at] = __half_as_ushort(nrm);
  if constexpr (BITS == 3) {
    constexpr int GL = 32 / E;          // lanes of a 32-code group
    const int m0 = E * (lane & (GL - 1));
    uint32_t w[3] = {0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int m = m0 + e;             // code m of the group
      const uint32_t body = code[e] << (4 * (m & 7));
#pragma unroll
      for (int r = 0; r < 3; ++r)
        w[r] |= m < 24 ? ((m >> 3) == r ? body : 0u) : ((code[e] >> r) & 1u) << (4 * (m & 7) + 3);
    }
#pragma unroll
    for (int o = 1; o < GL; o <<= 1)
#pragma unroll
      for (int r = 0; r < 3; ++r) w[r] |= __shfl_xor_sync(0xffffffffu, w[r], o);
    if ((lane & (GL - 1)) == 0) {
      uint32_t *g = reinterpret_cast<uint32_t *>(dst) + 3 * (lane / GL);
#pragma unroll
      for (int r = 0; r < 3; ++r) g[r] = w[r];
    }
  } else {
    constexpr int NB = E * BITS;        // bits of a lane: 8, 16, 32 or 64
    uint64_t w = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) w |= static_cast<uint64_t>(code[e]) << (BITS * e);
    if constexpr (NB == 8) dst[lane] = static_cast<uint8_t>(w);
    else if constexpr (NB == 16) reinterpret_cast<uint16_t *>(dst)[lane] = static_cast<uint16_t>(w);
    else if constexpr (NB == 32) reinterpret_cast<uint32_t *>(dst)[lane] = static_cast<uint32_t>(w);
    else reinterpret_cast<uint64_t *>(dst)[lane] = w;
  }
}

template <typename T, int D, int BITS>
int launch_paged_append(int variant, const PagedAppendArgs &a, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((a.n_vec + 3) / 4), 2);
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
