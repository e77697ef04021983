// CUDA-core split of the serving attention: any query dtype, d and bits, any
// group, any alignment that the entry points take.  Included by
// isoq_serve.cu inside namespace isoq::decode.
//
// Per query row: z_j = s^K_j <q~, c[K_j]> scale over the tokens it sees, one
// pass with the running reference maximum and sum of the softmax, and
// acc += p_j s^V_j c[V_j], all in float32 and in the rotated domain; one
// partial state (m, l, acc[d]) per query row and split, merged by
// combine_kernel.
//
// A CTA's four warps take the split's 32-token blocks in turn, up to RG query
// rows at once, so that one unpacking of a code serves all of them.  The next
// block arrives by 16-byte asynchronous copies (two stages per warp; a row's
// stride is an odd number of 16-byte units: no bank conflicts).
//   Scores: lane (t, s) = (lane mod 8, lane / 8) takes tokens t, t + 8, t + 16,
//   t + 24 and the 32-code groups s, s + 4, ...: every query value it loads
//   (RG rows of one dimension, broadcast over t) serves four tokens, every
//   centroid it looks up RG rows, two per f32x2 instruction.  Two exchanges
//   add the four slices and leave lane L with token L.
//   Values: a lane takes d / 32 dimensions, the weights broadcast.
//
// Bound: issue slots (0.59 per cycle), the ALU and FMA pipes (43 % busy each)
// and the LSU pipe (36 %): about 110 warp instructions per token and KV head for
// 8 rows, of which the two products are 32, the code lookups 32.  16 rows of 4,096 to 8,192 tokens x 4 KV heads,
// d = 128, 4 bits, 8 rows: a token per lane in the score loop took 92 us (every
// query value loaded again for each token), this form 78; half a warp per token
// in the value loop 84 (168 registers, 3 CTAs per SM instead of 4).

constexpr int kAnyWarps = 4;
constexpr int kAnyThreads = 32 * kAnyWarps;

template <int D, int BITS, int RG>
struct AnyCfg {
  static constexpr int PB = D * BITS / 8;
  static constexpr int RS = ((PB / 16) | 1) * 16;           // row stride in shared memory
  static constexpr int STAGE = 2 * 32 * RS;                 // K rows, V rows of a block
  // Rotated queries [32-code group][dim][RG], 8 floats between groups: the
  // four groups that a warp reads at once lie in different banks.
  static constexpr int Q_GROUP = 32 * RG + 8;
  static constexpr int OFF_Q = 2 * kAnyWarps * STAGE;
  static constexpr int OFF_W = OFF_Q + (D / 32) * Q_GROUP * 4;      // [warp][32][RG] weights
  static constexpr int OFF_TAB = OFF_W + kAnyWarps * 32 * RG * 4;   // [16] centroids
  static constexpr int OFF_ML = OFF_TAB + 16 * 4;           // [warp][RG] (m, l)
  static constexpr int MIN_BLOCKS = D == 128 ? 4 : 1;
  static constexpr int SMEM = OFF_ML + kAnyWarps * RG * 8;
  // CTAs that an SM holds: by registers (128 a thread at d = 128, 168 at
  // d = 256 up to 4 rows, up to 254 otherwise) and by shared memory.
  static constexpr int BY_REGS = D == 128 ? 4 : (D == 256 && RG <= 4 ? 3 : 2), BY_SMEM = 233472 / (SMEM + 1024);
  static constexpr int SLOTS = BY_REGS < BY_SMEM ? BY_REGS : BY_SMEM;
  static_assert(kAnyWarps * RG * D * 4 <= OFF_Q, "the warps' accumulators fit the stages");
};

// Codes 4 quad .. + 3 of a packed row (32-bit words) as four 4-bit fields.
template <int BITS>
__device__ __forceinline__ uint32_t quad_fields(const uint32_t *w, int quad) {
  if constexpr (BITS == 2) {
    uint32_t x = (w[quad >> 2] >> (8 * (quad & 3))) & 0xFFu;
    x = (x | (x << 4)) & 0x0F0Fu;
    return (x | (x << 2)) & 0x3333u;
  } else if constexpr (BITS == 4) {
    return (w[quad >> 1] >> (16 * (quad & 1))) & 0xFFFFu;
  } else {
    const uint32_t *g = w + 3 * (quad >> 3);
    const int q = quad & 7;
    const uint32_t w0 = g[0], w1 = g[1], w2 = g[2];
    const uint32_t body = (q < 2 ? w0 : (q < 4 ? w1 : w2)) & 0x77777777u;
    const uint32_t tail = ((w0 & 0x88888888u) >> 3) + ((w1 & 0x88888888u) >> 2) + ((w2 & 0x88888888u) >> 1);
    return ((q < 6 ? body : tail) >> (16 * (q & 1))) & 0x7777u;
  }
}

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// q~ = R_K q scale log2(e) of one query row by one warp, lane j holding dims
// E j .. E j + E - 1 (E = d / 32) before and after: the Walsh-Hadamard stages
// h < E inside the lane, the others by shuffles, then 1 / sqrt(d) and the block
// maps (the order of prep_i8_kernel).
template <int D>
__device__ __forceinline__ void rotate_query(float (&x)[D / 32], const float *prm, bool full, float scale, int lane) {
  constexpr int E = D / 32;
#pragma unroll
  for (int hs = 1; hs < E; hs <<= 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (!(e & hs)) {
        const float u = x[e], v = x[e + hs];
        x[e] = u + v;
        x[e + hs] = u - v;
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
  const float sc = scale * 1.4426950408889634f;
#pragma unroll
  for (int u = 0; u < E / 4; ++u) {
    const int bi = (E / 4) * lane + u;
    const Quat v{x[4 * u] * inv, x[4 * u + 1] * inv, x[4 * u + 2] * inv, x[4 * u + 3] * inv};
    const Quat y = block_forward(load_quat(prm + 8 * bi), load_quat(prm + 8 * bi + 4), v, full);
    x[4 * u] = y.w * sc;
    x[4 * u + 1] = y.x * sc;
    x[4 * u + 2] = y.y * sc;
    x[4 * u + 3] = y.z * sc;
  }
}

// The rotated queries of all rows, one warp per row.
template <typename T, int D, bool FULL>
__global__ void __launch_bounds__(128) prep_rotate_kernel(const SplitArgs a) {
  constexpr int E = D / 32;
  pdl_launch_dependents();
  const long long r = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (r >= static_cast<long long>(a.batch) * a.hq) return;
  const int kvh = static_cast<int>(r % a.hq) / a.group;
  const T *q = static_cast<const T *>(a.q) + r * D + E * lane;
  float x[E];
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = to_f32<T>(q[e]);
  rotate_query<D>(x, a.params_k + static_cast<size_t>(kvh) * 2 * D, FULL, a.scale, lane);
  float *out = a.ws_qrot + r * D + E * lane;
#pragma unroll
  for (int e = 0; e < E; e += 4) *reinterpret_cast<float4 *>(out + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
}

template <int D, int BITS, int RG>
__global__ void __launch_bounds__(kAnyThreads, AnyCfg<D, BITS, RG>::MIN_BLOCKS) split_any_kernel(const SplitArgs a) {
  using C = AnyCfg<D, BITS, RG>;
  constexpr int PB = C::PB, RS = C::RS, KD = D / 32, RP = RG / 2;
  extern __shared__ __align__(128) unsigned char smem[];
  float *qs = reinterpret_cast<float *>(smem + C::OFF_Q);
  unsigned char *tab = smem + C::OFF_TAB;
  float2 *ml = reinterpret_cast<float2 *>(smem + C::OFF_ML);
  const int split = blockIdx.x, kvh = blockIdx.y, z = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool paged = a.mode == kSplitPaged;
  const RowGroup grp = row_group(a, a.mode, z);
  const int row = grp.row, rows = grp.rows;
  const long long chunk = grp.prefix ? a.chunk_p : a.chunk;
  // The grid covers the longer of the two split counts (kSplitPrefix).
  if (split >= (grp.prefix ? a.n_splits_p : a.n_splits)) return;
  const uint8_t *pk = grp.prefix ? a.prefix_k : a.packed_k, *pv = grp.prefix ? a.prefix_v : a.packed_v;
  const uint16_t *nk = grp.prefix ? a.prefix_nk : a.norms_k, *nv = grp.prefix ? a.prefix_nv : a.norms_v;
  if (tid < 16) *reinterpret_cast<float *>(tab + 4 * tid) = a.centroid[tid];

  const long long tmax = grp.prefix ? a.prefix_max : a.tmax;
  int tlen = grp.prefix ? *a.prefix_len : a.seq_lens[row];
  tlen = tlen < 0 ? 0 : (tlen > tmax ? static_cast<int>(tmax) : tlen);
  const SeenBlocks seen = seen_blocks(tlen, a.window, a.n_sink);   // kSplitPrefix: no window
  const int per = static_cast<int>(chunk) / 32, v0 = split * per;
  int n_blk = seen.n_blocks - v0;
  n_blk = n_blk < 0 ? 0 : (n_blk > per ? per : n_blk);
  const long long cache0 = paged ? 0 : grp.prefix ? kvh * a.head_stride : (static_cast<long long>(row) * a.hkv + kvh) * a.tmax;

  // Cache row of token t (the same for 16 tokens from a multiple of 16 on,
  // plus t mod 16).  Where the query sees none of those tokens (which a page of
  // 16 may hold alone) the table is not followed; a page index out of range is
  // reported.  Page 0 stands in for both.
  auto row16 = [&](int t) -> long long {
    if (!paged) return cache0 + t;
    int page = 0;
    if (a.page_shift > 4 || t < seen.sink || max(t, seen.lo) < min(t + 16, seen.len))
      page = a.block_table[static_cast<long long>(row) * a.max_pages + (t >> a.page_shift)];
    if (page < 0 || page >= a.n_pages) {
      atomicOr(&g_decode_error, kErrBadPage);
      page = 0;
    }
    return ((static_cast<long long>(page) * a.hkv + kvh) << a.page_shift) + (t & ((1 << a.page_shift) - 1));
  };
  unsigned char *stage = smem + warp * 2 * C::STAGE;
  // Copies of block v's rows below tlen into stage s, and this lane's norms.
  uint16_t nk_next = 0, nv_next = 0;
  auto fetch = [&](int v, int s) {
    const int block = v < seen.n_sink_blocks ? v : v - seen.n_sink_blocks + seen.first;
    const int t0 = 32 * block, n = tlen - t0 < 32 ? tlen - t0 : 32;
    const long long ra = row16(t0), rb = n > 16 ? (paged ? row16(t0 + 16) : ra + 16) : 0;
    unsigned char *dk = stage + s * C::STAGE, *dv = dk + 32 * RS;
    for (int i = lane; i < n * (PB / 16); i += 32) {
      const int t = i / (PB / 16), p = 16 * (i % (PB / 16));
      const long long src = (t < 16 ? ra + t : rb + t - 16) * PB + p;
      cp_async16(dk + t * RS + p, pk + src);
      cp_async16(dv + t * RS + p, pv + src);
    }
    nk_next = nv_next = 0;
    if (lane < n) {
      const long long at = lane < 16 ? ra + lane : rb + lane - 16;
      nk_next = nk[at];
      nv_next = nv[at];
    }
  };
  if (warp < n_blk) fetch(v0 + warp, 0);
  cp_async_commit();

  __shared__ float2 fused_ml[8];
  if (a.fused) {   // the cluster has no earlier launch: this CTA rotates its own rows
    constexpr int E = D / 32;
    for (int h = warp; h < RG; h += kAnyWarps) {
      float x[E];
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = 0.f;
      if (h < rows) {
        const long long at = group_query(a, grp, kvh, h) * D + E * lane;
#pragma unroll
        for (int e = 0; e < E; ++e)
          x[e] = a.half_out ? __half2float(static_cast<const __half *>(a.q)[at + e]) : static_cast<const float *>(a.q)[at + e];
      }
      rotate_query<D>(x, a.params_k + static_cast<size_t>(kvh) * 2 * D, a.full, a.scale, lane);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int dim = E * lane + e;
        qs[(dim >> 5) * C::Q_GROUP + (dim & 31) * RG + h] = x[e];
      }
    }
  } else {
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the rotated queries
  pdl_launch_dependents();
  for (int i = tid; i < RG * D; i += kAnyThreads) {
    const int h = i / D, e = i % D;
    qs[(e >> 5) * C::Q_GROUP + (e & 31) * RG + h] = h < rows ? a.ws_qrot[group_query(a, grp, kvh, h) * D + e] : 0.f;
  }
  }
  __syncthreads();

  uint64_t acc[KD][RP];
  float m[RG], l[RG];
#pragma unroll
  for (int k = 0; k < KD; ++k)
#pragma unroll
    for (int r = 0; r < RP; ++r) acc[k][r] = 0ull;
#pragma unroll
  for (int r = 0; r < RG; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
  }
  float *wts = reinterpret_cast<float *>(smem + C::OFF_W) + warp * 32 * RG;

  int it = 0;
  for (int bi = warp; bi < n_blk; bi += kAnyWarps, ++it) {
    const int s = it & 1, v = v0 + bi;
    const float sk = __half2float(__ushort_as_half(nk_next)), svr = __half2float(__ushort_as_half(nv_next));
    if (bi + kAnyWarps < n_blk) fetch(v + kAnyWarps, s ^ 1);
    cp_async_commit();
    cp_async_wait<1>();
    __syncwarp();
    const unsigned char *kc = stage + s * C::STAGE, *vc = kc + 32 * RS;
    const int block = v < seen.n_sink_blocks ? v : v - seen.n_sink_blocks + seen.first;
    const unsigned mask = seen_mask(seen, block);
    const bool ok = (mask >> lane) & 1u;

    // ---- scores: four tokens and a quarter of the dimensions per lane ----
    uint64_t dot[4][RP];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < RP; ++r) dot[i][r] = 0ull;
    const int tl = lane & 7, sl = lane >> 3;
#pragma unroll 1
    for (int seg = 0; seg < D / 128; ++seg) {
      const int grp32 = 4 * seg + sl;                 // this lane's 32-code group
      uint32_t w[4][BITS];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const unsigned char *src = kc + (tl + 8 * i) * RS + grp32 * (4 * BITS);
        if constexpr (BITS == 4) {
          const uint4 u = *reinterpret_cast<const uint4 *>(src);
          w[i][0] = u.x;
          w[i][1] = u.y;
          w[i][2] = u.z;
          w[i][3] = u.w;
        } else if constexpr (BITS == 2) {
          const uint2 u = *reinterpret_cast<const uint2 *>(src);
          w[i][0] = u.x;
          w[i][1] = u.y;
        } else {
#pragma unroll
          for (int k = 0; k < 3; ++k) w[i][k] = *reinterpret_cast<const uint32_t *>(src + 4 * k);
        }
      }
      const float *qd = qs + grp32 * C::Q_GROUP;
#pragma unroll
      for (int quad = 0; quad < 8; ++quad) {
        uint32_t f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = quad_fields<BITS>(w[i], quad);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float *qe = qd + (4 * quad + e) * RG;
          uint64_t qv[RP];
          if constexpr (RG >= 4) {
#pragma unroll
            for (int r = 0; r < RG / 4; ++r) {
              const ulonglong2 u = *reinterpret_cast<const ulonglong2 *>(qe + 4 * r);
              qv[2 * r] = u.x;
              qv[2 * r + 1] = u.y;
            }
          } else {
            qv[0] = *reinterpret_cast<const uint64_t *>(qe);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float c = *reinterpret_cast<const float *>(tab + (e == 0 ? (f[i] << 2) & 0x3Cu : (f[i] >> (4 * e - 2)) & 0x3Cu));
            const uint64_t c2 = f2_pack(c, c);
#pragma unroll
            for (int r = 0; r < RP; ++r) dot[i][r] = f2_fma(c2, qv[r], dot[i][r]);
          }
        }
      }
    }
    // Add the four slices: lanes s and s ^ 2 share tokens (0, 1) and (2, 3),
    // then s and s ^ 1 one each; lane L = t + 8 s is left with token L.
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        const uint64_t give = (sl & 2) ? dot[i][r] : dot[i + 2][r], keep = (sl & 2) ? dot[i + 2][r] : dot[i][r];
        dot[i][r] = f2_add(keep, __shfl_xor_sync(0xffffffffu, give, 16));
      }
#pragma unroll
    for (int r = 0; r < RP; ++r) {
      const uint64_t give = (sl & 1) ? dot[0][r] : dot[1][r], keep = (sl & 1) ? dot[1][r] : dot[0][r];
      dot[0][r] = f2_add(keep, __shfl_xor_sync(0xffffffffu, give, 8));
    }
    // ---- softmax (log2 domain); the reference maximum moves only when a
    // score passes it by 8, so p <= 2^8 ----
    float x[RG];
    bool over = false;
#pragma unroll
    for (int r = 0; r < RP; ++r) {
      f2_unpack(dot[0][r], x[2 * r], x[2 * r + 1]);
      x[2 * r] = ok ? x[2 * r] * sk : -INFINITY;
      x[2 * r + 1] = ok ? x[2 * r + 1] * sk : -INFINITY;
      over |= x[2 * r] > m[2 * r] + 8.f || x[2 * r + 1] > m[2 * r + 1] + 8.f;
    }
    if (__any_sync(0xffffffffu, over)) {
      float f[RG];
#pragma unroll
      for (int r = 0; r < RG; ++r) {
        float mx = x[r];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        mx = fmaxf(m[r], mx);
        f[r] = m[r] == -INFINITY ? 0.f : exp2f(m[r] - mx);
        l[r] *= f[r];
        m[r] = mx;
      }
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        const uint64_t f2 = f2_pack(f[2 * r], f[2 * r + 1]);
#pragma unroll
        for (int k = 0; k < KD; ++k) acc[k][r] = f2_mul(acc[k][r], f2);
      }
    }
    const float sv = ok ? svr : 0.f;
#pragma unroll
    for (int r = 0; r < RG; ++r) {
      const float p = ok ? exp2f(x[r] - m[r]) : 0.f;
      l[r] += p;
      x[r] = p * sv;
    }
#pragma unroll
    for (int r = 0; r < RP; ++r) *reinterpret_cast<float2 *>(wts + lane * RG + 2 * r) = make_float2(x[2 * r], x[2 * r + 1]);
    __syncwarp();

    // ---- values: this lane's dimensions over the block's tokens; a token that
    // is not seen has weight 0 (and codes of whatever the stage held) ----
    const int n_tok = 32 - __clz(mask);              // past the last token seen
#pragma unroll 2
    for (int j = 0; j < n_tok; ++j) {
      uint64_t w2[RP];
      if constexpr (RG >= 4) {
#pragma unroll
        for (int r = 0; r < RG / 4; ++r) {
          const ulonglong2 u = *reinterpret_cast<const ulonglong2 *>(wts + j * RG + 4 * r);
          w2[2 * r] = u.x;
          w2[2 * r + 1] = u.y;
        }
      } else {
        w2[0] = *reinterpret_cast<const uint64_t *>(wts + j * RG);
      }
      const uint32_t *vr = reinterpret_cast<const uint32_t *>(vc + j * RS);
#pragma unroll
      for (int u = 0; u < KD / 4; ++u) {
        const uint32_t f = quad_fields<BITS>(vr, (KD / 4) * lane + u);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float c = *reinterpret_cast<const float *>(tab + (e == 0 ? (f << 2) & 0x3Cu : (f >> (4 * e - 2)) & 0x3Cu));
          const uint64_t c2 = f2_pack(c, c);
#pragma unroll
          for (int r = 0; r < RP; ++r) acc[4 * u + e][r] = f2_fma(c2, w2[r], acc[4 * u + e][r]);
        }
      }
    }
    __syncwarp();   // the stage and the weights may be overwritten
  }

  // ---- merge the four warps in a fixed order, one state per query row ----
  cp_async_wait<0>();
#pragma unroll
  for (int r = 0; r < RG; ++r) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
    if (lane == 0) ml[warp * RG + r] = make_float2(m[r], l[r]);
  }
  __syncthreads();   // every warp is done with its stages
  float *sl = reinterpret_cast<float *>(smem);   // [warp][RG][D]
#pragma unroll
  for (int r = 0; r < RP; ++r) {
#pragma unroll
    for (int k = 0; k < KD; ++k) {
      float u0, u1;
      f2_unpack(acc[k][r], u0, u1);
      sl[(warp * RG + 2 * r) * D + KD * lane + k] = u0;
      sl[(warp * RG + 2 * r + 1) * D + KD * lane + k] = u1;
    }
  }
  __syncthreads();
  for (int h = 0; h < rows; ++h) {
    float mx = -INFINITY, f[kAnyWarps], lt = 0.f;
#pragma unroll
    for (int w = 0; w < kAnyWarps; ++w) mx = fmaxf(mx, ml[w * RG + h].x);
#pragma unroll
    for (int w = 0; w < kAnyWarps; ++w) {
      const float2 u = ml[w * RG + h];
      f[w] = u.x == -INFINITY ? 0.f : exp2f(u.x - mx);
      lt += u.y * f[w];
    }
    const long long slot = a.fused ? 0 : group_slot(a, grp, kvh, h, split);
    float *acc_out = a.fused ? qs + h * D : a.ws_acc + slot * D;   // fused: over the queries
    for (int i = tid; i < D; i += kAnyThreads) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kAnyWarps; ++w) sum += sl[(w * RG + h) * D + i] * f[w];
      acc_out[i] = sum;
    }
    if (a.fused) {
      if (tid == 0) fused_ml[h] = make_float2(mx, lt);   // log2 domain
    } else if (tid == 0) a.ws_ml[slot] = make_float2(mx == -INFINITY ? -INFINITY : mx * 0.69314718055994531f, lt);
  }
  if (a.fused) cluster_finish<D>(a, grp, kvh, qs, fused_ml, warp, lane, kAnyWarps);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

template <typename T, int D>
int launch_prep_rotate(int variant, const SplitArgs &a, cudaStream_t st) {
  const long long rows = static_cast<long long>(a.batch) * a.hq;
  const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
  if (variant == ISOQ_FULL)
    prep_rotate_kernel<T, D, true><<<grid, 128, 0, st>>>(a);
  else
    prep_rotate_kernel<T, D, false><<<grid, 128, 0, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ISOQ_OK : set_error(ISOQ_ERR_CUDA, "query rotation launch: %s", cudaGetErrorString(e));
}

int run_prep_rotate(int dtype, int d, int variant, const SplitArgs &a, cudaStream_t st) {
  if (dtype == ISOQ_F16) {
    if (d == 128) return launch_prep_rotate<__half, 128>(variant, a, st);
    if (d == 256) return launch_prep_rotate<__half, 256>(variant, a, st);
    return launch_prep_rotate<__half, 512>(variant, a, st);
  }
  if (d == 128) return launch_prep_rotate<float, 128>(variant, a, st);
  if (d == 256) return launch_prep_rotate<float, 256>(variant, a, st);
  return launch_prep_rotate<float, 512>(variant, a, st);
}

template <int D, int BITS, int RG>
int launch_split_any(const SplitArgs &a, cudaStream_t st) {
  using C = AnyCfg<D, BITS, RG>;
  auto kernel = split_any_kernel<D, BITS, RG>;
  static std::atomic<unsigned long long> allowed;
  const cudaError_t c = allow_smem(allowed, reinterpret_cast<const void *>(kernel), C::SMEM);
  if (c != cudaSuccess) return set_error(ISOQ_ERR_CUDA, "split: %s", cudaGetErrorString(c));
  if (a.fused) {
    cudaError_t e = launch_cluster(kernel, dim3(a.n_splits, a.hkv, group_count(a, a.mode)), dim3(kAnyThreads), C::SMEM, st, a.n_splits, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? ISOQ_OK : set_error(ISOQ_ERR_CUDA, "split cluster launch: %s", cudaGetErrorString(e));
  }
  const int nx = a.mode == kSplitPrefix && a.n_splits_p > a.n_splits ? a.n_splits_p : a.n_splits;
  cudaError_t e = launch_pdl(kernel, dim3(nx, a.hkv, group_count(a, a.mode)), dim3(kAnyThreads), C::SMEM, st, a);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? ISOQ_OK : set_error(ISOQ_ERR_CUDA, "split launch: %s", cudaGetErrorString(e));
}

template <int D, int BITS>
int run_split_any_r(const SplitArgs &a, cudaStream_t st) {
  const int rows = a.mode == kSplitPrefix && a.zrow_size_p > a.zrow_size ? a.zrow_size_p : a.zrow_size;
  if (rows <= 2) return launch_split_any<D, BITS, 2>(a, st);
  if (rows <= 4) return launch_split_any<D, BITS, 4>(a, st);
  return launch_split_any<D, BITS, 8>(a, st);
}

template <int D>
int run_split_any_b(int bits, const SplitArgs &a, cudaStream_t st) {
  if (bits == 2) return run_split_any_r<D, 2>(a, st);
  if (bits == 3) return run_split_any_r<D, 3>(a, st);
  return run_split_any_r<D, 4>(a, st);
}

int run_split_any(int d, int bits, const SplitArgs &a, cudaStream_t st) {
  if (d == 128) return run_split_any_b<128>(bits, a, st);
  if (d == 256) return run_split_any_b<256>(bits, a, st);
  return run_split_any_b<512>(bits, a, st);
}
