// The shared prefix on the 5th-generation tensor cores: a KV head's batch x
// group query rows, 128 to a tile, against chunks of the prefix (the
// kPfPrefix kind of prefill.cuh), so that one unpacking of a code serves 128
// rows.  Included by isoq_serve.cu inside namespace isoq::decode.

// Query rows in the operand layout: row r of KV head kvh is rotated (the order
// of prep_i8_kernel), scaled (query_scale), split into float16 hi and lo parts
// and written to its 128-row tile, 128B-swizzled K-major, its inverse scale
// behind the two; rows past the batch are zeros.  One warp per row.
template <int D, bool FULL>
__global__ void __launch_bounds__(128) prep_prefix_kernel(const SplitArgs a, unsigned char *tiles, int row_tiles) {
  using C = TcCfg<D>;
  constexpr int E = D / 32, QBLK = kTcRows * 128;
  const int r = static_cast<int>(blockIdx.x) * 4 + (threadIdx.x >> 5), kvh = blockIdx.y, lane = threadIdx.x & 31;
  float x[E];
  if (r < a.batch * a.group) {
    const __half *q = static_cast<const __half *>(a.q) +
                      (static_cast<long long>(r / a.group) * a.hq + kvh * a.group + r % a.group) * D + E * lane;
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = __half2float(q[e]);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = 0.f;
  }
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
  const float *prm = a.params_k + static_cast<size_t>(kvh) * 2 * D;
  const int m = r % kTcRows;
  unsigned char *hi = tiles + (static_cast<long long>(kvh) * row_tiles + r / kTcRows) * C::Q_TILE;
  unsigned char *lo = hi + C::Q_BYTES;
  Quat rot[E / 4];
  float big = 0.f, back;
#pragma unroll
  for (int u = 0; u < E / 4; ++u) {
    const int bi = (E / 4) * lane + u;
    const Quat v{x[4 * u] * inv, x[4 * u + 1] * inv, x[4 * u + 2] * inv, x[4 * u + 3] * inv};
    rot[u] = block_forward(load_quat(prm + 8 * bi), load_quat(prm + 8 * bi + 4), v, FULL);
    big = fmaxf(fmaxf(fmaxf(big, fabsf(rot[u].w)), fabsf(rot[u].x)), fmaxf(fabsf(rot[u].y), fabsf(rot[u].z)));
  }
  big = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(big)));   // (not negative: ordered as integers)
  const float sc = query_scale(big, back);
  if (lane == 0) reinterpret_cast<float *>(hi + 2 * C::Q_BYTES)[m] = back;
#pragma unroll
  for (int u = 0; u < E / 4; ++u) {
    const int bi = (E / 4) * lane + u;
    const Quat y{rot[u].w * sc, rot[u].x * sc, rot[u].y * sc, rot[u].z * sc};
    const __half2 h0 = __floats2half2_rn(y.w, y.x), h1 = __floats2half2_rn(y.y, y.z);
    const float2 f0 = __half22float2(h0), f1 = __half22float2(h1);
    const uint32_t off = tc_off(m, 4 * bi, QBLK);
    *reinterpret_cast<uint2 *>(hi + off) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&h0), *reinterpret_cast<const uint32_t *>(&h1));
    *reinterpret_cast<uint2 *>(lo + off) = make_uint2(pack_f16x2(y.w - f0.x, y.x - f0.y), pack_f16x2(y.y - f1.x, y.z - f1.y));
  }
}

bool tc_prefix(int dtype, int d, int bits) { return dtype == ISOQ_F16 && bits == 3 && (d == 128 || d == 256); }

template <int D>
int launch_prep_prefix(int variant, const SplitArgs &a, unsigned char *tiles, int row_tiles, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(row_tiles * kTcRows / 4), static_cast<unsigned>(a.hkv));
  if (variant == ISOQ_FULL)
    prep_prefix_kernel<D, true><<<grid, 128, 0, st>>>(a, tiles, row_tiles);
  else
    prep_prefix_kernel<D, false><<<grid, 128, 0, st>>>(a, tiles, row_tiles);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ISOQ_OK : set_error(ISOQ_ERR_CUDA, "prefix query launch: %s", cudaGetErrorString(e));
}

int run_prep_prefix(int d, int variant, const SplitArgs &a, unsigned char *tiles, int row_tiles, cudaStream_t st) {
  (void)d;   // 256: at d = 128 the kernel prepares its queries itself
  return launch_prep_prefix<256>(variant, a, tiles, row_tiles, st);
}

template <int D>
int launch_prefix_tc(const PrefillArgs &p, int splits, cudaStream_t st) {
  using C = TcCfg<D>;
  auto kernel = prefill_tc_kernel<__half, D, true, 1, kPfPrefix>;
  static std::atomic<unsigned long long> allowed;
  const cudaError_t c = allow_smem(allowed, reinterpret_cast<const void *>(kernel), C::SMEM);
  if (c != cudaSuccess) return set_error(ISOQ_ERR_CUDA, "prefix: %s", cudaGetErrorString(c));
  cudaError_t e = launch_pdl(kernel, dim3(p.row_tiles, p.hkv, splits), dim3(kTcThreads), C::SMEM, st, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? ISOQ_OK : set_error(ISOQ_ERR_CUDA, "prefix launch: %s", cudaGetErrorString(e));
}

int run_prefix_tc(int d, int variant, const SplitArgs &a, const unsigned char *tiles, int row_tiles, int splits,
                  int chunk, cudaStream_t st) {
  PrefillArgs p{};
  p.q = a.q;
  p.params_k = a.params_k;
  p.packed_k = a.prefix_k;
  p.packed_v = a.prefix_v;
  p.norms_k = a.prefix_nk;
  p.norms_v = a.prefix_nv;
  p.prefix_len = a.prefix_len;
  p.q_tiles = tiles;
  p.row_tiles = row_tiles;
  p.chunk = chunk;
  p.head_stride = a.head_stride;
  p.tmax = a.prefix_max;
  p.batch = a.batch;
  p.hq = a.hq;
  p.hkv = a.hkv;
  p.group = a.group;
  p.ws_acc = a.ws_acc;
  p.ws_ml = a.ws_ml;
  p.slot_stride = a.slot_stride;
  p.score_unit = static_cast<float>(a.scale * 1.4426950408889634);
  prefill_tables(p, d);
  if (d == 256) return launch_prefix_tc<256>(p, splits, st);
  const dim3 grid(static_cast<unsigned>(row_tiles), static_cast<unsigned>(a.hkv), static_cast<unsigned>(splits));
  return variant == ISOQ_FULL ? launch_rows_tc<kPfPrefix, true>(p, grid, 1, st) : launch_rows_tc<kPfPrefix, false>(p, grid, 1, st);
}

// Windowed chunked prefill at d = 128.
int run_window_rows(int variant, PrefillArgs a, cudaStream_t st) {
  prefill_tables(a, 128);
  const int per = kTcRows / a.group;
  const dim3 grid(static_cast<unsigned>((a.tq + per - 1) / per), static_cast<unsigned>(a.hkv), static_cast<unsigned>(a.batch));
  // CTAs per row tile: as many as the SMs hold at once, at most 8, each with
  // two tiles of tokens or more (of the most that a row tile can see).
  const int64_t ctas = static_cast<int64_t>(grid.x) * grid.y * grid.z;
  const int64_t tiles = most_blocks(a.tmax, static_cast<int64_t>(a.window) + per, a.n_sink) / 4 + 1;
  int64_t ranks = 148 / ctas < kMaxClusterSplits ? 148 / ctas : kMaxClusterSplits;
  ranks = ranks < tiles / 2 ? ranks : tiles / 2;
  const int n = ranks > 1 ? static_cast<int>(ranks) : 1;
  return variant == ISOQ_FULL ? launch_rows_tc<kPfWindow, true>(a, grid, n, st) : launch_rows_tc<kPfWindow, false>(a, grid, n, st);
}
