// Device helpers shared by the decode translation units (isoq_decode.cu,
// isoq_serve.cu), each of which includes this file inside namespace
// isoq::decode: the error word, programmatic dependent launch, the rotation
// of vectors held in shared memory, element conversions.
#pragma once

using namespace isoq::dev;

// The translation unit's device error word (isoq_check_device_error).
static __device__ unsigned int g_decode_error = 0;

// Launch with programmatic dependent launch: the kernel may start while the
// previous kernel on the stream is still running (once that kernel's CTAs
// have all started or signalled), and must execute griddepcontrol.wait
// before reading anything the previous kernel writes.  Used only for
// kernels whose predecessor is one of ours (prep -> split -> combine).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                       Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Lets `kernel` take `bytes` of dynamic shared memory on the current device.
// The attribute belongs to the device: `done` has a bit for each one that has
// it already.
inline cudaError_t allow_smem(std::atomic<unsigned long long> &done, const void *kernel, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Barrier over the threads taking part in a shared-memory rotation: the whole
// CTA (bar_id 0 -> __syncthreads) or a named barrier over `nthreads` threads.
__device__ __forceinline__ void rotation_sync(int bar_id, int nthreads) {
  if (bar_id == 0)
    __syncthreads();
  else
    named_barrier(bar_id, nthreads);
}

// Forward rotation q~ = R q of `nvec` vectors v[nvec][D] held in shared
// memory, all sharing one head's parameters, by threads [0, nthreads): WHT
// butterflies (stride h = 1 ... d/2) for all vectors per barrier, 1/sqrt(d),
// then the per-block quaternion map.
template <int D, bool FULL>
__device__ void rotate_forward_smem(float *v, int nvec, const float *params_head, int tid,
                                    int nthreads, int bar_id) {
#pragma unroll 1
  for (int h = 1; h < D; h <<= 1) {
    for (int idx = tid; idx < nvec * (D / 2); idx += nthreads) {
      const int g = idx / (D / 2), p = idx % (D / 2);
      float *w = v + g * D;
      const int i = (p / h) * 2 * h + (p % h);
      const float a = w[i], b = w[i + h];
      w[i] = a + b;
      w[i + h] = a - b;
    }
    rotation_sync(bar_id, nthreads);
  }
  const float inv = rsqrtf(static_cast<float>(D));
  for (int idx = tid; idx < nvec * (D / 4); idx += nthreads) {
    const int g = idx / (D / 4), bi = idx % (D / 4);
    float *w = v + g * D + 4 * bi;
    const Quat x{w[0] * inv, w[1] * inv, w[2] * inv, w[3] * inv};
    const Quat u = block_forward(load_quat(params_head + 8 * bi), load_quat(params_head + 8 * bi + 4), x, FULL);
    w[0] = u.w;
    w[1] = u.x;
    w[2] = u.y;
    w[3] = u.z;
  }
  rotation_sync(bar_id, nthreads);
}

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

inline bool aligned(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// ---------------------------------------------------------------------------
// The last step of a fused decode: the CTAs of a cluster hold the partial
// states of the same `rows` query rows (at most 8), acc [rows][D] relative to
// 2^m and (m, l) per row, in their shared memory.  One warp per row, the rows
// dealt out over the cluster: the states are read from every CTA, merged in
// rank order, normalised, rotated back by R_V^T (lane: D / 32 dims; the order
// of combine_kernel) and stored.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_address(const void *p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 peer_load4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ float2 peer_load2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

constexpr int kMaxClusterSplits = 8;

template <int D>
__device__ void cluster_finish(const SplitArgs &a, const RowGroup &g, int kvh, const float *acc, const float2 *ml,
                               int warp, int lane, int warps) {
  constexpr int E = D / 32;
  cluster_sync();   // every CTA's states are in place
  const int n = static_cast<int>(cluster_size());
  for (int h = static_cast<int>(cluster_rank()) + n * warp; h < g.rows; h += n * warps) {
    // Lane r reads rank r's (m, l); all ranks' accumulators are on their way
    // at once.
    const float2 mine = lane < n ? peer_load2(peer_address(ml + h, lane)) : make_float2(-INFINITY, 0.f);
    float4 v[kMaxClusterSplits][E / 4];
#pragma unroll
    for (int r = 0; r < kMaxClusterSplits; ++r) {
      const uint32_t at = peer_address(acc + h * D + E * lane, r < n ? r : 0);
#pragma unroll
      for (int e = 0; e < E / 4; ++e) v[r][e] = peer_load4(at + 16 * e);
    }
    float m = mine.x;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    m = __shfl_sync(0xffffffffu, m, 0);
    const float w_mine = mine.x == -INFINITY ? 0.f : exp2f(mine.x - m), l_mine = mine.y * w_mine;
    float l = 0.f, x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = 0.f;
#pragma unroll
    for (int r = 0; r < kMaxClusterSplits; ++r) {
      const float w = __shfl_sync(0xffffffffu, w_mine, r);   // 0 past the cluster
      l += __shfl_sync(0xffffffffu, l_mine, r);
      if (r < n) {
#pragma unroll
        for (int e = 0; e < E / 4; ++e) {
          x[4 * e] = fmaf(v[r][e].x, w, x[4 * e]);
          x[4 * e + 1] = fmaf(v[r][e].y, w, x[4 * e + 1]);
          x[4 * e + 2] = fmaf(v[r][e].z, w, x[4 * e + 2]);
          x[4 * e + 3] = fmaf(v[r][e].w, w, x[4 * e + 3]);
        }
      }
    }
    const float inv_l = l > 0.f ? 1.f / l : 0.f;
    const float *prm = a.params_v + static_cast<size_t>(kvh) * 2 * D;
#pragma unroll
    for (int u = 0; u < E / 4; ++u) {
      const int bi = (E / 4) * lane + u;
      const Quat q = block_inverse(load_quat(prm + 8 * bi), load_quat(prm + 8 * bi + 4),
                                   Quat{x[4 * u] * inv_l, x[4 * u + 1] * inv_l, x[4 * u + 2] * inv_l, x[4 * u + 3] * inv_l}, a.full);
      x[4 * u] = q.w;
      x[4 * u + 1] = q.x;
      x[4 * u + 2] = q.y;
      x[4 * u + 3] = q.z;
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
      const float sgn = (lane & lm) ? -1.f : 1.f;
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = fmaf(x[e], sgn, __shfl_xor_sync(0xffffffffu, x[e], lm));
    }
    const float inv = rsqrtf(static_cast<float>(D));
    const long long at = group_query(a, g, kvh, h) * D + E * lane;
#pragma unroll
    for (int e = 0; e < E; e += 4) {
      if (a.half_out) {
        const __half2 p = __floats2half2_rn(x[e] * inv, x[e + 1] * inv), q = __floats2half2_rn(x[e + 2] * inv, x[e + 3] * inv);
        *reinterpret_cast<uint2 *>(static_cast<__half *>(a.out) + at + e) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&p), *reinterpret_cast<const uint32_t *>(&q));
      } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at + e) = make_float4(x[e] * inv, x[e + 1] * inv, x[e + 2] * inv, x[e + 3] * inv);
      }
    }
  }
  cluster_sync();   // no CTA ends while its shared memory is read
}

// Launch with clusters of `ranks` CTAs along x.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, int ranks,
                           Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
