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

