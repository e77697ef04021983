// Device error word collection: each kernel translation unit owns one 32-bit
// word per device that its kernels set bits of when they meet an error.

#include <cuda_runtime.h>

#include <cstdio>

#include "internal.h"

extern "C" __attribute__((visibility("hidden"))) cudaError_t isoq_detail_quant_error_word(void **word);
extern "C" __attribute__((visibility("hidden"))) cudaError_t isoq_detail_decode_error_word(void **word);
extern "C" __attribute__((visibility("hidden"))) cudaError_t isoq_detail_serve_error_word(void **word);

namespace {

// The three words, cleared where they are set; one synchronisation, and
// another one where there is something to clear.
cudaError_t take_words(unsigned (&w)[3], cudaStream_t s) {
  void *at[3] = {};
  cudaError_t e = isoq_detail_quant_error_word(&at[0]);
  if (e == cudaSuccess) e = isoq_detail_decode_error_word(&at[1]);
  if (e == cudaSuccess) e = isoq_detail_serve_error_word(&at[2]);
  for (int i = 0; i < 3 && e == cudaSuccess; ++i)
    e = cudaMemcpyAsync(&w[i], at[i], sizeof(unsigned), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess || !(w[0] | w[1] | w[2])) return e;
  for (int i = 0; i < 3 && e == cudaSuccess; ++i)
    if (w[i]) e = cudaMemsetAsync(at[i], 0, sizeof(unsigned), s);
  return e == cudaSuccess ? cudaStreamSynchronize(s) : e;
}

}  // namespace

extern "C" int isoq_check_device_error(isoq_stream_t stream) {
  isoq::clear_error();
  unsigned w[3] = {};
  const cudaError_t e = take_words(w, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return isoq::set_error(ISOQ_ERR_CUDA, "error word: %s", cudaGetErrorString(e));
  const unsigned all = w[0] | w[1] | w[2];
  if (!all) return ISOQ_OK;
  // The first one's status; the message names every one.
  const struct { unsigned bit; int status; const char *what; } kinds[] = {
      {1u, ISOQ_ERR_TIMEOUT, "device wait timed out"},
      {8u, ISOQ_ERR_INVALID_ARG, "paged cache: a page index or slot outside the pages"},
      {16u, ISOQ_ERR_INVALID_ARG, "block tables: no room for a request"},
      {2u, ISOQ_ERR_INVALID_ARG, "decode append: a row already held Tmax tokens"},
      {4u, ISOQ_ERR_CUDA, "prefill: dynamic shared memory not 1024-byte aligned"}};
  int status = ISOQ_OK, n = 0;
  char text[400] = "";
  for (const auto &k : kinds)
    if (all & k.bit) {
      if (status == ISOQ_OK) status = k.status;
      n += snprintf(text + n, sizeof(text) - n, "%s%s", n ? "; " : "", k.what);
    }
  return isoq::set_error(status, "%s (quantize=%u, decode=%u, serve=%u)", text, w[0], w[1], w[2]);
}
