// kmip_ffn.cu -- entry points of the gated feed-forward block (kmip_ffn_fwd,
// kmip_ffn_bwd): argument checks, scratch and the order of the kernels.
#include "kmip_ffn.h"

namespace kmip {
namespace {

kmip_status_t check_ffn(int64_t N, int C, int F, int act, int dtype) {
  if (N < 0 || N > INT32_MAX || C < 1 || F < 1) return KMIP_ERR_INVALID_ARG;
  if (dtype != KMIP_BF16 && dtype != KMIP_F32) return KMIP_ERR_INVALID_ARG;
  if (act < KMIP_ACT_NONE || act > KMIP_ACT_RELU) return KMIP_ERR_INVALID_ARG;
  if (N > kMaxRows || C % 8 || F % 8 || C > 65536 || F > 65536) return KMIP_ERR_UNSUPPORTED;
  // tiles are counted in 32 bits
  const int64_t wide = C > F ? C : F;
  if ((N / 64 + 1) * (wide / 64 + 1) * 3 > INT32_MAX) return KMIP_ERR_UNSUPPORTED;
  return KMIP_OK;
}

kmip_status_t to_status(cudaError_t e) {
  if (e == cudaSuccess) return KMIP_OK;
  cudaGetLastError();
  return KMIP_ERR_CUDA;
}

template <typename... P>
bool all_aligned(P... ptrs) {
  return (... && (ptrs && aligned16(ptrs)));
}

size_t round16(size_t n) { return (n + 15) & ~(size_t)15; }

}  // namespace
}  // namespace kmip

using namespace kmip;

extern "C" __attribute__((visibility("default"))) kmip_status_t kmip_ffn_fwd(
    const void* x, const void* Wg, const void* Wu, const void* Wd, int64_t N, int C, int F,
    kmip_act_t act, void* y, kmip_stream_t stream_, kmip_dtype_t dtype) {
  const kmip_status_t st = check_ffn(N, C, F, act, dtype);
  if (st != KMIP_OK) return st;
  if (N == 0) return KMIP_OK;
  if (!all_aligned(x, Wg, Wu, Wd, y)) return KMIP_ERR_INVALID_ARG;
  const size_t es = dtype == KMIP_BF16 ? 2 : 4, nc = es * N * C, cf = es * C * F;
  if (overlapping({{y, nc}, {x, nc}, {Wg, cf}, {Wu, cf}, {Wd, cf}}, 1))
    return KMIP_ERR_INVALID_ARG;
  int* status = status_ptr();
  if (!status) return KMIP_ERR_CUDA;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const FfnArgs a{x, Wg, Wu, Wd, (int)N, C, F, act, status};
  const size_t nf = (size_t)N * F;
  void* scratch = nullptr;
  cudaError_t e;
  if (N <= kFfnFewRows) {
    e = scratch_alloc(&scratch, 4 * nf, stream);
    if (e != cudaSuccess) return to_status(e);
    e = launch_ffn_rows_fwd(dtype, a, static_cast<float*>(scratch), y, stream);
  } else if (dtype == KMIP_BF16) {
    const size_t mat = round16(2 * nf);
    e = scratch_alloc(&scratch, mat + ffn_fwd_scratch(a), stream);
    if (e != cudaSuccess) return to_status(e);
    e = launch_ffn_glu(a, scratch, stream);
    if (e == cudaSuccess)
      e = launch_ffn_down(a, scratch, y, static_cast<char*>(scratch) + mat, stream);
  } else {
    e = scratch_alloc(&scratch, 4 * nf + ffn_f32_scratch(), stream);
    if (e != cudaSuccess) return to_status(e);
    float* h = static_cast<float*>(scratch);
    e = launch_ffn_f32_fwd(a, h, static_cast<float*>(y), h + nf, stream);
  }
  const cudaError_t ef = cudaFreeAsync(scratch, stream);
  return to_status(e != cudaSuccess ? e : ef);
}

extern "C" __attribute__((visibility("default"))) kmip_status_t kmip_ffn_bwd(
    const void* dy, const void* x, const void* Wg, const void* Wu, const void* Wd, int64_t N,
    int C, int F, kmip_act_t act, void* dx, void* dWg, void* dWu, void* dWd,
    kmip_stream_t stream_, kmip_dtype_t dtype) {
  const kmip_status_t st = check_ffn(N, C, F, act, dtype);
  if (st != KMIP_OK) return st;
  if (!all_aligned(Wg, Wu, Wd, dWg, dWu, dWd)) return KMIP_ERR_INVALID_ARG;
  if (N > 0 && !all_aligned(dy, x, dx)) return KMIP_ERR_INVALID_ARG;
  const size_t es = dtype == KMIP_BF16 ? 2 : 4, nf = (size_t)N * F;
  const size_t nc = es * N * C, cf = es * C * F;
  if (overlapping({{dx, nc}, {dWg, cf}, {dWu, cf}, {dWd, cf}, {dy, nc}, {x, nc}, {Wg, cf},
                   {Wu, cf}, {Wd, cf}}, 4))
    return KMIP_ERR_INVALID_ARG;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  cudaError_t e;
  if (N == 0) {
    e = cudaMemsetAsync(dWg, 0, cf, stream);
    if (e == cudaSuccess) e = cudaMemsetAsync(dWu, 0, cf, stream);
    if (e == cudaSuccess) e = cudaMemsetAsync(dWd, 0, cf, stream);
    return to_status(e);
  }
  int* status = status_ptr();
  if (!status) return KMIP_ERR_CUDA;
  const FfnArgs a{x, Wg, Wu, Wd, (int)N, C, F, act, status};
  void* scratch = nullptr;
  if (dtype == KMIP_BF16) {
    const size_t mat = round16(2 * nf);
    e = scratch_alloc(&scratch, 3 * mat + ffn_bwd_scratch(a), stream);
    if (e != cudaSuccess) return to_status(e);
    char *da = static_cast<char*>(scratch), *db = da + mat, *h = db + mat;
    e = launch_ffn_glu_bwd(a, dy, da, db, h, stream);
    if (e == cudaSuccess) e = launch_ffn_dx(a, da, db, dx, h + mat, stream);
    if (e == cudaSuccess)
      e = launch_ffn_wgrad(a, dy, da, db, h, dWg, dWu, dWd, h + mat, stream);
  } else {
    e = scratch_alloc(&scratch, 12 * nf + ffn_f32_scratch(), stream);
    if (e != cudaSuccess) return to_status(e);
    float* abd = static_cast<float*>(scratch);
    e = launch_ffn_f32_bwd(a, static_cast<const float*>(dy), abd, static_cast<float*>(dx),
                           static_cast<float*>(dWg), static_cast<float*>(dWu),
                           static_cast<float*>(dWd), abd + 3 * nf, stream);
  }
  const cudaError_t ef = cudaFreeAsync(scratch, stream);
  return to_status(e != cudaSuccess ? e : ef);
}
