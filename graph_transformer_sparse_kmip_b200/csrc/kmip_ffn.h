// kmip_ffn.h -- launchers of the gated feed-forward block, shared between its
// entry points (kmip_ffn.cu) and its kernels.
#pragma once

#include "kmip_internal.h"

namespace kmip {

struct FfnArgs {
  const void* x;   // [N, C]
  const void* wg;  // [F, C]
  const void* wu;  // [F, C]
  const void* wd;  // [C, F]
  int N, C, F;
  int act;
  int* status;
};

// tcgen05 kernels (bf16, kmip_ffn_tc.cu); C and F multiples of 8.
cudaError_t launch_ffn_glu(const FfnArgs& a, void* h, cudaStream_t stream);
cudaError_t launch_ffn_down(const FfnArgs& a, const void* h, void* y, void* scratch,
                            cudaStream_t stream);
cudaError_t launch_ffn_glu_bwd(const FfnArgs& a, const void* dy, void* da, void* db, void* h,
                               cudaStream_t stream);
cudaError_t launch_ffn_dx(const FfnArgs& a, const void* da, const void* db, void* dx,
                          void* scratch, cudaStream_t stream);
cudaError_t launch_ffn_wgrad(const FfnArgs& a, const void* dy, const void* da, const void* db,
                             const void* h, void* dwg, void* dwu, void* dwd, void* scratch,
                             cudaStream_t stream);
// Partial tiles of the forward's (down) and of the backward's (dx, then wgrad)
// products.
size_t ffn_fwd_scratch(const FfnArgs& a);
size_t ffn_bwd_scratch(const FfnArgs& a);

// A few rows, either type (kmip_ffn_rows.cu): h [N, F] fp32 scratch.
constexpr int kFfnFewRows = 16;
cudaError_t launch_ffn_rows_fwd(kmip_dtype_t dtype, const FfnArgs& a, float* h, void* y,
                                cudaStream_t stream);

// fp32 kernels (kmip_ffn_f32.cu); C and F multiples of 4.  h: [N, F], abd:
// [3][N, F], part: ffn_f32_scratch() bytes, all scratch.
size_t ffn_f32_scratch();
cudaError_t launch_ffn_f32_fwd(const FfnArgs& a, float* h, float* y, float* part,
                               cudaStream_t stream);
cudaError_t launch_ffn_f32_bwd(const FfnArgs& a, const float* dy, float* abd, float* dx,
                               float* dwg, float* dwu, float* dwd, float* part,
                               cudaStream_t stream);

}  // namespace kmip
