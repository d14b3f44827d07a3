// Interface between the C-ABI layer (ssm_api.hip) and layer norm's launchers.  Arguments have already been validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssm {

// Layer norm over rows of W elements (ssm_layernorm.hip).
struct LayerNormArgs {
  const void* x;        // [rows, H, W]
  const float* weight;  // [H, W], nullable
  const float* bias;    // [H, W], nullable
  float eps;
  void* y;
  float* mean;          // [rows, H]: written by the forward (nullable), read by the backward
  float* rstd;          // as mean
  // backward
  const void* dy;
  void* dx;
  float* dweight;       // [H, W]; both parameter gradients or neither
  float* dbias;
  int64_t rows, H, W;
  int dtype;
  hipStream_t stream;
};
int64_t layernorm_max_width();
size_t layernorm_workspace_bytes(const LayerNormArgs& a);  // of the backward, for tensors of any alignment
hipError_t launch_layernorm_fwd(const LayerNormArgs& a);
hipError_t launch_layernorm_bwd(const LayerNormArgs& a, void* workspace);

}  // namespace ssm
