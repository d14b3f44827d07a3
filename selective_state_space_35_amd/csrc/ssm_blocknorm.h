// Interface between the C-ABI layer (ssm_api.hip) and the launchers of the norms around a block.  Arguments have already been
// validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssm {

// RMS norm after a block, gate, scale, residual, RMS norm before the next block (ssm_blocknorm.hip).
struct BlockNormArgs {
  const void* x;             // [rows, H, W]
  const float* post_weight;  // [H, W], nullable
  const void* z;             // [rows, H, W], nullable
  const float* scale;        // [H, W], nullable
  const void* residual;      // [rows, H, W] of the residual's type, nullable
  const float* pre_weight;   // [H, W], nullable
  float eps;
  bool post, pre;            // which norms there are
  void* h;                   // of the residual's type; nullable with pre
  void* n;                   // with pre
  float* rstd_post;          // [rows, H]: written by the forward (nullable), read by the backward
  float* rstd_pre;
  // backward
  const void* dh;            // of the residual's type; nullable with pre
  const void* dn;            // with pre
  void* dx;
  void* dz;                  // with z
  void* dresidual;           // of the residual's type, nullable
  float* dpost_weight;       // [H, W] each, nullable
  float* dscale;
  float* dpre_weight;
  int64_t rows, H, W;
  int dtype, rdtype;
  hipStream_t stream;
};
int64_t blocknorm_max_width();
size_t blocknorm_workspace_bytes(const BlockNormArgs& a);  // of the backward, for all gradients
hipError_t launch_blocknorm_fwd(const BlockNormArgs& a);
hipError_t launch_blocknorm_bwd(const BlockNormArgs& a, void* workspace);

}  // namespace ssm
