// Interface between the C-ABI layer (ssm_api.hip) and linear attention's launchers.  Arguments have already been validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssm {

// Linear attention with a decay for each head (ssm_linattn.hip).
struct LinAttnArgs {
  const void* q;           // [b, L, G, Dk] (token form: [b, G, Dk])
  const void* k;           // as q
  const void* v;           // [b, L, H, Dv]
  const void* g;           // [b, L, H], nullable
  const float* A;          // [H], nullable
  const int32_t* lengths;  // [b], nullable
  float scale;
  const float* h0;         // [b, H, Dk, Dv], nullable
  void* y;                 // [b, L, H, Dv]
  float* last;             // [b, H, Dk, Dv], nullable; token form: the state, in place
  // backward
  const void* dy;
  const float* dlast;      // nullable
  void* dq;
  void* dk;
  void* dv;
  void* dg;                // null when g is
  float* dh0;              // nullable
  int64_t b, L, H, G, Dk, Dv;
  int dtype;
  hipStream_t stream;
};
int64_t linattn_max_dim();    // largest Dk and Dv
int64_t linattn_max_heads();  // largest H: a chunk's rows are addressed with 32-bit offsets
// Workspace of the forward or the backward of these sizes (nullable arguments taken as given).
size_t linattn_workspace_bytes(const LinAttnArgs& a, bool backward);
hipError_t launch_linattn_fwd(const LinAttnArgs& a, void* workspace);
hipError_t launch_linattn_bwd(const LinAttnArgs& a, void* workspace);
hipError_t launch_linattn_update(const LinAttnArgs& a);

}  // namespace ssm
