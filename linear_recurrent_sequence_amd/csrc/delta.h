// Launches of the gated delta rule (delta_*.hip), called by the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mlstm {

constexpr int64_t kDeltaMaxKeyDim = 512;
constexpr int64_t kDeltaMaxValueDim = 1024;
constexpr int kDeltaChunk = 64;

struct DeltaShape {
  int64_t B, NHK, NH, T, dk, dv;
  bool is_bf16;
  bool exp_forget;
};

// One token (T is 1): C_out and h.  C_in may be NULL (zeros) or C_out.
hipError_t launch_delta_step(const DeltaShape& s, const void* q, const void* k, const void* v,
                             const float* beta, const float* fgate, const float* C_in,
                             float* C_out, void* h, hipStream_t stream);

// A whole sequence in chunks; C_in may be NULL (zeros) or C_out.  `workspace`:
// delta_fwd_workspace_bytes(s), 256-byte aligned.
size_t delta_fwd_workspace_bytes(const DeltaShape& s);
hipError_t launch_delta_fwd(const DeltaShape& s, const void* q, const void* k, const void* v,
                            const float* beta, const float* fgate, const float* C_in, void* h,
                            float* C_out, void* workspace, hipStream_t stream);

struct DeltaGrads {
  const void* dh;      // [B][NH][T][dv]
  const float* dC_in;  // gradient of the memory after the sequence, or NULL (zeros)
  void *dq, *dk, *dv;
  float *dbeta, *dfgate;
  float* dC_out;       // gradient of the memory before it, or NULL
};
size_t delta_bwd_workspace_bytes(const DeltaShape& s);
hipError_t launch_delta_bwd(const DeltaShape& s, const void* q, const void* k, const void* v,
                            const float* beta, const float* fgate, const float* C_in,
                            const DeltaGrads& d, void* workspace, hipStream_t stream);

}  // namespace mlstm
