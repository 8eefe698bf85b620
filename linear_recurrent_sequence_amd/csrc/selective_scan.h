// Launches of the selective state space scan (selective_fwd.hip,
// selective_bwd.hip, selective_step.hip), called by the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mlstm {

constexpr int64_t kScanMaxStates = 64;

struct SelectiveScan {
  const void* u;   // [batch][T] rows of `channels`, u_row elements apart
  const void* dt;  // likewise
  const float* A;  // [channels][N]
  const void* B;   // [batch][T] rows of [G][N]
  const void* C;   // likewise
  const float* D;        // [channels] or NULL
  const void* gate;      // rows of `channels`, or NULL
  const float* dt_bias;  // [channels] or NULL
  const float* state;    // [batch][channels][N] or NULL (zeros)
  const int32_t* lengths;  // [batch] or NULL (T)
  int64_t u_row, dt_row, B_row, C_row, gate_row;
  int64_t batch, T, channels, G, N;
  bool is_bf16;
};

struct SelectiveGrads {
  const void* dy;       // [batch][T][channels]
  const float* dstate;  // [batch][channels][N] or NULL (zeros): of the state after
  void *du, *ddt, *dB, *dC, *dgate;       // contiguous; dgate with gate
  float *dA, *dD, *ddt_bias, *dstate_out;  // dD and ddt_bias with theirs; dstate_out may be NULL
};

size_t selective_fwd_workspace_bytes(const SelectiveScan& a);
hipError_t launch_selective_fwd(const SelectiveScan& a, void* y, float* state_out, void* workspace,
                                hipStream_t stream);
size_t selective_bwd_workspace_bytes(const SelectiveScan& a);
hipError_t launch_selective_bwd(const SelectiveScan& a, const SelectiveGrads& g, void* workspace,
                                hipStream_t stream);
// T = 1
hipError_t launch_selective_step(const SelectiveScan& a, void* y, float* state_out,
                                 hipStream_t stream);

}  // namespace mlstm
