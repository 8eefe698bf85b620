// Launches of the short causal convolution (short_conv.hip), called by the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mlstm {

constexpr int kConvMinWidth = 2, kConvMaxWidth = 8;

struct ShortConv {
  const void* x;           // [B][T] rows of C = NH d channels, x_row elements apart
  const float* weight;     // [C][W]
  const float* bias;       // [C] or NULL
  const void* state;       // [B][W - 1][C] or NULL (zeros)
  const int32_t* lengths;  // [B] or NULL (T)
  int64_t x_row, B, NH, T, d;
  int W;
  bool silu;
  bool is_bf16;
};

struct ShortConvGrads {
  const void* dy;      // [B][NH][T][d]
  const void* dstate;  // [B][W - 1][C] or NULL (zeros): of the state after
  void* dx;            // [B][T][C]
  float* dweight;      // [C][W]
  float* dbias;        // [C], with bias
  void* dstate_out;    // [B][W - 1][C] or NULL: of the state before
};

hipError_t launch_short_conv_fwd(const ShortConv& a, void* y, void* state_out, hipStream_t stream);
size_t short_conv_bwd_workspace_bytes(int64_t B, int64_t C, int64_t T, int W);
hipError_t launch_short_conv_bwd(const ShortConv& a, const ShortConvGrads& g, void* workspace,
                                 hipStream_t stream);

}  // namespace mlstm
