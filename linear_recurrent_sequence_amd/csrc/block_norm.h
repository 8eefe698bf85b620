// Launches of the block norm (block_norm.hip), called by the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mlstm {

constexpr int64_t kBlockNormMaxRow = 8192;  // NH * d

struct BlockNorm {
  const void* p;             // [B][NH][T][d]
  const void* gate;          // [B][NH][T][d] or NULL
  const void* residual;      // [B][T][NH * d] or NULL
  const float* weight;       // [NH * d]
  const float* scale;        // [NH * d] or NULL
  const float* next_weight;  // [NH * d] or NULL
  int64_t B, NH, T, d;
  float eps;
  bool layer;    // centred (layer) norm, else root mean square
  bool silu;     // gate activation g sigma(g), else sigma(g)
  bool is_bf16;
};

struct BlockNormGrads {
  const void* dr;     // [B][T][NH * d] or NULL
  const void* dy;     // [B][T][NH * d], given with next_weight
  void* dp;           // [B][NH][T][d]
  void* dgate;        // with gate
  void* dresidual;    // with residual
  float* dweight;     // [NH * d]
  float* dscale;      // with scale
  float* dnext_weight;  // with next_weight
};

hipError_t launch_block_norm_fwd(const BlockNorm& a, void* r_out, void* y_out, hipStream_t stream);
// `partials`: block_norm_partial_bytes(...) bytes, 256-byte aligned
size_t block_norm_partial_bytes(int64_t B, int64_t NH, int64_t T, int64_t d);
hipError_t launch_block_norm_bwd(const BlockNorm& a, const BlockNormGrads& g, float* partials,
                                 hipStream_t stream);

}  // namespace mlstm
