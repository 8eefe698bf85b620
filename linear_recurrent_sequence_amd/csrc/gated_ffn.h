// Launches of the gated feed-forward (gated_ffn.hip), called by the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mlstm {

// a tile's 256 rows of any operand stay within a buffer's 2^30 bytes
constexpr int64_t kFfnMaxRows = int64_t(1) << 20, kFfnMaxWidth = int64_t(1) << 16;

struct GatedFfn {
  const void* x;       // [M][D]
  const void* w_gate;  // [F][D]
  const void* w_up;    // [F][D]
  int64_t M, D, F;
  bool gelu;  // activation g Phi(g), else g sigma(g)
  bool is_bf16;
};

struct GatedFfnGrads {
  const void* dh;  // [M][F]
  void* dx;        // [M][D]
  void* dw_gate;   // [F][D]
  void* dw_up;     // [F][D]
};

// The products of a call: g and u forward, g and u again backward, dx, and the weights'
// gradients; and the tiles that one is taken in (none where rows are few)
enum class FfnProduct { kForward, kAgain, kDx, kWeights };
struct GatedFfnTiles {
  int64_t columns, rows;        // of a tile's outputs
  int64_t whole, split, shares;  // tiles in one piece, and those split into so many shares
};
GatedFfnTiles gated_ffn_tiles(const GatedFfn& a, FfnProduct which);

size_t gated_ffn_fwd_workspace_bytes(const GatedFfn& a);
hipError_t launch_gated_ffn_fwd(const GatedFfn& a, void* h, void* workspace, hipStream_t stream);
size_t gated_ffn_bwd_workspace_bytes(const GatedFfn& a);
hipError_t launch_gated_ffn_bwd(const GatedFfn& a, const GatedFfnGrads& g, void* workspace,
                                hipStream_t stream);

}  // namespace mlstm
