// C ABI of the gated delta rule and the block norm (declared in
// include/mlstm.h): argument validation and launches.
#include <math.h>

#include "abi_common.h"
#include "block_norm.h"
#include "delta.h"

namespace {

using mlstm::BlockNorm;
using mlstm::BlockNormGrads;
using mlstm::DeltaShape;
using mlstm::abi::check_alias;
using mlstm::abi::check_aligned;
using mlstm::abi::check_given;
using mlstm::abi::hip_status;

constexpr int64_t kMaxT = int64_t(1) << 30;
constexpr int64_t kMaxElems = int64_t(1) << 46;
// a launch takes fewer than 2^32 threads: a token's workgroups of 256 have at
// least 16 value columns, a sequence has at most 16 of 768 to a head and 4 of 256
// to a head's chunk
constexpr int64_t kMaxTokenTiles = (int64_t(1) << 24) - 1;
constexpr int64_t kMaxDeltaHeads = (int64_t(1) << 18) - 1;
constexpr int64_t kMaxDeltaChunks = (int64_t(1) << 22) - 1;
constexpr int64_t kMaxGrid = (int64_t(1) << 31) - 1;

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }
bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255) == 0; }

int check_common(int64_t B, int64_t NH, int64_t T, int dtype) {
  if (dtype != MLSTM_FP32 && dtype != MLSTM_BF16) return MLSTM_ERR_DTYPE;
  if (B < 1 || NH < 1 || T < 1) return MLSTM_ERR_SHAPE;
  if (T > kMaxT || B > kMaxGrid || NH > kMaxGrid || B * NH > kMaxGrid) return MLSTM_ERR_SHAPE;
  return MLSTM_OK;
}

// one_token: T = 1 forward, the step kernel's
int check_delta(int64_t B, int64_t NHK, int64_t NH, int64_t T, int64_t dk, int64_t dv, int dtype,
                bool one_token) {
  const int st = check_common(B, NH, T, dtype);
  if (st != MLSTM_OK) return st;
  if (NHK < 1 || dk < 1 || dv < 1) return MLSTM_ERR_SHAPE;
  if (NH % NHK != 0) return MLSTM_ERR_HEADS;
  if (dk % 16 != 0 || dk > mlstm::kDeltaMaxKeyDim || dv % 16 != 0 ||
      dv > mlstm::kDeltaMaxValueDim)
    return MLSTM_ERR_HEAD_DIM;
  const int64_t H = B * NH, chunks = (T + mlstm::kDeltaChunk - 1) / mlstm::kDeltaChunk;
  if (one_token ? H > kMaxTokenTiles / (dv / 16)
                : H > kMaxDeltaHeads || H > kMaxDeltaChunks / chunks)
    return MLSTM_ERR_SHAPE;
  return MLSTM_OK;
}

DeltaShape delta_shape(int64_t B, int64_t NHK, int64_t NH, int64_t T, int64_t dk, int64_t dv,
                       int dtype, int forget_activation) {
  return {B, NHK, NH, T, dk, dv, dtype == MLSTM_BF16, forget_activation == MLSTM_FORGET_EXP};
}

struct DeltaBytes {
  size_t qk, vh, gate, C;
};
DeltaBytes delta_bytes(const DeltaShape& s) {
  const size_t e = s.is_bf16 ? 2 : 4, t = size_t(s.B) * size_t(s.T);
  return {t * size_t(s.NHK * s.dk) * e, t * size_t(s.NH * s.dv) * e, t * size_t(s.NH) * 4,
          size_t(s.B * s.NH) * size_t(s.dv * s.dk) * 4};
}

bool known_forget(int a) { return a == MLSTM_FORGET_SIGMOID || a == MLSTM_FORGET_EXP; }

int check_norm(int64_t B, int64_t NH, int64_t T, int64_t d, int dtype, int norm,
               int gate_activation, float eps) {
  const int st = check_common(B, NH, T, dtype);
  if (st != MLSTM_OK) return st;
  if (d < 1) return MLSTM_ERR_SHAPE;
  if (d % 8 != 0 || d > mlstm::kBlockNormMaxRow || NH > mlstm::kBlockNormMaxRow / d)
    return MLSTM_ERR_HEAD_DIM;
  if (B > kMaxElems / T / (NH * d)) return MLSTM_ERR_SHAPE;
  if ((norm != MLSTM_NORM_LAYER && norm != MLSTM_NORM_RMS) ||
      (gate_activation != MLSTM_GATE_SIGMOID && gate_activation != MLSTM_GATE_SILU) ||
      !(eps >= 0.0f) || isinf(eps))
    return MLSTM_ERR_NORM;
  return MLSTM_OK;
}

BlockNorm block_norm(const void* p, const void* gate, const void* residual, const float* weight,
                     const float* scale, const float* next_weight, int64_t B, int64_t NH,
                     int64_t T, int64_t d, int dtype, int norm, int gate_activation, float eps) {
  BlockNorm a;
  a.p = p;
  a.gate = gate;
  a.residual = residual;
  a.weight = weight;
  a.scale = scale;
  a.next_weight = next_weight;
  a.B = B;
  a.NH = NH;
  a.T = T;
  a.d = d;
  a.eps = eps;
  a.layer = norm == MLSTM_NORM_LAYER;
  a.silu = gate_activation == MLSTM_GATE_SILU;
  a.is_bf16 = dtype == MLSTM_BF16;
  return a;
}

}  // namespace

extern "C" {

size_t mlstm_delta_workspace_bytes(int64_t B, int64_t NHK, int64_t NH, int64_t T, int64_t dk,
                                   int64_t dv, int dtype, int backward) {
  if (check_delta(B, NHK, NH, T, dk, dv, dtype, T == 1 && !backward) != MLSTM_OK) return 0;
  const DeltaShape s = delta_shape(B, NHK, NH, T, dk, dv, dtype, MLSTM_FORGET_SIGMOID);
  if (backward) return mlstm::delta_bwd_workspace_bytes(s);
  return T == 1 ? 0 : mlstm::delta_fwd_workspace_bytes(s);
}

int mlstm_delta_fwd(const void* q, const void* k, const void* v, const float* beta,
                    const float* fgate, const float* C_in, void* h, float* C_out, void* workspace,
                    size_t workspace_bytes, int64_t B, int64_t NHK, int64_t NH, int64_t T,
                    int64_t dk, int64_t dv, int dtype, int forget_activation, void* stream) {
  int st = check_delta(B, NHK, NH, T, dk, dv, dtype, T == 1);
  if (st != MLSTM_OK) return st;
  if (!known_forget(forget_activation)) return MLSTM_ERR_ACTIVATION;
  if ((st = check_given({q, k, v, beta, fgate, h, C_out})) != MLSTM_OK) return st;
  if ((st = check_aligned({q, k, v, h, C_in, C_out})) != MLSTM_OK) return st;
  if (!aligned4(beta) || !aligned4(fgate) || !aligned256(workspace)) return MLSTM_ERR_ALIGN;
  const DeltaShape s = delta_shape(B, NHK, NH, T, dk, dv, dtype, forget_activation);
  const size_t need = T == 1 ? 0 : mlstm::delta_fwd_workspace_bytes(s);
  if (need && !workspace) return MLSTM_ERR_NULL;
  if (workspace_bytes < need) return MLSTM_ERR_WORKSPACE;
  const DeltaBytes n = delta_bytes(s);
  // the memory may be updated in place, but not through a shifted window
  const bool in_place = C_in == C_out;
  st = check_alias({{q, n.qk}, {k, n.qk}, {v, n.vh}, {beta, n.gate}, {fgate, n.gate},
                    {in_place ? nullptr : C_in, n.C}},
                   {{h, n.vh}, {C_out, n.C}, {workspace, need}});
  if (st != MLSTM_OK) return st;
  const hipStream_t on = static_cast<hipStream_t>(stream);
  if (T == 1)
    return hip_status(mlstm::launch_delta_step(s, q, k, v, beta, fgate, C_in, C_out, h, on));
  return hip_status(
      mlstm::launch_delta_fwd(s, q, k, v, beta, fgate, C_in, h, C_out, workspace, on));
}

int mlstm_delta_step(const void* q, const void* k, const void* v, const float* beta,
                     const float* fgate, const float* C_in, float* C_out, void* h, int64_t B,
                     int64_t NHK, int64_t NH, int64_t dk, int64_t dv, int dtype,
                     int forget_activation, void* stream) {
  if (!C_in) return MLSTM_ERR_NULL;
  return mlstm_delta_fwd(q, k, v, beta, fgate, C_in, h, C_out, nullptr, 0, B, NHK, NH, 1, dk, dv,
                         dtype, forget_activation, stream);
}

int mlstm_delta_bwd(const void* q, const void* k, const void* v, const float* beta,
                    const float* fgate, const float* C_in, const void* dh, const float* dC_in,
                    void* dq, void* dk, void* dv, float* dbeta, float* dfgate, float* dC_out,
                    void* workspace, size_t workspace_bytes, int64_t B, int64_t NHK, int64_t NH,
                    int64_t T, int64_t dk_dim, int64_t dv_dim, int dtype, int forget_activation,
                    void* stream) {
  int st = check_delta(B, NHK, NH, T, dk_dim, dv_dim, dtype, false);
  if (st != MLSTM_OK) return st;
  if (!known_forget(forget_activation)) return MLSTM_ERR_ACTIVATION;
  st = check_given({q, k, v, beta, fgate, dh, dq, dk, dv, dbeta, dfgate, workspace});
  if (st != MLSTM_OK) return st;
  st = check_aligned({q, k, v, C_in, dh, dC_in, dq, dk, dv, dC_out});
  if (st != MLSTM_OK) return st;
  if (!aligned4(beta) || !aligned4(fgate) || !aligned4(dbeta) || !aligned4(dfgate) ||
      !aligned256(workspace))
    return MLSTM_ERR_ALIGN;
  const DeltaShape s = delta_shape(B, NHK, NH, T, dk_dim, dv_dim, dtype, forget_activation);
  const size_t need = mlstm::delta_bwd_workspace_bytes(s);
  if (workspace_bytes < need) return MLSTM_ERR_WORKSPACE;
  const DeltaBytes n = delta_bytes(s);
  st = check_alias({{q, n.qk}, {k, n.qk}, {v, n.vh}, {beta, n.gate}, {fgate, n.gate},
                    {C_in, n.C}, {dh, n.vh}, {dC_in, n.C}},
                   {{dq, n.qk}, {dk, n.qk}, {dv, n.vh}, {dbeta, n.gate}, {dfgate, n.gate},
                    {dC_out, n.C}, {workspace, need}});
  if (st != MLSTM_OK) return st;
  const mlstm::DeltaGrads g = {dh, dC_in, dq, dk, dv, dbeta, dfgate, dC_out};
  return hip_status(mlstm::launch_delta_bwd(s, q, k, v, beta, fgate, C_in, g, workspace,
                                            static_cast<hipStream_t>(stream)));
}

int mlstm_block_norm_fwd(const void* p, const void* gate, const void* residual,
                         const float* weight, const float* scale, const float* next_weight,
                         void* r_out, void* y_out, int64_t B, int64_t NH, int64_t T, int64_t d,
                         int dtype, int norm, int gate_activation, float eps, void* stream) {
  int st = check_norm(B, NH, T, d, dtype, norm, gate_activation, eps);
  if (st != MLSTM_OK) return st;
  if ((st = check_given({p, weight, r_out})) != MLSTM_OK) return st;
  if ((next_weight == nullptr) != (y_out == nullptr)) return MLSTM_ERR_NULL;
  st = check_aligned({p, gate, residual, weight, scale, next_weight, r_out, y_out});
  if (st != MLSTM_OK) return st;
  const size_t w = size_t(NH * d) * 4, n = size_t(B) * size_t(T) * size_t(NH * d) *
                                           (dtype == MLSTM_BF16 ? 2 : 4);
  st = check_alias({{p, n}, {gate, n}, {residual, n}, {weight, w}, {scale, w}, {next_weight, w}},
                   {{r_out, n}, {y_out, n}});
  if (st != MLSTM_OK) return st;
  return hip_status(mlstm::launch_block_norm_fwd(
      block_norm(p, gate, residual, weight, scale, next_weight, B, NH, T, d, dtype, norm,
                 gate_activation, eps),
      r_out, y_out, static_cast<hipStream_t>(stream)));
}

size_t mlstm_block_norm_workspace_bytes(int64_t B, int64_t NH, int64_t T, int64_t d) {
  if (check_norm(B, NH, T, d, MLSTM_BF16, MLSTM_NORM_LAYER, MLSTM_GATE_SIGMOID, 0.0f) != MLSTM_OK)
    return 0;
  return mlstm::block_norm_partial_bytes(B, NH, T, d);
}

int mlstm_block_norm_bwd(const void* p, const void* gate, const void* residual,
                         const float* weight, const float* scale, const float* next_weight,
                         const void* dr, const void* dy, void* dp, void* dgate, void* dresidual,
                         float* dweight, float* dscale, float* dnext_weight, void* workspace,
                         size_t workspace_bytes, int64_t B, int64_t NH, int64_t T, int64_t d,
                         int dtype, int norm, int gate_activation, float eps, void* stream) {
  int st = check_norm(B, NH, T, d, dtype, norm, gate_activation, eps);
  if (st != MLSTM_OK) return st;
  if ((st = check_given({p, weight, dp, dweight, workspace})) != MLSTM_OK) return st;
  // a gradient for each input that is given, and for no other
  if ((gate == nullptr) != (dgate == nullptr) || (residual == nullptr) != (dresidual == nullptr) ||
      (scale == nullptr) != (dscale == nullptr) ||
      (next_weight == nullptr) != (dnext_weight == nullptr) ||
      (next_weight == nullptr) != (dy == nullptr))
    return MLSTM_ERR_NULL;
  st = check_aligned({p, gate, residual, weight, scale, next_weight, dr, dy, dp, dgate, dresidual,
                      dweight, dscale, dnext_weight});
  if (st != MLSTM_OK) return st;
  if (!aligned256(workspace)) return MLSTM_ERR_ALIGN;
  const size_t need = mlstm::block_norm_partial_bytes(B, NH, T, d);
  if (workspace_bytes < need) return MLSTM_ERR_WORKSPACE;
  const size_t w = size_t(NH * d) * 4, n = size_t(B) * size_t(T) * size_t(NH * d) *
                                           (dtype == MLSTM_BF16 ? 2 : 4);
  st = check_alias({{p, n}, {gate, n}, {residual, n}, {weight, w}, {scale, w}, {next_weight, w},
                    {dr, n}, {dy, n}},
                   {{dp, n}, {dgate, n}, {dresidual, n}, {dweight, w}, {dscale, w},
                    {dnext_weight, w}, {workspace, need}});
  if (st != MLSTM_OK) return st;
  const BlockNormGrads g = {dr, dy, dp, dgate, dresidual, dweight, dscale, dnext_weight};
  return hip_status(mlstm::launch_block_norm_bwd(
      block_norm(p, gate, residual, weight, scale, next_weight, B, NH, T, d, dtype, norm,
                 gate_activation, eps),
      g, static_cast<float*>(workspace), static_cast<hipStream_t>(stream)));
}

}  // extern "C"
