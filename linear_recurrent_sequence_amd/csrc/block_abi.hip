// C ABI of the short convolution, the selective scan and the gated feed-forward
// (declared in include/mlstm.h): argument validation and launches.
#include "abi_common.h"
#include "gated_ffn.h"
#include "selective_scan.h"
#include "short_conv.h"

namespace {

using mlstm::GatedFfn;
using mlstm::SelectiveScan;
using mlstm::ShortConv;
using mlstm::abi::check_alias;
using mlstm::abi::check_aligned;
using mlstm::abi::check_given;
using mlstm::abi::hip_status;

// a launch takes fewer than 2^32 threads
constexpr int64_t kMaxChannels = int64_t(1) << 20;
constexpr int64_t kMaxTokens = int64_t(1) << 36;
constexpr int64_t kMaxElements = int64_t(1) << 58;  // byte offsets stay within 62 bits
// 32 rows of a scan's sequence stay within a buffer's 2^30 bytes
constexpr int64_t kMaxScanPitch = int64_t(1) << 23;
constexpr int64_t kMaxWorkgroups = (int64_t(1) << 24) - 1;

bool aligned_to(const void* p, uintptr_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

size_t size_of(int dtype) { return dtype == MLSTM_BF16 ? 2 : 4; }

// bytes from the first to the last element of `rows` rows of `width`, `pitch` apart
size_t rows_bytes(int64_t rows, int64_t width, int64_t pitch, int dtype) {
  return (size_t(rows - 1) * size_t(pitch) + size_t(width)) * size_of(dtype);
}

int check_tokens(int64_t B, int64_t T, int dtype) {
  if (dtype != MLSTM_FP32 && dtype != MLSTM_BF16) return MLSTM_ERR_DTYPE;
  if (B < 1 || T < 1 || B > kMaxTokens || T > kMaxTokens / B) return MLSTM_ERR_SHAPE;
  return MLSTM_OK;
}

// rows that vectors of 16 bytes are read from
int check_pitch(int64_t pitch, int64_t width, int64_t most) {
  return pitch < width || pitch % 8 != 0 || pitch > most ? MLSTM_ERR_ROW : MLSTM_OK;
}

// ---- short convolution

int check_conv(int64_t B, int64_t NH, int64_t T, int64_t d, int64_t width, int dtype) {
  const int st = check_tokens(B, T, dtype);
  if (st != MLSTM_OK) return st;
  if (NH < 1 || d < 1) return MLSTM_ERR_SHAPE;
  if (d % 8 != 0 || d > kMaxChannels || NH > kMaxChannels / d) return MLSTM_ERR_HEAD_DIM;
  if (width < mlstm::kConvMinWidth || width > mlstm::kConvMaxWidth) return MLSTM_ERR_WIDTH;
  // a workgroup has 128 channels and 64 tokens at least
  if (B > kMaxWorkgroups / ((T + 63) / 64) / ((NH * d + 127) / 128)) return MLSTM_ERR_SHAPE;
  return MLSTM_OK;
}

bool known_conv_activation(int a) { return a == MLSTM_CONV_NONE || a == MLSTM_CONV_SILU; }

struct ConvBytes {
  size_t x, rows, state, weight, bias, lengths;
};
ConvBytes conv_bytes(const ShortConv& a, int dtype) {
  const int64_t C = a.NH * a.d;
  return {rows_bytes(a.B * a.T, C, a.x_row, dtype), rows_bytes(a.B * a.T, C, C, dtype),
          size_t(a.B * (a.W - 1)) * size_t(C) * size_of(dtype), size_t(C * a.W) * 4,
          size_t(C) * 4, size_t(a.B) * 4};
}

// ---- selective scan

int check_scan(int64_t batch, int64_t T, int64_t channels, int64_t G, int64_t N, int dtype) {
  const int st = check_tokens(batch, T, dtype);
  if (st != MLSTM_OK) return st;
  if (channels < 1 || G < 1 || N < 1) return MLSTM_ERR_SHAPE;
  if (channels % G != 0) return MLSTM_ERR_HEADS;
  if (channels / G % 8 != 0 || channels > kMaxChannels) return MLSTM_ERR_HEAD_DIM;
  if (N > mlstm::kScanMaxStates) return MLSTM_ERR_WIDTH;
  const int64_t most = int64_t(1) << 31;
  if (batch > (int64_t(1) << 25) / channels || T > most / batch / (G * N) ||
      batch > (int64_t(1) << 22) / (G * ((channels / G + 63) / 64)))
    return MLSTM_ERR_SHAPE;
  return MLSTM_OK;
}

// (the kernel of one token takes rows that are any distance apart)
int check_scan_pitches(const SelectiveScan& a, bool one_token) {
  const int64_t most = one_token ? kMaxElements / a.batch : kMaxScanPitch;
  int st = check_pitch(a.u_row, a.channels, most);
  if (st == MLSTM_OK) st = check_pitch(a.dt_row, a.channels, most);
  if (st == MLSTM_OK && a.gate) st = check_pitch(a.gate_row, a.channels, most);
  if (st == MLSTM_OK &&
      (a.B_row < a.G * a.N || a.C_row < a.G * a.N || a.B_row > most || a.C_row > most))
    st = MLSTM_ERR_ROW;
  return st;
}

struct ScanBytes {
  size_t u, dt, gate, B, C, rows, shared, A, channel, state, lengths;
};
ScanBytes scan_bytes(const SelectiveScan& a, int dtype) {
  const int64_t n = a.batch * a.T;
  return {rows_bytes(n, a.channels, a.u_row, dtype),
          rows_bytes(n, a.channels, a.dt_row, dtype),
          a.gate ? rows_bytes(n, a.channels, a.gate_row, dtype) : 0,
          rows_bytes(n, a.G * a.N, a.B_row, dtype),
          rows_bytes(n, a.G * a.N, a.C_row, dtype),
          rows_bytes(n, a.channels, a.channels, dtype),
          rows_bytes(n, a.G * a.N, a.G * a.N, dtype),
          size_t(a.channels * a.N) * 4,
          size_t(a.channels) * 4,
          size_t(a.batch) * size_t(a.channels * a.N) * 4,
          size_t(a.batch) * 4};
}

// what is read, but for the state
int check_scan_inputs(const SelectiveScan& a, bool one_token) {
  int st = check_given({a.u, a.dt, a.A, a.B, a.C});
  if (st != MLSTM_OK) return st;
  if ((st = check_scan_pitches(a, one_token)) != MLSTM_OK) return st;
  st = check_aligned({a.u, a.dt, a.gate, a.A, a.D, a.dt_bias, a.state});
  if (st != MLSTM_OK) return st;
  const uintptr_t e = a.is_bf16 ? 2 : 4;
  if (!aligned_to(a.B, e) || !aligned_to(a.C, e) || !aligned_to(a.lengths, 4))
    return MLSTM_ERR_ALIGN;
  return MLSTM_OK;
}

// ---- gated feed-forward

int check_ffn(int64_t M, int64_t D, int64_t F, int dtype) {
  if (dtype != MLSTM_FP32 && dtype != MLSTM_BF16) return MLSTM_ERR_DTYPE;
  if (M < 1 || D < 1 || F < 1 || M > mlstm::kFfnMaxRows) return MLSTM_ERR_SHAPE;
  if (D % 8 != 0 || F % 8 != 0 || D > mlstm::kFfnMaxWidth || F > mlstm::kFfnMaxWidth)
    return MLSTM_ERR_HEAD_DIM;
  if (M > (int64_t(1) << 33) / (D > 2 * F ? D : 2 * F)) return MLSTM_ERR_SHAPE;
  return MLSTM_OK;
}

bool known_ffn_activation(int a) { return a == MLSTM_FFN_SILU || a == MLSTM_FFN_GELU; }

GatedFfn gated_ffn(const void* x, const void* w_gate, const void* w_up, int64_t M, int64_t D,
                   int64_t F, int dtype, int activation) {
  return {x, w_gate, w_up, M, D, F, activation == MLSTM_FFN_GELU, dtype == MLSTM_BF16};
}

}  // namespace

extern "C" {

int mlstm_short_conv_fwd(const void* x, int64_t x_row, const float* weight, const float* bias,
                         const void* state_in, const int32_t* lengths, void* y, void* state_out,
                         int64_t B, int64_t NH, int64_t T, int64_t d, int64_t width, int dtype,
                         int activation, void* stream) {
  int st = check_conv(B, NH, T, d, width, dtype);
  if (st != MLSTM_OK) return st;
  if (!known_conv_activation(activation)) return MLSTM_ERR_ACTIVATION;
  if ((st = check_given({x, weight, y, state_out})) != MLSTM_OK) return st;
  if ((st = check_pitch(x_row, NH * d, kMaxElements / (B * T))) != MLSTM_OK) return st;
  st = check_aligned({x, weight, bias, state_in, y, state_out});
  if (st != MLSTM_OK) return st;
  if (!aligned_to(lengths, 4)) return MLSTM_ERR_ALIGN;
  const ShortConv a = {x, weight, bias, state_in, lengths, x_row, B, NH, T, d, int(width),
                       activation == MLSTM_CONV_SILU, dtype == MLSTM_BF16};
  const ConvBytes n = conv_bytes(a, dtype);
  // the state may be updated in place, but not through a shifted window
  st = check_alias({{x, n.x}, {weight, n.weight}, {bias, n.bias},
                    {state_in == state_out ? nullptr : state_in, n.state}, {lengths, n.lengths}},
                   {{y, n.rows}, {state_out, n.state}});
  if (st != MLSTM_OK) return st;
  return hip_status(
      mlstm::launch_short_conv_fwd(a, y, state_out, static_cast<hipStream_t>(stream)));
}

size_t mlstm_short_conv_workspace_bytes(int64_t B, int64_t NH, int64_t T, int64_t d,
                                        int64_t width, int dtype) {
  if (check_conv(B, NH, T, d, width, dtype) != MLSTM_OK) return 0;
  return mlstm::short_conv_bwd_workspace_bytes(B, NH * d, T, int(width));
}

int mlstm_short_conv_bwd(const void* x, int64_t x_row, const float* weight, const float* bias,
                         const void* state_in, const int32_t* lengths, const void* dy,
                         const void* dstate, void* dx, float* dweight, float* dbias,
                         void* dstate_out, void* workspace, size_t workspace_bytes, int64_t B,
                         int64_t NH, int64_t T, int64_t d, int64_t width, int dtype,
                         int activation, void* stream) {
  int st = check_conv(B, NH, T, d, width, dtype);
  if (st != MLSTM_OK) return st;
  if (!known_conv_activation(activation)) return MLSTM_ERR_ACTIVATION;
  if ((st = check_given({x, weight, dy, dx, dweight, workspace})) != MLSTM_OK) return st;
  if ((bias == nullptr) != (dbias == nullptr)) return MLSTM_ERR_NULL;
  if ((st = check_pitch(x_row, NH * d, kMaxElements / (B * T))) != MLSTM_OK) return st;
  st = check_aligned({x, weight, bias, state_in, dy, dstate, dx, dweight, dbias, dstate_out});
  if (st != MLSTM_OK) return st;
  if (!aligned_to(lengths, 4) || !aligned_to(workspace, 256)) return MLSTM_ERR_ALIGN;
  const ShortConv a = {x, weight, bias, state_in, lengths, x_row, B, NH, T, d, int(width),
                       activation == MLSTM_CONV_SILU, dtype == MLSTM_BF16};
  const size_t need = mlstm::short_conv_bwd_workspace_bytes(B, NH * d, T, a.W);
  if (workspace_bytes < need) return MLSTM_ERR_WORKSPACE;
  const ConvBytes n = conv_bytes(a, dtype);
  st = check_alias({{x, n.x}, {weight, n.weight}, {bias, n.bias}, {state_in, n.state},
                    {lengths, n.lengths}, {dy, n.rows}, {dstate, n.state}},
                   {{dx, n.rows}, {dweight, n.weight}, {dbias, n.bias}, {dstate_out, n.state},
                    {workspace, need}});
  if (st != MLSTM_OK) return st;
  return hip_status(mlstm::launch_short_conv_bwd(a, {dy, dstate, dx, dweight, dbias, dstate_out},
                                                 workspace, static_cast<hipStream_t>(stream)));
}

size_t mlstm_scan_workspace_bytes(int64_t batch, int64_t T, int64_t channels, int64_t G, int64_t N,
                                  int dtype, int backward) {
  if (check_scan(batch, T, channels, G, N, dtype) != MLSTM_OK) return 0;
  SelectiveScan a = {};
  a.batch = batch;
  a.T = T;
  a.channels = channels;
  a.G = G;
  a.N = N;
  a.is_bf16 = dtype == MLSTM_BF16;
  if (backward) return mlstm::selective_bwd_workspace_bytes(a);
  return T == 1 ? 0 : mlstm::selective_fwd_workspace_bytes(a);
}

int mlstm_scan_fwd(const void* u, int64_t u_row, const void* dt, int64_t dt_row, const float* A,
                   const void* B, int64_t B_row, const void* C, int64_t C_row, const float* D,
                   const void* gate, int64_t gate_row, const float* dt_bias,
                   const float* state_in, const int32_t* lengths, void* y, float* state_out,
                   void* workspace, size_t workspace_bytes, int64_t batch, int64_t T,
                   int64_t channels, int64_t G, int64_t N, int dtype, void* stream) {
  int st = check_scan(batch, T, channels, G, N, dtype);
  if (st != MLSTM_OK) return st;
  const SelectiveScan a = {u, dt, A, B, C, D, gate, dt_bias, state_in, lengths, u_row, dt_row,
                           B_row, C_row, gate_row, batch, T, channels, G, N, dtype == MLSTM_BF16};
  if ((st = check_scan_inputs(a, T == 1)) != MLSTM_OK) return st;
  if ((st = check_given({y, state_out})) != MLSTM_OK) return st;
  if ((st = check_aligned({y, state_out})) != MLSTM_OK) return st;
  if (!aligned_to(workspace, 256)) return MLSTM_ERR_ALIGN;
  const size_t need = T == 1 ? 0 : mlstm::selective_fwd_workspace_bytes(a);
  if (need && !workspace) return MLSTM_ERR_NULL;
  if (workspace_bytes < need) return MLSTM_ERR_WORKSPACE;
  const ScanBytes n = scan_bytes(a, dtype);
  st = check_alias({{u, n.u}, {dt, n.dt}, {A, n.A}, {B, n.B}, {C, n.C}, {D, n.channel},
                    {gate, n.gate}, {dt_bias, n.channel},
                    {state_in == state_out ? nullptr : state_in, n.state}, {lengths, n.lengths}},
                   {{y, n.rows}, {state_out, n.state}, {workspace, need}});
  if (st != MLSTM_OK) return st;
  const hipStream_t on = static_cast<hipStream_t>(stream);
  if (T == 1) return hip_status(mlstm::launch_selective_step(a, y, state_out, on));
  return hip_status(mlstm::launch_selective_fwd(a, y, state_out, workspace, on));
}

int mlstm_scan_bwd(const void* u, int64_t u_row, const void* dt, int64_t dt_row, const float* A,
                   const void* B, int64_t B_row, const void* C, int64_t C_row, const float* D,
                   const void* gate, int64_t gate_row, const float* dt_bias,
                   const float* state_in, const int32_t* lengths, const void* dy,
                   const float* dstate, void* du, void* ddt, float* dA, void* dB, void* dC,
                   float* dD, void* dgate, float* ddt_bias, float* dstate_out, void* workspace,
                   size_t workspace_bytes, int64_t batch, int64_t T, int64_t channels, int64_t G,
                   int64_t N, int dtype, void* stream) {
  int st = check_scan(batch, T, channels, G, N, dtype);
  if (st != MLSTM_OK) return st;
  const SelectiveScan a = {u, dt, A, B, C, D, gate, dt_bias, state_in, lengths, u_row, dt_row,
                           B_row, C_row, gate_row, batch, T, channels, G, N, dtype == MLSTM_BF16};
  if ((st = check_scan_inputs(a, false)) != MLSTM_OK) return st;
  if ((st = check_given({dy, du, ddt, dA, dB, dC, workspace})) != MLSTM_OK) return st;
  if ((D == nullptr) != (dD == nullptr) || (gate == nullptr) != (dgate == nullptr) ||
      (dt_bias == nullptr) != (ddt_bias == nullptr))
    return MLSTM_ERR_NULL;
  st = check_aligned({dy, dstate, du, ddt, dA, dB, dC, dD, dgate, ddt_bias, dstate_out});
  if (st != MLSTM_OK) return st;
  if (!aligned_to(workspace, 256)) return MLSTM_ERR_ALIGN;
  const size_t need = mlstm::selective_bwd_workspace_bytes(a);
  if (workspace_bytes < need) return MLSTM_ERR_WORKSPACE;
  const ScanBytes n = scan_bytes(a, dtype);
  st = check_alias({{u, n.u}, {dt, n.dt}, {A, n.A}, {B, n.B}, {C, n.C}, {D, n.channel},
                    {gate, n.gate}, {dt_bias, n.channel}, {state_in, n.state},
                    {lengths, n.lengths}, {dy, n.rows}, {dstate, n.state}},
                   {{du, n.rows}, {ddt, n.rows}, {dA, n.A}, {dB, n.shared}, {dC, n.shared},
                    {dD, n.channel}, {dgate, n.rows}, {ddt_bias, n.channel},
                    {dstate_out, n.state}, {workspace, need}});
  if (st != MLSTM_OK) return st;
  const mlstm::SelectiveGrads g = {dy, dstate, du, ddt, dB, dC, dgate, dA, dD, ddt_bias,
                                   dstate_out};
  return hip_status(
      mlstm::launch_selective_bwd(a, g, workspace, static_cast<hipStream_t>(stream)));
}

size_t mlstm_gated_ffn_workspace_bytes(int64_t M, int64_t D, int64_t F, int dtype, int backward) {
  if (check_ffn(M, D, F, dtype) != MLSTM_OK) return 0;
  const GatedFfn a = gated_ffn(nullptr, nullptr, nullptr, M, D, F, dtype, MLSTM_FFN_SILU);
  return backward ? mlstm::gated_ffn_bwd_workspace_bytes(a)
                  : mlstm::gated_ffn_fwd_workspace_bytes(a);
}

int mlstm_gated_ffn_tiles(int64_t M, int64_t D, int64_t F, int dtype, int product,
                          int64_t tiles[5]) {
  const int st = check_ffn(M, D, F, dtype);
  if (st != MLSTM_OK) return st;
  if (product < MLSTM_FFN_FORWARD || product > MLSTM_FFN_WEIGHTS) return MLSTM_ERR_SHAPE;
  if (!tiles) return MLSTM_ERR_NULL;
  const mlstm::GatedFfnTiles t =
      mlstm::gated_ffn_tiles(gated_ffn(nullptr, nullptr, nullptr, M, D, F, dtype, MLSTM_FFN_SILU),
                             static_cast<mlstm::FfnProduct>(product));
  const int64_t all[5] = {t.columns, t.rows, t.whole, t.split, t.shares};
  for (int i = 0; i < 5; ++i) tiles[i] = all[i];
  return MLSTM_OK;
}

int mlstm_gated_ffn_fwd(const void* x, const void* w_gate, const void* w_up, void* h,
                        void* workspace, size_t workspace_bytes, int64_t M, int64_t D, int64_t F,
                        int dtype, int activation, void* stream) {
  int st = check_ffn(M, D, F, dtype);
  if (st != MLSTM_OK) return st;
  if (!known_ffn_activation(activation)) return MLSTM_ERR_ACTIVATION;
  if ((st = check_given({x, w_gate, w_up, h})) != MLSTM_OK) return st;
  if ((st = check_aligned({x, w_gate, w_up, h})) != MLSTM_OK) return st;
  if (!aligned_to(workspace, 256)) return MLSTM_ERR_ALIGN;
  const GatedFfn a = gated_ffn(x, w_gate, w_up, M, D, F, dtype, activation);
  const size_t need = mlstm::gated_ffn_fwd_workspace_bytes(a), e = size_of(dtype);
  if (need && !workspace) return MLSTM_ERR_NULL;
  if (workspace_bytes < need) return MLSTM_ERR_WORKSPACE;
  st = check_alias({{x, size_t(M * D) * e}, {w_gate, size_t(F * D) * e}, {w_up, size_t(F * D) * e}},
                   {{h, size_t(M * F) * e}, {workspace, need}});
  if (st != MLSTM_OK) return st;
  return hip_status(
      mlstm::launch_gated_ffn_fwd(a, h, workspace, static_cast<hipStream_t>(stream)));
}

int mlstm_gated_ffn_bwd(const void* x, const void* w_gate, const void* w_up, const void* dh,
                        void* dx, void* dw_gate, void* dw_up, void* workspace,
                        size_t workspace_bytes, int64_t M, int64_t D, int64_t F, int dtype,
                        int activation, void* stream) {
  int st = check_ffn(M, D, F, dtype);
  if (st != MLSTM_OK) return st;
  if (!known_ffn_activation(activation)) return MLSTM_ERR_ACTIVATION;
  st = check_given({x, w_gate, w_up, dh, dx, dw_gate, dw_up, workspace});
  if (st != MLSTM_OK) return st;
  if ((st = check_aligned({x, w_gate, w_up, dh, dx, dw_gate, dw_up})) != MLSTM_OK) return st;
  if (!aligned_to(workspace, 256)) return MLSTM_ERR_ALIGN;
  const GatedFfn a = gated_ffn(x, w_gate, w_up, M, D, F, dtype, activation);
  const size_t need = mlstm::gated_ffn_bwd_workspace_bytes(a), e = size_of(dtype);
  if (workspace_bytes < need) return MLSTM_ERR_WORKSPACE;
  const size_t rows = size_t(M * D) * e, wide = size_t(M * F) * e, w = size_t(F * D) * e;
  st = check_alias({{x, rows}, {w_gate, w}, {w_up, w}, {dh, wide}},
                   {{dx, rows}, {dw_gate, w}, {dw_up, w}, {workspace, need}});
  if (st != MLSTM_OK) return st;
  return hip_status(mlstm::launch_gated_ffn_bwd(a, {dh, dx, dw_gate, dw_up}, workspace,
                                                static_cast<hipStream_t>(stream)));
}

}  // extern "C"
