// One token of the selective scan (generation): the state is read and written
// once, which bounds it.  A channel's states lie side by side in memory and take
// the smallest power of two of lanes that covers them, 16 bytes (or 4, where N is
// not a multiple of 4) to a lane; C.s is summed over those lanes.  64 x 2048 channels of
// 16 states: 6.7 to 7.1 us (18 MB; 3.7 at a copy's rate and one memory latency), 7.9 with the
// loads behind one another.
#include "selective_common.h"

namespace mlstm {
namespace selective {
namespace {

template <typename T, int V>
__global__ __launch_bounds__(256) void step_kernel(SelectiveScan a, T* y, float* state_out,
                                                   int lane_shift) {
  const int64_t at = (int64_t(blockIdx.x) * 256 + threadIdx.x) >> lane_shift;
  const int n = (threadIdx.x & ((1 << lane_shift) - 1)) * V;
  const bool on = at < a.batch * a.channels;
  const int64_t row = on ? at : 0;  // lanes beyond take part in the sums
  const int64_t b = row / a.channels, c = row % a.channels, group = c / (a.channels / a.G);
  // every load is issued before the first is waited for
  const bool mine = n < a.N;
  const int64_t at_n = mine ? n : 0;
  const float u_in = rowvec::to_float(static_cast<const T*>(a.u)[b * a.u_row + c]);
  const float dt = rowvec::to_float(static_cast<const T*>(a.dt)[b * a.dt_row + c]);
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.0f, skip = a.D ? a.D[c] : 0.0f;
  const float z = a.gate ? rowvec::to_float(static_cast<const T*>(a.gate)[b * a.gate_row + c])
                         : 0.0f;
  const T* Bp = static_cast<const T*>(a.B) + b * a.B_row + group * a.N + at_n;
  const T* Cp = static_cast<const T*>(a.C) + b * a.C_row + group * a.N + at_n;
  float A[V], s[V] = {}, B[V], C[V];
  rowvec::load(a.A + c * a.N + at_n, A);
  if (a.state) rowvec::load(a.state + row * a.N + at_n, s);
#pragma unroll
  for (int e = 0; e < V; ++e) B[e] = rowvec::to_float(Bp[e]), C[e] = rowvec::to_float(Cp[e]);
  const bool live = rowvec::length_of(a.lengths, b, 1) == 1;
  const float u = live ? u_in : 0.0f, delta = live ? softplus(dt + bias) : 0.0f, v = delta * u;
  float p = 0.0f;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float in = live ? v * B[e] : 0.0f;
    s[e] = __builtin_fmaf(rowvec::exp2_fast(delta * rate_of(A[e])), s[e], in);
    if (live && mine) p = __builtin_fmaf(C[e], s[e], p);
  }
  if (on && mine) rowvec::store(state_out + row * a.N + n, s);
  for (int m = 1; m < (1 << lane_shift); m *= 2) p += __shfl_xor(p, m);
  if (on && n == 0) {
    p = __builtin_fmaf(skip, u, p);
    if (a.gate) p = live ? p * (z * rowvec::sigmoid(z)) : 0.0f;
    rowvec::put(y + row, p);
  }
}

template <typename T>
void launch(const SelectiveScan& a, void* y, float* state_out, hipStream_t stream) {
  const int vec = a.N % 4 == 0 ? 4 : 1;
  int shift = 0;
  while ((int64_t(vec) << shift) < a.N) ++shift;
  const int64_t groups = (((a.batch * a.channels) << shift) + 255) / 256;
  T* out = static_cast<T*>(y);
  if (vec == 4)
    step_kernel<T, 4><<<unsigned(groups), 256, 0, stream>>>(a, out, state_out, shift);
  else
    step_kernel<T, 1><<<unsigned(groups), 256, 0, stream>>>(a, out, state_out, shift);
}

}  // namespace
}  // namespace selective

hipError_t launch_selective_step(const SelectiveScan& a, void* y, float* state_out,
                                 hipStream_t stream) {
  if (a.is_bf16)
    selective::launch<__hip_bfloat16>(a, y, state_out, stream);
  else
    selective::launch<float>(a, y, state_out, stream);
  return hipGetLastError();
}

}  // namespace mlstm
