// Short causal convolution with an activation: what the inputs of a recurrent
// cell pass through, channel by channel, over the last W of them.
//
//   z   = the state's W - 1 inputs, then x_0 .. x_{n-1}
//   a_t = b + sum_j w_j z_{t+j}        y_t = a_t sigma(a_t) (or a_t)
//
// Backward, from dy and the gradient of the state after the sequence:
//
//   g_t  = dy_t act'(a_t)              dw_j = sum_t g_t z_{t+j},  db = sum_t g_t
//   dz_i = sum_j w_j g_{i-j}  (+ the state's gradient for i >= n)
//
// x, dx and the states are rows of all channels, as a projection writes them; y
// and dy are head-major, as the cells read them.
//
// A lane holds V neighbouring channels and walks a run of tokens with
// the last W inputs in registers, so an input is read once but for the W - 1 at
// the start of a run.  The backward forms a_t again and keeps the last W of g as
// well; its weights' sums stay in registers over the run, are joined over the
// runs of a workgroup through LDS and over workgroups by a second kernel, in a
// fixed order: no atomics, results are bitwise reproducible.
//
// Bound by memory.  Measured, bf16, W = 4, 8 x 2048 rows of 1536: forward 19.6 us (100 MB,
// a copy's rate), backward 35 us (150 MB, 86 % of it) and 4 us for the weights' sums.
#include "short_conv.h"

#include "row_vec.h"

namespace mlstm {
namespace {

using rowvec::length_of;

constexpr int kLanes = 32;  // neighbouring vectors of a workgroup
constexpr int kRuns = 8;    // runs of tokens of a workgroup

struct Place {
  int64_t b, c, t0, t1;
  bool on;
};

// workgroup -> (sequence, channels, kRuns runs of `run` tokens); channels fastest
template <int V>
__device__ inline Place place(int64_t B, int64_t C, int64_t T, int run) {
  const int64_t cols = (C / V + kLanes - 1) / kLanes;
  const int64_t span = int64_t(run) * kRuns, spans = (T + span - 1) / span;
  int64_t wg = blockIdx.x;
  Place p;
  const int64_t col = wg % cols;
  wg /= cols;
  p.b = wg / spans;
  p.c = (col * kLanes + threadIdx.x % kLanes) * V;
  p.t0 = (wg % spans) * span + (threadIdx.x / kLanes) * run;
  p.t1 = p.t0 + run < T ? p.t0 + run : T;
  p.on = p.c < C && p.t0 < T;
  return p;
}

template <int V, int W>
__device__ inline void load_weights(const float* weight, const float* bias, int64_t c,
                                    float (&w)[W][V], float (&b)[V]) {
  float raw[V * W];
  const float4* p = reinterpret_cast<const float4*>(weight + c * W);
#pragma unroll
  for (int i = 0; i < V * W / 4; ++i) {
    const float4 f = p[i];
    raw[4 * i] = f.x, raw[4 * i + 1] = f.y, raw[4 * i + 2] = f.z, raw[4 * i + 3] = f.w;
  }
#pragma unroll
  for (int j = 0; j < W; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) w[j][e] = raw[e * W + j];
#pragma unroll
  for (int e = 0; e < V; ++e) b[e] = 0.0f;
  if (bias) rowvec::load(bias + c, b);
}

template <typename T, int V, int W>
__global__ __launch_bounds__(kLanes* kRuns) void conv_fwd_kernel(ShortConv a, T* y, T* state_out,
                                                                 int run) {
  using rowvec::Raw;
  const int64_t C = a.NH * a.d;
  const Place p = place<V>(a.B, C, a.T, run);
  if (!p.on) return;
  const int64_t n = length_of(a.lengths, p.b, a.T);
  const T* x = static_cast<const T*>(a.x) + p.b * a.T * a.x_row + p.c;
  const int64_t head = p.c / a.d;
  T* out = y + (p.b * a.NH + head) * a.T * a.d + p.c % a.d;
  float w[W][V], bias[V];
  load_weights<V, W>(a.weight, a.bias, p.c, w, bias);

  // the last W inputs; z[W - 1] is the current one
  float z[W][V] = {};
  if (p.t0 > 0) {  // a run is longer than W - 1 tokens
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      rowvec::load(x + (p.t0 - (W - 1) + j) * a.x_row, z[j]);
  } else if (a.state) {
    const T* s = static_cast<const T*>(a.state) + p.b * (W - 1) * C + p.c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) rowvec::load(s + j * C, z[j]);
  }
  if (p.t0 == 0) {
    // the state after: rows n .. n + W - 2 of (state, x).  This thread alone reads
    // the state of its channels, and has done so: it may be overwritten.
    T* s = state_out + p.b * (W - 1) * C + p.c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int64_t i = n + j;
      float v[V];
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = 0.0f;
#pragma unroll
      for (int m = 0; m < W - 1; ++m)
        if (i == m)
#pragma unroll
          for (int e = 0; e < V; ++e) v[e] = z[m][e];
      if (i >= W - 1) rowvec::load(x + (i - (W - 1)) * a.x_row, v);
      rowvec::store(s + j * C, v);
    }
  }
  auto step = [&](int64_t t, const Raw<T, V>& raw) {
    rowvec::floats(raw, z[W - 1]);
    float o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float s = bias[e];
#pragma unroll
      for (int j = 0; j < W; ++j) s = __builtin_fmaf(w[j][e], z[j][e], s);
      o[e] = a.silu ? s * rowvec::sigmoid(s) : s;
    }
    rowvec::store(out + t * a.d, o);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) z[j][e] = z[j + 1][e];
  };
  const int64_t end = p.t1 < n ? p.t1 : n;
  constexpr int kAhead = 8;  // inputs in flight
  int64_t t = p.t0;
  for (; t + kAhead <= end; t += kAhead) {
    Raw<T, V> r[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) r[i] = rowvec::load_raw<T, V>(x + (t + i) * a.x_row);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) step(t + i, r[i]);
  }
  for (; t < end; ++t) step(t, rowvec::load_raw<T, V>(x + t * a.x_row));
  const float none[V] = {};
  for (t = t < p.t0 ? p.t0 : t; t < p.t1; ++t) rowvec::store(out + t * a.d, none);
}

// Partial sums of a workgroup: [W + 1][C] floats (w_0 .. w_{W-1}, b)
template <typename T, int V, int W>
__global__ __launch_bounds__(kLanes* kRuns) void conv_bwd_kernel(ShortConv a, ShortConvGrads g,
                                                                 float* partials, int run) {
  using rowvec::Raw;
  const int64_t C = a.NH * a.d;
  const Place p = place<V>(a.B, C, a.T, run);
  float dw[W][V] = {}, db[V] = {};
  if (p.on) {
    const int64_t n = length_of(a.lengths, p.b, a.T);
    const T* x = static_cast<const T*>(a.x) + p.b * a.T * a.x_row + p.c;
    const int64_t head = p.c / a.d;
    const T* dy = static_cast<const T*>(g.dy) + (p.b * a.NH + head) * a.T * a.d + p.c % a.d;
    T* dx = static_cast<T*>(g.dx) + p.b * a.T * C + p.c;
    const T* ds = g.dstate ? static_cast<const T*>(g.dstate) + p.b * (W - 1) * C + p.c : nullptr;
    T* dso = g.dstate_out ? static_cast<T*>(g.dstate_out) + p.b * (W - 1) * C + p.c : nullptr;
    float w[W][V], bias[V];
    load_weights<V, W>(a.weight, a.bias, p.c, w, bias);
    float z[W][V] = {};
    float gs[W][V] = {};  // g of the last W tokens, gs[W - 1] the current one
    if (p.t0 > 0) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
        rowvec::load(x + (p.t0 - (W - 1) + j) * a.x_row, z[j]);
    } else if (a.state) {
      const T* s = static_cast<const T*>(a.state) + p.b * (W - 1) * C + p.c;
#pragma unroll
      for (int j = 0; j < W - 1; ++j) rowvec::load(s + j * C, z[j]);
    }
    // token t: g_t and, with t < t1, its share of the weights' sums; then row
    // t of dz: an input W - 1 tokens back, or the state before the sequence
    auto step = [&](int64_t t, bool inside, const Raw<T, V>& rx, const Raw<T, V>& rdy) {
      if (inside) {
        float d[V];
        rowvec::floats(rx, z[W - 1]);
        rowvec::floats(rdy, d);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float s = bias[e];
#pragma unroll
          for (int j = 0; j < W; ++j) s = __builtin_fmaf(w[j][e], z[j][e], s);
          gs[W - 1][e] = a.silu ? d[e] * rowvec::silu_slope(s, rowvec::sigmoid(s)) : d[e];
        }
        if (t < p.t1) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            db[e] += gs[W - 1][e];
#pragma unroll
            for (int j = 0; j < W; ++j)
              dw[j][e] = __builtin_fmaf(gs[W - 1][e], z[j][e], dw[j][e]);
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) gs[W - 1][e] = 0.0f;
      }
      const bool before = t < W - 1;  // a row of the state, in the first run
      if (before ? p.t0 == 0 : t - (W - 1) >= p.t0) {
        float o[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          o[e] = 0.0f;
#pragma unroll
          for (int j = 0; j < W; ++j) o[e] = __builtin_fmaf(w[j][e], gs[W - 1 - j][e], o[e]);
        }
        if (ds && t >= n && t < n + W - 1) {
          float more[V];
          rowvec::load(ds + (t - n) * C, more);
#pragma unroll
          for (int e = 0; e < V; ++e) o[e] += more[e];
        }
        if (!before)
          rowvec::store(dx + (t - (W - 1)) * C, o);
        else if (dso)
          rowvec::store(dso + t * C, o);
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          z[j][e] = z[j + 1][e];
          gs[j][e] = gs[j + 1][e];
        }
    };
    const int64_t last = p.t1 + W - 1, end = last < n ? last : n;
    constexpr int kAhead = 4;
    int64_t t = p.t0;
    for (; t + kAhead <= end; t += kAhead) {
      Raw<T, V> rx[kAhead], ry[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        rx[i] = rowvec::load_raw<T, V>(x + (t + i) * a.x_row);
        ry[i] = rowvec::load_raw<T, V>(dy + (t + i) * a.d);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) step(t + i, true, rx[i], ry[i]);
    }
    const Raw<T, V> zero = {};
    for (; t < last; ++t) {
      const bool inside = t < end;
      step(t, inside, inside ? rowvec::load_raw<T, V>(x + t * a.x_row) : zero,
           inside ? rowvec::load_raw<T, V>(dy + t * a.d) : zero);
    }
  }
  // the workgroup's runs, in order
  __shared__ float sums[kRuns][kLanes * V];
  const int lane = threadIdx.x % kLanes, row = threadIdx.x / kLanes;
  const int64_t cols = (C / V + kLanes - 1) / kLanes;
  const int64_t first = (blockIdx.x % cols) * kLanes * V;
  float* mine = partials + (blockIdx.x / cols) * (W + 1) * C + first;
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < V; ++e) sums[row][lane * V + e] = j < W ? dw[j < W ? j : 0][e] : db[e];
    __syncthreads();
    for (int c = threadIdx.x; c < kLanes * V; c += kLanes * kRuns)
      if (first + c < C) {
        float s = 0.0f;
#pragma unroll
        for (int r = 0; r < kRuns; ++r) s += sums[r][c];
        mine[j * C + c] = s;
      }
  }
}

// sums over `n` rows of partials [n][W + 1][C]: a workgroup takes 32 columns, its
// eight rows of lanes every eighth partial, joined in order
__global__ __launch_bounds__(256) void conv_weight_sums_kernel(const float* partials, int64_t n,
                                                               int64_t C, int W, float* dweight,
                                                               float* dbias) {
  __shared__ float sums[8][32];
  const int lane = threadIdx.x % 32, row = threadIdx.x / 32;
  const int64_t all = (W + 1) * C, i = int64_t(blockIdx.x) * 32 + lane;
  float s = 0.0f;
  if (i < all)
    for (int64_t k = row; k < n; k += 8) s += partials[k * all + i];
  sums[row][lane] = s;
  __syncthreads();
  if (row == 0 && i < all) {
    for (int r = 1; r < 8; ++r) s += sums[r][lane];
    const int64_t j = i / C, c = i % C;
    if (j < W)
      dweight[c * W + j] = s;
    else if (dbias)
      dbias[c] = s;
  }
}

// Forward vectors of 16 bytes; with five and more weights to a channel bf16 takes 8,
// as the weights and the last inputs would not fit the registers.  Backward 8 bytes
// of bf16: with 16 a lane needs 203 registers and two waves fill a SIMD (8 x 2048 rows
// of 1536: 44 us, with 8 bytes 37).
constexpr int kBwdVec = 4;
constexpr int vec_of(int W, bool is_bf16) { return is_bf16 && W <= 4 ? 8 : 4; }

// Tokens of a run: 32, fewer where that leaves less than two waves to a SIMD, but
// no fewer than 8 (W - 1 at most are read twice).
int run_of(int64_t B, int64_t vectors, int64_t T) {
  int run = 32;
  while (run > 8 && B * vectors * ((T + run - 1) / run) < 2048 * 64) run /= 2;
  return run;
}

struct Grid {
  int64_t cols, spans;
  int run;
};
Grid grid_of(int64_t B, int64_t C, int64_t T, int vec) {
  const int64_t vectors = C / vec;
  const int run = run_of(B, vectors, T);
  return {(vectors + kLanes - 1) / kLanes, B * ((T + run * kRuns - 1) / (run * kRuns)), run};
}

template <typename T, int W>
void fwd(const ShortConv& a, void* y, void* state_out, const Grid& g, hipStream_t stream) {
  conv_fwd_kernel<T, vec_of(W, sizeof(T) == 2), W>
      <<<unsigned(g.cols * g.spans), kLanes * kRuns, 0, stream>>>(
          a, static_cast<T*>(y), static_cast<T*>(state_out), g.run);
}
template <typename T, int W>
void bwd(const ShortConv& a, const ShortConvGrads& gr, float* partials, const Grid& g,
         hipStream_t stream) {
  conv_bwd_kernel<T, kBwdVec, W><<<unsigned(g.cols * g.spans), kLanes * kRuns, 0, stream>>>(
      a, gr, partials, g.run);
}

// f<W>() for the call's width
template <typename F>
void with_width(int W, F&& f) {
  switch (W) {
    case 2: return f(std::integral_constant<int, 2>{});
    case 3: return f(std::integral_constant<int, 3>{});
    case 4: return f(std::integral_constant<int, 4>{});
    case 5: return f(std::integral_constant<int, 5>{});
    case 6: return f(std::integral_constant<int, 6>{});
    case 7: return f(std::integral_constant<int, 7>{});
    default: return f(std::integral_constant<int, 8>{});
  }
}

}  // namespace

hipError_t launch_short_conv_fwd(const ShortConv& a, void* y, void* state_out,
                                 hipStream_t stream) {
  const Grid g = grid_of(a.B, a.NH * a.d, a.T, vec_of(a.W, a.is_bf16));
  with_width(a.W, [&](auto w) {
    if (a.is_bf16)
      fwd<__hip_bfloat16, w()>(a, y, state_out, g, stream);
    else
      fwd<float, w()>(a, y, state_out, g, stream);
  });
  return hipGetLastError();
}

size_t short_conv_bwd_workspace_bytes(int64_t B, int64_t C, int64_t T, int W) {
  return size_t(grid_of(B, C, T, kBwdVec).spans) * size_t(W + 1) * size_t(C) * 4;
}

hipError_t launch_short_conv_bwd(const ShortConv& a, const ShortConvGrads& gr, void* workspace,
                                 hipStream_t stream) {
  const int64_t C = a.NH * a.d;
  const Grid g = grid_of(a.B, C, a.T, kBwdVec);
  float* partials = static_cast<float*>(workspace);
  with_width(a.W, [&](auto w) {
    if (a.is_bf16)
      bwd<__hip_bfloat16, w()>(a, gr, partials, g, stream);
    else
      bwd<float, w()>(a, gr, partials, g, stream);
  });
  conv_weight_sums_kernel<<<unsigned(((a.W + 1) * C + 31) / 32), 256, 0, stream>>>(
      partials, g.spans, C, a.W, gr.dweight, gr.dbias);
  return hipGetLastError();
}

}  // namespace mlstm
