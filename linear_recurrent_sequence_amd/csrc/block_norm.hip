// Block norm: the norm of a cell's output per head, its output gate, the
// scaled residual and the next block's norm, in one pass over the rows.
//
// For one token, with p in NH heads of d channels and D = NH d,
//
//   n1 = norm_d(p_head)          z = act(g) * w1 * n1
//   r  = x + s * z               n2 = norm_D(r)          y = w2 * n2
//
// norm(a) = (a - mean(a)) / sqrt(var(a) + eps)  (layer), or
//           a / sqrt(mean(a^2) + eps)           (root mean square);
// act is sigma(g) or g sigma(g).  p and g come head-major [B][NH][T][d], as
// the cells of this library write them; x, r and y are rows [B][T][D].
//
// Backward, from dr and dy (everything forward is formed again from p, g and
// x, which the pass reads in any case):
//
//   norm'(g, n) = inv (g - n mean(g n) - mean(g))   (the last term: layer only)
//   dr' = dr + norm'(w2 dy, n2),  dx = dr',  dz = s dr'
//   dg = dz w1 n1 act'(g),  dp = norm'(dz w1 act(g), n1)
//   dw1 = sum_rows dz act(g) n1,  ds = sum_rows dr' z,  dw2 = sum_rows dy n2
//
// The work is bound by memory: each element is read and written once and
// nothing else leaves the registers.  A lane holds vectors of 8 neighbouring
// channels (16 bytes of bf16).  A head takes the smallest power of two of
// lanes that covers d, so small heads share a wave and its sums are
// butterflies inside the head's lanes; a row takes as many waves as it needs,
// joined through LDS by one barrier per sum.  A workgroup keeps its share of
// the weights in registers over all rows it takes.  Sums of squares are taken
// about the wave's own mean and joined as (mean, M2) pairs, so a row far from
// zero loses nothing.  The weight gradients are summed per workgroup in
// registers, then over the workgroups in a fixed order by a second kernel: no
// atomics, results are bitwise reproducible.
//
// Measured (bf16, layer norm, gate and residual): forward on 8 x 2048 rows of
// 4 x 384 67 us, 51 us being a copy's time for the same bytes; 4 x 2048 rows of
// 8 x 512 95 us (67); backward there 176 us and 6 us for the weights' sums (108).
// What is left is the vector work of a row beside its loads: about 280
// instructions per 8 channels forward and 600 backward (bf16 spills 16 registers
// there, 60 bytes a lane).  Rows of more vectors of 8 channels than eight waves have
// lanes take two or four of them a lane, and with four the backward spills 137 to 231
// registers: 4 x 2048 rows of 20 x 384 in bf16 take 244 us forward and 1177 us
// backward (a copy of the same bytes 126 and 202), of 1 x 4096, two vectors, 78 and
// 169 (67 and 108).  The next row is loaded
// while one is worked on (two rows ahead gain nothing); with divisions by T per
// row, sums through LDS shuffles and the precise exponential the same took 96 us
// and 324 us.
#include "block_norm.h"

#include <hip/hip_bf16.h>

namespace mlstm {
namespace {

constexpr int kVec = 8;
constexpr int kMaxWaves = 8;  // of a row, and of a workgroup

struct Geometry {
  int64_t rows;         // B * T
  int64_t T;
  int NH, d, D;
  int lane_shift;       // log2 of a head's lanes
  int heads_per_pass;   // heads that a wave holds side by side
  int waves_per_head;   // > 1: a head spans several waves
  int waves_per_row;
  int rows_per_wg;
};

// 8 neighbouring elements as they lie in memory
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  float4 a, b;
};
template <>
struct Raw<__hip_bfloat16> {
  uint4 a;
};
template <typename T>
__device__ inline Raw<T> raw8(const T* p) {
  return *reinterpret_cast<const Raw<T>*>(p);
}
__device__ inline void floats(const Raw<float>& r, float* x) {
  x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w;
  x[4] = r.b.x; x[5] = r.b.y; x[6] = r.b.z; x[7] = r.b.w;
}
__device__ inline void floats(const Raw<__hip_bfloat16>& r, float* x) {
  const unsigned u[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ inline void load8(const float* p, float* x) { floats(raw8(p), x); }
__device__ inline void store8(float* p, const float* x) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ inline void store8(__hip_bfloat16* p, const float* x) {
  __bf16 b[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) b[i] = static_cast<__bf16>(x[i]);  // to nearest even
  *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(b);
}

// Butterflies in registers: x plus that of lane ^ 1, ^ 2 (quads), the mirrored
// lane of 8 and of 16 (whose halves are equal by then), lane ^ 16, lane ^ 32.
template <int kCtrl>
__device__ inline float plus_dpp(float x) {
  return x + __int_as_float(
                 __builtin_amdgcn_update_dpp(0, __float_as_int(x), kCtrl, 0xF, 0xF, true));
}
__device__ inline float plus_16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ inline float plus_32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// sum over the 2^shift lanes of a head (every lane gets it)
__device__ inline float head_sum(float x, int shift) {
  if (shift > 0) x = plus_dpp<0xB1>(x);
  if (shift > 1) x = plus_dpp<0x4E>(x);
  if (shift > 2) x = plus_dpp<0x141>(x);
  if (shift > 3) x = plus_dpp<0x140>(x);
  if (shift > 4) x = plus_16(x);
  if (shift > 5) x = plus_32(x);
  return x;
}
__device__ inline float wave_sum(float x) { return head_sum(x, 6); }

// mean and sum of squares about it of `n` values, joined with another set's
struct Moments {
  float n, mean, m2;
};
__device__ inline Moments join(Moments a, Moments b) {
  const float n = a.n + b.n, t = b.mean - a.mean;
  if (n == 0.0f) return a;
  return {n, a.mean + t * (b.n / n), a.m2 + b.m2 + t * t * (a.n * b.n / n)};
}

// One wave's share of a row: VPL vectors of each of NP sets of heads.
template <int VPL, int NP>
struct Lane {
  int64_t head_off[NP];    // of p and gate, from the (b, t) base: head * T * d
  int channel[NP * VPL];   // in the head
  int column[NP * VPL];    // in the row
  bool on[NP * VPL];
  float count;             // channels of the row that this wave holds
  float head_count;        // channels of one head that this wave holds

  __device__ Lane(const Geometry& g, int wave, int lane) {
    const int lph = 1 << g.lane_shift;
    const int pass0 = wave / g.waves_per_head * NP, part = wave % g.waves_per_head;
    float mine = 0.0f, in_head = 0.0f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int head = (pass0 + i) * g.heads_per_pass + (lane >> g.lane_shift);
      head_off[i] = int64_t(head) * g.T * g.d;
#pragma unroll
      for (int u = 0; u < VPL; ++u) {
        const int c = i * VPL + u;
        channel[c] = ((part * VPL + u) * lph + (lane & (lph - 1))) * kVec;
        on[c] = head < g.NH && channel[c] < g.d;
        column[c] = head * g.d + channel[c];
        if (on[c]) mine += kVec;
        if (i == 0 && channel[c] < g.d) in_head += kVec;
      }
    }
    count = wave_sum(mine);
    head_count = head_sum(in_head, g.lane_shift);
  }
};

// A wave's rows one after the other: (b, t) by addition, no division per row.
struct Rows {
  int64_t row, b, t, step, step_b, step_t;

  __device__ Rows(const Geometry& g, int sub) {
    step = int64_t(gridDim.x) * g.rows_per_wg;
    step_b = step / g.T;
    step_t = step % g.T;
    row = int64_t(blockIdx.x) * g.rows_per_wg + sub;
    b = row / g.T;
    t = row % g.T;
  }
  __device__ void next(const Geometry& g) {
    row += step;
    b += step_b;
    t += step_t;
    if (t >= g.T) t -= g.T, ++b;
  }
  __device__ bool live(const Geometry& g) const { return row < g.rows; }
  // of p and gate, before the head's offset
  __device__ int64_t base(const Geometry& g) const { return (b * g.NH * g.T + t) * g.d; }
};

// A wave's inputs of one row, zeros where off (and behind the end).
template <typename T, int VPL, int NP>
struct Inputs {
  Raw<T> p[VPL * NP], g[VPL * NP], x[VPL * NP];

  __device__ void load(const Geometry& geo, const Lane<VPL, NP>& L, const T* from_p,
                       const T* gate, const T* residual, const Rows& rows) {
    const int64_t base = rows.base(geo);
#pragma unroll
    for (int c = 0; c < VPL * NP; ++c) {
      p[c] = g[c] = x[c] = Raw<T>{};
      if (!L.on[c] || !rows.live(geo)) continue;
      const int64_t at = base + L.head_off[c / VPL] + L.channel[c];
      p[c] = raw8(from_p + at);
      if (gate) g[c] = raw8(gate + at);
      if (residual) x[c] = raw8(residual + rows.row * geo.D + L.column[c]);
    }
  }
};
template <typename T, int NC>
struct RowGrads {
  Raw<T> r[NC], y[NC];

  template <typename L>
  __device__ void load(const Geometry& geo, const L& lane, const T* dr, const T* dy,
                       const Rows& rows) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      r[c] = y[c] = Raw<T>{};
      if (!lane.on[c] || !rows.live(geo)) continue;
      const int64_t at = rows.row * geo.D + lane.column[c];
      if (dr) r[c] = raw8(dr + at);
      if (dy) y[c] = raw8(dy + at);
    }
  }
};

// Sums over a row's (or a head's) waves through LDS.  `slot` alternates
// between two from row to row: a wave writes a slot again only after the
// barrier of the row between.
__device__ inline Moments join_waves(Moments m, Moments* slot, int wave0, int wave, int n) {
  if (n == 1) return m;
  if ((threadIdx.x & 63) == 0) slot[wave] = m;
  __syncthreads();
  Moments a = slot[wave0];
  for (int w = 1; w < n; ++w) a = join(a, slot[wave0 + w]);
  return a;
}
__device__ inline float2 add_waves(float2 x, float2* slot, int wave0, int wave, int n) {
  if (n == 1) return x;
  if ((threadIdx.x & 63) == 0) slot[wave] = x;
  __syncthreads();
  float2 a = slot[wave0];
  for (int w = 1; w < n; ++w) {
    a.x += slot[wave0 + w].x;
    a.y += slot[wave0 + w].y;
  }
  return a;
}

template <bool kLayer>
__device__ inline float inverse(Moments m, float eps) {
  // root mean square: `mean` stays 0 and m2 is the sum of squares
  return 1.0f / sqrtf(m.m2 / m.n + eps);
}

struct Shared {
  Moments row[2][kMaxWaves], head[2][kMaxWaves];
  float2 row_grad[2][kMaxWaves], head_grad[2][kMaxWaves];
};

// n1 in place of p, and each head's 1 / sqrt(...)
template <bool kLayer, int VPL, int NP>
__device__ inline void head_norms(const Geometry& g, const Lane<VPL, NP>& L, float (*p)[kVec],
                                  float* inv, float eps, Moments* slot, int wave0, int wave) {
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    Moments m = {L.head_count, 0.0f, 0.0f};
    if (kLayer) {
      float s = 0.0f;
#pragma unroll
      for (int u = 0; u < VPL; ++u)
#pragma unroll
        for (int e = 0; e < kVec; ++e) s += p[i * VPL + u][e];  // 0 where off
      s = head_sum(s, g.lane_shift);
      m.mean = m.n > 0.0f ? s / m.n : 0.0f;
    }
    float q = 0.0f;
#pragma unroll
    for (int u = 0; u < VPL; ++u)
      if (L.on[i * VPL + u])
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const float t = p[i * VPL + u][e] - m.mean;
          q += t * t;
        }
    m.m2 = head_sum(q, g.lane_shift);
    // a head over several waves is the wave's only one (NP = 1, all lanes)
    if (g.waves_per_head > 1)
      m = join_waves(m, slot, wave0 + (wave - wave0) / g.waves_per_head * g.waves_per_head, wave,
                     g.waves_per_head);
    inv[i] = inverse<kLayer>(m, eps);
#pragma unroll
    for (int u = 0; u < VPL; ++u)
#pragma unroll
      for (int e = 0; e < kVec; ++e)
        p[i * VPL + u][e] = L.on[i * VPL + u] ? (p[i * VPL + u][e] - m.mean) * inv[i] : 0.0f;
  }
}

// the row's mean and 1 / sqrt(...)
template <bool kLayer, int NC>
__device__ inline float2 row_norm(const float (*r)[kVec], const bool* on, float count, float eps,
                                  Moments* slot, int wave0, int wave, int waves) {
  Moments m = {count, 0.0f, 0.0f};
  if (kLayer) {
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int e = 0; e < kVec; ++e) s += r[c][e];  // 0 where off
    s = wave_sum(s);
    m.mean = count > 0.0f ? s / count : 0.0f;
  }
  float q = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c)
    if (on[c])
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const float t = r[c][e] - m.mean;
        q += t * t;
      }
  m.m2 = wave_sum(q);
  m = join_waves(m, slot, wave0, wave, waves);
  return make_float2(m.mean, inverse<kLayer>(m, eps));
}

// sigma(x) and sigma(-x) from e^-|x|: neither overflows nor cancels.  For bf16
// the exponential and the reciprocal are the hardware's (an exponent of x log2 e
// rounded once, 2^-24 |x|, and 1 ulp): far below the output's rounding, and a
// third of the instructions, which bounded the pass.
struct Sigmoid {
  float plus, minus;
};
template <typename T>
__device__ inline Sigmoid sigmoid(float x) {
  float t, s;
  if (sizeof(T) == 2) {
    t = __builtin_amdgcn_exp2f(-1.44269504f * fabsf(x));
    s = __builtin_amdgcn_rcpf(1.0f + t);
  } else {
    t = expf(-fabsf(x));
    s = 1.0f / (1.0f + t);
  }
  return x >= 0.0f ? Sigmoid{s, t * s} : Sigmoid{t * s, s};
}

template <typename T, bool kLayer, int VPL, int NP>
__global__ __launch_bounds__(kMaxWaves * 64) void block_norm_fwd_kernel(
    Geometry g, const T* __restrict__ p, const T* __restrict__ gate,
    const T* __restrict__ residual, const float* __restrict__ weight,
    const float* __restrict__ scale, const float* __restrict__ next_weight,
    T* __restrict__ r_out, T* __restrict__ y_out, float eps, int silu) {
  constexpr int NC = VPL * NP;
  __shared__ Shared sh;
  const int all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), sub = all / g.waves_per_row;
  const int wave = all % g.waves_per_row, wave0 = sub * g.waves_per_row;
  const Lane<VPL, NP> L(g, wave, threadIdx.x & 63);
  float w1[NC][kVec], sc[NC][kVec], w2[NC][kVec];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int e = 0; e < kVec; ++e) w1[c][e] = w2[c][e] = 0.0f, sc[c][e] = 1.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c)
    if (L.on[c]) {
      load8(weight + L.column[c], w1[c]);
      if (scale) load8(scale + L.column[c], sc[c]);
      if (next_weight) load8(next_weight + L.column[c], w2[c]);
    }
  int parity = 0;
  constexpr bool kAhead = NC <= 2;  // where registers allow it (two rows ahead gain nothing)
  Rows next(g, sub);
  Inputs<T, VPL, NP> now;
  if (kAhead) now.load(g, L, p, gate, residual, next);
  // the same number of turns for all of a workgroup's rows: they share barriers
  for (int64_t first = int64_t(blockIdx.x) * g.rows_per_wg; first < g.rows;
       first += next.step, parity ^= 1) {
    if (!kAhead) now.load(g, L, p, gate, residual, next);
    const bool live = next.live(g);
    const int64_t row = next.row;
    next.next(g);
    float z[NC][kVec], gt[NC][kVec], r[NC][kVec];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      floats(now.p[c], z[c]);
      floats(now.g[c], gt[c]);
      floats(now.x[c], r[c]);
    }
    // the next row is on its way while this one is worked on
    if (kAhead) now.load(g, L, p, gate, residual, next);
    float inv1[NP];
    head_norms<kLayer, VPL, NP>(g, L, z, inv1, eps, sh.head[parity], wave0, all);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        float v = z[c][e] * w1[c][e];
        if (gate) {
          const float sg = sigmoid<T>(gt[c][e]).plus;
          v *= silu ? gt[c][e] * sg : sg;
        }
        // off: 0 by a select, since a weight or gate of 0 times it is not 0 for infinities
        r[c][e] = L.on[c] ? r[c][e] + sc[c][e] * v : 0.0f;
      }
      if (L.on[c] && live) store8(r_out + row * g.D + L.column[c], r[c]);
    }
    if (next_weight) {
      const float2 m = row_norm<kLayer, NC>(r, L.on, L.count, eps, sh.row[parity], wave0, all,
                                            g.waves_per_row);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) r[c][e] = (r[c][e] - m.x) * m.y * w2[c][e];
        if (L.on[c] && live) store8(y_out + row * g.D + L.column[c], r[c]);
      }
    }
  }
}

// The weight gradients of one workgroup's rows go to partials[...][2][D]: a =
// sum_rows dr' act(g) n1 (dw1 = s a and ds = w1 a, both constant in a column)
// and dw2.  The weights stay in LDS: with them in registers fewer waves fit.
template <typename T, bool kLayer, int VPL, int NP>
__global__ __launch_bounds__(
    kMaxWaves * 64, VPL * NP > 1 ? 2 : sizeof(T) == 2 ? 4 : 3) void block_norm_bwd_kernel(
    Geometry g, const T* __restrict__ p, const T* __restrict__ gate,
    const T* __restrict__ residual, const float* __restrict__ weight,
    const float* __restrict__ scale, const float* __restrict__ next_weight,
    const T* __restrict__ dr, const T* __restrict__ dy, T* __restrict__ dp,
    T* __restrict__ dgate, T* __restrict__ dresidual, float* __restrict__ partials, float eps,
    int silu) {
  constexpr int NC = VPL * NP;
  __shared__ Shared sh;
  const int all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), sub = all / g.waves_per_row;
  const int wave = all % g.waves_per_row, wave0 = sub * g.waves_per_row;
  const Lane<VPL, NP> L(g, wave, threadIdx.x & 63);
  float da[NC][kVec], dw2[NC][kVec];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int e = 0; e < kVec; ++e) da[c][e] = dw2[c][e] = 0.0f;
  // w1, s and w2 (`what` 0 - 2) of a lane's channels: with one vector per lane
  // from LDS, written and read by the same lane (6 KiB a wave); with more they
  // would not fit, and come from the cache
  constexpr bool kHeld = NC == 1;
  extern __shared__ __attribute__((aligned(16))) float weights[];
  auto cached = [&](int what, int c, float* w) {
    const float* from = what == 0 ? weight : what == 1 ? scale : next_weight;
#pragma unroll
    for (int e = 0; e < kVec; ++e) w[e] = what == 1 ? 1.0f : 0.0f;
    if (from && L.on[c]) load8(from + L.column[c], w);
  };
  auto held = [&](int what, int c, float* w) {
    if (!kHeld) return cached(what, c, w);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float4 x = *reinterpret_cast<const float4*>(
          weights + ((what * 2 + q) * blockDim.x + threadIdx.x) * 4);
      w[4 * q] = x.x; w[4 * q + 1] = x.y; w[4 * q + 2] = x.z; w[4 * q + 3] = x.w;
    }
  };
  if (kHeld)
#pragma unroll
    for (int what = 0; what < 3; ++what) {
      float w[kVec];
      cached(what, 0, w);
#pragma unroll
      for (int q = 0; q < 2; ++q)
        *reinterpret_cast<float4*>(weights + ((what * 2 + q) * blockDim.x + threadIdx.x) * 4) =
            make_float4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    }
  const float inv_d = 1.0f / float(g.d), inv_D = 1.0f / float(g.D);
  int parity = 0;
  const T* const x_in = next_weight ? residual : nullptr;  // only r needs it
  const T* const dy_in = next_weight ? dy : nullptr;
  constexpr bool kAhead = NC == 1;
  Rows next(g, sub);
  Inputs<T, VPL, NP> now;
  RowGrads<T, NC> grads;
  if (kAhead) {
    now.load(g, L, p, gate, x_in, next);
    grads.load(g, L, dr, dy_in, next);
  }
  for (int64_t first = int64_t(blockIdx.x) * g.rows_per_wg; first < g.rows;
       first += next.step, parity ^= 1) {
    if (!kAhead) {
      now.load(g, L, p, gate, x_in, next);
      grads.load(g, L, dr, dy_in, next);
    }
    const bool live = next.live(g);
    const int64_t row = next.row, base = next.base(g);
    next.next(g);
    float n1[NC][kVec], gt[NC][kVec], r[NC][kVec], gr[NC][kVec], gy[NC][kVec];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      floats(now.p[c], n1[c]);
      floats(now.g[c], gt[c]);
      floats(now.x[c], r[c]);
      floats(grads.r[c], gr[c]);
      floats(grads.y[c], gy[c]);
    }
    if (kAhead) {
      now.load(g, L, p, gate, x_in, next);
      grads.load(g, L, dr, dy_in, next);
    }
    float inv1[NP];
    head_norms<kLayer, VPL, NP>(g, L, n1, inv1, eps, sh.head[parity], wave0, all);
    // act(g), and its slope in g's place
    float act[NC][kVec];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float w1[kVec], sc[kVec];
      if (next_weight) {
        held(0, c, w1);
        held(1, c, sc);
      }
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        float a = 1.0f, slope = 0.0f;
        if (gate) {
          const float x = gt[c][e];
          const Sigmoid sg = sigmoid<T>(x);
          a = silu ? x * sg.plus : sg.plus;
          slope = silu ? sg.plus * (1.0f + x * sg.minus) : sg.plus * sg.minus;
        }
        act[c][e] = a;
        gt[c][e] = slope;
        if (next_weight) r[c][e] = L.on[c] ? r[c][e] + sc[e] * (n1[c][e] * w1[e] * a) : 0.0f;
      }
    }
    if (next_weight) {
      const float2 m = row_norm<kLayer, NC>(r, L.on, L.count, eps, sh.row[parity], wave0, all,
                                            g.waves_per_row);
      float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (L.on[c]) {
          float w2[kVec];
          held(2, c, w2);
#pragma unroll
          for (int e = 0; e < kVec; ++e) {
            r[c][e] = (r[c][e] - m.x) * m.y;  // n2
            if (live) dw2[c][e] += gy[c][e] * r[c][e];
            gy[c][e] *= w2[e];
            s.x += gy[c][e] * r[c][e];
            s.y += gy[c][e];
          }
        }
      s = add_waves(make_float2(wave_sum(s.x), wave_sum(s.y)), sh.row_grad[parity], wave0, all,
                    g.waves_per_row);
      s.x *= inv_D;
      s.y = kLayer ? s.y * inv_D : 0.0f;
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (L.on[c])
#pragma unroll
          for (int e = 0; e < kVec; ++e) gr[c][e] += m.y * (gy[c][e] - r[c][e] * s.x - s.y);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (!L.on[c]) continue;
      if (residual && live) store8(dresidual + row * g.D + L.column[c], gr[c]);
      float dg[kVec], w1[kVec], sc[kVec];
      held(0, c, w1);
      held(1, c, sc);
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        if (live) da[c][e] += gr[c][e] * (n1[c][e] * act[c][e]);
        const float dz = gr[c][e] * sc[e] * w1[e];
        dg[e] = dz * n1[c][e] * gt[c][e];
        gr[c][e] = dz * act[c][e];
      }
      if (gate && live) store8(dgate + base + L.head_off[c / VPL] + L.channel[c], dg);
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int u = 0; u < VPL; ++u)
        if (L.on[i * VPL + u])
#pragma unroll
          for (int e = 0; e < kVec; ++e) {
            s.x += gr[i * VPL + u][e] * n1[i * VPL + u][e];
            s.y += gr[i * VPL + u][e];
          }
      s = make_float2(head_sum(s.x, g.lane_shift), head_sum(s.y, g.lane_shift));
      if (g.waves_per_head > 1)
        s = add_waves(s, sh.head_grad[parity],
                      wave0 + wave / g.waves_per_head * g.waves_per_head, all, g.waves_per_head);
      s.x *= inv_d;
      s.y = kLayer ? s.y * inv_d : 0.0f;
#pragma unroll
      for (int u = 0; u < VPL; ++u) {
        const int c = i * VPL + u;
        if (!L.on[c] || !live) continue;
#pragma unroll
        for (int e = 0; e < kVec; ++e) gr[c][e] = inv1[i] * (gr[c][e] - n1[c][e] * s.x - s.y);
        store8(dp + base + L.head_off[i] + L.channel[c], gr[c]);
      }
    }
  }
  // several rows of a workgroup side by side write a partial each
  float* out = partials + (int64_t(blockIdx.x) * g.rows_per_wg + sub) * 2 * g.D;
#pragma unroll
  for (int c = 0; c < NC; ++c)
    if (L.on[c]) {
      store8(out + L.column[c], da[c]);
      if (next_weight) store8(out + g.D + L.column[c], dw2[c]);
    }
}

// Sums of the partials over the workgroups: 64 columns and 16 shares of the
// partials to a workgroup, each share in order, then the shares in order.
constexpr int kShares = 16;
__global__ __launch_bounds__(64 * kShares) void block_norm_weights_kernel(
    const float* __restrict__ partials, const float* __restrict__ weight,
    const float* __restrict__ scale, float* dweight, float* dscale, float* dnext_weight, int n,
    int D) {
  __shared__ float part[kShares][64];
  const int lane = threadIdx.x & 63, share = threadIdx.x >> 6, col = blockIdx.x * 64 + lane;
  if (blockIdx.y == 1 && !dnext_weight) return;  // the same for the whole workgroup
  float s = 0.0f;
  if (col < D)
#pragma unroll 4
    for (int i = share; i < n; i += kShares) s += partials[(int64_t(i) * 2 + blockIdx.y) * D + col];
  part[share][lane] = s;
  __syncthreads();
  if (share == 0 && col < D) {
    for (int i = 1; i < kShares; ++i) s += part[i][lane];
    if (blockIdx.y == 1) {
      dnext_weight[col] = s;
    } else {
      dweight[col] = scale ? scale[col] * s : s;
      if (dscale) dscale[col] = weight[col] * s;
    }
  }
}

struct Shape {
  Geometry g;
  int vpl, np;
};

// Vectors per lane and head, sets of heads per wave, and waves per row: one
// vector per wave if 8 waves then hold a row (the most waves share it, and the
// fewest registers hold weights), else two, else four.  At least half of a
// wave's lanes hold channels whatever d is, so 8 waves of 4 vectors hold any
// row of kBlockNormMaxRow.
Shape shape_of(int64_t B, int64_t NH, int64_t T, int64_t d) {
  Shape s;
  Geometry& g = s.g;
  g.rows = B * T;
  g.T = T;
  g.NH = int(NH);
  g.d = int(d);
  g.D = int(NH * d);
  const int vecs = int((d + kVec - 1) / kVec);
  g.lane_shift = 0;
  while (g.lane_shift < 6 && (1 << g.lane_shift) < vecs) ++g.lane_shift;
  g.heads_per_pass = 64 >> g.lane_shift;
  const int per_head = (vecs + 63) / 64;  // waves a head takes at one vector per lane
  const int passes = (int(NH) + g.heads_per_pass - 1) / g.heads_per_pass;
  if (per_head == 1) {
    s.vpl = 1;
    s.np = passes <= 8 ? 1 : passes <= 16 ? 2 : 4;
    g.waves_per_head = 1;
  } else if (per_head == 2) {
    s.vpl = 2;
    s.np = passes <= 8 ? 1 : 2;
    g.waves_per_head = 1;
  } else {
    s.vpl = (per_head + 1) / 2 * passes <= 8 ? 2 : 4;
    s.np = 1;
    g.waves_per_head = (per_head + s.vpl - 1) / s.vpl;
  }
  g.waves_per_row = (passes + s.np - 1) / s.np * g.waves_per_head;
  g.rows_per_wg = g.waves_per_row >= 4 ? 1 : 4 / g.waves_per_row;
  return s;
}

// Workgroups: as many as the card holds at once (the waves that a CU has
// registers for, by vectors per lane: a second round of workgroups would leave
// part of it idle), and no more than there are rows.
constexpr int kCUs = 256;
unsigned grid_of(const Geometry& g, int waves) {
  const int64_t need = (g.rows + g.rows_per_wg - 1) / g.rows_per_wg;
  const int64_t most = kCUs * (waves / (g.waves_per_row * g.rows_per_wg));
  return unsigned(need < most ? need : most);
}
unsigned fwd_grid(const Geometry& g, int vectors) {
  return grid_of(g, vectors == 1 ? 20 : vectors == 2 ? 12 : 8);
}
// backward: a workgroup's partials are worth about a row's traffic, so from two
// workgroups per CU on each takes at least four rows
unsigned bwd_grid(const Geometry& g, int vectors) {
  const unsigned most = grid_of(g, vectors == 1 ? 16 : 8);
  const int64_t four = (g.rows + 4 * g.rows_per_wg - 1) / (4 * g.rows_per_wg);
  const int64_t n = four > 2 * kCUs ? four : 2 * kCUs;
  return n < most ? unsigned(n) : most;
}

template <typename T, bool kLayer, int VPL, int NP>
hipError_t fwd(const Shape& s, const BlockNorm& a, void* r, void* y, hipStream_t stream) {
  const Geometry& g = s.g;
  block_norm_fwd_kernel<T, kLayer, VPL, NP>
      <<<fwd_grid(g, VPL * NP), 64 * g.waves_per_row * g.rows_per_wg, 0, stream>>>(
          g, static_cast<const T*>(a.p), static_cast<const T*>(a.gate),
          static_cast<const T*>(a.residual), a.weight, a.scale, a.next_weight,
          static_cast<T*>(r), static_cast<T*>(y), a.eps, int(a.silu));
  return hipGetLastError();
}

template <typename T, bool kLayer, int VPL, int NP>
hipError_t bwd(const Shape& s, const BlockNorm& a, const BlockNormGrads& d, float* partials,
               hipStream_t stream) {
  const Geometry& g = s.g;
  const unsigned grid = bwd_grid(g, VPL * NP);
  const unsigned threads = 64 * g.waves_per_row * g.rows_per_wg;
  block_norm_bwd_kernel<T, kLayer, VPL, NP>
      <<<grid, threads, VPL * NP == 1 ? threads * 3 * kVec * sizeof(float) : 0, stream>>>(
          g, static_cast<const T*>(a.p), static_cast<const T*>(a.gate),
          static_cast<const T*>(a.residual), a.weight, a.scale, a.next_weight,
          static_cast<const T*>(d.dr), static_cast<const T*>(d.dy), static_cast<T*>(d.dp),
          static_cast<T*>(d.dgate), static_cast<T*>(d.dresidual), partials, a.eps, int(a.silu));
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  block_norm_weights_kernel<<<dim3((g.D + 63) / 64, 2), 64 * kShares, 0, stream>>>(
      partials, a.weight, a.scale, d.dweight, a.scale ? d.dscale : nullptr,
      a.next_weight ? d.dnext_weight : nullptr, int(grid) * g.rows_per_wg, g.D);
  return hipGetLastError();
}

// the kernel of a shape, type and norm
template <typename F>
hipError_t dispatch(const Shape& s, const BlockNorm& a, F&& f) {
  using B16 = __hip_bfloat16;
#define MLSTM_NORM_CASE(V, N)                                                        \
  if (s.vpl == V && s.np == N) {                                                     \
    if (a.is_bf16)                                                                   \
      return a.layer ? f.template operator()<B16, true, V, N>()                      \
                     : f.template operator()<B16, false, V, N>();                    \
    return a.layer ? f.template operator()<float, true, V, N>()                      \
                   : f.template operator()<float, false, V, N>();                    \
  }
  MLSTM_NORM_CASE(1, 1)
  MLSTM_NORM_CASE(1, 2)
  MLSTM_NORM_CASE(1, 4)
  MLSTM_NORM_CASE(2, 1)
  MLSTM_NORM_CASE(2, 2)
  MLSTM_NORM_CASE(4, 1)
#undef MLSTM_NORM_CASE
  return hipErrorInvalidValue;
}

struct Fwd {
  const Shape& s;
  const BlockNorm& a;
  void *r, *y;
  hipStream_t stream;
  template <typename T, bool kLayer, int VPL, int NP>
  hipError_t operator()() {
    return fwd<T, kLayer, VPL, NP>(s, a, r, y, stream);
  }
};
struct Bwd {
  const Shape& s;
  const BlockNorm& a;
  const BlockNormGrads& d;
  float* partials;
  hipStream_t stream;
  template <typename T, bool kLayer, int VPL, int NP>
  hipError_t operator()() {
    return bwd<T, kLayer, VPL, NP>(s, a, d, partials, stream);
  }
};

}  // namespace

size_t block_norm_partial_bytes(int64_t B, int64_t NH, int64_t T, int64_t d) {
  const Shape s = shape_of(B, NH, T, d);
  return size_t(bwd_grid(s.g, s.vpl * s.np)) * s.g.rows_per_wg * 2 * s.g.D * sizeof(float);
}

hipError_t launch_block_norm_fwd(const BlockNorm& a, void* r_out, void* y_out,
                                 hipStream_t stream) {
  const Shape s = shape_of(a.B, a.NH, a.T, a.d);
  return dispatch(s, a, Fwd{s, a, r_out, y_out, stream});
}

hipError_t launch_block_norm_bwd(const BlockNorm& a, const BlockNormGrads& d, float* partials,
                                 hipStream_t stream) {
  const Shape s = shape_of(a.B, a.NH, a.T, a.d);
  return dispatch(s, a, Bwd{s, a, d, partials, stream});
}

}  // namespace mlstm
