// Backward pass of the gated delta rule, in chunks of 64 tokens.
//
// With the forward's terms of a chunk (delta_fwd.hip: S at its start, R = V -
// e^G K S, X = (I + At)^-1 R, U = beta X), dh, and Z = dL/dS at its end,
//
//   dU = P^T dh + e^(G_C - G) K Z,   dR = (I + At)^-T (beta dU),   dV = dR
//   dS = e^(G_C) Z + (e^G Q^)^T dh - (e^G K)^T dR
//
// and, with B_ij = D_ij (dh_i . U_j) (j <= i) and N_ij = D_ij (dR_i . U_j) (j < i),
//
//   dq^ = e^G dh S^T + B K
//   dk  = e^(G_C - G) U Z^T + B^T Q^ - e^G dR S^T - (N + N^T) K
//   dbeta_j = X_j . dU_j - sum_i D_ij (dR_i . X_j) (k_i . k_j)
//   dG_j = e^(G_j) dh_j . (S^T q^_j) + sum_(i<j) P_ji (dh_j . U_i) - sum_(i>j) P_ij (dh_i . U_j)
//          - dR_j . (V_j - X_j) + sum_(i>j) N_ij (k_i . k_j) - e^(G_C - G_j) U_j . (Z^T k_j)
//   dG_C += sum_j e^(G_C - G_j) U_j . (Z^T k_j) + e^(G_C) <S, Z>
//
// (V_j - X_j is what the memory predicted for token j), and dlog f is the sum
// of dG from its token to the chunk's end, so no sum is longer than a chunk.
//
// Four passes: the terms that all columns share (delta_prep.hip), the memory
// forward once more (its start and X of every chunk are kept, float32), the
// gradient of the memory backward (Z and dR kept), and, over all chunks at
// once, the gradients of q, k, beta and the gates.  The two chains hold 16
// value columns per wave in the accumulators, as the forward does.  Everything
// that the float32 gradients (beta, gates, memory) come from has float32
// accuracy (three bf16 planes); for bf16 inputs the products that only dq and
// dk take carry two planes per operand (16 bits), dq and dk being rounded to 8.
#include "delta_common.h"
#include "delta_internal.h"

namespace mlstm {
namespace delta {
namespace {

constexpr int kWaves = 4;

// the position of accumulator (tile i, lane group g, element 0)
__device__ inline int acc_row(int i, int g) { return (i >> 1) * 32 + 8 * g + 4 * (i & 1); }

template <typename T>
struct Chain {
  const T *q, *k, *v, *dh;
  Work ws;
  Saved sv;
  int64_t T_len, H;
  int chunks, NH, NHK, dk, dv, per_head, tiles;
  float scale;
};

// left operand tile i, columns t * 32 + 8 g ..: rows of q or k (bf16, those
// behind the end repeat the last: their results are dropped), or their planes
template <typename T, int KS>
__device__ inline auto key_frag(const Chain<T>& a, const T* x, const __bf16* planes,
                                int64_t khead, int64_t chunk, int valid, int t, int i, int lane) {
  const int g = lane >> 4, m = lane & 15;
  if constexpr (sizeof(T) == 2) {
    const int tok = (i >> 1) * 32 + row_of(i & 1, m), c = t * 32 + g * 8;
    return load_row<1>(
        x, (khead * a.T_len + chunk * kC + (tok < valid ? tok : valid - 1)) * a.dk + c, c < a.dk);
  } else {
    constexpr int64_t kPlane = int64_t(KS) * 32 * kC;
    return load_frag<3>(planes + (khead * a.chunks + chunk) * 3 * kPlane, kPlane, t * 4 + i, lane);
  }
}

// The memory once more: S at each chunk's start, X, and the part e^G dh . (S^T q^)
// of dG that each 16 value columns give.
template <typename T, int KS>
__global__ __launch_bounds__(64 * kWaves) void delta_again_kernel(Chain<T> a, const float* C_in) {
  constexpr int NPL = sizeof(T) == 2 ? 1 : 3;
  constexpr int64_t kPlane = int64_t(KS) * 32 * kC;
  int64_t head;
  int block;
  map_head(blockIdx.x, a.H, a.per_head, head, block);
  const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
  const int tile = block * kWaves + (threadIdx.x >> 6), col = tile * 16 + m;
  if (col >= a.dv) return;  // whole waves; no barrier follows
  const int64_t khead = head / a.NH * a.NHK + head % a.NH / (a.NH / a.NHK);

  f32x4 S[2 * KS];
#pragma unroll
  for (int i = 0; i < 2 * KS; ++i) {
    S[i] = f32x4{};
    if (C_in && acc_row(i, g) < a.dk)
      S[i] = *reinterpret_cast<const f32x4*>(C_in + (head * a.dv + col) * a.dk + acc_row(i, g));
  }
  for (int chunk = 0; chunk < a.chunks; ++chunk) {
    const int64_t at = head * a.chunks + chunk, kat = khead * a.chunks + chunk;
    const int64_t tok0 = int64_t(chunk) * kC;
    const int valid = a.T_len - tok0 < kC ? int(a.T_len - tok0) : kC;
    const float* decay = a.ws.decay + at * 3 * kC;
#pragma unroll
    for (int i = 0; i < 2 * KS; ++i)
      if (acc_row(i, g) < a.dk)
        *reinterpret_cast<f32x4*>(a.sv.S + (at * a.dv + col) * a.dk + acc_row(i, g)) = S[i];

    f32x4 ks[4] = {}, qs[4] = {};
#pragma unroll
    for (int t = 0; t < KS; ++t) {
      const Planes<3> s = split<3>(pair(S[2 * t], S[2 * t + 1]));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ks[i] = mma_planes<3>(
            key_frag<T, KS>(a, a.k, a.ws.key, khead, chunk, valid, t, i, lane), s, ks[i]);
        qs[i] = mma_planes<3>(
            key_frag<T, KS>(a, a.q, a.ws.query, khead, chunk, valid, t, i, lane), s, qs[i]);
      }
    }
    f32x4 R[4], U[4] = {};
    float* part = a.sv.part + (at * a.tiles + tile) * 3 * kC;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = acc_row(i, g);
      const f32x4 e = *reinterpret_cast<const f32x4*>(decay + tok);
      f32x4 s;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        R[i][r] = 0.0f;
        float x = 0.0f;
        if (tok + r < valid) {
          const int64_t from = (head * a.T_len + tok0 + tok + r) * a.dv + col;
          R[i][r] = load_elem(a.v + from) - e[r] * ks[i][r];
          x = load_elem(a.dh + from) * (a.scale * e[r] * qs[i][r]);
        }
        s[r] = row_sum(x);
      }
      if (m == 0) *reinterpret_cast<f32x4*>(part + tok) = s;
    }
    const __bf16* inv = a.ws.inv + at * 3 * kSquare;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const Planes<3> b = split<3>(pair(R[2 * s], R[2 * s + 1]));
#pragma unroll
      for (int i = 2 * s; i < 4; ++i)
        U[i] = mma_planes<3>(load_frag<3>(inv, kSquare, i * 2 + s, lane), b, U[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = acc_row(i, g);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (tok + r < valid) a.sv.X[(head * a.T_len + tok0 + tok + r) * a.dv + col] = U[i][r];
      U[i] *= *reinterpret_cast<const f32x4*>(decay + 2 * kC + tok) *
              *reinterpret_cast<const f32x4*>(decay + kC + tok);
    }
    const float e_all = decay[kC - 1];
    const Planes<3> u0 = split<3>(pair(U[0], U[1])), u1 = split<3>(pair(U[2], U[3]));
    const __bf16* keyT = a.ws.keyT + kat * NPL * kPlane;
#pragma unroll
    for (int i = 0; i < 2 * KS; ++i) {
      S[i] *= e_all;
      S[i] = mma_planes<3>(load_frag<NPL>(keyT, kPlane, i * 2, lane), u0, S[i]);
      S[i] = mma_planes<3>(load_frag<NPL>(keyT, kPlane, i * 2 + 1, lane), u1, S[i]);
    }
  }
}

// The memory's gradient backward: Z at each chunk's end, dR (and dV), and the
// parts X . (e^(G_C - G) Z^T k) and dR . (V - X) that each 16 columns give.
template <typename T, int KS>
__global__ __launch_bounds__(64 * kWaves) void delta_back_kernel(Chain<T> a, const float* dC_in,
                                                                 T* dv_out, float* dC_out) {
  constexpr int NPL = sizeof(T) == 2 ? 1 : 3;
  constexpr int64_t kPlane = int64_t(KS) * 32 * kC;
  int64_t head;
  int block;
  map_head(blockIdx.x, a.H, a.per_head, head, block);
  const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
  const int tile = block * kWaves + (threadIdx.x >> 6), col = tile * 16 + m;
  if (col >= a.dv) return;
  const int64_t khead = head / a.NH * a.NHK + head % a.NH / (a.NH / a.NHK);

  f32x4 Z[2 * KS];
#pragma unroll
  for (int i = 0; i < 2 * KS; ++i) {
    Z[i] = f32x4{};
    if (dC_in && acc_row(i, g) < a.dk)
      Z[i] = *reinterpret_cast<const f32x4*>(dC_in + (head * a.dv + col) * a.dk + acc_row(i, g));
  }
  for (int chunk = a.chunks - 1; chunk >= 0; --chunk) {
    const int64_t at = head * a.chunks + chunk, kat = khead * a.chunks + chunk;
    const int64_t tok0 = int64_t(chunk) * kC;
    const int valid = a.T_len - tok0 < kC ? int(a.T_len - tok0) : kC;
    const float* decay = a.ws.decay + at * 3 * kC;
#pragma unroll
    for (int i = 0; i < 2 * KS; ++i)
      if (acc_row(i, g) < a.dk)
        *reinterpret_cast<f32x4*>(a.sv.Z + (at * a.dv + col) * a.dk + acc_row(i, g)) = Z[i];

    // K Z
    f32x4 kz[4] = {};
#pragma unroll
    for (int t = 0; t < KS; ++t) {
      const Planes<3> s = split<3>(pair(Z[2 * t], Z[2 * t + 1]));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        kz[i] = mma_planes<3>(
            key_frag<T, KS>(a, a.k, a.ws.key, khead, chunk, valid, t, i, lane), s, kz[i]);
    }
    f32x4 dh[4], X[4], pred[4];
    float* part = a.sv.part + (at * a.tiles + tile) * 3 * kC;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = acc_row(i, g);
      const f32x4 e = *reinterpret_cast<const f32x4*>(decay + kC + tok);
      f32x4 s;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        dh[i][r] = X[i][r] = pred[i][r] = 0.0f;
        kz[i][r] = tok + r < valid ? kz[i][r] * e[r] : 0.0f;
        if (tok + r < valid) {
          const int64_t from = (head * a.T_len + tok0 + tok + r) * a.dv + col;
          dh[i][r] = load_elem(a.dh + from);
          X[i][r] = a.sv.X[from];
          pred[i][r] = load_elem(a.v + from) - X[i][r];
        }
        s[r] = row_sum(X[i][r] * kz[i][r]);
      }
      if (m == 0) *reinterpret_cast<f32x4*>(part + kC + tok) = s;
    }
    // dU = P^T dh + e^(G_C - G) K Z  (upper triangular), times beta
    const __bf16* scoreT = a.ws.scoreT + at * 3 * kSquare;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const Planes<NPL> b = split<NPL>(pair(dh[2 * s], dh[2 * s + 1]));
#pragma unroll
      for (int i = 0; i < 2 * s + 2; ++i)
        kz[i] = mma_planes<3>(load_frag<3>(scoreT, kSquare, i * 2 + s, lane), b, kz[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      kz[i] *= *reinterpret_cast<const f32x4*>(decay + 2 * kC + acc_row(i, g));
    // dR
    f32x4 dR[4] = {};
    const __bf16* invT = a.ws.invT + at * 3 * kSquare;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const Planes<3> b = split<3>(pair(kz[2 * s], kz[2 * s + 1]));
#pragma unroll
      for (int i = 0; i < 2 * s + 2; ++i)
        dR[i] = mma_planes<3>(load_frag<3>(invT, kSquare, i * 2 + s, lane), b, dR[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = acc_row(i, g);
      const f32x4 e = *reinterpret_cast<const f32x4*>(decay + tok);
      f32x4 s;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        s[r] = row_sum(dR[i][r] * pred[i][r]);
        if (tok + r < valid) {
          const int64_t to = (head * a.T_len + tok0 + tok + r) * a.dv + col;
          store_elem(dv_out + to, dR[i][r]);
          if (sizeof(T) == 2) a.sv.dR[to] = dR[i][r];
        }
        dR[i][r] *= -e[r];
        dh[i][r] *= a.scale * e[r];
      }
      if (m == 0) *reinterpret_cast<f32x4*>(part + 2 * kC + tok) = s;
    }
    // Z at the chunk's start
    const float e_all = decay[kC - 1];
    const Planes<3> r0 = split<3>(pair(dR[0], dR[1])), r1 = split<3>(pair(dR[2], dR[3]));
    const Planes<3> h0 = split<3>(pair(dh[0], dh[1])), h1 = split<3>(pair(dh[2], dh[3]));
    const __bf16* keyT = a.ws.keyT + kat * NPL * kPlane;
    const __bf16* queryT = a.ws.queryT + kat * NPL * kPlane;
#pragma unroll
    for (int i = 0; i < 2 * KS; ++i) {
      Z[i] *= e_all;
      Z[i] = mma_planes<3>(load_frag<NPL>(queryT, kPlane, i * 2, lane), h0, Z[i]);
      Z[i] = mma_planes<3>(load_frag<NPL>(queryT, kPlane, i * 2 + 1, lane), h1, Z[i]);
      Z[i] = mma_planes<3>(load_frag<NPL>(keyT, kPlane, i * 2, lane), r0, Z[i]);
      Z[i] = mma_planes<3>(load_frag<NPL>(keyT, kPlane, i * 2 + 1, lane), r1, Z[i]);
    }
  }
  if (dC_out)
#pragma unroll
    for (int i = 0; i < 2 * KS; ++i)
      if (acc_row(i, g) < a.dk)
        *reinterpret_cast<f32x4*>(dC_out + (head * a.dv + col) * a.dk + acc_row(i, g)) = Z[i];
}

// planes of 8 neighbouring float32 values, scaled; zeros where off
template <int N>
__device__ inline Planes<N> load_scaled(const float* x, int64_t at, float by, bool on) {
  f32x8 v = {};
  if (on) v = *reinterpret_cast<const f32x8*>(x + at) * by;
  return split<N>(v);
}

template <typename T>
struct Grads {
  const T *q, *k, *dh;
  const float* fgate;
  const float* dR;
  Work ws;
  Saved sv;
  T *dq, *dk;
  float *dbeta, *dfgate;
  int64_t T_len;
  int chunks, NH, NHK, dk_dim, dv, ks, tiles, exp_forget;
  float scale;
};

constexpr int kPitch = kC + 1;

// writes N planes of m (or its transpose) in load order
template <int N, bool kTranspose>
__device__ inline void write_planes(const float (*m)[kPitch], __bf16* to) {
  for (int i = threadIdx.x; i < kSquare / 8; i += 64 * kWaves) {
    const int lane = i & 63, frag = i >> 6;
    const int row = (frag >> 2) * 32 + row_of((frag >> 1) & 1, lane & 15);
    const int col = (frag & 1) * 32 + (lane >> 4) * 8;
    f32x8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = kTranspose ? m[col + e][row] : m[row][col + e];
    const Planes<N> s = split<N>(v);
#pragma unroll
    for (int n = 0; n < N; ++n) *reinterpret_cast<bf16x8*>(to + n * kSquare + i * 8) = s.p[n];
  }
}

// The gradients of q, k, beta and the gates: one workgroup per key head and
// chunk, its value heads one after the other.
template <typename T>
__global__ __launch_bounds__(64 * kWaves) void delta_grads_kernel(Grads<T> a) {
  constexpr bool kBf16 = sizeof(T) == 2;
  constexpr int NPL = kBf16 ? 1 : 3;  // planes of q, k, dh
  constexpr int NPD = kBf16 ? 2 : 3;  // planes of what only dq and dk take
  __shared__ double G[kC];
  __shared__ float e0[kC], e1[kC], bt[kC], row_g[kC], col_g[kWaves][kC], col_b[kWaves][kC];
  __shared__ float inner[kWaves], mat[kC][kPitch];
  __shared__ __attribute__((aligned(16))) __bf16 planes[3][NPD * kSquare];  // B, B^T, -(N + N^T)
  const int chunk = blockIdx.x % a.chunks;
  const int64_t khead = blockIdx.x / a.chunks;
  const int group = a.NH / a.NHK;
  const int64_t tok0 = int64_t(chunk) * kC;
  const int valid = a.T_len - tok0 < kC ? int(a.T_len - tok0) : kC;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, g = lane >> 4, m = lane & 15;
  const int64_t krow0 = khead * a.T_len + tok0;
  const int64_t plane = int64_t(a.ks) * 32 * kC;

  for (int hh = 0; hh < group; ++hh) {
    const int64_t head = khead / a.NHK * a.NH + khead % a.NHK * group + hh;
    const int64_t at = head * a.chunks + chunk, row0 = head * a.T_len + tok0;
    __syncthreads();
    if (w == 0) {
      const float* decay = a.ws.decay + at * 3 * kC;
      G[lane] = chunk_decay(a.fgate + row0, lane, valid, a.exp_forget);
      e0[lane] = decay[lane];
      e1[lane] = decay[kC + lane];
      bt[lane] = decay[2 * kC + lane];
    }
    // rows 16 w ..: dh . X, dR . X, k . k, q . k
    f32x4 hx[4] = {}, rx[4] = {}, kk[4] = {}, qk[4] = {};
    const bool r_on = 16 * w + m < valid;
    for (int s = 0; s < a.dv; s += 32) {
      const int c = s + g * 8;
      const bool c_on = c < a.dv;
      const Planes<NPL> h = load_row<NPL>(a.dh, (row0 + 16 * w + m) * a.dv + c, c_on && r_on);
      const Planes<3> r = load_row<3>(a.dR, (row0 + 16 * w + m) * a.dv + c, c_on && r_on);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j <= w) {
          const Planes<3> x =
              load_row<3>(a.sv.X, (row0 + 16 * j + m) * a.dv + c, c_on && 16 * j + m < valid);
          hx[j] = mma_planes<3>(h, x, hx[j]);
          rx[j] = mma_planes<3>(r, x, rx[j]);
        }
    }
    for (int t = 0; t < a.dk_dim; t += 32) {
      const int c = t + g * 8;
      const bool c_on = c < a.dk_dim;
      const Planes<NPL> qa = load_row<NPL>(a.q, (krow0 + 16 * w + m) * a.dk_dim + c, c_on && r_on);
      const Planes<NPL> ka = load_row<NPL>(a.k, (krow0 + 16 * w + m) * a.dk_dim + c, c_on && r_on);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j <= w) {
          const Planes<NPL> kb = load_row<NPL>(a.k, (krow0 + 16 * j + m) * a.dk_dim + c,
                                               c_on && 16 * j + m < valid);
          kk[j] = mma_planes<NPL>(ka, kb, kk[j]);
          qk[j] = mma_planes<NPL>(qa, kb, qk[j]);
        }
    }
    __syncthreads();
    f32x4 rows = {};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float cg = 0.0f, cb = 0.0f;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * w + 4 * g + r, c = 16 * j + m;
        const float d = c <= row ? exp2_once(G[row] - G[c]) : 0.0f, b = bt[c];
        const float p = d * qk[j][r] * a.scale;
        mat[row][c] = c <= row ? d * b * hx[j][r] : 0.0f;
        float n = 0.0f;
        if (c <= row) cb += p * hx[j][r];
        if (c < row) {
          n = d * b * rx[j][r];
          cb -= d * rx[j][r] * kk[j][r];
          rows[r] += p * b * hx[j][r];
          cg += n * kk[j][r] - p * b * hx[j][r];
        }
        rx[j][r] = n;
      }
      cg += __shfl_xor(cg, 16, 64);
      cg += __shfl_xor(cg, 32, 64);
      cb += __shfl_xor(cb, 16, 64);
      cb += __shfl_xor(cb, 32, 64);
      if (g == 0) {
        col_g[w][16 * j + m] = cg;
        col_b[w][16 * j + m] = cb;
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float s = row_sum(rows[r]);
      if (m == 0) row_g[16 * w + 4 * g + r] = s;
    }
    __syncthreads();
    write_planes<NPD, false>(mat, planes[0]);
    write_planes<NPD, true>(mat, planes[1]);
    __syncthreads();
    // -(N + N^T): the strict lower part by its owners, then the upper by theirs
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * w + 4 * g + r, c = 16 * j + m;
        if (c < row) mat[row][c] = mat[c][row] = -rx[j][r];
        if (c == row) mat[row][c] = 0.0f;
      }
    __syncthreads();
    write_planes<NPD, false>(mat, planes[2]);
    __syncthreads();

    // 32 columns of dq and dk at a time per wave
    float dot = 0.0f;
    for (int blk = w; blk * 32 < a.dk_dim; blk += kWaves) {
      f32x4 dq[4][2] = {}, dk[4][2] = {};
      for (int s = 0; s < a.dv; s += 32) {
        Planes<NPD> S[2], Z[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int kc = blk * 32 + row_of(p, m);
          f32x8 x = {}, z = {};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int vr = s + g * 8 + e;
            if (vr < a.dv && kc < a.dk_dim) {
              x[e] = a.sv.S[(at * a.dv + vr) * a.dk_dim + kc];
              z[e] = a.sv.Z[(at * a.dv + vr) * a.dk_dim + kc];
            }
            dot += x[e] * z[e];
          }
          S[p] = split<NPD>(x);
          Z[p] = split<NPD>(z);
        }
        const int c = s + g * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = (i >> 1) * 32 + row_of(i & 1, m);
          const bool on = tok < valid && c < a.dv;
          const int64_t from = (row0 + tok) * a.dv + c;
          const Planes<NPL> h = load_row<NPL>(a.dh, from, on);
          const Planes<NPD> r = load_scaled<NPD>(a.dR, from, -e0[tok], on);
          const Planes<NPD> x = load_scaled<NPD>(a.sv.X, from, e1[tok] * bt[tok], on);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            dq[i][p] = mma_planes<NPD>(h, S[p], dq[i][p]);
            dk[i][p] = mma_planes<NPD>(r, S[p], dk[i][p]);
            dk[i][p] = mma_planes<NPD>(x, Z[p], dk[i][p]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float e = e0[acc_row(i, g) + r];
          dq[i][0][r] *= e;
          dq[i][1][r] *= e;
        }
      const __bf16* keyT = a.ws.keyT + (khead * a.chunks + chunk) * NPL * plane;
      const __bf16* queryT = a.ws.queryT + (khead * a.chunks + chunk) * NPL * plane;
      f32x4 bq[4][2] = {};
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int frag = (blk * 2 + p) * 2 + s;
          const Planes<NPL> kf = load_frag<NPL>(keyT, plane, frag, lane);
          const Planes<NPL> qf = load_frag<NPL>(queryT, plane, frag, lane);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int f = i * 2 + s;
            if (i >= 2 * s)  // B is lower triangular
              dq[i][p] =
                  mma_planes<NPD>(load_frag<NPD>(planes[0], kSquare, f, lane), kf, dq[i][p]);
            if (i < 2 * s + 2)
              bq[i][p] =
                  mma_planes<NPD>(load_frag<NPD>(planes[1], kSquare, f, lane), qf, bq[i][p]);
            dk[i][p] =
                mma_planes<NPD>(load_frag<NPD>(planes[2], kSquare, f, lane), kf, dk[i][p]);
          }
        }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int tok = acc_row(i, g) + r, kc = blk * 32 + row_of(p, m);
            if (tok >= valid || kc >= a.dk_dim) continue;
            const int64_t to = (krow0 + tok) * a.dk_dim + kc;
            float x = a.scale * dq[i][p][r], y = dk[i][p][r] + a.scale * bq[i][p][r];
            // value heads of one key head: summed in float32, by this thread
            if (hh > 0) {
              x += a.sv.dq[to];
              y += a.sv.dk[to];
            }
            if (hh + 1 < group) {
              a.sv.dq[to] = x;
              a.sv.dk[to] = y;
            } else {
              store_elem(a.dq + to, x);
              store_elem(a.dk + to, y);
            }
          }
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) dot += __shfl_xor(dot, o, 64);
    if (lane == 0) inner[w] = dot;
    __syncthreads();
    if (w == 0) {
      double dg = 0.0;
      float t1 = 0.0f, t3 = 0.0f, t2 = 0.0f;
      const float* part = a.sv.part + at * a.tiles * 3 * kC;
      for (int i = 0; i < a.tiles; ++i) {
        t1 += part[i * 3 * kC + lane];
        t3 += part[i * 3 * kC + kC + lane];
        t2 += part[i * 3 * kC + 2 * kC + lane];
      }
      float cg = 0.0f, cb = 0.0f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) {
        cg += col_g[i][lane];
        cb += col_b[i][lane];
      }
      const double s3 = double(bt[lane]) * t3;
      dg = double(t1) + row_g[lane] + cg - t2 - s3;
      // to the chunk's end: the tokens' writes and what the memory keeps
      double all = s3;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) all += __shfl_xor(all, o, 64);
      if (lane == 63)
        dg += all + double(e0[63]) * ((double(inner[0]) + inner[1]) + (double(inner[2]) + inner[3]));
      // sums from each token to the end
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const double right = __shfl_down(dg, o, 64);
        if (lane + o < 64) dg += right;
      }
      if (lane < valid) {
        const float x = a.fgate[row0 + lane];
        // d log sigma(x) = sigma(-x), from e^-|x|
        const double t = exp(-fabs(double(x)));
        a.dfgate[row0 + lane] =
            float(a.exp_forget ? dg : dg * ((x >= 0.0f ? t : 1.0) / (1.0 + t)));
        a.dbeta[row0 + lane] = cb + t3;
      }
    }
  }
}

template <typename T, int KS>
hipError_t chains(const Chain<T>& a, const float* C_in, const float* dC_in, T* dv, float* dC_out,
                  hipStream_t stream) {
  const unsigned grid = unsigned(a.H * a.per_head);
  delta_again_kernel<T, KS><<<grid, 64 * kWaves, 0, stream>>>(a, C_in);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  delta_back_kernel<T, KS><<<grid, 64 * kWaves, 0, stream>>>(a, dC_in, dv, dC_out);
  return hipGetLastError();
}

template <typename T>
hipError_t backward(const DeltaShape& s, const DeltaGrads& d, const Layout& l, const void* q,
                    const void* k, const void* v, const float* fgate, const float* C_in,
                    hipStream_t stream) {
  const int chunks = int((s.T + kC - 1) / kC), tiles = int(s.dv / 16);
  const int per_head = (tiles + kWaves - 1) / kWaves;
  const float scale = 1.0f / sqrtf(float(s.dk));
  const Chain<T> a = {static_cast<const T*>(q), static_cast<const T*>(k),
                      static_cast<const T*>(v), static_cast<const T*>(d.dh), l.ws, l.sv, s.T,
                      s.B * s.NH, chunks, int(s.NH), int(s.NHK), int(s.dk), int(s.dv), per_head,
                      tiles, scale};
  T* dv = static_cast<T*>(d.dv);
  hipError_t e = hipErrorInvalidValue;
#define MLSTM_CHAINS(KS)                                            \
  case KS:                                                          \
    e = chains<T, KS>(a, C_in, d.dC_in, dv, d.dC_out, stream);      \
    break
  switch (l.ks) {
    MLSTM_CHAINS(2);
    MLSTM_CHAINS(4);
    MLSTM_CHAINS(6);
    MLSTM_CHAINS(8);
    MLSTM_CHAINS(12);
    MLSTM_CHAINS(16);
  }
#undef MLSTM_CHAINS
  if (e != hipSuccess) return e;
  const float* dR = sizeof(T) == 2 ? l.sv.dR : static_cast<const float*>(d.dv);
  const Grads<T> b = {a.q, a.k, a.dh, fgate, dR, l.ws, l.sv, static_cast<T*>(d.dq),
                      static_cast<T*>(d.dk), d.dbeta, d.dfgate, s.T, chunks, int(s.NH),
                      int(s.NHK), int(s.dk), int(s.dv), l.ks, tiles, int(s.exp_forget), scale};
  delta_grads_kernel<T><<<unsigned(s.B * s.NHK * chunks), 64 * kWaves, 0, stream>>>(b);
  return hipGetLastError();
}

}  // namespace
}  // namespace delta

using namespace delta;

size_t delta_bwd_workspace_bytes(const DeltaShape& s) { return layout(s, true, nullptr).bytes; }

hipError_t launch_delta_bwd(const DeltaShape& s, const void* q, const void* k, const void* v,
                            const float* beta, const float* fgate, const float* C_in,
                            const DeltaGrads& d, void* workspace, hipStream_t stream) {
  const Layout l = layout(s, true, workspace);
  const hipError_t e = launch_prep(s, q, k, beta, fgate, l.ws, l.ks, true, stream);
  if (e != hipSuccess) return e;
  return s.is_bf16 ? backward<__hip_bfloat16>(s, d, l, q, k, v, fgate, C_in, stream)
                   : backward<float>(s, d, l, q, k, v, fgate, C_in, stream);
}

}  // namespace mlstm
