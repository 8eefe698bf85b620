// Gated delta rule over a sequence, in chunks of 64 tokens.
//
// With S the memory at the chunk's start (dk x dv, the transpose of C), G, D,
// At and P as in delta_prep.hip, row by row of the chunk
//
//   X  = (I + At)^-1 (V - e^G K S),   U = beta X
//   h  = e^G (Q / sqrt(dk)) S + P U
//   S' = e^(G_C) S + (e^(G_C - G) K)^T U
//
// which is the recurrence C_t = f_t C_{t-1} + beta_t (v_t - f_t C_{t-1} k_t) k_t^T,
// h_t = C_t q_t / sqrt(dk), 64 steps at a time.  One wave holds the memory of 16
// value columns in its accumulators and goes through the chunks of its head;
// the four products of a chunk run on the bf16 matrix instruction with float32
// operands as sums of bf16 planes (delta_common.h).  What is rounded to fewer
// bits: for bf16 inputs the operands of h alone (S, U and P to 16 bits; h is
// then rounded to 8), never what the memory takes in.
#include "delta_common.h"
#include "delta_internal.h"

namespace mlstm {
namespace delta {
namespace {

constexpr int kWaves = 4;  // value tiles of 16 per workgroup

// T: element type of q, k, v, h.  KS: 32-column blocks of dk.
template <typename T, int KS>
__global__ __launch_bounds__(64 * kWaves) void delta_fwd_kernel(
    const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, const float* C_in,
    Work ws, T* __restrict__ h, float* C_out, int64_t T_len, int chunks, int64_t H, int NH,
    int NHK, int dk, int dv, int per_head, float scale) {
  constexpr bool kBf16 = sizeof(T) == 2;
  constexpr int NPL = kBf16 ? 1 : 3;   // planes of q and k
  constexpr int NPP = kBf16 ? 2 : 3;   // planes of P, and of S and U where h is formed
  constexpr int64_t kPlane = int64_t(KS) * 32 * kC;
  int64_t head;
  int block;
  map_head(blockIdx.x, H, per_head, head, block);
  const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
  const int col = (block * kWaves + (threadIdx.x >> 6)) * 16 + m;  // value column
  if (col >= dv) return;  // dv is a multiple of 16: whole waves; no barrier follows
  const int64_t khead = head / NH * NHK + head % NH / (NH / NHK);

  // tile 2 t + p, element r: memory row t * 32 + 8 g + 4 p + r
  f32x4 S[2 * KS];
#pragma unroll
  for (int i = 0; i < 2 * KS; ++i) {
    const int row = (i >> 1) * 32 + 8 * g + 4 * (i & 1);
    S[i] = f32x4{};
    if (C_in && row < dk)
      S[i] = *reinterpret_cast<const f32x4*>(C_in + (head * dv + col) * dk + row);
  }

  for (int chunk = 0; chunk < chunks; ++chunk) {
    const int64_t at = head * chunks + chunk, kat = khead * chunks + chunk;
    const int64_t tok0 = int64_t(chunk) * kC;
    const int valid = T_len - tok0 < kC ? int(T_len - tok0) : kC;
    const float* decay = ws.decay + at * 3 * kC;

    // K S and Q S
    f32x4 ks[4] = {}, qs[4] = {};
#pragma unroll
    for (int t = 0; t < KS; ++t) {
      const Planes<3> s = split<3>(pair(S[2 * t], S[2 * t + 1]));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        Planes<NPL> kf, qf;
        if constexpr (kBf16) {
          // rows of the inputs; those behind the end repeat the last one and
          // are dropped below
          const int tok = (i >> 1) * 32 + row_of(i & 1, m), c = t * 32 + g * 8;
          const int64_t from = (khead * T_len + tok0 + (tok < valid ? tok : valid - 1)) * dk + c;
          kf.p[0] = qf.p[0] = bf16x8{};
          if (c < dk) {
            kf.p[0] = *reinterpret_cast<const bf16x8*>(reinterpret_cast<const __bf16*>(k) + from);
            qf.p[0] = *reinterpret_cast<const bf16x8*>(reinterpret_cast<const __bf16*>(q) + from);
          }
        } else {
          kf = load_frag<NPL>(ws.key + kat * NPL * kPlane, kPlane, t * 4 + i, lane);
          qf = load_frag<NPL>(ws.query + kat * NPL * kPlane, kPlane, t * 4 + i, lane);
        }
        ks[i] = mma_planes<3>(kf, s, ks[i]);
        qs[i] = mma_planes<NPP>(qf, s, qs[i]);
      }
    }

    // R = V - e^G K S
    f32x4 R[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = (i >> 1) * 32 + 8 * g + 4 * (i & 1);
      const f32x4 e = *reinterpret_cast<const f32x4*>(decay + tok);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        R[i][r] = 0.0f;  // behind the end: nothing, whatever ks holds
        if (tok + r < valid)
          R[i][r] = load_elem(v + (head * T_len + tok0 + tok + r) * dv + col) - e[r] * ks[i][r];
      }
    }
    // X, then U = beta X
    f32x4 U[4] = {};
    {
      const __bf16* inv = ws.inv + at * 3 * kSquare;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const Planes<3> b = split<3>(pair(R[2 * s], R[2 * s + 1]));
#pragma unroll
        for (int i = 2 * s; i < 4; ++i)  // lower triangular
          U[i] = mma_planes<3>(load_frag<3>(inv, kSquare, i * 2 + s, lane), b, U[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      U[i] *= *reinterpret_cast<const f32x4*>(decay + 2 * kC + (i >> 1) * 32 + 8 * g + 4 * (i & 1));
    // h = e^G Q^ S + P U
    {
      const __bf16* score = ws.score + at * NPP * kSquare;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        qs[i] *= scale *
                 *reinterpret_cast<const f32x4*>(decay + (i >> 1) * 32 + 8 * g + 4 * (i & 1));
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const Planes<NPP> b = split<NPP>(pair(U[2 * s], U[2 * s + 1]));
#pragma unroll
        for (int i = 2 * s; i < 4; ++i)
          qs[i] = mma_planes<NPP>(load_frag<NPP>(score, kSquare, i * 2 + s, lane), b, qs[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tok = (i >> 1) * 32 + 8 * g + 4 * (i & 1);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (tok + r < valid)
            store_elem(h + (head * T_len + tok0 + tok + r) * dv + col, qs[i][r]);
      }
    }
    // S = e^(G_C) S + K^T (e^(G_C - G) U)
    const float e_all = decay[kC - 1];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      U[i] *= *reinterpret_cast<const f32x4*>(decay + kC + (i >> 1) * 32 + 8 * g + 4 * (i & 1));
    const Planes<3> u0 = split<3>(pair(U[0], U[1])), u1 = split<3>(pair(U[2], U[3]));
    const __bf16* keyT = ws.keyT + kat * NPL * kPlane;
#pragma unroll
    for (int i = 0; i < 2 * KS; ++i) {
      S[i] *= e_all;
      S[i] = mma_planes<3>(load_frag<NPL>(keyT, kPlane, i * 2, lane), u0, S[i]);
      S[i] = mma_planes<3>(load_frag<NPL>(keyT, kPlane, i * 2 + 1, lane), u1, S[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 2 * KS; ++i) {
    const int row = (i >> 1) * 32 + 8 * g + 4 * (i & 1);
    if (row < dk) *reinterpret_cast<f32x4*>(C_out + (head * dv + col) * dk + row) = S[i];
  }
}

template <typename T, int KS>
hipError_t launch(const DeltaShape& s, const void* q, const void* k, const void* v,
                  const float* C_in, const Work& ws, void* h, float* C_out, hipStream_t stream) {
  const int chunks = int((s.T + kC - 1) / kC);
  const int per_head = int((s.dv + 16 * kWaves - 1) / (16 * kWaves));
  delta_fwd_kernel<T, KS><<<unsigned(s.B * s.NH * per_head), 64 * kWaves, 0, stream>>>(
      static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v), C_in, ws,
      static_cast<T*>(h), C_out, s.T, chunks, s.B * s.NH, int(s.NH), int(s.NHK), int(s.dk),
      int(s.dv), per_head, 1.0f / sqrtf(float(s.dk)));
  return hipGetLastError();
}

}  // namespace
}  // namespace delta

using namespace delta;

size_t delta_fwd_workspace_bytes(const DeltaShape& s) { return layout(s, false, nullptr).bytes; }

hipError_t launch_delta_fwd(const DeltaShape& s, const void* q, const void* k, const void* v,
                            const float* beta, const float* fgate, const float* C_in, void* h,
                            float* C_out, void* workspace, hipStream_t stream) {
  const Layout l = layout(s, false, workspace);
  hipError_t e = launch_prep(s, q, k, beta, fgate, l.ws, l.ks, false, stream);
  if (e != hipSuccess) return e;
#define MLSTM_FWD(KS)                                                                     \
  case KS:                                                                                \
    return s.is_bf16                                                                      \
               ? launch<__hip_bfloat16, KS>(s, q, k, v, C_in, l.ws, h, C_out, stream)     \
               : launch<float, KS>(s, q, k, v, C_in, l.ws, h, C_out, stream)
  switch (l.ks) {
    MLSTM_FWD(1);
    MLSTM_FWD(2);
    MLSTM_FWD(3);
    MLSTM_FWD(4);
    MLSTM_FWD(6);
    MLSTM_FWD(8);
    MLSTM_FWD(12);
    MLSTM_FWD(16);
  }
#undef MLSTM_FWD
  return hipErrorInvalidValue;
}

}  // namespace mlstm
