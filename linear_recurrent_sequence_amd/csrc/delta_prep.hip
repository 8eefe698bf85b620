// Gated delta rule: what a chunk of 64 tokens needs besides the memory.
//
// For each head and chunk, with G the inclusive sums of log f in the chunk
// (float64), D_ij = exp(G_i - G_j) (each exponent formed in float64 and rounded
// once, as everywhere in this library) and beta the strengths,
//
//   At_ij = D_ij (k_i . k_j) beta_j  (j < i),   P_ij = D_ij (q_i . k_j) / sqrt(dk)  (j <= i)
//
// the kernel forms (I + At)^-1 and P, and writes them as bf16 planes in the
// order in which the other kernels load them, with the transposed keys and the
// three vectors e^G, e^(G_C - G), beta.  One workgroup of four waves per chunk,
// all chunks at once.
//
// k_i . k_j and q_i . k_j run on the bf16 matrix instruction (float32 inputs:
// three planes, six products).  The inverse is by blocks, [[A, 0], [B, C]]^-1 =
// [[A^-1, 0], [-C^-1 B A^-1, C^-1]]: 16 x 16 blocks by forward substitution,
// one wave each, then 32 and 64 on the float32 matrix instruction.
#include "delta_common.h"
#include "delta_internal.h"

namespace mlstm {
namespace delta {
namespace {

constexpr int kThreads = 256;
constexpr int kPitch = kC + 1;  // floats between rows in LDS

__device__ inline f32x4 mma_f32(float a, float b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// one 16 x 16 tile of C = A B over n columns of A, from LDS (rows kPitch apart)
__device__ inline f32x4 tile_product(const float* a, const float* b, int n, int lane) {
  f32x4 c = {};
  const int m = lane & 15, g = lane >> 4;
  for (int k = 0; k < n; k += 4) c = mma_f32(a[m * kPitch + k + g], b[(k + g) * kPitch + m], c);
  return c;
}
__device__ inline void store_tile(float* to, f32x4 c, float sign, int lane) {
#pragma unroll
  for (int r = 0; r < 4; ++r) to[((lane >> 4) * 4 + r) * kPitch + (lane & 15)] = sign * c[r];
}

// Writes NP planes of the 64 x 64 matrix in LDS (or its transpose) in load order.
template <int NP, bool kTranspose>
__device__ inline void write_square(const float (*m)[kPitch], __bf16* to) {
  for (int i = threadIdx.x; i < kSquare / 8; i += kThreads) {
    const int lane = i & 63, frag = i >> 6;  // frag: [row tile][half]
    const int row = (frag >> 2) * 32 + row_of((frag >> 1) & 1, lane & 15);
    const int col = (frag & 1) * 32 + (lane >> 4) * 8;
    f32x8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = kTranspose ? m[col + e][row] : m[row][col + e];
    const Planes<NP> s = split<NP>(v);
#pragma unroll
    for (int n = 0; n < NP; ++n)
      *reinterpret_cast<bf16x8*>(to + n * kSquare + int64_t(i) * 8) = s.p[n];
  }
}

// Writes the planes of a tensor's chunk X (64 x dk) as it is, transposed, or
// both (what is NULL is left out).  `tile` holds 64 tokens of 32 columns at a time.
template <int NPL>
__device__ inline void write_rows(const void* x, int64_t row0, int valid, int dk, int ks,
                                  __bf16* natural, __bf16* transposed, float (*tile)[kPitch]) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, g = lane >> 4, m = lane & 15;
  for (int t = 0; t < ks; ++t) {
    // wave w: tokens of row tile w, 8 columns per lane
    const int tok = (w >> 1) * 32 + row_of(w & 1, m), col = t * 32 + g * 8;
    const bool on = tok < valid && col < dk;
    const Planes<NPL> s = load_row<NPL>(x, (row0 + tok) * dk + col, on);
    if (natural)
#pragma unroll
      for (int n = 0; n < NPL; ++n)
        *reinterpret_cast<bf16x8*>(natural + int64_t(n) * ks * 32 * kC +
                                   (int64_t(t * 4 + w) * 64 + lane) * 8) = s.p[n];
    if (!transposed) continue;
    // the sum of the planes is the value again
    f32x8 v = __builtin_convertvector(s.p[NPL - 1], f32x8);
#pragma unroll
    for (int n = NPL - 2; n >= 0; --n) v += __builtin_convertvector(s.p[n], f32x8);
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) tile[g * 8 + e][tok] = v[e];
    __syncthreads();
    // wave w: row tile 2 t + (w >> 1) of the transpose, half w & 1 of the tokens
    const int half = w >> 1, row = row_of(half, m), tok0 = (w & 1) * 32 + g * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = tile[row][tok0 + e];
    const Planes<NPL> u = split<NPL>(v);
#pragma unroll
    for (int n = 0; n < NPL; ++n)
      *reinterpret_cast<bf16x8*>(transposed + int64_t(n) * ks * 32 * kC +
                                 (int64_t((2 * t + half) * 2 + (w & 1)) * 64 + lane) * 8) = u.p[n];
  }
}

template <int NPL, bool kBackward>
__global__ __launch_bounds__(kThreads) void delta_prep_kernel(
    const void* __restrict__ q, const void* __restrict__ k, const float* __restrict__ beta,
    const float* __restrict__ fgate, Work ws, int64_t T, int chunks, int NH, int NHK, int dk,
    int ks, float scale, int exp_forget) {
  __shared__ double G[kC];
  __shared__ float bt[kC];
  __shared__ float A[kC][kPitch], S[kC][kPitch], tmp[32][kPitch];
  const int64_t head = blockIdx.x / chunks;
  const int chunk = blockIdx.x % chunks;
  const int64_t at = head * chunks + chunk;
  const int group = NH / NHK;
  const int64_t khead = head / NH * NHK + head % NH / group;
  const int64_t tok0 = int64_t(chunk) * kC;
  const int valid = T - tok0 < kC ? int(T - tok0) : kC;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, g = lane >> 4, m = lane & 15;
  const int64_t row0 = khead * T + tok0;

  if (w == 0) {
    const bool on = lane < valid;
    const double s = chunk_decay(fgate + head * T + tok0, lane, valid, exp_forget);
    const float b = on ? beta[head * T + tok0 + lane] : 0.0f;
    G[lane] = s;
    bt[lane] = b;
    float* v = ws.decay + at * 3 * kC;
    v[lane] = exp2_once(s);
    v[kC + lane] = exp2_once(__shfl(s, 63, 64) - s);
    v[2 * kC + lane] = b;
  }
  // wave w: rows 16 w .. of the scores
  f32x4 kk[4] = {}, qk[4] = {};
  for (int t = 0; t < ks; ++t) {
    const int col = t * 32 + g * 8;
    const bool c_on = col < dk;
    const bool r_on = c_on && 16 * w + m < valid;
    const Planes<NPL> qa = load_row<NPL>(q, (row0 + 16 * w + m) * dk + col, r_on);
    const Planes<NPL> ka = load_row<NPL>(k, (row0 + 16 * w + m) * dk + col, r_on);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j <= w) {
        const Planes<NPL> kb =
            load_row<NPL>(k, (row0 + 16 * j + m) * dk + col, c_on && 16 * j + m < valid);
        kk[j] = mma_planes<NPL>(ka, kb, kk[j]);
        qk[j] = mma_planes<NPL>(qa, kb, qk[j]);
      }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * w + 4 * g + r, c = 16 * j + m;
      // above the diagonal by a select: no product with what is there
      const float e = c <= row ? exp2_once(G[row] - G[c]) : 0.0f;
      A[row][c] = c < row ? e * kk[j][r] * bt[c] : 0.0f;
      S[row][c] = c <= row ? e * qk[j][r] * scale : 0.0f;
    }
  __syncthreads();
  constexpr int NPP = NPL == 1 && !kBackward ? 2 : 3;
  write_square<NPP, false>(S, ws.score + at * NPP * kSquare);
  if (kBackward) write_square<NPP, true>(S, ws.scoreT + at * NPP * kSquare);

  // 16 x 16 blocks on the diagonal: lane m holds column m of the inverse
  if (lane < 16) {
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == m ? 1.0f : 0.0f;
#pragma unroll
      for (int j = 0; j < i; ++j) s -= A[16 * w + i][16 * w + j] * x[j];
      x[i] = s;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) A[16 * w + i][16 * w + m] = x[i];
  }
  __syncthreads();
  // blocks (1, 0) and (3, 2), by waves 0 and 1
  if (w < 2)
    store_tile(&tmp[16 * w][0], tile_product(&A[32 * w + 16][32 * w], &A[32 * w][32 * w], 16, lane),
               1.0f, lane);
  __syncthreads();
  if (w < 2)
    store_tile(&A[32 * w + 16][32 * w],
               tile_product(&A[32 * w + 16][32 * w + 16], &tmp[16 * w][0], 16, lane), -1.0f, lane);
  __syncthreads();
  // the lower left 32 x 32 block, a 16 x 16 tile per wave
  {
    const int i = 16 * (w >> 1), j = 16 * (w & 1);
    store_tile(&tmp[i][j], tile_product(&A[32 + i][0], &A[0][j], 32, lane), 1.0f, lane);
    __syncthreads();
    const f32x4 c = tile_product(&A[32 + i][32], &tmp[0][j], 32, lane);
    __syncthreads();
    store_tile(&A[32 + i][j], c, -1.0f, lane);
  }
  __syncthreads();
  write_square<3, false>(A, ws.inv + at * 3 * kSquare);
  if (kBackward) write_square<3, true>(A, ws.invT + at * 3 * kSquare);
  if (head % group == 0) {  // NH is a multiple of the group: one head per key head
    const int64_t n = int64_t(ks) * 32 * kC, kat = (khead * chunks + chunk) * NPL * n;
    write_rows<NPL>(k, row0, valid, dk, ks, NPL == 3 ? ws.key + kat : nullptr, ws.keyT + kat, S);
    if (NPL == 3 || kBackward)
      write_rows<NPL>(q, row0, valid, dk, ks, NPL == 3 ? ws.query + kat : nullptr,
                      kBackward ? ws.queryT + kat : nullptr, S);
  }
}

}  // namespace

hipError_t launch_prep(const DeltaShape& s, const void* q, const void* k, const float* beta,
                       const float* fgate, const Work& ws, int ks, bool backward,
                       hipStream_t stream) {
  const int chunks = int((s.T + kC - 1) / kC);
  const unsigned grid = unsigned(s.B * s.NH * chunks);
  const float scale = 1.0f / sqrtf(float(s.dk));
#define MLSTM_PREP(NPL, BWD)                                                                    \
  delta_prep_kernel<NPL, BWD><<<grid, kThreads, 0, stream>>>(                                   \
      q, k, beta, fgate, ws, s.T, chunks, int(s.NH), int(s.NHK), int(s.dk), ks, scale,          \
      int(s.exp_forget))
  if (s.is_bf16) {
    if (backward)
      MLSTM_PREP(1, true);
    else
      MLSTM_PREP(1, false);
  } else {
    if (backward)
      MLSTM_PREP(3, true);
    else
      MLSTM_PREP(3, false);
  }
#undef MLSTM_PREP
  return hipGetLastError();
}

}  // namespace delta
}  // namespace mlstm
