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
// one wave each, then 32 and 64 on the float32 matrix instruction.  Powers of At
// (the inverse as a product of I + At^(2^n)) would be fewer steps, and lose most
// digits where neighbouring keys are alike: entries grow as binomials before
// they cancel.
//
// What bounds it: memory, about 84 KiB of reads and writes per chunk of a 128
// wide bf16 head.  4096 such chunks take 88 us, 69 us at a copy's rate; a chunk
// alone takes 11 us.  Before the transposes went through the matrix unit and one
// matrix in LDS served P and At (18 KiB instead of 42, six workgroups to a CU
// instead of three) they took 122 us.
#include "delta_common.h"
#include "delta_internal.h"

namespace mlstm {
namespace delta {
namespace {

constexpr int kThreads = 256;
// floats between rows in LDS: 16-byte rows, columns without conflicts
constexpr int kPitch = kC + 4;

__device__ inline f32x4 mma_f32(float a, float b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// one 16 x 16 tile of C = A B over n columns of A, from LDS (rows kPitch apart)
template <int n>
__device__ inline f32x4 tile_product(const float* a, const float* b, int lane) {
  f32x4 c = {};
  const int m = lane & 15, g = lane >> 4;
#pragma unroll
  for (int k = 0; k < n; k += 4) c = mma_f32(a[m * kPitch + k + g], b[(k + g) * kPitch + m], c);
  return c;
}
__device__ inline void store_tile(float* to, f32x4 c, float sign, int lane) {
#pragma unroll
  for (int r = 0; r < 4; ++r) to[((lane >> 4) * 4 + r) * kPitch + (lane & 15)] = sign * c[r];
}

// Writes the planes of the lower triangular 64 x 64 matrix in LDS (or of its
// transpose) in load order: the six (row tile, half) pairs that hold something.
template <bool kTranspose>
__device__ inline void write_square(const float (*m)[kPitch], __bf16* to) {
  for (int i = threadIdx.x; i < 6 * 64; i += kThreads) {
    const int lane = i & 63;
    const int frag = kTranspose ? high_pair(i >> 6) : low_pair(i >> 6);  // 2 * row tile + half
    const int row = (frag >> 2) * 32 + row_of((frag >> 1) & 1, lane & 15);
    const int col = (frag & 1) * 32 + (lane >> 4) * 8;
    f32x8 v;
    if constexpr (kTranspose) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = col + e >= row ? m[col + e][row] : 0.0f;
    } else {
      v = pair(*reinterpret_cast<const f32x4*>(&m[row][col]),
               *reinterpret_cast<const f32x4*>(&m[row][col + 4]));
    }
    const Planes<3> s = split<3>(v);
#pragma unroll
    for (int n = 0; n < 3; ++n)
      *reinterpret_cast<bf16x8*>(to + n * kSquare + (frag * 64 + lane) * 8) = s.p[n];
  }
}

// Writes the planes of a tensor's chunk X (64 x dk) as it is, transposed, or
// both (what is NULL is left out).  The transpose is a product with columns of
// the identity, which is exact: the accumulators of two token tiles hold 8
// neighbouring tokens of a column in one lane, as K^T's left operand needs them.
template <int NPL>
__device__ inline void write_rows(const void* x, int64_t row0, int valid, int dk, int ks,
                                  __bf16* natural, __bf16* transposed) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, g = lane >> 4, m = lane & 15;
  const int64_t plane = int64_t(ks) * 32 * kC;
  bf16x8 one[2];
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int e = 0; e < 8; ++e)
      one[half][e] = static_cast<__bf16>(8 * g + e == row_of(half, m) ? 1.0f : 0.0f);
  const int s = w & 1;  // half of the tokens
  for (int t = w >> 1; t < ks; t += 2) {
    Planes<NPL> f[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int tok = s * 32 + row_of(i, m), col = t * 32 + g * 8;
      f[i] = load_row<NPL>(x, (row0 + tok) * dk + col, tok < valid && col < dk);
      if (natural)
#pragma unroll
        for (int n = 0; n < NPL; ++n)
          *reinterpret_cast<bf16x8*>(natural + n * plane +
                                     (int64_t(t * 4 + 2 * s + i) * 64 + lane) * 8) = f[i].p[n];
    }
    if (!transposed) continue;
#pragma unroll
    for (int n = 0; n < NPL; ++n)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const f32x4 a = mma(f[0].p[n], one[half], f32x4{}), b = mma(f[1].p[n], one[half], f32x4{});
        *reinterpret_cast<bf16x8*>(transposed + n * plane +
                                   (int64_t((2 * t + half) * 2 + s) * 64 + lane) * 8) =
            split<1>(pair(a, b)).p[0];
      }
  }
}

template <int NPL, bool kBackward>
__global__ __launch_bounds__(kThreads, NPL == 1 ? 6 : 4) void delta_prep_kernel(
    const void* __restrict__ q, const void* __restrict__ k, const float* __restrict__ beta,
    const float* __restrict__ fgate, Work ws, int64_t T, int chunks, int NH, int NHK, int dk,
    int ks, float scale, int exp_forget) {
  __shared__ double G[kC];
  __shared__ float bt[kC];
  __shared__ __attribute__((aligned(16))) float A[kC][kPitch];
  const int64_t head = blockIdx.x / chunks;
  const int chunk = blockIdx.x % chunks;
  const int64_t at = head * chunks + chunk;
  const int group = NH / NHK;
  const int64_t khead = head / NH * NHK + head % NH / group;
  const int64_t tok0 = int64_t(chunk) * kC;
  const int valid = T - tok0 < kC ? int(T - tok0) : kC;
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, m = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
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
#pragma unroll 2
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
            j == w ? ka
                   : load_row<NPL>(k, (row0 + 16 * j + m) * dk + col, c_on && 16 * j + m < valid);
        kk[j] = mma_planes<NPL>(ka, kb, kk[j]);
        qk[j] = mma_planes<NPL>(qa, kb, qk[j]);
      }
  }
  if (head % group == 0) {  // NH is a multiple of the group: one head per key head
    const int64_t kat = (khead * chunks + chunk) * NPL * int64_t(ks) * 32 * kC;
    write_rows<NPL>(k, row0, valid, dk, ks, NPL == 3 ? ws.key + kat : nullptr, ws.keyT + kat);
    if (NPL == 3 || kBackward)
      write_rows<NPL>(q, row0, valid, dk, ks, NPL == 3 ? ws.query + kat : nullptr,
                      kBackward ? ws.queryT + kat : nullptr);
  }
  __syncthreads();
  // P to memory through the one matrix in LDS, then At into its place
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * w + 4 * g + r, c = 16 * j + m;
      // above the diagonal by a select: no product with what is there
      const float e = c <= row ? exp2_once(G[row] - G[c]) : 0.0f;
      A[row][c] = c <= row ? e * qk[j][r] * scale : 0.0f;
      kk[j][r] = c < row ? e * kk[j][r] * bt[c] : 0.0f;
    }
  __syncthreads();
  write_square<false>(A, ws.score + at * 3 * kSquare);
  if (kBackward) write_square<true>(A, ws.scoreT + at * 3 * kSquare);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) A[16 * w + 4 * g + r][16 * j + m] = kk[j][r];
  __syncthreads();

  // 16 x 16 blocks on the diagonal: lane m holds column m of the inverse
  if (lane < 16) {
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float row[16];
#pragma unroll
      for (int j = 0; j < i; j += 4)
        *reinterpret_cast<f32x4*>(row + j) =
            *reinterpret_cast<const f32x4*>(&A[16 * w + i][16 * w + j]);
      float s = i == m ? 1.0f : 0.0f, s1 = 0.0f;  // two chains of additions
#pragma unroll
      for (int j = 0; j < i; ++j)
        if (j & 1)
          s1 -= row[j] * x[j];
        else
          s -= row[j] * x[j];
      x[i] = s + s1;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) A[16 * w + i][16 * w + m] = x[i];
  }
  __syncthreads();
  // blocks (1, 0) and (3, 2), by waves 0 and 1; the upper right block, which
  // nobody reads, takes the first product of each
  float(*tmp)[kPitch] = reinterpret_cast<float(*)[kPitch]>(&A[0][32]);
  if (w < 2)
    store_tile(&tmp[16 * w][0], tile_product<16>(&A[32 * w + 16][32 * w], &A[32 * w][32 * w], lane),
               1.0f, lane);
  __syncthreads();
  if (w < 2)
    store_tile(&A[32 * w + 16][32 * w],
               tile_product<16>(&A[32 * w + 16][32 * w + 16], &tmp[16 * w][0], lane), -1.0f, lane);
  __syncthreads();
  // the lower left 32 x 32 block, a 16 x 16 tile per wave
  {
    const int i = 16 * (w >> 1), j = 16 * (w & 1);
    store_tile(&tmp[i][j], tile_product<32>(&A[32 + i][0], &A[0][j], lane), 1.0f, lane);
    __syncthreads();
    const f32x4 c = tile_product<32>(&A[32 + i][32], &tmp[0][j], lane);
    store_tile(&A[32 + i][j], c, -1.0f, lane);  // no wave reads this block any more
  }
  __syncthreads();
  write_square<false>(A, ws.inv + at * 3 * kSquare);
  if (kBackward) write_square<true>(A, ws.invT + at * 3 * kSquare);
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
