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
// h_t = C_t q_t / sqrt(dk), 64 steps at a time.  Two waves hold the memory of 16
// value columns in their accumulators, half of its rows each, and go through
// the chunks of their head; they add their parts of K S and Q S, and take half
// of the tokens' rows of X and h each, through LDS.  The four products of a
// chunk run on the bf16 matrix instruction with float32 operands as sums of bf16
// planes (delta_common.h), three to an operand that is no bf16 input.  Two (16 bits)
// for the operands of h would take 4 to 8 % off a call with bf16 inputs, and make
// h another neighbour than the rounded float32 value's now and then (1.5e-4 in the
// 2-norm, 7e-6 as it is): not done.
//
// What bounds it: the chain.  A chunk of 128 wide heads takes a workgroup 5.0 us
// (about 9400 cycles) whatever runs beside it; of these a SIMD's vector unit is
// busy 47 %, its matrix unit 37 %, the CU's LDS 31 %, and the five barriers and
// the chain's own latencies are the rest.  8 x 16 heads of 128 x 2048 in bf16:
// 161 us for this kernel and 88 us for delta_prep.hip, 58 us being what a copy of
// the inputs and outputs takes.  Measured on the way there (with 16 bits to the
// operands of h, 145 us at the end): one wave to a value tile that loads its
// operands from memory 750 us; through an LDS ring 195 us; with copying waves of its
// own 138 us.  Two waves to a tile are 5 % slower than that there, and take 317 -> 248
// us on 8 x 4 heads of 384 x 2048, where one wave's registers spilled (above dk = 384
// two waves' do, 8 to 32 of them).  Slots enough for a whole chunk ahead change nothing there (197 us with
// 7, 195 with 3, before the copying waves).
#include "delta_forward.h"

namespace mlstm {
namespace delta {
namespace {

template <typename T, int KS, Pass kPass>
__global__ __launch_bounds__(kThreads) void delta_fwd_kernel(Chain<T> a, Segments seg,
                                                             const float* C_in, T* h,
                                                             float* C_out) {
  __shared__ __attribute__((aligned(1024))) char lds[ForwardStages<T, KS, kPass>::kShared];
  forward_chain<T, KS, kPass>(a, seg, C_in, h, C_out, blockIdx.x, lds);
}

// The memories before segments 2 ..: S' = Phi S + B, one segment after the other,
// Phi and B as the map pass left them (S' takes B's place).  A workgroup has 8
// value columns; a thread has two of 256 rows and an eighth of the sum over Phi's
// columns, so that what it reads of S from LDS serves two rows.  First it copies
// C_in, which the forward's last segment may overwrite before its first has read
// it.
constexpr int kJoinCols = 8, kJoinLanes = 128, kJoinRows = 2 * kJoinLanes, kJoinShares = kJoinCols,
              kJoinMax = int(kDeltaMaxKeyDim) / kJoinRows;
constexpr int kJoinAhead = 16;  // loads on their way at a time
template <int kMax>  // blocks of rows
__global__ __launch_bounds__(kJoinLanes * kJoinShares) void delta_join_kernel(Segments seg,
                                                                              const float* C_in,
                                                                              int dk, int dv) {
  __shared__ __attribute__((aligned(16))) float S[kDeltaMaxKeyDim][kJoinCols];
  __shared__ float part[kJoinShares][kJoinCols][kJoinRows];
  const int64_t head = blockIdx.x / (dv / kJoinCols);
  const int col0 = int(blockIdx.x % (dv / kJoinCols)) * kJoinCols;
  const int r0 = threadIdx.x % kJoinLanes, share = threadIdx.x / kJoinLanes;
  const int n = dk / kJoinShares;  // dk is a multiple of 16
  if (C_in)
    for (int i = threadIdx.x; i < kJoinCols * dk; i += kJoinLanes * kJoinShares)
      seg.start[(head * dv + col0) * dk + i] = C_in[(head * dv + col0) * dk + i];
  for (int i = threadIdx.x; i < kJoinCols * dk; i += kJoinLanes * kJoinShares)
    S[i % dk][i / dk] = seg.after(head, 0, dk, dv)[int64_t(col0 + i / dk) * dk + i % dk];
  __syncthreads();
  for (int j = 1; j + 1 < seg.n; ++j) {
    float* const map = seg.after(head, j, dk, dv);
    float x[kMax][2][kJoinCols], B[kMax][2];
#pragma unroll
    for (int p = 0; p < kMax; ++p)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int r = p * kJoinRows + q * kJoinLanes + r0;
        B[p][q] = r < dk ? map[int64_t(col0 + share) * dk + r] : 0.0f;
      }
#pragma unroll
    for (int p = 0; p < kMax; ++p) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int c = 0; c < kJoinCols; ++c) x[p][i][c] = 0.0f;
      const int r = p * kJoinRows + r0;
      if (r >= dk) continue;
      const int more = r + kJoinLanes < dk ? kJoinLanes : 0;  // without a second row: the first
      for (int k = 0; k < n; k += kJoinAhead) {
        const float* const from = map + int64_t(dv + share * n + k) * dk + r;
        float phi[kJoinAhead][2];  // all on their way before one is used
#pragma unroll
        for (int i = 0; i < kJoinAhead; ++i) {
          phi[i][0] = k + i < n ? from[i * dk] : 0.0f;
          phi[i][1] = k + i < n ? from[i * dk + more] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kJoinAhead; ++i)
          if (k + i < n) {
            float s[kJoinCols];
#pragma unroll
            for (int c = 0; c < kJoinCols; ++c) s[c] = S[share * n + k + i][c];
#pragma unroll
            for (int c = 0; c < kJoinCols; ++c) {
              x[p][0][c] += phi[i][0] * s[c];
              x[p][1][c] += phi[i][1] * s[c];
            }
          }
      }
    }
#pragma unroll
    for (int p = 0; p < kMax; ++p) {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < kJoinCols; ++c) {
        part[share][c][r0] = x[p][0][c];
        part[share][c][r0 + kJoinLanes] = x[p][1][c];
      }
      __syncthreads();
      // every share has read S: its next value, two rows of column `share` each
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int r = p * kJoinRows + q * kJoinLanes + r0;
        if (r >= dk) continue;
        float y = B[p][q];
#pragma unroll
        for (int t = 0; t < kJoinShares; ++t) y += part[t][share][q * kJoinLanes + r0];
        map[int64_t(col0 + share) * dk + r] = y;
        S[r][share] = y;
      }
    }
    __syncthreads();
  }
}

template <typename T, int KS, Pass kPass>
hipError_t launch(const DeltaShape& s, const Layout& l, const void* q, const void* k, const void* v,
                  const float* C_in, void* h, float* C_out, hipStream_t stream) {
  Chain<T> a = chain<T>(s, l, q, k, v, nullptr);
  const Segments& seg = l.seg;
  if (kPass == kMapPass) a.per_head = int((s.dv + s.dk + 63) / 64);
  const unsigned grid = unsigned(a.H * a.per_head * seg.n_of(kPass == kMapPass));
  delta_fwd_kernel<T, KS, kPass><<<grid, kThreads, 0, stream>>>(a, seg, C_in, static_cast<T*>(h),
                                                                C_out);
  return hipGetLastError();
}

template <Pass kPass>
hipError_t dispatch(const DeltaShape& s, const Layout& l, const void* q, const void* k,
                    const void* v, const float* C_in, void* h, float* C_out, hipStream_t stream) {
#define MLSTM_FWD(KS)                                                                     \
  case KS:                                                                                \
    return s.is_bf16                                                                      \
               ? launch<__hip_bfloat16, KS, kPass>(s, l, q, k, v, C_in, h, C_out, stream) \
               : launch<float, KS, kPass>(s, l, q, k, v, C_in, h, C_out, stream)
  switch (l.ks) {
    MLSTM_FWD(2);
    MLSTM_FWD(4);
    MLSTM_FWD(6);
    MLSTM_FWD(8);
    MLSTM_FWD(12);
    MLSTM_FWD(16);
  }
#undef MLSTM_FWD
  return hipErrorInvalidValue;
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
  if (l.seg.n > 1) {
    e = dispatch<kMapPass>(s, l, q, k, v, C_in, nullptr, nullptr, stream);
    if (e != hipSuccess) return e;
    const auto join =
        s.dk <= kJoinRows ? delta_join_kernel<1> : delta_join_kernel<kJoinMax>;
    join<<<unsigned(s.B * s.NH * (s.dv / kJoinCols)), kJoinLanes * kJoinShares, 0, stream>>>(
        l.seg, C_in, int(s.dk), int(s.dv));
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (C_in) C_in = l.seg.start;
  }
  return dispatch<kForward>(s, l, q, k, v, C_in, h, C_out, stream);
}

}  // namespace mlstm
