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
#include "delta_internal.h"
#include "delta_ring.h"

namespace mlstm {
namespace delta {
namespace {

constexpr int kWaves = 4;  // value tiles of 16 per workgroup

// The stages of a chunk: K and Q by blocks of kT 32-column blocks, the inverse,
// the scores, K^T by kI row tiles.
template <typename T, int KS>
struct Stages {
  static constexpr bool kBf16 = sizeof(T) == 2;
  static constexpr int NPL = kBf16 ? 1 : 3;  // planes of q and k
  static constexpr int NPP = kBf16 ? 2 : 3;  // planes of P, and of S and U where h is formed
  static constexpr int kT = kBf16 ? 2 : 1, kI = kBf16 ? 8 : 4;
  static constexpr int nKQ = (KS + kT - 1) / kT, nKT = (2 * KS + kI - 1) / kI;
  static constexpr int kInv = nKQ, kScore = nKQ + 1, kKeyT = nKQ + 2, n = nKQ + 2 + nKT;
  static constexpr int kInvFrags = 18, kScoreFrags = 6 * NPP;
  static constexpr int kSlot = (kBf16 ? 20 : 24) * kFrag;
  static constexpr int kRow = 16 * kWaves * int(sizeof(T));  // bytes of a token's values
  static constexpr int kValue = kC * kRow;                   // of a chunk's
  static constexpr int kValueCopies = kValue / kFrag / kWaves;
  // at most a chunk ahead: the values and decays of two chunks have room
  static constexpr int kMost = kBf16 ? 6 : 4, kAhead = n < kMost ? n : kMost;
  static constexpr int kSlots = kAhead + 1;
  static constexpr int kShared = kSlots * kSlot + 2 * (kValue + kFrag);

  // copies of each wave in a stage
  static constexpr int copies(int s) {
    s %= n;
    if (s < nKQ) {
      const int t = KS - s * kT < kT ? KS - s * kT : kT;
      return 2 * NPL * t + (s == 0 ? kValueCopies + 1 : 0);
    }
    if (s == kInv) return (kInvFrags + kWaves - 1) / kWaves;
    if (s == kScore) return (kScoreFrags + kWaves - 1) / kWaves;
    const int i0 = (s - kKeyT) * kI, i = 2 * KS - i0 < kI ? 2 * KS - i0 : kI;
    return i * 2 * NPL / kWaves;
  }
  static constexpr int in_flight(int s) {
    int k = 0;
    for (int j = 1; j < kAhead; ++j) k += copies(s + j);
    return k;
  }
};

// T: element type of q, k, v, h.  KS: 32-column blocks of dk.
template <typename T, int KS>
__global__ __launch_bounds__(128 * kWaves, 1) void delta_fwd_kernel(
    const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, const float* C_in,
    Work ws, T* __restrict__ h, float* C_out, int64_t T_len, int chunks, int64_t H, int NH,
    int NHK, int dk, int dv, int per_head, float scale) {
  using St = Stages<T, KS>;
  constexpr int NPL = St::NPL, NPP = St::NPP;
  constexpr int64_t kPlane = int64_t(KS) * 32 * kC;
  __shared__ __attribute__((aligned(1024))) char lds[St::kShared];
  char* const values = lds + St::kSlots * St::kSlot;
  char* const decays = values + 2 * St::kValue;
  int64_t head;
  int block;
  map_head(blockIdx.x, H, per_head, head, block);
  const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
  // waves 0-3 compute, waves 4-7 copy for them
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = wave % kWaves;
  const int col = (block * kWaves + w) * 16 + m;  // value column
  const bool mine = col < dv;  // whole waves; the others keep the barriers company
  const int64_t khead = head / NH * NHK + head % NH / (NH / NHK);
  const unsigned lds0 = tilecommon::lds_addr(lds);

  // this wave's copies of stage s of a chunk into a slot
  const unsigned krow = ((w >> 1) * 32 + row_of(w & 1, m)) * dk * 2;  // row tile w (bf16)
  auto issue = [&](auto stage, int chunk, int slot) {
    constexpr int s = decltype(stage)::value;
    chunk = chunk < chunks ? chunk : chunks - 1;
    const int64_t at = head * chunks + chunk, kat = khead * chunks + chunk;
    const int64_t tok0 = int64_t(chunk) * kC;
    const int valid = T_len - tok0 < kC ? int(T_len - tok0) : kC;
    const unsigned dst = lds0 + slot * St::kSlot, lane16 = lane * 16;
    if constexpr (s == 0) {
      const unsigned to = lds0 + St::kSlots * St::kSlot + (chunk & 1) * St::kValue;
      const i32x4 from = tilecommon::rsrc_words(v + (head * T_len + tok0) * dv,
                                                int64_t(valid) * dv * sizeof(T));
      constexpr int kLanes = St::kRow / 16;  // of a token
#pragma unroll
      for (int j = 0; j < St::kValueCopies; ++j) {
        const int tok = (w * St::kValueCopies + j) * (64 / kLanes) + lane / kLanes;
        const int c = block * 16 * kWaves + lane % kLanes * (16 / int(sizeof(T)));
        copy_frag(from,
                  c < dv ? unsigned(tok * dv + c) * unsigned(sizeof(T)) : tilecommon::kOutOfRange,
                  0, to + (w * St::kValueCopies + j) * kFrag);
      }
      copy_frag(tilecommon::rsrc_words(ws.decay + at * 3 * kC, 3 * kC * 4), lane16, 0,
                lds0 + St::kSlots * St::kSlot + 2 * St::kValue + (chunk & 1) * kFrag);
    }
    if constexpr (s < St::nKQ) {
      // wave w: row tile w of K and of Q
      const int64_t bytes = int64_t(valid) * dk * 2;
#pragma unroll
      for (int t = s * St::kT; t < KS && t < (s + 1) * St::kT; ++t)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const unsigned to = dst + (((t - s * St::kT) * 2 + x) * NPL * 4 + w) * kFrag;
          if constexpr (St::kBf16) {
            const int c = t * 32 + g * 8;
            copy_frag(tilecommon::rsrc_words((x ? q : k) + (khead * T_len + tok0) * dk, bytes),
                      c < dk ? krow + c * 2 : tilecommon::kOutOfRange, 0, to);
          } else {
#pragma unroll
            for (int p = 0; p < NPL; ++p)
              copy_frag(
                  tilecommon::rsrc_words((x ? ws.query : ws.key) + (kat * NPL + p) * kPlane,
                                         kPlane * 2),
                  lane16, (t * 4 + w) * kFrag, to + p * 4 * kFrag);
          }
        }
    } else if constexpr (s < St::kKeyT) {
      constexpr int np = s == St::kInv ? 3 : NPP, frags = 6 * np;
      const i32x4 from = tilecommon::rsrc_words(
          (s == St::kInv ? ws.inv : ws.score) + at * np * kSquare, np * kSquare * 2);
#pragma unroll
      for (int j = 0; j < (frags + kWaves - 1) / kWaves; ++j) {
        const int f = j * kWaves + w < frags ? j * kWaves + w : frags - 1;
        copy_frag(from, lane16, f / 6 * (kSquare * 2) + low_pair(f % 6) * kFrag,
                  dst + (j * kWaves + w) * kFrag);
      }
    } else {
      constexpr int i0 = (s - St::kKeyT) * St::kI;
      constexpr int frags = (2 * KS - i0 < St::kI ? 2 * KS - i0 : St::kI) * 2;  // of a plane
#pragma unroll
      for (int p = 0; p < NPL; ++p)
#pragma unroll
        for (int j = 0; j < frags / kWaves; ++j)
          copy_frag(tilecommon::rsrc_words(ws.keyT + (kat * NPL + p) * kPlane, kPlane * 2), lane16,
                    (i0 * 2 + j * kWaves + w) * kFrag,
                    dst + (p * St::kI * 2 + j * kWaves + w) * kFrag);
    }
  };

  if (wave >= kWaves) {
    static_for<St::kAhead>(
        [&](auto s) { issue(std::integral_constant<int, s % St::n>{}, s / St::n, s); });
    int slot = St::kAhead;
    for (int chunk = 0; chunk < chunks; ++chunk)
      static_for<St::n>([&](auto stage) {
        constexpr int s = decltype(stage)::value, next = s + St::kAhead;
        stage_barrier<St::in_flight(s)>();
        issue(std::integral_constant<int, next % St::n>{}, chunk + next / St::n, slot);
        slot = slot + 1 == St::kSlots ? 0 : slot + 1;
      });
    // no copy may be in flight into LDS that another workgroup gets
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    return;
  }

  // tile 2 t + p, element r: memory row t * 32 + 8 g + 4 p + r
  f32x4 S[2 * KS];
#pragma unroll
  for (int i = 0; i < 2 * KS; ++i) {
    const int row = (i >> 1) * 32 + 8 * g + 4 * (i & 1);
    S[i] = f32x4{};
    if (C_in && mine && row < dk)
      S[i] = *reinterpret_cast<const f32x4*>(C_in + (head * dv + col) * dk + row);
  }

  int read = 0;  // the slot of the stage at hand
  auto enter = [&]() {
    join_barrier();
    const char* slot = lds + read * St::kSlot;
    read = read + 1 == St::kSlots ? 0 : read + 1;
    return slot;
  };

  for (int chunk = 0; chunk < chunks; ++chunk) {
    const int64_t tok0 = int64_t(chunk) * kC;
    const int valid = T_len - tok0 < kC ? int(T_len - tok0) : kC;
    const float* decay = reinterpret_cast<const float*>(decays + (chunk & 1) * kFrag);
    const T* value = reinterpret_cast<const T*>(values + (chunk & 1) * St::kValue);

    // K S and Q S
    f32x4 ks[4] = {}, qs[4] = {};
    static_for<St::nKQ>([&](auto stage) {
      constexpr int s = decltype(stage)::value;
      const char* slot = enter();
#pragma unroll
      for (int t = s * St::kT; t < KS && t < (s + 1) * St::kT; ++t) {
        const Planes<3> b = split<3>(pair(S[2 * t], S[2 * t + 1]));
        const char* at = slot + (t - s * St::kT) * 2 * NPL * 4 * kFrag;
        Planes<NPL> kf[4], qf[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) kf[i] = lds_frag<NPL>(at, i, 4, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) qf[i] = lds_frag<NPL>(at, NPL * 4 + i, 4, lane);
        each_product<3, NPL, 3>([&](int x, int y) {
#pragma unroll
          for (int i = 0; i < 4; ++i) ks[i] = mma(kf[i].p[x], b.p[y], ks[i]);
        });
        each_product<NPP, NPL, 3>([&](int x, int y) {
#pragma unroll
          for (int i = 0; i < 4; ++i) qs[i] = mma(qf[i].p[x], b.p[y], qs[i]);
        });
      }
    });

    // R = V - e^G K S
    f32x4 R[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = (i >> 1) * 32 + 8 * g + 4 * (i & 1);
      const f32x4 e = *reinterpret_cast<const f32x4*>(decay + tok);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float x = load_elem(value + (tok + r) * 16 * kWaves + w * 16 + m) - e[r] * ks[i][r];
        R[i][r] = tok + r < valid ? x : 0.0f;  // behind the end: nothing, whatever the memory holds
      }
      qs[i] *= scale * e;
    }
    // X, then U = beta X
    f32x4 U[4] = {};
    {
      const char* slot = enter();
      low_product<3>(slot, R, U, lane);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      U[i] *= *reinterpret_cast<const f32x4*>(decay + 2 * kC + (i >> 1) * 32 + 8 * g + 4 * (i & 1));
    // h = e^G Q^ S + P U
    {
      const char* slot = enter();
      low_product<NPP>(slot, U, qs, lane);
      if (mine)
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
    static_for<St::nKT>([&](auto stage) {
      constexpr int j = decltype(stage)::value;
      const char* slot = enter();
      constexpr int i0 = j * St::kI, n = 2 * KS - i0 < St::kI ? 2 * KS - i0 : St::kI;
#pragma unroll
      for (int i = i0; i < i0 + n; ++i) S[i] *= e_all;
      // four tiles at a time
#pragma unroll
      for (int f = 0; f < n; f += 4) {
        Planes<NPL> a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4 && f + i < n; ++i) {
          a[i] = lds_frag<NPL>(slot, 2 * (f + i), St::kI * 2, lane);
          b[i] = lds_frag<NPL>(slot, 2 * (f + i) + 1, St::kI * 2, lane);
        }
        each_product<3, NPL, 3>([&](int x, int y) {
#pragma unroll
          for (int i = 0; i < 4 && f + i < n; ++i) S[i0 + f + i] = mma(a[i].p[x], u0.p[y], S[i0 + f + i]);
#pragma unroll
          for (int i = 0; i < 4 && f + i < n; ++i) S[i0 + f + i] = mma(b[i].p[x], u1.p[y], S[i0 + f + i]);
        });
      }
    });
  }
  if (mine)
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
  delta_fwd_kernel<T, KS><<<unsigned(s.B * s.NH * per_head), 128 * kWaves, 0, stream>>>(
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
