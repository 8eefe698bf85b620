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
// of the tokens' rows of X and h each, through LDS.  The four products of a chunk run on the bf16 matrix instruction with float32
// operands as sums of bf16 planes (delta_common.h).  What is rounded to fewer
// bits: for bf16 inputs the operands of h alone (S, U and P to 16 bits; h is
// then rounded to 8), never what the memory takes in.
#include "delta_internal.h"
#include "delta_ring.h"

namespace mlstm {
namespace delta {
namespace {

constexpr int kWaves = 4;  // value tiles of 16 per workgroup

constexpr int kChainWaves = 2 * kWaves;            // two to a value tile
constexpr int kThreads = 64 * (kChainWaves + kWaves);  // and four that copy

// The stages of a chunk.  The two waves of a value tile hold one half each of
// the memory's rows (KS tiles), so a stage of K and Q (float32: of K, then of
// Q) and one of K^T serve both halves.
template <typename T, int KS>
struct Stages {
  static constexpr bool kBf16 = sizeof(T) == 2;
  static constexpr int NPL = kBf16 ? 1 : 3;  // planes of q and k
  static constexpr int NPP = kBf16 ? 2 : 3;  // planes of P, and of S and U where h is formed
  static constexpr int kI = kBf16 ? 4 : 2;   // row tiles of K^T for each half
  static constexpr int nKQ = kBf16 ? KS / 2 : KS, nKT = (KS + kI - 1) / kI;
  static constexpr int kInv = nKQ, kScore = nKQ + 1, kKeyT = nKQ + 2, n = nKQ + 2 + nKT;
  static constexpr int kInvFrags = 18, kScoreFrags = 6 * NPP;
  static constexpr int kSlot = (kBf16 ? 20 : 24) * kFrag;
  static constexpr int kRow = 16 * kWaves * int(sizeof(T));  // bytes of a token's values
  static constexpr int kPad = kRow / 4;                      // after 8 tokens: no bank conflicts
  static constexpr int kValue = kC * kRow + kC / 8 * kPad;   // of a chunk's values
  static constexpr int kValueCopies = kC * kRow / kFrag / kWaves;
  // at most a chunk ahead: the values and decays of two chunks have room
  static constexpr int kMost = kBf16 ? 4 : 2, kAhead = n < kMost ? n : kMost;
  static constexpr int kSlots = kAhead + 1;
  static constexpr int kPart = 10 * kFrag;  // a value tile's sums between its two waves
  static constexpr int kValueAt = kSlots * kSlot, kDecayAt = kValueAt + 2 * kValue,
                       kPartAt = kDecayAt + 2 * kFrag, kShared = kPartAt + kWaves * kPart;

  static constexpr int tiles_of(int s) {  // of K^T, for each half
    return KS - (s - kKeyT) * kI < kI ? KS - (s - kKeyT) * kI : kI;
  }
  // copies of each copying wave in a stage
  static constexpr int copies(int s) {
    s %= n;
    if (s < nKQ) return (kBf16 ? 4 : 6) + (s == 0 ? kValueCopies + 1 : 0);
    if (s == kInv) return (kInvFrags + kWaves - 1) / kWaves;
    if (s == kScore) return (kScoreFrags + kWaves - 1) / kWaves;
    return tiles_of(s) * NPL;
  }
  static constexpr int in_flight(int s) {
    int k = 0;
    for (int j = 1; j < kAhead; ++j) k += copies(s + j);
    return k;
  }
  // a token's values in LDS
  static __device__ int value_at(int tok) { return tok * kRow + (tok >> 3) * kPad; }
};

// T: element type of q, k, v, h.  KS: 32-column blocks of dk (even).
template <typename T, int KS>
__global__ __launch_bounds__(kThreads) void delta_fwd_kernel(
    const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, const float* C_in,
    Work ws, T* __restrict__ h, float* C_out, int64_t T_len, int chunks, int64_t H, int NH,
    int NHK, int dk, int dv, int per_head, float scale) {
  using St = Stages<T, KS>;
  constexpr int NPL = St::NPL, NPP = St::NPP;
  constexpr int64_t kPlane = int64_t(KS) * 32 * kC;
  __shared__ __attribute__((aligned(1024))) char lds[St::kShared];
  int64_t head;
  int block;
  map_head(blockIdx.x, H, per_head, head, block);
  const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t khead = head / NH * NHK + head % NH / (NH / NHK);

  if (wave >= kChainWaves) {
    // ------------------------------------------------------ the copying waves
    const int w = wave - kChainWaves;
    const unsigned lds0 = tilecommon::lds_addr(lds), lane16 = lane * 16;
    const unsigned krow = ((w >> 1) * 32 + row_of(w & 1, m)) * dk * 2;  // row tile w (bf16)
    // this wave's copies of stage s of a chunk into a slot
    auto issue = [&](auto stage, int chunk, int slot) {
      constexpr int s = decltype(stage)::value;
      // behind the last chunk: its data again, into the buffers of the one after
      const int side = chunk & 1;
      chunk = chunk < chunks ? chunk : chunks - 1;
      const int64_t at = head * chunks + chunk, kat = khead * chunks + chunk;
      const int64_t tok0 = int64_t(chunk) * kC;
      const int valid = T_len - tok0 < kC ? int(T_len - tok0) : kC;
      const unsigned dst = lds0 + slot * St::kSlot;
      if constexpr (s == 0) {
        const i32x4 from = tilecommon::rsrc_words(v + (head * T_len + tok0) * dv,
                                                  int64_t(valid) * dv * sizeof(T));
        constexpr int kLanes = St::kRow / 16;  // of a token
#pragma unroll
        for (int j = 0; j < St::kValueCopies; ++j) {
          const int first = (w * St::kValueCopies + j) * (64 / kLanes);  // token
          const int c = block * 16 * kWaves + lane % kLanes * (16 / int(sizeof(T)));
          copy_frag(from,
                    c < dv ? unsigned((first + lane / kLanes) * dv + c) * unsigned(sizeof(T))
                           : tilecommon::kOutOfRange,
                    0, lds0 + St::kValueAt + side * St::kValue + St::value_at(first));
        }
        copy_frag(tilecommon::rsrc_words(ws.decay + at * 3 * kC, 3 * kC * 4), lane16, 0,
                  lds0 + St::kDecayAt + side * kFrag);
      }
      if constexpr (s < St::nKQ) {
        // wave w: row tile w, for both halves
        const int64_t bytes = int64_t(valid) * dk * 2;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if constexpr (St::kBf16) {
            const int t = half * (KS / 2) + s, c = t * 32 + g * 8;
#pragma unroll
            for (int x = 0; x < 2; ++x)
              copy_frag(tilecommon::rsrc_words((x ? q : k) + (khead * T_len + tok0) * dk, bytes),
                        c < dk ? krow + c * 2 : tilecommon::kOutOfRange, 0,
                        dst + ((half * 2 + x) * 4 + w) * kFrag);
          } else {
            const int t = half * (KS / 2) + s / 2;
#pragma unroll
            for (int p = 0; p < NPL; ++p)
              copy_frag(tilecommon::rsrc_words(
                            (s % 2 ? ws.query : ws.key) + (kat * NPL + p) * kPlane, kPlane * 2),
                        lane16, (t * 4 + w) * kFrag, dst + ((half * NPL + p) * 4 + w) * kFrag);
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
        // wave w: half w & 1 of the tokens, of every tile of half w >> 1 of the rows
        constexpr int i0 = (s - St::kKeyT) * St::kI, tiles = St::tiles_of(s);
#pragma unroll
        for (int p = 0; p < NPL; ++p)
#pragma unroll
          for (int i = 0; i < tiles; ++i)
            copy_frag(
                tilecommon::rsrc_words(ws.keyT + (kat * NPL + p) * kPlane, kPlane * 2), lane16,
                (((w >> 1) * KS + i0 + i) * 2 + (w & 1)) * kFrag,
                dst + (((p * 2 + (w >> 1)) * St::kI + i) * 2 + (w & 1)) * kFrag);
      }
    };
    static_for<St::kAhead>(
        [&](auto s) { issue(std::integral_constant<int, s % St::n>{}, s / St::n, s); });
    int slot = St::kAhead;
    for (int chunk = 0; chunk < chunks; ++chunk)
      static_for<St::n>([&](auto stage) {
        constexpr int s = decltype(stage)::value, next = s + St::kAhead;
        stage_barrier<St::in_flight(s)>();
        issue(std::integral_constant<int, next % St::n>{}, chunk + next / St::n, slot);
        slot = slot + 1 == St::kSlots ? 0 : slot + 1;
        if constexpr (s == St::kKeyT) {
          // h is where the chunk's values were: 16 bytes a lane to memory
          constexpr int kLanes = St::kRow / 16;
          const int64_t tok0 = int64_t(chunk) * kC;
          const int valid = T_len - tok0 < kC ? int(T_len - tok0) : kC;
#pragma unroll
          for (int j = 0; j < St::kValueCopies; ++j) {
            const int tok = (w * St::kValueCopies + j) * (64 / kLanes) + lane / kLanes;
            const int c = block * 16 * kWaves + lane % kLanes * (16 / int(sizeof(T)));
            const uint4 x = *reinterpret_cast<const uint4*>(
                lds + St::kValueAt + (chunk & 1) * St::kValue + St::value_at(tok) +
                lane % kLanes * 16);
            if (tok < valid && c < dv)
              *reinterpret_cast<uint4*>(h + (head * T_len + tok0 + tok) * dv + c) = x;
          }
        }
      });
    // no copy may be in flight into LDS that another workgroup gets
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    return;
  }

  // ---------------------------------------------------------- the chain's waves
  const int tile = wave % kWaves, half = wave / kWaves;
  const int col = (block * kWaves + tile) * 16 + m;  // value column
  const bool mine = col < dv;  // whole waves; the others keep the barriers company
  // tile 2 t + p of this half, element r: memory row (half * KS / 2 + t) * 32 + 8 g + 4 p + r
  const int row0 = half * KS * 16 + 8 * g;
  f32x4 S[KS];
#pragma unroll
  for (int i = 0; i < KS; ++i) {
    const int row = row0 + (i >> 1) * 32 + 4 * (i & 1);
    S[i] = f32x4{};
    if (C_in && mine && row < dk)
      S[i] = *reinterpret_cast<const f32x4*>(C_in + (head * dv + col) * dk + row);
  }
  // to the first half's wave: K S and Q S of tokens 0-31 (four fragments); to
  // the second's: K S of all, Q S of tokens 32-63 (six).  What a wave has read
  // it overwrites with its X, for the other one.
  f32x4* const to_first = reinterpret_cast<f32x4*>(lds + St::kPartAt + tile * St::kPart) + lane;
  f32x4* const to_second = to_first + 4 * 64;

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
    const float* decay = reinterpret_cast<const float*>(lds + St::kDecayAt + (chunk & 1) * kFrag);
    char* value = lds + St::kValueAt + (chunk & 1) * St::kValue;
    auto value_of = [&](int tok) {
      return reinterpret_cast<T*>(value + St::value_at(tok)) + tile * 16 + m;
    };

    // K S and Q S over this half's rows
    f32x4 ks[4] = {}, qs[4] = {};
    static_for<KS / 2>([&](auto block_t) {
      constexpr int t = decltype(block_t)::value;
      Planes<NPL> kf[4], qf[4];
      const char* slot = enter() + half * (St::kBf16 ? 8 : NPL * 4) * kFrag;
#pragma unroll
      for (int i = 0; i < 4; ++i) kf[i] = lds_frag<NPL>(slot, i, 4, lane);
      if constexpr (St::kBf16)
#pragma unroll
        for (int i = 0; i < 4; ++i) qf[i] = lds_frag<NPL>(slot, 4 + i, 4, lane);
      const Planes<3> b = split<3>(pair(S[2 * t], S[2 * t + 1]));
      each_product<3, NPL, 3>([&](int x, int y) {
#pragma unroll
        for (int i = 0; i < 4; ++i) ks[i] = mma(kf[i].p[x], b.p[y], ks[i]);
      });
      if constexpr (!St::kBf16) {
        slot = enter() + half * NPL * 4 * kFrag;
#pragma unroll
        for (int i = 0; i < 4; ++i) qf[i] = lds_frag<NPL>(slot, i, 4, lane);
      }
      each_product<NPP, NPL, 3>([&](int x, int y) {
#pragma unroll
        for (int i = 0; i < 4; ++i) qs[i] = mma(qf[i].p[x], b.p[y], qs[i]);
      });
    });
    if (half == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) to_second[i * 64] = ks[i];
      to_second[4 * 64] = qs[2];
      to_second[5 * 64] = qs[3];
    } else {
      to_first[0] = ks[0];
      to_first[64] = ks[1];
      to_first[2 * 64] = qs[0];
      to_first[3 * 64] = qs[1];
    }

    // R = V - e^G K S of token tile i, from the sum of the halves
    auto rest = [&](int i, f32x4 ks) {
      const int tok = (i >> 1) * 32 + 8 * g + 4 * (i & 1);
      const f32x4 e = *reinterpret_cast<const f32x4*>(decay + tok);
      f32x4 R;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float x = load_elem(value_of(tok + r)) - e[r] * ks[r];
        R[r] = tok + r < valid ? x : 0.0f;  // behind the end: nothing, whatever the memory holds
      }
      return R;
    };
    auto at_tile = [&](int what, int i) {
      return *reinterpret_cast<const f32x4*>(decay + what * kC + (i >> 1) * 32 + 8 * g +
                                             4 * (i & 1));
    };
    // X (first half: tokens 0-31, second: 32-63), exchanged; then U = beta X
    f32x4 U[4], hs[2];
    {
      const char* slot = enter();
      f32x4 x0 = {}, x1 = {};
      if (half == 0) {
        Planes<3> a[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) a[i] = lds_frag<3>(slot, i, 6, lane);
        const f32x4 r0 = rest(0, ks[0] + to_first[0]), r1 = rest(1, ks[1] + to_first[64]);
        hs[0] = qs[0] + to_first[2 * 64];
        hs[1] = qs[1] + to_first[3 * 64];
        const Planes<3> b = split<3>(pair(r0, r1));
        each_product<3, 3, 3>([&](int i, int j) {
          x0 = mma(a[0].p[i], b.p[j], x0);
          x1 = mma(a[1].p[i], b.p[j], x1);
        });
        to_first[0] = x0;
        to_first[64] = x1;
      } else {
        Planes<3> a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = lds_frag<3>(slot, 2 + i, 6, lane);
        f32x4 R[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) R[i] = rest(i, ks[i] + to_second[i * 64]);
        hs[0] = qs[2] + to_second[4 * 64];
        hs[1] = qs[3] + to_second[5 * 64];
        const Planes<3> b0 = split<3>(pair(R[0], R[1])), b1 = split<3>(pair(R[2], R[3]));
        f32x4 y0 = {}, y1 = {};
        each_product<3, 3, 3>([&](int i, int j) {
          x0 = mma(a[0].p[i], b0.p[j], x0);
          x1 = mma(a[2].p[i], b0.p[j], x1);
          y0 = mma(a[1].p[i], b1.p[j], y0);
          y1 = mma(a[3].p[i], b1.p[j], y1);
        });
        x0 += y0;
        x1 += y1;
        to_second[0] = x0;
        to_second[64] = x1;
      }
      U[2] = x0;  // placed below
      U[3] = x1;
    }
    // h = e^G Q^ S + P U, for this wave's tokens
    {
      const char* slot = enter();
      Planes<NPP> a[4];
      if (half == 0) {
        U[0] = U[2];
        U[1] = U[3];
        U[2] = to_second[0];
        U[3] = to_second[64];
#pragma unroll
        for (int i = 0; i < 2; ++i) a[i] = lds_frag<NPP>(slot, i, 6, lane);
      } else {
        U[0] = to_first[0];
        U[1] = to_first[64];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = lds_frag<NPP>(slot, 2 + i, 6, lane);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) U[i] *= at_tile(2, i);
      hs[0] *= scale * at_tile(0, 2 * half);
      hs[1] *= scale * at_tile(0, 2 * half + 1);
      const Planes<NPP> b0 = split<NPP>(pair(U[0], U[1]));
      if (half == 0) {
        each_product<NPP, NPP, NPP>([&](int i, int j) {
          hs[0] = mma(a[0].p[i], b0.p[j], hs[0]);
          hs[1] = mma(a[1].p[i], b0.p[j], hs[1]);
        });
      } else {
        const Planes<NPP> b1 = split<NPP>(pair(U[2], U[3]));
        f32x4 y0 = {}, y1 = {};
        each_product<NPP, NPP, NPP>([&](int i, int j) {
          hs[0] = mma(a[0].p[i], b0.p[j], hs[0]);
          hs[1] = mma(a[2].p[i], b0.p[j], hs[1]);
          y0 = mma(a[1].p[i], b1.p[j], y0);
          y1 = mma(a[3].p[i], b1.p[j], y1);
        });
        hs[0] += y0;
        hs[1] += y1;
      }
      // to where the values were; the copying waves store it
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          store_elem(value_of(half * 32 + 8 * g + 4 * i + r), hs[i][r]);
    }
    // S = e^(G_C) S + K^T (e^(G_C - G) U)
    const float e_all = decay[kC - 1];
#pragma unroll
    for (int i = 0; i < 4; ++i) U[i] *= at_tile(1, i);
    const Planes<3> u0 = split<3>(pair(U[0], U[1])), u1 = split<3>(pair(U[2], U[3]));
    static_for<St::nKT>([&](auto stage) {
      constexpr int j = decltype(stage)::value, n = St::tiles_of(St::kKeyT + j);
      const char* slot = enter() + half * St::kI * 2 * kFrag;
      Planes<NPL> a[n], b[n];
#pragma unroll
      for (int i = 0; i < n; ++i) {
        a[i] = lds_frag<NPL>(slot, 2 * i, St::kI * 4, lane);
        b[i] = lds_frag<NPL>(slot, 2 * i + 1, St::kI * 4, lane);
        S[j * St::kI + i] *= e_all;
      }
      each_product<3, NPL, 3>([&](int x, int y) {
#pragma unroll
        for (int i = 0; i < n; ++i)
          S[j * St::kI + i] = mma(a[i].p[x], u0.p[y], S[j * St::kI + i]);
#pragma unroll
        for (int i = 0; i < n; ++i)
          S[j * St::kI + i] = mma(b[i].p[x], u1.p[y], S[j * St::kI + i]);
      });
    });
  }
  if (mine)
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      const int row = row0 + (i >> 1) * 32 + 4 * (i & 1);
      if (row < dk) *reinterpret_cast<f32x4*>(C_out + (head * dv + col) * dk + row) = S[i];
    }
}

template <typename T, int KS>
hipError_t launch(const DeltaShape& s, const void* q, const void* k, const void* v,
                  const float* C_in, const Work& ws, void* h, float* C_out, hipStream_t stream) {
  const int chunks = int((s.T + kC - 1) / kC);
  const int per_head = int((s.dv + 16 * kWaves - 1) / (16 * kWaves));
  delta_fwd_kernel<T, KS><<<unsigned(s.B * s.NH * per_head), kThreads, 0, stream>>>(
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

}  // namespace mlstm
