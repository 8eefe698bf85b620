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
//   dlog f_t = sum_(i>=t) (e^(G_i) dh_i . (S^T q^_i) - dR_i . Y_i)
//              + sum_(j<t) e^(G_C - G_j) U_j . (Z^T k_j) + e^(G_C) <S, Z>
//              + sum_(i>=t>j) (P_ij (dh_i . U_j) - N_ij (k_i . k_j)),   Y_i = e^(G_i) S^T k_i:
//
// what passes from before token t to behind it, and so has f_t as a factor in
// every term.  (As the sum of dL/dG from t to the chunk's end it would be a
// difference of terms without f_t, and noise where f_t is small.)  No sum is longer
// than a chunk.
//
// Six passes: the terms that all columns share (delta_prep.hip), the memory
// forward once more (delta_forward.h; its start, X and Y of every chunk are kept,
// float32), the gradient of the memory backward (Z and dR kept), and, over all
// chunks at once, the pairs of tokens, the gradients of q and k, and those of beta
// and the gates.  The two chains need each other only for sums of X with Z^T k
// and of dR with Y, and run in one launch where the card holds both (side_by_side).
// Everything that the gradients come from has float32 accuracy (three bf16 planes to
// an operand that is no bf16 input); for bf16 inputs dq, dk and dv are rounded once,
// at the end.
//
// What bounds it: the memories, 8 dk dv bytes per head and chunk, written by the
// chains and read once by the key gradients.  On 8 x 4 heads of 384 x 2048 in
// bf16: chunk terms 83 us, the chains 459 and 429, pairs 116, key gradients 436,
// gates 8; the 1.2 GB of memories alone are 240 us each way at a copy's rate.
// Stored all at once at a chunk's start the memories stood 7 us in the way of each
// chunk; and a chain's wave that loads from memory waits for its own stores first,
// so V, X, Y and dh come through LDS (bf16), which took the chains from 630 to 460
// us.  A chain's waves hold the memory in registers, and spill up to 20 of them for dk
// of 257 to 384 and up to 62 above; in float32 (more planes on the way) up to 24
// from dk = 65 on, 64 above 256 and 170 above 384.
#include "delta_forward.h"

namespace mlstm {
namespace delta {
namespace {

// The stages of a chunk: P^T, K by blocks for both halves of the memory's rows,
// (I + At)^-T, then Q^T and K^T by row tiles.
// kApart: without X and Y, as it has to be beside the memory's pass.
template <typename T, int KS, bool kApart>
struct BackStages {
  static constexpr bool kBf16 = sizeof(T) == 2;
  static constexpr int NPL = kBf16 ? 1 : 3;  // planes of q, k and dh
  static constexpr int kT = kBf16 ? 2 : 1;   // 32-column blocks of K for each half
  static constexpr int kI = kBf16 ? 4 : 2;   // row tiles of Q^T or K^T for each half
  static constexpr int nK = (KS / 2 + kT - 1) / kT, nT = (KS + kI - 1) / kI;
  static constexpr int kInv = 1 + nK, kQueryT = kInv + 1, kKeyT = kQueryT + nT, n = kKeyT + nT;
  static constexpr int kSlot = (kBf16 ? 20 : 24) * kFrag;
  // X and Y come through LDS, with the inverse (a wave that stores and then loads
  // waits for its stores); one buffer each, so less than a chunk ahead
  static constexpr bool kStaged = !kApart;
  static_assert(kApart || kBf16, "float32: LDS is full");
  static constexpr int kMost = kBf16 ? 3 : 2;
  static constexpr int kAhead = n - kStaged < kMost ? n - kStaged : kMost;
  static constexpr int kSlots = kAhead + 1;
  static constexpr int kPart = 6 * kFrag;  // a value tile's sums between its two waves
  static constexpr int kValueAt = kSlots * kSlot, kDecayAt = kValueAt + 2 * Values<T>::kBytes,
                       kPartAt = kDecayAt + 2 * kFrag, kXAt = kPartAt + kWaves * kPart,
                       kYAt = kXAt + (kStaged ? Values<float>::kBytes : 0),
                       kShared = kYAt + (kStaged ? Values<float>::kBytes : 0);

  static constexpr int blocks_of(int s) {  // of K, for each half
    return KS / 2 - (s - 1) * kT < kT ? KS / 2 - (s - 1) * kT : kT;
  }
  static constexpr int tiles_of(int j) { return KS - j * kI < kI ? KS - j * kI : kI; }
  static constexpr int copies(int s) {
    s %= n;
    if (s == 0) return Copier::square_copies(3) + Values<T>::kCopies + 1;
    if (s < kInv) return 2 * NPL * blocks_of(s);
    if (s == kInv)
      return Copier::square_copies(3) +
             (kStaged ? 2 * Values<float>::kCopies : 0);
    return tiles_of((s - kQueryT) % nT) * NPL;
  }
  static constexpr int in_flight(int s) {
    int k = 0;
    for (int j = 1; j < kAhead; ++j) k += copies(s + j);
    return k;
  }
};

// The memory's gradient backward: Z at each chunk's end, dR (and dV), and the
// parts X . (e^(G_C - G) Z^T k) and dR . Y that each 16 columns give (kApart:
// e^(G_C - G) Z^T k itself, from which delta_pairs_kernel forms them).
// Built as the forward is (delta_forward.h): the operands are upper triangular
// here, so the first half's wave takes what the second's does there.
template <typename T, int KS, bool kApart>
__device__ inline void back_chain(const Chain<T>& a, const float* dC_in, T* dv_out, float* dC_out,
                                  int64_t wg, char* lds) {
  using St = BackStages<T, KS, kApart>;
  using V = Values<T>;
  constexpr int NPL = St::NPL;
  constexpr int64_t kPlane = int64_t(KS) * 32 * kC;
  int64_t head;
  int block;
  map_head(wg, a.H, a.per_head, head, block);
  const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t khead = head / a.NH * a.NHK + head % a.NH / (a.NH / a.NHK);
  const int chunks = a.chunks, dk = a.dk, dv = a.dv;

  if (wave >= kChainWaves) {
    const Copier cp = {wave - kChainWaves, lane, tilecommon::lds_addr(lds)};
    // `turn` counts chunks from the last one
    auto issue = [&](auto stage, int turn, int slot) {
      constexpr int s = decltype(stage)::value;
      const int side = turn & 1, chunk = turn < chunks ? chunks - 1 - turn : 0;
      const int64_t at = head * chunks + chunk, kat = khead * chunks + chunk;
      const int64_t tok0 = int64_t(chunk) * kC;
      const int valid = a.T_len - tok0 < kC ? int(a.T_len - tok0) : kC;
      const unsigned dst = slot * St::kSlot;
      if constexpr (s == 0) {
        cp.values(a.dh, (head * a.T_len + tok0) * dv, valid, dv, block * 16 * kWaves,
                  St::kValueAt + side * V::kBytes);
        cp.decay(a.ws.decay + at * 3 * kC, St::kDecayAt + side * kFrag);
        cp.template square<3, false>(a.ws.scoreT + at * 3 * kSquare, dst);
      } else if constexpr (s < St::kInv) {
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int j = 0; j < St::blocks_of(s); ++j) {
            const int t = half * (KS / 2) + (s - 1) * St::kT + j;
            if constexpr (St::kBf16) {
              cp.rows(a.k, (khead * a.T_len + tok0) * dk, valid, dk, t,
                      dst + (half * 2 + j) * 4 * kFrag);
            } else {
#pragma unroll
              for (int p = 0; p < NPL; ++p)
                cp.frag(a.ws.key + (kat * NPL + p) * kPlane, kPlane * 2, t * 4 + cp.w,
                        dst + ((half * NPL + p) * 4 + cp.w) * kFrag);
            }
          }
      } else if constexpr (s == St::kInv) {
        if constexpr (St::kStaged) {
          const int64_t from = (head * a.T_len + tok0) * dv;
          cp.values(static_cast<const float*>(a.sv.X), from, valid, dv, block * 16 * kWaves,
                    St::kXAt);
          cp.values(static_cast<const float*>(a.sv.Y), from, valid, dv, block * 16 * kWaves,
                    St::kYAt);
        }
        cp.template square<3, false>(a.ws.invT + at * 3 * kSquare, dst);
      } else {
        constexpr int j = (s - St::kQueryT) % St::nT;
        cp.template transposed<NPL, KS, St::kI>(
            (s < St::kKeyT ? a.ws.queryT : a.ws.keyT) + kat * NPL * kPlane, j * St::kI,
            St::tiles_of(j), dst);
      }
    };
    static_for<St::kAhead>(
        [&](auto s) { issue(std::integral_constant<int, s % St::n>{}, s / St::n, s); });
    int slot = St::kAhead;
    for (int turn = 0; turn < chunks; ++turn)
      static_for<St::n>([&](auto stage) {
        constexpr int s = decltype(stage)::value, next = s + St::kAhead;
        stage_barrier<St::in_flight(s)>();
        issue(std::integral_constant<int, next % St::n>{}, turn + next / St::n, slot);
        slot = slot + 1 == St::kSlots ? 0 : slot + 1;
        if constexpr (s == St::kQueryT) {  // dV is where dh was
          const int64_t tok0 = int64_t(chunks - 1 - turn) * kC;
          cp.store_values(lds + St::kValueAt + (turn & 1) * V::kBytes, dv_out,
                          (head * a.T_len + tok0) * dv,
                          a.T_len - tok0 < kC ? int(a.T_len - tok0) : kC, dv,
                          block * 16 * kWaves);
        }
      });
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    return;
  }

  const int tile = wave % kWaves, half = wave / kWaves;
  const int col = (block * kWaves + tile) * 16 + m;
  const bool mine = col < dv;
  const int first_row = half * KS * 16;
  f32x4 Z[KS];
  load_memory<KS>(dC_in ? dC_in + head * dv * dk : nullptr, first_row, col, mine, dk, g, Z);
  // K Z of all tokens to the first half's wave, of tokens 32-63 to the
  // second's; then each one's dR to the other
  f32x4* const to_first = reinterpret_cast<f32x4*>(lds + St::kPartAt + tile * St::kPart) + lane;
  f32x4* const to_second = to_first + 4 * 64;
  const unsigned state_off = state_offset(dv, col, lane);
  int read = 0;
  auto enter = [&]() {
    join_barrier();
    const char* slot = lds + read * St::kSlot;
    read = read + 1 == St::kSlots ? 0 : read + 1;
    return slot;
  };

  for (int turn = 0; turn < chunks; ++turn) {
    const int chunk = chunks - 1 - turn;
    const int64_t at = head * chunks + chunk, tok0 = int64_t(chunk) * kC;
    const int valid = a.T_len - tok0 < kC ? int(a.T_len - tok0) : kC;
    const float* decay = reinterpret_cast<const float*>(lds + St::kDecayAt + (turn & 1) * kFrag);
    char* value = lds + St::kValueAt + (turn & 1) * V::kBytes;
    char* const my_value = value + V::lane_at(g) + (tile * 16 + m) * sizeof(T);
    auto value_of = [&](int i, int r) { return reinterpret_cast<T*>(my_value + V::acc_at(i, r)); };
    auto at_tile = [&](int what, int i) {
      return *reinterpret_cast<const f32x4*>(decay + what * kC + acc_row(i, g));
    };
    const int64_t rows = (head * a.T_len + tok0) * dv;  // of values
    // P^T dh: of this wave's tokens, and for the first half of the others too
    f32x4 dh[4], dU[4] = {};
    {
      const char* slot = enter();
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int tok = acc_row(i, g) + r;
          const float x = load_elem(value_of(i, r));
          dh[i][r] = tok < valid ? x : 0.0f;
        }
      const Planes<NPL> h0 = split<NPL>(pair(dh[0], dh[1])), h1 = split<NPL>(pair(dh[2], dh[3]));
      add_square<3, false>(slot, lane, kHighSecond, h1, h1, dU[2], dU[3]);
      if (half == 0) add_square<3, true>(slot, lane, kHighFirst, h0, h1, dU[0], dU[1]);
    }
    // this wave's tokens of X and Y
    f32x4 X[2] = {}, Y[2] = {};
    // K Z over this half's rows
    f32x4 kz[4] = {};
    static_for<St::nK>([&](auto stage) {
      constexpr int s = decltype(stage)::value, nb = St::blocks_of(s + 1);
      const char* slot = enter() + half * (St::kBf16 ? 8 : NPL * 4) * kFrag;
#pragma unroll
      for (int j = 0; j < nb; ++j) {
        Planes<NPL> kf[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) kf[i] = lds_frag<NPL>(slot, j * 4 + i, 4, lane);
        const int t = s * St::kT + j;
        const Planes<3> b = split<3>(pair(Z[2 * t], Z[2 * t + 1]));
        if (mine)
          store_rows(a.sv.Z + (at * dk + first_row + 32 * t) * dv, Z[2 * t], Z[2 * t + 1],
                     state_off, dk - first_row - 32 * t, dv, lane);
        each_product<3, NPL, 3>([&](int x, int y) {
#pragma unroll
          for (int i = 0; i < 4; ++i) kz[i] = mma(kf[i].p[x], b.p[y], kz[i]);
        });
      }
    });
    if (half == 0) {
      to_second[0] = kz[2];
      to_second[64] = kz[3];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) to_first[i * 64] = kz[i];
    }
    // dU, and dR = (I + At)^-T (beta dU) of this wave's tokens
    f32x4 dR[4], own[2] = {};
    float* const part = a.sv.part + (at * a.tiles + block * kWaves + tile) * 3 * kC;
    {
      const char* slot = enter();
      if constexpr (St::kStaged)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {  // zeros behind the end
            using F = Values<float>;
            const char* const x = lds + St::kXAt + F::lane_at(g) + (tile * 16 + m) * 4 +
                                  half * F::acc_at(2, 0) + F::acc_at(i, r);
            X[i][r] = *reinterpret_cast<const float*>(x);
            Y[i][r] = *reinterpret_cast<const float*>(x + (St::kYAt - St::kXAt));
          }
      // e^(G_C - G) K Z, nothing behind the end
      auto whole = [&](int i, f32x4 other) {
        f32x4 x = (kz[i] + other) * at_tile(1, i);
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = acc_row(i, g) + r < valid ? x[r] : 0.0f;
        return x;
      };
      auto write_part = [&](int what, int i, f32x4 x, f32x4 y) {
        f32x4 s;
#pragma unroll
        for (int r = 0; r < 4; ++r) s[r] = row_sum(x[r] * y[r]);
        if (mine && m == 0)
          elem4(part, what * kC + acc_row(2 * half + i, g)) = s;
      };
      auto keep = [&](int i, f32x4 x) {
        if constexpr (!kApart)
          write_part(1, i, X[i], x);
        else if (mine)
          store_tokens(a.sv.KZ + rows, x, acc_row(2 * half + i, g), valid, dv, col, lane);
      };
      if (half == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4 x = whole(i, to_first[i * 64]);
          if (i < 2) keep(i, x);
          dU[i] = (dU[i] + x) * at_tile(2, i);
        }
        add_square<3, true>(slot, lane, kHighFirst, split<3>(pair(dU[0], dU[1])),
                            split<3>(pair(dU[2], dU[3])), own[0], own[1]);
        to_first[0] = own[0];
        to_first[64] = own[1];
      } else {
#pragma unroll
        for (int i = 2; i < 4; ++i) {
          const f32x4 x = whole(i, to_second[(i - 2) * 64]);
          keep(i - 2, x);
          dU[i] = (dU[i] + x) * at_tile(2, i);
        }
        const Planes<3> b = split<3>(pair(dU[2], dU[3]));
        add_square<3, false>(slot, lane, kHighSecond, b, b, own[0], own[1]);
        to_second[0] = own[0];
        to_second[64] = own[1];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (!kApart) write_part(2, i, own[i], Y[i]);
        const int tok = acc_row(2 * half + i, g);
#pragma unroll
        for (int r = 0; r < 4; ++r)  // the other wave has read dh (before this stage's barrier)
          store_elem(reinterpret_cast<T*>(my_value + half * V::acc_at(2, 0) + V::acc_at(i, r)),
                     own[i][r]);
        if (sizeof(T) == 2 && mine)
          store_tokens(a.sv.dR + rows, own[i], tok, valid, dv, col, lane);
      }
    }
    // Z at the chunk's start
    const char* slot = enter();
    if (half == 0) {
      dR[0] = own[0];
      dR[1] = own[1];
      dR[2] = to_second[0];
      dR[3] = to_second[64];
    } else {
      dR[0] = to_first[0];
      dR[1] = to_first[64];
      dR[2] = own[0];
      dR[3] = own[1];
    }
    const float e_all = decay[kC - 1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 e = at_tile(0, i);
      dR[i] *= -e;
      dh[i] *= a.scale * e;
    }
#pragma unroll
    for (int i = 0; i < KS; ++i) Z[i] *= e_all;
    {
      const Planes<3> u0 = split<3>(pair(dh[0], dh[1])), u1 = split<3>(pair(dh[2], dh[3]));
      static_for<St::nT>([&](auto stage) {
        constexpr int j = decltype(stage)::value;
        if (j > 0) slot = enter();
        add_transposed<NPL, St::tiles_of(j), St::kI>(slot, half, u0, u1, Z + j * St::kI, lane);
      });
    }
    {
      const Planes<3> u0 = split<3>(pair(dR[0], dR[1])), u1 = split<3>(pair(dR[2], dR[3]));
      static_for<St::nT>([&](auto stage) {
        constexpr int j = decltype(stage)::value;
        slot = enter();
        add_transposed<NPL, St::tiles_of(j), St::kI>(slot, half, u0, u1, Z + j * St::kI, lane);
      });
    }
  }
  if (dC_out && mine)
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      const int row = first_row + acc_row(i, g);
      if (row < dk) *reinterpret_cast<f32x4*>(dC_out + (head * dv + col) * dk + row) = Z[i];
    }
}

// The two chains: one after the other, or (kBoth) side by side, one in the first
// half of the workgroups.  Float32's gradient never takes X: loads of values
// behind its own stores took a third of its time.
enum Chains { kMemory, kGradient, kBoth };

template <typename T, int KS, Chains kWhich>
__global__ __launch_bounds__(kThreads) void delta_chains_kernel(Chain<T> a, const float* C_in,
                                                                const float* dC_in, T* dv_out,
                                                                float* dC_out) {
  constexpr bool kApart = kWhich == kBoth || sizeof(T) == 4;
  constexpr int kAgain = ForwardStages<T, KS, kAgainPass>::kShared,
                kBack = BackStages<T, KS, kApart>::kShared;
  __shared__ __attribute__((aligned(1024))) char
      lds[kWhich == kMemory ? kAgain : kWhich == kGradient || kBack > kAgain ? kBack : kAgain];
  const int64_t first = kWhich == kBoth ? a.H * a.per_head : 0, wg = blockIdx.x;
  if (kWhich == kMemory || wg < first)
    forward_chain<T, KS, kAgainPass>(a, Segments{}, C_in, nullptr, nullptr, wg, lds);
  else
    back_chain<T, KS, kApart>(a, dC_in, dv_out, dC_out, wg - first, lds);
}

// planes of 8 neighbouring values
template <int N>
__device__ inline Planes<N> to_planes(const f32x8& x) {
  return split<N>(x);
}
template <int N>
__device__ inline Planes<N> to_planes(const bf16x8& x) {
  Planes<N> s = {};
  s.p[0] = x;
  return s;
}
template <typename T>
struct Eight {
  using type = f32x8;
};
template <>
struct Eight<__hip_bfloat16> {
  using type = bf16x8;
};
template <typename T>
__device__ inline typename Eight<T>::type load8(const T* x, int64_t at, bool on) {
  typename Eight<T>::type v = {};
  if (on) v = *reinterpret_cast<const typename Eight<T>::type*>(x + at);
  return v;
}

template <typename T>
__device__ inline typename Eight<T>::type load8(const T* x, unsigned at, bool on) {
  typename Eight<T>::type v = {};
  if (on) v = *reinterpret_cast<const typename Eight<T>::type*>(&elem(x, at));
  return v;
}

constexpr int kGradThreads = 256;
constexpr int kPitch = kC + 1;

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
  int chunks, NH, NHK, dk_dim, dv, ks, tiles, groups, exp_forget;
  float scale;
};

// writes the planes of m (or its transpose) in load order
template <bool kTranspose>
__device__ inline void write_planes(const float (*m)[kPitch], float by, __bf16* to) {
  for (int i = threadIdx.x; i < kSquare / 8; i += kGradThreads) {
    const int lane = i & 63, frag = i >> 6;
    const int row = (frag >> 2) * 32 + row_of((frag >> 1) & 1, lane & 15);
    const int col = (frag & 1) * 32 + (lane >> 4) * 8;
    f32x8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = by * (kTranspose ? m[col + e][row] : m[row][col + e]);
    const Planes<3> s = split<3>(v);
#pragma unroll
    for (int n = 0; n < 3; ++n) *reinterpret_cast<bf16x8*>(to + n * kSquare + i * 8) = s.p[n];
  }
}

// The 64 x 64 matrices of a head's chunk: B, B^T / sqrt(dk) and -(N + N^T) in
// planes for delta_grads_kernel, and what they give to the gates and dbeta.
// kApart: also X . (e^(G_C - G) Z^T k) and dR . Y, for the one tile of Saved::part.
template <typename T, bool kApart>
__global__ __launch_bounds__(kGradThreads, 2) void delta_pairs_kernel(Grads<T> a) {
  constexpr int NPL = sizeof(T) == 2 ? 1 : 3;
  __shared__ double G[kC];
  __shared__ float bt[kC], col_g[kWaves][kC], col_b[kWaves][kC];
  __shared__ float mat[kC][kPitch];
  const int chunk = blockIdx.x % a.chunks;
  const int64_t head = blockIdx.x / a.chunks, at = blockIdx.x;
  const int64_t khead = head / a.NH * a.NHK + head % a.NH / (a.NH / a.NHK);
  const int64_t tok0 = int64_t(chunk) * kC;
  const int valid = a.T_len - tok0 < kC ? int(a.T_len - tok0) : kC;
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, m = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t krow0 = khead * a.T_len + tok0, row0 = head * a.T_len + tok0;
  if (w == 0) {
    G[lane] = chunk_decay(a.fgate + row0, lane, valid, a.exp_forget);
    bt[lane] = a.ws.decay[at * 3 * kC + 2 * kC + lane];
  }
  // rows 16 w ..: dh . X, dR . X, k . k, q . k
  f32x4 hx[4] = {}, rx[4] = {}, kk[4] = {}, qk[4] = {};
  const bool r_on = 16 * w + m < valid;
  // the next 32 columns are on their way while these are worked on
  {
    typename Eight<T>::type h;
    f32x8 r, x[4], y, z;
    float xz = 0.0f, ry = 0.0f;
    auto load = [&](int s) {
      const int c = s + g * 8;
      const bool c_on = c < a.dv;
      h = load8(a.dh, (row0 + 16 * w + m) * a.dv + c, c_on && r_on);
      r = load8(a.dR, (row0 + 16 * w + m) * a.dv + c, c_on && r_on);
      if (kApart) {
        y = load8(a.sv.Y, (row0 + 16 * w + m) * a.dv + c, c_on && r_on);
        z = load8(a.sv.KZ, (row0 + 16 * w + m) * a.dv + c, c_on && r_on);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j <= w)
          x[j] = load8(a.sv.X, (row0 + 16 * j + m) * a.dv + c, c_on && 16 * j + m < valid);
    };
    load(0);
    for (int s = 0; s < a.dv; s += 32) {
      const Planes<NPL> hp = to_planes<NPL>(h);
      const Planes<3> rp = to_planes<3>(r);
      f32x8 now[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) now[j] = x[j];
      if (kApart) {
        const f32x8 own = w == 0 ? x[0] : w == 1 ? x[1] : w == 2 ? x[2] : x[3];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          xz += own[e] * z[e];
          ry += r[e] * y[e];
        }
      }
      load(s + 32);  // nothing behind the last column
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j <= w) {
          const Planes<3> xp = to_planes<3>(now[j]);
          hx[j] = mma_planes<3>(hp, xp, hx[j]);
          rx[j] = mma_planes<3>(rp, xp, rx[j]);
        }
    }
    if (kApart) {  // over the lane groups' columns
#pragma unroll
      for (int o = 16; o < 64; o <<= 1) {
        xz += __shfl_xor(xz, o, 64);
        ry += __shfl_xor(ry, o, 64);
      }
      float* const part = a.sv.part + at * a.tiles * 3 * kC + 16 * w + m;
      if (g == 0) {
        part[kC] = xz;
        part[2 * kC] = ry;
      }
    }
  }
  {
    typename Eight<T>::type q, k[4];
    auto load = [&](int t) {
      const int c = t + g * 8;
      const bool c_on = c < a.dk_dim;
      q = load8(a.q, (krow0 + 16 * w + m) * a.dk_dim + c, c_on && r_on);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j <= w)
          k[j] = load8(a.k, (krow0 + 16 * j + m) * a.dk_dim + c, c_on && 16 * j + m < valid);
    };
    load(0);
    for (int t = 0; t < a.dk_dim; t += 32) {
      const Planes<NPL> qa = to_planes<NPL>(q);
      Planes<NPL> kb[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j <= w) kb[j] = to_planes<NPL>(k[j]);
      Planes<NPL> ka;  // a plane at a time: a choice of structures goes through memory
#pragma unroll
      for (int n = 0; n < NPL; ++n)
        ka.p[n] = w == 0 ? kb[0].p[n] : w == 1 ? kb[1].p[n] : w == 2 ? kb[2].p[n] : kb[3].p[n];
      load(t + 32);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j <= w) {
          kk[j] = mma_planes<NPL>(ka, kb[j], kk[j]);
          qk[j] = mma_planes<NPL>(qa, kb[j], qk[j]);
        }
    }
  }
  __syncthreads();
  // To the gate of token t: the pairs (i, j) with j < t <= i.  A row's sums from its
  // first column on (16 lanes by DPP, `before` from the tiles before), added up
  // over the rows behind the column, are column t - 1's.
  f32x4 before = {};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float cg = 0.0f, cb = 0.0f;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * w + 4 * g + r, c = 16 * j + m;
      const float d = c <= row ? exp2_once(G[row] - G[c]) : 0.0f, b = bt[c];
      const float p = d * qk[j][r] * a.scale;
      mat[row][c] = c <= row ? d * b * hx[j][r] : 0.0f;
      float n = 0.0f, e = 0.0f;
      if (c <= row) cb += p * hx[j][r];
      if (c < row) {
        n = d * b * rx[j][r];
        cb -= d * rx[j][r] * kk[j][r];
        e = p * b * hx[j][r] - n * kk[j][r];
      }
      rx[j][r] = n;
      const float up_to = before[r] + row_prefix(e);
      if (c < row) cg += up_to;
      before[r] += row_sum(e);
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
  __syncthreads();
  __bf16* const out = a.sv.pairs + at * 9 * kSquare;
  write_planes<false>(mat, 1.0f, out);
  write_planes<true>(mat, a.scale, out + 3 * kSquare);
  if (w == 0) {
    float cg = 0.0f, cb = 0.0f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      cg += col_g[i][lane];
      cb += col_b[i][lane];
    }
    a.sv.gates[at * 2 * kC + lane] = cg;
    a.sv.gates[at * 2 * kC + kC + lane] = cb;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * w + 4 * g + r, c = 16 * j + m;
      if (c < row) mat[row][c] = mat[c][row] = -rx[j][r];
      if (c == row) mat[row][c] = 0.0f;
    }
  __syncthreads();
  write_planes<false>(mat, 1.0f, out + 6 * kSquare);
}

// The gradients of q and k: a workgroup takes a key head's chunk and 128
// columns of dk, a wave 32 of them, for the value heads one after the other.
// The contraction over dv runs 32 at a time: wave i splits token tile i of dh,
// dR and X into planes in LDS (two buffers, one barrier), and each wave the
// columns of S and Z that it alone needs; the next 32 are loaded meanwhile.
// Registers are what is short: kShared only where value heads share a key head,
// since dq then lives through the loop.  There bf16 spills 46 of them at two
// workgroups to a CU, and at one, without spills, 8 x 8 / 16 heads of 128 x 1024
// take 593 us instead of 573 backward (2 x 2 / 4 of 64 x 555, 114 instead of 126).
template <typename T, bool kShared>
__global__ __launch_bounds__(kGradThreads,
                             sizeof(T) == 2 ? 2 : 1) void delta_grads_kernel(Grads<T> a) {
  constexpr int NPL = sizeof(T) == 2 ? 1 : 3;  // planes of q, k, dh
  constexpr int kSet = NPL + 6;
  __shared__ __attribute__((aligned(16))) char lds[2][4][kSet][kFrag];
  __shared__ float e0[kC], inner[kWaves];
  const int64_t id = blockIdx.x / a.groups;
  const int chunk = id % a.chunks, blk = int(blockIdx.x % a.groups) * kWaves;
  const int64_t khead = id / a.chunks;
  const int group = kShared ? a.NH / a.NHK : 1;
  const int64_t tok0 = int64_t(chunk) * kC;
  const int valid = a.T_len - tok0 < kC ? int(a.T_len - tok0) : kC;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, g = lane >> 4, m = lane & 15;
  const int64_t krow0 = khead * a.T_len + tok0;
  const int64_t plane = int64_t(a.ks) * 32 * kC;
  const int col0 = (blk + w) * 32;  // this wave's columns
  const int tok = (w >> 1) * 32 + row_of(w & 1, m);  // token tile w
  f32x4 dq[4][2] = {}, dk[4][2] = {};

  for (int hh = 0; hh < group; ++hh) {
    const int64_t head = khead / a.NHK * a.NH + khead % a.NHK * group + hh;
    const int64_t at = head * a.chunks + chunk, row0 = head * a.T_len + tok0;
    const float* decay = a.ws.decay + at * 3 * kC;
    __syncthreads();
    if (w == 0) e0[lane] = decay[lane];
    const float by_r = -decay[tok], by_x = decay[kC + tok] * decay[2 * kC + tok];
    float dot = 0.0f;
    typename Eight<T>::type dh;
    f32x8 dR, X, S[2], Z[2];
    auto load = [&](int s) {
      const int c = s + g * 8;
      const bool on = tok < valid && c < a.dv;
      const unsigned from = tok * a.dv + c;
      dh = load8(a.dh + row0 * a.dv, from, on);
      dR = load8(a.dR + row0 * a.dv, from, on);
      X = load8(a.sv.X + row0 * a.dv, from, on);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int kc = col0 + row_of(p, m);
        const bool k_on = kc < a.dk_dim && c < a.dv;
        const unsigned k_from = kc * a.dv + c;
        S[p] = load8(a.sv.S + at * a.dk_dim * a.dv, k_from, k_on);
        Z[p] = load8(a.sv.Z + at * a.dk_dim * a.dv, k_from, k_on);
      }
    };
    load(0);
    f32x4 own[4][2] = {};  // dh S^T of this value head
    for (int s = 0, side = 0; s < a.dv; s += 32, side ^= 1) {
      {
        const Planes<NPL> h = to_planes<NPL>(dh);
        const Planes<3> r = split<3>(dR * by_r), x = split<3>(X * by_x);
        auto put = [&](int n, bf16x8 v) {
          *reinterpret_cast<bf16x8*>(&lds[side][w][n][lane * 16]) = v;
        };
#pragma unroll
        for (int n = 0; n < NPL; ++n) put(n, h.p[n]);
#pragma unroll
        for (int n = 0; n < 3; ++n) {
          put(NPL + n, r.p[n]);
          put(NPL + 3 + n, x.p[n]);
        }
      }
      Planes<3> Sp[2], Zp[2];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
#pragma unroll
        for (int e = 0; e < 8; ++e) dot += S[p][e] * Z[p][e];
        Sp[p] = split<3>(S[p]);
        Zp[p] = split<3>(Z[p]);
      }
      __syncthreads();
      load(s + 32);  // nothing behind the last column
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Planes<NPL> h = lds_frag<NPL>(lds[side][i][0], 0, 1, lane);
        const Planes<3> r = lds_frag<3>(lds[side][i][NPL], 0, 1, lane);
        const Planes<3> x = lds_frag<3>(lds[side][i][NPL + 3], 0, 1, lane);
        each_product<3, NPL, 3>([&](int y, int z) {
#pragma unroll
          for (int p = 0; p < 2; ++p) own[i][p] = mma(h.p[y], Sp[p].p[z], own[i][p]);
        });
        each_product<3, 3, 3>([&](int y, int z) {
#pragma unroll
          for (int p = 0; p < 2; ++p) dk[i][p] = mma(r.p[y], Sp[p].p[z], dk[i][p]);
#pragma unroll
          for (int p = 0; p < 2; ++p) dk[i][p] = mma(x.p[y], Zp[p].p[z], dk[i][p]);
        });
      }
    }
    // e^G dh S^T + B K, B^T Q^ - (N + N^T) K
    const __bf16* pairs = a.sv.pairs + at * 9 * kSquare;
    const __bf16* keyT = a.ws.keyT + (khead * a.chunks + chunk) * NPL * plane;
    const __bf16* queryT = a.ws.queryT + (khead * a.chunks + chunk) * NPL * plane;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float e = e0[acc_row(i, g) + r];
#pragma unroll
        for (int p = 0; p < 2; ++p) dq[i][p][r] += e * own[i][p][r];
      }
    if (col0 < a.dk_dim)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Planes<NPL> kf[2], qf[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          kf[p] = load_frag<NPL>(keyT, plane, ((blk + w) * 2 + p) * 2 + s, lane);
          qf[p] = load_frag<NPL>(queryT, plane, ((blk + w) * 2 + p) * 2 + s, lane);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int f = i * 2 + s;
          auto add = [&](int which, const Planes<NPL>(&b)[2], f32x4(&c)[2]) {
            const Planes<3> x = load_frag<3>(pairs + which * 3 * kSquare, kSquare, f, lane);
            each_product<3, 3, NPL>([&](int y, int z) {
#pragma unroll
              for (int p = 0; p < 2; ++p) c[p] = mma(x.p[y], b[p].p[z], c[p]);
            });
          };
          if (i >= 2 * s) add(0, kf, dq[i]);  // lower triangular
          if (i < 2 * s + 2) add(1, qf, dk[i]);
          add(2, kf, dk[i]);
        }
      }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) dot += __shfl_xor(dot, o, 64);
    if (lane == 0) inner[w] = dot;
    __syncthreads();
    if (threadIdx.x == 0)
      a.sv.inner[at * a.groups + blk / kWaves] = (inner[0] + inner[1]) + (inner[2] + inner[3]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = acc_row(i, g) + r, kc = col0 + row_of(p, m);
        if (t >= valid || kc >= a.dk_dim) continue;
        store_elem(a.dq + (krow0 + t) * a.dk_dim + kc, a.scale * dq[i][p][r]);
        store_elem(a.dk + (krow0 + t) * a.dk_dim + kc, dk[i][p][r]);
      }
}

// The gradients of beta and of the gates: a wave per head and chunk.
template <typename T, bool kApart>
__global__ __launch_bounds__(64) void delta_gates_kernel(Grads<T> a) {
  const int chunk = blockIdx.x % a.chunks, lane = threadIdx.x;
  const int64_t head = blockIdx.x / a.chunks, at = blockIdx.x;
  const int64_t row0 = head * a.T_len + int64_t(chunk) * kC;
  const int valid = a.T_len - int64_t(chunk) * kC < kC ? int(a.T_len - int64_t(chunk) * kC) : kC;
  float t1 = 0.0f, t3 = 0.0f, t2 = 0.0f;
  const float* part = a.sv.part + at * a.tiles * 3 * kC;
#pragma unroll 8
  for (int i = 0; i < a.tiles; ++i) {
    t1 += part[i * 3 * kC + lane];
    if (!kApart || i == 0) {
      t3 += part[i * 3 * kC + kC + lane];
      t2 += part[i * 3 * kC + 2 * kC + lane];
    }
  }
  const float* decay = a.ws.decay + at * 3 * kC;
  // reads of the memory from each token to the end, writes to it up to each token
  double reads = double(t1) - t2, writes = double(decay[2 * kC + lane]) * t3, kept = 0.0;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const double right = __shfl_down(reads, o, 64), left = __shfl_up(writes, o, 64);
    if (lane + o < 64) reads += right;
    if (lane >= o) writes += left;
  }
  for (int i = 0; i < a.groups; ++i) kept += a.sv.inner[at * a.groups + i];
  const double pairs = a.sv.gates[at * 2 * kC + (lane > 0 ? lane - 1 : 0)];
  writes = __shfl_up(writes, 1, 64);  // of the tokens before
  const double dg = reads + (lane > 0 ? writes + pairs : 0.0) + double(decay[kC - 1]) * kept;
  if (lane < valid) {
    const float x = a.fgate[row0 + lane];
    // d log sigma(x) = sigma(-x), from e^-|x|
    const double t = exp(-fabs(double(x)));
    a.dfgate[row0 + lane] = float(a.exp_forget ? dg : dg * ((x >= 0.0f ? t : 1.0) / (1.0 + t)));
    a.dbeta[row0 + lane] = a.sv.gates[at * 2 * kC + kC + lane] + t3;
  }
}

template <typename T>
hipError_t backward(const DeltaShape& s, const DeltaGrads& d, const Layout& l, const void* q,
                    const void* k, const void* v, const float* fgate, const float* C_in,
                    hipStream_t stream) {
  const Chain<T> a = chain<T>(s, l, q, k, v, d.dh);
  const unsigned wgs = unsigned(a.H * a.per_head);
  hipError_t e = hipSuccess;
  auto run = [&](auto blocks, auto which) {
    constexpr int KS = decltype(blocks)::value;
    constexpr Chains kWhich = decltype(which)::value;
    delta_chains_kernel<T, KS, kWhich><<<kWhich == kBoth ? 2 * wgs : wgs, kThreads, 0, stream>>>(
        a, C_in, d.dC_in, static_cast<T*>(d.dv), d.dC_out);
    return hipGetLastError();
  };
  auto chains = [&](auto blocks) {
    if (side_by_side(s)) return run(blocks, std::integral_constant<Chains, kBoth>{});
    const hipError_t first = run(blocks, std::integral_constant<Chains, kMemory>{});
    return first != hipSuccess ? first
                               : run(blocks, std::integral_constant<Chains, kGradient>{});
  };
#define MLSTM_CHAINS(KS)                            \
  case KS:                                          \
    e = chains(std::integral_constant<int, KS>{});  \
    break
  switch (l.ks) {
    MLSTM_CHAINS(2);
    MLSTM_CHAINS(4);
    MLSTM_CHAINS(6);
    MLSTM_CHAINS(8);
    MLSTM_CHAINS(12);
    MLSTM_CHAINS(16);
    default: return hipErrorInvalidValue;
  }
#undef MLSTM_CHAINS
  if (e != hipSuccess) return e;
  const float* dR = sizeof(T) == 2 ? l.sv.dR : static_cast<const float*>(d.dv);
  const int groups = int((s.dk + 127) / 128);
  const Grads<T> b = {a.q, a.k, a.dh, fgate, dR, l.ws, l.sv, static_cast<T*>(d.dq),
                      static_cast<T*>(d.dk), d.dbeta, d.dfgate, s.T, a.chunks, a.NH, a.NHK, a.dk,
                      a.dv, l.ks, a.tiles, groups, int(s.exp_forget), a.scale};
  const unsigned each = unsigned(a.H * a.chunks);
  constexpr bool kAlways = sizeof(T) == 4;
  const auto pairs = l.apart ? delta_pairs_kernel<T, true> : delta_pairs_kernel<T, kAlways>;
  pairs<<<each, kGradThreads, 0, stream>>>(b);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const auto grads = s.NH > s.NHK ? delta_grads_kernel<T, true> : delta_grads_kernel<T, false>;
  grads<<<unsigned(s.B * s.NHK * a.chunks * groups), kGradThreads, 0, stream>>>(b);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const auto gates = l.apart ? delta_gates_kernel<T, true> : delta_gates_kernel<T, kAlways>;
  gates<<<each, 64, 0, stream>>>(b);
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
