// The chain of the gated delta rule over a sequence's chunks: for the forward
// pass, for what a segment makes of a memory, and for the memory once more in the
// backward pass.  The mathematics and the measurements stand in delta_fwd.hip.
#pragma once

#include "delta_chain.h"
#include "delta_internal.h"

namespace mlstm {
namespace delta {

// What a pass over the chunks is for: h and the memory, the memory once more for
// the backward (no scores, no h), or what a segment of the sequence makes of a
// memory (no Q either).
enum Pass { kForward, kAgainPass, kMapPass };

// The stages of a chunk.  A stage of K and Q (float32: of K, then of Q) and one
// of K^T serve both halves of the memory's rows (KS tiles each).
template <typename T, int KS, Pass kPass>
struct ForwardStages {
  static constexpr bool kAgain = kPass == kAgainPass, kMap = kPass == kMapPass;
  static constexpr bool kBf16 = sizeof(T) == 2;
  static constexpr int NPL = kBf16 ? 1 : 3;             // planes of q and k
  static constexpr int kI = kBf16 ? 4 : 2;              // row tiles of K^T for each half
  static constexpr int nKQ = kBf16 || kMap ? KS / 2 : KS, nKT = (KS + kI - 1) / kI;
  static constexpr int kInv = nKQ, kKeyT = nKQ + (kPass == kForward ? 2 : 1),
                       n = kKeyT + nKT;
  static constexpr int kSlot = (kBf16 ? 18 : 24) * kFrag;
  // kAgain with bf16: dh comes through LDS too, with the inverse (a wave that
  // stores and then loads waits for its stores); one buffer, so less than a
  // chunk ahead.  Otherwise at most a chunk ahead: the values and decays of two
  // chunks have room.
  static constexpr bool kStaged = kAgain && kBf16;
  static constexpr int kMost = kStaged ? 3 : kBf16 ? 4 : 2;
  static constexpr int kAhead = n - kStaged < kMost ? n - kStaged : kMost;
  // between a value tile's two waves: to the first (K S and Q S of tokens 0-31,
  // then six planes made of U) and to the second
  static constexpr int kToFirst = 6, kPart = (kToFirst + 6) * kFrag;
  static constexpr int kSlots = kAhead + 1;
  static constexpr int kValueAt = kSlots * kSlot, kDecayAt = kValueAt + 2 * Values<T>::kBytes,
                       kPartAt = kDecayAt + 2 * kFrag, kDhAt = kPartAt + kWaves * kPart,
                       kShared = kDhAt + (kStaged ? Values<T>::kBytes : 0);

  static constexpr int tiles_of(int s) {  // of K^T, for each half
    return KS - (s - kKeyT) * kI < kI ? KS - (s - kKeyT) * kI : kI;
  }
  // copies of each copying wave in a stage
  static constexpr int copies(int s) {
    s %= n;
    if (s < nKQ) return (!kBf16 ? 6 : kMap ? 2 : 4) + (s == 0 ? Values<T>::kCopies + 1 : 0);
    if (s == kInv) return Copier::square_copies(3) + (kStaged ? Values<T>::kCopies : 0);
    if (s < kKeyT) return Copier::square_copies(3);
    return tiles_of(s) * NPL;
  }
  static constexpr int in_flight(int s) {
    int k = 0;
    for (int j = 1; j < kAhead; ++j) k += copies(s + j);
    return k;
  }
};

// T: element type of q, k, v, h.  KS: 32-column blocks of dk (even).
//
// A sequence may be cut into segments (Segments): each is a workgroup's own, from
// chunk first to chunk last.  The forward takes the memory before a segment from
// `seg.maps`; the map pass writes there what a segment makes of zero (segment 0:
// of C_in) with its values, and of each unit vector without them (value columns
// dv .. dv + dk).
//
// One workgroup's work, wg being its number.
template <typename T, int KS, Pass kPass>
__device__ inline void forward_chain(const Chain<T>& a, const Segments& seg, const float* C_in,
                                     T* h, float* C_out, int64_t wg, char* lds) {
  using St = ForwardStages<T, KS, kPass>;
  using V = Values<T>;
  constexpr bool kAgain = St::kAgain, kMap = St::kMap;
  constexpr int NPL = St::NPL;
  constexpr int64_t kPlane = int64_t(KS) * 32 * kC;
  int64_t head;
  int block;
  map_head(wg, a.H, a.per_head * (kAgain ? 1 : seg.n_of(kMap)), head, block);
  const int segment = kAgain ? 0 : block / a.per_head;  // the backward has one
  if (!kAgain) block %= a.per_head;
  const int columns = kMap ? a.dv + a.dk : a.dv;
  // segment 0 starts from a memory that is known
  if (kMap && segment == 0 && block * 16 * kWaves >= a.dv) return;  // the whole workgroup
  const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t khead = head / a.NH * a.NHK + head % a.NH / (a.NH / a.NHK);
  const int first = kAgain ? 0 : segment * seg.chunks;
  const int chunks =
      !kAgain && first + seg.chunks < a.chunks ? first + seg.chunks : a.chunks;
  const int dk = a.dk, dv = a.dv;

  if (wave >= kChainWaves) {
    // ------------------------------------------------------ the copying waves
    const Copier cp = {wave - kChainWaves, lane, tilecommon::lds_addr(lds)};
    // this wave's copies of stage s of a chunk into a slot
    auto issue = [&](auto stage, int chunk, int slot) {
      constexpr int s = decltype(stage)::value;
      // behind the last chunk: its data again, into the buffers of the one after
      const int side = chunk & 1;
      chunk = chunk < chunks ? chunk : chunks - 1;
      const int64_t at = head * a.chunks + chunk, kat = khead * a.chunks + chunk;
      const int64_t tok0 = int64_t(chunk) * kC;
      const int valid = a.T_len - tok0 < kC ? int(a.T_len - tok0) : kC;
      const unsigned dst = slot * St::kSlot;
      if constexpr (s == 0) {
        cp.values(a.v, (head * a.T_len + tok0) * dv, valid, dv, block * 16 * kWaves,
                  St::kValueAt + side * V::kBytes);
        cp.decay(a.ws.decay + at * 3 * kC, St::kDecayAt + side * kFrag);
      }
      if constexpr (s < St::nKQ) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if constexpr (St::kBf16) {
            const int t = half * (KS / 2) + s;
            const int64_t from = (khead * a.T_len + tok0) * dk;
            cp.rows(a.k, from, valid, dk, t, dst + half * 8 * kFrag);
            if (!kMap) cp.rows(a.q, from, valid, dk, t, dst + (half * 8 + 4) * kFrag);
          } else {
            const int t = half * (KS / 2) + (kMap ? s : s / 2);
#pragma unroll
            for (int p = 0; p < NPL; ++p)
              cp.frag((!kMap && s % 2 ? a.ws.query : a.ws.key) + (kat * NPL + p) * kPlane,
                      kPlane * 2, t * 4 + cp.w, dst + ((half * NPL + p) * 4 + cp.w) * kFrag);
          }
        }
      } else if constexpr (s == St::kInv) {
        if constexpr (St::kStaged)
          cp.values(a.dh, (head * a.T_len + tok0) * dv, valid, dv, block * 16 * kWaves, St::kDhAt);
        cp.template square<3, true>(a.ws.inv + at * 3 * kSquare, dst);
      } else if constexpr (s < St::kKeyT) {
        cp.template square<3, true>(a.ws.score + at * 3 * kSquare, dst);
      } else {
        cp.template transposed<NPL, KS, St::kI>(a.ws.keyT + kat * NPL * kPlane,
                                                (s - St::kKeyT) * St::kI, St::tiles_of(s), dst);
      }
    };
    static_for<St::kAhead>(
        [&](auto s) { issue(std::integral_constant<int, s % St::n>{}, first + s / St::n, s); });
    int slot = St::kAhead;
    for (int chunk = first; chunk < chunks; ++chunk)
      static_for<St::n>([&](auto stage) {
        constexpr int s = decltype(stage)::value, next = s + St::kAhead;
        stage_barrier<St::in_flight(s)>();
        issue(std::integral_constant<int, next % St::n>{}, chunk + next / St::n, slot);
        slot = slot + 1 == St::kSlots ? 0 : slot + 1;
        if constexpr (s == St::kKeyT && kPass == kForward) {  // h is where the chunk's values were
          const int64_t tok0 = int64_t(chunk) * kC;
          cp.store_values(lds + St::kValueAt + (chunk & 1) * V::kBytes, h,
                          (head * a.T_len + tok0) * dv,
                          a.T_len - tok0 < kC ? int(a.T_len - tok0) : kC, dv,
                          block * 16 * kWaves);
        }
      });
    // no copy may be in flight into LDS that another workgroup gets
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    return;
  }

  // ---------------------------------------------------------- the chain's waves
  const int tile = wave % kWaves, half = wave / kWaves;
  const int col = (block * kWaves + tile) * 16 + m;  // value column
  const bool mine = col < columns;  // whole waves; the others keep the barriers company
  const int first_row = half * KS * 16;
  const float* from = kMap || kAgain || segment == 0 ? C_in : seg.before(head, segment, dk, dv);
  if (kMap && segment != 0) from = nullptr;
  if (from && segment == 0) from += head * dv * dk;
  f32x4 S[KS];
  load_memory<KS>(from, first_row, col, col < dv, dk, g, S);
  if (kMap)
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        S[i][r] = first_row + acc_row(i, g) + r == col - dv ? 1.0f : S[i][r];
  // to the first half's wave: K S and Q S of tokens 0-31 (four fragments); to
  // the second's: V - e^G K S (kAgain: K S) of all, Q S of tokens 32-63 (six).  What a
  // wave has read it overwrites with planes of its U, for the other one.
  f32x4* const to_first = reinterpret_cast<f32x4*>(lds + St::kPartAt + tile * St::kPart) + lane;
  f32x4* const to_second = to_first + St::kToFirst * 64;

  const unsigned state_off = state_offset(dv, col, lane);

  int read = 0;  // the slot of the stage at hand
  auto enter = [&]() {
    join_barrier();
    const char* slot = lds + read * St::kSlot;
    read = read + 1 == St::kSlots ? 0 : read + 1;
    return slot;
  };

  for (int chunk = first; chunk < chunks; ++chunk) {
    const int64_t at = head * a.chunks + chunk, tok0 = int64_t(chunk) * kC;
    const int valid = a.T_len - tok0 < kC ? int(a.T_len - tok0) : kC;
    const float* decay = reinterpret_cast<const float*>(lds + St::kDecayAt + (chunk & 1) * kFrag);
    char* value = lds + St::kValueAt + (chunk & 1) * V::kBytes;
    char* const my_value = value + V::lane_at(g) + (tile * 16 + m) * sizeof(T);
    auto value_of = [&](int i, int r) { return reinterpret_cast<T*>(my_value + V::acc_at(i, r)); };
    auto at_tile = [&](int what, int i) {
      return *reinterpret_cast<const f32x4*>(decay + what * kC + acc_row(i, g));
    };
    // of values: this wave's tokens are rows + (4 i + r) dv + own
    const int64_t rows = (head * a.T_len + tok0) * dv;
    const unsigned own = (32 * half + 8 * g) * dv + col;
    f32x4 dh[2] = {};
    if constexpr (kAgain && !St::kStaged)
      if (mine)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int tok = acc_row(2 * half + i, g) + r;
            if (tok < valid) dh[i][r] = load_elem(&elem(a.dh + rows + (4 * i + r) * dv, own));
          }

    // K S and Q S over this half's rows
    f32x4 ks[4] = {}, qs[4] = {};
    static_for<KS / 2>([&](auto block_t) {
      constexpr int t = decltype(block_t)::value;
      Planes<NPL> kf[4], qf[4];
      const char* slot = enter() + half * (St::kBf16 ? 8 : NPL * 4) * kFrag;
#pragma unroll
      for (int i = 0; i < 4; ++i) kf[i] = lds_frag<NPL>(slot, i, 4, lane);
      if constexpr (St::kBf16 && kPass == kForward)
#pragma unroll
        for (int i = 0; i < 4; ++i) qf[i] = lds_frag<NPL>(slot, 4 + i, 4, lane);
      const Planes<3> b = split<3>(pair(S[2 * t], S[2 * t + 1]));
      if (kAgain && mine)
        store_rows(a.sv.S + (at * dk + first_row + 32 * t) * dv, S[2 * t], S[2 * t + 1], state_off,
                   dk - first_row - 32 * t, dv, lane);
      each_product<3, NPL, 3>([&](int x, int y) {
#pragma unroll
        for (int i = 0; i < 4; ++i) ks[i] = mma(kf[i].p[x], b.p[y], ks[i]);
      });
      if constexpr (kMap) {
        return;
      } else if constexpr (!St::kBf16) {
        slot = enter() + half * NPL * 4 * kFrag;
#pragma unroll
        for (int i = 0; i < 4; ++i) qf[i] = lds_frag<NPL>(slot, i, 4, lane);
      } else if constexpr (kAgain) {
        asm volatile("" ::: "memory");  // not before: registers are short
#pragma unroll
        for (int i = 0; i < 4; ++i) qf[i] = lds_frag<NPL>(slot, 4 + i, 4, lane);
      }
      each_product<3, NPL, 3>([&](int x, int y) {
#pragma unroll
        for (int i = 0; i < 4; ++i) qs[i] = mma(qf[i].p[x], b.p[y], qs[i]);
      });
    });
    // R = V - e^G K S, from the sum of the halves: the first half's wave takes the
    // values, so that the second's, which has more to do below, has less here
    f32x4 R[4];
    if (half == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (kAgain) {  // the memory's prediction by itself, see Y
          to_second[i * 64] = ks[i];
          continue;
        }
        const f32x4 e = at_tile(0, i);
#pragma unroll
        for (int r = 0; r < 4; ++r) R[i][r] = load_elem(value_of(i, r)) - e[r] * ks[i][r];
        to_second[i * 64] = R[i];
      }
      to_second[4 * 64] = qs[2];
      to_second[5 * 64] = qs[3];
    } else {
      to_first[0] = ks[0];
      to_first[64] = ks[1];
      to_first[2 * 64] = qs[0];
      to_first[3 * 64] = qs[1];
    }
    f32x4 Y[2];  // kAgain: e^G K S of this wave's tokens
    auto whole = [&](int i, f32x4 part, f32x4 ks) {
      f32x4 x;
      if constexpr (kAgain) {
        const f32x4 y = at_tile(0, i) * (part + ks);
        if ((i >> 1) == half) Y[i & 1] = y;
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = load_elem(value_of(i, r)) - y[r];
      } else {
        x = part - at_tile(0, i) * ks;
      }
#pragma unroll
      for (int r = 0; r < 4; ++r)  // behind the end: nothing, whatever the memory holds
        x[r] = acc_row(i, g) + r < valid ? x[r] : 0.0f;
      return x;
    };
    // X (first half: tokens 0-31, second: 32-63) and U = beta X; the planes that
    // the other wave takes of it go through LDS
    f32x4 x[2] = {}, hs[2];
    {
      const char* slot = enter();
      if (half == 0) {
        const f32x4 r0 = whole(0, kAgain ? ks[0] : R[0], to_first[0]),
                    r1 = whole(1, kAgain ? ks[1] : R[1], to_first[64]);
        hs[0] = qs[0] + to_first[2 * 64];
        hs[1] = qs[1] + to_first[3 * 64];
        const Planes<3> b = split<3>(pair(r0, r1));
        add_square<3, false>(slot, lane, kLowFirst, b, b, x[0], x[1]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) R[i] = whole(i, to_second[i * 64], ks[i]);
        hs[0] = qs[2] + to_second[4 * 64];
        hs[1] = qs[3] + to_second[5 * 64];
        add_square<3, true>(slot, lane, kLowSecond, split<3>(pair(R[0], R[1])),
                            split<3>(pair(R[2], R[3])), x[0], x[1]);
      }
      hs[0] *= a.scale * at_tile(0, 2 * half);
      hs[1] *= a.scale * at_tile(0, 2 * half + 1);
    }
    const f32x4 own_u[2] = {x[0] * at_tile(2, 2 * half), x[1] * at_tile(2, 2 * half + 1)};
    // of U for h, of e^(G_C - G) U for the memory
    Planes<3> for_h;
    if (kPass == kForward) for_h = split<3>(pair(own_u[0], own_u[1]));
    const Planes<3> for_s = split<3>(
        pair(own_u[0] * at_tile(1, 2 * half), own_u[1] * at_tile(1, 2 * half + 1)));
    asm volatile("" ::: "memory");  // what lies there has been read, as another type
    bf16x8* const out = reinterpret_cast<bf16x8*>(half == 0 ? to_first : to_second);
#pragma unroll
    for (int n = 0; n < 3; ++n) out[n * 64] = for_s.p[n];
    if (kPass == kForward && half == 0)
#pragma unroll
      for (int n = 0; n < 3; ++n) out[(3 + n) * 64] = for_h.p[n];
    if constexpr (kAgain) {
      // X, Y, and e^G dh . (S^T q^) summed over the tile's columns
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int tok = acc_row(2 * half + i, g);
        if (mine) {
          store_tokens(a.sv.X + rows, x[i], tok, valid, dv, col, lane);
          store_tokens(a.sv.Y + rows, Y[i], tok, valid, dv, col, lane);
        }
        f32x4 s;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if constexpr (St::kStaged)  // zeros behind the end
            dh[i][r] = load_elem(reinterpret_cast<const T*>(
                lds + St::kDhAt + V::lane_at(g) + (tile * 16 + m) * sizeof(T) +
                half * V::acc_at(2, 0) + V::acc_at(i, r)));
          s[r] = row_sum(dh[i][r] * hs[i][r]);
        }
        if (mine && m == 0)
          elem4(a.sv.part + (at * a.tiles + block * kWaves + tile) * 3 * kC, tok) = s;
      }
    }
    const char* slot = enter();
    const bf16x8* const in = reinterpret_cast<const bf16x8*>(half == 0 ? to_second : to_first);
    if constexpr (kPass == kForward) {
      // h = e^G Q^ S + P U, for this wave's tokens
      if (half == 0) {
        add_square<3, false>(slot, lane, kLowFirst, for_h, for_h, hs[0], hs[1]);
      } else {
        Planes<3> other;
#pragma unroll
        for (int n = 0; n < 3; ++n) other.p[n] = in[(3 + n) * 64];
        add_square<3, true>(slot, lane, kLowSecond, other, for_h, hs[0], hs[1]);
      }
      // to where the values were; the copying waves store it
      char* const my_half = my_value + half * V::acc_at(2, 0);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          store_elem(reinterpret_cast<T*>(my_half + V::acc_at(i, r)), hs[i][r]);
      slot = nullptr;
    }
    // S = e^(G_C) S + K^T (e^(G_C - G) U)
    const float e_all = decay[kC - 1];
    Planes<3> u0 = for_s, u1 = for_s;
#pragma unroll
    for (int n = 0; n < 3; ++n) (half == 0 ? u1 : u0).p[n] = in[n * 64];
#pragma unroll
    for (int i = 0; i < KS; ++i) S[i] *= e_all;
    static_for<St::nKT>([&](auto stage) {
      constexpr int j = decltype(stage)::value;
      if (kPass == kForward || j > 0) slot = enter();
      add_transposed<NPL, St::tiles_of(St::kKeyT + j), St::kI>(slot, half, u0, u1,
                                                               S + j * St::kI, lane);
    });
  }
  // the memory after the segment: the caller's, or the map pass's
  float* to = nullptr;
  if (kMap) to = seg.after(head, segment, dk, dv);
  if (kPass == kForward && chunks == a.chunks) to = C_out + head * dv * dk;
  if (to && mine)
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      const int row = first_row + acc_row(i, g);
      if (row < dk) *reinterpret_cast<f32x4*>(to + int64_t(col) * dk + row) = S[i];
    }
}

}  // namespace delta
}  // namespace mlstm
