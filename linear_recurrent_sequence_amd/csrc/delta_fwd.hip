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
// planes (delta_common.h).  What is rounded to fewer bits: for bf16 inputs the
// operands of h alone (S, U and P to 16 bits; h is then rounded to 8), never what
// the memory takes in.
//
// What bounds it: the chain.  A chunk of 128 wide heads takes a workgroup 4.5 us
// (about 8700 cycles) whatever runs beside it; of these a SIMD's vector unit is
// busy 47 %, its matrix unit 33 %, the CU's LDS 32 %, and the five barriers and
// the chain's own latencies are the rest.  8 x 16 heads of 128 x 2048 in bf16:
// 145 us for this kernel and 88 us for delta_prep.hip, 58 us being what a copy of
// the inputs and outputs takes.  Measured on the way there: one wave to a value
// tile that loads its operands from memory 750 us; through an LDS ring 195 us;
// with copying waves of its own 138 us, and no less with two waves to a tile, which
// take 317 -> 248 us on 8 x 4 heads of 384 x 2048, where one wave's registers
// spilled.  Slots enough for a whole chunk ahead change nothing there (197 us with
// 7, 195 with 3, before the copying waves).
#include "delta_chain.h"
#include "delta_internal.h"

namespace mlstm {
namespace delta {
namespace {

// What a pass over the chunks is for: h and the memory, the memory once more for
// the backward (no scores, no h), or what a segment of the sequence makes of a
// memory (no Q either).
enum Pass { kForward, kAgainPass, kMapPass };

// The stages of a chunk.  A stage of K and Q (float32: of K, then of Q) and one
// of K^T serve both halves of the memory's rows (KS tiles each).
template <typename T, int KS, Pass kPass>
struct Stages {
  static constexpr bool kAgain = kPass == kAgainPass, kMap = kPass == kMapPass;
  static constexpr bool kBf16 = sizeof(T) == 2;
  static constexpr int NPL = kBf16 ? 1 : 3;             // planes of q and k
  static constexpr int NPP = kBf16 && !kAgain ? 2 : 3;  // of P, and of S and U where h is formed
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
  // then U's planes) and to the second
  static constexpr int kToFirst = 4 > 3 + NPP ? 4 : 3 + NPP, kPart = (kToFirst + 6) * kFrag;
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
    if (s < kKeyT) return Copier::square_copies(NPP);
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
template <typename T, int KS, Pass kPass>
__global__ __launch_bounds__(kThreads) void delta_fwd_kernel(Chain<T> a, Segments seg,
                                                             const float* C_in, T* h,
                                                             float* C_out) {
  using St = Stages<T, KS, kPass>;
  using V = Values<T>;
  constexpr bool kAgain = St::kAgain, kMap = St::kMap;
  constexpr int NPL = St::NPL, NPP = St::NPP;
  constexpr int64_t kPlane = int64_t(KS) * 32 * kC;
  __shared__ __attribute__((aligned(1024))) char lds[St::kShared];
  int64_t head;
  int block;
  map_head(blockIdx.x, a.H, a.per_head * seg.n_of(kMap), head, block);
  const int segment = block / a.per_head;
  block %= a.per_head;
  const int columns = kMap ? a.dv + a.dk : a.dv;
  // segment 0 starts from a memory that is known
  if (kMap && segment == 0 && block * 16 * kWaves >= a.dv) return;  // the whole workgroup
  const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t khead = head / a.NH * a.NHK + head % a.NH / (a.NH / a.NHK);
  const int first = segment * seg.chunks;
  const int chunks = first + seg.chunks < a.chunks ? first + seg.chunks : a.chunks;
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
        cp.template square<NPP, true>(a.ws.score + at * NPP * kSquare, dst);
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
  const float* const from = kMap || segment == 0 ? C_in : seg.before(head, segment, dk, dv);
  f32x4 S[KS];
#pragma unroll
  for (int i = 0; i < KS; ++i) {
    const int row = first_row + acc_row(i, g);
    S[i] = f32x4{};
    if (kMap && col >= dv) {
#pragma unroll
      for (int r = 0; r < 4; ++r) S[i][r] = row + r == col - dv ? 1.0f : 0.0f;
    } else if (from && mine && row < dk && (!kMap || segment == 0)) {
      S[i] = *reinterpret_cast<const f32x4*>(
          from + (int64_t(segment == 0 ? head : 0) * dv + col) * dk + row);
    }
  }
  // to the first half's wave: K S and Q S of tokens 0-31 (four fragments); to
  // the second's: V - e^G K S of all, Q S of tokens 32-63 (six).  What a wave has read
  // it overwrites with planes of its U, for the other one.
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
      each_product<NPP, NPL, 3>([&](int x, int y) {
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
    auto whole = [&](int i, f32x4 part, f32x4 ks) {
      f32x4 x = part - at_tile(0, i) * ks;
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
        const f32x4 r0 = whole(0, R[0], to_first[0]), r1 = whole(1, R[1], to_first[64]);
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
    Planes<NPP> for_h;
    if (kPass == kForward) for_h = split<NPP>(pair(own_u[0], own_u[1]));
    const Planes<3> for_s = split<3>(
        pair(own_u[0] * at_tile(1, 2 * half), own_u[1] * at_tile(1, 2 * half + 1)));
    asm volatile("" ::: "memory");  // what lies there has been read, as another type
    bf16x8* const out = reinterpret_cast<bf16x8*>(half == 0 ? to_first : to_second);
#pragma unroll
    for (int n = 0; n < 3; ++n) out[n * 64] = for_s.p[n];
    if (kPass == kForward && half == 0)
#pragma unroll
      for (int n = 0; n < NPP; ++n) out[(3 + n) * 64] = for_h.p[n];
    if constexpr (kAgain) {
      // X, and e^G dh . (S^T q^) summed over the tile's columns
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int tok = acc_row(2 * half + i, g);
        if (mine) store_tokens(a.sv.X + rows, x[i], tok, valid, dv, col, lane);
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
        add_square<NPP, false>(slot, lane, kLowFirst, for_h, for_h, hs[0], hs[1]);
      } else {
        Planes<NPP> other;
#pragma unroll
        for (int n = 0; n < NPP; ++n) other.p[n] = in[(3 + n) * 64];
        add_square<NPP, true>(slot, lane, kLowSecond, other, for_h, hs[0], hs[1]);
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
                  const void* dh, const float* C_in, void* h, float* C_out, hipStream_t stream) {
  Chain<T> a = chain<T>(s, l, q, k, v, dh);
  Segments seg = l.seg;
  if (kPass == kAgainPass) seg = {1, a.chunks, nullptr, nullptr};
  if (kPass == kMapPass) a.per_head = int((s.dv + s.dk + 63) / 64);
  const unsigned grid = unsigned(a.H * a.per_head * seg.n_of(kPass == kMapPass));
  delta_fwd_kernel<T, KS, kPass><<<grid, kThreads, 0, stream>>>(a, seg, C_in, static_cast<T*>(h),
                                                                C_out);
  return hipGetLastError();
}

template <Pass kPass>
hipError_t dispatch(const DeltaShape& s, const Layout& l, const void* q, const void* k,
                    const void* v, const void* dh, const float* C_in, void* h, float* C_out,
                    hipStream_t stream) {
#define MLSTM_FWD(KS)                                                                         \
  case KS:                                                                                    \
    return s.is_bf16                                                                          \
               ? launch<__hip_bfloat16, KS, kPass>(s, l, q, k, v, dh, C_in, h, C_out, stream) \
               : launch<float, KS, kPass>(s, l, q, k, v, dh, C_in, h, C_out, stream)
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

hipError_t launch_again(const DeltaShape& s, const Layout& l, const void* q, const void* k,
                        const void* v, const void* dh, const float* C_in, hipStream_t stream) {
  return dispatch<kAgainPass>(s, l, q, k, v, dh, C_in, nullptr, nullptr, stream);
}

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
    e = dispatch<kMapPass>(s, l, q, k, v, nullptr, C_in, nullptr, nullptr, stream);
    if (e != hipSuccess) return e;
    const auto join =
        s.dk <= kJoinRows ? delta_join_kernel<1> : delta_join_kernel<kJoinMax>;
    join<<<unsigned(s.B * s.NH * (s.dv / kJoinCols)), kJoinLanes * kJoinShares, 0, stream>>>(
        l.seg, C_in, int(s.dk), int(s.dv));
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (C_in) C_in = l.seg.start;
  }
  return dispatch<kForward>(s, l, q, k, v, nullptr, C_in, h, C_out, stream);
}

}  // namespace mlstm
