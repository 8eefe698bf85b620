// What the chain kernels of the gated delta rule (the forward, the memory once
// more for the backward, and its gradient backward) have in common.
//
// A workgroup has four value tiles of 16 columns, two waves to each (one half of
// the memory's rows each) and four waves that copy.  All tiles read the same
// left operands, 1 KiB "fragments" (16 rows x 32 columns, 16 bytes per lane in
// the order of the matrix instruction's lanes).  A chunk is a fixed sequence of
// stages of at most kSlot bytes, copied global -> LDS without registers into a
// ring of slots, up to a chunk ahead: at the start of a stage each copying wave
// waits for its own copies of that stage (vmcnt counts in order), a barrier
// makes them whole and ends the reads of the stage before, whose slot then
// takes the copies of a later stage.  Every copying wave issues the same number
// of copies in each stage, so the counts are constants; behind the last chunk
// the copies repeat it.  A chain's wave is bound by what it issues and waits
// for, and the copies' addresses would be a quarter of its instructions.
#pragma once

#include "delta_common.h"
#include "tile_common.h"

namespace mlstm {
namespace delta {

using tilecommon::i32x4;
using tilecommon::static_for;

constexpr int kFrag = 1024;  // bytes

// 16 bytes per lane from rsrc + voffset + soffset to LDS at dst + 16 * lane;
// dst and soffset are wave-uniform.  The wait is the caller's.  The wait states
// cover scalar registers that a vector instruction has just written (5).
__device__ inline void copy_frag(i32x4 rsrc, unsigned voffset, unsigned soffset, unsigned dst) {
  rsrc = tilecommon::sreg(rsrc);
  dst = tilecommon::sreg(dst);
  soffset = tilecommon::sreg(soffset);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(dst), "v"(voffset), "s"(rsrc), "s"(soffset)
               : "memory", "m0");
}

// waits until at most N of this wave's vector memory operations are in flight
// (and its LDS reads are done), then for the workgroup
template <int N>
__device__ inline void stage_barrier() {
  static_assert(N < 64, "vmcnt has 6 bits");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// the same for a wave that copies nothing
__device__ inline void join_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <int N>
__device__ inline Planes<N> lds_frag(const char* slot, int first, int step, int lane) {
  Planes<N> s;
#pragma unroll
  for (int n = 0; n < N; ++n)
    s.p[n] = *reinterpret_cast<const bf16x8*>(slot + (first + n * step) * kFrag + lane * 16);
  return s;
}

constexpr int kWaves = 4;                              // value tiles, and copying waves
constexpr int kChainWaves = 2 * kWaves;                // two to a value tile
constexpr int kThreads = 64 * (kChainWaves + kWaves);

// A chunk's values (64 tokens of the workgroup's 64 columns) in LDS.
template <typename T>
struct Values {
  static constexpr int kRow = 16 * kWaves * int(sizeof(T));  // bytes of a token
  static constexpr int kPad = kRow / 4;                      // after 8 tokens: no bank conflicts
  static constexpr int kBytes = kC * kRow + kC / 8 * kPad;
  static constexpr int kCopies = kC * kRow / kFrag / kWaves;  // of each copying wave
  static constexpr int kLanes = kRow / 16;                    // of a token
  static __device__ int at(int tok) { return tok * kRow + (tok >> 3) * kPad; }
  // of token acc_row(i, g) + r: a lane's base and a constant
  static __device__ int lane_at(int g) { return g * (8 * kRow + kPad); }
  static constexpr int acc_at(int i, int r) {
    return (i >> 1) * (32 * kRow + 4 * kPad) + (4 * (i & 1) + r) * kRow;
  }
};

// The position of accumulator (tile i, lane group g, element 0): a token, or a
// memory row from the half's first on.
__device__ inline int acc_row(int i, int g) { return (i >> 1) * 32 + 8 * g + 4 * (i & 1); }

// A wave's slice of a memory x [dv][dk] (NULL: zeros): rows first_row .. of value
// column col, zeros beyond dk and where not `mine`.  Every lane loads, from the
// first row where it has none: around a branch the compiler may spill a register of
// all lanes while some are off (seen with 168 registers in use: the lane's number,
// stored before the branch's lanes are on again).
template <int KS>
__device__ inline void load_memory(const float* x, int first_row, int col, bool mine, int dk,
                                   int g, f32x4 (&S)[KS]) {
#pragma unroll
  for (int i = 0; i < KS; ++i) S[i] = f32x4{};
  if (!x) return;
  x += int64_t(mine ? col : 0) * dk;
#pragma unroll
  for (int i = 0; i < KS; ++i) {
    const int row = first_row + acc_row(i, g);
    const bool on = mine && row < dk;
    const f32x4 s = *reinterpret_cast<const f32x4*>(x + (row < dk ? row : 0));
#pragma unroll
    for (int r = 0; r < 4; ++r) S[i][r] = on ? s[r] : 0.0f;
  }
}

// Two tiles (32 rows from `row` on) of a wave's slice of the memory, one value
// column per lane, to x [dk][dv], and 4 tokens of a value column per lane to x
// [T][dv]: transposed over quads of lanes, so that a lane stores 16 bytes and 16
// lanes four runs of 64.  The memory goes out two tiles to a stage.
// x: from row `row` on; off: state_offset; more: dk - row.
__device__ inline unsigned state_offset(int dv, int col, int lane) {
  return (8 * (lane >> 4) + (lane & 3)) * dv + (col & ~3);
}
__device__ inline void store_rows(float* x, f32x4 s0, f32x4 s1, unsigned off, int more, int dv,
                                  int lane) {
  const int row = 8 * (lane >> 4) + (lane & 3);
  s0 = quad_transpose(s0, lane);
  if (row < more) elem4(x, off) = s0;
  s1 = quad_transpose(s1, lane);
  if (row + 4 < more) elem4(x + 4 * dv, off) = s1;
}
__device__ inline void store_tokens(float* x, f32x4 y, int tok, int valid, int dv, int col,
                                    int lane) {
  y = quad_transpose(y, lane);
  tok += lane & 3;
  if (tok < valid) elem4(x, tok * dv + (col & ~3)) = y;
}

// One copying wave's view: w of kWaves.
struct Copier {
  int w, lane;
  unsigned lds0;

  __device__ unsigned lane16() const { return lane * 16; }

  // values x [T][dv] of one head from token tok0 on, columns col0 ..
  template <typename T>
  __device__ void values(const T* x, int64_t from, int valid, int dv, int col0,
                         unsigned to) const {
    using V = Values<T>;
    const i32x4 r = tilecommon::rsrc_words(x + from, int64_t(valid) * dv * sizeof(T));
    const int c = col0 + lane % V::kLanes * (16 / int(sizeof(T)));
#pragma unroll
    for (int j = 0; j < V::kCopies; ++j) {
      const int first = (w * V::kCopies + j) * (64 / V::kLanes);  // token
      copy_frag(r,
                c < dv ? unsigned((first + lane / V::kLanes) * dv + c) * unsigned(sizeof(T))
                       : tilecommon::kOutOfRange,
                0, lds0 + to + V::at(first));
    }
  }
  // the way back: 16 bytes a lane
  template <typename T>
  __device__ void store_values(const char* values, T* x, int64_t to, int valid, int dv,
                               int col0) const {
    using V = Values<T>;
    const int c = col0 + lane % V::kLanes * (16 / int(sizeof(T)));
#pragma unroll
    for (int j = 0; j < V::kCopies; ++j) {
      const int tok = (w * V::kCopies + j) * (64 / V::kLanes) + lane / V::kLanes;
      const uint4 u =
          *reinterpret_cast<const uint4*>(values + V::at(tok) + lane % V::kLanes * 16);
      if (tok < valid && c < dv) *reinterpret_cast<uint4*>(x + to + int64_t(tok) * dv + c) = u;
    }
  }
  __device__ void decay(const float* from, unsigned to) const {
    copy_frag(tilecommon::rsrc_words(from, 3 * kC * 4), lane16(), 0, lds0 + to);
  }
  // row tile w of 32-column block t of a chunk of q or k (bf16)
  template <typename T>
  __device__ void rows(const T* x, int64_t from, int valid, int dk, int t, unsigned to) const {
    const int c = t * 32 + (lane >> 4) * 8;
    const unsigned row = ((w >> 1) * 32 + row_of(w & 1, lane & 15)) * dk * 2;
    copy_frag(tilecommon::rsrc_words(x + from, int64_t(valid) * dk * 2),
              c < dk ? row + c * 2 : tilecommon::kOutOfRange, 0, lds0 + to + w * kFrag);
  }
  // fragment f of a plane of `bytes` bytes
  __device__ void frag(const __bf16* plane, int64_t bytes, int f, unsigned to) const {
    copy_frag(tilecommon::rsrc_words(plane, bytes), lane16(), f * kFrag, lds0 + to);
  }
  // NP planes of a triangular 64 x 64 operand: six fragments each, in the order
  // of low_pair or high_pair
  template <int NP, bool kLow>
  __device__ void square(const __bf16* from, unsigned to) const {
    const i32x4 r = tilecommon::rsrc_words(from, NP * kSquare * 2);
#pragma unroll
    for (int j = 0; j < square_copies(NP); ++j) {
      const int f = j * kWaves + w < 6 * NP ? j * kWaves + w : 6 * NP - 1;
      copy_frag(r, lane16(),
                f / 6 * (kSquare * 2) + (kLow ? low_pair(f % 6) : high_pair(f % 6)) * kFrag,
                lds0 + to + f * kFrag);  // the last one more than once, where they do not divide
    }
  }
  static constexpr int square_copies(int np) { return (6 * np + kWaves - 1) / kWaves; }
  // row tiles i0 .. of each half of K^T or Q^T (NPL planes, KS tiles to a half):
  // this wave takes one half of the tokens of one half of the rows
  template <int NPL, int KS, int kI>
  __device__ void transposed(const __bf16* from, int i0, int tiles, unsigned to) const {
    constexpr int64_t kPlane = int64_t(KS) * 32 * kC;
#pragma unroll
    for (int p = 0; p < NPL; ++p)
#pragma unroll
      for (int i = 0; i < kI; ++i)
        if (i < tiles)
          frag(from + p * kPlane, kPlane * 2, ((w >> 1) * KS + i0 + i) * 2 + (w & 1),
               to + (((p * 2 + (w >> 1)) * kI + i) * 2 + (w & 1)) * kFrag);
  }
};

// S[i] += the staged tiles of K^T or Q^T times u (tokens 0-31, 32-63)
template <int NPL, int N, int kI>
__device__ inline void add_transposed(const char* slot, int half, const Planes<3>& u0,
                                      const Planes<3>& u1, f32x4* S, int lane) {
  slot += half * kI * 2 * kFrag;
  Planes<NPL> a[N], b[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    a[i] = lds_frag<NPL>(slot, 2 * i, kI * 4, lane);
    b[i] = lds_frag<NPL>(slot, 2 * i + 1, kI * 4, lane);
  }
  each_product<3, NPL, 3>([&](int x, int y) {
#pragma unroll
    for (int i = 0; i < N; ++i) S[i] = mma(a[i].p[x], u0.p[y], S[i]);
#pragma unroll
    for (int i = 0; i < N; ++i) S[i] = mma(b[i].p[x], u1.p[y], S[i]);
  });
}

// Two row tiles of a staged triangular operand (fragments first, first + 1 of
// each plane times x0; with kBoth `second`, second + 1 times x1), added to c0,
// c1: a plane of it at a time, the smallest first.
template <int NP, bool kBoth, int NX>
__device__ inline void add_square(const char* slot, int lane, const int (&frag)[4],
                                  const Planes<NX>& x0, const Planes<NX>& x1, f32x4& c0,
                                  f32x4& c1) {
  f32x4 y0 = {}, y1 = {};
#pragma unroll
  for (int i = NP - 1; i >= 0; --i) {
    bf16x8 a[4];
#pragma unroll
    for (int n = 0; n < (kBoth ? 4 : 2); ++n)
      a[n] = lds_frag<1>(slot, i * 6 + frag[n], 0, lane).p[0];
#pragma unroll
    for (int j = NX - 1; j >= 0; --j)
      if (i + j < NP) {
        c0 = mma(a[0], x0.p[j], c0);
        c1 = mma(a[1], x0.p[j], c1);
        if (kBoth) {
          y0 = mma(a[2], x1.p[j], y0);
          y1 = mma(a[3], x1.p[j], y1);
        }
      }
  }
  if (kBoth) {
    c0 += y0;
    c1 += y1;
  }
}
// (fragments by low_pair: tiles 0, 1 of tokens 0-31; tiles 2, 3 of 0-31, of 32-63;
// by high_pair: tiles 0, 1 of 0-31, of 32-63; tiles 2, 3 of 32-63)
constexpr int kLowFirst[4] = {0, 1, 0, 0}, kLowSecond[4] = {2, 4, 3, 5};
constexpr int kHighFirst[4] = {0, 2, 1, 3}, kHighSecond[4] = {4, 5, 0, 0};

}  // namespace delta
}  // namespace mlstm
