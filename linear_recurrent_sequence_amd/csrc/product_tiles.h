// Tiles of a matrix product on the bf16 matrix instruction, for the gated
// feed-forward: out[q][p] = sum_k L[p][k] R[q][k], both operands rows of k.
//
// A workgroup has BP x BQ outputs; its WP x WQ waves have a block each, in
// 16 x 16 accumulators.  The left operand's rows are the outputs' fast index, so
// a lane holds four neighbouring outputs of a row (lane l: q = l % 16, p = 4 (l /
// 16) ..) and stores them together.  Both operands' tiles of 64 columns are copied
// global -> LDS without registers into two buffers, the next tile's while one is
// multiplied; eight lanes copy a row of 128 bytes, and the 16-byte pieces of a row
// lie in the order piece ^ (row & 7), so that the 16 rows that an instruction's
// lanes read in one column do not share banks.  Rows beyond an operand's, and
// columns beyond k, are read out of the buffer's range: zeros.
//
// float32 operands come as three bf16 planes (24 bits: exact), and the product is
// the sum of the six plane products above 2^-24, taken one after the other as if k
// were six times as long, the smallest first: their roundings are then those of
// small sums.
#pragma once

#include "tile_common.h"

namespace mlstm {
namespace product {

using tilecommon::bf16x8;
using tilecommon::i32x4;
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kStep = 64;  // columns of a tile

// rows of k elements; planes of a float32 operand are `plane` elements apart
struct Operand {
  const uint16_t* p;
  int64_t rows, plane;
};

template <int BP, int BQ, int WP, int WQ>
struct Shape {
  static constexpr int kBP = BP, kBQ = BQ, kWP = WP, kWQ = WQ;
  static constexpr int kThreads = 64 * WP * WQ;
  static constexpr int kPassRows = kThreads / 8;  // rows that one copy of every thread covers
  static constexpr int kP = BP / WP / 16, kQ = BQ / WQ / 16;  // a wave's accumulators
  static constexpr int kBuffer = (BP + BQ) * kStep * 2;       // bytes
  static constexpr int kLds = 2 * kBuffer;
};

// The planes of term s of six (a bf16 operand has plane 0 only)
__device__ inline int left_plane(int s) { return (0x001102 >> (4 * s)) & 15; }   // 2 0 1 1 0 0
__device__ inline int right_plane(int s) { return (0x010120 >> (4 * s)) & 15; }  // 0 2 1 0 1 0

// workgroup -> tile.  Workgroups are dealt to the 8 XCDs round-robin: each XCD
// takes a run of neighbouring tiles, in blocks of 8 tiles of q whose operands its
// L2 then holds.
__device__ inline void map_tile(unsigned wg, unsigned np, unsigned nq, unsigned& ip, unsigned& iq) {
  const unsigned n = np * nq, x = wg & 7, i = wg >> 3;
  const unsigned each = n >> 3, more = n & 7;
  const unsigned at = x * each + (x < more ? x : more) + i;
  const unsigned block = at / (8 * np), in = at % (8 * np);
  const unsigned high = nq - 8 * block < 8 ? nq - 8 * block : 8;
  iq = 8 * block + in % high;
  ip = in / high;
}

// acc[i][j]: accumulators of the wave's p block i and q block j.  DUAL: the left
// rows are those of two operands in turn, a wave's first half of its blocks from L
// and the second half from L2, for the same output columns (BP / 2 of them from
// p0 on).
template <typename S, bool DUAL>
__device__ inline void multiply(const Operand& L, const Operand& L2, const Operand& R, int64_t k,
                                int terms, int64_t p0, int64_t q0, char* lds,
                                f32x4 (&acc)[S::kP][S::kQ]) {
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int wp = wave / S::kWQ, wq = wave % S::kWQ;
  // the copy of this lane: row threadIdx.x / 8 of a pass, LDS piece threadIdx.x % 8
  const int row = threadIdx.x / 8, piece = (threadIdx.x % 8) ^ (row & 7);
  const unsigned pitch = unsigned(k) * 2, at = row * pitch + piece * 16;
  const unsigned out = tilecommon::lds_addr(lds) + wave * 1024;
  const int steps = int((k + kStep - 1) / kStep);
  auto words = [&](const Operand& o, int64_t first, int plane) {
    const int64_t left = o.rows - first;
    return tilecommon::rsrc_words(o.p + plane * o.plane + first * k,
                                  left > 0 ? (left < 256 ? left : 256) * k * 2 : 0);
  };
  constexpr int kPassesP = S::kBP / S::kPassRows, kPassesQ = S::kBQ / S::kPassRows;
  constexpr int kHalf = DUAL ? S::kBP / S::kWP / 2 : 0;
  static_assert(!DUAL || kHalf == S::kPassRows, "a pass is of one operand");
  i32x4 left = {}, left2 = {}, right = {};
  auto copy = [&](int s, int step, int buffer) {
    if (step == 0) {
      const int lp = terms > 1 ? left_plane(s) : 0, rp = terms > 1 ? right_plane(s) : 0;
      left = words(L, p0, lp);
      if constexpr (DUAL) left2 = words(L2, p0, lp);
      right = words(R, q0, rp);
    }
    // columns beyond k (a multiple of 8) in the last tile
    const unsigned off =
        step * kStep + piece * 8 < k ? at + step * (kStep * 2) : tilecommon::kOutOfRange;
    const unsigned to = out + buffer * S::kBuffer;
#pragma unroll
    for (int i = 0; i < kPassesP; ++i) {
      const int first = DUAL ? i / 2 * S::kPassRows : i * S::kPassRows;
      tilecommon::copy16(DUAL && (i & 1) ? left2 : left, off + first * pitch,
                         to + i * S::kPassRows * 128);
    }
#pragma unroll
    for (int i = 0; i < kPassesQ; ++i)
      tilecommon::copy16(right, off + i * S::kPassRows * pitch,
                         to + (S::kBP + i * S::kPassRows) * 128);
  };
#pragma unroll
  for (int i = 0; i < S::kP; ++i)
#pragma unroll
    for (int j = 0; j < S::kQ; ++j) acc[i][j] = f32x4{};

  copy(0, 0, 0);
  int s = 0, step = 0, buffer = 0;
  for (;;) {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    int s1 = s, step1 = step + 1;
    if (step1 == steps) step1 = 0, ++s1;
    const bool more = s1 < terms;
    if (more) copy(s1, step1, buffer ^ 1);
    const char* base = lds + buffer * S::kBuffer;
    const char* lp = base + (wp * (S::kBP / S::kWP) + lane % 16) * 128;
    const char* rp = base + (S::kBP + wq * (S::kBQ / S::kWQ) + lane % 16) * 128;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const int slot = ((kk * 4 + lane / 16) ^ (lane & 7)) * 16;
      bf16x8 l[S::kP], r[S::kQ];
#pragma unroll
      for (int j = 0; j < S::kQ; ++j)
        r[j] = *reinterpret_cast<const bf16x8*>(rp + j * 16 * 128 + slot);
#pragma unroll
      for (int i = 0; i < S::kP; ++i)
        l[i] = *reinterpret_cast<const bf16x8*>(lp + i * 16 * 128 + slot);
#pragma unroll
      for (int i = 0; i < S::kP; ++i)
#pragma unroll
        for (int j = 0; j < S::kQ; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(l[i], r[j], acc[i][j], 0, 0, 0);
    }
    if (!more) break;
    s = s1, step = step1, buffer ^= 1;
  }
}

}  // namespace product
}  // namespace mlstm
