// Tiles of a matrix product on the bf16 matrix instruction, for the gated
// feed-forward: out[q][p] = sum_k L[p][k] R[q][k], both operands rows of k.
//
// A workgroup has BP x BQ outputs at a time; its WP x WQ waves have a block each,
// in 16 x 16 accumulators.  The left operand's rows are the outputs' fast index, so
// a lane holds four neighbouring outputs of a row (lane l: q = l % 16, p = 4 (l /
// 16) ..) and stores them together.  Both operands' pieces of 64 columns are copied
// global -> LDS without registers into two or three slots.  A wave reads the fragments
// of 32 columns into registers while it multiplies those of the 32 before, so a slot is
// free when half of its products are done, and is filled again, as many pieces ahead as
// there are slots, beside the other half's.  Workgroups stay for several tiles: the
// copies run on into the next tile, whose first pieces come in while this one is stored.  Eight
// lanes copy a row's 128 bytes, a cache line, and its 16-byte parts lie in the order
// part ^ (row & 7), so that the 16 rows that an instruction's lanes read in one
// column do not share banks.  Rows beyond an operand's, and columns beyond k, are
// read out of the buffer's range: zeros.
//
// Measured: 8192 x 16384 x 1536 with the gate's epilogue 330 us, 1250 TFLOP/s (the
// library's product alone 358 to 373); 2048 x 8192 x 11008 in two terms 550 us, 1340
// TFLOP/s.  Without copies the same loop takes 0.78 of the time, without
// products 0.77, without reads 0.95: the copies and the matrix unit are each other's
// limit.  Copies and reads spread over the products, at a raised wave priority, gave
// 4.5 % over copies in one burst.
//
// float32 operands come as three bf16 planes (24 bits: exact), and the product is
// the sum of the six plane products above 2^-24, taken one after the other as if k
// were six times as long, the smallest first: their roundings are then those of
// small sums.
#pragma once

#include "row_vec.h"
#include "tile_common.h"

namespace mlstm {
namespace product {

using tilecommon::bf16x8;
using tilecommon::i32x4;
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kStep = 64;  // columns of a piece

// rows of k elements; planes of a float32 operand are `plane` elements apart.  A
// right operand may be several groups of rows, `group` elements apart, each with
// tiles of its own.
struct Operand {
  const uint16_t* p;
  int64_t rows, plane, group;
};

template <int BP, int BQ, int WP, int WQ, int SLOTS>
struct Shape {
  static constexpr int kBP = BP, kBQ = BQ, kWP = WP, kWQ = WQ;
  static constexpr int kThreads = 64 * WP * WQ;
  static constexpr int kPassRows = kThreads / 8;  // rows that one copy of every thread covers
  static constexpr int kPassesP = BP / kPassRows, kPassesQ = BQ / kPassRows;
  static constexpr int kP = BP / WP / 16, kQ = BQ / WQ / 16;  // a wave's accumulators
  static constexpr int kSlot = (BP + BQ) * kStep * 2;         // bytes
  static constexpr int kSlots = SLOTS, kLds = SLOTS * kSlot;
};

// 16 bytes per lane from rsrc + voffset to LDS at dst + 16 * lane (dst is
// wave-uniform).  The wait is the caller's.  The wait states cover scalar registers
// that a vector instruction has just written (5).
__device__ inline void copy_piece(i32x4 rsrc, unsigned voffset, unsigned dst) {
  rsrc = tilecommon::sreg(rsrc);
  dst = tilecommon::sreg(dst);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(dst), "v"(voffset), "s"(rsrc)
               : "memory", "m0");
}

// The planes of term s of `terms`: six of two float32 operands, two of a bf16 one (left)
// with two planes of a float32 one, and one of two bf16 operands
__device__ inline int left_plane(int s, int terms) {
  return terms == 6 ? (0x001102 >> (4 * s)) & 15 : 0;  // 2 0 1 1 0 0
}
__device__ inline int right_plane(int s, int terms) {
  return terms == 6 ? (0x010120 >> (4 * s)) & 15 : terms - 1 - s;  // 0 2 1 0 1 0
}

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

// What a wave multiplies at a time: 32 columns of its rows
template <typename S>
struct Fragments {
  bf16x8 l[S::kP], r[S::kQ];
};

// The tiles of a product.  The first `whole` of np x nq are taken as they are; the
// others by `splits` workgroups each, with a share of the pieces, so that the CUs that
// the last round of tiles would leave idle have work.
struct Plan {
  unsigned np, nq, groups;  // nq / groups tiles of each of R's groups
  unsigned whole;
  int splits;
  __host__ __device__ unsigned tiles() const { return np * nq; }
  __host__ __device__ unsigned rest() const { return tiles() - whole; }
  __host__ __device__ unsigned items() const { return whole + rest() * unsigned(splits); }
};
// An item of the plan: a tile, and its share (-1: whole)
struct Item {
  unsigned tile;
  int split;
};
__device__ inline Item item_of(const Plan& p, unsigned i) {
  if (i < p.whole) return {i, -1};
  const unsigned r = i - p.whole;
  return {p.whole + r % p.rest(), p.splits > 1 ? int(r / p.rest()) : -1};
}

// The workgroup's items, one after the other; store(ip, iq, item, acc) with
// acc[i][j] the accumulators of the wave's p block i and q block j.  DUAL: the left
// rows are those of two operands in turn, a wave's first half of its blocks from L
// and the second half from L2, for the same output columns (BP / 2 to a tile).
// `store` issues STORES stores at least, whatever the tile: the completion of that many
// is not waited for with the next tile's first copies, which are older.
template <typename S, bool DUAL, int STORES, typename F>
__device__ inline void tiles(const Operand& L, const Operand& L2, const Operand& R, int64_t k,
                             int terms, const Plan& plan, char* lds, F&& store) {
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int wp = wave / S::kWQ, wq = wave % S::kWQ;
  const unsigned n = plan.items(), np = plan.np, nq = plan.nq, of_group = nq / plan.groups;
  const int steps = int((k + kStep - 1) / kStep), pieces = steps * terms;
  const int share = (pieces + plan.splits - 1) / plan.splits;  // none is without a piece
  auto first_of = [&](const Item& t) { return t.split < 0 ? 0 : t.split * share; };
  auto last_of = [&](const Item& t) {
    return t.split < 0 || (t.split + 1) * share > pieces ? pieces : (t.split + 1) * share;
  };

  // ---- copies: a cursor over the pieces of all tiles
  constexpr int kHalf = S::kBP / S::kWP / 2;  // DUAL: rows of one operand
  static_assert(kHalf % 8 == 0, "a wave's copy is of one operand");
  const int row = threadIdx.x / 8, part = (threadIdx.x % 8) ^ (row & 7);
  const unsigned pitch = unsigned(k) * 2, lane_at = (lane / 8) * pitch + part * 16;
  const unsigned out = tilecommon::lds_addr(lds) + wave * 1024;  // LDS
  auto words = [&](const Operand& o, int64_t first, int plane, unsigned group) {
    const int64_t left = o.rows - first;
    return tilecommon::rsrc_words(o.p + plane * o.plane + group * o.group + first * k,
                                  left > 0 ? (left < 256 ? left : 256) * k * 2 : 0);
  };
  i32x4 left = {}, left2 = {}, right = {};
  unsigned at = blockIdx.x;  // the item; there are no more workgroups than items
  Item item = item_of(plan, at);
  int piece = first_of(item), step = piece % steps, term = piece / steps, slot = 0;
  bool fresh = true;  // a tile, or a plane, begins
  // The next piece's copies, for which begin() makes ready; beyond the last tile
  // they read zeros, so that as many are in flight at any time.
  unsigned col = 0;
  bool in = false;
  auto begin = [&]() {
    if (fresh && at < n) {
      unsigned ip, iq;
      map_tile(item.tile, np, nq, ip, iq);
      const int64_t p0 = int64_t(ip) * (DUAL ? S::kBP / 2 : S::kBP), q0 = int64_t(iq % of_group) * S::kBQ;
      const int lp = left_plane(term, terms), rp = right_plane(term, terms);
      left = words(L, p0, lp, 0);
      if constexpr (DUAL) left2 = words(L2, p0, lp, 0);
      right = words(R, q0, rp, iq / of_group);
    }
    // columns beyond k (a multiple of 8) in a plane's last piece are zeros
    in = at < n && step * kStep + part * 8 < k;
    col = step * (kStep * 2);
    fresh = false;
    if (++step == steps) step = 0, ++term, fresh = true;
    if (at < n && ++piece == last_of(item)) {
      at += gridDim.x;
      fresh = true;
      if (at < n) {
        item = item_of(plan, at);
        piece = first_of(item), step = piece % steps, term = piece / steps;
      }
    }
  };
  auto copy = [&](int i) {  // pass i of kPassesP + kPassesQ
    const int first = i * S::kPassRows + wave * 8;
    const unsigned to = out + slot * S::kSlot + i * S::kPassRows * (kStep * 2);
    if (i < S::kPassesP) {
      const bool second = DUAL && (first / kHalf & 1);
      const int from = DUAL ? first / (2 * kHalf) * kHalf + first % kHalf : first;
      copy_piece(second ? left2 : left,
                 in ? lane_at + col + from * pitch : tilecommon::kOutOfRange, to);
    } else {
      const int from = first - S::kBP;
      copy_piece(right, in ? lane_at + col + from * pitch : tilecommon::kOutOfRange, to);
    }
  };
  constexpr int kCopies = S::kPassesP + S::kPassesQ;

  // ---- reads and products
  const int half[2] = {((lane / 16) ^ (lane & 7)) * 16, ((4 + lane / 16) ^ (lane & 7)) * 16};
  const char* lp = lds + (wp * (S::kBP / S::kWP) + lane % 16) * (kStep * 2);
  const char* rp = lds + (S::kBP + wq * (S::kBQ / S::kWQ) + lane % 16) * (kStep * 2);
  auto read_l = [&](int from, int h, int i, Fragments<S>& f) {
    f.l[i] = *reinterpret_cast<const bf16x8*>(lp + from * S::kSlot + i * 16 * (kStep * 2) + half[h]);
  };
  auto read_r = [&](int from, int h, int j, Fragments<S>& f) {
    f.r[j] = *reinterpret_cast<const bf16x8*>(rp + from * S::kSlot + j * 16 * (kStep * 2) + half[h]);
  };
  f32x4 acc[S::kP][S::kQ];
  // The products of `now`, and in turn with them the reads of half h of slot `from`
  // into `next`, and if `with` says so the next piece's copies.
  auto multiply = [&](const Fragments<S>& now, Fragments<S>& next, int from, int h, auto with) {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int i = 0; i < S::kP; ++i) {
      if constexpr (with()) {
#pragma unroll
        for (int c = i; c < kCopies; c += S::kP) copy(c);
      }
#pragma unroll
      for (int j = i; j < S::kQ; j += S::kP) read_r(from, h, j, next);
      read_l(from, h, i, next);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < S::kQ; ++j)
        acc[i][j] =
            __builtin_amdgcn_mfma_f32_16x16x32_bf16(now.l[i], now.r[j], acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_setprio(0);
  };
  // waits for this wave's copies but for the newest `left` operations, and its
  // reads, then for the workgroup's
  auto arrive = [&](auto newer) {
    static_assert(newer() < 64, "vmcnt has 6 bits");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(newer()) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

#pragma unroll
  for (int s = 0; s < S::kSlots; ++s) {
    begin();
#pragma unroll
    for (int i = 0; i < kCopies; ++i) copy(i);
    if (++slot == S::kSlots) slot = 0;
  }
  arrive(std::integral_constant<int, (S::kSlots - 1) * kCopies>{});
  Fragments<S> a, b;
#pragma unroll
  for (int j = 0; j < S::kQ; ++j) read_r(0, 0, j, a);
#pragma unroll
  for (int i = 0; i < S::kP; ++i) read_l(0, 0, i, a);
  bool stored = false;
  for (unsigned t = blockIdx.x; t < n; t += gridDim.x) {
#pragma unroll
    for (int i = 0; i < S::kP; ++i)
#pragma unroll
      for (int j = 0; j < S::kQ; ++j) acc[i][j] = f32x4{};
    const Item mine = item_of(plan, t);
    for (int s = last_of(mine) - first_of(mine); s > 0; --s) {
      multiply(a, b, slot, 1, std::false_type{});
      // this slot has been read, and the next one is whole; the copies behind that
      // one's, and after a tile the stores, may still be on their way
      constexpr int kNewer = (S::kSlots - 2) * kCopies;
      if (stored)
        arrive(std::integral_constant<int, kNewer + STORES>{});
      else
        arrive(std::integral_constant<int, kNewer>{});
      stored = false;
      begin();
      const int next = slot + 1 == S::kSlots ? 0 : slot + 1;
      multiply(b, a, next, 0, std::true_type{});
      slot = next;
    }
    unsigned ip, iq;
    map_tile(mine.tile, np, nq, ip, iq);
    store(ip, iq, mine, acc);
    stored = true;
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
}

// Where an item's share of a tile is kept: [split][tile of the rest][BQ][BP] float32
template <typename S>
__device__ inline float* share_at(const Plan& p, float* shares, const Item& item) {
  return shares + (int64_t(item.split) * p.rest() + (item.tile - p.whole)) * (S::kBP * S::kBQ);
}
// A wave's accumulators of a share
template <typename S, typename R>
__device__ inline void put_share(const R& rows, const f32x4 (&acc)[S::kP][S::kQ]) {
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int p = wave / S::kWQ * (S::kBP / S::kWP) + lane / 16 * 4,
            q = wave % S::kWQ * (S::kBQ / S::kWQ) + lane % 16;
#pragma unroll
  for (int j = 0; j < S::kQ; ++j)
#pragma unroll
    for (int i = 0; i < S::kP; ++i) rows.put(q + j * 16, p + i * 16, S::kBP, acc[i][j]);
}

// Rows of outputs, 256 at most, from `first` on.  Stores beyond the last row or a
// row's end are dropped, but issued all the same (see `tiles`).
template <typename T>
struct Rows {
  __amdgpu_buffer_rsrc_t rsrc;
  int width;
  __device__ Rows(T* base, int64_t first, int64_t rows, int width_)
      : rsrc(tilecommon::make_rsrc(
            base + first * width_,
            (rows - first < 256 ? rows - first : 256) * width_ * int64_t(sizeof(T)))),
        width(width_) {}
  // columns c .. c + 3 of row `first` + i, where c is below `columns`
  __device__ void put(int i, int c, int columns, f32x4 x) const {
    typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
    typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
    const unsigned at = c < columns ? unsigned(i * width + c) * unsigned(sizeof(T))
                                    : tilecommon::kOutOfRange;
    if constexpr (sizeof(T) == 4)
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), rsrc, at, 0, 0);
    else
      __builtin_amdgcn_raw_buffer_store_b64(
          u32x2{rowvec::to_bf16(x[0], x[1]), rowvec::to_bf16(x[2], x[3])}, rsrc, at, 0, 0);
  }
};

// Four float32 values as two bf16 planes, 16 bits of them
struct TwoPlanes {
  f32x4 high, low;  // rounded to bf16, and what is left
  __device__ explicit TwoPlanes(f32x4 x) {
    rowvec::Raw<__hip_bfloat16, 4> r;
    r.w[0] = rowvec::to_bf16(x[0], x[1]), r.w[1] = rowvec::to_bf16(x[2], x[3]);
    float h[4];
    rowvec::floats(r, h);
    high = f32x4{h[0], h[1], h[2], h[3]};
    low = x - high;
  }
};

}  // namespace product
}  // namespace mlstm
