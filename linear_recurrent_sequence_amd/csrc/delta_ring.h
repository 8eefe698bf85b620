// Staging of a chunk's left operands through LDS for the chain kernels of the
// gated delta rule.
//
// The four waves of a workgroup hold different value columns and read the same
// left operands, 1 KiB "fragments" (16 rows x 32 columns, 16 bytes per lane in
// the order of the matrix instruction's lanes).  A chunk is a fixed sequence of
// stages of at most kSlot bytes, copied global -> LDS without registers into a
// ring of kSlots slots, two stages ahead: at the start of a stage each wave
// waits for its own copies of that stage (vmcnt counts in order), a barrier
// makes them whole and ends the reads of the stage before, whose slot then
// takes the copies of the stage after next.  Every wave issues the same number
// of copies in each stage, so the counts are constants; behind the last chunk
// the copies repeat it.
#pragma once

#include "delta_common.h"
#include "tile_common.h"

namespace mlstm {
namespace delta {

using tilecommon::i32x4;
using tilecommon::static_for;

constexpr int kSlots = 3;
constexpr int kAhead = kSlots - 1;
constexpr int kFrag = 1024;  // bytes

// 16 bytes per lane from rsrc + voffset + soffset to LDS at dst + 16 * lane;
// dst and soffset are wave-uniform.  The wait is the caller's.
__device__ inline void copy_frag(i32x4 rsrc, unsigned voffset, unsigned soffset, unsigned dst) {
  rsrc = tilecommon::sreg(rsrc);
  dst = tilecommon::sreg(dst);
  soffset = tilecommon::sreg(soffset);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
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

// The (row tile, half) pairs of a lower triangular 64 x 64 left operand that
// are not zero, as indexes 2 i + s; of an upper triangular one likewise.
__device__ inline int low_pair(int n) { return n < 2 ? 2 * n : n + 2; }   // 0 2 4 5 6 7
__device__ inline int high_pair(int n) { return n < 4 ? n : 2 * n - 3; }  // 0 1 2 3 5 7

template <int N>
__device__ inline Planes<N> lds_frag(const char* slot, int first, int step, int lane) {
  Planes<N> s;
#pragma unroll
  for (int n = 0; n < N; ++n)
    s.p[n] = *reinterpret_cast<const bf16x8*>(slot + (first + n * step) * kFrag + lane * 16);
  return s;
}

}  // namespace delta
}  // namespace mlstm
