// Staging of a chunk's left operands through LDS for the chain kernels of the
// gated delta rule.
//
// The four waves of a workgroup hold different value columns and read the same
// left operands, 1 KiB "fragments" (16 rows x 32 columns, 16 bytes per lane in
// the order of the matrix instruction's lanes).  A chunk is a fixed sequence of
// stages of at most kSlot bytes, copied global -> LDS without registers into a
// ring of slots, up to a chunk ahead: at the start of a stage each copying wave
// waits for its own copies of that stage (vmcnt counts in order), a barrier
// makes them whole and ends the reads of the stage before, whose slot then
// takes the copies of a later stage.  Every copying wave issues the same number
// of copies in each stage, so the counts are constants; behind the last chunk
// the copies repeat it.  Four waves copy and four compute: a chain's wave has a
// SIMD almost to itself and is bound by the instructions it issues, and the
// copies' addresses are a quarter of them.
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

// c += L x for a lower triangular 64 x 64 left operand in a slot (planes six
// fragments apart) and x in the accumulators' order
template <int NP>
__device__ inline void low_product(const char* slot, const f32x4 (&x)[4], f32x4 (&c)[4], int lane) {
  Planes<NP> a[6];
#pragma unroll
  for (int n = 0; n < 6; ++n) a[n] = lds_frag<NP>(slot, n, 6, lane);
  const Planes<NP> b0 = split<NP>(pair(x[0], x[1])), b1 = split<NP>(pair(x[2], x[3]));
  f32x4 low[2] = {};  // rows 32 .. of the second half: accumulators of their own
  each_product<NP, NP, NP>([&](int i, int j) {
    c[0] = mma(a[0].p[i], b0.p[j], c[0]);
    c[1] = mma(a[1].p[i], b0.p[j], c[1]);
    c[2] = mma(a[2].p[i], b0.p[j], c[2]);
    c[3] = mma(a[4].p[i], b0.p[j], c[3]);
    low[0] = mma(a[3].p[i], b1.p[j], low[0]);
    low[1] = mma(a[5].p[i], b1.p[j], low[1]);
  });
  c[2] += low[0];
  c[3] += low[1];
}

}  // namespace delta
}  // namespace mlstm
