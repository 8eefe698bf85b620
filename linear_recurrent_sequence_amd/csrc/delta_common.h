// Device pieces shared by the chunked kernels of the gated delta rule.
//
// Arithmetic.  The memory is held in float32 and a rounding of it to bf16
// would be carried from chunk to chunk, so a float32 operand of a matrix
// product is split into bf16 planes, x = hi + mid + lo (8 bits each, 24 in
// all: exact up to float32's own spacing), and the product is the sum of the
// planes' products on the bf16 matrix instruction, float32 accumulation.  A
// bf16 input needs one plane (three instructions against a float32 operand);
// two float32 operands take the six products above 2^-24: hh, hm, mh, mm, hl,
// lh.  Against the float32 matrix instruction, 1/16 of the bf16 one's rate,
// that is 5.3 and 2.7 times the rate for the same accuracy.
//
// Operand order.  A wave owns 16 value columns of a head and keeps its slice
// of the memory in the accumulators (float32, 16x16 tiles: lane l holds column
// l % 16 and rows 4 (l / 16) .. + 3).  Rows of a product are free to be
// permuted, so the left operand's rows are taken in the order `row_of`, which
// makes the accumulators of two neighbouring tiles the right operand (8
// consecutive rows 8 (l / 16) .. of 32) of the next product, with no exchange
// between lanes: the whole chain memory -> X -> memory stays in one wave's
// registers.  The left operands that a chunk shares between its value columns
// (the inverse, the scores, the transposed keys) are written once by a kernel
// over all chunks, in the order in which lanes load them.
#pragma once

#include <hip/hip_bf16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "delta.h"

namespace mlstm {
namespace delta {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

constexpr int kC = kDeltaChunk;  // 64 tokens

// the row of a 32-row block that the left operand's row m (0..15) of tile
// `half` (0, 1) holds: accumulator (half, lane group g, element r) is then row
// 8 g + 4 half + r
__device__ __host__ inline int row_of(int half, int m) {
  return (m >> 2) * 8 + half * 4 + (m & 3);
}

// The (row tile, half) pairs of a lower triangular 64 x 64 left operand that
// are not zero, as indexes 2 i + s; of an upper triangular one likewise.
__device__ inline int low_pair(int n) { return n < 2 ? 2 * n : n + 2; }   // 0 2 4 5 6 7
__device__ inline int high_pair(int n) { return n < 4 ? n : 2 * n - 3; }  // 0 1 2 3 5 7

__device__ inline f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// planes of 8 float32 values
template <int N>
struct Planes {
  bf16x8 p[N];
};
// two values to bf16, to nearest even, the first in the low half (one
// instruction; the compiler's own, since it has to see that a result of the
// matrix unit is read)
__device__ inline unsigned to_bf16(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(unsigned, __builtin_convertvector(f32x2{a, b}, bf16x2));
}
template <int N>
__device__ inline Planes<N> split(f32x8 x) {
  typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
  Planes<N> s;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    u32x4 u;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      u[e] = to_bf16(x[2 * e], x[2 * e + 1]);
      if (n + 1 < N) {
        x[2 * e] -= __uint_as_float(u[e] << 16);
        x[2 * e + 1] -= __uint_as_float(u[e] & 0xFFFF0000u);
      }
    }
    s.p[n] = __builtin_bit_cast(bf16x8, u);
  }
  return s;
}
__device__ inline f32x8 pair(f32x4 a, f32x4 b) {
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// c += a b over the products of planes above 2^-8 (NA + NB - 1 - ...): with
// `most` planes kept, products i + j < most; small ones first
template <int kMost, int NA, int NB>
__device__ inline f32x4 mma_planes(const Planes<NA>& a, const Planes<NB>& b, f32x4 c) {
#pragma unroll
  for (int s = kMost - 1; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int j = s - i;
      if (j >= 0 && j < NB) c = mma(a.p[i], b.p[j], c);
    }
  return c;
}

__device__ inline float load_elem(const float* p) { return *p; }
__device__ inline float load_elem(const __hip_bfloat16* p) { return __bfloat162float(*p); }
__device__ inline void store_elem(float* p, float x) { *p = x; }
__device__ inline void store_elem(__hip_bfloat16* p, float x) { *p = __float2bfloat16(x); }

__device__ inline float exp2_once(double x) { return __builtin_amdgcn_exp2f(float(x)); }

// log sigma(x) = min(x, 0) - log1p(exp(-|x|)) in float64.  -inf (an infinite
// or overflowing pre-activation: f = 0) is held at -1e4, whose exponential is
// 0 too, so that differences of sums stay numbers.
__device__ inline double log_forget(float x, int exp_forget) {
  const double v = double(x);
  const double f = exp_forget ? v : fmin(v, 0.0) - log1p(exp(-fabs(v)));
  return f < -1e4 ? -1e4 : f;  // NaN stays
}

// A chunk's log2-decay sums, one token per lane (inclusive, float64).
__device__ inline double chunk_decay(const float* fgate, int lane, int valid, int exp_forget) {
  double s = lane < valid ? log_forget(fgate[lane], exp_forget) : 0.0;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const double left = __shfl_up(s, o, 64);
    if (lane >= o) s += left;
  }
  return s * 1.4426950408889634;
}

// planes of 8 neighbouring elements of a row; zeros where off
template <int N>
__device__ inline Planes<N> load_row(const void* x, int64_t at, bool on);
template <>
__device__ inline Planes<1> load_row<1>(const void* x, int64_t at, bool on) {
  Planes<1> s;
  s.p[0] = bf16x8{};
  if (on) s.p[0] = *reinterpret_cast<const bf16x8*>(static_cast<const __bf16*>(x) + at);
  return s;
}
template <>
__device__ inline Planes<3> load_row<3>(const void* x, int64_t at, bool on) {
  f32x8 v = {};
  if (on) v = *reinterpret_cast<const f32x8*>(static_cast<const float*>(x) + at);
  return split<3>(v);
}

// the planes of a left operand in load order
template <int N>
__device__ inline Planes<N> load_frag(const __bf16* base, int64_t plane, int frag, int lane) {
  Planes<N> s;
#pragma unroll
  for (int n = 0; n < N; ++n)
    s.p[n] = *reinterpret_cast<const bf16x8*>(base + n * plane + (int64_t(frag) * 64 + lane) * 8);
  return s;
}

// x[i] with the same x in all lanes: the address is a scalar base and a 32-bit
// offset, one register instead of a pair for each access
template <typename T>
__device__ inline T& elem(T* x, unsigned i) {
  return *reinterpret_cast<T*>(
      reinterpret_cast<std::conditional_t<std::is_const<T>::value, const char, char>*>(x) +
      i * unsigned(sizeof(T)));
}
__device__ inline f32x4& elem4(float* x, unsigned i) {
  return *reinterpret_cast<f32x4*>(reinterpret_cast<char*>(x) + i * 4u);
}

// Transposes 4 registers over each 4 neighbouring lanes: lane j of a quad gets
// x[j] of its lanes 0 .. 3.
__device__ inline f32x4 quad_transpose(f32x4 x, int lane) {
  auto swap = [](float& a, float& b, bool odd, auto ctrl) {
    const float out = odd ? a : b;
    const float in = __int_as_float(__builtin_amdgcn_update_dpp(
        0, __float_as_int(out), decltype(ctrl)::value, 0xF, 0xF, true));
    a = odd ? in : a;
    b = odd ? b : in;
  };
  float a = x[0], b = x[1], c = x[2], d = x[3];
  const bool odd = lane & 1, high = lane & 2;
  swap(a, b, odd, std::integral_constant<int, 0xB1>{});  // lane ^ 1
  swap(c, d, odd, std::integral_constant<int, 0xB1>{});
  swap(a, c, high, std::integral_constant<int, 0x4E>{});  // lane ^ 2
  swap(b, d, high, std::integral_constant<int, 0x4E>{});
  return f32x4{a, b, c, d};
}

// sum over the 16 lanes of a row (every lane gets it), by DPP: lane i with
// i ^ 1, i ^ 2, 7 - i (of 8) and 15 - i
__device__ inline float row_sum(float x) {
  auto dpp = [](float v, auto ctrl) {
    return __int_as_float(
        __builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, 0xF, 0xF, true));
  };
  x += dpp(x, std::integral_constant<int, 0xB1>{});
  x += dpp(x, std::integral_constant<int, 0x4E>{});
  x += dpp(x, std::integral_constant<int, 0x141>{});
  x += dpp(x, std::integral_constant<int, 0x140>{});
  return x;
}

// sum over the lanes of a row up to this one
__device__ inline float row_prefix(float x) {
  auto dpp = [](float v, auto ctrl) {  // from the lane 1, 2, 4 or 8 before, 0 if there is none
    return __int_as_float(
        __builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, 0xF, 0xF, true));
  };
  x += dpp(x, std::integral_constant<int, 0x111>{});
  x += dpp(x, std::integral_constant<int, 0x112>{});
  x += dpp(x, std::integral_constant<int, 0x114>{});
  x += dpp(x, std::integral_constant<int, 0x118>{});
  return x;
}

// The products of planes i + j < kMost, small ones first, as one list: f(i, j)
// for each, so that a caller can run one product over independent accumulators
// before the next one (a dependent matrix instruction waits for the last).
template <int kMost, int NA, int NB, typename F>
__device__ inline void each_product(F&& f) {
#pragma unroll
  for (int s = kMost - 1; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (s - i >= 0 && s - i < NB) f(i, s - i);
}

// workgroups of one head on one XCD (they are dealt round-robin to the 8
// XCDs), so that what they share is read into one L2
__device__ inline void map_head(int64_t wg, int64_t H, int per_head, int64_t& head, int& block) {
  if ((H & 7) == 0) {
    const int64_t s = wg >> 3;
    head = (wg & 7) + 8 * (s / per_head);
    block = int(s % per_head);
  } else {
    head = wg / per_head;
    block = int(wg % per_head);
  }
}

// What the kernel over the chunks leaves for the others.  Counts of bf16
// elements of one chunk's planes; a plane of a 64 x 64 left operand is stored
// as [4 row tiles][2 halves of the columns][64 lanes][8], one of a K^T (dk x
// 64) as [2 ks row tiles][2][64][8], one of K (64 x dk) as [ks][4][64][8],
// with ks = ceil(dk / 32).
constexpr int kSquare = kC * kC;

struct Work {
  __bf16* inv;    // [H][chunks][3] planes of (I + At)^-1
  __bf16* invT;   // its transpose (backward)
  __bf16* score;  // [H][chunks][3] planes of P
  __bf16* scoreT; // its transpose (backward)
  __bf16* keyT;   // [HK][chunks][NPL] planes of K^T
  __bf16* queryT; // (backward)
  __bf16* key;    // [HK][chunks][3] planes of K, Q (float32 inputs)
  __bf16* query;
  float* decay;   // [H][chunks][3][64]: e^G, e^(G_C - G), beta (0 behind the end)
};

// What the backward keeps between its passes.
struct Saved {
  float* S;     // [H][chunks][dk][dv] memory at each chunk's start
  float* Z;     // [H][chunks][dk][dv] its gradient at each chunk's end
  float* X;     // [H][T][dv]
  float* Y;     // [H][T][dv] e^G S^T k, what the memory at the chunk's start predicts
  float* dR;    // [H][T][dv] (bf16 inputs: dV is rounded)
  float* KZ;    // [H][T][dv] e^(G_C - G) Z^T k (Layout::apart)
  float* part;  // [H][chunks][dv / 16][3][64] parts of the gates' gradients
  __bf16* pairs;  // [H][chunks][3][3] planes of B, B^T / sqrt(dk), -(N + N^T)
  float* gates;   // [H][chunks][2][64] what the pairs of tokens give to the gates, dbeta
  float* inner;   // [H][chunks][blocks of 128 dk] parts of <S, Z>
};

}  // namespace delta
}  // namespace mlstm
