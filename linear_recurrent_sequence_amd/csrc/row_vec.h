// Vectors of neighbouring channels of a row, and the activations, shared by the
// short convolution, the selective scan and the gated feed-forward.
#pragma once

#include <hip/hip_bf16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mlstm {
namespace rowvec {

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;

// V neighbouring elements as they lie in memory, where tensors are 16-byte aligned
template <typename T, int V>
struct alignas(sizeof(T) * V < 16 ? sizeof(T) * V : 16) Raw {
  unsigned w[sizeof(T) * V / 4];
};

template <typename T, int V>
__device__ inline Raw<T, V> load_raw(const T* p) {
  return *reinterpret_cast<const Raw<T, V>*>(p);
}
template <int V>
__device__ inline void floats(const Raw<float, V>& r, float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = __uint_as_float(r.w[i]);
}
template <int V>
__device__ inline void floats(const Raw<__hip_bfloat16, V>& r, float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    x[2 * i] = __uint_as_float(r.w[i] << 16);
    x[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
  }
}
template <typename T, int V>
__device__ inline void load(const T* p, float (&x)[V]) {
  floats(load_raw<T, V>(p), x);
}
// two values to bf16, to nearest even, the first in the low half
__device__ inline unsigned to_bf16(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(unsigned, __builtin_convertvector(f32x2{a, b}, bf16x2));
}
template <int V>
__device__ inline void store(float* p, const float (&x)[V]) {
  Raw<float, V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.w[i] = __float_as_uint(x[i]);
  *reinterpret_cast<Raw<float, V>*>(p) = r;
}
template <int V>
__device__ inline void store(__hip_bfloat16* p, const float (&x)[V]) {
  Raw<__hip_bfloat16, V> r;
#pragma unroll
  for (int i = 0; i < V / 2; ++i) r.w[i] = to_bf16(x[2 * i], x[2 * i + 1]);
  *reinterpret_cast<Raw<__hip_bfloat16, V>*>(p) = r;
}
__device__ inline float to_float(float x) { return x; }
__device__ inline float to_float(__hip_bfloat16 x) { return __bfloat162float(x); }
__device__ inline void put(float* p, float x) { *p = x; }
__device__ inline void put(__hip_bfloat16* p, float x) {
  *reinterpret_cast<unsigned short*>(p) = static_cast<unsigned short>(to_bf16(x, 0.0f));
}

// 2^x, and 1 / (1 + e^-x): the hardware's exponential and reciprocal are good to
// one unit in the last place, and the exponent's own rounding adds |x| 2^-24.
__device__ inline float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ inline float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + exp2_fast(-kLog2e * x));
}
// d(x sigma(x)) / dx, from sigma(x)
__device__ inline float silu_slope(float x, float sig) {
  return sig * __builtin_fmaf(x, 1.0f - sig, 1.0f);
}

// A sequence's length: `lengths` may be NULL, and what it holds is kept in [0, T]
__device__ inline int64_t length_of(const int32_t* lengths, int64_t b, int64_t T) {
  if (!lengths) return T;
  const int64_t n = lengths[b];
  return n < 0 ? 0 : n > T ? T : n;
}

}  // namespace rowvec
}  // namespace mlstm
