// One token of the gated delta rule (generation).
//
// Per head, with the memory C (dv x dk, rows by value), f = sigma(f~) or
// exp(f~), and q^ = q / sqrt(dk):
//
//   u = beta (v - f C k),   C' = f C + u k^T,   h = C' q^ = f C q^ + u (k . q^)
//
// C k and C q^ are taken in one pass over a row of C, so the row is in
// registers once and written back once.  The step is bound by the memory's
// traffic, 8 dk dv bytes per head.  A row of dk floats is held by the smallest
// power of two of lanes that covers it at 16 bytes a lane (up to 64, then
// several vectors per lane), the wave's other lanes take further rows; a wave
// loads all its rows before it stores any, so C may be updated in place.
// Reductions are butterflies in a fixed order: bitwise reproducible.  64
// sequences of 16 heads of 128 x 128: 27 us a token, what a copy of the memories
// takes; one sequence of 4 heads of 64: 4 us of kernel, 12 us with the call.
#include <hip/hip_bf16.h>

#include "delta.h"

namespace mlstm {
namespace {

constexpr int kThreads = 256;

__device__ inline float load_elem(const float* p) { return *p; }
__device__ inline float load_elem(const __hip_bfloat16* p) { return __bfloat162float(*p); }
__device__ inline float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ inline float4 load4(const __hip_bfloat16* p) {
  const uint2 a = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xFFFF0000u),
                     __uint_as_float(a.y << 16), __uint_as_float(a.y & 0xFFFF0000u));
}
__device__ inline void store_elem(float* p, float x) { *p = x; }
__device__ inline void store_elem(__hip_bfloat16* p, float x) { *p = __float2bfloat16(x); }
__device__ inline float dot4(float4 a, float4 b) {
  return a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
}
// sigma(x) from e^-|x|: no overflow
__device__ inline float sigmoid(float x) {
  const float e = expf(-fabsf(x));
  return (x >= 0.0f ? 1.0f : e) / (1.0f + e);
}

// R rows at a time per group of 2^shift lanes, VPL vectors of 4 per lane
template <typename T, int VPL, int R>
__global__ __launch_bounds__(kThreads) void delta_step_kernel(
    const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
    const float* __restrict__ beta, const float* __restrict__ fgate, const float* C_in,
    float* C_out, T* __restrict__ h, int group, int dk, int dv, int shift, int blocks_per_head,
    float scale, int exp_forget) {
  const int64_t head = blockIdx.x / blocks_per_head;
  const int block = blockIdx.x % blocks_per_head;
  const int lane = threadIdx.x & ((1 << shift) - 1);
  const int side = threadIdx.x >> shift;          // of the workgroup's groups of lanes
  const int sides = kThreads >> shift;
  const int64_t row0 = int64_t(block) * sides * R + side;
  const int64_t key = head / group * dk;

  float4 c[R][VPL];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t i = row0 + int64_t(r) * sides;
#pragma unroll
    for (int u = 0; u < VPL; ++u) {
      const int j = 4 * (lane + (u << shift));
      c[r][u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (C_in && i < dv && j < dk) c[r][u] = load4(C_in + (head * dv + i) * dk + j);
    }
  }
  float4 kv[VPL], qv[VPL];
  float kq = 0.0f;
#pragma unroll
  for (int u = 0; u < VPL; ++u) {
    const int j = 4 * (lane + (u << shift));
    kv[u] = qv[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (j < dk) {
      kv[u] = load4(k + key + j);
      qv[u] = load4(q + key + j);
    }
    kq += dot4(kv[u], qv[u]);
  }
  const float x = fgate[head], f = exp_forget ? expf(x) : sigmoid(x), b = beta[head];
  float ck[R], cq[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    ck[r] = cq[r] = 0.0f;
#pragma unroll
    for (int u = 0; u < VPL; ++u) {
      ck[r] += dot4(c[r][u], kv[u]);
      cq[r] += dot4(c[r][u], qv[u]);
    }
  }
  for (int o = 0; o < shift; ++o) {
    kq += __shfl_xor(kq, 1 << o, 64);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      ck[r] += __shfl_xor(ck[r], 1 << o, 64);
      cq[r] += __shfl_xor(cq[r], 1 << o, 64);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t i = row0 + int64_t(r) * sides;
    if (i >= dv) break;
    const float u_i = b * (load_elem(v + head * dv + i) - f * ck[r]);
#pragma unroll
    for (int u = 0; u < VPL; ++u) {
      const int j = 4 * (lane + (u << shift));
      if (j < dk)
        *reinterpret_cast<float4*>(C_out + (head * dv + i) * dk + j) =
            make_float4(f * c[r][u].x + u_i * kv[u].x, f * c[r][u].y + u_i * kv[u].y,
                        f * c[r][u].z + u_i * kv[u].z, f * c[r][u].w + u_i * kv[u].w);
    }
    if (lane == 0) store_elem(h + head * dv + i, scale * (f * cq[r] + u_i * kq));
  }
}

template <typename T, int VPL, int R>
hipError_t launch(const DeltaShape& s, const void* q, const void* k, const void* v,
                  const float* beta, const float* fgate, const float* C_in, float* C_out, void* h,
                  int shift, hipStream_t stream) {
  const int rows = (kThreads >> shift) * R;
  const int blocks = int((s.dv + rows - 1) / rows);
  delta_step_kernel<T, VPL, R><<<unsigned(s.B * s.NH * blocks), kThreads, 0, stream>>>(
      static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v), beta, fgate,
      C_in, C_out, static_cast<T*>(h), int(s.NH / s.NHK), int(s.dk), int(s.dv), shift, blocks,
      1.0f / sqrtf(float(s.dk)), int(s.exp_forget));
  return hipGetLastError();
}

template <typename T>
hipError_t dispatch(const DeltaShape& s, const void* q, const void* k, const void* v,
                    const float* beta, const float* fgate, const float* C_in, float* C_out,
                    void* h, hipStream_t stream) {
  int shift = 2;
  while (shift < 6 && (4 << shift) < s.dk) ++shift;
  if (s.dk <= 256)
    return launch<T, 1, 4>(s, q, k, v, beta, fgate, C_in, C_out, h, shift, stream);
  return launch<T, 2, 4>(s, q, k, v, beta, fgate, C_in, C_out, h, shift, stream);
}

}  // namespace

hipError_t launch_delta_step(const DeltaShape& s, const void* q, const void* k, const void* v,
                             const float* beta, const float* fgate, const float* C_in,
                             float* C_out, void* h, hipStream_t stream) {
  if (s.is_bf16)
    return dispatch<__hip_bfloat16>(s, q, k, v, beta, fgate, C_in, C_out, h, stream);
  return dispatch<float>(s, q, k, v, beta, fgate, C_in, C_out, h, stream);
}

}  // namespace mlstm
