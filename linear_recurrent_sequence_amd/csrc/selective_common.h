// Device pieces shared by the kernels of the selective scan.
//
// Per channel with N states, A' = A log2 e and Delta = softplus(dt + bias),
//
//   s_t = 2^(Delta_t A') s_{t-1} + (Delta_t u_t) B_t,   y_t = (C_t . s_t + D u_t) silu(z_t)
//
// A workgroup has 64 channels of one sequence, one to a lane, and its waves
// share the states: wave w has states NS w .. NS w + NS - 1 in registers, so B_t
// and C_t are the same for all lanes of a wave and come from LDS by broadcast,
// and no sum over states crosses lanes.  A tile of tokens is staged by all
// threads: Delta and Delta u (formed once per channel and token, whatever the
// number of states), B and C as float32.  The waves' shares of C.s go through
// LDS to the threads that store y, rows of 64 channels at a time.
#pragma once

#include "row_vec.h"
#include "mlstm_internal.h"
#include "scan_common.h"
#include "selective_scan.h"

namespace mlstm {
namespace selective {

using rowvec::Raw;

constexpr int kChannels = 64;  // of a workgroup

// log(1 + e^x); its slope is sigma(x)
__device__ inline float softplus(float x) {
  return fmaxf(x, 0.0f) + scan::log1p_unit(rowvec::exp2_fast(-rowvec::kLog2e * fabsf(x)));
}

// The channels of a workgroup: `tile` of all groups' tiles of 64
struct Channels {
  int64_t group, first;
  int count;  // of 64
};
__host__ __device__ inline int64_t tiles_of_group(int64_t channels, int64_t G) {
  return (channels / G + kChannels - 1) / kChannels;
}
__device__ inline Channels channels_of(const SelectiveScan& a, int64_t tile) {
  const int64_t per = a.channels / a.G, tiles = tiles_of_group(a.channels, a.G);
  const int64_t group = tile / tiles, at = (tile % tiles) * kChannels;
  return {group, group * per + at, int(per - at < kChannels ? per - at : kChannels)};
}

// A sequence cut into n segments of `tiles` tiles of tokens (the last one shorter)
struct Segments {
  int n;
  int64_t tiles;
};

// B and C of a tile, as float32 in LDS [token][wave][B: NS, C: NS], zeros for
// states beyond N and tokens from `end` on.  In two steps, so that the loads can
// be in flight while the tile before is worked on.
template <typename T, int NW, int NS, int TL>
struct Shared {
  static constexpr int kThreads = 64 * NW, kRow = 2 * NW * NS;
  static constexpr int kItems = TL * kRow / kThreads;
  static_assert(TL * kRow % kThreads == 0, "every thread has as many");
  T raw[kItems];

  __device__ void load(const SelectiveScan& a, int64_t b, int64_t group, int64_t t0, int64_t end) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int at = i * kThreads + threadIdx.x;
      const int t = at / kRow, k = at % kRow, n = k / (2 * NS) * NS + k % NS;
      const bool is_c = (k / NS) & 1;
      const T* p = static_cast<const T*>(is_c ? a.C : a.B) +
                   (b * a.T + t0 + t) * (is_c ? a.C_row : a.B_row) + group * a.N + n;
      raw[i] = t0 + t < end && n < a.N ? *p : T(0.0f);
    }
  }
  __device__ void put(float* lds) const {
#pragma unroll
    for (int i = 0; i < kItems; ++i) lds[i * kThreads + threadIdx.x] = rowvec::to_float(raw[i]);
  }
};

// NS neighbouring floats of LDS
template <int NS>
__device__ inline void read(const float* p, float (&x)[NS]) {
#pragma unroll
  for (int i = 0; i + 4 <= NS; i += 4) {
    const float4 f = *reinterpret_cast<const float4*>(p + i);
    x[i] = f.x, x[i + 1] = f.y, x[i + 2] = f.z, x[i + 3] = f.w;
  }
  if constexpr (NS == 2) {
    const float2 f = *reinterpret_cast<const float2*>(p);
    x[0] = f.x, x[1] = f.y;
  }
}

// A wave's share of A', zeros beyond N and the workgroup's channels
template <int NS>
__device__ inline void load_rates(const SelectiveScan& a, const Channels& ch, int wave, int lane,
                                  float (&A)[NS]) {
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    const int64_t n = wave * NS + j;
    A[j] = lane < ch.count && n < a.N ? a.A[(ch.first + lane) * a.N + n] * rowvec::kLog2e : 0.0f;
  }
}
// a state as callers keep it, [batch][channels][N]
template <int NS>
__device__ inline void load_state(const SelectiveScan& a, const float* x, int64_t b,
                                  const Channels& ch, int wave, int lane, float (&s)[NS]) {
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    const int64_t n = wave * NS + j;
    s[j] = x && lane < ch.count && n < a.N
               ? x[(b * a.channels + ch.first + lane) * a.N + n] : 0.0f;
  }
}
template <int NS>
__device__ inline void store_state(const SelectiveScan& a, float* x, int64_t b, const Channels& ch,
                                   int wave, int lane, const float (&s)[NS]) {
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    const int64_t n = wave * NS + j;
    if (lane < ch.count && n < a.N) x[(b * a.channels + ch.first + lane) * a.N + n] = s[j];
  }
}
// a state as the workspaces keep it, [N][channels] at x
template <int NS>
__device__ inline void load_kept(const SelectiveScan& a, const float* x, const Channels& ch,
                                 int wave, int lane, float (&s)[NS]) {
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    const int64_t n = wave * NS + j;
    s[j] = lane < ch.count && n < a.N ? x[n * a.channels + ch.first + lane] : 0.0f;
  }
}
template <int NS>
__device__ inline void store_kept(const SelectiveScan& a, float* x, const Channels& ch, int wave,
                                  int lane, const float (&s)[NS]) {
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    const int64_t n = wave * NS + j;
    if (lane < ch.count && n < a.N) x[n * a.channels + ch.first + lane] = s[j];
  }
}

inline size_t pad256(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace selective
}  // namespace mlstm
