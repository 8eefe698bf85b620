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

#include <float.h>

#include "row_vec.h"
#include "mlstm_internal.h"
#include "scan_common.h"
#include "selective_scan.h"
#include "tile_common.h"

namespace mlstm {
namespace selective {

using rowvec::Raw;

constexpr int kChannels = 64;  // of a workgroup

// log(1 + e^x); its slope is sigma(x)
__device__ inline float softplus(float x) {
  return fmaxf(x, 0.0f) + scan::log1p_unit(rowvec::exp2_fast(-rowvec::kLog2e * fabsf(x)));
}

// A' of a rate. It stays finite, for a step of 0 to leave the state as it is: 0 times an
// infinite one would be no number.
__device__ inline float rate_of(float a) {
  const float x = a * rowvec::kLog2e;
  return fabsf(x) > FLT_MAX ? __builtin_copysignf(FLT_MAX, x) : x;
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

// ---- rows of a tile, by buffer loads and stores: what lies beyond the tile's last
// row reads as zeros and is not stored, and a lane's offset is the same for all tiles

// A tensor's rows of the current tile
struct Rows {
  const char* base;
  unsigned pitch;  // bytes
  // from element `first` of `row` on; `pitch` elements apart
  __device__ Rows(const void* p, int64_t row, int64_t pitch_, int64_t first, int element)
      : base(static_cast<const char*>(p) + (row * pitch_ + first) * element),
        pitch(unsigned(pitch_ * element)) {}
  __device__ void move(int rows) { base += int64_t(rows) * pitch; }
  // `rows` of them, 32 at most
  __device__ __amdgpu_buffer_rsrc_t rsrc(int rows) const {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, rows * pitch,
                                             tilecommon::kRsrcFlags);
  }
};
__device__ inline int rows_left(int64_t from, int64_t end) {
  return end <= from ? 0 : end - from < 32 ? int(end - from) : 32;
}
// of element c of row r, where `on`
__device__ inline unsigned offset_of(bool on, int64_t r, int64_t pitch, int64_t c, int element) {
  const unsigned at = unsigned((r * pitch + c) * element);
  return on ? at : tilecommon::kOutOfRange;
}
template <typename T, int V>
__device__ inline Raw<T, V> load_rows(__amdgpu_buffer_rsrc_t rsrc, unsigned at) {
  constexpr int kWords = sizeof(T) * V / 4;
  typedef unsigned words __attribute__((ext_vector_type(kWords < 4 ? kWords : 4)));
  Raw<T, V> r;
#pragma unroll
  for (int i = 0; i < kWords; i += 4) {
    if constexpr (kWords == 1) {
      r.w[0] = __builtin_amdgcn_raw_buffer_load_b32(rsrc, at, 0, 0);
    } else {
      words x;
      if constexpr (kWords == 2)
        x = __builtin_amdgcn_raw_buffer_load_b64(rsrc, at, 0, 0);
      else
        x = __builtin_amdgcn_raw_buffer_load_b128(rsrc, at + i * 4, 0, 0);
#pragma unroll
      for (int e = 0; e < kWords && e < 4; ++e) r.w[i + e] = x[e];
    }
  }
  return r;
}
template <typename T, int V>
__device__ inline void store_rows(__amdgpu_buffer_rsrc_t rsrc, unsigned at, const float (&x)[V]) {
  constexpr int kWords = sizeof(T) * V / 4;
  typedef unsigned words __attribute__((ext_vector_type(kWords < 4 ? kWords : 4)));
  unsigned w[kWords];
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    if constexpr (sizeof(T) == 4)
      w[i] = __float_as_uint(x[i]);
    else
      w[i] = rowvec::to_bf16(x[2 * i], x[2 * i + 1]);
  }
#pragma unroll
  for (int i = 0; i < kWords; i += 4) {
    if constexpr (kWords == 1) {
      __builtin_amdgcn_raw_buffer_store_b32(w[0], rsrc, at, 0, 0);
    } else {
      words v;
#pragma unroll
      for (int e = 0; e < kWords && e < 4; ++e) v[e] = w[i + e];
      if constexpr (kWords == 2)
        __builtin_amdgcn_raw_buffer_store_b64(v, rsrc, at, 0, 0);
      else
        __builtin_amdgcn_raw_buffer_store_b128(v, rsrc, at + i * 4, 0, 0);
    }
  }
}

// B and C of a tile, as float32 in LDS [token][wave][B: NS, C: NS], zeros for
// states beyond N and tokens from `end` on.  In two steps, so that the loads can
// be in flight while the tile before is worked on.
template <typename T, int NW, int NS, int TL>
struct Shared {
  static constexpr int kThreads = 64 * NW, kN = NW * NS, kItems = TL * kN / kThreads;
  static_assert(TL * kN % kThreads == 0, "every thread has as many");
  unsigned B[kItems], C[kItems];  // as loaded
  unsigned B_at[kItems], C_at[kItems];

  __device__ explicit Shared(const SelectiveScan& a) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int at = i * kThreads + threadIdx.x, t = at / kN, n = at % kN;
      B_at[i] = offset_of(n < a.N, t, a.B_row, n, sizeof(T));
      C_at[i] = offset_of(n < a.N, t, a.C_row, n, sizeof(T));
    }
  }

  __device__ static unsigned one(__amdgpu_buffer_rsrc_t rsrc, unsigned at) {
    if constexpr (sizeof(T) == 4)
      return __builtin_amdgcn_raw_buffer_load_b32(rsrc, at, 0, 0);
    else
      return __builtin_amdgcn_raw_buffer_load_b16(rsrc, at, 0, 0);
  }
  __device__ static float value(unsigned x) {
    return __uint_as_float(sizeof(T) == 4 ? x : x << 16);
  }
  __device__ void load(const Rows& b_rows, const Rows& c_rows, int rows) {
    const auto rb = b_rows.rsrc(rows), rc = c_rows.rsrc(rows);
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      B[i] = one(rb, B_at[i]);
      C[i] = one(rc, C_at[i]);
    }
  }
  __device__ void put(float* lds) const {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int at = i * kThreads + threadIdx.x, t = at / kN, n = at % kN;
      float* p = lds + (t * NW + n / NS) * 2 * NS + n % NS;
      p[0] = value(B[i]);
      p[NS] = value(C[i]);
    }
  }
};

// dt_bias and D of the workgroup's channels (0 where they are not given)
struct alignas(16) Constants {
  float bias[kChannels], skip[kChannels];
  __device__ void load(const SelectiveScan& a, const Channels& ch) {
    const int c = threadIdx.x;
    if (c >= kChannels) return;
    bias[c] = a.dt_bias && c < ch.count ? a.dt_bias[ch.first + c] : 0.0f;
    skip[c] = a.D && c < ch.count ? a.D[ch.first + c] : 0.0f;
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

// Delta of V channels of a row, from dt as read; 0 where the row is not `on`
// (softplus(-infinity) = 0)
template <int V>
__device__ inline void deltas(const float (&dt)[V], const float* bias, bool on, float (&d)[V]) {
  const float mask = on ? 0.0f : -INFINITY;
  float b[V];
  read(bias, b);
#pragma unroll
  for (int e = 0; e < V; ++e) d[e] = softplus(dt[e] + b[e] + mask);
}

// What a wave reads of a token: Delta, Delta u, B, and C if it is asked for
template <int NS, bool WITH_C>
struct Token {
  float2 d;
  float B[NS], C[WITH_C ? NS : 1];
  __device__ void load(const float2 (*steps)[kChannels], const float* shared, int waves, int wave,
                       int t, int lane) {
    d = steps[t][lane];
    const float* row = shared + (t * waves + wave) * 2 * NS;
    read(row, B);
    if constexpr (WITH_C) read(row + NS, C);
  }
};

// A wave's share of A', zeros beyond N and the workgroup's channels
template <int NS>
__device__ inline void load_rates(const SelectiveScan& a, const Channels& ch, int wave, int lane,
                                  float (&A)[NS]) {
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    const int64_t n = wave * NS + j;
    A[j] = lane < ch.count && n < a.N ? rate_of(a.A[(ch.first + lane) * a.N + n]) : 0.0f;
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

// ---- how the work is cut, forward and backward

constexpr int64_t kCUs = 256, kSimds = 4 * kCUs;

// Waves of four states each (eight beyond 32)
inline int waves_of(int64_t N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : 8; }
inline int64_t workgroups_of(const SelectiveScan& a) {
  return a.batch * a.G * tiles_of_group(a.channels, a.G);
}

// The time of `n` tiles of tokens of `waves` waves: a SIMD with two waves keeps its
// vector unit three quarters busy, with one little more than half.
inline double time_of(int64_t n, int64_t waves) {
  return double(n) * (waves <= kSimds ? 0.65 : double((waves + 2 * kSimds - 1) / (2 * kSimds)));
}

}  // namespace selective
}  // namespace mlstm
