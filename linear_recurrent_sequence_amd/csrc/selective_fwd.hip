// The selective scan over a sequence.
//
// Bound by the vector unit: a state and token take a product, an exponential (a quarter
// of the rate) and three more, 8 issue slots, for 1/8 of a byte.  Measured, bf16, N = 16,
// gate: 8 x 2048 x 1536 177 us in a settled trace (192 workgroups on as many CUs, the unit
// there 73 % busy; at full rate on all CUs the states alone would take 82), 1 x 16384 x
// 2048 121 us for the effects of 15 of 16 segments, 5 to join them and 157 for the scan.  Blocks of four
// tokens whose LDS reads are issued a block ahead and whose exponentials come first gave
// 192 -> 175 us (calls) on the first and 358 -> 285 on the second.
#include "selective_common.h"

namespace mlstm {
namespace selective {
namespace {

constexpr int kTile = 32;  // tokens

// The ends of segments, and then the states before them.
struct Joints {
  float* states;  // [segment][batch][N][channels]
  float* deltas;  // [segment][batch][channels]: the sum of Delta
  __device__ float* state(const SelectiveScan& a, int64_t seg, int64_t b) const {
    return states + (seg * a.batch + b) * a.N * a.channels;
  }
  __device__ float* delta(const SelectiveScan& a, int64_t seg, int64_t b) const {
    return deltas + (seg * a.batch + b) * a.channels;
  }
};

// ENDS: a segment's effect from a state of zeros, and the sum of its Delta.
// Otherwise: y, and the state after the last segment.
template <typename T, int NW, int NS, bool GATE, bool ENDS>
__global__ __launch_bounds__(64 * NW) void scan_kernel(SelectiveScan a, T* y, float* state_out,
                                                       Segments seg, Joints joints) {
  constexpr int TL = kTile, kThreads = 64 * NW;
  constexpr int V = NW < 8 ? 8 : 4, kVecs = kChannels / V;
  constexpr int kItems = TL * kVecs / kThreads;
  static_assert(TL * kVecs % kThreads == 0, "every thread has as many");
  __shared__ float2 steps[TL][kChannels];  // Delta, Delta u
  __shared__ __align__(16) float shared[TL * 2 * NW * NS];
  __shared__ __align__(16) float parts[ENDS ? 1 : NW][ENDS ? 1 : TL][kChannels];
  __shared__ Constants constants;

  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t tiles = a.G * tiles_of_group(a.channels, a.G);
  const Channels ch = channels_of(a, blockIdx.x % tiles);
  const int64_t segments = ENDS ? seg.n - 1 : seg.n;
  const int64_t s_at = blockIdx.x / tiles % segments, b = blockIdx.x / tiles / segments;
  const int64_t first = s_at * seg.tiles * TL;
  const int64_t last = first + seg.tiles * TL < a.T ? first + seg.tiles * TL : a.T;
  const int64_t n = rowvec::length_of(a.lengths, b, a.T);

  float A[NS], s[NS];
  load_rates(a, ch, wave, lane, A);
  if constexpr (ENDS) {
#pragma unroll
    for (int j = 0; j < NS; ++j) s[j] = 0.0f;
  } else if (seg.n > 1) {
    load_kept(a, joints.state(a, s_at, b), ch, wave, lane, s);
  } else {
    load_state(a, a.state, b, ch, wave, lane, s);
  }
  float sum = 0.0f;

  Raw<T, V> u[kItems], dt[kItems], z[kItems];
  Shared<T, NW, NS, TL> bc(a);
  auto vec_of = [&](int i) { return (i * kThreads + int(threadIdx.x)) % kVecs * V; };
  auto row_of = [&](int i) { return (i * kThreads + int(threadIdx.x)) / kVecs; };
  const int64_t end = n < last ? n : last;  // of what is read
  constexpr int kSize = sizeof(T);
  unsigned u_at[kItems], dt_at[kItems], z_at[kItems], y_at[kItems];
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const bool on = vec_of(i) < ch.count;
    u_at[i] = offset_of(on, row_of(i), a.u_row, vec_of(i), kSize);
    dt_at[i] = offset_of(on, row_of(i), a.dt_row, vec_of(i), kSize);
    z_at[i] = offset_of(on, row_of(i), a.gate_row, vec_of(i), kSize);
    y_at[i] = offset_of(on, row_of(i), a.channels, vec_of(i), kSize);
  }
  const int64_t row0 = b * a.T + first;
  Rows u_rows(a.u, row0, a.u_row, ch.first, kSize), dt_rows(a.dt, row0, a.dt_row, ch.first, kSize),
      z_rows(a.gate, row0, a.gate_row, ch.first, kSize),
      y_rows(y, row0, a.channels, ch.first, kSize),
      b_rows(a.B, row0, a.B_row, ch.group * a.N, kSize),
      c_rows(a.C, row0, a.C_row, ch.group * a.N, kSize);
  auto load = [&](int64_t t0) {  // and on to the next tile
    const int rows = rows_left(t0, end);
    const auto ru = u_rows.rsrc(rows), rd = dt_rows.rsrc(rows), rz = z_rows.rsrc(rows);
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      u[i] = load_rows<T, V>(ru, u_at[i]);
      dt[i] = load_rows<T, V>(rd, dt_at[i]);
      if constexpr (GATE && !ENDS) z[i] = load_rows<T, V>(rz, z_at[i]);
    }
    bc.load(b_rows, c_rows, rows);
    u_rows.move(TL), dt_rows.move(TL), z_rows.move(TL), b_rows.move(TL), c_rows.move(TL);
  };

  constants.load(a, ch);
  load(first);
  __syncthreads();
  for (int64_t t0 = first; t0 < last; t0 += TL) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const bool on = t0 + row_of(i) < end;
      float x[V], v[V], d[V];
      rowvec::floats(dt[i], x);
      rowvec::floats(u[i], v);
      deltas(x, constants.bias + vec_of(i), on, d);
#pragma unroll
      for (int e = 0; e < V; ++e)
        steps[row_of(i)][vec_of(i) + e] = make_float2(d[e], d[e] * v[e]);
    }
    bc.put(shared);
    __syncthreads();
    Raw<T, V> u0[kItems], z0[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) u0[i] = u[i], z0[i] = z[i];
    if (t0 + TL < last) load(t0 + TL);

    // kBlock tokens at a time, the next ones' data read beside them
    constexpr int kBlock = NS <= 4 ? 4 : 2;
    Token<NS, !ENDS> now[kBlock], next[kBlock];
#pragma unroll
    for (int k = 0; k < kBlock; ++k) now[k].load(steps, shared, NW, wave, k, lane);
#pragma unroll
    for (int t = 0; t < TL; t += kBlock) {
      if (t + kBlock < TL)
#pragma unroll
        for (int k = 0; k < kBlock; ++k)
          next[k].load(steps, shared, NW, wave, t + kBlock + k, lane);
      __builtin_amdgcn_sched_barrier(0);
      float decay[kBlock][NS];
#pragma unroll
      for (int k = 0; k < kBlock; ++k)
#pragma unroll
        for (int j = 0; j < NS; ++j) decay[k][j] = rowvec::exp2_fast(now[k].d.x * A[j]);
#pragma unroll
      for (int k = 0; k < kBlock; ++k) {
        float p = 0.0f;
        if constexpr (ENDS) sum += now[k].d.x;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          s[j] = __builtin_fmaf(decay[k][j], s[j], now[k].d.y * now[k].B[j]);
          if constexpr (!ENDS) p = __builtin_fmaf(now[k].C[j], s[j], p);
        }
        if constexpr (!ENDS) parts[wave][t + k][lane] = p;
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = 0; k < kBlock; ++k) now[k] = next[k];
    }
    __syncthreads();
    if constexpr (!ENDS) {
      const auto ry = y_rows.rsrc(rows_left(t0, last));
      y_rows.move(TL);
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        float o[V], x[V];
        rowvec::floats(u0[i], x);
        read(constants.skip + vec_of(i), o);
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] *= x[e];
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          float part[V];
          read(&parts[w][row_of(i)][vec_of(i)], part);
#pragma unroll
          for (int e = 0; e < V; ++e) o[e] += part[e];
        }
        if constexpr (GATE) {
          rowvec::floats(z0[i], x);
#pragma unroll
          for (int e = 0; e < V; ++e) o[e] *= x[e] * rowvec::sigmoid(x[e]);
        }
        store_rows<T, V>(ry, y_at[i], o);
      }
    }
  }
  if constexpr (ENDS) {
    store_kept(a, joints.state(a, s_at, b), ch, wave, lane, s);
    if (wave == 0 && lane < ch.count) joints.delta(a, s_at, b)[ch.first + lane] = sum;
  } else if (s_at == seg.n - 1) {
    store_state(a, state_out, b, ch, wave, lane, s);
  }
}

// the state before each segment, in the place of the segment's end (of which the
// first pass leaves that of the last one out)
__global__ __launch_bounds__(256) void join_kernel(SelectiveScan a, Joints joints, int segments) {
  const int64_t all = a.N * a.channels, blocks = (all + 255) / 256;
  const int64_t b = blockIdx.x / blocks, i = (blockIdx.x % blocks) * 256 + threadIdx.x;
  if (i >= all) return;
  const int64_t c = i % a.channels, n = i / a.channels;
  const float A = rate_of(a.A[c * a.N + n]);
  float s = a.state ? a.state[(b * a.channels + c) * a.N + n] : 0.0f;
  constexpr int kAhead = 8;  // segments whose loads are in flight together
  for (int k0 = 0; k0 < segments; k0 += kAhead) {
    float end[kAhead], decay[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int k = k0 + j < segments - 1 ? k0 + j : 0;  // the last one's end is not needed
      end[j] = joints.state(a, k, b)[i];
      decay[j] = joints.delta(a, k, b)[c];
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (k0 + j >= segments) break;
      joints.state(a, k0 + j, b)[i] = s;
      s = __builtin_fmaf(rowvec::exp2_fast(A * decay[j]), s, end[j]);
    }
  }
}

// How many segments: those of a sequence run side by side, for the effect of each
// on a state (0.8 of the scan's time) taken first.  Both sides: 1 x 16384 x 2048 in 16
// segments 312 us, in 8 (one wave to a SIMD) 466, of one build; float32 2 x 555 x 208 in
// nine 34, in one piece 88.
Segments segments_of(const SelectiveScan& a) {
  const int64_t tiles = (a.T + kTile - 1) / kTile, waves = workgroups_of(a) * waves_of(a.N);
  Segments best = {1, tiles};
  double least = time_of(tiles, waves);
  for (int n = 2; n <= 64 && n * 2 <= tiles; ++n) {
    const int64_t len = (tiles + n - 1) / n;
    if ((tiles + len - 1) / len != n) continue;
    const double t = time_of(len, waves * n) + 0.8 * time_of(len, waves * (n - 1)) + 6.0;
    if (t < 0.9 * least) {
      least = t;
      best = {n, len};
    }
  }
  return best;
}

size_t state_bytes(const SelectiveScan& a, int n) {
  return align256(size_t(n) * size_t(a.batch * a.N * a.channels) * 4);
}

template <typename T, int NW, int NS, bool GATE>
void launch(const SelectiveScan& a, void* y, float* state_out, const Segments& seg,
            const Joints& joints, hipStream_t stream) {
  const int64_t per = workgroups_of(a);
  if (seg.n > 1) {
    scan_kernel<T, NW, NS, false, true><<<unsigned(per * (seg.n - 1)), 64 * NW, 0, stream>>>(
        a, nullptr, nullptr, seg, joints);
    join_kernel<<<unsigned(a.batch * ((a.N * a.channels + 255) / 256)), 256, 0, stream>>>(
        a, joints, seg.n);
  }
  scan_kernel<T, NW, NS, GATE, false><<<unsigned(per * seg.n), 64 * NW, 0, stream>>>(
      a, static_cast<T*>(y), state_out, seg, joints);
}

template <typename T, bool GATE>
void dispatch(const SelectiveScan& a, void* y, float* state_out, const Segments& seg,
              const Joints& joints, hipStream_t stream) {
  // two states to a wave where that gives a CU's one workgroup more waves: 8 x 2048 x
  // 1536 262 us with four, 201 with two
  const bool few = workgroups_of(a) * seg.n <= kCUs;
  if (few && a.N <= 4)
    launch<T, 2, 2, GATE>(a, y, state_out, seg, joints, stream);
  else if (few && a.N <= 8)
    launch<T, 4, 2, GATE>(a, y, state_out, seg, joints, stream);
  else if (few && a.N <= 16)
    launch<T, 8, 2, GATE>(a, y, state_out, seg, joints, stream);
  else if (a.N <= 4)
    launch<T, 1, 4, GATE>(a, y, state_out, seg, joints, stream);
  else if (a.N <= 8)
    launch<T, 2, 4, GATE>(a, y, state_out, seg, joints, stream);
  else if (a.N <= 16)
    launch<T, 4, 4, GATE>(a, y, state_out, seg, joints, stream);
  else if (a.N <= 32)
    launch<T, 8, 4, GATE>(a, y, state_out, seg, joints, stream);
  else
    launch<T, 8, 8, GATE>(a, y, state_out, seg, joints, stream);
}

}  // namespace
}  // namespace selective

size_t selective_fwd_workspace_bytes(const SelectiveScan& a) {
  const selective::Segments seg = selective::segments_of(a);
  if (seg.n == 1) return 0;
  return selective::state_bytes(a, seg.n) +
         align256(size_t(seg.n) * size_t(a.batch * a.channels) * 4);
}

hipError_t launch_selective_fwd(const SelectiveScan& a, void* y, float* state_out, void* workspace,
                                hipStream_t stream) {
  using namespace selective;
  const Segments seg = segments_of(a);
  char* ws = static_cast<char*>(workspace);
  Joints joints = {nullptr, nullptr};
  if (seg.n > 1)
    joints = {reinterpret_cast<float*>(ws), reinterpret_cast<float*>(ws + state_bytes(a, seg.n))};
  if (a.is_bf16) {
    if (a.gate)
      dispatch<__hip_bfloat16, true>(a, y, state_out, seg, joints, stream);
    else
      dispatch<__hip_bfloat16, false>(a, y, state_out, seg, joints, stream);
  } else {
    if (a.gate)
      dispatch<float, true>(a, y, state_out, seg, joints, stream);
    else
      dispatch<float, false>(a, y, state_out, seg, joints, stream);
  }
  return hipGetLastError();
}

}  // namespace mlstm
