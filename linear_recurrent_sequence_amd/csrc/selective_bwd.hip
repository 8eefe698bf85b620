// Gradients of the selective scan.
//
// With S_t the gradient of the state after token t (y_t's share of it included),
// g_t = dy_t silu(z_t) and a_t = exp(Delta_t A),
//
//   S_t = g_t C_t + a_{t+1} S_{t+1}              h_t = sum_n S_t B_t
//   f_t = S_t a_t s_{t-1}  (per state)           q_t = sum_n f_t A
//   du = D g + Delta h,   dDelta = q + u h,      ddt = dDelta sigma(dt + bias)
//   dA = sum_t f_t Delta_t,   dB_t = sum_c S_t Delta_t u_t,   dC_t = sum_c g_t s_t
//   dz = dy (C.s + D u) silu'(z),   dD = sum g u,   dbias = sum ddt
//
// Two passes over the tokens, in tiles.  The first goes forward and keeps the
// state before each tile.  The second takes the tiles from the last to the first:
// forward through a tile with its states s_t and a_t in registers (128 of them a
// lane), then back through it.  The products behind dC and dB take the registers
// of s_t and a_t as those are done with; at the tile's end the 128 of a wave are
// summed over its 64 channels by a halving butterfly (126 additions, two sums left
// on each lane), written per 64 channels, and summed over them by a small kernel.
// Sums over tokens (dA, dD, dbias) stay in registers and are joined over sequences
// and segments the same way.  No atomics: results are bitwise reproducible.
//
// A sequence of few channels is cut into segments side by side: the first pass
// then starts each from zeros and also takes what a segment makes of its own g
// for the gradient of the state before it (with the running product of a_t), a
// small kernel joins both, and the second pass adds what the state before the
// segment has become, exp(A sum Delta), to the states it kept.
//
// Bound by the vector unit.  Measured, bf16, N = 16, gate, 8 x 2048 x 1536 in 8 segments:
// first pass 123 us (unit 97 % busy), second 372 (83 %; 26 instructions a state and
// token: 5 forward, 10 back, 4.4 of the butterfly, the rest per token), sums 20.  With a
// tile's LDS reads kept over both ways and the sums sunk behind them, the second pass
// needed 440 registers and took 549 us on one wave to a SIMD; with its rows' addresses
// formed for every tile 514.
#include "selective_common.h"

namespace mlstm {
namespace selective {
namespace {

struct Kept {
  float* states;   // [batch][tile][N][channels]: the state before each tile
  float* sums;     // [batch][tile][channels]: Delta from the segment's start to the tile
  // of each segment [segment][batch][N][channels], and the sum of its Delta
  float* before;   // its effect on a state of zeros, then the state before it
  float* after;    // its share of the gradient before it, then the gradient after it
  float* deltas;   // [segment][batch][channels]
  float* weights;  // [segment][batch][N + 2][channels]: dA, dD, dbias
  float2* shared;  // [channel tile][batch][T][N]: dB, dC
};

template <int NW, int NS, int TL>
struct Vec {  // channels of a thread's vector in a tile
  static constexpr int V = TL * kChannels / (64 * NW) >= 8 ? 8 : TL * kChannels / (64 * NW) >= 4
                                                              ? 4 : 2;
};

struct Where {
  Channels ch;
  int64_t b, seg, first, last, n;
};
template <int TL>
__device__ inline Where where(const SelectiveScan& a, const Segments& seg) {
  const int64_t tiles = a.G * tiles_of_group(a.channels, a.G);
  Where w;
  w.ch = channels_of(a, blockIdx.x % tiles);
  w.seg = blockIdx.x / tiles % seg.n;
  w.b = blockIdx.x / tiles / seg.n;
  w.first = w.seg * seg.tiles * TL;
  w.last = w.first + seg.tiles * TL < a.T ? w.first + seg.tiles * TL : a.T;
  w.n = rowvec::length_of(a.lengths, w.b, a.T);
  return w;
}

// The offsets of a thread's vectors in a tile's rows
template <int ITEMS>
struct Offsets {
  unsigned u[ITEMS], dt[ITEMS], z[ITEMS], row[ITEMS];
  __device__ Offsets(const SelectiveScan& a, const Channels& ch, int tokens, int vec, int vecs,
                     int threads, int size) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int at = i * threads + threadIdx.x, r = at / vecs, c = at % vecs * vec;
      const bool on = r < tokens && c < ch.count;
      u[i] = offset_of(on, r, a.u_row, c, size);
      dt[i] = offset_of(on, r, a.dt_row, c, size);
      z[i] = offset_of(on, r, a.gate_row, c, size);
      row[i] = offset_of(on, r, a.channels, c, size);
    }
  }
};

struct Inputs {
  Rows u, dt, z, dy, b, c;
  __device__ Inputs(const SelectiveScan& a, const void* dy_, const Channels& ch, int64_t row,
                    int size)
      : u(a.u, row, a.u_row, ch.first, size), dt(a.dt, row, a.dt_row, ch.first, size),
        z(a.gate, row, a.gate_row, ch.first, size), dy(dy_, row, a.channels, ch.first, size),
        b(a.B, row, a.B_row, ch.group * a.N, size), c(a.C, row, a.C_row, ch.group * a.N, size) {}
  __device__ void move(int rows) {
    u.move(rows), dt.move(rows), z.move(rows), dy.move(rows), b.move(rows), c.move(rows);
  }
};

// ---- the first pass

template <typename T, int NW, int NS, int TL, bool GATE, bool CUT>
__global__ __launch_bounds__(64 * NW) void states_kernel(SelectiveScan a, const void* dy,
                                                         Segments seg, Kept kept) {
  constexpr int kThreads = 64 * NW, V = Vec<NW, NS, TL>::V, kVecs = kChannels / V;
  constexpr int kItems = (TL * kVecs + kThreads - 1) / kThreads;
  __shared__ float2 steps[TL][kChannels];                    // Delta, Delta u
  __shared__ float gs[CUT ? TL : 1][kChannels];              // g
  __shared__ __align__(16) float shared[TL * 2 * NW * NS];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const Where w = where<TL>(a, seg);
  const int64_t tiles = (a.T + TL - 1) / TL;

  float A[NS], s[NS], P[NS], S[NS], sum = 0.0f;
  load_rates(a, w.ch, wave, lane, A);
  load_state(a, CUT ? nullptr : a.state, w.b, w.ch, wave, lane, s);
#pragma unroll
  for (int j = 0; j < NS; ++j) P[j] = 1.0f, S[j] = 0.0f;

  Raw<T, V> u[kItems], dt[kItems], z[kItems], d[kItems];
  Shared<T, NW, NS, TL> bc(a);
  auto vec_of = [&](int i) { return (i * kThreads + int(threadIdx.x)) % kVecs * V; };
  auto row_of = [&](int i) { return (i * kThreads + int(threadIdx.x)) / kVecs; };
  const int64_t end = w.n < w.last ? w.n : w.last;
  constexpr int kSize = sizeof(T);
  const Offsets<kItems> at(a, w.ch, TL, V, kVecs, kThreads, kSize);
  Inputs in(a, dy, w.ch, w.b * a.T + w.first, kSize);
  auto load = [&](int64_t t0) {  // and on to the next tile
    const int rows = rows_left(t0, end);
    const auto ru = in.u.rsrc(rows), rt = in.dt.rsrc(rows), rd = in.dy.rsrc(rows),
               rz = in.z.rsrc(rows);
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      u[i] = load_rows<T, V>(ru, at.u[i]);
      dt[i] = load_rows<T, V>(rt, at.dt[i]);
      if constexpr (CUT) d[i] = load_rows<T, V>(rd, at.row[i]);
      if constexpr (CUT && GATE) z[i] = load_rows<T, V>(rz, at.z[i]);
    }
    bc.load(in.b, in.c, rows);
    in.move(TL);
  };
  __shared__ Constants constants;
  constants.load(a, w.ch);
  load(w.first);
  __syncthreads();
  for (int64_t t0 = w.first; t0 < w.last; t0 += TL) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      if (row_of(i) >= TL) continue;
      const bool on = t0 + row_of(i) < end;
      float x[V], v[V], dl[V];
      rowvec::floats(dt[i], x);
      rowvec::floats(u[i], v);
      deltas(x, constants.bias + vec_of(i), on, dl);
#pragma unroll
      for (int e = 0; e < V; ++e)
        steps[row_of(i)][vec_of(i) + e] = make_float2(dl[e], dl[e] * v[e]);
      if constexpr (CUT) {
        rowvec::floats(d[i], x);
        if constexpr (GATE) {
          rowvec::floats(z[i], v);
#pragma unroll
          for (int e = 0; e < V; ++e) x[e] *= v[e] * rowvec::sigmoid(v[e]);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) gs[row_of(i)][vec_of(i) + e] = x[e];
      }
    }
    bc.put(shared);
    __syncthreads();
    const int64_t tile = w.b * tiles + t0 / TL;
    store_kept(a, kept.states + tile * a.N * a.channels, w.ch, wave, lane, s);
    if (CUT && wave == 0 && lane < w.ch.count)
      kept.sums[tile * a.channels + w.ch.first + lane] = sum;
    if (t0 + TL < w.last) load(t0 + TL);
    // kBlock tokens at a time, the next ones' data read beside them
    constexpr int kBlock = NS <= 4 && !CUT ? 4 : 2;
    Token<NS, CUT> now[kBlock], next[kBlock];
    float g[kBlock], g_next[kBlock];
    auto fetch = [&](Token<NS, CUT>(&to)[kBlock], float(&to_g)[kBlock], int t) {
#pragma unroll
      for (int k = 0; k < kBlock; ++k) {
        to[k].load(steps, shared, NW, wave, t + k, lane);
        to_g[k] = CUT ? gs[CUT ? t + k : 0][lane] : 0.0f;
      }
    };
    fetch(now, g, 0);
#pragma unroll
    for (int t = 0; t < TL; t += kBlock) {
      if (t + kBlock < TL) fetch(next, g_next, t + kBlock);
      __builtin_amdgcn_sched_barrier(0);
      float decay[kBlock][NS];
#pragma unroll
      for (int k = 0; k < kBlock; ++k)
#pragma unroll
        for (int j = 0; j < NS; ++j) decay[k][j] = rowvec::exp2_fast(now[k].d.x * A[j]);
#pragma unroll
      for (int k = 0; k < kBlock; ++k) {
        if constexpr (CUT) sum += now[k].d.x;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          s[j] = __builtin_fmaf(decay[k][j], s[j], now[k].d.y * now[k].B[j]);
          if constexpr (CUT) {
            P[j] *= decay[k][j];
            S[j] = __builtin_fmaf(P[j], now[k].C[j] * g[k], S[j]);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = 0; k < kBlock; ++k) now[k] = next[k], g[k] = g_next[k];
    }
    __syncthreads();
  }
  if constexpr (CUT) {
    const int64_t at = w.seg * a.batch + w.b;
    store_kept(a, kept.before + at * a.N * a.channels, w.ch, wave, lane, s);
    store_kept(a, kept.after + at * a.N * a.channels, w.ch, wave, lane, S);
    if (wave == 0 && lane < w.ch.count) kept.deltas[at * a.channels + w.ch.first + lane] = sum;
  }
}

// the state before and the gradient after each segment, in place
__global__ __launch_bounds__(256) void join_kernel(SelectiveScan a, const float* dstate, Kept kept,
                                                   int segments) {
  const int64_t all = a.N * a.channels, blocks = (all + 255) / 256;
  const int64_t b = blockIdx.x / blocks, i = (blockIdx.x % blocks) * 256 + threadIdx.x;
  if (i >= all) return;
  const int64_t c = i % a.channels, n = i / a.channels, at = (b * a.channels + c) * a.N + n;
  const float A = rate_of(a.A[c * a.N + n]);
  auto kept_at = [&](int k) { return (k * a.batch + b) * all + i; };
  constexpr int kAhead = 8;  // segments whose loads are in flight together
  // x, with each segment's share added to what is left of it, in the order of `at`
  auto join = [&](float* shares, float x, auto at) {
    for (int k0 = 0; k0 < segments; k0 += kAhead) {
      float own[kAhead], decay[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int k = at(k0 + j < segments ? k0 + j : k0);
        own[j] = shares[kept_at(k)];
        decay[j] = kept.deltas[(k * a.batch + b) * a.channels + c];
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (k0 + j >= segments) break;
        shares[kept_at(at(k0 + j))] = x;
        x = __builtin_fmaf(rowvec::exp2_fast(A * decay[j]), x, own[j]);
      }
    }
  };
  join(kept.before, a.state ? a.state[at] : 0.0f, [](int k) { return k; });
  join(kept.after, dstate ? dstate[at] : 0.0f, [&](int k) { return segments - 1 - k; });
}

// ---- the second pass

// x[i] of 128 summed over the wave's lanes; lane l is left with those of i = 2 l
// and 2 l + 1, in x[0] and x[1].  Each step halves the values: a lane keeps the
// half of its own bit and gives the other to the lane across.
template <int CTRL>
__device__ inline float across(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, true));
}
template <int CTRL, int HALF>
__device__ inline void halve(float (&x)[128], bool upper) {
#pragma unroll
  for (int i = 0; i < HALF; ++i) {
    const float keep = upper ? x[i + HALF] : x[i], give = upper ? x[i] : x[i + HALF];
    x[i] = keep + across<CTRL>(give);
  }
}
__device__ inline void channel_sums(float (&x)[128], int lane) {
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x[i]),
                                                    __float_as_uint(x[i + 64]), false, false);
    x[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x[i]),
                                                    __float_as_uint(x[i + 32]), false, false);
    x[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  halve<0x128, 16>(x, lane & 8);  // row_ror:8
  halve<0x141, 8>(x, lane & 4);   // row_half_mirror: the other lanes of a quad follow
  halve<0x4E, 4>(x, lane & 2);    // quad_perm, lanes ^ 2
  halve<0xB1, 2>(x, lane & 1);    // lanes ^ 1
}

template <typename T, int NW, int NS, int TL, bool GATE, bool CUT>
__global__ __launch_bounds__(64 * NW, NW == 8 ? 1 : 2) void grads_kernel(SelectiveScan a, SelectiveGrads gr,
                                                        Segments seg, Kept kept) {
  static_assert(NS * TL == 64, "a wave's products of a tile are 128 to a lane");
  constexpr int kThreads = 64 * NW, V = Vec<NW, NS, TL>::V, kVecs = kChannels / V;
  constexpr int kItems = (TL * kVecs + kThreads - 1) / kThreads;
  constexpr int kParts = GATE ? 3 : 2;  // h, q, and C.s behind dz
  __shared__ float2 steps[TL][kChannels];
  __shared__ float gs[TL][kChannels];
  __shared__ __align__(16) float shared[TL * 2 * NW * NS];
  __shared__ __align__(16) float parts[kParts][NW][TL][kChannels];
  // what a thread read of the tile, for its end: registers are for the next one's
  __shared__ __align__(16) Raw<T, V> held[GATE ? 4 : 3][kItems][kThreads];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const Where w = where<TL>(a, seg);
  const int64_t tiles = (a.T + TL - 1) / TL, end = w.n < w.last ? w.n : w.last;

  float A[NS], dA[NS], S[NS], s0[NS];
  load_rates(a, w.ch, wave, lane, A);
#pragma unroll
  for (int j = 0; j < NS; ++j) dA[j] = 0.0f;
  if constexpr (CUT) {
    const int64_t at = (w.seg * a.batch + w.b) * a.N * a.channels;
    load_kept(a, kept.after + at, w.ch, wave, lane, S);
    load_kept(a, kept.before + at, w.ch, wave, lane, s0);
  } else {
    load_state(a, gr.dstate, w.b, w.ch, wave, lane, S);
  }
  float dD[kItems][V] = {}, dbias[kItems][V] = {};

  Raw<T, V> u[kItems], dt[kItems], z[kItems], d[kItems];
  Shared<T, NW, NS, TL> bc(a);
  float s[NS], sum = 0.0f;
  auto vec_of = [&](int i) { return (i * kThreads + int(threadIdx.x)) % kVecs * V; };
  auto row_of = [&](int i) { return (i * kThreads + int(threadIdx.x)) / kVecs; };
  constexpr int kSize = sizeof(T);
  const Offsets<kItems> at(a, w.ch, TL, V, kVecs, kThreads, kSize);
  int64_t t0 = w.first + (w.last - 1 - w.first) / TL * TL;  // the last tile
  Inputs in(a, gr.dy, w.ch, w.b * a.T + t0, kSize);
  auto load = [&](int64_t t0) {  // and on to the tile before
    const int rows = rows_left(t0, end);
    const auto ru = in.u.rsrc(rows), rt = in.dt.rsrc(rows), rd = in.dy.rsrc(rows),
               rz = in.z.rsrc(rows);
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      u[i] = load_rows<T, V>(ru, at.u[i]);
      dt[i] = load_rows<T, V>(rt, at.dt[i]);
      d[i] = load_rows<T, V>(rd, at.row[i]);
      if constexpr (GATE) z[i] = load_rows<T, V>(rz, at.z[i]);
    }
    bc.load(in.b, in.c, rows);
    in.move(-TL);
    const int64_t tile = w.b * tiles + t0 / TL;
    load_kept(a, kept.states + tile * a.N * a.channels, w.ch, wave, lane, s);
    if (CUT) sum = lane < w.ch.count ? kept.sums[tile * a.channels + w.ch.first + lane] : 0.0f;
  };

  const int64_t row0 = w.b * a.T + t0;
  Rows du_rows(gr.du, row0, a.channels, w.ch.first, kSize),
      ddt_rows(gr.ddt, row0, a.channels, w.ch.first, kSize),
      dz_rows(gr.dgate, row0, a.channels, w.ch.first, kSize);
  __shared__ Constants constants;
  constants.load(a, w.ch);
  load(t0);
  __syncthreads();
  for (; t0 >= w.first; t0 -= TL) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      if (row_of(i) >= TL) continue;
      const bool on = t0 + row_of(i) < end;
      float x[V], v[V], dl[V];
      rowvec::floats(dt[i], x);
      rowvec::floats(u[i], v);
      deltas(x, constants.bias + vec_of(i), on, dl);
#pragma unroll
      for (int e = 0; e < V; ++e)
        steps[row_of(i)][vec_of(i) + e] = make_float2(dl[e], dl[e] * v[e]);
      rowvec::floats(d[i], x);
      if constexpr (GATE) {
        rowvec::floats(z[i], v);
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] *= v[e] * rowvec::sigmoid(v[e]);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) gs[row_of(i)][vec_of(i) + e] = x[e];
      held[0][i][threadIdx.x] = u[i];
      held[1][i][threadIdx.x] = dt[i];
      held[2][i][threadIdx.x] = d[i];
      if constexpr (GATE) held[3][i][threadIdx.x] = z[i];
    }
    bc.put(shared);
    float start[NS], own[NS], through = 0.0f;
#pragma unroll
    for (int j = 0; j < NS; ++j)
      start[j] = CUT ? __builtin_fmaf(rowvec::exp2_fast(A[j] * sum), s0[j], s[j]) : s[j];
    __syncthreads();
    if (t0 > w.first) load(t0 - TL);

    float x[128];  // [token][state]: s and a, then the products behind dB and dC
    float now[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) now[j] = start[j], own[j] = 0.0f;
#pragma unroll
    for (int t = 0; t < TL; ++t) {
      const float2 st = steps[t][lane];
      const float* row = shared + (t * NW + wave) * 2 * NS;
      float B[NS], C[NS], p = 0.0f;
      read(row, B);
      if constexpr (GATE) read(row + NS, C);
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        const float e = rowvec::exp2_fast(st.x * A[j]);
        now[j] = __builtin_fmaf(e, now[j], st.y * B[j]);
        if constexpr (GATE) p = __builtin_fmaf(C[j], now[j], p);
        x[2 * (t * NS + j)] = e;
        x[2 * (t * NS + j) + 1] = now[j];
      }
      if constexpr (GATE) parts[2][wave][t][lane] = p;
      through += st.x;
      if (t % 4 == 3) __builtin_amdgcn_sched_barrier(0);
    }
    // the way back reads LDS again: kept from here, what it reads would take all the
    // registers that are left
    asm volatile("" ::: "memory");
    // what the tile's own g make of the gradient before it, beside the gradient
    // itself: that of the tokens behind then takes one rounded factor a tile, not one a
    // token, and what is left of it after thousands of tokens stays exact
    float last[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) last[j] = S[j];
#pragma unroll
    for (int t = TL - 1; t >= 0; --t) {
      const float2 st = steps[t][lane];
      const float gt = gs[t][lane];
      const float* row = shared + (t * NW + wave) * 2 * NS;
      float B[NS], C[NS], h = 0.0f, q = 0.0f;
      read(row, B);
      read(row + NS, C);
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        const int at = 2 * (t * NS + j);
        const float here = x[at + 1], old = t > 0 ? x[t > 0 ? at + 1 - 2 * NS : 0] : start[j];
        S[j] = __builtin_fmaf(gt, C[j], S[j]);
        own[j] = __builtin_fmaf(gt, C[j], own[j]) * x[at];
        h = __builtin_fmaf(S[j], B[j], h);
        const float e = S[j] * x[at], f = e * old;
        q = __builtin_fmaf(f, A[j], q);
        dA[j] = __builtin_fmaf(f, st.x, dA[j]);
        x[at] = S[j] * st.y;
        x[at + 1] = gt * here;
        S[j] = e;
      }
      parts[0][wave][t][lane] = h;
      parts[1][wave][t][lane] = q * rowvec::kLn2;  // A' is A log2 e
      // here, not where they are needed: their operands would have to be kept
#pragma unroll
      for (int j = 0; j < NS; ++j) asm volatile("" : "+v"(dA[j]), "+v"(own[j]));
      if (t % 4 == 0) __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int j = 0; j < NS; ++j)
      S[j] = __builtin_fmaf(rowvec::exp2_fast(A[j] * through), last[j], own[j]);
    channel_sums(x, lane);
    {
      const int64_t t = t0 + lane / NS, n = wave * NS + lane % NS;
      if (t < w.last && n < a.N)
        kept.shared[((blockIdx.x % (a.G * tiles_of_group(a.channels, a.G)) * a.batch + w.b) * a.T +
                     t) * a.N + n] = make_float2(x[0], x[1]);
    }
    __syncthreads();
    const int rows = rows_left(t0, w.last);
    const auto ru = du_rows.rsrc(rows), rt = ddt_rows.rsrc(rows), rz = dz_rows.rsrc(rows);
    du_rows.move(-TL), ddt_rows.move(-TL), dz_rows.move(-TL);
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int r = row_of(i), v0 = vec_of(i);
      if (r >= TL) continue;
      float uu[V], h[V] = {}, q[V] = {}, o[V];
      rowvec::floats(held[0][i][threadIdx.x], uu);
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        float ph[V], pq[V];
        read(&parts[0][k][r][v0], ph);
        read(&parts[1][k][r][v0], pq);
#pragma unroll
        for (int e = 0; e < V; ++e) h[e] += ph[e], q[e] += pq[e];
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float g = gs[r][v0 + e];  // this thread's own
        o[e] = __builtin_fmaf(steps[r][v0 + e].x, h[e], constants.skip[v0 + e] * g);
        dD[i][e] = __builtin_fmaf(g, uu[e], dD[i][e]);
      }
      store_rows<T, V>(ru, at.row[i], o);
      float pre[V];
      rowvec::floats(held[1][i][threadIdx.x], pre);
      const bool on = t0 + r < end;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float slope = on ? rowvec::sigmoid(pre[e] + constants.bias[v0 + e]) : 0.0f;
        // (q of a rate near the largest number may be infinite where there is no step)
        o[e] = slope != 0.0f ? __builtin_fmaf(uu[e], h[e], q[e]) * slope : 0.0f;
        dbias[i][e] += o[e];
      }
      store_rows<T, V>(rt, at.row[i], o);
      if constexpr (GATE) {
        float zz[V], dd[V];
        rowvec::floats(held[3][i][threadIdx.x], zz);
        rowvec::floats(held[2][i][threadIdx.x], dd);
        float raw[V];
        read(constants.skip + v0, raw);
#pragma unroll
        for (int e = 0; e < V; ++e) raw[e] *= uu[e];
#pragma unroll
        for (int k = 0; k < NW; ++k) {
          float part[V];
          read(&parts[2][k][r][v0], part);
#pragma unroll
          for (int e = 0; e < V; ++e) raw[e] += part[e];
        }
#pragma unroll
        for (int e = 0; e < V; ++e)
          o[e] = dd[e] * raw[e] * rowvec::silu_slope(zz[e], rowvec::sigmoid(zz[e]));
        store_rows<T, V>(rz, at.row[i], o);
      }
    }
  }
  __syncthreads();

  if (w.seg == 0 && gr.dstate_out) store_state(a, gr.dstate_out, w.b, w.ch, wave, lane, S);
  float* sums = kept.weights + (w.seg * a.batch + w.b) * (a.N + 2) * a.channels;
  store_kept(a, sums, w.ch, wave, lane, dA);
  // dD and dbias over the rows of the tile's threads, in order
  float(*rows)[kChannels] = parts[0][0];  // TL of them
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int i = 0; i < kItems; ++i)
      if (row_of(i) < TL)
#pragma unroll
        for (int e = 0; e < V; ++e)
          rows[row_of(i)][vec_of(i) + e] = k == 0 ? dD[i][e] : dbias[i][e];
    __syncthreads();
    if (int(threadIdx.x) < w.ch.count) {
      float v = 0.0f;
      for (int r = 0; r < TL; ++r) v += rows[r][threadIdx.x];
      sums[(a.N + k) * a.channels + w.ch.first + threadIdx.x] = v;
    }
    __syncthreads();
  }
}

// dB and dC: sums over the channel tiles of each group
template <typename T>
__global__ __launch_bounds__(256) void shared_sums_kernel(SelectiveScan a, const float2* parts,
                                                          T* dB, T* dC) {
  const int64_t rows = a.batch * a.T, all = rows * a.G * a.N;
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= all) return;
  const int64_t n = i % a.N, group = i / a.N % a.G, row = i / a.N / a.G;
  const int64_t tiles = tiles_of_group(a.channels, a.G);
  float b = 0.0f, c = 0.0f;
  const float2* p = parts + (group * tiles * rows + row) * a.N + n;
  for (int64_t k = 0; k < tiles; ++k, p += rows * a.N) b += p->x, c += p->y;
  rowvec::put(dB + i, b);
  rowvec::put(dC + i, c);
}

// dA, dD and dbias: sums over sequences and segments; a workgroup takes 32 columns,
// its eight rows of lanes every eighth partial, joined in order
__global__ __launch_bounds__(256) void weight_sums_kernel(SelectiveScan a, const float* parts,
                                                          int64_t n, float* dA, float* dD,
                                                          float* dbias) {
  __shared__ float sums[8][32];
  const int lane = threadIdx.x % 32, first = threadIdx.x / 32;
  const int64_t all = (a.N + 2) * a.channels, i = int64_t(blockIdx.x) * 32 + lane;
  float s = 0.0f;
  if (i < all)
    for (int64_t k = first; k < n; k += 8) s += parts[k * all + i];
  sums[first][lane] = s;
  __syncthreads();
  if (first != 0 || i >= all) return;
  for (int r = 1; r < 8; ++r) s += sums[r][lane];
  const int64_t row = i / a.channels, c = i % a.channels;
  if (row < a.N)
    dA[c * a.N + row] = s;
  else if (row == a.N && dD)
    dD[c] = s;
  else if (row == a.N + 1 && dbias)
    dbias[c] = s;
}

int tile_of(int64_t N) { return N <= 32 ? 16 : 8; }

// How many segments: operations to a state and token are 27 in one piece, 30 cut;
// see time_of.  Both sides, first and second pass, of one build: 8 x 2048 x
// 1536 in 8 segments 665 us, in 4 (one and a half rounds of workgroups) 722; float32 2 x
// 555 x 208 in 12 43, in 7 61.
Segments segments_of(const SelectiveScan& a) {
  const int64_t tiles = (a.T + tile_of(a.N) - 1) / tile_of(a.N);
  const int64_t waves = workgroups_of(a) * waves_of(a.N);
  Segments best = {1, tiles};
  double least = 27.0 * time_of(tiles, waves);
  for (int n = 2; n <= 64 && n * 2 <= tiles; ++n) {
    const int64_t len = (tiles + n - 1) / n;
    if ((tiles + len - 1) / len != n) continue;
    const double t = 30.0 * time_of(len, waves * n) + 60.0;
    if (t < 0.95 * least) {
      least = t;
      best = {n, len};
    }
  }
  return best;
}

// The workspace's parts, from `base` on; returns its size.
size_t lay_out(const SelectiveScan& a, const Segments& seg, char* base, Kept* k) {
  size_t at = 0;
  auto take = [&](size_t floats) {
    float* p = reinterpret_cast<float*>(base + at);
    at += align256(floats * 4);
    return p;
  };
  const size_t tiles = size_t((a.T + tile_of(a.N) - 1) / tile_of(a.N)), batch = size_t(a.batch),
               C = size_t(a.channels), N = size_t(a.N), n = size_t(seg.n);
  Kept x = {};
  x.states = take(batch * tiles * N * C);
  if (seg.n > 1) {
    x.sums = take(batch * tiles * C);
    x.before = take(n * batch * N * C);
    x.after = take(n * batch * N * C);
    x.deltas = take(n * batch * C);
  }
  x.weights = take(n * batch * (N + 2) * C);
  x.shared = reinterpret_cast<float2*>(
      take(size_t(a.G * tiles_of_group(a.channels, a.G)) * batch * size_t(a.T) * N * 2));
  if (k) *k = x;
  return at;
}

template <typename T, int NW, int NS, int TL, bool GATE, bool CUT>
void launch(const SelectiveScan& a, const SelectiveGrads& g, const Segments& seg, const Kept& kept,
            hipStream_t stream) {
  const unsigned wgs = unsigned(workgroups_of(a) * seg.n);
  states_kernel<T, NW, NS, TL, GATE, CUT><<<wgs, 64 * NW, 0, stream>>>(a, g.dy, seg, kept);
  if (CUT)
    join_kernel<<<unsigned(a.batch * ((a.N * a.channels + 255) / 256)), 256, 0, stream>>>(
        a, g.dstate, kept, seg.n);
  grads_kernel<T, NW, NS, TL, GATE, CUT><<<wgs, 64 * NW, 0, stream>>>(a, g, seg, kept);
}

template <typename T, bool GATE, bool CUT>
void by_states(const SelectiveScan& a, const SelectiveGrads& g, const Segments& seg,
               const Kept& kept, hipStream_t stream) {
  if (a.N <= 4)
    launch<T, 1, 4, 16, GATE, CUT>(a, g, seg, kept, stream);
  else if (a.N <= 8)
    launch<T, 2, 4, 16, GATE, CUT>(a, g, seg, kept, stream);
  else if (a.N <= 16)
    launch<T, 4, 4, 16, GATE, CUT>(a, g, seg, kept, stream);
  else if (a.N <= 32)
    launch<T, 8, 4, 16, GATE, CUT>(a, g, seg, kept, stream);
  else
    launch<T, 8, 8, 8, GATE, CUT>(a, g, seg, kept, stream);
}

template <typename T>
void dispatch(const SelectiveScan& a, const SelectiveGrads& g, const Segments& seg,
              const Kept& kept, hipStream_t stream) {
  if (a.gate && seg.n > 1)
    by_states<T, true, true>(a, g, seg, kept, stream);
  else if (a.gate)
    by_states<T, true, false>(a, g, seg, kept, stream);
  else if (seg.n > 1)
    by_states<T, false, true>(a, g, seg, kept, stream);
  else
    by_states<T, false, false>(a, g, seg, kept, stream);
  const int64_t all = a.batch * a.T * a.G * a.N;
  shared_sums_kernel<T><<<unsigned((all + 255) / 256), 256, 0, stream>>>(
      a, kept.shared, static_cast<T*>(g.dB), static_cast<T*>(g.dC));
  weight_sums_kernel<<<unsigned(((a.N + 2) * a.channels + 31) / 32), 256, 0, stream>>>(
      a, kept.weights, int64_t(seg.n) * a.batch, g.dA, g.dD, g.ddt_bias);
}

}  // namespace
}  // namespace selective

size_t selective_bwd_workspace_bytes(const SelectiveScan& a) {
  return selective::lay_out(a, selective::segments_of(a), nullptr, nullptr);
}

hipError_t launch_selective_bwd(const SelectiveScan& a, const SelectiveGrads& g, void* workspace,
                                hipStream_t stream) {
  using namespace selective;
  const Segments seg = segments_of(a);
  Kept kept;
  lay_out(a, seg, static_cast<char*>(workspace), &kept);
  if (a.is_bf16)
    dispatch<__hip_bfloat16>(a, g, seg, kept, stream);
  else
    dispatch<float>(a, g, seg, kept, stream);
  return hipGetLastError();
}

}  // namespace mlstm
