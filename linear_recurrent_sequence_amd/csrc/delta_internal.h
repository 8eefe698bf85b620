// Workspace and launches shared by the chunked forward and backward of the
// gated delta rule.
#pragma once

#include "delta_common.h"

namespace mlstm {
namespace delta {

// The 32-column blocks of dk that the kernels are built for (even: two waves
// share them).
inline int key_blocks(int64_t dk) {
  const int n = int((dk + 31) / 32);
  for (int ks : {2, 4, 6, 8, 12, 16})
    if (n <= ks) return ks;
  return 0;
}

constexpr int64_t kCUs = 256;

// A sequence cut into n segments of `chunks` chunks (the last one shorter).
struct Segments {
  int n, chunks;
  float* maps;   // [H][n - 1][dv + dk][dk]: the memory after each (see forward_chain)
  float* start;  // [H][dv][dk]: the memory before the first

  __host__ __device__ int n_of(bool map) const { return map ? n - 1 : n; }
  __device__ float* after(int64_t head, int segment, int dk, int dv) const {
    return maps + ((head * (n - 1) + segment) * (dv + dk)) * int64_t(dk);
  }
  __device__ const float* before(int64_t head, int segment, int dk, int dv) const {
    return after(head, segment - 1, dk, dv);
  }
};

// How many segments.  The chains of a sequence's chunks run one workgroup to a
// CU, so where heads times value columns leave CUs idle, a longer sequence is cut
// and each segment's effect on a memory taken first: (dv + dk) / dv times the
// work, but segments side by side.  In units of a chunk's time (5.9 us at dk =
// 256), from the rounds of workgroups that each pass takes, 0.8 for a chunk of the
// map pass, three for joining a segment at dk = 256 and four for the launches; taken
// if a fifth is won.  Whole calls in one piece and cut, bf16: 8 heads of 256 x 16384
// 1392 and 560 us (chunk terms 84; in eight segments 244 for the map pass, 41 to join,
// 188 for the forward), 8 of 128 x 8192 504 and 167, 2 x 4 of 384 x 8192 886 and 615,
// 4 of 64 x 1024 68 and 48; float32, 4 of 128 x 8192 705 and 167.  The charges are
// above what that first call shows (0.65 for a chunk of the map pass, 1.2 for a
// join), so some long sequences of few wide heads stay in one piece that might gain
// by a cut: 4 heads of 512 x 8192, 1042 us, and of 384 x 4096, 443.
inline Segments segments_of(const DeltaShape& s) {
  const int64_t chunks = (s.T + kC - 1) / kC, H = s.B * s.NH;
  auto rounds = [&](int64_t wgs) { return (wgs + kCUs - 1) / kCUs; };
  const int64_t per_head = (s.dv + 63) / 64, mapped = (s.dv + s.dk + 63) / 64;
  Segments best = {1, int(chunks), nullptr, nullptr};
  double least = 0.8 * double(chunks * rounds(H * per_head));
  for (int64_t n = 2; n <= 16 && n * 4 <= chunks; ++n) {
    const int64_t len = (chunks + n - 1) / n;
    if ((chunks + len - 1) / len != n) continue;  // as few segments of that length do
    const double join = 3.0 * double(s.dk) * double(s.dk) / 65536.0;
    const double t = double(len) * (0.8 * double(rounds(H * mapped * (n - 1))) +
                                    double(rounds(H * per_head * n))) +
                     double(n) * join + 4.0;
    if (t < least) {
      least = t;
      best = {int(n), int(len), nullptr, nullptr};
    }
  }
  return best;
}

// Whether the backward's two chains, the memory once more and its gradient, run
// in one launch (delta_pairs_kernel then forms what needs both): where that
// saves a tenth of the rounds of workgroups: up to 128 of them, and some numbers
// above.  The whole backward pass, one after the other and side by side: 4 x 4
// heads of 384 x 2048 (96 workgroups) in bf16 1051 and 821 us, 12 x 4 of 384 x
// 1024 (288) 1314 and 1209, 2 x 16 of 128 x 2048 (64) in float32 802 and 605.
// With as many rounds either way bf16's run one after the other, where the second
// has the sums with X and Y at hand (8 x 4 of 384 x 2048 1528 us, 1575 side by side,
// 1596 with the sums left to the pairs; in float32 the second chain always leaves
// them, as LDS has no room for X and Y: 8 x 16 of 128 x 1024 879 and 873).
inline bool side_by_side(const DeltaShape& s) {
  const int64_t wgs = s.B * s.NH * ((s.dv + 63) / 64);
  const int64_t apart = 2 * ((wgs + kCUs - 1) / kCUs), together = (2 * wgs + kCUs - 1) / kCUs;
  return 10 * (apart - together) >= apart;
}

struct Layout {
  Work ws;
  Saved sv;
  Segments seg;
  int ks;
  bool apart;  // the backward's gradient of the memory takes no X (see back_chain)
  size_t bytes;
};

// The workspace's parts from `base` (256-byte aligned) on; NULL gives the size.
inline Layout layout(const DeltaShape& s, bool backward, void* base) {
  Layout l = {};
  l.ks = key_blocks(s.dk);
  const size_t chunks = size_t((s.T + kC - 1) / kC), H = size_t(s.B * s.NH) * chunks,
               HK = size_t(s.B * s.NHK) * chunks;
  const size_t npl = s.is_bf16 ? 1 : 3;
  const size_t rows = size_t(l.ks) * 32 * kC * sizeof(__bf16), square = kSquare * sizeof(__bf16);
  auto take = [&](size_t n) {
    char* p = base ? static_cast<char*>(base) + l.bytes : nullptr;
    l.bytes += (n + 255) & ~size_t(255);
    return p;
  };
  auto planes = [&](size_t n) { return reinterpret_cast<__bf16*>(take(n)); };
  l.ws.inv = planes(H * 3 * square);
  l.ws.score = planes(H * 3 * square);
  l.ws.keyT = planes(HK * npl * rows);
  if (npl == 3) {
    l.ws.key = planes(HK * npl * rows);
    l.ws.query = planes(HK * npl * rows);
  }
  if (backward) l.ws.queryT = planes(HK * npl * rows);
  if (backward) {
    l.ws.invT = planes(H * 3 * square);
    l.ws.scoreT = planes(H * 3 * square);
  }
  l.ws.decay = reinterpret_cast<float*>(take(H * 3 * kC * sizeof(float)));
  l.seg = segments_of(s);
  if (!backward && l.seg.n > 1) {
    const size_t heads = size_t(s.B * s.NH), dk = size_t(s.dk), dv = size_t(s.dv);
    l.seg.maps = reinterpret_cast<float*>(
        take(heads * size_t(l.seg.n - 1) * (dv + dk) * dk * sizeof(float)));
    l.seg.start = reinterpret_cast<float*>(take(heads * dv * dk * sizeof(float)));
  }
  if (backward) {
    auto floats = [&](size_t n) { return reinterpret_cast<float*>(take(n * sizeof(float))); };
    const size_t state = size_t(s.dk * s.dv), rows = size_t(s.B * s.T);
    l.sv.S = floats(H * state);
    l.sv.Z = floats(H * state);
    l.sv.X = floats(rows * size_t(s.NH * s.dv));
    l.sv.Y = floats(rows * size_t(s.NH * s.dv));
    if (s.is_bf16) l.sv.dR = floats(rows * size_t(s.NH * s.dv));
    l.apart = side_by_side(s) || !s.is_bf16;
    if (l.apart) l.sv.KZ = floats(rows * size_t(s.NH * s.dv));
    l.sv.part = floats(H * size_t(s.dv / 16) * 3 * kC);
    l.sv.pairs = planes(H * 9 * square);
    l.sv.gates = floats(H * 2 * kC);
    l.sv.inner = floats(H * size_t((s.dk + 127) / 128));
  }
  return l;
}

// What a chain kernel takes.
template <typename T>
struct Chain {
  const T *q, *k, *v, *dh;
  Work ws;
  Saved sv;
  int64_t T_len, H;
  int chunks, NH, NHK, dk, dv, tiles, per_head;
  float scale;
};
template <typename T>
Chain<T> chain(const DeltaShape& s, const Layout& l, const void* q, const void* k, const void* v,
               const void* dh) {
  const int tiles = int(s.dv / 16);
  return {static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v),
          static_cast<const T*>(dh), l.ws, l.sv, s.T, s.B * s.NH, int((s.T + kC - 1) / kC),
          int(s.NH), int(s.NHK), int(s.dk), int(s.dv), tiles, (tiles + 3) / 4,
          1.0f / sqrtf(float(s.dk))};
}

// ks: the 32-column blocks that the kernels are built for, >= ceil(dk / 32)
hipError_t launch_prep(const DeltaShape& s, const void* q, const void* k, const float* beta,
                       const float* fgate, const Work& ws, int ks, bool backward,
                       hipStream_t stream);

}  // namespace delta
}  // namespace mlstm
