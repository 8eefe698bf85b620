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

struct Layout {
  Work ws;
  Saved sv;
  int ks;
  size_t bytes;
};

// The workspace's parts from `base` (256-byte aligned) on; NULL gives the size.
inline Layout layout(const DeltaShape& s, bool backward, void* base) {
  Layout l = {};
  l.ks = key_blocks(s.dk);
  const size_t chunks = size_t((s.T + kC - 1) / kC), H = size_t(s.B * s.NH) * chunks,
               HK = size_t(s.B * s.NHK) * chunks;
  const size_t npl = s.is_bf16 ? 1 : 3, npp = s.is_bf16 && !backward ? 2 : 3;
  const size_t rows = size_t(l.ks) * 32 * kC * sizeof(__bf16), square = kSquare * sizeof(__bf16);
  auto take = [&](size_t n) {
    char* p = base ? static_cast<char*>(base) + l.bytes : nullptr;
    l.bytes += (n + 255) & ~size_t(255);
    return p;
  };
  auto planes = [&](size_t n) { return reinterpret_cast<__bf16*>(take(n)); };
  l.ws.inv = planes(H * 3 * square);
  l.ws.score = planes(H * npp * square);
  l.ws.keyT = planes(HK * npl * rows);
  if (npl == 3) {
    l.ws.key = planes(HK * npl * rows);
    l.ws.query = planes(HK * npl * rows);
  }
  if (backward) l.ws.queryT = planes(HK * npl * rows);
  if (backward) {
    l.ws.invT = planes(H * 3 * square);
    l.ws.scoreT = planes(H * npp * square);
  }
  l.ws.decay = reinterpret_cast<float*>(take(H * 3 * kC * sizeof(float)));
  if (backward) {
    auto floats = [&](size_t n) { return reinterpret_cast<float*>(take(n * sizeof(float))); };
    const size_t state = size_t(s.dk * s.dv), rows = size_t(s.B * s.T);
    l.sv.S = floats(H * state);
    l.sv.Z = floats(H * state);
    l.sv.X = floats(rows * size_t(s.NH * s.dv));
    if (s.is_bf16) l.sv.dR = floats(rows * size_t(s.NH * s.dv));
    l.sv.part = floats(H * size_t(s.dv / 16) * 3 * kC);
    const size_t npd = s.is_bf16 ? 2 : 3;
    l.sv.pairs = planes(H * 3 * npd * square);
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

// the memory once more for the backward (Saved::S, X and the first of part)
hipError_t launch_again(const DeltaShape& s, const Layout& l, const void* q, const void* k,
                        const void* v, const void* dh, const float* C_in, hipStream_t stream);

// ks: the 32-column blocks that the kernels are built for, >= ceil(dk / 32)
hipError_t launch_prep(const DeltaShape& s, const void* q, const void* k, const float* beta,
                       const float* fgate, const Work& ws, int ks, bool backward,
                       hipStream_t stream);

}  // namespace delta
}  // namespace mlstm
