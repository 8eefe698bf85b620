// Gated feed-forward: h = act(x Wg^T) * (x Wu^T), rows of x.
//
// Forward: both products share the tiles of x, and a wave holds g and u of the
// same outputs, so the activation and the product are formed in its registers and
// h is all that is written.  Backward, with g and u formed again the same way:
//
//   dg = dh u act'(g),  du = dh act(g)             (G = [dg | du], M x 2F)
//   dx = G [Wg ; Wu],   [dWg ; dWu] = G^T x
//
// All products run on one kind of tile (product_tiles.h), whose operands are rows
// of the summed index: the weights, x and G are transposed into the workspace for
// the last two.  For bf16, G is rounded to bf16 as the operand of those products
// (2^-9 of each term, as much as the rounding of the results); everything before
// is float32.
#include "gated_ffn.h"

#include "product_tiles.h"
#include "row_vec.h"

namespace mlstm {
namespace ffn {
namespace {

using product::f32x4;
using product::Operand;

using Large = product::Shape<256, 256, 2, 4>;
using Medium = product::Shape<128, 256, 2, 4>;
using Small = product::Shape<128, 128, 2, 2>;

constexpr int kPlanes = 3, kTerms = 6;  // of float32

struct Act {
  float value, slope;
};
__device__ inline Act activation(float g, bool gelu) {
  if (gelu) {  // g Phi(g); the slope is Phi(g) + g phi(g)
    const float phi = 0.3989422804014327f * rowvec::exp2_fast(-0.5f * rowvec::kLog2e * g * g);
    const float cdf = 0.5f * erfcf(-0.7071067811865476f * g);
    return {g * cdf, __builtin_fmaf(g, phi, cdf)};
  }
  const float s = rowvec::sigmoid(g);
  return {g * s, rowvec::silu_slope(g, s)};
}

struct Sizes {
  int64_t M, D, F;
  int terms;
  bool gelu;
};

// h, or with GRAD G = [dg | du], in tiles of rows and of F
template <typename T, typename S, bool GRAD>
__global__ __launch_bounds__(S::kThreads) void gate_up_kernel(Operand wg, Operand wu, Operand x,
                                                              Sizes n, const T* dh, T* out) {
  __shared__ __align__(1024) char lds[S::kLds];
  constexpr int kF = S::kBP / 2, kStores = (GRAD ? S::kP : S::kP / 2) * S::kQ;
  const unsigned np = unsigned((n.F + kF - 1) / kF), nq = unsigned((n.M + S::kBQ - 1) / S::kBQ);
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  product::tiles<S, true, kStores>(
      wg, wu, x, n.D, n.terms, np, nq, 1, 1, lds,
      [&](unsigned ip, unsigned iq, unsigned, const f32x4(&acc)[S::kP][S::kQ]) {
        const int64_t f0 = int64_t(ip) * kF + wave / S::kWQ * (kF / S::kWP) + lane / 16 * 4,
                      q0 = int64_t(iq) * S::kBQ;
        const int m0 = wave % S::kWQ * (S::kBQ / S::kWQ) + lane % 16;
        const product::Rows<T> rows(out, q0, n.M, GRAD ? 2 * n.F : n.F);
#pragma unroll
        for (int j = 0; j < S::kQ; ++j)
#pragma unroll
          for (int i = 0; i < S::kP / 2; ++i) {
            const int64_t f = f0 + i * 16, m = q0 + m0 + j * 16;
            const f32x4 g = acc[i][j], u = acc[i + S::kP / 2][j];
            f32x4 a, b;
            if constexpr (GRAD) {
              float d[4] = {};
              if (m < n.M && f < n.F) rowvec::load(dh + m * n.F + f, d);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const Act act = activation(g[e], n.gelu);
                a[e] = d[e] * u[e] * act.slope;
                b[e] = d[e] * act.value;
              }
              rows.put(m0 + j * 16, f, n.F, a);
              rows.put(m0 + j * 16, n.F + f, 2 * n.F, b);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) a[e] = activation(g[e], n.gelu).value * u[e];
              rows.put(m0 + j * 16, f, n.F, a);
            }
          }
      });
}

// out[q][p], with two groups of q the second one in out2; with splits, each one's
// share in rows of its own, all groups of q behind one another
template <typename T, typename S>
__global__ __launch_bounds__(S::kThreads) void product_kernel(Operand left, Operand right,
                                                              int64_t k, int terms, int groups,
                                                              int splits, T* out, T* out2) {
  __shared__ __align__(1024) char lds[S::kLds];
  const unsigned np = unsigned((left.rows + S::kBP - 1) / S::kBP),
                 of_group = unsigned((right.rows + S::kBQ - 1) / S::kBQ);
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  product::tiles<S, false, S::kP * S::kQ>(
      left, left, right, k, terms, np, of_group * groups, groups, splits, lds,
      [&](unsigned ip, unsigned iq, unsigned split, const f32x4(&acc)[S::kP][S::kQ]) {
        const int64_t p0 = int64_t(ip) * S::kBP + wave / S::kWQ * (S::kBP / S::kWP) + lane / 16 * 4;
        const int q0 = wave % S::kWQ * (S::kBQ / S::kWQ) + lane % 16;
        T* to = iq < of_group ? out : out2;
        if (splits > 1)
          to = out + (int64_t(split) * groups + iq / of_group) * right.rows * left.rows;
        const product::Rows<T> rows(to, int64_t(iq % of_group) * S::kBQ, right.rows, left.rows);
#pragma unroll
        for (int j = 0; j < S::kQ; ++j)
#pragma unroll
          for (int i = 0; i < S::kP; ++i)
            rows.put(q0 + j * 16, p0 + i * 16, left.rows, acc[i][j]);
      });
}

// out, out2 = sums of `splits` shares, in order; n values to each (a multiple of 4)
template <typename T>
__global__ __launch_bounds__(256) void join_kernel(const float* shares, int64_t n, int groups,
                                                   int splits, T* out, T* out2) {
  const int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (i >= n * groups) return;
  float s[4] = {};
  for (int k = 0; k < splits; ++k) {
    float x[4];
    rowvec::load(shares + k * n * groups + i, x);
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] += x[e];
  }
  rowvec::store(i < n ? out + i : out2 + (i - n), s);
}

// ---- few rows

// h for up to 16 MT rows: bound by the weights' bytes, which a wave reads straight
// into the registers of its products.  A workgroup has 16 columns of h; its eight
// waves have a share of D each, and their sums are joined through LDS in order.
constexpr int kFewRows = 64, kFewWaves = 8;

template <typename T>
struct FewProduct;
// 32 columns of D: lane l has row l % 16 and 8 columns from 8 (l / 16) on
template <>
struct FewProduct<__hip_bfloat16> {
  static constexpr int kStep = 32, kLane = 8;
  typedef __bf16 Piece __attribute__((ext_vector_type(8)));
  __device__ static f32x4 add(Piece a, Piece b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
// 16 columns, 4 to a lane, on the float32 instruction, of which each takes one
template <>
struct FewProduct<float> {
  static constexpr int kStep = 16, kLane = 4;
  typedef f32x4 Piece;
  __device__ static f32x4 add(Piece a, Piece b, f32x4 c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
  }
};

template <typename T, int MT>
__global__ __launch_bounds__(64 * kFewWaves) void few_rows_kernel(const T* wg, const T* wu,
                                                                  const T* x, Sizes n, T* h) {
  using P = FewProduct<T>;
  using Piece = typename P::Piece;
  __shared__ f32x4 sums[kFewWaves][2 * MT][64];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t f0 = int64_t(blockIdx.x) * 16, f = f0 + lane % 16;
  const int64_t row = (f < n.F ? f : n.F - 1) * n.D;
  const int64_t steps = (n.D + P::kStep - 1) / P::kStep,
                share = (steps + kFewWaves - 1) / kFewWaves;
  const int64_t from = wave * share, to = from + share < steps ? from + share : steps;
  f32x4 g[MT], u[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) g[m] = u[m] = f32x4{};
  constexpr int kAhead = MT <= 2 ? 4 : 2;  // steps whose loads are in flight together
  for (int64_t s = from; s < to; s += kAhead) {
    Piece a[kAhead], b[kAhead], v[kAhead][MT];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t k = (s + i) * P::kStep + lane / 16 * P::kLane;
      const bool on = s + i < to && k < n.D;  // D is a multiple of a lane's columns
      const int64_t at = on ? k : 0;
      a[i] = *reinterpret_cast<const Piece*>(wg + row + at);
      b[i] = *reinterpret_cast<const Piece*>(wu + row + at);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int64_t r = m * 16 + lane % 16;
        const Piece p = *reinterpret_cast<const Piece*>(x + (r < n.M ? r : 0) * n.D + at);
        v[i][m] = on && r < n.M ? p : Piece{};
      }
      if (!on) a[i] = b[i] = Piece{};
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        g[m] = P::add(a[i], v[i][m], g[m]);
        u[m] = P::add(b[i], v[i][m], u[m]);
      }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) sums[wave][2 * m][lane] = g[m], sums[wave][2 * m + 1][lane] = u[m];
  __syncthreads();
  if (wave >= MT) return;
  f32x4 a = {}, b = {};
#pragma unroll
  for (int w = 0; w < kFewWaves; ++w) {
    a += sums[w][2 * wave][lane];
    b += sums[w][2 * wave + 1][lane];
  }
  // lane l: columns 4 (l / 16) .. of row l % 16
  const int64_t r = wave * 16 + lane % 16, c = f0 + lane / 16 * 4;
  if (r >= n.M || c >= n.F) return;
  float o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = activation(a[e], n.gelu).value * b[e];
  rowvec::store(h + r * n.F + c, o);
}

template <typename T>
hipError_t few_rows(const GatedFfn& a, void* h, hipStream_t stream) {
  const T *wg = static_cast<const T*>(a.w_gate), *wu = static_cast<const T*>(a.w_up),
          *x = static_cast<const T*>(a.x);
  const Sizes n = {a.M, a.D, a.F, 1, a.gelu};
  const unsigned wgs = unsigned((a.F + 15) / 16);
  T* out = static_cast<T*>(h);
  if (a.M <= 16)
    few_rows_kernel<T, 1><<<wgs, 64 * kFewWaves, 0, stream>>>(wg, wu, x, n, out);
  else if (a.M <= 32)
    few_rows_kernel<T, 2><<<wgs, 64 * kFewWaves, 0, stream>>>(wg, wu, x, n, out);
  else
    few_rows_kernel<T, 4><<<wgs, 64 * kFewWaves, 0, stream>>>(wg, wu, x, n, out);
  return hipGetLastError();
}

// ---- operands: planes of float32, and transposes

// three bf16 planes of x
__device__ inline void planes_of(float x, uint16_t (&p)[kPlanes]) {
#pragma unroll
  for (int i = 0; i < kPlanes; ++i) {
    p[i] = uint16_t(rowvec::to_bf16(x, 0.0f));
    x -= __uint_as_float(unsigned(p[i]) << 16);
  }
}

// planes of n values (a multiple of 4)
__global__ __launch_bounds__(256) void split_kernel(const float* x, int64_t n, uint16_t* out,
                                                    int64_t plane) {
  const int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  const float4 f = *reinterpret_cast<const float4*>(x + i);
  const float v[4] = {f.x, f.y, f.z, f.w};
  uint16_t p[4][kPlanes];
#pragma unroll
  for (int e = 0; e < 4; ++e) planes_of(v[e], p[e]);
#pragma unroll
  for (int k = 0; k < kPlanes; ++k)
    *reinterpret_cast<ushort4*>(out + k * plane + i) =
        make_ushort4(p[0][k], p[1][k], p[2][k], p[3][k]);
}

// out[c][r] = in[r][c] with rows of `width` outputs, `pitch` apart, zeros for r from
// `rows` on; in 64 x 64 tiles through LDS.  float32 becomes planes.
template <typename T>
__global__ __launch_bounds__(256) void transpose_kernel(const T* in, int64_t rows, int64_t cols,
                                                        uint16_t* out, int64_t width,
                                                        int64_t pitch, int64_t plane) {
  constexpr int N = sizeof(T) == 4 ? kPlanes : 1;
  __shared__ uint16_t tile[N][64][66];
  const int64_t tiles = (cols + 63) / 64;
  const int64_t c0 = blockIdx.x % tiles * 64, r0 = blockIdx.x / tiles * 64;
  for (int i = threadIdx.x; i < 64 * 16; i += 256) {
    const int r = i / 16, c = i % 16 * 4;
    float v[4] = {};
    if (r0 + r < rows && c0 + c < cols) rowvec::load(in + (r0 + r) * cols + c0 + c, v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (N == 1) {
        tile[0][c + e][r] = uint16_t(__float_as_uint(v[e]) >> 16);
      } else {
        uint16_t p[kPlanes];
        planes_of(v[e], p);
#pragma unroll
        for (int k = 0; k < N; ++k) tile[k][c + e][r] = p[k];
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * 16; i += 256) {
    const int c = i / 16, r = i % 16 * 4;
    if (c0 + c < cols && r0 + r < width)
#pragma unroll
      for (int k = 0; k < N; ++k)
        *reinterpret_cast<ushort4*>(out + k * plane + (c0 + c) * pitch + r0 + r) = make_ushort4(
            tile[k][c][r], tile[k][c][r + 1], tile[k][c][r + 2], tile[k][c][r + 3]);
  }
}

// ---- launches

size_t pad256(size_t n) { return (n + 255) & ~size_t(255); }

// a workspace taken in order; with a null base, its size
struct Arena {
  char* base;
  size_t at = 0;
  template <typename T>
  T* take(int64_t n) {
    T* p = reinterpret_cast<T*>(base + at);
    at += pad256(size_t(n) * sizeof(T));
    return p;
  }
};

template <typename T>
constexpr int kCopies = sizeof(T) == 4 ? kPlanes : 1;
template <typename T>
constexpr int kTermsOf = sizeof(T) == 4 ? kTerms : 1;

// an operand of the products: a bf16 matrix as it is, the planes of a float32 one
template <typename T>
Operand as_rows(const void* p, int64_t rows, int64_t k, Arena& ws, hipStream_t stream, bool run) {
  if constexpr (sizeof(T) == 2) {
    return {static_cast<const uint16_t*>(p), rows, 0, 0};
  } else {
    uint16_t* out = ws.take<uint16_t>(kPlanes * rows * k);
    if (run)
      split_kernel<<<unsigned((rows * k + 1023) / 1024), 256, 0, stream>>>(
          static_cast<const float*>(p), rows * k, out, rows * k);
    return {out, rows, rows * k, 0};
  }
}

// a matrix [rows][cols] as `cols` rows of `width` (rows, rounded up to 8)
template <typename T>
void transposed(const void* p, int64_t rows, int64_t cols, uint16_t* out, int64_t width,
                int64_t pitch, int64_t plane, hipStream_t stream) {
  const int64_t n = ((cols + 63) / 64) * ((width + 63) / 64);
  transpose_kernel<T><<<unsigned(n), 256, 0, stream>>>(static_cast<const T*>(p), rows, cols, out,
                                                       width, pitch, plane);
}

constexpr int64_t kCUs = 256;

template <typename S>
int64_t tiles_of(int64_t p, int64_t q) {
  return ((p + S::kBP - 1) / S::kBP) * ((q + S::kBQ - 1) / S::kBQ);
}
// Workgroups that a CU holds at a time
template <typename S>
constexpr int kPerCu = S::kLds <= 64 * 1024 ? 2 : 1;

// f(shape) with the tile of the least time for p x q outputs (in each of `groups`):
// the rounds of tiles that a CU takes, at what each takes.
template <typename F>
hipError_t with_shape(int64_t p, int64_t q, int64_t groups, F&& f) {
  auto rounds = [&](int64_t tiles, int64_t at_once) {
    return double((tiles * groups + kCUs * at_once - 1) / (kCUs * at_once));
  };
  const double large = rounds(tiles_of<Large>(p, q), 1),
               medium = 0.6 * rounds(tiles_of<Medium>(p, q), 1);
  const int64_t n = tiles_of<Small>(p, q) * groups;
  const double small = n <= kCUs ? 0.4 : 0.65 * rounds(tiles_of<Small>(p, q), 2);
  if (small < large && small < medium) return f(Small{});
  if (medium < large) return f(Medium{});
  return f(Large{});
}

template <typename T, bool GRAD>
hipError_t gate_up(const Operand& wg, const Operand& wu, const Operand& x, const Sizes& n,
                   const void* dh, void* out, hipStream_t stream) {
  return with_shape(2 * n.F, n.M, 1, [&](auto shape) {
    using S = decltype(shape);
    const int64_t tiles = tiles_of<S>(2 * n.F, n.M), most = kCUs * kPerCu<S>;
    gate_up_kernel<T, S, GRAD><<<unsigned(tiles < most ? tiles : most), S::kThreads, 0, stream>>>(
        wg, wu, x, n, static_cast<const T*>(dh), static_cast<T*>(out));
    return hipGetLastError();
  });
}

// How often a product's summed index is split, so that tiles that leave CUs idle are
// taken by several: each share at least eight pieces long.
template <typename T>
int splits_of(int64_t p, int64_t q, int64_t k, int groups) {
  const int64_t tiles = tiles_of<Small>(p, q) * groups,
                pieces = (k + product::kStep - 1) / product::kStep * kTermsOf<T>;
  int64_t n = kCUs / tiles;
  if (n > pieces / 8) n = pieces / 8;
  if (n < 2) return 1;
  const int64_t share = (pieces + n - 1) / n;
  return int((pieces + share - 1) / share);  // every share has a piece
}

template <typename T>
hipError_t multiply(const Operand& l, const Operand& r, int64_t k, int groups, void* out,
                    void* out2, Arena& ws, hipStream_t stream, bool run) {
  const int splits = splits_of<T>(l.rows, r.rows, k, groups);
  if (splits > 1) {
    const int64_t n = l.rows * r.rows;
    float* shares = ws.take<float>(splits * groups * n);
    if (!run) return hipSuccess;
    product_kernel<float, Small><<<unsigned(tiles_of<Small>(l.rows, r.rows) * groups * splits),
                                   Small::kThreads, 0, stream>>>(l, r, k, kTermsOf<T>, groups,
                                                                 splits, shares, shares);
    join_kernel<T><<<unsigned((n * groups + 1023) / 1024), 256, 0, stream>>>(
        shares, n, groups, splits, static_cast<T*>(out), static_cast<T*>(out2));
    return hipGetLastError();
  }
  if (!run) return hipSuccess;
  return with_shape(l.rows, r.rows, groups, [&](auto shape) {
    using S = decltype(shape);
    const int64_t tiles = tiles_of<S>(l.rows, r.rows) * groups, most = kCUs * kPerCu<S>;
    product_kernel<T, S><<<unsigned(tiles < most ? tiles : most), S::kThreads, 0, stream>>>(
        l, r, k, kTermsOf<T>, groups, 1, static_cast<T*>(out), static_cast<T*>(out2));
    return hipGetLastError();
  });
}

// `run` false: only the workspace's size
template <typename T>
hipError_t forward(const GatedFfn& a, void* h, Arena& ws, hipStream_t stream, bool run) {
  if (a.M <= kFewRows) return run ? few_rows<T>(a, h, stream) : hipSuccess;
  const Operand wg = as_rows<T>(a.w_gate, a.F, a.D, ws, stream, run),
                wu = as_rows<T>(a.w_up, a.F, a.D, ws, stream, run),
                x = as_rows<T>(a.x, a.M, a.D, ws, stream, run);
  if (!run) return hipSuccess;
  return gate_up<T, false>(wg, wu, x, {a.M, a.D, a.F, kTermsOf<T>, a.gelu}, nullptr, h, stream);
}

template <typename T>
hipError_t backward(const GatedFfn& a, const GatedFfnGrads& g, Arena& ws, hipStream_t stream,
                    bool run) {
  const int64_t M = a.M, D = a.D, F = a.F, pitch = (M + 7) / 8 * 8;
  const Operand wg = as_rows<T>(a.w_gate, F, D, ws, stream, run),
                wu = as_rows<T>(a.w_up, F, D, ws, stream, run),
                x = as_rows<T>(a.x, M, D, ws, stream, run);
  T* G = ws.take<T>(M * 2 * F);
  const int64_t wt_plane = D * 2 * F, xt_plane = D * pitch, gt_plane = 2 * F * pitch;
  uint16_t* wt = ws.take<uint16_t>(kCopies<T> * wt_plane);  // [D][Wg^T | Wu^T]
  uint16_t* xt = ws.take<uint16_t>(kCopies<T> * xt_plane);  // [D][M]
  uint16_t* gt = ws.take<uint16_t>(kCopies<T> * gt_plane);  // [2F][M]
  if (run) {
    const hipError_t e =
        gate_up<T, true>(wg, wu, x, {M, D, F, kTermsOf<T>, a.gelu}, g.dh, G, stream);
    if (e != hipSuccess) return e;
  }
  const Operand G_rows = as_rows<T>(G, M, 2 * F, ws, stream, run);
  if (run) {  // the two halves of wt, each [D] rows of 2 F
    transposed<T>(a.w_gate, F, D, wt, F, 2 * F, wt_plane, stream);
    transposed<T>(a.w_up, F, D, wt + F, F, 2 * F, wt_plane, stream);
    transposed<T>(a.x, M, D, xt, pitch, pitch, xt_plane, stream);
    transposed<T>(G, M, 2 * F, gt, pitch, pitch, gt_plane, stream);
  }
  const hipError_t e =
      multiply<T>({wt, D, wt_plane, 0}, G_rows, 2 * F, 1, g.dx, nullptr, ws, stream, run);
  if (e != hipSuccess) return e;
  return multiply<T>({xt, D, xt_plane, 0}, {gt, F, gt_plane, F * pitch}, pitch, 2, g.dw_gate,
                     g.dw_up, ws, stream, run);
}

}  // namespace
}  // namespace ffn

size_t gated_ffn_fwd_workspace_bytes(const GatedFfn& a) {
  ffn::Arena ws{nullptr};
  if (a.is_bf16)
    (void)ffn::forward<__hip_bfloat16>(a, nullptr, ws, nullptr, false);
  else
    (void)ffn::forward<float>(a, nullptr, ws, nullptr, false);
  return ws.at;
}

hipError_t launch_gated_ffn_fwd(const GatedFfn& a, void* h, void* workspace, hipStream_t stream) {
  ffn::Arena ws{static_cast<char*>(workspace)};
  return a.is_bf16 ? ffn::forward<__hip_bfloat16>(a, h, ws, stream, true)
                   : ffn::forward<float>(a, h, ws, stream, true);
}

size_t gated_ffn_bwd_workspace_bytes(const GatedFfn& a) {
  ffn::Arena ws{nullptr};
  if (a.is_bf16)
    (void)ffn::backward<__hip_bfloat16>(a, {}, ws, nullptr, false);
  else
    (void)ffn::backward<float>(a, {}, ws, nullptr, false);
  return ws.at;
}

hipError_t launch_gated_ffn_bwd(const GatedFfn& a, const GatedFfnGrads& g, void* workspace,
                                hipStream_t stream) {
  ffn::Arena ws{static_cast<char*>(workspace)};
  return a.is_bf16 ? ffn::backward<__hip_bfloat16>(a, g, ws, stream, true)
                   : ffn::backward<float>(a, g, ws, stream, true);
}

}  // namespace mlstm
