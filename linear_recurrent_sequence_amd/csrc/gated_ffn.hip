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
// the last two.  For bf16, G has two bf16 planes, 16 bits, as the operand of those
// products: up to 2^-17 of each term, little beside the rounding of the results, which are
// then the float32 gradients rounded once.  (One plane takes half the time of two, but its
// errors of up to 2^-8 of each term do not average out in a sum of terms of either sign,
// however long it is: the results would be off by as much again as by their own rounding.)
// Everything before is float32.
//
// Measured: 16384 rows of 1536 to 4096 forward 330 us (in a settled trace;
// product_tiles.h has what bounds it); 8192 rows of 2048 to 5504 forward 319, backward
// 466 for G, 550 for dx and 607 for the weights' gradients, 177 for turned operands and
// 10 for joined shares (with one plane of G 365, 287, 309, 95 and 11).  8 rows of 1536 to 4096 7.8 us (25 MB, 5.1 at a copy's rate), 17 as
// tiles.  float32, 999 rows of 392 to 1048, training: 145 us, 350 before split tiles,
// operands made in one launch and three pieces ahead (158 with two).
#include "gated_ffn.h"

#include "mlstm_internal.h"
#include "product_tiles.h"
#include "row_vec.h"

namespace mlstm {
namespace ffn {
namespace {

using product::f32x4;
using product::Operand;
using product::Plan;

using Large = product::Shape<256, 256, 2, 4, 2>;
using Medium = product::Shape<128, 256, 2, 4, 3>;
using Small = product::Shape<128, 128, 2, 2, 2>;

constexpr int kPlanes = 3, kTerms = 6;  // of float32
constexpr int kGradPlanes = 2;          // of G, behind bf16 gradients

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

// Four outputs from g and u: h (a), or with GRAD dg and du, from dh
struct Pair {
  f32x4 a, b;
};
template <bool GRAD>
__device__ inline Pair gate_up_of(f32x4 g, f32x4 u, const float (&d)[4], bool gelu) {
  Pair o;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const Act act = activation(g[e], gelu);
    if constexpr (GRAD) {
      o.a[e] = d[e] * u[e] * act.slope;
      o.b[e] = d[e] * act.value;
    } else {
      o.a[e] = act.value * u[e];
    }
  }
  return o;
}

// h, or with GRAD G = [dg | du] (for bf16 its two planes, one behind the other), in tiles
// of rows and of F
template <typename T, typename S, bool GRAD>
__global__ __launch_bounds__(S::kThreads) void gate_up_kernel(Operand wg, Operand wu, Operand x,
                                                              Sizes n, Plan plan, const T* dh,
                                                              T* out, float* shares) {
  __shared__ __align__(1024) char lds[S::kLds];
  constexpr bool kTwoPlanes = GRAD && sizeof(T) == 2;
  // two planes are twice as many stores, but a share of a tile has no more than these
  constexpr int kF = S::kBP / 2, kStores = (GRAD ? S::kP : S::kP / 2) * S::kQ;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  product::tiles<S, true, kStores>(
      wg, wu, x, n.D, n.terms, plan, lds,
      [&](unsigned ip, unsigned iq, const product::Item& item,
          const f32x4(&acc)[S::kP][S::kQ]) {
        if (item.split >= 0)
          return product::put_share<S>(
              product::Rows<float>(product::share_at<S>(plan, shares, item), 0, S::kBQ, S::kBP),
              acc);
        const int f0 = int(ip) * kF + wave / S::kWQ * (kF / S::kWP) + lane / 16 * 4,
                  q0 = int(iq) * S::kBQ, F = int(n.F), M = int(n.M);
        const int m0 = wave % S::kWQ * (S::kBQ / S::kWQ) + lane % 16;
        const product::Rows<T> rows(out, q0, M, GRAD ? 2 * F : F),
            low_rows(out + (kTwoPlanes ? n.M * 2 * n.F : 0), q0, M, GRAD ? 2 * F : F);
        auto put = [&](int i, int c, int columns, f32x4 v) {
          if constexpr (kTwoPlanes) {
            const product::TwoPlanes p(v);
            rows.put(i, c, columns, p.high);
            low_rows.put(i, c, columns, p.low);
          } else {
            rows.put(i, c, columns, v);
          }
        };
        // dh of kAhead blocks of rows at a time, ahead of their stores
        constexpr int kAhead = GRAD && sizeof(T) == 2 ? S::kQ : 1;
#pragma unroll
        for (int j0 = 0; j0 < S::kQ; j0 += kAhead) {
          rowvec::Raw<T, 4> raw[kAhead][S::kP / 2] = {};
          if constexpr (GRAD) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
#pragma unroll
              for (int i = 0; i < S::kP / 2; ++i) {
                const int f = f0 + i * 16, m = q0 + m0 + (j0 + j) * 16;
                if (m < M && f < F)
                  raw[j][i] = rowvec::load_raw<T, 4>(dh + int64_t(m) * F + f);
              }
          }
#pragma unroll
          for (int jj = 0; jj < kAhead; ++jj)
#pragma unroll
            for (int i = 0; i < S::kP / 2; ++i) {
              const int j = j0 + jj, f = f0 + i * 16;
              float d[4];
              rowvec::floats(raw[jj][i], d);
              const Pair o = gate_up_of<GRAD>(acc[i][j], acc[i + S::kP / 2][j], d, n.gelu);
              put(m0 + j * 16, f, F, o.a);
              if constexpr (GRAD) put(m0 + j * 16, f < F ? F + f : 2 * F, 2 * F, o.b);
            }
        }
      });
}

// out[q][p], with two groups of q the second one in out2
template <typename T, typename S>
__global__ __launch_bounds__(S::kThreads) void product_kernel(Operand left, Operand right,
                                                              int64_t k, int terms, Plan plan,
                                                              T* out, T* out2, float* shares) {
  __shared__ __align__(1024) char lds[S::kLds];
  const unsigned of_group = plan.nq / plan.groups;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  product::tiles<S, false, S::kP * S::kQ>(
      left, left, right, k, terms, plan, lds,
      [&](unsigned ip, unsigned iq, const product::Item& item,
          const f32x4(&acc)[S::kP][S::kQ]) {
        if (item.split >= 0)
          return product::put_share<S>(
              product::Rows<float>(product::share_at<S>(plan, shares, item), 0, S::kBQ, S::kBP),
              acc);
        const int p0 = int(ip) * S::kBP + wave / S::kWQ * (S::kBP / S::kWP) + lane / 16 * 4,
                  q0 = wave % S::kWQ * (S::kBQ / S::kWQ) + lane % 16, width = int(left.rows);
        const product::Rows<T> rows(iq < of_group ? out : out2, int64_t(iq % of_group) * S::kBQ,
                                    right.rows, width);
#pragma unroll
        for (int j = 0; j < S::kQ; ++j)
#pragma unroll
          for (int i = 0; i < S::kP; ++i)
            rows.put(q0 + j * 16, p0 + i * 16, width, acc[i][j]);
      });
}

// Four neighbouring columns of a tile of the plan's rest: its shares added in order
template <typename S>
__device__ inline f32x4 joined(const Plan& plan, const float* shares, unsigned rest, int q, int p) {
  f32x4 s = {};
  for (int k = 0; k < plan.splits; ++k)
    s += *reinterpret_cast<const f32x4*>(
        shares + ((int64_t(k) * plan.rest() + rest) * S::kBQ + q) * S::kBP + p);
  return s;
}

// The rest of product_kernel's tiles; four rows of a tile to a workgroup of 256
template <typename T, typename S>
__global__ __launch_bounds__(S::kBP) void join_kernel(Plan plan, const float* shares, int64_t p_rows,
                                                      int64_t q_rows, T* out, T* out2) {
  const unsigned rest = blockIdx.x / (S::kBQ / 4), of_group = plan.nq / plan.groups;
  unsigned ip, iq;
  product::map_tile(plan.whole + rest, plan.np, plan.nq, ip, iq);
  const int q = int(blockIdx.x % (S::kBQ / 4)) * 4 + threadIdx.x / (S::kBP / 4),
            p = threadIdx.x % (S::kBP / 4) * 4;
  const int64_t row = int64_t(iq % of_group) * S::kBQ + q, col = int64_t(ip) * S::kBP + p;
  if (row >= q_rows || col >= p_rows) return;
  const f32x4 s = joined<S>(plan, shares, rest, q, p);
  const float x[4] = {s[0], s[1], s[2], s[3]};
  rowvec::store((iq < of_group ? out : out2) + row * p_rows + col, x);
}

// The rest of gate_up_kernel's tiles, eight rows of a tile to a workgroup
template <typename T, typename S, bool GRAD>
__global__ __launch_bounds__(S::kBP) void join_gate_up_kernel(Plan plan, const float* shares,
                                                              Sizes n, const T* dh, T* out) {
  constexpr int kF = S::kBP / 2, kHalf = kF / S::kWP;  // columns; of a wave's rows of one operand
  const unsigned rest = blockIdx.x / (S::kBQ / 8);
  unsigned ip, iq;
  product::map_tile(plan.whole + rest, plan.np, plan.nq, ip, iq);
  const int q = int(blockIdx.x % (S::kBQ / 8)) * 8 + threadIdx.x / (kF / 4),
            c = threadIdx.x % (kF / 4) * 4, p = c / kHalf * 2 * kHalf + c % kHalf;
  const int64_t m = int64_t(iq) * S::kBQ + q, f = int64_t(ip) * kF + c;
  if (m >= n.M || f >= n.F) return;
  float d[4] = {};
  if (GRAD) rowvec::load(dh + m * n.F + f, d);
  const Pair o = gate_up_of<GRAD>(joined<S>(plan, shares, rest, q, p),
                                  joined<S>(plan, shares, rest, q, p + kHalf), d, n.gelu);
  auto put = [&](int64_t at, f32x4 v) {
    const float x[4] = {v[0], v[1], v[2], v[3]};
    rowvec::store(out + at, x);
  };
  if constexpr (!GRAD) {
    put(m * n.F + f, o.a);
  } else if constexpr (sizeof(T) == 2) {
    const product::TwoPlanes a(o.a), b(o.b);
    const int64_t low = n.M * 2 * n.F;
    put(m * 2 * n.F + f, a.high);
    put(m * 2 * n.F + f + low, a.low);
    put((m * 2 + 1) * n.F + f, b.high);
    put((m * 2 + 1) * n.F + f + low, b.low);
  } else {
    put(m * 2 * n.F + f, o.a);
    put((m * 2 + 1) * n.F + f, o.b);
  }
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

// A matrix [rows][cols] made an operand: as it lies (`straight`), and turned into
// `cols` rows of `width` (rows, rounded up to 8; zeros there), `pitch` apart
// (`turned`); either may be NULL.  float32 becomes planes, `plane` and `turned_plane`
// elements apart.  64 x 64 tiles through LDS; up to three matrices in a launch.
struct Job {
  const void* in;
  int64_t rows, cols;
  uint16_t* straight;
  int64_t plane;
  uint16_t* turned;
  int64_t width, pitch, turned_plane;
  __host__ __device__ int64_t tiles() const {
    const int64_t high = width > rows ? width : rows;
    return ((cols + 63) / 64) * ((high + 63) / 64);
  }
};
struct Jobs {
  Job job[3];
  int n;
};
template <typename T>
__global__ __launch_bounds__(256) void operands_kernel(Jobs jobs) {
  constexpr int N = sizeof(T) == 4 ? kPlanes : 1;
  __shared__ uint16_t tile[N][64][66];
  int64_t at = blockIdx.x;
  int which = 0;
  while (which + 1 < jobs.n && at >= jobs.job[which].tiles()) at -= jobs.job[which++].tiles();
  const Job& j = jobs.job[which];
  const T* in = static_cast<const T*>(j.in);
  const int64_t across = (j.cols + 63) / 64;
  const int64_t c0 = at % across * 64, r0 = at / across * 64;
  for (int i = threadIdx.x; i < 64 * 16; i += 256) {
    const int r = i / 16, c = i % 16 * 4;
    const bool on = r0 + r < j.rows && c0 + c < j.cols;
    float v[4] = {};
    if (on) rowvec::load(in + (r0 + r) * j.cols + c0 + c, v);
    uint16_t p[4][N];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (N == 1)
        p[e][0] = uint16_t(__float_as_uint(v[e]) >> 16);
      else
        planes_of(v[e], p[e]);
#pragma unroll
      for (int k = 0; k < N; ++k) tile[k][c + e][r] = p[e][k];
    }
    if (on && j.straight)
#pragma unroll
      for (int k = 0; k < N; ++k)
        *reinterpret_cast<ushort4*>(j.straight + k * j.plane + (r0 + r) * j.cols + c0 + c) =
            make_ushort4(p[0][k], p[1][k], p[2][k], p[3][k]);
  }
  if (!j.turned) return;
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * 16; i += 256) {
    const int c = i / 16, r = i % 16 * 4;
    if (c0 + c < j.cols && r0 + r < j.width)
#pragma unroll
      for (int k = 0; k < N; ++k)
        *reinterpret_cast<ushort4*>(j.turned + k * j.turned_plane + (c0 + c) * j.pitch + r0 + r) =
            make_ushort4(tile[k][c][r], tile[k][c][r + 1], tile[k][c][r + 2], tile[k][c][r + 3]);
  }
}

// ---- launches

// a workspace taken in order; with a null base, its size
struct Arena {
  char* base;
  size_t at = 0;
  template <typename T>
  T* take(int64_t n) {
    T* p = reinterpret_cast<T*>(base + at);
    at += align256(size_t(n) * sizeof(T));
    return p;
  }
};

template <typename T>
constexpr int kCopies = sizeof(T) == 4 ? kPlanes : 1;
// rows of turned operands: whole vectors
int64_t pitch_of(int64_t M) { return (M + 7) / 8 * 8; }

// a matrix as an operand: a bf16 one as it is, a float32 one as planes, which `job`
// is told to make
template <typename T>
Operand as_rows(const void* p, int64_t rows, int64_t k, Arena& ws, Job& job) {
  job = {p, rows, k, nullptr, 0, nullptr, 0, 0, 0};
  if constexpr (sizeof(T) == 2) return {static_cast<const uint16_t*>(p), rows, 0, 0};
  job.straight = ws.take<uint16_t>(kPlanes * rows * k);
  job.plane = rows * k;
  return {job.straight, rows, rows * k, 0};
}
// and turned
void turn(Job& job, uint16_t* out, int64_t width, int64_t pitch, int64_t plane) {
  job.turned = out;
  job.width = width;
  job.pitch = pitch;
  job.turned_plane = plane;
}
template <typename T>
void prepare(const Jobs& jobs, hipStream_t stream) {
  int64_t n = 0;
  for (int i = 0; i < jobs.n; ++i) n += jobs.job[i].tiles();
  operands_kernel<T><<<unsigned(n), 256, 0, stream>>>(jobs);
}

constexpr int64_t kCUs = 256;

// Workgroups that a CU holds at a time
template <typename S>
constexpr int kPerCu = S::kLds <= 64 * 1024 ? 2 : 1;

// The plan for p x q outputs (in each of `groups`) of `pieces` pieces, and the
// microseconds that it is expected to take: a round of tiles takes 4 and `piece` for
// each piece, and the tiles that do not fill a round are split where that takes less,
// with 6 for joining the shares and their way to memory and back at 4.5 TB/s.
struct Choice {
  Plan plan;
  double time;
};
template <typename S>
Choice choose(int64_t p, int64_t q, unsigned groups, int64_t pieces, double piece) {
  const unsigned np = unsigned((p + S::kBP - 1) / S::kBP),
                 nq = unsigned((q + S::kBQ - 1) / S::kBQ) * groups;
  const unsigned at_once = unsigned(kCUs) * kPerCu<S>, n = np * nq;
  auto rounds = [&](unsigned items) { return double((items + at_once - 1) / at_once); };
  auto round = [&](int64_t m) { return 4.0 + piece * double(m); };
  Choice best = {{np, nq, groups, n, 1}, rounds(n) * round(pieces)};
  const unsigned rest = n % at_once;
  if (rest == 0) return best;
  for (int s = 2; s <= 16 && int64_t(s) * 4 <= pieces; ++s) {
    const int64_t share = (pieces + s - 1) / s;
    if ((pieces + share - 1) / share != s) continue;  // every share has a piece
    const double t = rounds(n - rest) * round(pieces) + rounds(rest * s) * round(share) + 6.0 +
                     double(rest) * s * (S::kBP * S::kBQ * 8) / 4.5e6;
    if (t < 0.97 * best.time) best = {{np, nq, groups, n - rest, s}, t};
  }
  return best;
}

// A product of a call: p x q outputs (in each of `groups`), sums over k in `terms`
struct Product {
  int64_t p, q;
  unsigned groups;
  int64_t k;
  int terms;
};
Product product_of(const GatedFfn& a, FfnProduct which) {
  const int terms = a.is_bf16 ? 1 : kTerms, of_grads = a.is_bf16 ? kGradPlanes : kTerms;
  switch (which) {
    case FfnProduct::kDx: return {a.D, a.M, 1, 2 * a.F, of_grads};
    case FfnProduct::kWeights: return {a.D, a.F, 2, pitch_of(a.M), of_grads};
    default: return {2 * a.F, a.M, 1, a.D, terms};  // g and u
  }
}

// f(shape, plan) with the tiles of the least time.  A piece takes 1.7 us in tiles of
// 256 x 256 on all CUs, 0.92 in 128 x 256, and 1.2 in 128 x 128, two to a CU: measured
// on 2048 x 8192 x 11008, one round of the first (293 us) and two of the others (323
// and 422).  With 1.05 for the second, backward passes of ten other sizes took from 7 %
// more (float32, 8192 rows of 392 to 1048: 490 for 459 us) to 2 % less (float32, 4096
// rows of 1536 to 4096: 1814 for 1845), 2 % more on average.
template <typename F>
hipError_t with_shape(const Product& m, F&& f) {
  const int64_t pieces = (m.k + product::kStep - 1) / product::kStep * m.terms;
  const Choice large = choose<Large>(m.p, m.q, m.groups, pieces, 1.7),
               medium = choose<Medium>(m.p, m.q, m.groups, pieces, 0.92),
               small = choose<Small>(m.p, m.q, m.groups, pieces, 1.2);
  if (small.time < large.time && small.time < medium.time) return f(Small{}, small.plan);
  if (medium.time < large.time) return f(Medium{}, medium.plan);
  return f(Large{}, large.plan);
}

template <typename S>
unsigned workgroups_of(const Plan& plan) {
  const unsigned most = unsigned(kCUs) * kPerCu<S>;
  return plan.items() < most ? plan.items() : most;
}
template <typename S>
float* take_shares(const Plan& plan, Arena& ws) {
  return plan.splits > 1
             ? ws.take<float>(int64_t(plan.rest()) * plan.splits * (S::kBP * S::kBQ)) : nullptr;
}

template <typename T, bool GRAD>
hipError_t gate_up(const GatedFfn& a, const Operand& wg, const Operand& wu, const Operand& x,
                   const void* dh, void* out, Arena& ws, hipStream_t stream, bool run) {
  const Product m = product_of(a, GRAD ? FfnProduct::kAgain : FfnProduct::kForward);
  const Sizes n = {a.M, a.D, a.F, m.terms, a.gelu};
  return with_shape(m, [&](auto shape, const Plan& plan) {
    using S = decltype(shape);
    float* shares = take_shares<S>(plan, ws);
    if (!run) return hipSuccess;
    const T* d = static_cast<const T*>(dh);
    T* o = static_cast<T*>(out);
    gate_up_kernel<T, S, GRAD><<<workgroups_of<S>(plan), S::kThreads, 0, stream>>>(
        wg, wu, x, n, plan, d, o, shares);
    if (shares)
      join_gate_up_kernel<T, S, GRAD><<<plan.rest() * (S::kBQ / 8), S::kBP, 0, stream>>>(
          plan, shares, n, d, o);
    return hipGetLastError();
  });
}

template <typename T>
hipError_t multiply(const Product& m, const Operand& l, const Operand& r, void* out, void* out2,
                    Arena& ws, hipStream_t stream, bool run) {
  return with_shape(m, [&](auto shape, const Plan& plan) {
    using S = decltype(shape);
    float* shares = take_shares<S>(plan, ws);
    if (!run) return hipSuccess;
    T *o = static_cast<T*>(out), *o2 = static_cast<T*>(out2);
    product_kernel<T, S><<<workgroups_of<S>(plan), S::kThreads, 0, stream>>>(
        l, r, m.k, m.terms, plan, o, o2, shares);
    if (shares)
      join_kernel<T, S><<<plan.rest() * (S::kBQ / 4), S::kBP, 0, stream>>>(plan, shares, m.p, m.q,
                                                                           o, o2);
    return hipGetLastError();
  });
}

// `run` false: only the workspace's size
template <typename T>
hipError_t forward(const GatedFfn& a, void* h, Arena& ws, hipStream_t stream, bool run) {
  if (a.M <= kFewRows) return run ? few_rows<T>(a, h, stream) : hipSuccess;
  Jobs jobs;
  jobs.n = 3;
  const Operand wg = as_rows<T>(a.w_gate, a.F, a.D, ws, jobs.job[0]),
                wu = as_rows<T>(a.w_up, a.F, a.D, ws, jobs.job[1]),
                x = as_rows<T>(a.x, a.M, a.D, ws, jobs.job[2]);
  if (run && sizeof(T) == 4) prepare<T>(jobs, stream);
  return gate_up<T, false>(a, wg, wu, x, nullptr, h, ws, stream, run);
}

template <typename T>
hipError_t backward(const GatedFfn& a, const GatedFfnGrads& g, Arena& ws, hipStream_t stream,
                    bool run) {
  const int64_t M = a.M, D = a.D, F = a.F, pitch = pitch_of(M);
  Jobs jobs;
  jobs.n = 3;
  const Operand wg = as_rows<T>(a.w_gate, F, D, ws, jobs.job[0]),
                wu = as_rows<T>(a.w_up, F, D, ws, jobs.job[1]),
                x = as_rows<T>(a.x, M, D, ws, jobs.job[2]);
  constexpr bool kFloat = sizeof(T) == 4;
  constexpr int kOfG = kFloat ? kPlanes : kGradPlanes;
  T* G = ws.take<T>((kFloat ? 1 : kGradPlanes) * M * 2 * F);  // float32, or planes
  const int64_t g_plane = M * 2 * F, wt_plane = D * 2 * F, xt_plane = D * pitch,
                gt_plane = 2 * F * pitch;
  uint16_t* wt = ws.take<uint16_t>(kCopies<T> * wt_plane);  // [D][Wg^T | Wu^T]
  uint16_t* xt = ws.take<uint16_t>(kCopies<T> * xt_plane);  // [D][M]
  uint16_t* gt = ws.take<uint16_t>(kOfG * gt_plane);        // [2F][M]
  turn(jobs.job[0], wt, F, 2 * F, wt_plane);
  turn(jobs.job[1], wt + F, F, 2 * F, wt_plane);
  turn(jobs.job[2], xt, pitch, pitch, xt_plane);
  if (run) prepare<T>(jobs, stream);
  hipError_t e = gate_up<T, true>(a, wg, wu, x, g.dh, G, ws, stream, run);
  if (e != hipSuccess) return e;
  Jobs more;
  more.n = kFloat ? 1 : kGradPlanes;
  Operand G_rows = as_rows<T>(G, M, 2 * F, ws, more.job[0]);
  turn(more.job[0], gt, pitch, pitch, gt_plane);
  if constexpr (!kFloat) {  // the second plane is a matrix of its own
    G_rows.plane = g_plane;
    (void)as_rows<T>(G + g_plane, M, 2 * F, ws, more.job[1]);
    turn(more.job[1], gt + gt_plane, pitch, pitch, gt_plane);
  }
  if (run) prepare<T>(more, stream);
  e = multiply<T>(product_of(a, FfnProduct::kDx), {wt, D, wt_plane, 0}, G_rows, g.dx, nullptr, ws,
                  stream, run);
  if (e != hipSuccess) return e;
  return multiply<T>(product_of(a, FfnProduct::kWeights), {xt, D, xt_plane, 0},
                     {gt, F, gt_plane, F * pitch}, g.dw_gate, g.dw_up, ws, stream, run);
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

GatedFfnTiles gated_ffn_tiles(const GatedFfn& a, FfnProduct which) {
  GatedFfnTiles t = {};
  if (which == FfnProduct::kForward && a.M <= ffn::kFewRows) return t;
  (void)ffn::with_shape(ffn::product_of(a, which), [&](auto shape, const ffn::Plan& plan) {
    using S = decltype(shape);
    t = {S::kBP, S::kBQ, plan.whole, plan.rest(), plan.splits};
    return hipSuccess;
  });
  return t;
}

hipError_t launch_gated_ffn_bwd(const GatedFfn& a, const GatedFfnGrads& g, void* workspace,
                                hipStream_t stream) {
  ffn::Arena ws{static_cast<char*>(workspace)};
  return a.is_bf16 ? ffn::backward<__hip_bfloat16>(a, g, ws, stream, true)
                   : ffn::backward<float>(a, g, ws, stream, true);
}

}  // namespace mlstm
