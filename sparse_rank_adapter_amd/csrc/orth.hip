// Updates orthogonalised by Newton-Schulz steps: X_0 = G / (|G| + eps), X <- a X + (b A + c A^2) X with
// A = X X^T, for n matrices of d x L ("wide") or L x d ("tall": the same on the transpose), d <= 256.
//
// Every X is Q G with Q a polynomial in the Gram matrix A_0 = G G^T, so the steps run on d x d matrices:
//   P = a I + b A + c A^2,  Q <- P Q,  A <- P (P A)   (all of them commute)
// and G itself is read twice, once for A_0 and once for Q G, where step by step on X it would be read and
// written ten times.  Small singular values grow by a factor of up to a^steps (485), and the rounding of
// A_0 with them: fp32 Gram matrices gave results 2e-4 off, and a last product summed in fp32 1e-5 to 3e-5
// (128 x 5120, singular values over three to four decades), so everything from A_0 on is fp64, on
// v_mfma_f64_16x16x4_f64.  The norm is the square root of A_0's trace.
//
// Measured: 8 fp32 matrices of 20480 x 128 253 us: A_0 63 us (3.0 GFLOP, bound by the fp64 matrix unit, 38 us at its peak, and
// by uneven shares: 480 workgroups on 256 CUs), 14 launches of 128 x 128 products 6 us each (latency), Q G 102 us (5.4 GFLOP,
// 68 us at the peak).  12 of 16 x 1024: 15 us, three launches.  4 of 64 x 8192: 71 us, 45 of them the steps (k_orth_small); in
// bf16 73, 8 of 20480 x 128 in bf16 276 (half the bytes, but the fp64 unit bounds both).
//
// The fp64 matrix instruction: lane l gives a[l % 16][l / 16] and b[l / 16][l % 16], and holds rows
// 4 v + l / 16 (v = 0 .. 3) of column l % 16 of the result.
#include <algorithm>

#include "rowvec.h"

namespace {
using sra_row::RowVec;

typedef double f64x4 __attribute__((ext_vector_type(4)));
typedef double f64x2 __attribute__((ext_vector_type(2)));

SRA_DEV f64x4 mfma(double a, double b, f64x4 c) { return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0); }
// (Kernels are bound to two waves a SIMD at least: with a wave's 512 registers allowed the compiler keeps accumulators in
// accumulation registers and copies them to and fro in every step.)
SRA_DEV int drow(int q, int v) { return 4 * v + q; }  // row of a result's element v in lane group q

// Operands come from a matrix through a buffer resource (under 2 GiB): one 32-bit addition an address, and what is outside
// reads as zero by the resource's length, or by an offset past it (kOut).  With 64-bit addresses and zeros selected for every
// element the vector instructions between the fp64 products took about as long as the products, which they do not run beside.
// (BUF = 1: rows of any number of whole words, whose last vector may run on into the next row; BUF = 2: rows of whole vectors.
// 6 x 250 x 20481 640 us, 20480 columns 584 without the masks and 621 with them.)
constexpr uint32_t kOut = 0x80000000u;
template <int N, typename E>
SRA_DEV void load_n(__amdgpu_buffer_rsrc_t r, uint32_t at, float (&f)[N]) {
  union { E e[N]; uint32_t w; u32x2 d; u32x4 q; } c;
  if constexpr (N * sizeof(E) == 16) c.q = __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0);
  else if constexpr (N * sizeof(E) == 8) c.d = __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, 0);
  else c.w = __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if constexpr (sizeof(E) == 4) f[k] = c.e[k];
    else f[k] = bf16_to_f32(c.e[k]);
  }
}
SRA_DEV __amdgpu_buffer_rsrc_t matrix(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, (int)bytes, 0x00020000);
}
// Without that (bf16 in odd rows, longer matrices): N consecutive elements at base + at, `left` of which are inside the row; what is
// outside is read from the matrix's first elements and replaced by zeros, so that loads still go out together.
template <int N, typename E>
SRA_DEV void load_each(const E* __restrict__ base, int64_t at, int64_t left, float (&f)[N]) {
  E e[N];
#pragma unroll
  for (int k = 0; k < N; ++k) e[k] = base[k < left ? at + k : 0];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    float v;
    if constexpr (sizeof(E) == 4) v = e[k];
    else v = bf16_to_f32(e[k]);
    f[k] = k < left ? v : 0.f;
  }
}
typedef uint32_t u32x2w __attribute__((ext_vector_type(2), aligned(4)));  // in memory at any whole word
typedef uint32_t u32x4w __attribute__((ext_vector_type(4), aligned(4)));
// N elements to p, `left` of which are inside the row.  VEC: p is a whole word's address
template <int N, bool VEC, typename E>
SRA_DEV void store_n(E* __restrict__ p, int64_t left, const double (&d)[N]) {
  if (VEC && left >= N) {
    union { float f[N]; __bf16 h[N]; uint32_t w[N]; } o;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if constexpr (sizeof(E) == 4) o.f[k] = (float)d[k];
      else o.h[k] = (__bf16)(float)d[k];
    }
    constexpr int W = N * sizeof(E) / 4;
    if constexpr (W == 4) *reinterpret_cast<u32x4w*>(p) = u32x4w{o.w[0], o.w[1], o.w[2], o.w[3]};
    else if constexpr (W == 2) *reinterpret_cast<u32x2w*>(p) = u32x2w{o.w[0], o.w[1]};
    else *reinterpret_cast<uint32_t*>(p) = o.w[0];
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (k < left) {
        float one[1] = {(float)d[k]};
        RowVec<E, 1>::store(p + k, one);
      }
  }
}

// ---- A_0's lower triangle in blocks of 32 x 32: part [n][pair][S][32][32], one slice of L per workgroup.
// A wave takes every fourth chunk of 16 of the slice; the four join in LDS.  Operands come straight from
// global memory (the waves of a CU share them in its cache): the product is bound by the matrix unit.
struct GramArgs {
  const void* G;
  int64_t L;
  int d, S;
  double* part;
};
template <typename E, bool TALL, int BUF>
struct GramRows {  // a block of 32 rows of X, of which a chunk of 16 columns makes the lane's operands f[row][4]
  const E* G;
  int64_t L;
  int d, row0;
  __amdgpu_buffer_rsrc_t r;
  uint32_t off[TALL ? 4 : 2];
  SRA_DEV GramRows(const E* G_, int64_t L_, int d_, int row0_) : G(G_), L(L_), d(d_), row0(row0_) {
    if constexpr (BUF) {
      const int l = threadIdx.x & 63, q = l >> 4, i = l & 15, E_ = (int)sizeof(E);
      r = matrix(TALL ? G : G + (int64_t)row0 * L, (TALL ? d : d - row0) * L * E_);
      if constexpr (TALL) {
#pragma unroll
        for (int j = 0; j < 4; ++j) off[j] = row0 + 2 * i < d ? (uint32_t)(((4 * j + q) * d + row0 + 2 * i) * E_) : kOut;
      } else {
#pragma unroll
        for (int x = 0; x < 2; ++x) off[x] = row0 + 16 * x + i < d ? (uint32_t)(((16 * x + i) * L + 4 * q) * E_) : kOut;
      }
    }
  }
  SRA_DEV void load(int64_t chunk, float (&f)[2][4]) const {
    const int l = threadIdx.x & 63, q = l >> 4, i = l & 15;
    if constexpr (!TALL) {  // rows row0 + 16 x + i; columns 16 chunk + 4 q + j
      const int64_t k = chunk * 16 + 4 * q;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if constexpr (BUF) {
          const int inside = (int)L - (int)chunk * 16;  // columns from the chunk's first on
          load_n<4, E>(r, 4 * q < inside ? off[x] + (uint32_t)chunk * (16 * sizeof(E)) : kOut, f[x]);
          if (BUF == 1 && inside < 16) {  // the last chunk: what follows the row's end is the next row
#pragma unroll
            for (int j = 1; j < 4; ++j) f[x][j] = 4 * q + j < inside ? f[x][j] : 0.f;
          }
        } else {
          const int row = row0 + 16 * x + i;
          load_each<4, E>(G, (int64_t)row * L + k, row < d ? L - k : 0, f[x]);
        }
      }
    } else {  // rows row0 + 2 i + x; columns 16 chunk + 4 j + q
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float two[2];
        if constexpr (BUF) {
          load_n<2, E>(r, off[j] + (uint32_t)chunk * (uint32_t)(16 * d * sizeof(E)), two);
          if (BUF == 1 && row0 + 32 > d) two[1] = row0 + 2 * i + 1 < d ? two[1] : 0.f;
        } else {
          const int64_t k = chunk * 16 + 4 * j + q;
          const int row = row0 + 2 * i;
          load_each<2, E>(G, k * d + row, k < L ? d - row : 0, two);
        }
        f[0][j] = two[0], f[1][j] = two[1];
      }
    }
  }
  static SRA_DEV int at(int x, int i) { return TALL ? 2 * i + x : 16 * x + i; }  // operand row (x, i) in the block
};

template <typename E, bool TALL, int BUF, bool DIAG>
SRA_DEV void gram_slice(const GramRows<E, TALL, BUF>& ra, const GramRows<E, TALL, BUF>& rb, int64_t c, int64_t c1, f64x4 (&acc)[2][2]) {
  float a[2][2][4], b[2][2][4];
  const auto load = [&](int64_t at, int k) {
    ra.load(at, a[k]);
    if constexpr (!DIAG) rb.load(at, b[k]);
    __builtin_amdgcn_sched_barrier(0);
  };
  const auto sum = [&](int k) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (!DIAG || r <= p) acc[p][r] = mfma((double)a[k][p][j], (double)(DIAG ? a : b)[k][r][j], acc[p][r]);
  };
  if (c >= c1) return;
  // the next chunk's loads go out before this one's products (and every load is used on every path: the compiler moves one
  // that is not behind the products)
  load(c, 0);
  for (; c + 8 < c1; c += 8) {
    load(c + 4, 1);
    sum(0);
    load(c + 8, 0);
    sum(1);
  }
  if (c + 4 < c1) {
    load(c + 4, 1);
    sum(0);
    sum(1);
  } else {
    sum(0);
  }
}

template <typename E, bool TALL, int BUF>
SRA_DEV void gram_body(const GramArgs& g, double (&red)[4][32 * 33]) {
  const int l = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = l >> 4, i = l & 15;
  int bi = 0, pair = blockIdx.x;  // pairs (bi, bj), bj <= bi, row after row
  while (pair > bi) pair -= ++bi;
  const int bj = pair;
  const E* const G = (const E*)g.G + (int64_t)blockIdx.z * g.d * g.L;
  const int64_t chunks = (g.L + 15) / 16;
  const int64_t c0 = chunks * blockIdx.y / g.S, c1 = chunks * (blockIdx.y + 1) / g.S;
  f64x4 acc[2][2];
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int y = 0; y < 2; ++y) acc[x][y] = f64x4{0., 0., 0., 0.};
  using B = GramRows<E, TALL, BUF>;
  const B ra(G, g.L, g.d, 32 * bi), rb(G, g.L, g.d, 32 * bj);
  if (bi == bj) gram_slice<E, TALL, BUF, true>(ra, rb, c0 + w, c1, acc);
  else gram_slice<E, TALL, BUF, false>(ra, rb, c0 + w, c1, acc);
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int r = B::at(x, drow(q, v)), c = B::at(y, i);
        if (bi != bj || y <= x) red[w][r * 33 + c] = acc[x][y][v];
        if (bi == bj && y < x) red[w][c * 33 + r] = acc[x][y][v];  // a diagonal block's fourth tile mirrors this one
      }
  __syncthreads();
  double* const out = g.part + (((int64_t)blockIdx.z * gridDim.x + blockIdx.x) * g.S + blockIdx.y) * 1024;
  for (int e = threadIdx.x; e < 1024; e += 256) {
    const int at = (e >> 5) * 33 + (e & 31);
    out[e] = (red[0][at] + red[1][at]) + (red[2][at] + red[3][at]);
  }
}
template <typename E, bool TALL, int BUF>
__global__ __launch_bounds__(256, 2) void k_orth_gram(GramArgs g) {
  __shared__ double red[4][32 * 33];
  gram_body<E, TALL, BUF>(g, red);
}
// A_0 [n][D][D] from the slices, in order, zeros past d (D = 16: a corner of the only block)
__global__ __launch_bounds__(256) void k_orth_join(const double* __restrict__ part, int S, int D, double* __restrict__ A) {
  const int t = (D + 31) / 32, pairs = t * (t + 1) / 2;
  const int e = blockIdx.x * 256 + threadIdx.x, r = e / D, c = e % D;
  const int hi = max(r, c), lo = min(r, c), bi = hi >> 5, bj = lo >> 5;
  // inside a diagonal block both triangles are there, equal up to rounding: take the lower
  const double* p = part + ((int64_t)(blockIdx.y * pairs + bi * (bi + 1) / 2 + bj) * S) * 1024 + (hi & 31) * 32 + (lo & 31);
  constexpr int U = 8;  // loads in flight
  double s = 0.;
  for (int k = 0; k < S; k += U) {
    double v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = p[(int64_t)min(k + u, S - 1) * 1024];
#pragma unroll
    for (int u = 0; u < U; ++u) s += k + u < S ? v[u] : 0.;
  }
  A[(int64_t)blockIdx.y * D * D + e] = s;
}

struct Steps {
  double a, b, c, eps;
  int n;
};
// 1 / (|G| + eps) from |G|^2.  It is multiplied up to its fifth power, which overflows where eps alone is far below fp32's
// range: a zero matrix takes 0, which gives its zeros as well.
SRA_DEV double scale_of(double trace, double eps) { return trace == 0. && eps > 0. ? 0. : 1. / (sqrt(trace) + eps); }

// ---- d <= 64: all steps of one matrix in one workgroup, its matrices in LDS.  All of them are symmetric (polynomials of
// A_0): wave w owns one 16 x 16 tile on or below the diagonal of every product and writes it on both sides.  Rows are
// D + 4 doubles apart, so 16 rows x 4 columns spread over the banks.
template <int D>
SRA_DEV f64x4 lds_mm(const double* A, const double* B, int ti, int tj) {  // tile (ti, tj) of A B, B symmetric
  constexpr int LD = D + 4;
  const int l = threadIdx.x & 63, q = l >> 4, i = l & 15;
  f64x4 acc = {0., 0., 0., 0.};
  const double *pa = A + (16 * ti + i) * LD + q, *pb = B + (16 * tj + i) * LD + q;
#pragma unroll
  for (int k = 0; k < D; k += 4) acc = mfma(pa[k], pb[k], acc);
  return acc;
}
// JOIN: A0 is the slices' sums [n][S][32][32], joined here in k_orth_join's order, up to kJoinSlices of them: 12 x 16 x 1024 with
// 8 slices 17.0 us with the launch, 14.9 without; at 32 slices 12 x 32 x 4096 takes 28.4 us with it and 32.7 without.
constexpr int kJoinSlices = 16;
template <int D, bool JOIN>
__global__ __launch_bounds__(64 * (D / 16) * (D / 16 + 1) / 2, 2) void k_orth_small(const double* __restrict__ A0, int S, int d,
                                                                              Steps st, double* __restrict__ Q) {
  constexpr int LD = D + 4, NT = 64 * (D / 16) * (D / 16 + 1) / 2, PER = (D * D + NT - 1) / NT;
  __shared__ double lds[4 * D * LD];
  double *const A = lds, *const P = A + D * LD, *const W = P + D * LD, *const X = W + D * LD;
  const int l = threadIdx.x & 63, w = threadIdx.x >> 6, q = l >> 4, i = l & 15;
  int ti = 0, tj = w;  // tiles (ti, tj), tj <= ti, row after row
  while (tj > ti) tj -= ++ti;
  double own[PER];  // this thread's elements of A_0
  if constexpr (JOIN) {
    static_assert(D <= 32, "one block of 32 x 32");
    A0 += (int64_t)blockIdx.x * S * 1024;
#pragma unroll
    for (int k = 0; k < PER; ++k) own[k] = 0.;
    constexpr int U = 8;  // slices in flight
    for (int c = 0; c < S; c += U) {
      double v[U][PER];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          const int e = min((int)threadIdx.x + k * NT, D * D - 1), row = e / D, cl = e % D;
          v[u][k] = A0[min(c + u, S - 1) * 1024 + max(row, cl) * 32 + min(row, cl)];
        }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < PER; ++k) own[k] += c + u < S ? v[u][k] : 0.;
    }
  } else {
    A0 += (int64_t)blockIdx.x * D * D;
#pragma unroll
    for (int k = 0; k < PER; ++k) own[k] = A0[min((int)threadIdx.x + k * NT, D * D - 1)];
  }
  const auto put_own = [&](double f) {
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int e = threadIdx.x + k * NT;
      if (e < D * D) A[(e / D) * LD + e % D] = own[k] * f;
    }
  };
  put_own(1.);
  __syncthreads();
  double tr = 0.;
  for (int k = l; k < d; k += 64) tr += A[k * (LD + 1)];
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) tr += __shfl_xor(tr, m, 64);
  const double s = scale_of(tr, st.eps);
  __syncthreads();
  put_own(s * s);
  __syncthreads();
  const int col = 16 * tj + i;
  const auto put = [&](double* M, const f64x4& v) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = 16 * ti + drow(q, k);
      M[row * LD + col] = v[k];
      if (ti != tj) M[col * LD + row] = v[k];
    }
  };
  for (int k = 0; k < st.n; ++k) {
    f64x4 p = lds_mm<D>(A, A, ti, tj);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int row = 16 * ti + drow(q, v);
      p[v] = (row == col ? st.a : 0.) + st.b * A[row * LD + col] + st.c * p[v];
    }
    put(P, p);
    __syncthreads();
    f64x4 x = p;
    if (k > 0) x = lds_mm<D>(P, X, ti, tj);
    if (k + 1 == st.n) {
      double* const o = Q + (int64_t)blockIdx.x * D * D;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int row = 16 * ti + drow(q, v);
        o[row * D + col] = s * x[v];
        if (ti != tj) o[col * D + row] = s * x[v];
      }
      break;
    }
    put(W, lds_mm<D>(P, A, ti, tj));
    __syncthreads();  // P A is there, and A and X have been read
    const f64x4 n = lds_mm<D>(P, W, ti, tj);
    put(A, n);
    put(X, x);
    __syncthreads();
  }
}

// ---- d > 64: every product of a step as a launch of its own (one workgroup would take 14 us a product at d = 128, its CU's
// share of the fp64 rate).  A workgroup has a 16 x 16 tile on or below the diagonal and writes it on both sides, its waves a
// quarter of the reduction each, all of whose
// operands are loaded at once: a launch is bound by that latency.
// job z: C_z = u I + v A_z + w (A_z B_z), B_z symmetric; u, v and w are multiplied by the powers pu, pv and pw
// of s = 1 / (sqrt(trace of `norm`) + eps)
struct MmJob {
  const double *A, *B;
  double* C;
  double u, v, w;
  int pu, pv, pw;
};
struct MmArgs {
  MmJob job[2];
  const double* norm;
  int D, d, n;
  double eps;
};
__global__ __launch_bounds__(256, 2) void k_orth_mm(MmArgs g) {
  __shared__ double part[4][256], scale;
  const int t = threadIdx.x, l = t & 63, w = t >> 6, q = l >> 4, i = l & 15, D = g.D, KW = D / 4;
  // the matrix in the low digits: with eight of them (or 16, ...) each stays on one XCD, whose L2 holds it
  const int mat = blockIdx.x % g.n;
  int ti = 0, tj = blockIdx.x / g.n;  // tiles (ti, tj), tj <= ti, row after row
  while (tj > ti) tj -= ++ti;
  const int r0 = 16 * ti, c0 = 16 * tj;
  const MmJob& j = g.job[blockIdx.y];
  const int64_t at = (int64_t)mat * D * D;
  const double *const pa = j.A + at + (int64_t)(r0 + i) * D + KW * w + 2 * q, *const pb = j.B + at + (int64_t)(c0 + i) * D + KW * w + 2 * q;
  f64x2 a[8], b[8];  // KW <= 64: everything the wave needs, in flight at once
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int k8 = min(8 * k, KW - 8);  // past the end: not used
    a[k] = *reinterpret_cast<const f64x2*>(pa + k8);
    b[k] = *reinterpret_cast<const f64x2*>(pb + k8);
  }
  const int row = r0 + (t >> 4), col = c0 + (t & 15);  // this thread's element of the result
  const double own = j.v != 0. ? j.A[at + (int64_t)row * D + col] : 0.;
  if ((j.pu | j.pv | j.pw) && w == 0) {
    double tr = 0.;
    for (int k = l; k < g.d; k += 64) tr += g.norm[at + (int64_t)k * (D + 1)];
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) tr += __shfl_xor(tr, m, 64);
    if (l == 0) scale = scale_of(tr, g.eps);
  }
  f64x4 acc = {0., 0., 0., 0.};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (8 * k < KW) {
      acc = mfma(a[k][0], b[k][0], acc);
      acc = mfma(a[k][1], b[k][1], acc);
    }
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) part[w][drow(q, v) * 16 + i] = acc[v];
  __syncthreads();
  double u = j.u, v = j.v, wt = j.w;
  for (int k = 0; k < j.pu; ++k) u *= scale;
  for (int k = 0; k < j.pv; ++k) v *= scale;
  for (int k = 0; k < j.pw; ++k) wt *= scale;
  const double sum = (part[0][t] + part[1][t]) + (part[2][t] + part[3][t]);
  const double r = wt * sum + v * own + (row == col ? u : 0.);
  j.C[at + (int64_t)row * D + col] = r;
  if (ti != tj) j.C[at + (int64_t)col * D + row] = r;
}

// ---- O = Q X.  A wave owns 16 FR rows of Q against 64 columns of X (rows of the tall matrix); the waves of a
// workgroup take neighbouring rows of Q, so they share X in the CU's cache.  Q [n][D][D] is symmetric.
template <typename E, bool TALL, int BUF, int FR>
SRA_DEV void apply_body(const double* __restrict__ Q, const E* __restrict__ G, int64_t L, int d, int D, E* __restrict__ O) {
  const int l = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = l >> 4, i = l & 15, E_ = (int)sizeof(E);
  const int nrb = (d + 16 * FR - 1) / (16 * FR);
  const int64_t job = (int64_t)blockIdx.x * 4 + w, cb = job / nrb * 64;
  const int r0 = (int)(job % nrb) * 16 * FR;
  if (cb >= L) return;
  const int64_t at = (int64_t)blockIdx.y * d * L;
  G += at;
  O += at;
  const __amdgpu_buffer_rsrc_t rq = matrix(Q + (int64_t)blockIdx.y * D * D, (int64_t)D * D * 8);
  const __amdgpu_buffer_rsrc_t rg = matrix(TALL ? G + cb * d : G, (TALL ? (L - cb) * d : (int64_t)d * L) * E_);
  uint32_t qo[FR], go[4];  // the lane's first operands
#pragma unroll
  for (int x = 0; x < FR; ++x) qo[x] = (uint32_t)(((r0 + (TALL ? FR * i + x : 16 * x + i)) * D + 4 * q) * 8);
  if constexpr (BUF) {
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      if constexpr (TALL) go[y] = (uint32_t)(((16 * y + i) * d + 4 * q) * E_);
      else go[y] = cb + 4 * i < L ? (uint32_t)(((4 * q + y) * L + cb + 4 * i) * E_) : kOut;
    }
  }
  f64x4 acc[FR][4];
#pragma unroll
  for (int x = 0; x < FR; ++x)
#pragma unroll
    for (int g = 0; g < 4; ++g) acc[x][g] = f64x4{0., 0., 0., 0.};
  struct Step {  // the operands of 16 of the reduction
    f64x2 a[FR][2];  // Q's rows: wide r0 + 16 x + i, tall r0 + FR i + x; columns k0 + 4 q ..
    float f[4][4];   // wide f[j][g] = X[k0 + 4 q + j][cb + 4 i + g]; tall f[g][j] = G[cb + 16 g + i][k0 + 4 q + j]
  };
  const auto load = [&](int k0, Step& s) {
#pragma unroll
    for (int x = 0; x < FR; ++x)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        union { u32x4 w; f64x2 d; } c;
        c.w = __builtin_amdgcn_raw_buffer_load_b128(rq, qo[x] + (uint32_t)k0 * 8 + 16 * h, 0, 0);
        s.a[x][h] = c.d;
      }
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      if constexpr (!TALL) {
        if constexpr (BUF) {
          load_n<4, E>(rg, go[y] + (uint32_t)k0 * (uint32_t)(L * E_), s.f[y]);
        } else {
          const int k = k0 + 4 * q + y;
          load_each<4, E>(G, (int64_t)k * L + cb + 4 * i, k < d ? L - cb - 4 * i : 0, s.f[y]);
        }
      } else {
        if constexpr (BUF) {
          load_n<4, E>(rg, k0 < d - 4 * q ? go[y] + (uint32_t)(k0 * E_) : kOut, s.f[y]);
          if (BUF == 1 && k0 + 16 > d) {
#pragma unroll
            for (int j = 1; j < 4; ++j) s.f[y][j] = k0 + 4 * q + j < d ? s.f[y][j] : 0.f;
          }
        } else {
          const int64_t c = cb + 16 * y + i;
          load_each<4, E>(G, c * d + k0 + 4 * q, c < L ? d - k0 - 4 * q : 0, s.f[y]);
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // as above: before the products
  };
  const auto sum = [&](const Step& s) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int x = 0; x < FR; ++x)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const double a = s.a[x][j / 2][j % 2];
          if constexpr (!TALL) acc[x][g] = mfma(a, (double)s.f[j][g], acc[x][g]);
          else acc[x][g] = mfma((double)s.f[g][j], a, acc[x][g]);
        }
  };
  Step s0, s1;
  int k0 = 0;
  load(0, s0);
  for (; k0 + 32 < d; k0 += 32) {
    load(k0 + 16, s1);
    sum(s0);
    load(k0 + 32, s0);
    sum(s1);
  }
  if (k0 + 16 < d) {
    load(k0 + 16, s1);
    sum(s0);
    sum(s1);
  } else {
    sum(s0);
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    if constexpr (!TALL) {  // rows r0 + 16 x + drow, columns cb + 4 i + g
#pragma unroll
      for (int x = 0; x < FR; ++x) {
        const int row = r0 + 16 * x + drow(q, v);
        const double o[4] = {acc[x][0][v], acc[x][1][v], acc[x][2][v], acc[x][3][v]};
        store_n<4, BUF != 0, E>(O + (int64_t)row * L + cb + 4 * i, row < d ? L - cb - 4 * i : 0, o);
      }
    } else {  // rows cb + 16 g + drow of the tall matrix, columns r0 + FR i + x
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int64_t c = cb + 16 * g + drow(q, v);
        double o[FR];
#pragma unroll
        for (int x = 0; x < FR; ++x) o[x] = acc[x][g][v];
        store_n<FR, BUF != 0 && FR == 2, E>(O + c * d + r0 + FR * i, c < L ? d - r0 - FR * i : 0, o);
      }
    }
  }
}
template <typename E, bool TALL, int BUF, int FR>
__global__ __launch_bounds__(256, 2) void k_orth_apply(const double* __restrict__ Q, const E* __restrict__ G, int64_t L, int d,
                                                    int D, E* __restrict__ O) {
  apply_body<E, TALL, BUF, FR>(Q, G, L, d, D, O);
}

// slices of L: about 512 workgroups over the matrices and pairs, each with 8 chunks of 16 at least
int slices_of(int64_t n, int pairs, int64_t L) {
  const int64_t chunks = (L + 15) / 16;
  return (int)std::max<int64_t>(1, std::min<int64_t>(chunks / 8, 512 / std::max<int64_t>(1, n * pairs)));
}
int dim_of(int64_t d) { return d <= 16 ? 16 : (int)((d + 31) / 32 * 32); }
struct Layout {
  int d, D, pairs, S;
  int64_t L;
  size_t part, mat;  // bytes of the slices and of one set of D x D matrices
};
Layout layout_of(int64_t n, int64_t rows, int64_t cols) {
  Layout y;
  y.d = (int)std::min(rows, cols);
  y.L = std::max(rows, cols);
  y.D = dim_of(y.d);
  const int t = (y.D + 31) / 32;
  y.pairs = t * (t + 1) / 2;
  y.S = slices_of(n, y.pairs, y.L);
  y.part = (size_t)n * y.pairs * y.S * 1024 * sizeof(double);
  y.mat = (size_t)n * y.D * y.D * sizeof(double);
  return y;
}

}  // namespace

namespace sra {

bool orth_ok(int64_t rows, int64_t cols) { return std::min(rows, cols) <= 256; }
// slices of the Gram matrix, the Gram matrix, Q, and above d = 64 also A twice, P, P A and a second Q
size_t orth_ws(int64_t n, int64_t rows, int64_t cols) {
  if (n <= 0 || rows <= 0 || cols <= 0) return 0;
  const Layout y = layout_of(n, rows, cols);
  return y.part + y.mat * (y.D <= 64 ? 2 : 7);
}

template <typename E, bool TALL>
static hipError_t orth(const E* G, int64_t n, const Layout& y, const Steps& st, E* O, void* ws, hipStream_t s) {
  double* const part = (double*)ws;
  double* const m0 = (double*)((uint8_t*)ws + y.part);
  const size_t me = y.mat / sizeof(double);
  const GramArgs g{G, y.L, y.d, y.S, part};
  const dim3 gg((unsigned)y.pairs, (unsigned)y.S, (unsigned)n);
  // rows that begin at whole words (loads need no more than that), and 32-bit offsets up to the 16 rows past the last that a
  // step of the reduction may ask for
  const bool small = ((int64_t)y.d + 16) * y.L * (int64_t)sizeof(E) < ((int64_t)1 << 31);
  const bool words = small && (sizeof(E) == 4 || (TALL ? y.d : y.L) % 2 == 0);
#define SRA_GRAM(BUF) launch(SRA_KERNEL_ORTH, k_orth_gram<E, TALL, BUF>, gg, dim3(256), 0, s, g)
  if (words && (TALL ? y.d % 2 == 0 : y.L % 4 == 0)) SRA_GRAM(2);
  else if (words) SRA_GRAM(1);
  else SRA_GRAM(0);
#undef SRA_GRAM
  double* const a0 = m0;
  double* q0 = m0 + me;
  const bool join = y.D <= 32 && y.S <= kJoinSlices;
  if (!join)
    hipLaunchKernelGGL(k_orth_join, dim3((unsigned)(y.D * y.D / 256), (unsigned)n), dim3(256), 0, s, part, y.S, y.D, a0);
#define SRA_SMALL(D, JOIN, NT) \
  hipLaunchKernelGGL((k_orth_small<D, JOIN>), dim3((unsigned)n), dim3(NT), 0, s, JOIN ? part : a0, y.S, y.d, st, q0)
  if (y.D == 16) {
    if (join) SRA_SMALL(16, true, 64);
    else SRA_SMALL(16, false, 64);
  } else if (y.D == 32) {
    if (join) SRA_SMALL(32, true, 192);
    else SRA_SMALL(32, false, 192);
  } else if (y.D == 64) {
    SRA_SMALL(64, false, 640);
#undef SRA_SMALL
  } else {
    double *q1 = m0 + 2 * me, *a = m0 + 3 * me, *an = m0 + 4 * me, *const p = m0 + 5 * me, *const w = m0 + 6 * me;
    const unsigned tiles = (unsigned)(y.D / 16 * (y.D / 16 + 1) / 2);
    MmArgs m{};
    m.norm = a0, m.D = y.D, m.d = y.d, m.n = (int)n, m.eps = st.eps;
    const auto run = [&](unsigned jobs) { hipLaunchKernelGGL(k_orth_mm, dim3(tiles * (unsigned)n, jobs), dim3(256), 0, s, m); };
    const double* cur = a0;  // A of this step; the first is A_0 itself, with the norm's powers in the factors
    for (int k = 0; k < st.n; ++k) {
      const bool first = k == 0, last = k + 1 == st.n;
      const int s1 = first && last ? 1 : 0;
      double* const P = first ? q0 : p;  // the first Q is P itself
      m.job[0] = first ? MmJob{cur, cur, P, st.a, st.b, st.c, s1, 2 + s1, 4 + s1} : MmJob{cur, cur, P, st.a, st.b, st.c, 0, 0, 0};
      run(1);
      unsigned jobs = 0;
      if (!first) m.job[jobs++] = MmJob{P, q0, q1, 0., 0., 1., 0, 0, last ? 1 : 0};  // Q <- P Q, times s at the end
      if (!last) m.job[jobs++] = MmJob{P, cur, w, 0., 0., 1., 0, 0, first ? 2 : 0};
      if (jobs) run(jobs);
      if (!last) {
        m.job[0] = MmJob{P, w, an, 0., 0., 1., 0, 0, 0};
        run(1);
      }
      if (!first) std::swap(q0, q1);
      std::swap(a, an);
      cur = a;
    }
  }
  const double* const Q = q0;
  // 32 rows of Q a wave, or 16 where that leaves fewer than 1024 waves
  const int fr = y.d <= 16 || n * ((y.L + 63) / 64) * ((y.d + 31) / 32) < 1024 ? 1 : 2;
  const int nrb = (y.d + 16 * fr - 1) / (16 * fr);
  const int64_t jobs = (y.L + 63) / 64 * nrb;
  const dim3 ga((unsigned)((jobs + 3) / 4), (unsigned)n);
  const int buf = !words ? 0 : (TALL ? y.d : y.L) % 4 == 0 ? 2 : 1;
#define SRA_APPLY(BUF, FR) launch(SRA_KERNEL_ORTH, k_orth_apply<E, TALL, BUF, FR>, ga, dim3(256), 0, s, Q, G, y.L, y.d, y.D, O)
  if (fr == 1) {
    if (buf == 2) SRA_APPLY(2, 1);
    else if (buf == 1) SRA_APPLY(1, 1);
    else SRA_APPLY(0, 1);
  } else {
    if (buf == 2) SRA_APPLY(2, 2);
    else if (buf == 1) SRA_APPLY(1, 2);
    else SRA_APPLY(0, 2);
  }
#undef SRA_APPLY
  return hipGetLastError();
}

hipError_t launch_orth(int dtype, const void* G, int64_t n, int64_t rows, int64_t cols, int steps, const double* abc,
                       double eps, void* O, void* ws, hipStream_t s) {
  if (n <= 0 || rows <= 0 || cols <= 0) return hipSuccess;
  const Layout y = layout_of(n, rows, cols);
  const Steps st{abc[0], abc[1], abc[2], eps, steps};
  const bool tall = rows > cols;
  if (dtype == SRA_BF16)
    return tall ? orth<uint16_t, true>((const uint16_t*)G, n, y, st, (uint16_t*)O, ws, s)
                : orth<uint16_t, false>((const uint16_t*)G, n, y, st, (uint16_t*)O, ws, s);
  return tall ? orth<float, true>((const float*)G, n, y, st, (float*)O, ws, s)
              : orth<float, false>((const float*)G, n, y, st, (float*)O, ws, s);
}

}  // namespace sra
