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
// The fp64 matrix instruction: lane l gives a[l % 16][l / 16] and b[l / 16][l % 16], and holds rows
// 4 v + l / 16 (v = 0 .. 3) of column l % 16 of the result.
#include <algorithm>

#include "rowvec.h"

namespace {
using sra_row::RowVec;

typedef double f64x4 __attribute__((ext_vector_type(4)));
typedef double f64x2 __attribute__((ext_vector_type(2)));

SRA_DEV f64x4 mfma(double a, double b, f64x4 c) { return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0); }
SRA_DEV int drow(int q, int v) { return 4 * v + q; }  // row of a result's element v in lane group q

// N consecutive elements at p, `left` of which are inside the row (VEC: aligned, and a whole vector is in or out)
template <int N, bool VEC, typename E>
SRA_DEV void load_n(const E* __restrict__ p, int64_t left, float (&f)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) f[k] = 0.f;
  if constexpr (VEC && sizeof(E) == 4 && N == 4) {
    if (left > 0) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] = v[k];
    }
  } else if constexpr (VEC && sizeof(E) == 4) {
    if (left > 0) {
      const u32x2 v = *reinterpret_cast<const u32x2*>(p);
      f[0] = __uint_as_float(v[0]), f[1] = __uint_as_float(v[1]);
    }
  } else if constexpr (VEC) {
    if (left > 0) {
      uint32_t w[N / 2];
      if constexpr (N == 4) {
        const u32x2 v = *reinterpret_cast<const u32x2*>(p);
        w[0] = v[0], w[1] = v[1];
      } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
      }
#pragma unroll
      for (int k = 0; k < N / 2; ++k) {
        f[2 * k] = __uint_as_float(w[k] << 16);
        f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (k < left) {
        float one[1];
        RowVec<E, 1>::load(p + k, one);
        f[k] = one[0];
      }
  }
}
template <int N, bool VEC, typename E>
SRA_DEV void store_n(E* __restrict__ p, int64_t left, const double (&d)[N]) {
  if constexpr (VEC) {
    if (left <= 0) return;
    if constexpr (sizeof(E) == 4) {
      if constexpr (N == 4) *reinterpret_cast<f32x4*>(p) = f32x4{(float)d[0], (float)d[1], (float)d[2], (float)d[3]};
      else *reinterpret_cast<u32x2*>(p) = u32x2{__float_as_uint((float)d[0]), __float_as_uint((float)d[1])};
    } else {
      union { __bf16 h[N]; uint32_t w[N / 2]; } o;
#pragma unroll
      for (int k = 0; k < N; ++k) o.h[k] = (__bf16)(float)d[k];
      if constexpr (N == 4) *reinterpret_cast<u32x2*>(p) = u32x2{o.w[0], o.w[1]};
      else *reinterpret_cast<uint32_t*>(p) = o.w[0];
    }
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
template <typename E, bool TALL, bool VEC>
struct GramBlock {  // a block of 32 rows of X over a chunk of 16 columns, as the lane's operands
  float f[2][4];
  SRA_DEV void load(const E* __restrict__ G, int64_t L, int d, int row0, int64_t chunk, int64_t end) {
    const int l = threadIdx.x & 63, q = l >> 4, i = l & 15;
    if constexpr (!TALL) {  // rows row0 + 16 x + i; columns 16 chunk + 4 q + j
      const int64_t k = chunk * 16 + 4 * q;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int row = row0 + 16 * x + i;
        load_n<4, VEC, E>(G + (int64_t)row * L + k, row < d ? min(end, L) - k : 0, f[x]);
      }
    } else {  // rows row0 + 2 i + x; columns 16 chunk + 4 j + q
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t k = chunk * 16 + 4 * j + q;
        const int row = row0 + 2 * i;
        float two[2];
        load_n<2, VEC, E>(G + k * d + row, k < min(end, L) ? d - row : 0, two);
        f[0][j] = two[0], f[1][j] = two[1];
      }
    }
  }
  static SRA_DEV int at(int x, int i) { return TALL ? 2 * i + x : 16 * x + i; }  // operand row (x, i) in the block
};

template <typename E, bool TALL, bool VEC>
__global__ __launch_bounds__(256) void k_orth_gram(GramArgs g) {
  __shared__ double red[4][32 * 33];
  const int l = threadIdx.x & 63, w = threadIdx.x >> 6, q = l >> 4, i = l & 15;
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
  using B = GramBlock<E, TALL, VEC>;
  B a, b, an, bn;
  const bool diag = bi == bj;
  int64_t c = c0 + w;
  if (c < c1) {
    a.load(G, g.L, g.d, 32 * bi, c, g.L);
    if (!diag) b.load(G, g.L, g.d, 32 * bj, c, g.L);
  }
  for (; c < c1; c += 4) {
    if (c + 4 < c1) {
      an.load(G, g.L, g.d, 32 * bi, c + 4, g.L);
      if (!diag) bn.load(G, g.L, g.d, 32 * bj, c + 4, g.L);
    }
    if (diag) b = a;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) acc[x][y] = mfma((double)a.f[x][j], (double)b.f[y][j], acc[x][y]);
    a = an;
    b = bn;
  }
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int v = 0; v < 4; ++v) red[w][B::at(x, drow(q, v)) * 33 + B::at(y, i)] = acc[x][y][v];
  __syncthreads();
  double* const out = g.part + (((int64_t)blockIdx.z * gridDim.x + blockIdx.x) * g.S + blockIdx.y) * 1024;
  for (int e = threadIdx.x; e < 1024; e += 256) {
    const int at = (e >> 5) * 33 + (e & 31);
    out[e] = (red[0][at] + red[1][at]) + (red[2][at] + red[3][at]);
  }
}
SRA_DEV double gram_at(const double* part, int S, int r, int c) {  // element (r, c) of A_0 from the slices, in order
  const int hi = max(r, c), lo = min(r, c), bi = hi >> 5, bj = lo >> 5;
  // inside a diagonal block both triangles are there, equal up to rounding: take the lower
  const double* p = part + ((int64_t)(bi * (bi + 1) / 2 + bj) * S) * 1024 + (hi & 31) * 32 + (lo & 31);
  double s = 0.;
  for (int k = 0; k < S; ++k) s += p[(int64_t)k * 1024];
  return s;
}

struct Steps {
  double a, b, c, eps;
  int n;
};

// ---- d <= 64: all steps of one matrix in one workgroup, its matrices in LDS.  Wave w owns the 16 x 16 tile
// (w / T, w % T) of every product.  Rows are D + 4 doubles apart, so 16 rows x 4 columns spread over the banks.
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
template <int D>
__global__ __launch_bounds__(D * D / 4) void k_orth_small(const double* __restrict__ part, int S, int d, Steps st,
                                                          double* __restrict__ Q) {
  constexpr int LD = D + 4, T = D / 16;
  __shared__ double lds[4 * D * LD];
  double *const A = lds, *const P = A + D * LD, *const W = P + D * LD, *const X = W + D * LD;
  const int l = threadIdx.x & 63, w = threadIdx.x >> 6, q = l >> 4, i = l & 15, ti = w / T, tj = w % T;
  constexpr int pairs = (D / 32) * (D / 32 + 1) / 2;
  part += (int64_t)blockIdx.x * pairs * S * 1024;
  for (int e = threadIdx.x; e < D * D; e += blockDim.x) A[(e / D) * LD + e % D] = gram_at(part, S, e / D, e % D);
  __syncthreads();
  double tr = 0.;
  for (int k = 0; k < d; ++k) tr += A[k * LD + k];
  const double s = 1. / (sqrt(tr) + st.eps);
  __syncthreads();
  for (int e = threadIdx.x; e < D * D; e += blockDim.x) A[(e / D) * LD + e % D] *= s * s;
  __syncthreads();
  const int col = 16 * tj + i;
  for (int k = 0; k < st.n; ++k) {
    f64x4 p = lds_mm<D>(A, A, ti, tj);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int row = 16 * ti + drow(q, v);
      p[v] = (row == col ? st.a : 0.) + st.b * A[row * LD + col] + st.c * p[v];
      P[row * LD + col] = p[v];
    }
    __syncthreads();
    f64x4 x = p;
    if (k > 0) x = lds_mm<D>(P, X, ti, tj);
    if (k + 1 == st.n) {
      double* const o = Q + (int64_t)blockIdx.x * D * D;
#pragma unroll
      for (int v = 0; v < 4; ++v) o[(16 * ti + drow(q, v)) * D + col] = s * x[v];
      break;
    }
    const f64x4 t = lds_mm<D>(P, A, ti, tj);
#pragma unroll
    for (int v = 0; v < 4; ++v) W[(16 * ti + drow(q, v)) * LD + col] = t[v];
    __syncthreads();  // P A is there, and A and X have been read
    const f64x4 n = lds_mm<D>(P, W, ti, tj);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      A[(16 * ti + drow(q, v)) * LD + col] = n[v];
      X[(16 * ti + drow(q, v)) * LD + col] = x[v];
    }
    __syncthreads();
  }
}

// ---- d > 64: A_0 from its slices, then every product of a step as a launch of its own, 32 x 32 of the result a
// workgroup (one workgroup would take 14 us a product at d = 128, its CU's share of the fp64 rate).
__global__ __launch_bounds__(256) void k_orth_join(const double* __restrict__ part, int S, int D, double* __restrict__ A) {
  const int pairs = (D / 32) * (D / 32 + 1) / 2;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  A[(int64_t)blockIdx.y * D * D + e] =
      gram_at(part + (int64_t)blockIdx.y * pairs * S * 1024, S, (int)(e / D), (int)(e % D));
}
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
  int D, d;
  double eps;
};
__global__ __launch_bounds__(256) void k_orth_mm(MmArgs g) {
  const int l = threadIdx.x & 63, w = threadIdx.x >> 6, q = l >> 4, i = l & 15, D = g.D, T = D / 32;
  const int mat = blockIdx.y, r0 = 32 * (blockIdx.x / T) + 16 * (w >> 1), c0 = 32 * (blockIdx.x % T) + 16 * (w & 1);
  const MmJob& j = g.job[blockIdx.z];
  const int64_t at = (int64_t)mat * D * D;
  double s = 1.;
  if (j.pu | j.pv | j.pw) {
    double tr = 0.;
    for (int k = l; k < g.d; k += 64) tr += g.norm[at + (int64_t)k * (D + 1)];
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) tr += __shfl_xor(tr, m, 64);
    s = 1. / (sqrt(tr) + g.eps);
  }
  f64x4 acc = {0., 0., 0., 0.};
  const double *pa = j.A + at + (int64_t)(r0 + i) * D + 4 * q, *pb = j.B + at + (int64_t)(c0 + i) * D + 4 * q;
#pragma unroll 4
  for (int k = 0; k < D; k += 16) {
    const f64x2 a0 = *reinterpret_cast<const f64x2*>(pa + k), a1 = *reinterpret_cast<const f64x2*>(pa + k + 2);
    const f64x2 b0 = *reinterpret_cast<const f64x2*>(pb + k), b1 = *reinterpret_cast<const f64x2*>(pb + k + 2);
    acc = mfma(a0[0], b0[0], acc);
    acc = mfma(a0[1], b0[1], acc);
    acc = mfma(a1[0], b1[0], acc);
    acc = mfma(a1[1], b1[1], acc);
  }
  double u = j.u, v = j.v, wt = j.w;
  for (int k = 0; k < j.pu; ++k) u *= s;
  for (int k = 0; k < j.pv; ++k) v *= s;
  for (int k = 0; k < j.pw; ++k) wt *= s;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int row = r0 + drow(q, e), col = c0 + i;
    double o = wt * acc[e];
    if (j.v != 0.) o += v * j.A[at + (int64_t)row * D + col];
    if (row == col) o += u;
    j.C[at + (int64_t)row * D + col] = o;
  }
}

// ---- O = Q X.  A wave owns 16 FR rows of Q against 64 columns of X (rows of the tall matrix); the waves of a
// workgroup take neighbouring rows of Q, so they share X in the CU's cache.  Q [n][D][D] is symmetric.
template <typename E, bool TALL, bool VEC, int FR>
__global__ __launch_bounds__(256) void k_orth_apply(const double* __restrict__ Q, const E* __restrict__ G, int64_t L, int d,
                                                    int D, E* __restrict__ O) {
  const int l = threadIdx.x & 63, w = threadIdx.x >> 6, q = l >> 4, i = l & 15;
  const int nrb = (d + 16 * FR - 1) / (16 * FR);
  const int64_t job = (int64_t)blockIdx.x * 4 + w, cb = job / nrb * 64;
  const int r0 = (int)(job % nrb) * 16 * FR;
  if (cb >= L) return;
  const int64_t at = (int64_t)blockIdx.y * d * L;
  Q += (int64_t)blockIdx.y * D * D;
  G += at;
  O += at;
  f64x4 acc[FR][4];
#pragma unroll
  for (int x = 0; x < FR; ++x)
#pragma unroll
    for (int g = 0; g < 4; ++g) acc[x][g] = f64x4{0., 0., 0., 0.};
  for (int k0 = 0; k0 < d; k0 += 16) {
    double a[FR][4];  // Q's rows: wide r0 + 16 x + i, tall r0 + FR i + x; columns k0 + 4 q + j
#pragma unroll
    for (int x = 0; x < FR; ++x) {
      const double* p = Q + (int64_t)(r0 + (TALL ? FR * i + x : 16 * x + i)) * D + k0 + 4 * q;
      const f64x2 lo = *reinterpret_cast<const f64x2*>(p), hi = *reinterpret_cast<const f64x2*>(p + 2);
      a[x][0] = lo[0], a[x][1] = lo[1], a[x][2] = hi[0], a[x][3] = hi[1];
    }
    float f[4][4];
    if constexpr (!TALL) {  // f[j][g] = X[k0 + 4 q + j][cb + 4 i + g]
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + 4 * q + j;
        load_n<4, VEC, E>(G + (int64_t)k * L + cb + 4 * i, k < d ? L - cb - 4 * i : 0, f[j]);
      }
    } else {  // f[g][j] = X[cb + 16 g + i][k0 + 4 q + j], X as it lies, L x d
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int64_t c = cb + 16 * g + i;
        load_n<4, VEC, E>(G + c * d + k0 + 4 * q, c < L ? d - k0 - 4 * q : 0, f[g]);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int x = 0; x < FR; ++x)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if constexpr (!TALL) acc[x][g] = mfma(a[x][j], (double)f[j][g], acc[x][g]);
          else acc[x][g] = mfma((double)f[g][j], a[x][j], acc[x][g]);
        }
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    if constexpr (!TALL) {  // rows r0 + 16 x + drow, columns cb + 4 i + g
#pragma unroll
      for (int x = 0; x < FR; ++x) {
        const int row = r0 + 16 * x + drow(q, v);
        const double o[4] = {acc[x][0][v], acc[x][1][v], acc[x][2][v], acc[x][3][v]};
        store_n<4, VEC, E>(O + (int64_t)row * L + cb + 4 * i, row < d ? L - cb - 4 * i : 0, o);
      }
    } else {  // rows cb + 16 g + drow of the tall matrix, columns r0 + FR i + x
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int64_t c = cb + 16 * g + drow(q, v);
        double o[FR];
#pragma unroll
        for (int x = 0; x < FR; ++x) o[x] = acc[x][g][v];
        store_n<FR, VEC && FR == 2, E>(O + c * d + r0 + FR * i, c < L ? d - r0 - FR * i : 0, o);
      }
    }
  }
}

// slices of L: about 512 workgroups over the matrices and pairs, each with 8 chunks of 16 at least
int slices_of(int64_t n, int pairs, int64_t L) {
  const int64_t chunks = (L + 15) / 16;
  return (int)std::max<int64_t>(1, std::min<int64_t>(chunks / 8, 512 / std::max<int64_t>(1, n * pairs)));
}
int dim_of(int64_t d) { return (int)((d + 31) / 32 * 32); }
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
  const int t = y.D / 32;
  y.pairs = t * (t + 1) / 2;
  y.S = slices_of(n, y.pairs, y.L);
  y.part = (size_t)n * y.pairs * y.S * 1024 * sizeof(double);
  y.mat = (size_t)n * y.D * y.D * sizeof(double);
  return y;
}

}  // namespace

namespace sra {

bool orth_ok(int64_t rows, int64_t cols) { return std::min(rows, cols) <= 256; }
// slices of the Gram matrix, Q, and above d = 64 also the Gram matrix, A twice, P, P A and a second Q
size_t orth_ws(int64_t n, int64_t rows, int64_t cols) {
  if (n <= 0 || rows <= 0 || cols <= 0) return 0;
  const Layout y = layout_of(n, rows, cols);
  return y.part + y.mat * (y.D <= 64 ? 1 : 7);
}

template <typename E, bool TALL>
static hipError_t orth(const E* G, int64_t n, const Layout& y, const Steps& st, E* O, void* ws, hipStream_t s) {
  double* const part = (double*)ws;
  double* const m0 = (double*)((uint8_t*)ws + y.part);
  const size_t me = y.mat / sizeof(double);
  const GramArgs g{G, y.L, y.d, y.S, part};
  const dim3 gg((unsigned)y.pairs, (unsigned)y.S, (unsigned)n);
  if (TALL ? y.d % 2 == 0 : y.L % 4 == 0) launch(SRA_KERNEL_ORTH, k_orth_gram<E, TALL, true>, gg, dim3(256), 0, s, g);
  else launch(SRA_KERNEL_ORTH, k_orth_gram<E, TALL, false>, gg, dim3(256), 0, s, g);
  const double* Q = m0;
  if (y.D == 32) {
    hipLaunchKernelGGL(k_orth_small<32>, dim3((unsigned)n), dim3(256), 0, s, part, y.S, y.d, st, m0);
  } else if (y.D == 64) {
    hipLaunchKernelGGL(k_orth_small<64>, dim3((unsigned)n), dim3(1024), 0, s, part, y.S, y.d, st, m0);
  } else {
    double *q0 = m0, *q1 = m0 + me, *const a0 = m0 + 2 * me, *a = m0 + 3 * me, *an = m0 + 4 * me, *const p = m0 + 5 * me,
           *const w = m0 + 6 * me;
    hipLaunchKernelGGL(k_orth_join, dim3((unsigned)(y.D * y.D / 256), (unsigned)n), dim3(256), 0, s, part, y.S, y.D, a0);
    const unsigned tiles = (unsigned)((y.D / 32) * (y.D / 32));
    MmArgs m{};
    m.norm = a0, m.D = y.D, m.d = y.d, m.eps = st.eps;
    const auto run = [&](unsigned jobs) { hipLaunchKernelGGL(k_orth_mm, dim3(tiles, (unsigned)n, jobs), dim3(256), 0, s, m); };
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
    Q = q0;
  }
  const int fr = y.d <= 16 ? 1 : 2;
  const int nrb = (y.d + 16 * fr - 1) / (16 * fr);
  const int64_t jobs = (y.L + 63) / 64 * nrb;
  const dim3 ga((unsigned)((jobs + 3) / 4), (unsigned)n);
  const bool vec = TALL ? y.d % 4 == 0 : y.L % 4 == 0;
#define SRA_APPLY(V, FR) launch(SRA_KERNEL_ORTH, k_orth_apply<E, TALL, V, FR>, ga, dim3(256), 0, s, Q, G, y.L, y.d, y.D, O)
  if (fr == 1) {
    if (vec) SRA_APPLY(true, 1);
    else SRA_APPLY(false, 1);
  } else {
    if (vec) SRA_APPLY(true, 2);
    else SRA_APPLY(false, 2);
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
