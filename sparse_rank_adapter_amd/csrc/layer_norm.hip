// Layer norm over the rows of X [T][H], forward and backward.
//
//   forward   mean = sum(x) / H,  rstd = 1 / sqrt(sum((x - mean)^2) / H + eps)
//             y = (x - mean) rstd gamma + beta
//   backward  g = dy gamma,  xh = (x - mean) rstd
//             dx = rstd (g - mean(g) - xh mean(g xh)),  dgamma = sum_t dy xh,  dbeta = sum_t dy
//
// Both are bound by HBM: the forward reads and writes each element once, the backward reads two
// tensors and writes one.  A workgroup holds a whole row in registers (EPT elements a thread, as
// vectors of VEC), so the variance is summed from the deviations with no second read.
// All sums are fp32.
//
// The backward's workgroups walk over rows (gridDim.x apart): a thread keeps its columns, so its
// parts of dgamma and dbeta stay in registers until the end, are written as one partial row per
// workgroup, and are summed over the workgroups in a fixed order by a second launch: no atomics,
// the same result on every run.
#include <algorithm>

#include "rowvec.h"

namespace {
using namespace sra_row;

template <int N>
SRA_DEV void wave_sum(float (&v)[N]) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor(v[k], d, 64);
}
// Sum over the workgroup (up to 16 waves), the same value in every thread.  `red` is LDS that no
// wave still reads: calls alternate between two areas, so one barrier each is enough.
template <int N>
SRA_DEV void block_sum(float (&v)[N], float* red) {
  wave_sum<N>(v);
  const int nw = blockDim.x >> 6;
  if (nw == 1) return;
  const int w = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) red[w * N + k] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = 0.f;
  for (int i = 0; i < nw; ++i)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += red[i * N + k];
}

// one workgroup per row
template <typename E, int VEC, int EPT, bool CK>
__global__ __launch_bounds__(EPT == 8 ? 256 : 1024) void k_ln_fwd(const E* __restrict__ x, const E* __restrict__ gamma,
                                                 const E* __restrict__ beta, float eps, int64_t H, E* __restrict__ y,
                                                 float* __restrict__ mean, float* __restrict__ rstd,
                                                 int8_t* __restrict__ codes, uint8_t* __restrict__ exps) {
  constexpr int V = EPT / VEC;
  __shared__ float red[2][16];
  const int64_t t = blockIdx.x;
  const int nvec = (int)(H / VEC), nt = blockDim.x;
  float f[V][VEC];
  float s[1] = {0.f};
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = threadIdx.x + v * nt;
#pragma unroll
    for (int k = 0; k < VEC; ++k) f[v][k] = 0.f;
    if (i < nvec) RowVec<E, VEC>::load(x + t * H + (int64_t)i * VEC, f[v]);
#pragma unroll
    for (int k = 0; k < VEC; ++k) s[0] += f[v][k];
  }
  block_sum<1>(s, red[0]);
  const float mu = s[0] / (float)H;
  float q[1] = {0.f};
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const bool in = threadIdx.x + v * nt < nvec;
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      f[v][k] = in ? f[v][k] - mu : 0.f;
      q[0] += f[v][k] * f[v][k];
    }
  }
  block_sum<1>(q, red[1]);
  const float rs = 1.f / sqrtf(q[0] / (float)H + eps);
  if (threadIdx.x == 0) {
    mean[t] = mu;
    rstd[t] = rs;
  }
  const int64_t nblk = (H + kCkBlock - 1) / kCkBlock;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = threadIdx.x + v * nt;
    float o[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) o[k] = 0.f;
    if (i < nvec) {
      float ga[VEC], be[VEC];
      RowVec<E, VEC>::load(gamma + (int64_t)i * VEC, ga);
      RowVec<E, VEC>::load(beta + (int64_t)i * VEC, be);
#pragma unroll
      for (int k = 0; k < VEC; ++k) o[k] = fmaf(f[v][k] * rs, ga[k], be[k]);
      RowVec<E, VEC>::store(y + t * H + (int64_t)i * VEC, o);  // o becomes what is stored
    }
    if constexpr (CK) {  // the checkpoint codes the stored (rounded) output
      const Coded<VEC> c = ck_encode<VEC>(o);
      if (i < nvec) {
        ck_store_codes<VEC>(codes + t * H + (int64_t)i * VEC, c.codes);
        if ((threadIdx.x & (kCkBlock / VEC - 1)) == 0) exps[t * nblk + (int64_t)i * VEC / kCkBlock] = (uint8_t)c.exp;
      }
    }
  }
}

// part [gridDim.x][2][H]: this workgroup's sums of dy xh and dy over its rows
template <typename E, int VEC, int EPT>
__global__ __launch_bounds__(EPT == 8 ? 256 : 1024) void k_ln_bwd(const E* __restrict__ dy, const E* __restrict__ x,
                                                 const E* __restrict__ gamma, const float* __restrict__ mean,
                                                 const float* __restrict__ rstd, int64_t T, int64_t H,
                                                 E* __restrict__ dx, float* __restrict__ part) {
  constexpr int V = EPT / VEC;
  __shared__ float red[2][2 * 16];
  const int nvec = (int)(H / VEC), nt = blockDim.x;
  float dg[V][VEC], db[V][VEC];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int k = 0; k < VEC; ++k) dg[v][k] = db[v][k] = 0.f;
  int flip = 0;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x, flip ^= 1) {
    const float mu = mean[t], rs = rstd[t];
    float g[V][VEC], xh[V][VEC];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = threadIdx.x + v * nt;
      if (i < nvec) {
        float ga[VEC];
        RowVec<E, VEC>::load(dy + t * H + (int64_t)i * VEC, g[v]);
        RowVec<E, VEC>::load(x + t * H + (int64_t)i * VEC, xh[v]);
        RowVec<E, VEC>::load(gamma + (int64_t)i * VEC, ga);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          xh[v][k] = (xh[v][k] - mu) * rs;
          dg[v][k] = fmaf(g[v][k], xh[v][k], dg[v][k]);
          db[v][k] += g[v][k];
          g[v][k] *= ga[k];
          s[0] += g[v][k];
          s[1] = fmaf(g[v][k], xh[v][k], s[1]);
        }
      }
    }
    block_sum<2>(s, red[flip]);
    const float a = s[0] / (float)H, b = s[1] / (float)H;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = threadIdx.x + v * nt;
      if (i < nvec) {
        float o[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) o[k] = rs * (g[v][k] - a - xh[v][k] * b);
        RowVec<E, VEC>::store(dx + t * H + (int64_t)i * VEC, o);
      }
    }
  }
  float* pg = part + (int64_t)blockIdx.x * 2 * H;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = threadIdx.x + v * nt;
    if (i < nvec) {
      RowVec<float, VEC>::store(pg + (int64_t)i * VEC, dg[v]);
      RowVec<float, VEC>::store(pg + H + (int64_t)i * VEC, db[v]);
    }
  }
}

// dgamma (columns 0 .. H-1 of a partial row) and dbeta (H .. 2H-1): P partials per column, 16 rows
// at a time by the 16 groups of a workgroup, joined through LDS in a fixed order
__global__ __launch_bounds__(1024) void k_ln_params(const float* __restrict__ part, int P, int64_t H,
                                                    float* __restrict__ dgamma, float* __restrict__ dbeta) {
  __shared__ float red[16][64];
  const int c = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 64 + c;
  float s = 0.f;
  if (col < 2 * H)
    for (int p = w; p < P; p += 16) s += part[(int64_t)p * 2 * H + col];
  red[w][c] = s;
  __syncthreads();
  if (w == 0 && col < 2 * H) {
    for (int i = 1; i < 16; ++i) s += red[i][c];
    if (col < H) dgamma[col] = s;
    else dbeta[col - H] = s;
  }
}

// Elements a thread holds: 8 up to 2048 columns (at most 256 threads), 16 above (at most 1024, so
// rows of up to 16384), in as many whole waves as the row then needs.
int ept_for(int64_t H) { return H <= 2048 ? 8 : 16; }
int threads_for(int64_t H, int ept) { return 64 * (int)((H + 64 * ept - 1) / (64 * ept)); }
int bwd_groups(int64_t T) { return (int)std::min<int64_t>(T, 512); }

}  // namespace

namespace sra {

bool layer_norm_ok(int64_t H) { return H <= 16384; }
size_t layer_norm_bwd_ws(int64_t T, int64_t H) { return (size_t)bwd_groups(T) * 2 * (size_t)H * sizeof(float); }

// VEC and EPT of a call, as template arguments of `body`
#define SRA_LN_PICK(E, BODY)                                          \
  do {                                                                \
    const int vec_ = row_vec(H), ept_ = ept_for(H);                   \
    if (vec_ == 8) {                                                  \
      if (ept_ == 8) BODY(E, 8, 8);                                   \
      else BODY(E, 8, 16);                                            \
    } else if (vec_ == 2) {                                           \
      if (ept_ == 8) BODY(E, 2, 8);                                   \
      else BODY(E, 2, 16);                                            \
    } else {                                                          \
      if (ept_ == 8) BODY(E, 1, 8);                                   \
      else BODY(E, 1, 16);                                            \
    }                                                                 \
  } while (0)

hipError_t launch_layer_norm_fwd(int dtype, const void* x, const void* gamma, const void* beta, float eps, int64_t T,
                                 int64_t H, void* y, float* mean, float* rstd, int8_t* codes, uint8_t* exps,
                                 hipStream_t s) {
  if (T <= 0 || H <= 0) return hipSuccess;
  const dim3 grid((unsigned)T), block((unsigned)threads_for(H, ept_for(H)));
#define SRA_LN_FWD(E, VEC, EPT)                                                                                   \
  do {                                                                                                            \
    if (codes)                                                                                                    \
      launch(SRA_KERNEL_LAYER_NORM, k_ln_fwd<E, VEC, EPT, true>, grid, block, 0, s, (const E*)x, (const E*)gamma, \
             (const E*)beta, eps, H, (E*)y, mean, rstd, codes, exps);                                             \
    else                                                                                                          \
      launch(SRA_KERNEL_LAYER_NORM, k_ln_fwd<E, VEC, EPT, false>, grid, block, 0, s, (const E*)x, (const E*)gamma, \
             (const E*)beta, eps, H, (E*)y, mean, rstd, codes, exps);                                             \
  } while (0)
  if (dtype == SRA_BF16) SRA_LN_PICK(uint16_t, SRA_LN_FWD);
  else SRA_LN_PICK(float, SRA_LN_FWD);
#undef SRA_LN_FWD
  return hipGetLastError();
}

hipError_t launch_layer_norm_bwd(int dtype, const void* dy, const void* x, const void* gamma, const float* mean,
                                 const float* rstd, int64_t T, int64_t H, void* dx, float* dgamma, float* dbeta,
                                 void* ws, hipStream_t s) {
  if (H <= 0) return hipSuccess;
  const int P = bwd_groups(T);  // 0 partials when T = 0: the second launch writes zeros
  if (T > 0) {
    const dim3 grid((unsigned)P), block((unsigned)threads_for(H, ept_for(H)));
#define SRA_LN_BWD(E, VEC, EPT)                                                                               \
  launch(SRA_KERNEL_LAYER_NORM, k_ln_bwd<E, VEC, EPT>, grid, block, 0, s, (const E*)dy, (const E*)x, (const E*)gamma, \
         mean, rstd, T, H, (E*)dx, (float*)ws)
    if (dtype == SRA_BF16) SRA_LN_PICK(uint16_t, SRA_LN_BWD);
    else SRA_LN_PICK(float, SRA_LN_BWD);
#undef SRA_LN_BWD
  }
  hipLaunchKernelGGL(k_ln_params, dim3((unsigned)((2 * H + 63) / 64)), dim3(1024), 0, s, (const float*)ws, P, H, dgamma,
                     dbeta);
  return hipGetLastError();
}

}  // namespace sra
