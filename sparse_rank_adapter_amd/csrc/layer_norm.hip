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
// Terms are summed in fp32 within a thread (8 or 16 of them) and in fp64 over the threads.
//
// The backward's workgroups walk over rows (gridDim.x apart): a thread keeps its columns, so its
// parts of dgamma and dbeta stay in registers until the end, are written as one partial row per
// workgroup, and are summed over the workgroups in a fixed order by a second launch: no atomics,
// the same result on every run.
//
// Measured: 8192 rows of 5120 in bf16 with the checkpoint 49 us (211 MB: 4.3 TB/s, where a copy of 2 GiB
// reaches 4.9), the backward 51 + 5 us (252 MB: 4.9 TB/s in its first launch); 17 rows of 1024 3.2 us and
// the backward of 333 fp32 rows of 1024 4.6 + 4.2 us, all latency.
#include <algorithm>
#include <cmath>

#include "rowvec.h"

namespace {
using namespace sra_row;

// Sum over the wave in fp64 by DPP row shifts and broadcasts (lane 63 ends with it), the same value in
// every lane, with no LDS round trips (lane exchanges through LDS: 52 us against 48-50 at 8192 x 5120);
// fp32 sums here moved the statistics by enough to flip over half as many codes of a checkpoint again.
template <int CTRL, int ROWS>
SRA_DEV double dpp_add(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xf, false);
  return x + __longlong_as_double((int64_t)(((uint64_t)hi << 32) | lo));
}
SRA_DEV double wave_sum(double x) {
  x = dpp_add<0x111, 0xf>(x);  // row_shr 1, 2, 4, 8: lane 15 of each row of 16 holds the row's sum
  x = dpp_add<0x112, 0xf>(x);
  x = dpp_add<0x114, 0xf>(x);
  x = dpp_add<0x118, 0xf>(x);
  x = dpp_add<0x142, 0xa>(x);  // row_bcast 15 into rows 1 and 3
  x = dpp_add<0x143, 0xc>(x);  // row_bcast 31 into rows 2 and 3
  const uint64_t u = (uint64_t)__double_as_longlong(x);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, 63), hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63);
  return __longlong_as_double((int64_t)(((uint64_t)hi << 32) | lo));
}
// Sums over the workgroup (up to 16 waves, added in fp64), the same values in every thread.  `red` is
// LDS that no wave still reads: calls alternate between two areas, so one barrier each is enough.
template <int N>
SRA_DEV void block_sum(const float (&v)[N], double (&out)[N], double* red) {
  double s[N];
#pragma unroll
  for (int k = 0; k < N; ++k) s[k] = wave_sum((double)v[k]);
  const int nw = blockDim.x >> 6;
  if (nw == 1) {
#pragma unroll
    for (int k = 0; k < N; ++k) out[k] = s[k];
    return;
  }
  const int w = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) red[w * N + k] = s[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) out[k] = 0.0;
  for (int i = 0; i < nw; ++i)
#pragma unroll
    for (int k = 0; k < N; ++k) out[k] += red[i * N + k];
}

// sum of N terms as a tree
template <int N>
SRA_DEV float tree_sum(const float* v) {
  if constexpr (N == 1) return v[0];
  else return tree_sum<N / 2>(v) + tree_sum<N - N / 2>(v + N / 2);
}

// one workgroup per row
template <typename E, int VEC, int EPT, bool CK>
__global__ __launch_bounds__(EPT == 8 ? 256 : 1024) void k_ln_fwd(const E* __restrict__ x, const E* __restrict__ gamma,
                                                 const E* __restrict__ beta, float eps, int64_t H, E* __restrict__ y,
                                                 float* __restrict__ mean, float* __restrict__ rstd,
                                                 int8_t* __restrict__ codes, uint8_t* __restrict__ exps) {
  constexpr int V = EPT / VEC;
  __shared__ double red[2][16];
  const int64_t t = blockIdx.x;
  const int nvec = (int)(H / VEC), nt = blockDim.x;
  float f[V][VEC];
  float part[1] = {0.f};
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = threadIdx.x + v * nt;
#pragma unroll
    for (int k = 0; k < VEC; ++k) f[v][k] = 0.f;
    if (i < nvec) RowVec<E, VEC>::load(x + t * H + (int64_t)i * VEC, f[v]);
    part[0] += tree_sum<VEC>(f[v]);
  }
  double s[1];
  block_sum<1>(part, s, red[0]);
  const double inv_h = 1.0 / (double)H;
  const float mu = (float)(s[0] * inv_h);
  part[0] = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const bool in = threadIdx.x + v * nt < nvec;
    float sq[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      f[v][k] = in ? f[v][k] - mu : 0.f;
      sq[k] = f[v][k] * f[v][k];
    }
    part[0] += tree_sum<VEC>(sq);
  }
  double q[1];
  block_sum<1>(part, q, red[1]);
  const float rs = 1.f / sqrtf((float)(q[0] * inv_h) + eps);
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
  __shared__ double red[2][2 * 16];
  const int nvec = (int)(H / VEC), nt = blockDim.x;
  float dg[V][VEC], db[V][VEC];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int k = 0; k < VEC; ++k) dg[v][k] = db[v][k] = 0.f;
  const double inv_h = 1.0 / (double)H;
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
    double m[2];
    block_sum<2>(s, m, red[flip]);
    const float a = (float)(m[0] * inv_h), b = (float)(m[1] * inv_h);
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
  constexpr int U = 8;  // loads in flight: the partials are few and the launch is bound by their latency
  float s = 0.f;
  const float* src = part + min(col, 2 * H - 1);
  for (int p = w; p < P; p += 16 * U) {
    float v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = src[(int64_t)min(p + 16 * u, P - 1) * 2 * H];
#pragma unroll
    for (int u = 0; u < U; ++u) s += p + 16 * u < P ? v[u] : 0.f;
  }
  red[w][c] = s;
  __syncthreads();
  if (w == 0 && col < 2 * H) {
#pragma unroll
    for (int i = 1; i < 16; ++i) s += red[i][c];
    if (col < H) dgamma[col] = s;
    else dbeta[col - H] = s;
  }
}

// Elements a thread holds: 8 up to 2048 columns (at most 256 threads), 16 above (at most 1024, so
// rows of up to 16384), in as many whole waves as the row then needs.
int ept_for(int64_t H) { return H <= 2048 ? 8 : 16; }
int threads_for(int64_t H, int ept) { return 64 * (int)((H + 64 * ept - 1) / (64 * ept)); }
// Rows of one forward launch: a launch has fewer than 2^32 threads, and a row takes up to 1024 of them
constexpr int64_t kFwdRows = (int64_t)1 << 21;
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
  if (T <= 0) return hipSuccess;
  if (H <= 0) {  // a sum of no terms over no terms
    hipError_t err = mean ? launch_fill_f32(mean, T, NAN, s) : hipSuccess;
    return err == hipSuccess && rstd ? launch_fill_f32(rstd, T, NAN, s) : err;
  }
  const dim3 block((unsigned)threads_for(H, ept_for(H)));
  const int64_t blocks_per_row = (H + kCkBlock - 1) / kCkBlock, esz = dtype == SRA_BF16 ? 2 : 4;
  for (int64_t t0 = 0; t0 < T; t0 += kFwdRows) {
    const dim3 grid((unsigned)std::min<int64_t>(kFwdRows, T - t0));
    const void* const xt = (const uint8_t*)x + t0 * H * esz;
    void* const yt = (uint8_t*)y + t0 * H * esz;
    int8_t* const ct = codes ? codes + t0 * H : nullptr;
    uint8_t* const et = codes ? exps + t0 * blocks_per_row : nullptr;
#define SRA_LN_FWD(E, VEC, EPT)                                                                                    \
  do {                                                                                                             \
    if (codes)                                                                                                     \
      launch(SRA_KERNEL_LAYER_NORM, k_ln_fwd<E, VEC, EPT, true>, grid, block, 0, s, (const E*)xt, (const E*)gamma, \
             (const E*)beta, eps, H, (E*)yt, mean + t0, rstd + t0, ct, et);                                        \
    else                                                                                                           \
      launch(SRA_KERNEL_LAYER_NORM, k_ln_fwd<E, VEC, EPT, false>, grid, block, 0, s, (const E*)xt, (const E*)gamma, \
             (const E*)beta, eps, H, (E*)yt, mean + t0, rstd + t0, ct, et);                                        \
  } while (0)
    if (dtype == SRA_BF16) SRA_LN_PICK(uint16_t, SRA_LN_FWD);
    else SRA_LN_PICK(float, SRA_LN_FWD);
#undef SRA_LN_FWD
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
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
