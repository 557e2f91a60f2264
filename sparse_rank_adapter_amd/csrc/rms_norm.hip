// Root-mean-square norm over the rows of H = X + R (R the residual, optional), forward and backward.
//
//   forward   h = x + r,  rstd = 1 / sqrt(sum(h^2) / H + eps),  y = h rstd gamma
//   backward  g = dy gamma,  xh = h rstd,  dx = rstd (g - xh mean(g xh)) + dh,  dgamma = sum_t dy xh
//
// Bound by HBM: each tensor is read or written once.  A workgroup holds a whole row in registers (EPT
// elements a thread, as vectors of VEC), so the sum of squares, the stored H, Y and its 8-bit code come
// from one read.  The norm is that of the fp32 sum x + r; H, Y and the codes are each rounded once from fp32.
// A row's sum is fp32 within a thread (8 or 16 terms) and fp64 over the threads.
//
// The backward's workgroups walk over rows, gridDim.x apart, with their part of dgamma in registers;
// one partial row per workgroup is summed by a second launch in a fixed order: no atomics.
//
// Measured: 8192 rows of 5120 in bf16 with residual, Y and codes 64 us (378 MB, 5.9 TB/s: part of what is read is still in the
// Infinity Cache; a copy of 1 GiB reaches 5.1), the backward of 8191 rows with dH 69 + 4 us (336 MB, 4.9 TB/s); 17 rows of
// 1024 3 us and the backward of 333 fp32 rows of 1024 3.7 + 4.2 us, all latency.
#include <algorithm>
#include <cmath>

#include "fp8.h"

namespace {
using namespace sra_f8;
using sra_row::block_sum;
using sra_row::tree_sum;

// OUT: 1 = Y, 2 = codes, 3 = both
template <typename E, int VEC, int EPT, int OUT>
__global__ __launch_bounds__(1024) void k_rms_fwd(const E* x, const E* r, const E* __restrict__ gamma,
                                                                   float eps, int64_t H, E* h, E* __restrict__ y,
                                                                   float* __restrict__ rstd, uint8_t* __restrict__ codes,
                                                                   uint8_t* __restrict__ exps) {
  constexpr int V = EPT / VEC;
  __shared__ double red[16];
  const int64_t t = blockIdx.x;
  const int nt = blockDim.x;
  // all loads go out before any is used; in fp32, where they take twice the registers, gamma only ahead of the row's sum
  // (8192 x 5120 with the residual, Y and codes 118 us, 122 with gamma up here, rows of 5121 172 and 192)
  Stored<E, VEC> xs[V], res[V], gs[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int64_t c = (int64_t)(threadIdx.x + v * nt) * VEC;
    xs[v] = fetch<E, VEC>(x + t * H, c, H);
    if constexpr (sizeof(E) == 2) gs[v] = fetch<E, VEC>(gamma, c, H);
  }
  if (r) {
#pragma unroll
    for (int v = 0; v < V; ++v) res[v] = fetch<E, VEC>(r + t * H, (int64_t)(threadIdx.x + v * nt) * VEC, H);
  }
  float f[V][VEC];
#pragma unroll
  for (int v = 0; v < V; ++v) as_floats<E, VEC>(xs[v], H - (int64_t)(threadIdx.x + v * nt) * VEC, f[v]);
  if (r) {  // h may be x or r: a row's elements are read and written by the same thread
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t c = (int64_t)(threadIdx.x + v * nt) * VEC;
      float g[VEC];
      as_floats<E, VEC>(res[v], H - c, g);
#pragma unroll
      for (int k = 0; k < VEC; ++k) f[v][k] += g[k];
      store_row<E, VEC>(h + t * H + c, H - c, f[v]);
    }
  }
  float part[1] = {0.f};
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float sq[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) sq[k] = f[v][k] * f[v][k];
    part[0] += tree_sum<VEC>(sq);
  }
  if constexpr (sizeof(E) == 4) {
#pragma unroll
    for (int v = 0; v < V; ++v) gs[v] = fetch<E, VEC>(gamma, (int64_t)(threadIdx.x + v * nt) * VEC, H);
  }
  double s[1];
  block_sum<1>(part, s, red);
  const float rs = (float)(1.0 / sqrt(s[0] / (double)H + (double)eps));
  if (threadIdx.x == 0) rstd[t] = rs;
  const int64_t ld = (H + kBlock - 1) / kBlock * kBlock;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int64_t c = (int64_t)(threadIdx.x + v * nt) * VEC;
    float ga[VEC];
    as_floats<E, VEC>(gs[v], H - c, ga);
#pragma unroll
    for (int k = 0; k < VEC; ++k) f[v][k] = f[v][k] * rs * ga[k];
    if constexpr (OUT & 1) store_row<E, VEC>(y + t * H + c, H - c, f[v]);
    if constexpr (OUT & 2) {
      // past the row's end the elements are zeros (or NaN, from a rstd that is not finite)
#pragma unroll
      for (int k = 0; k < VEC; ++k) f[v][k] = c + k < H ? f[v][k] : 0.f;
      const Coded<SRA_FP8_E4M3, VEC> q = encode<SRA_FP8_E4M3, VEC>(f[v]);
      if (c < ld) {
        store_codes<SRA_FP8_E4M3, VEC>(codes + t * ld + c, q);
        if ((threadIdx.x & (kBlock / VEC - 1)) == 0) exps[t * (ld / kBlock) + c / kBlock] = (uint8_t)q.exp;
      }
    }
  }
}

// part [gridDim.x][H]: this workgroup's sum of dy xh over its rows.  DH: dh is given
template <typename E, int VEC, int EPT, bool DH>
__global__ __launch_bounds__(1024) void k_rms_bwd(const E* dy, const E* h, const E* __restrict__ gamma,
                                                                   const float* __restrict__ rstd, const E* dh, int64_t T,
                                                                   int64_t H, E* dx, float* __restrict__ part) {
  constexpr int V = EPT / VEC;
  __shared__ double red[2][16];
  const int nt = blockDim.x;
  float dg[V][VEC], ga[V][VEC];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int64_t c = (int64_t)(threadIdx.x + v * nt) * VEC;
    load_row<E, VEC>(gamma + c, H - c, ga[v]);
#pragma unroll
    for (int k = 0; k < VEC; ++k) dg[v][k] = 0.f;
  }
  const double inv_h = 1.0 / (double)H;
  // A row's three tensors are fetched while the row before is worked on.  dx may be any of them: a row is fetched by the
  // threads that write it, and always before.
  struct Row {
    Stored<E, VEC> g[V], x[V], o[V];
    float rs;
  };
  const auto load = [&](int64_t t, Row& r) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t c = (int64_t)(threadIdx.x + v * nt) * VEC;
      r.g[v] = fetch<E, VEC>(dy + t * H, c, H);
      r.x[v] = fetch<E, VEC>(h + t * H, c, H);
      if constexpr (DH) r.o[v] = fetch<E, VEC>(dh + t * H, c, H);
    }
    r.rs = rstd[t];
  };
  constexpr bool AHEAD = EPT == 8;  // with 16 elements the two rows do not fit a thread's 128 registers
  Row cur, nxt;
  int flip = 0;
  int64_t t = blockIdx.x;
  if (AHEAD && t < T) load(t, cur);
  for (; t < T; t += gridDim.x, flip ^= 1) {
    if (!AHEAD) load(t, cur);
    else if (t + gridDim.x < T) load(t + gridDim.x, nxt);
    const float rs = cur.rs;
    float g[V][VEC], xh[V][VEC];
    float s[1] = {0.f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t left = H - (int64_t)(threadIdx.x + v * nt) * VEC;
      as_floats<E, VEC>(cur.g[v], left, g[v]);
      as_floats<E, VEC>(cur.x[v], left, xh[v]);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        xh[v][k] *= rs;
        dg[v][k] = fmaf(g[v][k], xh[v][k], dg[v][k]);
        g[v][k] *= ga[v][k];
        s[0] = fmaf(g[v][k], xh[v][k], s[0]);
      }
    }
    double m[1];
    block_sum<1>(s, m, red[flip]);
    const float b = (float)(m[0] * inv_h);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t c = (int64_t)(threadIdx.x + v * nt) * VEC;
#pragma unroll
      for (int k = 0; k < VEC; ++k) g[v][k] = rs * (g[v][k] - xh[v][k] * b);
      if constexpr (DH) {
        float o[VEC];
        as_floats<E, VEC>(cur.o[v], H - c, o);
#pragma unroll
        for (int k = 0; k < VEC; ++k) g[v][k] += o[k];
      }
      store_row<E, VEC>(dx + t * H + c, H - c, g[v]);
    }
    if (AHEAD) cur = nxt;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int64_t c = (int64_t)(threadIdx.x + v * nt) * VEC;
    store_row<float, VEC>(part + (int64_t)blockIdx.x * H + c, H - c, dg[v]);
  }
}

// dgamma from P partial rows, 16 rows at a time by the 16 waves of a workgroup, joined in a fixed order
__global__ __launch_bounds__(1024) void k_rms_param(const float* __restrict__ part, int P, int64_t H,
                                                    float* __restrict__ dgamma) {
  __shared__ float red[16][64];
  const int c = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 64 + c;
  constexpr int U = 8;  // loads in flight: the launch is bound by their latency
  float s = 0.f;
  const float* src = part + min(col, H - 1);
  for (int p = w; p < P; p += 16 * U) {
    float v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = src[(int64_t)min(p + 16 * u, P - 1) * H];
#pragma unroll
    for (int u = 0; u < U; ++u) s += p + 16 * u < P ? v[u] : 0.f;
  }
  red[w][c] = s;
  __syncthreads();
  if (w == 0 && col < H) {
#pragma unroll
    for (int i = 1; i < 16; ++i) s += red[i][c];
    dgamma[col] = s;
  }
}

// Elements a thread holds, in at most 1024 threads: the forward 8 up to 2048 columns, 16 above (8192 rows of 5120 in bf16
// with H, Y and codes: 64 us, with 8 elements 74, each before loads went out ahead), the backward 8 up to 8192 columns, which leaves registers for the
// next row (8191 rows of 5120 with dH: 69 us, with 16 elements and no row ahead 85).  Rows above 8192 columns that are no
// multiple of 8 spill 27 to 54 registers there (2048 rows of 9001 with dH 96 us).
int fwd_ept(int64_t H) { return H <= 2048 ? 8 : 16; }
int bwd_ept(int64_t H) { return H <= 8192 ? 8 : 16; }
int threads_for(int64_t H, int ept) { return 64 * (int)((H + 64 * ept - 1) / (64 * ept)); }
// rows of one forward launch: a launch has fewer than 2^32 threads, and a row takes up to 1024 of them
constexpr int64_t kFwdRows = (int64_t)1 << 21;
int bwd_groups(int64_t T) { return (int)std::min<int64_t>(T, 512); }

}  // namespace

namespace sra {

bool rms_norm_ok(int64_t H) { return H <= 16384; }
size_t rms_norm_bwd_ws(int64_t T, int64_t H) { return (size_t)bwd_groups(T) * (size_t)H * sizeof(float); }

// VEC and EPT of a call, as template arguments of `body`
#define SRA_RMS_PICK(E, BODY)         \
  do {                                \
    if (vec8(H)) {                    \
      if (ept == 8) BODY(E, 8, 8);    \
      else BODY(E, 8, 16);            \
    } else {                          \
      if (ept == 8) BODY(E, 2, 8);    \
      else BODY(E, 2, 16);            \
    }                                 \
  } while (0)

hipError_t launch_rms_norm_fwd(int dtype, const void* x, const void* r, const void* gamma, float eps, int64_t T,
                               int64_t H, void* h, void* y, float* rstd, uint8_t* codes, uint8_t* exps, hipStream_t s) {
  if (T <= 0) return hipSuccess;
  if (H <= 0) return launch_fill_f32(rstd, T, NAN, s);  // the mean of no terms
  const int ept = fwd_ept(H);
  const dim3 block((unsigned)threads_for(H, ept));
  const int64_t ld = ld_of(H), esz = dtype == SRA_BF16 ? 2 : 4;
  for (int64_t t0 = 0; t0 < T; t0 += kFwdRows) {
    const dim3 grid((unsigned)std::min<int64_t>(kFwdRows, T - t0));
    const int64_t at = t0 * H * esz;
    const void *const xt = (const uint8_t*)x + at, *const rt = r ? (const uint8_t*)r + at : nullptr;
    void *const ht = h ? (uint8_t*)h + at : nullptr, *const yt = y ? (uint8_t*)y + at : nullptr;
    uint8_t* const ct = codes ? codes + t0 * ld : nullptr;
    uint8_t* const et = codes ? exps + t0 * (ld / kBlock) : nullptr;
#define SRA_RMS_ONE(E, VEC, EPT, OUT)                                                                              \
  launch(SRA_KERNEL_RMS_NORM, k_rms_fwd<E, VEC, EPT, OUT>, grid, block, 0, s, (const E*)xt, (const E*)rt,          \
         (const E*)gamma, eps, H, (E*)ht, (E*)yt, rstd + t0, ct, et)
#define SRA_RMS_FWD(E, VEC, EPT)                      \
  do {                                                \
    if (y && codes) SRA_RMS_ONE(E, VEC, EPT, 3);      \
    else if (codes) SRA_RMS_ONE(E, VEC, EPT, 2);      \
    else SRA_RMS_ONE(E, VEC, EPT, 1);                 \
  } while (0)
    if (dtype == SRA_BF16) SRA_RMS_PICK(uint16_t, SRA_RMS_FWD);
    else SRA_RMS_PICK(float, SRA_RMS_FWD);
#undef SRA_RMS_FWD
#undef SRA_RMS_ONE
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

hipError_t launch_rms_norm_bwd(int dtype, const void* dy, const void* h, const void* gamma, const float* rstd,
                               const void* dh, int64_t T, int64_t H, void* dx, float* dgamma, void* ws, hipStream_t s) {
  if (H <= 0) return hipSuccess;
  const int P = bwd_groups(T), ept = bwd_ept(H);  // no partials when T = 0: the second launch writes zeros
  if (T > 0) {
    const dim3 grid((unsigned)P), block((unsigned)threads_for(H, ept));
#define SRA_RMS_ONE(E, VEC, EPT, DH)                                                                                     \
  launch(SRA_KERNEL_RMS_NORM, k_rms_bwd<E, VEC, EPT, DH>, grid, block, 0, s, (const E*)dy, (const E*)h, (const E*)gamma, \
         rstd, (const E*)dh, T, H, (E*)dx, (float*)ws)
#define SRA_RMS_BWD(E, VEC, EPT)                 \
  do {                                           \
    if (dh) SRA_RMS_ONE(E, VEC, EPT, true);      \
    else SRA_RMS_ONE(E, VEC, EPT, false);        \
  } while (0)
    if (dtype == SRA_BF16) SRA_RMS_PICK(uint16_t, SRA_RMS_BWD);
    else SRA_RMS_PICK(float, SRA_RMS_BWD);
#undef SRA_RMS_BWD
#undef SRA_RMS_ONE
  }
  hipLaunchKernelGGL(k_rms_param, dim3((unsigned)((H + 63) / 64)), dim3(1024), 0, s, (const float*)ws, P, H, dgamma);
  return hipGetLastError();
}

}  // namespace sra
