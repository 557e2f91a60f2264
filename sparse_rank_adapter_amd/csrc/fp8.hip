// Matrices in 8-bit floating point with power-of-two scales (fp8.h has the code): encoding by rows, by
// 128 x 128 blocks and with the transpose, and decoding.  All are bound by HBM.
//
// Codes lie in rows of whole 128-byte blocks, filled up with zeros, so a product never masks its
// reduction.  Blocks of one row: 16 lanes hold a block (8 columns each) and find its maximum by DPP
// rotations.  With the transpose, or with blocks of 128 rows, a workgroup holds a 128 x 128 tile in
// registers (8 x 8 elements a thread), so the matrix is read once for both forms; the transposed codes
// cross through LDS and leave in whole 128-byte lines.
//
// Measured: 20480 x 5120 in bf16 by 128 x 128 blocks with the transpose 75-88 us (419 MB, 4.8-5.6 TB/s), decoded again 49 and
// 54 us (5.5-6.4 TB/s); 2047 x 4096 by rows with the transpose 13-16 us (34 MB: 512 workgroups of one tile each, so nothing
// overlaps a tile's loads, maxima and stores), decoded 6.5 us, and 9.4 us where rows of 2047 allow two elements at a time.
// By rows alone 8192 x 5120 takes 22-23 us in bf16 and 31 in fp32 (126 and 210 MB), 8192 x 5121 in bf16 42-44.
#include <algorithm>

#include "fp8.h"

namespace {
using namespace sra_f8;

constexpr int kThreads = 256, kU = 4;
// A launch has fewer than 2^32 threads: column tiles go out in spans of 2^23, the kernels' `first` the span's first tile.
constexpr int64_t kSpan = (int64_t)1 << 23;

// blocks of one row; grid: (vector tiles of a filled-up row, rows in steps of gridDim.y)
template <typename E, int KIND, int VEC>
__global__ __launch_bounds__(kThreads) void k_fp8_rows(const E* __restrict__ x, int64_t R, int64_t C, int64_t ld, int64_t first,
                                                       uint8_t* __restrict__ codes, uint8_t* __restrict__ exps) {
  const int64_t nvec = ld / VEC, nblk = ld / kBlock;
  const int64_t i0 = (first + blockIdx.x) * (kThreads * kU) + threadIdx.x;
  // slots of this wave that begin inside the row: a wave at a ragged row's end does no work for the others (262144 x 40 in bf16
  // 74 us, 362 with it)
  const int64_t w0 = i0 - threadIdx.x + 64 * __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int live = (int)min(max((nvec - w0 + kThreads - 1) / kThreads, (int64_t)0), (int64_t)kU);
  for (int64_t t = blockIdx.y; t < R; t += gridDim.y) {
    const auto get = [&](int u) { return fetch<E, VEC>(x + t * C, (i0 + u * kThreads) * VEC, C); };
    const auto put = [&](int u, const Stored<E, VEC>& in) {
      const int64_t i = i0 + u * kThreads;
      float f[VEC];
      as_floats<E, VEC>(in, C - i * VEC, f);
      const Coded<KIND, VEC> c = encode<KIND, VEC>(f);
      if (i < nvec) {
        store_codes<KIND, VEC>(codes + t * ld + i * VEC, c);
        if ((threadIdx.x & (kBlock / VEC - 1)) == 0) exps[t * nblk + i * VEC / kBlock] = (uint8_t)c.exp;
      }
    };
    if (live == kU) {
      Stored<E, VEC> in[kU];  // all loads go out before any is used
#pragma unroll
      for (int u = 0; u < kU; ++u) in[u] = get(u);
#pragma unroll
      for (int u = 0; u < kU; ++u) put(u, in[u]);
    } else {
#pragma unroll 1
      for (int u = 0; u < live; ++u) put(u, get(u));
    }
  }
}

// One 128 x 128 tile: thread (a, b) = (tid / 16, tid % 16) holds rows 8 a .. +7, columns 8 b .. +7.
// BLK: one scale for the tile (else one per row, and one per column for the transpose).
// codes / exps and codes_t / exps_t: either pair may be absent.
template <typename E, int KIND, bool BLK, bool VEC>
__global__ __launch_bounds__(kThreads) void k_fp8_tile(const E* __restrict__ x, int64_t R, int64_t C, int64_t first,
                                                       uint8_t* __restrict__ codes, uint8_t* __restrict__ exps,
                                                       uint8_t* __restrict__ codes_t, uint8_t* __restrict__ exps_t) {
  __shared__ uint32_t red[4][kBlock];
  __shared__ __align__(16) uint8_t turn[kBlock * kBlock];  // the transposed codes: column c's 16-byte chunk q at (q ^ (c / 8 % 8))
  const int a = threadIdx.x >> 4, b = threadIdx.x & 15, w = threadIdx.x >> 6;
  const int64_t tile_c = first + blockIdx.x, c0 = tile_c * kBlock + 8 * b;
  const int64_t nbc = (C + kBlock - 1) / kBlock, nbr = (R + kBlock - 1) / kBlock;
  for (int64_t tile_r = blockIdx.y; tile_r < nbr; tile_r += gridDim.y) {
    const int64_t r0 = tile_r * kBlock + 8 * a;
    // Every row's load goes out before any is used (in branches of their own each waited for the one before).  In tiles at an edge
    // what is outside is read from inside, and replaced by zeros; doing so in every tile cost an eighth (8192 x 5120 with the
    // transpose 41 us in fp32 and 32 in bf16, 46 and 39 with it).
    float f[8][8];
    const bool inside = VEC && (tile_r + 1) * kBlock <= R && (tile_c + 1) * kBlock <= C;
    if (inside) {
      Stored<E, 8> in[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) in[i] = fetch<E, 8>(x + (r0 + i) * C, c0, INT64_MAX);
#pragma unroll
      for (int i = 0; i < 8; ++i) as_floats<E, 8>(in[i], 8, f[i]);
    } else {
      Stored<E, 8> in[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const E* const row = x + min(r0 + i, R - 1) * C;
        if constexpr (VEC) {
          in[i] = fetch<E, 8>(row, c0, C);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) in[i].e[k] = row[c0 + k < C ? c0 + k : 0];
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t left = r0 + i < R ? C - c0 : 0;
        as_floats<E, 8>(in[i], left, f[i]);
        if constexpr (!VEC) {
#pragma unroll
          for (int k = 1; k < 8; ++k) f[i][k] = k < left ? f[i][k] : 0.f;
        }
      }
    }
    uint32_t rm[8], cm[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) rm[i] = cm[i] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t m = mag(f[i][k]);
        rm[i] = max(rm[i], m);
        cm[k] = max(cm[k], m);
      }
    if constexpr (BLK) {
#pragma unroll
      for (int k = 1; k < 8; ++k) cm[0] = max(cm[0], cm[k]);
      uint32_t m = max16(cm[0]);
      m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
      m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
      if ((threadIdx.x & 63) == 0) red[w][0] = m;
      __syncthreads();
      m = max(max(red[0][0], red[1][0]), max(red[2][0], red[3][0]));
#pragma unroll
      for (int k = 0; k < 8; ++k) rm[k] = cm[k] = m;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) rm[i] = max16(rm[i]);
      if (codes_t) {  // over the 16 row groups: four in this wave (lanes 16 apart), four waves
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          cm[k] = max(cm[k], (uint32_t)__shfl_xor((int)cm[k], 16, 64));
          cm[k] = max(cm[k], (uint32_t)__shfl_xor((int)cm[k], 32, 64));
          if ((threadIdx.x & 63) < 16) red[w][8 * b + k] = cm[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 8; ++k)
          cm[k] = max(max(red[0][8 * b + k], red[1][8 * b + k]), max(red[2][8 * b + k], red[3][8 * b + k]));
      }
    }
    if (codes) {
      const int64_t ld = nbc * kBlock;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = exp_of<KIND>(rm[i]);
        const float inv = pow2(-e);
        if (r0 + i < R) {
          u32x2 o;
          o[0] = code4<KIND>(f[i][0], f[i][1], f[i][2], f[i][3], inv);
          o[1] = code4<KIND>(f[i][4], f[i][5], f[i][6], f[i][7], inv);
          *reinterpret_cast<u32x2*>(codes + (r0 + i) * ld + c0) = o;
          if (!BLK && b == 0) exps[(r0 + i) * nbc + tile_c] = (uint8_t)(e + 127);
        }
        if (BLK && i == 0 && threadIdx.x == 0) exps[tile_r * nbc + tile_c] = (uint8_t)(e + 127);
      }
    }
    if (codes_t) {
      const int64_t ld = nbr * kBlock;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int e = exp_of<KIND>(cm[k]);
        const float inv = pow2(-e);
        u32x2 o;
        o[0] = code4<KIND>(f[0][k], f[1][k], f[2][k], f[3][k], inv);
        o[1] = code4<KIND>(f[4][k], f[5][k], f[6][k], f[7][k], inv);
        const int c = 8 * b + k;
        *reinterpret_cast<u32x2*>(turn + c * kBlock + (((a >> 1) ^ (b & 7)) << 4) + 8 * (a & 1)) = o;
        if (!BLK && a == 0 && c0 + k < C) exps_t[(c0 + k) * nbr + tile_r] = (uint8_t)(e + 127);
        if (BLK && k == 0 && threadIdx.x == 0) exps_t[tile_c * nbr + tile_r] = (uint8_t)(e + 127);
      }
      __syncthreads();
      for (int v = threadIdx.x; v < kBlock * 8; v += kThreads) {  // 8 lanes write a column's 128 bytes
        const int c = v >> 3, q = v & 7;
        if (tile_c * kBlock + c < C)
          *reinterpret_cast<u32x4*>(codes_t + (tile_c * kBlock + c) * ld + tile_r * kBlock + 16 * q) =
              *reinterpret_cast<const u32x4*>(turn + c * kBlock + ((q ^ ((c >> 3) & 7)) << 4));
      }
    }
    __syncthreads();  // the next tile writes `red` and `turn` again
  }
}

// blk = 7 for blocks of 128 rows, else 0
template <typename E, int KIND, int VEC>
__global__ __launch_bounds__(kThreads) void k_fp8_decode(const uint8_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ exps, int64_t R, int64_t C,
                                                         int64_t ld, int blk, int64_t first, E* __restrict__ x) {
  const int64_t nvec = (C + VEC - 1) / VEC, nblk = ld / kBlock;
  const int64_t i0 = (first + blockIdx.x) * (kThreads * kU) + threadIdx.x;
  for (int64_t t = blockIdx.y; t < R; t += gridDim.y) {
    uint32_t c[kU][2], e[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t i = i0 + u * kThreads;
      c[u][0] = c[u][1] = 0;
      e[u] = 127;
      if (i < nvec) {
        const uint8_t* p = codes + t * ld + i * VEC;
        if constexpr (VEC == 8) {
          const u32x2 v = *reinterpret_cast<const u32x2*>(p);
          c[u][0] = v[0], c[u][1] = v[1];
        } else {
          c[u][0] = *reinterpret_cast<const uint16_t*>(p);
        }
        e[u] = exps[(t >> blk) * nblk + i * VEC / kBlock];
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t i = i0 + u * kThreads;
      float lo[4], f[VEC];
      const float s = scale_of(e[u]);
      Kind<KIND>::unpack4(c[u][0], lo);
#pragma unroll
      for (int k = 0; k < (VEC == 8 ? 4 : VEC); ++k) f[k] = lo[k] * s;
      if constexpr (VEC == 8) {
        Kind<KIND>::unpack4(c[u][1], lo);
#pragma unroll
        for (int k = 0; k < 4; ++k) f[4 + k] = lo[k] * s;
      }
      if (i < nvec) store_row<E, VEC>(x + t * C + i * VEC, C - i * VEC, f);
    }
  }
}

// launch_one(first, grid) for each span of `tiles` column tiles, over R rows or row tiles
template <typename F>
void in_spans(int64_t tiles, int64_t R, const F& launch_one) {
  for (int64_t first = 0; first < tiles; first += kSpan)
    launch_one(first, dim3((unsigned)std::min(kSpan, tiles - first), (unsigned)std::min<int64_t>(R, 32768)));
}
int64_t vec_tiles(int64_t nvec) { return (nvec + kThreads * kU - 1) / (kThreads * kU); }

template <typename E, int KIND>
void encode_rows(const void* x, int64_t R, int64_t C, uint8_t* codes, uint8_t* exps, hipStream_t s) {
  if (C % kBlock == 0) C *= R, R = 1;  // rows of whole blocks follow each other without a gap: one long row
  const int64_t ld = ld_of(C);
  in_spans(vec_tiles(ld / (vec8(C) ? 8 : 2)), R, [&](int64_t first, dim3 grid) {
    if (vec8(C))
      sra::launch(SRA_KERNEL_FP8_CODE, k_fp8_rows<E, KIND, 8>, grid, dim3(kThreads), 0, s, (const E*)x, R, C, ld, first, codes, exps);
    else
      sra::launch(SRA_KERNEL_FP8_CODE, k_fp8_rows<E, KIND, 2>, grid, dim3(kThreads), 0, s, (const E*)x, R, C, ld, first, codes, exps);
  });
}
template <typename E, int KIND, bool BLK>
void encode_tiles(const void* x, int64_t R, int64_t C, uint8_t* codes, uint8_t* exps, uint8_t* codes_t,
                  uint8_t* exps_t, hipStream_t s) {
  in_spans(blocks_of(C), blocks_of(R), [&](int64_t first, dim3 grid) {
    if (vec8(C))
      sra::launch(SRA_KERNEL_FP8_CODE, k_fp8_tile<E, KIND, BLK, true>, grid, dim3(kThreads), 0, s, (const E*)x, R, C, first,
                  codes, exps, codes_t, exps_t);
    else
      sra::launch(SRA_KERNEL_FP8_CODE, k_fp8_tile<E, KIND, BLK, false>, grid, dim3(kThreads), 0, s, (const E*)x, R, C, first,
                  codes, exps, codes_t, exps_t);
  });
}
template <typename E, int KIND>
void decode(const uint8_t* codes, const uint8_t* exps, int64_t R, int64_t C, int block_rows, void* x, hipStream_t s) {
  const int64_t ld = ld_of(C);
  const int blk = block_rows == 1 ? 0 : 7;
  in_spans(vec_tiles(vec8(C) ? C / 8 : (C + 1) / 2), R, [&](int64_t first, dim3 grid) {
    if (vec8(C))
      sra::launch(SRA_KERNEL_FP8_CODE, k_fp8_decode<E, KIND, 8>, grid, dim3(kThreads), 0, s, codes, exps, R, C, ld, blk, first, (E*)x);
    else
      sra::launch(SRA_KERNEL_FP8_CODE, k_fp8_decode<E, KIND, 2>, grid, dim3(kThreads), 0, s, codes, exps, R, C, ld, blk, first, (E*)x);
  });
}

}  // namespace

namespace sra {

hipError_t launch_fp8_encode(int dtype, int kind, const void* x, int64_t R, int64_t C, int block_rows, uint8_t* codes,
                             uint8_t* exps, uint8_t* codes_t, uint8_t* exps_t, hipStream_t s) {
  if (R <= 0 || C <= 0) return hipSuccess;
#define SRA_FP8_ENC(E, K)                                                                          \
  do {                                                                                             \
    if (block_rows == 1 && !codes_t) encode_rows<E, K>(x, R, C, codes, exps, s);                   \
    else if (block_rows == 1) encode_tiles<E, K, false>(x, R, C, codes, exps, codes_t, exps_t, s); \
    else encode_tiles<E, K, true>(x, R, C, codes, exps, codes_t, exps_t, s);                       \
  } while (0)
  if (dtype == SRA_BF16) {
    if (kind == SRA_FP8_E4M3) SRA_FP8_ENC(uint16_t, SRA_FP8_E4M3);
    else SRA_FP8_ENC(uint16_t, SRA_FP8_E5M2);
  } else {
    if (kind == SRA_FP8_E4M3) SRA_FP8_ENC(float, SRA_FP8_E4M3);
    else SRA_FP8_ENC(float, SRA_FP8_E5M2);
  }
#undef SRA_FP8_ENC
  return hipGetLastError();
}

hipError_t launch_fp8_decode(int dtype, int kind, const uint8_t* codes, const uint8_t* exps, int64_t R, int64_t C,
                             int block_rows, void* x, hipStream_t s) {
  if (R <= 0 || C <= 0) return hipSuccess;
  if (block_rows == 1 && C % kBlock == 0) C *= R, R = 1;
  if (dtype == SRA_BF16) {
    if (kind == SRA_FP8_E4M3) decode<uint16_t, SRA_FP8_E4M3>(codes, exps, R, C, block_rows, x, s);
    else decode<uint16_t, SRA_FP8_E5M2>(codes, exps, R, C, block_rows, x, s);
  } else {
    if (kind == SRA_FP8_E4M3) decode<float, SRA_FP8_E4M3>(codes, exps, R, C, block_rows, x, s);
    else decode<float, SRA_FP8_E5M2>(codes, exps, R, C, block_rows, x, s);
  }
  return hipGetLastError();
}

}  // namespace sra
