// Gradients of many adapters beside one projection (each token t takes adapter ids[t]):
//
//   dA_g[j][k] = sum over the tokens of g of dU[t][j] X[t][k]
//   dB_g[n][j] = sum over the tokens of g of dY[t][n] U[t][j]
//
// k_multi_prep, one launch for what the products need from ids, A and B:
//   workgroup 0 sorts the tokens by adapter (a stable counting sort, so sums run in token order):
//     adapter g's tokens fill blocks gblk[g] .. gblk[g+1]-1 of 32 entries of perm, the last block
//     of each adapter padded with -1; tokens with no adapter are left out;
//   the other workgroups transpose every B_g (the dU product's operand, contiguous along N) and
//     every A_g (the dX epilogue's rows of r entries), in 64 x 64 tiles.
//
// k_multi_grads: a workgroup owns one adapter, 64 MF columns of dY or X and up to 128 adapter
// columns, and walks over the adapter's blocks, so an output element is summed by one workgroup in
// a fixed order and written once: no atomics and no partials.  A 32-token step gathers the tokens'
// rows into LDS as they lie ([t][m], 16-byte chunks; an 8-bit checkpoint is decoded on the way,
// exactly) and U or dU as three bf16 parts [part][j][t] that together carry its 24 bits (the sums
// cancel, so V's rounding would be amplified).  The products are v_mfma_f32_16x16x32_bf16: A
// operand V^T rows (16-byte LDS reads), B operand Act columns by ds_read_b64_tr_b16, the
// transposing LDS read.  The next step's rows are in flight (registers) while a step multiplies;
// two LDS buffers, one barrier per step.
#include <algorithm>

#include "rowvec.h"

namespace {

constexpr int kMaxAdapters = 1023, kPrepThreads = 1024, kPrepWaves = kPrepThreads / 64;

struct PrepArgs {
  const int32_t* ids;  // nullptr: no sort
  int64_t T;
  int n;
  int32_t* gblk;
  int32_t* perm;
  const uint16_t* B;  // [n][N][r] -> wt [n][r][N]; nullptr: none
  int64_t N;
  uint16_t* wt;
  const uint16_t* A;  // [n][r][K] -> at [n][K][lda]; nullptr: none
  int64_t K, lda;
  uint16_t* at;
  int r, b_tiles, a_tiles;  // 64 x 64 tiles per adapter
};

struct SortLds {
  int hist[kPrepWaves][kMaxAdapters + 1];
  int base[kMaxAdapters + 1];
  int wsum[kPrepWaves];
};
struct TileLds {
  uint16_t t[64][66];
};
union PrepLds {
  SortLds s;
  TileLds t;
};

SRA_DEV void sort_tokens(const PrepArgs& a, SortLds& s) {
  const int tid = threadIdx.x, w = tid >> 6, l = tid & 63;
  for (int i = tid; i < kPrepWaves * (kMaxAdapters + 1); i += kPrepThreads) (&s.hist[0][0])[i] = 0;
  __syncthreads();
  // wave w takes tokens [w * chunk, (w + 1) * chunk)
  const int64_t chunk = ((a.T + kPrepWaves - 1) / kPrepWaves + 63) / 64 * 64;
  const int64_t lo = w * chunk, hi = min(a.T, lo + chunk);
  for (int64_t t = lo + l; t < hi; t += 64) {
    const int g = a.ids[t];
    if (g >= 0 && g < a.n) atomicAdd(&s.hist[w][g], 1);  // LDS counts: the order does not matter
  }
  __syncthreads();
  // thread g: where each wave's tokens of adapter g start, and the adapter's blocks
  int cnt = 0, blocks = 0;
  if (tid < a.n) {
    for (int i = 0; i < kPrepWaves; ++i) {
      const int c = s.hist[i][tid];
      s.hist[i][tid] = cnt;
      cnt += c;
    }
    blocks = (cnt + 31) / 32;
  }
  int incl = blocks;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(incl, d, 64);
    if (l >= d) incl += v;
  }
  if (l == 63) s.wsum[w] = incl;
  __syncthreads();
  for (int i = 0; i < w; ++i) incl += s.wsum[i];
  const int first = incl - blocks;
  if (tid < a.n) {
    s.base[tid] = first;
    a.gblk[tid] = first;
    if (tid == a.n - 1) a.gblk[a.n] = incl;
    for (int p = cnt; p < 32 * blocks; ++p) a.perm[(int64_t)first * 32 + p] = -1;
  }
  __syncthreads();
  volatile int* const at = s.hist[w];  // this wave's running positions (only this wave uses them)
  for (int64_t t0 = lo; t0 < hi; t0 += 64) {
    const int64_t t = t0 + l;
    const int g = t < hi ? a.ids[t] : -1;
    uint64_t todo = __ballot(g >= 0 && g < a.n);
    while (todo) {
      const int lead = __builtin_ctzll(todo);
      const int cur = __builtin_amdgcn_readlane(g, lead);
      const uint64_t same = __ballot(g == cur);
      todo &= ~same;
      const int start = at[cur];
      if (g == cur) a.perm[(int64_t)s.base[cur] * 32 + start + __popcll(same & ((1ull << l) - 1))] = (int32_t)t;
      if (l == lead) at[cur] = start + __popcll(same);
    }
  }
}

// dst[y][x] = src[x][y] for one 64 x 64 tile (X x Y source, dst rows of stride ld)
SRA_DEV void transpose64(const uint16_t* __restrict__ src, int64_t X, int64_t Y, uint16_t* __restrict__ dst, int64_t ld,
                         int64_t x0, int64_t y0, TileLds& s) {
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
#pragma unroll
  for (int k = 0; k < 64 / kPrepWaves; ++k) {
    const int i = ty + kPrepWaves * k;
    const int64_t x = x0 + i, y = y0 + tx;
    s.t[i][tx] = (x < X && y < Y) ? src[x * Y + y] : (uint16_t)0;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 64 / kPrepWaves; ++k) {
    const int i = ty + kPrepWaves * k;
    const int64_t y = y0 + i, x = x0 + tx;
    if (y < Y && x < X) dst[y * ld + x] = s.t[tx][i];
  }
}

__global__ __launch_bounds__(kPrepThreads) void k_multi_prep(PrepArgs a) {
  __shared__ PrepLds lds;
  int64_t b = blockIdx.x;
  if (a.ids) {
    if (b == 0) {
      sort_tokens(a, lds.s);
      return;
    }
    --b;
  }
  const int64_t nb = (int64_t)a.n * a.b_tiles;
  if (b < nb) {
    const int64_t g = b / a.b_tiles, i = b % a.b_tiles, yt = (a.r + 63) / 64;
    transpose64(a.B + g * a.N * a.r, a.N, a.r, a.wt + g * a.N * a.r, a.N, i / yt * 64, i % yt * 64, lds.t);
  } else {
    b -= nb;
    const int64_t g = b / a.a_tiles, i = b % a.a_tiles, xt = (a.r + 63) / 64;
    transpose64(a.A + g * a.r * a.K, a.r, a.K, a.at + g * a.K * a.lda, a.lda, i % xt * 64, i / xt * 64, lds.t);
  }
}

// ------------------------------------------------------------------------------------ gradients
struct GradJob {
  const uint16_t* act;   // [T][M] bf16, or
  const int8_t* codes;   // its 8-bit checkpoint (act == nullptr)
  const uint8_t* exps;
  const float* V;        // [T][r]
  float* out;            // [n][r][M] (out_t) or [n][M][r]
  int64_t M;
  int mb;                // column tiles
  bool out_t;
};
struct GradArgs {
  GradJob job[2];
  const int32_t* gblk;
  const int32_t* perm;
  int r;
};

typedef short v4s __attribute__((ext_vector_type(4)));
SRA_DEV v4s lds_tr(const uint8_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)p);
}

// chunk swizzle of the Act tile's token row t (8 chunks per row, or 16 and more): over the rows of
// one transposing read the 32-byte windows spread over the LDS banks
template <int MT>
SRA_DEV int act_swz(int t) {
  return MT == 64 ? 2 * (((t >> 1) ^ (t >> 3)) & 3) : 2 * ((t & 3) | (((t >> 3) & 1) << 2));
}

template <int JT, int MF>
struct GradTile {
  static constexpr int JR = 16 * JT, MT = 64 * MF, AROW = MT * 2;
  static constexpr int A_BYTES = 32 * AROW, V_BYTES = 3 * JR * 64, BUF = A_BYTES + V_BYTES;
  static constexpr int NA = 32 * MT / 8 / 256;                // 16-byte Act chunks per thread
  static constexpr int NV = (JR * 4 + 255) / 256;             // (adapter column, 8 tokens) pieces per thread
};

template <int JT, int MF>
__global__ __launch_bounds__(256) void k_multi_grads(GradArgs ga) {
  using G = GradTile<JT, MF>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * G::BUF];
  const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, l16 = l & 15, q4 = l >> 4;
  const bool second = (int)blockIdx.x >= ga.job[0].mb;
  const GradJob& job = second ? ga.job[1] : ga.job[0];
  const int64_t m0 = ((int64_t)blockIdx.x - (second ? ga.job[0].mb : 0)) * G::MT, M = job.M;
  const int g = blockIdx.y, j0 = blockIdx.z * G::JR, r = ga.r;
  const int b0 = ga.gblk[g], b1 = ga.gblk[g + 1];
  const int64_t nblk = (M + sra_row::kCkBlock - 1) / sra_row::kCkBlock;

  u32x4 ar[G::NA];       // bf16 chunks, or codes in the low half and the exponent
  float vr[G::NV][8];
  auto load = [&](int b) {
    const int32_t* p = ga.perm + (int64_t)b * 32;
#pragma unroll
    for (int i = 0; i < G::NA; ++i) {
      const int v = tid + 256 * i, t = v / (G::MT / 8), c = v % (G::MT / 8);
      const int64_t tok = p[t], m = m0 + 8 * c;
      ar[i] = u32x4{0, 0, 0, 0};
      if (tok >= 0 && m < M) {  // M % 8 == 0: a chunk is inside a row or past it
        if (job.act) {
          ar[i] = *reinterpret_cast<const u32x4*>(job.act + tok * M + m);
        } else {
          const u32x2 q = *reinterpret_cast<const u32x2*>(job.codes + tok * M + m);
          ar[i] = u32x4{q[0], q[1], job.exps[tok * nblk + m / sra_row::kCkBlock], 0};
        }
      }
    }
#pragma unroll
    for (int i = 0; i < G::NV; ++i) {
      const int v = tid + 256 * i, j = v % G::JR, t8 = v / G::JR;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        vr[i][e] = 0.f;
        if (t8 < 4 && j0 + j < r) {
          const int64_t tok = p[8 * t8 + e];
          if (tok >= 0) vr[i][e] = job.V[tok * r + j0 + j];
        }
      }
    }
  };
  auto store = [&](uint8_t* buf) {
#pragma unroll
    for (int i = 0; i < G::NA; ++i) {
      const int v = tid + 256 * i, t = v / (G::MT / 8), c = v % (G::MT / 8);
      u32x4 x = ar[i];
      if (!job.act) {
        float f[8];
        sra_row::ck_decode<8>((uint64_t)ar[i][0] | ((uint64_t)ar[i][1] << 32), ar[i][2], f);
#pragma unroll
        for (int k = 0; k < 4; ++k)  // exact in bf16: the high halves are the values
          x[k] = (__float_as_uint(f[2 * k]) >> 16) | (__float_as_uint(f[2 * k + 1]) & 0xffff0000u);
      }
      *reinterpret_cast<u32x4*>(buf + t * G::AROW + ((c ^ act_swz<G::MT>(t)) << 4)) = x;
    }
    uint8_t* vb = buf + G::A_BYTES;
#pragma unroll
    for (int i = 0; i < G::NV; ++i) {
      const int v = tid + 256 * i, j = v % G::JR, t8 = v / G::JR;
      if (t8 < 4) {
        union { uint16_t h[8]; u32x4 v; } p[3];
#pragma unroll
        for (int e = 0; e < 8; ++e) split3_bf16(vr[i][e], p[0].h[e], p[1].h[e], p[2].h[e]);
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const int x = k * G::JR + j;
          *reinterpret_cast<u32x4*>(vb + x * 64 + ((t8 ^ ((x >> 2) & 3)) << 4)) = p[k].v;
        }
      }
    }
  };

  f32x4 acc[JT][MF];
#pragma unroll
  for (int a = 0; a < JT; ++a)
#pragma unroll
    for (int f = 0; f < MF; ++f) acc[a][f] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int fr = l16 >> 2, fs = l16 & 3;
  auto compute = [&](const uint8_t* buf) {
    bf16x8 bf[MF];
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      union { v4s h[2]; bf16x8 b; } u;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t = 8 * q4 + 4 * h + fr, col = (w * MF + f) * 16 + 4 * fs;
        u.h[h] = lds_tr(buf + t * G::AROW + (((col >> 3) ^ act_swz<G::MT>(t)) << 4) + (col & 7) * 2);
      }
      bf[f] = u.b;
    }
    const uint8_t* vb = buf + G::A_BYTES;
#pragma unroll
    for (int a = 0; a < JT; ++a)
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const int x = k * G::JR + 16 * a + l16;
        const bf16x8 vf = *reinterpret_cast<const bf16x8*>(vb + x * 64 + ((q4 ^ ((x >> 2) & 3)) << 4));
#pragma unroll
        for (int f = 0; f < MF; ++f) acc[a][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, bf[f], acc[a][f], 0, 0, 0);
      }
  };

  if (b0 < b1) load(b0);
  for (int b = b0; b < b1; ++b) {
    uint8_t* buf = lds + ((b - b0) & 1) * G::BUF;
    store(buf);
    __syncthreads();  // the buffer is written; every wave is done with the other one's last use
    if (b + 1 < b1) load(b + 1);
    compute(buf);
  }

  // D layout: adapter column 4 (l / 16) + e of fragment a, Act column l % 16 of fragment f
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    const int64_t m = m0 + (w * MF + f) * 16 + l16;
    if (m >= M) continue;
#pragma unroll
    for (int a = 0; a < JT; ++a)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = j0 + 16 * a + 4 * q4 + e;
        if (j < r) job.out[job.out_t ? ((int64_t)g * r + j) * M + m : ((int64_t)g * M + m) * r + j] = acc[a][f][e];
      }
  }
}

int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

namespace sra {

int multi_max_adapters() { return kMaxAdapters; }
int64_t multi_perm_entries(int64_t T, int n) { return 32 * (T / 32 + std::min<int64_t>(n, T)); }

hipError_t launch_multi_prep(const MultiPrep& p, hipStream_t s) {
  PrepArgs a{};
  a.ids = p.gblk ? p.ids : nullptr;
  a.T = p.T;
  a.n = p.n;
  a.gblk = p.gblk;
  a.perm = p.perm;
  a.B = p.B;
  a.N = p.N;
  a.wt = p.wt;
  a.A = p.A;
  a.K = p.K;
  a.lda = packed_at_ld(p.r);
  a.at = p.at;
  a.r = p.r;
  a.b_tiles = p.wt ? (int)(cdiv64(p.N, 64) * cdiv64(p.r, 64)) : 0;
  a.a_tiles = p.at ? (int)(cdiv64(p.K, 64) * cdiv64(p.r, 64)) : 0;
  const int64_t blocks = (a.ids ? 1 : 0) + (int64_t)p.n * (a.b_tiles + a.a_tiles);
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL(k_multi_prep, dim3((unsigned)blocks), dim3(kPrepThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_multi_grads(const MultiGrad* g, int n_jobs, const int32_t* gblk, const int32_t* perm, int n, int r,
                              hipStream_t s) {
  if (n_jobs <= 0 || r <= 0 || n <= 0) return hipSuccess;
  GradArgs ga{};
  ga.gblk = gblk;
  ga.perm = perm;
  ga.r = r;
  int64_t cols = 0;
  for (int i = 0; i < n_jobs; ++i) cols += g[i].M;
  const int jt = r <= 16 ? 1 : r <= 32 ? 2 : r <= 64 ? 4 : 8;
  const bool wide = cdiv64(cols, 128) * n >= 512;
  const int mt = wide ? 128 : 64;
  int64_t mb = 0;
  for (int i = 0; i < n_jobs; ++i) {
    GradJob& j = ga.job[i];
    j.act = g[i].act;
    j.codes = g[i].codes;
    j.exps = g[i].exps;
    j.V = g[i].V;
    j.out = g[i].out;
    j.M = g[i].M;
    j.mb = (int)cdiv64(g[i].M, mt);
    j.out_t = g[i].out_t;
    mb += j.mb;
  }
  if (mb == 0) return hipSuccess;
  const dim3 grid((unsigned)mb, (unsigned)n, (unsigned)cdiv64(r, 16 * jt));
#define SRA_MG(JT)                                                                                    \
  do {                                                                                                \
    if (wide) launch(SRA_KERNEL_ADAPTER, k_multi_grads<JT, 2>, grid, dim3(256), 0, s, ga);             \
    else launch(SRA_KERNEL_ADAPTER, k_multi_grads<JT, 1>, grid, dim3(256), 0, s, ga);                  \
  } while (0)
  if (jt == 1) SRA_MG(1);
  else if (jt == 2) SRA_MG(2);
  else if (jt == 4) SRA_MG(4);
  else SRA_MG(8);
#undef SRA_MG
  return hipGetLastError();
}

}  // namespace sra
