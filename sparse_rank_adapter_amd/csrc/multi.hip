// Gradients of many adapters beside one projection (each token t takes adapter ids[t]):
//
//   dA_g[j][k] = sum over the tokens of g of dU[t][j] X[t][k]
//   dB_g[n][j] = sum over the tokens of g of dY[t][n] U[t][j]
//
// k_multi_prep, one launch for what the products need from ids, A and B:
//   workgroup 0 sorts the tokens by adapter (a stable counting sort, so sums run in token order):
//     each adapter's tokens fill blocks of 32 entries of perm, the last block padded with -1 (loads
//     there read token 0 and are cleared); tokens with no adapter are left out; the adapters' list
//     runs by falling block count (up to 64 adapters), so that the longest start first;
//   the other workgroups transpose every B_g (the dU product's operand, contiguous along N) and
//     every A_g (the dX epilogue's rows of r entries), in tiles of 8192 elements.
//   It is bound by the sort's chain of dependent steps at small sizes (5.3 us: 2047 tokens, 12 adapters,
//   rank 16, K + N = 5120) and by HBM at large ones (13.7 us for the 105 MB that 8 adapters of rank 128
//   and K + N = 25600 read and write).
//
// The gradients are sums over an adapter's tokens of products of one Act value (dY or X, bf16, or an
// 8-bit checkpoint decoded on the way, exactly) with one V value (U or dU, fp32, split into three
// bf16 parts that together carry its 24 bits: the sums cancel, so V's rounding would be amplified).
// The products are v_mfma_f32_16x16x32_bf16, 32 tokens a step: A operand V^T rows, B operand Act
// columns by ds_read_b64_tr_b16, the transposing LDS read, from tiles that hold the tokens' gathered
// rows as they lie ([t][m], swizzled 16-byte chunks).  Sums run in a fixed order; where an adapter's
// tiles would leave most of the GPU idle, its tokens are cut into slices whose fp32 partials one
// more launch adds in slice order.
//
// Ranks up to 32 (k_multi_grads_few) are bound by reading Act and by latency.  A workgroup owns one
// adapter and 64 columns; its NW waves take every NW-th 32-token block, each through its own LDS
// tile with no barrier, and join their sums at the end, so an adapter's chain of steps is 1 / NW as
// long and 16 waves a CU keep loads in flight.  V is read and split by each wave itself.  10 us for dA
// and dB of 2047 tokens, 12 adapters, rank 16, K = 4096, N = 1024: 21 MB of Act at 2.1 TB/s, bound by
// the longest adapter's chain of steps.
//
// Larger ranks (k_multi_grads) are bound by the matrix cores and by LDS reads of V.  V is split once
// (k_multi_vt) into tiles of 32 tokens in the sorted order, contiguous per step; a workgroup of
// eight waves owns 256 columns and 64 or 128 adapter columns (wave: 64 adapter columns by 32 or 64
// columns), has both tiles two steps ahead and double-buffers LDS.  182 us for 8192 tokens, 8
// adapters, rank 128, K = 5120 (a checkpoint), N = 20480: 161 GFLOP of the three parts at 0.88
// PFLOP/s, where a large bf16 matrix product reaches 1.34; the matrix cores are busy for 40% of the
// cycles and the 800 workgroups take unequal shares of the tokens.
//
// Both load whole 16-byte pieces of Act's rows (8-byte ones of codes up to rank 32): rows of any other
// length are copied to whole ones first (k_multi_pad).
#include <algorithm>

#include "rowvec.h"

namespace {

constexpr int kMaxAdapters = 1023, kPrepThreads = 1024, kPrepWaves = kPrepThreads / 64;

struct PrepArgs {
  const int32_t* ids;  // nullptr: no sort
  int64_t T;
  int n;
  int32_t* gblk;       // gblk[n]: the block count; then, 16-byte aligned, per adapter in falling order
                       // of its blocks {adapter, first block, end, 0}
  int32_t* perm;
  const uint16_t* B;  // [n][N][r] -> wt [n][r][N]; nullptr: none
  int64_t N;
  uint16_t* wt;
  const uint16_t* A;  // [n][r][K] -> at [n][K][lda]; nullptr: none
  int64_t K, lda;
  uint16_t* at;
  int r, b_tiles, a_tiles;  // tiles per adapter
};

// offset (entries) of the adapters' list after gblk [n + 1], 16-byte aligned
__host__ __device__ inline int group_list(int n) { return (n + 1 + 3) / 4 * 4; }

struct SortLds {
  int hist[kPrepWaves][kMaxAdapters + 1];
  int base[kMaxAdapters + 1];
  int wsum[kPrepWaves];
};
// 512 x (16 + 2), the largest of the tile shapes with their padding
struct TileLds {
  uint16_t t[512 * 18];
};
union PrepLds {
  SortLds s;
  TileLds t;
};

// The lanes of a wave that name the same adapter: the number of them and this lane's place among
// them (g < 0: none).
struct Match {
  int count, place;
};
SRA_DEV Match match_adapter(int g, int l) {
  Match m{0, 0};
  uint64_t todo = __ballot(g >= 0);
  while (todo) {
    const int lead = __builtin_ctzll(todo);
    const uint64_t same = __ballot(g == __builtin_amdgcn_readlane(g, lead));
    todo &= ~same;
    if ((same >> l) & 1) m = {(int)__popcll(same), (int)__popcll(same & ((1ull << l) - 1))};
  }
  return m;
}
SRA_DEV void sort_tokens(const PrepArgs& a, SortLds& s) {
  const int tid = threadIdx.x, w = tid >> 6, l = tid & 63;
  // wave w takes tokens [w * chunk, (w + 1) * chunk)
  const int64_t chunk = ((a.T + kPrepWaves - 1) / kPrepWaves + 63) / 64 * 64;
  const int64_t lo = w * chunk, hi = min(a.T, lo + chunk);
  constexpr int KEEP = 4;  // the wave's first tokens are walked once: adapter and place stay in registers
  int kept[KEEP], at[KEEP];
  auto load_id = [&](int64_t t) {
    const int g = t < hi ? a.ids[t] : -1;
    return g < a.n ? g : -1;
  };
#pragma unroll
  for (int k = 0; k < KEEP; ++k) kept[k] = load_id(lo + 64 * k + l);
  volatile int* const mine = s.hist[w];  // this wave's counts: only this wave uses them until the barrier
  for (int i = l; i < a.n; i += 64) mine[i] = 0;
  // this wave's tokens of the same adapter before the lane's: one LDS round trip for 64 tokens
  auto take = [&](int g) {
    const Match m = match_adapter(g, l);
    int before = 0;
    if (g >= 0) before = mine[g];
    if (g >= 0 && m.place == 0) mine[g] = before + m.count;
    return before + m.place;
  };
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    at[k] = 0;
    if (lo + 64 * k < hi) at[k] = take(kept[k]);
  }
  for (int64_t t0 = lo + 64 * KEEP; t0 < hi; t0 += 64) {  // counted here, placed by the second walk
    const int g = load_id(t0 + l);
    if (g >= 0) atomicAdd(&s.hist[w][g], 1);  // LDS integers: the order does not matter
  }
  __syncthreads();
  // thread g: where each wave's tokens of adapter g start, and the adapter's blocks
  int cnt = 0, blocks = 0;
  if (tid < a.n) {
    int c[kPrepWaves];
#pragma unroll
    for (int i = 0; i < kPrepWaves; ++i) c[i] = s.hist[i][tid];
#pragma unroll
    for (int i = 0; i < kPrepWaves; ++i) {
      s.hist[i][tid] = cnt;
      cnt += c[i];
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
  int sums[kPrepWaves];
#pragma unroll
  for (int i = 0; i < kPrepWaves; ++i) sums[i] = s.wsum[i];
#pragma unroll
  for (int i = 0; i < kPrepWaves; ++i) incl += i < w ? sums[i] : 0;
  const int first = incl - blocks;
  if (tid < a.n) {
    s.base[tid] = first;
    if (tid == a.n - 1) a.gblk[a.n] = incl;
  }
  __syncthreads();
  int start[KEEP];
#pragma unroll
  for (int k = 0; k < KEEP; ++k) start[k] = kept[k] >= 0 ? s.base[kept[k]] * 32 + s.hist[w][kept[k]] : 0;
#pragma unroll
  for (int k = 0; k < KEEP; ++k)
    if (kept[k] >= 0) a.perm[start[k] + at[k]] = (int32_t)(lo + 64 * k + l);
  if (a.n > 64) {
    if (tid < a.n) reinterpret_cast<int4*>(a.gblk + group_list(a.n))[tid] = int4{tid, first, first + blocks, 0};
  } else if (w == 0) {  // by falling block count, ties by index
    int rank = 0;
    for (int i = 0; i < a.n; ++i) {
      const int b = __builtin_amdgcn_readlane(blocks, i);
      rank += b > blocks || (b == blocks && i < tid);
    }
    if (tid < a.n) reinterpret_cast<int4*>(a.gblk + group_list(a.n))[rank] = int4{tid, first, first + blocks, 0};
  }
  if (tid < a.n)
    for (int i = cnt; i < 32 * blocks; ++i) a.perm[(int64_t)first * 32 + i] = -1;
  if (lo + 64 * KEEP >= hi) return;
  // the wave's later tokens: its counts become running places, which start behind the kept tokens
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    const Match m = match_adapter(kept[k], l);
    if (kept[k] >= 0 && m.place == 0) mine[kept[k]] = mine[kept[k]] + m.count;
  }
  for (int64_t t0 = lo + 64 * KEEP; t0 < hi; t0 += 64) {
    const int g = load_id(t0 + l), p = take(g);
    if (g >= 0) a.perm[s.base[g] * 32 + p] = (int32_t)(t0 + l);
  }
}

// dst[y][x] = src[x][y] for one tile of 2^lx by 2^ly (X x Y source, dst rows of stride ld), 16 bytes a
// lane on both sides where the rows allow (X, Y and ld multiples of 8: the matrices' bases are 16-byte
// aligned).  A tile has 8192 elements whatever its shape, one load and one store a thread: tiles of
// 64 x 64 left three quarters of the lanes idle at rank 16.
SRA_DEV void transpose_tile(const uint16_t* __restrict__ src, int64_t X, int64_t Y, uint16_t* __restrict__ dst, int64_t ld,
                            int lx, int ly, int64_t x0, int64_t y0, TileLds& s) {
  const int tid = threadIdx.x, pitch = (1 << ly) + 2;
  // chunk i of 1024 -> (row, chunk of the row): eight chunks (128 bytes) of a row, then the rows, so that
  // the gathering reads spread over the banks
  auto place = [](int i, int lrows, int lchunks, int& row, int& c) {
    const int lc = min(lchunks, 3);
    c = (i & ((1 << lc) - 1)) | (i >> (lrows + lc) << lc);
    row = (i >> lc) & ((1 << lrows) - 1);
  };
  if (((X | Y | ld) & 7) == 0) {
    int i, c;
    place(tid, lx, ly - 3, i, c);
    {
      const int64_t x = x0 + i, y = y0 + 8 * c;
      union { u32x4 v; uint32_t w[4]; } u;
      u.v = u32x4{0, 0, 0, 0};
      if (x < X && y < Y) u.v = *reinterpret_cast<const u32x4*>(src + x * Y + y);
#pragma unroll
      for (int k = 0; k < 4; ++k) *reinterpret_cast<uint32_t*>(&s.t[i * pitch + 8 * c + 2 * k]) = u.w[k];
    }
    __syncthreads();
    place(tid, ly, lx - 3, i, c);  // row y0 + i, columns x0 + 8 c ..
    const int64_t y = y0 + i, x = x0 + 8 * c;
    union { u32x4 v; uint16_t h[8]; } u;
#pragma unroll
    for (int k = 0; k < 8; ++k) u.h[k] = s.t[(8 * c + k) * pitch + i];
    if (y < Y && x < X) *reinterpret_cast<u32x4*>(dst + y * ld + x) = u.v;
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int e = tid + kPrepThreads * k, i = e >> ly, j = e & ((1 << ly) - 1);
    const int64_t x = x0 + i, y = y0 + j;
    s.t[i * pitch + j] = (x < X && y < Y) ? src[x * Y + y] : (uint16_t)0;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int e = tid + kPrepThreads * k, i = e >> lx, j = e & ((1 << lx) - 1);
    const int64_t y = y0 + i, x = x0 + j;
    if (y < Y && x < X) dst[y * ld + x] = s.t[j * pitch + i];
  }
}
// a tile's extent along the rank, as a power of two: 2^13 elements lie in one
__host__ __device__ inline int tile_lr(int r) { return r <= 16 ? 4 : r <= 32 ? 5 : 6; }

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
  const int lr = tile_lr(a.r), lm = 13 - lr;
  const int64_t rt = (a.r + (1 << lr) - 1) >> lr;  // tiles along the rank
  if (b < nb) {
    const int64_t g = b / a.b_tiles, i = b % a.b_tiles;
    transpose_tile(a.B + g * a.N * a.r, a.N, a.r, a.wt + g * a.N * a.r, a.N, lm, lr, i / rt << lm, i % rt << lr, lds.t);
  } else {
    b -= nb;
    const int64_t g = b / a.a_tiles, i = b % a.a_tiles;
    transpose_tile(a.A + g * a.r * a.K, a.r, a.K, a.at + g * a.K * a.lda, a.lda, lr, lm, i % rt << lr, i / rt << lm, lds.t);
  }
}

// ------------------------------------------------------------------------------------ gradients
struct GradJob {
  const uint16_t* act;   // [T][M] bf16, or
  const int8_t* codes;   // its 8-bit checkpoint (act == nullptr)
  const uint8_t* exps;
  const float* V;        // [T][r]
  uint16_t* vt;          // its parts [block][3][rp][32], ranks above 32
  float* out;            // [n][r][M] (out_t) or [n][M][r]; with slices, partials of slice 0
  int64_t M, ld;         // columns, act's row length (multi_grad_fits)
  int mb;                // column tiles
  bool out_t;
};
struct GradArgs {
  GradJob job[2];
  const int32_t* gblk;
  const int32_t* perm;
  int n, r, rp;
  int S;                 // slices of an adapter's blocks
  int64_t slice;         // elements from one slice's partials to the next
};

union Bf8 {
  __bf16 h[8];
  u32x4 v;
  bf16x8 b;
  tr_v4s half[2];
};
// x = a + b + c with bf16 parts (below fp32's rounding; the differences are exact)
SRA_DEV void split3(float x, __bf16& a, __bf16& b, __bf16& c) {
  a = (__bf16)x;
  const float r1 = x - (float)a;
  b = (__bf16)r1;
  c = (__bf16)(r1 - (float)b);
}
// eight codes of a checkpoint as bf16: q 2^e is exact, so the high halves of the fp32 values are it
SRA_DEV u32x4 decode8(uint32_t lo, uint32_t hi, uint32_t exp) {
  float f[8];
  sra_row::ck_decode<8>((uint64_t)lo | ((uint64_t)hi << 32), exp, f);
  u32x4 x;
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = __builtin_amdgcn_perm(__float_as_uint(f[2 * k + 1]), __float_as_uint(f[2 * k]), 0x07060302u);
  return x;
}

// chunk swizzle of a tile's row t (8 chunks of 16 bytes per row, or 16 and more): over the rows of one
// transposing read the 32-byte windows spread over the LDS banks.  Bit 2 of t is not used, so the two
// reads of a fragment, four rows apart, have one swizzle (and so have rows 32 apart).
template <int MT>
SRA_DEV int act_swz(int t) {
  return MT == 64 ? 2 * (((t >> 1) & 1) | (((t >> 3) & 1) << 1)) : 2 * ((t & 3) | (((t >> 3) & 1) << 2));
}
// B operand of 16 columns from m0 (a multiple of 16) of an Act tile [32][MT]
template <int MT>
SRA_DEV bf16x8 act_frag(const uint8_t* tile, int m0, int l16, int q4) {
  Bf8 u;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int t = 8 * q4 + 4 * h + (l16 >> 2), col = m0 + 4 * (l16 & 3);
    u.half[h] = lds_tr(tile + t * (2 * MT) + (((col >> 3) ^ act_swz<MT>(t)) << 4) + (col & 7) * 2);
  }
  return u.b;
}

// the k-th adapter of the list (the longest first) and the blocks [lo, hi) of its slice z
SRA_DEV int slice_of(const GradArgs& ga, int k, int z, int& lo, int& hi) {
  const int4 e = reinterpret_cast<const int4*>(ga.gblk + group_list(ga.n))[k];
  const int per = (e.z - e.y + ga.S - 1) / ga.S;
  lo = min(e.z, e.y + z * per);
  hi = min(e.z, lo + per);
  return e.x;
}
// D layout: adapter column 4 (l / 16) + e, Act column l % 16
SRA_DEV void grad_store(const GradArgs& ga, const GradJob& job, int g, int z, int j0, int64_t m0, const f32x4& c, int l16,
                        int q4) {
  const int64_t m = m0 + l16;
  if (m >= job.M) return;
  float* out = job.out + (int64_t)z * ga.slice;
  const int j = j0 + 4 * q4;
  if (!job.out_t) {
    float* o = out + ((int64_t)g * job.M + m) * ga.r + j;
    if ((ga.r & 3) == 0 && j + 4 <= ga.r) {
      *reinterpret_cast<f32x4*>(o) = c;
      return;
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (j + e < ga.r) out[job.out_t ? ((int64_t)g * ga.r + j + e) * job.M + m : ((int64_t)g * job.M + m) * ga.r + j + e] = c[e];
}

// ---- ranks up to 32
template <int JT, int NW>
__global__ __launch_bounds__(64 * NW) void k_multi_grads_few(GradArgs ga) {
  constexpr int MT = 64, TILE = 32 * MT * 2;
  constexpr int RED = NW * JT * 4 * 64 * 16;  // the waves' sums: [wave][a][f][lane]
  __shared__ __attribute__((aligned(16))) uint8_t lds[RED > NW * TILE ? RED : NW * TILE];
  const int tid = threadIdx.x, l = tid & 63, l16 = l & 15, q4 = l >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const bool second = (int)blockIdx.x >= ga.job[0].mb;
  const GradJob job = second ? ga.job[1] : ga.job[0];
  const int64_t m0 = ((int64_t)blockIdx.x - (second ? ga.job[0].mb : 0)) * MT, ld = job.ld;
  const int z = blockIdx.z, r = ga.r;
  int b0, b1;
  const int g = slice_of(ga, blockIdx.y, z, b0, b1);
  const int64_t nblk = (ld + sra_row::kCkBlock - 1) / sra_row::kCkBlock;
  uint8_t* const tile = lds + w * TILE;

  // a lane's share of a block: chunk l % 8 of rows l / 8 + 8 i, and V of adapter column l % 16 at the
  // tokens 8 (l / 16) + e
  const int c8 = l & 7, r8 = l >> 3;
  const int64_t mc = min(m0 + 8 * c8, ld - 8);  // past the row (ld % 8 == 0): any columns, their sums are not stored
  u32x4 ar[4];
  float vr[JT][8];
  uint32_t a_ok = 0, v_ok = 0;  // bit: the row (token) is no padding.  Clearing waits for the data, so it
                                // happens where the data is used, not where it is loaded
  auto perm_of = [&](int b) { return ga.perm[(int64_t)min(b, b1 - 1) * 32 + (l & 31)]; };
  auto load = [&](int p) {  // p: lane l % 32 holds the block's token l % 32 (-1: padding)
    a_ok = v_ok = 0;
    int64_t tok[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = __shfl(p, r8 + 8 * i, 64);
      a_ok |= (uint32_t)(q >= 0) << i;
      tok[i] = max(q, 0);
    }
    if (job.act) {
#pragma unroll
      for (int i = 0; i < 4; ++i) ar[i] = *reinterpret_cast<const u32x4*>(job.act + tok[i] * ld + mc);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const u32x2 q = *reinterpret_cast<const u32x2*>(job.codes + tok[i] * ld + mc);
        ar[i] = u32x4{q[0], q[1], job.exps[tok[i] * nblk + mc / sra_row::kCkBlock], 0};
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int q = __shfl(p, 8 * q4 + e, 64);
      v_ok |= (uint32_t)(q >= 0) << e;
      const float* v = job.V + (int64_t)max(q, 0) * r;
#pragma unroll
      for (int a = 0; a < JT; ++a) vr[a][e] = v[min(16 * a + l16, r - 1)];
    }
  };
  f32x4 acc[JT][4];
#pragma unroll
  for (int a = 0; a < JT; ++a)
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[a][f] = f32x4{0.f, 0.f, 0.f, 0.f};

  int p = 0, pn = 0;
  if (b0 + w < b1) {
    p = perm_of(b0 + w);
    pn = perm_of(b0 + w + NW);
    load(p);
  }
  for (int b = b0 + w; b < b1; b += NW) {
    p = pn;
    pn = perm_of(b + 2 * NW);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = r8 + 8 * i;
      const u32x4 x = job.act ? ar[i] : decode8(ar[i][0], ar[i][1], ar[i][2]);
      *reinterpret_cast<u32x4*>(tile + t * (2 * MT) + ((c8 ^ act_swz<MT>(t)) << 4)) =
          (a_ok >> i) & 1u ? x : u32x4{0, 0, 0, 0};
    }
    Bf8 vf[JT][3];
#pragma unroll
    for (int a = 0; a < JT; ++a)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        split3((v_ok >> e) & 1u && 16 * a + l16 < r ? vr[a][e] : 0.f, vf[a][0].h[e], vf[a][1].h[e], vf[a][2].h[e]);
    if (b + NW < b1) load(p);  // in flight while this block multiplies
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const bf16x8 bf = act_frag<MT>(tile, 16 * f, l16, q4);  // this wave's own writes: in order
#pragma unroll
      for (int a = 0; a < JT; ++a)
#pragma unroll
        for (int k = 0; k < 3; ++k)
          acc[a][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf[a][k].b, bf, acc[a][f], 0, 0, 0);
    }
  }
  // join: fragment i = (a, f) is finished by wave i % NW, adding the waves in order
  __syncthreads();
  f32x4* const red = reinterpret_cast<f32x4*>(lds);
#pragma unroll
  for (int a = 0; a < JT; ++a)
#pragma unroll
    for (int f = 0; f < 4; ++f) red[((w * JT + a) * 4 + f) * 64 + l] = acc[a][f];
  __syncthreads();
  for (int i = w; i < 4 * JT; i += NW) {
    const int a = i >> 2, f = i & 3;
    f32x4 c = red[i * 64 + l];
#pragma unroll
    for (int k = 1; k < NW; ++k) c += red[(k * JT * 4 + i) * 64 + l];
    grad_store(ga, job, g, z, 16 * a, m0 + 16 * f, c, l16, q4);
  }
}

// ---- ranks above 32
template <int N>
SRA_DEV void wait_vm_all() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
// V in three parts, in the sorted order: tile b is [3][rp][32] bf16, zeros for padding and for
// adapter columns past r; 64 adapter columns per workgroup, gathered along r and written in whole
// lines through LDS.  grid: (blocks, jobs, 64-column parts)
__global__ __launch_bounds__(256) void k_multi_vt(GradArgs ga) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[3 * 64 * 32];
  const int b = blockIdx.x, jb = blockIdx.z * 64, nj = min(64, ga.rp - jb);
  if (b >= ga.gblk[ga.n]) return;
  const GradJob& job = ga.job[blockIdx.y];
  const int32_t* p = ga.perm + (int64_t)b * 32;
  const int jl = threadIdx.x & 63, j = jb + jl, t8 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Bf8 s[3];
  float x[8];
  uint32_t ok = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int q = p[8 * t8 + e];
    x[e] = job.V[(int64_t)max(q, 0) * ga.r + min(j, ga.r - 1)];
    ok |= (uint32_t)(q >= 0 && j < ga.r) << e;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) split3((ok >> e) & 1u ? x[e] : 0.f, s[0].h[e], s[1].h[e], s[2].h[e]);
#pragma unroll
  for (int k = 0; k < 3; ++k)  // 16-byte piece t8 of row (k, jl), pieces swizzled against bank conflicts
    *reinterpret_cast<u32x4*>(lds + ((k * 64 + jl) * 4 + (t8 ^ ((jl >> 2) & 3))) * 8) = s[k].v;
  __syncthreads();
  uint16_t* vt = job.vt + (int64_t)b * 3 * ga.rp * 32;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const int row = threadIdx.x >> 2, c = threadIdx.x & 3;
    if (row < nj)
      *reinterpret_cast<u32x4*>(vt + ((int64_t)k * ga.rp + jb + row) * 32 + 8 * c) =
          *reinterpret_cast<const u32x4*>(lds + ((k * 64 + row) * 4 + (c ^ ((row >> 2) & 3))) * 8);
  }
}

// WJ = 1: 64 adapter columns, 2: 128.  grid: (column tiles, adapters, adapter column tiles x slices).
// The V tile goes to LDS by buffer -> LDS transfers, Act through registers (a checkpoint is decoded
// there), both two steps ahead: with one step ahead and two workgroups per CU every step waited for
// its loads (192 us; 131 us with the loads taken out, and as much with the products taken out).
template <int WJ>
__global__ __launch_bounds__(512, 2) void k_multi_grads(GradArgs ga) {
  constexpr int MT = 256, JR = 64 * WJ, MF = 2 * WJ;
  constexpr int A_BYTES = 32 * MT * 2, V_BYTES = 3 * JR * 64;
  constexpr int NV = V_BYTES / 1024;  // 1 KB transfers: 12 or 24
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * A_BYTES + 3 * V_BYTES];
  uint8_t* const vlds = lds + 2 * A_BYTES;
  const int tid = threadIdx.x, l = tid & 63, l16 = l & 15, q4 = l >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6), wj = w % WJ, wm = w / WJ;
  const bool second = (int)blockIdx.x >= ga.job[0].mb;
  const GradJob& job = ga.job[second ? 1 : 0];
  const int64_t m0 = ((int64_t)blockIdx.x - (second ? ga.job[0].mb : 0)) * MT, ld = job.ld;
  const int njt = (ga.r + JR - 1) / JR, j0 = ((int)blockIdx.z % njt) * JR, z = (int)blockIdx.z / njt;
  int b0, b1;
  const int g = slice_of(ga, blockIdx.y, z, b0, b1);

  // a thread's share of a step: bf16 chunk tid % 32 of rows tid / 32 and tid / 32 + 16, or 16 codes
  // tid % 16 of row tid / 16.  Every load is unconditional: columns past the row read its last ones
  // (not stored), padding reads token 0 and is cleared on the way to LDS.
  const bool bf = job.act != nullptr;
  const int t0 = bf ? tid >> 5 : tid >> 4, cc = bf ? tid & 31 : tid & 15;
  const int64_t mc = min(m0 + (bf ? 8 : 16) * cc, ld - (bf ? 8 : 16));  // ld is a multiple of 8, or of 16
  const uint8_t* const col = bf ? reinterpret_cast<const uint8_t*>(job.act + mc) : reinterpret_cast<const uint8_t*>(job.codes + mc);
  const int64_t rowb = bf ? 2 * ld : ld, nblk = (ld + sra_row::kCkBlock - 1) / sra_row::kCkBlock;
  // (bf16: the exponent's load stays, one per step for either kind, and reads Act's first byte)
  const uint8_t* const ecol = bf ? reinterpret_cast<const uint8_t*>(job.act) : job.exps + mc / sra_row::kCkBlock;
  struct Act {
    u32x4 a0, a1;
    uint32_t e;         // checkpoint: the scale's exponent
    uint32_t ok0, ok1;  // all ones: the rows of a0 / a1 are no padding
  };
  struct Toks {
    int p0, p1;
  };
  auto toks = [&](int b) {
    const int32_t* p = ga.perm + (int64_t)min(b, b1 - 1) * 32;
    return Toks{p[t0], p[(t0 + 16) & 31]};
  };
  auto load_act = [&](const Toks& t, Act& s) {
    const int64_t q0 = max(t.p0, 0), q1 = max(t.p1, 0);
    s.ok0 = ~(uint32_t)(t.p0 >> 31);
    s.ok1 = bf ? ~(uint32_t)(t.p1 >> 31) : s.ok0;
    s.a0 = *reinterpret_cast<const u32x4*>(col + q0 * rowb);
    s.a1 = *reinterpret_cast<const u32x4*>(col + (bf ? q1 : q0) * rowb);  // (checkpoint: the same line again)
    s.e = ecol[bf ? 0 : q0 * nblk];
  };
  auto store_act = [&](uint8_t* buf, const Act& s) {
    u32x4 x0 = s.a0, x1 = s.a1;
    if (!bf) {
      x0 = decode8(s.a0[0], s.a0[1], s.e);
      x1 = decode8(s.a0[2], s.a0[3], s.e);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x0[k] &= s.ok0;
      x1[k] &= s.ok1;
    }
    const int r1 = bf ? t0 + 16 : t0, c0 = bf ? cc : 2 * cc, c1 = bf ? cc : 2 * cc + 1;
    *reinterpret_cast<u32x4*>(buf + t0 * (2 * MT) + ((c0 ^ act_swz<MT>(t0)) << 4)) = x0;
    *reinterpret_cast<u32x4*>(buf + r1 * (2 * MT) + ((c1 ^ act_swz<MT>(r1)) << 4)) = x1;
  };
  // V: transfer k of 16 rows of 64 bytes; rows past rp read as zeros or another part's (not stored)
  const int vtile = 3 * ga.rp * 64;
  uint32_t v_off[(NV + 7) / 8];
#pragma unroll
  for (int i = 0; i < (NV + 7) / 8; ++i) {
    const int x = 16 * (8 * i + w) + (l >> 2), c = (l & 3) ^ ((x >> 2) & 3), k = x / JR, j = j0 + x % JR;
    v_off[i] = (uint32_t)((k * ga.rp + j) * 64 + 16 * c);
  }
  auto issue_v = [&](int b) {
    const uint32_t buf = lds_offset(vlds) + (b - b0) % 3 * V_BYTES;
    const dma_rsrc_t rv = dma_rsrc(job.vt + (int64_t)min(b, b1 - 1) * 3 * ga.rp * 32, (uint32_t)vtile);
#pragma unroll
    for (int i = 0; i < (NV + 7) / 8; ++i)
      if (8 * i + 8 <= NV || 8 * i + w < NV) lds_dma(rv, buf + (8 * i + w) * 1024, v_off[i], 0);
  };
  f32x4 acc[4][MF];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int f = 0; f < MF; ++f) acc[a][f] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](const uint8_t* buf, const uint8_t* vb) {
    bf16x8 b[MF];
#pragma unroll
    for (int f = 0; f < MF; ++f) b[f] = act_frag<MT>(buf, (wm * MF + f) * 16, l16, q4);
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const int x = k * JR + 64 * wj + 16 * a + l16;
        const bf16x8 v = *reinterpret_cast<const bf16x8*>(vb + x * 64 + ((q4 ^ ((x >> 2) & 3)) << 4));
#pragma unroll
        for (int f = 0; f < MF; ++f) acc[a][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, b[f], acc[a][f], 0, 0, 0);
      }
  };

  // Step b: its Act goes from registers to LDS; its transfers have landed when at most what was issued
  // after them is outstanding (two loads of tokens, three of Act, the V transfers: what step b - 1 issues,
  // and what the first step finds issued ahead of it); one barrier, after which every wave is past step
  // b - 1's reads, so the loads of step b + 2 may go to its buffers; then it multiplies.  Loads past the
  // last block repeat it, so every step issues the same number.  (The compiler's wait for step b's Act, which
  // is older than its transfers, does not know of the transfers and so waits for at least as much.)
  Act s0, s1;
  Toks tk{0, 0};
  if (b0 < b1) {
    const Toks ta = toks(b0), tb = toks(b0 + 1);
    load_act(ta, s0);
    issue_v(b0);
    __builtin_amdgcn_sched_barrier(0);
    tk = toks(b0 + 2);  // after step b0's transfers, as in every later step
    load_act(tb, s1);
    issue_v(b0 + 1);
    __builtin_amdgcn_sched_barrier(0);
  }
  auto step = [&](int b, Act& s, uint8_t* buf) {
    store_act(buf, s);
    if (NV % 8 == 0 || w < NV % 8) wait_vm_all<2 + 3 + (NV + 7) / 8>();
    else wait_vm_all<2 + 3 + NV / 8>();
    __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));  // lgkmcnt(0): this wave's LDS writes are done
    ring_barrier();
    const Toks next = toks(b + 3);
    load_act(tk, s);
    issue_v(b + 2);
    __builtin_amdgcn_sched_barrier(0);
    tk = next;
    compute(buf, vlds + (b - b0) % 3 * V_BYTES);
  };
  int b = b0;
  for (; b + 1 < b1; b += 2) {
    step(b, s0, lds);
    step(b + 1, s1, lds + A_BYTES);
  }
  if (b < b1) step(b, s0, lds);
  wait_vm_all<0>();  // the repeated transfers land before this workgroup gives its LDS back

#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int f = 0; f < MF; ++f)
      grad_store(ga, job, g, z, j0 + 64 * wj + 16 * a, m0 + (wm * MF + f) * 16, acc[a][f], l16, q4);
}

// Rows of M columns as bf16 rows of ld >= M (ld % 8 == 0), zeros past M: for the few row lengths that the
// gradient kernels' loads do not fit.  A thread writes eight columns; T * ld / 8 of them, walked by the grid.
__global__ __launch_bounds__(256) void k_multi_pad(const uint16_t* __restrict__ act, const int8_t* __restrict__ codes,
                                                   const uint8_t* __restrict__ exps, int64_t T, int64_t M, int64_t ld,
                                                   uint16_t* __restrict__ out) {
  const int64_t per = ld / 8, nblk = (M + sra_row::kCkBlock - 1) / sra_row::kCkBlock;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < T * per; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / per, m = i % per * 8;
    union { uint16_t h[8]; u32x4 v; } o;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      o.h[k] = 0;
      if (m + k >= M) continue;
      if (act) {
        o.h[k] = act[t * M + m + k];
      } else {  // q 2^e is exact in bf16: the high half of the fp32 value
        const float s = __uint_as_float((uint32_t)exps[t * nblk + (m + k) / sra_row::kCkBlock] << 23);
        o.h[k] = (uint16_t)(__float_as_uint((float)codes[t * M + m + k] * s) >> 16);
      }
    }
    *reinterpret_cast<u32x4*>(out + t * ld + m) = o.v;
  }
}

// out[i] = sum of the S slices' partials in slice order; both jobs' outputs one after the other (5.5 us
// for the slices of U or dU at 8192 tokens, rank 128)
__global__ void k_multi_join(const float* __restrict__ part, int64_t slice, int S, int64_t n0, int64_t n1,
                             float* __restrict__ out0, float* __restrict__ out1) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n0 + n1) return;
  float s = part[i];
  for (int k = 1; k < S; ++k) s += part[(int64_t)k * slice + i];
  if (i < n0) out0[i] = s;
  else out1[i - n0] = s;
}

// ------------------------------------------------------------------------------------ rows
// Out[t][j] = sum_c act[t][c] W_g[j][c] for ranks above 32: a workgroup owns 128 tokens and JR
// adapter columns over a slice of c, in 64-column stages (whole 128-byte lines of every row; five
// stages of 32 columns took 164 us where two of 64 took 133, OPT-13B's dU at 8 slices); both operands stream
// through an LDS ring of NS stages filled by buffer -> LDS transfers.  At most 80 KB of LDS and 128
// registers, so two workgroups share a CU and one's transfers run under the other's products.
// Eight waves: four of 32 tokens by two of JR / 2 adapter columns.
// TW: the weight is given as [C][r] (B_g as it lies) and its stage [SC][JR] is read with the
// transposing LDS read; else as [r][C].
// A tile whose tokens take several adapters runs one pass per distinct adapter and writes the tokens
// of that adapter after it; the grid holds `passes` workgroups per tile (as k_adapter_rows), the last
// of them taking what the others leave.
// Bound by the transfers' latency into LDS: 36 us for U of 8192 tokens at K = 5120, rank 128, 8
// adapters in 15 requests (84 MB of X, 2.3 TB/s) and 112 us for dU at N = 20480 (336 MB of dY, 3.0
// TB/s, where a copy reaches 4.9).
template <int JR, bool TW>
__global__ __launch_bounds__(512, 4) void k_multi_rows(const uint16_t* __restrict__ act, int64_t T, int64_t C,
                                                       const uint16_t* __restrict__ wgt, int r, int64_t c_per, int S,
                                                       float* __restrict__ part, float* __restrict__ out,
                                                       sra::AdapterIds ai) {
  constexpr int SC = 64, NS = JR == 128 ? 2 : 3, D = NS - 1;
  constexpr int RB = 2 * SC, CH = SC / 8;  // bytes and 16-byte chunks of a row of a stage
  constexpr int A_BYTES = 128 * RB, G_BYTES = JR * RB, STAGE = A_BYTES + G_BYTES, JW = JR / 32;
  constexpr int LA = A_BYTES / 8192, LG = G_BYTES / 8192, L = LA + LG;  // 1 KB transfers per wave
  __shared__ __attribute__((aligned(16))) uint8_t lds[NS * STAGE];
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, q4 = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6), wt = w & 3, wj = w >> 2;
  // workgroups go to the 8 XCDs in turn: XCD x takes an eighth of the (slice, adapter column tile,
  // token tile) list in one piece, so the token tiles that read the same weight slice share its L2
  const int n_tt = (int)((T + 127) / 128), n_jt = (r + JR - 1) / JR, n_wg = n_tt * n_jt * S;
  const int my = (int)blockIdx.x / n_wg, last = ai.passes - 1;
  const int id = (int)blockIdx.x % n_wg, xcd = id & 7, per = n_wg >> 3, rem = n_wg & 7;
  const int lin = xcd * per + min(xcd, rem) + (id >> 3);
  const int64_t t0 = (int64_t)(lin % n_tt) * 128;
  const int j0 = lin / n_tt % n_jt * JR, z = lin / n_tt / n_jt;
  const int64_t cb = (int64_t)z * c_per, ce = min(C, cb + c_per);
  const int n_st = (int)((ce - cb) / SC), toks = (int)min((int64_t)128, T - t0);

  const dma_rsrc_t ra = dma_rsrc(act + t0 * C + cb, (uint32_t)((toks * C - cb) * 2));
  auto swz = [](int x) { return (x >> 1) & 7; };
  uint32_t a_off[LA], g_off[LG];
#pragma unroll
  for (int k = 0; k < LA; ++k) {  // 1024 / RB rows a transfer
    const int x = (1024 / RB) * (k * 8 + w) + lane / CH, c = (lane % CH) ^ swz(x);
    a_off[k] = (uint32_t)((x * C + c * 8) * 2);
  }
#pragma unroll
  for (int k = 0; k < LG; ++k) {
    const int b = k * 8 + w;
    if constexpr (TW) {  // rows of JR columns; columns past r lie past the buffer's end
      constexpr int GH = JR / 8;
      const int x = (64 / GH) * b + lane / GH, c = (lane % GH) ^ act_swz<JR>(x);
      g_off[k] = (uint32_t)((x * r + j0 + 8 * c) * 2) | ((uint32_t)(j0 + 8 * c >= r) << 31);
    } else {
      const int x = (1024 / RB) * b + lane / CH, c = (lane % CH) ^ swz(x);
      g_off[k] = (uint32_t)((x * C + c * 8) * 2);
    }
  }
  auto weight = [&](int g) {
    const uint16_t* w0 = wgt + (int64_t)g * r * C;
    const int64_t first = TW ? cb * r : (int64_t)j0 * C + cb, len = TW ? (C - cb) * r : (r - j0) * C - cb;
    return dma_rsrc(w0 + first, (uint32_t)(len * 2));
  };
  dma_rsrc_t rg = weight(0);

  // TW: this wave's fragments (16 adapter columns each) of a stage's [SC][JR] tile; rows t and t + 4
  // share their swizzle, and so do k steps 32 rows apart
  const uint8_t* tr_at[JW];
#pragma unroll
  for (int a = 0; a < JW; ++a) {
    const int t = 8 * q4 + (l16 >> 2), col = 16 * (JW * wj + a) + 4 * (l16 & 3);
    tr_at[a] = lds + A_BYTES + t * (2 * JR) + (((col >> 3) ^ act_swz<JR>(t)) << 4) + (col & 7) * 2;
  }

  f32x4 acc[2][JW];
  auto pass = [&] {
    auto issue = [&](int st) {
      const uint32_t base = lds_offset(lds) + (st % NS) * STAGE;
#pragma unroll
      for (int k = 0; k < LA; ++k) lds_dma(ra, base + (k * 8 + w) * 1024, a_off[k], st * RB);
#pragma unroll
      for (int k = 0; k < LG; ++k)
        lds_dma(rg, base + A_BYTES + (k * 8 + w) * 1024, g_off[k], TW ? st * RB * r : st * RB);
    };
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int a = 0; a < JW; ++a) acc[i][a] = f32x4{0.f, 0.f, 0.f, 0.f};
    __syncthreads();  // every wave is done with the previous pass's stages
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (d < n_st) issue(d);
    for (int st = 0; st < n_st; ++st) {
      // stage st has landed when at most the later stages' transfers are outstanding
      const int later = n_st - 1 - st;
      if (D > 1 && later >= D - 1) wait_vm_all<(D - 1) * L>();
      else wait_vm_all<0>();
      ring_barrier();  // every wave's part of stage st is in LDS, stage st - 1 consumed
      if (st + D < n_st) issue(st + D);
      const uint8_t* A = lds + (st % NS) * STAGE;
      const uint8_t* G = A + A_BYTES;
#pragma unroll
      for (int ks = 0; ks < SC / 32; ++ks) {
        const int k = 4 * ks + q4;
        bf16x8 af[2], gf[JW];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int x = 32 * wt + 16 * i + l16;
          af[i] = *reinterpret_cast<const bf16x8*>(A + x * RB + ((k ^ swz(x)) << 4));
        }
        if constexpr (TW) {
#pragma unroll
          for (int a = 0; a < JW; ++a) {
            TrFrag u;
#pragma unroll
            for (int h = 0; h < 2; ++h) u.h[h] = lds_tr(tr_at[a] + (st % NS) * STAGE + (32 * ks + 4 * h) * 2 * JR);
            gf[a] = u.b;
          }
        } else {
#pragma unroll
          for (int a = 0; a < JW; ++a) {
            const int x = 16 * (JW * wj + a) + l16;
            gf[a] = *reinterpret_cast<const bf16x8*>(G + x * RB + ((k ^ swz(x)) << 4));
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int a = 0; a < JW; ++a) acc[i][a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af[i], gf[a], acc[i][a], 0, 0, 0);
      }
    }
  };
  // D layout: token 32 wt + 16 i + 4 (l / 16) + e, adapter column 16 (JW wj + a) + l % 16
  float* const dst = part ? part + (int64_t)z * T * r : out;
  int idr[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = 32 * wt + 16 * i + 4 * q4 + e;
      idr[i][e] = t < toks ? ai.ids[t0 + t] : -1;
      if (my == 0 && t < toks && (idr[i][e] < 0 || idr[i][e] >= ai.n)) {  // no adapter: zeros
#pragma unroll
        for (int a = 0; a < JW; ++a) {
          const int j = j0 + 16 * (JW * wj + a) + l16;
          if (j < r) dst[(t0 + t) * r + j] = 0.f;
        }
      }
    }
  const int id0 = lane < toks ? ai.ids[t0 + lane] : -1, id1 = 64 + lane < toks ? ai.ids[t0 + 64 + lane] : -1;
  uint64_t todo0 = __ballot(id0 >= 0 && id0 < ai.n), todo1 = __ballot(id1 >= 0 && id1 < ai.n);
  for (int k = 0; todo0 | todo1; ++k) {  // the same sequence in every wave
    const int g = todo0 ? __builtin_amdgcn_readlane(id0, __builtin_ctzll(todo0))
                        : __builtin_amdgcn_readlane(id1, __builtin_ctzll(todo1));
    todo0 &= ~__ballot(id0 == g);
    todo1 &= ~__ballot(id1 == g);
    if (min(k, last) != my) continue;
    rg = weight(g);
    pass();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (idr[i][e] == g) {
          const int64_t t = t0 + 32 * wt + 16 * i + 4 * q4 + e;
#pragma unroll
          for (int a = 0; a < JW; ++a) {
            const int j = j0 + 16 * (JW * wj + a) + l16;
            if (j < r) dst[t * r + j] = acc[i][a][e];
          }
        }
  }
}

int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

namespace sra {

int multi_max_adapters() { return kMaxAdapters; }
size_t multi_groups_bytes(int n) { return (size_t)(group_list(n) + 4 * n) * 4; }
int64_t multi_perm_entries(int64_t T, int n) { return 32 * (T / 32 + std::min<int64_t>(n, T)); }

namespace {
// The 128-token tiles: ranks above 32 with at least two tiles and whole 64-column stages.  Slices of
// the reduction (at least 4 stages) for about 512 workgroups, two per CU, with one adapter, and 256
// with several, whose further passes then run beside the first ones.  Measured at OPT-13B's dU (64
// tiles, r 128), 4 / 8 / 16 slices: one adapter 104 / 90 / 113 us, 8 adapters in 15 requests 124 /
// 141 / 153 us.
struct RowsPlan {
  bool ring;
  int jr, S;
  int64_t c_per;
};
RowsPlan multi_rows_plan(int64_t T, int64_t C, int n, int r) {
  RowsPlan p{};
  p.ring = r > 32 && T >= 256 && C > 0 && C % 64 == 0 && C < ((int64_t)1 << 23);  // 32-bit offsets in 128 rows
  p.jr = r <= 64 ? 64 : 128;
  p.S = 1;
  if (!p.ring) return p;
  const int64_t tiles = cdiv64(T, 128);
  int64_t S = (n > 1 ? 256 : 512) / (tiles * cdiv64(r, p.jr));
  S = std::min<int64_t>(S, C / 256);
  S = std::max<int64_t>(S, 1);
  p.c_per = cdiv64(cdiv64(C, S), 64) * 64;
  p.S = (int)cdiv64(C, p.c_per);
  return p;
}
}  // namespace

bool multi_rows_w_t(int64_t T, int64_t C, int r) { return multi_rows_plan(T, C, 1, r).ring && r % 8 == 0; }
size_t multi_rows_ws(int64_t T, int64_t C, int n, int r) {
  const RowsPlan p = multi_rows_plan(T, C, n, r);
  if (p.ring) return p.S > 1 ? (size_t)p.S * T * r * sizeof(float) : 0;
  return multi_rows_small_ws(T, C, r);
}
hipError_t launch_multi_rows(const uint16_t* act, int64_t T, int64_t C, const uint16_t* w, bool w_t, int r,
                             const int32_t* ids, int n, float* out, void* ws, hipStream_t s) {
  if (T == 0 || r == 0) return hipSuccess;
  if (C == 0) return launch_fill_f32(out, T * r, 0.f, s);
  AdapterIds ai;
  ai.ids = ids;
  ai.stride = (int64_t)r * C;
  ai.n = n;
  const RowsPlan p = multi_rows_plan(T, C, n, r);
  if (!p.ring) return w_t ? hipErrorInvalidValue : launch_multi_rows_small(act, T, C, w, C, r, ai, out, ws, s);
  if (w_t && r % 8 != 0) return hipErrorInvalidValue;
  // eight workgroups share a tile's adapters, and up to 32 as long as the grid stays at 1024: 256 / 512 tokens
  // of 32 adapters side by side, C = N = 4096, r = 64: forward 67 / 101 us where eight took 100 / 107 (one
  // adapter: 41 / 42 and 39 / 41)
  const int64_t wgs = cdiv64(T, 128) * cdiv64(r, p.jr) * p.S;
  ai.passes = (int)std::min<int64_t>(n, std::max<int64_t>(8, std::min<int64_t>(32, 1024 / wgs)));
  // a launch has fewer than 2^32 threads (of 512 a workgroup): two column tiles of nearly 2^26 tokens leave seven
  ai.passes = (int)std::min<int64_t>(ai.passes, (((int64_t)1 << 23) - 1) / wgs);
  float* part = p.S > 1 ? (float*)ws : nullptr;
  const dim3 grid((unsigned)(cdiv64(T, 128) * cdiv64(r, p.jr) * p.S * ai.passes));
#define SRA_MR(JR, TWV) \
  launch(SRA_KERNEL_ADAPTER, k_multi_rows<JR, TWV>, grid, dim3(512), 0, s, act, T, C, w, r, p.c_per, p.S, part, out, ai)
  if (p.jr == 64) {
    if (w_t) SRA_MR(64, true);
    else SRA_MR(64, false);
  } else {
    if (w_t) SRA_MR(128, true);
    else SRA_MR(128, false);
  }
#undef SRA_MR
  if (p.S > 1)
    hipLaunchKernelGGL(k_multi_join, dim3((unsigned)cdiv64(T * r, 256)), dim3(256), 0, s, part, T * r, p.S, T * r, (int64_t)0,
                       out, (float*)nullptr);
  return hipGetLastError();
}

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
  const int lr = tile_lr(p.r), lm = 13 - lr;
  const int64_t rt = cdiv64(p.r, 1 << lr);
  a.b_tiles = p.wt ? (int)(cdiv64(p.N, 1 << lm) * rt) : 0;
  a.a_tiles = p.at ? (int)(cdiv64(p.K, 1 << lm) * rt) : 0;
  const int64_t blocks = (a.ids ? 1 : 0) + (int64_t)p.n * (a.b_tiles + a.a_tiles);
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL(k_multi_prep, dim3((unsigned)blocks), dim3(kPrepThreads), 0, s, a);
  return hipGetLastError();
}

namespace {
constexpr int kFewRank = 32;  // ranks up to this: k_multi_grads_few
struct GradPlan {
  bool few;
  int mt, wj, S, njt;
  int64_t vt, slice;  // bytes of one job's V parts, elements of one slice's partials
};
// Slices so that about 512 (few: four waves each) or 256 workgroups run, of at least 8 blocks of a
// batch spread evenly over the adapters.
GradPlan grad_plan(const MultiGrad* g, int n_jobs, int64_t T, int n, int r) {
  GradPlan p{};
  p.few = r <= kFewRank;
  p.mt = p.few ? 64 : 256;
  p.wj = r <= 64 ? 1 : 2;
  p.njt = p.few ? 1 : (int)cdiv64(r, 64 * p.wj);
  int64_t tiles = 0;
  for (int i = 0; i < n_jobs; ++i) {
    tiles += cdiv64(g[i].M, p.mt);
    p.slice += (int64_t)n * r * g[i].M;
  }
  const int64_t wg = tiles * n * p.njt;
  int64_t S = wg > 0 ? (p.few ? 512 : 256) / wg : 1;
  S = std::min<int64_t>(S, cdiv64(cdiv64(T, 32), n) / 8);
  p.S = (int)std::max<int64_t>(1, S);
  p.vt = p.few ? 0 : multi_perm_entries(T, n) * 3 * cdiv64(r, 16) * 16 * 2;
  return p;
}
}  // namespace

// 16-byte loads of bf16, 8-byte loads of codes, and above kFewRank 16-byte loads of codes
bool multi_grad_fits(int64_t row, bool ckpt, int r) { return row % (ckpt && r > kFewRank ? 16 : 8) == 0; }
int64_t multi_pad_ld(int64_t M) { return cdiv64(M, 32) * 32; }
hipError_t launch_multi_pad(const uint16_t* act, const int8_t* codes, const uint8_t* exps, int64_t T, int64_t M,
                            uint16_t* out, hipStream_t s) {
  const int64_t ld = multi_pad_ld(M);
  if (T <= 0 || M <= 0) return hipSuccess;
  const unsigned grid = (unsigned)std::min<int64_t>(cdiv64(T * (ld / 8), 256), 1 << 16);
  hipLaunchKernelGGL(k_multi_pad, dim3(grid), dim3(256), 0, s, act, codes, exps, T, M, ld, out);
  return hipGetLastError();
}

size_t multi_grads_ws(const MultiGrad* g, int n_jobs, int64_t T, int n, int r) {
  const GradPlan p = grad_plan(g, n_jobs, T, n, r);
  return (size_t)(((p.vt + 255) / 256 * 256) * n_jobs + (p.S > 1 ? p.S * p.slice * 4 : 0));
}

hipError_t launch_multi_grads(const MultiGrad* g, int n_jobs, int64_t T, const int32_t* gblk, const int32_t* perm, int n,
                              int r, void* ws, hipStream_t s) {
  if (n_jobs <= 0 || r <= 0 || n <= 0) return hipSuccess;
  for (int i = 0; i < n_jobs; ++i) {
    const int64_t ld = g[i].ld ? g[i].ld : g[i].M;
    if (ld < g[i].M || !multi_grad_fits(ld, !g[i].act, r)) return hipErrorInvalidValue;
  }
  const GradPlan p = grad_plan(g, n_jobs, T, n, r);
  GradArgs ga{};
  ga.gblk = gblk;
  ga.perm = perm;
  ga.n = n;
  ga.r = r;
  ga.rp = (int)(cdiv64(r, 16) * 16);
  ga.S = p.S;
  ga.slice = p.slice;
  uint8_t* at = (uint8_t*)ws;
  int64_t mb = 0, done = 0;
  float* part = (float*)(at + (p.vt + 255) / 256 * 256 * n_jobs);
  for (int i = 0; i < n_jobs; ++i) {
    GradJob& j = ga.job[i];
    j.act = g[i].act;
    j.codes = g[i].codes;
    j.exps = g[i].exps;
    j.V = g[i].V;
    j.vt = (uint16_t*)at;
    at += (p.vt + 255) / 256 * 256;
    j.out = p.S > 1 ? part + done : g[i].out;
    done += (int64_t)n * r * g[i].M;
    j.M = g[i].M;
    j.ld = g[i].ld ? g[i].ld : g[i].M;
    j.mb = (int)cdiv64(g[i].M, p.mt);
    j.out_t = g[i].out_t;
    mb += j.mb;
  }
  if (mb == 0) return hipSuccess;
  const dim3 grid((unsigned)mb, (unsigned)n, (unsigned)(p.njt * p.S));
  if (p.few) {
    if (r <= 16) launch(SRA_KERNEL_ADAPTER, k_multi_grads_few<1, 8>, grid, dim3(512), 0, s, ga);
    else launch(SRA_KERNEL_ADAPTER, k_multi_grads_few<2, 4>, grid, dim3(256), 0, s, ga);
  } else {
    hipLaunchKernelGGL(k_multi_vt, dim3((unsigned)(multi_perm_entries(T, n) / 32), (unsigned)n_jobs, (unsigned)cdiv64(r, 64)),
                       dim3(256), 0, s, ga);
    if (p.wj == 1) launch(SRA_KERNEL_ADAPTER, k_multi_grads<1>, grid, dim3(512), 0, s, ga);
    else launch(SRA_KERNEL_ADAPTER, k_multi_grads<2>, grid, dim3(512), 0, s, ga);
  }
  if (p.S > 1) {
    const int64_t n0 = (int64_t)n * r * g[0].M, n1 = n_jobs > 1 ? (int64_t)n * r * g[1].M : 0;
    hipLaunchKernelGGL(k_multi_join, dim3((unsigned)cdiv64(n0 + n1, 256)), dim3(256), 0, s, part, p.slice, p.S, n0, n1,
                       g[0].out, n_jobs > 1 ? g[1].out : nullptr);
  }
  return hipGetLastError();
}

}  // namespace sra
