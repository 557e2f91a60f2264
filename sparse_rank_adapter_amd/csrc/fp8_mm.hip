// Products of 8-bit floating point matrices with a power-of-two scale for each block of 128 columns
// (fp8.h): Out[m][n] = sum_k a[m][k] b[n][k], both operands reduced along their rows.
//
// The scaled matrix instruction v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 x 128 by 128 x 16 codes
// and applies one E8M0 byte per row and 32 columns; a block's byte is given for all four of its quarters.
// The sum over the whole reduction stays in its fp32 accumulators.  The order of the 128 codes inside a
// step does not matter as long as both operands use the same: a lane (row l % 16) takes 16-byte chunks
// l / 16 and l / 16 + 4 of its row's 128 bytes.
//
// Scales of four consecutive blocks are one dword of a row's exponents; the instruction's op_sel picks
// the byte, so they cost one read per row and 512 columns.
//
// The instruction first adds the products of each eight neighbouring codes, every one truncated to a multiple of 2^(E - 13), E
// the largest sum of two codes' exponents among them (codes below the smallest normal value count as that), and then these sums
// and the accumulator in fp32 (measured; the plain fp8 instructions do the same).  A block's sum is so 1e-5 to 4e-5 off for
// normally distributed values, and by 7 2^-13 of the eights' largest products at worst: less than a bf16 result's rounding
// unless large products cancel, so bf16 results accept it for the rate (8192 x 20480 over 5120: 619 us, 1826 with fp32
// results), but not less than fp32's.  fp32 results (EX) go over bf16: every code is exact in bf16, v_mfma_f32_16x16x32_bf16
// adds with full fp32 accuracy, and each block's sum enters the accumulator over its scale, an exact ldexp.
#include <algorithm>
#include <type_traits>

#include "fp8.h"

namespace {
using namespace sra_f8;

typedef int v8i __attribute__((ext_vector_type(8)));

struct Mat {
  const uint8_t* codes;
  const uint8_t* exps;
  int64_t rows, ld, nblk;  // ld = 128 nblk bytes a row
  int shift;               // log2 of the rows that share a scale (0 or 7)
};
struct Out {
  void* p;
  int64_t M, N;
  bool f32;
};

union Frag {
  u32x4 h[2];
  v8i v;
};

// s_waitcnt vmcnt(N) alone (expcnt / lgkmcnt at their maxima)
template <int N>
SRA_DEV void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// Buffer -> LDS transfers as lds_dma makes them (unseen by the compiler, which would put a wait for all of them before
// any LDS read), with scalar operands given as such: a readfirstlane of what is scalar already costs vector registers,
// and these kernels have none to spare.  base and bytes are uniform; offsets past `bytes` read zeros.
SRA_DEV dma_rsrc_t rows_rsrc(const uint8_t* base, int rows, int ld) {
  const uint64_t p = (uint64_t)(uintptr_t)base;
  return dma_rsrc_t{(int)(uint32_t)p, (int)((uint32_t)(p >> 32) & 0xffff), max(0, rows) * ld, 0x00020000};
}
SRA_DEV void dma(const dma_rsrc_t& rs, uint32_t block, uint32_t off, int soff) {
  // one wait state after M0 is written, five after a vector instruction writes a scalar register that is read here; M0 is
  // reserved and may not be in the clobber list: this file has no builtin transfer, which keeps its target there
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(block), "v"(off), "s"(rs), "s"(soff)
               : "memory");
}

// exponents of blocks kb .. kb + 3 of `row` (those past the row's end are of no use to the caller); nothing past
// the array's end is read.  `whole`: the array has four bytes at least.
SRA_DEV int64_t exps_total(const Mat& m) { return (((m.rows - 1) >> m.shift) + 1) * m.nblk; }
SRA_DEV uint32_t scales4(const Mat& m, int64_t row, int64_t kb, int64_t total, bool whole) {
  const int64_t at = (min(row, m.rows - 1) >> m.shift) * m.nblk + kb;
  uint32_t v = 0;
  if (whole) {
    const int64_t o = min(at, total - 4);
    __builtin_memcpy(&v, m.exps + o, 4);
    return v >> (8 * (int)(at - o));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v |= (uint32_t)m.exps[min(at + i, total - 1)] << (8 * i);
  return v;
}
SRA_DEV int byte_of(uint32_t w, int j) { return (int)((w >> (8 * j)) & 0xffu); }

// 32 codes as bf16, exactly: fragment s holds the 8 codes of dwords 2 s and 2 s + 1
struct Wide {
  bf16x8 s[4];
};
template <int K>
SRA_DEV Wide widen(const Frag& f) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  Wide o;
#pragma unroll
  for (int d = 0; d < 8; ++d) {
    bf16x2 lo, hi;
    if constexpr (K == SRA_FP8_E4M3) {
      lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)f.v[d], 1.f, false);
      hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)f.v[d], 1.f, true);
    } else {
      lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((uint32_t)f.v[d], 1.f, false);
      hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((uint32_t)f.v[d], 1.f, true);
    }
    o.s[d / 2][4 * (d % 2)] = lo[0];
    o.s[d / 2][4 * (d % 2) + 1] = lo[1];
    o.s[d / 2][4 * (d % 2) + 2] = hi[0];
    o.s[d / 2][4 * (d % 2) + 3] = hi[1];
  }
  return o;
}
SRA_DEV f32x4 mfma_wide(const Wide& x, const Wide& y) {
  f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x.s[s], y.s[s], c, 0, 0, 0);
  return c;
}

// j (a constant once unrolled): which byte of the scale dwords
template <int KX, int KY>
SRA_DEV f32x4 mfma(const Frag& x, const Frag& y, f32x4 c, uint32_t sx, uint32_t sy, int j) {
  if (j == 0) return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x.v, y.v, c, KX, KY, 0, (int)sx, 0, (int)sy);
  if (j == 1) return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x.v, y.v, c, KX, KY, 1, (int)sx, 1, (int)sy);
  if (j == 2) return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x.v, y.v, c, KX, KY, 2, (int)sx, 2, (int)sy);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x.v, y.v, c, KX, KY, 3, (int)sx, 3, (int)sy);
}

SRA_DEV void store_out(const Out& o, int64_t m, int64_t n, float v) {
  if (o.f32) reinterpret_cast<float*>(o.p)[m * o.N + n] = v;
  else {
    float one[1] = {v};
    sra_row::RowVec<uint16_t, 1>::store(reinterpret_cast<uint16_t*>(o.p) + m * o.N + n, one);
  }
}

// ---- few rows of a (up to 16 MT): b streams once from memory into registers.
// A workgroup owns 16 RT rows of b; its waves take groups of four blocks of the reduction in turn, so that together they
// read on along the rows, and join in LDS.  a comes from the caches: RT row tiles share what a wave loads of it.
// 16 x 36864 over 9216: 69 us for 340 MB (4.9 TB/s; a copy reaches 5.1).
template <int KA, int KB, int MT, int RT, int NW, bool EX>
__global__ __launch_bounds__(64 * NW) void k_fp8_few(Mat a, Mat b, Out out) {
  __shared__ float red[NW][RT * MT * 256];
  const int l = threadIdx.x & 63, w = threadIdx.x >> 6, q = l >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * RT);
  const uint8_t *bp[RT], *ap[MT];
#pragma unroll
  for (int r = 0; r < RT; ++r) bp[r] = b.codes + min(n0 + 16 * r + (l & 15), b.rows - 1) * b.ld + 16 * q;
#pragma unroll
  for (int f = 0; f < MT; ++f) ap[f] = a.codes + min((int64_t)(16 * f + (l & 15)), a.rows - 1) * a.ld + 16 * q;
  f32x4 acc[RT][MT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int f = 0; f < MT; ++f) acc[r][f] = f32x4{0.f, 0.f, 0.f, 0.f};
  uint32_t poison = 0;  // EX: scales of 255 met, bit 4 r + v for row 16 r + 4 q + v of b, bit 4 RT + f for a's
  const int64_t ta = exps_total(a), tb = exps_total(b);
  const bool whole = ta >= 4 && tb >= 4;
  constexpr int SB = EX ? 4 : 1;  // b's rows whose scales a lane holds: those of its results, or that of its operand
  for (int64_t kb = 4 * w; kb < b.nblk; kb += 4 * NW) {
    Frag fb[4][RT], fa[4][MT];
    uint32_t sa[MT], sb[RT][SB];
    const int left = (int)min(b.nblk - kb, (int64_t)4);
    const auto scales = [&](bool ok) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int v = 0; v < SB; ++v) sb[r][v] = scales4(b, n0 + 16 * r + (EX ? 4 * q + v : l & 15), kb, tb, ok);
#pragma unroll
      for (int f = 0; f < MT; ++f) sa[f] = scales4(a, 16 * f + (l & 15), kb, ta, ok);
    };
    if (whole) scales(true);
    else scales(false);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t at = (kb + min(j, left - 1)) * kBlock;  // past the row's end: a block that is read anyway
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        fb[j][r].h[0] = *reinterpret_cast<const u32x4*>(bp[r] + at);
        fb[j][r].h[1] = *reinterpret_cast<const u32x4*>(bp[r] + at + 64);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t at = (kb + min(j, left - 1)) * kBlock;
#pragma unroll
      for (int f = 0; f < MT; ++f) {
        fa[j][f].h[0] = *reinterpret_cast<const u32x4*>(ap[f] + at);
        fa[j][f].h[1] = *reinterpret_cast<const u32x4*>(ap[f] + at + 64);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= left) continue;
      if constexpr (!EX) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int f = 0; f < MT; ++f) acc[r][f] = mfma<KB, KA>(fb[j][r], fa[j][f], acc[r][f], sb[r][0], sa[f], j);
      } else {
#pragma unroll
        for (int f = 0; f < MT; ++f) poison |= byte_of(sa[f], j) == 255 ? 1u << (4 * RT + f) : 0u;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const Wide wb = widen<KB>(fb[j][r]);
#pragma unroll
          for (int v = 0; v < 4; ++v) poison |= byte_of(sb[r][v], j) == 255 ? 1u << (4 * r + v) : 0u;
#pragma unroll
          for (int f = 0; f < MT; ++f) {
            const f32x4 p = mfma_wide(wb, widen<KA>(fa[j][f]));
#pragma unroll
            for (int v = 0; v < 4; ++v)
              acc[r][f][v] += __builtin_amdgcn_ldexpf(p[v], byte_of(sb[r][v], j) + byte_of(sa[f], j) - 254);
          }
        }
      }
    }
  }
  // acc[r][f][v]: row 16 f + l % 16 of a, row n0 + 16 r + 4 q + v of b
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int f = 0; f < MT; ++f)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        if (EX && (poison & (1u << (4 * r + v) | 1u << (4 * RT + f)))) acc[r][f][v] = __uint_as_float(0x7fc00000u);
        red[w][(16 * f + (l & 15)) * (16 * RT) + 16 * r + 4 * q + v] = acc[r][f][v];
      }
  __syncthreads();
  for (int i = threadIdx.x; i < RT * MT * 256; i += 64 * NW) {
    float s = red[0][i];
#pragma unroll
    for (int k = 1; k < NW; ++k) s += red[k][i];
    const int64_t m = i / (16 * RT), n = n0 + i % (16 * RT);
    if (m < out.M && n < out.N) store_out(out, m, n, s);
  }
}

// ---- tiles of BM x BN, WM x WN waves, a ring of ST = 2 or 4 stages of 128 columns in LDS.
// Rows are 128 bytes; chunk c of row i lies at (c ^ key(i)), key = i % 8 for a and (i / FN) % 8 for b, whose
// fragments take rows FN (l % 16) + g, so that a lane's FN accumulators are neighbouring columns of Out.
template <int BM, int BN, int WM, int WN, int ST>
struct Cfg {
  static constexpr int NW = WM * WN, FM = BM / WM / 16, FN = BN / WN / 16;
  static constexpr int stage = (BM + BN) * kBlock;
  static constexpr int DA = BM / 8 / NW, DB = BN / 8 / NW;  // transfers of a wave per stage
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "whole transfers");
  static_assert(ST == 2 || ST == 4, "slots by the step modulo four");
  static constexpr int bytes = ST * stage;
};

// Workgroup ids go round-robin over the 8 XCDs: give each XCD a contiguous range of tiles, and order the
// tiles in groups of 8 row tiles so that the workgroups of one XCD share operands in its L2.
SRA_DEV void tile_of(int bid, int n, int nm, int nn, int& tm, int& tn) {
  const int full = n & ~7;
  const int t = bid >= full ? bid : (bid & 7) * (full >> 3) + (bid >> 3);
  constexpr int G = 8;
  const int per = G * nn, g = t / per, gs = min(G, nm - g * G), in = t - g * per;
  tm = g * G + in % gs;
  tn = in / gs;
}

// acc[g][v]: row m0 + 4 q + v, column n0 + FN (l % 16) + g of Out, or of this split's fp32 partial product
template <int FN, bool F32>
SRA_DEV void store_row16(const f32x4 (&acc)[FN], void* o, const Out& out, int64_t m0, int64_t n0) {
  static_assert(FN % 4 == 0, "stores of four columns");
  const int l = threadIdx.x & 63, q = l >> 4, i16 = l & 15;
  const int64_t n = n0 + FN * i16;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int64_t m = m0 + 4 * q + v, at = m * out.N + n;
    const int have = m < out.M ? (int)min(max(out.N - n, (int64_t)0), (int64_t)FN) : 0;  // columns inside
    if constexpr (F32) {
      float* const p = (float*)o + at;
      if (have == FN && out.N % 4 == 0) {
#pragma unroll
        for (int g = 0; g < FN; g += 4)
          *reinterpret_cast<f32x4*>(p + g) = f32x4{acc[g][v], acc[g + 1][v], acc[g + 2][v], acc[g + 3][v]};
      } else {
#pragma unroll
        for (int g = 0; g < FN; ++g)
          if (g < have) p[g] = acc[g][v];
      }
    } else {
      union { __bf16 h[FN]; uint16_t e[FN]; u32x2 w[FN / 4]; u32x4 x[(FN + 7) / 8]; } c;
#pragma unroll
      for (int g = 0; g < FN; ++g) c.h[g] = (__bf16)acc[g][v];
      uint16_t* const p = (uint16_t*)o + at;
      if (have == FN && out.N % FN == 0) {
        if constexpr (FN == 8) __builtin_nontemporal_store(c.x[0], reinterpret_cast<u32x4*>(p));
        else *reinterpret_cast<u32x2*>(p) = c.w[0];
      } else {
#pragma unroll
        for (int g = 0; g < FN; ++g)
          if (g < have) p[g] = c.e[g];
      }
    }
  }
}
template <int FM, int FN>
SRA_DEV void store_tile(const f32x4 (&acc)[FM][FN], const Out& out, float* part, int64_t m0, int64_t n0) {
  if (part || out.f32) {
    void* const o = part ? part + (int64_t)blockIdx.y * out.M * out.N : out.p;
#pragma unroll
    for (int f = 0; f < FM; ++f) store_row16<FN, true>(acc[f], o, out, m0 + 16 * f, n0);
  } else {
#pragma unroll
    for (int f = 0; f < FM; ++f) store_row16<FN, false>(acc[f], out.p, out, m0 + 16 * f, n0);
  }
}

// Scales of a tile's rows, 16 blocks at a time: thread t keeps row t (a's BM rows, then b's BN)
struct ScaleRow {
  const uint8_t* p;  // the row's first byte of this reduction
  int n, left;       // its blocks; bytes from p to the array's end, where that is less than 2^30
  SRA_DEV ScaleRow(const Mat& m, int64_t row, int64_t k0, int n_kb) {
    const int64_t at = (min(row, m.rows - 1) >> m.shift) * m.nblk + k0;
    p = m.exps + at;
    n = n_kb;
    left = (int)min(exps_total(m) - at, (int64_t)1 << 30);
  }
  SRA_DEV u32x4 load(int chunk) const {  // 127 (a scale of one) past the reduction's end
    const int o = 16 * chunk;
    u32x4 v;
    if (o + 16 <= left) {
      __builtin_memcpy(&v, p + o, 16);
    } else {  // the array's last bytes
      v = u32x4{0, 0, 0, 0};
#pragma unroll 1
      for (int i = 0; i < 16 && o + i < left; ++i) {
        const uint32_t e = (uint32_t)p[o + i] << (8 * (i % 4));
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] |= i / 4 == k ? e : 0u;
      }
    }
    if (o + 16 > n) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int keep = min(max(n - o - 4 * k, 0), 4);  // bytes of this dword inside the reduction
        const uint32_t mask = keep == 4 ? ~0u : (1u << (8 * keep)) - 1u;
        v[k] = (v[k] & mask) | (0x7f7f7f7fu & ~mask);
      }
    }
    return v;
  }
};
constexpr int kScaleLd = 20;  // bytes between rows of a chunk in LDS: 16 rows fall on different banks

// (128 x 128 with four stages: 138 KB of LDS, one workgroup a CU.  The bound of two only keeps its registers to 256 a wave; the
// compiler says that it is not met.)
template <int KA, int KB, int BM, int BN, int WM, int WN, int ST, bool EX>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_fp8_tiles(Mat a, Mat b, Out out, int nm, int nn, float* part) {
  using C = Cfg<BM, BN, WM, WN, ST>;
  constexpr int FM = C::FM, FN = C::FN, DA = C::DA, DB = C::DB;
  __shared__ __align__(1024) uint8_t smem[C::bytes];
  __shared__ __align__(16) uint8_t scal[2][(BM + BN) * kScaleLd];
  const int l = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), q = l >> 4, i16 = l & 15;
  int tm, tn;
  tile_of(blockIdx.x, nm * nn, nm, nn, tm, tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int wm = (w / WN) * (BM / WM), wn = (w % WN) * (BN / WN);
  // this split's blocks of the reduction
  const int64_t k0 = a.nblk * blockIdx.y / gridDim.y, k1 = a.nblk * (blockIdx.y + 1) / gridDim.y;
  const int n_kb = (int)(k1 - k0);
  // A wave's transfer d of an operand fills 8 rows from 8 (w D + d) on; rows past the resource's end (the matrix's) read
  // zeros.  The transfers are issued unseen by the compiler, which would wait for all of them before any LDS read.
  const int ld = (int)a.ld;
  const int left_a = (int)min((int64_t)BM, a.rows - m0) - 8 * w * DA, left_b = (int)min((int64_t)BN, b.rows - n0) - 8 * w * DB;
  const uint8_t *const ga = a.codes + (m0 + 8 * w * DA) * a.ld, *const gb = b.codes + (n0 + 8 * w * DB) * b.ld;
  const uint32_t va = (uint32_t)((l >> 3) * ld) + 16 * ((l & 7) ^ (l >> 3));
  uint32_t vb[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) vb[d] = (uint32_t)((l >> 3) * ld) + 16 * ((l & 7) ^ (((8 * (w * DB + d) + (l >> 3)) / FN) & 7));
  auto issue = [&](int kb, int slot) {
    const uint32_t st = lds_offset(smem) + slot * C::stage;
    const int so = (int)((k0 + kb) * kBlock);
#pragma unroll
    for (int d = 0; d < DA; ++d)
      dma(rows_rsrc(ga + (int64_t)(8 * d) * ld, left_a - 8 * d, ld), st + 1024 * (w * DA + d), va, so);
#pragma unroll
    for (int d = 0; d < DB; ++d)
      dma(rows_rsrc(gb + (int64_t)(8 * d) * ld, left_b - 8 * d, ld), st + BM * kBlock + 1024 * (w * DB + d), vb[d], so);
  };
  const int t = threadIdx.x;
  const bool has_row = t < BM + BN;
  const ScaleRow sr(t < BM ? a : b, t < BM ? m0 + t : n0 + t - BM, k0, n_kb);
  u32x4 sreg = {0, 0, 0, 0};
  auto put_scales = [&](int chunk) {  // sreg, loaded before, into the chunk's half
    if (has_row) {
      uint32_t* const p = reinterpret_cast<uint32_t*>(scal[chunk & 1] + t * kScaleLd);
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = sreg[i];
    }
  };
  f32x4 acc[FM][FN];
#pragma unroll
  for (int f = 0; f < FM; ++f)
#pragma unroll
    for (int g = 0; g < FN; ++g) acc[f][g] = f32x4{0.f, 0.f, 0.f, 0.f};
  uint32_t poison = 0;            // EX: scales of 255 met, bit 4 f + v for a's row of acc[..][v], bit 4 FM + g for b's
  constexpr int SA = EX ? 4 : 1;  // a's rows per fragment whose scales a lane holds: its results', or its operand's
  uint32_t sa[FM][SA], sb[FN];
  // a lane's chunks of its first row of each operand; its other rows lie at fixed distances with the same key
  const uint8_t* const pa0 = smem + (wm + i16) * kBlock + 16 * (q ^ (i16 & 7));
  const uint8_t* const pa1 = smem + (wm + i16) * kBlock + 16 * ((q + 4) ^ (i16 & 7));
  const uint8_t* const pb0 = smem + (BM + wn + FN * i16) * kBlock + 16 * (q ^ (i16 & 7));
  const uint8_t* const pb1 = smem + (BM + wn + FN * i16) * kBlock + 16 * ((q + 4) ^ (i16 & 7));
  auto step = [&](int kb, int j) {  // kb % 4 == j, so the ring's slots are constants
    if (ST == 4 && kb + 2 < n_kb) wait_vm<2 * (DA + DB)>();  // the newer stages may still be in flight
    else if (ST == 4 && kb + 1 < n_kb) wait_vm<DA + DB>();
    else wait_vm<0>();
    ring_barrier();  // the stage is there for every wave, and every wave has read the one before it
    if (kb + ST - 1 < n_kb) issue(kb + ST - 1, (j + ST - 1) % ST);
    const int st = j % ST * C::stage;
    if (j == 0) {
      const uint8_t* const sc = scal[(kb >> 4) & 1] + (kb & 12);
#pragma unroll
      for (int f = 0; f < FM; ++f)
#pragma unroll
        for (int v = 0; v < SA; ++v)
          sa[f][v] = *reinterpret_cast<const uint32_t*>(sc + (wm + 16 * f + (EX ? 4 * q + v : i16)) * kScaleLd);
#pragma unroll
      for (int g = 0; g < FN; ++g) sb[g] = *reinterpret_cast<const uint32_t*>(sc + (BM + wn + FN * i16 + g) * kScaleLd);
    }
    Frag fb[FN];
#pragma unroll
    for (int g = 0; g < FN; ++g) {
      fb[g].h[0] = *reinterpret_cast<const u32x4*>(pb0 + st + g * kBlock);
      fb[g].h[1] = *reinterpret_cast<const u32x4*>(pb1 + st + g * kBlock);
    }
    Wide wb[EX ? FN : 1];
    if constexpr (EX) {
#pragma unroll
      for (int g = 0; g < FN; ++g) {
        wb[g] = widen<KB>(fb[g]);
        poison |= byte_of(sb[g], j) == 255 ? 1u << (4 * FM + g) : 0u;
      }
    }
#pragma unroll
    for (int f = 0; f < FM; ++f) {
      Frag fa;
      fa.h[0] = *reinterpret_cast<const u32x4*>(pa0 + st + 16 * f * kBlock);
      fa.h[1] = *reinterpret_cast<const u32x4*>(pa1 + st + 16 * f * kBlock);
      if constexpr (!EX) {
#pragma unroll
        for (int g = 0; g < FN; ++g) acc[f][g] = mfma<KA, KB>(fa, fb[g], acc[f][g], sa[f][0], sb[g], j);
      } else {
        const Wide wa = widen<KA>(fa);
#pragma unroll
        for (int v = 0; v < 4; ++v) poison |= byte_of(sa[f][v], j) == 255 ? 1u << (4 * f + v) : 0u;
#pragma unroll
        for (int g = 0; g < FN; ++g) {
          const f32x4 p = mfma_wide(wa, wb[g]);
#pragma unroll
          for (int v = 0; v < 4; ++v)
            acc[f][g][v] += __builtin_amdgcn_ldexpf(p[v], byte_of(sa[f][v], j) + byte_of(sb[g], j) - 254);
        }
      }
    }
  };
  if (n_kb > 0) {
    if (has_row) sreg = sr.load(0);
    put_scales(0);
    if (has_row && n_kb > 16) sreg = sr.load(1);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ST - 1; ++i)
      if (i < n_kb) issue(i, i);
  }
  for (int kb = 0; kb < n_kb; kb += 4) {
    if ((kb & 15) == 8 && (kb | 15) + 1 < n_kb) {  // the next chunk's half was last read before this chunk began
      put_scales((kb >> 4) + 1);
      if (has_row && (kb | 15) + 17 < n_kb) sreg = sr.load((kb >> 4) + 2);
      __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): written before the barriers that follow
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (kb + j < n_kb) step(kb + j, j);
  }
  if constexpr (EX) {
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
      for (int g = 0; g < FN; ++g)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (poison & (1u << (4 * f + v) | 1u << (4 * FM + g))) acc[f][g][v] = __uint_as_float(0x7fc00000u);
  }
  store_tile<FM, FN>(acc, out, part, m0 + wm, n0 + wn);
}

// 8192 x 20480 over 5120 with scales of 128 x 128 blocks: 600-672 us by box, 2.6-2.9 PFLOP/s (a library product with one scale a
// matrix 553 where this took 622); the matrix units are then busy 60% of the time at 2.1 GHz, the clock that power allows.
//
// ---- 256 x 256 tiles, four waves of 128 x 128, one to a SIMD: half the LDS traffic of eight waves of 128 x 64 (per 128
// columns 128 KB read and 64 KB written, 1536 cycles of 128 bytes, beside 2048 cycles of matrix instructions).  A step's
// 64 matrix instructions run in four quarters of 16; the operands of a quarter are read from LDS during the one before
// it, so the matrix unit does not wait for LDS:
//   a_lo b_lo (reads b_hi) | a_lo b_hi (reads a_hi) | barrier | a_hi b_lo (reads the next a_lo) | a_hi b_hi (the next b_lo)
// At the barrier in the middle of step k stage k has been read by every wave and stage k + 1 is there; stage k + 2 then
// goes into stage k's slot.  Rows are 128 bytes with chunk c at c ^ (position / 2 % 8), which spreads 16 rows over 64
// banks; b's row 8 i + g of a wave's 128 lies at position 16 g + i, so a lane's 8 columns are neighbours in Out.
//
// The accumulators fill the 256 accumulation registers; left to itself the compiler keeps operands there too and spills
// (186 registers), so the instruction is written out with its operands' classes.  It then does not know the
// instruction's latency: every read of a result has 62 others between, or the wait at the end.  The other operands come from
// LDS, whose waits the compiler does put in.
// 32 wait states behind the last matrix instructions of a group of steps, in the loop's own block, since the compiler may copy
// accumulators as soon as the loop is left.  The last ones pass through; the others were written 8 instructions, 64 wait
// states, earlier.  (A test looks for reads in the assembly that come too early.)
SRA_DEV void results_settle(f32x4 (&x)[8], f32x4 (&y)[8]) {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 15\n\ts_nop 15"
               : "+a"(x[4]), "+a"(x[5]), "+a"(x[6]), "+a"(x[7]), "+a"(y[4]), "+a"(y[5]), "+a"(y[6]), "+a"(y[7])::"memory");
  __builtin_amdgcn_sched_barrier(0);
}
#define SRA_MFMA_TEXT(C, X, Y, SX, SY, LO, HI) \
  "v_mfma_scale_f32_16x16x128_f8f6f4 " C ", " X ", " Y ", " C ", " SX ", " SY " op_sel:[" LO "," LO ",0] op_sel_hi:[" HI "," HI ",0] cbsz:%8 blgp:%9"
// two matrix instructions on one fragment of a and two of b
template <int KA, int KB>
SRA_DEV void mfma_pair(const Frag& x, const Frag& y0, const Frag& y1, f32x4& c0, f32x4& c1, uint32_t sx, uint32_t sy0,
                       uint32_t sy1, int j) {
#define SRA_PAIR(LO, HI)                                                                                            \
  asm(SRA_MFMA_TEXT("%0", "%2", "%3", "%5", "%6", LO, HI) "\n\t" SRA_MFMA_TEXT("%1", "%2", "%4", "%5", "%7", LO, HI) \
      : "+a"(c0), "+a"(c1)                                                                                          \
      : "v"(x.v), "v"(y0.v), "v"(y1.v), "v"(sx), "v"(sy0), "v"(sy1), "n"(KA), "n"(KB))
  if (j == 0) SRA_PAIR("0", "0");
  else if (j == 1) SRA_PAIR("1", "0");
  else if (j == 2) SRA_PAIR("0", "1");
  else SRA_PAIR("1", "1");
#undef SRA_PAIR
}
// The same with a transfer behind them, M0 set in front: the second instruction starts 8 wait states after the first, which
// covers what M0 and scalar registers written by vector instructions need before the transfer reads them.
template <int KA, int KB>
SRA_DEV void mfma_pair_dma(const Frag& x, const Frag& y0, const Frag& y1, f32x4& c0, f32x4& c1, uint32_t sx, uint32_t sy0,
                           uint32_t sy1, int j, const dma_rsrc_t& rs, uint32_t block, int more, uint32_t off, int soff) {
#define SRA_PAIR(LO, HI)                                                                                               \
  asm volatile("s_add_u32 m0, %10, %11\n\t" SRA_MFMA_TEXT("%0", "%2", "%3", "%5", "%6", LO, HI) "\n\t"                 \
               SRA_MFMA_TEXT("%1", "%2", "%4", "%5", "%7", LO, HI) "\n\tbuffer_load_dwordx4 %12, %13, %14 offen lds"   \
               : "+a"(c0), "+a"(c1)                                                                                    \
               : "v"(x.v), "v"(y0.v), "v"(y1.v), "v"(sx), "v"(sy0), "v"(sy1), "n"(KA), "n"(KB), "s"(block), "i"(more), \
                 "v"(off), "s"(rs), "s"(soff)                                                                          \
               : "memory", "scc")
  if (j == 0) SRA_PAIR("0", "0");
  else if (j == 1) SRA_PAIR("1", "0");
  else if (j == 2) SRA_PAIR("0", "1");
  else SRA_PAIR("1", "1");
#undef SRA_PAIR
}
#undef SRA_MFMA_TEXT
template <int KA, int KB>
__global__ __launch_bounds__(256, 1) void k_fp8_big(Mat a, Mat b, Out out, int nm, int nn) {
  constexpr int BM = 256, BN = 256, F = 8, D = 8;  // fragments a side, transfers of each operand per wave and stage
  constexpr int kSlot = BM * kBlock;               // a's two slots, then b's: all reads within 64 KB of a base
  __shared__ __align__(1024) uint8_t smem[4 * kSlot];
  __shared__ __align__(16) uint8_t scal[2][(BM + BN) * kScaleLd];
  const int t = threadIdx.x, l = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6), q = l >> 4, i16 = l & 15;
  const int wm = (w >> 1) * 128, wn = (w & 1) * 128;
  const int n_kb = (int)a.nblk, n_steps = (n_kb + 3) & ~3, n_chunks = (n_steps + 15) >> 4, ld = (int)a.ld;
  const int tiles = nm * nn;
  struct Tile {
    int64_t m0, n0;
    const uint8_t *ga, *gb;
    int left_a, left_b;  // rows of the operands that are there; none past the last tile
  };
  auto tile_at = [&](int id) {
    int tm, tn;
    tile_of(min(id, tiles - 1), tiles, nm, nn, tm, tn);
    Tile x;
    x.m0 = (int64_t)tm * BM, x.n0 = (int64_t)tn * BN;
    x.ga = a.codes + x.m0 * a.ld, x.gb = b.codes + x.n0 * b.ld;
    x.left_a = id < tiles ? (int)min((int64_t)BM, a.rows - x.m0) : 0;
    x.left_b = id < tiles ? (int)min((int64_t)BN, b.rows - x.n0) : 0;
    return x;
  };
  Tile cur = tile_at(blockIdx.x), nxt = tile_at(blockIdx.x + gridDim.x);
  uint32_t va[D], vb[D];  // rows past the end lie past the resource's size: they read zeros
#pragma unroll
  for (int d = 0; d < D; ++d) {
    const int pos = 64 * w + 8 * d + (l >> 3), chunk = 16 * ((l & 7) ^ ((pos >> 1) & 7));
    va[d] = (uint32_t)(pos * ld) + chunk;
    vb[d] = (uint32_t)(((pos & 128) + 8 * (pos & 15) + ((pos >> 4) & 7)) * ld) + chunk;
  }
  const uint32_t lds = lds_offset(smem) + 64 * kBlock * w;
  // where step s comes from: zeros from the reduction's end to the group's, then the next tile's first two stages (the
  // reduction has two blocks at least)
  struct Source {
    dma_rsrc_t a, b;
    int off;
  };
  auto source = [&](int s) {
    const bool on = s >= n_steps;
    Source x;
    x.a = rows_rsrc(on ? nxt.ga : cur.ga, on ? nxt.left_a : s < n_kb ? cur.left_a : 0, ld);
    x.b = rows_rsrc(on ? nxt.gb : cur.gb, on ? nxt.left_b : s < n_kb ? cur.left_b : 0, ld);
    x.off = (on ? s - n_steps : s) * kBlock;
    return x;
  };
  auto fill_a = [&](const Source& x, int slot, int d) { dma(x.a, lds + slot * kSlot + 1024 * d, va[d], x.off); };
  auto fill_b = [&](const Source& x, int slot, int d) { dma(x.b, lds + (2 + slot) * kSlot + 1024 * d, vb[d], x.off); };
  u32x4 ca, cb;
  auto load_scales = [&](const Tile& x, int chunk) {
    ca = ScaleRow(a, x.m0 + t, 0, n_kb).load(chunk);
    cb = ScaleRow(b, x.n0 + t, 0, n_kb).load(chunk);
  };
  auto put_scales = [&](int half) {
    uint32_t* const p = reinterpret_cast<uint32_t*>(scal[half] + t * kScaleLd);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i] = ca[i];
      p[BM * kScaleLd / 4 + i] = cb[i];
    }
  };
  const int key = (i16 >> 1) & 7, other = (q ^ key) & 4 ? -64 : 64;  // from chunk q ^ key to chunk (q + 4) ^ key
  const uint8_t* const pa = smem + (wm + i16) * kBlock + 16 * (q ^ key);
  const uint8_t* const pb = smem + 2 * kSlot + (wn + i16) * kBlock + 16 * (q ^ key);
  Frag fa[F], fb[F];
  auto read_a = [&](int slot, int f) {
#pragma unroll
    for (int h = 0; h < 2; ++h) fa[f].h[h] = *reinterpret_cast<const u32x4*>(pa + h * other + slot * kSlot + 16 * f * kBlock);
  };
  auto read_b = [&](int slot, int g) {
#pragma unroll
    for (int h = 0; h < 2; ++h) fb[g].h[h] = *reinterpret_cast<const u32x4*>(pb + h * other + slot * kSlot + 16 * g * kBlock);
  };
  uint32_t sa[F], sb[F];
  auto read_scales = [&](int half, int kb) {
    const uint8_t* const sc = scal[half] + (kb & 12);
#pragma unroll
    for (int f = 0; f < F; ++f) {
      sa[f] = *reinterpret_cast<const uint32_t*>(sc + (wm + 16 * f + i16) * kScaleLd);
      sb[f] = *reinterpret_cast<const uint32_t*>(sc + (BM + wn + 8 * i16 + f) * kScaleLd);
    }
  };
  f32x4 acc[F][F];
  // 16 matrix instructions on fragments f0 .. and g0 .., and after each two of them more(x), x = 0 .. 7
  auto quarter = [&](int f0, int g0, int j, auto more) {
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int f = f0 + x / 2, g = g0 + 2 * (x % 2);
      mfma_pair<KA, KB>(fa[f], fb[g], fb[g + 1], acc[f][g], acc[f][g + 1], sa[f], sb[g], sb[g + 1], j);
      more(x);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // the same with one transfer of a stage behind each two: of a's (part 0) or b's (part 2)
  auto quarter_fill = [&](int f0, int g0, int j, const Source& from, int part, int slot, auto more) {
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int f = f0 + x / 2, g = g0 + 2 * (x % 2);
      if (part == 0)
        mfma_pair_dma<KA, KB>(fa[f], fb[g], fb[g + 1], acc[f][g], acc[f][g + 1], sa[f], sb[g], sb[g + 1], j, from.a, lds,
                              slot * kSlot + 1024 * x, va[x], from.off);
      else
        mfma_pair_dma<KA, KB>(fa[f], fb[g], fb[g + 1], acc[f][g], acc[f][g + 1], sa[f], sb[g], sb[g + 1], j, from.b, lds,
                              (2 + slot) * kSlot + 1024 * x, vb[x], from.off);
      more(x);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  int half = 0;  // where the current chunk of scales lies
  load_scales(cur, 0);
  put_scales(0);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const Source from = source(s);
#pragma unroll
    for (int d = 0; d < D; ++d) fill_a(from, s, d);
#pragma unroll
    for (int d = 0; d < D; ++d) fill_b(from, s, d);
  }
  __builtin_amdgcn_s_waitcnt(0xc07f);
  wait_vm<2 * D>();
  ring_barrier();
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    read_a(0, x);
    read_b(0, x);
  }
#pragma unroll
  for (int f = 0; f < F; ++f)
#pragma unroll
    for (int g = 0; g < F; ++g) acc[f][g] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int id = blockIdx.x; id < tiles; id += gridDim.x) {
    // whole groups of four steps: stages past the reduction's end are zeros, under scales of one
    for (int kb = 0; kb < n_steps; kb += 4) {
      // the next chunk of scales (this tile's, or the next tile's first) is fetched in a chunk's first group and put down
      // in its last; its half was last read before this chunk began
      const bool first = (kb & 15) == 0, last = (kb & 15) == 12 || kb + 4 == n_steps;
      if (first) {
        const int c = (kb >> 4) + 1;
        if (c < n_chunks) load_scales(cur, c);
        else load_scales(nxt, 0);
      }
      if (last) put_scales(half ^ 1);
      read_scales(half, kb);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int slot = j % 2;
        const Source from = source(kb + j + 2);
        // a quarter's reads go out in its first half, so that they are back before the next begins
        quarter(0, 0, j, [&](int x) {
          if (x < 4) read_b(slot, 4 + x);
        });
        quarter(0, 4, j, [&](int x) {
          if (x < 4) read_a(slot, 4 + x);
        });
        __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
        wait_vm<0>();
        ring_barrier();
        quarter_fill(4, 0, j, from, 0, slot, [&](int x) {
          if (x < 4) read_a(1 - slot, x);
        });
        quarter_fill(4, 4, j, from, 2, slot, [&](int x) {
          if (x < 4) read_b(1 - slot, x);
        });
      }
      results_settle(acc[6], acc[7]);
      if (last) half ^= 1;
    }
#pragma unroll
    for (int f = 0; f < F; ++f) {
      store_row16<F, false>(acc[f], out.p, out, cur.m0 + wm + 16 * f, cur.n0 + wn);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int g = 0; g < F; ++g) acc[f][g] = f32x4{0.f, 0.f, 0.f, 0.f};
      __builtin_amdgcn_sched_barrier(0);
    }
    cur = nxt;
    nxt = tile_at(id + 2 * gridDim.x);
  }
  wait_vm<0>();  // no transfer may be under way when the workgroup's LDS is given up
}

// sum of the splits' partial products, in order
__global__ __launch_bounds__(256) void k_fp8_join(const float* __restrict__ part, int S, Out out) {
  const int64_t n = out.M * out.N, step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += step) {
    float s = part[i];
    for (int k = 1; k < S; ++k) s += part[k * n + i];
    store_out(out, 0, i, s);
  }
}

// ---- the choice of kernel
// Row tiles of b per workgroup with few rows of a.  More of them share a's loads, fewer spread better over the 256 CUs: the
// estimate is the tiles of the busiest CU, a quarter more where a workgroup has a single one.  9216 x 36864 by 16 rows
// (2304 tiles): three 70 us, two 78, one 88.
int few_tiles(int64_t N, int mt) {
  const int64_t tiles = (N + 15) / 16;
  int best = 1;
  int64_t cost = 5 * ((tiles + 255) / 256);
  for (int r = 2; r <= (mt == 1 ? 3 : 2); ++r) {
    const int64_t c = 4 * r * ((tiles + 256 * r - 1) / (256 * r));
    if (c <= cost) best = r, cost = c;
  }
  return best;
}
enum { kFew, kBig, kMid, kDeep, kSmall };  // kMid: 128 x 128 tiles, two stages; kDeep: four
struct Plan {
  int kernel;
  int splits;
};
// Up to 32 rows of a b streams, but see below.  Else the tiles with the least estimated time, in units of 10 ns, from what a step
// of 128 columns was measured to take on the busiest CU: 256 x 256 tiles 1.55 us; 128 x 128 tiles 0.72 us alone on a CU (a ring
// of four stages), 1.39 us for two at once (of two stages); 64 x 64 tiles 0.40 us alone, 0.53 us for two.  Where the small
// tiles are few they split the reduction, at least 4 blocks a split, and a second launch (3 us) joins the parts.
// Against it, at 512 x 20480 over 5120: 160 large tiles 57-61 us, 640 middle ones 63; 128 x 20480 over 5120: 160 middle tiles
// 30 us, 320 small ones 35; 2047 x 1024 over 4096: 512 small tiles 17 us, 128 middle ones 24.
// Where b has few rows too (16 for a CU at most), nothing but its waves shares out the streaming kernel's reduction: a round of 32
// blocks takes 2.35 us and 0.11 for each row of a.  The split small tiles are taken where they promise half of that, with
// 0.2 us for each split in the second launch: 32 x 64 over 2^20 1495 us streaming, 80 by tiles; 16 x 256 over 131072 128 and 29;
// 32 x 2048 over 16384 27 and 13; but 16 x 64 over 16384 18 and 15, streaming.
Plan own_plan(int64_t M, int64_t N, int64_t nblk, bool ex) {
  const auto tiles = [&](int64_t side) { return ((M + side - 1) / side) * ((N + side - 1) / side); };
  const auto rounds = [](int64_t t, int64_t one, int64_t two) {  // two workgroups a CU
    const int64_t r = t % 512;
    return t / 512 * two + (r == 0 ? 0 : r <= 256 ? one : two);
  };
  const int64_t big = (tiles(256) + 255) / 256 * 155 * ((nblk + 3) / 4 * 4), mid = rounds(tiles(128), 72, 139) * nblk;
  const int64_t t = tiles(64);
  int s = 1;
  while (t * s < 192 && nblk >= 8 * s) s *= 2;
  const int64_t small = rounds(t * s, 40, 53) * ((nblk + s - 1) / s) + (s > 1 ? 300 : 0);
  if (M <= 32) {
    const int64_t few = (N + 15) / 16 <= 256 ? (nblk + 31) / 32 * (235 + 11 * M) : 0;
    return few > 2 * (small + 20 * s) ? Plan{kSmall, s} : Plan{kFew, 1};
  }
  if (!ex && nblk >= 2 && big < mid && big < small) return {kBig, 1};
  if (mid > small) return {kSmall, s};
  return {ex || tiles(128) > 256 ? kMid : kDeep, 1};
}
Plan plan_of(int64_t M, int64_t N, int64_t nblk, bool ex) {
  const Plan p = own_plan(M, N, nblk, ex);
  switch (sra::tuning().fp8_tile) {
    case 64: return {kSmall, p.kernel == kSmall ? p.splits : 1};
    case 128: return {kMid, 1};
    case 132: return {ex ? kMid : kDeep, 1};
    case 256: return {ex || nblk < 2 ? kMid : kBig, 1};
    default: return p;
  }
}

}  // namespace

namespace sra {

// the planner's, whatever the knob says: a knob's tiles split no further, and a size that was asked for stays enough
static size_t ws_of(int64_t M, int64_t N, int64_t K, bool ex) {
  if (M <= 0 || N <= 0) return 0;
  const Plan p = own_plan(M, N, blocks_of(K), ex);
  return p.splits > 1 ? (size_t)p.splits * (size_t)M * (size_t)N * sizeof(float) : 0;
}

// enough for either type of the result
size_t fp8_matmul_ws(int64_t M, int64_t N, int64_t K) { return std::max(ws_of(M, N, K, false), ws_of(M, N, K, true)); }

template <int KA, int KB, bool EX>
static hipError_t matmul(const Mat& a, const Mat& b, const Out& out, const Plan& p, float* ws, hipStream_t s) {
  if (p.kernel == kFew) {
    const int mt = (int)((out.M + 15) / 16), rt = EX ? 1 : few_tiles(out.N, mt);
#define SRA_FEW(MT, RT, NW)                                                                                              \
  launch(SRA_KERNEL_FP8_MM, k_fp8_few<KA, KB, MT, RT, NW, EX>, dim3((unsigned)((out.N + 16 * RT - 1) / (16 * RT))), dim3(64 * NW), \
         0, s, a, b, out)
    if (mt <= 1) {
      if (rt == 1) SRA_FEW(1, 1, 8);
      else if constexpr (!EX) {
        if (rt == 2) SRA_FEW(1, 2, 4);
        else SRA_FEW(1, 3, 4);
      }
    } else {
      if (rt == 1) SRA_FEW(2, 1, 8);
      else if constexpr (!EX) SRA_FEW(2, 2, 4);
    }
#undef SRA_FEW
    return hipGetLastError();
  }
#define SRA_TILES(BM, BN, WM, WN, ST)                                                                               \
  do {                                                                                                              \
    const int nm = (int)((out.M + BM - 1) / BM), nn = (int)((out.N + BN - 1) / BN);                                 \
    launch(SRA_KERNEL_FP8_MM, k_fp8_tiles<KA, KB, BM, BN, WM, WN, ST, EX>, dim3((unsigned)(nm * nn), (unsigned)p.splits), \
           dim3(64 * WM * WN), 0, s, a, b, out, nm, nn, p.splits > 1 ? ws : nullptr);                               \
  } while (0)
  if (p.kernel == kSmall) {
    SRA_TILES(64, 64, 4, 1, 4);
  } else if (p.kernel == kMid) {
    SRA_TILES(128, 128, 2, 2, 2);
  } else if constexpr (!EX) {
    if (p.kernel == kDeep) {
      SRA_TILES(128, 128, 2, 2, 4);
      return hipGetLastError();
    }
    const int nm = (int)((out.M + 255) / 256), nn = (int)((out.N + 255) / 256);
    launch(SRA_KERNEL_FP8_MM, k_fp8_big<KA, KB>, dim3((unsigned)std::min(nm * nn, 256)), dim3(256), 0, s, a, b, out, nm, nn);
  }
#undef SRA_TILES
  hipError_t err = hipGetLastError();
  if (err == hipSuccess && p.splits > 1) {
    const int64_t n = out.M * out.N;
    hipLaunchKernelGGL(k_fp8_join, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 4096)), dim3(256), 0, s, ws, p.splits, out);
    err = hipGetLastError();
  }
  return err;
}

hipError_t launch_fp8_matmul(const Fp8Operand& x, const Fp8Operand& y, int64_t M, int64_t N, int64_t K, bool out_f32,
                             void* o, void* ws, hipStream_t s) {
  if (M <= 0 || N <= 0) return hipSuccess;
  const int64_t nblk = blocks_of(K);
  const Plan p = plan_of(M, N, nblk, out_f32);
  // a launch has fewer than 2^32 threads: at most 2^23 tiles of 256 each, by rows of a in whole blocks (N < 2^26)
  const int64_t side = p.kernel == kSmall ? 64 : 128;
  const int64_t rows = p.kernel == kFew ? M : std::max<int64_t>(256, ((int64_t)1 << 23) / ((N + side - 1) / side) * side & ~(int64_t)255);
  for (int64_t m0 = 0; m0 < M; m0 += rows) {
    // m0 is a multiple of 256: whole blocks of exponents
    const Mat a{x.codes + m0 * nblk * kBlock, x.exps + (x.block_rows == 1 ? m0 : m0 / 128) * nblk, std::min(rows, M - m0),
                nblk * kBlock, nblk, x.block_rows == 1 ? 0 : 7};
    const Mat b{y.codes, y.exps, N, nblk * kBlock, nblk, y.block_rows == 1 ? 0 : 7};
    const Out out{(uint8_t*)o + m0 * N * (out_f32 ? 4 : 2), a.rows, N, out_f32};
    const auto run = [&](auto ka, auto kb) {
      return out_f32 ? matmul<ka.value, kb.value, true>(a, b, out, p, (float*)ws, s)
                     : matmul<ka.value, kb.value, false>(a, b, out, p, (float*)ws, s);
    };
    const std::integral_constant<int, SRA_FP8_E4M3> e4{};
    const std::integral_constant<int, SRA_FP8_E5M2> e5{};
    const hipError_t err = x.kind == SRA_FP8_E4M3 ? (y.kind == SRA_FP8_E4M3 ? run(e4, e4) : run(e4, e5))
                                                  : (y.kind == SRA_FP8_E4M3 ? run(e5, e4) : run(e5, e5));
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace sra
