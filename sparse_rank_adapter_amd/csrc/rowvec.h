// Row-wise helpers of the layer norm and checkpoint kernels: vectors of VEC consecutive elements of
// a bf16 or fp32 row as floats, reductions over lanes, and the 8-bit block code.
#pragma once

#include "common.h"

namespace sra_row {

constexpr int kCkBlock = 32;  // columns that share one scale

// VEC consecutive elements (VEC = 8, 2 or 1; 8 needs 16-byte aligned rows, 2 a row of an even
// length on a 4-byte base) as floats, and back with one rounding to the storage type (NaN stays NaN)
template <typename E, int VEC>
struct RowVec;

template <int VEC>
struct RowVec<uint16_t, VEC> {
  static SRA_DEV void load(const uint16_t* __restrict__ p, float (&f)[VEC]) {
    if constexpr (VEC == 8) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f[2 * k] = __uint_as_float(v[k] << 16);
        f[2 * k + 1] = __uint_as_float(v[k] & 0xffff0000u);
      }
    } else if constexpr (VEC == 2) {
      const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
      f[0] = __uint_as_float(v << 16);
      f[1] = __uint_as_float(v & 0xffff0000u);
    } else {
      f[0] = bf16_to_f32(*p);
    }
  }
  // rounds f in place to what is stored
  static SRA_DEV void store(uint16_t* __restrict__ p, float (&f)[VEC]) {
    union { __bf16 b[VEC]; uint16_t h[VEC]; uint32_t w[VEC > 1 ? VEC / 2 : 1]; } o;
#pragma unroll
    for (int k = 0; k < VEC; ++k) o.b[k] = (__bf16)f[k];
#pragma unroll
    for (int k = 0; k < VEC; ++k) f[k] = bf16_to_f32(o.h[k]);
    if constexpr (VEC == 8) {
      u32x4 v;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = o.w[k];
      *reinterpret_cast<u32x4*>(p) = v;
    } else if constexpr (VEC == 2) {
      *reinterpret_cast<uint32_t*>(p) = o.w[0];
    } else {
      *p = o.h[0];
    }
  }
};

template <int VEC>
struct RowVec<float, VEC> {
  static SRA_DEV void load(const float* __restrict__ p, float (&f)[VEC]) {
    if constexpr (VEC == 8) {
      const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f[k] = a[k];
        f[k + 4] = b[k];
      }
    } else {
#pragma unroll
      for (int k = 0; k < VEC; ++k) f[k] = p[k];
    }
  }
  static SRA_DEV void store(float* __restrict__ p, float (&f)[VEC]) {
    if constexpr (VEC == 8) {
      *reinterpret_cast<f32x4*>(p) = f32x4{f[0], f[1], f[2], f[3]};
      *reinterpret_cast<f32x4*>(p + 4) = f32x4{f[4], f[5], f[6], f[7]};
    } else {
#pragma unroll
      for (int k = 0; k < VEC; ++k) p[k] = f[k];
    }
  }
};

// ---- the 8-bit block code.  A block of up to 32 consecutive columns shares the scale 2^e, e the
// smallest integer with max|x| <= 127 * 2^e (from the bits of max|x| = m 2^E, 1 <= m < 2:
// E - 6, one more when m > 127/64), clamped to [-126, 121] so that the scale is a normal float and
// 127 * 2^e is finite.  q = round-half-even(x 2^-e) in [-127, 127]: the product is exact, and
// q 2^e is exact in bf16 and fp32 (8 significant bits), so a decoded value is rounded once.
SRA_DEV int ck_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 6 + ((u & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return min(max(e, -126), 121);
}
SRA_DEV float ck_pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
SRA_DEV int ck_code(float x, float inv) { return (int)fminf(fmaxf(rintf(x * inv), -127.f), 127.f); }

// Codes and scale of this lane's VEC elements (LPB = 32 / VEC neighbouring lanes hold a block;
// lanes past the row's end pass zeros); returns the codes packed and sets the biased exponent.
// Non-finite inputs are outside the contract: they saturate (NaN gives some code in range).
template <int VEC>
struct Coded {
  uint64_t codes;  // VEC bytes, lowest column first
  uint32_t exp;    // e + 127
};
template <int VEC>
SRA_DEV Coded<VEC> ck_encode(const float (&f)[VEC]) {
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < VEC; ++k) m = fmaxf(m, fabsf(f[k]));
#pragma unroll
  for (int d = 1; d < kCkBlock / VEC; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
  const int e = ck_exp(m);
  const float inv = ck_pow2(-e);
  Coded<VEC> c;
  c.codes = 0;
  c.exp = (uint32_t)(e + 127);
#pragma unroll
  for (int k = 0; k < VEC; ++k) c.codes |= (uint64_t)(uint8_t)ck_code(f[k], inv) << (8 * k);
  return c;
}
template <int VEC>
SRA_DEV void ck_store_codes(int8_t* __restrict__ p, uint64_t codes) {
  if constexpr (VEC == 8)
    *reinterpret_cast<u32x2*>(p) = u32x2{(uint32_t)codes, (uint32_t)(codes >> 32)};
  else if constexpr (VEC == 2)
    *reinterpret_cast<uint16_t*>(p) = (uint16_t)codes;
  else
    *p = (int8_t)codes;
}
template <int VEC>
SRA_DEV uint64_t ck_load_codes(const int8_t* __restrict__ p) {
  if constexpr (VEC == 8) {
    const u32x2 v = *reinterpret_cast<const u32x2*>(p);
    return (uint64_t)v[0] | ((uint64_t)v[1] << 32);
  } else if constexpr (VEC == 2) {
    return *reinterpret_cast<const uint16_t*>(p);
  } else {
    return *reinterpret_cast<const uint8_t*>(p);
  }
}
template <int VEC>
SRA_DEV void ck_decode(uint64_t codes, uint32_t exp, float (&f)[VEC]) {
  const float s = __uint_as_float(exp << 23);
#pragma unroll
  for (int k = 0; k < VEC; ++k) f[k] = (float)(int8_t)(uint8_t)(codes >> (8 * k)) * s;
}

// vector width of rows of `len` elements on 16-byte aligned bases
inline int row_vec(int64_t len) { return len % 8 == 0 ? 8 : len % 2 == 0 ? 2 : 1; }

}  // namespace sra_row
