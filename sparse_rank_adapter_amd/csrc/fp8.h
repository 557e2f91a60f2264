// 8-bit floating point with a power-of-two scale for each block of 128 columns: the code shared by the
// encoder, the norm that writes it and the products that read it.
//
// A block with largest finite magnitude a has the scale 2^e, e the smallest integer with a <= lim 2^e
// (lim = 448 = 1.75 2^8 for e4m3, 57344 = 1.75 2^15 for e5m2; from the bits of a = m 2^E, 1 <= m < 2:
// E - 8 or E - 15, one more when m > 1.75), clamped so that the scale is a normal float and lim 2^e is
// finite.  The code is x 2^-e (exact, or far below the type's smallest value) rounded to nearest even
// by the hardware's conversion; past the clamp it saturates at lim.  The stored exponent e + 127 is an
// E8M0 byte, the form in which the scaled matrix instructions take a scale, so products apply it for nothing.
// An infinity or NaN becomes the code NaN and takes no part in its block's scale.
#pragma once

#include "rowvec.h"

namespace sra_f8 {

constexpr int kBlock = 128;  // columns (or, for blocks of 128 rows, columns and rows) that share one scale
inline int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }
inline int64_t ld_of(int64_t cols) { return blocks_of(cols) * kBlock; }  // bytes between rows of codes

template <int KIND>
struct Kind;
template <>
struct Kind<SRA_FP8_E4M3> {
  static constexpr int top = 8, most = 119;
  static constexpr float lim = 448.f;
  static SRA_DEV uint32_t pack4(float a, float b, float c, float d) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true);
  }
  static SRA_DEV void unpack4(uint32_t w, float (&f)[4]) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    f[0] = lo[0], f[1] = lo[1], f[2] = hi[0], f[3] = hi[1];
  }
};
template <>
struct Kind<SRA_FP8_E5M2> {
  static constexpr int top = 15, most = 112;
  static constexpr float lim = 57344.f;
  static SRA_DEV uint32_t pack4(float a, float b, float c, float d) {
    const int lo = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_bf8_f32(c, d, lo, true);
  }
  static SRA_DEV void unpack4(uint32_t w, float (&f)[4]) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_bf8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_bf8((int)w, true);
    f[0] = lo[0], f[1] = lo[1], f[2] = hi[0], f[3] = hi[1];
  }
};

constexpr uint32_t kInf = 0x7f800000u;
// magnitude bits of x, 0 where x is not finite: their unsigned maximum over a block gives its scale
SRA_DEV uint32_t mag(float x) {
  const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
  return u < kInf ? u : 0u;
}
template <int KIND>
SRA_DEV int exp_of(uint32_t m) {
  const int e = (int)(m >> 23) - 127 - Kind<KIND>::top + ((m & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, -126), Kind<KIND>::most);
}
SRA_DEV float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// x over its block's scale, inside the type's range; NaN where x is not finite
template <int KIND>
SRA_DEV float scaled(float x, float inv) {
  const float v = __builtin_amdgcn_fmed3f(x * inv, -Kind<KIND>::lim, Kind<KIND>::lim);
  return (__float_as_uint(x) & 0x7fffffffu) < kInf ? v : __uint_as_float(0x7fc00000u);
}
template <int KIND>
SRA_DEV uint32_t code4(float a, float b, float c, float d, float inv) {
  return Kind<KIND>::pack4(scaled<KIND>(a, inv), scaled<KIND>(b, inv), scaled<KIND>(c, inv), scaled<KIND>(d, inv));
}
// scale of an E8M0 byte (0: 2^-127, 255: NaN; the encoder writes neither)
SRA_DEV float scale_of(uint32_t e) {
  const uint32_t u = e == 0 ? 0x00400000u : e == 255 ? 0x7fc00000u : e << 23;
  return __uint_as_float(u);
}

// maximum over each 16 consecutive lanes (by DPP row rotations, no LDS), in all of them
SRA_DEV uint32_t max16(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x128, 0xf, 0xf, true));  // row_ror 8, 4, 2, 1
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x124, 0xf, 0xf, true));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x122, 0xf, 0xf, true));
  return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x121, 0xf, 0xf, true));
}
// The code of this lane's VEC elements where 128 / VEC neighbouring lanes hold a block (VEC = 8 or 2);
// lanes past the row's end pass zeros.  Every lane of the wave takes part.
template <int KIND, int VEC>
struct Coded {
  uint32_t w[VEC == 8 ? 2 : 1];  // VEC bytes, lowest column first
  uint32_t exp;                  // e + 127
};
template <int KIND, int VEC>
SRA_DEV Coded<KIND, VEC> encode(const float (&f)[VEC]) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < VEC; ++k) m = max(m, mag(f[k]));
  m = max16(m);
  if constexpr (VEC == 2) {
    m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
  }
  const int e = exp_of<KIND>(m);
  const float inv = pow2(-e);
  Coded<KIND, VEC> c;
  c.exp = (uint32_t)(e + 127);
  if constexpr (VEC == 8) {
    c.w[0] = code4<KIND>(f[0], f[1], f[2], f[3], inv);
    c.w[1] = code4<KIND>(f[4], f[5], f[6], f[7], inv);
  } else {
    c.w[0] = code4<KIND>(f[0], f[1], 0.f, 0.f, inv);
  }
  return c;
}
template <int KIND, int VEC>
SRA_DEV void store_codes(uint8_t* __restrict__ p, const Coded<KIND, VEC>& c) {
  if constexpr (VEC == 8) *reinterpret_cast<u32x2*>(p) = u32x2{c.w[0], c.w[1]};
  else *reinterpret_cast<uint16_t*>(p) = (uint16_t)c.w[0];
}

// VEC elements of a row of any length: VEC = 8 needs rows of whole 16-byte vectors, VEC = 2 takes the
// elements one by one, as many as there are
template <typename E, int VEC>
SRA_DEV void load_row(const E* __restrict__ p, int64_t left, float (&f)[VEC]) {
#pragma unroll
  for (int k = 0; k < VEC; ++k) f[k] = 0.f;
  if constexpr (VEC == 8) {
    if (left > 0) sra_row::RowVec<E, 8>::load(p, f);
  } else {
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      if (k < left) {
        float one[1];
        sra_row::RowVec<E, 1>::load(p + k, one);
        f[k] = one[0];
      }
    }
  }
}
template <typename E, int VEC>
SRA_DEV void store_row(E* __restrict__ p, int64_t left, const float (&f)[VEC]) {
  if constexpr (VEC == 8) {
    float o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = f[k];
    if (left > 0) sra_row::RowVec<E, 8>::store(p, o);
  } else {
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      float one[1] = {f[k]};
      if (k < left) sra_row::RowVec<E, 1>::store(p + k, one);
    }
  }
}
// The same in two steps, for loads that are to be in flight together: as stored (of what lies outside, the first elements
// of the row), and as floats with zeros outside
template <typename E, int VEC>
struct Stored {
  union { E e[VEC]; u32x4 q[VEC * sizeof(E) / 16 + 1]; };
};
template <typename E, int VEC>
SRA_DEV Stored<E, VEC> fetch(const E* __restrict__ row, int64_t c, int64_t len) {
  Stored<E, VEC> o;
  if constexpr (VEC == 8) {
    const E* const p = row + (c < len ? c : 0);
#pragma unroll
    for (int i = 0; i < (int)sizeof(E) / 2; ++i) o.q[i] = reinterpret_cast<const u32x4*>(p)[i];
  } else {
#pragma unroll
    for (int k = 0; k < VEC; ++k) o.e[k] = row[c + k < len ? c + k : 0];
  }
  return o;
}
template <typename E, int VEC>
SRA_DEV void as_floats(const Stored<E, VEC>& s, int64_t left, float (&f)[VEC]) {
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    float v;
    if constexpr (sizeof(E) == 4) v = s.e[k];
    else v = bf16_to_f32(s.e[k]);
    f[k] = (VEC == 8 ? left > 0 : k < left) ? v : 0.f;
  }
}
inline bool vec8(int64_t len) { return len % 8 == 0; }

}  // namespace sra_f8
