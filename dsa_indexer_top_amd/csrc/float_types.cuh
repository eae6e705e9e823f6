// Loads, conversions and reductions shared by the operators in front of the indexer: rows of
// bf16, fp16 or fp32 read eight elements per lane, FP8 E4M3FN packing, and butterflies over the
// lanes that hold one row.
#pragma once

#include "common.hpp"

namespace echo {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

struct bf16_t { uint16_t bits; };
struct fp16_t { _Float16 v; };

ECHO_DEV float to_f32(bf16_t x) { return __uint_as_float(static_cast<uint32_t>(x.bits) << 16); }
ECHO_DEV float to_f32(fp16_t x) { return static_cast<float>(x.v); }
ECHO_DEV float to_f32(float x) { return x; }

// Round to nearest even, the type's own overflow (infinity) and NaN.
template <typename T> ECHO_DEV T from_f32(float x);
template <> ECHO_DEV float from_f32<float>(float x) { return x; }
template <> ECHO_DEV fp16_t from_f32<fp16_t>(float x) { return fp16_t{static_cast<_Float16>(x)}; }
template <> ECHO_DEV bf16_t from_f32<bf16_t>(float x) {
  const __bf16 b = static_cast<__bf16>(x);
  return bf16_t{__builtin_bit_cast(uint16_t, b)};
}

constexpr int VEC = 8;           // elements per lane

// Eight consecutive elements as loaded: 16 bytes (bf16, fp16) or 32 (fp32).
template <typename T> struct Raw8 { u32x4 w[sizeof(T) * VEC / 16]; };

// Read once by the whole launch, so past the caches (8191 x 45 x 128 fp16 heads on MI355X: 40.1 us
// with plain loads, 36.8 with these).
template <typename T>
ECHO_DEV Raw8<T> load8(const T *__restrict__ p) {
  Raw8<T> r;
#pragma unroll
  for (unsigned i = 0; i < sizeof(T) * VEC / 16; ++i)
    r.w[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p) + i);
  return r;
}
// The same from any address the type allows: gfx950 reads 16 bytes at any of them.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));
template <typename T>
ECHO_DEV Raw8<T> load8_any(const T *__restrict__ p) {
  Raw8<T> r;
#pragma unroll
  for (unsigned i = 0; i < sizeof(T) * VEC / 16; ++i) r.w[i] = reinterpret_cast<const u32x4_any *>(p)[i];
  return r;
}
template <typename T>
ECHO_DEV Raw8<T> zero8() {
  Raw8<T> r;
#pragma unroll
  for (unsigned i = 0; i < sizeof(T) * VEC / 16; ++i) r.w[i] = u32x4{0, 0, 0, 0};
  return r;
}
// The first n of eight elements, one by one (rows whose address or end allows no wide load).
template <typename T>
ECHO_DEV Raw8<T> load8_part(const T *__restrict__ p, int n) {
  T e[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) e[i] = i < n ? p[i] : from_f32<T>(0.f);
  Raw8<T> r;
  __builtin_memcpy(&r, e, sizeof r);
  return r;
}
template <typename T>
ECHO_DEV void unpack8(const Raw8<T> &r, float (&x)[VEC]) {
  T e[VEC];
  __builtin_memcpy(e, &r, sizeof r);
#pragma unroll
  for (int i = 0; i < VEC; ++i) x[i] = to_f32(e[i]);
}
template <typename T>
ECHO_DEV void store8(T *__restrict__ p, const float (&x)[VEC]) {
  T e[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) e[i] = from_f32<T>(x[i]);
  Raw8<T> r;
  __builtin_memcpy(&r, e, sizeof r);
#pragma unroll
  for (unsigned i = 0; i < sizeof(T) * VEC / 16; ++i) reinterpret_cast<u32x4 *>(p)[i] = r.w[i];
}

// Eight values to FP8 E4M3FN, round to nearest even; the caller keeps |x| below 464, so nothing
// overflows.  NaN stays NaN.
ECHO_DEV u32x2 pack_fp8(const float (&x)[VEC]) {
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], hi, true);
  return u32x2{static_cast<unsigned>(lo), static_cast<unsigned>(hi)};
}

// ---------------------------------------------------------------- butterflies
// All G lanes of an aligned group receive OP over the group.  Within 16 lanes the partners come
// from DPP moves (quad swaps, then mirrors of 8 and 16 lanes, whose halves already hold equal
// values); every lane adds the same two partial results, so all G lanes get the same bits.
constexpr int DPP_QUAD_XOR1 = 0xB1, DPP_QUAD_XOR2 = 0x4E, DPP_HALF_MIRROR = 0x141, DPP_MIRROR = 0x140;

template <int G, typename OP>
ECHO_DEV uint32_t group_reduce(uint32_t v, OP op) {
  if (G > 1) v = op(v, dpp_mov<DPP_QUAD_XOR1, 0xF>(0u, v));
  if (G > 2) v = op(v, dpp_mov<DPP_QUAD_XOR2, 0xF>(0u, v));
  if (G > 4) v = op(v, dpp_mov<DPP_HALF_MIRROR, 0xF>(0u, v));
  if (G > 8) v = op(v, dpp_mov<DPP_MIRROR, 0xF>(0u, v));
  if (G > 16) v = op(v, __shfl_xor(v, 16, 64));
  return v;
}
struct OpAddF {
  ECHO_DEV uint32_t operator()(uint32_t a, uint32_t b) const {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }
};
template <int G> ECHO_DEV float group_sum(float v) {
  return __uint_as_float(group_reduce<G>(__float_as_uint(v), OpAddF{}));
}
// Largest |x|, as an integer maximum over the bits without the sign: a NaN is larger than every
// number there, so it is kept.
template <int G> ECHO_DEV float group_amax(const float (&x)[VEC]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const uint32_t b = __float_as_uint(x[i]) & 0x7FFFFFFFu;
    m = m > b ? m : b;
  }
  return __uint_as_float(group_reduce<G>(m, OpMax{}));
}

// ---------------------------------------------------------------- FP8 scales
// scale = amax / 448, the largest value going to the largest E4M3FN number, but at least 2^-126:
// a block of zeros has a positive scale, and 1/scale is finite.  A block with a NaN or an
// infinity gets a NaN or infinite scale, and what its codes stand for is NaN.
constexpr float FP8_MAX = 448.f;
constexpr float FP8_AMAX_MIN = 448.f * 1.17549435e-38f;     // 448 * 2^-126

// Codes of eight values: the fp32 quotient x / scale rounded to the nearest code.  Quotients on the
// border of two codes are common (one bf16 value in a thousand), so one that is off by its last bit
// gives another code, as x times a rounded reciprocal did.  A block shares its scale, so its reciprocal
// is made in two parts, hi + lo: x (hi + lo) is within 2^-44 of the quotient before its one rounding, which
// is then the quotient's own for every pair of 16-bit x and largest x (tried for all, with a first
// reciprocal off by one unit either way).  Values with all of their 24 bits (FULL) take one step more,
// q - (q scale - x) / scale, whose remainder is exact (Markstein).  The scale itself is a (1 / 448) with
// that constant in two parts, equal to the division for every significand of a (tried for all).  Waves
// with a block whose products could underflow or that has an infinity or a NaN divide.  On
// MI355X 32768 tokens of indexer inputs take 152 us (149 with one rounded reciprocal, 157 with two divisions
// a block, 193 with one per value), 32768 x 4096 bf16 values 72.6 (72.7, 73.0 and 85.7).
struct Fp8Scale { float scale, inv, hi, lo; bool divide; };
template <bool FULL>
ECHO_DEV Fp8Scale fp8_scale(float amax) {                      // every lane of the wave calls
  const float a = amax < FP8_AMAX_MIN ? FP8_AMAX_MIN : amax;   // a NaN passes
  const bool zeros = amax == 0.f;                              // padding: any reciprocal does
  if (__ballot(!zeros && !(a >= 0x1p-64f && a <= 0x1p64f))) return Fp8Scale{a / FP8_MAX, 0.f, 0.f, 0.f, true};
  constexpr float C_HI = 1.f / FP8_MAX, C_LO = static_cast<float>(1.0 / 448.0 - static_cast<double>(C_HI));
  const float scale = zeros ? FP8_AMAX_MIN / FP8_MAX : fmaf(a, C_HI, a * C_LO);
  const float inv = FULL ? 1.f / scale : __builtin_amdgcn_rcpf(scale);         // rounded, or off by a unit
  const float hi = __uint_as_float(__float_as_uint(inv) - 2u);                 // below 1 / scale: lo is positive
  return Fp8Scale{scale, inv, hi, fmaf(-scale, hi, 1.f) * inv, false};
}
template <bool FULL>
ECHO_DEV u32x2 quantise8(const float (&x)[VEC], const Fp8Scale &s) {
  float y[VEC];
  if (!s.divide) {                                                   // the same for the whole wave
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      y[i] = fmaf(x[i], s.hi, x[i] * s.lo);                          // a zero keeps its sign
      if (FULL) y[i] = fmaf(-fmaf(y[i], s.scale, -x[i]), s.inv, y[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) y[i] = x[i] / s.scale;
  }
  return pack_fp8(y);
}

}  // namespace echo
