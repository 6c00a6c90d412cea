// Device helpers of the training operators: unaligned row runs, wave
// reductions, and the 8-bit checkpoint's number format.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "train.h"

namespace muon {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4v __attribute__((ext_vector_type(4)));
// The same, read and written at any address: global memory instructions take
// unaligned addresses, so a row that starts anywhere (an odd pitch) moves in
// 16-byte runs like an aligned one.
typedef u32x4 u32x4_any __attribute__((aligned(1)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));

__device__ inline float bits_f32(uint32_t u) { return __builtin_bit_cast(float, u); }
__device__ inline uint32_t f32_bits(float f) { return __builtin_bit_cast(uint32_t, f); }

// Eight consecutive elements of a row as they lie in memory.
template <typename T>
struct Raw8;
template <>
struct Raw8<__bf16> {
  u32x4 v;
  __device__ float get(int i) const { return bits_f32(i & 1 ? v[i >> 1] & 0xffff0000u : v[i >> 1] << 16); }
};
template <>
struct Raw8<float> {
  u32x4 v[2];
  __device__ float get(int i) const { return bits_f32(v[i >> 2][i & 3]); }
};

// The first min(n, 8) of them (zeros behind; n <= 0: none is read). A run that is
// cut repeats its last element, so that its loads are in flight together.
__device__ inline Raw8<__bf16> load8(const __bf16 *p, int n) {
  Raw8<__bf16> r{};
  if (n >= 8) {
    r.v = *reinterpret_cast<const u32x4_any *>(p);
  } else if (n > 0) {
    const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
    uint32_t e[7];
#pragma unroll
    for (int i = 0; i < 7; ++i) e[i] = q[i < n ? i : n - 1];
#pragma unroll
    for (int i = 0; i < 7; ++i) r.v[i >> 1] |= (i < n ? e[i] : 0u) << (16 * (i & 1));
  }
  return r;
}
__device__ inline Raw8<float> load8(const float *p, int n) {
  Raw8<float> r{};
  if (n >= 8) {
    r.v[0] = *reinterpret_cast<const u32x4_any *>(p);
    r.v[1] = *reinterpret_cast<const u32x4_any *>(p + 4);
  } else if (n > 0) {
    const uint32_t *q = reinterpret_cast<const uint32_t *>(p);
    uint32_t e[7];
#pragma unroll
    for (int i = 0; i < 7; ++i) e[i] = q[i < n ? i : n - 1];
#pragma unroll
    for (int i = 0; i < 7; ++i) r.v[i >> 2][i & 3] = i < n ? e[i] : 0u;
  }
  return r;
}

// Two values of a word, one instruction.
__device__ inline uint32_t pack2(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}
__device__ inline Raw8<__bf16> pack8(const float (&f)[8], __bf16) {
  Raw8<__bf16> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[i] = pack2(f[2 * i], f[2 * i + 1]);
  }
  return r;
}
__device__ inline Raw8<float> pack8(const float (&f)[8], float) {
  Raw8<float> r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r.v[i >> 2][i & 3] = f32_bits(f[i]);
  return r;
}

__device__ inline void store8(__bf16 *p, const Raw8<__bf16> &r, int n) {
  if (n >= 8) {
    *reinterpret_cast<u32x4_any *>(p) = r.v;
  } else {
    uint16_t *q = reinterpret_cast<uint16_t *>(p);
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) q[i] = uint16_t(r.v[i >> 1] >> (16 * (i & 1)));
  }
}
__device__ inline void store8(float *p, const Raw8<float> &r, int n) {
  if (n >= 8) {
    *reinterpret_cast<u32x4_any *>(p) = r.v[0];
    *reinterpret_cast<u32x4_any *>(p + 4) = r.v[1];
  } else {
    uint32_t *q = reinterpret_cast<uint32_t *>(p);
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) q[i] = r.v[i >> 2][i & 3];
  }
}

// Lane permutations inside rows of 16 lanes.
template <int kCtrl>
__device__ inline float dpp(float v) {
  return bits_f32(__builtin_amdgcn_update_dpp(0, int(f32_bits(v)), kCtrl, 0xf, 0xf, false));
}
template <int kCtrl>
__device__ inline uint32_t dpp(uint32_t v) {
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), kCtrl, 0xf, 0xf, false));
}
constexpr int kQuadSwap1 = 0xB1, kQuadSwap2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

// A value of this lane's row of 16 and the neighbouring row's (the even row's
// first), or of both halves of the wave (the lower's first), without LDS.
struct Pair {
  float a, b;
};
__device__ inline Pair rows_16(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(f32_bits(v), f32_bits(v), false, false);
  return {bits_f32(r[0]), bits_f32(r[1])};
}
__device__ inline Pair halves_32(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(f32_bits(v), f32_bits(v), false, false);
  return {bits_f32(r[0]), bits_f32(r[1])};
}

// Sum over the 64 lanes, the same value in each (a fixed tree: the result
// depends on nothing but the inputs).
__device__ inline float wave_sum(float v) {
  v += dpp<kQuadSwap1>(v);
  v += dpp<kQuadSwap2>(v);
  v += dpp<kHalfMirror>(v);
  v += dpp<kMirror>(v);
  const Pair p = rows_16(v);
  const Pair q = halves_32(p.a + p.b);
  return q.a + q.b;
}
// Maximum of unsigned values over rows of 16 lanes, in each of them.
__device__ inline uint32_t row16_max(uint32_t v) {
  v = max(v, dpp<kQuadSwap1>(v));
  v = max(v, dpp<kQuadSwap2>(v));
  v = max(v, dpp<kHalfMirror>(v));
  v = max(v, dpp<kMirror>(v));
  return v;
}

// ---- the checkpoint's number format ---------------------------------------

// |x| as ordered bits, 0 where x is not finite: a group's scale comes from
// its finite values.
__device__ inline uint32_t finite_mag(float x) {
  const uint32_t u = f32_bits(x) & 0x7fffffffu;
  return u < 0x7f800000u ? u : 0u;
}
// Scale byte b of a group with largest magnitude amax (bits): 2^(b - 127) is
// the smallest power of two with amax <= 448 * 2^(b - 127), at least 2^-127.
// 448 = 1.75 * 2^8, so b is amax's exponent field less 8, and one more when
// its significand exceeds 1.75.
__device__ inline uint32_t scale_byte(uint32_t amax) {
  const int b = int(amax >> 23) - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return b > 0 ? uint32_t(b) : 0u;
}
__device__ inline float scale_inverse(uint32_t b) { return bits_f32((254u - b) << 23); }        // 2^(127 - b)
__device__ inline float scale_value(uint32_t b) { return b ? bits_f32(b << 23) : bits_f32(0x400000u); }  // 2^(b - 127)

// Eight values over the group's scale as e4m3 codes (nearest even; NaN and
// infinities become NaN, nothing else overflows).
__device__ inline u32x2 encode8(const float (&f)[8], float inv) {
  u32x2 c;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h] * inv, f[4 * h + 1] * inv, 0, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h + 2] * inv, f[4 * h + 3] * inv, v, true);
    c[h] = uint32_t(v);
  }
  return c;
}
__device__ inline void store_codes8(uint8_t *p, const u32x2 &c, int n) {
  if (n >= 8) {
    *reinterpret_cast<u32x2_any *>(p) = c;
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) p[i] = uint8_t(c[i >> 2] >> (8 * (i & 3)));
  }
}
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
// Two codes of a dword (half 0 or 1) times the scale, as packed bf16. Exact:
// a value has four significant bits (only below 2^-133 is it rounded).
template <int kHalf>
__device__ inline uint32_t decode2(uint32_t c, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, scale, kHalf != 0));
}

}  // namespace muon
