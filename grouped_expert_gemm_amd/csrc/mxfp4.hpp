// MXFP4 conversion of one block's values, shared by the packer and by the product
// that quantises its activations.
#pragma once

#include "geg_device.hpp"

namespace geg {

// Code of t = x / 2^X (exact) by arithmetic: round to nearest on the grid of the
// value's binade (steps 0.5, 1, 2), ties to even; a tie between binades lands on
// the even code too.
__device__ __forceinline__ uint32_t e2m1_rne_sat(float t) {
  const uint32_t s = (__float_as_uint(t) >> 28) & 8u;
  const float a = fabsf(t);
  uint32_t c;
  if (a < 2.f)
    c = (uint32_t)__builtin_rintf(2.f * a);
  else if (a < 4.f)
    c = (uint32_t)__builtin_rintf(a) + 2u;
  else
    c = min((uint32_t)__builtin_rintf(0.5f * fminf(a, 16.f)) + 4u, 7u);
  return c | s;
}

__device__ __forceinline__ float e2m1_to_f32(uint32_t c) {
  const uint32_t m = c & 7u;
  const float a = m < 4u ? 0.5f * (float)m : (m < 6u ? (float)m - 2.f : 2.f * (float)m - 8.f);
  return (c & 8u) ? -a : a;
}

// 16 bytes of a row as fp32 values.
template <int DT>
__device__ __forceinline__ void unpack16(const u32x4& v, float* f) {
  if constexpr (DT == kF32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = v[i];
      if constexpr (DT == kBF16) {
        f[2 * i] = __uint_as_float(w << 16);
        f[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
      } else {
        const f16x2 h = __builtin_bit_cast(f16x2, w);
        const _Float16 h0 = h[0], h1 = h[1];
        f[2 * i] = (float)h0;
        f[2 * i + 1] = (float)h1;
      }
    }
  }
}

template <int DT>
__device__ __forceinline__ u32x4 pack16(const float* f) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == kF32) {
      r[i] = __float_as_uint(f[i]);
    } else if constexpr (DT == kBF16) {
      r[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    } else {
      f16x2 h;
      h[0] = (_Float16)f[2 * i];
      h[1] = (_Float16)f[2 * i + 1];
      r[i] = __builtin_bit_cast(uint32_t, h);
    }
  }
  return r;
}

// EPT (4 or 8) consecutive values of a 32-block, held by 32 / EPT consecutive lanes
// that all call it: their codes in `word` (first value in the low nibble), the block's
// scale byte as the result and, with VALUES, the values of the codes in q.
template <int EPT, bool VALUES>
__device__ __forceinline__ int mxfp4_block_piece(const float (&f)[EPT], uint32_t& word, float (&q)[EPT]) {
  constexpr int LPB = 32 / EPT;
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < EPT; ++i) mx = max(mx, __float_as_uint(f[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = 1; o < LPB; o <<= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, o));
  const int field = (int)(mx >> 23);
  // floor(log2 amax) - 2 + 127 = field - 2 for a normal amax; smaller ones clamp to 0
  const int byte = mx == 0 ? 127 : (field == 255 ? 255 : max(field - 2, 0));
  word = 0;
  if (byte >= 27 && byte < 255) {
    const float sc = __uint_as_float((uint32_t)byte << 23);
    word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, f[0], f[1], sc, 0);
    word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, f[2], f[3], sc, 1);
    if constexpr (EPT == 8) {
      word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, f[4], f[5], sc, 2);
      word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, f[6], f[7], sc, 3);
    }
    if constexpr (VALUES) {
#define GEG_PAIR(p)                                                              \
  {                                                                              \
    const auto d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, sc, p);        \
    const float d0 = d[0], d1 = d[1];                                            \
    q[2 * p] = d0;                                                               \
    q[2 * p + 1] = d1;                                                           \
  }
      GEG_PAIR(0)
      GEG_PAIR(1)
      if constexpr (EPT == 8) {
        GEG_PAIR(2)
        GEG_PAIR(3)
      }
#undef GEG_PAIR
    }
  } else if (byte == 255) {
#pragma unroll
    for (int i = 0; i < EPT; ++i) q[i] = __uint_as_float(0x7FC00000u);
  } else {
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const uint32_t c = e2m1_rne_sat(__builtin_ldexpf(f[i], 127 - byte));
      word |= c << (4 * i);
      q[i] = __builtin_ldexpf(e2m1_to_f32(c), byte - 127);
    }
  }
  return byte;
}

}  // namespace geg
