// What the kernels on 16-bit matrices (bf16, fp16) share: bounded windows on memory, the matrix
// instruction by type, rounding in pairs.
#pragma once

#include "geg_device.hpp"

namespace geg {

namespace {

__device__ __forceinline__ uint32_t oob_unless(bool ok, uint32_t off) { return off | ((uint32_t)!ok << 31); }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t window(const void* base, int64_t bytes) {
  const int32_t n = bytes <= 0 ? 0 : (bytes > 0x7FFFFFF0 ? 0x7FFFFFF0 : (int32_t)bytes);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, n, 0x00020000);
}

// acc += first . second for one 16x16x32 block; a lane's results are four adjacent indices of
// the first operand for one of the second.
template <int T>
__device__ __forceinline__ f32x4 mfma(const u32x4& first, const u32x4& second, const f32x4& acc) {
  return mfma16<T == kBF16 ? MXFP4 : NF4>(first, second, acc);
}

template <int T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (T == kBF16) {
    return pack_bf16x2(a, b);
  } else {
    f16x2 h;
    h[0] = (_Float16)a;
    h[1] = (_Float16)b;
    return __builtin_bit_cast(uint32_t, h);
  }
}

}  // namespace

}  // namespace geg
