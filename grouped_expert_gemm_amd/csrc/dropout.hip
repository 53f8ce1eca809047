// Dropout with the mask of philox.hpp, never stored: out = [residual +] keep ? x * scale : 0.
// Its gradient is the same pass over dout without a residual. A dropped value does not enter
// the result, whatever it holds (an infinity or NaN leaves 0).
#include <algorithm>

#include "geg_device.hpp"
#include "geg_launch.hpp"
#include "philox.hpp"

namespace geg {

namespace {

template <int T>
struct Eight {   // 8 values of a type
  u32x4 v[T == kF32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, int64_t block) {
    const u32x4* q = reinterpret_cast<const u32x4*>(p) + block * (T == kF32 ? 2 : 1);
#pragma unroll
    for (int i = 0; i < (T == kF32 ? 2 : 1); ++i) v[i] = q[i];
  }
  __device__ __forceinline__ void store(void* p, int64_t block) const {
    u32x4* q = reinterpret_cast<u32x4*>(p) + block * (T == kF32 ? 2 : 1);
#pragma unroll
    for (int i = 0; i < (T == kF32 ? 2 : 1); ++i) q[i] = v[i];
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (T == kF32) return __uint_as_float(v[i >> 2][i & 3]);
    const uint32_t h = (v[0][i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
    if constexpr (T == kBF16) return __uint_as_float(h << 16);
    return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
  }
  __device__ __forceinline__ void put2(int i, float a, float b) {   // values 2 i, 2 i + 1
    if constexpr (T == kF32) {
      v[i >> 1][2 * (i & 1)] = __float_as_uint(a);
      v[i >> 1][2 * (i & 1) + 1] = __float_as_uint(b);
    } else if constexpr (T == kBF16) {
      v[0][i] = pack_bf16x2(a, b);
    } else {
      f16x2 h;
      h[0] = (_Float16)a;
      h[1] = (_Float16)b;
      v[0][i] = __builtin_bit_cast(uint32_t, h);
    }
  }
};

template <int T>
__device__ __forceinline__ float one(const void* p, int64_t i) {
  if constexpr (T == kF32) return reinterpret_cast<const float*>(p)[i];
  if constexpr (T == kBF16) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << 16);
  return (float)reinterpret_cast<const _Float16*>(p)[i];
}
template <int T>
__device__ __forceinline__ void put_one(void* p, int64_t i, float v) {
  if constexpr (T == kF32)
    reinterpret_cast<float*>(p)[i] = v;
  else if constexpr (T == kBF16)
    reinterpret_cast<uint16_t*>(p)[i] = to_bf16(v);
  else
    reinterpret_cast<_Float16*>(p)[i] = (_Float16)v;
}

// One block of 8 values per thread at a time; WIDE: 16-byte accesses, the tensors aligned. Bound by
// memory: 16384 x 4096 bf16 with a residual 403 MB in 78 us (5.2 TB/s), its gradient 268 MB in 44 us; the
// ten rounds per 8 values hide behind that. 64 x 2048: 2.5 us.
// BITS: the mask is written too.
template <int T, bool RES, bool WIDE, bool BITS = false>
__global__ __launch_bounds__(kThreads) void dropout_kernel(const void* x, const void* res, void* out, uint8_t* bits, int64_t n,
                                                           DropoutArgs d) {
  const PhiloxState g(d);
  const int64_t whole = n / 8, stride = (int64_t)gridDim.x * kThreads;
  const int64_t first = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  for (int64_t b = first; b < (n + 7) / 8; b += stride) {
    uint32_t w[4];
    if (WIDE && b < whole) {
      Eight<T> v, r;
      v.load(x, b);
      if constexpr (RES) r.load(res, b);
      g.bits((uint64_t)b, w);
      if constexpr (BITS) {
        int kept = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) kept |= (int)philox_kept(w, i, d.threshold) << i;
        bits[b] = (uint8_t)kept;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float o[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          o[h] = philox_kept(w, 2 * i + h, d.threshold) ? v.get(2 * i + h) * d.scale : 0.f;
          if constexpr (RES) o[h] = r.get(2 * i + h) + o[h];
        }
        v.put2(i, o[0], o[1]);
      }
      v.store(out, b);
    } else {
      g.bits((uint64_t)b, w);
      for (int i = 0; i < 8 && 8 * b + i < n; ++i) {
        const uint32_t half = i < 4 ? (i < 2 ? w[0] : w[1]) : (i < 6 ? w[2] : w[3]);
        float o = ((half >> (16 * (i & 1))) & 0xFFFFu) >= d.threshold ? one<T>(x, 8 * b + i) * d.scale : 0.f;
        if constexpr (RES) o = one<T>(res, 8 * b + i) + o;
        put_one<T>(out, 8 * b + i, o);
      }
    }
  }
}

}  // namespace

hipError_t launch_dropout(const void* x, const void* res, void* out, uint8_t* bits, int dtype, int64_t n, const DropoutArgs& d,
                          int cus, hipStream_t s) {
  const bool wide = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(res) | reinterpret_cast<uintptr_t>(out)) & 15) == 0;
  const int64_t blocks = ((n + 7) / 8 + kThreads - 1) / kThreads;
  const dim3 grid((unsigned)std::max<int64_t>(1, std::min<int64_t>(blocks, (int64_t)cus * 32)));
  if (bits) {
    hipLaunchKernelGGL((dropout_kernel<kBF16, false, true, true>), grid, dim3(kThreads), 0, s, x, res, out, bits, n, d);
    return hipGetLastError();
  }
  auto run = [&](auto t) {
    constexpr int T = decltype(t)::value;
    if (res) {
      if (wide)
        hipLaunchKernelGGL((dropout_kernel<T, true, true>), grid, dim3(kThreads), 0, s, x, res, out, bits, n, d);
      else
        hipLaunchKernelGGL((dropout_kernel<T, true, false>), grid, dim3(kThreads), 0, s, x, res, out, bits, n, d);
    } else {
      if (wide)
        hipLaunchKernelGGL((dropout_kernel<T, false, true>), grid, dim3(kThreads), 0, s, x, res, out, bits, n, d);
      else
        hipLaunchKernelGGL((dropout_kernel<T, false, false>), grid, dim3(kThreads), 0, s, x, res, out, bits, n, d);
    }
  };
  if (dtype == kBF16)
    run(std::integral_constant<int, kBF16>{});
  else if (dtype == kF16)
    run(std::integral_constant<int, kF16>{});
  else
    run(std::integral_constant<int, kF32>{});
  return hipGetLastError();
}

}  // namespace geg
