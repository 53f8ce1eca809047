// MXFP4 quantisation (OCP MX v1.0 conversion) of bf16, fp16 or fp32 rows: per 32
// consecutive values with largest magnitude amax,
//     X = max(floor(log2 amax) - 2, -127)     (0 for an all-zero block)
//     code = nearest e2m1 value of x / 2^X, ties to the even code, saturating at 6,
// the sign kept (-0 for negatives that round to 0); the scale byte is X + 127. A
// block that holds an inf or a NaN gets scale byte 255, which decodes to NaN.
//
// Memory bound: a value is read once and 17/32 of a byte written (plus the value
// itself when asked for). A thread takes one 16-byte piece of its row (8 or 4
// values), the 4 or 8 lanes of a block share amax through lane exchanges, and the
// codes come from gfx950's scaled fp4 conversion (two values per instruction,
// round to nearest even, saturating; the division by 2^X is exact). Values that it
// might flush (blocks whose scale is below 2^-100) go through exact fp32
// arithmetic instead. 46080 x 2880 fp32 with the decoded values, 1.13 GB: 198 us, 5.7
// TB/s, what a large copy reaches; 8192 x 2880 bf16 with them, 107 MB: 16.9 us; four
// rows: 2.4 us, the launch.
#include <algorithm>

#include "geg_device.hpp"
#include "geg_launch.hpp"
#include "mxfp4.hpp"

namespace geg {

namespace {

// One 16-byte piece: codes (16 or 32 bits) and, on the block's first lane, the
// scale byte; with VALUES also the decoded piece. Every lane of a block calls it.
template <int DT, bool VALUES>
__device__ __forceinline__ void quantize_piece(const u32x4& v, int64_t piece, uint8_t* __restrict__ codes,
                                               uint8_t* __restrict__ scales, void* __restrict__ values) {
  constexpr int EPT = DT == kF32 ? 4 : 8;   // values per piece
  constexpr int LPB = 32 / EPT;             // pieces per block
  float f[EPT], q[EPT];
  unpack16<DT>(v, f);
  uint32_t word;
  const int byte = mxfp4_block_piece<EPT, VALUES>(f, word, q);
  if constexpr (EPT == 8)
    reinterpret_cast<uint32_t*>(codes)[piece] = word;
  else
    reinterpret_cast<uint16_t*>(codes)[piece] = (uint16_t)word;
  if ((piece & (LPB - 1)) == 0) scales[piece / LPB] = (uint8_t)byte;
  if constexpr (VALUES) reinterpret_cast<u32x4*>(values)[piece] = pack16<DT>(q);
}

// UNR pieces per thread, 256 apart, their loads all in flight first. Pieces of a
// row are consecutive; `ppr` pieces per row, rows `ld16` 16-byte units apart
// (ld16 == ppr: the matrix is one run of pieces).
template <int DT, bool VALUES, int UNR>
__global__ __launch_bounds__(kThreads) void mxfp4_quantize_kernel(const u32x4* __restrict__ x, int64_t pieces,
                                                                  int64_t ppr, int64_t ld16,
                                                                  uint8_t* __restrict__ codes,
                                                                  uint8_t* __restrict__ scales,
                                                                  void* __restrict__ values) {
  const int64_t p0 = (int64_t)blockIdx.x * (UNR * kThreads) + threadIdx.x;
  u32x4 v[UNR];
#pragma unroll
  for (int u = 0; u < UNR; ++u) {
    const int64_t p = p0 + u * kThreads;
    if (p < pieces) {
      const int64_t at = ld16 == ppr ? p : (p / ppr) * ld16 + p % ppr;
      v[u] = x[at];
    }
  }
#pragma unroll
  for (int u = 0; u < UNR; ++u) {
    // pieces come in whole blocks of 4 or 8 consecutive lanes, so the lanes of a
    // block pass this test together
    const int64_t p = p0 + u * kThreads;
    if (p < pieces) quantize_piece<DT, VALUES>(v[u], p, codes, scales, values);
  }
}

template <int DT, bool VALUES>
hipError_t launch_dt(const void* x, int64_t rows, int64_t K, int64_t ld, uint8_t* codes, uint8_t* scales,
                     void* values, int cus, hipStream_t s) {
  constexpr int EPT = DT == kF32 ? 4 : 8;
  const int64_t ppr = K / EPT, pieces = rows * ppr;
  const u32x4* xv = reinterpret_cast<const u32x4*>(x);
  // four pieces per thread once that still fills the chip
  if (pieces >= (int64_t)cus * kThreads * 8) {
    const int64_t grid = (pieces + 4 * kThreads - 1) / (4 * kThreads);
    hipLaunchKernelGGL((mxfp4_quantize_kernel<DT, VALUES, 4>), dim3((unsigned)grid), dim3(kThreads), 0, s, xv, pieces,
                       ppr, ld / EPT, codes, scales, values);
  } else {
    const int64_t grid = (pieces + kThreads - 1) / kThreads;
    hipLaunchKernelGGL((mxfp4_quantize_kernel<DT, VALUES, 1>), dim3((unsigned)grid), dim3(kThreads), 0, s, xv, pieces,
                       ppr, ld / EPT, codes, scales, values);
  }
  return hipGetLastError();
}

template <int DT>
hipError_t launch_values(const void* x, int64_t rows, int64_t K, int64_t ld, uint8_t* codes, uint8_t* scales,
                         void* values, int cus, hipStream_t s) {
  return values ? launch_dt<DT, true>(x, rows, K, ld, codes, scales, values, cus, s)
                : launch_dt<DT, false>(x, rows, K, ld, codes, scales, values, cus, s);
}

}  // namespace

hipError_t launch_mxfp4_quantize(const void* x, int dtype, int64_t rows, int64_t K, int64_t ld, uint8_t* codes,
                                 uint8_t* scales, void* values, int cus, hipStream_t s) {
  if (dtype == kBF16) return launch_values<kBF16>(x, rows, K, ld, codes, scales, values, cus, s);
  if (dtype == kF16) return launch_values<kF16>(x, rows, K, ld, codes, scales, values, cus, s);
  return launch_values<kF32>(x, rows, K, ld, codes, scales, values, cus, s);
}

}  // namespace geg
