// Low-rank adapters of many requests in one batch, beside a projection that they share
// (LoRA, Hu et al. 2021, eq. 3, with each row's own adapter i = ids[t]):
//     out_t = y_t + s_i (x_t A_i^T) B_i^T,     A_i [r, K], B_i [N, r], sums in fp32.
// Two launches: u = x A^T, then the rest. A block of 16 RB rows walks the adapters that its
// rows name, whatever their order: no sort, no list. For each, every row of the block is
// multiplied and the rows that name it keep the result, so a value of another row's adapter
// never reaches a row. A request's rows usually stand together (one adapter per block), and
// in a decode batch, where they do not, the adapters' bytes are the work anyway.
#include <algorithm>

#include "geg_device.hpp"
#include "geg_launch.hpp"

namespace geg {

namespace {

constexpr int kWaves = kThreads / 64;

__device__ __forceinline__ uint32_t oob_unless(bool ok, uint32_t off) { return off | ((uint32_t)!ok << 31); }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t window(const void* base, int64_t bytes) {
  const int32_t n = bytes <= 0 ? 0 : (bytes > 0x7FFFFFF0 ? 0x7FFFFFF0 : (int32_t)bytes);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, n, 0x00020000);
}

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
template <int T>
__device__ __forceinline__ void unpack2(uint32_t v, float& a, float& b) {
  if constexpr (T == kBF16) {
    a = __uint_as_float(v << 16);
    b = __uint_as_float(v & 0xFFFF0000u);
  } else {
    const f16x2 h = __builtin_bit_cast(f16x2, v);
    a = (float)h[0];
    b = (float)h[1];
  }
}

// The adapters that the rows of a block name: lane l holds those of rows 16 b + l % 16.
template <int RB>
struct Ids {
  int id[RB];        // -1: none
  bool open[RB];     // not walked yet
  __device__ __forceinline__ Ids(const RequestArgs& g, int64_t row0, bool flag) {
    bool bad = false;
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int64_t row = row0 + 16 * b + (threadIdx.x & 15);
      int v = row < g.M ? g.ids[row] : -1;
      if (v >= g.L) {
        bad = true;
        v = -1;
      }
      id[b] = v < 0 ? -1 : v;
      open[b] = v >= 0;
    }
    if (flag && bad) atomicOr(g.err, kErrBadExpertId);
  }
  // The next adapter, -1 behind the last one; `mine` marks its rows.
  __device__ __forceinline__ int next(bool* mine) {
    int cur = -1;
#pragma unroll
    for (int b = RB - 1; b >= 0; --b) {
      const uint64_t m = __ballot(open[b]);
      if (m) cur = __builtin_amdgcn_readlane(id[b], __builtin_ctzll(m));
    }
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      mine[b] = cur >= 0 && id[b] == cur;
      open[b] = open[b] && !mine[b];
    }
    return cur;
  }
};

// U[split][t, j] = sum over the split's k of x[t, k] A_i[j, k], for rows with an adapter. A
// workgroup has 16 RB rows and one range of 32-wide steps, dealt to its wavefronts in turn;
// they are added in wavefront order.
template <int T, int RB, int NCB>
__global__ __launch_bounds__(kThreads) void request_down_kernel(RequestArgs g) {
  __shared__ f32x4 red[kWaves - 1][RB][NCB][64];
  constexpr int kU = NCB + RB <= 5 ? 4 : 2;   // steps in flight
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, grp = lane >> 4;
  const int64_t row0 = (int64_t)(blockIdx.x / g.splits) * 16 * RB;
  const int split = blockIdx.x % g.splits;
  const int steps = (int)((g.K + 31) / 32);
  const int lo = (int)((int64_t)steps * split / g.splits), hi = (int)((int64_t)steps * (split + 1) / g.splits);
  const int rows = (int)min<int64_t>(16 * RB, g.M - row0);
  const __amdgpu_buffer_rsrc_t X = window(g.x + row0 * g.ldx, ((rows - 1) * g.ldx + g.K) * 2);
  const uint32_t xat = (uint32_t)((r16 * g.ldx + 8 * grp) * 2), xnext = 32 * (uint32_t)g.ldx;
  const uint32_t aat = (uint32_t)((r16 * g.K + 8 * grp) * 2), anext = 32 * (uint32_t)g.K;
  Ids<RB> ids(g, row0, split == 0 && wave == 0);
  f32x4 keep[RB][NCB] = {};
  bool mine[RB];
  for (int cur; (cur = ids.next(mine)) >= 0;) {
    const __amdgpu_buffer_rsrc_t A = window(g.a + (int64_t)cur * g.r * g.K, (int64_t)g.r * g.K * 2);
    f32x4 acc[RB][NCB] = {};
    for (int s0 = lo + wave; s0 < hi; s0 += kU * kWaves) {
      u32x4 xf[kU][RB], af[kU][NCB];
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        const int s = s0 + i * kWaves;
        const bool ok = s < hi && 32 * (int64_t)s + 8 * grp < g.K;
#pragma unroll
        for (int c = 0; c < NCB; ++c)
          af[i][c] = __builtin_amdgcn_raw_buffer_load_b128(A, oob_unless(ok, aat + c * anext + 64 * (uint32_t)s), 0, 0);
#pragma unroll
        for (int b = 0; b < RB; ++b)
          xf[i][b] = __builtin_amdgcn_raw_buffer_load_b128(X, oob_unless(ok, xat + b * xnext + 64 * (uint32_t)s), 0, 0);
      }
#pragma unroll
      for (int i = 0; i < kU; ++i)
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
          for (int c = 0; c < NCB; ++c) acc[b][c] = mfma<T>(af[i][c], xf[i][b], acc[b][c]);
    }
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int c = 0; c < NCB; ++c) keep[b][c] = mine[b] ? acc[b][c] : keep[b][c];
  }
  if (wave > 0) {
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int c = 0; c < NCB; ++c) red[wave - 1][b][c][lane] = keep[b][c];
  }
  __syncthreads();
  if (wave == 0) {
    float* U = g.u + ((int64_t)split * g.M + row0) * g.r;
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int c = 0; c < NCB; ++c) {
#pragma unroll
        for (int w = 0; w < kWaves - 1; ++w) keep[b][c] += red[w][b][c][lane];
        const int row = 16 * b + r16, j = 16 * c + 4 * grp;   // r % 8 == 0: whole groups of four
        if (row < rows && j < g.r && ids.id[b] >= 0) *reinterpret_cast<f32x4*>(U + (int64_t)row * g.r + j) = keep[b][c];
      }
  }
}

// out[t, n] = y[t, n] + sum_j (s_i u[t, j]) B_i[n, j]. A wavefront has 16 RB rows and 64
// columns. u enters the matrix instructions in two 16-bit parts, high and rest (together 16
// bits of it in bf16, 22 in fp16), laid side by side along the contraction: slot group q (8
// wide) of the 2 r / 8 holds part q / (r / 8) of j = 8 (q % (r / 8)) .., against the same B.
// fp16 has too few exponents for that: a row of u is scaled by a power of two that brings its
// largest value to [2^10, 2^11), undone in the fp32 sums.
template <int T, int RB, int NM>
__global__ __launch_bounds__(kThreads) void request_up_kernel(RequestArgs g) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, grp = lane >> 4;
  const int chunks = (int)((g.N + 63) / 64);
  const int64_t unit = (int64_t)blockIdx.x * kWaves + wave;
  const int64_t row0 = unit / chunks * 16 * RB;
  const int64_t n0 = unit % chunks * 64;
  if (row0 >= g.M) return;
  const int rows = (int)min<int64_t>(16 * RB, g.M - row0);
  const int cols = (int)min<int64_t>(64, g.N - n0);

  // y first: a lane has 8 adjacent columns of each row block and pair of column blocks
  const int col = 16 * (grp & 1) + 8 * (grp >> 1);
  u32x4 y[RB][2];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      y[b][p] = u32x4{0, 0, 0, 0};
      const int row = 16 * b + r16, c = 32 * p + col;
      if (g.y && row < rows && c < cols) y[b][p] = *reinterpret_cast<const u32x4*>(g.y + (row0 + row) * g.ldy + n0 + c);
    }

  Ids<RB> ids(g, row0, false);
  const int pr = g.r / 8;   // slot groups of a part
  u32x4 uf[RB][NM];
  int ex[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    const int row = 16 * b + r16;
    const bool any = ids.id[b] >= 0;
    float v[NM][8];
    float top = 0.f;
    const float s = any ? (g.scales ? g.scales[ids.id[b]] : 1.0f) : 0.f;
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      const int q = 4 * m + grp;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[m][i] = 0.f;
      if (any && q < 2 * pr) {
        const float* U = g.u + (row0 + row) * g.r + 8 * (q < pr ? q : q - pr);
        for (int k = 0; k < g.splits; ++k, U += g.M * g.r) {
          const f32x4 lo = *reinterpret_cast<const f32x4*>(U), hi = *reinterpret_cast<const f32x4*>(U + 4);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[m][i] += lo[i];
            v[m][4 + i] += hi[i];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[m][i] *= s;
        top = fmaxf(top, fabsf(v[m][i]));
      }
    }
    ex[b] = 0;
    if constexpr (T == kF16) {
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      if (top > 0.f && top < __builtin_inff()) ex[b] = (int)__builtin_amdgcn_frexp_expf(top) - 11;
    }
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      const bool rest = 4 * m + grp >= pr;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float a = v[m][2 * i], c = v[m][2 * i + 1];
        if constexpr (T == kF16) {
          a = __builtin_amdgcn_ldexpf(a, -ex[b]);
          c = __builtin_amdgcn_ldexpf(c, -ex[b]);
        }
        uint32_t h = pack2<T>(a, c);
        if (rest) {
          float ha, hc;
          unpack2<T>(h, ha, hc);
          // (an infinity has no rest)
          h = pack2<T>(fabsf(ha) < __builtin_inff() ? a - ha : 0.f, fabsf(hc) < __builtin_inff() ? c - hc : 0.f);
        }
        uf[b][m][i] = h;
      }
    }
  }

  f32x4 keep[RB][4] = {};
  bool mine[RB];
  for (int cur; (cur = ids.next(mine)) >= 0;) {
    const __amdgpu_buffer_rsrc_t B = window(g.b + ((int64_t)cur * g.N + n0) * g.r, (int64_t)cols * g.r * 2);
    f32x4 acc[RB][4] = {};
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      const int q = 4 * m + grp;
      u32x4 bf[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        bf[j] = __builtin_amdgcn_raw_buffer_load_b128(
            B, oob_unless(q < 2 * pr, (uint32_t)(((16 * j + r16) * g.r + 8 * (q < pr ? q : q - pr)) * 2)), 0, 0);
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[b][j] = mfma<T>(bf[j], uf[b][m], acc[b][j]);
    }
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int j = 0; j < 4; ++j) keep[b][j] = mine[b] ? acc[b][j] : keep[b][j];
  }

#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      // rows of 16 lanes of two neighbouring column blocks trade places: 8 adjacent columns each
      float d[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float lo = keep[b][2 * p][i], hi = keep[b][2 * p + 1][i];
        if constexpr (T == kF16) {
          lo = __builtin_amdgcn_ldexpf(lo, ex[b]);
          hi = __builtin_amdgcn_ldexpf(hi, ex[b]);
        }
        const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(lo), __float_as_uint(hi), false, false);
        d[i] = __uint_as_float(x[0]);
        d[4 + i] = __uint_as_float(x[1]);
      }
      const int row = 16 * b + r16, c = 32 * p + col;
      if (row < rows && c < cols) {
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float a, e;
          unpack2<T>(y[b][p][i], a, e);
          o[i] = pack2<T>(a + d[2 * i], e + d[2 * i + 1]);
        }
        // a row without an adapter keeps its bits
        if (ids.id[b] < 0) o = y[b][p];
        if (ids.id[b] >= 0 || g.out != g.y) *reinterpret_cast<u32x4*>(g.out + (row0 + row) * g.ldo + n0 + c) = o;
      }
    }
}

template <int T, int RB, int NCB>
hipError_t request_one(const RequestArgs& g, hipStream_t s) {
  const int64_t blocks = (g.M + 16 * RB - 1) / (16 * RB);
  hipLaunchKernelGGL((request_down_kernel<T, RB, NCB>), dim3((unsigned)(blocks * g.splits)), dim3(kThreads), 0, s, g);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t units = blocks * ((g.N + 63) / 64);
  hipLaunchKernelGGL((request_up_kernel<T, RB, NCB>), dim3((unsigned)((units + kWaves - 1) / kWaves)), dim3(kThreads), 0,
                     s, g);
  return hipGetLastError();
}

}  // namespace

// Row blocks of 16 per workgroup: more rows read an adapter's bytes less often, fewer leave
// more workgroups.
int request_rows(int64_t M, int32_t r) { return M <= 512 ? 1 : (r > 64 ? 2 : 4); }

// Ranges that the first product's contraction is cut into, by the sizes alone (the sums, so the
// results, do not depend on the device): about two workgroups per CU, each of at least one step
// per wavefront.
int request_splits(int64_t M, int64_t K, int32_t r) {
  const int64_t blocks = (M + 16 * request_rows(M, r) - 1) / (16 * request_rows(M, r));
  const int64_t steps = (K + 31) / 32;
  return (int)std::max<int64_t>(1, std::min<int64_t>({512 / std::max<int64_t>(blocks, 1), (steps + kWaves - 1) / kWaves, 32}));
}

hipError_t launch_request_lora(const RequestArgs& g, int dtype, hipStream_t s) {
  const int rb = request_rows(g.M, g.r), ncb = (g.r + 15) / 16;
  auto run = [&](auto t, auto n) {
    constexpr int T = decltype(t)::value, NCB = decltype(n)::value;
    if (rb == 1) return request_one<T, 1, NCB>(g, s);
    return request_one<T, NCB <= 4 ? 4 : 2, NCB>(g, s);
  };
  auto by_rank = [&](auto t) {
    if (ncb == 1) return run(t, std::integral_constant<int, 1>{});
    if (ncb == 2) return run(t, std::integral_constant<int, 2>{});
    if (ncb <= 4) return run(t, std::integral_constant<int, 4>{});
    return run(t, std::integral_constant<int, 8>{});
  };
  return dtype == kBF16 ? by_rank(std::integral_constant<int, kBF16>{}) : by_rank(std::integral_constant<int, kF16>{});
}

}  // namespace geg
