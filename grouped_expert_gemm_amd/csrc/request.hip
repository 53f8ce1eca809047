// Low-rank adapters of many requests in one batch, beside a projection that they share
// (LoRA, Hu et al. 2021, eq. 3, with each row's own adapter i = ids[t]):
//     out_t = y_t + s_i (x_t A_i^T) B_i^T,     A_i [r, K], B_i [N, r], sums in fp32.
// The work goes in units of up to 16 RB rows that name one adapter, wherever they stand in the
// batch: an adapter's bytes are then read once per unit, and a value of another row's adapter
// cannot reach a row. Two products follow each other in two launches, u = x A^T and the rest.
//
// Up to kRequestScan rows the units come from the ids directly: a workgroup is started for every
// row, and works if its row is the first, or the 17th, ... that names its adapter (ballots over
// the ids, a few instructions). Larger batches get a launch before that lists the units.
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

// Ids outside [0, L) name no adapter.
__device__ __forceinline__ int named(int id, int L) { return id >= 0 && id < L ? id : -1; }

// ------------------------------------------------------------------ the units
// One workgroup lists a batch's units: rows counted by adapter (key L: none), offsets and unit
// numbers by a scan over the keys, rows dealt to their places (in no fixed order: a row's result
// does not depend on its place).
constexpr int kPlanThreads = 1024;

__device__ __forceinline__ int wave_scan(int v) { return (int)wave_scan_sat((uint32_t)v); }

__global__ __launch_bounds__(kPlanThreads) void request_plan_kernel(RequestArgs g, int unit_rows) {
  extern __shared__ int32_t count[];   // [L + 1]
  __shared__ int32_t sums[2][kPlanThreads / 64];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int keys = g.L + 1;
  for (int k = t; k < keys; k += kPlanThreads) count[k] = 0;
  __syncthreads();
  // Place of each lane's row among those of its key, `base` rows counted so far: one atomic for a
  // wavefront whose rows all have one key (a prompt's).
  auto place = [&](int key, bool any) {
    const uint64_t m = __ballot(any);
    if (m == 0) return 0;
    const int first = __builtin_amdgcn_readlane(key, __builtin_ctzll(m));
    if (__ballot(any && key == first) == m) {
      int base = 0;
      if (lane == __builtin_ctzll(m)) base = atomicAdd(&count[first], __builtin_popcountll(m));
      base = __builtin_amdgcn_readlane(base, __builtin_ctzll(m));
      return base + (int)__builtin_popcountll(m & ((1ull << lane) - 1));
    }
    return any ? atomicAdd(&count[key], 1) : 0;
  };
  constexpr int kU = 8;   // ids in flight per thread
  bool bad = false;
  for (int64_t r0 = 0; r0 < g.M; r0 += kU * kPlanThreads) {
    int id[kU];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int64_t r = r0 + i * kPlanThreads + t;
      id[i] = r < g.M ? g.ids[r] : -1;
    }
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      bad |= id[i] >= g.L;
      const int n = named(id[i], g.L);
      place(n < 0 ? g.L : n, r0 + i * kPlanThreads + t < g.M);
    }
  }
  if (bad) atomicOr(g.err, kErrBadExpertId);
  __syncthreads();
  // exclusive scans of rows and units over the keys, a run of keys per thread
  const int per = (keys + kPlanThreads - 1) / kPlanThreads, k0 = min(keys, t * per), k1 = min(keys, k0 + per);
  int rows = 0, units = 0;
  for (int k = k0; k < k1; ++k) {
    rows += count[k];
    units += (count[k] + unit_rows - 1) / unit_rows;
  }
  const int rs = wave_scan(rows), us = wave_scan(units);
  if (lane == 63) {
    sums[0][wave] = rs;
    sums[1][wave] = us;
  }
  __syncthreads();
  int row = rs - rows, unit = us - units;
  for (int w = 0; w < wave; ++w) {
    row += sums[0][w];
    unit += sums[1][w];
  }
  for (int k = k0; k < k1; ++k) {
    const int n = count[k];
    for (int d = 0; d < n; d += unit_rows) {
      int32_t* to = g.units + 4 * (int64_t)unit++;
      to[0] = k < g.L ? k : -1;
      to[1] = row + d;
      to[2] = min(unit_rows, n - d);
    }
    count[k] = row;
    row += n;
  }
  if (t == kPlanThreads - 1) *g.n_units = unit;
  __syncthreads();
  for (int64_t r0 = 0; r0 < g.M; r0 += kU * kPlanThreads) {
    int id[kU];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int64_t r = r0 + i * kPlanThreads + t;
      id[i] = r < g.M ? g.ids[r] : -1;
    }
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int64_t r = r0 + i * kPlanThreads + t;
      const int n = named(id[i], g.L);
      const int at = place(n < 0 ? g.L : n, r < g.M);
      if (r < g.M) g.rows[at] = (int32_t)r;
    }
  }
}

// A unit's adapter (-1: none) and number of rows (0: no such unit), the same for the whole
// workgroup, and in lane l the rows 16 b + l % 16 of it (past the last: the first).
template <int RB>
struct Unit {
  int id, n;
  int row[RB];
  // `pick`: 16 RB words of LDS; every thread comes here
  __device__ __forceinline__ Unit(const RequestArgs& g, int unit, int32_t* pick, bool flag) {
    const int lane = threadIdx.x & 63, r16 = lane & 15;
    if (g.units) {
      n = 0;
      id = -1;
      if (unit < __builtin_amdgcn_readfirstlane(*g.n_units)) {
        const int32_t* u = g.units + 4 * (int64_t)unit;
        id = __builtin_amdgcn_readfirstlane(u[0]);
        n = __builtin_amdgcn_readfirstlane(u[2]);
        const int first = __builtin_amdgcn_readfirstlane(u[1]);
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          const int i = 16 * b + r16;
          row[b] = g.rows[first + (i < n ? i : 0)];
        }
      }
      return;
    }
    const int M = (int)g.M;
    const int raw0 = lane < M ? g.ids[lane] : -1, raw1 = lane + 64 < M ? g.ids[lane + 64] : -1;
    if (flag && (raw0 >= g.L || raw1 >= g.L)) atomicOr(g.err, kErrBadExpertId);
    const int id0 = named(raw0, g.L), id1 = named(raw1, g.L);
    id = unit < 64 ? __builtin_amdgcn_readlane(id0, unit) : __builtin_amdgcn_readlane(id1, unit - 64);
    const uint64_t m0 = __ballot(lane < M && id0 == id), m1 = __ballot(lane + 64 < M && id1 == id);
    // this lane's two rows' places among those of the adapter, and the unit's first row's
    const uint64_t below = (1ull << lane) - 1;
    const int c0 = __builtin_popcountll(m0);
    const int p0 = __builtin_popcountll(m0 & below), p1 = c0 + __builtin_popcountll(m1 & below);
    const int all = c0 + __builtin_popcountll(m1);
    const int at = unit < 64 ? __builtin_popcountll(m0 & ((1ull << unit) - 1))
                             : c0 + __builtin_popcountll(m1 & ((1ull << (unit - 64)) - 1));
    n = at % (16 * RB) == 0 ? min(16 * RB, all - at) : 0;
    if (n == 0) return;
    // (every wavefront writes the same words)
    if (((m0 >> lane) & 1) && p0 >= at && p0 < at + n) pick[p0 - at] = lane;
    if (((m1 >> lane) & 1) && p1 >= at && p1 < at + n) pick[p1 - at] = lane + 64;
    __syncthreads();
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int i = 16 * b + r16;
      row[b] = pick[i < n ? i : 0];
    }
  }
};

// ------------------------------------------------------------------ u = x A^T
// U[split][t, j] = sum over the split's k of x[t, k] A_i[j, k]. A workgroup has one unit and one
// range of 32-wide steps, dealt to its wavefronts in turn; they are added in wavefront order.
template <int T, int RB, int NCB>
__global__ __launch_bounds__(kThreads) void request_down_kernel(RequestArgs g) {
  __shared__ f32x4 red[kWaves - 1][RB][NCB][64];
  __shared__ int32_t pick[16 * RB];
  constexpr int kU = NCB + RB <= 5 ? 4 : 2;   // steps in flight
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, grp = lane >> 4;
  const int split = blockIdx.x % g.splits;
  const Unit<RB> u(g, blockIdx.x / g.splits, pick, blockIdx.x == 0);
  if (u.n == 0 || u.id < 0) return;
  const int steps = (int)((g.K + 31) / 32);
  const int lo = (int)((int64_t)steps * split / g.splits), hi = (int)((int64_t)steps * (split + 1) / g.splits);
  const __amdgpu_buffer_rsrc_t A = window(g.a + (int64_t)u.id * g.r * g.K, (int64_t)g.r * g.K * 2);
  const uint32_t aat = (uint32_t)((r16 * g.K + 8 * grp) * 2), anext = 32 * (uint32_t)g.K;
  const uint16_t* x[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) x[b] = g.x + u.row[b] * g.ldx;
  f32x4 acc[RB][NCB] = {};
  for (int s0 = lo + wave; s0 < hi; s0 += kU * kWaves) {
    u32x4 xf[kU][RB], af[kU][NCB];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int s = s0 + i * kWaves;
      const int64_t k = 32 * (int64_t)s + 8 * grp;
      const bool ok = s < hi && k < g.K;
#pragma unroll
      for (int c = 0; c < NCB; ++c)
        af[i][c] = __builtin_amdgcn_raw_buffer_load_b128(A, oob_unless(ok, aat + c * anext + 64 * (uint32_t)s), 0, 0);
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        xf[i][b] = u32x4{0, 0, 0, 0};
        if (ok && (b == 0 || 16 * b < u.n)) xf[i][b] = *reinterpret_cast<const u32x4*>(x[b] + k);
      }
    }
#pragma unroll
    for (int i = 0; i < kU; ++i)
#pragma unroll
      for (int b = 0; b < RB; ++b)
        if (b == 0 || 16 * b < u.n)
#pragma unroll
          for (int c = 0; c < NCB; ++c) acc[b][c] = mfma<T>(af[i][c], xf[i][b], acc[b][c]);
  }
  if (wave > 0) {
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int c = 0; c < NCB; ++c) red[wave - 1][b][c][lane] = acc[b][c];
  }
  __syncthreads();
  if (wave == 0) {
    float* U = g.u + (int64_t)split * g.M * g.r;
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int c = 0; c < NCB; ++c) {
#pragma unroll
        for (int w = 0; w < kWaves - 1; ++w) acc[b][c] += red[w][b][c][lane];
        const int j = 16 * c + 4 * grp;   // r % 8 == 0: whole groups of four
        if (16 * b + r16 < u.n && j < g.r) *reinterpret_cast<f32x4*>(U + u.row[b] * (int64_t)g.r + j) = acc[b][c];
      }
  }
}

// ------------------------------------------------------------------ out = y + s u B^T
// out[t, n] = y[t, n] + sum_j (s_i u[t, j]) B_i[n, j]. A workgroup has one unit, its wavefronts
// `per` chunks of 64 columns each. u enters the matrix instructions in two 16-bit parts, high and
// rest (together 16 bits of it in bf16, 22 in fp16), laid side by side along the contraction: slot
// group q (8 wide) of the 2 r / 8 holds part q / (r / 8) of j = 8 (q % (r / 8)) .., against the
// same B. fp16 has too few exponents for that: a row of u is scaled by a power of two that brings
// its largest value to [2^10, 2^11), undone in the fp32 sums. The parts are made once per
// workgroup, in LDS.
template <int T, int RB, int NM>
__global__ __launch_bounds__(kThreads) void request_up_kernel(RequestArgs g, int per) {
  __shared__ u32x4 parts[RB][NM][64];
  __shared__ int32_t pick[16 * RB], power[16 * RB];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, grp = lane >> 4;
  const int chunks = (int)((g.N + 63) / 64), groups = (chunks + kWaves * per - 1) / (kWaves * per);
  const int unit = blockIdx.x / groups;
  const Unit<RB> u(g, unit, pick, false);
  if (u.n == 0 || (u.id < 0 && g.out == g.y)) return;
  const int pr = g.r / 8;   // slot groups of a part
  int ex[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) ex[b] = 0;
  if (u.id >= 0) {
    const float s = g.scales ? g.scales[u.id] : 1.0f;
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      if (RB > 1 && b % kWaves != wave) continue;   // (one block: every wavefront, so that none waits)
      float v[NM][8];
      float top = 0.f;
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        const int q = 4 * m + grp;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[m][i] = 0.f;
        if (q < 2 * pr && 16 * b + r16 < u.n) {
          const float* U = g.u + u.row[b] * (int64_t)g.r + 8 * (q < pr ? q : q - pr);
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
      int e = 0;
      if constexpr (T == kF16) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        if (top > 0.f && top < __builtin_inff()) e = (int)__builtin_amdgcn_frexp_expf(top) - 11;
        if (grp == 0) power[16 * b + r16] = e;
      }
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        const bool rest = 4 * m + grp >= pr;
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float a = v[m][2 * i], c = v[m][2 * i + 1];
          if constexpr (T == kF16) {
            a = __builtin_amdgcn_ldexpf(a, -e);
            c = __builtin_amdgcn_ldexpf(c, -e);
          }
          uint32_t h = pack2<T>(a, c);
          if (rest) {
            float ha, hc;
            unpack2<T>(h, ha, hc);
            // (an infinity has no rest)
            h = pack2<T>(fabsf(ha) < __builtin_inff() ? a - ha : 0.f, fabsf(hc) < __builtin_inff() ? c - hc : 0.f);
          }
          w[i] = h;
        }
        parts[b][m][lane] = w;
      }
    }
  }
  __syncthreads();
  if constexpr (T == kF16) {
    if (u.id >= 0) {
#pragma unroll
      for (int b = 0; b < RB; ++b) ex[b] = power[16 * b + r16];
    }
  }
  // a lane has 8 adjacent columns of each row block and pair of column blocks
  const int col = 16 * (grp & 1) + 8 * (grp >> 1);
  const int c0 = (blockIdx.x % groups) * kWaves * per + wave;
  for (int ch = c0; ch < min(chunks, c0 + kWaves * per); ch += kWaves) {
    const int64_t n0 = 64 * (int64_t)ch;
    const int cols = (int)min<int64_t>(64, g.N - n0);
    u32x4 y[RB][2];
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        y[b][p] = u32x4{0, 0, 0, 0};
        if (g.y && 16 * b + r16 < u.n && 32 * p + col < cols)
          y[b][p] = *reinterpret_cast<const u32x4*>(g.y + u.row[b] * g.ldy + n0 + 32 * p + col);
      }
    f32x4 acc[RB][4] = {};
    if (u.id >= 0) {
      const __amdgpu_buffer_rsrc_t B = window(g.b + ((int64_t)u.id * g.N + n0) * g.r, (int64_t)cols * g.r * 2);
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        const int q = 4 * m + grp;
        u32x4 bf[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          bf[j] = __builtin_amdgcn_raw_buffer_load_b128(
              B, oob_unless(q < 2 * pr, (uint32_t)(((16 * j + r16) * g.r + 8 * (q < pr ? q : q - pr)) * 2)), 0, 0);
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          if (b > 0 && 16 * b >= u.n) continue;
          const u32x4 uf = parts[b][m][lane];
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[b][j] = mfma<T>(bf[j], uf, acc[b][j]);
        }
      }
    }
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      if (b > 0 && 16 * b >= u.n) continue;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        // rows of 16 lanes of two neighbouring column blocks trade places
        float d[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float lo = acc[b][2 * p][i], hi = acc[b][2 * p + 1][i];
          if constexpr (T == kF16) {
            lo = __builtin_amdgcn_ldexpf(lo, ex[b]);
            hi = __builtin_amdgcn_ldexpf(hi, ex[b]);
          }
          const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(lo), __float_as_uint(hi), false, false);
          d[i] = __uint_as_float(x[0]);
          d[4 + i] = __uint_as_float(x[1]);
        }
        if (16 * b + r16 < u.n && 32 * p + col < cols) {
          u32x4 o = y[b][p];   // (without an adapter: the same bits)
          if (u.id >= 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float a, e;
              unpack2<T>(y[b][p][i], a, e);
              o[i] = pack2<T>(a + d[2 * i], e + d[2 * i + 1]);
            }
          }
          *reinterpret_cast<u32x4*>(g.out + u.row[b] * g.ldo + n0 + 32 * p + col) = o;
        }
      }
    }
  }
}

template <int T, int RB, int NCB>
hipError_t request_one(const RequestArgs& g, hipStream_t s) {
  const int64_t units = request_units(g.M, g.L, g.r);
  hipLaunchKernelGGL((request_down_kernel<T, RB, NCB>), dim3((unsigned)(units * g.splits)), dim3(kThreads), 0, s, g);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // chunks of 64 columns per wavefront: one while that gives at most about 16 wavefronts per CU
  const int64_t chunks = (g.N + 63) / 64;
  const int64_t per = std::max<int64_t>(1, std::min<int64_t>(8, units * chunks / 4096));
  const int64_t groups = (chunks + kWaves * per - 1) / (kWaves * per);
  hipLaunchKernelGGL((request_up_kernel<T, RB, NCB>), dim3((unsigned)(units * groups)), dim3(kThreads), 0, s, g, (int)per);
  return hipGetLastError();
}

}  // namespace

// Rows of a unit, in blocks of 16: more rows read an adapter's bytes less often, a small batch has
// few rows per adapter.
int request_rows(int64_t M, int32_t r) { return M <= kRequestScan ? 1 : (r > 64 ? 2 : 4); }

// An upper bound of a batch's units.
int64_t request_units(int64_t M, int32_t L, int32_t r) {
  if (M <= kRequestScan) return M;
  const int rows = 16 * request_rows(M, r);
  return (M + rows - 1) / rows + std::min<int64_t>((int64_t)L + 1, M);
}

// Ranges that the first product's contraction is cut into, by the sizes alone (the sums, so the
// results, do not depend on the device): about two workgroups per CU, each of at least two steps
// per wavefront.
int request_splits(int64_t M, int64_t K, int32_t r) {
  const int rows = 16 * request_rows(M, r);
  const int64_t blocks = (M + rows - 1) / rows, steps = (K + 31) / 32;
  return (int)std::max<int64_t>(1, std::min<int64_t>({512 / std::max<int64_t>(blocks, 1), steps / (2 * kWaves), 16}));
}

hipError_t launch_request_lora(const RequestArgs& g, int dtype, hipStream_t s) {
  const int rb = request_rows(g.M, g.r), ncb = (g.r + 15) / 16;
  if (g.units) {
    const size_t bytes = ((size_t)g.L + 1) * 4;
    if (bytes > (48u << 10)) {
      hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(request_plan_kernel),
                                         hipFuncAttributeMaxDynamicSharedMemorySize, (kRequestMaxAdapters + 1) * 4);
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(request_plan_kernel, dim3(1), dim3(kPlanThreads), (unsigned)bytes, s, g, 16 * rb);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
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
