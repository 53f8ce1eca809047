// Low-rank adapters of many requests in one batch, beside a projection that they share
// (LoRA, Hu et al. 2021, eq. 3, with each row's own adapter i = ids[t]):
//     out_t = y_t + s_i (x_t A_i^T) B_i^T,     A_i [r, K], B_i [N, r], sums in fp32.
// The work goes in units of up to 16 RB rows that name one adapter, wherever they stand in the
// batch: an adapter's bytes are then read once per unit, and a value of another row's adapter
// cannot reach a row. Two products follow each other in two launches, u = x A^T and the rest.
//
// In small batches (request_scan()) the units come from the ids directly: a workgroup is started for
// every row, and works if its row is the first, or the 17th, ... that names its adapter (ballots over
// the ids, a few instructions). Others get a launch before that lists the units.
#include <algorithm>

#include "geg_device.hpp"
#include "geg_launch.hpp"
#include "wide16.hpp"

namespace geg {

namespace {

constexpr int kWaves = kThreads / 64;

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

// Two 16-bit values, infinities and NaN replaced by 0.
template <int T>
__device__ __forceinline__ uint32_t finite2(uint32_t v) {
  constexpr uint32_t top = T == kBF16 ? 0x7F80u : 0x7C00u;
  return ((v & 0x7FFFu) >= top ? 0 : v & 0xFFFFu) | (((v >> 16) & 0x7FFFu) >= top ? 0 : v & 0xFFFF0000u);
}

// Ids outside [0, L) name no adapter.
__device__ __forceinline__ int named(int id, int L) { return id >= 0 && id < L ? id : -1; }

// ------------------------------------------------------------------ the units
// One workgroup lists a batch's units (8000 rows: 9 us, two reads of the ids): rows counted by adapter (key L: none), offsets and unit
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
    constexpr int kWords = kRequestScan / 64;
    const int M = (int)g.M;
    int ids[kWords];   // of rows 64 w + lane
    bool bad = false;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      const int raw = 64 * w + lane < M ? g.ids[64 * w + lane] : -1;
      bad |= raw >= g.L;
      ids[w] = named(raw, g.L);
    }
    if (flag && bad) atomicOr(g.err, kErrBadExpertId);
    id = 0;
#pragma unroll
    for (int w = 0; w < kWords; ++w)
      if (unit >> 6 == w) id = __builtin_amdgcn_readlane(ids[w], unit & 63);
    // the places of the unit's first row and of this lane's among the adapter's
    const uint64_t below = (1ull << lane) - 1;
    uint64_t m[kWords];
    int all = 0, at = 0;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      m[w] = __ballot(64 * w + lane < M && ids[w] == id);
      if (unit >> 6 == w) at = all + __builtin_popcountll(m[w] & ((1ull << (unit & 63)) - 1));
      all += __builtin_popcountll(m[w]);
    }
    n = at % (16 * RB) == 0 ? min(16 * RB, all - at) : 0;
    if (n == 0) return;
    // (every wavefront writes the same words)
    int place = -at;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      const int mine = place + (int)__builtin_popcountll(m[w] & below);
      if (((m[w] >> lane) & 1) && mine >= 0 && mine < n) pick[mine] = 64 * w + lane;
      place += __builtin_popcountll(m[w]);
    }
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
// range of 32-wide steps, dealt to its wavefronts in turn; they are added in wavefront order. Bound by
// x (8000 x 4096: 65.5 MB in 21 us where x is in the last cache, 28 where not), a small batch by
// latency; loads a step ahead of the products gained nothing (28 to 32 us).
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
// out[t, n] = y[t, n] + sum_j (s_i u[t, j]) B_i[n, j]. The work is (unit, 4 chunks of 64 columns, one
// per wavefront): one of these to a workgroup where the units come from the ids, equal runs of them to
// two workgroups per CU for others, so that a unit's start (its rows, the parts of u) is paid once per
// run and no second round of workgroups is half empty. Bound by y and out: 8000 rows of 14336
// columns, fp16, rank 64, read and write 459 MB in 116 to 125 us, 3.8 TB/s (a copy of 1 GiB: 5.2);
// both pass the L2 by, 160 -> 152 us with the launches before. u enters the matrix instructions in two 16-bit parts, high and
// rest (together within 2^-17 of it in bf16; in fp16 within 2^-22, or 2^-35 of its row's largest): for r <= 16 (PACK) side by side in one
// instruction's contraction (slot group q, 8 wide, holds part q / (r / 8) of j = 8 (q % (r / 8)) ..),
// else NB blocks of 32 of either against the same B. fp16 has too few exponents for that: a row of u
// is scaled by a power of two that brings its largest value to [2^10, 2^11), undone in the fp32
// sums. The parts are made once per workgroup, in LDS.
template <int T, int RB, int NB, bool PACK>
__global__ __launch_bounds__(kThreads, 2) void request_up_kernel(RequestArgs g, int units) {
  static_assert(!PACK || NB == 1, "two parts in one block");
  constexpr int kParts = PACK ? 1 : 2 * NB;
  __shared__ u32x4 parts[RB][kParts][64];
  __shared__ int32_t pick[16 * RB], power[16 * RB];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, grp = lane >> 4;
  const int chunks = (int)((g.N + 63) / 64), groups = (chunks + kWaves - 1) / kWaves;
  const int pr = g.r / 8;   // slot groups of a part
  // slot group q of block m, here: its j / 8, or past the end
  auto slot = [&](int m) {
    const int q = 4 * m + grp;
    if constexpr (PACK) return q < pr ? q : (q < 2 * pr ? q - pr : 16);
    return q < pr ? q : 16;
  };
  auto run = [&](const Unit<RB>& u, int g0, int g1) {
    int ex[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) ex[b] = 0;
    if (u.id >= 0) {
      const float s = g.scales ? g.scales[u.id] : 1.0f;
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        if (RB > 1 && b % kWaves != wave) continue;   // (one block: every wavefront, so that none waits)
        float v[NB][8];
        float top = 0.f;
#pragma unroll
        for (int m = 0; m < NB; ++m) {
          const int q = slot(m);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[m][i] = 0.f;
          if (q < 16 && 16 * b + r16 < u.n) {
            const float* U = g.u + u.row[b] * (int64_t)g.r + 8 * q;
#pragma unroll 4
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
            if (fabsf(v[m][i]) < __builtin_inff()) top = fmaxf(top, fabsf(v[m][i]));   // of the finite ones
          }
        }
        int e = 0;
        if constexpr (T == kF16) {
          top = fmaxf(top, __shfl_xor(top, 16));
          top = fmaxf(top, __shfl_xor(top, 32));
          if (top > 0.f) e = (int)__builtin_amdgcn_frexp_expf(top) - 11;
          if (grp == 0) power[16 * b + r16] = e;
        }
#pragma unroll
        for (int m = 0; m < NB; ++m) {
          u32x4 high, rest;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float a = v[m][2 * i], c = v[m][2 * i + 1];
            if constexpr (T == kF16) {
              a = __builtin_amdgcn_ldexpf(a, -e);
              c = __builtin_amdgcn_ldexpf(c, -e);
            }
            high[i] = pack2<T>(a, c);
            float ha, hc;
            unpack2<T>(high[i], ha, hc);
            // (an infinity has no rest)
            rest[i] = pack2<T>(fabsf(ha) < __builtin_inff() ? a - ha : 0.f, fabsf(hc) < __builtin_inff() ? c - hc : 0.f);
          }
          if constexpr (PACK) {
            parts[b][0][lane] = grp < pr ? high : rest;
          } else {
            parts[b][m][lane] = high;
            parts[b][NB + m][lane] = rest;
          }
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
    // The matrix instructions leave a lane 8 adjacent columns of one row in each half chunk; its loads of
    // y and its stores are of whole 128-byte lines, 8 rows an instruction: rows 8 h + r16 % 8.
    const bool low = r16 < 8;
    const int col = 32 * (r16 >> 3) + 16 * (grp & 1) + 8 * (grp >> 1);
    int row[RB][2];
    uint32_t live = 0;
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = 8 * h + (r16 & 7);
        row[b][h] = __shfl(u.row[b], i);
        live |= (uint32_t)(16 * b + i < u.n) << (2 * b + h);
      }
    const int c0 = g0 * kWaves + wave, c1 = min(chunks, g1 * kWaves);
    uint32_t bat[NB];
#pragma unroll
    for (int m = 0; m < NB; ++m) bat[m] = oob_unless(slot(m) < 16, (uint32_t)((r16 * g.r + 8 * slot(m)) * 2));
    auto b_window = [&](int ch) {
      const int64_t n0 = 64 * (int64_t)ch;
      return window(g.b + ((int64_t)u.id * g.N + n0) * g.r, std::min<int64_t>(64, g.N - n0) * g.r * 2);
    };
    auto load_b = [&](int ch, u32x4 (&bf)[NB][4]) {
      const __amdgpu_buffer_rsrc_t B = b_window(ch);
#pragma unroll
      for (int m = 0; m < NB; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) bf[m][j] = __builtin_amdgcn_raw_buffer_load_b128(B, bat[m] + 32 * j * (uint32_t)g.r, 0, 0);
    };
    // Loads of y are unconditional (rows and columns past the end: some that are there).
    auto load_y = [&](int ch, int b, u32x4 (&y)[RB][2]) {
      const int64_t n = std::min<int64_t>(64 * (int64_t)ch + col, g.N - 8);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        y[b][h] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(g.y + row[b][h] * g.ldy + n));
    };
    auto store = [&](int ch, int b, int h, u32x4 o, bool all) {
      const int64_t n = 64 * (int64_t)ch + col;
      if (all || (((live >> (2 * b + h)) & 1) && n < g.N))
        __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(g.out + row[b][h] * g.ldo + n));
    };
    auto product = [&](int ch, const u32x4 (&bf)[NB][4], int b, float (&d)[2][8]) {
      f32x4 acc[4] = {};
#pragma unroll
      for (int m = 0; m < NB; ++m) {
        const u32x4 high = parts[b][m][lane];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = mfma<T>(bf[m][j], high, acc[j]);
        if constexpr (!PACK) {
          const u32x4 rest = parts[b][NB + m][lane];
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[j] = mfma<T>(bf[m][j], rest, acc[j]);
        }
      }
      // An infinity in B times the second part (0, or of the other sign) makes its column NaN: a product
      // with a result that is not finite is done again, the infinities beside the first part only.
      f32x4 z;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        z[i] = __builtin_fmaf(acc[0][i], 0.f, __builtin_fmaf(acc[1][i], 0.f, __builtin_fmaf(acc[2][i], 0.f, acc[3][i] * 0.f)));
      const float odd = (z[0] + z[1]) + (z[2] + z[3]);   // 0, or NaN
      if (__builtin_expect(__ballot(odd != odd) != 0, 0)) {
        const __amdgpu_buffer_rsrc_t B = b_window(ch);   // (read again: kept, B would cost the others registers)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int m = 0; m < NB; ++m) {
            const u32x4 q = __builtin_amdgcn_raw_buffer_load_b128(B, bat[m] + 32 * j * (uint32_t)g.r, 0, 0);
            u32x4 f;
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = finite2<T>(q[i]);
            if constexpr (PACK) {
              acc[j] = mfma<T>(grp < pr ? q : f, parts[b][m][lane], acc[j]);
            } else {
              acc[j] = mfma<T>(q, parts[b][m][lane], acc[j]);
              acc[j] = mfma<T>(f, parts[b][NB + m][lane], acc[j]);
            }
            __builtin_amdgcn_sched_barrier(0);   // one piece at a time: registers
          }
        }
      }
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        // rows of 16 lanes of two neighbouring column blocks trade places
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float lo = acc[2 * p][i], hi = acc[2 * p + 1][i];
          if constexpr (T == kF16) {
            lo = __builtin_amdgcn_ldexpf(lo, ex[b]);
            hi = __builtin_amdgcn_ldexpf(hi, ex[b]);
          }
          const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(lo), __float_as_uint(hi), false, false);
          d[p][i] = __uint_as_float(x[0]);
          d[p][4 + i] = __uint_as_float(x[1]);
        }
      }
      // and the second half of a low row with the first of the row 8 below
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int give = __float_as_int(low ? d[1][i] : d[0][i]);
        const float got = __int_as_float(__builtin_amdgcn_update_dpp(0, give, 0x128, 0xF, 0xF, false));   // row_ror:8
        d[0][i] = low ? d[0][i] : got;
        d[1][i] = low ? got : d[1][i];
      }
    };
    auto add = [&](const u32x4& y, const float (&d)[8]) {
      u32x4 o;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float a, e;
        unpack2<T>(y[i], a, e);
        o[i] = pack2<T>(a + d[2 * i], e + d[2 * i + 1]);
      }
      return o;
    };
    if (u.id < 0) {
      for (int ch = c0; ch < c1; ch += kWaves) {
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          u32x4 y[RB][2] = {};
          if (g.y) load_y(ch, b, y);
#pragma unroll
          for (int h = 0; h < 2; ++h) store(ch, b, h, y[b][h], false);   // the same bits
        }
      }
    } else if (RB == 1 || !g.y) {
      for (int ch = c0; ch < c1; ch += kWaves) {
        u32x4 bf[NB][4], y[RB][2] = {};
        load_b(ch, bf);
        if (g.y) {
#pragma unroll
          for (int b = 0; b < RB; ++b) load_y(ch, b, y);
        }
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          if (b > 0 && 16 * b >= u.n) continue;
          float d[2][8];
          product(ch, bf, b, d);
#pragma unroll
          for (int h = 0; h < 2; ++h) store(ch, b, h, add(y[b][h], d[h]), false);
        }
      }
    } else if (c0 < c1) {
      // The next chunk's B is asked for before this one's products, its y of a row block as soon as this
      // chunk's is used.
      auto walk = [&](int lo, int hi, auto all) {
        if (lo >= hi) return;
        u32x4 bf[NB][4], y[RB][2];
        load_b(lo, bf);
#pragma unroll
        for (int b = 0; b < RB; ++b) load_y(lo, b, y);
#pragma unroll 1
        for (int ch = lo; ch < hi; ch += kWaves) {
          const int next = ch + kWaves < hi ? ch + kWaves : ch;
          // (row * pitch anew for every chunk: 64-bit addresses would take 32 registers)
#pragma unroll
          for (int b = 0; b < RB; ++b) asm volatile("" : "+v"(row[b][0]), "+v"(row[b][1]));
          u32x4 nf[NB][4];
          if constexpr (NB <= 2) load_b(next, nf);
#pragma unroll
          for (int b = 0; b < RB; ++b) {
            float d[2][8];
            product(ch, bf, b, d);
#pragma unroll
            for (int h = 0; h < 2; ++h) store(ch, b, h, add(y[b][h], d[h]), decltype(all)::value);
            load_y(next, b, y);
          }
          if constexpr (NB <= 2) {
#pragma unroll
            for (int m = 0; m < NB; ++m)
#pragma unroll
              for (int j = 0; j < 4; ++j) bf[m][j] = nf[m][j];
          } else {
            load_b(next, bf);
          }
        }
      };
      if (u.n == 16 * RB && 64 * (int64_t)c1 <= g.N)
        walk(c0, c1, std::true_type{});
      else
        walk(c0, c1, std::false_type{});
    }
  };
  if constexpr (RB == 1) {
    const int unit = blockIdx.x / groups, g0 = blockIdx.x % groups;
    const Unit<RB> u(g, unit, pick, false);
    if (u.n > 0 && (u.id >= 0 || g.out != g.y)) run(u, g0, g0 + 1);
    return;
  }
  if (g.units) units = __builtin_amdgcn_readfirstlane(*g.n_units);
  // neighbouring ranges on one XCD, whose L2 then holds their adapters
  const int W = gridDim.x, xcd = blockIdx.x % 8, w = xcd * (W / 8) + min(xcd, W % 8) + blockIdx.x / 8;
  const int64_t items = (int64_t)units * groups;
  int64_t item = items * w / W;
  const int64_t end = items * (w + 1) / W;
  while (item < end) {
    const int unit = __builtin_amdgcn_readfirstlane((int)(item / groups));
    const int g0 = __builtin_amdgcn_readfirstlane((int)(item - (int64_t)unit * groups));
    const int g1 = __builtin_amdgcn_readfirstlane((int)min((int64_t)groups, g0 + end - item));
    item += g1 - g0;
    const Unit<RB> u(g, unit, pick, false);
    if (u.n > 0 && (u.id >= 0 || g.out != g.y)) run(u, g0, g1);
    __syncthreads();
  }
}

template <int T, int RB, int NCB, int NB, bool PACK>
hipError_t request_one(const RequestArgs& g, int cus, hipStream_t s) {
  const int64_t units = request_units(g.M, g.L, g.r, !g.units);
  hipLaunchKernelGGL((request_down_kernel<T, RB, NCB>), dim3((unsigned)(units * g.splits)), dim3(kThreads), 0, s, g);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t items = units * ((g.N + 64 * kWaves - 1) / (64 * kWaves));
  const int64_t grid = RB == 1 ? items : std::min<int64_t>(items, 2 * (int64_t)cus);
  hipLaunchKernelGGL((request_up_kernel<T, RB, NB, PACK>), dim3((unsigned)grid), dim3(kThreads), 0, s, g, (int)units);
  return hipGetLastError();
}

}  // namespace

// Rows of a unit, in blocks of 16: more rows read an adapter's bytes less often, a small batch has
// few rows per adapter.
int request_rows(int32_t r, bool scan) { return scan ? 1 : (r > 64 ? 2 : 4); }

// An upper bound of a batch's units.
int64_t request_units(int64_t M, int32_t L, int32_t r, bool scan) {
  if (scan) return M;
  const int rows = 16 * request_rows(r, scan);
  return (M + rows - 1) / rows + std::min<int64_t>((int64_t)L + 1, M);
}

// Ranges that the first product's contraction is cut into, by the sizes alone (the sums, so the
// results, do not depend on the device): about two workgroups per CU, each of at least eight steps
// per wavefront, for the second product reads every range's sums again (96 rows, 4096 x 4096,
// rank 16: 16, 8, 4 ranges 4.5 + 8.6, 4.9 + 6.8, 5.1 + 5.6 us).
int request_splits(int64_t M, int64_t K, int32_t r) {
  const int rows = 16 * request_rows(r, M <= kRequestScan / 2);
  const int64_t blocks = (M + rows - 1) / rows, steps = (K + 31) / 32;
  return (int)std::max<int64_t>(1, std::min<int64_t>({512 / std::max<int64_t>(blocks, 1), steps / (8 * kWaves), 16}));
}

hipError_t launch_request_lora(const RequestArgs& g, int dtype, int cus, hipStream_t s) {
  const int rb = request_rows(g.r, !g.units), ncb = (g.r + 15) / 16;
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
    constexpr int T = decltype(t)::value, NCB = decltype(n)::value, NB = NCB <= 2 ? 1 : NCB / 2;
    if (rb == 1) return request_one<T, 1, NCB, NB, NCB == 1>(g, cus, s);
    return request_one<T, NCB <= 4 ? 4 : 2, NCB, NB, NCB == 1>(g, cus, s);
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
