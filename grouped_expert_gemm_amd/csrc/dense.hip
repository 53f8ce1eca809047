// Grouped products with 16-bit weights (bf16 or fp16), in each direction of training:
//     forward   out_e = a_e W_e^T          contracts over K   (a [M, K], W [E, N, K])
//     dgrad     dx_e  = dy_e W_e           contracts over N   (dy [M, N])
//     wgrad     dW_e  = dy_e^T a_e         contracts over the expert's rows
// for the rows of each expert e, grouped by `sizes`; products of 16-bit values are exact in
// fp32, sums run in fp32 and are rounded once.
//
// Each is a product D[r, c] = sum_k P[r, k] Q[c, k] of 256 x 256 tiles, and differs in how
// memory holds the operands: with the contraction along a row (a, dy of the dgrad, W of the
// forward: "along") or with a row per contraction index (W of the dgrad, both of the wgrad:
// "across").
#include <algorithm>

#include "geg_device.hpp"
#include "geg_launch.hpp"

namespace geg {

namespace {

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef __attribute__((address_space(3))) uint8_t lds_u8;

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

template <int N>
__device__ __forceinline__ void step_barrier() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | 0x0070);   // vmcnt(N), lgkmcnt(0)
  asm volatile("s_barrier" ::: "memory");
}

// Rows [row0, M) of a 16-bit matrix set to zero by the whole grid.
__device__ __forceinline__ void zero_rows(uint16_t* out, int64_t row0, int64_t M, int64_t width) {
  const int64_t n = (M - row0) * width, stride = (int64_t)gridDim.x * blockDim.x;
  uint16_t* p = out + row0 * width;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += stride) p[i] = 0;
}

// ------------------------------------------------------------------ tiles
constexpr int TM = 256, TN = 256, TK = 64;
constexpr int TThreads = 512;            // 8 wavefronts: 2 (rows of 128) x 4 (columns of 64)
constexpr int kStage = 256 * TK * 2;     // bytes of one operand per stage

// A stage of an operand held along its rows: 256 rows of 128 bytes, 16-byte chunk c of row r
// at c ^ (r % 8). Held across: 64 contraction rows of 512 bytes, 32-byte unit u of row r at
// u ^ h(r), h(r) = r % 4 + 4 (r / 8 % 2): the eight rows that 32 lanes of a transposing read
// touch at once (4 of lane group g, 4 of g + 1) then lie in different banks.
template <int D, int T>
struct Tiles {
  static constexpr bool kPAlong = D != kDenseWgrad, kQAlong = D == kDenseFwd;

  const DenseArgs& g;
  const int lane, wave;
  const int32_t* p_off;
  const int32_t* p_u;
  int64_t C, O;          // contraction width of P's memory rows (along), output width
  int pb, qb;            // wgrad: row blocks (of N) and column blocks (of K) of an expert

  struct Tile {
    const uint16_t* p;   // first element of the tile's P and Q
    const uint16_t* q;
    int64_t row0, c0;    // first row of the output matrix, first column
    int64_t n0;          // wgrad: first column of dy
    int rows, cols;      // valid
    int n;               // contraction length
    int stages;
  };

  __device__ __forceinline__ Tile tile_of(int32_t u) const {
    Tile x;
    if constexpr (D == kDenseWgrad) {
      const int e = u / (pb * qb), lu = u - e * (pb * qb);
      const int qi = lu / pb, pi = lu - qi * pb;
      const int32_t o0 = __builtin_amdgcn_readfirstlane(p_off[e]), o1 = __builtin_amdgcn_readfirstlane(p_off[e + 1]);
      const int64_t n0 = (int64_t)pi * TM, k0 = (int64_t)qi * TN;
      x.n0 = n0;
      x.p = g.p + (int64_t)o0 * g.N + n0;
      x.q = g.q + (int64_t)o0 * g.K + k0;
      x.row0 = (int64_t)e * g.N + n0;
      x.c0 = k0;
      x.rows = (int)min<int64_t>(TM, g.N - n0);
      x.cols = (int)min<int64_t>(TN, g.K - k0);
      x.n = o1 - o0;
    } else {
      const int e = __builtin_amdgcn_readfirstlane(find_expert(p_u, g.E, u));
      const int32_t lu = u - __builtin_amdgcn_readfirstlane(p_u[e]);
      const int32_t o0 = __builtin_amdgcn_readfirstlane(p_off[e]), o1 = __builtin_amdgcn_readfirstlane(p_off[e + 1]);
      const int rblocks = (o1 - o0 + TM - 1) / TM;
      const int ct = lu / rblocks, rt = lu - ct * rblocks;
      x.row0 = o0 + (int64_t)rt * TM;
      x.rows = (int)min<int64_t>(TM, o1 - x.row0);
      x.c0 = (int64_t)ct * TN;
      x.cols = (int)min<int64_t>(TN, O - x.c0);
      x.p = g.p + x.row0 * C;
      x.q = D == kDenseFwd ? g.q + ((int64_t)e * g.N + x.c0) * g.K : g.q + (int64_t)e * g.N * g.K + x.c0;
      x.n0 = 0;
      x.n = (int)C;
    }
    x.stages = max(1, (x.n + TK - 1) / TK);
    return x;
  }

  // Loads of a stage straight into LDS: 16 bytes per lane, 1 KB (8 rows along, 2 across) per
  // instruction, four per wavefront and operand; what lies past the tile's rows or the
  // contraction reads as zeros, columns past an across operand's as anything (they meet only
  // results that are not stored).
  __device__ __forceinline__ void along(const uint16_t* base, int rows, int64_t pitch, int n, int st, uint8_t* L) const {
    const int chunk = (lane & 7) ^ (lane >> 3);
    const __amdgpu_buffer_rsrc_t R = window(base + (int64_t)st * TK, (rows * pitch - (int64_t)st * TK) * 2);
    const uint32_t at = (uint32_t)((8 * wave + (lane >> 3)) * (uint32_t)pitch * 2 + 16 * chunk), next = 128 * (uint32_t)pitch;
    const uint32_t off = oob_unless(st * TK + 8 * chunk < n, at);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(R, (lds_ptr_t)(L + (wave + 8 * i) * 1024), 16, off + i * next, 0, 0, 0);
  }
  __device__ __forceinline__ void across(const uint16_t* base, int64_t col0, int64_t pitch, int n, int st,
                                         uint8_t* L) const {
    const int r = 2 * wave + (lane >> 5);
    const int h = (r & 3) | ((r >> 1) & 4);
    const int chunk = (lane & 31) ^ (2 * h);
    const int rows = min(TK, n - st * TK);
    const __amdgpu_buffer_rsrc_t R = window(base + (int64_t)st * TK * pitch, rows > 0 ? (rows * pitch - col0) * 2 : 0);
    const uint32_t off = (uint32_t)(r * (uint32_t)pitch * 2 + 16 * chunk), next = 32 * (uint32_t)pitch;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(R, (lds_ptr_t)(L + (wave + 8 * i) * 1024), 16, off + i * next, 0, 0, 0);
  }
  __device__ __forceinline__ void load(const Tile& x, bool any, int st, uint8_t* P, uint8_t* Q) const {
    if constexpr (kPAlong)
      along(x.p, any ? x.rows : 0, C, x.n, st, P);
    else
      across(x.p, x.n0, g.N, any ? x.n : 0, st, P);
    if constexpr (kQAlong)
      along(x.q, any ? x.cols : 0, g.K, x.n, st, Q);
    else
      across(x.q, x.c0, g.K, any ? x.n : 0, st, Q);
  }
};

template <bool ALONG>
struct Frag {
  uint32_t at;
  // block0: the first of the operand's 16-wide blocks that the wavefront reads
  __device__ __forceinline__ Frag(int lane, int block0) {
    const int r16 = lane & 15, grp = lane >> 4;
    if constexpr (ALONG) {
      at = (uint32_t)((16 * block0 + r16) * 128 + ((grp ^ (r16 & 7)) << 4));
    } else {
      const int j = r16 >> 2, h = j | ((grp & 1) << 2);
      at = (uint32_t)((8 * grp + j) * 512 + ((block0 ^ h) << 5) + ((r16 & 3) << 3));
    }
  }
  // Block i (of the wavefront's), 32-wide substep q of the stage.
  __device__ __forceinline__ u32x4 read(const uint8_t* L, int i, int q) const {
    if constexpr (ALONG) {
      return *reinterpret_cast<const u32x4*>(L + (at ^ (64 * q)) + 2048 * i);
    } else {
      const uint8_t* p = L + (at ^ (32 * i)) + 16384 * q;
      const u32x2 lo = tr(p), hi = tr(p + 2048);
      return u32x4{lo[0], lo[1], hi[0], hi[1]};
    }
  }
  static __device__ __forceinline__ u32x2 tr(const uint8_t* p) {
    const i16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)(lds_u8*)p);
    return __builtin_bit_cast(u32x2, v);
  }
};

template <int D, int T, bool F32>
__global__ __launch_bounds__(TThreads, 1) void dense_tile_kernel(DenseArgs g) {
  __shared__ int32_t p_off[kMaxExperts + 1];
  __shared__ int32_t p_u[kMaxExperts + 1];
  __shared__ __attribute__((aligned(16))) uint8_t pa[kStage];
  __shared__ __attribute__((aligned(16))) uint8_t pb[kStage];
  __shared__ __attribute__((aligned(16))) uint8_t qa[kStage];
  __shared__ __attribute__((aligned(16))) uint8_t qb[kStage];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int r16 = lane & 15, grp = lane >> 4;
  using W = Tiles<D, T>;
  const int64_t O = D == kDenseFwd ? g.N : g.K;
  const int blocks_n = (int)((g.N + TM - 1) / TM), blocks_k = (int)((g.K + TN - 1) / TN);
  const int c_tiles = (int)((O + TN - 1) / TN);
  int32_t total = build_plan(p_off, p_u, g.sizes, g.E, g.M, g.err,
                             [&](int32_t s) -> int32_t { return D == kDenseWgrad ? 0 : (s + TM - 1) / TM * c_tiles; });
  if constexpr (D == kDenseWgrad) total = g.E * blocks_n * blocks_k;
  if constexpr (D != kDenseWgrad) {
    if (g.zero_rest) zero_rows((uint16_t*)g.out, p_off[g.E], g.M, O);
  }
  const W w{g, lane, wave, p_off, p_u, D == kDenseDgrad ? g.N : g.K, O, blocks_n, blocks_k};
  // each XCD its own run of tiles
  const int G = gridDim.x;
  const int parts = G % 8 == 0 ? 8 : 1, step = G / parts, part = blockIdx.x % parts;
  const int32_t end = (int32_t)((int64_t)total * (part + 1) / parts);
  int32_t u = (int32_t)((int64_t)total * part / parts) + blockIdx.x / parts;
  if (u >= end) return;

  const Frag<W::kPAlong> fp(lane, 8 * wm);
  const Frag<W::kQAlong> fq(lane, 4 * wn);
  u32x4 q[2][4], plo[4], phi[4];
  f32x4 acc[8][4];
  auto read_q = [&](const uint8_t* L, int s, u32x4* d) {
#pragma unroll
    for (int j = 0; j < 4; ++j) d[j] = fq.read(L, j, s);
  };
  auto read_p = [&](const uint8_t* L, int i0, int s, u32x4* d) {
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = fp.read(L, i0 + i, s);
  };

  // The loads run two stages ahead of the products, across tiles: their own place in the list.
  typename W::Tile lt = w.tile_of(u), cur = lt;
  int32_t lu = u;
  int lst = 0;
  bool lany = true;
  auto load_next = [&](uint8_t* P, uint8_t* Q) {
    w.load(lt, lany, lst, P, Q);
    if (++lst == lt.stages) {
      lst = 0;
      lu += step;
      lany = lu < end;
      if (lany) lt = w.tile_of(lu);
    }
  };
  load_next(pa, qa);
  load_next(pb, qb);
  step_barrier<8>();
  read_q(qa, 0, q[0]);
  read_p(pa, 0, 0, plo);

  int st = 0;
  bool lo, hi;
  auto begin = [&]() {
    lo = 128 * wm < cur.rows && 64 * wn < cur.cols;
    hi = 128 * wm + 64 < cur.rows && 64 * wn < cur.cols;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  };
  auto multiply = [&](int i0, const u32x4* p, const u32x4* qq) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i0 + i][j] = mfma<T>(qq[j], p[i], acc[i0 + i][j]);
  };
  auto store = [&]() {
    if (!lo) return;
    if constexpr (F32) {
      float* dst = reinterpret_cast<float*>(g.out) + (cur.row0 + 128 * wm + r16) * O + cur.c0 + 64 * wn + 4 * grp;
      const int rows = cur.rows - 128 * wm - r16, left = cur.cols - 64 * wn - 4 * grp;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (16 * i < rows && 16 * j < left) *reinterpret_cast<f32x4*>(dst + (int64_t)(16 * i) * O + 16 * j) = acc[i][j];
    } else {
      // lane groups 0, 2 end up with columns 0-7, 8-15 of block j, groups 1, 3 of block j + 1
      const bool wide = (O & 7) == 0;
      const int col = 16 * (grp & 1) + 8 * (grp >> 1);
      uint16_t* dst = reinterpret_cast<uint16_t*>(g.out) + (cur.row0 + 128 * wm + r16) * O + cur.c0 + 64 * wn + col;
      const int rows = cur.rows - 128 * wm - r16, left = cur.cols - 64 * wn - col;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          u32x4 v;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x = pack2<T>(acc[i][j][2 * h], acc[i][j][2 * h + 1]);
            const uint32_t y = pack2<T>(acc[i][j + 1][2 * h], acc[i][j + 1][2 * h + 1]);
            const auto r = __builtin_amdgcn_permlane16_swap(x, y, false, false);
            v[h] = r[0];
            v[2 + h] = r[1];
          }
          if (16 * i < rows && 16 * j < left) {
            uint16_t* d = dst + (int64_t)(16 * i) * O + 16 * j;
            if (wide) {
              *reinterpret_cast<u32x4*>(d) = v;
            } else {
#pragma clang loop unroll(disable)
              for (int b = 0; b < min(8, left - 16 * j); ++b) {
                const uint32_t x = b < 4 ? (b < 2 ? v[0] : v[1]) : (b < 6 ? v[2] : v[3]);
                d[b] = (uint16_t)(x >> (16 * (b & 1)));
              }
            }
          }
        }
      }
    }
  };
  // One stage from buffers P, Q, the next one's in P1, Q1. Behind the last tile an odd one out
  // runs without products: a way out between the two copies of this body would, to the
  // compiler, lead back to the first, which then waits for all loads.
  bool more = true;
  auto stage = [&](uint8_t* P, uint8_t* Q, const uint8_t* P1, const uint8_t* Q1) {
    read_p(P, 4, 0, phi);
    if (lo) multiply(0, plo, q[0]);
    __builtin_amdgcn_sched_barrier(0);
    read_q(Q, 1, q[1]);
    read_p(P, 0, 1, plo);
    if (hi) multiply(4, phi, q[0]);
    __builtin_amdgcn_sched_barrier(0);
    read_p(P, 4, 1, phi);
    if (lo) multiply(0, plo, q[1]);
    __builtin_amdgcn_sched_barrier(0);
    // every read of this stage is done and the next one's loads have landed
    step_barrier<0>();
    read_q(Q1, 0, q[0]);
    read_p(P1, 0, 0, plo);
    load_next(P, Q);
    if (hi) multiply(4, phi, q[1]);
    __builtin_amdgcn_sched_barrier(0);
    if (++st == cur.stages) {
      store();
      u += step;
      st = 0;
      more = u < end;
      if (more) {
        cur = w.tile_of(u);
      } else {
        cur.rows = 0;
        cur.stages = 2;
      }
      begin();
    }
  };
  begin();
  do {
    stage(pa, qa, pb, qb);
    stage(pb, qb, pa, qa);
  } while (more);
  __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0): no load into LDS outlives the workgroup
}

// ------------------------------------------------------------------ forward, few rows
// A unit is 16 output columns of one expert and up to 16 RB of its rows over the whole
// contraction; the wavefront streams the 16 weight rows from memory into registers, PD steps
// of 32 k ahead, and reads the activations beside them (rows past the expert's cost nothing).
constexpr int NThreads = 256, NWaves = NThreads / 64;

template <int T, int RB, int PD>
__global__ __launch_bounds__(NThreads) void dense_narrow_kernel(DenseArgs g) {
  __shared__ int32_t p_off[kMaxExperts + 1];
  __shared__ int32_t p_u[kMaxExperts + 1];
  const int64_t K = g.K, N = g.N;
  const int nblk = (int)((N + 15) / 16);
  const int32_t total = build_plan(p_off, p_u, g.sizes, g.E, g.M, g.err, [&](int32_t s) -> int32_t {
    return (s + 16 * RB - 1) / (16 * RB) * nblk;
  });
  if (g.zero_rest) zero_rows((uint16_t*)g.out, p_off[g.E], g.M, N);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, grp = lane >> 4;
  const int steps = (int)((K + 31) / 32), batches = (steps + PD - 1) / PD;
  const int stride = gridDim.x * NWaves;

  struct Unit {
    __amdgpu_buffer_rsrc_t W, A;
    int64_t row0, n0;
    int rows;
  };
  auto unit_of = [&](int u, bool any) {
    Unit x;
    const int e = any ? __builtin_amdgcn_readfirstlane(find_expert(p_u, g.E, u)) : 0;
    const int32_t lu = any ? u - __builtin_amdgcn_readfirstlane(p_u[e]) : 0;
    const int chunk = lu / nblk;
    const int32_t o0 = __builtin_amdgcn_readfirstlane(p_off[e]), o1 = __builtin_amdgcn_readfirstlane(p_off[e + 1]);
    x.n0 = 16 * (int64_t)(lu - chunk * nblk);
    x.row0 = o0 + (int64_t)chunk * 16 * RB;
    x.rows = (int)min<int64_t>(16 * RB, o1 - x.row0);
    x.W = window(g.q + ((int64_t)e * N + x.n0) * K, any ? min<int64_t>(16, N - x.n0) * K * 2 : 0);
    x.A = window(g.p + x.row0 * K, any ? x.rows * K * 2 : 0);
    return x;
  };
  u32x4 wf[PD], af[PD][RB];
  const uint32_t at = (uint32_t)(r16 * K * 2 + 16 * grp);
  auto load = [&](int i, const Unit& x, int s) {
    const uint32_t off = oob_unless(32 * (int64_t)s + 8 * grp < K, at + 64 * (uint32_t)s);
    wf[i] = __builtin_amdgcn_raw_buffer_load_b128(x.W, off, 0, 0);
#pragma unroll
    for (int b = 0; b < RB; ++b) af[i][b] = __builtin_amdgcn_raw_buffer_load_b128(x.A, off + b * 32 * (uint32_t)K, 0, 0);
  };
  int u = blockIdx.x * NWaves + wave;
  if (u >= total) return;
  Unit cur = unit_of(u, true);
#pragma unroll
  for (int i = 0; i < PD; ++i) load(i, cur, i);
  for (; u < total; u += stride) {
    const Unit nxt = unit_of(u + stride, u + stride < total);
    f32x4 acc[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int c = 0; c < batches; ++c) {
      const bool last = c + 1 == batches;
      const Unit from = last ? nxt : cur;
      const int s0 = last ? 0 : (c + 1) * PD;
#pragma unroll
      for (int i = 0; i < PD; ++i) {
#pragma unroll
        for (int b = 0; b < RB; ++b) acc[b] = mfma<T>(wf[i], af[i][b], acc[b]);
        load(i, from, s0 + i);
      }
    }
    const int64_t n = cur.n0 + 4 * grp;
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int r = 16 * b + r16;
      if (r < cur.rows) {
        uint16_t* dst = reinterpret_cast<uint16_t*>(g.out) + (cur.row0 + r) * N + n;
        const u32x2 v = u32x2{pack2<T>(acc[b][0], acc[b][1]), pack2<T>(acc[b][2], acc[b][3])};
        if ((N & 3) == 0) {
          if (n < N) *reinterpret_cast<u32x2*>(dst) = v;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (n + i < N) dst[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
        }
      }
    }
    cur = nxt;
  }
}

template <int T, int RB, int PD>
hipError_t narrow_one(const DenseArgs& g, int cus, hipStream_t s) {
  const int64_t units = ((g.M + 16 * RB - 1) / (16 * RB) + std::min<int64_t>(g.E, g.M)) * ((g.N + 15) / 16);
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>((units + NWaves - 1) / NWaves, (int64_t)cus * 4));
  hipLaunchKernelGGL((dense_narrow_kernel<T, RB, PD>), dim3((unsigned)grid), dim3(NThreads), 0, s, g);
  return hipGetLastError();
}

template <int D, int T, bool F32>
hipError_t tile_one(const DenseArgs& g, int cus, hipStream_t s) {
  const int64_t bn = (g.N + TM - 1) / TM, bk = (g.K + TN - 1) / TN;
  const int64_t bound = D == kDenseWgrad ? g.E * bn * bk
                                         : ((g.M + TM - 1) / TM + std::min<int64_t>(g.E, g.M)) * (D == kDenseFwd ? bn : bk);
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(bound, (int64_t)cus));
  hipLaunchKernelGGL((dense_tile_kernel<D, T, F32>), dim3((unsigned)grid), dim3(TThreads), 0, s, g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dense_tile(int dir, int dtype, bool f32_out, const DenseArgs& g, int cus, hipStream_t s) {
  const bool b = dtype == kBF16;
  if (dir == kDenseFwd) return b ? tile_one<kDenseFwd, kBF16, false>(g, cus, s) : tile_one<kDenseFwd, kF16, false>(g, cus, s);
  if (dir == kDenseDgrad)
    return b ? tile_one<kDenseDgrad, kBF16, false>(g, cus, s) : tile_one<kDenseDgrad, kF16, false>(g, cus, s);
  if (f32_out) return b ? tile_one<kDenseWgrad, kBF16, true>(g, cus, s) : tile_one<kDenseWgrad, kF16, true>(g, cus, s);
  return b ? tile_one<kDenseWgrad, kBF16, false>(g, cus, s) : tile_one<kDenseWgrad, kF16, false>(g, cus, s);
}

hipError_t launch_dense_narrow(int dtype, const DenseArgs& g, int cus, hipStream_t s) {
  const int64_t avg = (g.M + g.E - 1) / g.E;
  auto run = [&](auto t) {
    constexpr int T = decltype(t)::value;
    return avg <= 8 ? narrow_one<T, 1, 8>(g, cus, s) : narrow_one<T, 2, 4>(g, cus, s);
  };
  return dtype == kBF16 ? run(std::integral_constant<int, kBF16>{}) : run(std::integral_constant<int, kF16>{});
}

}  // namespace geg
