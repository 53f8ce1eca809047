// Grouped products with 16-bit weights (bf16 or fp16), in each direction of training:
//     forward   out_e = a_e W_e^T          contracts over K   (a [M, K], W [E, N, K])
//     dgrad     dx_e  = dy_e W_e           contracts over N   (dy [M, N])
//     wgrad     dW_e  = dy_e^T a_e         contracts over the expert's rows
// for the rows of each expert e, grouped by `sizes`; products of 16-bit values are exact in
// fp32, sums run in fp32 and are rounded once.
//
// Each is a product D[r, c] = sum_k P[r, k] Q[c, k] in tiles of 256 x 256 or 128 x 128, and differs in how
// memory holds the operands: with the contraction along a row (a, dy of the dgrad, W of the
// forward: "along") or with a row per contraction index (W of the dgrad, both of the wgrad:
// "across").
#include <algorithm>

#include "geg_device.hpp"
#include "geg_launch.hpp"
#include "wide16.hpp"

namespace geg {

namespace {

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef __attribute__((address_space(3))) uint8_t lds_u8;

template <int N>
__device__ __forceinline__ void step_barrier() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | 0x0070);   // vmcnt(N), lgkmcnt(0)
  asm volatile("s_barrier" ::: "memory");
}

// The lane's number, worked out where it is used: kept in a register over a tile's stages, it (and
// what follows from it) would cost registers that they need.
__device__ __forceinline__ int fresh_lane() {
  int l = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
  asm volatile("" : "+v"(l));
  return l;
}

// Blocks of d that hold n rows, n up to the largest int32.
__device__ __forceinline__ int32_t blocks_of(int32_t n, int32_t d) { return (int32_t)(((uint32_t)n + (uint32_t)d - 1) / (uint32_t)d); }

// Rows [row0, M) of a 16-bit matrix set to zero by the whole grid.
__device__ __forceinline__ void zero_rows(uint16_t* out, int64_t row0, int64_t M, int64_t width) {
  const int64_t n = (M - row0) * width, stride = (int64_t)gridDim.x * blockDim.x;
  uint16_t* p = out + row0 * width;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += stride) p[i] = 0;
}

// ------------------------------------------------------------------ tiles
constexpr int TK = 64;
constexpr int TThreads = 512;            // 8 wavefronts: per 128 x 128 results 4 (rows of 32) x 2 (columns of 64)
constexpr int kHalf = 128 * TK * 2;      // bytes of half an operand per stage

// Half an operand's stage, 128 rows (columns) of the tile by 64 of the contraction. Held along
// its rows: 128 rows of 128 bytes, 16-byte chunk c of row r at c ^ (r % 8). Held across: 64
// contraction rows of 256 bytes, 32-byte unit u of row r at u ^ h(r), h(r) = r % 4 + 4 (r / 8 %
// 2): the eight rows that 32 lanes of a transposing read touch at once (4 of lane group g, 4 of
// g + 1) then lie in different banks. Neither meets a bank conflict.
template <int D, int S>
struct Tiles {
  static constexpr int TM = S, TN = S;
  static constexpr int kRing = S == 256 ? 2 : 4;   // sets of buffers
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
    int k0;              // where the contraction starts (a piece of it)
    int stages;          // a multiple of the sets of buffers
  };

  __device__ __forceinline__ Tile tile_of(int32_t u) const {
    Tile x;
    if constexpr (D == kDenseWgrad) {
      // (divisions run on the vector ALUs)
      const int e = __builtin_amdgcn_readfirstlane(u / (pb * qb)), lu = u - e * (pb * qb);
      const int qi = __builtin_amdgcn_readfirstlane(lu / pb), pi = lu - qi * pb;
      const int32_t o0 = __builtin_amdgcn_readfirstlane(p_off[e]), o1 = __builtin_amdgcn_readfirstlane(p_off[e + 1]);
      const int64_t n0 = (int64_t)pi * TM, k0 = (int64_t)qi * TN;
      x.n0 = n0;
      x.p = g.p + (int64_t)o0 * g.N + n0;
      x.q = g.q + (int64_t)o0 * g.K + k0;
      x.row0 = (int64_t)e * g.N + n0;
      x.c0 = k0;
      x.rows = min(TM, (int)(g.N - n0));
      x.cols = min(TN, (int)(g.K - k0));
      x.n = o1 - o0;
    } else {
      const int e = __builtin_amdgcn_readfirstlane(find_expert(p_u, g.E, u, fresh_lane()));
      const int32_t lu = u - __builtin_amdgcn_readfirstlane(p_u[e]);
      const int32_t o0 = __builtin_amdgcn_readfirstlane(p_off[e]), o1 = __builtin_amdgcn_readfirstlane(p_off[e + 1]);
      const int rblocks = blocks_of(o1 - o0, TM);
      const int ct = __builtin_amdgcn_readfirstlane(lu / rblocks), rt = lu - ct * rblocks;   // (vector ALUs)
      x.row0 = o0 + (int64_t)rt * TM;
      x.rows = min(TM, o1 - o0 - rt * TM);
      x.c0 = (int64_t)ct * TN;
      x.cols = min(TN, (int)(O - x.c0));
      x.p = g.p + x.row0 * C;
      x.q = D == kDenseFwd ? g.q + ((int64_t)e * g.N + x.c0) * g.K : g.q + (int64_t)e * g.N * g.K + x.c0;
      x.n0 = 0;
      x.n = (int)C;
    }
    x.k0 = 0;
    x.stages = stages_of(x.n);
    return x;
  }
  static __device__ __forceinline__ int stages_of(int n) { return max(kRing, kRing * blocks_of(n, kRing * TK)); }
  // Piece `i` of `split` of a tile's contraction, in whole stages.
  __device__ __forceinline__ Tile piece_of(int32_t u, int split) const {
    const int32_t t = __builtin_amdgcn_readfirstlane(u / split);   // (vector ALUs)
    const int i = u - t * split;
    Tile x = tile_of(t);
    const int len = __builtin_amdgcn_readfirstlane((blocks_of(x.n, TK) + split - 1) / split) * TK;
    x.k0 = min(i * len, x.n);
    x.n = min(len, x.n - x.k0);
    x.p += x.k0 * (kPAlong ? 1 : g.N);
    x.q += x.k0 * (kQAlong ? 1 : g.K);
    x.stages = stages_of(x.n);
    return x;
  }

  // The place of the loads: the memory of P's and Q's next stage and what is left of it.
  struct Cursor {
    const uint8_t* p;
    const uint8_t* q;
    int64_t left_p, left_q;
    int rest;            // contraction left
    int st, stages;
  };
  __device__ __forceinline__ void aim(Cursor& c, const Tile& x, bool any) const {
    c.p = reinterpret_cast<const uint8_t*>(x.p);
    c.left_p = !any ? 0 : (kPAlong ? x.rows * C - x.k0 : x.n * g.N - x.n0) * 2;
    c.q = reinterpret_cast<const uint8_t*>(x.q);
    c.left_q = !any ? 0 : (kQAlong ? x.cols * g.K - x.k0 : x.n * g.K - x.c0) * 2;
    c.rest = x.n;
    c.st = 0;
    c.stages = x.stages;
  }
  __device__ __forceinline__ void next(Cursor& c) const {
    const int64_t dp = kPAlong ? TK * 2 : TK * g.N * 2, dq = kQAlong ? TK * 2 : TK * g.K * 2;
    c.p += dp;
    c.left_p -= dp;
    c.q += dq;
    c.left_q -= dq;
    c.rest -= TK;
    ++c.st;
  }

  // Loads of half an operand's stage straight into LDS: 16 bytes per lane, 1 KB (8 rows along,
  // 4 across) per instruction, two per wavefront; what lies past the tile's rows or the
  // contraction reads as zeros, columns past an across operand's as anything (they meet only
  // results that are not stored).
  static __device__ __forceinline__ uint32_t lane_at(bool along, int lane, int wave, int64_t pitch) {
    if (along) return (uint32_t)((8 * wave + (lane >> 3)) * (uint32_t)pitch * 2 + 16 * ((lane & 7) ^ (lane >> 3)));
    const int r = 4 * wave + (lane >> 4), h = (r & 3) | ((r >> 1) & 4);
    return (uint32_t)(r * (uint32_t)pitch * 2 + 16 * ((lane & 15) ^ (2 * h)));
  }
  // Instruction i of half h.
  template <bool ALONG>
  __device__ __forceinline__ void load(const uint8_t* base, int64_t left, int rest, uint32_t at, int64_t pitch, int h, int i,
                                       uint8_t* L) const {
    const int64_t skip = h * (ALONG ? 256 * pitch : 256);
    const __amdgpu_buffer_rsrc_t R = window(base + skip, left - skip);
    if constexpr (ALONG) at = oob_unless(8 * ((lane & 7) ^ (lane >> 3)) < rest, at);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(R, (lds_ptr_t)(L + (wave + 8 * i) * 1024), 16,
                                             at + i * ((ALONG ? 128 : 64) * (uint32_t)pitch), 0, 0, 0);
  }
};

template <bool ALONG>
struct Frag {
  uint32_t at;
  // block0: the first of the half's 16-wide blocks that the wavefront reads
  __device__ __forceinline__ Frag(int lane, int block0) {
    const int r16 = lane & 15, grp = lane >> 4;
    if constexpr (ALONG) {
      at = (uint32_t)((16 * block0 + r16) * 128 + ((grp ^ (r16 & 7)) << 4));
    } else {
      const int j = r16 >> 2, h = j | ((grp & 1) << 2);
      at = (uint32_t)((8 * grp + j) * 256 + ((block0 ^ h) << 5) + ((r16 & 3) << 3));
    }
  }
  // Block i (of the wavefront's), 32-wide substep q of the stage.
  __device__ __forceinline__ u32x4 read(const uint8_t* L, int i, int q) const {
    if constexpr (ALONG) {
      return *reinterpret_cast<const u32x4*>(L + (at ^ (64 * q)) + 2048 * i);
    } else {
      const uint8_t* p = L + (at ^ (32 * i)) + 8192 * q;
      const u32x2 lo = tr(p), hi = tr(p + 1024);
      return u32x4{lo[0], lo[1], hi[0], hi[1]};
    }
  }
  static __device__ __forceinline__ u32x2 tr(const uint8_t* p) {
    const i16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)(lds_u8*)p);
    return __builtin_bit_cast(u32x2, v);
  }
};

// Cache policy of the tiles' stores: streamed past the XCD's L2, where they would displace the
// operands that its tiles share (non-temporal, system scope). Both gradients of 1200 rows over 32
// experts of 2880 x 2880, the weights' in fp32: 387 us without, 346 with; of 16384 rows over 64 of 2048 x
// 2048, 16 bits: 432, 409.
constexpr int kStream = 18;

// How results are stored: 16 bits in rows of whole 16-byte pieces, fp32, or 16 bits in rows of any
// width, value by value (forward; a tile's stores are waited for before the next tile: one column less
// than 5760 in 3108 rows over 32 experts of 2880 238 us for 217, than 14336 in 4096 over 8 of 4096 547 for
// 463; the narrow kernel and tiles of 128 with one row per expert lose nothing).
enum Out : int { kWide = 0, kF32Out = 1, kAnyWidth = 2 };
// Stores per wavefront of 128 x 128 results (what lies past the rows and columns is dropped by the
// window); value by value, none is left in flight.
template <int OUT>
constexpr int kQuadrantStores = OUT == kAnyWidth ? 0 : OUT == kF32Out ? 8 : 4;

// 16 of a wavefront's 32 x 64 of 128 x 128 results, row block i: output rows from row0 (rows of them
// valid), columns from c0 + cv, of cols from c0.
template <int T, int OUT>
__device__ __forceinline__ void store_block(void* out, int64_t O, int64_t row0, int64_t c0, int rows, int cv, int cols, int wm,
                                            int wn, int i, const f32x4 (&acc)[4]) {
  constexpr bool F32 = OUT == kF32Out;
  const int l = fresh_lane();
  const int r16 = l & 15, grp = l >> 4;
  if constexpr (OUT == kAnyWidth) {
    const int left = rows - 32 * wm - r16, c = cv + 64 * wn + 4 * grp;
    uint16_t* dst = reinterpret_cast<uint16_t*>(out) + (row0 + 32 * wm + r16) * O + c0 + c;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (16 * i < left && 16 * j + b < cols - c)
          dst[(int64_t)(16 * i) * O + 16 * j + b] = (uint16_t)pack2<T>(acc[j][b], 0.f);
    return;
  }
  // Whole 128-byte lines: a lane has 16 bytes of its row in each of two 64-byte halves (16
  // bits: of two pairs of column blocks, whose rows of 16 lanes have traded places); the lanes of
  // rows 8-15 and 0-7 of the block trade a half, and a store then writes 8 rows of 128 bytes.
  constexpr int size = F32 ? 4 : 2;
  const bool low = r16 < 8;
  const int col = (F32 ? 4 * grp : 16 * (grp & 1) + 8 * (grp >> 1)) + (low ? 0 : F32 ? 16 : 32);
  const __amdgpu_buffer_rsrc_t R =
      window(reinterpret_cast<uint8_t*>(out) + (row0 * O + c0) * size, rows > 0 ? (rows * O - c0) * size : 0);
  const uint32_t row = (uint32_t)(32 * wm + (r16 & 7)) * (uint32_t)O * size;
#pragma unroll
  for (int j = 0; j < 4; j += F32 ? 2 : 4) {
    u32x4 a, b;
    if constexpr (F32) {
      a = __builtin_bit_cast(u32x4, acc[j]);
      b = __builtin_bit_cast(u32x4, acc[j + 1]);
    } else {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        auto two = [&](int jj) { return pack2<T>(acc[jj][2 * x], acc[jj][2 * x + 1]); };
        const auto r = __builtin_amdgcn_permlane16_swap(two(0), two(1), false, false);
        const auto s = __builtin_amdgcn_permlane16_swap(two(2), two(3), false, false);
        a[x] = r[0];
        a[2 + x] = r[1];
        b[x] = s[0];
        b[2 + x] = s[1];
      }
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const uint32_t give = low ? b[x] : a[x];
      const uint32_t got = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)give, 0x128, 0xF, 0xF, true);   // row_ror:8
      a[x] = low ? a[x] : got;
      b[x] = low ? got : b[x];
    }
    const int c = cv + 64 * wn + 16 * j + col;
    const uint32_t at = row + (uint32_t)(16 * i) * (uint32_t)O * size + c * size;
    __builtin_amdgcn_raw_buffer_store_b128(a, R, oob_unless(c < cols, at), 0, kStream);
    __builtin_amdgcn_raw_buffer_store_b128(b, R, oob_unless(c < cols, at + 8 * (uint32_t)O * size), 0, kStream);
  }
}

template <int T, int OUT>
__device__ __forceinline__ void store_quadrant(void* out, int64_t O, int64_t row0, int64_t c0, int rows, int cv, int cols, int wm,
                                               int wn, const f32x4 (&acc)[2][4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) store_block<T, OUT>(out, O, row0, c0, rows, cv, cols, wm, wn, i, acc[i]);
}

// One workgroup per CU, persistent over tiles. A stage is four quadrants of 128 x 128 results,
// P half h by Q half v, in the order (0, 0), (1, 0), (0, 1), (1, 1), of 16 instructions per
// wavefront each (32 x 64 results). Fragments are read a little ahead of their products, so a
// half of an operand is needed in LDS for half a stage only; its buffer then takes the stage
// after the next, and the loads have one and a half stages to land. Reads and loads stand between
// the products, four at a time. A load into LDS takes 16 clocks of the CU's one path from the L2 and
// holds its wavefront up while that is busy, so there is at most one per wavefront between four products
// and the next four (in twos and threes: 4% slower with all CUs at work, 10% with half). The loads run on
// across tiles, at their own place in the list.
// Measured: 8192 rows over 8 experts of 28672 x 4096 1.47 ms with 1024 each, 1.31 PFLOP/s, 1.63 ms with the
// sizes that a router gives (to 1.74 on other cards; a library product of that many rows by one such expert: 1.33 to 1.48): an
// expert's last row block of 6 rows costs 0.4 of a whole one. LDS is as busy as the matrix pipes: 192 KB of
// fragments and 64 KB of loads per stage, 2048 clocks, as 2048 of products; a stage takes 1.24 us on
// one CU in eight at 2.4 GHz and 1.7 on all at 1.8. (Four wavefronts of 128 x 128 read a third less
// and were slower, 1.36 and 1.9: alone on its SIMD a wavefront's loads hold its products up.) 3108 rows
// over 32 experts of 5760 x 2880 210 to 219 us, 1.1 GB at 5.2 TB/s. 16384 rows over 64 of 2048 x 2048, both
// gradients one after the other, 406 to 432 us: tiles of four stages in the weights', whose bursts of stores the
// next tile's loads wait behind (with the stores dropped it takes 184 of its 270), and whose contraction, an
// expert's rows, is rounded up to two stages (257 rows run six of 64).
template <int D, int T, int OUT>
__global__ __launch_bounds__(TThreads, 1) void dense_tile_kernel(DenseArgs g) {
  __shared__ int32_t p_off[kMaxExperts + 1];
  __shared__ int32_t p_u[kMaxExperts + 1];
  // distinct objects, named at compile time: the compiler then adds no wait for loads that fill
  // the others
  // (placed by alignment: each operand's 64 KB together, within reach of one address register)
  __shared__ __attribute__((aligned(128))) uint8_t qa0[kHalf], qa1[kHalf], qb0[kHalf], qb1[kHalf];
  __shared__ __attribute__((aligned(64))) uint8_t pa0[kHalf], pa1[kHalf], pb0[kHalf], pb1[kHalf];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  using W = Tiles<D, 256>;
  constexpr int TM = W::TM, TN = W::TN;
  const int64_t O = D == kDenseFwd ? g.N : g.K;
  const int blocks_n = (int)((g.N + TM - 1) / TM), blocks_k = (int)((g.K + TN - 1) / TN);
  const int c_tiles = (int)((O + TN - 1) / TN);
  int32_t total = build_plan(p_off, p_u, g.sizes, g.E, g.M, g.err,
                             [&](int32_t s) -> int32_t { return D == kDenseWgrad ? 0 : blocks_of(s, TM) * c_tiles; });
  total = D == kDenseWgrad ? g.E * blocks_n * blocks_k : __builtin_amdgcn_readfirstlane(total);
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

  const Frag<W::kPAlong> fp(lane, 2 * wm);
  const Frag<W::kQAlong> fq(lane, 4 * wn);
  u32x4 q[2][4], p0[2][2], p1[2][2];   // [substep][block] of one Q half and of both P halves
  f32x4 acc[2][2][2][4];

  typename W::Tile cur = w.tile_of(u);   // of the products
  typename W::Cursor lc;                 // of the loads
  w.aim(lc, cur, true);
  int32_t lu = u;
  const int64_t pitch_p = W::kPAlong ? w.C : g.N;
  const uint32_t at_p = W::lane_at(W::kPAlong, lane, wave, pitch_p), at_q = W::lane_at(W::kQAlong, lane, wave, g.K);
  auto load_p = [&](int h, int i, uint8_t* L) {
    w.template load<W::kPAlong>(lc.p, lc.left_p, lc.rest, at_p, pitch_p, h, i, L);
  };
  auto load_q = [&](int h, int i, uint8_t* L) {
    w.template load<W::kQAlong>(lc.q, lc.left_q, lc.rest, at_q, g.K, h, i, L);
  };
  auto advance = [&]() {
    w.next(lc);
    if (lc.st == lc.stages) {
      lu += step;
      const bool any = lu < end;
      w.aim(lc, any ? w.tile_of(lu) : cur, any);
    }
  };
  auto load_all = [&](uint8_t* P0, uint8_t* P1, uint8_t* Q0, uint8_t* Q1) {
#pragma unroll
    for (int i = 0; i < 2; ++i) load_q(0, i, Q0);
#pragma unroll
    for (int i = 0; i < 2; ++i) load_p(0, i, P0);
#pragma unroll
    for (int i = 0; i < 2; ++i) load_p(1, i, P1);
#pragma unroll
    for (int i = 0; i < 2; ++i) load_q(1, i, Q1);
    advance();
  };
  load_all(pa0, pa1, qa0, qa1);
  load_all(pb0, pb1, qb0, qb1);
  step_barrier<10>();
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int i = 0; i < 2; ++i) p0[s][i] = fp.read(pa0, i, s);
#pragma unroll
  for (int j = 0; j < 4; ++j) q[0][j] = fq.read(qa0, j, 0);

  int on;   // bit 2 h + v: the quadrant has results of this wavefront's
  auto begin = [&]() {
    on = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int v = 0; v < 2; ++v)
        on |= (int)(128 * h + 32 * wm < cur.rows && 128 * v + 64 * wn < cur.cols) << (2 * h + v);
    on = __builtin_amdgcn_readfirstlane(on);
  };
  // A quadrant: 16 products, four at a time (two columns of a substep), if they are wanted; due(k)
  // goes before the four, so that reads and loads stand between the products. `on` is made
  // opaque: otherwise paths with and without products each get a copy of what stands between.
  auto quadrant = [&](int h, int v, const u32x4 (&p)[2][2], auto due) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      due(k);
      asm volatile("" : "+s"(on));
      if (on & (1 << (2 * h + v))) {
#pragma unroll
        for (int j = 2 * (k & 1); j < 2 * (k & 1) + 2; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) acc[h][v][i][j] = mfma<T>(q[k >> 1][j], p[k >> 1][i], acc[h][v][i][j]);
      }
    }
  };
  // Stores of row block i of a quadrant, which then starts over.
  constexpr int kStores = kQuadrantStores<OUT>;
  auto store = [&](int h, int v, int i) {
    store_block<T, OUT>(g.out, O, cur.row0 + 128 * h, cur.c0, cur.rows - 128 * h, 128 * v, cur.cols, wm, wn, i, acc[h][v][i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[h][v][i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  };
  auto read_q = [&](const uint8_t* L, int s, int k) {   // two blocks
#pragma unroll
    for (int j = 2 * k; j < 2 * k + 2; ++j) q[s][j] = fq.read(L, j, s);
  };
  auto read_p = [&](const uint8_t* L, int s, u32x4 (&d)[2][2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) d[s][i] = fp.read(L, i, s);
  };
  // One stage from the buffers of P and Q, the next one's first halves in N0 and M0. A, B: stores that
  // may be in flight behind the loads which the first and second barrier wait for. FIN: a tile's last
  // stage, which stores each quadrant during the products of the next.
  auto stage = [&](auto sa, auto sb, auto fin, uint8_t* P0, uint8_t* P1, uint8_t* Q0, uint8_t* Q1, const uint8_t* N0,
                   const uint8_t* M0) {
    constexpr int A = decltype(sa)::value, B = decltype(sb)::value;
    constexpr bool FIN = decltype(fin)::value && OUT != kAnyWidth;
    quadrant(0, 0, p0, [&](int k) {
      if (k < 2)
        read_q(Q0, 1, k);
      else
        read_p(P1, k - 2, p1);
    });
    step_barrier<8 + A>();   // Q0, P0 and P1 are read; Q1 has landed
    quadrant(1, 0, p1, [&](int k) {
      if (FIN && k < 2) store(0, 0, k);
      if (k >= 2) read_q(Q1, 0, k - 2);   // over what the first substep's products are done with
      if (k == 0 || k == 1) load_q(0, k, Q0);
      if (k == 3) load_p(0, 0, P0);
    });
    quadrant(0, 1, p0, [&](int k) {
      if (FIN && k == 0) {
        store(1, 0, 0);
        store(1, 0, 1);
      }
      if (k < 2) read_q(Q1, 1, k);
      if (k == 1) load_p(0, 1, P0);
      if (k >= 2) load_p(1, k - 2, P1);
    });
    step_barrier<8 + B>();   // Q1 is read; the next M0 and both halves of the next P have landed
    quadrant(1, 1, p1, [&](int k) {
      if (k < 2) {
        read_p(N0, k, p0);
      } else {
        if (FIN) store(0, 1, k - 2);
        read_q(M0, 0, k - 2);
      }
      if (k & 1) load_q(1, k >> 1, Q1);
    });
    if (FIN) {
      store(1, 1, 0);
      store(1, 1, 1);
    }
    advance();
  };
  // A tile's first stage stands behind the stores of the tile before (for the first tile: as many
  // that store nothing). Its place in the program is its own, so that on every way to a wait the
  // number of memory operations in flight is the same: the compiler, which checks each read of
  // LDS against the loads, then adds no wait. A tile's odd last stage has no products.
  constexpr std::integral_constant<int, 0> none{};
  constexpr std::integral_constant<int, 2 * kStores> half{};
  constexpr std::integral_constant<int, 4 * kStores> whole{};
  constexpr std::false_type more{};
  constexpr std::true_type last{};
#pragma unroll
  for (int i = 0; i < 4 * kStores; ++i)   // at places of their own, or the compiler keeps one of them
    __builtin_amdgcn_raw_buffer_store_b128(u32x4{0, 0, 0, 0}, window(g.out, 0), 16 * i, 0, 0);
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int v = 0; v < 2; ++v)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[h][v][i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (;;) {
    begin();
    int real = blocks_of(cur.n, TK);
    auto second = [&]() {   // the products of a pair's second stage
      real -= 2;
      on = __builtin_amdgcn_readfirstlane(real < 0 ? 0 : on);
    };
    stage(whole, half, more, pa0, pa1, qa0, qa1, pb0, qb0);
    second();
    for (int st = 2; st < cur.stages; st += 2) {
      stage(none, none, more, pb0, pb1, qb0, qb1, pa0, qa0);
      stage(none, none, more, pa0, pa1, qa0, qa1, pb0, qb0);
      second();
    }
    stage(none, half, last, pb0, pb1, qb0, qb1, pa0, qa0);
    if constexpr (OUT == kAnyWidth) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
          for (int i = 0; i < 2; ++i) store(h, v, i);
      __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
    }
    u += step;
    if (u >= end) break;
    cur = w.tile_of(u);
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0): no load into LDS outlives the workgroup
}

// ------------------------------------------------------------------ tiles of 128 x 128
// For few tiles, and few rows per expert (the rule and both sides' times: dense_small()). A stage is
// one quadrant of the above, in a ring of four sets of buffers, three under way while one is used;
// one barrier per stage. Alone on its CU it is bound by the loads' latency, 0.4 us per stage of 64
// (a stage of 256 x 256: 1.24), with many tiles by the weights: 128 experts of
// 1536 x 2048, one row each, 805 MB in 134 us, 6.0 TB/s.
// SPLIT: so few tiles that each tile's contraction is cut into g.split pieces for workgroups of their own; the
// fp32 sums go to the workspace, in the order that the lanes hold them, and a second launch adds the
// pieces in their order.
constexpr int64_t kPart = 128 * 128 * 4;   // bytes of a piece's sums
template <int D, int T, int OUT, bool SPLIT>
__global__ __launch_bounds__(TThreads, 1) void dense_small_kernel(DenseArgs g) {
  __shared__ int32_t p_off[kMaxExperts + 1];
  __shared__ int32_t p_u[kMaxExperts + 1];
  __shared__ __attribute__((aligned(128))) uint8_t qa[kHalf], qb[kHalf], qc[kHalf], qd[kHalf];
  __shared__ __attribute__((aligned(64))) uint8_t pa[kHalf], pb[kHalf], pc[kHalf], pd[kHalf];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  using W = Tiles<D, 128>;
  constexpr int TM = W::TM, TN = W::TN;
  const int64_t O = D == kDenseFwd ? g.N : g.K;
  const int blocks_n = (int)((g.N + TM - 1) / TM), blocks_k = (int)((g.K + TN - 1) / TN);
  const int c_tiles = (int)((O + TN - 1) / TN);
  int32_t total = build_plan(p_off, p_u, g.sizes, g.E, g.M, g.err,
                             [&](int32_t s) -> int32_t { return D == kDenseWgrad ? 0 : blocks_of(s, TM) * c_tiles; });
  total = D == kDenseWgrad ? g.E * blocks_n * blocks_k : __builtin_amdgcn_readfirstlane(total);
  if constexpr (D != kDenseWgrad) {
    if (g.zero_rest) zero_rows((uint16_t*)g.out, p_off[g.E], g.M, O);
  }
  if constexpr (SPLIT) total *= g.split;
  const W w{g, lane, wave, p_off, p_u, D == kDenseDgrad ? g.N : g.K, O, blocks_n, blocks_k};
  auto unit_of = [&](int32_t v) { return SPLIT ? w.piece_of(v, g.split) : w.tile_of(v); };
  const int G = gridDim.x;
  const int parts = G % 8 == 0 ? 8 : 1, step = G / parts, part = blockIdx.x % parts;
  const int32_t end = (int32_t)((int64_t)total * (part + 1) / parts);
  int32_t u = (int32_t)((int64_t)total * part / parts) + blockIdx.x / parts;
  if (u >= end) return;

  const Frag<W::kPAlong> fp(lane, 2 * wm);
  const Frag<W::kQAlong> fq(lane, 4 * wn);
  f32x4 acc[2][4];
  typename W::Tile cur = unit_of(u);     // of the products
  typename W::Cursor lc;                 // of the loads
  w.aim(lc, cur, true);
  int32_t lu = u;
  const int64_t pitch_p = W::kPAlong ? w.C : g.N;
  const uint32_t at_p = W::lane_at(W::kPAlong, lane, wave, pitch_p), at_q = W::lane_at(W::kQAlong, lane, wave, g.K);
  auto load = [&](uint8_t* P, uint8_t* Q) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w.template load<W::kQAlong>(lc.q, lc.left_q, lc.rest, at_q, g.K, 0, i, Q);
      w.template load<W::kPAlong>(lc.p, lc.left_p, lc.rest, at_p, pitch_p, 0, i, P);
    }
    w.next(lc);
    if (lc.st == lc.stages) {
      lu += step;
      const bool any = lu < end;
      w.aim(lc, any ? unit_of(lu) : cur, any);
    }
  };
  int on;   // the wavefront has results
  // One stage from P and Q; the one after the next two is asked for into NP and NQ, which the stage
  // before has used. S: stores of the tile before that may be in flight.
  auto stage = [&](auto behind, const uint8_t* P, const uint8_t* Q, uint8_t* NP, uint8_t* NQ) {
    constexpr int S = decltype(behind)::value;
    step_barrier<8 + S>();   // P and Q have landed; every wavefront has read the stage before
    u32x4 p[2][2], q[2][4];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int i = 0; i < 2; ++i) p[s][i] = fp.read(P, i, s);
#pragma unroll
      for (int j = 0; j < 4; ++j) q[s][j] = fq.read(Q, j, s);
    }
    load(NP, NQ);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      asm volatile("" : "+s"(on));
      if (on) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) acc[i][j] = mfma<T>(q[s][j], p[s][i], acc[i][j]);
      }
    }
  };
  constexpr int kStores = SPLIT ? 8 : kQuadrantStores<OUT>;
  constexpr std::integral_constant<int, 0> none{};
  constexpr std::integral_constant<int, kStores> some{};
  load(pa, qa);
  load(pb, qb);
  load(pc, qc);
#pragma unroll
  for (int i = 0; i < kStores; ++i)   // (see dense_tile_kernel)
    __builtin_amdgcn_raw_buffer_store_b128(u32x4{0, 0, 0, 0}, window(g.out, 0), 16 * i, 0, 0);
  for (;;) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int want = __builtin_amdgcn_readfirstlane((int)(32 * wm < cur.rows && 64 * wn < cur.cols));
    int real = blocks_of(cur.n, TK);   // stages with products
    auto due = [&]() {
      on = __builtin_amdgcn_readfirstlane(real > 0 ? want : 0);
      --real;
    };
    due();
    stage(some, pa, qa, pd, qd);
    due();
    stage(some, pb, qb, pa, qa);
    due();
    stage(some, pc, qc, pb, qb);
    due();
    stage(none, pd, qd, pc, qc);
    for (int st = 4; st < cur.stages; st += 4) {
      due();
      stage(none, pa, qa, pd, qd);
      due();
      stage(none, pb, qb, pa, qa);
      due();
      stage(none, pc, qc, pb, qb);
      due();
      stage(none, pd, qd, pc, qc);
    }
    if constexpr (SPLIT) {
      const __amdgpu_buffer_rsrc_t R = window(g.parts + (int64_t)u * kPart, kPart);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[i][j]), R,
                                                 (uint32_t)(((wave * 2 + i) * 4 + j) * 1024 + lane * 16), 0, 0);
    } else {
      store_quadrant<T, OUT>(g.out, O, cur.row0, cur.c0, cur.rows, 0, cur.cols, wm, wn, acc);
      if constexpr (OUT == kAnyWidth) __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
    }
    u += step;
    if (u >= end) break;
    cur = unit_of(u);
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0): no load into LDS outlives the workgroup
}

// The pieces of a tile added in their order, rounded and stored.
template <int D, int T, int OUT>
__global__ __launch_bounds__(TThreads) void dense_join_kernel(DenseArgs g) {
  __shared__ int32_t p_off[kMaxExperts + 1];
  __shared__ int32_t p_u[kMaxExperts + 1];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  using W = Tiles<D, 128>;
  constexpr int TM = W::TM, TN = W::TN;
  const int64_t O = D == kDenseFwd ? g.N : g.K;
  const int blocks_n = (int)((g.N + TM - 1) / TM), blocks_k = (int)((g.K + TN - 1) / TN);
  const int c_tiles = (int)((O + TN - 1) / TN);
  int32_t total = build_plan(p_off, p_u, g.sizes, g.E, g.M, g.err,
                             [&](int32_t s) -> int32_t { return D == kDenseWgrad ? 0 : blocks_of(s, TM) * c_tiles; });
  total = D == kDenseWgrad ? g.E * blocks_n * blocks_k : __builtin_amdgcn_readfirstlane(total);
  const W w{g, lane, wave, p_off, p_u, D == kDenseDgrad ? g.N : g.K, O, blocks_n, blocks_k};
  for (int32_t u = blockIdx.x; u < total; u += gridDim.x) {
    const typename W::Tile x = w.tile_of(u);
    f32x4 acc[2][4] = {};
    const uint8_t* from = g.parts + (int64_t)u * g.split * kPart + wave * 8192 + lane * 16;
#pragma unroll 4
    for (int p = 0; p < g.split; ++p, from += kPart)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += *reinterpret_cast<const f32x4*>(from + (i * 4 + j) * 1024);
    store_quadrant<T, OUT>(g.out, O, x.row0, x.c0, x.rows, 0, x.cols, wave >> 1, wave & 1, acc);
  }
}

// ------------------------------------------------------------------ forward, few rows
// A unit is 16 output columns of one expert and up to 16 of its rows over the whole contraction;
// the wavefront streams the 16 weight rows from memory into registers, PD steps of 32 k ahead, and
// reads the activations beside them (rows past the expert's cost nothing). Bound by the weights: 8
// experts of 8192 x 4096, one row each, 537 MB in 102 us, 5.3 TB/s. (Units of 32 rows, 4 steps
// ahead: 110 there and behind at every size where the tiles are not ahead of both.)
constexpr int NThreads = 256, NWaves = NThreads / 64, PD = 8;

template <int T>
__global__ __launch_bounds__(NThreads) void dense_narrow_kernel(DenseArgs g) {
  __shared__ int32_t p_off[kMaxExperts + 1];
  __shared__ int32_t p_u[kMaxExperts + 1];
  const int64_t K = g.K, N = g.N;
  const int nblk = (int)((N + 15) / 16);
  const int32_t total = __builtin_amdgcn_readfirstlane(build_plan(
      p_off, p_u, g.sizes, g.E, g.M, g.err, [&](int32_t s) -> int32_t { return blocks_of(s, 16) * nblk; }));
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
    x.row0 = o0 + (int64_t)chunk * 16;
    x.rows = (int)min<int64_t>(16, o1 - x.row0);
    x.W = window(g.q + ((int64_t)e * N + x.n0) * K, any ? min<int64_t>(16, N - x.n0) * K * 2 : 0);
    x.A = window(g.p + x.row0 * K, any ? x.rows * K * 2 : 0);
    return x;
  };
  u32x4 wf[PD], af[PD];
  const uint32_t at = (uint32_t)(r16 * K * 2 + 16 * grp);
  auto load = [&](int i, const Unit& x, int s) {
    const uint32_t off = oob_unless(32 * (int64_t)s + 8 * grp < K, at + 64 * (uint32_t)s);
    wf[i] = __builtin_amdgcn_raw_buffer_load_b128(x.W, off, 0, 0);
    af[i] = __builtin_amdgcn_raw_buffer_load_b128(x.A, off, 0, 0);
  };
  int u = blockIdx.x * NWaves + wave;
  if (u >= total) return;
  Unit cur = unit_of(u, true);
#pragma unroll
  for (int i = 0; i < PD; ++i) load(i, cur, i);
  for (; u < total; u += stride) {
    const Unit nxt = unit_of(u + stride, u + stride < total);
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int c = 0; c < batches; ++c) {
      const bool last = c + 1 == batches;
      const Unit from = last ? nxt : cur;
      const int s0 = last ? 0 : (c + 1) * PD;
#pragma unroll
      for (int i = 0; i < PD; ++i) {
        acc = mfma<T>(wf[i], af[i], acc);
        load(i, from, s0 + i);
      }
    }
    const int64_t n = cur.n0 + 4 * grp;
    if (r16 < cur.rows) {
      uint16_t* dst = reinterpret_cast<uint16_t*>(g.out) + (cur.row0 + r16) * N + n;
      const u32x2 v = u32x2{pack2<T>(acc[0], acc[1]), pack2<T>(acc[2], acc[3])};
      if ((N & 3) == 0) {
        if (n < N) *reinterpret_cast<u32x2*>(dst) = v;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < N) dst[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
      }
    }
    cur = nxt;
  }
}

template <int T>
hipError_t narrow_one(const DenseArgs& g, int cus, hipStream_t s) {
  const int64_t units = ((g.M + 15) / 16 + std::min<int64_t>(g.E, g.M)) * ((g.N + 15) / 16);
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>((units + NWaves - 1) / NWaves, (int64_t)cus * 4));
  hipLaunchKernelGGL((dense_narrow_kernel<T>), dim3((unsigned)grid), dim3(NThreads), 0, s, g);
  return hipGetLastError();
}

template <int D, int T, int OUT>
hipError_t tile_one(const DenseArgs& g, bool small, int cus, hipStream_t s) {
  const int64_t tiles = std::max<int64_t>(1, dense_tiles(D, g.M, g.N, g.K, g.E, small ? 128 : 256));
  const dim3 grid((unsigned)std::min<int64_t>(tiles * (small ? g.split : 1), cus));
  if (!small) {
    hipLaunchKernelGGL((dense_tile_kernel<D, T, OUT>), grid, dim3(TThreads), 0, s, g);
  } else if (g.split == 1) {
    hipLaunchKernelGGL((dense_small_kernel<D, T, OUT, false>), grid, dim3(TThreads), 0, s, g);
  } else {
    hipLaunchKernelGGL((dense_small_kernel<D, T, kWide, true>), grid, dim3(TThreads), 0, s, g);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((dense_join_kernel<D, T, OUT>), dim3((unsigned)std::min<int64_t>(tiles, cus)), dim3(TThreads), 0, s, g);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dense_tile(int dir, int dtype, bool f32_out, bool small, const DenseArgs& g, int cus, hipStream_t s) {
  auto run = [&](auto t) {
    constexpr int T = decltype(t)::value;
    if (dir == kDenseDgrad) return tile_one<kDenseDgrad, T, kWide>(g, small, cus, s);
    if (dir == kDenseWgrad)
      return f32_out ? tile_one<kDenseWgrad, T, kF32Out>(g, small, cus, s) : tile_one<kDenseWgrad, T, kWide>(g, small, cus, s);
    return g.N % 8 ? tile_one<kDenseFwd, T, kAnyWidth>(g, small, cus, s) : tile_one<kDenseFwd, T, kWide>(g, small, cus, s);
  };
  return dtype == kBF16 ? run(std::integral_constant<int, kBF16>{}) : run(std::integral_constant<int, kF16>{});
}

hipError_t launch_dense_narrow(int dtype, const DenseArgs& g, int cus, hipStream_t s) {
  return dtype == kBF16 ? narrow_one<kBF16>(g, cus, s) : narrow_one<kF16>(g, cus, s);
}

}  // namespace geg
