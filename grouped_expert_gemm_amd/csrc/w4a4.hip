// Grouped expert GEMM with both operands in MXFP4 (e2m1 codes, one e8m0 scale per 32 k):
//     out_e = bf16( Q(a_e) . W_e^T ),  Q the MXFP4 conversion of mxfp4.hpp,
// on gfx950's block-scaled matrix instruction with two 4-bit operands
// (v_mfma_scale_f32_16x16x128_f8f6f4, twice the rate of the 8-bit forms), fp32
// accumulation. The released weight bytes and scales feed it as they are.
//
// Operand layout (both operands alike): lane l holds row l % 16, the 16 consecutive
// bytes of k = 32 (l / 16) .. +31 of the 128-wide step, and in a byte of its scale
// register the e8m0 byte of that row and 32-block. The weights are the first operand,
// so a lane's four results are four adjacent output columns (4 (l / 16) .. +3 of the 16)
// of one activation row (l % 16).
//
// Two kernels. With at most kW4A4NarrowAvg rows per expert on average the narrow one
// streams the weights straight into registers, larger batches run 256 x 256 tiles through
// LDS. A launch of its own quantises the activations, except for the smallest batches,
// where the narrow kernel does.
#include <algorithm>

#include "geg_device.hpp"
#include "geg_launch.hpp"
#include "mxfp4.hpp"

namespace geg {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int BK = 128;   // k per step

__device__ __forceinline__ uint32_t oob_unless(bool ok, uint32_t off) { return off | ((uint32_t)!ok << 31); }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t wrsrc(const void* base, int64_t bytes) {
  const int32_t n = bytes <= 0 ? 0 : (bytes > 0x7FFFFFF0 ? 0x7FFFFFF0 : (int32_t)bytes);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, n, 0x00020000);
}

__device__ __forceinline__ v8i fp4_operand(const u32x4& v) {
  return v8i{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}

// acc += weights (first operand) . activations, scale bytes S of the two registers.
template <int S>
__device__ __forceinline__ f32x4 mfma_fp4(const u32x4& w, const u32x4& a, const f32x4& acc, uint32_t sw, uint32_t sa) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(w), fp4_operand(a), acc, 4, 4, S, (int)sw, S,
                                                          (int)sa);
}

// ------------------------------------------------------------------ activations for the tiles
// bf16 [M, K] -> codes and scales. For the narrow kernel codes [M, K/2] and scales
// [M, K/32]; for the tiles codes [K/128 rounded up][M][64] (what lies past K is not written:
// the weights read as zeros there) and scales [K/512 rounded up][M][16]: byte 4 b + s of a row's 16 is the scale of 32-block 4 s + b of
// the 512-wide piece, so a lane of group b reads the bytes of its four steps s as one
// dword; blocks past K get 0. One thread per 8 values, four lanes to a block. Rows that
// belong to no expert are converted like the others (what they hold is never read), but not
// flagged: a thread that meets a block with an inf or NaN sums the sizes, once. 8192 x 2880:
// 14 us for 60 MB.
template <bool TILES>
__global__ __launch_bounds__(kThreads) void w4a4_quantize_kernel(const uint16_t* __restrict__ a, int64_t M, int64_t KS,
                                                                 const int32_t* __restrict__ sizes, int32_t E,
                                                                 uint32_t* __restrict__ codes,
                                                                 uint8_t* __restrict__ scales, uint32_t* err) {
  const int64_t pieces = M * KS * 4;
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  int64_t owned = -1;   // the experts' rows, once they are needed
  for (int64_t p = (int64_t)blockIdx.x * kThreads + threadIdx.x; p < pieces; p += stride) {
    float f[8], q[8];
    unpack16<kBF16>(reinterpret_cast<const u32x4*>(a)[p], f);
    uint32_t word;
    const int byte = mxfp4_block_piece<8, false>(f, word, q);
    const int64_t b = p >> 2;
    if ((p & 3) == 0 && byte == 255) {
      if (owned < 0) {
        owned = 0;
        for (int e = 0; e < E; ++e) owned += max(sizes[e], 0);
      }
      if (b < owned * KS) atomicOr(err, kErrNonFinite);
    }
    if constexpr (TILES) {
      const int64_t m = b / KS, kb = b - m * KS;
      codes[((kb >> 2) * M + m) * 16 + 4 * (kb & 3) + (p & 3)] = word;
      if ((p & 3) == 0) scales[((kb >> 4) * M + m) * 16 + 4 * (kb & 3) + ((kb >> 2) & 3)] = (uint8_t)byte;
    } else {
      codes[p] = word;
      if ((p & 3) == 0) scales[b] = (uint8_t)byte;
    }
  }
  if constexpr (!TILES) return;
  const int64_t pad = ((KS + 15) & ~(int64_t)15) - KS;   // blocks past K of the last piece
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < M * pad; i += stride) {
    const int64_t m = i / pad, kb = KS + i - m * pad;
    scales[((kb >> 4) * M + m) * 16 + 4 * (kb & 3) + ((kb >> 2) & 3)] = 0;
  }
}

// ------------------------------------------------------------------ tiles
constexpr int TM = 256, TN = 256;          // rows, columns per tile
constexpr int TThreads = 512;              // 8 wavefronts: 2 (rows of 128) x 4 (columns of 64)
constexpr int kRowStage = TM * (BK / 2);   // bytes of the activations per step
constexpr int kColStage = TN * BK;         // bytes of the weights per two steps

// A row of the staged activations holds 4 chunks of 16 bytes, chunk c of row r at
// c ^ (2 ((r / 4) % 2)); a row of the staged weights 8, at c ^ (r % 8). A fragment read
// (16 rows, chunk g for lane group g) then meets no bank conflict (with the activations'
// chunks at c ^ ((r / 4) % 4) every read took twice its time).
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return (uint32_t)(r * (BK / 2) + ((c ^ ((r >> 1) & 2)) << 4));
}

// This wavefront's LDS accesses are done and at most N of its loads in flight, then the
// workgroup meets (__syncthreads would wait for every load).
template <int N>
__device__ __forceinline__ void step_barrier() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | 0x0070);
  asm volatile("s_barrier" ::: "memory");
}

// One workgroup per CU, persistent over tiles (expert, column block, row block; row
// blocks fastest, so that the tiles that share weights run together on one XCD). Loads
// write LDS directly (16 bytes per lane, 1 KB per instruction): the activations a step at
// a time into four buffers, the weights two steps at a time into two, all distinct LDS
// objects named at compile time: the compiler then adds no wait for loads that fill the
// others. What a load instruction covers decides its speed: rows of 64 bytes came at 37
// GB/s per CU, 128 at 50 and whole runs at 65 (1440-byte rows from L2). So the
// activations are quantised into step order, where a step's rows are one run, and a
// weight row is read 128 bytes at a time.
//
// A wavefront computes 128 x 64, 8 + 4 fragments for the 32 instructions of a step, in
// two halves:
//   half 1: the second half's row fragments are read and the activations three steps
//           ahead start into the previous step's buffer while the first half's multiply;
//   barrier: every read of this step's buffers is done, the next step's have landed;
//   half 2: the next step's first fragments are read and, every other step, the weights
//           of the pair after the next start while the second half's rows multiply.
// So the matrix pipes work while LDS is read. The steps run on across tiles: the last
// ones of a tile start the next tile's first (a tile's steps are padded to whole pieces
// of four). Scales go by pieces of four steps through registers into LDS in lane order
// (byte 4 b + s of a row's 16: block b of step s): one dword per lane serves four steps,
// the instruction picking the byte.
//
// 2048 tokens x 4 of 32 experts, K 2880, N 5760: 151-157 us, 1219 tiles in five rounds of
// the 256 CUs. Before its last step (161 us) it took 111 us without its loads, 124 without
// its multiplications and 135 without its stores: no one of the three bounds it alone. Not kept: stores that the
// next tile's first waits leave in flight (nothing gained), stores past the caches
// (3% slower).
template <bool SHORT>
__device__ __forceinline__ void w4a4_tiles(const W4A4Args& g) {
  __shared__ int32_t p_off[kMaxExperts + 1];
  __shared__ int32_t p_u[kMaxExperts + 1];
  __shared__ __attribute__((aligned(16))) uint8_t a0[kRowStage];
  __shared__ __attribute__((aligned(16))) uint8_t a1[kRowStage];
  __shared__ __attribute__((aligned(16))) uint8_t a2[kRowStage];
  __shared__ __attribute__((aligned(16))) uint8_t a3[kRowStage];
  __shared__ __attribute__((aligned(16))) uint8_t w0[kColStage];
  __shared__ __attribute__((aligned(16))) uint8_t w1[kColStage];
  __shared__ __attribute__((aligned(16))) uint8_t sc[2][(TM + TN) * 16];
  const int64_t K = g.K, N = g.N, M = g.M;
  const int KS = (int)(K >> 5), KB = (int)(K >> 1);
  const int n_tiles = (int)((N + TN - 1) / TN);
  const int32_t total = build_plan(p_off, p_u, g.sizes, g.E, M, g.err,
                                   [&](int32_t s) -> int32_t { return (s + TM - 1) / TM * n_tiles; });
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int r16 = lane & 15, grp = lane >> 4;
  const int nss = (KS + 15) / 16;   // pieces of four steps
  const int G = gridDim.x;
  const int P = G % 8 == 0 ? 8 : 1, step = G / P, part = blockIdx.x % P;
  const int32_t end = (int32_t)((int64_t)total * (part + 1) / P);
  int32_t u = (int32_t)((int64_t)total * part / P) + blockIdx.x / P;
  if (u >= end) return;

  struct Tile {
    int64_t row0, n0, w0;   // first row, first column, first weight row in [E N]
    int rows, ncols;
  };
  auto tile_of = [&](int32_t u) {
    Tile x;
    const int e = __builtin_amdgcn_readfirstlane(find_expert(p_u, g.E, u));
    const int32_t lu = u - __builtin_amdgcn_readfirstlane(p_u[e]);
    const int32_t o0 = __builtin_amdgcn_readfirstlane(p_off[e]), o1 = __builtin_amdgcn_readfirstlane(p_off[e + 1]);
    const int rblocks = (o1 - o0 + TM - 1) / TM;
    const int nt = lu / rblocks, mt = lu - nt * rblocks;
    x.row0 = o0 + (int64_t)mt * TM;
    x.rows = (int)min<int64_t>(TM, o1 - x.row0);
    x.n0 = (int64_t)nt * TN;
    x.ncols = (int)min<int64_t>(TN, N - x.n0);
    x.w0 = (int64_t)e * N + x.n0;
    return x;
  };

  // Staging: of the activations a wavefront fills rows 16 wave + 128 i .. +15 (i = 0, 1), 4
  // lanes to a row, of the weights rows 8 wave + 64 i .. +7 (i = 0 .. 3), 8 lanes to a row;
  // lane l lands in slot l % 4 (l % 8) of its row and fetches the chunk that belongs there.
  // Rows past the expert's and columns past N (any = false: all) read as zeros, and so do
  // the weights' chunks past K.
  const int cp_r = 16 * wave + (lane >> 2), cp_c = (lane & 3) ^ ((cp_r >> 1) & 2);
  const uint32_t cp_a = (uint32_t)(cp_r * 64 + 16 * cp_c);
  const int cp_k = (lane & 7) ^ (lane >> 3);
  const uint32_t cp_w = (uint32_t)((8 * wave + (lane >> 3)) * KB + 16 * cp_k), cp_next = (uint32_t)(64 * KB);
  const int nst = (KS + 3) / 4;
  auto stage_a = [&](const Tile& x, bool any, int st, uint8_t* L) {
    const __amdgpu_buffer_rsrc_t R = wrsrc(g.aq + (st * M + x.row0) * 64, any && st < nst ? x.rows * 64 : 0);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(R, (lds_ptr_t)(L + (16 * wave + 128 * i) * 64), 16, cp_a + i * 8192, 0, 0,
                                               0);
  };
  auto stage_w = [&](const Tile& x, bool any, int pr, uint8_t* L) {
    const __amdgpu_buffer_rsrc_t R = wrsrc(g.wq + x.w0 * KB, any ? (int64_t)x.ncols * KB : 0);
    const uint32_t off = oob_unless(8 * pr + cp_k < KS, cp_w + 128 * pr);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(R, (lds_ptr_t)(L + (8 * wave + 64 * i) * 128), 16, off + i * cp_next, 0, 0,
                                               0);
  };
  // Scales of a piece: thread t has bytes 8 (t % 2) .. +7 of row (column) t / 2's 16. The
  // activations' are in lane order already; the weights' rows hold K / 32 bytes at any
  // alignment: 8 bytes that end with the row at the latest, shifted, so that blocks past K
  // get 0 (SHORT: rows of fewer than 8 bytes, byte by byte).
  const int s_row = t >> 1, s_half = t & 1;
  u32x2 s_a, s_w;
  auto load_scales = [&](const Tile& x, bool any, int ss) {
    const __amdgpu_buffer_rsrc_t RS = wrsrc(g.as + ((int64_t)ss * M + x.row0) * 16, any ? (M - x.row0) * 16 : 0);
    s_a = __builtin_amdgcn_raw_buffer_load_b64(RS, (uint32_t)(16 * s_row + 8 * s_half), 0, 0);
    const uint8_t* row = g.ws + (x.w0 + min(s_row, x.ncols - 1)) * KS;
    const int o = 16 * ss + 8 * s_half;
    if constexpr (!SHORT) {
      __builtin_memcpy(&s_w, row + min(o, KS - 8), 8);
    } else {
      s_w = u32x2{0, 0};
#pragma unroll
      for (int b = 0; b < 8; ++b)
        if (o + b < KS) s_w[b >> 2] |= (uint32_t)row[o + b] << (8 * (b & 3));
    }
  };
  auto put_scales = [&](int ss, uint8_t* to) {
    *reinterpret_cast<u32x2*>(to + 16 * s_row + 8 * s_half) = s_a;
    const int o = 16 * ss + 8 * s_half, over = SHORT ? 0 : o - min(o, KS - 8);   // bytes loaded too early
    uint64_t v = __builtin_bit_cast(uint64_t, s_w);
    v = over >= 8 ? 0 : v >> (8 * over);
    // (block pairs of this half's two steps; the other thread of the row has the other two)
    const uint32_t d0 = (uint32_t)v, d1 = (uint32_t)(v >> 32);
    const uint32_t b01 = perm(d1, d0, 0x05010400u), b23 = perm(d1, d0, 0x07030602u);
    const uint32_t mine = s_half ? b23 : b01;
    const uint32_t other = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(s_half ? b01 : b23), 0xB1, 0xF, 0xF, true);
    const uint32_t lo = s_half ? other : mine, hi = s_half ? mine : other;
    *reinterpret_cast<u32x2*>(to + (TM + s_row) * 16 + 8 * s_half) =
        u32x2{perm(hi, lo, 0x05040100u), perm(hi, lo, 0x07060302u)};
  };

  const uint32_t rd_a = chunk_at(128 * wm + r16, grp);               // row fragment i: + 1024 i
  // column fragment j: + 2048 j; second step of the two: ^ 64
  const uint32_t rd_w = (uint32_t)((64 * wn + r16) * 128 + ((grp ^ (r16 & 7)) << 4));
  const uint32_t rd_sa = (uint32_t)((128 * wm + r16) * 16 + 4 * grp);       // + 256 i
  const uint32_t rd_sw = (uint32_t)((TM + 64 * wn + r16) * 16 + 4 * grp);   // + 256 j
  u32x4 w[2][4], alo[4], ahi[4];
  uint32_t sw[2][4], slo[4], shi[4];
  f32x4 acc[8][4];
  auto read_w = [&](const uint8_t* L, int odd, u32x4* d) {
#pragma unroll
    for (int j = 0; j < 4; ++j) d[j] = *reinterpret_cast<const u32x4*>(L + (rd_w ^ (64 * odd)) + 2048 * j);
  };
  auto read_a = [&](const uint8_t* L, int i0, u32x4* d) {
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = *reinterpret_cast<const u32x4*>(L + rd_a + 1024 * (i0 + i));
  };
  auto read_s = [&](const uint8_t* from, uint32_t at, uint32_t* d) {
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = *reinterpret_cast<const uint32_t*>(from + at + 256 * i);
  };

  Tile cur = tile_of(u);
  bool live = 128 * wm < cur.rows;
  int par = 0;   // scale buffer of the piece at hand
  load_scales(cur, true, 0);
  stage_w(cur, true, 0, w0);
  stage_a(cur, true, 0, a0);
  stage_a(cur, true, 1, a1);
  stage_a(cur, true, 2, a2);
  stage_w(cur, true, 1, w1);
  put_scales(0, sc[0]);
  step_barrier<8>();
  read_w(w0, 0, w[0]);
  read_a(a0, 0, alo);
  read_s(sc[0], rd_sw, sw[0]);
  read_s(sc[0], rd_sa, slo);

  for (;;) {
    const bool more = u + step < end;
    const Tile nxt = more ? tile_of(u + step) : cur;
    const bool nlive = more && 128 * wm < nxt.rows;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int ss = 0; ss < nss; ++ss) {
      const bool last = ss + 1 == nss;
      // Step S of the piece in buffer `L`, the next one in `L1`. A piece's scales stay in
      // registers; sw alternates between two sets, as the weights' fragments do.
      auto one_step = [&](auto Sc, const uint8_t* L, const uint8_t* L1, uint8_t* L3, const uint8_t* W1, uint8_t* W2) {
        constexpr int S = decltype(Sc)::value;
        constexpr int c = S & 1, n = c ^ 1;
        if constexpr (S == 0) load_scales(last ? nxt : cur, !last || more, last ? 0 : ss + 1);
        if (live) {
          read_a(L, 4, ahi);
          if constexpr (S == 0) read_s(sc[par], rd_sa + 1024, shi);
        }
        // the stage three ahead: of this tile, or of the next one (its first three)
        if constexpr (S == 0)
          stage_a(cur, true, 4 * ss + 3, L3);
        else
          stage_a(last ? nxt : cur, !last || more, last ? S - 1 : 4 * ss + S + 3, L3);
        if (live) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = mfma_fp4<S>(w[c][j], alo[i], acc[i][j], sw[0][j], slo[i]);
        }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (S == 3) put_scales(last ? 0 : ss + 1, sc[par ^ 1]);
        // what may stay in flight: the loads begun after those the next step reads. Per
        // step: 0 the scales' two, a3; 1 a4, w of 4 and 5; 2 a5; 3 a6, w of 6 and 7.
        constexpr int scale_loads = SHORT ? 0 : 2;
        step_barrier<S == 0 ? 8 + scale_loads : S == 1 ? 4 + scale_loads : S == 2 ? 8 : 4>();
        if (S == 3 && last ? nlive : live) {
          read_w(W1, n, w[n]);
          read_a(L1, 0, alo);
          if constexpr (S == 3) {
            read_s(sc[par ^ 1], rd_sw, sw[1]);
            read_s(sc[par ^ 1], rd_sa, slo);
          }
        }
        if constexpr (S == 1) stage_w(last ? nxt : cur, !last || more, last ? 0 : 2 * ss + 2, W2);
        if constexpr (S == 3) stage_w(last ? nxt : cur, !last || more, last ? 1 : 2 * ss + 3, W2);
        if (live) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[4 + i][j] = mfma_fp4<S>(w[c][j], ahi[i], acc[4 + i][j], sw[0][j], shi[i]);
        }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (S == 3) {
#pragma unroll
          for (int j = 0; j < 4; ++j) sw[0][j] = sw[1][j];
        }
      };
      one_step(std::integral_constant<int, 0>{}, a0, a1, a3, w0, w0);
      one_step(std::integral_constant<int, 1>{}, a1, a2, a0, w1, w0);
      one_step(std::integral_constant<int, 2>{}, a2, a3, a1, w1, w1);
      one_step(std::integral_constant<int, 3>{}, a3, a0, a2, w0, w1);
      par ^= 1;
    }

    // Results. Lane (r16, grp) has columns 16 j + 4 grp .. +3 of row 16 i + r16; trading
    // rows of 16 lanes between two neighbouring j gives every lane 8 adjacent columns, 64
    // consecutive bytes of each of 16 rows per store.
    if (live) {
      const bool wide = (N & 7) == 0 && (reinterpret_cast<uintptr_t>(g.out) & 15) == 0;
      // lane groups 0, 2: columns 0-7, 8-15 of block j; 1, 3: of block j + 1
      const int col = 16 * (grp & 1) + 8 * (grp >> 1);
      uint16_t* dst = g.out + (cur.row0 + 128 * wm + r16) * N + cur.n0 + 64 * wn + col;
      const int left = (int)(min<int64_t>(N - cur.n0, TN)) - 64 * wn - col;   // columns from this lane's first on
      const int rows = cur.rows - 128 * wm - r16;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          u32x4 v;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t p = pack_bf16x2(acc[i][j][2 * h], acc[i][j][2 * h + 1]);
            const uint32_t q = pack_bf16x2(acc[i][j + 1][2 * h], acc[i][j + 1][2 * h + 1]);
            const auto r = __builtin_amdgcn_permlane16_swap(p, q, false, false);
            v[h] = r[0];
            v[2 + h] = r[1];
          }
          if (16 * i < rows && 16 * j < left) {
            uint16_t* d = dst + (int64_t)(16 * i) * N + 16 * j;
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
    if (!more) break;
    u += step;
    cur = nxt;
    live = nlive;
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0): no load into LDS outlives the workgroup
}

__global__ __launch_bounds__(TThreads, 1) void w4a4_tile_kernel(W4A4Args g) { w4a4_tiles<false>(g); }
__global__ __launch_bounds__(TThreads, 1) void w4a4_tile_short_kernel(W4A4Args g) { w4a4_tiles<true>(g); }

// ------------------------------------------------------------------ narrow
// Wavefront units: 16 output columns of one expert and up to 16 RB of its rows (a group),
// over the whole contraction. A workgroup takes a contiguous run of units, group by
// group: it quantises a group's rows into LDS once, then its wavefronts stream the weight
// rows of their units straight into registers (64 consecutive bytes of each of 16 rows per
// instruction and pair), PD pairs of steps ahead at all times, across units and groups: no
// barrier and no cross-wavefront sum between them. Bound by the weights' bytes: 64 tokens
// x 4 of 32 experts, 2880 x 2880: 32.7 us for 143 MB (4.4 TB/s) after 5 us of
// quantisation; one token x 4, 2880 x 5760: 9.6 us for 35 MB (3.7 TB/s, the ramp included).
constexpr int NThreads = 512, NWaves = NThreads / 64;
constexpr int PD = 4;   // pairs of steps in flight per wavefront; a unit's pairs are padded to whole PDs

// Steps go in pairs of 256 k whose eight 32-blocks are dealt so that lane group g takes
// blocks 2 g and 2 g + 1, one per step (both operands alike, so the sums are the same): a
// lane's scale bytes of a pair are then adjacent: one 2-byte load instead of two of a byte
// (EVEN: rows of an even number of scales at an even address; otherwise two all the same).

template <int RB, bool PRE, bool EVEN>
__global__ __launch_bounds__(NThreads, 4) void w4a4_narrow_kernel(W4A4Args g) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int64_t K = g.K, N = g.N, KS = K >> 5;
  const int np = (int)((K + 2 * BK - 1) / (2 * BK)), nch = (np + PD - 1) / PD;   // pairs; PDs of them
  const int ld = np * 128 + 16;   // bytes of a quantised row (an odd number of 16-byte units)
  const int sld = np * 8;         // bytes of a row's scales
  uint8_t* codes = lds;                     // [16 RB][ld]
  uint8_t* ascale = codes + 16 * RB * ld;   // [16 RB][sld]
  int32_t* p_off = reinterpret_cast<int32_t*>(ascale + 16 * RB * sld);
  int32_t* p_u = p_off + g.E + 1;
  const int nblk = (int)((N + 15) / 16);
  const int32_t total = build_plan(p_off, p_u, g.sizes, g.E, g.M, g.err, [&](int32_t s) -> int32_t {
    return (s + 16 * RB - 1) / (16 * RB) * nblk;
  });
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int r16 = lane & 15, grp = lane >> 4;
  const int lo = (int)((int64_t)total * blockIdx.x / gridDim.x);
  const int hi = (int)((int64_t)total * (blockIdx.x + 1) / gridDim.x);

  // The group of unit u: its expert, its chunk of rows, its first unit.
  struct Group {
    int e, chunk, u0;
  };
  auto group_of = [&](int u) {
    Group w;
    w.e = __builtin_amdgcn_readfirstlane(find_expert(p_u, g.E, u));
    const int base = __builtin_amdgcn_readfirstlane(p_u[w.e]);
    w.chunk = (u - base) / nblk;
    w.u0 = base + w.chunk * nblk;
    return w;
  };
  u32x4 code[PD][2];
  uint32_t scale[PD], scale1[EVEN ? 1 : PD];
  // Pairs ch PD .. +PD-1 of the unit at columns 16 nb of expert e into the PD slots (none:
  // zeros, without a memory access). Rows past N lie past the buffers and read zeros. What
  // a lane reads past its row's end (the last pair's blocks past K, padding pairs) meets
  // zero activations or is skipped; only scales there are masked (0xFF would be a NaN).
  struct Next {
    __amdgpu_buffer_rsrc_t W, S;
    uint32_t wo, so;
  };
  auto aim = [&](bool any, int e, int nb, int ch) {
    Next x;
    x.W = wrsrc(g.wq + (int64_t)e * N * (K >> 1), any ? N * (K >> 1) : 0);
    x.S = wrsrc(g.ws + (int64_t)e * N * KS, any ? N * KS : 0);
    const int64_t n = 16 * (int64_t)nb + r16;
    x.wo = (uint32_t)(n * (K >> 1) + 128 * PD * (int64_t)ch + 32 * grp);
    x.so = (uint32_t)(n * KS + 8 * PD * (int64_t)ch + 2 * grp);
    return x;
  };
  auto load = [&](int i, const Next& x) {
    code[i][0] = __builtin_amdgcn_raw_buffer_load_b128(x.W, x.wo + 128 * i, 0, 0);
    code[i][1] = __builtin_amdgcn_raw_buffer_load_b128(x.W, x.wo + 128 * i + 16, 0, 0);
    if constexpr (EVEN) {
      scale[i] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(x.S, x.so + 8 * i, 0, 0);
    } else {
      scale[i] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(x.S, x.so + 8 * i, 0, 0);
      scale1[i] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(x.S, x.so + 8 * i + 1, 0, 0);
    }
  };

  bool have = false;   // this wavefront's next unit has its first PD steps in flight
  Group cur = lo < hi ? group_of(lo) : Group{0, 0, 0};
  for (int s0 = lo; s0 < hi;) {
    const int s1 = min(hi, cur.u0 + nblk);   // this group's units in the run: [s0, s1)
    const Group nxt = s1 < hi ? group_of(s1) : cur;
    const int s2 = s1 < hi ? min(hi, nxt.u0 + nblk) : s1;
    int u = s0 + wave;
    if (!have && u < s1) {
      const Next x = aim(true, cur.e, u - cur.u0, 0);
#pragma unroll
      for (int i = 0; i < PD; ++i) load(i, x);
    }
    const int64_t row0 = p_off[cur.e] + (int64_t)cur.chunk * 16 * RB;
    const int rows = (int)min<int64_t>(16 * RB, p_off[cur.e + 1] - row0);
    lds_barrier();   // the rows before are no longer read
    if constexpr (PRE) {
      // 16 bytes of codes or 4 of scales at a time; what lies past K is zero
      const int cpr = np * 8, words = np * 2;
      for (int p0 = t; p0 < rows * cpr; p0 += 4 * NThreads) {
        u32x4 v[4];
        int at[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int p = p0 + i * NThreads, r = p / cpr, c = p - r * cpr;
          at[i] = p < rows * cpr ? r * ld + 16 * c : -1;
          v[i] = u32x4{0, 0, 0, 0};
          if (at[i] >= 0 && c < KS) v[i] = reinterpret_cast<const u32x4*>(g.aq + (row0 + r) * (K >> 1))[c];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (at[i] >= 0) *reinterpret_cast<u32x4*>(codes + at[i]) = v[i];
      }
      for (int p = t; p < rows * words; p += NThreads) {
        const int r = p / words, w = p - r * words;
        const uint8_t* src = g.as + (row0 + r) * KS + 4 * w;
        uint32_t v = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (4 * w + b < KS) v |= (uint32_t)src[b] << (8 * b);
        *reinterpret_cast<uint32_t*>(ascale + r * sld + 4 * w) = v;
      }
    } else {
      const int ppr = np * 32, pieces = rows * ppr;   // 8-value pieces per padded row
      for (int p0 = t; p0 < pieces; p0 += 4 * NThreads) {
        u32x4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int p = p0 + i * NThreads, r = p / ppr, c = p % ppr;
          v[i] = u32x4{0, 0, 0, 0};
          if (p < pieces && 8 * (int64_t)c < K) v[i] = reinterpret_cast<const u32x4*>(g.a + (row0 + r) * K)[c];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int p = p0 + i * NThreads, r = p / ppr, c = p % ppr;
          if (p < pieces) {   // whole blocks: the four lanes of one pass together
            float f[8], q[8];
            unpack16<kBF16>(v[i], f);
            uint32_t word;
            const int byte = mxfp4_block_piece<8, false>(f, word, q);
            *reinterpret_cast<uint32_t*>(codes + r * ld + 4 * c) = word;
            if ((c & 3) == 0) {
              ascale[r * sld + (c >> 2)] = (uint8_t)(8 * (int64_t)c < K ? byte : 0);
              if (byte == 255) atomicOr(g.err, kErrNonFinite);
            }
          }
        }
      }
    }
    lds_barrier();
    const bool some = u < s1;
    for (; u < s1; u += NWaves) {
      // where this wavefront goes next: its next unit here, or its first of the next group
      const bool here = u + NWaves < s1;
      const int u2 = here ? u + NWaves : s1 + wave;
      have = here || u2 < s2;
      const int e2 = here ? cur.e : nxt.e, nb2 = u2 - (here ? cur.u0 : nxt.u0);
      f32x4 acc[RB];
#pragma unroll
      for (int b = 0; b < RB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int ch = 0; ch < nch; ++ch) {
        const bool more = ch + 1 < nch;
        const Next x = aim(more || have, more ? cur.e : e2, more ? u - cur.u0 : nb2, more ? ch + 1 : 0);
#pragma unroll
        for (int i = 0; i < PD; ++i) {
          const int p = ch * PD + i;
          if (p < np) {
            // blocks 2 grp, 2 grp + 1 of the pair; those past K: 0
            const int left = (int)(KS - 8 * (int64_t)p) - 2 * grp;
            const uint32_t both = EVEN ? scale[i] : scale[i] | (scale1[EVEN ? 0 : i] << 8);
            const uint32_t sw = left >= 2 ? both : (left == 1 ? both & 0xFFu : 0u);
#pragma unroll
            for (int b = 0; b < RB; ++b)
              if (b == 0 || 16 * b < rows) {
                const int r = 16 * b + r16;
                const uint8_t* row = codes + r * ld + 128 * p + 32 * grp;
                const u32x4 a0 = *reinterpret_cast<const u32x4*>(row), a1 = *reinterpret_cast<const u32x4*>(row + 16);
                const uint32_t sa = *reinterpret_cast<const uint16_t*>(ascale + r * sld + 8 * p + 2 * grp);
                acc[b] = mfma_fp4<0>(code[i][0], a0, acc[b], sw, sa);
                acc[b] = mfma_fp4<1>(code[i][1], a1, acc[b], sw, sa);
              }
          }
          load(i, x);
        }
      }
      const int64_t n = 16 * (int64_t)(u - cur.u0) + 4 * grp;
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        const int r = 16 * b + r16;
        if (r < rows) {
          uint16_t* dst = g.out + (row0 + r) * N + n;
          if ((N & 3) == 0 && (reinterpret_cast<uintptr_t>(g.out) & 7) == 0) {
            if (n < N)
              *reinterpret_cast<u32x2*>(dst) = u32x2{pack_bf16x2(acc[b][0], acc[b][1]), pack_bf16x2(acc[b][2], acc[b][3])};
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (n + q < N) dst[q] = to_bf16(acc[b][q]);
          }
        }
      }
    }
    if (!some) have = false;   // no unit in this group: nothing was started for the next
    cur = nxt;
    s0 = s1;
  }
}

template <int RB>
size_t narrow_lds(int64_t K, int32_t E) {
  const int64_t np = (K + 2 * BK - 1) / (2 * BK);
  return (size_t)(16 * RB * (np * 128 + 16 + np * 8) + 8 * ((int64_t)E + 1));
}

template <int RB, bool PRE, bool EVEN>
hipError_t narrow_one(const W4A4Args& g, int cus, hipStream_t s) {
  const size_t bytes = narrow_lds<RB>(g.K, g.E);
  auto k = w4a4_narrow_kernel<RB, PRE, EVEN>;
  if (bytes > (64u << 10)) {
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize,
                                       kMaxLds);
    if (e != hipSuccess) return e;
  }
  const int64_t nblk = (g.N + 15) / 16;
  const int64_t units = ((g.M + 16 * RB - 1) / (16 * RB) + std::min<int64_t>(g.E, g.M)) * nblk;
  // two workgroups of 8 wavefronts per CU where the rows leave room for both
  const int64_t per_cu = 2 * (int64_t)bytes <= kMaxLds ? 2 : 1;
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(units, per_cu * cus));
  hipLaunchKernelGGL(k, dim3((unsigned)grid), dim3(NThreads), (unsigned)bytes, s, g);
  return hipGetLastError();
}

}  // namespace

// Row blocks of 16 per unit of the narrow kernel for a batch of M rows over E experts,
// 0 for the tiles: two once experts hold more than four rows on average (larger ones then
// read their weights half as often), as long as the rows fit in LDS. `force`: 0 by size,
// 2 the tiles, 4 the narrow kernel wherever the rows fit.
int w4a4_narrow_rb(int64_t M, int64_t K, int32_t E, int force) {
  if (force == 2 || (force == 0 && M > kW4A4NarrowAvg * (int64_t)E)) return 0;
  if (M > 4 * (int64_t)E && narrow_lds<2>(K, E) <= (size_t)kMaxLds) return 2;
  return narrow_lds<1>(K, E) <= (size_t)kMaxLds ? 1 : 0;
}

// Whether the narrow kernel quantises its rows itself (each workgroup a group's rows again)
// instead of reading what a launch before it quantised: up to one row per expert on
// average. At 8 (K = 2880, E = 32) it took 46 us of which 14 were the conversion.
bool w4a4_narrow_fused(int64_t M, int32_t E) { return M <= (int64_t)E; }

hipError_t launch_w4a4_narrow(const W4A4Args& g, int rb, int cus, hipStream_t s) {
  const bool even = ((g.K >> 5) & 1) == 0 && (reinterpret_cast<uintptr_t>(g.ws) & 1) == 0;
  auto run = [&](auto r, auto p) {
    constexpr int RB = decltype(r)::value;
    constexpr bool PRE = decltype(p)::value;
    return even ? narrow_one<RB, PRE, true>(g, cus, s) : narrow_one<RB, PRE, false>(g, cus, s);
  };
  constexpr std::integral_constant<int, 1> one{};
  constexpr std::integral_constant<int, 2> two{};
  if (g.aq) return rb == 2 ? run(two, std::true_type{}) : run(one, std::true_type{});
  return run(one, std::false_type{});   // no more rows than experts: one block of 16
}

hipError_t launch_w4a4_quantize(const W4A4Args& g, uint8_t* codes, uint8_t* scales, bool tiles, int cus, hipStream_t s) {
  const int64_t M = g.M, K = g.K;
  const int64_t KS = K >> 5, pieces = M * KS * 4;
  const dim3 grid((unsigned)std::min<int64_t>((pieces + kThreads - 1) / kThreads, (int64_t)cus * 16)), block(kThreads);
  uint32_t* c = reinterpret_cast<uint32_t*>(codes);
  if (tiles)
    hipLaunchKernelGGL(w4a4_quantize_kernel<true>, grid, block, 0, s, g.a, M, KS, g.sizes, g.E, c, scales, g.err);
  else
    hipLaunchKernelGGL(w4a4_quantize_kernel<false>, grid, block, 0, s, g.a, M, KS, g.sizes, g.E, c, scales, g.err);
  return hipGetLastError();
}

hipError_t launch_w4a4_tile(const W4A4Args& g, int cus, hipStream_t s) {
  const int64_t n_tiles = (g.N + TN - 1) / TN;
  const int64_t bound = ((g.M + TM - 1) / TM + std::min<int64_t>(g.E, g.M)) * n_tiles;
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(bound, (int64_t)cus));
  if (g.K < 256)
    hipLaunchKernelGGL(w4a4_tile_short_kernel, dim3((unsigned)grid), dim3(TThreads), 0, s, g);
  else
    hipLaunchKernelGGL(w4a4_tile_kernel, dim3((unsigned)grid), dim3(TThreads), 0, s, g);
  return hipGetLastError();
}

}  // namespace geg
