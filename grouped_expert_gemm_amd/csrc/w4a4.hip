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
// bf16 [M, K] -> codes [M, K/2] and scales. For the narrow kernel [M, K/32]; for the tiles
// [K/512 rounded up][M][16]: byte 4 b + s of a row's 16 is the scale of 32-block 4 s + b of
// the 512-wide piece, so a lane of group b reads the bytes of its four steps s as one
// dword; blocks past K get 0. One thread per 8 values, four lanes to a block.
template <bool TILES>
__global__ __launch_bounds__(kThreads) void w4a4_quantize_kernel(const uint16_t* __restrict__ a, int64_t M, int64_t KS,
                                                                 uint32_t* __restrict__ codes,
                                                                 uint8_t* __restrict__ scales, uint32_t* err) {
  const int64_t pieces = M * KS * 4;
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  for (int64_t p = (int64_t)blockIdx.x * kThreads + threadIdx.x; p < pieces; p += stride) {
    float f[8], q[8];
    unpack16<kBF16>(reinterpret_cast<const u32x4*>(a)[p], f);
    uint32_t word;
    const int byte = mxfp4_block_piece<8, false>(f, word, q);
    codes[p] = word;
    if ((p & 3) == 0) {
      if (byte == 255) atomicOr(err, kErrNonFinite);
      const int64_t b = p >> 2;
      if constexpr (TILES) {
        const int64_t m = b / KS, kb = b - m * KS;
        scales[((kb >> 4) * M + m) * 16 + 4 * (kb & 3) + ((kb >> 2) & 3)] = (uint8_t)byte;
      } else {
        scales[b] = (uint8_t)byte;
      }
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
constexpr int kSideStage = TM * (BK / 2);  // bytes of one operand per step
constexpr int kTileStage = 2 * kSideStage;
static_assert(TM == TN, "both operands stage alike");

// Row r of a staged operand holds 4 chunks of 16 bytes, chunk c at c ^ ((r / 4) % 4): the
// fragment reads (16 rows at one chunk each) then touch 8 distinct 16-byte bank groups
// per 8 lanes.
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return (uint32_t)(r * (BK / 2) + ((c ^ ((r >> 2) & 3)) << 4));
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
// blocks fastest, so that the tiles that share weights run together on one XCD). Each
// 128-wide step is staged by loads that write LDS directly (16 bytes per lane, 1 KB per
// instruction), three steps ahead in four buffers, which are distinct LDS objects named
// at compile time: the compiler then adds no wait for loads that fill the others. Scales
// go by pieces of four steps: the activations' 4 KB by direct loads, the weights' bytes
// (rows of K / 32 bytes, of any alignment) through registers, put in lane order on the
// way to LDS; one dword per lane then serves four steps, the instruction picking the
// byte. A wavefront computes 128 x 64: per step 8 + 4 fragments for 32 instructions, so
// LDS (12 KB per wavefront and step) and the matrix pipes are about equally loaded, and
// the HBM stream of the weights is what the kernel waits for.
__global__ __launch_bounds__(TThreads, 1) void w4a4_tile_kernel(W4A4Args g) {
  __shared__ int32_t p_off[kMaxExperts + 1];
  __shared__ int32_t p_u[kMaxExperts + 1];
  __shared__ __attribute__((aligned(16))) uint8_t lds0[kTileStage];
  __shared__ __attribute__((aligned(16))) uint8_t lds1[kTileStage];
  __shared__ __attribute__((aligned(16))) uint8_t lds2[kTileStage];
  __shared__ __attribute__((aligned(16))) uint8_t lds3[kTileStage];
  __shared__ __attribute__((aligned(16))) uint8_t sc0[(TM + TN) * 16];
  __shared__ __attribute__((aligned(16))) uint8_t sc1[(TM + TN) * 16];
  const int64_t K = g.K, N = g.N, KS = K >> 5, M = g.M;
  const int n_tiles = (int)((N + TN - 1) / TN);
  const int32_t total = build_plan(p_off, p_u, g.sizes, g.E, M, g.err,
                                   [&](int32_t s) -> int32_t { return (s + TM - 1) / TM * n_tiles; });
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int r16 = lane & 15, grp = lane >> 4;
  const int nst = (int)((K + BK - 1) / BK), nss = (nst + 3) / 4;
  const int G = gridDim.x;
  const int slot = (G % 8 == 0) ? (blockIdx.x % 8) * (G / 8) + blockIdx.x / 8 : blockIdx.x;

  // Staging: a wavefront fills rows 16 wave + 128 i .. +15 (i = 0, 1) of each operand;
  // lane l lands in slot l % 4 of row l / 4 and fetches the chunk that belongs there.
  const int cp_r = 16 * wave + (lane >> 2), cp_c = (lane & 3) ^ ((cp_r >> 2) & 3);
  const uint32_t rd_a = chunk_at(128 * wm + r16, grp);               // fragment i: + 1024 i
  const uint32_t rd_w = kSideStage + chunk_at(64 * wn + r16, grp);   // fragment j: + 1024 j
  const uint32_t rd_sa = (uint32_t)((128 * wm + r16) * 16 + 4 * grp);       // + 256 i
  const uint32_t rd_sw = (uint32_t)((TM + 64 * wn + r16) * 16 + 4 * grp);   // + 256 j

  for (int32_t base = 0; base < total; base += G) {
    const int32_t u = base + slot;
    if (u >= total) break;
    const int e = find_expert(p_u, g.E, u);
    const int32_t lu = u - p_u[e];
    const int rblocks = (p_off[e + 1] - p_off[e] + TM - 1) / TM;
    const int nt = lu / rblocks, mt = lu % rblocks;
    const int64_t row0 = p_off[e] + (int64_t)mt * TM;
    const int rows = (int)min<int64_t>(TM, p_off[e + 1] - row0);
    const int64_t n0 = (int64_t)nt * TN;
    const int ncols = (int)min<int64_t>(TN, N - n0);
    // rows past the expert's and columns past N read as zeros
    const __amdgpu_buffer_rsrc_t RA = wrsrc(g.aq + row0 * (K >> 1), (int64_t)rows * (K >> 1));
    const __amdgpu_buffer_rsrc_t RW = wrsrc(g.wq + ((int64_t)e * N + n0) * (K >> 1), (int64_t)ncols * (K >> 1));

    auto stage = [&](int st, uint8_t* L) {
      const bool ok = (int64_t)st * 4 + cp_c < KS;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t off = oob_unless(ok, (uint32_t)((cp_r + 128 * i) * (K >> 1) + 64 * (int64_t)st + 16 * cp_c));
        __builtin_amdgcn_raw_ptr_buffer_load_lds(RA, (lds_ptr_t)(L + (16 * wave + 128 * i) * (BK / 2)), 16, off, 0, 0,
                                                 0);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            RW, (lds_ptr_t)(L + kSideStage + (16 * wave + 128 * i) * (BK / 2)), 16, off, 0, 0, 0);
      }
    };
    // Scales of piece ss: wavefronts 0-3 load the activations' straight into `sc` (64 rows
    // each); every thread loads half a weight column's 16 bytes (two steps' four) into
    // registers. (All wavefronts alike: a value that only some load would be copied where
    // the paths join, behind a wait for every load in flight.)
    const int wcol = t >> 1, whalf = t & 1;
    const uint8_t* wsp = g.ws + ((int64_t)e * N + n0 + min(wcol, ncols - 1)) * KS + 8 * whalf;
    // rows of the tile past M read zeros, rows of the next expert their own bytes
    const int64_t sleft = (M - row0) * 16;
    auto scales = [&](int ss, uint8_t* sc, u32x2& d) {
      if (wave < 4) {
        const __amdgpu_buffer_rsrc_t RS = wrsrc(g.as + ((int64_t)min(ss, nss - 1) * M + row0) * 16, sleft);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(RS, (lds_ptr_t)(sc + wave * 1024), 16,
                                                 (uint32_t)(wave * 1024 + 16 * lane), 0, 0, 0);
      }
      if (16 * (ss + 1) <= (int)KS) {
        __builtin_memcpy(&d, wsp + 16 * ss, 8);
      } else {
        // the last piece, byte by byte; blocks past K get 0
        d = u32x2{0, 0};
#pragma unroll
        for (int b = 0; b < 8; ++b)
          if (16 * ss + 8 * whalf + b < (int)KS) d[b >> 2] |= (uint32_t)wsp[16 * ss + b] << (8 * (b & 3));
      }
    };
    // byte 4 b + s of a column's 16 in LDS: block b of step s (from byte 4 s + b)
    auto put_scales = [&](uint8_t* sc, const u32x2& d) {
      uint8_t* p = sc + (TM + wcol) * 16 + 2 * whalf;
      const uint32_t lo = perm(d[1], d[0], 0x05010400u), hi = perm(d[1], d[0], 0x07030602u);
      *reinterpret_cast<uint16_t*>(p) = (uint16_t)lo;
      *reinterpret_cast<uint16_t*>(p + 4) = (uint16_t)(lo >> 16);
      *reinterpret_cast<uint16_t*>(p + 8) = (uint16_t)hi;
      *reinterpret_cast<uint16_t*>(p + 12) = (uint16_t)(hi >> 16);
    };

    const bool live = 128 * wm < rows;
    f32x4 acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    u32x2 d = u32x2{0, 0};

    // Step S of piece ss: its operands are in `cur` (barrier of the step before); stage
    // st + 3 goes to `nxt`, the buffer that step st - 1 read. With S == 0 the next piece's
    // scales start, with S == 3 they are published. At the end stage st + 1 has landed
    // (the 8 loads of the two stages after it may be in flight).
    auto step = [&](auto Sc, int ss, const uint8_t* cur, uint8_t* nxt, const uint8_t* sc, uint8_t* scn) {
      constexpr int S = decltype(Sc)::value;
      if constexpr (S == 0) scales(ss + 1, scn, d);
      stage(4 * ss + S + 3, nxt);
      if (live) {
        u32x4 w[4], a[8];
        uint32_t sw[4], sa[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          w[j] = *reinterpret_cast<const u32x4*>(cur + rd_w + 1024 * j);
          sw[j] = *reinterpret_cast<const uint32_t*>(sc + rd_sw + 256 * j);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a[i] = *reinterpret_cast<const u32x4*>(cur + rd_a + 1024 * i);
          sa[i] = *reinterpret_cast<const uint32_t*>(sc + rd_sa + 256 * i);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = mfma_fp4<S>(w[j], a[i], acc[i][j], sw[j], sa[i]);
      }
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (S == 3) put_scales(scn, d);
      step_barrier<8>();
    };
    constexpr std::integral_constant<int, 0> s0{};
    constexpr std::integral_constant<int, 1> s1{};
    constexpr std::integral_constant<int, 2> s2{};
    constexpr std::integral_constant<int, 3> s3{};

    scales(0, sc0, d);
    stage(0, lds0);
    stage(1, lds1);
    stage(2, lds2);
    put_scales(sc0, d);
    step_barrier<8>();
    int ss = 0;
    for (; 4 * (ss + 2) <= nst; ss += 2) {
      step(s0, ss, lds0, lds3, sc0, sc1);
      step(s1, ss, lds1, lds0, sc0, sc1);
      step(s2, ss, lds2, lds1, sc0, sc1);
      step(s3, ss, lds3, lds2, sc0, sc1);
      step(s0, ss + 1, lds0, lds3, sc1, sc0);
      step(s1, ss + 1, lds1, lds0, sc1, sc0);
      step(s2, ss + 1, lds2, lds1, sc1, sc0);
      step(s3, ss + 1, lds3, lds2, sc1, sc0);
    }
    const int rest = nst - 4 * ss;
    if (rest > 0) step(s0, ss, lds0, lds3, sc0, sc1);
    if (rest > 1) step(s1, ss, lds1, lds0, sc0, sc1);
    if (rest > 2) step(s2, ss, lds2, lds1, sc0, sc1);
    if (rest > 3) step(s3, ss, lds3, lds2, sc0, sc1);
    if (rest > 4) step(s0, ss + 1, lds0, lds3, sc1, sc0);
    if (rest > 5) step(s1, ss + 1, lds1, lds0, sc1, sc0);
    if (rest > 6) step(s2, ss + 1, lds2, lds1, sc1, sc0);
    step_barrier<0>();   // loads past the last step have landed: the buffers are free

    // Epilogue: the wavefront's 128 x 64 block as bf16 rows of 128 bytes in its own 16 KB
    // (16-byte piece p of row r at p ^ (r % 8)), then 16-byte pieces of whole rows.
    if (live) {
      uint8_t* L = (wave < 4 ? (wave < 2 ? lds0 : lds1) : (wave < 6 ? lds2 : lds3)) + (wave & 1) * (kTileStage / 2);
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = 16 * i + r16;
          const u32x2 v = u32x2{pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3])};
          *reinterpret_cast<u32x2*>(L + r * 128 + (((2 * j + (grp >> 1)) ^ (r & 7)) << 4) + 8 * (grp & 1)) = v;
        }
      __builtin_amdgcn_wave_barrier();
      asm volatile("" ::: "memory");
      const bool wide = (N & 7) == 0 && (reinterpret_cast<uintptr_t>(g.out) & 15) == 0;
      const int pc = lane & 7;
      const int64_t col = n0 + 64 * wn + 8 * pc;
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const int r = 8 * q + (lane >> 3), lr = 128 * wm + r;
        const u32x4 v = *reinterpret_cast<const u32x4*>(L + r * 128 + ((pc ^ (r & 7)) << 4));
        if (lr < rows) {
          uint16_t* dst = g.out + (row0 + lr) * N + col;
          if (wide) {
            if (col < N) *reinterpret_cast<u32x4*>(dst) = v;
          } else {
#pragma unroll
            for (int b = 0; b < 8; ++b)
              if (col + b < N) dst[b] = (uint16_t)(v[b >> 1] >> (16 * (b & 1)));
          }
        }
      }
    }
    step_barrier<63>();   // LDS reads done before the next tile's loads land
  }
}

// ------------------------------------------------------------------ narrow
// Wavefront units: 16 output columns of one expert and up to 16 RB of its rows (a group),
// over the whole contraction. A workgroup takes a contiguous run of units, group by
// group: it quantises a group's rows into LDS once, then its wavefronts stream the weight
// rows of their units straight into registers (64 consecutive bytes of each of 16 rows per
// instruction and pair), PD pairs of steps ahead at all times, across units and groups: no
// barrier and no cross-wavefront sum between them.
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
  return rb == 2 ? run(two, std::false_type{}) : run(one, std::false_type{});
}

hipError_t launch_w4a4_quantize(const uint16_t* a, int64_t M, int64_t K, uint8_t* codes, uint8_t* scales, uint32_t* err,
                                bool tiles, int cus, hipStream_t s) {
  const int64_t KS = K >> 5, pieces = M * KS * 4;
  const dim3 grid((unsigned)std::min<int64_t>((pieces + kThreads - 1) / kThreads, (int64_t)cus * 16)), block(kThreads);
  uint32_t* c = reinterpret_cast<uint32_t*>(codes);
  if (tiles)
    hipLaunchKernelGGL(w4a4_quantize_kernel<true>, grid, block, 0, s, a, M, KS, c, scales, err);
  else
    hipLaunchKernelGGL(w4a4_quantize_kernel<false>, grid, block, 0, s, a, M, KS, c, scales, err);
  return hipGetLastError();
}

hipError_t launch_w4a4_tile(const W4A4Args& g, int cus, hipStream_t s) {
  const int64_t n_tiles = (g.N + TN - 1) / TN;
  const int64_t bound = ((g.M + TM - 1) / TM + std::min<int64_t>(g.E, g.M)) * n_tiles;
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(bound, (int64_t)cus));
  hipLaunchKernelGGL(w4a4_tile_kernel, dim3((unsigned)grid), dim3(TThreads), 0, s, g);
  return hipGetLastError();
}

}  // namespace geg
