// The routed experts of a whole MoE layer for a few tokens, in two kernels:
//     act[s, i] = silu(x_t . G_i) * (x_t . U_i)        for every (token, slot) s of t
//     out[t]    = sum_s w_s (act[s] . W2_e(s)^T)
// with e(s) the slot's expert, G_i / U_i rows 2i / 2i+1 of its fused gate/up weight.
// The first kernel reads the tokens and the gate/up weights, the second the down
// weights; the router's weighted sum is taken in the second one's fp32 sums, so
// neither a sort, a gathered copy of the rows nor a combine pass runs.
//
// Bound by streaming the packed weights of the experts that the tokens touch, each
// byte once: the (token, slot) entries are grouped by expert in LDS (at most 256
// entries: their places come from counting, no sort), and a wavefront that holds a
// piece of an expert's weight rows in registers takes the dot products of all of
// that expert's tokens with it, two at a time, before it moves on.
//
// A wavefront takes ROWS weight rows at a time: LPR lanes per row (64, 32 or 16, by the
// row length), U = ROWS LPR / 64 row groups, each lane a 16-byte chunk of 32 codes per
// row and pass, against the tokens' same 32 values with packed fp32-accumulated dot
// products. NF4 codes go through the byte table in LDS (two fp16 values per 32-bit
// read), MXFP4 through the scaled fp4 conversion; the block scale multiplies the
// chunk's fp32 dot product. One workgroup of 16 wavefronts per CU shares the table, the
// grouping and the staged tokens.
//
// act goes from one kernel to the other as fp16 with a power-of-two scale per 32 values
// that puts the block's largest in [2^14, 2^15): 11 bits for everything within 2^-29 of
// it, whatever the layer's scale, and a lane's 32 values are one such block, so the
// scale joins the weight's in the one product per chunk. (fp32 activations against
// mixed-precision fmas took twice the arithmetic and three times the registers: 714
// against 92 us for the second kernel of 8 experts of 4096 x 14336, four tokens.)
#include <algorithm>

#include "geg_device.hpp"
#include "geg_launch.hpp"

namespace geg {

namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));

constexpr int MT = 1024;             // threads per workgroup
constexpr int MW = MT / 64;          // wavefronts
constexpr int MG = 4;                // entries per item (an expert with more gets several)
constexpr int UP_ROWS = 4;           // first kernel: weight rows per wavefront and unit,
constexpr int UNIT_ROWS = UP_ROWS * MW;   // per workgroup: 64, the 32 act values of a block
static_assert(UNIT_ROWS == 64, "a unit of the first kernel makes one block of act");

__device__ __forceinline__ __amdgpu_buffer_rsrc_t mrsrc(const void* base, int64_t bytes) {
  const int32_t n = bytes > 0x7FFFFFF0 ? 0x7FFFFFF0 : (int32_t)bytes;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, n, 0x00020000);
}

__device__ __forceinline__ float fdot2(uint32_t a, uint32_t b, float c, std::integral_constant<int, NF4>) {
  return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, a), __builtin_bit_cast(f16x2, b), c, false);
}
__device__ __forceinline__ float fdot2(uint32_t a, uint32_t b, float c, std::integral_constant<int, MXFP4>) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2v, a), __builtin_bit_cast(bf16x2v, b), c, false);
}

// v + the value r lanes away, cyclically, in the lane's row of 16.
template <int R>
__device__ __forceinline__ float ror_add(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x120 + R, 0xF, 0xF,
                                                                   false));
}

// a's and b's sums over pairs of half wavefronts (or of 16-lane rows): lanes of the
// lower half (even rows) get a's, the others b's.
__device__ __forceinline__ float fold32(float a, float b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  const uint32_t x = r[0], y = r[1];
  return __uint_as_float(x) + __uint_as_float(y);
}
__device__ __forceinline__ float fold16(float a, float b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  const uint32_t x = r[0], y = r[1];
  return __uint_as_float(x) + __uint_as_float(y);
}

// Grouping of the T k entries by expert, in LDS. Entry f's place is the number of
// entries with a smaller expert, or the same and a smaller index; dropped entries
// (an id outside [0, E)) get none. item[q] is the q-th run of at most MG places of one
// expert.
struct Groups {
  int32_t id[kMoeMaxEntries];       // expert of each entry, -1 for a dropped one
  int32_t ent[kMoeMaxEntries];      // entry at each place
  int32_t lead[kMoeMaxEntries];     // at a run's first place its expert, else -1
  int32_t count[kMoeMaxEntries];    // at a run's first place its entries
  int32_t expert[kMoeMaxEntries];   // of each item: expert, first place, entries
  int32_t first[kMoeMaxEntries];
  int32_t size[kMoeMaxEntries];
  int32_t items;
};

// Every thread of the workgroup calls it (barriers inside). `err` (may be NULL)
// receives the flag of a dropped entry. `mine` is entry threadIdx.x's expert.
__device__ __forceinline__ void group_entries(Groups& g, int mine, int n, int E, uint32_t* err) {
  const int t = threadIdx.x;
  if (t < n && (mine < 0 || mine >= E)) {
    if (err) atomicOr(err, kErrBadExpertId);
    mine = -1;
  }
  if (t < kMoeMaxEntries) {
    g.id[t] = t < n ? mine : -1;
    g.lead[t] = -1;
  }
  lds_barrier();
  if (t < n && mine >= 0) {
    int place = 0, rank = 0, cnt = 0;
    for (int f0 = 0; f0 < n; f0 += 4) {   // the same address on every lane: broadcast reads
      const i32x4 v = *reinterpret_cast<const i32x4*>(g.id + f0);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = v[j];
        const bool before = f0 + j < t;
        place += e >= 0 && (e < mine || (e == mine && before));
        rank += e == mine && before;
        cnt += e == mine;
      }
    }
    g.ent[place] = t;
    if (rank % MG == 0) {
      g.lead[place] = mine;
      g.count[place] = min(MG, cnt - rank);
    }
  }
  lds_barrier();
  if (t < 64) {
    int q = 0;   // runs so far, 64 places per ballot
    for (int base = 0; base < n; base += 64) {
      const int e = g.lead[base + t];
      const uint64_t at = __ballot(e >= 0);
      if (e >= 0) {
        const int to = q + __builtin_popcountll(at & ((1ull << t) - 1));
        g.expert[to] = e;
        g.first[to] = base + t;
        g.size[to] = g.count[base + t];
      }
      q += __builtin_popcountll(at);
    }
    if (t == 0) g.items = q;
  }
  lds_barrier();
}

// Sums of per-lane values d[u][m] over the LPR lanes of their rows, added into
// acc[(m0 + m) * R + row], R = U * 64 / LPR rows, by the lanes that end up with them.
// (An odd count's missing second entry adds a duplicate to a row that nobody reads.)
template <int LPR, int U, int RV>
__device__ __forceinline__ void add_sums(const float (&d)[U][RV], int lane, int m0, float* acc) {
  constexpr int G = 64 / LPR, R = U * G;
  constexpr int F = LPR / 16;   // row groups folded into the wavefront's four rows of 16 lanes
  static_assert(U % F == 0, "whole folds");
  const int row16 = lane >> 4;
  float v[U / F][RV];
#pragma unroll
  for (int u = 0; u < U; u += F)
#pragma unroll
    for (int m = 0; m < RV; ++m) {
      float x;
      if constexpr (F == 4)
        x = fold16(fold32(d[u][m], d[u + 1][m]), fold32(d[u + 2][m], d[u + 3][m]));
      else if constexpr (F == 2)
        x = fold16(d[u][m], d[u + 1][m]);
      else
        x = d[u][m];
      x = ror_add<8>(x);
      x = ror_add<4>(x);
      x = ror_add<2>(x);
      v[u / F][m] = ror_add<1>(x);
    }
  // the rows of 16 lanes hold u + 0, 2, 1, 3 (F = 4); u, u + 1 of lane group 0, then of 1
  // (F = 2); lane groups 0..3 (F = 1)
  const int row = F == 4 ? (((row16 & 1) << 1) | (row16 >> 1)) : (F == 2 ? G * (row16 & 1) + (row16 >> 1) : row16);
  if ((lane & 15) == 0) {
    float* p = acc + m0 * R + row;
#pragma unroll
    for (int u = 0; u < U / F; ++u)
#pragma unroll
      for (int m = 0; m < RV; ++m) p[m * R + u * F * G] += v[u][m];
  }
}

// 8 e2m1 codes to fp16, natural order (exact).
__device__ __forceinline__ u32x4 mxfp4_decode8_f16(uint32_t x) {
  u32x4 r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(x, 1.0f, 0));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(x, 1.0f, 1));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(x, 1.0f, 2));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(x, 1.0f, 3));
  return r;
}

// The packed codes and scales of one pass: chunk c of rows n0 + G u + gl.
template <Fmt F, int LPR, int U>
struct Codes {
  u32x4 code[U];
  uint32_t scale[U];
  __device__ __forceinline__ void load(const __amdgpu_buffer_rsrc_t& W, const __amdgpu_buffer_rsrc_t& S, int64_t n0,
                                       int gl, int64_t K, int c, uint32_t off_mask) {
    constexpr int G = 64 / LPR;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t n = n0 + G * u + gl;   // rows past the matrix read as zero (buffer bounds)
      code[u] = __builtin_amdgcn_raw_buffer_load_b128(W, (uint32_t)(n * (K >> 1) + 16 * c) | off_mask, 0, 0);
      if constexpr (F == NF4)
        scale[u] = __builtin_amdgcn_raw_buffer_load_b32(S, (uint32_t)((n * (K >> 6) + (c >> 1)) * 4) | off_mask, 0, 0);
      else
        scale[u] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(S, (uint32_t)(n * (K >> 5) + c) | off_mask, 0, 0);
    }
  }
  // Makes row group u's codes new values to the compiler, and keeps what follows behind
  // what came before: decoded values are then neither kept from one pair of tokens to the
  // next nor made for several row groups at once (16 registers per code word: spills).
  __device__ __forceinline__ void next(int u) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t v = code[u][j];
      asm volatile("" : "+v"(v));
      code[u][j] = v;
    }
  }
  __device__ __forceinline__ float scale_f32(int u) const {
    return F == NF4 ? __uint_as_float(scale[u]) : e8m0_to_f32(scale[u]);
  }
};

template <Fmt F>
__device__ __forceinline__ const void* expert_scales(const void* s, int e, int64_t N, int64_t K) {
  if constexpr (F == NF4)
    return reinterpret_cast<const float*>(s) + (int64_t)e * N * (K >> 6);
  else
    return reinterpret_cast<const uint8_t*>(s) + (int64_t)e * N * (K >> 5);
}
template <Fmt F>
__device__ __forceinline__ int64_t scale_bytes(int64_t N, int64_t K) {
  return F == NF4 ? N * (K >> 6) * 4 : N * (K >> 5);
}

// The staged tokens: chunk c of token t as four 16-byte pieces, piece j at
// ((4 t + j) C + c) 16 bytes, so that the lanes of a wavefront (consecutive chunks)
// read consecutive pieces.
template <Fmt F>
constexpr int x_lds_bytes() { return F == NF4 ? 64 << 10 : 140 << 10; }

// First kernel. Units (item, 64 rows of its gate/up weight = 32 values of act) over a grid
// of one workgroup per CU, 4 rows per wavefront; a wavefront's codes of the next unit are
// in flight while it works on this one. x is staged in LDS when all tokens fit (XL), as
// fp16 for NF4 (flagged when it overflows; MXFP4 keeps bf16, exact), else each lane loads
// its slice from memory. The sums meet in LDS, where a half wavefront per entry forms the
// 32 act values, their scale and their fp16 form (value i = 32 c + 8 j + b of a row at
// ((j (I / 32) + c) 8 + b): the order in which the second kernel's lanes read it).
// Workgroup 0 also writes the grouping.
template <Fmt F, int LPR, int RV, bool XL>
__global__ __launch_bounds__(MT) void moe_up_kernel(MoeArgs g) {
  constexpr int G = 64 / LPR, U = UP_ROWS / G;
  constexpr std::integral_constant<int, F> fmt{};
  __shared__ __attribute__((aligned(16))) Groups grp;
  __shared__ __attribute__((aligned(16))) uint32_t blut[F == NF4 ? kNf4ByteLutWords : 4];
  __shared__ __attribute__((aligned(16))) uint8_t xs[XL ? x_lds_bytes<F>() : 16];
  __shared__ float accs[2][MW][MG * UP_ROWS];
  const int n = g.T * g.k;
  const int64_t H = g.H, N = 2 * g.I;
  const int C = (int)(H >> 5), CI = (int)(g.I >> 5);
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  uint32_t range = 0;
  const int my_id = t < n ? g.ids[t] : 0;   // in flight during the set-up
  if constexpr (XL) {
    const int pieces = g.T * 4 * C;   // 8 values each
    for (int p = t; p < pieces; p += MT) {
      const int tok = p / (4 * C), q = p % (4 * C);   // piece q of the token: chunk q / 4, piece q % 4
      u32x4 v = reinterpret_cast<const u32x4*>(g.x)[p];
      if constexpr (F == NF4) v = bf16x8_to_f16(v, range);
      *reinterpret_cast<u32x4*>(xs + ((4 * tok + (q & 3)) * C + (q >> 2)) * 16) = v;
    }
  }
  if constexpr (F == NF4) nf4_byte_lut_fill<64, MT>(blut);
  group_entries(grp, my_id, n, g.E, blockIdx.x == 0 ? g.err : nullptr);
  const int items = grp.items;
  if (blockIdx.x == 0 && t < kMoeMaxEntries) {
    if (t == 0) g.plan[0] = items;
    if (t < items) {
      g.plan[4 + 2 * t] = grp.expert[t];
      g.plan[4 + 2 * t + 1] = grp.first[t] | (grp.size[t] << 16);
    }
    if (t < n) g.plan[4 + 2 * kMoeMaxEntries + t] = grp.ent[t];
  }
  const int gl = lane / LPR, li = lane % LPR;
  const uint32_t lane_off = nf4_byte_lut_lane(lane);
  const int total = items * CI;
  const __amdgpu_buffer_rsrc_t X = mrsrc(g.x, (int64_t)g.T * H * 2);
  // codes of pass c0 of a unit
  auto load = [&](int unit, int c0, Codes<F, LPR, U>& w) {
    const int e = __builtin_amdgcn_readfirstlane(grp.expert[unit / CI]);
    const __amdgpu_buffer_rsrc_t W = mrsrc(g.w13 + (int64_t)e * N * (H >> 1), N * (H >> 1));
    const __amdgpu_buffer_rsrc_t S = mrsrc(expert_scales<F>(g.s13, e, N, H), scale_bytes<F>(N, H));
    const int c = c0 + li;
    // chunks past the row read as zero: their offsets lie past every buffer
    w.load(W, S, (int64_t)(unit % CI) * UNIT_ROWS + UP_ROWS * wave, gl, H, c, c < C ? 0u : 0xFFFFFFF0u);
  };
  Codes<F, LPR, U> nxt;
  int par = 0;
  if ((int)blockIdx.x < total) load(blockIdx.x, 0, nxt);
  for (int unit = blockIdx.x; unit < total; unit += gridDim.x, par ^= 1) {
    const int q = unit / CI;
    const int first = __builtin_amdgcn_readfirstlane(grp.first[q]);
    const int cnt = __builtin_amdgcn_readfirstlane(grp.size[q]);
    float* acc = accs[par][wave];
    if (lane < MG * UP_ROWS) acc[lane] = 0.f;
    __builtin_amdgcn_wave_barrier();
    for (int c0 = 0; c0 < C; c0 += LPR) {
      const int c = c0 + li;
      const uint32_t off_mask = c < C ? 0u : 0xFFFFFFF0u;
      Codes<F, LPR, U> w = nxt;
      if (c0 + LPR < C)
        load(unit, c0 + LPR, nxt);
      else if (unit + (int)gridDim.x < total)
        load(unit + gridDim.x, 0, nxt);
      for (int m0 = 0; m0 < cnt; m0 += RV) {
        u32x4 xv[RV][4];
#pragma unroll
        for (int m = 0; m < RV; ++m) {
          const int tok = __builtin_amdgcn_readfirstlane(grp.ent[first + min(m0 + m, cnt - 1)]) / g.k;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (XL) {
              xv[m][j] = *reinterpret_cast<const u32x4*>(xs + ((4 * tok + j) * C + min(c, C - 1)) * 16);
            } else {
              xv[m][j] = __builtin_amdgcn_raw_buffer_load_b128(
                  X, (uint32_t)(((int64_t)tok * H + 32 * c) * 2 + 16 * j) | off_mask, 0, 0);
              if constexpr (F == NF4) xv[m][j] = bf16x8_to_f16(xv[m][j], range);
            }
          }
        }
        float d[U][RV];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          w.next(u);
#pragma unroll
          for (int m = 0; m < RV; ++m) d[u][m] = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            u32x4 v;   // values k = 8j .. 8j+7, natural order
            if constexpr (F == NF4)
              v = nf4_byte_lut_decode8(blut, w.code[u][j], lane_off);
            else
              v = mxfp4_decode8(w.code[u][j], 1.0f);
#pragma unroll
            for (int m = 0; m < RV; ++m)
#pragma unroll
              for (int p = 0; p < 4; ++p) d[u][m] = fdot2(v[p], xv[m][j][p], d[u][m], fmt);
          }
          const float s = w.scale_f32(u);
#pragma unroll
          for (int m = 0; m < RV; ++m) {
            d[u][m] = off_mask ? 0.f : s * d[u][m];
            asm volatile("" : "+v"(d[u][m]));   // finished here, not where it is used
          }
        }
        add_sums<LPR, U, RV>(d, lane, m0, acc);
      }
    }
    lds_barrier();   // the sums of this unit; the other parity's are free again after the next one
    const int m = t >> 5, i = t & 31;
    if (m < cnt) {
      const float* a = accs[par][i >> 1] + m * UP_ROWS + 2 * (i & 1);
      const float v = swiglu(a[0], a[1]);
      uint32_t mx = __float_as_uint(v) & 0x7FFFFFFFu;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, o));
      // the block's largest to [2^14, 2^15); 2^ex stays a normal fp32 value
      const int ex = max((int)(mx >> 23) - 127 - 14, -126);
      const int64_t slot = grp.ent[first + m];
      const int c = unit % CI;
      const _Float16 h = (_Float16)__builtin_ldexpf(v, -ex);
      g.act[slot * g.I + ((i >> 3) * CI + c) * 8 + (i & 7)] = __builtin_bit_cast(uint16_t, h);
      if (i == 0) g.act_scale[slot * CI + c] = __uint_as_float((uint32_t)(ex + 127) << 23);
    }
  }
  if constexpr (F == NF4) {
    if ((blockIdx.x == 0 || !XL) && range_overflowed(range)) atomicOr(g.err, kErrFp16Range);
  }
}

// Second kernel. A workgroup owns RB rows of W2 (columns of out), RB / ROWS subgroups; its
// wavefronts share the (item, subgroup) pieces of work, each adding its weighted sums
// into an own [RB][T] array in LDS; the arrays are added in wavefront order, so results
// do not depend on timing.
template <Fmt F, int LPR, int RV, int ROWS>
__global__ __launch_bounds__(MT) void moe_down_kernel(MoeArgs g) {
  constexpr int G = 64 / LPR, U = ROWS / G;
  constexpr std::integral_constant<int, NF4> f16{};   // both formats multiply fp16 pairs
  __shared__ __attribute__((aligned(16))) uint32_t blut[F == NF4 ? kNf4ByteLutWords : 4];
  __shared__ float outs[MW][kMoeRowBlock * kMoeMaxTokens];   // [wavefront][row][token]
  __shared__ float accs[MW][MG * ROWS];
  const int64_t H = g.H, K = g.I;
  const int C = (int)(K >> 5);
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int gl = lane / LPR, li = lane % LPR;
  const uint32_t lane_off = nf4_byte_lut_lane(lane);
  const int items = g.plan[0];
  if constexpr (F == NF4) nf4_byte_lut_fill<64, MT>(blut);
  const int RB = g.rb, subs = RB / ROWS;
  const int64_t blocks = (H + RB - 1) / RB;
  float* acc = accs[wave];
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
    for (int i = t; i < MW * kMoeRowBlock * kMoeMaxTokens; i += MT) (&outs[0][0])[i] = 0.f;
    __syncthreads();
    for (int wk = wave; wk < items * subs; wk += MW) {
      const int q = wk / subs, sub = wk % subs;
      const int64_t n0 = b * RB + (int64_t)sub * ROWS;
      const int e = g.plan[4 + 2 * q];
      const int fc = g.plan[4 + 2 * q + 1];
      const int first = fc & 0xFFFF, cnt = fc >> 16;
      const __amdgpu_buffer_rsrc_t W = mrsrc(g.w2 + (int64_t)e * H * (K >> 1), H * (K >> 1));
      const __amdgpu_buffer_rsrc_t S = mrsrc(expert_scales<F>(g.s2, e, H, K), scale_bytes<F>(H, K));
      const int32_t* ent = g.plan + 4 + 2 * kMoeMaxEntries + first;
      for (int i = lane; i < MG * ROWS; i += 64) acc[i] = 0.f;
      __builtin_amdgcn_wave_barrier();
      for (int c0 = 0; c0 < C; c0 += LPR) {
        const int c = c0 + li, cc = min(c, C - 1);
        const uint32_t off_mask = c < C ? 0u : 0xFFFFFFF0u;
        Codes<F, LPR, U> w;
        w.load(W, S, n0, gl, K, c, off_mask);
        for (int m0 = 0; m0 < cnt; m0 += RV) {
            u32x4 xv[RV][4];
          float xs[RV];
#pragma unroll
          for (int m = 0; m < RV; ++m) {
            const int64_t f = ent[min(m0 + m, cnt - 1)];
            const u32x4* a = reinterpret_cast<const u32x4*>(g.act + f * K) + cc;
#pragma unroll
            for (int j = 0; j < 4; ++j) xv[m][j] = a[j * C];
            xs[m] = g.act_scale[f * C + cc] * g.weights[f];
          }
          float d[U][RV];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            w.next(u);
#pragma unroll
            for (int m = 0; m < RV; ++m) d[u][m] = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              u32x4 v;
              if constexpr (F == NF4)
                v = nf4_byte_lut_decode8(blut, w.code[u][j], lane_off);
              else
                v = mxfp4_decode8_f16(w.code[u][j]);
#pragma unroll
              for (int m = 0; m < RV; ++m)
#pragma unroll
                for (int p = 0; p < 4; ++p) d[u][m] = fdot2(v[p], xv[m][j][p], d[u][m], f16);
            }
            const float s = w.scale_f32(u);
#pragma unroll
            for (int m = 0; m < RV; ++m) {
              d[u][m] = off_mask ? 0.f : (s * xs[m]) * d[u][m];
              asm volatile("" : "+v"(d[u][m]));
            }
          }
          add_sums<LPR, U, RV>(d, lane, m0, acc);
        }
      }
      __builtin_amdgcn_wave_barrier();
      asm volatile("" ::: "memory");
      // one lane per row of the subgroup adds the item's rows to its tokens
      if (lane < ROWS)
        for (int m = 0; m < cnt; ++m)
          outs[wave][(sub * ROWS + lane) * kMoeMaxTokens + ent[m] / g.k] += acc[m * ROWS + lane];
      __builtin_amdgcn_wave_barrier();
      asm volatile("" ::: "memory");
    }
    __syncthreads();
    for (int i = t; i < RB * g.T; i += MT) {
      const int row = i % RB, tok = i / RB;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < MW; ++w) v += outs[w][row * kMoeMaxTokens + tok];
      const int64_t col = b * RB + row;
      if (col < H) g.out[(int64_t)tok * H + col] = to_bf16(v);
    }
    __syncthreads();
  }
}

template <Fmt F, int LPR, int RV>
hipError_t up_x(const MoeArgs& g, int cus, hipStream_t s) {
  const bool xl = (int64_t)g.T * g.H * 2 <= x_lds_bytes<F>();
  if (xl)
    hipLaunchKernelGGL((moe_up_kernel<F, LPR, RV, true>), dim3((unsigned)cus), dim3(MT), 0, s, g);
  else
    hipLaunchKernelGGL((moe_up_kernel<F, LPR, RV, false>), dim3((unsigned)cus), dim3(MT), 0, s, g);
  return hipGetLastError();
}

// Rows of W2 per workgroup: one round of the chip where that stays within the LDS
// arrays, in whole subgroups of ROWS.
template <Fmt F, int LPR, int RV, int ROWS>
hipError_t down_one(MoeArgs g, int cus, hipStream_t s) {
  const int64_t rb = ((g.H + cus - 1) / cus + ROWS - 1) / ROWS * ROWS;
  g.rb = (int)std::min<int64_t>(rb, kMoeRowBlock);
  const int64_t blocks = (g.H + g.rb - 1) / g.rb;
  hipLaunchKernelGGL((moe_down_kernel<F, LPR, RV, ROWS>), dim3((unsigned)std::min<int64_t>(blocks, cus)), dim3(MT), 0,
                     s, g);
  return hipGetLastError();
}

// f(LPR) with the lanes per weight row for a contraction of K: enough for the row's
// chunks in one pass, at most 64.
template <typename Fn>
hipError_t by_lanes(int64_t K, Fn f) {
  const int64_t C = K >> 5;
  if (C <= 16) return f(std::integral_constant<int, 16>{});
  if (C <= 32) return f(std::integral_constant<int, 32>{});
  return f(std::integral_constant<int, 64>{});
}

template <Fmt F>
hipError_t layer(const MoeArgs& g, int cus, hipStream_t s) {
  const bool single = g.T == 1;
  hipError_t e = by_lanes(g.H, [&](auto l) {
    constexpr int LPR = decltype(l)::value;
    return single ? up_x<F, LPR, 1>(g, cus, s) : up_x<F, LPR, 2>(g, cus, s);
  });
  if (e != hipSuccess) return e;
  return by_lanes(g.I, [&](auto l) {
    constexpr int LPR = decltype(l)::value;
    return single ? down_one<F, LPR, 1, 4>(g, cus, s) : down_one<F, LPR, 2, 8>(g, cus, s);
  });
}

}  // namespace

hipError_t launch_moe_layer(int fmt, const MoeArgs& g, int cus, hipStream_t s) {
  return fmt == NF4 ? layer<NF4>(g, cus, s) : layer<MXFP4>(g, cus, s);
}

}  // namespace geg
