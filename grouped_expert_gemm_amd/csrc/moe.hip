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
// entries: their places come from counting, no sort) into items of one expert and at
// most four entries, and a wavefront decodes a piece of an item's weight rows once for
// the dot products of all its entries.
//
// A wavefront takes ROWS weight rows at a time: LPR lanes per row (64, 32 or 16, by the
// row length), U = ROWS LPR / 64 row groups, each lane a 16-byte chunk of 32 codes per
// row and pass, against the tokens' same 32 values with packed fp32-accumulated dot
// products. NF4 codes go through the byte table in LDS (two fp16 values per 32-bit
// read), MXFP4 through the scaled fp4 conversion; the block scale multiplies the
// chunk's fp32 dot product. A workgroup shares the table, the grouping and the staged
// tokens.
//
// NF4 multiplies fp16 values: each token is first multiplied by a power of two that puts its
// largest magnitude in [2^14, 2^15) and the sums by the inverse, both exact, so that no token
// under- or overflows, whatever its scale. MXFP4 multiplies bf16 as it is.
//
// act goes from one kernel to the other as fp16 with a power-of-two scale per 32 values
// that puts the block's largest in [2^14, 2^15): 11 bits for everything within 2^-29 of
// it, whatever the layer's scale, and a lane's 32 values are one such block, so the
// scale joins the weight's in the one product per chunk. (fp32 activations against
// mixed-precision fmas took twice the arithmetic and three times the registers: for the
// second kernel of 8 experts of 4096 x 14336, four tokens, 714 us against 37 now.)
//
// Both kernels together, in a kernel trace: 8 experts of 4096 x 14336, top 2, four tokens:
// 99 to 103 us for 542 MB (5.4 TB/s). 128 experts of 2048 x 768, top 8: one token 13 us (21
// MB), 16 tokens 55 us (219 MB); 32 experts of 2880 x 2880, top 4, MXFP4, one token 18.5 us
// (53 MB), 8 tokens 70. One token is bound by latency and issue as much as by bytes:
// two kernels each ask for their weights two microseconds after their start, wait two more
// for the first, and lie 1.3 apart; 16 wavefronts pay 16 clocks of a CU for every vector
// instruction they share. So nothing is grouped for one token (item q is slot q, the ids
// stay in a register) and no unit costs a division: 21.8 -> 20.1 us in a kernel trace. Not
// kept: units of 32 rows, and loops unrolled over a ring of loads with all of a workgroup's
// begun at its start: 12.2 to 17 us for the MXFP4 first kernel against 12.8 then, the second
// slower by 1 to 6 (instructions that run once come from memory).
#include <algorithm>

#include "geg_device.hpp"
#include "geg_launch.hpp"

namespace geg {

namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));

constexpr int MG = 4;   // most entries per item

// Workgroups of the second kernel. One token (k <= 64): 16 wavefronts of 4 weight rows and
// one entry each, so that every load is out as soon as possible. More: 8 wavefronts of 8
// rows and up to four entries (with twice the registers each; 16 would spill).
template <bool ONE>
struct Shape {
  static constexpr int kMT = ONE ? 1024 : 512;   // threads per workgroup
  static constexpr int kMW = kMT / 64;
  static constexpr int kRows = ONE ? 4 : 8;      // weight rows per wavefront
  static constexpr int kMost = ONE ? 1 : MG;     // entries taken at once
  static constexpr int kAhead = ONE ? 3 : 1;     // passes whose codes are in flight
};
// Of the first, whose units are 64 rows, the 32 values of a block of act. The same, but for
// one token in MXFP4 two workgroups of 8 wavefronts share a CU: a unit past one per CU then
// runs beside another instead of after it, and a unit's 8 wavefronts meet sooner than 16. Units
// of 64 rows, in workgroups of 8 against 16: 48 of 2880 values 6.3 / 7.5-8.4 us, 192 of 2048
// 5.8 / 6.1, 240 of 2880 7.6-8.8 / 9.5-9.9, 256 of 4096 9.6-10.5 / 11.6-12.0, 360 of 2880
// 10.8-11.6 / 12.6, 896 of 4096 26.4 / 28.9. NF4's table leaves no room for a second workgroup:
// with 8 wavefronts it took 8.0 us for 192 units, with 16 6.9.
template <Fmt F, bool ONE>
struct UpShape {
  static constexpr bool kTwo = ONE && F == MXFP4;
  static constexpr int kMT = ONE && !kTwo ? 1024 : 512;
  static constexpr int kMW = kMT / 64;
  static constexpr int kRows = 64 / kMW;
  static constexpr int kMost = ONE ? 1 : MG;
  static constexpr int kAhead = ONE && !kTwo ? 3 : 1;
  static constexpr int kWavesPerSimd = kTwo ? 4 : kMT / 256;
};

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

// Maximum over each half wavefront, on all its lanes.
__device__ __forceinline__ uint32_t max32(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, false));   // row_ror:8
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xF, 0xF, false));
  const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  const uint32_t x = r[0], y = r[1];
  return max(x, y);
}

// Largest |x| of 8 bf16 values, as its bits.
__device__ __forceinline__ uint32_t max_abs8(const u32x4& x) {
  u16x2 m = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = x[i] & 0x7FFF7FFFu;
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w));
  }
  const uint16_t lo = m[0], hi = m[1];
  return max((uint32_t)lo, (uint32_t)hi);
}

// The exponent ex for which bf16 magnitudes of at most `mx` times 2^-ex lie below 2^15, the
// largest at 2^14 or more; 2^ex and 2^-ex are normal fp32 values. (inf and NaN stay so.)
__device__ __forceinline__ int fit_exponent(uint32_t mx) { return max((int)(mx >> 7) - 127 - 14, -126); }
__device__ __forceinline__ float pow2(int ex) { return __uint_as_float((uint32_t)(ex + 127) << 23); }
constexpr uint32_t kBf16PastF16 = 0x4780;   // 65536, the smallest bf16 magnitude past fp16's range

// 8 bf16 values times m as fp16, natural order.
__device__ __forceinline__ u32x4 bf16x8_times_to_f16(const u32x4& x, float m) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f16x2 h;
    h[0] = (_Float16)(__uint_as_float(x[i] << 16) * m);
    h[1] = (_Float16)(__uint_as_float(x[i] & 0xFFFF0000u) * m);
    r[i] = __builtin_bit_cast(uint32_t, h);
  }
  return r;
}

// Grouping of the T k entries by expert, in LDS. An entry's place is the number of
// entries with a smaller expert, or the same and a smaller index; dropped entries (an id
// outside [0, E)) get none. An item is a run of at most MOST places of one expert.
struct Groups {
  int32_t key[kMoeMaxEntries];         // of each entry: expert * 256 + index; dropped: the largest
  int32_t id[kMoeMaxEntries + MG];     // at each place: its expert (-1 past the last), its
  int32_t ent[kMoeMaxEntries];         // entry and token
  int32_t tok[kMoeMaxEntries];
  int32_t expert[kMoeMaxEntries];      // of each item: expert, first place, entries
  int32_t first[kMoeMaxEntries];
  int32_t size[kMoeMaxEntries];
  int32_t items;
};

// Every thread of the workgroup calls it (barriers inside). `err` (may be NULL)
// receives the flag of a dropped entry. `mine` is entry threadIdx.x's id.
template <int MT, int MOST>
__device__ __forceinline__ void group_entries(Groups& g, int mine, int n, int k, int E, uint32_t* err) {
  constexpr int TPE = MT / kMoeMaxEntries;   // lanes per entry, each counting a share of the others
  static_assert(TPE == 4 || TPE == 2, "two or four lanes per entry");
  static_assert(kMaxExperts * kMoeMaxEntries < INT32_MAX, "keys fit");
  const int t = threadIdx.x;
  if (t < kMoeMaxEntries) {
    const bool ok = t < n && mine >= 0 && mine < E;
    if (t < n && !ok && err) atomicOr(err, kErrBadExpertId);
    g.key[t] = ok ? mine * kMoeMaxEntries + t : INT32_MAX;
  }
  if (t < kMoeMaxEntries + MG) g.id[t] = -1;
  lds_barrier();
  const int f = t / TPE, key = g.key[f];
  int place = 0;
  for (int f0 = 4 * (t % TPE); f0 < n; f0 += 4 * TPE) {
    const i32x4 v = *reinterpret_cast<const i32x4*>(g.key + f0);
#pragma unroll
    for (int j = 0; j < 4; ++j) place += v[j] < key;
  }
  place += __builtin_amdgcn_update_dpp(0, place, 0xB1, 0xF, 0xF, false);                  // lane ^ 1
  if (TPE == 4) place += __builtin_amdgcn_update_dpp(0, place, 0x4E, 0xF, 0xF, false);   // lane ^ 2
  if (t % TPE == 0 && key != INT32_MAX) {
    g.id[place] = key / kMoeMaxEntries;
    g.ent[place] = f;
    g.tok[place] = f / k;
  }
  lds_barrier();
  if (t < 64) {
    // items of three and four entries first: the work that is left for a last, partial
    // round is then the cheap one
    int items = 0;
    for (int big = 1; big >= 0; --big) {
      int run = 0;   // first place of the run that reaches into the window of 64 places
      for (int base = 0; base < n; base += 64) {
        const int p = base + t, e = g.id[p];
        const uint64_t starts = __ballot(e >= 0 && (p == 0 || g.id[p - 1] != e));
        const uint64_t upto = starts & (~0ull >> (63 - t));
        const int start = upto ? base + 63 - __builtin_clzll(upto) : run;
        int cnt = 1;
#pragma unroll
        for (int j = 1; j < MOST; ++j) cnt += g.id[p + j] == e;
        const bool lead = e >= 0 && (p - start) % MOST == 0 && (cnt > 2) == (big != 0);
        const uint64_t leads = __ballot(lead);
        if (lead) {
          const int to = items + __builtin_popcountll(leads & ((1ull << t) - 1));
          g.expert[to] = e;
          g.first[to] = p;
          g.size[to] = cnt;
        }
        items += __builtin_popcountll(leads);
        if (starts) run = base + 63 - __builtin_clzll(starts);
      }
    }
    if (t == 0) g.items = items;
  }
  lds_barrier();
}

// Sums of per-lane values d[u][m] over the LPR lanes of their rows: put(row, m, sum) on
// one lane for each of the unit's rows and entries.
template <int LPR, int U, int RV, typename Put>
__device__ __forceinline__ void sum_lanes(const float (&d)[U][RV], int lane, Put put) {
  constexpr int G = 64 / LPR;
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
#pragma unroll
    for (int u = 0; u < U / F; ++u)
#pragma unroll
      for (int m = 0; m < RV; ++m) put(u * F * G + row, m, v[u][m]);
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
  __device__ __forceinline__ float scale_f32(int u) const {
    return F == NF4 ? __uint_as_float(scale[u]) : e8m0_to_f32(scale[u]);
  }
};

// tot[u][m] += scale[u] xscale[m] (dot product of row group u's chunk with entry m's 32
// values), for the four quarters j of the chunk in turn: a quarter's values of all row
// groups are decoded once for all entries. x(j, m): entry m's 8 values of quarter j as
// fp16 (FT = NF4) or bf16 (MXFP4) pairs. Lanes past the row (`on` false) hold zero codes and
// another chunk's values, and add nothing: 0 times an infinity there would be NaN.
template <Fmt F, int FT, int LPR, int U, int RV, typename X>
__device__ __forceinline__ void dot_pass(const Codes<F, LPR, U>& w, X x, const float* xscale, bool on,
                                         const uint32_t* blut, uint32_t lane_off, float (&tot)[U][RV]) {
  constexpr std::integral_constant<int, FT> ft{};
  float d[U][RV];
  u32x4 xv[2][RV];   // the next quarter's values are fetched ahead
#pragma unroll
  for (int m = 0; m < RV; ++m) xv[0][m] = x(0, m);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    u32x4 v[U];
    if (j < 3) {
#pragma unroll
      for (int m = 0; m < RV; ++m) xv[(j + 1) & 1][m] = x(j + 1, m);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {   // values k = 8j .. 8j+7, natural order
      if constexpr (F == NF4)
        v[u] = nf4_byte_lut_decode8(blut, w.code[u][j], lane_off);
      else if constexpr (FT == NF4)
        v[u] = mxfp4_decode8_f16(w.code[u][j]);
      else
        v[u] = mxfp4_decode8(w.code[u][j], 1.0f);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < RV; ++m) {
        if (j == 0) d[u][m] = 0.f;
#pragma unroll
        for (int p = 0; p < 4; ++p) d[u][m] = fdot2(v[u][p], xv[j & 1][m][p], d[u][m], ft);
        // finished here, not where it is used: with a quarter's values live at a time
        // nothing spills
        asm volatile("" : "+v"(d[u][m]));
      }
    __builtin_amdgcn_sched_barrier(0);
  }
  if (!on) return;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float s = w.scale_f32(u);
#pragma unroll
    for (int m = 0; m < RV; ++m) tot[u][m] += d[u][m] * (xscale ? s * xscale[m] : s);
  }
}

// f(RV) with the entries taken at once for an item of cnt: 1, 2 or 4.
template <int MOST, typename Fn>
__device__ __forceinline__ void by_entries(int cnt, Fn f) {
  if constexpr (MOST == 1) {
    f(std::integral_constant<int, 1>{});
  } else {
    if (cnt == 1)
      f(std::integral_constant<int, 1>{});
    else if (cnt == 2)
      f(std::integral_constant<int, 2>{});
    else
      f(std::integral_constant<int, 4>{});
  }
}

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
template <Fmt F, bool ONE>
constexpr int x_lds_bytes() { return F == NF4 || ONE ? 64 << 10 : 140 << 10; }

// First kernel. Units (item, 64 rows of its gate/up weight = 32 values of act) over a grid
// of one or two workgroups per CU; a wavefront's codes of the next pass are in flight
// while it works on this one. x is staged in LDS when all tokens fit (XL), else each lane loads
// its slice from memory. For NF4 every workgroup finds the tokens' largest magnitudes before it
// scales them: from the registers they pass through on their way into LDS (0.4 us for one
// token, nothing at 16 of 2048, where a second pass over LDS cost 3.7), or in a pass of its
// own over tokens that are not staged (1.9 us for 16 of 4096). Workgroup 0 flags what plain
// fp16 could not hold. The sums meet in LDS, where a half wavefront per entry forms the 32 act
// values, their scale and their fp16 form (value i = 32 c + 8 j + b of a row at
// ((j (I / 32) + c) 8 + b): the order in which the second kernel's lanes read it). Workgroup 0
// also writes the grouping.
template <Fmt F, int LPR, bool XL, bool ONE>
__global__ __launch_bounds__((UpShape<F, ONE>::kMT), (UpShape<F, ONE>::kWavesPerSimd)) void moe_up_kernel(MoeArgs g) {
  using Form = UpShape<F, ONE>;
  constexpr int MT = Form::kMT, MW = Form::kMW, ROWS = Form::kRows, MOST = Form::kMost, AHEAD = Form::kAhead;
  constexpr int G = 64 / LPR, U = ROWS / G;
  // the byte table first: at LDS address 0 a code byte's address needs no base added
  __shared__ struct __attribute__((aligned(16))) {
    uint32_t blut[F == NF4 ? kNf4ByteLutWords : 4];
    uint8_t xs[XL ? x_lds_bytes<F, ONE>() : 16];
    Groups grp;
    float accs[2][MW][MOST * ROWS];
    uint32_t xmax[F == NF4 ? kMoeMaxTokens : 4];   // NF4: the tokens' largest |x|, as bf16 bits
  } lds;
  uint32_t* const blut = lds.blut;
  uint8_t* const xs = lds.xs;
  Groups& grp = lds.grp;
  const int n = g.T * g.k;
  const int64_t H = g.H, N = 2 * g.I;
  const int C = (int)(H >> 5), CI = (int)(g.I >> 5);
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  if constexpr (F == NF4) {
    if (t < kMoeMaxTokens) lds.xmax[t] = 0;
    if constexpr (ONE) lds_barrier();   // else the grouping's barriers come before its first use
  }
  // The tokens' loads go out before the weights' (loads complete in order): the first XP
  // pieces of 8 values per thread wait in registers (NF4: all), more are stored right away.
  constexpr int XP = F == NF4 ? x_lds_bytes<F, ONE>() / (16 * MT) : 4;
  static_assert(F != NF4 || XP * 16 * MT == x_lds_bytes<F, ONE>(), "every staged piece of an NF4 call has a register");
  const int pieces = g.T * 4 * C;
  u32x4 xp[XP];
  auto put_x = [&](int p, u32x4 v) {
    if (p < pieces) {
      const int tok = ONE ? 0 : p / (4 * C), q = ONE ? p : p % (4 * C);   // piece q of the token: chunk q / 4, piece q % 4
      *reinterpret_cast<u32x4*>(xs + ((4 * tok + (q & 3)) * C + (q >> 2)) * 16) = v;
    }
  };
  // one token: every wavefront holds the k <= 64 ids
  const int my_id = ONE ? g.ids[min(lane, n - 1)] : (t < n ? g.ids[t] : 0);
  if constexpr (XL) {
#pragma unroll
    for (int i = 0; i < XP; ++i)
      if (t + i * MT < pieces) xp[i] = reinterpret_cast<const u32x4*>(g.x)[t + i * MT];
    if constexpr (F != NF4)
      for (int p = t + XP * MT; p < pieces; p += MT) put_x(p, reinterpret_cast<const u32x4*>(g.x)[p]);
  }
  int items = n;
  if constexpr (ONE) {   // item q is slot q
    if (blockIdx.x == 0 && t < n && (my_id < 0 || my_id >= g.E)) atomicOr(g.err, kErrBadExpertId);
  } else {
    group_entries<MT, MOST>(grp, my_id, n, g.k, g.E, blockIdx.x == 0 ? g.err : nullptr);
    items = grp.items;
    if (blockIdx.x == 0 && t < kMoeMaxEntries) {
      if (t == 0) g.plan[0] = items;
      if (t < items) {
        g.plan[4 + 2 * t] = grp.expert[t];
        g.plan[4 + 2 * t + 1] = grp.first[t] | (grp.size[t] << 16);
      }
      if (t < n) g.plan[4 + 2 * kMoeMaxEntries + t] = grp.ent[t];
    }
  }
  const int gl = lane / LPR, li = lane % LPR;
  const uint32_t lane_off = nf4_byte_lut_lane(lane);
  const __amdgpu_buffer_rsrc_t X = mrsrc(g.x, (int64_t)g.T * H * 2);
  // The passes of this workgroup's units in turn, AHEAD of them with their codes in flight.
  Codes<F, LPR, U> pre[AHEAD];
  // Units are stepped through as (item, block of act): every division less counts, as 16
  // wavefronts make each
  struct Unit {
    int q, c;
  };
  const Unit stride{(int)gridDim.x / CI, (int)gridDim.x % CI};
  auto advance = [&](Unit& u) {
    u.q += stride.q;
    u.c += stride.c;
    if (u.c >= CI) {
      u.c -= CI;
      ++u.q;
    }
  };
  Unit at{(int)blockIdx.x / CI, (int)blockIdx.x % CI};
  Unit l = at;   // the next pass to load
  int l_c0 = 0;
  auto load_next = [&](Codes<F, LPR, U>& w) {
    if (l.q >= items) return;
    const int e = ONE ? __builtin_amdgcn_readlane(my_id, l.q) : __builtin_amdgcn_readfirstlane(grp.expert[l.q]);
    const bool ok = !ONE || (e >= 0 && e < g.E);   // else zeros, without an access
    const __amdgpu_buffer_rsrc_t W = mrsrc(g.w13 + (int64_t)e * N * (H >> 1), ok ? N * (H >> 1) : 0);
    const __amdgpu_buffer_rsrc_t S = mrsrc(expert_scales<F>(g.s13, e, N, H), ok ? scale_bytes<F>(N, H) : 0);
    const int c = l_c0 + li;
    // chunks past the row read as zero: their offsets lie past every buffer
    w.load(W, S, (int64_t)l.c * 64 + ROWS * wave, gl, H, c, c < C ? 0u : 0xFFFFFFF0u);
    if ((l_c0 += LPR) >= C) {
      l_c0 = 0;
      advance(l);
    }
  };
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) load_next(pre[i]);
  // the table and the tokens while the first weights are on their way
  if constexpr (F == NF4) nf4_byte_lut_fill<64, MT>(blut);
  if constexpr (XL && F == NF4) {
    // token and place of each piece; H % 64 == 0, so eight adjacent lanes hold pieces of one token
    int tok[XP], q[XP];
    const int dt = ONE ? 0 : MT / (4 * C), dq = MT - dt * 4 * C;
    tok[0] = ONE ? 0 : t / (4 * C), q[0] = t - tok[0] * 4 * C;
#pragma unroll
    for (int i = 1; i < XP; ++i) {
      const bool over = !ONE && q[i - 1] + dq >= 4 * C;
      tok[i] = tok[i - 1] + dt + over;
      q[i] = q[i - 1] + dq - (over ? 4 * C : 0);
    }
#pragma unroll
    for (int i = 0; i < XP; ++i)
      if (t + i * MT < pieces) {
        uint32_t mx = max_abs8(xp[i]);
        mx = max(mx, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)mx, 0xB1, 0xF, 0xF, false));    // lane ^ 1
        mx = max(mx, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)mx, 0x4E, 0xF, 0xF, false));    // lane ^ 2
        mx = max(mx, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)mx, 0x141, 0xF, 0xF, false));   // 7 - lane
        if ((lane & 7) == 0) atomicMax(&lds.xmax[tok[i]], mx);   // a maximum: the same in any order
      }
    lds_barrier();
#pragma unroll
    for (int i = 0; i < XP; ++i)
      if (t + i * MT < pieces)
        *reinterpret_cast<u32x4*>(xs + ((4 * tok[i] + (q[i] & 3)) * C + (q[i] >> 2)) * 16) =
            bf16x8_times_to_f16(xp[i], pow2(-fit_exponent(lds.xmax[tok[i]])));
  } else if constexpr (XL) {
#pragma unroll
    for (int i = 0; i < XP; ++i) put_x(t + i * MT, xp[i]);
  } else if constexpr (F == NF4) {
    constexpr int UN = 8;   // pieces per lane in flight
    const int runs = (4 * C + 64 * UN - 1) / (64 * UN);
    for (int r = wave; r < g.T * runs; r += MW) {
      const int tok = r / runs, p0 = (r - tok * runs) * 64 * UN + lane;
      u32x4 v[UN];
#pragma unroll
      for (int i = 0; i < UN; ++i) {
        v[i] = u32x4{0, 0, 0, 0};
        if (p0 + 64 * i < 4 * C) v[i] = reinterpret_cast<const u32x4*>(g.x)[(int64_t)tok * 4 * C + p0 + 64 * i];
      }
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < UN; ++i) mx = max(mx, max_abs8(v[i]));
      mx = max32(mx);
      if ((lane & 31) == 0) atomicMax(&lds.xmax[tok], mx);
    }
  }
  lds_barrier();
  if constexpr (F == NF4) {
    if (blockIdx.x == 0 && t < g.T && lds.xmax[t] >= kBf16PastF16) atomicOr(g.err, kErrFp16Range);
  }
  int seq = 0;
  for (; at.q < items; advance(at), ++seq) {
    const int first = ONE ? at.q : __builtin_amdgcn_readfirstlane(grp.first[at.q]);
    const int cnt = ONE ? 1 : __builtin_amdgcn_readfirstlane(grp.size[at.q]);
    float(*acc)[MOST * ROWS] = lds.accs[seq & 1];
    // two wavefronts, others from unit to unit, form the block of act: 32 lanes per entry
    const int m = ((wave - 2 * seq) & (MW - 1)) * 2 + (lane >> 5), i = lane & 31;
    float back = 1.f;
    if constexpr (F == NF4) back = pow2(fit_exponent(lds.xmax[ONE ? 0 : grp.tok[min(first + m, n - 1)]]));
    by_entries<MOST>(cnt, [&](auto rv) {
      constexpr int RV = decltype(rv)::value;
      int tok[RV];
#pragma unroll
      for (int m = 0; m < RV; ++m) tok[m] = ONE ? 0 : __builtin_amdgcn_readfirstlane(grp.tok[first + min(m, cnt - 1)]);
      float fit[RV];   // of a token's values that were not staged
#pragma unroll
      for (int m = 0; m < RV; ++m)
        fit[m] = F == NF4 && !XL ? pow2(-fit_exponent(__builtin_amdgcn_readfirstlane(lds.xmax[tok[m]]))) : 1.f;
      float tot[U][RV];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int m = 0; m < RV; ++m) tot[u][m] = 0.f;
      for (int c0 = 0; c0 < C; c0 += LPR) {
        const int c = c0 + li, cc = min(c, C - 1);
        const uint32_t off_mask = c < C ? 0u : 0xFFFFFFF0u;
        const Codes<F, LPR, U> w = pre[0];
#pragma unroll
        for (int i = 0; i + 1 < AHEAD; ++i) pre[i] = pre[i + 1];
        load_next(pre[AHEAD - 1]);
        dot_pass<F, F>(
            w,
            [&](int j, int m) -> u32x4 {
              if constexpr (XL) {
                return *reinterpret_cast<const u32x4*>(xs + ((4 * tok[m] + j) * C + cc) * 16);
              } else {
                u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(
                    X, (uint32_t)(((int64_t)tok[m] * H + 32 * c) * 2 + 16 * j) | off_mask, 0, 0);
                if constexpr (F == NF4) v = bf16x8_times_to_f16(v, fit[m]);
                return v;
              }
            },
            nullptr, c < C, blut, lane_off, tot);
      }
      sum_lanes<LPR, U, RV>(tot, lane, [&](int row, int m, float v) { acc[wave][m * ROWS + row] = v; });
    });
    lds_barrier();   // the sums of this unit; the other parity's are free again after the next one
    if (m < cnt) {
      const float* a = acc[2 * i / ROWS] + m * ROWS + 2 * i % ROWS;
      const float v = F == NF4 ? swiglu(a[0] * back, a[1] * back) : swiglu(a[0], a[1]);
      const uint32_t mx = max32(__float_as_uint(v) & 0x7FFFFFFFu);
      // the block's largest to [2^14, 2^15); 2^ex stays a normal fp32 value
      const int ex = max((int)(mx >> 23) - 127 - 14, -126);
      const int64_t slot = ONE ? at.q : grp.ent[first + m];
      const int c = at.c;
      const _Float16 h = (_Float16)__builtin_ldexpf(v, -ex);
      g.act[slot * g.I + ((i >> 3) * CI + c) * 8 + (i & 7)] = __builtin_bit_cast(uint16_t, h);
      if (i == 0) g.act_scale[slot * CI + c] = __uint_as_float((uint32_t)(ex + 127) << 23);
    }
  }
}

// Second kernel. A workgroup owns RB rows of W2 (columns of out), RB / ROWS subgroups; its
// wavefronts share the (item, subgroup) pieces of work, the codes of the next piece in
// flight while one is worked on, each adding its weighted sums into an own [RB][T] array
// in LDS; the arrays are added in wavefront order, so results do not depend on timing.
template <Fmt F, int LPR, bool ONE>
__global__ __launch_bounds__(Shape<ONE>::kMT) void moe_down_kernel(MoeArgs g) {
  constexpr int MT = Shape<ONE>::kMT, MW = Shape<ONE>::kMW, ROWS = Shape<ONE>::kRows, MOST = Shape<ONE>::kMost;
  constexpr int AHEAD = Shape<ONE>::kAhead;
  constexpr int G = 64 / LPR, U = ROWS / G;
  __shared__ struct __attribute__((aligned(16))) {
    uint32_t blut[F == NF4 ? kNf4ByteLutWords : 4];    // at LDS address 0
    float outs[MW][kMoeRowBlock * kMoeMaxTokens];      // [wavefront][row][token]
    int32_t item[2 * kMoeMaxEntries];                  // expert; first place | entries << 16
    int32_t ent[kMoeMaxEntries], tok[kMoeMaxEntries];  // at each place
    float weight[kMoeMaxEntries];
  } lds;
  uint32_t* const blut = lds.blut;
  const int64_t H = g.H, K = g.I;
  const int C = (int)(K >> 5), T = g.T, n = T * g.k;
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int gl = lane / LPR, li = lane % LPR;
  const uint32_t lane_off = nf4_byte_lut_lane(lane);
  const int RB = g.rb, subs = RB / ROWS;
  int items = n, my_id = 0;
  float my_weight = 0.f;
  uint64_t valid = 0;
  if constexpr (ONE) {   // item q is slot q; every wavefront holds the k <= 64 ids and weights
    my_id = g.ids[min(lane, n - 1)];
    my_weight = g.weights[min(lane, n - 1)];
    valid = __builtin_amdgcn_ballot_w64(my_id >= 0 && my_id < g.E);
  } else {
    items = g.plan[0];
    for (int i = t; i < 2 * n; i += MT) lds.item[i] = g.plan[4 + i];
    if (t < n) {
      // places past the last hold nothing: any entry will do
      const int f = min((uint32_t)g.plan[4 + 2 * kMoeMaxEntries + t], (uint32_t)(n - 1));
      lds.ent[t] = f;
      lds.tok[t] = f / g.k;
      lds.weight[t] = g.weights[f];
    }
    lds_barrier();
  }
  const int64_t blocks = (H + RB - 1) / RB;
  const int works = items * subs;
  // the passes of this wavefront's pieces of work, block by block
  Codes<F, LPR, U> pre[AHEAD];
  struct Work {
    int q, sub;   // item, ROWS rows of the block
  };
  const Work stride{MW / subs, MW % subs}, w0{wave / subs, wave % subs};
  auto advance = [&](Work& w) {
    w.q += stride.q;
    w.sub += stride.sub;
    if (w.sub >= subs) {
      w.sub -= subs;
      ++w.q;
    }
  };
  int64_t l_b = blockIdx.x;
  Work l = w0;
  int l_c0 = 0;
  auto load_next = [&](Codes<F, LPR, U>& w) {
    if (l_b >= blocks || wave >= works) return;
    const int e = ONE ? __builtin_amdgcn_readlane(my_id, l.q) : __builtin_amdgcn_readfirstlane(lds.item[2 * l.q]);
    const bool ok = !ONE || (valid >> l.q) & 1;   // else zeros, without an access
    const __amdgpu_buffer_rsrc_t W = mrsrc(g.w2 + (int64_t)e * H * (K >> 1), ok ? H * (K >> 1) : 0);
    const __amdgpu_buffer_rsrc_t S = mrsrc(expert_scales<F>(g.s2, e, H, K), ok ? scale_bytes<F>(H, K) : 0);
    const int c = l_c0 + li;
    w.load(W, S, l_b * RB + l.sub * ROWS, gl, K, c, c < C ? 0u : 0xFFFFFFF0u);
    if ((l_c0 += LPR) >= C) {
      l_c0 = 0;
      advance(l);
      if (l.q >= items) {
        l = w0;
        l_b += gridDim.x;
      }
    }
  };
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) load_next(pre[i]);
  for (int i = lane; i < RB * T; i += 64) lds.outs[wave][i] = 0.f;
  if constexpr (F == NF4) nf4_byte_lut_fill<64, MT>(blut);
  lds_barrier();
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
    for (Work wk = w0; wk.q < items; advance(wk)) {
      const int sub = wk.sub;
      const int fc = ONE ? 0 : __builtin_amdgcn_readfirstlane(lds.item[2 * wk.q + 1]);
      const int first = ONE ? wk.q : fc & 0xFFFF, cnt = ONE ? (int)((valid >> wk.q) & 1) : fc >> 16;
      by_entries<MOST>(cnt, [&](auto rv) {
        constexpr int RV = decltype(rv)::value;
        float tot[U][RV];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int m = 0; m < RV; ++m) tot[u][m] = 0.f;
        for (int c0 = 0; c0 < C; c0 += LPR) {
          const int c = c0 + li, cc = min(c, C - 1);
          const Codes<F, LPR, U> w = pre[0];
          const u32x4* a[RV];
          float xs[RV];
#pragma unroll
          for (int m = 0; m < RV; ++m) {
            const int64_t f = ONE ? first : __builtin_amdgcn_readfirstlane(lds.ent[first + min(m, cnt - 1)]);
            a[m] = reinterpret_cast<const u32x4*>(g.act + f * K);
            xs[m] = g.act_scale[f * C + cc];
          }
#pragma unroll
          for (int i = 0; i + 1 < AHEAD; ++i) pre[i] = pre[i + 1];
          load_next(pre[AHEAD - 1]);
          dot_pass<F, NF4>(w, [&](int j, int m) -> u32x4 { return a[m][j * C + cc]; }, xs, c < C, blut, lane_off,
                           tot);
        }
        sum_lanes<LPR, U, RV>(tot, lane, [&](int row, int m, float v) {
          if constexpr (ONE) {
            const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(my_weight), first));
            if (cnt) lds.outs[wave][sub * ROWS + row] += w * v;
          } else if (m < cnt) {
            lds.outs[wave][(sub * ROWS + row) * T + lds.tok[first + m]] += lds.weight[first + m] * v;
          }
        });
      });
    }
    lds_barrier();
    for (int i = t; i < RB * T; i += MT) {
      float o[MW], v = 0.f;
#pragma unroll
      for (int w = 0; w < MW; ++w) o[w] = lds.outs[w][i];
#pragma unroll
      for (int w = 0; w < MW; ++w) {
        v += o[w];
        lds.outs[w][i] = 0.f;
      }
      const int64_t col = b * RB + i / T;
      if (col < H) g.out[(int64_t)(i % T) * H + col] = to_bf16(v);
    }
    lds_barrier();
  }
}

template <Fmt F, int LPR, bool ONE>
hipError_t up(const MoeArgs& g, int cus, hipStream_t s) {
  const dim3 grid((unsigned)(UpShape<F, ONE>::kTwo ? 2 * cus : cus)), block(UpShape<F, ONE>::kMT);
  if ((int64_t)g.T * g.H * 2 <= x_lds_bytes<F, ONE>())
    hipLaunchKernelGGL((moe_up_kernel<F, LPR, true, ONE>), grid, block, 0, s, g);
  else
    hipLaunchKernelGGL((moe_up_kernel<F, LPR, false, ONE>), grid, block, 0, s, g);
  return hipGetLastError();
}

// Rows of W2 per workgroup: no more than one round of the chip where that stays within the
// LDS arrays. (Fewer than ROWS rows per CU leave CUs idle: neither the items nor the
// contraction are split.)
template <Fmt F, int LPR, bool ONE>
hipError_t down(MoeArgs g, int cus, hipStream_t s) {
  constexpr int ROWS = Shape<ONE>::kRows;
  const int64_t rb = ((g.H + cus - 1) / cus + ROWS - 1) / ROWS * ROWS;
  g.rb = (int)std::min<int64_t>(rb, kMoeRowBlock);
  const int64_t blocks = (g.H + g.rb - 1) / g.rb;
  hipLaunchKernelGGL((moe_down_kernel<F, LPR, ONE>), dim3((unsigned)std::min<int64_t>(blocks, cus)),
                     dim3(Shape<ONE>::kMT), 0, s, g);
  return hipGetLastError();
}

// f(LPR) with the lanes per weight row for a contraction of K (C chunks): the number up to
// MOST that leaves the fewest lanes idle over the row's passes, the larger on a tie (90
// chunks: three passes of 32 lanes; two of 64 would idle 38 of 128).
template <int MOST, typename Fn>
hipError_t by_lanes(int64_t K, Fn f) {
  const int64_t C = K >> 5;
  auto lanes = [&](int64_t l) { return (C + l - 1) / l * l; };
  if constexpr (MOST >= 64)
    if (lanes(64) <= lanes(32) && lanes(64) <= lanes(16)) return f(std::integral_constant<int, 64>{});
  if (lanes(32) <= lanes(16)) return f(std::integral_constant<int, 32>{});
  return f(std::integral_constant<int, 16>{});
}

template <Fmt F, bool ONE>
hipError_t layer(const MoeArgs& g, int cus, hipStream_t s) {
  const hipError_t e = by_lanes<UpShape<F, ONE>::kTwo ? 32 : 64>(g.H, [&](auto l) { return up<F, decltype(l)::value, ONE>(g, cus, s); });
  if (e != hipSuccess) return e;
  return by_lanes<64>(g.I, [&](auto l) { return down<F, decltype(l)::value, ONE>(g, cus, s); });
}

}  // namespace

hipError_t launch_moe_layer(int fmt, const MoeArgs& g, int cus, hipStream_t s) {
  if (g.T == 1 && g.k <= 64) return fmt == NF4 ? layer<NF4, true>(g, cus, s) : layer<MXFP4, true>(g, cus, s);
  return fmt == NF4 ? layer<NF4, false>(g, cus, s) : layer<MXFP4, false>(g, cus, s);
}

}  // namespace geg
