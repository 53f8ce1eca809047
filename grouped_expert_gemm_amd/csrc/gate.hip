// The router's gate and the gradients of the gate and of the weighted combine.
//
// Forward, per token t with logits l over E experts: the k largest logits, ties to
// the lower expert, and their softmax weights
//     w_s = exp(l_s - m) / sum_j exp(l_j - m),  m = max l,
// the sum over all experts, or (renormalised) over the chosen k. A NaN logit counts
// as -inf (and is flagged); a token whose logits are all -inf gets weights 0; +inf
// logits share the weight equally.
//
// Backward, from dw: with S = sum_s w_s dw_s, dl of a chosen expert is
// w_s (dw_s - S); without renormalisation the softmax runs over all experts and
// every other expert gets -p_i S. The combine out_t = sum_s w_ts y[row(t, s)] gives
// dy[row(t, s)] = w_ts dout_t and dw_ts = <dout_t, y[row(t, s)]>.
//
// One wavefront per token: lane l holds the logits l + 64 j, so E <= 1024 takes at
// most 16 registers. Each of the k rounds is a DPP maximum over order-preserving
// integer keys and a ballot for the lowest index that attains it: no shuffles, no
// LDS, no sort. The combine's gradient is one wavefront per (token, slot), bound by
// reading y once and writing dy once.
//
// 4096 tokens, 128 experts, k 8: the gate 4.4 us, its gradient 5.0; with rows of 2048 the
// combine's gradient 49.6 us for 285 MB (5.7 TB/s). 64 tokens: the gate 3.7 us, of which
// the launch is 2.
#include <algorithm>

#include "geg_device.hpp"
#include "geg_launch.hpp"

namespace geg {

namespace {

// Order-preserving integer key of a float: larger float, larger key; 0 is below
// every key of a number (the key of -inf is 0x007FFFFF).
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xFFFFFFFFu));
}

// Maximum over the 64 lanes, on every lane: row shifts by 1, 2, 4, 8 and row
// broadcasts bring it to lane 63.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Sum over the 64 lanes, on every lane (a fixed tree).
__device__ __forceinline__ float wave_sum(float v) {
  auto add = [](float x, int y) { return x + __builtin_bit_cast(float, y); };
  v = add(v, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x111, 0xF, 0xF, false));
  v = add(v, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x112, 0xF, 0xF, false));
  v = add(v, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x114, 0xF, 0xF, false));
  v = add(v, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x118, 0xF, 0xF, false));
  v = add(v, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x142, 0xA, 0xF, false));
  v = add(v, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x143, 0xC, 0xF, false));
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

template <int DT>
__device__ __forceinline__ float load_as_f32(const void* p, int64_t i) {
  if constexpr (DT == kF32)
    return reinterpret_cast<const float*>(p)[i];
  else if constexpr (DT == kBF16)
    return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << 16);
  else
    return (float)reinterpret_cast<const _Float16*>(p)[i];
}

template <int DT>
__device__ __forceinline__ void store_from_f32(void* p, int64_t i, float v) {
  if constexpr (DT == kF32)
    reinterpret_cast<float*>(p)[i] = v;
  else if constexpr (DT == kBF16)
    reinterpret_cast<uint16_t*>(p)[i] = to_bf16(v);
  else
    reinterpret_cast<_Float16*>(p)[i] = (_Float16)v;
}

// A token's logits in registers (lane l: experts l + 64 j; -inf past E), their
// maximum and, with SUM, sum of exp(l - m).
constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ float exp_from_max(float l, float m) {
  return m == kNegInf ? 0.f : (l == m ? 1.f : expf(l - m));
}

template <int DT, int V>
__device__ __forceinline__ bool load_logits(const void* logits, int64_t t, int E, int lane, float* l) {
  bool nan = false;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = lane + 64 * j;
    l[j] = kNegInf;
    if (e < E) {
      const float v = load_as_f32<DT>(logits, t * E + e);
      if (v != v)
        nan = true;
      else
        l[j] = v;
    }
  }
  return nan;
}

template <int DT, int V>
__global__ __launch_bounds__(kThreads) void topk_kernel(const void* __restrict__ logits, int64_t T, int E, int k,
                                                        int renorm, float* __restrict__ weights,
                                                        int32_t* __restrict__ ids, uint32_t* err) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (t >= T) return;
  float l[V];
  const bool nan = load_logits<DT, V>(logits, t, E, lane, l);
  if (err && __ballot(nan) && lane == 0) atomicOr(err, kErrNonFinite);
  uint32_t key[V];
#pragma unroll
  for (int j = 0; j < V; ++j) key[j] = lane + 64 * j < E ? key_of(l[j] == 0.f ? 0.f : l[j]) : 0u;
  float m = 0.f, mine = 0.f;   // the maximum; lane s keeps the s-th choice
  int my_id = 0;
  for (int s = 0; s < k; ++s) {
    uint32_t best = key[0];
#pragma unroll
    for (int j = 1; j < V; ++j) best = max(best, key[j]);
    const uint32_t top = wave_max(best);
    int id = 0;
    bool found = false;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint64_t at = __ballot(key[j] == top);
      if (!found && at) {
        found = true;
        const int who = __builtin_ctzll(at);
        id = 64 * j + who;
        if (lane == who) key[j] = 0u;
      }
    }
    const float v = value_of(top);
    if (s == 0) m = v;
    if (lane == s) {
      mine = v;
      my_id = id;
    }
  }
  float e = lane < k ? exp_from_max(mine, m) : 0.f;
  float sum;
  if (renorm) {
    sum = wave_sum(e);
  } else {
    float part = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) part += exp_from_max(l[j], m);
    sum = wave_sum(part);
  }
  if (lane < k) {
    weights[t * k + lane] = sum > 0.f ? e / sum : 0.f;
    ids[t * k + lane] = my_id;
  }
}

template <int DT, int V>
__global__ __launch_bounds__(kThreads) void topk_grad_kernel(const float* __restrict__ dw,
                                                             const void* __restrict__ logits,
                                                             const int32_t* __restrict__ ids,
                                                             const float* __restrict__ weights, int64_t T, int E,
                                                             int k, int renorm, void* __restrict__ dlogits) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (t >= T) return;
  int id = -1;
  float w = 0.f, d = 0.f;
  if (lane < k) {
    id = ids[t * k + lane];
    if (id >= 0 && id < E) {
      w = weights[t * k + lane];
      d = dw[t * k + lane];
    } else {
      id = -1;
    }
  }
  const float S = wave_sum(w * d);
  float g[V];
  if (renorm) {
#pragma unroll
    for (int j = 0; j < V; ++j) g[j] = 0.f;
  } else {
    float l[V];
    load_logits<DT, V>(logits, t, E, lane, l);
    uint32_t best = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) best = max(best, key_of(l[j]));
    const float m = value_of(wave_max(best));
    float part = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      l[j] = exp_from_max(l[j], m);
      part += l[j];
    }
    const float sum = wave_sum(part);
    const float c = sum > 0.f ? -S / sum : 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) g[j] = c * l[j];
  }
  // the chosen experts' own terms, one slot after the other (an expert named twice
  // gets both)
  const float own = renorm ? w * (d - S) : w * d;
  for (int s = 0; s < k; ++s) {
    const int e = __builtin_amdgcn_readlane(id, s);
    const float v = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, own), s));
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (e == lane + 64 * j) g[j] += v;
  }
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (lane + 64 * j < E) store_from_f32<DT>(dlogits, t * E + lane + 64 * j, g[j]);
}

// One wavefront per flat entry f = t k + s: dy[row_of[f]] = bf16(w_f dout_t) and
// dw_f = sum_n dout_t[n] y[row_of[f]][n], fp32 products and a fixed order of sums.
// U 16-byte pieces of each row per lane in flight. A dropped entry gets dw 0; with
// src_of, a row that no entry lands on (src_of < 0) gets dy 0.
__global__ __launch_bounds__(kThreads) void combine_grad_kernel(const uint16_t* __restrict__ dout,
                                                                const uint16_t* __restrict__ y,
                                                                const int32_t* __restrict__ row_of,
                                                                const int32_t* __restrict__ src_of,
                                                                const float* __restrict__ w, int64_t n, int32_t k,
                                                                int64_t N, uint16_t* __restrict__ dy,
                                                                float* __restrict__ dw) {
  constexpr int U = 4;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t chunks = N >> 3;
  const int64_t f = (int64_t)blockIdx.x * (kThreads / 64) + wave;
  if (f >= n) return;
  const int32_t r = row_of[f];
  if (src_of && src_of[f] < 0)
    for (int64_t c = lane; c < chunks; c += 64) reinterpret_cast<u32x4*>(dy + f * N)[c] = u32x4{0, 0, 0, 0};
  if (r < 0 || r >= n) {
    if (dw && lane == 0) dw[f] = 0.f;
    return;
  }
  const float ws = w ? w[f] : 1.f;
  const u32x4* dp = reinterpret_cast<const u32x4*>(dout + (f / k) * N);
  const u32x4* yp = reinterpret_cast<const u32x4*>(y + (int64_t)r * N);
  u32x4* op = reinterpret_cast<u32x4*>(dy + (int64_t)r * N);
  float acc = 0.f;
  for (int64_t c0 = lane; c0 < chunks; c0 += 64 * U) {
    u32x4 d[U], v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + 64 * u < chunks) {
        d[u] = dp[c0 + 64 * u];
        if (dw) v[u] = yp[c0 + 64 * u];
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + 64 * u < chunks) {
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float d0 = __uint_as_float(d[u][i] << 16), d1 = __uint_as_float(d[u][i] & 0xFFFF0000u);
          if (dw) {
            acc += d0 * __uint_as_float(v[u][i] << 16);
            acc += d1 * __uint_as_float(v[u][i] & 0xFFFF0000u);
          }
          o[i] = pack_bf16x2(ws * d0, ws * d1);
        }
        op[c0 + 64 * u] = o;
      }
  }
  if (dw) {
    const float sum = wave_sum(acc);
    if (lane == 0) dw[f] = sum;
  }
}

template <int DT, int V>
hipError_t topk_one(const void* logits, int64_t T, int E, int k, int renorm, float* weights, int32_t* ids,
                    uint32_t* err, hipStream_t s) {
  const int64_t grid = (T + kThreads / 64 - 1) / (kThreads / 64);
  hipLaunchKernelGGL((topk_kernel<DT, V>), dim3((unsigned)grid), dim3(kThreads), 0, s, logits, T, E, k, renorm,
                     weights, ids, err);
  return hipGetLastError();
}

template <int DT, int V>
hipError_t topk_grad_one(const float* dw, const void* logits, const int32_t* ids, const float* weights, int64_t T,
                         int E, int k, int renorm, void* dlogits, hipStream_t s) {
  const int64_t grid = (T + kThreads / 64 - 1) / (kThreads / 64);
  hipLaunchKernelGGL((topk_grad_kernel<DT, V>), dim3((unsigned)grid), dim3(kThreads), 0, s, dw, logits, ids, weights,
                     T, E, k, renorm, dlogits);
  return hipGetLastError();
}

// f<DT, V>() with V the registers that hold E logits per wavefront.
template <int DT, typename Fn>
hipError_t by_width(int E, Fn f) {
  if (E <= 64) return f(std::integral_constant<int, 1>{});
  if (E <= 128) return f(std::integral_constant<int, 2>{});
  if (E <= 256) return f(std::integral_constant<int, 4>{});
  if (E <= 512) return f(std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 16>{});
}

template <typename Fn>
hipError_t by_type(int dtype, Fn f) {
  if (dtype == kBF16) return f(std::integral_constant<int, kBF16>{});
  if (dtype == kF16) return f(std::integral_constant<int, kF16>{});
  return f(std::integral_constant<int, kF32>{});
}

}  // namespace

hipError_t launch_route_topk(const void* logits, int dtype, int64_t T, int32_t E, int32_t k, int renorm,
                             float* weights, int32_t* ids, uint32_t* err, hipStream_t s) {
  return by_type(dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    return by_width<DT>(E, [&](auto v) {
      return topk_one<DT, decltype(v)::value>(logits, T, E, k, renorm, weights, ids, err, s);
    });
  });
}

hipError_t launch_route_topk_grad(const float* dw, const void* logits, int dtype, const int32_t* ids,
                                  const float* weights, int64_t T, int32_t E, int32_t k, int renorm, void* dlogits,
                                  hipStream_t s) {
  return by_type(dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    return by_width<DT>(E, [&](auto v) {
      return topk_grad_one<DT, decltype(v)::value>(dw, logits, ids, weights, T, E, k, renorm, dlogits, s);
    });
  });
}

hipError_t launch_route_combine_grad(const uint16_t* dout, const uint16_t* y, const int32_t* row_of,
                                     const int32_t* src_of, const float* w, int64_t T, int32_t k, int64_t N,
                                     uint16_t* dy, float* dw, hipStream_t s) {
  const int64_t n = T * k, grid = (n + kThreads / 64 - 1) / (kThreads / 64);
  hipLaunchKernelGGL(combine_grad_kernel, dim3((unsigned)grid), dim3(kThreads), 0, s, dout, y, row_of, src_of, w, n,
                     k, N, dy, dw);
  return hipGetLastError();
}

}  // namespace geg
