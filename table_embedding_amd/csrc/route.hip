// Router: softmax statistics and the k largest logits of each token, and the
// gradient of the chosen weights.
//
// A token's E logits lie in the registers of L lanes (a wave serves 64 / L
// tokens), V a lane in pieces of 16 bytes, the lanes' pieces side by side, so
// that loads are whole lines.  Steps across a token's lanes are register
// exchanges (DPP) up to 16 lanes.
//
// The k largest are found by k rounds of a maximum.  A logit is mapped to a
// 32-bit key with the order of the floats (-0 equal to +0, every NaN above
// +inf, 0 reserved for "not a candidate": -inf and masked rows); a round takes
// the largest key, then the lowest index that has it, and clears it.  A 16-bit
// logit's key takes 16 bits and its index the other 16, largest first, so that
// one maximum finds both.
//
// The forward reads the logits once and is bound by the rounds' comparisons
// (about five vector instructions a logit and round): 65536 tokens, 256 float32
// experts, 8 choices take 30.5 us, 67 MB read at 2.2 TB/s.  32 lanes of 8 logits
// (more exchanges) took 49.7 us; masks kept from the search to clear a key with,
// in place of comparing the index again, 32.3 us.
#include "experts_common.h"

namespace tbe {
namespace {

// Order-preserving key of a logit; 0 for -inf (never chosen).
__device__ __forceinline__ uint32_t key_of(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.f);  // -0 to +0
  if (u == 0xff800000u) return 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// e^x for x <= 0 (NaN and -inf as exp has them): 2^(x log2 e) with the
// product's rounding error carried as a factor 1 + r ln 2, so the error does
// not grow with |x|.
__device__ __forceinline__ float exp_neg(float x) {
  const float l2e = 1.44269504f, l2e_lo = 1.92596299e-8f;
  const float t = x * l2e;
  const float r = fmaf(x, l2e, -t) + x * l2e_lo;
  const float p = __builtin_amdgcn_exp2f(t);
  return x < -104.f ? 0.f : fmaf(p, r * 0.69314718f, p);
}

// The value M lanes across (M = 1, 2, 4, 8: mirrored inside blocks of 2 M whose
// halves hold one value each by then).
template <int M>
__device__ __forceinline__ uint32_t across(uint32_t v) {
  if constexpr (M == 1) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xb1, 0xf, 0xf, true);
  else if constexpr (M == 2) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4e, 0xf, 0xf, true);
  else if constexpr (M == 4) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xf, 0xf, true);
  else if constexpr (M == 8) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xf, 0xf, true);
  else return (uint32_t)__shfl_xor((int)v, M, kWave);
}
struct Max {
  static __device__ __forceinline__ uint32_t of(uint32_t a, uint32_t b) { return a > b ? a : b; }
};
struct Min {
  static __device__ __forceinline__ uint32_t of(uint32_t a, uint32_t b) { return a < b ? a : b; }
};
struct Sum {  // of floats
  static __device__ __forceinline__ uint32_t of(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
  }
};
// Over the token's L lanes, in all of them.
template <typename Op, int L, int M = 1>
__device__ __forceinline__ uint32_t lanes(uint32_t v) {
  if constexpr (M < L) return lanes<Op, L, M * 2>(Op::of(v, across<M>(v)));
  else return v;
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  return __builtin_bit_cast(float, lanes<Sum, L>(__builtin_bit_cast(uint32_t, v)));
}

// Expert of the lane's value i: pieces of C, side by side over the lanes.
template <int WD, int L>
__device__ __forceinline__ int expert_of(int lane, int i) {
  constexpr int C = kVec16<WD>;
  return (i / C) * (C * L) + lane * C + i % C;
}

// The lane's V logits of the row at element `row`; -inf beyond E.
template <int WD, int L, int V>
__device__ __forceinline__ void load_logits(const void* p, int64_t row, int lane, int E, bool vec,
                                            float* v) {
  constexpr int C = kVec16<WD>;
#pragma unroll
  for (int i = 0; i < V; i += C) {
    const int e = expert_of<WD, L>(lane, i);
    if (vec && e + C <= E) {
      load_w<WD, C>(p, row + e, v + i);
    } else {
#pragma unroll
      for (int x = 0; x < C; ++x)
        v[i + x] = e + x < E ? ld_elem<WD>(p, row + e + x) : -__builtin_inff();
    }
  }
}

template <int WD, int L, int V>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs a, bool vec) {
  constexpr int R = (kMaxChoices + L - 1) / L;  // choice j is kept by lane j % L
  constexpr bool PACKED = WD != WD_F32;
  const int lane = threadIdx.x % L;
  const int64_t t = (int64_t)blockIdx.x * (kThreads / L) + threadIdx.x / L;
  const bool live = t < a.tokens && !(a.valid && a.valid[t < a.tokens ? t : 0] == 0);
  const int E = a.experts;
  float v[V];
  if (live) load_logits<WD, L, V>(a.logits, t * a.ld, lane, E, vec, v);
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    uint32_t q = live ? key_of(v[i]) : 0u;
    if (PACKED) {
      // the low half of a 16-bit type's key holds nothing of its order but ties
      // (float16 widens by 13 zero bits: its key is taken from its own bits)
      if constexpr (WD == WD_F16) {
        const uint32_t h = __builtin_bit_cast(uint16_t, (_Float16)v[i]);
        if (q != 0u && q != 0xffffffffu)
          q = ((h & 0x7fffu) == 0u ? 0x8000u : (h & 0x8000u) ? ~h & 0xffffu : h | 0x8000u) << 16;
      }
      q = q ? (q & 0xffff0000u) | (uint32_t)(0xffff - expert_of<WD, L>(lane, i)) : 0u;
    }
    key[i] = q;
  }
  float x_mine[R];
  uint32_t id_mine[R];
  float top = 0.f;
#pragma unroll
  for (int jb = 0; jb < R; ++jb) {
    x_mine[jb] = -__builtin_inff();
    id_mine[jb] = 0xffffffffu;
#pragma unroll 1
    for (int jj = 0; jj < L; ++jj) {
      const int j = jb * L + jj;
      if (j >= a.k) break;
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) m = m > key[i] ? m : key[i];
      const uint32_t best = lanes<Max, L>(m);
      uint32_t id;
      float x;
      if constexpr (PACKED) {
        id = best ? 0xffffu - (best & 0xffffu) : 0xffffffffu;
        const uint32_t u = best >> 16, h = (u & 0x8000u) ? u & 0x7fffu : ~u & 0xffffu;
        x = WD == WD_F16 ? f16_bits_to_float(h) : bf16_bits_to_float(h);
        if (u == 0xffffu) x = __builtin_nanf("");
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = key[i] == best ? 0u : key[i];
      } else {
        uint32_t at = 0xffffffffu;
#pragma unroll
        for (int i = V - 1; i >= 0; --i)
          at = key[i] == best ? (uint32_t)expert_of<WD, L>(lane, i) : at;
        id = best ? lanes<Min, L>(at) : 0xffffffffu;
#pragma unroll
        for (int i = 0; i < V; ++i)
          key[i] = id == (uint32_t)expert_of<WD, L>(lane, i) ? 0u : key[i];
        const uint32_t u = (best & 0x80000000u) ? best & 0x7fffffffu : ~best;
        x = best == 0xffffffffu ? __builtin_nanf("") : __builtin_bit_cast(float, u);
      }
      if (j == 0) top = x;
      if (jj == lane) {
        x_mine[jb] = best ? x : -__builtin_inff();
        id_mine[jb] = id;
      }
    }
  }
  float over = 0.f;
#pragma unroll
  for (int jb = 0; jb < R; ++jb) {
    x_mine[jb] = x_mine[jb] == -__builtin_inff() ? 0.f : exp_neg(x_mine[jb] - top);
    over += x_mine[jb];
  }
  if (!a.renorm) {  // the sum over all experts
    over = 0.f;
    if (live) {
#pragma unroll
      for (int i = 0; i < V; ++i) over += v[i] == -__builtin_inff() ? 0.f : exp_neg(v[i] - top);
    }
  }
  over = lanes_sum<L>(over);
  const float inv = over == 0.f ? 0.f : 1.f / over;
  if (t < a.tokens) {
#pragma unroll
    for (int jb = 0; jb < R; ++jb) {
      const int j = jb * L + lane;
      if (j < a.k) {
        a.ids[t * a.k + j] = (int32_t)id_mine[jb];
        // (a choice that is not there weighs 0 also where inv is NaN)
        a.weights[t * a.k + j] = id_mine[jb] == 0xffffffffu ? 0.f : x_mine[jb] * inv;
      }
    }
  }
}

// Lane j % L of a token takes choice j: its logit, its softmax term, its part of
// the dot product.  What belongs to a chosen expert (its gradient, or dw where
// the softmax is over all) goes to the expert's place through LDS, where a
// token's row starts as zeros.  A token's lanes are in one wave.  Renormalized,
// only the chosen logits are read and the time is the gradient's write: 17.5 us
// for 65536 x 256 float32, 8 choices (67 MB, 3.8 TB/s; 40.6 us with each lane
// searching the token's ids for its experts).
template <int WD, int L, int V>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(RouteArgs a, bool vec) {
  constexpr int R = (kMaxChoices + L - 1) / L;
  __shared__ float place[kThreads * V];
  const int lane = threadIdx.x % L, E = a.experts;
  const int64_t t = (int64_t)blockIdx.x * (kThreads / L) + threadIdx.x / L;
  const bool here = t < a.tokens;
  float* row = place + threadIdx.x / L * (L * V);
  uint32_t id[R];
  float dw[R], x[R];
#pragma unroll
  for (int jb = 0; jb < R; ++jb) {
    const int j = jb * L + lane;
    id[jb] = here && j < a.k ? (uint32_t)a.ids[t * a.k + j] : 0xffffffffu;
    dw[jb] = id[jb] < (uint32_t)E ? a.grad_weights[t * a.k + j] : 0.f;
  }
#pragma unroll
  for (int jb = 0; jb < R; ++jb)
    x[jb] = id[jb] < (uint32_t)E ? ld_elem<WD>(a.logits, t * a.ld + id[jb]) : -__builtin_inff();
  const uint32_t any = lanes<Min, L>(id[0]);  // a row with a choice has its first
  float p[V];
  if (!a.renorm && any < (uint32_t)E) load_logits<WD, L, V>(a.logits, t * a.ld, lane, E, vec, p);
#pragma unroll
  for (int i = 0; i < V; ++i) row[i * L + lane] = 0.f;
  // the first choice has the largest logit (NaN in it reaches every term)
  const float top = __shfl(x[0], 0, L);
  float sum = 0.f, dot = 0.f;
#pragma unroll
  for (int jb = 0; jb < R; ++jb) {
    x[jb] = x[jb] == -__builtin_inff() ? 0.f : exp_neg(x[jb] - top);
    sum += x[jb];
    dot = fmaf(x[jb], dw[jb], dot);
  }
  if (!a.renorm) {
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] = any >= (uint32_t)E || p[i] == -__builtin_inff() ? 0.f : exp_neg(p[i] - top);
      sum += p[i];
    }
  }
  sum = lanes_sum<L>(sum);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  dot = lanes_sum<L>(dot) * inv;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int jb = 0; jb < R; ++jb)
    if (id[jb] < (uint32_t)E) row[id[jb]] = a.renorm ? x[jb] * inv * (dw[jb] - dot) : dw[jb];
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  if (!here) return;
  constexpr int C = kVec16<WD>;
#pragma unroll
  for (int i = 0; i < V; i += C) {
    const int e = expert_of<WD, L>(lane, i);
    float g[C];
#pragma unroll
    for (int q = 0; q < C; ++q) {
      g[q] = row[e + q];
      if (!a.renorm) g[q] = p[i + q] * inv * (g[q] - dot);
    }
    if (vec && e + C <= E) {
      store_w<WD, C>(a.grad_logits, t * a.ldg + e, g);
    } else {
#pragma unroll
      for (int q = 0; q < C; ++q)
        if (e + q < E) st_elem<WD>(a.grad_logits, t * a.ldg + e + q, g[q]);
    }
  }
}

template <int WD, int L, int V>
hipError_t run(const RouteArgs& a, bool backward, hipStream_t s) {
  const int es = WD == WD_F32 ? 4 : 2;
  const int64_t wgs = cdiv(a.tokens, kThreads / L);
  if (!fits_grid(wgs)) return hipErrorInvalidConfiguration;
  const dim3 grid((uint32_t)wgs);
  const bool in16 = aligned16(a.logits) && (a.ld * es) % 16 == 0;
  if (backward) {
    const bool vec = in16 && aligned16(a.grad_logits) && (a.ldg * es) % 16 == 0;
    TBE_LAUNCH("route_backward", (route_backward_kernel<WD, L, V>), grid, dim3(kThreads), s, a, vec);
  } else {
    TBE_LAUNCH("route", (route_kernel<WD, L, V>), grid, dim3(kThreads), s, a, in16);
  }
  return hipGetLastError();
}

// Lanes and logits a lane by E: 16 logits a lane (half the exchanges of 8 logits
// a lane: 30.5 against 49.7 us at 256 experts), 8 for E <= 64 so that a token
// still has 8 lanes.
template <int WD>
hipError_t by_experts(const RouteArgs& a, bool backward, hipStream_t s) {
  if (a.experts <= 64) return run<WD, 8, 8>(a, backward, s);
  if (a.experts <= 128) return run<WD, 8, 16>(a, backward, s);
  if (a.experts <= 256) return run<WD, 16, 16>(a, backward, s);
  if (a.experts <= 512) return run<WD, 32, 16>(a, backward, s);
  return run<WD, 64, 16>(a, backward, s);
}

hipError_t route_any(const RouteArgs& a, bool backward, hipStream_t s) {
  if (a.tokens == 0) return hipSuccess;
  switch (a.dtype) {
    case WD_F32: return by_experts<WD_F32>(a, backward, s);
    case WD_F16: return by_experts<WD_F16>(a, backward, s);
    default: return by_experts<WD_BF16>(a, backward, s);
  }
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s) { return route_any(a, false, s); }
hipError_t launch_route_backward(const RouteArgs& a, hipStream_t s) {
  return route_any(a, true, s);
}

}  // namespace tbe
