// Internal declarations of the expert-layer operators (include/tbe_experts.h):
// argument blocks and launchers that each kernel file provides to the C-ABI
// layer, and small device helpers they share.
#pragma once

#include "tbe_common.h"

namespace tbe {

constexpr int kF8Block = 128;       // contraction elements that share one scale
constexpr int kMaxExperts = 1024;
constexpr int kMaxChoices = 32;

inline int64_t up_to(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
inline int64_t cdiv(int64_t x, int64_t m) { return (x + m - 1) / m; }
// Whether a launch of so many workgroups of kThreads fits: its threads are counted
// in 32 bits.  (A launcher answers hipErrorInvalidConfiguration where it does not.)
inline bool fits_grid(int64_t wgs) { return wgs <= 0xffffffffll / kThreads; }
inline int64_t f8_ld(int64_t c) { return up_to(c, kF8Block); }                 // bytes a value row
inline int64_t f8_scale_ld(int64_t c) { return up_to(cdiv(c, kF8Block), 4); }  // bytes a scale row

struct RouteArgs {
  int64_t tokens;
  int32_t experts, k;
  int dtype;
  const void* logits;
  int64_t ld;
  const uint8_t* valid;
  bool renorm;
  int32_t* ids;
  float* weights;
  const float* grad_weights;  // backward
  void* grad_logits;
  int64_t ldg;
};
hipError_t launch_route(const RouteArgs& a, hipStream_t s);
hipError_t launch_route_backward(const RouteArgs& a, hipStream_t s);

struct ExpertSortArgs {
  int64_t n;  // tokens * k
  int32_t experts, align, itype;
  const void* ids;
  int32_t *offsets, *slots, *source;
  int64_t rows;
  uint32_t* ws;
};
size_t expert_sort_ws(int64_t n, int32_t experts, int64_t rows);
hipError_t launch_expert_sort(const ExpertSortArgs& a, hipStream_t s);

struct ExpertRowArgs {
  int64_t tokens;
  int32_t k;
  int64_t rows, width;
  int dtype;
  const void* x;  // dispatch: token rows; combine backward: grad_out
  int64_t ldx;
  const void* y;  // combine: expert rows
  int64_t ldy;
  const int32_t *slots, *source;
  const float* weights;
  void* out;  // dispatch: expert rows; combine: token rows; combine backward: grad_y
  int64_t ldo;
  float* grad_weights;
  uint8_t* scales;  // dispatch to the 8-bit form
};
hipError_t launch_expert_dispatch(const ExpertRowArgs& a, hipStream_t s);
hipError_t launch_expert_dispatch_f8(const ExpertRowArgs& a, hipStream_t s);
hipError_t launch_expert_combine(const ExpertRowArgs& a, hipStream_t s);
hipError_t launch_expert_combine_backward(const ExpertRowArgs& a, hipStream_t s);

struct QuantArgs {
  int64_t batch, rows, cols;
  int dtype;
  const void* x;
  int64_t ldx, batch_stride;
  bool square;
  void* row_values;
  uint8_t* row_scales;
  void* col_values;
  uint8_t* col_scales;
};
hipError_t launch_quantize_f8(const QuantArgs& a, hipStream_t s);

struct MatmulF8Args {
  int32_t experts;
  int64_t m, n, k;  // k: bytes of a value row (a multiple of 128); segments: the rows
  const uint8_t *a, *sa, *b, *sb;
  int64_t lds;  // bytes of a scale row
  bool square;
  const int32_t* offsets;
  int dtype;
  void* out;
  int64_t ldo;
};
hipError_t launch_matmul_f8(const MatmulF8Args& a, hipStream_t s);
hipError_t launch_matmul_f8_segments(const MatmulF8Args& a, hipStream_t s);

size_t clip_ws(int32_t n, const int64_t* sizes);
hipError_t launch_clip(int32_t n, const void* const* grads, void* const* outs,
                       const int64_t* sizes, const int32_t* dtypes, float max_norm, float* norm,
                       void* ws, hipStream_t s);

// ------------------------------------------------------------- device helpers

// One element of storage type WD at element index e, as float, and back
// (one rounding, to nearest even).
template <int WD>
__device__ __forceinline__ float ld_elem(const void* p, int64_t e) {
  if constexpr (WD == WD_F32) return gload(reinterpret_cast<const float*>(p) + e);
  const uint32_t u = *((const __attribute__((address_space(1))) uint16_t*)p + e);
  if constexpr (WD == WD_F16) return f16_bits_to_float(u); else return bf16_bits_to_float(u);
}
template <int WD>
__device__ __forceinline__ void st_elem(void* p, int64_t e, float v) {
  if constexpr (WD == WD_F32) { gstore(reinterpret_cast<float*>(p) + e, v); return; }
  *((__attribute__((address_space(1))) uint16_t*)p + e) =
      WD == WD_F16 ? float_to_f16_bits(v) : float_to_bf16_bits(v);
}

// VEC consecutive elements (VEC = 1, or the 16 bytes of the type).
template <int WD> constexpr int kVec16 = WD == WD_F32 ? 4 : 8;
template <int WD, int VEC>
__device__ __forceinline__ void st_vec(void* p, int64_t e, const float* v) {
  if constexpr (VEC == 1) st_elem<WD>(p, e, v[0]); else store_w<WD, VEC>(p, e, v);
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

}  // namespace tbe
