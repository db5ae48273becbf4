// The 8-bit form of a matrix: e4m3 values with one power-of-two scale for each
// 128 elements along the contraction (or each 128 x 128 square).
//
// The scale's exponent is the smallest e >= -126 with max|x| / 448 <= 2^e.
// 448 is 1.75 * 2^8, so e + 127 is the maximum's own exponent field less 8,
// plus one where its significand is above 1.75: an integer addition on its
// bits.  Scaling by 2^-e is exact, so a value is rounded once, by the
// conversion, and every order of work gives the same bytes.
//
// All of it is one read of the matrix and one write of each form, bound by memory
// where the matrix is large: 65536 x 2048 bfloat16 by rows 70 us (404 MB,
// 5.8 TB/s), 34816 x 4096 in both forms 100 us (570 MB, 5.7 TB/s); the weights of
// 16 experts of 4096 x 2048 by squares, from float32 118 us and in both
// orientations 143 (671 and 805 MB, 5.6 TB/s), from bfloat16 76 and 101.
#include "experts_common.h"

namespace tbe {
namespace {

constexpr uint32_t kInfBits = 0x7f800000u;

// Scale byte e + 127 of a block whose largest finite magnitude has bits u.
__device__ __forceinline__ uint32_t scale_byte(uint32_t u) {
  const int s = (int)((u + 0x1fffffu) >> 23) - 8;
  return s < 1 ? 1u : (uint32_t)s;
}
// 2^-e for scale byte e + 127.
__device__ __forceinline__ float scale_inv(uint32_t s) {
  return __builtin_bit_cast(float, (254u - s) << 23);
}

// Four floats to e4m3, scaled.
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d, float inv) {
  const int v = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, v, true);
}

// Eight consecutive elements as they are stored.  `most` of two packs is taken
// element by element on their magnitudes: a 16-bit float's order is that of its
// bits, two to a word.
typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
template <int WD>
struct Pack {
  static constexpr int W = WD == WD_F32 ? 8 : 4;  // words
  static constexpr uint32_t INF = WD == WD_F32 ? 0x7f800000u : WD == WD_F16 ? 0x7c00u : 0x7f80u;
  static constexpr uint32_t ABS = WD == WD_F32 ? 0x7fffffffu : 0x7fff7fffu;
  uint32_t w[W];

  __device__ __forceinline__ void load(const void* p, int64_t e, int64_t n, bool vec) {
    if (vec && n >= 8) {
#pragma unroll
      for (int i = 0; i < W; i += 4) {
        const u32x4_t x = ld16<false>((const uint8_t*)p + e * (W / 2) + i * 4);
        w[i] = x.x; w[i + 1] = x.y; w[i + 2] = x.z; w[i + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if constexpr (WD == WD_F32) {
          w[i] = i < n ? __builtin_bit_cast(uint32_t, ld_elem<WD>(p, e + i)) : 0u;
        } else {
          const auto* h = (const __attribute__((address_space(1))) uint16_t*)p + e;
          w[i] = (2 * i < n ? (uint32_t)h[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)h[2 * i + 1] << 16 : 0u);
        }
      }
    }
  }
  __device__ __forceinline__ float value(int i) const {
    if constexpr (WD == WD_F32) return __builtin_bit_cast(float, w[i]);
    const uint32_t u = i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu;
    if constexpr (WD == WD_F16) return f16_bits_to_float(u); else return bf16_bits_to_float(u);
  }
  __device__ __forceinline__ void most(const Pack& o) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = word_max(w[i], o.w[i] & ABS);
  }
  // largest magnitude of the eight, as the bits of a float
  __device__ __forceinline__ uint32_t largest() const {
    uint32_t m = w[0] & ABS;
#pragma unroll
    for (int i = 1; i < W; ++i) m = word_max(m, w[i] & ABS);
    if constexpr (WD != WD_F32) m = (m >> 16) > (m & 0xffffu) ? m >> 16 : m & 0xffffu;
    return bits(m);
  }
  __device__ __forceinline__ uint32_t magnitude(int i) const {  // of element i, as float bits
    if constexpr (WD == WD_F32) return w[i] & ABS;
    return bits((i & 1 ? w[i / 2] >> 16 : w[i / 2]) & 0x7fffu);
  }
  // Infinities become NaN, which no scale changes; `finite` is the pack with both
  // set to 0.  (Only where some element is not finite.)
  __device__ __forceinline__ void to_nan(Pack* finite) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      finite->w[i] = 0;
      constexpr int H = WD == WD_F32 ? 1 : 2;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const uint32_t m = WD == WD_F32 ? w[i] & ABS : (w[i] >> (16 * h)) & 0x7fffu;
        if (m >= INF) w[i] |= WD == WD_F32 ? 0x7fffffffu : 0x7fffu << (16 * h);
        else finite->w[i] |= m << (16 * h);
      }
    }
  }
  static __device__ __forceinline__ uint32_t word_max(uint32_t a, uint32_t b) {
    if constexpr (WD == WD_F32) return a > b ? a : b;
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a),
                                                                  __builtin_bit_cast(u16x2_t, b)));
  }
  static __device__ __forceinline__ uint32_t bits(uint32_t m) {
    if constexpr (WD == WD_F32) return m;
    if constexpr (WD == WD_BF16) return m << 16;
    return __builtin_bit_cast(uint32_t, f16_bits_to_float(m));
  }
};

// Largest of a row of 16 lanes, in all of them.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xf, 0xf, false);
  return v > o ? v : o;
}
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  v = dpp_max<0x128>(v);  // rotations of the row by 8, 4, 2, 1
  v = dpp_max<0x124>(v);
  v = dpp_max<0x122>(v);
  return dpp_max<0x121>(v);
}

constexpr int kT = kF8Block;      // tile edge
constexpr int kPitch = kT + 8;    // bytes of a transposed tile row in LDS

// One 128 x 128 tile a workgroup.  Thread t holds rows 8 (t / 16) + 0..7 of
// columns 8 (t % 16) + 0..7: a row's 128 columns are 16 neighbouring lanes; a
// column's 128 rows are the 16 row groups, four of a wave joined by lane
// exchanges, then the four waves through LDS.  The transposed bytes go through
// LDS eight rows at a time; the group's place there is turned by the column so
// that a wave's writes fall evenly on the banks.  Elements stay packed as they
// are stored until they are scaled, which keeps the 64 of a thread in 32
// registers.  (34816 x 4096 both forms and 34816 x 2048 transposed: 141 us; with
// float32 elements and column maxima by LDS atomics 366.)
template <int WD, bool SQUARE, bool ROWS, bool COLS>
__global__ __launch_bounds__(kThreads) void quant_tile_kernel(QuantArgs a, uint32_t ctiles,
                                                              bool vec) {
  using P = Pack<WD>;
  __shared__ __attribute__((aligned(16))) uint32_t red[4][kT];
  __shared__ __attribute__((aligned(16))) uint8_t tr[COLS ? kT * kPitch : 16];
  const int cg = threadIdx.x % 16, rg = threadIdx.x / 16, wave = threadIdx.x / kWave;
  const uint32_t rt = blockIdx.x / ctiles, ct = blockIdx.x % ctiles;
  const int64_t r0 = (int64_t)rt * kT, c0 = (int64_t)ct * kT, b = blockIdx.y;
  const int64_t R = a.rows, C = a.cols;
  P v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + rg * 8 + i, c = c0 + cg * 8;
    v[i].load(a.x, b * a.batch_stride + r * a.ldx + c, r < R ? C - c : 0, vec);
  }
  P col{};  // largest of each column over this thread's rows
#pragma unroll
  for (int i = 0; i < 8; ++i) col.most(v[i]);
  uint32_t row[8];
  if constexpr (ROWS && !SQUARE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) row[i] = v[i].largest();
  }
  if (__any(col.largest() >= kInfBits)) {
    col = P{};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      P finite;
      v[i].to_nan(&finite);
      col.most(finite);
      if constexpr (ROWS && !SQUARE) row[i] = finite.largest();
    }
  }
  uint32_t sq = 0, scol[8];
  if constexpr (SQUARE) {
    uint32_t m = row16_max(col.largest());
#pragma unroll
    for (int x = 16; x < kWave; x <<= 1) {
      const uint32_t o = (uint32_t)__shfl_xor((int)m, x, kWave);
      m = m > o ? m : o;
    }
    if (threadIdx.x % kWave == 0) red[0][wave] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) m = m > red[0][w] ? m : red[0][w];
    sq = scale_byte(m);
  } else if constexpr (COLS) {
#pragma unroll
    for (int x = 16; x < kWave; x <<= 1) {
      P o;
#pragma unroll
      for (int i = 0; i < P::W; ++i) o.w[i] = (uint32_t)__shfl_xor((int)col.w[i], x, kWave);
      col.most(o);
    }
    constexpr int W = P::W;
    if (threadIdx.x % kWave < 16) {
#pragma unroll
      for (int i = 0; i < W; ++i) red[wave][cg * W + i] = col.w[i];
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      P o;
#pragma unroll
      for (int i = 0; i < W; ++i) o.w[i] = red[w][cg * W + i];
      col.most(o);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) scol[q] = scale_byte(col.magnitude(q));
  }
  if constexpr (ROWS) {
    const int64_t ld = (C + kT - 1) / kT * kT, blocks = ld / kT, lds = (blocks + 3) / 4 * 4;
    uint8_t* val = reinterpret_cast<uint8_t*>(a.row_values) + b * R * ld;
    const bool last = (int64_t)ct == blocks - 1;
    const int64_t at = (int64_t)ct + cg;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = r0 + rg * 8 + i;
      const uint32_t s = SQUARE ? sq : scale_byte(row16_max(row[i]));
      const float inv = scale_inv(s);
      if (r < R) {
        *reinterpret_cast<uint2*>(val + r * ld + c0 + cg * 8) =
            make_uint2(pack4(v[i].value(0), v[i].value(1), v[i].value(2), v[i].value(3), inv),
                       pack4(v[i].value(4), v[i].value(5), v[i].value(6), v[i].value(7), inv));
        const int64_t sr = SQUARE ? b * ((R + kT - 1) / kT) + rt : b * R + r;
        if ((!SQUARE || (i == 0 && rg == 0)) && (cg == 0 || (last && at < lds)))
          a.row_scales[sr * lds + at] = cg == 0 ? (uint8_t)s : (uint8_t)0;
      }
    }
  }
  if constexpr (COLS) {
    const int64_t ld = (R + kT - 1) / kT * kT, blocks = ld / kT, lds = (blocks + 3) / 4 * 4;
    const bool last = (int64_t)rt == blocks - 1;
    const int64_t at = (int64_t)rt + rg;
    const int place = (rg ^ ((cg >> 2) * 4)) * 8;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const uint32_t s = SQUARE ? sq : scol[q];
      const float inv = scale_inv(s);
      *reinterpret_cast<uint2*>(&tr[(cg * 8 + q) * kPitch + place]) =
          make_uint2(pack4(v[0].value(q), v[1].value(q), v[2].value(q), v[3].value(q), inv),
                     pack4(v[4].value(q), v[5].value(q), v[6].value(q), v[7].value(q), inv));
      const int64_t c = c0 + cg * 8 + q;
      const int64_t sr = SQUARE ? b * ((C + kT - 1) / kT) + ct : b * C + c;
      if (c < C && (!SQUARE || (q == 0 && cg == 0)) && (rg == 0 || (last && at < lds)))
        a.col_scales[sr * lds + at] = rg == 0 ? (uint8_t)s : (uint8_t)0;
    }
    __syncthreads();
    uint8_t* val = reinterpret_cast<uint8_t*>(a.col_values) + b * C * ld;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = i * kThreads + threadIdx.x;  // 16-byte pieces, 8 a column
      const int c = n / 8, piece = n % 8;
      const uint8_t* p = &tr[c * kPitch + (piece ^ ((c >> 5) * 2)) * 16];
      const uint2 lo = *reinterpret_cast<const uint2*>(p);
      const uint2 hi = *reinterpret_cast<const uint2*>(p + 8);
      if (c0 + c < C)
        *reinterpret_cast<uint4*>(val + (c0 + c) * ld + r0 + piece * 16) =
            make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
  }
}

// Rows alone, a scale a row block: 16 lanes take a block, without LDS or a
// meeting.  (24 rows of 2048: 4.0 us, 4.8 by the tile kernel; 65536 rows: the
// memory's rate with both.)
template <int WD>
__global__ __launch_bounds__(kThreads) void quant_rows_kernel(QuantArgs a, uint32_t blocks,
                                                              int64_t lds, bool vec) {
  const uint32_t group = (blockIdx.x * kThreads + threadIdx.x) / 16, l = threadIdx.x % 16;
  const uint32_t q = group / blocks, blk = group - q * blocks;
  const int64_t row = q, b = blockIdx.y, ld = (int64_t)blocks * kT;
  if (row >= a.rows) return;
  const int64_t c = (int64_t)blk * kT + l * 8;
  Pack<WD> v;
  v.load(a.x, b * a.batch_stride + row * a.ldx + c, a.cols - c, vec);
  uint32_t m = v.largest();
  if (__any(m >= kInfBits)) {
    Pack<WD> finite;
    v.to_nan(&finite);
    m = finite.largest();
  }
  const uint32_t s = scale_byte(row16_max(m));
  const float inv = scale_inv(s);
  const int64_t r = b * a.rows + row;
  *reinterpret_cast<uint2*>((uint8_t*)a.row_values + r * ld + c) =
      make_uint2(pack4(v.value(0), v.value(1), v.value(2), v.value(3), inv),
                 pack4(v.value(4), v.value(5), v.value(6), v.value(7), inv));
  // the last block's lanes write the zeros that end the scale row
  if (l == 0 || (blk == blocks - 1 && blk + l < lds))
    a.row_scales[r * lds + blk + l] = l == 0 ? (uint8_t)s : (uint8_t)0;
}

// Token rows to the 8-bit form of their expert rows: a wave a token, four
// blocks of 128 columns a step (16 lanes each), written to every slot.  Bound by
// memory: 32768 tokens of 2048 bfloat16 columns, 4 choices, 139264 rows take 90 us,
// 134 MB read and 287 MB written, 4.7 TB/s (dispatch and quantize_f8 after each
// other 277); 8 tokens 5.4 us, four steps' latency.
constexpr int kClearRows = 16;
template <int WD>
__global__ __launch_bounds__(kThreads) void dispatch_f8_kernel(ExpertRowArgs a, int64_t clear_units,
                                                               int64_t ld, int64_t lds, bool vec) {
  const int lane = threadIdx.x % kWave;
  int64_t unit = (int64_t)blockIdx.x * (kThreads / kWave) + threadIdx.x / kWave;
  uint8_t* out = reinterpret_cast<uint8_t*>(a.out);
  if (unit < clear_units) {
    const int64_t mine = unit * kClearRows + lane;
    const bool clear = lane < kClearRows && mine < a.rows &&
                       (a.source[mine] < 0 || a.source[mine] >= a.tokens * a.k);
    uint64_t todo = __ballot(clear);
    while (todo) {
      const int64_t r = unit * kClearRows + __ffsll((unsigned long long)todo) - 1;
      todo &= todo - 1;
      for (int64_t c = lane * 8; c < ld; c += kWave * 8)
        *reinterpret_cast<uint2*>(out + r * ld + c) = make_uint2(0, 0);
      for (int64_t c = lane; c < lds; c += kWave) a.scales[r * lds + c] = c < ld / kT ? 1 : 0;
    }
    return;
  }
  unit -= clear_units;
  if (unit >= a.tokens) return;
  for (int64_t c = (int64_t)lane * 8; c < lds * kT; c += kWave * 8) {  // 512 columns a step: four scale bytes
    Pack<WD> v;
    v.load(a.x, unit * a.ldx + c, a.width - c, vec);
    uint32_t m = v.largest();
    if (__any(m >= kInfBits)) {
      Pack<WD> finite;
      v.to_nan(&finite);
      m = finite.largest();
    }
    const uint32_t s = scale_byte(row16_max(m));
    const float inv = scale_inv(s);
    const uint2 w = make_uint2(pack4(v.value(0), v.value(1), v.value(2), v.value(3), inv),
                               pack4(v.value(4), v.value(5), v.value(6), v.value(7), inv));
    for (int j = 0; j < a.k; ++j) {
      const uint32_t r = (uint32_t)a.slots[unit * a.k + j];
      if (r >= (uint64_t)a.rows) continue;
      if (c < ld) *reinterpret_cast<uint2*>(out + (int64_t)r * ld + c) = w;
      if (lane % 16 == 0) a.scales[(int64_t)r * lds + c / kT] = c < ld ? (uint8_t)s : (uint8_t)0;
    }
  }
}

template <int WD>
hipError_t run_quant(const QuantArgs& a, hipStream_t s) {
  const int es = WD == WD_F32 ? 4 : 2;
  const bool vec = aligned16(a.x) && (a.ldx * es) % 16 == 0 && (a.batch_stride * es) % 16 == 0;
  if (!a.square && !a.col_values) {
    const uint32_t blocks = (uint32_t)cdiv(a.cols, kT);
    const int64_t wgs = cdiv(a.rows * blocks, kThreads / 16);
    if (!fits_grid(wgs)) return hipErrorInvalidConfiguration;
    const dim3 grid((uint32_t)wgs, (uint32_t)a.batch);
    TBE_LAUNCH("quantize_f8", (quant_rows_kernel<WD>), grid, dim3(kThreads), s, a, blocks,
               f8_scale_ld(a.cols), vec);
    return hipGetLastError();
  }
  const uint32_t ctiles = (uint32_t)cdiv(a.cols, kT);
  if (!fits_grid(cdiv(a.rows, kT) * ctiles)) return hipErrorInvalidConfiguration;
  const dim3 grid((uint32_t)cdiv(a.rows, kT) * ctiles, (uint32_t)a.batch);
  const dim3 blk(kThreads);
#define TBE_QUANT(SQ, RW, CL) \
  TBE_LAUNCH("quantize_f8", (quant_tile_kernel<WD, SQ, RW, CL>), grid, blk, s, a, ctiles, vec)
  if (a.square) {
    if (a.row_values && a.col_values) TBE_QUANT(true, true, true);
    else if (a.row_values) TBE_QUANT(true, true, false);
    else TBE_QUANT(true, false, true);
  } else {
    if (a.row_values && a.col_values) TBE_QUANT(false, true, true);
    else TBE_QUANT(false, false, true);
  }
#undef TBE_QUANT
  return hipGetLastError();
}

template <int WD>
hipError_t run_dispatch_f8(const ExpertRowArgs& a, hipStream_t s) {
  const int es = WD == WD_F32 ? 4 : 2;
  const bool vec = aligned16(a.x) && (a.ldx * es) % 16 == 0;
  const int64_t clear = cdiv(a.rows, kClearRows);
  if (!fits_grid(cdiv(clear + a.tokens, kThreads / kWave))) return hipErrorInvalidConfiguration;
  TBE_LAUNCH("expert_dispatch_f8", (dispatch_f8_kernel<WD>),
             dim3((uint32_t)cdiv(clear + a.tokens, kThreads / kWave)), dim3(kThreads), s, a, clear,
             f8_ld(a.width), f8_scale_ld(a.width), vec);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_f8(const QuantArgs& a, hipStream_t s) {
  if (a.batch == 0 || a.rows == 0 || a.cols == 0) return hipSuccess;
  switch (a.dtype) {
    case WD_F32: return run_quant<WD_F32>(a, s);
    case WD_F16: return run_quant<WD_F16>(a, s);
    default: return run_quant<WD_BF16>(a, s);
  }
}

hipError_t launch_expert_dispatch_f8(const ExpertRowArgs& a, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  switch (a.dtype) {
    case WD_F32: return run_dispatch_f8<WD_F32>(a, s);
    case WD_F16: return run_dispatch_f8<WD_F16>(a, s);
    default: return run_dispatch_f8<WD_BF16>(a, s);
  }
}

}  // namespace tbe
