// Token rows sorted by expert, and back.
//
// The sort is a stable counting sort of n = tokens * k expert ids: per-tile
// counts, an exclusive prefix of each expert's counts over the tiles, then the
// placement, where a choice's rank inside its tile is the number of equal ids
// before it.  Everything that follows is row traffic, bound by memory: each
// kernel walks the tokens, so a token's row is read once however many experts
// take it (the combination's gradient reads it once for every four choices), and
// the rows that hold no choice are zeroed by workgroups of the same launch.
//
// Measured with 32768 tokens of 2048 bfloat16 columns, 4 choices of 64 experts,
// segments aligned to 128 (139264 rows):
//   sort       count 5.4, prefix 4.0, placement 7.3 us: launches and LDS atomics
//   dispatch   141 us, 134 MB read and 570 MB written: 5.0 TB/s
//   combine    125 us, 537 MB read and 134 MB written: 5.4 TB/s
//   its gradient 230 us, 671 MB read and 570 MB written: 5.4 TB/s
// against 4.8 TB/s of a large copy.
#include "experts_common.h"

#include <algorithm>

namespace tbe {
namespace {

// ------------------------------------------------------------------ the sort

constexpr int kSortItems = 8;                          // ids a thread
constexpr int kSortTile = kThreads * kSortItems;       // ids a tile
constexpr int kWaves = kThreads / kWave;

template <typename IT>
__device__ __forceinline__ uint32_t expert_at(const void* ids, int64_t i, int64_t n, uint32_t E) {
  if (i >= n) return E;
  const int64_t v = (int64_t)reinterpret_cast<const IT*>(ids)[i];
  return v < 0 || v >= (int64_t)E ? E : (uint32_t)v;  // E: dropped
}

// cnt[tile * E + e]: ids of expert e in the tile.
template <typename IT>
__global__ __launch_bounds__(kThreads) void expert_count_kernel(const void* ids, int64_t n,
                                                                uint32_t E, uint32_t* cnt) {
  __shared__ uint32_t h[kMaxExperts];
  for (uint32_t e = threadIdx.x; e < E; e += kThreads) h[e] = 0;
  __syncthreads();
  const int64_t b = (int64_t)blockIdx.x * kSortTile;
#pragma unroll
  for (int i = 0; i < kSortItems; ++i) {
    const uint32_t e = expert_at<IT>(ids, b + i * kThreads + threadIdx.x, n, E);
    if (e < E) atomicAdd(&h[e], 1u);
  }
  __syncthreads();
  for (uint32_t e = threadIdx.x; e < E; e += kThreads) cnt[(size_t)blockIdx.x * E + e] = h[e];
}

// One workgroup an expert: exclusive prefix of its counts over the tiles (in
// place) and its total.
__global__ __launch_bounds__(kThreads) void expert_prefix_kernel(uint32_t* cnt, uint32_t tiles,
                                                                 uint32_t E, uint32_t* total) {
  __shared__ uint32_t sh[kWaves];
  const uint32_t e = blockIdx.x;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  uint32_t run = 0;
  for (uint32_t t0 = 0; t0 < tiles; t0 += kThreads) {
    const uint32_t t = t0 + threadIdx.x;
    const uint32_t c = t < tiles ? cnt[(size_t)t * E + e] : 0u;
    uint32_t x = c;
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1) {
      const uint32_t o = (uint32_t)__shfl_up((int)x, m, kWave);
      x += lane >= m ? o : 0u;
    }
    if (lane == kWave - 1) sh[wave] = x;
    __syncthreads();
    uint32_t before = run, all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      before += w < wave ? sh[w] : 0u;
      all += sh[w];
    }
    if (t < tiles) cnt[(size_t)t * E + e] = before + x - c;
    run += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) total[e] = run;
}

// start[e] = first row of expert e's segment, start[E] the end: an exclusive
// prefix of the aligned totals, by the whole workgroup of TH threads.
template <int TH>
__device__ __forceinline__ void segment_starts(const uint32_t* total, uint32_t E, uint32_t align,
                                               uint32_t* start, uint32_t* sh) {
  constexpr int P = kMaxExperts / TH;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  uint32_t v[P], s = 0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const uint32_t e = threadIdx.x * P + i;
    v[i] = e < E ? (total[e] + align - 1) & ~(align - 1) : 0u;  // align is a power of two
    s += v[i];
  }
  uint32_t x = s;
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) {
    const uint32_t o = (uint32_t)__shfl_up((int)x, m, kWave);
    x += lane >= m ? o : 0u;
  }
  if (lane == kWave - 1) sh[wave] = x;
  __syncthreads();
  uint32_t at = x - s;
#pragma unroll
  for (int w = 0; w < TH / kWave; ++w) at += w < wave ? sh[w] : 0u;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const uint32_t e = threadIdx.x * P + i;
    if (e <= E) start[e] = at;
    at += v[i];
  }
  if (threadIdx.x == TH - 1 && E == kMaxExperts) start[E] = at;
  __syncthreads();
}

// Rows that hold no choice become -1 in `source`: the end of every segment, a
// wave each, and all rows past the last.  This is worker `w` of `n` workgroups.
__device__ __forceinline__ void clear_unheld(const uint32_t* start, const uint32_t* total,
                                             uint32_t E, int64_t rows, uint32_t w, uint32_t n,
                                             int32_t* source) {
  const uint32_t waves = blockDim.x / kWave, lane = threadIdx.x % kWave;
  for (uint32_t e = w * waves + threadIdx.x / kWave; e < E; e += n * waves)
    for (uint32_t r = start[e] + total[e] + lane; r < start[e + 1]; r += kWave) source[r] = -1;
  for (int64_t r = (int64_t)start[E] + w * blockDim.x + threadIdx.x; r < rows; r += n * blockDim.x)
    source[r] = -1;
}

// Places a round of 64 choices, lane's at flat position p with expert id (E:
// dropped): a choice's row is its expert's next one (at[id], this wave's) plus
// the lanes before it with the same id; the last of those moves at[id] on.
__device__ __forceinline__ void place_round(const ExpertSortArgs& a, uint32_t E, uint32_t id,
                                            int64_t p, uint32_t* at) {
  const int lane = threadIdx.x % kWave, bits = 32 - __builtin_clz(E);
  uint64_t same = ~0ull;
  for (int q = 0; q < bits; ++q) {
    const uint64_t m = __ballot((id >> q) & 1u);
    same &= (id >> q) & 1u ? m : ~m;
  }
  const bool kept = id < E;
  uint32_t r = 0;
  if (kept) r = at[id] + __popcll(same & ((1ull << lane) - 1));
  // every lane's read above comes before the write below
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (p < a.n) a.slots[p] = kept ? (int32_t)r : -1;
  if (kept) {
    a.source[r] = (int32_t)p;
    if ((same >> lane) == 1ull) at[id] = r + 1;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// Placement.  Workgroups [0, tiles) place their tile's choices; the ones from
// `tiles` on clear the rows that hold none; workgroup 0 also writes the offsets.
template <typename IT>
__global__ __launch_bounds__(kThreads) void expert_place_kernel(ExpertSortArgs a, uint32_t tiles,
                                                                const uint32_t* cnt,
                                                                const uint32_t* total) {
  __shared__ uint32_t start[kMaxExperts + 1];
  __shared__ uint32_t at[kWaves][kMaxExperts];  // next row of each expert, a wave
  __shared__ uint32_t sh[kWaves];
  const uint32_t E = (uint32_t)a.experts;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  segment_starts<kThreads>(total, E, (uint32_t)a.align, start, sh);
  if (blockIdx.x == 0)
    for (uint32_t e = threadIdx.x; e <= E; e += kThreads) a.offsets[e] = (int32_t)start[e];
  if (blockIdx.x >= tiles) {
    clear_unheld(start, total, E, a.rows, blockIdx.x - tiles, gridDim.x - tiles, a.source);
    return;
  }
  // the wave's ids are consecutive: kSortItems rounds of 64
  const int64_t b = (int64_t)blockIdx.x * kSortTile + wave * (kSortItems * kWave);
  uint32_t id[kSortItems];
#pragma unroll
  for (int i = 0; i < kSortItems; ++i) id[i] = expert_at<IT>(a.ids, b + i * kWave + lane, a.n, E);
  for (uint32_t e = threadIdx.x; e < E; e += kThreads)
    for (int w = 0; w < kWaves; ++w) at[w][e] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSortItems; ++i)
    if (id[i] < E) atomicAdd(&at[wave][id[i]], 1u);
  __syncthreads();
  for (uint32_t e = threadIdx.x; e < E; e += kThreads) {
    uint32_t r = start[e] + cnt[(size_t)blockIdx.x * E + e];
    for (int w = 0; w < kWaves; ++w) {
      const uint32_t c = at[w][e];
      at[w][e] = r;
      r += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSortItems; ++i)
    place_round(a, E, id[i], b + i * kWave + lane, at[wave]);
}

// The whole sort in one workgroup of 1024 threads, for batches of at most
// kSortOneIds choices and kSortOneRows rows: a wave takes ROUNDS consecutive
// rounds of 64 ids, all loaded at once; counts and placements stay in LDS, one
// launch.  The limit, us on the device by one launch / by three:
//   choices       1024          4096          8192
//   24 experts    4.9 / 15.4    6.0 / 15.0    9.3 / 14.9
//   256           6.8 / 16.4    8.8 / 16.0   13.1 / 15.7
//   1024         11.7 / 35.6   15.2 / 24.2   19.0 / 17.5
// (segments aligned to 128 take up to 2 us more by one launch, the same by three).
constexpr int kOneThreads = 1024, kOneWaves = kOneThreads / kWave, kOneRounds = 8;
constexpr int64_t kSortOneIds = kOneThreads * kOneRounds, kSortOneRows = 65536;
template <typename IT, int ROUNDS>
__global__ __launch_bounds__(kOneThreads) void expert_sort_one_kernel(ExpertSortArgs a) {
  __shared__ uint32_t start[kMaxExperts + 1];
  __shared__ uint32_t total[kMaxExperts];
  __shared__ uint32_t at[kOneWaves][kMaxExperts];
  __shared__ uint32_t sh[kOneWaves];
  const uint32_t E = (uint32_t)a.experts, n = (uint32_t)a.n;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  // the rounds that there are, shared out evenly
  const uint32_t rounds = ROUNDS == 1 ? 1 : (n + kOneThreads - 1) / kOneThreads;
  const uint32_t b = wave * rounds * kWave + lane;
  uint32_t id[ROUNDS];
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i)
    id[i] = (uint32_t)i < rounds ? expert_at<IT>(a.ids, b + i * kWave, n, E) : E;
  for (uint32_t x = threadIdx.x; x < E * kOneWaves; x += kOneThreads) at[x / E][x % E] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i)
    if (id[i] < E) atomicAdd(&at[wave][id[i]], 1u);
  __syncthreads();
  for (uint32_t e = threadIdx.x; e < E; e += kOneThreads) {
    uint32_t t = 0;
#pragma unroll
    for (int w = 0; w < kOneWaves; ++w) t += at[w][e];
    total[e] = t;
  }
  __syncthreads();
  segment_starts<kOneThreads>(total, E, (uint32_t)a.align, start, sh);
  for (uint32_t e = threadIdx.x; e <= E; e += kOneThreads) {
    uint32_t r = start[e];
    a.offsets[e] = (int32_t)r;
    if (e == E) break;
#pragma unroll
    for (int w = 0; w < kOneWaves; ++w) {
      const uint32_t c = at[w][e];
      at[w][e] = r;
      r += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i)
    if ((uint32_t)i < rounds) place_round(a, E, id[i], b + i * kWave, at[wave]);
  clear_unheld(start, total, E, a.rows, 0, 1, a.source);
}

// --------------------------------------------------------------- row traffic

// Zeroes the rows of a wave's kClearRows that hold no choice (source < 0, or
// out of range).
constexpr int kClearRows = 16;
template <typename U>
__device__ __forceinline__ void zero_rows(const ExpertRowArgs& a, int64_t unit, int64_t width,
                                          int64_t ld, U* out) {
  const int lane = threadIdx.x % kWave;
  const int64_t r0 = unit * kClearRows;
  const int64_t mine = r0 + lane;
  const bool clear = lane < kClearRows && mine < a.rows &&
                     (a.source[mine] < 0 || a.source[mine] >= a.tokens * a.k);
  uint64_t todo = __ballot(clear);
  while (todo) {
    const int r = __ffsll((unsigned long long)todo) - 1;
    todo &= todo - 1;
    U* o = out + (r0 + r) * ld;
    for (int64_t c = lane; c < width; c += kWave) o[c] = U{};
  }
}

// A wave takes one token's columns [part * CH * 64 * VEC, ...), CH loads a lane:
// one of 16 bytes (with four, waves are fewer and longer: combine 153 against
// 122 us, dispatch 151 against 141 at the sizes above), four of one element.
template <bool WIDE>
constexpr int kLoads = WIDE ? 1 : 4;
struct Part {
  int64_t token;
  int64_t col;  // this lane's first column
};
template <int CH, int VEC>
__device__ __forceinline__ Part part_of(uint32_t unit, uint32_t parts) {
  const uint32_t t = unit / parts, p = unit - t * parts;
  return {(int64_t)__builtin_amdgcn_readfirstlane((int)t),
          ((int64_t)p * CH * kWave + threadIdx.x % kWave) * VEC};
}

// Row of choice j of token t, or -1; the same in all lanes.
__device__ __forceinline__ int32_t row_of(const ExpertRowArgs& a, int64_t t, int j) {
  const int32_t r = j < a.k ? a.slots[t * a.k + j] : -1;
  return (uint32_t)r < (uint64_t)a.rows ? r : -1;
}

// Moves of 16 bytes, or of one element of 4 or 2 bytes: a token's columns are
// read once and stored to each of its rows.  (Stores past the caches: 147 against
// 118 us without the zeroed rows.)
template <typename U, int CH = kLoads<sizeof(U) == 16>>
__global__ __launch_bounds__(kThreads) void dispatch_kernel(ExpertRowArgs a, uint32_t clear_units,
                                                            uint32_t units, uint32_t parts,
                                                            int64_t width, int64_t ldx,
                                                            int64_t ldo) {
  uint32_t unit = blockIdx.x * kWaves + threadIdx.x / kWave;
  U* out = reinterpret_cast<U*>(a.out);
  if (unit < clear_units) {
    zero_rows<U>(a, unit, width, ldo, out);
    return;
  }
  unit -= clear_units;
  if (unit >= units) return;
  const Part at = part_of<CH, 1>(unit, parts);
  const U* x = reinterpret_cast<const U*>(a.x) + at.token * ldx;
  U v[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int64_t c = at.col + i * kWave;
    if (c < width) v[i] = x[c];
  }
  for (int j = 0; j < a.k; ++j) {
    const int32_t r = row_of(a, at.token, j);
    if (r < 0) continue;
    U* o = out + (int64_t)r * ldo;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int64_t c = at.col + i * kWave;
      if (c < width) o[c] = v[i];
    }
  }
}

// VEC elements as they are stored (16 bytes, or one element).
template <int WD, int VEC>
struct Held {
  uint32_t w[VEC == 1 ? 1 : 4];
  __device__ __forceinline__ void load(const void* p, int64_t e) {
    if constexpr (VEC == 1) {
      w[0] = __builtin_bit_cast(uint32_t, ld_elem<WD>(p, e));
    } else {
      // past the caches: a row is read once, but for grad_out with more than four choices
      const u32x4_t x = ld16<true>((const uint8_t*)p + e * (16 / VEC));
      w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    }
  }
  __device__ __forceinline__ void get(float* f) const {
    if constexpr (VEC == 1 || WD == WD_F32) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) f[i] = __builtin_bit_cast(float, w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const uint32_t u = i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu;
        f[i] = WD == WD_F16 ? f16_bits_to_float(u) : bf16_bits_to_float(u);
      }
    }
  }
};

// Four choices' columns are under way at a time; a choice without a row reads
// row 0 and takes no part.  Rows are read once, past the caches (160 -> 147 us at
// the sizes above).  Where k is no multiple of four, the loads of row 0 cost: 16384
// tokens of 2048 bfloat16 columns take 36.0 us with k = 1, 46.3 with 2, 67.6 with 4
// and 98.9 with 6; two choices at a time 30.7, 37.4, 65.9 and 94.2.
template <int WD, int VEC, int CH = kLoads<(VEC > 1)>>
__global__ __launch_bounds__(kThreads) void combine_kernel(ExpertRowArgs a, uint32_t units,
                                                           uint32_t parts) {
  constexpr int J = 4;
  const uint32_t unit = blockIdx.x * kWaves + threadIdx.x / kWave;
  if (unit >= units) return;
  const Part at = part_of<CH, VEC>(unit, parts);
  float s[CH][VEC] = {};
  for (int j0 = 0; j0 < a.k; j0 += J) {
    int32_t row[J];
    float w[J];
    Held<WD, VEC> v[J][CH];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      row[j] = row_of(a, at.token, j0 + j);
      w[j] = a.weights && row[j] >= 0 ? a.weights[at.token * a.k + j0 + j] : 1.f;
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int64_t c = at.col + i * kWave * VEC;
        if (c < a.width)
          v[j][i].load(a.y, (int64_t)(row[j] < 0 ? 0 : row[j]) * a.ldy + c);
      }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (row[j] < 0) continue;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        float f[VEC];
        v[j][i].get(f);
#pragma unroll
        for (int x = 0; x < VEC; ++x) s[i][x] = fmaf(w[j], f[x], s[i][x]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int64_t c = at.col + i * kWave * VEC;
    if (c < a.width) st_vec<WD, VEC>(a.out, at.token * a.ldo + c, s[i]);
  }
}

// Lane l's part of J = 4 sums to the whole sum l % 4: halves of the sums change
// lanes in the first two steps (7 exchanges, where a sum at a time takes 24).
template <int CTRL>
__device__ __forceinline__ float lane_moved(float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float four_sums(const float* d) {
  const bool odd = threadIdx.x & 1, high = threadIdx.x & 2;
  const float a = (odd ? d[1] : d[0]) + lane_moved<0xb1>(odd ? d[0] : d[1]);  // lane ^ 1
  const float b = (odd ? d[3] : d[2]) + lane_moved<0xb1>(odd ? d[2] : d[3]);
  float s = (high ? b : a) + lane_moved<0x4e>(high ? a : b);  // lane ^ 2
  s += lane_moved<0x124>(s);                                  // turned by 4, then 8, in 16 lanes
  s += lane_moved<0x128>(s);
  s += __shfl_xor(s, 16, kWave);
  return s + __shfl_xor(s, 32, kWave);
}

// WPT waves a token (1, or the 4 of a workgroup) share its columns; four choices
// at a time.  A choice's gradient is a dot product over the columns: the lanes'
// parts are added in float32 by exchanges, the waves' in LDS.  (One pass: a
// choice's row is read for the dot product beside the write of its gradient.
// grad_out's row is read again for every four choices: 16384 tokens of 2048
// bfloat16 columns take 114.6 us with k = 4 and 236.8 with k = 8, of whose traffic
// the second reading is a seventeenth.)
template <int WD, int VEC, int WPT>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(ExpertRowArgs a,
                                                                    uint32_t clear_wgs) {
  constexpr int J = 4;
  __shared__ float part[kWaves][J];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  if (blockIdx.x < clear_wgs) {
    const uint32_t unit = blockIdx.x * kWaves + wave;
    if constexpr (VEC == 1) {
      if constexpr (WD == WD_F32) zero_rows<float>(a, unit, a.width, a.ldo, reinterpret_cast<float*>(a.out));
      else zero_rows<uint16_t>(a, unit, a.width, a.ldo, reinterpret_cast<uint16_t*>(a.out));
    } else {
      zero_rows<u32x4_t>(a, unit, a.width / VEC, a.ldo / VEC, reinterpret_cast<u32x4_t*>(a.out));
    }
    return;
  }
  const uint32_t unit = (blockIdx.x - clear_wgs) * (kWaves / WPT) + (WPT > 1 ? 0 : wave);
  if (unit >= a.tokens) return;
  const int64_t t = __builtin_amdgcn_readfirstlane((int)unit);
  for (int j0 = 0; j0 < a.k; j0 += J) {
    int32_t row[J];
    float w[J], dot[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      row[j] = row_of(a, t, j0 + j);
      w[j] = row[j] >= 0 ? a.weights[t * a.k + j0 + j] : 0.f;
      dot[j] = 0.f;
    }
    for (int64_t c = (int64_t)(threadIdx.x % (WPT * kWave)) * VEC; c < a.width; c += WPT * kWave * VEC) {
      Held<WD, VEC> g, y[J];
      g.load(a.x, t * a.ldx + c);
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (a.rows > 0) y[j].load(a.y, (int64_t)(row[j] < 0 ? 0 : row[j]) * a.ldy + c);
      float fg[VEC];
      g.get(fg);
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (row[j] < 0) continue;
        float fy[VEC];
        y[j].get(fy);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          dot[j] = fmaf(fg[i], fy[i], dot[j]);
          fy[i] = w[j] * fg[i];
        }
        st_vec<WD, VEC>(a.out, (int64_t)row[j] * a.ldo + c, fy);
      }
    }
    float sum = four_sums(dot);
    if constexpr (WPT > 1) {
      if (lane < J) part[wave][lane] = sum;
      __syncthreads();
      sum = (part[0][lane % J] + part[1][lane % J]) + (part[2][lane % J] + part[3][lane % J]);
      __syncthreads();
    }
    if ((WPT == 1 || wave == 0) && lane < J && j0 + lane < a.k)
      a.grad_weights[t * a.k + j0 + lane] = sum;
  }
}

dim3 wave_grid(int64_t units) { return dim3((uint32_t)cdiv(units, kWaves)); }

template <typename U>
hipError_t run_dispatch(const ExpertRowArgs& a, int es, hipStream_t s) {
  const int64_t per = (int64_t)sizeof(U) / es, clear = cdiv(a.rows, kClearRows);
  const int64_t parts = cdiv(a.width / per, kLoads<sizeof(U) == 16> * kWave);
  const int64_t units = a.tokens * parts;
  if (!fits_grid(cdiv(clear + units, kWaves))) return hipErrorInvalidConfiguration;
  TBE_LAUNCH("expert_dispatch", (dispatch_kernel<U>), wave_grid(clear + units), dim3(kThreads), s,
             a, (uint32_t)clear, (uint32_t)units, (uint32_t)parts, a.width / per, a.ldx / per,
             a.ldo / per);
  return hipGetLastError();
}

bool rows16(const void* p, int64_t ld, int es) { return aligned16(p) && (ld * es) % 16 == 0; }

template <int WD, int VEC>
hipError_t run_combine(const ExpertRowArgs& a, bool backward, hipStream_t s) {
  if (backward) {
    // A wave a token where its columns take two steps at most: the four waves' meeting
    // costs more than it saves.  (16384 tokens, four choices, a wave each / a workgroup
    // each: 256 bfloat16 columns 20.7 / 40.9 us, 1024 51.4 / 57.6, 2048 99.5 / 94.8;
    // 2048 tokens of 2048 columns 22.0 / 19.7.)
    const int64_t clear = cdiv(cdiv(a.rows, kClearRows), kWaves);
    const bool one = a.width <= 2 * kWave * VEC;
    const int64_t wgs = clear + (one ? cdiv(a.tokens, kWaves) : a.tokens);
    if (!fits_grid(wgs)) return hipErrorInvalidConfiguration;
    if (one)
      TBE_LAUNCH("expert_combine_backward", (combine_backward_kernel<WD, VEC, 1>),
                 dim3((uint32_t)wgs), dim3(kThreads), s, a, (uint32_t)clear);
    else
      TBE_LAUNCH("expert_combine_backward", (combine_backward_kernel<WD, VEC, kWaves>),
                 dim3((uint32_t)wgs), dim3(kThreads), s, a, (uint32_t)clear);
  } else {
    const int64_t parts = cdiv(a.width, kLoads<(VEC > 1)> * kWave * VEC);
    const int64_t units = a.tokens * parts;
    if (!fits_grid(cdiv(units, kWaves))) return hipErrorInvalidConfiguration;
    TBE_LAUNCH("expert_combine", (combine_kernel<WD, VEC>), wave_grid(units), dim3(kThreads), s, a,
               (uint32_t)units, (uint32_t)parts);
  }
  return hipGetLastError();
}

template <int WD>
hipError_t combine_any(const ExpertRowArgs& a, bool backward, hipStream_t s) {
  constexpr int es = WD == WD_F32 ? 4 : 2;
  bool vec = (a.width * es) % 16 == 0 && rows16(a.y, a.ldy, es) && rows16(a.out, a.ldo, es);
  if (backward) vec = vec && rows16(a.x, a.ldx, es);
  return vec ? run_combine<WD, kVec16<WD>>(a, backward, s) : run_combine<WD, 1>(a, backward, s);
}

hipError_t combine_type(const ExpertRowArgs& a, bool backward, hipStream_t s) {
  switch (a.dtype) {
    case WD_F32: return combine_any<WD_F32>(a, backward, s);
    case WD_F16: return combine_any<WD_F16>(a, backward, s);
    default: return combine_any<WD_BF16>(a, backward, s);
  }
}

bool sort_one(int64_t n, int64_t rows) { return n <= kSortOneIds && rows <= kSortOneRows; }

uint32_t sort_tiles(int64_t n) { return (uint32_t)cdiv(n, kSortTile); }

template <typename IT>
hipError_t run_sort(const ExpertSortArgs& a, hipStream_t s) {
  if (sort_one(a.n, a.rows)) {
    if (a.n <= kOneThreads)
      TBE_LAUNCH("expert_sort", (expert_sort_one_kernel<IT, 1>), dim3(1), dim3(kOneThreads), s, a);
    else
      TBE_LAUNCH("expert_sort", (expert_sort_one_kernel<IT, kOneRounds>), dim3(1),
                 dim3(kOneThreads), s, a);
    return hipGetLastError();
  }
  const uint32_t tiles = sort_tiles(a.n), E = (uint32_t)a.experts;
  uint32_t* total = a.ws;
  uint32_t* cnt = a.ws + up_to(E, 64);
  const uint32_t clears = (uint32_t)std::min<int64_t>(256, cdiv(a.rows, kSortTile));
  if (tiles)
    TBE_LAUNCH("expert_count", (expert_count_kernel<IT>), dim3(tiles), dim3(kThreads), s, a.ids,
               a.n, E, cnt);
  TBE_LAUNCH("expert_prefix", expert_prefix_kernel, dim3(E), dim3(kThreads), s, cnt, tiles, E,
             total);
  TBE_LAUNCH("expert_place", (expert_place_kernel<IT>), dim3(std::max(1u, tiles + clears)),
             dim3(kThreads), s, a, tiles, (const uint32_t*)cnt, (const uint32_t*)total);
  return hipGetLastError();
}

}  // namespace

size_t expert_sort_ws(int64_t n, int32_t experts, int64_t rows) {
  if (sort_one(n, rows)) return 0;
  return (size_t)up_to((up_to(experts, 64) + (int64_t)sort_tiles(n) * experts) * 4,
                       (int64_t)kWsAlign);
}

hipError_t launch_expert_sort(const ExpertSortArgs& a, hipStream_t s) {
  return a.itype == IT_I32 ? run_sort<int32_t>(a, s) : run_sort<int64_t>(a, s);
}

hipError_t launch_expert_dispatch(const ExpertRowArgs& a, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  const int es = a.dtype == WD_F32 ? 4 : 2;
  if ((a.width * es) % 16 == 0 && rows16(a.x, a.ldx, es) && rows16(a.out, a.ldo, es))
    return run_dispatch<u32x4_t>(a, es, s);
  return es == 4 ? run_dispatch<uint32_t>(a, es, s) : run_dispatch<uint16_t>(a, es, s);
}

hipError_t launch_expert_combine(const ExpertRowArgs& a, hipStream_t s) {
  if (a.tokens == 0) return hipSuccess;
  ExpertRowArgs b = a;
  if (a.rows == 0) b.k = 0;  // no row to read: zeros
  return combine_type(b, false, s);
}

hipError_t launch_expert_combine_backward(const ExpertRowArgs& a, hipStream_t s) {
  if (a.rows == 0 && a.tokens == 0) return hipSuccess;
  return combine_type(a, true, s);
}

}  // namespace tbe
