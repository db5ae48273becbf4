// Matrix products of 8-bit block-scaled operands over experts, on the matrix
// cores.
//
//   matmul_f8   out[m, n] = sum_b 2^(sa[m,b] + sb[n,b]) sum_{c in b} a[m, c] w_e[n, c]
//   segments    out[e][i, j] = the same over the blocks b of segment e of a[i, .], b[j, .]
//
// v_mfma_scale_f32_32x32x64_f8f6f4 multiplies 32 rows by 32 columns over 64
// contraction elements, half a block, and takes each operand row's scale byte
// itself, so the blocks' scales cost nothing beside the product.  The weights
// are the instruction's first operand: a lane then holds four neighbouring n
// of one row m, which it stores together.
//
// Sums are float32.  The instruction cuts each product of eight neighbours toward
// zero at 2^-13 of the power of two of their largest, and rounds the sum once in
// sixteen products (both found by single terms beside known ones): the bound that
// the header states.
//
// What bounds it, measured:
//   large products are bound by the matrix cores.  65536 rows of 16 experts of
//     4096 x 2048: 500 us, 2.2 PFLOP/s, of it 57% of the matrix cores' cycles;
//     the rest is the results' way out (16 steps, then 128 KB of results a tile)
//     and waits for operands.  8192 x 8192 over 2048: 134 us, over 8192: 440 us,
//     2.5 PFLOP/s.  The clock falls under this load, so that variants of fewer
//     cycles and more LDS or L2 traffic came out slower.
//   few rows an expert are bound by reading the weights.  24 rows of those
//     experts: 22 us, 106 MB at 4.8 TB/s.
//   small products are bound by the chain of loads of one tile: 1001 x 1100 over
//     1000: 10 us.
#include "experts_common.h"

namespace tbe {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr int kBK = kF8Block;

__device__ __forceinline__ int64_t clamp_row(int32_t r, int64_t rows) {
  return r < 0 ? 0 : ((int64_t)r > rows ? rows : (int64_t)r);
}

// Row tiles of `bm` rows that do not cross stretches: `start` holds 0, the E + 1
// segment starts and the end of all rows, so that stretch 0 and stretch E + 1 are
// the rows of no segment.  Every wave finds tile `idx` by a prefix of the
// stretches' tile counts across its lanes; *tiles is their number when idx < 0.
__device__ __forceinline__ void find_tile(const int32_t* start, int32_t E, int bm, int32_t idx,
                                          int32_t* e, int64_t* row0, int64_t* hi, int32_t* tiles) {
  const int lane = threadIdx.x % kWave;
  int32_t run = 0;
  for (int32_t e0 = 0; e0 <= E + 1; e0 += kWave) {
    const int32_t q = e0 + lane;
    const int32_t lo = q <= E + 1 ? start[q] : 0, up = q <= E + 1 ? start[q + 1] : 0;
    const int32_t t = up > lo ? (up - lo - 1) / bm + 1 : 0;  // up - lo may be all of 31 bits
    int32_t x = t;
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1) {
      const int32_t o = __shfl_up(x, m, kWave);
      x += lane >= m ? o : 0;
    }
    const uint64_t past = __ballot(idx >= 0 && run + x > idx);
    if (past) {
      const int l = __builtin_ctzll(past);
      *e = e0 + l;
      *row0 = __builtin_amdgcn_readlane(lo, l) +
              (int64_t)(idx - run - __builtin_amdgcn_readlane(x - t, l)) * bm;
      *hi = __builtin_amdgcn_readlane(up, l);
      return;
    }
    run += __builtin_amdgcn_readlane(x, kWave - 1);
  }
  *tiles = run;
}

// The value of lane 0, in scalar registers: what every lane holds alike.
__device__ __forceinline__ int64_t uniform(int64_t x) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)x);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)x >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
template <int WD>
__device__ __forceinline__ uint32_t pack2(float a, float b) {  // one rounding, to nearest even
  if constexpr (WD == WD_F16) return __builtin_bit_cast(uint32_t, (f16x2_t){(_Float16)a, (_Float16)b});
  return __builtin_bit_cast(uint32_t, (bf16x2_t){(__bf16)a, (__bf16)b});
}

// A sum of the 256-row tile, from the accumulation registers that it fills (read
// one by one: taken over together they would not fit beside the rest).
template <bool ACC>
__device__ __forceinline__ float sum_at(float v) {
  if constexpr (ACC) {
    float f;
    asm("v_accvgpr_read_b32 %0, %1" : "=v"(f) : "a"(v));
    return f;
  }
  return v;
}

// A tile of 64 WM rows m by 64 WN rows n; four waves, two by two, each WM x WN
// products of 32 x 32.  An LDS stage holds 128 contraction bytes of every row, and
// a word of four scale bytes of every row.  A row's eight 16-byte
// pieces are stored at piece ^ swz(row), which spreads the sixteen rows that a
// read touches over all banks.
template <int WM, int WN>
struct Tile {
  static constexpr int TM = 64 * WM, TN = 64 * WN, ROWS = TM + TN;
  static constexpr int BYTES = ROWS * kBK + ROWS * 4;  // a stage: m rows, n rows, scale words
  // Workgroups that share a CU: what its 160 KB of LDS hold.  (24 rows of 16
  // experts of 4096 x 2048 by the smallest tile: two of two stages 31 us, two of
  // four stages 25.6, four of two stages 22.1: bound by reading the weights.)
  static constexpr int STAGES = 2, PER_CU = WM >= 4 ? 1 : WM >= 2 ? 2 : 4;
};

__device__ __forceinline__ int swz(int row) { return (row & 6) | ((row ^ (row >> 3)) & 1); }

// 64 lanes x 16 (or 4) bytes from a buffer straight into LDS: lane l's bytes
// at off + at land at LDS address lds + 16 l (4 l).  A buffer of no bytes gives
// zeros.  Written as instructions because the compiler would wait for every such
// load before the next LDS read, of whichever stage; meet() holds the waits.
// There is no output register: what they write is LDS.  (m0 is reserved: the
// compiler sets it before each use of its own.)
typedef __attribute__((address_space(3))) void lds_void_t;
typedef int i32x4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ i32x4_t bytes_at(const uint8_t* p, uint32_t bytes) {
  const uint64_t a = (uint64_t)(uintptr_t)p;
  return (i32x4_t){(int)(uint32_t)a, (int)((uint32_t)(a >> 32) & 0xffffu), (int)bytes, kBufDword3};
}
__device__ __forceinline__ void to_lds16(i32x4_t b, uint32_t off, uint32_t at, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               ::"s"(lds), "v"(off), "s"(b), "s"(at) : "memory");
}
__device__ __forceinline__ void to_lds4(i32x4_t b, uint32_t off, uint32_t at, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
               ::"s"(lds), "v"(off), "s"(b), "s"(at) : "memory");
}

// The workgroup meets when each of its waves has at most N loads under way and
// (READ) its LDS reads are done.
template <int N, bool READ = true>
__device__ __forceinline__ void meet() {
  __builtin_amdgcn_sched_barrier(0);
  if (READ) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
  else asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Row `row` of a tile, or its last one: rows past the end are read as that one
// and their results not stored.
__device__ __forceinline__ uint32_t row_at(int row, uint32_t rows) {
  return (uint32_t)row < rows ? (uint32_t)row : rows - 1;
}

// SEG: the contraction runs over segment e's blocks and out is [E][m][n];
// otherwise the rows are tiled by segment and the contraction is all of k.
//
// Workgroups stay for several tiles.  Workgroups of one XCD (blockIdx mod 8, the
// order in which they are given out) take one stretch of the tiles, kBand row
// tiles by all n at a time, so that its L2 holds the operands they share.
//
// The fragments of a step are in registers when it begins.  Its products run
// row by row of n; after row 0 the workgroup meets (the next block has landed,
// every wave has read this one), and each fragment is replaced by the next
// block's as soon as its last product is issued.  The first two blocks of the
// next tile are sent for before this tile's results are stored.
constexpr int kXcds = 8, kBand = 4;
template <int WD, bool SEG, bool SQ, int WM, int WN>
__global__ __launch_bounds__(kThreads, (Tile<WM, WN>::PER_CU)) void matmul_f8_kernel(
    MatmulF8Args g, uint32_t ntiles, uint32_t mtiles, bool vec) {
  using T = Tile<WM, WN>;
  __shared__ __attribute__((aligned(1024))) uint8_t stage[T::STAGES * T::BYTES];
  __shared__ int32_t start[SEG ? 1 : kMaxExperts + 3];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) & 3;
  const int r = lane % 32, h = lane / 32;
  const uint32_t k = (uint32_t)g.k, lds = (uint32_t)g.lds;
  int32_t total = 0;  // row tiles of all segments
  if (SEG) {
  } else if (!g.offsets) {
    total = (int32_t)mtiles;
  } else {
    for (int32_t q = threadIdx.x; q <= g.experts; q += kThreads)
      start[q + 1] = (int32_t)clamp_row(g.offsets[q], g.m);
    if (threadIdx.x == 0) start[0] = 0, start[g.experts + 2] = (int32_t)g.m;
    __syncthreads();
    int32_t e;
    int64_t a, b;
    find_tile(start, g.experts, T::TM, -1, &e, &a, &b, &total);
    total = __builtin_amdgcn_readfirstlane(total);
  }
  // places: bands of kBand row tiles by all n, some of the last band empty
  const uint32_t band_places = kBand * ntiles;
  // (segments: band b of every expert in turn, so that a stretch has many experts'
  // lengths in it)
  const uint32_t seg_bands = (mtiles + kBand - 1) / kBand;
  const uint32_t all = (SEG ? seg_bands * (uint32_t)g.experts : (uint32_t)(total + kBand - 1) / kBand) *
                       band_places;
  // this XCD's stretch, and this workgroup's first place in it
  const uint32_t xcd = blockIdx.x % kXcds, per = (all + kXcds - 1) / kXcds;
  const uint32_t last = (xcd + 1) * per < all ? (xcd + 1) * per : all;
  const uint32_t stride = (gridDim.x + kXcds - 1 - xcd) / kXcds;
  uint32_t place = xcd * per + blockIdx.x / kXcds;

  // the tile at hand
  int32_t e = 0, kb0 = 0, kb1 = 0;
  int64_t row0 = 0, hi = 0, n0 = 0;
  const uint8_t *va = nullptr, *vb = nullptr, *sa = nullptr, *sb = nullptr;
  uint32_t rows_a = 1, rows_b = 1;
  // a load takes eight rows, lane / 8, pieces lane % 8 (or 64 rows' scale words)
  const int lrow = wave * 8 + lane / 8;
  const uint32_t lpiece = (uint32_t)(((lane % 8) ^ swz(lrow)) * 16);
  uint32_t off_a[2 * WM], off_b[2 * WN], soff_a[(WM + 3) / 4], soff_b[(WN + 3) / 4];
  // the next place that holds a tile; false when there is none
  const auto next_tile = [&]() __attribute__((always_inline)) {
    for (; place < last; place += stride) {
      const uint32_t band = place / band_places, in = place - band * band_places;
      const int32_t mt = (int32_t)((SEG ? band / (uint32_t)g.experts : band) * kBand + in % kBand);
      if (mt >= (SEG ? (int32_t)mtiles : total)) continue;
      n0 = (int64_t)(in / kBand) * T::TN;
      kb0 = 0;
      kb1 = (int32_t)(g.k / kBK);  // blocks of the contraction
      if constexpr (SEG) {
        e = (int32_t)(band % (uint32_t)g.experts);
        row0 = (int64_t)mt * T::TM;
        hi = g.m;
        kb0 = (int32_t)(clamp_row(g.offsets[e], g.k) / kBK);
        kb1 = (int32_t)((clamp_row(g.offsets[e + 1], g.k) + kBK - 1) / kBK);
        kb0 = __builtin_amdgcn_readfirstlane(kb0);
        kb1 = __builtin_amdgcn_readfirstlane(kb1);
      } else if (!g.offsets) {
        row0 = (int64_t)mt * T::TM;
        hi = g.m;
      } else {
        int32_t none;
        find_tile(start, g.experts, T::TM, mt, &e, &row0, &hi, &none);
        e = __builtin_amdgcn_readfirstlane(e) - 1;
        row0 = uniform(row0);
        hi = uniform(hi);
        if ((uint32_t)e >= (uint32_t)g.experts) kb1 = e = 0;  // rows of no segment: zeros
      }
      const int64_t eb = SEG ? 0 : e;
      va = reinterpret_cast<const uint8_t*>(uniform((int64_t)(g.a + row0 * g.k)));
      sa = reinterpret_cast<const uint8_t*>(uniform((int64_t)(g.sa + row0 * g.lds)));
      vb = reinterpret_cast<const uint8_t*>(uniform((int64_t)(g.b + (eb * g.n + n0) * g.k)));
      sb = reinterpret_cast<const uint8_t*>(uniform((int64_t)(
          g.sb + (SQ ? eb * ((g.n + kBK - 1) / kBK) + n0 / kBK : eb * g.n + n0) * g.lds)));
      rows_a = (uint32_t)uniform(hi - row0 < T::TM ? hi - row0 : T::TM);
      rows_b = (uint32_t)uniform(g.n - n0 < T::TN ? g.n - n0 : T::TN);
#pragma unroll
      for (int i = 0; i < 2 * WM; ++i) off_a[i] = row_at(i * 32 + lrow, rows_a) * k + lpiece;
#pragma unroll
      for (int i = 0; i < 2 * WN; ++i) off_b[i] = row_at(i * 32 + lrow, rows_b) * k + lpiece;
#pragma unroll
      for (int i = 0; i < (WM + 3) / 4; ++i)
        soff_a[i] = row_at((i * 4 + wave) * 64 % T::TM + lane, rows_a) * lds;
#pragma unroll
      for (int i = 0; i < (WN + 3) / 4; ++i) {
        const uint32_t row = row_at((i * 4 + wave) * 64 % T::TN + lane, rows_b);
        soff_b[i] = (SQ ? row / kBK : row) * lds;
      }
      place += stride;
      return true;
    }
    return false;
  };
  const uint32_t base = (uint32_t)(uintptr_t)(lds_void_t*)stage;  // LDS address
  // Load x of the LOADS that a wave sends for block kb: n rows, scale words, then
  // m rows.  Past the last block the buffers have no bytes, so that a step has no
  // branch around it.
  constexpr int SCALES = (WM + 3) / 4 + (WN + 3) / 4, FIRST = 2 * WN + SCALES, LOADS = FIRST + 2 * WM;
  const auto send = [&](int x, int32_t kb, uint32_t st) __attribute__((always_inline)) {
    const bool on = kb < kb1;
    const uint32_t at = on ? (uint32_t)kb * kBK : 0u, sat = on ? (uint32_t)kb & ~3u : 0u;
    st += base;
    const uint32_t sc = st + T::ROWS * kBK;
    if (x < 2 * WN) {
      to_lds16(bytes_at(vb, on ? rows_b * k : 0u), off_b[x], at,
               st + (T::TM + x * 32 + wave * 8) * kBK);
    } else if (x < 2 * WN + (WN + 3) / 4) {  // fewer than 256 rows: waves bring the same words
      const int i = x - 2 * WN;
      to_lds4(bytes_at(sb, on ? rows_b * lds : 0u), soff_b[i], sat,
              sc + (T::TM + ((i * 4 + wave) * 64) % T::TN) * 4);
    } else if (x < FIRST) {
      const int i = x - 2 * WN - (WN + 3) / 4;
      to_lds4(bytes_at(sa, on ? rows_a * lds : 0u), soff_a[i], sat,
              sc + ((i * 4 + wave) * 64) % T::TM * 4);
    } else {
      const int i = x - FIRST;
      to_lds16(bytes_at(va, on ? rows_a * k : 0u), off_a[i], at, st + (i * 32 + wave * 8) * kBK);
    }
  };
  // Fragments of 32 rows: lane (r, h) holds pieces h, h + 2 of its row for the
  // block's first product and h + 4, h + 6 for the second; both operands do, and
  // a block has one scale, so the order inside it does not matter.
  const int wm = (wave >> 1) * 32 * WM, wn = (wave & 1) * 32 * WN;
  i32x8_t fm[WM][2], fn[WN][2];
  int cm[WM], cn[WN];
  // A stage's addresses in LDS: four piece addresses of the lane's first m row and
  // of its first n row, and its first scale words; further fragments lie at
  // constant distances.  (Kept from being spread into one register a fragment.)
  struct At {
    uint32_t m[4], n[4], sm, sn;
  };
  const uint32_t lane_at = (uint32_t)(r * kBK + (h ^ swz(r)) * 16);
  const auto at_stage = [&](uint32_t st) __attribute__((always_inline)) {
    At a;
    const uint32_t m = base + st + (uint32_t)wm * kBK + lane_at;
    const uint32_t n = base + st + (uint32_t)(T::TM + wn) * kBK + lane_at;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      a.m[p] = m ^ (uint32_t)(p * 32);
      a.n[p] = n ^ (uint32_t)(p * 32);
      asm volatile("" : "+v"(a.m[p]), "+v"(a.n[p]));
    }
    a.sm = base + st + (uint32_t)(T::ROWS * kBK + (wm + r) * 4);
    a.sn = base + st + (uint32_t)(T::ROWS * kBK + (T::TM + wn + r) * 4);
    asm volatile("" : "+v"(a.sm), "+v"(a.sn));
    return a;
  };
  typedef __attribute__((address_space(3))) const u32x4_t lds_u32x4_t;
  typedef __attribute__((address_space(3))) const int lds_int_t;
  const auto frag = [&](const uint32_t* a, int t, i32x8_t* f) __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const u32x4_t lo = *(lds_u32x4_t*)(uintptr_t)(a[2 * p] + t * 32 * kBK);
      const u32x4_t up = *(lds_u32x4_t*)(uintptr_t)(a[2 * p + 1] + t * 32 * kBK);
      f[p] = (i32x8_t){(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w,
                       (int)up.x, (int)up.y, (int)up.z, (int)up.w};
    }
  };
  const auto read_m = [&](const At& a, int t) __attribute__((always_inline)) {
    frag(a.m, t, fm[t]);
    cm[t] = *(lds_int_t*)(uintptr_t)(a.sm + t * 32 * 4);
  };
  const auto read_n = [&](const At& a, int t) __attribute__((always_inline)) {
    frag(a.n, t, fn[t]);
    cn[t] = *(lds_int_t*)(uintptr_t)(a.sn + t * 32 * 4);
  };
  f32x16_t acc[WN][WM];
  // Products of block kb (in registers), fragments of kb + 1 from the stage at
  // `other`, loads of kb + STAGES into the one at `cur`: one after each product
  // from row 1 on, the rate at which they are taken.  A wave's loads complete in
  // order.
  constexpr bool TWO = WN > 2;  // a second meeting before the last row, for the m rows
  constexpr int SLOTS = WN > 1 ? (WN - 1) * WM * 2 : 1;
  const auto step = [&](int32_t kb, uint32_t cur, uint32_t other) __attribute__((always_inline)) {
    const int sh = (kb & 3) * 8;  // this block's byte of the scale words
    const At next = at_stage(other);
#pragma unroll
    for (int i = 0; i < WN; ++i) {
      if (TWO && i == WN - 1) {
        // what this step has sent so far may be under way
        meet<(WN - 2) * WM * 2 < LOADS ? (WN - 2) * WM * 2 : LOADS, false>();
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
#pragma unroll
        for (int j = 0; j < WM; ++j) {
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              fn[i][q], fm[j][q], acc[i][j], 0, 0, 0, cn[i] >> sh, 0, cm[j] >> sh);
          if (i > 0) {
            const int slot = ((i - 1) * 2 + q) * WM + j;
#pragma unroll
            for (int x = 0; x < LOADS; ++x)
              if (TWO ? x == slot : x >= slot * LOADS / SLOTS && x < (slot + 1) * LOADS / SLOTS)
                send(x, kb + T::STAGES, cur);
            __builtin_amdgcn_sched_barrier(0);
          }
          if (WN > 1 && i == WN - 1 && q == 1) {
            read_m(next, j);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
      if (i == 0) {
        __builtin_amdgcn_sched_barrier(0);
        meet<TWO ? 2 * WM : (T::STAGES - 2) * LOADS>();  // the next block's n rows and scales have landed
        if (WN == 1) {
#pragma unroll
          for (int x = 0; x < LOADS; ++x) send(x, kb + T::STAGES, cur);
#pragma unroll
          for (int j = 0; j < WM; ++j) read_m(next, j);
        }
      }
      read_n(next, i);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  const auto send_first = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < T::STAGES; ++t)
#pragma unroll
      for (int x = 0; x < LOADS; ++x) send(x, kb0 + t, t * T::BYTES);
  };
  // Results go through LDS: memory of its own where the next tile's first blocks
  // are under way meanwhile, the stages where more workgroups share a CU.
  constexpr bool EARLY = WM >= 4;
  constexpr int CH = WN < 2 ? WN : 2, PITCH = CH * 64 + 16, STORES = 2 * WM * WN;
  __shared__ __attribute__((aligned(16))) uint8_t results[EARLY ? 4 * 32 * PITCH : 16];
  uint8_t* const tr = (EARLY ? results : stage) + wave * 32 * PITCH;
  if (!next_tile()) return;
  send_first();
  meet<(T::STAGES - 1) * LOADS>();
  for (;;) {
#pragma unroll
    for (int t = 0; t < WM; ++t) read_m(at_stage(0), t);
#pragma unroll
    for (int t = 0; t < WN; ++t) read_n(at_stage(0), t);
    // the last step reads a stage that nothing was loaded into, and uses none of it
    uint32_t at = 0;
#pragma unroll
    for (int i = 0; i < WN; ++i)
#pragma unroll
      for (int j = 0; j < WM; ++j) acc[i][j] = (f32x16_t)(0.f);
    for (int32_t kb = kb0; kb < kb1; ++kb) {
      const uint32_t next = at + T::BYTES < T::STAGES * T::BYTES ? at + T::BYTES : 0;
      step(kb, at, next);
      at = next;
    }
    // Both stages are free.  sum_at() reads accumulation registers by instructions of
    // its own: the last product has long written them (it takes 64 cycles).
    if (EARLY) asm volatile("s_nop 15\n\ts_nop 15\n\ts_nop 15");
    meet<0>();
    const int64_t m0 = row0 + wm, c0 = n0 + wn, end = hi;
    uint16_t* out = reinterpret_cast<uint16_t*>(g.out) + (SEG ? (int64_t)e * g.m * g.ldo : 0);
    const bool full = vec && rows_a == T::TM && rows_b == T::TN;
    bool more = false;
    if (EARLY) {
      more = next_tile();
      if (more) send_first();
    }
    // 32 rows by 32 CH columns at a time through LDS: a lane has four neighbouring
    // n of one row (eight apart), and stores eight of a row beside its neighbours'.
    // The next piece is rounded while this one's reads are under way.
    constexpr int PIECES = WM * WN / CH;
    uint2 rounded[4 * CH];
    const auto round = [&](int x) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const f32x16_t& v = acc[x % (WN / CH) * CH + i][x / (WN / CH)];
          float f[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) f[y] = sum_at<EARLY>(v[4 * p + y]);
          rounded[i * 4 + p] = make_uint2(pack2<WD>(f[0], f[1]), pack2<WD>(f[2], f[3]));
        }
    };
    round(0);
#pragma unroll
    for (int x = 0; x < PIECES; ++x) {
#pragma unroll
      for (int i = 0; i < 4 * CH; ++i)
        *reinterpret_cast<uint2*>(tr + r * PITCH + (i * 8 + h * 4) * 2) = rounded[i];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      u32x4_t v[2 * CH];
#pragma unroll
      for (int w = 0; w < 2 * CH; ++w)
        v[w] = *reinterpret_cast<const u32x4_t*>(
            tr + (w * (16 / CH) + lane / (4 * CH)) * PITCH + lane % (4 * CH) * 16);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (x + 1 < PIECES) round(x + 1);
      const int64_t n = c0 + x % (WN / CH) * CH * 32 + lane % (4 * CH) * 8;
#pragma unroll
      for (int w = 0; w < 2 * CH; ++w) {
        const int64_t m = m0 + x / (WN / CH) * 32 + w * (16 / CH) + lane / (4 * CH);
        uint16_t* o = out + m * g.ldo + n;
        if (full) {
          st16<true>(o, v[w]);  // the results are not read here: they do not push out the operands
        } else if (m < end) {
          if (vec && n + 8 <= g.n) {
            *reinterpret_cast<u32x4_t*>(o) = v[w];
          } else {
#pragma unroll
            for (int y = 0; y < 8; ++y)
              if (n + y < g.n) o[y] = (uint16_t)(v[w][y / 2] >> (y % 2 * 16));
          }
        }
      }
    }
    if (EARLY) {
      if (!more) return;
      if (full) meet<(LOADS + STORES < 63 ? LOADS + STORES : 63)>();
      else meet<(T::STAGES - 1) * LOADS>();
    } else {
      if (!next_tile()) return;
      meet<63>();  // every wave has read its part of the stages
      send_first();
      meet<(T::STAGES - 1) * LOADS>();
    }
  }
}

template <bool SEG, bool SQ, int WM, int WN>
hipError_t run(const MatmulF8Args& g, hipStream_t s) {
  using T = Tile<WM, WN>;
  const uint32_t ntiles = (uint32_t)cdiv(g.n, T::TN), mtiles = (uint32_t)cdiv(g.m, T::TM);
  // at most so many row tiles: every segment may end in a part of one
  const int64_t most = SEG ? up_to(mtiles, kBand) * g.experts
                           : g.offsets ? g.m / T::TM + g.experts + 2 : mtiles;
  const bool vec = aligned16(g.out) && g.ldo % 8 == 0 && (!SEG || (g.m * g.ldo) % 8 == 0);
  const int64_t places = up_to(most, kBand) * ntiles;
  const int64_t resident = 256 * T::PER_CU;  // workgroups that fit the chip
  const dim3 grid((uint32_t)(places < resident ? places : resident));
  const char* name = SEG ? "matmul_f8_segments" : "matmul_f8";
  if (g.dtype == WD_F16)
    TBE_LAUNCH(name, (matmul_f8_kernel<WD_F16, SEG, SQ, WM, WN>), grid, dim3(kThreads), s, g, ntiles,
               mtiles, vec);
  else
    TBE_LAUNCH(name, (matmul_f8_kernel<WD_BF16, SEG, SQ, WM, WN>), grid, dim3(kThreads), s, g, ntiles,
               mtiles, vec);
  return hipGetLastError();
}

// Tile by the number of tiles: the largest that still gives a workgroup to more
// than half of the chip's 256 CUs.  Below that a smaller tile is done sooner: its
// step is shorter and more CUs share the work.  Times of one product over 2048 by
// tile 64 / 128 / 256, with the numbers of 128- and 256-row tiles:
//   1024 x 1536  (96, 24)    10.3 / 11.4 / 24.3 us
//   2048 x 1280 (160, 40)    14.2 / 11.9 / 24.4
//   2048 x 4096 (512, 128)   36.8 / 20.3 / 27.0
//   4096 x 2560 (640, 160)   45.1 / 31.6 / 26.4
// The tiles are counted as if all rows were one segment.  With experts the rows of
// a tile that its segment does not fill are loaded and multiplied all the same, but
// such products are bound by reading the weights.  4096 columns over 2048, rows an
// expert (mean), by tile 64 / 128 / 256, the rule's own marked:
//   16 experts,  32 rows   25.5* / 25.5 / 32.8 us    256 rows   88.9 / 55.0 / 61.8*
//   64 experts,   2 rows   88.2* / 95.6 / 124.1       64 rows    154 / 126 / 149*
//   256 experts,  8 rows    409 / 405* / 513          32 rows    493 / 463 / 531*
//   256 experts, 64 rows    630 / 509 / 552*         256 rows   1545 / 973 / 820*
// so the 256-row tile, taken for rows that many short segments share, costs up to a
// fifth there.
constexpr int64_t kFewTiles = 144;
template <bool SEG, bool SQ>
hipError_t by_size(const MatmulF8Args& g, hipStream_t s) {
  const int64_t groups = SEG ? g.experts : 1;
  if (cdiv(g.m, 256) * cdiv(g.n, 256) * groups >= kFewTiles) return run<SEG, SQ, 4, 4>(g, s);
  if (cdiv(g.m, 128) * cdiv(g.n, 128) * groups >= kFewTiles) return run<SEG, SQ, 2, 2>(g, s);
  return run<SEG, SQ, 1, 1>(g, s);
}

}  // namespace

hipError_t launch_matmul_f8(const MatmulF8Args& g, hipStream_t s) {
  if (g.m == 0 || g.n == 0) return hipSuccess;
  return g.square ? by_size<false, true>(g, s) : by_size<false, false>(g, s);
}
hipError_t launch_matmul_f8_segments(const MatmulF8Args& g, hipStream_t s) {
  if (g.m == 0 || g.n == 0 || g.experts == 0) return hipSuccess;
  return by_size<true, false>(g, s);
}

}  // namespace tbe
