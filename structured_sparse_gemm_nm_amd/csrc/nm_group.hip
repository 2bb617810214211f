// Products of packed N:M weights grouped by expert: Y[t] = W_e act[t] for the rows
// t of expert e, rows ordered by expert (nm_group.h).  Operand layouts and the
// widening of 1:4 and 1:8 rows to the 2:4 operand are those of nm_spmm.hip.
#include "nm_group.h"

#include "nm_internal.h"
#include "nm_widen.h"

#include <algorithm>
#include <type_traits>

namespace nm {
namespace {

// ---------------------------------------------------------------------------
// The table of token tiles (nm_group.h), by one workgroup: a prefix sum of the
// experts' tile counts, 1024 experts at a time, then every thread looks up the
// expert of its share of the tiles.
// ---------------------------------------------------------------------------
constexpr int kTableThreads = 1024;

__global__ __launch_bounds__(kTableThreads) void group_tiles_kernel(const int32_t* __restrict__ offsets, int E, int T,
                                                                    int BT, int max_tiles, int4* __restrict__ table) {
  __shared__ int start[kTableThreads + 1], first[kTableThreads], last[kTableThreads], wsum[kTableThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int before = 0;
  for (int e0 = 0; e0 < E; e0 += kTableThreads) {
    int lo = 0, hi = 0;
    if (e0 + tid < E) group_range(offsets, e0 + tid, T, lo, hi);
    const int tiles = (hi - lo + BT - 1) / BT;
    int sum = tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int up = __shfl_up(sum, o, 64);
      if (lane >= o) sum = tile_sum(sum, up);
    }
    if (lane == 63) wsum[wave] = sum;
    first[tid] = lo;
    last[tid] = hi;
    __syncthreads();
    int base = before;
    for (int w = 0; w < wave; ++w) base = tile_sum(base, wsum[w]);
    const int up = __shfl_up(sum, 1, 64);
    start[tid] = tile_sum(base, lane > 0 ? up : 0);
    if (tid == kTableThreads - 1) start[kTableThreads] = tile_sum(base, sum);
    __syncthreads();
    const int end = min(start[kTableThreads], max_tiles);
    for (int i = before + tid; i < end; i += kTableThreads) {
      int a = 0, b = kTableThreads;   // the last expert that starts at or before tile i
      while (b - a > 1) {
        const int m = (a + b) >> 1;
        if (start[m] <= i) a = m;
        else b = m;
      }
      table[1 + i] = make_int4(e0 + a, first[a] + (i - start[a]) * BT, last[a], 0);
    }
    before = start[kTableThreads];
    __syncthreads();
  }
  if (tid == 0) table[0] = make_int4(min(before, max_tiles), 0, 0, 0);
}

struct GroupDims {
  int E, R, K, T, words, tilesR;
  int64_t ldx, ldy;
  int share = 0;            // steps of K a workgroup takes (0: all), parts part_stride apart
  int64_t part_stride = 0;
};

template <int DT, int OUT>
__device__ inline void store4(void* Y, int64_t o, bool whole, int left, const f32x4& v) {
  if constexpr (OUT == NM_F32) {
    float* y = static_cast<float*>(Y) + o;
    if (whole) *reinterpret_cast<f32x4*>(y) = v;
    else for (int e = 0; e < 4 && e < left; ++e) y[e] = v[e];
  } else {
    uint16_t* y = static_cast<uint16_t*>(Y) + o;
    const u32x2 h = {pack_half2<DT>(v[0], v[1]), pack_half2<DT>(v[2], v[3])};
    if (whole) *reinterpret_cast<u32x2*>(y) = h;
    else for (int e = 0; e < 4 && e < left; ++e) y[e] = uint16_t(h[e >> 1] >> (16 * (e & 1)));
  }
}

// ---------------------------------------------------------------------------
// Few rows an expert: bound by streaming the packed weights of the experts that
// have any.  A wave owns 16 RB rows of one expert's weight and up to 16 NT of its
// tokens; the 8 waves of a workgroup take KS shares of K (in wave order added in
// LDS) and 8 / KS blocks of rows, KS so that the waves fill the chip.
//
// The order of the reduction is free, as long as both operands keep it: so a lane
// quarter takes a run of consecutive columns that makes whole 16-byte loads of
// packed values whatever the pattern, and one load of their index bits:
//   2:4  32 columns (2 x 16 bytes, 32 bits), a unit of 128 columns in 2 products;
//   1:4  32 columns (16 bytes, 16 bits), the same;
//   1:8  64 columns (16 bytes, 24 bits), a unit of 256 columns in 4 products.
// (One 64-column step a load, 8 or 4 bytes a lane, ran 41 experts of 2816 x 2048 in
// 1:4 in 94 us.)  Product p of a unit takes columns 16p .. 16p+15 of each quarter's
// run.  Loads of U units go out before the first product.
// 2 tokens on 2 experts of 4096 x 4096 in 2:4: 11 us, 3.3 TB/s (the search for the
// tile and two round trips to memory before the first product; 1 / 2 / 4 units of loads
// at a time 11.9 / 11.2 / 12.4 us).
// ---------------------------------------------------------------------------
constexpr int kFewWaves = 8;

template <int P>
struct FewUnit {
  static constexpr int RUN = P == 2 ? 64 : 32;     // columns of a lane quarter
  static constexpr int COLS = 4 * RUN, PRODUCTS = RUN / 16;
  static constexpr int WORDS = P == 0 ? 8 : 4;     // packed values of a run
  uint32_t v[WORDS];
  uint32_t i0, i1;                                 // index bits (1:8: the two words that hold them)
};

// A lane's run of columns k .. k + RUN - 1 of a row, zeros past K and where `on` is
// false.  Offsets past an edge are selected to lie outside the descriptors, not
// branched on: behind branches the loads of a unit waited for those before them.
// WIDE: K is a multiple of RUN, a run's values come whole; otherwise 16 columns a load.

template <int P, bool WIDE>
__device__ inline void load_unit(FewUnit<P>& f, __amdgpu_buffer_rsrc_t rv, __amdgpu_buffer_rsrc_t ri, uint32_t vrow,
                                 uint32_t irow, int words, int k, int K, bool on) {
  using F = FewUnit<P>;
  on &= k < K;
  const uint32_t v0 = vrow + uint32_t(k / pat_m(P) * pat_n(P)) * 2u;
  if constexpr (P == 0 || WIDE) {
#pragma unroll
    for (int q = 0; q < F::WORDS / 4; ++q) {
      const bool live = on & ((P != 0) | (k + 16 * q < K));
      const u32x4 t = __builtin_bit_cast(
          u32x4, __builtin_amdgcn_raw_buffer_load_b128(rv, live_offset(live, v0 + 16u * q), 0, 0));
#pragma unroll
      for (int e = 0; e < 4; ++e) f.v[4 * q + e] = t[e];
    }
  } else {
#pragma unroll
    for (int q = 0; q < F::PRODUCTS; ++q) {
      const bool live = on & (k + 16 * q < K);
      if constexpr (P == 1) {
        const u32x2 t = __builtin_bit_cast(
            u32x2, __builtin_amdgcn_raw_buffer_load_b64(rv, live_offset(live, v0 + 8u * q), 0, 0));
        f.v[2 * q] = t[0];
        f.v[2 * q + 1] = t[1];
      } else {
        f.v[q] = __builtin_amdgcn_raw_buffer_load_b32(rv, live_offset(live, v0 + 4u * q), 0, 0);
      }
    }
  }
  if constexpr (P == 0) {
    f.i0 = __builtin_amdgcn_raw_buffer_load_b32(ri, live_offset(on, irow + uint32_t(k >> 5) * 4u), 0, 0);
  } else if constexpr (P == 1) {
    f.i0 = uint16_t(__builtin_amdgcn_raw_buffer_load_b16(ri, live_offset(on, irow + uint32_t(k >> 5) * 2u), 0, 0));
  } else {   // 24 bits from bit 24 (k / 64) on; past the row's last word nothing is needed
    const int w = (k >> 6) * 24 >> 5;
    f.i0 = __builtin_amdgcn_raw_buffer_load_b32(ri, live_offset(on, irow + uint32_t(w) * 4u), 0, 0);
    f.i1 = __builtin_amdgcn_raw_buffer_load_b32(ri, live_offset(on, irow + uint32_t(min(w + 1, words - 1)) * 4u), 0, 0);
  }
}

// The 2:4 operand of product p.
template <int P>
__device__ inline void unit_operand(const FewUnit<P>& f, int k, int p, u32x4& a, uint32_t& ix) {
  if constexpr (P == 0) {
    a = u32x4{f.v[4 * p], f.v[4 * p + 1], f.v[4 * p + 2], f.v[4 * p + 3]};
    ix = (f.i0 >> (16 * p)) & 0xFFFFu;
  } else if constexpr (P == 1) {
    AFrag t;
    t.v[0] = f.v[2 * p];
    t.v[1] = f.v[2 * p + 1];
    t.ib = (f.i0 >> (8 * p)) & 0xFFu;
    widen<1>(t, a, ix);
  } else {
    AFrag t;
    t.v[0] = f.v[p];
    t.v[1] = f.i0;
    t.v[2] = f.i1;
    t.ib = uint32_t((((k >> 6) * 24) & 31) + 6 * p);
    widen<2>(t, a, ix);
  }
}

template <int P, int DT, int OUT, int RB, int NT, int U, bool WIDE>
__global__ __launch_bounds__(kFewWaves * 64) void group_few_kernel(const uint16_t* __restrict__ values,
                                                                   const uint32_t* __restrict__ idx,
                                                                   const uint16_t* __restrict__ act,
                                                                   const int32_t* __restrict__ offsets, GroupDims d,
                                                                   int ks, void* __restrict__ Y) {
  using F = FewUnit<P>;
  __shared__ f32x4 part[kFewWaves][RB * NT][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const int tile = __builtin_amdgcn_readfirstlane(blockIdx.x / d.tilesR);
  // its share of K and its rows (ks is a power of two)
  const int share = wave & (ks - 1);
  const int r0 = (((int(blockIdx.x) - tile * d.tilesR) * kFewWaves + wave - share) >> __builtin_ctz(ks)) * (16 * RB);
  GroupTile g;
  if (!group_find(offsets, d.E, d.T, 16 * NT, tile, g)) return;
  const int64_t S = int64_t(d.K) / pat_m(P) * pat_n(P);
  const int toks = min(16 * NT, g.t1 - g.t0);
  // (clamping to two sides is a vector operation: back to a scalar for the descriptors)
  const int rows = __builtin_amdgcn_readfirstlane(max(min(16 * RB, d.R - r0), 0));
  const uint32_t vbytes = uint32_t(S * 2), ibytes = uint32_t(d.words) * 4u;
  const int64_t first = int64_t(g.e) * d.R + r0;
  const __amdgpu_buffer_rsrc_t rv = make_rsrc(values + first * S, uint32_t(rows) * vbytes);
  const __amdgpu_buffer_rsrc_t ri = make_rsrc(idx + first * d.words, uint32_t(rows) * ibytes);
  const __amdgpu_buffer_rsrc_t rx =
      make_rsrc(act + int64_t(g.t0) * d.ldx, uint32_t((int64_t(toks - 1) * d.ldx + d.K) * 2));
  const int units = (d.K + F::COLS - 1) / F::COLS;
  const int per = (units + ks - 1) / ks;
  const int u_end = min(units, (share + 1) * per);

  f32x4 acc[RB][NT];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Batch {
    F a[U][RB];
    u32x8 b[U][F::PRODUCTS][NT];
  };
  auto load = [&](int u0, Batch& s) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (u0 + u) * F::COLS + lq * F::RUN;
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        const int r = i * 16 + li;
        load_unit<P, WIDE>(s.a[u][i], rv, ri, uint32_t(r) * vbytes, uint32_t(r) * ibytes, d.words, k, d.K,
                           (u0 + u < u_end) & (r < rows));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int p = 0; p < F::PRODUCTS; ++p)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int t = j * 16 + li;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // the product's columns 32h + 8 lq .. +7: half of a quarter's 16
            const int k = (u0 + u) * F::COLS + (2 * h + (lq >> 1)) * F::RUN + 16 * p + 8 * (lq & 1);
            const bool live = (u0 + u < u_end) & (t < toks) & (k < d.K);
            const u32x4 v = __builtin_bit_cast(
                u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                           rx, live_offset(live, (uint32_t(t) * uint32_t(d.ldx) + uint32_t(k)) * 2u), 0, 0));
#pragma unroll
            for (int e = 0; e < 4; ++e) s.b[u][p][j][4 * h + e] = v[e];
          }
        }
  };
  auto multiply = [&](int u0, const Batch& s) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int p = 0; p < F::PRODUCTS; ++p)
#pragma unroll
        for (int i = 0; i < RB; ++i) {
          u32x4 w;
          uint32_t ix;
          unit_operand<P>(s.a[u][i], (u0 + u) * F::COLS + lq * F::RUN, p, w, ix);
#pragma unroll
          for (int j = 0; j < NT; ++j) acc[i][j] = smfmac<DT>(w, s.b[u][p][j], acc[i][j], ix);
        }
  };
  for (int u = share * per; u < u_end; u += U) {
    Batch b;
    load(u, b);
    __builtin_amdgcn_sched_barrier(0);   // every load goes out before the first product
    multiply(u, b);
  }
  auto store = [&](int f, int first, const f32x4& sum) {   // fragment f of the rows from `first` on
    const int t = (f % NT) * 16 + li, r = first + (f / NT) * 16 + lq * 4;
    if (t < toks && r < d.R)
      store4<DT, OUT>(Y, int64_t(g.t0 + t) * d.ldy + r, (d.ldy & 3) == 0 && r + 3 < d.R, d.R - r, sum);
  };
  if (ks == 1) {
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) store(i * NT + j, r0, acc[i][j]);
    return;
  }
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) part[wave][i * NT + j][lane] = acc[i][j];
  __syncthreads();
  for (int f = share; f < RB * NT; f += ks) {
    const int w0 = wave - share;
    f32x4 sum = part[w0][f][lane];
    for (int w = 1; w < ks; ++w) sum += part[w0 + w][f][lane];
    store(f, r0, sum);
  }
}

// ---------------------------------------------------------------------------
// The same for rows of whole 16-byte pieces and K <= 4096: one workgroup a compute
// unit streams the weights without a pause.  The kernel above spends most of a
// workgroup's life waiting (the search, two round trips to memory, the sum over its
// waves); here a workgroup takes a run of one tile's rows, its waves keep their
// shares of the tokens in registers and fetch packed rows by direct loads into rings
// of D stages in LDS of their own: a stage is refilled as soon as its fragments are
// in registers.
//
// A unit is 16 rows x 128 bytes of values (2:4 128, 1:4 256, 1:8 512 columns), two
// loads of 8 whole rows' lines each, and their index words; slot (row, 16-byte
// piece c) of a unit at row*8 + (c ^ (row & 7)).  A stage is KU units.  As above a
// lane quarter's run is 16 values, so the products differ only in the widening.
// Of the 8 waves KS share K and 8 / KS take rows of their own; the KS partial tiles
// are added in wave order through LDS, one barrier a step.
// 96 tokens of 41 experts of 2816 x 2048 in 1:4: 32 to 34 us with inputs in turn, 3.9 to
// 4.2 TB/s of packed bytes.
// ---------------------------------------------------------------------------
template <int N, int I = 0, class F>
__device__ inline void static_for(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<N, I + 1>(f);
  }
}

template <int P, int KU>
struct Stream {
  static constexpr int RUN = P == 0 ? 32 : P == 1 ? 64 : 128;   // columns of a lane quarter
  static constexpr int COLS = 4 * RUN, PRODUCTS = RUN / 16;
  static constexpr int IWORDS = P == 2 ? 6 : 4;                 // index words of a row's unit
  static constexpr int ILOADS = P == 2 ? 2 : 1;
  static constexpr int UNIT = 2048 + ILOADS * 256, STAGE = KU * UNIT;
  static constexpr int LOADS = KU * (2 + ILOADS);               // a wave's direct loads a stage
  static constexpr int PART = 2 * kFewWaves * 64 * 16;
  static constexpr int D = (160 * 1024 - PART) / (kFewWaves * STAGE) < 8 ? (160 * 1024 - PART) / (kFewWaves * STAGE) : 8;
  static constexpr int LDS = kFewWaves * D * STAGE + PART;
  static_assert(D >= 2 && D * LOADS < 64, "stages, and a count of their loads");
};

template <int P, int DT, int OUT, int KU>
__global__ __launch_bounds__(kFewWaves * 64, 2) void group_stream_kernel(const uint16_t* __restrict__ values,
                                                                         const uint32_t* __restrict__ idx,
                                                                         const uint16_t* __restrict__ act,
                                                                         const int32_t* __restrict__ offsets,
                                                                         GroupDims d, int max_tiles, int ks,
                                                                         void* __restrict__ Y) {
  using C = Stream<P, KU>;
  extern __shared__ __align__(16) unsigned char smem[];
  f32x4* part = reinterpret_cast<f32x4*>(smem + kFewWaves * C::D * C::STAGE);   // [2][waves][64]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lq = lane >> 4;
  unsigned char* ring = smem + wave * (C::D * C::STAGE);
  const int share = wave & (ks - 1), rg = kFewWaves >> __builtin_ctz(ks);   // row groups; the wave's:
  const int mine = wave >> __builtin_ctz(ks);
  const int row_bytes = d.K / pat_m(P) * pat_n(P) * 2, idx_bytes = d.words * 4;
  const int rsteps = (d.R + 16 * rg - 1) / (16 * rg);   // steps of 16 rows a group over all rows
  const int unit0 = share * KU;

  // Parts of a tile's rows: enough that every workgroup has one, or, of many tiles,
  // so many that the last round is nearly full.
  const int tiles = min(group_count(offsets, d.E, d.T, 16), max_tiles), grid = gridDim.x;
  int parts = 1;
  if (2 * tiles <= grid) {
    parts = tiles > 0 ? min(grid / tiles, rsteps) : 1;
  } else {
    int best = 0x7FFFFFFF;
    for (int w = 1; w <= min(8, rsteps); ++w) {
      const int cost = ((tiles * w + grid - 1) / grid) * ((rsteps + w - 1) / w + 3);   // (3: a start's worth of steps)
      if (cost < best) best = cost, parts = w;
    }
  }
  for (int job = blockIdx.x; job < tiles * parts; job += grid) {
    GroupTile g;
    if (!group_find(offsets, d.E, d.T, 16, job / parts, g)) return;
    const int p = job % parts;
    const int step0 = __builtin_amdgcn_readfirstlane(int(int64_t(rsteps) * p / parts));
    const int n = __builtin_amdgcn_readfirstlane(int(int64_t(rsteps) * (p + 1) / parts)) - step0;
    const int toks = g.t1 - g.t0 < 16 ? g.t1 - g.t0 : 16;
    const __amdgpu_buffer_rsrc_t rv =
        make_rsrc(reinterpret_cast<const unsigned char*>(values) + int64_t(g.e) * d.R * row_bytes);
    const __amdgpu_buffer_rsrc_t ri = make_rsrc(idx + int64_t(g.e) * d.R * d.words);
    const __amdgpu_buffer_rsrc_t rx =
        make_rsrc(act + int64_t(g.t0) * d.ldx, uint32_t((int64_t(toks - 1) * d.ldx + d.K) * 2));

    // step i's rows; rows past R reread the last one, pieces and words past K the row's first
    auto issue = [&](int i, int slot) {
      const int r0 = ((step0 + i) * rg + mine) * 16;
      unsigned char* st = ring + slot * C::STAGE;
#pragma unroll
      for (int u = 0; u < KU; ++u) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int row = j * 8 + (lane >> 3), c = (lane & 7) ^ (row & 7);
          const int at = (unit0 + u) * 128 + c * 16;
          dma16(rv, uint32_t(min(r0 + row, d.R - 1)) * uint32_t(row_bytes) + uint32_t(at < row_bytes ? at : 0), 0u,
                st + u * C::UNIT + j * 1024);
        }
#pragma unroll
        for (int j = 0; j < C::ILOADS; ++j) {
          const int s = min(j * 64 + lane, 16 * C::IWORDS - 1), row = s / C::IWORDS;
          const int at = (unit0 + u) * C::IWORDS + s % C::IWORDS;
          __builtin_amdgcn_raw_ptr_buffer_load_lds(
              ri, (lds_byte*)(st + u * C::UNIT + 2048 + j * 256), 4,
              int(uint32_t(min(r0 + row, d.R - 1)) * uint32_t(idx_bytes) + uint32_t(at < d.words ? at : 0) * 4u), 0, 0, 0);
        }
      }
    };
    // the tokens' operands of the wave's units, kept over all steps
    u32x8 b[KU][C::PRODUCTS];
    auto load_tokens = [&] {
#pragma unroll
      for (int u = 0; u < KU; ++u)
#pragma unroll
        for (int q = 0; q < C::PRODUCTS; ++q)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int k = (unit0 + u) * C::COLS + (2 * h + (lq >> 1)) * C::RUN + 16 * q + 8 * (lq & 1);
            const bool live = (li < toks) & (k < d.K);
            const u32x4 v = __builtin_bit_cast(
                u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                           rx, live_offset(live, (uint32_t(li) * uint32_t(d.ldx) + uint32_t(k)) * 2u), 0, 0));
#pragma unroll
            for (int e = 0; e < 4; ++e) b[u][q][4 * h + e] = v[e];
          }
    };
#pragma unroll
    for (int s = 0; s < C::D; ++s)
      if (s < n) issue(s, s);
    load_tokens();

    int slot = 0;
    for (int i = 0; i < n; ++i) {
      // stage i has landed once at most the loads of the stages after it remain
      // (tokens and stores issued since only make the wait stricter)
      const int behind = min(n - 1 - i, C::D - 1);
      static_for<C::D>([&](auto c) {
        if (behind == decltype(c)::value) wait_vmcnt<decltype(c)::value * C::LOADS>();
      });
      asm volatile("" ::: "memory");
      const unsigned char* st = ring + slot * C::STAGE;
      u32x4 v[KU][2];
      uint32_t w0[KU], w1[KU];
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        const unsigned char* un = st + u * C::UNIT;
#pragma unroll
        for (int x = 0; x < 2; ++x)
          v[u][x] = *reinterpret_cast<const u32x4*>(un + (li * 8 + ((2 * lq + x) ^ (li & 7))) * 16);
        // the run's 32 index bits (1:8: 48, from bit 0 or 16 of two words)
        const uint32_t* w = reinterpret_cast<const uint32_t*>(
            un + 2048 + (P == 2 ? li * 24 + (3 * lq >> 1) * 4 : li * 16 + lq * 4));
        w0[u] = w[0];
        w1[u] = 0u;
        if constexpr (P == 2) w1[u] = w[1];
      }
      wait_lgkm0();
      asm volatile("" ::: "memory");
      if (i + C::D < n) issue(i + C::D, slot);
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < KU; ++u) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if ((unit0 + u) * 128 + (2 * lq + x) * 16 >= row_bytes) v[u][x] = u32x4{0u, 0u, 0u, 0u};   // past K
        uint64_t bits = w0[u];
        if constexpr (P == 2) bits = (bits | uint64_t(w1[u]) << 32) >> (16 * (lq & 1));
#pragma unroll
        for (int q = 0; q < C::PRODUCTS; ++q) {
          u32x4 a;
          uint32_t ix;
          if constexpr (P == 0) {
            a = v[u][q];
            ix = uint32_t(bits >> (16 * q)) & 0xFFFFu;
          } else {
            AFrag t;
            if constexpr (P == 1) {
              t.v[0] = v[u][q >> 1][2 * (q & 1)];
              t.v[1] = v[u][q >> 1][2 * (q & 1) + 1];
              t.ib = uint32_t(bits >> (8 * q)) & 0xFFu;
            } else {
              t.v[0] = v[u][q >> 2][q & 3];
              t.v[1] = uint32_t(bits >> (6 * q)) & 63u;
              t.v[2] = 0u;
              t.ib = 0u;
            }
            widen<P>(t, a, ix);
          }
          acc = smfmac<DT>(a, b[u][q], acc, ix);
        }
      }
      const int r = ((step0 + i) * rg + mine) * 16 + lq * 4;
      const bool inside = li < toks && r < d.R;
      const int64_t o = int64_t(g.t0 + li) * d.ldy + r;
      const bool whole = (d.ldy & 3) == 0 && r + 3 < d.R;
      if (ks == 1) {
        if (inside) store4<DT, OUT>(Y, o, whole, d.R - r, acc);
      } else {
        f32x4* buf = part + (i & 1) * (kFewWaves * 64);
        buf[wave * 64 + lane] = acc;
        wait_lgkm0();
        barrier_no_fence();   // (the other buffer's sums were read before this one was written)
        if (share == (i & (ks - 1))) {
          f32x4 sum = buf[(wave - share) * 64 + lane];
          for (int w = 1; w < ks; ++w) sum += buf[(wave - share + w) * 64 + lane];
          if (inside) store4<DT, OUT>(Y, o, whole, d.R - r, sum);
        }
      }
      slot = slot == C::D - 1 ? 0 : slot + 1;
    }
    if (ks > 1) barrier_no_fence();   // the last sums are read before the next job's are written
  }
}

// ---------------------------------------------------------------------------
// Any shape: 128 rows x BT tokens by 4 waves (2 x 2), K in steps of 64.  Each
// thread loads its share of a step two steps ahead into registers (zeros past the
// edges of W, of K and of the expert's rows), widens it to the 2:4 operand, and
// writes it to a double-buffered stage in LDS, so every pattern runs the same
// products.  One barrier a step publishes one stage and retires the other.
// 1333 tokens of 5 experts of 1000 x 1056 in 1:8, 208 workgroups of 17 steps: 14.8 us,
// the matrix cores 3% busy: bound by launch, first loads and epilogue.
// ---------------------------------------------------------------------------
constexpr int kBR = 128;
constexpr int kStageA = kBR * 64, kStageI = kBR * 8;
template <int P, int DT, int OUT, int BT>
__global__ __launch_bounds__(256, 2) void group_tile_kernel(const uint16_t* __restrict__ values,
                                                            const uint32_t* __restrict__ idx,
                                                            const uint16_t* __restrict__ act,
                                                            GroupRows experts, GroupDims d, void* __restrict__ Y) {
  constexpr int FR = 4, FT = BT / 32;
  constexpr int kStageB = BT * 128, kStage = kStageA + kStageI + kStageB;
  constexpr int PB = BT / 32;   // 16-byte pieces of the tokens a thread loads a step
  __shared__ __align__(16) unsigned char smem[2 * kStage];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const int wr = wave >> 1, wt = wave & 1;
  const int b0 = blockIdx.x;
  const int tt = b0 / d.tilesR, tr = b0 - tt * d.tilesR;
  GroupTile g;
  if (!experts.tile(tt, d.T, BT, g)) return;
  const int r0 = tr * kBR;
  const int rows = min(kBR, d.R - r0), toks = min(BT, g.t1 - g.t0);
  const int64_t S = int64_t(d.K) / pat_m(P) * pat_n(P);
  const __amdgpu_buffer_rsrc_t rv = make_rsrc(values + (int64_t(g.e) * d.R + r0) * S, uint32_t(rows * S * 2));
  const __amdgpu_buffer_rsrc_t ri =
      make_rsrc(idx + (int64_t(g.e) * d.R + r0) * d.words, uint32_t(int64_t(rows) * d.words * 4));
  const __amdgpu_buffer_rsrc_t rx =
      make_rsrc(act + int64_t(g.t0) * d.ldx, uint32_t((int64_t(toks - 1) * d.ldx + d.K) * 2));
  // the steps this workgroup reduces over: all, or its share (an even number) of them
  int first = 0, steps = (d.K + 63) >> 6;
  if (d.share > 0) {
    first = int(blockIdx.y) * d.share;
    steps = min(steps, first + d.share);
    Y = static_cast<float*>(Y) + int64_t(blockIdx.y) * d.part_stride;
  }

  // this thread's share of W: 32 columns (half wh of the step) of row wrow
  const int wrow = tid >> 1, wh = tid & 1;
  constexpr int VB = P == 0 ? 32 : P == 1 ? 16 : 8;   // bytes of values of 32 columns
  struct Share {
    uint32_t v[VB / 4];
    uint32_t w0, w1;
    u32x4 x[PB];
  };
  const uint32_t vbase = uint32_t(wrow * S * 2), ibase = uint32_t(wrow * d.words * 4);
  uint32_t xoff[PB];
  int xcol[PB];
#pragma unroll
  for (int j = 0; j < PB; ++j) {
    const int slot = j * 256 + tid, tok = slot >> 3, c = (slot & 7) ^ (tok & 7);
    xoff[j] = live_offset(tok < toks, uint32_t(tok) * uint32_t(d.ldx) * 2u + uint32_t(c) * 16u);
    xcol[j] = c * 8;
  }
  auto load = [&](int s, Share& o) {
    const int k = s * 64 + wh * 32;
    const bool on = (s < steps) & (wrow < rows) & (k < d.K), on2 = on & (k + 16 < d.K);
    const uint32_t v0 = vbase + uint32_t(s * 2 + wh) * VB;
    if constexpr (P == 0) {
      const u32x4 a = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rv, live_offset(on, v0), 0, 0));
      const u32x4 b =
          __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rv, live_offset(on2, v0 + 16u), 0, 0));
#pragma unroll
      for (int e = 0; e < 4; ++e) o.v[e] = a[e], o.v[4 + e] = b[e];
      o.w0 = __builtin_amdgcn_raw_buffer_load_b32(ri, live_offset(on, ibase + uint32_t(s * 2 + wh) * 4u), 0, 0);
    } else if constexpr (P == 1) {
      const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rv, live_offset(on, v0), 0, 0));
      const u32x2 b =
          __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rv, live_offset(on2, v0 + 8u), 0, 0));
      o.v[0] = a[0], o.v[1] = a[1], o.v[2] = b[0], o.v[3] = b[1];
      o.w0 = __builtin_amdgcn_raw_buffer_load_b32(ri, live_offset(on, ibase + uint32_t(s) * 4u), 0, 0);
    } else {
      o.v[0] = __builtin_amdgcn_raw_buffer_load_b32(rv, live_offset(on, v0), 0, 0);
      o.v[1] = __builtin_amdgcn_raw_buffer_load_b32(rv, live_offset(on2, v0 + 4u), 0, 0);
      const int bit = 24 * s + 12 * wh, w = bit >> 5;
      o.w0 = __builtin_amdgcn_raw_buffer_load_b32(ri, live_offset(on, ibase + uint32_t(w) * 4u), 0, 0);
      // (the row's last word holds every bit it needs: the next one is not looked at)
      o.w1 = __builtin_amdgcn_raw_buffer_load_b32(ri, live_offset(on, ibase + uint32_t(min(w + 1, d.words - 1)) * 4u), 0, 0);
    }
#pragma unroll
    for (int j = 0; j < PB; ++j) {
      const bool live = (s < steps) & (s * 64 + xcol[j] < d.K) & (xoff[j] < kDeadOffset);
      o.x[j] = __builtin_bit_cast(
          u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, live_offset(live, xoff[j] + uint32_t(s) * 128u), 0, 0));
    }
  };
  auto stage = [&](int s, const Share& o) {
    unsigned char* st = smem + (s & 1) * kStage;
    uint32_t v[8], ix;
    if constexpr (P == 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = o.v[e];
      ix = o.w0;
    } else if constexpr (P == 1) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (o.v[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
      uint32_t y = (o.w0 >> (16 * wh)) & 0xFFFFu;   // eight 2-bit positions, each to a nibble p | p << 2
      y = (y | (y << 8)) & 0x00FF00FFu;
      y = (y | (y << 4)) & 0x0F0F0F0Fu;
      y = (y | (y << 2)) & 0x33333333u;
      ix = y * 5u;
    } else {
      const uint32_t bits = uint32_t((uint64_t(o.w0) | uint64_t(o.w1) << 32) >> ((24 * s + 12 * wh) & 31));
      ix = 0u;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t h = (o.v[e >> 1] >> (16 * (e & 1))) & 0xFFFFu, p = (bits >> (3 * e)) & 7u;
        v[2 * e] = p < 4u ? h : 0u;
        v[2 * e + 1] = p < 4u ? 0u : h;
        ix |= ((p & 3u) * 5u) << (8 * e + (p < 4u ? 0 : 4));
      }
    }
    const int sw = (wrow >> 1) & 3;
    *reinterpret_cast<u32x4*>(st + (wrow * 4 + ((2 * wh) ^ sw)) * 16) = u32x4{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<u32x4*>(st + (wrow * 4 + ((2 * wh + 1) ^ sw)) * 16) = u32x4{v[4], v[5], v[6], v[7]};
    *reinterpret_cast<uint32_t*>(st + kStageA + wrow * 8 + wh * 4) = ix;
#pragma unroll
    for (int j = 0; j < PB; ++j) *reinterpret_cast<u32x4*>(st + kStageA + kStageI + (j * 256 + tid) * 16) = o.x[j];
  };

  f32x4 acc[FR][FT];
#pragma unroll
  for (int i = 0; i < FR; ++i)
#pragma unroll
    for (int j = 0; j < FT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  Share sh[2];
  load(first, sh[0]);
  load(first + 1, sh[1]);
  stage(first, sh[0]);
  load(first + 2, sh[0]);
  auto step = [&](auto par_c, int s) {
    constexpr int PAR = decltype(par_c)::value;
    wait_lgkm0();
    barrier_no_fence();
    const unsigned char* st = smem + PAR * kStage;
    u32x4 a[FR];
    uint32_t ix[FR];
    u32x8 b[FT];
#pragma unroll
    for (int i = 0; i < FR; ++i) {
      const int row = wr * 64 + i * 16 + li;
      a[i] = *reinterpret_cast<const u32x4*>(st + (row * 4 + (lq ^ ((row >> 1) & 3))) * 16);
      ix[i] = *reinterpret_cast<const uint16_t*>(st + kStageA + row * 8 + lq * 2);
    }
#pragma unroll
    for (int j = 0; j < FT; ++j) {
      const int tok = wt * (BT / 2) + j * 16 + li;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(st + kStageA + kStageI + (tok * 8 + ((lq + 4 * h) ^ (tok & 7))) * 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) b[j][4 * h + e] = v[e];
      }
    }
#pragma unroll
    for (int i = 0; i < FR; ++i)
#pragma unroll
      for (int j = 0; j < FT; ++j) acc[i][j] = smfmac<DT>(a[i], b[j], acc[i][j], ix[i]);
    if (s + 1 < steps) stage(s + 1, sh[PAR ^ 1]);
    load(s + 3, sh[PAR ^ 1]);
  };
  int s = first;
  for (; s + 1 < steps; s += 2) {
    step(std::integral_constant<int, 0>{}, s);
    step(std::integral_constant<int, 1>{}, s + 1);
  }
  if (s < steps) step(std::integral_constant<int, 0>{}, s);
  wait_vmcnt<0>();

  const bool vec = (d.ldy & 3) == 0;
#pragma unroll
  for (int i = 0; i < FR; ++i) {
    const int r = wr * 64 + i * 16 + lq * 4;
#pragma unroll
    for (int j = 0; j < FT; ++j) {
      const int t = wt * (BT / 2) + j * 16 + li;
      if (t < toks && r < rows)
        store4<DT, OUT>(Y, int64_t(g.t0 + t) * d.ldy + r0 + r, vec && r + 3 < rows, rows - r, acc[i][j]);
    }
  }
}

// The parts of a shared reduction, added in their order (bound by its launch: the parts
// are a few MB and come from the cache).
template <int OUT>
__global__ __launch_bounds__(256) void group_join_kernel(const float* __restrict__ part, int n, int T, int C, int64_t ld,
                                                         const int32_t* __restrict__ offsets, int E,
                                                         void* __restrict__ out, int64_t ldo) {
  int lo = 0, hi = T;
  if (offsets) lo = rows_lo(offsets[0], T), hi = rows_hi(offsets[E], lo, T);
  const int t = lo + int(blockIdx.x), c = (int(blockIdx.y) * 256 + int(threadIdx.x)) * 4;
  if (t >= hi || c >= C) return;
  const int64_t stride = int64_t(T) * ld;
  const float* p = part + t * ld + c;
  f32x4 sum = *reinterpret_cast<const f32x4*>(p);
  for (int i = 1; i < n; ++i) sum += *reinterpret_cast<const f32x4*>(p + i * stride);
  store4<OUT, OUT>(out, int64_t(t) * ldo + c, (ldo & 3) == 0 && c + 3 < C, C - c, sum);
}

GroupDims dims_of(const GroupArgs& a, int rows) {
  GroupDims d;
  d.E = int(a.E);
  d.R = int(a.base.R);
  d.K = int(a.base.K);
  d.T = int(a.base.T);
  d.words = int(a.base.idx_row_words);
  d.tilesR = int((a.base.R + rows - 1) / rows);
  d.ldx = a.base.ldx;
  d.ldy = a.base.ldy;
  return d;
}

template <int P, int DT, int OUT, int RB, int NT, int U>
hipError_t launch_few(const GroupArgs& a, hipStream_t s) {
  const int64_t experts = std::min(a.base.T, a.E);
  // shares of K while the waves fit the chip a few times over, but none below two units
  const int64_t blocks = (a.base.R + 16 * RB - 1) / (16 * RB), units = a.base.K / FewUnit<P>::COLS;
  int ks = 1;
  while (ks < kFewWaves && experts * blocks * ks < 16 * 1024 && units >= 2 * ks) ks *= 2;
  const GroupDims d = dims_of(a, 16 * RB * (kFewWaves / ks));
  const int64_t grid = group_max_tiles(a.base.T, a.E, 16 * NT) * d.tilesR;
  if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
  const bool wide = P == 0 || a.base.K % FewUnit<P>::RUN == 0;
  const auto kern = wide ? group_few_kernel<P, DT, OUT, RB, NT, U, true> : group_few_kernel<P, DT, OUT, RB, NT, U, P == 0>;
  hipLaunchKernelGGL(kern, dim3(unsigned(grid)), dim3(kFewWaves * 64), 0, s, a.base.values, a.base.idx, a.base.act,
                     a.offsets, d, ks, a.base.Y);
  return hipGetLastError();
}

// Units a wave of the streaming kernel keeps its tokens for: as many as its registers
// hold (fewer, in more shares of K, mean more sums: 41 experts of 2816 x 2048 in 1:4
// with 1 / 2 / 4 units 37.9 / 34.2 / 35.2 us with inputs in turn, 34.6 / 27.1 / 28.1 with
// the same ones, which the cache keeps).
constexpr int stream_units(int P) { return P == 0 ? 4 : 2; }
int stream_shares(const SpmmArgs& b) {
  const int P = b.n == 2 ? 0 : b.m == 4 ? 1 : 2;
  const int64_t cols = 128 << P;   // of a unit
  int ks = 1;
  while (ks * stream_units(P) * cols < b.K) ks *= 2;
  return ks;
}

template <int P, int DT, int OUT, int KU>
hipError_t launch_stream(const GroupArgs& a, hipStream_t s) {
  using C = Stream<P, KU>;
  static_assert(C::COLS == 128 << P, "a unit's columns");
  const int ks = stream_shares(a.base);
  const auto kern = group_stream_kernel<P, DT, OUT, KU>;
  if (hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(kern), C::LDS); e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3(unsigned(device_cu_count())), dim3(kFewWaves * 64), C::LDS, s, a.base.values, a.base.idx,
                     a.base.act, a.offsets, dims_of(a, 16), int(group_max_tiles(a.base.T, a.E, 16)), ks, a.base.Y);
  return hipGetLastError();
}

int64_t part_ld(int64_t R) { return (R + 3) / 4 * 4; }   // rows on 16 bytes

Shares tile_shares(const SpmmArgs& b, int64_t E, int BT) {
  return group_shares((b.R + kBR - 1) / kBR * group_max_tiles(b.T, E, BT), (b.K + 63) / 64);
}

template <int P, int DT, int OUT, int BT>
hipError_t launch_tile(const GroupArgs& a, hipStream_t s) {
  const GroupDims d = dims_of(a, kBR);
  const int64_t tiles = group_max_tiles(a.base.T, a.E, BT);
  if (tiles * d.tilesR > 0x7FFFFFFF) return hipErrorInvalidValue;
  GroupRows rows;
  if (hipError_t e = group_rows(a.offsets, a.E, a.base.T, BT, tiles, a.workspace, s, rows); e != hipSuccess) return e;
  const Shares sh = tile_shares(a.base, a.E, BT);
  if (sh.n > 1) {
    // partial sums behind the table, joined by a second launch
    float* part = reinterpret_cast<float*>(static_cast<unsigned char*>(a.workspace) + group_rows_bytes(a.E, tiles));
    const int64_t ld = part_ld(a.base.R);
    GroupDims p = d;
    p.ldy = ld;
    p.share = sh.size;
    p.part_stride = a.base.T * ld;
    hipLaunchKernelGGL((group_tile_kernel<P, DT, NM_F32, BT>), dim3(unsigned(tiles * d.tilesR), unsigned(sh.n)), dim3(256),
                       0, s, a.base.values, a.base.idx, a.base.act, rows, p, static_cast<void*>(part));
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    return launch_group_join(part, sh.n, a.base.T, a.base.R, ld, a.offsets, int(a.E), a.base.Y, a.base.ldy, OUT, s);
  }
  hipLaunchKernelGGL((group_tile_kernel<P, DT, OUT, BT>), dim3(unsigned(tiles * d.tilesR)), dim3(256), 0, s,
                     a.base.values, a.base.idx, a.base.act, rows, d, a.base.Y);
  return hipGetLastError();
}

// Tokens an expert has on average, of the experts that can have any.
int64_t mean_rows(int64_t T, int64_t E) { return T / std::max<int64_t>(1, std::min(T, E)); }

// Whether the streaming kernel takes the weight (whole 16-byte pieces a row, K in its
// waves' registers, one expert's packed bytes in 32-bit offsets) and has at least four
// steps a workgroup to stream (2 experts of 4096 x 4096, two steps: 12.4 us against
// 11.5; 4 experts 19.8 against 20.4; 8 experts 33.9 against 39.1).
bool stream_applies(const SpmmArgs& b, int64_t E) {
  const int64_t piece = b.n == 2 ? 16 : b.m == 4 ? 32 : 64, row_bytes = b.K / b.m * b.n * 2;
  if (b.K % piece != 0 || b.K > 4096 || b.R * row_bytes >= (int64_t(1) << 32)) return false;
  const int64_t rows = 16 * (kFewWaves / stream_shares(b));
  return std::min(b.T, E) * ((b.R + rows - 1) / rows) >= 4 * 256;
}

// Which kernel: by the rows an expert has on average, of those that can have any.  Both
// sides of the limits, us with inputs in turn, on 41 experts of 2816 x 2048 and on 8 of
// 4096 x 4096, each in 2:4 and in 1:4:
//   rows        41: 2:4      41: 1:4      8: 2:4       8: 1:4
//      8     59.0  68.4   36.9  52.1   35.7  43.8   23.1  29.1   stream, few2
//     12     64.7  71.4   40.8  54.1   39.2  45.1   26.0  30.7   (it leads here as well)
//     20     80.0  84.4   62.7  66.9   50.9  53.2   36.8  41.1   few2, tile64
//     24     88.7  85.2   70.0  67.9   59.2  53.4   45.3  41.3
//     32    101.0  86.7   80.9  69.8   64.3  53.9   49.8  41.8
//     64    113.9  98.4   99.5  82.9   75.8  65.2   57.7  56.4   tile64, tile128; in 2:4
//     96    138.5 126.6  124.1 113.8   85.6  88.9   68.1  70.5   lds 72.2, 86.9; 59.9, 61.9
enum class Pick { stream, few1, few1_wide, few2, tile64, tile128, lds };

Pick pick(const SpmmArgs& b, int64_t E) {
  const int64_t mean = mean_rows(b.T, E);
  // 64 rows a wave (the tokens are read a quarter as often) where that leaves waves enough;
  // 16 and 64 rows, in 2:4 / 1:4 / 1:8: 2 experts of 4096 x 4096 11.5 and 15.9 us / 9.2 and
  // 12.5 / 8.3 and 10.9; 3 of them 15.2 and 16.6 / 12.2 and 13.0 / 11.8 and 11.7; 8 of 1571 x
  // 4128 17.2 and 17.7 / 13.3 and 12.7 / 18.3 and 13.7; 3 of 8192 x 4128 32.2 and 41.0 / 18.4
  // and 23.1 / 25.4 and 21.8 (where the rows are many it is 1:8 alone that gains)
  if (mean <= 8) {
    if (stream_applies(b, E)) return Pick::stream;
    return std::min(b.T, E) * b.R >= 12288 ? Pick::few1_wide : Pick::few1;
  }
  if (mean <= 24) return Pick::few2;
  if (mean <= 64) return Pick::tile64;
  // (by numbers alone: the workspace's size is asked for without a device)
  // the single weight's large tiles and their table's launch where 96 of them fill the
  // chip (8 experts of 1024 x 1024: 2048 tokens, 64 tiles, 20.4 us against 13.9 below;
  // 16 experts of 1408 x 2048: 2048 tokens, 96 tiles, 29.4 against 36.4, 8192 tokens of
  // 4096 x 2048, 1024 tiles, 108 against 180; all with the same inputs, from the cache)
  if (b.n == 2 && b.K % 128 == 0 && b.R >= 256 && (b.R + 255) / 256 * ((b.T + 127) / 128) >= 96) return Pick::lds;
  // tiles of 128 tokens where there is one for every compute unit (4 experts of 2048 x 2048
  // in 1:4 / 1:8, tiles of 64 and of 128: 1536 tokens, 192 tiles, 30.3 and 29.5 us / 33.3 and
  // 31.2; 2048, 256 tiles, 43.0 and 37.1 / 47.6 and 40.9)
  const int64_t tiles = (b.R + kBR - 1) / kBR * ((b.T + 127) / 128);
  return tiles >= 256 ? Pick::tile128 : Pick::tile64;
}

template <int P, int DT, int OUT>
hipError_t launch_pick(const GroupArgs& a, hipStream_t s) {
  switch (pick(a.base, a.E)) {
    case Pick::stream: return launch_stream<P, DT, OUT, stream_units(P)>(a, s);
    case Pick::few1: return launch_few<P, DT, OUT, 1, 1, 2>(a, s);
    case Pick::few1_wide: return launch_few<P, DT, OUT, 4, 1, 1>(a, s);
    case Pick::few2: return launch_few<P, DT, OUT, 4, 2, 1>(a, s);
    case Pick::tile64: return launch_tile<P, DT, OUT, 64>(a, s);
    case Pick::tile128: return launch_tile<P, DT, OUT, 128>(a, s);
    default: break;
  }
  const int64_t tiles = group_max_tiles(a.base.T, a.E, spmm_lds_tile());
  int4* table = static_cast<int4*>(a.workspace);
  if (hipError_t e = launch_group_tiles(a.offsets, a.E, a.base.T, spmm_lds_tile(), tiles, table, s); e != hipSuccess)
    return e;
  return launch_spmm_lds_group(a.base, table, int(tiles), s);
}

template <int P>
hipError_t pick_type(const GroupArgs& a, hipStream_t s) {
  const bool f32 = a.base.out_dtype == NM_F32;
  if (a.base.dtype == NM_F16) return f32 ? launch_pick<P, NM_F16, NM_F32>(a, s) : launch_pick<P, NM_F16, NM_F16>(a, s);
  return f32 ? launch_pick<P, NM_BF16, NM_F32>(a, s) : launch_pick<P, NM_BF16, NM_BF16>(a, s);
}

}  // namespace

hipError_t launch_group_tiles(const int32_t* offsets, int64_t E, int64_t T, int BT, int64_t max_tiles, int4* table,
                              hipStream_t s) {
  hipLaunchKernelGGL(group_tiles_kernel, dim3(1), dim3(kTableThreads), 0, s, offsets, int(E), int(T), BT,
                     int(max_tiles), table);
  return hipGetLastError();
}

// Shares of at least four steps, an even number of them each (the tiles' stages go by
// a step's parity), while the workgroups fit the chip twice, and three or more: of 32
// steps or more, or, where at most 64 tiles leave three quarters of the chip idle (and the
// parts are small), of 16.  A step is a third to a whole microsecond, the join a launch
// and 2 to 4.  (One token of ten experts of 3184 x 480, dX, 4 tiles of 50 steps: 36.4 us
// in one, 11.8 in shares.  2130 tokens of 12 experts of 160 x 2912, forward: 25.6 and
// 20.5.  8192 tokens of 2 experts of 64 x 64, dW: 69.5 and 16.0.  Two shares: 2376
// tokens of 2 experts of 520 x 2016, forward, 20.7 in one, 25.6 in two.  64 tokens of 4
// experts of 1536 x 1024, dX, 32 tiles of 24 steps: 20.3 and 10.9; 200 tokens of 512 x
// 1280, forward, 16 of 20: 11.5 and 8.7; 900 tokens of 1024 x 512, dW, 16 of 28: 21.0 and
// 15.2; but 1333 tokens of 5 experts of 1000 x 1056, dX, 135 of 16: 15.7 and 23.1.)
Shares group_shares(int64_t tiles, int64_t steps) {
  Shares s;
  if (tiles <= 0 || tiles >= 256 || steps < (tiles <= 64 ? 16 : 32)) return s;   // (none: a weight without rows)
  const int64_t most = std::min<int64_t>(std::min<int64_t>(512 / tiles, steps / 4), 16);
  if (most < 3) return s;
  s.size = int((steps + most - 1) / most + 1) & ~1;
  s.n = int((steps + s.size - 1) / s.size);
  return s;
}

hipError_t launch_group_join(const float* part, int n, int64_t T, int64_t C, int64_t ld, const int32_t* offsets, int E,
                             void* out, int64_t ldo, int out_dtype, hipStream_t s) {
  const dim3 grid(unsigned(T), unsigned((C + 1023) / 1024));
  const auto kern = out_dtype == NM_F32 ? group_join_kernel<NM_F32>
                    : out_dtype == NM_F16 ? group_join_kernel<NM_F16> : group_join_kernel<NM_BF16>;
  hipLaunchKernelGGL(kern, grid, dim3(256), 0, s, part, n, int(T), int(C), ld, offsets, E, out, ldo);
  return hipGetLastError();
}

size_t group_workspace(const SpmmArgs& base, int64_t E) {
  const Pick p = pick(base, E);
  if (p == Pick::lds) return group_table_bytes(group_max_tiles(base.T, E, spmm_lds_tile()));
  if (p != Pick::tile64 && p != Pick::tile128) return 0;
  const int BT = p == Pick::tile64 ? 64 : 128;
  const Shares sh = tile_shares(base, E, BT);
  return group_rows_bytes(E, group_max_tiles(base.T, E, BT)) +
         (sh.n > 1 ? size_t(sh.n) * size_t(base.T) * size_t(part_ld(base.R)) * 4 : 0);
}

size_t group_dx_workspace(int64_t R, int64_t K, int64_t T, int64_t E) {
  const Shares sh = spmm_dx_shares(R, K, T, E);
  return group_rows_bytes(E, spmm_dx_max_tiles(T, E)) + (sh.n > 1 ? size_t(sh.n) * size_t(T) * size_t(K) * 4 : 0);
}

size_t group_dw_workspace(int64_t R, int64_t K, int64_t S, int64_t T, int64_t E) {
  const int n = spmm_dw_shares(R, K, T, E);
  return n > 1 ? size_t(n) * size_t(E) * size_t(R) * size_t(S) * 4 : 0;
}

hipError_t launch_group(const GroupArgs& a, hipStream_t s) {
  if (a.base.n == 2) return pick_type<0>(a, s);
  return a.base.m == 4 ? pick_type<1>(a, s) : pick_type<2>(a, s);
}

}  // namespace nm
