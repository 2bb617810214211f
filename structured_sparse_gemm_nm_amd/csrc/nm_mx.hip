// Microscaled 4-bit floats (E2M1 values, one power of two for every 32 along a
// row) on gfx950: quantisation, its inverse, and the product
//   Y[t][r] = sum_k x[t][k] w[r][k]
// of two such operands on v_mfma_scale_f32_16x16x128_f8f6f4, one weight or one
// for each expert of tokens ordered by expert (nm_group.h).
//
// Format.  Two values a byte, the even one in the low bits.  The exponent bytes
// of a row come eight at a time in panels of 256 columns,
//   scale[panel][row][8],
// so that the scales of a tile's rows for one step of the product are one
// contiguous run: with each row's bytes kept together they would be a 128-byte
// line fetched per row for 8 bytes of it.
#include "nm_device.h"
#include "nm_group.h"
#include "nm_internal.h"

#include <algorithm>
#include <type_traits>

namespace nm {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((ext_vector_type(2))) float f32x2;

// D = C + A x B on 16 x 16 x 128 4-bit values: lane (i, q) holds 32 consecutive
// reduction values (16 bytes) of row i of A and of column i of B, and byte SA
// (SB) of its scale register their exponent; D rows 4q..4q+3 of column i.
template <int SA, int SB>
__device__ inline f32x4 mfma_fp4(const u32x4& a, const u32x4& b, const f32x4& c, uint32_t sa, uint32_t sb) {
  const i32x8 av = {int(a[0]), int(a[1]), int(a[2]), int(a[3]), 0, 0, 0, 0};
  const i32x8 bv = {int(b[0]), int(b[1]), int(b[2]), int(b[3]), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, SA, int(sa), SB, int(sb));
}

// ---------------------------------------------------------------------------
// Quantisation.  A block's exponent is that of its largest magnitude less 2, so
// that this one lies in [4, 8) (6 is the largest value: above it saturates), and
// each value goes to the nearest of the eight magnitudes, ties to the even
// mantissa.  Four lanes share a block, 8 values each.  A block that holds Inf or
// NaN gets the exponent byte 255, which makes all of it NaN.  Of a stack, workgroups
// (.., e) take matrix e, `stride` elements of x (y) behind the one before.
// Bound by its bytes: 2 (or 4) read and 17/32 written a value.  11008 x 4096 fp32:
// 45 us, 4.6 TB/s.
// ---------------------------------------------------------------------------
template <int DT>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const void* __restrict__ x, int64_t T, int64_t K, int64_t ldx,
                                                          int64_t stride, bool vec, uint32_t* __restrict__ q,
                                                          uint8_t* __restrict__ scale) {
  const int64_t per_row = K / 8;   // shares of 8 values
  const int64_t panels = (K + 255) / 256;
  const int64_t total = T * panels * 32;   // whole panels: the last one's missing blocks get the byte 0
  x = static_cast<const unsigned char*>(x) + blockIdx.y * stride * (DT == NM_F32 ? 4 : 2);
  q += blockIdx.y * (T * per_row);
  scale += blockIdx.y * (panels * T * 8);
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < total; i += int64_t(gridDim.x) * 256) {
    const int64_t t = i / (panels * 32), c = i - t * (panels * 32);
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
    if (c < per_row) {
      if constexpr (DT == NM_F32) {
        const float* p = static_cast<const float*>(x) + t * ldx + c * 8;
        if (vec) {
          const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = a[e], v[4 + e] = b[e];
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = p[e];
        }
      } else {
        const uint16_t* p = static_cast<const uint16_t*>(x) + t * ldx + c * 8;
        if (vec) {
          const u32x4 a = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = half_to_f32<DT>((a[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = half_to_f32<DT>(p[e]);
        }
      }
    }
    // magnitudes compare as their bits, NaN above Inf above every number
    uint32_t top = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __builtin_bit_cast(uint32_t, v[e]) & 0x7FFFFFFFu);
    top = max(top, uint32_t(__shfl_xor(int(top), 1, 64)));
    top = max(top, uint32_t(__shfl_xor(int(top), 2, 64)));
    const int field = int(top >> 23);
    const int byte = field == 255 ? 255 : max(field - 2, 0);
    // 2^(127 - byte) = 2^(254 - byte - 127): exact, and normal for every byte up to 252
    const float up = __builtin_bit_cast(float, uint32_t(254 - min(byte, 253)) << 23);
    uint32_t out = 0u;
    if (field != 255) {
      out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[0] * up, v[1] * up, 1.f, 0);
      out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[2] * up, v[3] * up, 1.f, 1);
      out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[4] * up, v[5] * up, 1.f, 2);
      out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[6] * up, v[7] * up, 1.f, 3);
    }
    if (c < per_row) q[t * per_row + c] = out;
    if ((c & 3) == 0) {
      const int64_t block = c >> 2;
      scale[((block >> 3) * T + t) * 8 + (block & 7)] = uint8_t(c < per_row ? byte : 0);
    }
  }
}

// The values that 4 bits and an exponent stand for, rounded to DT (exact in bf16
// and fp32 where they fit its range).  Bound by its bytes: 11008 x 4096 to fp32 in 34 us,
// 6 TB/s.
template <int DT>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint32_t* __restrict__ q,
                                                            const uint8_t* __restrict__ scale, int64_t T, int64_t K,
                                                            void* __restrict__ y, int64_t ldy, int64_t stride,
                                                            bool vec) {
  const int64_t per_row = K / 8;
  const int64_t total = T * per_row;
  q += blockIdx.y * total;
  scale += blockIdx.y * ((K + 255) / 256 * T * 8);
  y = static_cast<unsigned char*>(y) + blockIdx.y * stride * (DT == NM_F32 ? 4 : 2);
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < total; i += int64_t(gridDim.x) * 256) {
    const int64_t t = i / per_row, c = i - t * per_row;
    const int64_t block = c >> 2;
    const uint32_t byte = scale[((block >> 3) * T + t) * 8 + (block & 7)];
    const uint32_t w = q[i];
    const float s = __builtin_bit_cast(float, byte == 255 ? 0x7FC00000u : byte == 0 ? 0x00400000u : byte << 23);
    const f32x2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 1),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 3)};
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = p[e >> 1][e & 1] * s;
    if constexpr (DT == NM_F32) {
      float* o = static_cast<float*>(y) + t * ldy + c * 8;
      if (vec) {
        *reinterpret_cast<f32x4*>(o) = f32x4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f32x4*>(o + 4) = f32x4{v[4], v[5], v[6], v[7]};
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = v[e];
      }
    } else {
      uint16_t* o = static_cast<uint16_t*>(y) + t * ldy + c * 8;
      const u32x4 h = {pack_half2<DT>(v[0], v[1]), pack_half2<DT>(v[2], v[3]), pack_half2<DT>(v[4], v[5]),
                       pack_half2<DT>(v[6], v[7])};
      if (vec) {
        *reinterpret_cast<u32x4*>(o) = h;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = uint16_t(h[e >> 1] >> (16 * (e & 1)));
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Product for few tokens: bound by streaming the weight.  A wave owns 16 RB rows x
// 16 NT tokens; the 8 waves of a workgroup take KS shares of K (added in wave order
// in LDS) and 8 / KS blocks of rows.  Operands go straight into registers: a lane
// quarter takes 64 consecutive columns of a panel (two blocks, 32 bytes of values,
// 2 of scales) for two products, so rows are read in whole 128-byte lines.
// 7 tokens on 11008 x 4096: 8.5 us, 2.9 TB/s (24 MB: launch, one round trip and the sum
// over the waves are half of it).
// ---------------------------------------------------------------------------
struct MxDims {
  int E, R, K, T, tilesR;
  int64_t ldy;
};

constexpr int kFewWaves = 8;

template <int OUT, int RB, int NT, int U>
__global__ __launch_bounds__(kFewWaves * 64) void mx_few_kernel(const uint8_t* __restrict__ wq,
                                                                const uint8_t* __restrict__ ws,
                                                                const uint8_t* __restrict__ xq,
                                                                const uint8_t* __restrict__ xs,
                                                                const int32_t* __restrict__ offsets, MxDims d, int ks,
                                                                void* __restrict__ Y) {
  __shared__ f32x4 part[kFewWaves][RB * NT][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const int tile = __builtin_amdgcn_readfirstlane(blockIdx.x / d.tilesR);
  // its share of K and its rows (ks is a power of two)
  const int share = wave & (ks - 1);
  const int r0 = (((int(blockIdx.x) - tile * d.tilesR) * kFewWaves + wave - share) >> __builtin_ctz(ks)) * (16 * RB);
  GroupTile g{0, tile * 16 * NT, d.T};
  if (offsets && !group_find(offsets, d.E, d.T, 16 * NT, tile, g)) return;
  const int row_bytes = d.K >> 1, panels = (d.K + 255) >> 8;
  const int toks = min(16 * NT, g.t1 - g.t0);
  // (clamping to two sides is a vector operation: back to a scalar for the descriptors)
  const int rows = __builtin_amdgcn_readfirstlane(max(min(16 * RB, d.R - r0), 0));
  // Loads past the rows, the tokens or K read zeros: their offsets are selected, not
  // branched on (behind branches the loads of a unit waited for those before them).
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(wq + (int64_t(g.e) * d.R + r0) * row_bytes, uint32_t(rows * row_bytes));
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(xq + int64_t(g.t0) * row_bytes, uint32_t(toks * row_bytes));
  const uint32_t wstep = uint32_t(d.R) * 8u, xstep = uint32_t(d.T) * 8u;   // from a panel's scales to the next's
  const __amdgpu_buffer_rsrc_t rws = make_rsrc(ws + int64_t(g.e) * panels * wstep, uint32_t(panels) * wstep);
  const __amdgpu_buffer_rsrc_t rxs = make_rsrc(xs, uint32_t(panels) * xstep);
  const int per = (panels + ks - 1) / ks;
  const int u_end = min(panels, (share + 1) * per);

  f32x4 acc[RB][NT];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Batch {
    u32x4 a[U][RB][2], b[U][NT][2];
    uint32_t sa[U][RB], sb[U][NT];
  };
  auto load = [&](int u0, Batch& s) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (u0 + u) * 256 + lq * 64;
      const bool on0 = (u0 + u < u_end) & (k < d.K), on1 = on0 & (k + 32 < d.K);   // the two blocks
      auto take = [&](__amdgpu_buffer_rsrc_t r, __amdgpu_buffer_rsrc_t rs, int row, bool on, uint32_t sc,
                      u32x4 (&v)[2], uint32_t& scales) {
        const uint32_t o = uint32_t(row * row_bytes + (k >> 1));
        v[0] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, live_offset(on & on0, o), 0, 0));
        v[1] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, live_offset(on & on1, o + 16u), 0, 0));
        scales = uint16_t(__builtin_amdgcn_raw_buffer_load_b16(rs, live_offset(on & on0, sc + 2u * lq), 0, 0));
      };
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        const int r = i * 16 + li;
        take(rw, rws, r, r < rows, uint32_t(u0 + u) * wstep + uint32_t(r0 + r) * 8u, s.a[u][i], s.sa[u][i]);
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int t = j * 16 + li;
        take(rx, rxs, t, t < toks, uint32_t(u0 + u) * xstep + uint32_t(g.t0 + t) * 8u, s.b[u][j], s.sb[u][j]);
      }
    }
  };
  auto multiply = [&](int u0, Batch& s) {
    // a block past K: zeros already, and the scale 1 whatever the panel holds there
    if (d.K & 255) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if ((u0 + u) * 256 + lq * 64 + 32 >= d.K) {
#pragma unroll
          for (int i = 0; i < RB; ++i) s.sa[u][i] = (s.sa[u][i] & 0xFFu) | 0x7F00u;
#pragma unroll
          for (int j = 0; j < NT; ++j) s.sb[u][j] = (s.sb[u][j] & 0xFFu) | 0x7F00u;
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          acc[i][j] = mfma_fp4<0, 0>(s.a[u][i][0], s.b[u][j][0], acc[i][j], s.sa[u][i], s.sb[u][j]);
          acc[i][j] = mfma_fp4<1, 1>(s.a[u][i][1], s.b[u][j][1], acc[i][j], s.sa[u][i], s.sb[u][j]);
        }
  };
  for (int u = share * per; u < u_end; u += U) {
    Batch b;
    load(u, b);
    __builtin_amdgcn_sched_barrier(0);   // every load goes out before the first product
    multiply(u, b);
  }
  auto store = [&](int f, const f32x4& sum) {   // fragment f of the wave's rows
    const int t = (f % NT) * 16 + li, r = r0 + (f / NT) * 16 + lq * 4;
    if (t >= toks || r >= d.R) return;
    const int64_t o = int64_t(g.t0 + t) * d.ldy + r;
    const bool whole = (d.ldy & 3) == 0 && r + 3 < d.R;
    if constexpr (OUT == NM_F32) {
      float* y = static_cast<float*>(Y) + o;
      if (whole) *reinterpret_cast<f32x4*>(y) = sum;
      else for (int e = 0; e < 4 && r + e < d.R; ++e) y[e] = sum[e];
    } else {
      uint16_t* y = static_cast<uint16_t*>(Y) + o;
      const u32x2 h = {pack_half2<OUT>(sum[0], sum[1]), pack_half2<OUT>(sum[2], sum[3])};
      if (whole) *reinterpret_cast<u32x2*>(y) = h;
      else for (int e = 0; e < 4 && r + e < d.R; ++e) y[e] = uint16_t(h[e >> 1] >> (16 * (e & 1)));
    }
  };
  if (ks == 1) {
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) store(i * NT + j, acc[i][j]);
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
    store(f, sum);
  }
}

// ---------------------------------------------------------------------------
// Product for many tokens: BM rows of W x BN tokens a workgroup, both operands
// staged in LDS by direct loads in steps of 256 columns (128 bytes a row), two
// stages, fragments through two register sets: while one half step (128 columns,
// one instruction deep) is multiplied, the next half's fragments are read and the
// loads of the step after next are issued between the products, in chunks that
// scheduling barriers keep in order.  A stage is free once its second half is in
// registers, at mid-step, where the one barrier a step stands.
//
// Slot (row, 16-byte chunk c) of a stage sits at row*8 + (c ^ (row & 7)).  A chunk
// is one block of 32 values.  The order of the reduction is free, so half h of a
// step takes chunk 2q + h in lane quarter q: the two scale bytes a lane needs for
// a row and step are neighbours, one 16-bit read, and the product's own byte
// select picks the half's.  Two fragments' scales share a register.
//
// Columns past K (the last step's): chunks that reread chunk 0 and enter as zeros
// with the scale 1, whatever the panel holds there.  Rows past R and tokens past
// the tile's end reread the last one and are not stored.
// 4096 x 11008 x 4096 in 256 x 256 tiles: 91 to 98 us, 3.8 to 4.1 PFLOP/s (the instruction
// alone, from registers: 8.4), 688 tiles in 2.7 rounds of the chip.  The matrix cores are
// busy 33% of the time, LDS 31%, near half of that with bank conflicts; a wave issues 35%
// of its time, waits for its turn 37%, for data or the barrier 28%.  1999 rows of 7 experts
// of 2816 x 4096 in 128 x 128 tiles: 25 us, 1.9 PFLOP/s.
// ---------------------------------------------------------------------------
template <int BM_, int BN_, int WM_, int WN_>
struct MxTile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int WAVES = WM * WN, THREADS = WAVES * 64;
  static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
  static constexpr int DATA = (BM + BN) * 128, SCALES = (BM + BN) * 8;
  static constexpr int STAGE = DATA + SCALES, LDS = 2 * STAGE;
  static constexpr int LP = BM / 8 / WAVES, LQ = BN / 8 / WAVES;   // direct loads a wave issues a step
  static constexpr int LS = (BM + BN) * 2 / THREADS;
  static_assert(LP * 8 * WAVES == BM && LQ * 8 * WAVES == BN && LS * THREADS == (BM + BN) * 2, "whole loads");
  static_assert((LP + LQ) % FM == 0 && LS <= FM && FM % 2 == 0 && FN % 2 == 0 && FN <= 2 * FM, "chunks of a half");
};

template <int N, int I = 0, class F>
__device__ inline void static_for(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<N, I + 1>(f);
  }
}

struct MxTileDims {
  int R, K, T, tilesR, tilesT, group;
  int64_t ldy;
};

template <int OUT, class C>
__global__ __launch_bounds__(C::THREADS, 2) void mx_tile_kernel(
    const uint8_t* __restrict__ wq, const uint8_t* __restrict__ ws, const uint8_t* __restrict__ xq,
    const uint8_t* __restrict__ xs, GroupRows experts, MxTileDims d, void* __restrict__ Y) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const int wm = wave / C::WN, wn = wave % C::WN;
  int tt, tr;
  grouped_tile(xcd_tile(blockIdx.x, gridDim.x), d.tilesT, d.tilesR, d.group, tt, tr);
  GroupTile g;
  if (!experts.tile(tt, d.T, C::BN, g)) return;
  const int r0 = tr * C::BM;
  const int row_bytes = d.K >> 1, steps = (d.K + 255) >> 8;
  const int rem = d.K - (steps - 1) * 256;   // columns of the last step
  const int rlast = min(C::BM, d.R - r0) - 1, tlast = min(C::BN, g.t1 - g.t0) - 1;

  const __amdgpu_buffer_rsrc_t rw = make_rsrc(wq + (int64_t(g.e) * d.R + r0) * row_bytes);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(xq + int64_t(g.t0) * row_bytes);
  const __amdgpu_buffer_rsrc_t rws = make_rsrc(ws + (int64_t(g.e) * steps * d.R + r0) * 8);
  const __amdgpu_buffer_rsrc_t rxs = make_rsrc(xs + int64_t(g.t0) * 8);

  // direct loads: 0 .. LP-1 rows of W, then tokens, 8 rows each
  const uint32_t chunk = uint32_t((lane & 7) ^ ((lane >> 3) & 7));
  uint32_t off[C::LP + C::LQ];
#pragma unroll
  for (int j = 0; j < C::LP; ++j)
    off[j] = uint32_t(min((wave * C::LP + j) * 8 + (lane >> 3), rlast)) * uint32_t(row_bytes) + chunk * 16u;
#pragma unroll
  for (int j = 0; j < C::LQ; ++j)
    off[C::LP + j] = uint32_t(min((wave * C::LQ + j) * 8 + (lane >> 3), tlast)) * uint32_t(row_bytes) + chunk * 16u;
  // and the scales, a dword (half a row's eight) a lane: whole waves of W's rows, then of tokens
  uint32_t soff[C::LS];
  bool s_is_w[C::LS];
#pragma unroll
  for (int j = 0; j < C::LS; ++j) {
    const int row = (wave * C::LS + j) * 32 + (lane >> 1);
    s_is_w[j] = (wave * C::LS + j) * 32 < C::BM;
    soff[j] = uint32_t(s_is_w[j] ? min(row, rlast) : min(row - C::BM, tlast)) * 8u + uint32_t(lane & 1) * 4u;
  }
  const uint32_t wstep = uint32_t(d.R) * 8u, xstep = uint32_t(d.T) * 8u;

  auto last_back = [&](int s) { return s == steps - 1 && int(chunk) * 32 >= rem ? chunk * 16u : 0u; };
  auto issue = [&](auto j_c, int s, uint32_t back, unsigned char* st) {
    constexpr int j = decltype(j_c)::value;
    if constexpr (j < C::LP)
      dma16(rw, off[j] - back, uint32_t(s) * 128u, st + (wave * C::LP + j) * 1024);
    else
      dma16(rx, off[j] - back, uint32_t(s) * 128u, st + C::BM * 128 + (wave * C::LQ + j - C::LP) * 1024);
  };
  auto issue_scale = [&](auto j_c, int s, unsigned char* st) {
    constexpr int j = decltype(j_c)::value;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(s_is_w[j] ? rws : rxs, (lds_byte*)(st + C::DATA + (wave * C::LS + j) * 256), 4,
                                             int(soff[j]), int(uint32_t(s) * (s_is_w[j] ? wstep : xstep)), 0, 0);
  };

  f32x4 acc[C::FM][C::FN];
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // fragment addresses: fragment i's differs from fragment 0's by a constant
  const int prow = wm * C::FM * 16 + li, qrow = wn * C::FN * 16 + li;
  int pa[2], qa[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    pa[h] = (prow * 8 + ((2 * lq + h) ^ (prow & 7))) * 16;
    qa[h] = C::BM * 128 + (qrow * 8 + ((2 * lq + h) ^ (qrow & 7))) * 16;
  }
  const int psc = C::DATA + prow * 8 + 2 * lq, qsc = C::DATA + C::BM * 8 + qrow * 8 + 2 * lq;
  auto read_p = [&](const unsigned char* st, int h, int i) {
    return *reinterpret_cast<const u32x4*>(st + pa[h] + i * 2048);
  };
  auto read_q = [&](const unsigned char* st, int h, int j) {
    return *reinterpret_cast<const u32x4*>(st + qa[h] + j * 2048);
  };
  auto read_pair = [&](const unsigned char* p) {   // two fragments' scales, 16 rows apart
    const uint32_t lo = *reinterpret_cast<const uint16_t*>(p), hi = *reinterpret_cast<const uint16_t*>(p + 128);
    return lo | hi << 16;
  };

  u32x4 a0[C::FM], b0[C::FN], a1[C::FM], b1[C::FN];
  uint32_t sa[C::FM / 2], sb[C::FN / 2], na[C::FM / 2], nb[C::FN / 2];

  // One half step: products on (ca, cb) with byte H of the scales; with READ,
  // fragments of half RH of stage rst into (ra, rb), and for RH = 0 the scales of
  // that stage; with LOAD, the loads of step ls into stage lst.
  auto half = [&](auto h_c, auto read_c, auto load_c, const u32x4 (&ca)[C::FM], const u32x4 (&cb)[C::FN],
                  u32x4 (&ra)[C::FM], u32x4 (&rb)[C::FN], const unsigned char* rst, int ls, uint32_t back,
                  unsigned char* lst) {
    constexpr int H = decltype(h_c)::value, RH = H ^ 1;
    constexpr bool READ = decltype(read_c)::value, LOAD = decltype(load_c)::value;
    static_for<C::FM>([&](auto k_c) {
      constexpr int k = decltype(k_c)::value;
      // reads in the first half of the chunks (the next half step needs them right
      // at its start), loads spread over all
      if constexpr (READ && k < C::FM / 2) {
        constexpr int per = 2 * C::FN / C::FM;
#pragma unroll
        for (int j = 0; j < per; ++j) rb[k * per + j] = read_q(rst, RH, k * per + j);
        ra[2 * k] = read_p(rst, RH, 2 * k);
        ra[2 * k + 1] = read_p(rst, RH, 2 * k + 1);
        if constexpr (RH == 0) {
          na[k] = read_pair(rst + psc + k * 256);
          if constexpr (k < C::FN / 2) nb[k] = read_pair(rst + qsc + k * 256);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      static_for<C::FN>([&](auto j_c) {
        constexpr int j = decltype(j_c)::value;
        acc[k][j] = mfma_fp4<(k & 1) * 2 + H, (j & 1) * 2 + H>(ca[k], cb[j], acc[k][j], sa[k / 2], sb[j / 2]);
      });
      if constexpr (LOAD) {
        constexpr int per = (C::LP + C::LQ) / C::FM;
        static_for<per>([&](auto u_c) {
          issue(std::integral_constant<int, k * per + decltype(u_c)::value>{}, ls, back, lst);
        });
        if constexpr (k < C::LS) issue_scale(k_c, ls, lst);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  using yes = std::integral_constant<bool, true>;
  using no = std::integral_constant<bool, false>;
  using h0 = std::integral_constant<int, 0>;
  using h1 = std::integral_constant<int, 1>;
  auto take_scales = [&] {
#pragma unroll
    for (int i = 0; i < C::FM / 2; ++i) sa[i] = na[i];
#pragma unroll
    for (int j = 0; j < C::FN / 2; ++j) sb[j] = nb[j];
  };
  // the last step's chunks past K: zeros, and the scale 1 in half h's byte
  auto trim = [&](u32x4 (&a)[C::FM], u32x4 (&b)[C::FN], int h) {
    if ((2 * lq + h) * 32 < rem) return;
    const uint32_t keep = h ? 0x00FF00FFu : 0xFF00FF00u, one = h ? 0x7F007F00u : 0x007F007Fu;
#pragma unroll
    for (int i = 0; i < C::FM; ++i) a[i] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < C::FN; ++j) b[j] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < C::FM / 2; ++i) sa[i] = (sa[i] & keep) | one;
#pragma unroll
    for (int j = 0; j < C::FN / 2; ++j) sb[j] = (sb[j] & keep) | one;
  };
  auto load_all = [&](int s, unsigned char* st) {
    const uint32_t back = last_back(s);
    static_for<C::LP + C::LQ>([&](auto j_c) { issue(j_c, s, back, st); });
    static_for<C::LS>([&](auto j_c) { issue_scale(j_c, s, st); });
  };

  // steps 0 and 1 in stages 0 and 1, the first half step in set 0
  load_all(0, smem);
  load_all(min(1, steps - 1), smem + C::STAGE);
  wait_vmcnt<C::LP + C::LQ + C::LS>();
  barrier_no_fence();
#pragma unroll
  for (int i = 0; i < C::FM; ++i) a0[i] = read_p(smem, 0, i);
#pragma unroll
  for (int j = 0; j < C::FN; ++j) b0[j] = read_q(smem, 0, j);
#pragma unroll
  for (int i = 0; i < C::FM / 2; ++i) sa[i] = read_pair(smem + psc + i * 256);
#pragma unroll
  for (int j = 0; j < C::FN / 2; ++j) sb[j] = read_pair(smem + qsc + j * 256);
  for (int s = 0; s < steps - 1; ++s) {
    unsigned char* here = smem + (s & 1) * C::STAGE;
    unsigned char* next = smem + ((s & 1) ^ 1) * C::STAGE;
    half(h0{}, yes{}, no{}, a0, b0, a1, b1, here, 0, 0u, nullptr);
    wait_vmcnt<0>();
    wait_lgkm0();
    barrier_no_fence();
    const int ls = min(s + 2, steps - 1);   // past the end: the last step again, which nothing reads
    half(h1{}, yes{}, yes{}, a1, b1, a0, b0, next, ls, last_back(ls), here);
    take_scales();
  }
  if (rem < 256) trim(a0, b0, 0);
  half(h0{}, yes{}, no{}, a0, b0, a1, b1, smem + ((steps - 1) & 1) * C::STAGE, 0, 0u, nullptr);
  if (rem < 256) trim(a1, b1, 1);
  half(h1{}, no{}, no{}, a1, b1, a0, b0, nullptr, 0, 0u, nullptr);
  wait_vmcnt<0>();
  wait_lgkm0();
  barrier_no_fence();   // no load is in flight and no stage is read any more

  const int wr0 = wm * C::FM * 16, wt0 = wn * C::FN * 16;   // the wave's corner in the tile
  if constexpr (OUT == NM_F32) {
    const bool vec = (d.ldy & 3) == 0;
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
      const int t = wt0 + j * 16 + li;
      if (t > tlast) continue;
      float* y = static_cast<float*>(Y) + int64_t(g.t0 + t) * d.ldy + r0;
#pragma unroll
      for (int i = 0; i < C::FM; ++i) {
        const int r = wr0 + i * 16 + lq * 4;
        if (vec && r + 3 <= rlast) *reinterpret_cast<f32x4*>(y + r) = acc[i][j];
        else for (int e = 0; e < 4 && r + e <= rlast; ++e) y[r + e] = acc[i][j][e];
      }
    }
  } else {
    // 16-bit results pass through the wave's own part of LDS, token-major, and
    // leave in whole runs of its FM*16 rows (chunk c of token t at c ^ t)
    constexpr int CH = C::FM * 2;   // 16-byte chunks a token
    unsigned char* mine = smem + wave * (C::FN * 16 * CH * 16);
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int i = 0; i < C::FM; ++i) {
        const u32x2 h = {pack_half2<OUT>(acc[i][j][0], acc[i][j][1]), pack_half2<OUT>(acc[i][j][2], acc[i][j][3])};
        const int t = j * 16 + li, c = (2 * i + (lq >> 1)) ^ (t & (CH - 1));
        *reinterpret_cast<u32x2*>(mine + (t * CH + c) * 16 + (lq & 1) * 8) = h;
      }
    wait_lgkm0();
    asm volatile("" ::: "memory");
    const bool vec = (d.ldy & 7) == 0;
    const int c = lane % CH, r = wr0 + c * 8;
#pragma unroll
    for (int it = 0; it < C::FN * 16 * CH / 64; ++it) {
      const int t = it * (64 / CH) + lane / CH;
      const u32x4 v = *reinterpret_cast<const u32x4*>(mine + (t * CH + (c ^ (t & (CH - 1)))) * 16);
      if (wt0 + t > tlast) continue;
      uint16_t* y = static_cast<uint16_t*>(Y) + int64_t(g.t0 + wt0 + t) * d.ldy + r0 + r;
      if (vec && r + 7 <= rlast) {
        *reinterpret_cast<u32x4*>(y) = v;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t w = v[e >> 1];
          if (r + e <= rlast) y[e] = uint16_t(w >> (16 * (e & 1)));
        }
      }
    }
  }
}

using MxLarge = MxTile<256, 256, 2, 4>;
using MxMiddle = MxTile<128, 128, 2, 2>;

inline unsigned grid_of(int64_t items) {
  const int64_t blocks = (items + 255) / 256;
  return unsigned(blocks < 65536 ? blocks : 65536);
}

// Whether every row of every matrix at p begins on 16 bytes.
inline bool rows_aligned(const MxQuantArgs& a, const void* p, int64_t e) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (a.ldx * e) % 16 == 0 && (a.E == 1 || (a.stride * e) % 16 == 0);
}

template <int DT>
hipError_t quantize_dt(const MxQuantArgs& a, hipStream_t s) {
  const bool vec = rows_aligned(a, a.x, DT == NM_F32 ? 4 : 2);
  hipLaunchKernelGGL(mx_quantize_kernel<DT>, dim3(grid_of(a.T * ((a.K + 255) / 256) * 32), unsigned(a.E)), dim3(256), 0,
                     s, a.x, a.T, a.K, a.ldx, a.stride, vec, reinterpret_cast<uint32_t*>(a.q), a.scale);
  return hipGetLastError();
}

template <int DT>
hipError_t dequantize_dt(const MxQuantArgs& a, hipStream_t s) {
  const bool vec = rows_aligned(a, a.y, DT == NM_F32 ? 4 : 2);
  hipLaunchKernelGGL(mx_dequantize_kernel<DT>, dim3(grid_of(a.T * (a.K / 8)), unsigned(a.E)), dim3(256), 0, s,
                     reinterpret_cast<const uint32_t*>(a.q), a.scale, a.T, a.K, a.y, a.ldx, a.stride, vec);
  return hipGetLastError();
}

template <int OUT, int RB, int NT, int U>
hipError_t launch_few(const MxArgs& a, hipStream_t s) {
  MxDims d;
  d.E = int(a.E);
  d.R = int(a.R);
  d.K = int(a.K);
  d.T = int(a.T);
  d.ldy = a.ldy;
  // shares of K: until there are 16 waves a compute unit, but none below two panels
  // (11008 x 4096, 7 tokens, 1 / 2 / 4 / 8 shares: 15.6 / 10.1 / 9.7 / 8.4 us)
  const int64_t weights = a.offsets ? std::min(a.E, a.T) : 1, tiles = (a.T / weights + 16 * NT - 1) / (16 * NT);
  const int64_t blocks = (a.R + 16 * RB - 1) / (16 * RB), panels = (a.K + 255) / 256;
  int ks = 1;
  while (ks < kFewWaves && weights * tiles * blocks * ks < 16 * 256 && panels >= 2 * ks) ks *= 2;
  const int64_t rows = 16 * RB * (kFewWaves / ks);
  d.tilesR = int((a.R + rows - 1) / rows);
  const int64_t tilesT = a.offsets ? group_max_tiles(a.T, a.E, 16 * NT) : (a.T + 16 * NT - 1) / (16 * NT);
  if (tilesT * d.tilesR > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL((mx_few_kernel<OUT, RB, NT, U>), dim3(unsigned(tilesT * d.tilesR)), dim3(kFewWaves * 64), 0, s, a.wq,
                     a.ws, a.xq, a.xs, a.offsets, d, ks, a.Y);
  return hipGetLastError();
}

template <int OUT, class C>
hipError_t launch_tiles(const MxArgs& a, hipStream_t s) {
  const int64_t tilesR = (a.R + C::BM - 1) / C::BM;
  const int64_t tilesT = a.offsets ? group_max_tiles(a.T, a.E, C::BN) : (a.T + C::BN - 1) / C::BN;
  if (tilesR * tilesT > 0x7FFFFFFF) return hipErrorInvalidValue;
  MxTileDims d;
  d.R = int(a.R);
  d.K = int(a.K);
  d.T = int(a.T);
  d.tilesR = int(tilesR);
  d.tilesT = int(tilesT);
  d.group = int(std::min<int64_t>(tilesT, 4));
  d.ldy = a.ldy;
  GroupRows rows;
  if (hipError_t e = group_rows(a.offsets, a.E, a.T, C::BN, tilesT, a.workspace, s, rows); e != hipSuccess) return e;
  auto kern = mx_tile_kernel<OUT, C>;
  if (hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(kern), C::LDS); e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3(unsigned(tilesR * tilesT)), dim3(C::THREADS), C::LDS, s, a.wq, a.ws, a.xq, a.xs, rows, d,
                     a.Y);
  return hipGetLastError();
}

// Which kernel: by the rows that a weight meets on average, and, where those fill
// tiles, by whether the largest ones still give every compute unit one.  Both sides of the
// limits, us with inputs in turn, on 11008 x 4096, 4096 x 4096 and 4096 x 11008:
//   rows 16     9.5   9.9    5.3   9.2    9.1  19.0   few1, few2
//        17    13.8   9.8    6.6   9.1   12.8  19.0
//        32    10.5  12.0    9.8  11.4   20.5  23.8   few2, few4
//        33    15.0  11.9    9.7  11.3   19.9  23.8
//        64    13.4  14.6   12.6  14.1   27.5  31.6   few4, middle
//        65    21.5  14.5   12.5  14.1   26.7  31.6
//      1280    41.5  33.0   20.6  27.0   43.9  59.5   middle, large (215, 80, 80 tiles)
//      1536    51.6  57.9   21.1  27.3   47.1  60.7   (258, 96, 96)
//      4096   112.6  91.0   42.6  35.3   99.5  80.1   (688, 256, 256)
// The limits are those of the first: where the weight has fewer rows, the smaller kernel
// of a pair leads beyond its limit.  41 experts of 2816 x 2048: 300 rows, few1 and few2,
// 35.0 and 30.8; 700 rows 49.2 and 32.5; 2600 rows, few4 and middle, 65.9 and 56.9.
enum class MxPick { few1, few2, few4, middle, large };

MxPick pick(int64_t E, int64_t R, int64_t T, bool grouped) {
  const int64_t weights = grouped ? std::min(E, T) : 1, rows = T / weights;
  if (rows <= 16) return MxPick::few1;
  if (rows <= 32) return MxPick::few2;
  if (rows <= 64) return MxPick::few4;
  const int64_t large = weights * ((rows + 255) / 256) * ((R + 255) / 256);
  return large >= 256 ? MxPick::large : MxPick::middle;
}

template <int OUT>
hipError_t gemm_out(const MxArgs& a, hipStream_t s) {
  switch (pick(a.E, a.R, a.T, a.offsets != nullptr)) {
    case MxPick::few1: return launch_few<OUT, 1, 1, 2>(a, s);
    case MxPick::few2: return launch_few<OUT, 4, 2, 1>(a, s);
    case MxPick::few4: return launch_few<OUT, 4, 4, 1>(a, s);
    case MxPick::middle: return launch_tiles<OUT, MxMiddle>(a, s);
    default: return launch_tiles<OUT, MxLarge>(a, s);
  }
}

}  // namespace

// A stack's matrices, as many a launch as the second dimension of its grid takes.
template <class F>
static hipError_t over_stack(MxQuantArgs a, const F& launch) {
  const int64_t e = a.dtype == NM_F32 ? 4 : 2, E = a.E;
  for (int64_t m = 0; m < E; m += kGroupMaxExperts) {
    a.E = std::min(E - m, kGroupMaxExperts);
    if (hipError_t err = launch(a); err != hipSuccess) return err;
    if (a.x) a.x = static_cast<const unsigned char*>(a.x) + a.E * a.stride * e;
    if (a.y) a.y = static_cast<unsigned char*>(a.y) + a.E * a.stride * e;
    a.q += a.E * a.T * (a.K / 2);
    a.scale += a.E * ((a.K + 255) / 256) * a.T * 8;
  }
  return hipSuccess;
}

hipError_t launch_mx_quantize(const MxQuantArgs& a, hipStream_t s) {
  return over_stack(a, [s](const MxQuantArgs& a) {
    if (a.dtype == NM_F32) return quantize_dt<NM_F32>(a, s);
    return a.dtype == NM_F16 ? quantize_dt<NM_F16>(a, s) : quantize_dt<NM_BF16>(a, s);
  });
}

hipError_t launch_mx_dequantize(const MxQuantArgs& a, hipStream_t s) {
  return over_stack(a, [s](const MxQuantArgs& a) {
    if (a.dtype == NM_F32) return dequantize_dt<NM_F32>(a, s);
    return a.dtype == NM_F16 ? dequantize_dt<NM_F16>(a, s) : dequantize_dt<NM_BF16>(a, s);
  });
}

size_t mx_workspace(int64_t E, int64_t R, int64_t T, bool grouped) {
  const MxPick p = pick(E, R, T, grouped);
  if (!grouped || (p != MxPick::middle && p != MxPick::large)) return 0;
  return group_rows_bytes(E, group_max_tiles(T, E, p == MxPick::middle ? MxMiddle::BN : MxLarge::BN));
}

hipError_t launch_mx_gemm(const MxArgs& a, hipStream_t s) {
  if (a.out_dtype == NM_F32) return gemm_out<NM_F32>(a, s);
  return a.out_dtype == NM_F16 ? gemm_out<NM_F16>(a, s) : gemm_out<NM_BF16>(a, s);
}

}  // namespace nm
