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
// NaN gets the exponent byte 255, which makes all of it NaN.
// Bound by its bytes: 2 (or 4) read and 17/32 written a value.
// ---------------------------------------------------------------------------
template <int DT>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const void* __restrict__ x, int64_t T, int64_t K, int64_t ldx,
                                                          bool vec, uint32_t* __restrict__ q,
                                                          uint8_t* __restrict__ scale) {
  const int64_t per_row = K / 8;   // shares of 8 values
  const int64_t panels = (K + 255) / 256;
  const int64_t total = T * panels * 32;   // whole panels: the last one's missing blocks get the byte 0
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
// and fp32 where they fit its range).
template <int DT>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint32_t* __restrict__ q,
                                                            const uint8_t* __restrict__ scale, int64_t T, int64_t K,
                                                            void* __restrict__ y, int64_t ldy, bool vec) {
  const int64_t per_row = K / 8;
  const int64_t total = T * per_row;
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
// Product for few tokens (and any other shape): a workgroup of 8 waves owns
// 16 RB rows x 16 NT tokens, the waves take shares of K, operands go straight
// into registers, and the partial tiles are added in wave order.
// ---------------------------------------------------------------------------
struct MxDims {
  int E, R, K, T, tilesR;
  int64_t ldy;
};

constexpr int kFewWaves = 8;
constexpr uint32_t kDead = 0xFFFFFFF0u;   // no descriptor covers it: reads zeros

template <int OUT, int RB, int NT>
__global__ __launch_bounds__(kFewWaves * 64) void mx_few_kernel(const uint8_t* __restrict__ wq,
                                                                const uint8_t* __restrict__ ws,
                                                                const uint8_t* __restrict__ xq,
                                                                const uint8_t* __restrict__ xs,
                                                                const int32_t* __restrict__ offsets, MxDims d,
                                                                void* __restrict__ Y) {
  __shared__ f32x4 part[kFewWaves][RB * NT][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const int tile = blockIdx.x / d.tilesR;
  const int r0 = (blockIdx.x - tile * d.tilesR) * (16 * RB);
  GroupTile g{0, tile * 16 * NT, d.T};
  if (offsets && !group_find(offsets, d.E, d.T, 16 * NT, tile, g)) return;
  const int row_bytes = d.K >> 1, panels = (d.K + 255) >> 8, blocks = d.K >> 5;
  const int rows = min(16 * RB, d.R - r0), toks = min(16 * NT, g.t1 - g.t0);
  const __amdgpu_buffer_rsrc_t rw =
      make_rsrc(wq + (int64_t(g.e) * d.R + r0) * row_bytes, uint32_t(rows) * uint32_t(row_bytes));
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(xq + int64_t(g.t0) * row_bytes, uint32_t(toks) * uint32_t(row_bytes));
  const uint8_t* sw = ws + (int64_t(g.e) * panels * d.R + r0) * 8;
  const uint8_t* sx = xs + int64_t(g.t0) * 8;
  const int64_t wstep = int64_t(d.R) * 8, xstep = int64_t(d.T) * 8;   // bytes from a panel to the next

  const int steps = (d.K + 127) >> 7;
  const int share = (steps + kFewWaves - 1) / kFewWaves;
  const int s_end = min(steps, (wave + 1) * share);
  f32x4 acc[RB][NT];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  constexpr int U = 4 / (NT > 2 ? 2 : 1);
  for (int s0 = wave * share; s0 < s_end; s0 += U) {
    u32x4 a[U][RB], b[U][NT];
    uint32_t sa[U][RB], sb[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int block = (s0 + u) * 4 + lq;
      const bool live = s0 + u < s_end && block < blocks;
      const int64_t panel = block >> 3;
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        const int row = i * 16 + li;
        const bool on = live && row < rows;
        a[u][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                rw, on ? uint32_t(row * row_bytes + block * 16) : kDead, 0, 0));
        sa[u][i] = on ? sw[panel * wstep + row * 8 + (block & 7)] : 0u;
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int t = j * 16 + li;
        const bool on = live && t < toks;
        b[u][j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                rx, on ? uint32_t(t * row_bytes + block * 16) : kDead, 0, 0));
        sb[u][j] = on ? sx[panel * xstep + t * 8 + (block & 7)] : 0u;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = mfma_fp4<0, 0>(a[u][i], b[u][j], acc[i][j], sa[u][i], sb[u][j]);
  }
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) part[wave][i * NT + j][lane] = acc[i][j];
  __syncthreads();
  if (wave >= RB * NT) return;
  f32x4 sum = part[0][wave][lane];
#pragma unroll
  for (int w = 1; w < kFewWaves; ++w) sum += part[w][wave][lane];
  const int t = (wave % NT) * 16 + li, r = (wave / NT) * 16 + lq * 4;
  if (t >= toks || r >= rows) return;
  const int64_t o = int64_t(g.t0 + t) * d.ldy + r0 + r;
  const bool whole = (d.ldy & 3) == 0 && r + 3 < rows;
  if constexpr (OUT == NM_F32) {
    float* y = static_cast<float*>(Y) + o;
    if (whole) *reinterpret_cast<f32x4*>(y) = sum;
    else for (int e = 0; e < 4 && r + e < rows; ++e) y[e] = sum[e];
  } else {
    uint16_t* y = static_cast<uint16_t*>(Y) + o;
    const u32x2 h = {pack_half2<OUT>(sum[0], sum[1]), pack_half2<OUT>(sum[2], sum[3])};
    if (whole) *reinterpret_cast<u32x2*>(y) = h;
    else for (int e = 0; e < 4 && r + e < rows; ++e) y[e] = uint16_t(h[e >> 1] >> (16 * (e & 1)));
  }
}

inline unsigned grid_of(int64_t items) {
  const int64_t blocks = (items + 255) / 256;
  return unsigned(blocks < 65536 ? blocks : 65536);
}

template <int DT>
hipError_t quantize_dt(const MxQuantArgs& a, hipStream_t s) {
  const int64_t e = DT == NM_F32 ? 4 : 2;
  const bool vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && (a.ldx * e) % 16 == 0;
  hipLaunchKernelGGL(mx_quantize_kernel<DT>, dim3(grid_of(a.T * ((a.K + 255) / 256) * 32)), dim3(256), 0, s, a.x, a.T,
                     a.K, a.ldx, vec, reinterpret_cast<uint32_t*>(a.q), a.scale);
  return hipGetLastError();
}

template <int DT>
hipError_t dequantize_dt(const MxQuantArgs& a, hipStream_t s) {
  const int64_t e = DT == NM_F32 ? 4 : 2;
  const bool vec = reinterpret_cast<uintptr_t>(a.y) % 16 == 0 && (a.ldx * e) % 16 == 0;
  hipLaunchKernelGGL(mx_dequantize_kernel<DT>, dim3(grid_of(a.T * (a.K / 8))), dim3(256), 0, s,
                     reinterpret_cast<const uint32_t*>(a.q), a.scale, a.T, a.K, a.y, a.ldx, vec);
  return hipGetLastError();
}

template <int OUT, int RB, int NT>
hipError_t launch_few(const MxArgs& a, hipStream_t s) {
  MxDims d;
  d.E = int(a.E);
  d.R = int(a.R);
  d.K = int(a.K);
  d.T = int(a.T);
  d.tilesR = int((a.R + 16 * RB - 1) / (16 * RB));
  d.ldy = a.ldy;
  const int64_t tilesT = a.offsets ? group_max_tiles(a.T, a.E, 16 * NT) : (a.T + 16 * NT - 1) / (16 * NT);
  if (tilesT * d.tilesR > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL((mx_few_kernel<OUT, RB, NT>), dim3(unsigned(tilesT * d.tilesR)), dim3(kFewWaves * 64), 0, s, a.wq,
                     a.ws, a.xq, a.xs, a.offsets, d, a.Y);
  return hipGetLastError();
}

template <int OUT>
hipError_t gemm_out(const MxArgs& a, hipStream_t s) {
  const int64_t per = a.T / (a.offsets && a.E < a.T ? a.E : a.offsets ? a.T : 1);
  if (per <= 16) return launch_few<OUT, 1, 1>(a, s);
  if (per <= 32) return launch_few<OUT, 1, 2>(a, s);
  return launch_few<OUT, 2, 4>(a, s);
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantArgs& a, hipStream_t s) {
  if (a.dtype == NM_F32) return quantize_dt<NM_F32>(a, s);
  return a.dtype == NM_F16 ? quantize_dt<NM_F16>(a, s) : quantize_dt<NM_BF16>(a, s);
}

hipError_t launch_mx_dequantize(const MxQuantArgs& a, hipStream_t s) {
  if (a.dtype == NM_F32) return dequantize_dt<NM_F32>(a, s);
  return a.dtype == NM_F16 ? dequantize_dt<NM_F16>(a, s) : dequantize_dt<NM_BF16>(a, s);
}

size_t mx_workspace(int64_t E, int64_t R, int64_t K, int64_t T, bool grouped) { return 0; }

hipError_t launch_mx_gemm(const MxArgs& a, hipStream_t s) {
  if (a.out_dtype == NM_F32) return gemm_out<NM_F32>(a, s);
  return a.out_dtype == NM_F16 ? gemm_out<NM_F16>(a, s) : gemm_out<NM_BF16>(a, s);
}

}  // namespace nm
