// Low-rank adapters of many requests beside a shared N:M projection.
//
// Token t names adapter a = adapter[t] (outside [0, n): none); the packed
// weight W_nm is shared:
//   xa[t]   = A_a x_t                      (shrink: r numbers a token)
//   y_t     = W_nm x_t + s_a B_a xa[t]     (expand)
// and with g_t = dL/dy_t, W_nm frozen:
//   u[t]    = s_a B_a^T g_t                (shrink)
//   dx_t    = W_nm^T g_t + A_a^T u[t]      (expand)
//   dA_a    = sum_{t in a} u[t] x_t^T,   dB_a = s_a sum_{t in a} g_t xa[t]^T.
//
// Tokens of an adapter are found where they lie: a 16-token fragment is
// multiplied once for every adapter that occurs in it, and each token keeps its
// own adapter's result.  Requests whose tokens are adjacent cost one product a
// fragment; any other order is right and costs up to 16.
//
// The shrunk activations are fp32 (nothing between the two products is
// rounded to 16 bits).  All three kernels are bound by reading what they
// multiply: x or g once for the shrink and the gradients, Y once for the
// expand; the adapters themselves are small.
#include "nm_internal.h"
#include "nm_lowrank.h"

namespace nm {
namespace {

// Operand lane (row, quarter): 8 consecutive elements at row + c, zeros past C
// (C a multiple of 8).
__device__ inline u32x4 piece8(const uint16_t* row, int c, int C) {
  if (c >= C) return u32x4{0u, 0u, 0u, 0u};
  return *reinterpret_cast<const u32x4*>(row + c);
}

// ---------------------------------------------------------------------------
// Shrink: V[t][j] = s_a sum_c M_a[j][c] Z[t][c] for 16 tokens x RF*16 ranks.
// A workgroup of 16 waves splits the columns: wave w takes the 64-column steps
// w, w + 16, ..., and the waves' partial tiles are added in LDS in wave order.
// 16 tokens a workgroup keeps enough workgroups for short batches; Z is read
// once (rank tiles past the first reread it from L2).  blockIdx.z deals out
// the adapters that occur among the 16 tokens, so a batch of single tokens
// with an adapter each is not walked one after the other.
// TRANS: M_a is stored [C][r] (B), else [r][C] (A).
// ---------------------------------------------------------------------------
constexpr int kShrinkWaves = 16;

template <int DT, bool TRANS, int RF>
__global__ __launch_bounds__(kShrinkWaves * 64) void adapter_shrink_kernel(
    const int32_t* __restrict__ ids, int n, const uint16_t* __restrict__ M, const float* __restrict__ scale,
    const uint16_t* __restrict__ Z, int64_t ldz, int T, int C, int r, float* __restrict__ V) {
  __shared__ f32x4 part[kShrinkWaves][RF][64];
  const int lane = threadIdx.x & 63, li = lane & 15, lq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = blockIdx.x * 16, r0 = blockIdx.y * (RF * 16);
  const int t = t0 + li;
  const int id = t < T ? ids[t] : -1;
  const bool valid = uint32_t(id) < uint32_t(n);
  // every wave holds the same ids, so the loop and its barriers are uniform
  uint32_t todo = uint32_t(__ballot(valid)) & 0xFFFFu;
  if (blockIdx.z == 0 && wave < RF && !valid && t < T) {   // no adapter: zeros
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = r0 + wave * 16 + lq * 4 + e;
      if (j < r) V[int64_t(t) * r + j] = 0.f;
    }
  }
  const uint16_t* zrow = Z + int64_t(min(t, T - 1)) * ldz;
  const int steps = (C + 63) / 64;
  for (uint32_t d = 0; todo; ++d) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
    const bool mine = id == a;
    todo &= ~uint32_t(__ballot(mine));
    if (d % gridDim.z != blockIdx.z) continue;
    const uint16_t* Ma = M + int64_t(a) * r * C;
    f32x4 acc[RF];
#pragma unroll
    for (int f = 0; f < RF; ++f) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s = wave; s < steps; s += kShrinkWaves) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = s * 64 + h * 32 + lq * 8;
        const u32x4 z = piece8(zrow, c, C);
#pragma unroll
        for (int f = 0; f < RF; ++f) {
          const int j = min(r0 + f * 16 + li, r - 1);   // rows past r: results not stored
          u32x4 m = {0u, 0u, 0u, 0u};
          if constexpr (TRANS) {
            if (c < C) {
              const uint16_t* p = Ma + int64_t(c) * r + j;
#pragma unroll
              for (int e = 0; e < 8; ++e) m[e >> 1] |= uint32_t(p[e * r]) << (16 * (e & 1));
            }
          } else {
            m = piece8(Ma + int64_t(j) * C, c, C);
          }
          acc[f] = mfma32<DT>(m, z, acc[f]);
        }
      }
    }
#pragma unroll
    for (int f = 0; f < RF; ++f) part[wave][f][lane] = acc[f];
    __syncthreads();
    if (wave < RF) {
      f32x4 sum = part[0][wave][lane];
#pragma unroll
      for (int w = 1; w < kShrinkWaves; ++w) sum += part[w][wave][lane];
      const float sc = scale ? scale[a] : 1.f;
      if (mine && t < T) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = r0 + wave * 16 + lq * 4 + e;
          if (j < r) V[int64_t(t) * r + j] = sum[e] * sc;
        }
      }
    }
    __syncthreads();   // part is free for the next adapter
  }
}

// ---------------------------------------------------------------------------
// Expand: Y[t][c] = base[t][c] + (low-rank term), base fp32 (Y itself or a
// workspace).  A wave takes 16 tokens x 64 columns.
// ---------------------------------------------------------------------------
template <int DT, bool TRANS, int OUT>
__global__ __launch_bounds__(256) void adapter_expand_kernel(LowRank p, const float* base, int64_t ldb, void* Y,
                                                             int64_t ldy) {
  const int lane = threadIdx.x & 63, li = lane & 15, lq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = blockIdx.x * 16, c0 = blockIdx.y * 256 + wave * 64;
  const int t = t0 + li;
  f32x4 acc[4];
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int c = c0 + 16 * f + 4 * lq;
    if (t >= p.T) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < p.C) acc[f][e] = base[int64_t(t) * ldb + c + e];
  }
  lowrank_term<DT, TRANS, 4>(p, t0, c0, [&](int f, const f32x4& d, bool mine) {
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[f][e] = mine ? acc[f][e] + d[e] : acc[f][e];
  });
  if (t >= p.T) return;
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    const int c = c0 + 16 * f + 4 * lq;
    if constexpr (OUT == NM_F32) {
      float* y = static_cast<float*>(Y) + int64_t(t) * ldy + c;
      if ((ldy & 3) == 0 && c + 3 < p.C) *reinterpret_cast<f32x4*>(y) = acc[f];
      else
        for (int e = 0; e < 4 && c + e < p.C; ++e) y[e] = acc[f][e];
    } else {
      uint16_t* y = static_cast<uint16_t*>(Y) + int64_t(t) * ldy + c;
      const uint32_t p0 = pack_half2<OUT>(acc[f][0], acc[f][1]), p1 = pack_half2<OUT>(acc[f][2], acc[f][3]);
      if ((ldy & 3) == 0 && c + 3 < p.C) *reinterpret_cast<uint2*>(y) = make_uint2(p0, p1);
      else
        for (int e = 0; e < 4 && c + e < p.C; ++e) y[e] = uint16_t((e < 2 ? p0 : p1) >> (16 * (e & 1)));
    }
  }
}

// ---------------------------------------------------------------------------
// Gradients: D_a[j][c] = s_a sum_{t in a} V[t][j] Z[t][c], written [r][C] (dA,
// Z = x, V = u) or [C][r] (dB, Z = g, V = xa).  A workgroup of 8 waves owns one
// adapter, RF*16 ranks and CF*16 columns; wave w takes the 32-token chunks w,
// w + 8, ... that hold a token of the adapter, and the waves' tiles are added in
// LDS in a fixed order.  Tokens of other adapters enter as zeros in both
// operands (loads are not even made), so an Inf or NaN among them reaches
// nothing.  An adapter without tokens gets zeros.
// ---------------------------------------------------------------------------
constexpr int kGradWaves = 8;

struct GradArgs {
  const int32_t* ids;
  int n;
  const float* scale;   // or null: 1
  const float* V;       // [T][r]
  const uint16_t* Z;    // [T][C]
  int64_t ldz;
  int T, C, r;
  float* out;
  bool rank_minor;      // [C][r] instead of [r][C]
};

template <int DT, int RF, int CF>
__global__ __launch_bounds__(kGradWaves * 64) void adapter_grad_kernel(GradArgs g) {
  __shared__ f32x4 part[kGradWaves / 2][RF * CF][64];
  const int lane = threadIdx.x & 63, li = lane & 15, lq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c0 = blockIdx.x * (CF * 16), r0 = blockIdx.y * (RF * 16), a = blockIdx.z;
  f32x4 acc[RF][CF];
#pragma unroll
  for (int i = 0; i < RF; ++i)
#pragma unroll
    for (int j = 0; j < CF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int chunks = (g.T + 31) / 32;
  for (int k = wave; k < chunks; k += kGradWaves) {
    const int tl = k * 32 + (lane & 31);
    const uint32_t in = uint32_t(__ballot(tl < g.T && g.ids[min(tl, g.T - 1)] == a));
    if (in == 0) continue;
    const uint32_t mine = (in >> (8 * lq)) & 0xFFu;   // this lane's 8 tokens
    const int64_t t0 = int64_t(k) * 32 + 8 * lq;
    u32x4 vp[RF][3];
#pragma unroll
    for (int i = 0; i < RF; ++i) {
      const int j = min(r0 + i * 16 + li, g.r - 1);   // ranks past r: results not stored
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (mine >> e) & 1u ? g.V[(t0 + e) * g.r + j] : 0.f;
      split8(v, vp[i]);
    }
#pragma unroll
    for (int j = 0; j < CF; ++j) {
      const int c = min(c0 + j * 16 + li, g.C - 1);
      u32x4 z = {0u, 0u, 0u, 0u}, zp[operand_count<DT>()];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t x = (mine >> e) & 1u ? g.Z[(t0 + e) * g.ldz + c] : 0u;
        z[e >> 1] |= x << (16 * (e & 1));
      }
      operand_parts<DT>(z, zp);
#pragma unroll
      for (int i = 0; i < RF; ++i) acc[i][j] = mfma_parts(vp[i], zp, acc[i][j]);
    }
  }
  // waves 4..7 onto 0..3, 2..3 onto 0..1, 1 onto 0
#pragma unroll
  for (int half = kGradWaves / 2; half > 0; half >>= 1) {
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int i = 0; i < RF; ++i)
#pragma unroll
        for (int j = 0; j < CF; ++j) part[wave - half][i * CF + j][lane] = acc[i][j];
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int i = 0; i < RF; ++i)
#pragma unroll
        for (int j = 0; j < CF; ++j) acc[i][j] += part[wave][i * CF + j][lane];
    }
    __syncthreads();
  }
  if (wave != 0) return;
  const float s = g.scale ? g.scale[a] : 1.f;
  float* out = g.out + int64_t(a) * g.r * g.C;
#pragma unroll
  for (int i = 0; i < RF; ++i)
#pragma unroll
    for (int j = 0; j < CF; ++j) {
      const int c = c0 + j * 16 + li, q = r0 + i * 16 + lq * 4;
      if (c >= g.C) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (q + e >= g.r) break;
        const int64_t o = g.rank_minor ? int64_t(c) * g.r + q + e : int64_t(q + e) * g.C + c;
        out[o] = acc[i][j][e] * s;
      }
    }
}

template <int DT, bool TRANS>
hipError_t shrink(const int32_t* ids, int64_t n, const uint16_t* M, const float* scale, const uint16_t* Z, int64_t ldz,
                  int64_t T, int64_t C, int64_t r, float* V, hipStream_t s) {
  const unsigned tiles = unsigned((T + 15) / 16);
  // up to 16 adapters side by side while the batch alone does not fill the chip
  const unsigned z = unsigned(tiles <= 8 ? 16 : 1);
  auto go = [&](auto kern, int rf) {
    hipLaunchKernelGGL(kern, dim3(tiles, unsigned((r + rf * 16 - 1) / (rf * 16)), z), dim3(kShrinkWaves * 64), 0, s,
                       ids, int(n), M, scale, Z, ldz, int(T), int(C), int(r), V);
    return hipGetLastError();
  };
  // few tokens: a rank tile a workgroup; many: every rank of the tile, so Z is read once
  if (r <= 16 || tiles <= 8) return go(adapter_shrink_kernel<DT, TRANS, 1>, 1);
  if (r <= 32) return go(adapter_shrink_kernel<DT, TRANS, 2>, 2);
  return go(adapter_shrink_kernel<DT, TRANS, 4>, 4);
}

template <int DT, bool TRANS>
hipError_t expand(const LowRank& p, const float* base, int64_t ldb, void* Y, int64_t ldy, int out_dtype,
                  hipStream_t s) {
  const dim3 grid(unsigned((p.T + 15) / 16), unsigned((p.C + 255) / 256));
  if (out_dtype == NM_F32)
    hipLaunchKernelGGL((adapter_expand_kernel<DT, TRANS, NM_F32>), grid, dim3(256), 0, s, p, base, ldb, Y, ldy);
  else
    hipLaunchKernelGGL((adapter_expand_kernel<DT, TRANS, DT>), grid, dim3(256), 0, s, p, base, ldb, Y, ldy);
  return hipGetLastError();
}

template <int DT>
hipError_t gradient(const GradArgs& g, hipStream_t s) {
  auto go = [&](auto kern, int rf, int cf) {
    hipLaunchKernelGGL(kern, dim3(unsigned((g.C + cf * 16 - 1) / (cf * 16)), unsigned((g.r + rf * 16 - 1) / (rf * 16)),
                                  unsigned(g.n)),
                       dim3(kGradWaves * 64), 0, s, g);
    return hipGetLastError();
  };
  if (g.r <= 16) return go(adapter_grad_kernel<DT, 1, 4>, 1, 4);
  if (g.r <= 32) return go(adapter_grad_kernel<DT, 2, 4>, 2, 4);
  return go(adapter_grad_kernel<DT, 4, 4>, 4, 4);
}

template <int DT>
hipError_t forward_dt(const AdapterArgs& a, hipStream_t s) {
  hipError_t e = shrink<DT, false>(a.ids, a.n, a.A, nullptr, a.base.act, a.base.ldx, a.base.T, a.base.K, a.r, a.xa, s);
  if (e != hipSuccess) return e;
  // the product in fp32, in Y itself or in the workspace; then the low-rank term
  SpmmArgs b = a.base;
  if (a.base.out_dtype != NM_F32) {
    b.Y = a.workspace;
    b.ldy = a.base.R;
    b.out_dtype = NM_F32;
  }
  e = launch_spmm(b, s);
  if (e != hipSuccess) return e;
  LowRank p;
  p.ids = a.ids;
  p.M = a.B;
  p.scale = a.scale;
  p.V = a.xa;
  p.n = int(a.n);
  p.r = int(a.r);
  p.T = int(a.base.T);
  p.C = int(a.base.R);
  return expand<DT, false>(p, static_cast<const float*>(b.Y), b.ldy, a.base.Y, a.base.ldy, a.base.out_dtype, s);
}

template <int DT>
hipError_t backward_dt(const AdapterBwdArgs& a, hipStream_t s) {
  const TrainArgs& d = a.dx;
  float* u = static_cast<float*>(a.workspace);
  hipError_t e = hipSuccess;
  if (d.T > 0) e = shrink<DT, true>(a.ids, a.n, a.B, a.scale, d.G, d.ldg, d.T, d.R, a.r, u, s);
  if (e != hipSuccess) return e;
  if (d.out && d.T > 0) {
    TrainArgs b = d;
    if (d.out_dtype != NM_F32) {
      b.out = u + adapter_u_elems(d.T, a.r);
      b.ldo = d.K;
      b.out_dtype = NM_F32;
    }
    e = launch_spmm_dx(b, s);
    if (e != hipSuccess) return e;
    LowRank p;
    p.ids = a.ids;
    p.M = a.A;
    p.V = u;
    p.n = int(a.n);
    p.r = int(a.r);
    p.T = int(d.T);
    p.C = int(d.K);
    e = expand<DT, true>(p, static_cast<const float*>(b.out), b.ldo, d.out, d.ldo, d.out_dtype, s);
    if (e != hipSuccess) return e;
  }
  GradArgs g{a.ids, int(a.n), nullptr, u, d.act, d.ldx, int(d.T), int(d.K), int(a.r), a.dA, false};
  e = gradient<DT>(g, s);
  if (e != hipSuccess) return e;
  return gradient<DT>(GradArgs{a.ids, int(a.n), a.scale, a.xa, d.G, d.ldg, int(d.T), int(d.R), int(a.r), a.dB, true}, s);
}

}  // namespace

size_t adapter_workspace(int64_t R, int64_t T, int out_dtype) {
  return out_dtype == NM_F32 ? 0 : size_t(T) * size_t(R) * 4;
}

size_t adapter_bwd_workspace(int64_t K, int64_t T, int64_t r, int out_dtype) {
  return size_t(adapter_u_elems(T, r)) * 4 + (out_dtype == NM_F32 ? 0 : size_t(T) * size_t(K) * 4);
}

hipError_t launch_adapter(const AdapterArgs& a, hipStream_t s) {
  return a.base.dtype == NM_F16 ? forward_dt<NM_F16>(a, s) : forward_dt<NM_BF16>(a, s);
}

hipError_t launch_adapter_bwd(const AdapterBwdArgs& a, hipStream_t s) {
  return a.dx.dtype == NM_F16 ? backward_dt<NM_F16>(a, s) : backward_dt<NM_BF16>(a, s);
}

}  // namespace nm
