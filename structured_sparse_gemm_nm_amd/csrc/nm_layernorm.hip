// Layer norm over the features of each token, forward and backward.
//
//   mu = mean(x), var = mean((x - mu)^2), rstd = (var + eps)^(-1/2),
//   xh = (x - mu) rstd,  y = xh w + b;
//   with p = dy w:  dx = rstd (p - mean(p) - xh mean(p xh)),
//   dw = sum_t dy xh,  db = sum_t dy.
//
// Both directions are bound by memory.  A row is loaded once, 16 bytes a lane,
// and stays in the registers of the group of threads that owns it (64, 256,
// 512 or 1024 threads with at most 16 elements each), so the variance is taken
// about the mean in a second pass over registers, not as a difference of
// moments, and nothing is read twice.  Rows longer than the 16384 elements
// that 1024 threads hold are walked in loops instead.
// All statistics and sums are fp32; outputs are rounded once.
//
// Rows need not be aligned beyond their element: a 16-byte piece is loaded
// with the type's own alignment (the hardware takes unaligned vector accesses)
// and the piece a row ends inside is taken element by element.
#include "nm_device.h"
#include "nm_internal.h"

namespace nm {
namespace {

template <int DT>
struct Elem {
  static constexpr int V = DT == NM_F32 ? 4 : 8;   // elements of a 16-byte piece
  static constexpr int SIZE = DT == NM_F32 ? 4 : 2;
};

typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

// Piece of Elem::V elements at column c of a row of H: raw bits, zeros past H.
template <int DT>
__device__ inline u32x4 load_piece(const void* row, int c, int H) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (c + Elem<DT>::V <= H) {
    if constexpr (DT == NM_F32) v = *reinterpret_cast<const u32x4_a4*>(static_cast<const float*>(row) + c);
    else v = *reinterpret_cast<const u32x4_a2*>(static_cast<const uint16_t*>(row) + c);
  } else if (c < H) {
#pragma unroll
    for (int e = 0; e < Elem<DT>::V; ++e) {
      if (c + e >= H) break;
      if constexpr (DT == NM_F32) v[e] = static_cast<const uint32_t*>(row)[c + e];
      else v[e >> 1] |= uint32_t(static_cast<const uint16_t*>(row)[c + e]) << (16 * (e & 1));
    }
  }
  return v;
}

template <int DT>
__device__ inline float elem(const u32x4& v, int e) {
  // through a scalar: a bit cast of a vector's element itself reads element 0
  const uint32_t w = v[DT == NM_F32 ? e : e >> 1];
  if constexpr (DT == NM_F32) return __builtin_bit_cast(float, w);
  else return half_to_f32<DT>((w >> (16 * (e & 1))) & 0xFFFFu);
}

template <int DT>
__device__ inline void store_piece(void* row, int c, int H, const float* f) {
  if constexpr (DT == NM_F32) {
    float* p = static_cast<float*>(row) + c;
    if (c + 4 <= H) {
      *reinterpret_cast<u32x4_a4*>(p) =
          u32x4{__builtin_bit_cast(uint32_t, f[0]), __builtin_bit_cast(uint32_t, f[1]),
                __builtin_bit_cast(uint32_t, f[2]), __builtin_bit_cast(uint32_t, f[3])};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < H) p[e] = f[e];
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(row) + c;
    if (c + 8 <= H) {
      *reinterpret_cast<u32x4_a2*>(p) = u32x4{pack_half2<DT>(f[0], f[1]), pack_half2<DT>(f[2], f[3]),
                                              pack_half2<DT>(f[4], f[5]), pack_half2<DT>(f[6], f[7])};
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e < H) p[e] = to_half_bits<DT>(f[e]);
    }
  }
}

// Sum over a wave, the same bits in every lane: shifts within rows of 16 lanes,
// then row totals passed on, all on the vector ALUs (six LDS permutes a sum
// would take longer than a short row's arithmetic), and lane 63's total read
// back as a scalar.
template <int CTRL, int ROWS>
__device__ inline float dpp_add(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xF, true));
}
__device__ inline float wave_sum(float v) {
  v = dpp_add<0x111, 0xF>(v);   // row_shr 1, 2, 4, 8
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);   // row_bcast 15 into rows 1 and 3
  v = dpp_add<0x143, 0xC>(v);   // row_bcast 31 into rows 2 and 3
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// Sums of N values over the TPR threads of a row, the same bits in every
// thread: each wave sums itself, the waves' sums are added in wave order.
// `slot` alternates between two LDS areas, so one barrier a call suffices (a
// wave can be at most one call ahead of the slowest).
template <int TPR, int N>
__device__ inline void row_sum(float (&v)[N], float (*part)[16][2], int& slot) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) part[slot][wave][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) v[i] += part[slot][w][i];
    }
    slot ^= 1;
  }
}

// use(e) for the elements of the piece at column c that lie before H: without
// a test an element where the whole piece does.
template <int V, typename Use>
__device__ inline void each_inside(int c, int H, Use&& use) {
  if (c + V <= H) {
#pragma unroll
    for (int e = 0; e < V; ++e) use(e);
  } else if (c < H) {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (c + e < H) use(e);
  }
}

constexpr int block_of(int TPR) { return TPR < 256 ? 256 : TPR; }

// Forward.  EPT: elements a thread holds at most (8 or 16).
template <int DT, int TPR, int EPT>
__global__ __launch_bounds__(block_of(TPR)) void layernorm_kernel(const void* __restrict__ x, int T, int H, int64_t ldx,
                                                                  const void* __restrict__ weight,
                                                                  const void* __restrict__ bias, float eps,
                                                                  void* __restrict__ y, int64_t ldy,
                                                                  float* __restrict__ mean, float* __restrict__ rstd) {
  constexpr int V = Elem<DT>::V, NV = EPT / V, E = Elem<DT>::SIZE;
  constexpr int ROWS = block_of(TPR) / TPR;
  __shared__ float part[2][16][2];
  const int lane = threadIdx.x % TPR;
  u32x4 wr[NV], br[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * TPR + lane) * V;
    if (weight) wr[j] = load_piece<DT>(weight, c, H);
    if (bias) br[j] = load_piece<DT>(bias, c, H);
  }
  int slot = 0;
  // A group walks its rows, the next one's loads issued before the current
  // one's sums.  TPR > 64: the rows of a workgroup's loop are the same for every
  // wave, so its barriers are met by all.
  const int64_t stride = int64_t(gridDim.x) * ROWS;
  int64_t t = int64_t(blockIdx.x) * ROWS + threadIdx.x / TPR;
  auto load_row = [&](int64_t r, u32x4 (&v)[NV]) {
    const char* row = static_cast<const char*>(x) + r * ldx * E;
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j] = load_piece<DT>(row, (j * TPR + lane) * V, H);
  };
  u32x4 raw[NV], ahead[NV];
  if (t < T) load_row(t, raw);
  for (; t < T; t += stride) {
    if (t + stride < T) load_row(t + stride, ahead);
    float sum[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) sum[0] += elem<DT>(raw[j], e);
    row_sum<TPR>(sum, part, slot);
    const float mu = sum[0] / float(H);
    float q[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
      each_inside<V>((j * TPR + lane) * V, H, [&](int e) {
        const float d = elem<DT>(raw[j], e) - mu;
        q[0] += d * d;
      });
    row_sum<TPR>(q, part, slot);
    const float rs = 1.f / sqrtf(q[0] / float(H) + eps);
    if (mean && lane == 0) {
      mean[t] = mu;
      rstd[t] = rs;
    }
    char* out = static_cast<char*>(y) + t * ldy * E;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        f[e] = (elem<DT>(raw[j], e) - mu) * rs;
        if (weight) f[e] *= elem<DT>(wr[j], e);
        if (bias) f[e] += elem<DT>(br[j], e);
      }
      store_piece<DT>(out, (j * TPR + lane) * V, H, f);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) raw[j] = ahead[j];
  }
}

// Rows of any length: three walks over the row by 1024 threads.
template <int DT>
__global__ __launch_bounds__(1024) void layernorm_long_kernel(const void* __restrict__ x, int T, int H, int64_t ldx,
                                                              const void* __restrict__ weight,
                                                              const void* __restrict__ bias, float eps,
                                                              void* __restrict__ y, int64_t ldy,
                                                              float* __restrict__ mean, float* __restrict__ rstd) {
  constexpr int V = Elem<DT>::V, E = Elem<DT>::SIZE;
  __shared__ float part[2][16][2];
  int slot = 0;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    const char* row = static_cast<const char*>(x) + t * ldx * E;
    char* out = static_cast<char*>(y) + t * ldy * E;
    float sum[1] = {0.f};
    for (int c = threadIdx.x * V; c < H; c += 1024 * V) {
      const u32x4 v = load_piece<DT>(row, c, H);
#pragma unroll
      for (int e = 0; e < V; ++e) sum[0] += elem<DT>(v, e);
    }
    row_sum<1024>(sum, part, slot);
    const float mu = sum[0] / float(H);
    float q[1] = {0.f};
    for (int c = threadIdx.x * V; c < H; c += 1024 * V) {
      const u32x4 v = load_piece<DT>(row, c, H);
      each_inside<V>(c, H, [&](int e) {
        const float d = elem<DT>(v, e) - mu;
        q[0] += d * d;
      });
    }
    row_sum<1024>(q, part, slot);
    const float rs = 1.f / sqrtf(q[0] / float(H) + eps);
    if (mean && threadIdx.x == 0) {
      mean[t] = mu;
      rstd[t] = rs;
    }
    for (int c = threadIdx.x * V; c < H; c += 1024 * V) {
      const u32x4 v = load_piece<DT>(row, c, H);
      u32x4 wv = {}, bv = {};
      if (weight) wv = load_piece<DT>(weight, c, H);
      if (bias) bv = load_piece<DT>(bias, c, H);
      float f[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        f[e] = (elem<DT>(v, e) - mu) * rs;
        if (weight) f[e] *= elem<DT>(wv, e);
        if (bias) f[e] += elem<DT>(bv, e);
      }
      store_piece<DT>(out, c, H, f);
    }
  }
}

// Backward.  A group of TPR threads walks rows g, g + G, ... (G groups in
// all), keeping the sums of dy xh and dy of its columns in registers; the
// groups of a workgroup are added in LDS and the workgroup writes one row of
// partial sums, part_wb[2][grid][H] (dw's, then db's), added in order by
// layernorm_join_kernel.  The next row's loads are issued before the current
// row's sums, so a row's latency is hidden behind the one before it.
template <int DT, int TPR, int EPT>
__global__ __launch_bounds__(block_of(TPR)) void layernorm_bwd_kernel(
    const void* __restrict__ dy, int64_t ldg, const void* __restrict__ x, int64_t ldx, int T, int H,
    const float* __restrict__ mean, const float* __restrict__ rstd, const void* __restrict__ weight,
    void* __restrict__ dx, int64_t lddx, float* __restrict__ part_wb) {
  constexpr int V = Elem<DT>::V, NV = EPT / V, E = Elem<DT>::SIZE;
  constexpr int ROWS = block_of(TPR) / TPR;
  __shared__ float part[2][16][2];
  const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const int G = gridDim.x * ROWS;
  const float inv_h = 1.f / float(H);

  u32x4 wr[NV];
  float aw[EPT], ab[EPT];
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (weight) wr[j] = load_piece<DT>(weight, (j * TPR + lane) * V, H);
#pragma unroll
  for (int e = 0; e < EPT; ++e) aw[e] = ab[e] = 0.f;

  u32x4 xr[NV], gr[NV];
  float mu = 0.f, rs = 0.f;
  auto load_row = [&](int64_t t, u32x4 (&xv)[NV], u32x4 (&gv)[NV], float& m, float& r) {
    const char* xrow = static_cast<const char*>(x) + t * ldx * E;
    const char* grow = static_cast<const char*>(dy) + t * ldg * E;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      xv[j] = load_piece<DT>(xrow, (j * TPR + lane) * V, H);
      gv[j] = load_piece<DT>(grow, (j * TPR + lane) * V, H);
    }
    m = mean[t];
    r = rstd[t];
  };
  int64_t t = int64_t(blockIdx.x) * ROWS + grp;
  int slot = 0;
  if (t < T) load_row(t, xr, gr, mu, rs);
  for (; t < T; t += G) {   // TPR > 64: one group a workgroup, so its barriers are met by every wave
    u32x4 xn[NV], gn[NV];
    float mn = 0.f, rn = 0.f;
    if (t + G < T) load_row(t + G, xn, gn, mn, rn);
    float c[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
      each_inside<V>((j * TPR + lane) * V, H, [&](int e) {
        const float g = elem<DT>(gr[j], e);
        const float xh = (elem<DT>(xr[j], e) - mu) * rs;
        const float p = weight ? g * elem<DT>(wr[j], e) : g;
        c[0] += p;
        c[1] += p * xh;
        aw[j * V + e] += g * xh;
        ab[j * V + e] += g;
      });
    row_sum<TPR>(c, part, slot);
    const float c1 = c[0] * inv_h, c2 = c[1] * inv_h;
    char* out = static_cast<char*>(dx) + t * lddx * E;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float g = elem<DT>(gr[j], e);
        const float xh = (elem<DT>(xr[j], e) - mu) * rs;
        const float p = weight ? g * elem<DT>(wr[j], e) : g;
        f[e] = rs * (p - c1 - xh * c2);
      }
      store_piece<DT>(out, (j * TPR + lane) * V, H, f);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      xr[j] = xn[j];
      gr[j] = gn[j];
    }
    mu = mn;
    rs = rn;
  }
  if (!part_wb) return;

  float* pw = part_wb + int64_t(blockIdx.x) * H;
  float* pb = part_wb + (int64_t(gridDim.x) + blockIdx.x) * H;
  if constexpr (ROWS > 1) {   // TPR 64: add the groups' sums in group order
    __shared__ float sums[ROWS][64 * EPT];
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e)
          sums[grp][(j * TPR + lane) * V + e] = which ? ab[j * V + e] : aw[j * V + e];
      __syncthreads();
      for (int c = threadIdx.x; c < H; c += block_of(TPR)) {
        float v = sums[0][c];
#pragma unroll
        for (int g = 1; g < ROWS; ++g) v += sums[g][c];
        (which ? pb : pw)[c] = v;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int q = 0; q < V; q += 4) {
        const int c = (j * TPR + lane) * V + q;
        store_piece<NM_F32>(pw, c, H, aw + j * V + q);
        store_piece<NM_F32>(pb, c, H, ab + j * V + q);
      }
    }
  }
}

// Rows of any length: the row's two sums in one walk, dx in a second.
template <int DT>
__global__ __launch_bounds__(1024) void layernorm_bwd_long_kernel(
    const void* __restrict__ dy, int64_t ldg, const void* __restrict__ x, int64_t ldx, int T, int H,
    const float* __restrict__ mean, const float* __restrict__ rstd, const void* __restrict__ weight,
    void* __restrict__ dx, int64_t lddx) {
  constexpr int V = Elem<DT>::V, E = Elem<DT>::SIZE;
  __shared__ float part[2][16][2];
  int slot = 0;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    const char* xrow = static_cast<const char*>(x) + t * ldx * E;
    const char* grow = static_cast<const char*>(dy) + t * ldg * E;
    char* out = static_cast<char*>(dx) + t * lddx * E;
    const float mu = mean[t], rs = rstd[t];
    float sum[2] = {0.f, 0.f};
    auto each = [&](auto&& use) {
      for (int c = threadIdx.x * V; c < H; c += 1024 * V) {
        const u32x4 xv = load_piece<DT>(xrow, c, H), gv = load_piece<DT>(grow, c, H);
        u32x4 wv = {};
        if (weight) wv = load_piece<DT>(weight, c, H);
        float p[V], xh[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          p[e] = elem<DT>(gv, e) * (weight ? elem<DT>(wv, e) : 1.f);
          xh[e] = (elem<DT>(xv, e) - mu) * rs;
        }
        use(c, p, xh);
      }
    };
    each([&](int c, const float* p, const float* xh) {
      each_inside<V>(c, H, [&](int e) {
        sum[0] += p[e];
        sum[1] += p[e] * xh[e];
      });
    });
    row_sum<1024>(sum, part, slot);
    const float c1 = sum[0] / float(H), c2 = sum[1] / float(H);
    each([&](int c, const float* p, const float* xh) {
      float f[V];
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] = rs * (p[e] - c1 - xh[e] * c2);
      store_piece<DT>(out, c, H, f);
    });
  }
}

// Partial dw and db of rows t0, t0 + grid.y, ... for long rows: a thread a column.
template <int DT>
__global__ __launch_bounds__(256) void layernorm_columns_kernel(const void* __restrict__ dy, int64_t ldg,
                                                                const void* __restrict__ x, int64_t ldx, int T, int H,
                                                                const float* __restrict__ mean,
                                                                const float* __restrict__ rstd,
                                                                float* __restrict__ part_wb) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= H) return;
  float aw = 0.f, ab = 0.f;
  for (int64_t t = blockIdx.y; t < T; t += gridDim.y) {
    float g, v;
    if constexpr (DT == NM_F32) {
      g = static_cast<const float*>(dy)[t * ldg + c];
      v = static_cast<const float*>(x)[t * ldx + c];
    } else {
      g = half_to_f32<DT>(static_cast<const uint16_t*>(dy)[t * ldg + c]);
      v = half_to_f32<DT>(static_cast<const uint16_t*>(x)[t * ldx + c]);
    }
    aw += g * ((v - mean[t]) * rstd[t]);
    ab += g;
  }
  part_wb[int64_t(blockIdx.y) * H + c] = aw;
  part_wb[(int64_t(gridDim.y) + blockIdx.y) * H + c] = ab;
}

// dw (grid.y 0) and db (grid.y 1) from P partial rows: a workgroup takes 64
// columns, its 16 waves each every 16th partial row; the waves' sums are added
// in wave order, so the result does not depend on timing.
template <int OUT>
__global__ __launch_bounds__(1024) void layernorm_join_kernel(const float* __restrict__ part_wb, int P, int H,
                                                              void* __restrict__ dw, void* __restrict__ db) {
  __shared__ float sums[16][64];
  void* out = blockIdx.y ? db : dw;
  if (!out) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  const float* p = part_wb + int64_t(blockIdx.y) * P * H;
  float v = 0.f;
  if (c < H) {
#pragma unroll 8
    for (int i = wave; i < P; i += 16) v += p[int64_t(i) * H + c];
  }
  sums[wave][lane] = v;
  __syncthreads();
  if (wave != 0 || c >= H) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) v += sums[w][lane];
  if constexpr (OUT == NM_F32) static_cast<float*>(out)[c] = v;
  else static_cast<uint16_t*>(out)[c] = to_half_bits<OUT>(v);
}

// Threads a row of H elements takes, and elements a thread: the smallest group
// that holds the row (a wave up to 1024 elements).  0: walked in loops.
struct Shape {
  int tpr, ept;
};
Shape row_shape(int64_t H) {
  if (H <= 512) return {64, 8};
  if (H <= 1024) return {64, 16};
  if (H <= 2048) return {256, 8};
  if (H <= 4096) return {256, 16};
  if (H <= 8192) return {512, 16};
  if (H <= 16384) return {1024, 16};
  return {0, 0};
}

// Workgroups of a forward pass or of a long-row kernel; past this many they walk.
unsigned row_grid(int64_t n) { return unsigned(n < (int64_t(1) << 20) ? n : int64_t(1) << 20); }

// Workgroups of the forward pass: one a row group while they all fit the chip
// at once (2048 threads a CU), past that the fewest rounds, evenly filled, so
// that a group's next row arrives while it works on one (12608 x 768 fp16: 13.6
// us with a workgroup every 4 rows and sums by LDS permutes, 12.4 now; 8192 x
// 4096 bf16: 26.6, now 23.7, 5.7 TB/s).
unsigned fwd_grid(int64_t groups, int threads) {
  const int64_t resident = int64_t(256) * 2048 / threads;
  const int64_t rounds = (groups + resident - 1) / resident;
  return unsigned(rounds <= 1 ? groups : (groups + rounds - 1) / rounds);
}

template <int DT, int TPR, int EPT>
hipError_t fwd_cfg(const LayerNormArgs& a, hipStream_t s) {
  constexpr int ROWS = block_of(TPR) / TPR;
  hipLaunchKernelGGL((layernorm_kernel<DT, TPR, EPT>), dim3(fwd_grid((a.T + ROWS - 1) / ROWS, block_of(TPR))), dim3(block_of(TPR)), 0,
                     s, a.x, int(a.T), int(a.H), a.ldx, a.weight, a.bias, a.eps, a.y, a.ldy, a.mean_out, a.rstd_out);
  return hipGetLastError();
}

template <int DT>
hipError_t fwd_dt(const LayerNormArgs& a, hipStream_t s) {
  const Shape sh = row_shape(a.H);
  if (sh.tpr == 64) return sh.ept == 8 ? fwd_cfg<DT, 64, 8>(a, s) : fwd_cfg<DT, 64, 16>(a, s);
  if (sh.tpr == 256) return sh.ept == 8 ? fwd_cfg<DT, 256, 8>(a, s) : fwd_cfg<DT, 256, 16>(a, s);
  if (sh.tpr == 512) return fwd_cfg<DT, 512, 16>(a, s);
  if (sh.tpr == 1024) return fwd_cfg<DT, 1024, 16>(a, s);
  hipLaunchKernelGGL((layernorm_long_kernel<DT>), dim3(row_grid(a.T)), dim3(1024), 0, s, a.x, int(a.T), int(a.H),
                     a.ldx, a.weight, a.bias, a.eps, a.y, a.ldy, a.mean_out, a.rstd_out);
  return hipGetLastError();
}

// Workgroups of the backward pass (= rows of partial sums): two a CU, to keep its
// loads in flight.  Their partial sums, 8 H bytes each, written and read once, are
// small beside many rows (8192 x 4096 bf16: 16.8 MB beside 67 of dx) and as large as
// dx beside few (1999 x 1543 fp16: 6.3 MB beside 6.2, of the pass's 13 + 4 us).
int64_t bwd_groups(int64_t T, int64_t H) {
  const Shape sh = row_shape(H);
  const int64_t rows = sh.tpr == 64 ? 4 : 1;
  const int64_t want = sh.tpr == 0 ? 64 : 512;
  const int64_t all = (T + rows - 1) / rows;
  return all < want ? all : want;
}

template <int DT, int TPR, int EPT>
hipError_t bwd_cfg(const LayerNormArgs& a, float* part, hipStream_t s) {
  hipLaunchKernelGGL((layernorm_bwd_kernel<DT, TPR, EPT>), dim3(unsigned(bwd_groups(a.T, a.H))), dim3(block_of(TPR)),
                     0, s, a.dy, a.ldg, a.x, a.ldx, int(a.T), int(a.H), a.mean, a.rstd, a.weight, a.dx, a.lddx, part);
  return hipGetLastError();
}

template <int DT>
hipError_t bwd_dt(const LayerNormArgs& a, hipStream_t s) {
  const Shape sh = row_shape(a.H);
  const bool sums = a.dw || a.db;
  float* part = sums ? static_cast<float*>(a.workspace) : nullptr;
  const int64_t P = bwd_groups(a.T, a.H);
  hipError_t e = hipSuccess;
  if (a.T > 0) {
    if (sh.tpr == 64) e = sh.ept == 8 ? bwd_cfg<DT, 64, 8>(a, part, s) : bwd_cfg<DT, 64, 16>(a, part, s);
    else if (sh.tpr == 256) e = sh.ept == 8 ? bwd_cfg<DT, 256, 8>(a, part, s) : bwd_cfg<DT, 256, 16>(a, part, s);
    else if (sh.tpr == 512) e = bwd_cfg<DT, 512, 16>(a, part, s);
    else if (sh.tpr == 1024) e = bwd_cfg<DT, 1024, 16>(a, part, s);
    else {
      hipLaunchKernelGGL((layernorm_bwd_long_kernel<DT>), dim3(row_grid(a.T)), dim3(1024), 0, s, a.dy, a.ldg, a.x,
                         a.ldx, int(a.T), int(a.H), a.mean, a.rstd, a.weight, a.dx, a.lddx);
      e = hipGetLastError();
      if (e == hipSuccess && sums) {
        hipLaunchKernelGGL((layernorm_columns_kernel<DT>), dim3(unsigned((a.H + 255) / 256), unsigned(P)), dim3(256),
                           0, s, a.dy, a.ldg, a.x, a.ldx, int(a.T), int(a.H), a.mean, a.rstd, part);
        e = hipGetLastError();
      }
    }
  }
  if (e != hipSuccess || !sums) return e;
  // T == 0: no partial rows, so the sums are zeros
  const dim3 grid(unsigned((a.H + 63) / 64), 2);
  if (a.out_dtype == NM_F32)
    hipLaunchKernelGGL((layernorm_join_kernel<NM_F32>), grid, dim3(1024), 0, s, part, int(P), int(a.H), a.dw, a.db);
  else
    hipLaunchKernelGGL((layernorm_join_kernel<DT>), grid, dim3(1024), 0, s, part, int(P), int(a.H), a.dw, a.db);
  return hipGetLastError();
}

}  // namespace

size_t layernorm_bwd_workspace(int64_t T, int64_t H) { return size_t(bwd_groups(T, H)) * size_t(H) * 8; }

hipError_t launch_layernorm(const LayerNormArgs& a, hipStream_t s) {
  if (a.dtype == NM_F16) return fwd_dt<NM_F16>(a, s);
  if (a.dtype == NM_BF16) return fwd_dt<NM_BF16>(a, s);
  return fwd_dt<NM_F32>(a, s);
}

hipError_t launch_layernorm_bwd(const LayerNormArgs& a, hipStream_t s) {
  if (a.dtype == NM_F16) return bwd_dt<NM_F16>(a, s);
  if (a.dtype == NM_BF16) return bwd_dt<NM_BF16>(a, s);
  return bwd_dt<NM_F32>(a, s);
}

}  // namespace nm
