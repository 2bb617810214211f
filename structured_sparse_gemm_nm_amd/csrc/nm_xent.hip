// Softmax cross entropy over a large vocabulary, the logits never kept.
//
//   l[t][v] = x_t . w_v,  lse_t = log sum_v exp l[t][v],  loss_t = lse_t - l[t][y_t]
//   d[t][v] = g_t (exp(l[t][v] - lse_t) - [v = y_t]),   g = dL/dloss,
//   dx = d W,   dW = d^T x;
// a label outside [0, V) carries no loss and no gradient.
//
// Forward: one product X W^T whose tiles are reduced in registers to a running
// maximum and sum of exponentials per token (and the label's logit), 8 bytes a
// token and vocabulary tile, joined by a second small kernel.
// Backward: the vocabulary is walked in pieces.  For each, the logits are
// computed again and turned into d in the epilogue (written in both orders, so
// that every product reads its operands along the reduction), then the
// piece's rows of dW and its share of dx are two more products.  dx gathers in
// fp32 over the pieces.
// d enters the matrix cores in the inputs' 16-bit type, with as much of dloss
// as possible left to the fp32 results: dx's operand is q = softmax - onehot
// (its rows are multiplied by g_t at the end), dW's is q g_t / G with G the
// largest |g|, multiplied by G at the end.  With the usual constant g both are
// q itself; g q rounded as a whole would give every label's entry, all near -g,
// the same rounding error (4e-3 of dW measured, against 2e-3 now).  fp16 holds
// the operands times 2^14, so that probabilities down to 2^-38 are not flushed.
// An output of 16 bits takes the operand rounded once (its own rounding is as
// large: 2048 x 32000 x 4096 bf16, dx and dW 1.667e-3 from the exact ones, 1.662e-3
// with fp32 operands).  An fp32 output would show it (1.3e-4 there, 6e-4 at 7
// tokens), so it takes the operand in two parts that add up to q to 2^-16 (bf16)
// or 2^-22 (fp16) and a product of each (9e-7 and 1.5e-6; the backward pass of that
// size with both outputs in fp32 2.67 ms, in bf16 1.47).
#include "nm_gemm_nt.h"
#include "nm_internal.h"

#include <algorithm>
#include <type_traits>

namespace nm {
namespace {

constexpr float kInf = __builtin_inff();

// For few tokens, narrow tiles with a deeper ring (the product is then a stream
// of W).
using TileBig = GemmTilePiped;
using Tile128 = GemmTile<128, 128, 2, 2, 4>;
using Tile64 = GemmTile<128, 64, 4, 1, 4>;
using Tile16 = GemmTile<128, 16, 4, 1, 6>;

// The product of tile type C.
template <int DT, class C, class... Args>
__device__ inline void product_tile(Args&&... args) {
  if constexpr (std::is_same_v<C, GemmTilePiped>) gemm_nt_piped<DT, C>(static_cast<Args&&>(args)...);
  else gemm_nt<DT, C>(static_cast<Args&&>(args)...);
}

// A tile's 16-bit results leave through LDS, a wave its own part, so that every
// store writes whole lines (straight from the result layout a store covers 16
// rows of 32 bytes).  The wave's area holds rows by n (of its m) or by m (of
// its n), padded by 16 bytes.
template <class C>
struct OutArea {
  static constexpr int MW = C::FM * 16, NW = C::FN * 16;           // the wave's part
  static constexpr int ROW_N = MW * 2 + 16, ROW_M = NW * 2 + 16;   // bytes of a row
  static constexpr int BYTES = NW * ROW_N > MW * ROW_M ? NW * ROW_N : MW * ROW_M;
  static constexpr int ALL = C::WM * C::WN * BYTES;
  static constexpr int LDS = ALL > C::LDS ? ALL : C::LDS;          // of a kernel that uses it
  static_assert(LDS <= 160 * 1024, "fits a workgroup");

  // Fragment (i, j)'s 4 consecutive m of the lane's n, as two words, by n.
  __device__ static void put_by_n(unsigned char* area, int i, int j, int li, int lq, uint32_t lo, uint32_t hi) {
    *reinterpret_cast<u32x2*>(area + (j * 16 + li) * ROW_N + (i * 16 + 4 * lq) * 2) = u32x2{lo, hi};
  }
  // By m: neighbouring lanes (n, n + 1) exchange halves, so that each writes
  // two whole words.
  __device__ static void put_by_m(unsigned char* area, int i, int j, int li, int lq, uint32_t lo, uint32_t hi) {
    const bool odd = li & 1;
    const uint32_t got = uint32_t(__builtin_amdgcn_update_dpp(0, int(odd ? lo : hi), 0xB1, 0xF, 0xF, false));
    const uint32_t own = odd ? hi : lo;          // rows m, m + 1 (even lane) or m + 2, m + 3 (odd)
    const uint32_t first = odd ? got : own, second = odd ? own : got;
    unsigned char* p = area + (i * 16 + 4 * lq + (odd ? 2 : 0)) * ROW_M + (j * 16 + (li & ~1)) * 2;
    *reinterpret_cast<uint32_t*>(p) = (first & 0xFFFFu) | (second << 16);
    *reinterpret_cast<uint32_t*>(p + ROW_M) = (first >> 16) | (second & 0xFFFF0000u);
  }
  // Calls out(row, first column, 8 values) for the area's rows, 16 bytes a lane.
  template <bool BY_N, class Out>
  __device__ static void take(const unsigned char* area, Out&& out) {
    constexpr int ROWS = BY_N ? NW : MW, PIECES = (BY_N ? MW : NW) / 8, PITCH = BY_N ? ROW_N : ROW_M;
    constexpr int PER = 64 / PIECES;             // rows a pass
    static_assert(64 % PIECES == 0 && ROWS % PER == 0, "whole passes");
    const int lane = threadIdx.x & 63, piece = lane % PIECES;
    wait_lgkm0();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int k = 0; k < ROWS / PER; ++k) {
      const int row = k * PER + lane / PIECES;
      out(row, piece * 8, *reinterpret_cast<const u32x4*>(area + row * PITCH + piece * 16));
    }
    wait_lgkm0();
    asm volatile("" ::: "memory");
  }
};

// exp(m - top) for parts of a sum: 0 for an empty part (m = -inf).
__device__ inline float part_weight(float m, float top) { return m == -kInf ? 0.f : __expf(m - top); }

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------
struct XentArgsDev {
  const uint16_t* x;
  const uint16_t* w;
  const int32_t* labels;
  int64_t ldx, ldw;
  int T, V, H;
};

template <int DT, class C>
__global__ __launch_bounds__(C::THREADS) void xent_stats_kernel(XentArgsDev p, float2* __restrict__ part,
                                                                float* __restrict__ at_label, int tilesV, int tilesT,
                                                                int group) {
  extern __shared__ __align__(16) unsigned char smem[];
  int tv, tt;
  grouped_tile(xcd_tile(blockIdx.x, gridDim.x), tilesV, tilesT, group, tv, tt);
  product_tile<DT, C>(p.w, p.ldw, p.V, p.x, p.ldx, p.T, p.H, tv, tt, smem, [&](auto& acc, int wm, int wn, int li, int lq) {
    float2* red = reinterpret_cast<float2*>(smem);   // [WM][BN]
    const int v0 = tv * C::BM + wm * C::FM * 16 + 4 * lq;
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
      const int n = wn * C::FN * 16 + j * 16 + li, t = tt * C::BN + n;
      const int label = t < p.T ? p.labels[t] : -1;
      float m = -kInf;
#pragma unroll
      for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int v = v0 + i * 16 + e;
          if (v >= p.V) acc[i][j][e] = -kInf;
          m = fmaxf(m, acc[i][j][e]);
          if (v == label && v < p.V) at_label[t] = acc[i][j][e];
        }
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      const float base = m == -kInf ? 0.f : m;
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s += __expf(acc[i][j][e] - base);
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      if (lq == 0) red[wm * C::BN + n] = make_float2(m, s);
    }
    __syncthreads();
    for (int n = threadIdx.x; n < C::BN; n += C::THREADS) {
      const int t = tt * C::BN + n;
      if (t >= p.T) break;
      float m = red[n].x;
#pragma unroll
      for (int w = 1; w < C::WM; ++w) m = fmaxf(m, red[w * C::BN + n].x);
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < C::WM; ++w) s += red[w * C::BN + n].y * part_weight(red[w * C::BN + n].x, m);
      part[int64_t(tv) * p.T + t] = make_float2(m, s);
    }
  });
}

// lse and loss from the parts: a workgroup takes 64 tokens, its 16 waves every
// 16th vocabulary tile; the waves' sums are joined in wave order.
__global__ __launch_bounds__(1024) void xent_join_kernel(const float2* __restrict__ part,
                                                         const float* __restrict__ at_label,
                                                         const int32_t* __restrict__ labels, int tilesV, int T, int V,
                                                         float* __restrict__ loss, float* __restrict__ lse) {
  __shared__ float2 red[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = blockIdx.x * 64 + lane;
  float m = -kInf, s = 0.f;
  if (t < T) {
#pragma unroll 4
    for (int i = wave; i < tilesV; i += 16) {
      const float2 q = part[int64_t(i) * T + t];
      const float top = fmaxf(m, q.x);
      s = s * part_weight(m, top) + q.y * part_weight(q.x, top);
      m = top;
    }
  }
  red[wave][lane] = make_float2(m, s);
  __syncthreads();
  if (wave != 0 || t >= T) return;
  for (int w = 1; w < 16; ++w) m = fmaxf(m, red[w][lane].x);
  s = 0.f;
  for (int w = 0; w < 16; ++w) s += red[w][lane].y * part_weight(red[w][lane].x, m);
  const float l = m + logf(s);
  const int y = labels[t];
  lse[t] = l;
  loss[t] = uint32_t(y) < uint32_t(V) ? l - at_label[t] : 0.f;
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------

// out[c][r] = in[r][c] for a 16-bit matrix [rows][cols], cols a multiple of 8;
// out rows hold ldo elements (a multiple of 64), zeros past `rows` and, given
// labels, for rows whose label lies outside [0, V): whatever an ignored token
// holds, Inf and NaN among it, then meets its zero gradient as a zero.
__global__ __launch_bounds__(256) void xent_transpose_kernel(const uint16_t* __restrict__ in, int64_t ldi, int rows,
                                                             int cols, const int32_t* __restrict__ labels, int V,
                                                             uint16_t* __restrict__ out, int64_t ldo) {
  __shared__ uint16_t tile[64][64 + 2];
  const int r0 = blockIdx.x * 64, c0 = blockIdx.y * 64;
  const int piece = threadIdx.x & 7, line = threadIdx.x >> 3;   // 32 lines of 8 pieces
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = line + 32 * h, c = piece * 8;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (r0 + r < rows && c0 + c < cols && (!labels || uint32_t(labels[r0 + r]) < uint32_t(V)))
      v = *reinterpret_cast<const u32x4*>(in + int64_t(r0 + r) * ldi + c0 + c);
#pragma unroll
    for (int e = 0; e < 4; ++e) *reinterpret_cast<uint32_t*>(&tile[r][c + 2 * e]) = v[e];
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = line + 32 * h, r = piece * 8;
    if (c0 + c >= cols || r0 + r >= ldo) continue;
    u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      v[e] = uint32_t(tile[r + 2 * e][c]) | (uint32_t(tile[r + 2 * e + 1][c]) << 16);
    *reinterpret_cast<u32x4*>(out + int64_t(c0 + c) * ldo + r0 + r) = v;
  }
}

// The larger of two magnitudes, NaN if either is (fmaxf drops a NaN, and dW with it).
__device__ inline float larger(float a, float b) { return a >= b || a != a ? a : b; }

// The largest |dloss| of a counted token; NaN if one holds NaN, so that dW does.
__global__ __launch_bounds__(1024) void xent_largest_kernel(const float* __restrict__ dloss,
                                                            const int32_t* __restrict__ labels, int T, int V,
                                                            float* __restrict__ largest) {
  __shared__ float red[16];
  float m = 0.f;
  for (int t = threadIdx.x; t < T; t += 1024)
    if (uint32_t(labels[t]) < uint32_t(V)) m = larger(m, fabsf(dloss[t]));
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = larger(m, __shfl_xor(m, o));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < 16; ++w) m = larger(m, red[w]);
  *largest = m;
}

// What an operand is multiplied by before it is rounded to 16 bits.
template <int DT>
constexpr float kOperandScale = DT == NM_F16 ? 16384.f : 1.f;

// What is left of f after its rounding to 16 bits; nothing of what is not finite.
template <int DT>
__device__ inline float rest(float f) {
  const float r = f - half_to_f32<DT>(to_half_bits<DT>(f));
  return fabsf(r) < kInf ? r : 0.f;
}

struct XentBwdDev {
  XentArgsDev a;
  const float* lse;
  const float* dloss;
  const float* largest; // of |dloss|
  uint16_t* d;          // q [T][ldd], or null
  uint16_t* dt;         // q g / G, transposed: [piece][ldt], or null
  uint16_t* d_rest;     // what rounding left of them, or null
  uint16_t* dt_rest;
  int64_t ldd, ldt;
  int v0, vn, vpad;     // the piece: rows v0 .. v0 + vn of W, padded to vpad
};

template <int DT, class C>
__global__ __launch_bounds__(C::THREADS) void xent_dlogits_kernel(XentBwdDev p, int tilesV, int tilesT, int group) {
  extern __shared__ __align__(16) unsigned char smem[];
  int tv, tt;
  grouped_tile(xcd_tile(blockIdx.x, gridDim.x), tilesV, tilesT, group, tv, tt);
  const uint16_t* w = p.a.w + int64_t(p.v0) * p.a.ldw;
  product_tile<DT, C>(w, p.a.ldw, p.vn, p.a.x, p.a.ldx, p.a.T, p.a.H, tv, tt, smem,
                 [&](auto& acc, int wm, int wn, int li, int lq) {
    const float G = *p.largest;
    using Area = OutArea<C>;
    unsigned char* area = smem + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * Area::BYTES;
    const int v0 = tv * C::BM + wm * Area::MW, t0 = tt * C::BN + wn * Area::NW;   // the wave's corner
    // q, scaled for its 16-bit type, in place of the logits
    float ratio[C::FN];
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
      const int t = t0 + j * 16 + li;
      const bool live = t < p.a.T;
      const int label = live ? p.a.labels[t] : -1;
      const bool counted = uint32_t(label) < uint32_t(p.a.V);
      const float lse = live ? p.lse[t] : 0.f;
      // g == G gives exactly 1; G == 0 (no gradient at all) gives 0
      ratio[j] = counted && G != 0.f ? p.dloss[t] / G : 0.f;
      const int mine = label - p.v0;
#pragma unroll
      for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int v = v0 + i * 16 + 4 * lq + e;
          const float q = __expf(acc[i][j][e] - lse) - (v == mine ? 1.f : 0.f);
          acc[i][j][e] = counted && v < p.vn ? kOperandScale<DT> * q : 0.f;
        }
    }
    if (p.d) {
      auto write = [&](uint16_t* d, auto&& part) {
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
          for (int i = 0; i < C::FM; ++i)
            Area::put_by_n(area, i, j, li, lq, pack_half2<DT>(part(acc[i][j][0]), part(acc[i][j][1])),
                           pack_half2<DT>(part(acc[i][j][2]), part(acc[i][j][3])));
        // vpad is a multiple of 64: whole pieces
        Area::template take<true>(area, [&](int n, int m, const u32x4& w) {
          if (t0 + n < p.a.T && v0 + m < p.vpad) *reinterpret_cast<u32x4*>(d + int64_t(t0 + n) * p.ldd + v0 + m) = w;
        });
      };
      write(p.d, [](float f) { return f; });
      if (p.d_rest) write(p.d_rest, [](float f) { return rest<DT>(f); });
    }
    if (p.dt) {
      auto write = [&](uint16_t* dt, auto&& part) {
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
          for (int i = 0; i < C::FM; ++i)
            Area::put_by_m(area, i, j, li, lq,
                           pack_half2<DT>(part(ratio[j] * acc[i][j][0]), part(ratio[j] * acc[i][j][1])),
                           pack_half2<DT>(part(ratio[j] * acc[i][j][2]), part(ratio[j] * acc[i][j][3])));
        // so is ldt
        Area::template take<false>(area, [&](int m, int n, const u32x4& w) {
          if (v0 + m < p.vpad && t0 + n < p.ldt)
            *reinterpret_cast<u32x4*>(dt + int64_t(v0 + m) * p.ldt + t0 + n) = w;
        });
      };
      write(p.dt, [](float f) { return f; });
      if (p.dt_rest) write(p.dt_rest, [](float f) { return rest<DT>(f); });
    }
  });
}

// out[n][m] (+)= sum_k P[m][k] Q[n][k] over the split's share of K.
struct XentProduct {
  const uint16_t* P;
  const uint16_t* Q;
  int64_t ldp, ldq;
  int M, N, K, ksplit;  // a split takes ksplit of K (a multiple of 64)
  const float* largest; // G (dw: the result is multiplied by it), or null
  void* out;            // rows of ldo elements; split z at out + z * split_stride (fp32)
  int64_t ldo, split_stride;
  bool add;             // onto what out holds (fp32 only)
};

template <int DT, class C, int OUT>
__global__ __launch_bounds__(C::THREADS) void xent_product_kernel(XentProduct p, int tilesM, int tilesN, int group) {
  extern __shared__ __align__(16) unsigned char smem[];
  int tm, tn;
  grouped_tile(xcd_tile(blockIdx.x, gridDim.x), tilesM, tilesN, group, tm, tn);
  const int k0 = blockIdx.y * p.ksplit;
  const int K = min(p.K - k0, p.ksplit);
  product_tile<DT, C>(p.P + k0, p.ldp, p.M, p.Q + k0, p.ldq, p.N, K, tm, tn, smem,
                 [&](auto& acc, int wm, int wn, int li, int lq) {
    const float down = (p.largest ? *p.largest : 1.f) / kOperandScale<DT>;
    using Area = OutArea<C>;
    const int m0 = tm * C::BM + wm * Area::MW, n0 = tn * C::BN + wn * Area::NW;   // the wave's corner
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] *= down;
    if constexpr (OUT == NM_F32) {
#pragma unroll
      for (int j = 0; j < C::FN; ++j) {
        const int n = n0 + j * 16 + li;
        if (n >= p.N) continue;
#pragma unroll
        for (int i = 0; i < C::FM; ++i) {
          const int m = m0 + i * 16 + 4 * lq;
          if (m >= p.M) continue;        // M is a multiple of 8
          float* o = static_cast<float*>(p.out) + blockIdx.y * p.split_stride + int64_t(n) * p.ldo + m;
          f32x4 v = acc[i][j];
          if (p.add) v += *reinterpret_cast<const f32x4*>(o);
          *reinterpret_cast<f32x4*>(o) = v;
        }
      }
    } else {
      unsigned char* area = smem + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * Area::BYTES;
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
          Area::put_by_n(area, i, j, li, lq, pack_half2<OUT>(acc[i][j][0], acc[i][j][1]),
                         pack_half2<OUT>(acc[i][j][2], acc[i][j][3]));
      Area::template take<true>(area, [&](int r, int c, const u32x4& w) {
        const int n = n0 + r, m = m0 + c;
        if (n >= p.N || m >= p.M) return;
        uint16_t* o = static_cast<uint16_t*>(p.out) + int64_t(n) * p.ldo + m;
        if ((p.ldo & 7) == 0) {
          __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(o));   // not read again here: leave the caches to the operands
        } else {                         // rows on 8 bytes
          *reinterpret_cast<u32x2*>(o) = u32x2{w[0], w[1]};
          *reinterpret_cast<u32x2*>(o + 4) = u32x2{w[2], w[3]};
        }
      });
    }
  });
}

// dx for few tokens: acc[split][t][h] = sum over the split's v of q[t][v] w[v][h].
// The product is a stream of W, whose rows lie along h, not along the
// reduction: transposing W first, as the large products do, would read and
// write it once more.  A workgroup of 8 waves owns TF*16 tokens and 128
// columns; its waves take the split's 32-row chunks in turn, bring each into
// LDS (16 bytes a lane) and take the operands out by transpose reads, the next
// chunk's rows arriving meanwhile; in the end the waves' tiles are added in a
// fixed order.
struct FewDx {
  const uint16_t* w;    // the piece's rows [vn][H], ldw
  const uint16_t* d;    // q [T][ldd], zeros from vn to vpad
  int64_t ldw, ldd;
  int T, H, vn, vpad, vsplit;   // a split takes vsplit rows (a multiple of 32)
  float* acc;           // [splits][T][H]
  bool add;
};
constexpr int kFewWaves = 8;
constexpr int kFewPitch = 128 * 2 + 32;
__host__ __device__ constexpr int few_row(int v) { return v * kFewPitch + (((v >> 3) & 1) + (v >> 4)) * 128; }
constexpr int kFewTile = few_row(31) + 256;
static_assert(kFewTile % 16 == 0, "aligned tiles");

template <int DT, int TF>
__global__ __launch_bounds__(kFewWaves * 64) void xent_dx_few_kernel(FewDx p) {
  constexpr int LDS = kFewWaves * kFewTile > kFewWaves / 2 * TF * 8 * 1024 ? kFewWaves * kFewTile
                                                                             : kFewWaves / 2 * TF * 8 * 1024;
  __shared__ __align__(16) unsigned char smem[LDS];
  const int lane = threadIdx.x & 63, li = lane & 15, lq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h0 = blockIdx.x * 128, t0 = blockIdx.z * (TF * 16);
  const int v0 = blockIdx.y * p.vsplit, v1 = min(v0 + p.vsplit, p.vpad);
  unsigned char* tile = smem + wave * kFewTile;
  const int piece = lane & 15, prow = lane >> 4;
  const int col = h0 + piece * 8 < p.H ? h0 + piece * 8 : 0;   // columns past H: results not stored
  const int tr_row = 8 * (lane >> 4) + ((lane >> 2) & 3);
  const int tr_lo = few_row(tr_row) + 8 * (lane & 3), tr_hi = few_row(tr_row + 4) + 8 * (lane & 3);
  f32x4 acc[TF][8];
#pragma unroll
  for (int i = 0; i < TF; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  u32x4 x[8], q[TF];
  auto load = [&](int v) {   // rows past vn reread the last one and meet zeros of q
#pragma unroll
    for (int k = 0; k < 8; ++k)
      x[k] = *reinterpret_cast<const u32x4*>(p.w + int64_t(min(v + k * 4 + prow, p.vn - 1)) * p.ldw + col);
#pragma unroll
    for (int i = 0; i < TF; ++i)
      q[i] = *reinterpret_cast<const u32x4*>(p.d + int64_t(min(t0 + i * 16 + li, p.T - 1)) * p.ldd + v + 8 * lq);
    __builtin_amdgcn_sched_barrier(0);
  };
  int v = v0 + wave * 32;
  if (v < v1) load(v);
  for (; v < v1; v += kFewWaves * 32) {
    u32x4 a[TF];
#pragma unroll
    for (int k = 0; k < 8; ++k) *reinterpret_cast<u32x4*>(tile + few_row(k * 4 + prow) + piece * 16) = x[k];
#pragma unroll
    for (int i = 0; i < TF; ++i) a[i] = q[i];
    __builtin_amdgcn_sched_barrier(0);
    if (v + kFewWaves * 32 < v1) load(v + kFewWaves * 32);
    wait_lgkm0();            // a wave's LDS operations are carried out in order: no barrier
    asm volatile("" ::: "memory");
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const u32x2 lo = lds_read_tr(tile + tr_lo + 32 * j), hi = lds_read_tr(tile + tr_hi + 32 * j);
      const u32x4 b = {lo[0], lo[1], hi[0], hi[1]};
      // D[h][t]: the lane holds 4 consecutive h of token li
#pragma unroll
      for (int i = 0; i < TF; ++i) acc[i][j] = mfma32<DT>(b, a[i], acc[i][j]);
    }
    wait_lgkm0();
    asm volatile("" ::: "memory");   // the next chunk's writes stay behind these reads
  }
  f32x4 (*part)[TF * 8][64] = reinterpret_cast<f32x4 (*)[TF * 8][64]>(smem);
  for (int half = kFewWaves / 2; half > 0; half >>= 1) {
    __syncthreads();         // the tiles, then the sums of the round before, are read
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int i = 0; i < TF; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) part[wave - half][i * 8 + j][lane] = acc[i][j];
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int i = 0; i < TF; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] += part[wave][i * 8 + j][lane];
    }
  }
  if (wave != 0) return;
#pragma unroll
  for (int i = 0; i < TF; ++i) {
    const int t = t0 + i * 16 + li;
    if (t >= p.T) continue;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int h = h0 + j * 16 + 4 * lq;
      if (h >= p.H) continue;      // H is a multiple of 8
      float* o = p.acc + (int64_t(blockIdx.y) * p.T + t) * p.H + h;
      f32x4 r;
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] = acc[i][j][e] * (1.f / kOperandScale<DT>);
      if (p.add) r += *reinterpret_cast<const f32x4*>(o);
      *reinterpret_cast<f32x4*>(o) = r;
    }
  }
}

// dx = g times the sum of the splits' fp32 shares, in order, rounded once.  A
// token that carries no loss gets zeros whatever its g.
template <int OUT>
__global__ __launch_bounds__(256) void xent_finish_kernel(const float* __restrict__ acc, int splits, int T, int H,
                                                          const float* __restrict__ dloss,
                                                          const int32_t* __restrict__ labels, int V,
                                                          void* __restrict__ out, int64_t ldo) {
  const int64_t all = int64_t(T) * H;
  for (int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4; i < all; i += int64_t(gridDim.x) * 1024) {
    f32x4 v = *reinterpret_cast<const f32x4*>(acc + i);
    for (int z = 1; z < splits; ++z) v += *reinterpret_cast<const f32x4*>(acc + z * all + i);
    const int64_t t = i / H, h = i - t * H;
    const bool counted = uint32_t(labels[t]) < uint32_t(V);
    const float g = counted ? dloss[t] : 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = counted ? v[e] * g : 0.f;   // by selection: W may hold Inf or NaN
    if constexpr (OUT == NM_F32) {
      *reinterpret_cast<f32x4*>(static_cast<float*>(out) + t * ldo + h) = v;
    } else {
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + t * ldo + h) =
          make_uint2(pack_half2<OUT>(v[0], v[1]), pack_half2<OUT>(v[2], v[3]));
    }
  }
}

int64_t up_to(int64_t n, int64_t q) { return (n + q - 1) / q * q; }

// Launches kern on a tilesA x tilesB x splits grid of C's workgroups.
template <class C, typename Kern, typename Args, typename... Rest>
hipError_t launch_tiles(Kern kern, const Args& args, int64_t tilesA, int64_t tilesB, int64_t splits, hipStream_t s,
                        Rest... rest) {
  if (tilesA * tilesB * C::THREADS > 0xFFFFFFFFll) return hipErrorInvalidValue;
  constexpr int lds = OutArea<C>::LDS;
  if (hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(kern), lds); e != hipSuccess) return e;
  // an XCD's run of tiles covers about 4 tiles of A by what fits of B
  const int group = int(std::min<int64_t>(tilesA, 4));
  hipLaunchKernelGGL(kern, dim3(unsigned(tilesA * tilesB), unsigned(splits)), dim3(C::THREADS), lds, s, args,
                     rest..., int(tilesA), int(tilesB), group);
  return hipGetLastError();
}

XentArgsDev dev_args(const XentArgs& a) {
  return XentArgsDev{a.x, a.w, a.labels, a.ldx, a.ldw, int(a.T), int(a.V), int(a.H)};
}

// Tiles of a product over words and tokens: as wide as so few tokens are, with
// 128 words (more workgroups); past 128 tokens the 256 x 256 tiles, whose
// operands are read half as often (T = 512 on 32000 x 4096, forward: 110 us
// against 190 with 128 x 128; T = 128: 81 against 55), unless they would leave
// half the chip idle (T = 200 on 4000 x 1024: 28 us against 20).
template <class Use>
auto with_tile(int64_t T, int64_t words, Use&& use) {
  if (T <= 16) return use(Tile16{});
  if (T <= 64) return use(Tile64{});
  if (T <= 128 || (T + 255) / 256 * ((words + 255) / 256) <= 128) return use(Tile128{});
  return use(TileBig{});
}
int64_t stats_tile_v(int64_t T, int64_t V) {
  return with_tile(T, V, [](auto tile) { return int64_t(decltype(tile)::BM); });
}

template <int DT, class C>
hipError_t stats(const XentArgs& a, float2* part, float* at_label, hipStream_t s) {
  return launch_tiles<C>(xent_stats_kernel<DT, C>, dev_args(a), (a.V + C::BM - 1) / C::BM, (a.T + C::BN - 1) / C::BN,
                         1, s, part, at_label);
}

template <int DT>
hipError_t forward_dt(const XentArgs& a, hipStream_t s) {
  const int64_t tilesV = (a.V + stats_tile_v(a.T, a.V) - 1) / stats_tile_v(a.T, a.V);
  float2* part = static_cast<float2*>(a.workspace);
  float* at_label = reinterpret_cast<float*>(part + tilesV * a.T);
  const hipError_t e =
      with_tile(a.T, a.V, [&](auto tile) { return stats<DT, decltype(tile)>(a, part, at_label, s); });
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(xent_join_kernel, dim3(unsigned((a.T + 63) / 64)), dim3(1024), 0, s, part, at_label, a.labels,
                     int(tilesV), int(a.T), int(a.V), a.loss, a.lse_out);
  return hipGetLastError();
}

// Up to this many tokens dx is a stream of W as it lies, past it a product with
// W transposed (forward and backward on 32000 x 4096: T = 128 331 us against
// 427, T = 200 545 against 519).
constexpr int64_t kFewTokens = 128;

// Where the backward pass keeps things in its workspace (bytes).
struct BwdPlan {
  int64_t piece, ldt, ldd, splits, ksplit;
  size_t xt, wt, d, dt, d_rest, dt_rest, acc, largest, total;
};

// dx and dw: parts of their operand (0: not wanted, 2: an fp32 output).  The
// vocabulary is cut into pieces of at most 2^26 logits (128 MB in each order and
// part): large enough that dx's fp32 sums, read and written once a piece,
// stay a few percent of its products.
BwdPlan plan_bwd(int64_t T, int64_t V, int64_t H, int dx, int dw) {
  BwdPlan p;
  p.ldt = up_to(T, 64);
  const int64_t most = std::max<int64_t>((int64_t(1) << 26) / std::max<int64_t>(p.ldt, 1) / 256 * 256, 256);
  const int64_t pieces = (V + most - 1) / most;
  p.piece = up_to((V + pieces - 1) / pieces, 256);
  p.ldd = p.piece;
  // dx has few tiles: its reduction is split until the chip is covered (for few
  // tokens twice, with tiles of all tokens by 128)
  const int64_t tiles = T <= kFewTokens ? ((H + 127) / 128 + 1) / 2 : ((T + 255) / 256) * ((H + 255) / 256);
  p.splits = std::min<int64_t>(std::max<int64_t>(256 / tiles, 1), std::max<int64_t>(p.piece / 512, 1));
  p.ksplit = up_to((p.piece + p.splits - 1) / p.splits, 64);
  p.splits = (p.piece + p.ksplit - 1) / p.ksplit;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  p.largest = take(4);
  p.xt = take(dw ? size_t(H) * p.ldt * 2 : 0);
  p.dt = take(dw ? size_t(p.piece) * p.ldt * 2 : 0);
  p.d = take(dx ? size_t(T) * p.ldd * 2 : 0);
  p.wt = take(dx && T > kFewTokens ? size_t(H) * p.ldd * 2 : 0);
  p.dt_rest = take(dw > 1 ? size_t(p.piece) * p.ldt * 2 : 0);
  p.d_rest = take(dx > 1 ? size_t(T) * p.ldd * 2 : 0);
  p.acc = take(dx ? size_t(p.splits) * T * H * 4 : 0);
  p.total = at;
  return p;
}

hipError_t transpose(const uint16_t* in, int64_t ldi, int64_t rows, int64_t cols, const int32_t* labels, int64_t V,
                     uint16_t* out, int64_t ldo, hipStream_t s) {
  hipLaunchKernelGGL(xent_transpose_kernel, dim3(unsigned((ldo + 63) / 64), unsigned((cols + 63) / 64)), dim3(256), 0,
                     s, in, ldi, int(rows), int(cols), labels, int(V), out, ldo);
  return hipGetLastError();
}

template <int DT>
hipError_t product(const XentProduct& p, int out_dtype, int64_t splits, hipStream_t s) {
  using C = TileBig;
  const int64_t tm = (p.M + C::BM - 1) / C::BM, tn = (p.N + C::BN - 1) / C::BN;
  return out_dtype == NM_F32 ? launch_tiles<C>(xent_product_kernel<DT, C, NM_F32>, p, tm, tn, splits, s)
                             : launch_tiles<C>(xent_product_kernel<DT, C, DT>, p, tm, tn, splits, s);
}

template <int DT>
hipError_t backward_dt(const XentArgs& a, hipStream_t s) {
  const bool dx2 = a.dx && a.dx_dtype == NM_F32, dw2 = a.dw && a.dw_dtype == NM_F32;
  const BwdPlan pl = plan_bwd(a.T, a.V, a.H, a.dx ? 1 + dx2 : 0, a.dw ? 1 + dw2 : 0);
  char* ws = static_cast<char*>(a.workspace);
  float* largest = reinterpret_cast<float*>(ws + pl.largest);
  uint16_t* xt = reinterpret_cast<uint16_t*>(ws + pl.xt);
  uint16_t* wt = reinterpret_cast<uint16_t*>(ws + pl.wt);
  float* acc = reinterpret_cast<float*>(ws + pl.acc);
  hipLaunchKernelGGL(xent_largest_kernel, dim3(1), dim3(1024), 0, s, a.dloss, a.labels, int(a.T), int(a.V), largest);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.dw && (e = transpose(a.x, a.ldx, a.T, a.H, a.labels, a.V, xt, pl.ldt, s)) != hipSuccess) return e;
  XentBwdDev b;
  b.a = dev_args(a);
  b.lse = a.lse;
  b.dloss = a.dloss;
  b.largest = largest;
  b.d = a.dx ? reinterpret_cast<uint16_t*>(ws + pl.d) : nullptr;
  b.dt = a.dw ? reinterpret_cast<uint16_t*>(ws + pl.dt) : nullptr;
  b.d_rest = dx2 ? reinterpret_cast<uint16_t*>(ws + pl.d_rest) : nullptr;
  b.dt_rest = dw2 ? reinterpret_cast<uint16_t*>(ws + pl.dt_rest) : nullptr;
  b.ldd = pl.ldd;
  b.ldt = pl.ldt;
  for (int64_t v0 = 0; v0 < a.V; v0 += pl.piece) {
    const int64_t vn = std::min(pl.piece, a.V - v0), vpad = up_to(vn, 64);
    b.v0 = int(v0);
    b.vn = int(vn);
    b.vpad = int(vpad);
    // (ldt is a multiple of 64, which the narrowest tile here has to cover)
    e = with_tile(std::max<int64_t>(a.T, 17), vpad, [&](auto tile) {
      using C = decltype(tile);
      return launch_tiles<C>(xent_dlogits_kernel<DT, C>, b, (vpad + C::BM - 1) / C::BM, (pl.ldt + C::BN - 1) / C::BN, 1,
                             s);
    });
    if (e != hipSuccess) return e;
    const int64_t splits = (vpad + pl.ksplit - 1) / pl.ksplit;
    // each product once for the rounded operand and, where there is one, once more for what it left
    if (a.dx && a.T <= kFewTokens) {
      FewDx p{a.w + v0 * a.ldw, b.d, a.ldw, pl.ldd, int(a.T), int(a.H), int(vn), int(vpad), int(pl.ksplit), acc, v0 > 0};
      const dim3 grid(unsigned((a.H + 127) / 128), unsigned(splits), unsigned((a.T + 63) / 64));
      auto go = [&] {
        if (a.T <= 16) hipLaunchKernelGGL((xent_dx_few_kernel<DT, 1>), grid, dim3(kFewWaves * 64), 0, s, p);
        else hipLaunchKernelGGL((xent_dx_few_kernel<DT, 4>), grid, dim3(kFewWaves * 64), 0, s, p);
        return hipGetLastError();
      };
      if ((e = go()) != hipSuccess) return e;
      p.d = b.d_rest;
      p.add = true;
      if (dx2 && (e = go()) != hipSuccess) return e;
    } else if (a.dx) {
      if ((e = transpose(a.w + v0 * a.ldw, a.ldw, vn, a.H, nullptr, 0, wt, pl.ldd, s)) != hipSuccess) return e;
      XentProduct p{wt, b.d, pl.ldd, pl.ldd, int(a.H), int(a.T), int(vpad), int(pl.ksplit), nullptr, acc, a.H,
                    a.T * a.H, v0 > 0};
      // (a last piece shorter than the others may need fewer splits: the rest keep their sums)
      if ((e = product<DT>(p, NM_F32, splits, s)) != hipSuccess) return e;
      p.Q = b.d_rest;
      p.add = true;
      if (dx2 && (e = product<DT>(p, NM_F32, splits, s)) != hipSuccess) return e;
    }
    if (a.dw) {
      const size_t es = dw2 ? 4 : 2;
      XentProduct p{xt, b.dt, pl.ldt, pl.ldt, int(a.H), int(vn), int(pl.ldt), int(pl.ldt), largest,
                    static_cast<char*>(a.dw) + size_t(v0) * a.lddw * es, a.lddw, 0, false};
      if ((e = product<DT>(p, a.dw_dtype, 1, s)) != hipSuccess) return e;
      p.Q = b.dt_rest;
      p.add = true;
      if (dw2 && (e = product<DT>(p, a.dw_dtype, 1, s)) != hipSuccess) return e;
    }
  }
  if (a.dx) {
    const unsigned grid = unsigned(std::min<int64_t>((a.T * a.H / 4 + 255) / 256, int64_t(1) << 20));
    const int splits = int((std::min(pl.piece, up_to(a.V, 64)) + pl.ksplit - 1) / pl.ksplit);
    if (a.dx_dtype == NM_F32)
      hipLaunchKernelGGL((xent_finish_kernel<NM_F32>), dim3(grid), dim3(256), 0, s, acc, splits, int(a.T), int(a.H),
                         a.dloss, a.labels, int(a.V), a.dx, a.lddx);
    else
      hipLaunchKernelGGL((xent_finish_kernel<DT>), dim3(grid), dim3(256), 0, s, acc, splits, int(a.T), int(a.H),
                         a.dloss, a.labels, int(a.V), a.dx, a.lddx);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

size_t xent_workspace(int64_t T, int64_t V) {
  const int64_t tilesV = (V + stats_tile_v(T, V) - 1) / stats_tile_v(T, V);
  return size_t(tilesV) * T * 8 + size_t(T) * 4;
}

size_t xent_bwd_workspace(int64_t T, int64_t V, int64_t H, int dx, int dw) {
  return T == 0 ? 0 : plan_bwd(T, V, H, dx, dw).total;
}

hipError_t launch_xent(const XentArgs& a, hipStream_t s) {
  return a.dtype == NM_F16 ? forward_dt<NM_F16>(a, s) : forward_dt<NM_BF16>(a, s);
}

// T == 0: dw is zeros.
static __global__ __launch_bounds__(256) void xent_zero_kernel(uint16_t* out, int64_t ldo, int rows, int cols) {
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
    for (int c = threadIdx.x; c < cols; c += 256) out[r * ldo + c] = 0;
}

hipError_t launch_xent_bwd(const XentArgs& a, hipStream_t s) {
  if (a.T == 0) {
    if (!a.dw) return hipSuccess;
    const int64_t k = a.dw_dtype == NM_F32 ? 2 : 1;   // in 16-bit units
    hipLaunchKernelGGL(xent_zero_kernel, dim3(unsigned(std::min<int64_t>(a.V, 65536))), dim3(256), 0, s,
                       static_cast<uint16_t*>(a.dw), a.lddw * k, int(a.V), int(a.H * k));
    return hipGetLastError();
  }
  return a.dtype == NM_F16 ? backward_dt<NM_F16>(a, s) : backward_dt<NM_BF16>(a, s);
}

}  // namespace nm
