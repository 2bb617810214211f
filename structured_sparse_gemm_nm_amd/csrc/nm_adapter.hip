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
// Tokens of an adapter are found where they lie: a tile of 64 tokens is
// multiplied once for every adapter that occurs in it, and each token keeps its
// own adapter's result.  Requests whose tokens are adjacent cost one product a
// tile, two where they meet; any other order is right and costs more.
//
// The shrunk activations are fp32 (nothing between the two products is
// rounded to 16 bits).  All three kernels are bound by reading what they
// multiply: x or g once for the shrink and the gradients, Y once for the
// expand; the adapters themselves are small.  The expand step costs no pass of
// its own where the shared product's kernel holds its tile in registers and
// adds the term there (few tokens, 2:4 prefill, and dx).
#include "nm_gemm_nt.h"
#include "nm_internal.h"
#include "nm_lowrank.h"

#include <algorithm>
#include <type_traits>

namespace nm {
namespace {

__device__ inline u32x4 load16(__amdgpu_buffer_rsrc_t rsrc, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, off, 0, 0));
}

// ---------------------------------------------------------------------------
// Shrink: V[t][j] = s_a sum_c M_a[j][c] Z[t][c], M as [n][r][C].
// The product of a 64-token tile with one adapter's 32 or 64 ranks is far too
// small for the chip, so its columns are split over blockIdx.y and the shares,
// part[split][t][j], are added in order by adapter_join_kernel.  Loading whole
// 128-byte lines into LDS (gemm_nt) matters more than the few operations: with
// operand fragments loaded straight into registers (16 rows of 64 bytes an
// instruction) 2048 tokens x 4096, rank 32, took 13 us in place of SHRINK_US.
// Several adapters in a tile are dealt to blockIdx.z in turn.
// ---------------------------------------------------------------------------
struct ShrinkArgs {
  const int32_t* ids;
  const uint16_t* M;
  const uint16_t* Z;
  int64_t ldz;
  int n, T, C, r, csplit;   // a split takes csplit columns (a multiple of 64)
  float* part;              // [splits][T][r]
};

template <int DT, class C>
__global__ __launch_bounds__(C::THREADS) void adapter_shrink_kernel(ShrinkArgs p, int rank_tiles) {
  extern __shared__ __align__(16) unsigned char smem[];
  static_assert(C::BN == 64, "a lane a token");
  const int tt = blockIdx.x / rank_tiles, tr = blockIdx.x - tt * rank_tiles;
  const int t = tt * 64 + (threadIdx.x & 63);
  const int id = t < p.T ? p.ids[t] : -1;
  // every wave holds the same ids, so the loop and its barriers are uniform
  uint64_t todo = __ballot(uint32_t(id) < uint32_t(p.n));
  const int c0 = blockIdx.y * p.csplit, K = min(p.C - c0, p.csplit);
  float* part = p.part + int64_t(blockIdx.y) * p.T * p.r;
  for (uint32_t turn = 0; todo; ++turn) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    const uint64_t mine = __ballot(id == a);
    todo &= ~mine;
    if (turn % gridDim.z != blockIdx.z) continue;
    gemm_nt<DT, C>(p.M + int64_t(a) * p.r * p.C + c0, p.C, p.r, p.Z + c0, p.ldz, p.T, K, tr, tt, smem,
                   [&](auto& acc, int wm, int wn, int li, int lq) {
#pragma unroll
      for (int j = 0; j < C::FN; ++j) {
        const int k = wn * C::FN * 16 + j * 16 + li;
        if (!((mine >> k) & 1u)) continue;
        float* row = part + int64_t(tt * 64 + k) * p.r;
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int q = tr * C::BM + wm * C::FM * 16 + i * 16 + 4 * lq + e;
            if (q < p.r) row[q] = acc[i][j][e];
          }
      }
    });
  }
}

// One of the join's jobs: value = now_a sum of `splits` shares [T][r], in
// order; zero for a token without an adapter.  Written where wanted: the fp32
// value; next_a value in three bf16 parts, [T][3][r8] for the products over
// ranks (lowrank_add) and [3][r][ldt] for those over tokens (the gradients).
struct JoinJob {
  const float* part;
  int splits;
  const float* now;     // or null: 1
  const float* next;    // or null: 1
  float* V;
  uint16_t* P;
  uint16_t* PT;
};

// A thread an element (j runs to r8, where P holds zeros); blockIdx.y is the job.
__global__ __launch_bounds__(256) void adapter_join_kernel(JoinJob first, JoinJob second,
                                                           const int32_t* __restrict__ ids, int n, int T, int r,
                                                           int ldt) {
  const JoinJob& q = blockIdx.y ? second : first;
  const int r8 = (r + 7) & ~7;
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= int64_t(T) * r8) return;
  const int64_t t = i / r8, all = int64_t(T) * r;
  const int j = int(i - t * r8);
  float v = 0.f;
  if (j < r) {
    const int64_t at = t * r + j;
    const int a = ids[t];
#pragma unroll 8
    for (int s = 0; s < q.splits; ++s) v += q.part[s * all + at];
    const bool some = uint32_t(a) < uint32_t(n);
    v = some ? (q.now ? v * q.now[a] : v) : 0.f;
    if (q.V) q.V[at] = v;
    if (some && q.next) v *= q.next[a];
  }
  uint16_t h[3];
  split3(v, h);
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (q.P) q.P[(t * 3 + k) * r8 + j] = h[k];
    if (q.PT && j < r) q.PT[(int64_t(k) * r + j) * ldt + t] = h[k];
  }
}

// Mt[a][j][c] = M[a][c][j] for M [n][C][r]: B's columns along the reduction of
// the backward pass's shrink, and (with the roles of C and r exchanged) A's
// ranks along that of its expand; one launch does both, the first tiles B's.
// A workgroup takes 64 of the long and 32 of the short index.
struct TransposeSide {
  const uint16_t* M;
  uint16_t* Mt;
  int rows, cols;       // of M
  int tiles;            // workgroups
};

__global__ __launch_bounds__(256) void adapter_transpose_kernel(TransposeSide first, TransposeSide second) {
  __shared__ uint16_t tile[64][64 + 2];
  const bool two = int(blockIdx.x) >= first.tiles;
  const TransposeSide& s = two ? second : first;
  const int b = blockIdx.x - (two ? first.tiles : 0), across = (s.cols + 63) / 64;
  const int r0 = b / across * 64, c0 = b % across * 64;
  const int64_t each = int64_t(s.rows) * s.cols;
  const uint16_t* m = s.M + blockIdx.y * each;
  uint16_t* mt = s.Mt + blockIdx.y * each;
  const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int row = r0 + y + 4 * i, col = c0 + x;
    tile[y + 4 * i][x] = m[int64_t(min(row, s.rows - 1)) * s.cols + min(col, s.cols - 1)];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int col = c0 + y + 4 * i, row = r0 + x;
    if (col < s.cols && row < s.rows) mt[int64_t(col) * s.rows + row] = tile[x][y + 4 * i];
  }
}

// The same for few tokens, M as [r][C]: a wave takes one number, V[t][j], with
// all its loads (16 bytes a lane of both rows, 4096 columns at a time) in
// flight at once.  Every token may have its own adapter.
template <int DT>
__global__ __launch_bounds__(256) void adapter_dots_kernel(const int32_t* __restrict__ ids, int n,
                                                           const uint16_t* __restrict__ M,
                                                           const float* __restrict__ now,
                                                           const uint16_t* __restrict__ Z, int64_t ldz, int T, int C,
                                                           int r, float* __restrict__ V) {
  const int lane = threadIdx.x & 63;
  const int dot = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (dot >= T * r) return;
  const int t = dot / r, j = dot - t * r;
  const int a = ids[t];
  float sum = 0.f;
  if (uint32_t(a) < uint32_t(n)) {
    const __amdgpu_buffer_rsrc_t rz = make_rsrc(Z + int64_t(t) * ldz, uint32_t(C) * 2u);
    const __amdgpu_buffer_rsrc_t rm = make_rsrc(M + (int64_t(a) * r + j) * C, uint32_t(C) * 2u);
    for (int c0 = 0; c0 < C; c0 += 4096) {
      u32x4 z[8], m[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {   // pieces past C lie past both descriptors: zeros
        z[i] = load16(rz, uint32_t(c0 + (i * 64 + lane) * 8) * 2u);
        m[i] = load16(rm, uint32_t(c0 + (i * 64 + lane) * 8) * 2u);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          sum += half_to_f32<DT>((z[i][e >> 1] >> (16 * (e & 1))) & 0xFFFFu) *
                 half_to_f32<DT>((m[i][e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
    if (now) sum *= now[a];
  }
  if (lane == 0) V[dot] = sum;
}

// ---------------------------------------------------------------------------
// Expand: Y[t][c] = base[t][c] + (low-rank term), base fp32 (Y itself or a
// workspace).  A wave takes 16 tokens x 64 columns.
// ---------------------------------------------------------------------------
template <int DT, int OUT>
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
    const float* b = base + int64_t(t) * ldb + c;
    if ((ldb & 3) == 0 && c + 3 < p.C) acc[f] = *reinterpret_cast<const f32x4*>(b);
    else
      for (int e = 0; e < 4 && c + e < p.C; ++e) acc[f][e] = b[e];
  }
  lowrank_add<DT, 4, 1>(p, lowrank_ids<1>(p, t0), t0, c0, [&](int f, int) -> f32x4& { return acc[f]; });
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
// Gradients: D_a[j][c] = sum_{t in a} V[t][j] Z[t][c], written [r][C] (dA, Z =
// x, V = u) or [C][r] (dB, Z = g, V = s xa); one launch does both, the first
// column tiles dA's, the rest dB's.  A workgroup of 8 waves owns one adapter,
// RF*16 ranks and CF*16 columns.  The tokens are gone through 4096 at a time:
// the workgroup marks each 32-token chunk's tokens of the adapter in LDS and
// lists the chunks that hold any; the waves take them in turn, each loading its
// next chunk while it multiplies one, and in the end the waves' tiles are added
// in a fixed order.  The reduction runs over the rows of Z, so a wave brings
// its chunk's tile into LDS (16 bytes a lane, rows as they lie) and takes the
// operands out by transpose reads; V's parts lie along the tokens already (16
// bytes a lane and part).  Picking Z's operands 2 bytes a lane from memory, or
// V's 4, is bound by issuing loads (GRAD_US).  Tokens of other adapters are
// selected to zero in both operands, so an Inf or NaN among them reaches
// nothing.  An adapter without tokens gets zeros.
// ---------------------------------------------------------------------------
constexpr int kGradWaves = 8;
constexpr int kGradSpan = 4096, kGradChunks = kGradSpan / 32;

struct GradSide {
  const uint16_t* VT;   // [3][r][ldt]: V's parts
  const uint16_t* Z;    // [T][C]
  int64_t ldz;
  int C, tiles;
  float* out;
};
struct GradArgs {
  const int32_t* ids;
  int T, r, ldt;        // ldt: T rounded up to 32
  GradSide a, b;        // dA, written [r][C]; dB, written [C][r]
};

// A wave's staged tile: token row t starts at P t + 128 (t >> 3 & 1) + 128 (t >> 4)
// with P = 32 bytes past the row, so that the transpose reads of 32 lanes (rows
// 8g + j) fall in distinct banks.
template <int CF>
struct GradTile {
  static constexpr int PITCH = CF * 32 + 32;
  __host__ __device__ static constexpr int row(int t) { return t * PITCH + (((t >> 3) & 1) + (t >> 4)) * 128; }
  static constexpr int BYTES = (row(31) + CF * 32 + 15) / 16 * 16;
};

template <int DT, int RF, int CF>
__global__ __launch_bounds__(kGradWaves * 64) void adapter_grad_kernel(GradArgs g) {
  using Tile = GradTile<CF>;
  extern __shared__ __align__(16) unsigned char smem[];   // the waves' tiles; in the end their sums
  __shared__ uint32_t mark[kGradChunks];
  __shared__ uint8_t list[kGradChunks];
  const int lane = threadIdx.x & 63, li = lane & 15, lq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool rank_minor = int(blockIdx.x) >= g.a.tiles;
  const GradSide& z = rank_minor ? g.b : g.a;
  const int c0 = (blockIdx.x - (rank_minor ? g.a.tiles : 0)) * (CF * 16), r0 = blockIdx.y * (RF * 16), a = blockIdx.z;
  const int r = g.r, C = z.C;
  unsigned char* tile = smem + wave * Tile::BYTES;
  f32x4 acc[RF][CF];
#pragma unroll
  for (int i = 0; i < RF; ++i)
#pragma unroll
    for (int j = 0; j < CF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  // this lane's piece of a row of the tile, and its row among those of a load
  constexpr int PPR = CF * 2, RPL = 64 / PPR;   // 16-byte pieces a row, rows a load
  const int piece = lane % PPR, prow = lane / PPR;
  const bool inside = c0 + piece * 8 < C;       // C is a multiple of 8
  // transpose reads: lane 16g + 4j + e reads token rows 8g + j and 8g + j + 4
  const int tr_row = 8 * (lane >> 4) + ((lane >> 2) & 3);
  const int tr_lo = Tile::row(tr_row) + 8 * (lane & 3), tr_hi = Tile::row(tr_row + 4) + 8 * (lane & 3);

  bool any = false;                       // the same in every wave
  for (int64_t base = 0; base < g.T; base += kGradSpan) {
    __syncthreads();                      // the marks of the span before are read
#pragma unroll
    for (int i = 0; i < kGradSpan / (kGradWaves * 64); ++i) {
      const int64_t t = base + (i * kGradWaves + wave) * 64 + lane;
      const uint64_t in = __ballot(t < g.T && g.ids[t < g.T ? t : 0] == a);
      if (lane < 2) mark[(i * kGradWaves + wave) * 2 + lane] = uint32_t(in >> (32 * lane));
    }
    __syncthreads();
    // the chunks that hold a token of the adapter, listed in order
    const uint64_t some[2] = {__ballot(mark[lane] != 0), __ballot(mark[64 + lane] != 0)};
    const int count = __builtin_popcountll(some[0]) + __builtin_popcountll(some[1]);
    if (wave < 2) {
      const uint64_t below = some[wave] & ((uint64_t(1) << lane) - 1);
      if ((some[wave] >> lane) & 1u)
        list[__builtin_popcountll(below) + (wave ? __builtin_popcountll(some[0]) : 0)] = uint8_t(wave * 64 + lane);
    }
    __syncthreads();
    // chunk i's rows of Z and V; loads are unconditional (tokens past T reread
    // the last) and selected when used, so that all are in flight together
    auto load = [&](int i, u32x4 (&x)[32 / RPL], u32x4 (&v)[RF][3]) {
      const int64_t t0 = base + list[i] * 32;
#pragma unroll
      for (int k = 0; k < 32 / RPL; ++k) {
        const int64_t t = min(t0 + k * RPL + prow, int64_t(g.T) - 1);
        x[k] = *reinterpret_cast<const u32x4*>(z.Z + t * z.ldz + (inside ? c0 + piece * 8 : 0));
      }
#pragma unroll
      for (int i = 0; i < RF; ++i)
#pragma unroll
        for (int k = 0; k < 3; ++k)
          v[i][k] = *reinterpret_cast<const u32x4*>(
              z.VT + (int64_t(k) * r + min(r0 + i * 16 + li, r - 1)) * g.ldt + t0 + 8 * lq);
      __builtin_amdgcn_sched_barrier(0);
    };
    u32x4 x[32 / RPL], v[RF][3];
    if (wave < count) load(wave, x, v);
    for (int i = wave; i < count; i += kGradWaves) {
      const uint32_t mine = mark[list[i]];
#pragma unroll
      for (int k = 0; k < 32 / RPL; ++k) {
        const int row = k * RPL + prow;
        const bool sel = inside && ((mine >> row) & 1u);
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = sel ? x[k][e] : 0u;
        *reinterpret_cast<u32x4*>(tile + Tile::row(row) + piece * 16) = w;
      }
      // this lane's 8 tokens (8 lq ..) as a mask of halves
      uint32_t keep[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        keep[e] = ((mine >> (8 * lq + 2 * e)) & 1u ? 0xFFFFu : 0u) |
                  ((mine >> (8 * lq + 2 * e + 1)) & 1u ? 0xFFFF0000u : 0u);
      u32x4 vp[RF][3];
#pragma unroll
      for (int q = 0; q < RF; ++q)
#pragma unroll
        for (int k = 0; k < 3; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) vp[q][k][e] = v[q][k][e] & keep[e];
      __builtin_amdgcn_sched_barrier(0);
      // x and v are used up: the next chunk's rows arrive while this one is multiplied
      if (i + kGradWaves < count) load(i + kGradWaves, x, v);
      // a wave's LDS operations are carried out in order: no barrier
      wait_lgkm0();
      asm volatile("" ::: "memory");
#pragma unroll
      for (int j = 0; j < CF; ++j) {
        const u32x2 lo = lds_read_tr(tile + tr_lo + 32 * j), hi = lds_read_tr(tile + tr_hi + 32 * j);
        u32x4 zp[operand_count<DT>()];
        operand_parts<DT>(u32x4{lo[0], lo[1], hi[0], hi[1]}, zp);
#pragma unroll
        for (int q = 0; q < RF; ++q) acc[q][j] = mfma_parts(vp[q], zp, acc[q][j]);
      }
      wait_lgkm0();
      asm volatile("" ::: "memory");   // the next chunk's writes stay behind these reads
    }
    any |= count > 0;
  }
  // waves 4..7 onto 0..3, 2..3 onto 0..1, 1 onto 0
  f32x4 (*part)[RF * CF][64] = reinterpret_cast<f32x4 (*)[RF * CF][64]>(smem);
  if (any) __syncthreads();               // every wave is done with its tile
  for (int half = any ? kGradWaves / 2 : 0; half > 0; half >>= 1) {
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
  float* out = z.out + int64_t(a) * r * C;
#pragma unroll
  for (int i = 0; i < RF; ++i)
#pragma unroll
    for (int j = 0; j < CF; ++j) {
      const int c = c0 + j * 16 + li, q = r0 + i * 16 + lq * 4;
      if (c >= C) continue;
      if (rank_minor && (r & 3) == 0) {
        if (q < r) *reinterpret_cast<f32x4*>(out + int64_t(c) * r + q) = acc[i][j];
        continue;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (q + e < r) out[rank_minor ? int64_t(c) * r + q + e : int64_t(q + e) * C + c] = acc[i][j][e];
    }
}

// Up to this many tokens a wave computes one number of V: past it, a token's
// row would be read by too many waves.
constexpr int64_t kFewTokens = 16;

using ShrinkTile32 = GemmTile<32, 64, 2, 2, 4>;   // ranks x tokens, 48 KB: three workgroups a CU
using ShrinkTile64 = GemmTile<64, 64, 4, 1, 4>;

// Splits of the shrink's columns and their width: enough workgroups to cover
// the chip twice, shares of at least 256 columns.
struct ShrinkPlan {
  int64_t splits, csplit;
};
ShrinkPlan shrink_plan(int64_t T, int64_t C, int64_t r) {
  if (C == 0) return {0, 64};   // an empty sum
  const int64_t tiles = (T + 63) / 64 * (r <= 32 ? 1 : (r + 63) / 64);
  const int64_t want = std::min<int64_t>(std::max<int64_t>(512 / tiles, 1), std::max<int64_t>(C / 256, 1));
  const int64_t csplit = ((C + want - 1) / want + 63) / 64 * 64;
  return {(C + csplit - 1) / csplit, csplit};
}

// Bytes of the shrink's shares (0: none are kept).
size_t shrink_bytes(int64_t T, int64_t C, int64_t r) {
  return T <= kFewTokens ? 0 : size_t(shrink_plan(T, C, r).splits) * size_t(T) * size_t(r) * 4;
}

template <int DT, class C>
hipError_t launch_shrink(const ShrinkArgs& p, int64_t splits, hipStream_t s) {
  auto kern = adapter_shrink_kernel<DT, C>;
  if (hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(kern), C::LDS); e != hipSuccess) return e;
  const int rank_tiles = (p.r + C::BM - 1) / C::BM;
  // two adapters of a tile at a time, where there can be two
  hipLaunchKernelGGL(kern, dim3(unsigned((p.T + 63) / 64 * rank_tiles), unsigned(splits), p.n > 1 ? 2u : 1u),
                     dim3(C::THREADS), C::LDS, s, p, rank_tiles);
  return hipGetLastError();
}

hipError_t join(const JoinJob& first, const JoinJob* second, const int32_t* ids, int64_t n, int64_t T, int64_t r,
                int64_t ldt, hipStream_t s) {
  hipLaunchKernelGGL(adapter_join_kernel, dim3(unsigned((T * ((r + 7) / 8 * 8) + 255) / 256), second ? 2u : 1u),
                     dim3(256), 0, s, first, second ? *second : first, ids, int(n), int(T), int(r), int(ldt));
  return hipGetLastError();
}

// now_a M Z as `out` wants it (out.V is written in any case; out.part and
// out.splits are filled in here), and a second job along with it.
template <int DT>
hipError_t shrink(const int32_t* ids, int64_t n, const uint16_t* M, const uint16_t* Z, int64_t ldz, int64_t T, int64_t C,
                  int64_t r, float* part, JoinJob out, const JoinJob* second, int64_t ldt, hipStream_t s) {
  if (T <= kFewTokens) {
    hipLaunchKernelGGL((adapter_dots_kernel<DT>), dim3(unsigned((T * r + 3) / 4)), dim3(256), 0, s, ids, int(n), M,
                       out.now, Z, ldz, int(T), int(C), int(r), out.V);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    if (!out.P && !out.PT && !second) return hipSuccess;
    out.part = out.V;     // whole and scaled already
    out.V = nullptr;
    out.splits = 1;
    out.now = nullptr;
    return join(out, second, ids, n, T, r, ldt, s);
  }
  const ShrinkPlan pl = shrink_plan(T, C, r);
  const ShrinkArgs p{ids, M, Z, ldz, int(n), int(T), int(C), int(r), int(pl.csplit), part};
  if (n > 0 && pl.splits > 0) {
    const hipError_t e =
        r <= 32 ? launch_shrink<DT, ShrinkTile32>(p, pl.splits, s) : launch_shrink<DT, ShrinkTile64>(p, pl.splits, s);
    if (e != hipSuccess) return e;
  }
  out.part = part;
  out.splits = int(pl.splits);
  return join(out, second, ids, n, T, r, ldt, s);
}

template <int DT>
hipError_t expand(const LowRank& p, const float* base, int64_t ldb, void* Y, int64_t ldy, int out_dtype,
                  hipStream_t s) {
  const dim3 grid(unsigned((p.T + 15) / 16), unsigned((p.C + 255) / 256));
  if (out_dtype == NM_F32)
    hipLaunchKernelGGL((adapter_expand_kernel<DT, NM_F32>), grid, dim3(256), 0, s, p, base, ldb, Y, ldy);
  else
    hipLaunchKernelGGL((adapter_expand_kernel<DT, DT>), grid, dim3(256), 0, s, p, base, ldb, Y, ldy);
  return hipGetLastError();
}

template <int DT>
hipError_t gradients(GradArgs g, int64_t n, hipStream_t s) {
  auto go = [&](auto kern, auto rfc, auto cfc) {
    constexpr int RF = decltype(rfc)::value, CF = decltype(cfc)::value;
    constexpr int lds = std::max(kGradWaves * GradTile<CF>::BYTES, kGradWaves / 2 * RF * CF * 1024);
    if (hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(kern), lds); e != hipSuccess) return e;
    g.a.tiles = (g.a.C + CF * 16 - 1) / (CF * 16);
    g.b.tiles = (g.b.C + CF * 16 - 1) / (CF * 16);
    hipLaunchKernelGGL(kern, dim3(unsigned(g.a.tiles + g.b.tiles), unsigned((g.r + RF * 16 - 1) / (RF * 16)),
                                  unsigned(n)),
                       dim3(kGradWaves * 64), lds, s, g);
    return hipGetLastError();
  };
  using one = std::integral_constant<int, 1>;
  using two = std::integral_constant<int, 2>;
  using four = std::integral_constant<int, 4>;
  using eight = std::integral_constant<int, 8>;
  // 128 columns a workgroup where that still covers the chip, else 64
  const bool wide = (int64_t(g.a.C) + g.b.C) / 128 * n >= 256;
  if (g.r <= 16)
    return wide ? go(adapter_grad_kernel<DT, 1, 8>, one{}, eight{}) : go(adapter_grad_kernel<DT, 1, 4>, one{}, four{});
  if (g.r <= 32)
    return wide ? go(adapter_grad_kernel<DT, 2, 8>, two{}, eight{}) : go(adapter_grad_kernel<DT, 2, 4>, two{}, four{});
  return go(adapter_grad_kernel<DT, 4, 4>, four{}, four{});
}

// Whether the shared product's kernel adds the low-rank term itself: the
// few-token family (T <= 16) and the all-LDS family (prefill, 2:4).
bool fused_forward(const SpmmArgs& b) { return spmm_decode_applies(b) || spmm_lds_applies(b); }

// Parts of the workspaces, each on 256 bytes.
size_t padded(size_t bytes) { return (bytes + 255) / 256 * 256; }
size_t parts_bytes(int64_t T, int64_t r) { return padded(size_t(T) * 3 * ((r + 7) / 8 * 8) * 2); }

template <int DT>
hipError_t forward_dt(const AdapterArgs& a, hipStream_t s) {
  const int64_t T = a.base.T;
  // the few-token family multiplies V itself
  const bool few = spmm_decode_applies(a.base);
  char* ws = static_cast<char*>(a.workspace);
  uint16_t* P = few ? nullptr : reinterpret_cast<uint16_t*>(ws);
  char* rest = ws + (few ? 0 : parts_bytes(T, a.r));   // the shares, and when they are joined the fp32 product
  const JoinJob out{nullptr, 0, nullptr, a.scale, a.xa, P, nullptr};
  hipError_t e = shrink<DT>(a.ids, a.n, a.A, a.base.act, a.base.ldx, T, a.base.K, a.r, reinterpret_cast<float*>(rest),
                            out, nullptr, 0, s);
  if (e != hipSuccess || a.base.R == 0) return e;
  LowRank p;
  p.ids = a.ids;
  p.M = a.B;
  p.scale = a.scale;
  p.V = a.xa;
  p.P = P;
  p.n = int(a.n);
  p.r = int(a.r);
  p.T = int(T);
  p.C = int(a.base.R);
  SpmmArgs b = a.base;
  if (fused_forward(b)) {
    b.lowrank = &p;
    return few ? launch_spmm_decode(b, s) : launch_spmm_lds(b, s);
  }
  if (a.base.out_dtype != NM_F32) {
    b.Y = rest;
    b.ldy = a.base.R;
    b.out_dtype = NM_F32;
  }
  e = launch_spmm(b, s);
  if (e != hipSuccess) return e;
  return expand<DT>(p, static_cast<const float*>(b.Y), b.ldy, a.base.Y, a.base.ldy, a.base.out_dtype, s);
}

// The backward pass's workspace: u, its parts, u's and s xa's parts along the
// tokens, B and A transposed, the shares.
struct BwdParts {
  int64_t ldt;
  size_t u, p, ut, xt, bt, at, part, total;
};
BwdParts bwd_parts(int64_t R, int64_t K, int64_t T, int64_t n, int64_t r) {
  BwdParts b;
  b.ldt = (T + 31) / 32 * 32;
  b.u = 0;
  b.p = b.u + padded(size_t(T) * r * 4);
  b.ut = b.p + parts_bytes(T, r);
  b.xt = b.ut + padded(size_t(b.ldt) * r * 6);
  b.bt = b.xt + padded(size_t(b.ldt) * r * 6);
  b.at = b.bt + padded(size_t(n) * r * R * 2);
  b.part = b.at + padded(size_t(n) * r * K * 2);
  b.total = b.part + shrink_bytes(T, R, r);
  return b;
}

template <int DT>
hipError_t backward_dt(const AdapterBwdArgs& a, hipStream_t s) {
  TrainArgs d = a.dx;
  const BwdParts w = bwd_parts(d.R, d.K, d.T, a.n, a.r);
  char* ws = static_cast<char*>(a.workspace);
  float* u = reinterpret_cast<float*>(ws + w.u);
  uint16_t* P = reinterpret_cast<uint16_t*>(ws + w.p);
  uint16_t* ut = reinterpret_cast<uint16_t*>(ws + w.ut);
  uint16_t* xt = reinterpret_cast<uint16_t*>(ws + w.xt);
  uint16_t* bt = reinterpret_cast<uint16_t*>(ws + w.bt);
  uint16_t* at = reinterpret_cast<uint16_t*>(ws + w.at);
  hipError_t e = hipSuccess;
  if (d.T > 0) {
    if (a.n > 0) {
      auto tiles = [](int64_t rows, int64_t cols) { return int((rows + 63) / 64 * ((cols + 63) / 64)); };
      const TransposeSide tb{a.B, bt, int(d.R), int(a.r), tiles(d.R, a.r)};
      const TransposeSide ta{a.A, at, int(a.r), int(d.K), d.out ? tiles(a.r, d.K) : 0};
      if (tb.tiles + ta.tiles > 0)
        hipLaunchKernelGGL(adapter_transpose_kernel, dim3(unsigned(tb.tiles + ta.tiles), unsigned(a.n)), dim3(256), 0,
                           s, tb, ta);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const JoinJob mine{nullptr, 0, a.scale, nullptr, u, P, ut};
    const JoinJob other{a.xa, 1, a.scale, nullptr, nullptr, nullptr, xt};
    e = shrink<DT>(a.ids, a.n, bt, d.G, d.ldg, d.T, d.R, a.r, reinterpret_cast<float*>(ws + w.part), mine, &other, w.ldt,
                   s);
    if (e != hipSuccess) return e;
  }
  if (d.out && d.T > 0) {
    LowRank p;
    p.ids = a.ids;
    p.M = at;
    p.V = u;
    p.P = P;
    p.n = int(a.n);
    p.r = int(a.r);
    p.T = int(d.T);
    p.C = int(d.K);
    d.lowrank = &p;
    e = launch_spmm_dx(d, s);
    if (e != hipSuccess) return e;
  }
  if (a.n == 0) return e;
  const GradArgs g{a.ids, int(d.T), int(a.r), int(w.ldt), GradSide{ut, d.act, d.ldx, int(d.K), 0, a.dA},
                   GradSide{xt, d.G, d.ldg, int(d.R), 0, a.dB}};
  return gradients<DT>(g, a.n, s);
}

}  // namespace

size_t adapter_workspace(const SpmmArgs& base, int64_t r) {
  if (spmm_decode_applies(base)) return 0;
  const size_t y = base.out_dtype == NM_F32 || fused_forward(base) ? 0 : size_t(base.T) * size_t(base.R) * 4;
  return parts_bytes(base.T, r) + std::max(shrink_bytes(base.T, base.K, r), y);
}

size_t adapter_bwd_workspace(int64_t R, int64_t K, int64_t T, int64_t n, int64_t r) {
  return bwd_parts(R, K, T, n, r).total;
}

hipError_t launch_adapter(const AdapterArgs& a, hipStream_t s) {
  return a.base.dtype == NM_F16 ? forward_dt<NM_F16>(a, s) : forward_dt<NM_BF16>(a, s);
}

hipError_t launch_adapter_bwd(const AdapterBwdArgs& a, hipStream_t s) {
  return a.dx.dtype == NM_F16 ? backward_dt<NM_F16>(a, s) : backward_dt<NM_BF16>(a, s);
}

}  // namespace nm
