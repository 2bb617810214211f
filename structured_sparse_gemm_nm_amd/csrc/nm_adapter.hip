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
#include "nm_internal.h"
#include "nm_lowrank.h"
#include "nm_piece.h"

#include <algorithm>
#include <type_traits>

namespace nm {
namespace {

__device__ inline u32x4 load16(__amdgpu_buffer_rsrc_t rsrc, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, off, 0, 0));
}

// What is written of shrunk values V [T][r]: the fp32 value, and next_a V in
// three bf16 parts, P [T][3][r8] for the products over ranks (lowrank_add) and
// PT [3][r][ldt] for those over tokens (the gradients).  Each may be null.
struct ShrunkOut {
  const float* next;    // the adapter's factor in the parts, or null: 1
  float* V;
  uint16_t* P;
  uint16_t* PT;
  int ldt;
};

// Element j < r8 of token t, whose adapter is a (or none: zeros).
__device__ inline void put_shrunk(const ShrunkOut& o, int64_t t, int j, int r, bool some, int a, float v) {
  const int r8 = (r + 7) & ~7;
  v = some && j < r ? v : 0.f;
  if (o.V && j < r) o.V[t * r + j] = v;
  if (!o.P && !o.PT) return;
  if (some && o.next) v *= o.next[a];
  uint16_t h[3];
  split3(v, h);
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (o.P) o.P[(t * 3 + k) * r8 + j] = h[k];
    if (o.PT && j < r) o.PT[(int64_t(k) * r + j) * o.ldt + t] = h[k];
  }
}

// The parts of a V that is already there: a thread an element.
__device__ inline void parts_of(const float* V, const ShrunkOut& o, const int32_t* ids, int n, int T, int r,
                                int64_t i) {
  const int r8 = (r + 7) & ~7;
  if (i >= int64_t(T) * r8) return;
  const int64_t t = i / r8;
  const int j = int(i - t * r8), a = ids[t];
  put_shrunk(o, t, j, r, uint32_t(a) < uint32_t(n), a, j < r ? V[t * r + j] : 0.f);
}
__global__ __launch_bounds__(256) void adapter_parts_kernel(const float* __restrict__ V, ShrunkOut out,
                                                            const int32_t* __restrict__ ids, int n, int T, int r) {
  parts_of(V, out, ids, n, T, r, int64_t(blockIdx.x) * 256 + threadIdx.x);
}

// ---------------------------------------------------------------------------
// Shrink: V[t][j] = now_a sum_c M_a[j][c] Z[t][c], M as [n][r][C].
// A workgroup of 8 waves takes 16 tokens and RF*16 ranks: 16 tokens, so that
// few of them make many workgroups.  The columns are dealt to the waves in
// 64-wide steps; each wave brings its own steps' rows, whole 128-byte lines,
// straight into its own ring of LDS stages and needs no barrier until the
// waves' tiles are added, in wave order.  (Fragments loaded straight into
// registers, 16 rows of 64 bytes an instruction, took 13 us for 2048 tokens x
// 4096 at rank 32; tiles of 64 tokens with the columns split over workgroups
// and a second kernel to add the shares 10 + 5; this 8.8.)
// Several adapters in a tile are dealt to blockIdx.z in turn.
// ---------------------------------------------------------------------------
constexpr int kShrinkWaves = 8;

template <int RF>
struct ShrinkRing {
  static constexpr int ROWS = (1 + RF) * 16, STAGE = ROWS * 128, LOADS = ROWS / 8;
  static constexpr int NS = RF == 1 ? 4 : 3;    // 16 KB or 18 KB a wave
  static constexpr int LDS = kShrinkWaves * NS * STAGE;
};

template <int DT, int RF>
__global__ __launch_bounds__(kShrinkWaves * 64) void adapter_shrink_kernel(
    const int32_t* __restrict__ ids, int n, const uint16_t* __restrict__ M, const float* __restrict__ now,
    const uint16_t* __restrict__ Z, int64_t ldz, int T, int C, int r, ShrunkOut out) {
  using Ring = ShrinkRing<RF>;
  extern __shared__ __align__(16) unsigned char smem[];
  const int lane = threadIdx.x & 63, li = lane & 15, lq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = blockIdx.x * 16, r0 = blockIdx.y * (RF * 16);
  const int t = t0 + li;
  const int id = t < T ? ids[t] : -1;
  const bool valid = uint32_t(id) < uint32_t(n);
  // every wave holds the same ids, so the loop and its barriers are uniform
  uint32_t todo = uint32_t(__ballot(valid)) & 0xFFFFu;
  if (blockIdx.z == 0 && wave < RF && !valid && t < T) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = r0 + wave * 16 + lq * 4 + e;
      if (j < ((r + 7) & ~7)) put_shrunk(out, t, j, r, false, 0, 0.f);
    }
  }
  unsigned char* ring = smem + wave * (Ring::NS * Ring::STAGE);
  f32x4 (*part)[RF][64] = reinterpret_cast<f32x4 (*)[RF][64]>(smem);
  const int steps = (C + 63) >> 6, rem = C - (steps - 1) * 64;
  const int mine_steps = wave < steps ? (steps - 1 - wave) / kShrinkWaves + 1 : 0;
  // loads j: rows 8 j + lane / 8 of the tokens (j = 0, 1), then of the ranks
  const uint32_t chunk = uint32_t((lane & 7) ^ ((lane >> 3) & 7));
  const __amdgpu_buffer_rsrc_t rz = make_rsrc(Z + int64_t(t0) * ldz);
  uint32_t off[Ring::LOADS];
#pragma unroll
  for (int j = 0; j < Ring::LOADS; ++j) {
    const int row = 8 * j + (lane >> 3);
    off[j] = (j < 2 ? uint32_t(min(row, T - 1 - t0)) * uint32_t(ldz)
                    : uint32_t(min(r0 + row - 16, r - 1)) * uint32_t(C)) * 2u + chunk * 16u;
  }
  for (uint32_t turn = 0; todo; ++turn) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
    const bool sel = id == a;
    todo &= ~uint32_t(__ballot(sel));
    if (turn % gridDim.z != blockIdx.z) continue;
    const __amdgpu_buffer_rsrc_t rm = make_rsrc(M + int64_t(a) * r * C, uint32_t(r) * uint32_t(C) * 2u);
    // this wave's i-th step into stage i % NS; past its last step that step
    // again, into a stage nothing reads any more; chunks past C reread the
    // step's first one
    auto issue = [&](int i) {
      const int s = wave + min(i, mine_steps - 1) * kShrinkWaves;
      unsigned char* st = ring + i % Ring::NS * Ring::STAGE;
      const uint32_t back = s == steps - 1 && int(chunk) * 8 >= rem ? chunk * 16u : 0u;
#pragma unroll
      for (int j = 0; j < Ring::LOADS; ++j) dma16(j < 2 ? rz : rm, off[j] - back, uint32_t(s) * 128u, st + j * 1024);
    };
    f32x4 acc[RF];
#pragma unroll
    for (int f = 0; f < RF; ++f) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (mine_steps > 0) {
#pragma unroll
      for (int i = 0; i < Ring::NS - 1; ++i) issue(i);
      for (int i = 0; i < mine_steps; ++i) {
        wait_lgkm0();                                    // the stage about to be refilled has been read
        asm volatile("" ::: "memory");
        issue(i + Ring::NS - 1);
        wait_vmcnt<(Ring::NS - 1) * Ring::LOADS>();      // step i has landed
        asm volatile("" ::: "memory");
        const unsigned char* st = ring + i % Ring::NS * Ring::STAGE;
        const bool tail = wave + i * kShrinkWaves == steps - 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = 4 * h + lq;
          u32x4 z = *reinterpret_cast<const u32x4*>(st + (li * 8 + (c ^ (li & 7))) * 16);
          u32x4 m[RF];
#pragma unroll
          for (int f = 0; f < RF; ++f)
            m[f] = *reinterpret_cast<const u32x4*>(st + ((16 + f * 16 + li) * 8 + (c ^ (li & 7))) * 16);
          if (tail && c * 8 >= rem) {
            z = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
            for (int f = 0; f < RF; ++f) m[f] = u32x4{0u, 0u, 0u, 0u};
          }
#pragma unroll
          for (int f = 0; f < RF; ++f) acc[f] = mfma32<DT>(m[f], z, acc[f]);
        }
      }
      wait_vmcnt<0>();
      wait_lgkm0();
    }
    __syncthreads();                                     // every wave is done with its ring
#pragma unroll
    for (int f = 0; f < RF; ++f) part[wave][f][lane] = acc[f];
    __syncthreads();
    if (wave < RF && sel && t < T) {
      f32x4 sum = part[0][wave][lane];
#pragma unroll
      for (int w = 1; w < kShrinkWaves; ++w) sum += part[w][wave][lane];
      const float sc = now ? now[a] : 1.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = r0 + wave * 16 + lq * 4 + e;
        if (j < ((r + 7) & ~7)) put_shrunk(out, t, j, r, true, a, sum[e] * sc);
      }
    }
    __syncthreads();                                     // part is read
  }
}

// Mt[a][j][c] = M[a][c][j] for M [n][C][r]: B's columns along the reduction of
// the backward pass's shrink, and (with the roles of C and r exchanged) A's
// ranks along that of its expand.  One launch prepares the backward pass: the
// first tiles transpose B, the next A, the rest take xa apart.
struct TransposeSide {
  const uint16_t* M;
  uint16_t* Mt;
  int rows, cols;       // of M
  int tiles;            // workgroups
};

struct PartsJob {
  const float* V;
  ShrunkOut out;
  const int32_t* ids;
  int n, T, r;
};

__global__ __launch_bounds__(256) void adapter_prepare_kernel(TransposeSide first, TransposeSide second,
                                                              PartsJob parts) {
  __shared__ uint16_t tile[64][64 + 2];
  const int third = int(blockIdx.x) - first.tiles - second.tiles;
  if (third >= 0) {     // the parts of xa (one adapter index does them)
    if (blockIdx.y == 0)
      parts_of(parts.V, parts.out, parts.ids, parts.n, parts.T, parts.r, int64_t(third) * 256 + threadIdx.x);
    return;
  }
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
// Expand: Y[t][c] = sum of the base's shares, in order, + (low-rank term); the
// base fp32 (Y itself or a workspace).  A wave takes 16 tokens x F*16 columns;
// `readable` columns of a row of the base may be read.
// ---------------------------------------------------------------------------
template <int DT, int OUT, int F>
__global__ __launch_bounds__(256) void adapter_expand_kernel(LowRank p, const float* base, int64_t ldb,
                                                             int64_t readable, int splits, void* Y, int64_t ldy) {
  const int lane = threadIdx.x & 63, li = lane & 15, lq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = blockIdx.x * 16, c0 = (blockIdx.y * 4 + wave) * (F * 16);
  if (c0 >= p.C) return;
  const int t = t0 + li, tr = min(t, p.T - 1);
  const int id = lowrank_ids<1>(p, t0);
  f32x4 acc[F];
#pragma unroll
  for (int f = 0; f < F; ++f) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (whole_pieces(c0, F * 16, p.C, ldb, readable)) {
#pragma unroll 4
    for (int z = 0; z < splits; ++z) {
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const int c = piece_start(c0 + 16 * f + 4 * lq, p.C);
        acc[f] += *reinterpret_cast<const f32x4*>(base + (int64_t(z) * p.T + tr) * ldb + c);
      }
    }
  } else {
    for (int z = 0; z < splits; ++z) {
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[f][e] += base[(int64_t(z) * p.T + tr) * ldb + min(c0 + 16 * f + 4 * lq + e, p.C - 1)];
    }
  }
  lowrank_add<DT, F, 1>(p, id, t0, c0, [&](int f, int) -> f32x4& { return acc[f]; });
  if (t >= p.T) return;
#pragma unroll
  for (int f = 0; f < F; ++f) {
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
// V's 4, is bound by issuing loads (2048 tokens, 4 adapters of rank 32 on 4096 x
// 4096, both gradients: 43 us so, 16 now).  Tokens of other adapters are
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
  // the waves' tiles into LDS; then each wave adds up, in wave order, and writes
  // every 8th fragment
  f32x4 (*part)[RF * CF][64] = reinterpret_cast<f32x4 (*)[RF * CF][64]>(smem);
  if (any) {
    __syncthreads();                      // every wave is done with its staged tile
#pragma unroll
    for (int i = 0; i < RF; ++i)
#pragma unroll
      for (int j = 0; j < CF; ++j) part[wave][i * CF + j][lane] = acc[i][j];
    __syncthreads();
  }
  float* out = z.out + int64_t(a) * r * C;
  for (int f = wave; f < RF * CF; f += kGradWaves) {
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    if (any) {
#pragma unroll
      for (int w = 0; w < kGradWaves; ++w) sum += part[w][f][lane];
    }
    const int i = f / CF, j = f - i * CF;
    const int c = c0 + j * 16 + li, q = r0 + i * 16 + lq * 4;
    if (c >= C) continue;
    if (rank_minor && (r & 3) == 0) {
      if (q < r) *reinterpret_cast<f32x4*>(out + int64_t(c) * r + q) = sum;
      continue;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (q + e < r) out[rank_minor ? int64_t(c) * r + q + e : int64_t(q + e) * C + c] = sum[e];
  }
}

// Up to this many tokens a wave computes one number of V: past it, a token's
// row would be read by too many waves.
constexpr int64_t kFewTokens = 16;

int64_t round8(int64_t r) { return (r + 7) / 8 * 8; }

// now_a M Z as `out` wants it (out.V is written in any case).
template <int DT>
hipError_t shrink(const int32_t* ids, int64_t n, const uint16_t* M, const float* now, const uint16_t* Z, int64_t ldz,
                  int64_t T, int64_t C, int64_t r, const ShrunkOut& out, hipStream_t s) {
  if (T <= kFewTokens) {
    hipLaunchKernelGGL((adapter_dots_kernel<DT>), dim3(unsigned((T * r + 3) / 4)), dim3(256), 0, s, ids, int(n), M,
                       now, Z, ldz, int(T), int(C), int(r), out.V);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    if (!out.P && !out.PT) return hipSuccess;
    ShrunkOut rest = out;
    rest.V = nullptr;
    hipLaunchKernelGGL(adapter_parts_kernel, dim3(unsigned((T * round8(r) + 255) / 256)), dim3(256), 0, s, out.V, rest,
                       ids, int(n), int(T), int(r));
    return hipGetLastError();
  }
  auto go = [&](auto kern, int rf, int lds) {
    if (hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(kern), lds); e != hipSuccess) return e;
    // two adapters of a tile at a time, where there can be two
    hipLaunchKernelGGL(kern, dim3(unsigned((T + 15) / 16), unsigned((r + rf * 16 - 1) / (rf * 16)), n > 1 ? 2u : 1u),
                       dim3(kShrinkWaves * 64), lds, s, ids, int(n), M, now, Z, ldz, int(T), int(C), int(r), out);
    return hipGetLastError();
  };
  return r <= 16 ? go(adapter_shrink_kernel<DT, 1>, 1, ShrinkRing<1>::LDS)
                 : go(adapter_shrink_kernel<DT, 2>, 2, ShrinkRing<2>::LDS);
}

template <int DT>
hipError_t expand(const LowRank& p, const float* base, int64_t ldb, int64_t readable, int64_t splits, void* Y,
                  int64_t ldy, int out_dtype, hipStream_t s) {
  auto go = [&](auto kern, int f) {
    hipLaunchKernelGGL(kern, dim3(unsigned((p.T + 15) / 16), unsigned((p.C + f * 64 - 1) / (f * 64))), dim3(256), 0, s,
                       p, base, ldb, readable, int(splits), Y, ldy);
    return hipGetLastError();
  };
  // 64 columns a wave where that still covers the chip, else 16
  const bool wide = (int64_t(p.T) + 15) / 16 * ((p.C + 255) / 256) >= 256;
  if (out_dtype == NM_F32)
    return wide ? go(adapter_expand_kernel<DT, NM_F32, 4>, 4) : go(adapter_expand_kernel<DT, NM_F32, 1>, 1);
  return wide ? go(adapter_expand_kernel<DT, DT, 4>, 4) : go(adapter_expand_kernel<DT, DT, 1>, 1);
}

template <int DT>
hipError_t gradients(GradArgs g, int64_t n, hipStream_t s) {
  auto go = [&](auto kern, auto rfc, auto cfc) {
    constexpr int RF = decltype(rfc)::value, CF = decltype(cfc)::value;
    constexpr int lds = std::max(kGradWaves * GradTile<CF>::BYTES, kGradWaves * RF * CF * 1024);
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

// How the shared product is computed: by the few-token family (T <= 16) or the
// all-LDS family (2:4 prefill), which add the low-rank term themselves; in
// shares; or by whatever nm_spmm chooses, in fp32.  The last two leave the term
// to the expand kernel.
enum class Route { kFew, kPrefill, kShares, kPlain };
Route route(const SpmmArgs& b) {
  if (spmm_decode_applies(b)) return Route::kFew;
  if (adapter_product_applies(b)) return Route::kShares;
  return spmm_lds_applies(b) ? Route::kPrefill : Route::kPlain;
}

// Parts of the workspaces, each on 256 bytes.
size_t padded(size_t bytes) { return (bytes + 255) / 256 * 256; }
size_t parts_bytes(int64_t T, int64_t r) { return padded(size_t(T) * 3 * round8(r) * 2); }

template <int DT>
hipError_t forward_dt(const AdapterArgs& a, hipStream_t s) {
  const int64_t T = a.base.T;
  const Route way = route(a.base);
  const bool few = way == Route::kFew;   // that family multiplies V itself
  char* ws = static_cast<char*>(a.workspace);
  uint16_t* P = few ? nullptr : reinterpret_cast<uint16_t*>(ws);
  const ShrunkOut out{a.scale, a.xa, P, nullptr, 0};
  hipError_t e = shrink<DT>(a.ids, a.n, a.A, nullptr, a.base.act, a.base.ldx, T, a.base.K, a.r, out, s);
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
  if (few || way == Route::kPrefill) {
    b.lowrank = &p;
    return few ? launch_spmm_decode(b, s) : launch_spmm_lds(b, s);
  }
  float* base = reinterpret_cast<float*>(ws + parts_bytes(T, a.r));
  int64_t ldb = a.base.R, readable = ldb, splits = 1;   // in Y's last row nothing follows column R
  if (way == Route::kShares) {
    splits = adapter_product_splits(b);
    ldb = readable = adapter_product_ld(b);
    e = launch_adapter_product(b, base, s);
  } else {
    if (a.base.out_dtype == NM_F32) {
      base = static_cast<float*>(a.base.Y);
      ldb = a.base.ldy;
    }
    b.Y = base;
    b.ldy = ldb;
    b.out_dtype = NM_F32;
    e = launch_spmm(b, s);
  }
  if (e != hipSuccess) return e;
  return expand<DT>(p, base, ldb, readable, splits, a.base.Y, a.base.ldy, a.base.out_dtype, s);
}

// The backward pass's workspace: u, its parts, u's and s xa's parts along the
// tokens, B and A transposed.
struct BwdParts {
  int64_t ldt;
  size_t u, p, ut, xt, bt, at, total;
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
  b.total = b.at + padded(size_t(n) * r * K * 2);
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
      const PartsJob xp{a.xa, ShrunkOut{a.scale, nullptr, nullptr, xt, int(w.ldt)}, a.ids, int(a.n), int(d.T), int(a.r)};
      const int64_t blocks = tb.tiles + ta.tiles + (d.T * round8(a.r) + 255) / 256;
      hipLaunchKernelGGL(adapter_prepare_kernel, dim3(unsigned(blocks), unsigned(a.n)), dim3(256), 0, s, tb, ta, xp);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    e = shrink<DT>(a.ids, a.n, bt, a.scale, d.G, d.ldg, d.T, d.R, a.r, ShrunkOut{nullptr, u, P, ut, int(w.ldt)}, s);
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
  const size_t y = size_t(base.T) * size_t(base.R) * 4;
  switch (route(base)) {
    case Route::kFew: return 0;
    case Route::kPrefill: return parts_bytes(base.T, r);
    case Route::kShares:
      return parts_bytes(base.T, r) + size_t(adapter_product_splits(base)) * size_t(base.T) * adapter_product_ld(base) * 4;
    default: return parts_bytes(base.T, r) + (base.out_dtype == NM_F32 ? 0 : y);
  }
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
