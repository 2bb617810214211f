// Training-side products of an N:M layer on gfx950.
//
// Source: COE-592 lecture 04-2, "M:N sparsity on NVIDIA tensor cores",
// section "The recipe", step 3 (retrain with the zeros held fixed, so the
// pattern survives), and the RNM-TD3 abstract of thelatestinai.com's
// "Structured Sparsity" cards (row-wise N:M kept throughout training).  With
// G = dL/dYt [T, R] (the forward output's layout):
//   dX[T, K]  = G W_nm                          (nm_spmm_dx, this file);
//   dW[R, S]  = sum_t G[t, r] act[t, k(r, s)]   (nm_spmm_dw), the gradient of
//               each stored survivor, in the packed layout.
// In dX the reduction runs over R, across the rows of W, so the N:M groups
// (which run along K) give the instruction nothing to skip: the product is
// dense on the MFMA and what the packed form saves is the weight bytes read.
//
// LDS transpose reads.  ds_read_b64_tr_b16 reads 4 halves per lane like a
// plain 64-bit read and then exchanges them within each group of 16 lanes:
// lane 16g + 4a + b receives element b of what lane 16g + 4j + a read, for
// j = 0..3 (measured on the MI355X with a probe of the instruction).  So
// when lane 16g + 4j + a points at row 8g + j (plus 4 for a second read),
// columns 4a..4a+3, of a tile stored reduction-major (rows = reduction),
// lane 16g + 4a + b gets rows 8g..8g+7 of column 4a + b: the 8 consecutive
// reduction elements of one column that a v_mfma_f32_16x16x32 operand lane
// (column 4a + b, quarter g) holds.  Tiles that arrive reduction-major (the
// decompressed W for dX, G and act for dW) feed the MFMA through two such
// reads per operand, without a transposing copy.
#include "nm_device.h"
#include "nm_group.h"
#include "nm_internal.h"
#include "nm_lowrank.h"

#include <algorithm>
#include <type_traits>

namespace nm {
namespace {

// In the place of the experts' rows: one weight for all tokens.
struct NoGroup {};
// dX: the tiles, and from one expert's values (index words) to the next.
// share > 0: workgroup y reduces over that many chunks of R and leaves fp32 sums
// part_stride bytes from those before it.  (16 experts of 4096 x 2048 in 2:4, 8192
// tokens: 196 to 215 us, 0.64 to 0.70 PFLOP/s of the dense product.  Nothing is full: the
// matrix cores are busy 32% of the time, LDS 49%, a third of that with bank conflicts; a
// wave issues 41% of its time, waits for its turn to issue 41%, for data or the barrier
// 18%.  The grid is of the most tiles there can be, and those that exist lie in the first
// XCDs' runs, 158 each in seven and 78 in the last, 2.5 rounds of their compute units:
// these have work 84% of the time.)
struct GroupDx {
  GroupRows rows;
  int64_t values_stride, idx_stride;
  int share;
  int64_t part_stride;
};
// dW: the experts' rows, from one's index words to the next, and its gradient (bytes).
// shares > 1: workgroup y sums over a share of its expert's tokens and leaves it
// part_stride bytes from the one before.  (The same experts and tokens: 173 to 180 us,
// 0.76 to 0.79 PFLOP/s dense, the matrix cores 35% busy, LDS 31%; a wave issues 35% of its
// time, waits for its turn 44%, for data or the barrier 21%.)
struct GroupDw {
  const int32_t* offsets;
  int64_t idx_stride, dw_stride;
  int shares;
  int64_t part_stride;
};

constexpr int pat_n(int P) { return P == 0 ? 2 : 1; }
constexpr int pat_m(int P) { return P == 2 ? 8 : 4; }

// ---------------------------------------------------------------------------
// dX = G W_nm, computed as dX^T tiles: D[k][t] = sum_r W[r][k] G[t][r].
//
// A workgroup (4 waves, 2 x 2) owns 128 k x 128 t; a wave 64 x 64 (4 x 4
// fragments).  R is walked in chunks of 64 rows, each staged in LDS:
//   * G's tile (128 tokens x 64 r, 16 KB), 4 16-byte pieces per thread,
//     loaded into registers two chunks ahead and written to a double-buffered
//     stage, slot (token, 16-byte chunk c) at token*8 + (c ^ (token & 7)); a
//     B operand lane (token i, quarter q) reads chunk 4h + q of sub-step h
//     (r 32h + 8q ..) with one 16-byte read;
//   * W's chunk (64 rows x 128 columns) is decompressed by the workgroup's
//     256 threads, each one row and 32 columns, from packed values and index
//     bits it loaded into registers two chunks earlier, into a dense
//     double-buffered tile [64 r][128 k] (rows padded to 288 bytes); the A
//     operands (k rows, r reduction) come out of it by transpose reads.
// The stages are filled from registers, not by direct global->LDS loads: the
// compiler cannot tell which LDS bytes a transpose read touches, so after a
// direct load it would hold every transpose read until that load landed.
// One barrier per chunk publishes the chunk's stage and tile (written in the
// previous step) and retires the ones the step then refills.  At 68 KB of
// LDS two workgroups share a compute unit, each covering the other's barrier
// and epilogue.
// ---------------------------------------------------------------------------
constexpr int kDxBK = 128, kDxBT = 128, kDxRC = 64;
constexpr int kDxGStage = kDxBT * kDxRC * 2;     // 16 KB
constexpr int kDxWRow = kDxBK * 2 + 32;          // 288 bytes: padded row of the W tile
constexpr int kDxWTile = kDxRC * kDxWRow;        // 18 KB
constexpr int kDxLds = 2 * kDxGStage + 2 * kDxWTile;

// One thread's packed share of a chunk: values of 32 columns of one row
// (2:4 16 values, 1:4 8, 1:8 4) and the two index words holding its bits.
struct DxPack {
  u32x4 v0, v1;
  uint32_t i0, i1;
};

template <int P>
__device__ inline void dx_load(DxPack& d, __amdgpu_buffer_rsrc_t rv, __amdgpu_buffer_rsrc_t ri, uint32_t voff,
                               uint32_t ioff0, uint32_t ioff1) {
  if constexpr (P == 0) {
    d.v0 = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rv, voff, 0, 0));
    // a dead share stays dead: kDeadOffset + 16 would wrap to offset 0, and row
    // 0's values with zero index bits expand (two halves OR'ed into one
    // position) into arbitrary bits, Inf and NaN among them
    const uint32_t voff1 = voff == kDeadOffset ? kDeadOffset : voff + 16u;
    d.v1 = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rv, voff1, 0, 0));
  } else if constexpr (P == 1) {
    d.v0 = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rv, voff, 0, 0));
  } else {
    const u32x2 t = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rv, voff, 0, 0));
    d.v0 = u32x4{t[0], t[1], 0u, 0u};
  }
  d.i0 = __builtin_amdgcn_raw_buffer_load_b32(ri, ioff0, 0, 0);
  d.i1 = __builtin_amdgcn_raw_buffer_load_b32(ri, ioff1, 0, 0);
}

// Quarter q (8 columns, 4 dwords) of a thread's row segment from its packed share;
// ishift is the position of the segment's first index bit in word i0.
template <int P, int q>
__device__ inline void dx_expand(const DxPack& d, uint32_t ishift, u32x4& o) {
  const uint64_t bits = (uint64_t(d.i1) << 32 | d.i0) >> ishift;
  if constexpr (P == 0) {  // 2 groups of 4, two values each
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      constexpr int g0 = 2 * q;
      const int g = g0 + e;
      const uint32_t v = g < 4 ? d.v0[g & 3] : d.v1[g & 3];
      const uint32_t p0 = uint32_t(bits >> (4 * g)) & 3u, p1 = uint32_t(bits >> (4 * g + 2)) & 3u;
      const uint64_t w = (uint64_t(v & 0xFFFFu) << (16 * p0)) | (uint64_t(v >> 16) << (16 * p1));
      o[2 * e] = uint32_t(w);
      o[2 * e + 1] = uint32_t(w >> 32);
    }
  } else if constexpr (P == 1) {  // 2 groups of 4, one value each
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int g = 2 * q + e;
      const uint32_t h = (d.v0[g >> 1] >> (16 * (g & 1))) & 0xFFFFu;
      const uint32_t p = uint32_t(bits >> (2 * g)) & 3u;
      const uint64_t w = uint64_t(h) << (16 * p);
      o[2 * e] = uint32_t(w);
      o[2 * e + 1] = uint32_t(w >> 32);
    }
  } else {  // a group of 8, one value
    const uint32_t h = (d.v0[q >> 1] >> (16 * (q & 1))) & 0xFFFFu;
    const uint32_t p = uint32_t(bits >> (3 * q)) & 7u;
    const uint32_t x = h << (16 * (p & 1));
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = (p >> 1) == uint32_t(e) ? x : 0u;
  }
}

template <int P, int DT, int OUT, class LR, class GR>
__global__ __launch_bounds__(256, 2) void spmm_dx_kernel(const uint16_t* __restrict__ values, uint32_t values_bytes,
                                                      const uint32_t* __restrict__ idx, uint32_t idx_bytes, int R,
                                                      int K, int idx_row_words, const uint16_t* __restrict__ G,
                                                      int T, int64_t ldg, void* __restrict__ dX, int64_t lddx,
                                                      int tilesK, int tilesT, int group, LR lowrank, GR experts) {
  constexpr int N = pat_n(P), M = pat_m(P);
  constexpr int B = P == 2 ? 3 : 2;  // index bits per survivor
  extern __shared__ __align__(16) unsigned char smem[];
  unsigned char* gbuf = smem;                          // [2][16 KB]
  unsigned char* wbuf = smem + 2 * kDxGStage;          // [2][64][288 B]

  int tk, tt;
  grouped_tile(xcd_tile(blockIdx.x, gridDim.x), tilesK, tilesT, group, tk, tt);
  const int K0 = tk * kDxBK;
  int T0 = tt * kDxBT;
  if constexpr (std::is_same_v<GR, GroupDx>) {   // the tile's expert, its tokens up to T
    GroupTile g;
    if (!experts.rows.tile(tt, T, kDxBT, g)) return;
    values += g.e * experts.values_stride;
    idx += g.e * experts.idx_stride;
    T0 = g.t0;
    T = g.t1;
  }
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wk = wave >> 1, wt = wave & 1;
  const int li = lane & 15, lq = lane >> 4;
  // the chunks this workgroup reduces over: all, or its share of them
  int first = 0, nchunks = (R + kDxRC - 1) / kDxRC;
  if constexpr (std::is_same_v<GR, GroupDx>) {
    if (experts.share > 0) {
      first = int(blockIdx.y) * experts.share;
      nchunks = min(nchunks, first + experts.share);
      dX = static_cast<unsigned char*>(dX) + int64_t(blockIdx.y) * experts.part_stride;
    }
  }
  const int64_t S = int64_t(K) * N / M;

  // G: descriptor over the tile's token rows (rows past T reread row T - 1;
  // their outputs are dropped).  R % 8 == 0, so a 16-byte piece of a row lies
  // wholly before R or wholly past it; pieces past R read zeros, which meet
  // the zero rows of W's tile past R.
  const int tlast = min(T0 + kDxBT, T) - 1;
  const __amdgpu_buffer_rsrc_t rg =
      make_rsrc(G + int64_t(T0) * ldg, uint32_t((int64_t(tlast - T0) * ldg + R) * 2));
  // this thread's pieces of a chunk: LDS slot (wave*NG + j)*64 + lane, holding
  // (token, 16-byte piece c) of the tile (a piece's slot is its own inverse)
  uint32_t goff[4];
  int gcol[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int slot = (wave * 4 + j) * 64 + lane;
    const int tok = slot >> 3;
    const int c = (slot & 7) ^ (tok & 7);
    const int t = min(T0 + tok, T - 1) - T0;
    goff[j] = uint32_t(t) * uint32_t(ldg) * 2u + uint32_t(c) * 16u;
    gcol[j] = c * 8;
  }
  auto load_g = [&](int chunk, u32x4 (&gr)[4], int j) {
    const int r0 = chunk * kDxRC;
    // a piece past R (or of a chunk past the last) reads zeros
    const bool live = (chunk < nchunks) & (r0 + gcol[j] < R);
    gr[j] = __builtin_bit_cast(
        u32x4, __builtin_amdgcn_raw_buffer_load_b128(rg, live_offset(live, goff[j] + uint32_t(r0) * 2u), 0, 0));
  };
  auto write_g = [&](int stage, const u32x4 (&gr)[4], int j) {
    *reinterpret_cast<u32x4*>(gbuf + stage * kDxGStage + ((wave * 4 + j) * 64 + lane) * 16) = gr[j];
  };

  // W: this thread decompresses 32 columns of a row of the chunk
  const int wr = tid >> 2, wc = tid & 3;
  const __amdgpu_buffer_rsrc_t rv = make_rsrc(values, values_bytes);
  const __amdgpu_buffer_rsrc_t ri = make_rsrc(idx, idx_bytes);
  const int kc = K0 + 32 * wc;                      // first column of the segment
  const int64_t s0 = int64_t(kc) * N / M;           // its first survivor in the row
  const int64_t bit0 = s0 * B;                      // its first index bit in the row
  const uint32_t ishift = uint32_t(bit0 & 31);
  // the word holding the first bit and the next one, clamped to the row (the
  // row's last word then holds every bit the segment needs)
  const int64_t w0 = bit0 >> 5, w1 = min(w0 + 1, int64_t(idx_row_words) - 1);
  auto pack_offsets = [&](int chunk, uint32_t& voff, uint32_t& ioff0, uint32_t& ioff1) {
    const int64_t row = int64_t(chunk) * kDxRC + wr;
    const bool live = (chunk < nchunks) & (row < R) & (kc < K);
    voff = live_offset(live, uint32_t((row * S + s0) * 2));
    ioff0 = live_offset(live, uint32_t((row * idx_row_words + w0) * 4));
    ioff1 = live_offset(live, uint32_t((row * idx_row_words + w1) * 4));
  };
  // 8 columns (quarter q) of the segment, 16 bytes of the tile's row
  auto decompress = [&](const DxPack& d, int buf, auto q_c) {
    constexpr int q = decltype(q_c)::value;
    u32x4 o;
    dx_expand<P, q>(d, ishift, o);
    *reinterpret_cast<u32x4*>(wbuf + buf * kDxWTile + wr * kDxWRow + wc * 64 + 16 * q) = o;
  };

  f32x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // A operand addresses in the W tile: lane L = 16g + 4j + a reads row
  // 8g + j (+4) of the sub-step, columns 4a.. of fragment kf
  const int tr_row = 8 * (lane >> 4) + ((lane >> 2) & 3), tr_col = 4 * (lane & 3);
  auto read_a = [&](int buf, int h, int kf) {
    const unsigned char* base =
        wbuf + buf * kDxWTile + (32 * h + tr_row) * kDxWRow + (wk * (kDxBK / 2) + kf * 16 + tr_col) * 2;
    const u32x2 lo = lds_read_tr(base), hi = lds_read_tr(base + 4 * kDxWRow);
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
  };
  auto read_b = [&](int slot, int h, int tf) {
    const int tok = wt * 64 + tf * 16 + li;
    const int c = 4 * h + lq;
    return *reinterpret_cast<const u32x4*>(gbuf + slot * kDxGStage + (tok * 8 + (c ^ (tok & 7))) * 16);
  };

  // ---- prologue: chunks 0 and 1 in registers, chunk 0 staged and
  // decompressed, chunk 2 in registers
  DxPack pk[2];
  u32x4 gs[2][4];
  auto load_pack = [&](int chunk, DxPack& d) {
    uint32_t vo, i0, i1;
    pack_offsets(chunk, vo, i0, i1);
    dx_load<P>(d, rv, ri, vo, i0, i1);
  };
  [[maybe_unused]] int ids = 0;
  if constexpr (std::is_same_v<LR, LowRank>) ids = lowrank_ids<4>(lowrank, T0 + wt * 64);
  using std::integral_constant;
#pragma unroll
  for (int j = 0; j < 4; ++j) load_g(first, gs[0], j);
  load_pack(first, pk[0]);
#pragma unroll
  for (int j = 0; j < 4; ++j) load_g(first + 1, gs[1], j);
  load_pack(first + 1, pk[1]);
  decompress(pk[0], 0, integral_constant<int, 0>{});
  decompress(pk[0], 0, integral_constant<int, 1>{});
  decompress(pk[0], 0, integral_constant<int, 2>{});
  decompress(pk[0], 0, integral_constant<int, 3>{});
#pragma unroll
  for (int j = 0; j < 4; ++j) write_g(0, gs[0], j);
#pragma unroll
  for (int j = 0; j < 4; ++j) load_g(first + 2, gs[0], j);
  load_pack(first + 2, pk[0]);

  // Step c (parity PAR = c & 1, a compile-time constant: the loop is unrolled
  // by two so the register sets alternate without copies): the barrier
  // publishes G stage PAR and W tile PAR, written in step c-1 (or the
  // prologue), and retires stage and tile PAR ^ 1, read in step c-1.  The step
  // multiplies chunk c, stages chunk c+1 from register sets (c+1) & 1 into
  // stage and tile PAR ^ 1 and loads chunk c+3 into those sets.  Past the
  // last chunk the loads read zeros (dead offsets), and so are staged.
  // Eight slots of four products, which scheduling barriers keep in order: in the
  // first four a quarter of the next chunk is decompressed behind the products and
  // the second half's fragments are read, in the last four G is staged and the
  // loads go out (one after the other, products, decompression and stage writes
  // took the sum of their times).
  auto step = [&](auto par_c, int c) {
    constexpr int PAR = decltype(par_c)::value;
    DxPack& nextp = pk[PAR ^ 1];
    u32x4 (&nextg)[4] = gs[PAR ^ 1];
    wait_lgkm0();
    barrier_no_fence();
    u32x4 a0[4], b0[4], a1[4], b1[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      b0[f] = read_b(PAR, 0, f);
      a0[f] = read_a(PAR, 0, f);
    }
    auto slot = [&](auto k_c) {
      constexpr int k = decltype(k_c)::value;
      a1[k] = read_a(PAR, 1, k);
      b1[k] = read_b(PAR, 1, k);
#pragma unroll
      for (int tf = 0; tf < 4; ++tf) acc[k][tf] = mfma32<DT>(a0[k], b0[tf], acc[k][tf]);
      decompress(nextp, PAR ^ 1, k_c);
      __builtin_amdgcn_sched_barrier(0);
    };
    slot(integral_constant<int, 0>{});
    slot(integral_constant<int, 1>{});
    slot(integral_constant<int, 2>{});
    slot(integral_constant<int, 3>{});
    load_pack(c + 3, nextp);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
      for (int tf = 0; tf < 4; ++tf) acc[k][tf] = mfma32<DT>(a1[k], b1[tf], acc[k][tf]);
      write_g(PAR ^ 1, nextg, k);
      load_g(c + 3, nextg, k);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // whole pairs in the loop and an odd last chunk after it: a pair cut short
  // inside the loop would give the back edge a path on which the other
  // register set holds the newest loads, and the compiler's waits before
  // every later write of a set would then drain both sets
  int c = first;
  for (; c + 1 < nchunks; c += 2) {
    step(std::integral_constant<int, 0>{}, c);
    step(std::integral_constant<int, 1>{}, c + 1);
  }
  if (c < nchunks) step(std::integral_constant<int, 0>{}, c);
  wait_vmcnt<0>();

  // ---- the low-rank term
  if constexpr (std::is_same_v<LR, LowRank>)
    lowrank_add<DT, 4, 4>(lowrank, ids, T0 + wt * 64, K0 + wk * (kDxBK / 2), [&](int f, int n) -> f32x4& { return acc[f][n]; });

  // ---- epilogue: lane (t = li, quarter q) holds rows 4q..4q+3 (k) of column t of
  // each fragment.  A fragment of 16 tokens at a time is gathered in the wave's own
  // part of LDS and leaves in runs of the wave's BK / 2 columns (from the lanes a
  // token's columns would go out in pieces of 32 or 64 bytes).
  constexpr int ELT = OUT == NM_F32 ? 4 : 2, RUN = kDxBK / 2 * ELT, PITCH = RUN + 16, LPR = RUN / 16;
  static_assert(4 * 16 * PITCH <= kDxLds, "the waves' gather areas");
  wait_lgkm0();
  barrier_no_fence();   // every wave is done with the stages
  unsigned char* mine = smem + wave * (16 * PITCH);
  const int kw = K0 + wk * (kDxBK / 2);
  const bool vec_ok = (lddx * ELT) % 16 == 0;
#pragma unroll
  for (int tf = 0; tf < 4; ++tf) {
#pragma unroll
    for (int kf = 0; kf < 4; ++kf) {
      const f32x4 v = acc[kf][tf];
      unsigned char* o = mine + li * PITCH + (kf * 16 + lq * 4) * ELT;
      if constexpr (OUT == NM_F32) *reinterpret_cast<f32x4*>(o) = v;
      else *reinterpret_cast<u32x2*>(o) = u32x2{pack_half2<DT>(v[0], v[1]), pack_half2<DT>(v[2], v[3])};
    }
    wait_lgkm0();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int it = 0; it < 16 * LPR / 64; ++it) {
      const int slot = it * 64 + lane, row = slot / LPR, c = slot % LPR;
      const int t = T0 + wt * 64 + tf * 16 + row, k = kw + c * (16 / ELT);
      if (t >= T || k >= K) continue;   // (K is a multiple of 32: a piece is in or out)
      const u32x4 v = *reinterpret_cast<const u32x4*>(mine + row * PITCH + c * 16);
      unsigned char* y = static_cast<unsigned char*>(dX) + (int64_t(t) * lddx + k) * ELT;
      if (vec_ok) {
        *reinterpret_cast<u32x4*>(y) = v;
      } else {
#pragma unroll
        for (int e = 0; e < 16 / ELT; ++e) {
          const uint32_t w = v[e * ELT / 4];
          if constexpr (ELT == 4) reinterpret_cast<uint32_t*>(y)[e] = w;
          else reinterpret_cast<uint16_t*>(y)[e] = uint16_t(w >> (16 * (e & 1)));
        }
      }
    }
    wait_lgkm0();   // read before the next fragment is gathered
    asm volatile("" ::: "memory");
  }
}

// ---------------------------------------------------------------------------
// dW[r, s] = sum_t G[t, r] act[t, k(r, s)], computed as dense dW^T tiles
// D[k][r] = sum_t act[t][k] G[t][r] of which each lane keeps the stored
// entries.  A workgroup (4 waves, 2 x 2) owns 256 k x 128 r; a wave 128 k x
// 64 r (8 x 4 fragments), so one LDS byte feeds 43 MACs on average against
// 32 at 64 x 64.  T is walked in chunks of 32 tokens (one MFMA K step): act's
// [32 t][256 k] and G's [32 t][128 r] tiles are loaded into registers two
// chunks ahead (6 16-byte pieces per thread) and written to a double-buffered
// stage after the previous chunk's MFMAs; both operands come out by transpose
// reads (an operand lane needs 8 consecutive tokens of one column).  Staging
// from registers rather than by direct global->LDS loads keeps the compiler
// from holding each transpose read until every direct load in flight has
// landed.  Token row t of a tile starts at byte P t + 128 (((t >> 3) & 1) + (t
// >> 4)), P = 544 (act, 512-byte rows) or 288 (G, 256-byte rows): the 8-byte
// transpose reads of 32 lanes (rows 8g + j, g = 0, 1, j = 0..3) fall in
// distinct banks (64 banks of 4 bytes), the lanes writing one row write its
// bytes contiguously, and every fragment's address is a base register plus
// a constant.  At 2 x 27 KB of LDS two workgroups share a compute unit.
// A result lane (column r, quarter q) holds rows 4q..4q+3 of D, four
// consecutive columns k of W's row r: a whole group of four, or half of one
// of eight, whose stored positions it reads from the index bits and whose
// survivors it writes to the packed gradient.
// ---------------------------------------------------------------------------
constexpr int kDwBK = 256, kDwBR = 128, kDwTC = 32;
constexpr int kDwFK = 8, kDwFR = 4;                    // fragments per wave along k and r

__host__ __device__ constexpr int dw_row(int t, int pitch) {
  return t * pitch + (((t >> 3) & 1) + (t >> 4)) * 128;
}
constexpr int kDwActTile = dw_row(kDwTC - 1, 544) + 512;   // 17632 bytes
constexpr int kDwGTile = dw_row(kDwTC - 1, 288) + 256;     // 9440 bytes
constexpr int kDwStage = kDwActTile + kDwGTile;
constexpr int kDwLds = 2 * kDwStage;
static_assert(kDwActTile % 16 == 0 && kDwGTile % 16 == 0, "16-byte aligned tiles");

template <int P, int DT, int OUT, class GR>
__global__ __launch_bounds__(256, 2) void spmm_dw_kernel(const uint32_t* __restrict__ idx, uint32_t idx_bytes, int R,
                                                      int K, int idx_row_words, const uint16_t* __restrict__ G,
                                                      int T, int64_t ldg, const uint16_t* __restrict__ act,
                                                      int64_t ldx, void* __restrict__ dW, int tilesK, int tilesR,
                                                      int group, GR experts) {
  constexpr int N = pat_n(P), M = pat_m(P);
  constexpr int B = P == 2 ? 3 : 2;
  extern __shared__ __align__(16) unsigned char smem[];

  int block = blockIdx.x, blocks = gridDim.x;
  if constexpr (std::is_same_v<GR, GroupDw>) {
    // the expert's tokens, index words and gradient; its tiles are dealt to all
    // the XCDs, so that experts of many tokens do not fall to one of them
    blocks = tilesK * tilesR;
    const int e = block / blocks;
    block -= e * blocks;
    int lo, hi;
    group_range(experts.offsets, e, T, lo, hi);
    if (experts.shares > 1) {
      const int per = ((hi - lo + kDwTC - 1) / kDwTC + experts.shares - 1) / experts.shares * kDwTC;
      lo = min(lo + int(blockIdx.y) * per, hi);   // shares <= 16 and T <= 2^24: no overflow
      hi = min(lo + per, hi);
      dW = static_cast<unsigned char*>(dW) + int64_t(blockIdx.y) * experts.part_stride;
    }
    act += int64_t(lo) * ldx;
    G += int64_t(lo) * ldg;
    T = hi - lo;
    idx += e * experts.idx_stride;
    dW = static_cast<unsigned char*>(dW) + e * experts.dw_stride;
  }
  int tk, tr;
  grouped_tile(xcd_tile(block, blocks), tilesK, tilesR, group, tk, tr);
  const int K0 = tk * kDwBK, R0 = tr * kDwBR;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wk = wave >> 1, wr = wave & 1;
  const int li = lane & 15, lq = lane >> 4;
  const int nchunks = (T + kDwTC - 1) / kDwTC;
  const int64_t S = int64_t(K) * N / M;

  // A thread's pieces of a chunk: act rows (tid / 32) + 8 j, piece tid % 32
  // (j = 0..3), and G rows (tid / 16) + 16 j, piece tid % 16 (j = 0, 1).
  // Tokens past T read zeros, so they add nothing; columns past K or R are
  // whatever the descriptor allows and only reach outputs that are dropped
  // (with T == 0 nothing is read: the descriptors cover no bytes).
  const __amdgpu_buffer_rsrc_t ra =
      make_rsrc(act + K0, T > 0 ? uint32_t(((int64_t(T) - 1) * ldx + (K - K0)) * 2) : 0u);
  const __amdgpu_buffer_rsrc_t rg =
      make_rsrc(G + R0, T > 0 ? uint32_t(((int64_t(T) - 1) * ldg + (R - R0)) * 2) : 0u);
  int arow[4], grow[2];
  uint32_t aoff[4], goff[2], aloff[4], gloff[2];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    arow[j] = (tid >> 5) + 8 * j;
    aoff[j] = uint32_t(arow[j]) * uint32_t(ldx) * 2u + uint32_t(tid & 31) * 16u;
    aloff[j] = uint32_t(dw_row(arow[j], 544) + (tid & 31) * 16);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    grow[j] = (tid >> 4) + 16 * j;
    goff[j] = uint32_t(grow[j]) * uint32_t(ldg) * 2u + uint32_t(tid & 15) * 16u;
    gloff[j] = uint32_t(kDwActTile + dw_row(grow[j], 288) + (tid & 15) * 16);
  }
  // piece j of a chunk: 0 .. 3 act, 4 and 5 G
  auto load_piece = [&](int chunk, u32x4 (&v)[6], int j) {
    const int t0 = chunk * kDwTC;
    const bool is_act = j < 4;
    const int row = is_act ? arow[j & 3] : grow[j & 1];
    const bool live = t0 + row < T;      // false for every chunk past the last
    const uint32_t o = is_act ? aoff[j & 3] + uint32_t(t0) * uint32_t(ldx) * 2u : goff[j & 1] + uint32_t(t0) * uint32_t(ldg) * 2u;
    v[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(is_act ? ra : rg, live_offset(live, o), 0, 0));
  };
  auto load_chunk = [&](int chunk, u32x4 (&v)[6]) {
#pragma unroll
    for (int j = 0; j < 6; ++j) load_piece(chunk, v, j);
  };
  auto write_piece = [&](int stage, const u32x4 (&v)[6], int j) {
    unsigned char* st = smem + stage * kDwStage;
    *reinterpret_cast<u32x4*>(st + (j < 4 ? aloff[j & 3] : gloff[j & 1])) = v[j];
  };
  auto write_chunk = [&](int stage, const u32x4 (&v)[6]) {
#pragma unroll
    for (int j = 0; j < 6; ++j) write_piece(stage, v, j);
  };

  // transpose reads: lane L = 16g + 4j + a reads token rows 8g + j and
  // 8g + j + 4, columns 4a.. of a 16-column fragment
  const int tr_row = 8 * (lane >> 4) + ((lane >> 2) & 3), tr_a = lane & 3;
  const int a_lo = dw_row(tr_row, 544) + 8 * tr_a, a_hi = dw_row(tr_row + 4, 544) + 8 * tr_a;
  const int g_lo = kDwActTile + dw_row(tr_row, 288) + 8 * tr_a, g_hi = kDwActTile + dw_row(tr_row + 4, 288) + 8 * tr_a;
  auto read_tr = [&](const unsigned char* st, int lo, int hi, int col0) {
    const u32x2 l = lds_read_tr(st + lo + col0 * 2);
    const u32x2 h = lds_read_tr(st + hi + col0 * 2);
    return u32x4{l[0], l[1], h[0], h[1]};
  };

  f32x4 acc[kDwFK][kDwFR];
#pragma unroll
  for (int i = 0; i < kDwFK; ++i)
#pragma unroll
    for (int j = 0; j < kDwFR; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // chunk 0 staged, chunks 1 and 2 in registers; step c (parity PAR, the loop
  // unrolled by two): the barrier publishes stage PAR and retires stage
  // PAR ^ 1; the step multiplies chunk c, stages chunk c+1 from register set
  // PAR ^ 1 and loads chunk c+3 into it (past the last chunk, zeros)
  u32x4 vs[2][6];
  load_chunk(0, vs[0]);
  load_chunk(1, vs[1]);
  write_chunk(0, vs[0]);
  load_chunk(2, vs[0]);
  auto step = [&](auto par_c, int c) {
    constexpr int PAR = decltype(par_c)::value;
    u32x4 (&nextv)[6] = vs[PAR ^ 1];
    wait_lgkm0();
    barrier_no_fence();
    const unsigned char* st = smem + PAR * kDwStage;
    // Four slots of eight products, which scheduling barriers keep in order: the next
    // slot's operand is read, and the next chunk staged and the one after its loads
    // issued, behind the products (past the last chunk, zeros that nothing reads).
    u32x4 a[kDwFK], b[2];
    b[0] = read_tr(st, g_lo, g_hi, wr * 64);
#pragma unroll
    for (int kf = 0; kf < kDwFK; ++kf) a[kf] = read_tr(st, a_lo, a_hi, wk * 128 + kf * 16);
#pragma unroll
    for (int rf = 0; rf < kDwFR; ++rf) {
      if (rf + 1 < kDwFR) b[(rf + 1) & 1] = read_tr(st, g_lo, g_hi, wr * 64 + (rf + 1) * 16);
#pragma unroll
      for (int kf = 0; kf < kDwFK; ++kf) acc[kf][rf] = mfma32<DT>(a[kf], b[rf & 1], acc[kf][rf]);
#pragma unroll
      for (int j = rf; j < 6; j += 4) {
        write_piece(PAR ^ 1, nextv, j);
        load_piece(c + 3, nextv, j);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // whole pairs in the loop and an odd last chunk after it: a pair cut short
  // inside the loop would give the back edge a path on which the other
  // register set holds the newest loads, and the compiler's waits before
  // every later write of a set would then drain both sets
  int c = 0;
  for (; c + 1 < nchunks; c += 2) {
    step(std::integral_constant<int, 0>{}, c);
    step(std::integral_constant<int, 1>{}, c + 1);
  }
  if (c < nchunks) step(std::integral_constant<int, 0>{}, c);
  wait_vmcnt<0>();

  // ---- epilogue: lane (r = li of the fragment, quarter q) holds D rows
  // 4q..4q+3, columns k..k+3 of W's row r.  The wave's 128 columns of a row are VPR
  // stored values and up to four index words, which every quarter loads; a fragment
  // of 16 rows at a time is gathered in the wave's own part of LDS and leaves in
  // whole rows (written from the lanes, a row's 128 or 256 bytes went out in pieces
  // of 4 or 8, its index words came in two a fragment: 16 experts of 4096 x 2048,
  // 8192 tokens, 232 us).
  constexpr int VPR = 128 * N / M, ELT = OUT == NM_F32 ? 4 : 2;
  constexpr int ROW = VPR * ELT, PITCH = ROW + 16;
  constexpr int PIECE = P == 2 && ELT == 2 ? 8 : 16;   // bytes a store: whole 32 columns' worth
  constexpr int IW = P == 0 ? 4 : 2;                   // index words of 128 columns
  static_assert(4 * 16 * PITCH <= kDwLds, "the waves' gather areas");
  wait_lgkm0();
  barrier_no_fence();   // every wave is done with the stages
  unsigned char* mine = smem + wave * (16 * PITCH);
  const int kw = K0 + wk * 128;                        // the wave's first column
  const int wbit = kw / M * N * B, w0 = wbit >> 5;     // (1:8: at bit 0 or 16 of a word)
  const __amdgpu_buffer_rsrc_t ri = make_rsrc(idx, idx_bytes);
  uint32_t iw[kDwFR][IW];
#pragma unroll
  for (int rf = 0; rf < kDwFR; ++rf) {
    const int r = R0 + wr * 64 + rf * 16 + li;
#pragma unroll
    for (int e = 0; e < IW; ++e)
      iw[rf][e] = __builtin_amdgcn_raw_buffer_load_b32(
          ri, live_offset((r < R) & (w0 + e < idx_row_words), (uint32_t(r) * uint32_t(idx_row_words) + uint32_t(w0 + e)) * 4u),
          0, 0);
  }
  const int valid = min(128, K - kw) * N / M;          // stored values of the row inside W (none: 0 or less)
#pragma unroll
  for (int rf = 0; rf < kDwFR; ++rf) {
#pragma unroll
    for (int kf = 0; kf < kDwFK; ++kf) {
      const f32x4 v = acc[kf][rf];
      auto pick = [&](uint32_t p) {   // D value at in-lane column p (0..3)
        return p == 0 ? v[0] : p == 1 ? v[1] : p == 2 ? v[2] : v[3];
      };
      if constexpr (P == 0) {
        const uint32_t bits = iw[rf][kf >> 1] >> (16 * (kf & 1) + 4 * lq);
        const float x0 = pick(bits & 3u), x1 = pick((bits >> 2) & 3u);
        unsigned char* o = mine + li * PITCH + (kf * 4 + lq) * 2 * ELT;
        if constexpr (OUT == NM_F32) *reinterpret_cast<f32x2_t*>(o) = f32x2_t{x0, x1};
        else *reinterpret_cast<uint32_t*>(o) = pack_half2<DT>(x0, x1);
      } else {
        // 1:4: a group a lane; 1:8: a group two lanes, of which the one whose half
        // holds the survivor writes it
        const int g = P == 1 ? kf * 4 + lq : kf * 2 + (lq >> 1);
        uint32_t pos;
        if constexpr (P == 1) {
          pos = (iw[rf][kf >> 2] >> (8 * (kf & 3) + 2 * lq)) & 3u;
        } else {
          const uint64_t both = uint64_t(iw[rf][0]) | uint64_t(iw[rf][1]) << 32;
          pos = uint32_t(both >> ((wbit & 31) + 3 * g)) & 7u;
        }
        if (P == 1 || int(pos >> 2) == (lq & 1)) {
          const float x = pick(pos & 3u);
          unsigned char* o = mine + li * PITCH + g * ELT;
          if constexpr (OUT == NM_F32) *reinterpret_cast<float*>(o) = x;
          else *reinterpret_cast<uint16_t*>(o) = uint16_t(pack_half2<DT>(x, 0.f));
        }
      }
    }
    wait_lgkm0();
    asm volatile("" ::: "memory");
    constexpr int LPR = ROW / PIECE;   // lanes a row
    constexpr int PASSES = (16 * LPR + 63) / 64;
#pragma unroll
    for (int it = 0; it < PASSES; ++it) {
      const int slot = it * 64 + lane, row = slot / LPR, c = slot % LPR;
      const int r = R0 + wr * 64 + rf * 16 + row;
      if (r >= R || (c + 1) * (PIECE / ELT) > valid) continue;
      unsigned char* o = static_cast<unsigned char*>(dW) + (int64_t(r) * S + kw / M * N) * ELT + c * PIECE;
      if constexpr (PIECE == 16)
        *reinterpret_cast<u32x4*>(o) = *reinterpret_cast<const u32x4*>(mine + row * PITCH + c * 16);
      else
        *reinterpret_cast<u32x2*>(o) = *reinterpret_cast<const u32x2*>(mine + row * PITCH + c * 8);
    }
    wait_lgkm0();   // read before the next fragment is gathered
    asm volatile("" ::: "memory");
  }
}

// Group size for grouped_tile.  An XCD's run of about tiles / 8 tiles covers
// some bands of the grouped operand (at least min(group, run), more once the
// run spans several groups) and ceil(run / group) bands of the other, up to
// their counts; with band bytes in proportion band_a : band_b, the power of two
// with the fewest bytes is taken, so the XCD's L2 serves the rest.
int pick_group(int64_t tiles_a, int64_t tiles_b, double band_a, double band_b) {
  const int64_t run = (tiles_a * tiles_b + 7) / 8;
  int best = 1;
  double best_bytes = 0.0;
  for (int64_t g = 1; g <= tiles_a; g *= 2) {
    const int64_t na = std::min(tiles_a, std::max(std::min(g, run), (run + tiles_b - 1) / tiles_b));
    const int64_t nb = std::min(tiles_b, (run + g - 1) / g);
    const double bytes = double(na) * band_a + double(nb) * band_b;
    if (g == 1 || bytes < best_bytes) best = int(g), best_bytes = bytes;
  }
  return best;
}

template <int P, int DT, int OUT>
hipError_t launch_dw_cfg(const TrainArgs& a, hipStream_t s) {
  const int64_t tilesK = (a.K + kDwBK - 1) / kDwBK, tilesR = (a.R + kDwBR - 1) / kDwBR;
  if (tilesK * tilesR > 0x7FFFFFFF) return hipErrorInvalidValue;
  auto launch = [&](auto experts, int64_t grid) {
    unsigned shares = 1;
    if constexpr (std::is_same_v<decltype(experts), GroupDw>) shares = unsigned(experts.shares);
    auto kern = spmm_dw_kernel<P, DT, OUT, decltype(experts)>;
    if (hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(kern), kDwLds); e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3(unsigned(grid), shares), dim3(256), kDwLds, s, a.idx, uint32_t(a.idx_bytes), int(a.R),
                       int(a.K), int(a.idx_row_words), a.G, int(a.T), a.ldg, a.act, a.ldx, a.out, int(tilesK),
                       int(tilesR), pick_group(tilesK, tilesR, 2.0, 1.0), experts);
    return hipGetLastError();
  };
  if (!a.offsets) return launch(NoGroup{}, tilesK * tilesR);
  const int64_t grid = tilesK * tilesR * a.experts;
  if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
  GroupDw g{a.offsets, a.R * a.idx_row_words, a.R * (a.K / a.m * a.n) * (OUT == NM_F32 ? 4 : 2), 1, 0};
  if constexpr (OUT == NM_F32) {
    if (a.shares > 1) {
      g.shares = a.shares;
      g.part_stride = a.experts * g.dw_stride;
    }
  }
  return launch(g, grid);
}

template <int P, int DT>
hipError_t launch_dw_out(const TrainArgs& a, hipStream_t s) {
  const int64_t S = a.K / a.m * a.n;
  const int n = a.offsets ? spmm_dw_shares(a.R, a.K, a.T, a.experts) : 1;
  if (n > 1) {
    // partial sums, joined by a second launch
    TrainArgs part = a;
    part.out = a.table;
    part.shares = n;
    if (hipError_t e = launch_dw_cfg<P, DT, NM_F32>(part, s); e != hipSuccess) return e;
    return launch_group_join(static_cast<const float*>(a.table), n, a.experts * a.R, S, S, nullptr, 0, a.out, S,
                             a.out_dtype, s);
  }
  return a.out_dtype == NM_F32 ? launch_dw_cfg<P, DT, NM_F32>(a, s) : launch_dw_cfg<P, DT, DT>(a, s);
}

template <int P>
hipError_t launch_dw_dt(const TrainArgs& a, hipStream_t s) {
  return a.dtype == NM_F16 ? launch_dw_out<P, NM_F16>(a, s) : launch_dw_out<P, NM_BF16>(a, s);
}

template <int P, int DT, int OUT, class LR, class GR>
hipError_t launch_dx_cfg(const TrainArgs& a, const LR& lowrank, const GR& experts, hipStream_t s) {
  const int64_t tilesK = (a.K + kDxBK - 1) / kDxBK;
  const int64_t tilesT = a.offsets ? group_max_tiles(a.T, a.experts, kDxBT) : (a.T + kDxBT - 1) / kDxBT;
  if (tilesK * tilesT > 0x7FFFFFFF) return hipErrorInvalidValue;
  unsigned shares = 1;
  if constexpr (std::is_same_v<GR, GroupDx>)
    if (experts.share > 0) shares = unsigned(((a.R + kDxRC - 1) / kDxRC + experts.share - 1) / experts.share);
  auto kern = spmm_dx_kernel<P, DT, OUT, LR, GR>;
  if (hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(kern), kDxLds); e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3(unsigned(tilesK * tilesT), shares), dim3(256), kDxLds, s, a.values,
                     uint32_t(a.values_bytes), a.idx, uint32_t(a.idx_bytes), int(a.R), int(a.K),
                     int(a.idx_row_words), a.G, int(a.T), a.ldg, a.out, a.ldo, int(tilesK), int(tilesT),
                     // every column tile of an expert's tokens together: its weight is shared by few token
                     // tiles only (16 experts of 4096 x 2048, 8192 tokens: 237 us with a single weight's order)
                     a.offsets ? int(tilesK) : pick_group(tilesK, tilesT, double(pat_n(P)) / pat_m(P), 1.0), lowrank,
                     experts);
  return hipGetLastError();
}

template <int P, int DT>
hipError_t launch_dx_out(const TrainArgs& a, hipStream_t s) {
  const bool f32 = a.out_dtype == NM_F32;
  if (a.lowrank)
    return f32 ? launch_dx_cfg<P, DT, NM_F32>(a, *a.lowrank, NoGroup{}, s)
               : launch_dx_cfg<P, DT, DT>(a, *a.lowrank, NoGroup{}, s);
  if (a.offsets) {
    const int64_t tiles = spmm_dx_max_tiles(a.T, a.experts);
    GroupDx g{{}, a.R * (a.K / a.m * a.n), a.R * a.idx_row_words, 0, 0};
    if (hipError_t e = group_rows(a.offsets, a.experts, a.T, kDxBT, tiles, a.table, s, g.rows); e != hipSuccess) return e;
    const Shares sh = spmm_dx_shares(a.R, a.K, a.T, a.experts);
    if (sh.n > 1) {
      // partial sums behind the table, joined by a second launch
      TrainArgs part = a;
      part.out = static_cast<unsigned char*>(a.table) + group_rows_bytes(a.experts, tiles);
      part.ldo = a.K;
      g.share = sh.size;
      g.part_stride = a.T * a.K * 4;
      if (hipError_t e = launch_dx_cfg<P, DT, NM_F32>(part, NoLowRank{}, g, s); e != hipSuccess) return e;
      return launch_group_join(static_cast<const float*>(part.out), sh.n, a.T, a.K, a.K, a.offsets, int(a.experts), a.out,
                               a.ldo, a.out_dtype, s);
    }
    return f32 ? launch_dx_cfg<P, DT, NM_F32>(a, NoLowRank{}, g, s) : launch_dx_cfg<P, DT, DT>(a, NoLowRank{}, g, s);
  }
  return f32 ? launch_dx_cfg<P, DT, NM_F32>(a, NoLowRank{}, NoGroup{}, s)
             : launch_dx_cfg<P, DT, DT>(a, NoLowRank{}, NoGroup{}, s);
}

template <int P>
hipError_t launch_dx_dt(const TrainArgs& a, hipStream_t s) {
  return a.dtype == NM_F16 ? launch_dx_out<P, NM_F16>(a, s) : launch_dx_out<P, NM_BF16>(a, s);
}

}  // namespace

int64_t spmm_dx_max_tiles(int64_t T, int64_t E) { return group_max_tiles(T, E, kDxBT); }

Shares spmm_dx_shares(int64_t R, int64_t K, int64_t T, int64_t E) {
  return group_shares((K + kDxBK - 1) / kDxBK * spmm_dx_max_tiles(T, E), (R + kDxRC - 1) / kDxRC);
}

// dW's reduction is over an expert's tokens, of which the host knows the mean.
int spmm_dw_shares(int64_t R, int64_t K, int64_t T, int64_t E) {
  const int64_t tiles = (K + kDwBK - 1) / kDwBK * ((R + kDwBR - 1) / kDwBR) * E;
  return group_shares(tiles, T / std::max<int64_t>(1, std::min(T, E)) / kDwTC).n;
}

hipError_t launch_spmm_dw(const TrainArgs& a, hipStream_t s) {
  if (a.n == 2 && a.m == 4) return launch_dw_dt<0>(a, s);
  if (a.n == 1 && a.m == 4) return launch_dw_dt<1>(a, s);
  if (a.n == 1 && a.m == 8) return launch_dw_dt<2>(a, s);
  return hipErrorInvalidValue;
}

hipError_t launch_spmm_dx(const TrainArgs& a, hipStream_t s) {
  if (a.n == 2 && a.m == 4) return launch_dx_dt<0>(a, s);
  if (a.n == 1 && a.m == 4) return launch_dx_dt<1>(a, s);
  if (a.n == 1 && a.m == 8) return launch_dx_dt<2>(a, s);
  return hipErrorInvalidValue;
}

}  // namespace nm
