// Dense product of two 16-bit matrices stored along the reduction,
//   D[m][n] = sum_k P[m][k] Q[n][k],
// one BM x BN tile a workgroup, on v_mfma_f32_16x16x32, the tile handed to an
// epilogue in registers.
//
// Both operands go straight from memory into LDS (16 bytes a lane) through a
// ring of NS stages of 64 k each: slot (row, 16-byte chunk c) sits at row*8 +
// (c ^ (row & 7)), so the fragment reads of 8 consecutive rows hit distinct
// banks.  One barrier a step publishes the step's stage (each wave has waited
// for its own loads) and retires the one read before it, which the step's
// loads then refill.  Waves are WM x WN, each owning (BM / WM) x (BN / WN).
//
// Rows past M or N reread the last row (the epilogue drops them).  K is a
// multiple of 8; when it is no multiple of 64 the last step's chunks past K
// reread the step's first chunk and enter the product as zeros on both sides.
#pragma once

#include "nm_device.h"

namespace nm {

template <int BM_, int BN_, int WM_, int WN_, int NS_>
struct GemmTile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_;
  static constexpr int THREADS = WM * WN * 64;
  static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
  static constexpr int STAGE = (BM + BN) * 128;
  static constexpr int LDS = NS * STAGE;
  // direct loads a wave issues per step (a Q tile with fewer slots than
  // threads is loaded by several waves alike, so every wave counts the same)
  static constexpr int LP = BM * 8 / THREADS;
  static constexpr int LQ = BN * 8 >= THREADS ? BN * 8 / THREADS : 1;
  static constexpr int L = LP + LQ;
  static_assert(LP * THREADS == BM * 8 && (BN * 8) % 64 == 0 && LDS <= 160 * 1024, "whole loads");
};

// Tile (tm, tn); epi(acc) gets acc[FM][FN], lane (i, q) of fragment (fm, fn)
// holding rows m = tm*BM + wave_m*FM*16 + fm*16 + 4q .. +3 of column
// n = tn*BN + wave_n*FN*16 + fn*16 + i.  On entry to epi no load is in flight
// and every wave has passed a barrier, so smem is free.
template <int DT, class C, class Epi>
__device__ inline void gemm_nt(const uint16_t* P, int64_t ldp, int M, const uint16_t* Q, int64_t ldq, int N, int K,
                               int tm, int tn, unsigned char* smem, Epi&& epi) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const int wm = wave / C::WN, wn = wave % C::WN;
  const int m0 = tm * C::BM, n0 = tn * C::BN;
  const int steps = (K + 63) >> 6;
  const int rem = K - (steps - 1) * 64;   // valid k of the last step

  const __amdgpu_buffer_rsrc_t rp = make_rsrc(P + int64_t(m0) * ldp);
  const __amdgpu_buffer_rsrc_t rq = make_rsrc(Q + int64_t(n0) * ldq);
  uint32_t po[C::LP], qo[C::LQ];
  int qslot[C::LQ];
#pragma unroll
  for (int j = 0; j < C::LP; ++j) {
    const int slot = (wave * C::LP + j) * 64 + lane, row = slot >> 3, c = (slot & 7) ^ (row & 7);
    po[j] = uint32_t(min(row, M - 1 - m0)) * uint32_t(ldp) * 2u + uint32_t(c) * 16u;
  }
#pragma unroll
  for (int j = 0; j < C::LQ; ++j) {
    qslot[j] = ((wave * C::LQ + j) * 64) % (C::BN * 8);
    const int slot = qslot[j] + lane, row = slot >> 3, c = (slot & 7) ^ (row & 7);
    qo[j] = uint32_t(min(row, N - 1 - n0)) * uint32_t(ldq) * 2u + uint32_t(c) * 16u;
  }
  // chunk this lane loads: the same for every load (its slots are 64 apart)
  const uint32_t chunk = uint32_t((lane & 7) ^ ((lane >> 3) & 7));
  auto issue = [&](int s, int buf) {
    s = min(s, steps - 1);   // past the end: again the last step, into a stage nothing reads any more
    unsigned char* st = smem + buf * C::STAGE;
    const uint32_t back = s == steps - 1 && int(chunk) * 8 >= rem ? chunk * 16u : 0u;
#pragma unroll
    for (int j = 0; j < C::LP; ++j) dma16(rp, po[j] - back, uint32_t(s) * 128u, st + (wave * C::LP + j) * 1024);
#pragma unroll
    for (int j = 0; j < C::LQ; ++j)
      dma16(rq, qo[j] - back, uint32_t(s) * 128u, st + C::BM * 128 + qslot[j] * 16);
  };

  f32x4 acc[C::FM][C::FN];
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int prow = wm * C::FM * 16 + li, qrow = wn * C::FN * 16 + li;
  auto read = [&](const unsigned char* base, int row, int c) {
    return *reinterpret_cast<const u32x4*>(base + (row * 8 + (c ^ (row & 7))) * 16);
  };
  auto multiply = [&](int buf, bool tail) {
    const unsigned char* sp = smem + buf * C::STAGE;
    const unsigned char* sq = sp + C::BM * 128;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = 4 * h + lq;
      u32x4 a[C::FM], b[C::FN];
#pragma unroll
      for (int j = 0; j < C::FN; ++j) b[j] = read(sq, qrow + 16 * j, c);
#pragma unroll
      for (int i = 0; i < C::FM; ++i) a[i] = read(sp, prow + 16 * i, c);
      if (tail && c * 8 >= rem) {
#pragma unroll
        for (int j = 0; j < C::FN; ++j) b[j] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < C::FM; ++i) a[i] = u32x4{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) acc[i][j] = mfma32<DT>(a[i], b[j], acc[i][j]);
    }
  };

#pragma unroll
  for (int p = 0; p < C::NS - 1; ++p) issue(p, p);
  int buf = 0;
  auto step = [&](int s, bool tail) {
    wait_vmcnt<(C::NS - 2) * C::L>();
    wait_lgkm0();
    barrier_no_fence();
    const int fill = buf == 0 ? C::NS - 1 : buf - 1;
    issue(s + C::NS - 1, fill);
    multiply(buf, tail);
    buf = buf == C::NS - 1 ? 0 : buf + 1;
  };
  for (int s = 0; s < steps - 1; ++s) step(s, false);
  step(steps - 1, rem < 64);
  wait_vmcnt<0>();
  wait_lgkm0();
  barrier_no_fence();
  epi(acc, wm, wn, li, lq);
}

}  // namespace nm
