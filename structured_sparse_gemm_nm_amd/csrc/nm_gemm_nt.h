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

#include <type_traits>

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

// The same product for large shapes: 256 x 256 tiles by 8 waves of 128 x 64,
// two a SIMD, software-pipelined.  With fragments read right before their MFMAs
// both waves of a SIMD leave each barrier at the same time and wait for the
// same LDS port (2048 x 32003 x 4096 fp16 with the softmax epilogue: 479 us).
// Here they go through two register sets: while one half step (32 k) is
// multiplied the next half's fragments are read and the loads of the step after
// next are issued between the MFMAs, in eight chunks a half that scheduling
// barriers keep in order (425 us, 1.26 PFLOP/s; the library's product alone
// takes 458).  Two stages of 64 k; a step's stage is free once its second half
// is in registers, at mid-step, where the one barrier a step stands:
//   first half   MFMAs on set 0 (s, 0);  reads (s, 1) into set 1;
//   barrier      step s+1 has landed, stage s is free;
//   second half  MFMAs on set 1;  reads (s+1, 0) into set 0;  loads step s+2.
// (4 waves of 128 x 128 read a third fewer LDS bytes, but alone on its SIMD a
// wave covers none of another's waits: 558 us.)
struct GemmTilePiped {
  static constexpr int BM = 256, BN = 256, WM = 2, WN = 4, THREADS = 512, FM = 8, FN = 4;
  static constexpr int STAGE = (BM + BN) * 128, LDS = 2 * STAGE;
};

template <int DT, class C, class Epi>
__device__ inline void gemm_nt_piped(const uint16_t* P, int64_t ldp, int M, const uint16_t* Q, int64_t ldq, int N, int K,
                                    int tm, int tn, unsigned char* smem, Epi&& epi) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const int wm = wave >> 2, wn = wave & 3;
  const int m0 = tm * C::BM, n0 = tn * C::BN;
  const int steps = (K + 63) >> 6;
  const int rem = K - (steps - 1) * 64;

  const __amdgpu_buffer_rsrc_t rp = make_rsrc(P + int64_t(m0) * ldp);
  const __amdgpu_buffer_rsrc_t rq = make_rsrc(Q + int64_t(n0) * ldq);
  // loads j = 0..3: rows (wave*4 + j)*8 + lane/8 of P, 4..7 the same of Q
  const uint32_t chunk = uint32_t((lane & 7) ^ ((lane >> 3) & 7));
  uint32_t off[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int row = (wave * 4 + j) * 8 + (lane >> 3);
    off[j] = uint32_t(min(row, M - 1 - m0)) * uint32_t(ldp) * 2u + chunk * 16u;
    off[4 + j] = uint32_t(min(row, N - 1 - n0)) * uint32_t(ldq) * 2u + chunk * 16u;
  }
  // past the end: again the last step, into a stage nothing reads any more
  auto issue = [&](int j, int s, uint32_t back, unsigned char* st) {
    dma16(j < 4 ? rp : rq, off[j] - back, uint32_t(s) * 128u,
          st + (j < 4 ? 0 : C::BM * 128) + (wave * 4 + (j & 3)) * 1024);
  };
  auto last_back = [&](int s) { return s == steps - 1 && int(chunk) * 8 >= rem ? chunk * 16u : 0u; };

  f32x4 acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // fragment i of the wave's rows, half h: its address differs from fragment
  // 0's by a constant (16 rows apart the swizzle is the same)
  const int prow = wm * 128 + li, qrow = wn * 64 + li;
  int pa[2], qa[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    pa[h] = (prow * 8 + ((4 * h + lq) ^ (prow & 7))) * 16;
    qa[h] = C::BM * 128 + (qrow * 8 + ((4 * h + lq) ^ (qrow & 7))) * 16;
  }
  auto read_p = [&](const unsigned char* st, int h, int i) {
    return *reinterpret_cast<const u32x4*>(st + pa[h] + i * 2048);
  };
  auto read_q = [&](const unsigned char* st, int h, int j) {
    return *reinterpret_cast<const u32x4*>(st + qa[h] + j * 2048);
  };
  u32x4 a0[8], b0[4], a1[8], b1[4];

  // One half step: MFMAs on (ca, cb); with READ, fragments of half rh of stage
  // rst into (na, nb); with LOAD, the 8 loads of step ls into stage lst.
  auto half = [&](auto read_c, auto load_c, const u32x4 (&ca)[8], const u32x4 (&cb)[4], u32x4 (&na)[8], u32x4 (&nb)[4],
                  const unsigned char* rst, int rh, int ls, uint32_t back, unsigned char* lst) {
    constexpr bool READ = decltype(read_c)::value, LOAD = decltype(load_c)::value;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      // reads in the first four chunks (the next half needs them right at its
      // start), loads spread over all eight
      if (READ && k < 4) {
        nb[k] = read_q(rst, rh, k);
        na[2 * k] = read_p(rst, rh, 2 * k);
        na[2 * k + 1] = read_p(rst, rh, 2 * k + 1);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[k][j] = mfma32<DT>(ca[k], cb[j], acc[k][j]);
      if constexpr (LOAD) issue(k, ls, back, lst);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  using yes = std::integral_constant<bool, true>;
  using no = std::integral_constant<bool, false>;
  // the last step's chunks past K: zeros on both sides
  auto trim = [&](u32x4 (&a)[8], u32x4 (&b)[4], int h) {
    if ((4 * h + lq) * 8 < rem) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a[i] = u32x4{0u, 0u, 0u, 0u};
      if (i < 4) b[i] = a[i];
    }
  };

  // step 0 in stage 0, step 1 in stage 1, (0, 0) in set 0
#pragma unroll
  for (int j = 0; j < 8; ++j) issue(j, 0, last_back(0), smem);
  const int s1 = min(1, steps - 1);
#pragma unroll
  for (int j = 0; j < 8; ++j) issue(j, s1, last_back(s1), smem + C::STAGE);
  wait_vmcnt<8>();
  barrier_no_fence();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a0[i] = read_p(smem, 0, i);
    if (i < 4) b0[i] = read_q(smem, 0, i);
  }
  // every step but the last in the loop, which then holds no branch
  for (int s = 0; s < steps - 1; ++s) {
    unsigned char* here = smem + (s & 1) * C::STAGE;
    unsigned char* next = smem + ((s & 1) ^ 1) * C::STAGE;
    half(yes{}, no{}, a0, b0, a1, b1, here, 1, 0, 0u, nullptr);
    wait_vmcnt<0>();
    wait_lgkm0();
    barrier_no_fence();
    const int ls = min(s + 2, steps - 1);
    half(yes{}, yes{}, a1, b1, a0, b0, next, 0, ls, last_back(ls), here);
  }
  if (rem < 64) trim(a0, b0, 0);
  half(yes{}, no{}, a0, b0, a1, b1, smem + ((steps - 1) & 1) * C::STAGE, 1, 0, 0u, nullptr);
  if (rem < 64) trim(a1, b1, 1);
  half(no{}, no{}, a1, b1, a0, b0, nullptr, 0, 0, 0u, nullptr);
  wait_vmcnt<0>();
  wait_lgkm0();
  barrier_no_fence();
  epi(acc, wm, wn, li, lq);
}

}  // namespace nm
