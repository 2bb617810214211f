// The low-rank term of a token tile on the matrix cores, shared by the kernels
// that add it to a product they hold in registers.
//
//   D[c][t] = s_a sum_j M_a[c][j] V[t][j],   a = ids[t],
//
// for the 16 tokens of a fragment and any number of 16-column fragments.  V is
// fp32 (the shrunk activations or gradients).  The matrix cores take 16-bit
// operands, so V is split into three bf16 parts, which hold its 24 bits; an
// fp16 M is split into two, exactly, since bf16's exponent range covers fp16's
// and 8 + 8 bits its 11.  bf16 throughout also means that no V, however large
// or small, leaves the operand's range.  (Two parts for V would keep 16 bits:
// an fp32 output then has four times the error of an fp32 product.)
#pragma once

#include "nm_device.h"
#include "nm_internal.h"

namespace nm {

// Eight floats as N bf16 operands that add up to them, the largest first.  A
// part that is not finite (f infinite, NaN, or rounded up to infinity) stays in
// the first alone.
template <int N>
__device__ inline void split8(const float (&f)[8], u32x4 (&part)[N]) {
  float r[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = f[e];
#pragma unroll
  for (int n = 0; n < N; ++n) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t h = pack_half2<NM_BF16>(r[2 * e], r[2 * e + 1]);
      part[n][e] = h;
      const float r0 = r[2 * e] - __builtin_bit_cast(float, h << 16);
      const float r1 = r[2 * e + 1] - __builtin_bit_cast(float, h & 0xFFFF0000u);
      r[2 * e] = fabsf(r0) < __builtin_inff() ? r0 : 0.f;
      r[2 * e + 1] = fabsf(r1) < __builtin_inff() ? r1 : 0.f;
    }
  }
}

// A 16-bit operand as bf16 parts: bf16 as it is (one part), fp16 in two.
template <int DT>
constexpr int operand_count() { return DT == NM_BF16 ? 1 : 2; }

template <int DT>
__device__ inline void operand_parts(const u32x4& raw, u32x4 (&part)[operand_count<DT>()]) {
  if constexpr (DT == NM_BF16) {
    part[0] = raw;
  } else {
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = half_to_f32<DT>((raw[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
    split8(f, part);
  }
}

// acc += a x b with both operands in parts, the smallest products first;
// products of parts more than 2^-24 below the largest are left out.
template <int NA, int NB>
__device__ inline f32x4 mfma_parts(const u32x4 (&a)[NA], const u32x4 (&b)[NB], f32x4 acc) {
#pragma unroll
  for (int k = 2; k >= 0; --k)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (k - i >= 0 && k - i < NB) acc = mfma32<NM_BF16>(a[i], b[k - i], acc);
  return acc;
}

// Operand lane (row c, quarter q) of M: elements j0 .. j0 + 7 (zeros past r).
// TRANS: M is [r][C], the lane's elements lie C apart.
template <bool TRANS>
__device__ inline u32x4 lowrank_operand(const uint16_t* Ma, int c, int64_t C, int j0, int r) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (j0 >= r) return v;
  if constexpr (TRANS) {
    const uint16_t* p = Ma + int64_t(j0) * C + c;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t x = j0 + e < r ? p[int64_t(e) * C] : 0u;
      v[e >> 1] |= x << (16 * (e & 1));
    }
  } else {
    const uint16_t* p = Ma + int64_t(c) * r + j0;
    if ((r & 7) == 0) {
      v = *reinterpret_cast<const u32x4*>(p);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t x = j0 + e < r ? p[e] : 0u;
        v[e >> 1] |= x << (16 * (e & 1));
      }
    }
  }
  return v;
}

// Elements j0 .. j0 + 7 of a row of r floats, zeros past r.
__device__ inline void load_v8(const float* row, int j0, int r, float (&v)[8]) {
  if ((r & 7) == 0 && j0 < r) {   // whole, aligned pieces
    const f32x4 a = *reinterpret_cast<const f32x4*>(row + j0), b = *reinterpret_cast<const f32x4*>(row + j0 + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = a[e];
      v[4 + e] = b[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = j0 + e < r ? row[j0 + e] : 0.f;
  }
}

// sum[e] += s_a sum_j M_a[c + e][j] V[t][j] for 4 columns of one token, on the
// vector ALUs: for few tokens, where every token has its own adapter and a
// matrix-core fragment would hold one column of use.  Columns past C reread
// column C - 1.  M as [n][C][r].
template <int DT>
__device__ inline void lowrank_columns4(const LowRank& p, int t, int c, f32x4& sum) {
  const int a = p.ids[t];
  if (uint32_t(a) >= uint32_t(p.n)) return;
  const float s = p.scale ? p.scale[a] : 1.f;
  const uint16_t* Ma = p.M + int64_t(a) * p.r * p.C;
  const float* vrow = p.V + int64_t(t) * p.r;
  f32x4 d = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < p.r; j += 8) {
    float v[8];
    load_v8(vrow, j, p.r, v);
    u32x4 m[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) m[e] = lowrank_operand<false>(Ma, min(c + e, p.C - 1), p.C, j, p.r);
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int q = 0; q < 8; ++q)
        // past r both are zero
        d[e] += half_to_f32<DT>((m[e][q >> 1] >> (16 * (q & 1))) & 0xFFFFu) * v[q];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[e] += s * d[e];
}

// acc(f, n) += the term, for F column fragments from c0 and NT token fragments
// (16 NT <= 64 tokens) from t0, in the matrix cores' result layout (lane (i, q):
// columns 4q .. 4q+3 of token i).  Every adapter that occurs among the tokens
// takes one round: its operands are loaded once for all of them (one round for
// a request's adjacent tokens, two where requests meet, 64 at worst).  With one
// adapter the product accumulates in place; with several, each token takes the
// sum of its own adapter's round by selection, never by a mask's product, so
// Inf and NaN stay with their adapter's tokens.  The scale goes into V (one
// fp32 rounding).  Columns past C and tokens past T reread the last one.
template <int DT, bool TRANS, int F, int NT, typename Acc>
__device__ inline void lowrank_add(const LowRank& p, int t0, int c0, Acc&& acc) {
  const int lane = threadIdx.x & 63, li = lane & 15, lq = lane >> 4;
  if (t0 >= p.T) return;
  const int id = p.ids[min(t0 + lane % (16 * NT), p.T - 1)];
  uint64_t todo = __ballot(uint32_t(id) < uint32_t(p.n));
  while (todo) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    const uint64_t mine = __ballot(id == a);
    todo &= ~mine;
    const uint16_t* Ma = p.M + int64_t(a) * p.r * p.C;
    const float s = p.scale ? p.scale[a] : 1.f;
    for (int j = 0; j < p.r; j += 32) {
      const int j0 = j + 8 * lq;
      float v[NT][8];
      u32x4 raw[F];
#pragma unroll
      for (int n = 0; n < NT; ++n) load_v8(p.V + int64_t(min(t0 + 16 * n + li, p.T - 1)) * p.r, j0, p.r, v[n]);
#pragma unroll
      for (int f = 0; f < F; ++f)
        raw[f] = lowrank_operand<TRANS>(Ma, min(c0 + 16 * f + li, p.C - 1), p.C, j0, p.r);
      __builtin_amdgcn_sched_barrier(0);   // every load above in flight before the first use
      u32x4 vp[NT][3];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[n][e] *= s;
        split8(v[n], vp[n]);
      }
      if (mine == ~uint64_t(0)) {
#pragma unroll
        for (int f = 0; f < F; ++f) {
          u32x4 mp[operand_count<DT>()];
          operand_parts<DT>(raw[f], mp);
#pragma unroll
          for (int n = 0; n < NT; ++n) acc(f, n) = mfma_parts(mp, vp[n], acc(f, n));
        }
      } else {
#pragma unroll
        for (int f = 0; f < F; ++f) {
          u32x4 mp[operand_count<DT>()];
          operand_parts<DT>(raw[f], mp);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const bool sel = (mine >> (16 * n + li)) & 1u;
            const f32x4 d = mfma_parts(mp, vp[n], f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int e = 0; e < 4; ++e) acc(f, n)[e] = sel ? acc(f, n)[e] + d[e] : acc(f, n)[e];
          }
        }
      }
    }
  }
}

}  // namespace nm
