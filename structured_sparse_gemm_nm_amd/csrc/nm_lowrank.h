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

// One float in three bf16 parts.
__device__ inline void split3(float f, uint16_t (&h)[3]) {
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    h[k] = to_half_bits<NM_BF16>(f);
    f -= half_to_f32<NM_BF16>(h[k]);
    f = fabsf(f) < __builtin_inff() ? f : 0.f;   // what is not finite stays in the first part alone
  }
}

// Offset past every descriptor here: a load from it returns zeros.
constexpr uint32_t kLowRankDead = 0xFFFFFFF0u;

// Operand lane (row c, quarter q) of an adapter's M (its descriptor): elements
// j0 .. j0 + 7, zeros past r.  No branch over the lanes, so that a tile's loads
// are issued together.
__device__ inline u32x4 lowrank_operand(__amdgpu_buffer_rsrc_t rm, int c, int j0, int r) {
  const uint32_t at = (uint32_t(c) * uint32_t(r) + uint32_t(j0)) * 2u;
  if ((r & 7) == 0)
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rm, j0 < r ? at : kLowRankDead, 0, 0));
  u32x4 v;   // rows not on 16 bytes: element by element
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t lo = __builtin_amdgcn_raw_buffer_load_b16(rm, j0 + 2 * e < r ? at + 4u * e : kLowRankDead, 0, 0);
    const uint32_t hi =
        __builtin_amdgcn_raw_buffer_load_b16(rm, j0 + 2 * e + 1 < r ? at + 4u * e + 2u : kLowRankDead, 0, 0);
    v[e] = lo | (hi << 16);
  }
  return v;
}

// An adapter's M.
__device__ inline __amdgpu_buffer_rsrc_t lowrank_rsrc(const LowRank& p, int a) {
  return make_rsrc(p.M + int64_t(a) * p.r * p.C, uint32_t(p.r) * uint32_t(p.C) * 2u);
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
// matrix-core fragment would hold one column of use.  The token's adapter is
// loaded with the kernel's first loads, the first 16 ranks' operands while its
// waves still join their partial sums (11008 x 4096, 16 tokens of rank 16, the
// whole call: 19.2 us with all of it loaded at the end, 16.7 so).  Columns past
// C reread column C - 1.
template <int DT>
struct LowRankFew {
  int a = -1;           // none
  float s;
  u32x4 m[2][4];
  float v[2][8];

  __device__ void adapter(const LowRank& p, int t) {
    if (t < p.T) a = p.ids[t];
  }
  __device__ void load8(const LowRank& p, int t, int c, int j, u32x4 (&mm)[4], float (&vv)[8]) const {
    load_v8(p.V + int64_t(t) * p.r, j, p.r, vv);
    const uint16_t* Ma = p.M + int64_t(a) * p.r * p.C;   // the lanes' adapters differ: plain addresses
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint16_t* row = Ma + int64_t(min(c + e, p.C - 1)) * p.r + j;
      if ((p.r & 7) == 0) {
        mm[e] = *reinterpret_cast<const u32x4*>(row);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          mm[e][q] = (j + 2 * q < p.r ? uint32_t(row[2 * q]) : 0u) |
                     (j + 2 * q + 1 < p.r ? uint32_t(row[2 * q + 1]) << 16 : 0u);
      }
    }
  }
  __device__ void load(const LowRank& p, int t, int c) {
    if (uint32_t(a) >= uint32_t(p.n)) {
      a = -1;
      return;
    }
    s = p.scale ? p.scale[a] : 1.f;
    load8(p, t, c, 0, m[0], v[0]);
    if (p.r > 8) load8(p, t, c, 8, m[1], v[1]);
  }
  __device__ void add(const LowRank& p, int t, int c, f32x4& sum) {
    if (a < 0) return;
    f32x4 d = {0.f, 0.f, 0.f, 0.f};
    auto dot8 = [&](const u32x4 (&mm)[4], const float (&vv)[8]) {   // past r both are zero
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int q = 0; q < 8; ++q) d[e] += half_to_f32<DT>((mm[e][q >> 1] >> (16 * (q & 1))) & 0xFFFFu) * vv[q];
    };
    dot8(m[0], v[0]);
    if (p.r > 8) dot8(m[1], v[1]);
    for (int j = 16; j < p.r; j += 8) {
      load8(p, t, c, j, m[0], v[0]);
      dot8(m[0], v[0]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] += s * d[e];
  }
};

// The adapters of a tile of 16 NT tokens, a lane a token (tokens past T count
// as the last); loaded early by the kernels that add the term late.
template <int NT>
__device__ inline int lowrank_ids(const LowRank& p, int t0) {
  return p.ids[min(t0 + int(threadIdx.x & 63) % (16 * NT), p.T - 1)];
}

// acc(f, n) += the term, for F column fragments from c0 and NT token fragments
// (16 NT <= 64 tokens) from t0, in the matrix cores' result layout (lane (i, q):
// columns 4q .. 4q+3 of token i); id from lowrank_ids.  Every adapter that
// occurs among the tokens takes one round: its operands are loaded once for all
// of them (one round for a request's adjacent tokens, two where requests meet,
// 64 at worst).  With one adapter the product accumulates in place; with
// several, each token takes the sum of its own adapter's round by selection,
// never by a mask's product, so Inf and NaN stay with their adapter's tokens (the
// two differ in rounding: a token's last bit depends on its neighbours' adapters).
// Columns past C and tokens past T reread the last one.
template <int DT, int F, int NT, typename Acc>
__device__ inline void lowrank_add(const LowRank& p, int id, int t0, int c0, Acc&& acc) {
  const int lane = threadIdx.x & 63, li = lane & 15, lq = lane >> 4;
  if (t0 >= p.T) return;
  const int r8 = (p.r + 7) & ~7;
  const int rows = min(16 * NT, p.T - t0);
  const __amdgpu_buffer_rsrc_t rp = make_rsrc(p.P + int64_t(t0) * 3 * r8, uint32_t(rows) * 3u * uint32_t(r8) * 2u);
  uint64_t todo = __ballot(uint32_t(id) < uint32_t(p.n));
  while (todo) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    const uint64_t mine = __ballot(id == a);
    todo &= ~mine;
    const __amdgpu_buffer_rsrc_t rm = lowrank_rsrc(p, a);
    for (int j = 0; j < p.r; j += 32) {
      const int j0 = j + 8 * lq;
      u32x4 vp[NT][3], raw[F];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint32_t at = (uint32_t(min(16 * n + li, rows - 1)) * 3u * uint32_t(r8) + uint32_t(j0)) * 2u;
#pragma unroll
        for (int k = 0; k < 3; ++k)
          vp[n][k] = __builtin_bit_cast(
              u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                         rp, j0 < p.r ? at + uint32_t(k) * uint32_t(r8) * 2u : kLowRankDead, 0, 0));
      }
#pragma unroll
      for (int f = 0; f < F; ++f) raw[f] = lowrank_operand(rm, min(c0 + 16 * f + li, p.C - 1), j0, p.r);
      __builtin_amdgcn_sched_barrier(0);   // every load above in flight before the first use
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
