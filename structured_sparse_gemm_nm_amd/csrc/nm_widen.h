// The packed operand of one lane for one 64-wide K step, and its widening to
// the 2:4 operand v_smfmac takes (1:4 and 1:8 in registers).
#pragma once

#include "nm_device.h"

namespace nm {

constexpr int pat_n(int P) { return P == 0 ? 2 : 1; }
constexpr int pat_m(int P) { return P == 2 ? 8 : 4; }

struct AFrag {
  uint32_t v[4];
  uint32_t ib;
};

// Lane (row, lq) share of step s.  Rows past R and quarters past K load nothing.
template <int P>
__device__ inline void load_afrag(AFrag& f, const uint16_t* __restrict__ values,
                                  const uint32_t* __restrict__ idx, int64_t S, int64_t words, int row,
                                  int R, int K, int s, int lq) {
  f.v[0] = f.v[1] = f.v[2] = f.v[3] = 0u;
  f.ib = 0u;
  if (row >= R || s * 64 + lq * 16 >= K) return;
  const uint16_t* vrow = values + int64_t(row) * S;
  const unsigned char* irow = reinterpret_cast<const unsigned char*>(idx + int64_t(row) * words);
  if constexpr (P == 0) {
    const uint4 t = *reinterpret_cast<const uint4*>(vrow + s * 32 + lq * 8);
    f.v[0] = t.x; f.v[1] = t.y; f.v[2] = t.z; f.v[3] = t.w;
    f.ib = *reinterpret_cast<const uint16_t*>(irow + s * 8 + lq * 2);
  } else if constexpr (P == 1) {
    const uint2 t = *reinterpret_cast<const uint2*>(vrow + s * 16 + lq * 4);
    f.v[0] = t.x; f.v[1] = t.y;
    f.ib = irow[s * 4 + lq];
  } else {  // 1:8: 2 values (4 B), 6 index bits at bit 24 s + 6 lq of the row
    f.v[0] = *reinterpret_cast<const uint32_t*>(vrow + s * 8 + lq * 2);
    f.v[3] = 0u;
    // the aligned word holding the first bit and the next one (clamped to the
    // row's last word, whose bits then suffice): two loads from every lane,
    // kept as loaded (widen extracts the bits, so nothing here waits for them)
    const uint32_t* wrow = idx + int64_t(row) * words;
    const int bit = 24 * s + 6 * lq;
    const int w0 = bit >> 5;
    const int w1 = min(w0 + 1, int(words) - 1);
    f.v[1] = wrow[w0];
    f.v[2] = wrow[w1];
    f.ib = uint32_t(bit & 31);
  }
}

// 2:4: v = the 16 bytes of values, ib the 16 index bits.  1:4: v[0..1] = 4
// values, ib the byte of 4 positions.  1:8: v[0] = 2 values, v[1..2] the two
// words that hold the 6 index bits, ib the bit they start at.
template <int P>
__device__ inline void widen(const AFrag& f, u32x4& a, uint32_t& idx16) {
  if constexpr (P == 0) {
    a[0] = f.v[0]; a[1] = f.v[1]; a[2] = f.v[2]; a[3] = f.v[3];
    idx16 = f.ib & 0xFFFFu;
  } else if constexpr (P == 1) {
    a[0] = f.v[0] & 0xFFFFu; a[1] = f.v[0] >> 16; a[2] = f.v[1] & 0xFFFFu; a[3] = f.v[1] >> 16;
    const uint32_t ib = f.ib;
    const uint32_t t = (ib & 0x3u) | ((ib & 0xCu) << 2) | ((ib & 0x30u) << 4) | ((ib & 0xC0u) << 6);
    idx16 = t | (t << 2);
  } else {
    const uint32_t v0 = f.v[0] & 0xFFFFu, v1 = f.v[0] >> 16;
    const uint32_t ib = uint32_t((uint64_t(f.v[1]) | (uint64_t(f.v[2]) << 32)) >> f.ib);
    const uint32_t p0 = ib & 7u, p1 = (ib >> 3) & 7u;
    const bool h0 = p0 >= 4, h1 = p1 >= 4;
    a[0] = h0 ? 0u : v0; a[1] = h0 ? v0 : 0u;
    a[2] = h1 ? 0u : v1; a[3] = h1 ? v1 : 0u;
    const uint32_t f0 = (p0 & 3u) * 5u, f1 = (p1 & 3u) * 5u;
    idx16 = (h0 ? (f0 << 4) : f0) | (h1 ? (f1 << 12) : (f1 << 8));
  }
}

}  // namespace nm
