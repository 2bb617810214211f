// The shared N:M product of the adapters' forward pass where the prefill
// kernels' tiles would leave most of the chip idle: 17 to a few hundred tokens,
// few rows, or few tokens of a long K.
//
//   part[z][t][r] = sum over z's K steps of W_nm[r, k] act[t, k]   (fp32);
//
// the kernel that adds the low-rank term adds the shares, in order.  Bound by
// streaming the packed weight once per tile of 64 tokens and by the latency of
// the steps, so the K steps are dealt to many waves: a workgroup of 4 waves owns
// 32 rows x TB*16 tokens, its waves and blockIdx.z take 64-wide steps in turn.
// Every operand of a step comes straight into the wave's own ring of LDS stages
// (activations in whole 128-byte lines, packed values, index words), without a
// barrier until the waves' tiles are added in wave order.
// (4096 x 4096, 64 tokens, 2:4 bf16: 11.7 us, the register-prefetch kernel 37;
// 4096 x 11008, 16 tokens: 13, the generic kernel 92.  The whole call for 261
// tokens, 531 x 2848 1:8: 35 us, with the generic kernel 90.)
// Operand layouts and the 1:4 / 1:8 widening are those of nm_spmm.hip.
#include "nm_internal.h"
#include "nm_widen.h"

#include <algorithm>

namespace nm {
namespace {

constexpr int kWaves = 4, kRows = 32, kNS = 3;

template <int P, int TB>
struct Stage {
  static constexpr int ACT = TB * 2048;                 // [TB*16 tokens][128 bytes]
  static constexpr int VLOADS = P == 1 ? 1 : 2;
  static constexpr int VAL = P == 2 ? 512 : VLOADS * 1024;   // [32 rows][64, 32 or 16 bytes]
  static constexpr int BYTES = ACT + VAL + 256;         // + index words, 8 (1:4: 4) bytes a row
  static constexpr int LOADS = TB * 2 + VLOADS + 1;
  static constexpr int RING = kWaves * kNS * BYTES;
  static constexpr int PART = kWaves * 2 * TB * 1024;
  static constexpr int LDS = RING > PART ? RING : PART;
};

__device__ inline void dma4(__amdgpu_buffer_rsrc_t rsrc, uint32_t voff, unsigned char* lds_dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_byte*)lds_dst, 4, int(voff), 0, 0, 0);
}

template <int P, int DT, int TB>
__global__ __launch_bounds__(kWaves * 64) void adapter_product_kernel(const uint16_t* __restrict__ values,
                                                                      const uint32_t* __restrict__ idx, int words,
                                                                      int R, int K, const uint16_t* __restrict__ act,
                                                                      int64_t ldx, int T, float* __restrict__ part, int64_t ldp) {
  using St = Stage<P, TB>;
  extern __shared__ __align__(16) unsigned char smem[];
  const int lane = threadIdx.x & 63, li = lane & 15, lq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int R0 = blockIdx.x * kRows, T0 = blockIdx.y * (TB * 16);
  const int S = K / pat_m(P) * pat_n(P);
  const int steps = (K + 63) >> 6, rem = K - (steps - 1) * 64;   // 64 or 32
  const int first = blockIdx.z * kWaves + wave, stride = gridDim.z * kWaves;
  const int count = first < steps ? (steps - 1 - first) / stride + 1 : 0;

  const __amdgpu_buffer_rsrc_t ra = make_rsrc(act + int64_t(T0) * ldx);
  const __amdgpu_buffer_rsrc_t rv = make_rsrc(values + int64_t(R0) * S);
  const __amdgpu_buffer_rsrc_t ri = make_rsrc(idx + int64_t(R0) * words);
  // activations: slot (token, chunk c) at token*8 + (c ^ (token & 7))
  const uint32_t chunk = uint32_t((lane & 7) ^ ((lane >> 3) & 7));
  uint32_t aoff[TB * 2];
#pragma unroll
  for (int j = 0; j < TB * 2; ++j)
    aoff[j] = uint32_t(min(j * 8 + (lane >> 3), T - 1 - T0)) * uint32_t(ldx) * 2u + chunk * 16u;
  // values: 2:4 slot (row, quarter) at row*4 + (q ^ ((row >> 1) & 3)); 1:4 two
  // 16-byte pieces a row; 1:8 four of 4 bytes (its rows lie on 8 bytes where K is
  // an odd multiple of 32, and a short last step holds half of 16)
  constexpr uint32_t vbytes = P == 2 ? 4u : 16u;
  uint32_t voff[St::VLOADS], vpiece[St::VLOADS];
#pragma unroll
  for (int j = 0; j < St::VLOADS; ++j) {
    const int slot = j * 64 + lane;
    const int row = P == 1 ? slot >> 1 : slot >> 2;
    vpiece[j] = P == 0 ? uint32_t((slot & 3) ^ ((row >> 1) & 3)) : uint32_t(slot & (P == 1 ? 1 : 3));
    voff[j] = uint32_t(min(row, R - 1 - R0)) * uint32_t(S) * 2u + vpiece[j] * vbytes;
  }
  // index words: 2:4 and 1:8 two a row, 1:4 one (repeated)
  const int irow = P == 1 ? lane & 31 : lane >> 1;
  const uint32_t ioff = uint32_t(min(irow, R - 1 - R0)) * uint32_t(words) * 4u;
  unsigned char* ring = smem + wave * (kNS * St::BYTES);

  // The wave's i-th step into stage i % kNS (past its last one that step again,
  // into a stage nothing reads any more).  In a short last step the pieces past
  // K reread the step's first; they enter the product as zeros.
  auto issue = [&](int i) {
    const int s = first + min(i, count - 1) * stride;
    unsigned char* st = ring + i % kNS * St::BYTES;
    const bool tail = s == steps - 1;
    const uint32_t back = tail && int(chunk) * 8 >= rem ? chunk * 16u : 0u;
#pragma unroll
    for (int j = 0; j < TB * 2; ++j) dma16(ra, aoff[j] - back, uint32_t(s) * 128u, st + j * 1024);
    constexpr uint32_t vstep = P == 0 ? 64u : P == 1 ? 32u : 16u;
    constexpr int vk = P == 1 ? 32 : 16;     // K positions of a piece
#pragma unroll
    for (int j = 0; j < St::VLOADS; ++j) {
      const uint32_t vback = tail && int(vpiece[j]) * vk >= rem ? vpiece[j] * vbytes : 0u;
      if constexpr (P == 2) dma4(rv, voff[j] - vback + uint32_t(s) * vstep, st + St::ACT + j * 256);
      else dma16(rv, voff[j] - vback, uint32_t(s) * vstep, st + St::ACT + j * 1024);
    }
    const int word = P == 0 ? 2 * s + (lane & 1) : P == 1 ? s : ((24 * s) >> 5) + (lane & 1);
    dma4(ri, ioff + uint32_t(min(word, words - 1)) * 4u, st + St::ACT + St::VAL);
  };

  f32x4 acc[2][TB];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (count > 0) {
#pragma unroll
    for (int i = 0; i < kNS - 1; ++i) issue(i);
    for (int i = 0; i < count; ++i) {
      wait_lgkm0();                                // the stage about to be refilled has been read
      asm volatile("" ::: "memory");
      issue(i + kNS - 1);
      wait_vmcnt<(kNS - 1) * St::LOADS>();         // step i has landed
      asm volatile("" ::: "memory");
      const unsigned char* st = ring + i % kNS * St::BYTES;
      const unsigned char* sv = st + St::ACT;
      const unsigned char* si = sv + St::VAL;
      const int s = first + i * stride;
      const bool tail = s == steps - 1;
      u32x8 b[TB];
#pragma unroll
      for (int j = 0; j < TB; ++j) {
        const int tok = j * 16 + li;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = 4 * h + lq;
          u32x4 v = *reinterpret_cast<const u32x4*>(st + (tok * 8 + (c ^ (tok & 7))) * 16);
          if (tail && c * 8 >= rem) v = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
          for (int e = 0; e < 4; ++e) b[j][4 * h + e] = v[e];
        }
      }
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const int row = f * 16 + li;
        AFrag a;
        if constexpr (P == 0) {
          const u32x4 v = *reinterpret_cast<const u32x4*>(sv + (row * 4 + (lq ^ ((row >> 1) & 3))) * 16);
#pragma unroll
          for (int e = 0; e < 4; ++e) a.v[e] = v[e];
          a.ib = *reinterpret_cast<const uint16_t*>(si + row * 8 + lq * 2);
        } else if constexpr (P == 1) {
          const u32x2 v = *reinterpret_cast<const u32x2*>(sv + row * 32 + lq * 8);
          a.v[0] = v[0];
          a.v[1] = v[1];
          a.ib = si[row * 4 + lq];
        } else {
          const u32x2 w = *reinterpret_cast<const u32x2*>(si + row * 8);
          a.v[0] = *reinterpret_cast<const uint32_t*>(sv + row * 16 + lq * 4);
          a.v[1] = w[0];
          a.v[2] = w[1];
          a.ib = uint32_t((24 * s) & 31) + 6u * uint32_t(lq);
        }
        if (tail && lq * 16 >= rem) a = AFrag{};
        u32x4 m;
        uint32_t ix;
        widen<P>(a, m, ix);
#pragma unroll
        for (int j = 0; j < TB; ++j) acc[f][j] = smfmac<DT>(m, b[j], acc[f][j], ix);
      }
    }
    wait_vmcnt<0>();
    wait_lgkm0();
  }
  __syncthreads();                                 // every wave is done with its ring
  f32x4 (*sums)[2 * TB][64] = reinterpret_cast<f32x4 (*)[2 * TB][64]>(smem);
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int j = 0; j < TB; ++j) sums[wave][f * TB + j][lane] = acc[f][j];
  __syncthreads();
  for (int q = wave; q < 2 * TB; q += kWaves) {
    f32x4 v = sums[0][q][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += sums[w][q][lane];
    const int t = T0 + (q % TB) * 16 + li, r = R0 + (q / TB) * 16 + lq * 4;
    if (t >= T || r >= R) continue;
    *reinterpret_cast<f32x4*>(part + (int64_t(blockIdx.z) * T + t) * ldp + r) = v;   // ldp: R rounded up to 4
  }
}

int64_t token_frags(int64_t T) { return T <= 16 ? 1 : T <= 32 ? 2 : 4; }

template <int P, int DT, int TB>
hipError_t launch_tb(const SpmmArgs& a, float* part, hipStream_t s) {
  auto kern = adapter_product_kernel<P, DT, TB>;
  constexpr int lds = Stage<P, TB>::LDS;
  if (hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(kern), lds); e != hipSuccess) return e;
  const dim3 grid(unsigned((a.R + kRows - 1) / kRows), unsigned((a.T + TB * 16 - 1) / (TB * 16)),
                  unsigned(adapter_product_splits(a)));
  hipLaunchKernelGGL(kern, grid, dim3(kWaves * 64), lds, s, a.values, a.idx, int(a.idx_row_words), int(a.R), int(a.K),
                     a.act, a.ldx, int(a.T), part, adapter_product_ld(a));
  return hipGetLastError();
}

template <int P, int DT>
hipError_t launch_p(const SpmmArgs& a, float* part, hipStream_t s) {
  switch (token_frags(a.T)) {
    case 1: return launch_tb<P, DT, 1>(a, part, s);
    case 2: return launch_tb<P, DT, 2>(a, part, s);
    default: return launch_tb<P, DT, 4>(a, part, s);
  }
}

template <int DT>
hipError_t launch_dt(const SpmmArgs& a, float* part, hipStream_t s) {
  if (a.n == 2) return launch_p<0, DT>(a, part, s);
  return a.m == 4 ? launch_p<1, DT>(a, part, s) : launch_p<2, DT>(a, part, s);
}

}  // namespace

// Shares of the K steps: enough workgroups to cover the chip twice, four steps
// a wave at least.
int64_t adapter_product_splits(const SpmmArgs& a) {
  const int64_t per = token_frags(a.T) * 16;
  const int64_t tiles = (a.R + kRows - 1) / kRows * ((a.T + per - 1) / per), steps = (a.K + 63) / 64;
  return std::max<int64_t>(std::min<int64_t>(512 / std::max<int64_t>(tiles, 1), steps / (4 * kWaves)), 1);
}

// Shapes it takes (a short last step leaves whole pieces of values: K a multiple
// of 32; grid limits), and among them those where it is
// the fastest: a K of at least 16 steps (shorter ones leave nothing to share
// out) and prefill tiles, 256 x 128 (1:4 and 1:8: 128 x 64), that cover less
// than a quarter (a half) of the chip.
bool adapter_product_applies(const SpmmArgs& a) {
  if (a.R < 1 || a.T < 1 || a.K < 1024 || a.K % 32 != 0 || a.T > (int64_t(1) << 20)) return false;
  const int64_t wide = (a.R + 255) / 256 * ((a.T + 127) / 128), narrow = (a.R + 127) / 128 * ((a.T + 63) / 64);
  if (spmm_lds_applies(a)) return wide < 64;
  if (spmm_lds_nm_applies(a)) return narrow < 128;
  return wide < 128;
}

hipError_t launch_adapter_product(const SpmmArgs& a, float* part, hipStream_t s) {
  return a.dtype == NM_F16 ? launch_dt<NM_F16>(a, part, s) : launch_dt<NM_BF16>(a, part, s);
}

}  // namespace nm
