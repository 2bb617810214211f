// Internal declarations shared by the host API and the kernel launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "nmsparse.h"

namespace nm {

enum { NM_VARIANT_AUTO = 0, NM_VARIANT_GENERIC = 1, NM_VARIANT_PIPE = 2, NM_VARIANT_LDS = 3,
       NM_VARIANT_DECODE = 4, NM_VARIANT_RESIDENT = 5, NM_VARIANT_LDS_NM = 6, NM_VARIANT_MAX = 6 };

// Launchers (defined next to their kernels).  Arguments are already
// validated; each returns the hipError_t of its launch.
hipError_t launch_prune_pack(const uint16_t* W, int64_t R, int64_t K, int64_t ldw, int n, int m,
                             uint16_t* values, uint32_t* idx, int64_t idx_row_words,
                             hipStream_t s);

hipError_t launch_decompress(const uint16_t* values, const uint32_t* idx, int64_t R, int64_t K,
                             int n, int m, int64_t idx_row_words, uint16_t* W, int64_t ldw,
                             hipStream_t s);

// 8-bit 2:4 (nm_int8.hip): prune + pack, decompress (leading dimensions in
// bytes, multiples of 16; K % 32 == 0).  f8: FP8 E4M3 keys (bits & 0x7F)
// instead of int8 |w|; decompress moves bytes and serves both.
hipError_t launch_prune_pack_i8(const uint8_t* W, int64_t R, int64_t K, int64_t ldw, uint8_t* values,
                                uint32_t* idx, int64_t idx_row_words, bool f8, hipStream_t s);
hipError_t launch_decompress_i8(const uint8_t* values, const uint32_t* idx, int64_t R, int64_t K,
                                int64_t idx_row_words, uint8_t* W, int64_t ldw, hipStream_t s);

// The low-rank term s_a sum_j M_a[c][j] V[t][j], a = ids[t], of a product's
// columns c (nm_lowrank.h).  The few-token kernels read V and scale, the
// matrix-core kernels P.
struct LowRank {
  const int32_t* ids = nullptr;   // [T]: the token's adapter; outside [0, n): none
  const uint16_t* M = nullptr;    // [n][C][r]
  const float* scale = nullptr;   // [n], or null: 1
  const float* V = nullptr;       // [T][r]
  const uint16_t* P = nullptr;    // [T][3][r8]: s_a V in three bf16 parts, zeros from r to r8 (r rounded up to 8)
  int n = 0, r = 0, T = 0;
  int C = 0;                      // columns of the product
};
// In the place of a LowRank: none.
struct NoLowRank {};

struct SpmmArgs {
  const uint16_t* values;
  const uint32_t* idx;
  int64_t R, K;
  int n, m;
  int dtype;             // NM_F16 / NM_BF16 / NM_I8 / NM_FP8 (the last two: bytes)
  const uint16_t* act;   // [T, K], ldx (elements)
  int64_t T, ldx;
  const int32_t* perm;   // nullptr: identity
  void* Y;               // [T, R], ldy
  int64_t ldy;
  int out_dtype;         // NM_F32 or dtype
  int64_t idx_row_words;
  int variant;           // NM_VARIANT_* (0 = choose by shape)
  void* workspace;       // permuted product: caller memory for X' = act[:, perm], or null
  size_t workspace_bytes;
  const LowRank* lowrank = nullptr;   // added in the epilogue (few-token and all-LDS families, no map)
};

hipError_t launch_spmm(const SpmmArgs& a, hipStream_t s);
// Training-side products (nm_train.hip): dX = G W_nm and the packed dW.
struct TrainArgs {
  const uint16_t* values;  // packed W (dX only)
  size_t values_bytes;
  const uint32_t* idx;     // index words of the packed W
  size_t idx_bytes;
  int64_t R, K;
  int n, m;
  int dtype;               // NM_F16 / NM_BF16
  int64_t idx_row_words;
  const uint16_t* G;       // [T, R], ldg: gradient of the forward output
  int64_t T, ldg;
  const uint16_t* act;     // [T, K], ldx (dW only)
  int64_t ldx;
  void* out;               // dX [T, K] (ldo) or dW [R, S] (contiguous)
  int64_t ldo;
  int out_dtype;           // NM_F32 or dtype
  const LowRank* lowrank = nullptr;   // dX only: added in the epilogue
};
hipError_t launch_spmm_dx(const TrainArgs& a, hipStream_t s);
hipError_t launch_spmm_dw(const TrainArgs& a, hipStream_t s);

// 8-bit 2:4 GEMM (nm_int8.hip): Y int32 for NM_I8, fp32 for NM_FP8.
hipError_t launch_spmm_i8(const SpmmArgs& a, hipStream_t s);

// Pipelined large-tile kernel (nm_spmm_pipe.hip) and the shapes it takes.
bool spmm_pipe_applies(const SpmmArgs& a);
hipError_t launch_spmm_pipe(const SpmmArgs& a, hipStream_t s);

// Few-token kernel (nm_spmm_decode.hip) and the shapes it takes.
bool spmm_decode_applies(const SpmmArgs& a);
hipError_t launch_spmm_decode(const SpmmArgs& a, hipStream_t s);

// Permuted product as a gather pass X' = act[:, perm] into the caller's
// workspace followed by the plain GEMM on X' (nm_permute.hip): the bytes it
// needs (0 when the shape does not take it), and the launch.
size_t spmm_perm_gather_bytes(int64_t T, int64_t K, int dtype);
hipError_t launch_spmm_perm_gather(const SpmmArgs& a, void* workspace, hipStream_t s);

// The file-scope device array nm_spmm_perm_static uses as its workspace
// (nm_permute.hip): its size, and its address on the current device.
constexpr size_t kStaticWorkspaceBytes = size_t(32) << 20;
hipError_t static_workspace(void** ptr);

// 2:4 kernel with the token tile resident in LDS, plain or through the index
// map (nm_spmm_resident.hip), and the shapes it takes.
bool spmm_resident_applies(const SpmmArgs& a);
hipError_t launch_spmm_resident(const SpmmArgs& a, hipStream_t s);

// All-LDS 2:4 kernel (nm_spmm_lds.hip) and the shapes it takes.
bool spmm_lds_applies(const SpmmArgs& a);
hipError_t launch_spmm_lds(const SpmmArgs& a, hipStream_t s);

// All-LDS 1:4 / 1:8 kernel with 128 x 64 tiles (nm_spmm_lds_nm.hip) and the
// shapes it takes.
bool spmm_lds_nm_applies(const SpmmArgs& a);
hipError_t launch_spmm_lds_nm(const SpmmArgs& a, hipStream_t s);

// Hybrid dense / 2:4 weight tiles (nm_hybrid.hip): pack and product.  The
// layout tables are device arrays as nm_hybrid_layout writes them; values_bytes
// and idx_bytes bound every weight access (both below 2^32).
struct HybridArgs {
  const uint16_t* values = nullptr;   // product: packed weights
  const uint8_t* idx = nullptr;
  const int64_t* tile_meta = nullptr;
  const int64_t* row_meta = nullptr;
  int64_t R = 0, K = 0, tile_rows = 0, tile_cols = 0;
  int dtype = 0;
  uint64_t values_bytes = 0, idx_bytes = 0;
  const uint16_t* act = nullptr;      // product: activations and output
  int64_t T = 0, ldx = 0;
  void* Y = nullptr;
  int64_t ldy = 0;
  int out_dtype = 0;
  const uint16_t* W = nullptr;        // pack: dense weights and packed outputs
  int64_t ldw = 0;
  uint16_t* values_out = nullptr;
  uint8_t* idx_out = nullptr;
};
constexpr int64_t kHybridMaxTileCols = 8192;  // tile-columns per row the product takes
hipError_t launch_hybrid_pack(const HybridArgs& a, hipStream_t s);
hipError_t launch_hybrid_spmm(const HybridArgs& a, hipStream_t s);

// The column permutation on block-sparse and diagonal-sparse weights
// (nm_hosts.hip).  values_bytes and act_bytes bound the weight and activation
// reads (both below 2^32); row_ptr / col entries are clamped into range on the
// device, so a malformed structure gives wrong sums but no stray access.
struct HostArgs {
  bool diagonal = false;
  const uint16_t* values = nullptr;
  uint64_t values_bytes = 0;
  const int32_t* row_ptr = nullptr;   // block
  const int32_t* col = nullptr;
  const int32_t* offsets = nullptr;   // diagonal
  int64_t nnz = 0;                    // kept blocks, or diagonals
  int64_t R = 0, K = 0;
  int dtype = 0;
  const uint16_t* act = nullptr;
  uint64_t act_bytes = 0;
  int64_t ldx = 0, T = 0;
  const int32_t* perm = nullptr;      // NULL: act read as it is
  void* out = nullptr;
  int64_t ldy = 0;
  int out_dtype = 0;
};
constexpr int64_t kDiagMaxK = 1792;   // the diagonal product stages 80 bytes per column (and the offsets) in LDS
hipError_t launch_block_pack(const uint16_t* W, int64_t ldw, int64_t R, int64_t K, const int32_t* row_ptr,
                             const int32_t* col, int64_t nnzb, uint16_t* values, hipStream_t s);
hipError_t launch_diag_pack(const uint16_t* W, int64_t ldw, int64_t R, int64_t K, const int32_t* offsets, int64_t D,
                            uint16_t* values, hipStream_t s);
hipError_t launch_host_spmm(const HostArgs& a, hipStream_t s);

// Low-rank adapters beside an N:M product (nm_adapter.hip).
struct AdapterArgs {
  SpmmArgs base{};                  // the shared product, Y the final output
  const int32_t* ids = nullptr;     // [T]
  int64_t n = 0, r = 0;             // adapters, rank
  const uint16_t* A = nullptr;      // [n][r][K]
  const uint16_t* B = nullptr;      // [n][R][r]
  const float* scale = nullptr;     // [n]
  float* xa = nullptr;              // [T][r] (written)
  void* workspace = nullptr;        // adapter_workspace bytes
};
struct AdapterBwdArgs {
  TrainArgs dx{};                   // G, act and dX (out, may be null)
  const int32_t* ids = nullptr;
  int64_t n = 0, r = 0;
  const uint16_t* A = nullptr;
  const uint16_t* B = nullptr;
  const float* scale = nullptr;
  const float* xa = nullptr;
  float* dA = nullptr;              // [n][r][K]
  float* dB = nullptr;              // [n][R][r]
  void* workspace = nullptr;        // adapter_bwd_workspace bytes
};
constexpr int64_t kAdapterMaxRank = 256, kAdapterMaxCount = 65535;
constexpr int64_t kAdapterMaxTokens = int64_t(1) << 24, kAdapterMaxWidth = int64_t(1) << 22;   // grid limits
size_t adapter_workspace(const SpmmArgs& base, int64_t r);   // pointers are not looked at
size_t adapter_bwd_workspace(int64_t R, int64_t K, int64_t T, int64_t n, int64_t r);
hipError_t launch_adapter(const AdapterArgs& a, hipStream_t s);
// Their shared product as shares part[splits][T][ld] (nm_adapter_product.hip).
bool adapter_product_applies(const SpmmArgs& a);
int64_t adapter_product_splits(const SpmmArgs& a);
inline int64_t adapter_product_ld(const SpmmArgs& a) { return (a.R + 3) / 4 * 4; }   // rows on 16 bytes
hipError_t launch_adapter_product(const SpmmArgs& a, float* part, hipStream_t s);
hipError_t launch_adapter_bwd(const AdapterBwdArgs& a, hipStream_t s);

// Softmax cross entropy over a vocabulary (nm_xent.hip).
struct XentArgs {
  const uint16_t* x = nullptr;      // [T, H], ldx
  const uint16_t* w = nullptr;      // [V, H], ldw
  const int32_t* labels = nullptr;  // [T]
  int64_t ldx = 0, ldw = 0, T = 0, V = 0, H = 0;
  int dtype = 0;
  float* loss = nullptr;            // forward: [T]
  float* lse_out = nullptr;
  const float* lse = nullptr;       // backward: [T]
  const float* dloss = nullptr;
  void* dx = nullptr;               // [T, H], lddx, or null
  void* dw = nullptr;               // [V, H], lddw, or null
  int64_t lddx = 0, lddw = 0;
  int dx_dtype = 0, dw_dtype = 0;
  void* workspace = nullptr;
};
constexpr int64_t kXentMaxTokens = int64_t(1) << 22, kXentMaxVocab = int64_t(1) << 24, kXentMaxH = int64_t(1) << 20;
size_t xent_workspace(int64_t T, int64_t V);
// dx, dw: 0 not wanted, 1 in the inputs' type, 2 in fp32.
size_t xent_bwd_workspace(int64_t T, int64_t V, int64_t H, int dx, int dw);
hipError_t launch_xent(const XentArgs& a, hipStream_t s);
hipError_t launch_xent_bwd(const XentArgs& a, hipStream_t s);

// Layer norm (nm_layernorm.hip).  Forward: x, weight, bias -> y (and mean_out,
// rstd_out when given); backward: dy, x, mean, rstd, weight -> dx, dw, db (the
// last two through partial sums in `workspace`).
struct LayerNormArgs {
  int64_t T = 0, H = 0;
  int dtype = 0;
  const void* x = nullptr;
  int64_t ldx = 0;
  const void* weight = nullptr;
  const void* bias = nullptr;
  float eps = 0.f;
  void* y = nullptr;
  int64_t ldy = 0;
  float* mean_out = nullptr;
  float* rstd_out = nullptr;
  const void* dy = nullptr;
  int64_t ldg = 0;
  const float* mean = nullptr;
  const float* rstd = nullptr;
  void* dx = nullptr;
  int64_t lddx = 0;
  void* dw = nullptr;
  void* db = nullptr;
  int out_dtype = 0;
  void* workspace = nullptr;
};
size_t layernorm_bwd_workspace(int64_t T, int64_t H);
hipError_t launch_layernorm(const LayerNormArgs& a, hipStream_t s);
hipError_t launch_layernorm_bwd(const LayerNormArgs& a, hipStream_t s);

// Device properties and per-kernel launch set-up, kept per device and safe to
// call from several host threads (nm_api.cpp).
int device_cu_count();                 // CUs of the current device (256 if the query fails)
int device_max_lds();                  // its largest workgroup LDS allocation (0 if the query fails)
// Allow kern up to `bytes` of dynamic LDS on the current device (done once per
// device and kernel).
hipError_t ensure_lds_limit(const void* kern, int bytes);

inline int index_bits(int m) {
  int b = 0;
  while ((1 << b) < m) ++b;
  return b < 1 ? 1 : b;
}

}  // namespace nm
