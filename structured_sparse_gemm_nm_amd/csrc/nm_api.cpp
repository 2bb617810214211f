// C ABI of the N:M sparse library: argument validation and dispatch.
//
// Every check runs on the host before the first HIP call, so argument errors
// never touch the device and can be tested without a GPU.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <map>
#include <mutex>
#include <set>
#include <string>
#include <utility>
#include <vector>

#include "nm_internal.h"

namespace {

thread_local std::string g_last_error;

constexpr int64_t kMaxK = int64_t(1) << 24;
constexpr int64_t kMaxRT = int64_t(1) << 30;
constexpr int64_t kMaxElems = int64_t(1) << 40;

nm_status fail(nm_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = std::string(nm_status_string(st)) + ": " + buf;
  return st;
}

nm_status ok() {
  g_last_error.clear();
  return NM_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// One-byte weight types (INT8, FP8 E4M3).
bool byte_type(int dtype) { return dtype == NM_I8 || dtype == NM_FP8; }

bool supported_pattern(int n, int m) {
  return (n == 2 && m == 4) || (n == 1 && m == 4) || (n == 1 && m == 8);
}

// Checks shared by every entry point that names a packed weight.
nm_status check_format(int64_t R, int64_t K, int n, int m, int dtype) {
  if (dtype != NM_F16 && dtype != NM_BF16 && dtype != NM_I8 && dtype != NM_FP8)
    return fail(NM_ERR_UNSUPPORTED, "weight dtype %d is not NM_F16, NM_BF16, NM_I8 or NM_FP8", dtype);
  if (!supported_pattern(n, m))
    return fail(NM_ERR_UNSUPPORTED, "pattern %d:%d is not one of 2:4, 1:4, 1:8", n, m);
  if (byte_type(dtype) && !(n == 2 && m == 4))
    return fail(NM_ERR_UNSUPPORTED, "8-bit weights take the 2:4 pattern only");
  if (R < 0 || R > kMaxRT) return fail(NM_ERR_SHAPE, "R = %lld out of range", (long long)R);
  if (K < 16 || K > kMaxK) return fail(NM_ERR_SHAPE, "K = %lld out of range [16, 2^24]", (long long)K);
  if (K % 16) return fail(NM_ERR_SHAPE, "K = %lld is not a multiple of 16", (long long)K);
  if (byte_type(dtype) && K % 32)
    return fail(NM_ERR_SHAPE, "K = %lld is not a multiple of 32 (8-bit weights)", (long long)K);
  if (K % m) return fail(NM_ERR_SHAPE, "K = %lld is not a multiple of m = %d", (long long)K, m);
  if (R * K > kMaxElems) return fail(NM_ERR_SHAPE, "R*K too large");
  return NM_OK;
}

struct Sizes {
  int64_t S, words;
  size_t values_bytes, idx_bytes;
};

// Bytes per element of a storage type.
size_t elt_bytes(int dtype) { return byte_type(dtype) ? 1 : dtype == NM_F32 || dtype == NM_I32 ? 4 : 2; }

// Leading dimensions (elements) keep every row 16-byte aligned.
int64_t ld_quantum(int dtype) { return byte_type(dtype) ? 16 : 8; }

Sizes sizes_of(int64_t R, int64_t K, int n, int m, int dtype) {
  Sizes z;
  z.S = K / m * n;
  z.words = (z.S * nm::index_bits(m) + 31) / 32;
  z.values_bytes = size_t(R) * size_t(z.S) * elt_bytes(dtype);
  z.idx_bytes = size_t(R) * size_t(z.words) * 4;
  return z;
}

// Byte extent of a row-major [rows, cols] matrix with leading dimension ld.
size_t extent(int64_t rows, int64_t cols, int64_t ld, size_t elt) {
  if (rows <= 0 || cols <= 0) return 0;
  return (size_t(rows - 1) * size_t(ld) + size_t(cols)) * elt;
}

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}

struct Span {
  const void* p;
  size_t bytes;
};

// NM_ERR_ALIAS if an output overlaps an input or another output.
template <int NI, int NO>
nm_status check_alias(const Span (&in)[NI], const Span (&out)[NO]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j)
      if (overlaps(out[i].p, out[i].bytes, in[j].p, in[j].bytes))
        return fail(NM_ERR_ALIAS, "an output overlaps an input");
    for (int j = 0; j < i; ++j)
      if (overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
        return fail(NM_ERR_ALIAS, "outputs or workspace overlap each other");
  }
  return NM_OK;
}

nm_status hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return ok();
  return fail(NM_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

// Tile grid of the hybrid layout: tiles of tile_rows x tile_cols, both
// positive multiples of 64, tile_cols dividing K, at most kHybridMaxTileCols
// tile-columns; R up to 2^30, K up to 2^24.
nm_status check_hybrid_grid(int64_t R, int64_t K, int64_t tile_rows, int64_t tile_cols) {
  if (R < 0 || R > kMaxRT) return fail(NM_ERR_SHAPE, "R = %lld out of range", (long long)R);
  if (K < 64 || K > kMaxK) return fail(NM_ERR_SHAPE, "K = %lld out of range [64, 2^24]", (long long)K);
  if (tile_rows < 64 || tile_rows % 64 || tile_rows > kMaxRT)
    return fail(NM_ERR_SHAPE, "tile_rows = %lld is not a positive multiple of 64", (long long)tile_rows);
  if (tile_cols < 64 || tile_cols % 64 || K % tile_cols)
    return fail(NM_ERR_SHAPE, "tile_cols = %lld is not a multiple of 64 dividing K = %lld",
                (long long)tile_cols, (long long)K);
  if (K / tile_cols > nm::kHybridMaxTileCols)
    return fail(NM_ERR_SHAPE, "K / tile_cols = %lld tile-columns exceeds %lld", (long long)(K / tile_cols),
                (long long)nm::kHybridMaxTileCols);
  return NM_OK;
}

// Sizes of the packed hybrid arrays: the kernels address them with 32-bit
// byte offsets and use offsets from 2^31 up as "outside".
nm_status check_hybrid_totals(int64_t values_count, int64_t idx_bytes) {
  if (values_count < 0 || idx_bytes < 0) return fail(NM_ERR_SHAPE, "negative packed size");
  if (values_count * 2 >= (int64_t(1) << 31) || idx_bytes >= (int64_t(1) << 31))
    return fail(NM_ERR_SHAPE, "packed hybrid weight of %lld values / %lld index bytes reaches 2 GiB",
                (long long)values_count, (long long)idx_bytes);
  return NM_OK;
}

bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

nm_status spmm_common(const void* values, const uint32_t* idx, int64_t R, int64_t K, int n, int m,
                      int dtype, const void* act, int64_t T, int64_t ldx, const int32_t* perm,
                      bool want_perm, void* Y, int64_t ldy, int out_dtype, void* workspace,
                      size_t workspace_bytes, int variant, void* stream, bool static_ws = false) {
  nm_status st = check_format(R, K, n, m, dtype);
  if (st != NM_OK) return st;
  if (variant < 0 || variant > nm::NM_VARIANT_MAX)
    return fail(NM_ERR_UNSUPPORTED, "kernel family %d is not 0..%d", variant, int(nm::NM_VARIANT_MAX));
  if (T < 0 || T > kMaxRT) return fail(NM_ERR_SHAPE, "T = %lld out of range", (long long)T);
  if (dtype == NM_I8 || dtype == NM_FP8) {
    const int want = dtype == NM_I8 ? NM_I32 : NM_F32;
    if (out_dtype != want)
      return fail(NM_ERR_UNSUPPORTED, "%s weights give an %s output", dtype == NM_I8 ? "int8" : "fp8",
                  dtype == NM_I8 ? "NM_I32" : "NM_F32");
    if (want_perm) return fail(NM_ERR_UNSUPPORTED, "nm_spmm_perm does not take 8-bit weights");
  } else if (out_dtype != NM_F32 && out_dtype != dtype) {
    return fail(NM_ERR_UNSUPPORTED, "out_dtype %d must be NM_F32 or the input dtype", out_dtype);
  }
  if (ldx < K) return fail(NM_ERR_STRIDE, "ldx = %lld < K = %lld", (long long)ldx, (long long)K);
  if (ldy < R) return fail(NM_ERR_STRIDE, "ldy = %lld < R = %lld", (long long)ldy, (long long)R);
  // bounded before any product of sizes below, so no int64 product overflows
  if (ldx > kMaxElems || ldy > kMaxElems)
    return fail(NM_ERR_SHAPE, "leading dimension above 2^40 elements");
  if (R == 0 || T == 0) return ok();  // empty product: nothing to enqueue
  if (!values || !idx || !act || !Y || (want_perm && !perm))
    return fail(NM_ERR_NULL, "values, idx, act, Y%s must be non-NULL", want_perm ? ", perm" : "");
  if (ldx % ld_quantum(dtype))
    return fail(NM_ERR_ALIGN, "ldx = %lld is not a multiple of %lld", (long long)ldx,
                (long long)ld_quantum(dtype));
  if (!aligned16(values) || !aligned16(idx) || !aligned16(act) || !aligned16(Y) ||
      (want_perm && !aligned16(perm)))
    return fail(NM_ERR_ALIGN, "device pointers must be 16-byte aligned");
  if (T * ldx > kMaxElems || T * ldy > kMaxElems) return fail(NM_ERR_SHAPE, "T*ld too large");
  Sizes z = sizes_of(R, K, n, m, dtype);
  size_t ybytes = extent(T, R, ldy, elt_bytes(out_dtype));
  const size_t abytes = extent(T, K, ldx, elt_bytes(dtype));
  if (overlaps(Y, ybytes, values, z.values_bytes) || overlaps(Y, ybytes, idx, z.idx_bytes) ||
      overlaps(Y, ybytes, act, abytes) || (want_perm && overlaps(Y, ybytes, perm, size_t(K) * 4)))
    return fail(NM_ERR_ALIAS, "Y overlaps an input");
  if (static_ws) {
    // the library's own array: a size it cannot hold is refused (before any
    // HIP call); its address is looked up only once validation has passed
    const size_t need = nm::spmm_perm_gather_bytes(T, K, dtype);
    if (need > nm::kStaticWorkspaceBytes)
      return fail(NM_ERR_SHAPE, "T*K*2 = %zu bytes exceeds the static workspace (%zu bytes)", need,
                  nm::kStaticWorkspaceBytes);
    workspace = nullptr;
    workspace_bytes = 0;
    if (need > 0) {
      const hipError_t e = nm::static_workspace(&workspace);
      if (e != hipSuccess) return hip_status(e, "static workspace address");
      workspace_bytes = nm::kStaticWorkspaceBytes;
    }
  } else if (workspace_bytes == 0) {
    workspace = nullptr;
  }
  if (workspace && !static_ws) {
    if (!aligned16(workspace)) return fail(NM_ERR_ALIGN, "workspace must be 16-byte aligned");
    if (overlaps(workspace, workspace_bytes, Y, ybytes) || overlaps(workspace, workspace_bytes, act, abytes) ||
        overlaps(workspace, workspace_bytes, values, z.values_bytes) ||
        overlaps(workspace, workspace_bytes, idx, z.idx_bytes) ||
        (want_perm && overlaps(workspace, workspace_bytes, perm, size_t(K) * 4)))
      return fail(NM_ERR_ALIAS, "workspace overlaps an argument");
  }

  nm::SpmmArgs a;
  a.values = static_cast<const uint16_t*>(values);
  a.idx = idx;
  a.R = R;
  a.K = K;
  a.n = n;
  a.m = m;
  a.dtype = dtype;
  a.act = static_cast<const uint16_t*>(act);
  a.T = T;
  a.ldx = ldx;
  a.perm = want_perm ? perm : nullptr;
  a.Y = Y;
  a.ldy = ldy;
  a.out_dtype = out_dtype;
  a.idx_row_words = z.words;
  a.variant = variant;
  a.workspace = workspace;
  a.workspace_bytes = workspace_bytes;
  return hip_status(nm::launch_spmm(a, static_cast<hipStream_t>(stream)), "nm_spmm launch");
}

}  // namespace

namespace nm {
namespace {

std::mutex g_dev_mu;

int cached_attr(std::map<int, int>& cache, hipDeviceAttribute_t attr, int fallback) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return fallback;
  std::lock_guard<std::mutex> g(g_dev_mu);
  auto it = cache.find(dev);
  if (it != cache.end()) return it->second;
  int v = 0;
  if (hipDeviceGetAttribute(&v, attr, dev) != hipSuccess || v <= 0) v = fallback;
  cache[dev] = v;
  return v;
}

}  // namespace

int device_cu_count() {
  static std::map<int, int> cache;
  return cached_attr(cache, hipDeviceAttributeMultiprocessorCount, 256);
}

int device_max_lds() {
  static std::map<int, int> cache;
  return cached_attr(cache, hipDeviceAttributeMaxSharedMemoryPerBlock, 0);
}

hipError_t ensure_lds_limit(const void* kern, int bytes) {
  static std::set<std::pair<int, const void*>> done;
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  std::lock_guard<std::mutex> g(g_dev_mu);
  if (done.count({dev, kern})) return hipSuccess;
  e = hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess) done.insert({dev, kern});
  return e;
}

}  // namespace nm

extern "C" {

int nm_version(void) { return 201; }

const char* nm_status_string(int status) {
  switch (status) {
    case NM_OK: return "NM_OK";
    case NM_ERR_NULL: return "NM_ERR_NULL";
    case NM_ERR_SHAPE: return "NM_ERR_SHAPE";
    case NM_ERR_UNSUPPORTED: return "NM_ERR_UNSUPPORTED";
    case NM_ERR_STRIDE: return "NM_ERR_STRIDE";
    case NM_ERR_ALIAS: return "NM_ERR_ALIAS";
    case NM_ERR_HIP: return "NM_ERR_HIP";
    case NM_ERR_ALIGN: return "NM_ERR_ALIGN";
    default: return "NM_ERR_UNKNOWN";
  }
}

const char* nm_last_error(void) { return g_last_error.c_str(); }

nm_status nm_packed_sizes(int64_t R, int64_t K, int n, int m, int dtype, size_t* values_bytes,
                          size_t* idx_bytes, int64_t* idx_row_words) {
  nm_status st = check_format(R, K, n, m, dtype);
  if (st != NM_OK) return st;
  Sizes z = sizes_of(R, K, n, m, dtype);
  if (values_bytes) *values_bytes = z.values_bytes;
  if (idx_bytes) *idx_bytes = z.idx_bytes;
  if (idx_row_words) *idx_row_words = z.words;
  return ok();
}

nm_status nm_compress(const void* W, int64_t R, int64_t K, int64_t ldw, int dtype, int n, int m,
                      void* values, uint32_t* idx, void* stream) {
  nm_status st = check_format(R, K, n, m, dtype);
  if (st != NM_OK) return st;
  if (ldw < K) return fail(NM_ERR_STRIDE, "ldw = %lld < K = %lld", (long long)ldw, (long long)K);
  if (ldw > kMaxElems) return fail(NM_ERR_SHAPE, "ldw above 2^40 elements");
  if (R == 0) return ok();
  if (!W || !values || !idx) return fail(NM_ERR_NULL, "W, values and idx must be non-NULL");
  if (ldw % ld_quantum(dtype))
    return fail(NM_ERR_ALIGN, "ldw = %lld is not a multiple of %lld", (long long)ldw,
                (long long)ld_quantum(dtype));
  if (!aligned16(W) || !aligned16(values) || !aligned16(idx))
    return fail(NM_ERR_ALIGN, "device pointers must be 16-byte aligned");
  if (R * ldw > kMaxElems) return fail(NM_ERR_SHAPE, "R*ldw too large");
  Sizes z = sizes_of(R, K, n, m, dtype);
  size_t wbytes = extent(R, K, ldw, elt_bytes(dtype));
  if (overlaps(values, z.values_bytes, W, wbytes) || overlaps(idx, z.idx_bytes, W, wbytes) ||
      overlaps(values, z.values_bytes, idx, z.idx_bytes))
    return fail(NM_ERR_ALIAS, "outputs overlap each other or W");
  if (byte_type(dtype))
    return hip_status(nm::launch_prune_pack_i8(static_cast<const uint8_t*>(W), R, K, ldw,
                                               static_cast<uint8_t*>(values), idx, z.words,
                                               dtype == NM_FP8, static_cast<hipStream_t>(stream)),
                      "nm_compress launch");
  return hip_status(nm::launch_prune_pack(static_cast<const uint16_t*>(W), R, K, ldw, n, m,
                                          static_cast<uint16_t*>(values), idx, z.words,
                                          static_cast<hipStream_t>(stream)),
                    "nm_compress launch");
}

nm_status nm_decompress(const void* values, const uint32_t* idx, int64_t R, int64_t K, int n,
                        int m, int dtype, void* W_out, int64_t ldw, void* stream) {
  nm_status st = check_format(R, K, n, m, dtype);
  if (st != NM_OK) return st;
  if (ldw < K) return fail(NM_ERR_STRIDE, "ldw = %lld < K = %lld", (long long)ldw, (long long)K);
  if (ldw > kMaxElems) return fail(NM_ERR_SHAPE, "ldw above 2^40 elements");
  if (R == 0) return ok();
  if (!W_out || !values || !idx) return fail(NM_ERR_NULL, "values, idx and W_out must be non-NULL");
  if (ldw % ld_quantum(dtype))
    return fail(NM_ERR_ALIGN, "ldw = %lld is not a multiple of %lld", (long long)ldw,
                (long long)ld_quantum(dtype));
  if (!aligned16(W_out) || !aligned16(values) || !aligned16(idx))
    return fail(NM_ERR_ALIGN, "device pointers must be 16-byte aligned");
  if (R * ldw > kMaxElems) return fail(NM_ERR_SHAPE, "R*ldw too large");
  Sizes z = sizes_of(R, K, n, m, dtype);
  size_t wbytes = extent(R, K, ldw, elt_bytes(dtype));
  if (overlaps(W_out, wbytes, values, z.values_bytes) || overlaps(W_out, wbytes, idx, z.idx_bytes))
    return fail(NM_ERR_ALIAS, "W_out overlaps an input");
  if (byte_type(dtype))
    return hip_status(nm::launch_decompress_i8(static_cast<const uint8_t*>(values), idx, R, K, z.words,
                                               static_cast<uint8_t*>(W_out), ldw,
                                               static_cast<hipStream_t>(stream)),
                      "nm_decompress launch");
  return hip_status(nm::launch_decompress(static_cast<const uint16_t*>(values), idx, R, K, n, m,
                                          z.words, static_cast<uint16_t*>(W_out), ldw,
                                          static_cast<hipStream_t>(stream)),
                    "nm_decompress launch");
}

nm_status nm_spmm(const void* values, const uint32_t* idx, int64_t R, int64_t K, int n, int m,
                  int dtype, const void* act, int64_t T, int64_t ldx, void* Y, int64_t ldy,
                  int out_dtype, void* stream) {
  return spmm_common(values, idx, R, K, n, m, dtype, act, T, ldx, nullptr, false, Y, ldy,
                     out_dtype, nullptr, 0, 0, stream);
}

nm_status nm_spmm_perm_workspace_size(int64_t R, int64_t K, int64_t T, int n, int m, int dtype,
                                      size_t* bytes) {
  nm_status st = check_format(R, K, n, m, dtype);
  if (st != NM_OK) return st;
  if (T < 0 || T > kMaxRT) return fail(NM_ERR_SHAPE, "T = %lld out of range", (long long)T);
  if (!bytes) return fail(NM_ERR_NULL, "bytes must be non-NULL");
  *bytes = R == 0 ? 0 : nm::spmm_perm_gather_bytes(T, K, dtype);
  return ok();
}

nm_status nm_spmm_perm(const void* values, const uint32_t* idx, int64_t R, int64_t K, int n, int m,
                       int dtype, const void* act, int64_t T, int64_t ldx, const int32_t* perm,
                       void* Y, int64_t ldy, int out_dtype, void* workspace, size_t workspace_bytes,
                       void* stream) {
  return spmm_common(values, idx, R, K, n, m, dtype, act, T, ldx, perm, true, Y, ldy, out_dtype,
                     workspace, workspace_bytes, 0, stream);
}

nm_status nm_spmm_perm_static(const void* values, const uint32_t* idx, int64_t R, int64_t K, int n,
                              int m, int dtype, const void* act, int64_t T, int64_t ldx,
                              const int32_t* perm, void* Y, int64_t ldy, int out_dtype, void* stream) {
  return spmm_common(values, idx, R, K, n, m, dtype, act, T, ldx, perm, true, Y, ldy, out_dtype,
                     nullptr, 0, 0, stream, true);
}

nm_status nm_spmm_variant(const void* values, const uint32_t* idx, int64_t R, int64_t K, int n, int m,
                          int dtype, const void* act, int64_t T, int64_t ldx, const int32_t* perm,
                          void* Y, int64_t ldy, int out_dtype, void* workspace, size_t workspace_bytes,
                          int variant, void* stream) {
  return spmm_common(values, idx, R, K, n, m, dtype, act, T, ldx, perm, perm != nullptr, Y, ldy,
                     out_dtype, workspace, workspace_bytes, variant, stream);
}

nm_status nm_check_perm(const int32_t* perm, int64_t K, void* stream) {
  if (K < 1 || K > kMaxK) return fail(NM_ERR_SHAPE, "K = %lld out of range", (long long)K);
  if (!perm) return fail(NM_ERR_NULL, "perm must be non-NULL");
  std::vector<int32_t> host(static_cast<size_t>(K));
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = hipMemcpyAsync(host.data(), perm, size_t(K) * 4, hipMemcpyDeviceToHost, s);
  if (e == hipSuccess) e = hipStreamSynchronize(s);
  if (e != hipSuccess) return hip_status(e, "nm_check_perm copy");
  std::vector<char> seen(static_cast<size_t>(K), 0);
  for (int64_t k = 0; k < K; ++k) {
    int32_t p = host[size_t(k)];
    if (p < 0 || p >= K || seen[size_t(p)])
      return fail(NM_ERR_SHAPE, "perm[%lld] = %d breaks the permutation", (long long)k, p);
    seen[size_t(p)] = 1;
  }
  return ok();
}


// Shared checks of the training-side products: format, 16-bit types, output
// dtype, T and the G operand [T, R] (ldg).
static nm_status check_train(int64_t R, int64_t K, int n, int m, int dtype, int64_t T, int64_t ldg,
                             int out_dtype) {
  nm_status st = check_format(R, K, n, m, dtype);
  if (st != NM_OK) return st;
  if (dtype != NM_F16 && dtype != NM_BF16)
    return fail(NM_ERR_UNSUPPORTED, "training products take fp16 or bf16 weights");
  // whole 16-byte pieces of G's rows and whole 32-column segments of W's rows
  if (R % 8 || K % 32)
    return fail(NM_ERR_SHAPE, "training products need R %% 8 == 0 and K %% 32 == 0 (R = %lld, K = %lld)",
                (long long)R, (long long)K);
  if (out_dtype != NM_F32 && out_dtype != dtype)
    return fail(NM_ERR_UNSUPPORTED, "out_dtype %d must be NM_F32 or the input dtype", out_dtype);
  if (T < 0 || T > kMaxRT) return fail(NM_ERR_SHAPE, "T = %lld out of range", (long long)T);
  if (ldg < R) return fail(NM_ERR_STRIDE, "ldg = %lld < R = %lld", (long long)ldg, (long long)R);
  if (ldg > kMaxElems) return fail(NM_ERR_SHAPE, "ldg above 2^40 elements");
  return NM_OK;
}

nm_status nm_spmm_dx(const void* values, const uint32_t* idx, int64_t R, int64_t K, int n, int m, int dtype,
                     const void* G, int64_t T, int64_t ldg, void* dX, int64_t lddx, int out_dtype, void* stream) {
  nm_status st = check_train(R, K, n, m, dtype, T, ldg, out_dtype);
  if (st != NM_OK) return st;
  if (lddx < K) return fail(NM_ERR_STRIDE, "lddx = %lld < K = %lld", (long long)lddx, (long long)K);
  if (lddx > kMaxElems) return fail(NM_ERR_SHAPE, "lddx above 2^40 elements");
  if (T == 0) return ok();  // empty dX: nothing to enqueue (R == 0 writes zeros)
  if (!dX || (R > 0 && (!values || !idx || !G)))
    return fail(NM_ERR_NULL, "values, idx, G and dX must be non-NULL");
  if (ldg % 8) return fail(NM_ERR_ALIGN, "ldg = %lld is not a multiple of 8", (long long)ldg);
  if (!aligned16(values) || !aligned16(idx) || !aligned16(G) || !aligned16(dX))
    return fail(NM_ERR_ALIGN, "device pointers must be 16-byte aligned");
  if (T * ldg > kMaxElems || T * lddx > kMaxElems) return fail(NM_ERR_SHAPE, "T*ld too large");
  Sizes z = sizes_of(R, K, n, m, dtype);
  // the kernel's per-lane byte offsets are 32-bit: the packed arrays and a
  // 128-token block of G
  if (z.values_bytes >= (size_t(1) << 32) || z.idx_bytes >= (size_t(1) << 32) || 128 * ldg * 2 >= (int64_t(1) << 32))
    return fail(NM_ERR_SHAPE, "packed W of 4 GiB or more, or ldg of 2^24 or more");
  const size_t xbytes = extent(T, K, lddx, elt_bytes(out_dtype));
  const size_t gbytes = extent(T, R, ldg, 2);
  if (overlaps(dX, xbytes, values, z.values_bytes) || overlaps(dX, xbytes, idx, z.idx_bytes) ||
      overlaps(dX, xbytes, G, gbytes))
    return fail(NM_ERR_ALIAS, "dX overlaps an input");
  nm::TrainArgs a{};
  a.values = static_cast<const uint16_t*>(values);
  a.values_bytes = z.values_bytes;
  a.idx = idx;
  a.idx_bytes = z.idx_bytes;
  a.R = R;
  a.K = K;
  a.n = n;
  a.m = m;
  a.dtype = dtype;
  a.idx_row_words = z.words;
  a.G = static_cast<const uint16_t*>(G);
  a.T = T;
  a.ldg = ldg;
  a.out = dX;
  a.ldo = lddx;
  a.out_dtype = out_dtype;
  return hip_status(nm::launch_spmm_dx(a, static_cast<hipStream_t>(stream)), "nm_spmm_dx launch");
}

nm_status nm_spmm_dw(const uint32_t* idx, int64_t R, int64_t K, int n, int m, int dtype, const void* G, int64_t T,
                     int64_t ldg, const void* act, int64_t ldx, void* dW, int out_dtype, void* stream) {
  nm_status st = check_train(R, K, n, m, dtype, T, ldg, out_dtype);
  if (st != NM_OK) return st;
  if (ldx < K) return fail(NM_ERR_STRIDE, "ldx = %lld < K = %lld", (long long)ldx, (long long)K);
  if (ldx > kMaxElems) return fail(NM_ERR_SHAPE, "ldx above 2^40 elements");
  if (R == 0) return ok();  // no weights, no gradient (T == 0 writes zeros)
  if (!idx || !dW || (T > 0 && (!G || !act)))
    return fail(NM_ERR_NULL, "idx, G, act and dW must be non-NULL");
  if (ldg % 8 || ldx % 8) return fail(NM_ERR_ALIGN, "ldg and ldx must be multiples of 8");
  if (!aligned16(idx) || !aligned16(G) || !aligned16(act) || !aligned16(dW))
    return fail(NM_ERR_ALIGN, "device pointers must be 16-byte aligned");
  if (T * ldg > kMaxElems || T * ldx > kMaxElems) return fail(NM_ERR_SHAPE, "T*ld too large");
  // per-lane byte offsets are 32-bit: every token row of G and act
  if (T * ldg * 2 >= (int64_t(1) << 32) || T * ldx * 2 >= (int64_t(1) << 32))
    return fail(NM_ERR_SHAPE, "G or act of 4 GiB or more");
  Sizes z = sizes_of(R, K, n, m, dtype);
  if (z.idx_bytes >= (size_t(1) << 32)) return fail(NM_ERR_SHAPE, "index words of 4 GiB or more");
  const size_t wbytes = size_t(R) * size_t(z.S) * elt_bytes(out_dtype);
  const size_t gbytes = extent(T, R, ldg, 2), abytes = extent(T, K, ldx, 2);
  if (overlaps(dW, wbytes, idx, z.idx_bytes) || overlaps(dW, wbytes, G, gbytes) || overlaps(dW, wbytes, act, abytes))
    return fail(NM_ERR_ALIAS, "dW overlaps an input");
  nm::TrainArgs a{};
  a.idx = idx;
  a.idx_bytes = z.idx_bytes;
  a.R = R;
  a.K = K;
  a.n = n;
  a.m = m;
  a.dtype = dtype;
  a.idx_row_words = z.words;
  a.G = static_cast<const uint16_t*>(G);
  a.T = T;
  a.ldg = ldg;
  a.act = static_cast<const uint16_t*>(act);
  a.ldx = ldx;
  a.out = dW;
  a.out_dtype = out_dtype;
  return hip_status(nm::launch_spmm_dw(a, static_cast<hipStream_t>(stream)), "nm_spmm_dw launch");
}

nm_status nm_hybrid_layout(int64_t R, int64_t K, int64_t tile_rows, int64_t tile_cols, const uint8_t* flags,
                           int64_t* tile_meta, int64_t* row_meta, int64_t* values_count, int64_t* idx_bytes) {
  nm_status st = check_hybrid_grid(R, K, tile_rows, tile_cols);
  if (st != NM_OK) return st;
  const int64_t RB = (R + tile_rows - 1) / tile_rows, KB = K / tile_cols;
  if (R > 0 && !flags) return fail(NM_ERR_NULL, "flags must be non-NULL");
  for (int64_t t = 0; t < RB * KB; ++t)
    if (flags[t] > 1)
      return fail(NM_ERR_SHAPE, "flag %lld is %d: flags are 0 (2:4) or 1 (dense)", (long long)t, int(flags[t]));
  int64_t vbase = 0, ibase = 0;
  for (int64_t b = 0; b < RB; ++b) {
    int64_t v = 0, i = 0;  // position along the first row of tile-row b
    for (int64_t j = 0; j < KB; ++j) {
      const bool dense = flags[b * KB + j] != 0;
      if (tile_meta) {
        tile_meta[(b * KB + j) * 2] = vbase + v;
        tile_meta[(b * KB + j) * 2 + 1] = dense ? -1 : ibase + i;
      }
      v += dense ? tile_cols : tile_cols / 2;
      i += dense ? 0 : tile_cols / 8;
    }
    if (row_meta) {
      row_meta[b * 4] = v;
      row_meta[b * 4 + 1] = i;
      row_meta[b * 4 + 2] = vbase;
      row_meta[b * 4 + 3] = ibase;
    }
    const int64_t rows = (b + 1) * tile_rows <= R ? tile_rows : R - b * tile_rows;
    vbase += rows * v;
    ibase += rows * i;
  }
  ibase = (ibase + 15) / 16 * 16;  // whole 16-byte blocks (zero padding)
  st = check_hybrid_totals(vbase, ibase);
  if (st != NM_OK) return st;
  if (values_count) *values_count = vbase;
  if (idx_bytes) *idx_bytes = ibase;
  return ok();
}

nm_status nm_hybrid_compress(const void* W, int64_t R, int64_t K, int64_t ldw, int dtype, int64_t tile_rows,
                             int64_t tile_cols, const int64_t* tile_meta, const int64_t* row_meta,
                             int64_t values_count, int64_t idx_bytes, void* values, uint8_t* idx, void* stream) {
  if (dtype != NM_F16 && dtype != NM_BF16)
    return fail(NM_ERR_UNSUPPORTED, "hybrid tiles take NM_F16 or NM_BF16 weights, not dtype %d", dtype);
  nm_status st = check_hybrid_grid(R, K, tile_rows, tile_cols);
  if (st != NM_OK) return st;
  st = check_hybrid_totals(values_count, idx_bytes);
  if (st != NM_OK) return st;
  if (ldw < K) return fail(NM_ERR_STRIDE, "ldw = %lld < K = %lld", (long long)ldw, (long long)K);
  if (ldw > kMaxElems) return fail(NM_ERR_SHAPE, "ldw above 2^40 elements");
  if (R == 0) return ok();
  if (!W || !values || !tile_meta || !row_meta || (idx_bytes > 0 && !idx))
    return fail(NM_ERR_NULL, "W, values, tile_meta, row_meta (and idx with 2:4 tiles) must be non-NULL");
  if (ldw % 8) return fail(NM_ERR_ALIGN, "ldw = %lld is not a multiple of 8", (long long)ldw);
  if (!aligned16(W) || !aligned16(values) || (idx && !aligned16(idx)) || !aligned8(tile_meta) ||
      !aligned8(row_meta))
    return fail(NM_ERR_ALIGN, "W, values and idx must be 16-byte aligned, the layout tables 8-byte aligned");
  if (R * ldw > kMaxElems) return fail(NM_ERR_SHAPE, "R*ldw too large");
  const int64_t RB = (R + tile_rows - 1) / tile_rows, KB = K / tile_cols;
  const size_t wbytes = extent(R, K, ldw, 2), vbytes = size_t(values_count) * 2, ib = size_t(idx_bytes);
  const size_t tmb = size_t(RB * KB) * 16, rmb = size_t(RB) * 32;
  if (overlaps(values, vbytes, W, wbytes) || overlaps(idx, ib, W, wbytes) || overlaps(values, vbytes, idx, ib) ||
      overlaps(values, vbytes, tile_meta, tmb) || overlaps(values, vbytes, row_meta, rmb) ||
      overlaps(idx, ib, tile_meta, tmb) || overlaps(idx, ib, row_meta, rmb))
    return fail(NM_ERR_ALIAS, "outputs overlap each other, W or the layout tables");
  nm::HybridArgs a;
  a.W = static_cast<const uint16_t*>(W);
  a.ldw = ldw;
  a.R = R;
  a.K = K;
  a.tile_rows = tile_rows;
  a.tile_cols = tile_cols;
  a.dtype = dtype;
  a.tile_meta = tile_meta;
  a.row_meta = row_meta;
  a.values_out = static_cast<uint16_t*>(values);
  a.idx_out = idx;
  a.values_bytes = vbytes;
  a.idx_bytes = ib;
  return hip_status(nm::launch_hybrid_pack(a, static_cast<hipStream_t>(stream)), "nm_hybrid_compress launch");
}

nm_status nm_hybrid_spmm(const void* values, const uint8_t* idx, const int64_t* tile_meta, const int64_t* row_meta,
                         int64_t R, int64_t K, int64_t tile_rows, int64_t tile_cols, int64_t values_count,
                         int64_t idx_bytes, int dtype, const void* act, int64_t T, int64_t ldx, void* Y,
                         int64_t ldy, int out_dtype, void* stream) {
  if (dtype != NM_F16 && dtype != NM_BF16)
    return fail(NM_ERR_UNSUPPORTED, "hybrid tiles take NM_F16 or NM_BF16 weights, not dtype %d", dtype);
  if (out_dtype != NM_F32 && out_dtype != dtype)
    return fail(NM_ERR_UNSUPPORTED, "out_dtype %d must be NM_F32 or the input dtype", out_dtype);
  nm_status st = check_hybrid_grid(R, K, tile_rows, tile_cols);
  if (st != NM_OK) return st;
  st = check_hybrid_totals(values_count, idx_bytes);
  if (st != NM_OK) return st;
  if (T < 0 || T > kMaxRT) return fail(NM_ERR_SHAPE, "T = %lld out of range", (long long)T);
  if (ldx < K) return fail(NM_ERR_STRIDE, "ldx = %lld < K = %lld", (long long)ldx, (long long)K);
  if (ldy < R) return fail(NM_ERR_STRIDE, "ldy = %lld < R = %lld", (long long)ldy, (long long)R);
  if (ldx > kMaxElems || ldy > kMaxElems) return fail(NM_ERR_SHAPE, "leading dimension above 2^40 elements");
  if (ldx > (int64_t(1) << 22))
    return fail(NM_ERR_SHAPE, "ldx = %lld above 2^22 (a token tile's offsets are 31-bit)", (long long)ldx);
  if (R == 0 || T == 0) return ok();
  if (!values || !tile_meta || !row_meta || !act || !Y || (idx_bytes > 0 && !idx))
    return fail(NM_ERR_NULL, "values, tile_meta, row_meta, act, Y (and idx with 2:4 tiles) must be non-NULL");
  if (ldx % 8) return fail(NM_ERR_ALIGN, "ldx = %lld is not a multiple of 8", (long long)ldx);
  if (!aligned16(values) || (idx && !aligned16(idx)) || !aligned16(act) || !aligned16(Y) ||
      !aligned8(tile_meta) || !aligned8(row_meta))
    return fail(NM_ERR_ALIGN, "values, idx, act and Y must be 16-byte aligned, the layout tables 8-byte aligned");
  if (T * ldx > kMaxElems || T * ldy > kMaxElems) return fail(NM_ERR_SHAPE, "T*ld too large");
  const int64_t RB = (R + tile_rows - 1) / tile_rows, KB = K / tile_cols;
  const size_t ybytes = extent(T, R, ldy, elt_bytes(out_dtype)), abytes = extent(T, K, ldx, 2);
  const size_t vbytes = size_t(values_count) * 2, ib = size_t(idx_bytes);
  if (overlaps(Y, ybytes, values, vbytes) || overlaps(Y, ybytes, idx, ib) || overlaps(Y, ybytes, act, abytes) ||
      overlaps(Y, ybytes, tile_meta, size_t(RB * KB) * 16) || overlaps(Y, ybytes, row_meta, size_t(RB) * 32))
    return fail(NM_ERR_ALIAS, "Y overlaps an input");
  nm::HybridArgs a;
  a.values = static_cast<const uint16_t*>(values);
  a.idx = idx;
  a.tile_meta = tile_meta;
  a.row_meta = row_meta;
  a.R = R;
  a.K = K;
  a.tile_rows = tile_rows;
  a.tile_cols = tile_cols;
  a.dtype = dtype;
  a.values_bytes = vbytes;
  a.idx_bytes = ib;
  a.act = static_cast<const uint16_t*>(act);
  a.T = T;
  a.ldx = ldx;
  a.Y = Y;
  a.ldy = ldy;
  a.out_dtype = out_dtype;
  return hip_status(nm::launch_hybrid_spmm(a, static_cast<hipStream_t>(stream)), "nm_hybrid_spmm launch");
}

// ---------------------------------------------------------------------------
// Block-sparse and diagonal-sparse structures with the column permutation
// ---------------------------------------------------------------------------
static nm_status check_block_shape(int64_t R, int64_t K) {
  if (R < 0 || R > kMaxRT || R % 32)
    return fail(NM_ERR_SHAPE, "R = %lld must be a multiple of 32 in [0, 2^30]", (long long)R);
  if (K < 32 || K > kMaxK || K % 32)
    return fail(NM_ERR_SHAPE, "K = %lld must be a multiple of 32 in [32, 2^24]", (long long)K);
  return NM_OK;
}

static nm_status check_host_product(int dtype, int out_dtype, int64_t R, int64_t K, int64_t T, int64_t ldx,
                                    int64_t ldy) {
  if (dtype != NM_F16 && dtype != NM_BF16)
    return fail(NM_ERR_UNSUPPORTED, "block / diagonal products take NM_F16 or NM_BF16, not dtype %d", dtype);
  if (out_dtype != NM_F32 && out_dtype != dtype)
    return fail(NM_ERR_UNSUPPORTED, "out_dtype %d must be NM_F32 or the input dtype", out_dtype);
  if (T < 0 || T > kMaxRT) return fail(NM_ERR_SHAPE, "T = %lld out of range", (long long)T);
  if (ldx < K) return fail(NM_ERR_STRIDE, "ldx = %lld < K = %lld", (long long)ldx, (long long)K);
  if (ldy < R) return fail(NM_ERR_STRIDE, "ldy = %lld < R = %lld", (long long)ldy, (long long)R);
  if (ldx > kMaxElems || ldy > kMaxElems) return fail(NM_ERR_SHAPE, "leading dimension above 2^40 elements");
  if (T * ldx > kMaxElems || T * ldy > kMaxElems) return fail(NM_ERR_SHAPE, "T*ld too large");
  if (int64_t(extent(T, K, ldx, 2)) >= (int64_t(1) << 32))
    return fail(NM_ERR_SHAPE, "act of 4 GiB or more (its reads use 32-bit offsets)");
  return NM_OK;
}

nm_status nm_block_structure(int64_t R, int64_t K, const uint8_t* mask, int32_t* row_ptr, int32_t* col,
                             int64_t* nnzb) {
  nm_status st = check_block_shape(R, K);
  if (st != NM_OK) return st;
  const int64_t RB = R / 32, KB = K / 32;
  if (RB * KB > 0 && !mask) return fail(NM_ERR_NULL, "mask must be non-NULL");
  int64_t n = 0;
  for (int64_t b = 0; b < RB; ++b) {
    if (row_ptr) row_ptr[b] = int32_t(n);
    for (int64_t c = 0; c < KB; ++c) {
      const uint8_t f = mask[b * KB + c];
      if (f > 1) return fail(NM_ERR_SHAPE, "mask[%lld] = %d is neither 0 nor 1", (long long)(b * KB + c), f);
      if (f) {
        if (col) col[n] = int32_t(c);
        ++n;
      }
    }
  }
  if (n > (int64_t(1) << 21)) return fail(NM_ERR_SHAPE, "more than 2^21 kept blocks (values of 4 GiB)");
  if (row_ptr) row_ptr[RB] = int32_t(n);
  if (nnzb) *nnzb = n;
  return ok();
}

nm_status nm_block_compress(const void* W, int64_t R, int64_t K, int64_t ldw, int dtype, const int32_t* row_ptr,
                            const int32_t* col, int64_t nnzb, void* values, void* stream) {
  if (dtype != NM_F16 && dtype != NM_BF16)
    return fail(NM_ERR_UNSUPPORTED, "block structures take NM_F16 or NM_BF16 weights, not dtype %d", dtype);
  nm_status st = check_block_shape(R, K);
  if (st != NM_OK) return st;
  if (nnzb < 0 || nnzb > (R / 32) * (K / 32))
    return fail(NM_ERR_SHAPE, "nnzb = %lld outside [0, blocks of W]", (long long)nnzb);
  if (ldw < K) return fail(NM_ERR_STRIDE, "ldw = %lld < K = %lld", (long long)ldw, (long long)K);
  if (ldw > kMaxElems || R * ldw > kMaxElems) return fail(NM_ERR_SHAPE, "R*ldw too large");
  if (R == 0 || nnzb == 0) return ok();
  if (!W || !row_ptr || !col || !values) return fail(NM_ERR_NULL, "W, row_ptr, col and values must be non-NULL");
  if (ldw % 8) return fail(NM_ERR_ALIGN, "ldw = %lld is not a multiple of 8", (long long)ldw);
  if (!aligned16(W) || !aligned16(values) || !aligned16(row_ptr) || !aligned16(col))
    return fail(NM_ERR_ALIGN, "device pointers must be 16-byte aligned");
  const size_t vbytes = size_t(nnzb) * 2048;
  if (overlaps(values, vbytes, W, extent(R, K, ldw, 2)) || overlaps(values, vbytes, row_ptr, size_t(R / 32 + 1) * 4) ||
      overlaps(values, vbytes, col, size_t(nnzb) * 4))
    return fail(NM_ERR_ALIAS, "values overlaps an input");
  return hip_status(nm::launch_block_pack(static_cast<const uint16_t*>(W), ldw, R, K, row_ptr, col, nnzb,
                                          static_cast<uint16_t*>(values), static_cast<hipStream_t>(stream)),
                    "nm_block_compress launch");
}

nm_status nm_block_spmm(const void* values, const int32_t* row_ptr, const int32_t* col, int64_t nnzb, int64_t R,
                        int64_t K, int dtype, const void* act, int64_t T, int64_t ldx, const int32_t* perm,
                        void* Y, int64_t ldy, int out_dtype, void* stream) {
  nm_status st = check_block_shape(R, K);
  if (st != NM_OK) return st;
  st = check_host_product(dtype, out_dtype, R, K, T, ldx, ldy);
  if (st != NM_OK) return st;
  if (nnzb < 0 || nnzb > (R / 32) * (K / 32))
    return fail(NM_ERR_SHAPE, "nnzb = %lld outside [0, blocks of W]", (long long)nnzb);
  if (R == 0 || T == 0) return ok();
  if (!row_ptr || !act || !Y || (nnzb > 0 && (!values || !col)))
    return fail(NM_ERR_NULL, "row_ptr, act, Y (and values, col with kept blocks) must be non-NULL");
  if (ldx % 8) return fail(NM_ERR_ALIGN, "ldx = %lld is not a multiple of 8", (long long)ldx);
  if ((values && !aligned16(values)) || !aligned16(row_ptr) || (col && !aligned16(col)) || !aligned16(act) ||
      !aligned16(Y) || (perm && !aligned16(perm)))
    return fail(NM_ERR_ALIGN, "device pointers must be 16-byte aligned");
  const size_t ybytes = extent(T, R, ldy, elt_bytes(out_dtype)), abytes = extent(T, K, ldx, 2);
  const size_t vbytes = size_t(nnzb) * 2048;
  if (overlaps(Y, ybytes, values, vbytes) || overlaps(Y, ybytes, act, abytes) ||
      overlaps(Y, ybytes, row_ptr, size_t(R / 32 + 1) * 4) || overlaps(Y, ybytes, col, size_t(nnzb) * 4) ||
      overlaps(Y, ybytes, perm, perm ? size_t(K) * 4 : 0))
    return fail(NM_ERR_ALIAS, "Y overlaps an input");
  nm::HostArgs a;
  a.diagonal = false;
  a.values = static_cast<const uint16_t*>(values);
  a.values_bytes = vbytes;
  a.row_ptr = row_ptr;
  a.col = col;
  a.nnz = nnzb;
  a.R = R;
  a.K = K;
  a.dtype = dtype;
  a.act = static_cast<const uint16_t*>(act);
  a.act_bytes = abytes;
  a.ldx = ldx;
  a.T = T;
  a.perm = perm;
  a.out = Y;
  a.ldy = ldy;
  a.out_dtype = out_dtype;
  return hip_status(nm::launch_host_spmm(a, static_cast<hipStream_t>(stream)), "nm_block_spmm launch");
}

static nm_status check_diag_shape(int64_t R, int64_t K, int64_t D) {
  if (R < 0 || R > kMaxRT) return fail(NM_ERR_SHAPE, "R = %lld out of range", (long long)R);
  if (K < 8 || K > nm::kDiagMaxK || K % 8)
    return fail(NM_ERR_SHAPE, "K = %lld must be a multiple of 8 in [8, %lld]", (long long)K,
                (long long)nm::kDiagMaxK);
  if (D < 0 || D > K) return fail(NM_ERR_SHAPE, "D = %lld outside [0, K]", (long long)D);
  if (D * R * 2 >= (int64_t(1) << 32)) return fail(NM_ERR_SHAPE, "values of 4 GiB or more (32-bit offsets)");
  return NM_OK;
}

nm_status nm_diag_compress(const void* W, int64_t R, int64_t K, int64_t ldw, int dtype, const int32_t* offsets,
                           int64_t D, void* values, void* stream) {
  if (dtype != NM_F16 && dtype != NM_BF16)
    return fail(NM_ERR_UNSUPPORTED, "diagonal structures take NM_F16 or NM_BF16 weights, not dtype %d", dtype);
  nm_status st = check_diag_shape(R, K, D);
  if (st != NM_OK) return st;
  if (ldw < K) return fail(NM_ERR_STRIDE, "ldw = %lld < K = %lld", (long long)ldw, (long long)K);
  if (ldw > kMaxElems || R * ldw > kMaxElems) return fail(NM_ERR_SHAPE, "R*ldw too large");
  if (R == 0 || D == 0) return ok();
  if (!W || !offsets || !values) return fail(NM_ERR_NULL, "W, offsets and values must be non-NULL");
  if (!aligned16(W) || !aligned16(values) || !aligned16(offsets))
    return fail(NM_ERR_ALIGN, "device pointers must be 16-byte aligned");
  const size_t vbytes = size_t(D) * size_t(R) * 2;
  if (overlaps(values, vbytes, W, extent(R, K, ldw, 2)) || overlaps(values, vbytes, offsets, size_t(D) * 4))
    return fail(NM_ERR_ALIAS, "values overlaps an input");
  return hip_status(nm::launch_diag_pack(static_cast<const uint16_t*>(W), ldw, R, K, offsets, D,
                                         static_cast<uint16_t*>(values), static_cast<hipStream_t>(stream)),
                    "nm_diag_compress launch");
}

nm_status nm_diag_spmm(const void* values, const int32_t* offsets, int64_t D, int64_t R, int64_t K, int dtype,
                       const void* act, int64_t T, int64_t ldx, const int32_t* perm, void* Y, int64_t ldy,
                       int out_dtype, void* stream) {
  nm_status st = check_diag_shape(R, K, D);
  if (st != NM_OK) return st;
  st = check_host_product(dtype, out_dtype, R, K, T, ldx, ldy);
  if (st != NM_OK) return st;
  if (R == 0 || T == 0) return ok();
  if (!act || !Y || (D > 0 && (!values || !offsets)))
    return fail(NM_ERR_NULL, "act, Y (and values, offsets with D > 0) must be non-NULL");
  if (ldx % 8) return fail(NM_ERR_ALIGN, "ldx = %lld is not a multiple of 8", (long long)ldx);
  if ((values && !aligned16(values)) || (offsets && !aligned16(offsets)) || !aligned16(act) || !aligned16(Y) ||
      (perm && !aligned16(perm)))
    return fail(NM_ERR_ALIGN, "device pointers must be 16-byte aligned");
  const size_t ybytes = extent(T, R, ldy, elt_bytes(out_dtype)), abytes = extent(T, K, ldx, 2);
  if (overlaps(Y, ybytes, values, size_t(D) * size_t(R) * 2) || overlaps(Y, ybytes, act, abytes) ||
      overlaps(Y, ybytes, offsets, size_t(D) * 4) || overlaps(Y, ybytes, perm, perm ? size_t(K) * 4 : 0))
    return fail(NM_ERR_ALIAS, "Y overlaps an input");
  nm::HostArgs a;
  a.diagonal = true;
  a.values = static_cast<const uint16_t*>(values);
  a.values_bytes = size_t(D) * size_t(R) * 2;
  a.offsets = offsets;
  a.nnz = D;
  a.R = R;
  a.K = K;
  a.dtype = dtype;
  a.act = static_cast<const uint16_t*>(act);
  a.act_bytes = abytes;
  a.ldx = ldx;
  a.T = T;
  a.perm = perm;
  a.out = Y;
  a.ldy = ldy;
  a.out_dtype = out_dtype;
  return hip_status(nm::launch_host_spmm(a, static_cast<hipStream_t>(stream)), "nm_diag_spmm launch");
}

// Shared checks of layer norm: a 16-bit or fp32 matrix [T, H].
static nm_status check_norm(int64_t T, int64_t H, int dtype) {
  if (dtype != NM_F16 && dtype != NM_BF16 && dtype != NM_F32)
    return fail(NM_ERR_UNSUPPORTED, "layer norm takes NM_F16, NM_BF16 or NM_F32, not dtype %d", dtype);
  if (T < 0 || T > kMaxRT) return fail(NM_ERR_SHAPE, "T = %lld out of range", (long long)T);
  if (H < 1 || H > kMaxK) return fail(NM_ERR_SHAPE, "H = %lld out of range [1, 2^24]", (long long)H);
  return NM_OK;
}

// A leading dimension of a [T, W] matrix.
static nm_status check_ld(const char* name, int64_t ld, int64_t T, int64_t W) {
  if (ld < W) return fail(NM_ERR_STRIDE, "%s = %lld < %lld", name, (long long)ld, (long long)W);
  if (ld > kMaxElems || T * ld > kMaxElems) return fail(NM_ERR_SHAPE, "T*%s too large", name);
  return NM_OK;
}

static bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

nm_status nm_layernorm(const void* x, int64_t T, int64_t H, int64_t ldx, int dtype, const void* weight,
                       const void* bias, float eps, void* y, int64_t ldy, float* mean, float* rstd, void* stream) {
  nm_status st = check_norm(T, H, dtype);
  if (st != NM_OK) return st;
  if (!(eps >= 0.f)) return fail(NM_ERR_SHAPE, "eps = %g is negative or not a number", double(eps));
  if ((st = check_ld("ldx", ldx, T, H)) != NM_OK || (st = check_ld("ldy", ldy, T, H)) != NM_OK) return st;
  if (T == 0) return ok();
  if (!x || !y) return fail(NM_ERR_NULL, "x and y must be non-NULL");
  if (!mean != !rstd) return fail(NM_ERR_NULL, "mean and rstd go together");
  const size_t e = elt_bytes(dtype);
  if (!aligned_to(x, e) || !aligned_to(y, e) || !aligned_to(weight, e) || !aligned_to(bias, e) ||
      !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return fail(NM_ERR_ALIGN, "a pointer is not aligned to its element");
  const size_t xb = extent(T, H, ldx, e), yb = extent(T, H, ldy, e), wb = size_t(H) * e, sb = size_t(T) * 4;
  const void* outs[3] = {y, mean, rstd};
  const size_t outb[3] = {yb, sb, sb};
  for (int i = 0; i < 3; ++i) {
    if (overlaps(outs[i], outb[i], x, xb) || overlaps(outs[i], outb[i], weight, wb) ||
        overlaps(outs[i], outb[i], bias, wb))
      return fail(NM_ERR_ALIAS, "an output overlaps an input");
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], outb[i], outs[j], outb[j])) return fail(NM_ERR_ALIAS, "outputs overlap each other");
  }
  nm::LayerNormArgs a;
  a.T = T;
  a.H = H;
  a.dtype = dtype;
  a.x = x;
  a.ldx = ldx;
  a.weight = weight;
  a.bias = bias;
  a.eps = eps;
  a.y = y;
  a.ldy = ldy;
  a.mean_out = mean;
  a.rstd_out = rstd;
  return hip_status(nm::launch_layernorm(a, static_cast<hipStream_t>(stream)), "nm_layernorm launch");
}

nm_status nm_layernorm_bwd_workspace_size(int64_t T, int64_t H, size_t* bytes) {
  nm_status st = check_norm(T, H, NM_F32);
  if (st != NM_OK) return st;
  if (!bytes) return fail(NM_ERR_NULL, "bytes must be non-NULL");
  *bytes = nm::layernorm_bwd_workspace(T, H);
  return ok();
}

nm_status nm_layernorm_bwd(const void* dy, int64_t ldg, const void* x, int64_t ldx, int64_t T, int64_t H, int dtype,
                           const float* mean, const float* rstd, const void* weight, void* dx, int64_t lddx, void* dw,
                           void* db, int out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  nm_status st = check_norm(T, H, dtype);
  if (st != NM_OK) return st;
  if (out_dtype != NM_F32 && out_dtype != dtype)
    return fail(NM_ERR_UNSUPPORTED, "out_dtype %d must be NM_F32 or the input dtype", out_dtype);
  if ((st = check_ld("ldg", ldg, T, H)) != NM_OK || (st = check_ld("ldx", ldx, T, H)) != NM_OK ||
      (st = check_ld("lddx", lddx, T, H)) != NM_OK)
    return st;
  const bool sums = dw || db;
  if (T == 0 && !sums) return ok();
  if (T > 0 && (!dy || !x || !mean || !rstd || !dx))
    return fail(NM_ERR_NULL, "dy, x, mean, rstd and dx must be non-NULL");
  const size_t need = sums ? nm::layernorm_bwd_workspace(T, H) : 0;
  if (need > 0 && !workspace) return fail(NM_ERR_NULL, "dw and db need a workspace");
  if (workspace_bytes < need)
    return fail(NM_ERR_SHAPE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  const size_t e = elt_bytes(dtype), o = elt_bytes(out_dtype);
  if (!aligned_to(dy, e) || !aligned_to(x, e) || !aligned_to(dx, e) || !aligned_to(weight, e) ||
      !aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(dw, o) || !aligned_to(db, o))
    return fail(NM_ERR_ALIGN, "a pointer is not aligned to its element");
  if (need > 0 && !aligned16(workspace)) return fail(NM_ERR_ALIGN, "workspace must be 16-byte aligned");
  const void* ins[5] = {dy, x, mean, rstd, weight};
  const size_t inb[5] = {extent(T, H, ldg, e), extent(T, H, ldx, e), size_t(T) * 4, size_t(T) * 4, size_t(H) * e};
  const void* outs[4] = {dx, dw, db, need ? workspace : nullptr};
  const size_t outb[4] = {extent(T, H, lddx, e), size_t(H) * o, size_t(H) * o, need};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 5; ++j)
      if (overlaps(outs[i], outb[i], ins[j], inb[j])) return fail(NM_ERR_ALIAS, "an output overlaps an input");
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], outb[i], outs[j], outb[j])) return fail(NM_ERR_ALIAS, "outputs overlap each other");
  }
  nm::LayerNormArgs a;
  a.T = T;
  a.H = H;
  a.dtype = dtype;
  a.x = x;
  a.ldx = ldx;
  a.weight = weight;
  a.dy = dy;
  a.ldg = ldg;
  a.mean = mean;
  a.rstd = rstd;
  a.dx = dx;
  a.lddx = lddx;
  a.dw = dw;
  a.db = db;
  a.out_dtype = out_dtype;
  a.workspace = workspace;
  return hip_status(nm::launch_layernorm_bwd(a, static_cast<hipStream_t>(stream)), "nm_layernorm_bwd launch");
}

// Shared checks of the adapters: the packed weight (16-bit), the token count,
// the adapters' sizes and the output type.
static nm_status check_adapter(int64_t R, int64_t K, int n, int m, int dtype, int64_t T, int64_t adapters,
                               int64_t rank, int out_dtype) {
  nm_status st = check_format(R, K, n, m, dtype);
  if (st != NM_OK) return st;
  if (dtype != NM_F16 && dtype != NM_BF16) return fail(NM_ERR_UNSUPPORTED, "adapters take fp16 or bf16 weights");
  if (out_dtype != NM_F32 && out_dtype != dtype)
    return fail(NM_ERR_UNSUPPORTED, "out_dtype %d must be NM_F32 or the input dtype", out_dtype);
  if (T < 0 || T > nm::kAdapterMaxTokens)
    return fail(NM_ERR_SHAPE, "T = %lld out of range [0, 2^24]", (long long)T);
  if (R > nm::kAdapterMaxWidth || K > nm::kAdapterMaxWidth)
    return fail(NM_ERR_SHAPE, "R = %lld or K = %lld above 2^22", (long long)R, (long long)K);
  if (rank < 1 || rank > nm::kAdapterMaxRank)
    return fail(NM_ERR_SHAPE, "rank = %lld out of range [1, %lld]", (long long)rank, (long long)nm::kAdapterMaxRank);
  if (adapters < 0 || adapters > nm::kAdapterMaxCount)
    return fail(NM_ERR_SHAPE, "adapters = %lld out of range [0, %lld]", (long long)adapters,
                (long long)nm::kAdapterMaxCount);
  return NM_OK;
}

static nm::SpmmArgs adapter_base(int64_t R, int64_t K, int n, int m, int dtype, int64_t T, int64_t ldx,
                                 int out_dtype) {
  nm::SpmmArgs b{};
  b.R = R;
  b.K = K;
  b.n = n;
  b.m = m;
  b.dtype = dtype;
  b.T = T;
  b.ldx = ldx;
  b.out_dtype = out_dtype;
  b.idx_row_words = sizes_of(R, K, n, m, dtype).words;
  return b;
}

nm_status nm_adapter_spmm_workspace_size(int64_t R, int64_t K, int n, int m, int dtype, int64_t T, int64_t ldx,
                                         int64_t adapters, int64_t rank, int out_dtype, size_t* bytes) {
  nm_status st = check_adapter(R, K, n, m, dtype, T, adapters, rank, out_dtype);
  if (st != NM_OK) return st;
  if (!bytes) return fail(NM_ERR_NULL, "bytes must be non-NULL");
  nm::SpmmArgs b = adapter_base(R, K, n, m, dtype, T, ldx, out_dtype);
  *bytes = T == 0 ? 0 : nm::adapter_workspace(b, rank);
  return ok();
}

nm_status nm_adapter_spmm(const void* values, const uint32_t* idx, int64_t R, int64_t K, int n, int m, int dtype,
                          const void* act, int64_t T, int64_t ldx, const int32_t* adapter, const void* A,
                          const void* B, const float* scale, int64_t adapters, int64_t rank, float* xa, void* Y,
                          int64_t ldy, int out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  nm_status st = check_adapter(R, K, n, m, dtype, T, adapters, rank, out_dtype);
  if (st != NM_OK) return st;
  if ((st = check_ld("ldx", ldx, T, K)) != NM_OK || (st = check_ld("ldy", ldy, T, R)) != NM_OK) return st;
  if (ldx >= (int64_t(1) << 24)) return fail(NM_ERR_SHAPE, "ldx of 2^24 or more");
  if (T == 0) return ok();
  if (!act || !adapter || !xa || (R > 0 && (!values || !idx || !Y)) || (adapters > 0 && (!A || !scale)) ||
      (adapters > 0 && R > 0 && !B))
    return fail(NM_ERR_NULL, "values, idx, act, adapter, A, B, scale, xa and Y must be non-NULL");
  if (ldx % 8) return fail(NM_ERR_ALIGN, "ldx = %lld is not a multiple of 8", (long long)ldx);
  if (!aligned16(values) || !aligned16(idx) || !aligned16(act) || !aligned16(Y) || !aligned16(A) || !aligned16(B) ||
      !aligned16(xa) || !aligned16(workspace) || !aligned_to(adapter, 4) || !aligned_to(scale, 4))
    return fail(NM_ERR_ALIGN, "device pointers must be 16-byte aligned (adapter and scale: 4)");
  nm::AdapterArgs a;
  a.base = adapter_base(R, K, n, m, dtype, T, ldx, out_dtype);
  const size_t need = nm::adapter_workspace(a.base, rank);
  if (need > 0 && !workspace) return fail(NM_ERR_NULL, "workspace must be non-NULL");
  if (workspace_bytes < need)
    return fail(NM_ERR_SHAPE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  const Sizes z = sizes_of(R, K, n, m, dtype);
  const size_t ab = size_t(adapters) * size_t(rank) * size_t(K) * 2, bb = size_t(adapters) * size_t(rank) * size_t(R) * 2;
  const Span in[] = {{values, z.values_bytes}, {idx, z.idx_bytes}, {act, extent(T, K, ldx, 2)},
                     {adapter, size_t(T) * 4}, {A, ab}, {B, bb}, {scale, size_t(adapters) * 4}};
  const Span out[] = {{Y, extent(T, R, ldy, elt_bytes(out_dtype))}, {xa, size_t(T) * size_t(rank) * 4},
                      {workspace, need}};
  if ((st = check_alias(in, out)) != NM_OK) return st;
  a.base.values = static_cast<const uint16_t*>(values);
  a.base.idx = idx;
  a.base.act = static_cast<const uint16_t*>(act);
  a.base.Y = Y;
  a.base.ldy = ldy;
  a.ids = adapter;
  a.n = adapters;
  a.r = rank;
  a.A = static_cast<const uint16_t*>(A);
  a.B = static_cast<const uint16_t*>(B);
  a.scale = scale;
  a.xa = xa;
  a.workspace = workspace;
  return hip_status(nm::launch_adapter(a, static_cast<hipStream_t>(stream)), "nm_adapter_spmm launch");
}

nm_status nm_adapter_spmm_bwd_workspace_size(int64_t R, int64_t K, int n, int m, int dtype, int64_t T,
                                             int64_t adapters, int64_t rank, int out_dtype, size_t* bytes) {
  nm_status st = check_adapter(R, K, n, m, dtype, T, adapters, rank, out_dtype);
  if (st != NM_OK) return st;
  if (!bytes) return fail(NM_ERR_NULL, "bytes must be non-NULL");
  *bytes = nm::adapter_bwd_workspace(R, K, T, adapters, rank);
  return ok();
}

nm_status nm_adapter_spmm_bwd(const void* values, const uint32_t* idx, int64_t R, int64_t K, int n, int m, int dtype,
                              const void* G, int64_t T, int64_t ldg, const void* act, int64_t ldx, const float* xa,
                              const int32_t* adapter, const void* A, const void* B, const float* scale,
                              int64_t adapters, int64_t rank, void* dX, int64_t lddx, float* dA, float* dB,
                              int out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  nm_status st = check_train(R, K, n, m, dtype, T, ldg, out_dtype);
  if (st != NM_OK) return st;
  if ((st = check_adapter(R, K, n, m, dtype, T, adapters, rank, out_dtype)) != NM_OK) return st;
  if ((st = check_ld("ldg", ldg, T, R)) != NM_OK || (st = check_ld("ldx", ldx, T, K)) != NM_OK) return st;
  if (dX && (st = check_ld("lddx", lddx, T, K)) != NM_OK) return st;
  if (T == 0 && adapters == 0) return ok();
  if (T > 0 && (!act || !xa || !adapter || !workspace || (R > 0 && (!G || !values || !idx))))
    return fail(NM_ERR_NULL, "values, idx, G, act, xa, adapter and workspace must be non-NULL");
  if (adapters > 0 && (!A || !scale || !dA || (R > 0 && (!B || !dB))))
    return fail(NM_ERR_NULL, "A, B, scale, dA and dB must be non-NULL");
  if (ldg % 8 || ldx % 8) return fail(NM_ERR_ALIGN, "ldg and ldx must be multiples of 8");
  if (!aligned16(values) || !aligned16(idx) || !aligned16(G) || !aligned16(act) || !aligned16(xa) || !aligned16(A) ||
      !aligned16(B) || !aligned16(dX) || !aligned16(dA) || !aligned16(dB) || !aligned16(workspace) ||
      !aligned_to(adapter, 4) || !aligned_to(scale, 4))
    return fail(NM_ERR_ALIGN, "device pointers must be 16-byte aligned (adapter and scale: 4)");
  const size_t need = nm::adapter_bwd_workspace(R, K, T, adapters, rank);
  if (T > 0 && workspace_bytes < need)
    return fail(NM_ERR_SHAPE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  const Sizes z = sizes_of(R, K, n, m, dtype);
  // nm_spmm_dx's limits
  if (z.values_bytes >= (size_t(1) << 32) || z.idx_bytes >= (size_t(1) << 32) || 128 * ldg * 2 >= (int64_t(1) << 32))
    return fail(NM_ERR_SHAPE, "packed W of 4 GiB or more, or ldg of 2^24 or more");
  const size_t ab = size_t(adapters) * size_t(rank) * size_t(K), bb = size_t(adapters) * size_t(rank) * size_t(R);
  const Span in[] = {{values, z.values_bytes}, {idx, z.idx_bytes}, {G, extent(T, R, ldg, 2)},
                     {act, extent(T, K, ldx, 2)}, {xa, size_t(T) * size_t(rank) * 4}, {adapter, size_t(T) * 4},
                     {A, ab * 2}, {B, bb * 2}, {scale, size_t(adapters) * 4}};
  const Span out[] = {{dX, dX ? extent(T, K, lddx, elt_bytes(out_dtype)) : 0}, {dA, ab * 4}, {dB, bb * 4},
                      {workspace, T > 0 ? need : 0}};
  if ((st = check_alias(in, out)) != NM_OK) return st;
  nm::AdapterBwdArgs a;
  a.dx.values = static_cast<const uint16_t*>(values);
  a.dx.values_bytes = z.values_bytes;
  a.dx.idx = idx;
  a.dx.idx_bytes = z.idx_bytes;
  a.dx.R = R;
  a.dx.K = K;
  a.dx.n = n;
  a.dx.m = m;
  a.dx.dtype = dtype;
  a.dx.idx_row_words = z.words;
  a.dx.G = static_cast<const uint16_t*>(G);
  a.dx.T = T;
  a.dx.ldg = ldg;
  a.dx.act = static_cast<const uint16_t*>(act);
  a.dx.ldx = ldx;
  a.dx.out = dX;
  a.dx.ldo = lddx;
  a.dx.out_dtype = out_dtype;
  a.ids = adapter;
  a.n = adapters;
  a.r = rank;
  a.A = static_cast<const uint16_t*>(A);
  a.B = static_cast<const uint16_t*>(B);
  a.scale = scale;
  a.xa = xa;
  a.dA = dA;
  a.dB = dB;
  a.workspace = workspace;
  return hip_status(nm::launch_adapter_bwd(a, static_cast<hipStream_t>(stream)), "nm_adapter_spmm_bwd launch");
}

// Shared checks of cross entropy: x [T, H] and w [V, H] in a 16-bit type.
static nm_status check_xent(int64_t T, int64_t V, int64_t H, int dtype) {
  if (dtype != NM_F16 && dtype != NM_BF16)
    return fail(NM_ERR_UNSUPPORTED, "cross entropy takes NM_F16 or NM_BF16, not dtype %d", dtype);
  if (T < 0 || T > nm::kXentMaxTokens) return fail(NM_ERR_SHAPE, "T = %lld out of range [0, 2^22]", (long long)T);
  if (V < 1 || V > nm::kXentMaxVocab) return fail(NM_ERR_SHAPE, "V = %lld out of range [1, 2^24]", (long long)V);
  if (H < 8 || H > nm::kXentMaxH || H % 8)
    return fail(NM_ERR_SHAPE, "H = %lld is not a multiple of 8 in [8, 2^20]", (long long)H);
  // tiles of the products are counted in 32 bits
  if (((T + 15) / 16) * ((V + 127) / 128) > (int64_t(1) << 22) * 16)
    return fail(NM_ERR_SHAPE, "T x V = %lld x %lld is too large", (long long)T, (long long)V);
  return NM_OK;
}

// A 16-bit operand of cross entropy: rows on 16 bytes, 256 of them within 4 GiB.
static nm_status check_xent_ld(const char* name, int64_t ld, int64_t rows, int64_t H) {
  nm_status st = check_ld(name, ld, rows, H);
  if (st != NM_OK) return st;
  if (ld % 8) return fail(NM_ERR_ALIGN, "%s = %lld is not a multiple of 8", name, (long long)ld);
  if (ld >= (int64_t(1) << 23)) return fail(NM_ERR_SHAPE, "%s of 2^23 or more", name);
  return NM_OK;
}

nm_status nm_xent_workspace_size(int64_t T, int64_t V, int64_t H, int dtype, size_t* bytes) {
  nm_status st = check_xent(T, V, H, dtype);
  if (st != NM_OK) return st;
  if (!bytes) return fail(NM_ERR_NULL, "bytes must be non-NULL");
  *bytes = nm::xent_workspace(T, V);
  return ok();
}

nm_status nm_xent(const void* x, int64_t T, int64_t H, int64_t ldx, const void* w, int64_t V, int64_t ldw, int dtype,
                  const int32_t* labels, float* loss, float* lse, void* workspace, size_t workspace_bytes,
                  void* stream) {
  nm_status st = check_xent(T, V, H, dtype);
  if (st != NM_OK) return st;
  if ((st = check_xent_ld("ldx", ldx, T, H)) != NM_OK || (st = check_xent_ld("ldw", ldw, V, H)) != NM_OK) return st;
  if (T == 0) return ok();
  if (!x || !w || !labels || !loss || !lse || !workspace)
    return fail(NM_ERR_NULL, "x, w, labels, loss, lse and workspace must be non-NULL");
  if (!aligned16(x) || !aligned16(w) || !aligned16(workspace) || !aligned_to(labels, 4) || !aligned_to(loss, 4) ||
      !aligned_to(lse, 4))
    return fail(NM_ERR_ALIGN, "x, w and workspace must be 16-byte aligned, labels, loss and lse 4-byte");
  const size_t need = nm::xent_workspace(T, V);
  if (workspace_bytes < need)
    return fail(NM_ERR_SHAPE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  const size_t tb = size_t(T) * 4;
  const Span in[] = {{x, extent(T, H, ldx, 2)}, {w, extent(V, H, ldw, 2)}, {labels, tb}};
  const Span out[] = {{loss, tb}, {lse, tb}, {workspace, need}};
  if ((st = check_alias(in, out)) != NM_OK) return st;
  nm::XentArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.w = static_cast<const uint16_t*>(w);
  a.labels = labels;
  a.ldx = ldx;
  a.ldw = ldw;
  a.T = T;
  a.V = V;
  a.H = H;
  a.dtype = dtype;
  a.loss = loss;
  a.lse_out = lse;
  a.workspace = workspace;
  return hip_status(nm::launch_xent(a, static_cast<hipStream_t>(stream)), "nm_xent launch");
}

nm_status nm_xent_bwd_workspace_size(int64_t T, int64_t V, int64_t H, int dtype, int need_dx, int need_dw,
                                     size_t* bytes) {
  nm_status st = check_xent(T, V, H, dtype);
  if (st != NM_OK) return st;
  if (!bytes) return fail(NM_ERR_NULL, "bytes must be non-NULL");
  *bytes = nm::xent_bwd_workspace(T, V, H, need_dx ? 2 : 0, need_dw ? 2 : 0);   // enough for either type
  return ok();
}

nm_status nm_xent_bwd(const void* x, int64_t T, int64_t H, int64_t ldx, const void* w, int64_t V, int64_t ldw,
                      int dtype, const int32_t* labels, const float* lse, const float* dloss, void* dx, int64_t lddx,
                      int dx_dtype, void* dw, int64_t lddw, int dw_dtype, void* workspace, size_t workspace_bytes,
                      void* stream) {
  nm_status st = check_xent(T, V, H, dtype);
  if (st != NM_OK) return st;
  if ((dx && dx_dtype != NM_F32 && dx_dtype != dtype) || (dw && dw_dtype != NM_F32 && dw_dtype != dtype))
    return fail(NM_ERR_UNSUPPORTED, "dx_dtype and dw_dtype must be NM_F32 or the input dtype");
  if ((st = check_xent_ld("ldx", ldx, T, H)) != NM_OK || (st = check_xent_ld("ldw", ldw, V, H)) != NM_OK) return st;
  if ((dx && (st = check_ld("lddx", lddx, T, H)) != NM_OK) || (dw && (st = check_ld("lddw", lddw, V, H)) != NM_OK))
    return st;
  if (!dx && !dw) return ok();
  if (T == 0 && !dw) return ok();
  if (T > 0 && (!x || !w || !labels || !lse || !dloss || !workspace))
    return fail(NM_ERR_NULL, "x, w, labels, lse, dloss and workspace must be non-NULL");
  if ((dx && lddx % 4) || (dw && lddw % 4)) return fail(NM_ERR_ALIGN, "lddx and lddw must be multiples of 4");
  if (!aligned16(x) || !aligned16(w) || !aligned16(dx) || !aligned16(dw) || !aligned16(workspace) ||
      !aligned_to(labels, 4) || !aligned_to(lse, 4) || !aligned_to(dloss, 4))
    return fail(NM_ERR_ALIGN, "matrices and workspace must be 16-byte aligned, vectors 4-byte");
  const size_t need = nm::xent_bwd_workspace(T, V, H, dx ? 1 + (dx_dtype == NM_F32) : 0, dw ? 1 + (dw_dtype == NM_F32) : 0);
  if (workspace_bytes < need)
    return fail(NM_ERR_SHAPE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  const size_t tb = size_t(T) * 4;
  const Span in[] = {{x, extent(T, H, ldx, 2)}, {w, extent(V, H, ldw, 2)}, {labels, tb}, {lse, tb}, {dloss, tb}};
  const Span out[] = {{dx, dx ? extent(T, H, lddx, elt_bytes(dx_dtype)) : 0},
                      {dw, dw ? extent(V, H, lddw, elt_bytes(dw_dtype)) : 0}, {workspace, need}};
  if ((st = check_alias(in, out)) != NM_OK) return st;
  nm::XentArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.w = static_cast<const uint16_t*>(w);
  a.labels = labels;
  a.ldx = ldx;
  a.ldw = ldw;
  a.T = T;
  a.V = V;
  a.H = H;
  a.dtype = dtype;
  a.lse = lse;
  a.dloss = dloss;
  a.dx = dx;
  a.dw = dw;
  a.lddx = lddx;
  a.lddw = lddw;
  a.dx_dtype = dx_dtype;
  a.dw_dtype = dw_dtype;
  a.workspace = workspace;
  return hip_status(nm::launch_xent_bwd(a, static_cast<hipStream_t>(stream)), "nm_xent_bwd launch");
}

// Shared checks of the products grouped by expert: one expert's packed weight
// (16-bit), the counts, the output type and the offsets.
static nm_status check_group(int64_t E, int64_t R, int64_t K, int n, int m, int dtype, int64_t T, int out_dtype) {
  nm_status st = check_format(R, K, n, m, dtype);
  if (st != NM_OK) return st;
  if (dtype != NM_F16 && dtype != NM_BF16) return fail(NM_ERR_UNSUPPORTED, "grouped products take fp16 or bf16 weights");
  if (out_dtype != NM_F32 && out_dtype != dtype)
    return fail(NM_ERR_UNSUPPORTED, "out_dtype %d must be NM_F32 or the input dtype", out_dtype);
  if (E < 1 || E > nm::kGroupMaxExperts)
    return fail(NM_ERR_SHAPE, "E = %lld out of range [1, %lld]", (long long)E, (long long)nm::kGroupMaxExperts);
  if (T < 0 || T > nm::kGroupMaxTokens) return fail(NM_ERR_SHAPE, "T = %lld out of range [0, 2^24]", (long long)T);
  if (R > nm::kGroupMaxWidth || K > nm::kGroupMaxWidth)
    return fail(NM_ERR_SHAPE, "R = %lld or K = %lld above 2^22", (long long)R, (long long)K);
  return NM_OK;
}

// A 16-bit operand's leading dimension: rows on 16 bytes, 128 of them in 32-bit offsets.
static nm_status check_group_ld(const char* name, int64_t ld, int64_t T, int64_t W) {
  nm_status st = check_ld(name, ld, T, W);
  if (st != NM_OK) return st;
  if (ld >= nm::kGroupMaxLd) return fail(NM_ERR_SHAPE, "%s of 2^23 or more", name);
  if (ld % 8) return fail(NM_ERR_ALIGN, "%s = %lld is not a multiple of 8", name, (long long)ld);
  return NM_OK;
}

static nm_status check_workspace(const void* workspace, size_t have, size_t need) {
  if (need > 0 && !workspace) return fail(NM_ERR_NULL, "workspace must be non-NULL");
  if (have < need) return fail(NM_ERR_SHAPE, "workspace of %zu bytes, %zu needed", have, need);
  if (need > 0 && !aligned16(workspace)) return fail(NM_ERR_ALIGN, "workspace must be 16-byte aligned");
  return NM_OK;
}

static nm::SpmmArgs group_base(int64_t R, int64_t K, int n, int m, int dtype, int64_t T, int64_t ldx, int out_dtype) {
  return adapter_base(R, K, n, m, dtype, T, ldx, out_dtype);
}

nm_status nm_group_spmm_workspace_size(int64_t E, int64_t R, int64_t K, int n, int m, int dtype, int64_t T,
                                       int out_dtype, size_t* bytes) {
  nm_status st = check_group(E, R, K, n, m, dtype, T, out_dtype);
  if (st != NM_OK) return st;
  if (!bytes) return fail(NM_ERR_NULL, "bytes must be non-NULL");
  *bytes = T == 0 || R == 0 ? 0 : nm::group_workspace(group_base(R, K, n, m, dtype, T, K, out_dtype), E);
  return ok();
}

nm_status nm_group_spmm(const void* values, const uint32_t* idx, int64_t E, int64_t R, int64_t K, int n, int m,
                        int dtype, const void* act, int64_t T, int64_t ldx, const int32_t* offsets, void* Y,
                        int64_t ldy, int out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  nm_status st = check_group(E, R, K, n, m, dtype, T, out_dtype);
  if (st != NM_OK) return st;
  if ((st = check_group_ld("ldx", ldx, T, K)) != NM_OK || (st = check_ld("ldy", ldy, T, R)) != NM_OK) return st;
  if (T == 0 || R == 0) return ok();
  if (!values || !idx || !act || !offsets || !Y)
    return fail(NM_ERR_NULL, "values, idx, act, offsets and Y must be non-NULL");
  if (!aligned16(values) || !aligned16(idx) || !aligned16(act) || !aligned16(Y) || !aligned_to(offsets, 4))
    return fail(NM_ERR_ALIGN, "device pointers must be 16-byte aligned (offsets: 4)");
  nm::GroupArgs a;
  a.base = group_base(R, K, n, m, dtype, T, ldx, out_dtype);
  const size_t need = nm::group_workspace(a.base, E);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != NM_OK) return st;
  const Sizes z = sizes_of(R, K, n, m, dtype);
  const Span in[] = {{values, size_t(E) * z.values_bytes}, {idx, size_t(E) * z.idx_bytes},
                     {act, extent(T, K, ldx, 2)}, {offsets, size_t(E + 1) * 4}};
  const Span out[] = {{Y, extent(T, R, ldy, elt_bytes(out_dtype))}, {workspace, need}};
  if ((st = check_alias(in, out)) != NM_OK) return st;
  a.base.values = static_cast<const uint16_t*>(values);
  a.base.idx = idx;
  a.base.act = static_cast<const uint16_t*>(act);
  a.base.Y = Y;
  a.base.ldy = ldy;
  a.offsets = offsets;
  a.E = E;
  a.workspace = workspace;
  return hip_status(nm::launch_group(a, static_cast<hipStream_t>(stream)), "nm_group_spmm launch");
}

nm_status nm_group_spmm_dx_workspace_size(int64_t E, int64_t R, int64_t K, int64_t T, size_t* bytes) {
  nm_status st = check_group(E, R, K, 2, 4, NM_BF16, T, NM_F32);
  if (st != NM_OK) return st;
  if (!bytes) return fail(NM_ERR_NULL, "bytes must be non-NULL");
  *bytes = T == 0 ? 0 : nm::group_dx_workspace(R, K, T, E);
  return ok();
}

nm_status nm_group_spmm_dx(const void* values, const uint32_t* idx, int64_t E, int64_t R, int64_t K, int n, int m,
                           int dtype, const void* G, int64_t T, int64_t ldg, const int32_t* offsets, void* dX,
                           int64_t lddx, int out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  nm_status st = check_group(E, R, K, n, m, dtype, T, out_dtype);
  if (st != NM_OK) return st;
  if ((st = check_train(R, K, n, m, dtype, T, ldg, out_dtype)) != NM_OK) return st;
  if ((st = check_group_ld("ldg", ldg, T, R)) != NM_OK || (st = check_ld("lddx", lddx, T, K)) != NM_OK) return st;
  if (T == 0) return ok();
  if (!offsets || !dX || (R > 0 && (!values || !idx || !G)))
    return fail(NM_ERR_NULL, "values, idx, G, offsets and dX must be non-NULL");
  if (!aligned16(values) || !aligned16(idx) || !aligned16(G) || !aligned16(dX) || !aligned_to(offsets, 4))
    return fail(NM_ERR_ALIGN, "device pointers must be 16-byte aligned (offsets: 4)");
  const size_t need = nm::group_dx_workspace(R, K, T, E);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != NM_OK) return st;
  const Sizes z = sizes_of(R, K, n, m, dtype);
  if (z.values_bytes >= (size_t(1) << 32) || z.idx_bytes >= (size_t(1) << 32))
    return fail(NM_ERR_SHAPE, "one expert's packed W of 4 GiB or more");
  const Span in[] = {{values, size_t(E) * z.values_bytes}, {idx, size_t(E) * z.idx_bytes},
                     {G, extent(T, R, ldg, 2)}, {offsets, size_t(E + 1) * 4}};
  const Span out[] = {{dX, extent(T, K, lddx, elt_bytes(out_dtype))}, {workspace, need}};
  if ((st = check_alias(in, out)) != NM_OK) return st;
  nm::TrainArgs a{};
  a.values = static_cast<const uint16_t*>(values);
  a.values_bytes = z.values_bytes;
  a.idx = idx;
  a.idx_bytes = z.idx_bytes;
  a.R = R;
  a.K = K;
  a.n = n;
  a.m = m;
  a.dtype = dtype;
  a.idx_row_words = z.words;
  a.G = static_cast<const uint16_t*>(G);
  a.T = T;
  a.ldg = ldg;
  a.out = dX;
  a.ldo = lddx;
  a.out_dtype = out_dtype;
  a.offsets = offsets;
  a.experts = E;
  a.table = workspace;
  return hip_status(nm::launch_spmm_dx(a, static_cast<hipStream_t>(stream)), "nm_group_spmm_dx launch");
}

nm_status nm_group_spmm_dw_workspace_size(int64_t E, int64_t R, int64_t K, int n, int m, int64_t T, size_t* bytes) {
  nm_status st = check_group(E, R, K, n, m, NM_BF16, T, NM_F32);
  if (st != NM_OK) return st;
  if (!bytes) return fail(NM_ERR_NULL, "bytes must be non-NULL");
  *bytes = nm::group_dw_workspace(R, K, K / m * n, T, E);
  return ok();
}

nm_status nm_group_spmm_dw(const uint32_t* idx, int64_t E, int64_t R, int64_t K, int n, int m, int dtype, const void* G,
                           int64_t T, int64_t ldg, const void* act, int64_t ldx, const int32_t* offsets, void* dW,
                           int out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  nm_status st = check_group(E, R, K, n, m, dtype, T, out_dtype);
  if (st != NM_OK) return st;
  if ((st = check_train(R, K, n, m, dtype, T, ldg, out_dtype)) != NM_OK) return st;
  if ((st = check_group_ld("ldg", ldg, T, R)) != NM_OK || (st = check_group_ld("ldx", ldx, T, K)) != NM_OK) return st;
  if (R == 0) return ok();
  if (!idx || !offsets || !dW || (T > 0 && (!G || !act)))
    return fail(NM_ERR_NULL, "idx, G, act, offsets and dW must be non-NULL");
  if (!aligned16(idx) || !aligned16(G) || !aligned16(act) || !aligned16(dW) || !aligned_to(offsets, 4))
    return fail(NM_ERR_ALIGN, "device pointers must be 16-byte aligned (offsets: 4)");
  if (T * ldg * 2 >= (int64_t(1) << 32) || T * ldx * 2 >= (int64_t(1) << 32))
    return fail(NM_ERR_SHAPE, "G or act of 4 GiB or more");
  const Sizes z = sizes_of(R, K, n, m, dtype);
  if (z.idx_bytes >= (size_t(1) << 32)) return fail(NM_ERR_SHAPE, "one expert's index words of 4 GiB or more");
  const size_t need = nm::group_dw_workspace(R, K, z.S, T, E);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != NM_OK) return st;
  const Span in[] = {{idx, size_t(E) * z.idx_bytes}, {G, extent(T, R, ldg, 2)}, {act, extent(T, K, ldx, 2)},
                     {offsets, size_t(E + 1) * 4}};
  const Span out[] = {{dW, size_t(E) * size_t(R) * size_t(z.S) * elt_bytes(out_dtype)}, {workspace, need}};
  if ((st = check_alias(in, out)) != NM_OK) return st;
  nm::TrainArgs a{};
  a.idx = idx;
  a.idx_bytes = z.idx_bytes;
  a.R = R;
  a.K = K;
  a.n = n;
  a.m = m;
  a.dtype = dtype;
  a.idx_row_words = z.words;
  a.G = static_cast<const uint16_t*>(G);
  a.T = T;
  a.ldg = ldg;
  a.act = static_cast<const uint16_t*>(act);
  a.ldx = ldx;
  a.out = dW;
  a.out_dtype = out_dtype;
  a.offsets = offsets;
  a.experts = E;
  a.table = workspace;
  return hip_status(nm::launch_spmm_dw(a, static_cast<hipStream_t>(stream)), "nm_group_spmm_dw launch");
}

// Shared checks of the 4-bit format: rows and columns of a quantised matrix.
static nm_status check_mx(const char* rows_name, int64_t rows, int64_t K) {
  if (rows < 0 || rows > nm::kMxMaxRows)
    return fail(NM_ERR_SHAPE, "%s = %lld out of range [0, 2^24]", rows_name, (long long)rows);
  if (K < 32 || K > nm::kGroupMaxWidth || K % 32)
    return fail(NM_ERR_SHAPE, "K = %lld is not a multiple of 32 in [32, 2^22]", (long long)K);
  return NM_OK;
}

static nm_status check_mx_float(int dtype) {
  if (dtype != NM_F16 && dtype != NM_BF16 && dtype != NM_F32)
    return fail(NM_ERR_UNSUPPORTED, "dtype %d is not NM_F16, NM_BF16 or NM_F32", dtype);
  return NM_OK;
}

static size_t mx_scale_bytes(int64_t rows, int64_t K) { return size_t((K + 255) / 256) * size_t(rows) * 8; }

nm_status nm_mx_sizes(int64_t T, int64_t K, size_t* q_bytes, size_t* scale_bytes) {
  nm_status st = check_mx("T", T, K);
  if (st != NM_OK) return st;
  if (q_bytes) *q_bytes = size_t(T) * size_t(K / 2);
  if (scale_bytes) *scale_bytes = mx_scale_bytes(T, K);
  return ok();
}

// E matrices, `stride` elements of x (y) apart.
static nm_status check_mx_stack(const char* rows_name, int64_t E, int64_t R, int64_t K, int dtype, const char* ld_name,
                                int64_t ld, int64_t stride) {
  nm_status st = check_mx(rows_name, R, K);
  if (st != NM_OK || (st = check_mx_float(dtype)) != NM_OK || (st = check_ld(ld_name, ld, R, K)) != NM_OK) return st;
  if (E < 0 || E > nm::kMxMaxRows) return fail(NM_ERR_SHAPE, "E = %lld out of range [0, 2^24]", (long long)E);
  if (stride < 0) return fail(NM_ERR_STRIDE, "stride = %lld is negative", (long long)stride);
  if (E > 0 && (stride > kMaxElems / E || R * K > kMaxElems / E))
    return fail(NM_ERR_SHAPE, "a stack above 2^40 elements");
  return NM_OK;
}

static size_t mx_stack_extent(int64_t E, int64_t R, int64_t K, int64_t ld, int64_t stride, size_t e) {
  return size_t(E - 1) * size_t(stride) * e + extent(R, K, ld, e);
}

// An expert's scales are a multiple of 8 bytes long, so in a stack they begin on 8;
// the kernels read them by the byte (nm_mx_gemm: two or four).
static nm_status mx_quantize(const void* x, int64_t E, int64_t R, int64_t K, int64_t ldx, int64_t stride, int dtype,
                             uint8_t* q, uint8_t* scale, size_t scale_align, hipStream_t s) {
  if (E == 0 || R == 0) return ok();
  if (!x || !q || !scale) return fail(NM_ERR_NULL, "x, q and scale must be non-NULL");
  const size_t e = elt_bytes(dtype);
  if (!aligned_to(x, e) || !aligned16(q) || !aligned_to(scale, scale_align))
    return fail(NM_ERR_ALIGN, "q must be 16-byte aligned, scale %zu, x to its element", scale_align);
  const Span in[] = {{x, mx_stack_extent(E, R, K, ldx, stride, e)}};
  const Span out[] = {{q, size_t(E) * size_t(R) * size_t(K / 2)}, {scale, size_t(E) * mx_scale_bytes(R, K)}};
  if (nm_status st = check_alias(in, out); st != NM_OK) return st;
  nm::MxQuantArgs a;
  a.E = E;
  a.T = R;
  a.K = K;
  a.ldx = ldx;
  a.stride = stride;
  a.dtype = dtype;
  a.x = x;
  a.q = q;
  a.scale = scale;
  return hip_status(nm::launch_mx_quantize(a, s), "nm_mx_quantize launch");
}

nm_status nm_mx_quantize(const void* x, int64_t T, int64_t K, int64_t ldx, int dtype, uint8_t* q, uint8_t* scale,
                         void* stream) {
  nm_status st = check_mx_stack("T", 1, T, K, dtype, "ldx", ldx, 0);
  if (st != NM_OK) return st;
  return mx_quantize(x, 1, T, K, ldx, 0, dtype, q, scale, 16, static_cast<hipStream_t>(stream));
}

nm_status nm_mx_quantize_stack(const void* x, int64_t E, int64_t R, int64_t K, int64_t ldx, int64_t stride, int dtype,
                               uint8_t* q, uint8_t* scale, void* stream) {
  nm_status st = check_mx_stack("R", E, R, K, dtype, "ldx", ldx, stride);
  if (st != NM_OK) return st;
  return mx_quantize(x, E, R, K, ldx, stride, dtype, q, scale, 8, static_cast<hipStream_t>(stream));
}

static nm_status mx_dequantize(const uint8_t* q, const uint8_t* scale, size_t scale_align, int64_t E, int64_t R,
                               int64_t K, void* y, int64_t ldy, int64_t stride, int dtype, hipStream_t s) {
  if (E == 0 || R == 0) return ok();
  if (!y || !q || !scale) return fail(NM_ERR_NULL, "q, scale and y must be non-NULL");
  const size_t e = elt_bytes(dtype);
  if (!aligned_to(y, e) || !aligned16(q) || !aligned_to(scale, scale_align))
    return fail(NM_ERR_ALIGN, "q must be 16-byte aligned, scale %zu, y to its element", scale_align);
  const Span in[] = {{q, size_t(E) * size_t(R) * size_t(K / 2)}, {scale, size_t(E) * mx_scale_bytes(R, K)}};
  const Span out[] = {{y, mx_stack_extent(E, R, K, ldy, stride, e)}};
  if (nm_status st = check_alias(in, out); st != NM_OK) return st;
  nm::MxQuantArgs a;
  a.E = E;
  a.T = R;
  a.K = K;
  a.ldx = ldy;
  a.stride = stride;
  a.dtype = dtype;
  a.q = const_cast<uint8_t*>(q);
  a.scale = const_cast<uint8_t*>(scale);
  a.y = y;
  return hip_status(nm::launch_mx_dequantize(a, s), "nm_mx_dequantize launch");
}

nm_status nm_mx_dequantize(const uint8_t* q, const uint8_t* scale, int64_t T, int64_t K, void* y, int64_t ldy,
                           int dtype, void* stream) {
  nm_status st = check_mx_stack("T", 1, T, K, dtype, "ldy", ldy, 0);
  if (st != NM_OK) return st;
  return mx_dequantize(q, scale, 16, 1, T, K, y, ldy, 0, dtype, static_cast<hipStream_t>(stream));
}

nm_status nm_mx_dequantize_stack(const uint8_t* q, const uint8_t* scale, int64_t E, int64_t R, int64_t K, void* y,
                                 int64_t ldy, int64_t stride, int dtype, void* stream) {
  nm_status st = check_mx_stack("R", E, R, K, dtype, "ldy", ldy, stride);
  if (st != NM_OK) return st;
  if (E > 1 && R > 0 && stride < (R - 1) * ldy + K)   // the matrices written would overlap
    return fail(NM_ERR_STRIDE, "stride = %lld below one matrix", (long long)stride);
  return mx_dequantize(q, scale, 8, E, R, K, y, ldy, stride, dtype, static_cast<hipStream_t>(stream));
}

static nm_status check_mx_gemm(int64_t E, int64_t R, int64_t K, int64_t T, bool grouped, int out_dtype) {
  nm_status st = check_mx("R", R, K);
  if (st != NM_OK || (st = check_mx("T", T, K)) != NM_OK || (st = check_mx_float(out_dtype)) != NM_OK) return st;
  if (R > nm::kGroupMaxWidth) return fail(NM_ERR_SHAPE, "R = %lld above 2^22", (long long)R);
  if (E < 1 || E > nm::kGroupMaxExperts || (!grouped && E != 1))
    return fail(NM_ERR_SHAPE, "E = %lld out of range (1 without offsets, else [1, %lld])", (long long)E,
                (long long)nm::kGroupMaxExperts);
  // 32-bit offsets into one operand's scales
  if (mx_scale_bytes(R, K) >= (size_t(1) << 32) || mx_scale_bytes(T, K) >= (size_t(1) << 32))
    return fail(NM_ERR_SHAPE, "scales of 4 GiB or more");
  return NM_OK;
}

nm_status nm_mx_gemm_workspace_size(int64_t E, int64_t R, int64_t K, int64_t T, int grouped, int out_dtype,
                                    size_t* bytes) {
  nm_status st = check_mx_gemm(E, R, K, T, grouped != 0, out_dtype);
  if (st != NM_OK) return st;
  if (!bytes) return fail(NM_ERR_NULL, "bytes must be non-NULL");
  *bytes = T == 0 || R == 0 ? 0 : nm::mx_workspace(E, R, T, grouped != 0);
  return ok();
}

nm_status nm_mx_gemm(const uint8_t* wq, const uint8_t* wscale, int64_t E, int64_t R, int64_t K, const uint8_t* xq,
                     const uint8_t* xscale, int64_t T, const int32_t* offsets, void* Y, int64_t ldy, int out_dtype,
                     void* workspace, size_t workspace_bytes, void* stream) {
  nm_status st = check_mx_gemm(E, R, K, T, offsets != nullptr, out_dtype);
  if (st != NM_OK || (st = check_ld("ldy", ldy, T, R)) != NM_OK) return st;
  if (T == 0 || R == 0) return ok();
  if (!wq || !wscale || !xq || !xscale || !Y)
    return fail(NM_ERR_NULL, "wq, wscale, xq, xscale and Y must be non-NULL");
  if (!aligned16(wq) || !aligned_to(wscale, 8) || !aligned16(xq) || !aligned_to(xscale, 8) || !aligned16(Y) ||
      !aligned_to(offsets, 4))
    return fail(NM_ERR_ALIGN, "device pointers must be 16-byte aligned (scales: 8, offsets: 4)");
  const size_t need = nm::mx_workspace(E, R, T, offsets != nullptr);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != NM_OK) return st;
  const Span in[] = {{wq, size_t(E) * size_t(R) * size_t(K / 2)}, {wscale, size_t(E) * mx_scale_bytes(R, K)},
                     {xq, size_t(T) * size_t(K / 2)}, {xscale, mx_scale_bytes(T, K)},
                     {offsets, offsets ? size_t(E + 1) * 4 : 0}};
  const Span out[] = {{Y, extent(T, R, ldy, elt_bytes(out_dtype))}, {workspace, need}};
  if ((st = check_alias(in, out)) != NM_OK) return st;
  nm::MxArgs a;
  a.wq = wq;
  a.ws = wscale;
  a.xq = xq;
  a.xs = xscale;
  a.offsets = offsets;
  a.E = E;
  a.R = R;
  a.K = K;
  a.T = T;
  a.ldy = ldy;
  a.Y = Y;
  a.out_dtype = out_dtype;
  a.workspace = workspace;
  return hip_status(nm::launch_mx_gemm(a, static_cast<hipStream_t>(stream)), "nm_mx_gemm launch");
}

nm_status nm_grad_workspace_size(int64_t tensors, size_t* bytes) {
  if (tensors < 0 || tensors > nm::kGradMaxTensors)
    return fail(NM_ERR_SHAPE, "tensors = %lld out of range [0, %lld]", (long long)tensors,
                (long long)nm::kGradMaxTensors);
  if (!bytes) return fail(NM_ERR_NULL, "bytes must be non-NULL");
  *bytes = nm::grad_workspace(tensors);
  return ok();
}

// A written range and the tensor it belongs to.
struct Written {
  uintptr_t begin, end;
  int32_t tensor;
};

// The lists of a norm (out NULL) or a clipping: their types and counts, and that
// nothing written overlaps anything else, but for a tensor scaled in place.
static nm_status check_grads(const void* const* grads, const int64_t* counts, const int* dtypes, int64_t tensors,
                             void* const* out, const float* norm, const void* workspace, size_t workspace_bytes) {
  if (tensors < 0 || tensors > nm::kGradMaxTensors)
    return fail(NM_ERR_SHAPE, "tensors = %lld out of range [0, %lld]", (long long)tensors,
                (long long)nm::kGradMaxTensors);
  if (!norm || (tensors > 0 && (!grads || !counts || !dtypes)))
    return fail(NM_ERR_NULL, "grads, counts, dtypes and norm must be non-NULL");
  nm_status st = check_workspace(workspace, workspace_bytes, nm::grad_workspace(tensors));
  if (st != NM_OK) return st;
  if (!aligned_to(norm, 4)) return fail(NM_ERR_ALIGN, "norm must be 4-byte aligned");
  // The ranges of ordinary lists in 6 KB of the caller's stack; those of longer ones, up
  // to 400 KB, in one array for the process: a thread's whole stack may be smaller, and
  // no call allocates.
  constexpr int64_t kFew = 254;
  static Written many[nm::kGradMaxTensors + 2];
  static std::mutex many_mutex;
  Written few[kFew + 2], *w = few;
  std::unique_lock<std::mutex> hold(many_mutex, std::defer_lock);
  if (out && tensors > kFew) {
    hold.lock();
    w = many;
  }
  int64_t written = 0;
  auto add = [&](const void* p, size_t bytes, int32_t tensor) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(p);
    w[written++] = Written{b, b + bytes, tensor};
  };
  add(norm, 4, -1);
  add(workspace, nm::grad_workspace(tensors), -1);
  for (int64_t i = 0; i < tensors; ++i) {
    if (dtypes[i] != NM_F16 && dtypes[i] != NM_BF16 && dtypes[i] != NM_F32)
      return fail(NM_ERR_UNSUPPORTED, "tensor %lld: dtype %d is not NM_F16, NM_BF16 or NM_F32", (long long)i, dtypes[i]);
    if (counts[i] < 0 || counts[i] > nm::kGradMaxCount)
      return fail(NM_ERR_SHAPE, "tensor %lld: count %lld out of range [0, 2^36]", (long long)i, (long long)counts[i]);
    if (counts[i] == 0) continue;
    const size_t e = elt_bytes(dtypes[i]);
    if (!grads[i] || (out && !out[i])) return fail(NM_ERR_NULL, "tensor %lld is NULL", (long long)i);
    if (!aligned_to(grads[i], e) || (out && !aligned_to(out[i], e)))
      return fail(NM_ERR_ALIGN, "tensor %lld is not aligned to its element", (long long)i);
    if (out) add(out[i], size_t(counts[i]) * e, int32_t(i));
  }
  auto before = [](const Written& a, const Written& b) { return a.begin < b.begin; };
  if (!std::is_sorted(w, w + written, before)) std::sort(w, w + written, before);
  for (int64_t i = 1; i < written; ++i)
    if (w[i].begin < w[i - 1].end) return fail(NM_ERR_ALIAS, "outputs, norm or workspace overlap each other");
  for (int64_t i = 0; i < tensors; ++i) {
    if (counts[i] == 0) continue;
    const uintptr_t b = reinterpret_cast<uintptr_t>(grads[i]), end = b + size_t(counts[i]) * elt_bytes(dtypes[i]);
    // the written ranges do not overlap, so the last one that begins before `end` decides
    const Written* p = std::lower_bound(w, w + written, Written{end, 0, 0}, before);
    if (p == w) continue;
    --p;
    if (p->end > b && !(p->tensor == int32_t(i) && p->begin == b))
      return fail(NM_ERR_ALIAS, "tensor %lld overlaps an output of another, norm or workspace", (long long)i);
  }
  return NM_OK;
}

nm_status nm_grad_norm(const void* const* grads, const int64_t* counts, const int* dtypes, int64_t tensors, float* norm,
                       void* workspace, size_t workspace_bytes, void* stream) {
  nm_status st = check_grads(grads, counts, dtypes, tensors, nullptr, norm, workspace, workspace_bytes);
  if (st != NM_OK) return st;
  nm::GradArgs a;
  a.grads = grads;
  a.counts = counts;
  a.dtypes = dtypes;
  a.tensors = tensors;
  a.norm = norm;
  a.workspace = workspace;
  return hip_status(nm::launch_grad(a, static_cast<hipStream_t>(stream)), "nm_grad_norm launch");
}

nm_status nm_grad_clip(const void* const* grads, const int64_t* counts, const int* dtypes, int64_t tensors,
                       double max_norm, double eps, void* const* out, float* norm, void* workspace,
                       size_t workspace_bytes, void* stream) {
  if (!(max_norm >= 0.0) || !(eps >= 0.0) || std::isinf(eps))
    return fail(NM_ERR_SHAPE, "max_norm = %g or eps = %g is negative or not a number", max_norm, eps);
  if (tensors > 0 && !out) return fail(NM_ERR_NULL, "out must be non-NULL (grads for in place)");
  nm_status st = check_grads(grads, counts, dtypes, tensors, out, norm, workspace, workspace_bytes);
  if (st != NM_OK) return st;
  nm::GradArgs a;
  a.grads = grads;
  a.out = out;
  a.counts = counts;
  a.dtypes = dtypes;
  a.tensors = tensors;
  a.clip = true;
  a.in_place = true;
  for (int64_t i = 0; i < tensors && a.in_place; ++i) a.in_place = counts[i] == 0 || out[i] == grads[i];
  a.max_norm = max_norm;
  a.eps = eps;
  a.norm = norm;
  a.workspace = workspace;
  return hip_status(nm::launch_grad(a, static_cast<hipStream_t>(stream)), "nm_grad_clip launch");
}

}  // extern "C"
