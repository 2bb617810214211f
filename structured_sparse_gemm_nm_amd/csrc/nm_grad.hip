// Global norm of the gradients in many tensors, and their clipping:
//   norm = sqrt(sum over every tensor of g^2),
//   out  = g min(1, max_norm / (norm + eps)).
//
// Both passes only move bytes, so what bounds them is HBM (and, for a list of
// small tensors, the launches).  A launch takes the addresses, counts and types
// of up to a few hundred tensors as its arguments: they need no table in device
// memory, and a captured graph keeps them.  Tensors are cut into chunks of 32 KB;
// workgroups walk the chunks of all tensors of a launch, so one large tensor and
// hundreds of small ones fill the chip alike.
//
// Squares are summed in 64 bits: they neither overflow nor vanish for any fp32
// gradient, and the vector ALUs do it several times faster than HBM delivers.
// Each workgroup leaves one partial sum; they are added in a fixed order, so equal
// calls give equal bits.  The clipping pass adds them in every workgroup itself,
// which is cheaper than one more launch, and walks the chunks backwards, so that
// what the first pass read last is still in the cache.
//
// 88 tensors, 1.62 GB of bf16: 270 us the norm (6.0 TB/s), 608 the clipping (5.3); 256
// tensors of 256 KB of fp32: 14 us and two launches of 16.
#include "nm_device.h"
#include "nm_internal.h"

namespace nm {
namespace {

constexpr int kThreads = 256;
constexpr int kChunkBytes = 32768;
constexpr int kVecs = kChunkBytes / 16 / kThreads;   // 16-byte vectors a thread holds of a chunk

// 16 bytes at any element's address.
typedef u32x4 __attribute__((aligned(2))) u32x4_any;

// Tensors of one launch, in as few bytes as hold them: kernel arguments end at 4 KB,
// and every launch costs 3 us of the host's time.
template <int N, bool OUT>
struct Batch {
  const void* p[N];
  void* out[OUT ? N : 1];
  uint32_t start[N + 1];   // first chunk; start[count] is the launch's number of chunks
  uint16_t tail[N];        // elements of the last chunk, less one
  uint8_t dtype[N];
  int count;
};
constexpr int kNormTensors = 262, kClipTensors = 170;
using NormBatch = Batch<kNormTensors, false>;
using ClipBatch = Batch<kClipTensors, true>;
static_assert(int64_t(kNormTensors) * (kGradMaxCount / (kChunkBytes / 4)) < 0xFFFF0000, "chunks of a launch");
static_assert(sizeof(NormBatch) <= 3968 && sizeof(ClipBatch) <= 3968, "kernel argument size");

constexpr int chunk_elements(int dtype) { return kChunkBytes / (dtype == NM_F32 ? 4 : 2); }

template <class B>
__device__ inline int64_t count_of(const B& b, int t) {
  return int64_t(b.start[t + 1] - b.start[t] - 1) * chunk_elements(b.dtype[t]) + b.tail[t] + 1;
}

template <class B>
__device__ inline int find(const B& b, uint32_t chunk) {
  int lo = 0, hi = b.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.start[mid] <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <int DT>
__device__ inline float element(const u32x4& v, int e) {
  if constexpr (DT == NM_F32) {
    const uint32_t bits = v[e];   // (a cast of v[e] itself reads v[0])
    return __builtin_bit_cast(float, bits);
  } else {
    return half_to_f32<DT>((v[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
  }
}

template <int DT>
__device__ inline float scalar(const void* p, int64_t i) {
  if constexpr (DT == NM_F32) return static_cast<const float*>(p)[i];
  else return half_to_f32<DT>(static_cast<const uint16_t*>(p)[i]);
}

template <int DT>
__device__ inline void put(void* p, int64_t i, float v) {
  if constexpr (DT == NM_F32) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = to_half_bits<DT>(v);
}

template <int DT>
constexpr int kPer = DT == NM_F32 ? 4 : 8;   // elements a vector

// The thread's share of a chunk's sum of squares.
template <int DT>
__device__ inline double chunk_squares(const void* p, int64_t n, int64_t chunk) {
  constexpr int E = kPer<DT>;
  const int64_t v0 = chunk * (kChunkBytes / 16) + threadIdx.x;
  const int64_t whole = n / E;
  const u32x4_any* src = static_cast<const u32x4_any*>(p);
  u32x4 v[kVecs];
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    v[j] = u32x4{0u, 0u, 0u, 0u};
    if (v0 + j * kThreads < whole) v[j] = src[v0 + j * kThreads];
  }
  double s = 0.0;
#pragma unroll
  for (int j = 0; j < kVecs; ++j)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const double x = double(element<DT>(v[j], e));
      s = __builtin_fma(x, x, s);
    }
  // the last elements, fewer than a vector, by the thread whose vector they begin
  if (whole >= v0 && whole < v0 + kVecs * kThreads && (whole - v0) % kThreads == 0)
    for (int64_t i = whole * E; i < n; ++i) {
      const double x = double(scalar<DT>(p, i));
      s = __builtin_fma(x, x, s);
    }
  return s;
}

template <int W>
__device__ inline double wave_sum(double s) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
  return s;
}

// The sum over the workgroup, in every thread; `red` holds one double a wave.
template <int THREADS>
__device__ inline double block_sum(double s, double* red) {
  s = wave_sum<64>(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  s = red[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) s += red[w];
  return s;
}

__global__ __launch_bounds__(kThreads) void grad_norm_kernel(const NormBatch b, double* __restrict__ partial) {
  __shared__ double red[kThreads / 64];
  const uint32_t chunks = b.start[b.count];
  uint32_t c = blockIdx.x;
  int t = find(b, c);
  double s = 0.0;
  for (; c < chunks; c += gridDim.x) {
    while (c >= b.start[t + 1]) ++t;
    const int64_t local = int64_t(c - b.start[t]);
    const void* p = b.p[t];
    const int64_t n = count_of(b, t);
    const int dt = b.dtype[t];
    if (dt == NM_F32) s += chunk_squares<NM_F32>(p, n, local);
    else if (dt == NM_BF16) s += chunk_squares<NM_BF16>(p, n, local);
    else s += chunk_squares<NM_F16>(p, n, local);
  }
  s = block_sum<kThreads>(s, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// The sum of all partial sums, in one order whatever the workgroup.
template <int THREADS>
__device__ inline double total_of(const double* __restrict__ partial, int slots, double* red) {
  double s = 0.0;
  for (int i = threadIdx.x; i < slots; i += THREADS) s += partial[i];
  return block_sum<THREADS>(s, red);
}

// Norm alone, or many partial sums into one (total).
__global__ __launch_bounds__(1024) void grad_finish_kernel(const double* __restrict__ partial, int slots,
                                                           float* __restrict__ norm, double* __restrict__ total) {
  __shared__ double red[16];
  const double s = total_of<1024>(partial, slots, red);
  if (threadIdx.x == 0) {
    if (norm) *norm = float(__builtin_sqrt(s));
    if (total) *total = s;
  }
}

template <int DT>
__device__ inline void chunk_scale(const void* p, void* out, int64_t n, int64_t chunk, float pre, float coef) {
  constexpr int E = kPer<DT>;
  const int64_t v0 = chunk * (kChunkBytes / 16) + threadIdx.x;
  const int64_t whole = n / E;
  const u32x4_any* src = static_cast<const u32x4_any*>(p);
  u32x4_any* dst = static_cast<u32x4_any*>(out);
  u32x4 v[kVecs];
#pragma unroll
  for (int j = 0; j < kVecs; ++j)
    if (v0 + j * kThreads < whole) v[j] = src[v0 + j * kThreads];
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    if (v0 + j * kThreads >= whole) continue;
    u32x4 o;
    if constexpr (DT == NM_F32) {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = __builtin_bit_cast(uint32_t, element<DT>(v[j], e) * pre * coef);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o[e] = pack_half2<DT>(element<DT>(v[j], 2 * e) * pre * coef, element<DT>(v[j], 2 * e + 1) * pre * coef);
    }
    __builtin_nontemporal_store(o, dst + v0 + j * kThreads);
  }
  if (whole >= v0 && whole < v0 + kVecs * kThreads && (whole - v0) % kThreads == 0)
    for (int64_t i = whole * E; i < n; ++i) put<DT>(out, i, scalar<DT>(p, i) * pre * coef);
}

__global__ __launch_bounds__(kThreads) void grad_clip_kernel(const ClipBatch b, const double* __restrict__ partial,
                                                             int slots, double max_norm, double eps, int in_place,
                                                             float* __restrict__ norm_out) {
  __shared__ double red[kThreads / 64];
  const double norm = __builtin_sqrt(total_of<kThreads>(partial, slots, red));
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = float(norm);
  // a NaN norm gives a NaN factor; nothing to divide by, or no limit (Inf / Inf), gives 1
  const bool one = norm + eps == 0.0 || (__builtin_isinf(max_norm) && __builtin_isinf(norm));
  const double ratio = one ? 1.0 : max_norm / (norm + eps);
  // a factor that fp32 holds with fewer bits, beside gradients near its end, goes in two
  const bool tiny = ratio < 0x1p-64;
  const float pre = tiny ? 0x1p-64f : 1.f;
  const float coef = ratio > 1.0 ? 1.f : float(tiny ? ratio * 0x1p64 : ratio);
  if (in_place && coef == 1.f) return;   // every gradient stays as it is
  const uint32_t chunks = b.start[b.count];
  if (blockIdx.x >= chunks) return;
  // the same chunks as a forward walk, last first
  uint32_t c = blockIdx.x + (chunks - 1 - blockIdx.x) / gridDim.x * gridDim.x;
  int t = find(b, c);
  while (true) {
    while (c < b.start[t]) --t;
    const int64_t local = int64_t(c - b.start[t]);
    const void* p = b.p[t];
    void* o = b.out[t];
    const int64_t n = count_of(b, t);
    const int dt = b.dtype[t];
    if (dt == NM_F32) chunk_scale<NM_F32>(p, o, n, local, pre, coef);
    else if (dt == NM_BF16) chunk_scale<NM_BF16>(p, o, n, local, pre, coef);
    else chunk_scale<NM_F16>(p, o, n, local, pre, coef);
    if (c < gridDim.x) break;
    c -= gridDim.x;
  }
}

// Workgroups of a launch: enough to fill the chip, and few enough partial sums
// for the clipping pass to add them itself.
constexpr int kMaxGrid = 2048;
constexpr int kSelfSum = 4096;   // partial sums a clipping workgroup still adds itself

// Fills b with the tensors from i on (empty ones are left out), up to its size;
// returns the next tensor.
template <class B, int N>
int64_t fill(B& b, const GradArgs& a, int64_t i) {
  b.count = 0;
  b.start[0] = 0;
  for (; i < a.tensors && b.count < N; ++i) {
    if (a.counts[i] == 0) continue;
    const int k = b.count++;
    b.p[k] = a.grads[i];
    if constexpr (sizeof(b.out) > sizeof(void*)) b.out[k] = a.out[i];
    const int64_t per = chunk_elements(a.dtypes[i]), chunks = (a.counts[i] + per - 1) / per;
    b.tail[k] = uint16_t(a.counts[i] - (chunks - 1) * per - 1);
    b.dtype[k] = uint8_t(a.dtypes[i]);
    b.start[k + 1] = b.start[k] + uint32_t(chunks);   // below 2^32: kGradMaxCount
  }
  return i;
}

}  // namespace

// One double a workgroup of every norm launch, and before them one for their total.
size_t grad_workspace(int64_t tensors) {
  return size_t((tensors + kNormTensors - 1) / kNormTensors) * kMaxGrid * sizeof(double) + 64;
}

hipError_t launch_grad(const GradArgs& a, hipStream_t s) {
  double* total = static_cast<double*>(a.workspace);
  double* partial = total + 8;
  int slots = 0;
  for (int64_t i = 0; i < a.tensors;) {
    NormBatch b;
    i = fill<NormBatch, kNormTensors>(b, a, i);
    if (b.count == 0) break;
    const uint32_t chunks = b.start[b.count];
    const int grid = int(chunks < uint32_t(kMaxGrid) ? chunks : uint32_t(kMaxGrid));
    hipLaunchKernelGGL(grad_norm_kernel, dim3(unsigned(grid)), dim3(kThreads), 0, s, b, partial + slots);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    slots += grid;
  }
  const bool self = a.clip && slots <= kSelfSum && slots > 0;
  if (!self) {
    hipLaunchKernelGGL(grad_finish_kernel, dim3(1), dim3(1024), 0, s, partial, slots, a.norm, total);
    if (hipError_t e = hipGetLastError(); e != hipSuccess || !a.clip) return e;
  }
  float* norm = self ? a.norm : nullptr;
  for (int64_t i = 0; i < a.tensors;) {
    ClipBatch b;
    i = fill<ClipBatch, kClipTensors>(b, a, i);
    if (b.count == 0) break;
    const uint32_t chunks = b.start[b.count];
    const int grid = int(chunks < uint32_t(kMaxGrid) ? chunks : uint32_t(kMaxGrid));
    hipLaunchKernelGGL(grad_clip_kernel, dim3(unsigned(grid)), dim3(kThreads), 0, s, b, self ? partial : total,
                       self ? slots : 1, double(a.max_norm), double(a.eps), a.in_place ? 1 : 0, norm);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    norm = nullptr;   // the first launch has written it
  }
  return hipSuccess;
}

}  // namespace nm
