// cfc_clip.cu -- the norm of many gradients together, and the gradients scaled to it.
//
//   norm = sqrt(sum over all tensors of g^2)
//   out  = g min(1, max_norm / (norm + 1e-6))
//
// Memory is the bound: one operation a value.  The tensors are cut into items of
// at most kItem values that a fixed grid takes in turn; the table of tensors is a kernel
// parameter, so a captured launch keeps it.  A thread adds the squares of its up to 128
// values of an item in fp32, its items in 64 bits, and a block writes one sum: no
// atomics, and an order that depends on the sizes alone.  Every block of the second
// kernel adds those sums in the same order, which costs it a few kilobytes from L2
// and saves a launch; it takes the items backwards, so that it first meets those
// that the first kernel left in L2.  (Those sums are of all tables of kTensors: beyond some thousands of
// tensors each launch reads ever more of them.)  588 million values of both types: 165 us for the norm (1.18 GB,
// 7.1 TB/s), 360 to scale (2.35 GB, 6.4 TB/s, a copy's rate); with items of 8192 values 585 us in all.
#include "row_ops.cuh"

namespace cfc {
namespace clip {

constexpr int kThreads = 256;
constexpr int kTensors = 512;                    // of a launch: 15 KB of parameters (a table of 64 is no faster)
constexpr int kItem = 32768, kSmallItem = 2048;  // values of an item: the most, the fewest
constexpr int kMaxBlocks = 6 * kNumSMs;          // partial sums of a launch
constexpr int kScaleBlocks = 8 * kNumSMs;

enum : uint8_t { kBf16 = 1, kVector = 2 };       // what a tensor's flag says

struct Table {
  const void* in[kTensors];
  void* out[kTensors];
  long long n[kTensors];
  int first[kTensors + 1];                            // items before the tensor
  int item;                                      // values of an item
  uint8_t flags[kTensors];
  int count;
};

// The tensor of an item: the last that starts at or before it.
__device__ __forceinline__ int tensor_of(const Table& t, int item) {
  int lo = 0, hi = t.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= item) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The squares of a thread's values of an item, in fp32; in 64 bits (noticing zeros)
// where fp32 would overflow or lose them.
__device__ __forceinline__ float square_to(float s, float f) { return fmaf(f, f, s); }
__device__ __forceinline__ double square_to(double s, float f) { return f == 0.f ? s : fma((double)f, (double)f, s); }
template <class S, class V>
__device__ __forceinline__ S squares_as(const void* in, int n) {
  const typename V::T* p = static_cast<const typename V::T*>(in);
  S s[4] = {};
  const int nv = n / V::N;
#pragma unroll 8
  for (int i = threadIdx.x; i < nv; i += kThreads) {
    float f[V::N];
    V::get(f, p[i]);
#pragma unroll
    for (int e = 0; e < V::N; ++e) s[e & 3] = square_to(s[e & 3], f[e]);
  }
  const int i = nv * V::N + threadIdx.x;         // fewer than a vector's values are left
  if (V::N > 1 && i < n) s[0] = square_to(s[0], rows::load1(static_cast<const typename V::E*>(in) + i));
  return (s[0] + s[1]) + (s[2] + s[3]);
}
template <class V>
__device__ __noinline__ double squares_wide(const void* in, int n) { return squares_as<double, V>(in, n); }
template <class V>
__device__ __forceinline__ double squares(const void* in, int n) {
  const float s = squares_as<float, V>(in, n);
  return s >= 1e-30f && s <= 1e37f ? s : squares_wide<V>(in, n);
}

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double part[kThreads / 32];
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int i = 1; i < kThreads / 32; ++i) v += part[i];
  return v;
}

using bf16 = __nv_bfloat16;
using Bf = rows::Vec<bf16, 8>;
using Fp = rows::Vec<float, 4>;
using Bf1 = rows::Vec<bf16, 1>;
using Fp1 = rows::Vec<float, 1>;

// Item `item`'s tensor, its place in it and its number of values.
struct Span {
  int k, n;
  long long at;
  uint8_t flags;
};
__device__ __forceinline__ Span span_of(const Table& t, int item) {
  Span s;
  s.k = tensor_of(t, item);
  s.at = (long long)(item - t.first[s.k]) * t.item;
  const long long left = t.n[s.k] - s.at;
  s.n = left < t.item ? (int)left : t.item;
  s.flags = t.flags[s.k];
  return s;
}

__global__ void __launch_bounds__(kThreads) k_grad_squares(const __grid_constant__ Table t, double* sums) {
  double sum = 0;
  const int items = t.first[t.count];
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const Span s = span_of(t, item);
    const char* p = static_cast<const char*>(t.in[s.k]) + s.at * (s.flags & kBf16 ? 2 : 4);
    if (s.flags & kVector) sum += s.flags & kBf16 ? squares<Bf>(p, s.n) : squares<Fp>(p, s.n);
    else sum += s.flags & kBf16 ? squares<Bf1>(p, s.n) : squares<Fp1>(p, s.n);
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) sums[blockIdx.x] = sum;
}

template <class V>
__device__ __forceinline__ void scale(const void* in, void* out, int n, float c) {
  const typename V::T* p = static_cast<const typename V::T*>(in);
  typename V::T* o = static_cast<typename V::T*>(out);
  const int nv = n / V::N;
#pragma unroll 4
  for (int i = threadIdx.x; i < nv; i += kThreads) {
    float f[V::N];
    V::get(f, __ldcs(p + i));
#pragma unroll
    for (int e = 0; e < V::N; ++e) f[e] *= c;
    __stcs(o + i, V::make(f));
  }
  const int i = nv * V::N + threadIdx.x;
  if (V::N > 1 && i < n)
    rows::store1(static_cast<typename V::E*>(out) + i, rows::load1(static_cast<const typename V::E*>(in) + i) * c);
}

// c = min(1, most / (norm + 1e-6)); a NaN stays one, and an infinite norm gives 0, but for
// most = infinity, which is 1 whatever the norm (the quotient of the two would be a NaN).
__global__ void __launch_bounds__(kThreads) k_grad_scale(const __grid_constant__ Table t, const double* sums, int n_sums,
                                                         float most, float* norm) {
  double v = 0;
  for (int i = threadIdx.x; i < n_sums; i += kThreads) v += sums[i];
  const float length = (float)sqrt(block_sum(v));
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = length;
  float c = most / (length + 1e-6f);
  if (c > 1.f || (isinf(most) && !isnan(length))) c = 1.f;
  const int items = t.first[t.count];
  for (int j = blockIdx.x; j < items; j += gridDim.x) {
    const Span s = span_of(t, items - 1 - j);
    const long long at = s.at * (s.flags & kBf16 ? 2 : 4);
    const char* p = static_cast<const char*>(t.in[s.k]) + at;
    char* o = static_cast<char*>(t.out[s.k]) + at;
    if (c == 1.f && p == o) continue;
    if (s.flags & kVector) s.flags & kBf16 ? scale<Bf>(p, o, s.n, c) : scale<Fp>(p, o, s.n, c);
    else s.flags & kBf16 ? scale<Bf1>(p, o, s.n, c) : scale<Fp1>(p, o, s.n, c);
  }
}

// Values of an item: as many as leave each SM four, within bounds (26 small
// tensors: 9.9 us in a graph of calls, 16.4 with items of 32768).
static int item_of(const long long* n, int count) {
  long long all = 0;
  for (int i = 0; i < count; ++i) all += n[i];
  int item = kItem;
  while (item > kSmallItem && all / item < 4 * kNumSMs) item /= 2;
  return item;
}

// `go` is given tables of up to kTensors tensors, in order.
template <class F>
static cudaError_t tables(const void* const* in, void* const* out, const long long* n, const int* math, int count, F go) {
  int at = 0;
  const int item = item_of(n, count);
  do {
    Table t;
    t.item = item;
    t.count = 0;
    t.first[0] = 0;
    for (; at < count && t.count < kTensors; ++at) {
      if (n[at] == 0) continue;
      const int j = t.count++;
      t.in[j] = in[at];
      t.out[j] = out ? out[at] : nullptr;
      t.n[j] = n[at];
      const uintptr_t bits = reinterpret_cast<uintptr_t>(t.in[j]) | reinterpret_cast<uintptr_t>(t.out[j]);
      t.flags[j] = (math[at] == CFC_MATH_BF16 ? kBf16 : 0) | (bits % 16 == 0 ? kVector : 0);
      t.first[j + 1] = t.first[j] + (int)((n[at] + item - 1) / item);   // kTensors x kMaxGradValues stay below 2^31
    }
    const cudaError_t e = go(t);
    if (e != cudaSuccess) return e;
  } while (at < count);
  return cudaSuccess;
}

static int grid_of(const Table& t, int most) {
  const int items = t.first[t.count];
  return items < 1 ? 1 : items < most ? items : most;
}

static cudaError_t run(const void* const* in, void* const* out, const long long* n, const int* math, int count, float most,
                       float* norm, double* sums, cudaStream_t st) {
  int n_sums = 0;
  cudaError_t e = tables(in, out, n, math, count, [&](const Table& t) {
    if (t.count == 0) return cudaSuccess;
    TraceScope tr("k_grad_squares", st);
    k_grad_squares<<<grid_of(t, kMaxBlocks), kThreads, 0, st>>>(t, sums + n_sums);
    n_sums += grid_of(t, kMaxBlocks);
    return cudaGetLastError();
  });
  if (e != cudaSuccess) return e;
  // (no table: one block that writes the norm)
  return tables(in, out, n, math, out ? count : 0, [&](const Table& t) {
    TraceScope tr("k_grad_scale", st);
    k_grad_scale<<<grid_of(t, kScaleBlocks), kThreads, 0, st>>>(t, sums, n_sums, most, norm);
    return cudaGetLastError();
  });
}

static_assert(kTensors * (kMaxGradValues / kItem + 1) < (1ll << 31), "items of a launch");

}  // namespace clip

size_t grad_workspace(int count) {
  return (size_t)(count / clip::kTensors + 1) * clip::kMaxBlocks * sizeof(double);     // the sums of each launch
}

cudaError_t launch_grad_norm(const void* const* in, void* const* out, const long long* n, const int* math, int count,
                             float most, float* norm, double* sums, cudaStream_t st) {
  return clip::run(in, out, n, math, count, most, norm, sums, st);
}

}  // namespace cfc
