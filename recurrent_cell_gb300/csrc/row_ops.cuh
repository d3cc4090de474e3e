// row_ops.cuh -- what the row norms share: vectors of a row in registers, sums
// and maxima over a row's lanes or block, how many blocks an SM holds.
#pragma once

#include <atomic>

#include "cfc_internal.cuh"

namespace cfc {
namespace rows {

// N elements that a thread loads at once.
template <class EL, int NE> struct Vec;
template <> struct Vec<float, 4> {
  using E = float;
  static constexpr int N = 4;
  using T = float4;
  __device__ static __forceinline__ void get(float (&f)[4], const float4& v) { f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w; }
  __device__ static __forceinline__ float4 make(const float (&f)[4]) { return make_float4(f[0], f[1], f[2], f[3]); }
  __device__ static __forceinline__ float round(float v) { return v; }
};
template <> struct Vec<__nv_bfloat16, 8> {
  using E = __nv_bfloat16;
  static constexpr int N = 8;
  using T = uint4;
  __device__ static __forceinline__ void get(float (&f)[8], const uint4& v) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  __device__ static __forceinline__ uint4 make(const float (&f)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
  __device__ static __forceinline__ float round(float v) { return round_bf16(v); }
};

template <> struct Vec<float, 1> {
  using E = float;
  static constexpr int N = 1;
  using T = float;
  __device__ static __forceinline__ void get(float (&f)[1], float v) { f[0] = v; }
  __device__ static __forceinline__ float make(const float (&f)[1]) { return f[0]; }
  __device__ static __forceinline__ float round(float v) { return v; }
};
template <> struct Vec<__nv_bfloat16, 1> {
  using E = __nv_bfloat16;
  static constexpr int N = 1;
  using T = unsigned short;
  __device__ static __forceinline__ void get(float (&f)[1], unsigned short v) { f[0] = __uint_as_float((uint32_t)v << 16); }
  __device__ static __forceinline__ unsigned short make(const float (&f)[1]) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
  }
  __device__ static __forceinline__ float round(float v) { return round_bf16(v); }
};
template <class E> constexpr int kVecN = 16 / sizeof(E);

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float max_nan(float a, float b) {    // a NaN stays
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

struct Sum { __device__ static __forceinline__ float of(float a, float b) { return a + b; } };
struct Max { __device__ static __forceinline__ float of(float a, float b) { return max_nan(a, b); } };

// Over a row: a warp's shuffles and, where the row is a block's, its warps'
// values through `part`, two buffers in turn, so one barrier is enough.  The
// places of warps that the block lacks hold zeros, which both sums and maxima
// of magnitudes leave out.
constexpr int kWarps = 16;
struct Part {
  float4 v[2][kWarps / 4];
  __device__ __forceinline__ void clear() {
    if (threadIdx.x < 2 * kWarps) reinterpret_cast<float*>(v)[threadIdx.x] = 0.f;
    __syncthreads();
  }
};
// LANES: of the warp that share the row; 0: the block's.
template <class Op, int LANES>
__device__ __forceinline__ float over_row(float v, Part& part, int& turn) {
#pragma unroll
  for (int m = (LANES ? LANES : 32) / 2; m > 0; m >>= 1) v = Op::of(v, __shfl_xor_sync(0xffffffffu, v, m));
  if constexpr (LANES == 0) {
    if ((threadIdx.x & 31) == 0) reinterpret_cast<float*>(part.v[turn])[threadIdx.x >> 5] = v;
    __syncthreads();
    float4 x[kWarps / 4];
#pragma unroll
    for (int i = 0; i < kWarps / 4; ++i) x[i] = part.v[turn][i];
#pragma unroll
    for (int i = 0; i < kWarps / 4; ++i) x[i].x = Op::of(Op::of(x[i].x, x[i].y), Op::of(x[i].z, x[i].w));
    v = Op::of(Op::of(x[0].x, x[1].x), Op::of(x[2].x, x[3].x));
    turn ^= 1;
  }
  return v;
}

constexpr int kLaneThreads = 256;      // threads of a block whose rows are lanes of its warps
template <int LANES> constexpr int kRows = LANES ? kLaneThreads / (LANES ? LANES : 1) : 1;

// A thread's vectors of a row: j * L + l, L the threads of the row.
template <class V, int NV, int LANES>
struct Row {
  using E = typename V::E;
  using T = typename V::T;
  static constexpr int N = V::N;
  int l, L, nvec;
  __device__ __forceinline__ Row(int d) {
    L = LANES ? LANES : blockDim.x;
    l = LANES ? threadIdx.x % (LANES ? LANES : 1) : threadIdx.x;
    nvec = d / N;
  }
  __device__ __forceinline__ int at(int j) const { return j * L + l; }
  __device__ __forceinline__ bool in(int j) const { return at(j) < nvec; }
  __device__ __forceinline__ void load(T (&v)[NV], const void* p, long long row, long long rows, int d) const {
    const T* q = reinterpret_cast<const T*>(static_cast<const E*>(p) + row * d);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (row < rows && in(j)) v[j] = __ldcs(q + at(j));
  }
  __device__ __forceinline__ void weights(float (&w)[NV][N], const float* p) const {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if constexpr (N == 1) {
        w[j][0] = in(j) ? __ldg(p + at(j)) : 0.f;
      } else {
#pragma unroll
        for (int e = 0; e < N; e += 4) {
          const float4 f = in(j) ? __ldg(reinterpret_cast<const float4*>(p + at(j) * N + e))
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
          w[j][e] = f.x; w[j][e + 1] = f.y; w[j][e + 2] = f.z; w[j][e + 3] = f.w;
        }
      }
  }
};

// Blocks of `kernel` that an SM holds at once (asked once for each block size).
template <auto KERNEL>
static int resident(int threads, size_t smem) {
  static std::atomic<int> known[kWarps + 1] = {};
  int n = known[threads / 32].load(std::memory_order_relaxed);
  if (n > 0) return n;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, KERNEL, threads, smem) != cudaSuccess || n < 1) n = 1;
  known[threads / 32].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace rows
}  // namespace cfc
