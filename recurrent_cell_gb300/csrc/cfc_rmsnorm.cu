// cfc_rmsnorm.cu -- root-mean-square norm of a residual stream, forward and
// backward.
//
//   s = round(x + residual)        (the stream, in the stored type)
//   n = s rstd,  rstd = 1 / sqrt(mean(s^2) + eps),  y = n w
//   y8 = e4m3(y / c) with c = max|y| / 448 over each group of columns
//   grad_s = grad_residual_out + rstd (dn - n mean(dn n)),  dn = grad_y w
//   grad_w = sum over rows of grad_y n
//
// The stream is rounded before it is normalised: what the next layer adds to
// and what the backward reads is then what was normalised.  Everything else is
// fp32 and rounded once, on its way out.
//
// Memory is the bound in both directions (about one operation a byte), so a
// row is read once and kept in registers: 8 to 32 lanes a row up to 4 vectors
// of 16 bytes each, a block a row beyond that, of as many warps as leave each
// thread 4 (backward, where that fits: 2) vectors.  Rows that are no whole number of vectors go
// element by element in the same way.  Blocks are persistent: they keep their
// columns' weights, and in the backward their columns' grad_w, in registers,
// and load the next row before they finish the present one.  bf16, 16383 x 2560:
// forward 52 us, 6.5 TB/s; backward 54 us, 6.2 TB/s; 8 bits out, 16384 x 4096:
// 74 us, 6.3 TB/s.
#include <cuda_fp8.h>

#include <atomic>

#include "cfc_internal.cuh"

namespace cfc {
namespace rms {

struct Args {
  const void *x, *residual, *grad_y, *grad_s;
  const float *w, *rstd_in;
  void *y, *s_out, *grad_x;
  float *rstd, *scale, *part;
  uint8_t* y8;
  long long rows;
  int d, group;
  float eps;
};

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

// c = max / 448, so that the largest value of the group becomes e4m3's largest;
// 1 for a group of zeros, and never below the smallest normal number.
__device__ __forceinline__ float scale_of(float most) {
  return most > 0.f ? fmaxf(most * (1.f / 448.f), 1.17549435e-38f) : (most == 0.f ? 1.f : most);
}
__device__ __forceinline__ float max_nan(float a, float b) {    // a NaN stays
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint8_t e4m3(float v) {
  return __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {  // a in the low byte
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
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

// Threads of a block at most: what leaves each the registers it needs.
template <class V, int NV, int LANES, bool BWD>
constexpr int most_threads() { return LANES ? kLaneThreads : (BWD && V::N > 1 && NV > 2 ? 384 : 512); }

template <class V, int NV, int LANES>
__global__ void __launch_bounds__(most_threads<V, NV, LANES, false>(), !LANES && NV * V::N <= 16 ? 2 : 1) k_rmsnorm(Args a) {
  using R = Row<V, NV, LANES>;
  using E = typename V::E;
  using T = typename V::T;
  constexpr int N = V::N, RPB = kRows<LANES>;
  __shared__ Part part;
  int turn = 0;
  if (!LANES) part.clear();
  const R r(a.d);
  float w[NV][N];
  r.weights(w, a.w);
  const float inv_d = 1.f / (float)a.d;
  const long long step = (long long)gridDim.x * RPB;
  long long row = (long long)blockIdx.x * RPB + (LANES ? threadIdx.x / (LANES ? LANES : 1) : 0);
  T xv[NV], rv[NV];
  r.load(xv, a.x, row, a.rows, a.d);
  if (a.residual) r.load(rv, a.residual, row, a.rows, a.d);
  // (the lanes of a warp whose rows are over stay for the others' shuffles)
  for (long long first = (long long)blockIdx.x * RPB; first < a.rows; first += step, row += step) {
    const bool on = row < a.rows;
    float s[NV][N];
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int e = 0; e < N; ++e) s[j][e] = 0.f;
      if (on && r.in(j)) {
        V::get(s[j], xv[j]);
        if (a.residual) {
          float t[N];
          V::get(t, rv[j]);
#pragma unroll
          for (int e = 0; e < N; ++e) s[j][e] = V::round(s[j][e] + t[e]);
        }
        if (a.s_out) __stcs(reinterpret_cast<T*>(static_cast<E*>(a.s_out) + row * a.d) + r.at(j), V::make(s[j]));
      }
#pragma unroll
      for (int e = 0; e < N; ++e) sq = fmaf(s[j][e], s[j][e], sq);
    }
    r.load(xv, a.x, row + step, a.rows, a.d);
    if (a.residual) r.load(rv, a.residual, row + step, a.rows, a.d);
    sq = over_row<Sum, LANES>(sq, part, turn);
    const float rstd = 1.f / sqrtf(fmaf(sq, inv_d, a.eps));
    if (a.rstd && on && r.l == 0) a.rstd[row] = rstd;
    float most = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        s[j][e] = s[j][e] * rstd * w[j][e];
        most = max_nan(most, fabsf(s[j][e]));
      }
      if (a.y && on && r.in(j)) __stcs(reinterpret_cast<T*>(static_cast<E*>(a.y) + row * a.d) + r.at(j), V::make(s[j]));
    }
    if (a.y8) {
      const int gl = a.group / N;       // threads that share a scale, unless the row does
      if (a.group == a.d) most = over_row<Max, LANES>(most, part, turn);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int at = r.at(j);
        float c = most;
        if (a.group != a.d) {
          c = 0.f;
#pragma unroll
          for (int e = 0; e < N; ++e) c = max_nan(c, fabsf(s[j][e]));
          for (int m = gl / 2; m > 0; m >>= 1) c = max_nan(c, __shfl_xor_sync(0xffffffffu, c, m));
        }
        c = scale_of(c);
        const float inv = 1.f / c;
        if (on && r.in(j)) {
          if (a.group == a.d ? at == 0 : (at & (gl - 1)) == 0) a.scale[row * (a.d / a.group) + at * N / a.group] = c;
          if constexpr (N == 1) {
            a.y8[row * a.d + at] = e4m3(s[j][0] * inv);
          } else {
            uint32_t u[N / 4];
#pragma unroll
            for (int e = 0; e < N / 4; ++e)
              u[e] = e4m3x2(s[j][4 * e] * inv, s[j][4 * e + 1] * inv) |
                     e4m3x2(s[j][4 * e + 2] * inv, s[j][4 * e + 3] * inv) << 16;
            uint32_t* p = reinterpret_cast<uint32_t*>(a.y8 + row * a.d + (long long)at * N);
            if constexpr (N == 8) __stcs(reinterpret_cast<uint2*>(p), make_uint2(u[0], u[1]));
            else __stcs(p, u[0]);
          }
        }
      }
    }
  }
}

template <class V, int NV, int LANES>
__global__ void __launch_bounds__(most_threads<V, NV, LANES, true>()) k_rmsnorm_bwd(Args a) {
  using R = Row<V, NV, LANES>;
  using E = typename V::E;
  using T = typename V::T;
  constexpr int N = V::N, RPB = kRows<LANES>;
  extern __shared__ float sums[];                // [RPB][d] where a block has several rows
  __shared__ Part part;
  int turn = 0;
  if (!LANES) part.clear();
  const R r(a.d);
  float w[NV][N], gw[NV][N] = {};
  r.weights(w, a.w);
  const float inv_d = 1.f / (float)a.d;
  const long long step = (long long)gridDim.x * RPB;
  long long row = (long long)blockIdx.x * RPB + (LANES ? threadIdx.x / (LANES ? LANES : 1) : 0);
  T sv[NV], gv[NV], rv[NV];
  float rstd = 0.f;
  auto fetch = [&](long long row) {
    r.load(sv, a.x, row, a.rows, a.d);
    r.load(gv, a.grad_y, row, a.rows, a.d);
    if (a.grad_s) r.load(rv, a.grad_s, row, a.rows, a.d);
    if (row < a.rows) rstd = a.rstd_in[row];
  };
  fetch(row);
  for (long long first = (long long)blockIdx.x * RPB; first < a.rows; first += step, row += step) {
    const bool on = row < a.rows;
    const long long at = row * a.d;
    T cs[NV], cg[NV], cv[NV];
    const float rs = rstd;
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      cs[j] = sv[j];
      cg[j] = gv[j];
      cv[j] = rv[j];
    }
    fetch(row + step);
    // n = s rstd, dn = grad_y w; formed twice rather than kept, for the registers
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (on && r.in(j)) {
        float n[N], g[N];
        V::get(n, cs[j]);
        V::get(g, cg[j]);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          n[e] *= rs;
          gw[j][e] = fmaf(g[e], n[e], gw[j][e]);
          dot = fmaf(g[e] * w[j][e], n[e], dot);
        }
      }
    dot = over_row<Sum, LANES>(dot, part, turn) * inv_d;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (on && r.in(j)) {
        float n[N], g[N], o[N];
        V::get(n, cs[j]);
        V::get(g, cg[j]);
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] = rs * (g[e] * w[j][e] - n[e] * rs * dot);
        if (a.grad_s) {
          float t[N];
          V::get(t, cv[j]);
#pragma unroll
          for (int e = 0; e < N; ++e) o[e] += t[e];
        }
        __stcs(reinterpret_cast<T*>(static_cast<E*>(a.grad_x) + at) + r.at(j), V::make(o));
      }
  }
  // The block's row of partial sums, its rows' lanes in order.
  float* out = a.part + (long long)blockIdx.x * a.d;
  float* to = LANES ? sums + threadIdx.x / (LANES ? LANES : 1) * a.d : out;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (r.in(j))
#pragma unroll
      for (int e = 0; e < N; ++e) to[r.at(j) * N + e] = gw[j][e];
  if constexpr (LANES > 0) {
    __syncthreads();
    for (int i = threadIdx.x; i < a.d; i += kLaneThreads) {
      float v = sums[i];
      for (int g = 1; g < RPB; ++g) v += sums[g * a.d + i];
      out[i] = v;
    }
  }
}

// Rows longer than the registers hold, and scales of other widths: one block a row, element by element, each row read again
// from cache for its second pass.
constexpr int kAnyThreads = 256;

template <class E>
__global__ void __launch_bounds__(kAnyThreads) k_rmsnorm_any(Args a) {
  __shared__ Part part;
  int turn = 0;
  part.clear();
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const E* x = static_cast<const E*>(a.x) + row * a.d;
    const E* r = static_cast<const E*>(a.residual) + row * a.d;
    auto stream = [&](int i) {
      float v = load1(x + i);
      if (a.residual) v = Vec<E, 1>::round(v + load1(r + i));
      return v;
    };
    float sq = 0.f;
    for (int i = threadIdx.x; i < a.d; i += kAnyThreads) {
      const float v = stream(i);
      sq = fmaf(v, v, sq);
    }
    sq = over_row<Sum, 0>(sq, part, turn);
    const float rstd = 1.f / sqrtf(fmaf(sq, 1.f / (float)a.d, a.eps));
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    for (int i = threadIdx.x; i < a.d; i += kAnyThreads) {
      const float v = stream(i);
      if (a.y) store1(static_cast<E*>(a.y) + row * a.d + i, v * rstd * a.w[i]);
      if (a.s_out && !a.y8) store1(static_cast<E*>(a.s_out) + row * a.d + i, v);
    }
    if (a.y8) {
      for (int g0 = 0; g0 < a.d; g0 += a.group) {
        float most = 0.f;
        for (int i = g0 + threadIdx.x; i < g0 + a.group; i += kAnyThreads)
          most = max_nan(most, fabsf(stream(i) * rstd * a.w[i]));
        most = scale_of(over_row<Max, 0>(most, part, turn));
        const float inv = 1.f / most;
        if (threadIdx.x == 0) a.scale[row * (a.d / a.group) + g0 / a.group] = most;
        for (int i = g0 + threadIdx.x; i < g0 + a.group; i += kAnyThreads) {
          const float v = stream(i);
          a.y8[row * a.d + i] = e4m3(v * rstd * a.w[i] * inv);
          if (a.s_out) store1(static_cast<E*>(a.s_out) + row * a.d + i, v);
        }
      }
    }
  }
}

template <class E>
__global__ void __launch_bounds__(kAnyThreads) k_rmsnorm_bwd_any(Args a) {
  extern __shared__ float gw[];                  // [d], thread i % 256 owns column i
  __shared__ Part part;
  int turn = 0;
  part.clear();
  for (int i = threadIdx.x; i < a.d; i += kAnyThreads) gw[i] = 0.f;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const E* s = static_cast<const E*>(a.x) + row * a.d;
    const E* gy = static_cast<const E*>(a.grad_y) + row * a.d;
    const float rstd = a.rstd_in[row];
    float dot = 0.f;
    for (int i = threadIdx.x; i < a.d; i += kAnyThreads) {
      const float n = load1(s + i) * rstd, g = load1(gy + i);
      gw[i] = fmaf(g, n, gw[i]);
      dot = fmaf(g * a.w[i], n, dot);
    }
    dot = over_row<Sum, 0>(dot, part, turn) / (float)a.d;
    for (int i = threadIdx.x; i < a.d; i += kAnyThreads) {
      float o = rstd * (load1(gy + i) * a.w[i] - load1(s + i) * rstd * dot);
      if (a.grad_s) o += load1(static_cast<const E*>(a.grad_s) + row * a.d + i);
      store1(static_cast<E*>(a.grad_x) + row * a.d + i, o);
    }
  }
  for (int i = threadIdx.x; i < a.d; i += kAnyThreads) a.part[(long long)blockIdx.x * a.d + i] = gw[i];
}

// Blocks of the backward: at most kMaxBlocks rows of partial sums.
constexpr int kMaxBlocks = 4 * kNumSMs;

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

template <class V, int NV, int LANES>
static cudaError_t fwd(const Args& a, int threads, cudaStream_t st) {
  constexpr int RPB = kRows<LANES>;
  const long long need = (a.rows + RPB - 1) / RPB, most = (long long)resident<&k_rmsnorm<V, NV, LANES>>(threads, 0) * kNumSMs;
  TraceScope tr("k_rmsnorm", st);
  k_rmsnorm<V, NV, LANES><<<(unsigned)(need < most ? need : most), threads, 0, st>>>(a);
  return cudaGetLastError();
}
template <class V, int NV, int LANES>
static cudaError_t bwd(const Args& a, int threads, int* blocks, cudaStream_t st) {
  constexpr int RPB = kRows<LANES>;
  const size_t smem = LANES ? (size_t)RPB * a.d * 4 : 0;
  const long long need = (a.rows + RPB - 1) / RPB;
  long long most = (long long)resident<&k_rmsnorm_bwd<V, NV, LANES>>(threads, smem) * kNumSMs;
  if (most > kMaxBlocks) most = kMaxBlocks;
  *blocks = (int)(need < most ? need : most);
  TraceScope tr("k_rmsnorm_bwd", st);
  k_rmsnorm_bwd<V, NV, LANES><<<*blocks, threads, smem, st>>>(a);
  return cudaGetLastError();
}

// The variant by row length, f.operator()<V, NV, LANES>(threads).  `lanes`: at
// least so many lanes side by side (a scale's columns).  Both directions, bf16,
// a side against its neighbour: 65536 x 64 with 8 lanes a row 28 us, with 32 54;
// 65536 x 512 with a warp a row 97, a block 167; 16384 x 1024 with a warp and 4
// vectors a lane 61, a block 69; 16384 x 2560 with 2 vectors a thread 122, with 4
// in the backward too 132; forward alone, 8 bits out, 16384 x 8192: 2 vectors
// 167, 4 153.  What no variant's registers hold goes element by element, each row
// read twice (backward: FP32 from 6152 columns, bf16 from 12296; forward: FP32 from
// 8200, bf16 from 16392; rows that are no multiple of 8 from 8193).  That is a cliff:
// FP32 both ways, 16384 x 6144 510 us (475 by bytes), x 8192 1220 (634), x 12288 2400
// (951); scales of 256 of 4096 columns 457 us, of 128 96.
template <class V, bool BWD, class F>
static cudaError_t by_row(int d, int lanes, F f) {
  const int nvec = d / V::N;
  auto threads = [&](int nv) { return ((nvec + nv - 1) / nv + 31) / 32 * 32; };
  if constexpr (V::N > 1) {
    if (nvec <= 16 && lanes <= 8) return f.template operator()<V, 2, 8>(kLaneThreads);
    if (nvec <= 32 && lanes <= 16) return f.template operator()<V, 2, 16>(kLaneThreads);
    if (nvec <= 64) return f.template operator()<V, 2, 32>(kLaneThreads);
    if (nvec <= 128) return f.template operator()<V, 4, 32>(kLaneThreads);
    if constexpr (BWD)
      if (threads(2) <= most_threads<V, 2, 0, BWD>()) return f.template operator()<V, 2, 0>(threads(2));
    if (threads(4) <= most_threads<V, 4, 0, BWD>()) return f.template operator()<V, 4, 0>(threads(4));
  } else {
    if (threads(4) <= 128) return f.template operator()<V, 4, 0>(threads(4));
    if (threads(8) <= 256) return f.template operator()<V, 8, 0>(threads(8));
    if (threads(16) <= 512) return f.template operator()<V, 16, 0>(threads(16));
  }
  return cudaErrorNotSupported;
}

struct Fwd {
  const Args& a; cudaStream_t st;
  template <class V, int NV, int LANES> cudaError_t operator()(int threads) { return fwd<V, NV, LANES>(a, threads, st); }
};
struct Bwd {
  const Args& a; int* blocks; cudaStream_t st;
  template <class V, int NV, int LANES> cudaError_t operator()(int threads) {
    return bwd<V, NV, LANES>(a, threads, blocks, st);
  }
};

template <class E>
static cudaError_t forward(const Args& a, cudaStream_t st) {
  // scales of 32, 64 or 128 columns lie in neighbouring lanes
  constexpr int N = kVecN<E>;
  const bool parts = a.y8 && a.group != a.d;
  cudaError_t e = cudaErrorNotSupported;
  if (a.d % 8 == 0 && (!parts || a.group == 32 || a.group == 64 || a.group == 128))
    e = by_row<Vec<E, N>, false>(a.d, parts ? a.group / N : 0, Fwd{a, st});
  else if (!parts)
    e = by_row<Vec<E, 1>, false>(a.d, 0, Fwd{a, st});
  if (e != cudaErrorNotSupported) return e;
  TraceScope tr("k_rmsnorm_any", st);
  k_rmsnorm_any<E><<<(unsigned)(a.rows < 8 * kNumSMs ? a.rows : 8 * kNumSMs), kAnyThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <class E>
static cudaError_t backward(const Args& a, float* grad_w, cudaStream_t st) {
  int blocks = 0;
  cudaError_t e = cudaErrorNotSupported;
  if (a.rows == 0) e = cudaSuccess;              // grad_w = 0
  else if (a.d % 8 == 0) e = by_row<Vec<E, kVecN<E>>, true>(a.d, 0, Bwd{a, &blocks, st});
  else e = by_row<Vec<E, 1>, true>(a.d, 0, Bwd{a, &blocks, st});
  if (e == cudaErrorNotSupported) {
    const size_t bytes = (size_t)a.d * 4;
    e = allow_smem<k_rmsnorm_bwd_any<E>>(kMaxRmsWidth * sizeof(float));
    if (e != cudaSuccess) return e;
    blocks = (int)(a.rows < kMaxBlocks ? a.rows : kMaxBlocks);
    TraceScope tr("k_rmsnorm_bwd_any", st);
    k_rmsnorm_bwd_any<E><<<blocks, kAnyThreads, bytes, st>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  ReduceOut o{};
  o.nseg = 1;
  o.ptr[0] = grad_w;
  return launch_reduce(a.part, blocks, a.d, a.d, o, st);
}

}  // namespace rms

size_t rmsnorm_workspace(long long rows, int d) {
  const long long n = rows < rms::kMaxBlocks ? rows : rms::kMaxBlocks;
  return ((size_t)(n > 0 ? n : 1) * d * 4 + 255) & ~size_t(255);
}

cudaError_t launch_rmsnorm_forward(const void* x, const void* residual, const float* w, long long rows, int d, float eps,
                                   int math, void* y, void* residual_out, float* rstd, uint8_t* y8, float* y8_scale,
                                   int group, cudaStream_t st) {
  rms::Args a{};
  a.x = x; a.residual = residual; a.w = w; a.rows = rows; a.d = d; a.eps = eps;
  a.y = y; a.s_out = residual_out; a.rstd = rstd; a.y8 = y8; a.scale = y8_scale; a.group = group;
  return math == CFC_MATH_BF16 ? rms::forward<__nv_bfloat16>(a, st) : rms::forward<float>(a, st);
}

cudaError_t launch_rmsnorm_backward(const void* s, const float* w, const float* rstd, const void* grad_y,
                                    const void* grad_residual_out, long long rows, int d, int math, void* grad_x,
                                    float* grad_w, float* part, cudaStream_t st) {
  rms::Args a{};
  a.x = s; a.w = w; a.rstd_in = rstd; a.grad_y = grad_y; a.grad_s = grad_residual_out; a.rows = rows; a.d = d;
  a.grad_x = grad_x; a.part = part;
  return math == CFC_MATH_BF16 ? rms::backward<__nv_bfloat16>(a, grad_w, st) : rms::backward<float>(a, grad_w, st);
}

}  // namespace cfc
