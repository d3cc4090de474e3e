// cfc_layernorm.cu -- layer norm of a residual stream, forward and backward.
//
//   s = round(x + residual)        (the stream, in the stored type)
//   mean = sum(s) / d,  rstd = 1 / sqrt(sum((s - mean)^2) / d + eps)
//   n = (s - mean) rstd,  y = n w + b
//   grad_s = grad_residual_out + rstd (dn - mean(dn) - n mean(dn n)),  dn = grad_y w
//   grad_w = sum over rows of grad_y n,  grad_b = sum over rows of grad_y
//
// As in the root-mean-square norm the stream is rounded before it is normalised,
// and everything else is fp32 and rounded once on its way out.  The variance is
// summed from s - mean, not from squares less the square of the mean: a row far
// from zero keeps its digits.
//
// Memory is the bound in both directions, so a row is read once and kept in
// registers (row_ops.cuh): 8 to 32 lanes a row up to 4 vectors of 16 bytes
// each, a block a row beyond that.  Rows that outgrow the registers (k_*_wide) are
// read two or three times, from L2 after the first, and their grad_w and grad_b
// come from a pass over columns.  The block's partial grad_w and grad_b are rows of
// the workspace that reduce_axis0 adds: no atomics, the same bits every time.
#include "pair_math.cuh"
#include "row_ops.cuh"

namespace cfc {
namespace ln {

using namespace rows;

struct Args {
  const void *x, *residual, *grad_y, *grad_s;
  const float *w, *b, *mean_in, *rstd_in;
  void *y, *s_out, *grad_x;
  float *mean, *rstd, *part;
  long long rows;
  int d;
  float eps;
};

// Arithmetic on a vector's values, two at a time where there are two: r = a op b.
template <int N, class F2op, class F1op>
__device__ __forceinline__ void each(F2op two, F1op one) {
  if constexpr (N == 1) {
    one(0);
  } else {
#pragma unroll
    for (int e = 0; e < N; e += 2) two(e);
  }
}
using pairs::F2;
template <int N> __device__ __forceinline__ F2 at2(const float (&f)[N], int e) { return pairs::pack(f[e], f[(e + 1) % N]); }
template <int N> __device__ __forceinline__ void to2(float (&f)[N], int e, F2 v) { pairs::split(v, f[e], f[(e + 1) % N]); }
template <int N>
__device__ __forceinline__ void add(float (&r)[N], const float (&a)[N], const float (&b)[N]) {
  each<N>([&](int e) { to2(r, e, pairs::add2(at2(a, e), at2(b, e))); }, [&](int) { r[0] = a[0] + b[0]; });
}
template <int N>
__device__ __forceinline__ void add(float (&r)[N], const float (&a)[N], float b) {
  each<N>([&](int e) { to2(r, e, pairs::add2(at2(a, e), pairs::twice(b))); }, [&](int) { r[0] = a[0] + b; });
}
template <int N>
__device__ __forceinline__ void mul(float (&r)[N], const float (&a)[N], float b) {
  each<N>([&](int e) { to2(r, e, pairs::mul2(at2(a, e), pairs::twice(b))); }, [&](int) { r[0] = a[0] * b; });
}
template <int N>
__device__ __forceinline__ void mul(float (&r)[N], const float (&a)[N], const float (&b)[N]) {
  each<N>([&](int e) { to2(r, e, pairs::mul2(at2(a, e), at2(b, e))); }, [&](int) { r[0] = a[0] * b[0]; });
}
template <int N>
__device__ __forceinline__ void fma(float (&r)[N], const float (&a)[N], const float (&b)[N], const float (&c)[N]) {
  each<N>([&](int e) { to2(r, e, pairs::fma2(at2(a, e), at2(b, e), at2(c, e))); }, [&](int) { r[0] = fmaf(a[0], b[0], c[0]); });
}
template <int N>
__device__ __forceinline__ void fma(float (&r)[N], const float (&a)[N], float b, const float (&c)[N]) {
  each<N>([&](int e) { to2(r, e, pairs::fma2(at2(a, e), pairs::twice(b), at2(c, e))); }, [&](int) { r[0] = fmaf(a[0], b, c[0]); });
}
template <int N>
__device__ __forceinline__ float sum(const float (&a)[N]) {
  float s[N];
#pragma unroll
  for (int e = 0; e < N; ++e) s[e] = a[e];
#pragma unroll
  for (int m = N / 2; m > 0; m >>= 1)
#pragma unroll
    for (int e = 0; e < m; ++e) s[e] += s[e + m];
  return s[0];
}

// Two sums over a row at once, after the manner of over_row.
struct __align__(16) Part2 {
  float2 v[2][kWarps];
  __device__ __forceinline__ void clear() {
    if (threadIdx.x < 2 * kWarps) v[0][threadIdx.x] = make_float2(0.f, 0.f);
    __syncthreads();
  }
};
template <int LANES>
__device__ __forceinline__ float2 over_row2(float2 v, Part2& part, int& turn) {
#pragma unroll
  for (int m = (LANES ? LANES : 32) / 2; m > 0; m >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, m);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, m);
  }
  if constexpr (LANES == 0) {
    if ((threadIdx.x & 31) == 0) part.v[turn][threadIdx.x >> 5] = v;
    __syncthreads();
    F2 s[2] = {};
#pragma unroll
    for (int i = 0; i < kWarps; i += 2) {
      const ulonglong2 p = *reinterpret_cast<const ulonglong2*>(&part.v[turn][i]);
      s[0] = pairs::add2(s[0], p.x);
      s[1] = pairs::add2(s[1], p.y);
    }
    pairs::split(pairs::add2(s[0], s[1]), v.x, v.y);
    turn ^= 1;
  }
  return v;
}

// A thread's vectors of the rows ahead, K tensors: 16-byte vectors are copied into shared memory, each thread
// its own, STAGES - 1 rows ahead (no registers, and no barrier, since nobody else reads them);
// single values, too small for such copies, one row ahead into registers.
template <class V, int NV, int LANES, int K, int STAGES>
struct Ahead {
  using R = Row<V, NV, LANES>;
  using T = typename V::T;
  static constexpr bool RING = V::N > 1;
  static constexpr int kBytes = RING ? STAGES * K * NV * 16 : 0;       // of shared memory, a thread
  T regs[K][RING ? 1 : NV];
  unsigned char* base;
  const T* from[K];                    // the thread's first vector of the row that is sent for next (NULL: no such tensor)
  int stage = 0;
  __device__ __forceinline__ uint4* at(int s, int k, int j) const {
    return reinterpret_cast<uint4*>(base) + ((s * K + k) * NV + j) * blockDim.x + threadIdx.x;
  }
  __device__ __forceinline__ void fetch(const R& r, bool on, long long step, int s) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (from[k]) {
        if (on) {
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            if constexpr (RING) {
              if (r.in(j)) pairs::copy16(at(s, k, j), from[k] + j * r.L, true);
            } else {
              if (r.in(j)) regs[k][j] = __ldcs(from[k] + j * r.L);
            }
          }
        }
        from[k] += step;
      }
    if constexpr (RING) pairs::copies_end();
  }
  // p: the tensors; step, in rows, from one row of the thread's to the next.
  __device__ __forceinline__ void start(const R& r, const void* const (&p)[K], long long row, long long step, long long rows, int d) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      from[k] = p[k] ? reinterpret_cast<const T*>(static_cast<const typename V::E*>(p[k]) + row * d) + r.l : nullptr;
#pragma unroll
    for (int s = 0; s < (RING ? STAGES - 1 : 1); ++s) fetch(r, row + s * step < rows, step * r.nvec, s);
  }
  // The row at hand into v; the row STAGES - 1 (1) steps on is sent for.
  __device__ __forceinline__ void next(const R& r, long long row, long long step, long long rows, T (&v)[K][NV]) {
    if constexpr (RING) {
      pairs::copies_wait<STAGES - 2>();
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (from[k])
#pragma unroll
          for (int j = 0; j < NV; ++j) v[k][j] = *reinterpret_cast<const T*>(at(stage, k, j));
      // into the stage that was read in the last round
      fetch(r, row + (STAGES - 1) * step < rows, step * r.nvec, stage == 0 ? STAGES - 1 : stage - 1);
      stage = stage == STAGES - 1 ? 0 : stage + 1;
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < NV; ++j) v[k][j] = regs[k][j];
      fetch(r, row + step < rows, step * r.nvec, 0);
    }
  }
};
template <class V, int NV, int LANES> using FwdAhead = Ahead<V, NV, LANES, 2, 3>;
template <class V, int NV, int LANES> using BwdAhead = Ahead<V, NV, LANES, 3, (NV > 2 ? 2 : 3)>;

template <class V, int NV, int LANES>
__global__ void __launch_bounds__(LANES ? kLaneThreads : 512) k_layernorm(Args a) {
  using R = Row<V, NV, LANES>;
  using E = typename V::E;
  using T = typename V::T;
  constexpr int N = V::N, RPB = kRows<LANES>;
  __shared__ Part part_;
  int turn = 0;
  if (!LANES) part_.clear();
  const R r(a.d);
  float w[NV][N], b[NV][N] = {};
  r.weights(w, a.w);
  if (LANES && a.b) r.weights(b, a.b);
  const float inv_d = 1.f / (float)a.d;
  const long long step = (long long)gridDim.x * RPB;
  long long row = (long long)blockIdx.x * RPB + (LANES ? threadIdx.x / (LANES ? LANES : 1) : 0);
  extern __shared__ __align__(16) unsigned char ring[];
  FwdAhead<V, NV, LANES> ahead;
  ahead.base = ring;
  const void* const in[2] = {a.x, a.residual};
  ahead.start(r, in, row, step, a.rows, a.d);
  // (the lanes of a warp whose rows are over stay for the others' shuffles)
  for (long long first = (long long)blockIdx.x * RPB; first < a.rows; first += step, row += step) {
    const bool on = row < a.rows;
    T v[2][NV];
    ahead.next(r, row, step, a.rows, v);
    float s[NV][N], part[N] = {};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int e = 0; e < N; ++e) s[j][e] = 0.f;
      if (on && r.in(j)) {
        V::get(s[j], v[0][j]);
        T stored = v[0][j];
        if (a.residual) {
          float t[N];
          V::get(t, v[1][j]);
          add(t, s[j], t);
          stored = V::make(t);               // rounded once, for the store and for what follows
          V::get(s[j], stored);
        }
        if (a.s_out) __stcs(reinterpret_cast<T*>(static_cast<E*>(a.s_out) + row * a.d) + r.at(j), stored);
      }
      add(part, part, s[j]);
    }
    const float mean = over_row<Sum, LANES>(sum(part), part_, turn) * inv_d;
    float sq[N] = {};
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (r.in(j)) {
        add(s[j], s[j], -mean);
        fma(sq, s[j], s[j], sq);
      }
    const float var = over_row<Sum, LANES>(sum(sq), part_, turn);
    if (!LANES && a.b) r.weights(b, a.b);        // from L1: kept, it would spill
    const float rstd = 1.f / sqrtf(fmaf(var, inv_d, a.eps));
    if (on && r.l == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (on && r.in(j)) {
        mul(s[j], s[j], rstd);
        fma(s[j], s[j], w[j], b[j]);
        __stcs(reinterpret_cast<T*>(static_cast<E*>(a.y) + row * a.d) + r.at(j), V::make(s[j]));
      }
  }
}

template <class V, int NV, int LANES>
__global__ void __launch_bounds__(LANES ? kLaneThreads : 512) k_layernorm_bwd(Args a) {
  using R = Row<V, NV, LANES>;
  using E = typename V::E;
  using T = typename V::T;
  constexpr int N = V::N, RPB = kRows<LANES>;
  extern __shared__ __align__(16) float sums[];  // the rows ahead; in the end [RPB][d] where a block has several rows
  __shared__ Part2 part;
  int turn = 0;
  if (!LANES) part.clear();
  const R r(a.d);
  float w[NV][N], gw[NV][N] = {}, gb[NV][N] = {};
  r.weights(w, a.w);
  const float inv_d = 1.f / (float)a.d;
  const long long step = (long long)gridDim.x * RPB;
  long long row = (long long)blockIdx.x * RPB + (LANES ? threadIdx.x / (LANES ? LANES : 1) : 0);
  BwdAhead<V, NV, LANES> ahead;
  ahead.base = reinterpret_cast<unsigned char*>(sums);
  const void* const in[3] = {a.x, a.grad_y, a.grad_s};
  ahead.start(r, in, row, step, a.rows, a.d);
  float mean = 0.f, rstd = 0.f;
  auto scalars = [&](long long row) {
    if (row < a.rows) {
      mean = a.mean_in[row];
      rstd = a.rstd_in[row];
    }
  };
  scalars(row);
  for (long long first = (long long)blockIdx.x * RPB; first < a.rows; first += step, row += step) {
    const bool on = row < a.rows;
    const long long at = row * a.d;
    const float rs = rstd, mu = mean;
    T v[3][NV];
    ahead.next(r, row, step, a.rows, v);
    scalars(row + step);
    // n = (s - mean) rstd, dn = grad_y w
    float sn[N] = {}, sg[N] = {}, n[NV][N], g[NV][N];
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (on && r.in(j)) {
        V::get(n[j], v[0][j]);
        V::get(g[j], v[1][j]);
        add(gb[j], gb[j], g[j]);
        add(n[j], n[j], -mu);
        mul(n[j], n[j], rs);
        fma(gw[j], g[j], n[j], gw[j]);
        mul(g[j], g[j], w[j]);
        add(sg, sg, g[j]);
        fma(sn, g[j], n[j], sn);
      }
    const float2 dot = over_row2<LANES>(make_float2(sum(sg), sum(sn)), part, turn);
    const float k = -rs * (dot.y * inv_d), l = -rs * (dot.x * inv_d);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (on && r.in(j)) {
        float o[N];
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] = l;
        fma(o, n[j], k, o);
        fma(o, g[j], rs, o);
        if (a.grad_s) {
          float t[N];
          V::get(t, v[2][j]);
          add(o, o, t);
        }
        __stcs(reinterpret_cast<T*>(static_cast<E*>(a.grad_x) + at) + r.at(j), V::make(o));
      }
  }
  if constexpr (BwdAhead<V, NV, LANES>::RING) pairs::copies_wait<0>();
  // The block's row of partial sums [grad_w | grad_b], its rows' lanes in order.
  float* out = a.part + (long long)blockIdx.x * 2 * a.d;
  if constexpr (LANES > 0) {
    for (int which = 0; which < 2; ++which, out += a.d) {
      float* to = sums + threadIdx.x / (LANES ? LANES : 1) * a.d;
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (r.in(j))
#pragma unroll
          for (int e = 0; e < N; ++e) to[r.at(j) * N + e] = which ? gb[j][e] : gw[j][e];
      __syncthreads();
      for (int i = threadIdx.x; i < a.d; i += kLaneThreads) {
        float v = sums[i];
        for (int g = 1; g < RPB; ++g) v += sums[g * a.d + i];
        out[i] = v;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (r.in(j)) {
        if constexpr (N == 1) {
          out[r.at(j)] = gw[j][0];
          out[a.d + r.at(j)] = gb[j][0];
        } else {
#pragma unroll
          for (int e = 0; e < N; e += 4) {
            *reinterpret_cast<float4*>(out + r.at(j) * N + e) = make_float4(gw[j][e], gw[j][e + 1], gw[j][e + 2], gw[j][e + 3]);
            *reinterpret_cast<float4*>(out + a.d + r.at(j) * N + e) =
                make_float4(gb[j][e], gb[j][e + 1], gb[j][e + 2], gb[j][e + 3]);
          }
        }
      }
  }
}

// Rows longer than the registers hold: a block a row, each row read again from
// cache for its next pass.  With a residual the stream is formed anew each time,
// from operands that residual_out (written last) may overlay.
constexpr int kWideThreads = 512;

template <class V>
__global__ void __launch_bounds__(kWideThreads) k_layernorm_wide(Args a) {
  using E = typename V::E;
  using T = typename V::T;
  constexpr int N = V::N;
  __shared__ Part part;
  int turn = 0;
  part.clear();
  const int nvec = a.d / N;
  const float inv_d = 1.f / (float)a.d;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = reinterpret_cast<const T*>(static_cast<const E*>(a.x) + row * a.d);
    const T* r = reinterpret_cast<const T*>(static_cast<const E*>(a.residual) + row * a.d);
    auto stream = [&](int i, float (&s)[N]) {
      V::get(s, x[i]);
      if (a.residual) {
        float t[N];
        V::get(t, r[i]);
#pragma unroll
        for (int e = 0; e < N; ++e) s[e] = V::round(s[e] + t[e]);
      }
    };
    float sum = 0.f, sq = 0.f, s[N];
    for (int i = threadIdx.x; i < nvec; i += kWideThreads) {
      stream(i, s);
#pragma unroll
      for (int e = 0; e < N; ++e) sum += s[e];
    }
    const float mean = over_row<Sum, 0>(sum, part, turn) * inv_d;
    for (int i = threadIdx.x; i < nvec; i += kWideThreads) {
      stream(i, s);
#pragma unroll
      for (int e = 0; e < N; ++e) sq = fmaf(s[e] - mean, s[e] - mean, sq);
    }
    sq = over_row<Sum, 0>(sq, part, turn);
    const float rstd = 1.f / sqrtf(fmaf(sq, inv_d, a.eps));
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    for (int i = threadIdx.x; i < nvec; i += kWideThreads) {
      float y[N];
      stream(i, s);
#pragma unroll
      for (int e = 0; e < N; ++e)
        y[e] = fmaf((s[e] - mean) * rstd, __ldg(a.w + i * N + e), a.b ? __ldg(a.b + i * N + e) : 0.f);
      reinterpret_cast<T*>(static_cast<E*>(a.y) + row * a.d)[i] = V::make(y);
      if (a.s_out) reinterpret_cast<T*>(static_cast<E*>(a.s_out) + row * a.d)[i] = V::make(s);
    }
  }
}

template <class V>
__global__ void __launch_bounds__(kWideThreads) k_layernorm_bwd_wide(Args a) {
  using E = typename V::E;
  using T = typename V::T;
  constexpr int N = V::N;
  __shared__ Part2 part;
  int turn = 0;
  part.clear();
  const int nvec = a.d / N;
  const float inv_d = 1.f / (float)a.d;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* sp = reinterpret_cast<const T*>(static_cast<const E*>(a.x) + row * a.d);
    const T* gp = reinterpret_cast<const T*>(static_cast<const E*>(a.grad_y) + row * a.d);
    const T* cp = reinterpret_cast<const T*>(static_cast<const E*>(a.grad_s) + row * a.d);
    const float mu = a.mean_in[row], rs = a.rstd_in[row];
    float2 dot = make_float2(0.f, 0.f);
    float n[N], g[N];
    for (int i = threadIdx.x; i < nvec; i += kWideThreads) {
      V::get(n, sp[i]);
      V::get(g, gp[i]);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        g[e] *= __ldg(a.w + i * N + e);
        dot.x += g[e];
        dot.y = fmaf(g[e], (n[e] - mu) * rs, dot.y);
      }
    }
    dot = over_row2<0>(dot, part, turn);
    dot.x *= inv_d;
    dot.y *= inv_d;
    for (int i = threadIdx.x; i < nvec; i += kWideThreads) {
      float o[N];
      V::get(n, sp[i]);
      V::get(g, gp[i]);
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = rs * (fmaf(g[e], __ldg(a.w + i * N + e), -dot.x) - (n[e] - mu) * rs * dot.y);
      if (a.grad_s) {
        float t[N];
        V::get(t, cp[i]);
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] += t[e];
      }
      reinterpret_cast<T*>(static_cast<E*>(a.grad_x) + row * a.d)[i] = V::make(o);
    }
  }
}

// grad_w and grad_b of wide rows: a block's columns over every gridDim.y-th row.
// Runs before the kernel above, whose grad_x may be the buffer of grad_y.
constexpr int kColThreads = 128;
template <class V>
__global__ void __launch_bounds__(kColThreads) k_layernorm_cols(Args a) {
  using E = typename V::E;
  using T = typename V::T;
  constexpr int N = V::N;
  const int i = blockIdx.x * kColThreads + threadIdx.x;
  if (i * N >= a.d) return;
  float gw[N] = {}, gb[N] = {};
#pragma unroll 4
  for (long long row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float mu = __ldg(a.mean_in + row), rs = __ldg(a.rstd_in + row);
    float n[N], g[N];
    V::get(n, __ldg(reinterpret_cast<const T*>(static_cast<const E*>(a.x) + row * a.d) + i));
    V::get(g, __ldg(reinterpret_cast<const T*>(static_cast<const E*>(a.grad_y) + row * a.d) + i));
#pragma unroll
    for (int e = 0; e < N; ++e) {
      gw[e] = fmaf(g[e], (n[e] - mu) * rs, gw[e]);
      gb[e] += g[e];
    }
  }
  float* out = a.part + (long long)blockIdx.y * 2 * a.d + i * N;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    out[e] = gw[e];
    out[a.d + e] = gb[e];
  }
}

constexpr int kMaxBlocks = 4 * kNumSMs;          // rows of partial sums at most

template <class V, int NV, int LANES>
static cudaError_t fwd(const Args& a, int threads, cudaStream_t st) {
  constexpr int RPB = kRows<LANES>;
  using Ring = FwdAhead<V, NV, LANES>;
  const size_t smem = (size_t)threads * Ring::kBytes;
  const cudaError_t e = allow_smem<k_layernorm<V, NV, LANES>>((LANES ? kLaneThreads : 512) * Ring::kBytes);
  if (e != cudaSuccess) return e;
  const long long need = (a.rows + RPB - 1) / RPB;
  const long long most = (long long)resident<&k_layernorm<V, NV, LANES>>(threads, smem) * kNumSMs;
  TraceScope tr("k_layernorm", st);
  k_layernorm<V, NV, LANES><<<(unsigned)(need < most ? need : most), threads, smem, st>>>(a);
  return cudaGetLastError();
}
template <class V, int NV, int LANES>
static cudaError_t bwd(const Args& a, int threads, int* blocks, cudaStream_t st) {
  constexpr int RPB = kRows<LANES>;
  using Ring = BwdAhead<V, NV, LANES>;
  size_t smem = (size_t)threads * Ring::kBytes;
  if (LANES && smem < (size_t)RPB * a.d * 4) smem = (size_t)RPB * a.d * 4;
  cudaError_t e = allow_smem<k_layernorm_bwd<V, NV, LANES>>((LANES ? kLaneThreads : 512) * Ring::kBytes);
  if (e != cudaSuccess) return e;
  const long long need = (a.rows + RPB - 1) / RPB;
  long long most = (long long)resident<&k_layernorm_bwd<V, NV, LANES>>(threads, smem) * kNumSMs;
  if (most > kMaxBlocks) most = kMaxBlocks;
  *blocks = (int)(need < most ? need : most);
  TraceScope tr("k_layernorm_bwd", st);
  k_layernorm_bwd<V, NV, LANES><<<*blocks, threads, smem, st>>>(a);
  return cudaGetLastError();
}

// The variant by row length, f.operator()<V, NV, LANES>(threads): the lanes that
// the root-mean-square norm measured for its rows, which differ from these in one
// sum more.  The backward keeps three values a column (w, grad_w, grad_b), so its
// registers end at 512 threads of 2 vectors; cudaErrorNotSupported beyond.
template <class V, bool BWD, class F>
static cudaError_t by_row(int d, F f) {
  const int nvec = d / V::N;
  auto threads = [&](int nv) { return ((nvec + nv - 1) / nv + 31) / 32 * 32; };
  if constexpr (V::N > 1) {
    if (nvec <= 16) return f.template operator()<V, 2, 8>(kLaneThreads);
    if (nvec <= 32) return f.template operator()<V, 2, 16>(kLaneThreads);
    if (nvec <= 64) return f.template operator()<V, 2, 32>(kLaneThreads);
    if (nvec <= 128) return f.template operator()<V, 4, 32>(kLaneThreads);
    if (threads(2) <= 512) return f.template operator()<V, 2, 0>(threads(2));
    if constexpr (!BWD)
      if (threads(4) <= 512) return f.template operator()<V, 4, 0>(threads(4));
  } else {
    if (threads(4) <= 128) return f.template operator()<V, 4, 0>(threads(4));
    if (threads(8) <= 512) return f.template operator()<V, 8, 0>(threads(8));
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

template <class V>
static cudaError_t forward(const Args& a, cudaStream_t st) {
  const cudaError_t e = by_row<V, false>(a.d, Fwd{a, st});
  if (e != cudaErrorNotSupported) return e;
  TraceScope tr("k_layernorm_wide", st);
  k_layernorm_wide<V><<<(unsigned)(a.rows < 4 * kNumSMs ? a.rows : 4 * kNumSMs), kWideThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <class V>
static cudaError_t backward(const Args& a, float* grad_w, float* grad_b, cudaStream_t st) {
  int blocks = 0;
  cudaError_t e = cudaSuccess;
  if (a.rows > 0) e = by_row<V, true>(a.d, Bwd{a, &blocks, st});    // rows = 0: sums of nothing
  if (e == cudaErrorNotSupported) {
    const int cols = (a.d / V::N + kColThreads - 1) / kColThreads;
    blocks = (8 * kNumSMs + cols - 1) / cols;
    if (blocks > kMaxBlocks) blocks = kMaxBlocks;
    if (blocks > a.rows) blocks = (int)a.rows;
    {
      TraceScope tr("k_layernorm_cols", st);
      k_layernorm_cols<V><<<dim3(cols, blocks), kColThreads, 0, st>>>(a);
    }
    TraceScope tr("k_layernorm_bwd_wide", st);
    k_layernorm_bwd_wide<V><<<(unsigned)(a.rows < 4 * kNumSMs ? a.rows : 4 * kNumSMs), kWideThreads, 0, st>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  ReduceOut o{};
  o.nseg = grad_b ? 2 : 1;
  o.ptr[0] = grad_w;
  o.ptr[1] = grad_b;
  o.begin[1] = a.d;
  return launch_reduce(a.part, blocks, grad_b ? 2ll * a.d : a.d, 2ll * a.d, o, st);
}

}  // namespace ln

size_t layernorm_workspace(long long rows, int d) {
  const long long n = rows < ln::kMaxBlocks ? rows : ln::kMaxBlocks;
  return ((size_t)(n > 0 ? n : 1) * 2 * d * 4 + 255) & ~size_t(255);
}

cudaError_t launch_layernorm_forward(const void* x, const void* residual, const float* w, const float* b, long long rows,
                                     int d, float eps, int math, void* y, void* residual_out, float* mean, float* rstd,
                                     cudaStream_t st) {
  ln::Args a{};
  a.x = x; a.residual = residual; a.w = w; a.b = b; a.rows = rows; a.d = d; a.eps = eps;
  a.y = y; a.s_out = residual_out; a.mean = mean; a.rstd = rstd;
  if (math == CFC_MATH_BF16) {
    using E = __nv_bfloat16;
    return d % 8 == 0 ? ln::forward<rows::Vec<E, 8>>(a, st) : ln::forward<rows::Vec<E, 1>>(a, st);
  }
  return d % 4 == 0 ? ln::forward<rows::Vec<float, 4>>(a, st) : ln::forward<rows::Vec<float, 1>>(a, st);
}

cudaError_t launch_layernorm_backward(const void* s, const float* w, const float* mean, const float* rstd,
                                      const void* grad_y, const void* grad_residual_out, long long rows, int d, int math,
                                      void* grad_x, float* grad_w, float* grad_b, float* part, cudaStream_t st) {
  ln::Args a{};
  a.x = s; a.w = w; a.mean_in = mean; a.rstd_in = rstd; a.grad_y = grad_y; a.grad_s = grad_residual_out; a.rows = rows;
  a.d = d; a.grad_x = grad_x; a.part = part;
  if (math == CFC_MATH_BF16) {
    using E = __nv_bfloat16;
    return d % 8 == 0 ? ln::backward<rows::Vec<E, 8>>(a, grad_w, grad_b, st)
                      : ln::backward<rows::Vec<E, 1>>(a, grad_w, grad_b, st);
  }
  return d % 4 == 0 ? ln::backward<rows::Vec<float, 4>>(a, grad_w, grad_b, st)
                    : ln::backward<rows::Vec<float, 1>>(a, grad_w, grad_b, st);
}

}  // namespace cfc
