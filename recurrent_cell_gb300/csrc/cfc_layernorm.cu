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
// Memory is the bound in both directions, so a row is read once: 8 to 32 lanes a row up to 4
// vectors of 16 bytes each, a block a row beyond that (row_ops.cuh).  Vectors are copied into
// shared memory two rows ahead, each thread its own, and values go in pairs, since issue is
// the next bound: 16383 x 2560 in bfloat16 takes 55 us forward (6.1 TB/s) and 71 backward (4.7), with four
// blocks of five warps an SM (three, at 128 registers: 77); neither issue (64 and 61 %) nor DRAM (64 and 55 %)
// is at its end.  In fp32 119 us forward and 218 both ways, floors 99 and 198.
// Rows that outgrow the registers (k_*_wide) are
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

// A vector's values as the arithmetic takes them: pairs, or (rows of no whole vectors)
// one float.
using pairs::F2;
template <class V>
struct Vals {
  using X = F2;
  static constexpr int H = V::N / 2;
  using P = pairs::Pairs<typename V::E, V::N>;
  __device__ static __forceinline__ void get(F2 (&f)[H], const typename V::T& v) { P::get(f, *reinterpret_cast<const uint4*>(&v)); }
  __device__ static __forceinline__ typename V::T make(const F2 (&f)[H]) {
    const uint4 u = P::make(f);
    return *reinterpret_cast<const typename V::T*>(&u);
  }
};
template <class E>
struct Vals<Vec<E, 1>> {
  using X = float;
  static constexpr int H = 1;
  __device__ static __forceinline__ void get(float (&f)[1], const typename Vec<E, 1>::T& v) { Vec<E, 1>::get(f, v); }
  __device__ static __forceinline__ typename Vec<E, 1>::T make(const float (&f)[1]) { return Vec<E, 1>::make(f); }
};
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ F2 add(F2 a, F2 b) { return pairs::add2(a, b); }
__device__ __forceinline__ F2 mul(F2 a, F2 b) { return pairs::mul2(a, b); }
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) { return pairs::fma2(a, b, c); }
template <class X> __device__ __forceinline__ X all(float v) {
  if constexpr (sizeof(X) == 8) return pairs::twice(v);
  else return v;
}
template <int H> __device__ __forceinline__ float sum(const F2 (&a)[H]) {
  F2 s[H];
#pragma unroll
  for (int e = 0; e < H; ++e) s[e] = a[e];
#pragma unroll
  for (int m = H / 2; m > 0; m >>= 1)
#pragma unroll
    for (int e = 0; e < m; ++e) s[e] = pairs::add2(s[e], s[e + m]);
  return pairs::sum2(s[0]);
}
template <int H> __device__ __forceinline__ float sum(const float (&a)[H]) { return a[0]; }
// A row's weights of a thread.
template <class V, int NV, int LANES>
__device__ __forceinline__ void weights(const Row<V, NV, LANES>& r, typename Vals<V>::X (&w)[NV][Vals<V>::H], const float* p) {
  float f[NV][V::N];
  r.weights(f, p);
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if constexpr (V::N == 1) {
      w[j][0] = f[j][0];
    } else {
#pragma unroll
      for (int e = 0; e < V::N / 2; ++e) w[j][e] = pairs::pack(f[j][2 * e], f[j][2 * e + 1]);
    }
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
  // The row at hand once more, after next() (k, j: of its tensors and vectors).
  __device__ __forceinline__ T again(const T (&v)[K][NV], int k, int j) const {
    if constexpr (RING) return *reinterpret_cast<const T*>(at(stage == 0 ? STAGES - 1 : stage - 1, k, j));
    else return v[k][j];
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
__global__ void __launch_bounds__(LANES ? kLaneThreads : V::N > 1 && NV <= 2 ? 640 : 512) k_layernorm(Args a) {
  using R = Row<V, NV, LANES>;
  using E = typename V::E;
  using T = typename V::T;
  using X = typename Vals<V>::X;
  constexpr int H = Vals<V>::H, RPB = kRows<LANES>;
  __shared__ Part part_;
  int turn = 0;
  if (!LANES) part_.clear();
  const R r(a.d);
  X w[NV][H], b[NV][H] = {};
  weights<V, NV, LANES>(r, w, a.w);
  if (LANES && a.b) weights<V, NV, LANES>(r, b, a.b);
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
    X s[NV][H], part[H] = {};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int e = 0; e < H; ++e) s[j][e] = 0;
      if (on && r.in(j)) {
        Vals<V>::get(s[j], v[0][j]);
        T stored = v[0][j];
        if (a.residual) {
          X t[H];
          Vals<V>::get(t, v[1][j]);
#pragma unroll
          for (int e = 0; e < H; ++e) t[e] = add(s[j][e], t[e]);
          stored = Vals<V>::make(t);         // rounded once, for the store and for what follows
          Vals<V>::get(s[j], stored);
        }
        if (a.s_out) __stcs(reinterpret_cast<T*>(static_cast<E*>(a.s_out) + row * a.d) + r.at(j), stored);
      }
#pragma unroll
      for (int e = 0; e < H; ++e) part[e] = add(part[e], s[j][e]);
    }
    const float mean = over_row<Sum, LANES>(sum(part), part_, turn) * inv_d;
    X sq[H] = {};
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (r.in(j))
#pragma unroll
        for (int e = 0; e < H; ++e) {
          s[j][e] = add(s[j][e], all<X>(-mean));
          sq[e] = fma(s[j][e], s[j][e], sq[e]);
        }
    const float var = over_row<Sum, LANES>(sum(sq), part_, turn);
    if (!LANES && a.b) weights<V, NV, LANES>(r, b, a.b);     // from L1: kept, it would spill (4 vectors of bfloat16
                                                              // spill 176 bytes as it is)
    const float rstd = 1.f / sqrtf(fmaf(var, inv_d, a.eps));
    if (on && r.l == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (on && r.in(j)) {
#pragma unroll
        for (int e = 0; e < H; ++e) s[j][e] = fma(mul(s[j][e], all<X>(rstd)), w[j][e], b[j][e]);
        __stcs(reinterpret_cast<T*>(static_cast<E*>(a.y) + row * a.d) + r.at(j), Vals<V>::make(s[j]));
      }
  }
}

template <class V, int NV, int LANES>
__global__ void __launch_bounds__(LANES ? kLaneThreads : V::N > 1 ? 640 : 512) k_layernorm_bwd(Args a) {
  using R = Row<V, NV, LANES>;
  using E = typename V::E;
  using T = typename V::T;
  using X = typename Vals<V>::X;
  constexpr int N = V::N, H = Vals<V>::H, RPB = kRows<LANES>;
  extern __shared__ __align__(16) float sums[];  // the rows ahead; in the end [RPB][d] where a block has several rows
  __shared__ Part2 part;
  int turn = 0;
  if (!LANES) part.clear();
  const R r(a.d);
  X w[NV][H], gwx[NV][H] = {}, gbx[NV][H] = {};
  weights<V, NV, LANES>(r, w, a.w);
  const float inv_d = 1.f / (float)a.d;
  const long long step = (long long)gridDim.x * RPB;
  long long row = (long long)blockIdx.x * RPB + (LANES ? threadIdx.x / (LANES ? LANES : 1) : 0);
  BwdAhead<V, NV, LANES> ahead;
  ahead.base = reinterpret_cast<unsigned char*>(sums);
  const void* const in[3] = {a.x, a.grad_y, a.grad_s};
  ahead.start(r, in, row, step, a.rows, a.d);
  float mean, rstd;
  auto scalars = [&](long long row) {
    mean = pairs::load_here4(a.mean_in + row, row < a.rows);
    rstd = pairs::load_here4(a.rstd_in + row, row < a.rows);
  };
  scalars(row);
  for (long long first = (long long)blockIdx.x * RPB; first < a.rows; first += step, row += step) {
    const bool on = row < a.rows;
    pairs::use_here(mean);
    pairs::use_here(rstd);
    const float rs = rstd;
    const X mu = all<X>(-mean), rx = all<X>(rstd);
    T v[3][NV];
    ahead.next(r, row, step, a.rows, v);
    scalars(row + step);
    // n = (s - mean) rstd, dn = grad_y w; formed twice, from shared memory, rather than kept: with 96
    // registers a block of 5 warps fits an SM four times, with 128 three times
    X sn[H] = {}, sg[H] = {};
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (on && r.in(j)) {
        X n[H], g[H];
        Vals<V>::get(n, v[0][j]);
        Vals<V>::get(g, v[1][j]);
#pragma unroll
        for (int e = 0; e < H; ++e) {
          gbx[j][e] = add(gbx[j][e], g[e]);
          n[e] = mul(add(n[e], mu), rx);
          gwx[j][e] = fma(g[e], n[e], gwx[j][e]);
          g[e] = mul(g[e], w[j][e]);
          sg[e] = add(sg[e], g[e]);
          sn[e] = fma(g[e], n[e], sn[e]);
        }
      }
    const float2 dot = over_row2<LANES>(make_float2(sum(sg), sum(sn)), part, turn);
    // rs (dn - mean(dn) - n mean(dn n)) = rs dn + k (s - mu) + l
    const X k = all<X>(-rs * rs * (dot.y * inv_d)), l = all<X>(-rs * (dot.x * inv_d));
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (on && r.in(j)) {
        X n[H], g[H], o[H];
        Vals<V>::get(n, ahead.again(v, 0, j));
        Vals<V>::get(g, ahead.again(v, 1, j));
#pragma unroll
        for (int e = 0; e < H; ++e) o[e] = fma(mul(g[e], w[j][e]), rx, fma(add(n[e], mu), k, l));
        if (a.grad_s) {
          X t[H];
          Vals<V>::get(t, ahead.again(v, 2, j));
#pragma unroll
          for (int e = 0; e < H; ++e) o[e] = add(o[e], t[e]);
        }
        __stcs(reinterpret_cast<T*>(static_cast<E*>(a.grad_x) + row * a.d) + r.at(j), Vals<V>::make(o));
      }
  }
  float gw[NV][N], gb[NV][N];
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if constexpr (N == 1) {
      gw[j][0] = gwx[j][0];
      gb[j][0] = gbx[j][0];
    } else {
#pragma unroll
      for (int e = 0; e < H; ++e) {
        pairs::split(gwx[j][e], gw[j][2 * e], gw[j][2 * e + 1]);
        pairs::split(gbx[j][e], gb[j][2 * e], gb[j][2 * e + 1]);
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
