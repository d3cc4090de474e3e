// cfc_conv.cu -- the short causal convolution of each channel over the rows of
// its sequence, forward, backward and for the next tokens.
//
//   pre_t = b + sum_j w_j x_{t-W+1+j},  y = pre sigmoid(pre) or pre
//   p_t = grad_y_t act'(pre_t),  grad_x_t = sum_j w_j p_{t+W-1-j}
//   grad_w_j = sum_t p_t x_{t-W+1+j},  grad_b = sum_t p_t
//
// Before a sequence's first row lie the W - 1 inputs of its state (or zeros); its
// state afterwards is its last W - 1 inputs.
//
// Memory is the bound, W + 10 operations a value or not.  A thread owns 16 bytes
// of channels (backward: 4 channels, for the registers of grad_w) and walks down a
// tile of rows with the last W - 1 rows in registers, the next kBatch rows in
// flight; a tile reads W - 1 rows of its neighbours' again, from cache.  The
// backward walks its rows once: p_t is formed as soon as row t is there, and
// grad_x follows W - 1 rows behind.  Its tiles are as long as the GPU has threads
// for, since each is a row of partial grad_w that reduce_axis0 adds.
#include "row_ops.cuh"
#include "seq_rows.cuh"

namespace cfc {
namespace conv {

using rows::Vec;
using seqs::Seqs;
using seqs::Where;

struct Args {
  const void *x, *grad_y, *init, *grad_final;
  const float *w, *b;
  void *y, *final_state, *grad_x, *grad_init;
  float* part;
  long long ldx;
  Seqs s;
  int d, silu, tile, n_tiles;
};

constexpr int kThreads = 128;
constexpr int kBatch = 8;
constexpr int kTileFwd = 32;                 // rows of a forward tile

// pre sigmoid(pre).  bf16: the fast exponential and division, good to 1e-6.
template <bool EXACT>
__device__ __forceinline__ float sigmoid(float v) {
  return EXACT ? 1.f / (1.f + expf(-v)) : __fdividef(1.f, 1.f + __expf(-v));
}

template <class V, int W>
__device__ __forceinline__ void load_weights(const Args& a, int c, float (&w)[W][V::N], float (&b)[V::N]) {
#pragma unroll
  for (int e = 0; e < V::N; ++e) {
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][e] = __ldg(a.w + (long long)(c + e) * W + j);
    b[e] = a.b ? __ldg(a.b + c + e) : 0.f;
  }
}

// N channels of a row of x; of row `at` (negative) of a sequence's state.
template <class V>
__device__ __forceinline__ typename V::T x_at(const Args& a, long long row, int c) {
  return __ldg(reinterpret_cast<const typename V::T*>(static_cast<const typename V::E*>(a.x) + row * a.ldx + c));
}
template <class V, int W>
__device__ __forceinline__ void state_at(const Args& a, int seq, int at, int c, float (&f)[V::N]) {
#pragma unroll
  for (int e = 0; e < V::N; ++e) f[e] = 0.f;
  if (a.init)
    V::get(f, __ldg(reinterpret_cast<const typename V::T*>(static_cast<const typename V::E*>(a.init) +
                                                             ((long long)seq * (W - 1) + at + W - 1) * a.d + c)));
}

// The W - 1 rows before `row`, h[W - 2] being the last.
template <class V, int W>
__device__ __forceinline__ void window(const Args& a, const Where& q, long long row, int c, float (&h)[W - 1][V::N]) {
#pragma unroll
  for (int j = 1; j < W; ++j) {
    if (row - j >= q.begin) V::get(h[W - 1 - j], x_at<V>(a, row - j, c));
    else state_at<V, W>(a, q.i, (int)(row - q.begin) - j, c, h[W - 1 - j]);
  }
}

template <class V, int W>
__device__ __forceinline__ void pre_of(const float (&w)[W][V::N], const float (&b)[V::N], const float (&h)[W - 1][V::N],
                                       const float (&x)[V::N], float (&pre)[V::N]) {
#pragma unroll
  for (int e = 0; e < V::N; ++e) {
    pre[e] = b[e];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) pre[e] = fmaf(w[j][e], h[j][e], pre[e]);
    pre[e] = fmaf(w[W - 1][e], x[e], pre[e]);
  }
}
template <int W, int N>
__device__ __forceinline__ void shift(float (&h)[W][N], const float (&x)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) h[j][e] = h[j + 1][e];
    h[W - 1][e] = x[e];
  }
}
template <class V>
__device__ __forceinline__ void activate(int silu, float (&v)[V::N]) {
  if (silu)
#pragma unroll
    for (int e = 0; e < V::N; ++e) v[e] *= sigmoid<sizeof(typename V::E) == 4>(v[e]);
}

// The last W - 1 inputs of sequence seq, from its rows or the state before them.
template <class V, int W>
__device__ __forceinline__ void final_rows(const Args& a, int seq, int c) {
  long long begin, end;
  seqs::range_of(a.s, seq, &begin, &end);
  const long long len = end - begin;
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    const long long at = len - (W - 1) + i;
    float f[V::N];
    if (at >= 0) V::get(f, x_at<V>(a, begin + at, c));
    else state_at<V, W>(a, seq, (int)at, c, f);
    *reinterpret_cast<typename V::T*>(static_cast<typename V::E*>(a.final_state) +
                                      ((long long)seq * (W - 1) + i) * a.d + c) = V::make(f);
  }
}

template <class V, int W>
__global__ void __launch_bounds__(kThreads) k_conv(Args a) {
  constexpr int N = V::N;
  const int nvec = a.d / N;
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long tile = id / nvec;
  const int c = (int)(id % nvec) * N;
  if (tile >= a.n_tiles) {                   // behind the tiles: the states
    const long long seq = tile - a.n_tiles;
    if (a.final_state && seq < a.s.n) final_rows<V, W>(a, (int)seq, c);
    return;
  }
  float w[W][N], b[N], h[W - 1][N];
  load_weights<V, W>(a, c, w, b);
  const long long r0 = tile * a.tile;
  const int n = a.s.rows - r0 < a.tile ? (int)(a.s.rows - r0) : a.tile;
  Where q = seqs::find(a.s, r0);
  window<V, W>(a, q, r0, c, h);
  typename V::E* y = static_cast<typename V::E*>(a.y) + r0 * a.d + c;
  for (int i0 = 0; i0 < n; i0 += kBatch) {
    typename V::T in[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (i0 + i < n) in[i] = x_at<V>(a, r0 + i0 + i, c);
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (i0 + i < n) {
        const long long row = r0 + i0 + i;
        if (row >= q.end) {                  // the next sequence's first row
          q = seqs::find(a.s, row);
          window<V, W>(a, q, row, c, h);
        }
        float x[N], pre[N];
        V::get(x, in[i]);
        pre_of<V, W>(w, b, h, x, pre);
        shift<W - 1, N>(h, x);
        activate<V>(a.silu, pre);
        __stcs(reinterpret_cast<typename V::T*>(y + (long long)(i0 + i) * a.d), V::make(pre));
      }
  }
}

// p_t from pre_t and grad_y_t.
template <class V>
__device__ __forceinline__ void p_of(int silu, const float (&pre)[V::N], const float (&gy)[V::N], float (&p)[V::N]) {
#pragma unroll
  for (int e = 0; e < V::N; ++e) {
    p[e] = gy[e];
    if (silu) {
      const float s = sigmoid<sizeof(typename V::E) == 4>(pre[e]);
      p[e] *= s * fmaf(pre[e], 1.f - s, 1.f);
    }
  }
}
template <class V>
__device__ __forceinline__ typename V::T gy_at(const Args& a, long long row, int c) {
  return __ldg(reinterpret_cast<const typename V::T*>(static_cast<const typename V::E*>(a.grad_y) + row * a.d + c));
}
// Adds to g the gradient that the state after sequence seq sends to its input of place `at`.
template <class V, int W>
__device__ __forceinline__ void add_final(const Args& a, int seq, long long at, long long len, int c, float (&g)[V::N]) {
  const long long i = at - (len - (W - 1));
  if (!a.grad_final || i < 0) return;
  float f[V::N];
  V::get(f, __ldg(reinterpret_cast<const typename V::T*>(static_cast<const typename V::E*>(a.grad_final) +
                                                           ((long long)seq * (W - 1) + i) * a.d + c)));
#pragma unroll
  for (int e = 0; e < V::N; ++e) g[e] += f[e];
}

// The gradient of the state before sequence seq: of its inputs of places -(W-1) .. -1.
template <class V, int W>
__device__ __forceinline__ void init_rows(const Args& a, int seq, int c) {
  constexpr int N = V::N;
  float w[W][N], b[N], h[W - 1][N], p[W - 1][N];
  load_weights<V, W>(a, c, w, b);
  Where q;
  q.i = seq;
  seqs::range_of(a.s, seq, &q.begin, &q.end);
  const long long len = q.end - q.begin;
#pragma unroll
  for (int j = 1; j < W; ++j) state_at<V, W>(a, seq, -j, c, h[W - 1 - j]);
#pragma unroll
  for (int t = 0; t < W - 1; ++t) {
#pragma unroll
    for (int e = 0; e < N; ++e) p[t][e] = 0.f;
    if (t < len) {
      float x[N], pre[N], gy[N];
      V::get(x, x_at<V>(a, q.begin + t, c));
      V::get(gy, gy_at<V>(a, q.begin + t, c));
      pre_of<V, W>(w, b, h, x, pre);
      shift<W - 1, N>(h, x);
      p_of<V>(a.silu, pre, gy, p[t]);
    }
  }
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    float g[N] = {};
#pragma unroll
    for (int k = 0; k <= i; ++k)
#pragma unroll
      for (int e = 0; e < N; ++e) g[e] = fmaf(w[k][e], p[i - k][e], g[e]);
    add_final<V, W>(a, seq, i - (W - 1), len, c, g);
    *reinterpret_cast<typename V::T*>(static_cast<typename V::E*>(a.grad_init) +
                                      ((long long)seq * (W - 1) + i) * a.d + c) = V::make(g);
  }
}

template <class V, int W>
__global__ void __launch_bounds__(kThreads) k_conv_bwd(Args a) {
  constexpr int N = V::N;
  const int nvec = a.d / N;
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long tile = id / nvec;
  const int c = (int)(id % nvec) * N;
  if (tile >= a.n_tiles) {
    const long long seq = tile - a.n_tiles;
    if (a.grad_init && seq < a.s.n) init_rows<V, W>(a, (int)seq, c);
    return;
  }
  float w[W][N], b[N], h[W - 1][N], p[W][N] = {}, gw[W][N] = {}, gb[N] = {};
  load_weights<V, W>(a, c, w, b);
  const long long r0 = tile * a.tile;
  const long long r1 = a.s.rows - r0 < a.tile ? a.s.rows : r0 + a.tile;
  Where q = seqs::find(a.s, r0);
  window<V, W>(a, q, r0, c, h);
  // p moved on by one row, and grad_x of the row that then has all of its W
  auto emit = [&](long long row, const float (&now)[N]) {
    shift<W, N>(p, now);
    const long long at = row - (W - 1);
    if (at < r0 || at < q.begin) return;
    float g[N] = {};
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int e = 0; e < N; ++e) g[e] = fmaf(w[j][e], p[W - 1 - j][e], g[e]);
    add_final<V, W>(a, q.i, at - q.begin, q.end - q.begin, c, g);
    __stcs(reinterpret_cast<typename V::T*>(static_cast<typename V::E*>(a.grad_x) + at * a.d + c), V::make(g));
  };
  const float none[N] = {};
  for (long long i0 = r0; i0 < r1; i0 += kBatch) {
    typename V::T in[kBatch], gin[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (i0 + i < r1) {
        in[i] = x_at<V>(a, i0 + i, c);
        gin[i] = gy_at<V>(a, i0 + i, c);
      }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (i0 + i < r1) {
        const long long row = i0 + i;
        if (row >= q.end) {                  // the last rows of the one before, then the next sequence
#pragma unroll 1
          for (int k = 0; k < W - 1; ++k) emit(row + k, none);
          q = seqs::find(a.s, row);
          window<V, W>(a, q, row, c, h);
        }
        float x[N], gy[N], pre[N], now[N];
        V::get(x, in[i]);
        V::get(gy, gin[i]);
        pre_of<V, W>(w, b, h, x, pre);
        p_of<V>(a.silu, pre, gy, now);
#pragma unroll
        for (int e = 0; e < N; ++e) {
#pragma unroll
          for (int j = 0; j < W - 1; ++j) gw[j][e] = fmaf(now[e], h[j][e], gw[j][e]);
          gw[W - 1][e] = fmaf(now[e], x[e], gw[W - 1][e]);
          gb[e] += now[e];
        }
        shift<W - 1, N>(h, x);
        emit(row, now);
      }
  }
  // rows of the next tile, as far as they reach back into this one
#pragma unroll 1
  for (long long row = r1; row < r1 + W - 1; ++row) {
    float now[N] = {};
    if (row < q.end) {
      float x[N], gy[N], pre[N];
      V::get(x, x_at<V>(a, row, c));
      V::get(gy, gy_at<V>(a, row, c));
      pre_of<V, W>(w, b, h, x, pre);
      p_of<V>(a.silu, pre, gy, now);
      shift<W - 1, N>(h, x);
    }
    emit(row, now);
  }
  float* part = a.part + tile * ((W + 1ll) * a.d);          // [grad_w | grad_b]
#pragma unroll
  for (int e = 0; e < N; ++e) {
#pragma unroll
    for (int j = 0; j < W; ++j) part[(long long)(c + e) * W + j] = gw[j][e];
    part[(long long)W * a.d + c + e] = gb[e];
  }
}

// The next tokens: a sequence's state is a slot of a pool, updated in place.
struct StepArgs {
  Args a;
  const int* slots;
  long long n_slots;
  void* state;
  int tokens;
};

template <class V, int W>
__global__ void __launch_bounds__(kThreads) k_conv_step(StepArgs g) {
  constexpr int N = V::N;
  using E = typename V::E;
  using T = typename V::T;
  const Args& a = g.a;
  const int nvec = a.d / N;
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long seq = id / nvec;
  const int c = (int)(id % nvec) * N;
  if (seq >= a.s.n) return;
  const long long slot = g.slots ? g.slots[seq] : seq;
  const bool on = slot >= 0 && slot < g.n_slots;
  float w[W][N], b[N], h[W - 1][N] = {};
  E* state = static_cast<E*>(g.state) + (on ? slot : 0) * (W - 1) * a.d + c;
  if (on) {
    load_weights<V, W>(a, c, w, b);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) V::get(h[j], *reinterpret_cast<const T*>(state + (long long)j * a.d));
  }
  for (int t = 0; t < g.tokens; ++t) {
    const long long row = seq * g.tokens + t;
    float x[N], pre[N] = {};
    if (on) {
      V::get(x, x_at<V>(a, row, c));
      pre_of<V, W>(w, b, h, x, pre);
      shift<W - 1, N>(h, x);
      activate<V>(a.silu, pre);
    }
    *reinterpret_cast<T*>(static_cast<E*>(a.y) + row * a.d + c) = V::make(pre);
  }
  if (on)
#pragma unroll
    for (int j = 0; j < W - 1; ++j) *reinterpret_cast<T*>(state + (long long)j * a.d) = V::make(h[j]);
}

template <class F>
static cudaError_t by_width(int w, F f) {
  switch (w) {
    case 2: return f.template operator()<2>();
    case 3: return f.template operator()<3>();
    case 4: return f.template operator()<4>();
    case 5: return f.template operator()<5>();
    case 6: return f.template operator()<6>();
    case 7: return f.template operator()<7>();
    case 8: return f.template operator()<8>();
  }
  return cudaErrorNotSupported;
}

static unsigned blocks_of(long long threads) { return (unsigned)((threads + kThreads - 1) / kThreads); }

template <class V> struct Forward {
  Args& a; cudaStream_t st;
  template <int W> cudaError_t operator()() {
    const long long items = a.n_tiles + (a.final_state ? a.s.n : 0);
    if (items == 0) return cudaSuccess;
    TraceScope tr("k_conv", st);
    k_conv<V, W><<<blocks_of(items * (a.d / V::N)), kThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
};
template <class V> struct Backward {
  Args& a; cudaStream_t st;
  template <int W> cudaError_t operator()() {
    const long long items = a.n_tiles + (a.grad_init ? a.s.n : 0);
    if (items == 0) return cudaSuccess;
    TraceScope tr("k_conv_bwd", st);
    k_conv_bwd<V, W><<<blocks_of(items * (a.d / V::N)), kThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
};
template <class V> struct Step {
  StepArgs& g; cudaStream_t st;
  template <int W> cudaError_t operator()() {
    TraceScope tr("k_conv_step", st);
    k_conv_step<V, W><<<blocks_of((long long)g.a.s.n * (g.a.d / V::N)), kThreads, 0, st>>>(g);
    return cudaGetLastError();
  }
};

// Rows of a backward tile: about 16 warps of threads an SM.
static int bwd_tile(long long rows, int d) {
  const long long tiles = (16ll * 32 * kNumSMs + d / 4 - 1) / (d / 4);
  const long long n = (rows + tiles - 1) / tiles;
  return n < 16 ? 16 : (int)n;
}

static Args args_of(const ConvArgs& g) {
  Args a{};
  a.x = g.x; a.ldx = g.ldx; a.w = g.weight; a.b = g.bias; a.init = g.init; a.silu = g.silu; a.d = g.d;
  a.s = seqs::make_seqs(g.off, g.n_seq, g.rows);
  return a;
}

}  // namespace conv

size_t conv_workspace(long long rows, int d, int width) {
  const int tile = conv::bwd_tile(rows, d);
  const long long n = (rows + tile - 1) / tile;
  return ((size_t)(n > 0 ? n : 1) * (width + 1) * d * 4 + 255) & ~size_t(255);
}

cudaError_t launch_conv_forward(const ConvArgs& g, void* y, void* final_state, cudaStream_t st) {
  conv::Args a = conv::args_of(g);
  a.y = y;
  a.final_state = final_state;
  a.tile = conv::kTileFwd;
  a.n_tiles = (int)((g.rows + a.tile - 1) / a.tile);
  return g.math == CFC_MATH_BF16 ? conv::by_width(g.width, conv::Forward<rows::Vec<__nv_bfloat16, 8>>{a, st})
                                 : conv::by_width(g.width, conv::Forward<rows::Vec<float, 4>>{a, st});
}

cudaError_t launch_conv_backward(const ConvArgs& g, const void* grad_y, const void* grad_final, void* grad_x, float* grad_w,
                                 float* grad_b, void* grad_init, float* part, cudaStream_t st) {
  conv::Args a = conv::args_of(g);
  a.grad_y = grad_y;
  a.grad_final = grad_final;
  a.grad_x = grad_x;
  a.grad_init = grad_init;
  a.part = part;
  a.tile = conv::bwd_tile(g.rows, g.d);
  a.n_tiles = (int)((g.rows + a.tile - 1) / a.tile);
  const cudaError_t e = g.math == CFC_MATH_BF16
                            ? conv::by_width(g.width, conv::Backward<rows::Vec<__nv_bfloat16, 4>>{a, st})
                            : conv::by_width(g.width, conv::Backward<rows::Vec<float, 4>>{a, st});
  if (e != cudaSuccess) return e;
  ReduceOut o{};
  o.nseg = grad_b ? 2 : 1;
  o.ptr[0] = grad_w;
  o.ptr[1] = grad_b;
  o.begin[1] = (long long)g.width * g.d;
  return launch_reduce(part, a.n_tiles, (long long)(g.width + (grad_b ? 1 : 0)) * g.d, (g.width + 1ll) * g.d, o, st);
}

cudaError_t launch_conv_step(const ConvArgs& g, int tokens, void* state, long long n_slots, const int* slots, void* y,
                             cudaStream_t st) {
  conv::StepArgs s{};
  s.a = conv::args_of(g);
  s.a.y = y;
  s.state = state;
  s.n_slots = n_slots;
  s.slots = slots;
  s.tokens = tokens;
  return g.math == CFC_MATH_BF16 ? conv::by_width(g.width, conv::Step<rows::Vec<__nv_bfloat16, 8>>{s, st})
                                 : conv::by_width(g.width, conv::Step<rows::Vec<float, 4>>{s, st});
}

}  // namespace cfc
