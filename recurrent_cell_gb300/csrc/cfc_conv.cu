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
// Memory is the bound, if the arithmetic (W + 10 operations a value, the gate's
// exponential and reciprocal among them) is taken two channels at a time.  A thread owns
// 16 bytes of channels (backward: 4 channels, for the registers of grad_w) and walks down
// a tile of rows with the last W - 1 rows in registers and the next kBatch in flight; a
// tile reads W - 1 rows of its neighbours' again, from cache.  The backward walks its rows
// once: p_t is formed as soon as row t is there, and grad_x follows W - 1 rows behind.
// Tiles are as long as the GPU has threads for; a backward tile is a row of partial grad_w
// that reduce_axis0 adds.  16384 x 4096 in bfloat16, 4 weights: 48 us forward (268 MB, 5.5 TB/s), 90
// backward (403 MB, 4.5 TB/s), where arithmetic takes half of the issue slots.
#include "pair_math.cuh"
#include "seq_rows.cuh"

namespace cfc {
namespace conv {

using namespace pairs;
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
constexpr int kBatch = 4;

// A thread's channels: N of type E, as pairs.
template <class E_, int N_>
struct Chan {
  using E = E_;
  static constexpr int N = N_, H = N / 2;
  using P = Pairs<E, N>;
  using T = typename P::T;
  __device__ static __forceinline__ void read(F2 (&f)[H], const void* p, long long at) {
    P::get(f, P::load(static_cast<const E*>(p) + at));
  }
  __device__ static __forceinline__ void write(void* p, long long at, const F2 (&f)[H]) {
    __stcs(reinterpret_cast<T*>(static_cast<E*>(p) + at), P::make(f));
  }
  __device__ static __forceinline__ F2 sigmoid(F2 v) { return sizeof(E) == 4 ? sigmoid2_exact(v) : sigmoid2(v); }
};

// The weights [channels, W] of channels c on, as pairs of channels.
template <class C, int W>
__device__ __forceinline__ void load_weights(const Args& a, int c, F2 (&w)[W][C::H], F2 (&b)[C::H]) {
  float f[C::N * W];
#pragma unroll
  for (int i = 0; i < C::N * W; i += 4) {    // (c is a multiple of 4, so c W floats are whole vectors)
    const float4 v = __ldg(reinterpret_cast<const float4*>(a.w + (long long)c * W + i));
    f[i] = v.x; f[i + 1] = v.y; f[i + 2] = v.z; f[i + 3] = v.w;
  }
#pragma unroll
  for (int e = 0; e < C::H; ++e) {
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][e] = pack(f[2 * e * W + j], f[(2 * e + 1) * W + j]);
    b[e] = a.b ? pack(__ldg(a.b + c + 2 * e), __ldg(a.b + c + 2 * e + 1)) : 0;
  }
}

// Row `at` (negative) of what lies before a sequence.
template <class C, int W>
__device__ __forceinline__ void state_at(const Args& a, int seq, int at, int c, F2 (&f)[C::H]) {
#pragma unroll
  for (int e = 0; e < C::H; ++e) f[e] = 0;
  if (a.init) C::read(f, a.init, ((long long)seq * (W - 1) + at + W - 1) * a.d + c);
}

// The W - 1 rows before `row`, h[W - 2] being the last.
template <class C, int W>
__device__ __forceinline__ void window(const Args& a, const Where& q, long long row, int c, F2 (&h)[W - 1][C::H]) {
#pragma unroll
  for (int j = 1; j < W; ++j) {
    if (row - j >= q.begin) C::read(h[W - 1 - j], a.x, (row - j) * a.ldx + c);
    else state_at<C, W>(a, q.i, (int)(row - q.begin) - j, c, h[W - 1 - j]);
  }
}

template <int W, int H>
__device__ __forceinline__ void pre_of(const F2 (&w)[W][H], const F2 (&b)[H], const F2 (&h)[W - 1][H], const F2 (&x)[H],
                                       F2 (&pre)[H]) {
#pragma unroll
  for (int e = 0; e < H; ++e) {
    pre[e] = b[e];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) pre[e] = fma2(w[j][e], h[j][e], pre[e]);
    pre[e] = fma2(w[W - 1][e], x[e], pre[e]);
  }
}
// The same from W rows of an array, x[i] being the first.
template <int W, int H, int R>
__device__ __forceinline__ void pre_at(const F2 (&w)[W][H], const F2 (&b)[H], const F2 (&x)[R][H], int i, F2 (&pre)[H]) {
#pragma unroll
  for (int e = 0; e < H; ++e) {
    pre[e] = b[e];
#pragma unroll
    for (int j = 0; j < W; ++j) pre[e] = fma2(w[j][e], x[i + j][e], pre[e]);
  }
}
template <int W, int H>
__device__ __forceinline__ void shift(F2 (&h)[W][H], const F2 (&x)[H]) {
#pragma unroll
  for (int e = 0; e < H; ++e) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) h[j][e] = h[j + 1][e];
    h[W - 1][e] = x[e];
  }
}

// The last W - 1 inputs of sequence seq, from its rows or the state before them.
template <class C, int W>
__device__ __forceinline__ void final_rows(const Args& a, int seq, int c) {
  long long begin, end;
  seqs::range_of(a.s, seq, &begin, &end);
  const long long len = end - begin;
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    const long long at = len - (W - 1) + i;
    F2 f[C::H];
    if (at >= 0) C::read(f, a.x, (begin + at) * a.ldx + c);
    else state_at<C, W>(a, seq, (int)at, c, f);
    C::write(a.final_state, ((long long)seq * (W - 1) + i) * a.d + c, f);
  }
}

template <class C, int W>
__global__ void __launch_bounds__(kThreads) k_conv(Args a) {
  using P = typename C::P;
  constexpr int H = C::H;
  const int nvec = a.d / C::N;
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long tile = id / nvec;
  const int c = (int)(id % nvec) * C::N;
  if (tile >= a.n_tiles) {                   // behind the tiles: the states
    const long long seq = tile - a.n_tiles;
    if (a.final_state && seq < a.s.n) final_rows<C, W>(a, (int)seq, c);
    return;
  }
  a.s = seqs::trim(a.s);
  const long long r0 = tile * a.tile, r1 = a.s.rows - r0 < a.tile ? a.s.rows : r0 + a.tile;
  if (r0 >= r1) return;                      // rows behind the last sequence
  typename C::T in[kBatch], next[kBatch];
  auto fetch = [&](long long row) {
    const typename C::E* p = static_cast<const typename C::E*>(a.x) + row * a.ldx + c;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) next[i] = P::load(p + i * a.ldx, row + i < r1);
  };
  fetch(r0);
  F2 w[W][H], b[H], h[W - 1][H];
  load_weights<C, W>(a, c, w, b);
  Where q = seqs::find(a.s, r0);
  window<C, W>(a, q, r0, c, h);
  for (long long row = r0; row < r1; row += kBatch) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) in[i] = next[i];
    fetch(row + kBatch);
    if (row + kBatch <= q.end && row + kBatch <= r1) {       // a whole batch of one sequence: no row asks
      F2 x[W - 1 + kBatch][H];
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int e = 0; e < H; ++e) x[j][e] = h[j][e];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        F2 pre[H];
        P::get(x[W - 1 + i], in[i]);
        pre_at<W, H>(w, b, x, i, pre);
        if (a.silu)
#pragma unroll
          for (int e = 0; e < H; ++e) pre[e] = mul2(pre[e], C::sigmoid(pre[e]));
        C::write(a.y, (row + i) * a.d + c, pre);
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int e = 0; e < H; ++e) h[j][e] = x[kBatch + j][e];
    } else {
#pragma unroll 1
      for (int i = 0; i < kBatch && row + i < r1; ++i) {
        if (row + i >= q.end) {              // the next sequence's first row
          q = seqs::find(a.s, row + i);
          window<C, W>(a, q, row + i, c, h);
        }
        F2 x[H], pre[H];
        C::read(x, a.x, (row + i) * a.ldx + c);
        pre_of<W, H>(w, b, h, x, pre);
        shift<W - 1, H>(h, x);
        if (a.silu)
#pragma unroll
          for (int e = 0; e < H; ++e) pre[e] = mul2(pre[e], C::sigmoid(pre[e]));
        C::write(a.y, (row + i) * a.d + c, pre);
      }
    }
  }
}

// p_t from pre_t and grad_y_t: act' = s (1 + pre (1 - s)) = s + pre s (1 - s).
template <class C>
__device__ __forceinline__ void p_of(int silu, const F2 (&pre)[C::H], const F2 (&gy)[C::H], F2 (&p)[C::H]) {
#pragma unroll
  for (int e = 0; e < C::H; ++e) {
    p[e] = gy[e];
    if (silu) {
      const F2 s = C::sigmoid(pre[e]);
      p[e] = mul2(p[e], fma2(mul2(pre[e], s), fma2(s, twice(-1.f), twice(1.f)), s));
    }
  }
}
// Adds to g the gradient that the state after sequence seq sends to its input of place `at`.
template <class C, int W>
__device__ __forceinline__ void add_final(const Args& a, int seq, long long at, long long len, int c, F2 (&g)[C::H]) {
  const long long i = at - (len - (W - 1));
  if (!a.grad_final || i < 0) return;
  F2 f[C::H];
  C::read(f, a.grad_final, ((long long)seq * (W - 1) + i) * a.d + c);
#pragma unroll
  for (int e = 0; e < C::H; ++e) g[e] = add2(g[e], f[e]);
}

// The gradient of the state before sequence seq: of its inputs of places -(W-1) .. -1.
template <class C, int W>
__device__ __forceinline__ void init_rows(const Args& a, int seq, int c) {
  constexpr int H = C::H;
  F2 w[W][H], b[H], h[W - 1][H], p[W - 1][H];
  load_weights<C, W>(a, c, w, b);
  long long begin, end;
  seqs::range_of(a.s, seq, &begin, &end);
  const long long len = end - begin;
#pragma unroll
  for (int j = 1; j < W; ++j) state_at<C, W>(a, seq, -j, c, h[W - 1 - j]);
#pragma unroll
  for (int t = 0; t < W - 1; ++t) {
#pragma unroll
    for (int e = 0; e < H; ++e) p[t][e] = 0;
    if (t < len) {
      F2 x[H], pre[H], gy[H];
      C::read(x, a.x, (begin + t) * a.ldx + c);
      C::read(gy, a.grad_y, (begin + t) * a.d + c);
      pre_of<W, H>(w, b, h, x, pre);
      shift<W - 1, H>(h, x);
      p_of<C>(a.silu, pre, gy, p[t]);
    }
  }
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    F2 g[H] = {};
#pragma unroll
    for (int k = 0; k <= i; ++k)
#pragma unroll
      for (int e = 0; e < H; ++e) g[e] = fma2(w[k][e], p[i - k][e], g[e]);
    add_final<C, W>(a, seq, i - (W - 1), len, c, g);
    C::write(a.grad_init, ((long long)seq * (W - 1) + i) * a.d + c, g);
  }
}

template <class C, int W>
__global__ void __launch_bounds__(kThreads) k_conv_bwd(Args a) {
  using P = typename C::P;
  constexpr int H = C::H;
  const int nvec = a.d / C::N;
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long tile = id / nvec;
  const int c = (int)(id % nvec) * C::N;
  if (tile >= a.n_tiles) {
    const long long seq = tile - a.n_tiles;
    if (a.grad_init && seq < a.s.n) init_rows<C, W>(a, (int)seq, c);
    return;
  }
  a.s = seqs::trim(a.s);
  const long long r0 = tile * a.tile, r1 = a.s.rows - r0 < a.tile ? a.s.rows : r0 + a.tile;
  float* part = a.part + tile * ((W + 1ll) * a.d);          // [grad_w | grad_b]
  if (r0 >= r1) {                            // rows behind the last sequence: sums of nothing
#pragma unroll
    for (int e = 0; e < C::N; ++e) {
#pragma unroll
      for (int j = 0; j < W; ++j) part[(long long)(c + e) * W + j] = 0.f;
      part[(long long)W * a.d + c + e] = 0.f;
    }
    return;
  }
  typename C::T in[kBatch], gin[kBatch], next[kBatch], gnext[kBatch];
  auto fetch = [&](long long row) {
    const typename C::E* p = static_cast<const typename C::E*>(a.x) + row * a.ldx + c;
    const typename C::E* g = static_cast<const typename C::E*>(a.grad_y) + row * a.d + c;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      next[i] = P::load(p + i * a.ldx, row + i < r1);
      gnext[i] = P::load(g + i * (long long)a.d, row + i < r1);
    }
  };
  fetch(r0);
  F2 w[W][H], b[H], h[W - 1][H], p[W][H] = {}, gw[W][H] = {}, gb[H] = {};
  load_weights<C, W>(a, c, w, b);
  Where q = seqs::find(a.s, r0);
  window<C, W>(a, q, r0, c, h);
  // p moved on by one row, and grad_x of the row that then has all of its W
  auto emit = [&](long long row, const F2 (&now)[H]) {
    shift<W, H>(p, now);
    const long long at = row - (W - 1);
    if (at < r0 || at < q.begin) return;
    F2 g[H] = {};
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int e = 0; e < H; ++e) g[e] = fma2(w[j][e], p[W - 1 - j][e], g[e]);
    add_final<C, W>(a, q.i, at - q.begin, q.end - q.begin, c, g);
    C::write(a.grad_x, at * a.d + c, g);
  };
  const F2 none[H] = {};
  for (long long row = r0; row < r1; row += kBatch) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      in[i] = next[i];
      gin[i] = gnext[i];
    }
    fetch(row + kBatch);
    const bool inside = row - (W - 1) >= r0 && row - (W - 1) >= q.begin;       // grad_x of all the batch's rows is due
    if (inside && row + kBatch <= q.end && row + kBatch <= r1) {
      F2 x[W - 1 + kBatch][H], pp[W - 1 + kBatch][H];
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int e = 0; e < H; ++e) {
          x[j][e] = h[j][e];
          pp[j][e] = p[j + 1][e];
        }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        F2 gy[H], pre[H], g[H];
        P::get(x[W - 1 + i], in[i]);
        P::get(gy, gin[i]);
        pre_at<W, H>(w, b, x, i, pre);
        p_of<C>(a.silu, pre, gy, pp[W - 1 + i]);
#pragma unroll
        for (int e = 0; e < H; ++e) {
#pragma unroll
          for (int j = 0; j < W; ++j) {
            gw[j][e] = fma2(pp[W - 1 + i][e], x[i + j][e], gw[j][e]);
            g[e] = j == 0 ? mul2(w[0][e], pp[W - 1 + i][e]) : fma2(w[j][e], pp[W - 1 + i - j][e], g[e]);
          }
          gb[e] = add2(gb[e], pp[W - 1 + i][e]);
        }
        C::write(a.grad_x, (row + i - (W - 1)) * a.d + c, g);
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int e = 0; e < H; ++e) {
          h[j][e] = x[kBatch + j][e];
          p[j + 1][e] = pp[kBatch + j][e];
        }
    } else {
#pragma unroll 1
      for (int i = 0; i < kBatch && row + i < r1; ++i) {
        if (row + i >= q.end) {              // the last rows of the one before, then the next sequence
#pragma unroll 1
          for (int k = 0; k < W - 1; ++k) emit(row + i + k, none);
          q = seqs::find(a.s, row + i);
          window<C, W>(a, q, row + i, c, h);
        }
        F2 x[H], gy[H], pre[H], now[H];
        C::read(x, a.x, (row + i) * a.ldx + c);
        C::read(gy, a.grad_y, (row + i) * a.d + c);
        pre_of<W, H>(w, b, h, x, pre);
        p_of<C>(a.silu, pre, gy, now);
#pragma unroll
        for (int e = 0; e < H; ++e) {
#pragma unroll
          for (int j = 0; j < W - 1; ++j) gw[j][e] = fma2(now[e], h[j][e], gw[j][e]);
          gw[W - 1][e] = fma2(now[e], x[e], gw[W - 1][e]);
          gb[e] = add2(gb[e], now[e]);
        }
        shift<W - 1, H>(h, x);
        emit(row + i, now);
      }
    }
  }
  // rows of the next tile, as far as they reach back into this one
#pragma unroll 1
  for (long long row = r1; row < r1 + W - 1; ++row) {
    F2 now[H] = {};
    if (row < q.end) {
      F2 x[H], gy[H], pre[H];
      C::read(x, a.x, row * a.ldx + c);
      C::read(gy, a.grad_y, row * a.d + c);
      pre_of<W, H>(w, b, h, x, pre);
      p_of<C>(a.silu, pre, gy, now);
      shift<W - 1, H>(h, x);
    }
    emit(row, now);
  }
#pragma unroll
  for (int e = 0; e < H; ++e) {
    float f[2];
#pragma unroll
    for (int j = 0; j < W; ++j) {
      split(gw[j][e], f[0], f[1]);
      part[(long long)(c + 2 * e) * W + j] = f[0];
      part[(long long)(c + 2 * e + 1) * W + j] = f[1];
    }
    split(gb[e], f[0], f[1]);
    part[(long long)W * a.d + c + 2 * e] = f[0];
    part[(long long)W * a.d + c + 2 * e + 1] = f[1];
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

template <class C, int W>
__global__ void __launch_bounds__(kThreads) k_conv_step(StepArgs g) {
  constexpr int H = C::H;
  const Args& a = g.a;
  const int nvec = a.d / C::N;
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long seq = id / nvec;
  const int c = (int)(id % nvec) * C::N;
  if (seq >= a.s.n) return;
  const long long slot = g.slots ? g.slots[seq] : seq, row0 = seq * g.tokens;
  if (slot < 0 || slot >= g.n_slots) {       // a sequence without a state: zeros out, nothing kept
    const F2 none[H] = {};
    for (int t = 0; t < g.tokens; ++t) C::write(a.y, (row0 + t) * a.d + c, none);
    return;
  }
  const long long at = slot * (W - 1) * a.d + c;
  F2 w[W][H], b[H], h[W - 1][H], x[H], pre[H];
  typename C::T s[W - 1];                    // (the state is written below: plain reads)
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
    s[j] = *reinterpret_cast<const typename C::T*>(static_cast<const typename C::E*>(g.state) + at + (long long)j * a.d);
  C::read(x, a.x, row0 * a.ldx + c);
  load_weights<C, W>(a, c, w, b);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) C::P::get(h[j], s[j]);
  for (int t = 0; t < g.tokens; ++t) {
    if (t > 0) C::read(x, a.x, (row0 + t) * a.ldx + c);
    pre_of<W, H>(w, b, h, x, pre);
    shift<W - 1, H>(h, x);
    if (a.silu)
#pragma unroll
      for (int e = 0; e < H; ++e) pre[e] = mul2(pre[e], C::sigmoid(pre[e]));
    C::write(a.y, (row0 + t) * a.d + c, pre);
  }
#pragma unroll
  for (int j = 0; j < W - 1; ++j) C::write(g.state, at + (long long)j * a.d, h[j]);
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

template <class C> struct Forward {
  Args& a; cudaStream_t st;
  template <int W> cudaError_t operator()() {
    const long long items = a.n_tiles + (a.final_state ? a.s.n : 0);
    if (items == 0) return cudaSuccess;
    TraceScope tr("k_conv", st);
    k_conv<C, W><<<blocks_of(items * (a.d / C::N)), kThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
};
template <class C> struct Backward {
  Args& a; cudaStream_t st;
  template <int W> cudaError_t operator()() {
    const long long items = a.n_tiles + (a.grad_init ? a.s.n : 0);
    if (items == 0) return cudaSuccess;
    TraceScope tr("k_conv_bwd", st);
    k_conv_bwd<C, W><<<blocks_of(items * (a.d / C::N)), kThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
};
template <class C> struct Step {
  StepArgs& g; cudaStream_t st;
  template <int W> cudaError_t operator()() {
    TraceScope tr("k_conv_step", st);
    k_conv_step<C, W><<<blocks_of((long long)g.a.s.n * (g.a.d / C::N)), kThreads, 0, st>>>(g);
    return cudaGetLastError();
  }
};

// Rows of a backward tile: as many threads as the GPU holds at once, 12 warps an SM up to 5
// weights a channel and 8 beyond, by their registers (16384 x 4096 in bf16, 4 weights: 12
// warps 92 us, 16, a second round of blocks, 116).
static int bwd_tile(long long rows, int d, int width) {
  const long long warps = width <= 5 ? 12 : 8;
  const long long tiles = (warps * 32 * kNumSMs + d / 4 - 1) / (d / 4);
  const long long n = (rows + tiles - 1) / tiles;
  return n < 16 ? 16 : (int)n;
}

// Rows of a forward tile: 16 warps an SM, what it holds at once up to 4 weights a channel and
// twice beyond (16384 x 4096 in bf16, 4 weights: 16 warps 48.5 us, 12 52.8, 32 52.0, tiles of 128 rows
// 52.0; 8 weights 69.8, 85, 82, 78), and a batch at least (64 rows: tiles of 4 4.9 us, of 16 7.2,
// of 128 13.2).
static int fwd_tile(long long rows, int vectors) {
  const long long tiles = 16ll * 32 * kNumSMs / vectors;
  const long long n = tiles < 1 ? rows : (rows + tiles - 1) / tiles;
  return n < 1 ? kBatch : (int)((n + kBatch - 1) / kBatch * kBatch);
}

static Args args_of(const ConvArgs& g) {
  Args a{};
  a.x = g.x; a.ldx = g.ldx; a.w = g.weight; a.b = g.bias; a.init = g.init; a.silu = g.silu; a.d = g.d;
  a.s = seqs::make_seqs(g.off, g.n_seq, g.rows);
  return a;
}

}  // namespace conv

size_t conv_workspace(long long rows, int d, int width) {
  const int tile = conv::bwd_tile(rows, d, width);
  const long long n = (rows + tile - 1) / tile;
  return ((size_t)(n > 0 ? n : 1) * (width + 1) * d * 4 + 255) & ~size_t(255);
}

cudaError_t launch_conv_forward(const ConvArgs& g, void* y, void* final_state, cudaStream_t st) {
  conv::Args a = conv::args_of(g);
  a.y = y;
  a.final_state = final_state;
  a.tile = conv::fwd_tile(g.rows, g.d / (g.math == CFC_MATH_BF16 ? 8 : 4));
  a.n_tiles = (int)((g.rows + a.tile - 1) / a.tile);
  return g.math == CFC_MATH_BF16 ? conv::by_width(g.width, conv::Forward<conv::Chan<__nv_bfloat16, 8>>{a, st})
                                 : conv::by_width(g.width, conv::Forward<conv::Chan<float, 4>>{a, st});
}

cudaError_t launch_conv_backward(const ConvArgs& g, const void* grad_y, const void* grad_final, void* grad_x, float* grad_w,
                                 float* grad_b, void* grad_init, float* part, cudaStream_t st) {
  conv::Args a = conv::args_of(g);
  a.grad_y = grad_y;
  a.grad_final = grad_final;
  a.grad_x = grad_x;
  a.grad_init = grad_init;
  a.part = part;
  a.tile = conv::bwd_tile(g.rows, g.d, g.width);
  a.n_tiles = (int)((g.rows + a.tile - 1) / a.tile);
  const cudaError_t e = g.math == CFC_MATH_BF16
                            ? conv::by_width(g.width, conv::Backward<conv::Chan<__nv_bfloat16, 4>>{a, st})
                            : conv::by_width(g.width, conv::Backward<conv::Chan<float, 4>>{a, st});
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
  return g.math == CFC_MATH_BF16 ? conv::by_width(g.width, conv::Step<conv::Chan<__nv_bfloat16, 8>>{s, st})
                                 : conv::by_width(g.width, conv::Step<conv::Chan<float, 4>>{s, st});
}

}  // namespace cfc
