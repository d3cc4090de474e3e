// cfc_ssm_step.cu -- the selective scan for the next few tokens of many
// sequences, each with its state in a slot of a pool, updated in place.
//
// A step reads a state and writes it: 8 N bytes a channel, against an exponential and
// four multiply-adds a state, so memory is the floor.  A warp takes 32 channels: each
// lane forms dt, dt x and the gate of one of them, then eight channels at a time have four
// lanes each, with a quarter of the states in registers, and the sums over states
// come back to their channels' lanes.  Where there are sequences enough for every SM, a
// warp takes several with the same channels, so that A comes from L1 (192 sequences x 4096
// channels x 16 states: one a warp 32 us, 5 a warp 27).  Up to 16 states the next sequence is copied
// ahead into shared memory meanwhile (k_ssm_step_ahead): 23.4 us, 68 % of memory's rate, bound by instructions
// (596 a warp and sequence, 61 % of the issue slots) with the one round's start and end; 512 sequences 59 -> 54.  Ahead into registers it was slower (29), as were copies ahead of 32 states (42 -> 58): the
// blocks that fit are too few.
#include "ssm_common.cuh"

namespace cfc {
namespace ssm {

struct StepArgs {
  Args a;
  float* state;
  const int* slots;
  long long n_slots;
  int tokens, tiles, each;                     // tiles of 32 channels; sequences of a warp
};
constexpr int kStepThreads = 128;

// NS values of a lane's states of one row, zeros from `left` on.
template <class E, int NS, bool VEC>
__device__ __forceinline__ void lane_states(const E* p, int left, float (&f)[NS]) {
  if constexpr (VEC && sizeof(E) == 4) {
#pragma unroll
    for (int j = 0; j < NS; j += 2) {
      const float2 v = __ldg(reinterpret_cast<const float2*>(p + j));
      f[j] = v.x;
      f[j + 1] = v.y;
    }
  } else if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < NS; j += 2) {
      const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(p + j));
      f[j] = __uint_as_float(u << 16);
      f[j + 1] = __uint_as_float(u & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < NS; ++j) f[j] = j < left ? rows::load1(p + j) : 0.f;
  }
}

// A warp's channels and what is theirs.  VEC: N = 4 NS, and every row of B and C begins at a
// multiple of two values (192 x 4096 x 16: 24 us, value by value 34).
template <class E, int NS, bool VEC>
struct StepWarp {
  const StepArgs& g;
  int lane, sl, cl, c0, left;                  // (this lane's states are of channels c0 + 8 k + cl)
  bool in, one;                                // c0 + lane is a channel; all are of one group
  float bias, D;
  __device__ __forceinline__ StepWarp(const StepArgs& args, int tile) : g(args) {
    const Args& a = g.a;
    lane = threadIdx.x & 31;
    sl = lane & 3;
    cl = lane >> 2;
    c0 = tile * 32;
    left = a.N - sl * NS;
    in = c0 + lane < a.d;
    bias = a.bias && in ? __ldg(a.bias + c0 + lane) : 0.f;
    D = a.D && in ? __ldg(a.D + c0 + lane) : 0.f;
    one = c0 / a.per == (min(c0 + 31, a.d - 1)) / a.per;
  }
  __device__ __forceinline__ bool on(int k) const { return c0 + 8 * k < g.a.d; }      // (eight channels are all there or none, and of one group)
  __device__ __forceinline__ float* states(long long slot) const { return g.state + (slot * g.a.d + c0 + cl) * g.a.N + sl * NS; }
  __device__ __forceinline__ long long step() const { return 8ll * g.a.N; }
  __device__ __forceinline__ void load(const float* st, float (&h)[4][NS]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (VEC) {
#pragma unroll
        for (int j = 0; j < NS; j += NS >= 4 ? 4 : 2) {
          if constexpr (NS >= 4) {
            const float4 v = on(k) ? __ldcs(reinterpret_cast<const float4*>(st + k * step() + j)) : make_float4(0.f, 0.f, 0.f, 0.f);
            h[k][j] = v.x; h[k][j + 1] = v.y; h[k][j + 2] = v.z; h[k][j + 3] = v.w;
          } else {
            const float2 v = on(k) ? __ldcs(reinterpret_cast<const float2*>(st + k * step() + j)) : make_float2(0.f, 0.f);
            h[k][j] = v.x; h[k][j + 1] = v.y;
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < NS; ++j) h[k][j] = on(k) && j < left ? st[k * step() + j] : 0.f;
      }
    }
  }
  __device__ __forceinline__ void store(float* st, const float (&h)[4][NS]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (!on(k)) break;
      if constexpr (VEC) {
#pragma unroll
        for (int j = 0; j < NS; j += NS >= 4 ? 4 : 2) {
          if constexpr (NS >= 4)
            __stcs(reinterpret_cast<float4*>(st + k * step() + j), make_float4(h[k][j], h[k][j + 1], h[k][j + 2], h[k][j + 3]));
          else
            __stcs(reinterpret_cast<float2*>(st + k * step() + j), make_float2(h[k][j], h[k][j + 1]));
        }
      } else {
#pragma unroll
        for (int j = 0; j < NS; ++j)
          if (j < left) st[k * step() + j] = h[k][j];
      }
    }
  }
  __device__ __forceinline__ E* out(long long row) const { return static_cast<E*>(g.a.y) + row * g.a.d + c0 + lane; }
  // One token: x, delta, and z of the lane's channel as they are stored.
  __device__ __forceinline__ void token(long long row, float x, float dt, float z, float (&h)[4][NS]) const {
    const Args& a = g.a;
    dt = softplus(dt + bias);
    const float gate = a.z ? z * sigmoid(z) : 1.f, dx = dt * x;
    float part[4], b[NS], c[NS];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      part[k] = 0.f;
      const float dtk = __shfl_sync(0xffffffffu, dt, 8 * k + cl), dxk = __shfl_sync(0xffffffffu, dx, 8 * k + cl);
      if (on(k)) {
        if (k == 0 || !one) {
          const int group = (c0 + 8 * k) / a.per;
          lane_states<E, NS, VEC>(static_cast<const E*>(a.B) + row * a.ldb + group * a.N + sl * NS, left, b);
          lane_states<E, NS, VEC>(static_cast<const E*>(a.C) + row * a.ldc + group * a.N + sl * NS, left, c);
        }
        float A[NS];
        lane_states<float, NS, VEC>(a.A + (long long)(c0 + 8 * k + cl) * a.N + sl * NS, left, A);
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          h[k][j] = fmaf(decay(dtk, A[j] * kLog2e), h[k][j], dxk * b[j]);
          part[k] = fmaf(c[j], h[k][j], part[k]);
        }
      }
    }
    // the sums over four lanes: lane sl has that of k = sl, and hands it to its channel's lane
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float keep = sl & 1 ? part[2 * i + 1] : part[2 * i], send = sl & 1 ? part[2 * i] : part[2 * i + 1];
      part[i] = keep + __shfl_xor_sync(0xffffffffu, send, 1);
    }
    const float keep = sl & 2 ? part[1] : part[0], send = sl & 2 ? part[0] : part[1];
    float sum = keep + __shfl_xor_sync(0xffffffffu, send, 2);
    sum = __shfl_sync(0xffffffffu, sum, (lane & 7) * 4 + (lane >> 3));
    if (in) rows::store1(out(row), fmaf(D, x, sum) * gate);
  }
};

template <class E, int NS, bool VEC>
__global__ void __launch_bounds__(kStepThreads) k_ssm_step(StepArgs g) {
  const Args& a = g.a;
  const long long id = (long long)blockIdx.x * (kStepThreads / 32) + (threadIdx.x >> 5), first = id / g.tiles * g.each;
  const StepWarp<E, NS, VEC> w(g, (int)(id % g.tiles));
  for (long long seq = first; seq < first + g.each && seq < a.s.n; ++seq) {
    const long long slot = g.slots ? g.slots[seq] : seq, row0 = seq * g.tokens;
    if (slot < 0 || slot >= g.n_slots) {       // a sequence without a state: zeros out, nothing kept
      for (int t = 0; t < g.tokens; ++t)
        if (w.in) rows::store1(w.out(row0 + t), 0.f);
      continue;
    }
    float h[4][NS];
    w.load(w.states(slot), h);
    for (int t = 0; t < g.tokens; ++t) {
      const long long row = row0 + t, c = w.c0 + w.lane;
      float x = 0.f, dt = 0.f, z = 0.f;
      if (w.in) {
        x = rows::load1(static_cast<const E*>(a.x) + row * a.ldx + c);
        dt = rows::load1(static_cast<const E*>(a.delta) + row * a.ldd + c);
        if (a.z) z = rows::load1(static_cast<const E*>(a.z) + row * a.ldz + c);
      }
      w.token(row, x, dt, z, h);
    }
    w.store(w.states(slot), h);
  }
}

// The same with the next row and the next sequence's states on their way while one is worked on: x,
// delta and z as a warp's, states (NS = 4) each thread its own.
constexpr int kAheadBlocks = 6;                // of an SM at once
template <class E, int NS>
__global__ void __launch_bounds__(kStepThreads, kAheadBlocks) k_ssm_step_ahead(StepArgs g) {
  static_assert(NS == 2 || NS == 4, "a thread's states of a channel are half a vector or one");
  constexpr int VN = 16 / sizeof(E), IN = 32 / VN;           // vectors of a row's 32 channels
  __shared__ __align__(16) E rows_in[kStepThreads / 32][2][3][32];
  __shared__ uint4 states_in[NS == 4 ? 2 : 1][NS == 4 ? 4 : 1][kStepThreads];
  const Args& a = g.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long id = (long long)blockIdx.x * (kStepThreads / 32) + warp, first = id / g.tiles * g.each;
  if (first >= a.s.n) return;
  const int count = a.s.n - first < g.each ? (int)(a.s.n - first) : g.each;
  const StepWarp<E, NS, true> w(g, (int)(id % g.tiles));
  long long mine = first + lane;               // lane i: sequence first + i's slot, -1 if it has none
  if (g.slots) mine = lane < count ? g.slots[mine] : -1;
  if (mine >= g.n_slots) mine = -1;
  auto states_of = [&](int i) {
    const long long slot = __shfl_sync(0xffffffffu, mine, i);
    return slot < 0 ? nullptr : w.states(slot);
  };
  auto row_ahead = [&](long long row, int to) {              // lanes 0 .. 3 IN - 1: a vector each
    const int k = lane / IN, c = lane % IN * VN;
    const void* p = k == 0 ? a.x : k == 1 ? a.delta : a.z;
    const long long ld = k == 0 ? a.ldx : k == 1 ? a.ldd : a.ldz;
    if (k < 3 && p && w.c0 + c < a.d) copy16(&rows_in[warp][to][k][c], static_cast<const E*>(p) + row * ld + w.c0 + c, true);
  };
  auto states_ahead = [&](const float* st, int to) {
    if constexpr (NS == 4)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (st && w.on(k)) copy16(&states_in[to][k][threadIdx.x], st + k * w.step(), true);
  };
  float* st = states_of(0);
  row_ahead(first * g.tokens, 0);
  states_ahead(st, 0);
  copies_end();
  int at = 0;                                  // where the row at hand is
  for (int i = 0; i < count; ++i) {
    float* const next = i + 1 < count ? states_of(i + 1) : nullptr;
    float h[4][NS];
    for (int t = 0; t < g.tokens; ++t, at ^= 1) {
      const long long row = (first + i) * g.tokens + t;
      __syncwarp();                            // every lane has read the row before
      if (t + 1 < g.tokens || i + 1 < count) row_ahead(row + 1, at ^ 1);
      if (t == 0) states_ahead(next, (i + 1) & 1);
      copies_end();
      copies_wait<1>();
      __syncwarp();
      if (!st) {                               // a sequence without a state: zeros out, nothing kept
        if (w.in) rows::store1(w.out(row), 0.f);
        continue;
      }
      if (t == 0) {
        if constexpr (NS == 4) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 v = states_in[i & 1][k][threadIdx.x];
            h[k][0] = __uint_as_float(v.x); h[k][1] = __uint_as_float(v.y);
            h[k][2] = __uint_as_float(v.z); h[k][3] = __uint_as_float(v.w);
          }
        } else {
          w.load(st, h);
        }
      }
      const E(&v)[3][32] = rows_in[warp][at];
      w.token(row, w.in ? rows::load1(&v[0][lane]) : 0.f, w.in ? rows::load1(&v[1][lane]) : 0.f,
              w.in && a.z ? rows::load1(&v[2][lane]) : 0.f, h);
    }
    if (st) w.store(st, h);
    st = next;
  }
}

// Sequences of a warp: the fewest that fill the `resident` warps of the GPU a whole number of times, kMaxEach
// at most (192 sequences x 4096 channels: 7, all at once, 23.4 us; 6 at most, in two waves, 25.7).
constexpr int kMaxEach = 10;
inline int sequences_of_a_warp(int n, int tiles, int resident) {
  for (int k = 1;; ++k) {
    const long long groups = (long long)k * resident / tiles;
    if (groups * kMaxEach >= n) return (int)((n + groups - 1) / groups);
  }
}

template <class E, int NS>
static cudaError_t step_of(StepArgs& g, cudaStream_t st) {
  constexpr int kWarps = kStepThreads / 32;
  const Args& a = g.a;
  const uintptr_t bits = reinterpret_cast<uintptr_t>(a.B) | reinterpret_cast<uintptr_t>(a.C) |
                         (uintptr_t)(a.ldb * sizeof(E)) | (uintptr_t)(a.ldc * sizeof(E));
  const bool vec = a.N == 4 * NS && bits % (2 * sizeof(E)) == 0 && reinterpret_cast<uintptr_t>(a.A) % 8 == 0;
  if (vec && NS <= 4) {
    g.each = sequences_of_a_warp(a.s.n, g.tiles, kAheadBlocks * kWarps * kNumSMs);
  } else {                                     // about 32 warps an SM
    const long long each = (long long)a.s.n * g.tiles / (32 * kNumSMs);
    g.each = each < 1 ? 1 : each > 8 ? 8 : (int)each;
  }
  const long long warps = (long long)((a.s.n + g.each - 1) / g.each) * g.tiles;
  const unsigned blocks = (unsigned)((warps + kWarps - 1) / kWarps);
  TraceScope tr("k_ssm_step", st);
  bool done = false;
  if constexpr (NS <= 4)
    if (vec && (g.each > 1 || g.tokens > 1)) {   // (a warp of one row has nothing to come)
      k_ssm_step_ahead<E, NS><<<blocks, kStepThreads, 0, st>>>(g);
      done = true;
    }
  if (!done && vec) k_ssm_step<E, NS, true><<<blocks, kStepThreads, 0, st>>>(g);
  if (!vec) k_ssm_step<E, NS, false><<<blocks, kStepThreads, 0, st>>>(g);
  return cudaGetLastError();
}
template <class E>
static cudaError_t step(StepArgs& g, cudaStream_t st) {
  const int N = g.a.N;
  return N <= 8 ? step_of<E, 2>(g, st) : N <= 16 ? step_of<E, 4>(g, st) : N <= 32 ? step_of<E, 8>(g, st) : step_of<E, 16>(g, st);
}

}  // namespace ssm

cudaError_t launch_ssm_step(const SsmArgs& g, int tokens, float* state, long long n_slots, const int* slots, void* y,
                            cudaStream_t st) {
  ssm::StepArgs s{};
  s.a.x = g.x; s.a.delta = g.delta; s.a.z = g.z; s.a.B = g.B; s.a.C = g.C;
  s.a.ldx = g.ldx; s.a.ldd = g.ldd; s.a.ldz = g.ldz; s.a.ldb = g.ldb; s.a.ldc = g.ldc;
  s.a.A = g.A; s.a.D = g.D; s.a.bias = g.bias;
  s.a.s.n = g.n_seq;
  s.a.d = g.d; s.a.groups = g.groups; s.a.N = g.N; s.a.per = g.d / g.groups;
  s.a.y = y;
  s.state = state; s.slots = slots; s.n_slots = n_slots; s.tokens = tokens;
  s.tiles = (g.d + 31) / 32;
  return g.math == CFC_MATH_BF16 ? ssm::step<__nv_bfloat16>(s, st) : ssm::step<float>(s, st);
}

}  // namespace cfc
