// cfc_ssm_step.cu -- the selective scan for the next few tokens of many
// sequences, each with its state in a slot of a pool, updated in place.
//
// A step reads a state and writes it: 8 N bytes a channel, against an exponential and
// four multiply-adds a state, so memory is the bound.  A warp takes 32 channels: each
// lane forms dt, dt x and the gate of one of them, then eight channels at a time have four
// lanes each, with a quarter of the states in registers, and the sums over states
// come back to their channels' lanes.  Where there are sequences enough for every SM, a
// warp takes several with the same channels, so that A comes from L1 (192 sequences x 4096
// channels x 16 states: 5 a warp 31 us, one a warp 36).  Reading the next sequence's state ahead
// made it slower (29 against 27 us, in a graph): there are warps enough to hide it.
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

// VEC: N = 4 NS, and every row of B and C begins at a multiple of two values.
template <class E, int NS, bool VEC>
__global__ void __launch_bounds__(kStepThreads) k_ssm_step(StepArgs g) {
  const Args& a = g.a;
  const long long id = (long long)blockIdx.x * (kStepThreads / 32) + (threadIdx.x >> 5);
  const int tile = (int)(id % g.tiles), lane = threadIdx.x & 31, sl = lane & 3, cl = lane >> 2;
  const long long first = id / g.tiles * g.each;
  const int c0 = tile * 32, left = a.N - sl * NS;
  const bool in = c0 + lane < a.d;
  const float bias = a.bias && in ? __ldg(a.bias + c0 + lane) : 0.f, D = a.D && in ? __ldg(a.D + c0 + lane) : 0.f;
  const bool one = c0 / a.per == (min(c0 + 31, a.d - 1)) / a.per;      // one group's channels
  for (long long seq = first; seq < first + g.each && seq < a.s.n; ++seq) {
    const long long slot = g.slots ? g.slots[seq] : seq, row0 = seq * g.tokens;
    E* y = static_cast<E*>(a.y) + row0 * a.d + c0 + lane;
    if (slot < 0 || slot >= g.n_slots) {       // a sequence without a state: zeros out, nothing kept
      for (int t = 0; t < g.tokens; ++t)
        if (in) rows::store1(y + (long long)t * a.d, 0.f);
      continue;
    }
    // this lane's channels are c0 + 8 k + cl
    float* st = g.state + (slot * a.d + c0 + cl) * a.N + sl * NS;
    const long long step = 8ll * a.N;
    float h[4][NS];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool on = c0 + 8 * k < a.d;
      if constexpr (VEC) {
#pragma unroll
        for (int j = 0; j < NS; j += NS >= 4 ? 4 : 2) {
          if constexpr (NS >= 4) {
            const float4 v = on ? __ldcs(reinterpret_cast<const float4*>(st + k * step + j)) : make_float4(0.f, 0.f, 0.f, 0.f);
            h[k][j] = v.x; h[k][j + 1] = v.y; h[k][j + 2] = v.z; h[k][j + 3] = v.w;
          } else {
            const float2 v = on ? __ldcs(reinterpret_cast<const float2*>(st + k * step + j)) : make_float2(0.f, 0.f);
            h[k][j] = v.x; h[k][j + 1] = v.y;
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < NS; ++j) h[k][j] = on && j < left ? st[k * step + j] : 0.f;
      }
    }
    for (int t = 0; t < g.tokens; ++t) {
      const long long row = row0 + t;
      float x = 0.f, dt = 0.f, gate = 1.f;
      if (in) {
        x = rows::load1(static_cast<const E*>(a.x) + row * a.ldx + c0 + lane);
        dt = rows::load1(static_cast<const E*>(a.delta) + row * a.ldd + c0 + lane);
        if (a.z) gate = rows::load1(static_cast<const E*>(a.z) + row * a.ldz + c0 + lane);
      }
      dt = softplus(dt + bias);
      if (a.z) gate *= sigmoid(gate);
      const float dx = dt * x;
      float part[4], b[NS], c[NS];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        part[k] = 0.f;
        const float dtk = __shfl_sync(0xffffffffu, dt, 8 * k + cl), dxk = __shfl_sync(0xffffffffu, dx, 8 * k + cl);
        if (c0 + 8 * k < a.d) {                // (eight channels are all there or none, and of one group)
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
      if (in) rows::store1(y + (long long)t * a.d, fmaf(D, x, sum) * gate);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (c0 + 8 * k >= a.d) break;
      if constexpr (VEC) {
#pragma unroll
        for (int j = 0; j < NS; j += NS >= 4 ? 4 : 2) {
          if constexpr (NS >= 4)
            __stcs(reinterpret_cast<float4*>(st + k * step + j), make_float4(h[k][j], h[k][j + 1], h[k][j + 2], h[k][j + 3]));
          else
            __stcs(reinterpret_cast<float2*>(st + k * step + j), make_float2(h[k][j], h[k][j + 1]));
        }
      } else {
#pragma unroll
        for (int j = 0; j < NS; ++j)
          if (j < left) st[k * step + j] = h[k][j];
      }
    }
  }
}

template <class E, int NS>
static cudaError_t step_of(const StepArgs& g, cudaStream_t st) {
  const Args& a = g.a;
  const long long warps = (long long)((a.s.n + g.each - 1) / g.each) * g.tiles;
  const unsigned blocks = (unsigned)((warps + kStepThreads / 32 - 1) / (kStepThreads / 32));
  const uintptr_t bits = reinterpret_cast<uintptr_t>(a.B) | reinterpret_cast<uintptr_t>(a.C) |
                         (uintptr_t)(a.ldb * sizeof(E)) | (uintptr_t)(a.ldc * sizeof(E)) | reinterpret_cast<uintptr_t>(a.A);
  TraceScope tr("k_ssm_step", st);
  if (a.N == 4 * NS && bits % (2 * sizeof(E)) == 0 && reinterpret_cast<uintptr_t>(a.A) % 8 == 0)
    k_ssm_step<E, NS, true><<<blocks, kStepThreads, 0, st>>>(g);
  else
    k_ssm_step<E, NS, false><<<blocks, kStepThreads, 0, st>>>(g);
  return cudaGetLastError();
}
template <class E>
static cudaError_t step(const StepArgs& g, cudaStream_t st) {
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
  const long long each = (long long)g.n_seq * s.tiles / (32 * kNumSMs);
  s.each = each < 1 ? 1 : each > 8 ? 8 : (int)each;
  return g.math == CFC_MATH_BF16 ? ssm::step<__nv_bfloat16>(s, st) : ssm::step<float>(s, st);
}

}  // namespace cfc
