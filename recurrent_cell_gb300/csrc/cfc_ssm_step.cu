// cfc_ssm_step.cu -- the selective scan for the next few tokens of many
// sequences, each with its state in a slot of a pool, updated in place.
//
// A step reads a state and writes it: 8 N bytes a channel, against an exponential and
// four multiply-adds a state, so memory is the bound.  Four lanes share a channel, each
// with a quarter of its states in registers over the tokens of the call.
#include "ssm_common.cuh"

namespace cfc {
namespace ssm {

struct StepArgs {
  Args a;
  float* state;
  const int* slots;
  long long n_slots;
  int tokens, tiles;
};
constexpr int kStepThreads = 128, kStepChannels = kStepThreads / 4;

template <class E, int NS>
__global__ void __launch_bounds__(kStepThreads) k_ssm_step(StepArgs g) {
  const Args& a = g.a;
  const int tile = blockIdx.x % g.tiles, seq = blockIdx.x / g.tiles;
  const int sl = threadIdx.x & 3, c = tile * kStepChannels + (threadIdx.x >> 2);
  const bool on = c < a.d;                     // (whole warps of 8 channels: d is a multiple of 8)
  if (!on) return;
  const long long slot = g.slots ? g.slots[seq] : seq;
  const long long row0 = (long long)seq * g.tokens;
  E* y = static_cast<E*>(a.y) + row0 * a.d + c;
  if (slot < 0 || slot >= g.n_slots) {         // a sequence without a state: zeros out, nothing kept
    if (sl == 0)
      for (int t = 0; t < g.tokens; ++t) rows::store1(y + (long long)t * a.d, 0.f);
    return;
  }
  float* st = g.state + (slot * a.d + c) * a.N + sl * NS;
  const float* Ap = a.A + (long long)c * a.N + sl * NS;
  const int left = a.N - sl * NS;              // states of this lane's
  float h[NS], A2[NS];
  const bool whole = a.N == 4 * NS;
  if (whole) {
#pragma unroll
    for (int j = 0; j < NS; j += 2) {
      const float2 v = __ldcs(reinterpret_cast<const float2*>(st + j));
      h[j] = v.x; h[j + 1] = v.y;
    }
  }
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    if (!whole) h[j] = j < left ? st[j] : 0.f;
    A2[j] = j < left ? __ldg(Ap + j) * kLog2e : 0.f;
  }
  const float bias = a.bias ? __ldg(a.bias + c) : 0.f, D = a.D ? __ldg(a.D + c) : 0.f;
  const int group = c / a.per;
  for (int t = 0; t < g.tokens; ++t) {
    const long long row = row0 + t;
    const float x = rows::load1(static_cast<const E*>(a.x) + row * a.ldx + c);
    const float dt = softplus(rows::load1(static_cast<const E*>(a.delta) + row * a.ldd + c) + bias);
    const E* Bp = static_cast<const E*>(a.B) + row * a.ldb + group * a.N + sl * NS;
    const E* Cp = static_cast<const E*>(a.C) + row * a.ldc + group * a.N + sl * NS;
    const float dx = dt * x;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      const float b = j < left ? rows::load1(Bp + j) : 0.f, cc = j < left ? rows::load1(Cp + j) : 0.f;
      h[j] = fmaf(ex2(dt * A2[j]), h[j], dx * b);
      sum = fmaf(cc, h[j], sum);
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    if (sl == 0) {
      sum = fmaf(D, x, sum);
      if (a.z) {
        const float z = rows::load1(static_cast<const E*>(a.z) + row * a.ldz + c);
        sum *= z * sigmoid(z);
      }
      rows::store1(y + (long long)t * a.d, sum);
    }
  }
  if (whole) {
#pragma unroll
    for (int j = 0; j < NS; j += 2) __stcs(reinterpret_cast<float2*>(st + j), make_float2(h[j], h[j + 1]));
  } else {
#pragma unroll
    for (int j = 0; j < NS; ++j)
      if (j < left) st[j] = h[j];
  }
}

template <class E>
static cudaError_t step(const StepArgs& g, int NS, cudaStream_t st) {
  const unsigned blocks = (unsigned)((long long)g.a.s.n * g.tiles);
  TraceScope tr("k_ssm_step", st);
  if (NS == 2) k_ssm_step<E, 2><<<blocks, kStepThreads, 0, st>>>(g);
  else if (NS == 4) k_ssm_step<E, 4><<<blocks, kStepThreads, 0, st>>>(g);
  else if (NS == 8) k_ssm_step<E, 8><<<blocks, kStepThreads, 0, st>>>(g);
  else k_ssm_step<E, 16><<<blocks, kStepThreads, 0, st>>>(g);
  return cudaGetLastError();
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
  s.tiles = (g.d + ssm::kStepChannels - 1) / ssm::kStepChannels;
  const int NS = g.N <= 8 ? 2 : g.N <= 16 ? 4 : g.N <= 32 ? 8 : 16;
  return g.math == CFC_MATH_BF16 ? ssm::step<__nv_bfloat16>(s, NS, st) : ssm::step<float>(s, NS, st);
}

}  // namespace cfc
