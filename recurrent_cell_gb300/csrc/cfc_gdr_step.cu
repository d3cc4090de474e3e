// cfc_gdr_step.cu -- the gated delta rule for the next few tokens of many
// sequences, each with its state in a pool, updated in place.
//
// A step reads a state once and writes it once: 8 d_k d_v bytes a head against
// 9 d_k d_v operations, so memory is the bound and the state is the traffic.
// A block takes TDV value columns of one head with all d_k rows in registers
// (four columns a thread, so rows of 16 bytes a thread), applies the tokens
// one after another and writes back.  With a = exp(g), y = S^T k, z = S^T q
// from one pass over the registers,
//   u = beta (v - a y),  S <- a S + k u^T,  o = scale (a z + (k.q) u):
// one block-wide sum a token.  192 sequences x 32 heads of 128 x 128: 805 MB in
// 128 us, 6.3 TB/s; one sequence of 16 heads 2.7 us, a launch's latency.
#include "gdr_common.cuh"

namespace cfc {
namespace gdr {

struct StepArgs {
  const void *q, *k, *v;
  long long ldq, ldk, ldv;
  const float *g, *beta;
  float* state;
  const int* slots;
  long long n_slots;
  void* o;
  int tokens, hk, hv, dk, dv, ntile;
  float scale;
};

constexpr int kStepThreads = 256;
constexpr int kAhead = 4;      // tokens whose rows are fetched together

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// RPT rows of the state a thread: rows rg, rg + RG, ... of RG row groups.
template <class E, int TDV, int RPT>
__global__ void __launch_bounds__(kStepThreads, RPT <= 2 ? 6 : 4) k_gdr_step(StepArgs a) {
  constexpr int AC = TDV / 4;                   // threads across the columns
  constexpr int RG = kStepThreads / AC;
  constexpr int WARPS = kStepThreads / 32;
  __shared__ float ks[kAhead][kMaxDk], qs[kAhead][kMaxDk], gates[kAhead][2];
  __shared__ float4 vs[kAhead][AC];
  __shared__ float4 py[2][WARPS][AC], pz[2][WARPS][AC];
  __shared__ float pkq[2][WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ca = tid % AC, rg = tid / AC;
  const int tile = blockIdx.x % a.ntile;
  const long long sh = blockIdx.x / a.ntile;
  const int h = (int)(sh % a.hv);
  const long long n = sh / a.hv;
  const int hq = h / (a.hv / a.hk);
  const int col = tile * TDV + ca * 4;
  const bool on = col < a.dv;
  E* o = static_cast<E*>(a.o);
  const long long row0 = n * a.tokens;
  const long long slot = a.slots ? a.slots[n] : n;
  if (slot < 0 || slot >= a.n_slots) {          // a sequence without a state: zeros out, nothing kept
    if (rg == 0 && on)
      for (int t = 0; t < a.tokens; ++t)
        for (int e = 0; e < 4; ++e) put(o + ((row0 + t) * a.hv + h) * a.dv + col + e, 0.f);
    return;
  }
  float* st = a.state + (slot * a.hv + h) * a.dk * a.dv + col;
  float4 s[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = rg + i * RG;
    s[i] = on && r < a.dk ? __ldcs(reinterpret_cast<const float4*>(st + (long long)r * a.dv))
                          : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int t = 0; t < a.tokens; ++t) {
    const long long row = row0 + t;
    const int ta = t % kAhead;
    if (ta == 0) {
      if (t > 0) __syncthreads();               // the last rows have been read
      const int more = min(kAhead, a.tokens - t), r = tid & (kMaxDk - 1);
      const E* kq = (tid < kMaxDk ? static_cast<const E*>(a.k) + row * a.ldk : static_cast<const E*>(a.q) + row * a.ldq) +
                    (long long)hq * a.dk;
      const long long ld = tid < kMaxDk ? a.ldk : a.ldq;
#pragma unroll
      for (int x = 0; x < kAhead; ++x)
        if (x < more) (tid < kMaxDk ? ks : qs)[x][r] = r < a.dk ? to_f(kq[x * ld + r]) : 0.f;
      if (tid < more * AC) {
        const int x = tid / AC, cc = tile * TDV + (tid % AC) * 4;
        float4 v4 = make_float4(0.f, 0.f, 0.f, 0.f);
        if (cc < a.dv) {
          const E* v = static_cast<const E*>(a.v) + (row + x) * a.ldv + (long long)h * a.dv + cc;
          v4 = make_float4(to_f(v[0]), to_f(v[1]), to_f(v[2]), to_f(v[3]));
        }
        vs[x][tid % AC] = v4;
      }
      if (tid >= kStepThreads - 2 * kAhead) {
        const int x = (tid - (kStepThreads - 2 * kAhead)) >> 1;
        if (x < more) gates[x][tid & 1] = tid & 1 ? a.beta[(row + x) * a.hv + h] : expf(a.g[(row + x) * a.hv + h]);
      }
      __syncthreads();
    }
    const float al = gates[ta][0], be = gates[ta][1];
    const float4 vv = vs[ta][ca];
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f), z = y;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int r = rg + i * RG;
      if (r >= kMaxDk) continue;
      const float kk = ks[ta][r], qq = qs[ta][r];
      y.x = fmaf(s[i].x, kk, y.x); y.y = fmaf(s[i].y, kk, y.y); y.z = fmaf(s[i].z, kk, y.z); y.w = fmaf(s[i].w, kk, y.w);
      z.x = fmaf(s[i].x, qq, z.x); z.y = fmaf(s[i].y, qq, z.y); z.z = fmaf(s[i].z, qq, z.z); z.w = fmaf(s[i].w, qq, z.w);
    }
    float kq = 0.f;
    for (int r = tid; r < kMaxDk; r += kStepThreads) kq = fmaf(ks[ta][r], qs[ta][r], kq);
#pragma unroll
    for (int m = AC; m < 32; m <<= 1) {
      y.x += __shfl_xor_sync(0xffffffffu, y.x, m); y.y += __shfl_xor_sync(0xffffffffu, y.y, m);
      y.z += __shfl_xor_sync(0xffffffffu, y.z, m); y.w += __shfl_xor_sync(0xffffffffu, y.w, m);
      z.x += __shfl_xor_sync(0xffffffffu, z.x, m); z.y += __shfl_xor_sync(0xffffffffu, z.y, m);
      z.z += __shfl_xor_sync(0xffffffffu, z.z, m); z.w += __shfl_xor_sync(0xffffffffu, z.w, m);
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) kq += __shfl_xor_sync(0xffffffffu, kq, m);
    const int b = t & 1;
    if (lane < AC) { py[b][warp][lane] = y; pz[b][warp][lane] = z; }
    if (lane == 0) pkq[b][warp] = kq;
    __syncthreads();
    y = z = make_float4(0.f, 0.f, 0.f, 0.f);
    kq = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float4 u = py[b][w][ca], x = pz[b][w][ca];
      y.x += u.x; y.y += u.y; y.z += u.z; y.w += u.w;
      z.x += x.x; z.y += x.y; z.z += x.z; z.w += x.w;
      kq += pkq[b][w];
    }
    const float4 u = make_float4(be * (vv.x - al * y.x), be * (vv.y - al * y.y), be * (vv.z - al * y.z),
                                 be * (vv.w - al * y.w));
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int r = rg + i * RG;
      if (r >= kMaxDk) continue;
      const float kk = ks[ta][r];
      s[i].x = fmaf(kk, u.x, al * s[i].x); s[i].y = fmaf(kk, u.y, al * s[i].y);
      s[i].z = fmaf(kk, u.z, al * s[i].z); s[i].w = fmaf(kk, u.w, al * s[i].w);
    }
    if (rg == 0 && on) {
      E* p = o + (row * a.hv + h) * a.dv + col;
      put(p, a.scale * fmaf(kq, u.x, al * z.x));
      put(p + 1, a.scale * fmaf(kq, u.y, al * z.y));
      put(p + 2, a.scale * fmaf(kq, u.z, al * z.z));
      put(p + 3, a.scale * fmaf(kq, u.w, al * z.w));
    }
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = rg + i * RG;
    if (on && r < a.dk) __stcs(reinterpret_cast<float4*>(st + (long long)r * a.dv), s[i]);
  }
}

template <class E, int TDV>
static cudaError_t launch(StepArgs a, long long n_seq, cudaStream_t st) {
  constexpr int RG = kStepThreads / (TDV / 4);
  a.ntile = (a.dv + TDV - 1) / TDV;
  const unsigned blocks = (unsigned)(n_seq * a.hv * a.ntile);
  TraceScope tr("k_gdr_step", st);
  if (a.dk <= 64) k_gdr_step<E, TDV, (64 + RG - 1) / RG><<<blocks, kStepThreads, 0, st>>>(a);
  else k_gdr_step<E, TDV, (kMaxDk + RG - 1) / RG><<<blocks, kStepThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace gdr

cudaError_t launch_gdr_step(const GdrStepArgs& g, cudaStream_t st) {
  using namespace gdr;
  StepArgs a{g.q, g.k, g.v, g.ldq, g.ldk, g.ldv, g.g, g.beta, g.state, g.slots, g.n_slots, g.o,
             g.tokens, g.hk, g.hv, g.dk, g.dv, 0, g.scale};
  // Few heads: tiles of 32 columns, so that every SM takes part; many: of 64, unless the last would be half
  // empty.  Heads of 128 x 128, one token, 32 columns against 64: 96 heads 10.4, 10.6 us; 256 heads 14.4,
  // 12.8; 1024 heads 33.0, 30.5.
  const long long heads = (long long)g.n_seq * g.hv;
  const bool wide = (g.dv + 63) % 64 >= 32 && heads * ((g.dv + 63) / 64) >= 2 * kNumSMs;
  if (g.math == CFC_MATH_BF16)
    return wide ? launch<__nv_bfloat16, 64>(a, g.n_seq, st) : launch<__nv_bfloat16, 32>(a, g.n_seq, st);
  return wide ? launch<float, 64>(a, g.n_seq, st) : launch<float, 32>(a, g.n_seq, st);
}

}  // namespace cfc
