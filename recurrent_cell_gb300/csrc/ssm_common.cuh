// ssm_common.cuh -- what the selective scan's kernels share: the split of rows and
// channels, tiles of a chunk in shared memory, and the elementary functions.
//
// Per sequence and channel c, with a state h [N] in fp32, and per token
//   dt = softplus(delta + bias),  h <- exp(dt A) h + dt x B,
//   y = (C . h + D x) silu(z),
// B and C [N] shared by the channels of a group.
//
// A warp runs a tile of channels of one group over a segment of rows: 4 lanes
// share a channel's states and 8 lanes the tile's channels, so a thread keeps
// CPL channels x NS states in registers and sums over states need two lane steps,
// sums over channels three.  Rows go by chunks of kT: what depends on a token and
// channel alone (softplus, dt x, the gate) is formed once, by a second warp and through
// shared memory; the loop over tokens is left with an exponential and
// four multiply-adds a state.
//
// Segments are ranges of the rows of all sequences together, whatever the sequences'
// lengths: a state is set afresh where a sequence begins, and handed on where a
// segment's end cuts one.  Those states come from a pass of their own (the
// segment's own end state and sum of dt, since a product of decays is the exp of a
// sum) and a short serial pass over segments.
#pragma once

#include "pair_math.cuh"
#include "row_ops.cuh"
#include "seq_rows.cuh"

namespace cfc {
namespace ssm {

using namespace pairs;
using seqs::Seqs;
using seqs::Where;

constexpr int kResident = 8;                 // blocks of an SM at once, forward
constexpr int kT = 16;                       // rows of a chunk

struct Args {
  const void *x, *delta, *z, *B, *C;
  long long ldx, ldd, ldz, ldb, ldc;         // elements from row to row
  const float *A, *D, *bias;
  Seqs s;
  int d, groups, N;
  int per, tpg;                              // channels of a group, its tiles
  int vec_bc;                                // rows of B and C are whole 16-byte vectors (a prompt of 16384 x 2048, both
                                             // passes by events: 115 + 168 us, value by value 149 + 215)
  long long S;                               // rows of a segment
  int n_seg, tiles, cps;                     // chunks of a segment
  const float* init;
  void* y;
  float* final_state;
  // workspace
  float *local, *sdt, *ckpt;
  int* flags;
  // backward
  const void* grad_y;
  const float* grad_final;
  void *grad_x, *grad_delta, *grad_z, *grad_B, *grad_C;
  float *grad_init, *part, *bc;
};

// NS states and CPL channels a thread: 16 of them at most, whose values, decays and gradients registers hold.
template <class E_, int NS_, int CPL_>
struct Cfg {
  using E = E_;
  static constexpr int NS = NS_, CPL = CPL_, NP = 4 * NS, CW = 8 * CPL;
  static constexpr int VN = 16 / sizeof(E);                  // channels of a 16-byte vector
  static constexpr int LPR = CW / VN, RPP = 32 / LPR;        // lanes a row, rows a pass
  static constexpr int P = (kT + RPP - 1) / RPP;             // passes of a chunk
  static constexpr int BV = NP * (int)sizeof(E) / 16;        // vectors of a row of B
  static constexpr int PAIRS = CPL * NS / 2, CPAIRS = CPL > 1 ? CPL / 2 : 1, SPAIRS = CPL > 1 ? NS : NS / 2;
  static constexpr int BL = (kT * BV + 31) / 32;             // of a chunk, a lane
};

// softplus(v) = max(v, 0) + log1p(e), e = exp(-|v|), of two values.  The exponent's
// rounding is put right by a first-order term; log1p(e) = e P(e) on [0, 1] with P of
// degree 8, fitted for the smallest relative error (3e-8; 1.7e-7 with the roundings).
// A NaN comes through e.  e: for the caller's sigmoid.
__device__ __forceinline__ F2 softplus2(F2 v, F2* e_out = nullptr) {
  float a, b;
  split(v, a, b);
  // (beyond 100 e is zero: the parts of an infinite product would make a NaN)
  const F2 u = pack(min_nan(fabsf(a), 100.f), min_nan(fabsf(b), 100.f)), hi = mul2(u, twice(kLog2e));
  const F2 off = fma2(u, twice(-kLog2e), hi);                // hi less the exact product
  float ha, hb;
  split(hi, ha, hb);
  F2 e = pack(ex2(-ha), ex2(-hb));
  e = fma2(mul2(e, off), twice(kLn2), e);
  if (e_out) *e_out = e;
  F2 p = twice(0.0052326940931379795f);
  p = fma2(p, e, twice(-0.029505237936973572f));
  p = fma2(p, e, twice(0.07822595536708832f));
  p = fma2(p, e, twice(-0.13663245737552643f));
  p = fma2(p, e, twice(0.19106006622314453f));
  p = fma2(p, e, twice(-0.2484298199415207f));
  p = fma2(p, e, twice(0.3331909775733948f));
  p = fma2(p, e, twice(-0.4999949336051941f));
  p = fma2(p, e, twice(0.9999999403953552f));
  return fma2(p, e, pack(fmaxf(a, 0.f), fmaxf(b, 0.f)));
}
__device__ __forceinline__ float softplus(float v) {
  float a, b;
  split(softplus2(twice(v)), a, b);
  return a;
}
// exp(dt A) from dt and A / ln 2.  The hardware's exponential is low by 2e-8 on average (measured
// over [-1, 0]; 4e-8 in root mean square), which a state adds up over all the tokens it
// remembers: the gradient of A came out with twice the error of fp32 arithmetic.  A lift
// of the exponent by as much balances it; it leaves exp(0) at 1.
constexpr float kLift = 2.75e-8f;
__device__ __forceinline__ F2 decay2(F2 dt, F2 A2) { return ex2_2(fma2(dt, A2, twice(kLift))); }
__device__ __forceinline__ float decay(float dt, float A2) { return ex2(fmaf(dt, A2, kLift)); }

// The warp's tile of channels.
template <class G>
struct Tile {
  int lane, sl, cl;                          // state lane, channel lane
  int g, c0, cols;                           // group, first channel, channels (a multiple of 8; 0 or less: none)
  __device__ __forceinline__ Tile(const Args& a, int tile) {
    lane = threadIdx.x & 31;
    sl = lane & 3;
    cl = lane >> 2;
    g = tile / a.tpg;
    const int at = (tile % a.tpg) * G::CW;
    c0 = g * a.per + at;
    cols = a.per - at < G::CW ? a.per - at : G::CW;
  }
  __device__ __forceinline__ bool has(int i) const { return cl * G::CPL + i < cols; }
  __device__ __forceinline__ int channel(int i) const { return c0 + cl * G::CPL + i; }
  // the row and first column of pass p's vector
  __device__ __forceinline__ int row(int p) const { return p * G::RPP + lane / G::LPR; }
  __device__ __forceinline__ int col() const { return lane % G::LPR * G::VN; }
};

// A thread's states go in pairs: two channels of one state, or (one channel a thread)
// two states.  Element k of CPL * NS, pair k / 2: its channel and state.
template <class G>
__device__ __forceinline__ int channel_of(int k) { return G::CPL > 1 ? k / (2 * G::NS) * 2 + (k & 1) : 0; }
template <class G>
__device__ __forceinline__ int state_of(int k) { return G::CPL > 1 ? k / 2 % G::NS : k; }

template <class G>
__device__ __forceinline__ void load_A(const Args& a, const Tile<G>& w, F2 (&A2)[G::PAIRS]) {
#pragma unroll
  for (int p = 0; p < G::PAIRS; ++p) {
    float f[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int i = channel_of<G>(2 * p + m), n = w.sl * G::NS + state_of<G>(2 * p + m);
      f[m] = w.has(i) && n < a.N ? __ldg(a.A + (long long)w.channel(i) * a.N + n) * kLog2e : 0.f;
    }
    A2[p] = pack(f[0], f[1]);
  }
}

// States [sequence, d, N] as the caller has them.
template <class G>
__device__ __forceinline__ void load_state(const Args& a, const Tile<G>& w, const float* s, long long seq, F2 (&h)[G::PAIRS]) {
#pragma unroll
  for (int p = 0; p < G::PAIRS; ++p) {
    float f[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int i = channel_of<G>(2 * p + m), n = w.sl * G::NS + state_of<G>(2 * p + m);
      f[m] = s && w.has(i) && n < a.N ? s[(seq * a.d + w.channel(i)) * a.N + n] : 0.f;
    }
    h[p] = pack(f[0], f[1]);
  }
}
template <class G>
__device__ __forceinline__ void store_state(const Args& a, const Tile<G>& w, float* s, long long seq, const F2 (&h)[G::PAIRS]) {
#pragma unroll
  for (int p = 0; p < G::PAIRS; ++p) {
    float f[2];
    split(h[p], f[0], f[1]);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int i = channel_of<G>(2 * p + m), n = w.sl * G::NS + state_of<G>(2 * p + m);
      if (w.has(i) && n < a.N) s[(seq * a.d + w.channel(i)) * a.N + n] = f[m];
    }
  }
}
// States as the kernels hand them on: a warp's registers side by side.
template <class G>
__device__ __forceinline__ void load_lanes(const float* s, long long block, int lane, F2 (&h)[G::PAIRS]) {
#pragma unroll
  for (int p = 0; p < G::PAIRS; ++p) h[p] = reinterpret_cast<const F2*>(s)[(block * G::PAIRS + p) * 32 + lane];
}
template <class G>
__device__ __forceinline__ void store_lanes(float* s, long long block, int lane, const F2 (&h)[G::PAIRS]) {
#pragma unroll
  for (int p = 0; p < G::PAIRS; ++p) reinterpret_cast<F2*>(s)[(block * G::PAIRS + p) * 32 + lane] = h[p];
}

// N floats to or from shared memory, 16 bytes at a time.
template <int N>
__device__ __forceinline__ void put(float* p, const float (&v)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else if constexpr (N == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
  } else {
    p[0] = v[0];
  }
}
template <int N>
__device__ __forceinline__ void get(const float* p, float (&v)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 f = *reinterpret_cast<const float4*>(p + i);
      v[i] = f.x; v[i + 1] = f.y; v[i + 2] = f.z; v[i + 3] = f.w;
    }
  } else if constexpr (N == 2) {
    const float2 f = *reinterpret_cast<const float2*>(p);
    v[0] = f.x; v[1] = f.y;
  } else {
    v[0] = p[0];
  }
}

template <int N>
__device__ __forceinline__ void put_pairs(float* s, const F2 (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) *reinterpret_cast<ulonglong2*>(s + 2 * i) = make_ulonglong2(v[i], v[i + 1]);
}
template <int N>
__device__ __forceinline__ void get_pairs(const float* s, F2 (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(s + 2 * i);
    v[i] = u.x;
    v[i + 1] = u.y;
  }
}
// What a lane reads of a token, as pairs that fit its states': dt (or dt x, or g) of its
// channels, B (or C) of its states.  A value that goes with two channels is doubled in
// registers: from shared memory each register that a lane reads costs a quarter of the
// SM's cycle, and those reads are as scarce as instructions.
template <class G>
__device__ __forceinline__ void get_channels(const float* row, int cl, F2 (&v)[G::CPAIRS]) {
  if constexpr (G::CPL == 4) {
    const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(row + cl * 4);
    v[0] = u.x;
    v[1] = u.y;
  } else if constexpr (G::CPL == 2) {
    v[0] = *reinterpret_cast<const F2*>(row + cl * 2);
  } else {
    v[0] = twice(row[cl]);
  }
}
template <class G>
__device__ __forceinline__ void get_states(const float* row, int sl, F2 (&v)[G::SPAIRS]) {
  if constexpr (G::CPL == 1) {
    get_pairs(row + sl * G::NS, v);
  } else {
    float f[G::NS];
    get(row + sl * G::NS, f);
#pragma unroll
    for (int j = 0; j < G::NS; ++j) v[j] = twice(f[j]);
  }
}
// The pairs that state pair p needs.
template <class G>
constexpr __device__ __forceinline__ int cpair(int p) { return G::CPL > 1 ? p / G::NS : 0; }
template <class G>
constexpr __device__ __forceinline__ int spair(int p) { return G::CPL > 1 ? p % G::NS : p; }

// A chunk's vectors of a [rows, channels] tensor, zeros outside.
template <class G>
__device__ __forceinline__ void load_raw(const Tile<G>& w, const void* p, long long ld, long long row0, int n, uint4 (&v)[G::P]) {
  const typename G::E* q = static_cast<const typename G::E*>(p) + w.c0 + w.col();
#pragma unroll
  for (int k = 0; k < G::P; ++k) {
    v[k] = load_here(q + (row0 + w.row(k)) * ld, w.row(k) < n && w.col() < w.cols);
  }
}
// The lane's columns of a vector over channels (NULL: zeros).
template <class G>
__device__ __forceinline__ void load_pairs(const Tile<G>& w, const float* s, F2 (&v)[G::VN / 2]) {
#pragma unroll
  for (int e = 0; e < G::VN / 2; ++e) {
    const bool in = s && w.col() < w.cols;
    v[e] = pack(in ? __ldg(s + w.c0 + w.col() + 2 * e) : 0.f, in ? __ldg(s + w.c0 + w.col() + 2 * e + 1) : 0.f);
  }
}
// A segment's sums of dt, of each of the thread's channels.
template <class G>
__device__ __forceinline__ void store_sums(const Args& a, long long block, int lane, const F2 (&sum)[G::CPAIRS]) {
#pragma unroll
  for (int i = 0; i < G::CPAIRS; ++i) {
    float f[2];
    split(sum[i], f[0], f[1]);
#pragma unroll
    for (int m = 0; m < (G::CPL > 1 ? 2 : 1); ++m) a.sdt[(block * G::CPL + 2 * i + m) * 32 + lane] = f[m];
  }
}

// Half of a sum over lanes: v[2 i] plus the lane across m's for lanes without that bit, v[2 i + 1] for those
// with it, in v[i].
template <int N>
__device__ __forceinline__ void fold(float (&v)[N], int lane, int m) {
  const bool up = lane & m;
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const float keep = up ? v[2 * i + 1] : v[2 * i], send = up ? v[2 * i] : v[2 * i + 1];
    v[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
  }
}
template <int N>
__device__ __forceinline__ float all(float v, int m) { return v + __shfl_xor_sync(0xffffffffu, v, m); }

// Sums over the 4 state lanes of v[CPL]: lane sl has channel sl % CPL's.
template <int CPL>
__device__ __forceinline__ float over_states(float (&v)[CPL], int lane) {
  if constexpr (CPL == 4) {
    fold<4>(v, lane, 1);
    float u[2] = {v[0], v[1]};
    fold<2>(u, lane, 2);
    return u[0];
  } else if constexpr (CPL == 2) {
    fold<2>(v, lane, 1);
    return all<1>(v[0], 2);
  } else {
    return all<1>(all<1>(v[0], 1), 2);
  }
}
// Whether this warp is the one of its block's two that helps.  A warp's scheduler is its slot's, and blocks of two
// take slots in pairs, so were it always the second, the states would run on two of the four.
__device__ __forceinline__ bool helper_of_two() {
  __shared__ int swap;
  if (threadIdx.x == 0) {
    uint32_t slot;
    asm volatile("mov.u32 %0, %%warpid;" : "=r"(slot));
    swap = slot >> 2 & 1;
  }
  __syncthreads();
  return (threadIdx.x >= 32) != (swap != 0);
}

// A chunk's rows of B or C as the lanes have them (whole vectors), or element by element, into the tile [kT][NP].
template <class G>
struct Rows {
  uint4 v[G::BL];
  __device__ __forceinline__ void stage(const Args& a, const Tile<G>& w, const void* p, long long ld, long long row0, int n,
                                        float* tile) const {
    if (a.vec_bc) {
#pragma unroll
      for (int k = 0; k < G::BL; ++k) {
        const int i = k * 32 + w.lane;
        F2 f[G::VN / 2];
        Pairs<typename G::E, G::VN>::get(f, v[k]);
        if (i < kT * G::BV) put_pairs(tile + i * G::VN, f);
      }
    } else {
      const typename G::E* q = static_cast<const typename G::E*>(p) + w.g * a.N;
#pragma unroll 8
      for (int i = w.lane; i < kT * G::NP; i += 32) {
        const int r = i / G::NP, s = i % G::NP;
        tile[i] = r < n && s < a.N ? rows::load1(q + (row0 + r) * ld + s) : 0.f;
      }
    }
  }
};

// Whether sequence rows are cut by the end of segment seg, and whether one starts in it.
constexpr int kCut = 1, kStarts = 2;        // (backward: by its beginning; whether one ends in it)

// Thread: one state of a tile, over the segments in turn; local becomes the state at
// each segment's end.  BWD: the gradients' carries, over the segments from the last.
constexpr int kCarryThreads = 128;
template <class G, bool BWD>
__global__ void __launch_bounds__(kCarryThreads) k_ssm_carry(Args a) {
  constexpr int CN = G::CPL * G::NS;
  const long long id = (long long)blockIdx.x * kCarryThreads + threadIdx.x;      // (tile, pair, lane, one of the pair)
  if (id >= (long long)a.tiles * CN * 32) return;
  const int in = (int)(id % (CN * 32)), tile = (int)(id / (CN * 32));
  const int pair = in / 64, lane = in / 2 % 32, k = pair * 2 + in % 2, i = channel_of<G>(k), j = state_of<G>(k);
  const int c = tile % a.tpg * G::CW + (lane >> 2) * G::CPL + i, n = (lane & 3) * G::NS + j;
  if (c >= a.per || n >= a.N) return;
  const float A2 = __ldg(a.A + ((long long)(tile / a.tpg) * a.per + c) * a.N + n) * kLog2e;
  float carry = 0.f;
  constexpr int AHEAD = 8;                   // segments fetched together: only the sum is serial
  for (int t0 = 0; t0 < a.n_seg; t0 += AHEAD) {
    float v[AHEAD], d[AHEAD];
    int f[AHEAD];
#pragma unroll
    for (int t = 0; t < AHEAD; ++t)
      if (t0 + t < a.n_seg) {
        const int s = BWD ? a.n_seg - 1 - t0 - t : t0 + t;
        const long long block = (long long)s * a.tiles + tile;
        f[t] = a.flags[s];
        v[t] = a.local[block * CN * 32 + in];
        d[t] = a.sdt[(block * G::CPL + i) * 32 + lane];
      }
#pragma unroll
    for (int t = 0; t < AHEAD; ++t)
      if (t0 + t < a.n_seg && (f[t] & kCut)) {   // (else nothing is handed on, and what follows starts afresh)
        const int s = BWD ? a.n_seg - 1 - t0 - t : t0 + t;
        carry = f[t] & kStarts ? v[t] : fmaf(decay(d[t], A2), carry, v[t]);
        a.local[((long long)s * a.tiles + tile) * CN * 32 + in] = carry;
      }
  }
}
template <class G, bool BWD>
static cudaError_t launch_ssm_carry(const Args& a, cudaStream_t st) {
  TraceScope tr("k_ssm_carry", st);
  const long long n = (long long)a.tiles * G::CPL * G::NS * 32;
  const unsigned blocks = (unsigned)((n + kCarryThreads - 1) / kCarryThreads);
  k_ssm_carry<G, BWD><<<blocks, kCarryThreads, 0, st>>>(a);
  return cudaGetLastError();
}

// The plan: rows of a segment, segments, channels of a tile.  Cut into segments, every SM has its
// kResident warps, but the pass that hands states on costs half as much again as the scan, and two
// launches more; whole, a sequence takes the latency of all its tokens.  So sequences of one length
// (and packed rows, as if they were one) stay whole where there are kEnough of them and their tiles, and
// earlier the shorter they are.
// Measured, bfloat16, 16 states, whole | cut in us: 2048 tokens with 384 tiles in all 221 | 234 forward and
// 996 | 786 both ways, 512 226 | 298 and 1005 | 1014; 512 tokens with 256 58 | 66 and 269 | 201, 512 67 | 103 and
// 287 | 327; 128 tokens with 160 26 | 41.  One rule for both, between the two: a forward gives the
// same bits whether or not it saves.
struct Plan {
  int NS, CPL, tpg, tiles, n_seg, cps;
  long long S;
  bool cut;
};
constexpr long long kPlanWarps = (long long)kResident * kNumSMs, kPlanEnough = 3ll * kNumSMs,
                    kPlanShort = 75000;      // tokens x tiles that the launches and the handing on are worth
inline Plan make_plan(long long rows, int n_seq, int d, int groups, int N, bool packed) {
  Plan p{};
  p.NS = N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16;
  p.CPL = p.NS <= 4 ? 4 : p.NS == 8 ? 2 : 1;
  const int per = d / groups, cw = 8 * p.CPL;
  p.tpg = (per + cw - 1) / cw;
  p.tiles = p.tpg * groups;
  // (packed rows may be one sequence)
  const int n = packed ? 1 : n_seq;
  const long long tokens = n > 0 ? rows / n : 0;
  if (rows <= 0) {
    p.S = kT;
  } else if (tokens > 0 && n * (long long)p.tiles * tokens >= kPlanEnough * tokens - kPlanShort) {
    long long k = n * (long long)p.tiles / kPlanWarps;
    p.S = tokens * (k < 1 ? 1 : k < n ? k : n);
  } else {
    p.S = (rows * p.tiles + kPlanWarps - 1) / kPlanWarps;
    if (p.S < 4 * kT) p.S = 4 * kT;
    p.S = (p.S + kT - 1) / kT * kT;
    p.cut = true;
    if (tokens > 0 && p.S >= tokens) {
      p.S = p.S / tokens * tokens;
      p.cut = false;
    }
  }
  p.n_seg = (int)((rows + p.S - 1) / p.S);
  if (p.n_seg <= 1) p.cut = false;
  p.cps = (int)((p.S + kT - 1) / kT);
  return p;
}

// The workspace: flags, local states and sums of dt (also the backward's), then what a
// forward saves, then the backward's partial sums.
struct Work {
  size_t flags, local, sdt, ckpt, part, bc, total;
};
inline Work make_work(const Plan& p, long long rows, int d, bool save) {
  auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
  const size_t lanes = (size_t)p.CPL * p.NS * 32 * 4, seg = (size_t)(p.n_seg > 0 ? p.n_seg : 1);
  Work w{};
  w.flags = 0;
  w.local = up(seg * 4);
  w.sdt = w.local + (p.cut ? up(seg * p.tiles * lanes) : 0);
  w.ckpt = w.sdt + (p.cut ? up(seg * p.tiles * p.CPL * 32 * 4) : 0);
  w.part = w.ckpt + (save ? up(seg * p.cps * p.tiles * lanes) : 0);
  w.bc = w.part + (save ? up(seg * (size_t)d * (4 * p.NS + 2) * 4) : 0);
  const size_t blocks = (size_t)(p.tiles / p.tpg) * ((p.tpg + 3) / 4);     // of the backward, each a sum of grad_B and grad_C
  w.total = w.bc + (save ? up((size_t)rows * blocks * 2 * 4 * p.NS * 4) : 0);
  return w;
}

Args args_of(const SsmArgs& g, const Plan& p, const Work& k);

}  // namespace ssm
}  // namespace cfc
