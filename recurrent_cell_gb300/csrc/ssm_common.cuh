// ssm_common.cuh -- what the selective scan's kernels share: the split of rows and
// channels, tiles of a chunk in shared memory, and the elementary functions.
//
// Per sequence and channel c, with a state h [N] in fp32, and per token
//   dt = softplus(delta + bias),  h <- exp(dt A) h + dt x B,
//   y = (C . h + D x) silu(z),
// B and C [N] shared by the channels of a group.
//
// A warp takes a tile of channels of one group over a segment of rows: 4 lanes
// share a channel's states and 8 lanes the tile's channels, so a thread keeps
// CPL channels x NS states in registers and sums over states need two lane steps,
// sums over channels three.  Rows go by chunks of kT: what depends on a token and
// channel alone (softplus, dt x, the gate) is formed once by whichever lane loaded
// it, through shared memory; the loop over tokens is left with an exponential and
// four multiply-adds a state.
//
// Segments are ranges of the rows of all sequences together, whatever the sequences'
// lengths: a state is set afresh where a sequence begins, and handed on where a
// segment's end cuts one.  Those states come from a pass of their own (the
// segment's own end state and sum of dt, since a product of decays is the exp of a
// sum) and a short serial pass over segments.
#pragma once

#include "row_ops.cuh"
#include "seq_rows.cuh"

namespace cfc {
namespace ssm {

using seqs::Seqs;
using seqs::Where;

constexpr int kT = 16;                       // rows of a chunk
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

struct Args {
  const void *x, *delta, *z, *B, *C;
  long long ldx, ldd, ldz, ldb, ldc;         // elements from row to row
  const float *A, *D, *bias;
  Seqs s;
  int d, groups, N;
  int per, tpg;                              // channels of a group, its tiles
  int vec_bc;                                // rows of B and C are whole 16-byte vectors
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

// NS states and CPL channels a thread.
template <class E_, int NS_, int CPL_>
struct Cfg {
  using E = E_;
  static constexpr int NS = NS_, CPL = CPL_, NP = 4 * NS, CW = 8 * CPL;
  static constexpr int VN = 16 / sizeof(E);                  // channels of a 16-byte vector
  static constexpr int LPR = CW / VN, RPP = 32 / LPR;        // lanes a row, rows a pass
  static constexpr int P = (kT + RPP - 1) / RPP;             // passes of a chunk
  static constexpr int BV = NP * (int)sizeof(E) / 16;        // vectors of a row of B
  static constexpr int BL = (kT * BV + 31) / 32;             // of a chunk, a lane
};

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// exp(v), v <= 0, to about an fp32 unit and a half: 2^hi (1 + lo ln 2), hi + lo = v / ln 2.
__device__ __forceinline__ float exp_neg(float v) {
  const float hi = fmaxf(v, -126.f * kLn2) * kLog2e;         // (a NaN goes to the sum below)
  const float lo = fmaf(fmaxf(v, -126.f * kLn2), kLog2e, -hi);
  const float e = ex2(hi);
  return fmaf(e * lo, kLn2, e);
}
// softplus(v) = max(v, 0) + log1p(e), e = exp(-|v|); log1p(e) = 2 atanh(s), s = e / (2 + e) <= 1/3,
// by its Taylor series up to s^15 (the rest is below 2e-9 of it).  sig: sigmoid(v).
__device__ __forceinline__ float softplus(float v, float* sig = nullptr) {
  const float e = exp_neg(-fabsf(v));
  const float s = __fdividef(e, 2.f + e), q = s * s;
  float p = 1.f / 15.f;
  p = fmaf(p, q, 1.f / 13.f);
  p = fmaf(p, q, 1.f / 11.f);
  p = fmaf(p, q, 1.f / 9.f);
  p = fmaf(p, q, 1.f / 7.f);
  p = fmaf(p, q, 1.f / 5.f);
  p = fmaf(p, q, 1.f / 3.f);
  p = fmaf(p, q, 1.f);
  if (sig) {
    const float r = __fdividef(1.f, 1.f + e);
    *sig = v >= 0.f ? r : e * r;
  }
  return fmaf(2.f * s, p, v > 0.f || v != v ? v : 0.f);
}
__device__ __forceinline__ float sigmoid(float v) {
  const float e = exp_neg(-fabsf(v)), r = __fdividef(1.f, 1.f + e);
  return v != v ? v : (v >= 0.f ? r : e * r);
}

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

template <class G>
__device__ __forceinline__ void load_A(const Args& a, const Tile<G>& w, float (&A2)[G::CPL][G::NS]) {
#pragma unroll
  for (int i = 0; i < G::CPL; ++i)
#pragma unroll
    for (int j = 0; j < G::NS; ++j) {
      const int n = w.sl * G::NS + j;
      A2[i][j] = w.has(i) && n < a.N ? __ldg(a.A + (long long)w.channel(i) * a.N + n) * kLog2e : 0.f;
    }
}

// States [sequence, d, N] as the caller has them.
template <class G>
__device__ __forceinline__ void load_state(const Args& a, const Tile<G>& w, const float* p, long long seq, float (&h)[G::CPL][G::NS]) {
#pragma unroll
  for (int i = 0; i < G::CPL; ++i)
#pragma unroll
    for (int j = 0; j < G::NS; ++j) {
      const int n = w.sl * G::NS + j;
      h[i][j] = p && w.has(i) && n < a.N ? p[(seq * a.d + w.channel(i)) * a.N + n] : 0.f;
    }
}
template <class G>
__device__ __forceinline__ void store_state(const Args& a, const Tile<G>& w, float* p, long long seq, const float (&h)[G::CPL][G::NS]) {
#pragma unroll
  for (int i = 0; i < G::CPL; ++i)
#pragma unroll
    for (int j = 0; j < G::NS; ++j) {
      const int n = w.sl * G::NS + j;
      if (w.has(i) && n < a.N) p[(seq * a.d + w.channel(i)) * a.N + n] = h[i][j];
    }
}
// States as the kernels hand them on: a warp's registers side by side.
template <class G>
__device__ __forceinline__ long long lane_at(long long block, int k, int lane) {
  return (block * (G::CPL * G::NS / 2) + k) * 32 + lane;
}
template <class G>
__device__ __forceinline__ void load_lanes(const float* p, long long block, int lane, float (&h)[G::CPL][G::NS]) {
#pragma unroll
  for (int i = 0; i < G::CPL; ++i)
#pragma unroll
    for (int j = 0; j < G::NS; j += 2) {
      const float2 v = reinterpret_cast<const float2*>(p)[lane_at<G>(block, (i * G::NS + j) / 2, lane)];
      h[i][j] = v.x;
      h[i][j + 1] = v.y;
    }
}
template <class G>
__device__ __forceinline__ void store_lanes(float* p, long long block, int lane, const float (&h)[G::CPL][G::NS]) {
#pragma unroll
  for (int i = 0; i < G::CPL; ++i)
#pragma unroll
    for (int j = 0; j < G::NS; j += 2)
      reinterpret_cast<float2*>(p)[lane_at<G>(block, (i * G::NS + j) / 2, lane)] = make_float2(h[i][j], h[i][j + 1]);
}

// A chunk's vectors of a [rows, channels] tensor, zeros outside.
template <class G>
__device__ __forceinline__ void load_raw(const Tile<G>& w, const void* p, long long ld, long long row0, int n, uint4 (&v)[G::P]) {
  const typename G::E* q = static_cast<const typename G::E*>(p) + w.c0 + w.col();
#pragma unroll
  for (int k = 0; k < G::P; ++k) {
    v[k] = make_uint4(0, 0, 0, 0);
    if (w.row(k) < n && w.col() < w.cols) v[k] = __ldg(reinterpret_cast<const uint4*>(q + (row0 + w.row(k)) * ld));
  }
}
template <class E> struct Unpack;
template <> struct Unpack<__nv_bfloat16> {
  using V = rows::Vec<__nv_bfloat16, 8>;
  __device__ static __forceinline__ void get(float (&f)[8], const uint4& v) { V::get(f, v); }
  __device__ static __forceinline__ uint4 make(const float (&f)[8]) { return V::make(f); }
};
template <> struct Unpack<float> {
  __device__ static __forceinline__ void get(float (&f)[4], const uint4& v) {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y); f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
  }
  __device__ static __forceinline__ uint4 make(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

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

// A chunk's rows of B or C: fetched into registers ahead (whole vectors), or element
// by element when they are put into the tile [kT][NP].
template <class G>
struct Rows {
  uint4 v[G::BL];
  __device__ __forceinline__ void fetch(const Args& a, const Tile<G>& w, const void* p, long long ld, long long row0, int n) {
    if (!a.vec_bc) return;
    const typename G::E* q = static_cast<const typename G::E*>(p) + w.g * a.N;
#pragma unroll
    for (int k = 0; k < G::BL; ++k) {
      const int i = k * 32 + w.lane, r = i / G::BV;
      v[k] = make_uint4(0, 0, 0, 0);
      if (r < n) v[k] = __ldg(reinterpret_cast<const uint4*>(q + (row0 + r) * ld + i % G::BV * G::VN));
    }
  }
  __device__ __forceinline__ void stage(const Args& a, const Tile<G>& w, const void* p, long long ld, long long row0, int n,
                                        float* tile) const {
    if (a.vec_bc) {
#pragma unroll
      for (int k = 0; k < G::BL; ++k) {
        const int i = k * 32 + w.lane;
        float f[G::VN];
        Unpack<typename G::E>::get(f, v[k]);
        if (i < kT * G::BV) put(tile + i * G::VN, f);
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
  const int pair = in / 64, lane = in / 2 % 32, k = pair * 2 + in % 2, i = k / G::NS, j = k % G::NS;
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
        carry = f[t] & kStarts ? v[t] : fmaf(ex2(A2 * d[t]), carry, v[t]);
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

// The plan: rows of a segment, segments, channels of a tile.  Enough warps for every SM
// (kWarps in all) where sequences are long enough; sequences of one length stay whole
// where there are kEnough of them and their tiles, since the pass that hands states on costs
// about as much as half of the scan.
struct Plan {
  int NS, CPL, tpg, tiles, n_seg, cps;
  long long S;
  bool cut;
};
constexpr long long kPlanWarps = 16ll * kNumSMs, kPlanEnough = 4ll * kNumSMs;
inline Plan make_plan(long long rows, int n_seq, int d, int groups, int N, bool packed) {
  Plan p{};
  p.NS = N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16;
  p.CPL = p.NS <= 4 ? 4 : p.NS == 8 ? 2 : 1;
  const int per = d / groups, cw = 8 * p.CPL;
  p.tpg = (per + cw - 1) / cw;
  p.tiles = p.tpg * groups;
  const long long tokens = packed || n_seq == 0 ? 0 : rows / n_seq;
  if (rows <= 0) {
    p.S = kT;
  } else if (tokens > 0 && n_seq * (long long)p.tiles >= kPlanEnough) {
    long long k = n_seq * (long long)p.tiles / kPlanWarps;
    p.S = tokens * (k < 1 ? 1 : k);
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
