// gdr_common.cuh -- what the gated-delta-rule kernels share: sequence and
// workspace indexing, asynchronous tile copies, and warp-level matrix products
// (mma.sync fragments) in the two precision modes.
//
// The rule, per sequence and value head, with a state S [d_k, d_v]:
//   S <- exp(g_t) S,  u_t = beta_t (v_t - S^T k_t),  S <- S + k_t u_t^T,
//   o_t = scale S^T q_t.
// Over a chunk of C = 64 tokens, with G the running sum of g inside the chunk
// and S0 the state before it:
//   R_i = beta_i (v_i - exp(G_i) S0^T k_i)
//   U   = T R,  T = (I + A)^{-1},  A_ij = beta_i exp(G_i - G_j) k_i.k_j  (j < i)
//   O_i = scale exp(G_i) S0^T q_i + sum_{j<=i} P_ij U_j,
//         P_ij = scale exp(G_i - G_j) q_i.k_j
//   S1  = exp(G_C) S0 + sum_i exp(G_C - G_i) k_i U_i^T.
// T and P depend on q, k, g and beta alone, so one kernel forms them for all
// chunks at once; only S0 -> S1 is serial.  exp is only ever taken of sums of
// g over tokens that follow one another, never of their negatives, so nothing
// overflows whatever the decays are.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cfc_internal.cuh"
#include "tc_common.cuh"

namespace cfc {
namespace gdr {

constexpr int kC = 64;          // tokens of a chunk
constexpr int kMaxDk = 128;     // key width limit: the state's rows stay in one block's registers
constexpr int kMaxDv = 256;
constexpr int kPad = 4;         // floats between rows in shared memory: rows of a tile in different banks
constexpr int kLdT = kC + kPad; // a row of 64 x 64 in FP32: T - I and P in shared memory and workspace, R, U
// A serial pass takes tiles twice as wide where narrow ones no longer fit the
// SMs at once: a wide tile takes 1.4 to 1.6 times a narrow one's time, a second
// round of narrow ones 2.
constexpr bool wide_tiles(long long heads, int dv, int narrow) {
  return dv > narrow && heads * ((dv + narrow - 1) / narrow) > kNumSMs;
}
// Per chunk and head: exp(G), exp(G_C - G), beta, G / ln 2 as pairs of floats
// hi + lo, exp(G_C), and two words of bits (even rows, odd rows): the tokens that
// nothing passes, a factor of zero or a sequence's first from the zero state.
constexpr int kVec = 384;
constexpr int kVecEG = 0, kVecEGL = 64, kVecBeta = 128, kVecG2 = 192, kVecD = 320, kVecDead = 322;

// Log-decays below this are a zero factor in fp32 all the same
// (exp(-104) underflows); holding them here keeps -inf out of differences.
constexpr float kMinG = -110.f;

struct Shape {
  const int* off;     // n_seq + 1 row offsets, or NULL: n_seq sequences of rows / n_seq rows
  int n_seq;
  long long rows;
  int hk, hv, dk, dv;
  float scale;
  int per_seq;        // rows / n_seq
};

// Rows of sequence n.  Offsets are held inside [0, rows], so nothing outside
// the tensors is touched whatever the array holds.
__device__ __forceinline__ void seq_range(const Shape& s, int n, long long* start, int* len) {
  if (s.off) {
    long long a = s.off[n], b = s.off[n + 1];
    a = a < 0 ? 0 : (a > s.rows ? s.rows : a);
    b = b < a ? a : (b > s.rows ? s.rows : b);
    *start = a;
    *len = (int)(b - a);
  } else {
    *start = (long long)n * s.per_seq;
    *len = s.per_seq;
  }
}

// Chunk slots: sequence n's chunks are slots start_n / 64 + n, ...: the slots
// of different sequences never meet and need no prefix sum over lengths.
__host__ __device__ __forceinline__ long long slot_base(long long start, int n) { return start / kC + n; }
__host__ __device__ __forceinline__ long long slot_count(long long rows, int n_seq) { return rows / kC + n_seq; }

// The chunk of a slot, found by a whole warp (32 pivots a step, so up to 32
// sequences take one round of loads); false if the slot is none.  A sequence's
// slots may begin before an empty neighbour's, so the search is over
// slot_base, which rises strictly with n.
__device__ __forceinline__ bool slot_chunk(const Shape& s, long long slot, int* n_out, long long* start, int* len,
                                           int* c) {
  const int lane = threadIdx.x & 31;
  int lo = 0, size = s.n_seq;
  while (size > 1) {
    const int step = (size + 31) / 32, n = lo + lane * step;
    bool below = false;
    if (lane * step < size) {
      long long a;
      int l;
      seq_range(s, n, &a, &l);
      below = slot_base(a, n) <= slot;
    }
    const int hits = __popc(__ballot_sync(0xffffffffu, below)), skip = (hits > 0 ? hits - 1 : 0) * step;
    lo += skip;
    size = min(step, size - skip);
  }
  seq_range(s, lo, start, len);
  const long long d = slot - slot_base(*start, lo);
  *n_out = lo;
  *c = (int)d;
  return d >= 0 && d * kC < *len;
}

// ------------------------------------------------------------ async copies
__device__ __forceinline__ void cp16(void* dst, const void* src, bool on) {
  const int n = on ? 16 : 0;   // 0: the destination is filled with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Bulk copy of `bytes` (a multiple of 16, both ends 16-byte aligned) into
// shared memory; `bar` receives the bytes.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_addr(dst)), "l"(src), "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void bar_arrive_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}
// An arrival of this thread once all its cp.async so far have landed.
__device__ __forceinline__ void bar_arrive_cp(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// Barrier over the first `threads` threads that name it (1 .. 15).  A warp has
// to come to it as one, and the lanes of a wait may leave it one by one.
template <int ID, int THREADS>
__device__ __forceinline__ void group_sync() {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(THREADS) : "memory");
}
// The same, and whether `p` holds for any of them: one decision for all.
template <int ID, int THREADS>
__device__ __forceinline__ bool group_any(bool p) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)p), "n"(ID), "n"(THREADS)
      : "memory");
  return r != 0;
}
constexpr uint32_t kPolls = 1u << 20, kPollsBusy = 1u << 24;   // of a bounded wait that suspends, that polls

// rows x cols elements (cols x sizeof(E) a multiple of 16) from rows `stride`
// apart into rows `ld` apart; rows past row_end and columns past col_end are
// zeros.  col_end is a multiple of 16 bytes.
template <class E, int ROWS, int COLS, int THREADS>
__device__ __forceinline__ void load_tile(E* dst, int ld, const E* src, long long stride, int row_end, int col_end,
                                          int tid) {
  constexpr int V = 16 / sizeof(E);
  constexpr int PER = COLS / V;
  if constexpr (THREADS % PER == 0 && ROWS % (THREADS / PER) == 0) {
    constexpr int STEP = THREADS / PER;         // a thread keeps its column
    const int c = (tid % PER) * V;
    int r = tid / PER;
    const E* p = src + r * stride + c;
    E* d = dst + r * ld + c;
    const bool in = c < col_end;
#pragma unroll 8
    for (int i = 0; i < ROWS / STEP; ++i) {
      const bool on = in && r < row_end;
      cp16(d, on ? p : src, on);
      r += STEP;
      p += STEP * stride;
      d += STEP * ld;
    }
  } else {
    for (int i = tid; i < ROWS * PER; i += THREADS) {
      const int r = i / PER, c = (i % PER) * V;
      const bool on = r < row_end && c < col_end;
      cp16(dst + r * ld + c, on ? src + r * stride + c : src, on);
    }
  }
}

// Shared rows -> global rows (16-byte pieces).
template <class E, int ROWS, int COLS, int THREADS>
__device__ __forceinline__ void store_tile(E* dst, long long stride, const E* src, int ld, int row_end, int col_end,
                                           int tid) {
  constexpr int V = 16 / sizeof(E);
  constexpr int PER = COLS / V;
  for (int i = tid; i < ROWS * PER; i += THREADS) {
    const int r = i / PER, c = (i % PER) * V;
    if (r < row_end && c < col_end)
      *reinterpret_cast<uint4*>(dst + r * stride + c) = *reinterpret_cast<const uint4*>(src + r * ld + c);
  }
}

// ------------------------------------------------------------ warp products
// A matrix in shared memory, rows of ld elements.
template <class E>
struct Mat {
  E* p;
  int ld;
};

// Fragments of D[16 x 8] += A[16 x k] B[k x 8]: lane = 4 g + t holds rows g and
// g + 8, columns 2t and 2t + 1 of D.  load_b* fetches two adjacent 8-column
// tiles at once; h picks one.

// bf16 operands.
struct MBf16 {
  using E = __nv_bfloat16;
  using A = uint32_t[4];
  using B = uint32_t[4];
  __device__ static __forceinline__ void ldm(uint32_t (&r)[4], const void* p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(smem_addr(p)) : "memory");
  }
  __device__ static __forceinline__ void ldmt(uint32_t (&r)[4], const void* p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(smem_addr(p)) : "memory");
  }
  // A[m][k], k contiguous
  __device__ static __forceinline__ void load_a(A& a, const Mat<E>& m, int m0, int k0, int lane) {
    ldm(a, m.p + (m0 + (lane & 15)) * m.ld + k0 + (lane >> 4) * 8);
  }
  // B[k][n] stored [n][k], n0 .. n0 + 15
  __device__ static __forceinline__ void load_bn(B& b, const Mat<E>& m, int n0, int k0, int lane) {
    ldm(b, m.p + (n0 + (lane & 7) + (lane >> 4) * 8) * m.ld + k0 + ((lane >> 3) & 1) * 8);
  }
  __device__ static __forceinline__ void mma(float (&d)[4], const A& a, const B& b, int h) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[2 * h]), "r"(b[2 * h + 1]));
  }
};

// fp32 operands, split in registers into two TF32 values (22 significant
// bits); three TF32 products a step, the small ones into a sum of their own
// where a chain would otherwise be long.
struct MFp32 {
  static constexpr int KS = 8;        // k of one step
  struct A { uint32_t h[4], l[4]; };
  struct B { uint32_t h[4], l[4]; };
  __device__ static __forceinline__ uint32_t tf32(float x) {
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return r;
  }
  __device__ static __forceinline__ void split(uint32_t& h, uint32_t& l, float x) {
    h = tf32(x);
    l = tf32(x - __uint_as_float(h));
  }
  // A[m][k], k contiguous
  __device__ static __forceinline__ void load_a(A& a, const Mat<float>& m, int m0, int k0, int lane) {
    const float* p = m.p + (m0 + (lane >> 2)) * m.ld + k0 + (lane & 3);
    split(a.h[0], a.l[0], p[0]);
    split(a.h[1], a.l[1], p[8 * m.ld]);
    split(a.h[2], a.l[2], p[4]);
    split(a.h[3], a.l[3], p[8 * m.ld + 4]);
  }
  // A[m][k] stored [k][m]
  __device__ static __forceinline__ void load_at(A& a, const Mat<float>& m, int m0, int k0, int lane) {
    const float* p = m.p + (k0 + (lane & 3)) * m.ld + m0 + (lane >> 2);
    split(a.h[0], a.l[0], p[0]);
    split(a.h[1], a.l[1], p[8]);
    split(a.h[2], a.l[2], p[4 * m.ld]);
    split(a.h[3], a.l[3], p[4 * m.ld + 8]);
  }
  // B[k][n] stored [n][k], n0 .. n0 + 15
  __device__ static __forceinline__ void load_bn(B& b, const Mat<float>& m, int n0, int k0, int lane) {
    const float* p = m.p + (n0 + (lane >> 2)) * m.ld + k0 + (lane & 3);
    split(b.h[0], b.l[0], p[0]);
    split(b.h[1], b.l[1], p[4]);
    split(b.h[2], b.l[2], p[8 * m.ld]);
    split(b.h[3], b.l[3], p[8 * m.ld + 4]);
  }
  // B[k][n] stored [k][n]
  __device__ static __forceinline__ void load_bk(B& b, const Mat<float>& m, int n0, int k0, int lane) {
    const float* p = m.p + (k0 + (lane & 3)) * m.ld + n0 + (lane >> 2);
    split(b.h[0], b.l[0], p[0]);
    split(b.h[1], b.l[1], p[4 * m.ld]);
    split(b.h[2], b.l[2], p[8]);
    split(b.h[3], b.l[3], p[4 * m.ld + 8]);
  }
  __device__ static __forceinline__ void mma1(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  __device__ static __forceinline__ void mma(float (&d)[4], float (&lo)[4], const A& a, const B& b, int h) {
    mma1(lo, a.l, b.h[2 * h], b.h[2 * h + 1]);
    mma1(lo, a.h, b.l[2 * h], b.l[2 * h + 1]);
    mma1(d, a.h, b.h[2 * h], b.h[2 * h + 1]);
  }
  __device__ static __forceinline__ void mma(float (&d)[4], const A& a, const B& b, int h) { mma(d, d, a, b, h); }
  // two adjacent values of a row
  __device__ static __forceinline__ void put2(const Mat<float>& m, int row, int col, float v0, float v1) {
    *reinterpret_cast<float2*>(m.p + row * m.ld + col) = make_float2(v0, v1);
  }
};

using F = MFp32;                // the FP32 kernels' products

// 2^x to within 2 ulp, far below bf16's rounding.
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ------------------------------------------------------------ workspace
// Per (slot, value head).  FP32: T - I and P in rows of kLdT floats.  bf16: both as
// one image of the tensor cores' operand tiles, copied whole.  In both modes the
// vectors; when the backward is to follow also the state before the chunk and U;
// and the backward's own dS1 and dR, with dq and dk per value head where heads are
// shared.  (bf16: all of these as operand tiles too; FP32: plain rows.)
struct Workspace {
  size_t off_t, off_p, off_vec, off_order, off_s0, off_u, off_ds, off_dr, off_dq, off_dk, total;
};

Workspace plan(long long rows, int n_seq, int hk, int hv, int dk, int dv, int math, int save);

// Packed batches of up to this many sequences run longest first.  More even out
// by themselves, and ordering them, one against another by one block, would take
// longer than the rest of the preparation (1000 of 0 to 40 tokens: 68 us).
constexpr int kMaxOrder = 512;
constexpr uint32_t kImage = 32768;   // bf16: [T - I; P T] in two planes of 128 rows x 128 bytes

struct FwdArgs {
  Shape s;
  const void *q, *k, *v;
  long long ldq, ldk, ldv;        // elements from one row to the next
  const float *g, *beta;
  const float* init;
  float* final_state;
  void* o;
  char *t, *p, *s0, *u;
  float* vec;
  int* order;         // packed batches in bf16: the sequences, longest first
  int save;
  int ntile;
};

// A product reads a chunk's 64 tokens for each of its rows, the later ones with
// factors of zero: what it reads must be finite, also once rounded to bf16 or TF32.
constexpr float kLargest = 3.38953139e38f;      // bf16's largest
__device__ __forceinline__ bool finite(float v) { return fabsf(v) <= kLargest; }
// The preparation's part of that: entries of A or T that are not (from a NaN, an
// infinity or an overflow) become zeros, and the row's beta a NaN, by which the serial
// pass marks the token and all that follow.
__device__ __forceinline__ void drop(float& v, float* vec, int row) {
  if (finite(v)) return;
  v = 0.f;
  vec[kVecBeta + row] = nanf("");
}
// Sum of two pairs hi + lo.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  const float s = a.x + b.x, t = s - a.x, e = ((a.x - (s - t)) + (b.x - t)) + (a.y + b.y), h = s + e;
  return make_float2(h, e - (h - s));
}

// dg of a row, zero where its bit says so (a NaN stays).
__device__ __forceinline__ float alive(float dg, unsigned dead, int lane) { return (dead >> lane) & 1 ? 0.f * dg : dg; }

// g and beta of rows 2 lane and 2 lane + 1: (x, y) and (z, w).
__device__ __forceinline__ float4 load_gates(const FwdArgs& a, long long row0, int rows, int h, int lane) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  const long long at = (row0 + 2 * lane) * a.s.hv + h;
  if (2 * lane < rows) { v.x = a.g[at]; v.z = a.beta[at]; }
  if (2 * lane + 1 < rows) { v.y = a.g[at + a.s.hv]; v.w = a.beta[at + a.s.hv]; }
  return v;
}
// The decays of a chunk's head, by one warp with load_gates' values: into
// `vec`, and for the block G / ln 2 as pairs hi + lo and beta.
__device__ __forceinline__ void chunk_decays(const float4& gb, int lane, bool from_zero, float2* g2, float* bet,
                                             float* vec) {
  // dg is zero there; the sums it is a difference of would leave their rounding.
  const unsigned even = __ballot_sync(0xffffffffu, gb.x < kMinG || (from_zero && lane == 0));
  const unsigned odd = __ballot_sync(0xffffffffu, gb.y < kMinG);
  if (lane == 0) *reinterpret_cast<uint2*>(vec + kVecDead) = make_uint2(even, odd);
  // Running sum of g as a pair of floats hi + lo: differences of G then carry
  // no more than their own fp32 rounding, however far the sum has gone.  (In
  // double this was the longest part of the kernel: the fp64 rate is 1/64.)
  float2 x[2] = {make_float2(gb.x < kMinG ? kMinG : gb.x, 0.f), make_float2(gb.y < kMinG ? kMinG : gb.y, 0.f)};  // a NaN stays
  x[1] = add2(x[0], x[1]);
  float2 run = x[1];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const float2 y = make_float2(__shfl_up_sync(0xffffffffu, run.x, d), __shfl_up_sync(0xffffffffu, run.y, d));
    if (lane >= d) run = add2(run, y);
  }
  const float2 total = make_float2(__shfl_sync(0xffffffffu, run.x, 31), __shfl_sync(0xffffffffu, run.y, 31));
  float2 before = make_float2(__shfl_up_sync(0xffffffffu, run.x, 1), __shfl_up_sync(0xffffffffu, run.y, 1));
  if (lane == 0) before = make_float2(0.f, 0.f);
  const float2 G[2] = {add2(before, x[0]), run};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 2 * lane + i;
    // / ln 2 in the same form
    constexpr float kH = 1.442695041f, kL = (float)(1.4426950408889634074 - (double)kH);
    const float p = G[i].x * kH, e = fmaf(G[i].x, kH, -p) + fmaf(G[i].x, kL, G[i].y * kH), u = p + e;
    const float2 gu = make_float2(u, e - (u - p));
    g2[r] = gu;
    vec[kVecEG + r] = expf(G[i].x + G[i].y);
    vec[kVecEGL + r] = expf((total.x - G[i].x) + (total.y - G[i].y));
    bet[r] = vec[kVecBeta + r] = i ? gb.w : gb.z;
    reinterpret_cast<float2*>(vec + kVecG2)[r] = gu;
  }
  if (lane == 0) vec[kVecD] = expf(total.x + total.y);
}

// T = (I + A)^{-1} in place of A, 64 x 64 and strictly lower triangular in fp32
// with rows of LDA, by a block of 4 warps of which warp w wrote rows 16 w ..;
// ends with a block barrier.  The blocks off the diagonal come of fp32-accurate
// products, also where T is rounded to bf16 afterwards: an error of A21 T11 is
// multiplied by T22, whose rows have sums far above 1 where keys repeat.
template <int LDA>
__device__ __forceinline__ void invert(float* am, int warp, int lane) {
  const int m0 = warp * 16, g = lane >> 2, t2 = (lane & 3) * 2;
  // Diagonal blocks.
  if (lane < 16) {
    float x[16];
    const float* blk = am + m0 * LDA + m0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v = i == lane ? 1.f : 0.f, u = 0.f;
#pragma unroll
      for (int m = 0; m < i; m += 4) {
        const float4 b = *reinterpret_cast<const float4*>(blk + i * LDA + m);
        v = fmaf(-b.x, x[m], v);
        if (m + 1 < i) u = fmaf(-b.y, x[m + 1], u);
        if (m + 2 < i) v = fmaf(-b.z, x[m + 2], v);
        if (m + 3 < i) u = fmaf(-b.w, x[m + 3], u);
      }
      x[i] = v + u;
    }
    __syncwarp(0xffffu);
#pragma unroll
    for (int i = 0; i < 16; ++i) am[(m0 + i) * LDA + m0 + lane] = x[i];
  }
  __syncthreads();
  // 16 -> 32: warps 0 and 1, a pair each; y = A21 T11, then -T22 y.
  if (warp < 2) {
    float* t21 = am + (warp * 32 + 16) * LDA + warp * 32;
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
      float d[2][4] = {}, e[2][4] = {};
      const float* fa = pass == 0 ? t21 : t21 + 16;
      const float* fb = pass == 0 ? t21 - 16 * LDA : t21;
      const Mat<float> ma{const_cast<float*>(fa), LDA}, mb{const_cast<float*>(fb), LDA};
#pragma unroll
      for (int k0 = 0; k0 < 16; k0 += 8) {
        MFp32::A xa;
        MFp32::B xb;
        MFp32::load_a(xa, ma, 0, k0, lane);
        MFp32::load_bk(xb, mb, 0, k0, lane);
        MFp32::mma(d[0], e[0], xa, xb, 0);
        MFp32::mma(d[1], e[1], xa, xb, 1);
      }
      __syncwarp();
      const float sg = pass == 0 ? 1.f : -1.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        *reinterpret_cast<float2*>(t21 + g * LDA + j * 8 + t2) = make_float2(sg * (d[j][0] + e[j][0]), sg * (d[j][1] + e[j][1]));
        *reinterpret_cast<float2*>(t21 + (g + 8) * LDA + j * 8 + t2) = make_float2(sg * (d[j][2] + e[j][2]), sg * (d[j][3] + e[j][3]));
      }
      __syncwarp();
    }
  }
  __syncthreads();
  // 32 -> 64: warp w the rows 16 (w & 1) and the columns 16 (w >> 1) of each product.
  {
    float* t21 = am + 32 * LDA + (warp >> 1) * 16;
    float* mine = t21 + (warp & 1) * 16 * LDA;
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
      float d[2][4] = {}, e[2][4] = {};
      const float* fa = am + (32 + (warp & 1) * 16) * LDA + (pass == 0 ? 0 : 32);
      const float* fb = pass == 0 ? am + (warp >> 1) * 16 : t21;
      const Mat<float> ma{const_cast<float*>(fa), LDA}, mb{const_cast<float*>(fb), LDA};
#pragma unroll
      for (int k0 = 0; k0 < 32; k0 += 8) {
        MFp32::A xa;
        MFp32::B xb;
        MFp32::load_a(xa, ma, 0, k0, lane);
        MFp32::load_bk(xb, mb, 0, k0, lane);
        MFp32::mma(d[0], e[0], xa, xb, 0);
        MFp32::mma(d[1], e[1], xa, xb, 1);
      }
      __syncthreads();
      const float sg = pass == 0 ? 1.f : -1.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        *reinterpret_cast<float2*>(mine + g * LDA + j * 8 + t2) = make_float2(sg * (d[j][0] + e[j][0]), sg * (d[j][1] + e[j][1]));
        *reinterpret_cast<float2*>(mine + (g + 8) * LDA + j * 8 + t2) = make_float2(sg * (d[j][2] + e[j][2]), sg * (d[j][3] + e[j][3]));
      }
      __syncthreads();
    }
  }
}

struct BwdArgs {
  Shape s;
  const void *q, *k, *v, *go;
  long long ldq, ldk, ldv;
  const float* gfinal;
  float* ginit;
  void *gq, *gk, *gv, *gg, *gbeta;
  const char *t, *p, *s0, *u;
  char *ds, *dr;
  const float* vec;
  const int* order;
  float *pdq, *pdk;        // per value head [rows, hv, dk], or NULL
  int ntile;
};

// bf16 (cfc_gdr_tc.cu): what is formed for all chunks at once, the serial passes.
cudaError_t launch_prep_tc(const FwdArgs& a, int dk_tile, int planes, cudaStream_t st);
cudaError_t launch_scan_tc(const FwdArgs& a, int dk_tile, int planes, cudaStream_t st);
cudaError_t launch_scan_bwd_tc(const BwdArgs& a, int dk_tile, cudaStream_t st);
int* gdr_tc_error_word();      // on the device, or NULL
// The gradients that follow them (cfc_gdr_grad.cu).
cudaError_t launch_grad_tc(const BwdArgs& a, int dk_tile, cudaStream_t st);
int* gdr_grad_error_word();

}  // namespace gdr
}  // namespace cfc
