// cfc_gdr.cu -- forward of the gated delta rule over whole sequences, in
// chunks of 64 tokens (the formulas are at the top of gdr_common.cuh).
//
//   k_gdr_prep   one block per (chunk, value head): the decays, T and P
//   k_gdr_scan   one block per (sequence, value head, tile of value columns):
//                the serial pass over the chunks, the state in registers
//
// The state's columns do not touch one another, so a head's value columns are
// split over blocks: narrow tiles where there are few heads (the serial pass
// is then a chain of latencies, and every block shortens it by itself), wide
// tiles where the heads alone fill the GPU (then the tiles' shared operands
// are read fewer times).
#include "gdr_common.cuh"

namespace cfc {
namespace gdr {

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
  int save;
  int ntile;
};

// ------------------------------------------------------------------- prep
template <class P, int DK>
struct PrepSmem {
  using E = typename P::E;
  static constexpr int LDK = DK + P::PAD;
  static constexpr int LDA = kC + 1;
  E k[kC * LDK], q[kC * LDK];
  float a[kC * LDA];      // A, then T
  float x[32 * 33];       // A21 T11 of the last join
  float ghi[kC], glo[kC], beta[kC];
};

// T = (I + A)^{-1} of the unit lower triangular I + A: 16 x 16 diagonal blocks
// by forward substitution (one warp each, a column a lane), then pairs of
// blocks joined by T21 = -T22 A21 T11.  All in fp32: products of T feed the
// state, and its entries reach far above A's when keys repeat.
template <class P, int DK, int PL>
__global__ void __launch_bounds__(128) k_gdr_prep(FwdArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  using E = typename P::E;
  using S = PrepSmem<P, DK>;
  S& sm = *reinterpret_cast<S*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x % a.s.hv;
  const long long slot = blockIdx.x / a.s.hv;
  int n, len, c;
  long long start;
  if (!slot_chunk(a.s, slot, &n, &start, &len, &c)) return;
  const long long row0 = start + (long long)c * kC;
  const int rows = min(kC, len - c * kC);
  const int hq = h / (a.s.hv / a.s.hk);
  load_tile<E, kC, DK, 128>(sm.k, S::LDK, static_cast<const E*>(a.k) + row0 * a.ldk + (long long)hq * a.s.dk, a.ldk,
                            rows, a.s.dk, tid);
  load_tile<E, kC, DK, 128>(sm.q, S::LDK, static_cast<const E*>(a.q) + row0 * a.ldq + (long long)hq * a.s.dk, a.ldq,
                            rows, a.s.dk, tid);
  cp_commit();
  const long long id = slot * a.s.hv + h;
  float* vec = a.vec + id * kVec;
  if (warp == 0) {
    // Running sum of g in double: differences of G then carry no more than
    // their own fp32 rounding, however far the sum has gone.
    double x[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 2 * lane + i;
      x[i] = r < rows ? (double)fmaxf(a.g[(row0 + r) * a.s.hv + h], kMinG) : 0.0;
      // fmaxf drops a NaN: put it back
      if (r < rows && isnan(a.g[(row0 + r) * a.s.hv + h])) x[i] = (double)a.g[(row0 + r) * a.s.hv + h];
    }
    double run = x[0] + x[1];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, run, d);
      run += lane >= d ? y : 0.0;
    }
    const double total = __shfl_sync(0xffffffffu, run, 31);
    const double G[2] = {run - x[1], run};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 2 * lane + i;
      const float hi = (float)G[i], lo = (float)(G[i] - (double)hi);
      const float b = r < rows ? a.beta[(row0 + r) * a.s.hv + h] : 0.f;
      sm.ghi[r] = hi;
      sm.glo[r] = lo;
      sm.beta[r] = b;
      vec[kVecEG + r] = expf((float)G[i]);
      vec[kVecEGL + r] = expf((float)(total - G[i]));
      vec[kVecBeta + r] = b;
      vec[kVecGHi + r] = hi;
      vec[kVecGLo + r] = lo;
    }
    if (lane == 0) vec[kVecD] = expf((float)total);
  }
  cp_wait<0>();
  __syncthreads();

  // Rows 16 warp .. of q k^T and k k^T, columns up to the diagonal block.
  const Mat<E> mk{sm.k, S::LDK, 0}, mq{sm.q, S::LDK, 0};
  const int m0 = warp * 16, g = lane >> 2, t2 = (lane & 3) * 2;
  float aq[8][4] = {}, ak[8][4] = {};
  for (int k0 = 0; k0 < DK; k0 += P::KS) {
    typename P::template A<1> fq, fk;
    P::load_a(fq, mq, m0, k0, lane);
    P::load_a(fk, mk, m0, k0, lane);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j > warp) continue;
      typename P::template B<1> fb;
      P::load_bn(fb, mk, j * 16, k0, lane);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        P::mma(aq[2 * j + hf], fq, fb, hf);
        P::mma(ak[2 * j + hf], fk, fb, hf);
      }
    }
  }
  E* pout = reinterpret_cast<E*>(a.p) + id * (kC * kC);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      const int i = m0 + g + rr * 8;
      float pv[2];
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const int col = j * 8 + t2 + cc;
        float l = 0.f;
        if (col <= i) l = expf((sm.ghi[i] - sm.ghi[col]) + (sm.glo[i] - sm.glo[col]));
        pv[cc] = col <= i ? a.s.scale * l * aq[j][rr * 2 + cc] : 0.f;
        sm.a[i * S::LDA + col] = col < i ? sm.beta[i] * l * ak[j][rr * 2 + cc] : 0.f;
      }
      P::template put2<1>(Mat<E>{pout, kC, 0}, i, j * 8 + t2, pv[0], pv[1]);
    }
  }
  __syncthreads();

  // Diagonal blocks.
  if (lane < 16) {
    float x[16];
    const float* blk = sm.a + (m0)*S::LDA + m0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v = i == lane ? 1.f : 0.f;
#pragma unroll
      for (int m = 0; m < i; ++m) v = fmaf(-blk[i * S::LDA + m], x[m], v);
      x[i] = v;
    }
    __syncwarp(0xffffu);
    for (int i = 0; i < 16; ++i) sm.a[(m0 + i) * S::LDA + m0 + lane] = x[i];
  }
  __syncthreads();
  // 16 -> 32: warps 0, 1 the first pair, 2, 3 the second; y = A21 T11, then -T22 y.
  {
    const int b0 = (warp >> 1) * 32, half = tid & 63;
    const int r = half >> 2, c4 = (half & 3) * 4;
    float y[4] = {};
    for (int m = 0; m < 16; ++m) {
      const float av = sm.a[(b0 + 16 + r) * S::LDA + b0 + m];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = fmaf(av, sm.a[(b0 + m) * S::LDA + b0 + c4 + e], y[e]);
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) sm.a[(b0 + 16 + r) * S::LDA + b0 + c4 + e] = y[e];
    __syncthreads();
    float z[4] = {};
    for (int m = 0; m < 16; ++m) {
      const float tv = sm.a[(b0 + 16 + r) * S::LDA + b0 + 16 + m];
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] = fmaf(-tv, sm.a[(b0 + 16 + m) * S::LDA + b0 + c4 + e], z[e]);
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) sm.a[(b0 + 16 + r) * S::LDA + b0 + c4 + e] = z[e];
    __syncthreads();
  }
  // 32 -> 64
  {
    const int r = tid >> 2, c8 = (tid & 3) * 8;
    float y[8] = {};
    for (int m = 0; m < 32; ++m) {
      const float av = sm.a[(32 + r) * S::LDA + m];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = fmaf(av, sm.a[m * S::LDA + c8 + e], y[e]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sm.x[r * 33 + c8 + e] = y[e];
    __syncthreads();
    float z[8] = {};
    for (int m = 0; m < 32; ++m) {
      const float tv = sm.a[(32 + r) * S::LDA + 32 + m];
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = fmaf(-tv, sm.x[m * 33 + c8 + e], z[e]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sm.a[(32 + r) * S::LDA + c8 + e] = z[e];
    __syncthreads();
  }
  E* tout = reinterpret_cast<E*>(a.t) + id * (2 * kC * kC);
  const Mat<E> mt{tout, kC, kC * kC};
  for (int i = tid; i < kC * kC / 2; i += 128) {
    const int r = i / (kC / 2), col = (i % (kC / 2)) * 2;
    P::template put2<PL>(mt, r, col, sm.a[r * S::LDA + col], sm.a[r * S::LDA + col + 1]);
  }
}

// ------------------------------------------------------------------- scan
// WM x 4 warps: warp (wm, wn) holds 16 MT value columns (rows of S^T) by a
// quarter of the key width, and forms a quarter of the tokens of R, U and O.
// Operands that all four need pass through shared memory: three barriers a
// chunk.  PL = 2: the operands of the serial chain in two planes.
template <class P, int DK, int MT, int WM, int PL>
struct ScanCfg {
  using E = typename P::E;
  static constexpr int DVT = 16 * MT * WM, THREADS = 128 * WM;
  static constexpr int LDK = DK + P::PAD, LDT = kC + P::PAD, LDV = DVT + P::PAD;
  static constexpr int NTS = DK / 32;                 // 8-column tiles of S^T a warp
  static constexpr int ST = P::STAGES;
  static constexpr int kQ = kC * LDK;                 // elements of each staged operand
  static constexpr int kT = PL * kC * LDT, kP = kC * LDT, kV = kC * LDV;
  static constexpr int STAGE = 2 * kQ + kT + kP + kV;
  static constexpr int SOP = PL * DVT * LDK, ROP = PL * DVT * LDT, UOP = DVT * LDT;
  // U and its decayed copy lie over the state operand, which is free by then
  static constexpr bool ALIAS = (size_t)(ST * STAGE + SOP + 2 * ROP + UOP + kV) * sizeof(E) + 2 * kVec * 4 > 227u * 1024u;
  static constexpr int ELEMS = ST * STAGE + (ALIAS ? (SOP > UOP + ROP ? SOP : UOP + ROP) : SOP + UOP + ROP) + ROP + kV;
  static constexpr size_t BYTES = (size_t)ELEMS * sizeof(E) + (size_t)ST * kVec * 4;
  static constexpr bool FITS = BYTES <= 227u * 1024u;
};

template <class P, int DK, int MT, int WM, int PL>
__global__ void __launch_bounds__(128 * WM) k_gdr_scan(FwdArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  using C = ScanCfg<P, DK, MT, WM, PL>;
  using E = typename P::E;
  constexpr int NTS = C::NTS, ST = C::ST;
  float* vecs = reinterpret_cast<float*>(smem_raw);
  E* stage = reinterpret_cast<E*>(vecs + ST * kVec);
  E* sop_p = stage + ST * C::STAGE;
  E* uop_p = C::ALIAS ? sop_p : sop_p + C::SOP;
  E* ukop_p = uop_p + C::UOP;
  E* rop_p = sop_p + (C::ELEMS - ST * C::STAGE - C::ROP - C::kV);
  E* ost = rop_p + C::ROP;
  const Mat<E> sop{sop_p, C::LDK, C::DVT * C::LDK}, rop{rop_p, C::LDT, C::DVT * C::LDT}, uop{uop_p, C::LDT, 0},
      ukop{ukop_p, C::LDT, C::DVT * C::LDT};

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wn = warp & 3, wm = warp >> 2;
  const int g = lane >> 2, t2 = (lane & 3) * 2;
  const int tile = blockIdx.x % a.ntile;
  const long long sh = blockIdx.x / a.ntile;
  const int h = (int)(sh % a.s.hv), n = (int)(sh / a.s.hv);
  const int hq = h / (a.s.hv / a.s.hk);
  const int dk = a.s.dk, dv = a.s.dv, dv0 = tile * C::DVT, dvn = min(C::DVT, dv - dv0);
  const int m0 = wm * 16 * MT;
  long long start;
  int len;
  seq_range(a.s, n, &start, &len);
  const int nc = (len + kC - 1) / kC;
  const long long slot0 = slot_base(start, n);
  const E* q = static_cast<const E*>(a.q) + start * a.ldq + (long long)hq * dk;
  const E* k = static_cast<const E*>(a.k) + start * a.ldk + (long long)hq * dk;
  const E* v = static_cast<const E*>(a.v) + start * a.ldv + (long long)h * dv + dv0;
  E* o = static_cast<E*>(a.o) + (start * a.s.hv + h) * dv + dv0;
  const long long ldo = (long long)a.s.hv * dv;

  auto fetch = [&](int c, int st) {
    E* b = stage + st * C::STAGE;
    const int rows = min(kC, len - c * kC);
    const long long r0 = (long long)c * kC, id = (slot0 + c) * a.s.hv + h;
    load_tile<E, kC, DK, C::THREADS>(b, C::LDK, k + r0 * a.ldk, a.ldk, rows, dk, tid);
    load_tile<E, kC, DK, C::THREADS>(b + C::kQ, C::LDK, q + r0 * a.ldq, a.ldq, rows, dk, tid);
    load_tile<E, kC, C::DVT, C::THREADS>(b + 2 * C::kQ, C::LDV, v + r0 * a.ldv, a.ldv, rows, dvn, tid);
    const E* tp = reinterpret_cast<const E*>(a.t) + id * (2 * kC * kC);
#pragma unroll
    for (int i = 0; i < PL; ++i)
      load_tile<E, kC, kC, C::THREADS>(b + 2 * C::kQ + C::kV + i * kC * C::LDT, C::LDT, tp + i * kC * kC, kC, kC, kC,
                                       tid);
    load_tile<E, kC, kC, C::THREADS>(b + 2 * C::kQ + C::kV + C::kT, C::LDT,
                                     reinterpret_cast<const E*>(a.p) + id * (kC * kC), kC, kC, kC, tid);
    for (int i = tid; i < kVec / 4; i += C::THREADS) cp16(vecs + st * kVec + i * 4, a.vec + id * kVec + i * 4, true);
    cp_commit();
  };

  float s[MT][NTS][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < NTS; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = m0 + mt * 16 + g + (e >> 1) * 8, col = wn * (DK / 4) + nt * 8 + t2 + (e & 1);
        s[mt][nt][e] = a.init && r < dvn && col < dk ? a.init[(sh * dk + col) * dv + dv0 + r] : 0.f;
      }

  if (nc > 0) fetch(0, 0);
  for (int c = 0; c < nc; ++c) {
    const int st = ST == 2 ? (c & 1) : 0;
    E* b = stage + st * C::STAGE;
    const Mat<E> mk{b, C::LDK, 0}, mq{b + C::kQ, C::LDK, 0}, mt_{b + 2 * C::kQ + C::kV, C::LDT, kC * C::LDT},
        mp{b + 2 * C::kQ + C::kV + C::kT, C::LDT, 0};
    const E* vs = b + 2 * C::kQ;
    const float* vec = vecs + st * kVec;
    const int rows = min(kC, len - c * kC);
    cp_wait<0>();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NTS; ++nt)
#pragma unroll
        for (int rr = 0; rr < 2; ++rr)
          P::template put2<PL>(sop, m0 + mt * 16 + g + rr * 8, wn * (DK / 4) + nt * 8 + t2, s[mt][nt][2 * rr],
                               s[mt][nt][2 * rr + 1]);
    __syncthreads();
    if (ST == 2 && c + 1 < nc) fetch(c + 1, (c + 1) & 1);
    if (c > 0)
      store_tile<E, kC, C::DVT, C::THREADS>(o + (long long)(c - 1) * kC * ldo, ldo, ost, C::LDV, kC, dvn, tid);
    if (a.save)
      store_tile<E, C::DVT, DK, C::THREADS>(
          reinterpret_cast<E*>(a.s0) + (((slot0 + c) * a.s.hv + h) * dv + dv0) * dk, dk, sop_p, C::LDK, dvn, dk, tid);

    // S0^T k and S0^T q of this warp's 16 tokens
    float ar[MT][2][4] = {}, ao[MT][2][4] = {};
#pragma unroll
    for (int k0 = 0; k0 < DK; k0 += P::KS) {
      typename P::template B<1> bk, bq;
      P::load_bn(bk, mk, wn * 16, k0, lane);
      P::load_bn(bq, mq, wn * 16, k0, lane);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        typename P::template A<PL> fa;
        P::load_a(fa, sop, m0 + mt * 16, k0, lane);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          P::mma(ar[mt][hf], fa, bk, hf);
          // the outputs leave in the stored type: one plane of the state is enough
          if constexpr (PL == 2) P::mma1(ao[mt][hf], fa.r[0], bq.r[0][2 * hf], bq.r[0][2 * hf + 1]);
          else P::mma(ao[mt][hf], fa, bq, hf);
        }
      }
    }
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int i = wn * 16 + hf * 8 + t2;
      const float2 eg = *reinterpret_cast<const float2*>(vec + kVecEG + i);
      const float2 be = *reinterpret_cast<const float2*>(vec + kVecBeta + i);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          const int r = m0 + mt * 16 + g + rr * 8;
          const float v0 = to_f(vs[i * C::LDV + r]), v1 = to_f(vs[(i + 1) * C::LDV + r]);
          P::template put2<PL>(rop, r, i, be.x * (v0 - eg.x * ar[mt][hf][2 * rr]),
                               be.y * (v1 - eg.y * ar[mt][hf][2 * rr + 1]));
          ao[mt][hf][2 * rr] *= a.s.scale * eg.x;
          ao[mt][hf][2 * rr + 1] *= a.s.scale * eg.y;
        }
    }
    __syncthreads();
    // U = T R
    float au[MT][2][4] = {};
#pragma unroll
    for (int k0 = 0; k0 < kC; k0 += P::KS) {
      if (k0 >= wn * 16 + 16) break;
      typename P::template B<PL> bt;
      P::load_bn(bt, mt_, wn * 16, k0, lane);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        typename P::template A<PL> fa;
        P::load_a(fa, rop, m0 + mt * 16, k0, lane);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) P::mma(au[mt][hf], fa, bt, hf);
      }
    }
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int i = wn * 16 + hf * 8 + t2;
      const float2 el = *reinterpret_cast<const float2*>(vec + kVecEGL + i);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          const int r = m0 + mt * 16 + g + rr * 8;
          const float u0 = au[mt][hf][2 * rr], u1 = au[mt][hf][2 * rr + 1];
          P::template put2<1>(uop, r, i, u0, u1);
          P::template put2<PL>(ukop, r, i, el.x * u0, el.y * u1);
        }
    }
    __syncthreads();
    if (a.save)
      store_tile<E, C::DVT, kC, C::THREADS>(
          reinterpret_cast<E*>(a.u) + (((slot0 + c) * a.s.hv + h) * dv + dv0) * kC, kC, uop_p, C::LDT, dvn, kC, tid);
    // O += P U
#pragma unroll
    for (int k0 = 0; k0 < kC; k0 += P::KS) {
      if (k0 >= wn * 16 + 16) break;
      typename P::template B<1> bp;
      P::load_bn(bp, mp, wn * 16, k0, lane);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        typename P::template A<1> fa;
        P::load_a(fa, uop, m0 + mt * 16, k0, lane);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) P::mma(ao[mt][hf], fa, bp, hf);
      }
    }
#pragma unroll
    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          put(ost + (wn * 16 + hf * 8 + t2 + (e & 1)) * C::LDV + m0 + mt * 16 + g + (e >> 1) * 8, ao[mt][hf][e]);
    // S1 = exp(G_C) S0 + sum_i exp(G_C - G_i) U_i k_i^T
    const float d = vec[kVecD];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NTS; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[mt][nt][e] *= d;
#pragma unroll
    for (int k0 = 0; k0 < kC; k0 += P::KS) {
      typename P::template A<PL> fa[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) P::load_a(fa[mt], ukop, m0 + mt * 16, k0, lane);
#pragma unroll
      for (int j = 0; j < NTS / 2; ++j) {
        typename P::template B<1> bk;
        P::load_bk(bk, mk, wn * (DK / 4) + j * 16, k0, lane);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) P::mma(s[mt][2 * j + hf], fa[mt], bk, hf);
      }
    }
    if (ST == 1 || C::ALIAS) __syncthreads();
    if (ST == 1 && c + 1 < nc) fetch(c + 1, 0);
    (void)rows;
  }
  if (nc > 0) {
    __syncthreads();
    store_tile<E, kC, C::DVT, C::THREADS>(o + (long long)(nc - 1) * kC * ldo, ldo, ost, C::LDV, len - (nc - 1) * kC, dvn,
                                          tid);
  }
  if (a.final_state) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NTS; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = m0 + mt * 16 + g + (e >> 1) * 8, col = wn * (DK / 4) + nt * 8 + t2 + (e & 1);
          if (r < dvn && col < dk) a.final_state[(sh * dk + col) * dv + dv0 + r] = s[mt][nt][e];
        }
  }
}

template <class P, int DK, int PL>
static cudaError_t launch_prep(const FwdArgs& a, cudaStream_t st) {
  const long long blocks = slot_count(a.s.rows, a.s.n_seq) * a.s.hv;
  const size_t bytes = sizeof(PrepSmem<P, DK>);
  cudaError_t e = cudaFuncSetAttribute(k_gdr_prep<P, DK, PL>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) return e;
  TraceScope tr("k_gdr_prep", st);
  k_gdr_prep<P, DK, PL><<<(unsigned)blocks, 128, bytes, st>>>(a);
  return cudaGetLastError();
}

template <class P, int DK, int MT, int WM, int PL>
static cudaError_t launch_scan(FwdArgs a, cudaStream_t st) {
  using C = ScanCfg<P, DK, MT, WM, PL>;
  static_assert(C::FITS, "shared memory");
  a.ntile = (a.s.dv + C::DVT - 1) / C::DVT;
  const long long blocks = (long long)a.s.n_seq * a.s.hv * a.ntile;
  cudaError_t e =
      cudaFuncSetAttribute(k_gdr_scan<P, DK, MT, WM, PL>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::BYTES);
  if (e != cudaSuccess) return e;
  TraceScope tr("k_gdr_scan", st);
  k_gdr_scan<P, DK, MT, WM, PL><<<(unsigned)blocks, C::THREADS, C::BYTES, st>>>(a);
  return cudaGetLastError();
}

template <class P, int DK, int PL>
static cudaError_t forward(const FwdArgs& a, cudaStream_t st) {
  if (a.s.rows > 0) {
    cudaError_t e = launch_prep<P, DK, PL>(a, st);
    if (e != cudaSuccess) return e;
  }
  // The widest tile of value columns whose blocks still reach every SM.
  const long long heads = (long long)a.s.n_seq * a.s.hv;
  auto blocks = [&](int w) { return heads * ((a.s.dv + w - 1) / w); };
  if constexpr (P::kMode == CFC_MATH_BF16) {
    if constexpr (PL == 1)
      if (a.s.dv > 64 && blocks(128) >= 114) return launch_scan<P, DK, 2, 4, PL>(a, st);
    if (a.s.dv > 32 && blocks(64) >= 114) return launch_scan<P, DK, 2, 2, PL>(a, st);
  }
  if (a.s.dv > 16 && blocks(32) >= 114) return launch_scan<P, DK, 1, 2, PL>(a, st);
  return launch_scan<P, DK, 1, 1, PL>(a, st);
}

static size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

Workspace plan(long long rows, int n_seq, int hk, int hv, int dk, int dv, int math, int save) {
  Workspace w{};
  const size_t e = math == CFC_MATH_BF16 ? 2 : 4;
  const size_t slots = (size_t)slot_count(rows, n_seq) * hv;
  size_t off = 0;
  auto take = [&](size_t* at, size_t bytes) { *at = off; off = up256(off + bytes); };
  take(&w.off_t, slots * 2 * kC * kC * e);
  take(&w.off_p, slots * kC * kC * e);
  take(&w.off_vec, slots * kVec * 4);
  if (save) {
    take(&w.off_s0, slots * dk * dv * e);
    take(&w.off_u, slots * kC * dv * e);
    take(&w.off_ds, slots * dk * dv * e);
    take(&w.off_dr, slots * kC * dv * e);
    if (hv != hk) {
      take(&w.off_dq, (size_t)rows * hv * dk * 4);
      take(&w.off_dk, (size_t)rows * hv * dk * 4);
    }
  }
  w.total = off ? off : 256;
  return w;
}

}  // namespace gdr

bool gdr_shape_supported(int hk, int hv, int dk, int dv, int math) {
  return hk >= 1 && hv >= hk && hv % hk == 0 && hv <= 4096 && dk >= 8 && dk <= gdr::kMaxDk && dk % 8 == 0 && dv >= 8 &&
         dv <= gdr::kMaxDv && dv % 8 == 0 && (math == CFC_MATH_FP32 || math == CFC_MATH_BF16);
}

size_t gdr_workspace(long long rows, int n_seq, int hk, int hv, int dk, int dv, int math, int save) {
  return gdr::plan(rows, n_seq, hk, hv, dk, dv, math, save).total;
}

cudaError_t launch_gdr_forward(const GdrArgs& g, cudaStream_t st) {
  using namespace gdr;
  const Workspace w = plan(g.rows, g.n_seq, g.hk, g.hv, g.dk, g.dv, g.math, g.save);
  FwdArgs a{};
  a.s = Shape{g.off, g.n_seq, g.rows, g.hk, g.hv, g.dk, g.dv, g.scale};
  a.q = g.q; a.k = g.k; a.v = g.v;
  a.ldq = g.ldq; a.ldk = g.ldk; a.ldv = g.ldv;
  a.g = g.g; a.beta = g.beta; a.init = g.init; a.final_state = g.final_state; a.o = g.o;
  a.t = g.ws + w.off_t; a.p = g.ws + w.off_p;
  a.vec = reinterpret_cast<float*>(g.ws + w.off_vec);
  a.save = g.save;
  if (g.save) { a.s0 = g.ws + w.off_s0; a.u = g.ws + w.off_u; }
  if (g.math == CFC_MATH_BF16) {
    // A state that leaves the call is fp32: its chain keeps two planes.
    if (g.final_state)
      return g.dk <= 64 ? forward<MBf16, 64, 2>(a, st) : forward<MBf16, 128, 2>(a, st);
    return g.dk <= 64 ? forward<MBf16, 64, 1>(a, st) : forward<MBf16, 128, 1>(a, st);
  }
  return g.dk <= 64 ? forward<MFp32, 64, 1>(a, st) : forward<MFp32, 128, 1>(a, st);
}

}  // namespace cfc
