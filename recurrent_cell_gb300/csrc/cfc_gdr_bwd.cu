// cfc_gdr_bwd.cu -- backward of the gated delta rule over whole sequences
// (notation of gdr_common.cuh; the forward left T, P, the decays, S0 and U of
// every chunk in the workspace).
//
// With dO the gradient of the outputs and dS1 that of the state after a chunk,
//   dU_j  = exp(G_C - G_j) dS1^T k_j + sum_{i>=j} P_ij dO_i
//   dR    = T^T dU                      (U = T R)
//   dv_i  = beta_i dR_i
//   dS0   = exp(G_C) dS1 + sum_i scale exp(G_i) q_i dO_i^T - beta_i exp(G_i) k_i dR_i^T
// and, since dT = dU R^T and T^T dU R^T T^T = dR U^T,  dA_ij = -dR_i.U_j (j < i).
// With L_ij = exp(G_i - G_j), X = dR S0^T, dP_ij = scale L_ij dO_i.U_j (j <= i):
//   dq_i  = scale exp(G_i) S0 dO_i + sum_{j<=i} dP_ij k_j
//   E_i   = -exp(G_i) X_i + sum_{j<i} L_ij dA_ij k_j
//   dk_i  = beta_i E_i + exp(G_C - G_i) dS1 U_i + sum_{j>=i} dP_ji q_j + beta_j L_ji dA_ji k_j
//   dbeta_i = dR_i.v_i + k_i.E_i
// G enters through exp(G_i) of every row, exp(-G_j) of every column and
// exp(G_C).  The row and column sums of dP o P and of dA o A are dot products
// of the parts of dq and dk just formed, which leaves
//   dG_i  = q_i.dq_i - k_i.dk_i + 2 beta_i k_i.E_i  (+ for the last row:
//           sum_j exp(G_C - G_j) k_j.dS1 U_j + exp(G_C) <S0, dS1>),
//   dg_t  = sum_{i>=t} dG_i.
//
//   k_gdr_scan_bwd  the serial pass, last chunk first: dR, dv, dS1 of each chunk
//   k_gdr_grad      one block per (chunk, value head): dq, dk, dg, dbeta
//   k_gdr_heads     sums dq, dk over the value heads that share a key head
#include "gdr_common.cuh"

namespace cfc {
namespace gdr {

// -------------------------------------------------------------- serial pass
// The forward scan's split of warps: dS^T in registers, 16 MT value columns by
// a quarter of the key width a warp.
template <class P, int DK, int MT, int WM>
struct BwdCfg {
  using E = typename P::E;
  static constexpr int DVT = 16 * MT * WM, THREADS = 128 * WM;
  static constexpr int LDK = DK + P::PAD, LDT = kC + P::PAD, LDV = DVT + P::PAD;
  static constexpr int NTS = DK / 32, ST = P::STAGES;
  static constexpr int kQ = kC * LDK, kT = kC * LDT, kV = kC * LDV;
  static constexpr int STAGE = 2 * kQ + 2 * kT + kV;
  static constexpr int SOP = DVT * LDK, ROP = DVT * LDT;
  // dS operand, dU operand, scaled dO, dR, -beta exp(G) dR; the two dR matrices
  // lie over the dS operand where shared memory is short.  dv is staged over
  // the chunk's dO, which has been read by then.
  static constexpr bool ALIAS = (size_t)(ST * STAGE + SOP + 4 * ROP) * sizeof(E) + 2 * kVec * 4 > 227u * 1024u;
  static constexpr int ELEMS = ST * STAGE + (ALIAS ? (SOP > 2 * ROP ? SOP : 2 * ROP) : SOP + 2 * ROP) + 2 * ROP;
  static constexpr size_t BYTES = (size_t)ELEMS * sizeof(E) + (size_t)ST * kVec * 4;
  static constexpr bool FITS = BYTES <= 227u * 1024u;
};

template <class P, int DK, int MT, int WM>
__global__ void __launch_bounds__(128 * WM) k_gdr_scan_bwd(BwdArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  using C = BwdCfg<P, DK, MT, WM>;
  using E = typename P::E;
  constexpr int NTS = C::NTS, ST = C::ST;
  float* vecs = reinterpret_cast<float*>(smem_raw);
  E* stage = reinterpret_cast<E*>(vecs + ST * kVec);
  E* sop_p = stage + ST * C::STAGE;
  E* dr_p = C::ALIAS ? sop_p : sop_p + C::SOP;
  E* drk_p = dr_p + C::ROP;
  E* uop_p = sop_p + (C::ELEMS - ST * C::STAGE - 2 * C::ROP);
  E* dop_p = uop_p + C::ROP;
  const Mat<E> sop{sop_p, C::LDK, 0}, uop{uop_p, C::LDT, 0}, dop{dop_p, C::LDT, 0}, drk{drk_p, C::LDT, 0};

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
  const long long ldo = (long long)a.s.hv * dv;
  const E* q = static_cast<const E*>(a.q) + start * a.ldq + (long long)hq * dk;
  const E* k = static_cast<const E*>(a.k) + start * a.ldk + (long long)hq * dk;
  const E* go = static_cast<const E*>(a.go) + (start * a.s.hv + h) * dv + dv0;
  E* gv = static_cast<E*>(a.gv) + (start * a.s.hv + h) * dv + dv0;

  auto fetch = [&](int c, int st) {
    E* b = stage + st * C::STAGE;
    const int rows = min(kC, len - c * kC);
    const long long r0 = (long long)c * kC, id = (slot0 + c) * a.s.hv + h;
    load_tile<E, kC, DK, C::THREADS>(b, C::LDK, k + r0 * a.ldk, a.ldk, rows, dk, tid);
    load_tile<E, kC, DK, C::THREADS>(b + C::kQ, C::LDK, q + r0 * a.ldq, a.ldq, rows, dk, tid);
    load_tile<E, kC, kC, C::THREADS>(b + 2 * C::kQ, C::LDT,
                                     reinterpret_cast<const E*>(a.t) + id * (kTPlanes<P> * kC * C::LDT), C::LDT, kC, kC,
                                     tid);
    load_tile<E, kC, kC, C::THREADS>(b + 2 * C::kQ + C::kT, C::LDT, reinterpret_cast<const E*>(a.p) + id * (kTPlanes<P> * kC * C::LDT),
                                     C::LDT, kC, kC, tid);
    load_tile<E, kC, C::DVT, C::THREADS>(b + 2 * C::kQ + 2 * C::kT, C::LDV, go + r0 * ldo, ldo, rows, dvn, tid);
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
        s[mt][nt][e] = a.gfinal && r < dvn && col < dk ? a.gfinal[(sh * dk + col) * dv + dv0 + r] : 0.f;
      }

  if (nc > 0) fetch(nc - 1, (nc - 1) & (ST - 1));
  for (int c = nc - 1; c >= 0; --c) {
    const int st = c & (ST - 1);
    E* b = stage + st * C::STAGE;
    const Mat<E> mk{b, C::LDK, 0}, mq{b + C::kQ, C::LDK, 0}, mt_{b + 2 * C::kQ, C::LDT, 0},
        mp{b + 2 * C::kQ + C::kT, C::LDT, 0}, mo{b + 2 * C::kQ + 2 * C::kT, C::LDV, 0};
    const float* vec = vecs + st * kVec;
    const long long id = (slot0 + c) * a.s.hv + h;
    cp_wait<0>();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NTS; ++nt)
#pragma unroll
        for (int rr = 0; rr < 2; ++rr)
          P::template put2<1>(sop, m0 + mt * 16 + g + rr * 8, wn * (DK / 4) + nt * 8 + t2, s[mt][nt][2 * rr],
                              s[mt][nt][2 * rr + 1]);
    __syncthreads();
    if (ST == 2 && c > 0) fetch(c - 1, (c - 1) & 1);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NTS; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = m0 + mt * 16 + g + (e >> 1) * 8, col = wn * (DK / 4) + nt * 8 + t2 + (e & 1);
          if (r < dvn && col < dk) put(reinterpret_cast<E*>(a.ds) + (id * dk + col) * dv + dv0 + r, s[mt][nt][e]);
        }
    // dU of this warp's 16 tokens
    float ak[MT][2][4] = {}, ap[MT][2][4] = {}, ar[MT][2][4];
#pragma unroll
    for (int k0 = 0; k0 < DK; k0 += P::KS) {
      typename P::template B<1> bk;
      P::load_bn(bk, mk, wn * 16, k0, lane);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        typename P::template A<1> fa;
        P::load_a(fa, sop, m0 + mt * 16, k0, lane);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) P::mma(ak[mt][hf], fa, bk, hf);
      }
    }
#pragma unroll
    for (int k0 = 0; k0 < kC; k0 += P::KS) {
      if (k0 + P::KS <= wn * 16) continue;
      typename P::template B<1> bp;
      P::load_bk(bp, mp, wn * 16, k0, lane);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        typename P::template A<1> fa;
        P::load_at(fa, mo, m0 + mt * 16, k0, lane);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) P::mma(ap[mt][hf], fa, bp, hf);
      }
    }
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int i = wn * 16 + hf * 8 + t2;
      const float2 eg = *reinterpret_cast<const float2*>(vec + kVecEG + i);
      const float2 el = *reinterpret_cast<const float2*>(vec + kVecEGL + i);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          const int r = m0 + mt * 16 + g + rr * 8;
          // dR = dU + (T - I)^T dU: dU itself stays fp32
          ar[mt][hf][2 * rr] = el.x * ak[mt][hf][2 * rr] + ap[mt][hf][2 * rr];
          ar[mt][hf][2 * rr + 1] = el.y * ak[mt][hf][2 * rr + 1] + ap[mt][hf][2 * rr + 1];
          P::template put2<1>(uop, r, i, ar[mt][hf][2 * rr], ar[mt][hf][2 * rr + 1]);
          P::template put2<1>(dop, r, i, a.s.scale * eg.x * to_f(mo.p[i * C::LDV + r]),
                              a.s.scale * eg.y * to_f(mo.p[(i + 1) * C::LDV + r]));
        }
    }
    __syncthreads();
    E* gst = mo.p;
#pragma unroll
    for (int k0 = 0; k0 < kC; k0 += P::KS) {
      if (k0 + P::KS <= wn * 16) continue;
      typename P::template B<1> bt;
      P::load_bk(bt, mt_, wn * 16, k0, lane);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        typename P::template A<1> fa;
        P::load_a(fa, uop, m0 + mt * 16, k0, lane);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) P::mma(ar[mt][hf], fa, bt, hf);
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
          const float r0 = ar[mt][hf][2 * rr], r1 = ar[mt][hf][2 * rr + 1];
          if (r < dvn) {
            E* p = reinterpret_cast<E*>(a.dr) + (id * kC + i) * dv + dv0 + r;
            put(p, r0);
            put(p + dv, r1);
          }
          P::template put2<1>(drk, r, i, -be.x * eg.x * r0, -be.y * eg.y * r1);
          put(gst + i * C::LDV + r, be.x * r0);
          put(gst + (i + 1) * C::LDV + r, be.y * r1);
        }
    }
    __syncthreads();
    store_tile<E, kC, C::DVT, C::THREADS>(gv + (long long)c * kC * ldo, ldo, gst, C::LDV, len - c * kC, dvn, tid);
    const float d = vec[kVecD];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NTS; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[mt][nt][e] *= d;
#pragma unroll
    for (int k0 = 0; k0 < kC; k0 += P::KS) {
      typename P::template A<1> fd[MT], fr[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        P::load_a(fd[mt], dop, m0 + mt * 16, k0, lane);
        P::load_a(fr[mt], drk, m0 + mt * 16, k0, lane);
      }
#pragma unroll
      for (int j = 0; j < NTS / 2; ++j) {
        typename P::template B<1> bq, bk;
        P::load_bk(bq, mq, wn * (DK / 4) + j * 16, k0, lane);
        P::load_bk(bk, mk, wn * (DK / 4) + j * 16, k0, lane);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            P::mma(s[mt][2 * j + hf], fd[mt], bq, hf);
            P::mma(s[mt][2 * j + hf], fr[mt], bk, hf);
          }
      }
    }
    if (ST == 1 || C::ALIAS) __syncthreads();
    if (ST == 1 && c > 0) fetch(c - 1, 0);
  }
  if (a.ginit) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NTS; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = m0 + mt * 16 + g + (e >> 1) * 8, col = wn * (DK / 4) + nt * 8 + t2 + (e & 1);
          if (r < dvn && col < dk) a.ginit[(sh * dk + col) * dv + dv0 + r] = s[mt][nt][e];
        }
  }
}

// ------------------------------------------------------------- the gradients
template <class P, int DK>
struct GradSmem {
  using E = typename P::E;
  static constexpr int DVS = 32;                       // value columns of a slice
  static constexpr int ST = P::STAGES;
  static constexpr int LDK = DK + P::PAD, LDT = kC + P::PAD, LDV = DVS + P::PAD;
  E k[kC * LDK], q[kC * LDK];
  E go[ST][kC * LDV], v[ST][kC * LDV];
  E u[ST][kC * LDV], dr[ST][kC * LDV];
  E s0[ST][DK * LDV], ds[ST][DK * LDV];
  static constexpr int PL = kTPlanes<P>;
  E dp[PL * kC * LDT], da[PL * kC * LDT], dm[PL * kC * LDT];    // 17 bits in bf16: dg is a difference of large sums
  float vec[kVec];
  float dot[4][2][kC];    // q.dq, k.dk, k.E, k.dS1 U by half of the key width
  float drv[4][kC];
  float sum[8];
  float dg[kC];
};

template <class P, int DK>
__global__ void __launch_bounds__(256) k_gdr_grad(BwdArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  using S = GradSmem<P, DK>;
  using E = typename P::E;
  S& sm = *reinterpret_cast<S*>(smem_raw);
  constexpr int NT = DK / 16;           // 8-column tiles of half the key width
  constexpr int DVS = S::DVS, ST = S::ST;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wr = warp & 3, wc = warp >> 2;
  const int g = lane >> 2, t2 = (lane & 3) * 2;
  const int h = blockIdx.x % a.s.hv;
  const long long slot = blockIdx.x / a.s.hv;
  int n, len, c;
  long long start;
  if (!slot_chunk(a.s, slot, &n, &start, &len, &c)) return;
  const long long row0 = start + (long long)c * kC;
  const int rows = min(kC, len - c * kC);
  const int hq = h / (a.s.hv / a.s.hk);
  const int dk = a.s.dk, dv = a.s.dv;
  const long long id = slot * a.s.hv + h;
  const long long ldo = (long long)a.s.hv * dv;
  const E* go = static_cast<const E*>(a.go) + row0 * ldo + (long long)h * dv;
  const E* v = static_cast<const E*>(a.v) + row0 * a.ldv + (long long)h * dv;

  auto fetch = [&](int x, int st) {
    const int v0 = x * DVS, vn = min(DVS, dv - v0);
    load_tile<E, kC, DVS, 256>(sm.go[st], S::LDV, go + v0, ldo, rows, vn, tid);
    load_tile<E, kC, DVS, 256>(sm.v[st], S::LDV, v + v0, a.ldv, rows, vn, tid);
    load_tile<E, kC, DVS, 256>(sm.u[st], S::LDV, reinterpret_cast<const E*>(a.u) + id * kC * dv + v0, dv, kC, vn, tid);
    load_tile<E, kC, DVS, 256>(sm.dr[st], S::LDV, reinterpret_cast<const E*>(a.dr) + id * kC * dv + v0, dv, kC, vn, tid);
    load_tile<E, DK, DVS, 256>(sm.s0[st], S::LDV, reinterpret_cast<const E*>(a.s0) + id * dk * dv + v0, dv, dk, vn, tid);
    load_tile<E, DK, DVS, 256>(sm.ds[st], S::LDV, reinterpret_cast<const E*>(a.ds) + id * dk * dv + v0, dv, dk, vn, tid);
    cp_commit();
  };
  load_tile<E, kC, DK, 256>(sm.k, S::LDK, static_cast<const E*>(a.k) + row0 * a.ldk + (long long)hq * dk, a.ldk, rows,
                            dk, tid);
  load_tile<E, kC, DK, 256>(sm.q, S::LDK, static_cast<const E*>(a.q) + row0 * a.ldq + (long long)hq * dk, a.ldq, rows,
                            dk, tid);
  for (int i = tid; i < kVec / 4; i += 256) cp16(sm.vec + i * 4, a.vec + id * kVec + i * 4, true);
  fetch(0, 0);

  float aq[NT][4] = {}, ax[NT][4] = {}, au[NT][4] = {};   // S0 dO, X, dS1 U
  float ap[4][4] = {}, aa[4][4] = {};                     // dO.U, dR.U over 32 columns
  float drv = 0.f, ss = 0.f;
  const int ns = (dv + DVS - 1) / DVS;
  for (int x = 0; x < ns; ++x) {
    const int st = x & (ST - 1);
    cp_wait<0>();
    __syncthreads();
    if (ST == 2 && x + 1 < ns) fetch(x + 1, (x + 1) & 1);
    const Mat<E> mo{sm.go[st], S::LDV, 0}, mu{sm.u[st], S::LDV, 0}, mr{sm.dr[st], S::LDV, 0}, ms{sm.s0[st], S::LDV, 0},
        md{sm.ds[st], S::LDV, 0};
#pragma unroll
    for (int k0 = 0; k0 < DVS; k0 += P::KS) {
      typename P::template A<1> fo, fr, fu;
      P::load_a(fo, mo, wr * 16, k0, lane);
      P::load_a(fr, mr, wr * 16, k0, lane);
      P::load_a(fu, mu, wr * 16, k0, lane);
#pragma unroll
      for (int j = 0; j < NT / 2; ++j) {
        typename P::template B<1> bs, bd;
        P::load_bn(bs, ms, wc * (DK / 2) + j * 16, k0, lane);
        P::load_bn(bd, md, wc * (DK / 2) + j * 16, k0, lane);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          P::mma(aq[2 * j + hf], fo, bs, hf);
          P::mma(ax[2 * j + hf], fr, bs, hf);
          P::mma(au[2 * j + hf], fu, bd, hf);
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (wc * 32 + j * 16 > wr * 16) continue;        // above the diagonal
        typename P::template B<1> bu;
        P::load_bn(bu, mu, wc * 32 + j * 16, k0, lane);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          P::mma(ap[2 * j + hf], fo, bu, hf);
          P::mma(aa[2 * j + hf], fr, bu, hf);
        }
      }
    }
    {
      const int i = tid & 63, part = tid >> 6;
#pragma unroll
      for (int e = 0; e < DVS / 4; ++e)
        drv = fmaf(to_f(sm.dr[st][i * S::LDV + part * (DVS / 4) + e]),
                   to_f(sm.v[st][i * S::LDV + part * (DVS / 4) + e]), drv);
      for (int e = tid; e < DVS * DK / 2; e += 256) {
        const int r = e / (DVS / 2), cc = (e % (DVS / 2)) * 2;
        const float2 x0 = P::get2(sm.s0[st] + r * S::LDV + cc), x1 = P::get2(sm.ds[st] + r * S::LDV + cc);
        ss = fmaf(x0.x, x1.x, fmaf(x0.y, x1.y, ss));
      }
    }
    if (ST == 1) {
      __syncthreads();
      if (x + 1 < ns) fetch(x + 1, 0);
    }
  }

  const float* vec = sm.vec;
  const int i0 = wr * 16 + g;
  // dP and the two forms of dA as operands
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      const int i = i0 + rr * 8, col = wc * 32 + j * 8 + t2;
      float dp[2], da[2];
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const float2 gi = reinterpret_cast<const float2*>(vec + kVecG2)[i],
                     gj = reinterpret_cast<const float2*>(vec + kVecG2)[col + cc];
        const float l = P::exp2((gi.x - gj.x) + (gi.y - gj.y));
        dp[cc] = col + cc <= i ? a.s.scale * l * ap[j][2 * rr + cc] : 0.f;
        da[cc] = col + cc < i ? -l * aa[j][2 * rr + cc] : 0.f;
      }
      const float be = vec[kVecBeta + i];
      P::template put2<S::PL>(Mat<E>{sm.dp, S::LDT, kC * S::LDT}, i, col, dp[0], dp[1]);
      P::template put2<S::PL>(Mat<E>{sm.da, S::LDT, kC * S::LDT}, i, col, da[0], da[1]);
      P::template put2<S::PL>(Mat<E>{sm.dm, S::LDT, kC * S::LDT}, i, col, be * da[0], be * da[1]);
    }
  float dus[2] = {0.f, 0.f};
#pragma unroll
  for (int rr = 0; rr < 2; ++rr) {
    const int i = i0 + rr * 8;
    const float eg = vec[kVecEG + i], el = vec[kVecEGL + i];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const float2 kk = P::get2(sm.k + i * S::LDK + wc * (DK / 2) + j * 8 + t2);
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        aq[j][2 * rr + cc] *= a.s.scale * eg;
        ax[j][2 * rr + cc] *= -eg;
        au[j][2 * rr + cc] *= el;
        dus[rr] = fmaf(cc ? kk.y : kk.x, au[j][2 * rr + cc], dus[rr]);
      }
    }
  }
  __syncthreads();
  {
    const Mat<E> mk{sm.k, S::LDK, 0}, mq{sm.q, S::LDK, 0}, mp{sm.dp, S::LDT, kC * S::LDT},
        ma{sm.da, S::LDT, kC * S::LDT}, mm{sm.dm, S::LDT, kC * S::LDT};
#pragma unroll
    for (int k0 = 0; k0 < kC; k0 += P::KS) {
      if (k0 < wr * 16 + 16) {
        typename P::template A<S::PL> fp, fa;
        P::load_a(fp, mp, wr * 16, k0, lane);
        P::load_a(fa, ma, wr * 16, k0, lane);
#pragma unroll
        for (int j = 0; j < NT / 2; ++j) {
          typename P::template B<1> bk;
          P::load_bk(bk, mk, wc * (DK / 2) + j * 16, k0, lane);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            P::mma(aq[2 * j + hf], fp, bk, hf);
            P::mma(ax[2 * j + hf], fa, bk, hf);
          }
        }
      }
      if (k0 + P::KS > wr * 16) {
        typename P::template A<S::PL> fp, fm;
        P::load_at(fp, mp, wr * 16, k0, lane);
        P::load_at(fm, mm, wr * 16, k0, lane);
#pragma unroll
        for (int j = 0; j < NT / 2; ++j) {
          typename P::template B<1> bq, bk;
          P::load_bk(bq, mq, wc * (DK / 2) + j * 16, k0, lane);
          P::load_bk(bk, mk, wc * (DK / 2) + j * 16, k0, lane);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            P::mma(au[2 * j + hf], fp, bq, hf);
            P::mma(au[2 * j + hf], fm, bk, hf);
          }
        }
      }
    }
  }
  // row dots, dk, stores
#pragma unroll
  for (int rr = 0; rr < 2; ++rr) {
    const int i = i0 + rr * 8;
    const float be = vec[kVecBeta + i];
    float dq_ = 0.f, dk_ = 0.f, de_ = 0.f;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int col = wc * (DK / 2) + j * 8 + t2;
      const float2 kk = P::get2(sm.k + i * S::LDK + col), qq = P::get2(sm.q + i * S::LDK + col);
      const float q0 = aq[j][2 * rr], q1 = aq[j][2 * rr + 1], e0 = ax[j][2 * rr], e1 = ax[j][2 * rr + 1];
      const float k0 = fmaf(be, e0, au[j][2 * rr]), k1 = fmaf(be, e1, au[j][2 * rr + 1]);
      dq_ = fmaf(qq.x, q0, fmaf(qq.y, q1, dq_));
      dk_ = fmaf(kk.x, k0, fmaf(kk.y, k1, dk_));
      de_ = fmaf(kk.x, e0, fmaf(kk.y, e1, de_));
      if (i < rows && col < dk) {
        if (a.pdq) {
          const long long at = ((row0 + i) * a.s.hv + h) * dk + col;
          *reinterpret_cast<float2*>(a.pdq + at) = make_float2(q0, q1);
          *reinterpret_cast<float2*>(a.pdk + at) = make_float2(k0, k1);
        } else {
          const long long at = ((row0 + i) * a.s.hk + h) * dk + col;
          P::template put2<1>(Mat<E>{static_cast<E*>(a.gq) + at, 0, 0}, 0, 0, q0, q1);
          P::template put2<1>(Mat<E>{static_cast<E*>(a.gk) + at, 0, 0}, 0, 0, k0, k1);
        }
      }
    }
    float d[4] = {dq_, dk_, de_, dus[rr]};
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      d[m] += __shfl_xor_sync(0xffffffffu, d[m], 1);
      d[m] += __shfl_xor_sync(0xffffffffu, d[m], 2);
      if ((lane & 3) == 0) sm.dot[m][wc][i] = d[m];
    }
  }
  sm.drv[tid >> 6][tid & 63] = drv;
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
  if (lane == 0) sm.sum[warp] = ss;
  __syncthreads();
  if (tid < kC) {
    const int i = tid;
    const float be = vec[kVecBeta + i];
    const float z = sm.dot[2][0][i] + sm.dot[2][1][i];
    const float db = ((sm.drv[0][i] + sm.drv[1][i]) + (sm.drv[2][i] + sm.drv[3][i])) + z;
    sm.dg[i] = (sm.dot[0][0][i] + sm.dot[0][1][i]) - (sm.dot[1][0][i] + sm.dot[1][1][i]) + 2.f * be * z;
    if (i < rows) put(static_cast<E*>(a.gbeta) + (row0 + i) * a.s.hv + h, db);
  }
  __syncthreads();
  if (warp == 0) {
    // dg: the sums from each row to the chunk's end
    float us = (sm.dot[3][0][lane] + sm.dot[3][1][lane]) + (sm.dot[3][0][lane + 32] + sm.dot[3][1][lane + 32]);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) us += __shfl_xor_sync(0xffffffffu, us, m);
    float st_sum = 0.f;
#pragma unroll
    for (int m = 0; m < 8; ++m) st_sum += sm.sum[m];
    const float last = fmaf(vec[kVecD], st_sum, us);
    const float x0 = sm.dg[2 * lane], x1 = sm.dg[2 * lane + 1];
    float run = x0 + x1;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const float y = __shfl_down_sync(0xffffffffu, run, d);
      run += lane + d < 32 ? y : 0.f;
    }
    const float d0 = run + last, d1 = run - x0 + last;
    if (2 * lane < rows) put(static_cast<E*>(a.gg) + (row0 + 2 * lane) * a.s.hv + h, d0);
    if (2 * lane + 1 < rows) put(static_cast<E*>(a.gg) + (row0 + 2 * lane + 1) * a.s.hv + h, d1);
  }
}

// dq, dk of a key head: its value heads' parts, first to last.
template <class E>
__global__ void k_gdr_heads(const float* pdq, const float* pdk, E* gq, E* gk, long long rows, int hk, int group, int dk) {
  const long long total = rows * hk * (dk / 2);
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total;
       i += (long long)gridDim.x * blockDim.x) {
    const long long rh = i / (dk / 2);
    const int c = (int)(i % (dk / 2)) * 2;
    float2 x = make_float2(0.f, 0.f), y = x;
    for (int j = 0; j < group; ++j) {
      const long long at = (rh * group + j) * dk + c;
      const float2 u = *reinterpret_cast<const float2*>(pdq + at), w = *reinterpret_cast<const float2*>(pdk + at);
      x.x += u.x; x.y += u.y;
      y.x += w.x; y.y += w.y;
    }
    put(gq + rh * dk + c, x.x);
    put(gq + rh * dk + c + 1, x.y);
    put(gk + rh * dk + c, y.x);
    put(gk + rh * dk + c + 1, y.y);
  }
}

template <class P, int DK, int MT, int WM>
static cudaError_t launch_scan_bwd(BwdArgs a, cudaStream_t st) {
  using C = BwdCfg<P, DK, MT, WM>;
  static_assert(C::FITS, "shared memory");
  a.ntile = (a.s.dv + C::DVT - 1) / C::DVT;
  const long long blocks = (long long)a.s.n_seq * a.s.hv * a.ntile;
  cudaError_t e =
      cudaFuncSetAttribute(k_gdr_scan_bwd<P, DK, MT, WM>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::BYTES);
  if (e != cudaSuccess) return e;
  TraceScope tr("k_gdr_scan_bwd", st);
  k_gdr_scan_bwd<P, DK, MT, WM><<<(unsigned)blocks, C::THREADS, C::BYTES, st>>>(a);
  return cudaGetLastError();
}

template <class P, int DK>
static cudaError_t backward(const BwdArgs& a, cudaStream_t st) {
  using E = typename P::E;
  cudaError_t e;
  if constexpr (P::kMode == CFC_MATH_BF16) {
    e = launch_scan_bwd_tc(a, DK, st);
    return e != cudaSuccess || a.s.rows == 0 ? e : launch_grad_tc(a, DK, st);
  } else {
    const long long heads = (long long)a.s.n_seq * a.s.hv;
    if (a.s.dv > 16 && heads * ((a.s.dv + 31) / 32) >= 114) e = launch_scan_bwd<P, DK, 1, 2>(a, st);
    else e = launch_scan_bwd<P, DK, 1, 1>(a, st);
  }
  if (e != cudaSuccess || a.s.rows == 0) return e;
  const size_t bytes = sizeof(GradSmem<P, DK>);
  static_assert(sizeof(GradSmem<P, DK>) <= 227u * 1024u, "shared memory");
  e = cudaFuncSetAttribute(k_gdr_grad<P, DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) return e;
  {
    TraceScope tr("k_gdr_grad", st);
    k_gdr_grad<P, DK><<<(unsigned)(slot_count(a.s.rows, a.s.n_seq) * a.s.hv), 256, bytes, st>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || !a.pdq) return e;
  TraceScope tr("k_gdr_heads", st);
  const long long work = (a.s.rows * a.s.hk * (a.s.dk / 2) + 255) / 256;
  k_gdr_heads<E><<<(unsigned)(work < 16 * kNumSMs ? work : 16 * kNumSMs), 256, 0, st>>>(
      a.pdq, a.pdk, static_cast<E*>(a.gq), static_cast<E*>(a.gk), a.s.rows, a.s.hk, a.s.hv / a.s.hk, a.s.dk);
  return cudaGetLastError();
}

}  // namespace gdr

cudaError_t launch_gdr_backward(const GdrArgs& g, const GdrGrads& r, cudaStream_t st) {
  using namespace gdr;
  const Workspace w = plan(g.rows, g.n_seq, g.hk, g.hv, g.dk, g.dv, g.math, 1);
  BwdArgs a{};
  a.s = Shape{g.off, g.n_seq, g.rows, g.hk, g.hv, g.dk, g.dv, g.scale, (int)(g.rows / g.n_seq)};
  a.q = g.q; a.k = g.k; a.v = g.v; a.go = r.grad_o;
  a.ldq = g.ldq; a.ldk = g.ldk; a.ldv = g.ldv;
  a.gfinal = r.grad_final; a.ginit = r.grad_init;
  a.gq = r.grad_q; a.gk = r.grad_k; a.gv = r.grad_v; a.gg = r.grad_g; a.gbeta = r.grad_beta;
  a.t = g.ws + w.off_t; a.p = g.ws + w.off_p; a.s0 = g.ws + w.off_s0; a.u = g.ws + w.off_u;
  a.ds = g.ws + w.off_ds; a.dr = g.ws + w.off_dr;
  a.vec = reinterpret_cast<const float*>(g.ws + w.off_vec);
  if (g.off && g.math == CFC_MATH_BF16 && g.n_seq <= kMaxOrder)
    a.order = reinterpret_cast<const int*>(g.ws + w.off_order);
  if (g.hv != g.hk && g.math == CFC_MATH_FP32) {
    a.pdq = reinterpret_cast<float*>(g.ws + w.off_dq);
    a.pdk = reinterpret_cast<float*>(g.ws + w.off_dk);
  }
  if (g.math == CFC_MATH_BF16) return g.dk <= 64 ? backward<MBf16, 64>(a, st) : backward<MBf16, 128>(a, st);
  return g.dk <= 64 ? backward<MFp32, 64>(a, st) : backward<MFp32, 128>(a, st);
}

}  // namespace cfc
