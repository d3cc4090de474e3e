// cfc_gdr_bwd.cu -- backward of the gated delta rule over whole sequences: its
// formulas, dispatch, and the kernels in FP32 (bf16: cfc_gdr_tc.cu, cfc_gdr_grad.cu)
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
// The forward scan's split of the chain's warps: dS^T in registers, 16 value
// columns by a quarter of the key width a warp.
template <int DK, int WM>
struct BwdCfg {
  static constexpr int DVT = 16 * WM, THREADS = 128 * WM;
  static constexpr int LDK = DK + kPad, LDV = DVT + kPad, NTS = DK / 32;
  static constexpr int kQ = kC * LDK, kT = kC * kLdT, kV = kC * LDV;
  static constexpr int SOP = DVT * LDK, ROP = DVT * kLdT;
  // k, q, T - I, P, dO (then dv), the vectors; the operands dS, dU, scaled dO, -beta exp(G) dR
  static constexpr int ELEMS = 2 * kQ + 2 * kT + kV + kVec + SOP + 3 * ROP;
  static constexpr size_t BYTES = ELEMS * sizeof(float);
  static_assert(BYTES <= 227u * 1024u, "shared memory");
};

template <int DK, int WM>
__global__ void __launch_bounds__(128 * WM) k_gdr_scan_bwd(BwdArgs a) {
  extern __shared__ __align__(16) float smem[];
  using C = BwdCfg<DK, WM>;
  constexpr int NTS = C::NTS;
  const Mat<float> mk{smem, C::LDK}, mq{mk.p + C::kQ, C::LDK}, mt{mq.p + C::kQ, kLdT}, mp{mt.p + C::kT, kLdT},
      mo{mp.p + C::kT, C::LDV};
  float* vec = mo.p + C::kV;
  const Mat<float> sop{vec + kVec, C::LDK}, uop{sop.p + C::SOP, kLdT}, dop{uop.p + C::ROP, kLdT},
      drk{dop.p + C::ROP, kLdT};

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wn = warp & 3, m0 = (warp >> 2) * 16;
  const int g = lane >> 2, t2 = (lane & 3) * 2, i0 = wn * 16 + t2;
  const int tile = blockIdx.x % a.ntile;
  const long long sh = blockIdx.x / a.ntile;
  const int h = (int)(sh % a.s.hv), n = (int)(sh / a.s.hv);
  const int hq = h / (a.s.hv / a.s.hk);
  const int dk = a.s.dk, dv = a.s.dv, dv0 = tile * C::DVT, dvn = min(C::DVT, dv - dv0);
  long long start;
  int len;
  seq_range(a.s, n, &start, &len);
  const int nc = (len + kC - 1) / kC;
  const long long slot0 = slot_base(start, n);
  const long long ldo = (long long)a.s.hv * dv;
  const float* q = static_cast<const float*>(a.q) + start * a.ldq + (long long)hq * dk;
  const float* k = static_cast<const float*>(a.k) + start * a.ldk + (long long)hq * dk;
  const float* go = static_cast<const float*>(a.go) + (start * a.s.hv + h) * dv + dv0;
  float* gv = static_cast<float*>(a.gv) + (start * a.s.hv + h) * dv + dv0;

  auto fetch = [&](int c) {
    const int rows = min(kC, len - c * kC);
    const long long r0 = (long long)c * kC, id = (slot0 + c) * a.s.hv + h;
    load_tile<float, kC, DK, C::THREADS>(mk.p, C::LDK, k + r0 * a.ldk, a.ldk, rows, dk, tid);
    load_tile<float, kC, DK, C::THREADS>(mq.p, C::LDK, q + r0 * a.ldq, a.ldq, rows, dk, tid);
    load_tile<float, kC, kC, C::THREADS>(mt.p, kLdT, reinterpret_cast<const float*>(a.t) + id * C::kT, kLdT, kC, kC, tid);
    load_tile<float, kC, kC, C::THREADS>(mp.p, kLdT, reinterpret_cast<const float*>(a.p) + id * C::kT, kLdT, kC, kC, tid);
    load_tile<float, kC, C::DVT, C::THREADS>(mo.p, C::LDV, go + r0 * ldo, ldo, rows, dvn, tid);
    for (int i = tid; i < kVec / 4; i += C::THREADS) cp16(vec + i * 4, a.vec + id * kVec + i * 4, true);
    cp_commit();
  };
  // dS^T: element e of 8-column tile nt is value column m0 + g + 8 (e / 2), key column:
  auto key = [&](int nt, int e) { return wn * (DK / 4) + nt * 8 + t2 + (e & 1); };
  float s[NTS][4];
#pragma unroll
  for (int nt = 0; nt < NTS; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = m0 + g + (e >> 1) * 8;
      s[nt][e] = a.gfinal && r < dvn && key(nt, e) < dk ? a.gfinal[(sh * dk + key(nt, e)) * dv + dv0 + r] : 0.f;
    }

  if (nc > 0) fetch(nc - 1);
  for (int c = nc - 1; c >= 0; --c) {
    const long long id = (slot0 + c) * a.s.hv + h;
    cp_wait<0>();
    float* ds = reinterpret_cast<float*>(a.ds) + id * dk * dv + dv0;
#pragma unroll
    for (int nt = 0; nt < NTS; ++nt)
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const int r = m0 + g + rr * 8;
        F::put2(sop, r, key(nt, 0), s[nt][2 * rr], s[nt][2 * rr + 1]);
        if (r < dvn && key(nt, 0) < dk) {
          ds[(long long)key(nt, 0) * dv + r] = s[nt][2 * rr];
          ds[(long long)key(nt, 1) * dv + r] = s[nt][2 * rr + 1];
        }
      }
    __syncthreads();
    // dU of this warp's 16 tokens
    float ak[2][4] = {}, ap[2][4] = {}, al[2][4] = {}, ar[2][4], aw[2][4] = {};
#pragma unroll
    for (int k0 = 0; k0 < DK; k0 += F::KS) {
      F::A fa;
      F::B fb;
      F::load_a(fa, sop, m0, k0, lane);
      F::load_bn(fb, mk, wn * 16, k0, lane);
      F::mma(ak[0], al[0], fa, fb, 0);
      F::mma(ak[1], al[1], fa, fb, 1);
    }
#pragma unroll
    for (int k0 = 0; k0 < kC; k0 += F::KS) {
      if (k0 + F::KS <= wn * 16) continue;
      F::A fa;
      F::B fb;
      F::load_at(fa, mo, m0, k0, lane);
      F::load_bk(fb, mp, wn * 16, k0, lane);
      F::mma(ap[0], fa, fb, 0);
      F::mma(ap[1], fa, fb, 1);
    }
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int i = i0 + hf * 8;
      const float2 eg = *reinterpret_cast<const float2*>(vec + kVecEG + i);
      const float2 el = *reinterpret_cast<const float2*>(vec + kVecEGL + i);
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const int r = m0 + g + rr * 8;
        ar[hf][2 * rr] = el.x * (ak[hf][2 * rr] + al[hf][2 * rr]) + ap[hf][2 * rr];
        ar[hf][2 * rr + 1] = el.y * (ak[hf][2 * rr + 1] + al[hf][2 * rr + 1]) + ap[hf][2 * rr + 1];
        F::put2(uop, r, i, ar[hf][2 * rr], ar[hf][2 * rr + 1]);
        F::put2(dop, r, i, a.s.scale * eg.x * mo.p[i * C::LDV + r], a.s.scale * eg.y * mo.p[(i + 1) * C::LDV + r]);
      }
    }
    __syncthreads();
    // dR = dU + (T - I)^T dU
#pragma unroll
    for (int k0 = 0; k0 < kC; k0 += F::KS) {
      if (k0 + F::KS <= wn * 16) continue;
      F::A fa;
      F::B fb;
      F::load_a(fa, uop, m0, k0, lane);
      F::load_bk(fb, mt, wn * 16, k0, lane);
      F::mma(ar[0], aw[0], fa, fb, 0);
      F::mma(ar[1], aw[1], fa, fb, 1);
    }
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int i = i0 + hf * 8;
      const float2 eg = *reinterpret_cast<const float2*>(vec + kVecEG + i);
      const float2 be = *reinterpret_cast<const float2*>(vec + kVecBeta + i);
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const int r = m0 + g + rr * 8;
        const float r0 = ar[hf][2 * rr] + aw[hf][2 * rr], r1 = ar[hf][2 * rr + 1] + aw[hf][2 * rr + 1];
        if (r < dvn) {
          float* p = reinterpret_cast<float*>(a.dr) + (id * kC + i) * dv + dv0 + r;
          p[0] = r0;
          p[dv] = r1;
        }
        F::put2(drk, r, i, -be.x * eg.x * r0, -be.y * eg.y * r1);
        mo.p[i * C::LDV + r] = be.x * r0;              // dv, over dO
        mo.p[(i + 1) * C::LDV + r] = be.y * r1;
      }
    }
    __syncthreads();
    store_tile<float, kC, C::DVT, C::THREADS>(gv + (long long)c * kC * ldo, ldo, mo.p, C::LDV, len - c * kC, dvn, tid);
    // dS0 = exp(G_C) dS1 + sum_i scale exp(G_i) dO_i q_i^T - beta_i exp(G_i) dR_i k_i^T
    const float d = vec[kVecD];
#pragma unroll
    for (int nt = 0; nt < NTS; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] *= d;
#pragma unroll
    for (int k0 = 0; k0 < kC; k0 += F::KS) {
      F::A fd, fr;
      F::load_a(fd, dop, m0, k0, lane);
      F::load_a(fr, drk, m0, k0, lane);
#pragma unroll
      for (int j = 0; j < NTS / 2; ++j) {
        F::B bq, bk;
        F::load_bk(bq, mq, wn * (DK / 4) + j * 16, k0, lane);
        F::load_bk(bk, mk, wn * (DK / 4) + j * 16, k0, lane);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          F::mma(s[2 * j + hf], fd, bq, hf);
          F::mma(s[2 * j + hf], fr, bk, hf);
        }
      }
    }
    __syncthreads();
    if (c > 0) fetch(c - 1);
  }
  if (a.ginit)
#pragma unroll
    for (int nt = 0; nt < NTS; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = m0 + g + (e >> 1) * 8;
        if (r < dvn && key(nt, e) < dk) a.ginit[(sh * dk + key(nt, e)) * dv + dv0 + r] = s[nt][e];
      }
}

// ------------------------------------------------------------- the gradients
template <int DK>
struct GradSmem {
  static constexpr int DVS = 32;                       // value columns of a slice
  static constexpr int LDK = DK + kPad, LDV = DVS + kPad;
  float k[kC * LDK], q[kC * LDK];
  float go[kC * LDV], v[kC * LDV], u[kC * LDV], dr[kC * LDV];
  float s0[DK * LDV], ds[DK * LDV];
  float dp[kC * kLdT], da[kC * kLdT], dm[kC * kLdT];
  float vec[kVec];
  float dot[4][2][kC];    // q.dq, k.dk, k.E, k.dS1 U by half of the key width
  float drv[4][kC];
  float sum[8];
  float dg[kC];
};

template <int DK>
__global__ void __launch_bounds__(256) k_gdr_grad(BwdArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  using S = GradSmem<DK>;
  S& sm = *reinterpret_cast<S*>(smem_raw);
  constexpr int NT = DK / 16;           // 8-column tiles of half the key width
  constexpr int DVS = S::DVS;
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
  const float* go = static_cast<const float*>(a.go) + row0 * ldo + (long long)h * dv;
  const float* v = static_cast<const float*>(a.v) + row0 * a.ldv + (long long)h * dv;

  auto fetch = [&](int x) {
    const int v0 = x * DVS, vn = min(DVS, dv - v0);
    load_tile<float, kC, DVS, 256>(sm.go, S::LDV, go + v0, ldo, rows, vn, tid);
    load_tile<float, kC, DVS, 256>(sm.v, S::LDV, v + v0, a.ldv, rows, vn, tid);
    load_tile<float, kC, DVS, 256>(sm.u, S::LDV, reinterpret_cast<const float*>(a.u) + id * kC * dv + v0, dv, kC, vn, tid);
    load_tile<float, kC, DVS, 256>(sm.dr, S::LDV, reinterpret_cast<const float*>(a.dr) + id * kC * dv + v0, dv, kC, vn, tid);
    load_tile<float, DK, DVS, 256>(sm.s0, S::LDV, reinterpret_cast<const float*>(a.s0) + id * dk * dv + v0, dv, dk, vn, tid);
    load_tile<float, DK, DVS, 256>(sm.ds, S::LDV, reinterpret_cast<const float*>(a.ds) + id * dk * dv + v0, dv, dk, vn, tid);
    cp_commit();
  };
  load_tile<float, kC, DK, 256>(sm.k, S::LDK, static_cast<const float*>(a.k) + row0 * a.ldk + (long long)hq * dk, a.ldk, rows,
                            dk, tid);
  load_tile<float, kC, DK, 256>(sm.q, S::LDK, static_cast<const float*>(a.q) + row0 * a.ldq + (long long)hq * dk, a.ldq, rows,
                            dk, tid);
  for (int i = tid; i < kVec / 4; i += 256) cp16(sm.vec + i * 4, a.vec + id * kVec + i * 4, true);
  fetch(0);

  float aq[NT][4] = {}, ax[NT][4] = {}, au[NT][4] = {};   // S0 dO, X, dS1 U
  float ap[4][4] = {}, aa[4][4] = {};                     // dO.U, dR.U over 32 columns
  float drv = 0.f, ss = 0.f;
  const int ns = (dv + DVS - 1) / DVS;
  for (int x = 0; x < ns; ++x) {
    cp_wait<0>();
    __syncthreads();
    const Mat<float> mo{sm.go, S::LDV}, mu{sm.u, S::LDV}, mr{sm.dr, S::LDV}, ms{sm.s0, S::LDV},
        md{sm.ds, S::LDV};
#pragma unroll
    for (int k0 = 0; k0 < DVS; k0 += F::KS) {
      F::A fo, fr, fu;
      F::load_a(fo, mo, wr * 16, k0, lane);
      F::load_a(fr, mr, wr * 16, k0, lane);
      F::load_a(fu, mu, wr * 16, k0, lane);
#pragma unroll
      for (int j = 0; j < NT / 2; ++j) {
        F::B bs, bd;
        F::load_bn(bs, ms, wc * (DK / 2) + j * 16, k0, lane);
        F::load_bn(bd, md, wc * (DK / 2) + j * 16, k0, lane);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          F::mma(aq[2 * j + hf], fo, bs, hf);
          F::mma(ax[2 * j + hf], fr, bs, hf);
          F::mma(au[2 * j + hf], fu, bd, hf);
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (wc * 32 + j * 16 > wr * 16) continue;        // above the diagonal
        F::B bu;
        F::load_bn(bu, mu, wc * 32 + j * 16, k0, lane);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          F::mma(ap[2 * j + hf], fo, bu, hf);
          F::mma(aa[2 * j + hf], fr, bu, hf);
        }
      }
    }
    {
      const int i = tid & 63, part = tid >> 6;
#pragma unroll
      for (int e = 0; e < DVS / 4; ++e)
        drv = fmaf(sm.dr[i * S::LDV + part * (DVS / 4) + e],
                   sm.v[i * S::LDV + part * (DVS / 4) + e], drv);
      for (int e = tid; e < DVS * DK / 2; e += 256) {
        const int r = e / (DVS / 2), cc = (e % (DVS / 2)) * 2;
        const float2 x0 = *reinterpret_cast<const float2*>(sm.s0 + r * S::LDV + cc), x1 = *reinterpret_cast<const float2*>(sm.ds + r * S::LDV + cc);
        ss = fmaf(x0.x, x1.x, fmaf(x0.y, x1.y, ss));
      }
    }
    __syncthreads();
    if (x + 1 < ns) fetch(x + 1);
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
        const float l = exp2f((gi.x - gj.x) + (gi.y - gj.y));
        dp[cc] = col + cc <= i ? a.s.scale * l * ap[j][2 * rr + cc] : 0.f;
        da[cc] = col + cc < i ? -l * aa[j][2 * rr + cc] : 0.f;
      }
      const float be = vec[kVecBeta + i];
      F::put2(Mat<float>{sm.dp, kLdT}, i, col, dp[0], dp[1]);
      F::put2(Mat<float>{sm.da, kLdT}, i, col, da[0], da[1]);
      F::put2(Mat<float>{sm.dm, kLdT}, i, col, be * da[0], be * da[1]);
    }
  float dus[2] = {0.f, 0.f};
#pragma unroll
  for (int rr = 0; rr < 2; ++rr) {
    const int i = i0 + rr * 8;
    const float eg = vec[kVecEG + i], el = vec[kVecEGL + i];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const float2 kk = *reinterpret_cast<const float2*>(sm.k + i * S::LDK + wc * (DK / 2) + j * 8 + t2);
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
    const Mat<float> mk{sm.k, S::LDK}, mq{sm.q, S::LDK}, mp{sm.dp, kLdT},
        ma{sm.da, kLdT}, mm{sm.dm, kLdT};
#pragma unroll
    for (int k0 = 0; k0 < kC; k0 += F::KS) {
      if (k0 < wr * 16 + 16) {
        F::A fp, fa;
        F::load_a(fp, mp, wr * 16, k0, lane);
        F::load_a(fa, ma, wr * 16, k0, lane);
#pragma unroll
        for (int j = 0; j < NT / 2; ++j) {
          F::B bk;
          F::load_bk(bk, mk, wc * (DK / 2) + j * 16, k0, lane);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            F::mma(aq[2 * j + hf], fp, bk, hf);
            F::mma(ax[2 * j + hf], fa, bk, hf);
          }
        }
      }
      if (k0 + F::KS > wr * 16) {
        F::A fp, fm;
        F::load_at(fp, mp, wr * 16, k0, lane);
        F::load_at(fm, mm, wr * 16, k0, lane);
#pragma unroll
        for (int j = 0; j < NT / 2; ++j) {
          F::B bq, bk;
          F::load_bk(bq, mq, wc * (DK / 2) + j * 16, k0, lane);
          F::load_bk(bk, mk, wc * (DK / 2) + j * 16, k0, lane);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            F::mma(au[2 * j + hf], fp, bq, hf);
            F::mma(au[2 * j + hf], fm, bk, hf);
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
      const float2 kk = *reinterpret_cast<const float2*>(sm.k + i * S::LDK + col);
      const float2 qq = *reinterpret_cast<const float2*>(sm.q + i * S::LDK + col);
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
          *reinterpret_cast<float2*>(static_cast<float*>(a.gq) + at) = make_float2(q0, q1);
          *reinterpret_cast<float2*>(static_cast<float*>(a.gk) + at) = make_float2(k0, k1);
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
    if (i < rows) static_cast<float*>(a.gbeta)[(row0 + i) * a.s.hv + h] = db;
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
    const uint2 dead = *reinterpret_cast<const uint2*>(vec + kVecDead);
    const float d0 = alive(run + last, dead.x, lane), d1 = alive(run - x0 + last, dead.y, lane);
    if (2 * lane < rows) static_cast<float*>(a.gg)[(row0 + 2 * lane) * a.s.hv + h] = d0;
    if (2 * lane + 1 < rows) static_cast<float*>(a.gg)[(row0 + 2 * lane + 1) * a.s.hv + h] = d1;
  }
}

// dq, dk of a key head: its value heads' parts, first to last.
__global__ void k_gdr_heads(const float2* pdq, const float2* pdk, float2* gq, float2* gk, long long rows, int hk,
                            int group, int half) {
  const long long total = rows * hk * half;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total;
       i += (long long)gridDim.x * blockDim.x) {
    const long long rh = i / half;
    const int c = (int)(i % half);
    float2 x = make_float2(0.f, 0.f), y = x;
    for (int j = 0; j < group; ++j) {
      const float2 u = pdq[(rh * group + j) * half + c], w = pdk[(rh * group + j) * half + c];
      x.x += u.x; x.y += u.y;
      y.x += w.x; y.y += w.y;
    }
    gq[i] = x;
    gk[i] = y;
  }
}

template <int DK, int WM>
static cudaError_t scan_bwd(BwdArgs a, cudaStream_t st) {
  using C = BwdCfg<DK, WM>;
  a.ntile = (a.s.dv + C::DVT - 1) / C::DVT;
  cudaError_t e = allow_smem<k_gdr_scan_bwd<DK, WM>>(C::BYTES);
  if (e != cudaSuccess) return e;
  TraceScope tr("k_gdr_scan_bwd", st);
  k_gdr_scan_bwd<DK, WM><<<(unsigned)((long long)a.s.n_seq * a.s.hv * a.ntile), C::THREADS, C::BYTES, st>>>(a);
  return cudaGetLastError();
}

template <int DK>
static cudaError_t backward_fp32(const BwdArgs& a, cudaStream_t st) {
  // as in the forward (84 us, 133)
  cudaError_t e = wide_tiles((long long)a.s.n_seq * a.s.hv, a.s.dv, 16) ? scan_bwd<DK, 2>(a, st) : scan_bwd<DK, 1>(a, st);
  if (e != cudaSuccess || a.s.rows == 0) return e;
  constexpr size_t bytes = sizeof(GradSmem<DK>);
  static_assert(bytes <= 227u * 1024u, "shared memory");
  e = allow_smem<k_gdr_grad<DK>>(bytes);
  if (e != cudaSuccess) return e;
  {
    TraceScope tr("k_gdr_grad", st);
    k_gdr_grad<DK><<<(unsigned)(slot_count(a.s.rows, a.s.n_seq) * a.s.hv), 256, bytes, st>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || !a.pdq) return e;
  TraceScope tr("k_gdr_heads", st);
  const long long work = (a.s.rows * a.s.hk * (a.s.dk / 2) + 255) / 256;
  k_gdr_heads<<<(unsigned)(work < 16 * kNumSMs ? work : 16 * kNumSMs), 256, 0, st>>>(
      reinterpret_cast<const float2*>(a.pdq), reinterpret_cast<const float2*>(a.pdk), static_cast<float2*>(a.gq),
      static_cast<float2*>(a.gk), a.s.rows, a.s.hk, a.s.hv / a.s.hk, a.s.dk / 2);
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
  if (g.off && g.rows > 0 && g.math == CFC_MATH_BF16 && g.n_seq <= kMaxOrder)
    a.order = reinterpret_cast<const int*>(g.ws + w.off_order);
  if (g.hv != g.hk && g.math == CFC_MATH_FP32) {
    a.pdq = reinterpret_cast<float*>(g.ws + w.off_dq);
    a.pdk = reinterpret_cast<float*>(g.ws + w.off_dk);
  }
  const int tile = g.dk <= 64 ? 64 : 128;
  if (g.math == CFC_MATH_FP32) return tile == 64 ? backward_fp32<64>(a, st) : backward_fp32<128>(a, st);
  const cudaError_t e = launch_scan_bwd_tc(a, tile, st);
  return e != cudaSuccess || g.rows == 0 ? e : launch_grad_tc(a, tile, st);
}

}  // namespace cfc
