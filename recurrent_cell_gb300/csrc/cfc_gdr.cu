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

__device__ int g_gdr_error = 0;   // a bounded wait gave up

// ------------------------------------------------------------------- prep
template <class P, int DK>
struct PrepSmem {
  using E = typename P::E;
  static constexpr int LDK = DK + P::PAD;
  static constexpr int LDA = kC + 4;      // fp32 rows of A and T
  static constexpr int LDT = kLdt<P>;
  static constexpr size_t kTile = sizeof(E) * kC * LDK;
  static constexpr size_t kA = sizeof(float) * kC * LDA, kP = kTPlanes<P> * sizeof(E) * kC * LDT;
  // k, then A and T; q, then P: the products are done when the others begin
  static constexpr size_t kOffQ = kTile > kA ? kTile : kA;
  static constexpr size_t kOffG = kOffQ + (kTile > kP ? kTile : kP);
  static constexpr size_t kBytes = kOffG + 3 * kC * sizeof(float);      // G / ln 2 in pairs, beta
};


// T = (I + A)^{-1} of the unit lower triangular I + A: 16 x 16 diagonal blocks
// by forward substitution (one warp each, a column a lane), then pairs of
// blocks joined by T21 = -T22 A21 T11 with fp32-accurate products.  T stays in
// fp32 until it is stored: its entries reach far above A's when keys repeat.
template <class P, int DK, int PL>
__global__ void __launch_bounds__(128, 5) k_gdr_prep(FwdArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  using E = typename P::E;
  using S = PrepSmem<P, DK>;
  E* ks = reinterpret_cast<E*>(smem_raw);
  E* qs = reinterpret_cast<E*>(smem_raw + S::kOffQ);
  float* am = reinterpret_cast<float*>(smem_raw);
  E* ps = qs;
  float2* g2 = reinterpret_cast<float2*>(smem_raw + S::kOffG);
  float* bet = reinterpret_cast<float*>(g2 + kC);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x % a.s.hv;
  const long long slot = blockIdx.x / a.s.hv;
  int n, len, c;
  long long start;
  if (!slot_chunk(a.s, slot, &n, &start, &len, &c)) return;
  const long long row0 = start + (long long)c * kC;
  const int rows = min(kC, len - c * kC);
  const int hq = h / (a.s.hv / a.s.hk);
  // the gates are wanted after the products: asked for first, they are there by then
  const float4 gb = warp == 0 ? load_gates(a, row0, rows, h, lane) : make_float4(0.f, 0.f, 0.f, 0.f);
  load_tile<E, kC, DK, 128>(ks, S::LDK, static_cast<const E*>(a.k) + row0 * a.ldk + (long long)hq * a.s.dk, a.ldk, rows,
                            a.s.dk, tid);
  load_tile<E, kC, DK, 128>(qs, S::LDK, static_cast<const E*>(a.q) + row0 * a.ldq + (long long)hq * a.s.dk, a.ldq, rows,
                            a.s.dk, tid);
  cp_commit();
  const long long id = slot * a.s.hv + h;
  float* vec = a.vec + id * kVec;
  cp_wait<0>();
  __syncthreads();

  // Rows 16 warp .. of q k^T and k k^T, columns up to the diagonal block.
  const Mat<E> mk{ks, S::LDK, 0}, mq{qs, S::LDK, 0};
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
  if (warp == 0) chunk_decays(gb, lane, g2, bet, vec);      // the warp with the fewest products
  __syncthreads();
#pragma unroll
  for (int rr = 0; rr < 2; ++rr) {
    const int i = m0 + g + rr * 8;
    const float2 gi = g2[i];
    const float be = bet[i];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = j * 8 + t2;
      const float4 gj = *reinterpret_cast<const float4*>(g2 + col);
      const float l0 = P::exp2((gi.x - gj.x) + (gi.y - gj.y)), l1 = P::exp2((gi.x - gj.z) + (gi.y - gj.w));
      const float p0 = col <= i ? a.s.scale * l0 * aq[j][rr * 2] : 0.f,
                  p1 = col < i ? a.s.scale * l1 * aq[j][rr * 2 + 1] : 0.f;
      P::template put2<PL>(Mat<E>{ps, S::LDT, kC * S::LDT}, i, col, p0, p1);
      *reinterpret_cast<float2*>(am + i * S::LDA + col) =
          make_float2(col < i ? be * l0 * ak[j][rr * 2] : 0.f, col + 1 < i ? be * l1 * ak[j][rr * 2 + 1] : 0.f);
    }
  }
  __syncthreads();
  {
    E* out = reinterpret_cast<E*>(a.p) + id * (kTPlanes<P> * kC * S::LDT);
    constexpr int V = 16 / sizeof(E);
    for (int i = tid; i < PL * kC * S::LDT / V; i += 128)
      reinterpret_cast<uint4*>(out)[i] = reinterpret_cast<const uint4*>(ps)[i];
  }
  invert<S::LDA>(am, warp, lane);
  {
    E* tout = reinterpret_cast<E*>(a.t) + id * (kTPlanes<P> * kC * S::LDT);
    const Mat<E> mt{tout, S::LDT, kC * S::LDT};
    for (int i = tid; i < kC * kC / 4; i += 128) {
      const int r = i / (kC / 4), col = (i % (kC / 4)) * 4;
      float4 v = *reinterpret_cast<const float4*>(am + r * S::LDA + col);
      if (r == col) v.x = 0.f;            // T - I: the products add R itself in fp32
      if (r == col + 1) v.y = 0.f;
      if (r == col + 2) v.z = 0.f;
      if (r == col + 3) v.w = 0.f;
      P::template put4<PL>(mt, r, col, v);
    }
  }
}

// ------------------------------------------------------------------- scan
// Chain warps: (wm, wn) holds 16 MT value columns (rows of S^T) by a quarter
// of the key width, and forms a quarter of the tokens of R and U.  Operands
// that all four quarters need pass through shared memory.  SPLIT: as many
// warps again form the outputs beside the chain (what few heads need: the
// chain's length is the time); else the chain's warps form them too.  Two more
// warps fetch the next chunk.  PL = 2: the operands of the
// serial chain in two planes.
template <class P, int DK, int MT, int WM, int PL, bool SPLIT>
struct ScanCfg {
  using E = typename P::E;
  static constexpr int DVT = 16 * MT * WM, CHAIN = 128 * WM, WORK = SPLIT ? 2 * CHAIN : CHAIN, FETCH = 64,
                       THREADS = WORK + FETCH;
  static constexpr int LDK = DK + P::PAD, LDT = kLdt<P>, LDV = DVT + P::PAD;
  static constexpr int NTS = DK / 32;                 // 8-column tiles of S^T a warp
  static constexpr int ST = P::STAGES;
  static constexpr int kQ = kC * LDK;                 // elements of each staged operand
  static constexpr int kT = PL * kC * LDT, kP = kT, kV = kC * LDV;
  static constexpr int STAGE = 2 * kQ + kT + kP + kV + kVec * (int)(4 / sizeof(E));
  static constexpr int SOP = PL * DVT * LDK, ROP = PL * DVT * LDT, UOP = ROP;
  // U and its decayed copy lie over the state operand, which is free by then
  static constexpr bool ALIAS = (size_t)(ST * STAGE + SOP + 2 * ROP + UOP + kV) * sizeof(E) + 64 > 227u * 1024u;
  static constexpr int ELEMS = ST * STAGE + (ALIAS ? (SOP > UOP + ROP ? SOP : UOP + ROP) : SOP + UOP + ROP) + ROP + kV;
  static constexpr size_t BYTES = (size_t)ELEMS * sizeof(E) + 64;
  static constexpr bool FITS = BYTES <= 227u * 1024u;
};

template <class P, int DK, int MT, int WM, int PL, bool SPLIT>
__global__ void __launch_bounds__(ScanCfg<P, DK, MT, WM, PL, SPLIT>::THREADS) k_gdr_scan(FwdArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  using C = ScanCfg<P, DK, MT, WM, PL, SPLIT>;
  using E = typename P::E;
  constexpr int NTS = C::NTS, ST = C::ST;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem_raw);
  uint64_t* empty = full + 2;
  E* stage = reinterpret_cast<E*>(smem_raw + 64);
  E* sop_p = stage + ST * C::STAGE;
  E* uop_p = C::ALIAS ? sop_p : sop_p + C::SOP;
  E* ukop_p = uop_p + C::UOP;
  E* rop_p = sop_p + (C::ELEMS - ST * C::STAGE - C::ROP - C::kV);
  E* ost = rop_p + C::ROP;
  const Mat<E> sop{sop_p, C::LDK, C::DVT * C::LDK}, rop{rop_p, C::LDT, C::DVT * C::LDT}, uop{uop_p, C::LDT, C::DVT * C::LDT},
      ukop{ukop_p, C::LDT, C::DVT * C::LDT};

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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

  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      tc::mbar_init(full + i, C::FETCH + 1);
      tc::mbar_init(empty + i, C::WORK / 32);
    }
    tc::mbar_init_fence();
  }
  __syncthreads();

  bool lost = false;        // a wait gave up: no more waiting, the results are void
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!lost && !tc::mbar_wait(bar, parity, kPolls)) {
      lost = true;
      atomicExch(&g_gdr_error, 1);
    }
  };

  if (tid >= C::WORK) {     // ---- the fetching warps
    const int ft = tid - C::WORK;
    const E* q = static_cast<const E*>(a.q) + start * a.ldq + (long long)hq * dk;
    const E* k = static_cast<const E*>(a.k) + start * a.ldk + (long long)hq * dk;
    const E* v = static_cast<const E*>(a.v) + start * a.ldv + (long long)h * dv + dv0;
    constexpr uint32_t tb = C::kT * sizeof(E), pb = C::kP * sizeof(E);
    for (int c = 0; c < nc; ++c) {
      const int st = ST == 2 ? (c & 1) : 0;
      if (c >= ST) wait(empty + st, (c / ST - 1) & 1);
      E* b = stage + st * C::STAGE;
      const int rows = min(kC, len - c * kC);
      const long long r0 = (long long)c * kC, id = (slot0 + c) * a.s.hv + h;
      if (ft == 0) {
        E* x = b + 2 * C::kQ + C::kV;
        bar_arrive_tx(full + st, tb + pb + kVec * 4);
        bulk_load(x, reinterpret_cast<const E*>(a.t) + id * (kTPlanes<P> * kC * C::LDT), tb, full + st);
        bulk_load(x + C::kT, reinterpret_cast<const E*>(a.p) + id * (kTPlanes<P> * kC * C::LDT), pb, full + st);
        bulk_load(x + C::kT + C::kP, a.vec + id * kVec, kVec * 4, full + st);
      }
      load_tile<E, kC, DK, C::FETCH>(b, C::LDK, k + r0 * a.ldk, a.ldk, rows, dk, ft);
      load_tile<E, kC, DK, C::FETCH>(b + C::kQ, C::LDK, q + r0 * a.ldq, a.ldq, rows, dk, ft);
      load_tile<E, kC, C::DVT, C::FETCH>(b + 2 * C::kQ, C::LDV, v + r0 * a.ldv, a.ldv, rows, dvn, ft);
      bar_arrive_cp(full + st);
    }
    return;
  }

  const bool chain = tid < C::CHAIN, outs = !SPLIT || !chain;
  const int wn = warp & 3, wm = (warp >> 2) % WM, m0 = wm * 16 * MT, otid = SPLIT ? tid - C::CHAIN : tid;
  const int g = lane >> 2, t2 = (lane & 3) * 2;
  E* o = static_cast<E*>(a.o) + (start * a.s.hv + h) * dv + dv0;
  const long long ldo = (long long)a.s.hv * dv;
  float s[MT][NTS][4];
  if (chain)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NTS; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = m0 + mt * 16 + g + (e >> 1) * 8, col = wn * (DK / 4) + nt * 8 + t2 + (e & 1);
          s[mt][nt][e] = a.init && r < dvn && col < dk ? a.init[(sh * dk + col) * dv + dv0 + r] : 0.f;
        }

  for (int c = 0; c < nc; ++c) {
    const int st = ST == 2 ? (c & 1) : 0;
    E* b = stage + st * C::STAGE;
    E* x = b + 2 * C::kQ + C::kV;
    const Mat<E> mk{b, C::LDK, 0}, mq{b + C::kQ, C::LDK, 0}, mt_{x, C::LDT, kC * C::LDT}, mp{x + C::kT, C::LDT, kC * C::LDT};
    const E* vs = b + 2 * C::kQ;
    const float* vec = reinterpret_cast<const float*>(x + C::kT + C::kP);
    if (chain)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NTS; ++nt)
#pragma unroll
          for (int rr = 0; rr < 2; ++rr)
            P::template put2<PL>(sop, m0 + mt * 16 + g + rr * 8, wn * (DK / 4) + nt * 8 + t2, s[mt][nt][2 * rr],
                                 s[mt][nt][2 * rr + 1]);
    wait(full + st, (c / ST) & 1);
    group_sync<1, C::WORK>();
    if (!SPLIT && c > 0)
      store_tile<E, kC, C::DVT, C::CHAIN>(o + (long long)(c - 1) * kC * ldo, ldo, ost, C::LDV, kC, dvn, otid);
    if (chain && a.save)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NTS; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = m0 + mt * 16 + g + (e >> 1) * 8, col = wn * (DK / 4) + nt * 8 + t2 + (e & 1);
            if (r < dvn && col < dk)
              put(reinterpret_cast<E*>(a.s0) + (((slot0 + c) * a.s.hv + h) * dk + col) * dv + dv0 + r, s[mt][nt][e]);
          }

    // S0^T k and S0^T q of this warp's 16 tokens
    float ar[MT][2][4] = {}, al[MT][2][4] = {}, ao[MT][2][4] = {};
#pragma unroll
    for (int k0 = 0; k0 < DK; k0 += P::KS) {
      typename P::template B<1> bk, bq;
      if (chain) P::load_bn(bk, mk, wn * 16, k0, lane);
      if (outs) P::load_bn(bq, mq, wn * 16, k0, lane);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        typename P::template A<PL> fa;
        P::load_a(fa, sop, m0 + mt * 16, k0, lane);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          if (chain) P::mma(ar[mt][hf], al[mt][hf], fa, bk, hf);
          // the outputs leave in the stored type: one plane of the state is enough
          if (outs) P::mma_hi(ao[mt][hf], fa, bq, hf);
        }
      }
    }
    const int i0 = wn * 16 + t2;
    float au[MT][2][4];
    if (chain) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int i = i0 + hf * 8;
        const float2 eg = *reinterpret_cast<const float2*>(vec + kVecEG + i);
        const float2 be = *reinterpret_cast<const float2*>(vec + kVecBeta + i);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int rr = 0; rr < 2; ++rr) {
            const int r = m0 + mt * 16 + g + rr * 8;
            const float v0 = to_f(vs[i * C::LDV + r]), v1 = to_f(vs[(i + 1) * C::LDV + r]);
            float s0 = ar[mt][hf][2 * rr], s1 = ar[mt][hf][2 * rr + 1];
            if constexpr (P::two_sums(PL, 1)) { s0 += al[mt][hf][2 * rr]; s1 += al[mt][hf][2 * rr + 1]; }
            // U = R + (T - I) R: R itself stays fp32
            au[mt][hf][2 * rr] = be.x * (v0 - eg.x * s0);
            au[mt][hf][2 * rr + 1] = be.y * (v1 - eg.y * s1);
            P::template put2<PL>(rop, r, i, au[mt][hf][2 * rr], au[mt][hf][2 * rr + 1]);
          }
      }
    }
    if (outs)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const float2 eg = *reinterpret_cast<const float2*>(vec + kVecEG + i0 + hf * 8);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int rr = 0; rr < 2; ++rr) {
            ao[mt][hf][2 * rr] *= a.s.scale * eg.x;
            ao[mt][hf][2 * rr + 1] *= a.s.scale * eg.y;
          }
      }
    if (chain) {
      group_sync<2, C::CHAIN>();
      float aw[MT][2][4] = {};
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
          for (int hf = 0; hf < 2; ++hf) P::mma(au[mt][hf], aw[mt][hf], fa, bt, hf);
        }
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int i = i0 + hf * 8;
        const float2 el = *reinterpret_cast<const float2*>(vec + kVecEGL + i);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int rr = 0; rr < 2; ++rr) {
            const int r = m0 + mt * 16 + g + rr * 8;
            float u0 = au[mt][hf][2 * rr], u1 = au[mt][hf][2 * rr + 1];
            if constexpr (P::two_sums(PL, PL)) { u0 += aw[mt][hf][2 * rr]; u1 += aw[mt][hf][2 * rr + 1]; }
            if (a.save && r < dvn) {
              E* p = reinterpret_cast<E*>(a.u) + (((slot0 + c) * a.s.hv + h) * kC + i) * dv + dv0 + r;
              put(p, u0);
              put(p + dv, u1);
            }
            P::template put2<PL>(uop, r, i, u0, u1);
            P::template put2<PL>(ukop, r, i, el.x * u0, el.y * u1);
          }
      }
    }
    group_sync<1, C::WORK>();
    if (outs) {
      // O += P U
#pragma unroll
      for (int k0 = 0; k0 < kC; k0 += P::KS) {
        if (k0 >= wn * 16 + 16) break;
        typename P::template B<PL> bp;
        P::load_bn(bp, mp, wn * 16, k0, lane);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          typename P::template A<PL> fa;
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
            put(ost + (i0 + hf * 8 + (e & 1)) * C::LDV + m0 + mt * 16 + g + (e >> 1) * 8, ao[mt][hf][e]);
    }
    if (chain) {
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
    }
    __syncwarp();
    if (lane == 0) bar_arrive(empty + st);
    if (SPLIT) {
      if (!chain) {
        group_sync<3, C::CHAIN>();
        store_tile<E, kC, C::DVT, C::CHAIN>(o + (long long)c * kC * ldo, ldo, ost, C::LDV, len - c * kC, dvn, otid);
        group_sync<3, C::CHAIN>();     // ost is written again in the next chunk
      }
    } else if (C::ALIAS) {
      group_sync<1, C::WORK>();
    }
  }
  if (lost)                  // copies that may still be on their way
    for (int i = 0; i < ST; ++i) tc::mbar_wait(full + i, 0, kPolls);
  if (!SPLIT && nc > 0) {
    group_sync<1, C::WORK>();
    store_tile<E, kC, C::DVT, C::CHAIN>(o + (long long)(nc - 1) * kC * ldo, ldo, ost, C::LDV, len - (nc - 1) * kC, dvn,
                                        otid);
  }
  if (chain && a.final_state) {
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
  const size_t bytes = PrepSmem<P, DK>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(k_gdr_prep<P, DK, PL>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) return e;
  TraceScope tr("k_gdr_prep", st);
  k_gdr_prep<P, DK, PL><<<(unsigned)blocks, 128, bytes, st>>>(a);
  return cudaGetLastError();
}

template <class P, int DK, int MT, int WM, int PL, bool SPLIT>
static cudaError_t launch_scan(FwdArgs a, cudaStream_t st) {
  using C = ScanCfg<P, DK, MT, WM, PL, SPLIT>;
  static_assert(C::FITS, "shared memory");
  static_assert(!(SPLIT && C::ALIAS), "the output warps still read the state when U is written");
  a.ntile = (a.s.dv + C::DVT - 1) / C::DVT;
  const long long blocks = (long long)a.s.n_seq * a.s.hv * a.ntile;
  cudaError_t e = cudaFuncSetAttribute(k_gdr_scan<P, DK, MT, WM, PL, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)C::BYTES);
  if (e != cudaSuccess) return e;
  TraceScope tr("k_gdr_scan", st);
  k_gdr_scan<P, DK, MT, WM, PL, SPLIT><<<(unsigned)blocks, C::THREADS, C::BYTES, st>>>(a);
  return cudaGetLastError();
}

template <class P, int DK, int PL>
static cudaError_t forward(const FwdArgs& a, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if constexpr (P::kMode == CFC_MATH_BF16) {
    if (a.s.rows > 0) e = launch_prep_tc(a, DK, PL, st);
    return e != cudaSuccess ? e : launch_scan_tc(a, DK, PL, st);
  } else {
    if (a.s.rows > 0) e = launch_prep<P, DK, PL>(a, st);
    if (e != cudaSuccess) return e;
    // Tiles of 32 value columns where their blocks still reach every SM, else of 16.
    const long long heads = (long long)a.s.n_seq * a.s.hv;
    if (a.s.dv > 16 && heads * ((a.s.dv + 31) / 32) >= 114) return launch_scan<P, DK, 1, 2, PL, true>(a, st);
    return launch_scan<P, DK, 1, 1, PL, true>(a, st);
  }
}

static size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

Workspace plan(long long rows, int n_seq, int hk, int hv, int dk, int dv, int math, int save) {
  Workspace w{};
  const size_t e = math == CFC_MATH_BF16 ? 2 : 4;
  const size_t slots = (size_t)slot_count(rows, n_seq) * hv;
  size_t off = 0;
  auto take = [&](size_t* at, size_t bytes) { *at = off; off = up256(off + bytes); };
  const bool bf = math == CFC_MATH_BF16;
  take(&w.off_t, slots * (bf ? kImage : kC * kLdt<MFp32> * sizeof(float)));
  take(&w.off_p, bf ? 0 : slots * kC * kLdt<MFp32> * sizeof(float));
  take(&w.off_vec, slots * kVec * 4);
  take(&w.off_order, bf && n_seq <= kMaxOrder ? n_seq * sizeof(int) : 0);
  if (save) {
    const size_t wk = bf ? (dk <= 64 ? 64 : 128) : dk, wv = bf ? (dv + 63) / 64 * 64 : dv;
    take(&w.off_s0, slots * wk * wv * e);
    take(&w.off_u, slots * kC * wv * e);
    take(&w.off_ds, slots * wk * wv * e);
    take(&w.off_dr, slots * kC * wv * e);
    if (hv != hk && !bf) {
      take(&w.off_dq, (size_t)rows * hv * dk * 4);
      take(&w.off_dk, (size_t)rows * hv * dk * 4);
    }
  }
  w.total = off ? off : 256;
  return w;
}

}  // namespace gdr

int read_gdr_error(int clear) {
  const int t = gdr::read_gdr_tc_error(clear), r = gdr::read_gdr_grad_error(clear);
  if (t != 0 || r != 0) return t != 0 ? t : r;
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, gdr::g_gdr_error, sizeof(int)) != cudaSuccess) return CFC_ERR_DEVICE;
  if (clear && v) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(gdr::g_gdr_error, &zero, sizeof(int)) != cudaSuccess) return CFC_ERR_DEVICE;
  }
  return v;
}

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
  a.s = Shape{g.off, g.n_seq, g.rows, g.hk, g.hv, g.dk, g.dv, g.scale, (int)(g.rows / g.n_seq)};
  a.q = g.q; a.k = g.k; a.v = g.v;
  a.ldq = g.ldq; a.ldk = g.ldk; a.ldv = g.ldv;
  a.g = g.g; a.beta = g.beta; a.init = g.init; a.final_state = g.final_state; a.o = g.o;
  a.t = g.ws + w.off_t; a.p = g.ws + w.off_p;
  a.vec = reinterpret_cast<float*>(g.ws + w.off_vec);
  if (g.off && g.math == CFC_MATH_BF16 && g.n_seq <= kMaxOrder) a.order = reinterpret_cast<int*>(g.ws + w.off_order);
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
