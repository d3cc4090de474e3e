// cfc_gdr.cu -- the gated delta rule over whole sequences: workspace, dispatch,
// and the forward in FP32 (formulas at the top of gdr_common.cuh; bf16 is in
// cfc_gdr_tc.cu).
//
//   k_gdr_prep   one block per (chunk, value head): the decays, T - I and P
//   k_gdr_scan   one block per (sequence, value head, tile of value columns):
//                the serial pass over the chunks, the state in registers
//
// Products are mma.sync of TF32 pairs (three a step, fp32-accurate): tcgen05
// takes TF32 too, but its operands would have to be split and laid out in
// shared memory first, twice the bytes of a tile that already fills an SM.
// The state's columns do not touch one another, so a head's value columns are
// split over blocks; the serial pass is a chain of latencies, 7 us a chunk of
// 128 keys x 16 columns (32 x 64 tokens x 2 heads of 64: prep 10 us, scan 9,
// backward 10 and 16; 16384 tokens x 16 heads of 128: 1.9 ms, 80 us by bytes).
#include "gdr_common.cuh"

namespace cfc {
namespace gdr {

__device__ int g_gdr_error = 0;   // a bounded wait gave up

// ------------------------------------------------------------------- prep
template <int DK>
struct PrepSmem {
  static constexpr int LDK = DK + kPad;
  static constexpr int kTile = kC * LDK, kA = kC * kLdT;
  // k, then A and T; q, then P: the products are done when the others begin
  static constexpr int kOffQ = kTile > kA ? kTile : kA, kOffG = 2 * kOffQ;
  static constexpr size_t kBytes = (kOffG + 3 * kC) * sizeof(float);      // G / ln 2 in pairs, beta
};

template <int DK>
__global__ void __launch_bounds__(128) k_gdr_prep(FwdArgs a) {
  extern __shared__ __align__(16) float smem[];
  using S = PrepSmem<DK>;
  float *ks = smem, *am = smem, *qs = smem + S::kOffQ, *ps = qs;
  float2* g2 = reinterpret_cast<float2*>(smem + S::kOffG);
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
  load_tile<float, kC, DK, 128>(ks, S::LDK, static_cast<const float*>(a.k) + row0 * a.ldk + (long long)hq * a.s.dk,
                                a.ldk, rows, a.s.dk, tid);
  load_tile<float, kC, DK, 128>(qs, S::LDK, static_cast<const float*>(a.q) + row0 * a.ldq + (long long)hq * a.s.dk,
                                a.ldq, rows, a.s.dk, tid);
  cp_commit();
  const long long id = slot * a.s.hv + h;
  cp_wait<0>();
  __syncthreads();

  // Rows 16 warp .. of q k^T and k k^T, columns up to the diagonal block.
  const Mat<float> mk{ks, S::LDK}, mq{qs, S::LDK};
  const int m0 = warp * 16, g = lane >> 2, t2 = (lane & 3) * 2;
  float aq[8][4] = {}, ak[8][4] = {};
  for (int k0 = 0; k0 < DK; k0 += F::KS) {
    F::A fq, fk;
    F::load_a(fq, mq, m0, k0, lane);
    F::load_a(fk, mk, m0, k0, lane);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j > warp) continue;
      F::B fb;
      F::load_bn(fb, mk, j * 16, k0, lane);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        F::mma(aq[2 * j + hf], fq, fb, hf);
        F::mma(ak[2 * j + hf], fk, fb, hf);
      }
    }
  }
  float* vec = a.vec + id * kVec;
  if (warp == 0) chunk_decays(gb, lane, c == 0 && !a.init, g2, bet, vec);   // the warp with the fewest products
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
      const float l0 = exp2f((gi.x - gj.x) + (gi.y - gj.y)), l1 = exp2f((gi.x - gj.z) + (gi.y - gj.w));
      *reinterpret_cast<float2*>(ps + i * kLdT + col) =
          make_float2(col <= i ? a.s.scale * l0 * aq[j][rr * 2] : 0.f, col < i ? a.s.scale * l1 * aq[j][rr * 2 + 1] : 0.f);
      float a0 = col < i ? be * l0 * ak[j][rr * 2] : 0.f, a1 = col + 1 < i ? be * l1 * ak[j][rr * 2 + 1] : 0.f;
      if (!finite(fabsf(a0) + fabsf(a1))) {
        drop(a0, vec, i);
        drop(a1, vec, i);
      }
      *reinterpret_cast<float2*>(am + i * kLdT + col) = make_float2(a0, a1);
    }
  }
  __syncthreads();
  float4* pout = reinterpret_cast<float4*>(a.p) + id * (kC * kLdT / 4);
  for (int i = tid; i < kC * kLdT / 4; i += 128) pout[i] = reinterpret_cast<const float4*>(ps)[i];
  invert<kLdT>(am, warp, lane);
  float4* tout = reinterpret_cast<float4*>(a.t) + id * (kC * kLdT / 4);
  for (int i = tid; i < kC * kC / 4; i += 128) {
    const int r = i / (kC / 4), col = (i % (kC / 4)) * 4;
    float4 v = *reinterpret_cast<const float4*>(am + r * kLdT + col);
    if (!finite(fabsf(v.x) + fabsf(v.y) + fabsf(v.z) + fabsf(v.w))) {
      drop(v.x, vec, r);
      drop(v.y, vec, r);
      drop(v.z, vec, r);
      drop(v.w, vec, r);
    }
    if (r == col) v.x = 0.f;            // T - I: the products add R itself
    if (r == col + 1) v.y = 0.f;
    if (r == col + 2) v.z = 0.f;
    if (r == col + 3) v.w = 0.f;
    tout[(r * kLdT + col) / 4] = v;
  }
}

// ------------------------------------------------------------------- scan
// WM x 4 chain warps: (wm, wn) holds 16 value columns (rows of S^T) by a
// quarter of the key width, and forms a quarter of the tokens of R and U.
// Operands that all four quarters need pass through shared memory.  As many
// warps again form the outputs beside the chain, two more fetch the next chunk.
template <int DK, int WM>
struct ScanCfg {
  static constexpr int DVT = 16 * WM, CHAIN = 128 * WM, WORK = 2 * CHAIN, FETCH = 64, THREADS = WORK + FETCH;
  static constexpr int LDK = DK + kPad, LDV = DVT + kPad;
  static constexpr int NTS = DK / 32;                 // 8-column tiles of S^T a warp
  static constexpr int kQ = kC * LDK, kT = kC * kLdT, kV = kC * LDV;
  static constexpr int STAGE = 2 * kQ + 2 * kT + kV + kVec;
  static constexpr int SOP = DVT * LDK, ROP = DVT * kLdT;
  static constexpr size_t HEAD = 64 + 4 * DVT;        // barriers; each column's first bad token
  static constexpr size_t BYTES = (STAGE + SOP + 3 * ROP + kV) * sizeof(float) + HEAD;
  static_assert(BYTES <= 227u * 1024u, "shared memory");
};

template <int DK, int WM>
__global__ void __launch_bounds__(ScanCfg<DK, WM>::THREADS) k_gdr_scan(FwdArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  using C = ScanCfg<DK, WM>;
  constexpr int NTS = C::NTS;
  uint64_t *full = reinterpret_cast<uint64_t*>(smem_raw), *empty = full + 1;
  int *any_bad = reinterpret_cast<int*>(smem_raw + 32), *bad_from = reinterpret_cast<int*>(smem_raw + 64);
  float* stage = reinterpret_cast<float*>(smem_raw + C::HEAD);
  float* x = stage + 2 * C::kQ + C::kV;               // T - I, P, the vectors
  const float *vs = stage + 2 * C::kQ, *vec = x + 2 * C::kT;
  float* ops = stage + C::STAGE;
  const Mat<float> mk{stage, C::LDK}, mq{stage + C::kQ, C::LDK}, mt{x, kLdT}, mp{x + C::kT, kLdT};
  const Mat<float> sop{ops, C::LDK}, rop{ops + C::SOP, kLdT}, uop{ops + C::SOP + C::ROP, kLdT},
      ukop{ops + C::SOP + 2 * C::ROP, kLdT};
  float* ost = ops + C::SOP + 3 * C::ROP;

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
    tc::mbar_init(full, C::FETCH + 1);
    tc::mbar_init(empty, C::WORK / 32);
    tc::mbar_init_fence();
  }
  __syncthreads();
  bool lost = false;        // a wait gave up: no more waiting, the results are void
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!lost && !tc::mbar_wait(bar, parity, kPolls)) {
      lost = true;
      atomicExch(&g_gdr_error, 1);
    }
    lost = __any_sync(0xffffffffu, lost);      // a warp goes on as one
  };

  if (tid >= C::WORK) {     // ---- the fetching warps
    const int ft = tid - C::WORK;
    const float* q = static_cast<const float*>(a.q) + start * a.ldq + (long long)hq * dk;
    const float* k = static_cast<const float*>(a.k) + start * a.ldk + (long long)hq * dk;
    const float* v = static_cast<const float*>(a.v) + start * a.ldv + (long long)h * dv + dv0;
    for (int c = 0; c < nc; ++c) {
      if (c > 0) wait(empty, (c - 1) & 1);
      const int rows = min(kC, len - c * kC);
      const long long r0 = (long long)c * kC, id = (slot0 + c) * a.s.hv + h;
      if (ft == 0) {
        constexpr uint32_t bytes = C::kT * sizeof(float);
        bar_arrive_tx(full, 2 * bytes + kVec * 4);
        bulk_load(x, reinterpret_cast<const float*>(a.t) + id * C::kT, bytes, full);
        bulk_load(x + C::kT, reinterpret_cast<const float*>(a.p) + id * C::kT, bytes, full);
        bulk_load(x + 2 * C::kT, a.vec + id * kVec, kVec * 4, full);
      }
      load_tile<float, kC, DK, C::FETCH>(mk.p, C::LDK, k + r0 * a.ldk, a.ldk, rows, dk, ft);
      load_tile<float, kC, DK, C::FETCH>(mq.p, C::LDK, q + r0 * a.ldq, a.ldq, rows, dk, ft);
      load_tile<float, kC, C::DVT, C::FETCH>(stage + 2 * C::kQ, C::LDV, v + r0 * a.ldv, a.ldv, rows, dvn, ft);
      bar_arrive_cp(full);
    }
    return;
  }

  const bool chain = tid < C::CHAIN;
  const int wn = warp & 3, m0 = ((warp >> 2) % WM) * 16;
  const int g = lane >> 2, t2 = (lane & 3) * 2, i0 = wn * 16 + t2;
  float* o = static_cast<float*>(a.o) + (start * a.s.hv + h) * dv + dv0;
  const long long ldo = (long long)a.s.hv * dv;
  // S^T: element e of 8-column tile nt is value column m0 + g + 8 (e / 2), key column:
  auto key = [&](int nt, int e) { return wn * (DK / 4) + nt * 8 + t2 + (e & 1); };
  float s[NTS][4];
  if (chain)
#pragma unroll
    for (int nt = 0; nt < NTS; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = m0 + g + (e >> 1) * 8;
        s[nt][e] = a.init && r < dvn && key(nt, e) < dk ? a.init[(sh * dk + key(nt, e)) * dv + dv0 + r] : 0.f;
      }

  for (int c = 0; c < nc; ++c) {
    const long long id = (slot0 + c) * a.s.hv + h;
    if (chain) {
#pragma unroll
      for (int nt = 0; nt < NTS; ++nt)
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) F::put2(sop, m0 + g + rr * 8, key(nt, 0), s[nt][2 * rr], s[nt][2 * rr + 1]);
    }
    wait(full, c & 1);
    group_sync<1, C::WORK>();
    if (chain) {
      if (a.save) {
        float* s0 = reinterpret_cast<float*>(a.s0) + id * dk * dv + dv0;
#pragma unroll
        for (int nt = 0; nt < NTS; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = m0 + g + (e >> 1) * 8;
            if (r < dvn && key(nt, e) < dk) s0[(long long)key(nt, e) * dv + r] = s[nt][e];
          }
      }
      // R of this warp's 16 tokens
      float ar[2][4] = {}, al[2][4] = {}, au[2][4], aw[2][4] = {};
      bool bad = false;
#pragma unroll
      for (int k0 = 0; k0 < DK; k0 += F::KS) {
        F::A fa;
        F::B fb;
        F::load_a(fa, sop, m0, k0, lane);
        F::load_bn(fb, mk, wn * 16, k0, lane);
        F::mma(ar[0], al[0], fa, fb, 0);
        F::mma(ar[1], al[1], fa, fb, 1);
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int i = i0 + hf * 8;
        const float2 eg = *reinterpret_cast<const float2*>(vec + kVecEG + i);
        const float2 be = *reinterpret_cast<const float2*>(vec + kVecBeta + i);
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          const int r = m0 + g + rr * 8;
          au[hf][2 * rr] = be.x * (vs[i * C::LDV + r] - eg.x * (ar[hf][2 * rr] + al[hf][2 * rr]));
          au[hf][2 * rr + 1] = be.y * (vs[(i + 1) * C::LDV + r] - eg.y * (ar[hf][2 * rr + 1] + al[hf][2 * rr + 1]));
          F::put2(rop, r, i, au[hf][2 * rr], au[hf][2 * rr + 1]);
          bad |= !finite(fabsf(au[hf][2 * rr]) + fabsf(au[hf][2 * rr + 1]));
        }
      }
      // From a bad value of a column on its R reads as zero and its U is NaN.
      const bool some = group_any<2, C::CHAIN>(bad);
      if (tid == 0) *any_bad = some;
      if (some) {
        for (int r = tid; r < C::DVT; r += C::CHAIN) bad_from[r] = kC;
        group_sync<2, C::CHAIN>();
#pragma unroll
        for (int x = 0; x < 8; ++x)
          if (!finite(au[x >> 2][x & 3]))
            atomicMin(bad_from + m0 + g + ((x >> 1) & 1) * 8, i0 + (x >> 2) * 8 + (x & 1));
        group_sync<2, C::CHAIN>();
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int r = m0 + g + ((x >> 1) & 1) * 8, i = i0 + (x >> 2) * 8 + (x & 1);
          if (i >= bad_from[r]) {
            au[x >> 2][x & 3] = nanf("");
            rop.p[r * kLdT + i] = 0.f;
          }
        }
        group_sync<2, C::CHAIN>();
      }
      // U = R + (T - I) R
#pragma unroll
      for (int k0 = 0; k0 < kC; k0 += F::KS) {
        if (k0 >= wn * 16 + 16) break;
        F::A fa;
        F::B fb;
        F::load_a(fa, rop, m0, k0, lane);
        F::load_bn(fb, mt, wn * 16, k0, lane);
        F::mma(au[0], aw[0], fa, fb, 0);
        F::mma(au[1], aw[1], fa, fb, 1);
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int i = i0 + hf * 8;
        const float2 el = *reinterpret_cast<const float2*>(vec + kVecEGL + i);
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          const int r = m0 + g + rr * 8;
          const float u0 = au[hf][2 * rr] + aw[hf][2 * rr], u1 = au[hf][2 * rr + 1] + aw[hf][2 * rr + 1];
          if (a.save && r < dvn) {
            float* p = reinterpret_cast<float*>(a.u) + (id * kC + i) * dv + dv0 + r;
            p[0] = u0;
            p[dv] = u1;
          }
          const bool from = some && i + 1 >= bad_from[r];      // for the outputs alone: the state takes them as they are
          F::put2(uop, r, i, from && i >= bad_from[r] ? 0.f : u0, from ? 0.f : u1);
          F::put2(ukop, r, i, el.x * u0, el.y * u1);
        }
      }
      group_sync<1, C::WORK>();
      // S1 = exp(G_C) S0 + sum_i exp(G_C - G_i) U_i k_i^T
      const float d = vec[kVecD];
#pragma unroll
      for (int nt = 0; nt < NTS; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] *= d;
#pragma unroll
      for (int k0 = 0; k0 < kC; k0 += F::KS) {
        F::A fa;
        F::load_a(fa, ukop, m0, k0, lane);
#pragma unroll
        for (int j = 0; j < NTS / 2; ++j) {
          F::B fb;
          F::load_bk(fb, mk, wn * (DK / 4) + j * 16, k0, lane);
          F::mma(s[2 * j], fa, fb, 0);
          F::mma(s[2 * j + 1], fa, fb, 1);
        }
      }
      __syncwarp();
      if (lane == 0) bar_arrive(empty);
    } else {
      // O = scale exp(G) S0^T q + P U of this warp's 16 tokens
      float ao[2][4] = {};
#pragma unroll
      for (int k0 = 0; k0 < DK; k0 += F::KS) {
        F::A fa;
        F::B fb;
        F::load_a(fa, sop, m0, k0, lane);
        F::load_bn(fb, mq, wn * 16, k0, lane);
        F::mma(ao[0], fa, fb, 0);
        F::mma(ao[1], fa, fb, 1);
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const float2 eg = *reinterpret_cast<const float2*>(vec + kVecEG + i0 + hf * 8);
#pragma unroll
        for (int e = 0; e < 4; ++e) ao[hf][e] *= a.s.scale * ((e & 1) ? eg.y : eg.x);
      }
      group_sync<1, C::WORK>();
#pragma unroll
      for (int k0 = 0; k0 < kC; k0 += F::KS) {
        if (k0 >= wn * 16 + 16) break;
        F::A fa;
        F::B fb;
        F::load_a(fa, uop, m0, k0, lane);
        F::load_bn(fb, mp, wn * 16, k0, lane);
        F::mma(ao[0], fa, fb, 0);
        F::mma(ao[1], fa, fb, 1);
      }
      if (*any_bad)
#pragma unroll
        for (int x = 0; x < 8; ++x)
          if (i0 + (x >> 2) * 8 + (x & 1) >= bad_from[m0 + g + ((x >> 1) & 1) * 8]) ao[x >> 2][x & 3] = nanf("");
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          ost[(i0 + hf * 8 + (e & 1)) * C::LDV + m0 + g + (e >> 1) * 8] = ao[hf][e];
      __syncwarp();
      if (lane == 0) bar_arrive(empty);
      group_sync<3, C::CHAIN>();
      store_tile<float, kC, C::DVT, C::CHAIN>(o + (long long)c * kC * ldo, ldo, ost, C::LDV, len - c * kC, dvn,
                                              tid - C::CHAIN);
      group_sync<3, C::CHAIN>();     // ost is written again in the next chunk
    }
  }
  if (lost) tc::mbar_wait(full, 0, kPolls);      // copies that may still be on their way
  if (chain && a.final_state)
#pragma unroll
    for (int nt = 0; nt < NTS; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = m0 + g + (e >> 1) * 8;
        if (r < dvn && key(nt, e) < dk) a.final_state[(sh * dk + key(nt, e)) * dv + dv0 + r] = s[nt][e];
      }
}

template <int DK, int WM>
static cudaError_t scan(FwdArgs a, cudaStream_t st) {
  using C = ScanCfg<DK, WM>;
  a.ntile = (a.s.dv + C::DVT - 1) / C::DVT;
  cudaError_t e = allow_smem<k_gdr_scan<DK, WM>>(C::BYTES);
  if (e != cudaSuccess) return e;
  TraceScope tr("k_gdr_scan", st);
  k_gdr_scan<DK, WM><<<(unsigned)((long long)a.s.n_seq * a.s.hv * a.ntile), C::THREADS, C::BYTES, st>>>(a);
  return cudaGetLastError();
}

template <int DK>
static cudaError_t forward_fp32(const FwdArgs& a, cudaStream_t st) {
  if (a.s.rows > 0) {
    using S = PrepSmem<DK>;
    cudaError_t e = allow_smem<k_gdr_prep<DK>>(S::kBytes);
    if (e != cudaSuccess) return e;
    TraceScope tr("k_gdr_prep", st);
    k_gdr_prep<DK><<<(unsigned)(slot_count(a.s.rows, a.s.n_seq) * a.s.hv), 128, S::kBytes, st>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  // Tiles of 32 value columns or of 16 (32 heads of 128, 512 tokens: 86 us, 127).
  return wide_tiles((long long)a.s.n_seq * a.s.hv, a.s.dv, 16) ? scan<DK, 2>(a, st) : scan<DK, 1>(a, st);
}

static size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

Workspace plan(long long rows, int n_seq, int hk, int hv, int dk, int dv, int math, int save) {
  Workspace w{};
  const size_t e = math == CFC_MATH_BF16 ? 2 : 4;
  const size_t slots = (size_t)slot_count(rows, n_seq) * hv;
  size_t off = 0;
  auto take = [&](size_t* at, size_t bytes) { *at = off; off = up256(off + bytes); };
  const bool bf = math == CFC_MATH_BF16;
  take(&w.off_t, slots * (bf ? kImage : kC * kLdT * sizeof(float)));
  take(&w.off_p, bf ? 0 : slots * kC * kLdT * sizeof(float));
  take(&w.off_vec, slots * kVec * 4);
  take(&w.off_order, bf && n_seq <= kMaxOrder ? (n_seq + 2) * sizeof(int) : 0);
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

bool gdr_error_words(int* (&words)[kGdrErrorWords]) {
  void* p = nullptr;
  words[0] = cudaGetSymbolAddress(&p, gdr::g_gdr_error) == cudaSuccess ? static_cast<int*>(p) : nullptr;
  words[1] = gdr::gdr_tc_error_word();
  words[2] = gdr::gdr_grad_error_word();
  return words[0] && words[1] && words[2];
}

int read_gdr_error(int clear) {
  int* words[kGdrErrorWords];
  if (!gdr_error_words(words)) return CFC_ERR_DEVICE;
  int any = 0;
  for (int* word : words) {              // each is read and cleared, whatever the others hold
    int v = 0;
    const int zero = 0;
    if (cudaMemcpy(&v, word, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return CFC_ERR_DEVICE;
    if (clear && v && cudaMemcpy(word, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess) return CFC_ERR_DEVICE;
    any |= v;
  }
  return any;
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
  if (g.off && g.rows > 0 && g.math == CFC_MATH_BF16 && g.n_seq <= kMaxOrder)
    a.order = reinterpret_cast<int*>(g.ws + w.off_order);
  a.save = g.save;
  if (g.save) { a.s0 = g.ws + w.off_s0; a.u = g.ws + w.off_u; }
  const int tile = g.dk <= 64 ? 64 : 128;
  if (g.math == CFC_MATH_FP32) return tile == 64 ? forward_fp32<64>(a, st) : forward_fp32<128>(a, st);
  // A state that leaves the call is fp32: its chain keeps two planes.
  const int planes = g.final_state ? 2 : 1;
  const cudaError_t e = g.rows > 0 ? launch_prep_tc(a, tile, planes, st) : cudaSuccess;
  return e != cudaSuccess ? e : launch_scan_tc(a, tile, planes, st);
}

}  // namespace cfc
