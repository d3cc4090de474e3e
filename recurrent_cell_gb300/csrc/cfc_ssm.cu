// cfc_ssm.cu -- the selective scan over whole sequences, forward (ssm_common.cuh
// has the formulas and the split).
//
//   k_ssm<., true>   the end state of each segment from its own rows, and its sum of dt
//   k_ssm_carry      the states between segments: h_s = local_s + exp(A sum dt) h_{s-1}
//   k_ssm<., false>  the scan itself
//
// The first two run only where segments cut sequences.
#include "ssm_common.cuh"

namespace cfc {
namespace ssm {

template <class G, bool LOCAL>
struct __align__(16) FwdTiles {
  float dt[kT][G::CW], dx[kT][G::CW];        // dt, dt x
  float B[kT][G::NP];
  float C[LOCAL ? 1 : kT][G::NP];
  float y[LOCAL ? 1 : kT][4 * G::CW];        // C . h, a part from each state lane
};

// Where state lane sl's part of channels c .. c + CPL - 1 of row t lies.  With 4 channels a
// lane, 16-byte pieces permuted so that neither the lanes of a token nor those that add
// the parts of several rows meet in a bank.
template <class G>
__device__ __forceinline__ int y_at(int t, int sl, int c) {
  if constexpr (G::CPL == 4) return (c >> 3) * 32 + (((((c >> 2) & 1) * 4 + sl) ^ ((c >> 3) | (t & 1) << 2)) << 2);
  else return sl * G::CW + c;
}

// What a token reads of the tiles.
template <class G, bool LOCAL>
struct Operands {
  F2 dt[G::CPAIRS], dx[G::CPAIRS], b[G::SPAIRS], c[G::SPAIRS];
  __device__ __forceinline__ void read(const FwdTiles<G, LOCAL>& sm, const Tile<G>& w, int t) {
    get_channels<G>(sm.dt[t], w.cl, dt);
    get_channels<G>(sm.dx[t], w.cl, dx);
    get_states<G>(sm.B[t], w.sl, b);
    if constexpr (!LOCAL) get_states<G>(sm.C[t], w.sl, c);
  }
};

// One token: the states, and C . h of the lane's states.
template <class G, bool LOCAL>
__device__ __forceinline__ void token(FwdTiles<G, LOCAL>& sm, const Tile<G>& w, int t, const Operands<G, LOCAL>& o,
                                      const F2 (&A2)[G::PAIRS], F2 (&h)[G::PAIRS], F2 (&sum)[G::CPAIRS]) {
  F2 y[G::CPAIRS];
#pragma unroll
  for (int p = 0; p < G::PAIRS; ++p) {
    const int i = cpair<G>(p), j = spair<G>(p);
    h[p] = fma2(decay2(o.dt[i], A2[p]), h[p], mul2(o.dx[i], o.b[j]));
    if constexpr (!LOCAL) y[i] = j == 0 ? mul2(o.c[j], h[p]) : fma2(o.c[j], h[p], y[i]);
  }
  if constexpr (LOCAL) {
#pragma unroll
    for (int i = 0; i < G::CPAIRS; ++i) sum[i] = add2(sum[i], o.dt[i]);
  } else {
    float* to = sm.y[t] + y_at<G>(t, w.sl, w.cl * G::CPL);
    if constexpr (G::CPL == 4) *reinterpret_cast<ulonglong2*>(to) = make_ulonglong2(y[0], y[1]);
    else if constexpr (G::CPL == 2) *reinterpret_cast<F2*>(to) = y[0];
    else *to = sum2(y[0]);
  }
}

template <class G, bool LOCAL>
__global__ void __launch_bounds__(32, kResident) k_ssm(Args a, bool save) {
  using E = typename G::E;
  using U = Pairs<E, G::VN>;
  constexpr int P = G::P, VN = G::VN, VP = VN / 2;
  __shared__ FwdTiles<G, LOCAL> sm;
  const Tile<G> w(a, blockIdx.x);
  const int seg = blockIdx.y;
  F2 h[G::PAIRS];

  if (!LOCAL && seg >= a.n_seg) {            // the states after sequences without rows
    const int step = (gridDim.y - a.n_seg) * 32;
    for (long long i0 = (long long)(seg - a.n_seg) * 32; i0 < a.s.n; i0 += step) {
      long long begin = 0, end = 1;
      if (i0 + w.lane < a.s.n) seqs::range_of(a.s, (int)(i0 + w.lane), &begin, &end);
      unsigned none = __ballot_sync(0xffffffffu, begin >= end);
      while (none) {
        const long long i = i0 + __ffs(none) - 1;
        none &= none - 1;
        load_state<G>(a, w, a.init, i, h);
        store_state<G>(a, w, a.final_state, i, h);
      }
    }
    return;
  }

  a.s = seqs::trim(a.s);
  const long long r0 = seg * a.S, r1 = a.s.rows - r0 < a.S ? a.s.rows : r0 + a.S;
  Where q;
  long long row = r0;
  if (r0 >= r1) {                            // rows behind the last sequence
    if (LOCAL && blockIdx.x == 0 && w.lane == 0) a.flags[seg] = 0;
    return;
  }
  if constexpr (LOCAL) {
    q = seqs::find(a.s, r1 - 1);
    const bool cut = q.end > r1, starts = q.begin >= r0;
    if (blockIdx.x == 0 && w.lane == 0) a.flags[seg] = (cut ? kCut : 0) | (starts ? kStarts : 0);
    if (!cut) return;
    if (starts) row = q.begin;
#pragma unroll
    for (int p = 0; p < G::PAIRS; ++p) h[p] = 0;
  } else {
    q = seqs::find(a.s, r0);
    if (q.begin < r0) load_lanes<G>(a.local, (long long)(seg - 1) * a.tiles + blockIdx.x, w.lane, h);
  }
  F2 A2[G::PAIRS], bias[VP], D[VP], sum[G::CPAIRS] = {};
  load_A<G>(a, w, A2);
  load_pairs<G>(w, a.bias, bias);
  load_pairs<G>(w, LOCAL ? nullptr : a.D, D);

  uint4 xv[P], dv[P], zv[P];
  Rows<G> bv, cv;
  auto fetch = [&](long long at) {
    const int n = r1 - at < kT ? (int)(r1 - at) : kT;      // none behind the segment
    load_raw<G>(w, a.x, a.ldx, at, n, xv);
    load_raw<G>(w, a.delta, a.ldd, at, n, dv);
    bv.fetch(a, w, a.B, a.ldb, at, n);
    if (!LOCAL) cv.fetch(a, w, a.C, a.ldc, at, n);
  };
  fetch(row);
  for (int chunk = 0; row < r1; row += kT, ++chunk) {
    const int n = r1 - row < kT ? (int)(r1 - row) : kT;
    if (!LOCAL && save) store_lanes<G>(a.ckpt, ((long long)seg * a.cps + chunk) * a.tiles + blockIdx.x, w.lane, h);
    F2 y[P][LOCAL ? 1 : VP];                               // D x
#pragma unroll
    for (int k = 0; k < P; ++k) {
      F2 x[VP], dt[VP];
      U::get(x, xv[k]);
      U::get(dt, dv[k]);
#pragma unroll
      for (int e = 0; e < VP; ++e) {
        dt[e] = softplus2(add2(dt[e], bias[e]));
        if constexpr (!LOCAL) y[k][e] = mul2(D[e], x[e]);
        x[e] = mul2(x[e], dt[e]);
      }
      if (w.row(k) < kT) {
        put_pairs(&sm.dt[w.row(k)][w.col()], dt);
        put_pairs(&sm.dx[w.row(k)][w.col()], x);
      }
    }
    bv.stage(a, w, a.B, a.ldb, row, n, sm.B[0]);
    if constexpr (!LOCAL) {
      cv.stage(a, w, a.C, a.ldc, row, n, sm.C[0]);
      if (a.z) load_raw<G>(w, a.z, a.ldz, row, n, zv);
    }
    __syncwarp();
    fetch(row + kT);
    if (n == kT && q.begin < row && q.end > row + kT) {    // inside one sequence: no state comes or goes
      Operands<G, LOCAL> now, next;
      now.read(sm, w, 0);
#pragma unroll 4
      for (int t = 0; t < kT; ++t) {
        next.read(sm, w, t + 1 < kT ? t + 1 : t);
        token<G, LOCAL>(sm, w, t, now, A2, h, sum);
        now = next;
      }
    } else {
      for (int t = 0; t < n;) {
        if (row + t == q.begin) load_state<G>(a, w, a.init, q.i, h);
        const int m = q.end - row < n ? (int)(q.end - row) : n;
        for (; t < m; ++t) {
          Operands<G, LOCAL> now;
          now.read(sm, w, t);
          token<G, LOCAL>(sm, w, t, now, A2, h, sum);
        }
        if (!LOCAL && row + t == q.end) {
          if (a.final_state) store_state<G>(a, w, a.final_state, q.i, h);
          if (row + t < a.s.rows) q = seqs::find(a.s, row + t);
        }
      }
    }
    __syncwarp();
    if constexpr (!LOCAL) {
#pragma unroll
      for (int k = 0; k < P; ++k)
        if (w.row(k) < n && w.col() < w.cols) {
          F2 z[VP];
#pragma unroll
          for (int s = 0; s < 4; ++s) {
#pragma unroll
            for (int e = 0; e < VP; e += 2) {
              const float* part = sm.y[w.row(k)] + y_at<G>(w.row(k), s, w.col() + 2 * e);
              const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(part);
              y[k][e] = add2(y[k][e], u.x);
              y[k][e + 1] = add2(y[k][e + 1], u.y);
            }
          }
          if (a.z) {
            U::get(z, zv[k]);
#pragma unroll
            for (int e = 0; e < VP; ++e) y[k][e] = mul2(y[k][e], mul2(z[e], sigmoid2(z[e])));
          }
          E* to = static_cast<E*>(a.y) + (row + w.row(k)) * a.d + w.c0 + w.col();
          __stcs(reinterpret_cast<uint4*>(to), U::make(y[k]));
        }
    }
  }
  if constexpr (LOCAL) {
    const long long block = (long long)seg * a.tiles + blockIdx.x;
    store_lanes<G>(a.local, block, w.lane, h);
    store_sums<G>(a, block, w.lane, sum);
  }
}

template <class G>
static cudaError_t forward(const Args& a, const Plan& p, bool save, cudaStream_t st) {
  if (p.cut) {
    {
      TraceScope tr("k_ssm_local", st);
      k_ssm<G, true><<<dim3(a.tiles, a.n_seg), 32, 0, st>>>(a, false);
    }
    const cudaError_t e = launch_ssm_carry<G, false>(a, st);
    if (e != cudaSuccess) return e;
  }
  // warps behind the segments look for sequences without rows
  const bool empty = a.final_state && (a.s.off || a.s.rows == 0);
  const int more = empty ? (a.s.n < 32 * 64 ? (a.s.n + 31) / 32 : 64) : 0;
  if (a.n_seg + more == 0) return cudaSuccess;
  TraceScope tr("k_ssm", st);
  k_ssm<G, false><<<dim3(a.tiles, a.n_seg + more), 32, 0, st>>>(a, save);
  return cudaGetLastError();
}

template <class E>
static cudaError_t forward_of(const Args& a, const Plan& p, bool save, cudaStream_t st) {
  switch (p.NS) {
    case 2: return forward<Cfg<E, 2, 4>>(a, p, save, st);
    case 4: return forward<Cfg<E, 4, 4>>(a, p, save, st);
    case 8: return forward<Cfg<E, 8, 2>>(a, p, save, st);
    default: return forward<Cfg<E, 16, 1>>(a, p, save, st);
  }
}

Args args_of(const SsmArgs& g, const Plan& p, const Work& k) {
  Args a{};
  a.x = g.x; a.delta = g.delta; a.z = g.z; a.B = g.B; a.C = g.C;
  a.ldx = g.ldx; a.ldd = g.ldd; a.ldz = g.ldz; a.ldb = g.ldb; a.ldc = g.ldc;
  a.A = g.A; a.D = g.D; a.bias = g.bias;
  a.s = seqs::make_seqs(g.off, g.n_seq, g.rows);
  a.d = g.d; a.groups = g.groups; a.N = g.N; a.per = g.d / g.groups; a.tpg = p.tpg;
  const int size = g.math == CFC_MATH_BF16 ? 2 : 4;
  a.vec_bc = g.N == 4 * p.NS &&
             (reinterpret_cast<uintptr_t>(g.B) | reinterpret_cast<uintptr_t>(g.C) | (uintptr_t)(g.ldb * size) |
              (uintptr_t)(g.ldc * size)) % 16 == 0;
  a.S = p.S; a.n_seg = p.n_seg; a.tiles = p.tiles; a.cps = p.cps;
  a.init = g.init;
  a.flags = reinterpret_cast<int*>(g.ws + k.flags);
  a.local = reinterpret_cast<float*>(g.ws + k.local);
  a.sdt = reinterpret_cast<float*>(g.ws + k.sdt);
  a.ckpt = reinterpret_cast<float*>(g.ws + k.ckpt);
  a.part = reinterpret_cast<float*>(g.ws + k.part);
  a.bc = reinterpret_cast<float*>(g.ws + k.bc);
  return a;
}

}  // namespace ssm

size_t ssm_workspace(long long rows, int n_seq, int d, int groups, int N, int save) {
  size_t most = 0;
  for (int packed = 0; packed < 2; ++packed) {
    const ssm::Plan p = ssm::make_plan(rows, n_seq, d, groups, N, packed != 0);
    const size_t n = ssm::make_work(p, rows, d, save != 0).total;
    if (n > most) most = n;
  }
  return most;
}

cudaError_t launch_ssm_forward(const SsmArgs& g, void* y, float* final_state, int save, cudaStream_t st) {
  const ssm::Plan p = ssm::make_plan(g.rows, g.n_seq, g.d, g.groups, g.N, g.off != nullptr);
  ssm::Args a = ssm::args_of(g, p, ssm::make_work(p, g.rows, g.d, save != 0));
  a.y = y;
  a.final_state = final_state;
  return g.math == CFC_MATH_BF16 ? ssm::forward_of<__nv_bfloat16>(a, p, save != 0, st)
                                 : ssm::forward_of<float>(a, p, save != 0, st);
}

}  // namespace cfc
