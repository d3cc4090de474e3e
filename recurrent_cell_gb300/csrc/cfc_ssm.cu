// cfc_ssm.cu -- the selective scan over whole sequences, forward (ssm_common.cuh
// has the formulas and the split).
//
//   k_ssm<., true>   the end state of each segment from its own rows, and its sum of dt
//   k_ssm_carry      the states between segments: h_s = local_s + exp(A sum dt) h_{s-1}
//   k_ssm<., false>  the scan itself
//
// The first two run only where segments cut sequences.  The third is bound by instructions and
// their latencies, not by memory: with 16 states a thread has 16 exponentials (4 cycles of a
// scheduler each) and 32 multiply-adds of pairs (2) a token, 122 instructions with the reads and the sums,
// and two such warps a scheduler issue 56 % of its cycles.  More warps have no room: at 128
// registers it took 235 us where it now takes 168, partial sums of y through shared memory instead of
// lane steps 182.  bfloat16, 16 states: 1 x 16384 rows x 2048 channels 109 + 7 + 167 us
// (281 the call), 8 x 2048 x 4096 (whole) 378 us; fp32 317 and 425 the calls.
#include "ssm_common.cuh"

namespace cfc {
namespace ssm {

// Two of each: the chunk that the states run through, and the next or the one before.
template <class G, bool LOCAL>
struct __align__(16) FwdTiles {
  float dt[2][kT][G::CW], dx[2][kT][G::CW];  // dt, dt x
  float B[2][kT][G::NP];
  float C[LOCAL ? 1 : 2][kT][G::NP];
  float y[LOCAL ? 1 : 2][kT][G::CW];         // C . h
  uint4 raw[2][G::P][32], rawB[LOCAL ? 1 : 2][G::BL][32];    // x, delta; B, C: the chunk to come as the lanes take it
};

// What a token reads of the tiles.
template <class G, bool LOCAL>
struct Operands {
  F2 dt[G::CPAIRS], dx[G::CPAIRS], b[G::SPAIRS], c[G::SPAIRS];
  __device__ __forceinline__ void read(const FwdTiles<G, LOCAL>& sm, const Tile<G>& w, int k, int t) {
    get_channels<G>(sm.dt[k][t], w.cl, dt);
    get_channels<G>(sm.dx[k][t], w.cl, dx);
    get_states<G>(sm.B[k][t], w.sl, b);
    if constexpr (!LOCAL) get_states<G>(sm.C[k][t], w.sl, c);
  }
};

// One token: the states, and C . h.
template <class G, bool LOCAL>
__device__ __forceinline__ void token(FwdTiles<G, LOCAL>& sm, const Tile<G>& w, int k, int t, const Operands<G, LOCAL>& o,
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
    float f[G::CPL];
    if constexpr (G::CPL > 1) {
#pragma unroll
      for (int i = 0; i < G::CPAIRS; ++i) split(y[i], f[2 * i], f[2 * i + 1]);
    } else {
      f[0] = sum2(y[0]);
    }
    const float v = over_states<G::CPL>(f, w.lane);
    if (w.sl < G::CPL) sm.y[k][t][w.cl * G::CPL + w.sl] = v;
  }
}

// A block is two warps: one runs the states through a chunk's tokens while the other
// stages the next chunk (dt, dt x, B and C as floats) and finishes the one before (D x,
// the gate, the store).  Alone, a warp's phases follow one another's latencies; there
// are too few tiles of channels for more warps to fill them.
template <class G, bool LOCAL>
__global__ void __launch_bounds__(64, kResident) k_ssm(Args a, bool save) {
  using E = typename G::E;
  using U = Pairs<E, G::VN>;
  constexpr int P = G::P, VN = G::VN, VP = VN / 2;
  __shared__ FwdTiles<G, LOCAL> sm;
  const Tile<G> w(a, blockIdx.x);
  const int seg = blockIdx.y;
  const bool helper = helper_of_two();

  if (!LOCAL && seg >= a.n_seg) {            // the states after sequences without rows
    F2 h[G::PAIRS];
    const int step = (gridDim.y - a.n_seg) * 64;
    for (long long i0 = (long long)(seg - a.n_seg) * 64 + (helper ? 32 : 0); i0 < a.s.n; i0 += step) {
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
  if (r0 >= r1) {                            // rows behind the last sequence
    if (LOCAL && blockIdx.x == 0 && threadIdx.x == 0) a.flags[seg] = 0;
    return;
  }
  Where q = seqs::find(a.s, LOCAL ? r1 - 1 : r0);
  long long row = r0;
  if constexpr (LOCAL) {
    const bool cut = q.end > r1, starts = q.begin >= r0;
    if (blockIdx.x == 0 && threadIdx.x == 0) a.flags[seg] = (cut ? kCut : 0) | (starts ? kStarts : 0);
    if (!cut) return;
    if (starts) row = q.begin;
  }
  const int chunks = (int)((r1 - row + kT - 1) / kT);

  if (helper) {
    F2 bias[VP], D[VP];
    load_pairs<G>(w, a.bias, bias);
    load_pairs<G>(w, LOCAL ? nullptr : a.D, D);
    auto count = [&](int chunk) {
      const long long at = row + (long long)chunk * kT;
      return r1 - at < kT ? (int)(r1 - at) : kT;
    };
    auto vector = [&](const void* p, long long ld, long long r) { return static_cast<const E*>(p) + r * ld + w.c0 + w.col(); };
    auto fetch = [&](int chunk) {
      const long long at = row + (long long)chunk * kT;
      const int n = count(chunk);
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const bool in = w.row(k) < n && w.col() < w.cols;
        const long long r = in ? at + w.row(k) : at;
        copy16(&sm.raw[0][k][w.lane], in ? vector(a.x, a.ldx, r) : a.x, in);
        copy16(&sm.raw[1][k][w.lane], in ? vector(a.delta, a.ldd, r) : a.delta, in);
      }
      if (a.vec_bc)
#pragma unroll
        for (int k = 0; k < G::BL; ++k) {
          const int i = k * 32 + w.lane, r = i / G::BV;
          const bool in = r < n;
          const long long off = w.g * a.N + i % G::BV * VN;
          copy16(&sm.rawB[0][k][w.lane], in ? static_cast<const E*>(a.B) + (at + r) * a.ldb + off : a.B, in);
          if constexpr (!LOCAL)
            copy16(&sm.rawB[1][k][w.lane], in ? static_cast<const E*>(a.C) + (at + r) * a.ldc + off : a.C, in);
        }
      copies_end();
    };
    auto stage = [&](int chunk) {
      const long long at = row + (long long)chunk * kT;
      const int n = count(chunk), to = chunk & 1;
      copies_wait<0>();
#pragma unroll
      for (int k = 0; k < P; ++k) {
        F2 x[VP], dt[VP];
        U::get(x, sm.raw[0][k][w.lane]);
        U::get(dt, sm.raw[1][k][w.lane]);
#pragma unroll
        for (int e = 0; e < VP; ++e) {
          dt[e] = softplus2(add2(dt[e], bias[e]));
          x[e] = mul2(x[e], dt[e]);
        }
        if (w.row(k) < kT) {
          put_pairs(&sm.dt[to][w.row(k)][w.col()], dt);
          put_pairs(&sm.dx[to][w.row(k)][w.col()], x);
        }
      }
      Rows<G> bv, cv;
      if (a.vec_bc)
#pragma unroll
        for (int k = 0; k < G::BL; ++k) {
          bv.v[k] = sm.rawB[0][k][w.lane];
          if constexpr (!LOCAL) cv.v[k] = sm.rawB[1][k][w.lane];
        }
      bv.stage(a, w, a.B, a.ldb, at, n, sm.B[to][0]);
      if constexpr (!LOCAL) cv.stage(a, w, a.C, a.ldc, at, n, sm.C[to][0]);
    };
    uint4 xv[P], zv[P];
    auto reload = [&](int chunk) {             // x and z of a chunk that is about to be finished
      const long long at = row + (long long)chunk * kT;
      load_raw<G>(w, a.x, a.ldx, at, count(chunk), xv);
      if (a.z) load_raw<G>(w, a.z, a.ldz, at, count(chunk), zv);
    };
    auto finish = [&](int chunk) {
      const long long at = row + (long long)chunk * kT;
      const int n = count(chunk);
#pragma unroll
      for (int k = 0; k < P; ++k) {
        use_here(xv[k]);
        if (a.z) use_here(zv[k]);
      }
#pragma unroll
      for (int k = 0; k < P; ++k)
        if (w.row(k) < n && w.col() < w.cols) {
          F2 y[VP], x[VP];
          U::get(x, xv[k]);
          get_pairs(&sm.y[chunk & 1][w.row(k)][w.col()], y);
#pragma unroll
          for (int e = 0; e < VP; ++e) y[e] = fma2(D[e], x[e], y[e]);
          if (a.z) {
            // (fp32 too: the exponent's rounding is |z| 6e-8 of the gate, below what C . h has gathered by then, where
            // the convolution, whose sums are a few terms, puts it right)
            U::get(x, zv[k]);
#pragma unroll
            for (int e = 0; e < VP; ++e) y[e] = mul2(y[e], mul2(x[e], sigmoid2(x[e])));
          }
          __stcs(reinterpret_cast<uint4*>(static_cast<E*>(a.y) + (at + w.row(k)) * a.d + w.c0 + w.col()), U::make(y));
        }
    };
    fetch(0);
    stage(0);
    if (chunks > 1) fetch(1);
    for (int i = 0; i < chunks; ++i) {
      __syncthreads();                         // chunk i is staged, chunk i - 1 has been run through
      if (!LOCAL && i > 0) reload(i - 1);
      if (i + 1 < chunks) stage(i + 1);
      if (i + 2 < chunks) fetch(i + 2);
      if (!LOCAL && i > 0) finish(i - 1);
    }
    __syncthreads();
    if constexpr (!LOCAL) {
      reload(chunks - 1);
      finish(chunks - 1);
    }
    return;
  }

  F2 h[G::PAIRS], A2[G::PAIRS], sum[G::CPAIRS] = {};
  load_A<G>(a, w, A2);
  if (LOCAL || q.begin == r0) {
#pragma unroll
    for (int p = 0; p < G::PAIRS; ++p) h[p] = 0;
  } else {
    load_lanes<G>(a.local, (long long)(seg - 1) * a.tiles + blockIdx.x, w.lane, h);
  }
  for (int chunk = 0; chunk < chunks; ++chunk, row += kT) {
    const int n = r1 - row < kT ? (int)(r1 - row) : kT, k = chunk & 1;
    if (!LOCAL && save) store_lanes<G>(a.ckpt, ((long long)seg * a.cps + chunk) * a.tiles + blockIdx.x, w.lane, h);
    __syncthreads();
    if (n == kT && q.begin < row && q.end > row + kT) {      // inside one sequence: no state comes or goes
      Operands<G, LOCAL> now, next;
      now.read(sm, w, k, 0);
#pragma unroll
      for (int t = 0; t < kT; ++t) {
        next.read(sm, w, k, t + 1 < kT ? t + 1 : t);
        token<G, LOCAL>(sm, w, k, t, now, A2, h, sum);
        now = next;
      }
    } else {
      for (int t = 0; t < n;) {
        if (row + t == q.begin) load_state<G>(a, w, a.init, q.i, h);
        const int m = q.end - row < n ? (int)(q.end - row) : n;
        for (; t < m; ++t) {
          Operands<G, LOCAL> now;
          now.read(sm, w, k, t);
          token<G, LOCAL>(sm, w, k, t, now, A2, h, sum);
        }
        if (!LOCAL && row + t == q.end) {
          if (a.final_state) store_state<G>(a, w, a.final_state, q.i, h);
          if (row + t < a.s.rows) q = seqs::find(a.s, row + t);
        }
      }
    }
  }
  __syncthreads();
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
      k_ssm<G, true><<<dim3(a.tiles, a.n_seg), 64, 0, st>>>(a, false);
    }
    const cudaError_t e = launch_ssm_carry<G, false>(a, st);
    if (e != cudaSuccess) return e;
  }
  // warps behind the segments look for sequences without rows
  const bool empty = a.final_state && (a.s.off || a.s.rows == 0);
  const int more = empty ? (a.s.n < 32 * 64 ? (a.s.n + 31) / 32 : 64) : 0;
  if (a.n_seg + more == 0) return cudaSuccess;
  TraceScope tr("k_ssm", st);
  k_ssm<G, false><<<dim3(a.tiles, a.n_seg + more), 64, 0, st>>>(a, save);
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
