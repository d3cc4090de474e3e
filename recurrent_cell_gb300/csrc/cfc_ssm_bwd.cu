// cfc_ssm_bwd.cu -- the selective scan's backward (ssm_common.cuh has the formulas of
// the forward and the split of rows and channels).
//
// With g = grad_y silu(z), a_t = exp(dt_t A), h_t the state after token t and dh_t
// the gradient that reaches it,
//   dh_t  = C_t g_t + a_{t+1} dh_{t+1},    e_t = dh_t a_t h_{t-1}   (per channel and state)
//   dx    = dt sum_n dh B + D g            ddt = sum_n e A + x sum_n dh B
//   dA    = sum_t dt e                     ddelta = ddt sigmoid(delta + bias)
//   dB    = sum_c dt x dh                  dC = sum_c g h
//   dz    = grad_y (C . h + D x) silu'(z)  dD = sum_t g x,  dbias = sum_t ddelta
// A chunk starts from the state that the forward saved before it.  A first sweep runs
// it forward and puts every state into tensor memory, which here is nothing but memory: 32 KB
// a tile that the other warps' traffic through shared memory, as scarce as
// instructions in this kernel, does not see.  The second sweep goes back.  The two exponentials
// and some fifteen multiply-adds a state are the bound, not memory, and with tensor memory full
// at eight tiles an SM there are only two token warps a scheduler to hide them behind.  So
// a second warp a tile takes off the first what is not the recurrence (staging, outputs), the
// registers are split unevenly between the two, and a token's sums over the lanes are taken beside
// the next one's arithmetic.  16384 rows x 4096 channels x 16 states, bfloat16: 1261 us; with one
// warp that does everything 1360; helpers without the delayed sums 1311; registers 152 | 104,
// 168 | 88, 184 | 72: 1343, 1314, 1269; the second sweep unrolled 1, 3, 5, 15 times: 1470,
// 1261, 1327, 1442 (its code leaves the instruction cache); states read a token ahead: 1312.  The
// compiler still spills there: 192 bytes stored and 224 loaded a thread (180 and 240 with 64 states).  32 and
// 64 states, whose tiles are 16 and 8 channels wide: 2.6 and 8.4 ms; fp32 1314 us.
//
// Sums over a channel's states and over a tile's channels are taken by lane steps that
// halve the values as they go: 12 values over 4 lanes in 9 steps, 8 over 8 in 7.  Four
// tiles of a block add their dB and dC in shared memory, so that what goes to the
// workspace is a sum over 128 channels; k_ssm_bc adds those.  dA is kept in shared memory, dD
// and dbias in registers over a segment; reduce_axis0 adds the segments.
#include "ssm_common.cuh"
#include "tc_common.cuh"

namespace cfc {
namespace ssm {

constexpr int kBwdWarps = 4;

// Of a tile of channels; two of each: the chunk that the tokens run through, and the one to
// come or the one before.
template <class G>
struct __align__(16) BwdTiles {
  float dt[2][kT][G::CW], dx[2][kT][G::CW], g[2][kT][G::CW];         // dt, dt x, g; then sum e A, sum dh B, C . h
  float bc[2][kT][2 * G::NP];                                // dB, dC of the tile
  F2 gA[G::PAIRS][32];                                       // dA of the chunks so far
  uint4 raw[4][G::P][32];                                    // the chunk to come: x, delta, z, grad_y as the lanes take them
};
// Of a block, whose tiles are of one group.
template <class G>
struct __align__(16) BwdBlock {
  BwdTiles<G> tile[kBwdWarps];
  float B[2][kT][G::NP], C[2][kT][G::NP];
  uint4 rawB[2][(kT * G::BV + 127) / 128][128];
};

// A thread's states to and from tensor memory, at `at` of its warp's part.
template <int N>
__device__ __forceinline__ void tmem_put(uint32_t at, const F2 (&h)[N]) {
  static_assert(N == 4 || N == 8, "8 or 16 columns");
  uint32_t r[2 * N];
#pragma unroll
  for (int p = 0; p < N; ++p) {
    float a, b;
    split(h[p], a, b);
    r[2 * p] = __float_as_uint(a);
    r[2 * p + 1] = __float_as_uint(b);
  }
  if constexpr (N == 8)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                 "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]));
  else
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]));
}
template <int N>
__device__ __forceinline__ void tmem_get(uint32_t at, F2 (&h)[N]) {
  // (no memory clobber: it takes part in nothing but tensor memory, and volatile statements keep their order)
  uint32_t r[2 * N];
  if constexpr (N == 8)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at));
  else
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(at));
#pragma unroll
  for (int p = 0; p < N; ++p) h[p] = pack(__uint_as_float(r[2 * p]), __uint_as_float(r[2 * p + 1]));
}
__device__ __forceinline__ void tmem_put_wait() { asm volatile("tcgen05.wait::st.sync.aligned;"); }

// Sums over the 8 channel lanes of v[N], N = 4, 8, 16 or 32: lane cl has those of
// values cl + 8 k, in v[k] (N = 4: value cl % 4's).
template <int N>
__device__ __forceinline__ void over_channels(float (&v)[N], int lane) {
  if constexpr (N == 4) {
    fold<4>(v, lane, 4);
    float u[2] = {v[0], v[1]};
    fold<2>(u, lane, 8);
    v[0] = all<1>(u[0], 16);
  } else {
    // value 8 k + 4 b2 + 2 b1 + b0 after folding by b0, b1, b2
    fold<N>(v, lane, 4);
    float u[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) u[i] = v[i];
    fold<N / 2>(u, lane, 8);
    float t[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i) t[i] = u[i];
    fold<N / 4>(t, lane, 16);
#pragma unroll
    for (int i = 0; i < N / 8; ++i) v[i] = t[i];
  }
}

// What a segment's own rows send to the state before it, and its sum of dt: for the
// segments whose first row continues a sequence.  Two warps as in the forward (16384 x 2048 channels
// x 16 states: 127 us, one warp that does both 174).
template <class G>
struct __align__(16) LocalTiles {
  float dt[2][kT][G::CW], g[2][kT][G::CW], C[2][kT][G::NP];
  uint4 raw[3][G::P][32], rawC[G::BL][32];                   // delta, z, grad_y; C: the chunk to come
};
template <class G>
__global__ void __launch_bounds__(64, kResident) k_ssm_local_bwd(Args a) {
  using E = typename G::E;
  using U = Pairs<E, G::VN>;
  constexpr int VN = G::VN, VP = VN / 2, P = G::P;
  __shared__ LocalTiles<G> sm;
  const Tile<G> w(a, blockIdx.x);
  const int seg = blockIdx.y;
  const bool helper = helper_of_two();
  a.s = seqs::trim(a.s);
  const long long r0 = seg * a.S, r1 = a.s.rows - r0 < a.S ? a.s.rows : r0 + a.S;
  if (r0 >= r1) {                            // rows behind the last sequence
    if (blockIdx.x == 0 && threadIdx.x == 0) a.flags[seg] = 0;
    return;
  }
  const Where q = seqs::find(a.s, r0);
  const bool cut = q.begin < r0, ends = q.end <= r1;
  if (blockIdx.x == 0 && threadIdx.x == 0) a.flags[seg] = (cut ? kCut : 0) | (ends ? kStarts : 0);
  if (!cut) return;
  const long long last = ends ? q.end : r1;
  const int chunks = (int)((last - r0 + kT - 1) / kT);
  auto count = [&](int chunk) { return last - (r0 + (long long)chunk * kT) < kT ? (int)(last - (r0 + (long long)chunk * kT)) : kT; };

  if (helper) {
    F2 bias[VP];
    load_pairs<G>(w, a.bias, bias);
    auto vector = [&](const void* p, long long ld, long long r) { return static_cast<const E*>(p) + r * ld + w.c0 + w.col(); };
    auto fetch = [&](int chunk) {
      const long long at = r0 + (long long)chunk * kT;
      const int n = count(chunk);
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const bool in = w.row(k) < n && w.col() < w.cols;
        const long long r = in ? at + w.row(k) : at;
        copy16(&sm.raw[0][k][w.lane], in ? vector(a.delta, a.ldd, r) : a.delta, in);
        if (a.z) copy16(&sm.raw[1][k][w.lane], in ? vector(a.z, a.ldz, r) : a.z, in);
        copy16(&sm.raw[2][k][w.lane], in ? vector(a.grad_y, a.d, r) : a.grad_y, in);
      }
      if (a.vec_bc)
#pragma unroll
        for (int k = 0; k < G::BL; ++k) {
          const int i = k * 32 + w.lane, r = i / G::BV;
          const bool in = r < n;
          copy16(&sm.rawC[k][w.lane], in ? static_cast<const E*>(a.C) + (at + r) * a.ldc + w.g * a.N + i % G::BV * VN : a.C, in);
        }
      copies_end();
    };
    auto stage = [&](int chunk) {
      const int to = chunk & 1;
      copies_wait<0>();
#pragma unroll
      for (int k = 0; k < P; ++k) {
        F2 f[VP], t[VP], u[VP];
        U::get(t, sm.raw[0][k][w.lane]);
#pragma unroll
        for (int e = 0; e < VP; ++e) t[e] = softplus2(add2(t[e], bias[e]));
        U::get(f, sm.raw[2][k][w.lane]);
        if (a.z) {
          U::get(u, sm.raw[1][k][w.lane]);
#pragma unroll
          for (int e = 0; e < VP; ++e) f[e] = mul2(f[e], mul2(u[e], sigmoid2(u[e])));
        }
        if (w.row(k) < kT) {
          put_pairs(&sm.dt[to][w.row(k)][w.col()], t);
          put_pairs(&sm.g[to][w.row(k)][w.col()], f);
        }
      }
      Rows<G> cv;
      if (a.vec_bc)
#pragma unroll
        for (int k = 0; k < G::BL; ++k) cv.v[k] = sm.rawC[k][w.lane];
      cv.stage(a, w, a.C, a.ldc, r0 + (long long)chunk * kT, count(chunk), sm.C[to][0]);
    };
    fetch(chunks - 1);
    stage(chunks - 1);
    if (chunks > 1) fetch(chunks - 2);
    for (int i = chunks - 1; i >= 0; --i) {
      __syncthreads();                         // chunk i is staged, chunk i + 1 has been run through
      if (i > 0) stage(i - 1);
      if (i > 1) fetch(i - 2);
    }
    return;
  }

  F2 A2[G::PAIRS], dh[G::PAIRS], sum[G::CPAIRS] = {};
  load_A<G>(a, w, A2);
  load_state<G>(a, w, ends ? a.grad_final : nullptr, q.i, dh);
  for (int chunk = chunks - 1; chunk >= 0; --chunk) {
    const int n = count(chunk), k = chunk & 1;
    __syncthreads();
    auto token = [&](int t) {
      F2 dt[G::CPAIRS], g[G::CPAIRS], c[G::SPAIRS];
      get_channels<G>(sm.dt[k][t], w.cl, dt);
      get_channels<G>(sm.g[k][t], w.cl, g);
      get_states<G>(sm.C[k][t], w.sl, c);
#pragma unroll
      for (int p = 0; p < G::PAIRS; ++p) {
        const int i = cpair<G>(p), j = spair<G>(p);
        dh[p] = mul2(decay2(dt[i], A2[p]), fma2(c[j], g[i], dh[p]));
      }
#pragma unroll
      for (int i = 0; i < G::CPAIRS; ++i) sum[i] = add2(sum[i], dt[i]);
    };
    if (n == kT) {
#pragma unroll
      for (int t = kT - 1; t >= 0; --t) token(t);
    } else {
#pragma unroll 1
      for (int t = n - 1; t >= 0; --t) token(t);
    }
  }
  const long long block = (long long)seg * a.tiles + blockIdx.x;
  store_lanes<G>(a.local, block, w.lane, dh);
  store_sums<G>(a, block, w.lane, sum);
}

// What a token reads of the tiles.
template <class G, bool BACK>
struct Token {
  F2 dt[G::CPAIRS], dx[G::CPAIRS], b[G::SPAIRS], g[G::CPAIRS], c[G::SPAIRS];
  __device__ __forceinline__ void read(const BwdBlock<G>& all, const BwdTiles<G>& sm, const Tile<G>& w, int k, int t) {
    get_channels<G>(sm.dt[k][t], w.cl, dt);
    get_channels<G>(sm.dx[k][t], w.cl, dx);
    get_states<G>(all.B[k][t], w.sl, b);
    if constexpr (BACK) {
      get_channels<G>(sm.g[k][t], w.cl, g);
      get_states<G>(all.C[k][t], w.sl, c);
    }
  }
  __device__ __forceinline__ void forward(const F2 (&A2)[G::PAIRS], F2 (&h)[G::PAIRS]) const {
#pragma unroll
    for (int p = 0; p < G::PAIRS; ++p)
      h[p] = fma2(decay2(dt[cpair<G>(p)], A2[p]), h[p], mul2(dx[cpair<G>(p)], b[spair<G>(p)]));
  }
};

// A lane's part of the sums of a token: over its states for each of its channels, and over
// its channels for each of its states.
template <class G>
struct Sums {
  F2 s1[G::CPAIRS], s2[G::CPAIRS], y[G::CPAIRS];
  float bc[2 * G::NS];
  // A token backward, h being the state before it; dh goes on to the token before it.
  __device__ __forceinline__ void token(const Token<G, true>& k, const F2 (&h)[G::PAIRS], const F2 (&A2)[G::PAIRS], F2 (&dh)[G::PAIRS],
                                        F2 (&gA)[G::PAIRS]) {
    F2 db[G::SPAIRS], dc[G::SPAIRS];
#pragma unroll
    for (int p = 0; p < G::PAIRS; ++p) {
      const int i = cpair<G>(p), j = spair<G>(p);
      const bool first_i = G::CPL > 1 ? j == 0 : p == 0, first_j = G::CPL > 1 ? i == 0 : true;
      const F2 e = decay2(k.dt[i], A2[p]);
      const F2 ah = mul2(e, h[p]), now = fma2(k.dx[i], k.b[j], ah), d = fma2(k.c[j], k.g[i], dh[p]), q = mul2(d, ah);
      y[i] = first_i ? mul2(k.c[j], now) : fma2(k.c[j], now, y[i]);
      s1[i] = first_i ? mul2(d, k.b[j]) : fma2(d, k.b[j], s1[i]);
      s2[i] = first_i ? mul2(q, A2[p]) : fma2(q, A2[p], s2[i]);
      gA[p] = fma2(q, k.dt[i], gA[p]);
      db[j] = first_j ? mul2(d, k.dx[i]) : fma2(d, k.dx[i], db[j]);
      dc[j] = first_j ? mul2(k.g[i], now) : fma2(k.g[i], now, dc[j]);
      dh[p] = mul2(e, d);
    }
    if constexpr (G::CPL > 1) {
#pragma unroll
      for (int j = 0; j < G::NS; ++j) {
        bc[j] = sum2(db[j]);
        bc[G::NS + j] = sum2(dc[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < G::NS / 2; ++j) {
        split(db[j], bc[2 * j], bc[2 * j + 1]);
        split(dc[j], bc[G::NS + 2 * j], bc[G::NS + 2 * j + 1]);
      }
    }
  }
  // The sums over the lanes, into the tiles in place of token t's own values.
  __device__ __forceinline__ void out(BwdTiles<G>& sm, const Tile<G>& w, int at, int t) {
    constexpr int CPL = G::CPL, NS = G::NS, NP = G::NP;
    float f1[CPL], f2[CPL], f3[CPL];
    if constexpr (CPL > 1) {
#pragma unroll
      for (int i = 0; i < CPL / 2; ++i) {
        split(s1[i], f1[2 * i], f1[2 * i + 1]);
        split(s2[i], f2[2 * i], f2[2 * i + 1]);
        split(y[i], f3[2 * i], f3[2 * i + 1]);
      }
    } else {
      f1[0] = sum2(s1[0]);
      f2[0] = sum2(s2[0]);
      f3[0] = sum2(y[0]);
    }
    const float o1 = over_states<CPL>(f1, w.lane), o2 = over_states<CPL>(f2, w.lane), o3 = over_states<CPL>(f3, w.lane);
    over_channels<2 * NS>(bc, w.lane);
    __syncwarp();                              // every lane has read the token's own values
    if (w.sl < CPL) {
      sm.dx[at][t][w.cl * CPL + w.sl] = o1;
      sm.dt[at][t][w.cl * CPL + w.sl] = o2 * kLn2;
      sm.g[at][t][w.cl * CPL + w.sl] = o3;
    }
    if constexpr (NS == 2) {
      if (w.cl < 4) sm.bc[at][t][(w.cl >> 1) * NP + w.sl * NS + (w.cl & 1)] = bc[0];
    } else {
#pragma unroll
      for (int i = 0; i < 2 * NS / 8; ++i) {
        const int v = i * 8 + w.cl;
        sm.bc[at][t][v / NS * NP + w.sl * NS + v % NS] = bc[i];
      }
    }
  }
};

// Registers of a thread: what the block is launched with, and what it comes to for the warps
// that run the tokens and those that help.
constexpr int kLaunchRegs = 128, kTokenRegs = 176, kHelperRegs = 80;
static_assert(kTokenRegs + kHelperRegs == 2 * kLaunchRegs, "the split draws on what the launch has");

// A block is four tiles, each with two warps: one runs the tokens of a chunk forward and
// back, the other stages the chunk to come and finishes the one behind (the outputs
// channel by channel, the block's sum of dB and dC).  They meet once a chunk.
template <class G>
__global__ void __launch_bounds__(64 * kBwdWarps, 2) k_ssm_bwd(Args a) {
  using E = typename G::E;
  using U = Pairs<E, G::VN>;
  constexpr int VN = G::VN, VP = VN / 2, NP = G::NP, PAIRS = G::PAIRS, P = G::P;
  constexpr uint32_t kColumns = 2 * PAIRS * kT;              // of tensor memory
  extern __shared__ __align__(16) unsigned char raw[];
  __shared__ uint32_t tmem;
  BwdBlock<G>& all = *reinterpret_cast<BwdBlock<G>*>(raw);
  const int warp = threadIdx.x >> 5, pair = warp & (kBwdWarps - 1);
  const bool helper = warp >= kBwdWarps;
  BwdTiles<G>& sm = all.tile[pair];
  const int quads = (a.tpg + kBwdWarps - 1) / kBwdWarps;     // blocks of a group
  const int group = blockIdx.x / quads, at = blockIdx.x % quads * kBwdWarps + pair;
  const bool on = at < a.tpg;                                // else warps without channels, there for the barriers
  const int tile = group * a.tpg + (on ? at : a.tpg - 1);
  const Tile<G> w(a, tile);
  const int seg = blockIdx.y;

  if (seg >= a.n_seg) {                        // sequences without rows: the gradient passes through
    F2 h[PAIRS];
    const int step = (gridDim.y - a.n_seg) * 32;
    for (long long i0 = (long long)(seg - a.n_seg) * 32; on && !helper && i0 < a.s.n; i0 += step) {
      long long begin = 0, end = 1;
      if (i0 + w.lane < a.s.n) seqs::range_of(a.s, (int)(i0 + w.lane), &begin, &end);
      unsigned none = __ballot_sync(0xffffffffu, begin >= end);
      while (none) {
        const long long i = i0 + __ffs(none) - 1;
        none &= none - 1;
        load_state<G>(a, w, a.grad_final, i, h);
        store_state<G>(a, w, a.grad_init, i, h);
      }
    }
    return;
  }

  const long long all_rows = a.s.rows;
  a.s = seqs::trim(a.s);
  const long long r0 = seg * a.S, r1 = a.s.rows - r0 < a.S ? a.s.rows : r0 + a.S;
  float* part = a.part + (long long)seg * a.d * (a.N + 2);   // the segment's dA, dD, dbias: [d, N | d | d]
  if (r0 >= r1) {                              // rows behind the last sequence: sums of nothing
    const int n = on && !helper ? w.cols : 0;
    for (int i = w.lane; i < n * a.N; i += 32) part[(long long)w.c0 * a.N + i] = 0.f;
    for (int i = w.lane; i < n; i += 32) part[(long long)a.d * a.N + w.c0 + i] = part[(long long)a.d * (a.N + 1) + w.c0 + i] = 0.f;
    return;
  }

  if (warp == 0) tc::tmem_alloc(&tmem, kColumns);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const int chunks = (int)((r1 - r0 + kT - 1) / kT);
  auto row_of = [&](int chunk) { return r0 + (long long)chunk * kT; };
  auto count = [&](int chunk) { return r1 - row_of(chunk) < kT ? (int)(r1 - row_of(chunk)) : kT; };

  if (helper) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kHelperRegs));
    const int ht = threadIdx.x - 32 * kBwdWarps;             // of the helpers' 128 threads
    F2 bias[VP], D[VP], gD[VP] = {}, gb[VP] = {};
    load_pairs<G>(w, a.bias, bias);
    load_pairs<G>(w, a.D, D);
    auto vector = [&](const void* p, long long ld, long long r) {
      return static_cast<const E*>(p) + r * ld + w.c0 + w.col();
    };
    auto fetch = [&](int chunk) {
      const long long row = row_of(chunk);
      const int n = count(chunk);
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const bool in = w.row(k) < n && w.col() < w.cols;
        const long long r = in ? row + w.row(k) : 0;
        copy16(&sm.raw[0][k][w.lane], in ? vector(a.x, a.ldx, r) : a.x, in);
        copy16(&sm.raw[1][k][w.lane], in ? vector(a.delta, a.ldd, r) : a.delta, in);
        if (a.z) copy16(&sm.raw[2][k][w.lane], in ? vector(a.z, a.ldz, r) : a.z, in);
        copy16(&sm.raw[3][k][w.lane], in ? vector(a.grad_y, a.d, r) : a.grad_y, in);
      }
      if (a.vec_bc)
        for (int i = ht, k = 0; i < kT * G::BV; i += 128, ++k) {
          const int r = i / G::BV;
          const bool in = r < n;
          const long long off = w.g * a.N + i % G::BV * VN;
          copy16(&all.rawB[0][k][ht], in ? static_cast<const E*>(a.B) + (row + r) * a.ldb + off : a.B, in);
          copy16(&all.rawB[1][k][ht], in ? static_cast<const E*>(a.C) + (row + r) * a.ldc + off : a.C, in);
        }
      copies_end();
    };
    // dt, dt x, g, B and C of a chunk's tokens, from what fetch() copied
    auto stage = [&](int chunk) {
      const int to = chunk & 1;
      copies_wait<0>();
#pragma unroll
      for (int k = 0; k < P; ++k) {
        F2 x[VP], dt[VP], z[VP], g[VP];
        U::get(x, sm.raw[0][k][w.lane]);
        U::get(dt, sm.raw[1][k][w.lane]);
        U::get(g, sm.raw[3][k][w.lane]);
        if (a.z) {
          U::get(z, sm.raw[2][k][w.lane]);
#pragma unroll
          for (int e = 0; e < VP; ++e) g[e] = mul2(g[e], mul2(z[e], sigmoid2(z[e])));
        }
#pragma unroll
        for (int e = 0; e < VP; ++e) {
          dt[e] = softplus2(add2(dt[e], bias[e]));
          x[e] = mul2(x[e], dt[e]);
        }
        if (w.row(k) < kT) {
          put_pairs(&sm.dt[to][w.row(k)][w.col()], dt);
          put_pairs(&sm.dx[to][w.row(k)][w.col()], x);
          put_pairs(&sm.g[to][w.row(k)][w.col()], g);
        }
      }
      if (a.vec_bc) {
        for (int i = ht, k = 0; i < kT * G::BV; i += 128, ++k) {
          F2 f[VP];
          U::get(f, all.rawB[0][k][ht]);
          put_pairs(all.B[to][0] + i * VN, f);
          U::get(f, all.rawB[1][k][ht]);
          put_pairs(all.C[to][0] + i * VN, f);
        }
      } else {
        const long long row = row_of(chunk);
        const int n = count(chunk);
        for (int i = ht; i < kT * NP; i += 128) {
          const int r = i / NP, s = i % NP;
          const bool in = r < n && s < a.N;
          all.B[to][0][i] = in ? rows::load1(static_cast<const E*>(a.B) + (row + r) * a.ldb + w.g * a.N + s) : 0.f;
          all.C[to][0][i] = in ? rows::load1(static_cast<const E*>(a.C) + (row + r) * a.ldc + w.g * a.N + s) : 0.f;
        }
      }
    };
    // the gradients of a chunk that has been run through, channel by channel
    auto finish = [&](int chunk) {
      const long long row = row_of(chunk);
      const int n = count(chunk), from = chunk & 1;
      F2 cD[VP] = {}, cb[VP] = {};             // dD and dbias of the chunk
#pragma unroll
      for (int k = 0; k < P; ++k)
        if (w.row(k) < n && w.col() < w.cols && on) {
          const long long r = row + w.row(k);
          auto out = [&](void* p, const F2 (&f)[VP]) {
            __stcs(reinterpret_cast<uint4*>(static_cast<E*>(p) + r * a.d + w.c0 + w.col()), U::make(f));
          };
          const uint4 xv = load_here(vector(a.x, a.ldx, r)), gv = load_here(vector(a.grad_y, a.d, r)),
                      dv = load_here(vector(a.delta, a.ldd, r)), zv = load_here(vector(a.z, a.ldz, r), a.z != nullptr);
          F2 x[VP], g[VP], f[VP], s1[VP], u[VP];
          U::get(x, xv);
          U::get(g, gv);
          if (a.z) {
            F2 z[VP];
            U::get(z, zv);
            get_pairs(&sm.g[from][w.row(k)][w.col()], u);
#pragma unroll
            for (int e = 0; e < VP; ++e) {
              // silu'(z) = s (1 + z (1 - s)) = s + z s (1 - s)
              const F2 s = sigmoid2(z[e]), zs = mul2(z[e], s);
              u[e] = mul2(fma2(D[e], x[e], u[e]), g[e]);
              u[e] = mul2(u[e], fma2(zs, fma2(s, twice(-1.f), twice(1.f)), s));
              g[e] = mul2(g[e], zs);
            }
            out(a.grad_z, u);
          }
          get_pairs(&sm.dx[from][w.row(k)][w.col()], s1);
          get_pairs(&sm.dt[from][w.row(k)][w.col()], f);
          U::get(u, dv);
#pragma unroll
          for (int e = 0; e < VP; ++e) {
            F2 en;
            const F2 v = add2(u[e], bias[e]), dt = softplus2(v, &en);
            float va, vb, ea, eb;              // sigmoid(v) = 1 / (1 + e), or e / (1 + e) below zero
            split(v, va, vb);
            split(en, ea, eb);
            const F2 sig = pack((va >= 0.f ? 1.f : ea) * rcp(1.f + ea), (vb >= 0.f ? 1.f : eb) * rcp(1.f + eb));
            cD[e] = fma2(g[e], x[e], cD[e]);
            f[e] = mul2(fma2(x[e], s1[e], f[e]), sig);
            cb[e] = add2(cb[e], f[e]);
            g[e] = fma2(dt, s1[e], mul2(D[e], g[e]));
          }
          out(a.grad_delta, f);
          out(a.grad_x, g);
        }
#pragma unroll
      for (int e = 0; e < VP; ++e) {
        gD[e] = add2(gD[e], cD[e]);
        gb[e] = add2(gb[e], cb[e]);
      }
      // the block's sum of dB and dC
      const int warps = a.tpg - blockIdx.x % quads * kBwdWarps;
      for (int i = ht; i < n * 2 * NP; i += 128) {
        const int t = i / (2 * NP), s = i % (2 * NP);
        float v = all.tile[0].bc[from][t][s];
#pragma unroll
        for (int k = 1; k < kBwdWarps; ++k)
          if (k < warps) v += all.tile[k].bc[from][t][s];
        a.bc[((long long)blockIdx.x * all_rows + row + t) * (2 * NP) + s] = v;
      }
    };
    fetch(chunks - 1);
    stage(chunks - 1);
    if (chunks > 1) fetch(chunks - 2);
    for (int i = chunks - 1; i >= 0; --i) {
      __syncthreads();                         // chunk i is staged, chunk i + 1 has been run through
      if (i + 1 < chunks) finish(i + 1);
      // (what other helpers may still be reading, the tiles' dB and dC, is not staged over)
      if (i > 0) stage(i - 1);
      if (i > 1) fetch(i - 2);
    }
    __syncthreads();
    finish(0);
    if (on) {
      float fD[VN], fb[VN];
#pragma unroll
      for (int e = 0; e < VP; ++e) {
        split(gD[e], fD[2 * e], fD[2 * e + 1]);
        split(gb[e], fb[2 * e], fb[2 * e + 1]);
      }
#pragma unroll
      for (int e = 0; e < VN; ++e)
#pragma unroll
        for (int m = G::LPR; m < 32; m <<= 1) {
          fD[e] += __shfl_xor_sync(0xffffffffu, fD[e], m);
          fb[e] += __shfl_xor_sync(0xffffffffu, fb[e], m);
        }
      if (w.lane < G::LPR && w.col() < w.cols) {
        put(part + (long long)a.d * a.N + w.c0 + w.col(), fD);
        put(part + (long long)a.d * (a.N + 1) + w.c0 + w.col(), fb);
      }
    }
    return;
  }

  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTokenRegs));
  const uint32_t states = tmem + ((uint32_t)warp * 32u << 16);
  F2 h[PAIRS], dh[PAIRS], A2[PAIRS];
  load_A<G>(a, w, A2);
#pragma unroll
  for (int p = 0; p < PAIRS; ++p) sm.gA[p][w.lane] = 0;
  Where q = seqs::find(a.s, r1 - 1);           // the sequence of the row at hand, from the last back
  if (q.end > r1) load_lanes<G>(a.local, (long long)(seg + 1) * a.tiles + tile, w.lane, dh);
  else load_state<G>(a, w, a.grad_final, q.i, dh);

  for (int chunk = chunks - 1; chunk >= 0; --chunk) {
    const long long row = row_of(chunk);
    const int n = count(chunk), k = chunk & 1;
    load_lanes<G>(a.ckpt, ((long long)seg * a.cps + chunk) * a.tiles + tile, w.lane, h);
    __syncthreads();
    F2 gA[PAIRS];
#pragma unroll
    for (int p = 0; p < PAIRS; ++p) gA[p] = 0;
    if (q.begin < row && n == kT) {            // inside one sequence
      {
        Token<G, false> now, ahead;
        now.read(all, sm, w, k, 0);
#pragma unroll
        for (int t = 0; t < kT - 1; ++t) {
          ahead.read(all, sm, w, k, t + 1);
          tmem_put(states + t * 2 * PAIRS, h);
          now.forward(A2, h);
          now = ahead;
        }
        tmem_put(states + (kT - 1) * 2 * PAIRS, h);
        tmem_put_wait();
      }
      // a token's sums over the lanes are taken beside the next one's arithmetic
      Token<G, true> now, ahead;
      Sums<G> sums;
      now.read(all, sm, w, k, kT - 1);
      ahead.read(all, sm, w, k, kT - 2);
      sums.token(now, h, A2, dh, gA);
#pragma unroll 3
      for (int t = kT - 2; t >= 0; --t) {
        now = ahead;
        if (t > 0) ahead.read(all, sm, w, k, t - 1);
        tmem_get(states + t * 2 * PAIRS, h);
        Sums<G> last = sums;
        sums.token(now, h, A2, dh, gA);
        last.out(sm, w, k, t + 1);
      }
      sums.out(sm, w, k, 0);
    } else {
      Where f = seqs::find(a.s, row);
      for (int t = 0; t < n; ++t) {
        if (row + t >= f.end) f = seqs::find(a.s, row + t);
        if (row + t == f.begin) load_state<G>(a, w, a.init, f.i, h);
        tmem_put(states + t * 2 * PAIRS, h);
        Token<G, false> now;
        now.read(all, sm, w, k, t);
        now.forward(A2, h);
      }
      tmem_put_wait();
      for (int t = n - 1; t >= 0; --t) {
        tmem_get(states + t * 2 * PAIRS, h);
        Token<G, true> now;
        now.read(all, sm, w, k, t);
        Sums<G> sums;
        sums.token(now, h, A2, dh, gA);
        sums.out(sm, w, k, t);
        if (row + t == q.begin) {              // the first row of its sequence: out, and on with the one before
          if (a.grad_init && on) store_state<G>(a, w, a.grad_init, q.i, dh);
          if (row + t > r0) {
            q = seqs::find(a.s, row + t - 1);
            load_state<G>(a, w, a.grad_final, q.i, dh);
          }
        }
      }
    }
#pragma unroll
    for (int p = 0; p < PAIRS; ++p) sm.gA[p][w.lane] = add2(sm.gA[p][w.lane], gA[p]);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (on) {
    F2 gA[PAIRS];
#pragma unroll
    for (int p = 0; p < PAIRS; ++p) gA[p] = sm.gA[p][w.lane];
    store_state<G>(a, w, part, 0, gA);
  }
  // every token warp has left tensor memory by the barrier above
  if (warp == 0) tc::tmem_dealloc(tmem, kColumns);
}

// grad_B and grad_C from the blocks' sums.
constexpr int kBcThreads = 256;
template <class E>
__global__ void __launch_bounds__(kBcThreads) k_ssm_bc(Args a, int NP, int quads) {
  const long long id = (long long)blockIdx.x * kBcThreads + threadIdx.x;     // (row, group, B or C, state)
  const int s = (int)(id % (2 * NP));
  const long long rg = id / (2 * NP);
  const int g = (int)(rg % a.groups), n = s % NP;
  const long long row = rg / a.groups;
  if (row >= seqs::trim(a.s).rows || n >= a.N) return;
  float v = 0.f;
#pragma unroll 8
  for (int q = 0; q < quads; ++q) v += __ldcs(a.bc + (((long long)g * quads + q) * a.s.rows + row) * (2 * NP) + s);
  rows::store1(static_cast<E*>(s < NP ? a.grad_B : a.grad_C) + (row * a.groups + g) * a.N + n, v);
}

// Registers that a kernel's threads are launched with, asked for once.
template <auto KERNEL>
static int launch_regs() {
  static std::atomic<int> known{0};
  int n = known.load(std::memory_order_relaxed);
  if (n == 0) {
    cudaFuncAttributes f;
    if (cudaFuncGetAttributes(&f, KERNEL) != cudaSuccess) return 0;
    known.store(n = f.numRegs, std::memory_order_relaxed);
  }
  return n;
}

template <class G>
static cudaError_t backward(const Args& a, const Plan& p, cudaStream_t st) {
  using E = typename G::E;
  if (p.cut) {
    {
      TraceScope tr("k_ssm_local_bwd", st);
      k_ssm_local_bwd<G><<<dim3(a.tiles, a.n_seg), 64, 0, st>>>(a);
    }
    const cudaError_t e = launch_ssm_carry<G, true>(a, st);
    if (e != cudaSuccess) return e;
  }
  const bool empty = a.grad_init && (a.s.off || a.s.rows == 0);
  const int more = empty ? (a.s.n < 32 * 64 ? (a.s.n + 31) / 32 : 64) : 0;
  if (a.n_seg + more == 0) return cudaSuccess;
  constexpr size_t smem = sizeof(BwdBlock<G>);
  static_assert(smem <= 226 * 1024, "shared memory");
  cudaError_t e = allow_smem<k_ssm_bwd<G>>(smem);
  // A block launched with fewer registers than the split hands out would wait for them for ever.  (By the count that
  // the compiler reports, which is 128 for every variant; that the hardware may round a smaller one up is not relied on.)
  if (e == cudaSuccess) e = launch_regs<k_ssm_bwd<G>>() >= kLaunchRegs ? cudaSuccess : cudaErrorLaunchOutOfResources;
  if (e != cudaSuccess) return e;
  const int quads = (a.tpg + kBwdWarps - 1) / kBwdWarps;
  {
    TraceScope tr("k_ssm_bwd", st);
    k_ssm_bwd<G><<<dim3(quads * a.groups, a.n_seg + more), 64 * kBwdWarps, smem, st>>>(a);
  }
  if (a.s.rows > 0) {
    TraceScope tr("k_ssm_bc", st);
    const long long n = a.s.rows * a.groups * 2 * G::NP;
    k_ssm_bc<E><<<(unsigned)((n + kBcThreads - 1) / kBcThreads), kBcThreads, 0, st>>>(a, G::NP, quads);
  }
  return cudaGetLastError();
}

template <class E>
static cudaError_t backward_of(const Args& a, const Plan& p, cudaStream_t st) {
  switch (p.NS) {
    case 2: return backward<Cfg<E, 2, 4>>(a, p, st);
    case 4: return backward<Cfg<E, 4, 4>>(a, p, st);
    case 8: return backward<Cfg<E, 8, 2>>(a, p, st);
    default: return backward<Cfg<E, 16, 1>>(a, p, st);
  }
}

}  // namespace ssm

cudaError_t launch_ssm_backward(const SsmArgs& g, const SsmGrads& r, cudaStream_t st) {
  const ssm::Plan p = ssm::make_plan(g.rows, g.n_seq, g.d, g.groups, g.N, g.off != nullptr);
  ssm::Args a = ssm::args_of(g, p, ssm::make_work(p, g.rows, g.d, true));
  a.grad_y = r.grad_y; a.grad_final = r.grad_final;
  a.grad_x = r.grad_x; a.grad_delta = r.grad_delta; a.grad_z = r.grad_z; a.grad_B = r.grad_B; a.grad_C = r.grad_C;
  a.grad_init = r.grad_init;
  cudaError_t e = g.math == CFC_MATH_BF16 ? ssm::backward_of<__nv_bfloat16>(a, p, st) : ssm::backward_of<float>(a, p, st);
  if (e != cudaSuccess) return e;
  // [dA | dD | dbias] of the segments
  ReduceOut o{};
  const long long d = g.d, ld = d * (g.N + 2);
  o.ptr[0] = r.grad_A;
  o.nseg = 1;
  long long n = d * g.N;
  if (r.grad_D) {
    o.ptr[1] = r.grad_D;
    o.begin[1] = n;
    o.nseg = 2;
    n += d;
    if (r.grad_bias) {
      o.ptr[2] = r.grad_bias;
      o.begin[2] = n;
      o.nseg = 3;
      n += d;
    }
  }
  e = launch_reduce(a.part, p.n_seg, n, ld, o, st);
  if (e != cudaSuccess || r.grad_D || !r.grad_bias) return e;
  ReduceOut b{};
  b.ptr[0] = r.grad_bias;
  b.nseg = 1;
  return launch_reduce(a.part + d * (g.N + 1), p.n_seg, d, ld, b, st);
}

}  // namespace cfc
