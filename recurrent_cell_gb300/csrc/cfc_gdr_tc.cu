// cfc_gdr_tc.cu -- the serial passes of the gated delta rule in bf16 on the
// 5th-generation tensor cores (notation of gdr_common.cuh).
//
// Value columns do not touch one another, so a head is split into tiles of NV
// columns, a block each.  A chunk takes three products of 128 rows, each
// waiting for the one before:
//   D1 = [K; Q] S0        rows 0-63:  R = beta (V - exp(G) D1)
//                         rows 64-127: scale exp(G) D1, the outputs' first part
//   D2 = [T - I; P T] R   rows 0-63:  U = R + D2
//                         rows 64-127: the outputs' second part (P U = P T R)
//   D3 = K^T (exp(G_C - G) U),  S1 = exp(G_C) S0 + D3.
// Tokens, and for D3 the key index, are the accumulator's lanes: S lives in
// registers, one key row a thread, and S, R and U go to shared memory row by
// row as MN-major operand tiles.  R and S stay fp32 where they are added.
//
// PL = 2 (a state leaves the call): S, R, U and [T - I; P T] as two bf16
// planes, 17 significant bits.  The planes lie side by side in the operand's
// 64 NB columns, NV = 64 NB / PL, one product for both.
//
// A NaN or an infinity reaches no earlier token although D2 multiplies it by zeros
// for them: its place in R is zero, its U is NaN (and so the state), and the fetching
// warps, which copy the outputs, write NaN from there on.  The preparation finds bad k, g
// and beta, the pass itself bad V.  Looking for them takes 2 us of 78 and 8 of 410
// (16384 tokens x 16 heads); joining a vote to a barrier of the chain took 26.
//
// What bounds a pass over few heads is the length of that chain: 1.6 us a chunk
// of 32 columns with PL = 2 (16384 tokens x 16 heads 418 us; 40 us by bytes),
// of which the products, bound by their operands' reads of shared memory, are
// 0.5 us and the rest three times accumulator -> registers -> operand ->
// barrier.  With many heads and no state asked for a chunk of 128 columns moves
// 121 KB in 3.3 us; 128 heads on as many SMs come to 4.7 TB/s forward, 4.2 backward,
// 70 and 62 % of a copy's rate, the chain being what they wait for (8 x 2048 x 16
// heads 108 us and 119).
#include "gdr_tc.cuh"

namespace cfc {
namespace gdr {

__device__ int g_gdr_tc_error = 0;

// ------------------------------------------------------------ all chunks at once
// One block of 4 warps a (chunk, value head): the decays, T - I and P T.
// T = (I + A)^{-1} comes from 16 x 16 diagonal blocks by forward substitution
// (a warp each, a column a lane), then pairs of blocks joined by
// T21 = -T22 A21 T11, all in fp32 or fp32-accurate products: T's entries reach
// far above A's when keys repeat.  P T = P + P (T - I) takes P from the
// registers that q k^T left it in and T - I, both as two bf16 planes; PL = 1 only
// rounds the results.  One pass of TF32 and bf16 products there takes 62 us instead
// of 74 for 4096 chunks and heads, but where keys repeat the terms cancel after their
// rounding: o of a chunk of equal keys 1.5e-2 from exact instead of 2.5e-3.
template <int DK>
struct PrepTc {
  static constexpr int LDK = DK + 8, LDA = kC + 4;
  static constexpr uint32_t K = kC * LDK * 2, A = kC * LDA * 4;
  // k, then A and T, then P T; q, then T - I: each is done with when the next begins
  static constexpr uint32_t OFF_I = (K > A ? K : A), OFF_G = OFF_I + (K > kImage / 2 ? K : kImage / 2);
  static constexpr uint32_t BYTES = OFF_G + 3 * kC * 4;
  static_assert(BYTES >= kMaxOrder * 4, "the sequences' lengths");
};

// The sequences' order by falling length (ties by number): the longest one's
// serial pass is the least that the whole takes, so it has to begin first (16
// prompts of 0 to 4100 tokens x 16 heads 222 us, in their own order 233).
// `lens`: kMaxOrder ints of shared memory.
__device__ __noinline__ void longest_first(const FwdArgs& a, int* lens, int tid) {
  const int n4 = (a.s.n_seq + 3) / 4 * 4;
  for (int n = tid; n < n4; n += 128) {
    long long s;
    int len = -1;
    if (n < a.s.n_seq) seq_range(a.s, n, &s, &len);
    lens[n] = len;
  }
  __syncthreads();
  for (int n = tid; n < a.s.n_seq; n += 128) {
    const int len = lens[n];
    int rank = 0;
#pragma unroll 4
    for (int m = 0; m < n4; m += 4) {
      const int4 l = *reinterpret_cast<const int4*>(lens + m);
      // as long, and before it
      rank += (l.x + (m < n) > len) + (l.y + (m + 1 < n) > len) + (l.z + (m + 2 < n) > len) + (l.w + (m + 3 < n) > len);
    }
    a.order[rank] = n;
  }
  // How many of them to halve (see work_of), for tiles of 64 and of 128 columns.
  if (tid < 32) {
    long long sum = 0;
    for (int n = tid; n < a.s.n_seq; n += 32) sum += (lens[n] + kC - 1) / kC;
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const long long share = sum * a.s.hv * ((a.s.dv + (64 << w) - 1) / (64 << w)) / kNumSMs;
      int count = 0;
      for (int n = tid; n < a.s.n_seq; n += 32) count += 4ll * ((lens[n] + kC - 1) / kC) > 5 * share;
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) count += __shfl_xor_sync(0xffffffffu, count, m);
      if (tid == 0) a.order[a.s.n_seq + w] = count;
    }
  }
  __syncthreads();
}

template <int DK, int PL>
__global__ void __launch_bounds__(128, 5) k_gdr_prep_tc(FwdArgs a) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  using P = MBf16;
  using S = PrepTc<DK>;
  bf16* ks = reinterpret_cast<bf16*>(smem_raw);
  bf16* qs = reinterpret_cast<bf16*>(smem_raw + S::OFF_I);
  float* am = reinterpret_cast<float*>(smem_raw);
  unsigned char *img = smem_raw + S::OFF_I, *pimg = smem_raw;      // 64 rows each, the lo plane 8 KB on
  float2* g2 = reinterpret_cast<float2*>(smem_raw + S::OFF_G);
  float* bet = reinterpret_cast<float*>(g2 + kC);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x % a.s.hv;
  const long long slot = blockIdx.x / a.s.hv;
  int n, len, c;
  long long start;
  if (a.order && blockIdx.x == 0) longest_first(a, reinterpret_cast<int*>(smem_raw), tid);
  if (!slot_chunk(a.s, slot, &n, &start, &len, &c)) return;
  const long long row0 = start + (long long)c * kC;
  const int rows = min(kC, len - c * kC);
  const int hq = h / (a.s.hv / a.s.hk);
  // the gates are wanted after the products: asked for first, they are there by then
  const float4 gb = warp == 0 ? load_gates(a, row0, rows, h, lane) : make_float4(0.f, 0.f, 0.f, 0.f);
  load_tile<bf16, kC, DK, 128>(ks, S::LDK, static_cast<const bf16*>(a.k) + row0 * a.ldk + (long long)hq * a.s.dk, a.ldk,
                               rows, a.s.dk, tid);
  load_tile<bf16, kC, DK, 128>(qs, S::LDK, static_cast<const bf16*>(a.q) + row0 * a.ldq + (long long)hq * a.s.dk, a.ldq,
                               rows, a.s.dk, tid);
  cp_commit();
  const long long id = slot * a.s.hv + h;
  float* vec = a.vec + id * kVec;
  cp_wait<0>();
  __syncthreads();

  // Rows 16 warp .. of q k^T and k k^T, columns up to the diagonal block.
  const Mat<bf16> mk{ks, S::LDK}, mq{qs, S::LDK};
  const int m0 = warp * 16, g = lane >> 2, t2 = (lane & 3) * 2;
  float pr[8][4] = {}, ak[8][4] = {};
#pragma unroll 2
  for (int k0 = 0; k0 < DK; k0 += 16) {
    P::A fq, fk;
    P::load_a(fq, mq, m0, k0, lane);
    P::load_a(fk, mk, m0, k0, lane);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j > warp) continue;
      P::B fb;
      P::load_bn(fb, mk, j * 16, k0, lane);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        P::mma(pr[2 * j + hf], fq, fb, hf);
        P::mma(ak[2 * j + hf], fk, fb, hf);
      }
    }
  }
  if (warp == 0) chunk_decays(gb, lane, c == 0 && !a.init, g2, bet, vec);   // the warp with the fewest products
  __syncthreads();
  // P in the registers, A in shared memory.  (The first row has no entries in A: its |k|^2, not a number or infinite
  // as soon as one of k is, and its g speak for it.)
  float sum = tid == 0 ? fabsf(ak[0][0]) + fabsf(g2[0].x) : 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int col = j * 8 + t2;
    float av[4] = {};
    if (j <= 2 * warp + 1) {
      const float4 gj = *reinterpret_cast<const float4*>(g2 + col);
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const int i = m0 + g + rr * 8;
        const float2 gi = g2[i];
        const float l0 = exp2_approx((gi.x - gj.x) + (gi.y - gj.y)), l1 = exp2_approx((gi.x - gj.z) + (gi.y - gj.w));
        const float be = bet[i];
        av[2 * rr] = col < i ? be * l0 * ak[j][2 * rr] : 0.f;
        av[2 * rr + 1] = col + 1 < i ? be * l1 * ak[j][2 * rr + 1] : 0.f;
        pr[j][2 * rr] = col <= i ? a.s.scale * l0 * pr[j][2 * rr] : 0.f;
        pr[j][2 * rr + 1] = col < i ? a.s.scale * l1 * pr[j][2 * rr + 1] : 0.f;
      }
      sum += fabsf(av[0]) + fabsf(av[1]) + fabsf(av[2]) + fabsf(av[3]);
    }
    *reinterpret_cast<float2*>(am + (m0 + g) * S::LDA + col) = make_float2(av[0], av[1]);
    *reinterpret_cast<float2*>(am + (m0 + g + 8) * S::LDA + col) = make_float2(av[2], av[3]);
  }
  if (!finite(sum)) {
#pragma unroll 1
    for (int x = 0; x < 32; ++x) {
      const int row = m0 + g + (x & 1) * 8;
      drop(am[row * S::LDA + (x >> 2) * 8 + t2 + ((x >> 1) & 1)], vec, row);
    }
    if (tid == 0 && !(finite(ak[0][0]) && finite(g2[0].x))) vec[kVecBeta] = nanf("");
  }
  __syncwarp();
  invert<S::LDA>(am, warp, lane);
  // T - I into the image, both planes
  __nv_bfloat162 z = __float2bfloat162_rn(0.f);
#pragma unroll
  for (int e = 0; e < kC * 8 / 128; ++e) {
    const int r = (e * 128 + tid) >> 3, ch = tid & 7;
    float v[8] = {};
    if (ch * 8 <= r) {
      const float* src = am + r * S::LDA + ch * 8;
      *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(src);
      *reinterpret_cast<float4*>(v + 4) = *reinterpret_cast<const float4*>(src + 4);
      if (r >> 3 == ch)
#pragma unroll
        for (int x = 0; x < 8; ++x) v[x] = (r & 7) == x ? 0.f : v[x];
    }
    const uint4 hi = pack8(v);
    *reinterpret_cast<uint4*>(img + chunk_at(r, ch)) = hi;
    z = times_zero(hi, z);
    float hv[8];
    unpack8(hv, hi);
#pragma unroll
    for (int x = 0; x < 8; ++x) hv[x] = v[x] - hv[x];
    *reinterpret_cast<uint4*>(img + 8192 + chunk_at(r, ch)) = pack8(hv);
  }
  if (!zeros(z)) {                       // T has overflowed: as for A
#pragma unroll 1
    for (int e = 0; e < kC * 8 * 8 / 128; ++e) {
      const int r = ((e >> 3) * 128 + tid) >> 3;
      bf16* p = reinterpret_cast<bf16*>(img + chunk_at(r, tid & 7)) + (e & 7);
      if (finite(__bfloat162float(*p))) continue;
      *p = p[4096] = __float2bfloat16_rn(0.f);
      vec[kVecBeta + r] = nanf("");
    }
  }
  __syncthreads();
  // P T, 16 rows a warp
  float d[8][4];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) d[j][e] = pr[j][e];
#pragma unroll
  for (int kb = 0; kb < 4; ++kb) {
    if (kb > warp) continue;
    P::A ah, al;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float* p = pr[2 * kb + (x >> 1)] + (x & 1) * 2;
      ah[x] = pack2(p[0], p[1]);
      al[x] = pack2(p[0] - lo_f(ah[x]), p[1] - hi_f(ah[x]));
    }
    const int r = kb * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
    for (int jb = 0; jb < 4; ++jb) {
      if (jb > kb) continue;
      P::B bh, bl;
      const unsigned char* src = img + chunk_at(r, jb * 2 + (lane >> 4));
      P::ldmt(bh, src);
      P::ldmt(bl, src + 8192);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        P::mma(d[2 * jb + hf], al, bh, hf);
        P::mma(d[2 * jb + hf], ah, bl, hf);
        P::mma(d[2 * jb + hf], ah, bh, hf);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      const uint32_t o = chunk_at(m0 + g + rr * 8, j) + t2 * 2;
      const uint32_t hi = pack2(d[j][2 * rr], d[j][2 * rr + 1]);
      *reinterpret_cast<uint32_t*>(pimg + o) = hi;
      if constexpr (PL == 2)
        *reinterpret_cast<uint32_t*>(pimg + 8192 + o) =
            pack2(d[j][2 * rr] - lo_f(hi), d[j][2 * rr + 1] - hi_f(hi));
    }
  tc::fence_proxy_async_smem();
  __syncthreads();
  if (tid == 0) {
    char* out = a.t + id * kImage;
#pragma unroll
    for (int pl = 0; pl < PL; ++pl) {
      bulk_store(out + pl * (kImage / 2), img + pl * 8192, 8192);
      bulk_store(out + pl * (kImage / 2) + 8192, pimg + pl * 8192, 8192);
    }
    bulk_store_read();
  }
}

template <int DK, int PL, int NB, bool BWD>
struct TcCfg {
  // Warps that share the columns; 4: 16 ragged prompts 222 -> 233 us, training 447 -> 462.
  static constexpr int CW = 2;
  static constexpr int NV = 64 * NB / PL, ATOMS = DK / 64, FETCH = 128, WORK = 128 * CW, THREADS = WORK + FETCH;
  static constexpr int NC = NV / CW;                    // columns a thread
  static constexpr int LO = NV;                         // from the hi to the lo plane's accumulator columns
  static constexpr uint32_t KQ = ATOMS * 16384u;        // per 64 key columns: 64 rows of K, 64 of Q
  static constexpr uint32_t A2 = PL * 16384u;
  static constexpr uint32_t VT = 64 * NV * 2;           // V (or dO): 64 rows
  static constexpr uint32_t STAGE = (KQ + A2 + VT + kVec * 4 + 1023) / 1024 * 1024;
  // S; R, then its decayed U; U as it is (PL = 1); backward: dO scaled.  NB blocks each.
  static constexpr uint32_t SB = DK * 128u, RB = 8192u, S = NB * SB, R = NB * RB;
  // forward, for each stage: each column's first bad token, and whether there is one
  static constexpr uint32_t BAD = BWD ? 0 : 2 * (NV + 1) * 4;
  static constexpr uint32_t BYTES = 2048 + 2 * STAGE + S + (PL == 1 ? 2 : 1) * R + (BWD ? R : 0) + BAD;
  static constexpr uint32_t TMEM = NB * 128;            // D1 / D2 and D3
  static_assert(BYTES <= 227u * 1024u, "shared memory");
};

// Columns col .. col + 7 of a row into a tile of blocks of BB bytes: PL = 1,
// blocks of 64 columns; PL = 2, the lo plane in the second block or, with one
// block, in its second half.
template <int PL, int NB, uint32_t BB>
__device__ __forceinline__ void put8(unsigned char* tile, int row, int col, const float* v) {
  const uint4 h = pack8(v);
  if constexpr (PL == 1) {
    *reinterpret_cast<uint4*>(tile + (NB > 1 ? (col >> 6) * BB : 0) + chunk_at(row, (col & 63) >> 3)) = h;
  } else {
    *reinterpret_cast<uint4*>(tile + chunk_at(row, col >> 3)) = h;
    float l[8];
    unpack8(l, h);
#pragma unroll
    for (int i = 0; i < 8; ++i) l[i] = v[i] - l[i];
    *reinterpret_cast<uint4*>(tile + (NB > 1 ? BB + chunk_at(row, col >> 3) : chunk_at(row, (col >> 3) + 4))) = pack8(l);
  }
}

struct TcArgs {
  Shape s;
  const bf16 *q, *k, *v;        // v: the backward's grad_o
  long long ldq, ldk, ldv;
  const float* init;            // the backward's grad_final_state
  float* final_state;           // the backward's grad_initial_state
  bf16* o;                      // the backward's grad_v
  const unsigned char* a2;
  const float* vec;
  // per chunk and 64 value columns, as operand tiles: S0 and U (backward: dS1, dR), or NULL
  unsigned char *st, *u;
  const int* order;             // the sequences, longest first; then how many to halve
  int ntile, tma;
  int twice;                    // so many of the longest may go in tiles of half the width; 0: none
};

// The n-th sequence to run; held to the batch whatever the workspace holds.
__device__ __forceinline__ int nth(const TcArgs& a, int i) {
  const int n = a.order ? a.order[i] : i;
  return (unsigned)n < (unsigned)a.s.n_seq ? n : i;
}

// What a block does: a tile of a head of a sequence; tile < 0: nothing.  The
// longest sequences, those that would outlast by a quarter and more an even
// share of the whole, take tiles of half the width, two thirds of the time a
// chunk.  (Training of 3000 of 6470 tokens x 16 heads 28 % less, now 305 us, prompts of
// 8000 of 8530 tokens x 16 heads 26 % less, now 257; at 1.05 of the share 194 -> 220, so
// not there.  A batch in which nothing is halved loses 5 % by the joint kernel.)
struct Work {
  int n, h, tile, len;
  long long start;
  bool half;
};
__device__ __forceinline__ Work work_of(const TcArgs& a, int wide) {
  Work w;
  int b = blockIdx.x, k = 0;
  if (a.twice > 0) {
    k = a.order[a.s.n_seq + (wide == 128)];
    k = k < 0 || k > a.twice ? 0 : k;
  }
  const int two = 2 * a.ntile, first = k * a.s.hv * two;
  w.half = b < first;
  const int tiles = w.half ? two : a.ntile;
  if (!w.half) b -= first;
  w.tile = b % tiles;
  b /= tiles;
  w.h = b % a.s.hv;
  b = b / a.s.hv + (w.half ? 0 : k);
  if (b >= a.s.n_seq) {
    w.tile = -1;
    return w;
  }
  w.n = nth(a, b);
  seq_range(a.s, w.n, &w.start, &w.len);
  return w;
}

// The fetching warps' loop.  The chunk before last's output rows (o, or the
// backward's dv), which lie in the place of its V (dO), go to global memory;
// then the next chunk's tiles come into that stage: the prepared images by bulk
// copy, q, k and v as tensor-map boxes where the chunk is whole, else by the
// fetching threads' 16-byte copies (rows past the end as zeros).  With
// copies alone, both passes and the gradients: 16384 tokens x 16 heads 532 us
// against 487, training of 8 x 2048 x 16 heads 478 against 434.
template <int DK, class C, class W>
__device__ __forceinline__ void fetch_chunks(const TcArgs& a, const Maps& maps, const CUtensorMap* v_map,
                                             unsigned char* stage, uint64_t* full,
                                             uint64_t* empty, uint64_t* outs, int ft, int h, long long start, int len,
                                             long long slot0, int v0, bool backwards, int* bad_from, W wait) {
  constexpr int NV = C::NV;
  const int hq = h / (a.s.hv / a.s.hk), dk = a.s.dk, nc = (len + kC - 1) / kC;
  const bf16* q = a.q + start * a.ldq + (long long)hq * dk;
  const bf16* k = a.k + start * a.ldk + (long long)hq * dk;
  const bf16* v = a.v + start * a.ldv + (long long)h * a.s.dv + v0;
  const int vn = a.s.dv - v0;
  const long long ldo = (long long)a.s.hv * a.s.dv;
  for (int i = 0; i < nc + 2; ++i) {
    const int c = backwards ? nc - 1 - i : i, st = i & 1;
    unsigned char* b = stage + st * C::STAGE;
    if (i >= 2 && i - 2 < nc) {
      const int cl = backwards ? c + 2 : c - 2;
      bf16* o = a.o + (start + (long long)cl * kC) * ldo + (long long)h * a.s.dv + v0;
      wait(outs + st, (i / 2 - 1) & 1);
      if (bad_from && bad_from[st * (NV + 1) + NV]) {      // outputs from a bad token on
        int* from = bad_from + st * (NV + 1);
        group_sync<15, C::FETCH>();
        for (int x = ft; x < NV; x += C::FETCH) {
          for (int r = from[x]; r < kC; ++r)
            reinterpret_cast<unsigned short*>(b + C::KQ + C::A2 + v_at<NV>(r, x / 8))[x % 8] = 0x7fff;
          from[x] = kC;
        }
        if (ft == 0) from[NV] = 0;
        group_sync<15, C::FETCH>();
      }
      // 4 warps: 32 rows by half of the columns each
      const int w = ft >> 5;
      rows_out<NV, NV / 2>(o, ldo, b + C::KQ + C::A2, (w & 1) * 32, (w >> 1) * (NV / 16), min(kC, len - cl * kC), vn,
                           ft & 31);
      group_sync<15, C::FETCH>();          // the tiles are filled again by other threads
      if (!wait(empty + st, (i / 2 - 1) & 1)) continue;      // nothing more is fetched after a wait that gave up
    }
    if (i >= nc) continue;
    const int rows = min(kC, len - c * kC);
    const long long r0 = (long long)c * kC, id = (slot0 + c) * a.s.hv + h;
    const bool boxes = a.tma && rows == kC;
    if (ft == 0) {
      tc::fence_proxy_async_smem();      // output rows were written where boxes now go
      bar_arrive_tx(full + st, C::A2 + kVec * 4 + (boxes ? C::KQ + C::VT : 0));
      if (boxes) {
        const int row = (int)(start + r0);
#pragma unroll
        for (int x = 0; x < C::ATOMS; ++x) {
          tma_tile(b + x * 16384, &maps.k, x * 64, hq, row, full + st);
          tma_tile(b + x * 16384 + 8192, &maps.q, x * 64, hq, row, full + st);
        }
        constexpr int VB = NV < 64 ? NV : 64;
#pragma unroll
        for (int x = 0; x < NV / VB; ++x)
          tma_tile(b + C::KQ + C::A2 + x * 8192, v_map, v0 + x * VB, h, row, full + st);
      }
      bulk_load(b + C::KQ, a.a2 + id * 32768, C::A2, full + st);
      bulk_load(b + C::KQ + C::A2 + C::VT, a.vec + id * kVec, kVec * 4, full + st);
    }
    if (!boxes) {
      {
        constexpr int PER = DK / 8, STEP = C::FETCH / PER;      // 16-byte pieces of a row; rows a pass
        const int ch = ft % PER, rr = ft / PER;
        const bool in = ch * 8 < dk;
        unsigned char* d = b + (ch >> 3) * 16384;
#pragma unroll 4
        for (int r = rr; r < kC; r += STEP) {
          const bool on = in && r < rows;
          cp16(d + chunk_at(r, ch & 7), on ? k + (r0 + r) * a.ldk + ch * 8 : k, on);
          cp16(d + 8192 + chunk_at(r, ch & 7), on ? q + (r0 + r) * a.ldq + ch * 8 : q, on);
        }
      }
      {
        constexpr int PER = NV / 8, STEP = C::FETCH / PER;
        const int ch = ft % PER;
        const bool in = ch * 8 < vn;
        unsigned char* d = b + C::KQ + C::A2;
#pragma unroll 4
        for (int r = ft / PER; r < kC; r += STEP) {
          const bool on = in && r < rows;
          cp16(d + v_at<NV>(r, ch), on ? v + (r0 + r) * a.ldv + ch * 8 : v, on);
        }
      }
      cp_commit();
      cp_wait<0>();
      tc::fence_proxy_async_smem();      // read by the tensor cores
    }
    bar_arrive(full + st);
  }
}

// ------------------------------------------------------------------- forward
// A block's work: a tile of a head of sequence n, the rows start .. start + len.
template <int DK, int PL, int NB>
__device__ __forceinline__ void scan_tile(const TcArgs& a, const Maps& maps, const CUtensorMap* v_map,
                                          unsigned char* smem_raw, int n, int h, int tile, long long start, int len) {
  using C = TcCfg<DK, PL, NB, false>;
  constexpr int NC = C::NC, NV = C::NV, NP = 16;      // columns a thread; at a time
  unsigned char* base = smem_raw + (1024 - (smem_addr(smem_raw) & 1023)) % 1024;
  uint64_t* full = reinterpret_cast<uint64_t*>(base);
  uint64_t *empty = full + 2, *done = full + 4, *outs = full + 6;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(base + 128);
  unsigned char* stage = base + 1024;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long sh = (long long)n * a.s.hv + h;
  const int nc = (len + kC - 1) / kC;
  const long long slot0 = slot_base(start, n);
  int* bad_from = reinterpret_cast<int*>(stage + 2 * C::STAGE + C::S + (PL == 1 ? 2 : 1) * C::R);
  for (int x = tid; x < 2 * (NV + 1); x += C::THREADS) bad_from[x] = x % (NV + 1) < NV ? kC : 0;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(full + i, C::FETCH + 1);
      tc::mbar_init(empty + i, 1);             // a chunk's last product
      tc::mbar_init(outs + i, 2 * C::CW);         // the warps that form output rows
      tc::mbar_init(done + i, 1);
    }
    tc::mbar_init_fence();
  }
  if (warp == 0) tc::tmem_alloc(tmem_at, C::TMEM);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_at;
  bool lost = false;        // a wait gave up: no more waiting, the results are void
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!lost && !tc::mbar_wait(bar, parity, kPolls)) {
      lost = true;
      atomicExch(&g_gdr_tc_error, 1);
    }
    lost = __any_sync(0xffffffffu, lost);      // a warp goes on as one
    return !lost;
  };
  // (a warp comes to it as one, and one instruction's answer is the same for all its lanes)
  auto poll = [&](uint64_t* bar, uint32_t parity) {
    if (!lost && !poll_wait(bar, parity, kPollsBusy)) {
      lost = true;
      atomicExch(&g_gdr_tc_error, 1);
    }
  };

  if (tid >= C::WORK) {
    fetch_chunks<DK, C>(a, maps, v_map, stage, full, empty, outs, tid - C::WORK, h, start, len, slot0,
                                     tile * NV, false, bad_from, wait);
  } else {
    const int quad = warp & 3, cg = warp >> 2, row = quad * 32 + lane;
    const int v0 = tile * NV, c0 = cg * NC, dk = a.s.dk, dv = a.s.dv;
    const bool token = quad < 2;             // rows of K; else rows of Q
    const bool issuer = quad == 0 && cg == 0;
    const int i = row & 63;                  // the row's token
    unsigned char* stile = stage + 2 * C::STAGE;
    unsigned char* rtile = stile + C::S;
    unsigned char* utile = rtile + C::R;
    const uint32_t d12 = tmem, d3 = tmem + 64 * NB, at = ((uint32_t)(quad * 32) << 16) + c0;
    const uint32_t id_kq = tc::idesc(128, 64 * NB, tc::kFmtBF16) | kBmn;
    const uint32_t id_lo = tc::idesc(128, NV, tc::kFmtBF16) | kBmn;
    const uint32_t id_kt = tc::idesc(128, 64 * NB, tc::kFmtBF16) | kAmn | kBmn;
    const uint64_t bs = mn_desc(smem_addr(stile), C::SB), br = mn_desc(smem_addr(rtile), C::RB);
    uint32_t phase = 0;
    const bool srow = row < dk && row < DK;
    float s[NC];
#pragma unroll
    for (int j = 0; j < NC; j += 4) {
      const int col = v0 + c0 + j;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (a.init && srow && col < dv) x = *reinterpret_cast<const float4*>(a.init + (sh * dk + row) * dv + col);
      s[j] = x.x; s[j + 1] = x.y; s[j + 2] = x.z; s[j + 3] = x.w;
    }
    for (int c = 0; c < nc; ++c) {
      const int st = c & 1;
      unsigned char* b = stage + st * C::STAGE;
      unsigned char* vt = b + C::KQ + C::A2;
      const float* vec = reinterpret_cast<const float*>(b + C::KQ + C::A2 + C::VT);
      const long long img = ((slot0 + c) * a.s.hv + h) * ((dv + 63) / 64) + v0 / 64;
      if (row < DK) {
#pragma unroll
        for (int j = 0; j < NC; j += 8) put8<PL, NB, C::SB>(stile, row, c0 + j, s + j);
      }
      if (c == 0 && issuer) wait(full, 0);
      tc::fence_proxy_async_smem();
      tc::fence_before_sync();
      group_sync<1, C::WORK>();
      if (issuer) {
        tc::fence_after_sync();
        const uint64_t ad = tc::sdesc_k_sw128(smem_addr(b));
        if (tc::elect_one()) {
#pragma unroll
          for (int ks = 0; ks < DK / 16; ++ks)
            tc::mma_bf16(d12, tc::sdesc_advance(ad, (ks >> 2) * 16384 + (ks & 3) * kStepK),
                         tc::sdesc_advance(bs, ks * kStepMN), id_kq, ks > 0);
          tc::mma_commit(done);
          if (PL == 1 && a.st) bulk_store(a.st + img * C::SB, stile, min(NB, (dv - v0 + 63) / 64) * C::SB);
        }
        __syncwarp();
      }
      if (PL == 2 && a.st && row < DK)      // only the hi plane
#pragma unroll
        for (int j = 0; j < NC; j += 8)
          *reinterpret_cast<uint4*>(a.st + img * C::SB + chunk_at(row, ((v0 & 63) + c0 + j) / 8)) = pack8(s + j);
      const float eg = vec[kVecEG + i], be = vec[kVecBeta + i], el = vec[kVecEGL + i], dec = vec[kVecD];
      float r[NC];                     // beta V; then R; in the rows of Q, O
      bool bad = false;                // a token with a NaN or an infinity, in V or marked by the preparation
      if (token) {
        __nv_bfloat162 z = __float2bfloat162_rn(0.f);
#pragma unroll
        for (int j = 0; j < NC; j += 8) {
          const uint4 u = *reinterpret_cast<const uint4*>(vt + v_at<NV>(i, (c0 + j) / 8));
          z = times_zero(u, z);
          unpack8(r + j, u);
#pragma unroll
          for (int e = 0; e < 8; ++e) r[j + e] *= be;
        }
        bad = !zeros(z) || !finite(be);
        if (bad) {
#pragma unroll
          for (int j = 0; j < NC; ++j)
            if (!finite(r[j])) atomicMin(bad_from + st * (NV + 1) + c0 + j, i);
          bad_from[st * (NV + 1) + NV] = 1;
        }
        __syncwarp();
      }
      const float f = token ? -be * eg : a.s.scale * eg;
      poll(done, phase);
      phase ^= 1;
      tc::fence_after_sync();
#pragma unroll
      for (int j = 0; j < NC; j += NP) {
        float x[NP];
        ld_sum<NP, PL, C::LO>(d12 + at + j, x);
        if (token) {
#pragma unroll
          for (int e = 0; e < NP; ++e) r[j + e] = fmaf(f, x[e], r[j + e]);
#pragma unroll
          for (int e = 0; e < NP; e += 8) put8<PL, NB, C::RB>(rtile, i, c0 + j + e, r + j + e);
        } else {
#pragma unroll
          for (int e = 0; e < NP; ++e) r[j + e] = f * x[e];
        }
      }
      if (PL == 1 && issuer) bulk_store_read();      // S and the last chunk's U have left their tiles
      if (bad) {
        // The product reads all 64 tokens for each, the later ones with factors of zero: a bad value's place in it is zero.
#pragma unroll
        for (int j = 0; j < NC; j += 8) {
          float w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = finite(r[j + e]) ? r[j + e] : 0.f;
          put8<PL, NB, C::RB>(rtile, i, c0 + j, w);
        }
      }
      tc::fence_proxy_async_smem();
      tc::fence_before_sync();
      group_sync<1, C::WORK>();
      if (issuer) {
        tc::fence_after_sync();
        const uint64_t ad = tc::sdesc_k_sw128(smem_addr(b + C::KQ));
        if (tc::elect_one()) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            tc::mma_bf16(d12, tc::sdesc_advance(ad, ks * kStepK), tc::sdesc_advance(br, ks * kStepMN), id_kq, ks > 0);
          if constexpr (PL == 2) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              tc::mma_bf16(d12, tc::sdesc_advance(ad, 16384 + ks * kStepK), tc::sdesc_advance(br, ks * kStepMN), id_lo,
                           1u);
          }
          tc::mma_commit(done);
        }
        __syncwarp();
      }
      poll(done, phase);
      phase ^= 1;
      tc::fence_after_sync();
#pragma unroll
      for (int j = 0; j < NC; j += NP) {
        float x[NP];
        ld_sum<NP, PL, C::LO>(d12 + at + j, x);
#pragma unroll
        for (int e = 0; e < NP; ++e) r[j + e] += x[e];
      }
      if (token) {
#pragma unroll
        for (int j = 0; j < NC; j += 8) {
          float w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = el * r[j + e];
          put8<PL, NB, C::RB>(rtile, i, c0 + j, w);
          if (a.u) {
            if constexpr (PL == 1) put8<PL, NB, C::RB>(utile, i, c0 + j, r + j);
            else
              *reinterpret_cast<uint4*>(a.u + img * C::RB + chunk_at(i, ((v0 & 63) + c0 + j) / 8)) = pack8(r + j);
          }
        }
      }
      tc::fence_proxy_async_smem();
      tc::fence_before_sync();
      group_sync<1, C::WORK>();
      if (issuer) {
        tc::fence_after_sync();
        const uint64_t ad = mn_desc(smem_addr(b), DK == 128 ? 16384 : 8192);   // DK = 64: rows 64.. unused
        if (tc::elect_one()) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            tc::mma_bf16(d3, tc::sdesc_advance(ad, ks * kStepMN), tc::sdesc_advance(br, ks * kStepMN), id_kt, ks > 0);
          tc::mma_commit(done);
          tc::mma_commit(empty + st);
          if (PL == 1 && a.u) bulk_store(a.u + img * C::RB, utile, min(NB, (dv - v0 + 63) / 64) * C::RB);
        }
        __syncwarp();
      }
      // While it runs, the outputs into V's tile, which has been read.
      if (!token) {
#pragma unroll
        for (int j = 0; j < NC; j += 8)
          *reinterpret_cast<uint4*>(vt + v_at<NV>(i, (c0 + j) / 8)) = pack8(r + j);
        __syncwarp();
        if (lane == 0) bar_arrive(outs + st);
        __syncwarp();
      }
      // the next chunk's tiles, long there: the block's barrier passes it on
      if (issuer && c + 1 < nc) wait(full + (st ^ 1), ((c + 1) >> 1) & 1);
      poll(done, phase);
      phase ^= 1;
      tc::fence_after_sync();
#pragma unroll
      for (int j = 0; j < NC; j += NP) {
        float x[NP];
        ld_sum<NP, PL, C::LO>(d3 + at + j, x);
#pragma unroll
        for (int e = 0; e < NP; ++e) s[j + e] = fmaf(dec, s[j + e], x[e]);
      }
    }
    if (a.final_state && srow) {
#pragma unroll
      for (int j = 0; j < NC; j += 4)
        if (v0 + c0 + j < dv)
          *reinterpret_cast<float4*>(a.final_state + (sh * dk + row) * dv + v0 + c0 + j) =
              make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
    }
    if (issuer) bulk_store_read();
  }
  if (lost)                  // copies and products that may still be on their way
    for (int j = 0; j < 2; ++j) {
      tc::mbar_wait(full + j, 0, kPolls);
      tc::mbar_wait(done + j, 0, kPolls);
    }
  tc::fence_before_sync();
  __syncwarp();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::TMEM);
  }
}

template <int DK, int PL, int NB>
__global__ void __launch_bounds__(TcCfg<DK, PL, NB, false>::THREADS, 1)
    k_gdr_scan_tc(TcArgs a, const __grid_constant__ Maps maps) {
  extern __shared__ unsigned char smem_raw[];
  const Work w = work_of(a, 0);
  scan_tile<DK, PL, NB>(a, maps, &maps.v, smem_raw, w.n, w.h, w.tile, w.start, w.len);
}

template <int DK, int PL>
__global__ void __launch_bounds__(TcCfg<DK, PL, 2, false>::THREADS, 1)
    k_gdr_scan_mixed_tc(TcArgs a, const __grid_constant__ Maps maps) {
  extern __shared__ unsigned char smem_raw[];
  const Work w = work_of(a, TcCfg<DK, PL, 2, false>::NV);
  if (w.tile < 0) return;
  if (w.half) {
    // (kept in tiles of 64 columns: two of 32 fill one)
    if (PL == 2 || w.tile * 64 < a.s.dv)
      scan_tile<DK, PL, 1>(a, maps, PL == 2 ? &maps.w : &maps.v, smem_raw, w.n, w.h, w.tile, w.start, w.len);
  } else {
    scan_tile<DK, PL, 2>(a, maps, &maps.v, smem_raw, w.n, w.h, w.tile, w.start, w.len);
  }
}

// ------------------------------------------------------------------ backward
// Last chunk first, the state gradient dS in registers:
//   D1 = [K; .] dS1               X = exp(G_C - G) D1
//   D2 = (T - I)^T X + (P T)^T dO dR = X + D2 (= T^T dU),  dv = beta dR
//   D3 = Q^T (scale exp(G) dO) - K^T (beta exp(G) dR),  dS0 = exp(G_C) dS1 + D3.
// The warps on lanes 64-127 scale dO for D3 meanwhile; its Q^T part runs under
// the wait for D1.
template <int DK, int NB>
__device__ __forceinline__ void scan_bwd_tile(const TcArgs& a, const Maps& maps, unsigned char* smem_raw, int n, int h,
                                              int tile, long long start, int len) {
  using C = TcCfg<DK, 1, NB, true>;
  constexpr int PL = 1, NC = C::NC, NV = C::NV, NP = 16;
  unsigned char* base = smem_raw + (1024 - (smem_addr(smem_raw) & 1023)) % 1024;
  uint64_t* full = reinterpret_cast<uint64_t*>(base);
  uint64_t *empty = full + 2, *done = full + 4, *outs = full + 6;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(base + 128);
  unsigned char* stage = base + 1024;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long sh = (long long)n * a.s.hv + h;
  const int nc = (len + kC - 1) / kC;
  const long long slot0 = slot_base(start, n);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(full + i, C::FETCH + 1);
      tc::mbar_init(empty + i, 1);             // a chunk's last product
      tc::mbar_init(outs + i, 2 * C::CW);         // the warps that form output rows
      tc::mbar_init(done + i, 1);
    }
    tc::mbar_init_fence();
  }
  if (warp == 0) tc::tmem_alloc(tmem_at, C::TMEM);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_at;
  bool lost = false;        // a wait gave up: no more waiting, the results are void
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!lost && !tc::mbar_wait(bar, parity, kPolls)) {
      lost = true;
      atomicExch(&g_gdr_tc_error, 1);
    }
    lost = __any_sync(0xffffffffu, lost);      // a warp goes on as one
    return !lost;
  };
  // (a warp comes to it as one, and one instruction's answer is the same for all its lanes)
  auto poll = [&](uint64_t* bar, uint32_t parity) {
    if (!lost && !poll_wait(bar, parity, kPollsBusy)) {
      lost = true;
      atomicExch(&g_gdr_tc_error, 1);
    }
  };

  if (tid >= C::WORK) {
    fetch_chunks<DK, C>(a, maps, &maps.v, stage, full, empty, outs, tid - C::WORK, h, start, len, slot0,
                                    tile * NV, true, nullptr, wait);
  } else {
    const int quad = warp & 3, cg = warp >> 2, row = quad * 32 + lane;
    const int v0 = tile * NV, c0 = cg * NC, dk = a.s.dk, dv = a.s.dv;
    const bool token = quad < 2;             // rows of K; else rows of Q
    const bool issuer = quad == 0 && cg == 0;
    const int i = row & 63;                  // the row's token
    unsigned char* stile = stage + 2 * C::STAGE;
    unsigned char* rtile = stile + C::S;
    unsigned char* utile = rtile + C::R;
    unsigned char* otile = utile + C::R;
    const uint32_t d12 = tmem, d3 = tmem + 64 * NB, at = ((uint32_t)(quad * 32) << 16) + c0;
    const uint32_t id_k = tc::idesc(128, 64 * NB, tc::kFmtBF16) | kBmn;
    const uint32_t id_t = tc::idesc(128, 64 * NB, tc::kFmtBF16) | kAmn | kBmn;
    const uint64_t bs = mn_desc(smem_addr(stile), C::SB), bx = mn_desc(smem_addr(rtile), C::RB),
                   bo = mn_desc(smem_addr(otile), C::RB);
    uint32_t phase = 0;
    const bool srow = row < dk && row < DK;
    float s[NC];
#pragma unroll
    for (int j = 0; j < NC; j += 4) {
      const int col = v0 + c0 + j;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (a.init && srow && col < dv) x = *reinterpret_cast<const float4*>(a.init + (sh * dk + row) * dv + col);
      s[j] = x.x; s[j + 1] = x.y; s[j + 2] = x.z; s[j + 3] = x.w;
    }
    for (int it = 0; it < nc; ++it) {
      const int c = nc - 1 - it, st = it & 1;
      unsigned char* b = stage + st * C::STAGE;
      unsigned char* dot = b + C::KQ + C::A2;
      const float* vec = reinterpret_cast<const float*>(b + C::KQ + C::A2 + C::VT);
      const long long img = ((slot0 + c) * a.s.hv + h) * ((dv + 63) / 64) + v0 / 64;
      if (row < DK) {
#pragma unroll
        for (int j = 0; j < NC; j += 8) put8<PL, NB, C::SB>(stile, row, c0 + j, s + j);
      }
      wait(full + st, (it >> 1) & 1);
      const float eg = vec[kVecEG + i], be = vec[kVecBeta + i], el = vec[kVecEGL + i], dec = vec[kVecD];
      if (!token) {
        const float f = a.s.scale * eg;
#pragma unroll
        for (int j = 0; j < NC; j += 8) {
          float w[8];
          unpack8(w, *reinterpret_cast<const uint4*>(dot + v_at<NV>(i, (c0 + j) / 8)));
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] *= f;
          put8<PL, NB, C::RB>(otile, i, c0 + j, w);
        }
      }
      tc::fence_proxy_async_smem();
      tc::fence_before_sync();
      group_sync<1, C::WORK>();
      if (issuer) {
        tc::fence_after_sync();
        const uint64_t ad = tc::sdesc_k_sw128(smem_addr(b));
        const uint64_t aq = mn_desc(smem_addr(b + 8192), DK == 128 ? 16384 : 8192);
        if (tc::elect_one()) {
#pragma unroll
          for (int ks = 0; ks < DK / 16; ++ks)
            tc::mma_bf16(d12, tc::sdesc_advance(ad, (ks >> 2) * 16384 + (ks & 3) * kStepK),
                         tc::sdesc_advance(bs, ks * kStepMN), id_k, ks > 0);
          tc::mma_commit(done);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            tc::mma_bf16(d3, tc::sdesc_advance(aq, ks * kStepMN), tc::sdesc_advance(bo, ks * kStepMN), id_t, ks > 0);
          bulk_store(a.st + img * C::SB, stile, min(NB, (dv - v0 + 63) / 64) * C::SB);
        }
        __syncwarp();
      }
      poll(done, phase);
      phase ^= 1;
      tc::fence_after_sync();
      float r[NC];
      if (token) {
        ld_sum<NC, 1, 0>(d12 + at, r);
#pragma unroll
        for (int j = 0; j < NC; ++j) r[j] *= el;
#pragma unroll
        for (int j = 0; j < NC; j += 8) put8<PL, NB, C::RB>(rtile, i, c0 + j, r + j);
      }
      if (issuer) bulk_store_read();      // dS1 and the last chunk's dR have left their tiles
      tc::fence_proxy_async_smem();
      tc::fence_before_sync();
      group_sync<1, C::WORK>();
      if (issuer) {
        tc::fence_after_sync();
        // transposed: columns of T - I, then of P T (the block after each is not used)
        const uint64_t at_ = mn_desc(smem_addr(b + C::KQ), 8192), ap = mn_desc(smem_addr(b + C::KQ + 8192), 8192);
        const uint64_t bd = mn_desc(smem_addr(dot), 8192);
        if (tc::elect_one()) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            tc::mma_bf16(d12, tc::sdesc_advance(at_, ks * kStepMN), tc::sdesc_advance(bx, ks * kStepMN), id_t, ks > 0);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            tc::mma_bf16(d12, tc::sdesc_advance(ap, ks * kStepMN), tc::sdesc_advance(bd, ks * kStepMN), id_t, 1u);
          tc::mma_commit(done);
        }
        __syncwarp();
      }
      poll(done, phase);
      phase ^= 1;
      tc::fence_after_sync();
      if (token) {
#pragma unroll
        for (int j = 0; j < NC; j += NP) {
          float x[NP];
          ld_sum<NP, PL, C::LO>(d12 + at + j, x);
#pragma unroll
          for (int e = 0; e < NP; ++e) r[j + e] += x[e];
        }
        const float f = -be * eg;
#pragma unroll
        for (int j = 0; j < NC; j += 8) {
          float w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = f * r[j + e];
          put8<PL, NB, C::RB>(rtile, i, c0 + j, w);
          put8<PL, NB, C::RB>(utile, i, c0 + j, r + j);
        }
      }
      tc::fence_proxy_async_smem();
      tc::fence_before_sync();
      group_sync<1, C::WORK>();
      if (issuer) {
        tc::fence_after_sync();
        const uint64_t ak = mn_desc(smem_addr(b), DK == 128 ? 16384 : 8192);
        if (tc::elect_one()) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            tc::mma_bf16(d3, tc::sdesc_advance(ak, ks * kStepMN), tc::sdesc_advance(bx, ks * kStepMN), id_t, 1u);
          tc::mma_commit(done);
          tc::mma_commit(empty + st);
          bulk_store(a.u + img * C::RB, utile, min(NB, (dv - v0 + 63) / 64) * C::RB);
        }
        __syncwarp();
      }
      // While it runs, dv into dO's tile, which the products have read.
      if (token) {
#pragma unroll
        for (int j = 0; j < NC; j += 8) {
          float w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = be * r[j + e];
          *reinterpret_cast<uint4*>(dot + v_at<NV>(i, (c0 + j) / 8)) = pack8(w);
        }
        __syncwarp();
        if (lane == 0) bar_arrive(outs + st);
        __syncwarp();
      }
      poll(done, phase);
      phase ^= 1;
      tc::fence_after_sync();
#pragma unroll
      for (int j = 0; j < NC; j += NP) {
        float x[NP];
        ld_sum<NP, PL, C::LO>(d3 + at + j, x);
#pragma unroll
        for (int e = 0; e < NP; ++e) s[j + e] = fmaf(dec, s[j + e], x[e]);
      }
    }
    if (a.final_state && srow) {
#pragma unroll
      for (int j = 0; j < NC; j += 4)
        if (v0 + c0 + j < dv)
          *reinterpret_cast<float4*>(a.final_state + (sh * dk + row) * dv + v0 + c0 + j) =
              make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
    }
    if (issuer) bulk_store_read();
  }
  if (lost)                  // copies and products that may still be on their way
    for (int j = 0; j < 2; ++j) {
      tc::mbar_wait(full + j, 0, kPolls);
      tc::mbar_wait(done + j, 0, kPolls);
    }
  tc::fence_before_sync();
  __syncwarp();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::TMEM);
  }
}

template <int DK, int NB>
__global__ void __launch_bounds__(TcCfg<DK, 1, NB, true>::THREADS, 1)
    k_gdr_scan_bwd_tc(TcArgs a, const __grid_constant__ Maps maps) {
  extern __shared__ unsigned char smem_raw[];
  const Work w = work_of(a, 0);
  scan_bwd_tile<DK, NB>(a, maps, smem_raw, w.n, w.h, w.tile, w.start, w.len);
}

template <int DK>
__global__ void __launch_bounds__(TcCfg<DK, 1, 2, true>::THREADS, 1)
    k_gdr_scan_bwd_mixed_tc(TcArgs a, const __grid_constant__ Maps maps) {
  extern __shared__ unsigned char smem_raw[];
  const Work w = work_of(a, TcCfg<DK, 1, 2, true>::NV);
  if (w.tile < 0) return;
  if (w.half) {
    if (w.tile * 64 < a.s.dv) scan_bwd_tile<DK, 1>(a, maps, smem_raw, w.n, w.h, w.tile, w.start, w.len);
  } else {
    scan_bwd_tile<DK, 2>(a, maps, smem_raw, w.n, w.h, w.tile, w.start, w.len);
  }
}

// ------------------------------------------------------------------- launches
bool tile_map(CUtensorMap* m, const void* base, int width, int heads, long long rows, long long ld, int box) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<Encode>(p);
  }();
  if (!fn || !base || rows < 1) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)width * 2, (cuuint64_t)ld * 2};
  const cuuint32_t boxes[3] = {(cuuint32_t)box, 1u, (cuuint32_t)kC}, es[3] = {1u, 1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, boxes, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, box == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static int maps_of(const TcArgs& a, int v_box, Maps* m) {
  return tile_map(&m->q, a.q, a.s.dk, a.s.hk, a.s.rows, a.ldq, 64) &&
         tile_map(&m->k, a.k, a.s.dk, a.s.hk, a.s.rows, a.ldk, 64) &&
         tile_map(&m->v, a.v, a.s.dv, a.s.hv, a.s.rows, a.ldv, v_box);
}

template <int DK, int PL, int NB>
static cudaError_t scan(TcArgs a, cudaStream_t st) {
  using C = TcCfg<DK, PL, NB, false>;
  // What the backward reads is kept in tiles of 64 columns: narrower blocks also fill the last one's zeros.
  constexpr int UP = C::NV < 64 ? 64 : C::NV;
  a.ntile = a.st ? (a.s.dv + UP - 1) / UP * (UP / C::NV) : (a.s.dv + C::NV - 1) / C::NV;
  cudaError_t e = allow_smem<k_gdr_scan_tc<DK, PL, NB>>(C::BYTES);
  if (e != cudaSuccess) return e;
  Maps m;
  a.tma = maps_of(a, C::NV < 64 ? C::NV : 64, &m);
  TraceScope tr("k_gdr_scan_tc", st);
  k_gdr_scan_tc<DK, PL, NB><<<(unsigned)((long long)a.s.n_seq * a.s.hv * a.ntile), C::THREADS, C::BYTES, st>>>(a, m);
  return cudaGetLastError();
}
// How many sequences can be so much longer than an even share.
static void allow_half(TcArgs* a, int wide) {
  a->ntile = (a->s.dv + wide - 1) / wide;
  const int most = kNumSMs * 4 / (5 * a->s.hv * a->ntile) + 1;
  a->twice = a->s.n_seq < most ? a->s.n_seq : most;
}
static unsigned mixed_blocks(const TcArgs& a) {
  return (unsigned)((long long)(a.s.n_seq + a.twice) * a.s.hv * a.ntile);
}
template <int DK, int PL>
static cudaError_t scan_mixed(TcArgs a, cudaStream_t st) {
  using W = TcCfg<DK, PL, 2, false>;
  static_assert(W::BYTES >= TcCfg<DK, PL, 1, false>::BYTES && W::THREADS == TcCfg<DK, PL, 1, false>::THREADS, "both fit");
  allow_half(&a, W::NV);
  const cudaError_t e = allow_smem<k_gdr_scan_mixed_tc<DK, PL>>(W::BYTES);
  if (e != cudaSuccess) return e;
  Maps m;
  a.tma = maps_of(a, 64, &m) && (PL == 1 || tile_map(&m.w, a.v, a.s.dv, a.s.hv, a.s.rows, a.ldv, 32));
  TraceScope tr("k_gdr_scan_tc", st);
  k_gdr_scan_mixed_tc<DK, PL><<<mixed_blocks(a), W::THREADS, W::BYTES, st>>>(a, m);
  return cudaGetLastError();
}
template <int DK>
static cudaError_t scan_bwd_mixed(TcArgs a, cudaStream_t st) {
  using W = TcCfg<DK, 1, 2, true>;
  static_assert(W::BYTES >= TcCfg<DK, 1, 1, true>::BYTES && W::THREADS == TcCfg<DK, 1, 1, true>::THREADS, "both fit");
  allow_half(&a, W::NV);
  const cudaError_t e = allow_smem<k_gdr_scan_bwd_mixed_tc<DK>>(W::BYTES);
  if (e != cudaSuccess) return e;
  Maps m;
  a.tma = maps_of(a, 64, &m);
  TraceScope tr("k_gdr_scan_bwd_tc", st);
  k_gdr_scan_bwd_mixed_tc<DK><<<mixed_blocks(a), W::THREADS, W::BYTES, st>>>(a, m);
  return cudaGetLastError();
}
template <int DK, int NB>
static cudaError_t scan_bwd(TcArgs a, cudaStream_t st) {
  using C = TcCfg<DK, 1, NB, true>;
  a.ntile = (a.s.dv + C::NV - 1) / C::NV;
  cudaError_t e = allow_smem<k_gdr_scan_bwd_tc<DK, NB>>(C::BYTES);
  if (e != cudaSuccess) return e;
  Maps m;
  a.tma = maps_of(a, 64, &m);
  TraceScope tr("k_gdr_scan_bwd_tc", st);
  k_gdr_scan_bwd_tc<DK, NB><<<(unsigned)((long long)a.s.n_seq * a.s.hv * a.ntile), C::THREADS, C::BYTES, st>>>(a, m);
  return cudaGetLastError();
}

template <int DK, int PL>
static cudaError_t prep(const FwdArgs& a, cudaStream_t st) {
  using S = PrepTc<DK>;
  cudaError_t e = allow_smem<k_gdr_prep_tc<DK, PL>>(S::BYTES);
  if (e != cudaSuccess) return e;
  TraceScope tr("k_gdr_prep_tc", st);
  k_gdr_prep_tc<DK, PL><<<(unsigned)(slot_count(a.s.rows, a.s.n_seq) * a.s.hv), 128, S::BYTES, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_prep_tc(const FwdArgs& a, int dk_tile, int planes, cudaStream_t st) {
  if (dk_tile == 64) return planes == 2 ? prep<64, 2>(a, st) : prep<64, 1>(a, st);
  return planes == 2 ? prep<128, 2>(a, st) : prep<128, 1>(a, st);
}

// Heads of 128, 1024 tokens, narrow tiles against wide, us:
//   state asked for (32 columns, 64):   32 heads 32, 43;  64 heads  61,  45;  256 heads 205, 162
//   not (64, 128):                      64 heads 36, 52;  96 heads  65,  53;  256 heads 133, 106
//   backward (64, 128):                 64 heads 39, 60;  96 heads  74,  59;  256 heads 145, 119
template <int DK>
static cudaError_t scan_by_size(const TcArgs& t, int planes, cudaStream_t st) {
  const long long heads = (long long)t.s.n_seq * t.s.hv;
  if (planes == 2) {
    if (!wide_tiles(heads, t.s.dv, 32)) return scan<DK, 2, 1>(t, st);
    return t.order ? scan_mixed<DK, 2>(t, st) : scan<DK, 2, 2>(t, st);
  }
  if (!wide_tiles(heads, t.s.dv, 64)) return scan<DK, 1, 1>(t, st);
  return t.order ? scan_mixed<DK, 1>(t, st) : scan<DK, 1, 2>(t, st);
}
template <int DK>
static cudaError_t scan_bwd_by_size(const TcArgs& t, cudaStream_t st) {
  if (!wide_tiles((long long)t.s.n_seq * t.s.hv, t.s.dv, 64)) return scan_bwd<DK, 1>(t, st);
  return t.order ? scan_bwd_mixed<DK>(t, st) : scan_bwd<DK, 2>(t, st);
}

cudaError_t launch_scan_tc(const FwdArgs& a, int dk_tile, int planes, cudaStream_t st) {
  TcArgs t{};
  t.s = a.s;
  t.q = static_cast<const bf16*>(a.q); t.k = static_cast<const bf16*>(a.k); t.v = static_cast<const bf16*>(a.v);
  t.ldq = a.ldq; t.ldk = a.ldk; t.ldv = a.ldv;
  t.init = a.init; t.final_state = a.final_state; t.o = static_cast<bf16*>(a.o);
  t.a2 = reinterpret_cast<const unsigned char*>(a.t);
  t.vec = a.vec;
  t.order = a.order;
  if (a.save) { t.st = reinterpret_cast<unsigned char*>(a.s0); t.u = reinterpret_cast<unsigned char*>(a.u); }
  return dk_tile == 64 ? scan_by_size<64>(t, planes, st) : scan_by_size<128>(t, planes, st);
}

cudaError_t launch_scan_bwd_tc(const BwdArgs& a, int dk_tile, cudaStream_t st) {
  TcArgs t{};
  t.s = a.s;
  t.q = static_cast<const bf16*>(a.q); t.k = static_cast<const bf16*>(a.k); t.v = static_cast<const bf16*>(a.go);
  t.ldq = a.ldq; t.ldk = a.ldk; t.ldv = (long long)a.s.hv * a.s.dv;
  t.init = a.gfinal; t.final_state = a.ginit; t.o = static_cast<bf16*>(a.gv);
  t.a2 = reinterpret_cast<const unsigned char*>(a.t);
  t.vec = a.vec;
  t.order = a.order;
  t.st = reinterpret_cast<unsigned char*>(a.ds); t.u = reinterpret_cast<unsigned char*>(a.dr);
  return dk_tile == 64 ? scan_bwd_by_size<64>(t, st) : scan_bwd_by_size<128>(t, st);
}

int* gdr_tc_error_word() {
  void* p = nullptr;
  return cudaGetSymbolAddress(&p, g_gdr_tc_error) == cudaSuccess ? static_cast<int*>(p) : nullptr;
}

}  // namespace gdr
}  // namespace cfc
