// cfc_gdr_grad.cu -- the parallel part of the gated delta rule's backward in
// bf16 on the tensor cores: dq, dk, dg, dbeta of every chunk (formulas at the
// top of cfc_gdr_bwd.cu, notation of gdr_common.cuh).
//
// Persistent blocks, one an SM, take a chunk of a key head at a time and walk
// over its value heads, whose parts of dq and dk add up in registers.  A head
// takes five products; rows 0-63 and 64-127 of the accumulators are tokens:
//   D1 = [dR; dO] S0^T     X                 | S0 dO
//   D2 = [dR; dO] U^T      dR_i.U_j          | dO_i.U_j
//   D3 = [U; dR] dS1^T     dS1 U             | (not used)
//   D4 = [dA; dP] K        of E              | of dq
//   D5 = dP^T Q + (beta dA)^T K   of dk      | (not used)
// with dA = -L o D2 strictly below the diagonal and dP = scale L o D2 up to it,
// each in two bf16 planes: dg is a difference of their sums.  S0, U, dS1 and dR
// come as operand tiles, as the serial passes left them; with the inputs they
// are the traffic (about 160 KB a chunk and head in, 32 KB out).  Two warps
// keep two 64-column stages and the next chunk's K and Q on their way, one
// issues the products, eight do the arithmetic between them; a head's first
// products run under the last one's end.  194 KB a chunk and head of 128 x 128
// in 41 ns, 4.8 TB/s (8 x 2048 x 16 heads 167 us): 71 % of a copy's rate.  What
// holds it below is latency: the 11 warps of an SM wait for shared and tensor
// memory in 44 % of the samples, and DRAM is active in 62 % of the cycles.  (With
// shared heads and d_k = 128 the sums over a group cost 220 bytes of spills a thread;
// 16 value on 8 key heads take the whole call from 460 us to 502.)
#include "gdr_tc.cuh"

namespace cfc {
namespace gdr {

__device__ int g_gdr_grad_error = 0;

struct GradArgs {
  Shape s;
  const bf16 *q, *k, *v, *go;
  long long ldq, ldk, ldv;
  bf16 *gq, *gk, *gg, *gbeta;
  const unsigned char *s0, *u, *ds, *dr;
  const float* vec;
  int tma;
};

template <int DK>
struct GradCfg {
  static constexpr int ATOMS = DK / 64, FETCH = 64, WORK = 256, THREADS = WORK + FETCH + 32;
  static constexpr uint32_t T = 8192;                   // 64 rows x 128 bytes
  static constexpr uint32_t S = DK * 128u;
  // a stage: U, dR, dO, V, S0, dS1 of 64 value columns, the vectors
  static constexpr uint32_t OFF_DO = 2 * T, OFF_V = 3 * T, OFF_S0 = 4 * T, OFF_DS = OFF_S0 + S, OFF_VEC = OFF_DS + S;
  static constexpr uint32_t STAGE = OFF_VEC + 2048;     // + what the chunk is
  static constexpr uint32_t OPS = 6 * T;                // dA, dP, beta dA; then their lo planes
  static constexpr uint32_t KQ = 2 * ATOMS * T;
  static constexpr uint32_t SMALL = (4 * 2 * 64 + 4 * 64 + 8 + 128) * 4;
  static constexpr uint32_t BYTES = 2048 + 2 * STAGE + OPS + KQ + SMALL;
  static_assert(BYTES <= 227u * 1024u, "shared memory");
};

struct Chunk {
  long long row0, slot;
  int rows, hk;           // rows < 0: no more
};

// SHARED: several value heads to a key head, dq and dk added up in registers.
template <int DK, bool SHARED>
__global__ void __launch_bounds__(GradCfg<DK>::THREADS, 1) k_gdr_grad_tc(GradArgs a, const __grid_constant__ Maps maps) {
  extern __shared__ unsigned char smem_raw[];
  using C = GradCfg<DK>;
  unsigned char* base = smem_raw + (1024 - (smem_addr(smem_raw) & 1023)) % 1024;
  uint64_t* full = reinterpret_cast<uint64_t*>(base);      // stages 0, 1; K and Q
  uint64_t *empty = full + 3, *done = full + 6;            // done: D1 - D3; D4, D5
  uint64_t *ops_in = full + 8, *acc_out = full + 9;        // dA, dP are there; the accumulators have been read
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(base + 128);
  unsigned char* stage = base + 1024;
  unsigned char* ops = stage + 2 * C::STAGE;
  unsigned char* kq = ops + C::OPS;
  float* dot = reinterpret_cast<float*>(kq + C::KQ);       // [4][2][64]: q.dq, k.dk, k.E, k.dS1 U
  float *drv = dot + 4 * 2 * 64, *sums = drv + 4 * 64, *gs = sums + 8;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = a.s.hv / a.s.hk, dk = a.s.dk, dv = a.s.dv, nt = (dv + 63) / 64;
  if (tid == 0) {
    for (int i = 0; i < 3; ++i) {
      tc::mbar_init(full + i, C::FETCH + 1);
      tc::mbar_init(empty + i, C::WORK / 32 + (i < 2 ? 1 : 0));        // K and Q: dk and dq lie in their place
    }
    tc::mbar_init(done, 1);
    tc::mbar_init(done + 1, 1);
    tc::mbar_init(ops_in, C::WORK / 32);
    tc::mbar_init(acc_out, C::WORK / 32);
    tc::mbar_init_fence();
  }
  if (warp == 0) tc::tmem_alloc(tmem_at, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_at;
  bool lost = false;        // a wait gave up: no more waiting, the results are void
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!lost && !tc::mbar_wait(bar, parity, kPolls)) {
      lost = true;
      atomicExch(&g_gdr_grad_error, 1);
    }
    lost = __any_sync(0xffffffffu, lost);      // a warp goes on as one
  };

  if (tid >= C::WORK && tid < C::WORK + C::FETCH) {     // ---- the fetching warps
    const int ft = tid - C::WORK;
    uint64_t* pending = nullptr;           // copies under way whose arrival is still to come
    auto flush = [&]() {
      if (!pending) return;
      cp_wait<0>();
      tc::fence_proxy_async_smem();
      bar_arrive(pending);
      pending = nullptr;
    };
    auto claim = [&](int i, uint32_t use) {      // buffer i for its use-th time
      if (use == 0) return;
      if (__all_sync(0xffffffffu, !lost && tc::mbar_try_wait(empty + i, (use - 1) & 1))) return;
      flush();
      wait(empty + i, (use - 1) & 1);
    };
    auto issued = [&](uint64_t* bar) {
      cp_commit();
      if (pending) {
        cp_wait<1>();
        tc::fence_proxy_async_smem();
        bar_arrive(pending);
      }
      pending = bar;
    };
    uint32_t it = 0, kqi = 0;
    Chunk last{};
    // dk and dq of the chunk before, from K's and Q's tiles
    auto rows_of = [&](const Chunk& c) {
      flush();
      wait(empty + 2, (kqi - 1) & 1);
      const bool q = ft >= 32;             // a warp each
#pragma unroll 1
      for (int r0 = 0; r0 < kC; r0 += 32)
#pragma unroll
        for (int b = 0; b < C::ATOMS; ++b)
          rows_out<64, 64>((q ? a.gq : a.gk) + (c.row0 * a.s.hk + c.hk) * dk + b * 64, (long long)a.s.hk * dk,
                           kq + (q ? C::ATOMS + b : b) * C::T, r0, 0, c.rows, dk - b * 64, lane);
      // the tiles are filled again by other threads
      group_sync<2, C::FETCH>();
    };
    const long long ldo = (long long)a.s.hv * dv;
    const long long items = slot_count(a.s.rows, a.s.n_seq) * a.s.hk;
    for (long long item = blockIdx.x; item < items; item += gridDim.x) {
      if (group_any<2, C::FETCH>(lost)) break;       // nothing more is fetched after a wait that gave up
      const long long slot = item / a.s.hk;
      const int hk = (int)(item % a.s.hk);
      int n, len, c;
      long long start;
      if (!slot_chunk(a.s, slot, &n, &start, &len, &c)) continue;
      const long long row0 = start + (long long)c * kC;
      const int rows = min(kC, len - c * kC);
      const bool boxes = a.tma && rows == kC;    // else 16-byte copies: rows past a sequence's end are zeros
      for (int g = 0; g < group; ++g) {
        const int h = hk * group + g;
        const long long id = slot * a.s.hv + h;
        const bf16 *go = a.go + row0 * ldo + (long long)h * dv, *v = a.v + row0 * a.ldv + (long long)h * dv;
        for (int t = 0; t < nt; ++t, ++it) {
          const int st = it & 1;
          claim(st, it >> 1);
          unsigned char* b = stage + st * C::STAGE;
          if (ft == 0) {
            bar_arrive_tx(full + st, 2 * C::T + 2 * C::S + kVec * 4 + (boxes ? 2 * C::T : 0));
            if (boxes) {
              tma_tile(b + C::OFF_DO, &maps.w, t * 64, h, (int)row0, full + st);
              tma_tile(b + C::OFF_V, &maps.v, t * 64, h, (int)row0, full + st);
            }
            bulk_load(b, a.u + (id * nt + t) * C::T, C::T, full + st);
            bulk_load(b + C::T, a.dr + (id * nt + t) * C::T, C::T, full + st);
            bulk_load(b + C::OFF_S0, a.s0 + (id * nt + t) * C::S, C::S, full + st);
            bulk_load(b + C::OFF_DS, a.ds + (id * nt + t) * C::S, C::S, full + st);
            bulk_load(b + C::OFF_VEC, a.vec + id * kVec, kVec * 4, full + st);
            *reinterpret_cast<Chunk*>(b + C::OFF_VEC + kVec * 4) = Chunk{row0, slot, rows, hk};
          }
          if (boxes) {
            bar_arrive(full + st);
            continue;
          }
          const int ch = ft & 7, col = t * 64 + ch * 8;
#pragma unroll
          for (int r = ft >> 3; r < kC; r += C::FETCH / 8) {
            const bool on = r < rows && col < dv;
            cp16(b + C::OFF_DO + chunk_at(r, ch), on ? go + r * ldo + col : go, on);
            cp16(b + C::OFF_V + chunk_at(r, ch), on ? v + r * a.ldv + col : v, on);
          }
          issued(full + st);
        }
        if (g == 0) {
          if (kqi > 0) rows_of(last);
          ++kqi;
          last = Chunk{row0, slot, rows, hk};
          const bf16 *k = a.k + row0 * a.ldk + (long long)hk * dk, *q = a.q + row0 * a.ldq + (long long)hk * dk;
          if (ft == 0) {
            tc::fence_proxy_async_smem();        // dk and dq were written where boxes now go
            bar_arrive_tx(full + 2, boxes ? C::KQ : 0);
            if (boxes)
#pragma unroll
              for (int x = 0; x < C::ATOMS; ++x) {
                tma_tile(kq + x * C::T, &maps.k, x * 64, hk, (int)row0, full + 2);
                tma_tile(kq + (C::ATOMS + x) * C::T, &maps.q, x * 64, hk, (int)row0, full + 2);
              }
          }
          if (boxes) {
            bar_arrive(full + 2);
            continue;
          }
          constexpr int PER = DK / 8;
          const int ch = ft % PER;
          unsigned char* d = kq + (ch >> 3) * C::T;
#pragma unroll 4
          for (int r = ft / PER; r < kC; r += C::FETCH / PER) {
            const bool on = r < rows && ch * 8 < dk;
            cp16(d + chunk_at(r, ch & 7), on ? k + r * a.ldk + ch * 8 : k, on);
            cp16(d + C::ATOMS * C::T + chunk_at(r, ch & 7), on ? q + r * a.ldq + ch * 8 : q, on);
          }
          issued(full + 2);
        }
      }
    }
    flush();
    if (kqi > 0) rows_of(last);
    claim(it & 1, it >> 1);
    if (ft == 0) {
      reinterpret_cast<Chunk*>(stage + (it & 1) * C::STAGE + C::OFF_VEC + kVec * 4)->rows = -1;
      bar_arrive_tx(full + (it & 1), 0);
    }
    bar_arrive(full + (it & 1));
  } else if (tid >= C::WORK) {   // ---- the warp that issues the products
    const uint32_t d1 = tmem, d3 = tmem + 128, d4 = tmem + 256, d5 = tmem + 384, d2 = d5;
    const uint32_t id_dk = tc::idesc(128, DK, tc::kFmtBF16), id_64 = tc::idesc(128, 64, tc::kFmtBF16);
    const uint64_t ap = tc::sdesc_k_sw128(smem_addr(ops)), tp = mn_desc(smem_addr(ops + C::T), C::T),
                   tm = mn_desc(smem_addr(ops + 2 * C::T), C::T), bk = mn_desc(smem_addr(kq), C::T),
                   bq = mn_desc(smem_addr(kq + C::ATOMS * C::T), C::T);
    uint32_t it = 0, kqi = 0;
    int g = 0;
    for (uint32_t heads = 0;; ++heads) {
      for (int t = 0; t < nt; ++t, ++it) {
        const int st = it & 1;
        unsigned char* b = stage + st * C::STAGE;
        wait(full + st, (it >> 1) & 1);
        if (t == 0) {
          if (__any_sync(0xffffffffu, lost || reinterpret_cast<const Chunk*>(b + C::OFF_VEC + kVec * 4)->rows < 0)) goto over;
          if (heads > 0) wait(acc_out, (heads - 1) & 1);
        }
        tc::fence_after_sync();
        const uint64_t au = tc::sdesc_k_sw128(smem_addr(b)), ar = tc::sdesc_k_sw128(smem_addr(b + C::T)),
                       b0 = tc::sdesc_k_sw128(smem_addr(b + C::OFF_S0)), bd = tc::sdesc_k_sw128(smem_addr(b + C::OFF_DS));
        if (tc::elect_one()) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint32_t o = ks * kStepK, ac = (t > 0 || ks > 0) ? 1u : 0u;
            tc::mma_bf16(d2, tc::sdesc_advance(ar, o), tc::sdesc_advance(au, o), id_64, ac);
            tc::mma_bf16(d1, tc::sdesc_advance(ar, o), tc::sdesc_advance(b0, o), id_dk, ac);
            tc::mma_bf16(d3, tc::sdesc_advance(au, o), tc::sdesc_advance(bd, o), id_dk, ac);
          }
          tc::mma_commit(empty + st);
          if (t == nt - 1) tc::mma_commit(done);
        }
        __syncwarp();
      }
      wait(ops_in, heads & 1);
      if (g == 0) wait(full + 2, kqi & 1);
      if (++g == group) {
        g = 0;
        ++kqi;
      }
      tc::fence_after_sync();
      if (tc::elect_one()) {
#pragma unroll
        for (int pl = 0; pl < 2; ++pl)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint32_t lo = pl * 3 * C::T, ac = pl + ks > 0 ? 1u : 0u;
            const uint64_t kd = tc::sdesc_advance(bk, ks * kStepMN), qd = tc::sdesc_advance(bq, ks * kStepMN);
            tc::mma_bf16(d4, tc::sdesc_advance(ap, lo + ks * kStepK), kd, id_dk | kBmn, ac);
            tc::mma_bf16(d5, tc::sdesc_advance(tp, lo + ks * kStepMN), qd, id_dk | kAmn | kBmn, ac);
            tc::mma_bf16(d5, tc::sdesc_advance(tm, lo + ks * kStepMN), kd, id_dk | kAmn | kBmn, 1u);
          }
        tc::mma_commit(done + 1);
      }
      __syncwarp();
    }
  over:;
  } else {
    constexpr int NC = DK / 2;             // columns of dq, dk a thread
    const int quad = warp & 3, cg = warp >> 2, row = quad * 32 + lane, i = row & 63;
    const bool lower = quad < 2;
    const uint32_t d1 = tmem, d3 = tmem + 128, d4 = tmem + 256, d5 = tmem + 384, d2 = d5;
    const uint32_t at = (uint32_t)(quad * 32) << 16;
    unsigned char* krow = kq + (DK == 128 ? cg * C::T : 0);          // the block of this thread's columns
    unsigned char* tile = lower ? krow : krow + C::ATOMS * C::T;     // K, then dk; Q, then dq
    const int ch0 = DK == 128 ? 0 : cg * 4;
    uint32_t it = 0;
    float acc[SHARED ? NC : 1];            // dk of the chunk (rows 0-63), dq
    int g = 0;
    for (uint32_t heads = 0;; ++heads) {
      wait(full + (it & 1), (it >> 1) & 1);
      const Chunk ck = *reinterpret_cast<const Chunk*>(stage + (it & 1) * C::STAGE + C::OFF_VEC + kVec * 4);
      // a wait that gave up ends it for all at once, so that nobody stays behind at a barrier
      if (group_any<1, C::WORK>(ck.rows < 0 || lost)) break;
      const float* vec = reinterpret_cast<const float*>(stage + (it & 1) * C::STAGE + C::OFF_VEC);
      const float eg = vec[kVecEG + i], el = vec[kVecEGL + i], be = vec[kVecBeta + i], dec = vec[kVecD];
      const float2 be2 = *reinterpret_cast<const float2*>(vec + kVecBeta + 2 * lane);
      const uint2 dead = *reinterpret_cast<const uint2*>(vec + kVecDead);
      if (tid < 128) gs[tid] = vec[kVecG2 + tid];
      float ss = 0.f, dr = 0.f;            // <S0, dS1> and dR.v, while the products run
      for (int t = 0; t < nt; ++t, ++it) {
        const int st = it & 1;
        unsigned char* b = stage + st * C::STAGE;
        if (t > 0) wait(full + st, (it >> 1) & 1);
#pragma unroll 2
        for (int e = 0; e < DK * 8 / C::WORK; ++e) {
          const uint32_t o = (e * C::WORK + tid) * 16;
          float x[8], y[8];
          unpack8(x, *reinterpret_cast<const uint4*>(b + C::OFF_S0 + o));
          unpack8(y, *reinterpret_cast<const uint4*>(b + C::OFF_DS + o));
#pragma unroll
          for (int z = 0; z < 8; ++z) ss = fmaf(x[z], y[z], ss);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t o = chunk_at(tid & 63, (tid >> 6) * 2 + e);
          float x[8], y[8];
          unpack8(x, *reinterpret_cast<const uint4*>(b + C::T + o));
          unpack8(y, *reinterpret_cast<const uint4*>(b + C::OFF_V + o));
#pragma unroll
          for (int z = 0; z < 8; ++z) dr = fmaf(x[z], y[z], dr);
        }
        __syncwarp();
        if (lane == 0) bar_arrive(empty + st);
      }
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
      group_sync<1, C::WORK>();            // gs is there; warp 7 has done the last head's sums
      drv[tid] = dr;
      if (lane == 0) sums[warp] = ss;
      wait(done, heads & 1);
      tc::fence_after_sync();
      {
        const float2 gi = reinterpret_cast<const float2*>(gs)[i];
        const float f = lower ? -1.f : a.s.scale;
        const int end = cg * 32 <= i ? (lower ? i : i + 1) : 0;    // columns that count
        unsigned char* to = ops + (lower ? 0 : C::T);
#pragma unroll 1
        for (int j = 0; j < 32; j += 16) {
          float x[16];
          ld_sum<16, 1, 0>(d2 + at + cg * 32 + j, x);
#pragma unroll
          for (int z = 0; z < 16; z += 8) {
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const int col = cg * 32 + j + z + e;
              const float4 gj = *reinterpret_cast<const float4*>(gs + 2 * col);
              const float w0 = f * x[z + e] * exp2_approx((gi.x - gj.x) + (gi.y - gj.y));
              const float w1 = f * x[z + e + 1] * exp2_approx((gi.x - gj.z) + (gi.y - gj.w));
              w[e] = col < end ? w0 : 0.f;
              w[e + 1] = col + 1 < end ? w1 : 0.f;
            }
            const uint32_t o = chunk_at(i, cg * 4 + (j + z) / 8);
            auto two = [&](unsigned char* p) {
              const uint4 h = pack8(w);
              *reinterpret_cast<uint4*>(p + o) = h;
              float hv[8];
              unpack8(hv, h);
#pragma unroll
              for (int e = 0; e < 8; ++e) hv[e] = w[e] - hv[e];
              *reinterpret_cast<uint4*>(p + 3 * C::T + o) = pack8(hv);
            };
            two(to);
            if (lower) {
#pragma unroll
              for (int e = 0; e < 8; ++e) w[e] *= be;
              two(ops + 2 * C::T);
            }
          }
        }
      }
      tc::fence_proxy_async_smem();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) bar_arrive(ops_in);
      wait(done + 1, heads & 1);
      tc::fence_after_sync();
      float s0 = 0.f, s1 = 0.f, s2 = 0.f;  // k.dk or q.dq; k.E; k.dS1 U
      const float f = lower ? -eg : a.s.scale * eg;
      // 16 columns from j of dk or dq
      auto part = [&](int j, float* d) {
        const uint32_t o = at + cg * NC + j;
        float x[16], y[16], u[16], p[16];
        ld_cols<16>(d1 + o, x);
        ld_cols<16>(d4 + o, y);
        if (lower) {
          ld_cols<16>(d3 + o, u);
          ld_cols<16>(d5 + o, p);
        }
        ld_wait<16>(x);
        ld_wait<16>(y);
        if (lower) {
          ld_wait<16>(u);
          ld_wait<16>(p);
        }
#pragma unroll
        for (int z = 0; z < 16; z += 8) {
          float kk[8];
          unpack8(kk, *reinterpret_cast<const uint4*>(tile + chunk_at(i, ch0 + (j + z) / 8)));
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float en = fmaf(f, x[z + e], y[z + e]);
            float dd = en;
            if (lower) {
              const float us = el * u[z + e];
              s1 = fmaf(kk[e], en, s1);
              s2 = fmaf(kk[e], us, s2);
              dd = fmaf(be, en, us + p[z + e]);
            }
            s0 = fmaf(kk[e], dd, s0);
            d[z + e] = dd;
          }
        }
      };
      if constexpr (SHARED) {
#pragma unroll
        for (int j = 0; j < NC; j += 16) {
          float d[16];
          part(j, d);
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[j + e] = g == 0 ? d[e] : acc[j + e] + d[e];
        }
      } else {
#pragma unroll 1
        for (int j = 0; j < NC; j += 16) {
          float d[16];
          part(j, d);                      // K or Q has been read there: the result takes its place
          *reinterpret_cast<uint4*>(tile + chunk_at(i, ch0 + j / 8)) = pack8(d);
          *reinterpret_cast<uint4*>(tile + chunk_at(i, ch0 + j / 8 + 1)) = pack8(d + 8);
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) bar_arrive(acc_out);
      if (lower) {
        dot[128 + cg * 64 + i] = s0;
        dot[256 + cg * 64 + i] = s1;
        dot[384 + cg * 64 + i] = s2;
      } else {
        dot[cg * 64 + i] = s0;
      }
      const int h = ck.hk * group + g;
      if (++g == group) {                  // the fetching warps take dk and dq from K's and Q's place
        g = 0;
        if constexpr (SHARED)
#pragma unroll
          for (int j = 0; j < NC; j += 8) *reinterpret_cast<uint4*>(tile + chunk_at(i, ch0 + j / 8)) = pack8(acc + j);
        __syncwarp();
        if (lane == 0) bar_arrive(empty + 2);
      }
      group_sync<1, C::WORK>();
      if (warp == 7) {
        // dbeta, and dg: the sums of dG from each row to the chunk's end
        float dg[2], us = 0.f, tot = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 2 * lane + e;
          const float z = dot[256 + r] + dot[320 + r];
          const float db = ((drv[r] + drv[64 + r]) + (drv[128 + r] + drv[192 + r])) + z;
          dg[e] = (dot[r] + dot[64 + r]) - (dot[128 + r] + dot[192 + r]) + 2.f * (e ? be2.y : be2.x) * z;
          us += dot[384 + r] + dot[448 + r];
          if (r < ck.rows) a.gbeta[(ck.row0 + r) * a.s.hv + h] = __float2bfloat16_rn(db);
        }
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) us += __shfl_xor_sync(0xffffffffu, us, m);
#pragma unroll
        for (int m = 0; m < 8; ++m) tot += sums[m];
        const float last = fmaf(dec, tot, us);
        float run = dg[0] + dg[1];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const float y = __shfl_down_sync(0xffffffffu, run, d);
          run += lane + d < 32 ? y : 0.f;
        }
        const float g0 = alive(run + last, dead.x, lane), g1 = alive(run - dg[0] + last, dead.y, lane);
        if (2 * lane < ck.rows) a.gg[(ck.row0 + 2 * lane) * a.s.hv + h] = __float2bfloat16_rn(g0);
        if (2 * lane + 1 < ck.rows) a.gg[(ck.row0 + 2 * lane + 1) * a.s.hv + h] = __float2bfloat16_rn(g1);
      }
    }
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
    tc::tmem_dealloc(tmem, 512);
  }
}

template <int DK, bool SHARED>
static cudaError_t launch(GradArgs g, cudaStream_t st) {
  using C = GradCfg<DK>;
  const long long items = slot_count(g.s.rows, g.s.n_seq) * g.s.hk;
  cudaError_t e = allow_smem<k_gdr_grad_tc<DK, SHARED>>(C::BYTES);
  if (e != cudaSuccess) return e;
  Maps m;
  g.tma = tile_map(&m.q, g.q, g.s.dk, g.s.hk, g.s.rows, g.ldq, 64) &&
          tile_map(&m.k, g.k, g.s.dk, g.s.hk, g.s.rows, g.ldk, 64) &&
          tile_map(&m.v, g.v, g.s.dv, g.s.hv, g.s.rows, g.ldv, 64) &&
          tile_map(&m.w, g.go, g.s.dv, g.s.hv, g.s.rows, (long long)g.s.hv * g.s.dv, 64);
  TraceScope tr("k_gdr_grad_tc", st);
  k_gdr_grad_tc<DK, SHARED><<<(unsigned)(items < kNumSMs ? items : kNumSMs), C::THREADS, C::BYTES, st>>>(g, m);
  return cudaGetLastError();
}

cudaError_t launch_grad_tc(const BwdArgs& a, int dk_tile, cudaStream_t st) {
  GradArgs g{};
  g.s = a.s;
  g.q = static_cast<const bf16*>(a.q); g.k = static_cast<const bf16*>(a.k);
  g.v = static_cast<const bf16*>(a.v); g.go = static_cast<const bf16*>(a.go);
  g.ldq = a.ldq; g.ldk = a.ldk; g.ldv = a.ldv;
  g.gq = static_cast<bf16*>(a.gq); g.gk = static_cast<bf16*>(a.gk);
  g.gg = static_cast<bf16*>(a.gg); g.gbeta = static_cast<bf16*>(a.gbeta);
  g.s0 = reinterpret_cast<const unsigned char*>(a.s0); g.u = reinterpret_cast<const unsigned char*>(a.u);
  g.ds = reinterpret_cast<const unsigned char*>(a.ds); g.dr = reinterpret_cast<const unsigned char*>(a.dr);
  g.vec = a.vec;
  if (a.s.hv == a.s.hk) return dk_tile == 64 ? launch<64, false>(g, st) : launch<128, false>(g, st);
  return dk_tile == 64 ? launch<64, true>(g, st) : launch<128, true>(g, st);
}

int* gdr_grad_error_word() {
  void* p = nullptr;
  return cudaGetSymbolAddress(&p, g_gdr_grad_error) == cudaSuccess ? static_cast<int*>(p) : nullptr;
}

}  // namespace gdr
}  // namespace cfc
