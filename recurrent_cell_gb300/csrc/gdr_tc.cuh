// gdr_tc.cuh -- tensor-core pieces of the gated delta rule's bf16 kernels:
// operand tiles of 64 columns (128 bytes a row, 128-byte swizzle), their
// descriptors, accumulator reads, and copies of tiles to global memory.
//
// A tile's rows are tokens or key indexes, its columns what lies contiguous in
// memory.  Read with a K-major descriptor its columns are contracted, read with
// an MN-major one its rows are: the same tile serves both.
#pragma once

#include <cuda.h>

#include "gdr_common.cuh"

namespace cfc {
namespace gdr {

// Tensor maps of [rows, heads, width] bf16 tensors: boxes of up to 64 columns
// of one head by a chunk's 64 rows, zeros past the width.  w: the gradients'
// grad_o; in a scan of both widths with PL = 2, v in boxes of 32 columns.
struct Maps {
  CUtensorMap q, k, v, w;
};
// False: the driver cannot say (the kernels then copy by 16 bytes).
bool tile_map(CUtensorMap* m, const void* base, int width, int heads, long long rows, long long ld, int box);

__device__ __forceinline__ void tma_tile(void* dst, const CUtensorMap* map, int col, int head, int row, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(col), "r"(head), "r"(row), "r"(smem_addr(bar))
      : "memory");
}

using bf16 = __nv_bfloat16;

__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr, uint32_t next_block) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)(next_block >> 4) << 16;    // the next 64 columns
  d |= (uint64_t)(1024u >> 4) << 32;         // the next 8 rows
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}
constexpr uint32_t kAmn = 1u << 15, kBmn = 1u << 16;
constexpr uint32_t kStepK = 32, kStepMN = 2048;    // bytes of 16 along K

__device__ __forceinline__ uint32_t chunk_at(int row, int ch) { return row * 128 + ((ch ^ (row & 7)) << 4); }

// N accumulator columns of this warp's lanes; PL = 2: the columns LO on, the
// products of the lo plane, added.
template <int N>
__device__ __forceinline__ void ld_cols(uint32_t t, float* v) {
  static_assert(N % 16 == 0, "columns");
#pragma unroll
  for (int j = 0; j + 16 <= N; j += 16) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(t + j)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[j + i] = __uint_as_float(r[i]);
  }
}
// The loads above are valid after this: it holds their registers back.
template <int N>
__device__ __forceinline__ void ld_wait(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i])::"memory");
}
template <int N, int PL, int LO>
__device__ __forceinline__ void ld_sum(uint32_t t, float (&v)[N]) {
  ld_cols<N>(t, v);
  if constexpr (PL == 2) {
    float w[N];
    ld_cols<N>(t + LO, w);
    ld_wait<N>(v);
    ld_wait<N>(w);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += w[i];
  } else {
    ld_wait<N>(v);
  }
}

// Bounded wait by polling: the products' round trips are the serial passes'
// time, and a poll answers some 80 cycles sooner than a suspended wait.
__device__ __forceinline__ bool poll_wait(uint64_t* bar, uint32_t parity, uint32_t max_polls) {
  for (uint32_t i = 0; i < max_polls; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
  }
  return false;
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}
__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ void unpack8(float* v, const uint4& u) {
  v[0] = lo_f(u.x); v[1] = hi_f(u.x); v[2] = lo_f(u.y); v[3] = hi_f(u.y);
  v[4] = lo_f(u.z); v[5] = hi_f(u.z); v[6] = lo_f(u.w); v[7] = hi_f(u.w);
}
// z + 0 x eight bf16 values: zeros as long as all of them are finite.
__device__ __forceinline__ __nv_bfloat162 times_zero(const uint4& u, __nv_bfloat162 z) {
  const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162*>(&u), o = __float2bfloat162_rn(0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) z = __hfma2(p[i], o, z);
  return z;
}
__device__ __forceinline__ bool zeros(__nv_bfloat162 z) {
  return (*reinterpret_cast<const uint32_t*>(&z) & 0x7fff7fffu) == 0;
}
// Shared -> global copy of a tile by the calling thread, and the wait until
// its copies have read their tiles.
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_addr(src)), "r"(bytes)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void bulk_store_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// Row r, 16-byte piece ch of a V, dO or output tile of NV columns (blocks of 64).
template <int NV>
__device__ __forceinline__ uint32_t v_at(int r, int ch) {
  if (NV < 64) return r * 64 + ((ch ^ ((r >> 1) & 3)) << 4);
  return (NV > 64 ? (ch >> 3) * 8192 : 0) + chunk_at(r, ch & 7);
}
// The warp's 32 rows (from r0) x NC columns (from piece ch0) of such a tile to
// rows of global memory, 16 bytes a lane, whole rows side by side.  Rows from
// row_end and columns from col_end on are left out.
template <int NV, int NC>
__device__ __forceinline__ void rows_out(bf16* dst, long long ld, const unsigned char* tile, int r0, int ch0, int row_end,
                                         int col_end, int lane) {
  constexpr int PC = NC / 8, RP = 32 / PC;
  const int ch = ch0 + lane % PC, r = r0 + lane / PC;
  bf16* p = dst + r * ld + ch * 8;
  uint4 v[PC];
#pragma unroll
  for (int i = 0; i < PC; ++i) v[i] = *reinterpret_cast<const uint4*>(tile + v_at<NV>(r + i * RP, ch));
  if (ch * 8 < col_end) {
#pragma unroll
    for (int i = 0; i < PC; ++i)
      if (r + i * RP < row_end) *reinterpret_cast<uint4*>(p + i * RP * ld) = v[i];
  }
}

}  // namespace gdr
}  // namespace cfc
