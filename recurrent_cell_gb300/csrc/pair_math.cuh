// pair_math.cuh -- arithmetic on two floats at a time, and the fast elementary functions.
#pragma once

#include <stdint.h>

#include "cfc_internal.cuh"

namespace cfc {
namespace pairs {

constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ float min_nan(float a, float b) {     // a NaN stays
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Two floats at a time: kernels that are bound by instructions issued do the work of two with one.
using F2 = unsigned long long;
__device__ __forceinline__ F2 pack(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 twice(float a) { return pack(a, a); }
__device__ __forceinline__ void split(F2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 ex2_2(F2 v) {
  float a, b;
  split(v, a, b);
  return pack(ex2(a), ex2(b));
}
__device__ __forceinline__ float sum2(F2 v) {
  float a, b;
  split(v, a, b);
  return a + b;
}

// 1 / (1 + exp(-v)) of two values: 0 where the exponential is infinite.
__device__ __forceinline__ F2 sigmoid2(F2 v) {
  const F2 e = add2(ex2_2(mul2(v, twice(-kLog2e))), twice(1.f));
  float a, b;
  split(e, a, b);
  return pack(rcp(a), rcp(b));
}
__device__ __forceinline__ float sigmoid(float v) { return rcp(1.f + ex2(v * -kLog2e)); }
// The same with the exponent's rounding put right, for outputs in fp32.
__device__ __forceinline__ F2 sigmoid2_exact(F2 v) {
  const F2 x = mul2(v, twice(-kLog2e)), off = fma2(v, twice(kLog2e), x);      // x less the exact product
  const F2 e = ex2_2(x);
  float a, b, ea, eb, fa, fb;
  split(fma2(mul2(e, off), twice(-kLn2), e), a, b);
  split(e, ea, eb);
  split(x, fa, fb);
  a = 1.f + (fabsf(fa) < 126.f ? a : ea);      // (an infinite product has no part to put right)
  b = 1.f + (fabsf(fb) < 126.f ? b : eb);
  return pack(rcp(a), rcp(b));
}

// 16 bytes of global memory, or zeros.  One opaque statement: from a branch and a load the
// compiler makes a read whose value is unpacked, and so waited for, at once.
__device__ __forceinline__ uint4 load_here(const void* p, bool on = true) {
  uint4 v;
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %5, 0;\n mov.b32 %0, 0;\n mov.b32 %1, 0;\n mov.b32 %2, 0;\n mov.b32 %3, 0;\n"
      " @p ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"((int)on));
  return v;
}

// What was read ahead may be used from here on, and not before: the compiler would move its
// unpacking up to the read, and the wait for it with it.
__device__ __forceinline__ void use_here(uint4& v) { asm volatile("" : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)); }
__device__ __forceinline__ void use_here(float& v) { asm volatile("" : "+f"(v)); }
__device__ __forceinline__ float load_here4(const float* p, bool on = true) {
  float v;
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %2, 0;\n mov.b32 %0, 0;\n @p ld.global.nc.f32 %0, [%1];\n}"
               : "=&f"(v)
               : "l"(p), "r"((int)on));
  return v;
}
__device__ __forceinline__ uint2 load_here8(const void* p, bool on = true) {
  uint2 v;
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %3, 0;\n mov.b32 %0, 0;\n mov.b32 %1, 0;\n @p ld.global.nc.v2.u32 {%0, %1}, [%2];\n}"
      : "=&r"(v.x), "=&r"(v.y)
      : "l"(p), "r"((int)on));
  return v;
}

// 16 bytes of global memory (or zeros) to shared memory, asynchronously; the copies since the
// last call as one group; the wait until at most N groups are on their way.
__device__ __forceinline__ void copy16(void* to, const void* from, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(to)), "l"(from), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// N stored values as pairs, and back (rounded to nearest even).
template <class E, int N> struct Pairs;
template <> struct Pairs<__nv_bfloat16, 8> {
  using T = uint4;
  __device__ static __forceinline__ F2 one(uint32_t u) { return pack(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)); }
  __device__ static __forceinline__ uint32_t word(F2 v) {
    float a, b;
    split(v, a, b);
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&x);
  }
  __device__ static __forceinline__ void get(F2 (&p)[4], const uint4& v) { p[0] = one(v.x); p[1] = one(v.y); p[2] = one(v.z); p[3] = one(v.w); }
  __device__ static __forceinline__ uint4 make(const F2 (&p)[4]) { return make_uint4(word(p[0]), word(p[1]), word(p[2]), word(p[3])); }
  __device__ static __forceinline__ uint4 load(const void* q, bool on = true) { return load_here(q, on); }
};
template <> struct Pairs<__nv_bfloat16, 4> {
  using T = uint2;
  using B = Pairs<__nv_bfloat16, 8>;
  __device__ static __forceinline__ void get(F2 (&p)[2], const uint2& v) { p[0] = B::one(v.x); p[1] = B::one(v.y); }
  __device__ static __forceinline__ uint2 make(const F2 (&p)[2]) { return make_uint2(B::word(p[0]), B::word(p[1])); }
  __device__ static __forceinline__ uint2 load(const void* q, bool on = true) { return load_here8(q, on); }
};
template <> struct Pairs<float, 4> {
  using T = uint4;
  __device__ static __forceinline__ void get(F2 (&p)[2], const uint4& v) {
    p[0] = pack(__uint_as_float(v.x), __uint_as_float(v.y));
    p[1] = pack(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  __device__ static __forceinline__ uint4 make(const F2 (&p)[2]) {
    float f[4];
    split(p[0], f[0], f[1]);
    split(p[1], f[2], f[3]);
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  __device__ static __forceinline__ uint4 load(const void* q, bool on = true) { return load_here(q, on); }
};

}  // namespace pairs
}  // namespace cfc
