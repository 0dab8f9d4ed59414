// Small fp32 arithmetic shared by the elementwise kernels: approximate powers
// and reciprocals, and pairs of values in one register pair.
#pragma once

#include <cuda_runtime.h>

namespace kda {

constexpr float kLog2e = 1.4426950408889634f;

// 2^x and 1 / x to 2 ulp, subnormal results flushed to 0: one instruction each, where
// exp and division take several, in kernels that fill up to two thirds of the issue
// slots.  Their 4 half steps of fp32 are within what the operators state.
__device__ __forceinline__ float fast_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// V fp32 values of one lane.  Two are one register pair, and one instruction
// of the packed fp32 kind works on both: elementwise kernels are bound by
// instruction issue before they are by anything else but HBM.
template <int V> struct Vec;
template <> struct Vec<1> {
  float v;
  __device__ __forceinline__ float get(int) const { return v; }
};
template <> struct Vec<2> {
  unsigned long long v;
  __device__ __forceinline__ float get(int i) const { return __uint_as_float((unsigned)(i ? v >> 32 : v)); }
};
__device__ __forceinline__ Vec<2> pair(float x, float y) {
  Vec<2> r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
template <int V> __device__ __forceinline__ Vec<V> all(float x);
template <> __device__ __forceinline__ Vec<1> all<1>(float x) { return Vec<1>{x}; }
template <> __device__ __forceinline__ Vec<2> all<2>(float x) { return pair(x, x); }
__device__ __forceinline__ Vec<1> fma(Vec<1> a, Vec<1> b, Vec<1> c) { return Vec<1>{fmaf(a.v, b.v, c.v)}; }
__device__ __forceinline__ Vec<1> mul(Vec<1> a, Vec<1> b) { return Vec<1>{a.v * b.v}; }
__device__ __forceinline__ Vec<1> add(Vec<1> a, Vec<1> b) { return Vec<1>{a.v + b.v}; }
__device__ __forceinline__ Vec<2> fma(Vec<2> a, Vec<2> b, Vec<2> c) {
  Vec<2> r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ Vec<2> mul(Vec<2> a, Vec<2> b) {
  Vec<2> r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Vec<2> add(Vec<2> a, Vec<2> b) {
  Vec<2> r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
// f of every value's index
template <int V, typename F> __device__ __forceinline__ Vec<V> lanes(F f) {
  if constexpr (V == 2) return pair(f(0), f(1));
  else return Vec<1>{f(0)};
}

}  // namespace kda
