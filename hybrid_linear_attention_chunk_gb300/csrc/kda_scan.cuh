// Device pieces that the kernels of the gated linear recurrence share
// (kda_scan.cu, kda_scan_bwd.cu).
//
// Numerics.  With alpha near 1 (a memory of thousands of tokens) rounding
// alpha to fp32 costs up to 3e-8 / (1 - alpha) of the state, the same way at
// every token of a constant decay.  So the decay of a whole 16-token tile, by
// which a state is carried on, comes from the sum of its logs: h' = h + (e h + B)
// with e = expm1(sum g) when sum g > -1/8, whose rounding error is relative to
// 1 - alpha, and alpha itself below that, so that a strong decay (alpha = 0 at
// the least) leaves nothing of h behind.  Inside a tile the products of up to 16
// rounded alphas are off by at most 16 roundings, of the tile's own sums alone.
// w = 1 - alpha comes from expm1(g) too.  Everything is fp32.
//
// The decay of a tile or span is one float c: the sign bit set means c = e
// (e <= 0; -0 for a sum of 0), clear means c = alpha.
#pragma once

#include "kda_internal.cuh"

namespace kda {

constexpr float kNearOne = -0.125f;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ bool is_near(float c) { return __float_as_int(c) < 0; }

// min(g, 0) that passes a NaN on (log_alpha above 0 counts as 0).
__device__ __forceinline__ float at_most_zero(float g) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(g), "f"(0.f));
  return r;
}

// 2^x and 1 / x to 2 ulp, subnormal results flushed to 0.
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

// expm1(g) on (-1/8, 0] as g + g^2 q(g), q the quadratic with the least maximum
// relative error there (a reweighted least-squares fit to the series): 1.8e-8
// of the value, a third of half a step.
__device__ __forceinline__ float expm1_near(float g) {
  float q = fmaf(g, 0.03972300514578819f, 0.16652730107307434f);
  q = fmaf(g, q, 0.4999971389770508f);
  return fmaf(g * g, q, g);
}

__device__ __forceinline__ float decay_code(float g) {
  return g > kNearOne ? -fabsf(expm1_near(g)) : fast_exp2(g * kLog2e);
}

// alpha h + u
__device__ __forceinline__ float decay_apply(float c, float h, float u) {
  float r = fmaf(c, h, u);
  if (is_near(c)) r += h;
  return r;
}

// alpha and w of one token from its g <= 0.
__device__ __forceinline__ float alpha_of(float g) { return fast_exp2(g * kLog2e); }
__device__ __forceinline__ float one_minus(float g, float alpha) {
  return g > kNearOne ? -expm1_near(g) : 1.f - alpha;
}

// -exp(A) log2(e), never 0: the product with z = -inf, a masked token, stays inf.
__device__ __forceinline__ float gate_scale(float A_log) { return fminf(-kLog2e * expf(A_log), -1e-37f); }

// g = g_min Sigmoid(s z) from z and ns = -s log2(e); 2^x = inf gives g = -0.
__device__ __forceinline__ float gate_code(float z, float ns, float g_min) {
  return g_min * fast_rcp(1.f + fast_exp2(ns * z));
}

__device__ __forceinline__ void scan_range(const ScanArgs &a, int n, int &bos, int &eos) {
  if (a.cu) {  // clamped: cu_seqlens that break their precondition reach no other memory
    bos = min(max(a.cu[n], 0), a.T_total);
    eos = min(max(a.cu[n + 1], bos), a.T_total);
  } else {
    bos = n * a.T_seq;
    eos = bos + a.T_seq;
  }
}

// V consecutive elements as they lie in memory, and their fp32 values.
template <typename T, int V> struct Pack;
template <> struct Pack<float, 2> {
  float2 v;
  __device__ __forceinline__ void load(const void *p) { v = __ldcs(static_cast<const float2 *>(p)); }
  __device__ __forceinline__ float get(int i) const { return i ? v.y : v.x; }
  __device__ __forceinline__ void fill(float f) { v = make_float2(f, f); }
};
template <> struct Pack<float, 1> {
  float v;
  __device__ __forceinline__ void load(const void *p) { v = __ldcs(static_cast<const float *>(p)); }
  __device__ __forceinline__ float get(int) const { return v; }
  __device__ __forceinline__ void fill(float f) { v = f; }
};
template <> struct Pack<__nv_bfloat16, 2> {
  unsigned v;
  __device__ __forceinline__ void load(const void *p) { v = __ldcs(static_cast<const unsigned *>(p)); }
  __device__ __forceinline__ float get(int i) const { return __uint_as_float(i ? v & 0xffff0000u : v << 16); }
  __device__ __forceinline__ void fill(float f) { v = __float_as_uint(f) | __float_as_uint(f) >> 16; }  // f exact in bf16
};
template <> struct Pack<__nv_bfloat16, 1> {
  unsigned short v;
  __device__ __forceinline__ void load(const void *p) { v = __ldcs(static_cast<const unsigned short *>(p)); }
  __device__ __forceinline__ float get(int) const { return __uint_as_float((unsigned)v << 16); }
  __device__ __forceinline__ void fill(float f) { v = (unsigned short)(__float_as_uint(f) >> 16); }
};

// A warp's tile of one array: tokens t .. t + 15, `col` the lane's byte offset
// in a row.  The row pointers are the same in a whole warp.  Tokens past `len`
// get `pad`.
template <typename T, int V>
__device__ __forceinline__ void load_tile(Pack<T, V> (&v)[kScanTile], const void *base, int D, int t, unsigned col,
                                          int len, bool full, float pad) {
  const size_t row = (size_t)D * sizeof(T);
  const char *p = static_cast<const char *>(base) + (size_t)t * row;
  if (full) {
#pragma unroll
    for (int j = 0; j < kScanTile; ++j, p += row) v[j].load(p + col);
  } else {
#pragma unroll
    for (int j = 0; j < kScanTile; ++j, p += row) {
      v[j].fill(pad);
      if (j < len) v[j].load(p + col);
    }
  }
}

template <int V> __device__ __forceinline__ void store(float *p, const float *v) {
  if (V == 2) *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[V - 1]);
  else *p = v[0];
}
template <int V> __device__ __forceinline__ void store(__nv_bfloat16 *p, const float *v) {
  if (V == 2) *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v[0], v[V - 1]);
  else *p = __float2bfloat16_rn(v[0]);
}
template <int V> __device__ __forceinline__ void load_f32(const float *p, float *v) {
  if (V == 2) {
    const float2 t = *reinterpret_cast<const float2 *>(p);
    v[0] = t.x;
    v[V - 1] = t.y;
  } else {
    v[0] = *p;
  }
}

// ------------------------------------------------------------------ clusters
// A chain block (one sequence, 32 V channels) runs on one cluster; its CTAs take
// consecutive spans of tokens of a round.  The hardware schedules a cluster's
// CTAs together, so its barrier needs no spinning on memory.
__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ unsigned cluster_size() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Stores at the same shared-memory place of CTA `rank`.
template <typename T>
__device__ __forceinline__ void store_remote(T *local, int rank, const T &v) {
  const unsigned addr = (unsigned)__cvta_generic_to_shared(local);
  unsigned remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  const float *f = reinterpret_cast<const float *>(&v);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 8); ++i)
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(remote + 8 * i), "f"(f[2 * i]), "f"(f[2 * i + 1])
                 : "memory");
}

constexpr int kScanWarps = 8;                               // warps of a CTA
constexpr int kScanThreads = 32 * kScanWarps;
constexpr int kScanSpan = kScanWarps * kScanTile;           // tokens of a CTA in one round
constexpr int kScanMaxCluster = 8;

// What a span of tokens does to the state, per channel of a lane: the decay
// code of its log-sum, and what it adds.
template <int V> struct __align__(8 * V) Span {
  float c[V], add[V];
  __device__ __forceinline__ void run(float (&h)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) h[i] = decay_apply(c[i], h[i], add[i]);
  }
};

// Joins the tiles of one round, in the order the recurrence runs (warp 0 of
// CTA 0 first).  Tile by tile each warp runs the state that entered the round
// through the spans before its own.
//   One CTA: the last warp leaves the state that enters the next round in
//   `carry`, which the others read after the next round's barrier.
//   A cluster: warp 0 joins its CTA's eight tiles into one span and stores it
//   in every CTA; each thread keeps the round's state in registers.
// Two buffers: a round's spans are read until the next round's barrier.
template <int V>
struct ScanJoin {
  Span<V> tile[2][kScanWarps][32];
  Span<V> cta[2][kScanMaxCluster][32];
  float logs[2][kScanWarps][32 * V];
  float carry[2][32 * V];
};

template <int V>
__device__ __forceinline__ void join_one(ScanJoin<V> &sh, int par, int warp, int lane, const Span<V> &mine,
                                         float (&entry)[V]) {
  sh.tile[par][warp][lane] = mine;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < V; ++i) entry[i] = sh.carry[par][lane * V + i];
  for (int w = 0; w < warp; ++w) sh.tile[par][w][lane].run(entry);
}

template <int V>
__device__ __forceinline__ void join_cluster(ScanJoin<V> &sh, int par, int warp, int lane, int rank, int ranks,
                                             const Span<V> &mine, const float (&logs)[V], float (&state)[V],
                                             float (&entry)[V]) {
  sh.tile[par][warp][lane] = mine;
#pragma unroll
  for (int i = 0; i < V; ++i) sh.logs[par][warp][lane * V + i] = logs[i];
  __syncthreads();
  if (warp == 0) {
    float sum[V] = {}, add[V] = {};
#pragma unroll
    for (int w = 0; w < kScanWarps; ++w) {
      sh.tile[par][w][lane].run(add);
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] += sh.logs[par][w][lane * V + i];
    }
    Span<V> all;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      all.c[i] = decay_code(sum[i]);
      all.add[i] = add[i];
    }
    for (int r = 0; r < ranks; ++r) store_remote(&sh.cta[par][rank][lane], r, all);
  }
  cluster_sync_all();
  for (int r = 0; r < rank; ++r) sh.cta[par][r][lane].run(state);
#pragma unroll
  for (int i = 0; i < V; ++i) entry[i] = state[i];
  for (int r = rank; r < ranks; ++r) sh.cta[par][r][lane].run(state);
  for (int w = 0; w < warp; ++w) sh.tile[par][w][lane].run(entry);
}

// Whether every given pointer allows 2-element accesses on rows of D elements.
inline bool scan_pairs(int D, std::initializer_list<const void *> ptrs) {
  uintptr_t bits = (D & 1) ? 8 : 0;
  for (const void *p : ptrs) bits |= reinterpret_cast<uintptr_t>(p);
  return (bits & 15) == 0;
}

// CTAs of a cluster: see the rule in kda_scan.cu.
int scan_cluster(const ScanArgs &a, int channels);

}  // namespace kda
