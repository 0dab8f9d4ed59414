// Device pieces that the kernels of the gated linear recurrence share
// (kda_scan.cu, kda_scan_bwd.cu).
//
// Numerics.  With alpha near 1 (a memory of thousands of tokens) rounding
// alpha to fp32 costs up to 3e-8 / (1 - alpha) of the state, the same way at
// every token of a constant decay.  So for g > -1/8 a step uses
// h' = h + (e h + u) with e = expm1(g), whose rounding error is relative to
// 1 - alpha, and below that alpha itself, so that a strong decay (alpha = 0 at
// the least) leaves nothing of h behind.  Everything is fp32.
//
// A decay is one float c: the sign bit set means c = e (e <= 0; -0 for g = 0),
// clear means c = alpha.
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

// expm1 on (-1/8, 0] by its series through g^5: the next term is 4.3e-8 of the
// first, below half a step.
__device__ __forceinline__ float decay_code(float g) {
  g = at_most_zero(g);
  float p = fmaf(g, 1.f / 120.f, 1.f / 24.f);
  p = fmaf(g, p, 1.f / 6.f);
  p = fmaf(g, p, 0.5f);
  p = fmaf(g * g, p, g);
  return g > kNearOne ? -fabsf(p) : fast_exp2(g * kLog2e);
}

__device__ __forceinline__ float decay_alpha(float c) { return is_near(c) ? 1.f + c : c; }
__device__ __forceinline__ float decay_one_minus(float c) { return is_near(c) ? -c : 1.f - c; }

// alpha h + u
__device__ __forceinline__ float decay_apply(float c, float h, float u) {
  float r = fmaf(c, h, u);
  if (is_near(c)) r += h;
  return r;
}

// One token: alpha h + w x; with w = 1 - alpha it is h + e (h - x) = x + alpha (h - x).
template <bool kComp>
__device__ __forceinline__ float scan_token(float c, float h, float x) {
  if (!kComp) return decay_apply(c, h, x);
  return fmaf(c, h - x, is_near(c) ? h : x);
}

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
template <int V> struct Pack<float, V> {
  float v[V];
  __device__ __forceinline__ void load(const float *p) {
    if (V == 2) {
      const float2 t = __ldcs(reinterpret_cast<const float2 *>(p));
      v[0] = t.x;
      v[V - 1] = t.y;
    } else {
      v[0] = __ldcs(p);
    }
  }
  __device__ __forceinline__ float get(int i) const { return v[i]; }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.f;
  }
};
template <> struct Pack<__nv_bfloat16, 2> {
  unsigned v;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { v = __ldcs(reinterpret_cast<const unsigned *>(p)); }
  __device__ __forceinline__ float get(int i) const { return __uint_as_float(i ? v & 0xffff0000u : v << 16); }
  __device__ __forceinline__ void zero() { v = 0u; }
};
template <> struct Pack<__nv_bfloat16, 1> {
  unsigned short v;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { v = __ldcs(reinterpret_cast<const unsigned short *>(p)); }
  __device__ __forceinline__ float get(int) const { return __uint_as_float((unsigned)v << 16); }
  __device__ __forceinline__ void zero() { v = 0; }
};

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
// Stores two floats at the same shared-memory place of CTA `rank`.
__device__ __forceinline__ void store_remote(void *local, unsigned rank, float x, float y) {
  unsigned addr = (unsigned)__cvta_generic_to_shared(local), remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(remote), "f"(x), "f"(y) : "memory");
}

constexpr int kScanWarps = 8;                               // warps of a CTA
constexpr int kScanThreads = 32 * kScanWarps;
constexpr int kScanSpan = kScanWarps * kScanTile;           // tokens of a CTA in one round
constexpr int kScanMaxCluster = 8;

// Joins the spans of one round.  Every warp gives the decay code c and log-sum
// G of its tile and what the tile adds (B) per channel, in the order the
// recurrence runs (warp 0 of CTA 0 first); each thread gets back the state that
// enters its warp's tile, and `carry` becomes the state that leaves the round.
template <int V>
struct ScanJoin {
  float2 tile[2][kScanWarps][32 * V];          // (c, B)
  float G[2][kScanWarps][32 * V];
  float2 cta[2][kScanMaxCluster][32 * V];      // (c, B) of whole CTAs

  __device__ __forceinline__ void join(int par, int warp, int lane, unsigned rank, unsigned ranks,
                                       const float (&g)[V], const float (&b)[V], float (&carry)[V],
                                       float (&entry)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      tile[par][warp][lane * V + i] = make_float2(decay_code(g[i]), b[i]);
      if (ranks > 1) G[par][warp][lane * V + i] = g[i];
    }
    __syncthreads();
    if (ranks > 1) {
      if (warp == 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float sum = 0.f, add = 0.f;
#pragma unroll
          for (int w = 0; w < kScanWarps; ++w) {
            const float2 t = tile[par][w][lane * V + i];
            sum += G[par][w][lane * V + i];
            add = decay_apply(t.x, add, t.y);
          }
          const float c = decay_code(sum);
          for (unsigned r = 0; r < ranks; ++r) store_remote(&cta[par][rank][lane * V + i], r, c, add);
        }
      }
      cluster_sync_all();
#pragma unroll
      for (int i = 0; i < V; ++i) {
        entry[i] = carry[i];
        for (unsigned r = 0; r < ranks; ++r) {
          if (r == rank) entry[i] = carry[i];
          const float2 t = cta[par][r][lane * V + i];
          carry[i] = decay_apply(t.x, carry[i], t.y);
        }
        for (int w = 0; w < warp; ++w) {
          const float2 t = tile[par][w][lane * V + i];
          entry[i] = decay_apply(t.x, entry[i], t.y);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int w = 0; w < kScanWarps; ++w) {
          if (w == warp) entry[i] = carry[i];
          const float2 t = tile[par][w][lane * V + i];
          carry[i] = decay_apply(t.x, carry[i], t.y);
        }
      }
    }
  }
};

// Whether every given pointer allows 2-element accesses on rows of D elements.
inline bool scan_pairs(int D, std::initializer_list<const void *> ptrs) {
  uintptr_t bits = (D & 1) ? 8 : 0;
  for (const void *p : ptrs) bits |= reinterpret_cast<uintptr_t>(p);
  return (bits & 15) == 0;
}

// CTAs of a cluster: see the rule in kda_scan.cu.
int scan_cluster(const ScanArgs &a, int channels);

}  // namespace kda
