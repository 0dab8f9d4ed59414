// Norms before and after a block, fused with its gate and residual scale, and
// their backward (formulas in include/kda.h).
//
// A row is read once, held in registers across its sums, and written once:
// a group of kThreads threads (half a warp to 512 threads, by the width) holds
// kChunks pieces of V elements per thread.  Sums run in fp32, per thread, then
// by shuffles, then over the warps in order.
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

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

// Sigmoid(g), and 1 - Sigmoid(g): the difference below a half, e r above it,
// where the power e is finite.
__device__ __forceinline__ float sigmoid_fast(float g, float &e) {
  e = fast_exp2(-kLog2e * g);
  return fast_rcp(1.f + e);
}
__device__ __forceinline__ float sigmoid_rest(float r, float e) { return r <= 0.5f ? 1.f - r : e * r; }

// V elements as they lie in memory.
template <typename T, int V> struct Piece;
template <> struct Piece<__nv_bfloat16, 8> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { v = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ float get(int i) const {
    const unsigned w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
};
template <> struct Piece<float, 8> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = *reinterpret_cast<const float4 *>(p);
    b = *reinterpret_cast<const float4 *>(p + 4);
  }
  __device__ __forceinline__ float get(int i) const {
    const float4 &q = i < 4 ? a : b;
    return (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w;
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
};
template <> struct Piece<__nv_bfloat16, 1> {
  __nv_bfloat16 v;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { v = *p; }
  __device__ __forceinline__ float get(int) const { return __bfloat162float(v); }
  __device__ __forceinline__ void zero() { v = __float2bfloat16_rn(0.f); }
};
template <> struct Piece<float, 1> {
  float v;
  __device__ __forceinline__ void load(const float *p) { v = *p; }
  __device__ __forceinline__ float get(int) const { return v; }
  __device__ __forceinline__ void zero() { v = 0.f; }
};

template <int V> __device__ __forceinline__ void put(float *p, const float (&f)[V]) {
  if constexpr (V == 8) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    *p = f[0];
  }
}
template <int V> __device__ __forceinline__ void put(__nv_bfloat16 *p, const float (&f)[V]) {
  if constexpr (V == 8) {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<uint4 *>(h);
  } else {
    *p = __float2bfloat16_rn(f[0]);
  }
}
// A weight row's piece; ones when it is absent.
template <int V> __device__ __forceinline__ void weight(const float *w, int j, float (&f)[V]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = 1.f;
  } else if constexpr (V == 8) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(w + j)), b = __ldg(reinterpret_cast<const float4 *>(w + j) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
    f[0] = __ldg(w + j);
  }
}

template <typename T_, typename R_, int V_, int kChunks_, int kThreads_>
struct Shape {
  using T = T_;                                              // y, gate, normed
  using R = R_;                                              // residual, out
  static constexpr int V = V_, kChunks = kChunks_, kThreads = kThreads_;
  static constexpr int kBlock = kThreads > 32 ? kThreads : 256, kGroups = kBlock / kThreads;
  static constexpr int kMaxWidth = V * kChunks * kThreads;
};

// Sums of kN values over the threads of a row, the same in each of them.
// `sh`: kN x 16 floats, not in use by an earlier sum of the same place.
template <int kThreads, int kN>
__device__ __forceinline__ void row_sum(float (&v)[kN], float (*sh)[16]) {
#pragma unroll
  for (int k = 0; k < kN; ++k)
#pragma unroll
    for (int off = (kThreads < 32 ? kThreads : 32) / 2; off > 0; off >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
  if constexpr (kThreads > 32) {
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int k = 0; k < kN; ++k) sh[k][threadIdx.x >> 5] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      v[k] = 0.f;
#pragma unroll
      for (int i = 0; i < kThreads / 32; ++i) v[k] += sh[k][i];
    }
  }
}

template <typename S>
__global__ void __launch_bounds__(S::kBlock) norm_fwd_kernel(NormArgs a) {
  using T = typename S::T;
  using R = typename S::R;
  constexpr int V = S::V, C = S::kChunks;
  __shared__ float sh[2][1][16];
  const long long row = (long long)blockIdx.x * S::kGroups + threadIdx.x / S::kThreads;
  const bool valid = row < a.rows;  // (a whole warp stays for the shuffles)
  const int t = threadIdx.x % S::kThreads;
  const size_t base = (size_t)(valid ? row : 0) * a.width;
  Piece<T, V> y[C], g[C];
  Piece<R, V> r[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int j = (c * S::kThreads + t) * V;
    const bool in = j < a.width;
    y[c].zero();
    if (in) y[c].load(static_cast<const T *>(a.y) + base + j);
    if (in && a.gate) g[c].load(static_cast<const T *>(a.gate) + base + j);
    if (in && a.res) r[c].load(static_cast<const R *>(a.res) + base + j);
  }
  const float inv = 1.f / (float)a.width;
  float r1 = 1.f;
  if (a.post) {
    float ss[1] = {0.f};
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < V; ++i) ss[0] = fmaf(y[c].get(i), y[c].get(i), ss[0]);
    row_sum<S::kThreads, 1>(ss, sh[0]);
    r1 = rsqrtf(ss[0] * inv + a.e1);
  }
  float o[C][V], so[1] = {0.f};
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int j = (c * S::kThreads + t) * V;
    const bool in = j < a.width;
    float w[V], s[V];
    if (in) {
      weight<V>(a.w1, j, w);
      weight<V>(a.sc, j, s);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float b = 0.f;
      if (in) {
        b = y[c].get(i) * r1 * w[i];
        float e;
        if (a.gate) b *= sigmoid_fast(g[c].get(i), e);
        b = a.res ? fmaf(b, s[i], r[c].get(i)) : b * s[i];
      }
      o[c][i] = b;
      so[0] = fmaf(b, b, so[0]);
    }
    if (in && valid && a.out) put<V>(static_cast<R *>(a.out) + base + j, o[c]);
  }
  if (!a.normed) return;
  row_sum<S::kThreads, 1>(so, sh[1]);
  const float r2 = rsqrtf(so[0] * inv + a.e2);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int j = (c * S::kThreads + t) * V;
    if (j < a.width && valid) {
      float w[V];
      weight<V>(a.w2, j, w);
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] *= o[c][i] * r2;
      put<V>(static_cast<T *>(a.normed) + base + j, w);
    }
  }
}

constexpr int kBwdBlocks = 304;  // at most; a block leaves one set of weight-gradient partials

// Backward.  With tr = scale o b the branch's part of out, everything that the
// row's gradients need of the row as a whole are sums that are known as soon as
// r1 is: sum out^2, and with q = d_normed w2
//     sum q out,  sum d_out tr,  sum q tr,  sum out tr
// since sum dy yh = sum D tr = sum (d_out + r2 q - back out) tr.  So a row takes
// two sums over its threads, not three.  Blocks walk over rows; a thread owns
// fixed channels, so its sums of the weight gradients stay in registers.
template <typename S>
__global__ void __launch_bounds__(S::kBlock) norm_bwd_kernel(NormArgs a, NormBwdIo io, float *part) {
  using T = typename S::T;
  using R = typename S::R;
  constexpr int V = S::V, C = S::kChunks;
  __shared__ float sh1[2][1][16], sh2[2][5][16];
  const int t = threadIdx.x % S::kThreads, group = threadIdx.x / S::kThreads;
  const float inv = 1.f / (float)a.width;
  float p1[C][V], ps[C][V], p2[C][V];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < V; ++i) p1[c][i] = ps[c][i] = p2[c][i] = 0.f;
  int par = 0;
  for (long long r0 = (long long)blockIdx.x * S::kGroups; r0 < a.rows; r0 += (long long)gridDim.x * S::kGroups, par ^= 1) {
    const bool valid = r0 + group < a.rows;
    const size_t base = (size_t)(valid ? r0 + group : 0) * a.width;
    Piece<T, V> y[C], g[C], dn[C];
    Piece<R, V> res[C], dout[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = (c * S::kThreads + t) * V;
      const bool in = j < a.width && valid;
      y[c].zero();
      g[c].zero();
      dn[c].zero();
      res[c].zero();
      dout[c].zero();
      if (in) {
        y[c].load(static_cast<const T *>(a.y) + base + j);
        if (a.gate) g[c].load(static_cast<const T *>(a.gate) + base + j);
        if (a.res) res[c].load(static_cast<const R *>(a.res) + base + j);
        if (io.dout) dout[c].load(static_cast<const R *>(io.dout) + base + j);
        if (io.dn) dn[c].load(static_cast<const T *>(io.dn) + base + j);
      }
    }
    float r1 = 1.f;
    if (a.post) {
      float ss[1] = {0.f};
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < V; ++i) ss[0] = fmaf(y[c].get(i), y[c].get(i), ss[0]);
      row_sum<S::kThreads, 1>(ss, sh1[par]);
      r1 = rsqrtf(ss[0] * inv + a.e1);
    }
    float sums[5] = {0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = (c * S::kThreads + t) * V;
      if (j >= a.width) continue;
      float w1[V], sc[V], w2[V];
      weight<V>(a.w1, j, w1);
      weight<V>(a.sc, j, sc);
      weight<V>(a.w2, j, w2);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float tr = y[c].get(i) * r1 * w1[i], e;
        if (a.gate) tr *= sigmoid_fast(g[c].get(i), e);
        tr *= sc[i];
        const float o = a.res ? tr + res[c].get(i) : tr;
        const float q = dn[c].get(i) * w2[i];
        sums[0] = fmaf(o, o, sums[0]);
        sums[1] = fmaf(q, o, sums[1]);
        sums[2] = fmaf(dout[c].get(i), tr, sums[2]);
        sums[3] = fmaf(q, tr, sums[3]);
        sums[4] = fmaf(o, tr, sums[4]);
      }
    }
    row_sum<S::kThreads, 5>(sums, sh2[par]);
    const float r2 = io.dn ? rsqrtf(sums[0] * inv + a.e2) : 0.f;
    const float back = r2 * r2 * r2 * sums[1] * inv;
    const float m = (sums[2] + r2 * sums[3] - back * sums[4]) * inv;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = (c * S::kThreads + t) * V;
      if (j >= a.width || !valid) continue;
      float w1[V], sc[V], w2[V], dres[V], dgate[V], dy[V];
      weight<V>(a.w1, j, w1);
      weight<V>(a.sc, j, sc);
      weight<V>(a.w2, j, w2);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float yh = y[c].get(i) * r1;
        float sg = 1.f, rest = 0.f;
        if (a.gate) {
          float e;
          sg = sigmoid_fast(g[c].get(i), e);
          rest = sigmoid_rest(sg, e);
        }
        const float b = yh * w1[i] * sg;
        const float o = a.res ? fmaf(b, sc[i], res[c].get(i)) : b * sc[i];
        const float n = dn[c].get(i);
        const float D = fmaf(r2 * w2[i], n, fmaf(-back, o, dout[c].get(i)));
        p2[c][i] = fmaf(n * r2, o, p2[c][i]);
        ps[c][i] = fmaf(D, b, ps[c][i]);
        const float db = D * sc[i], du = db * sg;
        p1[c][i] = fmaf(du, yh, p1[c][i]);
        dres[i] = D;
        dgate[i] = db * b * rest;
        dy[i] = a.post ? r1 * fmaf(du, w1[i], -yh * m) : du;
      }
      put<V>(static_cast<T *>(io.dy) + base + j, dy);
      if (io.dgate) put<V>(static_cast<T *>(io.dgate) + base + j, dgate);
      if (io.dres) put<V>(static_cast<R *>(io.dres) + base + j, dres);
    }
  }
  if (!part) return;
  // the groups of a block in order, then one row of partials
  extern __shared__ float sums[];  // [kGroups][kMaxWidth]
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    float *to = part + ((size_t)k * gridDim.x + blockIdx.x) * a.width;
    if constexpr (S::kGroups > 1) {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < V; ++i)
          sums[group * S::kMaxWidth + (c * S::kThreads + t) * V + i] = k == 0 ? p1[c][i] : k == 1 ? ps[c][i] : p2[c][i];
      __syncthreads();
      for (int j = threadIdx.x; j < a.width; j += S::kBlock) {
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < S::kGroups; ++q) s += sums[q * S::kMaxWidth + j];
        to[j] = s;
      }
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int j = (c * S::kThreads + t) * V;
        if (j < a.width)
#pragma unroll
          for (int i = 0; i < V; ++i) to[j + i] = k == 0 ? p1[c][i] : k == 1 ? ps[c][i] : p2[c][i];
      }
    }
  }
}

// Weight gradients: the blocks' partials summed, 32 columns and 16 strides of
// blocks to a CTA.
__global__ void __launch_bounds__(512) norm_weights_kernel(const float *part, int blocks, int width, NormBwdIo io) {
  const int lane = threadIdx.x & 31, stride = threadIdx.x >> 5, j = blockIdx.x * 32 + lane, k = blockIdx.y;
  float *out = k == 0 ? io.dw1 : k == 1 ? io.dsc : io.dw2;
  if (!out) return;
  __shared__ float sh[16][32];
  float s = 0.f;
  if (j < width)
    for (int b = stride; b < blocks; b += 16) s += part[((size_t)k * blocks + b) * width + j];
  sh[stride][lane] = s;
  __syncthreads();
  if (stride == 0 && j < width) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += sh[i][lane];
    out[j] = s;
  }
}

template <typename S> cudaError_t fwd(const NormArgs &a, cudaStream_t s) {
  norm_fwd_kernel<S><<<(unsigned)((a.rows + S::kGroups - 1) / S::kGroups), S::kBlock, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename S> cudaError_t bwd(const NormArgs &a, const NormBwdIo &io, float *ws, cudaStream_t s) {
  const bool weights = io.dw1 || io.dsc || io.dw2;
  const long long groups = (a.rows + S::kGroups - 1) / S::kGroups;
  const int blocks = (int)(groups < 1 ? 1 : groups < kBwdBlocks ? groups : kBwdBlocks);
  const size_t smem = S::kGroups > 1 ? sizeof(float) * S::kGroups * S::kMaxWidth : 0;
  norm_bwd_kernel<S><<<blocks, S::kBlock, smem, s>>>(a, io, weights ? ws : nullptr);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !weights) return e;
  norm_weights_kernel<<<dim3((a.width + 31) / 32, 3), 512, 0, s>>>(ws, blocks, a.width, io);
  return cudaGetLastError();
}

// Calls f with the row shape for this width: pieces of 8 elements when every
// row of every tensor starts on 16 bytes, else single elements.
template <typename T, typename R, typename F>
cudaError_t with_shape(int width, bool vectors, F f) {
  if (vectors) {
    if (width <= 128) return f(Shape<T, R, 8, 1, 16>());
    if (width <= 256) return f(Shape<T, R, 8, 1, 32>());
    if (width <= 512) return f(Shape<T, R, 8, 2, 32>());
    if (width <= 1024) return f(Shape<T, R, 8, 1, 128>());
    if (width <= 2048) return f(Shape<T, R, 8, 1, 256>());
    if (width <= 4096) return f(Shape<T, R, 8, 2, 256>());
    return f(Shape<T, R, 8, 2, 512>());
  }
  if (width <= 128) return f(Shape<T, R, 1, 4, 32>());
  if (width <= 1024) return f(Shape<T, R, 1, 4, 256>());
  return f(Shape<T, R, 1, 16, 512>());
}

template <typename F> cudaError_t with_types(const NormArgs &a, bool vectors, F f) {
  using B = __nv_bfloat16;
  if (a.t == KDA_BF16)
    return a.rt == KDA_BF16 ? with_shape<B, B>(a.width, vectors, f) : with_shape<B, float>(a.width, vectors, f);
  return a.rt == KDA_BF16 ? with_shape<float, B>(a.width, vectors, f) : with_shape<float, float>(a.width, vectors, f);
}

template <int kN> bool on_16_bytes(const NormArgs &a, const void *const (&p)[kN]) {
  uintptr_t bits = 0;
  for (const void *q : p) bits |= reinterpret_cast<uintptr_t>(q);
  return (bits & 15) == 0 && a.width % 8 == 0;
}

}  // namespace

size_t norm_bwd_workspace_bytes(int width) { return (size_t)3 * kBwdBlocks * width * sizeof(float); }

cudaError_t launch_norm_fwd(const NormArgs &a, cudaStream_t s) {
  if (a.rows == 0) return cudaSuccess;
  const void *const p[] = {a.y, a.res, a.gate, a.w1, a.sc, a.w2, a.out, a.normed};
  return with_types(a, on_16_bytes(a, p), [&](auto shape) { return fwd<decltype(shape)>(a, s); });
}

cudaError_t launch_norm_bwd(const NormArgs &a, const NormBwdIo &io, void *ws, cudaStream_t s) {
  const void *const p[] = {a.y, a.res, a.gate, a.w1, a.sc, a.w2, io.dout, io.dn, io.dy, io.dres, io.dgate};
  return with_types(a, on_16_bytes(a, p),
                    [&](auto shape) { return bwd<decltype(shape)>(a, io, static_cast<float *>(ws), s); });
}

}  // namespace kda
