// Norms before and after a block, fused with its gate and residual scale, and
// their backward (formulas in include/kda.h).
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kBwdBlocks = 304;  // row groups of the backward; one set of weight-gradient partials each

// Sum over the block, the same in every thread and in a fixed order.
__device__ __forceinline__ float block_sum(float v, float *sh) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) s += sh[i];
  return s;
}

// Sigmoid(g) and 1 - Sigmoid(g).  The exponential's argument is capped (a NaN
// passes), past which Sigmoid is below 1e-34, so that e / (1 + e) stays finite.
__device__ __forceinline__ float gate_sigmoid(float g, float &rest) {
  const float e = expf(-g > 80.f ? 80.f : -g);
  const float s = 1.f / (1.f + e);
  rest = e * s;
  return s;
}

__device__ __forceinline__ float pick(const float *p, int j) { return p ? p[j] : 1.f; }

// One block per row; the row's `out` values wait in shared memory for the
// second norm.
__global__ void __launch_bounds__(kThreads) norm_fwd_kernel(NormArgs a) {
  extern __shared__ float row[];
  __shared__ float sh[kThreads / 32];
  const size_t base = (size_t)blockIdx.x * a.width;
  float ss = 0.f;
  for (int j = threadIdx.x; j < a.width; j += kThreads) {
    const float y = ld_elem(a.y, base + j, a.t);
    row[j] = y;
    ss += y * y;
  }
  const float r1 = a.post ? rsqrtf(block_sum(ss, sh) / (float)a.width + a.e1) : 1.f;
  float so = 0.f;
  for (int j = threadIdx.x; j < a.width; j += kThreads) {
    float b = row[j] * r1 * pick(a.w1, j);
    if (a.gate) b *= sigmoid_f(ld_elem(a.gate, base + j, a.t));
    float o = b * pick(a.sc, j);
    if (a.res) o += ld_elem(a.res, base + j, a.rt);
    row[j] = o;
    so += o * o;
    if (a.out) st_elem(a.out, base + j, o, a.rt);
  }
  if (!a.normed) return;
  const float r2 = rsqrtf(block_sum(so, sh) / (float)a.width + a.e2);
  for (int j = threadIdx.x; j < a.width; j += kThreads) st_elem(a.normed, base + j, row[j] * r2 * pick(a.w2, j), a.t);
}

// One block per group of rows; a thread owns fixed channels, so its sums of
// the weight gradients need no exchange.  part: [3][gridDim.x][width].
__global__ void __launch_bounds__(kThreads) norm_bwd_kernel(NormArgs a, NormBwdIo io, float *part) {
  extern __shared__ float smem[];
  __shared__ float sh[kThreads / 32];
  float *row = smem, *p1 = smem + a.width, *ps = p1 + a.width, *p2 = ps + a.width;
  for (int j = threadIdx.x; j < a.width; j += kThreads) p1[j] = ps[j] = p2[j] = 0.f;
  const float inv = 1.f / (float)a.width;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const size_t base = (size_t)r * a.width;
    float ss = 0.f;
    if (a.post)
      for (int j = threadIdx.x; j < a.width; j += kThreads) {
        const float y = ld_elem(a.y, base + j, a.t);
        ss += y * y;
      }
    const float r1 = a.post ? rsqrtf(block_sum(ss, sh) * inv + a.e1) : 1.f;
    float so = 0.f, dot = 0.f;
    if (io.dn) {
      for (int j = threadIdx.x; j < a.width; j += kThreads) {
        float b = ld_elem(a.y, base + j, a.t) * r1 * pick(a.w1, j);
        if (a.gate) b *= sigmoid_f(ld_elem(a.gate, base + j, a.t));
        float o = b * pick(a.sc, j);
        if (a.res) o += ld_elem(a.res, base + j, a.rt);
        so += o * o;
        dot += o * ld_elem(io.dn, base + j, a.t) * pick(a.w2, j);
      }
      so = block_sum(so, sh);
      dot = block_sum(dot, sh);
    }
    const float r2 = io.dn ? rsqrtf(so * inv + a.e2) : 0.f;
    const float back = r2 * r2 * r2 * dot * inv;
    float dd = 0.f;
    for (int j = threadIdx.x; j < a.width; j += kThreads) {
      const float yh = ld_elem(a.y, base + j, a.t) * r1, u = yh * pick(a.w1, j);
      float rest = 0.f;
      const float sg = a.gate ? gate_sigmoid(ld_elem(a.gate, base + j, a.t), rest) : 1.f;
      const float b = u * sg;
      float o = b * pick(a.sc, j);
      if (a.res) o += ld_elem(a.res, base + j, a.rt);
      float D = io.dout ? ld_elem(io.dout, base + j, a.rt) : 0.f;
      if (io.dn) {
        const float dn = ld_elem(io.dn, base + j, a.t);
        D += r2 * dn * pick(a.w2, j) - back * o;
        p2[j] += dn * o * r2;
      }
      if (io.dres) st_elem(io.dres, base + j, D, a.rt);
      ps[j] += D * b;
      const float db = D * pick(a.sc, j);
      if (io.dgate) st_elem(io.dgate, base + j, db * b * rest, a.t);
      const float du = db * sg;
      p1[j] += du * yh;
      const float dy = du * pick(a.w1, j);
      row[j] = dy;
      dd += dy * yh;
    }
    const float m = a.post ? block_sum(dd, sh) * inv : 0.f;
    for (int j = threadIdx.x; j < a.width; j += kThreads) {
      const float yh = ld_elem(a.y, base + j, a.t) * r1;
      st_elem(io.dy, base + j, a.post ? r1 * (row[j] - yh * m) : row[j], a.t);
    }
  }
  for (int j = threadIdx.x; j < a.width; j += kThreads) {
    part[((size_t)0 * gridDim.x + blockIdx.x) * a.width + j] = p1[j];
    part[((size_t)1 * gridDim.x + blockIdx.x) * a.width + j] = ps[j];
    part[((size_t)2 * gridDim.x + blockIdx.x) * a.width + j] = p2[j];
  }
}

__global__ void __launch_bounds__(kThreads) norm_weights_kernel(const float *part, int blocks, int width, NormBwdIo io) {
  const int j = blockIdx.x * kThreads + threadIdx.x, k = blockIdx.y;
  float *out = k == 0 ? io.dw1 : k == 1 ? io.dsc : io.dw2;
  if (!out || j >= width) return;
  float s = 0.f;
  for (int b = 0; b < blocks; ++b) s += part[((size_t)k * blocks + b) * width + j];
  out[j] = s;
}

}  // namespace

size_t norm_bwd_workspace_bytes(int width) { return (size_t)3 * kBwdBlocks * width * sizeof(float); }

cudaError_t launch_norm_fwd(const NormArgs &a, cudaStream_t s) {
  if (a.rows == 0) return cudaSuccess;
  const size_t smem = sizeof(float) * a.width;
  cudaError_t e = cudaFuncSetAttribute(norm_fwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  norm_fwd_kernel<<<(unsigned)a.rows, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_norm_bwd(const NormArgs &a, const NormBwdIo &io, void *ws, cudaStream_t s) {
  const int blocks = kBwdBlocks;
  const size_t smem = sizeof(float) * 4 * (size_t)a.width;
  if (smem > 220 * 1024) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(norm_bwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  float *part = static_cast<float *>(ws);
  norm_bwd_kernel<<<blocks, kThreads, smem, s>>>(a, io, part);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  norm_weights_kernel<<<dim3((a.width + kThreads - 1) / kThreads, 3), kThreads, 0, s>>>(part, blocks, a.width, io);
  return cudaGetLastError();
}

}  // namespace kda
