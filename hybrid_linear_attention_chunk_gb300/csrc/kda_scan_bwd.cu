// Backward of the gated linear recurrence (formulas in include/kda.h).
#include <initializer_list>

#include "kda_scan.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float alpha_of(float g) { return fast_exp2(g * kLog2e); }
__device__ __forceinline__ float one_minus(float g, float alpha) { return g > kNearOne ? -expm1_near(g) : 1.f - alpha; }

__device__ __forceinline__ float gate_slope(float z, float s, float g_min, float *slope) {
  const float v = -s * z;
  const float e = expf(v > 80.f ? 80.f : v);
  const float r = 1.f / (1.f + e);
  const float g = g_min * r;
  *slope = g * (e * r) * s;
  return g;
}

// One thread per chain: tiles from the last to the first, each rerun forward
// from its stored state.
__global__ void __launch_bounds__(kThreads) scan_bwd_kernel(ScanArgs a, ScanBwdIo io, float *dA_part) {
  const int cblocks = (a.D + kThreads - 1) / kThreads;
  const int c = (int)(blockIdx.x % cblocks) * kThreads + threadIdx.x, n = blockIdx.x / cblocks;
  if (c >= a.D) return;
  int bos, eos;
  scan_range(a, n, bos, eos);
  const size_t chain = (size_t)n * a.D + c;
  const float scale = a.A_log ? expf(a.A_log[c / a.d]) : 0.f;
  float carry = io.dST ? io.dST[chain] : 0.f;  // gradient of the state that leaves token t
  float dA = 0.f;
  const int tiles = (eos - bos + kScanTile - 1) / kScanTile;
  for (int j = tiles - 1; j >= 0; --j) {
    const int t0 = bos + j * kScanTile, len = min(kScanTile, eos - t0);
    float prev[kScanTile];
    float h = a.states[((size_t)(bos / kScanTile) + n + j) * a.D + c];
    for (int i = 0; i < len; ++i) {
      prev[i] = h;
      const size_t at = (size_t)(t0 + i) * a.D + c;
      float g = ld_elem(a.g, at, a.gdt());
      float sl;
      if (a.A_log) g = gate_slope(g, scale, a.g_min, &sl);
      const float al = alpha_of(g);
      const float x = ld_elem(a.x, at, a.t);
      h = decay_apply(decay_code(g), h, a.complement ? one_minus(g, al) * x : x);
    }
    float dA_tile = 0.f;
    for (int i = len - 1; i >= 0; --i) {
      const size_t at = (size_t)(t0 + i) * a.D + c;
      const float z = ld_elem(a.g, at, a.gdt());
      float slope = 1.f;
      const float g = a.A_log ? gate_slope(z, scale, a.g_min, &slope) : z;
      const float al = alpha_of(g);
      const float x = ld_elem(a.x, at, a.t);
      const float D = ld_elem(io.dO, at, a.t) + carry;
      st_elem(io.dx, at, a.complement ? one_minus(g, al) * D : D, a.t);
      const float dg = al * D * (a.complement ? prev[i] - x : prev[i]) * slope;
      st_elem(io.dg, at, dg, a.gdt());
      if (a.A_log && !isinf(z)) dA_tile += dg * z;  // (dg is 0 at z = +-inf)
      carry = decay_apply(decay_code(g), D, 0.f);
    }
    dA += dA_tile;
  }
  if (io.ds0) io.ds0[chain] = carry;
  if (a.A_log) dA_part[chain] = dA;
}

// dA_log[h]: the sum of the partials [rows][D] over rows and the head's channels.
__global__ void __launch_bounds__(256) scan_dA_kernel(const float *part, int rows, int D, int d, float *dA) {
  const int h = blockIdx.x;
  const long long total = (long long)rows * d;
  double s = 0.0;
  for (long long i = threadIdx.x; i < total; i += 256) s += part[(size_t)(i / d) * D + (size_t)h * d + i % d];
  __shared__ double sh[256];
  sh[threadIdx.x] = s;
  __syncthreads();
  for (int k = 128; k > 0; k >>= 1) {
    if (threadIdx.x < k) sh[threadIdx.x] += sh[threadIdx.x + k];
    __syncthreads();
  }
  if (threadIdx.x == 0) dA[h] = (float)sh[0];
}

}  // namespace

size_t scan_dA_bytes(const ScanArgs &a) { return (size_t)a.N * a.D * sizeof(float); }

static unsigned scan_blocks(const ScanArgs &a) { return (unsigned)((size_t)((a.D + kThreads - 1) / kThreads) * a.N); }

cudaError_t launch_scan_bwd(const ScanArgs &a, const ScanBwdIo &io, float *dA_part, cudaStream_t s) {
  scan_bwd_kernel<<<scan_blocks(a), kThreads, 0, s>>>(a, io, dA_part);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && a.A_log) {
    scan_dA_kernel<<<a.H, 256, 0, s>>>(dA_part, a.N, a.D, a.d, io.dA);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace kda
