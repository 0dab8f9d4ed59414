// Gated linear recurrence: h_t = alpha_t h_{t-1} + w_t x_t per channel, its
// backward, and the single-token step (formulas in include/kda.h).
//
// Numerics.  With alpha near 1 (a memory of thousands of tokens) rounding
// alpha to fp32 costs up to 3e-8 / (1 - alpha) of the state, the same way at
// every token of a constant decay.  So a step uses expm1: h' = h + (e h + u)
// with e = expm1(g), whose rounding error is relative to 1 - alpha; for
// g <= -ln 2 it uses alpha itself, so that a strong decay (alpha = 0 at the
// least) leaves nothing of h behind.  Everything is fp32.
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr float kNearOne = -0.6931472f;  // expm1 form above, exp form below

struct Decay {
  float c;     // expm1(g) or alpha
  bool near_;
  __device__ __forceinline__ float alpha() const { return near_ ? 1.f + c : c; }
  __device__ __forceinline__ float one_minus() const { return near_ ? -c : 1.f - c; }
  // alpha h + u
  __device__ __forceinline__ float apply(float h, float u) const {
    const float r = fmaf(c, h, u);
    return near_ ? h + r : r;
  }
};

__device__ __forceinline__ Decay decay_of(float g) {
  Decay d;
  d.near_ = g > kNearOne;
  d.c = d.near_ ? expm1f(g) : expf(g);
  return d;
}

// g = g_min Sigmoid(s z); slope = dg/dz.  The exponential's argument is capped
// (a NaN passes), past which Sigmoid is below 1e-34: e / (1 + e) stays finite.
__device__ __forceinline__ float gate_of(float z, float s, float g_min, float *slope) {
  const float v = -s * z;
  const float e = expf(v > 80.f ? 80.f : v);
  const float r = 1.f / (1.f + e);
  const float g = g_min * r;
  if (slope) *slope = g * (e * r) * s;
  return g;
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

constexpr int kThreads = 128;

// One thread per chain.
__global__ void __launch_bounds__(kThreads) scan_fwd_kernel(ScanArgs a) {
  const int cblocks = (a.D + kThreads - 1) / kThreads;
  const int c = (int)(blockIdx.x % cblocks) * kThreads + threadIdx.x, n = blockIdx.x / cblocks;
  if (c >= a.D) return;
  int bos, eos;
  scan_range(a, n, bos, eos);
  const size_t chain = (size_t)n * a.D + c;
  const float scale = a.A_log ? expf(a.A_log[c / a.d]) : 0.f;
  float h = a.s0 ? a.s0[chain] : 0.f;
  size_t slot = (size_t)(bos / kScanTile) + n;
  for (int t = bos; t < eos; ++t) {
    if (a.states && (t - bos) % kScanTile == 0) a.states[slot++ * a.D + c] = h;
    const size_t i = (size_t)t * a.D + c;
    float g = ld_elem(a.g, i, a.gdt());
    if (a.A_log) g = gate_of(g, scale, a.g_min, nullptr);
    const Decay dc = decay_of(g);
    const float x = ld_elem(a.x, i, a.t);
    h = dc.apply(h, a.complement ? dc.one_minus() * x : x);
    if (a.o) st_elem(a.o, i, h, a.t);
  }
  if (a.sT) a.sT[chain] = h;
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
      if (a.A_log) g = gate_of(g, scale, a.g_min, nullptr);
      const Decay dc = decay_of(g);
      const float x = ld_elem(a.x, at, a.t);
      h = dc.apply(h, a.complement ? dc.one_minus() * x : x);
    }
    float dA_tile = 0.f;
    for (int i = len - 1; i >= 0; --i) {
      const size_t at = (size_t)(t0 + i) * a.D + c;
      const float z = ld_elem(a.g, at, a.gdt());
      float slope = 1.f;
      const float g = a.A_log ? gate_of(z, scale, a.g_min, &slope) : z;
      const Decay dc = decay_of(g);
      const float x = ld_elem(a.x, at, a.t);
      const float D = ld_elem(io.dO, at, a.t) + carry;
      st_elem(io.dx, at, a.complement ? dc.one_minus() * D : D, a.t);
      const float dg = dc.alpha() * D * (a.complement ? prev[i] - x : prev[i]) * slope;
      st_elem(io.dg, at, dg, a.gdt());
      if (a.A_log && !isinf(z)) dA_tile += dg * z;  // (dg is 0 at z = +-inf)
      carry = dc.apply(D, 0.f);
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

__global__ void __launch_bounds__(kThreads) scan_step_kernel(ScanArgs a) {
  const size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= (size_t)a.N * a.D) return;
  float g = ld_elem(a.g, i, a.gdt());
  if (a.A_log) g = gate_of(g, expf(a.A_log[(i % a.D) / a.d]), a.g_min, nullptr);
  const Decay dc = decay_of(g);
  const float x = ld_elem(a.x, i, a.t);
  const float h = dc.apply(a.s0[i], a.complement ? dc.one_minus() * x : x);
  a.sT[i] = h;
  st_elem(a.o, i, h, a.t);
}

__global__ void __launch_bounds__(256) validate_scan_kernel(ScanArgs a, int *flag) {
  const size_t n = (size_t)a.T_total * a.D, stride = (size_t)gridDim.x * blockDim.x;
  int bad = 0;
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += stride) {
    const float g = ld_elem(a.g, i, a.gdt());
    if (a.A_log ? isnan(g) : !(g <= 0.f)) bad = 1;
  }
  if (blockIdx.x == 0) {
    if (a.A_log)
      for (int h = threadIdx.x; h < a.H; h += blockDim.x)
        if (!isfinite(a.A_log[h])) bad = 1;
    if (a.cu)
      for (int i = threadIdx.x; i <= a.N; i += blockDim.x) {
        const int c = a.cu[i];
        if ((i == 0 && c != 0) || c > a.T_total || (i > 0 && c < a.cu[i - 1])) bad = 1;
      }
  }
  if (bad) atomicOr(flag, bad);
}

}  // namespace

size_t scan_dA_bytes(const ScanArgs &a) { return (size_t)a.N * a.D * sizeof(float); }

static unsigned scan_blocks(const ScanArgs &a) { return (unsigned)((size_t)((a.D + kThreads - 1) / kThreads) * a.N); }

cudaError_t launch_scan_fwd(const ScanArgs &a, cudaStream_t s) {
  scan_fwd_kernel<<<scan_blocks(a), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_scan_states(const ScanArgs &a, cudaStream_t s) {
  ScanArgs b = a;
  b.o = nullptr;
  b.sT = nullptr;
  return launch_scan_fwd(b, s);
}

cudaError_t launch_scan_bwd(const ScanArgs &a, const ScanBwdIo &io, float *dA_part, cudaStream_t s) {
  scan_bwd_kernel<<<scan_blocks(a), kThreads, 0, s>>>(a, io, dA_part);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && a.A_log) {
    scan_dA_kernel<<<a.H, 256, 0, s>>>(dA_part, a.N, a.D, a.d, io.dA);
    e = cudaGetLastError();
  }
  return e;
}

cudaError_t launch_scan_step(const ScanArgs &a, cudaStream_t s) {
  const size_t n = (size_t)a.N * a.D;
  scan_step_kernel<<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_validate_scan(const ScanArgs &a, int *d_flag, cudaStream_t s) {
  validate_scan_kernel<<<512, 256, 0, s>>>(a, d_flag);
  return cudaGetLastError();
}

}  // namespace kda
