// Host-side checks and plumbing that the entry points of the C ABI share.
#pragma once

#include "kda_internal.cuh"

namespace kda {

// Keeps the text of a CUDA error for kda_last_cuda_error and returns KDA_ERR_CUDA.
kda_status cuda_fail(cudaError_t e);

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool aligned_to(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

inline bool dim_ok(int d) { return d == kMinDim || d == 32 || d == 64 || d == kMaxDim; }

inline bool dtype_ok(kda_dtype t) { return t == KDA_F32 || t == KDA_BF16; }

inline size_t esize(kda_dtype t) { return t == KDA_BF16 ? 2 : 4; }

struct Range {
  uintptr_t lo, hi;
};

inline Range span(const void *p, size_t bytes) {
  uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Range{a, a + bytes};
}

inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo; }

// Runs a check kernel, waits for it and reports KDA_ERR_RANGE on a bad value.
template <class Launch>
kda_status run_validation(cudaStream_t s, Launch launch) {
  int *d_flag = nullptr;
  cudaError_t e = cudaMallocAsync(reinterpret_cast<void **>(&d_flag), sizeof(int), s);
  if (e != cudaSuccess) return cuda_fail(e);
  int h_flag = 0;
  e = cudaMemsetAsync(d_flag, 0, sizeof(int), s);
  if (e == cudaSuccess) e = launch(d_flag);
  if (e == cudaSuccess) e = cudaMemcpyAsync(&h_flag, d_flag, sizeof(int), cudaMemcpyDeviceToHost, s);
  cudaError_t ef = cudaFreeAsync(d_flag, s);
  if (e == cudaSuccess) e = ef;
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e);
  return h_flag ? KDA_ERR_RANGE : KDA_OK;
}

// No output may overlap an input or another output, but for the listed pairs
// (in, out) that may be the same buffer.
inline bool aliased(const Range *in, int n_in, const Range *out, int n_out, int same_in = -1, int same_out = -1) {
  for (int o = 0; o < n_out; ++o) {
    for (int i = 0; i < n_in; ++i) {
      if (i == same_in && o == same_out && in[i].lo == out[o].lo && in[i].hi == out[o].hi) continue;
      if (overlap(in[i], out[o])) return true;
    }
    for (int p = 0; p < o; ++p)
      if (overlap(out[p], out[o])) return true;
  }
  return false;
}

// A workspace of `need` bytes: the caller's, or one allocated on s around `run`.
template <class Run>
kda_status with_workspace(void *ws, size_t ws_bytes, size_t need, cudaStream_t s, Run run) {
  if (ws) {
    if (ws_bytes < need) return KDA_ERR_SHAPE;
    if (!aligned16(ws)) return KDA_ERR_ALIGN;
  }
  cudaError_t e;
  if (ws || need == 0) {
    e = run(ws);
  } else {
    void *tmp = nullptr;
    e = cudaMallocAsync(&tmp, need, s);
    if (e == cudaSuccess) {
      e = run(tmp);
      const cudaError_t ef = cudaFreeAsync(tmp, s);
      if (e == cudaSuccess) e = ef;
    }
  }
  return e == cudaSuccess ? KDA_OK : cuda_fail(e);
}

inline size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace kda
