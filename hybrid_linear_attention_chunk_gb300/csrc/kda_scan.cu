// Gated linear recurrence: forward scan and single-token step (formulas in
// include/kda.h, numerics in kda_scan.cuh).
//
// The scan.  A chain (one channel of one sequence) is serial, and a batch has
// too few chains to keep HBM busy, so time is split.  A warp takes a tile of 16
// tokens x 64 channels (2 per lane) straight into registers and scans it from a
// zero state, keeping each token's sum and product of alphas; once the state
// that enters the tile is known, a token's output is sum + product * state: one
// read of the inputs, one write of the output.  Eight warps hold 128 consecutive
// tokens of a round; what their tiles do to a state meets in shared memory.
// When there are few chain blocks, the CTAs of a cluster take consecutive
// 128-token spans of a round and exchange theirs through distributed shared
// memory.  A state passes through the tiles in the recurrence's order, so it
// keeps the error of a token-by-token run and is the same from run to run.
// The loads of the next round are issued as soon as the raw inputs have been
// used, so they are in flight under the join and the stores.
#include <initializer_list>

#include "kda_scan.cuh"

namespace kda {
namespace {

template <typename X, typename G, bool kLogit, bool kComp, int V>
__global__ void __launch_bounds__(kScanThreads, 2) scan_fwd_kernel(ScanArgs a, int cblocks) {
  __shared__ ScanJoin<V> sh;
  const int ranks = (int)cluster_size(), rank = (int)cluster_rank();
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int block = blockIdx.x / ranks, n = block / cblocks, c0 = (block % cblocks) * 32 * V;
  const int c = c0 + lane * V, D = a.D;
  const bool live = c < D, whole = c0 + 32 * V <= D;  // (D is a multiple of V)
  int bos, eos;
  scan_range(a, n, bos, eos);
  const size_t chain = (size_t)n * D + c;
  float h[V], state[V], ns[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    h[i] = state[i] = live && a.s0 ? a.s0[chain + i] : 0.f;
    ns[i] = kLogit && live ? gate_scale(a.A_log[(c + i) / a.d]) : -1.f;
  }
  if (ranks == 1 && warp == kScanWarps - 1)
#pragma unroll
    for (int i = 0; i < V; ++i) sh.carry[0][lane * V + i] = h[i];

  if (ranks > 1) cluster_sync_all();  // every CTA has started before another stores in it

  Pack<X, V> xs[kScanTile];
  Pack<G, V> gs[kScanTile];
  int t = bos + rank * kScanSpan + warp * kScanTile;
  // a token past the end has alpha = 1 (z = -inf) and adds nothing
  auto fetch = [&](int at, Pack<X, V>(&xv)[kScanTile], Pack<G, V>(&gv)[kScanTile]) {
    const int left = eos - at;
    const bool full = whole && left >= kScanTile;
    load_tile<G, V>(gv, a.g, D, at, (unsigned)(c * sizeof(G)), live ? left : 0, full, kLogit ? -INFINITY : 0.f);
    load_tile<X, V>(xv, a.x, D, at, (unsigned)(c * sizeof(X)), live ? left : 0, full, 0.f);
  };
  fetch(t, xs, gs);
  int par = 0;
  for (int t0 = bos; t0 < eos; t0 += kScanSpan * ranks, t += kScanSpan * ranks, par ^= 1) {
    // from a zero state: sum[j] the state after token j, keep[j] the product of
    // the alphas up to it
    float keep[kScanTile][V], sum[kScanTile][V], logs[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      logs[i] = 0.f;
      float k = 1.f, u = 0.f;
#pragma unroll
      for (int j = 0; j < kScanTile; ++j) {
        const float g = kLogit ? gate_code(gs[j].get(i), ns[i], a.g_min) : at_most_zero(gs[j].get(i));
        const float al = alpha_of(g), x = xs[j].get(i);
        logs[i] += g;
        k *= al;
        u = fmaf(al, u, kComp ? one_minus(g, al) * x : x);
        keep[j][i] = k;
        sum[j][i] = u;
      }
    }
    // the next round's loads run under the rest of this round
    fetch(t + kScanSpan * ranks, xs, gs);
    Span<V> mine;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      mine.c[i] = decay_code(logs[i]);
      mine.add[i] = sum[kScanTile - 1][i];
    }
    if (ranks == 1) join_one<V>(sh, par, warp, lane, mine, h);
    else join_cluster<V>(sh, par, warp, lane, rank, ranks, mine, logs, state, h);
    const int left = live ? eos - t : 0;
    if (a.states && left > 0) {
      const size_t slot = (size_t)(bos / kScanTile) + n + (t - bos) / kScanTile;
      store<V>(a.states + slot * D + c, h);
    }
    char *o = static_cast<char *>(a.o) + ((size_t)t * D + c) * sizeof(X);
    const size_t row = (size_t)D * sizeof(X);
    const int rows = a.o ? left : 0;
#pragma unroll
    for (int j = 0; j < kScanTile; ++j, o += row) {
      float v[V];
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = fmaf(keep[j][i], h[i], sum[j][i]);
      if (j < rows) store<V>(reinterpret_cast<X *>(o), v);
    }
    if (ranks == 1) {
      mine.run(h);
      if (warp == kScanWarps - 1)
#pragma unroll
        for (int i = 0; i < V; ++i) sh.carry[par ^ 1][lane * V + i] = h[i];
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) h[i] = state[i];
    }
  }
  if (a.sT && live && rank == 0 && warp == kScanWarps - 1)
#pragma unroll
    for (int i = 0; i < V; ++i) a.sT[chain + i] = h[i];
}

constexpr int kStepThreads = 128;

__global__ void __launch_bounds__(kStepThreads) scan_step_kernel(ScanArgs a) {
  const size_t i = (size_t)blockIdx.x * kStepThreads + threadIdx.x;
  if (i >= (size_t)a.N * a.D) return;
  float g = ld_elem(a.g, i, a.gdt());
  if (a.A_log) g = gate_code(g, gate_scale(a.A_log[(i % a.D) / a.d]), a.g_min);
  g = at_most_zero(g);
  const float x = ld_elem(a.x, i, a.t);
  const float h = decay_apply(decay_code(g), a.s0[i], a.complement ? one_minus(g, alpha_of(g)) * x : x);
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

template <typename X, typename G, bool kLogit, bool kComp, int V>
cudaError_t fwd_v(const ScanArgs &a, cudaStream_t s) {
  const int cblocks = (a.D + 32 * V - 1) / (32 * V), ranks = scan_cluster(a, 32 * V);
  const long long blocks = (long long)cblocks * a.N * ranks;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kScanThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ranks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, scan_fwd_kernel<X, G, kLogit, kComp, V>, a, cblocks);
}

template <typename X, typename G, bool kLogit>
cudaError_t fwd_t(const ScanArgs &a, cudaStream_t s) {
  const bool pairs = scan_pairs(a.D, {a.x, a.g, a.o, a.states});
  if (a.complement) return pairs ? fwd_v<X, G, kLogit, true, 2>(a, s) : fwd_v<X, G, kLogit, true, 1>(a, s);
  return pairs ? fwd_v<X, G, kLogit, false, 2>(a, s) : fwd_v<X, G, kLogit, false, 1>(a, s);
}

}  // namespace

// A cluster grows until the grid fills the 152 SMs three times over or a round
// covers the average sequence.
int scan_cluster(const ScanArgs &a, int channels) {
  const long long blocks = (long long)((a.D + channels - 1) / channels) * a.N;
  const long long tokens = a.T_total / a.N;
  int r = 1;
  while (r < kScanMaxCluster && blocks * r < 3 * 152 && (long long)r * kScanSpan < tokens) r *= 2;
  return r;
}

cudaError_t launch_scan_fwd(const ScanArgs &a, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (a.A_log) return a.t == KDA_BF16 ? fwd_t<B, B, true>(a, s) : fwd_t<float, float, true>(a, s);
  if (a.t == KDA_BF16) return a.gate == KDA_BF16 ? fwd_t<B, B, false>(a, s) : fwd_t<B, float, false>(a, s);
  return a.gate == KDA_BF16 ? fwd_t<float, B, false>(a, s) : fwd_t<float, float, false>(a, s);
}

cudaError_t launch_scan_states(const ScanArgs &a, cudaStream_t s) {
  ScanArgs b = a;
  b.o = nullptr;
  b.sT = nullptr;
  return launch_scan_fwd(b, s);
}

cudaError_t launch_scan_step(const ScanArgs &a, cudaStream_t s) {
  const size_t n = (size_t)a.N * a.D;
  scan_step_kernel<<<(unsigned)((n + kStepThreads - 1) / kStepThreads), kStepThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_validate_scan(const ScanArgs &a, int *d_flag, cudaStream_t s) {
  validate_scan_kernel<<<512, 256, 0, s>>>(a, d_flag);
  return cudaGetLastError();
}

}  // namespace kda
