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

template <typename X, typename G, bool kLogit, int V>
struct FwdSmem {
  static constexpr int kWarpBytes = 2 * (Tile<X, V, false>::kBytes + Tile<G, V, kLogit>::kBytes);
  static constexpr int kBytes = (int)sizeof(ScanJoin<V>) + kScanWarps * kWarpBytes;
};

template <typename X, typename G, bool kLogit, bool kComp, int V>
__global__ void __launch_bounds__(kScanThreads, FwdSmem<X, G, kLogit, V>::kBytes <= 115712 ? 2 : 1)
scan_fwd_kernel(ScanArgs a, int cblocks) {
  extern __shared__ __align__(128) char smem[];
  ScanJoin<V> &sh = *reinterpret_cast<ScanJoin<V> *>(smem);
  const int ranks = (int)cluster_size(), rank = (int)cluster_rank();
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int block = blockIdx.x / ranks, n = block / cblocks, c0 = (block % cblocks) * 32 * V;
  const int c = c0 + lane * V, D = a.D;
  const bool live = c < D;  // (with V = 2, D is a multiple of 4)
  int bos, eos;
  scan_range(a, n, bos, eos);
  const size_t chain = (size_t)n * D + c;
  const Gate<kLogit, V> gate(a, c, live);
  float h[V], state[V];
#pragma unroll
  for (int i = 0; i < V; ++i) h[i] = state[i] = live && a.s0 ? a.s0[chain + i] : 0.f;
  if (ranks == 1 && warp == kScanWarps - 1)
#pragma unroll
    for (int i = 0; i < V; ++i) sh.carry[0][lane * V + i] = h[i];
  if (ranks > 1) cluster_sync_all();  // every CTA has started before another stores in it

  Tile<X, V, false> xs;
  Tile<G, V, kLogit> gs;
  if constexpr (V == 2) {
    char *mine = smem + sizeof(ScanJoin<V>) + warp * FwdSmem<X, G, kLogit, V>::kWarpBytes;
    xs.buf = reinterpret_cast<X *>(mine);
    gs.buf = reinterpret_cast<G *>(mine + 2 * Tile<X, V, false>::kBytes);
  }
  const int step = kScanSpan * ranks;
  int t = bos + rank * kScanSpan + warp * kScanTile;
  // a token past the end has alpha = 1 (z = -inf) and adds nothing
  auto fetch = [&](int stage, int at) {
    gs.issue(stage, a.g, D, at, c0, eos - at, lane);
    xs.issue(stage, a.x, D, at, c0, eos - at, lane);
    if (V == 2) copies_commit();
  };
  if (bos < eos) {
    fetch(0, t);
    if (V == 2) fetch(1, t + step);
  }
  int par = 0;
  for (int t0 = bos; t0 < eos; t0 += step, t += step, par ^= 1) {
    if (V == 2) {
      copies_wait<1>();
      __syncwarp();
      gs.pad(par, eos - t, lane);
      __syncwarp();
    }
    // from a zero state: sum[j] the state after token j, keep[j] the product of
    // the alphas up to it
    Vec<V> keep[kScanTile], sum[kScanTile], log = all<V>(0.f);
#pragma unroll
    for (int j = 0; j < kScanTile; ++j) {
      const Vec<V> l = gate.log(gs.at(par, j, lane)), al = gate.alpha(l);
      Vec<V> u = xs.at(par, j, lane);
      if (kComp) u = mul(u, gate.one_minus(l, al));
      log = add(log, l);
      keep[j] = j ? mul(keep[j - 1], al) : al;
      sum[j] = j ? fma(al, sum[j - 1], u) : u;
    }
    // later rounds' loads run under the rest of this round
    __syncwarp();
    if (V == 2) fetch(par, t + 2 * step);
    else fetch(0, t + step);
    Span<V> mine;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      mine.c[i] = decay_code(gate.unit * log.get(i));
      mine.add[i] = sum[kScanTile - 1].get(i);
    }
    if (ranks == 1) join_one<V>(sh, par, warp, lane, mine, h);
    else join_cluster<V>(sh, par, warp, lane, rank, ranks, mine, state, h);
    const int left = live ? eos - t : 0;
    const Vec<V> hv = lanes<V>([&](int i) { return h[i]; });
    if (a.states && left > 0) {
      const size_t slot = (size_t)(bos / kScanTile) + n + (t - bos) / kScanTile;
      store<V>(a.states + slot * D + c, hv);
    }
    if (a.o) {
      X *o = static_cast<X *>(a.o) + (size_t)t * D + c;
      if (__all_sync(0xffffffffu, left >= kScanTile)) {
#pragma unroll
        for (int j = 0; j < kScanTile; ++j) store<V>(o + (unsigned)(j * D), fma(keep[j], hv, sum[j]));
      } else {
#pragma unroll
        for (int j = 0; j < kScanTile; ++j)
          if (j < left) store<V>(o + (unsigned)(j * D), fma(keep[j], hv, sum[j]));
      }
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
  if (V == 2) copies_wait<0>();
  if (a.sT && live && rank == 0 && warp == kScanWarps - 1)
#pragma unroll
    for (int i = 0; i < V; ++i) a.sT[chain + i] = h[i];
}

constexpr int kStepThreads = 128;

template <bool kLogit>
__device__ __forceinline__ float step(const ScanArgs &a, int c, Vec<1> z, Vec<1> x, float h) {
  const Gate<kLogit, 1> gate(a, c, true);
  const Vec<1> l = gate.log(z);
  return decay_apply(decay_code(gate.unit * l.v), h, a.complement ? gate.one_minus(l, gate.alpha(l)).v * x.v : x.v);
}

__global__ void __launch_bounds__(kStepThreads) scan_step_kernel(ScanArgs a) {
  const size_t i = (size_t)blockIdx.x * kStepThreads + threadIdx.x;
  if (i >= (size_t)a.N * a.D) return;
  const Vec<1> z{ld_elem(a.g, i, a.gdt())}, x{ld_elem(a.x, i, a.t)};
  const float h = a.A_log ? step<true>(a, (int)(i % a.D), z, x, a.s0[i]) : step<false>(a, 0, z, x, a.s0[i]);
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
  const auto kernel = scan_fwd_kernel<X, G, kLogit, kComp, V>;
  constexpr int smem = FwdSmem<X, G, kLogit, V>::kBytes;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kScanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ranks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, cblocks);
}

template <typename X, typename G, bool kLogit>
cudaError_t fwd_t(const ScanArgs &a, cudaStream_t s) {
  const bool v = scan_vectors(a.D, {{a.x, sizeof(X)}, {a.g, sizeof(G)}, {a.o, sizeof(X)}, {a.states, 4}});
  if (a.complement) return v ? fwd_v<X, G, kLogit, true, 2>(a, s) : fwd_v<X, G, kLogit, true, 1>(a, s);
  return v ? fwd_v<X, G, kLogit, false, 2>(a, s) : fwd_v<X, G, kLogit, false, 1>(a, s);
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
