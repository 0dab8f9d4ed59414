// Gated linear recurrence: forward scan and single-token step (formulas in
// include/kda.h, numerics in kda_scan.cuh).
//
// The scan.  A chain (one channel of one sequence) is serial, and a batch has
// too few chains to keep HBM busy, so time is split.  Each lane takes 16 tokens of
// 2 channels, scans them from a zero state and keeps, per token, that sum and the
// product of alphas; once the state that enters the tile is known, a token's
// output is sum + product * state: one read of the inputs, one write of the
// output.  The state passes from tile to tile in the recurrence's order (ScanJoin
// in kda_scan.cuh) by the tiles' own log-sums, so its error grows no faster than in a
// token-by-token run, and it is the same from run to run.  Inputs come in two tiles ahead, so loads are in flight under
// everything else.
//
// Bounds and measurements (6.78 TB/s is a measured copy on the same GPU):
//   bound by HBM where chains are many: 24 packed sequences, 49152 x 4096, bf16
//   with fp32 log-decay, 240 us, 6.7 TB/s (0.99 of the copy); 15 instructions an
//   element, issue slots 41 % used;
//   few chains (262144 x 2048 of one sequence, decay logits): 661 us, 4.9 TB/s
//   (0.72): rows of 16 channels are 32-byte requests, and the logits' two
//   exponentials, reciprocal and expm1 make 28 instructions an element (67 % of
//   issue slots).  Blocks of 64 channels on clusters of 8 CTAs took 1008 us: the
//   cluster barrier of every 1024 tokens cost 1.2 us.
//   A step is one launch: 4.1 us for one sequence of 4096 channels, 6.2 us for 256.
#include <initializer_list>

#include "kda_scan.cuh"

namespace kda {
namespace {

template <typename X, typename G, bool kLogit, typename L>
struct FwdSmem {
  static constexpr int kWarpBytes = 2 * (Tile<X, L, false>::kBytes + Tile<G, L, kLogit>::kBytes);
  static constexpr size_t bytes(int warps, int ranks) { return ScanJoin<L>::bytes(warps, ranks) + (size_t)warps * kWarpBytes; }
  static constexpr int kMaxWarps = bytes(16, kScanMaxCluster) <= 227 * 1024 ? 16 : 8;
  static constexpr size_t kMost = bytes(kMaxWarps, kScanMaxCluster);
  static_assert(kMost <= 227 * 1024);
};

template <typename X, typename G, bool kLogit, bool kComp, typename L>
__global__ void __launch_bounds__(32 * FwdSmem<X, G, kLogit, L>::kMaxWarps, 1) scan_fwd_kernel(ScanArgs a, int cblocks) {
  constexpr int V = L::V;
  extern __shared__ __align__(128) char smem[];
  ScanJoin<L> sh(smem);
  const int lane = sh.lane, ranks = sh.ranks, D = a.D;
  const int block = blockIdx.x / ranks, n = block / cblocks, c0 = (block % cblocks) * L::kWide;
  const int wide = (lane % L::kLanes) * V, c = c0 + wide;
  const bool live = c < D;  // (with V = 2, D is a multiple of 4)
  int bos, eos;
  scan_range(a, n, bos, eos);
  const size_t chain = (size_t)n * D + c;
  const Gate<kLogit, V> gate(a, c, live);
  float h[V], state[V];
#pragma unroll
  for (int i = 0; i < V; ++i) h[i] = state[i] = live && a.s0 ? a.s0[chain + i] : 0.f;
  if (ranks > 1) cluster_sync_all();  // every CTA has started before another stores in it

  Tile<X, L, false> xs;
  Tile<G, L, kLogit> gs;
  if constexpr (V == 2) {
    char *mine = smem + ScanJoin<L>::bytes(sh.warps, ranks) + sh.warp * FwdSmem<X, G, kLogit, L>::kWarpBytes;
    xs.buf = reinterpret_cast<X *>(mine);
    gs.buf = reinterpret_cast<G *>(mine + 2 * Tile<X, L, false>::kBytes);
  }
  const int step = sh.warps * L::kTokens * ranks;
  int tw = bos + (sh.rank * sh.warps + sh.warp) * L::kTokens;  // the warp's first token
  // a token past the end has alpha = 1 (z = -inf) and adds nothing
  auto fetch = [&](int stage, int t) {
    gs.issue(stage, a.g, D, t, c0, eos - t, sh.group, lane);
    xs.issue(stage, a.x, D, t, c0, eos - t, sh.group, lane);
    if (V == 2) copies_commit();
  };
  if (bos < eos) {
    fetch(0, tw);
    if (V == 2) fetch(1, tw + step);
  }
  int par = 0;
  // alone, a warp stops at the sequence's end; the CTAs of a cluster run the same rounds
  for (int t0 = ranks > 1 ? bos : tw; t0 < eos; t0 += step, tw += step, par ^= 1) {
    if (V == 2) {
      copies_wait<1>();
      __syncwarp();
      gs.pad(par, eos - tw, lane);
      __syncwarp();
    }
    // from a zero state: sum[j] the state after token j, keep[j] the product of
    // the alphas up to it
    Vec<V> keep[kScanTile], sum[kScanTile], log = all<V>(0.f);
#pragma unroll
    for (int j = 0; j < kScanTile; ++j) {
      const Vec<V> l = gate.log(gs.at(par, j, sh.group, lane)), al = gate.alpha(l);
      Vec<V> u = xs.at(par, j, sh.group, lane);
      if (kComp) u = mul(u, gate.one_minus(l, al));
      log = add(log, l);
      keep[j] = j ? mul(keep[j - 1], al) : al;
      sum[j] = j ? fma(al, sum[j - 1], u) : u;
    }
    // later rounds' loads run under the rest of this round
    __syncwarp();
    if (V == 2) fetch(par, tw + 2 * step);
    else fetch(0, tw + step);
    Span<V> mine;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      mine.c[i] = decay_code(gate.unit * log.get(i));
      mine.add[i] = sum[kScanTile - 1].get(i);
    }
    const bool ends = eos - tw <= L::kTokens;  // the sequence's last tile
    float leave[V];
    if (ranks == 1) sh.ring(par, mine, tw == bos, !ends, h, leave);
    else sh.cluster(par, mine, state, h);
    const int t = tw + sh.group * kScanTile, left = live ? eos - t : 0;
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
    if (ranks == 1 && ends && a.sT && live && sh.group == L::kGroups - 1)
#pragma unroll
      for (int i = 0; i < V; ++i) a.sT[chain + i] = leave[i];
  }
  if (V == 2) copies_wait<0>();
  if ((ranks > 1 || bos == eos) && a.sT && live && sh.rank == 0 && sh.warp == 0 && sh.group == 0)
#pragma unroll
    for (int i = 0; i < V; ++i) a.sT[chain + i] = state[i];
}

constexpr int kStepThreads = 128;

// One token of every chain, V channels of one sequence per thread.
template <typename X, typename G, bool kLogit, bool kComp, int V>
__global__ void __launch_bounds__(kStepThreads) scan_step_kernel(ScanArgs a) {
  const size_t i = ((size_t)blockIdx.x * kStepThreads + threadIdx.x) * V;
  if (i >= (size_t)a.N * a.D) return;
  const Vec<V> z = values(*reinterpret_cast<const Raw<G, V> *>(static_cast<const G *>(a.g) + i));
  const Vec<V> x = values(*reinterpret_cast<const Raw<X, V> *>(static_cast<const X *>(a.x) + i));
  const Vec<V> s = values(*reinterpret_cast<const Raw<float, V> *>(a.s0 + i));
  const Gate<kLogit, V> gate(a, (int)(i % a.D), true);
  const Vec<V> l = gate.log(z);
  const Vec<V> u = kComp ? mul(x, gate.one_minus(l, gate.alpha(l))) : x;
  const Vec<V> h = lanes<V>([&](int k) { return decay_apply(decay_code(gate.unit * l.get(k)), s.get(k), u.get(k)); });
  store<V>(a.sT + i, h);
  store<V>(static_cast<X *>(a.o) + i, h);
}

__global__ void __launch_bounds__(256) validate_scan_kernel(ScanArgs a, int *flag) {
  const int tokens = a.cu ? min(max(a.cu[a.N], 0), a.T_total) : a.T_total;  // rows behind the last sequence are not read
  const size_t n = (size_t)tokens * a.D, stride = (size_t)gridDim.x * blockDim.x;
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

template <typename X, typename G, bool kLogit, bool kComp, typename L>
cudaError_t fwd_l(const ScanArgs &a, int warps, int ranks, cudaStream_t s) {
  return launch_chains<L>(scan_fwd_kernel<X, G, kLogit, kComp, L>, a, warps, ranks,
                          FwdSmem<X, G, kLogit, L>::bytes(warps, ranks),
                          FwdSmem<X, G, kLogit, L>::kMost, s, a, (a.D + L::kWide - 1) / L::kWide);
}

template <typename X, typename G, bool kLogit, bool kComp, typename Wide, typename Narrow>
cudaError_t fwd_c(const ScanArgs &a, cudaStream_t s) {
  const ScanPlan p = scan_plan(a, Wide::V == 2, FwdSmem<X, G, kLogit, Narrow>::kMaxWarps);
  return p.narrow ? fwd_l<X, G, kLogit, kComp, Narrow>(a, p.warps, p.ranks, s)
                  : fwd_l<X, G, kLogit, kComp, Wide>(a, p.warps, p.ranks, s);
}

template <typename X, typename G, bool kLogit>
cudaError_t fwd_t(const ScanArgs &a, cudaStream_t s) {
  using W = Layout<64, 2>;
  using N = Layout<16, 2>;
  using EW = Layout<32, 1>;
  using EN = Layout<8, 1>;
  if (!scan_vectors(a.D, {{a.x, sizeof(X)}, {a.g, sizeof(G)}, {a.o, sizeof(X)}, {a.states, 4}}))
    return a.complement ? fwd_c<X, G, kLogit, true, EW, EN>(a, s) : fwd_c<X, G, kLogit, false, EW, EN>(a, s);
  return a.complement ? fwd_c<X, G, kLogit, true, W, N>(a, s) : fwd_c<X, G, kLogit, false, W, N>(a, s);
}

template <typename X, typename G, bool kLogit, bool kComp, int V>
cudaError_t step_v(const ScanArgs &a, cudaStream_t s) {
  const size_t threads = ((size_t)a.N * a.D + V - 1) / V;
  scan_step_kernel<X, G, kLogit, kComp, V>
      <<<(unsigned)((threads + kStepThreads - 1) / kStepThreads), kStepThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename X, typename G, bool kLogit>
cudaError_t step_t(const ScanArgs &a, cudaStream_t s) {
  const bool v = scan_vectors(a.D, {{a.x, sizeof(X)}, {a.g, sizeof(G)}, {a.o, sizeof(X)}, {a.s0, 4}, {a.sT, 4}});
  if (a.complement) return v ? step_v<X, G, kLogit, true, 2>(a, s) : step_v<X, G, kLogit, true, 1>(a, s);
  return v ? step_v<X, G, kLogit, false, 2>(a, s) : step_v<X, G, kLogit, false, 1>(a, s);
}

}  // namespace

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
  using B = __nv_bfloat16;
  if (a.A_log) return a.t == KDA_BF16 ? step_t<B, B, true>(a, s) : step_t<float, float, true>(a, s);
  if (a.t == KDA_BF16) return a.gate == KDA_BF16 ? step_t<B, B, false>(a, s) : step_t<B, float, false>(a, s);
  return a.gate == KDA_BF16 ? step_t<float, B, false>(a, s) : step_t<float, float, false>(a, s);
}

cudaError_t launch_validate_scan(const ScanArgs &a, int *d_flag, cudaStream_t s) {
  validate_scan_kernel<<<512, 256, 0, s>>>(a, d_flag);
  return cudaGetLastError();
}

}  // namespace kda
