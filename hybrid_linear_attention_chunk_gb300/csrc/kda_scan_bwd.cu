// Backward of the gated linear recurrence (formulas in include/kda.h, numerics
// and the layout of warps in kda_scan.cuh).
//
// The gradient of the state runs through the tiles from the last to the first,
// by the same alphas: c_{t-1} = alpha_t (d_out_t + c_t).  So a tile acts on it
// as in the forward, with (log-sum of g, what the tile adds to a zero gradient),
// and passes it on in the same ring.  The states that the tile needs come from
// the one before its first token, which the forward stored (4 bytes in 16 tokens
// of a channel); with it the tile's 16 states are rebuilt in registers.  Each
// input is read once, each gradient written once.
//
// Measured on 32768 x 4096 (4 sequences, bf16, decay logits, w = 1 - alpha): 284 us
// of the 436 us that forward and backward take, 10.25 bytes an element at 4.8 TB/s
// (0.71 of a measured copy).  It issues 53 instructions an element into 68 % of the
// slots; the two CTAs of 8 warps that 128 registers leave on an SM do not cover the
// rest of the latency.  The gate and 1 - alpha are formed twice, since keeping them
// across the hand-on of the gradient would take 64 registers more.
#include <initializer_list>

#include "kda_scan.cuh"

namespace kda {
namespace {

template <typename X, typename G, bool kLogit, typename L>
struct BwdSmem {
  static constexpr int kStates = L::V == 2 ? 32 * L::V * (int)sizeof(float) : 0;
  static constexpr int kWarpBytes = 2 * (2 * Tile<X, L, false>::kBytes + Tile<G, L, kLogit>::kBytes + kStates);
  // the ring's buffers, and after it the sums of dA_log
  static constexpr size_t join(int warps, int ranks) {
    const size_t j = ScanJoin<L>::bytes(warps, ranks), d = (size_t)warps * 32 * L::V * sizeof(float);
    return j > d ? j : d;
  }
  static constexpr size_t bytes(int warps, int ranks) { return join(warps, ranks) + (size_t)warps * kWarpBytes; }
  static constexpr int kMaxWarps = bytes(16, kScanMaxCluster) <= 227 * 1024 ? 16 : 8;
  static constexpr size_t kMost = bytes(kMaxWarps, kScanMaxCluster);
  static_assert(kMost <= 227 * 1024);
};

// sum += low, and low what that addition's rounding left out, to be added the next time.
template <int V> __device__ __forceinline__ void settle(Vec<V> &sum, Vec<V> &low) {
  const Vec<V> s = add(sum, low), part = fma(sum, all<V>(-1.f), s);
  low = fma(part, all<V>(-1.f), low);
  sum = s;
}

template <typename X, typename G, bool kLogit, bool kComp, typename L>
__global__ void __launch_bounds__(32 * BwdSmem<X, G, kLogit, L>::kMaxWarps,
                                  BwdSmem<X, G, kLogit, L>::kMaxWarps == 8 &&
                                  BwdSmem<X, G, kLogit, L>::bytes(8, 1) <= 115712 ? 2 : 1)
scan_bwd_kernel(ScanArgs a, ScanBwdIo io, float *dA_part, int cblocks) {
  constexpr int V = L::V;
  using Smem = BwdSmem<X, G, kLogit, L>;
  extern __shared__ __align__(128) char smem[];
  ScanJoin<L> sh(smem);
  const int lane = sh.lane, ranks = sh.ranks, D = a.D;
  const int block = blockIdx.x / ranks, n = block / cblocks, c0 = (block % cblocks) * L::kWide;
  const int wide = (lane % L::kLanes) * V, c = c0 + wide;
  const int tg = L::kGroups - 1 - sh.group;  // the ring's first group holds the last tokens
  const bool live = c < D;
  int bos, eos;
  scan_range(a, n, bos, eos);
  const size_t chain = (size_t)n * D + c;
  const Gate<kLogit, V> gate(a, c, live);
  float h[V], state[V];
#pragma unroll
  for (int i = 0; i < V; ++i) h[i] = state[i] = live && io.dST ? io.dST[chain + i] : 0.f;
  if (ranks > 1) cluster_sync_all();  // every CTA has started before another stores in it

  Tile<X, L, false> xs, ds;
  Tile<G, L, kLogit> gs;
  float *ss = nullptr;
  if constexpr (V == 2) {
    char *mine = smem + Smem::join(sh.warps, ranks) + sh.warp * Smem::kWarpBytes;
    xs.buf = reinterpret_cast<X *>(mine);
    ds.buf = reinterpret_cast<X *>(mine += 2 * Tile<X, L, false>::kBytes);
    gs.buf = reinterpret_cast<G *>(mine += 2 * Tile<X, L, false>::kBytes);
    ss = reinterpret_cast<float *>(mine + 2 * Tile<G, L, kLogit>::kBytes) + lane * V;
  }
  const int tiles = (eos - bos + L::kTokens - 1) / L::kTokens;  // warp tiles
  const int step = sh.warps * ranks;
  int q = sh.rank * sh.warps + sh.warp;  // the warp's place in the ring: tile tiles - 1 - q
  float s0[V];
  // first token of tile q and how many are left from it (0: no such tile)
  auto first = [&](int q) { return bos + max(tiles - 1 - q, 0) * L::kTokens; };
  auto length = [&](int q) { return q < tiles ? eos - first(q) : 0; };
  auto fetch = [&](int stage, int q) {
    const int t = first(q), len = length(q);
    gs.issue(stage, a.g, D, t, c0, len, tg, lane);
    xs.issue(stage, a.x, D, t, c0, len, tg, lane);
    ds.issue(stage, io.dO, D, t, c0, len, tg, lane);
    // the state before the lane's tile
    const bool ok = live && tg * kScanTile < len;
    const size_t slot = (size_t)(bos / kScanTile) + n + (t - bos) / kScanTile + tg;
    if constexpr (V == 2) {
      const float *from = ok ? a.states + slot * D + c : a.states;
      const unsigned to = (unsigned)__cvta_generic_to_shared(ss + stage * 32 * V);
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(from), "r"(ok ? 8 : 0) : "memory");
      copies_commit();
    } else {
      s0[0] = ok ? a.states[slot * D + c] : 0.f;
    }
  };
  if (tiles > 0) {
    fetch(0, q);
    if (V == 2) fetch(1, q + step);
  }
  // Over the lane's tiles, of which there may be thousands: a running sum, and the tile's own on top of what the
  // roundings of the running one left out.  (Where tokens are alike, so are these: of 131072 equal ones a plain sum
  // was off by 3856 half steps.)
  Vec<V> dA = all<V>(0.f), dA_tile = all<V>(0.f);
  int par = 0;
  for (int q0 = ranks > 1 ? 0 : q; q0 < tiles; q0 += step, q += step, par ^= 1) {
    const int len = length(q);
    if (V == 2) {
      copies_wait<1>();
      __syncwarp();
      gs.pad(par, len, lane);
      __syncwarp();
    }
    // forward through the tile: alpha, and what d_out meets in dg
    Vec<V> al[kScanTile], meet[kScanTile], log = all<V>(0.f), hv;
    if constexpr (V == 2) hv = pair(ss[par * 32 * V], ss[par * 32 * V + 1]);
    else hv = Vec<1>{s0[0]};
#pragma unroll
    for (int j = 0; j < kScanTile; ++j) {
      const Vec<V> l = gate.log(gs.at(par, j, tg, lane)), x = xs.at(par, j, tg, lane);
      al[j] = gate.alpha(l);
      log = add(log, l);
      meet[j] = kComp ? fma(x, all<V>(-1.f), hv) : hv;
      hv = fma(al[j], hv, kComp ? mul(x, gate.one_minus(l, al[j])) : x);
    }
    // what the tile adds to a zero gradient
    Vec<V> c1 = all<V>(0.f);
#pragma unroll
    for (int j = kScanTile - 1; j >= 0; --j) c1 = mul(al[j], add(ds.at(par, j, tg, lane), c1));
    Span<V> mine;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      mine.c[i] = decay_code(gate.unit * log.get(i));
      mine.add[i] = c1.get(i);
    }
    const bool ends = q == tiles - 1;  // (one CTA) the sequence's first tile
    float leave[V];
    if (ranks == 1) sh.ring(par, mine, q == 0, !ends, h, leave);
    else sh.cluster(par, mine, state, h);
    Vec<V> cv = lanes<V>([&](int i) { return h[i]; });
    const int rows = live ? len - tg * kScanTile : 0;
    const size_t at = (size_t)(first(q) + tg * kScanTile) * D + c;
    X *dx = static_cast<X *>(io.dx) + at;
    G *dg = static_cast<G *>(io.dg) + at;
#pragma unroll
    for (int j = kScanTile - 1; j >= 0; --j) {
      const Vec<V> grad = add(ds.at(par, j, tg, lane), cv);
      const Vec<V> z = gs.at(par, j, tg, lane);
      Vec<V> slope, scaled, l = z;
      if (kLogit) l = gate.log(z, slope, scaled);
      cv = mul(al[j], grad);
      Vec<V> out = mul(cv, meet[j]);
      if (kLogit) {
        out = mul(out, slope);
        dA_tile = fma(out, scaled, dA_tile);
      }
      if (j < rows) {
        store<V>(dx + (unsigned)(j * D), kComp ? mul(grad, gate.one_minus(l, al[j])) : grad);
        store<V>(dg + (unsigned)(j * D), out);
      }
    }
    if (kLogit) settle(dA, dA_tile);
    if (ranks == 1 && ends && io.ds0 && live && sh.group == L::kGroups - 1)
#pragma unroll
      for (int i = 0; i < V; ++i) io.ds0[chain + i] = leave[i];
    __syncwarp();
    fetch(V == 2 ? par : 0, V == 2 ? q + 2 * step : q + step);
  }
  if (V == 2) copies_wait<0>();
  if ((ranks > 1 || tiles == 0) && io.ds0 && live && sh.rank == 0 && sh.warp == 0 && sh.group == 0)
#pragma unroll
    for (int i = 0; i < V; ++i) io.ds0[chain + i] = state[i];
  if (kLogit) {  // the block's sums over time, per channel: warps and groups in order
    // The cluster's barrier, also where the cluster is one CTA: the ring's warps may
    // still wait at the CTA's barriers, barrier 0 (that of __syncthreads) among them.
    cluster_sync_all();
    float *sums = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int i = 0; i < V; ++i)
      sums[(sh.warp * L::kGroups + sh.group) * L::kWide + wide + i] = dA.get(i) / gate.ns.get(i);  // dz z = dz scaled / ns
    cluster_sync_all();
    for (int i = threadIdx.x; i < L::kWide && c0 + i < D; i += blockDim.x) {
      double s = 0.0;
      for (int w = 0; w < sh.warps * L::kGroups; ++w) s += sums[w * L::kWide + i];
      dA_part[((size_t)n * ranks + sh.rank) * D + c0 + i] = (float)s;
    }
  }
}

constexpr int kSlices = 64;  // of a head's partial sums

// Partials [rows][D] over a slice of the rows and the head's channels: to
// sums[h][slice] (doubles), or, when one slice holds all rows, to dA[h].
__global__ void __launch_bounds__(256) scan_dA_kernel(const float *part, int rows, int D, int d, double *sums, float *dA) {
  const int h = blockIdx.x, slice = blockIdx.y;
  const long long lo = (long long)rows * slice / gridDim.y, hi = (long long)rows * (slice + 1) / gridDim.y;
  double s = 0.0;
  for (long long i = lo * d + threadIdx.x; i < hi * d; i += 256) s += part[(size_t)(i / d) * D + (size_t)h * d + i % d];
  __shared__ double sh[256];
  sh[threadIdx.x] = s;
  __syncthreads();
  for (int k = 128; k > 0; k >>= 1) {
    if (threadIdx.x < k) sh[threadIdx.x] += sh[threadIdx.x + k];
    __syncthreads();
  }
  if (threadIdx.x != 0) return;
  if (gridDim.y == 1) dA[h] = (float)sh[0];
  else sums[(size_t)h * gridDim.y + slice] = sh[0];
}

__global__ void __launch_bounds__(256) scan_dA_final_kernel(const double *sums, int H, int slices, float *dA) {
  const int h = blockIdx.x * 256 + threadIdx.x;
  if (h >= H) return;
  double s = 0.0;
  for (int i = 0; i < slices; ++i) s += sums[(size_t)h * slices + i];
  dA[h] = (float)s;
}

template <typename X, typename G, bool kLogit, bool kComp, typename L>
cudaError_t bwd_l(const ScanArgs &a, const ScanBwdIo &io, float *part, int warps, int ranks, cudaStream_t s) {
  return launch_chains<L>(scan_bwd_kernel<X, G, kLogit, kComp, L>, a, warps, ranks,
                          BwdSmem<X, G, kLogit, L>::bytes(warps, ranks),
                          BwdSmem<X, G, kLogit, L>::kMost, s, a, io, part, (a.D + L::kWide - 1) / L::kWide);
}

template <typename X, typename G, bool kLogit, bool kComp, typename Wide, typename Narrow>
cudaError_t bwd_c(const ScanArgs &a, const ScanBwdIo &io, float *part, int *ranks, cudaStream_t s) {
  const ScanPlan p = scan_plan(a, Wide::V == 2, BwdSmem<X, G, kLogit, Narrow>::kMaxWarps);
  *ranks = p.ranks;
  return p.narrow ? bwd_l<X, G, kLogit, kComp, Narrow>(a, io, part, p.warps, p.ranks, s)
                  : bwd_l<X, G, kLogit, kComp, Wide>(a, io, part, p.warps, p.ranks, s);
}

template <typename X, typename G, bool kLogit>
cudaError_t bwd_t(const ScanArgs &a, const ScanBwdIo &io, float *part, int *ranks, cudaStream_t s) {
  using W = Layout<64, 2>;
  using N = Layout<16, 2>;
  using EW = Layout<32, 1>;
  using EN = Layout<8, 1>;
  if (!scan_vectors(a.D, {{a.x, sizeof(X)}, {a.g, sizeof(G)}, {io.dO, sizeof(X)}, {io.dx, sizeof(X)}, {io.dg, sizeof(G)},
                          {a.states, 4}}))
    return a.complement ? bwd_c<X, G, kLogit, true, EW, EN>(a, io, part, ranks, s)
                        : bwd_c<X, G, kLogit, false, EW, EN>(a, io, part, ranks, s);
  return a.complement ? bwd_c<X, G, kLogit, true, W, N>(a, io, part, ranks, s)
                      : bwd_c<X, G, kLogit, false, W, N>(a, io, part, ranks, s);
}

cudaError_t bwd(const ScanArgs &a, const ScanBwdIo &io, float *part, int *ranks, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (a.A_log) return a.t == KDA_BF16 ? bwd_t<B, B, true>(a, io, part, ranks, s) : bwd_t<float, float, true>(a, io, part, ranks, s);
  if (a.t == KDA_BF16)
    return a.gate == KDA_BF16 ? bwd_t<B, B, false>(a, io, part, ranks, s) : bwd_t<B, float, false>(a, io, part, ranks, s);
  return a.gate == KDA_BF16 ? bwd_t<float, B, false>(a, io, part, ranks, s) : bwd_t<float, float, false>(a, io, part, ranks, s);
}

size_t slice_bytes(const ScanArgs &a) { return (size_t)a.H * kSlices * sizeof(double); }

}  // namespace

// Slices first (8-byte aligned), then one row of channel sums per sequence and
// CTA of its cluster.  Alignment decides the cluster size, so the larger counts.
size_t scan_dA_bytes(const ScanArgs &a) {
  const int ranks = max(scan_plan(a, true, 8).ranks, scan_plan(a, false, 8).ranks);
  return slice_bytes(a) + (size_t)a.N * ranks * a.D * sizeof(float);
}

cudaError_t launch_scan_bwd(const ScanArgs &a, const ScanBwdIo &io, float *ws, cudaStream_t s) {
  double *sums = reinterpret_cast<double *>(ws);
  float *part = a.A_log ? reinterpret_cast<float *>(reinterpret_cast<char *>(ws) + slice_bytes(a)) : nullptr;
  int ranks = 1;
  cudaError_t e = bwd(a, io, part, &ranks, s);
  if (e == cudaSuccess && a.A_log) {
    const int rows = a.N * ranks, slices = min(kSlices, (int)(((long long)rows * a.d + 16383) / 16384));
    scan_dA_kernel<<<dim3(a.H, slices), 256, 0, s>>>(part, rows, a.D, a.d, sums, io.dA);
    e = cudaGetLastError();
    if (e != cudaSuccess || slices == 1) return e;
    scan_dA_final_kernel<<<(a.H + 255) / 256, 256, 0, s>>>(sums, a.H, slices, io.dA);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace kda
