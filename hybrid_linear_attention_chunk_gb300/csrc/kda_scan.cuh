// Device pieces that the kernels of the gated linear recurrence share
// (kda_scan.cu, kda_scan_bwd.cu).
//
// Numerics, in half steps of fp32 (2^-24 relative).  With alpha near 1 (a memory of
// thousands of tokens) rounding alpha to fp32 costs up to 3e-8 / (1 - alpha) of the
// state, the same way at every token of a constant decay.  So the decay of a whole
// 16-token tile, by which a state is carried on, comes from the sum of its logs:
// h' = h + (e h + B) with e = expm1(sum g) when sum g > -1/8, whose rounding error is
// relative to 1 - alpha, and alpha itself below that, so that a strong decay (alpha
// = 0 at the least) leaves nothing of h behind.  What is left of a state after a tile
// of log-sum G is off by at most 9 + 18 |G| more: 16 |G| from the sum, 4 + 2 |G| from the
// power (less from expm1), 3 where spans join, 2 where they act.  (With logits g itself
// is off by (10 + 7 |s z|) |g|, 6 of the 7 from s.)
//   Inside a tile, products of up to 16 alphas multiply the state (or gradient) that
// enters it.  Each alpha is a power off by up to 4 half steps and by |g| from its
// argument, and each product rounds: 16 (5 + |g|) at the tile's last token.  They
// reach the tile's outputs (in the backward its gradients, and the states that it
// rebuilds), and nothing that is carried on: out of a sequence's last token and its
// final state may differ by as much.
//   w = 1 - alpha comes from expm1(g) too.  Everything is fp32; alphas below 2^-126 are 0.
//
// The decay of a tile or span is one float c: the sign bit set means c = e
// (e <= 0; -0 for a sum of 0), clear means c = alpha.
#pragma once

#include "kda_internal.cuh"
#include "kda_packed.cuh"

namespace kda {

constexpr float kNearOne = -0.125f;

__device__ __forceinline__ bool is_near(float c) { return __float_as_int(c) < 0; }

// expm1(g) on (-1/8, 0] as g + g^2 q(g), q the quadratic with the least maximum
// relative error there (a reweighted least-squares fit to the series): 1.96e-8
// of the value, a third of half a step.
constexpr float kExpm1C0 = 0.4999971389770508f, kExpm1C1 = 0.16652730107307434f, kExpm1C2 = 0.03972300514578819f;
__device__ __forceinline__ float expm1_near(float g) {
  return fmaf(g * g, fmaf(g, fmaf(g, kExpm1C2, kExpm1C1), kExpm1C0), g);
}

__device__ __forceinline__ float decay_code(float g) {
  return g > kNearOne && g <= 0.f ? -fabsf(expm1_near(g)) : fast_exp2(g * kLog2e);
}

// The code of two spans in a row, c after d.  Near 1 both, e = c + d + c d; past
// -1/8 it becomes the product of the alphas, as 1 + e would lose what e has
// rounded to: e's error is relative to e, and alpha may be far smaller.
__device__ __forceinline__ float decay_join(float c, float d) {
  const float e = fmaf(c, d, c + d);
  const float alpha = (is_near(c) ? 1.f + c : c) * (is_near(d) ? 1.f + d : d);
  return is_near(c) && is_near(d) && e > kNearOne ? -fabsf(e) : alpha;  // (0 keeps its sign bit)
}

// alpha h + u
__device__ __forceinline__ float decay_apply(float c, float h, float u) {
  float r = fmaf(c, h, u);
  if (is_near(c)) r += h;
  return r;
}

// -exp(A) log2(e), never 0: the product with z = -inf, a masked token, stays inf.  A NaN stays one.
__device__ __forceinline__ float gate_scale(float A_log) {
  float s = -kLog2e * expf(A_log);
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(s) : "f"(-1e-37f));
  return s;
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

// V consecutive elements as they lie in memory, as fp32.
__device__ __forceinline__ Vec<1> values(float v) { return Vec<1>{v}; }
__device__ __forceinline__ Vec<2> values(float2 v) { return pair(v.x, v.y); }
__device__ __forceinline__ Vec<1> values(unsigned short v) { return Vec<1>{__uint_as_float((unsigned)v << 16)}; }
__device__ __forceinline__ Vec<2> values(unsigned v) { return pair(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)); }
template <typename T, int V> struct RawOf;
template <> struct RawOf<float, 1> { using type = float; };
template <> struct RawOf<float, 2> { using type = float2; };
template <> struct RawOf<__nv_bfloat16, 1> { using type = unsigned short; };
template <> struct RawOf<__nv_bfloat16, 2> { using type = unsigned; };
template <typename T, int V> using Raw = typename RawOf<T, V>::type;
__device__ __forceinline__ float raw_of(const float (&f)[1]) { return f[0]; }
__device__ __forceinline__ float2 raw_of(const float (&f)[2]) { return make_float2(f[0], f[1]); }

template <int V> __device__ __forceinline__ void store(float *p, Vec<V> v) {
  if constexpr (V == 2) *reinterpret_cast<float2 *>(p) = make_float2(v.get(0), v.get(1));
  else *p = v.v;
}
template <int V> __device__ __forceinline__ void store(__nv_bfloat16 *p, Vec<V> v) {
  if constexpr (V == 2) *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v.get(0), v.get(1));
  else *p = __float2bfloat16_rn(v.v);
}

// --------------------------------------------------------- layout of a warp
// Each lane holds V channels of 16 consecutive tokens.  The lanes of a warp are
// kGroups groups along the sequence, of kWide / V lanes that cover kWide
// channels: 64 channels x 16 tokens where there are many chains, 16 x 64 where
// there are few (32 x 16 and 8 x 64 in the elementwise form, V = 1).
template <int kWide_, int V_>
struct Layout {
  static constexpr int kWide = kWide_, V = V_;
  static constexpr int kLanes = kWide / V, kGroups = 32 / kLanes, kTokens = kScanTile * kGroups;
  static constexpr bool kClusters = kWide < 64;  // as scan_plan() has it
};

// The input tiles of a warp, of one array.  Two ways in:
//  V = 2: 16-byte asynchronous copies into the warp's own shared memory, two
//  tiles ahead, so that what is in flight costs no registers (needs 16-byte
//  aligned arrays and rows).  Token j of group g lies in row 16 g + (j ^ g), so
//  that the groups' rows of one j fall into different banks;
//  V = 1: elementwise loads into registers, for everything else.
// Tokens past the end, and channels past D, read as 0 (kPad: -inf).
template <typename T, typename L, bool kPad, int V = L::V> struct Tile;

template <typename T, typename L, bool kPad> struct Tile<T, L, kPad, 2> {
  static constexpr int kChunk = 16 / (int)sizeof(T);        // elements of a copy
  static constexpr int kPerRow = L::kWide / kChunk;
  static constexpr int kElems = L::kTokens * L::kWide;
  static constexpr int kBytes = kElems * (int)sizeof(T);
  T *buf;                                                   // [2][kTokens][kWide]
  __device__ __forceinline__ static int place(int r) { return (r & ~(kScanTile - 1)) | ((r ^ r / kScanTile) & (kScanTile - 1)); }
  __device__ __forceinline__ void issue(int stage, const void *base, int D, int t, int c0, int len, int, int lane) {
    T *dst = buf + stage * kElems;
    const int row = lane / kPerRow, col = (lane % kPerRow) * kChunk;
    const T *src = static_cast<const T *>(base) + ((size_t)t * D + c0 + col);
    const unsigned to = (unsigned)__cvta_generic_to_shared(dst + col);
    const bool in = c0 + col < D;
#pragma unroll
    for (int k = 0; k < L::kTokens * kPerRow / 32; ++k) {
      const int r = row + k * (32 / kPerRow);
      const bool ok = in && r < len;
      copy(to + place(r) * L::kWide * (int)sizeof(T), ok ? src + (size_t)(unsigned)r * (unsigned)D : static_cast<const T *>(base),
           ok ? 16 : 0);
    }
  }
  static __device__ __forceinline__ void copy(unsigned to, const void *from, int size) {
    if (L::kWide == 64)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(size) : "memory");
    else  // the neighbouring channels' blocks read the rest of the line at about the same time
      asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(size) : "memory");
  }
  // after the copies have landed, before the first read
  __device__ __forceinline__ void pad(int stage, int len, int lane) {
    if (kPad && len < L::kTokens) {
      T *dst = buf + stage * kElems;
      for (int i = max(len, 0) * L::kWide + lane; i < kElems; i += 32)
        dst[place(i / L::kWide) * L::kWide + i % L::kWide] = (T)-INFINITY;
    }
  }
  // token j of group g, for a lane
  __device__ __forceinline__ Vec<2> at(int stage, int j, int g, int lane) const {
    const T *p = buf + stage * kElems + (g * kScanTile + (j ^ g)) * L::kWide;
    return values(reinterpret_cast<const Raw<T, 2> *>(p)[lane % L::kLanes]);
  }
};

template <typename T, typename L, bool kPad> struct Tile<T, L, kPad, 1> {
  static constexpr int kBytes = 0;
  Raw<T, 1> v[kScanTile];
  // (a lane loads what it will use: group g's tokens)
  __device__ __forceinline__ void issue(int, const void *base, int D, int t, int c0, int len, int g, int lane) {
    const int c = c0 + lane % L::kLanes;
    const T *src = static_cast<const T *>(base) + ((size_t)(t + g * kScanTile) * D + c);
    len = c < D ? len - g * kScanTile : 0;
#pragma unroll
    for (int j = 0; j < kScanTile; ++j) {
      v[j] = sizeof(T) == 2 ? (kPad ? 0xff80 : 0) : (kPad ? -INFINITY : 0.f);
      if (j < len) v[j] = __ldcs(reinterpret_cast<const Raw<T, 1> *>(src + (unsigned)(j * D)));
    }
  }
  __device__ __forceinline__ void pad(int, int, int) {}
  __device__ __forceinline__ Vec<1> at(int, int j, int, int) const { return values(v[j]); }
};

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft> __device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

__device__ __forceinline__ float clamp_127(float x) {
  asm("min.NaN.f32 %0, %0, %1;\n\tmax.NaN.f32 %0, %0, %2;" : "+f"(x) : "f"(127.f), "f"(-127.f));
  return x;
}

// How a token's alpha and 1 - alpha come from its log-decay, or from its logit
// through r = Sigmoid(s z), g = g_min r.  `log` is g or r; tile sums of it give
// the tile's log-decay as `unit` times the sum.
template <bool kLogit, int V>
struct Gate {
  Vec<V> ns;                     // -s log2(e)
  float unit, rate, edge;        // g = unit log; log2(alpha) = rate log; near 1 on log's near side of edge
  float a0, a1, a2, a3;          // 1 - alpha near 1, a cubic times log
  __device__ __forceinline__ Gate(const ScanArgs &a, int c, bool live) {
    ns = lanes<V>([&](int i) { return kLogit && live ? gate_scale(a.A_log[(c + i) / a.d]) : -1.f; });
    unit = kLogit ? a.g_min : 1.f;
    rate = unit * kLog2e;
    edge = kNearOne / unit;
    a0 = -unit;
    a1 = -unit * unit * kExpm1C0;
    a2 = -unit * unit * unit * kExpm1C1;
    a3 = -unit * unit * unit * unit * kExpm1C2;
  }
  __device__ __forceinline__ Vec<V> log(Vec<V> z) const {
    if (!kLogit) return z;
    const Vec<V> e = mul(ns, z);
    const Vec<V> d = add(all<V>(1.f), lanes<V>([&](int i) { return fast_exp2(e.get(i)); }));
    return lanes<V>([&](int i) { return fast_rcp(d.get(i)); });
  }
  // The same, with dg/dz = g (1 - Sigmoid) s and `x` = -s log2(e) z.  With e = 2^x,
  // Sigmoid = r = 1 / (1 + e) and 1 - Sigmoid = e r.  x is held in +-127 (a NaN
  // passes): there e is finite, and at the ends r, or e, is flushed to 0, so that
  // z = +-inf has slope 0 exactly, and x times a gradient is finite there.
  __device__ __forceinline__ Vec<V> log(Vec<V> z, Vec<V> &slope, Vec<V> &x) const {
    const Vec<V> v = mul(ns, z);
    x = lanes<V>([&](int i) { return clamp_127(v.get(i)); });
    const Vec<V> e = lanes<V>([&](int i) { return fast_exp2(x.get(i)); });
    const Vec<V> d = add(all<V>(1.f), e), r = lanes<V>([&](int i) { return fast_rcp(d.get(i)); });
    slope = mul(mul(mul(ns, all<V>(-unit / kLog2e)), r), mul(e, r));
    return r;
  }
  __device__ __forceinline__ Vec<V> alpha(Vec<V> l) const {
    const Vec<V> e = mul(all<V>(rate), l);
    return lanes<V>([&](int i) { return fast_exp2(e.get(i)); });
  }
  __device__ __forceinline__ Vec<V> one_minus(Vec<V> l, Vec<V> al) const {
    Vec<V> p = fma(l, all<V>(a3), all<V>(a2));
    p = mul(l, fma(l, fma(l, p, all<V>(a1)), all<V>(a0)));
    const Vec<V> f = fma(al, all<V>(-1.f), all<V>(1.f));
    return lanes<V>([&](int i) { return (kLogit ? l.get(i) < edge : l.get(i) > edge) ? p.get(i) : f.get(i); });
  }
};

// ------------------------------------------------------------------ clusters
// A chain block (one sequence, kWide channels) runs on one cluster; its CTAs take
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
// Stores at the same shared-memory place of CTA `rank`.
template <typename T>
__device__ __forceinline__ void store_remote(T *local, int rank, const T &v) {
  const unsigned addr = (unsigned)__cvta_generic_to_shared(local);
  unsigned remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  const float *f = reinterpret_cast<const float *>(&v);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 8); ++i)
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(remote + 8 * i), "f"(f[2 * i]), "f"(f[2 * i + 1])
                 : "memory");
}

constexpr int kScanMaxCluster = 8;

// What a span of tokens does to the state, per channel of a lane: the decay
// code of its log-sum, and what it adds.
template <int V> struct __align__(8 * V) Span {
  float c[V], add[V];
  __device__ __forceinline__ void run(float (&h)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) h[i] = decay_apply(c[i], h[i], add[i]);
  }
  // this span after `first`
  __device__ __forceinline__ void after(const Span &first) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      add[i] = decay_apply(c[i], first.add[i], add[i]);
      c[i] = decay_join(c[i], first.c[i]);
    }
  }
  __device__ __forceinline__ Span up(int lanes) const {
    Span r;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      r.c[i] = __shfl_up_sync(0xffffffffu, c[i], lanes);
      r.add[i] = __shfl_up_sync(0xffffffffu, add[i], lanes);
    }
    return r;
  }
};

__device__ __forceinline__ void barrier_sync(int id, int threads) {
  asm volatile("barrier.cta.sync.aligned %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void barrier_arrive(int id, int threads) {
  asm volatile("barrier.cta.arrive.aligned %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Brings every tile the state that enters it, in the order the recurrence runs.
//   One CTA for a chain block: the warps take the tiles of a sequence in turn
//   and hand the state on in a ring.  A warp knows beforehand what its tile does,
//   so a state waits for a load, a step and a store per tile, and one warp's
//   arithmetic runs under another's waiting.  Warp w waits at named barrier w for
//   its predecessor's arrival, which is never a round ahead, as the predecessor's
//   own next state comes through the waiter.  So the ring has every barrier of the
//   CTA, that of __syncthreads (0) among them, and uses with different thread counts
//   must not meet: a kernel on this path has the cluster's barrier for anything else.
//   (Rings of teams of 2, 4 and 8 warps that join their tiles first were slower:
//   262144 x 2048 in 0.68 to 0.99 ms against 0.65 to 0.75.)
//   A cluster: its CTAs take consecutive spans of a round.  Warp 0 joins its
//   CTA's warps into one span and stores it in every CTA; each thread keeps the
//   round's state in registers.
// Two buffers each: what one round reads, the round after next overwrites.
template <typename L>
struct ScanJoin {
  static constexpr int V = L::V;
  float *carry;                 // one CTA's: [2][warps][kWide]
  Span<V> *tile, *cta;          // a cluster's: [2][warps][kLanes], [2][ranks][kLanes]
  int warps, warp, lane, group, rank, ranks;

  static constexpr size_t bytes(int warps, int ranks) {
    return ranks > 1 ? (2 * warps + 2 * ranks) * L::kLanes * sizeof(Span<V>) : 2 * warps * L::kWide * sizeof(float);
  }
  __device__ __forceinline__ explicit ScanJoin(char *smem) {
    warps = blockDim.x / 32;
    warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    lane = threadIdx.x & 31;
    group = lane / L::kLanes;
    ranks = L::kClusters ? (int)cluster_size() : 1;
    rank = L::kClusters ? (int)cluster_rank() : 0;
    carry = reinterpret_cast<float *>(smem);
    tile = reinterpret_cast<Span<V> *>(smem);
    cta = tile + 2 * warps * L::kLanes;
  }

  // A lane's tile -> `upto`, with the tiles before it in its warp; `before`, those alone.
  __device__ __forceinline__ void groups(const Span<V> &mine, Span<V> &upto, Span<V> &before) const {
    upto = mine;
    if (L::kGroups > 1) {
#pragma unroll
      for (int d = 1; d < L::kGroups; d *= 2) {
        const Span<V> o = upto.up(d * L::kLanes);
        if (group >= d) upto.after(o);
      }
      before = upto.up(L::kLanes);
    }
  }

  // h: in, the sequence's first state (read with `first`); out, the state that
  // enters the tile.  out: the state that leaves the warp's tiles, in the last
  // group.  `more`: a tile of another warp follows.
  __device__ __forceinline__ void ring(int par, const Span<V> &mine, bool first, bool more, float (&h)[V],
                                       float (&out)[V]) {
    const int wide = (lane % L::kLanes) * V, next = warp + 1 < warps ? warp + 1 : 0, npar = next ? par : par ^ 1;
    using F = Raw<float, V>;
    const F *in = reinterpret_cast<const F *>(carry + (par * warps + warp) * L::kWide + wide);
    F *to = reinterpret_cast<F *>(carry + (npar * warps + next) * L::kWide + wide);
    const bool gives = more && group == L::kGroups - 1;
    Span<V> upto, before;
    groups(mine, upto, before);
    if (!first) {
      barrier_sync(warp, 64);
      const Vec<V> v = values(*in);
#pragma unroll
      for (int i = 0; i < V; ++i) h[i] = v.get(i);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = h[i];
    upto.run(out);
    if (gives) *to = raw_of(out);
    if (more) barrier_arrive(next, 64);
    if (group > 0) before.run(h);
  }

  // state: in, the state that enters the cluster's round, out, the one that
  // leaves it; h: the one that enters the tile.
  __device__ __forceinline__ void cluster(int par, const Span<V> &mine, float (&state)[V], float (&h)[V]) {
    const int l = lane % L::kLanes;
    Span<V> upto, before;
    groups(mine, upto, before);
    Span<V> *tiles = tile + par * warps * L::kLanes + l, *spans = cta + par * ranks * L::kLanes + l;
    if (group == L::kGroups - 1) tiles[warp * L::kLanes] = upto;
    __syncthreads();
    if (warp == 0) {
      Span<V> all = tiles[0];
      for (int w = 1; w < warps; ++w) {
        Span<V> t = tiles[w * L::kLanes];
        t.after(all);
        all = t;
      }
      for (int r = group; r < ranks; r += L::kGroups) store_remote(spans + rank * L::kLanes, r, all);
    }
    cluster_sync_all();
    for (int r = 0; r < rank; ++r) spans[r * L::kLanes].run(state);
#pragma unroll
    for (int i = 0; i < V; ++i) h[i] = state[i];
    for (int r = rank; r < ranks; ++r) spans[r * L::kLanes].run(state);
    for (int w = 0; w < warp; ++w) tiles[w * L::kLanes].run(h);
    if (group > 0) before.run(h);
  }
};

// How chains and time are laid over the GPU.
//   Blocks of 64 channels (two CTAs of 8 warps on an SM, as far as shared memory
//   goes) when there are enough of them for the 152 SMs; else blocks of 16
//   channels, whose warps span four times the tokens: 32768 x 4096 of one
//   sequence took 200 us against 240 in blocks of 64 with clusters, 262144 x 128
//   0.2 ms against 0.7.  When even those are at most one for an SM, CTAs of
//   `most` warps, and clusters along the sequence while the grid has room for
//   them and the sequences are longer than a round.
//   The elementwise form has blocks of 32 and 8 channels, the narrow ones only
//   when clusters alone would leave most SMs without work.
struct ScanPlan {
  bool narrow;
  int warps, ranks;
};
inline ScanPlan scan_plan(const ScanArgs &a, bool vectors, int most) {
  const int wide = vectors ? 64 : 32, narrow = wide / 4;
  const long long tokens = a.T_total / a.N;
  const auto blocks = [&](int w) { return (long long)((a.D + w - 1) / w) * a.N; };
  ScanPlan p{blocks(wide) < (vectors ? 152 : 40), 8, 1};
  const long long b = blocks(p.narrow ? narrow : wide);
  const int span = p.narrow ? 64 : 16;  // tokens of a warp
  if (p.narrow && b <= 152 && tokens > 512) p.warps = most;
  if (p.narrow || !vectors)
    while (p.ranks < kScanMaxCluster && b * p.ranks * 2 <= (p.narrow ? 152 : 304) &&
           (long long)p.ranks * p.warps * span < tokens)
      p.ranks *= 2;
  return p;
}

// Launches one cluster of `ranks` CTAs for each chain block.  `most`: the most
// shared memory that any layout of this kernel takes.  The limit belongs to the
// kernel, which other threads may be about to launch on another layout, so every
// call sets the same.
template <typename L, typename... P>
cudaError_t launch_chains(void (*kernel)(P...), const ScanArgs &a, int warps, int ranks, size_t smem, size_t most,
                          cudaStream_t s, P... args) {
  const long long blocks = (long long)((a.D + L::kWide - 1) / L::kWide) * a.N * ranks;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(32 * warps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ranks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;  // (of one CTA too: the cluster barrier is then a barrier of that CTA)
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Whether rows of D elements of every given array can be copied 16 bytes at a
// time: (address, element size) pairs.
struct RowArray {
  const void *p;
  int size;
};
inline bool scan_vectors(int D, std::initializer_list<RowArray> arrays) {
  for (const RowArray &r : arrays)
    if (r.p && ((reinterpret_cast<uintptr_t>(r.p) & 15) || ((size_t)D * r.size) % 16)) return false;
  return true;
}

}  // namespace kda
