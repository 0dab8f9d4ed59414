// Norms before and after a block, fused with its gate and residual scale, and
// their backward (formulas in include/kda.h).
//
// A row is read once, held in registers across its sums, and written once:
// a group of kThreads threads (2 lanes to 512 threads, by the width) holds
// kChunks pieces of V elements per thread.  Sums run in fp32, per thread, then
// by shuffles, then over the warps in order.
//
// Measured (6.78 TB/s is a measured copy on the same GPU): the forward is bound by
// HBM, 32768 x 4096 with gate and fp32 residual 272 us, 6.9 TB/s; rows of 128
// (262144, gate) 35.1 us, 5.7 TB/s (0.85), where latency of the short rows shows.
// Forward and backward of 16384 x 4096 in bf16 take 342 us, of them the backward
// 225 us: 16 bytes an element at 4.8 TB/s (0.70).  It issues 77 instructions an
// element into 59 % of the slots: 128 registers leave two blocks of 256 on an SM, too
// few to run under one another's two sums over each row.
#include <initializer_list>
#include <type_traits>

#include "kda_internal.cuh"
#include "kda_packed.cuh"

namespace kda {
namespace {

// Sigmoid(g), with the power e = exp(-g) it came from.
template <int P> __device__ __forceinline__ Vec<P> sigmoid_of(Vec<P> g, Vec<P> &e) {
  const Vec<P> x = mul(g, all<P>(-kLog2e));
  e = lanes<P>([&](int i) { return fast_exp2(x.get(i)); });
  const Vec<P> d = add(e, all<P>(1.f));
  return lanes<P>([&](int i) { return fast_rcp(d.get(i)); });
}
// 1 - Sigmoid: the difference below a half, e r above it, where e is finite.
template <int P> __device__ __forceinline__ Vec<P> sigmoid_rest(Vec<P> r, Vec<P> e) {
  return lanes<P>([&](int i) { return r.get(i) <= 0.5f ? 1.f - r.get(i) : e.get(i) * r.get(i); });
}

// V elements as they lie in memory, read as V / P vectors of P.  open(): a gate
// of 128, whose Sigmoid is 1 and whose 1 - Sigmoid is 0.
template <typename T, int V> struct Piece;
template <> struct Piece<__nv_bfloat16, 8> {
  uint4 v;
  static constexpr int kParts = 1;                           // 16-byte parts
  __device__ __forceinline__ void load(const void *p) { v = *static_cast<const uint4 *>(p); }
  __device__ __forceinline__ void part(int, uint4 x) { v = x; }
  __device__ __forceinline__ Vec<2> get(int i) const {
    const unsigned w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
    return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void open() { v = make_uint4(0x43004300, 0x43004300, 0x43004300, 0x43004300); }  // 128
};
template <> struct Piece<float, 8> {
  uint4 a, b;
  static constexpr int kParts = 2;
  __device__ __forceinline__ void load(const void *p) {
    a = static_cast<const uint4 *>(p)[0];
    b = static_cast<const uint4 *>(p)[1];
  }
  __device__ __forceinline__ void part(int k, uint4 x) {
    if (k) b = x;
    else a = x;
  }
  __device__ __forceinline__ Vec<2> get(int i) const {
    const uint4 &q = i < 2 ? a : b;
    return i & 1 ? pair(__uint_as_float(q.z), __uint_as_float(q.w)) : pair(__uint_as_float(q.x), __uint_as_float(q.y));
  }
  __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void open() { a = b = make_uint4(0x43000000, 0x43000000, 0x43000000, 0x43000000); }  // 128
};
template <> struct Piece<__nv_bfloat16, 1> {
  __nv_bfloat16 v;
  __device__ __forceinline__ void load(const void *p) { v = *static_cast<const __nv_bfloat16 *>(p); }
  __device__ __forceinline__ Vec<1> get(int) const { return Vec<1>{__bfloat162float(v)}; }
  __device__ __forceinline__ void zero() { v = __float2bfloat16_rn(0.f); }
  __device__ __forceinline__ void open() { v = __float2bfloat16_rn(128.f); }
};
template <> struct Piece<float, 1> {
  float v;
  __device__ __forceinline__ void load(const void *p) { v = *static_cast<const float *>(p); }
  __device__ __forceinline__ Vec<1> get(int) const { return Vec<1>{v}; }
  __device__ __forceinline__ void zero() { v = 0.f; }
  __device__ __forceinline__ void open() { v = 128.f; }
};

__device__ __forceinline__ void put(float *p, const Vec<1> (&f)[1]) { *p = f[0].v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, const Vec<1> (&f)[1]) { *p = __float2bfloat16_rn(f[0].v); }
__device__ __forceinline__ void put(float *p, const Vec<2> (&f)[4]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(f[0].get(0), f[0].get(1), f[1].get(0), f[1].get(1));
  reinterpret_cast<float4 *>(p)[1] = make_float4(f[2].get(0), f[2].get(1), f[3].get(0), f[3].get(1));
}
__device__ __forceinline__ void put(__nv_bfloat16 *p, const Vec<2> (&f)[4]) {
  __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[i].get(0), f[i].get(1));
  *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<uint4 *>(h);
}
// A weight row's piece; ones when it is absent.
__device__ __forceinline__ void weight(const float *w, int j, Vec<1> (&f)[1]) { f[0].v = w ? __ldg(w + j) : 1.f; }
__device__ __forceinline__ void weight(const float *w, int j, Vec<2> (&f)[4]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = all<2>(1.f);
  } else {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(w + j)), b = __ldg(reinterpret_cast<const float4 *>(w + j) + 1);
    f[0] = pair(a.x, a.y);
    f[1] = pair(a.z, a.w);
    f[2] = pair(b.x, b.y);
    f[3] = pair(b.z, b.w);
  }
}
__device__ __forceinline__ float total(Vec<1> v) { return v.v; }
__device__ __forceinline__ float total(Vec<2> v) { return v.get(0) + v.get(1); }

template <typename T_, typename R_, int V_, int kChunks_, int kThreads_, int kRows_ = 1>
struct Shape {
  using T = T_;                                              // y, gate, normed
  using R = R_;                                              // residual, out
  static constexpr int V = V_, kChunks = kChunks_, kThreads = kThreads_;
  static constexpr int rows() { return kRows_; }              // at once, in the forward
  static constexpr int P = V == 8 ? 2 : 1, kVecs = V / P;    // values of one instruction
  static constexpr int kBlock = kThreads >= 128 ? kThreads : 256, kGroups = kBlock / kThreads;
  static constexpr int max_width() { return V * kChunks * kThreads; }
};

// Sums of kN (at most 8) values over the threads of a row, the same in each of
// them.  `sh`: 16 warps' values of each, not in use by an earlier sum.
// Behind the warps' own sums, one value is read from every warp of the row by
// every thread.  With more of them that would be most of a row's instructions, so
// lane l takes value l % 8 of every fourth warp from l / 8, two steps join these,
// and the lanes 0 .. kN - 1 hand the values out.
template <int kThreads, int kN>
__device__ __forceinline__ void row_sum(float (&v)[kN], float (*sh)[16]) {
#pragma unroll
  for (int k = 0; k < kN; ++k)
#pragma unroll
    for (int off = (kThreads < 32 ? kThreads : 32) / 2; off > 0; off >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
  if constexpr (kThreads > 32) {
    constexpr int kWarps = kThreads / 32;
    const int lane = threadIdx.x & 31, first = threadIdx.x / kThreads * kWarps;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < kN; ++k) sh[k][threadIdx.x >> 5] = v[k];
    __syncthreads();
    if constexpr (kN == 1) {
      v[0] = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) v[0] += sh[0][first + i];
    } else {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; i += 4)
        if (i + lane / 8 < kWarps && lane % 8 < kN) s += sh[lane % 8][first + i + lane / 8];
      s += __shfl_xor_sync(0xffffffffu, s, 8);
      s += __shfl_xor_sync(0xffffffffu, s, 16);
#pragma unroll
      for (int k = 0; k < kN; ++k) v[k] = __shfl_sync(0xffffffffu, s, k);
    }
  }
}

// Forward.  A group takes kRows rows at once where a row is only a piece or two
// per thread, so that weights and addresses are spread over several rows.
template <typename S>
__global__ void __launch_bounds__(S::kBlock, (sizeof(typename S::T) + sizeof(typename S::R) <= 6 ? 1024 : 768) / S::kBlock)
norm_fwd_kernel(NormArgs a) {
  using T = typename S::T;
  using R = typename S::R;
  constexpr int V = S::V, C = S::kChunks, P = S::P, N = S::kVecs, K = S::rows();
  __shared__ float sh[2][K][16];
  const int t = threadIdx.x % S::kThreads;
  const long long row = ((long long)blockIdx.x * S::kGroups + threadIdx.x / S::kThreads) * K;
  const size_t base = (size_t)row * a.width;
  const int rows = (int)max(min((long long)K, a.rows - row), 0LL);  // (a whole warp stays for the shuffles)
  Piece<T, V> y[K][C], g[K][C];
  Piece<R, V> r[K][C];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = (c * S::kThreads + t) * V;
      const bool in = j < a.width && k < rows;
      const size_t at = base + (size_t)k * a.width + j;
      y[k][c].zero();
      g[k][c].zero();
      r[k][c].zero();
      if (in) {
        y[k][c].load(static_cast<const T *>(a.y) + at);
        if (a.gate) g[k][c].load(static_cast<const T *>(a.gate) + at);
        if (a.res) r[k][c].load(static_cast<const R *>(a.res) + at);
      }
    }
  const float inv = 1.f / (float)a.width;
  float r1[K], r2[K];
#pragma unroll
  for (int k = 0; k < K; ++k) r1[k] = 1.f;
  if (a.post) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      Vec<P> s = all<P>(0.f);
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < N; ++i) s = fma(y[k][c].get(i), y[k][c].get(i), s);
      r1[k] = total(s);
    }
    row_sum<S::kThreads, K>(r1, sh[0]);
#pragma unroll
    for (int k = 0; k < K; ++k) r1[k] = rsqrtf(r1[k] * inv + a.e1);
  }
  Vec<P> o[K][C][N], sum[K];
#pragma unroll
  for (int k = 0; k < K; ++k) sum[k] = all<P>(0.f);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int j = (c * S::kThreads + t) * V;
    if (j >= a.width) continue;
    Vec<P> w[N], sc[N];
    weight(a.w1, j, w);
    weight(a.sc, j, sc);
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = mul(w[i], sc[i]);
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        Vec<P> b = mul(mul(y[k][c].get(i), all<P>(r1[k])), w[i]), e;
        if (a.gate) b = mul(b, sigmoid_of(g[k][c].get(i), e));
        o[k][c][i] = add(b, r[k][c].get(i));
        sum[k] = fma(o[k][c][i], o[k][c][i], sum[k]);
      }
      if (k < rows && a.out) put(static_cast<R *>(a.out) + base + (size_t)k * a.width + j, o[k][c]);
    }
  }
  if (!a.normed) return;
#pragma unroll
  for (int k = 0; k < K; ++k) r2[k] = total(sum[k]);
  row_sum<S::kThreads, K>(r2, sh[1]);
#pragma unroll
  for (int k = 0; k < K; ++k) r2[k] = rsqrtf(r2[k] * inv + a.e2);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int j = (c * S::kThreads + t) * V;
    if (j >= a.width) continue;
    Vec<P> w[N], v[N];
    weight(a.w2, j, w);
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (k < rows) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = mul(mul(o[k][c][i], all<P>(r2[k])), w[i]);
        put(static_cast<T *>(a.normed) + base + (size_t)k * a.width + j, v);
      }
  }
}

constexpr int kSms = 152;  // the backward's grid fills these once; each block leaves one set of weight-gradient partials

// Backward.  With tr = scale o b the branch's part of out, everything that the
// row's gradients need of the row as a whole are sums that are known as soon as
// r1 is: sum out^2, and with q = d_normed w2
//     sum q out,  sum d_out tr,  sum q tr,  sum out tr
// since sum dy yh = sum D tr = sum (d_out + r2 q - back out) tr.  So a row takes
// two sums over its threads, not three.  Blocks walk over rows; a thread owns
// fixed channels, so its sums of the weight gradients stay in registers: with
// b = yh w1 s (s the gate) and du yh = D scale s yh, both d_scale = w1 Q and
// d_post_weight = scale Q come from Q = sum over rows of D s yh.  These sums are
// fp32, over a thread's rows (at most a 152nd of all), then groups and blocks: with
// compensation they would take 32 more registers, which wide rows do not have.  Where
// all rows are alike, and so the roundings too, they are off by up to 30 half steps
// (2^-24) at 32768 x 4096, 212 at 262144 x 4096, 394 at 1000000 x 1000.
//
// In pieces of 8 elements the rows come in by asynchronous copies, up to two
// rows ahead as far as shared memory goes, each thread into places of its own that no other thread reads.
template <typename S> struct RowStages {
  using T = typename S::T;
  using R = typename S::R;
  static constexpr int parts() {
    if constexpr (S::V == 8) return 3 * Piece<T, 8>::kParts + 2 * Piece<R, 8>::kParts;
    else return 0;
  }
  static constexpr int kStage = parts() * S::kChunks * S::kBlock * 16;  // bytes
  static constexpr int kLimit = S::kBlock > 256 ? 227 * 1024 : 225 * 1024 / (512 / S::kBlock);
  static constexpr int kStages = 3 * kStage <= kLimit ? 3 : 2 * kStage <= kLimit ? 2 : 1;
  static constexpr int kSums = S::kGroups > 1 ? (int)sizeof(float) * S::kGroups * S::max_width() : 0;
  static constexpr int kBytes = kStages * kStage > kSums ? kStages * kStage : kSums;
  // an SM's: single elements have no copies in flight ahead of them, and need few registers
  static constexpr int kBlocks = (S::V == 1 && S::kChunks <= 4 ? 1024 : 512) / S::kBlock;
};

template <typename S>
__global__ void __launch_bounds__(S::kBlock, RowStages<S>::kBlocks) norm_bwd_kernel(NormArgs a, NormBwdIo io, float *part) {
  using T = typename S::T;
  using R = typename S::R;
  using St = RowStages<S>;
  constexpr int V = S::V, C = S::kChunks, P = S::P, N = S::kVecs;
  extern __shared__ __align__(16) uint4 stage_mem[];
  __shared__ float sh1[2][1][16], sh2[2][5][16];
  const int t = threadIdx.x % S::kThreads, group = threadIdx.x / S::kThreads;
  const float inv = 1.f / (float)a.width;
  Vec<P> p1[C][N], p2[C][N];  // Q, and d_pre_weight
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < N; ++i) p1[c][i] = p2[c][i] = all<P>(0.f);
  const long long step = (long long)gridDim.x * S::kGroups;
  const long long first = (long long)blockIdx.x * S::kGroups + group;

  Piece<T, V> y[C], g[C], dn[C];
  Piece<R, V> res[C], dout[C];
  // absent tensors: no bytes of y
  const void *const src[5] = {a.y, a.gate ? a.gate : a.y, io.dn ? io.dn : a.y, a.res ? a.res : a.y, io.dout ? io.dout : a.y};
  const bool here[5] = {true, a.gate != nullptr, io.dn != nullptr, a.res != nullptr, io.dout != nullptr};
  // `row` into stage `k`, as zeros past the last row and for absent tensors
  auto fetch = [&](long long row, int k) {
    if constexpr (V == 8) {
      unsigned to = (unsigned)__cvta_generic_to_shared(stage_mem + (size_t)k * (St::kStage / 16) + threadIdx.x);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int j = (c * S::kThreads + t) * V;
        const bool in = j < a.width && row < a.rows;
        const size_t at = in ? (size_t)row * a.width + j : 0;
#pragma unroll
        for (int m = 0; m < 5; ++m) {
          constexpr int kT = (int)sizeof(T), kR = (int)sizeof(R);
          const char *from = static_cast<const char *>(src[m]) + (here[m] ? at * (m < 3 ? kT : kR) : 0);
          const int size = in && here[m] ? 16 : 0;
#pragma unroll
          for (int h = 0; h < (m < 3 ? kT : kR) / 2; ++h, to += 16 * S::kBlock)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from + (here[m] ? 16 * h : 0)), "r"(size)
                         : "memory");
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  };
  auto take = [&](long long row, int k) {
    if constexpr (V == 8) {
      asm volatile("cp.async.wait_group %0;" ::"n"(St::kStages - 1) : "memory");
      const uint4 *from = stage_mem + (size_t)k * (St::kStage / 16) + threadIdx.x;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        auto read = [&](auto &piece) {
#pragma unroll
          for (int h = 0; h < std::remove_reference_t<decltype(piece)>::kParts; ++h, from += S::kBlock) piece.part(h, *from);
        };
        read(y[c]);
        read(g[c]);
        read(dn[c]);
        read(res[c]);
        read(dout[c]);
      }
      if (!a.gate)
#pragma unroll
        for (int c = 0; c < C; ++c) g[c].open();
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int j = c * S::kThreads + t;
        const size_t at = (size_t)row * a.width + j;
        const bool in = j < a.width && row < a.rows;
        y[c].zero();
        g[c].open();
        dn[c].zero();
        res[c].zero();
        dout[c].zero();
        if (in) {
          y[c].load(static_cast<const T *>(a.y) + at);
          if (a.gate) g[c].load(static_cast<const T *>(a.gate) + at);
          if (io.dn) dn[c].load(static_cast<const T *>(io.dn) + at);
          if (a.res) res[c].load(static_cast<const R *>(a.res) + at);
          if (io.dout) dout[c].load(static_cast<const R *>(io.dout) + at);
        }
      }
    }
  };
#pragma unroll
  for (int k = 0; k < St::kStages - 1; ++k) fetch(first + k * step, k);
  int par = 0, stage = 0;
  // the groups of a block run the same number of rows
  for (long long r0 = (long long)blockIdx.x * S::kGroups; r0 < a.rows; r0 += step, par ^= 1) {
    const long long row = r0 + group;
    const bool valid = row < a.rows;
    {
      int k = stage + St::kStages - 1;
      fetch(row + (St::kStages - 1) * step, k >= St::kStages ? k - St::kStages : k);
    }
    take(row, stage);
    stage = stage + 1 < St::kStages ? stage + 1 : 0;
    float r1 = 1.f;
    if (a.post) {
      Vec<P> s = all<P>(0.f);
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < N; ++i) s = fma(y[c].get(i), y[c].get(i), s);
      float ss[1] = {total(s)};
      row_sum<S::kThreads, 1>(ss, sh1[par]);
      r1 = rsqrtf(ss[0] * inv + a.e1);
    }
    Vec<P> v[5];
#pragma unroll
    for (int k = 0; k < 5; ++k) v[k] = all<P>(0.f);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = (c * S::kThreads + t) * V;
      if (j >= a.width) continue;
      Vec<P> w1[N], sc[N], w2[N];
      weight(a.w1, j, w1);
      weight(a.sc, j, sc);
      weight(a.w2, j, w2);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        Vec<P> tr = mul(mul(y[c].get(i), all<P>(r1)), mul(w1[i], sc[i])), e;
        tr = mul(tr, sigmoid_of(g[c].get(i), e));
        const Vec<P> o = add(tr, res[c].get(i)), q = mul(dn[c].get(i), w2[i]);
        v[0] = fma(o, o, v[0]);
        v[1] = fma(q, o, v[1]);
        v[2] = fma(dout[c].get(i), tr, v[2]);
        v[3] = fma(q, tr, v[3]);
        v[4] = fma(o, tr, v[4]);
      }
    }
    float sums[5];
#pragma unroll
    for (int k = 0; k < 5; ++k) sums[k] = total(v[k]);
    row_sum<S::kThreads, 5>(sums, sh2[par]);
    // without d_normed nothing depends on out, however large or infinite it is
    const float r2 = io.dn ? rsqrtf(sums[0] * inv + a.e2) : 0.f;
    const float back = io.dn ? r2 * r2 * r2 * sums[1] * inv : 0.f;
    const float m = !a.post ? 0.f : io.dn ? (sums[2] + r2 * sums[3] - back * sums[4]) * inv : sums[2] * inv;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = (c * S::kThreads + t) * V;
      if (j >= a.width || !valid) continue;
      Vec<P> w1[N], sc[N], w2[N], dres[N], dgate[N], dy[N];
      weight(a.w1, j, w1);
      weight(a.sc, j, sc);
      weight(a.w2, j, w2);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const Vec<P> yh = mul(y[c].get(i), all<P>(r1));
        Vec<P> e;
        const Vec<P> sg = sigmoid_of(g[c].get(i), e), rest = sigmoid_rest(sg, e);
        const Vec<P> ys = mul(yh, sg), b = mul(ys, w1[i]);
        const Vec<P> o = io.dn ? fma(b, sc[i], res[c].get(i)) : all<P>(0.f);
        const Vec<P> n = mul(dn[c].get(i), all<P>(r2));
        const Vec<P> D = fma(n, w2[i], fma(o, all<P>(-back), dout[c].get(i)));
        p2[c][i] = fma(n, o, p2[c][i]);
        p1[c][i] = fma(D, ys, p1[c][i]);
        const Vec<P> db = mul(D, sc[i]), du = mul(db, sg);
        dres[i] = D;
        dgate[i] = mul(mul(db, b), rest);
        dy[i] = a.post ? mul(fma(du, w1[i], mul(yh, all<P>(-m))), all<P>(r1)) : du;
      }
      const size_t at = (size_t)row * a.width + j;
      put(static_cast<T *>(io.dy) + at, dy);
      if (io.dgate) put(static_cast<T *>(io.dgate) + at, dgate);
      if (io.dres) put(static_cast<R *>(io.dres) + at, dres);
    }
  }
  if constexpr (V == 8) asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (!part) return;
  // the groups of a block in order, then one row of partials
  float *sums = reinterpret_cast<float *>(stage_mem);  // [kGroups][max_width]
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float *to = part + ((size_t)k * gridDim.x + blockIdx.x) * a.width;
    if constexpr (S::kGroups > 1) __syncthreads();
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = (c * S::kThreads + t) * V;
      const Vec<P>(&p)[N] = k == 0 ? p1[c] : p2[c];
      if constexpr (S::kGroups > 1) put(sums + group * S::max_width() + j, p);
      else if (j < a.width) put(to + j, p);
    }
    if constexpr (S::kGroups > 1) {
      __syncthreads();
      for (int j = threadIdx.x; j < a.width; j += S::kBlock) {
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < S::kGroups; ++q) s += sums[q * S::max_width() + j];
        to[j] = s;
      }
    }
  }
}

// Weight gradients: the blocks' partials summed, 32 columns and 16 strides of
// blocks to a CTA.
__global__ void __launch_bounds__(512) norm_weights_kernel(NormArgs a, const float *part, int blocks, NormBwdIo io) {
  const int lane = threadIdx.x & 31, stride = threadIdx.x >> 5, j = blockIdx.x * 32 + lane, k = blockIdx.y;
  if (k == 0 ? !io.dw1 && !io.dsc : !io.dw2) return;
  __shared__ float sh[16][32];
  float s = 0.f;
  if (j < a.width)
    for (int b = stride; b < blocks; b += 16) s += part[((size_t)k * blocks + b) * a.width + j];
  sh[stride][lane] = s;
  __syncthreads();
  if (stride == 0 && j < a.width) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += sh[i][lane];
    if (k == 1) {
      io.dw2[j] = s;
    } else {
      if (io.dw1) io.dw1[j] = a.sc ? s * a.sc[j] : s;
      if (io.dsc) io.dsc[j] = a.w1 ? s * a.w1[j] : s;
    }
  }
}

template <typename S> cudaError_t fwd(const NormArgs &a, cudaStream_t s) {
  const long long rows = (long long)S::kGroups * S::rows();
  norm_fwd_kernel<S><<<(unsigned)((a.rows + rows - 1) / rows), S::kBlock, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename S> cudaError_t bwd(const NormArgs &a, const NormBwdIo &io, float *ws, cudaStream_t s) {
  const bool weights = io.dw1 || io.dsc || io.dw2;
  const long long groups = (a.rows + S::kGroups - 1) / S::kGroups, most = kSms * RowStages<S>::kBlocks;
  const int blocks = (int)(groups < most ? groups : most);
  constexpr int smem = RowStages<S>::kBytes;  // with the kernel's own sums, below 2 KB, past 48 KB only after leave
  cudaError_t e = cudaSuccess;
  if (smem > 46 * 1024) e = cudaFuncSetAttribute(norm_bwd_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  norm_bwd_kernel<S><<<blocks, S::kBlock, smem, s>>>(a, io, weights ? ws : nullptr);
  e = cudaGetLastError();
  if (e != cudaSuccess || !weights) return e;
  norm_weights_kernel<<<dim3((a.width + 31) / 32, 2), 512, 0, s>>>(a, ws, blocks, io);
  return cudaGetLastError();
}

// Calls f with the row shape for this width: pieces of 8 elements when every
// row of every tensor starts on 16 bytes, else single elements.  Two pieces per
// thread where rows are wide enough (65536 x 2048 forward: 310 us against 350 of
// one; 32768 x 2048 forward and backward in bf16: 359 against 430), in the
// backward from 1025 on (32768 x 1024 in bf16: 131 us against 142 of two).  Wider
// types fill its registers and shared memory with fewer: all-fp32 rows take one
// piece (16384 x 2048: 299 us against 367); rows of one fp32 and one bf16 type take
// one up to 2048 (bf16 y with fp32 residual 204 us against 289, fp32 y with bf16
// residual 240 against 285) and two above, where one would leave a single block on
// an SM (16384 x 4096: 406 against 496, and 564 against 583).
// Narrow rows take as few lanes as hold them, and in the forward two rows at once when
// there are many: in bf16 of two pieces a lane from 65 to 256 (262144 rows of 128: 35.1
// us against 38.3 of one row, 36.9 on 16 lanes of one piece; 4194304 rows of 32: 157 us
// against 440 on 16 lanes), where a tensor is fp32 of one, as two do not fit the
// registers (262144 x 128, bf16 y with fp32 residual: 74 us against 98, 80 of one row;
// fp32 y with bf16 residual 84, 123, 86; all fp32 102, 143, 102).
// Rows of single elements have a step of threads for each doubling of the width, as
// a piece past the row costs as much as one in it: bf16 with every part, 258111 x 130
// on 64 threads 139 us forward and 363 backward, on 256 threads 416 and 1215;
// 31359 x 1070 on 4 pieces of 512 threads 172 and 340, on 16 pieces 321 and 851.
template <typename T, typename R, bool kBwd, typename F>
cudaError_t with_shape(int width, bool vectors, bool many, F f) {
  if (vectors) {
    constexpr int bytes = sizeof(T) + sizeof(R);
    constexpr bool one2048 = kBwd && bytes > 4, one4096 = kBwd && bytes > 6;
    if constexpr (!kBwd) {
      constexpr int c = bytes > 4 ? 1 : 2;
      if (many && width <= 16) return f(Shape<T, R, 8, 1, 2, 2>());
      if (many && width <= 32) return f(Shape<T, R, 8, 1, 4, 2>());
      if (many && width <= 64) return f(Shape<T, R, 8, 1, 8, 2>());
      if (many && width <= 128) return f(Shape<T, R, 8, c, 16 / c, 2>());
      if (many && width <= 256) return f(Shape<T, R, 8, c, 32 / c, 2>());
    } else {
      if (width <= 16) return f(Shape<T, R, 8, 1, 2>());
      if (width <= 32) return f(Shape<T, R, 8, 1, 4>());
      if (width <= 64) return f(Shape<T, R, 8, 1, 8>());
    }
    if (width <= 128) return f(Shape<T, R, 8, 1, 16>());
    if (width <= 256) return f(Shape<T, R, 8, 1, 32>());
    if (width <= 512) return f(Shape<T, R, 8, kBwd ? 1 : 2, kBwd ? 64 : 32>());
    if (width <= 1024) return f(Shape<T, R, 8, kBwd ? 1 : 2, kBwd ? 128 : 64>());
    if (width <= 2048) return f(Shape<T, R, 8, one2048 ? 1 : 2, one2048 ? 256 : 128>());
    if (width <= 4096) return f(Shape<T, R, 8, one4096 ? 1 : 2, one4096 ? 512 : 256>());
    return f(Shape<T, R, 8, 2, 512>());
  }
  if (width <= 32) return f(Shape<T, R, 1, 1, 32>());
  if (width <= 64) return f(Shape<T, R, 1, 2, 32>());
  if (width <= 128) return f(Shape<T, R, 1, 4, 32>());
  if (width <= 256) return f(Shape<T, R, 1, 4, 64>());
  if (width <= 512) return f(Shape<T, R, 1, 4, 128>());
  if (width <= 1024) return f(Shape<T, R, 1, 4, 256>());
  if (width <= 2048) return f(Shape<T, R, 1, 4, 512>());
  if (width <= 4096) return f(Shape<T, R, 1, 8, 512>());
  return f(Shape<T, R, 1, 16, 512>());
}

template <bool kBwd, typename F> cudaError_t with_types(const NormArgs &a, bool vectors, F f) {
  using B = __nv_bfloat16;
  const bool many = a.rows >= 16384;
  if (a.t == KDA_BF16)
    return a.rt == KDA_BF16 ? with_shape<B, B, kBwd>(a.width, vectors, many, f) : with_shape<B, float, kBwd>(a.width, vectors, many, f);
  return a.rt == KDA_BF16 ? with_shape<float, B, kBwd>(a.width, vectors, many, f) : with_shape<float, float, kBwd>(a.width, vectors, many, f);
}

template <int kN> bool on_16_bytes(const NormArgs &a, const void *const (&p)[kN]) {
  uintptr_t bits = 0;
  for (const void *q : p) bits |= reinterpret_cast<uintptr_t>(q);
  return (bits & 15) == 0 && a.width % 8 == 0;
}

}  // namespace

// (an SM holds up to 8 blocks, of 128 threads, where rows have at most 512 elements, and 4 above)
size_t norm_bwd_workspace_bytes(int width) { return (size_t)2 * kSms * (width <= 512 ? 8 : 4) * width * sizeof(float); }

cudaError_t launch_norm_fwd(const NormArgs &a, cudaStream_t s) {
  if (a.rows == 0) return cudaSuccess;
  const void *const p[] = {a.y, a.res, a.gate, a.w1, a.sc, a.w2, a.out, a.normed};
  return with_types<false>(a, on_16_bytes(a, p), [&](auto shape) { return fwd<decltype(shape)>(a, s); });
}

cudaError_t launch_norm_bwd(const NormArgs &args, const NormBwdIo &io, void *ws, cudaStream_t s) {
  NormArgs a = args;
  if (!io.dn) a.w2 = nullptr;  // not read, whatever it holds
  if (a.rows == 0) {
    cudaError_t e = cudaSuccess;
    for (float *w : {io.dw1, io.dsc, io.dw2})
      if (w && e == cudaSuccess) e = cudaMemsetAsync(w, 0, sizeof(float) * a.width, s);
    return e;
  }
  const void *const p[] = {a.y, a.res, a.gate, a.w1, a.sc, a.w2, io.dout, io.dn, io.dy, io.dres, io.dgate};
  return with_types<true>(a, on_16_bytes(a, p),
                          [&](auto shape) { return bwd<decltype(shape)>(a, io, static_cast<float *>(ws), s); });
}

}  // namespace kda
