// Norm and position rotation of query and key rows, forward and backward, and
// the append of keys and values to a paged cache with both on the way.
//
// A row of d channels belongs to d / 8 lanes.  Lane l < rot / 8 holds the four
// rotation pairs 4l .. 4l + 3, so that a rotation never leaves its lane: with
// half pairs channels 4l .. and rot / 2 + 4l .., interleaved 8l .. 8l + 7; the
// lanes behind hold eight channels that are not rotated.  The norm's sum is over
// the lanes, by shuffles.
//
// A block takes a few tokens with all their heads.  Its threads first form the
// sine and cosine of each (token, pair) once, into shared memory, for all the
// heads: the sine costs more than everything else that a row's lane does.  The
// angle is position * inv_freq in turns modulo one, a 64-bit product of integers:
// fp32 would lose 2^-24 of it, all of it at positions of 10^6.
#include <type_traits>

#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;   // of a block
constexpr int kBwdBlocks = 152 * 4;

// Row pieces: 4 channels at c0 and 4 at c1.
struct Piece {
  int c0, c1;
  bool turned;
};
template <bool kInter> __device__ __forceinline__ Piece piece_of(int l, int rot) {
  Piece p;
  p.turned = l < rot / 8;
  const bool half = !kInter && p.turned;
  p.c0 = half ? 4 * l : 8 * l;
  p.c1 = half ? rot / 2 + 4 * l : 8 * l + 4;
  return p;
}

template <typename T> struct Raw;  // 4 channels as they lie in memory
template <> struct Raw<float> { using V = float4; };
template <> struct Raw<__nv_bfloat16> { using V = uint2; };

__device__ __forceinline__ void unpack(float4 r, float *v) { v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w; }
__device__ __forceinline__ void unpack(uint2 r, float *v) {
  const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&r.x));
  const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&r.y));
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}
__device__ __forceinline__ void pack(float4 &r, const float *v) { r = make_float4(v[0], v[1], v[2], v[3]); }
__device__ __forceinline__ void pack(uint2 &r, const float *v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  r.x = *reinterpret_cast<const unsigned *>(&a);
  r.y = *reinterpret_cast<const unsigned *>(&b);
}

// A row's 8 channels of this lane.
template <typename T> struct Eight {
  typename Raw<T>::V lo, hi;
  __device__ __forceinline__ void load(const T *row, Piece p) {
    lo = *reinterpret_cast<const typename Raw<T>::V *>(row + p.c0);
    hi = *reinterpret_cast<const typename Raw<T>::V *>(row + p.c1);
  }
  __device__ __forceinline__ void get(float *v) const {
    unpack(lo, v);
    unpack(hi, v + 4);
  }
  __device__ __forceinline__ void store(T *row, Piece p, const float *v) {
    pack(lo, v);
    pack(hi, v + 4);
    *reinterpret_cast<typename Raw<T>::V *>(row + p.c0) = lo;
    *reinterpret_cast<typename Raw<T>::V *>(row + p.c1) = hi;
  }
};

// Turns of one step of the position, in 2^-64 of a turn, to 2 of them: freq has 24
// bits, so its product with the first 29 of 1 / (2 pi) is exact in fp64.
__device__ __forceinline__ unsigned long long turns_of(float freq) {
  constexpr double hi = 85445659.0 / 536870912.0;             // 2^29 / (2 pi), rounded down
  constexpr double lo = 8.3270286903304391962e-10;          // and what it leaves
  double x = (double)freq * hi, y = (double)freq * lo;
  x -= floor(x);
  y -= rint(y);
  return (unsigned long long)(x * 18446744073709551616.0) + (unsigned long long)(long long)(y * 18446744073709551616.0);
}

// cos and sin of position * inv_freq, times scale.
__device__ __forceinline__ float2 angle(unsigned long long turns, int pos, float scale) {
  const unsigned long long f = turns * (unsigned long long)(long long)pos;  // modulo one turn
  float s, c;
  sincospif((float)(int)(f >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31: in half turns, -1 to 1
  return make_float2(c * scale, s * scale);
}

// Angles of nt tokens to cs[token][pair].
__device__ __forceinline__ void fill_angles(float2 *cs, const int *pos, int nt, const RopeArgs &a) {
  const int half = a.rot / 2;
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int tok = i / half, f = i - tok * half;
    cs[i] = angle(turns_of(a.freq[f]), pos[tok], a.rot_scale);
  }
}

// (a, b) -> (a cos - b sin, b cos + a sin) of the lane's pairs; kBack turns back.
template <bool kInter, bool kBack> __device__ __forceinline__ void turn(float *v, const float2 *cs) {
  const float4 p = reinterpret_cast<const float4 *>(cs)[0], q = reinterpret_cast<const float4 *>(cs)[1];
  const float c[4] = {p.x, p.z, q.x, q.z}, s[4] = {p.y, p.w, q.y, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float &x = v[kInter ? 2 * i : i], &y = v[kInter ? 2 * i + 1 : 4 + i];
    const float sn = kBack ? -s[i] : s[i], x0 = x;
    x = x0 * c[i] - y * sn;
    y = y * c[i] + x0 * sn;
  }
}

template <int L> __device__ __forceinline__ float lane_sum(float x) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

// The lane's 8 weights (ones when absent).
__device__ __forceinline__ void load_weight(const float *w, Piece p, float *v) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = w ? w[(i < 4 ? p.c0 : p.c1 - 4) + i] : 1.f;
}

// Where rows of a tensor go: row (token, head) is base + at(token) + head * step.
struct TokenRows {
  long long first, stride, step;
  __device__ __forceinline__ long long at(int tok, int head) const { return first + tok * stride + head * step; }
};
struct SlotRows {          // slots[token] < 0: not stored
  const long long *slots;
  long long step;
  __device__ __forceinline__ long long at(int tok, int head) const {
    return slots[tok] < 0 ? -1 : slots[tok] + head * step;
  }
};

// Rows of nt tokens of one tensor: x -> norm, rotation -> y, or a copy without kTurn.
template <typename T, int L, bool kInter, bool kTurn, class To>
__device__ __forceinline__ void rows_fwd(const RopeArgs &a, const T *x, long long xs, T *y, To to, const float *weight,
                                         int t0, int nt, int H, const float2 *cs) {
  constexpr int G = kThreads / L, U = 2;  // rows at a time of a block, of a lane
  const int l = threadIdx.x % L, g = threadIdx.x / L, total = nt * H, half = a.rot / 2;
  const Piece p = kTurn ? piece_of<kInter>(l, a.rot) : piece_of<true>(l, 0);
  float w[8];
  if (kTurn) load_weight(a.norm ? weight : nullptr, p, w);
  for (int r0 = 0; r0 < total; r0 += G * U) {  // (the whole warp stays, for its shuffles)
    Eight<T> e[U];
    int tok[U], head[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * G + g;
      tok[u] = r < total ? r / H : -1;
      head[u] = r - tok[u] * H;
      if (tok[u] >= 0) e[u].load(x + (t0 + tok[u]) * xs + head[u] * (8 * L), p);
      else e[u].lo = e[u].hi = {};
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v[8];
      if (kTurn) {
        e[u].get(v);
        if (a.norm) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
          const float r = rsqrtf(lane_sum<L>(ss) * (1.f / (8 * L)) + a.eps);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] *= r * w[i];
        }
      }
      if (tok[u] < 0) continue;
      const long long o = to.at(tok[u], head[u]);
      if (o < 0) continue;
      if (kTurn) {
        if (p.turned) turn<kInter, false>(v, cs + tok[u] * half + 4 * l);
        e[u].store(y + o, p, v);
      } else {
        *reinterpret_cast<typename Raw<T>::V *>(y + o + p.c0) = e[u].lo;
        *reinterpret_cast<typename Raw<T>::V *>(y + o + p.c1) = e[u].hi;
      }
    }
  }
}

template <typename T, int L, bool kInter>
__global__ void __launch_bounds__(kThreads) rope_fwd_kernel(const RopeArgs a, int per) {
  extern __shared__ float4 smem4[];
  float2 *cs = reinterpret_cast<float2 *>(smem4);
  __shared__ int pos[kMaxTokens];
  const int t0 = blockIdx.x * per, nt = min(per, a.tokens - t0);
  if (a.rot) {
    if (threadIdx.x < nt) pos[threadIdx.x] = a.positions[t0 + threadIdx.x];
    __syncthreads();
    fill_angles(cs, pos, nt, a);
    __syncthreads();
  }
  rows_fwd<T, L, kInter, true>(a, static_cast<const T *>(a.q), a.qs, static_cast<T *>(a.qo),
                               TokenRows{t0 * a.qos, a.qos, 8 * L}, a.qw, t0, nt, a.Hq, cs);
  if (a.Hk)
    rows_fwd<T, L, kInter, true>(a, static_cast<const T *>(a.k), a.ks, static_cast<T *>(a.ko),
                                 TokenRows{t0 * a.kos, a.kos, 8 * L}, a.kw, t0, nt, a.Hk, cs);
}

// ------------------------------------------------------------------- append

// Position and cache slot of nt <= kMaxTokens tokens from t0; a slot below 0 is none.
// The first token's sequence is the number of entries of cu_seqlens[1 ..] at or
// below it, counted by the block in one round of loads; the others walk on from there.
__device__ __forceinline__ void place_tokens(const PagedArgs &p, int t0, int nt, int *pos, long long *slot, bool *mine) {
  int n0 = 0;
  if (p.cu) {
    for (int i = 1; i <= p.N; i += kThreads) {
      const int j = i + threadIdx.x, c = __syncthreads_count(j <= p.N && p.cu[j] <= t0);
      n0 += c;
      if (c < kThreads) break;
    }
  }
  if (threadIdx.x < nt) {
    const int t = t0 + threadIdx.x;
    int n = p.cu ? n0 : t / p.T_seq;
    if (p.cu)
      while (n < p.N && p.cu[n + 1] <= t) ++n;
    bool in = n < p.N;
    int ps = 0;
    long long at = -1;
    if (in) {
      const PagedSeq s = paged_seq(p, n);
      in = t >= s.bos && t < s.bos + s.len;
      ps = s.kv - (s.bos + s.len - t);
      if (in && ps >= 0) {
        const int id = p.table[(long long)n * p.max_pages + ps / p.page];
        if (id >= 0 && id < p.pages) at = id * p.cs + (long long)(ps % p.page) * p.d;
      }
    }
    pos[threadIdx.x] = ps;
    slot[threadIdx.x] = at;
    mine[threadIdx.x] = in;
  }
}

template <typename T, int L, bool kInter>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const RopeArgs a, const PagedArgs p, const T *v,
                                                             long long vs, T *kc, T *vc, int per) {
  extern __shared__ float4 smem4[];
  float2 *cs = reinterpret_cast<float2 *>(smem4);
  __shared__ int pos[kMaxTokens];
  __shared__ long long slot[kMaxTokens], qrow[kMaxTokens];
  __shared__ bool mine[kMaxTokens];
  const int t0 = blockIdx.x * per, nt = min(per, a.tokens - t0);
  place_tokens(p, t0, nt, pos, slot, mine);
  if (threadIdx.x < nt) qrow[threadIdx.x] = mine[threadIdx.x] ? (t0 + threadIdx.x) * a.qos : -1;
  __syncthreads();
  if (a.rot) {
    fill_angles(cs, pos, nt, a);
    __syncthreads();
  }
  const long long head = (long long)p.page * (8 * L);
  if (a.q)
    rows_fwd<T, L, kInter, true>(a, static_cast<const T *>(a.q), a.qs, static_cast<T *>(a.qo), SlotRows{qrow, 8 * L},
                                 a.qw, t0, nt, a.Hq, cs);
  rows_fwd<T, L, kInter, true>(a, static_cast<const T *>(a.k), a.ks, kc, SlotRows{slot, head}, a.kw, t0, nt, a.Hk, cs);
  rows_fwd<T, L, kInter, false>(a, v, vs, vc, SlotRows{slot, head}, nullptr, t0, nt, a.Hk, cs);
}

// ----------------------------------------------------------------- backward

// Rows of nt tokens of one tensor: dy -> dx, the lane's weight gradients added to dw.
template <typename T, int L, bool kInter>
__device__ __forceinline__ void rows_bwd(const RopeArgs &a, const T *x, long long xs, const T *dy, long long dys, T *dx,
                                         long long dxs, const float *w, int t0, int nt, int H, const float2 *cs,
                                         float *dw) {
  constexpr int G = kThreads / L, U = 2;
  const int l = threadIdx.x % L, g = threadIdx.x / L, total = nt * H, half = a.rot / 2;
  const Piece p = piece_of<kInter>(l, a.rot);
  for (int r0 = 0; r0 < total; r0 += G * U) {
    Eight<T> ex[U], ey[U];
    int tok[U], head[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * G + g;
      tok[u] = r < total ? r / H : -1;
      head[u] = r - tok[u] * H;
      ex[u].lo = ex[u].hi = ey[u].lo = ey[u].hi = {};
      if (tok[u] >= 0) {
        if (a.norm) ex[u].load(x + (t0 + tok[u]) * xs + head[u] * (8 * L), p);
        ey[u].load(dy + (t0 + tok[u]) * dys + head[u] * (8 * L), p);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v[8], gr[8];
      ex[u].get(v);
      ey[u].get(gr);
      if (p.turned && tok[u] >= 0) turn<kInter, true>(gr, cs + tok[u] * half + 4 * l);
      if (a.norm) {
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss = fmaf(v[i], v[i], ss);
          dot = fmaf(gr[i] * w[i], v[i], dot);
        }
        const float r = rsqrtf(lane_sum<L>(ss) * (1.f / (8 * L)) + a.eps);
        const float m = lane_sum<L>(dot) * (1.f / (8 * L)) * r * r;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (tok[u] >= 0) dw[i] = fmaf(gr[i], v[i] * r, dw[i]);
          gr[i] = r * (gr[i] * w[i] - v[i] * m);
        }
      }
      if (tok[u] >= 0) ey[u].store(dx + (t0 + tok[u]) * dxs + head[u] * (8 * L), p, gr);
    }
  }
}

// Sum of dw over the block's rows of lanes, to out[d].
template <int L, bool kInter>
__device__ __forceinline__ void block_weight(float *sums, const float *dw, int rot, float *out) {
  constexpr int G = kThreads / L, D = 8 * L;
  const Piece p = piece_of<kInter>(threadIdx.x % L, rot);
  __syncthreads();  // sums is free
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[threadIdx.x / L * D + (i < 4 ? p.c0 : p.c1 - 4) + i] = dw[i];
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += kThreads) {
    float s = 0.f;
    for (int g = 0; g < G; ++g) s += sums[g * D + c];
    out[c] = s;
  }
}

// Blocks walk over the tokens, so that each leaves one row of weight gradients.
template <typename T, int L, bool kInter>
__global__ void __launch_bounds__(kThreads) rope_bwd_kernel(const RopeArgs a, const RopeBwdIo io, int per, float *part) {
  __shared__ float4 smem4[kThreads * 2];  // kMaxTokens * 64 angles, then a row of d floats for each d / 8 lanes
  float2 *cs = reinterpret_cast<float2 *>(smem4);
  __shared__ int pos[kMaxTokens];
  float wq[8], wk[8], dwq[8] = {}, dwk[8] = {};
  const Piece p = piece_of<kInter>(threadIdx.x % L, a.rot);
  load_weight(a.qw, p, wq);
  load_weight(a.kw, p, wk);
  for (long long t = (long long)blockIdx.x * per; t < a.tokens; t += (long long)gridDim.x * per) {
    const int t0 = (int)t, nt = min(per, a.tokens - t0);
    if (a.rot) {
      if (threadIdx.x < nt) pos[threadIdx.x] = a.positions[t0 + threadIdx.x];
      __syncthreads();  // (and the last tokens' angles are read)
      fill_angles(cs, pos, nt, a);
      __syncthreads();
    }
    rows_bwd<T, L, kInter>(a, static_cast<const T *>(a.q), a.qs, static_cast<const T *>(io.dqo), a.qos,
                           static_cast<T *>(io.dq), io.dqs, wq, t0, nt, a.Hq, cs, dwq);
    if (a.Hk)
      rows_bwd<T, L, kInter>(a, static_cast<const T *>(a.k), a.ks, static_cast<const T *>(io.dko), a.kos,
                             static_cast<T *>(io.dk), io.dks, wk, t0, nt, a.Hk, cs, dwk);
  }
  if (!part) return;
  float *sums = reinterpret_cast<float *>(smem4);
  block_weight<L, kInter>(sums, dwq, a.rot, part + (size_t)blockIdx.x * 16 * L);
  block_weight<L, kInter>(sums, dwk, a.rot, part + (size_t)blockIdx.x * 16 * L + 8 * L);
}

// Column sums of part[blocks][2 d] in fp64: 32 columns a block, 8 threads to each.
__global__ void __launch_bounds__(256) rope_weight_kernel(const float *part, int blocks, int d, float *dqw, float *dkw) {
  __shared__ double s[8][32];
  const int c = blockIdx.x * 32 + threadIdx.x % 32, y = threadIdx.x / 32;
  double x = 0.0;
  for (int b = y; b < blocks; b += 8) x += part[(size_t)b * 2 * d + c];
  s[y][threadIdx.x % 32] = x;
  __syncthreads();
  if (y == 0) {
    for (int i = 1; i < 8; ++i) x += s[i][threadIdx.x];
    float *to = c < d ? dqw : dkw;
    if (to) to[c < d ? c : c - d] = (float)x;
  }
}

// Tokens of a block: enough blocks for the SMs first, then up to kMaxTokens, over
// whose heads a lane's weights and the block's start are spread.
int tokens_per_block(int tokens) {
  const int n = tokens / (152 * 4);
  return n < 1 ? 1 : n > kMaxTokens ? kMaxTokens : n;
}

template <typename F> cudaError_t for_shape(const RopeArgs &a, F f) {
#define KDA_ROPE_CASE(T, L)                                                      \
  if (a.d == 8 * L)                                                              \
    return a.inter ? f(T{}, std::integral_constant<int, L>{}, std::true_type{})  \
                   : f(T{}, std::integral_constant<int, L>{}, std::false_type{})
  if (a.t == KDA_BF16) {
    KDA_ROPE_CASE(__nv_bfloat16, 2);
    KDA_ROPE_CASE(__nv_bfloat16, 4);
    KDA_ROPE_CASE(__nv_bfloat16, 8);
    KDA_ROPE_CASE(__nv_bfloat16, 16);
  } else {
    KDA_ROPE_CASE(float, 2);
    KDA_ROPE_CASE(float, 4);
    KDA_ROPE_CASE(float, 8);
    KDA_ROPE_CASE(float, 16);
  }
#undef KDA_ROPE_CASE
  return cudaErrorInvalidValue;
}

}  // namespace

size_t rope_bwd_workspace_bytes(int d) { return (size_t)kBwdBlocks * 2 * d * sizeof(float); }

cudaError_t launch_rope_fwd(const RopeArgs &a, cudaStream_t s) {
  if (a.tokens == 0) return cudaSuccess;
  const int per = tokens_per_block(a.tokens), grid = (int)(((long long)a.tokens + per - 1) / per);
  return for_shape(a, [&](auto t, auto l, auto inter) {
    rope_fwd_kernel<decltype(t), decltype(l)::value, decltype(inter)::value>
        <<<grid, kThreads, per * a.rot * sizeof(float), s>>>(a, per);
    return cudaGetLastError();
  });
}

cudaError_t launch_kv_append(const RopeArgs &r, const PagedArgs &p, const void *v, long long vs, void *kc, void *vc,
                             cudaStream_t s) {
  if (r.tokens == 0) return cudaSuccess;
  const int per = tokens_per_block(r.tokens), grid = (int)(((long long)r.tokens + per - 1) / per);
  return for_shape(r, [&](auto t, auto l, auto inter) {
    using T = decltype(t);
    kv_append_kernel<T, decltype(l)::value, decltype(inter)::value>
        <<<grid, kThreads, per * r.rot * sizeof(float), s>>>(r, p, static_cast<const T *>(v), vs, static_cast<T *>(kc),
                                                             static_cast<T *>(vc), per);
    return cudaGetLastError();
  });
}

cudaError_t launch_rope_bwd(const RopeArgs &a, const RopeBwdIo &io, float *ws, cudaStream_t s) {
  const int per = tokens_per_block(a.tokens);
  const long long need = ((long long)a.tokens + per - 1) / per;
  const int grid = (int)(need < kBwdBlocks ? need : kBwdBlocks);
  const bool weights = io.dqw || io.dkw;
  if (grid) {
    const cudaError_t e = for_shape(a, [&](auto t, auto l, auto inter) {
      rope_bwd_kernel<decltype(t), decltype(l)::value, decltype(inter)::value>
          <<<grid, kThreads, 0, s>>>(a, io, per, weights ? ws : nullptr);
      return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
  }
  if (weights) rope_weight_kernel<<<a.d / 16, 256, 0, s>>>(ws, grid, a.d, io.dqw, io.dkw);
  return cudaGetLastError();
}

}  // namespace kda
