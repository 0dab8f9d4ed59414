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
// heads: the sine costs more than everything else that a row's lane does.  Each group of
// d / 8 lanes then has one token and every so-many-th of its heads, with the pairs' angles
// and the weights in registers.  Each lane copies the pieces that it will need kStages rows ahead into
// shared memory of its own, from before the angles are formed on: HBM latency is all that
// bounds these kernels otherwise.  The angle is
// position * inv_freq in turns modulo one, a 64-bit product of integers: fp32
// would lose 2^-24 of it, all of it at positions of 10^6.
//
// Bound by HBM and, close behind, by instruction issue (71 % of the slots), which is why
// channels are taken two to an fp32 instruction.  32768 tokens x 40 heads of 128 in bf16:
// forward 112 us (0.88 of the copy's rate on its bytes), backward 166 us (0.89) and 8 us for
// the weights' sums; append of 16384 tokens x (32 + 2 x 8) heads 71 us (0.84).  Rings of 16 rows
// instead of 8 leave room for fewer blocks (159 us forward); blocks of 8 tokens instead of
// 16 take the backward from 172 to 190 us.
#include <type_traits>

#include "kda_internal.cuh"
#include "kda_packed.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;   // of a block
constexpr int kSms = 152, kBwdBlocks = kSms * 32;  // of the card; the backward's blocks, which its workspace's size goes by

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

// A lane's 8 channels as its pairs (x, y), two pairs to a register pair: what issues
// packed fp32 instructions.  (Lanes that are not turned have some order of theirs.)
struct Eight {
  Vec<2> x[2], y[2];
};
__device__ __forceinline__ float bf_lo(unsigned w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(unsigned w) { return __uint_as_float(w & 0xffff0000u); }
template <bool kInter> __device__ __forceinline__ Eight unpack(float4 a, float4 b) {
  if (kInter) return Eight{{pair(a.x, a.z), pair(b.x, b.z)}, {pair(a.y, a.w), pair(b.y, b.w)}};
  return Eight{{pair(a.x, a.y), pair(a.z, a.w)}, {pair(b.x, b.y), pair(b.z, b.w)}};
}
template <bool kInter> __device__ __forceinline__ Eight unpack(uint2 a, uint2 b) {
  return unpack<kInter>(make_float4(bf_lo(a.x), bf_hi(a.x), bf_lo(a.y), bf_hi(a.y)),
                        make_float4(bf_lo(b.x), bf_hi(b.x), bf_lo(b.y), bf_hi(b.y)));
}
template <bool kInter> __device__ __forceinline__ void pack(const Eight &v, float4 &a, float4 &b) {
  if (kInter) {
    a = make_float4(v.x[0].get(0), v.y[0].get(0), v.x[0].get(1), v.y[0].get(1));
    b = make_float4(v.x[1].get(0), v.y[1].get(0), v.x[1].get(1), v.y[1].get(1));
  } else {
    a = make_float4(v.x[0].get(0), v.x[0].get(1), v.x[1].get(0), v.x[1].get(1));
    b = make_float4(v.y[0].get(0), v.y[0].get(1), v.y[1].get(0), v.y[1].get(1));
  }
}
__device__ __forceinline__ unsigned bf_pair(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const unsigned *>(&b);
}
template <bool kInter> __device__ __forceinline__ void pack(const Eight &v, uint2 &a, uint2 &b) {
  float4 p, q;
  pack<kInter>(v, p, q);
  a = make_uint2(bf_pair(p.x, p.y), bf_pair(p.z, p.w));
  b = make_uint2(bf_pair(q.x, q.y), bf_pair(q.z, q.w));
}
template <typename T> __device__ __forceinline__ void store_raw(T *row, Piece p, typename Raw<T>::V lo, typename Raw<T>::V hi) {
  *reinterpret_cast<typename Raw<T>::V *>(row + p.c0) = lo;
  *reinterpret_cast<typename Raw<T>::V *>(row + p.c1) = hi;
}
template <typename T, bool kInter> __device__ __forceinline__ void store8(T *row, Piece p, const Eight &v) {
  typename Raw<T>::V lo, hi;
  pack<kInter>(v, lo, hi);
  store_raw(row, p, lo, hi);
}

// Rows on their way: kN tensors' pieces of each of kStages rows, in a place of its own for each lane.
template <typename T, int kN> struct Ring {
  using V = typename Raw<T>::V;
  static constexpr int kStages = (sizeof(T) == 2 ? 8 : 4) / kN;  // a power of two
  static constexpr size_t kBytes = (size_t)kStages * kN * 2 * kThreads * sizeof(V);
  V *mine;  // + threadIdx.x
  __device__ __forceinline__ V *at(int stage, int n, int piece) const { return mine + ((stage * kN + n) * 2 + piece) * kThreads; }
  __device__ __forceinline__ void copy(int stage, int n, const T *row, Piece p, bool there) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const unsigned dst = (unsigned)__cvta_generic_to_shared(at(stage, n, i));
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(row + (i ? p.c1 : p.c0)), "n"(sizeof(V)),
                   "r"(there ? (int)sizeof(V) : 0) : "memory");
    }
  }
  __device__ __forceinline__ void commit() const { asm volatile("cp.async.commit_group;" ::: "memory"); }
  __device__ __forceinline__ void wait() const { asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory"); }
  template <bool kInter> __device__ __forceinline__ Eight get(int stage, int n) const {
    return unpack<kInter>(*at(stage, n, 0), *at(stage, n, 1));
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

// cos and sin of position * inv_freq, times scale.  The nearest quarter of a turn is taken out while the angle is an
// integer: what is left, within an eighth, rounds to fp32 by 2^-27 of a half turn at most, where a whole angle would by 2^-25.
__device__ __forceinline__ float2 angle(unsigned long long turns, int pos, float scale) {
  const unsigned long long f = turns * (unsigned long long)(long long)pos;  // modulo one turn
  const unsigned q = (unsigned)((f + (1ull << 61)) >> 62);                  // quarters, modulo 4
  const int rest = (int)((long long)(f - ((unsigned long long)q << 62)) >> 30);  // of 2^34 a turn, -2^31 to 2^31 - 1
  float s, c;
  sincospif((float)rest * 1.1641532182693481e-10f, &s, &c);  // 2^-33: in half turns, -1/4 to 1/4
  const float x = q & 1u ? -s : c, y = q & 1u ? c : s;
  return q & 2u ? make_float2(-x * scale, -y * scale) : make_float2(x * scale, y * scale);
}

// Angles of nt tokens: rot / 2 cosines of a token, then its sines.  A thread has one pair, of several tokens.
__device__ __forceinline__ void fill_angles(float *cs, const int *pos, int nt, const RopeArgs &a) {
  const int half = a.rot / 2, step = kThreads / half, f = threadIdx.x % half;
  if ((int)threadIdx.x >= step * half) return;
  const unsigned long long turns = turns_of(a.freq[f]);
  for (int tok = threadIdx.x / half; tok < nt; tok += step) {
    const float2 x = angle(turns, pos[tok], a.rot_scale);
    cs[tok * a.rot + f] = x.x;
    cs[tok * a.rot + half + f] = x.y;
  }
}

// The lane's four pairs' cosines and sines.
struct Turn {
  Vec<2> c[2], s[2];
  bool turned;
  // cs: the token's; kBack turns back
  template <bool kBack> __device__ __forceinline__ void load(const float *cs, int rot, int l, bool turned_) {
    turned = turned_;
    float4 p = make_float4(1.f, 1.f, 1.f, 1.f), q = make_float4(0.f, 0.f, 0.f, 0.f);
    if (turned) {
      p = *reinterpret_cast<const float4 *>(cs + 4 * l);
      q = *reinterpret_cast<const float4 *>(cs + rot / 2 + 4 * l);
    }
    c[0] = pair(p.x, p.y);
    c[1] = pair(p.z, p.w);
    s[0] = kBack ? pair(-q.x, -q.y) : pair(q.x, q.y);
    s[1] = kBack ? pair(-q.z, -q.w) : pair(q.z, q.w);
  }
  // (x, y) -> (x cos - y sin, y cos + x sin)
  __device__ __forceinline__ void apply(Eight &v) const {
    if (!turned) return;
    const Vec<2> minus = pair(-1.f, -1.f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const Vec<2> x = v.x[i], y = v.y[i];
      v.x[i] = fma(mul(y, s[i]), minus, mul(x, c[i]));
      v.y[i] = fma(x, s[i], mul(y, c[i]));
    }
  }
};

template <int L> __device__ __forceinline__ float lane_sum(float x) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

// The lane's 8 weights (ones when absent).
template <bool kInter> __device__ __forceinline__ Eight load_weight(const float *w, Piece p) {
  float4 a = make_float4(1.f, 1.f, 1.f, 1.f), b = a;
  if (w) {
    a = make_float4(w[p.c0], w[p.c0 + 1], w[p.c0 + 2], w[p.c0 + 3]);
    b = make_float4(w[p.c1], w[p.c1 + 1], w[p.c1 + 2], w[p.c1 + 3]);
  }
  return unpack<kInter>(a, b);
}

__device__ __forceinline__ float sum_of(const Eight &a, const Eight &b) {  // of products
  const Vec<2> s = fma(a.x[0], b.x[0], mul(a.y[0], b.y[0])), t = fma(a.x[1], b.x[1], mul(a.y[1], b.y[1]));
  const Vec<2> u = add(s, t);
  return u.get(0) + u.get(1);
}
__device__ __forceinline__ Eight times(const Eight &a, const Eight &b) {
  return Eight{{mul(a.x[0], b.x[0]), mul(a.x[1], b.x[1])}, {mul(a.y[0], b.y[0]), mul(a.y[1], b.y[1])}};
}
__device__ __forceinline__ Eight times(const Eight &a, float f) {
  const Vec<2> b = pair(f, f);
  return Eight{{mul(a.x[0], b), mul(a.x[1], b)}, {mul(a.y[0], b), mul(a.y[1], b)}};
}
__device__ __forceinline__ Eight add_times(const Eight &a, const Eight &b, float f) {  // a + b f
  const Vec<2> c = pair(f, f);
  return Eight{{fma(b.x[0], c, a.x[0]), fma(b.x[1], c, a.x[1])}, {fma(b.y[0], c, a.y[0]), fma(b.y[1], c, a.y[1])}};
}
__device__ __forceinline__ Eight add_times(const Eight &a, const Eight &b, const Eight &c) {  // a + b c
  return Eight{{fma(b.x[0], c.x[0], a.x[0]), fma(b.x[1], c.x[1], a.x[1])},
               {fma(b.y[0], c.y[0], a.y[0]), fma(b.y[1], c.y[1], a.y[1])}};
}

// A group's place in its block: one token, and heads h0, h0 + step, ...
struct Place {
  int tok, h0, step;
};
template <int L> __device__ __forceinline__ Place place_of(int per) {  // per: tokens of a block, a power of two
  constexpr int G = kThreads / L;
  const int g = threadIdx.x / L;
  Place p;
  p.step = per < G ? G / per : 1;
  p.tok = g / p.step;
  p.h0 = g % p.step;
  return p;
}

// Rows of up to three tensors of the group's token, one after the other: the queries, the keys
// and, in the append, the values.
template <typename T> struct Tensor {
  const T *x;         // of the token
  T *y;               // nullptr: nothing to do
  long long ystep;    // from head to head in y
  int H;
};
template <typename T, int L, bool kInter, int kTensors> struct Rows {
  Tensor<T> t[kTensors];
  Place at;
  Piece p;
  Ring<T, 1> ring;
  // the next row to copy: its tensor's, head h of H, of x unless there is nothing to do
  const T *x;
  int h, H, tensor = -1, put = 0, got = 0;
  bool open;
  __device__ __forceinline__ void next_tensor() {
    h = at.h0;
    ++tensor;
    if (tensor == 0 && t[0].H == 0) tensor = 1;
    if (tensor == 1 && t[1].H == 0) tensor = 2;
    if (tensor == 0) x = t[0].x, H = t[0].H, open = t[0].y != nullptr;
    if (tensor == 1) x = t[1].x, H = t[1].H, open = t[1].y != nullptr;
    if (kTensors > 2 && tensor == 2) x = t[kTensors - 1].x, H = t[kTensors - 1].H, open = t[kTensors - 1].y != nullptr;
    x += at.h0 * (8 * L);
  }
  __device__ __forceinline__ void issue() {
    if (tensor < kTensors) {
      const bool there = open && h < H;
      ring.copy(put, 0, there ? x : t[0].x, p, there);
      put = (put + 1) % Ring<T, 1>::kStages;
      x += at.step * (8 * L);
      h += at.step;
      if (h - at.h0 >= H) next_tensor();  // (the same for the whole warp)
    }
    ring.commit();
  }
  __device__ __forceinline__ void start() {
    next_tensor();
#pragma unroll 1
    for (int i = 0; i < Ring<T, 1>::kStages; ++i) issue();
  }
  // Rows of tensor i: x -> norm, rotation -> y, or a copy without kTurn (of the bits: a NaN keeps its sign and payload).
  template <int i, bool kTurn> __device__ __forceinline__ void run(const RopeArgs &a, const float *weight, const Turn &turn) {
    Eight w;
    if (kTurn) w = load_weight<kInter>(a.norm ? weight : nullptr, p);
    T *y = t[i].y + at.h0 * t[i].ystep;
    const long long step = at.step * t[i].ystep;
    for (int b = 0; b < t[i].H; b += at.step, y += step) {  // (the same count for the whole warp, for its shuffles)
      ring.wait();
      const bool there = t[i].y && b + at.h0 < t[i].H;
      if constexpr (kTurn) {
        Eight v = ring.template get<kInter>(got, 0);
        got = (got + 1) % Ring<T, 1>::kStages;
        issue();
        if (a.norm) v = times(v, times(w, rsqrtf(lane_sum<L>(sum_of(v, v)) * (1.f / (8 * L)) + a.eps)));
        turn.apply(v);
        if (there) store8<T, kInter>(y, p, v);
      } else {
        const typename Raw<T>::V lo = *ring.at(got, 0, 0), hi = *ring.at(got, 0, 1);
        got = (got + 1) % Ring<T, 1>::kStages;
        issue();
        if (there) store_raw(y, p, lo, hi);
      }
    }
  }
};

template <typename T, int L, bool kInter>
__global__ void __launch_bounds__(kThreads, 4) rope_fwd_kernel(const RopeArgs a, int per) {
  extern __shared__ float4 smem4[];
  float *cs = reinterpret_cast<float *>(smem4 + Ring<T, 1>::kBytes / 16);
  __shared__ int pos[kMaxTokens];
  const int t0 = blockIdx.x * per, nt = min(per, a.tokens - t0), l = threadIdx.x % L;
  Rows<T, L, kInter, 2> rows;
  rows.at = place_of<L>(per);
  rows.p = piece_of<kInter>(l, a.rot);
  rows.ring.mine = reinterpret_cast<typename Raw<T>::V *>(smem4) + threadIdx.x;
  const bool mine = rows.at.tok < nt;
  const long long t = t0 + (mine ? rows.at.tok : 0);
  rows.t[0] = Tensor<T>{static_cast<const T *>(a.q) + t * a.qs, mine ? static_cast<T *>(a.qo) + t * a.qos : nullptr,
                        8 * L, a.Hq};
  rows.t[1] = Tensor<T>{static_cast<const T *>(a.k) + t * a.ks, mine ? static_cast<T *>(a.ko) + t * a.kos : nullptr,
                        8 * L, a.Hk};
  rows.start();
  if (a.rot) {
    if (threadIdx.x < nt) pos[threadIdx.x] = a.positions[t0 + threadIdx.x];
    __syncthreads();
    fill_angles(cs, pos, nt, a);
    __syncthreads();
  }
  Turn turn;
  turn.load<false>(cs + rows.at.tok * a.rot, a.rot, l, mine && rows.p.turned);
  rows.template run<0, true>(a, a.qw, turn);
  rows.template run<1, true>(a, a.kw, turn);
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
__global__ void __launch_bounds__(kThreads, 4) kv_append_kernel(const RopeArgs a, const PagedArgs p, const T *v,
                                                                long long vs, T *kc, T *vc, int per) {
  extern __shared__ float4 smem4[];
  float *cs = reinterpret_cast<float *>(smem4 + Ring<T, 1>::kBytes / 16);
  __shared__ int pos[kMaxTokens];
  __shared__ long long slot[kMaxTokens];
  __shared__ bool in[kMaxTokens];
  const int t0 = blockIdx.x * per, nt = min(per, a.tokens - t0), l = threadIdx.x % L;
  Rows<T, L, kInter, 3> rows;
  rows.at = place_of<L>(per);
  rows.p = piece_of<kInter>(l, a.rot);
  rows.ring.mine = reinterpret_cast<typename Raw<T>::V *>(smem4) + threadIdx.x;
  const bool mine = rows.at.tok < nt;
  const long long t = t0 + (mine ? rows.at.tok : 0), head = (long long)p.page * (8 * L);
  // (rows of tokens that turn out not to be stored are read all the same: they lie within the tensors)
  const T *k = static_cast<const T *>(a.k) + t * a.ks;
  rows.t[0] = Tensor<T>{a.q ? static_cast<const T *>(a.q) + t * a.qs : k,
                        mine ? static_cast<T *>(a.qo) + t * a.qos : nullptr, 8 * L, a.q ? a.Hq : 0};
  rows.t[1] = Tensor<T>{k, mine ? kc : nullptr, head, a.Hk};
  rows.t[2] = Tensor<T>{v + t * vs, mine ? vc : nullptr, head, a.Hk};
  rows.start();
  place_tokens(p, t0, nt, pos, slot, in);
  __syncthreads();
  if (a.rot) {
    fill_angles(cs, pos, nt, a);
    __syncthreads();
  }
  Turn turn;
  turn.load<false>(cs + rows.at.tok * a.rot, a.rot, l, mine && rows.p.turned);
  const bool query = mine && in[rows.at.tok];
  const long long to = mine ? slot[rows.at.tok] : -1;
  if (!query) rows.t[0].y = nullptr;
  rows.t[1].y = to >= 0 ? kc + to : nullptr;
  rows.t[2].y = to >= 0 ? vc + to : nullptr;
  rows.template run<0, true>(a, a.qw, turn);
  rows.template run<1, true>(a, a.kw, turn);
  rows.template run<2, false>(a, nullptr, turn);
}

// ----------------------------------------------------------------- backward

// Sum of dw over the block's rows of lanes, to out[d].
template <int L, bool kInter> __device__ __forceinline__ void block_weight(float *sums, const Eight &dw, Piece p, float *out) {
  constexpr int G = kThreads / L, D = 8 * L;
  float4 a, b;
  pack<kInter>(dw, a, b);
  __syncthreads();  // sums is free
  *reinterpret_cast<float4 *>(sums + threadIdx.x / L * D + p.c0) = a;
  *reinterpret_cast<float4 *>(sums + threadIdx.x / L * D + p.c1) = b;
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += kThreads) {
    float s = 0.f;
    for (int g = 0; g < G; ++g) s += sums[g * D + c];
    out[c] = s;
  }
}

// Blocks have the tokens of one tensor: the first `q_blocks` q's and the others k's (both
// at once would hold twice the weights and sums in registers).  Each leaves one row of weight
// gradients; there are up to kBwdBlocks, which walk over the tokens when these are more.
template <typename T, int L, bool kInter>
__global__ void __launch_bounds__(kThreads, 3) rope_bwd_kernel(const RopeArgs a, const RopeBwdIo io, int per,
                                                               int q_blocks, float *part) {
  using R = Ring<T, 2>;
  extern __shared__ float4 smem4[];  // the ring (and in the end a row of d floats for each d / 8 lanes), angles
  float *cs = reinterpret_cast<float *>(smem4 + R::kBytes / 16);
  __shared__ int pos[kMaxTokens];
  const bool isq = (int)blockIdx.x < q_blocks;
  const int H = isq ? a.Hq : a.Hk, first = isq ? blockIdx.x : blockIdx.x - q_blocks;
  const long long step = (long long)(isq ? q_blocks : gridDim.x - q_blocks) * per;
  const T *x = static_cast<const T *>(isq ? a.q : a.k), *dy = static_cast<const T *>(isq ? io.dqo : io.dko);
  T *dx = static_cast<T *>(isq ? io.dq : io.dk);
  const long long xs = isq ? a.qs : a.ks, dys = isq ? a.qos : a.kos, dxs = isq ? io.dqs : io.dks;
  const Place at = place_of<L>(per);
  const Piece p = piece_of<kInter>(threadIdx.x % L, a.rot);
  R ring;
  ring.mine = reinterpret_cast<typename Raw<T>::V *>(smem4) + threadIdx.x;
  const Eight w = load_weight<kInter>(isq ? a.qw : a.kw, p);
  Eight dw = Eight{{pair(0.f, 0.f), pair(0.f, 0.f)}, {pair(0.f, 0.f), pair(0.f, 0.f)}};
  for (long long t = (long long)first * per; t < a.tokens; t += step) {
    const int t0 = (int)t, nt = min(per, a.tokens - t0);
    const bool mine = at.tok < nt;
    const long long tok = t0 + (mine ? at.tok : 0);
    const T *dyt = dy + tok * dys + (mine ? at.h0 * (8 * L) : 0), *xt = a.norm ? x + tok * xs + (mine ? at.h0 * (8 * L) : 0) : dyt;
    T *dxt = dx + tok * dxs + at.h0 * (8 * L);
    int h = 0, put = 0, got = 0;  // the next heads to copy
    auto issue = [&]() {
      if (h < H) {
        const bool there = mine && h + at.h0 < H;
        const int o = there ? h * (8 * L) : 0;
        ring.copy(put, 0, xt + o, p, there && a.norm);
        ring.copy(put, 1, dyt + o, p, there);
        put = (put + 1) % R::kStages;
        h += at.step;
      }
      ring.commit();
    };
#pragma unroll 1
    for (int i = 0; i < R::kStages; ++i) issue();
    if (a.rot) {
      if (threadIdx.x < nt) pos[threadIdx.x] = a.positions[t0 + threadIdx.x];
      __syncthreads();  // (and the last tokens' angles are read)
      fill_angles(cs, pos, nt, a);
      __syncthreads();
    }
    Turn turn;
    turn.load<true>(cs + at.tok * a.rot, a.rot, threadIdx.x % L, mine && p.turned);
    for (int b = 0; b < H; b += at.step, dxt += at.step * (8 * L)) {
      const bool there = mine && b + at.h0 < H;
      ring.wait();
      const Eight v = ring.template get<kInter>(got, 0);
      Eight gr = ring.template get<kInter>(got, 1);
      got = (got + 1) % R::kStages;
      issue();
      turn.apply(gr);
      if (a.norm) {
        const Eight gw = times(gr, w);
        const float r = rsqrtf(lane_sum<L>(sum_of(v, v)) * (1.f / (8 * L)) + a.eps);
        const float m = lane_sum<L>(sum_of(gw, v)) * (1.f / (8 * L)) * r * r;
        if (there) dw = add_times(dw, gr, times(v, r));
        gr = times(add_times(gw, v, -m), r);
      }
      if (there) store8<T, kInter>(dxt, p, gr);
    }
  }
  if (part) block_weight<L, kInter>(reinterpret_cast<float *>(smem4), dw, p, part + (size_t)blockIdx.x * 8 * L);
}

// Column sums of part[blocks][d], q's rows first: 8 columns a block, 128 threads to each, which
// have up to 39 rows each and join them by halves (fp64 would take ten times as long here).
__global__ void __launch_bounds__(1024) rope_weight_kernel(const float *part, int q_blocks, int blocks, int d,
                                                           float *dqw, float *dkw) {
  __shared__ float s[8][128 + 1];
  const int c0 = blockIdx.x % (d / 8) * 8, c = threadIdx.x % 8, y = threadIdx.x / 8;
  const bool isq = (int)blockIdx.x < d / 8;
  float *to = isq ? dqw : dkw;
  if (!to) return;
  float x = 0.f;
#pragma unroll 8
  for (int b = (isq ? 0 : q_blocks) + y; b < (isq ? q_blocks : blocks); b += 128) x += part[(size_t)b * d + c0 + c];
  s[c][y] = x;
  __syncthreads();
  const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (w >= 8) return;
  float sum = (s[w][lane] + s[w][lane + 32]) + (s[w][lane + 64] + s[w][lane + 96]);  // warp w has column w
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  if (lane == 0) to[c0 + w] = sum;
}

// Tokens of a block: enough blocks for the SMs first, then up to kMaxTokens, over
// whose heads a lane's weights and the block's start are spread.
int tokens_per_block(int tokens) {
  int n = 1;
  while (n < kMaxTokens && tokens / (2 * n) >= kSms * 4) n *= 2;
  return n;
}

// Blocks of the backward, q's and k's by their shares of the rows.
struct BwdBlocks {
  int q, k;
};
BwdBlocks bwd_blocks(int tokens, int Hq, int Hk) {
  const int per = tokens_per_block(tokens);
  const long long need = ((long long)tokens + per - 1) / per;
  const int share = (int)((long long)kBwdBlocks * Hq / (Hq + Hk)), q = share > 1 ? share : 1;
  const int k = Hk ? (kBwdBlocks - q > 1 ? kBwdBlocks - q : 1) : 0;
  return BwdBlocks{(int)(need < q ? need : q), (int)(need < k ? need : k)};
}

// Ring and angles fit the shared memory that a kernel may have without asking.
template <typename T, int kN> constexpr size_t ring_bytes() {
  static_assert(Ring<T, kN>::kBytes + kMaxTokens * kMaxDim * sizeof(float) + 1024 <= 48 * 1024, "within the default limit");
  return Ring<T, kN>::kBytes;
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

size_t rope_bwd_workspace_bytes(int tokens, int Hq, int Hk, int d) {
  const BwdBlocks b = bwd_blocks(tokens, Hq, Hk);
  return (size_t)(b.q + b.k + 1) * d * sizeof(float);
}

cudaError_t launch_rope_fwd(const RopeArgs &a, cudaStream_t s) {
  if (a.tokens == 0) return cudaSuccess;
  const int per = tokens_per_block(a.tokens), grid = (int)(((long long)a.tokens + per - 1) / per);
  return for_shape(a, [&](auto t, auto l, auto inter) {
    using T = decltype(t);
    auto kernel = rope_fwd_kernel<T, decltype(l)::value, decltype(inter)::value>;
    kernel<<<grid, kThreads, ring_bytes<T, 1>() + per * a.rot * sizeof(float), s>>>(a, per);
    return cudaGetLastError();
  });
}

cudaError_t launch_kv_append(const RopeArgs &r, const PagedArgs &p, const void *v, long long vs, void *kc, void *vc,
                             cudaStream_t s) {
  if (r.tokens == 0) return cudaSuccess;
  const int per = tokens_per_block(r.tokens), grid = (int)(((long long)r.tokens + per - 1) / per);
  return for_shape(r, [&](auto t, auto l, auto inter) {
    using T = decltype(t);
    auto kernel = kv_append_kernel<T, decltype(l)::value, decltype(inter)::value>;
    kernel<<<grid, kThreads, ring_bytes<T, 1>() + per * r.rot * sizeof(float), s>>>(
        r, p, static_cast<const T *>(v), vs, static_cast<T *>(kc), static_cast<T *>(vc), per);
    return cudaGetLastError();
  });
}

cudaError_t launch_rope_bwd(const RopeArgs &a, const RopeBwdIo &io, float *ws, cudaStream_t s) {
  const BwdBlocks b = bwd_blocks(a.tokens, a.Hq, a.Hk);
  const int per = tokens_per_block(a.tokens), q_blocks = b.q, k_blocks = b.k;
  const bool weights = io.dqw || io.dkw;
  if (q_blocks) {
    const cudaError_t e = for_shape(a, [&](auto t, auto l, auto inter) {
      using T = decltype(t);
      auto kernel = rope_bwd_kernel<T, decltype(l)::value, decltype(inter)::value>;
      kernel<<<q_blocks + k_blocks, kThreads, ring_bytes<T, 2>() + per * a.rot * sizeof(float), s>>>(a, io, per, q_blocks,
                                                                                        weights ? ws : nullptr);
      return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
  }
  if (weights) {
    rope_weight_kernel<<<a.d / 8 * 2, 1024, 0, s>>>(ws, q_blocks, q_blocks + k_blocks, a.d, io.dqw, io.dkw);
  }
  return cudaGetLastError();
}

}  // namespace kda
