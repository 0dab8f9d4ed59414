// Attention over a paged cache: the choice of its kernel and the joining of parts.
#include "kda_attn.cuh"

namespace kda {
namespace {

// A row of an item that several blocks hold parts of:
//     M = max m_p,  l = sum l_p 2^(m_p - M),  out = sum o_p 2^(m_p - M) / l.
// Both kernels below are launched as the first one's blocks end (their launch passes meanwhile) and
// wait for all of it before they read anything.
struct Joined {
  float m = -INFINITY, l = 0.f;
  // Takes in a part; what has been summed counts `f` and the part `g`.
  __device__ __forceinline__ void add(float2 x, float &f, float &g) {
    const float top = fmaxf(m, x.x), ref = top == -INFINITY ? 0.f : top;
    f = exp2f(m - ref);
    g = exp2f(x.x - ref);
    l = l * f + x.y * g;
    m = top;
  }
  __device__ __forceinline__ float log_sum() const { return (m + log2f(l)) * 0.6931471805599453f; }
};

template <typename T, int V> __device__ __forceinline__ void store_row(T *to, const float (&o)[V], float l, bool none) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float x = none ? 0.f : o[i] / l;
    if constexpr (sizeof(T) == 2) to[i] = __float2bfloat16_rn(x);
    else to[i] = x;
  }
}

// Items of many rows: a warp has four rows at once, a lane D / 32 channels of each, and goes over the parts one after the
// other.  These are two or three where a call has more items than blocks (8192 tokens, 32 heads on 8 of 128: 15 us), and up
// to one for each block where it has few: 32 rows of one head over 262144 keys are 152 parts, 80 of the call's 121 us.
template <int D, typename T> __global__ void __launch_bounds__(256) attn_join_rows_kernel(const AttnArgs a, int grid, int R) {
  constexpr int V = D >= 32 ? D / 32 : 1, kLanes = D / V, kN = 4;
  attn_wait_for_first();
  const AttnRec rec = reinterpret_cast<const AttnRec *>(a.part)[blockIdx.x];
  if (rec.parts == 0) return;
  const PagedSeq s = paged_seq(a, rec.n);
  const int lane = threadIdx.x % 32, row0 = (blockIdx.y * 8 + threadIdx.x / 32) * kN;
  const int rows = min(R, s.len * a.G - rec.r * R);
  if (row0 >= rows) return;
  Joined j[kN];
  float o[kN][V] = {};
  for (int p = 0; p < rec.parts; ++p) {
    const int block = blockIdx.x + p, slot = p == 0;
    float2 x[kN];
    float v[kN][V];
#pragma unroll
    for (int r = 0; r < kN; ++r) {  // (rows behind the last are not written, but lie in the workspace)
      x[r] = *attn_part_ml(a, grid, block, slot, R, row0 + r);
      const float *src = attn_part_out(a, grid, block, slot, R, row0 + r) + lane * V;
#pragma unroll
      for (int i = 0; i < V; ++i) v[r][i] = lane < kLanes ? src[i] : 0.f;
    }
#pragma unroll
    for (int r = 0; r < kN; ++r) {
      float f, g;
      j[r].add(x[r], f, g);
#pragma unroll
      for (int i = 0; i < V; ++i) o[r][i] = o[r][i] * f + v[r][i] * g;
    }
  }
#pragma unroll
  for (int r = 0; r < kN; ++r) {
    if (row0 + r >= rows) break;
    const int at = rec.r * R + row0 + r, rg = a.by_G(at), head = rec.h * a.G + at - rg * a.G;
    const size_t tok = s.bos + rg;
    const bool none = attn_end(a, s, at) == 0;
    if (lane < kLanes) store_row(static_cast<T *>(a.o) + tok * a.os + head * D + lane * V, o[r], j[r].l, none);
    if (a.lse && lane == 0) a.lse[tok * a.Hq + head] = none ? -INFINITY : j[r].log_sum();
  }
}

// Items of few rows may have a part in every block (one long sequence): a block has one row at a time, its 8 warps
// take the parts in turn, and the row is the sum of theirs in the warps' order.
template <int D, typename T> __global__ void __launch_bounds__(256) attn_join_parts_kernel(const AttnArgs a, int grid, int R) {
  constexpr int W = 8, V = D >= 32 ? D / 32 : 1, kLanes = D / V;
  __shared__ float2 ml[W];
  __shared__ float sums[W][D];
  attn_wait_for_first();
  const AttnRec rec = reinterpret_cast<const AttnRec *>(a.part)[blockIdx.x];
  if (rec.parts == 0) return;
  const PagedSeq s = paged_seq(a, rec.n);
  const int w = threadIdx.x / 32, lane = threadIdx.x % 32, rows = min(R, s.len * a.G - rec.r * R);
  for (int row = blockIdx.y; row < rows; row += gridDim.y) {
    Joined j;
    float o[V] = {};
#pragma unroll 4
    for (int p = w; p < rec.parts; p += W) {
      const int block = blockIdx.x + p, slot = p == 0;
      const float2 x = *attn_part_ml(a, grid, block, slot, R, row);
      const float *src = attn_part_out(a, grid, block, slot, R, row) + lane * V;
      float f, g;
      j.add(x, f, g);
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = o[i] * f + (lane < kLanes ? src[i] : 0.f) * g;
    }
    __syncthreads();  // the row before is read
    if (lane == 0) ml[w] = make_float2(j.m, j.l);
    if (lane < kLanes)
#pragma unroll
      for (int i = 0; i < V; ++i) sums[w][lane * V + i] = o[i];
    __syncthreads();
    if (threadIdx.x >= kLanes) continue;
    Joined all;
    float x[V] = {};
#pragma unroll
    for (int i = 0; i < W; ++i) all.m = fmaxf(all.m, ml[i].x);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float f = exp2f(ml[i].x - (all.m == -INFINITY ? 0.f : all.m));
      all.l += ml[i].y * f;
#pragma unroll
      for (int c = 0; c < V; ++c) x[c] += sums[i][lane * V + c] * f;
    }
    const int at = rec.r * R + row, rg = a.by_G(at), head = rec.h * a.G + at - rg * a.G;
    const size_t tok = s.bos + rg;
    const bool none = attn_end(a, s, at) == 0;
    store_row(static_cast<T *>(a.o) + tok * a.os + head * D + lane * V, x, all.l, none);
    if (a.lse && lane == 0) a.lse[tok * a.Hq + head] = none ? -INFINITY : all.log_sum();
  }
}

}  // namespace

cudaError_t launch_attn_join(const AttnArgs &a, int grid, int R, cudaStream_t s) {
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.blockDim = dim3(256);
  c.gridDim = dim3(grid, R > 32 ? R / 32 : 4);
  c.stream = s;
  c.attrs = &early;
  c.numAttrs = 1;
#define KDA_JOIN(D, T)                                                                 \
  return R > 32 ? cudaLaunchKernelEx(&c, attn_join_rows_kernel<D, T>, a, grid, R)      \
                : cudaLaunchKernelEx(&c, attn_join_parts_kernel<D, T>, a, grid, R)
#define KDA_JOINS(T)                    \
  switch (a.d) {                        \
    case 16: KDA_JOIN(16, T);           \
    case 32: KDA_JOIN(32, T);           \
    case 64: KDA_JOIN(64, T);           \
    default: KDA_JOIN(128, T);          \
  }
  if (a.t == KDA_BF16) KDA_JOINS(__nv_bfloat16)
  KDA_JOINS(float)
#undef KDA_JOINS
#undef KDA_JOIN
}

// The tensor cores' tiles of 128 rows against products of 16 or 32: by the rows of a
// (sequence, head) on average, us with tiles / with products of few:
//     heads of 128   128 x 4 rows over 4000   336 / 325     64 x 20 rows over 2000   110 / 118     64 x 64 rows   115 / 220
//     heads of 64    128 x 4 rows over 4000   275 / 177     128 x 32 rows over 4000  278 / 242     64 x 64 rows    98 / 144
// A packed batch of one long chunk among single tokens goes by the same, since only the device knows its lengths: 256
// tokens and a chunk of 2048 over 1000 319 / 615 (36 rows on average), 2047 tokens and that chunk 1834 / 1481 (8 rows).
// Over short contexts, where the chunk outweighs the single tokens, the average misses it: 2000 tokens (4 rows each) over
// 16, 256 and 1000 beside a chunk of 4096 from an empty cache (12 rows on average) take 838 / 1620, 1230 / 1615 and 1791 /
// 2158 with heads of 128, 792 / 1256, 1207 / 1158 and 1688 / 1587 with heads of 64.
static bool many_rows(const AttnArgs &a) {
  return (long long)a.T_total * a.G > (a.d == 128 ? 16LL : 32LL) * a.N && attn_tc_supports(a);
}

// fp32: few rows of a (sequence, head) on average run in items of 4 or 8 by warps of their own, more in items of 64 by
// whole blocks: the first reads a key once for 8 rows, from HBM or L2, the second wastes what an item lacks.  64
// sequences over 4000, us with few / with 64 rows:
//     heads of 128   12 rows 193 / 481   24 rows 281 / 481   32 rows 366 / 483   48 rows 532 / 483
//     heads of 64    12 rows 142 / 247   24 rows 222 / 262   32 rows 270 / 247
//     heads of 32    12 rows 111 / 156   20 rows 157 / 155   32 rows 204 / 154
//     heads of 16    12 rows 104 / 113   20 rows 145 / 115
// and 256 single tokens beside a chunk of 512 over 1000 (12 rows) 225 / 589, 167 / 292, 128 / 184, 119 / 134.
// A third form, items of 16 rows by whole blocks, was faster for narrow heads of 9 to 16 rows (12 rows: heads of 32 96 us,
// of 16 65) and slower for wide ones (354 against 193), and is not kept.
static bool few_rows(const AttnArgs &a) {
  return (long long)a.T_total * a.G <= (a.d == 128 ? 32LL : a.d == 64 ? 24LL : 16LL) * a.N;
}

size_t attn_workspace_bytes(const AttnArgs &a) {
  const size_t floats = a.t == KDA_F32 ? (few_rows(a) ? attn_f32_few_floats(a) : attn_f32_floats(a))
                                       : (many_rows(a) ? attn_tc_floats(a) : attn_mma_floats(a));
  return floats * sizeof(float);
}

cudaError_t launch_attn(const AttnArgs &a, cudaStream_t s) {
  if (a.T_total == 0) return cudaSuccess;
  if (a.t == KDA_F32) return few_rows(a) ? launch_attn_f32_few(a, s) : launch_attn_f32(a, s);
  return many_rows(a) ? launch_attn_tc(a, s) : launch_attn_mma(a, s);
}

}  // namespace kda
