// Attention over a paged cache: the choice of its kernel and the joining of parts.
#include "kda_attn.cuh"

namespace kda {
namespace {

// A row of an item that several blocks hold parts of:
//     M = max m_p,  l = sum l_p 2^(m_p - M),  out = sum o_p 2^(m_p - M) / l.
// A block's 8 warps have 8 / W rows at a time: W of them take a row's parts in turn, and the
// row is the sum of theirs in the warps' order.  Items of few rows may have a part in every block
// (one long sequence), which W = 8 reads at once; those of many rows have two or three.
// The kernel is launched as the first one's blocks end (its launch passes meanwhile) and waits for
// all of it before it reads anything.
template <int D, typename T, int W>
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnArgs a, int grid, int R) {
  constexpr int V = D >= 32 ? D / 32 : 1, kLanes = D / V, kRows = 8 / W;
  __shared__ float2 mls[kRows][W];
  __shared__ float sum[kRows][W][D];
  attn_wait_for_first();
  const AttnRec rec = reinterpret_cast<const AttnRec *>(a.part)[blockIdx.x];
  if (rec.parts == 0) return;
  const PagedSeq s = paged_seq(a, rec.n);
  const int w = threadIdx.x / 32 % W, lane = threadIdx.x % 32, mine = threadIdx.x / 32 / W;
  const int rows = min(R, s.len * a.G - rec.r * R);
  for (int row0 = blockIdx.y * kRows; row0 < rows; row0 += gridDim.y * kRows) {
    const int row = row0 + mine, at = rec.r * R + row;
    float m = -INFINITY, l = 0.f, o[V] = {};
    if (row < rows) {
#pragma unroll 4
      for (int p = w; p < rec.parts; p += W) {
        const int block = blockIdx.x + p, slot = p == 0;
        const float2 x = *attn_part_ml(a, grid, block, slot, R, row);
        const float *src = attn_part_out(a, grid, block, slot, R, row) + lane * V;
        float v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = lane < kLanes ? src[i] : 0.f;
        const float top = fmaxf(m, x.x), ref = top == -INFINITY ? 0.f : top;
        const float f = exp2f(m - ref), g = exp2f(x.x - ref);
        l = l * f + x.y * g;
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = o[i] * f + v[i] * g;
        m = top;
      }
    }
    __syncthreads();  // the rows before are read
    if (lane == 0) mls[mine][w] = make_float2(m, l);
    if (lane < kLanes)
#pragma unroll
      for (int i = 0; i < V; ++i) sum[mine][w][lane * V + i] = o[i];
    __syncthreads();
    if (row >= rows) continue;
    const float2 *ml = mls[mine];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < W; ++i) top = fmaxf(top, ml[i].x);
    const float ref = top == -INFINITY ? 0.f : top;
    float all = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) all += ml[i].y * exp2f(ml[i].x - ref);
    const int rg = a.by_G(at), head = rec.h * a.G + at - rg * a.G;
    const size_t tok = s.bos + rg;
    const bool none = attn_end(a, s, at) == 0;
    for (int c = threadIdx.x % (32 * W); c < D; c += 32 * W) {
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) x += sum[mine][i][c] * exp2f(ml[i].x - ref);
      x = none ? 0.f : x / all;
      T *out = static_cast<T *>(a.o) + tok * a.os + head * D + c;
      if constexpr (sizeof(T) == 2) *out = __float2bfloat16_rn(x);
      else *out = x;
    }
    if (a.lse && threadIdx.x % (32 * W) == 0)
      a.lse[tok * a.Hq + head] = none ? -INFINITY : (top + log2f(all)) * 0.6931471805599453f;
  }
}

}  // namespace

cudaError_t launch_attn_join(const AttnArgs &a, int grid, int R, cudaStream_t s) {
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.blockDim = dim3(256);
  c.gridDim = dim3(grid, R > 32 ? R / 8 : 4);
  c.stream = s;
  c.attrs = &early;
  c.numAttrs = 1;
#define KDA_JOIN(D, T)                                                                  \
  return R > 32 ? cudaLaunchKernelEx(&c, attn_join_kernel<D, T, 1>, a, grid, R)         \
                : cudaLaunchKernelEx(&c, attn_join_kernel<D, T, 8>, a, grid, R)
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

// The tensor cores' tiles of 128 rows against products of 16 or 32 rows: by the
// rows of a (sequence, head) on average.
static bool many_rows(const AttnArgs &a) { return (long long)a.T_total * a.G > 32LL * a.N && attn_tc_supports(a); }

size_t attn_workspace_bytes(const AttnArgs &a) {
  return (a.t == KDA_F32 ? attn_f32_floats(a) : many_rows(a) ? attn_tc_floats(a) : attn_mma_floats(a)) * sizeof(float);
}

cudaError_t launch_attn(const AttnArgs &a, cudaStream_t s) {
  if (a.T_total == 0) return cudaSuccess;
  return a.t == KDA_F32 ? launch_attn_f32(a, s) : many_rows(a) ? launch_attn_tc(a, s) : launch_attn_mma(a, s);
}

}  // namespace kda
