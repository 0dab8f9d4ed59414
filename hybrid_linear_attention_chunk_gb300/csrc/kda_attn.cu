// Attention over a paged cache: the choice of its kernel and the joining of parts.
#include "kda_attn.cuh"

namespace kda {
namespace {

// A row of an item that several blocks hold parts of:
//     M = max m_p,  l = sum l_p 2^(m_p - M),  out = sum o_p 2^(m_p - M) / l.
// A block has one row; its 8 warps take the parts in turn, so that many parts of
// few rows (one long sequence) are read at once, and are summed in the warps' order.
template <int D, typename T>
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnArgs a, int grid, int R) {
  constexpr int W = 8, V = D >= 32 ? D / 32 : 1, kLanes = D / V;
  __shared__ float2 ml[W];
  __shared__ float sums[W][D];
  const AttnRec rec = reinterpret_cast<const AttnRec *>(a.part)[blockIdx.x];
  if (rec.parts == 0) return;
  const PagedSeq s = paged_seq(a, rec.n);
  const int row = blockIdx.y, at = rec.r * R + row;
  if (at >= s.len * a.G) return;
  const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
  float m = -INFINITY, l = 0.f, o[V] = {};
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
  if (lane == 0) ml[w] = make_float2(m, l);
  if (lane < kLanes)
#pragma unroll
    for (int i = 0; i < V; ++i) sums[w][lane * V + i] = o[i];
  __syncthreads();
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < W; ++i) top = fmaxf(top, ml[i].x);
  const float ref = top == -INFINITY ? 0.f : top;
  float all = 0.f;
#pragma unroll
  for (int i = 0; i < W; ++i) all += ml[i].y * exp2f(ml[i].x - ref);
  const size_t tok = s.bos + at / a.G;
  const int head = rec.h * a.G + at % a.G;
  const bool none = attn_end(a, s, at) == 0;
  for (int c = threadIdx.x; c < D; c += 256) {
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) x += sums[i][c] * exp2f(ml[i].x - ref);
    x = none ? 0.f : x / all;
    T *out = static_cast<T *>(a.o) + tok * a.os + head * D + c;
    if constexpr (sizeof(T) == 2) *out = __float2bfloat16_rn(x);
    else *out = x;
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[tok * a.Hq + head] = none ? -INFINITY : (top + log2f(all)) * 0.6931471805599453f;
}

}  // namespace

cudaError_t launch_attn_join(const AttnArgs &a, int grid, int R, cudaStream_t s) {
  const dim3 g(grid, R);
#define KDA_JOIN(D)                                                                                     \
  if (a.d == D) {                                                                                       \
    if (a.t == KDA_BF16) attn_join_kernel<D, __nv_bfloat16><<<g, 256, 0, s>>>(a, grid, R);              \
    else attn_join_kernel<D, float><<<g, 256, 0, s>>>(a, grid, R);                                      \
  }
  KDA_JOIN(16) KDA_JOIN(32) KDA_JOIN(64) KDA_JOIN(128)
#undef KDA_JOIN
  return cudaGetLastError();
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
