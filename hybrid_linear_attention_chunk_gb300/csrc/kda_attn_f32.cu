// Attention over a paged cache in fp32, on CUDA cores.  Tensor cores have no fp32 product, and a single tf32 one would
// show in the 24 bits of the result; operands split in two tf32 parts each, three products to one, would keep them (as
// the delta rule's backward does), at a rate that is above that of the CUDA cores.  This kernel does not do that.
//
// An item of 64 rows runs over the keys in tiles of 64, by 256 threads as
// 16 x 16.  Scores: a thread has 4 rows and 4 keys, both from shared memory as
// float4.  Outputs: the same rows and d / 16 channels, probabilities through shared memory.
// The next tile's keys and values are copied meanwhile (16-byte asynchronous copies into a second buffer).
//
// 2048 tokens over 8192, 8 heads on 2 of 128: 2030 us (38 TFLOP/s, 0.51 of the CUDA cores' rate); 1203 tokens of 5
// ragged sequences over 700 on average, 6 heads on 3 of 32, 45 us with the join.  Bound by latencies, with 8 warps on
// an SM for heads of 128: shared memory's pipe is 60 % busy (a load of 16 bytes takes 2 to 4 of its cycles whatever
// its lanes share) and 38 % of the issue slots are taken.  8 rows and 4 keys a thread load a third less: 0 to 12 %
// faster on long runs with three blocks of 128 threads, 17 % slower on the short ragged one.  One barrier a tile, a
// page looked up once a key and warp: 3 % against three and a division for each copy.  Probabilities are read four
// keys at a time, products are of two channels to an instruction.  Few rows leave most of an item's threads without
// work and run elsewhere (kda_attn_f32_few.cu).
#include "kda_attn.cuh"

namespace kda {
namespace {

constexpr int kRows = 64, kKeys = 64, kThreads = 256;
// Tiles that an item counts for its start and end.  0 and 2 against 1: 5 ragged sequences, 6 heads on 3 of 32, 44 and 46
// against 41 us; 4 x 1024 tokens, 8 heads on 2 of 128, 291 and 287 against 276; 20 x 100 over 300, of 64, 66 and 73 against
// 73.
constexpr int kStart = 1;
// Blocks of an SM, as many as shared memory holds.
constexpr int f32_blocks(int d) { return d == 128 ? 1 : 2; }

template <int D> struct F32Smem {
  static constexpr int kRow = D + 4, kProw = kKeys + 4;  // padded: rows of a quarter warp in distinct banks
  static constexpr size_t kBytes = ((size_t)(kRows + 4 * kKeys) * kRow + (size_t)kRows * kProw) * 4;
};

// acc += p v of the tile.  With kMask keys that the row may not see are left out,
// whatever their values are (0 times a non-finite value is not 0).
template <int D, int RT, int V, bool kMask>
__device__ __forceinline__ void add_values(float (&o)[RT][V], const float *P, const float *Vs, int tx, const int *lim,
                                           int key0) {
  constexpr int kRow = D + 4, kProw = kKeys + 4;
#pragma unroll 2
  for (int k0 = 0; k0 < kKeys; k0 += 4) {
    float4 p4[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) p4[i] = *reinterpret_cast<const float4 *>(P + i * kProw + k0);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int k = k0 + x;
      float v[V];
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = Vs[k * kRow + (V >= 4 ? tx * 4 + (j / 4) * 64 + j % 4 : tx * V + j)];
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const float p = x == 0 ? p4[i].x : x == 1 ? p4[i].y : x == 2 ? p4[i].z : p4[i].w;
        if (kMask && key0 + k >= lim[i]) continue;
        if constexpr (V >= 2) {
#pragma unroll
          for (int j = 0; j < V; j += 2) {
            const Vec<2> y = fma(pair(p, p), pair(v[j], v[j + 1]), pair(o[i][j], o[i][j + 1]));
            o[i][j] = y.get(0);
            o[i][j + 1] = y.get(1);
          }
        } else {
          o[i][0] = fmaf(p, v[0], o[i][0]);
        }
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, f32_blocks(D)) attn_f32_kernel(const AttnArgs a) {
  constexpr int kRow = F32Smem<D>::kRow, kProw = F32Smem<D>::kProw, RT = kRows / 16, V = D / 16;
  extern __shared__ float4 smem4[];
  float *Qs = reinterpret_cast<float *>(smem4), *KV = Qs + kRows * kRow, *Ps = KV + 4 * kKeys * kRow;
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16, grid = gridDim.x;
  attn_let_join();
  AttnWalk walk = attn_walk<kRows, kKeys, kStart, kThreads>(a, blockIdx.x, grid);
  AttnRec rec{0, 0, 0, 0};
  AttnPart p;
  while (attn_next<kRows, kKeys, kStart>(a, walk, p)) {
    if (p.parts) rec = AttnRec{p.n, p.h, p.r, p.parts};
    const float *q = static_cast<const float *>(a.q), *kc = static_cast<const float *>(a.kc),
                *vc = static_cast<const float *>(a.vc);
    const int rows = p.s.len * a.G, row0 = p.r * kRows;
    __syncthreads();  // the part before is done with shared memory
    for (int i = tid; i < kRows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), c = i % (D / 4) * 4, at = row0 + r;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (at < rows)
        x = *reinterpret_cast<const float4 *>(q + (p.s.bos + a.by_G(at)) * a.qs + (p.h * a.G + at - a.by_G(at) * a.G) * D + c);
      *reinterpret_cast<float4 *>(Qs + r * kRow + c) = x;
    }
    int lim[RT];  // keys that each of the thread's rows may see
    float m[RT], l[RT], o[RT][V];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int at = row0 + ty * RT + i;
      lim[i] = at < rows ? attn_end(a, p.s, at) : 0;
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) o[i][j] = 0.f;
    }
    const int all = attn_end(a, p.s, row0);            // keys that every row sees
    const int most = attn_end(a, p.s, min(row0 + kRows, rows) - 1);
    const int32_t *table = a.table + (long long)p.n * a.max_pages;
    auto copy_tile = [&](int t) {  // keys, then values, of tile t to buffer t % 2
      float *to = KV + (t & 1) * 2 * kKeys * kRow;
      long long at[2];  // where the tile's first 32 keys and its last 32 lie, a lane each
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int j = t * kKeys + i * 32 + tid % 32;
        at[i] = j < most ? key_offset(a, table[j / a.page], j % a.page, p.h) : 0;
      }
#pragma unroll
      for (int i = 0; i < kKeys * (D / 4) / kThreads; ++i) {
        const int x = i * kThreads + tid, k = x / (D / 4), c = x % (D / 4) * 4, j = t * kKeys + k;
        const bool there = j < most;
        const long long off = __shfl_sync(~0u, k & 32 ? at[1] : at[0], k & 31) + c;  // (a warp's keys are in one half)
        const unsigned dst = (unsigned)__cvta_generic_to_shared(to + k * kRow + c);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(kc + off), "r"(there ? 16 : 0) : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + kKeys * kRow * 4), "l"(vc + off),
                     "r"(there ? 16 : 0) : "memory");
      }
    };
    copy_tile(p.t0);
    for (int t = p.t0; t < p.t1; ++t) {
      const int key0 = t * kKeys;
      const float *Ks = KV + (t & 1) * 2 * kKeys * kRow, *Vs = Ks + kKeys * kRow;
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncthreads();  // tile t (and Qs) is there, and the other buffer is free
      if (t + 1 < p.t1) copy_tile(t + 1);
      // even channels' products and odd ones' side by side: two to an instruction, as they lie
      Vec<2> s2[RT][4];
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s2[i][j] = pair(0.f, 0.f);
#pragma unroll 2
      for (int c = 0; c < D; c += 4) {
        float4 x[RT], y[4];
#pragma unroll
        for (int i = 0; i < RT; ++i) x[i] = *reinterpret_cast<const float4 *>(Qs + (ty * RT + i) * kRow + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4 *>(Ks + (tx + 16 * j) * kRow + c);
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            s2[i][j] = fma(pair(x[i].z, x[i].w), pair(y[j].z, y[j].w), fma(pair(x[i].x, x[i].y), pair(y[j].x, y[j].y), s2[i][j]));
      }
      float s[RT][4];
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = s2[i][j].get(0) + s2[i][j].get(1);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        float top = m[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = key0 + tx + 16 * j < lim[i] ? s[i][j] * a.scale2 : -INFINITY;
          top = fmaxf(top, s[i][j]);
        }
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, x));
        const float ref = top == -INFINITY ? 0.f : top, f = exp2f(m[i] - ref);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = exp2f(s[i][j] - ref);
          Ps[(ty * RT + i) * kProw + tx + 16 * j] = e;
          sum += e;
        }
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(~0u, sum, x);
        l[i] = l[i] * f + sum;
        m[i] = top;
#pragma unroll
        for (int j = 0; j < V; ++j) o[i][j] *= f;
      }
      __syncwarp();  // (a half-warp writes and reads its own rows of Ps)
      if (key0 + kKeys <= all) add_values<D, RT, V, false>(o, Ps + ty * RT * kProw, Vs, tx, lim, key0);
      else add_values<D, RT, V, true>(o, Ps + ty * RT * kProw, Vs, tx, lim, key0);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int r = ty * RT + i, at = row0 + r;
      if (at >= rows) continue;
      const size_t tok = p.s.bos + a.by_G(at);
      const int head = p.h * a.G + at - a.by_G(at) * a.G;
      const bool none = lim[i] == 0;
      float *out = p.whole ? static_cast<float *>(a.o) + tok * a.os + head * D
                           : attn_part_out(a, grid, blockIdx.x, p.slot, kRows, r);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = V >= 4 ? tx * 4 + (j / 4) * 64 + j % 4 : tx * V + j;
        out[c] = p.whole ? (none ? 0.f : o[i][j] / l[i]) : o[i][j];
      }
      if (tx != 0) continue;
      if (!p.whole) *attn_part_ml(a, grid, blockIdx.x, p.slot, kRows, r) = make_float2(m[i], l[i]);
      else if (a.lse) a.lse[tok * a.Hq + head] = none ? -INFINITY : (m[i] + log2f(l[i])) * 0.6931471805599453f;
    }
  }
  if (tid == 0) reinterpret_cast<AttnRec *>(a.part)[blockIdx.x] = rec;
}

template <int D> int f32_grid() { return kSms * f32_blocks(D); }

template <int D> cudaError_t launch_f32(const AttnArgs &a, cudaStream_t s) {
  const size_t bytes = F32Smem<D>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(attn_f32_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) return e;
  attn_f32_kernel<D><<<f32_grid<D>(), kThreads, bytes, s>>>(a);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_attn_join(a, f32_grid<D>(), kRows, s) : e;
}

}  // namespace

size_t attn_f32_floats(const AttnArgs &a) { return attn_part_floats(2 * kSms, kRows, a.d); }

cudaError_t launch_attn_f32(const AttnArgs &a, cudaStream_t s) {
  switch (a.d) {
    case 16: return launch_f32<16>(a, s);
    case 32: return launch_f32<32>(a, s);
    case 64: return launch_f32<64>(a, s);
    default: return launch_f32<128>(a, s);
  }
}

}  // namespace kda
