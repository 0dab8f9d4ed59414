// Attention over a paged cache in bf16 for few query rows to a head of the cache:
// generation, where each key and value is read once for a handful of rows and the
// kernel's one task is to keep HBM busy.
//
// Warps are independent.  An item of 16 or 32 rows has its queries in the registers
// of every warp; a tile of 64 keys is 16 keys for each of 4 warps, which copies them
// (16-byte asynchronous copies, swizzled so that the fragments' loads have no bank
// conflicts) several tiles ahead into shared memory of its own and runs its own
// online softmax: there is no barrier in the loop.  At the end of a part the warps'
// maxima, sums and outputs are joined through shared memory.
//
// For wide heads two blocks of 4 warps with three tiles each keep 96 to 128 KB in flight on an SM.  128 sequences of 8192 on
// average, 32 heads on 8 of 128: 642 to 649 us for the call, 0.97 of the copy's rate; one of 262144, 16 heads on
// 4: 84 us for this kernel, 0.94.  One of 4096 takes 10.6 us, of which 2 find the block's stretch, 2 reach its
// first keys by way of the page table and 1 joins the warps.
#include "kda_attn.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace {

using sm100::smem_u32;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kWarpKeys = 16, kKeys = kWarps * kWarpKeys;
constexpr int kStages = 3;
// Tiles that an item counts for its start and end.  0 and 2 against 1, one token each: 128 ragged sequences of 32 to 11600,
// 32 heads on 8 of 128, 223 and 195 against 210 us, 16 heads on 4 of 32 53 and 40 against 44; 256 of 200 57 and 56 against 56.
constexpr int kStart = 1;
// Blocks of an SM: as many as shared memory holds for wide heads; narrow ones, whose tiles are small, are bound by the
// warps' own instructions and take twice as many (64 sequences of 8000, 16 heads on 4 of 32: 61 us against 80, of 16 52
// against 73; one sequence of 100000 26 against 24).
constexpr int blocks_of(int d) { return d >= 64 ? 2 : 4; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&x);
}

template <int D> struct Tile {
  static constexpr int kChunks = D / 8;                       // 16-byte pieces of a row
  static constexpr uint32_t kBytes = kWarpKeys * D * 2;       // 16 keys (or values)
  // Rows of 8 matrices' worth of keys fall into distinct banks: the piece is permuted
  // by the row, or by the 128-byte line where a line holds several rows.
  static __device__ __forceinline__ uint32_t at(int row, int chunk) {
    constexpr int per = D >= 64 ? 1 : 64 / D;
    return row * (D * 2) + ((chunk ^ ((row / per) & (kChunks < 8 ? kChunks - 1 : 7))) * 16);
  }
};

template <int D, int MT> struct MmaSmem {
  static constexpr uint32_t kStage = 2 * Tile<D>::kBytes;
  static constexpr uint32_t kJoin = kWarps * MT * 16 * (D + 2) * 4;
  static constexpr uint32_t kRing = kWarps * kStages * kStage;
  static constexpr uint32_t kBytes = kRing > kJoin ? kRing : kJoin;
};

template <int D, int MT>
__global__ void __launch_bounds__(kThreads, blocks_of(D)) attn_mma_kernel(const AttnArgs a) {
  constexpr int R = 16 * MT, kChunks = Tile<D>::kChunks, kCopies = kWarpKeys * kChunks / 32;
  constexpr uint32_t kStage = MmaSmem<D, MT>::kStage;
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, tq = lane % 4, grid = gridDim.x;
  const uint32_t ring = smem_u32(smem) + warp * kStages * kStage;
  const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q), *kc = static_cast<const __nv_bfloat16 *>(a.kc),
                      *vc = static_cast<const __nv_bfloat16 *>(a.vc);
  attn_let_join();
  AttnWalk walk = attn_walk<R, kKeys, kStart, kThreads>(a, blockIdx.x, grid);
  AttnRec rec{0, 0, 0, 0};
  AttnPart p;
  while (attn_next<R, kKeys, kStart>(a, walk, p)) {
    if (p.parts) rec = AttnRec{p.n, p.h, p.r, p.parts};
    const int rows = p.s.len * a.G, row0 = p.r * R, tiles = p.t1 - p.t0;
    const int most = attn_end(a, p.s, min(row0 + R, rows) - 1), all = attn_end(a, p.s, row0);
    const int32_t *table = a.table + (long long)p.n * a.max_pages;

    // Copies of the warp's 16 keys of tile i: lane k finds key k's page a tile ahead.
    auto page_of = [&](int i) {
      const int j = (p.t0 + i) * kKeys + warp * kWarpKeys + (lane & 15);
      return i < tiles && j < most ? table[j / a.page] : 0;
    };
    int page = page_of(0);
    auto issue = [&](int i) {
      if (i < tiles) {
        const int key0 = (p.t0 + i) * kKeys + warp * kWarpKeys, j = key0 + (lane & 15);
        const long long off = key_offset(a, page, j % a.page, p.h);
        const uint32_t dst = ring + i % kStages * kStage;
#pragma unroll
        for (int c = 0; c < kCopies; ++c) {
          const int x = c * 32 + lane, row = x / kChunks, ch = x % kChunks;
          const bool there = key0 + row < most;
          const long long at = __shfl_sync(~0u, off, row) + ch * 8, o = there ? at : 0;
          cp_async16(dst + Tile<D>::at(row, ch), kc + o, there);
          cp_async16(dst + Tile<D>::kBytes + Tile<D>::at(row, ch), vc + o, there);
        }
        page = page_of(i + 1);
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i);

    uint32_t qf[MT][D / 16][4];
    int lim[MT][2];  // keys that rows g and g + 8 of each 16 may see
    float m[MT][2], l[MT][2], o[MT][D / 8][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int at = row0 + t * 16 + x * 8 + g;
        const bool there = at < rows;
        const __nv_bfloat16 *src = q + (there ? (p.s.bos + a.by_G(at)) * a.qs + (p.h * a.G + at - a.by_G(at) * a.G) * D : 0) + tq * 2;
        lim[t][x] = there ? attn_end(a, p.s, at) : 0;
        m[t][x] = -INFINITY;
        l[t][x] = 0.f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          qf[t][k][x] = there ? *reinterpret_cast<const uint32_t *>(src + k * 16) : 0u;
          qf[t][k][2 + x] = there ? *reinterpret_cast<const uint32_t *>(src + k * 16 + 8) : 0u;
        }
      }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int c = 0; c < D / 8; ++c) o[t][c][0] = o[t][c][1] = o[t][c][2] = o[t][c][3] = 0.f;

    for (int i = 0; i < tiles; ++i) {
      const int key0 = (p.t0 + i) * kKeys + warp * kWarpKeys;
      issue(i + kStages - 1);
      cp_wait<kStages - 1>();
      __syncwarp();
      const uint32_t ks = ring + i % kStages * kStage, vs = ks + Tile<D>::kBytes;
      if (key0 < most) {
        float s[MT][2][4] = {};
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t b[4];
          ldsm4(ks + Tile<D>::at((lane / 16) * 8 + lane % 8, k * 2 + (lane / 8) % 2), b);
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            mma16816(s[t][0], qf[t][k], b[0], b[1]);
            mma16816(s[t][1], qf[t][k], b[2], b[3]);
          }
        }
        const bool masked = key0 + kWarpKeys > all;
        uint32_t pf[MT][4];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float e[4] = {s[t][0][2 * x], s[t][0][2 * x + 1], s[t][1][2 * x], s[t][1][2 * x + 1]};
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              e[j] *= a.scale2;
              if (masked && key0 + (j / 2) * 8 + tq * 2 + (j & 1) >= lim[t][x]) e[j] = -INFINITY;
              top = fmaxf(top, e[j]);
            }
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
            if (__any_sync(~0u, top > m[t][x])) {
              top = fmaxf(top, m[t][x]);
              const float f = fast_exp2(m[t][x] - (top == -INFINITY ? 0.f : top));
              m[t][x] = top;
              l[t][x] *= f;
#pragma unroll
              for (int c = 0; c < D / 8; ++c) {
                o[t][c][2 * x] *= f;
                o[t][c][2 * x + 1] *= f;
              }
            }
            const float ref = m[t][x] == -INFINITY ? 0.f : m[t][x];
#pragma unroll
            for (int j = 0; j < 4; ++j) e[j] = fast_exp2(e[j] - ref);
            // (rounded to the values' type, as the product's operands are; the sum is of the unrounded ones)
            l[t][x] += (e[0] + e[1]) + (e[2] + e[3]);
            pf[t][x] = bf2(e[0], e[1]);
            pf[t][2 + x] = bf2(e[2], e[3]);
          }
        if (masked) {
          // A value that is not finite must reach the rows that see its key and no
          // others, but 0 times it is not 0: it goes to those rows by addition, and a
          // 0 takes its place for the product.  Seldom; the test is one pass of 16-byte reads.
          bool odd = false;
#pragma unroll
          for (int c = 0; c < kCopies; ++c) {
            const int x = c * 32 + lane, row = x / kChunks, ch = x % kChunks;
            uint4 w;
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                         : "r"(vs + Tile<D>::at(row, ch)) : "memory");
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              odd |= (u[j] & 0x7f80u) == 0x7f80u || (u[j] & 0x7f800000u) == 0x7f800000u;
          }
          if (__any_sync(~0u, odd)) {
            for (int k = 0; k < kWarpKeys; ++k)
#pragma unroll
              for (int c = 0; c < D / 8; ++c) {
                uint32_t w;  // channels c * 8 + tq * 2 and + 1 of key k
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(vs + Tile<D>::at(k, c) + tq * 4) : "memory");
                const uint32_t h[2] = {w & 0xffffu, w >> 16};
#pragma unroll
                for (int y = 0; y < 2; ++y)
                  if ((h[y] & 0x7f80u) == 0x7f80u) {
                    const float v = __uint_as_float(h[y] << 16);
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                      for (int x = 0; x < 2; ++x)
                        if (key0 + k < lim[t][x]) o[t][c][2 * x + y] += v;
                  }
              }
            __syncwarp();
#pragma unroll
            for (int c = 0; c < kCopies * 4; ++c) {
              const int x = c * 32 + lane, row = x / (D / 2), w2 = x % (D / 2);
              const uint32_t at = vs + Tile<D>::at(row, w2 / 4) + (w2 % 4) * 4;
              uint32_t w;
              asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(at) : "memory");
              if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
              if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
              asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(w) : "memory");
            }
            __syncwarp();
          }
        }
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          uint32_t b[4];
          ldsm4t(vs + Tile<D>::at(((lane / 8) % 2) * 8 + lane % 8, c * 2 + lane / 16), b);
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            mma16816(o[t][2 * c], pf[t], b[0], b[1]);
            mma16816(o[t][2 * c + 1], pf[t], b[2], b[3]);
          }
        }
      }
      __syncwarp();  // the stage may be refilled
    }
    cp_wait<0>();
    __syncthreads();  // every warp is done with its ring

    // Join of the warps: outputs [warp][row][D], then (m, l) [warp][row].
    float *jo = reinterpret_cast<float *>(smem);
    float2 *jm = reinterpret_cast<float2 *>(jo + kWarps * R * D);
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float sum = l[t][x];
        sum += __shfl_xor_sync(~0u, sum, 1);
        sum += __shfl_xor_sync(~0u, sum, 2);
        const int r = t * 16 + x * 8 + g;
        if (tq == 0) jm[warp * R + r] = make_float2(m[t][x], sum);
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
          *reinterpret_cast<float2 *>(jo + (warp * R + r) * D + c * 8 + tq * 2) =
              make_float2(o[t][c][2 * x], o[t][c][2 * x + 1]);
      }
    __syncthreads();
    for (int i = tid; i < R * (D / 4); i += kThreads) {
      const int r = i / (D / 4), c = i % (D / 4) * 4, at = row0 + r;
      if (at >= rows) break;
      float2 w[kWarps];
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        w[x] = jm[x * R + r];
        top = fmaxf(top, w[x].x);
      }
      const bool none = attn_end(a, p.s, at) == 0;
      const float ref = top == -INFINITY ? 0.f : top;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        const float f = fast_exp2(w[x].x - ref);
        const float4 v = *reinterpret_cast<const float4 *>(jo + (x * R + r) * D + c);
        sum += w[x].y * f;
        y.x += v.x * f;
        y.y += v.y * f;
        y.z += v.z * f;
        y.w += v.w * f;
      }
      if (!p.whole) {
        *reinterpret_cast<float4 *>(attn_part_out(a, grid, blockIdx.x, p.slot, R, r) + c) = y;
        if (c == 0) *attn_part_ml(a, grid, blockIdx.x, p.slot, R, r) = make_float2(top, sum);
        continue;
      }
      const float inv = 1.f / sum;
      const size_t tok = p.s.bos + a.by_G(at);
      const int head = p.h * a.G + at - a.by_G(at) * a.G;
      *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) + tok * a.os + head * D + c) =
          none ? make_uint2(0u, 0u) : make_uint2(bf2(y.x * inv, y.y * inv), bf2(y.z * inv, y.w * inv));
      if (a.lse && c == 0) a.lse[tok * a.Hq + head] = none ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    }
    __syncthreads();  // the ring is free again
  }
  if (tid == 0) reinterpret_cast<AttnRec *>(a.part)[blockIdx.x] = rec;
}

int grid_of(int d) { return kSms * blocks_of(d); }

// Up to 16 rows of a (sequence, head) on average, one product of 16 rows, else two.
bool one_tile(const AttnArgs &a) { return (long long)a.T_total * a.G <= 16LL * a.N; }

template <int D, int MT> cudaError_t launch_mma(const AttnArgs &a, cudaStream_t s) {
  constexpr uint32_t bytes = MmaSmem<D, MT>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(attn_mma_kernel<D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) return e;
  attn_mma_kernel<D, MT><<<grid_of(D), kThreads, bytes, s>>>(a);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_attn_join(a, grid_of(D), 16 * MT, s) : e;
}

}  // namespace

size_t attn_mma_floats(const AttnArgs &a) { return attn_part_floats(grid_of(a.d), one_tile(a) ? 16 : 32, a.d); }

cudaError_t launch_attn_mma(const AttnArgs &a, cudaStream_t s) {
  const bool one = one_tile(a);
  switch (a.d) {
    case 16: return one ? launch_mma<16, 1>(a, s) : launch_mma<16, 2>(a, s);
    case 32: return one ? launch_mma<32, 1>(a, s) : launch_mma<32, 2>(a, s);
    case 64: return one ? launch_mma<64, 1>(a, s) : launch_mma<64, 2>(a, s);
    default: return one ? launch_mma<128, 1>(a, s) : launch_mma<128, 2>(a, s);
  }
}

}  // namespace kda
