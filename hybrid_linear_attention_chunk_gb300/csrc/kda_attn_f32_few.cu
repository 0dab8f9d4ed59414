// Attention over a paged cache in fp32 for a few query rows to a head of the cache:
// generation, where the kernel's task is to keep HBM busy, as in bf16 (kda_attn_mma.cu),
// but without tensor products.
//
// Warps are independent.  An item has 4 or 8 rows; a tile of 32 keys is 8 keys for each of 4
// warps, copied tiles ahead into shared memory of its own.  Scores: a half-warp has 4 of the 8
// keys and a lane d / 16 channels of all rows' queries in registers, so that a key is read once for all rows;
// the 4 x rows partial sums are added over the 16 lanes by halves, each step handing on half of them, which
// leaves every (key, row) with one lane after 15 or 30 shuffles instead of 64 or 128.  Outputs: a
// lane has d / 32 channels of all rows, probabilities through shared memory.
//
// Bound by HBM for wide heads: one token of 64 sequences of 8000, 16 heads on 4 of 128, 328 us (6.40 TB/s, 0.94 of the
// copy), of 64 186 us (5.63 TB/s); of 32 by instruction issue, 131 us (4.0 TB/s).
#include "kda_attn.cuh"

namespace kda {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kWarpKeys = 8, kKeys = kWarps * kWarpKeys;
constexpr int kStages = 3;
// Tiles that an item counts for its start and end.  1 and 3 against 2, one token each, 16 heads on 4 of 128: 64 ragged
// sequences 114-117 and 114 against 115 us, 64 of 200 17.6 and 16.6 against 17.1.
constexpr int kStart = 2;
// Blocks of an SM: as many as shared memory holds for wide heads; narrow ones, whose tiles are small, are bound by the
// warps' own instructions and take twice as many (64 sequences of 8000, 16 heads on 4 of 32: 131 us against 163, of 16
// 122 against 151; one sequence of 100000 loses, 29 against 25, to a join of more parts).
constexpr int blocks_of(int d) { return d >= 64 ? 2 : 4; }
int grid_of(int d) { return kSms * blocks_of(d); }

template <int D, int NR> struct FewSmem {
  static constexpr int kStage = 2 * kWarpKeys * D;                 // floats: keys, then values
  static constexpr int kRing = kWarps * kStages * kStage, kJoin = kWarps * NR * (D + 2);
  static constexpr int kP = kWarps * kWarpKeys * NR;
  static constexpr size_t kBytes = (size_t)((kRing > kJoin ? kRing : kJoin) + kP) * 4;
};

// N floats as they lie.
template <int N> __device__ __forceinline__ void load_row(const float *p, float *v) {
  if constexpr (N >= 4) {
    const float4 x = *reinterpret_cast<const float4 *>(p);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  } else if constexpr (N == 2) {
    const float2 x = *reinterpret_cast<const float2 *>(p);
    v[0] = x.x; v[1] = x.y;
  } else {
    v[0] = *p;
  }
}

template <int D, int NR>
__global__ void __launch_bounds__(kThreads, blocks_of(D)) attn_f32_few_kernel(const AttnArgs a) {
  using Smem = FewSmem<D, NR>;
  constexpr int CH = D / 16, CV = CH < 4 ? CH : 4;           // channels of a lane's scores, in vectors of CV
  constexpr int VC = D >= 32 ? D / 32 : 1, kLanes = D / VC;  // channels of a lane's outputs
  constexpr int NS = NR / 4, NV = 4 * NR;                    // scores that a lane ends up with; partial sums
  extern __shared__ float4 smem4[];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, half = lane / 16, l16 = lane % 16, grid = gridDim.x;
  float *ring = reinterpret_cast<float *>(smem4) + warp * kStages * Smem::kStage;
  float *P = reinterpret_cast<float *>(smem4) + (Smem::kRing > Smem::kJoin ? Smem::kRing : Smem::kJoin) + warp * kWarpKeys * NR;
  const float *q = static_cast<const float *>(a.q), *kc = static_cast<const float *>(a.kc), *vc = static_cast<const float *>(a.vc);
  const int mine = half * 4 + l16 / 4, r0 = l16 % 4 * NS;    // the key and first row of the lane's scores
  attn_let_join();
  AttnWalk walk = attn_walk<NR, kKeys, kStart, kThreads>(a, blockIdx.x, grid);
  AttnRec rec{0, 0, 0, 0};
  AttnPart p;
  while (attn_next<NR, kKeys, kStart>(a, walk, p)) {
    if (p.parts) rec = AttnRec{p.n, p.h, p.r, p.parts};
    const int rows = p.s.len * a.G, row0 = p.r * NR, tiles = p.t1 - p.t0;
    const int most = attn_end(a, p.s, min(row0 + NR, rows) - 1), all = attn_end(a, p.s, row0);
    const int32_t *table = a.table + (long long)p.n * a.max_pages;
    // copies of the warp's 8 keys of tile i; lane k finds key k's page a tile ahead
    auto page_of = [&](int i) {
      const int j = (p.t0 + i) * kKeys + warp * kWarpKeys + (lane & 7);
      return i < tiles && j < most ? table[j / a.page] : 0;
    };
    int page = page_of(0);
    auto issue = [&](int i) {
      if (i < tiles) {
        const int key0 = (p.t0 + i) * kKeys + warp * kWarpKeys, j = key0 + (lane & 7);
        const long long off = key_offset(a, page, j % a.page, p.h);
        float *to = ring + i % kStages * Smem::kStage;
#pragma unroll
        for (int c = 0; c < kWarpKeys * D / 4 / 32; ++c) {
          const int x = c * 32 + lane, row = x / (D / 4), ch = x % (D / 4) * 4;
          const bool there = key0 + row < most;
          const long long at = __shfl_sync(~0u, off, row) + ch, o = there ? at : 0;
          const unsigned dst = (unsigned)__cvta_generic_to_shared(to + row * D + ch);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(kc + o), "r"(there ? 16 : 0) : "memory");
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + kWarpKeys * D * 4), "l"(vc + o),
                       "r"(there ? 16 : 0) : "memory");
        }
        page = page_of(i + 1);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i);

    float qr[NR][CH], o[NR][VC], m[NS], l[NS];
    int lim[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int at = row0 + r, rg = a.by_G(min(at, rows - 1));
      const float *src = q + (p.s.bos + rg) * a.qs + (p.h * a.G + min(at, rows - 1) - rg * a.G) * D;
      lim[r] = at < rows ? attn_end(a, p.s, at) : 0;
#pragma unroll
      for (int c = 0; c < CH; c += CV) load_row<CV>(src + l16 * CV + c / CV * 16 * CV, qr[r] + c);
#pragma unroll
      for (int c = 0; c < VC; ++c) o[r][c] = 0.f;
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) m[s] = -INFINITY, l[s] = 0.f;

    for (int i = 0; i < tiles; ++i) {
      const int key0 = (p.t0 + i) * kKeys + warp * kWarpKeys;
      issue(i + kStages - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      __syncwarp();
      const float *ks = ring + i % kStages * Smem::kStage, *vs = ks + kWarpKeys * D;
      if (key0 < most) {
        const bool masked = key0 + kWarpKeys > all;
        float s[NV];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float x[CH];
#pragma unroll
          for (int c = 0; c < CH; c += CV) load_row<CV>(ks + (half * 4 + k) * D + l16 * CV + c / CV * 16 * CV, x + c);
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            if constexpr (CH >= 2) {
              Vec<2> y = mul(pair(qr[r][0], qr[r][1]), pair(x[0], x[1]));
#pragma unroll
              for (int c = 2; c < CH; c += 2) y = fma(pair(qr[r][c], qr[r][c + 1]), pair(x[c], x[c + 1]), y);
              s[k * NR + r] = y.get(0) + y.get(1);
            } else {
              s[k * NR + r] = qr[r][0] * x[0];
            }
          }
        }
        // sums over the half-warp by halves: what a lane hands on is the half that its partner keeps
#pragma unroll
        for (int step = 8, n = NV; step > 0; step >>= 1) {
          const bool upper = l16 & step;
          if (n > NS) {
            n >>= 1;
#pragma unroll
            for (int x = 0; x < NV / 2; ++x)
              if (x < n) {
                const float keep = upper ? s[x + n] : s[x], give = upper ? s[x] : s[x + n];
                s[x] = keep + __shfl_xor_sync(~0u, give, step);
              }
          }
        }
        bool moved = false;
        float top[NS];
#pragma unroll
        for (int x = 0; x < NS; ++x) {
          int see = most;  // (what lies behind `most` is zero in shared memory, not a key)
          if (masked) {
            see = lim[0];
#pragma unroll
            for (int r = 1; r < NR; ++r)
              if (r0 + x == r) see = lim[r];
          }
          s[x] = key0 + mine < see ? s[x] * a.scale2 : -INFINITY;
          top[x] = s[x];
#pragma unroll
          for (int y = 4; y < 32; y <<= 1) top[x] = fmaxf(top[x], __shfl_xor_sync(~0u, top[x], y));
          moved |= top[x] > m[x];
        }
        if (__any_sync(~0u, moved)) {
          float f[NS];
#pragma unroll
          for (int x = 0; x < NS; ++x) {
            top[x] = fmaxf(top[x], m[x]);
            f[x] = exp2f(m[x] - (top[x] == -INFINITY ? 0.f : top[x]));
            m[x] = top[x];
            l[x] *= f[x];
          }
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const float by = __shfl_sync(~0u, f[r % NS], r / NS);
#pragma unroll
            for (int c = 0; c < VC; ++c) o[r][c] *= by;
          }
        }
#pragma unroll
        for (int x = 0; x < NS; ++x) {
          const float e = exp2f(s[x] - (m[x] == -INFINITY ? 0.f : m[x]));
          l[x] += e;
          P[mine * NR + r0 + x] = e;
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kWarpKeys; ++k) {
          float v[VC], pr[NR];
          if (lane < kLanes) load_row<VC>(vs + k * D + lane * VC, v);
          else v[0] = 0.f;
#pragma unroll
          for (int r = 0; r < NR; r += 4) load_row<4>(P + k * NR + r, pr + r);
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            if (masked && key0 + k >= lim[r]) continue;  // (0 times a value that is not finite is not 0)
            if constexpr (VC >= 2) {
#pragma unroll
              for (int c = 0; c < VC; c += 2) {
                const Vec<2> y = fma(pair(pr[r], pr[r]), pair(v[c], v[c + 1]), pair(o[r][c], o[r][c + 1]));
                o[r][c] = y.get(0);
                o[r][c + 1] = y.get(1);
              }
            } else {
              o[r][0] = fmaf(pr[r], v[0], o[r][0]);
            }
          }
        }
      }
      __syncwarp();  // the stage and P may be written again
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // every warp is done with its ring

    // Join of the warps: outputs [warp][row][D], then (m, l) [warp][row].
    float *jo = reinterpret_cast<float *>(smem4);
    float2 *jm = reinterpret_cast<float2 *>(jo + kWarps * NR * D);
#pragma unroll
    for (int x = 0; x < NS; ++x) {
      float sum = l[x];
#pragma unroll
      for (int y = 4; y < 32; y <<= 1) sum += __shfl_xor_sync(~0u, sum, y);
      if (lane < 4) jm[warp * NR + r0 + x] = make_float2(m[x], sum);
    }
    if (lane < kLanes)
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int c = 0; c < VC; ++c) jo[(warp * NR + r) * D + lane * VC + c] = o[r][c];
    __syncthreads();
    for (int i = tid; i < NR * D; i += kThreads) {
      const int r = i / D, c = i % D, at = row0 + r;
      if (at >= rows) break;
      float top = -INFINITY, sum = 0.f, y = 0.f;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) top = fmaxf(top, jm[x * NR + r].x);
      const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        const float f = exp2f(jm[x * NR + r].x - ref);
        sum += jm[x * NR + r].y * f;
        y += jo[(x * NR + r) * D + c] * f;
      }
      if (!p.whole) {
        attn_part_out(a, grid, blockIdx.x, p.slot, NR, r)[c] = y;
        if (c == 0) *attn_part_ml(a, grid, blockIdx.x, p.slot, NR, r) = make_float2(top, sum);
        continue;
      }
      const bool none = attn_end(a, p.s, at) == 0;
      const int rg = a.by_G(at), head = p.h * a.G + at - rg * a.G;
      const size_t tok = p.s.bos + rg;
      (static_cast<float *>(a.o) + tok * a.os + head * D)[c] = none ? 0.f : y / sum;
      if (a.lse && c == 0) a.lse[tok * a.Hq + head] = none ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    }
    __syncthreads();  // the ring is free again
  }
  if (tid == 0) reinterpret_cast<AttnRec *>(a.part)[blockIdx.x] = rec;
}

template <int D, int NR> cudaError_t launch_few(const AttnArgs &a, cudaStream_t s) {
  constexpr size_t bytes = FewSmem<D, NR>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(attn_f32_few_kernel<D, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) return e;
  attn_f32_few_kernel<D, NR><<<grid_of(D), kThreads, bytes, s>>>(a);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_attn_join(a, grid_of(D), NR, s) : e;
}

// Up to 4 rows of a (sequence, head) on average, items of 4, else of 8.
bool four(const AttnArgs &a) { return (long long)a.T_total * a.G <= 4LL * a.N; }

}  // namespace

size_t attn_f32_few_floats(const AttnArgs &a) { return attn_part_floats(grid_of(a.d), four(a) ? 4 : 8, a.d); }

cudaError_t launch_attn_f32_few(const AttnArgs &a, cudaStream_t s) {
  const bool f = four(a);
  switch (a.d) {
    case 16: return f ? launch_few<16, 4>(a, s) : launch_few<16, 8>(a, s);
    case 32: return f ? launch_few<32, 4>(a, s) : launch_few<32, 8>(a, s);
    case 64: return f ? launch_few<64, 4>(a, s) : launch_few<64, 8>(a, s);
    default: return f ? launch_few<128, 4>(a, s) : launch_few<128, 8>(a, s);
  }
}

}  // namespace kda
