// Attention over a paged cache: the division of the work, shared by its kernels.
//
// The query rows of a sequence and a head of the cache are its new tokens times
// the G query heads that share the head, token by token: row i is token i / G,
// head h G + i % G.  An item is R of these rows; it runs over the keys that they
// may see in tiles of KT.  All items' tiles, in the order (sequence, head, rows),
// are cut into one stretch of equal length for each block of the grid: blocks
// then finish together whatever the lengths are, which only the device knows.  An
// item that a stretch does not hold whole leaves, for each block that has a part of it, the
// maxima, sums and unnormalised outputs of that part in the workspace, and a second
// kernel joins them in order.  An item counts kStart tiles more than it has, for what it
// costs to begin and end: blocks whose items are short would otherwise be last.  A block has two such parts at most: one that goes on
// with an item (slot 0) and one that begins one (slot 1).
#pragma once

#include "kda_internal.cuh"
#include "kda_packed.cuh"

namespace kda {

// SMs of the card: the grids, and with them the workspaces' sizes, are whole multiples.  (With fewer SMs blocks would run
// in a second wave, with the same results.)
constexpr int kSms = 152;

// The joining record of a block: the item that it begins and does not end.
struct AttnRec {
  int n, h, r, parts;  // parts: blocks that hold some of it; 0: there is none
};

__host__ __device__ inline size_t attn_rec_floats(int grid) { return (size_t)grid * 4; }
// floats of the workspace: records, then [grid][2][R] rows of d + 2
__host__ __device__ inline size_t attn_part_floats(int grid, int R, int d) {
  return attn_rec_floats(grid) + (size_t)grid * 2 * R * (d + 2);
}
__device__ __forceinline__ float *attn_part_out(const AttnArgs &a, int grid, int block, int slot, int R, int row) {
  return a.part + attn_rec_floats(grid) + ((size_t)(block * 2 + slot) * R + row) * a.d;
}
__device__ __forceinline__ float2 *attn_part_ml(const AttnArgs &a, int grid, int block, int slot, int R, int row) {
  return reinterpret_cast<float2 *>(a.part + attn_rec_floats(grid) + (size_t)grid * 2 * R * a.d) +
         ((size_t)(block * 2 + slot) * R + row);
}

// a / b for a >= 0, b > 0; 64-bit divisions take several times as long as 32-bit ones.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return (unsigned long long)(a | b) >> 32 ? a / b : (long long)((unsigned)a / (unsigned)b);
}

// Keys that rows up to `row` of a sequence may see: the first `end` ones.
__device__ __forceinline__ int attn_end(const AttnArgs &a, const PagedSeq &s, int row) {
  if (!a.causal) return s.kv;
  return min(max(s.kv - s.len + a.by_G(row) + 1, 0), s.kv);
}

// Items of a (sequence, head), and tiles of one: at least one, so that rows
// without keys are written too.
template <int R> __device__ __forceinline__ int attn_items(const AttnArgs &a, const PagedSeq &s) {
  return (s.len * a.G + R - 1) / R;
}
template <int R, int KT> __device__ __forceinline__ int attn_tiles(const AttnArgs &a, const PagedSeq &s, int r) {
  return max(1, (attn_end(a, s, min((r + 1) * R, s.len * a.G) - 1) + KT - 1) / KT);
}
// sum of floor((k i + b) / m) over 0 <= i < n, for k, b >= 0, by Euclid's algorithm on (k, m): whole multiples come out of
// the sum, and what is left is the sum over the exchanged k and m (Graham, Knuth, Patashnik, Concrete Mathematics, 3.5).
__device__ __forceinline__ unsigned long long floor_sum(unsigned long long n, unsigned long long m, unsigned long long k,
                                                        unsigned long long b) {
  unsigned long long sum = 0;
  while (true) {
    sum += (n * (n - 1) / 2) * (k / m) + n * (b / m);
    k %= m;
    b %= m;
    const unsigned long long top = k * n + b;
    if (top < m) return sum;
    n = top / m;
    b = top % m;
    const unsigned long long x = m;
    m = k;
    k = x;
  }
}
// Tiles of the first n items: whole ones have floor(((kv - len + KT) G + (r + 1) R - 1) / (G KT)) or one.
template <int R, int KT> __device__ __forceinline__ long long attn_tiles_before(const AttnArgs &a, const PagedSeq &s, int n) {
  if (n == 0) return 0;
  const int items = attn_items<R>(a, s);
  if (items == 1) return attn_tiles<R, KT>(a, s, 0);
  if (!a.causal) return (long long)n * attn_tiles<R, KT>(a, s, 0);
  long long sum = 0;
  if (n == items) {  // the last one may have fewer rows
    sum = attn_tiles<R, KT>(a, s, --n);
    if (n == 0) return sum;
  }
  const long long m = (long long)a.G * KT, first = (long long)(s.kv - s.len + KT) * a.G + R - 1;
  const long long low = first >= m ? 0 : min((long long)n, quotient(m - first + R - 1, R));  // items of one tile at the start
  sum += low;
  if (low < n) sum += floor_sum(n - low, m, R, first + low * R);
  return sum;
}
// Units of the stretches: an item has its tiles and kStart more.
template <int R, int KT, int kStart> __device__ __forceinline__ long long attn_units_before(const AttnArgs &a, const PagedSeq &s, int n) {
  return attn_tiles_before<R, KT>(a, s, n) + (long long)n * kStart;
}

// Where a block's stretch begins and what is left of it.
struct AttnWalk {
  int n, h, r, u;   // sequence, head, rows, unit of the item
  PagedSeq s;       // of n
  int block, blocks;  // this block, and those that have a stretch
  long long left, at, total;  // units left; index of the next one among `total`
};

// The stretch of block c of `grid`, by all NT threads of the block.
template <int R, int KT, int kStart, int NT>
__device__ __forceinline__ AttnWalk attn_walk(const AttnArgs &a, int c, int grid) {
  __shared__ long long warp_sums[NT / 32];
  __shared__ AttnWalk walk;
  const int tid = threadIdx.x, per = (a.N + NT - 1) / NT;
  const int lo = min(tid * per, a.N), hi = min(lo + per, a.N);
  long long sum = 0;
  for (int n = lo; n < hi; ++n) {
    const PagedSeq s = paged_seq(a, n);
    sum += attn_units_before<R, KT, kStart>(a, s, attn_items<R>(a, s)) * a.Hk;
  }
  long long upto = sum;  // sum of this thread and those below, first within the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(~0u, upto, o);
    if ((tid & 31) >= o) upto += x;
  }
  if ((tid & 31) == 31) warp_sums[tid >> 5] = upto;
  if (tid == 0) walk.left = walk.total = 0;
  __syncthreads();
  long long total = 0;
  for (int w = 0; w < NT / 32; ++w) {
    if (w < (tid >> 5)) upto += warp_sums[w];
    total += warp_sums[w];
  }
  // no stretch is empty, so that the parts of an item lie in consecutive blocks
  const int blocks = (int)min(total, (long long)grid);
  const long long begin = c < blocks ? quotient(total * c, blocks) : 0, end = c < blocks ? quotient(total * (c + 1), blocks) : 0;
  if (begin < end && begin >= upto - sum && begin < upto) {
    // the thread whose sequences hold the first tile: which of them, and how far in
    long long rest = begin - (upto - sum), head = 1;
    AttnWalk w{};
    for (w.n = lo; w.n < hi; ++w.n) {
      w.s = paged_seq(a, w.n);
      head = attn_units_before<R, KT, kStart>(a, w.s, attn_items<R>(a, w.s));
      if (rest < head * a.Hk) break;
      rest -= head * a.Hk;
    }
    w.h = (int)quotient(rest, head);
    w.at = rest - w.h * head;  // within the head, for the search below
    w.block = c;
    w.blocks = blocks;
    w.left = end - begin;
    w.total = total;
    walk = w;
  }
  __syncthreads();
  AttnWalk w = walk;
  if (w.left > 0) {  // the item: each thread looks at a few
    const int items = attn_items<R>(a, w.s), each = (items + NT - 1) / NT;
    const int r0 = min(tid * each, items), r1 = min(r0 + each, items);
    long long before = attn_units_before<R, KT, kStart>(a, w.s, r0);
    for (int r = r0; r < r1; ++r) {
      const int units = attn_tiles<R, KT>(a, w.s, r) + kStart;
      if (w.at >= before && w.at < before + units) {
        walk.r = r;
        walk.u = (int)(w.at - before);
      }
      before += units;
    }
  }
  __syncthreads();
  w = walk;
  w.at = begin;
  return w;
}

// One part of a stretch: tiles [t0, t1) of an item.
struct AttnPart {
  PagedSeq s;
  int n, h, r, t0, t1;
  bool whole;
  int slot;     // of the workspace, unless whole
  int parts;    // when it begins an item that it does not end: blocks that hold some of it
};
template <int R, int KT, int kStart>
__device__ __forceinline__ bool attn_next(const AttnArgs &a, AttnWalk &w, AttnPart &p) {
  while (w.left > 0) {
    int items = attn_items<R>(a, w.s);
    while (w.r >= items) {  // past the last item of a head
      w.r = 0;
      if (items == 0 || ++w.h >= a.Hk) {
        w.h = 0;
        w.s = paged_seq(a, ++w.n);  // (some sequence follows as long as units are left)
        items = attn_items<R>(a, w.s);
      }
    }
    const int nt = attn_tiles<R, KT>(a, w.s, w.r), units = nt + kStart;
    const int take = (int)min(w.left, (long long)units - w.u);
    p.s = w.s;
    p.n = w.n;
    p.h = w.h;
    p.r = w.r;
    p.t0 = max(w.u - kStart, 0);
    p.t1 = max(w.u + take - kStart, 0);
    p.whole = p.t0 == 0 && p.t1 == nt;
    p.slot = p.t0 == 0 ? 1 : 0;
    p.parts = 0;
    if (p.t0 == 0 && !p.whole) {
      // up to the block whose stretch holds its last unit; stretch c begins at floor(total c / blocks)
      p.parts = (int)quotient((w.at - w.u + units) * w.blocks - 1, w.total) - w.block + 1;
    }
    w.at += take;
    w.left -= take;
    w.u = 0;
    ++w.r;
    if (p.t1 > p.t0) return true;  // (else the stretch ends within what counts for the item's start)
  }
  return false;
}

// Element offset of (page of key j, slot, head h) in the cache.
__device__ __forceinline__ long long key_offset(const AttnArgs &a, int page_id, int slot, int h) {
  return min(max(page_id, 0), a.pages - 1) * a.cs + ((long long)h * a.page + slot) * a.d;
}

// Lets the joining kernel's launch begin while this one runs, and waits there for the end of it.
__device__ __forceinline__ void attn_let_join() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void attn_wait_for_first() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Joins the parts of the items that blocks of `grid` began and did not end.
cudaError_t launch_attn_join(const AttnArgs &a, int grid, int R, cudaStream_t s);

// kda_attn_f32.cu, kda_attn_f32_few.cu, kda_attn_mma.cu, kda_attn_tc.cu
size_t attn_f32_few_floats(const AttnArgs &a);
cudaError_t launch_attn_f32_few(const AttnArgs &a, cudaStream_t s);
size_t attn_f32_floats(const AttnArgs &a);
cudaError_t launch_attn_f32(const AttnArgs &a, cudaStream_t s);
size_t attn_mma_floats(const AttnArgs &a);
cudaError_t launch_attn_mma(const AttnArgs &a, cudaStream_t s);
bool attn_tc_supports(const AttnArgs &a);
size_t attn_tc_floats(const AttnArgs &a);
cudaError_t launch_attn_tc(const AttnArgs &a, cudaStream_t s);

}  // namespace kda
