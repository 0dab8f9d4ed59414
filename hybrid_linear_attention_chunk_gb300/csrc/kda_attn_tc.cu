// Attention over a paged cache in bf16 for many query rows to a head of the cache:
// prefills and chunks, bound by the tensor cores.
//
// An item is 256 query rows as two tiles of 128, each with its scores S = Q K^T
// and its outputs O += P V on tcgen05 with fp32 accumulators in TMEM; P, in bf16,
// takes the place of its S there and is the second product's operand as it lies.  Two
// warpgroups hold one row of a tile in each thread, so that the softmax needs no
// exchange between threads.  While one tile's softmax runs, the tensor cores have the
// other tile's products.  One warp issues the products, one the copies of keys and values
// (TMA from the pages, 128 keys at a time), and two go over the values of tiles that some row does not see
// whole: slots behind the sequence's end are zeroed there, since 0 times what lies in
// them need not be 0, and values that are not finite are taken out and listed, to be
// added in the end to the rows that see them.
//
// A row's outputs stand relative to a reference that follows its running maximum in steps: it is set 2^8 above
// the maximum, and the outputs need not be rescaled until the maximum is above the reference.  Probabilities are then
// at most 1, as where the reference is the maximum itself, so that values of up to fp32's range over the number of
// keys do not overflow the outputs; a factor of 2^-8 costs bf16 and fp32 no bits.
//
// Every wait on an mbarrier is bounded (2 s).  On a time-out all warps leave their loops, products and copies in flight
// are waited for, TMEM is freed and a bit is set in a device word the host can read (kda_device_watchdog).
//
// P is rounded to bf16 since both operands of the product have one type and V is bf16: 2^-8 of each probability at most,
// while their sum is of the unrounded ones.  The outputs' error against fp64 grows by it from 0.0016, their own rounding, to
// 0.0018-0.0023.  A second product with what the rounding leaves out would make the two products three.
//
// Measured with heads of 128, 32 on 8: 8192 tokens from an empty cache 371 us and 16 us for the
// join, 380 together (1.45 PFLOP/s, tensor pipe 67 % active); 2048 tokens over 65536 in 1440 us (tensor pipe 76 %
// active) while the card's clock holds and 1650 us (1.36 PFLOP/s) when it runs for seconds, at 1.37 kW and 1500 of 2070 MHz.
// 8192 tokens with heads of 64 take 335 us (0.82 PFLOP/s, tensor pipe 37 % active), 2048 over 65536 1135 us (1.0
// PFLOP/s): their products of 64 channels are issued no faster than those of 128.  A tile of 128 keys takes about 2900
// cycles, its products 2048 of them: the rest is waits between products (a ready one costs about 100 cycles, five a tile),
// since the two tiles of scores and outputs fill TMEM and no third product can be in line.  A part costs
// about 12000 cycles beside its tiles: queries, the first softmax, outputs.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <string.h>

#include "kda_attn.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int kThreads = 384, kRows = 256, kKeys = 128;
// Tiles that an item counts for its start and end, about 12000 cycles to a tile's 2900.  2 and 4 against 3: 8192 tokens 377
// and 375 against 372 us, 20 x 300 tokens over 500 116 and 112 against 113, the mixed batch of heads of 64 the same.
constexpr int kStart = 3;
constexpr int kMaxStages = 4;
constexpr float kSlack = 8.f;  // powers of two that a row's reference is set above its maximum
constexpr uint32_t kHalf = 16384;  // 128 rows of 64 channels

enum Bar {
  B_Q = 0,                        // [2] queries in shared memory
  B_S = 2,                        // [2] scores in TMEM
  B_P = 4,                        // [2] probabilities in TMEM, outputs rescaled
  B_O = 6,                        // [2] the part's outputs are complete
  B_KFULL = 8,                    // [stages] keys landed
  B_KEMPTY = B_KFULL + kMaxStages,
  B_VFULL = B_KEMPTY + kMaxStages,
  B_VEMPTY = B_VFULL + kMaxStages,
  B_VOK = B_VEMPTY + kMaxStages,  // values gone over, where they need it
  B_DRAIN = B_VOK + kMaxStages,
  B_FULL,                         // [4] a part is told
  B_EMPTY = B_FULL + 4,           // [4] every warp is done with a part
  B_COUNT = B_EMPTY + 4
};

// What a wait that runs out reports, by what it waited for: bits of KDA_WATCHDOG_PAGED_ATTN.
enum Code : unsigned {
  C_QUERIES = 1u << 16,
  C_SCORES = 1u << 17,
  C_PROBS = 1u << 18,
  C_OUTPUTS = 1u << 19,
  C_KEYS = 1u << 21,
  C_VALUES = 1u << 22,
  C_PART = 1u << 28,
  C_DRAIN = 1u << 29   // what is in flight after an abort
};
static_assert((C_QUERIES | C_SCORES | C_PROBS | C_OUTPUTS | C_KEYS | C_VALUES | C_PART | C_DRAIN) == KDA_WATCHDOG_PAGED_ATTN &&
                  C_QUERIES + C_SCORES + C_PROBS + C_OUTPUTS + C_KEYS + C_VALUES + C_PART + C_DRAIN == KDA_WATCHDOG_PAGED_ATTN,
              "a bit to each kind of wait, none shared");

// A part, as the copy warp works it out for all: it runs ahead of the others.
constexpr int kParts = 4;         // told at a time
struct Part {
  int n, h;                       // sequence, head of the cache
  int t0, t1;                     // tiles; t1 = 0: there are no more parts
  int bos, before, kv;            // first new token, position of it, length
  int rows, row0;                 // rows of the (sequence, head); of the item
  int most, all[2];               // keys that some row sees; that every row of each 128 sees
  int count[2];                   // tiles of each 128 rows within the part
  int whole, slot;
  // keys that a row sees
  __device__ __forceinline__ int end(const AttnArgs &a, int row) const {
    return a.causal ? min(max(before + a.by_G(row) + 1, 0), kv) : kv;
  }
  // whether tile t has keys that some row does not see
  __device__ __forceinline__ bool at_end(int t) const { return (t + 1) * kKeys > all[0]; }
};

struct Ctl {
  uint64_t bar[B_COUNT];
  uint32_t tmem;
  int abort;
  Part part[kParts];
  uint32_t odd[kParts][3][4];  // [part % 4][tile at the end][32 keys]: keys with values that are not finite
};

template <int D> struct Tc {
  static constexpr uint32_t kTile = D / 64 * kHalf;
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr uint32_t kK = 2 * kTile, kV = kK + kStages * kTile, kCtl = kV + kStages * kTile;
  static constexpr uint32_t kBytes = kCtl + sizeof(Ctl) + 1024;
};

struct TcArgs {
  AttnArgs a;
  unsigned int *err;
  int box;  // rows of a copy: a page's, at most 128
};

struct Waits {
  Ctl *ctl;
  unsigned int *err;
  // By a whole warp; false when any of its lanes gave up.
  __device__ __forceinline__ bool operator()(int b, uint32_t parity, Code code) const {
    return __all_sync(~0u, mbar_wait(smem_u32(&ctl->bar[b]), parity & 1u, &ctl->abort, err, code));
  }
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *m, uint32_t bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// 32 bytes to global memory: whole sectors where the address allows it.
__device__ __forceinline__ void store32(void *to, const uint32_t (&w)[8], bool aligned) {
  if (aligned) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
  } else {
    reinterpret_cast<uint4 *>(to)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4 *>(to)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The parts in turn, for a warp that is told of them.
struct Parts {
  Ctl *ctl;
  Waits wait;
  int at = 0;
  // The next part, or nullptr behind the last one or after an abort.
  __device__ __forceinline__ const Part *next() const {
    if (!wait(B_FULL + at % kParts, at / kParts, C_PART)) return nullptr;
    const Part *p = &ctl->part[at % kParts];
    return p->t1 ? p : nullptr;
  }
  __device__ __forceinline__ void done() {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&ctl->bar[B_EMPTY + at % kParts]));
    ++at;
  }
};

// ------------------------------------------------------------------ softmax

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0],"
      " {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
      "%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// Probabilities of 64 scores relative to kSlack powers of two above m, in pairs of bf16 to w; returns their sum in two parts.
__device__ __forceinline__ Vec<2> half_of(const float *s, float scale2, float m, uint32_t (&w)[32]) {
  const float r = m == -INFINITY ? 0.f : fmaf(-m, scale2, -kSlack);
  const Vec<2> scale = pair(scale2, scale2), ref = pair(r, r);
  Vec<2> sum = pair(0.f, 0.f);
#pragma unroll
  for (int x = 0; x < 32; ++x) {
    const Vec<2> e = fma(pair(s[2 * x], s[2 * x + 1]), scale, ref);
    const float lo = fast_exp2(e.get(0)), hi = fast_exp2(e.get(1));
    sum = add(sum, pair(lo, hi));
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    w[x] = *reinterpret_cast<const uint32_t *>(&b);
  }
  return sum;
}

__device__ __forceinline__ float max_of(const float (&s)[128]) {
  float t[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
  for (int c = 4; c < 124; c += 8)
#pragma unroll
    for (int x = 0; x < 4; ++x) t[x] = max3(t[x], s[c + 2 * x], s[c + 2 * x + 1]);
  return max3(max3(t[0], t[1], fmaxf(s[124], s[125])), max3(t[2], t[3], s[126]), s[127]);
}

template <int D>
__device__ __forceinline__ void softmax_role(const AttnArgs &a, Ctl *ctl, const Waits &wait, unsigned char *smem, int i) {
  const int grid = gridDim.x, tid = threadIdx.x % 128, qw = tid / 32;
  const uint32_t tb = ctl->tmem + ((uint32_t)(32 * qw) << 16), ts = tb + 128 * i, to = tb + 256 + 128 * i;
  const uint32_t qs = smem_u32(smem) + i * Tc<D>::kTile;
  const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q), *vc = static_cast<const __nv_bfloat16 *>(a.vc);
  uint32_t seen_s = 0, seen_o = 0;
  // Queries of a part: asynchronous 16-byte copies, D / 8 of a row, into the swizzled operand tile.  The last
  // product that read it is complete once this warpgroup has seen its scores.
  auto issue_queries = [&](const Part *p) {
    const int first = p->row0 + 128 * i, rows = p->rows;
    if (p->count[i] == 0) return false;
    const __nv_bfloat16 *base = q + p->bos * a.qs + p->h * a.G * D + tid % (D / 8) * 8;
    const uint32_t dst = qs + (tid % (D / 8) / 8) * kHalf;
#pragma unroll 4
    for (int x = 0; x < D / 8; ++x) {
      const int r = x * (1024 / D) + tid / (D / 8), rt = min(first + r, rows - 1), rg = a.by_G(rt);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + sw128_offset(r, tid % 8 * 8)),
                   "l"(base + rg * a.qs + (rt - rg * a.G) * D), "r"(first + r < rows ? 16 : 0) : "memory");
    }
    return true;
  };
  auto land_queries = [&]() {
    asm volatile("cp.async.wait_all;" ::: "memory");
    fence_proxy_async_smem();
    mbar_arrive(smem_u32(&ctl->bar[B_Q + i]));
  };
  Parts parts{ctl, wait};
  const Part *p = parts.next();
  if (p && issue_queries(p)) land_queries();
  while (p) {
    const int first = p->row0 + 128 * i, n = p->count[i];
    if (first >= p->rows) {
      parts.done();
      p = parts.next();
      if (p && issue_queries(p)) land_queries();
      continue;
    }
    const int lim = first + tid < p->rows ? p->end(a, first + tid) : 0, all = p->all[i], t0 = p->t0;
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < n; ++j) {
      const int key0 = (t0 + j) * kKeys;
      if (!wait(B_S + i, seen_s++, C_SCORES)) return;
      tc_fence_after();
      float s[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, *reinterpret_cast<float(*)[32]>(s + 32 * c));
      tmem_wait_ld();
      const int nv = key0 + kKeys > all ? lim - key0 : kKeys;  // keys that the row sees
      if (key0 + kKeys > all) {
#pragma unroll
        for (int c = 0; c < 128; ++c) s[c] = c < nv ? s[c] : -INFINITY;
      }
      // The first half's probabilities by the reference as it is, beside the search for the maximum; seldom
      // this is above the reference, then the reference moves and they are formed anew.
      uint32_t w[32];
      Vec<2> sum = pair(0.f, 0.f);
      float top;
      if (j > 0) {
        sum = half_of(s, a.scale2, m, w);
        top = max_of(s);
      } else {
        top = max_of(s);
      }
      if (j == 0 || __any_sync(~0u, top * a.scale2 > m * a.scale2 + kSlack)) {
        const float next = fmaxf(m, top);
        const float f = next == -INFINITY ? 1.f : fast_exp2((m - next) * a.scale2);
        l *= f;
        m = next;
        if (j > 0) {  // (these scores came after the products that O holds)
#pragma unroll
          for (int c = 0; c < D; c += 16) {
            float o[16];
            tmem_ld16(to + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 16; ++x) o[x] *= f;
            tmem_st16(to + c, o);
          }
        }
        float again[64];
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_ld32(ts + 32 * c, *reinterpret_cast<float(*)[32]>(again + 32 * c));
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 64; ++c) again[c] = c < nv ? again[c] : -INFINITY;
        sum = half_of(again, a.scale2, m, w);
      }
      tmem_st32(ts, w);
      sum = add(sum, half_of(s + 64, a.scale2, m, w));
      tmem_st32(ts + 32, w);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(smem_u32(&ctl->bar[B_P + i]));
      l += sum.get(0) + sum.get(1);
    }
    // The next part's queries come while the last products run, and its first scores are
    // computed while this one's outputs are written.
    Parts ahead = parts;
    ++ahead.at;
    const Part *next = ahead.next();
    const bool queries = next && issue_queries(next);
    if (n > 0) {
      if (!wait(B_O + i, seen_o++, C_OUTPUTS)) return;
      tc_fence_after();
    }
    if (queries) land_queries();
    const int at = first + tid, rg = a.by_G(at), head = p->h * a.G + at - rg * a.G;
    const size_t tok = p->bos + rg;
    const bool mine = at < p->rows, none = lim == 0, whole = p->whole;
    const float inv = 1.f / l;
    uint32_t any = 0;  // listed keys of the tiles at the end
    const int end0 = p->all[0] / kKeys, from = max(t0, end0), ring = parts.at % kParts;
    for (int t = from; t < t0 + n; ++t)
#pragma unroll
      for (int x = 0; x < 4; ++x) any |= ctl->odd[ring][t - end0][x];
    float *to_part = attn_part_out(a, grid, blockIdx.x, p->slot, kRows, 128 * i + tid);
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      float o[32];
      if (n > 0) {
        tmem_ld32(to + c, o);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int x = 0; x < 32; ++x) o[x] = 0.f;
      }
      if (any && mine) {
        for (int k = from * kKeys; k < min(lim, (t0 + n) * kKeys); ++k) {
          if (!((ctl->odd[ring][k / kKeys - end0][k % kKeys / 32] >> (k % 32)) & 1u)) continue;
          const int id = a.table[(long long)p->n * a.max_pages + k / a.page];
          const __nv_bfloat16 *v = vc + key_offset(a, id, k % a.page, p->h) + c;
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            const float y = __bfloat162float(v[x]);
            if (!isfinite(y)) o[x] += y;
          }
        }
      }
      if (!mine) continue;
      if (whole) {
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.o) + tok * a.os + head * D + c;
        const bool aligned = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
#pragma unroll
        for (int x = 0; x < 32; x += 16) {
          uint32_t w[8];
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const __nv_bfloat162 b = none ? __floats2bfloat162_rn(0.f, 0.f)
                                          : __floats2bfloat162_rn(o[x + 2 * y] * inv, o[x + 2 * y + 1] * inv);
            w[y] = *reinterpret_cast<const uint32_t *>(&b);
          }
          store32(out + x, w, aligned);
        }
      } else {
        const bool aligned = (reinterpret_cast<uintptr_t>(to_part) & 31u) == 0;
#pragma unroll
        for (int x = 0; x < 32; x += 8) {
          uint32_t w[8];
#pragma unroll
          for (int y = 0; y < 8; ++y) w[y] = __float_as_uint(o[x + y]);
          store32(to_part + c + x, w, aligned);
        }
      }
    }
    tc_fence_before();
    if (mine) {
      if (!whole) *attn_part_ml(a, grid, blockIdx.x, p->slot, kRows, 128 * i + tid) = make_float2(fmaf(m, a.scale2, kSlack), l);
      else if (a.lse)  // (l in terms of the maximum, so that the logarithm of a sum of few keys is not the small difference of two)
        a.lse[tok * a.Hq + head] = none ? -INFINITY : fmaf(m, a.scale2, log2f(l * exp2f(kSlack))) * 0.6931471805599453f;
    }
    parts.done();
    p = next;
  }
}

// ----------------------------------------------------------------- products

// Products are issued by a whole warp in step, one lane elected in the instruction:
// what an instruction needs is then uniform, and a product of 64 cycles is not held up by moving its operands.
// Low words of descriptors are the address / 16 and LBO / 16; the high word is the same for all operands here.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);  // SBO 1024, version, 128-byte swizzle
template <bool kFirst>
__device__ __forceinline__ void issue_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t.reg .b64 x, y;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(kDescHigh),
      "r"(idesc), "n"(kFirst ? 0 : 1)
      : "memory");
}
__device__ __forceinline__ void issue_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t.reg .b64 y;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 y, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(kDescHigh),
      "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void issue_commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar) : "memory");
}
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(~0u, x, 0); }

template <int D>
__device__ __forceinline__ void product_role(Ctl *ctl, const Waits &wait, unsigned char *smem) {
  constexpr uint32_t S = Tc<D>::kStages;
  constexpr uint32_t kIdS = idesc_bf16_f32(128, kKeys, 0, 0), kIdO = idesc_bf16_f32(128, D, 0, 1);
  const uint32_t base = uniform(smem_u32(smem)), tb = uniform(ctl->tmem), bars = uniform(smem_u32(&ctl->bar[0]));
  uint32_t ks = 0, kp = 0, vs = 0, vp = 0;  // stage and parity of the next keys and values
  auto scores = [&](int i) {                // S_i = Q_i K^T
    const uint32_t q = ((base + i * Tc<D>::kTile) >> 4) | 1u << 16;
    const uint32_t k = uniform(((base + Tc<D>::kK + ks * Tc<D>::kTile) >> 4) | 1u << 16);
    issue_ss<true>(tb + 128 * i, q, k, kIdS);
#pragma unroll
    for (int x = 1; x < D / 16; ++x) {
      const uint32_t off = ((x / 4) * kHalf + (x % 4) * 32) >> 4;
      issue_ss<false>(tb + 128 * i, q + off, k + off, kIdS);
    }
    issue_commit(bars + 8 * (B_S + i));
  };
  auto keys_done = [&]() {
    issue_commit(bars + 8 * (B_KEMPTY + ks));
    if (++ks == S) ks = 0, kp ^= 1u;
  };
  uint32_t nq[2] = {0, 0}, np[2] = {0, 0};
  Parts parts{ctl, wait};
  while (const Part *p = parts.next()) {
    const int count = p->t1 - p->t0, n0 = p->count[0], n1 = p->count[1];
    parts.done();
    if (n0 > 0 && !wait(B_Q, nq[0]++, C_QUERIES)) return;
    if (n1 > 0 && !wait(B_Q + 1, nq[1]++, C_QUERIES)) return;
    if (!wait(B_KFULL + ks, kp, C_KEYS)) return;
    tc_fence_after();
    if (n0 > 0) scores(0);
    if (n1 > 0) scores(1);
    keys_done();
    if (!wait(B_VOK + vs, vp, C_VALUES)) return;
    for (int j = 0; j < count; ++j) {
      const uint32_t v = uniform(((base + Tc<D>::kV + vs * Tc<D>::kTile) >> 4) | (kHalf >> 4) << 16);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int n = i ? n1 : n0;
        if (j < n) {
          if (!wait(B_P + i, np[i]++, C_PROBS)) return;
          tc_fence_after();
          issue_ts(tb + 256 + 128 * i, tb + 128 * i, v, kIdO, j > 0);
#pragma unroll
          for (int x = 1; x < kKeys / 16; ++x) issue_ts(tb + 256 + 128 * i, tb + 128 * i + 8 * x, v + x * (2048 >> 4), kIdO, 1u);
          if (j == n - 1) issue_commit(bars + 8 * (B_O + i));
        }
        if (i == 1) issue_commit(bars + 8 * (B_VEMPTY + vs));
        if (j + 1 < count && i == 0 && !wait(B_KFULL + ks, kp, C_KEYS)) return;
        if (j + 1 < n) scores(i);
      }
      if (++vs == S) vs = 0, vp ^= 1u;
      if (j + 1 < count) {
        keys_done();
        if (!wait(B_VOK + vs, vp, C_VALUES)) return;  // (while the last products run)
      }
    }
  }
}

// ------------------------------------------------------------------- copies

template <int D>
__device__ __forceinline__ void copy_role(const TcArgs &args, const CUtensorMap *mk, const CUtensorMap *mv, AttnWalk walk,
                                          Ctl *ctl, const Waits &wait, unsigned char *smem, int lane) {
  constexpr int S = Tc<D>::kStages;
  const AttnArgs &a = args.a;
  const int box = args.box, boxes = kKeys / box, b = lane % boxes, half = lane / boxes;  // (boxes is a power of two)
  const uint32_t base = smem_u32(smem), to_smem = half * kHalf + b * box * 128;
  uint32_t n = 0, issued[2] = {0, 0};  // tiles; copies of keys, of values
  bool alive = true;
  AttnRec rec{0, 0, 0, 0};
  AttnPart p;
  for (int at = 0; alive; ++at) {
    const bool more = attn_next<kRows, kKeys, kStart>(a, walk, p);
    if (!wait(B_EMPTY + at % kParts, at / kParts + 1, C_PART)) break;
    const int rows = p.s.len * a.G, row0 = p.r * kRows, most = more ? attn_end(a, p.s, min(row0 + kRows, rows) - 1) : 0;
    if (lane == 0) {
      Part *to = &ctl->part[at % kParts];
      to->t1 = 0;
      if (more) {
        if (p.parts) rec = AttnRec{p.n, p.h, p.r, p.parts};
        *to = Part{p.n, p.h, p.t0, p.t1, p.s.bos, p.s.kv - p.s.len, p.s.kv, rows, row0, most, {0, 0}, {0, 0}, p.whole, p.slot};
        for (int i = 0; i < 2; ++i) {
          const int first = row0 + 128 * i;
          if (first >= rows) continue;
          const int end = attn_end(a, p.s, min(first + 128, rows) - 1);
          to->all[i] = attn_end(a, p.s, first);
          to->count[i] = max(min(p.t1, max(1, (end + kKeys - 1) / kKeys)) - p.t0, 0);
        }
      }
      mbar_arrive(smem_u32(&ctl->bar[B_FULL + at % kParts]));
    }
    if (!more) break;
    const int32_t *table = a.table + (long long)p.n * a.max_pages;
    auto page_of = [&](int t) {
      const int j = t * kKeys + b * box;
      return t < p.t1 && half < D / 64 && j < most ? min(max(table[j / a.page], 0), a.pages - 1) : -1;
    };
    int id = page_of(p.t0);
    for (int t = p.t0; t < p.t1 && alive; ++t) {
      const int j = t * kKeys + b * box, slot = j % a.page;
      const uint32_t st = n % S, bytes = __popc(__ballot_sync(~0u, id >= 0)) * box * 128;
      const int next = page_of(t + 1);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        if (!alive || !wait((kv ? B_VEMPTY : B_KEMPTY) + st, n / S + 1, kv ? C_VALUES : C_KEYS)) {
          alive = false;
          continue;
        }
        const uint32_t bar = smem_u32(&ctl->bar[(kv ? B_VFULL : B_KFULL) + st]);
        if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
        ++issued[kv];
        __syncwarp();
        if (id >= 0)
          tma_load_4d(base + (kv ? Tc<D>::kV : Tc<D>::kK) + st * Tc<D>::kTile + to_smem, kv ? mv : mk, bar, half * 64, slot, p.h, id);
      }
      ++n;
      id = next;
    }
  }
  if (lane == 0) reinterpret_cast<AttnRec *>(a.part)[blockIdx.x] = rec;
  // copies still in flight after an abort land before the CTA retires
  volatile int no_abort = 0;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
    for (uint32_t x = issued[kv] > S ? issued[kv] - S : 0; x < issued[kv]; ++x)
      mbar_wait(smem_u32(&ctl->bar[(kv ? B_VFULL : B_KFULL) + x % S]), x / S & 1, &no_abort, args.err, C_DRAIN);
}

// ------------------------------------------------------------ values at the end

__device__ __forceinline__ uint32_t odd_bf16(uint32_t w) {  // mask of the halves that are not finite
  return ((w & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) | ((w & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}

template <int D>
__device__ __forceinline__ void value_role(Ctl *ctl, const Waits &wait, unsigned char *smem, int w, int lane) {
  constexpr int S = Tc<D>::kStages, kPieces = D / 8, kStep = 32 / kPieces;  // pieces of a row; rows at a time
  uint32_t n = 0;
  Parts parts{ctl, wait};
  while (const Part *p = parts.next()) {
    for (int t = p->t0; t < p->t1; ++t, ++n) {
      if (!wait(B_VFULL + n % S, n / S, C_VALUES)) return;
      if (!p->at_end(t)) {
        if (lane == 0) mbar_arrive(smem_u32(&ctl->bar[B_VOK + n % S]));
        continue;
      }
      const int valid = p->most - t * kKeys, c = lane % kPieces;  // rows up to `valid` hold values
      const uint32_t v = smem_u32(smem) + Tc<D>::kV + n % S * Tc<D>::kTile + (c / 8) * kHalf;
      auto at = [&](int r0) { return v + sw128_offset(w * 64 + r0 + lane / kPieces, (c % 8) * 8); };
      uint32_t list[2] = {0u, 0u};
      uint32_t top = 0;  // largest magnitudes of either half of the words, as integers: 0x7f80 and above are not finite
#pragma unroll 8
      for (int r0 = 0; r0 < 64; r0 += kStep) {
        uint4 x;
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at(r0)) : "memory");
        const uint32_t m = 0x7fff7fffu;
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & m, x.y & m), __vmaxu2(x.z & m, x.w & m)));
      }
      if (valid < w * 64 + 64) {
        for (int r0 = 0; r0 < 64; r0 += kStep)
          if (w * 64 + r0 + lane / kPieces >= valid)
            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(at(r0)), "r"(0u) : "memory");
        __syncwarp();
      }
      // (what lies behind the end counts here too, and is zero for the closer look)
      const bool odd = (top & 0xffffu) >= 0x7f80u || (top >> 16) >= 0x7f80u;
      if (__any_sync(~0u, odd)) {  // seldom
        for (int r0 = 0; r0 < 64; r0 += kStep) {
          uint4 x;
          asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at(r0)) : "memory");
          const uint32_t o[4] = {odd_bf16(x.x), odd_bf16(x.y), odd_bf16(x.z), odd_bf16(x.w)};
          const bool any = o[0] | o[1] | o[2] | o[3];  // (rows behind the end are zero by now)
          if (any)
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at(r0)), "r"(x.x & ~o[0]), "r"(x.y & ~o[1]),
                         "r"(x.z & ~o[2]), "r"(x.w & ~o[3]) : "memory");
          const uint32_t found = __ballot_sync(~0u, any);
          for (int y = 0; y < kStep; ++y)
            if ((found >> (y * kPieces)) & ((1u << kPieces) - 1u)) list[(r0 + y) / 32] |= 1u << ((r0 + y) % 32);
        }
      }
      if (lane < 2) ctl->odd[parts.at % kParts][t - p->all[0] / kKeys][2 * w + lane] = lane ? list[1] : list[0];
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->bar[B_VOK + n % S]));
    }
    parts.done();
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                   const __grid_constant__ TcArgs args) {
  extern __shared__ unsigned char raw[];
  unsigned char *smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  Ctl *ctl = reinterpret_cast<Ctl *>(smem + Tc<D>::kCtl);
  const AttnArgs &a = args.a;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, grid = gridDim.x;
  if (tid == 0) {
    ctl->abort = 0;
    for (int b = 0; b < B_COUNT; ++b) {
      const bool group = (b >= B_Q && b < B_Q + 2) || (b >= B_P && b < B_P + 2);
      const bool pair = b >= B_VOK && b < B_VOK + kMaxStages, empty = b >= B_EMPTY;
      mbar_init(smem_u32(&ctl->bar[b]), group ? 128 : pair ? 2 : empty ? 11 : 1);  // (11 warps are told of a part)
    }
    fence_mbar_init();
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(&ctl->tmem), 512);
    tmem_relinquish();
  }
  attn_let_join();
  const AttnWalk walk = attn_walk<kRows, kKeys, kStart, kThreads>(a, blockIdx.x, grid);  // (with barriers of the whole block)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const Waits wait{ctl, args.err};
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;" ::: "memory");
    softmax_role<D>(a, ctl, wait, smem, warp / 4);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;" ::: "memory");
    if (warp == 8) {
      product_role<D>(ctl, wait, smem);
      __syncwarp();
      if (lane == 0) {  // products in flight after an abort
        volatile int no_abort = 0;
        mma_commit(smem_u32(&ctl->bar[B_DRAIN]));
        mbar_wait(smem_u32(&ctl->bar[B_DRAIN]), 0, &no_abort, args.err, C_DRAIN);
      }
    } else if (warp == 9) {
      copy_role<D>(args, &mk, &mv, walk, ctl, wait, smem, lane);
    } else {
      value_role<D>(ctl, wait, smem, warp - 10, lane);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(ctl->tmem, 512);
  }
}

template <int D> cudaError_t launch_tc(const CUtensorMap &mk, const CUtensorMap &mv, const TcArgs &args, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(attn_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Tc<D>::kBytes);
  if (e != cudaSuccess) return e;
  attn_tc_kernel<D><<<kSms, kThreads, Tc<D>::kBytes, s>>>(mk, mv, args);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_attn_join(args.a, kSms, kRows, s) : e;
}

// [pages, Hk, page, d] as (channel, slot, head, page); boxes of 64 channels by `box` slots.
bool encode_cache(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap *m, const void *base, const AttnArgs &a, int box) {
  memset(m, 0, sizeof(*m));
  const cuuint64_t dims[4] = {(cuuint64_t)a.d, (cuuint64_t)a.page, (cuuint64_t)a.Hk, (cuuint64_t)a.pages};
  const cuuint64_t strides[3] = {(cuuint64_t)a.d * 2, (cuuint64_t)a.page * a.d * 2, (cuuint64_t)a.cs * 2};
  const cuuint32_t boxes[4] = {64u, (cuuint32_t)box, 1u, 1u}, es[4] = {1u, 1u, 1u, 1u};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, boxes, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// Heads of 64 or 128 channels, pages that tiles of 128 keys are made of, or that are made of such
// tiles, in boxes of at least 8 slots (a swizzled row group).
bool attn_tc_supports(const AttnArgs &a) {
  if (a.t != KDA_BF16 || (a.d != 64 && a.d != 128) || a.cs >= 1LL << 39) return false;  // (a tensor map's strides end at 2^40 bytes)
  return a.page % 8 == 0 && (a.page < kKeys ? kKeys % a.page == 0 : a.page % kKeys == 0);
}

size_t attn_tc_floats(const AttnArgs &a) { return attn_part_floats(kSms, kRows, a.d); }

cudaError_t launch_attn_tc(const AttnArgs &a, cudaStream_t s) {
  auto encode = tensor_map_encoder();
  if (!encode) return cudaErrorNotSupported;
  TcArgs args;
  args.a = a;
  args.box = a.page < kKeys ? a.page : kKeys;
  CUtensorMap mk, mv;
  if (!encode_cache(encode, &mk, a.kc, a, args.box) || !encode_cache(encode, &mv, a.vc, a, args.box))
    return cudaErrorInvalidValue;
  const cudaError_t e = tc_watchdog_word(&args.err);
  if (e != cudaSuccess) return e;
  return a.d == 128 ? launch_tc<128>(mk, mv, args, s) : launch_tc<64>(mk, mv, args, s);
}

}  // namespace kda
