// Entry points of the rotation, the append and the attention over a paged cache
// (include/kda.h): argument checks and launches.
#include <math.h>

#include "kda_check.cuh"

namespace kda {
namespace {

constexpr long long kMostElements = 1LL << 44;

// Rows of one tensor: `n` of them, `bytes` long, `stride` bytes apart.
struct Rows {
  uintptr_t base;
  size_t n, bytes, stride;
};

bool overlap(const Rows &a, const Rows &b) {
  if (!a.base || !b.base || !a.n || !b.n) return false;
  const Range ra{a.base, a.base + (a.n - 1) * a.stride + a.bytes}, rb{b.base, b.base + (b.n - 1) * b.stride + b.bytes};
  if (!overlap(ra, rb)) return false;
  if (a.stride != b.stride || a.n == 1 || b.n == 1) return true;
  // beside each other in rows of the same stride: b starts `off` behind a row of a
  const size_t off = b.base >= a.base ? (b.base - a.base) % a.stride
                                      : (a.stride - (a.base - b.base) % a.stride) % a.stride;
  return !(off >= a.bytes && a.stride - off >= b.bytes);
}

bool same(const Rows &a, const Rows &b) { return a.base == b.base && (a.stride == b.stride || a.n <= 1); }

// No output may overlap an input or an output before it; out[i] may be in[same_in[i]] itself.
bool aliased_rows(const Rows *in, int n_in, const Rows *out, int n_out, const int *same_in) {
  for (int o = 0; o < n_out; ++o) {
    for (int i = 0; i < n_in; ++i)
      if (!(same_in[o] == i && same(in[i], out[o])) && overlap(in[i], out[o])) return true;
    for (int p = 0; p < o; ++p)
      if (overlap(out[p], out[o])) return true;
  }
  return false;
}

Rows rows_of(const void *p, long long n, long long width, long long stride, size_t e) {
  return Rows{reinterpret_cast<uintptr_t>(p), (size_t)n, (size_t)width * e, (size_t)stride * e};
}
Rows flat(const void *p, size_t bytes) { return Rows{reinterpret_cast<uintptr_t>(p), bytes ? 1u : 0u, bytes, bytes}; }

// A token stride in elements (0: dense), or -1 when it does not do.
long long token_stride(int64_t stride, long long width, kda_dtype t) {
  if (stride == 0) return width;
  return stride < width || stride >= (1LL << 32) || stride % (t == KDA_BF16 ? 8 : 4) ? -1 : (long long)stride;
}

kda_status check_turn(int rot, int layout, float rot_scale, int norm, float eps, int d, const float *freq,
                      const float *qw, const float *kw, RopeArgs *a) {
  if (rot < 0 || rot > d || rot % 8) return KDA_ERR_SHAPE;
  if (layout != KDA_ROPE_HALF && layout != KDA_ROPE_INTERLEAVED) return KDA_ERR_SHAPE;
  if (rot && !freq) return KDA_ERR_NULL;
  if ((qw || kw) && !norm) return KDA_ERR_UNSUPPORTED;
  if ((norm && !(eps >= 0.f)) || !isfinite(rot_scale)) return KDA_ERR_RANGE;
  if (!aligned_to(freq, 4) || !aligned_to(qw, 4) || !aligned_to(kw, 4)) return KDA_ERR_ALIGN;
  a->d = d;
  a->rot = rot;
  a->inter = layout == KDA_ROPE_INTERLEAVED;
  a->norm = norm != 0;
  a->rot_scale = rot_scale;
  a->eps = eps;
  a->freq = freq;
  a->qw = qw;
  a->kw = kw;
  return KDA_OK;
}

kda_status rope_sizes(const kda_rope_desc *d) {
  if (!dtype_ok(d->dtype)) return KDA_ERR_DTYPE;
  if (d->tokens < 0 || d->tokens >= (1LL << 31) - 65536 || d->Hq <= 0 || d->Hk < 0 || !dim_ok(d->d)) return KDA_ERR_SHAPE;
  if (((long long)d->Hq + d->Hk) * d->d >= (1LL << 27)) return KDA_ERR_SHAPE;
  return KDA_OK;
}

// Strides and alignment of a tensor pair; the spans in elements stay below kMostElements.
kda_status pair_rows(const kda_rope_desc *d, const void *q, const void *k, int64_t qs, int64_t ks, Rows *rq, Rows *rk,
                     long long *sq, long long *sk) {
  const size_t e = esize(d->dtype);
  *sq = token_stride(qs, (long long)d->Hq * d->d, d->dtype);
  *sk = token_stride(ks, (long long)d->Hk * d->d, d->dtype);
  if (*sq < 0 || *sk < 0 || *sq * d->tokens >= kMostElements || *sk * d->tokens >= kMostElements) return KDA_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(k)) return KDA_ERR_ALIGN;
  *rq = rows_of(q, d->tokens, (long long)d->Hq * d->d, *sq, e);
  *rk = rows_of(k, d->Hk ? d->tokens : 0, (long long)d->Hk * d->d, *sk, e);
  return KDA_OK;
}

kda_status check_rope(const kda_rope_desc *d, const int32_t *positions, const float *freq, const float *qw,
                      const float *kw, RopeArgs *a) {
  kda_status st = rope_sizes(d);
  if (st != KDA_OK) return st;
  st = check_turn(d->rot, d->layout, d->rot_scale, d->norm, d->eps, d->d, freq, qw, kw, a);
  if (st != KDA_OK) return st;
  if (d->rot && !positions) return KDA_ERR_NULL;
  if (!aligned_to(positions, 4)) return KDA_ERR_ALIGN;
  a->tokens = d->tokens;
  a->Hq = d->Hq;
  a->Hk = d->Hk;
  a->t = d->dtype;
  a->positions = positions;
  return KDA_OK;
}

// ------------------------------------------------------------- paged cache

// Sizes of a descriptor.
kda_status paged_sizes(const kda_paged_desc *d, bool varlen, PagedArgs *a) {
  if (!dtype_ok(d->dtype)) return KDA_ERR_DTYPE;
  if (d->B <= 0 || d->T < 0 || d->num_seqs < 0 || !dim_ok(d->d)) return KDA_ERR_SHAPE;
  if (varlen ? (d->B != 1 || d->num_seqs <= 0) : d->num_seqs != 0) return KDA_ERR_SHAPE;
  if (d->Hk <= 0 || d->Hq <= 0 || d->Hq % d->Hk) return KDA_ERR_SHAPE;
  if (d->page_size <= 0 || d->num_pages <= 0 || d->max_pages <= 0) return KDA_ERR_SHAPE;
  const long long tokens = (long long)d->B * d->T, page = (long long)d->Hk * d->page_size * d->d;
  if (tokens * (d->Hq / d->Hk) >= (1LL << 31) - 65536 || (long long)d->Hq * d->d >= (1LL << 27)) return KDA_ERR_SHAPE;
  if ((long long)d->max_pages * d->page_size >= (1LL << 31) - 65536 || page >= (1LL << 40)) return KDA_ERR_SHAPE;
  const long long cs = d->cache_stride ? d->cache_stride : page;
  if (cs < page || cs % (d->dtype == KDA_BF16 ? 8 : 4) || cs >= (1LL << 40) || cs * d->num_pages >= kMostElements)
    return KDA_ERR_SHAPE;
  a->N = varlen ? d->num_seqs : d->B;
  a->T_total = (int)tokens;
  a->T_seq = varlen ? 0 : d->T;
  a->Hq = d->Hq;
  a->Hk = d->Hk;
  a->d = d->d;
  a->page = d->page_size;
  a->pages = d->num_pages;
  a->max_pages = d->max_pages;
  a->t = d->dtype;
  a->cs = cs;
  a->lens = a->cu = a->table = nullptr;
  return KDA_OK;
}

kda_status check_paged(const kda_paged_desc *d, const int32_t *lens, const int32_t *cu, const int32_t *table,
                       const void *kc, const void *vc, PagedArgs *a) {
  if (!d || !lens || !table || !kc || !vc) return KDA_ERR_NULL;
  const kda_status st = paged_sizes(d, cu != nullptr, a);
  if (st != KDA_OK) return st;
  if (!aligned_to(lens, 4) || !aligned_to(cu, 4) || !aligned_to(table, 4) || !aligned16(kc) || !aligned16(vc))
    return KDA_ERR_ALIGN;
  a->lens = lens;
  a->cu = cu;
  a->table = table;
  return KDA_OK;
}

Rows cache_rows(const PagedArgs &a, const void *p) {
  return rows_of(p, a.pages, (long long)a.Hk * a.page * a.d, a.cs, esize(a.t));
}

kda_status validate_paged(const kda_paged_desc *d, const PagedArgs &a, cudaStream_t s) {
  if (!d->validate) return KDA_OK;
  return run_validation(s, [&](int *flag) { return launch_validate_paged(a, flag, s); });
}

kda_status attn_args(const kda_paged_desc *d, AttnArgs *a) {
  a->scale2 = d->scale * 1.4426950408889634f;
  if (!(d->scale > 0.f) || !isfinite(a->scale2)) return KDA_ERR_RANGE;
  a->G = d->Hq / d->Hk;
  // the multiple of 1 / G by 2^(31 + s), 2^s the power of two at or above G, rounded up: it is off by less than
  // G of 2^(31 + s), so that x < 2^31 times it falls short of the next whole number
  int shift = 0;
  while ((1LL << shift) < a->G) ++shift;
  a->g_shift = shift ? shift - 1 : 0;
  a->g_mul = (unsigned)(((1ULL << (31 + shift)) + a->G - 1) / a->G);
  a->causal = d->causal != 0;
  a->q = a->kc = a->vc = nullptr;
  a->o = nullptr;
  a->lse = a->part = nullptr;
  a->qs = token_stride(d->q_stride, (long long)d->Hq * d->d, d->dtype);
  a->os = token_stride(d->out_stride, (long long)d->Hq * d->d, d->dtype);
  if (a->qs < 0 || a->os < 0 || a->qs * a->T_total >= kMostElements || a->os * a->T_total >= kMostElements)
    return KDA_ERR_SHAPE;
  return KDA_OK;
}

__global__ void validate_paged_kernel(PagedArgs a, int *flag) {
  int bad = 0;
  const int step = gridDim.x * blockDim.x, first = blockIdx.x * blockDim.x + threadIdx.x;
  for (int n = first; n <= a.N; n += step) {
    if (a.cu) {
      const int c = a.cu[n];
      if (n == 0 && c != 0) bad |= 1;
      if (c > a.T_total || (n > 0 && c < a.cu[n - 1])) bad |= 1;
    }
    if (n < a.N && (a.lens[n] < 0 || (long long)a.lens[n] > (long long)a.max_pages * a.page)) bad |= 2;
  }
  for (int n = blockIdx.x; n < a.N; n += gridDim.x) {
    const PagedSeq s = paged_seq(a, n);
    for (long long j = threadIdx.x; j < ((long long)s.kv + a.page - 1) / a.page; j += blockDim.x) {
      const int id = a.table[(long long)n * a.max_pages + j];
      if (id < 0 || id >= a.pages) bad |= 4;
    }
  }
  if (bad) atomicOr(flag, bad);
}

}  // namespace

cudaError_t launch_validate_paged(const PagedArgs &a, int *d_flag, cudaStream_t s) {
  validate_paged_kernel<<<256, 256, 0, s>>>(a, d_flag);
  return cudaGetLastError();
}

}  // namespace kda

using namespace kda;

kda_status kda_qk_rope_fwd(const kda_rope_desc *desc, const void *q, const void *k, const int32_t *positions,
                           const float *inv_freq, const float *q_weight, const float *k_weight, void *q_out,
                           void *k_out, kda_stream_t stream) {
  if (!desc || !q || !q_out || (desc->Hk > 0 && (!k || !k_out))) return KDA_ERR_NULL;
  RopeArgs a;
  kda_status st = check_rope(desc, positions, inv_freq, q_weight, k_weight, &a);
  if (st != KDA_OK) return st;
  Rows in[6], out[2];
  st = pair_rows(desc, q, k, desc->q_stride, desc->k_stride, &in[0], &in[1], &a.qs, &a.ks);
  if (st == KDA_OK)
    st = pair_rows(desc, q_out, k_out, desc->q_out_stride, desc->k_out_stride, &out[0], &out[1], &a.qos, &a.kos);
  if (st != KDA_OK) return st;
  in[2] = flat(positions, (size_t)desc->tokens * 4);
  in[3] = flat(inv_freq, (size_t)desc->rot * 2);
  in[4] = flat(q_weight, (size_t)desc->d * 4);
  in[5] = flat(k_weight, (size_t)desc->d * 4);
  const int same_in[] = {0, 1};
  if (aliased_rows(in, 6, out, 2, same_in)) return KDA_ERR_ALIAS;
  a.q = q;
  a.k = k;
  a.qo = q_out;
  a.ko = k_out;
  const cudaError_t e = launch_rope_fwd(a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KDA_OK : cuda_fail(e);
}

kda_status kda_qk_rope_bwd_workspace_size(const kda_rope_desc *desc, size_t *bytes) {
  if (!desc || !bytes) return KDA_ERR_NULL;
  *bytes = 0;
  const kda_status st = rope_sizes(desc);
  if (st != KDA_OK) return st;
  *bytes = rope_bwd_workspace_bytes(desc->tokens, desc->Hq, desc->Hk, desc->d);
  return KDA_OK;
}

kda_status kda_qk_rope_bwd(const kda_rope_desc *desc, const void *q, const void *k, const int32_t *positions,
                           const float *inv_freq, const float *q_weight, const float *k_weight,
                           const void *d_q_out, const void *d_k_out, void *dq, void *dk, float *dq_weight,
                           float *dk_weight, void *workspace, size_t workspace_bytes, kda_stream_t stream) {
  if (!desc || !d_q_out || !dq || (desc->Hk > 0 && (!d_k_out || !dk))) return KDA_ERR_NULL;
  if (desc->norm && (!q || (desc->Hk > 0 && !k))) return KDA_ERR_NULL;
  RopeArgs a;
  kda_status st = check_rope(desc, positions, inv_freq, q_weight, k_weight, &a);
  if (st != KDA_OK) return st;
  if ((dq_weight || dk_weight) && !a.norm) return KDA_ERR_UNSUPPORTED;
  Rows in[8], out[5];
  RopeBwdIo io{d_q_out, d_k_out, dq, dk, 0, 0, dq_weight, dk_weight};
  st = pair_rows(desc, q, k, desc->q_stride, desc->k_stride, &in[0], &in[1], &a.qs, &a.ks);
  if (st == KDA_OK)
    st = pair_rows(desc, d_q_out, d_k_out, desc->q_out_stride, desc->k_out_stride, &in[2], &in[3], &a.qos, &a.kos);
  if (st == KDA_OK) st = pair_rows(desc, dq, dk, desc->dq_stride, desc->dk_stride, &out[0], &out[1], &io.dqs, &io.dks);
  if (st != KDA_OK) return st;
  if (!aligned_to(dq_weight, 4) || !aligned_to(dk_weight, 4)) return KDA_ERR_ALIGN;
  if (!a.norm) in[0].n = in[1].n = 0;  // not read
  in[4] = flat(positions, (size_t)desc->tokens * 4);
  in[5] = flat(inv_freq, (size_t)desc->rot * 2);
  in[6] = flat(q_weight, (size_t)desc->d * 4);
  in[7] = flat(k_weight, (size_t)desc->d * 4);
  out[2] = flat(dq_weight, (size_t)desc->d * 4);
  out[3] = flat(dk_weight, (size_t)desc->d * 4);
  out[4] = flat(workspace, workspace ? workspace_bytes : 0);
  const int same_in[] = {2, 3, -1, -1, -1};
  if (aliased_rows(in, 8, out, 5, same_in)) return KDA_ERR_ALIAS;
  const size_t full = rope_bwd_workspace_bytes(a.tokens, a.Hq, a.Hk, a.d);
  if (workspace && workspace_bytes < full) return KDA_ERR_SHAPE;
  a.q = q;
  a.k = k;
  a.qo = a.ko = nullptr;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return with_workspace(workspace, workspace_bytes, dq_weight || dk_weight ? full : 0, s,
                        [&](void *ws) { return launch_rope_bwd(a, io, static_cast<float *>(ws), s); });
}

kda_status kda_kv_append(const kda_paged_desc *desc, const void *q, const void *k, const void *v,
                         const int32_t *lens, const int32_t *cu_seqlens, const int32_t *page_table,
                         const float *inv_freq, const float *q_weight, const float *k_weight, void *q_out,
                         void *k_cache, void *v_cache, kda_stream_t stream) {
  if (!k || !v || (q != nullptr) != (q_out != nullptr)) return KDA_ERR_NULL;
  PagedArgs p;
  kda_status st = check_paged(desc, lens, cu_seqlens, page_table, k_cache, v_cache, &p);
  if (st != KDA_OK) return st;
  RopeArgs a;
  st = check_turn(desc->rot, desc->layout, desc->rot_scale, desc->norm, desc->eps, desc->d, inv_freq, q_weight,
                  k_weight, &a);
  if (st != KDA_OK) return st;
  if (q_weight && !q) return KDA_ERR_UNSUPPORTED;
  const long long wq = (long long)p.Hq * p.d, wk = (long long)p.Hk * p.d, T = p.T_total;
  const long long vs = token_stride(desc->v_stride, wk, p.t);
  a.qs = token_stride(desc->q_stride, wq, p.t);
  a.ks = token_stride(desc->k_stride, wk, p.t);
  a.qos = token_stride(desc->out_stride, wq, p.t);
  a.kos = 0;
  if (a.qs < 0 || a.ks < 0 || a.qos < 0 || vs < 0 || a.qs * T >= kMostElements || a.ks * T >= kMostElements ||
      a.qos * T >= kMostElements || vs * T >= kMostElements)
    return KDA_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out)) return KDA_ERR_ALIGN;
  const size_t e = esize(p.t);
  const Rows in[] = {rows_of(q, T, wq, a.qs, e), rows_of(k, T, wk, a.ks, e), rows_of(v, T, wk, vs, e),
                     flat(lens, (size_t)p.N * 4), flat(cu_seqlens, cu_seqlens ? (size_t)(p.N + 1) * 4 : 0),
                     flat(page_table, (size_t)p.N * p.max_pages * 4), flat(inv_freq, (size_t)desc->rot * 2),
                     flat(q_weight, (size_t)p.d * 4), flat(k_weight, (size_t)p.d * 4)};
  const Rows out[] = {rows_of(q_out, T, wq, a.qos, e), cache_rows(p, k_cache), cache_rows(p, v_cache)};
  const int same_in[] = {0, -1, -1};
  if (aliased_rows(in, 9, out, 3, same_in)) return KDA_ERR_ALIAS;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  st = validate_paged(desc, p, s);
  if (st != KDA_OK) return st;
  a.tokens = p.T_total;
  a.Hq = p.Hq;
  a.Hk = p.Hk;
  a.t = p.t;
  a.positions = nullptr;
  a.q = q;
  a.k = k;
  a.qo = q_out;
  a.ko = nullptr;
  const cudaError_t err = launch_kv_append(a, p, v, vs, k_cache, v_cache, s);
  return err == cudaSuccess ? KDA_OK : cuda_fail(err);
}

kda_status kda_paged_attn_workspace_size(const kda_paged_desc *desc, size_t *bytes) {
  if (!desc || !bytes) return KDA_ERR_NULL;
  *bytes = 0;
  AttnArgs a;
  kda_status st = paged_sizes(desc, desc->num_seqs > 0, &a);
  if (st == KDA_OK) st = attn_args(desc, &a);
  if (st != KDA_OK) return st;
  *bytes = round256(attn_workspace_bytes(a));
  return KDA_OK;
}

kda_status kda_paged_attn(const kda_paged_desc *desc, const void *q, const void *k_cache, const void *v_cache,
                          const int32_t *lens, const int32_t *cu_seqlens, const int32_t *page_table, void *out,
                          float *lse, void *workspace, size_t workspace_bytes, kda_stream_t stream) {
  if (!q || !out) return KDA_ERR_NULL;
  AttnArgs a;
  kda_status st = check_paged(desc, lens, cu_seqlens, page_table, k_cache, v_cache, &a);
  if (st == KDA_OK) st = attn_args(desc, &a);
  if (st != KDA_OK) return st;
  if (!aligned16(q) || !aligned16(out) || !aligned_to(lse, 4)) return KDA_ERR_ALIGN;
  const long long wq = (long long)a.Hq * a.d, T = a.T_total;
  const size_t e = esize(a.t);
  const Rows in[] = {rows_of(q, T, wq, a.qs, e), cache_rows(a, k_cache), cache_rows(a, v_cache),
                     flat(lens, (size_t)a.N * 4), flat(cu_seqlens, cu_seqlens ? (size_t)(a.N + 1) * 4 : 0),
                     flat(page_table, (size_t)a.N * a.max_pages * 4)};
  const Rows outs[] = {rows_of(out, T, wq, a.os, e), flat(lse, lse ? (size_t)T * a.Hq * 4 : 0),
                       flat(workspace, workspace ? workspace_bytes : 0)};
  const int same_in[] = {-1, -1, -1};
  if (aliased_rows(in, 6, outs, 3, same_in)) return KDA_ERR_ALIAS;
  const size_t need = round256(attn_workspace_bytes(a));
  if (workspace && workspace_bytes < need) return KDA_ERR_SHAPE;
  if (workspace && !aligned16(workspace)) return KDA_ERR_ALIGN;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  st = validate_paged(desc, a, s);
  if (st != KDA_OK) return st;
  a.q = q;
  a.kc = k_cache;
  a.vc = v_cache;
  a.o = out;
  a.lse = lse;
  return with_workspace(workspace, workspace_bytes, a.T_total ? need : 0, s, [&](void *ws) {
    AttnArgs b = a;
    b.part = static_cast<float *>(ws);
    return launch_attn(b, s);
  });
}
