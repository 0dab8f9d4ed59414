/* Calls kda_scan_fwd and kda_scan_bwd over and over without Python in between,
 * so that threads really overlap inside them.  Returns the first status that is
 * not 0. */
#include "kda.h"

typedef kda_status (*fwd_fn)(const kda_scan_desc *, const void *, const void *, const float *, float, const float *,
                             const int32_t *, void *, float *, float *, kda_stream_t);
typedef kda_status (*bwd_fn)(const kda_scan_desc *, const void *, const void *, const float *, float, const float *,
                             const int32_t *, const float *, const void *, const float *, void *, void *, float *, float *,
                             void *, size_t, kda_stream_t);

int hammer(fwd_fn fwd, bwd_fn bwd, const kda_scan_desc *desc, const void *x, const void *z, const float *A, const void *d_out,
           void *out, float *states, void *dx, void *dz, float *dA, void *workspace, size_t bytes, kda_stream_t stream, int n) {
  for (int i = 0; i < n; ++i) {
    kda_status s = fwd(desc, x, z, A, -5.0f, 0, 0, out, 0, states, stream);
    if (s == KDA_OK) s = bwd(desc, x, z, A, -5.0f, 0, 0, states, d_out, 0, dx, dz, dA, 0, workspace, bytes, stream);
    if (s != KDA_OK) return s;
  }
  return 0;
}

typedef kda_status (*chunk_fwd_fn)(const kda_chunk_desc *, const void *, const void *, const void *, const void *, const void *,
                                   const float *, const int32_t *, void *, float *, kda_stream_t);
typedef kda_status (*chunk_bwd_fn)(const kda_chunk_desc *, const void *, const void *, const void *, const void *, const void *,
                                   const float *, const int32_t *, const void *, const float *, float *, float *, float *,
                                   float *, float *, float *, void *, size_t, kda_stream_t);

/* The same with kda_chunk_fwd and kda_chunk_bwd. */
int hammer_chunk(chunk_fwd_fn fwd, chunk_bwd_fn bwd, const kda_chunk_desc *desc, const void *q, const void *k, const void *v,
                 const void *g, const void *beta, const void *d_out, void *out, float *dq, float *dk, float *dv, float *dg,
                 float *dbeta, void *workspace, size_t bytes, kda_stream_t stream, int n) {
  for (int i = 0; i < n; ++i) {
    kda_status s = fwd(desc, q, k, v, g, beta, 0, 0, out, 0, stream);
    if (s == KDA_OK)
      s = bwd(desc, q, k, v, g, beta, 0, 0, d_out, 0, dq, dk, dv, dg, dbeta, 0, workspace, bytes, stream);
    if (s != KDA_OK) return s;
  }
  return 0;
}
