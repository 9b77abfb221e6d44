// tq_kv_attn.hip -- tq_kv_attn: attention of new rows over the paged 8-bit
// key/value cache (its kernels: tq_kv_attn_kernel.h).
#include "tq_kv_attn_kernel.h"

extern "C" size_t tq_kv_attn_workspace_bytes(int64_t rows, int64_t seqs, int64_t q_heads, int64_t kv_heads,
                                             int64_t head_dim, int64_t max_kv_len) {
  if (shape_check(rows, seqs, q_heads, kv_heads, head_dim, 1, 1) != TQ_OK || max_kv_len < 1 ||
      max_kv_len > 0x7fffffff)
    return 0;
  return make_plan(rows, seqs, q_heads, kv_heads, head_dim, max_kv_len).bytes;
}

extern "C" int tq_kv_attn(int64_t rows, int64_t seqs, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                          const void *q, int64_t q_stride, const int32_t *cu_rows, const int32_t *kv_len,
                          const int32_t *page_table, int64_t max_pages, const uint8_t *k_cache,
                          const uint8_t *v_cache, const float *k_scale, const float *v_scale, int64_t num_pages,
                          int64_t max_kv_len, float softmax_scale, int64_t window, int64_t sinks, void *out,
                          int64_t out_stride, void *ws, size_t ws_bytes, void *stream) {
  if (!q || !cu_rows || !kv_len || !page_table || !k_cache || !v_cache || !k_scale || !v_scale || !out)
    return TQ_ERR_NULL;
  const int rc = shape_check(rows, seqs, q_heads, kv_heads, head_dim, max_pages, num_pages);
  if (rc != TQ_OK) return rc;
  const int64_t width = q_heads * head_dim;
  if (q_stride < width || q_stride % 8 != 0 || q_stride > ((int64_t)1 << 31) || out_stride < width ||
      out_stride % 8 != 0 || out_stride > ((int64_t)1 << 31) || max_kv_len < 1 || max_kv_len > 0x7fffffff)
    return TQ_ERR_SHAPE;
  if (window < 0 || window > 0x7fffffff || sinks < 0 || sinks > 0x7fffff00 || !(softmax_scale > 0.0f) ||
      softmax_scale > 3.0e38f)
    return TQ_ERR_VALUE;
  if (!aligned_to(q, 16) || !aligned_to(out, 16) || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) ||
      !aligned_to(ws, 16) || !aligned_to(k_scale, 4) || !aligned_to(v_scale, 4) || !aligned_to(cu_rows, 4) ||
      !aligned_to(kv_len, 4) || !aligned_to(page_table, 4))
    return TQ_ERR_ALIGN;
  const Plan P = make_plan(rows, seqs, q_heads, kv_heads, head_dim, max_kv_len);
  if (P.bytes && !ws) return TQ_ERR_NULL;
  if (ws_bytes < P.bytes) return TQ_ERR_SIZE;
  if (!plan_fits(P, rows, seqs, q_heads, kv_heads, max_pages)) return TQ_ERR_SHAPE;
  AttnArgs A = {};
  A.q = (const _Float16 *)q; A.out = (_Float16 *)out;
  A.cu = cu_rows; A.kv_len = kv_len; A.table = page_table;
  A.k = k_cache; A.v = v_cache; A.ks = k_scale; A.vs = v_scale;
  A.q_stride = q_stride; A.out_stride = out_stride; A.max_pages = max_pages; A.num_pages = num_pages;
  A.scale_log2 = softmax_scale * 1.4426950408889634f;
  A.rows = (int)rows; A.hkv = (int)kv_heads; A.group = (int)(q_heads / kv_heads);
  A.window = (int)window; A.sinks = (int)sinks;
  set_plan(A, P, seqs, (char *)ws);
  if (window && P.nsplit > 1) A.chunk = 4;  // a window leaves fewer pages than max_kv_len says
  launch_attn<kAllKeys>(P, head_dim, A, (hipStream_t)stream);
  return hipGetLastError() == hipSuccess ? TQ_OK : TQ_ERR_HIP;
}
