// tq_kv_shared.hip -- tq_kv_attn_shared: attention over the paged 8-bit
// key/value cache for groups of sequences that share their first pages.
//
// The rows of a group's sequences lie next to each other, so against the shared
// prefix they are the rows of one sequence, every one of which sees all of it: the
// kernels for one sequence's rows (tq_kv_attn_kernel.h) read it once for all of
// them.  A first launch takes the prefixes and leaves each row's output, maximum
// and sum in the workspace; a second one takes the sequences' own keys and joins
// the two, o = (2^(m1 - m) l1 o1 + 2^(m2 - m) l2 o2) / (2^(m1 - m) l1 + 2^(m2 - m) l2).
#include "tq_kv_attn_kernel.h"

namespace {

constexpr size_t kMidBytes = (size_t)1 << 27;  // of the prefixes' results at most

struct SharedPlan {
  bool shared;  // else one launch over all keys
  Plan prefix, own;
  size_t bytes;
};

SharedPlan make_shared_plan(int64_t rows, int64_t seqs, int64_t groups, int64_t q_heads, int64_t kv_heads,
                            int64_t head_dim, int64_t max_prefix, int64_t max_own) {
  SharedPlan P = {};
  const size_t mid = (size_t)(rows * q_heads * (head_dim + 2)) * 4;
  P.shared = max_prefix >= kPage && mid <= kMidBytes;
  if (!P.shared) {
    P.own = make_plan(rows, seqs, q_heads, kv_heads, head_dim, max_prefix + max_own);
    P.bytes = P.own.bytes;
    return P;
  }
  P.prefix = make_plan(rows, groups, q_heads, kv_heads, head_dim, max_prefix);
  P.own = make_plan(rows, seqs, q_heads, kv_heads, head_dim, max_own + kPage - 1);  // (with the prefix's last part of a page)
  P.bytes = P.prefix.bytes + P.own.bytes + mid;
  return P;
}

int check_lens(int64_t groups, int64_t max_prefix, int64_t max_own) {
  return groups < 1 || groups > ((int64_t)1 << 20) || max_prefix < 0 || max_own < 1 || max_prefix + max_own > 0x7fffffff - kPage
             ? TQ_ERR_SHAPE
             : TQ_OK;
}

}  // namespace

extern "C" size_t tq_kv_attn_shared_workspace_bytes(int64_t rows, int64_t seqs, int64_t groups, int64_t q_heads,
                                                    int64_t kv_heads, int64_t head_dim, int64_t max_prefix_len,
                                                    int64_t max_own_len) {
  if (shape_check(rows, seqs, q_heads, kv_heads, head_dim, 1, 1) != TQ_OK ||
      check_lens(groups, max_prefix_len, max_own_len) != TQ_OK)
    return 0;
  return make_shared_plan(rows, seqs, groups, q_heads, kv_heads, head_dim, max_prefix_len, max_own_len).bytes;
}

extern "C" int tq_kv_attn_shared(int64_t rows, int64_t seqs, int64_t groups, int64_t q_heads, int64_t kv_heads,
                                 int64_t head_dim, const void *q, int64_t q_stride, const int32_t *cu_rows,
                                 const int32_t *kv_len, const int32_t *cu_seqs, const int32_t *prefix_len,
                                 const int32_t *page_table, int64_t max_pages, const uint8_t *k_cache,
                                 const uint8_t *v_cache, const float *k_scale, const float *v_scale,
                                 int64_t num_pages, int64_t max_prefix_len, int64_t max_own_len, float softmax_scale,
                                 void *out, int64_t out_stride, void *ws, size_t ws_bytes, void *stream) {
  if (!q || !cu_rows || !kv_len || !cu_seqs || !prefix_len || !page_table || !k_cache || !v_cache || !k_scale ||
      !v_scale || !out)
    return TQ_ERR_NULL;
  int rc = shape_check(rows, seqs, q_heads, kv_heads, head_dim, max_pages, num_pages);
  if (rc == TQ_OK) rc = check_lens(groups, max_prefix_len, max_own_len);
  if (rc != TQ_OK) return rc;
  const int64_t width = q_heads * head_dim;
  if (q_stride < width || q_stride % 8 != 0 || q_stride > ((int64_t)1 << 31) || out_stride < width ||
      out_stride % 8 != 0 || out_stride > ((int64_t)1 << 31))
    return TQ_ERR_SHAPE;
  if (!(softmax_scale > 0.0f) || softmax_scale > 3.0e38f) return TQ_ERR_VALUE;
  if (!aligned_to(q, 16) || !aligned_to(out, 16) || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) ||
      !aligned_to(ws, 16) || !aligned_to(k_scale, 4) || !aligned_to(v_scale, 4) || !aligned_to(cu_rows, 4) ||
      !aligned_to(kv_len, 4) || !aligned_to(cu_seqs, 4) || !aligned_to(prefix_len, 4) || !aligned_to(page_table, 4))
    return TQ_ERR_ALIGN;
  const SharedPlan P =
      make_shared_plan(rows, seqs, groups, q_heads, kv_heads, head_dim, max_prefix_len, max_own_len);
  if (P.bytes && !ws) return TQ_ERR_NULL;
  if (ws_bytes < P.bytes) return TQ_ERR_SIZE;
  if (!P.shared)
    return tq_kv_attn(rows, seqs, q_heads, kv_heads, head_dim, q, q_stride, cu_rows, kv_len, page_table, max_pages, k_cache,
                      v_cache, k_scale, v_scale, num_pages, max_prefix_len + max_own_len, softmax_scale, 0, 0, out, out_stride,
                      ws, ws_bytes, stream);
  if (!plan_fits(P.own, rows, seqs, q_heads, kv_heads, max_pages) ||
      !plan_fits(P.prefix, rows, groups, q_heads, kv_heads, max_pages))
    return TQ_ERR_SHAPE;
  AttnArgs A = {};
  A.q = (const _Float16 *)q; A.out = (_Float16 *)out;
  A.cu = cu_rows; A.kv_len = kv_len; A.table = page_table;
  A.k = k_cache; A.v = v_cache; A.ks = k_scale; A.vs = v_scale;
  A.q_stride = q_stride; A.out_stride = out_stride; A.max_pages = max_pages; A.num_pages = num_pages;
  A.scale_log2 = softmax_scale * 1.4426950408889634f;
  A.rows = (int)rows; A.hkv = (int)kv_heads; A.group = (int)(q_heads / kv_heads);
  A.cu_seqs = cu_seqs; A.prefix = prefix_len; A.groups = (int)groups; A.all_seqs = (int)seqs;
  hipStream_t st = (hipStream_t)stream;
  char *p = (char *)ws;
  A.mid_o = (float *)(p + P.prefix.bytes + P.own.bytes);
  A.mid_ml = A.mid_o + rows * q_heads * head_dim;
  set_plan(A, P.prefix, groups, p);
  launch_attn<kPrefixKeys>(P.prefix, head_dim, A, st);
  set_plan(A, P.own, seqs, p + P.prefix.bytes);
  launch_attn<kOwnKeys>(P.own, head_dim, A, st);
  return hipGetLastError() == hipSuccess ? TQ_OK : TQ_ERR_HIP;
}
