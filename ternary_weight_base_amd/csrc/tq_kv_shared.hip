// tq_kv_shared.hip -- tq_kv_attn_shared: attention over the paged 8-bit
// key/value cache for groups of sequences that share their first pages.
//
// The rows of a group's sequences lie next to each other, so against the shared
// prefix they are the rows of one sequence, every one of which sees all of it: the
// kernels for one sequence's rows (tq_kv_attn_kernel.h) read it once for all of
// them.  A first launch takes the prefixes and leaves each row's output, maximum
// and sum in the workspace; a second one takes the sequences' own keys and joins
// the two, o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i.  Calls in which a prefix
// is read too few times to pay for that run as tq_kv_attn.
//
// Bound: the prefix by the matrix, vector and LDS pipes (as a prompt), own keys by
// HBM.  Measured, 64 query and 8 KV heads of 128: 64 tokens on up to 1001 own tokens
// behind 16384, 78 us, of them the prefix 49 (700 TFLOP/s) and the own keys, with 34
// MB of the prefix's pieces read and cleared, 28; read for each sequence it was 261.
#include "tq_kv_attn_kernel.h"

namespace {

constexpr size_t kMidBytes = (size_t)1 << 27;  // of the prefixes' results at most
// Workgroups of the prefix launch, two a CU, where its keys are cut (64 tokens behind
// 16384: 79 us, with one a CU 87, with three 90; 37 x 2 rows behind four prefixes 46, 59
// and 46), and pages of a piece at least.
constexpr int kPreFill = 2 * kCus, kPreLeast = 4;

struct SharedPlan {
  bool shared;  // else one launch over all keys
  Plan prefix, own;
  int64_t slots;    // of the prefix launch's tiles of 128 rows; 0: tiles of 16 or 32, results row by row
  int64_t mid_ml;
  size_t bytes;
};

// us that a tile of `tile_rows` rows takes for a page of 64 keys with all CUs at work
// on such tiles: from calls of 8 to 128 sequences on 2000 to 33000 tokens.
double page_us(int tile_rows, int64_t head_dim) {
  const bool wide = head_dim == 128;
  return tile_rows == kTileRows ? (wide ? 0.0047 : 0.0030) : tile_rows == 2 * kRows ? (wide ? 0.0026 : 0.0012) : (wide ? 0.0016 : 0.00105);
}
double tiles_us(int64_t rows, int64_t seqs, int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t keys, int tile_rows) {
  const int64_t each = (rows * (q_heads / kv_heads) + seqs - 1) / seqs, tiles = (each + tile_rows - 1) / tile_rows * seqs * kv_heads;
  return (double)(tiles * ((keys + kPage - 1) / kPage)) * page_us(tile_rows, head_dim);
}

SharedPlan make_shared_plan(int64_t rows, int64_t seqs, int64_t groups, int64_t q_heads, int64_t kv_heads,
                            int64_t head_dim, int64_t max_prefix, int64_t max_own) {
  SharedPlan P = {};
  const int64_t flat = rows * (q_heads / kv_heads), pages = max_prefix / kPage;
  const Plan all = make_plan(rows, seqs, q_heads, kv_heads, head_dim, max_prefix + max_own);
  P.bytes = all.bytes;
  if (pages == 0) return P;
  SharedPlan S = {};
  size_t mid;
  if (flat <= 2 * kRows * groups) {
    S.prefix = make_plan(rows, groups, q_heads, kv_heads, head_dim, max_prefix);
    S.mid_ml = rows * q_heads * head_dim;
    mid = (size_t)(rows * q_heads * (head_dim + 2)) * 4;
  } else {
    Plan &T = S.prefix;
    S.slots = flat / kTileRows + groups;
    const int64_t full = (flat + kTileRows - 1) / kTileRows, units = (full > groups ? full : groups) * kv_heads;
    const size_t piece = (size_t)partial_floats(kTileRows, (int)head_dim) * 4 * (size_t)(S.slots * kv_heads);
    int64_t n = kPreFill / units;
    if (n > kPrePieces) n = kPrePieces;
    if (n > pages / kPreLeast) n = pages / kPreLeast;
    if (n > (int64_t)(kMidBytes / piece)) n = (int64_t)(kMidBytes / piece);
    if (n < 1) n = 1;
    T.tile_rows = kTileRows;
    T.waves = kPreWaves;
    T.wgs = S.slots * kv_heads * n;
    T.nsplit = (int)n;
    T.chunk = (int)((pages + n - 1) / n);
    mid = piece * (size_t)n;
  }
  if (mid > kMidBytes) return P;
  S.own = make_plan(rows, seqs, q_heads, kv_heads, head_dim, max_own);
  // Own parts of a few pages in tiles of 16 rows, three workgroups of four waves a CU:
  // their end (the join with the prefix) is as long as their keys.  (64 x 4 rows, 300 own
  // tokens behind 2048: 64 against 90 us with tiles of 32; 64 x 1, 2000 behind 8192: 85
  // against 90 with cut units.)
  const int64_t own_pages = (max_own + kPage - 1) / kPage, own_units = (flat / kRows + seqs) * kv_heads;
  if (S.own.tile_rows != kTileRows && own_units > kCus &&
      own_pages <= (S.own.tile_rows == kRows ? 2 * kWhole : kWhole)) {
    S.own = Plan{};
    S.own.tile_rows = kRows;
    S.own.waves = 4;
    S.own.wgs = own_units;
    S.own.nsplit = 1;
    S.own.chunk = 0x7fffffff;
  }
  // Two launches where they should take less time: what a page takes a tile, what a
  // launch takes besides, and the prefix's results, written, read and cleared.  (8 x 1
  // rows, 300 behind 2048: 15.6 us in one, 23.2 in two; 4 x 1 behind 8192 18.7 and 38,
  // 16 x 1 38 and 36, 64 x 1 121 and 54, 64 x 1 behind 16384 261 and 78; 16 x 150,
  // 32 heads, 203 behind 4096, 205 and 225.  Of 22 calls around the border 17
  // take the faster way, four lose 5 to 10 % and one 16 %: 16 x 20, 32 heads, 200 behind
  // 4096, 65 in one against 56 in two, for 50 and 60 by the estimate.)
  const double one = 9.0 + tiles_us(rows, seqs, q_heads, kv_heads, head_dim, max_prefix + max_own, all.tile_rows);
  const double two = 24.0 + tiles_us(rows, groups < seqs ? groups : seqs, q_heads, kv_heads, head_dim, max_prefix, S.prefix.tile_rows) +
                     tiles_us(rows, seqs, q_heads, kv_heads, head_dim, max_own, S.own.tile_rows) + (double)mid * 2.0 / 8.5e6;
  if (one <= two) return P;
  S.shared = true;
  S.bytes = S.prefix.bytes + S.own.bytes + mid;
  return S;
}

int check_lens(int64_t groups, int64_t max_prefix, int64_t max_own) {
  // (each by itself first: their sum could pass 64 bits)
  return groups < 1 || groups > ((int64_t)1 << 20) || max_prefix < 0 || max_own < 1 || max_prefix > 0x7fffffff ||
                 max_own > 0x7fffffff || max_prefix + max_own > 0x7fffffff - kPage
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
  A.mid = (float *)(p + P.prefix.bytes + P.own.bytes);
  A.mid_ml = P.mid_ml;
  A.pre_slots = (int)P.slots;
  A.pre_nsplit = P.slots ? P.prefix.nsplit : 0;
  A.pre_chunk = P.prefix.chunk;
  set_plan(A, P.prefix, groups, p);
  launch_attn<kPrefixKeys>(P.prefix, head_dim, A, st);
  set_plan(A, P.own, seqs, p + P.prefix.bytes);
  launch_attn<kOwnKeys>(P.own, head_dim, A, st);
  return hipGetLastError() == hipSuccess ? TQ_OK : TQ_ERR_HIP;
}
