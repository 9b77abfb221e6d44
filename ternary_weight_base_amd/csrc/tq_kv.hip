// tq_kv.hip -- appending keys and values to the paged 8-bit cache with the
// position rotation on the way, and reading pages back.
//
// A cache byte b stands for (b - 127.5) * s with one scale s, a power of two,
// for each page of 64 tokens and KV head (keys and values apart): s is the
// smallest 2^e with max |x| < 128 s over the page's tokens, and
// b = floor(x / s) + 128, so the value is within s / 2 of x.  A later token
// that needs a larger scale shifts the codes that are there,
// c -> c >> log2(s_new / s_old) with c = b - 128: floor(floor(x / s) / 2^k) =
// floor(x / (2^k s)), so a page holds the same bytes however its tokens were
// cut into calls, and growing a scale never adds a second rounding error.
// (Round-to-nearest codes with an arbitrary scale would be rounded again at
// each growth.)
//
// The rotation of a pair (a, b) by its angle's (cos, sin) = (c, s) is
// (a c - b s, b c + a s): the products of two fp32 are exact in double, so
// one rounding of the double to fp32 is the only other one.
//
// Bound: memory, or launch latency for a few rows.  A prompt reads
// (q_heads + 2 kv_heads) head_dim values a row once and writes the rotated
// queries (fp16) and a byte per key and value element.  Workgroups: one per
// (page that receives rows, KV head, key or value), which holds the page's
// new rows in registers between its maximum and its codes, and after those
// the queries' workgroups of the same launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tq.h"
#include "tq_device.h"
#include "tq_kv.h"

namespace {

using namespace tqkv;

constexpr int kThreads = 256;
constexpr int kQuadsPerWg = 512;  // 4-element pieces of one row that a query workgroup rotates

struct AppendArgs {
  const void *qkv;
  const float *rope;
  const int *cu, *kv_len, *table;
  uint8_t *k, *v;
  float *ks, *vs;
  _Float16 *q_out;
  int64_t row_stride, max_pages, num_pages, rope_rows;
  int rows, seqs, hq, hkv, rot, pairs;
  int page_wgs, q_chunks;  // workgroups of the page part; query workgroups of a row
};

__device__ __forceinline__ f4 load4(const float *p) { return *reinterpret_cast<const f4 *>(p); }
__device__ __forceinline__ f4 load4(const _Float16 *p) {
  const h4 a = *reinterpret_cast<const h4 *>(p);
  return (f4){(float)a[0], (float)a[1], (float)a[2], (float)a[3]};
}

__device__ __forceinline__ float turn(float x, float c, float y, float s, bool plus) {
  const double p = (double)x * (double)c, q = (double)y * (double)s;  // both exact
  return tqdev::round_f32(plus ? p + q : p - q);
}

// Elements d..d+3 of the head vector at `head`, rotated.  t: the position's
// row of the table, rot / 2 cosines, then rot / 2 sines.
template <typename T>
__device__ __forceinline__ f4 load_rotated(const T *head, int d, const float *t, int rot, bool pairs) {
  const f4 x = load4(head + d);
  if (d >= rot) return x;
  const int h = rot >> 1;
  f4 r;
  if (pairs) {
    const float c0 = t[d >> 1], c1 = t[(d >> 1) + 1], s0 = t[h + (d >> 1)], s1 = t[h + (d >> 1) + 1];
    r[0] = turn(x[0], c0, x[1], s0, false);
    r[1] = turn(x[1], c0, x[0], s0, true);
    r[2] = turn(x[2], c1, x[3], s1, false);
    r[3] = turn(x[3], c1, x[2], s1, true);
    return r;
  }
  const bool hi = d >= h;
  const int a = hi ? d - h : d;
  const f4 y = load4(head + (hi ? d - h : d + h)), c = load4(t + a), s = load4(t + h + a);
#pragma unroll
  for (int i = 0; i < 4; i++) r[i] = turn(x[i], c[i], y[i], s[i], hi);
  return r;
}

// The four biased codes of w, shifted: c = b - 128, c >> k.
__device__ __forceinline__ uint32_t shift_codes(uint32_t w, int k) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int c = (int)((w >> (8 * i)) & 255u) - 128;
    r |= (uint32_t)((c >> k) + 128) << (8 * i);
  }
  return r;
}

// The exponent field of the smallest 2^e with m < 128 * 2^e (2^-126 at
// least, 2^121 at most), 0 for m = 0.
__device__ __forceinline__ int need_field(float m) {
  const uint32_t b = __float_as_uint(m);
  return b == 0 ? 0 : min(max((int)(b >> 23) - 6, 1), 248);
}

template <int D, typename T>
__global__ __launch_bounds__(kThreads) void append_kernel(const AppendArgs A) {
  constexpr int kQuads = D / 4, kRowsStep = kThreads / kQuads, kSteps = kPage / kRowsStep;
  const int tid = threadIdx.x;
  const T *qkv = (const T *)A.qkv;
  int blk = blockIdx.x;
  if (blk >= A.page_wgs) {  // queries: one row, kQuadsPerWg quads
    blk -= A.page_wgs;
    const int row = blk / A.q_chunks, chunk = blk % A.q_chunks;
    if (row >= cu_at(A.cu, A.seqs, A.rows)) return;
    const int s = find_seq<1, 0>(A.cu, A.seqs, A.rows, row, 1);
    const int64_t pos = (int64_t)A.kv_len[s] - (cu_at(A.cu, s + 1, A.rows) - row);
    const bool ok = pos >= 0 && (A.rot == 0 || pos < A.rope_rows);
    const float *t = A.rope + (ok ? pos : 0) * A.rot;
    const T *x = qkv + (int64_t)row * A.row_stride;
    _Float16 *o = A.q_out + (int64_t)row * A.hq * D;
    const int end = min((chunk + 1) * kQuadsPerWg, A.hq * kQuads);
    for (int i = chunk * kQuadsPerWg + tid; i < end; i += kThreads) {
      const int head = i / kQuads, d = (i % kQuads) * 4;
      f4 r = {0, 0, 0, 0};
      if (ok) r = load_rotated(x + head * D, d, t, A.rot, A.pairs);
      *reinterpret_cast<h4 *>(o + i * 4) = (h4){(_Float16)r[0], (_Float16)r[1], (_Float16)r[2], (_Float16)r[3]};
    }
    return;
  }
  const bool is_v = blk & 1;
  const int h = (blk >> 1) % A.hkv, slot = (blk >> 1) / A.hkv;
  const int s = find_seq<kPage, 2>(A.cu, A.seqs, A.rows, slot, 1);
  const int begin = cu_at(A.cu, s, A.rows), end = max(cu_at(A.cu, s + 1, A.rows), begin);
  const int local = slot - slot_base<kPage, 2>(begin, s, 1);
  const int64_t kvl = A.kv_len[s], p0 = kvl - (end - begin), first = p0 > 0 ? p0 : 0;
  const int64_t pg = first / kPage + local;
  if (local < 0 || pg >= A.max_pages) return;
  int64_t last = kvl;  // tokens at `last` and behind are not stored
  if (A.rot && last > A.rope_rows) last = A.rope_rows;
  const int64_t lo = first > pg * kPage ? first : pg * kPage;
  const int64_t hi = last < (pg + 1) * kPage ? last : (pg + 1) * kPage;
  if (lo >= hi) return;
  const int64_t id = A.table[(int64_t)s * A.max_pages + pg];
  if (id < 0 || id >= A.num_pages) return;
  const int a = (int)(lo - pg * kPage), m = (int)(hi - lo);  // slots a .. a + m - 1 receive rows
  const int64_t row0 = begin + (lo - p0), ph = id * A.hkv + h;
  float *scale = (is_v ? A.vs : A.ks) + ph;

  __shared__ float wmax[kThreads / 64];
  __shared__ uint32_t tile[D * (kPage / 4 + 1)];
  // the page's present scale: none if the page is new (or holds no power of two)
  const uint32_t ob = a > 0 ? __float_as_uint(*scale) : 0u;
  const int old_f = (ob & 0x807fffffu) == 0 && (ob >> 23) <= 248 ? (int)(ob >> 23) : 0;
  const int quad = tid % kQuads, r0 = tid / kQuads, d = quad * 4;
  const T *src = qkv + row0 * A.row_stride + (int64_t)(A.hq + (is_v ? A.hkv : 0) + h) * D;
  f4 x[kSteps];
  float mx = 0.0f;
#pragma unroll
  for (int i = 0; i < kSteps; i++) {
    const int r = i * kRowsStep + r0;
    x[i] = (f4){0, 0, 0, 0};
    if (r < m) {
      const T *p = src + r * A.row_stride;
      x[i] = is_v ? load4(p + d) : load_rotated(p, d, A.rope + (lo + r) * A.rot, A.rot, A.pairs);
    }
#pragma unroll
    for (int j = 0; j < 4; j++) mx = fmaxf(mx, fabsf(x[i][j]));
  }
  mx = tqdev::wave_max64(mx);
  if ((tid & 63) == 0) wmax[tid >> 6] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; w++) mx = fmaxf(mx, wmax[w]);
  const int f = max(need_field(mx), old_f);
  const int grow = old_f ? min(f - old_f, 8) : 0;
  if (tid == 0) *scale = __uint_as_float((uint32_t)f << 23);
  // 1 / s as a double; codes of a page of zeros are those of 0
  const double inv = f ? __longlong_as_double((long long)(1023 + 127 - f) << 52) : 0.0;

  uint32_t *page = reinterpret_cast<uint32_t *>((is_v ? A.v : A.k) + ph * (kPage * D));
  if (!is_v && grow)
    for (int i = tid; i < a * kQuads; i += kThreads) page[i] = shift_codes(page[i], grow);
#pragma unroll
  for (int i = 0; i < kSteps; i++) {
    const int r = i * kRowsStep + r0;
    if (r < m) {
      uint32_t w = 0;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        // in double: x / s must not be rounded before its floor is taken
        const double c = fmin(fmax(floor((double)x[i][j] * inv), -128.0), 127.0);
        const uint32_t b = (uint32_t)((int)c + 128);
        if (is_v)
          reinterpret_cast<uint8_t *>(tile)[(d + j) * (kPage + 4) + a + r] = (uint8_t)b;
        else
          w |= b << (8 * j);
      }
      if (!is_v) page[(a + r) * kQuads + quad] = w;
    }
  }
  if (!is_v) return;
  // values lie with their tokens side by side: whole words from the tile, words
  // that also hold other tokens merged with what is there
  __syncthreads();
  const int w0 = grow ? 0 : a >> 2, nw = ((a + m - 1) >> 2) - w0 + 1;
  for (int i = tid; i < D * nw; i += kThreads) {
    const int dim = i / nw, wd = w0 + i % nw, t0 = wd * 4;
    uint32_t w = tile[dim * (kPage / 4 + 1) + wd];
    if (t0 < a || t0 + 4 > a + m) {
      const uint32_t old = page[dim * (kPage / 4) + wd];
      const uint32_t moved = grow ? shift_codes(old, grow) : old;
      uint32_t mask_new = 0, mask_old = 0;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const int t = t0 + j;
        if (t >= a && t < a + m) mask_new |= 255u << (8 * j);
        if (t < a) mask_old |= 255u << (8 * j);
      }
      w = (w & mask_new) | (moved & mask_old) | (old & ~(mask_new | mask_old));
    }
    page[dim * (kPage / 4) + wd] = w;
  }
}

// values[2][n][heads][64][D] of the listed pages: keys, then values.
template <int D, typename T>
__global__ __launch_bounds__(kThreads) void read_kernel(const int *ids, int n, int hkv, int64_t num_pages,
                                                        const uint8_t *k, const uint8_t *v, const float *ks,
                                                        const float *vs, T *out) {
  constexpr int kWords = kPage * D / 4;
  __shared__ uint32_t tile[D * (kPage / 4 + 1)];
  const int tid = threadIdx.x;
  const bool is_v = (int)blockIdx.x >= n * hkv;
  const int b = blockIdx.x - (is_v ? n * hkv : 0), h = b % hkv;
  const int64_t id = ids[b / hkv];
  const bool ok = id >= 0 && id < num_pages;
  const int64_t ph = ok ? id * hkv + h : 0;
  const float s = ok ? (is_v ? vs : ks)[ph] : 0.0f;
  const uint32_t *page = reinterpret_cast<const uint32_t *>((is_v ? v : k) + ph * (kPage * D));
  T *o = out + (int64_t)blockIdx.x * (kPage * D);
  if (is_v) {
    for (int i = tid; i < kWords; i += kThreads)
      tile[(i / (kPage / 4)) * (kPage / 4 + 1) + i % (kPage / 4)] = page[i];
    __syncthreads();
  }
  for (int i = tid; i < kWords; i += kThreads) {
    const int t = i / (D / 4), d = (i % (D / 4)) * 4;
    const uint32_t w = is_v ? 0u : page[i];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const uint32_t c = is_v ? reinterpret_cast<const uint8_t *>(tile)[(d + j) * (kPage + 4) + t] : (w >> (8 * j)) & 255u;
      o[i * 4 + j] = ok ? (T)(((float)c - 127.5f) * s) : (T)0.0f;
    }
  }
}

bool aligned_to(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

}  // namespace

extern "C" int tq_kv_append(int dtype, int64_t rows, int64_t seqs, int64_t q_heads, int64_t kv_heads,
                            int64_t head_dim, const void *qkv, int64_t row_stride, const float *rope,
                            int64_t rope_rows, int64_t rot, int rope_mode, const int32_t *cu_rows,
                            const int32_t *kv_len, const int32_t *page_table, int64_t max_pages,
                            uint8_t *k_cache, uint8_t *v_cache, float *k_scale, float *v_scale,
                            int64_t num_pages, void *q_out, void *stream) {
  if (!qkv || !cu_rows || !kv_len || !page_table || !k_cache || !v_cache || !k_scale || !v_scale ||
      (!rope && rot != 0))
    return TQ_ERR_NULL;
  if (dtype != TQ_F16 && dtype != TQ_F32) return TQ_ERR_DTYPE;
  if (rope_mode != TQ_ROPE_HALVES && rope_mode != TQ_ROPE_PAIRS) return TQ_ERR_VALUE;
  const int rc = shape_check(rows, seqs, q_heads, kv_heads, head_dim, max_pages, num_pages);
  if (rc != TQ_OK) return rc;
  if (rot < 0 || rot > head_dim || rot % 8 != 0 || (rot && (rope_rows < 1 || rope_rows > ((int64_t)1 << 31))) ||
      row_stride < (q_heads + 2 * kv_heads) * head_dim || row_stride % 8 != 0 || row_stride > ((int64_t)1 << 31))
    return TQ_ERR_SHAPE;
  if (!aligned_to(qkv, 16) || !aligned_to(rope, 16) || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) ||
      !aligned_to(q_out, 16) || !aligned_to(k_scale, 4) || !aligned_to(v_scale, 4) || !aligned_to(cu_rows, 4) ||
      !aligned_to(kv_len, 4) || !aligned_to(page_table, 4))
    return TQ_ERR_ALIGN;
  AppendArgs A;
  A.qkv = qkv; A.rope = rope; A.cu = cu_rows; A.kv_len = kv_len; A.table = page_table;
  A.k = k_cache; A.v = v_cache; A.ks = k_scale; A.vs = v_scale; A.q_out = (_Float16 *)q_out;
  A.row_stride = row_stride; A.max_pages = max_pages; A.num_pages = num_pages; A.rope_rows = rope_rows;
  A.rows = (int)rows; A.seqs = (int)seqs; A.hq = (int)q_heads; A.hkv = (int)kv_heads; A.rot = (int)rot;
  A.pairs = rope_mode == TQ_ROPE_PAIRS;
  const int64_t slots = rows / kPage + 2 * seqs;
  A.q_chunks = (int)((q_heads * head_dim / 4 + kQuadsPerWg - 1) / kQuadsPerWg);
  const int64_t page_wgs = slots * kv_heads * 2, wgs = page_wgs + (q_out ? rows * A.q_chunks : 0);
  if (wgs > 0x7fffffff) return TQ_ERR_SHAPE;
  A.page_wgs = (int)page_wgs;
  const dim3 grid((unsigned)wgs), block(kThreads);
  hipStream_t st = (hipStream_t)stream;
#define TQ_APPEND(D, T) hipLaunchKernelGGL((append_kernel<D, T>), grid, block, 0, st, A)
  if (head_dim == 128) {
    if (dtype == TQ_F16) TQ_APPEND(128, _Float16); else TQ_APPEND(128, float);
  } else {
    if (dtype == TQ_F16) TQ_APPEND(64, _Float16); else TQ_APPEND(64, float);
  }
#undef TQ_APPEND
  return hipGetLastError() == hipSuccess ? TQ_OK : TQ_ERR_HIP;
}

extern "C" int tq_debug_kv_read(int dtype, int64_t n, int64_t kv_heads, int64_t head_dim, const int32_t *pages,
                                const uint8_t *k_cache, const uint8_t *v_cache, const float *k_scale,
                                const float *v_scale, int64_t num_pages, void *values, void *stream) {
  if (!pages || !k_cache || !v_cache || !k_scale || !v_scale || !values) return TQ_ERR_NULL;
  if (dtype != TQ_F16 && dtype != TQ_F32) return TQ_ERR_DTYPE;
  const int rc = shape_check(n, 1, kv_heads, kv_heads, head_dim, 1, num_pages);
  if (rc != TQ_OK) return rc;
  if (n * kv_heads > ((int64_t)1 << 29)) return TQ_ERR_SHAPE;
  if (!aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) || !aligned_to(k_scale, 4) || !aligned_to(v_scale, 4) ||
      !aligned_to(pages, 4) || !aligned_to(values, 16))
    return TQ_ERR_ALIGN;
  const dim3 grid((unsigned)(2 * n * kv_heads)), block(kThreads);
  hipStream_t st = (hipStream_t)stream;
#define TQ_READ(D, T)                                                                                         \
  hipLaunchKernelGGL((read_kernel<D, T>), grid, block, 0, st, pages, (int)n, (int)kv_heads, num_pages, k_cache, \
                     v_cache, k_scale, v_scale, (T *)values)
  if (head_dim == 128) {
    if (dtype == TQ_F16) TQ_READ(128, _Float16); else TQ_READ(128, float);
  } else {
    if (dtype == TQ_F16) TQ_READ(64, _Float16); else TQ_READ(64, float);
  }
#undef TQ_READ
  return hipGetLastError() == hipSuccess ? TQ_OK : TQ_ERR_HIP;
}
