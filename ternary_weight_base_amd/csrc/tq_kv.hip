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
// queries (fp16) and a byte per key and value element.  A thread's piece is 8
// elements of a head that are rotated together: 4 and their 4 partners, or 8
// side by side.  Workgroups: one per (page that receives rows, KV head, key
// or value), and after those the queries' of the same launch.  For many rows
// (256 threads) a page's new rows stay in registers between its maximum and
// its codes, and the values turn through LDS; for a few rows a sequence (one
// wave) every lane still has a piece of a row, and values are merged into
// their words straight from the rows.
//
// Measured: three prompts of up to 2051 rows, 64 query and 8 KV heads of 128,
// fp32, 57 us, 5.0 TB/s (a large copy reaches 4.8); 64 sequences of one row, 32
// and 8 heads, fp16, 6.5 us; one row of 64 and 8 heads 4.3 us (latency); the
// prompts in fp16 43 us, 4.4 TB/s.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tq.h"
#include "tq_device.h"
#include "tq_kv.h"
#include "tq_wave.h"

namespace {

using namespace tqkv;

constexpr int kThreads = 256;

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
  int by_row;              // page workgroups are numbered by rows, not by slots (tq_kv.h)
};

__device__ __forceinline__ f4 load4(const float *p) { return *reinterpret_cast<const f4 *>(p); }
__device__ __forceinline__ f4 load4(const _Float16 *p) {
  const h4 a = *reinterpret_cast<const h4 *>(p);
  return (f4){(float)a[0], (float)a[1], (float)a[2], (float)a[3]};
}

// Piece i (of D / 8) of a head: two groups of 4 elements, at lo and hi.
// Rotated pairs i, i + rot / 2: 4 elements and their partners; else, and
// behind the rotated elements, 8 side by side.
struct Piece {
  int lo, hi;
  bool turned;
};
__device__ __forceinline__ Piece piece_at(int i, int rot, bool pairs) {
  Piece p;
  p.turned = 8 * i < rot;
  p.lo = p.turned && !pairs ? 4 * i : 8 * i;
  p.hi = p.turned && !pairs ? 4 * i + (rot >> 1) : 8 * i + 4;
  return p;
}

__device__ __forceinline__ float turn(float x, float c, float y, float s, bool plus) {
  const double p = (double)x * (double)c, q = (double)y * (double)s;  // both exact
  return tqdev::round_f32(plus ? p + q : p - q);
}

// Rotates a piece's 8 elements in place by c, s, the cosines and sines of
// its four pairs.
__device__ __forceinline__ void rotate(f4 &a, f4 &b, f4 c, f4 s, bool pairs) {
  if (pairs) {
    const f4 x = a, y = b;
#pragma unroll
    for (int i = 0; i < 2; i++) {
      a[2 * i] = turn(x[2 * i], c[i], x[2 * i + 1], s[i], false);
      a[2 * i + 1] = turn(x[2 * i + 1], c[i], x[2 * i], s[i], true);
      b[2 * i] = turn(y[2 * i], c[2 + i], y[2 * i + 1], s[2 + i], false);
      b[2 * i + 1] = turn(y[2 * i + 1], c[2 + i], y[2 * i], s[2 + i], true);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const float x = a[i], y = b[i];
    a[i] = turn(x, c[i], y, s[i], false);
    b[i] = turn(y, c[i], x, s[i], true);
  }
}

// A byte's code and the shift of earlier ones.
//
// x / s must not be rounded before its floor is taken: in double.
__device__ __forceinline__ uint32_t code(float x, double inv) {
  const double c = fmin(fmax(floor((double)x * inv), -128.0), 127.0);
  return (uint32_t)((int)c + 128);
}
__device__ __forceinline__ uint32_t codes4(f4 x, double inv) {
  return code(x[0], inv) | code(x[1], inv) << 8 | code(x[2], inv) << 16 | code(x[3], inv) << 24;
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

// Word `wd` (4 tokens) of a value row: the new codes in w where slots
// a .. a + m - 1 are, earlier tokens' from `old`, shifted, later bytes as they are.
__device__ __forceinline__ uint32_t merge_word(uint32_t w, uint32_t old, int wd, int a, int m, int grow) {
  const uint32_t moved = grow ? shift_codes(old, grow) : old;
  uint32_t mask_new = 0, mask_old = 0;
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const int t = 4 * wd + j;
    if (t >= a && t < a + m) mask_new |= 255u << (8 * j);
    if (t < a) mask_old |= 255u << (8 * j);
  }
  return (w & mask_new) | (moved & mask_old) | (old & ~(mask_new | mask_old));
}

// The rotated queries of one row: pieces chunk * NT * IT ..., IT a thread,
// whose loads are sent for before the row's position is known.
template <int D, typename T, int NT, int IT>
__device__ __forceinline__ void rotate_queries(const AppendArgs &A, int row, int chunk) {
  constexpr int kPieces = D / 8;
  const int total = A.hq * kPieces, i0 = chunk * (NT * IT) + threadIdx.x;
  const Piece p = piece_at(i0 % kPieces, A.rot, A.pairs);  // the same for each of a thread's: NT % kPieces = 0
  const T *x = (const T *)A.qkv + (int64_t)row * A.row_stride;
  f4 a[IT], b[IT];
#pragma unroll
  for (int k = 0; k < IT; k++) {
    const int head = min(i0 + k * NT, total - 1) / kPieces;
    a[k] = load4(x + head * D + p.lo);
    b[k] = load4(x + head * D + p.hi);
  }
  if (row >= cu_at(A.cu, A.seqs, A.rows)) return;
  const int s = find_seq<1, 0>(A.cu, A.seqs, A.rows, row, 1);
  const int64_t pos = (int64_t)A.kv_len[s] - (cu_at(A.cu, s + 1, A.rows) - row);
  const bool ok = pos >= 0 && (A.rot == 0 || pos < A.rope_rows);
  f4 c = {0, 0, 0, 0}, sn = c;
  if (ok && p.turned) {
    const float *t = A.rope + pos * A.rot + 4 * (i0 % kPieces);
    c = load4(t);
    sn = load4(t + (A.rot >> 1));
  }
  _Float16 *o = A.q_out + (int64_t)row * A.hq * D;
#pragma unroll
  for (int k = 0; k < IT; k++) {
    const int i = i0 + k * NT;
    if (i >= total) break;
    if (!ok) a[k] = b[k] = (f4){0, 0, 0, 0};
    else if (p.turned) rotate(a[k], b[k], c, sn, A.pairs);
    _Float16 *d = o + i / kPieces * D;
    *reinterpret_cast<h4 *>(d + p.lo) = (h4){(_Float16)a[k][0], (_Float16)a[k][1], (_Float16)a[k][2], (_Float16)a[k][3]};
    *reinterpret_cast<h4 *>(d + p.hi) = (h4){(_Float16)b[k][0], (_Float16)b[k][1], (_Float16)b[k][2], (_Float16)b[k][3]};
  }
}

// The rows that a page workgroup stores: row0 .. row0 + m - 1 at positions
// pos .. into slots a .. of a page (and KV head) ph.
struct Run {
  int64_t row0, pos, ph;
  int a, m;
};

__device__ __forceinline__ bool find_run(const AppendArgs &A, int unit, int h, Run &r) {
  int s, begin, end;
  int64_t kvl, p0, pg;
  if (A.by_row) {
    // the workgroup of a sequence's first row, or of the row at a page's start
    if (unit >= cu_at(A.cu, A.seqs, A.rows)) return false;
    s = find_seq<1, 0>(A.cu, A.seqs, A.rows, unit, 1);
    begin = cu_at(A.cu, s, A.rows);
    end = max(cu_at(A.cu, s + 1, A.rows), begin);
    kvl = A.kv_len[s];
    p0 = kvl - (end - begin);
    const int64_t pos = p0 + (unit - begin);
    if (unit < begin || unit >= end || pos < 0) return false;
    if (unit != begin && pos != 0 && pos % kPage != 0) return false;
    pg = pos / kPage;
  } else {
    s = find_seq<kPage, 2>(A.cu, A.seqs, A.rows, unit, 1);
    begin = cu_at(A.cu, s, A.rows);
    end = max(cu_at(A.cu, s + 1, A.rows), begin);
    const int local = unit - slot_base<kPage, 2>(begin, s, 1);
    kvl = A.kv_len[s];
    p0 = kvl - (end - begin);
    if (local < 0) return false;
    pg = (p0 > 0 ? p0 : 0) / kPage + local;
  }
  if (pg >= A.max_pages) return false;
  int64_t last = kvl;  // tokens at `last` and behind are not stored
  if (A.rot && last > A.rope_rows) last = A.rope_rows;
  const int64_t first = p0 > 0 ? p0 : 0;
  const int64_t lo = first > pg * kPage ? first : pg * kPage;
  const int64_t hi = last < (pg + 1) * kPage ? last : (pg + 1) * kPage;
  if (lo >= hi) return false;
  const int64_t id = A.table[(int64_t)s * A.max_pages + pg];
  if (id < 0 || id >= A.num_pages) return false;
  r.a = (int)(lo - pg * kPage);
  r.m = (int)(hi - lo);
  r.row0 = begin + (lo - p0);
  r.pos = lo;
  r.ph = id * A.hkv + h;
  return true;
}

// The exponent field of a page's present scale: 0 if the page is new (or
// holds no power of two).
__device__ __forceinline__ int present_field(const float *scale, int a) {
  const uint32_t b = a > 0 ? __float_as_uint(*scale) : 0u;
  return (b & 0x807fffffu) == 0 && (b >> 23) <= 248 ? (int)(b >> 23) : 0;
}
// 1 / s as a double; a page of zeros has the codes of 0
__device__ __forceinline__ double inverse_scale(int f) {
  return f ? __longlong_as_double((long long)(1023 + 127 - f) << 52) : 0.0;
}

template <int D, typename T>
__global__ __launch_bounds__(kThreads) void append_kernel(const AppendArgs A) {
  constexpr int kPieces = D / 8, kRowsStep = kThreads / kPieces, kSteps = kPage / kRowsStep, kIt = 4;
  const int tid = threadIdx.x, blk = blockIdx.x;
  if (blk >= A.page_wgs) {
    rotate_queries<D, T, kThreads, kIt>(A, (blk - A.page_wgs) / A.q_chunks, (blk - A.page_wgs) % A.q_chunks);
    return;
  }
  const bool is_v = blk & 1;
  const int h = (blk >> 1) % A.hkv;
  Run R;
  if (!find_run(A, (blk >> 1) / A.hkv, h, R)) return;
  float *scale = (is_v ? A.vs : A.ks) + R.ph;
  __shared__ float wmax[kThreads / 64];
  __shared__ uint32_t tile[D * (kPage / 4 + 1)];
  const int old_f = present_field(scale, R.a), i = tid % kPieces, r0 = tid / kPieces;
  const Piece p = piece_at(i, is_v ? 0 : A.rot, A.pairs);
  const T *src = (const T *)A.qkv + R.row0 * A.row_stride + (int64_t)(A.hq + (is_v ? A.hkv : 0) + h) * D;
  f4 x[kSteps][2];
  float mx = 0.0f;
#pragma unroll
  for (int k = 0; k < kSteps; k++) {
    const int r = k * kRowsStep + r0;
    x[k][0] = x[k][1] = (f4){0, 0, 0, 0};
    if (r < R.m) {
      x[k][0] = load4(src + r * A.row_stride + p.lo);
      x[k][1] = load4(src + r * A.row_stride + p.hi);
    }
  }
#pragma unroll
  for (int k = 0; k < kSteps; k++) {
    const int r = k * kRowsStep + r0;
    if (r < R.m && p.turned) {
      const float *t = A.rope + (R.pos + r) * A.rot + 4 * i;
      rotate(x[k][0], x[k][1], load4(t), load4(t + (A.rot >> 1)), A.pairs);
    }
#pragma unroll
    for (int j = 0; j < 8; j++) mx = fmaxf(mx, fabsf(x[k][j >> 2][j & 3]));
  }
  mx = tqdev::wave_max64(mx);
  if ((tid & 63) == 0) wmax[tid >> 6] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; w++) mx = fmaxf(mx, wmax[w]);
  const int f = max(need_field(mx), old_f);
  const int grow = old_f ? min(f - old_f, 8) : 0;
  if (tid == 0) *scale = __uint_as_float((uint32_t)f << 23);
  const double inv = inverse_scale(f);

  constexpr int kWords = D / 4;
  uint32_t *page = reinterpret_cast<uint32_t *>((is_v ? A.v : A.k) + R.ph * (kPage * D));
  if (!is_v && grow)
    for (int k = tid; k < R.a * kWords; k += kThreads) page[k] = shift_codes(page[k], grow);
#pragma unroll
  for (int k = 0; k < kSteps; k++) {
    const int r = k * kRowsStep + r0;
    if (r < R.m) {
      if (is_v) {
#pragma unroll
        for (int j = 0; j < 8; j++)
          reinterpret_cast<uint8_t *>(tile)[(8 * i + j) * (kPage + 4) + R.a + r] = (uint8_t)code(x[k][j >> 2][j & 3], inv);
      } else {
        page[(R.a + r) * kWords + p.lo / 4] = codes4(x[k][0], inv);
        page[(R.a + r) * kWords + p.hi / 4] = codes4(x[k][1], inv);
      }
    }
  }
  if (!is_v) return;
  // values lie with their tokens side by side: whole words from the tile, words
  // that also hold other tokens merged with what is there
  __syncthreads();
  const int w0 = grow ? 0 : R.a >> 2, nw = ((R.a + R.m - 1) >> 2) - w0 + 1;
  for (int k = tid; k < D * nw; k += kThreads) {
    const int dim = k / nw, wd = w0 + k % nw, at = dim * (kPage / 4) + wd;
    uint32_t w = tile[dim * (kPage / 4 + 1) + wd];
    if (4 * wd < R.a || 4 * wd + 4 > R.a + R.m) w = merge_word(w, page[at], wd, R.a, R.m, grow);
    page[at] = w;
  }
}

// The same for a few rows a sequence, one wave a workgroup (right for any
// number: rows beyond the first four of a page are read twice).
template <int D, typename T>
__global__ __launch_bounds__(64) void append_few_kernel(const AppendArgs A) {
  constexpr int kPieces = D / 8, kRowsStep = 64 / kPieces;
  const int lane = threadIdx.x, blk = blockIdx.x;
  if (blk >= A.page_wgs) {
    rotate_queries<D, T, 64, 1>(A, (blk - A.page_wgs) / A.q_chunks, (blk - A.page_wgs) % A.q_chunks);
    return;
  }
  const bool is_v = blk & 1;
  const int h = (blk >> 1) % A.hkv;
  Run R;
  if (!find_run(A, (blk >> 1) / A.hkv, h, R)) return;
  float *scale = (is_v ? A.vs : A.ks) + R.ph;
  const int old_f = present_field(scale, R.a), i = lane % kPieces, r0 = lane / kPieces;
  const Piece p = piece_at(i, is_v ? 0 : A.rot, A.pairs);
  const T *src = (const T *)A.qkv + R.row0 * A.row_stride + (int64_t)(A.hq + (is_v ? A.hkv : 0) + h) * D;
  auto fetch = [&](int r, f4 &a, f4 &b) {
    a = b = (f4){0, 0, 0, 0};
    if (r >= R.m) return;
    a = load4(src + r * A.row_stride + p.lo);
    b = load4(src + r * A.row_stride + p.hi);
    if (p.turned) {
      const float *t = A.rope + (R.pos + r) * A.rot + 4 * i;
      rotate(a, b, load4(t), load4(t + (A.rot >> 1)), A.pairs);
    }
  };
  f4 a0, b0;
  fetch(r0, a0, b0);
  float mx = 0.0f;
  auto widen = [&](f4 a, f4 b) {
#pragma unroll
    for (int j = 0; j < 4; j++) mx = fmaxf(mx, fmaxf(fabsf(a[j]), fabsf(b[j])));
  };
  widen(a0, b0);
  for (int r = kRowsStep; r < R.m; r += kRowsStep) {
    f4 a, b;
    fetch(r + r0, a, b);
    widen(a, b);
  }
  mx = tqdev::wave_max64(mx);
  const int f = max(need_field(mx), old_f);
  const int grow = old_f ? min(f - old_f, 8) : 0;
  if (lane == 0) *scale = __uint_as_float((uint32_t)f << 23);
  const double inv = inverse_scale(f);
  constexpr int kWords = D / 4;
  uint32_t *page = reinterpret_cast<uint32_t *>((is_v ? A.v : A.k) + R.ph * (kPage * D));
  if (is_v) {
    const int w0 = grow ? 0 : R.a >> 2, w1 = (R.a + R.m - 1) >> 2;
    for (int dim = lane; dim < D; dim += 64)
      for (int wd = w0; wd <= w1; wd++) {
        const uint32_t old = page[dim * (kPage / 4) + wd];
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const int r = 4 * wd + j - R.a;
          if (r >= 0 && r < R.m) w |= code((float)src[r * A.row_stride + dim], inv) << (8 * j);
        }
        page[dim * (kPage / 4) + wd] = merge_word(w, old, wd, R.a, R.m, grow);
      }
    return;
  }
  if (grow)
    for (int k = lane; k < R.a * kWords; k += 64) page[k] = shift_codes(page[k], grow);
  for (int r = 0; r < R.m; r += kRowsStep) {
    f4 a = a0, b = b0;
    if (r) fetch(r + r0, a, b);
    if (r + r0 < R.m) {
      page[(R.a + r + r0) * kWords + p.lo / 4] = codes4(a, inv);
      page[(R.a + r + r0) * kWords + p.hi / 4] = codes4(b, inv);
    }
  }
}

// values[2][n][heads][64][D] of the listed pages: keys, then values.  Bound:
// memory (77 pages of 8 heads to fp16, 30 MB, 8.9 us; one page 3.9 us, a launch).
template <int D, typename T>
__global__ __launch_bounds__(kThreads) void read_kernel(const int *ids, int n, int hkv, int64_t num_pages,
                                                        const uint8_t *k, const uint8_t *v, const float *ks,
                                                        const float *vs, T *out) {
  const int tid = threadIdx.x;
  const bool is_v = (int)blockIdx.x >= n * hkv;
  const int b = blockIdx.x - (is_v ? n * hkv : 0), h = b % hkv;
  const int64_t id = ids[b / hkv];
  const bool ok = id >= 0 && id < num_pages;
  const int64_t ph = ok ? id * hkv + h : 0;
  const float s = ok ? (is_v ? vs : ks)[ph] : 0.0f;
  const uint32_t *page = reinterpret_cast<const uint32_t *>((is_v ? v : k) + ph * (kPage * D));
  T *o = out + (int64_t)blockIdx.x * (kPage * D);
  typedef T T4 __attribute__((ext_vector_type(4)));
  auto put = [&](int token, int d, uint32_t w) {  // elements d .. d + 3 of a token
    T4 x;
#pragma unroll
    for (int j = 0; j < 4; j++) x[j] = ok ? (T)(((float)((w >> (8 * j)) & 255u) - 127.5f) * s) : (T)0.0f;
    *reinterpret_cast<T4 *>(o + token * D + d) = x;
  };
  // 4 tokens by 4 elements a thread and turn
  for (int i = tid; i < kPage * D / 16; i += kThreads) {
    const int d = i % (D / 4) * 4, t = i / (D / 4) * 4;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; j++) w[j] = is_v ? page[(d + j) * (kPage / 4) + t / 4] : page[(t + j) * (D / 4) + d / 4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      uint32_t x = w[j];
      if (is_v) {
        x = 0;
#pragma unroll
        for (int e = 0; e < 4; e++) x |= ((w[e] >> (8 * j)) & 255u) << (8 * e);
      }
      put(t + j, d, x);
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
  // a row's worth of lanes has work in a wave, not in 256 threads: one row a
  // sequence (64 of them: 14.1 against 14.4 us with a read-back; 1: 7.05, 7.2), or a
  // few in each of many (64 x 2: 15.2, 16.8; 64 x 4: 16.8, 17.5).  In fewer sequences
  // the wave's second trip costs more (8 x 4: 8.35, 7.75; 32 x 4: 13.3, 12.1)
  const bool few = rows <= seqs || (rows <= 4 * seqs && seqs >= 64);
  const int64_t slots = rows / kPage + 2 * seqs;
  A.by_row = rows < slots;
  const int64_t per_wg = few ? 64 : 4 * kThreads;
  A.q_chunks = (int)((q_heads * head_dim / 8 + per_wg - 1) / per_wg);
  const int64_t page_wgs = (A.by_row ? rows : slots) * kv_heads * 2, wgs = page_wgs + (q_out ? rows * A.q_chunks : 0);
  if (!grid_ok(wgs, few ? 64 : kThreads)) return TQ_ERR_SHAPE;
  A.page_wgs = (int)page_wgs;
  const dim3 grid((unsigned)wgs), block(few ? 64 : kThreads);
  hipStream_t st = (hipStream_t)stream;
#define TQ_APPEND(D, T)                                                     \
  {                                                                         \
    if (few) hipLaunchKernelGGL((append_few_kernel<D, T>), grid, block, 0, st, A); \
    else hipLaunchKernelGGL((append_kernel<D, T>), grid, block, 0, st, A);  \
  }
  if (head_dim == 128) {
    if (dtype == TQ_F16) TQ_APPEND(128, _Float16) else TQ_APPEND(128, float)
  } else {
    if (dtype == TQ_F16) TQ_APPEND(64, _Float16) else TQ_APPEND(64, float)
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
  if (!grid_ok(2 * n * kv_heads, kThreads)) return TQ_ERR_SHAPE;
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
