// tq_kv_attn.hip -- attention of new rows over the paged 8-bit key/value cache.
//
//   o[row][head] = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale * q . k_j),
// over the keys j <= the row's position that its window (or the sink tokens)
// leaves; keys and values are (b - 127.5) * s (tq_kv.hip).
//
// One pass over the keys with a running maximum and sum per query row.  A
// tile is one page, 64 tokens with one key scale and one value scale, so the
// scales never enter the matrix products: q . k = s_k (sum q c + sum q / 2)
// with c = b - 128 exact in fp16, the key scale joins the softmax factor, and
// the output accumulates c in units of a value scale (below).
//
// Products run on v_mfma_f32_16x16x32_f16.  Scores are made transposed,
// S^T = K Q^T: a lane then holds one query row and, with the tile's key rows
// handed to the four 16-row products in the order 16 (r / 4) + 4 t + r % 4,
// the 16 consecutive tokens 16 g .. 16 g + 15 (g = lane / 16).  That is the
// order in which the second product O^T = V^T P^T wants its weights (8
// consecutive tokens a lane and product) and in which 16 bytes of the
// token-fastest value page arrive, so weights go from one product into the
// next within a lane: no LDS, no lane exchange, and every softmax quantity is
// lane-local but for two exchanges of the running maximum.
//
// The weights are rounded to fp16 for the second product.  The decode kernel
// adds the rounding error back as a second fp16 term (its matrix units are
// idle anyway), so there only the output's own rounding to fp16 is left.
//
// Bound: few rows (decode) read 2 head_dim bytes a token and KV head and are
// bound by HBM; the work along the keys is split over workgroups, whose
// partial (max, sum, output) meet in the workspace, where the last one to
// arrive joins them in order.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tq.h"
#include "tq_kv.h"

namespace {

using namespace tqkv;

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kRows = 16;  // (token, query head) rows of a decode workgroup
constexpr float kNone = -1e30f;  // running maximum before the first visible key

struct AttnArgs {
  const _Float16 *q;
  _Float16 *out;
  const int *cu, *kv_len, *table;
  const uint8_t *k, *v;
  const float *ks, *vs;
  int64_t q_stride, out_stride, max_pages, num_pages;
  uint32_t *counters;
  float *partials;
  float scale_log2;
  int rows, seqs, hkv, group, window, sinks;
  int nsplit, chunk;  // splits of the keys at most; pages of a split at least
};

// The visible pages of a row tile whose positions are pmin .. pmax: pages
// with sinks, then from the page where the first row's window starts.  A
// position may lie behind the page table; such pages are not there.
struct Tiles {
  int sink, first, count;
  __device__ __forceinline__ int page(int i) const { return i < sink ? i : first + i - sink; }
};

__device__ __forceinline__ Tiles visible_tiles(int pmin, int pmax, int64_t max_pages, int window, int sinks) {
  Tiles t = {0, 0, 0};
  if (pmax < 0) return t;
  const int total = (int)min((int64_t)(pmax / kPage + 1), max_pages);
  if (window) {
    t.first = min(max(max(pmin, 0) - window + 1, 0) / kPage, total);
    t.sink = min(t.first, (sinks + kPage - 1) / kPage);
  }
  t.count = t.sink + total - t.first;
  return t;
}

__device__ __forceinline__ void store_dev(float *p, float v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float load_dev(const float *p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The bytes of one page and KV head that a lane takes part in.
template <int D>
struct Raw {
  uint4 k[4][D / 64], v[D / 16];
  float ks, vs;  // wave-uniform; ks < 0: no such page
};

template <int D>
__device__ __forceinline__ void load_tile(const AttnArgs &A, int s, int h, int pg, Raw<D> &t) {
  const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
  const int id = __builtin_amdgcn_readfirstlane(A.table[(int64_t)s * A.max_pages + pg]);
  const bool ok = id >= 0 && id < A.num_pages;
  const int64_t ph = (int64_t)(ok ? id : 0) * A.hkv + h;
  const uint8_t *kp = A.k + ph * (kPage * D), *vp = A.v + ph * (kPage * D);
  t.ks = ok ? A.ks[ph] : -1.0f;
  t.vs = A.vs[ph];
#pragma unroll
  for (int i = 0; i < 4; i++)
#pragma unroll
    for (int j = 0; j < D / 64; j++)
      t.k[i][j] = *reinterpret_cast<const uint4 *>(kp + (16 * (m >> 2) + 4 * i + (m & 3)) * D + 64 * j + 16 * g);
#pragma unroll
  for (int i = 0; i < D / 16; i++) t.v[i] = *reinterpret_cast<const uint4 *>(vp + (16 * i + m) * kPage + 16 * g);
}

// Running state of a lane's query row.  The output is held as
//   unit * (o + corr / 2), corr = sum of the weights that o's products took,
// where `unit` is a value scale: pages whose scale is within 2^4 of it have
// the ratio folded into their weights, others move the state to their own.
template <int D>
struct State {
  f4 o[D / 16];
  float m, l, corr, unit;
};

template <int D>
__device__ __forceinline__ void step(const AttnArgs &A, const Raw<D> &t, const h8 (&qf)[D / 32], float qsum, int pg,
                                     int pos, bool masked, State<D> &st) {
  const int g = (threadIdx.x & 63) >> 4;
  if (t.ks < 0.0f) return;  // wave-uniform
  float x[16];
  const float sc = t.ks * A.scale_log2;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    f4 acc = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < D / 64; j++) {
      const uint4 w = t.k[i][j];
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes8(w.x, w.y), qf[2 * j], acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes8(w.z, w.w), qf[2 * j + 1], acc, 0, 0, 0);
    }
#pragma unroll
    for (int r = 0; r < 4; r++) x[4 * i + r] = (acc[r] + qsum) * sc;
  }
  if (masked) {
    const int j0 = pg * kPage + 16 * g;
#pragma unroll
    for (int i = 0; i < 16; i++) {
      const int j = j0 + i;
      const bool see = j <= pos && (A.window == 0 || j > pos - A.window || j < A.sinks);
      x[i] = see ? x[i] : -__builtin_inff();
    }
  }
  float mx = x[0];
#pragma unroll
  for (int i = 1; i < 16; i++) mx = fmaxf(mx, x[i]);
  mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
  mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
  float shift = 0.0f;  // log2 of this page's value scale over the unit
  float alpha = 1.0f;
  const float m_new = fmaxf(st.m, mx);
  alpha = __builtin_amdgcn_exp2f(st.m - m_new);
  st.m = m_new;
  st.l *= alpha;
  const bool has_v = t.vs > 0.0f;  // a page of zeros adds to the sum only
  if (has_v) {
    const float ratio = t.vs / st.unit;
    if (!(ratio > 0.0625f && ratio < 16.0f)) {
      alpha *= fminf(st.unit / t.vs, 3.0e38f);
      st.unit = t.vs;
    } else {
      shift = __builtin_amdgcn_logf(ratio);
    }
  }
  st.corr *= alpha;
#pragma unroll
  for (int i = 0; i < D / 16; i++) st.o[i] *= alpha;
  float sum = 0.0f;
  h8 p[2], e[2];
#pragma unroll
  for (int i = 0; i < 16; i++) {
    const float w = __builtin_amdgcn_exp2f(x[i] - m_new + shift);
    sum += w;
    const _Float16 r = (_Float16)w;
    p[i >> 3][i & 7] = r;
    e[i >> 3][i & 7] = (_Float16)(w - (float)r);
  }
  st.l += sum * __builtin_amdgcn_exp2f(-shift);
  if (!has_v) return;
  st.corr += sum;
#pragma unroll
  for (int i = 0; i < D / 16; i++) {
    const uint4 w = t.v[i];
    const h8 a = codes8(w.x, w.y), b = codes8(w.z, w.w);
    st.o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, p[0], st.o[i], 0, 0, 0);
    st.o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b, p[1], st.o[i], 0, 0, 0);
    st.o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, e[0], st.o[i], 0, 0, 0);
    st.o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b, e[1], st.o[i], 0, 0, 0);
  }
}

// Floats of one split's partial result: outputs, then (max, sum) per row.
constexpr int partial_floats(int D) { return kRows * (D + 2); }

template <int D>
__global__ __launch_bounds__(kThreads, 2) void decode_kernel(const AttnArgs A) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n16 = lane & 15, g = lane >> 4;
  const int h = blockIdx.x % A.hkv, c = blockIdx.x / A.hkv % A.nsplit, slot = blockIdx.x / A.hkv / A.nsplit;
  const int s = find_seq(A.cu, A.seqs, A.rows, slot, A.group, kRows, 1);
  const int begin = cu_at(A.cu, s, A.rows), n = max(cu_at(A.cu, s + 1, A.rows) - begin, 0);
  const int64_t f0 = (slot - slot_base(A.cu, s, A.rows, A.group, kRows, 1)) * kRows;
  if (f0 < 0 || f0 >= (int64_t)n * A.group) return;
  const int nrows = (int)min((int64_t)kRows, (int64_t)n * A.group - f0);
  const int tok0 = (int)(f0 / A.group), tokl = (int)((f0 + nrows - 1) / A.group);
  const int p0 = max(A.kv_len[s], 0) - n;  // may be negative: such rows see nothing
  const int pmin = p0 + tok0, pmax = p0 + tokl;
  const Tiles T = visible_tiles(pmin, pmax, A.max_pages, A.window, A.sinks);
  const int per = max(A.chunk, (T.count + A.nsplit - 1) / A.nsplit);
  const int splits = max((T.count + per - 1) / per, 1);
  if (c >= splits) return;

  const int64_t fl = f0 + n16;
  const bool valid = n16 < nrows;
  const int tok = (int)(fl / A.group), head = h * A.group + (int)(fl % A.group);
  const int pos = valid ? p0 + tok : -1;
  const _Float16 *qr = A.q + (int64_t)(begin + (valid ? tok : 0)) * A.q_stride + (valid ? head : 0) * D;
  h8 qf[D / 32];
  float qsum = 0.0f;
#pragma unroll
  for (int j = 0; j < D / 64; j++)
#pragma unroll
    for (int u = 0; u < 2; u++) {
      h8 x = *reinterpret_cast<const h8 *>(qr + 64 * j + 16 * g + 8 * u);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        x[i] = valid ? x[i] : (_Float16)0.0f;
        qsum += (float)x[i];
      }
      qf[2 * j + u] = x;
    }
  qsum += __shfl_xor(qsum, 16, 64);
  qsum += __shfl_xor(qsum, 32, 64);
  qsum *= 0.5f;

  State<D> st;
#pragma unroll
  for (int i = 0; i < D / 16; i++) st.o[i] = (f4){0, 0, 0, 0};
  st.m = kNone;
  st.l = st.corr = 0.0f;
  st.unit = 1.0f;
  const int end = min(T.count, (c + 1) * per);
  Raw<D> raw[2];
  int i = c * per + wave;
  auto run = [&](const Raw<D> &t, int ti) {
    const int pg = T.page(ti), j1 = pg * kPage + kPage - 1;
    const bool all = j1 <= pmin && (A.window == 0 || pg * kPage > pmax - A.window || j1 < A.sinks);
    step<D>(A, t, qf, qsum, pg, pos, !all, st);
  };
  if (i < end) load_tile<D>(A, s, h, T.page(i), raw[0]);
  while (i < end) {
    if (i + kWaves < end) load_tile<D>(A, s, h, T.page(i + kWaves), raw[1]);
    run(raw[0], i);
    i += kWaves;
    if (i >= end) break;
    if (i + kWaves < end) load_tile<D>(A, s, h, T.page(i + kWaves), raw[0]);
    run(raw[1], i);
    i += kWaves;
  }

  // the waves' results meet in LDS
  constexpr int kStride = D + 4;
  __shared__ float so[kWaves][kRows][kStride];
  __shared__ float sm[kWaves][kRows], sl[kWaves][kRows];
  st.l += __shfl_xor(st.l, 16, 64);
  st.l += __shfl_xor(st.l, 32, 64);
  st.corr += __shfl_xor(st.corr, 16, 64);
  st.corr += __shfl_xor(st.corr, 32, 64);
#pragma unroll
  for (int d = 0; d < D / 16; d++) {
    f4 o;
#pragma unroll
    for (int r = 0; r < 4; r++) o[r] = (st.o[d][r] + 0.5f * st.corr) * st.unit;
    *reinterpret_cast<f4 *>(&so[wave][n16][16 * d + 4 * g]) = o;
  }
  if (g == 0) {
    sm[wave][n16] = st.m;
    sl[wave][n16] = st.l;
  }
  __syncthreads();
  constexpr int kPer = D / 16;  // outputs of a thread: row tid / 16
  const int row = tid >> 4, d0 = (tid & 15) * kPer;
  float M = kNone, L = 0.0f, o[kPer];
#pragma unroll
  for (int w = 0; w < kWaves; w++) M = fmaxf(M, sm[w][row]);
#pragma unroll
  for (int j = 0; j < kPer; j++) o[j] = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; w++) {
    const float f = __builtin_amdgcn_exp2f(sm[w][row] - M);
    L += f * sl[w][row];
#pragma unroll
    for (int j = 0; j < kPer; j++) o[j] += f * so[w][row][d0 + j];
  }

  if (splits > 1) {
    __shared__ int last;
    const int64_t tile = (int64_t)slot * A.hkv + h;
    float *base = A.partials + tile * A.nsplit * partial_floats(D);
    float *mine = base + (int64_t)c * partial_floats(D);
    if (row < nrows) {
#pragma unroll
      for (int j = 0; j < kPer; j++) store_dev(mine + row * D + d0 + j, o[j]);
      if ((tid & 15) == 0) {
        store_dev(mine + kRows * D + 2 * row, M);
        store_dev(mine + kRows * D + 2 * row + 1, L);
      }
    }
    __builtin_amdgcn_s_waitcnt(0);  // this thread's words have reached device scope
    __syncthreads();                // ... and so have every other thread's
    if (tid == 0)
      last = __hip_atomic_fetch_add(&A.counters[tile], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
             (uint32_t)(splits - 1);
    __syncthreads();
    if (!last) return;  // another split finishes this tile
    M = kNone;
    L = 0.0f;
#pragma unroll
    for (int j = 0; j < kPer; j++) o[j] = 0.0f;
    if (row < nrows) {
      for (int k = 0; k < splits; k++) {
        float *p = base + (int64_t)k * partial_floats(D);
        const float mk = load_dev(p + kRows * D + 2 * row), lk = load_dev(p + kRows * D + 2 * row + 1);
        const float mn = fmaxf(M, mk), fa = __builtin_amdgcn_exp2f(M - mn), fb = __builtin_amdgcn_exp2f(mk - mn);
        M = mn;
        L = L * fa + lk * fb;
#pragma unroll
        for (int j = 0; j < kPer; j++) o[j] = o[j] * fa + load_dev(p + row * D + d0 + j) * fb;
      }
      // consumed: leave the workspace zero for the next call, whatever its shape
      for (int k = 0; k < splits; k++) {
        float *p = base + (int64_t)k * partial_floats(D);
#pragma unroll
        for (int j = 0; j < kPer; j++) store_dev(p + row * D + d0 + j, 0.0f);
      }
    }
    __syncthreads();  // every thread of the row has read its maximum and sum
    if (row < nrows && (tid & 15) == 0)
      for (int k = 0; k < splits; k++) {
        float *p = base + (int64_t)k * partial_floats(D) + kRows * D + 2 * row;
        store_dev(p, 0.0f);
        store_dev(p + 1, 0.0f);
      }
    if (tid == 0) __hip_atomic_store(&A.counters[tile], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (row < nrows) {
    const int64_t f = f0 + row;
    _Float16 *dst = A.out + (int64_t)(begin + f / A.group) * A.out_stride + (h * A.group + f % A.group) * D + d0;
    const float r = L > 0.0f || L != L ? 1.0f / L : 0.0f;  // no visible key: zeros
#pragma unroll
    for (int j = 0; j < kPer; j++) dst[j] = (_Float16)(o[j] * r);
  }
}

// The launch of a call: how the keys are split, and the workspace it needs.
struct Plan {
  int64_t slots;
  int nsplit, chunk;
  size_t counter_bytes, bytes;
};

constexpr int kTargetWgs = 512;  // two workgroups a CU
constexpr int kMinChunk = 4, kMaxChunk = 32;

Plan make_plan(int64_t rows, int64_t seqs, int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t max_kv) {
  Plan P;
  const int64_t group = q_heads / kv_heads;
  P.slots = rows * group / kRows + seqs;
  const int64_t tiles = (max_kv + kPage - 1) / kPage;
  const int64_t full = (rows * group + kRows - 1) / kRows, units = (full > seqs ? full : seqs) * kv_heads;
  int64_t chunk = (tiles * units + kTargetWgs - 1) / kTargetWgs;
  if (chunk < kMinChunk) chunk = kMinChunk;
  if (full <= 4 * seqs && chunk > kMaxChunk) chunk = kMaxChunk;
  int64_t nsplit = (tiles + chunk - 1) / chunk;
  if (nsplit < 1) nsplit = 1;
  P.chunk = (int)(chunk < 0x7fffffff ? chunk : 0x7fffffff);
  P.nsplit = (int)nsplit;
  P.counter_bytes = 0;
  P.bytes = 0;
  if (nsplit > 1) {
    P.counter_bytes = ((size_t)P.slots * kv_heads * 4 + 15) / 16 * 16;
    P.bytes = P.counter_bytes + (size_t)P.slots * kv_heads * nsplit * partial_floats((int)head_dim) * 4;
  }
  return P;
}

bool aligned_to(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

}  // namespace

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
  const int64_t wgs = P.slots * kv_heads * P.nsplit;
  if (wgs > 0x7fffffff) return TQ_ERR_SHAPE;
  AttnArgs A;
  A.q = (const _Float16 *)q; A.out = (_Float16 *)out;
  A.cu = cu_rows; A.kv_len = kv_len; A.table = page_table;
  A.k = k_cache; A.v = v_cache; A.ks = k_scale; A.vs = v_scale;
  A.q_stride = q_stride; A.out_stride = out_stride; A.max_pages = max_pages; A.num_pages = num_pages;
  A.counters = (uint32_t *)ws;
  A.partials = (float *)((char *)ws + P.counter_bytes);
  A.scale_log2 = softmax_scale * 1.4426950408889634f;
  A.rows = (int)rows; A.seqs = (int)seqs; A.hkv = (int)kv_heads; A.group = (int)(q_heads / kv_heads);
  A.window = (int)window; A.sinks = (int)sinks;
  A.nsplit = P.nsplit; A.chunk = P.chunk;
  const dim3 grid((unsigned)wgs), block(kThreads);
  if (head_dim == 128)
    hipLaunchKernelGGL(decode_kernel<128>, grid, block, 0, (hipStream_t)stream, A);
  else
    hipLaunchKernelGGL(decode_kernel<64>, grid, block, 0, (hipStream_t)stream, A);
  return hipGetLastError() == hipSuccess ? TQ_OK : TQ_ERR_HIP;
}
