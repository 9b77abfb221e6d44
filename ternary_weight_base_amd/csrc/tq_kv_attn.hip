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

typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

constexpr int kRows = 16;  // (token, query head) rows of a decode workgroup
constexpr int kDecThreads = 512, kDecWaves = kDecThreads / 64;
constexpr int kDecSplits = 128;  // splits of the keys at most, decode
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

// 16-byte accesses at device scope (past the XCD's own cache, as other XCDs'
// workgroups read and write these words).
typedef __amdgpu_buffer_rsrc_t Rsrc;
constexpr int kDevScope = 16;  // the sc1 bit of the cache policy
__device__ __forceinline__ Rsrc make_rsrc(void *p) { return __builtin_amdgcn_make_buffer_rsrc(p, 0, 0x7fffffff, 0x00027000); }
__device__ __forceinline__ void store_dev(Rsrc r, int i, f4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, v), r, i * 4, 0, kDevScope);
}
__device__ __forceinline__ f4 load_dev(Rsrc r, int i) {
  return __builtin_bit_cast(f4, __builtin_amdgcn_raw_buffer_load_b128(r, i * 4, 0, kDevScope));
}
__device__ __forceinline__ void store_dev2(Rsrc r, int i, float a, float b) {
  __builtin_amdgcn_raw_buffer_store_b64((u2){__float_as_uint(a), __float_as_uint(b)}, r, i * 4, 0, kDevScope);
}
__device__ __forceinline__ void load_dev2(Rsrc r, int i, float &a, float &b) {
  const u2 v = __builtin_amdgcn_raw_buffer_load_b64(r, i * 4, 0, kDevScope);
  a = __uint_as_float(v[0]);
  b = __uint_as_float(v[1]);
}

// The larger of a lane's value and its partner's in the other half of the wave.
__device__ __forceinline__ float half_max(float v) {
  const uint32_t b = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float v) {
  const uint32_t b = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Over the four lanes lane % 16 + 16 g.
__device__ __forceinline__ float quarter_max(float v) {
  const uint32_t b = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  return half_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float quarter_sum(float v) {
  const uint32_t b = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  return half_sum(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// The bytes of one page and KV head that a lane takes part in.
template <int D>
struct Raw {
  uint4 k[4][D / 64], v[D / 16];
  float ks, vs;  // wave-uniform; ks < 0: no such page
};

template <int D>
__device__ __forceinline__ void load_tile(const AttnArgs &A, int h, int id, Raw<D> &t) {
  const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
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
  mx = quarter_max(mx);
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

// Floats of one split's partial result for R rows: outputs, then (max, sum)
// of each row.
constexpr int partial_floats(int R, int D) { return R * (D + 2); }

// After a workgroup has stored its split's partial result (store_dev) at
// `base` + c * partial_floats: whether it is the last of `splits`, in which
// case it leaves the counter zero for the next call.
__device__ __forceinline__ bool last_split(uint32_t *counter, int splits) {
  __shared__ int last;
  __builtin_amdgcn_s_waitcnt(0);  // this thread's words have reached device scope
  __syncthreads();                // ... and so have every other thread's
  if (threadIdx.x == 0) {
    last = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)(splits - 1);
    if (last) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  return last;
}

// 1 / sum of weights; 0 for a row that saw no key.
__device__ __forceinline__ float inverse(float l) { return l > 0.0f || l != l ? 1.0f / l : 0.0f; }

// The last split's join of a tile: the partial results at `part`, summed in
// the order of the splits; `out(row, d, f4)` takes the outputs.  First every
// split's weight per row, then the outputs, 16 bytes a thread, several
// splits' loads in flight; where the rows are fewer than the threads, the
// splits are dealt over `parts` groups of threads that meet in LDS.  The
// words read are left zero for the next call, whatever its shape.
template <int R, int D, int NT, int MAXS, typename Out>
__device__ __forceinline__ void join(Rsrc part, int splits, int nrows, float *lds, const Out &out) {
  constexpr int PF = partial_floats(R, D), kBatch = 8;
  const int tid = threadIdx.x;
  float *wm = lds, *wl = lds + R * MAXS;
  for (int i = tid; i < splits * R; i += NT) {
    const int k = i / R, r = i % R;
    float m = kNone, l = 0.0f;
    if (r < nrows) {
      load_dev2(part, k * PF + R * D + 2 * r, m, l);
      store_dev2(part, k * PF + R * D + 2 * r, 0.0f, 0.0f);
    }
    wm[i] = m;
    wl[i] = l;
  }
  __syncthreads();
  if (tid < R) {
    float M = kNone, L = 0.0f;
    for (int k = 0; k < splits; k++) M = fmaxf(M, wm[k * R + tid]);
    for (int k = 0; k < splits; k++) L += wl[k * R + tid] * __builtin_amdgcn_exp2f(wm[k * R + tid] - M);
    const float inv = inverse(L);
    for (int k = 0; k < splits; k++) wm[k * R + tid] = inv * __builtin_amdgcn_exp2f(wm[k * R + tid] - M);
  }
  __syncthreads();
  const int quads = nrows * (D / 4);
  const int parts = quads * 4 <= NT ? 4 : quads * 2 <= NT ? 2 : 1;
  const int per = NT / parts, p = tid / per;
  f4 *red = reinterpret_cast<f4 *>(lds + 2 * R * MAXS);
  for (int q = tid - p * per; q < quads; q += per) {  // one round where parts > 1
    const int row = q / (D / 4), w = q * 4;
    f4 o = {0, 0, 0, 0};
    for (int k0 = p; k0 < splits; k0 += kBatch * parts) {
      f4 v[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; b++) v[b] = load_dev(part, min(k0 + b * parts, splits - 1) * PF + w);
#pragma unroll
      for (int b = 0; b < kBatch; b++)
        if (k0 + b * parts < splits) o += v[b] * wm[(k0 + b * parts) * R + row];
    }
    for (int k = p; k < splits; k += parts) store_dev(part, k * PF + w, (f4){0, 0, 0, 0});
    if (parts == 1)
      out(row, w - row * D, o);
    else
      red[tid] = o;
  }
  if (parts == 1) return;
  __syncthreads();
  if (tid < quads) {
    f4 o = red[tid];
    for (int k = 1; k < parts; k++) o += red[k * per + tid];
    out(tid / (D / 4), tid * 4 % D, o);
  }
}
template <int R, int MAXS, int NT>
constexpr int kJoinFloats = 2 * R * MAXS + 4 * NT;

// A workgroup's place: R consecutive (token, query head) rows of a sequence
// and KV head, and its share of their pages.
struct Place {
  int h, s, begin, n, nrows, f0, p0, pmin, pmax, lo, hi, splits, split;
  int64_t tile;
  Tiles T;
};

template <int R>
__device__ __forceinline__ bool find_place(const AttnArgs &A, Place &P) {
  P.h = blockIdx.x % (uint32_t)A.hkv;
  const uint32_t b = blockIdx.x / (uint32_t)A.hkv;
  P.split = b % (uint32_t)A.nsplit;
  const int slot = b / (uint32_t)A.nsplit;
  P.s = find_seq<R, 1>(A.cu, A.seqs, A.rows, slot, A.group);
  P.begin = cu_at(A.cu, P.s, A.rows);
  P.n = max(cu_at(A.cu, P.s + 1, A.rows) - P.begin, 0);
  const int local = slot - slot_base<R, 1>(P.begin, P.s, A.group), all = P.n * A.group;
  P.f0 = local * R;
  if (local < 0 || P.f0 >= all) return false;
  P.nrows = min(R, all - P.f0);
  P.p0 = max(A.kv_len[P.s], 0) - P.n;  // may be negative: such rows see nothing
  P.pmin = P.p0 + (uint32_t)P.f0 / (uint32_t)A.group;
  P.pmax = P.p0 + (uint32_t)(P.f0 + P.nrows - 1) / (uint32_t)A.group;
  P.T = visible_tiles(P.pmin, P.pmax, A.max_pages, A.window, A.sinks);
  const int per = max(A.chunk, (int)((uint32_t)(P.T.count + A.nsplit - 1) / (uint32_t)A.nsplit));
  P.splits = max((int)((uint32_t)(P.T.count + per - 1) / (uint32_t)per), 1);
  P.lo = P.split * per;
  P.hi = min(P.T.count, P.lo + per);
  P.tile = (int64_t)slot * A.hkv + P.h;
  return P.split < P.splits;
}

__device__ __forceinline__ int page_id(const AttnArgs &A, int s, int pg) {
  return __builtin_amdgcn_readfirstlane(A.table[(int64_t)s * A.max_pages + pg]);
}

template <int D>
__global__ __launch_bounds__(kDecThreads, 2) void decode_kernel(const AttnArgs A) {
  constexpr int kStride = D + 4;
  union Shared {
    struct {
      float o[kDecWaves][kRows][kStride], m[kDecWaves][kRows], l[kDecWaves][kRows];
    } w;
    float join[kJoinFloats<kRows, kDecSplits, kDecThreads>];
  };
  __shared__ __attribute__((aligned(16))) Shared S;
  const int tid = threadIdx.x, lane = tid & 63, n16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  Place P;
  if (!find_place<kRows>(A, P)) return;
  int i = P.lo + wave, id = 0, id_next = 0;
  if (i < P.hi) id = page_id(A, P.s, P.T.page(i));
  if (i + kDecWaves < P.hi) id_next = page_id(A, P.s, P.T.page(i + kDecWaves));
  const bool valid = n16 < P.nrows;
  const uint32_t fl = P.f0 + (valid ? n16 : 0);
  const int tok = fl / (uint32_t)A.group, head = P.h * A.group + fl % (uint32_t)A.group;
  const int pos = valid ? P.p0 + tok : -1;
  const _Float16 *qr = A.q + (int64_t)(P.begin + tok) * A.q_stride + head * D;
  h8 qf[D / 32];
#pragma unroll
  for (int j = 0; j < D / 64; j++)
#pragma unroll
    for (int u = 0; u < 2; u++) qf[2 * j + u] = *reinterpret_cast<const h8 *>(qr + 64 * j + 16 * g + 8 * u);
  Raw<D> raw[2];
  if (i < P.hi) load_tile<D>(A, P.h, id, raw[0]);
  float qsum = 0.0f;
#pragma unroll
  for (int j = 0; j < D / 32; j++)
#pragma unroll
    for (int r = 0; r < 8; r++) {
      qf[j][r] = valid ? qf[j][r] : (_Float16)0.0f;
      qsum += (float)qf[j][r];
    }
  qsum = 0.5f * quarter_sum(qsum);

  State<D> st;
#pragma unroll
  for (int d = 0; d < D / 16; d++) st.o[d] = (f4){0, 0, 0, 0};
  st.m = kNone;
  st.l = st.corr = 0.0f;
  st.unit = 1.0f;
  auto run = [&](const Raw<D> &t, int ti) {
    const int pg = P.T.page(ti), j1 = pg * kPage + kPage - 1;
    const bool all = j1 <= P.pmin && (A.window == 0 || pg * kPage > P.pmax - A.window || j1 < A.sinks);
    step<D>(A, t, qf, qsum, pg, pos, !all, st);
  };
  // the next page's bytes are on their way while a page is worked on, the id
  // of the one after that too
  auto ahead = [&](Raw<D> &t) {
    if (i + kDecWaves < P.hi) load_tile<D>(A, P.h, id_next, t);
    if (i + 2 * kDecWaves < P.hi) id_next = page_id(A, P.s, P.T.page(i + 2 * kDecWaves));
  };
  while (i < P.hi) {
    ahead(raw[1]);
    run(raw[0], i);
    i += kDecWaves;
    if (i >= P.hi) break;
    ahead(raw[0]);
    run(raw[1], i);
    i += kDecWaves;
  }

  // the waves' results meet in LDS
  st.l = quarter_sum(st.l);
  st.corr = 0.5f * quarter_sum(st.corr);
#pragma unroll
  for (int d = 0; d < D / 16; d++)
    *reinterpret_cast<f4 *>(&S.w.o[wave][n16][16 * d + 4 * g]) = (st.o[d] + st.corr) * st.unit;
  if (g == 0) {
    S.w.m[wave][n16] = st.m;
    S.w.l[wave][n16] = st.l;
  }
  __syncthreads();
  // outputs 4 c .. 4 c + 3 of a row, for the rows that are there
  constexpr int kQuads = D / 4, kRound = kDecThreads / kQuads;
  auto write_out = [&](int row, int d, f4 o) {
    const uint32_t f = P.f0 + row;
    _Float16 *dst = A.out + (int64_t)(P.begin + f / (uint32_t)A.group) * A.out_stride +
                    (P.h * A.group + f % (uint32_t)A.group) * D + d;
    *reinterpret_cast<h4 *>(dst) = (h4){(_Float16)o[0], (_Float16)o[1], (_Float16)o[2], (_Float16)o[3]};
  };
  Rsrc base = make_rsrc(A.partials + P.tile * A.nsplit * partial_floats(kRows, D));
  for (int row = tid / kQuads; row < P.nrows; row += kRound) {
    const int c = tid % kQuads;
    float M = kNone, L = 0.0f;
#pragma unroll
    for (int w = 0; w < kDecWaves; w++) M = fmaxf(M, S.w.m[w][row]);
    f4 o = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kDecWaves; w++) {
      const float f = __builtin_amdgcn_exp2f(S.w.m[w][row] - M);
      L += f * S.w.l[w][row];
      o += f * *reinterpret_cast<const f4 *>(&S.w.o[w][row][4 * c]);
    }
    if (P.splits > 1) {
      const int at = P.split * partial_floats(kRows, D);
      store_dev(base, at + row * D + 4 * c, o);
      if (c == 0) store_dev2(base, at + kRows * D + 2 * row, M, L);
    } else {
      write_out(row, 4 * c, o * inverse(L));
    }
  }
  if (P.splits > 1 && last_split(A.counters + P.tile, P.splits))
    join<kRows, D, kDecThreads, kDecSplits>(base, P.splits, P.nrows, S.join, write_out);
}

// ---- many rows -----------------------------------------------------------
//
// A workgroup takes 128 (token, query head) rows, 32 a wave, over the same
// pages.  Each page's codes are converted to fp16 once for all waves, on
// their way into LDS (two buffers, the next page's bytes in registers
// meanwhile, one barrier a page); K rows of D + 8 and V rows of 64 + 8 fp16
// keep the 16-byte reads of both products free of bank conflicts.  Products
// are v_mfma_f32_32x32x16_f16, scores transposed as in the decode kernel: with
// key rows handed over in the order of row_token() a lane holds, for its query
// row, 8 consecutive tokens per 16, half a wave each half: what the second
// product's operand is.
//
// The running maximum is a reference, not the maximum: it moves only when a
// score exceeds it by 2^8 in weight, so the output is hardly ever rescaled
// (fp16 weights reach 2^8, times 2^4 for the page's value scale).
constexpr int kTileRows = 128, kWaveRows = 32;
constexpr int kThreads = 256;
constexpr int kPreSplits = 16;
typedef float f16x __attribute__((ext_vector_type(16)));

// The token of a 32-token group that row r of the score product takes.
__device__ __forceinline__ int row_token(int r) { return (r & 16) + ((r >> 2) & 1) * 8 + ((r >> 3) & 1) * 4 + (r & 3); }

template <int D>
struct Page {
  uint4 k[D / 64], v[D / 64];
  float ks, vs;  // ks < 0: no such page
};

template <int D>
__device__ __forceinline__ void load_page(const AttnArgs &A, int h, int id, Page<D> &t) {
  const bool ok = id >= 0 && id < A.num_pages;
  const int64_t ph = (int64_t)(ok ? id : 0) * A.hkv + h;
  t.ks = ok ? A.ks[ph] : -1.0f;
  t.vs = A.vs[ph];
  const uint4 *kp = reinterpret_cast<const uint4 *>(A.k + ph * (kPage * D));
  const uint4 *vp = reinterpret_cast<const uint4 *>(A.v + ph * (kPage * D));
#pragma unroll
  for (int i = 0; i < D / 64; i++) {
    t.k[i] = kp[i * kThreads + threadIdx.x];
    t.v[i] = vp[i * kThreads + threadIdx.x];
  }
}

template <int D>
struct Lds {
  _Float16 k[kPage][D + 8], v[D][kPage + 8];
};

template <int D>
__device__ __forceinline__ void put_page(const Page<D> &t, Lds<D> &l) {
#pragma unroll
  for (int i = 0; i < D / 64; i++) {
    const int idx = i * kThreads + threadIdx.x;
    h8 *kd = reinterpret_cast<h8 *>(&l.k[idx / (D / 16)][idx % (D / 16) * 16]);
    kd[0] = codes8(t.k[i].x, t.k[i].y);
    kd[1] = codes8(t.k[i].z, t.k[i].w);
    h8 *vd = reinterpret_cast<h8 *>(&l.v[idx / 4][idx % 4 * 16]);
    vd[0] = codes8(t.v[i].x, t.v[i].y);
    vd[1] = codes8(t.v[i].z, t.v[i].w);
  }
}

template <int D>
__global__ __launch_bounds__(kThreads, 2) void prefill_kernel(const AttnArgs A) {
  union Shared {
    Lds<D> page[2];
    float join[kJoinFloats<kTileRows, kPreSplits, kThreads>];
  };
  __shared__ __attribute__((aligned(16))) Shared S;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 31, half = lane >> 5;
  Place P;
  if (!find_place<kTileRows>(A, P)) return;
  const int row = wave * kWaveRows + n;
  const bool valid = row < P.nrows;
  const uint32_t fl = P.f0 + (valid ? row : 0);
  const int tok = fl / (uint32_t)A.group, head = P.h * A.group + fl % (uint32_t)A.group;
  const int pos = valid ? P.p0 + tok : -1;
  const _Float16 *qr = A.q + (int64_t)(P.begin + tok) * A.q_stride + head * D;
  h8 qf[D / 16];
  float qsum = 0.0f;
#pragma unroll
  for (int j = 0; j < D / 16; j++) {
    h8 x = *reinterpret_cast<const h8 *>(qr + 16 * j + 8 * half);
#pragma unroll
    for (int i = 0; i < 8; i++) {
      x[i] = valid ? x[i] : (_Float16)0.0f;
      qsum += (float)x[i];
    }
    qf[j] = x;
  }
  qsum = 0.5f * half_sum(qsum);
  // the wave's own rows: positions wmin .. wmax (none: wmax = -1)
  const int r0 = wave * kWaveRows, r1 = min(r0 + kWaveRows, P.nrows) - 1;
  const int wmin = P.p0 + (uint32_t)(P.f0 + r0) / (uint32_t)A.group;
  const int wmax = r1 < r0 ? -1 : P.p0 + (int)((uint32_t)(P.f0 + r1) / (uint32_t)A.group);

  f16x o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; i++)
#pragma unroll
    for (int r = 0; r < 16; r++) o[i][r] = 0.0f;
  float m = kNone, l = 0.0f, corr = 0.0f, unit = 1.0f;
  Page<D> next;
  float ks, vs;
  int id_next = 0;
  if (P.lo < P.hi) {
    load_page<D>(A, P.h, page_id(A, P.s, P.T.page(P.lo)), next);
    if (P.lo + 1 < P.hi) id_next = page_id(A, P.s, P.T.page(P.lo + 1));
    put_page<D>(next, S.page[0]);
  }
  ks = next.ks;
  vs = next.vs;
  __syncthreads();
  for (int i = P.lo; i < P.hi; i++) {
    const Lds<D> &L = S.page[(i - P.lo) & 1];
    const bool more = i + 1 < P.hi;
    if (more) load_page<D>(A, P.h, id_next, next);
    if (i + 2 < P.hi) id_next = page_id(A, P.s, P.T.page(i + 2));
    const int pg = P.T.page(i), j0 = pg * kPage, j1 = j0 + kPage - 1;
    const bool none = ks < 0.0f || j0 > wmax || (A.window && j1 <= wmin - A.window && j0 >= A.sinks);
    if (!none) {
      f16x acc[2];
#pragma unroll
      for (int t = 0; t < 2; t++) {
#pragma unroll
        for (int r = 0; r < 16; r++) acc[t][r] = 0.0f;
        const _Float16 *kr = &L.k[32 * t + row_token(n)][8 * half];
#pragma unroll
        for (int j = 0; j < D / 16; j++)
          acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(*reinterpret_cast<const h8 *>(kr + 16 * j), qf[j], acc[t], 0, 0, 0);
      }
      const bool all = j1 <= wmin && (A.window == 0 || j0 > wmax - A.window || j1 < A.sinks);
      if (!all) {
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
          for (int r = 0; r < 16; r++) {
            const int j = j0 + 32 * t + (r >> 3) * 16 + 8 * half + (r & 7);
            const bool see = j <= pos && (A.window == 0 || j > pos - A.window || j < A.sinks);
            acc[t][r] = see ? acc[t][r] : -__builtin_inff();
          }
      }
      // a page of zeros has scale 0: its (zero) scores stay finite, masked ones -inf
      const float sc = fmaxf(ks * A.scale_log2, 1e-37f);
      float mx = acc[0][0];
#pragma unroll
      for (int r = 1; r < 16; r++) mx = fmaxf(mx, acc[0][r]);
#pragma unroll
      for (int r = 0; r < 16; r++) mx = fmaxf(mx, acc[1][r]);
      mx = (half_max(mx) + qsum) * sc;
      const bool has_v = vs > 0.0f;  // a page of zeros adds to the sum only
      const float ratio = has_v ? vs / unit : 1.0f;
      const bool far = !(ratio > 0.0625f && ratio < 16.0f);
      const float shift = far ? 0.0f : __builtin_amdgcn_logf(ratio);
      if (far || __any(mx > m + 8.0f)) {
        const float mn = mx > m + 8.0f ? mx : m;
        float alpha = __builtin_amdgcn_exp2f(m - mn);
        m = mn;
        l *= alpha;
        if (far) {
          alpha *= fminf(unit / vs, 3.0e38f);
          unit = vs;
        }
        corr *= alpha;
#pragma unroll
        for (int d = 0; d < D / 32; d++)
#pragma unroll
          for (int r = 0; r < 16; r++) o[d][r] *= alpha;
      }
      const float bias = qsum * sc + shift - m;
      float sum = 0.0f;
      h8 p[2][2];
#pragma unroll
      for (int t = 0; t < 2; t++)
#pragma unroll
        for (int r = 0; r < 16; r++) {
          const float w = __builtin_amdgcn_exp2f(acc[t][r] * sc + bias);
          sum += w;
          p[t][r >> 3][r & 7] = (_Float16)w;
        }
      l += sum * __builtin_amdgcn_exp2f(-shift);
      if (has_v) {
        corr += sum;
#pragma unroll
        for (int d = 0; d < D / 32; d++)
#pragma unroll
          for (int t = 0; t < 2; t++)
#pragma unroll
            for (int u = 0; u < 2; u++) {
              const h8 a = *reinterpret_cast<const h8 *>(&L.v[32 * d + n][32 * t + 16 * u + 8 * half]);
              o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, p[t][u], o[d], 0, 0, 0);
            }
      }
    }
    if (more) {
      put_page<D>(next, S.page[(i + 1 - P.lo) & 1]);
      ks = next.ks;
      vs = next.vs;
    }
    __syncthreads();
  }
  l = half_sum(l);
  corr = 0.5f * half_sum(corr);
#pragma unroll
  for (int d = 0; d < D / 32; d++)
#pragma unroll
    for (int r = 0; r < 16; r++) o[d][r] = (o[d][r] + corr) * unit;

  // element r of o[d] is output 32 d + 8 (r / 4) + 4 half + r % 4
  if (P.splits > 1) {
    Rsrc base = make_rsrc(A.partials + P.tile * A.nsplit * partial_floats(kTileRows, D));
    const int at = P.split * partial_floats(kTileRows, D);
    if (valid) {
#pragma unroll
      for (int d = 0; d < D / 32; d++)
#pragma unroll
        for (int r = 0; r < 16; r += 4)
          store_dev(base, at + row * D + 32 * d + 2 * r + 4 * half, (f4){o[d][r], o[d][r + 1], o[d][r + 2], o[d][r + 3]});
      if (half == 0) store_dev2(base, at + kTileRows * D + 2 * row, m, l);
    }
    if (last_split(A.counters + P.tile, P.splits))
      join<kTileRows, D, kThreads, kPreSplits>(base, P.splits, P.nrows, S.join, [&](int jr, int d, f4 v) {
        const uint32_t f = P.f0 + jr;
        *reinterpret_cast<h4 *>(A.out + (int64_t)(P.begin + f / (uint32_t)A.group) * A.out_stride +
                                (P.h * A.group + f % (uint32_t)A.group) * D + d) =
            (h4){(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
      });
    return;
  }
  if (valid) {
    const float inv = inverse(l);
    _Float16 *dst = A.out + (int64_t)(P.begin + tok) * A.out_stride + head * D;
#pragma unroll
    for (int d = 0; d < D / 32; d++)
#pragma unroll
      for (int r = 0; r < 16; r += 4)
        *reinterpret_cast<h4 *>(dst + 32 * d + 2 * r + 4 * half) =
            (h4){(_Float16)(o[d][r] * inv), (_Float16)(o[d][r + 1] * inv), (_Float16)(o[d][r + 2] * inv),
                 (_Float16)(o[d][r + 3] * inv)};
  }
}

// The launch of a call: which kernel, how the keys are split, and the
// workspace that needs.
struct Plan {
  bool prefill;
  int64_t slots;
  int nsplit, chunk;
  size_t counter_bytes, bytes;
};

constexpr int kCus = 256;
constexpr int kMaxChunk = 64;

Plan make_plan(int64_t rows, int64_t seqs, int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t max_kv) {
  Plan P;
  const int64_t group = q_heads / kv_heads;
  P.prefill = rows * group > 32 * seqs;
  const int R = P.prefill ? kTileRows : kRows;
  P.slots = rows * group / R + seqs;
  const int64_t tiles = (max_kv + kPage - 1) / kPage;
  const int64_t full = (rows * group + R - 1) / R, units = (full > seqs ? full : seqs) * kv_heads;
  const int64_t target = P.prefill ? 2 * kCus : kCus, least = P.prefill ? 4 : kDecWaves, most = P.prefill ? kPreSplits : kDecSplits;
  int64_t chunk = (tiles * units + target - 1) / target;
  if (chunk < least) chunk = least;
  if (!P.prefill && chunk > kMaxChunk) chunk = kMaxChunk;
  int64_t nsplit = (tiles + chunk - 1) / chunk;
  if (nsplit > most) nsplit = most;
  if (nsplit < 1) nsplit = 1;
  P.chunk = (int)(chunk < 0x7fffffff ? chunk : 0x7fffffff);
  P.nsplit = (int)nsplit;
  P.counter_bytes = 0;
  P.bytes = 0;
  if (nsplit > 1) {
    P.counter_bytes = ((size_t)P.slots * kv_heads * 4 + 15) / 16 * 16;
    P.bytes = P.counter_bytes + (size_t)P.slots * kv_heads * nsplit * partial_floats(R, (int)head_dim) * 4;
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
  const dim3 grid((unsigned)wgs), block(P.prefill ? kThreads : kDecThreads);
  hipStream_t st = (hipStream_t)stream;
  if (P.prefill) {
    if (head_dim == 128) hipLaunchKernelGGL(prefill_kernel<128>, grid, block, 0, st, A);
    else hipLaunchKernelGGL(prefill_kernel<64>, grid, block, 0, st, A);
  } else {
    if (head_dim == 128) hipLaunchKernelGGL(decode_kernel<128>, grid, block, 0, st, A);
    else hipLaunchKernelGGL(decode_kernel<64>, grid, block, 0, st, A);
  }
  return hipGetLastError() == hipSuccess ? TQ_OK : TQ_ERR_HIP;
}
