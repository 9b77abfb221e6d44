// tq_kv_attn_kernel.h -- attention of new rows over the paged 8-bit key/value cache.
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
// The weights are rounded to fp16 for the second product, half a step of 2^-11
// each; their sum is of the fp32 weights.  The kernel for up to 16 rows adds the
// rounding error back as a second fp16 term (its matrix units are idle anyway).
// With 32 rows the term takes the registers (8 sequences with 4 rows on up to 6001
// tokens 35.7 against 27.9 us, with 16 rows 86 against 57), with 128 a third more
// products where the matrix units bound.  fp16 ends at 2^-24, so the
// largest weight of a row is put at 2^11 to 2^15, not at 1: a weight keeps its
// eleven bits down to 2^-25 of the largest one, and what is lost of a smaller one
// is at most 2^-36 of that.  (With the largest at 1 the 2^17 keys of a long
// context 2^-24 below a first token that draws all attention were rounded to a
// single bit, all the same way.)
//
// Bound: few rows (decode) read 2 head_dim bytes a token and KV head and are
// bound by HBM; the work along the keys is split over workgroups, whose
// partial (max, sum, output) meet in the workspace, where the last one to
// arrive joins them in order.  Many rows (prefill) are bound by the matrix,
// vector and LDS pipes together.
//
// Measured, 64 query and 8 KV heads of 128 (a plain streaming read reaches 6.9
// TB/s, a large fp16 matrix product 1202 TFLOP/s):
//   one token over 517 tokens            9 us
//   one token over 131001 tokens        53 us   5.0 TB/s
//   64 sequences of up to 8190 tokens  125 us   5.4 TB/s
//   64 sequences of up to 32 K tokens  436 us   6.2 TB/s
//   8 sequences of up to 6001, 4 rows   27 us   2.6 TB/s
//   a prompt of 4096 tokens            315 us   870 TFLOP/s
// decode_kernel<128, 2, false> takes 256 registers and spills 12 more (over own keys
// behind a prefix 23, over a prefix 10), and prefill_kernel<128> over own keys 4.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tq.h"
#include "tq_device.h"
#include "tq_kv.h"
#include "tq_wave.h"

namespace {

using namespace tqkv;

typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

constexpr int kRows = 16;  // (token, query head) rows of a decode workgroup
constexpr int kWaves = 8;  // of a decode workgroup
constexpr int kDecPieces = 128;  // pieces of a unit at most (and one or two more)
// Pages, see "few rows".  A piece has kLeast at least: one token of 1100 10.9 us, of
// 4096 12.1 (8: 13.7, 13.0; 3: 10.9, 13.1).  Units of up to kWhole stay whole: 64
// sequences of up to 700 tokens 17.6 us (8: 35; 32: 17.5).  A cut leaves kSnap at
// least on both sides (the workspace's two results a workgroup rest on per >= kSnap).
constexpr int kSnap = 4, kLeast = 4, kWhole = 16;
static_assert(kSnap <= kLeast, "a share's two borders must not meet in one unit's end");
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
  int slots, solo;    // prefill: row tiles; units that stay whole
  int nsplit, chunk;  // prefill: pieces of the others at most; pages of a piece at least
  int whole;          // decode: units of up to so many pages stay whole
  // sequences that share a prefix (below): their groups, the prefixes' results
  const int *cu_seqs, *prefix;
  float *mid;
  int64_t mid_ml;                         // where the (maximum, sum) pairs start, without tiles
  int groups, all_seqs;
  int pre_slots, pre_nsplit, pre_chunk;   // the prefix launch's tiles of 128 rows (nsplit 0: results row by row)
};

// Which keys a launch is about.  kAllKeys: all that a row sees.  Sequences that
// share their first pages (a prefix of whole pages a group of sequences) take two
// launches.  kPrefixKeys: the prefixes, whose "sequences" are the groups, with the
// rows of all their sequences, every one of which sees all of the prefix; the
// results (sums of weighted values, maximum and sum of the weights) go to mid: row
// by row, or as the pieces of tiles of 128 rows.  kOwnKeys: the keys behind the
// prefix, joined with what mid holds, which is left zero.
enum Keys { kAllKeys = 0, kPrefixKeys, kOwnKeys };

// The first row of sequence (or group) i.
template <int KEYS>
__device__ __forceinline__ int row_at(const AttnArgs &A, int i) {
  if (KEYS == kPrefixKeys) i = min(max(A.cu_seqs[i], 0), A.all_seqs);
  return cu_at(A.cu, i, A.rows);
}
// Keys of a sequence (of a group's prefix: of whole pages).
template <int KEYS>
__device__ __forceinline__ int keys_of(const AttnArgs &A, int s) {
  return KEYS == kPrefixKeys ? max(A.prefix[s], 0) / kPage * kPage : max(A.kv_len[s], 0);
}
// The group of a sequence: the last one that starts at or before it, if it is in
// it; else -1.
__device__ __forceinline__ int group_of(const AttnArgs &A, int s) {
  int lo = 0, hi = A.groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (A.cu_seqs[mid] <= s) lo = mid;
    else hi = mid;
  }
  return A.cu_seqs[lo] <= s && s < A.cu_seqs[lo + 1] ? lo : -1;
}
// Pages before a sequence's own.
template <int KEYS>
__device__ __forceinline__ int pages_before(const AttnArgs &A, int s) {
  if (KEYS != kOwnKeys) return 0;
  const int g = group_of(A, s);
  return g >= 0 ? max(A.prefix[g], 0) / kPage : 0;
}

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

// ... without the `before` first pages.
template <int KEYS>
__device__ __forceinline__ void leave_out(Tiles &t, int before) {
  if (KEYS != kOwnKeys) return;
  const int n = min(before, t.count);
  t.first += n;
  t.count -= n;
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

// A value that all lanes have alike, in a scalar register.
__device__ __forceinline__ float uniform(float v) { return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v))); }

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

// The bytes of one page and KV head that a lane takes part in.  Keys and
// values are fetched apart: the next page's keys as soon as this page's have
// been used, its values after this page's.
template <int D>
struct Raw {
  uint4 k[4][D / 64], v[D / 16];
  float ks, vs;  // wave-uniform; ks < 0: no such page
};

template <int D>
__device__ __forceinline__ void load_keys(const AttnArgs &A, int h, int id, Raw<D> &t) {
  const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
  const bool ok = id >= 0 && id < A.num_pages;
  const int64_t ph = (int64_t)(ok ? id : 0) * A.hkv + h;
  const uint8_t *kp = A.k + ph * (kPage * D) + (16 * (m >> 2) + (m & 3)) * D + 16 * g;
  t.ks = ok ? A.ks[ph] : -1.0f;
#pragma unroll
  for (int i = 0; i < 4; i++)
#pragma unroll
    for (int j = 0; j < D / 64; j++) t.k[i][j] = *reinterpret_cast<const uint4 *>(kp + 4 * i * D + 64 * j);
}

// Values are streamed past the caches (64 contexts of up to 8190 tokens 125
// against 137 us, 131001 tokens 55.5 against 59.9); not the keys, whose lines
// two of a lane's loads share (129.6 and 55.3 us with both).
template <int D>
__device__ __forceinline__ void load_values(const AttnArgs &A, int h, int id, Raw<D> &t) {
  const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
  const int64_t ph = (int64_t)(id >= 0 && id < A.num_pages ? id : 0) * A.hkv + h;
  const uint8_t *vp = A.v + ph * (kPage * D) + m * kPage + 16 * g;
  t.vs = A.vs[ph];
#pragma unroll
  for (int i = 0; i < D / 16; i++) t.v[i] = tqdev::ld_stream16(vp + 16 * i * kPage);
}

// A page with a smaller value scale counts as zeros: its values are below
// 2^-30, nothing to an fp16 output (half its least step is 2^-25).  So the
// state's unit (below) never falls by more than the largest scale's 2^50 over
// this, and 2^87 times what the products can sum up to stays within fp32.
constexpr float kLeastScale = 0x1p-37f;

// Running state of a lane's query row.  The output is held as
//   unit * (o + corr / 2), corr = sum of the weights that o's products took,
// where `unit` (one for the wave) is a value scale: pages with 2^-7 to 1 of it
// have the ratio folded into their weights, larger and smaller ones move the
// state to their own.  (A ratio below one takes bits from weights of values that
// are as much smaller; room for ratios above one would take them from all.)
// m is a reference for the weights' exponents: kLift below the score it was set
// by, moved only when a score exceeds it by kTop, so the outputs are hardly ever
// rescaled and weights reach 2^15.25 in fp16, which ends at 2^16.  (kLift 9 or 7, for
// scores that rise further, measured the same.)  The 0.75 between are for the
// exponent's roundings: those of the reference, of the half-code term and of their
// difference, together 8 of 2^-24 of 2^20.5, 0.71, at scores of 2^20.
constexpr float kLift = 11.0f, kTop = 15.0f;
constexpr float kNoUnit = -1000.0f;  // log2 of the unit before the first page with values

// Whether the state moves to the scale of a page, whose log2 is `over` above
// the unit's: outside -7.75 .. 0.25 (weights stay below 2^15.25).
__device__ __forceinline__ bool unit_moves(float over) { return !(fabsf(over + 3.75f) < 4.0f); }

template <int D>
struct State {
  f4 o[D / 16];
  float m, l, corr;
};

// Scores of RT tiles of 16 rows against a page's keys, before any scale.
template <int D, int RT>
__device__ __forceinline__ void scores(const Raw<D> &t, const h8 (&qf)[RT][D / 32], f4 (&x)[RT][4]) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
#pragma unroll
    for (int a = 0; a < RT; a++) x[a][i] = (f4){0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < D / 64; j++) {
      const uint4 w = t.k[i][j];
      const h8 k0 = codes8(w.x, w.y), k1 = codes8(w.z, w.w);
#pragma unroll
      for (int a = 0; a < RT; a++) {
        x[a][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, qf[a][2 * j], x[a][i], 0, 0, 0);
        x[a][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, qf[a][2 * j + 1], x[a][i], 0, 0, 0);
      }
    }
  }
}

// The weights of one row tile: hi (+ lo, if LO) fp16 terms of w * 2^shift.
template <int D, bool LO>
__device__ __forceinline__ void weights(const AttnArgs &A, f4 (&x)[4], float qsum, float sc, float shift, float moves,
                                        bool masked, int j0, int pos, bool has_v, State<D> &st, h8 (&hi)[2], h8 (&lo)[2]) {
  if (masked) {
#pragma unroll
    for (int i = 0; i < 16; i++) {
      const int j = j0 + i;
      const bool see = j <= pos && (A.window == 0 || j > pos - A.window || j < A.sinks);
      x[i >> 2][i & 3] = see ? x[i >> 2][i & 3] : -__builtin_inff();
    }
  }
  float mx = x[0][0];
#pragma unroll
  for (int i = 1; i < 16; i++) mx = fmaxf(mx, x[i >> 2][i & 3]);
  mx = (quarter_max(mx) + qsum) * sc;
  if (moves != 1.0f || __any(mx > st.m + kTop)) {
    const float mn = mx > st.m + kTop ? mx - kLift : st.m;
    float alpha = __builtin_amdgcn_exp2f(st.m - mn);
    st.m = mn;
    st.l *= alpha;
    alpha *= moves;
    st.corr *= alpha;
#pragma unroll
    for (int i = 0; i < D / 16; i++) st.o[i] *= alpha;
  }
  const float bias = qsum * sc + shift - st.m;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; i++) {
    const float w = __builtin_amdgcn_exp2f(x[i >> 2][i & 3] * sc + bias);
    sum += w;
    const _Float16 r = (_Float16)w;
    hi[i >> 3][i & 7] = r;
    if (LO) lo[i >> 3][i & 7] = (_Float16)(w - (float)r);
  }
  st.l += sum * __builtin_amdgcn_exp2f(-shift);
  if (has_v) st.corr += sum;
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

// What the prefix launch left of a sequence's rows in mid: for each row `pieces`
// results `step` floats apart.
constexpr int kPreRows = 128, kPrePieces = 32;
struct Before {
  int pieces, first, slot0;  // the group's first row and first tile
  int64_t step;
  __device__ __forceinline__ Before() : pieces(0), first(0), slot0(0), step(0) {}
  __device__ __forceinline__ Before(const AttnArgs &A, int s, int D) : pieces(0), first(0), slot0(0), step(0) {
    const int g = group_of(A, s);
    if (g < 0) return;
    pieces = 1;
    if (A.pre_nsplit == 0) return;
    const int count = (int)min((int64_t)(max(A.prefix[g], 0) / kPage), A.max_pages);
    const int per = max(A.pre_chunk, (int)((uint32_t)(count + A.pre_nsplit - 1) / (uint32_t)A.pre_nsplit));
    pieces = max((int)((uint32_t)(count + per - 1) / (uint32_t)per), 1);
    first = row_at<kPrefixKeys>(A, g);
    slot0 = slot_base<kPreRows, 1>(first, g, A.group);
    step = partial_floats(kPreRows, D);
  }
  // where the first result of a row (of query head `head`) has its sums, and its (maximum, sum)
  __device__ __forceinline__ void at(const AttnArgs &A, int row, int head, int D, int64_t &o, int64_t &ml) const {
    if (A.pre_nsplit == 0) {
      const int64_t i = (int64_t)row * (A.hkv * A.group) + head;
      o = i * D;
      ml = A.mid_ml + 2 * i;
      return;
    }
    const uint32_t h = (uint32_t)head / (uint32_t)A.group, f = (row - first) * A.group + ((uint32_t)head - h * A.group);
    // (a row that the prefix launch has no tile of, by arrays out of order: the last one's)
    const int slot = min(max(slot0 + (int)(f / (uint32_t)kPreRows), 0), A.pre_slots - 1);
    const int64_t base = ((int64_t)(A.pre_slots - 1 - slot) * A.hkv + h) * A.pre_nsplit * step;
    const int r = f % (uint32_t)kPreRows;
    o = base + r * D;
    ml = base + kPreRows * D + 2 * r;
  }
};

// A row's (maximum, sum) over its own keys joined to those over its prefix by 16
// lanes, `j` each one's number: `w` takes the prefix's pieces' factors, and the
// one that the sums over its own keys take is returned.  Leaves zeros (`live`).
__device__ __forceinline__ float join_before(float *mid, int64_t ml, const Before &B, int j, bool live, float M, float L,
                                             float *w) {
  float m[kPrePieces / 16], l[kPrePieces / 16], most = M, sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kPrePieces / 16; i++) {
    const int k = 16 * i + j;
    m[i] = kNone;
    l[i] = 0.0f;
    if (live && k < B.pieces) {
      float *p = mid + ml + k * B.step;
      m[i] = p[0];
      l[i] = p[1];
      p[0] = p[1] = 0.0f;
      if (!(l[i] > 0.0f || l[i] != l[i])) m[i] = kNone;  // nothing there
    }
    most = fmaxf(most, m[i]);
  }
  most = tqdev::row16_max(most);
#pragma unroll
  for (int i = 0; i < kPrePieces / 16; i++) {
    m[i] = __builtin_amdgcn_exp2f(m[i] - most);
    sum += m[i] * l[i];
  }
  const float f = __builtin_amdgcn_exp2f(M - most), inv = inverse(f * L + tqdev::row16_sum(sum));
#pragma unroll
  for (int i = 0; i < kPrePieces / 16; i++)
    if (live && 16 * i + j < B.pieces) w[16 * i + j] = m[i] * inv;
  return f * inv;
}
// The prefix's part of four outputs; leaves zeros.
__device__ __forceinline__ f4 take_before(float *mid, int64_t o, const Before &B, const float *w) {
  f4 sum = {0, 0, 0, 0};
#pragma unroll 1
  for (int k0 = 0; k0 < B.pieces; k0 += 8) {
    f4 v[8];
#pragma unroll
    for (int k = 0; k < 8; k++) v[k] = *reinterpret_cast<const f4 *>(mid + o + min(k0 + k, B.pieces - 1) * B.step);
#pragma unroll
    for (int k = 0; k < 8; k++)
      if (k0 + k < B.pieces) {
        sum += w[k0 + k] * v[k];
        *reinterpret_cast<f4 *>(mid + o + (k0 + k) * B.step) = (f4){0, 0, 0, 0};
      }
  }
  return sum;
}

// The last piece's join of a tile of R rows: the partial results, piece k's at
// float `at(k)` of `part`, summed in the order of the pieces;
// `out(row, d, f4)` takes the outputs.  Each row's maximum and sum over the
// pieces come from 16 lanes; the outputs take 16 bytes a thread with kBatch
// pieces' loads in flight (the first of them before the weights are known);
// where the rows are fewer than the threads, the pieces are dealt over
// `parts` groups of threads that meet in LDS.  The words read are left zero
// for the next call, whatever its shape.
// `more(row, j, live, M, L)`, by 16 lanes a row (j: each one's number), returns the
// factor of the pieces' sums, whose weights have the maximum M and the sum L.
template <int R, int D, int NT, int MAXP, typename At, typename Out, typename More>
__device__ __forceinline__ void join(int tid, Rsrc part, int pieces, int nrows, float *lds, const At &at, const Out &out,
                                     const More &more) {
  // loads of 16 bytes in flight a thread: of 8 pieces (32 rows: for each of two
  // outputs), or (many rows, few pieces) of 2 pieces for each of 4 outputs
  constexpr int kPer16 = (MAXP + 15) / 16, kQ = R > 32 ? 4 : R > 16 ? 2 : 1, kBatch = R > 32 ? 2 : 8;
  const int quads = nrows * (D / 4);
  const int parts = quads * 4 <= NT ? 4 : quads * 2 <= NT ? 2 : 1;
  const int per = NT / parts, p = tid / per, q0 = tid - p * per;
  f4 v[kQ][kBatch];
  auto fetch = [&](int k0, int q) {
    auto some = [&](int b0) {
#pragma unroll
      for (int a = 0; a < kQ; a++)
#pragma unroll
        for (int b = b0; b < b0 + kBatch / 2; b++)
          v[a][b] = load_dev(part, at(min(k0 + b * parts, pieces - 1)) + 4 * min(q + a * per, quads - 1));
    };
    some(0);
    if (pieces > kBatch / 2 * parts) some(kBatch / 2);
  };
  if (q0 < quads) fetch(p, q0);
  float *wt = lds;  // the pieces' weights, [MAXP][R]
  const int j = tid & 15;
#pragma unroll 1
  for (int r0 = 0; r0 < nrows; r0 += NT / 16) {
    const int r = r0 + tid / 16, rr = min(r, nrows - 1);
    float m[kPer16], l[kPer16], M = kNone, L = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer16; i++) {
      m[i] = kNone;
      l[i] = 0.0f;
      if (16 * i < pieces) load_dev2(part, at(min(16 * i + j, pieces - 1)) + R * D + 2 * rr, m[i], l[i]);
    }
#pragma unroll
    for (int i = 0; i < kPer16; i++) {
      if (16 * i + j >= pieces) m[i] = kNone, l[i] = 0.0f;
      M = fmaxf(M, m[i]);
    }
    M = tqdev::row16_max(M);
#pragma unroll
    for (int i = 0; i < kPer16; i++) {
      m[i] = __builtin_amdgcn_exp2f(m[i] - M);
      L += m[i] * l[i];
    }
    L = tqdev::row16_sum(L);
    const float inv = more(rr, j, r < nrows, M, L);
#pragma unroll
    for (int i = 0; i < kPer16; i++) {
      const int k = 16 * i + j;
      if (k < pieces && r < nrows) {
        wt[k * R + r] = m[i] * inv;
        store_dev2(part, at(k) + R * D + 2 * r, 0.0f, 0.0f);
      }
    }
  }
  __syncthreads();
  f4 *red = reinterpret_cast<f4 *>(lds + R * MAXP);
#pragma unroll 1
  for (int q = q0; q < quads; q += kQ * per) {  // one round where parts > 1
    f4 o[kQ];
#pragma unroll
    for (int a = 0; a < kQ; a++) o[a] = (f4){0, 0, 0, 0};
#pragma unroll 1
    for (int k0 = p; k0 < pieces; k0 += kBatch * parts) {
      if (q != q0 || k0 != p) fetch(k0, q);
#pragma unroll
      for (int b = 0; b < kBatch; b++)
        if (k0 + b * parts < pieces)
#pragma unroll
          for (int a = 0; a < kQ; a++)
            o[a] += v[a][b] * wt[(k0 + b * parts) * R + min(q + a * per, quads - 1) / (D / 4)];
    }
#pragma unroll
    for (int a = 0; a < kQ; a++) {
      const int e = q + a * per;
      if (e >= quads) break;
#pragma unroll 1
      for (int k = p; k < pieces; k += parts) store_dev(part, at(k) + 4 * e, (f4){0, 0, 0, 0});
      if (parts == 1)
        out(e / (D / 4), 4 * e % D, o[a]);
      else if (a == 0)
        red[tid] = o[a];
    }
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
constexpr int kJoinFloats = R * MAXS + 4 * NT;

// A workgroup's place: R consecutive (token, query head) rows of a sequence
// and KV head, and its share of their pages.
struct Place {
  int h, s, begin, n, nrows, f0, p0, pmin, pmax, lo, hi, splits, split, nsplit, tile;
  Tiles T;
};

template <int R, int KEYS>
__device__ __forceinline__ bool find_place(const AttnArgs &A, Place &P) {
  // units are numbered from the last tile on: the later rows of a sequence
  // see more keys, and the longest work should start first.  The first `solo`
  // units are whole, the others in up to nsplit pieces.
  int unit = blockIdx.x;
  P.split = 0;
  P.nsplit = 1;
  if (unit >= A.solo) {
    const uint32_t b = unit - A.solo;
    unit = A.solo + b / (uint32_t)A.nsplit;
    P.split = b % (uint32_t)A.nsplit;
    P.nsplit = A.nsplit;
  }
  P.h = unit % (uint32_t)A.hkv;
  const int slot = A.slots - 1 - (int)(unit / (uint32_t)A.hkv);
  P.tile = unit - A.solo;
  const auto first_row = [&](int i) { return row_at<KEYS>(A, i); };
  P.s = find_seq<R, 1>(first_row, A.seqs, slot, A.group);
  P.begin = first_row(P.s);
  P.n = max(first_row(P.s + 1) - P.begin, 0);
  const int local = slot - slot_base<R, 1>(P.begin, P.s, A.group), all = P.n * A.group;
  P.f0 = local * R;
  if (local < 0 || P.f0 >= all) return false;
  P.nrows = min(R, all - P.f0);
  const int keys = keys_of<KEYS>(A, P.s);
  if (KEYS == kPrefixKeys) {
    P.p0 = P.pmin = P.pmax = keys - 1;
  } else {
    P.p0 = keys - P.n;  // may be negative: such rows see nothing
    P.pmin = P.p0 + (uint32_t)P.f0 / (uint32_t)A.group;
    P.pmax = P.p0 + (uint32_t)(P.f0 + P.nrows - 1) / (uint32_t)A.group;
  }
  P.T = visible_tiles(P.pmin, P.pmax, A.max_pages, A.window, A.sinks);
  leave_out<KEYS>(P.T, pages_before<KEYS>(A, P.s));
  const int per = max(A.chunk, (int)((uint32_t)(P.T.count + P.nsplit - 1) / (uint32_t)P.nsplit));
  P.splits = max((int)((uint32_t)(P.T.count + per - 1) / (uint32_t)per), 1);
  P.lo = P.split * per;
  P.hi = min(P.T.count, P.lo + per);
  return P.split < P.splits;
}

template <int KEYS>
__device__ __forceinline__ int page_id(const AttnArgs &A, int s, int pg) {
  if (KEYS == kPrefixKeys) s = min(max(A.cu_seqs[s], 0), A.all_seqs - 1);
  return __builtin_amdgcn_readfirstlane(A.table[(int64_t)s * A.max_pages + pg]);
}

// ---- few rows ------------------------------------------------------------
//
// A unit of work is a tile of R rows of a sequence and one KV head, and has
// `pages` pages (the most that a row tile of the sequence sees; what a tile does not
// see is cut off later).  The workgroups share the units out by the lengths
// that they read, whatever the host knows of them:
//  - as many units as workgroups at most: each is cut into equal pieces of up
//    to `per` pages, `per` the least for which the pieces are no more than the
//    workgroups; a workgroup has one piece.  (Shares of the same length that
//    run over unit borders are two units' work for most workgroups, with two
//    starts and ends: 39 against 26 us for 8 sequences with 4 drafted rows.)
//  - more: workgroup w takes pages w * per .. (w + 1) * per - 1 of the list of
//    all units' pages.  A border that would cut off less than kSnap pages of a
//    unit, or that falls into a unit of at most `whole` pages, moves to the
//    unit's end or start.
// A unit that is cut is joined by the last of its workgroups; only a
// workgroup's first and last unit can be cut, so two partial results a
// workgroup are all the workspace there is.
struct Seq {
  int begin, n, kv, units, pages;  // units: row tiles * KV heads
  int before;                      // pages left out
};

template <int R, int KEYS>
__device__ __forceinline__ Seq seq_load(const AttnArgs &A, int s) {
  Seq q;
  q.begin = row_at<KEYS>(A, s);
  q.n = max(row_at<KEYS>(A, s + 1) - q.begin, 0);
  q.kv = keys_of<KEYS>(A, s);
  q.before = pages_before<KEYS>(A, s);
  int64_t pages = min((int64_t)((q.kv + (int64_t)kPage - 1) / kPage), A.max_pages) - q.before;
  if (A.window) {
    const int64_t seen = ((int64_t)A.sinks + kPage - 1) / kPage + ((int64_t)A.window + R) / kPage + 2;
    pages = min(pages, seen);
  }
  q.pages = (int)max(pages, (int64_t)1);  // a unit that sees nothing still has its zeros to write
  q.units = (int)((uint32_t)(q.n * A.group + R - 1) / (uint32_t)R) * A.hkv;
  return q;
}

// The list of the units' pages, or of their pieces of `per` pages (per > 0):
// its length, and the sequence of a position in it (the last one that starts
// at or before it and is not empty).  Lanes take a sequence each, 64 at a
// time; with up to 64 sequences everything stays in registers.
template <int R, int KEYS>
struct List {
  int total, units, longest, per;
  int count, incl;  // this lane's sequence
  Seq seq;

  __device__ __forceinline__ static int scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // lane 15 of rows 0, 2 to rows 1, 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // lane 31 to rows 2, 3
    return v;
  }

  __device__ __forceinline__ void tally() {
    count = seq.units * (per ? (int)((uint32_t)(seq.pages + per - 1) / (uint32_t)per) : seq.pages);
    incl = scan(count);
  }
  __device__ __forceinline__ void load(const AttnArgs &A, int s) {
    seq.pages = seq.units = seq.n = 0;
    if (s < A.seqs) seq = seq_load<R, KEYS>(A, s);
    tally();
  }

  // all units' pages
  __device__ __forceinline__ void init(const AttnArgs &A) {
    const int lane = threadIdx.x & 63;
    total = units = per = 0;
    int64_t rows = 0;
    float most = 0.0f;  // exact up to 2^24 pages, more than enough for a bound
    for (int s0 = 0; s0 < A.seqs; s0 += 64) {
      load(A, s0 + lane);
      total += __builtin_amdgcn_readlane(incl, 63);
      units += __builtin_amdgcn_readlane(scan(seq.units), 63);
      rows += __builtin_amdgcn_readlane(scan(seq.n), 63);
      most = fmaxf(most, count ? (float)seq.pages : 0.0f);
    }
    longest = (int)tqdev::wave_max64(most);
    // sequences that overlap (cu_rows out of order) could make the list longer
    // than 32 bits count: nothing is done
    if (rows > A.rows) total = units = 0;
  }
  // all units' pieces of `p` pages at most
  __device__ __forceinline__ void cut(const AttnArgs &A, int p) {
    per = p;
    if (A.seqs <= 64) {
      tally();
      total = __builtin_amdgcn_readlane(incl, 63);
      return;
    }
    total = 0;
    for (int s0 = 0; s0 < A.seqs; s0 += 64) {
      load(A, s0 + (threadIdx.x & 63));
      total += __builtin_amdgcn_readlane(incl, 63);
    }
  }

  // -> the sequence, its first position in `start`
  __device__ __forceinline__ int find(const AttnArgs &A, int b, int &start, Seq &q) {
    int s0 = 0, before = 0;
    if (A.seqs > 64) {
      for (;; s0 += 64) {
        load(A, s0 + (threadIdx.x & 63));
        const int sum = __builtin_amdgcn_readlane(incl, 63);
        if (b < before + sum || s0 + 64 >= A.seqs) break;
        before += sum;
      }
    }
    const uint64_t behind = __ballot(incl > b - before);
    const int l = behind ? __builtin_ctzll(behind) : 63;
    start = before + __builtin_amdgcn_readlane(incl, l) - __builtin_amdgcn_readlane(count, l);
    q.begin = __builtin_amdgcn_readlane(seq.begin, l);
    q.n = __builtin_amdgcn_readlane(seq.n, l);
    q.kv = __builtin_amdgcn_readlane(seq.kv, l);
    q.units = __builtin_amdgcn_readlane(seq.units, l);
    q.pages = __builtin_amdgcn_readlane(seq.pages, l);
    q.before = KEYS == kOwnKeys ? __builtin_amdgcn_readlane(seq.before, l) : 0;
    return s0 + l;
  }

  // A border of the workgroups' shares, moved as said above.
  __device__ __forceinline__ int snap(const AttnArgs &A, int64_t b64) {
    if (b64 >= total) return total;
    const int b = (int)b64;
    if (b <= 0) return 0;
    int start;
    Seq q;
    find(A, b, start, q);
    const int u0 = start + (uint32_t)(b - start) / (uint32_t)q.pages * q.pages;
    if (b == u0) return b;
    if (q.pages <= A.whole || u0 + q.pages - b < kSnap) return u0 + q.pages;
    return b - u0 < kSnap ? u0 : b;
  }
};

// WHOLE: no unit is cut; a workgroup per unit, found as the prefill kernel
// finds its tile, without the list and the join (2 to 4 us less for short
// contexts, where the call is latency).
template <int D, int RT, bool WHOLE, int NW, int KEYS = kAllKeys>
__global__ __launch_bounds__(NW * 64, NW == 4 ? 3 : 2) void decode_kernel(const AttnArgs A) {
  constexpr int kDecWaves = NW, kDecThreads = NW * 64;
  constexpr int kStride = D + 4, R = kRows * RT, PF = partial_floats(R, D);
  union Shared {
    struct {
      float o[kDecWaves][R][kStride], m[kDecWaves][R], l[kDecWaves][R];
    } w;
    float join[WHOLE ? 1 : kJoinFloats<R, kDecPieces + 2, kDecThreads>];
  };
  __shared__ __attribute__((aligned(16))) Shared S;
  __shared__ float pre_w[KEYS == kOwnKeys ? R * kPrePieces : 1], keep[KEYS == kOwnKeys ? R : 1];
  const int wg = blockIdx.x;
  List<R, KEYS> list;
  int at = 0, stop = 1, per = 1;
  bool equal = false;  // one piece a workgroup
  if constexpr (!WHOLE) {
    list.init(A);
    const int wgs = gridDim.x;
    const int even = (int)((uint32_t)(list.total + wgs - 1) / (uint32_t)wgs);
    per = max(max(even, kLeast), (list.longest + kDecPieces - 1) / kDecPieces);
    if (list.total <= 0) return;
    equal = list.units <= wgs;
    if (equal) {
      for (list.cut(A, per); list.total > wgs; list.cut(A, per)) per += max(per / 8, 1);
      at = wg;
      stop = min(wg + 1, list.total);
    } else {
      at = list.snap(A, (int64_t)wg * per);
      stop = list.snap(A, (int64_t)(wg + 1) * per);
    }
  }
  const Rsrc parts = make_rsrc(A.partials);
  const int lane = threadIdx.x & 63, n16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // What a workgroup works on: rows f0 .. f0 + nrows - 1 of a sequence and KV
  // head, pages i, i + kDecWaves, ... < hi of its list T (i: this wave's first).
  struct Unit {
    int s, h, begin, f0, nrows, p0, pmin, pmax, i, hi, pieces, first;
    Tiles T;
  };
  // the unit at list position `at`, which moves behind it; false: none
  auto next_unit = [&](Unit &u) -> bool {
    Seq q;
    int from = 0, upto = 0x7fffffff;
    u.pieces = 1;
    u.first = wg;
    if constexpr (WHOLE) {
      u.h = wg % (uint32_t)A.hkv;
      const int slot = wg / (uint32_t)A.hkv;
      u.s = find_seq<R, 1>([&](int i) { return row_at<KEYS>(A, i); }, A.seqs, slot, A.group);
      q = seq_load<R, KEYS>(A, u.s);
      u.f0 = (slot - slot_base<R, 1>(q.begin, u.s, A.group)) * R;
      at = stop;
      if (u.f0 < 0 || u.f0 >= q.n * A.group) return false;
    } else {
      if (at >= stop) return false;
      int start;
      u.s = list.find(A, at, start, q);
      int unit;
      if (equal) {
        u.pieces = (uint32_t)(q.pages + per - 1) / (uint32_t)per;
        unit = (uint32_t)(at - start) / (uint32_t)u.pieces;
        const int k = at - start - unit * u.pieces, size = (uint32_t)(q.pages + u.pieces - 1) / (uint32_t)u.pieces;
        u.first = wg - k;
        from = k * size;
        upto = min(from + size, q.pages);
        at = stop;
      } else {
        unit = (uint32_t)(at - start) / (uint32_t)q.pages;
        const int u0 = start + unit * q.pages, end = min(u0 + q.pages, stop);
        // the pieces of a cut unit belong to workgroups first, first + 1, ...
        if (at != u0 || end != u0 + q.pages) {
          const int cut = (uint32_t)(u0 + kSnap + per - 1) / (uint32_t)per;
          u.pieces = (int)((uint32_t)(u0 + q.pages - kSnap) / (uint32_t)per) - cut + 2;
          u.first = cut - 1;
        }
        from = at - u0;
        upto = end - u0;
        at = end;
      }
      u.h = (uint32_t)unit % (uint32_t)A.hkv;
      u.f0 = (int)((uint32_t)unit / (uint32_t)A.hkv) * R;
    }
    u.begin = q.begin;
    u.nrows = min(R, q.n * A.group - u.f0);
    if (KEYS == kPrefixKeys) {
      u.p0 = u.pmin = u.pmax = q.kv - 1;
    } else {
      u.p0 = q.kv - q.n;  // may be negative: such rows see nothing
      u.pmin = u.p0 + (uint32_t)u.f0 / (uint32_t)A.group;
      u.pmax = u.p0 + (uint32_t)(u.f0 + u.nrows - 1) / (uint32_t)A.group;
    }
    u.T = visible_tiles(u.pmin, u.pmax, A.max_pages, A.window, A.sinks);
    leave_out<KEYS>(u.T, q.before);
    u.i = from + wave;
    u.hi = min(upto, u.T.count);
    return true;
  };
  int id_next = 0, pos[RT];
  h8 qf[RT][D / 32];
  Raw<D> raw;
  auto first_page = [&](const Unit &u) {
    if (u.i < u.hi) {
      const int id = page_id<KEYS>(A, u.s, u.T.page(u.i));
      if (u.i + kDecWaves < u.hi) id_next = page_id<KEYS>(A, u.s, u.T.page(u.i + kDecWaves));
      load_keys<D>(A, u.h, id, raw);
      load_values<D>(A, u.h, id, raw);
    }
  };
  auto queries = [&](const Unit &u) {
#pragma unroll
    for (int a = 0; a < RT; a++) {
      const int row = kRows * a + n16;
      const bool valid = row < u.nrows;
      const uint32_t fl = u.f0 + (valid ? row : 0);
      const int tok = fl / (uint32_t)A.group, head = u.h * A.group + fl % (uint32_t)A.group;
      pos[a] = !valid ? -1 : KEYS == kPrefixKeys ? u.p0 : u.p0 + tok;
      const _Float16 *qr = A.q + (int64_t)(u.begin + tok) * A.q_stride + head * D;
#pragma unroll
      for (int j = 0; j < D / 64; j++)
#pragma unroll
        for (int k = 0; k < 2; k++) qf[a][2 * j + k] = *reinterpret_cast<const h8 *>(qr + 64 * j + 16 * g + 8 * k);
    }
  };

  Unit u;
  if (!next_unit(u)) return;
  for (;;) {
    // the queries are sent for first: their sums are taken while the page's
    // bytes arrive (one token of 4096: 12.8 against 13.0 us).  Not with 32
    // rows, whose registers are short (8 sequences with 4 rows: 28.2 against
    // 27.7 us)
    if (RT == 1) queries(u);
    first_page(u);
    if (RT > 1) queries(u);
    const int s = u.s, h = u.h, pmin = u.pmin, pmax = u.pmax, hi = u.hi;
    const Tiles T = u.T;
    int i = u.i, id;
    State<D> st[RT];
    float qsum[RT], unit = kNoUnit;  // log2 of the outputs' unit
#pragma unroll
    for (int a = 0; a < RT; a++) {
      qsum[a] = 0.0f;
#pragma unroll
      for (int j = 0; j < D / 32; j++)
#pragma unroll
        for (int r = 0; r < 8; r++) {
          qf[a][j][r] = pos[a] >= 0 ? qf[a][j][r] : (_Float16)0.0f;
          qsum[a] += (float)qf[a][j][r];
        }
      qsum[a] = 0.5f * quarter_sum(qsum[a]);
#pragma unroll
      for (int d = 0; d < D / 16; d++) st[a].o[d] = (f4){0, 0, 0, 0};
      st[a].m = kNone;
      st[a].l = st[a].corr = 0.0f;
    }
    for (; i < hi; i += kDecWaves) {
      const bool more = i + kDecWaves < hi;
      const int pg = T.page(i), j0 = pg * kPage, j1 = j0 + kPage - 1;
      const bool masked = !(j1 <= pmin && (A.window == 0 || j0 > pmax - A.window || j1 < A.sinks));
      const float ks = raw.ks, vs = raw.vs;
      f4 x[RT][4];
      scores<D, RT>(raw, qf, x);
      id = id_next;
      if (more) load_keys<D>(A, h, id, raw);
      if (i + 2 * kDecWaves < hi) id_next = page_id<KEYS>(A, s, T.page(i + 2 * kDecWaves));
      if (ks >= 0.0f) {  // wave-uniform, as all of this page's scales
        // a page of zeros has scale 0: its (zero) scores stay finite, masked ones -inf
        const float sc = fmaxf(ks * A.scale_log2, 1e-37f);
        const bool has_v = vs >= kLeastScale;  // a page of zeros adds to the sum only
        const float lv = uniform(__builtin_amdgcn_logf(vs)), over = has_v ? lv - unit : 0.0f;
        const bool far = unit_moves(over);
        const float shift = far ? 0.0f : over;
        const float moves = far ? __builtin_amdgcn_exp2f(-over) : 1.0f;
        if (far) unit = lv;
        h8 hi16[RT][2], lo16[RT][2];
#pragma unroll
        for (int a = 0; a < RT; a++)
          weights<D, RT == 1>(A, x[a], qsum[a], sc, shift, moves, masked, j0 + 16 * g, pos[a], has_v, st[a], hi16[a], lo16[a]);
        if (has_v) {
#pragma unroll
          for (int d = 0; d < D / 16; d++) {
            const uint4 w = raw.v[d];
            const h8 v0 = codes8(w.x, w.y), v1 = codes8(w.z, w.w);
#pragma unroll
            for (int a = 0; a < RT; a++) {
              st[a].o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, hi16[a][0], st[a].o[d], 0, 0, 0);
              st[a].o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, hi16[a][1], st[a].o[d], 0, 0, 0);
              if (RT == 1) {
                st[a].o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, lo16[a][0], st[a].o[d], 0, 0, 0);
                st[a].o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, lo16[a][1], st[a].o[d], 0, 0, 0);
              }
            }
          }
        }
      }
      if (more) load_values<D>(A, h, id, raw);
    }

    // the waves' results meet in LDS (the thread number through an empty asm:
    // what follows is not to be computed ahead of the loop and kept)
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const float unit_scale = __builtin_amdgcn_exp2f(unit);
#pragma unroll
    for (int a = 0; a < RT; a++) {
      const int row = kRows * a + n16;
      const float l = quarter_sum(st[a].l), corr = 0.5f * quarter_sum(st[a].corr);
      if (row < u.nrows) {
#pragma unroll
        for (int d = 0; d < D / 16; d++)
          *reinterpret_cast<f4 *>(&S.w.o[wave][row][16 * d + 4 * g]) = (st[a].o[d] + corr) * unit_scale;
        if (g == 0) {
          S.w.m[wave][row] = st[a].m;
          S.w.l[wave][row] = l;
        }
      }
    }
    __syncthreads();
    // outputs 4 c .. 4 c + 3 of a row, for the rows that are there
    constexpr int kQuads = D / 4, kRound = kDecThreads / kQuads;
    auto token_of = [&](int row) { return u.begin + (int)((uint32_t)(u.f0 + row) / (uint32_t)A.group); };
    auto head_of = [&](int row) { return h * A.group + (int)((uint32_t)(u.f0 + row) % (uint32_t)A.group); };
    auto write_out = [&](int row, int d, f4 o) {
      if constexpr (KEYS == kPrefixKeys) {
        *reinterpret_cast<f4 *>(A.mid + ((int64_t)token_of(row) * (A.hkv * A.group) + head_of(row)) * D + d) = o;
        return;
      }
      const uint32_t f = u.f0 + row;
      _Float16 *dst = A.out + (int64_t)(u.begin + f / (uint32_t)A.group) * A.out_stride +
                      (h * A.group + f % (uint32_t)A.group) * D + d;
      *reinterpret_cast<h4 *>(dst) = (h4){(_Float16)o[0], (_Float16)o[1], (_Float16)o[2], (_Float16)o[3]};
    };
    const int mine = (2 * wg + (u.first == wg)) * PF;
    auto put_sums = [&](int row, float M, float L) {  // (kPrefixKeys)
      float *ml = A.mid + A.mid_ml + 2 * ((int64_t)token_of(row) * (A.hkv * A.group) + head_of(row));
      ml[0] = M;
      ml[1] = L;
    };
    const Before before = KEYS == kOwnKeys ? Before(A, s, D) : Before();
    auto join_row = [&](int row, int j, bool live, float M, float L) {  // (kOwnKeys)
      int64_t o, ml;
      before.at(A, token_of(row), head_of(row), D, o, ml);
      return join_before(A.mid, ml, before, j, live, M, L, pre_w + row * kPrePieces);
    };
    auto taken = [&](int row, int d) {
      int64_t o, ml;
      before.at(A, token_of(row), head_of(row), D, o, ml);
      return take_before(A.mid, o + d, before, pre_w + row * kPrePieces);
    };
    if (KEYS == kOwnKeys && u.pieces == 1) {
      for (int r0 = 0; r0 < u.nrows; r0 += kDecThreads / 16) {
        const int row = r0 + tid / 16, rr = min(row, u.nrows - 1);
        float M = kNone, L = 0.0f;
#pragma unroll
        for (int w = 0; w < kDecWaves; w++) M = fmaxf(M, S.w.m[w][rr]);
#pragma unroll
        for (int w = 0; w < kDecWaves; w++) L += __builtin_amdgcn_exp2f(S.w.m[w][rr] - M) * S.w.l[w][rr];
        const float f = join_row(rr, tid & 15, row < u.nrows, M, L);
        if ((tid & 15) == 0 && row < u.nrows) keep[row] = f;
      }
      __syncthreads();
    }
    for (int row = tid / kQuads; row < u.nrows; row += kRound) {
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
      if (u.pieces > 1) {
        store_dev(parts, mine + row * D + 4 * c, o);
        if (c == 0) store_dev2(parts, mine + R * D + 2 * row, M, L);
      } else {
        if constexpr (KEYS == kPrefixKeys) {
          if (c == 0) put_sums(row, M, L);
          write_out(row, 4 * c, o);
        } else if constexpr (KEYS == kOwnKeys) {
          write_out(row, 4 * c, o * keep[row] + taken(row, 4 * c));
        } else {
          write_out(row, 4 * c, o * inverse(L));
        }
      }
    }
    if constexpr (WHOLE) {
      return;
    } else {
      if (u.pieces > 1 && last_split(A.counters + u.first, u.pieces))
        join<R, D, kDecThreads, kDecPieces + 2>(
            tid, parts, u.pieces, u.nrows, S.join, [&](int k) { return (2 * (u.first + k) + (k == 0)) * PF; },
            [&](int row, int d, f4 o) {
              if constexpr (KEYS == kOwnKeys) o += taken(row, d);
              write_out(row, d, o);
            },
            [&](int row, int j, bool live, float M, float L) {
              if constexpr (KEYS == kPrefixKeys) {
                if (j == 0 && live) put_sums(row, M, L);
                return 1.0f;
              } else if constexpr (KEYS == kOwnKeys) {
                return join_row(row, j, live, M, L);
              } else {
                return inverse(L);
              }
            });
      if (at >= stop) return;
      list.load(A, lane);  // (not kept in registers through the unit)
      next_unit(u);
      __syncthreads();  // LDS is used anew
    }
  }
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
// What else was built: 256 rows and 8 waves with four buffers, which halves the
// conversions (a prompt of 4096 tokens 314 against 323 us, two chunks of 1025
// rows 139 against 119); 64 rows a wave, which halves the LDS reads but leaves
// one wave a SIMD (374 against 309, 173 against 115).
//
// The running maximum is a reference, not the maximum, as in the decode kernel
// (kLift, kTop), and so is the output's unit.
constexpr int kWaveRows = 32;
constexpr int kPreWaves = 4, kTileRows = kPreWaves * kWaveRows;
constexpr int kPreSplits = 16;  // pieces of a tile at most
typedef float f16x __attribute__((ext_vector_type(16)));

// The token of a 32-token group that row r of the score product takes.
__device__ __forceinline__ int row_token(int r) { return (r & 16) + ((r >> 2) & 1) * 8 + ((r >> 3) & 1) * 4 + (r & 3); }

// The 16-byte pieces of a page's keys (and of its values) that a thread of NT fetches.
template <int D, int NT>
constexpr int kPieces = kPage * D / 16 / NT;

// The same bytes of a page, keys or values, on their way into LDS.
template <int D, int NT>
struct Half {
  uint4 r[kPieces<D, NT>];
  __device__ __forceinline__ void load(const uint8_t *p) {
#pragma unroll
    for (int i = 0; i < kPieces<D, NT>; i++) r[i] = reinterpret_cast<const uint4 *>(p)[i * NT + threadIdx.x];
  }
};

template <int D>
struct Lds {
  _Float16 k[kPage][D + 8], v[D][kPage + 8];
};

template <int D, int NT>
__device__ __forceinline__ void put_keys(const Half<D, NT> &t, Lds<D> &l) {
#pragma unroll
  for (int i = 0; i < kPieces<D, NT>; i++) {
    const int idx = i * NT + threadIdx.x;
    h8 *d = reinterpret_cast<h8 *>(&l.k[idx / (D / 16)][idx % (D / 16) * 16]);
    d[0] = codes8(t.r[i].x, t.r[i].y);
    d[1] = codes8(t.r[i].z, t.r[i].w);
  }
}
// (live: the page's scale counts; else its bytes, whatever they are, stand for zeros)
template <int D, int NT>
__device__ __forceinline__ void put_values(const Half<D, NT> &t, bool live, Lds<D> &l) {
  const uint32_t zero = 0x80808080u;
#pragma unroll
  for (int i = 0; i < kPieces<D, NT>; i++) {
    const int idx = i * NT + threadIdx.x;
    h8 *d = reinterpret_cast<h8 *>(&l.v[idx / 4][idx % 4 * 16]);
    d[0] = codes8(live ? t.r[i].x : zero, live ? t.r[i].y : zero);
    d[1] = codes8(live ? t.r[i].z : zero, live ? t.r[i].w : zero);
  }
}

template <int D, int NW, int KEYS = kAllKeys>
__global__ __launch_bounds__(NW * 64, 2) void prefill_kernel(const AttnArgs A) {
  constexpr int kThreads = NW * 64, kTileRows = NW * kWaveRows;
  union Shared {
    Lds<D> page[2];
    struct {
      float join[kJoinFloats<kTileRows, kPreSplits, kThreads>];
      float pre_w[KEYS == kOwnKeys ? kTileRows * kPrePieces : 1], row_ml[KEYS == kOwnKeys ? kTileRows : 1][2];
    } end;
  };
  __shared__ __attribute__((aligned(16))) Shared S;
  const int lane = threadIdx.x & 63, n = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Place P;
  if (!find_place<kTileRows, KEYS>(A, P)) return;
  const int row = wave * kWaveRows + n;
  const bool valid = row < P.nrows;
  const uint32_t fl = P.f0 + (valid ? row : 0);
  const int tok = fl / (uint32_t)A.group, head = P.h * A.group + fl % (uint32_t)A.group;
  const int pos = !valid ? -1 : KEYS == kPrefixKeys ? P.p0 : P.p0 + tok;
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
  // the wave's own rows: positions wmin .. wmax (none: wmax = -1); not below 0,
  // from where a window of 2^31 - 1 could not be taken off
  const int r0 = wave * kWaveRows, r1 = min(r0 + kWaveRows, P.nrows) - 1;
  const int wmin = KEYS == kPrefixKeys ? max(P.p0, 0) : max(P.p0 + (int)((uint32_t)(P.f0 + r0) / (uint32_t)A.group), 0);
  const int wmax = r1 < r0 ? -1 : KEYS == kPrefixKeys ? P.p0 : P.p0 + (int)((uint32_t)(P.f0 + r1) / (uint32_t)A.group);

  f16x o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; i++)
#pragma unroll
    for (int r = 0; r < 16; r++) o[i][r] = 0.0f;
  // keys up to `lowest` are outside the row's window (no window: none are)
  const int lowest = A.window ? pos - A.window : -1;
  float m = kNone, l = 0.0f, corr = 0.0f, unit = kNoUnit;  // unit: its log2

  // A page's scales: the score's factor (finite for a page of zeros, so that a
  // masked score stays -inf), log2 of the value scale (a page of zeros adds to
  // the sum only: its values are put into LDS as zeros).  A page that is not
  // there is read as page 0, whose scales may be anything: none of them counts.
  struct Scales {
    float sc, lv;
    bool there, live;
  };
  auto scales = [&](int id) {
    Scales t;
    const bool ok = id >= 0 && id < A.num_pages;
    const int64_t ph = (int64_t)(ok ? id : 0) * A.hkv + P.h;
    float ks = A.ks[ph], vs = A.vs[ph];
    t.there = ok && ks >= 0.0f;
    // (by a mask: selects spill two registers, 1 x 256 rows on 2000 51.1 against 50.9 us)
    const uint32_t keep = t.there ? 0xffffffffu : 0u;
    ks = __uint_as_float(__float_as_uint(ks) & keep);
    vs = __uint_as_float(__float_as_uint(vs) & keep);
    t.sc = fmaxf(ks * A.scale_log2, 1e-37f);
    t.live = vs >= kLeastScale;
    t.lv = __builtin_amdgcn_logf(vs);
    return t;
  };
  auto key_bytes = [&](int id) { return A.k + ((int64_t)(id >= 0 && id < A.num_pages ? id : 0) * A.hkv + P.h) * (kPage * D); };
  auto value_bytes = [&](int id) { return A.v + ((int64_t)(id >= 0 && id < A.num_pages ? id : 0) * A.hkv + P.h) * (kPage * D); };
  auto id_at = [&](int i) { return page_id<KEYS>(A, P.s, P.T.page(i)); };

  // S^T of a page's keys
  auto dot = [&](const Lds<D> &L, f16x (&acc)[2]) {
#pragma unroll
    for (int t = 0; t < 2; t++) {
#pragma unroll
      for (int r = 0; r < 16; r++) acc[t][r] = 0.0f;
      const _Float16 *kr = &L.k[32 * t + row_token(n)][8 * half];
#pragma unroll
      for (int j = 0; j < D / 16; j++)
        acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(*reinterpret_cast<const h8 *>(kr + 16 * j), qf[j], acc[t], 0, 0, 0);
    }
  };
  auto largest = [&](const f16x (&acc)[2]) {
    float mx = acc[0][0];
#pragma unroll
    for (int r = 1; r < 16; r++) mx = fmaxf(mx, acc[0][r]);
#pragma unroll
    for (int r = 0; r < 16; r++) mx = fmaxf(mx, acc[1][r]);
    return mx;
  };
  // moves the references to a page's scores and value scale; -> log2 of the factor its weights take
  auto refer = [&](const Scales &t, float mx) {
    mx = t.there ? (half_max(mx) + qsum) * t.sc : -__builtin_inff();
    const float over = t.live ? t.lv - unit : 0.0f;
    const bool far = unit_moves(over);
    if (far || __any(mx > m + kTop)) {
      const float mn = mx > m + kTop ? mx - kLift : m;
      float alpha = __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      l *= alpha;
      if (far) {
        alpha *= __builtin_amdgcn_exp2f(-over);
        unit = t.lv;
      }
      corr *= alpha;
#pragma unroll
      for (int d = 0; d < D / 32; d++)
#pragma unroll
        for (int r = 0; r < 16; r++) o[d][r] *= alpha;
    }
    return far ? 0.0f : over;
  };
  // the weights of a page's scores (in fp16), summed into l and corr
  auto weigh = [&](const Scales &t, float shift, const f16x (&acc)[2], h8 (&p)[2][2]) {
    const float bias = t.there ? qsum * t.sc + shift - m : -__builtin_inff();
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 2; k++)
#pragma unroll
      for (int r = 0; r < 16; r++) {
        const float w = __builtin_amdgcn_exp2f(acc[k][r] * t.sc + bias);
        sum += w;
        p[k][r >> 3][r & 7] = (_Float16)w;
      }
    l += sum * __builtin_amdgcn_exp2f(-shift);
    corr += t.live ? sum : 0.0f;
  };
  auto add_values = [&](const Lds<D> &L, const h8 (&p)[2][2]) {
#pragma unroll
    for (int d = 0; d < D / 32; d++)
#pragma unroll
      for (int t = 0; t < 2; t++)
#pragma unroll
        for (int u = 0; u < 2; u++) {
          const h8 a = *reinterpret_cast<const h8 *>(&L.v[32 * d + n][32 * t + 16 * u + 8 * half]);
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, p[t][u], o[d], 0, 0, 0);
        }
  };

  // Pages [ca, cb) of the list are seen whole by every row; the few before
  // (sinks, a window's first pages) and behind (the rows' own) go one by one, with masks.
  int ca = P.T.sink, cb = P.pmin < 0 ? 0 : (P.pmin + 1) / kPage - P.T.first + P.T.sink;
  if (A.window && P.pmax >= A.window) ca = max(ca, (P.pmax - A.window) / kPage + 1 - P.T.first + P.T.sink);
  ca = max(ca, P.lo);
  cb = min(cb, P.hi);
  if (cb - ca < 2) ca = cb = P.hi;
  Half<D, kThreads> rk, rv;
#pragma unroll 1
  for (int part = 0; part < 2; part++) {
    const int lo = part ? cb : P.lo, hi = part ? P.hi : ca;
    if (lo < hi) {
      // one page after the other, the next one's bytes on their way
      int id = id_at(lo), id1 = lo + 1 < hi ? id_at(lo + 1) : 0;
      Scales t = scales(id);
      rk.load(key_bytes(id));
      rv.load(value_bytes(id));
      put_keys<D, kThreads>(rk, S.page[0]);
      put_values<D, kThreads>(rv, t.live, S.page[0]);
      __syncthreads();
#pragma unroll 1
      for (int i = lo; i < hi; i++) {
        const Lds<D> &L = S.page[(i - lo) & 1];
        const bool more = i + 1 < hi;
        if (more) {
          rk.load(key_bytes(id1));
          rv.load(value_bytes(id1));
        }
        const Scales next = scales(id1);
        if (i + 2 < hi) id1 = id_at(i + 2);
        const int j0 = P.T.page(i) * kPage, j1 = j0 + kPage - 1;
        if (t.there && j0 <= wmax && !(A.window && j1 <= wmin - A.window && j0 >= A.sinks)) {
          f16x acc[2];
          h8 p[2][2];
          dot(L, acc);
          // (whole expressions, no short cuts: branches would cost more)
#pragma unroll
          for (int k = 0; k < 2; k++)
#pragma unroll
            for (int r = 0; r < 16; r++) {
              const int j = j0 + 32 * k + (r >> 3) * 16 + 8 * half + (r & 7);
              const bool see = (j <= pos) & ((j > lowest) | (j < A.sinks));
              acc[k][r] = see ? acc[k][r] : -__builtin_inff();
            }
          const float shift = refer(t, largest(acc));
          weigh(t, shift, acc, p);
          add_values(L, p);
        }
        if (more) {
          put_keys<D, kThreads>(rk, S.page[(i + 1 - lo) & 1]);
          put_values<D, kThreads>(rv, next.live, S.page[(i + 1 - lo) & 1]);
          t = next;
        }
        __syncthreads();
      }
    }
    if (part || ca >= cb) continue;
    // The run of whole pages, two pages deep: while page i's weights are made
    // (vector unit) the scores of page i + 1 are (matrix unit), while its values
    // are added (matrix unit) the next pages' bytes are converted into LDS and
    // page i + 1's maximum is taken.  The order is as written, held by the
    // sched_barriers: one product, then what the vector unit does beside it (a
    // prompt of 4096 tokens: 310 us; the compiler's own order 322, patterns of
    // sched_group_barrier 341 to 354).
    const int id0 = id_at(ca);
    int id1 = id_at(ca + 1), id2 = id_at(min(ca + 2, cb - 1)), id3 = id_at(min(ca + 3, cb - 1));
    Scales t = scales(id0), t1;
    rk.load(key_bytes(id0));
    rv.load(value_bytes(id0));
    put_keys<D, kThreads>(rk, S.page[0]);
    put_values<D, kThreads>(rv, t.live, S.page[0]);
    rk.load(key_bytes(id1));
    put_keys<D, kThreads>(rk, S.page[1]);
    rk.load(key_bytes(id2));
    rv.load(value_bytes(id1));
    __syncthreads();
    f16x even[2], odd[2];
    dot(S.page[0], even);
    float shift = refer(t, largest(even));
    __syncthreads();  // page[0]'s keys are read by all
    // page i: `cur` its scores, `here` its values, `there` page i + 1's keys;
    // on their way: the keys of page i + 2 and the values of page i + 1
    auto step = [&](int i, f16x (&cur)[2], f16x (&nxt)[2], Lds<D> &here, Lds<D> &there) {
      t1 = scales(id1);
      // piece u of the 16-byte halves that this thread converts into LDS: keys, then values
      auto put = [&](int u) {
        constexpr int N = 2 * kPieces<D, kThreads>;
        const uint32_t zero = 0x80808080u;
        const int q = u % N / 2, idx = q * kThreads + threadIdx.x;
        const uint4 w = u < N ? rk.r[q] : rv.r[q];
        uint32_t a = u & 1 ? w.z : w.x, b = u & 1 ? w.w : w.y;
        if (u >= N) a = t1.live ? a : zero, b = t1.live ? b : zero;
        h8 *d = u < N ? reinterpret_cast<h8 *>(&here.k[idx / (D / 16)][idx % (D / 16) * 16])
                      : reinterpret_cast<h8 *>(&there.v[idx / 4][idx % 4 * 16]);
        d[u & 1] = codes8(a, b);
      };
      // products of page i + 1's keys and the weights of page i, side by side
      constexpr int NQ = D / 8, E = 32 / NQ, AHEAD = 2;
      const _Float16 *kr = &there.k[row_token(n)][8 * half], *vr = &here.v[n][8 * half];
      // operand z of the score products (32 tokens, then the other 32) and of the value products
      auto key = [&](int z) { return *reinterpret_cast<const h8 *>(kr + z / (D / 16) * 32 * (D + 8) + z % (D / 16) * 16); };
      auto value = [&](int z) { return *reinterpret_cast<const h8 *>(vr + z / 4 * 32 * (kPage + 8) + z % 4 * 16); };
      h8 ops[AHEAD + 1], p[2][2];
      const float bias = t.there ? qsum * t.sc + shift - m : -__builtin_inff();
      float sum = 0.0f;
#pragma unroll
      for (int z = 0; z < AHEAD; z++) ops[z] = key(z);
#pragma unroll
      for (int z = 0; z < NQ; z++) {
        ops[(z + AHEAD) % (AHEAD + 1)] = z + AHEAD < NQ ? key(z + AHEAD) : value(z + AHEAD - NQ);
        const int k = z / (D / 16), jj = z % (D / 16);
        nxt[k] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ops[z % (AHEAD + 1)], qf[jj],
                                                        jj == 0 ? (f16x)(0.0f) : nxt[k], 0, 0, 0);
#pragma unroll
        for (int e = 0; e < E; e++) {
          const int x = z * E + e;
          const float w = __builtin_amdgcn_exp2f(cur[x >> 4][x & 15] * t.sc + bias);
          sum += w;
          p[x >> 4][(x & 15) >> 3][x & 7] = (_Float16)w;
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      l += sum * __builtin_amdgcn_exp2f(-shift);
      corr += t.live ? sum : 0.0f;
      // page i's values; beside them page i + 1's maximum and the bytes for LDS
      float mx = -__builtin_inff();
#pragma unroll
      for (int z = 0; z < NQ; z++) {
        if (z + AHEAD < NQ) ops[(NQ + z + AHEAD) % (AHEAD + 1)] = value(z + AHEAD);
        o[z / 4] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ops[(NQ + z) % (AHEAD + 1)], p[(z >> 1) & 1][z & 1], o[z / 4], 0, 0, 0);
#pragma unroll
        for (int e = 0; e < E; e++) mx = fmaxf(mx, nxt[(z * E + e) >> 4][(z * E + e) & 15]);
        if (z & 1) put(z >> 1);
        // as soon as a half's registers are free its next bytes are sent for
        if (z == NQ / 2) rk.load(key_bytes(id3));
        if (z == NQ - 1) rv.load(value_bytes(id2));
        __builtin_amdgcn_sched_barrier(0);
      }
      id1 = id2;
      id2 = id3;
      id3 = id_at(min(i + 4, cb - 1));
      t = t1;
      if (i + 1 < cb) shift = refer(t, mx);
      __syncthreads();
    };
#pragma unroll 1
    for (int i = ca; i < cb; i += 2) {
      step(i, even, odd, S.page[0], S.page[1]);
      if (i + 1 < cb) step(i + 1, odd, even, S.page[1], S.page[0]);
    }
  }
  l = half_sum(l);
  corr = 0.5f * half_sum(corr);
  unit = __builtin_amdgcn_exp2f(unit);
#pragma unroll
  for (int d = 0; d < D / 32; d++)
#pragma unroll
    for (int r = 0; r < 16; r++) o[d][r] = (o[d][r] + corr) * unit;

  // element r of o[d] is output 32 d + 8 (r / 4) + 4 half + r % 4
  if constexpr (KEYS == kPrefixKeys) {
    // every piece as it is: the launch over the own keys joins them
    float *to = A.mid + ((int64_t)P.tile * A.nsplit + P.split) * partial_floats(kTileRows, D);
    if (valid) {
#pragma unroll
      for (int d = 0; d < D / 32; d++)
#pragma unroll
        for (int r = 0; r < 16; r += 4)
          *reinterpret_cast<f4 *>(to + row * D + 32 * d + 2 * r + 4 * half) =
              (f4){o[d][r], o[d][r + 1], o[d][r + 2], o[d][r + 3]};
      if (half == 0) {
        to[kTileRows * D + 2 * row] = m;
        to[kTileRows * D + 2 * row + 1] = l;
      }
    }
    return;
  }
  const Before before = KEYS == kOwnKeys ? Before(A, P.s, D) : Before();
  auto join_row = [&](int jr, int j, bool live, float M, float L) {  // (kOwnKeys)
    const uint32_t f = P.f0 + jr;
    int64_t at, ml;
    before.at(A, P.begin + f / (uint32_t)A.group, P.h * A.group + f % (uint32_t)A.group, D, at, ml);
    return join_before(A.mid, ml, before, j, live, M, L, S.end.pre_w + jr * kPrePieces);
  };
  if (P.splits > 1) {
    Rsrc base = make_rsrc(A.partials + (int64_t)P.tile * A.nsplit * partial_floats(kTileRows, D));
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
      join<kTileRows, D, kThreads, kPreSplits>(
          threadIdx.x, base, P.splits, P.nrows, S.end.join, [](int k) { return k * partial_floats(kTileRows, D); },
          [&](int jr, int d, f4 v) {
            const uint32_t f = P.f0 + jr;
            const int t = P.begin + f / (uint32_t)A.group, qh = P.h * A.group + f % (uint32_t)A.group;
            if constexpr (KEYS == kOwnKeys) {
              int64_t at, ml;
              before.at(A, t, qh, D, at, ml);
              v += take_before(A.mid, at + d, before, S.end.pre_w + jr * kPrePieces);
            }
            *reinterpret_cast<h4 *>(A.out + (int64_t)t * A.out_stride + qh * D + d) =
                (h4){(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
          },
          [&](int jr, int j, bool live, float M, float L) {
            if constexpr (KEYS == kOwnKeys) return join_row(jr, j, live, M, L);
            else return inverse(L);
          });
    return;
  }
  float inv = inverse(l);
  int64_t pre_o = 0;
  if constexpr (KEYS == kOwnKeys) {
    // 16 lanes a row, its maximum and sum through LDS, the factor on the way back
    if (half == 0) {
      S.end.row_ml[row][0] = m;
      S.end.row_ml[row][1] = l;
    }
    __syncthreads();
    for (int r0 = 0; r0 < P.nrows; r0 += kThreads / 16) {
      const int jr = r0 + threadIdx.x / 16, rr = min(jr, P.nrows - 1);
      const float f = join_row(rr, threadIdx.x & 15, jr < P.nrows, S.end.row_ml[rr][0], S.end.row_ml[rr][1]);
      if ((threadIdx.x & 15) == 0 && jr < P.nrows) S.end.row_ml[jr][1] = f;
    }
    __syncthreads();
    inv = S.end.row_ml[row][1];
    int64_t ml;
    before.at(A, P.begin + tok, head, D, pre_o, ml);
  }
  if (valid) {
    _Float16 *dst = A.out + (int64_t)(P.begin + tok) * A.out_stride + head * D;
#pragma unroll
    for (int d = 0; d < D / 32; d++)
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        f4 v = (f4){o[d][r], o[d][r + 1], o[d][r + 2], o[d][r + 3]} * inv;
        const int e = 32 * d + 2 * r + 4 * half;
        if constexpr (KEYS == kOwnKeys) v += take_before(A.mid, pre_o + e, before, S.end.pre_w + row * kPrePieces);
        *reinterpret_cast<h4 *>(dst + e) = (h4){(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
      }
  }
}

constexpr int kCus = 256;

// The launch of a call: which kernel, its workgroups, how the keys are split,
// and the workspace that needs.
struct Plan {
  int tile_rows;  // 16, 32: decode; 128: prefill
  int64_t wgs, solo;
  int waves;  // of a workgroup
  int nsplit, chunk;
  int whole;  // decode: units of up to so many pages stay whole; 0: all do
  size_t counter_bytes, bytes;
};

Plan make_plan(int64_t rows, int64_t seqs, int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t max_kv) {
  Plan P;
  const int64_t group = q_heads / kv_heads, flat = rows * group;
  // The decode kernel converts a page for each 32 rows, the prefill kernel for
  // 128, but it starts and ends sooner, cuts the keys finer and shares them out
  // by the lengths there are.  It takes (us of decode against prefill; 64 query
  // and 8 KV heads of 128, sequences x rows on up to so many tokens)
  //  - up to 32 (row, query head) rows a sequence;
  //  - up to half a tile of 32 a CU (1 x 16 on 600 12.5 against 21.7, on 6001 25.3
  //    against 56.9; 1 x 64 on 30000 118 against 139), up to a tile a CU on up to
  //    12 K tokens (1 x 96 on 12000 92 against 96, on 30000 213 against 152), up to
  //    two on up to 1024 (1 x 180 on 1000 28.8 against 30.2, on 4000 82 against 62;
  //    1 x 256 on 600 23.5 against 22.7);
  //  - up to two tiles a CU of up to 64 rows a sequence, which fill half of a tile of
  //    128, on more than 3500 tokens (32 x 8 on 4000 87 against 128, on 8000 147
  //    against 183; 24 x 8 on 2000 56 against 47; 24 x 12, three tiles each, on 8000
  //    163 against 146; 64 x 8, four a CU, on 4000 170 against 149).
  // The tiles are counted as of sequences with the same number of rows.
  const int64_t each = (flat + seqs - 1) / seqs, tiles32 = (each + 31) / 32 * seqs * kv_heads;
  const int64_t most = max_kv <= 1024 || (each <= 64 && max_kv > 3500) ? 2 * kCus : max_kv <= 12288 ? kCus : kCus / 2;
  const bool prefill = each > 32 && tiles32 > most;
  const int R = prefill ? kTileRows : flat > kRows * seqs ? 2 * kRows : kRows;
  P.tile_rows = R;
  const int64_t tiles = (max_kv + kPage - 1) / kPage;
  const int64_t full = (flat + R - 1) / R, units = (full > seqs ? full : seqs) * kv_heads;
  P.nsplit = 1;
  P.solo = 0;
  P.chunk = 0x7fffffff;
  P.whole = 0;
  P.waves = prefill ? kPreWaves : kWaves;
  P.counter_bytes = P.bytes = 0;
  if (prefill) {
    // Two workgroups a CU run together.  Full rounds of them take whole units;
    // the rest of a last round is cut into pieces for all CUs.  With many rounds
    // the longest-first order levels the load by itself.
    const int64_t slots = flat / R + seqs, all = slots * kv_heads, round = 2 * kCus;
    const int64_t rest = all < 4 * round ? all % round : 0;
    const int64_t idle = all - units, real = rest > idle ? rest - idle : rest;  // some tiles may hold no row
    int64_t nsplit = rest ? round / real : 1;
    if (nsplit > kPreSplits) nsplit = kPreSplits;
    // (where most of the rest holds no row, what is launched and kept for it is bounded)
    if (rest && nsplit > 2 * round / rest) nsplit = 2 * round / rest;
    if (nsplit > tiles / 4) nsplit = tiles / 4;
    if (rest == all && tiles <= 32 && each >= R) {
      // One round of full tiles and few pages: the number of pieces that should take
      // least, in 10 ns.  A page takes a workgroup 1.25 us alone on its CU and 2.34
      // beside another (64 elements: 0.98 and 1.37, slopes of 1 x 264 and 3 x 264 rows);
      // pieces cost 12 us (64 elements: 3.5, and 0.5 each) and the time of their partial
      // results, 66 (33) KB each, written and read.  (1 x 256 rows on 2000, 64 and 8
      // heads: one piece 49 us, two 47, four 60; 1 x 300, 32 and 8 heads: one 50, two
      // 45, three 42, four 48.  Heads of 64: 1 x 256 on 2000, 64 and 8 heads, one 38, two
      // 33, four 37; 1 x 300, 32 and 8, one 38, three 29, four 32; 1 x 1200, 16 and 4,
      // one 36, three 34; 3 x 300, 24 and 4, one 40, two 43, on 1000 one 23, two 30.
      // More pages: 1 x 180 on 4000 one 92, two 64, five 62; 3 x 200 on 3000, 32 and 8
      // heads, two 73, four 63.  Tiles half empty: 30 x 13 on 2000, 40 and 8 heads, one
      // 63, two 51.)
      const bool wide = head_dim == 128;
      const int64_t pages = tiles - rows / seqs / (2 * kPage);
      int64_t least = 0, best = 1;
      for (int64_t n = 1; n <= nsplit; n++) {
        const int64_t wgs = real * n, page = wgs <= kCus ? (wide ? 125 : 98) : (wide ? 234 : 137);
        const int64_t cut = (wide ? 1200 : 350 + 50 * n) + wgs * head_dim * 27 / 1280;
        const int64_t t = (pages + n - 1) / n * page + (n > 1 ? cut : 0);
        if (n == 1 || t < least) least = t, best = n;
      }
      nsplit = best;
    }
    P.wgs = P.solo = all;
    if (nsplit > 1) {
      P.nsplit = (int)nsplit;
      P.solo = all - rest;
      P.wgs = P.solo + rest * nsplit;
      const int64_t chunk = (tiles + nsplit - 1) / nsplit;
      P.chunk = (int)(chunk < 0x7fffffff ? chunk : 0x7fffffff);
      P.counter_bytes = ((size_t)rest * 4 + 15) / 16 * 16;
      P.bytes = P.counter_bytes + (size_t)rest * nsplit * partial_floats(R, (int)head_dim) * 4;
    }
    return P;
  }
  if (tiles <= kWhole) {
    // eight waves where there is a CU for each unit (9 pages: 9.1 against 9.4
    // us), else four and three workgroups a CU (512 units of up to 11 pages:
    // 17.5 against 23.4 us)
    P.wgs = (flat / R + seqs) * kv_heads;
    if (units > kCus && R == kRows) P.waves = 4;
    return P;
  }
  // one workgroup a CU: a second one's start and end cost more than its
  // waves bring (131001 tokens: 58 against 82 us with two a CU)
  P.whole = kWhole;
  P.wgs = units * ((tiles + kLeast - 1) / kLeast);
  if (P.wgs > kCus) P.wgs = kCus;
  P.counter_bytes = ((size_t)P.wgs * 4 + 15) / 16 * 16;
  P.bytes = P.counter_bytes + (size_t)P.wgs * 2 * partial_floats(R, (int)head_dim) * 4;
  return P;
}

bool aligned_to(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// What the plan sets of a call's arguments, without a window; its words start at ws.
void set_plan(AttnArgs &A, const Plan &P, int64_t seqs, char *ws) {
  A.counters = (uint32_t *)ws;
  A.partials = (float *)(ws + P.counter_bytes);
  A.seqs = (int)seqs;
  A.slots = (int)((int64_t)A.rows * A.group / P.tile_rows + seqs);
  A.nsplit = P.nsplit;
  A.solo = (int)P.solo;
  A.chunk = P.chunk;
  A.whole = P.whole;
}

// Whether its launch is small enough, and (where units are cut their list counts
// the pages of all of them in 32 bits) its units.
bool plan_fits(const Plan &P, int64_t rows, int64_t seqs, int64_t q_heads, int64_t kv_heads, int64_t max_pages) {
  const int64_t units = (rows * (q_heads / kv_heads) / P.tile_rows + seqs) * kv_heads;
  return grid_ok(P.wgs, P.waves * 64) && !(P.whole && units > 0x7fffffff / max_pages);
}

// A plan's launch.
template <int KEYS>
void launch_attn(const Plan &P, int64_t head_dim, const AttnArgs &A, hipStream_t st) {
  const dim3 grid((unsigned)P.wgs), block(P.waves * 64);
#define TQ_ATTN(...) hipLaunchKernelGGL((__VA_ARGS__), grid, block, 0, st, A)
#define TQ_DECODE(D)                                                    \
  if (P.tile_rows == kRows) {                                           \
    if (P.whole) TQ_ATTN(decode_kernel<D, 1, false, kWaves, KEYS>);     \
    else if (P.waves == 4) TQ_ATTN(decode_kernel<D, 1, true, 4, KEYS>); \
    else TQ_ATTN(decode_kernel<D, 1, true, kWaves, KEYS>);              \
  } else {                                                              \
    if (P.whole) TQ_ATTN(decode_kernel<D, 2, false, kWaves, KEYS>);     \
    else TQ_ATTN(decode_kernel<D, 2, true, kWaves, KEYS>);              \
  }
  if (P.tile_rows == kTileRows) {
    if (head_dim == 128) TQ_ATTN(prefill_kernel<128, kPreWaves, KEYS>);
    else TQ_ATTN(prefill_kernel<64, kPreWaves, KEYS>);
  } else if (head_dim == 128) {
    TQ_DECODE(128)
  } else {
    TQ_DECODE(64)
  }
#undef TQ_ATTN
#undef TQ_DECODE
}

}  // namespace
