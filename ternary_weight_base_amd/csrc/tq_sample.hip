// tq_sample.hip -- the next token of each row of logits by temperature, top-k,
// top-p and min-p, from a given uniform number.
//
//   w_i = exp((x_i - max x) / temperature); of the tokens in descending order
//   (equal logits: the lower index first) the first top_k, of these the fewest
//   with a sum of at least top_p of theirs, of these the ones with w >= min_p;
//   the token is the first, in index order, whose running sum exceeds u times
//   the kept tokens' sum.
//
// The kept tokens are all down to a last one in that order (a cut: its logit and
// index) that reach min_p, so no list of them is made.  Weights and sums are in
// double, every sum in a fixed order or of integers: a token's place in the
// running sum decides, and a row's token depends on nothing but the row.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tq.h"
#include "tq_device.h"
#include "tq_wave.h"

namespace {

constexpr int kSeg = 4096;           // tokens of a segment
constexpr int kMaxVocab = 1 << 20;
constexpr int kMaxSegs = kMaxVocab / kSeg;
constexpr int kParts = 64;           // of a power of two, in the table of weights

struct SampleArgs {
  const void *logits;
  const float *temperature, *top_p, *min_p, *u;
  const int *top_k;
  int *token;
  float *logprob;
  int64_t row_stride;
  int rows, vocab;
  int row0, segs;  // a pass over the rows: its first; segments of a row
  bool wide;       // every row aligned to 16 bytes
};

// A row's settings.
struct Rule {
  double per;       // 64 log2 e / temperature
  double top_p, min_p;
  int top_k;        // vocab: all
  bool greedy;
};

__device__ __forceinline__ Rule rule_of(const SampleArgs &A, int row) {
  Rule r;
  const float t = A.temperature ? A.temperature[row] : 1.0f;
  r.greedy = !(t > 0.0f);
  r.per = r.greedy ? 0.0 : kParts * 1.4426950408889634 / (double)t;
  const int k = A.top_k ? A.top_k[row] : 0;
  r.top_k = k > 0 ? min(k, A.vocab) : A.vocab;
  const float p = A.top_p ? A.top_p[row] : 1.0f;
  r.top_p = p < 1.0f ? (double)p : 1.0;
  const float m = A.min_p ? A.min_p[row] : 0.0f;
  r.min_p = m > 0.0f ? fmin((double)m, 1.0) : 0.0;
  return r;
}

// A logit: NaN counts as -inf, -0 as 0.
__device__ __forceinline__ float clean(float x) { return x == x ? x + 0.0f : -__builtin_inff(); }

// Its order as an unsigned integer.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// 2^(t / 64) for t <= 0, to some 2^-51 of it; 0 from 2^-1000 on (and for -inf, NaN): a
// power of two, a 64th of one from a table in LDS and exp's series up to its fifth
// power for the rest, up to (ln 2) / 128 (the next term is below 2^-54).
__device__ __forceinline__ double power2(double t, const double *table) {
  constexpr double c = 0.6931471805599453 / kParts;
  const double u = fmax(t, -1100.0 * kParts), n = rint(u), r = u - n;
  const int k = (int)n;
  const double s = fma(r, fma(r, fma(r, fma(r, fma(r, c * c * c * c * c / 120.0, c * c * c * c / 24.0), c * c * c / 6.0), c * c / 2.0), c), 1.0);
  // (the power of two goes into the exponent: no result is below 2^-1001)
  const uint64_t b = __builtin_bit_cast(uint64_t, s * table[k & (kParts - 1)]) + ((uint64_t)((uint32_t)(k >> 6) << 20) << 32);
  return t > -1000.0 * kParts ? __builtin_bit_cast(double, b) : 0.0;
}

// The table, 2^(i / 64): exp's series at up to 0.3466, whose 14th term is below 2^-57.
struct Powers {
  double v[kParts];
  constexpr Powers() : v() {
    for (int i = 0; i < kParts; i++) {
      const double f = (i < kParts / 2 ? i : i - kParts) * (0.6931471805599453 / kParts);
      double s = 1.0;
      for (int k = 13; k > 0; k--) s = s * f / k + 1.0;
      v[i] = i < kParts / 2 ? s : 2.0 * s;
    }
  }
};
__device__ constexpr Powers kPowers;

// ... into LDS.  (A barrier before its use.)
__device__ __forceinline__ void fill_table(double *table) {
  if (threadIdx.x < kParts) table[threadIdx.x] = kPowers.v[threadIdx.x];
}

// A weight (at most 1) in steps of 1 / steps, a power of two up to 2^48, to the
// nearest: the sum with 2^52 has it in its low bits.
__device__ __forceinline__ uint64_t fixed(double w, double steps) {
  return __builtin_bit_cast(uint64_t, fma(w, steps, 0x1p52)) - __builtin_bit_cast(uint64_t, 0x1p52);
}

// The row's logits as its weights are taken from them: where one is +inf those
// weigh 1 and all others nothing.
struct Weigher {
  float most;
  double per;
  const double *table;
  __device__ __forceinline__ double operator()(float x) const {
    if (most == __builtin_inff()) return x == most ? 1.0 : 0.0;
    return power2(((double)x - (double)most) * per, table);  // (-inf: 0)
  }
};

// What is kept: tokens of a larger key, or of that key up to an index.
struct Cut {
  uint32_t key;
  int index;
  __device__ __forceinline__ bool keeps(uint32_t k, int i) const { return k > key || (k == key && i <= index); }
};

// Sums over a workgroup in a fixed order, for all threads.  `room`: a word a wave.
template <int NT>
__device__ __forceinline__ double block_sum(double v, double *room) {
  v = tqdev::wave_sum64(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) room[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = room[0];
#pragma unroll
  for (int i = 1; i < NT / 64; i++) s += room[i];
  return s;
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)b, lane), hi = __builtin_amdgcn_readlane((int)(b >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// ... of the threads before this one (`all`: of all threads).
template <int NT>
__device__ __forceinline__ double block_before(double v, double *room, double *all = nullptr) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const double sum = tqdev::wave_upto(v);
  __syncthreads();
  if (lane == 63) room[wave] = sum;
  __syncthreads();
  double s = 0.0, t = 0.0;
#pragma unroll
  for (int i = 0; i < NT / 64; i++) {
    s = i == wave ? t : s;
    t += room[i];
  }
  if (all) *all = t;
  return s + (sum - v);
}

// ---- one workgroup a row -----------------------------------------------------

// The cut where the sum of a measure (1 a token, or its weight) reaches
// `target`, among the tokens that `cut` keeps: a radix search over the keys,
// eight bits at a time, then over the indices of the last key.  Weights are
// counted in the smallest steps of which the row's stay in 62 bits.
template <typename T, int NT>
__device__ void narrow(const T *x, int vocab, const Weigher &weigh, bool weights, double target, Cut &cut, uint64_t *hist,
                       double *room) {
  __shared__ uint32_t found;
  __shared__ double left;
  __shared__ int last;
  uint32_t prefix = 0;
  double rest = target;
  const int bits = min(62 - (32 - __builtin_clz(vocab)), 48);
  const double steps = weights ? ldexp(1.0, bits) : 1.0, unit = weights ? ldexp(1.0, -bits) : 1.0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += NT) hist[i] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0 : ~0u << (shift + 8);
    for (int i = threadIdx.x; i < vocab; i += NT) {
      const float v = clean((float)x[i]);
      const uint32_t k = key_of(v);
      if (v > -__builtin_inff() && (k & mask) == prefix && cut.keeps(k, i))
        atomicAdd((unsigned long long *)&hist[k >> shift & 255], weights ? (unsigned long long)fixed(weigh(v), steps) : 1ull);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      int d = 255, some = -1;
      for (; d >= 0; d--) {
        const double h = (double)hist[d] * unit;
        if (hist[d]) {
          some = d;
          if (h >= rest) break;
          rest -= h;
        }
      }
      // (the target is never reached by a rounding of sums: the last token there is)
      if (d < 0 && some >= 0) rest += (double)hist[some] * unit;
      found = prefix | (uint32_t)(d < 0 ? max(some, 0) : d) << shift;
      left = rest;
    }
    __syncthreads();
    prefix = found;
    rest = left;
    __syncthreads();
  }
  // equal keys: as many, in index order, as reach what is left
  const uint32_t b = prefix & 0x80000000u ? prefix & 0x7fffffffu : ~prefix;
  const double each = weights ? weigh(__uint_as_float(b)) : 1.0;
  const double need = each > 0.0 ? ceil(rest / each) : (double)vocab;
  const int want = (int)fmin(fmax(need, 1.0), (double)vocab);
  int before = 0;
  if (threadIdx.x == 0) last = -1;
  for (int i0 = 0; i0 < vocab && before < want; i0 += NT) {
    const int i = i0 + threadIdx.x;
    const bool same = i < vocab && key_of(clean((float)x[i])) == prefix && cut.keeps(prefix, i);
    const int at = before + (int)block_before<NT>(same ? 1.0 : 0.0, room);
    if (same && at < want) atomicMax(&last, i);
    before += (int)block_sum<NT>(same ? 1.0 : 0.0, room);
  }
  __syncthreads();
  cut.key = prefix;
  cut.index = last;
  __syncthreads();
}

// A segment's logits into LDS, -inf behind the vocabulary; `wide`: rows aligned to
// 16 bytes.
template <typename T, int NT>
__device__ __forceinline__ void stage(const T *x, bool wide, int vocab, int seg, float *xs) {
  constexpr int kV = (int)(16 / sizeof(T)) < kSeg / NT ? 16 / sizeof(T) : kSeg / NT;
  typedef T Wide __attribute__((ext_vector_type(kV)));
  const int tid = threadIdx.x;
  x += seg * kSeg;
  if (wide && (seg + 1) * kSeg <= vocab) {
    Wide v[kSeg / NT / kV];
#pragma unroll
    for (int i = 0; i < kSeg / NT / kV; i++) v[i] = reinterpret_cast<const Wide *>(x)[i * NT + tid];
#pragma unroll
    for (int i = 0; i < kSeg / NT / kV; i++)
#pragma unroll
      for (int j = 0; j < kV; j++) xs[(i * NT + tid) * kV + j] = clean((float)v[i][j]);
  } else {
    const int n = vocab - seg * kSeg;
    T v[kSeg / NT];
#pragma unroll
    for (int i = 0; i < kSeg / NT; i++) v[i] = i * NT + tid < n ? x[i * NT + tid] : (T)-__builtin_inff();
#pragma unroll
    for (int i = 0; i < kSeg / NT; i++) xs[i * NT + tid] = clean((float)v[i]);
  }
}

// Where a running sum over the lanes from `before` on exceeds `target`: the first
// lane, or the last one that adds something; the sum before it.
__device__ __forceinline__ int crossing(double own, double before, double target, double &from) {
  const double upto = before + tqdev::wave_upto(own);
  const uint64_t some = __ballot(own > 0.0), above = __ballot(own > 0.0 && upto > target);
  const int at = above ? __builtin_ctzll(above) : some ? 63 - __builtin_clzll(some) : 0;
  from = lane_value(upto - own, at);
  return at;
}

// The token of a segment (its logits in LDS) at which the running sum from
// `before` on exceeds `target`: the first one, or the last that weighs something;
// its weight.  A wave has 64 consecutive tokens of each NT.
template <int NT>
__device__ int pick(const float *xs, int seg, const Weigher &weigh, const Cut &cut, double min_p, double before, double target,
                    double &weight) {
  constexpr int kCells = kSeg / 64;
  __shared__ double cell[kCells];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  auto weight_of = [&](int i) {
    const float c = xs[i];
    double w = 0.0;
    if (cut.keeps(key_of(c), seg * kSeg + i)) {
      w = weigh(c);
      if (!(w >= min_p)) w = 0.0;
    }
    return w;
  };
  __syncthreads();
#pragma unroll 4
  for (int j = 0; j < kCells / (NT / 64); j++) {
    const int i = j * (NT / 64) + wave;
    const double sum = tqdev::wave_sum64(weight_of(i * 64 + lane));
    if (lane == 0) cell[i] = sum;
  }
  __syncthreads();
  // the cell that crosses the target, or the last with a sum: every wave finds it
  static_assert(kCells == 64, "a cell a lane");
  double from;
  const int at = crossing(cell[lane], before, target, from);
  const double w = weight_of(at * 64 + lane);
  const int l = crossing(w, from, target, from);
  weight = lane_value(w, l);
  return seg * kSeg + at * 64 + l;
}

__device__ __forceinline__ void answer(const SampleArgs &A, int row, int token, double weight, double total) {
  A.token[row] = token;
  if (A.logprob) A.logprob[row] = token < 0 ? -__builtin_inff() : weight == total ? 0.0f : (float)log(weight / total);
}

// The segment in which the running sum of the segments' sums (in LDS) exceeds u
// times all of them; the sum before it, that target and all.
__device__ int find_segment(float u, int segs, const double *seg_sum, double &from, double &target, double &total) {
  // every wave finds it by itself: a lane has four of them
  static_assert(kMaxSegs <= 256, "four segments a lane");
  const int lane = threadIdx.x & 63;
  double mine[4], own = 0.0;
#pragma unroll
  for (int j = 0; j < 4; j++) {
    mine[j] = 4 * lane + j < segs ? seg_sum[4 * lane + j] : 0.0;
    own += mine[j];
  }
  const double upto = tqdev::wave_upto(own);
  total = lane_value(upto, 63);
  // (from u = 1 on nothing crosses, whatever the sums' roundings: the last that weighs something)
  target = u >= 1.0f ? (double)__builtin_inff() : (u > 0.0f ? (double)u : 0.0) * total;
  double r = upto - own, before_above = 0.0, before_some = 0.0;
  int above = -1, some = -1;
#pragma unroll
  for (int j = 0; j < 4; j++) {
    if (mine[j] > 0.0) {
      if (above < 0 && r + mine[j] > target) {
        above = j;
        before_above = r;
      }
      some = j;
      before_some = r;
    }
    r += mine[j];
  }
  const uint64_t has_above = __ballot(above >= 0), has_some = __ballot(some >= 0);
  const int l = has_above ? __builtin_ctzll(has_above) : has_some ? 63 - __builtin_clzll(has_some) : 0;
  from = lane_value(has_above ? before_above : before_some, l);
  return 4 * l + max(__builtin_amdgcn_readlane(has_above ? above : some, l), 0);
}

// The token from the segments' sums of kept weights (in LDS); xs: room for a
// segment's logits.
template <typename T, int NT>
__device__ void choose(const SampleArgs &A, int row, int segs, const double *seg_sum, const Weigher &weigh, const Cut &cut,
                       double min_p, float *xs) {
  double from, target, total, weight;
  const int seg = find_segment(A.u[row], segs, seg_sum, from, target, total);
  stage<T, NT>((const T *)A.logits + row * A.row_stride, A.wide, A.vocab, seg, xs);
  const int i = pick<NT>(xs, seg, weigh, cut, min_p, from, target, weight);
  if (threadIdx.x == 0) answer(A, row, i, weight, total);
}

// A row's token by one workgroup: where the segments' way (below) does not lead
// on, and for vocabularies of one segment without limits.
template <typename T, int NT>
__device__ void whole_row(const SampleArgs &A, int row, const double *table, float *xs) {
  __shared__ uint64_t hist[256];
  __shared__ double room[NT / 64], seg_sum[kMaxSegs];
  __shared__ float wave_most[NT / 64];
  __shared__ int where;
  const int tid = threadIdx.x, vocab = A.vocab;
  const T *x = (const T *)A.logits + row * A.row_stride;
  const Rule rule = rule_of(A, row);
  float most = -__builtin_inff();
  for (int i = tid; i < vocab; i += NT) most = fmaxf(most, clean((float)x[i]));
  most = tqdev::wave_max64(most);
  __syncthreads();
  if ((tid & 63) == 0) wave_most[tid >> 6] = most;
  if (tid == 0) where = 0x7fffffff;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NT / 64; i++) most = fmaxf(most, wave_most[i]);
  if (rule.greedy || most == -__builtin_inff()) {
    for (int i = tid; i < vocab; i += NT)
      if (clean((float)x[i]) == most) {
        atomicMin(&where, i);
        break;
      }
    __syncthreads();
    if (tid == 0) answer(A, row, most == -__builtin_inff() ? -1 : where, 1.0, 1.0);
    return;
  }
  const Weigher weigh = {most, rule.per, table};
  Cut cut = {0, -1};
  if (rule.top_k < vocab) narrow<T, NT>(x, vocab, weigh, false, (double)rule.top_k, cut, hist, room);
  if (rule.top_p < 1.0) {
    double sum = 0.0;
    for (int i = tid; i < vocab; i += NT) {
      const float v = clean((float)x[i]);
      if (cut.keeps(key_of(v), i)) sum += weigh(v);
    }
    sum = block_sum<NT>(sum, room);
    narrow<T, NT>(x, vocab, weigh, true, rule.top_p * sum, cut, hist, room);
  }
  const int segs = (vocab + kSeg - 1) / kSeg;
  for (int s = 0; s < segs; s++) {
    double sum = 0.0;
    for (int i = s * kSeg + tid; i < min(vocab, (s + 1) * kSeg); i += NT) {
      const float v = clean((float)x[i]);
      const double w = weigh(v);
      if (cut.keeps(key_of(v), i) && w >= rule.min_p) sum += w;
    }
    sum = block_sum<NT>(sum, room);
    if (tid == 0) seg_sum[s] = sum;
  }
  __syncthreads();
  choose<T, NT>(A, row, segs, seg_sum, weigh, cut, rule.min_p, xs);
}

template <typename T, int NT>
__global__ __launch_bounds__(NT) void row_kernel(const SampleArgs A) {
  __shared__ __attribute__((aligned(16))) float xs[kSeg];
  __shared__ double table[kParts];
  fill_table(table);  // (whole_row has barriers before its first use)
  whole_row<T, NT>(A, blockIdx.x, table, xs);
}

// ---- a workgroup a segment -----------------------------------------------------
//
// Four launches, two with a workgroup a segment and two with one a row behind them:
//  - each segment's largest logit and, in units of its weight, either the sum of
//    its weights or how many tokens (and what weight) fall into each of 255 steps
//    of the logits;
//  - a row without limits gets its token; else the step is found in which the
//    limit falls;
//  - the tokens of that step (top-k up to kFewK: of all steps down to it) are
//    gathered, with their weights and 256ths of the step, and each segment's weights
//    in the steps above summed;
//  - the gathered ones are narrowed down by the 256ths, what is left is sorted and
//    cut, and the token taken.
// A row that gathers more than kGather tokens or has more than kSort left (flat
// logits), or has a top_k above kFewK and top_p too, is done by the last launch's
// workgroup alone, as above: one row of 131072 logits by top-k and top-p takes 26 us
// with a top_k of 1024 and 853 with 1025, 64 rows 35 and 991 (kFewK tokens are two
// a thread of that launch; top-k beyond it alone 26 and 39).  Bound: a row's workgroups by their instructions (a CU
// issues one a cycle) and dependent trips to memory, the segments' for many rows by
// the weights in double (64 rows of 131072 by top-p: 18 us, by top-k, which needs none
// there, 9, reading 34 MB).  (Instead of the launches for a row, the last of its
// segments' workgroups did their work at first: 64 against 51 us for 64 rows, since
// what it meets in had to be written past the caches and its room in LDS was
// every workgroup's.)

constexpr int kThreads = 256, kOwn = kSeg / kThreads;
constexpr int kLast = 512;      // threads of the last launch (one row 22 us; 1024: 23, 256: 24)
constexpr int kSteps = 256;     // the last one: everything below the others
constexpr int kGather = 16384;  // tokens of a row
constexpr int kSort = 4096;     // ... of them sorted
constexpr int kFewK = 1024;
// Threads of the second launch, steps that they take at once (256 threads: 64 rows by
// top-p 55 against 51 us; 1024: 53, and one row 22 against 21).
constexpr int kLimit = 512, kQuarters = 4, kTogether = kLimit / kQuarters;
constexpr int kLine = 32;       // words of a cache line
constexpr double kFixed = 0x1p48;  // weights as integers: kGather of them stay in 62 bits

enum Mode { kDone = 0, kTopK, kManyK, kTopP, kMinP, kAlone };

__device__ __forceinline__ int mode_of(const SampleArgs &A, const Rule &r) {
  const bool by_k = r.top_k < A.vocab, by_p = r.top_p < 1.0;
  if (r.greedy) return kDone;
  if (by_k) return r.top_k <= kFewK ? kTopK : by_p ? kAlone : kManyK;
  return by_p ? kTopP : r.min_p > 0.0 ? kMinP : kDone;
}

struct SegInfo {
  float most;
  int index;   // of the largest logit, where that is the answer
  double sum;  // of the segment's weights, in units of its largest one's
};

// What the later launches have to know of a row.
struct RowInfo {
  int mode;
  float most;
  int step;      // the gathered step
  int top_step;  // of the largest logit
  double left;   // top_k's tokens, or top_p's sum, to be found in that step
};

// The workspace: all zero between calls.
struct SampleWs {
  int64_t room;        // tokens gathered of a row at most: kGather, or all
  RowInfo *info;
  SegInfo *seg;
  double *seg_sum;
  uint32_t *found;     // a row's gathered tokens, a cache line each (one line for 32 rows: 24 against 14 us)
  uint32_t *count;     // [row][segment][step]
  uint64_t *weight;
  uint64_t *gathered;  // [row][room]: key, then the index's complement
  uint64_t *worth;     // ... with its 256th of the step, whether it reaches min_p, its weight (kTopP, kManyK)
};

// The steps are of an eighth of a logit (for top-p of the temperature, where that
// is below 1): the 255 reach 32 logits, or weights of 2^-46, down.  Rounding keeps
// the order, and segments count from steps of the same grid.
struct Steps {
  float per;
  __device__ __forceinline__ Steps(const Rule &r, int mode)
      : per(mode == kTopP ? fminf(8.0f * fmaxf((float)(r.per * (0.6931471805599453 / kParts)), 1.0f), 1e30f) : 8.0f) {}
  __device__ __forceinline__ int operator()(float x) const { return (int)floorf(fminf(fmaxf(x * per, -1e9f), 1e9f)); }
  // the 256th of step `at` (of the grid) that x lies in, from its upper end; below the step: the last
  __device__ __forceinline__ int part(float x, int at) const {
    const float f = (fminf(fmaxf(x * per, -1e9f), 1e9f) - (float)at) * 256.0f;
    return 255 - (int)fminf(fmaxf(f, 0.0f), 255.0f);
  }
};

template <int NT>
__device__ __forceinline__ float block_most(float v, float *room) {
  v = tqdev::wave_max64(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) room[threadIdx.x >> 6] = v;
  __syncthreads();
  v = room[0];
#pragma unroll
  for (int i = 1; i < NT / 64; i++) v = fmaxf(v, room[i]);
  return v;
}

// A thread's logits of a segment, -inf behind the vocabulary.
template <typename T>
struct Own {
  static constexpr int kV = 16 / sizeof(T);
  float v[kOwn];
  bool packed;  // 16 bytes of consecutive ones at a time
  __device__ __forceinline__ Own(const SampleArgs &A, int row, int seg) {
    typedef T Wide __attribute__((ext_vector_type(kV)));
    const T *x = (const T *)A.logits + row * A.row_stride + seg * kSeg;
    const int n = A.vocab - seg * kSeg, tid = threadIdx.x;
    packed = A.wide && n >= kSeg;
    if (packed) {
      Wide w[kOwn / kV];
#pragma unroll
      for (int i = 0; i < kOwn / kV; i++) w[i] = reinterpret_cast<const Wide *>(x)[i * kThreads + tid];
#pragma unroll
      for (int i = 0; i < kOwn; i++) v[i] = clean((float)w[i / kV][i % kV]);
    } else {
      T w[kOwn];
#pragma unroll
      for (int i = 0; i < kOwn; i++) w[i] = i * kThreads + tid < n ? x[i * kThreads + tid] : (T)-__builtin_inff();
#pragma unroll
      for (int i = 0; i < kOwn; i++) v[i] = clean((float)w[i]);
    }
  }
  // Four at a time, the next ones moved down: f(value, number in the thread).  (All
  // at once are so much code that fetching it takes longer than the moves.)
  template <typename F>
  __device__ __forceinline__ void each(const F &f) {
#pragma unroll 1
    for (int g = 0; g < kOwn; g += 4) {
#pragma unroll
      for (int j = 0; j < 4; j++) f(v[j], g + j);
#pragma unroll
      for (int j = 4; j < kOwn; j++) v[j - 4] = v[j];
    }
  }
  // the place of the j-th in the segment
  __device__ __forceinline__ int at(int j) const {
    const int tid = threadIdx.x;
    return packed ? (j / kV * kThreads + tid) * kV + j % kV : j * kThreads + tid;
  }
};

template <typename T>
__global__ __launch_bounds__(kThreads) void segment_kernel(const SampleArgs A, const SampleWs W) {
  __shared__ uint32_t count[kSteps];
  __shared__ unsigned long long weight[kSteps];
  __shared__ double room[kThreads / 64], table[kParts];
  __shared__ float froom[kThreads / 64];
  __shared__ int where;
  const int tid = threadIdx.x, segs = A.segs;
  const int rel = blockIdx.x / (uint32_t)segs, seg = blockIdx.x % (uint32_t)segs, row = A.row0 + rel;
  Own<T> x(A, row, seg);
  const Rule rule = rule_of(A, row);
  const int mode = mode_of(A, rule);
  const Steps step(rule, mode);
  if (mode == kDone || mode == kTopP) fill_table(table);
  if (tid == 0) where = 0x7fffffff;
  count[tid] = 0;
  weight[tid] = 0;
  __syncthreads();
  float most = x.v[0];
#pragma unroll
  for (int j = 1; j < kOwn; j++) most = fmaxf(most, x.v[j]);
  most = block_most<kThreads>(most, froom);
  const Weigher weigh = {most, rule.per, table};
  SegInfo mine = {most, 0, 0.0};
  const int64_t at = (int64_t)rel * segs + seg;
  if (rule.greedy) {
    int first = kSeg;
#pragma unroll
    for (int j = kOwn - 1; j >= 0; j--) first = x.v[j] == most ? x.at(j) : first;
    if (first < kSeg) atomicMin(&where, seg * kSeg + first);
    __syncthreads();
    mine.index = where;
  } else if (mode == kDone) {
    double sum = 0.0;
    x.each([&](float v, int) { sum += weigh(v); });
    mine.sum = block_sum<kThreads>(sum, room);
  } else if (mode == kTopK || mode == kManyK || mode == kTopP) {
    // (a thread's run of the same step is added at once: equal logits would queue)
    const int top = step(most);
    const bool weights = mode == kTopP;
    int run = -1;
    unsigned long long sum = 0;
    auto add = [&]() {
      if (run < 0) return;
      if (weights) atomicAdd(&weight[run], sum);
      else atomicAdd(&count[run], (uint32_t)sum);
    };
    x.each([&](float v, int) {
      if (!(v > -__builtin_inff())) return;
      const int b = min(top - step(v), kSteps - 1);
      if (b != run) {
        add();
        run = b;
        sum = 0;
      }
      sum += weights ? fixed(weigh(v), kFixed) : 1ull;
    });
    add();
    __syncthreads();
    if (!weights) {
      W.count[at * kSteps + tid] = count[tid];
    } else {
      W.weight[at * kSteps + tid] = weight[tid];
      mine.sum = block_sum<kThreads>((double)weight[tid] / kFixed, room);
    }
  }
  if (tid == 0) W.seg[at] = mine;
}

template <typename T>
__global__ __launch_bounds__(kLimit) void limit_kernel(const SampleArgs A, const SampleWs W) {
  __shared__ __attribute__((aligned(16))) float xs[kSeg];
  __shared__ double room[kLimit / 64], seg_sum[kMaxSegs], share[kMaxSegs], part[kQuarters][kTogether], upto[kTogether], table[kParts];
  __shared__ float froom[kLimit / 64];
  __shared__ int seg_step[kMaxSegs], first[kTogether / 64], where;
  const int tid = threadIdx.x, segs = A.segs, rel = blockIdx.x, row = A.row0 + rel;
  SegInfo mine = {-__builtin_inff(), 0, 0.0};
  if (tid < segs) mine = W.seg[(int64_t)rel * segs + tid];
  const Rule rule = rule_of(A, row);
  const int mode = mode_of(A, rule);
  const Steps step(rule, mode);
  fill_table(table);
  if (tid == 0) where = 0x7fffffff;
  const float most = block_most<kLimit>(mine.most, froom);
  const bool none = most == -__builtin_inff();
  const Weigher weigh = {most, rule.per, table};
  const int top = step(most);
  if (tid < segs) {
    share[tid] = weigh(mine.most);  // of a segment's unit
    seg_sum[tid] = mine.sum * share[tid];
    // (a segment without a token that may come counts from far below)
    seg_step[tid] = mine.most == -__builtin_inff() ? 2 * kSteps : min(top - step(mine.most), 2 * kSteps);
    // (the next launch takes, and clears, what it needs to sum the weights above a step)
    const bool more = mode == kTopP && !none;
    W.seg[(int64_t)rel * segs + tid] = SegInfo{0.0f, more ? seg_step[tid] : 0, more ? share[tid] : 0.0};
    if (mine.most == most) atomicMin(&where, mine.index);
  }
  __syncthreads();
  if (none || rule.greedy) {
    if (tid == 0) answer(A, row, none ? -1 : where, 1.0, 1.0);
    return;
  }
  if (mode == kDone) {
    choose<T, kLimit>(A, row, segs, seg_sum, weigh, Cut{0, -1}, 0.0, xs);
    return;
  }
  RowInfo info = {mode, most, kSteps - 1, top, 0.0};
  if (mode == kTopK || mode == kManyK || mode == kTopP) {
    // kTogether steps at a time (mostly the first ones are enough, and one workgroup
    // reads them slowly), a thread a step and a quarter of the segments
    const uint32_t *c = W.count + (int64_t)rel * segs * kSteps;
    const uint64_t *w = W.weight + (int64_t)rel * segs * kSteps;
    const int at = tid % kTogether, quarter = tid / kTogether;
    double target = (double)rule.top_k, before = 0.0;
    if (mode == kTopP) target = rule.top_p * block_sum<kLimit>(tid < segs ? seg_sum[tid] : 0.0, room);
#pragma unroll 1
    for (int s0 = 0; s0 < kSteps; s0 += kTogether) {
      const int t = s0 + at;
      double have = 0.0;
      if (mode == kTopP) {
#pragma unroll 8
        for (int i = quarter; i < segs; i += kQuarters) {
          const int b = t - seg_step[i];
          const uint64_t v = w[i * kSteps + max(b, 0)];
          have += b >= 0 ? (double)v / kFixed * share[i] : 0.0;
        }
      } else {
#pragma unroll 8
        for (int i = quarter; i < segs; i += kQuarters) {
          const int b = t - seg_step[i];
          const uint32_t v = c[i * kSteps + max(b, 0)];
          have += b >= 0 ? (double)v : 0.0;
        }
      }
      part[quarter][at] = have;
      __syncthreads();
      have = 0.0;
      // (the last step is not whole: other segments' last steps belong to it too)
      if (tid < kTogether && t < kSteps - 1) have = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
      double all;
      const double from = before + block_before<kLimit>(have, room, &all);
      const uint64_t there = __ballot(have > 0.0 && from + have >= target);
      if (tid < kTogether) {
        if ((tid & 63) == 0) first[tid / 64] = there ? tid + __builtin_ctzll(there) : kTogether;
        upto[tid] = from;
      }
      __syncthreads();
      int to = kTogether;
#pragma unroll
      for (int i = 0; i < kTogether / 64; i++) to = min(to, first[i]);
      if (to < kTogether) {
        info.step = s0 + to;
        before = upto[to];
        break;
      }
      before += all;  // (nothing above reaches the target: the last step)
    }
    info.left = target - before;
  }
  if (tid == 0) W.info[rel] = info;
}

__device__ __forceinline__ float logit_of(uint64_t entry) {  // of a key and index
  const uint32_t k = (uint32_t)(entry >> 32);
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// A weight in steps; what weighs something has one, so that with u of 1 the last kept
// token is taken.
__device__ __forceinline__ uint64_t steps_of(double w) { return max(fixed(w, kFixed), (uint64_t)1); }
constexpr int kPartBit = 56, kKeepBit = 55;  // above a weight of at most 2^48 steps

template <typename T>
__global__ __launch_bounds__(kThreads) void gather_kernel(const SampleArgs A, const SampleWs W) {
  __shared__ double room[kThreads / 64], table[kParts];
  __shared__ int base;
  const int tid = threadIdx.x, segs = A.segs;
  const int rel = blockIdx.x / (uint32_t)segs, seg = blockIdx.x % (uint32_t)segs, row = A.row0 + rel;
  const RowInfo info = W.info[rel];
  if (info.mode == kDone || info.mode == kAlone) return;
  const int64_t at = (int64_t)rel * segs + seg;
  Own<T> x(A, row, seg);
  const Rule rule = rule_of(A, row);
  const Steps step(rule, info.mode);
  const Weigher weigh = {info.most, rule.per, table};
  // the weights above the step: of top-p from the segment's steps, else one by one
  const bool by_steps = info.mode == kTopP && rule.min_p == 0.0;
  double sum = 0.0;
  if (info.mode == kTopP) {
    const SegInfo mine = W.seg[at];
    if (tid < info.step - mine.index) sum = (double)W.weight[at * kSteps + tid] / kFixed * mine.sum;
    if (!by_steps) sum = 0.0;
    W.weight[at * kSteps + tid] = 0;
  } else if (info.mode != kMinP) {
    W.count[at * kSteps + tid] = 0;
  }
  if (info.mode != kTopK) fill_table(table);
  __syncthreads();
  if (info.mode == kTopP && tid == 0) W.seg[at] = SegInfo{0.0f, 0, 0.0};
  uint32_t mine = 0;  // this thread's tokens that are gathered
  if (info.mode == kTopK || by_steps) {
#pragma unroll
    for (int j = 0; j < kOwn; j++) {
      const int b = min(info.top_step - step(x.v[j]), kSteps - 1);
      if (x.v[j] > -__builtin_inff() && (info.mode == kTopK ? b <= info.step : b == info.step)) mine |= 1u << j;
    }
  } else {
    Own<T> y = x;
    y.each([&](float v, int j) {
      const int b = info.mode == kMinP ? -1 : min(info.top_step - step(v), kSteps - 1);
      if (!(v > -__builtin_inff()) || b > info.step) return;
      if (b == info.step) {
        mine |= 1u << j;
      } else {
        const double w = weigh(v);
        if (w >= rule.min_p) sum += w;
      }
    });
  }
  if (info.mode != kTopK) {
    sum = block_sum<kThreads>(sum, room);
    if (tid == 0) W.seg_sum[at] = sum;
  }
  double all;
  int to = (int)block_before<kThreads>((double)__popc(mine), room, &all);
  if (all == 0.0) return;
  if (tid == 0) base = (int)atomicAdd(W.found + rel * kLine, (uint32_t)all);
  __syncthreads();
  to += base;
  uint64_t *gathered = W.gathered + (int64_t)rel * W.room;
  uint64_t *worth = W.worth + (int64_t)rel * W.room;
#pragma unroll
  for (int j = 0; j < kOwn; j++)
    if (mine >> j & 1) {
      if (to < kGather) gathered[to] = (uint64_t)key_of(x.v[j]) << 32 | (uint32_t)~(seg * kSeg + x.at(j));
      to++;
    }
  if (info.mode == kTopK) return;
  // (their weights once they lie next to each other: few lanes have one at the same j)
  __syncthreads();
  for (int i = base + tid; i < min(base + (int)all, kGather); i += kThreads) {
    const float v = logit_of(gathered[i]);
    const double w = weigh(v);
    worth[i] = (uint64_t)step.part(v, info.top_step - info.step) << kPartBit | (uint64_t)(w > 0.0 && w >= rule.min_p) << kKeepBit | steps_of(w);
  }
}

// Sorts n <= kSort words in descending order (room behind them for the next
// power of two).
__device__ __forceinline__ void sort_equal(uint64_t *v, int n) {
  int size = 64;
  while (size < n) size *= 2;
  for (int i = n + threadIdx.x; i < size; i += kLast) v[i] = 0;
  __syncthreads();
  for (int k = 2; k <= size; k *= 2)
    for (int j = k / 2; j > 0; j /= 2) {
      for (int t = threadIdx.x; t < size / 2; t += kLast) {
        const int a = 2 * t - (t & (j - 1)), b = a + j;  // the bit of j clear, set
        const uint64_t x = v[a], y = v[b];
        if ((x < y) == ((a & k) == 0)) {
          v[a] = y;
          v[b] = x;
        }
      }
      __syncthreads();
    }
}

// The same for up to kSort / 2 words, `other` with room for as many: by kLast equal
// parts of the range between the least and the largest logit, and within a part by
// counting larger ones; where a part holds many (nearly equal logits) as above.
__device__ __forceinline__ void sort_down(uint64_t *v, uint64_t *other, int n, double *room) {
  constexpr int kCrowd = 64;
  __shared__ int count[kLast], next[kLast], crowded;
  __shared__ float ends[kLast / 64][2];
  const int tid = threadIdx.x;
  float lo = __builtin_inff(), hi = -__builtin_inff();
  for (int i = tid; i < n; i += kLast) {
    lo = fminf(lo, logit_of(v[i]));
    hi = fmaxf(hi, logit_of(v[i]));
  }
  hi = tqdev::wave_max64(hi);
  lo = -tqdev::wave_max64(-lo);
  if ((tid & 63) == 0) {
    ends[tid >> 6][0] = lo;
    ends[tid >> 6][1] = hi;
  }
  count[tid] = 0;
  if (tid == 0) crowded = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kLast / 64; i++) {
    lo = fminf(lo, ends[i][0]);
    hi = fmaxf(hi, ends[i][1]);
  }
  const float per = hi > lo ? (float)kLast / (hi - lo) : 0.0f;
  auto part = [&](uint64_t e) { return (int)fminf(fmaxf((hi - logit_of(e)) * per, 0.0f), (float)(kLast - 1)); };
  for (int i = tid; i < n; i += kLast) atomicAdd(&count[part(v[i])], 1);
  __syncthreads();
  const int mine = count[tid];
  if (mine > kCrowd) crowded = 1;
  next[tid] = (int)block_before<kLast>((double)mine, room);
  __syncthreads();
  if (crowded) {
    sort_equal(v, n);
    return;
  }
  for (int i = tid; i < n; i += kLast) other[atomicAdd(&next[part(v[i])], 1)] = v[i];
  __syncthreads();
  for (int i = tid; i < n; i += kLast) {
    const uint64_t e = other[i];
    const int p = part(e), end = next[p], first = end - count[p];
    int at = first;
    for (int k = first; k < end; k++) at += other[k] > e;
    v[at] = e;
  }
  __syncthreads();
}

// The same for few words, by a wave: a word's place is the number of larger ones.
__device__ __forceinline__ void sort_few(uint64_t *v, int n) {
  const int tid = threadIdx.x;
  const uint64_t a = tid < n ? v[tid] : 0;
  int at = 0;
  if (tid < 64) {
#pragma unroll 8
    for (int i = 0; i < n; i++) at += v[i] > a;
  }
  __syncthreads();
  if (tid < n) v[at] = a;
  __syncthreads();
}

template <typename T>
__global__ __launch_bounds__(kLast) void token_kernel(const SampleArgs A, const SampleWs W) {
  __shared__ __attribute__((aligned(16))) uint64_t list[kSort];
  __shared__ double room[kLast / 64], seg_sum[kMaxSegs], table[kParts], one[64], upto[kSteps];
  __shared__ unsigned long long extra[kMaxSegs], fine[kSteps], cell[kSeg / 64];
  __shared__ int found, kept, first[kSteps / 64], last[kSteps / 64];
  const int tid = threadIdx.x, segs = A.segs, rel = blockIdx.x, row = A.row0 + rel;
  const RowInfo info = W.info[rel];
  if (info.mode == kDone) return;
  const int n = (int)W.found[rel * kLine];
  const Rule rule = rule_of(A, row);
  const Weigher weigh = {info.most, rule.per, table};
  uint64_t *gathered = W.gathered + (int64_t)rel * W.room, *worth = W.worth + (int64_t)rel * W.room;
  fill_table(table);
  if (tid < segs) {
    seg_sum[tid] = W.seg_sum[(int64_t)rel * segs + tid];
    W.seg_sum[(int64_t)rel * segs + tid] = 0.0;
    extra[tid] = 0;
  }
  if (tid < kSteps) fine[tid] = 0;
  if (tid < 64) {
    cell[tid] = 0;
    one[tid] = 0.0;
  }
  if (tid == 0) {
    kept = kGather;
    found = 0;
  }
  __syncthreads();
  if (tid == 0) {
    W.info[rel] = RowInfo{0, 0.0f, 0, 0, 0.0};
    W.found[rel * kLine] = 0;
  }
  auto keep = [&](uint64_t entry) {
    const double w = weigh(logit_of(entry));
    if (w > 0.0 && w >= rule.min_p) atomicAdd(&extra[(int)~(uint32_t)entry / kSeg], (unsigned long long)steps_of(w));
  };
  double left = info.left;
  bool alone = info.mode == kAlone || n > kGather;
  int m = n;  // tokens to be sorted
  if (!alone && (info.mode == kTopK || n <= 64)) {
    alone = n > kSort;
    for (int i = tid; i < min(n, kSort); i += kLast) list[i] = gathered[i];
    __syncthreads();
  } else if (!alone) {
    // by 256ths of the step: those above the one in which the limit falls are kept
    const bool weights = info.mode == kTopP;
    constexpr uint64_t kWeight = ((uint64_t)1 << kKeepBit) - 1;
#pragma unroll 4
    for (int i = tid; i < n; i += kLast) {
      const uint64_t v = worth[i];
      atomicAdd(&fine[v >> kPartBit], weights ? (unsigned long long)(v & kWeight) : 1ull);
    }
    __syncthreads();
    const double have = tid < kSteps ? (double)fine[tid] / (weights ? kFixed : 1.0) : 0.0, before = block_before<kLast>(have, room);
    const uint64_t some = __ballot(have > 0.0), there = __ballot(have > 0.0 && before + have >= left);
    if (tid < kSteps) upto[tid] = before;
    if (tid < kSteps && (tid & 63) == 0) {
      first[tid / 64] = there ? tid + __builtin_ctzll(there) : kSteps;
      last[tid / 64] = some ? tid + 63 - __builtin_clzll(some) : 0;
    }
    __syncthreads();
    // (where roundings of the sums leave the limit unreached: the last one there is)
    int at_part = kSteps, end = 0;
#pragma unroll
    for (int i = 0; i < kSteps / 64; i++) {
      at_part = min(at_part, first[i]);
      end = max(end, last[i]);
    }
    if (at_part == kSteps) at_part = end;
    left -= upto[at_part];
#pragma unroll 4
    for (int i = tid; i < n; i += kLast) {
      const uint64_t v = worth[i], e = gathered[i];
      const int q = (int)(v >> kPartBit);
      if (q < at_part && (v >> kKeepBit & 1)) atomicAdd(&extra[(int)~(uint32_t)e / kSeg], (unsigned long long)(v & kWeight));
      if (q == at_part) {
        const int k = atomicAdd(&found, 1);
        if (k < kSort) list[k] = e;
      }
    }
    __syncthreads();
    m = found;
    alone = m > kSort;
  }
  for (int i = tid; i < min(n, kGather); i += kLast) gathered[i] = 0;
  if (info.mode != kTopK)
    for (int i = tid; i < min(n, kGather); i += kLast) worth[i] = 0;
  if (alone) {
    whole_row<T, kLast>(A, row, table, reinterpret_cast<float *>(list));
    return;
  }
  Cut cut = {0, -1};
  if (info.mode != kMinP) {
    if (m > kSort / 2) sort_equal(list, m);
    else if (m > 64) sort_down(list, list + kSort / 2, m, room);
    else sort_few(list, m);
    if (info.mode == kTopK) {
      // all tokens that may be kept are in the list, one a thread: the limit, the
      // segment, its 64 tokens and the token by their sums alone
      const int top = min(rule.top_k, m);
      constexpr int kPer = kFewK / kLast;
      int index[kPer];
      double w[kPer], own = 0.0;
#pragma unroll
      for (int j = 0; j < kPer; j++) {
        const int i = tid * kPer + j;
        const uint64_t entry = i < top ? list[i] : 0;
        index[j] = (int)~(uint32_t)entry;
        w[j] = i < top ? weigh(logit_of(entry)) : 0.0;
        own += w[j];
      }
      if (rule.top_p < 1.0) {
        double all, c = block_before<kLast>(own, room, &all);
        int spare = kGather;  // the first that is not needed
#pragma unroll
        for (int j = 0; j < kPer; j++) {
          const int i = tid * kPer + j;
          if (i > 0 && i < top && c >= rule.top_p * all) spare = min(spare, i);
          c += w[j];
        }
        const uint64_t some = __ballot(spare < kGather);
        if (some) {
          spare = __builtin_amdgcn_readlane(spare, __builtin_ctzll(some));
          if ((tid & 63) == 0) atomicMin(&kept, spare);
        }
        __syncthreads();
      }
#pragma unroll
      for (int j = 0; j < kPer; j++) {
        if (tid * kPer + j >= kept || !(w[j] >= rule.min_p)) w[j] = 0.0;
        if (w[j] > 0.0) atomicAdd(&extra[index[j] / kSeg], (unsigned long long)steps_of(w[j]));
      }
      __syncthreads();
      if (tid < segs) seg_sum[tid] = (double)extra[tid] / kFixed;
      __syncthreads();
      double from, target, total;
      const int seg = find_segment(A.u[row], segs, seg_sum, from, target, total);
#pragma unroll
      for (int j = 0; j < kPer; j++)
        if (w[j] > 0.0 && index[j] / kSeg == seg) atomicAdd(&cell[index[j] % kSeg / 64], (unsigned long long)steps_of(w[j]));
      __syncthreads();
      const int at = seg * (kSeg / 64) + crossing((double)cell[tid & 63] / kFixed, from, target, from);
#pragma unroll
      for (int j = 0; j < kPer; j++)
        if (w[j] > 0.0 && index[j] / 64 == at) one[index[j] % 64] = w[j];
      __syncthreads();
      const int l = crossing(one[tid & 63], from, target, from);
      if (tid == 0) answer(A, row, at * 64 + l, one[l], total);
      return;
    }
    // the limit, kLast sorted tokens at a time
    const int top = info.mode == kManyK ? min((int)left, m) : m;
    int keeps = top;
    if (rule.top_p < 1.0) {
      const double target = left;
      double before = 0.0;
#pragma unroll 1
      for (int i0 = 0; i0 < top; i0 += kLast) {
        const int i = i0 + tid;
        const double w = i < top ? weigh(logit_of(list[i])) : 0.0;
        double all;
        const double c = before + block_before<kLast>(w, room, &all);
        const uint64_t spare = __ballot(i < top && i > 0 && c >= target);
        if (spare && (tid & 63) == 0) atomicMin(&kept, i + __builtin_ctzll(spare));  // the first that is not needed
        __syncthreads();
        if (kept < top) break;
        before += all;
      }
      keeps = min(kept, top);
    }
    // (nothing is there where the limit falls behind the last token: all are kept)
    const uint64_t lowest = keeps ? list[keeps - 1] : 0xffffffffull;
    cut = Cut{(uint32_t)(lowest >> 32), (int)~(uint32_t)lowest};
    for (int i = tid; i < keeps; i += kLast) keep(list[i]);
    __syncthreads();
    if (tid < segs) seg_sum[tid] += (double)extra[tid] / kFixed;
    __syncthreads();
  }
  choose<T, kLast>(A, row, segs, seg_sum, weigh, cut, rule.min_p, reinterpret_cast<float *>(list));
}

bool aligned_to(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int check_shape(int64_t rows, int64_t vocab) {
  return rows < 1 || rows > (1 << 20) || vocab < 1 || vocab > kMaxVocab ? TQ_ERR_SHAPE : TQ_OK;
}

// A call's rows in passes whose words fit kWsBytes.
constexpr size_t kWsBytes = (size_t)1 << 27;

struct Plan {
  int64_t segs, pass, room;
  size_t bytes;
};

Plan make_plan(int64_t rows, int64_t vocab) {
  Plan P = {(vocab + kSeg - 1) / kSeg, 0, kGather, 0};
  if (P.room > P.segs * kSeg) P.room = P.segs * kSeg;
  const size_t each = sizeof(RowInfo) + ((size_t)P.room * 4 + kLine) * 4 + (size_t)P.segs * (sizeof(SegInfo) + 8 + kSteps * 12);
  P.pass = (int64_t)(kWsBytes / each);
  if (P.pass > rows) P.pass = rows;
  P.bytes = ((size_t)P.pass * each + 15) / 16 * 16;
  return P;
}

}  // namespace

extern "C" size_t tq_sample_workspace_bytes(int64_t rows, int64_t vocab) {
  return check_shape(rows, vocab) == TQ_OK ? make_plan(rows, vocab).bytes : 0;
}

extern "C" int tq_sample(int dtype, int64_t rows, int64_t vocab, const void *logits, int64_t row_stride,
                         const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                         const float *u, int32_t *token, float *logprob, void *ws, size_t ws_bytes, void *stream) {
  if (!logits || !u || !token) return TQ_ERR_NULL;
  if (dtype != TQ_F16 && dtype != TQ_F32) return TQ_ERR_DTYPE;
  const int rc = check_shape(rows, vocab);
  if (rc != TQ_OK) return rc;
  if (row_stride < vocab || row_stride > ((int64_t)1 << 31)) return TQ_ERR_SHAPE;
  if (!aligned_to(logits, 16) || !aligned_to(ws, 16) || !aligned_to(temperature, 4) || !aligned_to(top_k, 4) ||
      !aligned_to(top_p, 4) || !aligned_to(min_p, 4) || !aligned_to(u, 4) || !aligned_to(token, 4) ||
      !aligned_to(logprob, 4))
    return TQ_ERR_ALIGN;
  const Plan P = make_plan(rows, vocab);
  if (P.bytes && !ws) return TQ_ERR_NULL;
  if (ws_bytes < P.bytes) return TQ_ERR_SIZE;
  const int64_t unit = dtype == TQ_F16 ? 8 : 4;
  SampleArgs A = {logits, temperature, top_p, min_p, u, top_k, token, logprob, row_stride, (int)rows, (int)vocab,
                  0, (int)P.segs, rows == 1 || row_stride % unit == 0};
  hipStream_t st = (hipStream_t)stream;
  const bool limits = top_k || top_p || min_p;
  // A workgroup a row, in one launch, where there is one segment and no limit: one row of
  // 4000 9 against 11 us, 64 of 4000 10 against 12 (with limits: 92 against 21, 106
  // against 32).
  if (P.segs == 1 && !limits) {
    if (dtype == TQ_F16) hipLaunchKernelGGL((row_kernel<_Float16, 1024>), dim3((unsigned)rows), dim3(1024), 0, st, A);
    else hipLaunchKernelGGL((row_kernel<float, 1024>), dim3((unsigned)rows), dim3(1024), 0, st, A);
    return hipGetLastError() == hipSuccess ? TQ_OK : TQ_ERR_HIP;
  }
  char *p = (char *)ws;
  const size_t n = (size_t)P.pass, ns = n * (size_t)P.segs;
  SampleWs W;
  W.room = P.room;
  W.info = (RowInfo *)p;
  W.seg = (SegInfo *)(p += n * sizeof(RowInfo));
  W.gathered = (uint64_t *)(p += ns * sizeof(SegInfo));
  W.worth = (uint64_t *)(p += n * (size_t)P.room * 8);
  W.weight = (uint64_t *)(p += n * (size_t)P.room * 8);
  W.seg_sum = (double *)(p += ns * kSteps * 8);
  W.count = (uint32_t *)(p += ns * 8);
  W.found = (uint32_t *)(p += ns * kSteps * 4);
  for (int64_t r = 0; r < rows; r += P.pass) {
    A.row0 = (int)r;
    const int64_t m = rows - r < P.pass ? rows - r : P.pass;
    const dim3 each((unsigned)(m * P.segs)), one((unsigned)m);
#define TQ_SAMPLE(T)                                                                  \
  {                                                                                   \
    hipLaunchKernelGGL((segment_kernel<T>), each, dim3(kThreads), 0, st, A, W);       \
    hipLaunchKernelGGL((limit_kernel<T>), one, dim3(kLimit), 0, st, A, W);            \
    if (!limits) continue;                                                            \
    hipLaunchKernelGGL((gather_kernel<T>), each, dim3(kThreads), 0, st, A, W);        \
    hipLaunchKernelGGL((token_kernel<T>), one, dim3(kLast), 0, st, A, W);             \
  }
    if (dtype == TQ_F16) TQ_SAMPLE(_Float16) else TQ_SAMPLE(float)
#undef TQ_SAMPLE
  }
  return hipGetLastError() == hipSuccess ? TQ_OK : TQ_ERR_HIP;
}
