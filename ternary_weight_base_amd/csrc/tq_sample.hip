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

struct SampleArgs {
  const void *logits;
  const float *temperature, *top_p, *min_p, *u;
  const int *top_k;
  int *token;
  float *logprob;
  int64_t row_stride;
  int rows, vocab;
};

// A row's settings.
struct Rule {
  double per;       // log2 e / temperature
  double top_p, min_p;
  int top_k;        // vocab: all
  bool greedy;
};

__device__ __forceinline__ Rule rule_of(const SampleArgs &A, int row) {
  Rule r;
  const float t = A.temperature ? A.temperature[row] : 1.0f;
  r.greedy = !(t > 0.0f);
  r.per = r.greedy ? 0.0 : 1.4426950408889634 / (double)t;
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

// 2^t for t <= 0, to some 2^-51 of it; 0 from 2^-1000 on (and for -inf, NaN).
__device__ __forceinline__ double power2(double t) {
  if (!(t > -1000.0)) return 0.0;
  const double n = rint(t), f = (t - n) * 0.6931471805599453;
  // exp's series: |f| <= 0.3466, its 14th term is below 2^-57
  double s = 1.0 / 6227020800.0;
  s = fma(s, f, 1.0 / 479001600.0);
  s = fma(s, f, 1.0 / 39916800.0);
  s = fma(s, f, 1.0 / 3628800.0);
  s = fma(s, f, 1.0 / 362880.0);
  s = fma(s, f, 1.0 / 40320.0);
  s = fma(s, f, 1.0 / 5040.0);
  s = fma(s, f, 1.0 / 720.0);
  s = fma(s, f, 1.0 / 120.0);
  s = fma(s, f, 1.0 / 24.0);
  s = fma(s, f, 1.0 / 6.0);
  s = fma(s, f, 0.5);
  s = fma(s, f, 1.0);
  s = fma(s, f, 1.0);
  return ldexp(s, (int)n);
}

// The row's logits as its weights are taken from them: where one is +inf those
// weigh 1 and all others nothing.
struct Weigher {
  float most;
  double per;
  __device__ __forceinline__ double operator()(float x) const {
    if (most == __builtin_inff()) return x == most ? 1.0 : 0.0;
    return x == -__builtin_inff() ? 0.0 : power2(((double)x - (double)most) * per);
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
// ... of the threads before this one.
template <int NT>
__device__ __forceinline__ double block_before(double v, double *room) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double sum = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const double o = __shfl_up(sum, d);
    if (lane >= d) sum += o;
  }
  __syncthreads();
  if (lane == 63) room[wave] = sum;
  __syncthreads();
  double s = 0.0;
  for (int i = 0; i < wave; i++) s += room[i];
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
  const int bits = 62 - (32 - __builtin_clz(vocab));
  const double steps = weights ? ldexp(1.0, bits) : 1.0, unit = weights ? ldexp(1.0, -bits) : 1.0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += NT) hist[i] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0 : ~0u << (shift + 8);
    for (int i = threadIdx.x; i < vocab; i += NT) {
      const float v = clean((float)x[i]);
      const uint32_t k = key_of(v);
      if (v > -__builtin_inff() && (k & mask) == prefix && cut.keeps(k, i))
        atomicAdd((unsigned long long *)&hist[k >> shift & 255], weights ? (unsigned long long)rint(weigh(v) * steps) : 1ull);
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

// The token of a segment at which the running sum from `before` on exceeds
// `target`: the first one, or the last that is kept; its weight.
template <typename T, int NT>
__device__ int pick(const T *x, int vocab, int seg, const Weigher &weigh, const Cut &cut, double min_p, double before,
                    double target, double *room, double &weight) {
  constexpr int kEach = kSeg / NT;
  __shared__ int first, end;
  if (threadIdx.x == 0) {
    first = 0x7fffffff;
    end = -1;
  }
  double w[kEach], sum = 0.0;
  const int i0 = seg * kSeg + threadIdx.x * kEach;
#pragma unroll
  for (int j = 0; j < kEach; j++) {
    w[j] = 0.0;
    if (i0 + j < vocab) {
      const float v = clean((float)x[i0 + j]);
      const double e = weigh(v);
      if (cut.keeps(key_of(v), i0 + j) && e >= min_p) w[j] = e;
    }
    sum += w[j];
  }
  double c = before + block_before<NT>(sum, room);
#pragma unroll
  for (int j = 0; j < kEach; j++) {
    c += w[j];
    if (w[j] > 0.0) {
      if (c > target) atomicMin(&first, i0 + j);
      atomicMax(&end, i0 + j);
    }
  }
  __syncthreads();
  const int i = first < 0x7fffffff ? first : end;
  weight = i >= 0 ? weigh(clean((float)x[i])) : 0.0;
  return i;
}

template <typename T, int NT>
__global__ __launch_bounds__(NT) void row_kernel(const SampleArgs A) {
  __shared__ uint64_t hist[256];
  __shared__ double room[NT / 64], seg_sum[kMaxSegs];
  __shared__ float wave_most[NT / 64];
  __shared__ int where;
  const int row = blockIdx.x, tid = threadIdx.x, vocab = A.vocab;
  const T *x = (const T *)A.logits + row * A.row_stride;
  const Rule rule = rule_of(A, row);
  float most = -__builtin_inff();
  for (int i = tid; i < vocab; i += NT) most = fmaxf(most, clean((float)x[i]));
  most = tqdev::wave_max64(most);
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
    if (tid == 0) {
      const bool none = most == -__builtin_inff();
      A.token[row] = none ? -1 : where;
      if (A.logprob) A.logprob[row] = none ? -__builtin_inff() : 0.0f;
    }
    return;
  }
  const Weigher weigh = {most, rule.per};
  Cut cut = {key_of(-__builtin_inff()), -1};
  if (rule.top_k < vocab) narrow<T, NT>(x, vocab, weigh, false, (double)rule.top_k, cut, hist, room);
  if (rule.top_p < 1.0) {
    double sum = 0.0;
    for (int i = tid; i < vocab; i += NT) {
      const float v = clean((float)x[i]);
      if (cut.keeps(key_of(v), i)) sum += weigh(v);
    }
    sum = block_sum<NT>(sum, room);
    narrow<T, NT>(x, vocab, weigh, true, fmax(rule.top_p, 0.0) * sum, cut, hist, room);
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
  double total = 0.0;
  for (int s = 0; s < segs; s++) total += seg_sum[s];
  const float u = A.u[row];
  const double target = (u > 0.0f ? (double)u : 0.0) * total;
  double before = 0.0;
  int seg = -1;
  for (int s = 0; s < segs; s++) {
    if (!(seg_sum[s] > 0.0)) continue;
    if (seg >= 0) before += seg_sum[seg];
    seg = s;
    if (before + seg_sum[s] > target) break;
  }
  double weight;
  const int i = pick<T, NT>(x, vocab, seg, weigh, cut, rule.min_p, before, target, room, weight);
  if (tid == 0) {
    A.token[row] = i;
    if (A.logprob) A.logprob[row] = (float)log(weight / total);
  }
}

bool aligned_to(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int check_shape(int64_t rows, int64_t vocab) {
  return rows < 1 || rows > (1 << 20) || vocab < 1 || vocab > kMaxVocab ? TQ_ERR_SHAPE : TQ_OK;
}

}  // namespace

extern "C" size_t tq_sample_workspace_bytes(int64_t rows, int64_t vocab) {
  (void)rows;
  (void)vocab;
  return 0;
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
  const size_t need = tq_sample_workspace_bytes(rows, vocab);
  if (need && !ws) return TQ_ERR_NULL;
  if (ws_bytes < need) return TQ_ERR_SIZE;
  const SampleArgs A = {logits, temperature, top_p, min_p, u, top_k, token, logprob, row_stride, (int)rows, (int)vocab};
  hipStream_t st = (hipStream_t)stream;
  if (dtype == TQ_F16) hipLaunchKernelGGL((row_kernel<_Float16, 1024>), dim3((unsigned)rows), dim3(1024), 0, st, A);
  else hipLaunchKernelGGL((row_kernel<float, 1024>), dim3((unsigned)rows), dim3(1024), 0, st, A);
  return hipGetLastError() == hipSuccess ? TQ_OK : TQ_ERR_HIP;
}
