// tq_linear.hip -- linear attention with a decay for each head.
//
//   S_t = a_t S_{t-1} + k_t v_t^T,   o_t = scale q_t^T S_t,   a_t = exp(log_decay_t)
//
// with an fp32 state S [head_dim][head_dim] (key index first) a sequence and
// KV head.  Two forms:
//
// Few rows a sequence: the recurrence itself, in fp32.  A workgroup holds 64
// columns of a state in registers, a wave a quarter of their rows.  Bound: the
// states' bytes, read and written once (64 tokens, 8 KV heads of 128: 67 MB in 13 us,
// 5.1 TB/s; one token: 5 us, a launch and two dependent loads).
//
// Prompts, in chunks of 128 rows (G: the chunk's running sum of log2 a):
//   o_i = scale (2^G_i q_i S + sum_{j <= i} 2^(G_i - G_j) (q_i . k_j) v_j)
//   S'  = 2^G_n S + U,   U = sum_j 2^(G_n - G_j) k_j v_j^T
// in three launches: every chunk's U; the states before each chunk, element by
// element along the chunks; every chunk's outputs.
//
// Products run on v_mfma_f32_32x32x16_f16, sums in fp32.  fp16 operands are scaled by
// powers of two, each row by its own size and by what is left of it where it is used, so
// that no size of input overflows them and no row takes another's bits.
// U is of two fp16 terms a factor (fp16 inputs: the keys with their weights two, the
// values are exact down to 2^-38 of the row's largest): a term is within 2^-22 of itself,
// the state as near as fp32 sums (a prompt's: 1.1e-7 off, plain fp32 0.8e-7).
// For the outputs, which are fp16, queries, keys and weights have two terms each; fp32
// values and the states before a chunk are rounded to fp16 once (outputs 0.00029 off
// in place of 0.00021, which their own rounding is).  Second terms of those would take
// 64 KB more LDS than a CU has beside fp32 keys of 128, and a third more products.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>
#include <utility>

#include "tq.h"
#include "tq_device.h"
#include "tq_kv.h"
#include "tq_wave.h"

namespace {

using namespace tqkv;

constexpr int kChunk = 128;     // rows of a chunk
constexpr int kStep = 64;       // ... of them that U's kernel takes at once
constexpr int kScanRun = 8;    // chunks of a wave's run in the scan
constexpr int kFewRows = 16;    // up to so many rows a sequence (on average): the recurrence
constexpr size_t kPassBytes = (size_t)1 << 27;  // scratch of a pass over the chunks
constexpr int kNoState = -100000;  // exponent of a snapshot that is zero

typedef float f8 __attribute__((ext_vector_type(8)));
typedef float f16x __attribute__((ext_vector_type(16)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s4 lds_s4;

struct Meta {
  float decay, most_u, most_s;  // log2 of the chunk's decay; max |U|; max |S| before the pass's first chunk
  int e;                        // the snapshot holds S * 2^-e
};

struct LinArgs {
  const void *qkv;
  const float *log_decay;
  const int *cu, *from, *to;
  float *states;
  _Float16 *out;
  int64_t row_stride, decay_stride, out_stride, num_states;
  float scale;
  int rows, seqs, hq, hkv, group;
  // a pass over the chunks: slots slot0 .. slot0 + slots - 1
  float *u, *carry;  // carry: where the pass leaves the state of a sequence that goes on behind it
  const float *carried;  // ... and where the last one left it
  _Float16 *snap;
  Meta *meta;
  int slot0, slots, parts;
};

__device__ __forceinline__ bool state_ok(const LinArgs &A, int id) { return id >= 0 && id < A.num_states; }

// log2 of a row's decay: above 0 (growth) counts as 0, below -2000 as -2000 (a factor of 0).
__device__ __forceinline__ double log2_decay(const LinArgs &A, int row, int h) {
  const double g = (double)A.log_decay[row * A.decay_stride + h] * 1.4426950408889634;
  return fmin(fmax(g, -2000.0), 0.0);
}

__device__ __forceinline__ f8 load8(const float *p) {
  const f4 a = *reinterpret_cast<const f4 *>(p), b = *reinterpret_cast<const f4 *>(p + 4);
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ __forceinline__ h8 load8(const _Float16 *p) { return *reinterpret_cast<const h8 *>(p); }

// ---- few rows a sequence ---------------------------------------------------

constexpr int kHeads = 8;  // query heads taken together

template <int D, typename T>
__global__ __launch_bounds__(256) void recur_kernel(const LinArgs A) {
  constexpr int kOwn = D / 4;  // rows of the state a wave
  __shared__ __attribute__((aligned(16))) float ks[D], qs[kHeads][D], red[4][kHeads][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t blk = blockIdx.x % (uint32_t)(D / 64), sh = blockIdx.x / (uint32_t)(D / 64);
  const int h = sh % (uint32_t)A.hkv, s = sh / (uint32_t)A.hkv;
  const int begin = cu_at(A.cu, s, A.rows), n = cu_at(A.cu, s + 1, A.rows) - begin;
  if (n <= 0) return;
  const int from = A.from[s], to = A.to[s], col = blk * 64 + lane;
  float S[kOwn];
#pragma unroll
  for (int i = 0; i < kOwn; i++) S[i] = 0.0f;
  if (state_ok(A, from)) {
    const float *p = A.states + ((int64_t)from * A.hkv + h) * (D * D) + wave * kOwn * D + col;
#pragma unroll
    for (int i = 0; i < kOwn; i++) S[i] = p[i * D];
  }
  for (int r = 0; r < n; r++) {
    const T *x = (const T *)A.qkv + (int64_t)(begin + r) * A.row_stride;
    const float v = (float)x[(A.hq + A.hkv + h) * D + col];
    const float a = __builtin_amdgcn_exp2f((float)log2_decay(A, begin + r, h));
    for (int g0 = 0; g0 < A.group; g0 += kHeads) {
      const int heads = min(kHeads, A.group - g0);
      __syncthreads();
      if (g0 == 0)
        for (int i = tid; i < D; i += 256) ks[i] = (float)x[(A.hq + h) * D + i];
      for (int i = tid; i < heads * D; i += 256) qs[i / D][i % D] = (float)x[(h * A.group + g0) * D + i] * A.scale;
      __syncthreads();
      if (g0 == 0) {
#pragma unroll
        for (int i = 0; i < kOwn; i++) S[i] = a * S[i] + ks[wave * kOwn + i] * v;
      }
      for (int g = 0; g < heads; g++) {
        float o = 0.0f;
#pragma unroll
        for (int i = 0; i < kOwn; i++) o += qs[g][wave * kOwn + i] * S[i];
        red[wave][g][lane] = o;
      }
      __syncthreads();
      for (int i = tid; i < heads * 64; i += 256) {
        const int g = i / 64, c = i % 64;
        const float o = (red[0][g][c] + red[1][g][c]) + (red[2][g][c] + red[3][g][c]);
        A.out[(int64_t)(begin + r) * A.out_stride + (h * A.group + g0 + g) * D + blk * 64 + c] = (_Float16)o;
      }
    }
  }
  if (state_ok(A, to)) {
    float *p = A.states + ((int64_t)to * A.hkv + h) * (D * D) + wave * kOwn * D + col;
#pragma unroll
    for (int i = 0; i < kOwn; i++) p[i * D] = S[i];
  }
}

// ---- prompts ---------------------------------------------------------------

// A chunk: n rows from `begin` on, the `local`-th of sequence s.
struct Chunk {
  int s, begin, n, local;
};
__device__ __forceinline__ bool find_chunk(const LinArgs &A, int slot, Chunk &c) {
  int first, end;
  if (A.seqs < 64) {  // (a lane an entry: no second trip to memory for what was found)
    const int lane = threadIdx.x & 63, v = cu_at(A.cu, min(lane, A.seqs), A.rows);
    const bool le = lane < A.seqs && slot_base<kChunk, 1>(v, lane, 1) <= slot;
    c.s = max((int)__popcll(__ballot(le)), 1) - 1;
    first = __builtin_amdgcn_readlane(v, c.s);
    end = __builtin_amdgcn_readlane(v, c.s + 1);
  } else {
    c.s = find_seq<kChunk, 1>(A.cu, A.seqs, A.rows, slot, 1);
    first = cu_at(A.cu, c.s, A.rows);
    end = cu_at(A.cu, c.s + 1, A.rows);
  }
  c.local = slot - slot_base<kChunk, 1>(first, c.s, 1);
  if (c.local < 0 || c.local >= (end - first + kChunk - 1) / kChunk || end <= first) return false;
  c.begin = first + c.local * kChunk;
  c.n = min(kChunk, end - c.begin);
  return true;
}

// Running sums of the chunk's log2 decays, by one wave: lane l's are of rows
// 2 l and 2 l + 1; rows behind the chunk do not decay.
__device__ __forceinline__ void decay_sums(const LinArgs &A, const Chunk &c, int h, double &g0, double &g1) {
  const int lane = threadIdx.x & 63;
  const double d0 = 2 * lane < c.n ? log2_decay(A, c.begin + 2 * lane, h) : 0.0;
  const double d1 = 2 * lane + 1 < c.n ? log2_decay(A, c.begin + 2 * lane + 1, h) : 0.0;
  const double sum = tqdev::wave_upto(d0 + d1);
  g1 = sum;
  g0 = sum - d1;
}

// The largest of the lanes up to this one.
template <int CTRL, int ROWS>
__device__ __forceinline__ float most_below(float v) {  // (or its own)
  const int b = __float_as_int(v);
  return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(b, b, CTRL, ROWS, 0xF, false)));
}
__device__ __forceinline__ float wave_most_upto(float v) {
  v = most_below<0x111, 0xF>(v);  // (the moves of wave_upto)
  v = most_below<0x112, 0xF>(v);
  v = most_below<0x114, 0xF>(v);
  v = most_below<0x118, 0xF>(v);
  v = most_below<0x142, 0xA>(v);
  return most_below<0x143, 0xC>(v);
}

// A tile of fp16 rows in LDS whose operands are read transposed (below):
// 64-byte blocks of a row in an order that puts the same block of four
// consecutive rows into different banks.  -> byte offset of a block
template <int D>
__device__ __forceinline__ int block_at(int row, int blk) {
  return row * 2 * D + ((blk ^ (D == 128 ? row & 3 : (row >> 1) & 1)) << 6);
}
template <int D>
__device__ __forceinline__ int piece_at(int row, int piece) {  // 8 elements
  return block_at<D>(row, piece >> 2) + (piece & 3) * 16;
}

// A matrix operand from such a tile: lane l takes column 32 blk + l % 32 of rows
// row0 + 8 (l / 32) + 0 .. 7.  ds_read_b64_tr_b16 turns 4 rows x 16 columns
// among 16 lanes.
template <int D>
struct Turned {
  int at;  // this lane's byte offset in rows 0 .. 15, block 0 but for the order
  int sw;
  __device__ __forceinline__ Turned() {
    const int lane = threadIdx.x & 63, row = 8 * (lane >> 5) + ((lane & 15) >> 2);
    sw = D == 128 ? row & 3 : (row >> 1) & 1;
    at = row * 2 * D + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
  }
  __device__ __forceinline__ h8 operator()(const uint8_t *tile, int row0, int blk) const {
    const uint8_t *p = tile + at + ((blk ^ sw) << 6) + row0 * 2 * D;
    const s4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)p);
    const s4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(p + 8 * D));
    const h4 x = __builtin_bit_cast(h4, a), y = __builtin_bit_cast(h4, b);
    return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};

// x as two fp16 terms, together within 2^-23 of it (or half the least fp16 step), two
// elements an instruction.
__device__ __forceinline__ void two_terms(const f8 &x, h8 &hi, h8 &lo) {
  hi = __builtin_convertvector(x, h8);
  lo = __builtin_convertvector(x - __builtin_convertvector(hi, f8), h8);
}

// 2^e as a factor, e within fp32's exponents
__device__ __forceinline__ float power(int e) { return __uint_as_float((uint32_t)(min(max(e, -126), 127) + 127) << 23); }

// The largest of what D / 8 consecutive lanes hold.
template <int D, typename V, typename F>
__device__ __forceinline__ V row_most(V v, const F &most) {
  auto step = [&](int moved) { v = most(v, __builtin_bit_cast(V, moved)); };
  step(tqdev::dpp_move<tqdev::kDppSwap1>(__builtin_bit_cast(int, v)));
  step(tqdev::dpp_move<tqdev::kDppSwap2>(__builtin_bit_cast(int, v)));
  if (D == 128) {
    step(tqdev::dpp_move<tqdev::kDppRor4>(__builtin_bit_cast(int, v)));
    step(tqdev::dpp_move<tqdev::kDppRor8>(__builtin_bit_cast(int, v)));
  } else {
    step(tqdev::dpp_move<0x141>(__builtin_bit_cast(int, v)));  // (eight lanes mirrored)
  }
  return v;
}
// The exponent of a row's largest value (`some`: not all are 0), by which eight values a
// lane are scaled to below 2^14, unless SCALE says no.
template <int D, bool SCALE = true>
__device__ __forceinline__ int scale_row(f8 &v, bool &some) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; j++) m = fmaxf(m, fabsf(v[j]));
  m = row_most<D>(m, [](float a, float b) { return fmaxf(a, b); });
  some = m > 0.0f;
  const int e = __builtin_amdgcn_frexp_expf(m);
#pragma unroll
  for (int j = 0; j < 8; j++)
    if (SCALE) v[j] = ldexpf(v[j], 14 - e);
  return e;
}
template <int D, bool SCALE = true>
__device__ __forceinline__ int scale_row(h8 &v, bool &some) {
  // (values without their signs are in the order of their bits: two at a time)
  typedef uint16_t s2 __attribute__((ext_vector_type(2)));
  typedef uint16_t s8 __attribute__((ext_vector_type(8)));
  const s8 bits = __builtin_bit_cast(s8, __builtin_bit_cast(u4, v) & 0x7fff7fffu);
  const s2 a = __builtin_elementwise_max(bits.s01, bits.s23), b = __builtin_elementwise_max(bits.s45, bits.s67);
  s2 m = __builtin_elementwise_max(a, b);
  m = row_most<D>(m, [](s2 x, s2 y) { return __builtin_elementwise_max(x, y); });
  const float most = tqdev::half_bits(m[0] > m[1] ? m[0] : m[1]);
  some = most > 0.0f;
  const int e = __builtin_amdgcn_frexp_expf(most);
#pragma unroll
  for (int j = 0; j < 8; j++)
    if (SCALE) v[j] = __builtin_amdgcn_ldexph(v[j], 14 - e);
  return e;
}

// Size (an exponent) of a row whose key or value is zero: far below any other's.
constexpr int kNothing = -4000;

// U of a chunk and KV head, 64 rows at a time; further workgroups take the
// largest element of the state that each sequence starts the pass from.  Bound: one
// workgroup a CU in turn waits for its rows, converts and multiplies them (4096 fp32
// rows of 8 KV heads of 128, 50 MB: 14 to 16.5 us, of them 6.5 the loads and 3 the stores;
// in halves of 64 columns, two workgroups a CU, no faster).
template <int D, typename T>
__global__ __launch_bounds__(512) void chunk_state_kernel(const LinArgs A) {
  constexpr bool kWide = std::is_same<T, float>::value;
  constexpr int kSteps = kChunk / kStep, kPer = kStep * (D / 8) / 512;  // pieces of 8 elements a thread and step
  constexpr int kNb = D == 128 ? 2 : 1;  // column blocks of 32 a wave
  constexpr int kTile = kStep * 2 * D;
  __shared__ __attribute__((aligned(16))) uint8_t kh[2 * kTile], vh[kTile], vl[kWide ? kTile : 16];
  uint8_t *const kl = kh + kTile;
  __shared__ float left[kChunk], red[8];
  __shared__ int size[kChunk];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = blockIdx.x % (uint32_t)A.hkv, rel = blockIdx.x / (uint32_t)A.hkv;
  auto most_of = [&](float m) {  // over the workgroup, in thread 0
    m = tqdev::wave_max64(m);
    if (lane == 0) red[wave] = m;
    __syncthreads();
    float r = red[0];
#pragma unroll
    for (int i = 1; i < 8; i++) r = fmaxf(r, red[i]);
    return r;
  };
  if (rel >= A.slots) {
    const int s = rel - A.slots, first = cu_at(A.cu, s, A.rows), n = cu_at(A.cu, s + 1, A.rows) - first;
    const int base = slot_base<kChunk, 1>(first, s, 1), slot = max(base, A.slot0);
    if (n <= 0 || slot >= min(base + (n + kChunk - 1) / kChunk, A.slot0 + A.slots)) return;
    const int from = A.from[s];
    const float *p = base < slot ? A.carried + (int64_t)h * (D * D) : A.states + ((int64_t)from * A.hkv + h) * (D * D);
    float m = 0.0f;
    if (base < slot || state_ok(A, from)) {
#pragma unroll
      for (int i = 0; i < D * D / 2048; i++) {
        const f4 x = *reinterpret_cast<const f4 *>(p + (i * 512 + tid) * 4);
        m = fmaxf(m, fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))));
      }
    }
    m = most_of(m);
    if (tid == 0) A.meta[(int64_t)(slot - A.slot0) * A.hkv + h].most_s = m;
    return;
  }
  Chunk c;
  if (!find_chunk(A, A.slot0 + rel, c)) return;
  Meta *meta = A.meta + (int64_t)rel * A.hkv + h;
  const T *kp = (const T *)A.qkv + (int64_t)c.begin * A.row_stride + (A.hq + h) * D;
  const T *vp = kp + A.hkv * D;
  // all rows are sent for at once
  typedef typename std::conditional<kWide, f8, h8>::type Eight;
  Eight k[kSteps][kPer], v[kSteps][kPer];
#pragma unroll
  for (int t = 0; t < kSteps; t++)
#pragma unroll
    for (int i = 0; i < kPer; i++) {
      const int p = i * 512 + tid, row = t * kStep + p / (D / 8), at = p % (D / 8) * 8;
      k[t][i] = v[t][i] = (Eight)(0);
      if (row < c.n) {
        k[t][i] = load8(kp + row * A.row_stride + at);
        v[t][i] = load8(vp + row * A.row_stride + at);
      }
    }
  if (wave == 0) {
    double g0, g1;
    decay_sums(A, c, h, g0, g1);
    const double all = __shfl(g1, 63);
    left[2 * lane] = (float)(all - g0);
    left[2 * lane + 1] = (float)(all - g1);
    if (lane == 0) meta->decay = (float)all;
  }
  const int mb = D == 128 ? wave & 3 : wave & 1, nb0 = D == 128 ? 2 * (wave >> 2) : (wave >> 1) & 1;
  const Turned<D> turned;
  f16x acc[kNb];
#pragma unroll
  for (int b = 0; b < kNb; b++) acc[b] = (f16x)(0.0f);
  // each row by the exponents of its own largest key and value
#pragma unroll
  for (int t = 0; t < kSteps; t++)
#pragma unroll
    for (int i = 0; i < kPer; i++) {
      const int p = i * 512 + tid;
      bool a, b;
      const int e = scale_row<D>(k[t][i], a) + scale_row<D>(v[t][i], b);
      if (p % (D / 8) == 0) size[t * kStep + p / (D / 8)] = a && b ? e : kNothing;
    }
  __syncthreads();
  // the largest that is left at the chunk's end: acc holds U * 2^(28 - unit)
  const int unit = (int)ceilf(tqdev::wave_max64(fmaxf(left[lane] + (float)size[lane], left[64 + lane] + (float)size[64 + lane])));
#pragma unroll
  for (int t = 0; t < kSteps; t++) {
    if (t * kStep >= c.n) break;
    if (t) __syncthreads();  // (the last step's operands are read)
#pragma unroll
    for (int i = 0; i < kPer; i++) {
      const int p = i * 512 + tid, row = p / (D / 8), at = piece_at<D>(row, p % (D / 8)), all = t * kStep + row;
      const float f = __builtin_amdgcn_exp2f(left[all] + (float)(size[all] - unit));
      const f8 kw = __builtin_convertvector(k[t][i], f8) * f;
      h8 a, b, x, y;
      two_terms(kw, a, b);
      if constexpr (kWide) {
        two_terms(v[t][i], x, y);
      } else {
        x = v[t][i];
      }
      *reinterpret_cast<h8 *>(kh + at) = a;
      *reinterpret_cast<h8 *>(kl + at) = b;
      *reinterpret_cast<h8 *>(vh + at) = x;
      if constexpr (kWide) *reinterpret_cast<h8 *>(vl + at) = y;
    }
    __syncthreads();
    // (head_dim 64: the upper four waves take the other half of the rows)
    constexpr int kRows = D == 128 ? kStep : kStep / 2;
    const int r0 = D == 128 ? 0 : (wave >> 2) * kRows;
#pragma unroll
    for (int r = 0; r < kRows; r += 16) {
      const h8 a = turned(kh, r0 + r, mb), b = turned(kl, r0 + r, mb);
#pragma unroll
      for (int nb = 0; nb < kNb; nb++) {
        const h8 x = turned(vh, r0 + r, nb0 + nb);
        acc[nb] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, x, acc[nb], 0, 0, 0);
        acc[nb] = __builtin_amdgcn_mfma_f32_32x32x16_f16(b, x, acc[nb], 0, 0, 0);
        if constexpr (kWide) acc[nb] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, turned(vl, r0 + r, nb0 + nb), acc[nb], 0, 0, 0);
      }
    }
  }
  __syncthreads();
  if constexpr (D == 64) {  // the halves' sums meet
    float *half = reinterpret_cast<float *>(kh);  // [4 waves][16][64], over kh and kl
    static_assert(sizeof(kh) >= 4 * 16 * 64 * 4, "room for the sums of four waves");
    if (wave >= 4) {
#pragma unroll
      for (int r = 0; r < 16; r++) half[((wave - 4) * 16 + r) * 64 + lane] = acc[0][r];
    }
    __syncthreads();
    if (wave < 4) {
#pragma unroll
      for (int r = 0; r < 16; r++) acc[0][r] += half[(wave * 16 + r) * 64 + lane];
    }
  }
  // acc[b][r] is row 32 mb + 8 (r / 4) + 4 (lane / 32) + r % 4, column 32 (nb0 + b) + lane % 32
  float *u = A.u + ((int64_t)rel * A.hkv + h) * (D * D) + (32 * mb + 4 * (lane >> 5)) * D + 32 * nb0 + (lane & 31);
  float m = 0.0f;
  if (D == 128 || wave < 4) {
#pragma unroll
    for (int b = 0; b < kNb; b++)
#pragma unroll
      for (int r = 0; r < 16; r++) {
        const float x = ldexpf(acc[b][r], unit - 28);
        u[(8 * (r >> 2) + (r & 3)) * D + 32 * b] = x;
        m = fmaxf(m, fabsf(x));
      }
  }
  m = most_of(m);
  if (tid == 0) meta->most_u = m;
}

// The sum over a lane's eight.
__device__ __forceinline__ float row_sum8(float v) {
  v += __int_as_float(tqdev::dpp_move<tqdev::kDppSwap1>(__float_as_int(v)));
  v += __int_as_float(tqdev::dpp_move<tqdev::kDppSwap2>(__float_as_int(v)));
  return v + __int_as_float(tqdev::dpp_move<0x141>(__float_as_int(v)));
}

// A decay, as a product of two factors (of which the second is mostly 1): one alone may
// be below fp32's least number while what it leaves of a large state is not.
struct Factors {
  float a, b;
  __device__ __forceinline__ Factors(float log2) {
    const float whole = ceilf(log2);
    const int e = max((int)whole, -1000), e1 = max(e, -125);
    a = ldexpf(__builtin_amdgcn_exp2f(log2 - whole), e1);
    b = ldexpf(1.0f, e - e1);
  }
  __device__ __forceinline__ Factors(float a, float b) : a(a), b(b) {}
  __device__ __forceinline__ Factors at(int lane) const {
    return Factors(__uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(a), lane)),
                   __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(b), lane)));
  }
  template <typename V>
  __device__ __forceinline__ V operator*(V v) const { return v * a * b; }
};

// The states before each chunk (fp16, scaled), and the last one: 256 elements a
// workgroup, four a thread, and a run of kRun chunks a wave.  With four waves, each
// takes its run from zero first, S' = P S + T; what the runs before it make of the
// state it gets from their P and T.  Bound: latency (32 chunks of 8 KV heads of 128,
// 25 MB: 9 us; by one wave, chunk after chunk, 14; decays as one factor: 8).
template <int D, int kWaves>
__global__ __launch_bounds__(kWaves * 64) void scan_kernel(const LinArgs A) {
  constexpr uint32_t kBlocks = D * D / 256;
  constexpr int kRun = kScanRun, kSpan = kRun * kWaves;
  static_assert(kRun == 8, "a run's decays are summed over eight lanes");
  __shared__ f4 runs[kWaves > 1 ? kWaves : 1][64];
  // (heads fastest, as in the other launches, so that a head stays on an XCD: 8.1 against 8.9 us)
  const uint32_t rest = blockIdx.x / (uint32_t)A.hkv, blk = rest % kBlocks;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = blockIdx.x % (uint32_t)A.hkv, s = rest / kBlocks, at = blk * 256 + lane * 4;
  const int begin = cu_at(A.cu, s, A.rows), n = cu_at(A.cu, s + 1, A.rows) - begin;
  if (n <= 0) return;
  const int base = slot_base<kChunk, 1>(begin, s, 1), end = base + (n + kChunk - 1) / kChunk;
  const int lo = max(base, A.slot0), hi = min(end, A.slot0 + A.slots);
  if (lo >= hi) return;
  const int from = A.from[s], to = A.to[s], count = hi - lo;
  const int64_t r0 = (int64_t)(lo - A.slot0) * A.hkv + h;
  const float *u = A.u + r0 * (D * D) + at;
  const int64_t step = (int64_t)A.hkv * (D * D);
  _Float16 *snap = A.snap + r0 * (D * D) + at;
  Meta *meta = A.meta + r0;
  f4 x[kRun];
  Factors decay(0.0f), decay8(0.0f);  // of chunk c0 + lane, of the run that it is in
  float most;
  auto send_for = [&](int c0) {
#pragma unroll
    for (int i = 0; i < kRun; i++) x[i] = *reinterpret_cast<const f4 *>(u + min(c0 + wave * kRun + i, count - 1) * step);
    const Meta m = meta[(int64_t)min(c0 + lane, count - 1) * A.hkv];
    const float d = c0 + lane < count ? m.decay : 0.0f;
    decay = Factors(d);
    if (kWaves > 1) decay8 = Factors(row_sum8(d));
    most = c0 + lane < count ? m.most_u : 0.0f;
  };
  send_for(0);
  float *carry = A.carry + (int64_t)h * (D * D) + at;  // (one sequence may read it as another one writes: two of them)
  f4 S = {0, 0, 0, 0};
  if (lo > base) S = *reinterpret_cast<const f4 *>(A.carried + (int64_t)h * (D * D) + at);
  else if (state_ok(A, from)) S = *reinterpret_cast<const f4 *>(A.states + ((int64_t)from * A.hkv + h) * (D * D) + at);
  // of |S|, from the chunks' largest elements, held within fp32 (an infinite one would stay, as NaN, behind a reset)
  auto within = [](float v) { return fminf(v, 3.4e38f); };
  float bound = within(meta->most_s);
  auto most_of = [&](int c) { return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(most), c)); };
#pragma unroll 1
  for (int c0 = 0; c0 < count; c0 += kSpan) {
    const int c1 = c0 + wave * kRun;
    f4 mine = S;  // this run's start, and a bound of it
    float reach = bound;
    if constexpr (kWaves > 1) {
      f4 T = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < kRun; i++) {
        if (c1 + i >= count) x[i] = (f4){0, 0, 0, 0};
        T = decay.at(wave * kRun + i) * T + x[i];
      }
      runs[wave][lane] = T;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWaves; w++) {
        if (w == wave) {
          mine = S;
          reach = bound;
        }
        if (c0 + w * kRun >= count) break;
#pragma unroll
        for (int i = 0; i < kRun; i++) bound = within(decay.at(w * kRun + i) * bound + most_of(w * kRun + i));
        S = decay8.at(w * kRun) * S + runs[w][lane];
      }
    }
#pragma unroll
    for (int i = 0; i < kRun; i++) {
      const int c = c1 + i;
      if (c >= count) break;
      const int e = reach > 0.0f ? __builtin_amdgcn_frexp_expf(reach) - 15 : kNoState;
      const int sh16 = reach > 0.0f ? -e : 0;
      h4 o;
#pragma unroll
      for (int j = 0; j < 4; j++) o[j] = (_Float16)ldexpf(mine[j], sh16);
      *reinterpret_cast<h4 *>(snap + c * step) = o;
      if (blk == 0 && lane == 0) meta[(int64_t)c * A.hkv].e = e;
      const Factors f = decay.at(wave * kRun + i);
      reach = within(f * reach + most_of(wave * kRun + i));
      mine = f * mine + x[i];
    }
    if constexpr (kWaves == 1) {
      S = mine;
      bound = reach;
    }
    if (c0 + kSpan < count) {
      send_for(c0 + kSpan);
      if constexpr (kWaves > 1) __syncthreads();  // (the runs are read)
    }
  }
  if (wave) return;
  if (hi < end) *reinterpret_cast<f4 *>(carry) = S;
  else if (state_ok(A, to)) *reinterpret_cast<f4 *>(A.states + ((int64_t)to * A.hkv + h) * (D * D) + at) = S;
}

// The token of a 32-token group that row r of the score product takes: a lane
// then holds 8 consecutive tokens per 16, as the second product wants them.
__device__ __forceinline__ int row_token(int r) { return (r & 16) + ((r >> 2) & 1) * 8 + ((r >> 3) & 1) * 4 + (r & 3); }

__device__ __forceinline__ float half_max(float v) {
  const uint32_t b = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Outputs of a chunk: keys, values and the state in LDS; a wave takes 32 rows
// of a query head, then of another one (NW = 8: two heads at a time), its next
// queries on their way meanwhile.  The block of 32 rows changes from head to
// head, so that the waves' shares of the causal triangle come out even.
//
// Values, and fp32 keys and queries, have the unit of their own row (fp16 keys and
// queries stay as they are), and a row's weights, which take up the keys' and values',
// one by what they can reach: with z_j the exponent of a token's largest key times its
// largest value, h_j = z_j - G_j and H_i the largest h_j up to i (and 60 below the
// state's), a weight is at most 2^(h_j - H_i) times head_dim max |q|, whatever was
// forgotten before the row or comes behind it.  2^(h_j - H_i) is a factor of the row and
// one of the token, both at most 1, with H at the end of the token's 32 between them;
// among the row's own 32 tokens it is made as it stands.  (H_i is raised so that
// H_i + G_i is whole.)
//
// Bound: 4096 fp32 rows, 64 and 8 heads of 128, 240 MB and 17 GFLOP (44 issued, for
// second terms and whole blocks): 60 to 69 us, of them some 10 before the first
// product, one workgroup a CU (139 KB of LDS).  Matrix pipes busy 34 %, VALU 33 %.
template <int D, typename T, int NW>
__global__ __launch_bounds__(NW * 64) void chunk_out_kernel(const LinArgs A) {
  constexpr bool kWide = std::is_same<T, float>::value;
  constexpr int NT = NW * 64, kPer = kChunk * (D / 8) / NT, kTogether = NW / 4, kTerms = kWide ? 2 : 1;
  constexpr int kLogD = D == 128 ? 7 : 6;
  __shared__ __attribute__((aligned(16))) _Float16 kt[kTerms][kChunk][D + 8];
  __shared__ __attribute__((aligned(16))) uint8_t vt[kChunk * 2 * D], stt[D * 2 * D];
  // of tokens: h in two terms, 2^(h - H of its 32); of rows and of 32 tokens: H
  __shared__ __attribute__((aligned(16))) float hhi[kChunk], hlo[kChunk], wt[kChunk];
  __shared__ float khi[kChunk], klo[kChunk], block[kChunk / 32];
  __shared__ int size[kChunk], bias[kWide ? 1 : kChunk], ex[kChunk];  // z; 14 less an fp16 key's exponent; H + G
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t part = blockIdx.x % (uint32_t)A.parts, rh = blockIdx.x / (uint32_t)A.parts;
  const int h = rh % (uint32_t)A.hkv, rel = rh / (uint32_t)A.hkv;
  Chunk c;
  if (!find_chunk(A, A.slot0 + rel, c)) return;
  // this wave's head and row block of round i
  const int per = (A.group + A.parts - 1) / A.parts, g0 = part * per, heads = min(per, A.group - g0);
  const int rounds = (heads + kTogether - 1) / kTogether;
  auto head_of = [&](int i) { return i * kTogether + (wave >> 2); };
  auto block_of = [&](int i) { return wave < 4 ? (wave + i) & 3 : 3 - ((wave + i) & 3); };
  typedef typename std::conditional<kWide, f4, h8>::type Piece;
  constexpr int kPieces = D / 16 * (kWide ? 2 : 1);
  Piece raw[kPieces];
  // fp32 queries come in two halves, the second once the operands made of the last
  // ones are done with: all at once do not fit into the registers
  constexpr int kFirst = kWide ? kPieces / 2 : kPieces;
  auto send_for = [&](int i, int from, int to) {
    const int row = 32 * block_of(i) + n, head = h * A.group + g0 + min(head_of(i), heads - 1);
    const T *qp = (const T *)A.qkv + (int64_t)(c.begin + min(row, c.n - 1)) * A.row_stride + head * D + 8 * half;
#pragma unroll
    for (int j = 0; j < kPieces; j++)
      if (j >= from && j < to) raw[j] = *reinterpret_cast<const Piece *>(qp + (kWide ? 16 * (j >> 1) + 4 * (j & 1) : 16 * j));
  };
  if (heads <= 0) return;
  send_for(0, 0, kPieces);
  const int64_t rs = (int64_t)rel * A.hkv + h;
  const int es = A.meta[rs].e;
  const T *kp = (const T *)A.qkv + (int64_t)c.begin * A.row_stride + (A.hq + h) * D;
  const T *vp = kp + A.hkv * D;
  {
    typedef typename std::conditional<kWide, f8, h8>::type Eight;
    Eight k[kPer], v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i++) {
      const int p = i * NT + tid, row = p / (D / 8), at = p % (D / 8) * 8;
      k[i] = v[i] = (Eight)(0);
      if (row < c.n) {
        k[i] = load8(kp + row * A.row_stride + at);
        v[i] = load8(vp + row * A.row_stride + at);
      }
    }
    u4 sp[D * (D / 8) / NT];
    // (sent for before its exponent is known: without a state it is not used)
#pragma unroll
    for (int i = 0; i < D * (D / 8) / NT; i++) sp[i] = reinterpret_cast<const u4 *>(A.snap + rs * (D * D))[i * NT + tid];
    double g0 = 0.0, g1 = 0.0;
    if (wave == 0) decay_sums(A, c, h, g0, g1);
#pragma unroll
    for (int i = 0; i < kPer; i++) {
      const int p = i * NT + tid;
      bool a, b;
      const int ek = scale_row<D, kWide>(k[i], a), ev = scale_row<D>(v[i], b);
      if (p % (D / 8) == 0) {
        size[p / (D / 8)] = a && b ? ek + ev : kNothing;
        if (!kWide) bias[p / (D / 8)] = 14 - ek;
      }
    }
    if (es != kNoState) {
#pragma unroll
      for (int i = 0; i < D * (D / 8) / NT; i++) {
        const int p = i * NT + tid;
        *reinterpret_cast<u4 *>(stt + piece_at<D>(p / (D / 8), p % (D / 8))) = sp[i];
      }
    }
#pragma unroll
    for (int i = 0; i < kPer; i++) {
      const int p = i * NT + tid, row = p / (D / 8), at = p % (D / 8);
      h8 a, l, b;
      if constexpr (kWide) {
        two_terms(k[i], a, l);
        b = __builtin_convertvector(v[i], h8);
      } else {
        a = k[i];
        b = v[i];
      }
      *reinterpret_cast<h8 *>(&kt[0][row][8 * at]) = a;
      if constexpr (kWide) *reinterpret_cast<h8 *>(&kt[1][row][8 * at]) = l;
      *reinterpret_cast<h8 *>(vt + piece_at<D>(row, at)) = b;
    }
    __syncthreads();
    if (wave == 0) {
      double h0 = size[2 * lane] - g0, h1 = size[2 * lane + 1] - g1;
      // (largest ones to fp32's accuracy are enough: a weight may then pass its bound by as much)
      const float least = es != kNoState ? (float)(es + 15 - kLogD - 60) : -1e9f;
      const float m1 = fmaxf(wave_most_upto(fmaxf((float)h0, (float)h1)), least);
      const float before = __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(least), __float_as_int(m1), 0x138, 0xF, 0xF, false));
      const float m0 = fmaxf(before, (float)h0), last = __shfl(m1, lane | 15);  // up to the row, up to the end of its 32
      const double e0 = ceil((double)m0 + g0), e1 = ceil((double)m1 + g1), k0 = e0 - g0, k1 = e1 - g1;
      const int r = 2 * lane;
      if (!kWide) h0 += bias[r], h1 += bias[r + 1];  // (keys as they are)
      ex[r] = (int)e0, ex[r + 1] = (int)e1;
      khi[r] = (float)k0, klo[r] = (float)(k0 - (double)(float)k0);
      khi[r + 1] = (float)k1, klo[r + 1] = (float)(k1 - (double)(float)k1);
      hhi[r] = (float)h0, hlo[r] = (float)(h0 - (double)(float)h0);
      hhi[r + 1] = (float)h1, hlo[r + 1] = (float)(h1 - (double)(float)h1);
      wt[r] = __builtin_amdgcn_exp2f((float)(h0 - (double)last));
      wt[r + 1] = __builtin_amdgcn_exp2f((float)(h1 - (double)last));
      if ((lane & 15) == 15) block[lane >> 4] = last;
    }
  }
  __syncthreads();
  int scale_e;
  const float scale_m = frexpf(A.scale, &scale_e);
  const Turned<D> turned;

  // Outputs go through a buffer whose end drops the rows that are not there, so
  // that every round has the same stores behind its loads: the wait for the next
  // queries is then not a wait for the stores.
  const __amdgpu_buffer_rsrc_t out = __builtin_amdgcn_make_buffer_rsrc(A.out + (int64_t)c.begin * A.out_stride, 0, 0x7fffffff, 0x00027000);
  constexpr uint32_t kNowhere = 0x80000000u;

  // one round: rows 32 RB + n of a head.  (One copy for all four blocks, its tiles in a
  // loop: with a copy a block, 28 to 43 KB of code against 11 to 15, most of which a
  // wave runs once, fetching it took longer: 3 x 2051 fp16 rows 39 against 34 us.)
  auto rows = [&](int RB, int i, const h8 (&qf)[kTerms][D / 16], int bq) {
    const int row = 32 * RB + n, head = h * A.group + g0 + head_of(i);
    if (32 * RB >= c.n || head_of(i) >= heads) {
      send_for(min(i + 1, rounds - 1), kFirst, kPieces);
#pragma unroll
      for (int k = 0; k < D / 16; k++) __builtin_amdgcn_raw_buffer_store_b128((u4){0, 0, 0, 0}, out, kNowhere, 0, 0);
      return;
    }
    // o^T: o[d][r] is element 32 d + 8 (r / 4) + 4 half + r % 4 of the row, in
    // units of 2^(ex + bq + kLogD - 29): weights are below 2^15 in it, the state's part
    // below 2^97 (fp32 queries are scaled by 2^(14 - bq), fp16 ones as they are)
    const float kh = khi[row], kl = klo[row];
    const float unit = power((kWide ? 0 : 14 - bq) - 13 - kLogD);
    f16x o[D / 32];
#pragma unroll
    for (int d = 0; d < D / 32; d++) o[d] = (f16x)(0.0f);
    if (es != kNoState) {
#pragma unroll
      for (int j = 0; j < D / 16; j++)
#pragma unroll
        for (int d = 0; d < D / 32; d++) {
          const h8 a = turned(stt, 16 * j, d);
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, qf[0][j], o[d], 0, 0, 0);
          if constexpr (kWide) o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, qf[1][j], o[d], 0, 0, 0);
        }
      float f = __builtin_amdgcn_exp2f(((float)(es + 15 - kLogD) - kh) - kl);
      if (!kWide) f = ldexpf(f, 14 - bq);
#pragma unroll
      for (int d = 0; d < D / 32; d++)
#pragma unroll
        for (int r = 0; r < 16; r++) o[d][r] *= f;
    }
    auto tile = [&](auto last_tile, int t) {
      constexpr bool kLast = decltype(last_tile)::value;
      // scores S^T = K Q^T: sc[r] is token 32 t + 16 (r / 8) + 8 half + r % 8
      f16x sc = (f16x)(0.0f);
      const int key = 32 * t + row_token(n);
#pragma unroll
      for (int j = 0; j < D / 16; j++) {
        const h8 a = *reinterpret_cast<const h8 *>(&kt[0][key][16 * j + 8 * half]);
        sc = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, qf[0][j], sc, 0, 0, 0);
        if constexpr (kWide) {
          sc = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, qf[1][j], sc, 0, 0, 0);
          const h8 b = *reinterpret_cast<const h8 *>(&kt[1][key][16 * j + 8 * half]);
          sc = __builtin_amdgcn_mfma_f32_32x32x16_f16(b, qf[0][j], sc, 0, 0, 0);
        }
      }
      if (kLast) send_for(min(i + 1, rounds - 1), kFirst, kPieces);
      // weights: two fp16 terms, so that they lose nothing to the outputs' rounding
      const int j0 = 32 * t + 8 * half;
      h8 p[2], pl[2];
      const float f = kLast ? 0.0f : __builtin_amdgcn_exp2f((block[t] - kh) - kl) * unit;
#pragma unroll
      for (int u = 0; u < 2; u++) {
        f8 w;
#pragma unroll
        for (int r = 0; r < 8; r++) {
          const int j = j0 + 16 * u + r;
          if (kLast) {
            w[r] = sc[8 * u + r] * (__builtin_amdgcn_exp2f((hhi[j] - kh) + (hlo[j] - kl)) * unit);
            w[r] = j <= row ? w[r] : 0.0f;
          } else {
            w[r] = sc[8 * u + r] * (wt[j] * f);
          }
        }
        two_terms(w, p[u], pl[u]);
      }
#pragma unroll
      for (int u = 0; u < 2; u++)
#pragma unroll
        for (int d = 0; d < D / 32; d++) {
          const h8 a = turned(vt, 32 * t + 16 * u, d);
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, p[u], o[d], 0, 0, 0);
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, pl[u], o[d], 0, 0, 0);
        }
    };
#pragma unroll 1
    for (int t = 0; t < RB; t++) tile(std::false_type(), t);
    tile(std::true_type(), RB);
    // (held within fp32's exponents: sums are 0 or 2^-48 to 2^98, but for a state that is
    // nothing beside them, so a result that fp16 holds is not changed)
    const float last = scale_m * power(ex[row] + bq + kLogD - 29 + scale_e);
    // two quads' halves change places between the halves of the wave: 16 bytes a lane
    const uint32_t to = row < c.n ? 2u * (uint32_t)(row * (int)A.out_stride + head * D + 8 * half) : kNowhere;
#pragma unroll
    for (int d = 0; d < D / 32; d++)
#pragma unroll
      for (int r = 0; r < 16; r += 8) {
        uint32_t w[4];
#pragma unroll
        for (int i2 = 0; i2 < 4; i2++) {
          const h2 y = {(_Float16)(o[d][r + 2 * i2] * last), (_Float16)(o[d][r + 2 * i2 + 1] * last)};
          w[i2] = __builtin_bit_cast(uint32_t, y);
        }
        const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
        const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
        __builtin_amdgcn_raw_buffer_store_b128((u4){a[0], b[0], a[1], b[1]}, out, to + 2 * (32 * d + 2 * r), 0, 0);
      }
  };
#pragma unroll 1
  for (int i = 0; i < rounds; i++) {
    // the queries that have arrived, as operands (fp32: scaled, in two terms)
    h8 qf[kTerms][D / 16];
    float mq = 0.0f;
#pragma unroll
    for (int j = 0; j < kPieces; j++)
#pragma unroll
      for (int r = 0; r < (kWide ? 4 : 8); r++) mq = fmaxf(mq, fabsf((float)raw[j][r]));
    const int bq = __builtin_amdgcn_frexp_expf(half_max(mq));
    if constexpr (kWide) {
#pragma unroll
      for (int j = 0; j < D / 16; j++) {
        f8 x;
#pragma unroll
        for (int r = 0; r < 8; r++) x[r] = ldexpf((float)raw[kPieces / (D / 16) * j + (r >> 2)][r & 3], 14 - bq);
        two_terms(x, qf[0][j], qf[kTerms - 1][j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kPieces; j++)
#pragma unroll
        for (int r = 0; r < 8; r++) qf[0][j][r] = (_Float16)raw[j][r];
    }
    send_for(min(i + 1, rounds - 1), 0, kFirst);  // (again the last one's behind it, from the cache)
    rows(block_of(i), i, qf, bq);
  }
}

// (a chunk's outputs are addressed in 31 bits)
constexpr int64_t kMaxOutStride = (int64_t)1 << 22;

constexpr int kCus = 256;

struct Plan {
  bool chunked;
  int64_t slots, pass;  // chunks, and those of a pass
  size_t carry_bytes, meta_bytes, u_bytes, bytes;
};

Plan make_plan(int64_t rows, int64_t seqs, int64_t kv_heads, int64_t head_dim) {
  Plan P = {};
  P.chunked = rows > kFewRows * seqs;
  if (!P.chunked) return P;
  P.slots = rows / kChunk + seqs;
  const size_t state = (size_t)(kv_heads * head_dim * head_dim);
  const size_t each = state * 6 + (size_t)kv_heads * sizeof(Meta);
  P.pass = (int64_t)(kPassBytes / each);
  if (P.pass < 1) P.pass = 1;
  if (P.pass > P.slots) P.pass = P.slots;
  P.carry_bytes = P.pass < P.slots ? state * 8 : 0;
  P.meta_bytes = (size_t)(P.pass * kv_heads) * sizeof(Meta);
  P.u_bytes = (size_t)P.pass * state * 4;
  P.bytes = P.carry_bytes + P.meta_bytes + P.u_bytes + P.u_bytes / 2;
  return P;
}

int check_shape(int64_t rows, int64_t seqs, int64_t q_heads, int64_t kv_heads, int64_t head_dim) {
  const int rc = shape_check(rows, seqs, q_heads, kv_heads, head_dim, 1, 1);
  if (rc != TQ_OK) return rc;
  const Plan P = make_plan(rows, seqs, kv_heads, head_dim);
  const int64_t blocks = head_dim * head_dim / 256;
  const bool ok = P.chunked ? grid_ok(P.pass * q_heads + seqs * kv_heads, 512) && grid_ok(seqs * kv_heads * blocks, 256)
                            : grid_ok(seqs * kv_heads * (head_dim / 64), 256);
  return ok ? TQ_OK : TQ_ERR_SHAPE;
}

bool aligned_to(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

template <int D, typename T>
void launch_passes(LinArgs A, const Plan &P, hipStream_t st) {
  float *carried = A.carry + (int64_t)A.hkv * D * D;
  for (int64_t s0 = 0; s0 < P.slots; s0 += P.pass) {
    A.slot0 = (int)s0;
    std::swap(A.carry, carried);
    A.carried = carried;
    A.slots = (int)(P.slots - s0 < P.pass ? P.slots - s0 : P.pass);
    const int64_t units = (int64_t)A.slots * A.hkv;
    hipLaunchKernelGGL((chunk_state_kernel<D, T>), dim3((unsigned)(units + (int64_t)A.seqs * A.hkv)), dim3(512), 0, st, A);
    // four waves where sequences have more chunks than a run, on average (64 sequences
    // of 100 rows: 187 us with four waves, 111 with one)
    const dim3 blocks((unsigned)((int64_t)A.seqs * A.hkv * (D * D / 256)));
    if (P.slots > kScanRun * (int64_t)A.seqs) hipLaunchKernelGGL((scan_kernel<D, 4>), blocks, dim3(256), 0, st, A);
    else hipLaunchKernelGGL((scan_kernel<D, 1>), blocks, dim3(64), 0, st, A);
    // the query heads of a KV head over as many workgroups as fill the CUs
    const int most = A.group >= 2 ? A.group / 2 : 1;
    int64_t parts = kCus / units;
    A.parts = (int)(parts < 1 ? 1 : parts > most ? most : parts);
    const dim3 grid((unsigned)(units * A.parts));
    if (A.group >= 2) hipLaunchKernelGGL((chunk_out_kernel<D, T, 8>), grid, dim3(512), 0, st, A);
    else hipLaunchKernelGGL((chunk_out_kernel<D, T, 4>), grid, dim3(256), 0, st, A);
  }
}

}  // namespace

extern "C" size_t tq_linear_attn_scratch_bytes(int64_t rows, int64_t seqs, int64_t q_heads, int64_t kv_heads,
                                               int64_t head_dim) {
  if (check_shape(rows, seqs, q_heads, kv_heads, head_dim) != TQ_OK) return 0;
  return make_plan(rows, seqs, kv_heads, head_dim).bytes;
}

extern "C" int tq_linear_attn(int dtype, int64_t rows, int64_t seqs, int64_t q_heads, int64_t kv_heads,
                              int64_t head_dim, const void *qkv, int64_t row_stride, const float *log_decay,
                              int64_t decay_stride, const int32_t *cu_rows, const int32_t *state_from,
                              const int32_t *state_to, float *states, int64_t num_states, float scale, void *out,
                              int64_t out_stride, void *scratch, size_t scratch_bytes, void *stream) {
  if (!qkv || !log_decay || !cu_rows || !state_from || !state_to || !states || !out) return TQ_ERR_NULL;
  if (dtype != TQ_F16 && dtype != TQ_F32) return TQ_ERR_DTYPE;
  const int rc = check_shape(rows, seqs, q_heads, kv_heads, head_dim);
  if (rc != TQ_OK) return rc;
  if (row_stride < (q_heads + 2 * kv_heads) * head_dim || row_stride % 8 != 0 || row_stride > ((int64_t)1 << 31) ||
      (decay_stride != 0 && decay_stride < kv_heads) || decay_stride > ((int64_t)1 << 31) || num_states < 1 ||
      num_states > 0x7fffffff || out_stride < q_heads * head_dim || out_stride % 8 != 0 ||
      out_stride > kMaxOutStride)
    return TQ_ERR_SHAPE;
  if (!(scale > -3.0e38f && scale < 3.0e38f)) return TQ_ERR_VALUE;
  if (!aligned_to(qkv, 16) || !aligned_to(states, 16) || !aligned_to(out, 16) || !aligned_to(scratch, 16) ||
      !aligned_to(log_decay, 4) || !aligned_to(cu_rows, 4) || !aligned_to(state_from, 4) || !aligned_to(state_to, 4))
    return TQ_ERR_ALIGN;
  const Plan P = make_plan(rows, seqs, kv_heads, head_dim);
  if (P.bytes && !scratch) return TQ_ERR_NULL;
  if (scratch_bytes < P.bytes) return TQ_ERR_SIZE;
  LinArgs A = {};
  A.qkv = qkv; A.log_decay = log_decay; A.cu = cu_rows; A.from = state_from; A.to = state_to;
  A.states = states; A.out = (_Float16 *)out;
  A.row_stride = row_stride; A.decay_stride = decay_stride; A.out_stride = out_stride; A.num_states = num_states;
  A.scale = scale;
  A.rows = (int)rows; A.seqs = (int)seqs; A.hq = (int)q_heads; A.hkv = (int)kv_heads; A.group = (int)(q_heads / kv_heads);
  char *p = (char *)scratch;
  A.carry = (float *)p;
  A.meta = (Meta *)(p + P.carry_bytes);
  A.u = (float *)(p + P.carry_bytes + P.meta_bytes);
  A.snap = (_Float16 *)(p + P.carry_bytes + P.meta_bytes + P.u_bytes);
  hipStream_t st = (hipStream_t)stream;
#define TQ_LINEAR(D, T)                                                                                       \
  {                                                                                                           \
    if (P.chunked) launch_passes<D, T>(A, P, st);                                                             \
    else hipLaunchKernelGGL((recur_kernel<D, T>), dim3((unsigned)(seqs * kv_heads * (D / 64))), dim3(256), 0, st, A); \
  }
  if (head_dim == 128) {
    if (dtype == TQ_F16) TQ_LINEAR(128, _Float16) else TQ_LINEAR(128, float)
  } else {
    if (dtype == TQ_F16) TQ_LINEAR(64, _Float16) else TQ_LINEAR(64, float)
  }
#undef TQ_LINEAR
  return hipGetLastError() == hipSuccess ? TQ_OK : TQ_ERR_HIP;
}
