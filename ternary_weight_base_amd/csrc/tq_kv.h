// tq_kv.h -- what the kernels of the paged 8-bit key/value cache share: the
// cache's geometry, the search of the sequence a workgroup belongs to, and
// the conversion of cache bytes.  Internal to the library.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tq.h"

namespace tqkv {

constexpr int kPage = 64;  // tokens of a page = tokens that share a scale

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));

// The rows of sequence s are cu[s] .. cu[s+1]-1.  Entries are clamped to
// 0..rows, so a caller's bad array can give wrong rows but no access outside
// the tensors.
__device__ __forceinline__ int cu_at(const int *cu, int i, int rows) { return min(max(cu[i], 0), rows); }

// Work is numbered without a scan over the sequences: sequence s owns the
// slots from base(s) = floor(cu[s] * mul / DIV) + s * ADD up to base(s+1).
// With DIV units of work a slot, floor(x) + 1 slots hold ceil(x) of them
// wherever the sequence starts, so every sequence has slots enough and the
// number of slots, floor(rows * mul / DIV) + seqs * ADD, is known on the
// host; slots past a sequence's need are left at once.  (shape_check bounds
// rows * q_heads below 2^31.)
template <int DIV, int ADD>
__device__ __forceinline__ int slot_base(int cu, int i, int mul) {
  return (int)((uint32_t)(cu * mul) / (uint32_t)DIV) + i * ADD;
}

// The last sequence whose base is <= w, searched 64 ways at a time by the
// lanes of a wave (every lane active; one round for up to 64 sequences).
// `first_row(i)`: a sequence's first row.
template <int DIV, int ADD, typename Rows>
__device__ __forceinline__ int find_seq(const Rows &first_row, int seqs, int w, int mul) {
  int lo = 0, hi = seqs;
  const int lane = threadIdx.x & 63;
  while (hi - lo > 1) {
    const int step = (int)((uint32_t)(hi - lo + 63) / 64u);
    const int i = lo + lane * step;
    const bool le = i < hi && slot_base<DIV, ADD>(first_row(min(i, hi)), i, mul) <= w;
    const int k = max((int)__popcll(__ballot(le)), 1);
    lo += (k - 1) * step;
    hi = min(hi, lo + step);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}
template <int DIV, int ADD>
__device__ __forceinline__ int find_seq(const int *cu, int seqs, int rows, int w, int mul) {
  return find_seq<DIV, ADD>([=](int i) { return cu_at(cu, i, rows); }, seqs, w, mul);
}

// Cache bytes as fp16 c = b - 128, exact: a byte under the fp16
// pattern of 1024 (0x64) reads 1024 + b.
__device__ __forceinline__ h2 codes2(uint32_t w, uint32_t sel) {
  const h2 x = __builtin_bit_cast(h2, __builtin_amdgcn_perm(w, 0x64646464u, sel));
  return x - (h2){(_Float16)1152.0f, (_Float16)1152.0f};
}
__device__ __forceinline__ h8 codes8(uint32_t w0, uint32_t w1) {
  const h2 a = codes2(w0, 0x00050004u), b = codes2(w0, 0x00070006u), c = codes2(w1, 0x00050004u),
           d = codes2(w1, 0x00070006u);
  return (h8){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Shape checks that the calls on the cache share.
inline int shape_check(int64_t rows, int64_t seqs, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                       int64_t max_pages, int64_t num_pages) {
  if (rows < 1 || rows > ((int64_t)1 << 24) || seqs < 1 || seqs > ((int64_t)1 << 20) || kv_heads < 1 ||
      q_heads < kv_heads || q_heads > 4096 || q_heads % kv_heads != 0 || (head_dim != 64 && head_dim != 128) ||
      rows * q_heads >= ((int64_t)1 << 30) || max_pages < 1 || max_pages > ((int64_t)1 << 25) || num_pages < 1 || num_pages > 0x7fffffff)
    return TQ_ERR_SHAPE;
  return TQ_OK;
}

// A launch counts its threads in 32 bits.
inline bool grid_ok(int64_t wgs, int64_t threads) { return wgs <= 0xffffffffll / threads; }

}  // namespace tqkv
