// tq_norm.hip -- the step between two blocks of a decoder layer in one pass:
// norm of the block's output, its gate, the scaled residual addition, and the
// norm of the next block's input, rounded or quantised for its projection.
//
//   u  = y / rms(y) * post_w                 (rms(v) = sqrt(mean v^2 + eps))
//   r' = round(res + res_scale * gate * u)   stored
//   x  = r' / rms(r') * pre_w                of the stored r'
//
// Sums and products run in double: the squares of fp32 values are exact there,
// and the results do not depend on the order of the sums but in one rounding
// to fp32 out of some 2^28, so x and its int8 codes match a plain evaluation
// in 64 bits.  Its rate is not what bounds the kernel.
//
// Bound: memory (each input read once, each output written once), or for few
// rows the latency of one load, two reductions and a store.  One workgroup
// per row; the row stays in registers from the first load to the last store.
//
// Measured: 2048 rows of 5120, fp32 with a gate row each, to the residual and
// int8, 39 us, 4.5 TB/s of 178 MB (a large copy reaches 4.8); one row 4.1 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tq.h"
#include "tq_device.h"
#include "tq_wave.h"

namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));

struct NormArgs {
  const void *y, *gate, *res;
  void *res_out, *x;
  const float *post_w, *pre_w;
  int8_t *q;
  float *a_scale;
  int64_t gate_stride;
  double res_scale, eps;
  int H, x_f32;
};

// V consecutive elements (1 or 4), as floats.
template <int V>
__device__ __forceinline__ void load(const float *p, float (&v)[V]) {
  if constexpr (V == 4) {
    const f4 a = *reinterpret_cast<const f4 *>(p);
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = a[i];
  } else {
    v[0] = *p;
  }
}
template <int V>
__device__ __forceinline__ void load(const _Float16 *p, float (&v)[V]) {
  if constexpr (V == 4) {
    const h4 a = *reinterpret_cast<const h4 *>(p);
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = (float)a[i];
  } else {
    v[0] = (float)*p;
  }
}
template <int V>
__device__ __forceinline__ void store(float *p, const float (&v)[V]) {
  if constexpr (V == 4)
    *reinterpret_cast<f4 *>(p) = (f4){v[0], v[1], v[2], v[3]};
  else
    *p = v[0];
}
template <int V>
__device__ __forceinline__ void store(_Float16 *p, const float (&v)[V]) {
  if constexpr (V == 4)
    *reinterpret_cast<h4 *>(p) = (h4){(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
  else
    *p = (_Float16)v[0];
}

template <int NT>
__device__ __forceinline__ double block_sum(double v, double *part) {
  v = tqdev::wave_sum64(v);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < NT / 64; w++) s += part[w];
  return s;
}

// EARLY: the weights and the gate are sent for with the row, else where they
// are used.  It pays where a thread has one item (1 x 1024: 3.07 against 3.16 us,
// 2048 x 1024: 9.2 against 9.4), not with more registers to hold (1 x 5120:
// 5.11 against 4.71 us, 1024 x 5120: 23.3 against 16.4).
template <typename TY, typename TR, int V, int NT, int ITEMS>
__global__ __launch_bounds__(NT) void residual_norm_kernel(const NormArgs A) {
  __shared__ double part[2][NT / 64];
  __shared__ float wmax[NT / 64];
  const int tid = threadIdx.x, H = A.H;
  const int64_t row = blockIdx.x;
  const TY *y = A.y ? (const TY *)A.y + row * H : nullptr;
  const TY *gate = A.gate ? (const TY *)A.gate + row * A.gate_stride : nullptr;
  const TR *res = (const TR *)A.res + row * H;
  float r[ITEMS][V], u[ITEMS][V];
  constexpr bool EARLY = ITEMS == 1;
  float ew[V], eg[V], ep[V];
  // weight, gate and next weight of item i (ones where there are none)
  auto get = [&](const auto *p, int e, float (&v)[V]) {
#pragma unroll
    for (int j = 0; j < V; j++) v[j] = 1.0f;
    if (p && e < H) load<V>(p + e, v);
  };
#pragma unroll
  for (int i = 0; i < ITEMS; i++) {
    const int e = (i * NT + tid) * V;
#pragma unroll
    for (int j = 0; j < V; j++) r[i][j] = u[i][j] = 0.0f;
    if (e < H) {
      load<V>(res + e, r[i]);
      if (y) load<V>(y + e, u[i]);
    }
    if constexpr (EARLY) {
      get(A.post_w, e, ew);
      get(gate, e, eg);
      get(A.pre_w, e, ep);
    }
  }
  if (y) {
    double inv = 1.0;
    if (A.post_w) {
      double ss = 0.0;
#pragma unroll
      for (int i = 0; i < ITEMS; i++)
#pragma unroll
        for (int j = 0; j < V; j++) ss += (double)u[i][j] * (double)u[i][j];
      inv = 1.0 / sqrt(block_sum<NT>(ss, part[0]) / H + A.eps);
    }
#pragma unroll
    for (int i = 0; i < ITEMS; i++) {
      const int e = (i * NT + tid) * V;
      if (e < H) {
        if constexpr (!EARLY) {
          get(A.post_w, e, ew);
          get(gate, e, eg);
        }
#pragma unroll
        for (int j = 0; j < V; j++)
          r[i][j] = (float)(TR)tqdev::round_f32(
              (double)r[i][j] + A.res_scale * ((double)u[i][j] * inv * (double)ew[j] * (double)eg[j]));
      }
    }
  }
  if (A.res_out) {
    TR *o = (TR *)A.res_out + row * H;
#pragma unroll
    for (int i = 0; i < ITEMS; i++) {
      const int e = (i * NT + tid) * V;
      if (e < H) store<V>(o + e, r[i]);
    }
  }
  if (!A.x && !A.q) return;
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < ITEMS; i++)
#pragma unroll
    for (int j = 0; j < V; j++) ss += (double)r[i][j] * (double)r[i][j];
  const double inv = 1.0 / sqrt(block_sum<NT>(ss, part[1]) / H + A.eps);
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < ITEMS; i++) {
    const int e = (i * NT + tid) * V;
    if (e < H) {
      if constexpr (!EARLY) get(A.pre_w, e, ep);
#pragma unroll
      for (int j = 0; j < V; j++) {
        r[i][j] = tqdev::round_f32((double)r[i][j] * inv * (double)ep[j]);
        m = fmaxf(m, fabsf(r[i][j]));
      }
      if (A.x) {
        if (A.x_f32)
          store<V>((float *)A.x + row * H + e, r[i]);
        else
          store<V>((_Float16 *)A.x + row * H + e, r[i]);
      }
    }
  }
  if (!A.q) return;
  // int8 by absmax as tq_quant_act, the factor by a reciprocal: 127 (1 / a).  That is
  // what x * (127 / a) comes to for a tensor a in torch, and what the header says:
  // a plain evaluation there gives the same codes.  (tq_quant_act divides once, 127 / a;
  // at most one code in 2^15 differs, by one step, as the factors differ by 2^-23.)
  m = tqdev::wave_max64(m);
  if ((tid & 63) == 0) wmax[tid >> 6] = m;
  __syncthreads();
  float amax = 0.0f;
#pragma unroll
  for (int w = 0; w < NT / 64; w++) amax = fmaxf(amax, wmax[w]);
  const bool zero = amax == 0.0f;
  // a maximum whose reciprocal would overflow is moved up first, and so are
  // the values (exact: powers of two)
  const float up = amax < 0x1p-100f ? 0x1p100f : 1.0f;
  const float qi = zero ? 0.0f : 127.0f * (1.0f / (amax * up));  // two IEEE roundings
  int8_t *q = A.q + row * H;
#pragma unroll
  for (int i = 0; i < ITEMS; i++) {
    const int e = (i * NT + tid) * V;
    if (e < H) {
      uint32_t pk = 0;
#pragma unroll
      for (int j = 0; j < V; j++) {
        const float t = fminf(fmaxf(rintf(r[i][j] * up * qi), -127.0f), 127.0f);
        pk |= (uint32_t)(uint8_t)(int8_t)(zero ? 0 : (int)t) << (8 * j);
      }
      if constexpr (V == 4)
        *reinterpret_cast<uint32_t *>(q + e) = pk;
      else
        q[e] = (int8_t)pk;
    }
  }
  if (tid == 0) A.a_scale[row] = zero ? 0.0f : amax / 127.0f;
}

template <typename TY, typename TR>
void launch(const NormArgs &A, int64_t M, hipStream_t st) {
  const dim3 grid((unsigned)M);
  const int H = A.H;
#define TQ_NORM(V, NT, ITEMS) hipLaunchKernelGGL((residual_norm_kernel<TY, TR, V, NT, ITEMS>), grid, dim3(NT), 0, st, A)
  // threads for 4 to 16 elements each (2048 x 5120: 512 threads 36.8 us, 256 38.3,
  // 1024 38.0; 1 x 5120: 4.75, 6.4, 4.8; 4096 x 4096: 512 51.3, 256 55.4, 1024 57.3)
  if (H % 4 == 0) {
    if (H <= 1024) {
      TQ_NORM(4, 256, 1);
    } else if (H <= 4096) {
      TQ_NORM(4, 512, 2);
    } else if (H <= 6144) {
      TQ_NORM(4, 512, 3);
    } else if (H <= 8192) {
      TQ_NORM(4, 512, 4);
    } else if (H <= 16384) {
      TQ_NORM(4, 1024, 4);
    } else {
      TQ_NORM(4, 1024, 8);
    }
  } else {
    if (H <= 1024) TQ_NORM(1, 256, 4);
    else if (H <= 8192) TQ_NORM(1, 512, 16);
    else TQ_NORM(1, 1024, 32);
  }
#undef TQ_NORM
}

bool aligned_to(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool is_act(int t) { return t == TQ_F16 || t == TQ_F32; }

}  // namespace

extern "C" int tq_residual_norm(int y_dtype, int res_dtype, int x_dtype, int64_t M, int64_t H, const void *y,
                                const float *post_w, const void *gate, int64_t gate_stride, double res_scale,
                                const void *res, void *res_out, const float *pre_w, double eps, void *x,
                                int8_t *q, float *a_scale, void *stream) {
  if (!res || (q && !a_scale) || (!x && !q && !res_out) || (y && !res_out) || (!y && (post_w || gate)))
    return TQ_ERR_NULL;
  if (!is_act(res_dtype) || (y && !is_act(y_dtype)) || (x && !is_act(x_dtype))) return TQ_ERR_DTYPE;
  // a launch counts its threads, up to 1024 a row, in 32 bits
  if (M < 1 || M >= ((int64_t)1 << 22) || H < 1 || H > 32768 ||
      (gate && gate_stride != 0 && (gate_stride < H || gate_stride > ((int64_t)1 << 31) || (H % 4 == 0 && gate_stride % 4 != 0))))
    return TQ_ERR_SHAPE;
  if (!(eps >= 0.0) || !(eps < 1e30) || !(res_scale > -1e30 && res_scale < 1e30)) return TQ_ERR_VALUE;
  if (!aligned_to(y, 16) || !aligned_to(post_w, 16) || !aligned_to(gate, 16) || !aligned_to(res, 16) ||
      !aligned_to(res_out, 16) || !aligned_to(pre_w, 16) || !aligned_to(x, 16) || !aligned_to(q, 16) ||
      !aligned_to(a_scale, 4))
    return TQ_ERR_ALIGN;
  NormArgs A;
  A.y = y; A.gate = gate; A.res = res; A.res_out = res_out; A.x = x;
  A.post_w = post_w; A.pre_w = pre_w; A.q = q; A.a_scale = a_scale;
  A.gate_stride = gate_stride; A.res_scale = res_scale; A.eps = eps;
  A.H = (int)H; A.x_f32 = x_dtype == TQ_F32;
  hipStream_t st = (hipStream_t)stream;
  if (!y) y_dtype = TQ_F32;
  if (y_dtype == TQ_F16) {
    if (res_dtype == TQ_F16) launch<_Float16, _Float16>(A, M, st);
    else launch<_Float16, float>(A, M, st);
  } else {
    if (res_dtype == TQ_F16) launch<float, _Float16>(A, M, st);
    else launch<float, float>(A, M, st);
  }
  return hipGetLastError() == hipSuccess ? TQ_OK : TQ_ERR_HIP;
}
