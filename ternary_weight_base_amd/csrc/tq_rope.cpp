// tq_rope.cpp -- the table of rotation angles that tq_kv_append reads.
#include <math.h>

#include "tq.h"

// cos and sin of position * base^(-2 i / rot): angles of far positions need
// 64 bits (position 131000 times a frequency rounded to fp32 is off by up to
// 0.008 rad), the table's entries are rounded to fp32 once.
extern "C" int tq_rope_table(int64_t positions, int64_t rot, double base, float *table) {
  if (!table) return TQ_ERR_NULL;
  if (positions < 1 || positions > ((int64_t)1 << 31) || rot < 8 || rot > 128 || rot % 8 != 0) return TQ_ERR_SHAPE;
  if (!(base > 1.0) || !isfinite(base)) return TQ_ERR_VALUE;
  const int64_t half = rot / 2;
  double freq[64];
  for (int64_t i = 0; i < half; i++) freq[i] = pow(base, -2.0 * (double)i / (double)rot);
#pragma omp parallel for schedule(static)
  for (int64_t p = 0; p < positions; p++)
    for (int64_t i = 0; i < half; i++) {
      const double a = (double)p * freq[i];
      table[p * rot + i] = (float)cos(a);
      table[p * rot + half + i] = (float)sin(a);
    }
  return TQ_OK;
}
