// Host side of the rotary positions: the table of frequencies.
#include <cmath>

#include "host_internal.h"

extern "C" svdq_status svdq_rope_frequencies(int32_t axes, const int32_t* dims, double theta, int32_t shared,
                                             float* turns, int32_t* axis) {
  if (!dims || !turns || !axis || !(theta > 0.0) || !std::isfinite(theta)) return SVDQ_ERR_ARG;
  if (axes < 1 || axes > SVDQ_ROPE_MAX_AXES) return SVDQ_ERR_SHAPE;
  int64_t total = 0;
  for (int a = 0; a < axes; ++a) {
    if (dims[a] < 0 || dims[a] % 2 != 0) return SVDQ_ERR_SHAPE;
    total += dims[a];
  }
  if (total < 16 || total > 512 || total % 16 != 0) return SVDQ_ERR_SHAPE;
  const double two_pi = 6.283185307179586476925286766559;
  int j = 0;
  for (int a = 0; a < axes; ++a) {
    for (int i = 0; i < dims[a] / 2; ++i, ++j) {
      const double e = shared ? 2.0 * j / (double)total : 2.0 * i / (double)dims[a];
      const double f = std::pow(theta, -e) / two_pi;
      if (!(f < 0x1p103)) return SVDQ_ERR_ARG;   // times a position below 2^24: within fp32
      const float hi = (float)f;
      turns[2 * j] = hi;
      turns[2 * j + 1] = (float)(f - (double)hi);
      axis[j] = a;
    }
  }
  return SVDQ_OK;
}
