// Scores of the attention kernels: scale, cap, powers of two.  P is a kernel's
// arguments: a.softcap and what set_score() fills in.
#pragma once

#include "device_block.h"

namespace svdq {
namespace {

constexpr float kLow = -3.402823466e38f;
__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// Capped score in powers of two of a raw dot product s: cap tanh(x) log2 e with
// x = s scale / cap, scale > 0, in one of two forms.
//   by_exp    cap - 2 cap / (e^2x + 1): five instructions, but a difference of two
//             numbers of the cap's size, so the score is off by up to 2e-7 cap
//             whatever its own size.
//   by_series s (scale log2 e) tanh(x) / x, the quotient a polynomial of degree 6
//             in x^2 (minimax on |x| <= 1, 5.6e-8 relative); beyond, by_exp, whose
//             error there is 3e-7 of the result.  As exact under a cap of 1e30 as
//             without one.
// Caps up to kSmallCap take by_exp: its error is then below 1.3e-5, that of the
// weight 2^-16, and the 16-bit weights are off by 2^-11 or 2^-8 anyway.
// The series is slower (2 x 1000 causal queries of 16 heads of 128 36.9 against
// 34.1 us, 4 x 1024 of 8 heads of 64 30.3 against 26.9; the latter under a cap of
// 2, where tiles need both, 39.4).
constexpr float kSmallCap = 64.0f;
constexpr float kTanh[7] = {1.0f,           -0.33332987f,   0.13326409f, -0.053498708f,
                            0.020359759f,   -0.0062593391f, 0.0010582646f};
template <class P>
__device__ __forceinline__ float by_exp(const P& p, float s) {
  return fmaf(-2.0f * p.c3, __builtin_amdgcn_rcpf(exp2_(s * p.c2) + 1.0f), p.c3);
}
template <class P>
__device__ __forceinline__ float by_series(const P& p, float s) {   // |x| <= 1
  const float x = s * p.c4, u = x * x;
  float q = p.cap[6];
#pragma unroll
  for (int i = 5; i >= 0; --i) q = fmaf(q, u, p.cap[i]);
  return s * q;
}
template <class P>
__device__ __forceinline__ float capped(const P& p, float s) {
  return p.a.softcap <= kSmallCap || !(fabsf(s * p.c4) <= 1.0f) ? by_exp(p, s) : by_series(p, s);
}

template <class P>
void set_score(P* p, float by, float softcap) {
  // A negative scale turns the signs of Q, scale 0 makes Q zero; what remains
  // is positive, so a hidden score of -infinity stays one when scaled.
  constexpr float log2e = 1.44269504088896f;
  const float scale = by < 0.f ? -by : by > 0.f ? by : 1.f;
  p->flip = by < 0.f;
  p->qmul = by < 0.f ? -1.f : by > 0.f ? 1.f : 0.f;
  // all finite, so that a score of 0 stays 0 at the largest scale and under the
  // smallest cap
  p->c1 = fminf(scale * log2e, 3.0e38f);
  p->c2 = softcap > 0.f ? fminf(2.f * scale / softcap * log2e, 3.0e38f) : 0.f;
  p->c3 = softcap * log2e;
  p->c4 = softcap > 0.f ? fminf(scale / softcap, 3.0e38f) : 0.f;
  for (int i = 0; i < 7; ++i) p->cap[i] = p->c1 * kTanh[i];
}

}  // namespace
}  // namespace svdq
