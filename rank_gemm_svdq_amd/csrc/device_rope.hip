// Rotary positions with several axes, for queries and keys in one launch.
//
// Pair j of every head of token m turns by t = 2 pi f_j p with
// p = positions[m, axis[j]].  f_j comes as hi + lo in turns: p hi is split
// into its rounded value and the rounding error (one fma), whole turns are
// dropped from the rounded value exactly, and the error and p lo are added to
// the fraction.  The angle is then good to about 2^-24 of a turn at any
// position.
//
// A lane owns 8 elements of a head (4 neighbouring pairs, or 8 firsts and
// their 8 partners half a head on), computes its sines once and walks over
// heads of its token with them.  Bytes bound it: every element is read and
// written once.

#include "device_block.h"

namespace svdq {
namespace {

struct RopeP {
  const int32_t* pos;
  const float* turns;
  const int32_t* axis;
  const uint16_t* x[2];
  uint16_t* y[2];
  int64_t xt[2], xh[2], yt[2], yh[2];
  int M, axes, pairs, D, heads0, heads, units, hstep;
};

__device__ __forceinline__ void angle(const RopeP& p, int m, int j, float* c, float* s) {
  const int a = p.axis[j];
  const float at = (float)p.pos[(size_t)m * p.axes + ((unsigned)a < (unsigned)p.axes ? a : 0)];
  const float hi = p.turns[2 * j], lo = p.turns[2 * j + 1];
  const float t = at * hi;
  const float err = fmaf(at, hi, -t);
  const float f = (t - rintf(t)) + fmaf(at, lo, err);
  sincospif(2.0f * f, s, c);
}

template <int DT, bool INTER>
__global__ __launch_bounds__(256) void rope_kernel(RopeP p) {
  constexpr int NP = INTER ? 4 : 8;   // pairs of a lane
  // units: lanes that cover one head (rotated chunks first, then copied ones)
  const int per = blockDim.x / p.units;                       // head slots of a block
  const int u = threadIdx.x % p.units, slot = threadIdx.x / p.units;
  if (slot >= per) return;
  const int m = blockIdx.x;
  const int turned = p.pairs / NP;
  const int d0 = INTER ? 8 * u : (u < turned ? 8 * u : 2 * p.pairs + 8 * (u - turned));
  float c[NP], s[NP];
  const bool turn = u < turned;
  if (turn) {
#pragma unroll
    for (int i = 0; i < NP; ++i) angle(p, m, NP * u + i, &c[i], &s[i]);
  }
  for (int h = blockIdx.y * per + slot; h < p.heads; h += p.hstep) {
    const int grp = h >= p.heads0;
    const int hh = grp ? h - p.heads0 : h;
    const uint16_t* xp = p.x[grp] + (size_t)m * p.xt[grp] + (size_t)hh * p.xh[grp] + d0;
    uint16_t* yp = p.y[grp] + (size_t)m * p.yt[grp] + (size_t)hh * p.yh[grp] + d0;
    const b4i a = *reinterpret_cast<const b4i*>(xp);
    if (!turn) {
      *reinterpret_cast<b4i*>(yp) = a;
      continue;
    }
    float va[8], o[8];
    widen8<DT>(a, va);
    if constexpr (INTER) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[2 * i] = va[2 * i] * c[i] - va[2 * i + 1] * s[i];
        o[2 * i + 1] = va[2 * i] * s[i] + va[2 * i + 1] * c[i];
      }
      *reinterpret_cast<b4i*>(yp) = narrow8<DT>(o);
    } else {
      const b4i b = *reinterpret_cast<const b4i*>(xp + p.pairs);
      float vb[8], o2[8];
      widen8<DT>(b, vb);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[i] = va[i] * c[i] - vb[i] * s[i];
        o2[i] = va[i] * s[i] + vb[i] * c[i];
      }
      *reinterpret_cast<b4i*>(yp) = narrow8<DT>(o);
      *reinterpret_cast<b4i*>(yp + p.pairs) = narrow8<DT>(o2);
    }
  }
}

}  // namespace
}  // namespace svdq

using namespace svdq;

extern "C" svdq_status svdq_rope(const svdq_rope_args* a, void* stream) {
  if (!a || !a->positions || !a->turns || !a->axis || !a->x[0] || !a->y[0]) return SVDQ_ERR_ARG;
  if (!is_dtype(a->dtype)) return SVDQ_ERR_UNSUPPORTED;
  if (a->M < 1 || a->M > (1 << 20) || a->axes < 1 || a->axes > SVDQ_ROPE_MAX_AXES) return SVDQ_ERR_SHAPE;
  if (a->head_dim < 16 || a->head_dim > 512 || a->head_dim % 8 != 0) return SVDQ_ERR_SHAPE;
  if (a->pairs < 8 || a->pairs % 8 != 0 || 2 * a->pairs > a->head_dim) return SVDQ_ERR_SHAPE;
  if (a->heads[0] < 1 || a->heads[1] < 0 || (int64_t)a->heads[0] + a->heads[1] > 65536) return SVDQ_ERR_SHAPE;
  if (a->heads[1] > 0 && (!a->x[1] || !a->y[1])) return SVDQ_ERR_ARG;
  if (!on4(a->positions) || !on4(a->turns) || !on4(a->axis)) return SVDQ_ERR_ALIGN;
  for (int g = 0; g < (a->heads[1] > 0 ? 2 : 1); ++g) {
    if (!on16(a->x[g]) || !on16(a->y[g]) || a->x_token[g] % 8 || a->x_head[g] % 8 || a->y_token[g] % 8 ||
        a->y_head[g] % 8)
      return SVDQ_ERR_ALIGN;
    if (a->x[g] == a->y[g] && (a->x_token[g] != a->y_token[g] || a->x_head[g] != a->y_head[g])) return SVDQ_ERR_ARG;
  }
  const svdq_status ok = device_ok();
  if (ok != SVDQ_OK) return ok;
  RopeP p;
  p.pos = a->positions;
  p.turns = a->turns;
  p.axis = a->axis;
  for (int g = 0; g < 2; ++g) {
    p.x[g] = a->x[g];
    p.y[g] = a->y[g];
    p.xt[g] = a->x_token[g];
    p.xh[g] = a->x_head[g];
    p.yt[g] = a->y_token[g];
    p.yh[g] = a->y_head[g];
  }
  p.M = a->M;
  p.axes = a->axes;
  p.pairs = a->pairs;
  p.D = a->head_dim;
  p.heads0 = a->heads[0];
  p.heads = a->heads[0] + a->heads[1];
  const bool inter = a->interleaved != 0;
  p.units = inter ? p.D / 8 : p.pairs / 8 + (p.D - 2 * p.pairs) / 8;
  const int per = 256 / p.units;
  const int need = (p.heads + per - 1) / per;
  const int gy = a->M >= 4 * device_cus() ? 1 : need;
  p.hstep = gy * per;
  const dim3 grid(a->M, gy), block(256);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (a->dtype == SVDQ_BF16) {
    if (inter) hipLaunchKernelGGL((rope_kernel<SVDQ_BF16, true>), grid, block, 0, st, p);
    else hipLaunchKernelGGL((rope_kernel<SVDQ_BF16, false>), grid, block, 0, st, p);
  } else {
    if (inter) hipLaunchKernelGGL((rope_kernel<SVDQ_FP16, true>), grid, block, 0, st, p);
    else hipLaunchKernelGGL((rope_kernel<SVDQ_FP16, false>), grid, block, 0, st, p);
  }
  return launched();
}
