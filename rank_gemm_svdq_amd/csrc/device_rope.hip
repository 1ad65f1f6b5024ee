// Rotary positions with several axes, for queries and keys in one launch.
//
// Pair j of every head of token m turns by t = 2 pi f_j p with
// p = positions[m, axis[j]].  f_j comes as hi + lo in turns: p hi is split
// into its rounded value and the rounding error (one fma), whole turns are
// dropped from the rounded value exactly, and the error and p lo are added to
// the fraction.  The angle is then good to about 2^-24 of a turn at any
// position.
//
// A block takes a few tokens (or a share of the heads of one): its angles go to
// LDS once, while the first elements are on their way, and its threads walk
// over (token, head) pairs with them, four in flight.  A lane owns 8 elements
// of a head: 4 neighbouring pairs, or 8 firsts and their 8 partners.  Bytes
// bound it: every element is read and written once.  4608 tokens x 48 heads of
// 128: 22.5 - 23.7 us, 4.8 - 5.0 TB/s (a large copy: 5.2 TB/s).

#include "device_block.h"

namespace svdq {
namespace {

constexpr int kTable = 256;   // angles of a block in LDS

struct RopeP {
  const int32_t* pos;
  const float* turns;
  const int32_t* axis;
  const uint16_t* x[2];
  uint16_t* y[2];
  int64_t xt[2], xh[2], yt[2], yh[2];
  int M, axes, pairs, heads0, heads, units, tokens, share;   // tokens of a block; heads of a block if tokens == 1
};

__device__ __forceinline__ float2 angle(const RopeP& p, int m, int j) {
  const int a = p.axis[j];
  const float at = (float)p.pos[(size_t)m * p.axes + ((unsigned)a < (unsigned)p.axes ? a : 0)];
  const float hi = p.turns[2 * j], lo = p.turns[2 * j + 1];
  const float t = at * hi;
  const float err = fmaf(at, hi, -t);
  const float f = (t - rintf(t)) + fmaf(at, lo, err);
  float s, c;
  sincospif(2.0f * f, &s, &c);
  return make_float2(c, s);
}

template <int DT, bool INTER>
__global__ __launch_bounds__(256) void rope_kernel(RopeP p) {
  constexpr int NP = INTER ? 4 : 8;   // pairs of a lane
  constexpr int IN = 4;               // elements in flight
  __shared__ __attribute__((aligned(16))) float2 table[kTable];
  const int per = 256 / p.units;                              // (token, head) pairs at a time
  const int u = threadIdx.x % p.units, slot = threadIdx.x / p.units;
  const int m0 = blockIdx.x * p.tokens, nt = min(p.tokens, p.M - m0);
  const int h0 = blockIdx.y * p.share, nh = min(p.share, p.heads - h0);
  const int turned = p.pairs / NP;    // units that turn; the others copy
  const bool turn = u < turned;
  const int d0 = INTER ? 8 * u : (turn ? 8 * u : 2 * p.pairs + 8 * (u - turned));
  const int items = slot < per ? nt * nh : 0;

  b4i a[IN], b[IN];
  int tok[IN];
  uint16_t* to[IN];
  int t = slot / nh, h = slot % nh, item = slot;              // of the next element to fetch
  auto fetch = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < IN; ++i) {
      to[i] = nullptr;
      if (item < items) {
        const int head = h0 + h, g = head >= p.heads0, hh = g ? head - p.heads0 : head;
        const uint16_t* xp = p.x[g] + (size_t)(m0 + t) * p.xt[g] + (size_t)hh * p.xh[g] + d0;
        a[i] = *reinterpret_cast<const b4i*>(xp);
        if (!INTER && turn) b[i] = *reinterpret_cast<const b4i*>(xp + p.pairs);
        to[i] = p.y[g] + (size_t)(m0 + t) * p.yt[g] + (size_t)hh * p.yh[g] + d0;
        tok[i] = t;
        item += per;
        h += per;
        while (h >= nh) {
          h -= nh;
          ++t;
        }
      }
    }
  };
  fetch();
  for (int i = threadIdx.x; i < nt * p.pairs; i += 256) table[i] = angle(p, m0 + i / p.pairs, i % p.pairs);
  __syncthreads();
  while (to[0] != nullptr) {
#pragma unroll
    for (int i = 0; i < IN; ++i) {
      if (to[i] == nullptr) continue;
      if (!turn) {
        *reinterpret_cast<b4i*>(to[i]) = a[i];
        continue;
      }
      const float2* cs = table + tok[i] * p.pairs + NP * u;
      float va[8], o[8];
      widen8<DT>(a[i], va);
      if constexpr (INTER) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 w = cs[k];
          o[2 * k] = va[2 * k] * w.x - va[2 * k + 1] * w.y;
          o[2 * k + 1] = va[2 * k] * w.y + va[2 * k + 1] * w.x;
        }
        *reinterpret_cast<b4i*>(to[i]) = narrow8<DT>(o);
      } else {
        float vb[8], o2[8];
        widen8<DT>(b[i], vb);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 w = cs[k];
          o[k] = va[k] * w.x - vb[k] * w.y;
          o2[k] = va[k] * w.y + vb[k] * w.x;
        }
        *reinterpret_cast<b4i*>(to[i]) = narrow8<DT>(o);
        *reinterpret_cast<b4i*>(to[i] + p.pairs) = narrow8<DT>(o2);
      }
    }
    fetch();
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
  p.heads0 = a->heads[0];
  p.heads = a->heads[0] + a->heads[1];
  const bool inter = a->interleaved != 0;
  p.units = inter ? a->head_dim / 8 : p.pairs / 8 + (a->head_dim - 2 * p.pairs) / 8;
  const int per = 256 / p.units;
  if (a->M > 256) {
    // all heads of a token, or of the few tokens that keep every thread at work
    // (4608 tokens x 48 heads of 128: 23.7 us with one token a block, 24.8 with
    // four, 29.1 with a third of the heads)
    const int fill = per / p.heads, most = kTable / p.pairs;
    p.tokens = fill > most ? most : fill > 1 ? fill : 1;
    p.share = p.heads;
  } else {
    // few tokens: heads spread over blocks (16 tokens x 40 heads: 2.9 us
    // against 3.3 us)
    p.tokens = 1;
    p.share = per < p.heads ? per : p.heads;
  }
  const dim3 grid((a->M + p.tokens - 1) / p.tokens, (p.heads + p.share - 1) / p.share), block(256);
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
