// The end of a block and the start of the next: norms on both sides of the
// block's gate and residual sum, modulation, 16-bit values and FP8 codes.
//
//   b = post(x) w';  h = a r + g b;  y = pre(h) w (1 + c) + d;
//   per 128 columns  s = max |y| / 448,  q = e4m3(y / s).
//
// The row stays in registers from x to the last store, so x and r are read once
// and h, y, q, s written once: the bytes are the floor.  W waves share a row; lane
// l of them owns the 8-element chunks l, l + 64 W, ..., so every load is 16 bytes a
// lane and the 16 lanes of one 128-column block are neighbours.  4608 x 4096 with
// gate, modulation and codes: 28.0 us, 4.7 TB/s; 1531 x 5000 normed on both sides:
// 16.5 us, bound by the start of a row and its three sums.  (Blocks that keep the
// parameters in fp32 for several rows, the next row on its way: 33 and 23 us, as fewer
// rows are under way at a time.)

#include "device_block.h"

namespace svdq {
namespace {

// Sum over a wave, in every lane: within rows of 16 lanes, then across them.
__device__ __forceinline__ float wave_sum(float v) {
  auto with = [&](auto ctrl) {
    v += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), decltype(ctrl)::value, 0xF, 0xF, true));
  };
  with(std::integral_constant<int, 0xB1>{});    // lanes 1, 0, 3, 2 of a quad
  with(std::integral_constant<int, 0x4E>{});    // 2, 3, 0, 1
  with(std::integral_constant<int, 0x141>{});   // half a row mirrored
  with(std::integral_constant<int, 0x140>{});   // a row mirrored
  const uint32_t u = __float_as_uint(v);
  return (__uint_as_float(__builtin_amdgcn_readlane(u, 0)) + __uint_as_float(__builtin_amdgcn_readlane(u, 16))) +
         (__uint_as_float(__builtin_amdgcn_readlane(u, 32)) + __uint_as_float(__builtin_amdgcn_readlane(u, 48)));
}

// MORE: y or its codes are asked for.
template <int DT, int NC, bool MORE>
__global__ __launch_bounds__(1024) void gated_kernel(svdq_gated_norm_args a, int W) {
  __shared__ __attribute__((aligned(16))) float part[2][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // W == 1: each wave has a row of its own; otherwise the block shares one
  const int row = W == 1 ? blockIdx.x * (blockDim.x >> 6) + wave : blockIdx.x;
  if (W == 1 && row >= a.M) return;
  const int first = W == 1 ? lane : (int)threadIdx.x;
  const int chunks = a.K >> 3, stride = 64 * W;
  const int blocks = (a.K + SVDQ_FP8_BLOCK - 1) / SVDQ_FP8_BLOCK;

  auto load = [&](const uint16_t* base, int64_t at, int c) __attribute__((always_inline)) -> b4i {
    const int k = first + c * stride;
    return base && k < chunks ? *reinterpret_cast<const b4i*>(base + at + 8 * (size_t)k) : (b4i){0, 0, 0, 0};
  };
  int e = 0;
  if (a.gate || a.scale || a.shift) e = a.entry ? min(max(a.entry[row], 0), a.E - 1) : row / (a.M / a.E);

  float v[NC][8];
  b4i rv[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const b4i x = load(a.x, row * a.x_row, c);
    rv[c] = load(a.residual, row * a.residual_row, c);
    widen8<DT>(x, v[c]);
  }
  b4i pv[NC], gv[NC], wv[NC], sv[NC], dv[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    pv[c] = load(a.post_weight, 0, c);
    gv[c] = load(a.gate, e * a.gate_row, c);
  }

  int turn = 0;   // the two halves of part[] in turn: one barrier a sum
  auto total = [&](float sum) __attribute__((always_inline)) -> float {   // over the row
    sum = wave_sum(sum);
    if (W > 1) {
      if (lane == 0) part[turn][wave] = sum;
      __syncthreads();
      sum = 0.f;
      for (int i = 0; i < W; ++i) sum += part[turn][i];
      turn ^= 1;
    }
    return sum;
  };
  // The norm of v as v inv + off.  Squares leave fp32 above
  // 2^64 and lose bits below 2^-63: such rows are scaled by a power of two (exactly) and
  // summed again.
  float inv, off;
  auto norm = [&](int kind) __attribute__((always_inline)) {
    inv = 1.f;
    off = 0.f;
    if (kind == SVDQ_NORM_NONE) return;
    float mean = 0.f;
    auto square = [&](float eps) __attribute__((always_inline)) -> float {   // mean square of v - mean, and eps
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float d = v[c][i] - mean;
          s = fmaf(d, d, s);
        }
        sum += first + c * stride < chunks ? s : 0.f;
      }
      return total(sum) / (float)a.K + eps;
    };
    auto centre = [&]() __attribute__((always_inline)) {
      if (kind != SVDQ_NORM_LAYER) return;
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += v[c][i];
      mean = total(sum) / (float)a.K;
    };
    centre();
    float var = square(a.eps);
    if (__builtin_expect(!(var >= 0x1p-80f && var < __builtin_inff()), 0)) {
      // the deviations themselves, as v
      float by = 0x1p90f;
      if (!(var < 1.f)) {
        by = 0x1p-90f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) v[c][i] *= by;
        centre();
      }
      const float up = by > 1.f ? by : 1.f;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] = first + c * stride < chunks ? (v[c][i] - mean) * up : 0.f;
      mean = 0.f;
      var = square(a.eps * by * by);
    }
    inv = 1.0f / sqrtf(var);
    off = -mean * inv;
  };

  norm(a.post);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    wv[c] = load(a.weight, 0, c);
    sv[c] = load(a.scale, e * a.scale_row, c);
    dv[c] = load(a.shift, e * a.shift_row, c);
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int k = first + c * stride;
    float t[8];
    if (a.post != SVDQ_NORM_NONE) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = fmaf(v[c][i], inv, off);
    }
    if (a.post_weight) {
      widen8<DT>(pv[c], t);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] *= t[i];
    }
    if (a.gate) {
      widen8<DT>(gv[c], t);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] *= t[i];
    }
    if (a.residual) {
      widen8<DT>(rv[c], t);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = fmaf(a.residual_scale, t[i], v[c][i]);
    }
    if (k >= chunks) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = 0.f;
    }
    if (a.h && k < chunks) {
      // The sum is read again after the next projections, y or its codes by what follows
      // at once: the sum goes past the caches and leaves them to those (4608 x 4096 with
      // codes 28.0 against 30.4 us, and the FP8 linear after it loses nothing: 41.0
      // against 43.1 together.  y or the codes past them too: 24.2 alone, 47.0 together.)
      b4i* to = reinterpret_cast<b4i*>(a.h + row * a.h_row + 8 * (size_t)k);
      if constexpr (MORE) __builtin_nontemporal_store(narrow8<DT>(v[c]), to);
      else *to = narrow8<DT>(v[c]);
    }
  }
  if constexpr (!MORE) return;
  norm(a.pre);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int k = first + c * stride;
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[c][i] = fmaf(v[c][i], inv, off);
    if (a.weight) {
      widen8<DT>(wv[c], t);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] *= t[i];
    }
    if (a.scale) {
      widen8<DT>(sv[c], t);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = fmaf(v[c][i], t[i], v[c][i]);
    }
    if (a.shift) {
      widen8<DT>(dv[c], t);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] += t[i];
    }
    if (a.y && k < chunks) *reinterpret_cast<b4i*>(a.y + row * a.y_row + 8 * (size_t)k) = narrow8<DT>(v[c]);
    if (!a.q) continue;
    // maximum of |y| as integers, so that a NaN is the largest of all
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[c][i]) & 0x7FFFFFFFu);
    if (k >= chunks) top = 0;
    auto with = [&](auto ctrl) {
      top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, top, decltype(ctrl)::value, 0xF, 0xF, true));
    };
    with(std::integral_constant<int, 0xB1>{});
    with(std::integral_constant<int, 0x4E>{});
    with(std::integral_constant<int, 0x141>{});
    with(std::integral_constant<int, 0x140>{});
    float sc = __uint_as_float(top) / 448.0f;
    if (sc < 1.17549435e-38f) sc = 0.f;
    const float by = sc > 0.f ? 1.0f / sc : 0.f;
    if (k < chunks) {
      int lo = 0, hi = 0;
      lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[c][0] * by, v[c][1] * by, lo, false);
      lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[c][2] * by, v[c][3] * by, lo, true);
      hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[c][4] * by, v[c][5] * by, hi, false);
      hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[c][6] * by, v[c][7] * by, hi, true);
      *reinterpret_cast<int2*>(a.q + (size_t)row * a.K + 8 * (size_t)k) = make_int2(lo, hi);
      if ((k & 15) == 0) a.s[(size_t)row * blocks + (k >> 4)] = sc;
    }
  }
}

template <int DT>
svdq_status launch_gated(const svdq_gated_norm_args& a, hipStream_t st) {
  const int chunks = a.K / 8;
  // Chunks of a lane: one where rows are few, so that a row's loads are one round
  // trip, otherwise two (4608 x 4096 30.3 us against 30.7 with one and 33.7 with four;
  // 1531 x 5000 16.9 against 18.8 and 17.9).
  const int per = a.M <= 512 ? 1 : 2;
  int W = (chunks + 64 * per - 1) / (64 * per);
  if (W > 16) W = 16;
  const int nc = (chunks + 64 * W - 1) / (64 * W);
  const dim3 block(W == 1 ? 256 : 64 * W), grid(W == 1 ? (a.M + 3) / 4 : a.M);
  auto go = [&](auto n, auto more) {
    hipLaunchKernelGGL((gated_kernel<DT, decltype(n)::value, decltype(more)::value>), grid, block, 0, st, a, W);
  };
  auto rows = [&](auto n) {
    if (a.y || a.q) go(n, std::true_type{});
    else go(n, std::false_type{});
  };
  if (nc <= 1) rows(std::integral_constant<int, 1>{});
  else rows(std::integral_constant<int, 2>{});   // 16 waves of two hold 16384 columns
  return launched();
}

svdq_status check(const svdq_gated_norm_args* a) {
  if (!a || !a->x || (!a->h && !a->y && !a->q) || (a->q == nullptr) != (a->s == nullptr)) return SVDQ_ERR_ARG;
  const float big = 3.0e38f;
  if (!(a->eps >= 0.f && a->eps <= big) || !(a->residual_scale >= -big && a->residual_scale <= big)) return SVDQ_ERR_ARG;
  if (!is_dtype(a->dtype) || a->post < SVDQ_NORM_NONE || a->post > SVDQ_NORM_LAYER || a->pre < SVDQ_NORM_NONE ||
      a->pre > SVDQ_NORM_LAYER)
    return SVDQ_ERR_UNSUPPORTED;
  if (a->M < 1 || a->M > (1 << 20) || a->K < 8 || a->K > 16384 || a->K % 8 != 0 || a->E < 1 || a->E > (1 << 20))
    return SVDQ_ERR_SHAPE;
  const bool rows = a->gate || a->scale || a->shift;
  if (rows && !a->entry && a->M % a->E != 0) return SVDQ_ERR_SHAPE;
  const struct { const void* p; int64_t row; int32_t n; } t[] = {
      {a->x, a->x_row, a->M}, {a->residual, a->residual_row, a->M}, {a->gate, a->gate_row, a->E},
      {a->scale, a->scale_row, a->E}, {a->shift, a->shift_row, a->E}, {a->h, a->h_row, a->M}, {a->y, a->y_row, a->M}};
  for (const auto& x : t)
    if (x.p && x.n > 1 && x.row < a->K) return SVDQ_ERR_SHAPE;
  for (const auto& x : t)
    if ((x.p && x.n > 1 && x.row % 8 != 0) || !on16(x.p)) return SVDQ_ERR_ALIGN;
  if (!on16(a->post_weight) || !on16(a->weight) || !on16(a->q) || !on4(a->s) || !on4(a->entry)) return SVDQ_ERR_ALIGN;
  // in place, element for element: with another stride rows would be written that
  // are still to be read
  auto in_place = [&](const uint16_t* o, int64_t row) {
    return o && a->M > 1 && ((o == a->x && row != a->x_row) || (o == a->residual && row != a->residual_row));
  };
  if (in_place(a->h, a->h_row) || in_place(a->y, a->y_row) || (a->h && a->h == a->y)) return SVDQ_ERR_ARG;
  return SVDQ_OK;
}

}  // namespace
}  // namespace svdq

using namespace svdq;

extern "C" svdq_status svdq_gated_norm(const svdq_gated_norm_args* args, void* stream) {
  svdq_status ok = check(args);
  if (ok != SVDQ_OK || (ok = device_ok()) != SVDQ_OK) return ok;
  svdq_gated_norm_args a = *args;
  // the row of a single row addresses nothing
  if (a.M == 1) a.x_row = a.residual_row = a.h_row = a.y_row = 0;
  if (a.E == 1) a.gate_row = a.scale_row = a.shift_row = 0;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return a.dtype == SVDQ_BF16 ? launch_gated<SVDQ_BF16>(a, st) : launch_gated<SVDQ_FP16>(a, st);
}
