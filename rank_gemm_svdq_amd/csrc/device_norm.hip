// Residual sum, root-mean-square norm and FP8 codes in one pass.
//
//   h = x + r;  y = h / sqrt(mean h^2 + eps) * w;
//   per 128 columns  s = max |y| / 448,  q = e4m3(y / s).
//
// The row stays in registers between the sum of squares and the codes, so x
// and r are read once and h, q and s written once: the bytes are the floor
// (7 per element with a residual).  W waves share a row; lane l of them owns
// the 8-element chunks l, l + 64 W, ... so every load is 16 bytes a lane, and
// the 16 lanes of one 128-column block are neighbours: its maximum is four
// lane exchanges.  4096 x 3072 with a residual: 17 - 18 us, 4.9 - 5.2 TB/s, the
// rate of a large copy; 8192 x 12288: 125 us, 5.6 TB/s.

#include "device_block.h"

namespace svdq {
namespace {

// h may lie where x or res does (a lane reads its chunks of both before it stores
// any), so neither is restrict.
template <int DT, int NC>
__global__ __launch_bounds__(1024) void norm_kernel(const uint16_t* x, int64_t xst, const uint16_t* res, int64_t rst,
                                                    const uint16_t* __restrict__ wt, float eps, int M, int K,
                                                    uint16_t* h, int64_t hst, uint8_t* __restrict__ q,
                                                    float* __restrict__ s, int W) {
  __shared__ float part[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // W == 1: each wave has a row of its own; otherwise the block shares one
  const int row = W == 1 ? blockIdx.x * (blockDim.x >> 6) + wave : blockIdx.x;
  if (W == 1 && row >= M) return;
  const int first = W == 1 ? lane : (int)threadIdx.x;
  const int chunks = K >> 3, stride = 64 * W;
  const uint16_t* xr = x + (size_t)row * xst;
  const uint16_t* rr = res ? res + (size_t)row * rst : nullptr;

  float v[NC][8];
  b4i xv[NC], rv[NC], wv[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int k = first + c * stride;
    xv[c] = rv[c] = (b4i){0, 0, 0, 0};
    if (k < chunks) {
      xv[c] = *reinterpret_cast<const b4i*>(xr + 8 * (size_t)k);
      if (rr) rv[c] = *reinterpret_cast<const b4i*>(rr + 8 * (size_t)k);
    }
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int k = first + c * stride;
    wv[c] = k < chunks ? *reinterpret_cast<const b4i*>(wt + 8 * (size_t)k) : (b4i){0, 0, 0, 0};
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    widen8<DT>(xv[c], v[c]);
    if (rr) {
      float t[8];
      widen8<DT>(rv[c], t);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] += t[i];
    }
    const int k = first + c * stride;
    if (h && k < chunks) *reinterpret_cast<b4i*>(h + (size_t)row * hst + 8 * (size_t)k) = narrow8<DT>(v[c]);
  }
  auto squares = [&]() {   // of the row
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(v[c][i], v[c][i], sum);
#pragma unroll
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
    if (W > 1) {
      if (lane == 0) part[wave] = sum;
      __syncthreads();
      sum = 0.f;
      for (int i = 0; i < W; ++i) sum += part[i];
    }
    return sum;
  };
  float mean = squares() / (float)K + eps;
  // The squares of bf16 values leave fp32 above 2^64 and below 2^-63.  Such rows,
  // whole or with a mean that small, are scaled by 2^-90 or 2^90 (exactly; their
  // squares are in range then) and summed again: y does not change with h's scale.
  if (DT == SVDQ_BF16 && !(mean >= 0x1p-80f && mean < __builtin_inff())) {
    const float by = mean < 1.f ? 0x1p90f : 0x1p-90f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] *= by;
    if (W > 1) __syncthreads();
    mean = squares() / (float)K + eps * by * by;
  }
  const float inv = 1.0f / sqrtf(mean);
  const int blocks = (K + SVDQ_FP8_BLOCK - 1) / SVDQ_FP8_BLOCK;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int k = first + c * stride;
    float t[8];
    widen8<DT>(wv[c], t);
    // maximum of |y| as integers, so that a NaN is the largest of all
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[c][i] = v[c][i] * inv * t[i];
      top = max(top, __float_as_uint(v[c][i]) & 0x7FFFFFFFu);
    }
    if (k >= chunks) top = 0;
#pragma unroll
    for (int d = 8; d; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    float sc = __uint_as_float(top) / 448.0f;
    if (sc < 1.17549435e-38f) sc = 0.f;
    const float by = sc > 0.f ? 1.0f / sc : 0.f;
    if (k < chunks) {
      int lo = 0, hi = 0;
      lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[c][0] * by, v[c][1] * by, lo, false);
      lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[c][2] * by, v[c][3] * by, lo, true);
      hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[c][4] * by, v[c][5] * by, hi, false);
      hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[c][6] * by, v[c][7] * by, hi, true);
      *reinterpret_cast<int2*>(q + (size_t)row * K + 8 * (size_t)k) = make_int2(lo, hi);
      if ((k & 15) == 0) s[(size_t)row * blocks + (k >> 4)] = sc;
    }
  }
}

template <int DT>
svdq_status launch_norm(const uint16_t* x, int64_t xst, const uint16_t* res, int64_t rst, const uint16_t* w, float eps,
                        int M, int K, uint16_t* h, int64_t hst, uint8_t* q, float* s, hipStream_t st) {
  const int chunks = K / 8;
  // Chunks of a lane.  Few rows: one, so that a row's loads are one round trip
  // (3072 columns: 1 row 3.0 us against 4.0 us with up to four chunks, 256
  // rows 3.6 against 4.6).  Many rows fill the chip by themselves and fewer,
  // fuller waves are better (4096 rows 18.1 us against 20.2 us).
  const int per = M <= 512 ? 1 : 4;
  int W = 1;
  while (W < 16 && 64 * W * per < chunks) W *= 2;
  const int nc = (chunks + 64 * W - 1) / (64 * W);
  const dim3 block(W == 1 ? 256 : 64 * W), grid(W == 1 ? (M + 3) / 4 : M);
  auto go = [&](auto n) {
    hipLaunchKernelGGL((norm_kernel<DT, decltype(n)::value>), grid, block, 0, st, x, xst, res, rst, w, eps, M, K, h,
                       hst, q, s, W);
  };
  if (nc <= 1) go(std::integral_constant<int, 1>{});
  else if (nc <= 2) go(std::integral_constant<int, 2>{});
  else if (nc <= 4) go(std::integral_constant<int, 4>{});
  else go(std::integral_constant<int, 8>{});
  return launched();
}

}  // namespace
}  // namespace svdq

using namespace svdq;

extern "C" svdq_status svdq_add_rmsnorm_quantize(const uint16_t* x, int64_t x_stride, const uint16_t* residual,
                                                 int64_t residual_stride, const uint16_t* weight, float eps,
                                                 int32_t M, int32_t K, int32_t dtype, uint16_t* h, int64_t h_stride,
                                                 uint8_t* q, float* s, void* stream) {
  if (!x || !weight || !q || !s || !(eps >= 0.f) || eps > 3.0e38f) return SVDQ_ERR_ARG;
  if (!is_dtype(dtype)) return SVDQ_ERR_UNSUPPORTED;
  if (M < 1 || M > (1 << 20) || K < 8 || K > 65536 || K % 8 != 0) return SVDQ_ERR_SHAPE;
  if (x_stride < K || (residual && residual_stride < K) || (h && h_stride < K)) return SVDQ_ERR_SHAPE;
  if (x_stride % 8 != 0 || (residual && residual_stride % 8 != 0) || (h && h_stride % 8 != 0)) return SVDQ_ERR_ALIGN;
  if (!on16(x) || !on16(residual) || !on16(weight) || !on16(h) || !on16(q) || !on4(s)) return SVDQ_ERR_ALIGN;
  // in place, element for element: with another stride rows would be written that
  // are still to be read
  if (h && M > 1 && ((h == x && h_stride != x_stride) || (h == residual && h_stride != residual_stride)))
    return SVDQ_ERR_ARG;
  const svdq_status ok = device_ok();
  if (ok != SVDQ_OK) return ok;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return dtype == SVDQ_BF16
             ? launch_norm<SVDQ_BF16>(x, x_stride, residual, residual_stride, weight, eps, M, K, h, h_stride, q, s, st)
             : launch_norm<SVDQ_FP16>(x, x_stride, residual, residual_stride, weight, eps, M, K, h, h_stride, q, s, st);
}
