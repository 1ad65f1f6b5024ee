// FP8 linear with fp32 scales per block of 128:
//   Y[m, n] = sum_b xs[m, b] ws[n / 128, b] (sum_{k in b} xq[m, k] wq[n, k]) + bias[n].
//
// MFMAs form the block sums of 16 out-features x 16 tokens (A = weight rows,
// B = token rows, from a zero accumulator); lane l then holds
// out-features 4 (l / 16) + i of token l % 16, so the scale product is one
// value per lane and step and the update one fma per output.

#include "device_block.h"

namespace svdq {
namespace {

template <int DT>
__device__ __forceinline__ void store4(uint16_t* y, const b4f& v) {
  *reinterpret_cast<uint2*>(y) = make_uint2(narrow2<DT>(v[0], v[1]), narrow2<DT>(v[2], v[3]));
}

// The FP8 products of the matrix unit are added in groups of 8 with only 13
// bits kept below the group's largest (measured: beside 2^16, 2^3 survives
// and 2^2 does not); bf16 operands keep fp32 sums, and every E4M3 value is a
// bf16 value.  So the codes are widened, two at a time, and the product of
// 128 is four bf16 MFMAs.  Lane group g supplies bytes 32 g .. + 32 of both
// operands' rows; MFMA s takes bytes 8 s .. + 8 of them.
__device__ __forceinline__ b8bf widen_codes(int lo, int hi) {
  const b2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const b2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const b2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const b2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return (b8bf){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ b4f dot128(const b8i& a, const b8i& b) {
  b4f p = (b4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < 4; ++s)
    p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_codes(a[2 * s], a[2 * s + 1]), widen_codes(b[2 * s], b[2 * s + 1]),
                                                p, 0, 0, 0);
  return p;
}

__device__ __forceinline__ b8i load32(const uint8_t* p) {
  const b4i a = *reinterpret_cast<const b4i*>(p), b = *reinterpret_cast<const b4i*>(p + 16);
  return (b8i){a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

template <int DT>
__global__ __launch_bounds__(256) void fp8_simple_kernel(const uint8_t* __restrict__ xq, const float* __restrict__ xs,
                                                         const uint8_t* __restrict__ wq, const float* __restrict__ ws,
                                                         const uint16_t* __restrict__ bias, int M, int K, int N,
                                                         uint16_t* __restrict__ Y) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, g = lane >> 4;
  const int n0 = (blockIdx.x * 4 + wave) * 16, m0 = blockIdx.y * 16;
  if (n0 >= N) return;
  const int m = min(m0 + l16, M - 1), kb = K / 128;
  const uint8_t* ap = wq + (size_t)(n0 + l16) * K + 32 * g;
  const uint8_t* bp = xq + (size_t)m * K + 32 * g;
  const float* sx = xs + (size_t)m * kb;
  const float* sw = ws + (size_t)(n0 >> 7) * kb;
  b4f acc = (b4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int t = 0; t < kb; ++t) {
    const b4f p = dot128(load32(ap + 128 * (size_t)t), load32(bp + 128 * (size_t)t));
    const float s = sx[t] * sw[t];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(p[i], s, acc[i]);
  }
  if (m0 + l16 >= M) return;
  const int n = n0 + 4 * g;
  if (bias) {
    const uint2 raw = *reinterpret_cast<const uint2*>(bias + n);
    const b2f b0 = widen2<DT>(raw.x), b1 = widen2<DT>(raw.y);
    acc += (b4f){b0[0], b0[1], b1[0], b1[1]};
  }
  store4<DT>(Y + (size_t)m * N + n, acc);
}

template <int DT>
svdq_status launch_fp8(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws, const uint16_t* bias,
                       int M, int K, int N, uint16_t* Y, hipStream_t st) {
  hipLaunchKernelGGL((fp8_simple_kernel<DT>), dim3((N / 16 + 3) / 4, (M + 15) / 16), dim3(256), 0, st, xq, xs, wq, ws,
                     bias, M, K, N, Y);
  return launched();
}

}  // namespace
}  // namespace svdq

using namespace svdq;

extern "C" svdq_status svdq_fp8_linear(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                                       const uint16_t* bias, int32_t M, int32_t K, int32_t N, int32_t dtype,
                                       uint16_t* Y, void* stream) {
  if (!xq || !xs || !wq || !ws || !Y) return SVDQ_ERR_ARG;
  if (!is_dtype(dtype)) return SVDQ_ERR_UNSUPPORTED;
  if (!valid_kn(K, N) || M < 1 || M > (1 << 20)) return SVDQ_ERR_SHAPE;
  if ((int64_t)M * K > (int64_t)1 << 32 || (int64_t)N * K > (int64_t)1 << 32) return SVDQ_ERR_SHAPE;
  if (!on16(xq) || !on16(wq) || !on16(bias) || !on16(Y) || !on4(xs) || !on4(ws)) return SVDQ_ERR_ALIGN;
  const svdq_status ok = device_ok();
  if (ok != SVDQ_OK) return ok;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return dtype == SVDQ_BF16 ? launch_fp8<SVDQ_BF16>(xq, xs, wq, ws, bias, M, K, N, Y, st)
                            : launch_fp8<SVDQ_FP16>(xq, xs, wq, ws, bias, M, K, N, Y, st);
}
