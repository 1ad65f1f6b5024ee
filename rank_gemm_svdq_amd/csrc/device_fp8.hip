// FP8 linear with fp32 scales per block of 128:
//   Y[m, n] = sum_b xs[m, b] ws[n / 128, b] (sum_{k in b} xq[m, k] wq[n, k]) + bias[n].
//
// Products.  The FP8 products of the matrix unit are added in groups of 8 with
// only 13 bits kept below the group's largest (measured: beside 2^16, 2^3
// survives and 2^2 does not; all FP8 forms alike); bf16 operands keep fp32
// sums, and every E4M3 value is a bf16 value.  So codes travel through memory
// and LDS as 8 bits and are widened, two at a time, on their way to bf16
// MFMAs: twice the matrix time of the FP8 forms, for sums that hold 24 bits.
//
// Tiles.  16x16x32 MFMAs, A = weight rows, B = token rows: lane l holds
// out-features 4 (l / 16) + i of token l % 16, so the scale of a block sum is
// one value per lane and the update one fma per output.  A row's 128 codes of
// a step are 8 chunks of 16 bytes; lane group g = l / 16 supplies chunks g and
// g + 4 of both operands' rows (the order of k inside a block is free as long
// as both agree), 8 codes per MFMA.  Weight rows are permuted inside pairs of
// 16-row tiles, row q of tile 2 p + h being out-feature 32 p + 8 (q / 4) +
// 4 h + q % 4, so that the pair's 4 + 4 outputs of a lane are 8 consecutive
// out-features: 16-byte stores.

#include "device_block.h"

namespace svdq {
namespace {

__device__ __forceinline__ b8bf widen_codes(int lo, int hi) {
  const b2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const b2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const b2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const b2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return (b8bf){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// out-feature (within the wave's) of MFMA row q of weight tile nt
__device__ __forceinline__ int feature_row(int nt, int q) {
  return 32 * (nt >> 1) + 8 * (q >> 2) + 4 * (nt & 1) + (q & 3);
}

template <int DT>
__device__ __forceinline__ void add_bias8(const uint16_t* bias, int n, float* v) {
  if (bias == nullptr) return;
  float t[8];
  widen8<DT>(*reinterpret_cast<const b4i*>(bias + n), t);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] += t[i];
}

// ---------------------------------------------------------- large tiles
//
// A block computes BM tokens x BN out-features; its waves (WM x WN) own MT x
// NT MFMA tiles each.  Steps of 128 k of both operands go to LDS by direct
// copies (1 KB: 8 rows x 128 codes), one step ahead, two buffers, one barrier
// a step.  Chunk c of a row sits at slot c ^ f(row) with f such that the 16
// lanes served together in a fragment read hit distinct 16-byte slots.

template <int NT, int MT, int WN, int WM>
struct LargeTile {
  static constexpr int WAVES = WN * WM, BN = 16 * NT * WN, BM = 16 * MT * WM;
  static constexpr int STEP = (BN + BM) * 128;
};

template <int DT, int NT, int MT, int WN, int WM>
__global__ __launch_bounds__(64 * WN * WM, 2) void fp8_large_kernel(
    const uint8_t* __restrict__ xq, const float* __restrict__ xs, const uint8_t* __restrict__ wq,
    const float* __restrict__ ws, const uint16_t* __restrict__ bias, int M, int K, int N, uint16_t* __restrict__ Y,
    int tiles_m, int tiles_n) {
  using T = LargeTile<NT, MT, WN, WM>;
  constexpr int UNITS = (T::BN + T::BM) / 8 / T::WAVES;   // copies per wave and step
  static_assert((T::BN / 8) % UNITS == 0, "a wave copies rows of one operand");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * T::STEP];
  __shared__ float sxl[2][T::BM];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int l16 = lane & 15, g = lane >> 4;
  // work ids run through groups of 8 token tiles, out-feature tile slower: the
  // blocks that an XCD holds at a time share their operand panels in its L2
  const int id = xcd_order(blockIdx.x, tiles_m * tiles_n);
  const int span = 8 * tiles_n, grp = id / span, in = id % span;
  const int high = min(8, tiles_m - 8 * grp);
  const int m0 = (8 * grp + in % high) * T::BM, n0 = (in / high) * T::BN;
  const int steps = K >> 7;

  // ---- copies: units of 8 rows, weights first.  N % 16 == 0, so a unit of
  // weight rows is whole or past the end (then the last one is repeated);
  // token rows past M repeat the last row, lane by lane.
  const int u0 = wave * UNITS;
  const bool wside = u0 < T::BN / 8;
  const int r8 = lane >> 3, slot = lane & 7;
  // weights: slot ^ (2 (u % 4) + r8 bit 1); tokens: slot ^ (4 (u % 2) + r8 / 2)
  const int f0 = wside ? (r8 >> 1) & 1 : r8 >> 1;
  const uint32_t voff = (uint32_t)r8 * (uint32_t)K + 16u * (slot ^ f0);
  const int edge = wside ? 7 : max(min(7, M - 1 - m0 - ((M - 1 - m0) & ~7)), 0);   // last row of the last unit
  const uint32_t voff_edge = (uint32_t)min(r8, edge) * (uint32_t)K + 16u * (slot ^ f0);
  const int last_unit = wside ? (N - n0) / 8 - 1 : (M - 1 - m0) >> 3;
  const uint8_t* base = wside ? wq + (size_t)n0 * K : xq + (size_t)m0 * K;
  const uint32_t lds0 = lds_address(lds);
  auto copy = [&](int t) __attribute__((always_inline)) {
    const uint8_t* src = base + (size_t)t * 128;
    const uint32_t dst = lds0 + (t & 1) * T::STEP + u0 * 1024;
#pragma unroll
    for (int j = 0; j < UNITS; ++j) {
      const int u = wside ? u0 + j : u0 + j - T::BN / 8;
      const int at = min(u, last_unit);
      const uint32_t x = wside ? 32u * (u & 3) : 64u * (u & 1);
      dma_16(src + (size_t)at * 8 * K, (at == last_unit ? voff_edge : voff) ^ x, dst + 1024 * j);
    }
  };

  // ---- fragment addresses: chunk g (and, 4 chunks on, g + 4) of the row
  int aoff[NT], boff[2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = 16 * NT * wn + feature_row(nt, l16);
    aoff[nt] = r * 128 + 16 * (g ^ (2 * ((r >> 3) & 3) + ((r >> 1) & 1)));
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = 16 * MT * wm + l16 + 16 * h;
    boff[h] = T::BN * 128 + r * 128 + 16 * (g ^ ((r >> 1) & 7));
  }

  b4f acc[NT][MT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[nt][mt] = (b4f){0.f, 0.f, 0.f, 0.f};

  // token scales of a step, one per thread, two steps ahead
  const float* sxp = xs + (size_t)min(m0 + tid, M - 1) * steps;
  const float* swp = ws + (size_t)((n0 + 16 * NT * wn) >> 7 < (N + 127) >> 7 ? (n0 + 16 * NT * wn) >> 7 : 0) * steps;
  copy(0);
  float sx_next = 0.f;
  if (tid < T::BM) {
    sxl[0][tid] = sxp[0];
    sx_next = sxp[min(1, steps - 1)];
  }
  for (int t = 0; t < steps; ++t) {
    dma_wait();
    __syncthreads();
    if (t + 1 < steps) copy(t + 1);
    if (tid < T::BM) {
      sxl[(t + 1) & 1][tid] = sx_next;
      sx_next = sxp[min(t + 2, steps - 1)];
    }
    const float sw = swp[t];
    const uint8_t* buf = lds + (t & 1) * T::STEP;
    b8bf a[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const b4i lo = *reinterpret_cast<const b4i*>(buf + aoff[nt]);
      const b4i hi = *reinterpret_cast<const b4i*>(buf + (aoff[nt] ^ 64));
      a[nt][0] = widen_codes(lo[0], lo[1]);
      a[nt][1] = widen_codes(lo[2], lo[3]);
      a[nt][2] = widen_codes(hi[0], hi[1]);
      a[nt][3] = widen_codes(hi[2], hi[3]);
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const b4i lo = *reinterpret_cast<const b4i*>(buf + boff[mt & 1] + (mt >> 1) * 32 * 128);
      const b4i hi = *reinterpret_cast<const b4i*>(buf + (boff[mt & 1] ^ 64) + (mt >> 1) * 32 * 128);
      const float s = sxl[t & 1][16 * MT * wm + 16 * mt + l16] * sw;
      b4f p[NT];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const b8bf b = x < 2 ? widen_codes(lo[2 * (x & 1)], lo[2 * (x & 1) + 1]) : widen_codes(hi[2 * (x & 1)], hi[2 * (x & 1) + 1]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          p[nt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[nt][x], b, x ? p[nt] : (b4f){0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][mt][i] = fmaf(p[nt][i], s, acc[nt][mt][i]);
    }
  }
#pragma unroll
  for (int p2 = 0; p2 < NT / 2; ++p2) {
    const int n = n0 + 16 * NT * wn + 32 * p2 + 8 * g;
    if (n >= N) continue;
    float bv[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) bv[i] = 0.f;
    add_bias8<DT>(bias, n, bv);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int m = m0 + 16 * MT * wm + 16 * mt + l16;
      if (m >= M) continue;
      float v[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = acc[2 * p2][mt][i] + bv[i];
        v[4 + i] = acc[2 * p2 + 1][mt][i] + bv[4 + i];
      }
      *reinterpret_cast<b4i*>(Y + (size_t)m * N + n) = narrow8<DT>(v);
    }
  }
}

// ------------------------------------------------------------ few tokens
//
// The weights are read once for at most 16 MT tokens of a block, so their
// bytes bound it.  A block owns 16 out-features, its waves take steps of 128 k
// in turn straight from memory (a row's step is one whole line) and are
// joined in LDS.

template <int DT, int MT>
__global__ __launch_bounds__(512) void fp8_few_kernel(const uint8_t* __restrict__ xq, const float* __restrict__ xs,
                                                      const uint8_t* __restrict__ wq, const float* __restrict__ ws,
                                                      const uint16_t* __restrict__ bias, int M, int K, int N,
                                                      uint16_t* __restrict__ Y) {
  constexpr int WV = 8;
  __shared__ float red[WV][MT][16][17];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16 * MT, steps = K >> 7;
  const uint8_t* ap = wq + (size_t)(n0 + l16) * K + 16 * g;
  const uint8_t* bp[MT];
  const float* sx[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int m = min(m0 + 16 * mt + l16, M - 1);
    bp[mt] = xq + (size_t)m * K + 16 * g;
    sx[mt] = xs + (size_t)m * steps;
  }
  const float* sw = ws + (size_t)(n0 >> 7) * steps;
  b4f acc[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) acc[mt] = (b4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int t = wave; t < steps; t += WV) {
    const b4i alo = *reinterpret_cast<const b4i*>(ap + 128 * (size_t)t);
    const b4i ahi = *reinterpret_cast<const b4i*>(ap + 128 * (size_t)t + 64);
    const float w = sw[t];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const b4i blo = *reinterpret_cast<const b4i*>(bp[mt] + 128 * (size_t)t);
      const b4i bhi = *reinterpret_cast<const b4i*>(bp[mt] + 128 * (size_t)t + 64);
      b4f p = (b4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_codes(alo[2 * x], alo[2 * x + 1]), widen_codes(blo[2 * x], blo[2 * x + 1]), p, 0, 0, 0);
        p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_codes(ahi[2 * x], ahi[2 * x + 1]), widen_codes(bhi[2 * x], bhi[2 * x + 1]), p, 0, 0, 0);
      }
      const float s = sx[mt][t] * w;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[mt][i] = fmaf(p[i], s, acc[mt][i]);
    }
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][mt][l16][4 * g + i] = acc[mt][i];
  __syncthreads();
  for (int o = threadIdx.x; o < MT * 256; o += 512) {
    const int mt = o >> 8, r = (o >> 4) & 15, c = o & 15, m = m0 + 16 * mt + r;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < WV; ++w) v += red[w][mt][r][c];
    if (m < M) {
      if (bias) v += widen2<DT>(bias[n0 + c])[0];
      Y[(size_t)m * N + n0 + c] = (uint16_t)narrow2<DT>(v, 0.f);
    }
  }
}

template <int DT>
svdq_status launch_fp8(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws, const uint16_t* bias,
                       int M, int K, int N, uint16_t* Y, hipStream_t st) {
  auto large = [&](auto nt, auto mt, auto wn, auto wm) {
    using T = LargeTile<decltype(nt)::value, decltype(mt)::value, decltype(wn)::value, decltype(wm)::value>;
    const int tm = (M + T::BM - 1) / T::BM, tn = (N + T::BN - 1) / T::BN;
    hipLaunchKernelGGL((fp8_large_kernel<DT, decltype(nt)::value, decltype(mt)::value, decltype(wn)::value, decltype(wm)::value>),
                       dim3(tm * tn), dim3(64 * T::WAVES), 0, st, xq, xs, wq, ws, bias, M, K, N, Y, tm, tn);
  };
  using std::integral_constant;
  typedef integral_constant<int, 2> I2;
  typedef integral_constant<int, 4> I4;
  typedef integral_constant<int, 8> I8;
  const int64_t t256 = (int64_t)((M + 255) / 256) * ((N + 255) / 256);
  const int64_t t128 = (int64_t)((M + 127) / 128) * ((N + 127) / 128);
  if (M <= 64) {
    if (M <= 16) hipLaunchKernelGGL((fp8_few_kernel<DT, 1>), dim3(N / 16, 1), dim3(512), 0, st, xq, xs, wq, ws, bias, M, K, N, Y);
    else hipLaunchKernelGGL((fp8_few_kernel<DT, 2>), dim3(N / 16, (M + 31) / 32), dim3(512), 0, st, xq, xs, wq, ws, bias, M, K, N, Y);
  } else if (t256 >= 256) {
    large(I4{}, I8{}, I4{}, I2{});
  } else if (t128 >= 200) {
    large(I4{}, I4{}, I2{}, I2{});
  } else {
    large(I2{}, I2{}, I2{}, I2{});
  }
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
