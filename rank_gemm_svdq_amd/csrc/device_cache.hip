// Writing keys and values into a paged cache, in 8 bits or as they are, and
// reading them back.
//
// Keys lie token by token, [page][head][place][D], and values element by element,
// [page][head][D][place], so that attention's matrix operands are 16-byte loads of
// either (device_paged.hip).  Values therefore turn on their way through LDS: a
// block takes a run of tokens of one head, and rows of it that lie side by side in a
// page are stored four tokens at a time, others one by one.
//
// Codes.  INT8: s = max (1 / 127), the code nearest to x / s.  The first guess
// rint(x / s) by a reciprocal is off by at most one, and x - code s, which one fma
// gives exactly, tells.  FP8: s is a power of two, so x / s is exact and the
// conversion's rounding is the only one.

#include "device_kv.h"

namespace svdq {
namespace {

// Sizes of a cache's elements and lanes: LPR lanes (8 elements each) hold a token's
// vector; a dword of a row in LDS holds QD elements.
template <int FMT, int LPR>
struct CacheShape {
  static constexpr int ES = FMT == SVDQ_KV_VALUES ? 2 : 1;
  static constexpr int QD = 4 / ES;
  static constexpr int ROW = LPR * 8 * ES / 4 + 1;   // dwords of a row, and one for the banks
};

// 4 x 4 bytes turned: out[i] = byte i of r[0], r[1], r[2], r[3]
__device__ __forceinline__ void turn4(const uint32_t (&r)[4], uint32_t (&out)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(r[1], r[0], 0x05010400), b = __builtin_amdgcn_perm(r[3], r[2], 0x05010400);
  const uint32_t c = __builtin_amdgcn_perm(r[1], r[0], 0x07030602), d = __builtin_amdgcn_perm(r[3], r[2], 0x07030602);
  out[0] = __builtin_amdgcn_perm(b, a, 0x05040100);
  out[1] = __builtin_amdgcn_perm(b, a, 0x07060302);
  out[2] = __builtin_amdgcn_perm(d, c, 0x05040100);
  out[3] = __builtin_amdgcn_perm(d, c, 0x07060302);
}

// Codes of 8 elements of a vector whose elements LPR lanes hold, and its scale.
template <int FMT, int DT, int LPR>
__device__ __forceinline__ uint2 encode(const b4i& w, float* scale) {
  float x[8];
  widen8<DT>(w, x);
  uint32_t top = 0;   // as integers, so that infinities and NaN are the largest
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int d = LPR / 2; d; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
  if (top >= 0x7F800000u) {
    *scale = __uint_as_float(0x7FC00000u);
    return make_uint2(0, 0);
  }
  const float most = __uint_as_float(top);
  if constexpr (FMT == SVDQ_KV_FP8) {
    // the power of two at or above max / 448
    const uint32_t t = __float_as_uint(most / 448.0f);
    const uint32_t e = max((t >> 23) + ((t & 0x7FFFFFu) != 0), 1u);
    *scale = top ? __uint_as_float(e << 23) : 0.f;
    const float by = __uint_as_float((254u - e) << 23);
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * by, x[1] * by, lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2] * by, x[3] * by, lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4] * by, x[5] * by, hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6] * by, x[7] * by, hi, true);
    return make_uint2((uint32_t)lo, (uint32_t)hi);
  } else {
    float s = most * (1.0f / 127.0f);
    if (s < 0x1p-126f) s = 0.f;
    *scale = s;
    const float by = s > 0.f ? 1.0f / s : 0.f;
    uint32_t out[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float c = rintf(x[i] * by);
      const float left = fmaf(-c, s, x[i]), twice = fabsf(left + left);
      // past the middle, or on it with an odd code: one further
      const bool odd = ((int)c & 1) != 0;
      if (s > 0.f && (twice > s || (twice == s && odd))) c += left < 0.f ? -1.f : 1.f;
      out[i / 4] |= ((uint32_t)(int)c & 0xFFu) << (8 * (i % 4));
    }
    return make_uint2(out[0], out[1]);
  }
}

// 8 elements of a vector from their codes
template <int FMT, int DT>
__device__ __forceinline__ b4i decode(const uint2& w, float s) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t c = i < 4 ? w.x : w.y;
    if constexpr (FMT == SVDQ_KV_INT8) x[i] = (float)(int8_t)(c >> (8 * (i % 4)));
  }
  if constexpr (FMT == SVDQ_KV_FP8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = (int)(i < 2 ? w.x : w.y);
      const b2f t = i % 2 ? __builtin_amdgcn_cvt_pk_f32_fp8(c, true) : __builtin_amdgcn_cvt_pk_f32_fp8(c, false);
      x[2 * i] = t[0];
      x[2 * i + 1] = t[1];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] *= s;
  return narrow8<DT>(x);
}

// A block: TOK tokens of one head, keys and values.
template <int FMT, int DT, int LPR, int TOK>
__global__ __launch_bounds__(256) void write_kernel(svdq_kv_cache c, svdq_cache_write_args a, int shift) {
  using S = CacheShape<FMT, LPR>;
  constexpr int ES = S::ES, QD = S::QD, ROW = S::ROW;
  constexpr int AT = 256 / LPR;                        // vectors at a time
  constexpr int IN = TOK * LPR > 256 ? TOK * LPR / 256 : 1;
  __shared__ uint32_t tile[TOK][ROW];
  __shared__ int page_of[TOK], place_of[TOK];
  const int tid = threadIdx.x;
  const int h = blockIdx.x % c.heads, m0 = blockIdx.x / c.heads * TOK;
  const int set = tid / LPR, d = 8 * (tid % LPR);

  b4i kw[IN], vw[IN];
#pragma unroll
  for (int i = 0; i < IN; ++i) {
    const int t = set + AT * i, m = m0 + t;
    kw[i] = vw[i] = (b4i){0, 0, 0, 0};
    if (t < TOK && m < a.M && d < c.D) {
      kw[i] = *reinterpret_cast<const b4i*>(a.k + m * a.k_token + h * a.k_head + d);
      vw[i] = *reinterpret_cast<const b4i*>(a.v + m * a.v_token + h * a.v_head + d);
    }
  }
  if (tid < TOK) {
    const int m = m0 + tid;
    int page = -1, place = 0;
    if (m < a.M) {
      const int e = a.entry ? a.entry[m] : m, pos = a.position[m];
      if ((unsigned)e < (unsigned)a.B && pos >= 0 && (pos >> shift) < a.T) {
        page = a.table[e * a.table_row + (pos >> shift)];
        place = pos & (c.page - 1);
        if ((unsigned)page >= (unsigned)c.pages) page = -1;
      }
    }
    page_of[tid] = page;
    place_of[tid] = place;
  }
  __syncthreads();

#pragma unroll
  for (int i = 0; i < IN; ++i) {
    const int t = set + AT * i;
    if (t >= TOK) break;                               // whole sets of lanes
    const int page = page_of[t], place = place_of[t];
    const bool live = page >= 0 && d < c.D;
    const size_t row = ((size_t)h << shift) + place;
    if constexpr (FMT == SVDQ_KV_VALUES) {
      if (live) *reinterpret_cast<b4i*>(static_cast<uint16_t*>(c.k) + page * c.k_page + row * c.D + d) = kw[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) tile[t][d / QD + j] = (uint32_t)vw[i][j];
    } else {
      float ks, vs;
      const uint2 kc = encode<FMT, DT, LPR>(kw[i], &ks), vc = encode<FMT, DT, LPR>(vw[i], &vs);
      if (live) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(c.k) + page * c.k_page + row * c.D + d) = kc;
        if (d == 0) {
          c.k_scale[page * c.scale_page + row] = ks;
          c.v_scale[page * c.scale_page + row] = vs;
        }
      }
      tile[t][d / QD] = vc.x;
      tile[t][d / QD + 1] = vc.y;
    }
  }
  __syncthreads();

  // values: items of 4 tokens x QD elements
  for (int i = tid; i < TOK / 4 * (c.D / QD); i += 256) {
    const int t = 4 * (i % (TOK / 4)), dq = i / (TOK / 4);
    const int page = page_of[t], place = place_of[t];
    uint32_t r[4];
    bool whole = page >= 0 && (place & 3) == 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      r[j] = tile[t + j][dq];
      whole = whole && page_of[t + j] == page && place_of[t + j] == place + j;
    }
    if (whole) {
      const size_t at = page * c.v_page + (((size_t)h * c.D + QD * dq) << shift) + place;
      if constexpr (ES == 1) {
        uint32_t o[4];
        turn4(r, o);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(c.v) + at + ((size_t)e << shift)) = o[e];
      } else {
        uint16_t* p = static_cast<uint16_t*>(c.v) + at;
        *reinterpret_cast<uint2*>(p) = make_uint2(__builtin_amdgcn_perm(r[1], r[0], 0x05040100),
                                                  __builtin_amdgcn_perm(r[3], r[2], 0x05040100));
        *reinterpret_cast<uint2*>(p + ((size_t)1 << shift)) =
            make_uint2(__builtin_amdgcn_perm(r[1], r[0], 0x07060302), __builtin_amdgcn_perm(r[3], r[2], 0x07060302));
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int pg = page_of[t + j];
        if (pg < 0) continue;
        const size_t at = pg * c.v_page + (((size_t)h * c.D + QD * dq) << shift) + place_of[t + j];
#pragma unroll
        for (int e = 0; e < QD; ++e) {
          if constexpr (ES == 1)
            static_cast<uint8_t*>(c.v)[at + ((size_t)e << shift)] = (uint8_t)(r[j] >> (8 * e));
          else
            static_cast<uint16_t*>(c.v)[at + ((size_t)e << shift)] = (uint16_t)(r[j] >> (16 * e));
        }
      }
    }
  }
}

// A block: 64 positions of one request and head, keys and values.
template <int FMT, int DT, int LPR>
__global__ __launch_bounds__(256) void read_kernel(svdq_kv_cache c, svdq_cache_read_args a, int shift, int tiles) {
  using S = CacheShape<FMT, LPR>;
  constexpr int ES = S::ES, QD = S::QD, ROW = S::ROW, TOK = 64;
  __shared__ uint32_t tile[TOK][ROW];
  __shared__ int page_of[TOK / 16];
  const int tid = threadIdx.x;
  const int h = blockIdx.x % c.heads, rest = blockIdx.x / c.heads, b = rest / tiles;
  const int64_t start = a.start ? a.start[b] : 0;
  const int64_t end = min(min((int64_t)a.kv_len[b], (int64_t)a.T << shift), start + a.S);
  const int64_t p0 = (max(start, (int64_t)0) / TOK + rest % tiles) * TOK;   // first position of the block
  if (p0 >= end) return;
  if (tid < TOK / 16) {
    const int64_t i = (p0 + 16 * tid) >> shift;
    int page = i < a.T ? a.table[b * a.table_row + i] : -1;
    if ((unsigned)page >= (unsigned)c.pages) page = -1;
    page_of[tid] = page;
  }
  __syncthreads();
  const int mask = c.page - 1;

  // values: items of 8 tokens x QD elements, turned into rows of tokens
  for (int i = tid; i < TOK / 8 * (c.D / QD); i += 256) {
    const int t = 8 * (i % (TOK / 8)), dq = i / (TOK / 8), page = page_of[t / 16];
    if (page < 0) continue;
    const size_t at = page * c.v_page + (((size_t)h * c.D + QD * dq) << shift) + ((p0 + t) & mask);
    if constexpr (ES == 1) {
      uint2 w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.v) + at + ((size_t)e << shift));
      const uint32_t lo[4] = {w[0].x, w[1].x, w[2].x, w[3].x}, hi[4] = {w[0].y, w[1].y, w[2].y, w[3].y};
      uint32_t o[4];
      turn4(lo, o);
#pragma unroll
      for (int j = 0; j < 4; ++j) tile[t + j][dq] = o[j];
      turn4(hi, o);
#pragma unroll
      for (int j = 0; j < 4; ++j) tile[t + 4 + j][dq] = o[j];
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(c.v) + at;
      const b4i x = *reinterpret_cast<const b4i*>(p), y = *reinterpret_cast<const b4i*>(p + ((size_t)1 << shift));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        tile[t + 2 * j][dq] = __builtin_amdgcn_perm((uint32_t)y[j], (uint32_t)x[j], 0x05040100);
        tile[t + 2 * j + 1][dq] = __builtin_amdgcn_perm((uint32_t)y[j], (uint32_t)x[j], 0x07060302);
      }
    }
  }
  __syncthreads();

  const int d = 8 * (tid % LPR);
  if (d >= c.D) return;
  for (int t = tid / LPR; t < TOK; t += 256 / LPR) {
    const int64_t pos = p0 + t, j = pos - start;
    const int page = page_of[t / 16];
    if (j < 0 || pos >= end || page < 0) continue;
    const size_t row = ((size_t)h << shift) + (pos & mask);
    b4i kv, vv;
    if constexpr (FMT == SVDQ_KV_VALUES) {
      kv = *reinterpret_cast<const b4i*>(static_cast<const uint16_t*>(c.k) + page * c.k_page + row * c.D + d);
#pragma unroll
      for (int i = 0; i < 4; ++i) vv[i] = (int)tile[t][d / QD + i];
    } else {
      const uint2 kc = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.k) + page * c.k_page + row * c.D + d);
      kv = decode<FMT, DT>(kc, c.k_scale[page * c.scale_page + row]);
      vv = decode<FMT, DT>(make_uint2(tile[t][d / QD], tile[t][d / QD + 1]), c.v_scale[page * c.scale_page + row]);
    }
    *reinterpret_cast<b4i*>(a.k + b * a.k_batch + j * a.k_token + h * a.k_head + d) = kv;
    *reinterpret_cast<b4i*>(a.v + b * a.v_batch + j * a.v_token + h * a.v_head + d) = vv;
  }
}

// go(format, type, lanes of a vector) as compile-time values
template <class Fn>
void dispatch(const svdq_kv_cache& c, int32_t dtype, Fn&& go) {
  auto lanes = [&](auto f, auto t) {
    if (c.D <= 64) go(f, t, std::integral_constant<int, 8>{});
    else go(f, t, std::integral_constant<int, 16>{});
  };
  auto type = [&](auto f) {
    if (dtype == SVDQ_BF16) lanes(f, std::integral_constant<int, SVDQ_BF16>{});
    else lanes(f, std::integral_constant<int, SVDQ_FP16>{});
  };
  if (c.format == SVDQ_KV_INT8) type(std::integral_constant<int, SVDQ_KV_INT8>{});
  else if (c.format == SVDQ_KV_FP8) type(std::integral_constant<int, SVDQ_KV_FP8>{});
  else lanes(std::integral_constant<int, SVDQ_KV_VALUES>{}, std::integral_constant<int, SVDQ_BF16>{});   // copies
}

}  // namespace
}  // namespace svdq

using namespace svdq;

extern "C" svdq_status svdq_cache_write(const svdq_kv_cache* cache, const svdq_cache_write_args* args, void* stream) {
  if (!cache || !args || !args->k || !args->v || !args->position || !args->table) return SVDQ_ERR_ARG;
  svdq_status ok = cache_check(*cache);
  if (ok != SVDQ_OK) return ok;
  svdq_cache_write_args a = *args;
  if (!is_dtype(a.dtype)) return SVDQ_ERR_UNSUPPORTED;
  if (!table_fits(*cache, a.B, a.T, a.table_row)) return SVDQ_ERR_SHAPE;
  if (a.M < 1 || a.M > (1 << 20) || (!a.entry && a.M > a.B)) return SVDQ_ERR_SHAPE;
  // Tokens of a block: 64 fill the stores of the turned values, 16 more compute
  // units.
  const int tok = (int64_t)((a.M + 63) / 64) * cache->heads >= kCus ? 64 : 16;
  const int64_t blocks = (int64_t)((a.M + tok - 1) / tok) * cache->heads;
  if (blocks >= (1 << 24)) return SVDQ_ERR_SHAPE;
  for (int64_t s : {a.k_token, a.k_head, a.v_token, a.v_head})
    if (s % 8 != 0) return SVDQ_ERR_ALIGN;
  if (!on16(a.k) || !on16(a.v) || !on4(a.table) || !on4(a.entry) || !on4(a.position)) return SVDQ_ERR_ALIGN;
  if ((ok = device_ok()) != SVDQ_OK) return ok;
  if (a.B == 1) a.table_row = 0;
  const int shift = __builtin_ctz(cache->page);
  hipStream_t st = static_cast<hipStream_t>(stream);
  dispatch(*cache, a.dtype, [&](auto f, auto t, auto l) {
    constexpr int F = decltype(f)::value, T = decltype(t)::value, L = decltype(l)::value;
    if (tok == 64) hipLaunchKernelGGL((write_kernel<F, T, L, 64>), dim3((unsigned)blocks), dim3(256), 0, st, *cache, a, shift);
    else hipLaunchKernelGGL((write_kernel<F, T, L, 16>), dim3((unsigned)blocks), dim3(256), 0, st, *cache, a, shift);
  });
  return launched();
}

extern "C" svdq_status svdq_cache_read(const svdq_kv_cache* cache, const svdq_cache_read_args* args, void* stream) {
  if (!cache || !args || !args->k || !args->v || !args->kv_len || !args->table) return SVDQ_ERR_ARG;
  svdq_status ok = cache_check(*cache);
  if (ok != SVDQ_OK) return ok;
  svdq_cache_read_args a = *args;
  if (!is_dtype(a.dtype)) return SVDQ_ERR_UNSUPPORTED;
  if (!table_fits(*cache, a.B, a.T, a.table_row) || a.S < 1 || a.S > (1 << 24)) return SVDQ_ERR_SHAPE;
  const int tiles = (a.S + 63) / 64 + (a.start ? 1 : 0);   // a start inside a tile: one more
  if ((int64_t)a.B * tiles > (1 << 24) || (int64_t)a.B * tiles * cache->heads >= (1 << 24)) return SVDQ_ERR_SHAPE;
  for (int64_t s : {a.k_batch, a.k_token, a.k_head, a.v_batch, a.v_token, a.v_head})
    if (s % 8 != 0) return SVDQ_ERR_ALIGN;
  if (!on16(a.k) || !on16(a.v) || !on4(a.table) || !on4(a.kv_len) || !on4(a.start)) return SVDQ_ERR_ALIGN;
  if ((ok = device_ok()) != SVDQ_OK) return ok;
  if (a.B == 1) a.table_row = 0;
  const int shift = __builtin_ctz(cache->page);
  const dim3 grid((unsigned)(a.B * tiles * cache->heads));
  hipStream_t st = static_cast<hipStream_t>(stream);
  dispatch(*cache, a.dtype, [&](auto f, auto t, auto l) {
    hipLaunchKernelGGL((read_kernel<decltype(f)::value, decltype(t)::value, decltype(l)::value>), grid, dim3(256), 0, st,
                       *cache, a, shift, tiles);
  });
  return launched();
}
