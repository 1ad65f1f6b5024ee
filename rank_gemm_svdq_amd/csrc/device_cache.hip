// Writing keys and values into a paged cache, in 8 bits or as they are, and
// reading them back.
//
// Keys lie token by token, [page][head][place][D], and values element by element,
// [page][head][D][place], so that attention's matrix operands are 16-byte loads of
// either (device_paged.hip).  Values therefore turn on their way through LDS: a
// block takes 64 tokens of one head, and eights of them that lie side by side in a
// page from a place that is a multiple of 8 are stored and loaded as one piece (four at
// a time 22.0 us for what takes 18.2 now), others one by one.  Few tokens go
// straight from registers (write_few_kernel).
//
// Both ways move each value once and each code once, and the memory's rate bounds
// them: 4608 tokens x 24 heads of 128 into E4M3 codes 18.2 us, out of them 17.8 us, 4.7
// and 4.8 TB/s.  (What is read back stored past the caches: the attention that reads it
// loses more.)
//
// Codes.  INT8: s = max (1 / 127), the code nearest to x / s.  The first guess
// rint(x / s) by a reciprocal is off by at most one, and x - code s, which one fma
// gives exactly, tells.  FP8: s is a power of two, so x / s is exact and the
// conversion's rounding is the only one.

#include "device_kv.h"

namespace svdq {
namespace {

// LPR lanes (8 elements each) hold a token's vector.  A value or code has ES bytes; a
// dword of a row in LDS holds QD elements.
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
  auto with = [&](auto ctrl) {
    top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, top, decltype(ctrl)::value, 0xF, 0xF, true));
  };
  with(std::integral_constant<int, 0xB1>{});    // lanes 1, 0, 3, 2 of a quad
  with(std::integral_constant<int, 0x4E>{});    // 2, 3, 0, 1
  with(std::integral_constant<int, 0x141>{});   // half a row of 16 mirrored
  if constexpr (LPR == 16) with(std::integral_constant<int, 0x140>{});   // a row mirrored
  if (top >= 0x7F800000u) {
    *scale = __uint_as_float(0x7FC00000u);
    return make_uint2(0, 0);
  }
  if constexpr (FMT == SVDQ_KV_FP8) {
    // the power of two at or above max / 448, 448 = 1.75 x 2^8
    const uint32_t e = (uint32_t)max((int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u), 1);
    *scale = top ? __uint_as_float(e << 23) : 0.f;
    const float by = __uint_as_float((254u - e) << 23);
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * by, x[1] * by, lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2] * by, x[3] * by, lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4] * by, x[5] * by, hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6] * by, x[7] * by, hi, true);
    return make_uint2((uint32_t)lo, (uint32_t)hi);
  } else {
    float s = __uint_as_float(top) * (1.0f / 127.0f);
    if (s < 0x1p-126f) s = 0.f;
    *scale = s;
    const float by = s > 0.f ? __builtin_amdgcn_rcpf(s) : 0.f;
    float c[8], left[8], most = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = rintf(x[i] * by);
      left[i] = fmaf(-c[i], s, x[i]);
      most = fmaxf(most, fabsf(left[i]));
    }
    if (s > 0.f && most + most >= s) {
      // past the middle between two codes, or on it with an odd one: one further
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float twice = fabsf(left[i] + left[i]);
        if (twice > s || (twice == s && ((int)c[i] & 1) != 0)) c[i] += left[i] < 0.f ? -1.f : 1.f;
      }
    }
    uint32_t v[8];   // the code in the low byte
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __float_as_uint(c[i] + 0x1.8p23f);
    auto four = [&](int i) {
      return __builtin_amdgcn_perm(__builtin_amdgcn_perm(v[i + 3], v[i + 2], 0x0C0C0400),
                                   __builtin_amdgcn_perm(v[i + 1], v[i], 0x0C0C0400), 0x05040100);
    };
    return make_uint2(four(0), four(4));
  }
}

// Where a token goes: its page (-1: nowhere) and place.
__device__ __forceinline__ int2 place_of_token(const svdq_kv_cache& c, const svdq_cache_write_args& a, int shift, int m) {
  const int e = a.entry ? a.entry[m] : m, pos = a.position[m];
  if ((unsigned)e >= (unsigned)a.B || pos < 0 || (pos >> shift) >= a.T) return make_int2(-1, 0);
  const int page = a.table[e * a.table_row + (pos >> shift)];
  return make_int2((unsigned)page < (unsigned)c.pages ? page : -1, pos & (c.page - 1));
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

// Few tokens: LPR lanes take one of one head, and store its values as they have them,
// one by one (each in a line of its own, as places of one element lie together).
template <int FMT, int DT, int LPR>
__global__ __launch_bounds__(256) void write_few_kernel(svdq_kv_cache c, svdq_cache_write_args a, int shift) {
  constexpr int ES = FMT == SVDQ_KV_VALUES ? 2 : 1;
  const int unit = blockIdx.x * (256 / LPR) + threadIdx.x / LPR, d = 8 * (threadIdx.x % LPR);
  const int m = unit / c.heads, h = unit - m * c.heads;
  if (m >= a.M) return;                              // whole sets of lanes
  b4i kw = (b4i){0, 0, 0, 0}, vw = kw;
  if (d < c.D) {
    kw = *reinterpret_cast<const b4i*>(a.k + m * a.k_token + h * a.k_head + d);
    vw = *reinterpret_cast<const b4i*>(a.v + m * a.v_token + h * a.v_head + d);
  }
  const int2 at = place_of_token(c, a, shift, m);
  const size_t row = ((size_t)h << shift) + at.y;
  const bool live = at.x >= 0 && d < c.D;
  const size_t vat = at.x * c.v_page + (((size_t)h * c.D + d) << shift) + at.y;
  if constexpr (ES == 2) {
    if (live) {
      *reinterpret_cast<b4i*>(static_cast<uint16_t*>(c.k) + at.x * c.k_page + row * c.D + d) = kw;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        static_cast<uint16_t*>(c.v)[vat + ((size_t)i << shift)] = (uint16_t)((uint32_t)vw[i / 2] >> (16 * (i % 2)));
    }
  } else {
    float ks, vs;
    const uint2 kc = encode<FMT, DT, LPR>(kw, &ks), vc = encode<FMT, DT, LPR>(vw, &vs);
    if (live) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(c.k) + at.x * c.k_page + row * c.D + d) = kc;
      if (d == 0) {
        c.k_scale[at.x * c.scale_page + row] = ks;
        c.v_scale[at.x * c.scale_page + row] = vs;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        static_cast<uint8_t*>(c.v)[vat + ((size_t)i << shift)] = (uint8_t)((i < 4 ? vc.x : vc.y) >> (8 * (i % 4)));
    }
  }
}

// Many tokens: a block takes 64 of one head, keys and values.
template <int FMT, int DT, int LPR>
__global__ __launch_bounds__(256) void write_kernel(svdq_kv_cache c, svdq_cache_write_args a, int shift) {
  using S = CacheShape<FMT, LPR>;
  constexpr int ES = S::ES, QD = S::QD, ROW = S::ROW, TOK = 64;
  constexpr int AT = 256 / LPR;                        // vectors at a time
  constexpr int IN = TOK / AT;
  __shared__ uint32_t tile[TOK][ROW];
  __shared__ int page_of[TOK], place_of[TOK];
  __shared__ int64_t run[TOK / 8];                     // where 8 tokens' values lie side by side, -1 if they do not
  __shared__ int phase;
  const int tid = threadIdx.x;
  // Eights of places begin where a page's do.  The blocks' first tokens are chosen so
  // for the call's first request, and within a block the eights begin at `phase`, the
  // first token on such a place by what the block's first live token says.
  const int h = blockIdx.x % c.heads, m0 = (int)(blockIdx.x / c.heads) * TOK - (a.position[0] & 7);
  const int set = tid / LPR, d = 8 * (tid % LPR);

  b4i kw[IN], vw[IN];
#pragma unroll
  for (int i = 0; i < IN; ++i) {
    const int m = m0 + set + AT * i;
    kw[i] = vw[i] = (b4i){0, 0, 0, 0};
    if (m >= 0 && m < a.M && d < c.D) {
      kw[i] = *reinterpret_cast<const b4i*>(a.k + m * a.k_token + h * a.k_head + d);
      vw[i] = *reinterpret_cast<const b4i*>(a.v + m * a.v_token + h * a.v_head + d);
    }
  }
  if (tid < TOK) {
    const int2 at = m0 + tid >= 0 && m0 + tid < a.M ? place_of_token(c, a, shift, m0 + tid) : make_int2(-1, 0);
    page_of[tid] = at.x;
    place_of[tid] = at.y;
    const uint64_t live = __ballot(at.x >= 0);         // the first wave
    const int ref = live ? __builtin_ctzll(live) : 0;
    if (tid == ref) phase = (ref - at.y) & 7;
  }
  __syncthreads();
  const int lead = phase;
  if (tid < TOK / 8) {
    const int t = lead + 8 * tid, page = page_of[t], place = place_of[t];
    bool whole = t + 7 < TOK && page >= 0 && (place & 7) == 0;
#pragma unroll
    for (int j = 1; j < 8; ++j) {
      const int k = min(t + j, TOK - 1);
      whole = whole && page_of[k] == page && place_of[k] == place + j;
    }
    run[tid] = whole ? ES * (page * c.v_page + ((int64_t)h * c.D << shift) + place) : -1;
  }

#pragma unroll
  for (int i = 0; i < IN; ++i) {
    const int t = set + AT * i, page = page_of[t], place = place_of[t];
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

  // values: items of 8 tokens x QD elements, stored 8 at a time where they lie side by
  // side, else one by one
  auto one = [&](int t, int dq, uint32_t r) __attribute__((always_inline)) {
    const int page = page_of[t];
    if (page < 0) return;
    const size_t at = page * c.v_page + (((size_t)h * c.D + QD * dq) << shift) + place_of[t];
#pragma unroll
    for (int e = 0; e < QD; ++e) {
      if constexpr (ES == 1) static_cast<uint8_t*>(c.v)[at + ((size_t)e << shift)] = (uint8_t)(r >> (8 * e));
      else static_cast<uint16_t*>(c.v)[at + ((size_t)e << shift)] = (uint16_t)(r >> (16 * e));
    }
  };
  for (int i = tid; i < lead * (c.D / QD); i += 256) one(i % lead, i / lead, tile[i % lead][i / lead]);
  for (int i = tid; i < TOK / 8 * (c.D / QD); i += 256) {
    const int g = i % (TOK / 8), t = lead + 8 * g, dq = i / (TOK / 8);
    uint32_t r[2][4];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j / 4][j % 4] = tile[min(t + j, TOK - 1)][dq];
    const int64_t at = run[g];
    if (at >= 0) {
      uint8_t* to = static_cast<uint8_t*>(c.v) + at + ((size_t)(ES * QD * dq) << shift);
      if constexpr (ES == 1) {
        uint32_t o[2][4];
        turn4(r[0], o[0]);
        turn4(r[1], o[1]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<uint2*>(to + ((size_t)e << shift)) = make_uint2(o[0][e], o[1][e]);
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          b4i o;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            o[j] = (int)__builtin_amdgcn_perm(r[j / 2][2 * (j % 2) + 1], r[j / 2][2 * (j % 2)], e ? 0x07060302 : 0x05040100);
          *reinterpret_cast<b4i*>(to + ((size_t)(2 * e) << shift)) = o;
        }
      }
      continue;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (t + j < TOK) one(t + j, dq, r[j / 4][j % 4]);
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

  // keys, on their way while the values turn
  constexpr int AT = 256 / LPR, IN = TOK / AT;
  const int d = 8 * (tid % LPR);
  typedef typename std::conditional<ES == 1, uint2, b4i>::type Piece;
  Piece kc[IN];
  float ks[IN], vs[IN];
#pragma unroll
  for (int i = 0; i < IN; ++i) {
    const int t = tid / LPR + AT * i, page = page_of[t / 16];
    kc[i] = Piece{};
    ks[i] = vs[i] = 0.f;
    if (page >= 0 && d < c.D) {
      const size_t row = ((size_t)h << shift) + ((p0 + t) & mask);
      kc[i] = *reinterpret_cast<const Piece*>(static_cast<const uint8_t*>(c.k) + ES * (page * c.k_page + row * c.D + d));
      if constexpr (ES == 1) {
        ks[i] = c.k_scale[page * c.scale_page + row];
        vs[i] = c.v_scale[page * c.scale_page + row];
      }
    }
  }

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

  if (d >= c.D) return;
#pragma unroll
  for (int i = 0; i < IN; ++i) {
    const int t = tid / LPR + AT * i;
    const int64_t pos = p0 + t, j = pos - start;
    if (j < 0 || pos >= end || page_of[t / 16] < 0) continue;
    b4i kv, vv;
    if constexpr (FMT == SVDQ_KV_VALUES) {
      kv = kc[i];
#pragma unroll
      for (int w = 0; w < 4; ++w) vv[w] = (int)tile[t][d / QD + w];
    } else {
      kv = decode<FMT, DT>(kc[i], ks[i]);
      vv = decode<FMT, DT>(make_uint2(tile[t][d / QD], tile[t][d / QD + 1]), vs[i]);
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
  // Blocks of 64 tokens and a head, or where those are few, 16 or 32 lots of one token and
  // one head (a run of 512 tokens x 8 heads of 128 5.9 us instead of 7.3, of 1024 8.9 instead of
  // 7.8; the next tokens of 16 requests 3.9 instead of 6.4, of 128 4.9 instead of 9.5).
  const bool few = (int64_t)((a.M + 63) / 64) * cache->heads < 128;
  const int lots = cache->D <= 64 ? 32 : 16;
  const int64_t blocks = few ? ((int64_t)a.M * cache->heads + lots - 1) / lots : (int64_t)((a.M + 7 + 63) / 64) * cache->heads;
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
    if (few) hipLaunchKernelGGL((write_few_kernel<F, T, L>), dim3((unsigned)blocks), dim3(256), 0, st, *cache, a, shift);
    else hipLaunchKernelGGL((write_kernel<F, T, L>), dim3((unsigned)blocks), dim3(256), 0, st, *cache, a, shift);
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
