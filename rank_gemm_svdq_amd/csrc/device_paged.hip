// Attention of one new token of each request over a paged cache, 16-bit values or
// codes: one pass over K and V, split over the cache's length and joined.
//
// Rows.  The G query heads that share a K/V head are the rows of one matrix, 16 to a
// row tile; a block of four waves takes one or two row tiles of one (request, K/V
// head) over a share of its keys, the waves in turn.
//
// A tile of TK keys (64 codes or 32 values), per wave, all operands straight from
// memory to registers (16x16x32 MFMA; lane l: c = l % 16, u = l / 16):
//   S^T = K Q^T   A = K.  Row 4 a + i of score tile t is key KPL a + 4 t + i (KPL =
//                 TK / 4), and the result's lane then holds row c of Q and
//                 the keys KPL u .. + KPL of the tile in order.
//   O^T += V^T P  P as it stands, rounded to 16 bits, is the B operand: 8 keys to an
//                 MFMA.  A = V^T: element 16 d + c of the keys KPL u .. + KPL, 16
//                 neighbouring bytes of the cache's order [head][D][place].
// A lane's KPL keys lie in one page (pages are multiples of 16), so a tile may span
// pages: every lane looks its own page up, two tiles ahead.  A tile's operands are asked
// for as soon as the registers that they go to have been used for the tile before.
//
// Codes.  E4M3 goes to fp16, exactly, and a query row with it, scaled by a power of two
// that brings its largest element to [1, 2): what falls below fp16's range is under
// 2^-24 of that.  INT8 keys are multiplied as they are by queries of 24 bits in three digits
// of 8, summed exactly in int32; INT8 values become fp16 of their bits (widen_codes).
// The key's scale multiplies the score, and the value's scale the weight; of these
// products a row's largest so far is kept between 2^6 and 2^14 by a power of two (iv), which
// rises and falls with the maximum, so that neither a scale without weight nor a weight
// without scale takes the bits of those that count.
//
// Softmax.  A row's maximum is raised when a tile exceeds it by more than kLag
// (powers of two), which a vote of the wave finds out without exchanges; weights
// then carry 2^kLift to the middle of their type's range.
//
// What bounds it.  Each key and value is read once, and the memory's rate is reached where
// all compute units have work: 16 requests of up to 16384 INT8 keys, 8 heads of 128,
// 67.1 us; one of 131072 E4M3 keys 54.4; 40 of up to 3001 fp16 keys within a window of
// 1500, 24 heads of 64, 63.5.  A compute unit by itself takes in 49 GB/s where eight do and
// 42 where 128 do, from memory and from the last-level cache alike, however many waves ask,
// so fewer blocks than units leave the rate behind; 600 INT8 keys take 8.2 us in one part,
// which is a launch and the chain length, page, K, scores, V, join of waves.  (Blocks of
// eight waves, a wave on two tiles at a time, K in whole lines with its pieces exchanged: the
// same time; K and V loaded past the caches: 5 to 10 % more.)
//
// Parts are shares of the table's width, which the host sees, not of the lengths: 4096 keys
// take 10.0 us in a table for as many and 28.9 in one for 131072; 15 requests of 512 keys
// beside one of 131072 take 356.
#include "device_kv.h"
#include "device_score.h"

namespace svdq {
namespace {

struct PagedPart {          // how the keys are split over blocks
  int32_t share, splits;    // keys of a block (a multiple of 256), parts at most
  float* o;                 // [splits][B Hq][DP]: means of the values
  float* ml;                // [splits][B Hq][2]: maximum (log2) and sum of weights
};

struct PagedP {
  svdq_paged_attention_args a;
  svdq_kv_cache c;
  int G, rows, shift;       // heads of a K/V head, blocks for its rows, log2 page
  uint32_t by_splits, by_heads;   // 2^32 / parts and / heads, rounded up (0: does not serve)
  float qmul, c1, c2, c3, c4;   // see set_score()
  float cap[7];
  bool flip;
  PagedPart part;
};

constexpr float kLag = 8.0f;
// fp16 weights between 2^6 and 2^14 at the maximum: the smallest that keeps its bits
// is 2^-20 of it, 2^-30 with half of them.  bf16: at most 2^-22, so that the sum of the 2^22
// keys that a wave may see stays in fp32 whatever their values (those under 2^-96 lose bits).
// Codes: at most 1, so that a weight times any scale of V stays in fp32; to fp16 go these
// products, with a range of their own.
template <int FMT, int DT>
constexpr float kLift = FMT != SVDQ_KV_VALUES ? -kLag : DT == SVDQ_BF16 ? -30.0f : 6.0f;

// FP16: codes or fp16 values
template <bool FP16>
__device__ __forceinline__ b4f mma16(const b4i& a, const b4i& b, const b4f& c) {
  if constexpr (FP16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(b8h, a), __builtin_bit_cast(b8h, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8bf, a), __builtin_bit_cast(b8bf, b), c, 0, 0, 0);
}

// 8 codes as fp16.  E4M3: as they are, in order.  INT8: (code + 128) 2^-24, fp16
// values below its normal range, in the order 0, 2, 1, 3, 4, 6, 5, 7: the bytes
// need no arithmetic, and the 128 is taken out of the sums at the end.
template <int FMT>
__device__ __forceinline__ b4i widen_codes(int lo, int hi) {
  b4i r;
  if constexpr (FMT == SVDQ_KV_INT8) {
    const uint32_t x = (uint32_t)lo ^ 0x80808080u, y = (uint32_t)hi ^ 0x80808080u;
    r[0] = (int)(x & 0x00FF00FFu);
    r[1] = (int)__builtin_amdgcn_perm(0, x, 0x0C030C01);
    r[2] = (int)(y & 0x00FF00FFu);
    r[3] = (int)__builtin_amdgcn_perm(0, y, 0x0C030C01);
  } else {
    r[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false));
    r[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true));
    r[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false));
    r[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true));
  }
  return r;
}

// what lane N of each row of 16 lanes holds
template <int N>
__device__ __forceinline__ float of_lane(float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x150 + N, 0xF, 0xF, true));
}
template <class Fn, int... I>
__device__ __forceinline__ void each(Fn&& fn, std::integer_sequence<int, I...>) {
  (fn(std::integral_constant<int, I>{}), ...);
}

// over the four lanes of a row
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float row_sum(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// The kernel's arguments, read again where they are used: what only the rare paths and
// the end need would otherwise sit in scalar registers, which run out in the loop.
__device__ __forceinline__ PagedP again() {
  uint64_t at = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(at));
  return *(const PagedP*)(__attribute__((address_space(4))) const PagedP*)at;
}

// Keys of request b that are visible, [lo, n), and its first part's first key.
struct Span {
  int lo, n, first;
};
__device__ __forceinline__ Span span_of(const PagedP& p, int b) {
  Span s;
  s.n = min(max(p.a.kv_len[b], 0), p.a.T << p.shift);
  s.lo = p.a.window > 0 ? max(s.n - p.a.window, 0) : 0;
  s.first = s.lo & ~63;
  return s;
}

template <int FMT, int DT, int DP, bool PAD, int RT>
__global__ __launch_bounds__(256, RT == 2 && DP == 128 ? 1 : 2) void paged_kernel(PagedP p) {
  constexpr bool CODES = FMT != SVDQ_KV_VALUES, INT8 = FMT == SVDQ_KV_INT8;
  constexpr bool FP16 = CODES || DT == SVDQ_FP16;
  constexpr int ES = CODES ? 1 : 2;
  constexpr int KPL = 16 / ES, TK = 4 * KPL;     // keys of a lane and of a tile
  constexpr int NT = TK / 16;                    // score tiles
  constexpr int NC = DP * ES / 64;               // 16-byte pieces of K a lane reads of a key
  constexpr int NS = DP / 32;                    // MFMA steps of a score tile (INT8: 3 NC, 64 wide, of three digits of Q)
  constexpr int ND = DP / 16;                    // element tiles of O
  constexpr int NU = TK / 32;                    // MFMA steps of O
  constexpr int NW = 4, STEP = NW * TK;          // waves, and keys from a wave's tile to its next
  constexpr float LIFT = kLift<FMT, DT>;
  __shared__ __attribute__((aligned(16))) float jo[NW][16 * RT][DP + 4];
  __shared__ float jm[NW][16 * RT][2];
  const svdq_paged_attention_args& a = p.a;
  const svdq_kv_cache& c = p.c;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lc = lane & 15, lu = lane >> 4;
  // Which part, rows and (request, K/V head).  Divisions of a few instructions: by what
  // the host worked out, or none where the divisor is 1.
  const uint32_t id = xcd_order(blockIdx.x, gridDim.x);
  const uint32_t rest = p.part.splits == 1 ? id : __umulhi(id, p.by_splits);
  const int sp = id - rest * p.part.splits;
  const uint32_t grp = p.rows == 1 ? rest : rest / p.rows;
  const int rb = rest - grp * p.rows;
  const uint32_t entry = p.a.B == 1 ? 0 : p.by_heads ? __umulhi(grp, p.by_heads) : grp / c.heads;
  const int b = entry, h = grp - entry * c.heads;
  const int D = PAD ? c.D : DP;
  // ---- Q: asked for before all else
  b4i qf[RT][NS], q8[RT][INT8 ? 3 * NC : 1];     // (q8: INT8's digits)
  float rq[RT], rk[RT], slope[RT];               // a row's factor, in two: at most 1, at least 1
  int qh[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    qh[r] = h * p.G + min(rb * 16 * RT + 16 * r + lc, p.G - 1);
    slope[r] = a.slopes ? a.slopes[qh[r]] * 1.44269504f : 0.f;
    const uint16_t* qp = a.q + b * a.q_batch + qh[r] * a.q_head;
    // the elements that meet K's piece of the same step in this lane
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int d = CODES ? 64 * (s / 2) + 16 * lu + 8 * (s % 2) : 32 * s + 8 * lu;
      qf[r][s] = (b4i){0, 0, 0, 0};
      if (!PAD || d < D) qf[r][s] = *reinterpret_cast<const b4i*>(qp + d);
    }
  }

  // page of key j of the request: -1 if there is none
  const int32_t* table = a.table + b * a.table_row;
  auto page_of = [&](int j) __attribute__((always_inline)) -> int {
    const int page = table[min(j >> p.shift, a.T - 1)];
    return (unsigned)page < (unsigned)c.pages ? page : -1;
  };
  const int mask = c.page - 1;
  const int kg = KPL * (lc >> 2), vg = KPL * lu;   // keys of a tile whose pages the lane needs: K's, V's and the scores'

  // Without a window the block's first key does not depend on the length, and the
  // first pages are looked up while that is on its way.
  int first = 0;
  if (a.window > 0) first = span_of(p, b).first;
  const int begin = first + sp * p.part.share;
  int j = begin + TK * wave;
  int kpage = page_of(j + kg), vpage = page_of(j + vg);   // pages of this tile and of the next
  int knext = page_of(j + STEP + kg), vnext = page_of(j + STEP + vg);
  const Span sn = span_of(p, b);
  const int end = min(sn.n, begin + p.part.share);
  if (sp > 0 && begin >= end) {                  // no such part: no weights
    for (int r = threadIdx.x; r < 16 * RT && rb * 16 * RT + r < p.G; r += 64 * NW)
      *reinterpret_cast<float2*>(p.part.ml + 2 * ((size_t)sp * ((size_t)a.B * a.Hq) + (size_t)b * a.Hq + h * p.G + rb * 16 * RT + r)) =
          make_float2(kLow, 0.f);
    return;
  }

  float m[RT], l[RT], iv[RT];                    // iv: what weights times V's scales are multiplied by, at most 2^126
  b4f o[RT][ND], ow[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    ow[r] = (b4f){0.f, 0.f, 0.f, 0.f};
    m[r] = kLow;
    l[r] = 0.f;
    iv[r] = 0x1p126f;
#pragma unroll
    for (int d = 0; d < ND; ++d) o[r][d] = (b4f){0.f, 0.f, 0.f, 0.f};
  }

  // ---- loads of the tile at j
  b4i kw[NT][NC], vw[ND];
  float ks = 0.f, vs = 0.f;                      // scales of key KPL lu + lc
  auto k_at = [&](int j, int page) __attribute__((always_inline)) -> const uint8_t* {
    return static_cast<const uint8_t*>(c.k) +
           ES * (max(page, 0) * c.k_page + (((int64_t)h << p.shift) + ((j + kg + (lc & 3)) & mask)) * D) + 16 * lu;
  };
  auto load_k = [&](const uint8_t* kp, int t) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (PAD) kw[t][i] = (b4i){0, 0, 0, 0};
      if (!PAD || 64 * i + 16 * lu < ES * D) kw[t][i] = *reinterpret_cast<const b4i*>(kp + 4 * t * ES * D + 64 * i);
    }
  };
  auto load_scales = [&](int j, int page) __attribute__((always_inline)) {
    if constexpr (CODES) {
      const int64_t at = max(page, 0) * c.scale_page + ((int64_t)h << p.shift) + ((j + vg) & mask) + lc;
      ks = c.k_scale[at];
      vs = c.v_scale[at];
    }
  };
  auto v_at = [&](int j, int page) __attribute__((always_inline)) -> const uint8_t* {
    return static_cast<const uint8_t*>(c.v) +
           ES * (max(page, 0) * c.v_page + (((int64_t)h * D + lc) << p.shift) + ((j + vg) & mask));
  };
  auto load_v = [&](const uint8_t* vp, int d) __attribute__((always_inline)) {
    if (PAD) vw[d] = (b4i){0, 0, 0, 0};
    if (!PAD || 16 * d < D) vw[d] = *reinterpret_cast<const b4i*>(vp + ((size_t)(16 * d * ES) << p.shift));
  };

  if (j < end) {
    const uint8_t *kp = k_at(j, kpage), *vp = v_at(j, vpage);
#pragma unroll
    for (int t = 0; t < NT; ++t) load_k(kp, t);
    load_scales(j, vpage);
#pragma unroll
    for (int d = 0; d < ND; ++d) load_v(vp, d);
  }

  // ---- Q as the B operand, while the first tile is on its way
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    rq[r] = rk[r] = 1.f;
    if constexpr (CODES) {
      // largest magnitude of the row, as bits: infinities and NaN are the largest
      typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
      u16x2 most = (u16x2){0, 0};
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, qf[r][s][i] & 0x7FFF7FFF));
      int tb = max((int)most[0], (int)most[1]);
      tb = max(tb, __shfl_xor(tb, 16));
      tb = max(tb, __shfl_xor(tb, 32));
      const float mag = widen2<DT>((uint32_t)tb)[0];
      const bool odd = tb >= (DT == SVDQ_BF16 ? 0x7F80 : 0x7C00);
      if constexpr (INT8) {
        // Whole numbers of 24 bits, in units of 2^-22 of a power of two that the largest element
        // is between 0.996 and 1.992 of, as three signed digits of 8 bits: a bf16 element above
        // 2^-15 of the largest keeps all its bits, and the sums of products are exact.  (Two
        // digits: the output 0.2 to 2.5 % off where a channel of the query is 300 to 3000 times
        // the others and the keys' is small in proportion; 600 keys 8.0 us, not 8.2.)
        const int e = max((int)((__float_as_uint(mag) + 0x10000u) >> 23), 1) - 127;
        rq[r] = odd ? __builtin_nanf("") : ldexpf(p.qmul, min(e - 22, 0));
        rk[r] = ldexpf(1.0f, max(e - 22, 0));
        const int keep = odd ? 0 : -1;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const b4i& q4 = qf[r][2 * i + w / 2];
            uint32_t v[4];                         // 128 more in each digit
#pragma unroll
            for (int k = 0; k < 4; ++k)
              v[k] = (uint32_t)((int)rintf(ldexpf(widen2<DT>((uint32_t)(q4[2 * (w % 2) + k / 2] & keep))[k % 2], 22 - e)) + 0x808080);
            const uint32_t x = __builtin_amdgcn_perm(v[1], v[0], 0x05040100), y = __builtin_amdgcn_perm(v[3], v[2], 0x05040100);
            q8[r][3 * i][w] = (int)((__builtin_amdgcn_perm(v[1], v[0], 0x0C0C0602) |
                                     __builtin_amdgcn_perm(v[3], v[2], 0x06020C0C)) ^ 0x80808080u);
            q8[r][3 * i + 1][w] = (int)(__builtin_amdgcn_perm(y, x, 0x07050301) ^ 0x80808080u);
            q8[r][3 * i + 2][w] = (int)(__builtin_amdgcn_perm(y, x, 0x06040200) ^ 0x80808080u);
          }
        }
      } else {
        // to [1, 2) by a power of two
        const int e = max((int)(__float_as_uint(mag) >> 23), 1) - 127;
        rq[r] = odd ? __builtin_nanf("") : __uint_as_float((uint32_t)(min(e, 0) + 127) << 23);
        rk[r] = __uint_as_float((uint32_t)(max(e, 0) + 127) << 23);
        const float by = ldexpf(p.qmul, -e);
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          float x[8];
          widen8<DT>(qf[r][s], x);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] *= by;
          qf[r][s] = narrow8<SVDQ_FP16>(x);
        }
      }
    } else if (!(p.qmul > 0.f)) {
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) qf[r][s][i] = p.flip ? qf[r][s][i] ^ (int)0x80008000 : 0;
    }
  }

  // The tile at j, whose loads are under way.  MORE: another follows, and each of its
  // operands is asked for as soon as this tile's has been used, into the same registers.
  auto tile = [&](int j, auto more) __attribute__((always_inline)) {
    constexpr bool MORE = decltype(more)::value;
    const int vj = j + vg;
    // keys [lo, hi) of the lane's are visible
    const int lo = vpage >= 0 ? sn.lo - vj : KPL, hi = vpage >= 0 ? end - vj : 0;
    const bool cut = __any(lo > 0 || hi < KPL);
    int kafter = -1, vafter = -1;
    if constexpr (MORE) {
      kafter = page_of(j + 2 * STEP + kg);
      vafter = page_of(j + 2 * STEP + vg);
    }

    // The next tile's K in four places among this tile's softmax, its V among the products
    // with V: a wave that asks for much at once waits until the unit has taken it in.
    const uint8_t* kp = nullptr;
    auto more_k = [&](int quarter) __attribute__((always_inline)) {
      if constexpr (MORE) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int t = NT * quarter / 4; t < NT * (quarter + 1) / 4; ++t) load_k(kp, t);
        __builtin_amdgcn_sched_barrier(0);
      }
    };

    // ---- scores
    b4f s[RT][NT];
    if constexpr (INT8) {
      if constexpr (MORE) kp = k_at(j + STEP, knext);
      b4i x[RT][NT], y[RT][NT];                    // of the two upper digits and of the last
#pragma unroll
      for (int step = 0; step < 3; ++step) {
        const int digit = step == 0 ? 0 : 3 - step;   // the last between the others, which wait for each other
        if (digit == 1)
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t) x[r][t] <<= 8;   // at most 128 x 128 x 128 x 256 = 2^29
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < RT; ++r) {
              b4i& to = digit < 2 ? x[r][t] : y[r][t];
              if (digit != 1 && i == 0) to = (b4i){0, 0, 0, 0};
              to = __builtin_amdgcn_mfma_i32_16x16x64_i8(kw[t][i], q8[r][3 * i + digit], to, 0, 0, 0);
            }
      }
      // K's first quarter before the sums are ready (after them 16 requests of up to 16384
      // keys 78.0 us, so 67.1)
      more_k(0);
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[r][t][i] = fmaf((float)x[r][t][i], 256.0f, (float)y[r][t][i]);
    } else {
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) s[r][t] = (b4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int st = 0; st < NS; ++st)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          b4i kf;
          if constexpr (CODES) kf = widen_codes<FMT>(kw[t][st / 2][2 * (st % 2)], kw[t][st / 2][2 * (st % 2) + 1]);
          else kf = kw[t][st];
#pragma unroll
          for (int r = 0; r < RT; ++r) s[r][t] = mma16<FP16>(kf, qf[r][st], s[r][t]);
        }
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (MORE) kp = k_at(j + STEP, knext);
      more_k(0);
    }
    if (CODES && (lc < lo || lc >= hi)) vs = 0.f;
    more_k(1);
    b4i pf[RT][NU];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      // a query's small factor before the key's scale, its large one after: no step leaves
      // fp32 unless q.k does
      if constexpr (CODES)
        each([&](auto x) { s[r][x / 4][x % 4] = s[r][x / 4][x % 4] * rq[r] * of_lane<x>(ks) * rk[r]; },
             std::make_integer_sequence<int, KPL>{});
      // in powers of two; rounded here and not in the exponent's sum, so that the largest
      // of enormous scores is the maximum itself
      if (a.softcap > 0.f) {
        const PagedP p = again();
        if (p.a.softcap <= kSmallCap) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[r][t][i] = by_exp(p, s[r][t][i]);
        } else {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float x = s[r][t][i], near = by_series(p, x), far = by_exp(p, x);
              s[r][t][i] = fabsf(x * p.c4) <= 1.0f ? near : far;
            }
        }
      } else {
#pragma unroll
        for (int t = 0; t < NT; ++t) s[r][t] *= p.c1;
      }
      if (a.slopes) {
        const float from = (float)(sn.n - 1 - vj);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[r][t][i] = fmaf(-slope[r], from - (float)(4 * t + i), s[r][t][i]);
      }
      if (cut) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (4 * t + i < lo || 4 * t + i >= hi) s[r][t][i] = -__builtin_inff();
      }
      if (r == 0) more_k(2);
      float top = s[r][0][0];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, s[r][t][i]);
      auto rescale = [&](float f) __attribute__((always_inline)) {
        ow[r] *= f;
#pragma unroll
        for (int d = 0; d < ND; ++d) o[r][d] *= f;
      };
      if (__any(top > m[r] + (LIFT + kLag))) {
        if constexpr (CODES) {
          // a whole number: by powers of two l falls and iv rises, as far as it may, in whose
          // place the sums fall
          const float up = fmaxf(m[r], floorf(row_max(top) - LIFT));
          const int k = (int)fminf(up - m[r], 300.0f);
          const float f = ldexpf(1.0f, -k), rise = fminf(ldexpf(1.0f, k), fminf(0x1p126f / iv[r], 0x1p126f));
          m[r] = up;
          l[r] *= f;
          iv[r] *= rise;
          if (__any(f * rise != 1.0f)) rescale(f * rise);
        } else {
          const float up = fmaxf(m[r], row_max(top) - LIFT);
          const float f = exp2_(m[r] - up);
          m[r] = up;
          l[r] *= f;
          rescale(f);
        }
      }
      if (r == 0) more_k(3);
      float w[4 * NT];
#pragma unroll
      for (int x = 0; x < 4 * NT; ++x) {
        w[x] = exp2_(s[r][x / 4][x % 4] - m[r]);
        l[r] += w[x];
      }
      if constexpr (CODES) {
        float big = 0.f;
        each([&](auto x) { big = fmaxf(big, w[x] *= of_lane<x>(vs)); }, std::make_integer_sequence<int, KPL>{});
        if (__any(big * iv[r] > 0x1p14f)) {
          big = row_max(big);
          // the largest to [2^6, 2^7)
          const float next = fminf(iv[r], ldexpf(1.0f, 133 - (int)(__float_as_uint(big) >> 23)));
          rescale(next * (1.0f / iv[r]));   // (powers of two: exact, or 0)
          iv[r] = next;
        }
#pragma unroll
        for (int x = 0; x < 4 * NT; ++x) w[x] *= iv[r];
      }
      // To the product with V the weights go in 16 bits, as the matrix unit takes them
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        constexpr int T16 = FP16 ? SVDQ_FP16 : SVDQ_BF16, I1 = INT8 ? 2 : 1, I2 = INT8 ? 1 : 2;   // in V's order
        pf[r][t / 2][2 * (t % 2)] = (int)narrow2<T16>(w[4 * t], w[4 * t + I1]);
        pf[r][t / 2][2 * (t % 2) + 1] = (int)narrow2<T16>(w[4 * t + I2], w[4 * t + 3]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (MORE) load_scales(j + STEP, vnext);
    __builtin_amdgcn_sched_barrier(0);

    // ---- values
    if (cut && !INT8) {                            // (codes of INT8 are all finite)
      // what is hidden takes no part, whatever is there
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t keep = 0;
#pragma unroll
        for (int k = 0; k < 4 / ES; ++k) {
          const int x = 4 / ES * i + k;
          if (x >= lo && x < hi) keep |= (ES == 1 ? 0xFFu : 0xFFFFu) << (8 * ES * k);
        }
#pragma unroll
        for (int d = 0; d < ND; ++d) vw[d][i] &= (int)keep;
      }
    }
    const uint8_t* vp = nullptr;
    if constexpr (MORE) vp = v_at(j + STEP, vnext);
#pragma unroll
    for (int d = 0; d < ND; ++d) {
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        b4i vf;
        if constexpr (CODES) vf = widen_codes<FMT>(vw[d][2 * u], vw[d][2 * u + 1]);
        else vf = vw[d];
#pragma unroll
        for (int r = 0; r < RT; ++r) o[r][d] = mma16<FP16>(vf, pf[r][u], o[r][d]);
      }
      if constexpr (MORE) {
        __builtin_amdgcn_sched_barrier(0);
        load_v(vp, d);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if constexpr (INT8) {
      // -128 2^-24 times the sum of the weights as rounded
      const int less = (int)0x80808080;
#pragma unroll
      for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int r = 0; r < RT; ++r) ow[r] = mma16<true>((b4i){less, less, less, less}, pf[r][u], ow[r]);
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (MORE) {
      kpage = knext;
      vpage = vnext;
      knext = kafter;
      vnext = vafter;
    }
  };
  if (j < end) {
    for (; j + STEP < end; j += STEP) tile(j, std::true_type{});
    tile(j, std::false_type{});
  }

  // ---- join the waves: means and (maximum, sum) through LDS
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const float sum = row_sum(l[r]);
    // a mean of codes is at most 448, so the scale comes back after the division; INT8's
    // 2^24 with the division, as together with the scale it may leave fp32
    const float by = sum != 0.f ? (INT8 ? 0x1p24f : 1.0f) / sum : 0.f, back = CODES ? 1.0f / iv[r] : 1.f;
#pragma unroll
    for (int d = 0; d < ND; ++d)
      *reinterpret_cast<b4f*>(&jo[wave][16 * r + lc][16 * d + 4 * lu]) =
          (INT8 ? o[r][d] + ow[r] : o[r][d]) * by * back;
    if (lu == 0) {
      jm[wave][16 * r + lc][0] = m[r];
      jm[wave][16 * r + lc][1] = sum;
    }
  }
  __syncthreads();
  const PagedP e = again();
  for (int i = threadIdx.x; i < 16 * RT * (DP / 4); i += 64 * NW) {
    const int r = i / (DP / 4), d = 4 * (i % (DP / 4)), row = rb * 16 * RT + r;
    if (row >= e.G || d >= D) continue;
    float up = jm[0][r][0], sum = 0.f, f[NW];
#pragma unroll
    for (int w = 1; w < NW; ++w) up = fmaxf(up, jm[w][r][0]);
#pragma unroll
    for (int w = 0; w < NW; ++w) sum += f[w] = jm[w][r][1] * exp2_(jm[w][r][0] - up);
    // shares of the sum, not weights: a mean near the type's largest value times a weight leaves fp32
    const float by = sum != 0.f ? 1.0f / sum : 0.f;
    b4f x = (b4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < NW; ++w) x += *reinterpret_cast<const b4f*>(&jo[w][r][d]) * (f[w] * by);
    const size_t at = (size_t)b * e.a.Hq + h * e.G + row;
    if (e.part.splits > 1) {
      const size_t pt = (size_t)sp * ((size_t)a.B * e.a.Hq) + at;
      *reinterpret_cast<b4f*>(e.part.o + pt * DP + d) = x;
      if (d == 0) *reinterpret_cast<float2*>(e.part.ml + 2 * pt) = make_float2(up, sum);
    } else {
      *reinterpret_cast<uint2*>(e.a.o + b * e.a.o_batch + (h * e.G + row) * e.a.o_head + d) =
          make_uint2(narrow2<DT>(x[0], x[1]), narrow2<DT>(x[2], x[3]));
      if (d == 0 && e.a.lse) e.a.lse[at] = sum != 0.f ? (up + __log2f(sum)) * 0.693147181f : -__builtin_inff();
    }
  }
}

// Joins the parts of the rows: DP / 8 lanes hold a row's 8-element pieces, and
// `across` such lane sets (1, 2, .. 16) of a block share the row's parts, two at a time.
// The sets of a wave are joined by exchanges and the waves through LDS (every set's sums
// through LDS in turn: 1.1 us more for 32 parts, 0.9 for 16).
template <int DT, int DP>
__global__ __launch_bounds__(256) void paged_join(PagedP p, int across) {
  const svdq_paged_attention_args& a = p.a;
  constexpr int LPR = DP / 8;
  __shared__ float part[4][LPR][11];   // of a wave: 8 means, maximum, sum of weights; 11: odd stride
  const size_t rows = (size_t)a.B * a.Hq;
  const int set = threadIdx.x / LPR, g = set % across, lane = threadIdx.x % LPR, d = 8 * lane;
  const size_t at = (size_t)blockIdx.x * (256 / LPR / across) + set / across;
  const bool live = at < rows;
  float top = kLow, sum = 0.f, o[8];             // o: the mean so far
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = 0.f;
  // The mean x of weights of sum f under maximum m joins this set's, each times its share
  // of the sum: a mean near the type's largest value times a weight leaves fp32.
  auto add = [&](float m, float f, const float* x) __attribute__((always_inline)) {
    const float up = fmaxf(top, m), mine = sum * exp2_(top - up), other = f * exp2_(m - up);
    top = up;
    sum = mine + other;
    const float by = sum != 0.f ? __builtin_amdgcn_rcpf(sum) : 0.f, b = other * by;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = fmaf(b, x[i], o[i] * (mine * by));
  };
  if (live) {
    for (int s = g; s < p.part.splits; s += 2 * across) {
      float2 ml[2] = {};
      b4f x[2][2] = {};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (k == 1 && p.part.splits <= across) break;   // one part a set
        const size_t pt = min(s + k * across, p.part.splits - 1) * rows + at;
        const float* op = p.part.o + pt * DP + d;
        ml[k] = *reinterpret_cast<const float2*>(p.part.ml + 2 * pt);
        x[k][0] = *reinterpret_cast<const b4f*>(op);
        x[k][1] = *reinterpret_cast<const b4f*>(op + 4);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        // no keys, and nothing stored; or no weights
        if (s + k * across >= p.part.splits || ml[k].y == 0.f) continue;
        const float t[8] = {x[k][0][0], x[k][0][1], x[k][0][2], x[k][0][3], x[k][1][0], x[k][1][1], x[k][1][2], x[k][1][3]};
        add(ml[k].x, ml[k].y, t);
      }
    }
  }
  // the sets of a wave
  if (across > 1) {
    float up = top;
#pragma unroll
    for (int w = LPR; w < 64; w *= 2)
      if (w < across * LPR) up = fmaxf(up, __shfl_xor(up, w));
    const float mine = sum * exp2_(top - up);
    top = up;
    sum = mine;
#pragma unroll
    for (int w = LPR; w < 64; w *= 2)
      if (w < across * LPR) sum += __shfl_xor(sum, w);
    const float share = sum != 0.f ? mine * __builtin_amdgcn_rcpf(sum) : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      o[i] *= share;
#pragma unroll
      for (int w = LPR; w < 64; w *= 2)
        if (w < across * LPR) o[i] += __shfl_xor(o[i], w);
    }
  }
  if (across * LPR > 64) {
    const int wave = threadIdx.x >> 6, waves = across * LPR / 64;
    if ((threadIdx.x & 63) < LPR) {
#pragma unroll
      for (int i = 0; i < 8; ++i) part[wave][lane][i] = o[i];
      part[wave][lane][8] = top;
      part[wave][lane][9] = sum;
    }
    __syncthreads();
    if (g == 0)
      for (int k = 1; k < waves; ++k) add(part[wave + k][lane][8], part[wave + k][lane][9], part[wave + k][lane]);
  }
  if (!live || g != 0 || d >= p.c.D) return;
  const int b = (int)(at / a.Hq), hq = (int)(at % a.Hq);
  *reinterpret_cast<b4i*>(a.o + b * a.o_batch + hq * a.o_head + d) = narrow8<DT>(o);
  if (d == 0 && a.lse) a.lse[at] = sum != 0.f ? (top + __log2f(sum)) * 0.693147181f : -__builtin_inff();
}

int padded_dim(int32_t D) { return D <= 64 ? 64 : 128; }

// The arrangement of a call.  keys: at most so many of a request are visible.
struct PagedPlan {
  int G, rows, share, splits;
};
// Parts of a row of keys by the least time, in ns.  A compute unit brings in what the four
// tiles of a block's step need (heads of 128) in 1490 where few blocks run, 2090 where 128
// do (what it can have under way at a time bounds it, and a second block beside the first
// does not help), or all of them at the rate of the memory.  A batch is priced at 0.7 of
// its table, the mean where lengths lie evenly between two fifths of it and all, as the host does
// not see them (one of equal lengths costs 1.4 times that).  Blocks are as many to a
// compute unit as the fullest has.  Start and end are 4500, 700 more for each block after the first, and the join
// 3900, 100 a part up to 16 and 8 a part.
// (us in 1, 2, 4, 8, 16, 32 parts, 8 K/V heads of 128, INT8: 600 keys 8.3, 10.2, 9.2, the
// same beyond; 4096 keys 25.0, 17.8, 12.6, 10.8, 10.1, 10.2; 16384 88, 49, 28.9, 18.7, 13.9,
// 12.8; 131072 704, 360, 187, 102, 61.6, 53.6, in 48 59.8; 16 requests of up to 16384 in 1,
// 2, 3, 4 97.5, 67.2, 84.1, 70.3; 64 of 1024 19.4, 25.0, 24.9, 32.7; 40 of 4096 58.4, 54.1, 55.5,
// 52.8.  A dearer join costs single long requests, a cheaper one batches of some hundred
// keys: 16 of 1280 11.4 in one part, 12.8 in two.)
PagedPlan plan_of(const svdq_kv_cache& c, int32_t B, int64_t keys, int32_t Hq) {
  PagedPlan p;
  p.G = Hq / c.heads;
  p.rows = p.G <= 16 ? 1 : (p.G + 31) / 32;
  const int64_t blocks = (int64_t)B * c.heads * p.rows;
  const int64_t tile_keys = c.format == SVDQ_KV_VALUES ? 32 : 64, tile_bytes = 128 * padded_dim(c.D) + 512;
  const int64_t tiles = (keys + tile_keys - 1) / tile_keys;
  const int64_t full = 4 * kCus * tile_bytes * (B > 1 ? 7 : 10) / 54000;
  int64_t least = 0, best = 1;
  for (int64_t k = 1; k <= 128 && (k == 1 || (4 * k < tiles + 4 && blocks * (k - 1) < 4 * kCus)); ++k) {
    const int64_t n = blocks * k, each = (n + kCus - 1) / kCus, steps = ((tiles + k - 1) / k + 3) / 4;
    const int64_t alone = 250 + tile_bytes * 71 / 1000 + tile_bytes * (n < 128 ? n : 128) / 3400;
    const int64_t step = n >= kCus ? full : full * n / kCus;
    const int64_t cost = each * (steps * (step > alone ? step : alone) + 700) + 3800 + (k > 1 ? 3900 + 100 * (k < 16 ? k : 16) + 8 * k : 0);
    if (k == 1 || cost < least) {
      least = cost;
      best = k;
    }
  }
  const int64_t share = ((keys + best - 1) / best + 255) / 256 * 256;
  p.share = (int)share;
  p.splits = (int)((keys + share - 1) / share);
  return p;
}
size_t plan_bytes(const PagedPlan& p, int32_t B, int32_t Hq, int32_t D) {
  if (p.splits == 1) return 0;
  const size_t rows = (size_t)B * Hq;
  return align256(p.splits * rows * padded_dim(D) * 4) + align256(p.splits * rows * 8);
}

template <int FMT, int DT, int DP, bool PAD>
svdq_status launch_rows(const PagedP& p, const PagedPlan& pl, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)p.a.B * p.c.heads * pl.rows * pl.splits));
  if (pl.G <= 16) hipLaunchKernelGGL((paged_kernel<FMT, DT, DP, PAD, 1>), grid, dim3(256), 0, st, p);
  else hipLaunchKernelGGL((paged_kernel<FMT, DT, DP, PAD, 2>), grid, dim3(256), 0, st, p);
  svdq_status s = launched();
  if (s == SVDQ_OK && pl.splits > 1) {
    int across = 1;
    while (across < 16 && across < pl.splits) across *= 2;
    const int per = 256 / (DP / 8) / across;
    const size_t rows = (size_t)p.a.B * p.a.Hq;
    hipLaunchKernelGGL((paged_join<DT, DP>), dim3((unsigned)((rows + per - 1) / per)), dim3(256), 0, st, p, across);
    s = launched();
  }
  return s;
}
template <int FMT, int DT>
svdq_status launch_dim(const PagedP& p, const PagedPlan& pl, hipStream_t st) {
  if (p.c.D == 128) return launch_rows<FMT, DT, 128, false>(p, pl, st);
  if (p.c.D > 64) return launch_rows<FMT, DT, 128, true>(p, pl, st);
  if (p.c.D == 64) return launch_rows<FMT, DT, 64, false>(p, pl, st);
  return launch_rows<FMT, DT, 64, true>(p, pl, st);
}
template <int FMT>
svdq_status launch_type(const PagedP& p, const PagedPlan& pl, hipStream_t st) {
  return p.a.dtype == SVDQ_BF16 ? launch_dim<FMT, SVDQ_BF16>(p, pl, st) : launch_dim<FMT, SVDQ_FP16>(p, pl, st);
}

bool sizes_fit(const svdq_kv_cache& c, int32_t B, int32_t T, int32_t Hq) {
  return B >= 1 && T >= 1 && (int64_t)T * c.page <= (1 << 24) && Hq >= 1 && Hq <= 65536 && Hq % c.heads == 0 &&
         (int64_t)B * Hq < (1 << 24);
}

}  // namespace
}  // namespace svdq

using namespace svdq;

extern "C" size_t svdq_paged_attention_workspace_bytes(const svdq_kv_cache* cache, int32_t B, int32_t T, int32_t Hq) {
  if (!cache || cache_sizes(*cache) != SVDQ_OK || !sizes_fit(*cache, B, T, Hq)) return 0;
  return plan_bytes(plan_of(*cache, B, (int64_t)T * cache->page, Hq), B, Hq, cache->D);
}

extern "C" svdq_status svdq_paged_attention(const svdq_kv_cache* cache, const svdq_paged_attention_args* a, void* ws,
                                            size_t ws_bytes, void* stream) {
  if (!cache || !a || !a->q || !a->o || !a->table || !a->kv_len) return SVDQ_ERR_ARG;
  svdq_status s = cache_check(*cache);
  if (s != SVDQ_OK) return s;
  if (!is_dtype(a->dtype)) return SVDQ_ERR_UNSUPPORTED;
  if (!sizes_fit(*cache, a->B, a->T, a->Hq) || (a->B > 1 && a->table_row < a->T)) return SVDQ_ERR_SHAPE;
  const float big = 3.0e38f;
  if (!(a->scale >= -big && a->scale <= big) || !(a->softcap >= 0.f && a->softcap <= big) || a->window < 0)
    return SVDQ_ERR_ARG;
  for (int64_t st : {a->q_batch, a->q_head, a->o_batch, a->o_head})
    if (st % 8 != 0) return SVDQ_ERR_ALIGN;
  if (!on16(a->q) || !on16(a->o) || !on4(a->table) || !on4(a->kv_len) || !on4(a->slopes) || !on4(a->lse))
    return SVDQ_ERR_ALIGN;
  const int64_t all = (int64_t)a->T * cache->page;
  // a window starts inside a tile: up to 63 keys before it are passed over
  const int64_t near = (int64_t)a->window + 63, keys = a->window > 0 && near < all ? near : all;
  PagedPlan pl = plan_of(*cache, a->B, keys, a->Hq);
  // the workspace is asked for without the window: no more parts than without it
  const PagedPlan whole = plan_of(*cache, a->B, all, a->Hq);
  if (pl.splits > whole.splits) pl = whole;
  const size_t need = plan_bytes(pl, a->B, a->Hq, cache->D);
  if (need > 0 && (!ws || ws_bytes < need)) return !ws ? SVDQ_ERR_ARG : SVDQ_ERR_WORKSPACE;
  if (((uintptr_t)ws & 255u) != 0) return SVDQ_ERR_ALIGN;
  if ((s = device_ok()) != SVDQ_OK) return s;
  PagedP p;
  p.a = *a;
  p.c = *cache;
  if (a->B == 1) p.a.table_row = 0;
  p.G = pl.G;
  p.rows = pl.rows;
  p.shift = __builtin_ctz(cache->page);
  // x / d is the upper half of x ceil(2^32 / d) as long as x d < 2^32; x < 2^24
  auto over = [](uint32_t d, uint64_t most) -> uint32_t {
    return d > 1 && most * d < (1ull << 32) ? (uint32_t)(((1ull << 32) + d - 1) / d) : 0;
  };
  const uint64_t groups = (uint64_t)a->B * cache->heads;
  p.by_splits = over(pl.splits, groups * pl.rows * pl.splits);
  p.by_heads = over(cache->heads, groups);
  set_score(&p, a->scale, a->softcap);
  p.part.share = pl.share;
  p.part.splits = pl.splits;
  p.part.o = static_cast<float*>(ws);
  p.part.ml = pl.splits > 1 ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) +
                                                       align256((size_t)pl.splits * a->B * a->Hq * padded_dim(cache->D) * 4))
                            : nullptr;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (cache->format == SVDQ_KV_INT8) return launch_type<SVDQ_KV_INT8>(p, pl, st);
  if (cache->format == SVDQ_KV_FP8) return launch_type<SVDQ_KV_FP8>(p, pl, st);
  return launch_type<SVDQ_KV_VALUES>(p, pl, st);
}
