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

// ------------------------------------------------------------ LDS tiles
//
// A block computes BM tokens x BN out-features; WM x WN waves own MT x NT MFMA
// tiles each, and WK such groups of waves take the steps of 128 k in turn
// (joined in LDS at the end).  Codes and token scales of the next step go to
// LDS by direct copies (1 KB: 8 rows x 128 codes), two buffers, one barrier a
// step.
// Chunk c of a row sits at slot c ^ f(row) with f such that the 16 lanes
// served together in a fragment read hit distinct 16-byte slots.
//
// The block sums of a pair of weight tiles are scaled while the MFMAs of the
// next pair run (two sets of them), and the token codes of the next tile are
// read ahead.  Two waves a SIMD hide most of the widening and scaling behind
// the other's MFMAs.  4096 x 3072 -> 9216 in 128 x 128 tiles, two blocks a
// compute unit: 203 us, 1.14 PFLOP/s (a large bf16 product of the vendor's
// library: 1.21).  When it took 214 us, timing it without the copies gave 180 us,
// without the widening 203 us.

template <int NT, int MT, int WN, int WM, int WK>
struct Tile {
  static constexpr int WAVES = WN * WM, BN = 16 * NT * WN, BM = 16 * MT * WM;
  static constexpr int CODES = (BN + BM) * 128;             // of a step
  static constexpr int STEP = CODES + WAVES * 256;          // and 64 token scales per wave
  static constexpr int UNITS = (BN + BM) / 8 / WAVES;       // code copies per wave and step
  static constexpr int JOIN = WK > 1 ? (WK - 1) * BN * BM * 4 : 0;
  static constexpr int LDS = 2 * WK * STEP > JOIN ? 2 * WK * STEP : JOIN;
};

// Long k and few tiles: a 128 x 128 tile moves half the bytes per product of a
// 64 x 64 one, but 333 x 12288 -> 3072 has 72 of them.  SPLIT: `parts` blocks share a tile's steps and leave their sums in `sums`, as
// [part][tile][wave][nt][mt][lane], for fp8_join_kernel.
template <int DT, int NT, int MT, int WN, int WM, int WK, bool SPLIT>
__global__ __launch_bounds__(64 * WN * WM * WK, 2) void fp8_tile_kernel(
    const uint8_t* __restrict__ xq, const float* __restrict__ xs, const uint8_t* __restrict__ wq,
    const float* __restrict__ ws, const uint16_t* __restrict__ bias, int M, int K, int N, uint16_t* __restrict__ Y,
    int tiles_m, int tiles_n, int parts, b4f* __restrict__ sums) {
  static_assert(!SPLIT || WK == 1, "blocks or groups share the steps");
  using T = Tile<NT, MT, WN, WM, WK>;
  constexpr int UNITS = T::UNITS;
  static_assert(MT <= 4 && NT % 2 == 0, "64 token scales per wave, pairs of weight tiles");
  __shared__ __attribute__((aligned(1024))) uint8_t lds_all[T::LDS];
  __shared__ float swl[512];                               // K <= 65536
  static_assert(128 % T::BN == 0, "one block of weight scales");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave_all = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wk = wave_all / T::WAVES, wave = wave_all % T::WAVES;
  const int wm = wave % WM, wn = wave / WM;
  const int l16 = lane & 15, g = lane >> 4;
  // work ids run through groups of 8 token tiles, out-feature tile slower: the
  // blocks that an XCD holds at a time share their operand panels in its L2
  int id = xcd_order(blockIdx.x, tiles_m * tiles_n * (SPLIT ? parts : 1)), part = 0;
  const int place = id;
  if constexpr (SPLIT) {
    part = id / (tiles_m * tiles_n);
    id -= part * (tiles_m * tiles_n);
  }
  const int span = 8 * tiles_n, grp = id / span, in = id % span;
  const int high = min(8, tiles_m - 8 * grp);
  const int m0 = (8 * grp + in % high) * T::BM, n0 = (in / high) * T::BN;
  const int steps = K >> 7;
  // steps wk, wk + WK, ..., or the part's
  const int first = SPLIT ? part * steps / parts : wk;
  const int mine = SPLIT ? (part + 1) * steps / parts - first : (steps - wk + WK - 1) / WK;
  const int turns = SPLIT ? mine : (steps + WK - 1) / WK;
  uint8_t* lds = lds_all + wk * 2 * T::STEP;

  // ---- copies: units of 8 rows, weights first.  N % 16 == 0, so a unit of
  // weight rows is whole or past the end (then the last one is repeated);
  // token rows past M repeat the last row, lane by lane.
  const int u0 = wave * UNITS;
  const int r8 = lane >> 3, slot = lane & 7;
  const uint8_t* wbase = wq + (size_t)n0 * K;
  const uint8_t* tbase = xq + (size_t)m0 * K;
  uint32_t voff[UNITS];
#pragma unroll
  for (int j = 0; j < UNITS; ++j) {
    const int u = u0 + j, ut = u - T::BN / 8;
    const bool wside = u < T::BN / 8;
    const int row = wside ? min(u, (N - n0) / 8 - 1) * 8 + r8 : min(8 * ut + r8, M - 1 - m0);
    const int f = wside ? 2 * (u & 3) + ((r8 >> 1) & 1) : 4 * (ut & 1) + (r8 >> 1);
    voff[j] = (uint32_t)row * (uint32_t)K + 16u * (slot ^ f);
  }
  const uint32_t lds0 = lds_address(lds);
  // scales: lane l the wave's token l (its 16 MT; the others repeat one)
  const int m_wave = m0 + 16 * MT * wm;
  const uint8_t* sbase = reinterpret_cast<const uint8_t*>(xs + (size_t)min(m_wave, M - 1) * steps);
  const uint32_t svoff = (uint32_t)max(min(lane < 16 * MT ? lane : 0, M - 1 - m_wave), 0) * (uint32_t)steps * 4u;
  auto copy = [&](int v) __attribute__((always_inline)) {   // the v-th of this group's steps
    const int t = v * WK + first;
    const uint32_t dst = lds0 + (v & 1) * T::STEP + u0 * 1024;
    const uint8_t *wt = wbase + (size_t)t * 128, *tt = tbase + (size_t)t * 128;
#pragma unroll
    for (int j = 0; j < UNITS; ++j) dma_16(u0 + j < T::BN / 8 ? wt : tt, voff[j], dst + 1024 * j);
    dma_4(sbase + (size_t)t * 4, svoff, lds0 + (v & 1) * T::STEP + T::CODES + 256 * wave);
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
  const int nb = n0 >> 7;                                   // the block's out-features share a scale block
  if (mine > 0) copy(0);
  // the weight scales of all steps; the first barrier below makes them visible
  for (int i = tid; i < steps; i += 64 * T::WAVES * WK) swl[i] = ws[(size_t)nb * steps + i];
  for (int v = 0; v < turns; ++v) {
    dma_wait();
    __syncthreads();
    if (v + 1 < mine) copy(v + 1);
    if (WK > 1 && v >= mine) break;                         // the last turn of a group with one step less
    const float sw = swl[v * WK + first];
    const uint8_t* buf = lds + (v & 1) * T::STEP;
    const float* sx = reinterpret_cast<const float*>(buf + T::CODES + 256 * wave);
    b4i blo, bhi;
    auto read_b = [&](int mt) __attribute__((always_inline)) {
      blo = *reinterpret_cast<const b4i*>(buf + boff[mt & 1] + (mt >> 1) * 32 * 128);
      bhi = *reinterpret_cast<const b4i*>(buf + (boff[mt & 1] ^ 64) + (mt >> 1) * 32 * 128);
    };
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
    read_b(0);
    constexpr int NP = NT / 2;
    b4f p[2][2];
    float s_old = 0.f;
    auto scale_pair = [&](int set, int mt, int pr, float s) __attribute__((always_inline)) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[2 * pr + h][mt][i] = fmaf(p[set][h][i], s, acc[2 * pr + h][mt][i]);
    };
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const float s = sx[16 * mt + l16] * sw;
      b8bf b[4];
      b[0] = widen_codes(blo[0], blo[1]);
      b[1] = widen_codes(blo[2], blo[3]);
      b[2] = widen_codes(bhi[0], bhi[1]);
      b[3] = widen_codes(bhi[2], bhi[3]);
      if (mt + 1 < MT) read_b(mt + 1);
#pragma unroll
      for (int pr = 0; pr < NP; ++pr) {
        const int set = (mt * NP + pr) & 1;
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            p[set][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[2 * pr + h][x], b[x],
                                                                x ? p[set][h] : (b4f){0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
        if (pr > 0) scale_pair(set ^ 1, mt, pr - 1, s);
        else if (mt > 0) scale_pair(set ^ 1, mt - 1, NP - 1, s_old);
      }
      s_old = s;
    }
    scale_pair((MT * NP - 1) & 1, MT - 1, NP - 1, s_old);
  }

  if constexpr (WK > 1) {
    // groups 1.. hand their sums to group 0, each wave to the wave of its place
    __syncthreads();
    b4f* j = reinterpret_cast<b4f*>(lds_all);               // [group][wave][nt][mt][lane]
    if (wk > 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          j[((((wk - 1) * T::WAVES + wave) * NT + nt) * MT + mt) * 64 + lane] = acc[nt][mt];
    }
    __syncthreads();
    if (wk > 0) return;
#pragma unroll
    for (int k = 0; k < WK - 1; ++k)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) acc[nt][mt] += j[(((k * T::WAVES + wave) * NT + nt) * MT + mt) * 64 + lane];
  }

  if constexpr (SPLIT) {
    b4f* out = sums + ((size_t)place * T::WAVES + wave) * NT * MT * 64 + lane;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) out[(nt * MT + mt) * 64] = acc[nt][mt];
    return;
  }

#pragma unroll
  for (int pr = 0; pr < NT / 2; ++pr) {
    const int n = n0 + 16 * NT * wn + 32 * pr + 8 * g;
    if (n >= N) continue;
    float bv[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) bv[i] = 0.f;
    add_bias8<DT>(bias, n, bv);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int m = m_wave + 16 * mt + l16;
      if (m >= M) continue;
      float v[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = acc[2 * pr][mt][i] + bv[i];
        v[4 + i] = acc[2 * pr + 1][mt][i] + bv[4 + i];
      }
      *reinterpret_cast<b4i*>(Y + (size_t)m * N + n) = narrow8<DT>(v);
    }
  }
}

// Adds the parts of a tile in their order.  A block takes one (pair of weight
// tiles, token tile) of all waves of a tile; lanes hold what they held there.
template <int DT, int NT, int MT, int WN, int WM>
__global__ __launch_bounds__(64 * WN * WM) void fp8_join_kernel(const b4f* __restrict__ sums,
                                                                const uint16_t* __restrict__ bias, int M, int N,
                                                                uint16_t* __restrict__ Y, int tiles_m, int tiles_n,
                                                                int parts) {
  using T = Tile<NT, MT, WN, WM, 1>;
  constexpr int PIECES = NT / 2 * MT;
  const int id = blockIdx.x / PIECES, piece = blockIdx.x % PIECES, pr = piece / MT, mt = piece % MT;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave % WM, wn = wave / WM;
  const int span = 8 * tiles_n, grp = id / span, in = id % span;
  const int high = min(8, tiles_m - 8 * grp);
  const int m = (8 * grp + in % high) * T::BM + 16 * MT * wm + 16 * mt + (lane & 15);
  const int n = (in / high) * T::BN + 16 * NT * wn + 32 * pr + 8 * (lane >> 4);
  if (m >= M || n >= N) return;
  const b4f* at = sums + (((size_t)id * T::WAVES + wave) * NT * MT + (2 * pr) * MT + mt) * 64 + lane;
  const size_t next = (size_t)tiles_m * tiles_n * T::WAVES * NT * MT * 64;
  b4f lo = at[0], hi = at[MT * 64];
#pragma unroll 4
  for (int p = 1; p < parts; ++p) {
    at += next;
    lo += at[0];
    hi += at[MT * 64];
  }
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = lo[i];
    v[4 + i] = hi[i];
  }
  add_bias8<DT>(bias, n, v);
  *reinterpret_cast<b4i*>(Y + (size_t)m * N + n) = narrow8<DT>(v);
}

// ------------------------------------------------------------ few tokens
//
// At most 16 tokens a block, so the weights' bytes bound it (16 x 3072 ->
// 9216: 12.5 us, 2.3 TB/s; token rows cost as many line accesses as weight
// rows).  A block owns 16 out-features; its 8 waves take steps of 128 k in turn
// straight from memory to registers (a row's step is one whole line) and are
// joined in LDS.

template <int DT>
__global__ __launch_bounds__(512) void fp8_few_kernel(const uint8_t* __restrict__ xq, const float* __restrict__ xs,
                                                      const uint8_t* __restrict__ wq, const float* __restrict__ ws,
                                                      const uint16_t* __restrict__ bias, int M, int K, int N,
                                                      uint16_t* __restrict__ Y) {
  constexpr int WV = 8;
  __shared__ float red[WV][16][17];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16, steps = K >> 7;
  const int m = min(m0 + l16, M - 1);
  const uint8_t* ap = wq + (size_t)(n0 + l16) * K + 16 * g;
  const uint8_t* bp = xq + (size_t)m * K + 16 * g;
  const float* sx = xs + (size_t)m * steps;
  const float* sw = ws + (size_t)(n0 >> 7) * steps;
  b4f acc = (b4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int t = wave; t < steps; t += WV) {
    const b4i alo = *reinterpret_cast<const b4i*>(ap + 128 * (size_t)t);
    const b4i ahi = *reinterpret_cast<const b4i*>(ap + 128 * (size_t)t + 64);
    const b4i blo = *reinterpret_cast<const b4i*>(bp + 128 * (size_t)t);
    const b4i bhi = *reinterpret_cast<const b4i*>(bp + 128 * (size_t)t + 64);
    const float s = sx[t] * sw[t];
    b4f p = (b4f){0.f, 0.f, 0.f, 0.f};
    p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_codes(alo[0], alo[1]), widen_codes(blo[0], blo[1]), p, 0, 0, 0);
    p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_codes(alo[2], alo[3]), widen_codes(blo[2], blo[3]), p, 0, 0, 0);
    p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_codes(ahi[0], ahi[1]), widen_codes(bhi[0], bhi[1]), p, 0, 0, 0);
    p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_codes(ahi[2], ahi[3]), widen_codes(bhi[2], bhi[3]), p, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(p[i], s, acc[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) red[wave][l16][4 * g + i] = acc[i];
  __syncthreads();
  if (threadIdx.x < 256) {
    const int r = threadIdx.x >> 4, c = threadIdx.x & 15;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < WV; ++w) v += red[w][r][c];
    if (m0 + r < M) {
      if (bias) v += widen2<DT>(bias[n0 + c])[0];
      Y[(size_t)(m0 + r) * N + n0 + c] = (uint16_t)narrow2<DT>(v, 0.f);
    }
  }
}

// ------------------------------------------------------------- one token
//
// No matrix unit: a wave reads RW weight rows 1 KB at a time (whole lines, 16
// codes a lane), multiplies them with the token's codes of the same places and
// keeps one fp32 sum per row and lane; a lane's codes of a kilobyte lie in one
// scale block.  The lanes are added at the end.  3072 -> 9216: 7.0 - 7.4 us, 3.8 -
// 4.1 TB/s.

template <int DT, int RW>
__global__ __launch_bounds__(256) void fp8_row_kernel(const uint8_t* __restrict__ xq, const float* __restrict__ xs,
                                                      const uint8_t* __restrict__ wq, const float* __restrict__ ws,
                                                      const uint16_t* __restrict__ bias, int K, int N,
                                                      uint16_t* __restrict__ Y) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = (blockIdx.x * 4 + wave) * RW, steps = K >> 7;
  if (n0 >= N) return;
  const uint8_t* wp = wq + (size_t)n0 * K;
  const float* sw = ws + (size_t)(n0 >> 7) * steps;
  float acc[RW];
#pragma unroll
  for (int r = 0; r < RW; ++r) acc[r] = 0.f;
#pragma unroll 4
  for (int k = 16 * lane; k < K; k += 1024) {
    b4i w[RW];
#pragma unroll
    for (int r = 0; r < RW; ++r) w[r] = *reinterpret_cast<const b4i*>(wp + (size_t)r * K + k);
    const b4i c = *reinterpret_cast<const b4i*>(xq + k);
    const float s = xs[k >> 7] * sw[k >> 7];
    float x[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const b2f lo = __builtin_amdgcn_cvt_pk_f32_fp8(c[i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(c[i], true);
      x[4 * i] = lo[0] * s;
      x[4 * i + 1] = lo[1] * s;
      x[4 * i + 2] = hi[0] * s;
      x[4 * i + 3] = hi[1] * s;
    }
#pragma unroll
    for (int r = 0; r < RW; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const b2f lo = __builtin_amdgcn_cvt_pk_f32_fp8(w[r][i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w[r][i], true);
        acc[r] = fmaf(lo[0], x[4 * i], acc[r]);
        acc[r] = fmaf(lo[1], x[4 * i + 1], acc[r]);
        acc[r] = fmaf(hi[0], x[4 * i + 2], acc[r]);
        acc[r] = fmaf(hi[1], x[4 * i + 3], acc[r]);
      }
  }
#pragma unroll
  for (int r = 0; r < RW; ++r) {
#pragma unroll
    for (int d = 32; d; d >>= 1) acc[r] += __shfl_xor(acc[r], d);
    if (lane == 0) {
      const float v = acc[r] + (bias ? widen2<DT>(bias[n0 + r])[0] : 0.f);
      Y[n0 + r] = (uint16_t)narrow2<DT>(v, 0.f);
    }
  }
}

// In how many parts the steps of a 128 x 128 tile are taken by blocks of their
// own, given memory for their sums: as many as the chip holds (two blocks a
// compute unit), where k is long enough to pay for the sums' way through
// memory and the second launch.  Measured, us (without -> with):
//   K      100 x 3072    200 x 3072    333 x 3072    512 x 3072    512 x 4096
//   6144   15 -> 19      20 -> 23      31 -> 26      32 -> 32      35 -> 36
//   8192   19 -> 19      25 -> 25      39 -> 31      40 -> 36      44 -> 43
//   12288  27 -> 22      35 -> 30      59 -> 39      61 -> 47      68 -> 57
//   16384  31 -> 25      44 -> 35      74 -> 46      76 -> 58      90 -> 76
// (M x N in the head.)  16 tiles lose at any K (100 x 16384 -> 2048 20 -> 25),
// and so do few tokens (64 x 12288 -> 3072 17.5 -> 21.7),
// and two parts (700 x 12288 -> 4096, 192 tiles: 79 -> 88).  The last condition of
// the rule is a line drawn between the shapes that lose and win above.
int64_t fp8_tiles(int M, int N) { return (int64_t)((M + 127) / 128) * ((N + 127) / 128); }
int fp8_parts(int M, int K, int N) {
  const int64_t tiles = fp8_tiles(M, N), steps = K / 128;
  if (M <= 64 || steps < 64 || tiles < 24 || tiles > 2 * kCus / 3 || 2 * tiles + 3 * steps < 336) return 1;
  return (int)(2 * kCus / tiles);                            // at most 21
}

template <int DT>
svdq_status launch_split(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws, const uint16_t* bias,
                         int M, int K, int N, uint16_t* Y, b4f* sums, hipStream_t st) {
  const int tm = (M + 127) / 128, tn = (N + 127) / 128, parts = fp8_parts(M, K, N);
  hipLaunchKernelGGL((fp8_tile_kernel<DT, 4, 4, 2, 2, 1, true>), dim3(tm * tn * parts), dim3(256), 0, st, xq, xs, wq,
                     ws, nullptr, M, K, N, nullptr, tm, tn, parts, sums);
  hipLaunchKernelGGL((fp8_join_kernel<DT, 4, 4, 2, 2>), dim3(tm * tn * 8), dim3(256), 0, st, sums, bias, M, N, Y, tm,
                     tn, parts);
  return launched();
}

bool fp8_sizes(int32_t M, int32_t K, int32_t N) {
  return valid_kn(K, N) && M >= 1 && M <= (1 << 20) && (int64_t)M * K <= (int64_t)1 << 32 &&
         (int64_t)N * K <= (int64_t)1 << 32;
}

// The variant of a call, by its sizes.  Tiles are taken as large as the chip
// can still be filled with: in one round with a block a compute unit (256),
// whose groups of waves take the steps of k in turn, or with two.  A larger
// tile moves fewer bytes per product, but a second round that is mostly empty
// costs more.  Measured, us (tokens x out-features of a tile / groups):
//   M x K x N          row   few   32/8  64x32/4  64/4   64/2   128/1
//   1 x 3072 x 9216    7.2   8.3   11    15       11     11     28
//   16 x 3072 x 9216         12.4  12.4  15       11     12     28
//   64 x 1024 x 1024         3.1   3.8   4.5      5.8    5.4    11
//   64 x 12288 x 3072        42    18    27       37     42     100
//   128 x 12288 x 3072       80    32    27       35     41     101
//   64 x 3072 x 9216         32    17    17       12.3   13.3   28
//   256 x 3072 x 3072        41    17    16       11.9   12.9   28
//
//   M x K x N           64/4   64/2   96x128/2  128/2  96x128/1  128/1
//   512 x 4096 x 4096   26.3   23.7   28.1      32.7   32.0      37.2
//   200 x 3072 x 9216   29.9   25.5   22.1      25.8   24.6      28.6
//   900 x 3072 x 3072   30.8   27.4   23.5      26.8   25.7      29.8
//   1024 x 3072 x 3072  31.0   27.6   42.4      26.5   36.9      29.4
//   1024 x 4096 x 4096  50.0   44.9   52.0      36.3   46.7      39.1
//   1500 x 3072 x 3072  48.6   41.0   41.0      50.6   37.5      43.7
//   512 x 3072 x 9216   48.5   40.8   41.3      49.9   38.5      43.3
//   1024 x 3072 x 9216  87.1   75.9   80.5      73.9   71.4      67.1
//   2048 x 3072 x 9216  170    141    139       124    124       112
//   4096 x 3072 x 9216         297                               203
// (At 16 x 3072 x 9216 64/4 is a tenth faster than few, which the rule takes for
// all of 2 to 16 tokens: 12.4 us, and 11.4 with 17 tokens.)
template <int DT>
svdq_status launch_fp8(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws, const uint16_t* bias,
                       int M, int K, int N, uint16_t* Y, hipStream_t st) {
  using std::integral_constant;
  typedef integral_constant<int, 1> I1;
  typedef integral_constant<int, 2> I2;
  typedef integral_constant<int, 3> I3;
  typedef integral_constant<int, 4> I4;
  typedef integral_constant<int, 8> I8;
  auto blocks = [&](int bm, int bn) { return (int64_t)((M + bm - 1) / bm) * ((N + bn - 1) / bn); };
  auto row = [&](auto rw) {
    constexpr int RW = decltype(rw)::value;
    hipLaunchKernelGGL((fp8_row_kernel<DT, RW>), dim3((N / RW + 3) / 4), dim3(256), 0, st, xq, xs, wq, ws, bias, K, N, Y);
  };
  auto tile = [&](auto nt, auto mt, auto wn, auto wm, auto wk) {   // two buffers per group
    constexpr int NT = decltype(nt)::value, MT = decltype(mt)::value, WN = decltype(wn)::value,
                  WM = decltype(wm)::value, WK = decltype(wk)::value;
    using T = Tile<NT, MT, WN, WM, WK>;
    const int tm = (M + T::BM - 1) / T::BM, tn = (N + T::BN - 1) / T::BN;
    hipLaunchKernelGGL((fp8_tile_kernel<DT, NT, MT, WN, WM, WK, false>), dim3(tm * tn), dim3(64 * T::WAVES * WK), 0, st,
                       xq, xs, wq, ws, bias, M, K, N, Y, tm, tn, 1, nullptr);
  };
  if (M == 1) {
    // two rows against one, us: 5120 -> 13824 13.2 / 13.6, 3072 -> 9216 7.1 / 7.5,
    // 3072 -> 5120 5.0 / 4.9, 8192 -> 4096 8.9 / 8.3, 3072 -> 2048 3.2 / 3.0
    // (12288 -> 3072 the other way, 8.8 / 9.2)
    if (N >= 6144) row(I2{});
    else row(I1{});
  } else if (M <= 16 || blocks(16, 16) <= 256) {
    hipLaunchKernelGGL((fp8_few_kernel<DT>), dim3(N / 16, (M + 15) / 16), dim3(512), 0, st, xq, xs, wq, ws, bias, M, K,
                       N, Y);
  } else if (blocks(32, 32) <= 256) {
    tile(I2{}, I2{}, I1{}, I1{}, I8{});
  } else if (blocks(64, 32) <= 256) {
    tile(I2{}, I2{}, I1{}, I2{}, I4{});
  } else if (blocks(64, 64) <= 256) {
    tile(I2{}, I2{}, I2{}, I2{}, I4{});
  } else if (blocks(64, 64) <= 512) {
    tile(I2{}, I2{}, I2{}, I2{}, I2{});
  } else if (blocks(96, 128) <= 256) {
    tile(I4{}, I3{}, I2{}, I2{}, I2{});
  } else if (blocks(128, 128) <= 256) {
    tile(I4{}, I4{}, I2{}, I2{}, I2{});
  } else if (blocks(96, 128) <= 512) {
    tile(I4{}, I3{}, I2{}, I2{}, I1{});
  } else {
    tile(I4{}, I4{}, I2{}, I2{}, I1{});
  }
  return launched();
}

}  // namespace
}  // namespace svdq

using namespace svdq;

namespace {

svdq_status fp8_check(const void* xq, const void* xs, const void* wq, const void* ws, const void* bias, int32_t M,
                      int32_t K, int32_t N, int32_t dtype, const void* Y) {
  if (!xq || !xs || !wq || !ws || !Y) return SVDQ_ERR_ARG;
  if (!is_dtype(dtype)) return SVDQ_ERR_UNSUPPORTED;
  if (!fp8_sizes(M, K, N)) return SVDQ_ERR_SHAPE;
  if (!on16(xq) || !on16(wq) || !on16(bias) || !on16(Y) || !on4(xs) || !on4(ws)) return SVDQ_ERR_ALIGN;
  return SVDQ_OK;
}

}  // namespace

extern "C" svdq_status svdq_fp8_linear(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                                       const uint16_t* bias, int32_t M, int32_t K, int32_t N, int32_t dtype,
                                       uint16_t* Y, void* stream) {
  svdq_status ok = fp8_check(xq, xs, wq, ws, bias, M, K, N, dtype, Y);
  if (ok == SVDQ_OK) ok = device_ok();
  if (ok != SVDQ_OK) return ok;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return dtype == SVDQ_BF16 ? launch_fp8<SVDQ_BF16>(xq, xs, wq, ws, bias, M, K, N, Y, st)
                            : launch_fp8<SVDQ_FP16>(xq, xs, wq, ws, bias, M, K, N, Y, st);
}

extern "C" size_t svdq_fp8_linear_workspace_bytes(int32_t M, int32_t K, int32_t N) {
  if (!fp8_sizes(M, K, N)) return 0;
  const int parts = fp8_parts(M, K, N);
  return parts > 1 ? (size_t)parts * fp8_tiles(M, N) * 128 * 128 * sizeof(float) : 0;
}

extern "C" svdq_status svdq_fp8_linear_shared(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                                              const uint16_t* bias, int32_t M, int32_t K, int32_t N, int32_t dtype,
                                              uint16_t* Y, void* workspace, size_t workspace_bytes, void* stream) {
  const size_t need = svdq_fp8_linear_workspace_bytes(M, K, N);
  if (need == 0) return svdq_fp8_linear(xq, xs, wq, ws, bias, M, K, N, dtype, Y, stream);
  svdq_status ok = fp8_check(xq, xs, wq, ws, bias, M, K, N, dtype, Y);
  if (ok != SVDQ_OK) return ok;
  if (!workspace) return SVDQ_ERR_ARG;
  if (workspace_bytes < need) return SVDQ_ERR_WORKSPACE;
  if (!on16(workspace)) return SVDQ_ERR_ALIGN;
  ok = device_ok();
  if (ok != SVDQ_OK) return ok;
  hipStream_t st = static_cast<hipStream_t>(stream);
  b4f* sums = static_cast<b4f*>(workspace);
  return dtype == SVDQ_BF16 ? launch_split<SVDQ_BF16>(xq, xs, wq, ws, bias, M, K, N, Y, sums, st)
                            : launch_split<SVDQ_FP16>(xq, xs, wq, ws, bias, M, K, N, Y, sums, st);
}
