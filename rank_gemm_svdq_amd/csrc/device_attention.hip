// Attention over visible keys, with shared K/V heads, score cap, distance
// bias, document numbers, a prefix and lengths: one pass over K and V with the
// running maximum and sum of the softmax, scores never leave registers.
//
// Rows.  The queries of all heads that share a K/V head are rows of one
// matrix: row r is query r / G of head hk G + r % G (G heads share).  A wave
// owns 32 rows, so one pass over K and V serves all G heads.
//
// One tile of 32 keys, per wave (32x32x16 MFMA; lane l: column l % 32,
// l / 32 = half):
//   S^T = K Q^T   A = 32 keys (LDS), B = the wave's rows (registers).  Lane l
//                 gets row l % 32, keys 8 (i / 4) + 4 half + i % 4 in register i.
//   softmax       a row's 32 scores sit in two lanes (l, l + 32): its maximum
//                 is a register reduction and one half exchange.
//   O^T += V^T P  the order of the keys inside an MFMA is free as long as both
//                 operands agree, and with keys 16 s + 4 half + {0..3, 8..11}
//                 in the 8 slots of a lane, registers 8 s' .. + 8 of S are the
//                 B operand as they stand, rounded to 16 bits: P does not
//                 cross lanes.  A comes from V as it lies in memory by
//                 transposing LDS reads (4 keys x 16 columns a read).
// K and V tiles go to LDS by direct copies.  16-byte chunks of a K row are
// XORed with row bits and 64-byte chunks of a V row likewise, so that the
// reads above hit all banks evenly (k_chunk, v_chunk).
//
// The maximum is raised only when a tile's exceeds it by more than 8 (in
// powers of two): the weights stay below 2^8 and the rescaling of O is rare.
//
// Two arrangements.  Many rows: the four waves of a block take 128 rows and
// share tiles of 64 keys.  Few rows (a few new tokens, short prompts): the waves
// share 32 rows and take tiles of 32 keys in turn, each with its own buffers
// and no barriers, and are joined at the end.  Where blocks are few,
// the keys are split over blocks too; a second kernel joins the parts.
//
// What bounds it.  Many rows: power and the serial chain of a wave's tile
// (scores 700 cycles, maximum 440, weights 740, values 800 and 560 for the
// barrier and the copies, two waves a SIMD, at 1.6 - 1.8 GHz under this load):
// 4608 tokens x 24 heads of 128: 287 - 300 us, 870 - 910 TFLOP/s; causal 153 us.  64 rows a
// wave with the two row tiles' softmax and MFMAs side by side (one wave a
// SIMD) took 525 us, eight waves sharing the copies half a tile apart 345 us.
// Heads of 64 have half the MFMAs of heads of 128 for the same softmax and are
// bound by its instructions: 5173 tokens x 24 heads of 64 218 us, 760 TFLOP/s, of
// 128 357 us, 920.
// One token: the bytes of K and V; 16 requests of 4096 - 16384 keys x 8 heads
// 130 - 136 us, 5.0 TB/s.
//
// Hidden keys.  A hidden score is -infinity, its weight 0, and 0 times what V
// holds there would be NaN if that is not finite.  O is checked at the end of a
// block's tiles: where a row with a finite sum of weights came out not finite, the
// block goes over its tiles once more (AGAIN), and each tile's values that are not
// finite are taken out of LDS and kept as marks of the rows that see them;
// everything else is worked out as before, so hidden values do not change a bit of
// the result.  A sum of weights that is not finite needs no second pass: hidden
// scores do not enter it, so the row is NaN.  (2048 tokens, all visible, 8 heads of
// 128 46 us, with one NaN in V 83, with nothing else in it 1.7 ms.)

#include "device_score.h"

namespace svdq {
namespace {

constexpr int kSeen = 2048;  // tiles of a block looked through for their documents

struct Part {               // how the keys are split over blocks
  int32_t splits;
  float* o;                 // [splits][rows][DP]: sums of weights times values
  float* ml;                // [splits][rows][2]: maximum (log2) and sum of weights
};

struct AttnP {
  svdq_attention_args a;
  int G, R, tiles, groups;  // heads per K/V head, rows per (entry, K/V head), row tiles, entries x K/V heads
  float qmul, c1, c2, c3, c4;   // see svdq_attention()
  float cap[7];                 // c1 x the coefficients of tanh(x) / x in x^2
  bool flip;
  Part part;
};

template <int DT>
__device__ __forceinline__ b16f mma(const b4i& a, const b4i& b, const b16f& c) {
  if constexpr (DT == SVDQ_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8bf, a), __builtin_bit_cast(b8bf, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(b8h, a), __builtin_bit_cast(b8h, b), c, 0, 0, 0);
}

// both halves' value of the lane pair (l, l + 32)
__device__ __forceinline__ float half_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Which (entry, K/V head) and which of its row tiles and key parts a block
// takes.  Blocks are dealt to the 8 XCDs round robin; with a multiple of 8
// groups an XCD keeps to groups of its own, so that its L2 holds their K and V.
// Neighbouring blocks take different groups, so that the longest rows of a causal
// mask come first in every group (4608 tokens x 24 heads of 128: 152 us, 164 with
// one group after the other; all visible 295 either way).
template <bool KEYS>
__device__ __forceinline__ void group_order(const AttnP& p, int b, int* grp, int* rest) {
  if constexpr (KEYS) {
    // nothing is shared between blocks: the parts of a group follow each other
    // (one token of 16 requests: 136 us, 147 the other way)
    const int id = xcd_order(b, gridDim.x), per = p.tiles * p.part.splits;
    *grp = id / per;
    *rest = id % per;
  } else if ((p.groups & 7) == 0) {
    const int own = p.groups >> 3, i = b >> 3;
    *grp = (b & 7) * own + i % own;
    *rest = i / own;
  } else {
    *grp = b % p.groups;
    *rest = b / p.groups;
  }
}

// The end of 32 rows of a wave (lane l: row row0 + l % 32, O^T as the MFMAs
// leave it, m and l of the whole row): stored as parts or finished.
template <int DT, int DP, bool PAD>
__device__ __forceinline__ void store_rows(const AttnP& p, int grp, int b, int hk, int sp, int row0, int lane, float m, float l,
                                           const b16f (&o)[DP / 32]) {
  const svdq_attention_args& a = p.a;
  constexpr int ND = DP / 32;
  const int l32 = lane & 31, half = lane >> 5;
  const int row = row0 + l32;
  const size_t rows_all = (size_t)p.groups * p.R;
  const bool parts = p.part.splits > 1;
  if (row < p.R) {
    if (parts) {
      const size_t at = (size_t)sp * rows_all + (size_t)grp * p.R + row;
      float* op = p.part.o + at * DP;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<b4f*>(op + 32 * d + 8 * g + 4 * half) =
              (b4f){o[d][4 * g], o[d][4 * g + 1], o[d][4 * g + 2], o[d][4 * g + 3]};
      if (half == 0) *reinterpret_cast<float2*>(p.part.ml + 2 * at) = make_float2(m, l);
    } else {
      const float by = l != 0.f ? 1.0f / l : 0.f;
      const int qi = row / p.G, qh = hk * p.G + row % p.G;
      uint16_t* op = a.o + b * a.o_batch + qi * a.o_token + qh * a.o_head;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int at = 32 * d + 8 * g + 4 * half;
          if (!PAD || at < a.D)
            *reinterpret_cast<uint2*>(op + at) = make_uint2(narrow2<DT>(o[d][4 * g] * by, o[d][4 * g + 1] * by),
                                                            narrow2<DT>(o[d][4 * g + 2] * by, o[d][4 * g + 3] * by));
        }
    }
  }
}

// LDS of a block.  KEYS: waves share 32 rows and take key tiles in turn; otherwise
// waves take rows and share key tiles.
template <int DP, bool KEYS>
struct Shared {
  static constexpr int KT = KEYS ? 1 : 2;          // 32-key subtiles of a tile
  static constexpr int TK = 32 * KT;
  static constexpr int TILE = TK * 2 * DP;         // one of K, V
  static constexpr int RING = 4 * TILE;            // K, V of two tiles
  static constexpr int LDS = KEYS ? 4 * RING : RING;
  __attribute__((aligned(1024))) uint8_t tiles[LDS];
  int docs[4][TK];
  uint32_t seen[KEYS ? 1 : kSeen / 32];
  uint32_t redo[4];                                // per wave: rows for the second pass
  uint32_t marks[DP / 32][256];                    // per lane, two bits per register of O: it saw +, - infinity (NaN: both)
};

// A block's rows over its share of the keys.  PAD: D < DP.  KEYS: returns whether
// rows have to be gone over again; the call with AGAIN does that, with weights up to
// 2^lag.
template <int DT, int DP, bool PAD, bool KEYS, bool AGAIN>
__device__ __forceinline__ bool attention_block(const AttnP& p, Shared<DP, KEYS>* sh, float lag) {
  const svdq_attention_args& a = p.a;
  using S = Shared<DP, KEYS>;
  constexpr int KT = S::KT, TK = S::TK, TILE = S::TILE, RING = S::RING, LDS = S::LDS;
  constexpr int ROWB = 2 * DP;                     // bytes of a row in LDS
  constexpr int CH = DP / 8;                       // 16-byte chunks of a row
  constexpr int RPI = 64 / CH;                     // rows of one 1 KB copy
  constexpr int COPIES = TILE / 1024;              // of K or V, per tile
  constexpr int MINE = KEYS ? COPIES : COPIES / 4; // per wave
  constexpr int NS = DP / 16;                      // MFMA steps of S
  constexpr int ND = DP / 32;                      // 32-column tiles of O
  constexpr int AHEAD_K = 4, AHEAD_V = 2;          // fragments read ahead
  uint8_t* lds = sh->tiles;
  auto& docs = sh->docs;
  auto& seen = sh->seen;
  auto& redo = sh->redo;
  auto& marks = sh->marks;

  int tid = threadIdx.x, block = blockIdx.x;
  if constexpr (AGAIN) asm volatile("" : "+v"(tid), "+s"(block));   // see attention_kernel
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, half = lane >> 5;
  int grp, rest;
  group_order<KEYS>(p, block, &grp, &rest);
  // the last rows see most keys under a causal mask: they go first
  const int rt = p.tiles - 1 - rest / p.part.splits, sp = rest % p.part.splits;
  const int b = grp / a.Hkv, hk = grp % a.Hkv;
  const int n = a.kv_len ? min(max(a.kv_len[b], 0), a.Skv) : a.Skv;
  const int pre = a.causal && a.prefix ? a.prefix[b] : 0;
  const int row_base = rt * (KEYS ? 32 : 128);
  const int row0 = row_base + (KEYS ? 0 : 32 * wave);
  const int row = min(row0 + l32, p.R - 1);
  const int qi = row / p.G, qh = hk * p.G + row % p.G;
  const int pos = n - a.Sq + qi;
  auto limit = [&](int r) {   // keys below it may be visible to row r
    return a.causal ? min(n, max(max(n - a.Sq + r / p.G + 1, pre), 0)) : n;
  };
  const int lim = limit(row);
  const int lim_first = limit(min(row0, p.R - 1)), lim_last = limit(min(row0 + 31, p.R - 1));
  const int end = limit(min(row_base + (KEYS ? 31 : 127), p.R - 1));
  const bool use_docs = a.q_doc != nullptr;
  const float slope = a.slopes ? a.slopes[qh] * 1.44269504f : 0.f;

  // this block's tiles
  const int all = (end + TK - 1) / TK;
  const int share = (all + p.part.splits - 1) / p.part.splits;
  const int t_begin = min(all, sp * share), t_end = min(all, t_begin + share);

  // ---- Q as the B operand: step s, elements 16 s + 8 half .. + 8 of the lane's row
  b4i qf[NS];
  {
    const uint16_t* qp = a.q + b * a.q_batch + qi * a.q_token + qh * a.q_head;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int d = 16 * s + 8 * half;
      qf[s] = (b4i){0, 0, 0, 0};
      if (!PAD || d < a.D) qf[s] = *reinterpret_cast<const b4i*>(qp + d);
    }
  }
  // its sign, or zero; after the first copies are on their way, as it waits for Q
  auto turn_q = [&]() __attribute__((always_inline)) {
    if (p.qmul > 0.f) return;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) qf[s][i] = p.flip ? qf[s][i] ^ (int)0x80008000 : 0;
  };
  const int qd = use_docs ? a.q_doc[(size_t)b * a.Sq + qi] : 0;
  int doc_lo = qd, doc_hi = qd;   // documents of the block's rows
  if (!KEYS && use_docs) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int d = a.q_doc[(size_t)b * a.Sq + min(row_base + 64 * k + lane, p.R - 1) / p.G];
      doc_lo = min(doc_lo, d);
      doc_hi = max(doc_hi, d);
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
      doc_lo = min(doc_lo, __shfl_xor(doc_lo, d));
      doc_hi = max(doc_hi, __shfl_xor(doc_hi, d));
    }
  }
  const int qd_first = __builtin_amdgcn_readfirstlane(qd);
  const bool one_doc = use_docs && __all(qd == qd_first);

  // ---- copies to LDS
  const uint32_t lbase = lds_address(lds) + (KEYS ? wave * RING : 0);
  if constexpr (PAD) {
    // columns D .. DP of the buffers are never copied: zero for good
    uint32_t* w = reinterpret_cast<uint32_t*>(lds);
    for (int i = tid; i < LDS / 4; i += 256) w[i] = 0;
    __syncthreads();
  }
  const uint8_t* kbase = reinterpret_cast<const uint8_t*>(a.k + b * a.k_batch + hk * a.k_head);
  const uint8_t* vbase = reinterpret_cast<const uint8_t*>(a.v + b * a.v_batch + hk * a.v_head);
  const int crow = lane / CH, cslot = lane % CH;   // row and 16-byte slot of a copy's lane
  // chunk of K row r at slot c and the other way round
  auto k_chunk = [&](int r, int c) { return DP == 128 ? c ^ (r & 15) : c ^ ((r >> 1) & 7); };
  auto v_chunk = [&](int r, int c) { return DP == 128 ? c ^ (4 * (r & 3)) : c ^ (4 * ((r >> 1) & 1)); };
  const uint32_t kst = 2u * (uint32_t)a.k_token, vst = 2u * (uint32_t)a.v_token;   // at most 2^26
  const int r_first = RPI * (KEYS ? 0 : MINE * wave);
  uint32_t koffs[MINE], voffs[MINE];
  bool klive[MINE], vlive[MINE];
#pragma unroll
  for (int c = 0; c < MINE; ++c) {
    const int r = r_first + RPI * c + crow, kc = k_chunk(r, cslot), vc = v_chunk(r, cslot);
    koffs[c] = (uint32_t)r * kst + 16 * kc;
    voffs[c] = (uint32_t)r * vst + 16 * vc;
    klive[c] = !PAD || 8 * kc < a.D;
    vlive[c] = !PAD || 8 * vc < a.D;
  }
  auto copy_tile = [&](int t, int buf) __attribute__((always_inline)) {
    const uint8_t *kp = kbase + (uint64_t)(t * TK) * kst, *vp = vbase + (uint64_t)(t * TK) * vst;
    const uint32_t dst = lbase + buf * 2 * TILE + r_first * ROWB;
    const int last = n - 1 - t * TK;
    if (last >= TK - 1) {
#pragma unroll
      for (int c = 0; c < MINE; ++c) {
        if (klive[c]) dma_16(kp, koffs[c], dst + 1024 * c);
        if (vlive[c]) dma_16(vp, voffs[c], dst + TILE + 1024 * c);
      }
    } else {
      // the last tile: rows past the last key in use repeat it
#pragma unroll
      for (int c = 0; c < MINE; ++c) {
        const int r = r_first + RPI * c + crow;
        const uint32_t over = (uint32_t)max(r - last, 0);
        if (klive[c]) dma_16(kp, koffs[c] - over * kst, dst + 1024 * c);
        if (vlive[c]) dma_16(vp, voffs[c] - over * vst, dst + TILE + 1024 * c);
      }
    }
  };

  // fragment addresses
  const uint8_t* wl = lds + (KEYS ? wave * RING : 0);
  int koff[NS], voff[ND];
#pragma unroll
  for (int s = 0; s < NS; ++s) koff[s] = l32 * ROWB + 16 * k_chunk(l32, 2 * s + half);
  {
    const int i16 = lane & 15, dh = (lane >> 4) & 1, kr = 4 * half + i16 / 4;
#pragma unroll
    for (int d = 0; d < ND; ++d) voff[d] = kr * ROWB + 16 * v_chunk(kr, 4 * d) + 32 * dh + 8 * (i16 % 4);
  }

  float m, l;
  b16f o[ND];

  const bool plain = !(a.softcap > 0.f) && !a.slopes;   // score = c1 x dot product

  b4i pf[2 * KT];   // weights of a tile, 16 bits

  // O += V P of the tile in `buf`, fragments AHEAD_V MFMAs ahead (the first of
  // them are read before the weights are worked out)
  b4i vf[AHEAD_V];
  auto read_v = [&](int buf, int i) __attribute__((always_inline)) {
    typedef short s4 __attribute__((ext_vector_type(4)));
    const uint8_t* vl = wl + buf * 2 * TILE + TILE + voff[i % ND] + 16 * (i / ND) * ROWB;
    const s4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((SVDQ_LDS s4*)vl);
    const s4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((SVDQ_LDS s4*)(vl + 8 * ROWB));
    const int2 lo = __builtin_bit_cast(int2, v0), hi = __builtin_bit_cast(int2, v1);
    vf[i % AHEAD_V] = (b4i){lo.x, lo.y, hi.x, hi.y};
  };
  auto first_values = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < AHEAD_V; ++i) read_v(buf, i);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto values = [&](int buf) __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 2 * KT * ND; ++i) {
      o[i % ND] = mma<DT>(vf[i % AHEAD_V], pf[i / ND], o[i % ND]);
      if (i + AHEAD_V < 2 * KT * ND) read_v(buf, i + AHEAD_V);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // Scores and weights of tile t, and the running maximum and sum.  kd:
  // document of key j0 + lane (where documents are used).
  auto scores = [&](int t, int buf, int kd) __attribute__((always_inline)) {
    const int j0 = t * TK;
    const uint8_t* kl = wl + buf * 2 * TILE;
    b16f s[KT];
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[k][i] = 0.f;
    // Consecutive MFMAs add to different registers, and fragments are read
    // AHEAD_K MFMAs ahead: left to itself the compiler puts each read right
    // before its MFMA and waits for it, hence the fences.
    b4i kf[AHEAD_K];
    auto read_k = [&](int i) __attribute__((always_inline)) {
      kf[i % AHEAD_K] = *reinterpret_cast<const b4i*>(kl + koff[i / KT] + (i % KT) * 32 * ROWB);
    };
#pragma unroll
    for (int i = 0; i < AHEAD_K; ++i) read_k(i);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < KT * NS; ++i) {
      s[i % KT] = mma<DT>(kf[i % AHEAD_K], qf[i / KT], s[i % KT]);
      if (i + AHEAD_K < KT * NS) read_k(i + AHEAD_K);
      __builtin_amdgcn_sched_barrier(0);
    }
    float c = p.c1;
    if (!plain) {
      c = 1.f;
      if (a.softcap > 0.f) {
        if (a.softcap <= kSmallCap) {
#pragma unroll
          for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int i = 0; i < 16; ++i) s[k][i] = by_exp(p, s[k][i]);
        } else {
          float big = 0.f;
#pragma unroll
          for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int i = 0; i < 16; ++i) big = fmaxf(big, fabsf(s[k][i]));
          if (__any(big * p.c4 > 1.0f)) {
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
              for (int i = 0; i < 16; ++i) s[k][i] = capped(p, s[k][i]);
          } else {
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
              for (int i = 0; i < 16; ++i) s[k][i] = by_series(p, s[k][i]);
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[k][i] *= p.c1;
      }
      if (a.slopes) {
        const float from = (float)(pos - j0 - 4 * half);
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[k][i] = fmaf(-slope, fabsf(from - (float)(32 * k + 8 * (i / 4) + i % 4)), s[k][i]);
      }
    }
    if (j0 + TK > lim_first) {
      const int rel = lim - j0 - 4 * half;
#pragma unroll
      for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (32 * k + 8 * (i / 4) + i % 4 >= rel) s[k][i] = -__builtin_inff();
    }
    if (use_docs && !(one_doc && __all(kd == qd_first))) {
      docs[wave][lane & (TK - 1)] = kd;
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const b4i kk = *reinterpret_cast<const b4i*>(&docs[wave][32 * k + 8 * g + 4 * half]);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (kk[i] != qd) s[k][4 * g + i] = -__builtin_inff();
        }
      __builtin_amdgcn_wave_barrier();
    }
    float top = s[0][0];
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[k][i]);
    top = half_max(top) * c;
    if (__any(top > m + lag)) {
      const float up = fmaxf(m, top);
      const float f = exp2_(m - up);
      m = up;
      l *= f;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= f;
    }
    first_values(buf);
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      float part = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[k][i] = exp2_(fmaf(s[k][i], c, -m));
        part += s[k][i];
      }
      l += part;
      // To the product with V the weights go in the call's type, as the matrix unit
      // takes it; their sum stays as they were.  The output is off by at most 2^-8
      // (bf16) or 2^-11 (fp16) of mean |v| for that (error against 64 bits 2.3e-3 and
      // 2.8e-4 of its norm, of which the store 1.7e-3 and 2.1e-4).
#pragma unroll
      for (int x = 0; x < 8; ++x) pf[2 * k + x / 4][x % 4] = (int)narrow2<DT>(s[k][2 * x], s[k][2 * x + 1]);
    }
  };
  auto doc_of = [&](int t) -> int {
    return use_docs && t < t_end ? a.k_doc[(size_t)b * a.Skv + min(t * TK + (lane & (TK - 1)), n - 1)] : 0;
  };

  // Second pass, tile t in `buf` before its scores: the keys whose values are not
  // all finite are found, each lane marks those values of its columns that its
  // row sees, and they are set to zero.  All waves find the same keys.
  auto take_out = [&](int t, int buf, int kd) __attribute__((always_inline)) {
    constexpr uint32_t EXP = DT == SVDQ_BF16 ? 0x7F80u : 0x7C00u;   // all ones: infinity or NaN
    uint8_t* vt = lds + (KEYS ? wave * RING : 0) + buf * 2 * TILE + TILE;
    auto odd = [&](uint32_t w) { return (w & EXP) == EXP || ((w >> 16) & EXP) == EXP; };
    // KEYS: a lane looks through half a key; otherwise through one
    constexpr int LOOK = KEYS ? CH / 2 : CH;
    const int key = lane & (TK - 1);               // its chunks in another order than its neighbours', for the banks
    uint8_t* own = vt + key * ROWB + (KEYS ? half * (ROWB / 2) : 0);
    bool any = false;
#pragma unroll 1
    for (int c = 0; c < LOOK; ++c) {
      const b4i w = *reinterpret_cast<const b4i*>(own + 16 * ((c + key) % LOOK));
#pragma unroll
      for (int i = 0; i < 4; ++i) any = any || odd((uint32_t)w[i]);
    }
    uint64_t keys = __ballot(any);
    if (KEYS) keys = (keys | (keys >> 32)) & 0xFFFFFFFFull;
    if (keys == 0) return;
#pragma unroll 1
    for (uint64_t left = keys; left; left &= left - 1) {
      const int j = __builtin_ctzll(left);
      const uint32_t sees = t * TK + j < lim && (!use_docs || __builtin_amdgcn_readlane(kd, j) == qd) ? ~0u : 0u;
#pragma unroll 1
      for (int c = 0; c < 4 * ND; ++c) {
        const uint2 w = *reinterpret_cast<const uint2*>(vt + j * ROWB + 16 * v_chunk(j, c) + 8 * half);
        uint32_t bits = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t v = (i < 2 ? w.x : w.y) >> (16 * (i & 1)) & 0xFFFFu;
          const uint32_t kind = (v & 0x7FFFu) > EXP ? 3u : v & 0x8000u ? 2u : 1u;
          if ((v & EXP) == EXP) bits |= kind << (2 * i);
        }
        marks[c >> 2][tid] |= (bits & sees) << (8 * (c & 3));
      }
    }
    // every wave that reads these values has marked them
    if constexpr (KEYS) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_wave_barrier();
    } else {
      __syncthreads();
    }
    if (KEYS || key / 16 == wave) {
#pragma unroll 1
      for (int c = 0; c < LOOK; ++c) {
        b4i w = *reinterpret_cast<const b4i*>(own + 16 * ((c + key) % LOOK));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t v = (uint32_t)w[i];
          if ((v & EXP) == EXP) v &= 0xFFFF0000u;
          if (((v >> 16) & EXP) == EXP) v &= 0x0000FFFFu;
          w[i] = (int)v;
        }
        *reinterpret_cast<b4i*>(own + 16 * ((c + key) % LOOK)) = w;
      }
    }
    if constexpr (KEYS) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_wave_barrier();
    } else {
      __syncthreads();
    }
  };

  // documents: which tiles the block has to visit (see below)
  if (!KEYS && use_docs) {
    for (int w = wave; w < (min(t_end - t_begin, kSeen) + 31) / 32; w += 4) {
      int kd[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const int j = (t_begin + 32 * w + k) * TK + lane;
        kd[k] = a.k_doc[(size_t)b * a.Skv + min(j, n - 1)];
      }
      uint32_t bits = 0;
#pragma unroll
      for (int k = 0; k < 32; ++k) bits |= (__any(kd[k] >= doc_lo && kd[k] <= doc_hi) ? 1u : 0u) << k;
      if (lane == 0) seen[w] = bits;
    }
    __syncthreads();
  }

  // One pass over the block's tiles.  SECOND: without what is not finite.
  auto pass = [&](auto second) __attribute__((always_inline)) {
    constexpr bool SECOND = decltype(second)::value;
    m = kLow;
    l = 0.f;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][i] = 0.f;

    if constexpr (KEYS) {
      // each wave on its own: tiles t_begin + wave, + 4, ...
      int t = t_begin + wave, buf = 0;
      if (t < t_end) copy_tile(t, 0);
      turn_q();
      int kd = doc_of(t);
      for (; t < t_end; t += 4, buf ^= 1) {
        dma_wait();
        __builtin_amdgcn_wave_barrier();
        if (t + 4 < t_end) copy_tile(t + 4, buf ^ 1);
        const int kd_next = doc_of(t + 4);
        if constexpr (SECOND) take_out(t, buf, kd);
        scores(t, buf, kd);
        values(buf);
        // this tile's LDS reads end before the next copy may overwrite it
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        kd = kd_next;
      }
    } else {
      // Tiles in turn; where documents are used, those that hold none of the
      // block's are passed over: the waves have looked through the first kSeen tiles
      // of the block's share beforehand (later ones are all visited).
      int word = -1;
      uint32_t bits = 0;
      auto next = [&](int t) -> int {
        if (!use_docs) return t;
        for (int i = t - t_begin; i < t_end - t_begin && i < kSeen; i = (i | 31) + 1) {
          if (i >> 5 != word) {
            word = i >> 5;
            bits = __builtin_amdgcn_readfirstlane(seen[word]);
          }
          const uint32_t left = bits >> (i & 31);
          if (left) return min(t_end, t_begin + i + __builtin_ctz(left));
        }
        return min(t_end, max(t, t_begin + kSeen));
      };
      int t = next(t_begin), buf = 0;
      if (t < t_end) copy_tile(t, 0);
      if constexpr (!SECOND) turn_q();
      int kd = doc_of(t);
      while (t < t_end) {
        // tile t has landed for every wave, and all are done with the one before
        dma_wait();
        __syncthreads();
        const int tn = next(t + 1);
        if (tn < t_end) copy_tile(tn, buf ^ 1);
        const int kd_next = doc_of(tn);
        if constexpr (SECOND) take_out(t, buf, kd);
        if (t * TK < lim_last) {
          scores(t, buf, kd);
          values(buf);
        }
        kd = kd_next;
        t = tn;
        buf ^= 1;
      }
    }
    l = half_sum(l);
  };
  pass(std::integral_constant<bool, AGAIN>{});

  if constexpr (KEYS) {
    // join the waves: O^T, m and l of waves 1..3 through LDS, where the tiles were,
    // to wave 0
    __syncthreads();
    float* jo = reinterpret_cast<float*>(lds);                 // [4][32 rows][DP + 4]
    float* jm = reinterpret_cast<float*>(lds) + 4 * 32 * (DP + 4);
    if (half == 0) {
      jm[(wave * 32 + l32) * 2] = m;
      jm[(wave * 32 + l32) * 2 + 1] = l;
    }
    if (wave > 0) {
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<b4f*>(jo + (wave * 32 + l32) * (DP + 4) + 32 * d + 8 * g + 4 * half) =
              (b4f){o[d][4 * g], o[d][4 * g + 1], o[d][4 * g + 2], o[d][4 * g + 3]};
    }
    __syncthreads();
    if (wave == 0) {
      float up = m;
#pragma unroll
      for (int w = 1; w < 4; ++w) up = fmaxf(up, jm[(w * 32 + l32) * 2]);
      const float f0 = exp2_(m - up);
      l *= f0;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= f0;
#pragma unroll
      for (int w = 1; w < 4; ++w) {
        const float f = exp2_(jm[(w * 32 + l32) * 2] - up);
        l = fmaf(f, jm[(w * 32 + l32) * 2 + 1], l);
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const b4f x = *reinterpret_cast<const b4f*>(jo + (w * 32 + l32) * (DP + 4) + 32 * d + 8 * g + 4 * half);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[d][4 * g + i] = fmaf(f, x[i], o[d][4 * g + i]);
          }
      }
      m = up;
    }
  }

  // Rows to be gone over again?  (KEYS: wave 0 has them all.)  A sum over O tells in
  // half the instructions of a look at each; should it overflow, the passes are
  // only in vain.
  auto any_odd = [&]() __attribute__((always_inline)) -> bool {
    bool odd = false;
    if (!KEYS || wave == 0) {
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[i % 4] += o[d][i];
      odd = !(fabsf(sum[0] + sum[1] + (sum[2] + sum[3])) < __builtin_inff()) && fabsf(l) < __builtin_inff() &&
            row0 + l32 < p.R;
    }
    uint32_t rows = __any(odd);
    if (lane == 0) redo[wave] = rows;
    __syncthreads();
    if (!KEYS || wave > 0) rows = __builtin_amdgcn_readfirstlane(redo[0] | redo[1] | redo[2] | redo[3]);
    return rows != 0;
  };
  // The second pass, and a third with weights up to 1 should sums of finite values
  // overflow.  KEYS: by the caller.
  bool marked = AGAIN;
  if (__builtin_expect(any_odd(), 0)) {
    if constexpr (KEYS) {
      if (lag != 0.f) return true;
    } else {
#pragma unroll 1
      for (;;) {
        __syncthreads();
#pragma unroll
        for (int d = 0; d < ND; ++d) marks[d][tid] = 0;
        pass(std::true_type{});
        if (!any_odd() || lag == 0.f) break;
        lag = 0.f;
      }
      marked = true;
    }
  }
  if (KEYS && wave > 0) return false;
  if (__builtin_expect(marked, KEYS)) {
    // O is finite where it is marked: add the infinity or NaN
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      uint32_t bits = marks[d][tid];
      if (KEYS) bits |= marks[d][64 + lane] | marks[d][128 + lane] | marks[d][192 + lane];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t plus = bits >> (2 * i) & 1u, minus = bits >> (2 * i + 1) & 1u;
        o[d][i] += __uint_as_float((plus | minus) * 0x7F800000u | (plus & minus) << 22 | (minus & ~plus) << 31);
      }
    }
  }

  store_rows<DT, DP, PAD>(p, grp, b, hk, sp, row0, lane, m, l, o);
  return false;
}

// With KEYS the second pass starts from the arguments, read again through an address
// that the compiler does not know, as a block does from its place in the grid: with
// anything kept for it from the first pass short calls took 0.4 - 0.8 us more.  128
// rows a block keep what they have (starting anew they would need scratch memory).
template <int DT, int DP, bool PAD, bool KEYS>
__global__ __launch_bounds__(256, KEYS && DP == 128 ? 1 : 2) void attention_kernel(AttnP p) {
  __shared__ Shared<DP, KEYS> sh;
  const bool again = attention_block<DT, DP, PAD, KEYS, false>(p, &sh, 8.0f);
  if constexpr (KEYS) {
    if (__builtin_expect(!again, 1)) return;
#pragma unroll 1
    for (float lag = 8.0f;; lag = 0.f) {
      uint64_t at = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr();
      asm volatile("" : "+s"(at));
      const AttnP q = *(const AttnP*)(__attribute__((address_space(4))) const AttnP*)at;
      __syncthreads();
#pragma unroll
      for (int d = 0; d < DP / 32; ++d) sh.marks[d][threadIdx.x] = 0;
      if (!attention_block<DT, DP, PAD, KEYS, true>(q, &sh, lag)) return;
    }
  }
}

// Joins the parts of the rows: DP / 8 lanes hold a row's 8-element pieces, and
// `across` such lane sets (1, 2, .. 16) of a block share the row's parts, so that
// many parts are a few rounds of loads.
template <int DT, int DP>
__global__ __launch_bounds__(256) void join_kernel(AttnP p, int across) {
  const svdq_attention_args& a = p.a;
  constexpr int LPR = DP / 8;
  __shared__ float part[256][11];   // 8 sums, maximum, sum of weights; 11: odd stride
  const size_t rows = (size_t)p.groups * p.R;
  const int set = threadIdx.x / LPR, g = set % across, d = 8 * (threadIdx.x % LPR);
  const size_t at = (size_t)blockIdx.x * (256 / LPR / across) + set / across;
  const bool live = at < rows;
  float top = kLow, sum = 0.f, o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = 0.f;
  if (live) {
    for (int s = g; s < p.part.splits; s += across) {
      const float2 ml = *reinterpret_cast<const float2*>(p.part.ml + 2 * (s * rows + at));
      const float* op = p.part.o + (s * rows + at) * DP + d;
      const b4f x = *reinterpret_cast<const b4f*>(op), y = *reinterpret_cast<const b4f*>(op + 4);
      const float up = fmaxf(top, ml.x), f0 = exp2_(top - up), f = exp2_(ml.x - up);
      sum = fmaf(f, ml.y, sum * f0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[i] = fmaf(f, x[i], o[i] * f0);
        o[4 + i] = fmaf(f, y[i], o[4 + i] * f0);
      }
      top = up;
    }
  }
  if (across > 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) part[threadIdx.x][i] = o[i];
    part[threadIdx.x][8] = top;
    part[threadIdx.x][9] = sum;
    __syncthreads();
    if (g == 0) {
      for (int k = 1; k < across; ++k) {
        const float* x = part[threadIdx.x + k * LPR];
        const float up = fmaxf(top, x[8]), f0 = exp2_(top - up), f = exp2_(x[8] - up);
        sum = fmaf(f, x[9], sum * f0);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = fmaf(f, x[i], o[i] * f0);
        top = up;
      }
    }
  }
  if (!live || g != 0 || d >= a.D) return;
  const float by = sum != 0.f ? 1.0f / sum : 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] *= by;
  const int grp = (int)(at / p.R), r = (int)(at % p.R);
  uint16_t* op = a.o + (grp / a.Hkv) * a.o_batch + (r / p.G) * a.o_token +
                 ((grp % a.Hkv) * p.G + r % p.G) * a.o_head + d;
  *reinterpret_cast<b4i*>(op) = narrow8<DT>(o);
}

svdq_status check(const svdq_attention_args* a) {
  if (!a || !a->q || !a->o) return SVDQ_ERR_ARG;
  if (!is_dtype(a->dtype)) return SVDQ_ERR_UNSUPPORTED;
  constexpr int64_t lim = 1 << 24;
  if (a->B < 1 || a->Sq < 1 || a->Sq > lim || a->Skv < 0 || a->Skv > lim || a->Hq < 1 || a->Hkv < 1 ||
      a->Hq > 65536 || a->Hq % a->Hkv != 0 || a->D < 8 || a->D > SVDQ_ATTENTION_MAX_HEAD_DIM || a->D % 8 != 0)
    return SVDQ_ERR_SHAPE;
  // at most a block of 256 threads per head and 32 rows: fewer than 2^32 threads
  if ((int64_t)a->B * a->Hq >= (1 << 24) || (int64_t)a->B * a->Hq * a->Sq > (int64_t)1 << 30) return SVDQ_ERR_SHAPE;
  if (a->Skv > 0 && (!a->k || !a->v)) return SVDQ_ERR_ARG;
  if ((a->q_doc == nullptr) != (a->k_doc == nullptr) && a->Skv > 0) return SVDQ_ERR_ARG;
  const float big = 3.0e38f;
  if (!(a->scale >= -big && a->scale <= big) || !(a->softcap >= 0.f && a->softcap <= big)) return SVDQ_ERR_ARG;
  const int64_t st[] = {a->q_batch, a->q_token, a->q_head, a->k_batch, a->k_token, a->k_head,
                        a->v_batch, a->v_token, a->v_head, a->o_batch, a->o_token, a->o_head};
  for (int64_t s : st)
    if (s % 8 != 0) return SVDQ_ERR_ALIGN;
  if (a->k_token < 0 || a->v_token < 0 || a->k_token > (1 << 25) || a->v_token > (1 << 25)) return SVDQ_ERR_SHAPE;
  if (!on16(a->q) || !on16(a->k) || !on16(a->v) || !on16(a->o) || !on4(a->slopes) || !on4(a->kv_len) ||
      !on4(a->prefix) || !on4(a->q_doc) || !on4(a->k_doc))
    return SVDQ_ERR_ALIGN;
  return SVDQ_OK;
}

// The arrangement of a call: by its sizes alone, so that a workspace fits
// every call of its shape.
struct Plan {
  bool keys;
  int G, R, tiles, groups, splits;
  size_t rows() const { return (size_t)groups * R; }
};
Plan plan_of(int32_t B, int32_t Sq, int32_t Skv, int32_t Hq, int32_t Hkv, int32_t D) {
  Plan p;
  p.G = Hq / Hkv;
  p.R = Sq * p.G;
  p.groups = B * Hkv;
  // Blocks of 32 rows whose waves share the keys, as long as the chip holds one
  // for every 32 rows (LDS: one a compute unit for heads above 64, two below) and
  // a pass over the keys for 32 rows instead of 128 is not what takes the time.
  // Measured, us (128 rows -> 32): 512 queries on as many keys, 8 heads of 128
  // 16.3 -> 11.1; 16 on 8192, 32 on 8 heads 29.6 -> 17.7; 2 x 64 on 512, 16 on
  // 4 16.9 -> 11.1; 200 on 3000, 8 heads (168000 keys) 22.0 -> 25.5; 6 x 16 on
  // 11453, 8 on 1 (275000 keys) 33.6 -> 40.5; 4 x 142 on 142, 16 on 2 (288
  // blocks) 10.7 -> 14.7.
  const int64_t fine = (int64_t)((p.R + 31) / 32) * p.groups;
  p.keys = p.R <= 32 || (fine <= (D <= 64 ? 2 : 1) * kCus && fine * Skv <= 160 * 1024);
  p.tiles = p.keys ? (p.R + 31) / 32 : (p.R + 127) / 128;
  const int64_t blocks = (int64_t)p.tiles * p.groups;
  // Blocks that the chip holds (twice, where LDS allows one a compute unit), and
  // the keys that are worth a block of their own.
  const int64_t fill = 2 * kCus, least = 512;
  int64_t most = ((int64_t)Skv + least - 1) / least;
  if (most > 64) most = 64;
  int64_t s = 1;
  if (p.keys) {
    // The least time, in steps of 128 keys (32 a wave): rounds of blocks, each
    // with its share of the keys and about a step of start and end, and the join.
    // The most parts among those within 8 %, as lengths may differ.  (One
    // request of 8192 keys x 8 K/V heads 15.5 us: with 1024 keys a part 18.0,
    // with 128 20.7.  Against as many parts as fill the chip twice: 3 such
    // requests 27 for 32 us, 5 of them 41 for 48, 16 of 2048 keys 33 for 37.)
    const int64_t t = ((int64_t)Skv + 127) / 128, slots = (D <= 64 ? 2 : 1) * kCus;
    if (most > (fill + blocks - 1) / blocks) most = (fill + blocks - 1) / blocks;
    auto cost = [&](int64_t k) { return (blocks * k + slots - 1) / slots * ((t + k - 1) / k + 1) + (k > 1); };
    int64_t best = cost(1);
    for (int64_t k = 2; k <= most; ++k)
      if (cost(k) < best) best = cost(k);
    for (int64_t k = 2; k <= most; ++k)
      if (cost(k) * 100 <= best * 108) s = k;
  } else if (blocks < fill) {
    // the least time, in half tiles of 64 keys: rounds of blocks, each with its
    // share of the keys and about 6 tiles' worth of start and end, and the join.
    // (Against as many parts as fill the chip: 2 x 700 queries of 16 heads on
    // 3001 keys, 68 for 73 us; 1024 of 24 on 4096, 78 for 95; 2500 of 16 on as
    // many, 81 for 87.)
    const int64_t t = ((int64_t)Skv + 63) / 64;
    int64_t best = 0;
    for (int64_t k = 1; k <= most; ++k) {
      const int64_t rounds = (blocks * k + fill - 1) / fill;
      const int64_t cost = 2 * rounds * ((t + k - 1) / k + 6) + (k > 1 ? 12 + 3 * k : 0);
      if (k == 1 || cost < best) {
        best = cost;
        s = k;
      }
    }
  }
  p.splits = s < 1 ? 1 : (int)s;
  return p;
}
int padded_dim(int32_t D) { return D <= 64 ? 64 : 128; }

template <int DT, int DP, bool PAD>
svdq_status launch3(const AttnP& p, const Plan& pl, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)pl.tiles * pl.groups * pl.splits));
  if (pl.keys) hipLaunchKernelGGL((attention_kernel<DT, DP, PAD, true>), grid, dim3(256), 0, st, p);
  else hipLaunchKernelGGL((attention_kernel<DT, DP, PAD, false>), grid, dim3(256), 0, st, p);
  svdq_status s = launched();
  if (s == SVDQ_OK && pl.splits > 1) {
    int across = 1;
    while (across < 16 && across < pl.splits) across *= 2;
    const int per = 256 / (DP / 8) / across;
    hipLaunchKernelGGL((join_kernel<DT, DP>), dim3((unsigned)((pl.rows() + per - 1) / per)), dim3(256), 0, st, p, across);
    s = launched();
  }
  return s;
}
template <int DT>
svdq_status launch2(const AttnP& p, const Plan& pl, hipStream_t st) {
  if (p.a.D == 128) return launch3<DT, 128, false>(p, pl, st);
  if (p.a.D > 64) return launch3<DT, 128, true>(p, pl, st);
  if (p.a.D == 64) return launch3<DT, 64, false>(p, pl, st);
  return launch3<DT, 64, true>(p, pl, st);
}

}  // namespace
}  // namespace svdq

using namespace svdq;

extern "C" size_t svdq_attention_workspace_bytes(int32_t B, int32_t Sq, int32_t Skv, int32_t Hq, int32_t Hkv,
                                                 int32_t D) {
  if (B < 1 || Sq < 1 || Skv < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || D < 8 || D > SVDQ_ATTENTION_MAX_HEAD_DIM ||
      (int64_t)B * Hq >= (1 << 24) || (int64_t)B * Hq * Sq > (int64_t)1 << 30)
    return 0;
  const Plan p = plan_of(B, Sq, Skv, Hq, Hkv, D);
  if (p.splits == 1) return 0;
  return align256(p.splits * p.rows() * padded_dim(D) * 4) + align256(p.splits * p.rows() * 8);
}

extern "C" svdq_status svdq_attention(const svdq_attention_args* a, void* ws, size_t ws_bytes, void* stream) {
  svdq_status s = check(a);
  if (s != SVDQ_OK) return s;
  const size_t need = svdq_attention_workspace_bytes(a->B, a->Sq, a->Skv, a->Hq, a->Hkv, a->D);
  if (need > 0 && (!ws || ws_bytes < need)) return !ws ? SVDQ_ERR_ARG : SVDQ_ERR_WORKSPACE;
  if (((uintptr_t)ws & 255u) != 0) return SVDQ_ERR_ALIGN;
  if ((s = device_ok()) != SVDQ_OK) return s;
  const Plan pl = plan_of(a->B, a->Sq, a->Skv, a->Hq, a->Hkv, a->D);
  AttnP p;
  p.a = *a;
  p.G = pl.G;
  p.R = pl.R;
  p.tiles = pl.tiles;
  p.groups = pl.groups;
  set_score(&p, a->scale, a->softcap);
  p.part.splits = pl.splits;
  p.part.o = static_cast<float*>(ws);
  p.part.ml = pl.splits > 1
                  ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) +
                                             align256(pl.splits * pl.rows() * padded_dim(a->D) * 4))
                  : nullptr;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return a->dtype == SVDQ_BF16 ? launch2<SVDQ_BF16>(p, pl, st) : launch2<SVDQ_FP16>(p, pl, st);
}
