// Attention over visible keys, with shared K/V heads, score cap, distance
// bias, document numbers, a prefix and lengths.
//
// One wave per (entry, head, query): lane l holds elements 2 l, 2 l + 1 of
// the head, each visible key is one dot product over the wave and one step of
// the running maximum and sum.

#include "device_block.h"

namespace svdq {
namespace {

template <int DT>
__global__ __launch_bounds__(256) void attention_row_kernel(svdq_attention_args a) {
  const int lane = threadIdx.x & 63;
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (id >= (int64_t)a.B * a.Hq * a.Sq) return;
  const int i = (int)(id % a.Sq), h = (int)(id / a.Sq % a.Hq), b = (int)(id / a.Sq / a.Hq);
  const int hk = h / (a.Hq / a.Hkv);
  const bool live = 2 * lane < a.D;
  const int n = a.kv_len ? min(max(a.kv_len[b], 0), a.Skv) : a.Skv;
  const int pos = n - a.Sq + i;
  const int pre = a.causal && a.prefix ? a.prefix[b] : 0;
  const int end = a.causal ? min(n, max(pos + 1, pre)) : n;
  const int doc = a.q_doc ? a.q_doc[(size_t)b * a.Sq + i] : 0;
  auto pair = [&](const uint16_t* p) { return live ? widen2<DT>(*reinterpret_cast<const uint32_t*>(p + 2 * lane)) : (b2f){0.f, 0.f}; };
  const b2f q = pair(a.q + b * a.q_batch + i * a.q_token + h * a.q_head);
  float top = -__builtin_inff(), sum = 0.f;
  b2f o = (b2f){0.f, 0.f};
  for (int j = 0; j < end; ++j) {
    if (a.q_doc && a.k_doc[(size_t)b * a.Skv + j] != doc) continue;
    const b2f k = pair(a.k + b * a.k_batch + j * a.k_token + hk * a.k_head);
    float s = fmaf(q[0], k[0], q[1] * k[1]);
#pragma unroll
    for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
    s *= a.scale;
    if (a.softcap > 0.f) s = a.softcap * tanhf(s / a.softcap);
    if (a.slopes) s -= a.slopes[h] * fabsf((float)(pos - j));
    const float up = fmaxf(top, s);
    const float base = up == -__builtin_inff() ? 0.f : up;
    const float f = __expf(top - base), w = __expf(s - base);
    const b2f v = pair(a.v + b * a.v_batch + j * a.v_token + hk * a.v_head);
    sum = fmaf(sum, f, w);
    o[0] = fmaf(o[0], f, w * v[0]);
    o[1] = fmaf(o[1], f, w * v[1]);
    top = up;
  }
  const float by = sum != 0.f ? 1.0f / sum : 0.f;
  if (live)
    *reinterpret_cast<uint32_t*>(a.o + b * a.o_batch + i * a.o_token + h * a.o_head + 2 * lane) =
        narrow2<DT>(o[0] * by, o[1] * by);
}

svdq_status check(const svdq_attention_args* a) {
  if (!a || !a->q || !a->o) return SVDQ_ERR_ARG;
  if (!is_dtype(a->dtype)) return SVDQ_ERR_UNSUPPORTED;
  constexpr int64_t lim = 1 << 24;
  if (a->B < 1 || a->Sq < 1 || a->Sq > lim || a->Skv < 0 || a->Skv > lim || a->Hq < 1 || a->Hkv < 1 ||
      a->Hq > 65536 || a->Hq % a->Hkv != 0 || a->D < 8 || a->D > SVDQ_ATTENTION_MAX_HEAD_DIM || a->D % 8 != 0)
    return SVDQ_ERR_SHAPE;
  if ((int64_t)a->B * a->Hq > (1 << 24) || (int64_t)a->B * a->Hq * a->Sq > (int64_t)1 << 31) return SVDQ_ERR_SHAPE;
  if (a->Skv > 0 && (!a->k || !a->v)) return SVDQ_ERR_ARG;
  if ((a->q_doc == nullptr) != (a->k_doc == nullptr) && a->Skv > 0) return SVDQ_ERR_ARG;
  const float big = 3.0e38f;
  if (!(a->scale >= -big && a->scale <= big) || !(a->softcap >= 0.f && a->softcap <= big)) return SVDQ_ERR_ARG;
  const int64_t st[] = {a->q_batch, a->q_token, a->q_head, a->k_batch, a->k_token, a->k_head,
                        a->v_batch, a->v_token, a->v_head, a->o_batch, a->o_token, a->o_head};
  for (int64_t s : st)
    if (s % 8 != 0) return SVDQ_ERR_ALIGN;
  if (!on16(a->q) || !on16(a->k) || !on16(a->v) || !on16(a->o) || !on4(a->slopes) || !on4(a->kv_len) ||
      !on4(a->prefix) || !on4(a->q_doc) || !on4(a->k_doc))
    return SVDQ_ERR_ALIGN;
  return SVDQ_OK;
}

}  // namespace
}  // namespace svdq

using namespace svdq;

extern "C" size_t svdq_attention_workspace_bytes(int32_t B, int32_t Sq, int32_t Skv, int32_t Hq, int32_t Hkv,
                                                 int32_t D) {
  (void)B, (void)Sq, (void)Skv, (void)Hq, (void)Hkv, (void)D;
  return 0;
}

extern "C" svdq_status svdq_attention(const svdq_attention_args* a, void* ws, size_t ws_bytes, void* stream) {
  svdq_status s = check(a);
  if (s != SVDQ_OK) return s;
  const size_t need = svdq_attention_workspace_bytes(a->B, a->Sq, a->Skv, a->Hq, a->Hkv, a->D);
  if (need > 0 && (!ws || ws_bytes < need)) return !ws ? SVDQ_ERR_ARG : SVDQ_ERR_WORKSPACE;
  if (((uintptr_t)ws & 255u) != 0) return SVDQ_ERR_ALIGN;
  if ((s = device_ok()) != SVDQ_OK) return s;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int64_t rows = (int64_t)a->B * a->Hq * a->Sq;
  const dim3 grid((unsigned)((rows + 3) / 4)), block(256);
  if (a->dtype == SVDQ_BF16) hipLaunchKernelGGL((attention_row_kernel<SVDQ_BF16>), grid, block, 0, st, *a);
  else hipLaunchKernelGGL((attention_row_kernel<SVDQ_FP16>), grid, block, 0, st, *a);
  return launched();
}
