// history_attn.cu -- wave_history_attention and wave_history_attention_frame:
// attention over the 8-bit history with grouped heads.
//
//   o = sum_{t <= p} w_t vs_t v_t / sum_{t <= p} w_t,   w_t = exp(scale ks_t q.k_t - m)
//
// for the token at position p of a session, with k_t, v_t the codes and ks_t,
// vs_t the scales of its history.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/wave.h"
#include "history_attn.h"

using namespace wave;

namespace wave {

template <int D, typename T>
__global__ void __launch_bounds__(256) k_history_attention(const __grid_constant__ HistoryAttnParams p, int tokens) {
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31;
  const long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int t = (int)(i / p.heads), head = (int)(i % p.heads);
  if (t >= tokens) return;
  int row, pos, slot;
  if (p.positions) {
    row = slot = t;
    pos = p.positions[t];
    if (pos < 0) return;
  } else {
    const int s = seq_of(p.b, t), n = t - p.b.cum[s];
    row = p.b.begin[s] + n;
    pos = p.b.start[s] + n;
    slot = p.b.slot[s];
  }
  T* out = (T*)p.out + (size_t)row * p.out_stride + head * D + lane * kPer;
  float acc[kPer] = {}, q[kPer], m = -INFINITY, l = 0.f;
  if (pos >= p.hist.T_max) {
    if (lane == 0 && head == 0) bad_position(p.err, p.err_out);
    l = 1.f;
    pos = -1;
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) q[e] = (float)((const T*)p.q)[(size_t)row * p.q_stride + head * D + lane * kPer + e];
  const size_t kr = p.hist.row(0, slot, head / p.group), vr = p.hist.row(1, slot, head / p.group);
  const uint8_t *kc = p.hist.codes + kr * p.hist.T_max * D, *vc = p.hist.codes + vr * p.hist.T_max * D;
  const float *ks = p.hist.scales + kr * p.hist.blocks, *vs = p.hist.scales + vr * p.hist.blocks;
  auto value = [](uint8_t c) { return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3))); };
  for (int j = 0; j <= pos; ++j) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) s += q[e] * value(kc[(size_t)j * D + lane * kPer + e]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= ks[j >> p.hist.shift] * p.scale2;
    const float top = fmaxf(m, s), a = exp2f(m - top), w = exp2f(s - top), v = vs[j >> p.hist.shift];
    m = top;
    l = l * a + w;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = acc[e] * a + w * (v * value(vc[(size_t)j * D + lane * kPer + e]));
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) out[e] = (T)(acc[e] / l);
}

// The sequences of `from` that have a length to keep.
template <typename F>
static void keep(SeqBatch* to, const SeqBatch from, F want) {
  to->n = 0;
  to->cum[0] = 0;
  for (int i = 0; i < from.n; ++i) {
    if (!want(from.len(i))) continue;
    to->begin[to->n] = from.begin[i];
    to->slot[to->n] = from.slot[i];
    to->start[to->n] = from.start[i];
    to->cum[to->n + 1] = to->cum[to->n] + from.len(i);
    ++to->n;
  }
}

static int attention(wave_t* h, HistoryAttnParams& p, int tokens, int type, const void* q, int64_t q_stride, float scale,
                     void* out, int64_t out_stride, void* stream) {
  const int H = h->pl.cfg.n_heads, D = h->pl.cfg.head_dim;
  if (!q || !out || (type != WAVE_BF16 && type != WAVE_F16)) return WAVE_EINVAL;
  const float scale2 = scale * 1.44269504088896340736f;  // log2(e)
  if (!(scale > 0.f) || !isfinite(scale2)) return WAVE_EINVAL;
  const int64_t strides[2] = {q_stride, out_stride};
  for (int64_t s : strides)
    if (s < (int64_t)H * D || s % 8 || s > kMaxStride) return WAVE_EINVAL;
  if (!aligned16(q) || !aligned16(out) || H / p.hist.heads > kMaxGroup) return WAVE_EINVAL;
  if (!on_device(h)) return WAVE_EINVAL;
  if (tokens == 0) return WAVE_OK;
  p.heads = H;
  p.group = H / p.hist.heads;
  p.q = (const uint16_t*)q;
  p.out = (uint16_t*)out;
  p.q_stride = q_stride;
  p.out_stride = out_stride;
  p.scale2 = scale2;
  p.err = h->ws.err;
  p.err_out = h->err_host_dev;
  cudaStream_t st = (cudaStream_t)stream;
  h->last_stream = st;
  // Sequences whose rows fit one tile of few rows, and the others.
  HistoryAttnParams many = p;
  if (p.positions) {
    p.n = tokens;
    many.b.n = 0;
  } else {
    keep(&p.b, many.b, [&](int len) { return (long long)len * p.group <= kFewRows; });
    keep(&many.b, many.b, [&](int len) { return (long long)len * p.group > kFewRows; });
    p.n = p.b.n;
  }
  p.part = h->ws.part_o;
  p.part_cnt = h->ws.hist_cnt;
  if (p.n) {
    const cudaError_t e = launch_history_few(p, D, type, h->pl.grid, st);
    if (e != cudaSuccess) return WAVE_ECUDA;
  }
  if (many.b.n) {
    const int rows = many.b.cum[many.b.n];
    const unsigned ctas = (unsigned)(((long long)rows * H + 7) / 8);
    if (D == 128)
      type == WAVE_F16 ? k_history_attention<128, __half><<<ctas, 256, 0, st>>>(many, rows)
                       : k_history_attention<128, __nv_bfloat16><<<ctas, 256, 0, st>>>(many, rows);
    else
      type == WAVE_F16 ? k_history_attention<64, __half><<<ctas, 256, 0, st>>>(many, rows)
                       : k_history_attention<64, __nv_bfloat16><<<ctas, 256, 0, st>>>(many, rows);
  }
  return cudaGetLastError() == cudaSuccess ? WAVE_OK : WAVE_ECUDA;
}

}  // namespace wave

extern "C" int wave_history_attention(wave_t* h, int layer, int n_seq, const int32_t* cu_seqlens, const int32_t* slots,
                                      const int32_t* starts, int type, const void* q, int64_t q_stride, const uint8_t* kv_fp8,
                                      const float* kv_scales, int n_kv_heads, int block, float scale, void* out,
                                      int64_t out_stride, void* stream) {
  HistoryAttnParams p;
  int rc = make_history(&p.hist, h, layer, n_kv_heads, block, kv_fp8, kv_scales);
  if (!rc) rc = make_batch(&p.b, n_seq, cu_seqlens, slots, starts, h->pl.S_max);
  if (rc) return rc;
  for (int i = 0; i < p.b.n; ++i)
    if (p.b.start[i] > h->pl.T_max - p.b.len(i)) return WAVE_EPOS;
  p.positions = nullptr;
  return attention(h, p, p.b.cum[p.b.n], type, q, q_stride, scale, out, out_stride, stream);
}

extern "C" int wave_history_attention_frame(wave_t* h, int layer, int S, const int32_t* positions, int type, const void* q,
                                            int64_t q_stride, const uint8_t* kv_fp8, const float* kv_scales, int n_kv_heads,
                                            int block, float scale, void* out, int64_t out_stride, void* stream) {
  HistoryAttnParams p;
  const int rc = make_history(&p.hist, h, layer, n_kv_heads, block, kv_fp8, kv_scales);
  if (rc) return rc;
  if (S < 1 || S > h->pl.S_max || !positions || ((uintptr_t)positions & 3)) return WAVE_EINVAL;
  p.b.n = 0;
  p.b.cum[0] = 0;
  p.positions = positions;
  return attention(h, p, S, type, q, q_stride, scale, out, out_stride, stream);
}
