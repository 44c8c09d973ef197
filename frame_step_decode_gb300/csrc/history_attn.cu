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

#include <algorithm>

#include "../../include/wave.h"
#include "history_attn.h"

using namespace wave;

namespace wave {

// The sequences of `from` that have a length to keep.
template <typename F>
static void keep(SeqBatch* to, const SeqBatch& from, F want) {
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
  // Sequences of few rows, and the others.  Where there are others, few rows with
  // no more than two blocks of 128 keys for each SM go along with them: a launch
  // of their own costs more.  300 tokens after 1000 with one prompt of 4 after 500
  // (32 blocks), 32/8 heads of 128: 23.9 us, apart 36.0; with nine of them (288) 31.6
  // and 38.8; 2001 after 4096 with 36 of 4 after 100 (288) 178 and 182; 300 with two of
  // 20 after 500, 32 heads, at 320 blocks, where both take 50, apart.
  HistoryAttnParams many = p;
  if (p.positions) {
    p.n = tokens;
    many.b.n = 0;
  } else {
    auto few = [&](int len) { return (long long)len * p.group <= kFewRows; };
    long long blocks = 0;
    bool others = false;
    for (int i = 0; i < p.b.n; ++i) {
      const int len = p.b.len(i);
      if (few(len))
        blocks += (long long)p.hist.heads * ((p.b.start[i] + len + 127) / 128);
      else
        others = true;
    }
    if (others && blocks <= 2LL * h->pl.grid) {
      p.b.n = 0;
    } else {
      const SeqBatch all = p.b;
      keep(&p.b, all, few);
      keep(&many.b, all, [&](int len) { return !few(len); });
    }
    p.n = p.b.n;
  }
  p.part = h->ws.part_o;
  p.part_cnt = h->ws.hist_cnt;
  if (p.n) {
    int rows = p.group;
    for (int i = 0; i < p.b.n; ++i) rows = std::max(rows, p.b.len(i) * p.group);
    const cudaError_t e = launch_history_few(p, D, type, rows, h->pl.grid, st);
    if (e != cudaSuccess) return WAVE_ECUDA;
  }
  if (many.b.n && launch_history_many(many, h, type, st) != cudaSuccess) return WAVE_ECUDA;
  return WAVE_OK;
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
