// prompt_state.cu -- wave_hybrid_prompt_state: the hybrid's selective-state
// block over packed prompts.  Per head, with dt_t = softplus(dt_t + dt_bias)
// and a_t = exp(-exp(A_log) dt_t):
//
//   h_t = a_t h_{t-1} + dt_t x_t B_t^T,   y_t = h_t C_t + D x_t,   out_t = bf16(y_t silu(z_t))
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/wave.h"
#include "ctx.h"
#include "prompt.h"

using namespace wave;

namespace wave {

struct StateParams {
  SeqBatch b;
  int Hs, S_max;
  const uint16_t* zx;      // [rows][zx_stride] bf16: z | x | B | C | dt
  const uint16_t* prm;     // A_log[Hs] | dt_bias[Hs] | D[Hs]
  const float* state_in;   // the layer's [S_max][Hs][64][128]
  float* state_out;
  uint16_t* out;           // [rows][out_stride] bf16
  long long zx_stride, out_stride;
};

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// The recurrent form: a CTA per (sequence, head), its 64 x 128 state in
// registers (warp w: rows 8w..8w+7, lane: states 4 lane..+3).
__global__ void __launch_bounds__(256) k_prompt_state_rows(const __grid_constant__ StateParams p) {
  const int h = blockIdx.x, i = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int di = p.Hs * kSsmP, n = p.b.len(i);
  const size_t base = ((size_t)p.b.slot[i] * p.Hs + h) * (kSsmP * kSsmN) + (size_t)warp * 8 * kSsmN + 4 * lane;
  float4 st[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    st[j] = p.b.start[i] > 0 ? __ldcs((const float4*)(p.state_in + base + j * kSsmN)) : make_float4(0.f, 0.f, 0.f, 0.f);
  const float a_neg = -expf(bf(p.prm[h])), bias = bf(p.prm[p.Hs + h]), Dh = bf(p.prm[2 * p.Hs + h]);
  const uint16_t* row = p.zx + (size_t)p.b.begin[i] * p.zx_stride;
  uint16_t* orow = p.out + (size_t)p.b.begin[i] * p.out_stride + h * kSsmP + warp * 8;
  for (int t = 0; t < n; ++t, row += p.zx_stride, orow += p.out_stride) {
    const float raw = bf(row[2 * di + 2 * kSsmN + h]) + bias;
    const float dt = raw > 0.f ? raw + log1pf(expf(-raw)) : log1pf(expf(raw));
    const float a = expf(a_neg * dt);
    const uint2 x0 = *(const uint2*)(row + di + h * kSsmP + warp * 8), x1 = *(const uint2*)(row + di + h * kSsmP + warp * 8 + 4);
    const uint2 Bq = *(const uint2*)(row + 2 * di + 4 * lane), Cq = *(const uint2*)(row + 2 * di + kSsmN + 4 * lane);
    const float4 B = make_float4(bf((uint16_t)Bq.x), bf((uint16_t)(Bq.x >> 16)), bf((uint16_t)Bq.y), bf((uint16_t)(Bq.y >> 16)));
    const float4 C = make_float4(bf((uint16_t)Cq.x), bf((uint16_t)(Cq.x >> 16)), bf((uint16_t)Cq.y), bf((uint16_t)(Cq.y >> 16)));
    const uint32_t xw[4] = {x0.x, x0.y, x1.x, x1.y};
    float x[8], y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = bf((uint16_t)(xw[j / 2] >> (16 * (j & 1))));
      const float u = dt * x[j];
      st[j].x = fmaf(a, st[j].x, u * B.x);
      st[j].y = fmaf(a, st[j].y, u * B.y);
      st[j].z = fmaf(a, st[j].z, u * B.z);
      st[j].w = fmaf(a, st[j].w, u * B.w);
      y[j] = st[j].x * C.x + st[j].y * C.y + st[j].z * C.z + st[j].w * C.w;
    }
    // row sums by recursive halving: lane bits 4, 3, 2 pick the row 4 b4 + 2 b3 + b2
    const bool h4 = lane & 16, h3 = lane & 8, h2 = lane & 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = (h4 ? y[j + 4] : y[j]) + __shfl_xor_sync(0xffffffffu, h4 ? y[j] : y[j + 4], 16);
#pragma unroll
    for (int j = 0; j < 2; ++j) y[j] = (h3 ? y[j + 2] : y[j]) + __shfl_xor_sync(0xffffffffu, h3 ? y[j] : y[j + 2], 8);
    y[0] = (h2 ? y[1] : y[0]) + __shfl_xor_sync(0xffffffffu, h2 ? y[0] : y[1], 4);
    y[0] += __shfl_xor_sync(0xffffffffu, y[0], 2);
    y[0] += __shfl_xor_sync(0xffffffffu, y[0], 1);
    if ((lane & 3) == 0) {
      const int j = (h4 ? 4 : 0) + (h3 ? 2 : 0) + (h2 ? 1 : 0);
      const float xp = bf(row[di + h * kSsmP + warp * 8 + j]), z = bf(row[h * kSsmP + warp * 8 + j]);
      orow[j] = __bfloat16_as_ushort(__float2bfloat16_rn((y[0] + Dh * xp) * z / (1.0f + expf(-z))));
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) __stcs((float4*)(p.state_out + base + j * kSsmN), st[j]);
}

}  // namespace wave

extern "C" int wave_hybrid_prompt_state(wave_t* h, int layer, const void* weights, int n_seq, const int32_t* cu_seqlens,
                                        const int32_t* slots, const int32_t* starts, const void* zxbcdt,
                                        int64_t zx_stride, const float* state_in, float* state_out, void* out,
                                        int64_t out_stride, void* stream) {
  if (!h || !h->pl.hybrid || !weights || !zxbcdt || !state_out || !out) return WAVE_EINVAL;
  const Plan& pl = h->pl;
  const int e = pl.hcfg.attn_every;
  if (layer < 0 || layer >= pl.hcfg.n_layers || layer % e == e - 1) return WAVE_EINVAL;
  if (zx_stride < pl.in_rows || zx_stride % 4 || out_stride < pl.d_inner || out_stride % 8 || !aligned16(weights) ||
      !aligned16(zxbcdt) || !aligned16(state_in) || !aligned16(state_out) || !aligned16(out))
    return WAVE_EINVAL;
  StateParams p;
  const int rc = make_batch(&p.b, n_seq, cu_seqlens, slots, starts, pl.S_max);
  if (rc) return rc;
  for (int i = 0; i < p.b.n; ++i)
    if (p.b.start[i] > 0 && !state_in) return WAVE_EINVAL;
  if (!on_device(h)) return WAVE_EINVAL;
  if (!p.b.n) return WAVE_OK;
  const int Hs = pl.hcfg.ssm_heads, lm = layer - layer / e;
  const size_t per_layer = (size_t)pl.S_max * Hs * kSsmP * kSsmN;
  p.Hs = Hs;
  p.S_max = pl.S_max;
  p.zx = (const uint16_t*)zxbcdt;
  p.prm = (const uint16_t*)weights + hyb_layer_offset(pl.pk_M, pl.pk_layer, e, layer) + pl.pk_a_log;
  p.state_in = state_in ? state_in + lm * per_layer : nullptr;
  p.state_out = state_out + lm * per_layer;
  p.out = (uint16_t*)out;
  p.zx_stride = zx_stride;
  p.out_stride = out_stride;
  cudaStream_t st = (cudaStream_t)stream;
  h->last_stream = st;
  k_prompt_state_rows<<<dim3(Hs, p.b.n), 256, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? WAVE_OK : WAVE_ECUDA;
}
