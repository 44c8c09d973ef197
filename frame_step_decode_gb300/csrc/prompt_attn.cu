// prompt_attn.cu -- wave_prompt_attention: causal attention over packed
// prompts with grouped heads.
//
//   o_i = sum_{j <= i} p_ij v_j / sum_{j <= i} p_ij,   p_ij = exp(scale q_i.k_j - m_i)
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/wave.h"
#include "ctx.h"
#include "prompt.h"
#include "ptx.cuh"

using namespace wave;

namespace wave {

struct AttnParams {
  SeqBatch b;
  int Hq, group;  // query heads, and how many of them share a K/V head
  const void *q, *k, *v;
  void* out;
  long long q_stride, k_stride, v_stride, out_stride;
  float scale2;   // scale * log2(e)
};

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// A warp per (token, head), a running maximum and sum over the keys.
template <int D, typename T>
__global__ void __launch_bounds__(256) k_prompt_attention_rows(const __grid_constant__ AttnParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int t = (int)(w / p.Hq), h = (int)(w % p.Hq);
  if (t >= p.b.cum[p.b.n]) return;
  const int i = seq_of(p.b, t), at = t - p.b.cum[i];
  const size_t first = p.b.begin[i];
  const T* q = (const T*)p.q + (first + at) * p.q_stride + h * D + lane * E;
  const T* k = (const T*)p.k + first * p.k_stride + (h / p.group) * D + lane * E;
  const T* v = (const T*)p.v + first * p.v_stride + (h / p.group) * D + lane * E;
  float qv[E], o[E] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) qv[e] = to_f32<T>(q[e]) * p.scale2;
  for (int j = 0; j <= at; ++j) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += qv[e] * to_f32<T>(k[(size_t)j * p.k_stride + e]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    const float m2 = fmaxf(m, s), a = m == m2 ? 1.f : ex2(m - m2), w2 = ex2(s - m2);
    m = m2;
    l = l * a + w2;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * a + w2 * to_f32<T>(v[(size_t)j * p.v_stride + e]);
  }
  T* out = (T*)p.out + (first + at) * p.out_stride + h * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = from_f32<T>(o[e] / l);
}

}  // namespace wave

extern "C" int wave_prompt_attention(wave_t* h, int n_seq, const int32_t* cu_seqlens, int n_kv_heads, int type,
                                     const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                     int64_t v_stride, float scale, void* out, int64_t out_stride, void* stream) {
  if (!h || !q || !k || !v || !out || !cu_ok(n_seq, cu_seqlens)) return WAVE_EINVAL;
  const int H = h->pl.cfg.n_heads, D = h->pl.cfg.head_dim;
  if (n_kv_heads < 1 || H % n_kv_heads || (type != WAVE_BF16 && type != WAVE_F16)) return WAVE_EINVAL;
  if (!(scale > 0.f) || !isfinite(scale)) return WAVE_EINVAL;
  const int64_t least[4] = {(int64_t)H * D, (int64_t)n_kv_heads * D, (int64_t)n_kv_heads * D, (int64_t)H * D};
  const int64_t strides[4] = {q_stride, k_stride, v_stride, out_stride};
  const void* ptrs[4] = {q, k, v, out};
  for (int i = 0; i < 4; ++i)
    if (strides[i] < least[i] || strides[i] % 8 || strides[i] >= (1LL << 31) || !aligned16(ptrs[i])) return WAVE_EINVAL;
  if (!on_device(h)) return WAVE_EINVAL;
  AttnParams p;
  p.b.n = 0;
  p.b.cum[0] = 0;
  for (int i = 0; i < n_seq; ++i) {
    const int len = cu_seqlens[i + 1] - cu_seqlens[i];
    if (!len) continue;
    p.b.begin[p.b.n] = cu_seqlens[i];
    p.b.cum[p.b.n + 1] = p.b.cum[p.b.n] + len;
    ++p.b.n;
  }
  if (!p.b.n) return WAVE_OK;
  p.Hq = H;
  p.group = H / n_kv_heads;
  p.q = q;
  p.k = k;
  p.v = v;
  p.out = out;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.out_stride = out_stride;
  p.scale2 = scale * 1.44269504088896340736f;
  cudaStream_t st = (cudaStream_t)stream;
  h->last_stream = st;
  const long long warps = (long long)p.b.cum[p.b.n] * H;
  const unsigned grid = (unsigned)((warps + 7) / 8);
  if (D == 128)
    type == WAVE_BF16 ? k_prompt_attention_rows<128, __nv_bfloat16><<<grid, 256, 0, st>>>(p)
                      : k_prompt_attention_rows<128, __half><<<grid, 256, 0, st>>>(p);
  else
    type == WAVE_BF16 ? k_prompt_attention_rows<64, __nv_bfloat16><<<grid, 256, 0, st>>>(p)
                      : k_prompt_attention_rows<64, __half><<<grid, 256, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? WAVE_OK : WAVE_ECUDA;
}
