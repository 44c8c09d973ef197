// prompt.cu -- wave_prompt_append: rotary embedding, FP8 quantisation and
// append of packed prompts to the sessions' history.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/wave.h"
#include "ctx.h"
#include "fp8.cuh"
#include "prompt.h"
#include "quotient.cuh"

using namespace wave;

namespace wave {

struct AppendParams {
  SeqBatch b;
  int H, S_max, T_max, layer;
  long long stride;      // elements between tokens of qkv
  const void* qkv;
  const float2* rope;    // [T_max][D/2]
  uint8_t* kv;
  float* scales;
  void *q, *k, *v;       // [rows][H][D] 16-bit, or null
};

constexpr int kAppendThreads = 128;

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
  return __ldg((const float4*)p);
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 u = __ldg((const uint2*)p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xFFFF0000u));
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *(uint32_t*)&t;
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  __half2 t = __floats2half2_rn(a, b);
  return *(uint32_t*)&t;
}
template <typename T>
__device__ __forceinline__ void store4(void* base, size_t at, const float* v) {
  *(uint2*)((T*)base + at) = make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
}

// A group of D/4 lanes per (token, head): four values of q, k and v each.
// The arithmetic is the step's append (rotate-half pairs (i, i + D/2), scale
// amax/448, code E4M3(v/scale) by an IEEE division), so that a prompt leaves
// the history that stepping through it would have left.  Bound by HBM: a CTA
// takes the same few heads of neighbouring tokens, so that the history's rows
// it writes lie together (16 prompts, 8005 tokens, 32 heads of 128, qkv fp32:
// 110 us = 5.99 TB/s; with the heads of one token in a CTA 126 us; qkv bf16
// 106 us = 4.35 TB/s: its loads are of 8 bytes a lane).
template <int D, int kHeads, typename In, typename Out>
__global__ void __launch_bounds__(kAppendThreads) k_prompt_append(const __grid_constant__ AppendParams p) {
  constexpr int G = D / 4;  // lanes per row: 32 or 16
  const int lane = threadIdx.x % G;
  const int chunks = (p.H + kHeads - 1) / kHeads;
  const int t = (int)(blockIdx.x / chunks) * (kAppendThreads / G) + (int)threadIdx.x / G;
  const int h0 = (int)(blockIdx.x % chunks) * kHeads;
  const bool live = t < p.b.cum[p.b.n];  // the shuffles below need whole warps
  const int i = live ? seq_of(p.b, t) : 0;
  const int at = live ? t - p.b.cum[i] : 0;
  const int row = p.b.begin[i] + at, pos = p.b.start[i] + at, slot = p.b.slot[i];
  const In* src = (const In*)p.qkv + (size_t)row * p.stride + lane * 4;
  const int HD = p.H * D;
  float c[4], s[4];
  {
    const float4* tab = (const float4*)(p.rope + (size_t)pos * (D / 2) + (lane % (G / 2)) * 4);
    const float4 a = __ldg(tab), b = __ldg(tab + 1);
    c[0] = a.x, s[0] = a.y, c[1] = a.z, s[1] = a.w;
    c[2] = b.x, s[2] = b.y, c[3] = b.z, s[3] = b.w;
  }
#pragma unroll
  for (int hh = 0; hh < kHeads; ++hh) {
    const int h = h0 + hh;
    const bool on = live && h < p.H;
    float x[3][4];
#pragma unroll
    for (int w = 0; w < 3; ++w) {
      const float4 v = on ? load4<In>(src + w * HD + h * D) : make_float4(0.f, 0.f, 0.f, 0.f);
      x[w][0] = v.x, x[w][1] = v.y, x[w][2] = v.z, x[w][3] = v.w;
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float y = __shfl_xor_sync(0xffffffffu, x[w][e], G / 2);
        x[w][e] = lane < G / 2 ? x[w][e] * c[e] - y * s[e] : y * s[e] + x[w][e] * c[e];
      }
    }
    const size_t o = ((size_t)row * p.H + h) * D + lane * 4;
    if (on && p.q) store4<Out>(p.q, o, x[0]);
#pragma unroll
    for (int w = 0; w < 2; ++w) {  // K, V
      float* v = x[1 + w];
      float amax = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
      for (int d = G / 2; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
      const float sc = __fdiv_rn(amax, 448.0f);
      const uint32_t codes = encode4(v, sc);
      if (!on) continue;
      const size_t r = ((((size_t)p.layer * 2 + w) * p.S_max + slot) * p.H + h) * p.T_max + pos;
      *(uint32_t*)(p.kv + r * D + lane * 4) = codes;
      if (lane == 0) p.scales[r] = sc;
      void* back = w ? p.v : p.k;
      if (back) {  // what the history now holds, rounded once to 16 bits
        uint32_t lo, hi;
        e4m3x4_to_f16x2x2(codes, lo, hi);
        const float2 a = __half22float2(*(__half2*)&lo), b = __half22float2(*(__half2*)&hi);
        const float z[4] = {a.x * sc, a.y * sc, b.x * sc, b.y * sc};
        store4<Out>(back, o, z);
      }
    }
  }
}

template <int D, typename In, typename Out>
static void launch_append(const AppendParams& p, int sms, cudaStream_t st) {
  // Many tokens: four heads to a group of lanes, their 12 loads in flight
  // together.  Few: one, a shorter chain (25 tokens of 16 heads of 64: 2.7
  // against 6.3 us; 32 heads of 128, qkv fp32, 300 tokens: 6.4 / 6.4, 1200:
  // 20.0 / 18.4, 16 x 511: 141 / 113).
  constexpr int kHeads = 4;
  const long long per_cta = kAppendThreads / (D / 4), groups = ((long long)p.b.cum[p.b.n] + per_cta - 1) / per_cta;
  const long long ctas = groups * ((p.H + kHeads - 1) / kHeads);
  if (ctas < 4 * sms)
    k_prompt_append<D, 1, In, Out><<<(unsigned)(groups * p.H), kAppendThreads, 0, st>>>(p);
  else
    k_prompt_append<D, kHeads, In, Out><<<(unsigned)ctas, kAppendThreads, 0, st>>>(p);
}

template <int D>
static void launch_append_types(const AppendParams& p, int in, int out, int sms, cudaStream_t st) {
  if (in == WAVE_F32)
    out == WAVE_BF16 ? launch_append<D, float, __nv_bfloat16>(p, sms, st) : launch_append<D, float, __half>(p, sms, st);
  else
    out == WAVE_BF16 ? launch_append<D, __nv_bfloat16, __nv_bfloat16>(p, sms, st)
                     : launch_append<D, __nv_bfloat16, __half>(p, sms, st);
}

}  // namespace wave

extern "C" int wave_prompt_append(wave_t* h, int layer, int n_seq, const int32_t* cu_seqlens, const int32_t* slots,
                                  const int32_t* starts, const void* qkv, int qkv_type, int64_t row_stride,
                                  uint8_t* kv_fp8, float* kv_scales, void* q, void* k, void* v, int out_type,
                                  void* stream) {
  if (!h || !qkv || !kv_fp8 || !kv_scales) return WAVE_EINVAL;
  const Plan& pl = h->pl;
  const int H = pl.cfg.n_heads, D = pl.cfg.head_dim;
  int la = layer;  // the history's layer
  if (pl.hybrid) {
    const int e = pl.hcfg.attn_every;
    if (layer < 0 || layer >= pl.hcfg.n_layers || layer % e != e - 1) return WAVE_EINVAL;
    la = layer / e;
  }
  if (la < 0 || la >= pl.cfg.n_layers) return WAVE_EINVAL;
  if ((qkv_type != WAVE_F32 && qkv_type != WAVE_BF16) || (out_type != WAVE_BF16 && out_type != WAVE_F16))
    return WAVE_EINVAL;
  if (row_stride < 3LL * H * D || row_stride % 8 || row_stride > kMaxStride || !aligned16(qkv) || !aligned16(kv_fp8) ||
      !aligned16(kv_scales) || !aligned16(q) || !aligned16(k) || !aligned16(v))
    return WAVE_EINVAL;
  AppendParams p;
  const int rc = make_batch(&p.b, n_seq, cu_seqlens, slots, starts, pl.S_max);
  if (rc) return rc;
  for (int i = 0; i < p.b.n; ++i)
    if (p.b.start[i] > pl.T_max - p.b.len(i)) return WAVE_EPOS;
  if (!on_device(h)) return WAVE_EINVAL;
  if (p.b.n == 0) return WAVE_OK;
  p.H = H;
  p.S_max = pl.S_max;
  p.T_max = pl.T_max;
  p.layer = la;
  p.stride = row_stride;
  p.qkv = qkv;
  p.rope = h->ws.rope;
  p.kv = kv_fp8;
  p.scales = kv_scales;
  p.q = q;
  p.k = k;
  p.v = v;
  cudaStream_t st = (cudaStream_t)stream;
  h->last_stream = st;
  if (D == 128)
    launch_append_types<128>(p, qkv_type, out_type, pl.grid, st);
  else
    launch_append_types<64>(p, qkv_type, out_type, pl.grid, st);
  return cudaGetLastError() == cudaSuccess ? WAVE_OK : WAVE_ECUDA;
}
