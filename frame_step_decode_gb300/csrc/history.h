// history.h -- what the calls on rotary positions and on the block-scaled
// history share: the turn of a pair at a position, the history's layout, and
// their checks on the host.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/wave.h"
#include "ctx.h"
#include "fp8.cuh"
#include "prompt.h"

namespace wave {

// ---- rotary positions

// The cosine and sine of `pos` times a frequency that is held as a fraction of
// a turn in 64 bits: the product's low 64 bits are the angle modulo a turn,
// exact for every position, so that far ones lose nothing.  The angle is
// brought into an eighth of a turn to either side of a quarter first, where
// fp32 holds it to 2^-25.
__device__ __forceinline__ float2 turn_at(uint64_t turns, uint32_t pos, float amplitude) {
  const int32_t a = (int32_t)((turns * pos) >> 32);  // 2^32 to a turn
  const int32_t q = (int32_t)((uint32_t)a + (1u << 29)) >> 30;
  const int32_t r = (int32_t)((uint32_t)a - ((uint32_t)q << 30));
  float s, c;
  sincospif((float)r * 0x1p-31f, &s, &c);
  const float x = q & 1 ? s : c, y = q & 1 ? c : s;
  return make_float2((q + 1) & 2 ? -x * amplitude : x * amplitude, q & 2 ? -y * amplitude : y * amplitude);
}

inline bool rope_ok(const wave_rope* r, int head_dim) {
  return (r->layout == WAVE_ROPE_HALF || r->layout == WAVE_ROPE_INTERLEAVED) && r->dims >= 16 && r->dims <= head_dim &&
         r->dims % 16 == 0;
}

// A head's values are worked on sixteen at a time, two groups of eight: those
// that a half layout pairs (8 j and 8 j + dims / 2), or neighbours.
template <typename Rope>
__device__ __forceinline__ void groups_of_item(const Rope& r, int item, int& a, int& b, bool& turned) {
  turned = item < r.dims / 16;
  if (turned && r.layout == WAVE_ROPE_HALF) {
    a = item;
    b = item + r.dims / 16;
  } else {
    a = 2 * item;
    b = a + 1;
  }
}

// x[0..7] and x[8..15] (groups a and b) turned by the item's eight pairs; cs
// holds them as four of two, `stride` apart.
template <bool kHalf>
__device__ __forceinline__ void turn_pairs(float* x, const float4* cs, int stride) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 t = cs[k * stride];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * k + e;  // the pair
      const float c = e ? t.z : t.x, s = e ? t.w : t.y;
      const int p = kHalf ? i : 2 * i, q = kHalf ? i + 8 : 2 * i + 1;
      const float u = x[p], v = x[q];
      x[p] = u * c - v * s;
      x[q] = u * s + v * c;
    }
  }
}
__device__ __forceinline__ void turn_item(float* x, const float4* cs, int stride, bool half) {
  if (half)
    turn_pairs<true>(x, cs, stride);
  else
    turn_pairs<false>(x, cs, stride);
}

// ---- eight values of a row

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* x);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float* x) {
  const float4 a = *(const float4*)p, b = *(const float4*)(p + 4);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float* x) {
  const uint4 u = *(const uint4*)p;
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
template <>
__device__ __forceinline__ void load8<__half>(const __half* p, float* x) {
  const uint4 u = *(const uint4*)p;
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*(const __half2*)&w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <typename T>
__device__ __forceinline__ uint32_t pair16(float a, float b);
template <>
__device__ __forceinline__ uint32_t pair16<__nv_bfloat16>(float a, float b) {
  __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *(uint32_t*)&t;
}
template <>
__device__ __forceinline__ uint32_t pair16<__half>(float a, float b) {
  __half2 t = __floats2half2_rn(a, b);
  return *(uint32_t*)&t;
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float* x) {
  *(uint4*)p = make_uint4(pair16<T>(x[0], x[1]), pair16<T>(x[2], x[3]), pair16<T>(x[4], x[5]), pair16<T>(x[6], x[7]));
}
template <>
__device__ __forceinline__ void store8<float>(float* p, const float* x) {
  *(float4*)p = make_float4(x[0], x[1], x[2], x[3]);
  *(float4*)(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// Sixteen values of a row as they come from memory, two groups of eight.
template <typename T>
struct Raw16 {
  uint4 v[sizeof(T)];  // 2 for 16-bit types, 4 for fp32
  __device__ __forceinline__ void load(const T* row, int a, int b) {
    constexpr int n = sizeof(T) / 2;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      v[i] = *((const uint4*)(row + 8 * a) + i);
      v[n + i] = *((const uint4*)(row + 8 * b) + i);
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float* x) const {
    load8<T>((const T*)v, x);
    load8<T>((const T*)(v + sizeof(T) / 2), x + 8);
  }
};

// ---- the history

// One layer: codes [2][S_max][heads][T_max][D], scales [2][S_max][heads][blocks].
struct History {
  uint8_t* codes;
  float* scales;
  int S_max, heads, T_max, block, shift, blocks;  // block = 1 << shift
  // the row of scales of (K or V, slot, head); its codes begin at row * T_max * D
  __device__ __forceinline__ size_t row(int which, int slot, int head) const {
    return ((size_t)which * S_max + slot) * heads + head;
  }
};

constexpr int kMaxGroup = 128;  // query heads to a K/V head in attention

inline bool block_ok(int block) { return block == 1 || (block >= 16 && block <= 128 && (block & (block - 1)) == 0); }

// The arguments that name a layer's history; WAVE_OK, or WAVE_EINVAL.
inline int make_history(History* v, const wave_ctx* h, int layer, int n_kv_heads, int block, const uint8_t* kv,
                        const float* scales) {
  if (!h || !kv || !scales) return WAVE_EINVAL;
  const Plan& pl = h->pl;
  int la = layer;  // the history's layer
  if (pl.hybrid) {
    const int e = pl.hcfg.attn_every;
    if (layer < 0 || layer >= pl.hcfg.n_layers || layer % e != e - 1) return WAVE_EINVAL;
    la = layer / e;
  }
  if (la < 0 || la >= pl.cfg.n_layers) return WAVE_EINVAL;
  if (n_kv_heads < 1 || pl.cfg.n_heads % n_kv_heads || !block_ok(block) || !aligned16(kv) || !aligned16(scales))
    return WAVE_EINVAL;
  v->S_max = pl.S_max;
  v->heads = n_kv_heads;
  v->T_max = pl.T_max;
  v->block = block;
  v->shift = 0;
  while ((1 << v->shift) < block) ++v->shift;
  v->blocks = (pl.T_max + block - 1) / block;
  const size_t rows = (size_t)la * 2 * pl.S_max * n_kv_heads;
  v->codes = (uint8_t*)kv + rows * pl.T_max * pl.cfg.head_dim;
  v->scales = (float*)scales + rows * v->blocks;
  return WAVE_OK;
}

// The least power of two s with amax <= 448 s, no smaller than the least
// ordinary number; 0 for 0.
__device__ __forceinline__ float block_scale(float amax) {
  if (amax == 0.f) return 0.f;
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u);  // 448 = 1.75 * 2^8
  return __uint_as_float((uint32_t)(max(e, -126) + 127) << 23);
}

// What a value counts for in its block's largest magnitude: values that are
// not finite only keep the scale from being 0.
__device__ __forceinline__ float counts(float v) {
  const float a = fabsf(v);
  return a < __int_as_float(0x7F800000) ? a : 0x1p-126f;
}

// Eight codes of x * inv.  Infinities saturate, NaN stays NaN.
__device__ __forceinline__ uint2 codes8(const float* x, float inv) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x[4 * i] * inv, x[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3) |
           (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2] * inv, x[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3)
               << 16;
  return make_uint2(w[0], w[1]);
}
// Eight codes of x / scale.  1 / scale is exact for the powers of two that
// blocks have; inv is 0 for a scale of 0, whose codes are 0 (without a sign).
__device__ __forceinline__ uint2 encode8(const float* x, float inv) { return inv == 0.f ? make_uint2(0, 0) : codes8(x, inv); }
__device__ __forceinline__ void decode8(uint2 c, float* x) {
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t lo, hi;
    e4m3x4_to_f16x2x2(w[i], lo, hi);
    const float2 a = __half22float2(*(__half2*)&lo), b = __half22float2(*(__half2*)&hi);
    x[4 * i] = a.x, x[4 * i + 1] = a.y, x[4 * i + 2] = b.x, x[4 * i + 3] = b.y;
  }
}

// Reports a position at or beyond T_max (see wave_status).
__device__ __forceinline__ void bad_position(int* err, int* err_out) { *(volatile int*)err_out = atomicOr(err, kErrPos) | kErrPos; }

}  // namespace wave
