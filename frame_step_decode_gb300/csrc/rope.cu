// rope.cu -- wave_rope_plan, wave_rope_apply, wave_rope_apply_at: rotary
// positions on packed rows.
//
//   (a, b) -> amplitude (a cos - b sin, a sin + b cos),  angle = position * frequency of the pair
//
// Measured (captured launches in a row): 8005 tokens of 40 heads of 128, bf16,
// 31 us = 5.3 TB/s of mixed reads and writes; 25 tokens of 32 heads of 64, 2.8 us.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/wave.h"
#include "history.h"

using namespace wave;

namespace wave {

struct RopeParams {
  SeqBatch b;
  const int32_t* positions;  // rows' positions on the device, or null
  long long tokens;
  wave_rope rope;
  int heads;
  const void* x;
  void* out;
  long long x_stride, out_stride;
};

constexpr int kRopeThreads = 256, kRopeRows = 4;

// Bound by HBM, x read and out written once.  A CTA takes four rows: a thread
// has the same sixteen values of each, whose loads are in flight while the turns
// of the rows' positions are made, into shared memory, for all their heads.
template <int D, typename In, typename Out>
__global__ void __launch_bounds__(kRopeThreads) k_rope(const __grid_constant__ RopeParams p) {
  __shared__ float4 turns[kRopeRows][D / 4];  // [row][4][dims / 16]: the items' pairs, two by two
  const int pairs = p.rope.dims / 2, per = p.rope.dims / 16;
  const long long first = (long long)blockIdx.x * kRopeRows;
  const int rows = (int)min((long long)kRopeRows, p.tokens - first);
  long long at[kRopeRows];  // the row in the buffers, or -1
  int pos[kRopeRows];
#pragma unroll
  for (int r = 0; r < kRopeRows; ++r) {
    at[r] = -1;
    pos[r] = 0;
    if (r >= rows) continue;
    if (p.positions) {
      pos[r] = p.positions[first + r];
      if (pos[r] >= 0) at[r] = first + r;
    } else {
      const int t = (int)first + r, s = seq_of(p.b, t), n = t - p.b.cum[s];
      at[r] = p.b.begin[s] + n;
      pos[r] = p.b.start[s] + n;
    }
  }
  constexpr int kItems = D / 16;
  const int items = p.heads * kItems;
  const bool half = p.rope.layout == WAVE_ROPE_HALF;
  for (int i = threadIdx.x; i < (items + (int)blockDim.x - 1) / (int)blockDim.x * (int)blockDim.x; i += blockDim.x) {
    const int head = i / kItems, item = i % kItems;
    int a, b;
    bool turned;
    groups_of_item(p.rope, item, a, b, turned);
    Raw16<In> raw[kRopeRows];
    if (i < items) {
#pragma unroll
      for (int r = 0; r < kRopeRows; ++r)
        if (at[r] >= 0) raw[r].load((const In*)p.x + at[r] * p.x_stride + head * D, a, b);
    }
    if (i < (int)blockDim.x) {  // once
      for (int k = threadIdx.x; k < kRopeRows * pairs; k += blockDim.x) {
        const int r = k / pairs, j = k - r * pairs, t = r == 0 ? pos[0] : r == 1 ? pos[1] : r == 2 ? pos[2] : pos[3];
        ((float2*)turns[r])[(j % 8 / 2 * per + j / 8) * 2 + j % 2] = turn_at(p.rope.turns[j], (uint32_t)max(t, 0), p.rope.amplitude);
      }
      __syncthreads();
    }
    if (i >= items) continue;
#pragma unroll
    for (int r = 0; r < kRopeRows; ++r) {
      if (at[r] < 0) continue;
      float x[16];
      raw[r].get(x);
      if (turned) turn_item(x, &turns[r][item], per, half);
      Out* dst = (Out*)p.out + at[r] * p.out_stride + head * D;
      store8<Out>(dst + 8 * a, x);
      store8<Out>(dst + 8 * b, x + 8);
    }
  }
}

template <int D, typename In>
static void launch_rope(const RopeParams& p, int out_type, unsigned ctas, cudaStream_t st) {
  const unsigned threads = std::min(kRopeThreads, (p.heads * (D / 16) + 31) / 32 * 32);
  if (out_type == WAVE_F32)
    k_rope<D, In, float><<<ctas, threads, 0, st>>>(p);
  else if (out_type == WAVE_BF16)
    k_rope<D, In, __nv_bfloat16><<<ctas, threads, 0, st>>>(p);
  else
    k_rope<D, In, __half><<<ctas, threads, 0, st>>>(p);
}
template <int D>
static void launch_rope_in(const RopeParams& p, int type, int out_type, unsigned ctas, cudaStream_t st) {
  if (type == WAVE_F32)
    launch_rope<D, float>(p, out_type, ctas, st);
  else if (type == WAVE_BF16)
    launch_rope<D, __nv_bfloat16>(p, out_type, ctas, st);
  else
    launch_rope<D, __half>(p, out_type, ctas, st);
}

static bool type_ok(int t) { return t == WAVE_F32 || t == WAVE_BF16 || t == WAVE_F16; }

static int apply(RopeParams& p, const wave_rope* rope, int n_heads, int head_dim, const void* x, int type, int64_t x_stride,
                 void* out, int out_type, int64_t out_stride, void* stream) {
  if (!rope || !x || !out || n_heads < 1 || n_heads > 65536 || (head_dim != 64 && head_dim != 128) || !rope_ok(rope, head_dim) ||
      !type_ok(type) || !type_ok(out_type))
    return WAVE_EINVAL;
  const int64_t width = (int64_t)n_heads * head_dim;
  const int64_t strides[2] = {x_stride, out_stride};
  for (int64_t s : strides)
    if (s < width || s % 8 || s > kMaxStride) return WAVE_EINVAL;
  if (!aligned16(x) || !aligned16(out) || (x == out && (type != out_type || x_stride != out_stride))) return WAVE_EINVAL;
  if (p.tokens == 0) return WAVE_OK;
  p.rope = *rope;
  p.heads = n_heads;
  p.x = x;
  p.out = out;
  p.x_stride = x_stride;
  p.out_stride = out_stride;
  const long long ctas = (p.tokens + kRopeRows - 1) / kRopeRows;
  if (ctas > 0x7fffffff) return WAVE_EINVAL;
  if (head_dim == 128)
    launch_rope_in<128>(p, type, out_type, (unsigned)ctas, (cudaStream_t)stream);
  else
    launch_rope_in<64>(p, type, out_type, (unsigned)ctas, (cudaStream_t)stream);
  return cudaGetLastError() == cudaSuccess ? WAVE_OK : WAVE_ECUDA;
}

}  // namespace wave

extern "C" int wave_rope_plan(const wave_rope_config* c, wave_rope* rope) {
  if (!c || !rope) return WAVE_EINVAL;
  if ((c->layout != WAVE_ROPE_HALF && c->layout != WAVE_ROPE_INTERLEAVED) || c->dims < 16 || c->dims > 128 || c->dims % 16)
    return WAVE_EINVAL;
  if (!(c->base > 0.f) || !isfinite(c->base) || !isfinite(c->amplitude)) return WAVE_EINVAL;
  const bool parts = c->scaling == WAVE_ROPE_PARTS;
  if (c->scaling != WAVE_ROPE_PLAIN && c->scaling != WAVE_ROPE_LINEAR && !parts) return WAVE_EINVAL;
  if (c->scaling != WAVE_ROPE_PLAIN && (!(c->factor > 0.f) || !isfinite(c->factor))) return WAVE_EINVAL;
  if (parts && (!(c->original > 0.f) || !isfinite(c->original) || !(c->fast > c->slow) || !(c->slow >= 0.f) || !isfinite(c->fast)))
    return WAVE_EINVAL;
  const double two_pi = 6.283185307179586476925;
  wave_rope r = {};
  for (int i = 0; i < c->dims / 2; ++i) {
    double f = pow((double)c->base, -2.0 * i / c->dims);
    if (c->scaling == WAVE_ROPE_LINEAR) f /= c->factor;
    if (parts) {
      const double g = ((double)c->original * f / two_pi - c->slow) / ((double)c->fast - c->slow);
      const double keep = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
      f = keep * f + (1.0 - keep) * f / c->factor;
    }
    double t = f / two_pi;
    if (!isfinite(t)) return WAVE_EINVAL;
    t -= floor(t);
    r.turns[i] = (uint64_t)rint(ldexp(t, 64));  // t < 1 has no more than 53 bits: below 2^64
  }
  r.layout = c->layout;
  r.dims = c->dims;
  r.amplitude = c->amplitude;
  *rope = r;
  return WAVE_OK;
}

extern "C" int wave_rope_apply(const wave_rope* rope, int n_seq, const int32_t* cu_seqlens, const int32_t* starts, int n_heads,
                               int head_dim, const void* x, int type, int64_t x_stride, void* out, int out_type,
                               int64_t out_stride, void* stream) {
  if (!starts || !cu_ok(n_seq, cu_seqlens)) return WAVE_EINVAL;
  RopeParams p;
  int32_t slots[WAVE_MAX_SEQS];
  for (int i = 0; i < n_seq; ++i) {
    slots[i] = i;
    if (starts[i] < 0 || starts[i] > INT32_MAX - (cu_seqlens[i + 1] - cu_seqlens[i])) return WAVE_EINVAL;
  }
  const int rc = make_batch(&p.b, n_seq, cu_seqlens, slots, starts, WAVE_MAX_SEQS);
  if (rc) return rc;
  p.positions = nullptr;
  p.tokens = p.b.cum[p.b.n];
  return apply(p, rope, n_heads, head_dim, x, type, x_stride, out, out_type, out_stride, stream);
}

extern "C" int wave_rope_apply_at(const wave_rope* rope, int64_t rows, const int32_t* positions, int n_heads, int head_dim,
                                  const void* x, int type, int64_t x_stride, void* out, int out_type, int64_t out_stride,
                                  void* stream) {
  if (!positions || ((uintptr_t)positions & 3) || rows < 0 || rows > INT32_MAX) return WAVE_EINVAL;
  RopeParams p;
  p.b.n = 0;
  p.b.cum[0] = 0;
  p.positions = positions;
  p.tokens = rows;
  return apply(p, rope, n_heads, head_dim, x, type, x_stride, out, out_type, out_stride, stream);
}
