// rope.cu -- wave_rope_plan, wave_rope_apply, wave_rope_apply_at: rotary
// positions on packed rows.
//
//   (a, b) -> amplitude (a cos - b sin, a sin + b cos),  angle = position * frequency of the pair
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/wave.h"
#include "history.h"

using namespace wave;

namespace wave {

struct RopeParams {
  SeqBatch b;
  const int32_t* positions;  // rows' positions on the device, or null
  long long tokens;
  wave_rope rope;
  int heads, rows_per_cta;
  const void* x;
  void* out;
  long long x_stride, out_stride;
};

constexpr int kRopeThreads = 256, kRopeRows = 16;

// Bound by HBM, x read and out written once.  A CTA takes a few rows: the
// turns of their positions are made once, into shared memory, and serve all
// heads of a row.
template <int D, typename In, typename Out>
__global__ void __launch_bounds__(kRopeThreads) k_rope(const __grid_constant__ RopeParams p) {
  __shared__ float4 turns[kRopeRows][D / 4];  // [row][4][dims / 16]: the items' pairs, two by two
  __shared__ long long at[kRopeRows];         // the row in the buffers, or -1
  const int pairs = p.rope.dims / 2, per = p.rope.dims / 16;
  const long long first = (long long)blockIdx.x * p.rows_per_cta;
  const int rows = (int)min((long long)p.rows_per_cta, p.tokens - first);
  for (int i = threadIdx.x; i < rows * pairs; i += kRopeThreads) {
    const int r = i / pairs, k = i % pairs;
    const long long t = first + r;
    long long row = t;
    int pos;
    if (p.positions) {
      pos = p.positions[t];
      if (pos < 0) row = -1;
    } else {
      const int s = seq_of(p.b, (int)t), n = (int)t - p.b.cum[s];
      row = p.b.begin[s] + n;
      pos = p.b.start[s] + n;
    }
    if (k == 0) at[r] = row;
    ((float2*)turns[r])[(k % 8 / 2 * per + k / 8) * 2 + k % 2] = turn_at(p.rope.turns[k], (uint32_t)max(pos, 0), p.rope.amplitude);
  }
  __syncthreads();
  constexpr int kItems = D / 16;
  const int items = p.heads * kItems;
  const bool half = p.rope.layout == WAVE_ROPE_HALF;
  for (int i = threadIdx.x; i < rows * items; i += kRopeThreads) {
    const int r = i / items, head = (i - r * items) / kItems, item = i % kItems;
    const long long row = at[r];
    if (row < 0) continue;
    int a, b;
    bool turned;
    groups_of_item(p.rope, item, a, b, turned);
    const In* src = (const In*)p.x + row * p.x_stride + head * D;
    Out* dst = (Out*)p.out + row * p.out_stride + head * D;
    float x[16];
    load8<In>(src + 8 * a, x);
    load8<In>(src + 8 * b, x + 8);
    if (turned) turn_item(x, &turns[r][item], per, half);
    store8<Out>(dst + 8 * a, x);
    store8<Out>(dst + 8 * b, x + 8);
  }
}

template <int D, typename In>
static void launch_rope(const RopeParams& p, int out_type, unsigned ctas, cudaStream_t st) {
  if (out_type == WAVE_F32)
    k_rope<D, In, float><<<ctas, kRopeThreads, 0, st>>>(p);
  else if (out_type == WAVE_BF16)
    k_rope<D, In, __nv_bfloat16><<<ctas, kRopeThreads, 0, st>>>(p);
  else
    k_rope<D, In, __half><<<ctas, kRopeThreads, 0, st>>>(p);
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
  p.rows_per_cta = 1;
  const long long ctas = (p.tokens + p.rows_per_cta - 1) / p.rows_per_cta;
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
