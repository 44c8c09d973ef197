// prompt_state.cu -- wave_hybrid_prompt_state: the hybrid's selective-state
// block over packed prompts.  Per head, with dt_t = softplus(dt_t + dt_bias)
// and a_t = exp(-exp(A_log) dt_t):
//
//   h_t = a_t h_{t-1} + dt_t x_t B_t^T,   y_t = h_t C_t + D x_t,   out_t = bf16(y_t silu(z_t))
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "../../include/wave.h"
#include "ctx.h"
#include "prompt.h"
#include "prompt_ptx.cuh"

using namespace wave;

namespace wave {

// Sequences of up to so many tokens go token by token, by how many heads they
// have together.  Up to half as many as SMs: 0.16 us a token and 2.5 to begin
// with, against 13 us for a chunk with any number of tokens (a sequence of 64
// heads, 25 tokens: 6.9 against 13.1; 48: 10.8 / 12.9; 64: 13.3 / 12.5).  More:
// both take their time per head (16 sequences of 64 heads, 16 tokens: 24
// against 40; 28: 41 / 39; two sequences, 24: 9 / 13; 48: 15 / 13).
constexpr int kRowTokensFew = 48, kRowTokensMany = 28;

struct StateParams {
  SeqBatch b;
  CUtensorMap tm;          // the rows of zx as tiles of 64 columns x 128 tokens
  int tiled;               // whether tm is there: a row stride of a multiple of 16 bytes
  int Hs;
  const uint16_t* zx;      // [rows][zx_stride] bf16: z | x | B | C | dt
  const uint16_t* prm;     // A_log[Hs] | dt_bias[Hs] | D[Hs]
  const float* state_in;   // the layer's [S_max][Hs][64][128]
  float* state_out;
  uint16_t* out;           // [rows][out_stride] bf16
  long long zx_stride, out_stride;
  // Few sequences and heads leave SMs idle: a long sequence is then cut into
  // segments of seg_chunks chunks, a CTA each.  A first launch makes every
  // segment's state from zero, a second one from these the states that the
  // segments begin from, the third goes through the segments again.  The last
  // segment's place first holds the state that the sequence begins from:
  // state_out, which the third launch writes, may be state_in.
  int seg_chunks;                      // 0: whole sequences
  int32_t seg_cum[WAVE_MAX_SEQS + 1];  // segments before sequence i
  float* seg_state;                    // [segment and head pair][128 rows (head, p)][128]
  float* seg_decay;                    // ... [2]: the decays of the segment, in powers of two
  ErrSink sink;
  int skip;  // testing hook: the copies end before this chunk of a CTA (-1: off)
};

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// The recurrent form: a CTA per sequence and R rows (p) of a head's state.
// Sixteen lanes have four rows, eight values of each row in registers, so that
// a value of B or C read from shared memory serves four rows.  What depends on
// the token only, or on token and row, is brought in for kRowBatch tokens at
// once and made fp32 in shared memory (B, C, x, the gate silu(z), dt and the
// decay); the loads of the next tokens run under the arithmetic of these.  All
// of it is fp32.  Single tokens are bound by HBM, reading and writing the
// state (56 sessions of 64 heads: 36.9 us = 6.40 TB/s, with three CTAs to an
// SM; two 41.1, four 37.9).
constexpr int kRowBatch = 16;

template <int R>
__global__ void __launch_bounds__(4 * R, R == 64 ? 3 : 1) k_prompt_state_rows(const __grid_constant__ StateParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kUnroll = R == 64 ? 1 : 2;
  constexpr int kThreads = 4 * R, kParts = kSsmP / R, kLoads = kRowBatch * 2 * kSsmN / 4 / kThreads;
  __shared__ float4 sbc[kRowBatch][2 * kSsmN / 4];  // B | C
  __shared__ float4 sx[kRowBatch][R / 4], sgate[kRowBatch][R / 4];
  __shared__ float2 sda[kRowBatch];                 // dt, decay
  const int tid = threadIdx.x, i = blockIdx.y, h = blockIdx.x / kParts, row0 = blockIdx.x % kParts * R;
  const int r = tid >> 4, col = tid & 15, di = p.Hs * kSsmP, n = p.b.len(i);  // rows 4 r .. 4 r + 3
  const uint16_t* rows = p.zx + (size_t)p.b.begin[i] * p.zx_stride;
  uint2 vbc[kLoads] = {}, vx = {}, vz = {};
  uint16_t vdt = 0;
  const int xt = tid / (R / 4), xc = h * kSsmP + row0 + tid % (R / 4) * 4;  // this thread's token and column of x and z
  auto load = [&](int t0) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int k = j * kThreads + tid, t = k / (2 * kSsmN / 4);
      if (t0 + t < n) vbc[j] = __ldg((const uint2*)(rows + (size_t)(t0 + t) * p.zx_stride + 2 * di) + k % (2 * kSsmN / 4));
    }
    if (t0 + xt < n) {
      const uint16_t* row = rows + (size_t)(t0 + xt) * p.zx_stride + xc;
      vx = __ldg((const uint2*)(row + di));
      vz = __ldg((const uint2*)row);
    }
    if (tid < kRowBatch && t0 + tid < n) vdt = rows[(size_t)(t0 + tid) * p.zx_stride + 2 * di + 2 * kSsmN + h];
  };
  auto f4 = [&](uint2 v) {
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xFFFF0000u));
  };
  const size_t base = (((size_t)p.b.slot[i] * p.Hs + h) * kSsmP + row0 + 4 * r) * kSsmN + 4 * col;
  float4 st[4][2];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    st[j >> 1][j & 1] = p.b.start[i] > 0 ? __ldcs((const float4*)(p.state_in + base + (j >> 1) * kSsmN + (j & 1) * 64))
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
  load(0);
  const float a_neg = -expf(bf(p.prm[h])), bias = bf(p.prm[p.Hs + h]), skip = bf(p.prm[2 * p.Hs + h]);
  // the sums over a row's lanes end, by recursive halving, with this row's in four of them
  const bool hi8 = tid & 8, hi4 = tid & 4;
  const int mine = 4 * r + (hi8 ? 2 : 0) + (hi4 ? 1 : 0);
  uint16_t* out = p.out + (size_t)p.b.begin[i] * p.out_stride + h * kSsmP + row0 + mine;
  for (int t0 = 0; t0 < n; t0 += kRowBatch) {
    if (t0) __syncthreads();  // the tokens before these have been read
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int k = j * kThreads + tid, t = k / (2 * kSsmN / 4);
      if (t0 + t < n) sbc[t][k % (2 * kSsmN / 4)] = f4(vbc[j]);
    }
    if (t0 + xt < n) {
      sx[xt][tid % (R / 4)] = f4(vx);
      const float4 z = f4(vz);
      sgate[xt][tid % (R / 4)] =
          make_float4(z.x / (1.f + expf(-z.x)), z.y / (1.f + expf(-z.y)), z.z / (1.f + expf(-z.z)), z.w / (1.f + expf(-z.w)));
    }
    if (tid < kRowBatch && t0 + tid < n) {
      const float raw = bf(vdt) + bias;
      const float dt = raw > 0.f ? raw + log1pf(expf(-raw)) : log1pf(expf(raw));
      sda[tid] = make_float2(dt, dt == 0.f && a_neg < 0.f ? 1.f : expf(a_neg * dt));  // an infinite rate too, not a NaN
    }
    __syncthreads();
    if (t0 + kRowBatch < n) load(t0 + kRowBatch);
    const int m = min(kRowBatch, n - t0);
#pragma unroll kUnroll
    for (int t = 0; t < m; ++t, out += p.out_stride) {
      const float2 da = sda[t], a2 = make_float2(da.y, da.y);
      const float4 x4 = sx[t][r];
      const float x[4] = {x4.x, x4.y, x4.z, x4.w};
      float y[4];
      float4 B[2], C[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) B[j] = sbc[t][16 * j + col], C[j] = sbc[t][kSsmN / 4 + 16 * j + col];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float u = da.x * x[e];
        const float2 u2 = make_float2(u, u);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float4& s = st[e][j];
          const float2 s0 = fma2(a2, make_float2(s.x, s.y), mul2(u2, make_float2(B[j].x, B[j].y)));
          const float2 s1 = fma2(a2, make_float2(s.z, s.w), mul2(u2, make_float2(B[j].z, B[j].w)));
          s = make_float4(s0.x, s0.y, s1.x, s1.y);
          sum = fma2(s0, make_float2(C[j].x, C[j].y), sum);
          sum = fma2(s1, make_float2(C[j].z, C[j].w), sum);
        }
        y[e] = sum.x + sum.y;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) y[e] = (hi8 ? y[e + 2] : y[e]) + __shfl_xor_sync(0xffffffffu, hi8 ? y[e] : y[e + 2], 8);
      y[0] = (hi4 ? y[1] : y[0]) + __shfl_xor_sync(0xffffffffu, hi4 ? y[0] : y[1], 4);
      y[0] += __shfl_xor_sync(0xffffffffu, y[0], 2);
      y[0] += __shfl_xor_sync(0xffffffffu, y[0], 1);
      if ((tid & 3) == 0)
        *out = __bfloat16_as_ushort(
            __float2bfloat16_rn((y[0] + skip * ((const float*)sx[t])[mine]) * ((const float*)sgate[t])[mine]));
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    __stcs((float4*)(p.state_out + base + (j >> 1) * kSsmN + (j & 1) * 64), st[j >> 1][j & 1]);
}

// ------------------------------------------------------------ chunked form
// Chunks of 128 tokens.  With c_i the sum of exp(A_log) dt over the chunk's
// tokens up to i (in powers of two) and H the state before the chunk:
//
//   Y = M X + diag(2^-c_i) C H^T,   M_ij = (C_i . B_j) dt_j 2^(c_j - c_i)  for j <= i
//   H <- 2^-c_last H + (w X)^T B,   w_j = dt_j 2^(c_j - c_last)
//
// Everything of size 128 x 128 is a tcgen05 product: G = C B^T (once for the
// two heads of a CTA: B and C are shared by all heads), C H^T, M X with M read
// from TMEM, and the state with (w X)^T read from TMEM and its accumulator,
// the fp32 state of both heads (row = head, p; column = n), staying in TMEM
// over the whole sequence.  M (with D on its diagonal: D x_i takes part in that
// rounding; out's error, 2-norm, is 2.3e-3 with it there and with D x apart)
// and the H of C H^T are rounded to bf16 once (the output is bf16).  The state
// is fp32, so (w X)^T is the sum of three bf16 parts, all of fp32's 24 bits:
// with two the state was 2.4e-6 off (2-norm), with three 3e-7.
//
// Two warpgroups in front (a head each: the state's pass between chunks, M),
// two behind (a head each: (w X)^T, the gated output), and a warp each for the
// MMAs, the copies of x and B, those of C and z, and the decays.  The chain from
// chunk to chunk is the state's: its pass, (w X)^T and its product.  It is
// what bounds the kernel: 4.8 us a chunk, 1.7 of them products (16 prompts of
// 64 heads: tensor cores 24% active, HBM 25%, issue 42%).
constexpr int kQ = 128;                 // tokens of a chunk
constexpr int kStateThreads = 640;      // 2 warpgroups in front, 2 behind, 4 single warps; 96 registers each
constexpr int kBehind = 256;
constexpr int kBC = kQ * kSsmN * 2;     // bytes of the B (or C) tile
constexpr int kXT = kQ * kSsmP * 2;     // ... of one head's x (or z) tile

struct StateSmem {
  // One each of B, C and z (which becomes out in place), x of two chunks: x is
  // read by the products of two chunks at once.
  static constexpr int kB = 0;
  static constexpr int kC = kB + kBC;
  static constexpr int kZ = kC + kBC;
  static constexpr int kX = kZ + kBC;
  static constexpr int kLo = kX + 2 * 2 * kXT;    // the last part of (w X)^T: [tokens / 64][128 rows (head, p) of 128 B]
  static constexpr int kH = kLo + kBC;            // bf16 H: [n / 64][128 rows (head, p) of 128 B]
  static constexpr int kAfter = kH + 2 * kXT;     // [head][128] the decays behind token j, to the chunk's end
  static constexpr int kV = kAfter + 2 * kQ * 4;  // [head][128] log2 dt_j - after_j
  static constexpr int kU = kV + 2 * kQ * 4;      // [head][96] dt_j 2^-(the decays behind j in its 32 tokens)
  static constexpr int kLast = kU + 2 * 96 * 4;   // [head] the decays of the whole chunk
  static constexpr int kBad = kLast + 8;  // byte chunk % 4, bit head * 4 + warp: an x that is not finite
  static constexpr int kMisc = kBad + 4;          // TMEM's address
  static constexpr int kAnswer = kMisc + 4;       // a CTA taken over
  static constexpr int kUnit = kAnswer + 16;      // ... as the other warps get it
  static constexpr int kBars = kUnit + 8;
  enum {
    kBFull = 0,
    kBEmpty,
    kXFull,
    kXEmpty = kXFull + 2,
    kCFull = kXEmpty + 2,
    kZFull = kCFull + 2,
    kOut = kZFull + 2,  // the output has left z's tile
    kG = kOut + 2,
    kY2,
    kHFull = kY2 + 2,
    kMFull,
    kYFull,
    kYFree = kYFull + 2,
    kWx,
    kS,
    kScan,
    kNext,
    kUnitFull,
    kUnitEmpty,
    kDone,
    kCount
  };
  static constexpr int kTotal = kBars + kCount * 8;
};
static_assert(StateSmem::kAnswer % 16 == 0 && StateSmem::kBars % 8 == 0, "alignment");
static_assert(StateSmem::kTotal <= 232448, "the chunked state form does not fit shared memory");

// TMEM columns: G (the heads' M later, 64 each), (w X)^T (its first two parts;
// there is no room for the third), the state, Y of each head.
constexpr int kTG = 0, kTWx = 128, kTState = 256, kTY = 384;

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Whether it holds for all of them.
__device__ __forceinline__ bool bar_and(int id, int threads, bool v) {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(r)
               : "r"((uint32_t)v), "r"(id), "r"(threads)
               : "memory");
  return r != 0;
}
// Rows that no tensor map can describe (a stride that is no multiple of 16
// bytes): a warp copies the tile, 128 tokens x 128 columns from (row0, col) on,
// 8 bytes at a time, as the same 128-byte swizzled blocks of 64 columns.  Rows
// from n on repeat row n - 1.
__device__ __forceinline__ void copy_tile(uint32_t dst, const uint16_t* zx, long long stride, int col, int row0, int n) {
  const int lane = threadIdx.x & 31, blk = lane >> 4, c = (lane >> 1) & 7;
  const uint16_t* src = zx + (size_t)row0 * stride + col + lane * 4;
  dst += blk * (kQ * 128) + (lane & 1) * 8;
#pragma unroll 8
  for (int r = 0; r < kQ; ++r, src += r < n ? stride : 0)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst + r * 128 + ((c ^ (r & 7)) << 4)), "l"(src) : "memory");
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Waits for all tiles that this warp has begun to copy but the last kOpen.
template <int kOpen>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kOpen) : "memory");
  fence_proxy_async_smem();
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int n>
__device__ __forceinline__ void scale_regs(uint32_t* v, float f) {
#pragma unroll
  for (int e = 0; e < n; e += 2) {
    const float2 r = mul2(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), make_float2(f, f));
    v[e] = __float_as_uint(r.x);
    v[e + 1] = __float_as_uint(r.y);
  }
}

// log(1 + e^raw) = max(raw, 0) + log1p(t), t = e^-|raw|, by the series
// log1p(t) = 2 (s + s^3/3 + s^5/5 + ...), s = t / (2 + t) <= 1/3: terms to
// s^13 leave 2^-27.  Short and without branches: it runs eight times per lane
// and chunk, and the library's expf and log1pf together did not fit the
// instruction cache beside the other warps' code.
__device__ __forceinline__ float softplus(float raw) {
  const float t = ex2(-1.44269504088896340736f * fabsf(raw));
  const float s = __fdividef(t, 2.f + t), s2 = s * s;
  float q = fmaf(s2, 2.f / 13.f, 2.f / 11.f);
  q = fmaf(s2, q, 2.f / 9.f);
  q = fmaf(s2, q, 2.f / 7.f);
  q = fmaf(s2, q, 2.f / 5.f);
  q = fmaf(s2, q, 2.f / 3.f);
  q = fmaf(s2, q, 2.f);
  return fmaxf(raw, 0.f) + s * q;
}

// The states that segments begin from, in the place of their own states from
// zero: a thread per four values of a sequence's head pair, eight segments'
// loads at once (with each CTA adding up those before it, a load after the
// other, 2048 tokens of 4 heads took 52 us instead of 28).
__global__ void __launch_bounds__(256) k_segment_states(const __grid_constant__ StateParams p) {
  const int e = blockIdx.x * 256 + threadIdx.x, pairs = gridDim.y, seq = blockIdx.z;
  const int first = p.seg_cum[seq], segs = p.seg_cum[seq + 1] - first;
  auto slot = [&](int i) { return (float4*)p.seg_state + ((size_t)(first + i) * pairs + blockIdx.y) * (128 * kSsmN / 4) + e; };
  const int hh = e / (kSsmP * kSsmN / 4);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float4 now = p.b.start[seq] > 0 ? *slot(segs - 1) : make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < segs; i0 += 8) {
    float4 own[8];
    float d[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i0 + j + 1 < segs) own[j] = *slot(i0 + j), d[j] = p.seg_decay[2 * ((first + i0 + j) * pairs + blockIdx.y) + hh];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (i0 + j >= segs) break;
      *slot(i0 + j) = now;
      const float f = ex2(-d[j]);
      if (i0 + j + 1 < segs)
        now = make_float4(fmaf(now.x, f, own[j].x), fmaf(now.y, f, own[j].y), fmaf(now.z, f, own[j].z), fmaf(now.w, f, own[j].w));
    }
  }
}

// What a CTA works on: a head pair of a sequence, or of a segment of one.
struct StateUnit {
  int seq, h0, first, len;  // first: its first row
  int chunks;
};

// kLocal: only the state of a segment from zero, into seg_state (the last
// segment of a sequence has none to give on).  kOnce: a unit per CTA, whole
// sequences or segments.  kMore: whole sequences, more of them than SMs; a CTA
// takes the place of CTAs that have not begun, so that a unit's first copies
// and products run under the last of the unit before (16 prompts of 8005
// tokens, 64 heads: 96 us, with a unit per CTA 102).
enum StateMode { kLocal, kOnce, kMore };

template <StateMode kMode>
__global__ void __launch_bounds__(kStateThreads, 1) k_prompt_state(const __grid_constant__ StateParams p) {
  using L = StateSmem;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if constexpr (kMode == kLocal) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int pairs = p.Hs / 2;
  auto whole = [&](int cta) {  // a CTA's sequence and head pair
    StateUnit u;
    u.seq = cta / pairs, u.h0 = cta % pairs * 2;
    u.len = p.b.len(u.seq), u.first = p.b.begin[u.seq];
    u.chunks = (u.len + kQ - 1) / kQ;
    return u;
  };
  StateUnit mine;
  int seg = 0;
  bool last_seg = true;
  if (kMode != kMore && p.seg_chunks) {
    const int unit = blockIdx.x / pairs;
    int lo = 0, hi = p.b.n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.seg_cum[mid] <= unit)
        lo = mid;
      else
        hi = mid - 1;
    }
    mine = whole(lo * pairs + blockIdx.x % pairs);
    seg = unit - p.seg_cum[lo];
    mine.first += seg * p.seg_chunks * kQ;
    mine.len -= seg * p.seg_chunks * kQ;
    last_seg = mine.len <= p.seg_chunks * kQ;
    if (!last_seg) mine.len = p.seg_chunks * kQ;
    mine.chunks = (mine.len + kQ - 1) / kQ;
    if (kMode == kLocal && last_seg) {
      if (p.b.start[mine.seq] > 0) {
        const float4* src = (const float4*)p.state_in + ((size_t)p.b.slot[mine.seq] * p.Hs + mine.h0) * (kSsmP * kSsmN / 4);
        float4* dst = (float4*)p.seg_state + (size_t)blockIdx.x * (128 * kSsmN / 4);
        for (int i = threadIdx.x; i < 128 * kSsmN / 4; i += kStateThreads) dst[i] = src[i];
      }
      asm volatile("griddepcontrol.wait;" ::: "memory");  // see the end
      return;
    }
  } else {
    mine = whole(blockIdx.x);
  }
  const int di = p.Hs * kSsmP;
  auto bar = [&](int b) { return sb + L::kBars + b * 8; };
  uint32_t* tmem_word = (uint32_t*)(smem + L::kMisc);
  if (sb & 1023) {  // the tiles' swizzle counts on it, and there is no room to align by hand
    if (threadIdx.x == 0) *(volatile int*)p.sink.err_out = atomicOr(p.sink.err, kErrTimeout) | kErrTimeout;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  if (__syncthreads_or(threadIdx.x == 0 && stopped(p.sink))) {  // a CTA that begins now would run into the same limit
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }

  if (warp == 16) {
    if (lane == 0) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(bar(L::kXFull + b), 1);
        mbar_init(bar(L::kXEmpty + b), 1);
        mbar_init(bar(L::kCFull + b), 1);
        mbar_init(bar(L::kZFull + b), 1);
        mbar_init(bar(L::kOut + b), kBehind / 32);
        mbar_init(bar(L::kY2 + b), 1);
        mbar_init(bar(L::kYFull + b), 1);
      }
      mbar_init(bar(L::kBFull), 1);
      mbar_init(bar(L::kBEmpty), 1);
      mbar_init(bar(L::kMFull), 8);
      mbar_init(bar(L::kG), 1);
      mbar_init(bar(L::kHFull), 8);  // warps
      mbar_init(bar(L::kYFree), kBehind / 32);
      mbar_init(bar(L::kScan), 1);
      mbar_init(bar(L::kWx), kBehind / 32);
      mbar_init(bar(L::kS), 1);
      mbar_init(bar(L::kNext), 1);
      mbar_init(bar(L::kUnitFull), 1);
      mbar_init(bar(L::kUnitEmpty), 19);  // every warp but the one that writes it
      mbar_init(bar(L::kDone), 1);
      fence_mbar_init();
      fence_proxy_async_smem();
    }
    __syncwarp();
    tmem_alloc(smem_u32(tmem_word), 512);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) *(uint32_t*)(smem + L::kBad) = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_word;

  // In the compute warps a wait that gives up leaves the rest of the unit
  // without waits (the named barriers need every warp), with its results
  // undefined, and then all leave; the other warps leave their loops.
  bool ok = true;
  auto wait_warp = [&](int b, uint32_t parity) {
    if (ok) ok = __all_sync(0xffffffffu, wait_bar(bar(b), parity, p.sink));
  };
  // One arrival for the warp's 32 threads (as many arrivals on one barrier would
  // go one after the other through the shared-memory pipe, 32 passes a warp).
  auto arrive_warp = [&](int b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(b));
  };
  const int h = (warp >> 2) & 1, quad = warp & 3, row = quad * 32 + lane;  // a thread per token of head h0 + h
  const uint32_t lanes = (uint32_t)(quad * 32) << 16;
  const int hh = row >> 6, pp = row & 63;  // for the state: row (head hh, p)
  // Whether a unit's state does not begin as zero.
  auto goes_on = [&](const StateUnit& u) { return kMode != kLocal && (seg > 0 || p.b.start[u.seq] > 0); };
  // The unit after the n - 1 before it, if there is one: a CTA that has not
  // begun, taken over by the warp of the decays, so that the first chunk of one
  // unit runs under the last of the one before.  group: the named barrier of a
  // group of 256 threads, which goes on together or not at all.
  auto next_unit = [&](StateUnit& u, uint32_t n, int group = 0) {
    if (kMode != kMore) return false;
    wait_warp(L::kUnitFull, (n - 1) & 1);
    if (group) ok = bar_and(group, 256, ok);
    if (!ok) return false;
    const int cta = *(volatile int*)(smem + L::kUnit);
    arrive_warp(L::kUnitEmpty);
    if (cta < 0) return false;
    u = whole(cta);
    return true;
  };
  float* sv = (float*)(smem + L::kV);
  float* su = (float*)(smem + L::kU);
  float* saft = (float*)(smem + L::kAfter);
  float* slast = (float*)(smem + L::kLast);
  uint32_t* sbad = (uint32_t*)(smem + L::kBad);

  if (warp < 8) {
    // -------------------------------------------------------------- in front
    float decayed = 0.f;  // kLocal: the decays so far, of head h
    StateUnit u = mine;
    uint32_t g = 0;  // the CTA's chunks
    // the states that segments begin from are there, and what state_in held has been read
    if (kMode == kOnce && p.seg_chunks) asm volatile("griddepcontrol.wait;" ::: "memory");
    for (uint32_t n = 0; n == 0 || next_unit(u, n, 1); ++n) {
      const float skip = bf(p.prm[2 * p.Hs + u.h0 + h]);
      const size_t state_at = (((size_t)p.b.slot[u.seq] * p.Hs + u.h0) * kSsmP + row) * kSsmN + h * 64;
      const float* begin = kMode != kMore && p.seg_chunks
                               ? p.seg_state + (size_t)blockIdx.x * (128 * kSsmN) + row * kSsmN + h * 64
                               : p.state_in + state_at;
      if (goes_on(u)) {
        asm volatile("prefetch.global.L1 [%0];" ::"l"(begin));
        asm volatile("prefetch.global.L1 [%0];" ::"l"(begin + 32));
      }
      for (int c = 0; c < u.chunks; ++c, ++g) {
        // ---- the state: its bf16 copy for C H^T, and the chunk's decay
        wait_warp(L::kScan, g & 1);
        if (g > 0) wait_warp(L::kS, (g - 1) & 1);
        tc_fence_after();
        const float after = saft[h * kQ + row];  // c_j - c_i = after_i - after_j
        const bool zero = c == 0 && !goes_on(u);
        if (!zero) {
          const float dec = ex2(-slast[hh]);
          uint8_t* hrow = smem + L::kH + h * (128 * 128) + row * 128;
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            uint32_t v[16];
            if (kMode != kLocal && c == 0) {
              const float4* src = (const float4*)(begin + 16 * q);
              float4 f[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) f[e] = src[e];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                v[4 * e] = __float_as_uint(f[e].x), v[4 * e + 1] = __float_as_uint(f[e].y);
                v[4 * e + 2] = __float_as_uint(f[e].z), v[4 * e + 3] = __float_as_uint(f[e].w);
              }
            } else {
              tmem_ld16_nowait(tmem + kTState + lanes + h * 64 + 16 * q, v);
              tmem_ld_wait();
            }
            if constexpr (kMode != kLocal) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                uint4 w;
                w.x = pack_bf16(__uint_as_float(v[8 * e]), __uint_as_float(v[8 * e + 1]));
                w.y = pack_bf16(__uint_as_float(v[8 * e + 2]), __uint_as_float(v[8 * e + 3]));
                w.z = pack_bf16(__uint_as_float(v[8 * e + 4]), __uint_as_float(v[8 * e + 5]));
                w.w = pack_bf16(__uint_as_float(v[8 * e + 6]), __uint_as_float(v[8 * e + 7]));
                *(uint4*)(hrow + (((2 * q + e) ^ (pp & 7)) << 4)) = w;
              }
            }
            scale_regs<16>(v, dec);
            tmem_st16(tmem + kTState + lanes + h * 64 + 16 * q, v);
          }
          tmem_st_wait();
          fence_proxy_async_smem();
        }
        tc_fence_before();
        if constexpr (kMode == kLocal) decayed += slast[h];
        arrive_warp(L::kHFull);
        if constexpr (kMode == kLocal) continue;
        // ---- M, over G once both heads have read G
        wait_warp(L::kG, g & 1);
        tc_fence_after();
        // Tokens 64..127 first, then 0..63: once both heads have read that half
        // of G, its 64 columns take the same half of both heads' M.
#pragma unroll 1
        for (int half = 1; half >= 0; --half) {
          uint32_t m[32];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int q = 2 * half + t;  // 32 tokens
            if (q > quad) {              // above the diagonal
#pragma unroll
              for (int e = 0; e < 16; ++e) m[16 * t + e] = 0;
              continue;
            }
            uint32_t gv[32];
            tmem_ld32(tmem + kTG + lanes + 32 * q, gv);
            if (q < quad) {
              // below: the decay from the end of token j's 32 to i is a factor
              // of the row, that from j to there is in u_j
              const float r = ex2(after - saft[h * kQ + 32 * q + 31]);
              const float2 r2 = make_float2(r, r);
              const float4* uj = (const float4*)(su + h * 96 + 32 * q);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float4 u4 = uj[e];
                const float2 m0 = mul2(mul2(make_float2(__uint_as_float(gv[4 * e]), __uint_as_float(gv[4 * e + 1])), r2),
                                       make_float2(u4.x, u4.y));
                const float2 m1 = mul2(mul2(make_float2(__uint_as_float(gv[4 * e + 2]), __uint_as_float(gv[4 * e + 3])), r2),
                                       make_float2(u4.z, u4.w));
                m[16 * t + 2 * e] = pack_bf16(m0.x, m0.y);
                m[16 * t + 2 * e + 1] = pack_bf16(m1.x, m1.y);
              }
            } else {
              // on it; D x_i is added to y_i as D on the diagonal
              const float2 ai = make_float2(after, after);
              const float4* vj = (const float4*)(sv + h * kQ + 32 * q);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float4 v4 = vj[e];
                const float2 t0 = add2(make_float2(v4.x, v4.y), ai), t1 = add2(make_float2(v4.z, v4.w), ai);
                const float2 m0 = mul2(make_float2(__uint_as_float(gv[4 * e]), __uint_as_float(gv[4 * e + 1])),
                                       make_float2(ex2(t0.x), ex2(t0.y)));
                const float2 m1 = mul2(make_float2(__uint_as_float(gv[4 * e + 2]), __uint_as_float(gv[4 * e + 3])),
                                       make_float2(ex2(t1.x), ex2(t1.y)));
                float f[4] = {m0.x, m0.y, m1.x, m1.y};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  if (4 * e + k > lane) f[k] = 0.f;
                  if (4 * e + k == lane) f[k] += skip;
                }
                m[16 * t + 2 * e] = pack_bf16(f[0], f[1]);
                m[16 * t + 2 * e + 1] = pack_bf16(f[2], f[3]);
              }
            }
          }
          tc_fence_before();
          bar_sync(1, 256);  // both heads have read this half of G
          tc_fence_after();
          tmem_st32(tmem + kTG + half * 64 + h * 32 + lanes, m);
        }
        // ---- C H^T, scaled in place: M X is added to it
        wait_warp(L::kY2 + (g & 1), (g >> 1) & 1);
        tc_fence_after();
        if (!zero) {
          const float ei = ex2(after - slast[h]);
#pragma unroll 1
          for (int q = 0; q < 2; ++q) {
            uint32_t v[32];
            tmem_ld32(tmem + kTY + h * 64 + lanes + 32 * q, v);
            tmem_ld_wait();
            scale_regs<32>(v, ei);
            tmem_st32(tmem + kTY + h * 64 + lanes + 32 * q, v);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        arrive_warp(L::kMFull);
      }
      if (kMode == kLocal && row == 0) p.seg_decay[2 * blockIdx.x + h] = decayed;
      // ---- the state after the last token
      wait_warp(L::kS, (g - 1) & 1);
      tc_fence_after();
#pragma unroll 1
      for (int q = 0; q < 2 && (kMode == kLocal || last_seg); ++q) {
        uint32_t v[32];
        tmem_ld32(tmem + kTState + lanes + h * 64 + q * 32, v);
        tmem_ld_wait();
        float4* dst = (float4*)(kMode == kLocal ? p.seg_state + (size_t)blockIdx.x * (128 * kSsmN) + row * kSsmN + h * 64 + 32 * q
                                       : p.state_out + state_at + 32 * q);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          dst[e] = make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]), __uint_as_float(v[4 * e + 2]),
                               __uint_as_float(v[4 * e + 3]));
      }
    }
  } else if (warp < 16) {
    // ---------------------------------------------------------------- behind
    // (w X)^T of a chunk is made before the output of the chunk before it: the
    // state's product does not wait for the gate
    StateUnit u = mine;
    uint32_t n = 0, g = 0;  // units; chunks, the next (w X)^T's
    int c = 0;              // ... and its chunk of u
    bool weigh = true, gate = false;
    int out_row = 0;  // the chunk whose output is next: the one before g
    int out_h0 = 0, out_left = 0;
    while (weigh || gate) {
      const int left = u.len - c * kQ;
      const int row0 = u.first + c * kQ;
      if (weigh) {
        const uint32_t k = g;
        const int b = k & 1;
        // ---- this token's x and B.  Behind the sequence's end lie other rows:
        // theirs become zero.  An x that is not finite would reach earlier
        // tokens as 0 * NaN in M X: it is noted here, becomes zero once the
        // state's weights have been made of it, and is put back at the output.
        const uint32_t parity = (k >> 1) & 1;
        wait_warp(L::kXFull + b, parity);
        uint8_t* xrow = smem + L::kX + (b * 2 + h) * kXT + row * 128;
        bool odd = false;
        if (row >= left) {
#pragma unroll 4
          for (int e = 0; e < 8; ++e) *(uint4*)(xrow + (e << 4)) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
        } else {
          uint32_t acc[2] = {0, 0};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint4 x = *(const uint4*)(xrow + ((e ^ (row & 7)) << 4));
            asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc[0]) : "r"(x.x), "r"(0));
            asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc[1]) : "r"(x.y), "r"(0));
            asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc[0]) : "r"(x.z), "r"(0));
            asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc[1]) : "r"(x.w), "r"(0));
          }
          odd = ((acc[0] | acc[1]) & 0x7fff7fffu) != 0;
          if (odd) atomicOr(sbad, 1u << ((k & 3) * 8 + h * 4 + quad));
        }
        bar_sync(4, kBehind);  // x and its flags are complete; every thread here is done with chunk k - 2
        // cleared two chunks ahead: nobody sets these before the next barrier
        if (threadIdx.x == 256) atomicAnd(sbad, ~(0xFFu << (((k + 2) & 3) * 8)));
        // ---- (w X)^T: row (hh, pp), tokens 64 h .. 64 h + 63
        wait_warp(L::kScan, k & 1);
        if (k > 0) wait_warp(L::kS, (k - 1) & 1);
        if (left < kQ) {  // B's phase before this one is over: the last state has been made of it
          wait_warp(L::kBFull, k & 1);
          if (row >= left) {
            uint8_t* brow = smem + L::kB + h * (kQ * 128) + row * 128;
#pragma unroll
            for (int e = 0; e < 8; ++e) *(uint4*)(brow + (e << 4)) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
          }
        }
        tc_fence_after();
        const uint8_t* xt = smem + L::kX + (b * 2 + hh) * kXT + (pp & 7) * 2;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          const int j0 = h * 64 + 16 * q;
          float v[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)  // j0 is a multiple of 8
            v[e] = bf(*(const uint16_t*)(xt + (j0 + e) * 128 + (((pp >> 3) ^ (e & 7)) << 4)));
          // w_j: u_j times the decay from its 32 tokens' end on; the last 32 have v_j only
          const bool tail_block = j0 >= 96;
          const float tail = tail_block ? 1.f : ex2(-saft[hh * kQ + (j0 | 31)]);
          const float4* uj = (const float4*)((tail_block ? sv + hh * kQ : su + hh * 96) + j0);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float4 u4 = uj[e];
            if (tail_block) u4 = make_float4(ex2(u4.x), ex2(u4.y), ex2(u4.z), ex2(u4.w));
            const float2 r0 = mul2(make_float2(v[4 * e], v[4 * e + 1]), mul2(make_float2(u4.x, u4.y), make_float2(tail, tail)));
            const float2 r1 = mul2(make_float2(v[4 * e + 2], v[4 * e + 3]), mul2(make_float2(u4.z, u4.w), make_float2(tail, tail)));
            v[4 * e] = r0.x, v[4 * e + 1] = r0.y, v[4 * e + 2] = r1.x, v[4 * e + 3] = r1.y;
          }
          uint32_t part[3][8];
#pragma unroll
          for (int t = 0; t < 3; ++t) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              part[t][e] = pack_bf16(v[2 * e], v[2 * e + 1]);
              if (t == 2) continue;
              const float2 r = sub2(make_float2(v[2 * e], v[2 * e + 1]),
                                    make_float2(__uint_as_float(part[t][e] << 16), __uint_as_float(part[t][e] & 0xFFFF0000u)));
              v[2 * e] = r.x, v[2 * e + 1] = r.y;
            }
          }
          tmem_st8(tmem + kTWx + lanes + h * 32 + q * 8, part[0]);
          tmem_st8(tmem + kTWx + 64 + lanes + h * 32 + q * 8, part[1]);
          uint8_t* lrow = smem + L::kLo + h * (128 * 128) + row * 128;
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *(uint4*)(lrow + (((2 * q + e) ^ (row & 7)) << 4)) =
                make_uint4(part[2][4 * e], part[2][4 * e + 1], part[2][4 * e + 2], part[2][4 * e + 3]);
        }
        fence_proxy_async_smem();
        tmem_st_wait();
        if (*(volatile uint32_t*)sbad >> ((k & 3) * 8) & 0xFFu) {  // seen by every thread or none
          bar_sync(4, kBehind);
          if (odd) {
#pragma unroll 1
            for (int e = 0; e < 64; ++e) {
              uint16_t* x = (uint16_t*)xrow + e;
              if ((*x & 0x7F80) == 0x7F80) *x = 0;
            }
            fence_proxy_async_smem();
          }
        }
        tc_fence_before();
        arrive_warp(L::kWx);
      }
      if (kMode != kLocal && gate) {
        const uint32_t k = g - 1;
        const int b = k & 1;
        // ---- the output: y, gated, over z's row and from there to global
        uint8_t* ztile = smem + L::kZ + h * kXT;
        const uint32_t any_bad = *(volatile uint32_t*)sbad >> ((k & 3) * 8 + h * 4) & 15u;
        wait_warp(L::kZFull + b, (k >> 1) & 1);
        wait_warp(L::kYFull + h, k & 1);
        tc_fence_after();
        uint8_t* zrow = ztile + row * 128;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          uint32_t y[32];
          tmem_ld32(tmem + kTY + h * 64 + lanes + 32 * half, y);
          tmem_ld_wait();
          if (half == 1) {
            tc_fence_before();
            arrive_warp(L::kYFree);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint4* zp = (uint4*)(zrow + (((half * 4 + e) ^ (row & 7)) << 4));
            const uint4 zv = *zp;
            const uint32_t zw[4] = {zv.x, zv.y, zv.z, zv.w};
            uint32_t o[4];
#pragma unroll
            for (int f = 0; f < 4; ++f) {
              const int i = 8 * e + 2 * f;
              const float2 z2 = make_float2(__uint_as_float(zw[f] << 16), __uint_as_float(zw[f] & 0xFFFF0000u));
              const float2 t = mul2(z2, make_float2(-1.44269504088896340736f, -1.44269504088896340736f));
              const float2 d = add2(make_float2(ex2(t.x), ex2(t.y)), make_float2(1.f, 1.f));
              const float2 g = mul2(z2, make_float2(rcp(d.x), rcp(d.y)));
              const float2 r = mul2(make_float2(__uint_as_float(y[i]), __uint_as_float(y[i + 1])), g);
              o[f] = pack_bf16(r.x, r.y);
            }
            *zp = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        if (any_bad) {  // tokens up to this one whose x is not finite
#pragma unroll 1
          for (int j = 0; j <= row && j < out_left; ++j) {
            if (!(any_bad >> (j >> 5) & 1)) continue;
            const uint16_t* x = p.zx + (size_t)(out_row + j) * p.zx_stride + di + (out_h0 + h) * kSsmP;
#pragma unroll 1
            for (int e = 0; e < 64; ++e)
              if ((x[e] & 0x7F80) == 0x7F80) *(uint16_t*)(zrow + (((e >> 3) ^ (row & 7)) << 4) + (e & 7) * 2) = 0x7FC0;
          }
        }
        __syncwarp();
        {
          const int r0 = quad * 32 + (lane >> 3), at = lane & 7;  // four rows at a time
          uint16_t* dst = p.out + (size_t)(out_row + r0) * p.out_stride + (out_h0 + h) * kSsmP + at * 8;
#pragma unroll 4
          for (int q = 0; q < 8; ++q, dst += 4 * p.out_stride) {
            const int r = r0 + 4 * q;
            const uint4 v = *(const uint4*)(ztile + r * 128 + ((at ^ (r & 7)) << 4));
            if (r < out_left) *(uint4*)dst = v;
          }
        }
        fence_proxy_async_smem();  // the next copies into this buffer come by the async proxy
        arrive_warp(L::kOut + b);
      }
      gate = kMode != kLocal && weigh;
      if (weigh) {
        out_row = row0, out_h0 = u.h0, out_left = left;
        ++g;
        if (++c == u.chunks) {
          c = 0;
          weigh = next_unit(u, ++n, 4);
        }
      }
    }
  } else {
    if (warp == 16) {
      // ---------------------------------------------------------------- MMAs
      constexpr uint32_t id_g = idesc_16(128, 128, false, false, false), id_y = idesc_16(128, 64, false, false, true),
                         id_s = idesc_16(128, 128, false, false, true);
      constexpr uint32_t kBlk = (kQ * 128) >> 4;  // the next 64 columns of a tile, as a descriptor counts
      StateUnit u = mine;
      uint32_t g = 0;  // the CTA's chunks
      for (uint32_t n = 0; ok && (n == 0 || next_unit(u, n)); ++n) {
        for (int c = 0; c < u.chunks; ++c, ++g) {
          const uint32_t ct = sb + L::kC, bt = sb + L::kB;
          const bool zero = c == 0 && !goes_on(u);
          wait_warp(L::kBFull, g & 1);
          if constexpr (kMode != kLocal) wait_warp(L::kCFull + (g & 1), (g >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          if (kMode != kLocal && elect_one()) {  // G = C B^T
            const uint32_t cm = sdesc_lo(ct), bm = sdesc_lo(bt);
            mma_ss<false>(tmem + kTG, cm, bm, id_g);
#pragma unroll
            for (int e = 1; e < 8; ++e)
              mma_ss<true>(tmem + kTG, cm + (e / 4) * kBlk + (e % 4) * 2, bm + (e / 4) * kBlk + (e % 4) * 2, id_g);
            tc_commit(bar(L::kG));
          }
          __syncwarp();
          wait_warp(L::kHFull, g & 1);
          wait_warp(L::kWx, g & 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {  // the state += (w X)^T B, its three parts
            const uint32_t bm = sdesc_lo(bt, kQ * 128), lm = sdesc_lo(sb + L::kLo);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              mma_ts(tmem + kTState, tmem + kTWx + 8 * e, bm + (e % 8) * (2048 >> 4), id_s, e > 0 ? 1u : zero ? 0u : 1u);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              mma_ss<true>(tmem + kTState, lm + (e / 4) * kBlk + (e % 4) * 2, bm + e * (2048 >> 4), id_s);
            tc_commit(bar(L::kS));
            tc_commit(bar(L::kBEmpty));
          }
          __syncwarp();
          if constexpr (kMode != kLocal) {
            if (g > 0) wait_warp(L::kYFree, (g - 1) & 1);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {  // Y = C H^T, of both heads at once
              if (!zero) {
                const uint32_t cm = sdesc_lo(ct), hm = sdesc_lo(sb + L::kH);
                mma_ss<false>(tmem + kTY, cm, hm, id_g);
#pragma unroll
                for (int e = 1; e < 8; ++e)
                  mma_ss<true>(tmem + kTY, cm + (e / 4) * kBlk + (e % 4) * 2, hm + (e / 4) * kBlk + (e % 4) * 2, id_g);
              }
              tc_commit(bar(L::kY2 + (g & 1)));
            }
            __syncwarp();
            wait_warp(L::kMFull, g & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // Y += M X
              if (elect_one()) {
                const uint32_t xm = sdesc_lo(sb + L::kX + ((g & 1) * 2 + h) * kXT, kQ * 128);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  mma_ts(tmem + kTY + h * 64, tmem + kTG + (e / 4) * 64 + h * 32 + (e % 4) * 8, xm + e * (2048 >> 4), id_y,
                         e > 0 ? 1u : zero ? 0u : 1u);
                tc_commit(bar(L::kYFull + h));
              }
              __syncwarp();
            }
          }
          if (elect_one()) tc_commit(bar(L::kXEmpty + (g & 1)));
          __syncwarp();
        }
      }
      if (!ok) {  // give-up: wait (bounded) for the MMAs issued so far
        if (elect_one()) tc_commit(bar(L::kDone));
        __syncwarp();
        for (int n = 0; n < (1 << 20) && !mbar_try_wait(bar(L::kDone), 0); ++n) {
        }
      }
      __syncwarp();
    } else if (warp < 19) {
      // ----------------------- copies: x and B by one warp, C and z by another
      auto copy = [&](uint32_t dst, int column, int r, int n, int b) {  // two blocks of 64 columns
        if (p.tiled) {
          if (elect_one()) {
            mbar_arrive_expect_tx(bar(b), kBC);
            tma_load_3d_plain(dst, &p.tm, column, 0, r, bar(b));
            tma_load_3d_plain(dst + kQ * 128, &p.tm, column + 64, 0, r, bar(b));
          }
          __syncwarp();
        } else {
          copy_tile(dst, p.zx, p.zx_stride, column, r, n);
        }
      };
      // Without a tensor map the warp itself says when a tile is there: the
      // first of a chunk's two once the second is under way (the CTA's first
      // chunk: both buffers are free), or before the second is waited for.
      auto landed = [&](int b, auto open) {
        if (p.tiled) return;
        copy_wait<open.value>();
        arrive_warp(b);
      };
      constexpr std::integral_constant<int, 0> kNone{};
      constexpr std::integral_constant<int, 1> kOne{};
      StateUnit u = mine;
      uint32_t g = 0;                           // the CTA's chunks
      uint32_t nx = 0, nb = 0, nc = 0, nz = 0;  // copies begun
      for (uint32_t n = 0; ok && (n == 0 || next_unit(u, n)); ++n) {
        for (int c = 0; c < u.chunks; ++c, ++g) {
          const int r = u.first + c * kQ, rows = min(kQ, u.len - c * kQ);
          if (g == (uint32_t)p.skip) {
            ok = false;
            break;
          }
          if (warp == 17) {
            wait_warp(L::kXEmpty + (g & 1), ((g >> 1) & 1) ^ 1);
            if (!ok) break;
            copy(sb + L::kX + (g & 1) * 2 * kXT, di + u.h0 * kSsmP, r, rows, L::kXFull + (g & 1));
            ++nx;
            if (g > 0) landed(L::kXFull + (g & 1), kNone);
            wait_warp(L::kBEmpty, (g & 1) ^ 1);
            if (!ok) break;
            copy(sb + L::kB, 2 * di, r, rows, L::kBFull);
            ++nb;
            if (g == 0) landed(L::kXFull, kOne);
            landed(L::kBFull, kNone);
          } else if constexpr (kMode != kLocal) {
            if (g > 0) wait_warp(L::kY2 + ((g - 1) & 1), ((g - 1) >> 1) & 1);  // C of the chunk before
            if (!ok) break;
            copy(sb + L::kC, 2 * di + kSsmN, r, rows, L::kCFull + (g & 1));
            ++nc;
            if (g > 0) {
              landed(L::kCFull + (g & 1), kNone);
              wait_warp(L::kOut + ((g - 1) & 1), ((g - 1) >> 1) & 1);
              if (!ok) break;
            }
            copy(sb + L::kZ, u.h0 * kSsmP, r, rows, L::kZFull + (g & 1));
            ++nz;
            if (g == 0) landed(L::kCFull, kOne);
            landed(L::kZFull + (g & 1), kNone);
          }
        }
      }
      if (!p.tiled) {
        copy_wait<0>();
      } else if (!ok) {  // give-up: the copies in flight land before the shared memory is left
        auto drain = [&](int b, uint32_t parity) {
          for (int n = 0; n < (1 << 20) && !mbar_try_wait(bar(b), parity); ++n) {
          }
        };
        auto drain2 = [&](int b, uint32_t n) {  // the last two of n copies by turns
          for (uint32_t i = n > 2 ? n - 2 : 0; i < n; ++i) drain(b + (i & 1), (i >> 1) & 1);
        };
        drain2(L::kXFull, nx);
        drain2(L::kCFull, nc);
        drain2(L::kZFull, nz);
        if (nb) drain(L::kBFull, (nb - 1) & 1);
      }
      __syncwarp();
    } else {
      // ------------------------------ the decays, a chunk ahead: lane l has
      // tokens 4 l .. 4 l + 3 of both heads.  They are summed from the chunk's
      // end, so that the weights of the state's newest tokens are exact to
      // fp32 whatever the sum over the chunk is.
      StateUnit u = mine;
      uint32_t g = 0;        // the CTA's chunks
      uint32_t asks = 0;     // requests for another CTA ...
      bool asked = false;    // ... and whether one is open
      for (uint32_t n = 0; ok; ++n) {
        const uint16_t* col = p.zx + (size_t)u.first * p.zx_stride + 2 * di + 2 * kSsmN + u.h0;  // two heads: 4 bytes
        uint32_t raw[4];
        auto fetch = [&](int c) {
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const int j = c * kQ + 4 * lane + t;
            raw[t] = j < u.len ? *(const uint32_t*)(col + (size_t)j * p.zx_stride) : 0;
          }
        };
        fetch(0);
        float rate[2], bias[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          rate[e] = expf(bf(p.prm[u.h0 + e])) * 1.44269504088896340736f;
          bias[e] = bf(p.prm[p.Hs + u.h0 + e]);
          if (rate[e] != rate[e]) bias[e] = rate[e];  // the cap of the decays would hide a NaN: it goes into dt
        }
        for (int c = 0; c < u.chunks; ++c, ++g) {
          if (kMode == kMore && c == u.chunks - 1) {
            if (lane == 0) {
              fence_proxy_async_smem();  // the last answer has been read
              mbar_arrive_expect_tx(bar(L::kNext), 16);
              cta_request(sb + L::kAnswer, bar(L::kNext));
            }
            __syncwarp();
            ++asks, asked = true;
          }
          const int left = u.len - c * kQ;
          float dt[2][4], after[2][4], last[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float lam[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              dt[e][t] = softplus((e ? __uint_as_float(raw[t] & 0xFFFF0000u) : __uint_as_float(raw[t] << 16)) + bias[e]);
              if (4 * lane + t >= left) dt[e][t] = 0.f;
              // the token's decay in powers of two; 2^-160 is zero in fp32: a larger
              // step changes nothing, and the cap bounds the rounding of the sums.
              // No step, no decay, also at a rate beyond fp32's range (inf * 0)
              lam[t] = dt[e][t] == 0.f ? 0.f : fminf(rate[e] * dt[e][t], 160.f);
            }
            float down = (lam[0] + lam[1]) + (lam[2] + lam[3]);  // this lane's and the later ones'
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
              const float v = __shfl_down_sync(0xffffffffu, down, d);
              if (lane + d < 32) down += v;
            }
            float a = __shfl_down_sync(0xffffffffu, down, 1);
            if (lane == 31) a = 0.f;
            last[e] = __shfl_sync(0xffffffffu, down, 0);
#pragma unroll
            for (int t = 3; t >= 0; --t) {
              after[e][t] = a;
              a += lam[t];
            }
          }
          if (c + 1 < u.chunks) fetch(c + 1);
          if (g > 0) {  // the last chunk's have been read
            wait_warp(L::kWx, (g - 1) & 1);
            wait_warp(kMode == kLocal ? L::kHFull : L::kMFull, (g - 1) & 1);
            if (!ok) break;
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            *(float4*)(saft + e * kQ + 4 * lane) = make_float4(after[e][0], after[e][1], after[e][2], after[e][3]);
            *(float4*)(sv + e * kQ + 4 * lane) = make_float4(lg2(dt[e][0]) - after[e][0], lg2(dt[e][1]) - after[e][1],
                                                             lg2(dt[e][2]) - after[e][2], lg2(dt[e][3]) - after[e][3]);
            const float end = __shfl_sync(0xffffffffu, after[e][3], lane | 7);  // behind these 32 tokens
            if (lane < 24)
              *(float4*)(su + e * 96 + 4 * lane) =
                  make_float4(dt[e][0] * ex2(end - after[e][0]), dt[e][1] * ex2(end - after[e][1]),
                              dt[e][2] * ex2(end - after[e][2]), dt[e][3] * ex2(end - after[e][3]));
            if (lane == 0) slast[e] = last[e];
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::kScan));
        }
        if (kMode != kMore || !ok) break;
        // ---- the next unit: asked for with the last chunk of this one
        wait_warp(L::kNext, n & 1);
        if (!ok) break;
        asked = false;
        int cta;
        const bool taken = cta_taken(sb + L::kAnswer, cta);
        wait_warp(L::kUnitEmpty, (n & 1) ^ 1);
        if (!ok) break;
        if (lane == 0) {
          *(volatile int*)(smem + L::kUnit) = taken ? cta : -1;
          mbar_arrive(bar(L::kUnitFull));
        }
        __syncwarp();
        if (!taken) break;
        u = whole(cta);
      }
      if (asked) {  // give-up: the answer lands before the shared memory is left
        for (int i = 0; i < (1 << 20) && !mbar_try_wait(bar(L::kNext), (asks - 1) & 1); ++i) {
        }
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 16) tmem_dealloc(tmem, 512);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // no launch after this one begins before the rows' is complete
}

// A launch whose CTAs may begin (early) when all of the launch before have
// begun or ended; the kernel itself waits for that launch to be complete.
template <typename K>
static cudaError_t launch(K kernel, dim3 grid, int threads, int smem, cudaStream_t st, bool early, const StateParams& p) {
  cudaLaunchAttribute a;
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = early;
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  c.attrs = &a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, p);
}

// Once per device, when a handle is made.
cudaError_t configure_prompt_state() {
  const void* kernels[3] = {(const void*)k_prompt_state<kLocal>, (const void*)k_prompt_state<kOnce>,
                            (const void*)k_prompt_state<kMore>};
  cudaError_t e = cudaSuccess;
  for (const void* k : kernels)
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, StateSmem::kTotal);
  return e;
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
  if (zx_stride < pl.in_rows || zx_stride % 4 || out_stride < pl.d_inner || out_stride % 8 || zx_stride > kMaxStride ||
      out_stride > kMaxStride || !aligned16(weights) || !aligned16(zxbcdt) || !aligned16(state_in) ||
      !aligned16(state_out) || !aligned16(out))
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
  p.zx = (const uint16_t*)zxbcdt;
  p.prm = (const uint16_t*)weights + hyb_layer_offset(pl.pk_M, pl.pk_layer, e, layer) + pl.pk_a_log;
  p.state_in = state_in ? state_in + lm * per_layer : nullptr;
  p.state_out = state_out + lm * per_layer;
  p.out = (uint16_t*)out;
  p.zx_stride = zx_stride;
  p.out_stride = out_stride;
  cudaStream_t st = (cudaStream_t)stream;
  h->last_stream = st;
  p.sink = make_sink(h->ws.err, h->err_host_dev, h->timeout_ns);
  p.skip = h->skip_sig_kind == 10 ? h->skip_sig : -1;
  // short sequences go token by token, the others in chunks, longest first
  SeqBatch all = p.b;
  int order[WAVE_MAX_SEQS];
  for (int i = 0; i < all.n; ++i) order[i] = i;
  std::stable_sort(order, order + all.n, [&](int a, int b) { return all.len(a) > all.len(b); });
  const int pairs = Hs / 2, sms = pl.grid;
  auto upto = [&](int tokens) {
    int c = 0;
    for (int i = 0; i < all.n; ++i) c += all.len(i) <= tokens;
    return c;
  };
  const int n_short = upto(Hs * upto(kRowTokensFew) <= sms / 2 ? kRowTokensFew : kRowTokensMany);
  const int n_between = n_short - upto(kRowTokensMany);  // those that are short in this call only
  int n_long = all.n - n_short;
  // Segments: the shortest that give no more CTAs than SMs, if that is worth
  // two more launches.  A chunk of the first costs about half of one of the
  // last, the launches about two (2048 tokens of 64 heads: 77 us as 32 CTAs
  // of 16 chunks, 49 in segments of 4; of 4 heads 23 in segments of 1).
  auto chunks = [&](int k) { return (all.len(order[k]) + kQ - 1) / kQ; };
  auto segments = [&](int t) {
    int n = 0;
    for (int k = 0; k < n_long; ++k) n += (chunks(k) + t - 1) / t;
    return n;
  };
  int t = 1;
  while (n_long * pairs <= sms && t < chunks(0) && segments(t) * pairs > sms) ++t;
  const bool cut = n_long && n_long * pairs <= sms && 3 * t + 4 < 2 * chunks(0);
  // What is short in this call only goes along with long ones where SMs are
  // left for it, and where long ones take all SMs several times over: a few
  // chunks more cost less than rows of their own.  Up to kRowTokensMany tokens
  // are always rows: their arithmetic does not depend on who else is there.
  const int left = sms - (cut ? segments(t) : n_long) * pairs;
  if (n_long && (n_between * pairs <= left || n_long * pairs > sms)) n_long += n_between;
  auto take = [&](int from, int to) {
    p.b.n = 0;
    for (int k = from; k < to; ++k) {
      const int i = order[k];
      p.b.begin[p.b.n] = all.begin[i];
      p.b.slot[p.b.n] = all.slot[i];
      p.b.start[p.b.n] = all.start[i];
      p.b.cum[p.b.n + 1] = p.b.cum[p.b.n] + all.len(i);
      ++p.b.n;
    }
    return p.b.n;
  };
  p.tiled = zx_stride % 8 == 0;
  if (n_long && p.tiled && encode_rows_map(&p.tm, zxbcdt, pl.in_rows, 1, cu_seqlens[n_seq], zx_stride, kQ)) return WAVE_ECUDA;
  // The rows first: the long ones' CTAs begin beside them (they are other
  // sessions') and end after them (16 prompts of 64 heads, two of them short:
  // 96 us, as with those two in chunks; 56 single tokens beside one of 600: 64
  // instead of 66; seven prompts of 32 heads that leave SMs idle: 36 instead
  // of 32).
  const bool rows = take(n_long, all.n);
  if (rows) {
    // Few heads are cut into four CTAs each while all of these run at once (64
    // heads, 25 tokens: 6.9 against 8.0 us; 256 heads, 16 tokens: 10.3 / 8.2).
    if (Hs * p.b.n * 4 <= sms * 2)
      k_prompt_state_rows<16><<<dim3(Hs * 4, p.b.n), 64, 0, st>>>(p);
    else
      k_prompt_state_rows<64><<<dim3(Hs, p.b.n), 256, 0, st>>>(p);
  }
  if (take(0, n_long)) {
    p.seg_chunks = cut ? t : 0;
    p.seg_cum[0] = 0;
    for (int k = 0; k < n_long; ++k) p.seg_cum[k + 1] = p.seg_cum[k] + (cut ? (chunks(k) + t - 1) / t : 1);
    p.seg_state = h->ws.seg_state;
    p.seg_decay = h->ws.seg_decay;
    const int ctas = p.seg_cum[n_long] * pairs;
    auto long_ones = [&](auto kernel, bool early) {
      return launch(kernel, dim3(ctas), kStateThreads, StateSmem::kTotal, st, early, p) == cudaSuccess;
    };
    if (cut) {
      // Where a third of the SMs is free, the CTAs of the second and third
      // launch begin beside those of the one before and wait for them (2048
      // tokens of 4 heads 28.4 -> 23.4 us; 128 CTAs 27.1 -> 28.6).
      const bool early = 3 * ctas <= 2 * sms;
      if (!long_ones(k_prompt_state<kLocal>, rows) ||
          launch(k_segment_states, dim3(128 * kSsmN / 4 / 256, pairs, p.b.n), 256, 0, st, early, p) != cudaSuccess ||
          !long_ones(k_prompt_state<kOnce>, early))
        return WAVE_ECUDA;
    } else if (!(ctas > sms ? long_ones(k_prompt_state<kMore>, rows) : long_ones(k_prompt_state<kOnce>, rows))) {
      return WAVE_ECUDA;
    }
  }
  return cudaGetLastError() == cudaSuccess ? WAVE_OK : WAVE_ECUDA;
}
