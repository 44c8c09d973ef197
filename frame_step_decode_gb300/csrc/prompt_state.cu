// prompt_state.cu -- wave_hybrid_prompt_state: the hybrid's selective-state
// block over packed prompts.  Per head, with dt_t = softplus(dt_t + dt_bias)
// and a_t = exp(-exp(A_log) dt_t):
//
//   h_t = a_t h_{t-1} + dt_t x_t B_t^T,   y_t = h_t C_t + D x_t,   out_t = bf16(y_t silu(z_t))
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/wave.h"
#include "ctx.h"
#include "prompt.h"
#include "prompt_ptx.cuh"

using namespace wave;

namespace wave {

// Sequences of at most this many tokens go token by token (a launch of the
// chunked form costs some microseconds whatever its length).
constexpr int kRowTokens = 8;

struct StateParams {
  SeqBatch b;
  CUtensorMap tm;          // the rows of zx as tiles of 64 columns x 128 tokens
  int tiled;               // whether tm is there: a row stride of a multiple of 16 bytes
  int Hs, S_max;
  const uint16_t* zx;      // [rows][zx_stride] bf16: z | x | B | C | dt
  const uint16_t* prm;     // A_log[Hs] | dt_bias[Hs] | D[Hs]
  const float* state_in;   // the layer's [S_max][Hs][64][128]
  float* state_out;
  uint16_t* out;           // [rows][out_stride] bf16
  long long zx_stride, out_stride;
  ErrSink sink;
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
// over the whole sequence.  M and the H of C H^T are rounded to bf16 once
// (the output is bf16); (w X)^T is split into a bf16 and the bf16 of its
// remainder (2^-18), since the state is carried on in fp32.
//
// Five warpgroups: two in front (a head each: the decays, the state's pass
// between chunks, M), two behind (the weights w, (w X)^T, the gated output),
// and one warp each for the MMAs, the copies of B, C, x and those of z.  The
// chain from chunk to chunk is the state's: its pass and its product.
constexpr int kQ = 128;                 // tokens of a chunk
constexpr int kStateThreads = 640;
// Registers: 640 threads are launched with 96 each (61440); the split is
// 256 x 112 + 256 x 104 + 128 x 48, the same sum.
constexpr int kRegsFront = 112, kRegsBehind = 104, kRegsRest = 48;
static_assert(256 * kRegsFront + 256 * kRegsBehind + 128 * kRegsRest <= kStateThreads * 96, "registers");
constexpr int kBC = kQ * kSsmN * 2;     // bytes of the B (or C) tile
constexpr int kXT = kQ * kSsmP * 2;     // ... of one head's x (or z) tile

struct StateSmem {
  static constexpr int kBuf = 2 * kBC + 2 * kXT;  // B, C (later z, then out, of both heads), x of both heads
  static constexpr int kH = 2 * kBuf;             // bf16 H of both heads: [2][n / 64][64 rows of 128 B]
  static constexpr int kV = kH + 2 * kXT;         // [head][128] log2 dt_j - (the decays behind j, to the chunk's end)
  static constexpr int kU = kV + 2 * kQ * 4;      // [head][96] dt_j 2^-(the decays behind j in its 32 tokens)
  static constexpr int kW = kU + 2 * 96 * 4;      // [head][128] w_j
  static constexpr int kTot = kW + 2 * kQ * 4;    // [in front, behind][head][32 tokens] sums of decays
  static constexpr int kBad = kTot + 2 * 2 * 4 * 4;  // [chunk % 4] bit head * 4 + warp: an x that is not finite
  static constexpr int kBars = kBad + 4 * 4;
  enum {
    kFull = 0,             // B and x
    kEmpty = kFull + 2,
    kCFull = kEmpty + 2,   // C
    kCEmpty = kCFull + 2,  // ... and the z and out that follow it
    kZFull = kCEmpty + 2,
    kG,
    kY2,
    kHFull,
    kMFull,
    kYFull = kMFull + 2,
    kYFree = kYFull + 2,
    kWx,
    kS,
    kDone,
    kCount
  };
  static constexpr int kMisc = kBars + kCount * 8;
  static constexpr int kTotal = kMisc + 16;
};
static_assert(StateSmem::kTotal <= 232448, "the chunked state form does not fit shared memory");

// TMEM columns: G (the heads' M later, 64 each), (w X)^T (high parts, then
// remainders), the state, Y of each head.
constexpr int kTG = 0, kTWx = 128, kTState = 256, kTY = 384;

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Rows that no tensor map can describe (a stride that is no multiple of 16
// bytes) are copied by the 256 threads behind, 8 bytes at a time: 128 tokens x
// kCols values at column `col` of the rows from row0 on, as the same 128-byte
// swizzled blocks of 64 columns.  Rows from n on repeat row n - 1.
template <int kCols>
__device__ __forceinline__ void copy_tile(uint32_t dst, const uint16_t* zx, long long stride, int col, size_t row0, int n) {
  constexpr int kPer = kCols * 2 / 8;  // pieces of a row
#pragma unroll 4
  for (int q = threadIdx.x & 255; q < kQ * kPer; q += 256) {
    const int r = q / kPer, b = (q % kPer) * 8, blk = b >> 7, c = (b >> 4) & 7;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst + blk * (kQ * 128) + r * 128 + ((c ^ (r & 7)) << 4) + (b & 15)),
                 "l"(zx + (row0 + min(r, n - 1)) * stride + col + b / 2)
                 : "memory");
  }
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

__global__ void __launch_bounds__(kStateThreads, 1) k_prompt_state(const __grid_constant__ StateParams p) {
  using L = StateSmem;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pairs = p.Hs / 2, seq = blockIdx.x / pairs, h0 = (blockIdx.x % pairs) * 2;
  const size_t first = p.b.begin[seq];
  const int len = p.b.len(seq), chunks = (len + kQ - 1) / kQ;
  const bool goes_on = p.b.start[seq] > 0;  // the state begins as state_in, not as zero
  const int di = p.Hs * kSsmP;
  auto bar = [&](int b) { return sb + L::kBars + b * 8; };
  uint32_t* tmem_word = (uint32_t*)(smem + L::kMisc);
  if (sb & 1023) {  // the tiles' swizzle counts on it, and there is no room to align by hand
    if (threadIdx.x == 0) *(volatile int*)p.sink.err_out = atomicOr(p.sink.err, kErrTimeout) | kErrTimeout;
    return;
  }

  if (warp == 16) {
    if (lane == 0) {
      const int copies = p.tiled ? 1 : 256;
      for (int b = 0; b < 2; ++b) {
        mbar_init(bar(L::kFull + b), copies);
        mbar_init(bar(L::kEmpty + b), 1);
        mbar_init(bar(L::kCFull + b), copies);
        mbar_init(bar(L::kCEmpty + b), 256);
        mbar_init(bar(L::kMFull + b), 128);
        mbar_init(bar(L::kYFull + b), 1);
      }
      mbar_init(bar(L::kZFull), copies);
      mbar_init(bar(L::kG), 1);
      mbar_init(bar(L::kY2), 1);
      mbar_init(bar(L::kHFull), 256);
      mbar_init(bar(L::kYFree), 256);
      mbar_init(bar(L::kWx), 256);
      mbar_init(bar(L::kS), 1);
      mbar_init(bar(L::kDone), 1);
      fence_mbar_init();
      fence_proxy_async_smem();
    }
    __syncwarp();
    tmem_alloc(smem_u32(tmem_word), 512);
    tmem_relinquish();
  }
  if (threadIdx.x < 4) ((uint32_t*)(smem + L::kBad))[threadIdx.x] = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_word;

  // In the compute warps a wait that gives up leaves the rest of the loop
  // without waits (the named barriers need every warp), with its results
  // undefined; the other warps leave their loops.
  bool ok = true;
  auto wait_warp = [&](int b, uint32_t parity) {
    if (ok) ok = __all_sync(0xffffffffu, wait_bar(bar(b), parity, p.sink));
  };
  auto wait = [&](int b, uint32_t parity) { return ok = wait_bar(bar(b), parity, p.sink); };
  const int h = (warp >> 2) & 1, quad = warp & 3, row = quad * 32 + lane;  // a thread per token of head h0 + h
  const uint32_t lanes = (uint32_t)(quad * 32) << 16;
  const int hh = row >> 6, pp = row & 63;  // for the state: row (head hh, p), half h of the columns or tokens
  const int head = h0 + h;
  float* sv = (float*)(smem + L::kV);
  float* su = (float*)(smem + L::kU);
  float* sw = (float*)(smem + L::kW);
  uint32_t* sbad = (uint32_t*)(smem + L::kBad);
  // the decays: this token's dt of chunk c (0 behind the sequence's end), the
  // sum of the later tokens' log-decays among its 32 (in powers of two), and
  // the sum of all 32 for the others.  Summed from the end: the state's newest
  // tokens are exact to fp32 whatever the sum over the chunk is.
  const uint16_t* dt_col = p.zx + first * p.zx_stride + 2 * di + 2 * kSsmN + head;
  const float rate = warp < 16 ? ex2(bf(p.prm[head]) * 1.44269504088896340736f) * 1.44269504088896340736f : 0.f;
  const float bias = warp < 16 ? bf(p.prm[p.Hs + head]) : 0.f;
  auto dt_at = [&](int c) { return c * kQ + row < len ? dt_col[(size_t)(c * kQ + row) * p.zx_stride] : (uint16_t)0; };
  auto decays = [&](int c, uint16_t raw, float& dt, float& inner) {
    dt = c * kQ + row < len ? softplus(bf(raw) + bias) : 0.f;
    // 2^-160 is zero in fp32: a larger step changes nothing, and the cap bounds the sums' rounding
    float down = fminf(rate * dt, 160.f);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const float v = __shfl_down_sync(0xffffffffu, down, d);
      if (lane + d < 32) down += v;
    }
    inner = __shfl_down_sync(0xffffffffu, down, 1);
    if (lane == 31) inner = 0.f;
    return down;  // lane 0: the sum of all 32
  };
  const size_t state_at = (((size_t)p.b.slot[seq] * p.Hs + h0) * kSsmP + row) * kSsmN + h * 64;

  if (warp < 8) {
    // -------------------------------------------------------------- in front
    regs_take<kRegsFront>();
    const float skip = bf(p.prm[2 * p.Hs + head]);
    uint16_t dt_next = dt_at(0);
    for (int c = 0; c < chunks; ++c) {
      // ---- the decays
      float dt, inner;
      const float sum = decays(c, dt_next, dt, inner);
      dt_next = dt_at(c + 1);
      float* tot = (float*)(smem + L::kTot);
      if (lane == 0) tot[h * 4 + quad] = sum;
      bar_sync(1, 256);  // also: the last chunk's sv and su have been read
      float end[4];  // behind each 32 tokens
      end[3] = 0.f;
#pragma unroll
      for (int q = 2; q >= 0; --q) end[q] = end[q + 1] + tot[h * 4 + q + 1];
      const float after = inner + (quad == 0 ? end[0] : quad == 1 ? end[1] : quad == 2 ? end[2] : 0.f);
      const float last = end[0] + tot[h * 4];
      sv[h * kQ + row] = lg2(dt) - after;
      if (row < 96) su[h * 96 + row] = dt * ex2(-inner);
      // ---- the state: its bf16 copy for C H^T, and the chunk's decay
      if (c > 0) wait_warp(L::kS, (c - 1) & 1);
      tc_fence_after();
      const bool zero = c == 0 && !goes_on;
      if (!zero) {
        const float dec = ex2(-((tot[hh * 4] + tot[hh * 4 + 1]) + (tot[hh * 4 + 2] + tot[hh * 4 + 3])));
        uint8_t* hrow = smem + L::kH + hh * kXT + h * (64 * 128) + pp * 128;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          uint32_t v[16];
          if (c == 0) {
            const float4* src = (const float4*)(p.state_in + state_at + 16 * q);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 f = src[e];
              v[4 * e] = __float_as_uint(f.x), v[4 * e + 1] = __float_as_uint(f.y);
              v[4 * e + 2] = __float_as_uint(f.z), v[4 * e + 3] = __float_as_uint(f.w);
            }
          } else {
            tmem_ld16_nowait(tmem + kTState + lanes + h * 64 + 16 * q, v);
            tmem_ld_wait();
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint4 w;
            w.x = pack_bf16(__uint_as_float(v[8 * e]), __uint_as_float(v[8 * e + 1]));
            w.y = pack_bf16(__uint_as_float(v[8 * e + 2]), __uint_as_float(v[8 * e + 3]));
            w.z = pack_bf16(__uint_as_float(v[8 * e + 4]), __uint_as_float(v[8 * e + 5]));
            w.w = pack_bf16(__uint_as_float(v[8 * e + 6]), __uint_as_float(v[8 * e + 7]));
            *(uint4*)(hrow + (((2 * q + e) ^ (pp & 7)) << 4)) = w;
          }
          scale_regs<16>(v, dec);
          tmem_st16(tmem + kTState + lanes + h * 64 + 16 * q, v);
        }
        tmem_st_wait();
        fence_proxy_async_smem();
      }
      tc_fence_before();
      mbar_arrive(bar(L::kHFull));
      bar_sync(2 + h, 128);  // the head's sv and su are complete
      // ---- M, over G once both heads have read G
      wait_warp(L::kG, c & 1);
      tc_fence_after();
      // 32 tokens at a time, from the diagonal down: m[16 t ..] is block quad - t
      uint32_t m[64];
      {
        // on the diagonal; D x_i is added to y_i as D on the diagonal
        uint32_t g[32];
        tmem_ld32(tmem + kTG + lanes + 32 * quad, g);
        const float2 ai = make_float2(after, after);
        const float4* vj = (const float4*)(sv + h * kQ + 32 * quad);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float4 v4 = vj[e];
          const float2 t0 = add2(make_float2(v4.x, v4.y), ai), t1 = add2(make_float2(v4.z, v4.w), ai);
          const float2 m0 = mul2(make_float2(__uint_as_float(g[4 * e]), __uint_as_float(g[4 * e + 1])),
                                 make_float2(ex2(t0.x), ex2(t0.y)));
          const float2 m1 = mul2(make_float2(__uint_as_float(g[4 * e + 2]), __uint_as_float(g[4 * e + 3])),
                                 make_float2(ex2(t1.x), ex2(t1.y)));
          float f[4] = {m0.x, m0.y, m1.x, m1.y};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (4 * e + k > lane) f[k] = 0.f;
            if (4 * e + k == lane) f[k] += skip;
          }
          m[2 * e] = pack_bf16(f[0], f[1]);
          m[2 * e + 1] = pack_bf16(f[2], f[3]);
        }
      }
#pragma unroll
      for (int t = 1; t < 4; ++t) {
        if (t > quad) continue;
        // below: the decay from the end of token j's block to i is a factor
        // of the row, that from j to there is in u_j
        const int q = quad - t;
        uint32_t g[32];
        tmem_ld32(tmem + kTG + lanes + 32 * q, g);
        const float r = ex2(after - (q == 0 ? end[0] : q == 1 ? end[1] : end[2]));
        const float2 r2 = make_float2(r, r);
        const float4* uj = (const float4*)(su + h * 96 + 32 * q);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float4 u4 = uj[e];
          const float2 m0 = mul2(mul2(make_float2(__uint_as_float(g[4 * e]), __uint_as_float(g[4 * e + 1])), r2),
                                 make_float2(u4.x, u4.y));
          const float2 m1 = mul2(mul2(make_float2(__uint_as_float(g[4 * e + 2]), __uint_as_float(g[4 * e + 3])), r2),
                                 make_float2(u4.z, u4.w));
          m[16 * t + 2 * e] = pack_bf16(m0.x, m0.y);
          m[16 * t + 2 * e + 1] = pack_bf16(m1.x, m1.y);
        }
      }
      tc_fence_before();
      bar_sync(1, 256);  // both heads have read G
      tc_fence_after();
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if (t <= quad) {
          tmem_st16(tmem + kTG + h * 64 + lanes + 16 * (quad - t), m + 16 * t);
        } else {  // above the diagonal
          uint32_t none[16] = {};
          tmem_st16(tmem + kTG + h * 64 + lanes + 16 * t, none);
        }
      }
      // ---- C H^T, scaled in place: M X is added to it
      wait_warp(L::kY2, c & 1);
      tc_fence_after();
      if (!zero) {
        const float ei = ex2(after - last);
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
      mbar_arrive(bar(L::kMFull + h));
    }
    // ---- the state after the last token
    wait_warp(L::kS, (chunks - 1) & 1);
    tc_fence_after();
#pragma unroll 1
    for (int q = 0; q < 2; ++q) {
      uint32_t v[32];
      tmem_ld32(tmem + kTState + lanes + h * 64 + q * 32, v);
      tmem_ld_wait();
      float4* dst = (float4*)(p.state_out + state_at + 32 * q);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        dst[e] = make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]), __uint_as_float(v[4 * e + 2]),
                             __uint_as_float(v[4 * e + 3]));
    }
  } else if (warp < 16) {
    // ---------------------------------------------------------------- behind
    regs_take<kRegsBehind>();
    // (w X)^T of a chunk is made before the output of the chunk before it: the
    // state's product does not wait for the gate
    uint16_t dt_next = dt_at(0);
    for (int c = -1; c < chunks; ++c) {
      if (c + 1 < chunks) {
        const int k = c + 1, b = k & 1, left = len - k * kQ;
        uint8_t* buf = smem + b * L::kBuf;
        // ---- this token's x and B.  Behind the sequence's end lie other rows:
        // theirs become zero.  An x that is not finite would reach earlier
        // tokens as 0 * NaN in M X: it is noted here, becomes zero once the
        // state's weights have been made of it, and is put back at the output.
        if (!p.tiled) {
          const size_t row0 = first + (size_t)k * kQ;
          const int n = min(kQ, left);
          wait_warp(L::kEmpty + b, ((k >> 1) & 1) ^ 1);
          wait_warp(L::kCEmpty + b, ((k >> 1) & 1) ^ 1);
          copy_tile<2 * kSsmN>(sb + b * L::kBuf, p.zx, p.zx_stride, 2 * di, row0, n);  // B, then C
          copy_tile<2 * kSsmP>(sb + b * L::kBuf + 2 * kBC, p.zx, p.zx_stride, di + h0 * kSsmP, row0, n);
          asm volatile("cp.async.wait_all;" ::: "memory");
          fence_proxy_async_smem();
          mbar_arrive(bar(L::kFull + b));
          mbar_arrive(bar(L::kCFull + b));
        }
        float dt, inner;
        const float sum = decays(k, dt_next, dt, inner);
        dt_next = dt_at(k + 1);
        float* tot = (float*)(smem + L::kTot) + 8;
        if (lane == 0) tot[h * 4 + quad] = sum;
        wait_warp(L::kFull + b, (k >> 1) & 1);
        uint8_t* xrow = buf + 2 * kBC + h * kXT + row * 128;
        bool odd = false;
        if (row >= left) {
          uint8_t* brow = buf + h * (kQ * 128) + row * 128;
#pragma unroll 4
          for (int e = 0; e < 8; ++e) {
            *(uint4*)(xrow + (e << 4)) = make_uint4(0, 0, 0, 0);
            *(uint4*)(brow + (e << 4)) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        } else {
          uint32_t acc[2] = {0, 0};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint4 x = *(const uint4*)(xrow + ((e ^ (lane & 7)) << 4));
            asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc[0]) : "r"(x.x), "r"(0));
            asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc[1]) : "r"(x.y), "r"(0));
            asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc[0]) : "r"(x.z), "r"(0));
            asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc[1]) : "r"(x.w), "r"(0));
          }
          odd = ((acc[0] | acc[1]) & 0x7fff7fffu) != 0;
          if (odd) atomicOr(&sbad[k & 3], 1u << (h * 4 + quad));
        }
        bar_sync(4, 256);  // x and its flags are complete; every thread here is done with chunk k - 2
        // cleared two chunks ahead: nobody sets these before the next barrier
        if ((threadIdx.x & 255) == 0) sbad[(k + 2) & 3] = 0;
        // ---- (w X)^T: row (hh, pp), tokens 64 h .. 64 h + 63
        {
          float after = inner;
#pragma unroll
          for (int q = 1; q < 4; ++q)
            if (q > quad) after += tot[h * 4 + q];
          sw[h * kQ + row] = dt * ex2(-after);
        }
        if (k > 0) wait_warp(L::kS, (k - 1) & 1);
        bar_sync(4, 256);  // sw is complete
        tc_fence_after();
        const uint8_t* xt = buf + 2 * kBC + hh * kXT + (pp & 7) * 2;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          const int j0 = h * 64 + 16 * q;
          float v[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)  // j0 is a multiple of 8
            v[e] = bf(*(const uint16_t*)(xt + (j0 + e) * 128 + (((pp >> 3) ^ (e & 7)) << 4)));
          const float4* wj = (const float4*)(sw + hh * kQ + j0);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 w4 = wj[e];
            const float2 r0 = mul2(make_float2(v[4 * e], v[4 * e + 1]), make_float2(w4.x, w4.y));
            const float2 r1 = mul2(make_float2(v[4 * e + 2], v[4 * e + 3]), make_float2(w4.z, w4.w));
            v[4 * e] = r0.x, v[4 * e + 1] = r0.y, v[4 * e + 2] = r1.x, v[4 * e + 3] = r1.y;
          }
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            hi[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
            const float2 r = sub2(make_float2(v[2 * e], v[2 * e + 1]),
                                  make_float2(__uint_as_float(hi[e] << 16), __uint_as_float(hi[e] & 0xFFFF0000u)));
            lo[e] = pack_bf16(r.x, r.y);
          }
          tmem_st8(tmem + kTWx + lanes + h * 32 + q * 8, hi);
          tmem_st8(tmem + kTWx + 64 + lanes + h * 32 + q * 8, lo);
        }
        tmem_st_wait();
        if (sbad[k & 3]) {  // seen by every thread or none
          bar_sync(4, 256);
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
        mbar_arrive(bar(L::kWx));
      }
      if (c < 0) continue;
      const int b = c & 1, left = len - c * kQ;
      uint8_t* buf = smem + b * L::kBuf;
      // ---- the output: y, gated, over z's row and from there to global
      uint8_t* ztile = buf + kBC + h * kXT;
      const uint32_t any_bad = sbad[c & 3] >> (h * 4) & 15u;
      if (!p.tiled) {
        wait_warp(L::kY2, c & 1);
        copy_tile<2 * kSsmP>(sb + b * L::kBuf + kBC, p.zx, p.zx_stride, h0 * kSsmP, first + (size_t)c * kQ, min(kQ, left));
        asm volatile("cp.async.wait_all;" ::: "memory");
        mbar_arrive(bar(L::kZFull));
      }
      wait_warp(L::kZFull, c & 1);
      wait_warp(L::kYFull + h, c & 1);
      tc_fence_after();
      uint8_t* zrow = ztile + row * 128;
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        uint32_t y[16];
        tmem_ld16_nowait(tmem + kTY + h * 64 + lanes + 16 * q, y);
        uint4 zv[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) zv[e] = *(const uint4*)(zrow + (((q * 2 + e) ^ (row & 7)) << 4));
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t zw[4] = {zv[e].x, zv[e].y, zv[e].z, zv[e].w};
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
          *(uint4*)(zrow + (((q * 2 + e) ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      tc_fence_before();
      mbar_arrive(bar(L::kYFree));
      if (any_bad) {  // tokens up to this one whose x is not finite
#pragma unroll 1
        for (int j = 0; j <= row && j < left; ++j) {
          if (!(any_bad >> (j >> 5) & 1)) continue;
          const uint16_t* x = p.zx + (first + (size_t)c * kQ + j) * p.zx_stride + di + head * kSsmP;
#pragma unroll 1
          for (int e = 0; e < 64; ++e)
            if ((x[e] & 0x7F80) == 0x7F80) *(uint16_t*)(zrow + (((e >> 3) ^ (row & 7)) << 4) + (e & 7) * 2) = 0x7FC0;
        }
      }
      __syncwarp();
      {
        const int r0 = quad * 32 + (lane >> 3), at = lane & 7;  // four rows at a time
        uint16_t* dst = p.out + (first + (size_t)c * kQ + r0) * p.out_stride + head * kSsmP + at * 8;
#pragma unroll 4
        for (int q = 0; q < 8; ++q, dst += 4 * p.out_stride) {
          const int r = r0 + 4 * q;
          const uint4 v = *(const uint4*)(ztile + r * 128 + ((at ^ (r & 7)) << 4));
          if (r < left) *(uint4*)dst = v;
        }
      }
      fence_proxy_async_smem();  // the next copies into this buffer come by the async proxy
      mbar_arrive(bar(L::kCEmpty + b));
    }
  } else {
    regs_give<kRegsRest>();
    if (warp == 16) {
      // ---------------------------------------------------------------- MMAs
      constexpr uint32_t id_g = idesc_16(128, 128, false, false, false), id_y2 = idesc_16(128, 64, false, false, false),
                         id_y = idesc_16(128, 64, false, false, true), id_s = idesc_16(128, 128, false, false, true);
      constexpr uint32_t kBlk = (kQ * 128) >> 4;  // the next 64 columns of a tile, as a descriptor counts
      for (int c = 0; c < chunks; ++c) {
        const uint32_t buf = sb + (c & 1) * L::kBuf;
        const bool zero = c == 0 && !goes_on;
        wait_warp(L::kFull + (c & 1), (c >> 1) & 1);
        wait_warp(L::kCFull + (c & 1), (c >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {  // G = C B^T
          const uint32_t cm = sdesc_lo(buf + kBC), bm = sdesc_lo(buf);
          mma_ss<false>(tmem + kTG, cm, bm, id_g);
#pragma unroll
          for (int e = 1; e < 8; ++e)
            mma_ss<true>(tmem + kTG, cm + (e / 4) * kBlk + (e % 4) * 2, bm + (e / 4) * kBlk + (e % 4) * 2, id_g);
          tc_commit(bar(L::kG));
        }
        __syncwarp();
        wait_warp(L::kHFull, c & 1);
        wait_warp(L::kWx, c & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {  // the state += (w X)^T B: the high parts, then the remainders
          const uint32_t bm = sdesc_lo(buf, kQ * 128);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            mma_ts(tmem + kTState, tmem + kTWx + 8 * e, bm + (e % 8) * (2048 >> 4), id_s, e > 0 ? 1u : zero ? 0u : 1u);
          tc_commit(bar(L::kS));
        }
        __syncwarp();
        if (c > 0) wait_warp(L::kYFree, (c - 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {  // Y = C H^T
          if (!zero) {
            const uint32_t cm = sdesc_lo(buf + kBC), hm = sdesc_lo(sb + L::kH);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              mma_ss<false>(tmem + kTY + h * 64, cm, hm + h * (kXT >> 4), id_y2);
#pragma unroll
              for (int e = 1; e < 8; ++e)
                mma_ss<true>(tmem + kTY + h * 64, cm + (e / 4) * kBlk + (e % 4) * 2,
                             hm + ((h * kXT + (e / 4) * (64 * 128)) >> 4) + (e % 4) * 2, id_y2);
            }
          }
          tc_commit(bar(L::kY2));
        }
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // Y += M X
          wait_warp(L::kMFull + h, c & 1);
          tc_fence_after();
          if (ok && elect_one()) {
            const uint32_t xm = sdesc_lo(buf + 2 * kBC + h * kXT, kQ * 128);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              mma_ts(tmem + kTY + h * 64, tmem + kTG + h * 64 + 8 * e, xm + e * (2048 >> 4), id_y, e > 0 ? 1u : zero ? 0u : 1u);
            tc_commit(bar(L::kYFull + h));
          }
          __syncwarp();
        }
        if (!ok) break;
        if (elect_one()) tc_commit(bar(L::kEmpty + (c & 1)));
        __syncwarp();
      }
      if (!ok) {  // give-up: wait (bounded) for the MMAs issued so far
        if (elect_one()) tc_commit(bar(L::kDone));
        __syncwarp();
        for (int n = 0; n < (1 << 20) && !mbar_try_wait(bar(L::kDone), 0); ++n) {
        }
      }
      __syncwarp();
    } else if (warp == 17) {
      // ------------------------------------------------ copies of B, C and x
      if (p.tiled) {
        if (lane == 0) {
          int c = 0;
          for (; c < chunks; ++c) {
            const uint32_t buf = sb + (c & 1) * L::kBuf, fb = bar(L::kFull + (c & 1)), fc = bar(L::kCFull + (c & 1));
            const uint32_t parity = ((c >> 1) & 1) ^ 1;
            const int r = (int)first + c * kQ;
            if (!wait(L::kEmpty + (c & 1), parity)) break;
            mbar_arrive_expect_tx(fb, kBC + 2 * kXT);
            tma_load_3d_plain(buf, &p.tm, 2 * di, 0, r, fb);
            tma_load_3d_plain(buf + kQ * 128, &p.tm, 2 * di + 64, 0, r, fb);
            tma_load_3d_plain(buf + 2 * kBC, &p.tm, di + h0 * kSsmP, 0, r, fb);
            tma_load_3d_plain(buf + 2 * kBC + kXT, &p.tm, di + (h0 + 1) * kSsmP, 0, r, fb);
            if (!wait(L::kCEmpty + (c & 1), parity)) {
              ++c;
              break;
            }
            mbar_arrive_expect_tx(fc, kBC);
            tma_load_3d_plain(buf + kBC, &p.tm, 2 * di + kSsmN, 0, r, fc);
            tma_load_3d_plain(buf + kBC + kQ * 128, &p.tm, 2 * di + kSsmN + 64, 0, r, fc);
          }
          if (!ok)  // give-up: the copies in flight land before the shared memory is left
            for (int i = max(0, c - 2); i < c; ++i) {
              for (int n = 0; n < (1 << 20) && !mbar_try_wait(bar(L::kFull + (i & 1)), (i >> 1) & 1); ++n) {
              }
              for (int n = 0; n < (1 << 12) && !mbar_try_wait(bar(L::kCFull + (i & 1)), (i >> 1) & 1); ++n) {
              }
            }
        }
      }
      __syncwarp();
    } else if (warp == 18) {
      // ---------------------------- copies of z, over C once its products are done
      if (p.tiled) {
        if (lane == 0) {
          int c = 0;
          for (; c < chunks; ++c) {
            const uint32_t dst = sb + (c & 1) * L::kBuf + kBC;
            const int r = (int)first + c * kQ;
            if (!wait(L::kY2, c & 1)) break;
            mbar_arrive_expect_tx(bar(L::kZFull), 2 * kXT);
            tma_load_3d_plain(dst, &p.tm, h0 * kSsmP, 0, r, bar(L::kZFull));
            tma_load_3d_plain(dst + kXT, &p.tm, (h0 + 1) * kSsmP, 0, r, bar(L::kZFull));
          }
          if (!ok && c > 0)
            for (int n = 0; n < (1 << 20) && !mbar_try_wait(bar(L::kZFull), (c - 1) & 1); ++n) {
            }
        }
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 16) tmem_dealloc(tmem, 512);
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
  p.sink = make_sink(h->ws.err, h->err_host_dev, h->timeout_ns);
  // short sequences go token by token, the others in chunks, longest first
  SeqBatch all = p.b;
  int order[WAVE_MAX_SEQS];
  for (int i = 0; i < all.n; ++i) order[i] = i;
  std::stable_sort(order, order + all.n, [&](int a, int b) { return all.len(a) > all.len(b); });
  auto take = [&](bool chunked) {
    p.b.n = 0;
    for (int k = 0; k < all.n; ++k) {
      const int i = order[k];
      if ((all.len(i) > kRowTokens) != chunked) continue;
      p.b.begin[p.b.n] = all.begin[i];
      p.b.slot[p.b.n] = all.slot[i];
      p.b.start[p.b.n] = all.start[i];
      p.b.cum[p.b.n + 1] = p.b.cum[p.b.n] + all.len(i);
      ++p.b.n;
    }
    return p.b.n;
  };
  p.tiled = zx_stride % 8 == 0;
  if (take(true)) {
    if (p.tiled && encode_rows_map(&p.tm, zxbcdt, pl.in_rows, 1, cu_seqlens[n_seq], zx_stride, kQ)) return WAVE_ECUDA;
    if (cudaFuncSetAttribute(k_prompt_state, cudaFuncAttributeMaxDynamicSharedMemorySize, StateSmem::kTotal) != cudaSuccess)
      return WAVE_ECUDA;
    k_prompt_state<<<p.b.n * (Hs / 2), kStateThreads, StateSmem::kTotal, st>>>(p);
  }
  if (take(false)) k_prompt_state_rows<<<dim3(Hs, p.b.n), 256, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? WAVE_OK : WAVE_ECUDA;
}
