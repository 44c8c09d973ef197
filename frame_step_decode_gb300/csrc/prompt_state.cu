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
constexpr int kQ = 128;                 // tokens of a chunk
constexpr int kStateThreads = 384;      // 8 compute warps, the MMA warp, 3 copy warps
constexpr int kCopyThreads = 96;
constexpr int kBC = kQ * kSsmN * 2;     // bytes of the B (or C) tile
constexpr int kXT = kQ * kSsmP * 2;     // ... of one head's x (or z) tile

struct StateSmem {
  static constexpr int kBuf = 2 * kBC + 2 * kXT;  // B, C (later z, then out, of both heads), x of both heads
  static constexpr int kH = 2 * kBuf;             // bf16 H of both heads: [2][n / 64][64 rows of 128 B]
  static constexpr int kA = kH + 2 * kXT;         // [head][128] c_j + log2 dt_j
  static constexpr int kW = kA + 2 * kQ * 4;      // [head][128] w_j
  static constexpr int kTot = kW + 2 * kQ * 4;    // [chunk parity][head][warp] sums of the warps' 32 tokens
  static constexpr int kBad = kTot + 2 * 2 * 4 * 4;  // [chunk parity][head][4] tokens with an x that is not finite
  static constexpr int kBars = kBad + 2 * 2 * 4 * 4;
  enum { kFull = 0, kEmpty = 2, kZFull = 4, kG = 5, kY2 = 6, kHFull = 7, kMFull = 8, kYFull = 10, kWx = 12, kS = 13, kDone = 14, kCount = 15 };
  static constexpr int kMisc = kBars + kCount * 8;
  static constexpr int kTotal = kMisc + 16;
};
static_assert(StateSmem::kTotal <= 232448, "the chunked state form does not fit shared memory");

// TMEM columns: G, then (w X)^T in its place (high parts, remainders); the
// state; M and Y of each head.
constexpr int kTG = 0, kTState = 128, kTM = 256, kTY = 384;

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool there) {  // zeros where it is not
  const int n = there ? kBytes : 0;
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// A tile of 128 tokens x kCols values at column `col` of the rows from `row0`
// on (n of them are there), 128-byte swizzled blocks of 64 columns.
template <int kCols, int kBytes>
__device__ __forceinline__ void copy_tile(uint32_t dst, const uint16_t* zx, long long stride, int col, size_t row0, int n,
                                          int tid) {
  constexpr int kPer = kCols * 2 / kBytes;  // pieces of a row
  for (int q = tid; q < kQ * kPer; q += kCopyThreads) {
    const int r = q / kPer, b = (q % kPer) * kBytes, blk = b >> 7, c = (b >> 4) & 7;
    const bool there = r < n;
    copy_async<kBytes>(dst + blk * (kQ * 128) + r * 128 + ((c ^ (r & 7)) << 4) + (b & 15),
                       zx + (row0 + (there ? r : 0)) * stride + col + b / 2, there);
  }
}

template <bool kWide>
__device__ __forceinline__ void state_copies(const StateParams& p, uint32_t sb, size_t first, int len, int h0, int tid,
                                             bool& ok) {
  using L = StateSmem;
  constexpr int kBytes = kWide ? 16 : 8;
  auto bar = [&](int i) { return sb + L::kBars + i * 8; };
  const int di = p.Hs * kSsmP, chunks = (len + kQ - 1) / kQ;
  for (int c = 0; c <= chunks && ok; ++c) {
    const uint32_t buf = sb + (c & 1) * L::kBuf;
    const size_t row0 = first + (size_t)c * kQ;
    const int n = min(kQ, len - c * kQ);
    if (c < chunks) {
      if (!(ok = wait_or_flag(bar(L::kEmpty + (c & 1)), ((c >> 1) & 1) ^ 1, p.sink, kErrTimeout))) break;
      copy_tile<kSsmN, kBytes>(buf, p.zx, p.zx_stride, 2 * di, row0, n, tid);
      copy_tile<kSsmN, kBytes>(buf + kBC, p.zx, p.zx_stride, 2 * di + kSsmN, row0, n, tid);
      for (int h = 0; h < 2; ++h)
        copy_tile<kSsmP, kBytes>(buf + 2 * kBC + h * kXT, p.zx, p.zx_stride, di + (h0 + h) * kSsmP, row0, n, tid);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (c > 0) {  // z of the chunk before, over its C once C's products are done
      if (!(ok = wait_or_flag(bar(L::kY2), (c - 1) & 1, p.sink, kErrTimeout))) break;
      for (int h = 0; h < 2; ++h)
        copy_tile<kSsmP, kBytes>(sb + ((c - 1) & 1) * L::kBuf + kBC + h * kXT, p.zx, p.zx_stride, (h0 + h) * kSsmP,
                                 row0 - kQ, min(kQ, len - (c - 1) * kQ), tid);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (c < chunks) {
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      fence_proxy_async_smem();
      mbar_arrive(bar(L::kFull + (c & 1)));
    }
    if (c > 0) {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      mbar_arrive(bar(L::kZFull));
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__global__ void __launch_bounds__(kStateThreads, 1) k_prompt_state(const __grid_constant__ StateParams p) {
  using L = StateSmem;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pairs = p.Hs / 2, i = blockIdx.x / pairs, h0 = (blockIdx.x % pairs) * 2;
  const size_t first = p.b.begin[i];
  const int len = p.b.len(i), chunks = (len + kQ - 1) / kQ;
  const bool goes_on = p.b.start[i] > 0;  // the state begins as state_in, not as zero
  auto bar = [&](int b) { return sb + L::kBars + b * 8; };
  uint32_t* tmem_word = (uint32_t*)(smem + L::kMisc);
  if (sb & 1023) {  // the tiles' swizzle counts on it, and there is no room to align by hand
    if (threadIdx.x == 0) *(volatile int*)p.sink.err_out = atomicOr(p.sink.err, kErrTimeout) | kErrTimeout;
    return;
  }

  if (warp == 8) {
    if (lane == 0) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(bar(L::kFull + b), kCopyThreads);
        mbar_init(bar(L::kEmpty + b), 257);  // the compute threads and the MMAs
        mbar_init(bar(L::kMFull + b), 128);
        mbar_init(bar(L::kYFull + b), 1);
      }
      mbar_init(bar(L::kZFull), kCopyThreads);
      mbar_init(bar(L::kG), 1);
      mbar_init(bar(L::kY2), 1);
      mbar_init(bar(L::kHFull), 256);
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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_word;

  bool ok = true;
  if (warp < 8) {
    // ------------------------------------------------------------- compute
    // Warps 4h..4h+3 have head h0 + h, a thread per token.  For the state a
    // thread has row (head hh, p) and half the columns.  A wait that gives up
    // leaves the rest of the loop without waits (the barriers below need
    // every warp), with its results undefined.
    auto wait = [&](int b, uint32_t parity) {
      if (ok) ok = __all_sync(0xffffffffu, wait_or_flag(bar(b), parity, p.sink, kErrTimeout));
    };
    const int h = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const int hh = row >> 6, pp = row & 63;  // the state's row
    const int head = h0 + h, di = p.Hs * kSsmP;
    float* sa = (float*)(smem + L::kA);
    float* sw = (float*)(smem + L::kW);
    float* tot = (float*)(smem + L::kTot);
    const float rate = expf(bf(p.prm[head])) * 1.44269504088896340736f, bias = bf(p.prm[p.Hs + head]);
    const float skip = bf(p.prm[2 * p.Hs + head]);
    const size_t state_at = (((size_t)p.b.slot[i] * p.Hs + h0) * kSsmP + row) * kSsmN + h * 64;
    const uint16_t* dt_col = p.zx + first * p.zx_stride + 2 * di + 2 * kSsmN + head;
    uint16_t dt_next = row < len ? dt_col[(size_t)row * p.zx_stride] : 0;
    if (threadIdx.x < 16) ((uint32_t*)(smem + L::kBad))[threadIdx.x] = 0;
    for (int c = 0; c < chunks; ++c) {
      const int b = c & 1, left = len - c * kQ;
      uint32_t* bad = (uint32_t*)(smem + L::kBad) + b * 8;
      uint8_t* buf = smem + b * L::kBuf;
      // ---- the decays
      float dt = 0.f;
      if (row < left) {
        const float raw = bf(dt_next) + bias;
        dt = raw > 0.f ? raw + log1pf(expf(-raw)) : log1pf(expf(raw));
      }
      if (row + kQ < left) dt_next = dt_col[(size_t)((c + 1) * kQ + row) * p.zx_stride];
      // 2^-160 is zero in fp32: a larger step changes nothing, and bounds the sums' rounding
      const float lam = fminf(rate * dt, 160.f);
      float up = lam, down = lam;  // sums of the warp's tokens up to this one, and from it on
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const float u = __shfl_up_sync(0xffffffffu, up, d), v = __shfl_down_sync(0xffffffffu, down, d);
        if (lane >= d) up += u;
        if (lane + d < 32) down += v;
      }
      float* tc = tot + b * 8;
      if (lane == 31) tc[h * 4 + quad] = up;
      bar_sync(1, 256);
      float ci = up, after = __shfl_down_sync(0xffffffffu, down, 1);  // the sum behind this token
      if (lane == 31) after = 0.f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (q < quad) ci += tc[h * 4 + q];
        if (q > quad) after += tc[h * 4 + q];
      }
      if (c > 0) wait(L::kS, (c - 1) & 1);  // also: nobody reads sa or sw of the last chunk any more
      tc_fence_after();
      sa[h * kQ + row] = ci + lg2(dt);
      sw[h * kQ + row] = dt * ex2(-after);
      // every thread is past the last chunk: its flags are cleared for the next one
      if (threadIdx.x < 8) ((uint32_t*)(smem + L::kBad))[(b ^ 1) * 8 + threadIdx.x] = 0;
      // ---- the state: its bf16 copy for C H^T, and the chunk's decay
      const bool zero = c == 0 && !goes_on;
      if (!zero) {
        const float* th = tc + hh * 4;
        const float dec = ex2(-((th[0] + th[1]) + (th[2] + th[3])));
        uint8_t* hrow = smem + L::kH + hh * kXT + h * (64 * 128) + pp * 128;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t v[32];
          if (c == 0) {
            const float4* src = (const float4*)(p.state_in + state_at + 32 * q);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 f = src[e];
              v[4 * e] = __float_as_uint(f.x), v[4 * e + 1] = __float_as_uint(f.y);
              v[4 * e + 2] = __float_as_uint(f.z), v[4 * e + 3] = __float_as_uint(f.w);
            }
          } else {
            tmem_ld32(tmem + kTState + lanes + h * 64 + q * 32, v);
            tmem_ld_wait();
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint4 w;
            w.x = pack_bf16(__uint_as_float(v[8 * e]), __uint_as_float(v[8 * e + 1]));
            w.y = pack_bf16(__uint_as_float(v[8 * e + 2]), __uint_as_float(v[8 * e + 3]));
            w.z = pack_bf16(__uint_as_float(v[8 * e + 4]), __uint_as_float(v[8 * e + 5]));
            w.w = pack_bf16(__uint_as_float(v[8 * e + 6]), __uint_as_float(v[8 * e + 7]));
            *(uint4*)(hrow + (((q * 4 + e) ^ (pp & 7)) << 4)) = w;
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * dec);
          tmem_st32(tmem + kTState + lanes + h * 64 + q * 32, v);
        }
        tmem_st_wait();
        fence_proxy_async_smem();
      }
      tc_fence_before();
      mbar_arrive(bar(L::kHFull));
      // ---- this token's x: a value that is not finite would reach earlier
      // tokens as 0 * NaN, so it is set to zero here and put back below
      wait(L::kFull + b, (c >> 1) & 1);
      uint8_t* xrow = buf + 2 * kBC + h * kXT + row * 128;
      {
        uint32_t acc = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint4 x = *(const uint4*)(xrow + (e << 4));
          asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x.x), "r"(0));
          asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x.y), "r"(0));
          asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x.z), "r"(0));
          asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x.w), "r"(0));
        }
        if (acc & 0x7fff7fffu) {
          for (int e = 0; e < 64; ++e) {
            uint16_t* x = (uint16_t*)xrow + e;
            if ((*x & 0x7F80) == 0x7F80) *x = 0;
          }
          atomicOr(&bad[h * 4 + quad], 1u << lane);
          fence_proxy_async_smem();
        }
      }
      bar_sync(1, 256);  // sa, sw and bad are complete
      // ---- M
      wait(L::kG, c & 1);
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t w[16];
        if (q <= quad) {
          uint32_t g[32];
          tmem_ld32(tmem + kTG + lanes + 32 * q, g);
          tmem_ld_wait();
          const float4* aj = (const float4*)(sa + h * kQ + 32 * q);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 a4 = aj[e];
            float m[4] = {__uint_as_float(g[4 * e]) * ex2(a4.x - ci), __uint_as_float(g[4 * e + 1]) * ex2(a4.y - ci),
                          __uint_as_float(g[4 * e + 2]) * ex2(a4.z - ci), __uint_as_float(g[4 * e + 3]) * ex2(a4.w - ci)};
            if (q == quad) {
#pragma unroll
              for (int f = 0; f < 4; ++f)
                if (4 * e + f > lane) m[f] = 0.f;
            }
            w[2 * e] = pack_bf16(m[0], m[1]);
            w[2 * e + 1] = pack_bf16(m[2], m[3]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = 0;
        }
        tmem_st16(tmem + kTM + h * 64 + lanes + 16 * q, w);
      }
      // ---- C H^T, scaled in place: M X is added to it
      wait(L::kY2, c & 1);
      tc_fence_after();
      if (!zero) {
        const float ei = ex2(-ci);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t v[32];
          tmem_ld32(tmem + kTY + h * 64 + lanes + 32 * q, v);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * ei);
          tmem_st32(tmem + kTY + h * 64 + lanes + 32 * q, v);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(bar(L::kMFull + h));
      bar_sync(1, 256);  // G has been read: (w X)^T goes in its place
      // ---- (w X)^T: row (hh, pp), tokens 64 h .. 64 h + 63
      const uint32_t any_bad = (bad[0] | bad[1] | bad[2] | bad[3]) | (bad[4] | bad[5] | bad[6] | bad[7]);
      {
        const uint8_t* xt = buf + 2 * kBC + hh * kXT + (pp & 7) * 2;
        const float* wj = sw + hh * kQ + h * 64;
        uint32_t hi[32], lo[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          float v[2];
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const int j = h * 64 + 2 * e + f;
            v[f] = wj[2 * e + f] * bf(*(const uint16_t*)(xt + j * 128 + (((pp >> 3) ^ (j & 7)) << 4)));
          }
          if (any_bad) {
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const int j = h * 64 + 2 * e + f;
              if (bad[hh * 4 + (j >> 5)] >> (j & 31) & 1)
                v[f] = wj[2 * e + f] * bf(p.zx[(first + (size_t)c * kQ + j) * p.zx_stride + di + (h0 + hh) * kSsmP + pp]);
            }
          }
          hi[e] = pack_bf16(v[0], v[1]);
          lo[e] = pack_bf16(v[0] - __uint_as_float(hi[e] << 16), v[1] - __uint_as_float(hi[e] & 0xFFFF0000u));
        }
        tmem_st32(tmem + kTG + lanes + h * 32, hi);
        tmem_st32(tmem + kTG + 64 + lanes + h * 32, lo);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(bar(L::kWx));
      // ---- the output: y + D x, gated, over z's row and from there to global
      wait(L::kYFull + h, c & 1);
      wait(L::kZFull, c & 1);
      tc_fence_after();
      uint8_t* ztile = buf + kBC + h * kXT;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t y[32];
        tmem_ld32(tmem + kTY + h * 64 + lanes + 32 * q, y);
        tmem_ld_wait();
        if (any_bad) {  // tokens up to this one whose x is not finite
          for (int j = 0; j <= row; ++j) {
            if (!(bad[h * 4 + (j >> 5)] >> (j & 31) & 1)) continue;
            const uint16_t* x = p.zx + (first + (size_t)c * kQ + j) * p.zx_stride + di + head * kSsmP + 32 * q;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if ((x[e] & 0x7F80) == 0x7F80) y[e] = 0x7FC00000u;
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int at = ((q * 4 + e) ^ (row & 7)) << 4;
          const uint4 xv = *(const uint4*)(xrow + at), zv = *(const uint4*)(ztile + row * 128 + at);
          const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w}, zw[4] = {zv.x, zv.y, zv.z, zv.w};
          uint32_t o[4];
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            float r[2];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const float x = __uint_as_float(g ? xw[f] & 0xFFFF0000u : xw[f] << 16);
              const float z = __uint_as_float(g ? zw[f] & 0xFFFF0000u : zw[f] << 16);
              const float yv = fmaf(skip, x, __uint_as_float(y[8 * e + 2 * f + g]));
              r[g] = yv * __fdividef(z, 1.f + ex2(-1.44269504088896340736f * z));
            }
            o[f] = pack_bf16(r[0], r[1]);
          }
          *(uint4*)(ztile + row * 128 + at) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      tc_fence_before();
      __syncwarp();
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int r = quad * 32 + q * 4 + (lane >> 3), at = lane & 7;
        const uint4 v = *(const uint4*)(ztile + r * 128 + ((at ^ (r & 7)) << 4));
        if (r < left) *(uint4*)(p.out + (first + (size_t)c * kQ + r) * p.out_stride + head * kSsmP + at * 8) = v;
      }
      mbar_arrive(bar(L::kEmpty + b));
    }
    // ---- the state after the last token
    wait(L::kS, (chunks - 1) & 1);
    tc_fence_after();
#pragma unroll
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
  } else if (warp == 8) {
    // ------------------------------------------------------------------ MMAs
    if (lane == 0) {
      auto wait = [&](int b, uint32_t parity) { return ok = wait_or_flag(bar(b), parity, p.sink, kErrTimeout); };
      constexpr uint32_t id_g = idesc_16(128, 128, false, false, false), id_y2 = idesc_16(128, 64, false, false, false),
                         id_y = idesc_16(128, 64, false, false, true), id_s = idesc_16(128, 128, false, false, true);
      for (int c = 0; c < chunks; ++c) {
        const uint32_t buf = sb + (c & 1) * L::kBuf, cm = buf + kBC, x = buf + 2 * kBC;
        const bool zero = c == 0 && !goes_on;
        if (!wait(L::kFull + (c & 1), (c >> 1) & 1)) break;
        tc_fence_after();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t o = (e / 4) * (kQ * 128) + (e % 4) * 32;
          mma_ss(tmem + kTG, sdesc_sw128(cm + o), sdesc_sw128(buf + o), id_g, e > 0);
        }
        tc_commit(bar(L::kG));
        if (!wait(L::kHFull, c & 1)) break;
        tc_fence_after();
        if (!zero) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              mma_ss(tmem + kTY + h * 64, sdesc_sw128(cm + (e / 4) * (kQ * 128) + (e % 4) * 32),
                     sdesc_sw128(sb + L::kH + h * kXT + (e / 4) * (64 * 128) + (e % 4) * 32), id_y2, e > 0);
        }
        tc_commit(bar(L::kY2));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!ok || !wait(L::kMFull + h, c & 1)) continue;
          tc_fence_after();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            mma_ts(tmem + kTY + h * 64, tmem + kTM + h * 64 + 8 * e, sdesc_mn_sw128(x + h * kXT + e * 2048, kQ * 128), id_y,
                   !zero || e > 0);
          tc_commit(bar(L::kYFull + h));
        }
        if (!ok || !wait(L::kWx, c & 1)) break;
        tc_fence_after();
#pragma unroll
        for (int e = 0; e < 16; ++e)  // the high parts, then the remainders
          mma_ts(tmem + kTState, tmem + kTG + 8 * e, sdesc_mn_sw128(buf + (e % 8) * 2048, kQ * 128), id_s, !zero || e > 0);
        tc_commit(bar(L::kS));
        tc_commit(bar(L::kEmpty + (c & 1)));
      }
      if (!ok) {  // give-up: wait (bounded) for the MMAs issued so far
        tc_commit(bar(L::kDone));
        for (int n = 0; n < (1 << 20) && !mbar_try_wait(bar(L::kDone), 0); ++n) {
        }
      }
    }
    __syncwarp();
  } else {
    const int tid = (int)threadIdx.x - 9 * 32;
    if (p.zx_stride % 8 == 0)
      state_copies<true>(p, sb, first, len, h0, tid, ok);
    else
      state_copies<false>(p, sb, first, len, h0, tid, ok);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
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
  p.sink = {h->ws.err, h->err_host_dev, h->timeout_ns};
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
  if (take(true)) {
    if (cudaFuncSetAttribute(k_prompt_state, cudaFuncAttributeMaxDynamicSharedMemorySize, StateSmem::kTotal) != cudaSuccess)
      return WAVE_ECUDA;
    k_prompt_state<<<p.b.n * (Hs / 2), kStateThreads, StateSmem::kTotal, st>>>(p);
  }
  if (take(false)) k_prompt_state_rows<<<dim3(Hs, p.b.n), 256, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? WAVE_OK : WAVE_ECUDA;
}
