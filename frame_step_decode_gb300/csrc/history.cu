// history.cu -- wave_history_append, wave_history_append_frame and
// wave_history_read: the 8-bit history with one scale for each block of tokens
// and head, written and read back.
//
//   block > 1:  scale = the least power of two s with |v| <= 448 s for all finite v of the block,
//               code = E4M3(v / s); when a block goes on and its scale grows, the codes that it
//               holds are encoded anew, which changes an exponent and loses nothing above the
//               codes' normal range
//   block = 1:  the step's rule, scale = amax / 448, code = E4M3(v / scale) by an IEEE division
//
// Bound by HBM.  Measured (captured launches in a row): append of 16 prompts,
// 8005 tokens, 32 query and 8 K/V heads of 128, qkv fp32, blocks of 64, 57 us =
// 4.9 TB/s; qkv bf16, blocks of 128, 54 us; 32 and 32 heads, blocks of 1, 103 us =
// 5.1 TB/s; a prompt of 25 tokens of 16 x 64 3.7 us, a frame of 80 sessions 3.4 us.
// Read back of 8005 tokens of 32 heads of 128 to bf16, blocks of 1, 35 us = 5.7
// TB/s.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/wave.h"
#include "history.h"
#include "quotient.cuh"

using namespace wave;

namespace wave {

struct HistoryAppendParams {
  SeqBatch b;
  int32_t first_block[WAVE_MAX_SEQS + 1];  // blocks of the sequences before sequence i
  const int32_t* positions;                // a frame's, on the device; null: the batch's
  History hist;
  wave_rope rope;                          // dims 0: no rotation
  int heads;                               // of q
  int per_cta;                             // head rows that a CTA works on
  int kv_ctas, q_team;                     // blocks: the CTAs of K and V; q's are behind them, in teams of so many threads
  long long stride;
  const void* qkv;
  void* q;                                 // [rows][heads][D], or null
  int *err, *err_out;
};

constexpr int kAppendThreads2 = 256;

// The turns of `tokens` positions from `pos` on, [token][4][dims / 16].
__device__ __forceinline__ void make_turns(const wave_rope& r, float4* turns, int quads, int tokens, int pos) {
  const int pairs = r.dims / 2, per = r.dims / 16;
  for (int i = threadIdx.x; i < tokens * pairs; i += blockDim.x) {
    const int t = i / pairs, k = i % pairs;
    ((float2*)(turns + t * quads))[(k % 8 / 2 * per + k / 8) * 2 + k % 2] = turn_at(r.turns[k], (uint32_t)(pos + t), r.amplitude);
  }
}

// Codes of tokens [from, to) of one head encoded anew under a scale that is
// 1 / ratio times the one they were made with.  NaN stays NaN, also where the
// ratio is 0 (a block whose values are not finite has the least scale).
template <int D>
__device__ __forceinline__ void recode(uint8_t* codes, int from, int to, float ratio, int lane, int lanes) {
  for (int i = from * (D / 8) + lane; i < to * (D / 8); i += lanes) {
    uint2* c = (uint2*)codes + i;
    float x[8];
    decode8(*c, x);
    *c = codes8(x, ratio);
  }
}

// Single tokens: blocks of 1, and frames.  D / 16 lanes to a head row of a token,
// sixteen values each, kFew rows of a lane's in flight together while the turns
// of the token's position are made.
template <int D, typename In, typename Out>
__global__ void __launch_bounds__(kAppendThreads2) k_append_tokens(const __grid_constant__ HistoryAppendParams p) {
  constexpr int kLanes = D / 16, kGroups = kAppendThreads2 / kLanes, kFew = 3;
  __shared__ float4 turns[D / 4];
  const int rows = p.heads + 2 * p.hist.heads, chunks = (rows + p.per_cta - 1) / p.per_cta;
  const int t = blockIdx.x / chunks, first = (blockIdx.x - t * chunks) * p.per_cta;
  int row, pos, slot;
  if (p.positions) {
    row = slot = t;
    pos = p.positions[t];
    if (pos < 0) return;
    if (pos >= p.hist.T_max) {
      if (threadIdx.x == 0) bad_position(p.err, p.err_out);
      return;
    }
  } else {
    const int s = seq_of(p.b, t), n = t - p.b.cum[s];
    row = p.b.begin[s] + n;
    pos = p.b.start[s] + n;
    slot = p.b.slot[s];
  }
  const int lane = threadIdx.x % kLanes, last = min(first + p.per_cta, rows);
  const uint32_t mates = ((1u << kLanes) - 1) << ((threadIdx.x & 31) / kLanes * kLanes);
  const bool half = p.rope.layout == WAVE_ROPE_HALF;
  int a, b;
  bool turned;
  groups_of_item(p.rope, lane, a, b, turned);
  const In* src = (const In*)p.qkv + (size_t)row * p.stride;
  for (int r0 = first + (int)threadIdx.x / kLanes, it = 0; it == 0 || r0 - (int)threadIdx.x / kLanes < last; r0 += kFew * kGroups, ++it) {
    Raw16<In> raw[kFew];
#pragma unroll
    for (int f = 0; f < kFew; ++f) {
      const int r = r0 + f * kGroups;
      if (r < last && (r >= p.heads || p.q)) raw[f].load(src + r * D, a, b);
    }
    if (it == 0) {
      make_turns(p.rope, turns, 0, 1, pos);
      __syncthreads();
    }
#pragma unroll
    for (int f = 0; f < kFew; ++f) {
      const int r = r0 + f * kGroups;
      if (r >= last || (r < p.heads && !p.q)) continue;
      const bool is_v = r >= p.heads + p.hist.heads;
      float x[16];
      raw[f].get(x);
      if (turned && !is_v) turn_item(x, &turns[lane], p.rope.dims / 16, half);
      if (r < p.heads) {
        Out* dst = (Out*)p.q + ((size_t)row * p.heads + r) * D;
        store8<Out>(dst + 8 * a, x);
        store8<Out>(dst + 8 * b, x + 8);
        continue;
      }
      const size_t hr = p.hist.row(is_v, slot, r - p.heads - (is_v ? p.hist.heads : 0));
      uint8_t* codes = p.hist.codes + hr * p.hist.T_max * D;
      float* scales = p.hist.scales + hr * p.hist.blocks;
      float amax = 0.f;
      uint2 c0, c1;
      if (p.hist.block == 1) {
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
        for (int d = kLanes / 2; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(mates, amax, d));
        const float sc = __fdiv_rn(amax, 448.0f);
        c0 = make_uint2(encode4(x, sc), encode4(x + 4, sc));
        c1 = make_uint2(encode4(x + 8, sc), encode4(x + 12, sc));
        if (lane == 0) scales[pos] = sc;
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = fmaxf(amax, counts(x[i]));
#pragma unroll
        for (int d = kLanes / 2; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(mates, amax, d));
        const int blk = pos >> p.hist.shift, from = blk << p.hist.shift;
        float sc = block_scale(amax);
        if (from < pos) {
          const float old = scales[blk];
          __syncwarp(mates);  // read before lane 0 writes it
          if (sc > old)
            recode<D>(codes, from, pos, old / sc, lane, kLanes);
          else
            sc = old;
        }
        const float inv = sc == 0.f ? 0.f : __frcp_rn(sc);
        c0 = encode8(x, inv), c1 = encode8(x + 8, inv);
        if (lane == 0) scales[blk] = sc;
      }
      uint8_t* dst = codes + (size_t)pos * D;
      *(uint2*)(dst + 8 * a) = c0;
      *(uint2*)(dst + 8 * b) = c1;
    }
  }
}

// Blocks of 16 to 128 tokens of prompts.  For K and V a CTA takes the tokens that
// the call has of one block, and some of the heads: one pass over them, values
// kept in registers between the block's largest magnitude and the codes, the
// next head's on their way meanwhile.  For q, which has no blocks, a team of
// threads takes four tokens with all heads.  So the turns of a position are made for few
// CTAs (into shared memory), and none for V.  kLog: the block is 1 << kLog tokens.
template <int D, int kLog>
struct BlockShape {
  static constexpr int kLanes = D / 16, kItems = (1 << kLog) * kLanes;  // of a head row
  static constexpr int kThreads = kItems > 512 ? 512 : 256;
  static constexpr int kPer = kItems > kThreads ? kItems / kThreads : 1;  // items of a thread
  static constexpr int kGroup = kItems / kPer;                           // threads to a head row
  static constexpr int kGroups = kThreads / kGroup;                      // head rows at a time
};
template <int D, int kLog, typename In, typename Out>
__global__ void __launch_bounds__((BlockShape<D, kLog>::kThreads)) k_append_blocks(const __grid_constant__ HistoryAppendParams p) {
  using B = BlockShape<D, kLog>;
  constexpr int kLanes = B::kLanes, kPer = B::kPer, kGroup = B::kGroup, kGroups = B::kGroups;
  extern __shared__ float4 turns[];  // [token][D / 4]
  __shared__ float most[2][B::kThreads / 32];
  const bool half = p.rope.layout == WAVE_ROPE_HALF;
  if ((int)blockIdx.x >= p.kv_ctas) {  // q
    constexpr int kTokens = 4;
    const int team = p.q_team, sub = threadIdx.x / team, tid = threadIdx.x % team, total = p.b.cum[p.b.n];
    const int first = (((int)blockIdx.x - p.kv_ctas) * (B::kThreads / team) + sub) * kTokens;
    float4* mine = turns + sub * kTokens * (D / 4);
    size_t row[kTokens];
    int pos[kTokens];
#pragma unroll
    for (int r = 0; r < kTokens; ++r) {
      const int t = min(first + r, total - 1), s = seq_of(p.b, t), n = t - p.b.cum[s];
      row[r] = p.b.begin[s] + n;
      pos[r] = p.b.start[s] + n;
    }
    const int items = p.heads * kLanes;
    for (int i = tid; i < (items + team - 1) / team * team; i += team) {
      const int r0 = i / kLanes;
      int a, b;
      bool turned;
      groups_of_item(p.rope, i % kLanes, a, b, turned);
      Raw16<In> raw[kTokens];
#pragma unroll
      for (int r = 0; r < kTokens; ++r)
        if (i < items && first + r < total) raw[r].load((const In*)p.qkv + row[r] * p.stride + r0 * D, a, b);
      if (i < team) {  // once
        const int pairs = p.rope.dims / 2, per = p.rope.dims / 16;
        for (int k = tid; k < kTokens * pairs; k += team) {
          const int r = k / pairs, j = k - r * pairs, t = r == 0 ? pos[0] : r == 1 ? pos[1] : r == 2 ? pos[2] : pos[3];
          ((float2*)(mine + r * (D / 4)))[(j % 8 / 2 * per + j / 8) * 2 + j % 2] = turn_at(p.rope.turns[j], (uint32_t)t, p.rope.amplitude);
        }
        __syncthreads();
      }
#pragma unroll
      for (int r = 0; r < kTokens; ++r) {
        if (i >= items || first + r >= total) continue;
        float x[16];
        raw[r].get(x);
        if (turned) turn_item(x, mine + r * (D / 4) + i % kLanes, p.rope.dims / 16, half);
        Out* dst = (Out*)p.q + (row[r] * p.heads + r0) * D;
        store8<Out>(dst + 8 * a, x);
        store8<Out>(dst + 8 * b, x + 8);
      }
    }
    return;
  }
  // K and V: (block, K or V, some heads)
  const int chunks = (p.hist.heads + p.per_cta - 1) / p.per_cta, unit = blockIdx.x / (2 * chunks);
  const int which = ((int)blockIdx.x - unit * 2 * chunks) / chunks, first = (blockIdx.x % chunks) * p.per_cta;
  const int last = min(first + p.per_cta, p.hist.heads);
  int lo = 0, hi = p.b.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.first_block[mid] <= unit)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int start = p.b.start[lo], end = start + p.b.len(lo), slot = p.b.slot[lo];
  const int blk = (start >> kLog) + unit - p.first_block[lo];
  const int from = max(start, blk << kLog), to = min(end, (blk + 1) << kLog);  // the call's tokens of the block
  const int held = from - (blk << kLog);                                      // what the block holds before them
  const int g = threadIdx.x / kGroup, in = threadIdx.x % kGroup, lane = in % kLanes, t0 = in / kLanes;
  constexpr int kStep = kGroup / kLanes;  // tokens between a thread's items
  int a, b;
  bool turned;
  groups_of_item(p.rope, lane, a, b, turned);
  turned = turned && !which;
  const size_t row0 = p.b.begin[lo] + (from - start);
  Raw16<In> raw[kPer];
  auto load = [&](int r) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int t = t0 + i * kStep;
      if (r < last && from + t < to)
        raw[i].load((const In*)p.qkv + (row0 + t) * p.stride + (p.heads + which * p.hist.heads + r) * D, a, b);
      else
        raw[i].clear();
    }
  };
  load(first + g);
  if (!which) {
    make_turns(p.rope, turns, D / 4, to - from, from);
    __syncthreads();
  }
  for (int it = 0, r0 = first; r0 < last; ++it, r0 += kGroups) {
    const int r = r0 + g;
    float x[kPer][16];
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) raw[i].get(x[i]);
    load(r + kGroups);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int t = t0 + i * kStep;
      if (turned && from + t < to) turn_item(x[i], turns + t * (D / 4) + lane, p.rope.dims / 16, half);
#pragma unroll
      for (int e = 0; e < 16; ++e) amax = fmaxf(amax, counts(x[i][e]));  // 0 where there is no token
    }
    const bool on = r < last;
    const size_t hr = p.hist.row(which, slot, on ? r : first);
    uint8_t* codes = p.hist.codes + hr * p.hist.T_max * D;
    float* scales = p.hist.scales + hr * p.hist.blocks;
    const float old = on && held ? scales[blk] : 0.f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
    if (threadIdx.x % 32 == 0) most[it & 1][threadIdx.x / 32] = amax;
    __syncthreads();  // most[it & 1] is written again after the next one, which comes after it has been read
    if (!on) continue;
#pragma unroll
    for (int w = 0; w < kGroup / 32; ++w) amax = fmaxf(amax, most[it & 1][g * (kGroup / 32) + w]);
    float sc = block_scale(amax);
    if (held) {
      if (sc > old)
        recode<D>(codes, blk << kLog, from, old / sc, in, kGroup);
      else
        sc = old;
    }
    const float inv = sc == 0.f ? 0.f : __frcp_rn(sc);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int t = t0 + i * kStep;
      if (from + t >= to) continue;
      uint8_t* dst = codes + (size_t)(from + t) * D;
      *(uint2*)(dst + 8 * a) = encode8(x[i], inv);
      *(uint2*)(dst + 8 * b) = encode8(x[i] + 8, inv);
    }
    if (in == 0) scales[blk] = sc;
  }
}

template <int D, int kLog, typename In, typename Out>
static cudaError_t launch_blocks(HistoryAppendParams& p, int sms, cudaStream_t st) {
  using B = BlockShape<D, kLog>;
  constexpr int kSmem = (1 << kLog) * D * 4;
  static_assert(kSmem <= 64 * 1024, "the turns of a block");
  if (kSmem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(k_append_blocks<D, kLog, In, Out>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
  }
  // Heads of a CTA: up to eight rounds of them, fewer where that leaves SMs
  // without work (a CTA of 512 threads has an SM to itself).
  const int units = p.first_block[p.b.n];
  const long long share = 2LL * units * p.hist.heads / ((B::kThreads > 256 ? 2LL : 4LL) * sms * B::kGroups);
  p.per_cta = B::kGroups * (int)std::max(1LL, std::min(8LL, share));
  const int chunks = (p.hist.heads + p.per_cta - 1) / p.per_cta;
  p.kv_ctas = units * 2 * chunks;
  p.q_team = 256;
  while (p.q_team > 64 && p.heads * B::kLanes <= p.q_team / 2) p.q_team /= 2;
  const int tokens = 4 * (B::kThreads / p.q_team), q_ctas = p.q ? (p.b.cum[p.b.n] + tokens - 1) / tokens : 0;
  static_assert(4 * B::kThreads / 64 * D * 4 <= kSmem, "q's turns");
  k_append_blocks<D, kLog, In, Out><<<(unsigned)(p.kv_ctas + q_ctas), B::kThreads, kSmem, st>>>(p);
  return cudaGetLastError();
}

template <int D, typename In, typename Out>
static cudaError_t launch_history_append(HistoryAppendParams& p, int tokens, int sms, cudaStream_t st) {
  if (p.positions || p.hist.block == 1) {
    const int rows = p.heads + 2 * p.hist.heads;
    // head rows of a CTA: all of them, or one for each group of lanes where tokens are few
    constexpr int kGroups = kAppendThreads2 / (D / 16);
    p.per_cta = tokens >= 8 * sms ? rows : kGroups;
    const int chunks = (rows + p.per_cta - 1) / p.per_cta;
    k_append_tokens<D, In, Out><<<(unsigned)((long long)tokens * chunks), kAppendThreads2, 0, st>>>(p);
    return cudaGetLastError();
  }
  p.first_block[0] = 0;
  for (int i = 0; i < p.b.n; ++i)
    p.first_block[i + 1] =
        p.first_block[i] + ((p.b.start[i] + p.b.len(i) - 1) >> p.hist.shift) - (p.b.start[i] >> p.hist.shift) + 1;
  switch (p.hist.shift) {
    case 4: return launch_blocks<D, 4, In, Out>(p, sms, st);
    case 5: return launch_blocks<D, 5, In, Out>(p, sms, st);
    case 6: return launch_blocks<D, 6, In, Out>(p, sms, st);
    default: return launch_blocks<D, 7, In, Out>(p, sms, st);
  }
}

template <int D>
static cudaError_t launch_history_append_types(HistoryAppendParams& p, int in, int out, int tokens, int sms, cudaStream_t st) {
  if (in == WAVE_F32)
    return out == WAVE_BF16 ? launch_history_append<D, float, __nv_bfloat16>(p, tokens, sms, st)
                            : launch_history_append<D, float, __half>(p, tokens, sms, st);
  return out == WAVE_BF16 ? launch_history_append<D, __nv_bfloat16, __nv_bfloat16>(p, tokens, sms, st)
                          : launch_history_append<D, __nv_bfloat16, __half>(p, tokens, sms, st);
}

static int append(wave_t* h, HistoryAppendParams& p, int tokens, const wave_rope* rope, const void* qkv, int qkv_type,
                  int64_t row_stride, void* q, int q_type, void* stream) {
  const int H = h->pl.cfg.n_heads, D = h->pl.cfg.head_dim;
  if (!qkv || (rope && !rope_ok(rope, D)) || (qkv_type != WAVE_F32 && qkv_type != WAVE_BF16) ||
      (q_type != WAVE_BF16 && q_type != WAVE_F16) || row_stride < (int64_t)(H + 2 * p.hist.heads) * D || row_stride % 8 ||
      row_stride > kMaxStride || !aligned16(qkv) || !aligned16(q))
    return WAVE_EINVAL;
  if (!on_device(h)) return WAVE_EINVAL;
  if (tokens == 0) return WAVE_OK;
  if (rope)
    p.rope = *rope;
  else
    p.rope = wave_rope{};
  p.heads = H;
  p.stride = row_stride;
  p.qkv = qkv;
  p.q = q;
  p.err = h->ws.err;
  p.err_out = h->err_host_dev;
  cudaStream_t st = (cudaStream_t)stream;
  h->last_stream = st;
  const cudaError_t e = D == 128 ? launch_history_append_types<128>(p, qkv_type, q_type, tokens, h->pl.grid, st)
                                 : launch_history_append_types<64>(p, qkv_type, q_type, tokens, h->pl.grid, st);
  return e == cudaSuccess ? WAVE_OK : WAVE_ECUDA;
}

struct HistoryReadParams {
  SeqBatch b;
  History hist;
  long long items;
  void *k, *v;
};

// Codes times their scale, rounded once.  Sixteen values of a row a thread.
template <int D, typename Out>
__global__ void __launch_bounds__(256) k_history_read(const __grid_constant__ HistoryReadParams p) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= p.items) return;
  constexpr int kLanes = D / 16;
  const int lane = (int)(i % kLanes), head = (int)(i / kLanes % p.hist.heads);
  const long long j = i / kLanes / p.hist.heads;
  const int t = (int)(j >> 1), which = (int)(j & 1);
  Out* out = (Out*)(which ? p.v : p.k);
  if (!out) return;
  const int s = seq_of(p.b, t), n = t - p.b.cum[s], pos = p.b.start[s] + n;
  const size_t hr = p.hist.row(which, p.b.slot[s], head);
  const uint4 c = *(const uint4*)(p.hist.codes + (hr * p.hist.T_max + pos) * D + 16 * lane);
  const float sc = p.hist.scales[hr * p.hist.blocks + (pos >> p.hist.shift)];
  float x[16];
  decode8(make_uint2(c.x, c.y), x);
  decode8(make_uint2(c.z, c.w), x + 8);
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] *= sc;
  Out* dst = out + ((size_t)(p.b.begin[s] + n) * p.hist.heads + head) * D + 16 * lane;
  store8<Out>(dst, x);
  store8<Out>(dst + 8, x + 8);
}

template <int D>
static void launch_read(const HistoryReadParams& p, int type, cudaStream_t st) {
  const unsigned ctas = (unsigned)((p.items + 255) / 256);
  if (type == WAVE_F32)
    k_history_read<D, float><<<ctas, 256, 0, st>>>(p);
  else if (type == WAVE_BF16)
    k_history_read<D, __nv_bfloat16><<<ctas, 256, 0, st>>>(p);
  else
    k_history_read<D, __half><<<ctas, 256, 0, st>>>(p);
}

}  // namespace wave

extern "C" int wave_history_append(wave_t* h, int layer, int n_seq, const int32_t* cu_seqlens, const int32_t* slots,
                                   const int32_t* starts, const wave_rope* rope, const void* qkv, int qkv_type,
                                   int64_t row_stride, uint8_t* kv_fp8, float* kv_scales, int n_kv_heads, int block, void* q,
                                   int q_type, void* stream) {
  HistoryAppendParams p;
  int rc = make_history(&p.hist, h, layer, n_kv_heads, block, kv_fp8, kv_scales);
  if (!rc) rc = make_batch(&p.b, n_seq, cu_seqlens, slots, starts, h->pl.S_max);
  if (rc) return rc;
  for (int i = 0; i < p.b.n; ++i)
    if (p.b.start[i] > h->pl.T_max - p.b.len(i)) return WAVE_EPOS;
  p.positions = nullptr;
  return append(h, p, p.b.cum[p.b.n], rope, qkv, qkv_type, row_stride, q, q_type, stream);
}

extern "C" int wave_history_append_frame(wave_t* h, int layer, int S, const int32_t* positions, const wave_rope* rope,
                                         const void* qkv, int qkv_type, int64_t row_stride, uint8_t* kv_fp8,
                                         float* kv_scales, int n_kv_heads, int block, void* q, int q_type, void* stream) {
  HistoryAppendParams p;
  const int rc = make_history(&p.hist, h, layer, n_kv_heads, block, kv_fp8, kv_scales);
  if (rc) return rc;
  if (S < 1 || S > h->pl.S_max || !positions || ((uintptr_t)positions & 3)) return WAVE_EINVAL;
  p.b.n = 0;
  p.b.cum[0] = 0;
  p.positions = positions;
  return append(h, p, S, rope, qkv, qkv_type, row_stride, q, q_type, stream);
}

extern "C" int wave_history_read(wave_t* h, int layer, int n_seq, const int32_t* cu_seqlens, const int32_t* slots,
                                 const int32_t* starts, const uint8_t* kv_fp8, const float* kv_scales, int n_kv_heads,
                                 int block, void* k, void* v, int out_type, void* stream) {
  HistoryReadParams p;
  int rc = make_history(&p.hist, h, layer, n_kv_heads, block, kv_fp8, kv_scales);
  if (!rc) rc = make_batch(&p.b, n_seq, cu_seqlens, slots, starts, h->pl.S_max);
  if (rc) return rc;
  if ((!k && !v) || !aligned16(k) || !aligned16(v) || (out_type != WAVE_F32 && out_type != WAVE_BF16 && out_type != WAVE_F16))
    return WAVE_EINVAL;
  for (int i = 0; i < p.b.n; ++i)
    if (p.b.start[i] > h->pl.T_max - p.b.len(i)) return WAVE_EPOS;
  if (!on_device(h)) return WAVE_EINVAL;
  if (p.b.n == 0) return WAVE_OK;
  const int D = h->pl.cfg.head_dim;
  p.items = (long long)p.b.cum[p.b.n] * 2 * n_kv_heads * (D / 16);
  if (p.items > 0x7fffffffLL * 256) return WAVE_EINVAL;
  p.k = k;
  p.v = v;
  cudaStream_t st = (cudaStream_t)stream;
  h->last_stream = st;
  if (D == 128)
    launch_read<128>(p, out_type, st);
  else
    launch_read<64>(p, out_type, st);
  return cudaGetLastError() == cudaSuccess ? WAVE_OK : WAVE_ECUDA;
}
