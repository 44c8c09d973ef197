// history_many.cu -- attention over the 8-bit history for prompts that go on:
// more rows than kFewRows for a K/V head.
//
// Bound by the tensor cores (4 D flops for a query head, a query and a key).
// Rows are (token, head of the group), so that the heads of a K/V head share its
// tiles; a pair of 128-row tiles is a unit, its two tiles are two streams, and
// while one stream's weights are computed the tensor core works for the other.
// S = Q K^T by tcgen05 into TMEM, a thread per row turns S into the weights P
// (fp16, written over S), O += P V by tcgen05 with P read from TMEM.
//
// Four warps bring the codes to fp16 operand tiles, an exact conversion: 16
// codes a load, held in registers a block ahead.  The K scale of a block of 128
// is a factor of the scores and the V scale an offset of the weights'
// exponents, so that neither costs anything an element; in tiles with several
// scales codes are brought to the largest of them in fp16 (exact for powers of
// two), and with a scale for each token the softmax's threads multiply the
// columns of S and of P in fp32; scales that lie far apart go another way (kApart).
//
// All units' key blocks are one line, cut evenly among the SMs: a unit's blocks
// in several CTAs leave fp32 sums, which a second launch joins.
//
// Measured (captured launches in a row): 1024 tokens after 7168, 32 heads of 128,
// fp16, blocks of 128, 113 us = 1.14 PFLOP/s (the join 14 us when profiled alone);
// 2001 after 4096 with 300, 17 and 1 others, 32/8 heads, bf16, blocks of 32, 177 us =
// 0.99 PFLOP/s; 2048 after 6144, 32 heads, a scale for each token, 288 us = 0.83
// PFLOP/s, 16 heads of 64, blocks of 64, 86 us; 8192 tokens from the first, 437 to
// 447 us.  A block of 128 keys and both streams takes about 3500 cycles, 2048 of
// them the tensor core's (its pipe is active 55% of the time): the MMAs wait for
// the chain from S to P, and the conversion shares the shared memory with them.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "history_attn.h"

using namespace wave;

namespace wave {

constexpr int kManyRows = 128;      // rows of a stream, and keys of a block
constexpr int kManyThreads = 512;   // 8 softmax warps (two streams), 4 that convert, MMAs, scheduler, prefetch, one idle
constexpr int kMaxCuts = 160;       // CTAs
constexpr int kRegsRows = 144, kRegsCodes = 128, kRegsMma = 96;
constexpr float kManyBias = 7.f;    // weights are held times 2^7, see below
enum { kScaleOfTile, kScaleOfBlock, kScaleOfToken };  // blocks of 128, of 16 to 64, of 1

// Where a CTA's part of the line begins: key block `block` of a unit.
struct ManyCut {
  int32_t seq, level, head, block;
};

struct ManyParams {
  HistoryAttnParams a;  // a.b: the sequences
  int tile_tokens;      // tokens of a 128-row tile: 128 / group
  int ctas;
  ManyCut cut[kMaxCuts + 1];
  float* part_o;        // [2 * CTA + (the unit begins there)][256 rows][D], in the values' own units over 2^kPartBias
  float2* part_ml;      // the sums of their weights (second) and the power of two that both are relative to
  int wide;             // out's rows are 32-byte aligned
  ErrSink sink;
  int skip;             // testing hook: no tile of K and V from this one on is made (-1: off)
};

// A unit's blocks [from, to) in this CTA.
struct ManyItem {
  int seq, level, head;
  int tok0, len;       // first token of stream 0, of the sequence's
  int n[2];            // key blocks of the streams, from the sequence's begin (0: no rows)
  int from, to;
  int valid;
  int start, row0;     // position of the sequence's first token, and its row
  __host__ __device__ int blocks() const { return n[0] > n[1] ? n[0] : n[1]; }
  __host__ __device__ bool whole() const { return from == 0 && to == blocks(); }
  __host__ __device__ int here(int st) const { return (n[st] < to ? n[st] : to) - from; }  // a stream's blocks in this CTA (or none)
};

__host__ __device__ inline void unit_blocks(const SeqBatch& b, int tile_tokens, ManyItem& it) {
  it.tok0 = it.level * 2 * tile_tokens;
  it.len = b.len(it.seq);
  it.start = b.start[it.seq];
  it.row0 = b.begin[it.seq];
  for (int st = 0; st < 2; ++st) {
    const int first = it.tok0 + st * tile_tokens, last = first + tile_tokens < it.len ? first + tile_tokens : it.len;
    it.n[st] = first < it.len ? (b.start[it.seq] + last - 1) / kManyRows + 1 : 0;
  }
}

// A CTA's walk along its part of the line.
struct ManyWalk {
  ManyItem it;
  __device__ __forceinline__ bool begin(const ManyParams& p) {
    const ManyCut& c = p.cut[blockIdx.x];
    it.seq = c.seq, it.level = c.level, it.head = c.head, it.from = c.block;
    return set(p);
  }
  __device__ __forceinline__ bool next(const ManyParams& p) {
    if (it.to < it.blocks()) return false;  // the rest is another CTA's
    it.from = 0;
    if (++it.head == p.a.hist.heads) {
      it.head = 0;
      if ((++it.level) * 2 * p.tile_tokens >= it.len) it.level = 0, ++it.seq;
    }
    return set(p);
  }
  __device__ __forceinline__ bool set(const ManyParams& p) {
    const ManyCut& e = p.cut[blockIdx.x + 1];
    const bool last = it.seq == e.seq && it.level == e.level && it.head == e.head;
    if (it.seq >= p.a.b.n || (last && it.from >= e.block)) return false;
    unit_blocks(p.a.b, p.tile_tokens, it);
    it.to = last ? e.block : it.blocks();
    return true;
  }
};

struct BlockMeta {
  float factor;       // of the scores: the tile's largest K scale, over 2^6
  float shift;        // of the weights' exponents: log2 of the largest V scale
  int apart;          // the codes are as they are in the tiles, and the scales are
  float pad;
  float k[kManyRows], v[kManyRows];  // scales for each token: K's, and V's over 2^shift (apart: log2 of V's); k alone for blocks: 8 of K, 8 of V
};

// A tile of 128 slots whose scales lie far apart is not brought to the largest
// of them, for which fp16 would cut the others' codes or weights: its codes stay
// as they are, its scales meet the scores and the weights token by token in fp32,
// relative to what a row sees.  Two passes over the scores and two exponentials
// each: a call of such tiles alone takes 268 us instead of 124 (1024 tokens after
// 7168, 32 heads of 128, blocks of 64).  How far, in powers of two of the largest
// scale over the least that is not 0: 8, which leaves codes their bits and weights
// theirs; of V's, where some row does not see all of the tile, 4, which is what a
// scale that it does not see may cost it; and there none 64 above the tiles
// before, whose sums it would leave nothing in fp32.
constexpr int kApart = 8, kApartCut = 4, kApartRise = 64;

template <int D>
struct ManySmem {
  static constexpr int kTile = kManyRows * D * 2;
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kMetas = 4;
  static constexpr int kRing = 2 * kTile;
  static constexpr int kMeta = kRing + kStages * kTile;
  static constexpr int kBad = kMeta + kMetas * (int)sizeof(BlockMeta);  // [2 units][converting warp][D]: the first token whose value is NaN
  static constexpr int kItems = kBad + 2 * 4 * D * 4;
  static constexpr int kBars = kItems + (2 * (int)sizeof(ManyItem) + 15) / 16 * 16;
  enum {
    kFull = 0,
    kEmpty = kFull + kStages,
    kMetaFull = kEmpty + kStages,
    kMetaEmpty = kMetaFull + kMetas,
    kQFull = kMetaEmpty + kMetas,
    kSFull = kQFull + 2,
    kPFull = kSFull + 2,
    kOFull = kPFull + 2,
    kItemFull = kOFull + 2,
    kItemEmpty = kItemFull + 2,
    kDone = kItemEmpty + 2,
    kCount
  };
  static constexpr int kMisc = (kBars + kCount * 8 + 15) / 16 * 16;
  static constexpr int kTotal = kMisc + 48 + 1024;  // + alignment
};
static_assert(ManySmem<128>::kTotal <= 232448 && ManySmem<64>::kTotal <= 232448, "shared memory of a CTA");

__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The exponent of the least power of two at or above x > 0.
__device__ __forceinline__ int exponent_up(float x) {
  const uint32_t u = __float_as_uint(x);
  return (int)(u >> 23) - 127 + ((u & 0x7FFFFFu) != 0);
}
__device__ __forceinline__ float power(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

template <int D, bool kF16, int kScale>
__global__ void __launch_bounds__(kManyThreads, 1) k_history_many(const __grid_constant__ ManyParams p) {
  using L = ManySmem<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base_raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024 - (base_raw & 1023)) & 1023);
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) { return sb + L::kBars + i * 8; };
  BlockMeta* metas = (BlockMeta*)(smem + L::kMeta);
  int* bad = (int*)(smem + L::kBad);
  const ManyItem* items = (const ManyItem*)(smem + L::kItems);
  uint32_t* tmem_word = (uint32_t*)(smem + L::kMisc);
  int* leave = (int*)(smem + L::kMisc + 8);
  int* odd_unit = (int*)(smem + L::kMisc + 16);  // [2 units][converting warp]: it has found NaN values

  if (warp == 12) {
    if (lane == 0) {
      for (int i = 0; i < L::kStages; ++i) {
        mbar_init(bar(L::kFull + i), 4);
        mbar_init(bar(L::kEmpty + i), 1);
      }
      for (int i = 0; i < L::kMetas; ++i) {
        mbar_init(bar(L::kMetaFull + i), 4);
        mbar_init(bar(L::kMetaEmpty + i), 8);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(bar(L::kQFull + i), 4);
        mbar_init(bar(L::kSFull + i), 1);
        mbar_init(bar(L::kPFull + i), 4);
        mbar_init(bar(L::kOFull + i), 1);
        mbar_init(bar(L::kItemFull + i), 1);
        mbar_init(bar(L::kItemEmpty + i), 14);  // softmax, conversion, MMAs, prefetch
      }
      mbar_init(bar(L::kDone), 1);
      fence_mbar_init();
      fence_proxy_async_smem();
      *leave = stopped(p.sink);
    }
    __syncwarp();
    tmem_alloc(smem_u32(tmem_word), 512);
    tmem_relinquish();
  }
  for (int i = threadIdx.x; i < 8 * D; i += kManyThreads) bad[i] = INT32_MAX;
  if (threadIdx.x < 8) odd_unit[threadIdx.x] = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_word;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the launch that joins parts
  const bool stop = *leave;
  auto tS = [&](int st) { return tmem + st * 128; };
  auto tO = [&](int st) { return tmem + 256 + st * D; };

  // Every wait is bounded; a give-up sets the error word and ends the role's
  // loop, which lets the waits of the others run out too; CTAs that begin
  // later leave at once.
  bool ok = true;
  auto wait_warp = [&](int b, uint32_t parity) {
    return ok = __all_sync(0xffffffffu, wait_bar(bar(b), parity, p.sink));
  };
  if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    regs_take<kRegsRows>();
    const int st = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int row_tok = row / p.a.group, row_head = row % p.a.group;  // of a tile and of a group
    uint32_t s_it = 0, o_it = 0, m_it = 0;
    // The row's q into the stream's operand tile (128-byte swizzle): fp16, bf16
    // times a power of two; the factor that its scores get in return.
    auto bring_q = [&](const ManyItem& it) {
      const int tok = it.tok0 + st * p.tile_tokens + row_tok;
      const bool on = row_tok < p.tile_tokens && tok < it.len;
      const uint16_t* src = p.a.q + (it.row0 + (on ? tok : 0)) * p.a.q_stride + (it.head * p.a.group + row_head) * D;
      uint4 v[D / 8];
#pragma unroll
      for (int i = 0; i < D / 8; ++i) v[i] = on ? __ldg((const uint4*)src + i) : make_uint4(0, 0, 0, 0);
      float factor = p.a.scale2, up = 1.f;
      if constexpr (!kF16) {
        uint32_t top = 0;  // the largest magnitude: bf16 bits compare as integers
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu), __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu)));
        top = max(top & 0xFFFFu, top >> 16);
        const int ex = min(max((int)(top >> 7) - 127, -113), 127);
        up = power(14 - ex);
        factor = p.a.scale2 * (power(ex) * 0x1p-14f);
      }
      uint8_t* dst = smem + st * L::kTile + row * 128;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        if constexpr (!kF16) {
#pragma unroll
          for (int c = 0; c < 4; ++c) w[c] = half2_of(__uint_as_float(w[c] << 16) * up, __uint_as_float(w[c] & 0xFFFF0000u) * up);
        }
        *(uint4*)(dst + (i / 8) * (kManyRows * 128) + (((i % 8) ^ (row & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::kQFull + st));
      return factor;
    };
    float factor = 0.f;
    if (wait_warp(L::kItemFull, 0) && items[0].valid && items[0].here(st) > 0) factor = bring_q(items[0]);
    for (uint32_t k = 0; ok && items[k & 1].valid; ++k) {
      const ManyItem& it = items[k & 1];
      const int n = it.here(st), all = it.to - it.from;  // this stream's blocks, and the unit's
      const int tile_tok = it.tok0 + st * p.tile_tokens;
      // what the row sees of the first block, and the first block that some row of the tile does not see all of
      int seen = it.start + tile_tok + row_tok - it.from * kManyRows;
      const int cut = (it.start + tile_tok) / kManyRows - it.from;
      // what the weights of O are relative to; the sum of the weights without V's
      // scales, and what it is relative to
      float m = -INFINITY, l = 0.f, base = 0.f;
#pragma unroll 1
      for (int j = 0; j < all; ++j, ++m_it, seen -= kManyRows) {
        const int mi = m_it % L::kMetas;
        if (!wait_warp(L::kMetaFull + mi, (m_it / L::kMetas) & 1)) break;
        if (j >= n) {  // the other stream's
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::kMetaEmpty + mi));
          continue;
        }
        const BlockMeta& meta = metas[mi];
        const float z = fmaxf(factor * meta.factor, 0x1p-126f), shift = meta.shift;
        const bool apart = kScale != kScaleOfTile && meta.apart, special = j >= cut || apart;
        if (!wait_warp(L::kSFull + st, s_it & 1)) break;
        ++s_it;
        tc_fence_after();
        // 32 columns, scaled and masked; and their largest
        auto ready = [&](int c, uint32_t* s, auto masked) {
          if constexpr (kScale == kScaleOfToken) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 f = ((const float4*)meta.k)[8 * c + i];
              s[4 * i] = __float_as_uint(__uint_as_float(s[4 * i]) * f.x);
              s[4 * i + 1] = __float_as_uint(__uint_as_float(s[4 * i + 1]) * f.y);
              s[4 * i + 2] = __float_as_uint(__uint_as_float(s[4 * i + 2]) * f.z);
              s[4 * i + 3] = __float_as_uint(__uint_as_float(s[4 * i + 3]) * f.w);
            }
          }
          if constexpr (masked.value) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * c + i > seen) s[i] = __float_as_uint(-INFINITY);
          }
        };
        constexpr std::true_type kMasked;
        constexpr std::false_type kAll;
        auto largest = [&](auto masked) {
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t s[32];
            tmem_ld32(tS(st) + lanes + 32 * c, s);
            tmem_ld_wait();
            ready(c, s, masked);
#pragma unroll
            for (int i = 0; i < 32; i += 8)
#pragma unroll
              for (int x = 0; x < 4; ++x) mx[x] = max3(mx[x], __uint_as_float(s[i + 2 * x]), __uint_as_float(s[i + 2 * x + 1]));
          }
          return fmaf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), z, shift);
        };
        // The weights' exponents are those of w times the tile's V scale.  What
        // they are relative to moves only when the weights of a row's block add
        // up to more than fp16 holds, so that O is rescaled seldom and weights
        // are made of S as it is read, with the maximum of the blocks before;
        // where that was too low they are made again.  The largest is then
        // between 2^7 and 2^16 and fp16 goes down to 2^-25, so that one 2^-32 of
        // it is still there.  (One fp32 product at a time: with packed ones the
        // loop takes 1290 cycles instead of 740 for a warp alone.)
        auto raise = [&](float top, bool up) {  // the maximum moves
          const float a = up ? (m == -INFINITY ? 0.f : ex2(m - top)) : 1.f;
          m = up ? top : m;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO(st) + lanes + 32 * c, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
            tmem_st32(tO(st) + lanes + 32 * c, o);
          }
        };
        float2 sum[4];
        auto weights = [&](int c, uint32_t* x, uint32_t* w, float neg, auto masked) {  // of 32 columns
          ready(c, x, masked);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float2 e = make_float2(ex2(fmaf(__uint_as_float(x[2 * i]), z, neg)), ex2(fmaf(__uint_as_float(x[2 * i + 1]), z, neg)));
            sum[i & 3] = add2(sum[i & 3], e);
            if constexpr (kScale == kScaleOfToken) {
              const float2 v = ((const float2*)meta.v)[16 * c + i];
              e = make_float2(e.x * v.x, e.y * v.y);
            }
            w[i] = half2_of(e.x, e.y);
          }
        };
        auto relative = [&]() { return (m == -INFINITY ? 0.f : shift - m) + kManyBias; };
        auto clear = [&]() { sum[0] = sum[1] = sum[2] = sum[3] = make_float2(0.f, 0.f); };
        auto add_up = [&]() {
          sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
          sum[0].x += sum[0].y;
        };
        // The sum of the weights has a reference of its own: every key counts in
        // it, also where V's scale is so far below another tile's that the
        // weights of O are nothing.  Without V's scales this tile's weights are
        // relative to -neg.  Where that is far above what the sum is relative to
        // they may all have been cut to 0, and the tile is added apart; where it
        // is because the maximum has just moved to a score of this tile they are
        // not, and the sum moves along.
        bool added = false;
        auto is_far = [&]() { return -relative() - base > 64.f; };
        auto add_apart = [&](bool far, auto masked) {
          float top = -INFINITY, more = 0.f;
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t s[32];
            tmem_ld32(tS(st) + lanes + 32 * (c & 3), s);
            tmem_ld_wait();
            ready(c & 3, s, masked);
            if (c == 4) top = fmaxf(base, top * z);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (c < 4)
                top = fmaxf(top, __uint_as_float(s[i]));
              else
                more += ex2(fmaf(__uint_as_float(s[i]), z, -top));
            }
          }
          l = far ? fmaf(l, ex2(base - top), more) : l;
          base = far ? top : base;
          added = far;
        };
        auto add_tile = [&](float neg) {
          const float d = -neg - base;
          if (added) return;
          if (d > 64.f) {
            l = fmaf(l, ex2(-d), sum[0].x);
            base = -neg;
          } else {
            l = fmaf(sum[0].x, ex2(d), l);
          }
        };
        // A tile apart: its scores times their K scales, in powers of two, and the
        // weights times their V scales relative to the largest that the row sees.
        auto apart_tile = [&]() {
          auto scores = [&](int c, auto use) {  // 16 columns: few at a time keep the code short
            uint32_t s[16];
            tmem_ld16_nowait(tS(st) + lanes + 16 * c, s);
            tmem_ld_wait();
            const int b = (16 * c) >> p.a.hist.shift;  // of blocks
            const float bk = kScale == kScaleOfBlock ? factor * meta.k[b] : z, bv = kScale == kScaleOfBlock ? lg2(meta.k[8 + b]) : 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float x = __uint_as_float(s[i]) * bk;
              if constexpr (kScale == kScaleOfToken) x *= meta.k[16 * c + i];
              use(i, 16 * c + i > seen ? -INFINITY : x, kScale == kScaleOfToken ? meta.v[16 * c + i] : bv);
            }
          };
          float top = -INFINITY, high = -INFINITY;  // of the scores, and with V's scales
#pragma unroll 1
          for (int c = 0; c < 8; ++c)
            scores(c, [&](int, float x, float v) {
              top = fmaxf(top, x);
              high = fmaxf(high, x + v);
            });
          if (j == 0) {
            m = high == -INFINITY ? top - 100.f : high;  // values of 0 alone: as a tile of them
            base = top == -INFINITY ? 0.f : top;
          } else {
            const bool up = high > m;
            if (__any_sync(0xffffffffu, up)) raise(high, up);
            const float to = fmaxf(base, top);
            l *= ex2(base - to);
            base = to;
          }
          const float mm = m == -INFINITY ? 0.f : m - kManyBias;
          float add = 0.f;
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t w[8];
            float even = 0.f;
            scores(c, [&](int i, float x, float v) {
              add += ex2(x - base);
              const float e = x == -INFINITY ? 0.f : ex2(x + (v - mm));
              if (i & 1)
                w[i / 2] = half2_of(even, e);
              else
                even = e;
            });
            tmem_st8(tS(st) + lanes + 8 * c, w);  // over scores that have been read
          }
          l += add;
        };
        if constexpr (kScale == kScaleOfToken) {
          // With a block's scales in registers too, P cannot be held back: the
          // maximum comes first, and P is written as it is made (over columns of
          // S that have been read).
          auto block = [&](auto masked) {
            const float top = largest(masked);
            if (j == 0) {
              m = top;
            } else {
              const bool up = top > m + 8.f, far = !up && is_far();
              if (__any_sync(0xffffffffu, up || far)) {
                raise(top, up);
                if (__any_sync(0xffffffffu, far)) add_apart(far, masked);
              }
            }
            const float neg = relative();
            if (j == 0) base = -neg;
            clear();
            uint32_t s[2][32];
            tmem_ld32(tS(st) + lanes, s[0]);
#pragma unroll 1
            for (int c = 0; c < 4; c += 2) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t w[16];
                tmem_ld_wait();
                if (c + h < 3) tmem_ld32(tS(st) + lanes + 32 * (c + h + 1), s[1 - h]);
                weights(c + h, s[h], w, neg, masked);
                tmem_st16(tS(st) + lanes + 16 * (c + h), w);
              }
            }
            add_up();
            add_tile(neg);
          };
          if (special) {  // one branch for tiles of the usual kind: with two, 292 us instead of 287 (2048 after 6144)
            if (apart)
              apart_tile();
            else
              block(kMasked);
          } else {
            block(kAll);
          }
        } else {
          if (special) {
            if (apart) {
              apart_tile();
              goto made;
            }
            // masked in place: the loop below has no branch
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t s[32];
              tmem_ld32(tS(st) + lanes + 32 * c, s);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (32 * c + i > seen) s[i] = __float_as_uint(-INFINITY);
              tmem_st32(tS(st) + lanes + 32 * c, s);
            }
            tmem_st_wait();
          }
          {
            if (j == 0) m = largest(kAll);
            float neg = relative();
            if (j == 0) base = -neg;
            const bool far = is_far();
            uint32_t w[64];
#pragma unroll 1
            for (bool again = false;; again = true) {
              clear();
              uint32_t s[2][32];
              tmem_ld32(tS(st) + lanes, s[0]);
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                tmem_ld_wait();
                if (c < 3) tmem_ld32(tS(st) + lanes + 32 * (c + 1), s[(c + 1) & 1]);
                weights(c, s[c & 1], w + 16 * c, neg, kAll);
              }
              add_up();
              if (j == 0 || again || !__any_sync(0xffffffffu, !(sum[0].x <= 60000.f) || far)) break;
              if (__any_sync(0xffffffffu, far)) add_apart(far, kAll);
              const float top = largest(kAll);
              raise(top, top > m);
              neg = relative();
            }
            tmem_st32(tS(st) + lanes, w);
            tmem_st32(tS(st) + lanes + 32, w + 32);
            add_tile(neg);
          }
        made:;
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(L::kPFull + st));
          mbar_arrive(bar(L::kMetaEmpty + mi));
        }
      }
      if (!ok) break;
      // the next unit's q, before this one's output is waited for (its last scores are done)
      if (!wait_warp(L::kItemFull + ((k + 1) & 1), ((k + 1) >> 1) & 1)) break;
      float next_factor = 0.f;
      if (items[(k + 1) & 1].valid && items[(k + 1) & 1].here(st) > 0) next_factor = bring_q(items[(k + 1) & 1]);
      if (n > 0) {
        if (!wait_warp(L::kOFull + st, o_it & 1)) break;
        ++o_it;
        tc_fence_after();
        const int4 found = *(const int4*)&odd_unit[(k & 1) * 4];
        const bool odd = (found.x | found.y | found.z | found.w) != 0, part = !it.whole();
        const int tok = tile_tok + row_tok;
        const bool on = row_tok < p.tile_tokens && tok < it.len;
        // the sum of the weights between 1 and 2, and O in the values' own units: times
        // 2^(m - bias - base), in halves where fp32 does not hold it
        const int le = exponent_of_sum(l);
        l *= power(-le);
        base += (float)le;
        const float units = m - kManyBias - base - (part ? kPartBias : 0.f);
        const bool wide = __any_sync(0xffffffffu, fabsf(units) > 100.f);  // one factor does for the others
        const float half = ex2(0.5f * units), factor_o = (wide ? half : ex2(units)) * (part ? 1.f : 1.f / l);
        uint16_t* orow = p.a.out + (it.row0 + (on ? tok : 0)) * p.a.out_stride + (it.head * p.a.group + row_head) * D;
        const size_t at = (size_t)(2 * blockIdx.x + (it.from == 0)) * (2 * kManyRows) + st * kManyRows + row;
        if (part && on) p.part_ml[at] = make_float2(l == 0.f ? -INFINITY : base, l);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(tO(st) + lanes + 32 * c, o);
          tmem_ld_wait();
          if (wide) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * half);
          }
          if (odd) {  // NaN that was left out of P V: for the rows that see it
#pragma unroll
            for (int i = 0; i < 32; ++i)
              for (int f = 0; f < 4; ++f)
                if (it.start + tok >= bad[((k & 1) * 4 + f) * D + 32 * c + i]) o[i] = 0x7FC00000u;
          }
          if (part) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * factor_o);
            if (on) {
#pragma unroll
              for (int i = 0; i < 4; ++i) store32(p.part_o + at * D + 32 * c + 8 * i, o + 8 * i);
            }
          } else if (on) {
            uint32_t v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 x = mul2(make_float2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), make_float2(factor_o, factor_o));
              v[i] = kF16 ? half2_of(x.x, x.y) : pair16<__nv_bfloat16>(x.x, x.y);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (p.wide)
                store32(orow + 32 * c + 16 * i, v + 8 * i);
              else
#pragma unroll
                for (int f = 0; f < 2; ++f)
                  *(uint4*)(orow + 32 * c + 16 * i + 8 * f) =
                      make_uint4(v[8 * i + 4 * f], v[8 * i + 4 * f + 1], v[8 * i + 4 * f + 2], v[8 * i + 4 * f + 3]);
            }
          }
          __syncwarp();
        }
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::kItemEmpty + (k & 1)));
      factor = next_factor;
    }
  } else if (warp < 12) {
    // -------------------------------------------------------- codes to tiles
    regs_give<kRegsCodes>();
    constexpr int kRowPieces = D / 16, kPieces = kManyRows * kRowPieces / 128;  // 16-byte pieces of a token; a thread's of a tile
    constexpr int kRowStep = 128 / kRowPieces;                                  // rows between them
    // a thread's row and piece: eight neighbouring lanes take two rows' halves of
    // 64 values, whose stores meet no bank twice
    const int prow = (warp - 8) * (kRowStep / 4) + (D == 128 ? (lane >> 2) & 3 : lane >> 2);
    const int pc = D == 128 ? (lane & 3) | (lane >> 4) << 2 : lane & 3;
    const uint32_t to = (pc / 4) * (kManyRows * 128) + prow * 128;  // rows are a multiple of 8 apart
    const uint32_t to0 = to + (((pc % 4 * 2) ^ (prow & 7)) << 4), to1 = to + (((pc % 4 * 2 + 1) ^ (prow & 7)) << 4);
    int* my_bad = bad + (warp - 8) * D;
    uint32_t tiles = 0, m_it = 0;
    uint4 code[2][kPieces];                     // the next K tile and the next V tile
    float sc[kScale == kScaleOfToken ? 4 : 1];  // the next block's scales (a scale for each token: warp 8 K's, warp 9 V's)
    const uint8_t *kc, *vc;                     // the thread's piece of the unit's codes
    const float *ks, *vs;
    int keys;                                   // what the unit's last row sees
    auto unit = [&](const ManyItem& it) {
      const int slot = p.a.b.slot[it.seq];
      const size_t kr = p.a.hist.row(0, slot, it.head), vr = p.a.hist.row(1, slot, it.head);
      kc = p.a.hist.codes + kr * p.a.hist.T_max * D + prow * D + pc * 16;
      vc = p.a.hist.codes + vr * p.a.hist.T_max * D + prow * D + pc * 16;
      ks = p.a.hist.scales + kr * p.a.hist.blocks;
      vs = p.a.hist.scales + vr * p.a.hist.blocks;
      keys = it.start + min(it.len, it.tok0 + 2 * p.tile_tokens);
    };
    auto load = [&](uint4* c, const uint8_t* src, int block) {  // of a tile; nothing behind the last key
      src += (size_t)block * (kManyRows * D);
      if ((block + 1) * kManyRows <= keys) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) c[i] = __ldg((const uint4*)(src + i * (kRowStep * D)));
      } else {
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
          c[i] = block * kManyRows + prow + i * kRowStep < keys ? __ldg((const uint4*)(src + i * (kRowStep * D))) : make_uint4(0, 0, 0, 0);
      }
    };
    auto scales = [&](int block) {
      if constexpr (kScale == kScaleOfToken) {
        if (warp < 10) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = block * kManyRows + lane * 4 + i;
            sc[i] = t < keys ? __ldg((warp == 8 ? ks : vs) + t) : 0.f;
          }
        }
      } else {  // lanes 0..7 K's, 8..15 V's
        const int t = (lane & 7) << p.a.hist.shift;
        sc[0] = lane < 16 && t < kManyRows && block * kManyRows + t < keys ? __ldg((lane < 8 ? ks : vs) + ((block * kManyRows + t) >> p.a.hist.shift)) : 0.f;
      }
    };
    if (wait_warp(L::kItemFull, 0) && items[0].valid) {
      unit(items[0]);
      load(code[0], kc, items[0].from);
      scales(items[0].from);
      load(code[1], vc, items[0].from);
    }
    for (uint32_t k = 0; ok && items[k & 1].valid; ++k) {
      const ManyItem& it = items[k & 1];
      const int first_cut = (it.start + it.tok0) / kManyRows, from = it.from, last = it.to;
      int v_exp = -100;  // of the V scale that the weights are times; a tile whose values are all 0 has the one before it
      int v_low = 1000;  // the least exponent of the V scales so far (blocks: lanes 8..15)
      // the list of NaN values is free: the unit before the last has been written
      for (int i = lane; i < D; i += 32) my_bad[(k & 1) * 4 * D + i] = INT32_MAX;
      if (lane == 0) odd_unit[(k & 1) * 4 + warp - 8] = 0;
      __syncwarp();
#pragma unroll 1
      for (int j = from; j < last && ok; ++j, ++m_it) {
        const int mi = m_it % L::kMetas;
        BlockMeta& meta = metas[mi];
        uint32_t ratio = 0;  // the lane's scale over the tile's (a block of 128: V's), as two fp16
        bool apart = false;
        if (!wait_warp(L::kMetaEmpty + mi, ((m_it / L::kMetas) & 1) ^ 1)) break;
        if constexpr (kScale == kScaleOfToken) {
          if (warp == 8) {
            *(float4*)&meta.k[4 * lane] = make_float4(sc[0], sc[1], sc[2], sc[3]);
          } else if (warp == 9) {
            // a V scale that is not finite makes all its token's values NaN
            bool odd = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) odd |= !(sc[i] <= 0x1.fffffep127f);
            if (__any_sync(0xffffffffu, odd)) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (!(sc[i] <= 0x1.fffffep127f))
#pragma unroll 1
                  for (int d = 0; d < D; ++d) atomicMin(&my_bad[(k & 1) * 4 * D + d], j * kManyRows + 4 * lane + i);
              odd_unit[(k & 1) * 4 + 1] = 1;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[i] = sc[i] <= 0x1.fffffep127f ? sc[i] : 0.f;
            float top = fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3]));
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const bool cut = j >= first_cut;
            const float least = top * power(cut ? -kApartCut : -kApart);
            if (top > 0.f) v_exp = min(exponent_up(top), 120);
            apart = cut && v_exp > v_low + kApartRise;
#pragma unroll
            for (int i = 0; i < 4; ++i) apart |= sc[i] > 0.f && sc[i] < least;
            apart = __any_sync(0xffffffffu, apart);
            if (top > 0.f) v_low = apart ? -126 : min(v_low, v_exp);
            const float r = power(-v_exp);
            *(float4*)&meta.v[4 * lane] = apart ? make_float4(lg2(sc[0]), lg2(sc[1]), lg2(sc[2]), lg2(sc[3]))
                                                : make_float4(sc[0] * r, sc[1] * r, sc[2] * r, sc[3] * r);
            if (lane == 0) meta.factor = 1.f, meta.shift = (float)v_exp, meta.apart = apart;
          }
        } else {
          float top = sc[0];
          if constexpr (kScale == kScaleOfBlock) {
#pragma unroll
            for (int d = 4; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
          }
          const int e = top > 0.f ? min(max(exponent_up(top), lane < 8 ? -120 : -126), 120) : v_exp;
          if constexpr (kScale == kScaleOfBlock) {
            const bool cut = (lane >= 8) & (j >= first_cut);
            const float least = top * (cut ? power(-kApartCut) : power(-kApart));
            const bool far = ((sc[0] > 0.f) & (sc[0] < least)) | (cut & (e > v_low + kApartRise));
            apart = __any_sync(0xffffffffu, far);
            v_low = top > 0.f ? (apart ? -126 : min(v_low, e)) : v_low;
          }
          // K's codes have room for 2^6 more in fp16; the scale of a block of 128 is a factor of K's scores as it is
          const float r = apart ? 1.f : sc[0] * power(-e) * (lane < 8 ? 64.f : 1.f);
          ratio = half2_of(r, r);
          v_exp = __shfl_sync(0xffffffffu, e, 8);
          if (warp == 8 && lane < (kScale == kScaleOfBlock ? 16 : 1)) {
            if (kScale == kScaleOfBlock) meta.k[lane] = sc[0];
            if (lane == 0) {
              meta.factor = kScale == kScaleOfTile ? sc[0] : power(e) * 0x1p-6f;
              meta.shift = (float)v_exp;
              meta.apart = apart;
            }
          }
          if constexpr (kScale == kScaleOfTile) ratio = __shfl_sync(0xffffffffu, ratio, 8);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kMetaFull + mi));
        // The tiles behind these are loaded as the registers become free: the
        // unit's next block, or the first one of the next unit.
        int ahead = j + 1;
        bool more = true;
#pragma unroll
        for (int which = 0; which < 2; ++which, ++tiles) {
          const int slot = tiles % L::kStages;
          if (tiles == (uint32_t)p.skip) {
            ok = false;
            break;
          }
          if (!wait_warp(L::kEmpty + slot, ((tiles / L::kStages) & 1) ^ 1)) break;
          uint8_t* dst = smem + L::kRing + slot * L::kTile;
          const bool look = which && j >= first_cut;
          bool odd = false;
          if (look) {  // apart: a branch in the loop below keeps its pieces from being worked on together (5% of the whole)
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
              const uint32_t c[4] = {code[which][i].x, code[which][i].y, code[which][i].z, code[which][i].w};
#pragma unroll
              for (int x = 0; x < 4; ++x) odd |= any_nan_code(c[x]);
            }
          }
#pragma unroll
          for (int i = 0; i < kPieces; ++i) {
            const uint32_t c[4] = {code[which][i].x, code[which][i].y, code[which][i].z, code[which][i].w};
            uint32_t h[8];
#pragma unroll
            for (int x = 0; x < 4; ++x) e4m3x4_to_f16x2x2(c[x], h[2 * x], h[2 * x + 1]);
            if constexpr (kScale == kScaleOfBlock) {
              const uint32_t r = __shfl_sync(0xffffffffu, ratio, ((prow + i * kRowStep) >> p.a.hist.shift) + 8 * which);
#pragma unroll
              for (int x = 0; x < 8; ++x) h[x] = mul_half2(h[x], r);
            }
            *(uint4*)(dst + to0 + i * (kRowStep * 128)) = make_uint4(h[0], h[1], h[2], h[3]);
            *(uint4*)(dst + to1 + i * (kRowStep * 128)) = make_uint4(h[4], h[5], h[6], h[7]);
          }
          if (kScale == kScaleOfTile && which && ratio != 0x3C003C00u) {  // a V scale that is no power of two, or 0
#pragma unroll 1
            for (int i = 0; i < 2 * kPieces; ++i) {
              uint4* at = (uint4*)(dst + (i & 1 ? to1 : to0) + (i >> 1) * (kRowStep * 128));
              const uint4 h = *at;
              *at = make_uint4(mul_half2(h.x, ratio), mul_half2(h.y, ratio), mul_half2(h.z, ratio), mul_half2(h.w, ratio));
            }
          }
          if (look && __any_sync(0xffffffffu, odd)) {
            // NaN in a tile that some row does not see all of (0 x NaN would
            // reach it): out of the tile, and noted for the rows that do
#pragma unroll 1
            for (int i = 0; i < kPieces; ++i)
#pragma unroll 1
              for (int x = 0; x < 16; ++x) {
                uint16_t* at = (uint16_t*)(dst + (x < 8 ? to0 : to1) + i * (kRowStep * 128)) + x % 8;
                if ((*at & 0x7FFF) > 0x7C00) {
                  *at = 0;
                  atomicMin(&my_bad[(k & 1) * 4 * D + pc * 16 + x], j * kManyRows + prow + i * kRowStep);
                  odd_unit[(k & 1) * 4 + warp - 8] = 1;
                }
              }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::kFull + slot));
          if (!which && ahead == last) {
            if (!wait_warp(L::kItemFull + ((k + 1) & 1), ((k + 1) >> 1) & 1)) break;
            const ManyItem& next = items[(k + 1) & 1];
            more = next.valid;
            if (more) unit(next);
            ahead = next.from;
          }
          if (more) {
            load(code[which], which ? vc : kc, ahead);
            if (!which) scales(ahead);
          }
        }
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::kItemEmpty + (k & 1)));
    }
  } else {
    regs_give<kRegsMma>();
    if (warp == 12) {
      // --------------------------------------------------------------- MMAs
      // In issue order on the tensor core, which is what lets Q K^T of block j
      // + 1 be issued behind P V of block j although both use the same TMEM
      // columns; a commit covers every MMA issued before it.
      constexpr uint32_t id_s = idesc_16(128, 128, true, false, false), id_o = idesc_16(128, D, true, false, true);
      uint32_t p_par[2] = {0, 0}, q_par[2] = {0, 0};
      int at = 0;           // the next tile of the ring ...
      uint32_t at_par = 0;  // ... and its parity
      auto next_tile = [&]() {  // waits for it; its slot
        wait_warp(L::kFull + at, at_par);
        const int slot = at;
        if (++at == L::kStages) at = 0, at_par ^= 1;
        return slot;
      };
      auto commit = [&](int b) {
        if (elect_one()) tc_commit(bar(b));
        __syncwarp();
      };
      auto scores = [&](int st, int slot) {  // S = Q K^T
        tc_fence_after();
        if (elect_one()) {
          const uint32_t q = sdesc_lo(sb + st * L::kTile), kt = sdesc_lo(sb + L::kRing + slot * L::kTile);
#pragma unroll
          for (int e = 0; e < D / 16; ++e) {
            const uint32_t o = ((e / 4) * (kManyRows * 128) + (e % 4) * 32) >> 4;
            if (e == 0)
              mma_ss<false>(tS(st), q, kt, id_s);
            else
              mma_ss<true>(tS(st), q + o, kt + o, id_s);
          }
          tc_commit(bar(L::kSFull + st));
        }
        __syncwarp();
      };
      auto values = [&](int st, int slot, bool first) {  // O += P V
        tc_fence_after();
        if (elect_one()) {
          const uint32_t vt = sdesc_lo(sb + L::kRing + slot * L::kTile, kManyRows * 128);
#pragma unroll
          for (int e = 0; e < kManyRows / 16; ++e)
            mma_ts(tO(st), tS(st) + 8 * e, vt + e * (2048 >> 4), id_o, e > 0 ? 1u : first ? 0u : 1u);
        }
        __syncwarp();
      };
      for (uint32_t k = 0; ok; ++k) {
        if (!wait_warp(L::kItemFull + (k & 1), (k >> 1) & 1)) break;
        const bool valid = items[k & 1].valid;
        const int n0 = items[k & 1].here(0), n1 = items[k & 1].here(1), nb = max(n0, n1);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kItemEmpty + (k & 1)));
        if (!valid) break;
        int ks = next_tile();
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          if (!ok || (st ? n1 : n0) <= 0 || !wait_warp(L::kQFull + st, q_par[st])) continue;
          q_par[st] ^= 1;
          scores(st, ks);
        }
        if (!ok) break;
        commit(L::kEmpty + ks);
        for (int j = 0; j < nb && ok; ++j) {
          const bool more = j + 1 < nb;
          const int vsl = next_tile();
          if (!ok) break;
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            const int n = st ? n1 : n0;
            if (j < n) {
              if (!wait_warp(L::kPFull + st, p_par[st])) break;
              p_par[st] ^= 1;
              values(st, vsl, j == 0);
            }
            if (st == 1) commit(L::kEmpty + vsl);
            if (st == 0 && more) ks = next_tile();
            if (!ok) break;
            if (j + 1 < n)
              scores(st, ks);
            else if (j + 1 == n)
              commit(L::kOFull + st);
          }
          if (ok && more) commit(L::kEmpty + ks);
        }
      }
      if (!ok) {  // give-up: wait (bounded) for the MMAs issued so far
        commit(L::kDone);
        for (int n = 0; n < (1 << 20) && !mbar_try_wait(bar(L::kDone), 0); ++n) {
        }
      }
      __syncwarp();
    } else if (warp == 13) {
      // ---------------------------------------------------------- scheduler
      ManyWalk walk;
      bool live = !stop && walk.begin(p);
      for (uint32_t k = 0;; ++k) {
        if (!wait_warp(L::kItemEmpty + (k & 1), ((k >> 1) & 1) ^ 1)) break;
        if (lane == 0) {
          walk.it.valid = live;
          *(ManyItem*)(smem + L::kItems + (k & 1) * sizeof(ManyItem)) = walk.it;
          mbar_arrive(bar(L::kItemFull + (k & 1)));
        }
        __syncwarp();
        if (!live) break;
        live = walk.next(p);
      }
    } else if (warp == 14) {
      // a unit's q on its way to L2 while the unit before is worked on
      for (uint32_t k = 0;; ++k) {
        if (!wait_warp(L::kItemFull + (k & 1), (k >> 1) & 1)) break;
        const ManyItem it = items[k & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kItemEmpty + (k & 1)));
        if (!it.valid) break;
        const int tokens = min(2 * p.tile_tokens, it.len - it.tok0), lines = p.a.group * D / 64;  // of 128 bytes, a token
        const char* q = (const char*)(p.a.q + (it.row0 + it.tok0) * p.a.q_stride + it.head * p.a.group * D);
        for (int i = lane; i < tokens * lines; i += 32)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(q + (i / lines) * p.a.q_stride * 2 + (i % lines) * 128));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(tmem, 512);
}

// A unit's parts joined: D / 4 threads to a row, a CTA for every 1024 / D rows of
// each place where the line is cut.  Four parts' loads are in flight together.
template <int D, bool kF16>
__global__ void __launch_bounds__(256) k_join_history(const __grid_constant__ ManyParams p) {
  constexpr int kLanes = D / 4, kRowsHere = 256 / kLanes, kCtas = 2 * kManyRows / kRowsHere;
  const int r = blockIdx.x % kCtas * kRowsHere + (int)threadIdx.x / kLanes, c = blockIdx.x / kCtas + 1;
  const ManyCut u = p.cut[c];
  auto same = [&](int i) { return p.cut[i].seq == u.seq && p.cut[i].level == u.level && p.cut[i].head == u.head && p.cut[i].block > 0; };
  if (u.block == 0 || (c > 1 && same(c - 1))) return;  // not where a unit is cut first
  int last = c;  // the last CTA that has a part
  while (last + 1 < p.ctas && same(last + 1)) ++last;
  const int st = r / kManyRows, row = r % kManyRows, row_tok = row / p.a.group;
  const int tok = u.level * 2 * p.tile_tokens + st * p.tile_tokens + row_tok, col = (int)threadIdx.x % kLanes * 4;
  const bool on = row_tok < p.tile_tokens && tok < p.a.b.len(u.seq);
  uint16_t* dst = p.a.out + (p.a.b.begin[u.seq] + tok) * p.a.out_stride + (u.head * p.a.group + row % p.a.group) * D + col;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are there
  if (!on) return;
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = c - 1; i <= last; i += 4) {
    float2 ml[4];
    float4 v[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const int k = min(i + f, last);
      const size_t at = (size_t)(2 * k + (k < c)) * (2 * kManyRows) + r;
      ml[f] = __ldcg(p.part_ml + at);
      v[f] = __ldcg((const float4*)(p.part_o + at * D + col));
    }
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      if (i + f > last) break;
      const float top = fmaxf(m, ml[f].x);
      const float a = m == -INFINITY ? 0.f : ex2(m - top), b = ml[f].x == -INFINITY ? 0.f : ex2(ml[f].x - top);
      l = l * a + ml[f].y * b;
      o = make_float4(o.x * a + v[f].x * b, o.y * a + v[f].y * b, o.z * a + v[f].z * b, o.w * a + v[f].w * b);
      m = top;
    }
  }
  const float inv = joined_factor(l);
  *(uint2*)dst = kF16 ? make_uint2(half2_of(o.x * inv, o.y * inv), half2_of(o.z * inv, o.w * inv))
                      : make_uint2(pair16<__nv_bfloat16>(o.x * inv, o.y * inv), pair16<__nv_bfloat16>(o.z * inv, o.w * inv));
}

// The line cut into even parts, by what its blocks cost: with both streams at
// work a block takes longer than with one.  A part has three blocks at least.
// No cut falls before the last block of a unit whose first stream ends a block
// earlier, so that each stream has a block in every part.
static bool cut_line(ManyParams& p, int sms) {
  const SeqBatch& b = p.a.b;
  const int heads = p.a.hist.heads;
  auto cost = [](const ManyItem& it) { return it.n[1] ? 4 : 3; };
  constexpr int kUnit = 10;  // what a unit costs beside its blocks
  long long total = 0, most = 3;
  ManyItem it;
  for (it.seq = 0; it.seq < b.n; ++it.seq)
    for (it.level = 0; it.level * 2LL * p.tile_tokens < b.len(it.seq); ++it.level) {
      unit_blocks(b, p.tile_tokens, it);
      total += ((long long)cost(it) * it.blocks() + kUnit) * heads;
      most = std::max(most, (long long)cost(it));
    }
  p.ctas = (int)std::max(1LL, std::min((long long)std::min(sms, kMaxCuts), total / (3 * most)));
  int c = 0;
  long long before = 0;  // cost in front of this level's units
  bool any = false;
  for (it.seq = 0; it.seq < b.n; ++it.seq)
    for (it.level = 0; it.level * 2LL * p.tile_tokens < b.len(it.seq); ++it.level) {
      unit_blocks(b, p.tile_tokens, it);
      const long long unit = (long long)cost(it) * it.blocks() + kUnit;
      for (; c < p.ctas; ++c) {
        const long long at = total * c / p.ctas - before;
        if (at >= unit * heads) break;
        int block = std::min((int)(std::max(at % unit - kUnit, 0LL) / cost(it)), it.blocks() - 1);
        if (block == it.blocks() - 1 && it.n[1] > it.n[0] && block > 0) --block;
        p.cut[c] = {it.seq, it.level, (int)(at / unit), block};
        any |= block > 0;
      }
      before += unit * heads;
    }
  p.cut[p.ctas] = {b.n, 0, 0, 0};
  return any;
}

template <int D, bool kF16, int kScale>
static cudaError_t configure() {
  return configure_split(k_history_many<D, kF16, kScale>, kManyThreads, 256 * kRegsRows + 128 * (kRegsCodes + kRegsMma), kRegsRows,
                         std::max(kRegsCodes, kRegsMma), ManySmem<D>::kTotal);
}

template <int D, bool kF16>
static cudaError_t configure_all() {
  const cudaError_t e[3] = {configure<D, kF16, kScaleOfTile>(), configure<D, kF16, kScaleOfBlock>(), configure<D, kF16, kScaleOfToken>()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

cudaError_t configure_history_many() {
  const cudaError_t e[4] = {configure_all<128, false>(), configure_all<128, true>(), configure_all<64, false>(), configure_all<64, true>()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

template <int D, bool kF16>
static cudaError_t launch(const ManyParams& p, bool join, cudaStream_t st) {
  if (p.a.hist.block == 1)
    k_history_many<D, kF16, kScaleOfToken><<<p.ctas, kManyThreads, ManySmem<D>::kTotal, st>>>(p);
  else if (p.a.hist.block < kManyRows)
    k_history_many<D, kF16, kScaleOfBlock><<<p.ctas, kManyThreads, ManySmem<D>::kTotal, st>>>(p);
  else
    k_history_many<D, kF16, kScaleOfTile><<<p.ctas, kManyThreads, ManySmem<D>::kTotal, st>>>(p);
  if (join) {  // its CTAs begin as the parts' end, and wait for all of them
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((p.ctas - 1) * (2 * kManyRows * D / 1024));
    c.blockDim = dim3(256);
    c.stream = st;
    c.attrs = &early;
    c.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&c, k_join_history<D, kF16>, p);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

cudaError_t launch_history_many(const HistoryAttnParams& a, const wave_ctx* h, int type, cudaStream_t st) {
  ManyParams p;
  p.a = a;
  p.tile_tokens = kManyRows / a.group;
  p.part_o = h->ws.part_o;
  p.part_ml = h->ws.part_ml;
  p.wide = ((uintptr_t)a.out & 31) == 0 && a.out_stride % 16 == 0;
  p.sink = make_sink(h->ws.err, h->err_host_dev, h->timeout_ns);
  p.skip = h->skip_sig_kind == 11 ? h->skip_sig : -1;
  const bool join = cut_line(p, h->pl.grid);
  if (h->pl.cfg.head_dim == 128) return type == WAVE_F16 ? launch<128, true>(p, join, st) : launch<128, false>(p, join, st);
  return type == WAVE_F16 ? launch<64, true>(p, join, st) : launch<64, false>(p, join, st);
}

}  // namespace wave
