// prompt_attn.cu -- wave_prompt_attention: causal attention over packed
// prompts with grouped heads.
//
//   o_i = sum_{j <= i} p_ij v_j / sum_{j <= i} p_ij,   p_ij = exp(scale q_i.k_j - m_i)
//
// Bound by the tensor cores for long prompts (4 D flops for a query and a key
// it attends to; the blocks on the diagonal are done whole), by HBM for short
// ones with many heads, by latency for a single short one.  Measured (captured
// launches in a row; 32 heads of 128): a prompt of 8192 tokens 370 to 405 us
// with the power limit active, 1.36 to 1.49 PFLOP/s of causal work; prompts of
// 4096, 1 and 2001 tokens, 8 K/V heads, fp16, 129 us = 1.32 PFLOP/s; 16 prompts
// of 1 to 1500 tokens, 8005 in all, 73 to 75 us; 8192 tokens of 16 heads of 64,
// 162 us = 0.85 PFLOP/s; a prompt of 25 tokens of 16 heads of 64, 6 us.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/wave.h"
#include "ctx.h"
#include "prompt.h"
#include "prompt_ptx.cuh"

using namespace wave;

namespace wave {

constexpr int kRows = 128;         // query rows of one stream, and keys of one block
constexpr int kAttnThreads = 384;  // 8 softmax warps (two streams), then copies, MMAs, guard, scheduler
constexpr int kMaxParts = 160;     // items, where keys are divided
constexpr int kRegsSoftmax = 208, kRegsRest = 80;  // a row's 128 scores stay in registers

// A pair's part `part` of `parts` has the key blocks from part_begin on: even
// shares, the last (with the diagonal blocks of both tiles) no smaller than two.
__host__ __device__ inline int part_begin(int blocks, int parts, int part) { return (int)((long long)blocks * part / parts); }

struct AttnParams {
  CUtensorMap tm_q, tm_k, tm_v;
  int n;                            // sequences, longest first
  int32_t begin[WAVE_MAX_SEQS], len[WAVE_MAX_SEQS];
  int Hq, group;                    // query heads, and how many of them share a K/V head
  const uint16_t* v;
  uint16_t* out;
  long long v_stride, out_stride;
  float scale2;                     // scale * log2(e)
  int wide;                         // out's rows are 32-byte aligned
  int more;                         // more items than SMs
  // Few items: the keys of a pair of row tiles are divided among several (see
  // attention_parts).  Then CTA i works on a part of pair j, where cut_first[j]
  // <= i, and leaves its sums in place i of the workspace.
  int cuts;                         // pairs, 0: not divided
  int32_t cut_first[kMaxParts + 1], cut_seq[kMaxParts], cut_level[kMaxParts];
  float* part_o;                    // [item][256 rows][D], not divided by the sums of weights
  float2* part_ml;                  // [item][256 rows]: the maximum and the sum
  ErrSink sink;
  int skip;  // testing hook: the copies end before this tile of K and V (-1: off)
};

// What the scheduler hands to the other warps.
struct AttnItem {
  int valid, head;
  int row0, left;      // first query row of the pair, rows from there to the sequence's end
  int kv0;             // the first row of its keys
  int diag;            // whether the last key blocks are the tiles' own
  int part;            // place of its sums in the workspace; -1: it has all keys
  int n0, n1;          // key blocks of stream 0 and 1 (0: no rows)
  uint32_t bad[2][4];  // keys of the last two V blocks that hold a value which is not finite
};

// Shared memory: the two streams' Q tiles, a ring of K and V tiles, barriers, items.
template <int D>
struct AttnSmem {
  static constexpr int kTile = kRows * D * 2;
  static constexpr int kStages = D == 128 ? 5 : 10;
  static constexpr int kRing = 2 * kTile;
  static constexpr int kBars = kRing + kStages * kTile;
  enum {
    kFull = 0,
    kEmpty = kFull + kStages,
    kQFull = kEmpty + kStages,
    kQEmpty = kQFull + 2,
    kSFull = kQEmpty + 2,
    kPFull = kSFull + 2,
    kOFull = kPFull + 2,
    kGo = kOFull + 2,
    kOk,
    kDone,
    kItemFull,
    kItemEmpty = kItemFull + 2,
    kNext = kItemEmpty + 2,
    kCount
  };
  static constexpr int kItems = kBars + kCount * 8;
  static constexpr int kAnswer = (kItems + 2 * (int)sizeof(AttnItem) + 15) / 16 * 16;
  static constexpr int kMisc = kAnswer + 16;
  static constexpr int kTotal = kMisc + 16 + 1024;  // + alignment
};

template <bool kF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  uint32_t r;
  if constexpr (kF16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The rank-th pair of row tiles in descending order of work: pairs with many
// key blocks first, so that the last ones to start are the shortest.  The
// level of a pair is its index in its sequence (its work is 2 level + 2 key
// blocks); the sequences that reach a level are the first ones, as they are
// sorted.  Called by a whole warp.
__device__ __forceinline__ void pair_of_rank(const AttnParams& p, int rank, int& seq, int& level) {
  const int lane = threadIdx.x & 31;
  int np[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int s = lane + 32 * i;
    np[i] = s < p.n ? (int)(((unsigned)p.len[s] + 2 * kRows - 1) / (2 * kRows)) : 0;
  }
  auto at_or_above = [&](int t) {  // pairs whose level is t or more
    int c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) c += max(0, np[i] - t);
    return (int)__reduce_add_sync(0xffffffffu, (unsigned)c);
  };
  int lo = 0, hi = (int)(((unsigned)p.len[0] + 2 * kRows - 1) / (2 * kRows)) - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (at_or_above(mid + 1) <= rank)
      hi = mid;
    else
      lo = mid + 1;
  }
  level = lo;
  seq = rank - at_or_above(lo + 1);
}

// Attention on the tensor cores, a pair of 128-row query tiles per work
// item.  One pass over the keys with the softmax's running maximum and sum:
// S = Q K^T by tcgen05 into TMEM, a thread per row turns S into the weights
// P (16 bits, written over S), O += P V by tcgen05 with P read from TMEM.  The
// two tiles are two streams: while one stream's weights are computed the
// tensor core works for the other.
//
// MMAs issued by one thread run in issue order, which is what lets Q K^T of
// block j + 1 be issued behind P V of block j although both use the same TMEM
// columns; a commit covers every MMA issued before it, so s_full of block
// j + 1 also says that P V of block j is complete.
// kCut: with few items, whose keys are divided (a variant of its own: as one
// with the rest 2% slower for many items).
template <int D, bool kF16, bool kCut>
__global__ void __launch_bounds__(kAttnThreads, 1) k_prompt_attention(const __grid_constant__ AttnParams p) {
  using L = AttnSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base_raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024 - (base_raw & 1023)) & 1023);
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) { return sb + L::kBars + i * 8; };
  AttnItem* items = (AttnItem*)(smem + L::kItems);
  uint32_t* tmem_word = (uint32_t*)(smem + L::kMisc);

  if (warp == 9) {
    if (lane == 0) {
      for (int i = 0; i < L::kStages; ++i) {
        mbar_init(bar(L::kFull + i), 1);
        mbar_init(bar(L::kEmpty + i), 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(bar(L::kQFull + i), 1);
        mbar_init(bar(L::kQEmpty + i), 1);
        mbar_init(bar(L::kSFull + i), 1);
        mbar_init(bar(L::kPFull + i), 4);  // a stream's softmax warps
        mbar_init(bar(L::kOFull + i), 1);
        mbar_init(bar(L::kItemFull + i), 1);
        mbar_init(bar(L::kItemEmpty + i), 11);  // 8 softmax warps, copies, MMAs, guard
      }
      mbar_init(bar(L::kNext), 1);
      mbar_init(bar(L::kGo), 1);
      mbar_init(bar(L::kOk), 1);
      mbar_init(bar(L::kDone), 1);
      fence_mbar_init();
      fence_proxy_async_smem();
    }
    __syncwarp();
    tmem_alloc(smem_u32(tmem_word), 512);
    tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    prefetch_tmap(&p.tm_q);
    prefetch_tmap(&p.tm_k);
    prefetch_tmap(&p.tm_v);
  }
  const bool stop = warp == 11 && stopped(p.sink);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_word;
  auto tS = [&](int st) { return tmem + st * 128; };
  auto tO = [&](int st) { return tmem + 256 + st * D; };

  // Every wait is bounded; a give-up sets the error word and ends the role's
  // loop, which lets the waits of the others run out too; CTAs that begin later
  // find no work.  wait: one thread;
  // wait_warp: a whole warp, which stays together.
  bool ok = true;
  auto wait = [&](int b, uint32_t parity) { return ok = wait_bar(bar(b), parity, p.sink); };
  auto wait_warp = [&](int b, uint32_t parity) {
    return ok = __all_sync(0xffffffffu, wait_bar(bar(b), parity, p.sink));
  };

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    regs_take<kRegsSoftmax>();
    const int st = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    uint32_t s_it = 0, o_it = 0;
    for (uint32_t k = 0; ok; ++k) {
      if (!wait_warp(L::kItemFull + (k & 1), (k >> 1) & 1)) break;
      const AttnItem& it = items[k & 1];
      const bool live = it.valid != 0;
      const int n = st ? it.n1 : it.n0;
      const bool diag = !kCut || it.diag;
      if (live && n > 0) {
        float m = -INFINITY, l = 0.f;
        for (int j = 0; j < n; ++j, ++s_it) {
          if (!wait_warp(L::kSFull + st, s_it & 1)) break;
          tc_fence_after();
          uint32_t s[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS(st) + lanes + 32 * c, s + 32 * c);
          tmem_ld_wait();
          if (j == n - 1 && diag) {  // the diagonal block
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (c > row) s[c] = __float_as_uint(-INFINITY);
          }
          float mx[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) mx[c] = __uint_as_float(s[c]);
#pragma unroll
          for (int c = 4; c < 124; c += 8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) mx[i] = max3(mx[i], __uint_as_float(s[c + 2 * i]), __uint_as_float(s[c + 2 * i + 1]));
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) mx[i] = fmaxf(mx[i], __uint_as_float(s[124 + i]));
          const float bm = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          // The maximum moves only when a weight would exceed 2^8 (the sums
          // and the 16-bit weights have room for that): O is rescaled seldom.
          if (j == 0) {
            m = bm;
          } else {
            const bool up = (bm - m) * p.scale2 > 8.f;
            if (__any_sync(0xffffffffu, up)) {
              const float m2 = up ? bm : m;
              const float a = up ? (m == -INFINITY ? 0.f : ex2((m - m2) * p.scale2)) : 1.f;
              l *= a;
              m = m2;
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(tO(st) + lanes + 32 * c, o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
                tmem_st32(tO(st) + lanes + 32 * c, o);
              }
            }
          }
          const float neg = m == -INFINITY ? 0.f : -m * p.scale2;
          const float2 scale = make_float2(p.scale2, p.scale2), neg2 = make_float2(neg, neg);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float2 t =
                  fma2(make_float2(__uint_as_float(s[64 * c + 2 * i]), __uint_as_float(s[64 * c + 2 * i + 1])), scale, neg2);
              const float2 e = make_float2(ex2(t.x), ex2(t.y));
              sum[i & 1] = add2(sum[i & 1], e);
              w[i] = pack16<kF16>(e.x, e.y);
            }
            tmem_st32(tS(st) + lanes + 32 * c, w);
          }
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::kPFull + st));
        }
        if (!ok || !wait_warp(L::kOFull + st, o_it & 1)) break;
        ++o_it;
        tc_fence_after();
        const float inv = 1.f / l;
        uint32_t bad = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) bad |= it.bad[0][i] | it.bad[1][i];
        uint16_t* orow = p.out + (size_t)(it.row0 + st * kRows + row) * p.out_stride + it.head * D;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(tO(st) + lanes + 32 * c, o);
          tmem_ld_wait();
          if (bad) {
            // values of the last blocks' keys that are not finite were left
            // out of P V; the rows that attend to them get them here
            for (int g = 0; g <= st; ++g)
              for (int w = 0; w < 4; ++w)
                for (uint32_t bits = it.bad[g][w]; bits; bits &= bits - 1) {
                  const int key = w * 32 + __ffs(bits) - 1;
                  const int kr = it.kv0 + (it.n0 - 1 + g) * kRows + key;
                  if ((g == st && key > row) || kr >= it.row0 + it.left) continue;
                  const uint16_t* vr = p.v + (size_t)kr * p.v_stride + (it.head / p.group) * D + 32 * c;
#pragma unroll
                  for (int i = 0; i < 32; ++i) {
                    const float v = kF16 ? __half2float(__ushort_as_half(vr[i])) : __uint_as_float((uint32_t)vr[i] << 16);
                    if (!isfinite(v)) o[i] = __float_as_uint(__uint_as_float(o[i]) + v);
                  }
                }
          }
          if (kCut && it.part >= 0) {
            if (st * kRows + row < it.left) {
              const size_t at = (size_t)it.part * (2 * kRows) + st * kRows + row;
#pragma unroll
              for (int i = 0; i < 4; ++i) store32(p.part_o + at * D + 32 * c + 8 * i, o + 8 * i);
              if (c == 0) p.part_ml[at] = make_float2(m, l);
            }
            __syncwarp();
            continue;
          }
          if (st * kRows + row < it.left) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 v = mul2(make_float2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), make_float2(inv, inv));
              w[i] = pack16<kF16>(v.x, v.y);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (p.wide)
                store32(orow + 32 * c + 16 * i, w + 8 * i);
              else
#pragma unroll
                for (int f = 0; f < 2; ++f)
                  *(uint4*)(orow + 32 * c + 16 * i + 8 * f) =
                      make_uint4(w[8 * i + 4 * f], w[8 * i + 4 * f + 1], w[8 * i + 4 * f + 2], w[8 * i + 4 * f + 3]);
            }
          }
          __syncwarp();
        }
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::kItemEmpty + (k & 1)));
      if (!live) break;
    }
  } else {
    regs_give<kRegsRest>();
    if (warp == 8) {
      // ------------------------------------------------------------- copies
      if (lane == 0) {
        uint32_t it_r = 0;  // tiles brought into the ring
        auto tile = [&](const CUtensorMap* map, uint32_t dst, int head, int r, uint32_t b) {
#pragma unroll
          for (int i = 0; i < D / 64; ++i) tma_load_3d_plain(dst + i * (kRows * 128), map, 64 * i, head, r, b);
        };
        uint32_t q_it[2] = {0, 0};
        for (uint32_t k = 0; ok; ++k) {
          if (!wait(L::kItemFull + (k & 1), (k >> 1) & 1)) break;
          const AttnItem& src = items[k & 1];
          const int valid = src.valid, head = src.head, row0 = src.row0, kv0 = src.kv0, n0 = src.n0, n1 = src.n1;
          mbar_arrive(bar(L::kItemEmpty + (k & 1)));
          if (!valid) break;
          const int nb = max(n0, n1), kvh = head / p.group;
          auto query = [&](int st) {
            if (!wait(L::kQEmpty + st, (q_it[st] & 1) ^ 1)) return;
            mbar_arrive_expect_tx(bar(L::kQFull + st), L::kTile);
            tile(&p.tm_q, sb + st * L::kTile, head, row0 + st * kRows, bar(L::kQFull + st));
            ++q_it[st];
          };
          query(0);
          for (int j = 0; j < 2 * nb && ok; ++j, ++it_r) {  // K_0, V_0, K_1, V_1, ...
            const int slot = it_r % L::kStages;
            if (it_r == (uint32_t)p.skip) {
              ok = false;
              break;
            }
            if (!wait(L::kEmpty + slot, ((it_r / L::kStages) & 1) ^ 1)) break;
            mbar_arrive_expect_tx(bar(L::kFull + slot), L::kTile);
            tile(j & 1 ? &p.tm_v : &p.tm_k, sb + L::kRing + slot * L::kTile, kvh, kv0 + (j >> 1) * kRows,
                 bar(L::kFull + slot));
            if (j == 0 && n1) query(1);
          }
        }
        if (!ok) {  // give-up: the copies in flight land before the shared memory is left
          auto drain = [&](int b, uint32_t parity) {
            for (int n = 0; n < (1 << 20) && !mbar_try_wait(bar(b), parity); ++n) {
            }
          };
          for (int st = 0; st < 2; ++st)
            if (q_it[st]) drain(L::kQFull + st, (q_it[st] - 1) & 1);
          for (uint32_t i = it_r > L::kStages ? it_r - L::kStages : 0; i < it_r; ++i)
            drain(L::kFull + i % L::kStages, (i / L::kStages) & 1);
        }
      }
      __syncwarp();
    } else if (warp == 9) {
      // --------------------------------------------------------------- MMAs
      {
        // A group of MMAs is issued hardly faster than it runs (some 400 cycles
        // of them are queued), so what stands between two groups is short:
        // waits for tiles are made while the group before them runs.
        constexpr uint32_t id_s = idesc_16(128, 128, kF16, false, false), id_o = idesc_16(128, D, kF16, false, true);
        uint32_t p_par[2] = {0, 0}, q_par[2] = {0, 0}, g_par = 0;
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
              const uint32_t o = ((e / 4) * (kRows * 128) + (e % 4) * 32) >> 4;
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
            const uint32_t vt = sdesc_lo(sb + L::kRing + slot * L::kTile, kRows * 128);
#pragma unroll
            for (int e = 0; e < kRows / 16; ++e)
              mma_ts(tO(st), tS(st) + 8 * e, vt + e * (2048 >> 4), id_o, e > 0 ? 1u : first ? 0u : 1u);
          }
          __syncwarp();
        };
        int n0 = 0, n1 = 0;  // key blocks of the streams (0: no item, or no second tile)
        bool diag = true;
        for (uint32_t k = 0; ok; ++k) {
          if (!wait_warp(L::kItemFull + (k & 1), (k >> 1) & 1)) break;
          {
            const AttnItem& it = items[k & 1];
            n0 = it.valid ? it.n0 : 0, n1 = it.valid ? it.n1 : 0;
            if constexpr (kCut) diag = it.diag;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::kItemEmpty + (k & 1)));
          if (!n0) break;
          const int nb = max(n0, n1);
          // the first scores, behind the last P V of the item before: its epilogue is not waited for
          int ks = next_tile();
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            const int n = st ? n1 : n0;
            if (!ok || !n || !wait_warp(L::kQFull + st, q_par[st])) continue;
            q_par[st] ^= 1;
            scores(st, ks);
            if (n == 1) commit(L::kQEmpty + st);
          }
          if (!ok) break;
          commit(L::kEmpty + ks);
          int vs = next_tile();
          if (diag && n0 == 1 && lane == 0) mbar_arrive(bar(L::kGo));
          for (int j = 0; j < nb && ok; ++j) {
            const bool more = j + 1 < nb;
            bool unchecked = diag && j >= n0 - 1;  // the guard looks over V
            int vnext = 0;
#pragma unroll
            for (int st = 0; st < 2; ++st) {
              const int n = st ? n1 : n0;
              if (j < n) {
                if (!wait_warp(L::kPFull + st, p_par[st])) break;
                p_par[st] ^= 1;
                if (unchecked) {
                  if (!wait_warp(L::kOk, g_par)) break;
                  g_par ^= 1;
                  unchecked = false;
                }
                values(st, vs, j == 0);
              }
              if (st == 1) commit(L::kEmpty + vs);
              if (st == 0 && more) ks = next_tile();
              if (!ok) break;
              if (j + 1 < n) {
                scores(st, ks);
                if (j + 2 == n) commit(L::kQEmpty + st);
              } else if (j < n) {
                commit(L::kOFull + st);
              }
              if (st == 0 && more) {
                vnext = next_tile();
                if (!ok) break;
                if (diag && j + 1 >= n0 - 1 && lane == 0) mbar_arrive(bar(L::kGo));
              }
            }
            if (ok && more) commit(L::kEmpty + ks);
            vs = vnext;
          }
        }
        if (!ok) {  // give-up: wait (bounded) for the MMAs issued so far
          commit(L::kDone);
          for (int n = 0; n < (1 << 20) && !mbar_try_wait(bar(L::kDone), 0); ++n) {
          }
        }
      }
      __syncwarp();
    } else if (warp == 10) {
      // -------------------------------------------------------------- guard
      // A weight of zero times a value that is not finite is NaN, so the V
      // tiles with keys that some of their rows do not attend to (the blocks
      // on the diagonal; behind a sequence's end lie other sequences) are
      // looked over first: such values become zero there, and the epilogue
      // adds them to the rows that do attend to them.
      uint32_t it_r = 0, g_it = 0;
      for (uint32_t k = 0; ok; ++k) {
        if (!wait_warp(L::kItemFull + (k & 1), (k >> 1) & 1)) break;
        AttnItem& it = items[k & 1];
        const int valid = it.valid, n0 = it.n0, nb = max(it.n0, it.n1);
        for (int j = n0 - 1; valid && (!kCut || it.diag) && j < nb; ++j) {
          if (!wait_warp(L::kGo, g_it & 1)) break;
          ++g_it;
          uint8_t* v = smem + L::kRing + ((it_r + 2 * j + 1) % L::kStages) * L::kTile;
          uint32_t acc[4] = {0, 0, 0, 0};  // x * 0 is NaN exactly where x is not finite
#pragma unroll 1
          for (int o = lane * 16; o < L::kTile; o += 8 * 512) {
            uint4 x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = *(const uint4*)(v + o + i * 512);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
              for (int f = 0; f < 4; ++f) {
                if constexpr (kF16)
                  asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc[f]) : "r"(w[f]), "r"(0));
                else
                  asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc[f]) : "r"(w[f]), "r"(0));
              }
            }
          }
          if (__any_sync(0xffffffffu, (((acc[0] | acc[1]) | (acc[2] | acc[3])) & 0x7fff7fffu) != 0)) {
            constexpr uint32_t kExp = kF16 ? 0x7C00u : 0x7F80u;
            for (int o = lane * 4; o < L::kTile; o += 128) {
              uint32_t w = *(uint32_t*)(v + o);
              const bool lo = (w & kExp) == kExp, hi = ((w >> 16) & kExp) == kExp;
              if (lo || hi) {
                if (lo) w &= 0xFFFF0000u;
                if (hi) w &= 0x0000FFFFu;
                *(uint32_t*)(v + o) = w;
                const int key = (o / 128) % kRows;
                atomicOr(&it.bad[j - (n0 - 1)][key >> 5], 1u << (key & 31));
              }
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::kOk));
        }
        if (!ok) break;
        it_r += 2 * nb;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kItemEmpty + (k & 1)));
        if (!valid) break;
      }
    } else {
      // ---------------------------------------------------------- scheduler
      // The first item is the CTA's own, the later ones those of CTAs that have
      // not begun: items go to whoever is free next, longest first, and the
      // copies and first scores of one run under the end of the one before.
      for (uint32_t k = 0; ok; ++k) {
        if (!wait_warp(L::kItemEmpty + (k & 1), ((k >> 1) & 1) ^ 1)) break;
        int idx = blockIdx.x;
        bool valid = !stop;
        if (k > 0) valid = !kCut && p.more;
        if (k > 0 && valid) {
          if (lane == 0) {
            fence_proxy_async_smem();  // the last answer has been read
            mbar_arrive_expect_tx(bar(L::kNext), 16);
            cta_request(sb + L::kAnswer, bar(L::kNext));
          }
          __syncwarp();
          if (!wait_warp(L::kNext, (k - 1) & 1)) {  // give-up: the answer lands before the shared memory is left
            for (int n = 0; n < (1 << 20) && !mbar_try_wait(bar(L::kNext), (k - 1) & 1); ++n) {
            }
            break;
          }
          valid = cta_taken(sb + L::kAnswer, idx);
        }
        int seq = 0, level = 0, head = idx % p.Hq, part = 0, parts = 1;
        if constexpr (!kCut) {
          if (valid) pair_of_rank(p, idx / p.Hq, seq, level);
        } else {
          int lo = 0, hi = p.cuts - 1;
          while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.cut_first[mid] <= idx)
              lo = mid;
            else
              hi = mid - 1;
          }
          seq = p.cut_seq[lo], level = p.cut_level[lo];
          parts = (p.cut_first[lo + 1] - p.cut_first[lo]) / p.Hq;
          head = (idx - p.cut_first[lo]) / parts, part = (idx - p.cut_first[lo]) % parts;
        }
        if (lane == 0) {
          AttnItem& it = items[k & 1];
          const int left = p.len[seq] - level * 2 * kRows;
          const int n0 = 2 * level + 1, n1 = left > kRows ? n0 + 1 : 0;
          int from = 0, to = max(n0, n1);
          if constexpr (kCut) {
            from = part_begin(max(n0, n1), parts, part), to = part_begin(max(n0, n1), parts, part + 1);
            it.diag = part == parts - 1;
            it.part = parts > 1 ? idx : -1;
          }
          it.valid = valid;
          it.head = head;
          it.kv0 = p.begin[seq] + from * kRows;
          it.row0 = p.begin[seq] + level * 2 * kRows;
          it.left = left;
          it.n0 = min(n0, to) - from;
          it.n1 = n1 ? to - from : 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) it.bad[i / 4][i % 4] = 0;
          mbar_arrive(bar(L::kItemFull + (k & 1)));
        }
        __syncwarp();
        if (!valid) break;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// A row's parts joined: a CTA per 32 rows of a tile and head, D / 4 threads to a row.
template <int D, bool kF16>
__global__ void __launch_bounds__(256) k_join_parts(const __grid_constant__ AttnParams p) {
  constexpr int kLanes = D / 4;
  const int block = blockIdx.x % 8, head = blockIdx.x / 8 % p.Hq, pair = blockIdx.x / 8 / p.Hq;
  const int parts = (p.cut_first[pair + 1] - p.cut_first[pair]) / p.Hq, col = (int)threadIdx.x % kLanes * 4;
  if (parts == 1) return;  // written by the attention itself
  const int seq = p.cut_seq[pair], first = p.cut_level[pair] * 2 * kRows;
  const size_t item = p.cut_first[pair] + head * parts;
  for (int r = block * 32 + (int)threadIdx.x / kLanes; r < block * 32 + 32; r += 256 / kLanes) {
    if (first + r >= p.len[seq]) return;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < parts; ++i) {
      const size_t at = (item + i) * (2 * kRows) + r;
      const float2 ml = p.part_ml[at];
      const float4 v = *(const float4*)(p.part_o + at * D + col);
      const float top = fmaxf(m, ml.x);
      const float a = m == -INFINITY ? 0.f : ex2((m - top) * p.scale2), b = ml.x == -INFINITY ? 0.f : ex2((ml.x - top) * p.scale2);
      l = l * a + ml.y * b;
      o = make_float4(o.x * a + v.x * b, o.y * a + v.y * b, o.z * a + v.z * b, o.w * a + v.w * b);
      m = top;
    }
    const float inv = 1.f / l;
    *(uint2*)(p.out + (size_t)(p.begin[seq] + first + r) * p.out_stride + head * D + col) =
        make_uint2(pack16<kF16>(o.x * inv, o.y * inv), pack16<kF16>(o.z * inv, o.w * inv));
  }
}

// Whether and how the keys are divided: the smallest shares that give no more
// items than SMs, if the longest then is shorter by more than the join costs
// (heads of 128: 5500 tokens of one head 28 instead of 69 us, 2000 of 8 heads
// 24 / 31, 1000 of 4 heads 16.5 / 18.6).
static int attention_parts(AttnParams& p, int sms) {
  auto blocks = [&](int seq, int level) {
    const int left = p.len[seq] - level * 2 * kRows;
    return left > kRows ? 2 * level + 2 : 2 * level + 1;
  };
  auto pairs = [&](int seq) { return (int)((p.len[seq] + 2LL * kRows - 1) / (2 * kRows)); };
  const int most = blocks(0, pairs(0) - 1), limit = std::min(sms, kMaxParts);
  auto lay = [&](int share) {  // the table, or false if there are too many items
    int n = 0, items = 0;
    p.cut_first[0] = 0;
    for (int seq = 0; seq < p.n; ++seq)
      for (int level = 0; level < pairs(seq); ++level) {
        items += (blocks(seq, level) + share - 1) / share * p.Hq;
        if (items > limit) return false;
        p.cut_seq[n] = seq, p.cut_level[n] = level;
        p.cut_first[++n] = items;
      }
    p.cuts = n;
    return true;
  };
  for (int share = 2; share + 3 < most; ++share)
    if (lay(share)) return p.cut_first[p.cuts];
  p.cuts = 0;
  return 0;
}

template <int D, bool kF16>
static cudaError_t launch_attention(const AttnParams& p, long long items, cudaStream_t st) {
  if (p.cuts) {
    k_prompt_attention<D, kF16, true><<<(unsigned)items, kAttnThreads, AttnSmem<D>::kTotal, st>>>(p);
    k_join_parts<D, kF16><<<(unsigned)(p.cuts * p.Hq * 8), 256, 0, st>>>(p);
  } else {
    k_prompt_attention<D, kF16, false><<<(unsigned)items, kAttnThreads, AttnSmem<D>::kTotal, st>>>(p);
  }
  return cudaGetLastError();
}

template <int D, bool kF16>
static cudaError_t configure() {
  constexpr int kSplit = 256 * kRegsSoftmax + 128 * kRegsRest;
  const cudaError_t e = configure_split(k_prompt_attention<D, kF16, false>, kAttnThreads, kSplit, kRegsSoftmax, kRegsRest,
                                        AttnSmem<D>::kTotal);
  return e != cudaSuccess ? e
                          : configure_split(k_prompt_attention<D, kF16, true>, kAttnThreads, kSplit, kRegsSoftmax, kRegsRest,
                                            AttnSmem<D>::kTotal);
}

// Once per device, when a handle is made.
cudaError_t configure_prompt_attention() {
  const cudaError_t e[4] = {configure<128, false>(), configure<128, true>(), configure<64, false>(), configure<64, true>()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

}  // namespace wave

extern "C" int wave_prompt_attention(wave_t* h, int n_seq, const int32_t* cu_seqlens, int n_kv_heads, int type,
                                     const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                     int64_t v_stride, float scale, void* out, int64_t out_stride, void* stream) {
  if (!h || !q || !k || !v || !out || !cu_ok(n_seq, cu_seqlens)) return WAVE_EINVAL;
  const int H = h->pl.cfg.n_heads, D = h->pl.cfg.head_dim;
  if (n_kv_heads < 1 || H % n_kv_heads || (type != WAVE_BF16 && type != WAVE_F16)) return WAVE_EINVAL;
  const float scale2 = scale * 1.44269504088896340736f;  // log2(e)
  if (!(scale > 0.f) || !isfinite(scale2)) return WAVE_EINVAL;
  const int64_t least[4] = {(int64_t)H * D, (int64_t)n_kv_heads * D, (int64_t)n_kv_heads * D, (int64_t)H * D};
  const int64_t strides[4] = {q_stride, k_stride, v_stride, out_stride};
  const void* ptrs[4] = {q, k, v, out};
  for (int i = 0; i < 4; ++i)
    if (strides[i] < least[i] || strides[i] % 8 || strides[i] > kMaxStride || !aligned16(ptrs[i])) return WAVE_EINVAL;
  if (!on_device(h)) return WAVE_EINVAL;
  AttnParams p;
  // the sequences that have tokens, longest first
  int order[WAVE_MAX_SEQS];
  p.n = 0;
  for (int i = 0; i < n_seq; ++i)
    if (cu_seqlens[i + 1] > cu_seqlens[i]) order[p.n++] = i;
  if (!p.n) return WAVE_OK;
  std::stable_sort(order, order + p.n, [&](int a, int b) {
    return cu_seqlens[a + 1] - cu_seqlens[a] > cu_seqlens[b + 1] - cu_seqlens[b];
  });
  long long pairs = 0;
  for (int i = 0; i < p.n; ++i) {
    p.begin[i] = cu_seqlens[order[i]];
    p.len[i] = cu_seqlens[order[i] + 1] - cu_seqlens[order[i]];
    pairs += (p.len[i] + 2LL * kRows - 1) / (2 * kRows);
  }
  const long long rows = cu_seqlens[n_seq];
  if (encode_rows_map(&p.tm_q, q, D, H, rows, q_stride, kRows) ||
      encode_rows_map(&p.tm_k, k, D, n_kv_heads, rows, k_stride, kRows) ||
      encode_rows_map(&p.tm_v, v, D, n_kv_heads, rows, v_stride, kRows))
    return WAVE_ECUDA;
  p.Hq = H;
  p.cuts = 0;
  const int cut = pairs * H <= h->pl.grid ? attention_parts(p, h->pl.grid) : 0;
  const long long items = cut ? cut : pairs * H;
  p.part_o = h->ws.part_o;
  p.part_ml = h->ws.part_ml;
  if (items > 0x7fffffff) return WAVE_EINVAL;
  p.more = items > h->pl.grid;
  p.group = H / n_kv_heads;
  p.v = (const uint16_t*)v;
  p.out = (uint16_t*)out;
  p.v_stride = v_stride;
  p.out_stride = out_stride;
  p.wide = ((uintptr_t)out & 31) == 0 && out_stride % 16 == 0;
  p.scale2 = scale2;
  p.sink = make_sink(h->ws.err, h->err_host_dev, h->timeout_ns);
  p.skip = h->skip_sig_kind == 9 ? h->skip_sig : -1;
  cudaStream_t st = (cudaStream_t)stream;
  h->last_stream = st;
  cudaError_t e;
  if (D == 128)
    e = type == WAVE_F16 ? launch_attention<128, true>(p, items, st) : launch_attention<128, false>(p, items, st);
  else
    e = type == WAVE_F16 ? launch_attention<64, true>(p, items, st) : launch_attention<64, false>(p, items, st);
  return e == cudaSuccess ? WAVE_OK : WAVE_ECUDA;
}
