// history_few.cu -- attention over the 8-bit history for few rows: a frame's
// single tokens, and prompts of so few tokens that a K/V head has at most
// kFewRows rows (tokens times heads of the group), in tiles of 8 or 16.
//
// Bound by HBM: every code is read once for all rows of its K/V head.  The
// keys of all sessions and heads are one line of chunks of 16 tokens, divided
// evenly among the warps of the GPU whatever the lengths, which only the device
// knows in a frame; what a unit (session, head, row tile) has in several warps
// is joined in shared memory, in several CTAs by the last of them to finish.
//
// A chunk's codes are brought into the warp's own ring by cp.async (tokens
// that no row sees as zeros) and become operands of mma.sync in registers, as A
// (16 tokens, or 16 dims), so that eight rows are B's columns and 9 to 16 rows
// two products: S^T = K Q^T, O^T += V^T P^T.  The order of a product's inner
// index is free as long as both operands have it, so that K needs no shuffle:
// lane (g, t) takes 16 bytes of token g, four to an MMA.  V's pairs of tokens
// are made by byte permutes, P is transposed by movmatrix.  The maxima move only
// when a weight would exceed 2^8 of them.  A code is an exact f16; the weights,
// times the V scale of their token, are held in f16 between 2^7 and 2^15 of the
// largest, so that one 2^-31 of it is still there.  bf16 queries are brought to
// f16 by a power of two for each row, which loses nothing above 2^-29 of the
// row's largest value.
//
// Measured (captured launches in a row): a frame of 80 sessions of up to 3000
// tokens, 32/8 heads of 128, blocks of 64, 54.6 us = 4.5 TB/s, of 20 sessions of
// 6000 tokens 46 us = 5.4 TB/s; 56 sessions of up to 1500 tokens, 32 heads, a scale
// for each token, 84 us = 4.25 TB/s; one session of 32001 tokens, 32/8 heads,
// 23.1 us; one after 1500 tokens, 16 x 64, 9.4 us; 25 tokens after 1475, 10.7 us.
// Of some 80,000 cycles of the frame of 80, about 8,000 are the begin (positions,
// the line, first loads) and 9,000 the joins; in the loop between the rate is
// about 5.7 TB/s, what HBM gives.
#include <cuda_runtime.h>
#include <stdint.h>

#include "history_attn.h"

using namespace wave;

namespace wave {

constexpr int kFewChunk = 16;
constexpr float kFewBias = 7.f;  // the largest weight is held as 2^7

// kN: groups of eight rows.  Two take twice the registers: half as many warps.
template <int D, int kN>
struct FewShape {
  static constexpr int kWarps = kN == 1 ? 16 : 8, kThreads = kWarps * 32, kRows = 8 * kN;
  static constexpr int kStages = kN == 1 ? (D == 128 ? 2 : 5) : D == 128 ? 4 : 8;
  static constexpr int kCodes = kFewChunk * D;  // of K, and of V
  static constexpr int kStage = 2 * kCodes + 2 * kFewChunk * 4;
  static constexpr int kRing = kStages * kStage;  // of a warp
  static constexpr int kSums = kRows * (D + 2);   // floats: a unit's sums, then the rows' maxima and sums of weights
  static_assert(kSums * 4 <= kRing, "a warp leaves its last unit's sums in its ring");
  static constexpr int kFirst = kWarps * kRing;   // the sums of the warps' first units, where another warp has a part
  static constexpr int kTotal = kFirst + kWarps * kSums * 4;
  static constexpr int kPart = 2 * kSums;         // of the workspace, for each CTA: two units that other CTAs have a part of
  static_assert(kPart <= 2 * 256 * D, "the workspace of a CTA");
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {  // an 8 x 8 tile of 16-bit values
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Where a chunk of the line lies.
struct FewPlace {
  int seq, unit;      // unit: head * row tiles + row tile
  int chunk, chunks;  // of the unit
  int keys;
};

struct FewTables {
  int first[WAVE_MAX_SEQS + 1];  // chunks before sequence i
  int keys[WAVE_MAX_SEQS];       // what its last token sees
};

// The line's `total` chunks divided evenly, in 32 bits (a 64-bit quotient takes
// 700 cycles).  Not the same number for every warp: with starts a constant
// distance apart the same work took from 87 to 110 us, by that distance.
struct FewDivision {
  int total, parts, share, rest;
  __device__ __forceinline__ FewDivision(int total, int parts)
      : total(total), parts(parts), share(total / parts), rest(total - share * parts) {}
  __device__ __forceinline__ int begin(int part) const { return part * share + part * rest / parts; }  // parts are fewer than 2^15
  __device__ __forceinline__ int part_of(int chunk) const {
    int c = min((int)((float)chunk * ((float)parts / (float)total)), parts - 1);  // off by one at most
    while (begin(c) > chunk) --c;
    while (begin(c + 1) <= chunk) ++c;
    return c;
  }
};

// Row tiles of a K/V head: the same for all of a frame, by a prompt's length.
template <int kR>
__device__ __forceinline__ int tiles_of(const HistoryAttnParams& p, int seq) {
  return p.positions ? p.tiles : (p.b.len(seq) * p.group + kR - 1) / kR;
}

__device__ __forceinline__ FewPlace place_of(const HistoryAttnParams& p, const FewTables& tab, int at) {  // by a whole warp
  const int lane = threadIdx.x & 31;
  int seq = -1;
#pragma unroll
  for (int k = 0; k < WAVE_MAX_SEQS / 32; ++k)
    seq += __popc(__ballot_sync(0xffffffffu, lane + 32 * k < p.n && tab.first[lane + 32 * k] <= at));
  FewPlace w;
  w.seq = seq;
  w.keys = tab.keys[seq];
  w.chunks = (w.keys + kFewChunk - 1) / kFewChunk;
  const int in = at - tab.first[seq];
  w.unit = in / w.chunks;
  w.chunk = in - w.unit * w.chunks;
  return w;
}
// The next chunk of the line, which has one.
template <int kR>
__device__ __forceinline__ void advance(const HistoryAttnParams& p, const FewTables& tab, FewPlace& w) {
  if (++w.chunk < w.chunks) return;
  w.chunk = 0;
  if (++w.unit < p.hist.heads * tiles_of<kR>(p, w.seq)) return;
  w.unit = 0;
  do ++w.seq;
  while (tab.keys[w.seq] == 0);
  w.keys = tab.keys[w.seq];
  w.chunks = (w.keys + kFewChunk - 1) / kFewChunk;
}

// A unit's row r (of the tile): whether there is one, and the row of q
// and out and the head that it is.
struct FewRow {
  bool on;
  int head, keys;
  long long row;
};
template <int kR>
__device__ __forceinline__ FewRow row_of(const HistoryAttnParams& p, const FewPlace& w, int r) {
  const int tiles = tiles_of<kR>(p, w.seq), head = w.unit / tiles, i = (w.unit - head * tiles) * kR + r;
  const int t = i / p.group, len = p.positions ? 1 : p.b.len(w.seq);
  FewRow x;
  x.on = t < len;
  x.head = head * p.group + i - t * p.group;
  x.row = p.positions ? w.seq : p.b.begin[w.seq] + (x.on ? t : 0);
  x.keys = w.keys - (len - 1) + (x.on ? t : 0);
  return x;
}

// Where four of a row's sums are among a unit's: moved about so that lanes meet
// less in a bank.
template <int D>
__device__ __forceinline__ int sums_at(int row, int quad) {
  return row * (D / 4) + (quad ^ (row & 7));
}

template <int D, bool kF16, int kN>
__global__ void __launch_bounds__((FewShape<D, kN>::kThreads), 1) k_history_few(const __grid_constant__ HistoryAttnParams p) {
  using L = FewShape<D, kN>;
  constexpr int kWarps = L::kWarps, kR = L::kRows;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ FewTables tab;
  __shared__ int scan[WAVE_MAX_SEQS / 32];
  // a warp's units that others have a part of: [0] the one that it goes on with, [1] the one that it leaves unfinished
  __shared__ FewPlace open[kWarps][2];
  __shared__ int is_open[kWarps][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  float* part = p.part + (size_t)blockIdx.x * L::kPart;

  // the line: sequences' chunks
  if (threadIdx.x < WAVE_MAX_SEQS) {
    const int s = threadIdx.x;
    int keys = 0, mine = 0;
    if (s < p.n) {
      if (!p.positions) {
        keys = p.b.start[s] + p.b.len(s);
      } else {
        const int pos = p.positions[s];
        keys = pos < 0 ? 0 : pos >= p.hist.T_max ? -1 : pos + 1;
      }
      if (keys > 0) mine = (keys + kFewChunk - 1) / kFewChunk * p.hist.heads * tiles_of<kR>(p, s);
    }
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += v;
    }
    if (lane == 31) scan[warp] = sum;
    tab.first[s + 1] = sum;
    tab.keys[s] = max(keys, 0);
    // a position beyond the history: a zero row, and the error
    if (keys < 0 && blockIdx.x == s % gridDim.x) {
      bad_position(p.err, p.err_out);
      for (int i = 0; i < p.heads * D / 8; ++i) *(uint4*)(p.out + s * p.out_stride + i * 8) = make_uint4(0, 0, 0, 0);
    }
  }
  if (threadIdx.x < 2 * kWarps) is_open[threadIdx.x >> 1][threadIdx.x & 1] = 0;
  if (threadIdx.x == 0) tab.first[0] = 0;
  __syncthreads();
  if (threadIdx.x < WAVE_MAX_SEQS) {
    int before = 0;
    for (int i = 0; i < warp; ++i) before += scan[i];
    tab.first[threadIdx.x + 1] += before;
  }
  __syncthreads();
  const int total = tab.first[p.n];
  if (total == 0) return;
  // no more CTAs than there are chunks for their warps
  int begin, end;
  {
    const int ctas = min((int)gridDim.x, (total + kWarps - 1) / kWarps);
    if ((int)blockIdx.x >= ctas) return;
    const FewDivision line(total, ctas * kWarps);
    begin = line.begin(blockIdx.x * kWarps + warp);
    end = line.begin(blockIdx.x * kWarps + warp + 1);
  }

  const uint32_t ring = smem_u32(smem) + warp * L::kRing;
  uint8_t* ring_p = smem + warp * L::kRing;
  constexpr int kH = D / 64;
  if (begin < end) {
    // ---- the unit at hand; its q is on its way before any key
    FewPlace at = place_of(p, tab, begin);
    uint32_t qb[kN][kH * 4][2];
    float acc[kN][D / 16][4], m[kN][2], e[kN][2], l[kN][2], rf[kN][2];  // of rows 2t, 2t + 1 of each eight
    int limit[kN][2];
    uint4 raw[kN][kH][2];
    auto load_q = [&]() {
#pragma unroll
      for (int b = 0; b < kN; ++b) {
        const FewRow r = row_of<kR>(p, at, 8 * b + g);
        const uint16_t* src = p.q + r.row * p.q_stride + r.head * D + t * 16;
#pragma unroll
        for (int h = 0; h < kH; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i) raw[b][h][i] = r.on ? __ldg((const uint4*)(src + h * 64 + i * 8)) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int x = 0; x < 2; ++x) limit[b][x] = __shfl_sync(0xffffffffu, r.keys, 4 * (2 * t + x));
      }
    };
    auto begin_unit = [&]() {
#pragma unroll
      for (int b = 0; b < kN; ++b) {
        float factor = p.scale2, up = 1.f;
        if constexpr (!kF16) {
          uint32_t top = 0;  // the largest magnitude: bf16 bits compare as integers
#pragma unroll
          for (int h = 0; h < kH; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint4 v = raw[b][h][i];
              top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
            }
          top = max(top & 0xFFFFu, top >> 16);
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int ex = min(max((int)(top >> 7) - 127, -113), 127);  // its exponent
          up = __int_as_float((14 - ex + 127) << 23);
          factor = p.scale2 * (__int_as_float((ex + 127) << 23) * 0x1p-14f);
        }
#pragma unroll
        for (int h = 0; h < kH; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t v[4] = {raw[b][h][i].x, raw[b][h][i].y, raw[b][h][i].z, raw[b][h][i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t z = v[k];
              if constexpr (!kF16) z = half2_of(__uint_as_float(z << 16) * up, __uint_as_float(z & 0xFFFF0000u) * up);
              // word k of 16 bytes: values 2k, 2k + 1 of eight; an MMA takes four values of a lane
              qb[b][h * 4 + i * 2 + (k >> 1)][k & 1] = z;
            }
          }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          rf[b][x] = __shfl_sync(0xffffffffu, factor, 4 * (2 * t + x));
          m[b][x] = e[b][x] = -INFINITY;
          l[b][x] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[b][j][k] = 0.f;
      }
    };
    load_q();

    // ---- copies: chunk by chunk along the line, kStages - 1 ahead
    FewPlace in = at;
    int issued = begin, slot_in = 0;
    const uint8_t *kc = nullptr, *vc = nullptr;
    const float *ks = nullptr, *vs = nullptr;
    auto unit_pointers = [&]() {
      const int slot = p.positions ? in.seq : p.b.slot[in.seq], head = in.unit / tiles_of<kR>(p, in.seq);
      const size_t kr = p.hist.row(0, slot, head), vr = p.hist.row(1, slot, head);
      kc = p.hist.codes + kr * p.hist.T_max * D;
      vc = p.hist.codes + vr * p.hist.T_max * D;
      ks = p.hist.scales + kr * p.hist.blocks;
      vs = p.hist.scales + vr * p.hist.blocks;
    };
    unit_pointers();
    constexpr int kRowPieces = D / 16, kPieces = kFewChunk * kRowPieces / 32;  // 16-byte pieces of a token; a lane's of K or V
    const int prow = lane / kRowPieces, pc = lane % kRowPieces;
    auto issue = [&]() {
      if (issued < end) {
        const uint32_t dst = ring + slot_in * L::kStage;
        const int t0 = in.chunk * kFewChunk;
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
          const int row = prow + k * (32 / kRowPieces);
          const bool there = t0 + row < in.keys;
          const size_t off = there ? (size_t)(t0 + row) * D + pc * 16 : 0;
          int ko, vo;
          if constexpr (D == 128) {
            ko = row * 128 + ((pc ^ (4 * (row & 1))) << 4);
            vo = row * 128 + ((pc ^ (((row >> 1) & 3) << 1)) << 4);
          } else {
            ko = row * 64 + (pc << 4);
            vo = ((row & ~3) | ((row & 1) << 1) | ((row >> 1) & 1)) * 64 + ((pc ^ (((row >> 2) & 1) << 1)) << 4);
          }
          cp16(dst + ko, kc + off, there);
          cp16(dst + L::kCodes + vo, vc + off, there);
        }
        const int tok = t0 + (lane & 15);
        const bool there = tok < in.keys;
        cp4(dst + 2 * L::kCodes + lane * 4, (lane < 16 ? ks : vs) + (there ? tok >> p.hist.shift : 0), there);
        if (++issued < end) {
          const int unit = in.unit, seq = in.seq;
          advance<kR>(p, tab, in);
          if (in.unit != unit || in.seq != seq) {
            unit_pointers();
            // its queries, on their way to L1 while the unit at hand is worked on
#pragma unroll
            for (int b = 0; b < kN; ++b) {
              const FewRow r = row_of<kR>(p, in, 8 * b + g);
              if (r.on && t < kH)
                asm volatile("prefetch.global.L1 [%0];" ::"l"(p.q + r.row * p.q_stride + r.head * D + t * 64));
            }
          }
        }
        if (++slot_in == L::kStages) slot_in = 0;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int i = 0; i < L::kStages - 1; ++i) issue();

    auto weights_of = [&](float sum) {  // over the lanes of a row
#pragma unroll
      for (int d = 4; d <= 16; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      return sum;
    };
    // The sums in the values' own units are times 2^(e - m - bias), which the least
    // scales take below fp32: twice the root of it.
    auto half_unit = [&](int b, int x, float less) { return e[b][x] == -INFINITY ? 0.f : ex2(0.5f * (e[b][x] - m[b][x] - kFewBias - less)); };
    // The unit's rows as sums that others join: divided by a power of two, which goes to the maxima m.
    auto leave_sums = [&](float* dst) {
#pragma unroll
      for (int b = 0; b < kN; ++b)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float sum = weights_of(l[b][x]);
          const int es = exponent_of_sum(sum);
          const float f = half_unit(b, x, (float)es + kPartBias);
          const int row = 8 * b + 2 * t + x;
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            *(float4*)(dst + 4 * sums_at<D>(row, g * (D / 32) + k)) =
                make_float4(f * acc[b][2 * k][x] * f, f * acc[b][2 * k][2 + x] * f, f * acc[b][2 * k + 1][x] * f, f * acc[b][2 * k + 1][2 + x] * f);
          if (g == 0) *(float2*)(dst + kR * D + 2 * row) = make_float2(m[b][x] + (float)es, sum * __int_as_float((127 - es) << 23));
        }
    };
    auto finish_unit = [&]() {
#pragma unroll
      for (int b = 0; b < kN; ++b)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const FewRow r = row_of<kR>(p, at, 8 * b + 2 * t + x);
          const float sum = weights_of(l[b][x]);
          if (!r.on) continue;
          const float f = half_unit(b, x, 0.f), inv = f / sum;
          uint16_t* dst = p.out + r.row * p.out_stride + r.head * D + g * (D / 8);
#pragma unroll
          for (int k = 0; k < D / 64; ++k) {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float u = acc[b][4 * k + i][x] * inv * f, v = acc[b][4 * k + i][2 + x] * inv * f;
              o[i] = kF16 ? pair16<__half>(u, v) : pair16<__nv_bfloat16>(u, v);
            }
            *(uint4*)(dst + 8 * k) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
    };

    int slot = 0;
    bool fresh = true, started = false;
    for (int c = begin; c < end; ++c) {
      if (fresh) {
        if (c > begin) load_q();
        begin_unit();
        fresh = false;
        started = at.chunk == 0;
      }
      asm volatile("cp.async.wait_group %0;" ::"n"(L::kStages - 2) : "memory");
      __syncwarp();
      issue();  // into the stage that was read last
      const uint8_t* st = ring_p + slot * L::kStage;
      if (++slot == L::kStages) slot = 0;
      const float* sc = (const float*)(st + 2 * L::kCodes);

      float s[kN][4] = {};
#pragma unroll
      for (int h = 0; h < kH; ++h) {
        const int off = D == 128 ? g * 128 + (((t + 4 * h) ^ (4 * (g & 1))) << 4) : g * 64 + (t << 4);
        const uint4 lo = *(const uint4*)(st + off), hi = *(const uint4*)(st + off + 8 * D);  // tokens g and g + 8
        const uint32_t lw[4] = {lo.x, lo.y, lo.z, lo.w}, hw[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_f16x2x2(lw[j], a0, a2);
          e4m3x4_to_f16x2x2(hw[j], a1, a3);
#pragma unroll
          for (int b = 0; b < kN; ++b) mma_f16_16816(s[b], a0, a1, a2, a3, qb[b][h * 4 + j][0], qb[b][h * 4 + j][1]);
        }
      }
      const float k0 = sc[g], k1 = sc[g + 8], lv0 = lg2(sc[16 + g]), lv1 = lg2(sc[24 + g]);
      const int t0 = at.chunk * kFewChunk;
      const bool cut = __any_sync(0xffffffffu, t0 + kFewChunk > limit[0][0]);  // some row does not see all of the chunk
      float top[kN][2], etop[kN][2];
      bool up = false;
#pragma unroll
      for (int b = 0; b < kN; ++b)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          s[b][x] *= k0 * rf[b][x];
          s[b][2 + x] *= k1 * rf[b][x];
          if (cut) {
            if (t0 + g >= limit[b][x]) s[b][x] = -INFINITY;
            if (t0 + g + 8 >= limit[b][x]) s[b][2 + x] = -INFINITY;
          }
          top[b][x] = fmaxf(s[b][x], s[b][2 + x]);
          etop[b][x] = fmaxf(s[b][x] + lv0, s[b][2 + x] + lv1);
          up |= top[b][x] > m[b][x] + 8.f || etop[b][x] > e[b][x] + 8.f;
        }
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int b = 0; b < kN; ++b)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int d = 4; d <= 16; d <<= 1) {
              top[b][x] = fmaxf(top[b][x], __shfl_xor_sync(0xffffffffu, top[b][x], d));
              etop[b][x] = fmaxf(etop[b][x], __shfl_xor_sync(0xffffffffu, etop[b][x], d));
            }
            const float m2 = fmaxf(m[b][x], top[b][x]), e2 = fmaxf(e[b][x], etop[b][x]);
            l[b][x] *= m[b][x] == -INFINITY ? 0.f : ex2(m[b][x] - m2);
            const float a = e[b][x] == -INFINITY ? 0.f : ex2(e[b][x] - e2);
            m[b][x] = m2;
            e[b][x] = e2;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              acc[b][j][x] *= a;
              acc[b][j][2 + x] *= a;
            }
          }
      }
      uint32_t pb[kN][2];
#pragma unroll
      for (int b = 0; b < kN; ++b) {
        float wt[4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float mm = m[b][x] == -INFINITY ? 0.f : m[b][x], ee = (e[b][x] == -INFINITY ? 0.f : e[b][x]) - kFewBias;
          l[b][x] += ex2(s[b][x] - mm) + ex2(s[b][2 + x] - mm);
          wt[x] = ex2(s[b][x] + (lv0 - ee));
          wt[2 + x] = ex2(s[b][2 + x] + (lv1 - ee));
          if (cut) {  // a scale behind a row's end counts for nothing there, whatever it is
            wt[x] = s[b][x] == -INFINITY ? 0.f : wt[x];
            wt[2 + x] = s[b][2 + x] == -INFINITY ? 0.f : wt[2 + x];
          }
        }
        pb[b][0] = transpose8(half2_of(wt[0], wt[1]));
        pb[b][1] = transpose8(half2_of(wt[2], wt[3]));
      }
      // V: the lane's D / 8 bytes of tokens 2t, 2t + 1, 2t + 8, 2t + 9
      constexpr int kWords = D / 32;
      uint32_t v[4][kWords];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 2 * t + (i & 1) + 8 * (i >> 1);
        if constexpr (D == 128) {
          const uint4 x = *(const uint4*)(st + L::kCodes + row * 128 + ((g ^ (((row >> 1) & 3) << 1)) << 4));
          v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
        } else {
          const uint2 x = *(const uint2*)(st + L::kCodes + ((row & ~3) | ((row & 1) << 1) | ((row >> 1) & 1)) * 64 +
                                          (((g >> 1) ^ (((row >> 2) & 1) << 1)) << 4) + (g & 1) * 8);
          v[i][0] = x.x, v[i][1] = x.y;
        }
      }
      bool odd = false;  // NaN among values that some row does not see: 0 x NaN would reach it
      if (cut) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < kWords; ++k) odd |= any_nan_code(v[i][k]);
        odd = __any_sync(0xffffffffu, odd);
        if (odd) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < kWords; ++k)
#pragma unroll
              for (int b = 0; b < 4; ++b)
                if ((v[i][k] >> (8 * b) & 0x7F) == 0x7F) v[i][k] &= ~(0xFFu << (8 * b));
        }
      }
#pragma unroll
      for (int k = 0; k < kWords; ++k) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {  // bytes 0, 1 and 2, 3 of a word: dims 4 k + 2 y, 4 k + 2 y + 1 of the lane's
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_f16x2x2(prmt(v[0][k], v[1][k], y ? 0x7362 : 0x5140), a0, a1);
          e4m3x4_to_f16x2x2(prmt(v[2][k], v[3][k], y ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
          for (int b = 0; b < kN; ++b) mma_f16_16816(acc[b][2 * k + y], a0, a1, a2, a3, pb[b][0], pb[b][1]);
        }
      }
      if (odd) {  // the rows that see them get NaN
#pragma unroll 1
        for (int row = 0; row < kFewChunk; ++row) {
          uint32_t bad = 0;  // of the lane's D / 8 values
#pragma unroll 1
          for (int d = 0; d < D / 8; ++d) {
            const int dim = g * (D / 8) + d, c16 = dim >> 4;
            const int o = D == 128 ? row * 128 + ((c16 ^ (((row >> 1) & 3) << 1)) << 4)
                                   : ((row & ~3) | ((row & 1) << 1) | ((row >> 1) & 1)) * 64 + ((c16 ^ (((row >> 2) & 1) << 1)) << 4);
            if ((st[L::kCodes + o + (dim & 15)] & 0x7F) == 0x7F) bad |= 1u << d;
          }
#pragma unroll
          for (int b = 0; b < kN; ++b)
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int d = 0; d < D / 8; ++d)
                if ((bad >> d & 1) && t0 + row < limit[b][x]) acc[b][d / 2][2 * (d & 1) + x] = __int_as_float(0x7FC00000);
        }
      }
      __syncwarp();
      const bool ends = at.chunk + 1 == at.chunks;
      if (ends || c + 1 == end) {
        if (started && ends) {
          finish_unit();
        } else {
          if (c + 1 == end) asm volatile("cp.async.wait_group 0;" ::: "memory");
          __syncwarp();
          leave_sums((float*)(started ? ring_p : smem + L::kFirst + warp * L::kSums * 4));
          if (lane == 0) {
            open[warp][started] = at;
            is_open[warp][started] = 1;
          }
        }
        fresh = true;
      }
      if (c + 1 < end) advance<kR>(p, tab, at);
    }
  }

  // ---- units in several warps: a CTA's chains of sums.  A warp joins a fourth of
  // a chain's rows; where other CTAs have a part of the unit it leaves what it
  // has for the last of them.
  __syncthreads();
  const int chunks = tab.first[p.n];  // read again: registers are scarce in between
  const FewDivision line(chunks, min((int)gridDim.x, (chunks + kWarps - 1) / kWarps));  // among CTAs: the same
  const int cta_begin = line.begin(blockIdx.x), cta_end = line.begin(blockIdx.x + 1);
  constexpr int kQuads = kR * D / 4, kEach = kQuads / 4 / 32;  // four sums at a time: of a unit, and of a lane
  // the open units in the line's order, and where chains begin
  uint32_t opens, starts;
  {
    const bool there = lane < 2 * kWarps && is_open[(lane >> 1) % kWarps][lane & 1];
    opens = __ballot_sync(0xffffffffu, there);
    const uint32_t before = opens & ((1u << lane) - 1);
    bool first = there;
    if (there && before) {
      const int b = 31 - __clz(before);
      const FewPlace &x = open[b >> 1][b & 1], &y = open[lane >> 1][lane & 1];
      first = x.seq != y.seq || x.unit != y.unit;
    }
    starts = __ballot_sync(0xffffffffu, first);
  }
  for (int task = warp; task < 4 * __popc(starts); task += kWarps) {
    uint32_t rest = starts;
    for (int i = 0; i < task / 4; ++i) rest &= rest - 1;
    const int start = __ffs(rest) - 1;
    rest &= rest - 1;
    uint32_t chain = opens & ~((1u << start) - 1) & (rest ? (1u << (__ffs(rest) - 1)) - 1 : 0xffffffffu);
    const FewPlace u = open[start >> 1][start & 1];
    const int u0 = tab.first[u.seq] + u.unit * u.chunks, u1 = u0 + u.chunks;  // the unit's part of the line
    const int q0 = (task & 3) * (kQuads / 4) + lane;
    float4 o[kEach];
    float mx[kEach], lx[kEach];
    auto clear = [&]() {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        mx[i] = -INFINITY;
        lx[i] = 0.f;
      }
    };
    auto add = [&](int i, float2 ml, float4 v) {
      const float top = fmaxf(mx[i], ml.x);
      const float a = mx[i] == -INFINITY ? 0.f : ex2(mx[i] - top), b = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);
      lx[i] = lx[i] * a + ml.y * b;
      o[i] = make_float4(o[i].x * a + v.x * b, o[i].y * a + v.y * b, o[i].z * a + v.z * b, o[i].w * a + v.w * b);
      mx[i] = top;
    };
    constexpr int kBatch = 4;  // sums whose loads are in flight together
    clear();
    while (chain) {
      float2 ml[kBatch][kEach];
      float4 v[kBatch][kEach];
#pragma unroll
      for (int f = 0; f < kBatch; ++f) {
        const int j = chain ? __ffs(chain) - 1 : -1;
        chain &= chain - 1;  // 0 stays 0
        const float* src = (const float*)(smem + (j & 1 ? (j >> 1) * L::kRing : L::kFirst + (j >> 1) * L::kSums * 4));
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const int row = (q0 + 32 * i) / (D / 4), quad = (q0 + 32 * i) % (D / 4);
          ml[f][i] = j < 0 ? make_float2(-INFINITY, 0.f) : *(const float2*)(src + kR * D + 2 * row);
          v[f][i] = j < 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : *(const float4*)(src + 4 * sums_at<D>(row, quad));
        }
      }
#pragma unroll
      for (int f = 0; f < kBatch; ++f)
#pragma unroll
        for (int i = 0; i < kEach; ++i) add(i, ml[f][i], v[f][i]);
    }
    bool write = u0 >= cta_begin && u1 <= cta_end;
    if (!write) {
      const int c0 = line.part_of(u0), c1 = line.part_of(u1 - 1);
      float* dst = part + (u0 >= cta_begin ? L::kSums : 0);
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int q = q0 + 32 * i;
        __stcg((float4*)dst + q, o[i]);
        if (q % (D / 4) == 0) __stcg((float2*)(dst + kR * D) + q / (D / 4), make_float2(mx[i], lx[i]));
      }
      __threadfence();
      __syncwarp();
      int* cnt = p.part_cnt + (u.seq * (kFewTiles * p.heads) + u.unit) * 4 + (task & 3);
      int there = 0;
      if (lane == 0) there = atomicAdd(cnt, 1);
      write = __shfl_sync(0xffffffffu, there, 0) == c1 - c0;
      if (write) {
        __threadfence();
        if (lane == 0) *cnt = 0;  // for the next launch
        clear();
        constexpr int kFar = 16 / kEach;
        for (int c = c0; c <= c1; c += kFar) {
          float2 ml[kFar][kEach];
          float4 v[kFar][kEach];
#pragma unroll
          for (int f = 0; f < kFar; ++f) {
            const float* src = p.part + (size_t)min(c + f, c1) * L::kPart + (c + f == c0 ? L::kSums : 0);
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
              ml[f][i] = __ldcg((const float2*)(src + kR * D) + (q0 + 32 * i) / (D / 4));
              v[f][i] = __ldcg((const float4*)src + q0 + 32 * i);
              if (c + f > c1) ml[f][i].x = -INFINITY;
            }
          }
#pragma unroll
          for (int f = 0; f < kFar; ++f)
#pragma unroll
            for (int i = 0; i < kEach; ++i)
              if (c + f <= c1) add(i, ml[f][i], v[f][i]);
        }
      }
    }
    if (write) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int row = (q0 + 32 * i) / (D / 4), quad = (q0 + 32 * i) % (D / 4);
        const FewRow r = row_of<kR>(p, u, row);
        if (!r.on) continue;
        const float inv = joined_factor(lx[i]);
        *(uint2*)(p.out + r.row * p.out_stride + r.head * D + 4 * quad) =
            kF16 ? make_uint2(pair16<__half>(o[i].x * inv, o[i].y * inv), pair16<__half>(o[i].z * inv, o[i].w * inv))
                 : make_uint2(pair16<__nv_bfloat16>(o[i].x * inv, o[i].y * inv), pair16<__nv_bfloat16>(o[i].z * inv, o[i].w * inv));
      }
    }
  }
}

template <int D, bool kF16, int kN>
static cudaError_t configure() {
  return cudaFuncSetAttribute(k_history_few<D, kF16, kN>, cudaFuncAttributeMaxDynamicSharedMemorySize, FewShape<D, kN>::kTotal);
}

cudaError_t configure_history_few() {
  const cudaError_t e[8] = {configure<128, false, 1>(), configure<128, false, 2>(), configure<128, true, 1>(), configure<128, true, 2>(),
                            configure<64, false, 1>(),  configure<64, false, 2>(),  configure<64, true, 1>(),  configure<64, true, 2>()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

template <int D, bool kF16>
static cudaError_t launch(HistoryAttnParams& p, int rows, int sms, cudaStream_t st) {
  const int tile = rows <= 8 ? 8 : kFewTile;
  p.tiles = (p.group + tile - 1) / tile;  // a frame's
  if (tile == 8)
    k_history_few<D, kF16, 1><<<sms, FewShape<D, 1>::kThreads, FewShape<D, 1>::kTotal, st>>>(p);
  else
    k_history_few<D, kF16, 2><<<sms, FewShape<D, 2>::kThreads, FewShape<D, 2>::kTotal, st>>>(p);
  return cudaGetLastError();
}

// rows: the most that a session has for a K/V head.
cudaError_t launch_history_few(HistoryAttnParams& p, int D, int type, int rows, int sms, cudaStream_t st) {
  if (D == 128) return type == WAVE_F16 ? launch<128, true>(p, rows, sms, st) : launch<128, false>(p, rows, sms, st);
  return type == WAVE_F16 ? launch<64, true>(p, rows, sms, st) : launch<64, false>(p, rows, sms, st);
}

}  // namespace wave
