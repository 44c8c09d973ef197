// history_few.cu -- attention over the 8-bit history for few rows: a frame's
// single tokens, and prompts of so few tokens that their heads' rows fit one
// tile of 16.
//
// Bound by HBM: every code is read once for all rows of its K/V head.  The
// keys of all sessions and heads are one line of chunks of 16 tokens, divided
// evenly among the warps of the GPU whatever the lengths, which only the device
// knows in a frame; what a unit (session, head, 16 rows) has in several warps
// is joined in shared memory, in several CTAs by the last of them to finish.
//
// A chunk's codes are brought into the warp's own ring by cp.async (tokens
// that no row sees as zeros) and become operands of mma.sync in registers:
// S = Q K^T with Q's 16 rows as A and eight tokens as B's columns, O += P V with
// S's registers as A.  The order of a product's inner index is free as long as
// both operands have it, so that K needs no shuffle: lane (g, t) takes 16
// bytes of token g, four to an MMA.  V's pairs of tokens are made by byte
// permutes.  The maxima move only when a weight would exceed 2^8 of them.  A
// code is an exact f16; the weights, times the V scale of their token, are held
// in f16 between 2^7 and 2^15 of the largest, so that one 2^-31 of it is still
// there.  bf16 queries are brought to f16 by a power of two for each row, which
// loses nothing above 2^-29 of the row's largest value.
#include <cuda_runtime.h>
#include <stdint.h>

#include "history_attn.h"

using namespace wave;

namespace wave {

constexpr int kFewWarps = 8, kFewThreads = kFewWarps * 32, kFewChunk = 16;
constexpr float kFewBias = 7.f;  // the largest weight is held as 2^7

template <int D>
struct FewSmem {
  static constexpr int kStages = 4;
  static constexpr int kCodes = kFewChunk * D;       // of K, and of V
  static constexpr int kStage = 2 * kCodes + 2 * kFewChunk * 4;
  static constexpr int kRing = kStages * kStage;     // of a warp
  static constexpr int kSums = kFewRows * (D + 2) * 4;
  static_assert(kSums <= kRing, "a warp leaves its last unit's sums in its ring");
  static constexpr int kFirst = kFewWarps * kRing;   // the warps' first units' sums
  static constexpr int kTotal = kFirst + kFewWarps * kSums;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ bool any_nan_code(uint32_t w) { return (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0; }

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

__device__ __forceinline__ int row_tiles(const HistoryAttnParams& p, int seq) {
  return ((p.positions ? 1 : p.b.len(seq)) * p.group + kFewRows - 1) / kFewRows;
}

__device__ __forceinline__ FewPlace place_of(const HistoryAttnParams& p, const FewTables& tab, int at) {
  int lo = 0, hi = p.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.first[mid] <= at)
      lo = mid;
    else
      hi = mid - 1;
  }
  FewPlace w;
  w.seq = lo;
  w.keys = tab.keys[lo];
  w.chunks = (w.keys + kFewChunk - 1) / kFewChunk;
  const int in = at - tab.first[lo];
  w.unit = in / w.chunks;
  w.chunk = in - w.unit * w.chunks;
  return w;
}
// The next chunk of the line, which has one.
__device__ __forceinline__ void advance(const HistoryAttnParams& p, const FewTables& tab, FewPlace& w) {
  if (++w.chunk < w.chunks) return;
  w.chunk = 0;
  if (++w.unit < p.hist.heads * row_tiles(p, w.seq)) return;
  w.unit = 0;
  do ++w.seq;
  while (tab.keys[w.seq] == 0);
  w.keys = tab.keys[w.seq];
  w.chunks = (w.keys + kFewChunk - 1) / kFewChunk;
}

// A unit's row r (0..15 of the tile): whether there is one, and the row of q
// and out and the head that it is.
struct FewRow {
  bool on;
  int head, keys;
  long long row;
};
__device__ __forceinline__ FewRow row_of(const HistoryAttnParams& p, const FewPlace& w, int r) {
  const int tiles = row_tiles(p, w.seq), head = w.unit / tiles, i = (w.unit - head * tiles) * kFewRows + r;
  const int t = i / p.group, len = p.positions ? 1 : p.b.len(w.seq);
  FewRow x;
  x.on = t < len;
  x.head = head * p.group + i - t * p.group;
  x.row = p.positions ? w.seq : p.b.begin[w.seq] + (x.on ? t : 0);
  x.keys = w.keys - (len - 1) + (x.on ? t : 0);
  return x;
}

// Sums of a unit in shared memory: [16 rows][D], then the rows' maxima and
// sums of weights.  The four values of a row that a lane writes together are
// moved about so that lanes do not meet in a bank.
template <int D>
__device__ __forceinline__ int sums_at(int row, int quad) {
  constexpr int kQuads = D / 16;  // of a lane
  const int t = quad / kQuads, k = quad % kQuads;
  return row * (D / 4) + t * kQuads + (k ^ ((2 * t + (row & 1)) & (kQuads - 1)));
}

template <int D, bool kF16>
__global__ void __launch_bounds__(kFewThreads, 1) k_history_few(const __grid_constant__ HistoryAttnParams p) {
  using L = FewSmem<D>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ FewTables tab;
  __shared__ int scan[WAVE_MAX_SEQS / 32];
  // a warp's units that others have a part of: [0] the one that it goes on with, [1] the one that it leaves unfinished
  __shared__ FewPlace open[kFewWarps][2];
  __shared__ int is_open[kFewWarps][2], last_cta;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

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
      if (keys > 0) mine = (keys + kFewChunk - 1) / kFewChunk * p.hist.heads * row_tiles(p, s);
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
  if (threadIdx.x < 2 * kFewWarps) is_open[threadIdx.x >> 1][threadIdx.x & 1] = 0;
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
  // CTAs: no more than there are chunks for their warps
  const int ctas = min((int)gridDim.x, (total + kFewWarps - 1) / kFewWarps);
  if ((int)blockIdx.x >= ctas) return;
  const int w = blockIdx.x * kFewWarps + warp;
  const int begin = (int)((long long)total * w / (ctas * kFewWarps)), end = (int)((long long)total * (w + 1) / (ctas * kFewWarps));

  const uint32_t ring = smem_u32(smem) + warp * L::kRing;
  uint8_t* ring_p = smem + warp * L::kRing;
  constexpr int kH = D / 64;
  if (begin < end) {
    // ---- copies: chunk by chunk along the line, kStages - 1 ahead
    FewPlace in = place_of(p, tab, begin);
    int issued = begin, slot_in = 0;
    const uint8_t *kc = nullptr, *vc = nullptr;
    const float *ks = nullptr, *vs = nullptr;
    auto unit_pointers = [&]() {
      const int slot = p.positions ? in.seq : p.b.slot[in.seq], head = in.unit / row_tiles(p, in.seq);
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
          advance(p, tab, in);
          if (in.unit != unit || in.seq != seq) unit_pointers();
        }
        if (++slot_in == L::kStages) slot_in = 0;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < L::kStages - 1; ++i) issue();

    // ---- the unit at hand
    FewPlace at = place_of(p, tab, begin);
    uint32_t qa[kH * 4][4];
    float acc[D / 8][4], m[2], e[2], l[2], rf[2];
    int limit[2];
    auto begin_unit = [&]() {
      uint4 raw[2][kH][2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const FewRow r = row_of(p, at, g + 8 * x);
        limit[x] = r.keys;
        const uint16_t* src = p.q + r.row * p.q_stride + r.head * D + t * 16;
#pragma unroll
        for (int h = 0; h < kH; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i) raw[x][h][i] = r.on ? __ldg((const uint4*)(src + h * 64 + i * 8)) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        rf[x] = p.scale2;
        float up = 1.f;
        if constexpr (!kF16) {
          uint32_t top = 0;  // the largest magnitude: bf16 bits compare as integers
#pragma unroll
          for (int h = 0; h < kH; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint4 v = raw[x][h][i];
              top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
            }
          top = max(top & 0xFFFFu, top >> 16);
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int ex = min(max((int)(top >> 7) - 127, -113), 127);  // its exponent
          up = __int_as_float((14 - ex + 127) << 23);
          rf[x] = p.scale2 * __int_as_float((ex + 127) << 23) * 0x1p-14f;
        }
#pragma unroll
        for (int h = 0; h < kH; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t v[4] = {raw[x][h][i].x, raw[x][h][i].y, raw[x][h][i].z, raw[x][h][i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t z = v[k];
              if constexpr (!kF16) z = half2_of(__uint_as_float(z << 16) * up, __uint_as_float(z & 0xFFFF0000u) * up);
              // word k of 16 bytes: values 2k, 2k + 1 of eight; an MMA takes four values of a lane
              qa[h * 4 + i * 2 + (k >> 1)][(k & 1) * 2 + x] = z;
            }
          }
        m[x] = e[x] = -INFINITY;
        l[x] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[j][k] = 0.f;
    };
    // The unit's rows as sums that others join: divided by nothing, relative to the maxima m.
    auto leave_sums = [&](float* dst) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float sum = l[x];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const float f = e[x] == -INFINITY ? 0.f : ex2(e[x] - m[x] - kFewBias);
        const int row = g + 8 * x;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          float v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int d = 4 * k + i;  // of the lane's D / 4 values
            v[i] = f * acc[d % (D / 8)][2 * x + d / (D / 8)];
          }
          *(float4*)(dst + 4 * sums_at<D>(row, t * (D / 16) + k)) = make_float4(v[0], v[1], v[2], v[3]);
        }
        if (t == 0) *(float2*)(dst + kFewRows * D + 2 * row) = make_float2(m[x], sum);
      }
    };
    auto finish_unit = [&]() {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const FewRow r = row_of(p, at, g + 8 * x);
        float sum = l[x];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (!r.on) continue;
        const float f = e[x] == -INFINITY ? 0.f : ex2(e[x] - m[x] - kFewBias), inv = f / sum;
        uint16_t* dst = p.out + r.row * p.out_stride + r.head * D + t * (D / 4);
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int d = 8 * k + 2 * i;
            const float a = acc[d % (D / 8)][2 * x + d / (D / 8)] * inv, b = acc[(d + 1) % (D / 8)][2 * x + d / (D / 8)] * inv;
            o[i] = kF16 ? pair16<__half>(a, b) : pair16<__nv_bfloat16>(a, b);
          }
          *(uint4*)(dst + 8 * k) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    };

    int slot = 0;
    bool fresh = true, started = false;
    for (int c = begin; c < end; ++c) {
      if (fresh) {
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

      float s[2][4] = {};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int h = 0; h < kH; ++h) {
          const int row = 8 * i + g;
          const uint4 k4 = *(const uint4*)(st + (D == 128 ? row * 128 + (((t + 4 * h) ^ (4 * (row & 1))) << 4) : row * 64 + (t << 4)));
          const uint32_t kw[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t b0, b1;
            e4m3x4_to_f16x2x2(kw[j], b0, b1);
            mma_f16_16816(s[i], qa[h * 4 + j][0], qa[h * 4 + j][1], qa[h * 4 + j][2], qa[h * 4 + j][3], b0, b1);
          }
        }
      }
      float lv[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 k2 = *(const float2*)(sc + 8 * i + 2 * t), v2 = *(const float2*)(sc + 16 + 8 * i + 2 * t);
        lv[2 * i] = lg2(v2.x);
        lv[2 * i + 1] = lg2(v2.y);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          s[i][2 * x] *= k2.x * rf[x];
          s[i][2 * x + 1] *= k2.y * rf[x];
        }
      }
      const int t0 = at.chunk * kFewChunk;
      const bool cut = __any_sync(0xffffffffu, t0 + kFewChunk > limit[0]);  // some row does not see all of the chunk
      if (cut) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (t0 + 8 * i + 2 * t + (k & 1) >= limit[k >> 1]) s[i][k] = -INFINITY;
      }
      float top[2], etop[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        top[x] = fmaxf(fmaxf(s[0][2 * x], s[0][2 * x + 1]), fmaxf(s[1][2 * x], s[1][2 * x + 1]));
        etop[x] = fmaxf(fmaxf(s[0][2 * x] + lv[0], s[0][2 * x + 1] + lv[1]), fmaxf(s[1][2 * x] + lv[2], s[1][2 * x + 1] + lv[3]));
      }
      const bool up = top[0] > m[0] + 8.f || top[1] > m[1] + 8.f || etop[0] > e[0] + 8.f || etop[1] > e[1] + 8.f;
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
          for (int d = 1; d <= 2; d <<= 1) {
            top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], d));
            etop[x] = fmaxf(etop[x], __shfl_xor_sync(0xffffffffu, etop[x], d));
          }
          const float m2 = fmaxf(m[x], top[x]), e2 = fmaxf(e[x], etop[x]);
          l[x] *= m[x] == -INFINITY ? 0.f : ex2(m[x] - m2);
          const float a = e[x] == -INFINITY ? 0.f : ex2(e[x] - e2);
          m[x] = m2;
          e[x] = e2;
#pragma unroll
          for (int j = 0; j < D / 8; ++j) {
            acc[j][2 * x] *= a;
            acc[j][2 * x + 1] *= a;
          }
        }
      }
      uint32_t pa[4];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float mm = m[x] == -INFINITY ? 0.f : m[x], ee = (e[x] == -INFINITY ? 0.f : e[x]) - kFewBias;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float a = s[i][2 * x], b = s[i][2 * x + 1];
          l[x] += ex2(a - mm) + ex2(b - mm);
          float wa = ex2(a + (lv[2 * i] - ee)), wb = ex2(b + (lv[2 * i + 1] - ee));
          if (cut) {  // a scale behind a row's end counts for nothing there, whatever it is
            wa = a == -INFINITY ? 0.f : wa;
            wb = b == -INFINITY ? 0.f : wb;
          }
          pa[2 * i + x] = half2_of(wa, wb);
        }
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
        const uint32_t x0 = prmt(v[0][k], v[1][k], 0x5140), y0 = prmt(v[0][k], v[1][k], 0x7362);
        const uint32_t x1 = prmt(v[2][k], v[3][k], 0x5140), y1 = prmt(v[2][k], v[3][k], 0x7362);
        uint32_t a0, a1, b0, b1;
        e4m3x4_to_f16x2x2(x0, a0, a1);
        e4m3x4_to_f16x2x2(x1, b0, b1);
        mma_f16_16816(acc[4 * k], pa[0], pa[1], pa[2], pa[3], a0, b0);
        mma_f16_16816(acc[4 * k + 1], pa[0], pa[1], pa[2], pa[3], a1, b1);
        e4m3x4_to_f16x2x2(y0, a0, a1);
        e4m3x4_to_f16x2x2(y1, b0, b1);
        mma_f16_16816(acc[4 * k + 2], pa[0], pa[1], pa[2], pa[3], a0, b0);
        mma_f16_16816(acc[4 * k + 3], pa[0], pa[1], pa[2], pa[3], a1, b1);
      }
      if (odd) {  // the rows that see them get NaN
#pragma unroll 1
        for (int row = 0; row < kFewChunk; ++row) {
          // the lane's sums: values t D / 4 .. of its rows
          uint32_t bad = 0;  // by value
#pragma unroll
          for (int d = 0; d < D / 4; ++d) {
            const int dim = t * (D / 4) + d, pc16 = dim >> 4;
            const int o = D == 128 ? row * 128 + ((pc16 ^ (((row >> 1) & 3) << 1)) << 4)
                                   : ((row & ~3) | ((row & 1) << 1) | ((row >> 1) & 1)) * 64 + ((pc16 ^ (((row >> 2) & 1) << 1)) << 4);
            if ((st[L::kCodes + o + (dim & 15)] & 0x7F) == 0x7F) bad |= 1u << d;
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (t0 + row >= limit[x]) continue;
#pragma unroll
            for (int d = 0; d < D / 4; ++d)
              if (bad >> d & 1) acc[d % (D / 8)][2 * x + d / (D / 8)] = __int_as_float(0x7FC00000);
          }
        }
      }
      __syncwarp();
      const bool ends = at.chunk + 1 == at.chunks;
      if (ends || c + 1 == end) {
        if (started && ends) {
          finish_unit();
        } else {
          if (c + 1 == end) asm volatile("cp.async.wait_group 0;" ::: "memory");
          leave_sums(started ? (float*)ring_p : (float*)(smem + L::kFirst + warp * L::kSums));
          if (lane == 0) {
            open[warp][started] = at;
            is_open[warp][started] = 1;
          }
        }
        fresh = true;
      }
      if (c + 1 < end) advance(p, tab, at);
    }
  }

  // ---- units in several warps: a chain of a CTA's sums, joined by all its threads
  __syncthreads();
  const int cta_begin = (int)((long long)total * blockIdx.x / ctas), cta_end = (int)((long long)total * (blockIdx.x + 1) / ctas);
  constexpr int kQuads = kFewRows * D / 4, kEach = kQuads / kFewThreads;
  for (int k = 0; k < 2 * kFewWarps;) {  // the warps' open units in the line's order
    if (!is_open[k >> 1][k & 1]) {
      ++k;
      continue;
    }
    const FewPlace u = open[k >> 1][k & 1];
    int last = k + 1;
    while (last < 2 * kFewWarps && (!is_open[last >> 1][last & 1] ||
                                    (open[last >> 1][last & 1].seq == u.seq && open[last >> 1][last & 1].unit == u.unit)))
      ++last;
    const int u0 = tab.first[u.seq] + u.unit * u.chunks, u1 = u0 + u.chunks;  // the unit's part of the line
    const bool here = u0 >= cta_begin && u1 <= cta_end;
    float4 o[kEach];
    float mx[kEach], lx[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int q = threadIdx.x + i * kFewThreads, row = q / (D / 4), quad = q % (D / 4);
      o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      mx[i] = -INFINITY;
      lx[i] = 0.f;
      for (int j = k; j < last; ++j) {
        if (!is_open[j >> 1][j & 1]) continue;
        const float* src = (const float*)(smem + (j & 1 ? (j >> 1) * L::kRing : L::kFirst + (j >> 1) * L::kSums));
        const float2 ml = *(const float2*)(src + kFewRows * D + 2 * row);
        const float4 v = *(const float4*)(src + 4 * sums_at<D>(row, quad));
        const float top = fmaxf(mx[i], ml.x);
        const float a = mx[i] == -INFINITY ? 0.f : ex2(mx[i] - top), b = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);
        lx[i] = lx[i] * a + ml.y * b;
        o[i] = make_float4(o[i].x * a + v.x * b, o[i].y * a + v.y * b, o[i].z * a + v.z * b, o[i].w * a + v.w * b);
        mx[i] = top;
      }
    }
    bool write = here;
    if (!here) {
      const int c0 = (int)(((long long)(u0 + 1) * ctas - 1) / total), c1 = (int)(((long long)u1 * ctas - 1) / total);
      const size_t floats = kFewRows * (D + 2);
      float* dst = p.part + ((size_t)blockIdx.x * 2 + (u0 >= cta_begin)) * floats;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int q = threadIdx.x + i * kFewThreads, row = q / (D / 4), quad = q % (D / 4);
        __stcg((float4*)dst + q, o[i]);
        if (quad == 0) __stcg((float2*)(dst + kFewRows * D) + row, make_float2(mx[i], lx[i]));
      }
      __threadfence();
      __syncthreads();
      int* cnt = p.part_cnt + u.seq * p.heads + u.unit;
      if (threadIdx.x == 0) last_cta = atomicAdd(cnt, 1) == c1 - c0;
      __syncthreads();
      write = last_cta;
      __syncthreads();
      if (write) {
        __threadfence();
        if (threadIdx.x == 0) *cnt = 0;  // for the next launch
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const int q = threadIdx.x + i * kFewThreads, row = q / (D / 4);
          o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          mx[i] = -INFINITY;
          lx[i] = 0.f;
          for (int c = c0; c <= c1; ++c) {
            const float* src = p.part + ((size_t)c * 2 + (c == c0)) * floats;
            const float2 ml = __ldcg((const float2*)(src + kFewRows * D) + row);
            const float4 v = __ldcg((const float4*)src + q);
            const float top = fmaxf(mx[i], ml.x);
            const float a = mx[i] == -INFINITY ? 0.f : ex2(mx[i] - top), b = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);
            lx[i] = lx[i] * a + ml.y * b;
            o[i] = make_float4(o[i].x * a + v.x * b, o[i].y * a + v.y * b, o[i].z * a + v.z * b, o[i].w * a + v.w * b);
            mx[i] = top;
          }
        }
      }
    }
    if (write) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int q = threadIdx.x + i * kFewThreads, row = q / (D / 4), quad = q % (D / 4);
        const FewRow r = row_of(p, u, row);
        if (!r.on) continue;
        const float inv = 1.f / lx[i];
        const float4 v = make_float4(o[i].x * inv, o[i].y * inv, o[i].z * inv, o[i].w * inv);
        const uint2 z = kF16 ? make_uint2(pair16<__half>(v.x, v.y), pair16<__half>(v.z, v.w))
                             : make_uint2(pair16<__nv_bfloat16>(v.x, v.y), pair16<__nv_bfloat16>(v.z, v.w));
        *(uint2*)(p.out + r.row * p.out_stride + r.head * D + 4 * quad) = z;
      }
    }
    k = last;
  }
}

cudaError_t configure_history_few() {
  const cudaError_t e[4] = {
      cudaFuncSetAttribute(k_history_few<128, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, FewSmem<128>::kTotal),
      cudaFuncSetAttribute(k_history_few<128, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, FewSmem<128>::kTotal),
      cudaFuncSetAttribute(k_history_few<64, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, FewSmem<64>::kTotal),
      cudaFuncSetAttribute(k_history_few<64, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, FewSmem<64>::kTotal)};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

cudaError_t launch_history_few(const HistoryAttnParams& p, int D, int type, int sms, cudaStream_t st) {
  if (D == 128)
    type == WAVE_F16 ? k_history_few<128, true><<<sms, kFewThreads, FewSmem<128>::kTotal, st>>>(p)
                     : k_history_few<128, false><<<sms, kFewThreads, FewSmem<128>::kTotal, st>>>(p);
  else
    type == WAVE_F16 ? k_history_few<64, true><<<sms, kFewThreads, FewSmem<64>::kTotal, st>>>(p)
                     : k_history_few<64, false><<<sms, kFewThreads, FewSmem<64>::kTotal, st>>>(p);
  return cudaGetLastError();
}

}  // namespace wave
