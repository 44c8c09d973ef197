// sessions.cu -- wave_sessions_copy: sessions forked into other slots of the
// batch, or moved into free ones.
//
// Bound by HBM: every byte a source holds is read once, however many slots it
// goes to, and written once per destination; a CTA moves pieces of 16 KB, four
// 16-byte loads of a thread in flight, and the grid (8 CTAs per SM) shares the
// pieces of all sources and layers evenly whatever the positions, which only
// the device knows (one session of 1500 positions to 8 slots, eight layers of
// 32 x 128 heads: 144.6 us = 6.31 TB/s; four hybrid sessions, ten state layers
// and two of history: 40.4 us = 5.79 TB/s).
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/wave.h"
#include "ctx.h"
#include "prompt.h"

using namespace wave;

namespace wave {

constexpr int kMaxSessions = 128;        // S_max's limit
constexpr int kPieceBytes = 16 * 1024;   // 256 threads x 4 x 16 bytes

struct CopyParams {
  int n_src;                             // sources, each with ...
  int first[kMaxSessions + 1];           // ... the pairs first[i]..first[i + 1] - 1
  uint8_t src[kMaxSessions], dst[kMaxSessions];  // slots (dst by pair)
  int S_max, H, T_max, D, La, Lm, move;
  long long state_bytes;                 // of one session in one selective-state layer
  uint8_t* kv;
  float* scales;
  float* state;
  int32_t* pos;
};

__device__ __forceinline__ int held(const CopyParams& p, int s) { return max(0, min(p.pos[s], p.T_max)); }

// One piece: up to kPieceBytes (a multiple of 4) at the same offset of every destination.
__device__ __forceinline__ void copy_piece(const CopyParams& p, int i, char* base, long long slot_bytes, long long at,
                                           int bytes) {
  const char* s = base + p.src[i] * slot_bytes + at;
  uint4 v[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int o = (k * 256 + (int)threadIdx.x) * 16;
    if (o + 16 <= bytes) v[k] = __ldcs((const uint4*)(s + o));
  }
  for (int d = p.first[i]; d < p.first[i + 1]; ++d) {
    char* t = base + p.dst[d] * slot_bytes + at;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int o = (k * 256 + (int)threadIdx.x) * 16;
      if (o + 16 <= bytes) __stcs((uint4*)(t + o), v[k]);
    }
    const int o = (bytes & ~15) + (int)threadIdx.x * 4;  // the last words, fewer than four
    if (o < bytes) *(uint32_t*)(t + o) = *(const uint32_t*)(s + o);
  }
}

__global__ void __launch_bounds__(256) k_sessions_copy(const __grid_constant__ CopyParams p) {
  __shared__ long long units[kMaxSessions + 1];
  const int rows = p.La * 2 * p.H;
  const int state_pieces = (int)(p.state_bytes / kPieceBytes);
  if (threadIdx.x == 0) {
    long long u = 0;
    for (int i = 0; i < p.n_src; ++i) {
      units[i] = u;
      const long long code_pieces = ((long long)held(p, p.src[i]) * p.D + kPieceBytes - 1) / kPieceBytes;
      const long long scale_pieces = ((long long)held(p, p.src[i]) * 4 + kPieceBytes - 1) / kPieceBytes;
      u += rows * (code_pieces + scale_pieces);
      if (p.pos[p.src[i]] >= 0) u += (long long)p.Lm * state_pieces;
    }
    units[p.n_src] = u;
  }
  __syncthreads();
  int i = 0;
  for (long long u = blockIdx.x; u < units[p.n_src]; u += gridDim.x) {
    while (u >= units[i + 1]) ++i;
    const int n = held(p, p.src[i]);
    const long long codes = (long long)n * p.D, sc = (long long)n * 4;
    const long long cp = (codes + kPieceBytes - 1) / kPieceBytes, sp = (sc + kPieceBytes - 1) / kPieceBytes;
    long long r = u - units[i];
    if (r < rows * cp) {
      const long long row = r / cp, at = (r - row * cp) * kPieceBytes, lw = row / p.H, h = row - lw * p.H;
      const long long slot = (long long)p.H * p.T_max * p.D;
      copy_piece(p, i, (char*)p.kv + lw * p.S_max * slot, slot, h * p.T_max * p.D + at,
                 (int)min((long long)kPieceBytes, codes - at));
    } else if ((r -= rows * cp) < rows * sp) {
      const long long row = r / sp, at = (r - row * sp) * kPieceBytes, lw = row / p.H, h = row - lw * p.H;
      const long long slot = (long long)p.H * p.T_max * 4;
      copy_piece(p, i, (char*)p.scales + lw * p.S_max * slot, slot, h * p.T_max * 4 + at,
                 (int)min((long long)kPieceBytes, sc - at));
    } else {
      r -= rows * sp;
      const long long lm = r / state_pieces, at = (r - lm * state_pieces) * kPieceBytes;
      copy_piece(p, i, (char*)p.state + lm * p.S_max * p.state_bytes, p.state_bytes, at, kPieceBytes);
    }
  }
  // no CTA reads a destination's position
  if (blockIdx.x == 0 && !p.move) {
    for (int s = 0; s < p.n_src; ++s)
      for (int d = p.first[s] + (int)threadIdx.x; d < p.first[s + 1]; d += 256) p.pos[p.dst[d]] = p.pos[p.src[s]];
  }
}

// A move ends with the sources' slots empty: after every CTA of the copy has read the positions.
__global__ void k_sessions_moved(const __grid_constant__ CopyParams p) {
  for (int s = threadIdx.x; s < p.n_src; s += blockDim.x) {
    for (int d = p.first[s]; d < p.first[s + 1]; ++d) p.pos[p.dst[d]] = p.pos[p.src[s]];
    p.pos[p.src[s]] = -1;
  }
}

}  // namespace wave

extern "C" int wave_sessions_copy(wave_t* h, int n, const int32_t* src, const int32_t* dst, int move, uint8_t* kv_fp8,
                                  float* kv_scales, float* ssm_state, int32_t* positions, void* stream) {
  if (!h || !src || !dst || !kv_fp8 || !kv_scales || !positions) return WAVE_EINVAL;
  const Plan& pl = h->pl;
  if (n < 1 || n > pl.S_max || (pl.hybrid ? !ssm_state : ssm_state != nullptr)) return WAVE_EINVAL;
  if (!aligned16(kv_fp8) || !aligned16(kv_scales) || !aligned16(ssm_state) || ((uintptr_t)positions & 3))
    return WAVE_EINVAL;
  bool is_src[kMaxSessions] = {false}, is_dst[kMaxSessions] = {false};
  for (int i = 0; i < n; ++i) {
    if (src[i] < 0 || src[i] >= pl.S_max || dst[i] < 0 || dst[i] >= pl.S_max || is_dst[dst[i]]) return WAVE_EINVAL;
    is_src[src[i]] = true;
    is_dst[dst[i]] = true;
  }
  for (int s = 0; s < pl.S_max; ++s)
    if (is_src[s] && is_dst[s]) return WAVE_EINVAL;  // it would be read and written at once
  if (!on_device(h)) return WAVE_EINVAL;
  CopyParams p;
  p.n_src = 0;
  p.first[0] = 0;
  int k = 0;
  for (int s = 0; s < pl.S_max; ++s) {
    if (!is_src[s]) continue;
    for (int i = 0; i < n; ++i)
      if (src[i] == s) p.dst[k++] = (uint8_t)dst[i];
    p.src[p.n_src++] = (uint8_t)s;
    p.first[p.n_src] = k;
  }
  p.S_max = pl.S_max;
  p.H = pl.cfg.n_heads;
  p.T_max = pl.T_max;
  p.D = pl.cfg.head_dim;
  p.La = pl.cfg.n_layers;
  p.Lm = pl.hybrid ? pl.hcfg.n_layers - pl.cfg.n_layers : 0;
  p.state_bytes = pl.hybrid ? (long long)pl.hcfg.ssm_heads * kSsmP * kSsmN * 4 : kPieceBytes;
  p.move = move != 0;
  p.kv = kv_fp8;
  p.scales = kv_scales;
  p.state = ssm_state;
  p.pos = positions;
  cudaStream_t st = (cudaStream_t)stream;
  h->last_stream = st;
  k_sessions_copy<<<pl.grid * 8, 256, 0, st>>>(p);
  if (p.move) k_sessions_moved<<<1, 128, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? WAVE_OK : WAVE_ECUDA;
}
