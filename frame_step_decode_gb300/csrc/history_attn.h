// history_attn.h -- what the two kernels of attention over the 8-bit history share.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "history.h"
#include "prompt_ptx.cuh"

namespace wave {

struct HistoryAttnParams {
  SeqBatch b;
  const int32_t* positions;  // a frame's, on the device; null: the batch's
  int n;                     // sequences, or rows of the frame
  History hist;
  int heads, group;
  int tiles;                 // few rows: a frame's, of a K/V head's rows
  const uint16_t* q;
  uint16_t* out;
  long long q_stride, out_stride;
  float scale2;              // scale * log2(e)
  float* part;               // few rows: sums of units that several warps or CTAs share, ...
  int* part_cnt;             // ... and how many CTAs have left theirs, for each fourth of a unit's rows (0 between launches)
  int *err, *err_out;
};

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
// Sums that are joined are held over 2^12 of the values' units and relative to
// their weights' sum brought between 1 and 2, so that the sums of values near
// fp32's end do not leave it.
constexpr float kPartBias = 12.f;
// The exponent of a sum of weights (0 for one that is 0, infinite or NaN) ...
__device__ __forceinline__ int exponent_of_sum(float l) { return l > 0.f && l < INFINITY ? (int)(__float_as_uint(l) >> 23) - 127 : 0; }
// ... and the factor that takes joined sums to the output.
__device__ __forceinline__ float joined_factor(float l) { return 4096.f / l; }

// Whether one of four codes is NaN.
__device__ __forceinline__ bool any_nan_code(uint32_t w) { return (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0; }

constexpr int kFewTile = 16;                     // rows (tokens times heads of a group) of a unit of few rows
constexpr int kFewTiles = 2;                     // units of a prompt and K/V head at most
constexpr int kFewRows = kFewTile * kFewTiles;

cudaError_t launch_history_few(HistoryAttnParams& p, int D, int type, int rows, int sms, cudaStream_t st);

cudaError_t launch_history_many(const HistoryAttnParams& p, const wave_ctx* h, int type, cudaStream_t st);

}  // namespace wave
