// ctx.h -- the handle behind wave_t, shared by the host sides of the C ABI.
#pragma once
#include "plan.h"

struct wave_ctx {
  wave::Plan pl;
  int device = 0;
  void* ws_block = nullptr;
  wave::Workspace ws;
  int* err_host = nullptr;      // pinned host word the kernel mirrors the error bits into
  int* err_host_dev = nullptr;  // its device-side address
  // cached tensor maps and what they were encoded for
  wave::Maps maps;
  const void* maps_weights = nullptr;
  const void* maps_kv = nullptr;
  const void* maps_sc = nullptr;
  int maps_S = -1;
  cudaStream_t last_stream = nullptr;
  long long timeout_ns = 2000000000LL;
  int skip_cta = -1, skip_bar = -1, skip_sig = -1, skip_sig_kind = -1;
  float* kv_dump = nullptr;
  float* act_dump = nullptr;
  int act_dump_n = 0;
  long long* phase_ts = nullptr;
  long long* arrive_ts = nullptr;
};
