// ssd_linattn_dev.cuh -- device code both kernels of linear attention share.
#pragma once

#include "ssd_linattn.cuh"

namespace ssd {
namespace {

__device__ __forceinline__ double log2_clamped(float log_decay) {
  const double l = (double)log_decay * 1.4426950408889634;
  return l < kLaLogMin ? kLaLogMin : l;  // a NaN stays one
}

__device__ __forceinline__ double log2_decay(const LaPass& a, int64_t t, int h) {
  return log2_clamped(a.log_decay[a.per_token ? t * a.H + h : h]);
}

// 2^(hi + lo) for whole hi <= 0, to fp32 rounding.
__device__ __forceinline__ float exp2_parts(float hi, float lo) { return exp2f(lo) * exp2f(hi); }

struct Unit {
  int seq;
  int64_t t0;
  int len, window;   // window: its number (a whole sequence: that of its first)
  bool first, last;  // the unit begins / ends its sequence
};

__device__ __forceinline__ bool get_unit(const LaPass& a, int u, Unit& r) {
  const bool whole = u < a.whole;
  if (a.win_count && (*a.win_count < 0 || (!whole && u >= *a.win_count))) return false;
  int64_t s0, s1;
  if (whole) {
    r.seq = u;
    s0 = a.cu ? a.cu[u] : (int64_t)u * a.seqlen;
    s1 = a.cu ? a.cu[u + 1] : s0 + a.seqlen;
    r.t0 = s0;
    r.len = (int)(s1 - s0);
    r.window = a.cu ? a.first_win[u] : u * a.dense_windows;
  } else if (a.cu) {
    const LaWindow w = a.win[u];
    r.seq = w.seq, r.t0 = w.t0, r.len = w.len, r.window = u;
    s0 = a.cu[r.seq], s1 = a.cu[r.seq + 1];
  } else {
    const int v = u - a.whole;
    r.seq = a.whole + v / a.dense_windows;
    s0 = (int64_t)r.seq * a.seqlen, s1 = s0 + a.seqlen;
    r.t0 = s0 + (int64_t)(v % a.dense_windows) * a.window;
    r.len = (int)min((int64_t)a.window, s1 - r.t0);
    r.window = a.whole * a.dense_windows + v;
  }
  r.first = r.t0 == s0;
  r.last = r.t0 + r.len == s1;
  return true;
}

}  // namespace
}  // namespace ssd
