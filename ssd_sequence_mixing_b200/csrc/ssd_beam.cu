// ssd_beam.cu -- beam search for a recurrent model: the selection of the best continuations
// over beams and vocabulary, and the reordering of the beams' states that follows it.
//
// Selection.  With lse_i = log sum_w exp(x[i,w]) of beam i's logits, the continuations' scores
// are scores[i] + (x[i,w] - lse_i), formed in 64 bits and compared in fp32, as they are returned; the
// best `count` over all (i, w) are wanted, equal ones by the lower beam, then the larger logit,
// then the lower token.  The logits are read once:
//   1. blocks of 256 threads, several to a row of logits.  A thread goes over its elements
//      once, four vectors of 16 bytes in flight, and keeps their running maximum, its place,
//      and the running sum of exp(x).  A term is a function t(x) of the logit times an exact
//      power of two, and the sum is held in 64 bits in a unit of a power of two near the
//      maximum, so rows of the same logits have sums that differ by the order of 64-bit
//      additions alone, however they are cut among threads: by some 2^-52, which fp32
//      scores do not show, but for a score that lies that close to the border of two
//      (terms taken from a reference near each thread's own maximum differed by 1e-8: one
//      in some hundred equal rows around 64 did not tie).  Logits beyond 2^20 in size are taken from
//      such references all the same.
//      Let K be the count-th best of the threads' maxima: an element among the
//      row's best is at or above K and belongs to one of the `count` threads whose maximum is
//      (count other threads would otherwise each hold a better one), so those threads alone go
//      over their elements (some dozens, still in cache) a second time and hand on what is at
//      or above K.
//   2. one block per batch item joins the sums, forms the scores in 64 bits and picks the best
//      of the rows' sorted lists by the same argument.
// Bound by the issue of instructions for large batches (64 x 8 fp32 rows of 128,000, a fifth of them
// finished and not read: 68 us, 3.3 TB/s of what is read; 20 instructions an element, issued in
// 69 % of the cycles) and by the latency of two
// launches for one batch item (4 bf16 rows of 50,003: 20 us).  What counted on the way there: a
// warp instead of a thread over a chosen thread's elements, all of the merge's entries at once
// (109 to 67 us), and four vectors in flight with ranks by warp and then by block (139 to 109).
//
// Reordering.  state[b, i] <- state[b, parents[b, i]] in place: the beams of one batch item
// exchange rows only among themselves, so a thread that holds the same 16 bytes of all its
// beams loads what moves, then stores it; nothing needs a second buffer.  Rows that stay are
// neither read nor written.  Bound by HBM (16 x 4 rows of 8 layers, 1.8 GB moved: 300 to 350 us, 0.78
// to 0.92 of the measured copy rate, by box).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <memory>
#include <new>
#include <utility>

#include "ssd.h"
#include "ssd_common.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxBeams = 64;
constexpr int kMaxSplits = 64;
constexpr int kPerThread = 128;  // elements of a row a thread takes at most
// Dynamic shared memory of a block at most.  The kernels' limit is set to this, never to what one
// call needs: it belongs to the process, and another thread's call may be about to launch
constexpr int kMaxDynamic = 200 * 1024;

// Whole numbers in the order of the values (-0 and 0 equal; 0 is below every value but NaNs).
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v == 0.f ? 0.f : v);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// A candidate's rank as one whole number: a larger value first, then a lower place.  0 is "none".
__device__ __forceinline__ uint64_t key_of(float v, uint32_t at) {
  return (uint64_t)ordered(v) << 32 | (uint32_t)~at;
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ uint32_t key_place(uint64_t k) { return ~(uint32_t)k; }

// The unit of a sum of exponentials: e^ref 2^e.  Logits of usual sizes have ref = 0, so that terms are
// e^x = t 2^n with t a function of x alone, and going from one unit to another is exact.
constexpr float kUsual = 1048576.f;  // beyond this, x log2(e) has too few bits after the point: x - ref instead
constexpr int kStepE = 512;          // e goes in such steps: a sum of 2^20 terms stays below 2^(kStepE + 22)
struct SumUnit {
  float ref;
  int e;
};
constexpr SumUnit kNoUnit{-INFINITY, 0};  // of no logit above -inf
__device__ __forceinline__ double log2_ratio(SumUnit a, SumUnit b) {
  return ((double)a.ref - (double)b.ref) * 1.4426950408889634 + (double)(a.e - b.e);
}
__device__ __forceinline__ SumUnit larger(SumUnit a, SumUnit b) { return log2_ratio(a, b) > 0.0 ? a : b; }
// The largest of a warp's.
__device__ __forceinline__ SumUnit warp_largest(SumUnit u) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const SumUnit v{__shfl_xor_sync(0xffffffffu, u.ref, o), __shfl_xor_sync(0xffffffffu, u.e, o)};
    u = larger(v, u);
  }
  return u;
}

struct Select {
  int beams, vocab, count, splits, per_split;  // per_split: elements of a row in one block
  const void* logits;
  const float* scores;
  const uint8_t* finished;
  int eos;
  // of each row and split: the sum of exponentials and its unit, the best `count` keys
  SumUnit* row_unit;
  double* row_sum;
  uint64_t* keys;
  float* out_scores;
  int32_t *out_tokens, *out_parents;
};

template <typename T>
struct Vec {
  static constexpr int n = 16 / sizeof(T);
  T v[n];
};

// Elements [8 j, 8 j + 8) (fp32: 4) of the flat logits.
template <typename T>
__device__ __forceinline__ void load_whole(const T* logits, int64_t j, float (&x)[Vec<T>::n]) {
  Vec<T> v;
  *reinterpret_cast<uint4*>(&v) = __ldg(reinterpret_cast<const uint4*>(logits) + j);
#pragma unroll
  for (int i = 0; i < Vec<T>::n; ++i) x[i] = to_f(v.v[i]);
}

// The same, those outside [lo, hi) as -inf.
template <typename T>
__device__ __forceinline__ void load_vec(const T* logits, int64_t j, int64_t lo, int64_t hi,
                                         float (&x)[Vec<T>::n]) {
  constexpr int n = Vec<T>::n;
  const int64_t e0 = j * n;
  if (e0 >= lo && e0 + n <= hi) {
    load_whole(logits, j, x);
  } else {  // the range begins or ends inside this vector
#pragma unroll
    for (int i = 0; i < n; ++i) x[i] = e0 + i >= lo && e0 + i < hi ? to_f(logits[e0 + i]) : -INFINITY;
  }
}

__device__ __forceinline__ SumUnit unit_for(float top) {
  if (!(fabsf(top) <= kUsual)) return SumUnit{128.f * rintf(top * (1.f / 128.f)), 0};
  return SumUnit{0.f, kStepE * (int)rintf(top * (1.4426950408889634f / kStepE))};
}

// add_term's constants.
__device__ __forceinline__ float unit_low(SumUnit u) { return ((float)u.e - 1000.f) * 0.693147180559945f; }
__device__ __forceinline__ uint32_t unit_bias(SumUnit u) { return (uint32_t)(1023 - u.e) << 20; }

// 2^d, exact for whole d (0 from -1080 down); NaN for NaN.
__device__ __forceinline__ double pow2(double d) {
  const double n = floor(d), f = d - n;
  return ldexp(f == 0.0 ? 1.0 : exp2(f), (int)fmax(n, -1080.0));
}

// s + e^d in units of 2^e; a term below 2^-1000 of the unit counts as that (a sum is at least 2^-258
// of it).  NaN from a NaN or an infinite d on.
__device__ __forceinline__ double add_term(double s, float d, float low, uint32_t bias) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(d) : "f"(low));
  constexpr float kL = 1.44269502162933349609375f, kLow = 1.92596299112661746887e-8f;  // log2(e)
  constexpr float kWhole = 12582912.f;  // 1.5 2^23: adding it rounds to whole numbers, kept in the lowest bits
  const float y = fmaf(d, kL, kWhole);
  const float f = fmaf(d, kLow, fmaf(d, kL, kWhole - y));  // the rest, to 2^-26
  float t;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(f));
  return fma((double)t, __hiloint2double((int)((__float_as_uint(y) << 20) + bias), 0), s);
}

// Rank of `mine` among keys[0 .. n): how many are larger.
__device__ __forceinline__ int rank_of(uint64_t mine, const uint64_t* keys, int n) {
  int r = 0;
#pragma unroll 8
  for (int i = 0; i < n; ++i) r += keys[i] > mine;
  return r;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) beam_rows_kernel(Select a) {
  constexpr int n = Vec<T>::n, kVecs = 4, kWarps = kThreads / 32;
  extern __shared__ uint64_t s_list[];  // count * elements per thread
  __shared__ uint64_t s_key[kThreads];
  __shared__ uint64_t s_sorted[kWarps][32];  // each warp's best keys, in order
  __shared__ double s_sum[kWarps];
  __shared__ SumUnit s_unit[kWarps];
  __shared__ int s_who[kMaxBeams];  // the threads with the best maxima, in order
  __shared__ uint64_t s_limit;
  __shared__ int s_n;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x / a.splits;
  if (a.finished && a.finished[row]) return;  // its logits do not matter
  const int split = blockIdx.x % a.splits;
  const T* logits = static_cast<const T*>(a.logits);
  const int64_t start = row * a.vocab;  // of the row in the flat array
  const int64_t lo = start + (int64_t)split * a.per_split;
  const int64_t hi = min(start + a.vocab, lo + a.per_split);
  const int64_t j0 = lo / n, j1 = (hi + n - 1) / n;  // 16-byte vectors that hold the range

  // vectors of the block: [0, vecs), those that lie in the range as a whole: [in0, in1)
  const int vecs = (int)(j1 - j0), in0 = lo % n != 0, in1 = (int)(hi / n - j0);
  float m = -INFINITY;
  SumUnit unit{0.f, 0};
  float low = unit_low(unit);
  uint32_t bias = unit_bias(unit);
  double s = 0.0;
  int from = 0;  // the group of vectors that holds the maximum first
  for (int u = tid; u < vecs; u += kVecs * kThreads) {
    float x[kVecs][n];
    if (u >= in0 && u + (kVecs - 1) * kThreads < in1) {
#pragma unroll
      for (int v = 0; v < kVecs; ++v) load_whole(logits, j0 + u + v * kThreads, x[v]);
    } else {
#pragma unroll
      for (int v = 0; v < kVecs; ++v) load_vec(logits, j0 + u + v * kThreads, lo, hi, x[v]);  // (past the range: -inf)
    }
    float top = -INFINITY;
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
#pragma unroll
      for (int i = 0; i < n; ++i) top = fmaxf(top, x[v][i]);
    if (top > m) {
      const bool none = m == -INFINITY;
      m = top;
      from = u;
      // the first value, one far above the unit, or a usual one after logits like -1e9
      if (none || (top - unit.ref) * 1.4426950408889634f - (float)unit.e > (float)kStepE ||
          (unit.ref < 0.f && top >= -kUsual)) {
        const SumUnit to = unit_for(top);
        s *= none ? 0.0 : pow2(log2_ratio(unit, to));  // (0: what -inf counted so far; a NaN stays)
        unit = to;
        low = unit_low(to), bias = unit_bias(to);
      }
    }
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
#pragma unroll
      for (int i = 0; i < n; ++i) s = add_term(s, x[v][i] - unit.ref, low, bias);
  }
  int best = -1;  // place of the maximum in the row
  if (m > -INFINITY) {  // looked up once: at every new maximum it cost a quarter of the loop
#pragma unroll
    for (int v = kVecs - 1; v >= 0; --v) {
      float x[n];
      load_vec(logits, j0 + from + v * kThreads, lo, hi, x);
#pragma unroll
      for (int i = n - 1; i >= 0; --i)
        if (x[i] == m) best = (int)((j0 + from + v * kThreads) * n + i - start);
    }
  }
  // a thread without an element above -inf has no key
  const uint64_t mine = best >= 0 ? key_of(m, (uint32_t)best) : 0;
  if (m == -INFINITY) unit = kNoUnit, s *= 0.0;  // (a NaN stays)
  SumUnit bm = warp_largest(unit);
  if (lane == 0) s_unit[warp] = bm;
  s_key[tid] = mine;
  s_sorted[warp][lane] = 0;
  if (tid < kMaxBeams) s_who[tid] = -1;
  if (tid == 0) s_n = 0, s_limit = 1;
  __syncwarp();
  int r = mine ? rank_of(mine, s_key + 32 * warp, 32) : kThreads;  // in the warp
  if (mine) s_sorted[warp][r] = mine;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) bm = larger(s_unit[w], bm);
  double sum = s == 0.0 ? 0.0 : s * pow2(log2_ratio(unit, bm));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_sum[warp] = sum;
  if (mine && r < a.count)  // ... and in the block, from the other warps' lists
    for (int w = 0; w < kWarps && r < a.count; ++w)
      if (w != warp)
        for (int i = 0; i < 32 && r < a.count && s_sorted[w][i] > mine; ++i) ++r;
  if (r == a.count - 1) s_limit = mine;
  if (r < a.count) s_who[r] = tid;
  __syncthreads();
  // a warp takes all vectors of one such thread at once
  const uint64_t limit = s_limit;
  for (int q = warp; q < a.count; q += kWarps) {
    if (s_who[q] < 0) break;
    for (int64_t j = j0 + s_who[q] + lane * kThreads; j < j1; j += 32 * kThreads) {
      float x[n];
      load_vec(logits, j, lo, hi, x);
#pragma unroll
      for (int i = 0; i < n; ++i) {
        if (!(x[i] > -INFINITY)) continue;
        const uint64_t k = key_of(x[i], (uint32_t)(j * n + i - start));
        if (k >= limit) s_list[atomicAdd(&s_n, 1)] = k;
      }
    }
  }
  __syncthreads();
  const int got = s_n;
  uint64_t* out = a.keys + (int64_t)blockIdx.x * a.count;
  for (int e = tid; e < got; e += kThreads) {
    const uint64_t k = s_list[e];
    const int at = rank_of(k, s_list, got);
    if (at < a.count) out[at] = k;
  }
  for (int e = got + tid; e < a.count; e += kThreads) out[e] = 0;
  if (tid == 0) {
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) t += s_sum[w];
    a.row_unit[blockIdx.x] = bm;
    a.row_sum[blockIdx.x] = t;
  }
}

struct Cand {
  uint32_t score, beam;  // ordered(score), 0: none
  uint64_t key;          // of the logit and the token
};
__device__ __forceinline__ bool before(const Cand& x, const Cand& y) {
  if (x.score != y.score) return x.score > y.score;
  if (x.beam != y.beam) return x.beam < y.beam;
  return x.key > y.key;
}
constexpr Cand kNone{0, 0xFFFFFFFFu, 0};

// Entry e, with key k, of a list of beam `beam` with the sum `lse`; none where the score is -inf or NaN.
__device__ __forceinline__ Cand candidate(const Select& a, uint64_t k, int beam, bool first_split, int e, double lse,
                                          double score, bool finished) {
  if (finished) {
    if (first_split && e == 0 && score > -INFINITY)
      return Cand{ordered((float)score), (uint32_t)beam, key_of(0.f, (uint32_t)a.eos)};
    return kNone;
  }
  if (!k) return kNone;
  const float v = (float)(score + ((double)key_value(k) - lse));
  if (!(v > -INFINITY)) return kNone;
  return Cand{ordered(v), (uint32_t)beam, k};
}

// One block per batch item.  Lists: (beam, split), each sorted.  A list's entry among the best
// `count` is at or above the count-th best of the lists' first entries.
__global__ void __launch_bounds__(kThreads) beam_merge_kernel(Select a) {
  extern __shared__ unsigned char s_raw[];
  const int lists = a.beams * a.splits;
  double* s_lse = reinterpret_cast<double*>(s_raw);                // beams
  Cand* s_head = reinterpret_cast<Cand*>(s_lse + kMaxBeams);       // lists
  Cand* s_cand = s_head + lists;                                   // count * count
  __shared__ Cand s_limit;
  __shared__ int s_n;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t b = blockIdx.x;
  const int64_t list0 = b * lists;
  if (tid == 0) s_n = 0, s_limit = Cand{1, 0xFFFFFFFFu, 0};
  // asked for now, needed after the sums (a finished beam's lists were not written: unused)
  const uint64_t first = tid < lists ? a.keys[(list0 + tid) * a.count] : 0;
  for (int i = warp; i < a.beams; i += kThreads / 32) {  // a warp per beam, a lane or more per split
    if (a.finished && a.finished[b * a.beams + i]) continue;  // (nothing was written for it)
    static_assert(kMaxSplits <= 64, "a lane takes two splits");
    SumUnit unit[2];
    double part[2], sum = 0.0;
    uint32_t top = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int e = lane + 32 * h;
      const bool in = e < a.splits;
      const int64_t l = list0 + i * a.splits + e;
      unit[h] = in ? a.row_unit[l] : kNoUnit;
      part[h] = in ? a.row_sum[l] : 0.0;
      top = max(top, in ? (uint32_t)(a.keys[l * a.count] >> 32) : 0);
    }
    const SumUnit all = warp_largest(larger(unit[1], unit[0]));
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (part[h] != 0.0) sum += part[h] * pow2(log2_ratio(unit[h], all));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    // The largest term anew in 64 bits, and the logarithm of the sum's ratio to it: what is left of a
    // row with one likely token is that token's 0, and no score is above its beam's
    const float x = key_value((uint64_t)__reduce_max_sync(0xffffffffu, top) << 32);
    const double exact = exp2(((double)x - (double)all.ref) * 1.4426950408889634 - (double)all.e);
    sum -= add_term(0.0, x - all.ref, unit_low(all), unit_bias(all));
    if (sum < 0.0) sum = 0.0;  // (by the rounding of references that differ, of logits beyond 2^20; a NaN stays)
    if (lane == 0) s_lse[i] = (double)x + log1p(sum / exact);  // (NaN for a row of -inf alone, which has no key)
  }
  for (int i = tid; i < a.count; i += kThreads) {  // what stays where there are too few continuations
    a.out_scores[b * a.count + i] = -INFINITY;
    a.out_tokens[b * a.count + i] = max(a.eos, 0);
    a.out_parents[b * a.count + i] = i % a.beams;
  }
  __syncthreads();
  for (int l = tid; l < lists; l += kThreads) {
    const int beam = l / a.splits;
    const bool fin = a.finished && a.finished[b * a.beams + beam];
    const uint64_t k = l == tid ? first : a.keys[(list0 + l) * a.count];
    s_head[l] = candidate(a, k, beam, l % a.splits == 0, 0, s_lse[beam], (double)a.scores[b * a.beams + beam], fin);
  }
  __syncthreads();
  for (int l = warp; l < lists; l += kThreads / 32) {  // a warp ranks a list
    const Cand mine = s_head[l];
    if (!mine.score) continue;
    int r = 0;
    for (int i = lane; i < lists; i += 32) r += before(s_head[i], mine);
    r = __reduce_add_sync(0xffffffffu, r);
    if (lane == 0 && r == a.count - 1) s_limit = mine;
  }
  __syncthreads();
  const Cand limit = s_limit;
  for (int q = tid; q < lists * a.count; q += kThreads) {  // all entries at once: one load's latency
    const int l = q / a.count, e = q - l * a.count;
    if (!s_head[l].score || before(limit, s_head[l])) continue;  // below the limit from the start
    const int beam = l / a.splits;
    const bool fin = a.finished && a.finished[b * a.beams + beam];
    const Cand c = candidate(a, a.keys[list0 * a.count + q], beam, l % a.splits == 0, e, s_lse[beam],
                             (double)a.scores[b * a.beams + beam], fin);
    if (c.score && !before(limit, c)) s_cand[atomicAdd(&s_n, 1)] = c;
  }
  __syncthreads();
  const int got = s_n;
  for (int e = tid; e < got; e += kThreads) {
    const Cand c = s_cand[e];
    int r = 0;
    for (int i = 0; i < got; ++i) r += before(s_cand[i], c);
    if (r < a.count) {
      a.out_scores[b * a.count + r] = key_value((uint64_t)c.score << 32);
      a.out_tokens[b * a.count + r] = (int32_t)key_place(c.key);
      a.out_parents[b * a.count + r] = (int32_t)c.beam;
    }
  }
}

// ------------------------------------------------------------------- reordering
constexpr int kMaxBuffers = 128;
constexpr int kReorderThreads = 256;

struct Reorder {
  const int32_t* parents;
  unsigned int* status;
  int beams, nbuf;
  int64_t batch;
  struct {
    void* base;
    int64_t row;       // units in a row
    int64_t first;     // first block of this buffer
    int tiles;         // blocks per batch item
  } buf[kMaxBuffers];
};

// Block: one batch item and kReorderThreads units' columns of one buffer.
template <typename V, int MAXB>
__global__ void __launch_bounds__(kReorderThreads) state_reorder_kernel(const __grid_constant__ Reorder a) {
  __shared__ int s_src[MAXB];
  int i = 0;
  {
    int lo = 0, hi = a.nbuf - 1;  // the last buffer that begins at or before this block
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.buf[mid].first <= (int64_t)blockIdx.x)
        lo = mid;
      else
        hi = mid - 1;
    }
    i = lo;
  }
  const int64_t local = (int64_t)blockIdx.x - a.buf[i].first;
  const int tiles = a.buf[i].tiles;
  const int64_t b = local / tiles, row = a.buf[i].row;
  const int64_t col = (local % tiles) * kReorderThreads + threadIdx.x;
  if (threadIdx.x < MAXB) {
    int p = threadIdx.x;
    if (p < a.beams) {
      p = a.parents[b * a.beams + p];
      if (p < 0 || p >= a.beams) {  // leave the row as it is and say so
        p = threadIdx.x;
        atomicOr(a.status, kStatusBadParent);
      }
    }
    s_src[threadIdx.x] = p;
  }
  __syncthreads();
  if (col >= row) return;
  V* base = static_cast<V*>(a.buf[i].base) + b * a.beams * row + col;
  V v[MAXB];
#pragma unroll
  for (int k = 0; k < MAXB; ++k)
    if (k < a.beams && s_src[k] != k) v[k] = base[s_src[k] * row];
#pragma unroll
  for (int k = 0; k < MAXB; ++k)
    if (k < a.beams && s_src[k] != k) base[k * row] = v[k];
}

constexpr int64_t kMaxBlocks = ((int64_t)1 << 31) - 1;  // of a launch; one buffer's are 2^30 + 2^24 at most

template <typename V>
cudaError_t launch_reorder(Reorder& a, cudaStream_t st) {
  int64_t blocks = 0;
  for (int i = 0; i < a.nbuf; ++i) {
    a.buf[i].row /= (int64_t)sizeof(V);
    a.buf[i].first = blocks;
    a.buf[i].tiles = (int)((a.buf[i].row + kReorderThreads - 1) / kReorderThreads);
    blocks += a.batch * a.buf[i].tiles;
  }
  if (a.beams <= 4)
    state_reorder_kernel<V, 4><<<(unsigned)blocks, kReorderThreads, 0, st>>>(a);
  else if (a.beams <= 8)
    state_reorder_kernel<V, 8><<<(unsigned)blocks, kReorderThreads, 0, st>>>(a);
  else if (sizeof(V) == 16 || a.beams <= 16)
    state_reorder_kernel<V, 16><<<(unsigned)blocks, kReorderThreads, 0, st>>>(a);
  else if constexpr (sizeof(V) < 16)
    state_reorder_kernel<V, kMaxBeams><<<(unsigned)blocks, kReorderThreads, 0, st>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace
}  // namespace ssd

extern "C" int ssd_beam_select(int64_t batch, int64_t beams, int64_t vocab, ssd_dtype logits_dtype, const void* logits,
                               const float* scores, const uint8_t* finished, int32_t eos, int64_t count,
                               float* out_scores, int32_t* out_tokens, int32_t* out_parents, ssd_stream_t stream) {
  using namespace ssd;
  if (batch < 0 || beams <= 0 || vocab <= 0 || count <= 0) return SSD_ERR_INVALID_ARG;
  if (logits_dtype != SSD_F32 && logits_dtype != SSD_BF16) return SSD_ERR_INVALID_ARG;
  if (beams > kMaxBeams || count > kMaxBeams || vocab > (1 << 20) || batch > (1 << 24)) return SSD_ERR_UNSUPPORTED;
  if (finished && (eos < 0 || eos >= vocab)) return SSD_ERR_INVALID_ARG;
  if (batch == 0) return SSD_OK;
  if (!logits || !scores || !out_scores || !out_tokens || !out_parents) return SSD_ERR_INVALID_ARG;
  for (const void* p : {logits, (const void*)scores, (const void*)finished, (const void*)out_scores,
                        (const void*)out_tokens, (const void*)out_parents})
    if (p && ((uintptr_t)p & 15u)) return SSD_ERR_MISALIGNED;
  const int64_t rows = batch * beams;
  if (!buffers_apart({{out_scores, batch * count * 4}, {out_tokens, batch * count * 4}, {out_parents, batch * count * 4}},
                     {{logits, rows * vocab * (logits_dtype == SSD_BF16 ? 2 : 4)}, {scores, rows * 4}, {finished, rows}}))
    return SSD_ERR_INVALID_ARG;
  // Splits of a row: enough blocks to fill the GPU, 2048 elements or more in each, and at
  // most kPerThread elements a thread.
  const int64_t fill = (8 * (int64_t)device_sm_count() + rows - 1) / rows;
  int64_t splits = std::max<int64_t>(1, std::min<int64_t>(fill, vocab / 2048));
  splits = std::min<int64_t>(splits, kMaxSplits);
  splits = std::max<int64_t>(splits, (vocab + kThreads * kPerThread - 1) / (kThreads * kPerThread));
  const int64_t per_split = ((vocab + splits - 1) / splits + 7) & ~(int64_t)7;
  splits = (vocab + per_split - 1) / per_split;
  if (rows * splits > ((int64_t)1 << 31) - 1) return SSD_ERR_UNSUPPORTED;
  Select a{};
  a.beams = (int)beams, a.vocab = (int)vocab, a.count = (int)count;
  a.splits = (int)splits, a.per_split = (int)per_split;
  a.logits = logits, a.scores = scores, a.finished = finished, a.eos = finished ? eos : std::max(eos, -1);
  a.out_scores = out_scores, a.out_tokens = out_tokens, a.out_parents = out_parents;
  const int es = logits_dtype == SSD_BF16 ? 2 : 4, per_vec = 16 / es;
  // vectors of a block's range (its ends may share one with a neighbour), per thread
  const int64_t vecs = per_split / per_vec + 2;
  const size_t list_bytes = sizeof(uint64_t) * (size_t)count * per_vec * (size_t)((vecs + kThreads - 1) / kThreads);
  const size_t cands = (size_t)beams * splits + (size_t)count * count;
  const size_t merge_bytes = sizeof(double) * kMaxBeams + sizeof(Cand) * cands;
  if (list_bytes > kMaxDynamic || merge_bytes > kMaxDynamic) return SSD_ERR_UNSUPPORTED;
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  const size_t n = (size_t)(rows * splits);
  const size_t o_sum = up(n * sizeof(SumUnit)), o_keys = o_sum + up(n * sizeof(double)),
               total = o_keys + up(n * (size_t)count * sizeof(uint64_t));
  cudaStream_t st = (cudaStream_t)stream;
  char* ws = nullptr;
  if (scratch_alloc((void**)&ws, total, st) != cudaSuccess) return SSD_ERR_CUDA;
  a.row_unit = (SumUnit*)ws, a.row_sum = (double*)(ws + o_sum), a.keys = (uint64_t*)(ws + o_keys);
  auto* rows_fn = logits_dtype == SSD_BF16 ? beam_rows_kernel<__nv_bfloat16> : beam_rows_kernel<float>;
  cudaError_t e = cudaSuccess;
  if (list_bytes > 40 * 1024)
    e = cudaFuncSetAttribute(rows_fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDynamic);
  if (e == cudaSuccess && merge_bytes > 40 * 1024)
    e = cudaFuncSetAttribute(beam_merge_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDynamic);
  if (e == cudaSuccess) {
    rows_fn<<<(unsigned)n, kThreads, list_bytes, st>>>(a);
    beam_merge_kernel<<<(unsigned)batch, kThreads, merge_bytes, st>>>(a);
    count_launches(2);
    e = cudaGetLastError();
  }
  const cudaError_t e2 = cudaFreeAsync(ws, st);
  return e != cudaSuccess || e2 != cudaSuccess ? SSD_ERR_CUDA : SSD_OK;
}

extern "C" int ssd_state_reorder(int64_t batch, int64_t beams, const int32_t* parents, int64_t nbuf,
                                 void* const* buffers, const int64_t* row_bytes, ssd_stream_t stream) {
  using namespace ssd;
  if (batch < 0 || beams <= 0 || nbuf < 0) return SSD_ERR_INVALID_ARG;
  if (beams > kMaxBeams || batch > (1 << 24) || nbuf > (1 << 20)) return SSD_ERR_UNSUPPORTED;
  if (batch == 0 || nbuf == 0) return SSD_OK;
  if (!parents || !buffers || !row_bytes) return SSD_ERR_INVALID_ARG;
  if ((uintptr_t)parents & 3u) return SSD_ERR_MISALIGNED;
  typedef std::pair<uintptr_t, uintptr_t> Span;
  std::unique_ptr<Span[]> spans(new (std::nothrow) Span[nbuf]);
  if (!spans) return SSD_ERR_CUDA;
  int64_t n = 0;
  for (int64_t i = 0; i < nbuf; ++i) {
    if (row_bytes[i] < 0) return SSD_ERR_INVALID_ARG;
    if (row_bytes[i] == 0) continue;
    if (!buffers[i]) return SSD_ERR_INVALID_ARG;
    if ((uintptr_t)buffers[i] & 15u) return SSD_ERR_MISALIGNED;
    if (row_bytes[i] > ((int64_t)1 << 38) / (batch * beams)) return SSD_ERR_UNSUPPORTED;
    spans[n++] = Span((uintptr_t)buffers[i], (uintptr_t)buffers[i] + (uintptr_t)(batch * beams * row_bytes[i]));
  }
  std::sort(spans.get(), spans.get() + n);
  for (int64_t i = 1; i < n; ++i)
    if (spans[i].first < spans[i - 1].second) return SSD_ERR_INVALID_ARG;  // one buffer would be moved twice
  for (int64_t i = 0; i < n; ++i)  // ... or the parents moved while others read them
    if (buffers_meet({parents, batch * beams * 4}, {(void*)spans[i].first, (int64_t)(spans[i].second - spans[i].first)}))
      return SSD_ERR_INVALID_ARG;
  unsigned int* status = device_status_word();
  if (!status) return SSD_ERR_CUDA;
  cudaStream_t st = (cudaStream_t)stream;
  // buffers whose rows are whole 16-byte units, then those of 4-byte units, then the rest; more
  // than 16 beams go by 4 bytes, so that a thread can hold one unit of each
  for (int unit : {16, 4, 1}) {
    Reorder a{};
    a.parents = parents, a.status = status, a.beams = (int)beams, a.batch = batch;
    int64_t blocks = 0;
    auto flush = [&]() {
      const cudaError_t e = !a.nbuf      ? cudaSuccess
                            : unit == 16 ? launch_reorder<uint4>(a, st)
                            : unit == 4  ? launch_reorder<uint32_t>(a, st)
                                         : launch_reorder<uint8_t>(a, st);
      a.nbuf = 0, blocks = 0;
      return e == cudaSuccess;
    };
    for (int64_t i = 0; i < nbuf; ++i) {
      if (row_bytes[i] == 0) continue;
      const int own = row_bytes[i] % 16 == 0 && beams <= 16 ? 16 : row_bytes[i] % 4 == 0 ? 4 : 1;
      if (own != unit) continue;
      const int64_t mine = batch * ((row_bytes[i] / unit + kReorderThreads - 1) / kReorderThreads);
      if ((a.nbuf == kMaxBuffers || blocks + mine > kMaxBlocks) && !flush()) return SSD_ERR_CUDA;
      a.buf[a.nbuf].base = buffers[i];
      a.buf[a.nbuf].row = row_bytes[i];
      ++a.nbuf, blocks += mine;
    }
    if (!flush()) return SSD_ERR_CUDA;
  }
  return SSD_OK;
}
