// ssd_linattn.cuh -- what the kernels of linear attention with a decay for each head share:
// the description of one pass and the launchers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace ssd {

// Log-decays are held in base 2 and kept at or above this: 2^-150 is zero in fp32, so a
// decay of exp(-inf) = 0 needs no case of its own and no difference of two sums is inf - inf.
constexpr double kLaLogMin = -150.0;
constexpr int kLaChunk = 64;   // tokens of a block of the chunked form (general kernel)
constexpr int kLaSlice = 64;   // rows of the value dimension one CTA takes (general kernel)
constexpr int kLaMinWindow = 128;  // tokens of the smallest window
constexpr int kLaMaxDim = 128; // largest query/key and value dimension

// A window: `len` tokens from t0, all of sequence `seq`.
struct LaWindow {
  int32_t seq, t0, len;
};

// One pass over every sequence and head h, in the order of the tokens or (reverse) against it:
//   out_i = scale * sum_j  decay(i, j) (query_i . key_j) value_j   over j <= i (reverse: j >= i)
// with decay(i, j) the product of the a_t between them, and the same from the state `start`.
// The state (value dimension x key dimension) of head h is
//   forward:  S_t = a_t S_{t-1} + value_t key_t^T,        out_t = scale * S_t query_t
//   reverse:  D_t = a_{t+1} D_{t+1} + scale * value_t key_t^T,  out_t = D_t query_t
// (the forward recurrence of the operator, and the one its gradients follow).
struct LaPass {
  // tokens
  int64_t tokens, seqlen;
  int nseq, H;
  const int32_t* cu;  // packed offsets, or null: nseq rows of seqlen tokens
  // windows of `window` tokens (a multiple of both kernels' chunks)
  int window, dense_windows;   // dense_windows: per row, max(1, ceil(seqlen / window))
  int max_windows;             // upper bound on their number
  const LaWindow* win;         // packed batches: the windows, ...
  const int32_t* first_win;    // ... each sequence's first one (nseq + 1), ...
  const int32_t* win_count;    // ... and their number, or -1 for invalid offsets
  int32_t* next;               // ... and two counters of units taken (tcgen05 kernel): the full passes', states_only's
  // operands: head h reads head h / div of an array with `heads` heads
  const void *query, *key, *value;
  int q_heads, k_heads, v_heads, q_div, k_div, v_div;
  int NK, PV;                  // key and value dimensions
  const float* log_decay;      // (tokens, H), or (H) when !per_token
  int per_token;
  float scale;
  int reverse;
  // states: element (r, c) of (sequence, head) at base + (seq * H + h) * NK * PV + r * sr + c * sc
  const float* start;          // before the first token (reverse: after the last), or null
  float* last;                 // after the last token (reverse: before the first), or null
  int64_t sr, sc;
  // units: the first `whole` sequences, then the windows of the others, each of which starts from
  // carry[window][H][PV][NK] (a packed batch has all of its sequences whole, or none)
  int whole;
  float* carry;                // states_only: the windows' end states from zero go here
  float* window_decay;         // states_only: (window, H) decay over the window
  int states_only;
  float* dump;                 // (window, H, PV, NK) state after each window (reverse: before
                               // it in processing order, the gradient of the state after it), or null
  // outputs
  void* out;                   // (tokens, H, PV), io type, or fp32 with out_f32
  int out_f32;
  const void* dot;             // dots = dot . out of each token (dot: (tokens, dot_heads, PV)), or null
  int dot_heads, dot_div;
  float* dots;                 // (slices, tokens, H)
};

inline bool la_segmented(const LaPass& p) { return p.whole < p.nseq; }
// Upper bound on the units (of one head).
inline int64_t la_units(const LaPass& p) {
  return !la_segmented(p) ? p.nseq : p.cu ? p.max_windows : p.whole + (int64_t)(p.nseq - p.whole) * p.dense_windows;
}

struct LaTable {
  LaWindow* win;
  int32_t *first_win, *count;  // count: the windows' number, then the two counters of units taken
};

cudaError_t launch_la_table(int64_t tokens, int nseq, const int32_t* cu, int window, int max_windows, LaTable t,
                            unsigned int* status, cudaStream_t st);
// bf16: io type; exact: the products that enter `out` keep fp32 accuracy (needed for dots).
cudaError_t launch_la_general(const LaPass& p, bool bf16, bool exact, cudaStream_t st);
int la_general_slices(int PV);
// The tcgen05 kernel (bf16): whether it takes the pass, and whether its CTAs take two heads each.
bool la_tc_supports(const LaPass& p);
bool la_tc_pairs(const LaPass& p);
// Up to three passes of one problem, side by side; a pass with `dots` keeps fp32 accuracy.
cudaError_t launch_la_tc(const LaPass* p, int passes, cudaStream_t st);
// carry[w] <- the state before window w (reverse: after it in time), from the windows' own states.
cudaError_t launch_la_scan(const LaPass& p, cudaStream_t st);

}  // namespace ssd
