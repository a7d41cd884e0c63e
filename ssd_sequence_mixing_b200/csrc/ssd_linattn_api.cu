// ssd_linattn_api.cu -- linear attention with a decay for each head: the entry points, the
// choice of windows, the gradients' plan and the kernels that finish them, and the
// single-token step.
//
// Gradients.  With D_t the gradient of the state S_t (D_t = a_{t+1} D_{t+1} + scale dy_t q_t^T,
// from dfinal after the last token),
//   dq_t = scale S_t^T dy_t,   dk_t = D_t^T v_t,   dv_t = D_t k_t,   dinit = a_1 D_1,
// and each of the first three is the operator again with its operands exchanged: dq is the
// pass (query, key, value) = (dy, v, k) in the order of the tokens from init^T; dk is
// (v, dy, q) and dv is (k, q, dy) against the order of the tokens from dfinal.  So the
// backward pass is three passes of the forward kernel and keeps nothing from the forward
// pass.  The decay's gradient a_t <D_t, S_{t-1}> is the difference of what q_t.dq_t and
// k_t.dk_t count (pairs i >= j with i at or after t, minus those with j at or after t):
//   dl_t = sum_{s >= t} (q_s . dq_s - k_s . dk_s) + <D_end, S_end>
// summed in 64 bits over windows of at most 1024 tokens, with <D, S> taken anew at every
// window's end, so that rounding errors do not pile up over a long sequence.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <initializer_list>

#include "ssd.h"
#include "ssd_common.cuh"
#include "ssd_linattn.cuh"

namespace ssd {
namespace {

// ------------------------------------------------------------------ finishing the gradients
struct LaGrad {
  int64_t tokens, seqlen;
  int H, size;  // size: NK * PV
  const int32_t* cu;
  int window, dense_windows;
  const LaWindow* win;
  const int32_t* win_count;
  const float *s_end, *d_end;     // (window, H, size): S after the window, and its gradient
  const float *q_dots, *k_dots;   // (slices, tokens, H)
  int slices;
  const float* log_decay;
  int per_token;
  int from_zero;   // sequences start from no state: their first decay has nothing to act on
  float* out;      // (tokens, H), or null:
  double* parts;   // (window, H) sums over the window's tokens
};

constexpr int kGradThreads = 128;

__device__ __forceinline__ double block_sum(double v, double* warp_sums) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kGradThreads / 32; ++w) s += warp_sums[w];
  return s;
}

// One block per window and head: <D, S> at the window's end, then the sums towards its start.
__global__ void __launch_bounds__(kGradThreads) la_decay_grad_kernel(LaGrad a) {
  __shared__ double s_warp[kGradThreads / 32];
  const int w = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t t0;
  int len;
  bool first;  // of its sequence
  if (a.cu) {
    if (w >= *a.win_count) return;  // (and where the offsets were invalid: -1)
    t0 = a.win[w].t0, len = a.win[w].len, first = t0 == a.cu[a.win[w].seq];
  } else {
    first = w % a.dense_windows == 0;
    t0 = (int64_t)(w / a.dense_windows) * a.seqlen + (int64_t)(w % a.dense_windows) * a.window;
    len = (int)min((int64_t)a.window, a.seqlen - (int64_t)(w % a.dense_windows) * a.window);
  }
  if (len <= 0) {
    if (a.parts && tid == 0) a.parts[(int64_t)w * a.H + h] = 0.0;
    return;
  }
  const float* s = a.s_end + ((int64_t)w * a.H + h) * a.size;
  const float* d = a.d_end + ((int64_t)w * a.H + h) * a.size;
  double v = 0.0;
  for (int e = tid; e < a.size; e += kGradThreads) v += (double)s[e] * (double)d[e];
  double carry = block_sum(v, s_warp);
  double total = 0.0;
  for (int hi = len; hi > 0; hi -= kGradThreads) {  // 128 tokens at a time, from the window's end
    const int i = hi - 1 - tid;                      // thread 0: the last one
    const int64_t t = t0 + i;
    double x = 0.0;
    if (i >= 0) {
      for (int n = 0; n < a.slices; ++n) {
        const int64_t at = ((int64_t)n * a.tokens + t) * a.H + h;
        x += (double)a.q_dots[at] - (double)a.k_dots[at];
      }
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    double before = 0.0, all = 0.0;
#pragma unroll
    for (int k = 0; k < kGradThreads / 32; ++k) {
      if (k < warp) before += s_warp[k];
      all += s_warp[k];
    }
    if (i >= 0) {
      const double l = (double)a.log_decay[a.per_token ? t * a.H + h : h] * 1.4426950408889634;
      // a decay of zero has no gradient in its log, nor has one of no state (the sums' difference is
      // rounding there)
      const bool none = l <= kLaLogMin || (a.from_zero && first && i == 0);
      const double g = none ? 0.0 : carry + before + x;
      if (a.out) a.out[t * a.H + h] = (float)g;
      total += g;
    }
    carry += all;
  }
  if (a.parts) {
    total = block_sum(total, s_warp);
    if (tid == 0) a.parts[(int64_t)w * a.H + h] = total;
  }
}

// Constant decays: the windows' sums, one block per head.
__global__ void __launch_bounds__(kGradThreads)
    la_decay_total_kernel(const double* parts, int windows, const int32_t* count, int H, float* out) {
  __shared__ double s_warp[kGradThreads / 32];
  const int h = blockIdx.x;
  const int n = count ? *count : windows;
  if (n < 0) return;
  double v = 0.0;
  for (int w = threadIdx.x; w < n; w += kGradThreads) v += parts[(int64_t)w * H + h];
  v = block_sum(v, s_warp);
  if (threadIdx.x == 0) out[h] = (float)v;
}

// dst[t][g][n] = sum over the group's heads of src[t][h][n], heads in order.
template <typename T>
__global__ void __launch_bounds__(256) la_group_sum_kernel(const float* src, T* dst, int64_t total, int N, int hpg,
                                                           const int32_t* count) {
  if (count && *count < 0) return;
  for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < total; e += (int64_t)gridDim.x * blockDim.x) {
    const int64_t tg = e / N;
    const int n = (int)(e - tg * N);
    const float* p = src + tg * hpg * N + n;
    float v = 0.f;
    for (int i = 0; i < hpg; ++i) v += p[(int64_t)i * N];
    dst[e] = from_f<T>(v);
  }
}

// ------------------------------------------------------------------------ the step
struct LaStep {
  int H, P, N, G, hpg;
  const void *q, *k, *v;
  const float* log_decay;
  int per_row;
  float scale;
  float* state;
  void* y;
};

constexpr int kStepRows = 8, kStepWarps = 4;

// Grid (rows * H, ceil(P / 32)); 4 warps, each advancing 8 rows of the state, all their loads
// in flight before the first use.  Lane l owns the columns 4 l .. 4 l + 3 (N <= 128).  The
// state is read and written once and is nearly all of the bytes: bound by HBM.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kStepWarps * 32) la_step_kernel(LaStep a) {
  const int64_t bh = blockIdx.x;
  const int64_t b = bh / a.H;
  const int h = (int)(bh % a.H), g = h / a.hpg;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int p0 = (blockIdx.y * kStepWarps + warp) * kStepRows, n0 = 4 * lane;
  float* S = a.state + bh * (int64_t)a.P * a.N;
  float s[kStepRows][4], vp[kStepRows], q[4], k[4];
#pragma unroll
  for (int r = 0; r < kStepRows; ++r) {
    const int p = p0 + r;
#pragma unroll
    for (int j = 0; j < 4; ++j) s[r][j] = 0.f;
    if (p < a.P) {
      const float* row = S + (int64_t)p * a.N + n0;
      if (VEC) {
        if (n0 < a.N) {
          const float4 x = *reinterpret_cast<const float4*>(row);
          s[r][0] = x.x, s[r][1] = x.y, s[r][2] = x.z, s[r][3] = x.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n0 + j < a.N) s[r][j] = row[j];
      }
    }
    vp[r] = p < a.P ? to_f(static_cast<const T*>(a.v)[bh * a.P + p]) : 0.f;
  }
  const T* qv = static_cast<const T*>(a.q) + (b * a.G + g) * a.N;
  const T* kv = static_cast<const T*>(a.k) + (b * a.G + g) * a.N;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    q[j] = n0 + j < a.N ? to_f(qv[n0 + j]) : 0.f;
    k[j] = n0 + j < a.N ? to_f(kv[n0 + j]) : 0.f;
  }
  const float decay = expf(a.log_decay[a.per_row ? bh : h]);
#pragma unroll
  for (int r = 0; r < kStepRows; ++r) {
    const int p = p0 + r;
    float acc = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s[r][j] = fmaf(decay, s[r][j], vp[r] * k[j]);
      acc = fmaf(q[j], s[r][j], acc);
    }
    if (p < a.P) {
      float* row = S + (int64_t)p * a.N + n0;
      if (VEC) {
        if (n0 < a.N) *reinterpret_cast<float4*>(row) = make_float4(s[r][0], s[r][1], s[r][2], s[r][3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n0 + j < a.N) row[j] = s[r][j];
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (lane == 0 && p < a.P) static_cast<T*>(a.y)[bh * a.P + p] = from_f<T>(acc * a.scale);
  }
}

// ------------------------------------------------------------------------ host side
size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

int la_validate(const ssd_shape* s, const int32_t* cu) {
  if (!s) return SSD_ERR_INVALID_ARG;
  if (s->batch < 0 || s->seqlen < 0 || s->nheads <= 0 || s->headdim <= 0 || s->dstate <= 0 || s->ngroups <= 0)
    return SSD_ERR_INVALID_ARG;
  if (s->io_dtype != SSD_F32 && s->io_dtype != SSD_BF16) return SSD_ERR_INVALID_ARG;
  if (cu && (s->batch != 1 || s->nseq < 1)) return SSD_ERR_INVALID_ARG;
  if (s->nheads % s->ngroups) return SSD_ERR_UNSUPPORTED;
  if (s->headdim > kLaMaxDim || s->dstate > kLaMaxDim || s->nheads > 65535) return SSD_ERR_UNSUPPORTED;
  if (s->batch > (1 << 30) || s->seqlen > (1 << 30) || (cu && s->nseq > (1 << 24))) return SSD_ERR_UNSUPPORTED;
  const int64_t tokens = s->batch * s->seqlen, rows = cu ? s->nseq : s->batch;
  if (tokens > ((int64_t)1 << 30) || rows > (1 << 24)) return SSD_ERR_UNSUPPORTED;
  // the longest list of units: the smallest windows, three passes (and room for a step past its end)
  if ((tokens / kLaMinWindow + rows + 1) * s->nheads * 3 > ((int64_t)1 << 31) - (1 << 16)) return SSD_ERR_UNSUPPORTED;
  if (s->cu_seqlens_host && cu) {
    const int32_t* c = s->cu_seqlens_host;
    if (c[0] != 0 || (int64_t)c[s->nseq] != tokens) return SSD_ERR_BAD_SEQLENS;
    for (int64_t i = 1; i <= s->nseq; ++i)
      if (c[i] < c[i - 1]) return SSD_ERR_BAD_SEQLENS;
  }
  return SSD_OK;
}

bool la_aligned(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (p && ((uintptr_t)p & 15u)) return false;
  return true;
}

// Bytes of the operands.
struct Sizes {
  int64_t qk, vy, decay, state, cu;
  Sizes(const ssd_shape* s, int64_t tokens, int64_t rows, bool per_token, bool packed) {
    const int64_t es = s->io_dtype == SSD_BF16 ? 2 : 4;
    qk = tokens * s->ngroups * s->dstate * es, vy = tokens * s->nheads * s->headdim * es;
    decay = (per_token ? tokens : 1) * s->nheads * 4, state = rows * s->nheads * s->headdim * s->dstate * 4;
    cu = packed ? (s->nseq + 1) * 4 : 0;
  }
};

struct Plan {
  int window, dense_windows, max_windows;
  int whole;  // sequences that are units by themselves; the others' windows are
  bool table;
  bool segmented(int64_t rows) const { return whole < rows; }
};

// Windows.  A sequence runs on `lanes` CTAs (of all `passes` together) of which `resident` fit the
// GPU at once.  Where whole sequences leave SMs idle (few of them, or a last round that is not
// full) some or all are cut into windows that run side by side, from states that a pass over key
// and value alone and a scan over the windows give; that pass costs about 0.6 of the full one,
// and the two launches before it the time of 12 + 4 passes blocks of 64 tokens (30 - 50 us).
// With k of the sequences of n blocks cut, in blocks' times,
//   n max(rounds of the others, all the work / resident) + 0.6 n k lanes / resident + launches
// and the k with the least is taken.  (2048 tokens: of 8 sequences x 40 pairs of heads one is
// cut, 306 us instead of 330; of 8 x 32 none.)
// The general kernel runs the passes one after another, so `lanes` counts one of them and the
// passes' number does not matter; its blocks take longer (fp32: 10 - 17 us), so the
// launches weigh less: `launches` = 5 blocks, 2 for fp32.  (Gradients of 2 fp32 sequences of 777
// tokens, 8 heads: windows of 128 tokens 204 us; whole, the passes in one launch, 231 us.)
Plan make_plan(const ssd_shape* s, const int32_t* cu, int64_t lanes, double launches, int64_t resident) {
  const int64_t tokens = s->batch * s->seqlen, rows = cu ? s->nseq : s->batch;
  Plan p{};
  p.window = 512;
  p.whole = (int)rows;
  int64_t cut = 0;
  if (cu) {
    // A packed batch may hold one long sequence among short ones, and its lengths are not known here:
    // all of them are cut unless there are enough to fill the GPU whatever their lengths.  Measured
    // (16 heads, G 4, N 64, P 128; cut / whole): 20,000 tokens and three short ones 216 / 680 us, 16 sequences of
    // 1 to 8192 205 / 296, 16 of 1850 237 / 150, 30 of 20 tokens 60 / 41
    if ((double)rows * (double)lanes < 4.0 * resident && tokens > 256) cut = rows;
  } else if (s->seqlen > kLaMinWindow) {
    const double n = (double)((s->seqlen + kLaChunk - 1) / kLaChunk);
    double best = n * (double)((rows * lanes + resident - 1) / resident);
    for (int64_t k = 1; k <= std::min<int64_t>(rows, 1024); ++k) {
      const double work = (double)(rows * lanes) / resident;
      const double whole = (double)(((rows - k) * lanes + resident - 1) / resident);
      const double least = (double)(kLaMinWindow / kLaChunk);  // a window's blocks follow one another
      const double time = std::max(n * std::max(whole, work), least) +
                          0.6 * std::max(n * (double)(k * lanes) / resident, least) + launches;
      if (time < best) best = time, cut = k;
    }
  }
  if (cut) {
    p.whole = (int)(rows - cut);
    const int64_t cut_tokens = cu ? tokens : cut * s->seqlen;
    // Enough windows for every CTA.  (Twice as many of a packed batch, whose windows are of all lengths: 16
    // sequences of 1850 tokens, 8 heads, N = P = 128, 211 us instead of 159; 20,000 tokens and three
    // short ones 159 instead of 172; 16 of 1 to 8192 162 instead of 155.)
    p.window = 1024;
    while (p.window > kLaMinWindow && cut_tokens / p.window * lanes < resident) p.window /= 2;
  }
  p.dense_windows = (int)std::max<int64_t>(1, (s->seqlen + p.window - 1) / p.window);
  const int64_t most = cu ? tokens / p.window + rows : rows * p.dense_windows;
  p.max_windows = (int)most;
  p.table = cu != nullptr;
  return p;
}

// The tcgen05 kernel takes bf16 operands of whole 16-byte rows; PATH_SIMT keeps to the general one.
bool wants_tc(const ssd_shape* s) {
  return s->io_dtype == SSD_BF16 && s->headdim % 8 == 0 && s->dstate % 8 == 0 && path_setting() != SSD_PATH_SIMT;
}
Plan plan_for(const ssd_shape* s, const int32_t* cu, bool tc, int64_t lanes, int passes) {
  const bool f32 = s->io_dtype == SSD_F32;
  return make_plan(s, cu, lanes, tc ? 12 + 4 * passes : f32 ? 2 : 5, (tc || f32 ? 1 : 3) * (int64_t)device_sm_count());
}

// Passes over one problem, with the windows' states first where it is segmented: side by side in
// one launch on the tcgen05 kernel (a batch that gives one pass too few CTAs may fill the GPU with
// three), one after another on the general one.  Pass i has the i-th part of carry and
// window_decay to itself.
cudaError_t run_passes(LaPass* p, int n, bool tc, bool bf16, float* carry, float* window_decay, cudaStream_t st) {
  const LaPass& q = p[0];
  const size_t states = (size_t)q.max_windows * q.H * q.NK * q.PV, decays = (size_t)q.max_windows * q.H;
  LaPass own[3];
  for (int i = 0; i < n; ++i) {
    p[i].carry = carry + i * states;
    p[i].window_decay = window_decay + i * decays;
    own[i] = p[i];
    own[i].states_only = 1;
    own[i].dump = nullptr, own[i].last = nullptr, own[i].dot = nullptr, own[i].dots = nullptr, own[i].out_f32 = 0;
  }
  auto launch = [&](const LaPass* l) {
    if (tc && la_tc_supports(l[0])) return launch_la_tc(l, n, st);
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < n && e == cudaSuccess; ++i) e = launch_la_general(l[i], bf16, l[i].dots != nullptr, st);
    return e;
  };
  cudaError_t e = cudaSuccess;
  if (la_segmented(q)) {
    e = launch(own);
    for (int i = 0; i < n && e == cudaSuccess; ++i) e = launch_la_scan(p[i], st);
  }
  return e == cudaSuccess ? launch(p) : e;
}

struct TableLayout {
  size_t win, first, count, total;
  TableLayout(const Plan& p, int64_t rows, size_t base) {
    win = base;
    first = win + (p.table ? up256(sizeof(LaWindow) * (size_t)p.max_windows) : 0);
    count = first + (p.table ? up256(sizeof(int32_t) * (size_t)(rows + 1)) : 0);
    total = count + (p.table ? 256 : 0);
  }
};

void set_common(LaPass& p, const ssd_shape* s, const Plan& plan, const int32_t* cu, char* ws, const TableLayout& t,
                const float* log_decay, int per_token, float scale) {
  p.tokens = s->batch * s->seqlen;
  p.seqlen = s->seqlen;
  p.nseq = (int)(cu ? s->nseq : s->batch);
  p.H = (int)s->nheads;
  p.cu = cu;
  p.window = plan.window;
  p.dense_windows = plan.dense_windows;
  p.max_windows = plan.max_windows;
  if (plan.table) {
    p.win = (const LaWindow*)(ws + t.win);
    p.first_win = (const int32_t*)(ws + t.first);
    p.win_count = (const int32_t*)(ws + t.count);
    p.next = (int32_t*)(ws + t.count) + 1;
  }
  p.log_decay = log_decay;
  p.per_token = per_token;
  p.scale = scale;
  p.whole = plan.whole;
}

cudaError_t build_table(const ssd_shape* s, const Plan& plan, const int32_t* cu, char* ws, const TableLayout& t,
                        unsigned int* status, cudaStream_t st) {
  if (!plan.table) return cudaSuccess;
  LaTable tab{(LaWindow*)(ws + t.win), (int32_t*)(ws + t.first), (int32_t*)(ws + t.count)};
  return launch_la_table(s->batch * s->seqlen, (int)s->nseq, cu, plan.window, plan.max_windows, tab, status, st);
}

}  // namespace
}  // namespace ssd

extern "C" int ssd_linear_attention_forward(const ssd_shape* s, const void* q, const void* k, const void* v,
                                            const float* log_decay, int decay_per_token, float scale,
                                            const float* init_state, const int32_t* cu, void* y, float* final_state,
                                            ssd_stream_t stream) {
  using namespace ssd;
  const int rc = la_validate(s, cu);
  if (rc) return rc;
  const int64_t tokens = s->batch * s->seqlen, rows = cu ? s->nseq : s->batch;
  if (!log_decay && (tokens > 0 || !decay_per_token)) return SSD_ERR_INVALID_ARG;
  if (tokens > 0 && (!q || !k || !v || !y)) return SSD_ERR_INVALID_ARG;
  if (!la_aligned({q, k, v, log_decay, init_state, cu, y, final_state})) return SSD_ERR_MISALIGNED;
  if (rows == 0) return SSD_OK;
  const Sizes z(s, tokens, rows, decay_per_token, cu);
  if (!buffers_apart({{y, z.vy}, {final_state, z.state}},
                {{q, z.qk}, {k, z.qk}, {v, z.vy}, {log_decay, z.decay}, {init_state, z.state}, {cu, z.cu}}))
    return SSD_ERR_INVALID_ARG;
  unsigned int* status = device_status_word();
  if (!status) return SSD_ERR_CUDA;
  cudaStream_t st = (cudaStream_t)stream;
  const int P = (int)s->headdim, N = (int)s->dstate, H = (int)s->nheads, hpg = (int)(s->nheads / s->ngroups);
  const bool tc = wants_tc(s);
  if (path_setting() == SSD_PATH_TC && !tc) return SSD_ERR_UNSUPPORTED;
  const Plan plan = plan_for(s, cu, tc, tc ? (P <= 64 && hpg % 2 == 0 ? H / 2 : H) : H * la_general_slices(P), 1);
  const TableLayout tl(plan, rows, 0);
  const size_t o_carry = tl.total;
  const size_t states = (size_t)plan.max_windows * H * P * N;
  const size_t o_dec = o_carry + (plan.segmented(rows) ? up256(sizeof(float) * states) : 0);
  const size_t total = o_dec + (plan.segmented(rows) ? up256(sizeof(float) * (size_t)plan.max_windows * H) : 0);
  char* ws = nullptr;
  if (total && scratch_alloc((void**)&ws, total, st) != cudaSuccess) return SSD_ERR_CUDA;
  LaPass p{};
  set_common(p, s, plan, cu, ws, tl, log_decay, decay_per_token, scale);
  p.query = q, p.key = k, p.value = v;
  p.q_heads = p.k_heads = (int)s->ngroups, p.v_heads = H;
  p.q_div = p.k_div = hpg, p.v_div = 1;
  p.NK = N, p.PV = P;
  p.start = init_state, p.last = final_state, p.sr = N, p.sc = 1;
  p.out = y;
  const bool bf16 = s->io_dtype == SSD_BF16;
  cudaError_t e = build_table(s, plan, cu, ws, tl, status, st);
  if (e == cudaSuccess) e = run_passes(&p, 1, tc, bf16, (float*)(ws + o_carry), (float*)(ws + o_dec), st);
  const cudaError_t e2 = ws ? cudaFreeAsync(ws, st) : cudaSuccess;
  return e != cudaSuccess || e2 != cudaSuccess ? SSD_ERR_CUDA : SSD_OK;
}

extern "C" int ssd_linear_attention_backward(const ssd_shape* s, const void* dy, const void* q, const void* k,
                                             const void* v, const float* log_decay, int decay_per_token, float scale,
                                             const float* init_state, const float* dfinal_state, const int32_t* cu,
                                             void* dq, void* dk, void* dv, float* dlog_decay, float* dinit_state,
                                             ssd_stream_t stream) {
  using namespace ssd;
  const int rc = la_validate(s, cu);
  if (rc) return rc;
  const int64_t tokens = s->batch * s->seqlen, rows = cu ? s->nseq : s->batch;
  if (!log_decay && (tokens > 0 || !decay_per_token)) return SSD_ERR_INVALID_ARG;
  if (tokens > 0 && (!dy || !q || !k || !v || !dq || !dk || !dv)) return SSD_ERR_INVALID_ARG;
  if (!la_aligned({dy, q, k, v, log_decay, init_state, dfinal_state, cu, dq, dk, dv, dlog_decay, dinit_state}))
    return SSD_ERR_MISALIGNED;
  cudaStream_t st = (cudaStream_t)stream;
  const int P = (int)s->headdim, N = (int)s->dstate, H = (int)s->nheads, G = (int)s->ngroups, hpg = H / G;
  if (rows == 0) {
    if (dlog_decay && !decay_per_token && cudaMemsetAsync(dlog_decay, 0, sizeof(float) * H, st) != cudaSuccess)
      return SSD_ERR_CUDA;
    return SSD_OK;
  }
  const Sizes z(s, tokens, rows, decay_per_token, cu);
  if (!buffers_apart({{dq, z.qk}, {dk, z.qk}, {dv, z.vy}, {dlog_decay, z.decay}, {dinit_state, z.state}},
                {{dy, z.vy}, {q, z.qk}, {k, z.qk}, {v, z.vy}, {log_decay, z.decay}, {init_state, z.state},
                 {dfinal_state, z.state}, {cu, z.cu}}))
    return SSD_ERR_INVALID_ARG;
  unsigned int* status = device_status_word();
  if (!status) return SSD_ERR_CUDA;
  const bool bf16 = s->io_dtype == SSD_BF16, decay_grad = dlog_decay != nullptr, shared = hpg > 1;
  const bool tc = wants_tc(s);
  if (path_setting() == SSD_PATH_TC && !tc) return SSD_ERR_UNSUPPORTED;
  const int slices = std::min(la_general_slices(P), la_general_slices(N));
  const int dot_slices = tc && tokens > 0 ? (N + 31) / 32 : la_general_slices(N);  // partial dots of a token
  const Plan plan = plan_for(s, cu, tc, tc ? 3 * H : H * slices, 3);
  const size_t W = (size_t)plan.max_windows, state = (size_t)H * P * N, th = (size_t)tokens * H;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += up256(bytes);
    return here;
  };
  const TableLayout tl(plan, rows, 0);
  at = tl.total;
  const size_t o_carry = take(plan.segmented(rows) ? 3 * 4 * W * state : 0);
  const size_t o_dec = take(plan.segmented(rows) ? 3 * 4 * W * H : 0);
  const size_t o_send = take(decay_grad ? 4 * W * state : 0), o_dend = take(decay_grad ? 4 * W * state : 0);
  const size_t o_qdot = take(decay_grad ? 4 * th * dot_slices : 0), o_kdot = take(decay_grad ? 4 * th * dot_slices : 0);
  const size_t o_parts = take(decay_grad && !decay_per_token ? 8 * W * H : 0);
  const size_t o_dq = take(shared ? 4 * th * N : 0), o_dk = take(shared ? 4 * th * N : 0);
  char* ws = nullptr;
  if (at && scratch_alloc((void**)&ws, at, st) != cudaSuccess) return SSD_ERR_CUDA;
  float *carry = (float*)(ws + o_carry), *dec = (float*)(ws + o_dec);
  cudaError_t e = build_table(s, plan, cu, ws, tl, status, st);
  const int32_t* count = plan.table ? (const int32_t*)(ws + tl.count) : nullptr;

  LaPass base{};
  set_common(base, s, plan, cu, ws, tl, log_decay, decay_per_token, scale);
  LaPass pass[3] = {base, base, base};
  {  // dq = pass (dy, v, k) from init^T
    LaPass& p = pass[0];
    p.query = dy, p.key = v, p.value = k;
    p.q_heads = p.k_heads = H, p.v_heads = G, p.q_div = p.k_div = 1, p.v_div = hpg;
    p.NK = P, p.PV = N;
    p.start = init_state, p.sr = 1, p.sc = N;
    p.out = shared ? (void*)(ws + o_dq) : dq, p.out_f32 = shared;
    if (decay_grad) {
      p.dump = (float*)(ws + o_send);
      p.dot = q, p.dot_heads = G, p.dot_div = hpg, p.dots = (float*)(ws + o_qdot);
    }
  }
  {  // dk = pass (v, dy, q), backwards from dfinal^T
    LaPass& p = pass[1];
    p.reverse = 1;
    p.query = v, p.key = dy, p.value = q;
    p.q_heads = p.k_heads = H, p.v_heads = G, p.q_div = p.k_div = 1, p.v_div = hpg;
    p.NK = P, p.PV = N;
    p.start = dfinal_state, p.sr = 1, p.sc = N;
    p.out = shared ? (void*)(ws + o_dk) : dk, p.out_f32 = shared;
    if (decay_grad) {
      p.dump = (float*)(ws + o_dend);
      p.dot = k, p.dot_heads = G, p.dot_div = hpg, p.dots = (float*)(ws + o_kdot);
    }
  }
  {  // dv = pass (k, q, dy), backwards from dfinal; its last state is dinit
    LaPass& p = pass[2];
    p.reverse = 1;
    p.query = k, p.key = q, p.value = dy;
    p.q_heads = p.k_heads = G, p.v_heads = H, p.q_div = p.k_div = hpg, p.v_div = 1;
    p.NK = N, p.PV = P;
    p.start = dfinal_state, p.last = dinit_state, p.sr = N, p.sc = 1;
    p.out = dv;
  }
  if (e == cudaSuccess) e = run_passes(pass, 3, tc, bf16, carry, dec, st);
  for (int i = 0; i < 2 && e == cudaSuccess && shared && tokens > 0; ++i) {
    const int64_t n = tokens * G * N;
    const unsigned blocks = (unsigned)std::min<int64_t>((n + 255) / 256, 148 * 32);
    const float* src = (const float*)(ws + (i ? o_dk : o_dq));
    if (bf16)
      la_group_sum_kernel<__nv_bfloat16><<<blocks, 256, 0, st>>>(src, (__nv_bfloat16*)(i ? dk : dq), n, N, hpg, count);
    else
      la_group_sum_kernel<float><<<blocks, 256, 0, st>>>(src, (float*)(i ? dk : dq), n, N, hpg, count);
    count_launches(1);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && decay_grad) {
    LaGrad g{};
    g.tokens = tokens, g.seqlen = s->seqlen, g.H = H, g.size = P * N;
    g.cu = cu, g.window = plan.window, g.dense_windows = plan.dense_windows;
    g.win = base.win, g.win_count = base.win_count;
    g.s_end = (const float*)(ws + o_send), g.d_end = (const float*)(ws + o_dend);
    g.q_dots = (const float*)(ws + o_qdot), g.k_dots = (const float*)(ws + o_kdot);
    g.slices = dot_slices;
    g.log_decay = log_decay, g.per_token = decay_per_token, g.from_zero = !init_state;
    g.out = decay_per_token ? dlog_decay : nullptr;
    g.parts = decay_per_token ? nullptr : (double*)(ws + o_parts);
    la_decay_grad_kernel<<<dim3((unsigned)plan.max_windows, (unsigned)H), kGradThreads, 0, st>>>(g);
    count_launches(1);
    if (!decay_per_token) {
      la_decay_total_kernel<<<H, kGradThreads, 0, st>>>(g.parts, plan.max_windows, count, H, dlog_decay);
      count_launches(1);
    }
    e = cudaGetLastError();
  }
  const cudaError_t e2 = ws ? cudaFreeAsync(ws, st) : cudaSuccess;
  return e != cudaSuccess || e2 != cudaSuccess ? SSD_ERR_CUDA : SSD_OK;
}

extern "C" int ssd_linear_attention_step(const ssd_shape* s, const void* q, const void* k, const void* v,
                                         const float* log_decay, int decay_per_row, float scale, float* state, void* y,
                                         ssd_stream_t stream) {
  using namespace ssd;
  const int rc = la_validate(s, nullptr);
  if (rc) return rc;
  if (s->seqlen != 1) return SSD_ERR_INVALID_ARG;
  if (s->batch == 0) return SSD_OK;
  if (!q || !k || !v || !log_decay || !state || !y) return SSD_ERR_INVALID_ARG;
  if (!la_aligned({q, k, v, log_decay, state, y})) return SSD_ERR_MISALIGNED;
  const Sizes z(s, s->batch, s->batch, decay_per_row, false);
  if (!buffers_apart({{y, z.vy}, {state, z.state}}, {{q, z.qk}, {k, z.qk}, {v, z.vy}, {log_decay, z.decay}}))
    return SSD_ERR_INVALID_ARG;
  LaStep a{};
  a.H = (int)s->nheads, a.P = (int)s->headdim, a.N = (int)s->dstate, a.G = (int)s->ngroups, a.hpg = a.H / a.G;
  a.q = q, a.k = k, a.v = v, a.log_decay = log_decay, a.per_row = decay_per_row, a.scale = scale;
  a.state = state, a.y = y;
  const int rows = kStepRows * kStepWarps;
  const dim3 grid((unsigned)(s->batch * s->nheads), (unsigned)((a.P + rows - 1) / rows));
  cudaStream_t st = (cudaStream_t)stream;
  const bool vec = a.N % 4 == 0;
  if (s->io_dtype == SSD_BF16)
    vec ? la_step_kernel<__nv_bfloat16, true><<<grid, kStepWarps * 32, 0, st>>>(a)
        : la_step_kernel<__nv_bfloat16, false><<<grid, kStepWarps * 32, 0, st>>>(a);
  else
    vec ? la_step_kernel<float, true><<<grid, kStepWarps * 32, 0, st>>>(a)
        : la_step_kernel<float, false><<<grid, kStepWarps * 32, 0, st>>>(a);
  count_launches(1);
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}
