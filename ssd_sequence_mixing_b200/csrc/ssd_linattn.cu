// ssd_linattn.cu -- the general kernel of linear attention with a decay for each head, and the
// small kernels around it: the table of windows of a packed batch and the scan of the
// windows' states.
//
// The chunked form: over a block of 64 tokens with c_i the inclusive sum of its log-decays,
//   out_i = scale * ( sum_{j<=i} 2^(c_i - c_j) (query_i . key_j) value_j  +  2^(c_i) S query_i )
//   S    <- 2^(c_end) S + sum_j 2^(c_end - c_j) value_j key_j^T
// and against the order of the tokens (the gradients of key and value) the same with j >= i,
// 2^(c_j - c_i), and the two per-token factors 2^(c) and 2^(c_end - c) exchanged.
//
// One CTA (4 warps) takes 64 rows of the value dimension of one head and walks the blocks of
// its unit with that part of the state (64 x NK, fp32) in registers, as the accumulators of
// mma.sync.  Everything is computed transposed (out^T = S query^T + value^T P^T), so the
// state's accumulators are themselves the A operand of the next block's S query^T and need no
// trip through shared memory.  It takes every size up to 128 x 128, both io types and any
// alignment; the tcgen05 kernel takes the common bf16 shapes.
//
// Precision: a bf16 operand enters a product as it is; an fp32 operand (an fp32 input, the
// state, the decayed value rows that feed the state) enters as three bf16 planes whose sum is
// the fp32 value to 24 bits, and the products of planes i + j <= 2 are summed, lowest first.
// With bf16 outputs the masked product P and the state's copy that meets the query are
// rounded to one plane each (about the output's own rounding); the state itself never is.
//
// Measured, fp32: gradients of 2 x 777 tokens, 8 heads, N 96, P 64: 204 us; 256 tokens of 2 heads of
// 16 x 16: 35 us.  Bound by latency: at 110 to 160 KB of tiles an SM holds one or two CTAs, a
// scheduler one or two warps, and an instruction takes 5 to 6 cycles (waits for its last one, for
// instructions and for loads in equal parts), some 5400 of them a warp and block.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "sm100_ptx.cuh"
#include "ssd.h"
#include "ssd_common.cuh"
#include "ssd_linattn.cuh"
#include "ssd_linattn_dev.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(sm100::smem_u32(p))
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(sm100::smem_u32(p))
               : "memory");
}
// d += a (16 x 16, row) b (16 x 8, col)
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// The planes of an fp32 pair: plane 0 its bf16 rounding, plane 1 that of what is left, ...
template <int NP>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&out)[NP]) {
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    out[p] = sm100::bf16x2(x, y);
    if (p + 1 < NP) x -= sm100::bf16_lo(out[p]), y -= sm100::bf16_hi(out[p]);
  }
}

template <int SP, int PO, int NT>
struct Smem {
  static constexpr int kQ = NT + 8, kV = kLaSlice + 8, kP = kLaChunk + 8;  // row pitches (bf16): no bank conflicts
  __nv_bfloat16 q[SP][kLaChunk][kQ];
  __nv_bfloat16 k[SP][kLaChunk][kQ];
  __nv_bfloat16 v[SP][kLaChunk][kV];
  __nv_bfloat16 p[PO][kLaChunk][kP];
  // c = chi + clo (chi whole, 0 <= clo < 1): differences of c keep their fraction bits
  float chi[kLaChunk], clo[kLaChunk], row[kLaChunk], upd[kLaChunk], decay;
  double total;
  float dots[4][kLaChunk];
};

// 64 rows (tokens) x COLS columns of a (tokens, heads, dim) array into planes; rows past
// `rows` and columns past dim - c0 become zeros.
template <int SP, int COLS, int PITCH>
__device__ __forceinline__ void load_tile(__nv_bfloat16 (*dst)[kLaChunk][PITCH], const void* src, int64_t t0, int rows,
                                          int heads, int head, int dim, int c0) {
  static_assert(COLS * kLaChunk / 4 % (8 * kThreads) == 0, "whole groups of loads");
  const int valid = min(COLS, dim - c0);
  if constexpr (SP == 1) {
    const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(src) + (t0 * heads + head) * (int64_t)dim + c0;
    const int64_t pitch = (int64_t)heads * dim;
    if (dim % 8 == 0) {  // every row starts on a 16-byte boundary
      constexpr int vec = COLS / 8;
      for (int e = threadIdx.x; e < kLaChunk * vec; e += kThreads) {
        const int r = e / vec, c = (e % vec) * 8;
        const bool in = r < rows && c < valid;
        const __nv_bfloat16* p = in ? base + r * pitch + c : static_cast<const __nv_bfloat16*>(src);
        const int bytes = in ? 16 : 0;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm100::smem_u32(&dst[0][r][c])), "l"(p),
                     "r"(bytes)
                     : "memory");
      }
    } else {
      for (int e = threadIdx.x; e < kLaChunk * COLS; e += kThreads) {
        const int r = e / COLS, c = e % COLS;
        dst[0][r][c] = r < rows && c < valid ? base[r * pitch + c] : __float2bfloat16_rn(0.f);
      }
    }
  } else {
    // eight loads of a thread in flight (one after another, a block of 64 tokens took 25 us more)
    constexpr int kFlight = 8;
    const float* base = static_cast<const float*>(src) + (t0 * heads + head) * (int64_t)dim + c0;
    const int64_t pitch = (int64_t)heads * dim;
    const int padded = min(COLS, (valid + 15) & ~15);  // columns that the products read
    auto put = [&](int r, int c, float x, float y) {
      uint32_t pl[SP];
      split2<SP>(x, y, pl);
#pragma unroll
      for (int p = 0; p < SP; ++p) *reinterpret_cast<uint32_t*>(&dst[p][r][c]) = pl[p];
    };
    if (dim % 4 == 0) {  // every row starts on a 16-byte boundary
      constexpr int kVec = COLS / 4;
      for (int e0 = threadIdx.x; e0 < kLaChunk * kVec; e0 += kFlight * kThreads) {
        float4 x[kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
          const int e = e0 + i * kThreads, r = e / kVec, c = (e % kVec) * 4;
          x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (r < rows && c < valid) x[i] = __ldg(reinterpret_cast<const float4*>(base + r * pitch + c));
        }
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
          const int e = e0 + i * kThreads, r = e / kVec, c = (e % kVec) * 4;
          if (c >= padded) continue;
          put(r, c, x[i].x, x[i].y);
          put(r, c + 2, x[i].z, x[i].w);
        }
      }
    } else {
      constexpr int kPairs = COLS / 2;
      for (int e0 = threadIdx.x; e0 < kLaChunk * kPairs; e0 += kFlight * kThreads) {
        float x[kFlight][2];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
          const int e = e0 + i * kThreads, r = e / kPairs, c = (e % kPairs) * 2;
          x[i][0] = r < rows && c < valid ? __ldg(base + r * pitch + c) : 0.f;
          x[i][1] = r < rows && c + 1 < valid ? __ldg(base + r * pitch + c + 1) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
          const int e = e0 + i * kThreads, r = e / kPairs, c = (e % kPairs) * 2;
          if (c < padded) put(r, c, x[i][0], x[i][1]);
        }
      }
    }
  }
}

// Grid: units x heads x slices (slices fastest, then heads, so that CTAs that read the same
// query and key run together).
template <int SP, int PO, int NT>
__global__ void __launch_bounds__(kThreads, SP == 1 ? 3 : 1) la_general_kernel(LaPass a, int slices) {
  using S = Smem<SP, PO, NT>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  S& sm = *reinterpret_cast<S*>(smem_raw);
  constexpr int KS = NT / 16, NTILES = NT / 8;
  // fp32 operands: the products of lower planes have accumulators of their own.  An accumulation
  // in the tensor core truncates to the sum's last bit, and the sum of the highest planes
  // then takes a sixth of them.  Their loops stay rolled where the registers' indices allow:
  // each instruction runs once a block, and fetching them is what a block of a short window
  // waits for.
  constexpr bool kLow = SP == 3;
  const int slice = blockIdx.x % slices;
  const int h = (blockIdx.x / slices) % a.H;
  const int u = blockIdx.x / slices / a.H;
  Unit un;
  if (!get_unit(a, u, un)) return;
  const bool begins = a.reverse ? un.last : un.first, ends = a.reverse ? un.first : un.last;
  if (a.states_only && ends) return;  // nothing follows this window
  const int lane = threadIdx.x & 31, hw = threadIdx.x >> 5;
  // the causal products give the warps unequal work: turn their parts from CTA to CTA, so
  // that every sub-partition of the SM gets each part
  const int warp = (hw + blockIdx.x) & 3;
  const int gr = lane >> 2, gc = (lane & 3) * 2;
  const int row0 = slice * kLaSlice;          // first value row of the CTA
  const int r_lo = row0 + 16 * warp + gr;     // this thread's value rows: r_lo, r_lo + 8
  const bool has_rows = row0 + 16 * warp < a.PV;  // (a warp without any still computes rows of P)
  const int qh = h / a.q_div, kh = h / a.k_div, vh = h / a.v_div;
  const int64_t state_at = ((int64_t)un.seq * a.H + h) * a.NK * a.PV;

  // the state: st[n][..] is the accumulator tile of columns 8 n ..
  float st[NTILES][4];
#pragma unroll
  for (int n = 0; n < NTILES; ++n) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = r_lo + 8 * (e >> 1), c = 8 * n + gc + (e & 1);
      float v = 0.f;
      if (r < a.PV && c < a.NK) {
        if (begins) {
          if (a.start) v = a.start[state_at + r * a.sr + c * a.sc];
        } else if (!a.states_only) {
          v = a.carry[(((int64_t)un.window * a.H + h) * a.PV + r) * a.NK + c];
        }
      }
      st[n][e] = v;
    }
  }
  const int chunks = (un.len + kLaChunk - 1) / kLaChunk;
  double total = 0.0;  // log2 of the decay over the unit
  for (int step = 0; step < chunks; ++step) {
    const int ci = a.reverse ? chunks - 1 - step : step;
    const int64_t t0 = un.t0 + (int64_t)ci * kLaChunk;
    const int rows = min(kLaChunk, un.len - ci * kLaChunk);
    if (a.dump && a.reverse && (ci == chunks - 1 || ((ci + 1) * kLaChunk) % a.window == 0)) {
      const int64_t w = un.window + ((int64_t)ci * kLaChunk) / a.window;
#pragma unroll
      for (int n = 0; n < NTILES; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = r_lo + 8 * (e >> 1), c = 8 * n + gc + (e & 1);
          if (r < a.PV && c < a.NK) a.dump[((w * a.H + h) * a.PV + r) * a.NK + c] = st[n][e];
        }
    }
    __syncthreads();  // the last block's tiles are no longer read
    if (!a.states_only) load_tile<SP, NT>(sm.q, a.query, t0, rows, a.q_heads, qh, a.NK, 0);
    load_tile<SP, NT>(sm.k, a.key, t0, rows, a.k_heads, kh, a.NK, 0);
    load_tile<SP, kLaSlice>(sm.v, a.value, t0, rows, a.v_heads, vh, a.PV, row0);
    if constexpr (SP == 1) sm100::cp_async_commit();
    if (hw == 0) {
      // lane l: tokens 2 l and 2 l + 1; tokens past the end do not decay
      const int i0 = 2 * lane, i1 = i0 + 1;
      const double l0 = i0 < rows ? log2_decay(a, t0 + i0, h) : 0.0;
      const double l1 = i1 < rows ? log2_decay(a, t0 + i1, h) : 0.0;
      double c1 = l0 + l1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double x = __shfl_up_sync(0xffffffffu, c1, o);
        if (lane >= o) c1 += x;
      }
      const double end = __shfl_sync(0xffffffffu, c1, 31);
      const double c0 = c1 - l1;
      const float sr = a.reverse ? 1.f : a.scale, su = a.reverse ? a.scale : 1.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const double c = j ? c1 : c0;
        const int i = j ? i1 : i0;
        const double f = floor(c), g = floor(end - c);
        const float hi = (float)f, lo = (float)(c - f);
        sm.chi[i] = hi, sm.clo[i] = lo;
        const float from_start = exp2_parts(hi, lo), to_end = exp2_parts((float)g, (float)(end - c - g));
        sm.row[i] = (a.reverse ? to_end : from_start) * sr;
        sm.upd[i] = (a.reverse ? from_start : to_end) * su;
      }
      if (lane == 31) {
        sm.decay = exp2f((float)end);
        sm.total = end;
      }
    }
    if constexpr (SP == 1) sm100::cp_async_wait_all();
    __syncthreads();
    total += sm.total;

    if (!a.states_only) {
      // P = decay o (query key^T) * scale: warp's rows i = 16 warp .., all columns j
      const int i_lo = 16 * warp + gr;
      float acc[8][4], low[kLow ? 8 : 1][4];
      auto clear = [&]() {
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            acc[n][e] = 0.f;
            if constexpr (kLow) low[n][e] = 0.f;
          }
      };
      auto join = [&]() {
        if constexpr (kLow)
#pragma unroll
          for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][e] += low[n][e];
      };
      clear();
      const int n0 = a.reverse ? 2 * warp : 0, n1 = a.reverse ? 8 : 2 * warp + 2;  // column tiles with any j in reach
#pragma unroll(kLow ? 1 : KS)
      for (int ks = 0; ks < KS; ++ks) {
        if (16 * ks >= a.NK) continue;
        uint32_t qa[SP][4];
#pragma unroll
        for (int p = 0; p < SP; ++p)
          ldsm4(qa[p], &sm.q[p][16 * warp + (lane & 7) + ((lane >> 3) & 1) * 8][16 * ks + ((lane >> 4) & 1) * 8]);
#pragma unroll
        for (int n = 0; n < 8; n += 2) {
          if (n < n0 || n >= n1) continue;
          uint32_t kb[SP][4];
#pragma unroll
          for (int p = 0; p < SP; ++p)
            ldsm4(kb[p], &sm.k[p][8 * n + (lane & 7) + ((lane >> 4) & 1) * 8][16 * ks + ((lane >> 3) & 1) * 8]);
#pragma unroll
          for (int i = SP - 1; i >= 0; --i)
#pragma unroll
            for (int j = SP - 1 - i; j >= 0; --j) {
              mma(kLow && i + j ? low[kLow ? n : 0] : acc[n], qa[i], kb[j][0], kb[j][1]);
              mma(kLow && i + j ? low[kLow ? n + 1 : 0] : acc[n + 1], qa[i], kb[j][2], kb[j][3]);
            }
        }
      }
      join();
      const float hi0 = sm.chi[i_lo], lo0 = sm.clo[i_lo], hi1 = sm.chi[i_lo + 8], lo1 = sm.clo[i_lo + 8];
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        if (n < n0 || n >= n1) continue;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = i_lo + 8 * (e >> 1), j = 8 * n + gc + (e & 1);
          const float dh = (e >> 1 ? hi1 : hi0) - sm.chi[j], dl = (e >> 1 ? lo1 : lo0) - sm.clo[j];
          const float d = a.reverse ? -dh - dl : dh + dl;
          const bool in = a.reverse ? j >= i : j <= i;
          v[e] = in ? acc[n][e] * sm100::ex2(d) * a.scale : 0.f;
        }
        uint32_t p0[PO], p1[PO];
        split2<PO>(v[0], v[1], p0);
        split2<PO>(v[2], v[3], p1);
#pragma unroll
        for (int p = 0; p < PO; ++p) {
          *reinterpret_cast<uint32_t*>(&sm.p[p][i_lo][8 * n + gc]) = p0[p];
          *reinterpret_cast<uint32_t*>(&sm.p[p][i_lo + 8][8 * n + gc]) = p1[p];
        }
      }
      __syncthreads();

      // out^T (16 value rows of the warp x 64 tokens) = row o (S query^T) + value^T P^T
      clear();
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        if (16 * ks >= a.NK || !has_rows) continue;
        uint32_t sa[4][PO];
        split2<PO>(st[2 * ks][0], st[2 * ks][1], sa[0]);
        split2<PO>(st[2 * ks][2], st[2 * ks][3], sa[1]);
        split2<PO>(st[2 * ks + 1][0], st[2 * ks + 1][1], sa[2]);
        split2<PO>(st[2 * ks + 1][2], st[2 * ks + 1][3], sa[3]);
#pragma unroll
        for (int n = 0; n < 8; n += 2) {
          uint32_t qb[SP][4];
#pragma unroll
          for (int p = 0; p < SP; ++p)
            ldsm4(qb[p], &sm.q[p][8 * n + (lane & 7) + ((lane >> 4) & 1) * 8][16 * ks + ((lane >> 3) & 1) * 8]);
#pragma unroll
          for (int i = PO - 1; i >= 0; --i) {
            const uint32_t af[4] = {sa[0][i], sa[1][i], sa[2][i], sa[3][i]};
#pragma unroll
            for (int j = SP - 1; j >= 0; --j) {
              if (i + j > 2) continue;
              mma(kLow && i + j ? low[kLow ? n : 0] : acc[n], af, qb[j][0], qb[j][1]);
              mma(kLow && i + j ? low[kLow ? n + 1 : 0] : acc[n + 1], af, qb[j][2], qb[j][3]);
            }
          }
        }
      }
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[n][e] *= sm.row[8 * n + gc + (e & 1)];
          if constexpr (kLow) low[n][e] *= sm.row[8 * n + gc + (e & 1)];
        }
#pragma unroll(kLow ? 1 : 4)
      for (int kk = 0; kk < 4; ++kk) {
        if (!has_rows) continue;
        uint32_t va[SP][4];
#pragma unroll
        for (int p = 0; p < SP; ++p)
          ldsm4t(va[p], &sm.v[p][16 * kk + (lane & 7) + ((lane >> 4) & 1) * 8][16 * warp + ((lane >> 3) & 1) * 8]);
#pragma unroll
        for (int n = 0; n < 8; n += 2) {
          // tokens i = 8 n .. 8 n + 15 against j = 16 kk .. 16 kk + 15
          if (a.reverse ? n > 2 * kk + 1 : n + 1 < 2 * kk) continue;
          uint32_t pb[PO][4];
#pragma unroll
          for (int p = 0; p < PO; ++p)
            ldsm4(pb[p], &sm.p[p][8 * n + (lane & 7) + ((lane >> 4) & 1) * 8][16 * kk + ((lane >> 3) & 1) * 8]);
#pragma unroll
          for (int i = SP - 1; i >= 0; --i)
#pragma unroll
            for (int j = PO - 1; j >= 0; --j) {
              if (i + j > 2) continue;
              mma(kLow && i + j ? low[kLow ? n : 0] : acc[n], va[i], pb[j][0], pb[j][1]);
              mma(kLow && i + j ? low[kLow ? n + 1 : 0] : acc[n + 1], va[i], pb[j][2], pb[j][3]);
            }
        }
      }
      join();
      // acc[n][e]: value row r_lo + 8 (e >> 1), token 8 n + gc + (e & 1)
      if (a.dot) {
        const int64_t dp = (int64_t)a.dot_heads * a.PV;
        const int64_t dot0 = t0 * dp + (int64_t)(h / a.dot_div) * a.PV;
        auto dot_at = [&](int i, int r) {  // (outside: any value of the array, unused)
          const int64_t at = dot0 + (int64_t)min(i, rows - 1) * dp + min(r, a.PV - 1);
          return SP == 1 ? to_f(static_cast<const __nv_bfloat16*>(a.dot)[at]) : static_cast<const float*>(a.dot)[at];
        };
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          float w[2][2];
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int x = 0; x < 2; ++x) w[b][x] = dot_at(8 * n + gc + b, r_lo + 8 * x);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int i = 8 * n + gc + b;
            float s = 0.f;
#pragma unroll
            for (int x = 0; x < 2; ++x)
              if (i < rows && r_lo + 8 * x < a.PV) s = fmaf(w[b][x], acc[n][2 * x + b], s);
            s += __shfl_xor_sync(0xffffffffu, s, 4);
            s += __shfl_xor_sync(0xffffffffu, s, 8);
            s += __shfl_xor_sync(0xffffffffu, s, 16);
            if (gr == 0) sm.dots[warp][i] = s;
          }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < rows; i += kThreads)
          a.dots[((int64_t)slice * a.tokens + t0 + i) * a.H + h] =
              (sm.dots[0][i] + sm.dots[1][i]) + (sm.dots[2][i] + sm.dots[3][i]);
      }
      const int64_t op = (int64_t)a.H * a.PV;
      if (SP == 1 && !a.out_f32) {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + t0 * op + (int64_t)h * a.PV + row0 + 16 * warp;
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            // 8 value rows x 8 tokens, turned: this thread gets token 8 n + gr, rows gc, gc + 1
            const uint32_t v = movmatrix(sm100::bf16x2(acc[n][2 * x], acc[n][2 * x + 1]));
            const int i = 8 * n + gr, r = 8 * x + gc, left = a.PV - (row0 + 16 * warp) - r;
            if (i < rows && left > 0) {
              __nv_bfloat16* p = o + i * op + r;
              if (left > 1 && a.PV % 2 == 0)
                *reinterpret_cast<uint32_t*>(p) = v;
              else {
                p[0] = __ushort_as_bfloat16((unsigned short)(v & 0xffffu));
                if (left > 1) p[1] = __ushort_as_bfloat16((unsigned short)(v >> 16));
              }
            }
          }
      } else {
        float* o = static_cast<float*>(a.out) + t0 * op + (int64_t)h * a.PV;
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = 8 * n + gc + (e & 1), r = r_lo + 8 * (e >> 1);
            if (i < rows && r < a.PV) o[i * op + r] = acc[n][e];
          }
      }
    }

    // S <- 2^(c_end) S + (upd o value)^T key, the sum over the block in accumulators of its
    // own: adding 64 tokens at a time in fp32 keeps the tensor core's truncating accumulation
    // from piling up over a long memory.  fp32 operands go by halves of the columns, whose
    // two sets of accumulators fit the registers.
    const float dec = sm.decay;
    constexpr int kPart = kLow ? NTILES / 2 : NTILES;
#pragma unroll
    for (int part = 0; part < NTILES; part += kPart) {
      if (8 * part >= a.NK || !has_rows) continue;
      float add[kPart][4], low[kLow ? kPart : 1][4];
#pragma unroll
      for (int n = 0; n < kPart; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          add[n][e] = 0.f;
          if constexpr (kLow) low[n][e] = 0.f;
        }
#pragma unroll(kLow ? 1 : 4)
      for (int kk = 0; kk < 4; ++kk) {
        uint32_t va[SP][4];
#pragma unroll
        for (int p = 0; p < SP; ++p)
          ldsm4t(va[p], &sm.v[p][16 * kk + (lane & 7) + ((lane >> 4) & 1) * 8][16 * warp + ((lane >> 3) & 1) * 8]);
        const float u0 = sm.upd[16 * kk + gc], u1 = sm.upd[16 * kk + gc + 1];
        const float u2 = sm.upd[16 * kk + gc + 8], u3 = sm.upd[16 * kk + gc + 9];
        uint32_t ua[4][3];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          float x = 0.f, y = 0.f;
#pragma unroll
          for (int p = SP - 1; p >= 0; --p) x += sm100::bf16_lo(va[p][m]), y += sm100::bf16_hi(va[p][m]);
          split2<3>(x * (m < 2 ? u0 : u2), y * (m < 2 ? u1 : u3), ua[m]);
        }
#pragma unroll
        for (int n = 0; n < kPart; n += 2) {
          if (8 * (part + n) >= a.NK) continue;
          uint32_t kb[SP][4];
#pragma unroll
          for (int p = 0; p < SP; ++p)
            ldsm4t(kb[p],
                   &sm.k[p][16 * kk + (lane & 7) + ((lane >> 3) & 1) * 8][8 * (part + n) + ((lane >> 4) & 1) * 8]);
#pragma unroll
          for (int i = 2; i >= 0; --i) {
            const uint32_t af[4] = {ua[0][i], ua[1][i], ua[2][i], ua[3][i]};
#pragma unroll
            for (int j = SP - 1; j >= 0; --j) {
              if (i + j > 2) continue;
              mma(kLow && i + j ? low[kLow ? n : 0] : add[n], af, kb[j][0], kb[j][1]);
              mma(kLow && i + j ? low[kLow ? n + 1 : 0] : add[n + 1], af, kb[j][2], kb[j][3]);
            }
          }
        }
      }
#pragma unroll
      for (int n = 0; n < kPart; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (kLow) add[n][e] += low[n][e];
          st[part + n][e] = fmaf(st[part + n][e], dec, add[n][e]);
        }
    }

    if (a.dump && !a.reverse && (ci == chunks - 1 || ((ci + 1) * kLaChunk) % a.window == 0)) {
      const int64_t w = un.window + ((int64_t)ci * kLaChunk) / a.window;
#pragma unroll
      for (int n = 0; n < NTILES; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = r_lo + 8 * (e >> 1), c = 8 * n + gc + (e & 1);
          if (r < a.PV && c < a.NK) a.dump[((w * a.H + h) * a.PV + r) * a.NK + c] = st[n][e];
        }
    }
  }
  if (a.states_only) {
#pragma unroll
    for (int n = 0; n < NTILES; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = r_lo + 8 * (e >> 1), c = 8 * n + gc + (e & 1);
        if (r < a.PV && c < a.NK) a.carry[(((int64_t)un.window * a.H + h) * a.PV + r) * a.NK + c] = st[n][e];
      }
    if (slice == 0 && threadIdx.x == 0) a.window_decay[(int64_t)un.window * a.H + h] = (float)exp2(total);
    return;
  }
  if (a.last && ends) {
#pragma unroll
    for (int n = 0; n < NTILES; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = r_lo + 8 * (e >> 1), c = 8 * n + gc + (e & 1);
        if (r < a.PV && c < a.NK) a.last[state_at + r * a.sr + c * a.sc] = st[n][e];
      }
  }
}

// Windows of a packed batch: sequence s has max(1, ceil(len / window)) of them, the first at
// first_win[s].  Checks the offsets (the status word and *count = -1 where they are wrong).
__global__ void __launch_bounds__(1024) la_table_kernel(int64_t tokens, int nseq, const int32_t* cu, int window,
                                                        int max_windows, LaTable t, unsigned int* status) {
  __shared__ int s_bad;
  __shared__ int s_warp[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) s_bad = t.count[1] = t.count[2] = 0;
  __syncthreads();
  for (int s = tid; s <= nseq; s += blockDim.x) {
    const int v = cu[s];
    if ((s == 0 && v != 0) || (s == nseq && (int64_t)v != tokens) || (s > 0 && v < cu[s - 1])) atomicOr(&s_bad, 1);
  }
  __syncthreads();
  if (s_bad) {
    if (tid == 0) {
      *t.count = -1;
      atomicOr(status, kStatusBadSeqlens);
    }
    return;
  }
  int carry = 0;
  for (int base = 0; base < nseq; base += blockDim.x) {
    const int s = base + tid;
    const int n = s < nseq ? max(1, (cu[s + 1] - cu[s] + window - 1) / window) : 0;
    int v = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, v, off);
      if (lane >= off) v += x;
    }
    if (lane == 31) s_warp[warp] = v;
    __syncthreads();
    if (warp == 0) {
      int x = s_warp[lane];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
      }
      s_warp[lane] = x;
    }
    __syncthreads();
    if (s < nseq) t.first_win[s] = carry + (warp > 0 ? s_warp[warp - 1] : 0) + v - n;
    carry += s_warp[31];
    __syncthreads();  // s_warp is rewritten by the next round; first_win is read below
  }
  if (tid == 0) t.first_win[nseq] = *t.count = carry;
  // every window by its own thread: its sequence is the last one that starts at or before it
  for (int w = tid; w < carry && w < max_windows; w += blockDim.x) {
    int lo = 0, hi = nseq - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (t.first_win[mid] <= w)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int t0 = cu[lo] + (w - t.first_win[lo]) * window;
    t.win[w] = LaWindow{lo, t0, min(window, cu[lo + 1] - t0)};
  }
}

// carry[w] holds window w's own end state (from zero; the first window's from `start`) and
// becomes the state that window w starts from.  One thread per V (1 or 4 elements) of a state; the
// loads of 8 windows are in flight together (one after another, each behind the last one's
// store, took 130 us for 64 states of 8 windows, and these 20).  A read and a write of every
// state but the last: bound by HBM.
template <typename V>
__global__ void __launch_bounds__(256) la_scan_kernel(LaPass a) {
  if (a.win_count && *a.win_count < 0) return;
  constexpr int kV = sizeof(V) / sizeof(float), kBatch = 8;
  const int64_t sh = blockIdx.x;
  const int seq = a.whole + (int)(sh / a.H), h = (int)(sh % a.H);
  const int64_t size = (int64_t)a.PV * a.NK;
  const int w0 = a.cu ? a.first_win[seq] : seq * a.dense_windows;
  const int n = a.cu ? a.first_win[seq + 1] - w0 : a.dense_windows;
  const int64_t e = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * kV;
  if (e >= size) return;
  const int64_t pitch = (a.reverse ? -1 : 1) * a.H * size;  // from a window to the next in order
  float* p = a.carry + ((int64_t)(a.reverse ? w0 + n - 1 : w0) * a.H + h) * size + e;
  const float* decay = a.window_decay + (int64_t)(a.reverse ? w0 + n - 1 : w0) * a.H + h;
  const int64_t dpitch = (a.reverse ? -1 : 1) * a.H;
  alignas(16) float state[kV];
#pragma unroll
  for (int k = 0; k < kV; ++k) state[k] = 0.f;
  for (int i0 = 0; i0 < n; i0 += kBatch) {
    alignas(16) float own[kBatch][kV];
    float dec[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const bool in = i0 + i + 1 < n;  // the last window's own state is not computed
      dec[i] = in && i0 + i > 0 ? decay[(i0 + i) * dpitch] : 0.f;
      if (in) {
        *reinterpret_cast<V*>(own[i]) = *reinterpret_cast<const V*>(p + (i0 + i) * pitch);
      } else {
#pragma unroll
        for (int k = 0; k < kV; ++k) own[i][k] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      // the first window starts from `start` itself
      if (i0 + i > 0 && i0 + i < n) *reinterpret_cast<V*>(p + (i0 + i) * pitch) = *reinterpret_cast<const V*>(state);
#pragma unroll
      for (int k = 0; k < kV; ++k) state[k] = i0 + i > 0 ? fmaf(state[k], dec[i], own[i][k]) : own[i][k];
    }
  }
}

template <int SP, int PO, int NT>
cudaError_t launch_one(const LaPass& p, cudaStream_t st) {
  auto* fn = la_general_kernel<SP, PO, NT>;
  constexpr size_t bytes = sizeof(Smem<SP, PO, NT>);
  static_assert(bytes <= 227 * 1024, "tiles must fit the SM's shared memory");
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) return e;
  const int slices = la_general_slices(p.PV);
  const int64_t units = la_units(p);
  const int64_t blocks = units * p.H * slices;
  if (blocks == 0) return cudaSuccess;
  fn<<<(unsigned)blocks, kThreads, bytes, st>>>(p, slices);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

int la_general_slices(int PV) { return (PV + kLaSlice - 1) / kLaSlice; }

cudaError_t launch_la_table(int64_t tokens, int nseq, const int32_t* cu, int window, int max_windows, LaTable t,
                            unsigned int* status, cudaStream_t st) {
  la_table_kernel<<<1, 1024, 0, st>>>(tokens, nseq, cu, window, max_windows, t, status);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_la_general(const LaPass& p, bool bf16, bool exact, cudaStream_t st) {
  const bool narrow = p.NK <= 64;
  if (!bf16) return narrow ? launch_one<3, 3, 64>(p, st) : launch_one<3, 3, 128>(p, st);
  if (exact) return narrow ? launch_one<1, 3, 64>(p, st) : launch_one<1, 3, 128>(p, st);
  return narrow ? launch_one<1, 1, 64>(p, st) : launch_one<1, 1, 128>(p, st);
}

cudaError_t launch_la_scan(const LaPass& p, cudaStream_t st) {
  const int64_t size = (int64_t)p.PV * p.NK;
  const bool vec = size % 4 == 0;
  const dim3 grid((unsigned)((int64_t)(p.nseq - p.whole) * p.H), (unsigned)((size / (vec ? 4 : 1) + 255) / 256));
  if (vec)
    la_scan_kernel<float4><<<grid, 256, 0, st>>>(p);
  else
    la_scan_kernel<float><<<grid, 256, 0, st>>>(p);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace ssd
