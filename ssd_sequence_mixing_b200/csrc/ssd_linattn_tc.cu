// ssd_linattn_tc.cu -- the tcgen05 kernel of linear attention with a decay for each head: bf16
// operands whose dimensions are multiples of 8.
//
// The mathematics is that of ssd_linattn.cu: blocks of 64 tokens, everything transposed so that
// the rows of the value dimension are the 128 rows of a product (lanes of tensor memory):
//   S1          = query key^T                          64 x 64,   both from shared memory
//   P           = decay o S1                           to shared memory (bf16)
//   Yi^T        = S query^T                            128 x 64,  S from tensor memory (bf16)
//   Ya^T        = value^T P^T                          128 x 64,  both from shared memory
//   out_i       = row_i Yi_i + Ya_i                    written from tensor memory
//   dS          = (upd o value)^T key                  128 x NK,  three bf16 planes of
//                                                      upd o value from tensor memory
//   S          <- 2^(c_end) S + dS                     S stays in registers, fp32
// dS does not depend on S, so only the last line is a recurrence; everything else of a block
// runs while the previous one finishes.
//
// One CTA per SM takes one head (up to 128 value rows), or two heads of up to 64 rows each
// that share query and key, and walks the blocks of its unit.  28 warps, each with one task, so
// that the tasks of several blocks overlap without any of them being interleaved by hand:
//   load  (1 warp)   query, key, value tiles by TMA, three stages; issues S1
//   dS    (1 warp)   issues the products of dS
//   Y     (1 warp)   issues Yi and Ya (one warp for all products took 110 cycles for each of a
//                    block's 32 and 10 commits, and was what a block's time was made of)
//   gates (1 warp)   the sums of log-decays in 64 bits and the factors from them
//   mask  (4 warps)  S1 -> P
//   decay (8 warps)  value -> the planes of upd o value, by transposing loads
//   state (8 warps)  dS -> S -> the bf16 planes of S
//   out   (4 warps)  Yi, Ya -> out
// Tensor memory (512 columns): S1 64, Yi 64, Ya 64, dS 128, planes of upd o value 2 x 32, planes
// of S 2 x 64 (two heads: Ya 128, S 64).
//
// With PL = 3 P and S enter their products as three bf16 planes each (fp32 accuracy), which
// the per-token dot products behind the decay's gradient need.
//
// Every wait is bounded; one that runs out stops the CTA's roles, which drain what is in
// flight, and SSD_ERR_DEVICE_TIMEOUT is recorded.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "sm100_ptx.cuh"
#include "ssd.h"
#include "ssd_common.cuh"
#include "ssd_linattn.cuh"
#include "ssd_linattn_dev.cuh"
#include "ssd_tc.cuh"

namespace ssd {
namespace {

using namespace sm100;

constexpr int kC = kLaChunk;  // tokens of a block
constexpr int kAtomBytes = kC * 128;  // 64 tokens x 64 columns of bf16, 128-byte rows
constexpr int kMaxStages = 3, kGateSlots = 4, kPlanes = 3;
constexpr int kWarpsTc = 28, kThreadsTc = 32 * kWarpsTc;
constexpr int kLoadWarp = 0, kDsWarp = 1, kGateWarp = 2, kYWarp = 3, kMaskWarp = 4, kDecayWarp = 8, kStateWarp = 16, kOutWarp = 24;

// tensor memory columns
constexpr int kColS1 = 0, kColYi = 64, kColYa = 128, kColDs = 256, kColUv = 384, kColSp0 = 448, kColSp1 = 192;
constexpr int kTmem = 512;
constexpr uint32_t kDrainPolls = 1u << 22;  // (a drain's bound is not the test hooks' to lower)

enum Bar {
  kFull = 0,                     // tiles of a stage have landed
  kReady = kFull + kMaxStages,   // ... and rows past the sequence's end are zero (decay warps)
  kFree = kReady + kMaxStages,      // every product that reads the stage is done
  kS1Full = kFree + kMaxStages, kS1Free,
  kPFull, kPFree = kPFull + 2,
  kUvFull = kPFree + 2, kUvFree = kUvFull + 2,
  kDsFull = kUvFree + 2, kDsFree,
  kSpFull, kSpFree = kSpFull + 2,
  kYFull = kSpFree + 2, kYFree,
  kGFull, kGFree = kGFull + kGateSlots,
  kDrain = kGFree + kGateSlots,  // every product of a warp that issues them is done
  kBars = kDrain + 3
};

struct Gate {
  float chi[kC], clo[kC], row[kC], upd[kC];
  float decay, pad[3];
};

// An output warp's own staging: 64 tokens x 32 rows of bf16 at 80 bytes a token, or 16 tokens of
// fp32 at 144 (neither pitch has bank conflicts); and as much for the rows of the dot products.
constexpr int kOutPitch = 80, kOutPitch32 = 144, kOutBytes = kC * kOutPitch, kDotBytes = kC * kOutPitch;

template <int NT, bool PAIR, int PL>
struct TcSmem {
  static constexpr int kStages = PL > 1 ? 2 : 3;   // (three planes of P leave room for two)
  static constexpr int kPTiles = PAIR ? 2 : PL;    // tiles of P: planes, or one per head
  static constexpr int kHeads = PAIR ? 2 : 1;
  static constexpr int kQ = 0, kK = NT / 64 * kAtomBytes, kV = 2 * kK, kStage = kV + 2 * kAtomBytes;
  static constexpr int kP = kStages * kStage;      // P: two buffers
  static constexpr int kGate = kP + 2 * kPTiles * kAtomBytes;
  static constexpr int kOut = kGate + (int)sizeof(Gate) * kHeads * kGateSlots;  // out warps: staged outputs, ...
  static constexpr int kDot = kOut + 4 * kOutBytes;                              // ... rows to multiply them with
  static constexpr int kBar = kDot + 4 * kDotBytes;
  static constexpr int kFlag = kBar + 8 * kBars;
  static constexpr int kBytes = kFlag + 16 + 1024;                  // 1024: alignment of the base
};

__device__ __forceinline__ void tmem_ld8(uint32_t t, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(t)
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t t, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(t), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t t, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(t)
      : "memory");
}
// 16 lanes x 16 (8) columns in the layout of mma.sync's accumulators: registers 4 t .. 4 t + 3 are
// columns 8 t + 2 (lane % 4), + 1 of row lane / 4, then of row lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x256_x1(uint32_t t, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(t)
               : "memory");
}
__device__ __forceinline__ void tmem_st_16x256_x1(uint32_t t, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x1.b32 [%0], {%1, %2, %3, %4};" ::"r"(t), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void tmem_ld_16x256_x2(uint32_t t, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(t)
               : "memory");
}
// 16 lanes x 16 columns: registers 2 t, 2 t + 1 are column 4 t + lane % 4 of rows lane / 4 and
// lane / 4 + 8 (a pair of bf16 per column: the layout of 8 x 8 matrices from ldmatrix).
__device__ __forceinline__ void tmem_st_16x128_x4(uint32_t t, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(t), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

template <int N>
__device__ __forceinline__ void set_regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Waits for the phase with the given parity, for at most `polls` polls of up to 1 us each (the
// hint; a poll may also return at once).  A tight loop: the waits are a good part of the code, and
// the block loop of all roles together has to stay in the instruction cache.
__device__ __forceinline__ bool wait_polls(uint32_t bar, uint32_t parity, uint32_t polls) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
      "mov.u32 n, %3;\n\t"
      "POLL_%=:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n\t"
      "@p bra DONE_%=;\n\t"
      "sub.u32 n, n, 1;\n\t"
      "setp.ne.u32 q, n, 0;\n\t"
      "@q bra POLL_%=;\n\t"
      "DONE_%=:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(polls)
      : "memory");
  return ok != 0;
}

// 2^c of a sum of log-decays c <= 0 (up to rounding), split as c = hi + lo with hi whole: 2^lo to
// the accuracy of ex2, times an exact power (0 below 2^-126, infinity from 2^128).  A NaN stays one.
__device__ __forceinline__ float exp2_split(double c, float& hi, float& lo) {
  const int whole = min(max(__double2int_rd(c), -100000), 128);
  hi = (float)whole;
  lo = (float)(c - (double)whole);
  return ex2(lo) * (whole < -126 ? 0.f : __int_as_float((whole + 127) << 23));
}

// What every role needs.
struct Cta {
  uint8_t* smem;
  uint64_t* bars;
  volatile int* abort_flag;
  uint32_t polls;
  uint32_t tmem;
  int chunks;
  int64_t t0;
  int len, lane;
  // A whole warp waits for the n-th completion of a barrier (n from 0).  A wait that gives up
  // ends the role; the others' waits run out in turn.
  __device__ __forceinline__ bool wait(int bar, int n) const {
    const bool mine = wait_polls(smem_u32(&bars[bar]), (uint32_t)n & 1u, polls);
    if (!__any_sync(0xffffffffu, !mine)) return true;
    *abort_flag = 1;
    return false;
  }
  // A producer's wait for the slot's consumers; use number n (from 0) of the slot.
  __device__ __forceinline__ bool wait_free(int bar, int n) const { return n == 0 || wait(bar, n - 1); }
  // One arrival for the warp, after every lane's accesses.
  __device__ __forceinline__ void arrive(int bar) const {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[bar]);
  }
  // The block processed at step c: its first token and its tokens.
  __device__ __forceinline__ int64_t token(const LaPass& a, int c) const {
    return t0 + (int64_t)(a.reverse ? chunks - 1 - c : c) * kC;
  }
  __device__ __forceinline__ int rows(const LaPass& a, int c) const {
    return min(kC, len - (a.reverse ? chunks - 1 - c : c) * kC);
  }
};

// What the three warps that issue products share.
struct Issue {
  const Cta& t;
  bool leader;
  uint64_t k_major, mn_major;  // descriptors of shared-memory tiles, without the address
  uint32_t base;
  __device__ __forceinline__ explicit Issue(const Cta& cta)
      : t(cta), leader(elect_one()), k_major(sdesc_sw128(0, 16, 1024)), mn_major(sdesc_sw128(0, kAtomBytes, 1024)),
        base(smem_u32(cta.smem)) {}
  __device__ __forceinline__ uint64_t at(uint64_t major, int off) const { return major | (uint64_t)((base + off) >> 4); }
  // K step kk of a K-major tile of 64-column atoms
  static __device__ __forceinline__ uint64_t koff(int kk) { return (uint64_t)(((kk >> 2) * kAtomBytes + (kk & 3) * 32) >> 4); }
  // Arrives on the barrier once every product this warp has issued so far is done.
  __device__ __forceinline__ void commit(int bar) const {
    if (leader) umma_commit(&t.bars[bar]);
    __syncwarp();
  }
  __device__ __forceinline__ void drain(int bar) const {
    commit(bar);
    if (!wait_polls(smem_u32(&t.bars[bar]), 0, kDrainPolls)) *t.abort_flag = 1;
  }
};

// Tiles by TMA, and S1 of each block.
template <int NT, bool PAIR, int PL>
__device__ __forceinline__ void load_role(const Cta& t, const LaPass& a, const CUtensorMap* tq, const CUtensorMap* tk,
                                          const CUtensorMap* tv, int h0, int withhold) {
  using L = TcSmem<NT, PAIR, PL>;
  const Issue mma(t);
  const int qh = h0 / a.q_div, kh = h0 / a.k_div, vh = h0 / a.v_div;  // (two heads: v_div is 1)
  const int v_atoms = PAIR || a.PV > 64 ? 2 : 1;
  const uint32_t bytes = ((a.states_only ? 1 : 2) * (NT / 64) + v_atoms) * kAtomBytes;
  constexpr uint32_t id_s1 = idesc_bf16(64, kC, 0, 0);
  constexpr int kAhead = L::kStages - 1;  // blocks loaded before they are needed
  bool ok = true;
  int s = 0, use = 0, ls = 0, luse = 0;  // stage and its use: of the products, of the loads
#pragma unroll 1
  for (int c = -kAhead; c < t.chunks; ++c) {
    if (c >= 0 && !a.states_only) {
      // the tiles as they landed: what a last block holds past its end is masked in P
      if (!(ok = t.wait(kFull + s, use)) || !(ok = t.wait_free(kS1Free, c))) break;
      tc_fence_after();
      if (mma.leader) {
        const uint64_t q = mma.at(mma.k_major, s * L::kStage + L::kQ), k = mma.at(mma.k_major, s * L::kStage + L::kK);
#pragma unroll
        for (int kk = 0; kk < NT / 16; ++kk)
          umma_f16(t.tmem + kColS1, q + Issue::koff(kk), k + Issue::koff(kk), id_s1, kk > 0);
      }
      __syncwarp();
      if (!withhold) mma.commit(kS1Full);
      if (++s == L::kStages) s = 0, ++use;
    }
    if (c + kAhead >= t.chunks) continue;
    if (!(ok = t.wait_free(kFree + ls, luse))) break;
    if (t.lane == 0) {
      uint64_t* bar = &t.bars[kFull + ls];
      uint8_t* to = t.smem + ls * L::kStage;
      const int tok = (int)t.token(a, c + kAhead);
      mbar_expect_tx(bar, bytes);
#pragma unroll
      for (int i = 0; i < NT / 64; ++i) tma_load_3d(to + L::kK + i * kAtomBytes, tk, 64 * i, kh, tok, bar);
      if (!a.states_only) {
#pragma unroll
        for (int i = 0; i < NT / 64; ++i) tma_load_3d(to + L::kQ + i * kAtomBytes, tq, 64 * i, qh, tok, bar);
      }
      tma_load_3d(to + L::kV, tv, 0, vh, tok, bar);
      if (v_atoms == 2) tma_load_3d(to + L::kV + kAtomBytes, tv, PAIR ? 0 : 64, PAIR ? vh + 1 : vh, tok, bar);
    }
    __syncwarp();
    if (++ls == L::kStages) ls = 0, ++luse;
  }
  mma.drain(kDrain);
  // after a failure: what was issued lands before the CTA ends
  if (!ok)
#pragma unroll 1
    for (int d = 0; d < L::kStages; ++d) {
      const int n = luse - (d >= ls);  // the last use of stage d that was loaded
      if (n >= 0) wait_polls(smem_u32(&t.bars[kFull + d]), (uint32_t)n & 1u, kDrainPolls);
    }
}

// dS = (upd o value)^T key, plane by plane.
template <int NT, bool PAIR, int PL>
__device__ __forceinline__ void ds_role(const Cta& t, const LaPass& a) {
  using L = TcSmem<NT, PAIR, PL>;
  const Issue mma(t);
  constexpr uint32_t id_ds = idesc_bf16(128, NT, 0, 1);
  bool ok = true;
  int s = 0, use = 0;
#pragma unroll 1
  for (int c = 0; ok && c < t.chunks; ++c) {
    if (!(ok = t.wait(kReady + s, use)) || !(ok = t.wait(kDsFree, c))) break;  // (the first time: S is loaded)
    const uint64_t k_mn = mma.at(mma.mn_major, s * L::kStage + L::kK);
#pragma unroll 1
    for (int p = 0; p < kPlanes; ++p) {
      const int m = kPlanes * c + p, slot = m & 1;
      if (!(ok = t.wait(kUvFull + slot, m >> 1))) break;
      tc_fence_after();
      if (mma.leader) {
#pragma unroll
        for (int kk = 0; kk < kC / 16; ++kk)
          umma_f16_ta(t.tmem + kColDs, t.tmem + kColUv + slot * 32 + kk * 8, k_mn + kk * 128, id_ds, p > 0 || kk > 0);
      }
      __syncwarp();
      mma.commit(kUvFree + slot);
    }
    if (!ok) break;
    mma.commit(kDsFull);
    mma.commit(kFree + s);
    if (++s == L::kStages) s = 0, ++use;
  }
  mma.drain(kDrain + 1);
}

// Yi^T = S query^T and Ya^T = value^T P^T.
template <int NT, bool PAIR, int PL>
__device__ __forceinline__ void y_role(const Cta& t, const LaPass& a) {
  using L = TcSmem<NT, PAIR, PL>;
  const Issue mma(t);
  constexpr uint32_t id_yi = idesc_bf16(128, kC, 0, 0), id_ya = idesc_bf16(128, PAIR ? 2 * kC : kC, 1, 0);
  constexpr int sp_slots = PAIR ? 1 : 2;
  bool ok = true;
  int s = 0, use = 0;
#pragma unroll 1
  for (int c = 0; ok && c < t.chunks; ++c) {
    if (!(ok = t.wait(kFull + s, use)) || !(ok = t.wait_free(kYFree, c))) break;
    const uint64_t q = mma.at(mma.k_major, s * L::kStage + L::kQ);
#pragma unroll 1
    for (int p = 0; p < PL; ++p) {
      const int m = PL * c + p, slot = m % sp_slots;
      if (!(ok = t.wait(kSpFull + slot, m / sp_slots))) break;
      tc_fence_after();
      if (mma.leader) {
        const uint32_t sp = t.tmem + (slot ? kColSp1 : kColSp0);
#pragma unroll
        for (int kk = 0; kk < NT / 16; ++kk)
          umma_f16_ta(t.tmem + kColYi, sp + kk * 8, q + Issue::koff(kk), id_yi, p > 0 || kk > 0);
      }
      __syncwarp();
      mma.commit(kSpFree + slot);
    }
    if (!ok) break;
    if (!(ok = t.wait(kReady + s, use)) || !(ok = t.wait(kPFull + (c & 1), c >> 1))) break;
    tc_fence_after();
    if (mma.leader) {
      const uint64_t v_mn = mma.at(mma.mn_major, s * L::kStage + L::kV);
#pragma unroll 1
      for (int p = 0; p < PL; ++p) {
        const uint64_t pm = mma.at(mma.k_major, L::kP + ((c & 1) * L::kPTiles + p) * kAtomBytes);
#pragma unroll
        for (int kk = 0; kk < kC / 16; ++kk)
          umma_f16(t.tmem + kColYa, v_mn + kk * 128, pm + kk * 2, id_ya, p > 0 || kk > 0);
      }
    }
    __syncwarp();
    mma.commit(kPFree + (c & 1));
    mma.commit(kYFull);
    mma.commit(kFree + s);  // (S1 of this block was done before its P)
    if (++s == L::kStages) s = 0, ++use;
  }
  mma.drain(kDrain + 2);
}

// One head: lane l takes tokens 2 l, 2 l + 1 of each block.  Two: half a warp each, 4 tokens a lane.
template <int NT, bool PAIR, int PL>
__device__ __forceinline__ void gate_role(const Cta& t, const LaPass& a, int h0, int unit) {
  using L = TcSmem<NT, PAIR, PL>;
  constexpr int kLanes = 32 / L::kHeads, kTok = kC / kLanes;
  const int which = PAIR ? t.lane >> 4 : 0, l = t.lane & (kLanes - 1), i0 = kTok * l, h = h0 + which;
  const float sr = a.reverse ? 1.f : a.scale, su = a.reverse ? a.scale : 1.f;
  const float* from = a.log_decay + h;
  double total = 0.0;
  float x[kTok];
  auto load = [&](int c) {
    if (c >= t.chunks) return;
    const int64_t tok = t.token(a, c) + i0;
    const int left = t.rows(a, c) - i0;
#pragma unroll
    for (int j = 0; j < kTok; ++j) x[j] = j < left ? from[a.per_token ? (tok + j) * a.H : 0] : 0.f;
  };
  load(0);
#pragma unroll 1
  for (int c = 0; c < t.chunks; ++c) {
    double sum[kTok];  // inclusive sums from the block's start
#pragma unroll
    for (int j = 0; j < kTok; ++j) sum[j] = log2_clamped(x[j]) + (j ? sum[j - 1] : 0.0);
    load(c + 1);
    double before = sum[kTok - 1];
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) {
      const double v = __shfl_up_sync(0xffffffffu, before, o, kLanes);
      if (l >= o) before += v;
    }
    const double end = __shfl_sync(0xffffffffu, before, kLanes - 1, kLanes);
    before -= sum[kTok - 1];
    const int slot = c % kGateSlots;
    if (!t.wait_free(kGFree + slot, c / kGateSlots)) return;
    Gate* g = reinterpret_cast<Gate*>(t.smem + L::kGate) + slot * L::kHeads + which;
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      const double cc = before + sum[j];
      float hi, lo;
      const float from_start = exp2_split(cc, hi, lo);
      g->chi[i0 + j] = hi, g->clo[i0 + j] = lo;
      const float to_end = exp2_split(end - cc, hi, lo);
      g->row[i0 + j] = (a.reverse ? to_end : from_start) * sr;
      g->upd[i0 + j] = (a.reverse ? from_start : to_end) * su;
    }
    if (l == 0) {
      float hi, lo;
      g->decay = exp2_split(end, hi, lo);
    }
    total += end;
    t.arrive(kGFull + slot);
  }
  if (a.states_only && l == 0) {
    float hi, lo;
    a.window_decay[(int64_t)unit * a.H + h] = exp2_split(total, hi, lo);
  }
}

// S1 -> P.  Warp q holds rows 16 q .. 16 q + 15 of S1 (lanes 0 .. 15 of its quarter of tensor
// memory: a product of 64 rows puts 16 in each quarter).
template <int NT, bool PAIR, int PL>
__device__ __forceinline__ void mask_role(const Cta& t, const LaPass& a) {
  constexpr int planes = PL;
  using L = TcSmem<NT, PAIR, PL>;
  const int q = threadIdx.x / 32 & 3;
  const int gr = t.lane >> 2, gc = (t.lane & 3) * 2;
  const int i0 = 16 * q + gr;
  uint8_t* P = t.smem + L::kP;
  const int sign = a.reverse ? -1 : 1;
  const float fsign = (float)sign;
  auto put = [&](uint8_t* tile, int i, int j, uint32_t v) {
    *reinterpret_cast<uint32_t*>(tile + sw128_off(i, j >> 3) + (j & 7) * 2) = v;
  };
  if (!a.states_only) {  // the tiles above the diagonal stay zero
#pragma unroll 1
    for (int n = 0; n < 8; ++n)
#pragma unroll 1
      for (int p = 0; p < 2 * L::kPTiles; ++p) {
        put(P + p * kAtomBytes, i0, 8 * n + gc, 0u);
        put(P + p * kAtomBytes, i0 + 8, 8 * n + gc, 0u);
      }
  }
#pragma unroll 1
  for (int c = 0; c < t.chunks; ++c) {
    const int slot = c % kGateSlots;
    if (!t.wait(kGFull + slot, c / kGateSlots)) return;
    if (!a.states_only) {
      const Gate* g = reinterpret_cast<const Gate*>(t.smem + L::kGate) + slot * L::kHeads;
      if (!t.wait(kS1Full, c) || !t.wait_free(kPFree + (c & 1), c >> 1)) return;
      tc_fence_after();
      // the column tiles with any j in reach, two at a time
      const int b0 = a.reverse ? q : 0, b1 = a.reverse ? 4 : q + 1;
#pragma unroll 1
      for (int b = b0; b < b1; ++b) {
        uint32_t r[8];
        tmem_ld_16x256_x2(t.tmem + ((uint32_t)(32 * q) << 16) + kColS1 + 16 * b, r);
        tmem_ld_wait();
#pragma unroll
        for (int hh = 0; hh < L::kHeads; ++hh) {
          const float hi0 = g[hh].chi[i0], hi1 = g[hh].chi[i0 + 8], lo0 = g[hh].clo[i0], lo1 = g[hh].clo[i0 + 8];
#pragma unroll
          for (int nn = 0; nn < 2; ++nn) {
            const int j = 16 * b + 8 * nn + gc;
            const float2 hj = *reinterpret_cast<const float2*>(&g[hh].chi[j]);
            const float2 lj = *reinterpret_cast<const float2*>(&g[hh].clo[j]);
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float dh = (e >> 1 ? hi1 : hi0) - (e & 1 ? hj.y : hj.x);
              const float dl = (e >> 1 ? lo1 : lo0) - (e & 1 ? lj.y : lj.x);
              const int ahead = i0 + 8 * (e >> 1) - j - (e & 1);  // i - j
              v[e] = sign * ahead >= 0 ? __uint_as_float(r[4 * nn + e]) * ex2(fsign * (dh + dl)) * a.scale : 0.f;
            }
#pragma unroll
            for (int p = 0; p < planes; ++p) {
              const uint32_t x = bf16x2(v[0], v[1]), y = bf16x2(v[2], v[3]);
              uint8_t* tile = P + ((c & 1) * L::kPTiles + (PAIR ? hh : p)) * kAtomBytes;
              put(tile, i0, j, x);
              put(tile, i0 + 8, j, y);
              v[0] -= bf16_lo(x), v[1] -= bf16_hi(x), v[2] -= bf16_lo(y), v[3] -= bf16_hi(y);
            }
          }
        }
      }
      tc_fence_before();
      t.arrive(kS1Free);
      fence_proxy_async();
      t.arrive(kPFull + (c & 1));
    }
    t.arrive(kGFree + slot);
  }
}

// value -> the planes of upd o value in tensor memory, transposed on the way.  Warp w makes rows
// 32 (w % 4) .. and half of the block's tokens.
template <int NT, bool PAIR, int PL>
__device__ __forceinline__ void decay_role(const Cta& t, const LaPass& a) {
  using L = TcSmem<NT, PAIR, PL>;
  const int w = threadIdx.x / 32 - kDecayWarp, q = w & 3, half = w >> 2, lane = t.lane;
  const int head = PAIR ? q >> 1 : 0;
  const bool active = (PAIR ? 32 * q & 63 : 32 * q) < a.PV;
  int s = 0, use = 0;
#pragma unroll 1
  for (int c = 0; c < t.chunks; ++c) {
    const int slot = c % kGateSlots, rows = t.rows(a, c);
    uint8_t* tiles = t.smem + s * L::kStage;
    if (!t.wait(kFull + s, use)) return;
    if (rows < kC) {
      // the sequence ends inside the block: what follows is another's, and 0 * NaN is NaN.  A
      // row of key and value is 8 pieces of 16 bytes in each of up to 4 atoms
      constexpr int kAtoms = NT / 64 + 2;
#pragma unroll 1
      for (int i = rows + w; i < kC; i += 8)
        if (lane < 8 * kAtoms)
          *reinterpret_cast<uint4*>(tiles + L::kK + (lane >> 3) * kAtomBytes + i * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
      fence_proxy_async();
    }
    t.arrive(kReady + s);
    if (rows < kC && !t.wait(kReady + s, use)) return;
    if (++s == L::kStages) s = 0, ++use;
    if (!t.wait(kGFull + slot, c / kGateSlots)) return;
    const float* u = (reinterpret_cast<const Gate*>(t.smem + L::kGate) + slot * L::kHeads + head)->upd + 32 * half;
    float x[2][8][2];  // [half of the rows][4 k step of 16 tokens + matrix][token of the pair]
    if (active) {
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const int j = 32 * half + 16 * kk + (lane & 7) + ((lane >> 4) & 1) * 8;
        const float2 ua = *reinterpret_cast<const float2*>(&u[16 * kk + 2 * (lane & 3)]);
        const float2 ub = *reinterpret_cast<const float2*>(&u[16 * kk + 8 + 2 * (lane & 3)]);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int p = 32 * q + 16 * hf + ((lane >> 3) & 1) * 8;
          uint32_t v[4];
          asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                       : "r"(smem_u32(tiles + L::kV + (p >> 6) * kAtomBytes + sw128_off(j, (p & 63) >> 3)))
                       : "memory");
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            x[hf][4 * kk + m][0] = bf16_lo(v[m]) * (m < 2 ? ua.x : ub.x);
            x[hf][4 * kk + m][1] = bf16_hi(v[m]) * (m < 2 ? ua.y : ub.y);
          }
        }
      }
    }
    t.arrive(kGFree + slot);
#pragma unroll 1
    for (int p = 0; p < kPlanes; ++p) {
      const int m = kPlanes * c + p, us = m & 1;
      if (!t.wait_free(kUvFree + us, m >> 1)) return;
      tc_fence_after();
      if (active) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[i] = bf16x2(x[hf][i][0], x[hf][i][1]);
            x[hf][i][0] -= bf16_lo(v[i]), x[hf][i][1] -= bf16_hi(v[i]);
          }
          tmem_st_16x128_x4(t.tmem + ((uint32_t)(32 * q + 16 * hf) << 16) + kColUv + 32 * us + 16 * half, v);
        }
        tmem_st_wait();
      }
      tc_fence_before();
      t.arrive(kUvFull + us);
    }
  }
}

// Where a state lies in memory: element (r, n) of the head at base + r * sr + n * sc.
struct StateAt {
  float* base;
  int64_t sr, sc;
};

// Moves the warp's 32 rows from row0 and NC columns from n0 between memory and the columns of dS
// in tensor memory (`ds`; no product uses them at that time), in small loops.  Rows are
// contiguous in memory (sc = 1: 8 rows x 32 bytes an access) or columns are (a lane per row).
template <int NC, bool STORE>
__device__ __forceinline__ void move_state(uint32_t ds, const StateAt& at, int lane, int row0, int n0, int rows, int cols) {
  if (at.sc == 1) {
    const int r0 = row0 + (lane >> 2), c0 = n0 + 2 * (lane & 3);
#pragma unroll 1
    for (int i = 0; i < NC / 4; ++i) {  // 8 columns, half of the rows
      const int r = r0 + 16 * (i & 1), n = 8 * (i >> 1);
      const uint32_t t = ds + ((uint32_t)(16 * (i & 1)) << 16) + n;
      float* p = at.base + r * at.sr + c0 + n;
      const bool in = c0 + n < cols, lo = in && r < rows, hi = in && r + 8 < rows;  // (both even)
      uint32_t v[4] = {0u, 0u, 0u, 0u};
      if (STORE) {
        tmem_ld_16x256_x1(t, v);
        tmem_ld_wait();
        if (lo) *reinterpret_cast<uint2*>(p) = make_uint2(v[0], v[1]);
        if (hi) *reinterpret_cast<uint2*>(p + 8 * at.sr) = make_uint2(v[2], v[3]);
      } else {
        if (lo) *reinterpret_cast<uint2*>(&v[0]) = *reinterpret_cast<const uint2*>(p);
        if (hi) *reinterpret_cast<uint2*>(&v[2]) = *reinterpret_cast<const uint2*>(p + 8 * at.sr);
        tmem_st_16x256_x1(t, v);
      }
    }
  } else {
    float* p = at.base + (row0 + lane) * at.sr + n0 * at.sc;
#pragma unroll 1
    for (int n = 0; n < NC; n += 8) {
      uint32_t v[8];
      if (STORE) {
        tmem_ld8(ds + n, v);
        tmem_ld_wait();
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool in = row0 + lane < rows && n0 + n + i < cols;
        if (!STORE)
          v[i] = in ? __float_as_uint(p[(n + i) * at.sc]) : 0u;
        else if (in)
          p[(n + i) * at.sc] = __uint_as_float(v[i]);
      }
      if (!STORE) tmem_st8(ds + n, v);
    }
  }
  if (!STORE) tmem_st_wait();
}
template <int NC>
__device__ __forceinline__ void put_state(uint32_t ds, const float (&S)[NC], const StateAt& at, int lane, int row0, int n0,
                                          int rows, int cols) {
#pragma unroll
  for (int b = 0; b < NC / 16; ++b) {
    uint32_t v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(S[16 * b + i]);
    tmem_st16(ds + 16 * b, v);
  }
  tmem_st_wait();
  move_state<NC, true>(ds, at, lane, row0, n0, rows, cols);
}

// Plane p of the state that step c's outputs see, to tensor memory.
template <int NT, bool PAIR, int PL>
__device__ __forceinline__ bool put_plane(const Cta& t, const float (&S)[NT / 2], bool active, uint32_t lanes, int half,
                                          int c, int p) {
  constexpr int NC = NT / 2, slots = PAIR ? 1 : 2;
  const int m = PL * c + p, slot = m % slots;
  if (!t.wait_free(kSpFree + slot, m / slots)) return false;
  tc_fence_after();
  if (active) {
    const uint32_t to = t.tmem + lanes + (slot ? kColSp1 : kColSp0) + half * (NC / 2);
#pragma unroll
    for (int b = 0; b < NC / 32; ++b) {
      uint32_t v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float x = S[32 * b + 2 * i], y = S[32 * b + 2 * i + 1];
        v[i] = bf16x2(x, y);
#pragma unroll
        for (int k = 0; k < PL - 1; ++k) {
          if (k >= p) break;
          x -= bf16_lo(v[i]), y -= bf16_hi(v[i]);
          v[i] = bf16x2(x, y);
        }
      }
      tmem_st16(to + 16 * b, v);
    }
    tmem_st_wait();
  }
  tc_fence_before();
  t.arrive(kSpFull + slot);
  return true;
}

// S in registers: warp w (of 8) holds rows 32 (w % 4) .. and half of the columns.
template <int NT, bool PAIR, int PL>
__device__ __forceinline__ void state_role(const Cta& t, const LaPass& a, const Unit& un, int u, int h0) {
  using L = TcSmem<NT, PAIR, PL>;
  constexpr int NC = NT / 2, sp_slots = PAIR ? 1 : 2;  // columns of a thread
  const int w = threadIdx.x / 32 - kStateWarp, q = w & 3, half = w >> 2;
  const int head = PAIR ? q >> 1 : 0, h = h0 + head;
  const int row0 = PAIR ? 32 * q & 63 : 32 * q;  // the warp's first row of the head
  const bool active = row0 < a.PV;
  const int n0 = half * NC;
  const bool begins = a.reverse ? un.last : un.first, ends = a.reverse ? un.first : un.last;
  const uint32_t lanes = (uint32_t)(32 * q) << 16;
  const int64_t state_at = ((int64_t)un.seq * a.H + h) * a.NK * a.PV;
  const uint32_t ds = t.tmem + lanes + kColDs + n0;  // the thread's part of dS
  auto window_at = [&](float* base, int64_t win) {
    return StateAt{base + (win * a.H + h) * a.PV * a.NK, (int64_t)a.NK, 1};
  };
  float S[NC];
  {
    StateAt from{nullptr, a.NK, 1};
    if (!begins && !a.states_only)
      from = window_at(a.carry, u);
    else if (begins && a.start)
      from = StateAt{const_cast<float*>(a.start) + state_at, a.sr, a.sc};
    move_state<NC, false>(ds, from, t.lane, row0, n0, from.base ? a.PV : 0, a.NK);
#pragma unroll
    for (int b = 0; b < NC / 16; ++b) {
      uint32_t v[16];
      tmem_ld16(ds + 16 * b, v);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) S[16 * b + i] = __uint_as_float(v[i]);
    }
  }
  // windows whose state is wanted: forward, after the window's last block; reverse, before it
  auto wanted = [&](int ci) { return a.dump && (ci == t.chunks - 1 || (ci + 1) * kC % a.window == 0); };
  auto dump_at = [&](int ci) { return window_at(a.dump, un.first_window + ci * kC / a.window); };
  if (a.reverse && t.chunks && wanted(t.chunks - 1)) put_state<NC>(ds, S, dump_at(t.chunks - 1), t.lane, row0, n0, a.PV, a.NK);
  tc_fence_before();
  t.arrive(kDsFree);
  if (!a.states_only && t.chunks)
#pragma unroll
    for (int p = 0; p < PL; ++p)
      if (!put_plane<NT, PAIR, PL>(t, S, active, lanes, half, 0, p)) return;
#pragma unroll 1
  for (int c = 0; c < t.chunks; ++c) {
    const int ci = a.reverse ? t.chunks - 1 - c : c;
    if (!t.wait(kGFull + c % kGateSlots, c / kGateSlots)) return;
    const float dec = (reinterpret_cast<const Gate*>(t.smem + L::kGate) + (c % kGateSlots) * L::kHeads + head)->decay;
    const bool more = !a.states_only && c + 1 < t.chunks;
    const int m = PL * (c + 1), slot = m % sp_slots;  // the next step's first plane goes out as S is made
    if (!t.wait(kDsFull, c) || (more && !t.wait_free(kSpFree + slot, m / sp_slots))) return;
    tc_fence_after();
    const uint32_t sp = t.tmem + lanes + (slot ? kColSp1 : kColSp0) + half * (NC / 2);
#pragma unroll
    for (int b = 0; b < NC / 16; ++b) {
      uint32_t d[16], v[8];
      tmem_ld16(ds + 16 * b, d);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) S[16 * b + i] = fmaf(S[16 * b + i], dec, __uint_as_float(d[i]));
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = bf16x2(S[16 * b + 2 * i], S[16 * b + 2 * i + 1]);
      if (more) tmem_st8(sp + 8 * b, v);
    }
    const int at = a.reverse ? ci - 1 : ci;  // the block whose window's state this may be
    if (at >= 0 && wanted(at)) put_state<NC>(ds, S, dump_at(at), t.lane, row0, n0, a.PV, a.NK);
    tc_fence_before();
    t.arrive(kDsFree);
    t.arrive(kGFree + c % kGateSlots);
    if (more) {
      tmem_st_wait();
      tc_fence_before();
      t.arrive(kSpFull + slot);
#pragma unroll
      for (int p = 1; p < PL; ++p)
        if (!put_plane<NT, PAIR, PL>(t, S, active, lanes, half, c + 1, p)) return;
    }
  }
  if (a.states_only)
    put_state<NC>(ds, S, window_at(a.carry, u), t.lane, row0, n0, a.PV, a.NK);
  else if (a.last && ends)
    put_state<NC>(ds, S, StateAt{a.last + state_at, a.sr, a.sc}, t.lane, row0, n0, a.PV, a.NK);
}

// Yi, Ya -> out: warp q writes rows 32 q .., 16 tokens at a time.  Tensor memory is read in the layout of mma.sync's accumulators (registers are pairs of
// tokens of one row), turned by transposing stores to shared memory, and written from there
// in 16-byte pieces (single 2-byte stores took 16 cycles each, 5 of a block's 9 thousand).
template <int NT, bool PAIR, int PL>
__device__ __forceinline__ void out_role(const Cta& t, const LaPass& a, int h0) {
  using L = TcSmem<NT, PAIR, PL>;
  const int q = threadIdx.x / 32 & 3;
  const int head = PAIR ? q >> 1 : 0, h = h0 + head;
  const int row0 = PAIR ? 32 * q & 63 : 32 * q;  // the warp's first row of the head
  const bool active = row0 < a.PV;
  const uint32_t lanes = (uint32_t)(32 * q) << 16;
  uint8_t* stage = t.smem + L::kOut + q * kOutBytes;
  uint8_t* dots_in = t.smem + L::kDot + q * kDotBytes;
  // The rows that step c's outputs are multiplied with, on their way while its products run.
  auto fetch_dots = [&](int c) {
    const int64_t tok = t.token(a, c);
    const int rows = t.rows(a, c);
    const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(a.dot) + (tok * a.dot_heads + h / a.dot_div) * a.PV + row0;
#pragma unroll 1
    for (int k = 0; k < 8; ++k) {
      const int i = 8 * k + (t.lane >> 2), p = (t.lane & 3) * 8;
      const bool in = i < rows && row0 + p < a.PV;
      const void* src = in ? from + (int64_t)i * a.dot_heads * a.PV + p : static_cast<const __nv_bfloat16*>(a.dot);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dots_in + i * kOutPitch + p * 2)),
                   "l"(src), "r"(in ? 16 : 0)
                   : "memory");
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int c = 0; c < t.chunks; ++c) {
    if constexpr (PL > 1) fetch_dots(c);
    const float* rowf = (reinterpret_cast<const Gate*>(t.smem + L::kGate) + (c % kGateSlots) * L::kHeads + head)->row;
    if (!t.wait(kGFull + c % kGateSlots, c / kGateSlots) || !t.wait(kYFull, c)) return;
    tc_fence_after();
    const int64_t tok = t.token(a, c);
    const int rows = t.rows(a, c);
    const int64_t pitch = (int64_t)a.H * a.PV, at = tok * pitch + (int64_t)h * a.PV + row0;
    const int gr = t.lane >> 2, gc = (t.lane & 3) * 2;
    if constexpr (PL > 1) {
      cp_async_wait_all();
      __syncwarp();
    }
    // Everything is read, and Yi and Ya are free for the next block's products, before anything
    // goes to memory: the products and this reading alternate, and are most of a block's time.
#pragma unroll 1
    for (int b = 0; b < 4; ++b) {
      uint32_t yi[2][8], ya[2][8];
      if (active) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint32_t from = t.tmem + lanes + ((uint32_t)(16 * hf) << 16) + 16 * b;
          tmem_ld_16x256_x2(from + kColYi, yi[hf]);
          tmem_ld_16x256_x2(from + kColYa + (PAIR ? kC * head : 0), ya[hf]);
        }
        tmem_ld_wait();
      }
      if (b == 3) {
        tc_fence_before();
        t.arrive(kYFree);
      }
      const float2 f0 = *reinterpret_cast<const float2*>(&rowf[16 * b + gc]);
      const float2 f1 = *reinterpret_cast<const float2*>(&rowf[16 * b + 8 + gc]);
      float o[2][8];  // [half of the rows][4 tile of 8 tokens + 2 (row + 8) + token of the pair]
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          o[hf][e] = fmaf(__uint_as_float(yi[hf][e]), e < 4 ? (e & 1 ? f0.y : f0.x) : (e & 1 ? f1.y : f1.x),
                          __uint_as_float(ya[hf][e]));
      if (!a.out_f32) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint8_t* to = stage + (16 * b + 8 * (t.lane >> 4) + (t.lane & 7)) * kOutPitch + 32 * hf + 16 * ((t.lane >> 3) & 1);
          asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(smem_u32(to)),
                       "r"(bf16x2(o[hf][0], o[hf][1])), "r"(bf16x2(o[hf][2], o[hf][3])),
                       "r"(bf16x2(o[hf][4], o[hf][5])), "r"(bf16x2(o[hf][6], o[hf][7]))
                       : "memory");
        }
      } else if (active) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<float*>(stage + (8 * (e >> 2) + gc + (e & 1)) * kOutPitch32 +
                                      (16 * hf + 8 * ((e >> 1) & 1) + gr) * 4) = o[hf][e];
        __syncwarp();
        float* to = static_cast<float*>(a.out) + at + 16 * b * pitch;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = 4 * k + (t.lane >> 3), p = (t.lane & 7) * 4;
          const float4 v = *reinterpret_cast<const float4*>(stage + i * kOutPitch32 + p * 4);
          if (16 * b + i < rows && row0 + p < a.PV) *reinterpret_cast<float4*>(to + i * pitch + p) = v;
        }
        __syncwarp();
      }
      if constexpr (PL > 1)
        if (active) {  // sums over the warp's rows of out * dot, for the decay's gradient
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t v[4];
          const uint8_t* from = dots_in + (16 * b + 8 * (t.lane >> 4) + (t.lane & 7)) * kOutPitch + 32 * hf + 16 * ((t.lane >> 3) & 1);
          asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                       : "r"(smem_u32(from))
                       : "memory");
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            sum[2 * (m >> 1)] = fmaf(o[hf][2 * m], bf16_lo(v[m]), sum[2 * (m >> 1)]);
            sum[2 * (m >> 1) + 1] = fmaf(o[hf][2 * m + 1], bf16_hi(v[m]), sum[2 * (m >> 1) + 1]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 4);
          sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 8);
          sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 16);
        }
        // lanes 0 .. 3 have tokens gc, gc + 1, gc + 8, gc + 9; lane 4 m + l writes the m-th
        const int m = t.lane >> 2, i = 16 * b + gc + (m & 1) + 8 * (m >> 1);
        if (m < 4 && i < rows)
          a.dots[((int64_t)q * a.tokens + tok + i) * a.H + h] = m == 0 ? sum[0] : m == 1 ? sum[1] : m == 2 ? sum[2] : sum[3];
      }
    }
    t.arrive(kGFree + c % kGateSlots);
    if (!active || a.out_f32) continue;
    __syncwarp();
    __nv_bfloat16* to = static_cast<__nv_bfloat16*>(a.out) + at;
#pragma unroll 4
    for (int k = 0; k < 8; ++k) {
      const int i = 8 * k + gr, p = (t.lane & 3) * 8;
      const uint4 v = *reinterpret_cast<const uint4*>(stage + i * kOutPitch + p * 2);
      if (i < rows && row0 + p < a.PV) *reinterpret_cast<uint4*>(to + i * pitch + p) = v;
    }
    __syncwarp();
  }
}

// Grid: units x heads (or pairs of heads), heads fastest.
template <int NT, bool PAIR, int PL>
__global__ void __launch_bounds__(kThreadsTc, 1)
    la_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                 const __grid_constant__ CUtensorMap tv, const __grid_constant__ LaPass a, unsigned int* status, uint32_t polls, int withhold) {
  using L = TcSmem<NT, PAIR, PL>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  const int lanes_of_heads = PAIR ? a.H / 2 : a.H;
  const int u = blockIdx.x / lanes_of_heads, h0 = (blockIdx.x % lanes_of_heads) * L::kHeads;
  Unit un;
  if (!get_unit(a, u, un)) return;
  if (a.states_only && (a.reverse ? un.first : un.last)) return;  // nothing follows this window
  const int warp = threadIdx.x >> 5;
  Cta t;
  t.smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // (an offset, so that accesses stay known as shared)
  t.bars = reinterpret_cast<uint64_t*>(t.smem + L::kBar);
  t.abort_flag = reinterpret_cast<volatile int*>(t.smem + L::kFlag);
  t.polls = polls;
  t.lane = threadIdx.x & 31;
  t.t0 = un.t0, t.len = un.len;
  t.chunks = (un.len + kC - 1) / kC;
  if (warp == 0) {
    tmem_alloc(&s_tmem, kTmem);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kBars; ++i) {
      int n = 1;
      if (i == kS1Free || (i >= kPFull && i < kPFree)) n = 4;
      if ((i >= kReady && i < kFree) || (i >= kUvFull && i < kUvFree)) n = 8;
      if (i == kYFree) n = 4;
      if (i == kDsFree || (i >= kSpFull && i < kSpFree)) n = 8;
      if (i >= kFree && i < kS1Full) n = a.states_only ? 1 : 2;
      if (i >= kGFree && i < kDrain) n = a.states_only ? 20 : 24;
      mbar_init(&t.bars[i], n);
    }
    *t.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_tensormap(&tq);
    prefetch_tensormap(&tk);
    prefetch_tensormap(&tv);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  t.tmem = s_tmem;

  // Registers: 896 threads start with 72 each (64512); the warpgroups' shares after the split,
  // 128 x (40 + 56 + 2 x 56 + 2 x 112 + 72) = 64512, are what the launch holds.
  if (warp < kMaskWarp) {
    set_regs_dec<40>();
    if (warp == kLoadWarp)
      load_role<NT, PAIR, PL>(t, a, &tq, &tk, &tv, h0, withhold);
    else if (warp == kDsWarp)
      ds_role<NT, PAIR, PL>(t, a);
    else if (warp == kGateWarp)
      gate_role<NT, PAIR, PL>(t, a, h0, u);
    else if (warp == kYWarp && !a.states_only)
      y_role<NT, PAIR, PL>(t, a);
  } else if (warp < kDecayWarp) {
    set_regs_dec<56>();
    mask_role<NT, PAIR, PL>(t, a);
  } else if (warp < kStateWarp) {
    set_regs_dec<56>();
    decay_role<NT, PAIR, PL>(t, a);
  } else if (warp < kOutWarp) {
    set_regs_inc<112>();
    state_role<NT, PAIR, PL>(t, a, un, u, h0);
  } else {
    set_regs_inc<72>();
    if (!a.states_only) out_role<NT, PAIR, PL>(t, a, h0);
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *t.abort_flag) atomicOr(status, kStatusTimeout);
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(s_tmem, kTmem);
  }
}

// {dim, heads, tokens} with boxes of 64 columns of one head and 64 tokens, 128-byte swizzle;
// what lies past the head's columns or the last token reads as zero.
bool make_map(CUtensorMap* m, const void* base, int dim, int heads, int64_t tokens) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)dim * 2, (cuuint64_t)dim * heads * 2};
  cuuint32_t box[3] = {64, 1, kC}, one[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT, bool PAIR, int PL>
cudaError_t launch_one(const LaPass& p, cudaStream_t st) {
  auto* fn = la_tc_kernel<NT, PAIR, PL>;
  using L = TcSmem<NT, PAIR, PL>;
  static_assert(L::kBytes <= 227 * 1024, "tiles must fit the SM's shared memory");
  CUtensorMap tq, tk, tv;
  if (!make_map(&tq, p.query, p.NK, p.q_heads, p.tokens) || !make_map(&tk, p.key, p.NK, p.k_heads, p.tokens) ||
      !make_map(&tv, p.value, p.PV, p.v_heads, p.tokens))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
  if (e != cudaSuccess) return e;
  // a poll takes 1 us (2000 cycles) at most: the bound in polls is within that of the wait limit
  const uint32_t polls = (uint32_t)std::min<long long>(std::max<long long>(device_wait_limit() / 2000, 1), 1u << 22);
  const int64_t units = p.segmented ? p.max_windows : p.nseq;
  fn<<<(unsigned)(units * (PAIR ? p.H / 2 : p.H)), kThreadsTc, L::kBytes, st>>>(
      tq, tk, tv, p, device_status_word(), polls, device_withhold() & 4);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

bool la_tc_supports(const LaPass& p) { return p.tokens > 0 && p.NK % 8 == 0 && p.PV % 8 == 0; }

bool la_tc_pairs(const LaPass& p) {
  return p.PV <= 64 && p.H % 2 == 0 && p.q_div % 2 == 0 && p.k_div % 2 == 0 && p.v_div == 1;
}

cudaError_t launch_la_tc(const LaPass& p, bool exact, cudaStream_t st) {
  const bool narrow = p.NK <= 64;
  if (exact) return narrow ? launch_one<64, false, kPlanes>(p, st) : launch_one<128, false, kPlanes>(p, st);
  if (la_tc_pairs(p)) return narrow ? launch_one<64, true, 1>(p, st) : launch_one<128, true, 1>(p, st);
  return narrow ? launch_one<64, false, 1>(p, st) : launch_one<128, false, 1>(p, st);
}

}  // namespace ssd
