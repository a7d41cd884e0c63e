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
// One CTA per SM (the shared memory is its own) walks a list of units: a sequence or a window of
// one, for one head of up to 128 value rows, or for two heads of up to 64 rows each that share
// query and key.  The list goes through up to three passes (the gradients of query, key and
// value are the same operator with exchanged operands), so that a batch too small for one pass
// fills the GPU with three and no CTA waits between them.  28 warps, each with one task, so that
// the tasks of several blocks and units overlap without any of them being interleaved by hand:
//   load  (1 warp)   finds the next unit; query, key and value tiles by TMA, three stages
//                    (two with PL = 3), and the rows that outputs are multiplied with
//   dS    (1 warp)   issues the products of dS
//   Y     (1 warp)   issues S1, a block ahead of Yi and Ya (one warp for all products took 110
//                    cycles for each of a block's 32 and 10 commits, and was what a block's time
//                    was made of)
//   gates (1 warp)   the sums of log-decays in 64 bits and the factors from them
//   mask  (4 warps)  S1 -> P
//   decay (8 warps)  value -> the planes of upd o value, by transposing loads
//   state (8 warps)  dS -> S -> the bf16 planes of S
//   out   (4 warps)  Yi, Ya -> out, and the dot products
// Tensor memory (512 columns): S1 64, Yi 64, Ya 64, dS 128, planes of upd o value 2 x 32, planes
// of S 2 x 64 (two heads: Ya 128, S 64).
//
// With one plane P and the copy of S that meets the query are rounded to bf16: about the output's own
// rounding each (y's error 2.3e-3 for 1.7e-3), where two planes of each would be a quarter more
// products and a second pass of the mask's and the state's stores.  With PL = 3 they enter their
// products as three bf16 planes each (fp32 accuracy), which the per-token dot products behind the
// decay's gradient need; a pass that has none runs in the same instance with one plane.
//
// Measured (a block is 64 tokens of a unit, NK = 128): 2.3 us for one head of 128 rows, 2.9 for
// two of 64, about 5 with three planes.  8 x 2048 tokens, 32 heads, N = P = 128: 187 us, of which
// HBM needs 87; 80 heads of 64 rows with one query and key: 278 of 57; gradients of 4 x 2048, 16
// heads: 310 of 36.  No unit of the SM is full: of the issue slots 62 % are used for one head of 128
// rows, 54 % for two of 64, 53 % with three planes; of the tensor pipe 27, 24 and 21 %.  A block is
// 12,800, 13,700 and (the mean of the gradients' passes) 19,100 warp instructions, of 28 warps
// that run their code once a block and wait for one another: most of the waiting is for tensor
// memory and barriers (4 to 6 of 11 to 13 cycles a warp spends on an instruction), 1 to 2 of them for
// instructions (a text of 75 to 95 KB, a seventh to a quarter of whose fetches miss).
// What changed most on the way: the state in registers and no spills in the block loops (a
// thread's local memory shares the little L1 that 215 KB of shared memory leave: 992 to 460 us for
// the first case), rolled loops where the text shrinks (460 to 396), and outputs through a staging
// buffer instead of 2-byte stores (396 to 325 us).  The two instances of one plane, one head and bf16
// outputs spill nothing; two heads 88 bytes of a thread, three planes 56, three planes with fp32
// outputs 108 (NK = 64: a little less), none of which has been timed apart.
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
constexpr int kMaxStages = 3, kGateSlots = 4, kPlanes = 3, kUnitSlots = 4;
constexpr int kWarpsTc = 28, kThreadsTc = 32 * kWarpsTc;
constexpr int kLoadWarp = 0, kDsWarp = 1, kGateWarp = 2, kMaskWarp = 4, kDecayWarp = 8, kStateWarp = 16, kOutWarp = 24;

// tensor memory columns
constexpr int kColS1 = 0, kColYi = 64, kColYa = 128, kColDs = 256, kColUv = 384, kColSp0 = 448, kColSp1 = 192;
constexpr int kTmem = 512;
constexpr uint32_t kDrainPolls = 1u << 22;  // (a drain's bound is not the test hooks' to lower)

enum Bar {
  kFull = 0,                     // tiles of a stage have landed
  kReady = kFull + kMaxStages,  // ... and rows past the sequence's end are zero (decay warps)
  kFree = kReady + kMaxStages,  // every product that reads the stage is done
  kS1Full = kFree + kMaxStages, kS1Free,
  kPFull, kPFree = kPFull + 2,
  kUvFull = kPFree + 2, kUvFree = kUvFull + 2,
  kDsFull = kUvFree + 2, kDsFree,
  kSpFull, kSpFree = kSpFull + 2,
  kYFull = kSpFree + 2, kYFree,
  kGFull, kGFree = kGFull + kGateSlots,
  kUnit = kGFree + kGateSlots, kUnitFree = kUnit + kUnitSlots,  // a unit's description
  kDotFull = kUnitFree + kUnitSlots, kDotFree = kDotFull + 2,  // rows that outputs are multiplied with
  kDrain = kDotFree + 2,  // every product of a warp that issues them is done
  kBars = kDrain + 2
};

// A unit as its CTA's roles see it, in shared memory; chunks < 0: there is none left.
struct alignas(16) UnitDesc {
  LaPass a;
  Unit un;
  int h0, chunks, planes;
  int begins, ends;
  // The block processed at step c: its place in the unit, its first token and its tokens.
  __device__ __forceinline__ int block(int c) const { return a.reverse ? chunks - 1 - c : c; }
  __device__ __forceinline__ int64_t token(int c) const { return un.t0 + (int64_t)block(c) * kC; }
  __device__ __forceinline__ int rows(int c) const { return min(kC, un.len - block(c) * kC); }
};

struct Gate {
  float chi[kC], clo[kC], row[kC], upd[kC];
  float decay, pad[3];
};

// An output warp's own staging: 64 tokens x 32 rows of bf16 at 80 bytes a token, or 16 tokens of
// fp32 at 144 (neither pitch has bank conflicts); and its dot products' parts.
constexpr int kOutPitch = 80, kOutPitch32 = 144, kOutBytes = kC * kOutPitch, kSumBytes = 4 * 32 * 16;

template <int NT, bool PAIR, int PL>
struct TcSmem {
  static constexpr int kStages = PL > 1 ? 2 : 3;   // (three planes of P leave room for two)
  static constexpr int kPTiles = PAIR ? 2 : PL;    // tiles of P: planes, or one per head
  static constexpr int kHeads = PAIR ? 2 : 1;
  static constexpr int kQ = 0, kK = NT / 64 * kAtomBytes, kV = 2 * kK, kStage = kV + 2 * kAtomBytes;
  static constexpr int kP = kStages * kStage;      // P: two buffers
  static constexpr int kDot = kP + 2 * kPTiles * kAtomBytes;  // rows that outputs are multiplied with: two buffers
  static constexpr int kGate = kDot + (PL > 1 ? 4 : 0) * kAtomBytes;
  static constexpr int kOut = kGate + (int)sizeof(Gate) * kHeads * kGateSlots;  // out warps: staged outputs, ...
  static constexpr int kSum = kOut + 4 * kOutBytes;                               // ... and the dot products' parts
  static constexpr int kBar = kSum + (PL > 1 ? 4 * kSumBytes : 0);
  static constexpr int kFlag = kBar + 8 * kBars;
  static constexpr int kUnits = (kFlag + 4 + 15) / 16 * 16;
  static constexpr int kBytes = kUnits + kUnitSlots * (int)sizeof(UnitDesc) + 1024;  // 1024: the base's alignment
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
  asm volatile("tcgen05.st.sync.aligned.16x256b.x1.b32 [%0], {%1, %2, %3, %4};" ::"r"(t), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
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

// Waits for the loads so far, and ties the wait to the registers they fill.
__device__ __forceinline__ void tmem_ld_wait8(uint32_t (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
               :
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

// One launch: up to three passes, each over its units (sequences or windows, times heads or pairs
// of heads), walked by a CTA per SM.
struct TcWork {
  int passes, total;   // total: units of all passes
  // First unit of each pass's whole sequences, and of each pass's windows: the long units come
  // first, so that the short ones even out the CTAs' shares
  int first[6];
  int exact[3];        // the pass wants P and S in three planes
  int8_t map[3][4];    // tensor maps of its query, key, value and dot
  int32_t* next;       // the next unit that no CTA has taken, or null: CTA b takes b, b + grid, ...
  LaPass pass[3];
};
struct TcMaps {
  CUtensorMap m[4];
};

// What every role needs.
struct Cta {
  uint8_t* smem;
  uint64_t* bars;
  volatile int* abort_flag;
  uint32_t polls;
  uint32_t tmem;
  int lane;
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
};

// A role's place in the CTA's list of units, which the load warp makes.  Blocks are numbered
// through all of it (`g` in the roles), which is what the barriers' phases go by.
struct Units {
  const Cta& t;
  const UnitDesc* ring;
  const UnitDesc* d;
  int n;
  __device__ __forceinline__ Units(const Cta& cta, int off)
      : t(cta), ring(reinterpret_cast<const UnitDesc*>(cta.smem + off)), d(nullptr), n(-1) {}
  __device__ __forceinline__ bool next() {
    if (n >= 0) t.arrive(kUnitFree + n % kUnitSlots);
    ++n;
    if (!t.wait(kUnit + n % kUnitSlots, n / kUnitSlots)) return false;
    d = ring + n % kUnitSlots;
    return d->chunks >= 0;
  }
  // The same without giving the last one back (for a second walk of one role).
  __device__ __forceinline__ bool peek() {
    ++n;
    if (!t.wait(kUnit + n % kUnitSlots, n / kUnitSlots)) return false;
    d = ring + n % kUnitSlots;
    return true;
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
  __device__ __forceinline__ uint64_t at(uint64_t major, int off) const {
    return major | (uint64_t)((base + off) >> 4);
  }
  // K step kk of a K-major tile of 64-column atoms
  static __device__ __forceinline__ uint64_t koff(int kk) {
    return (uint64_t)(((kk >> 2) * kAtomBytes + (kk & 3) * 32) >> 4);
  }
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

// Tiles by TMA.
template <int NT, bool PAIR, int PL>
__device__ __forceinline__ void load_role(const Cta& t, const TcWork& work, const TcMaps& maps) {
  using L = TcSmem<NT, PAIR, PL>;
  UnitDesc* ring = reinterpret_cast<UnitDesc*>(t.smem + L::kUnits);
  int s = 0, use = 0, dot = 0;  // stage, and its use; loads of rows for dot products
  bool ok = true, left = true;
#pragma unroll 1
  for (int n = 0, w = (int)blockIdx.x - (int)gridDim.x; ok && left;) {
    // the next unit that has work
    if (work.next) {
      if (t.lane == 0) w = atomicAdd(work.next, 1);
      w = __shfl_sync(0xffffffffu, w, 0);
    } else {
      w += (int)gridDim.x;
    }
    left = w < work.total;
    int part = 0;
#pragma unroll 1
    for (int i = 1; i < 2 * work.passes; ++i) part += w >= work.first[i];
    const int pass = part < work.passes ? part : part - work.passes;
    UnitDesc* d = ring + n % kUnitSlots;
    int h0 = 0, chunks = -1;
    Unit un{};
    if (left) {
      const LaPass& a = work.pass[pass];
      const int rel = w - work.first[part], per = a.H / L::kHeads;
      if (!get_unit(a, rel / per + (part == pass ? 0 : a.whole), un)) continue;
      const bool ends = a.reverse ? un.first : un.last;
      if (a.states_only && ends) continue;  // nothing follows this window
      h0 = rel % per * L::kHeads, chunks = (un.len + kC - 1) / kC;
      if (!chunks) {  // no tokens: the last state is the first (and no unit is without blocks)
        const int64_t size = (int64_t)a.NK * a.PV, from = ((int64_t)un.seq * a.H + h0) * size;
        if (a.last)
          for (int64_t i = t.lane; i < L::kHeads * size; i += 32) a.last[from + i] = a.start ? a.start[from + i] : 0.f;
        continue;
      }
      if (!(ok = t.wait_free(kUnitFree + n % kUnitSlots, n / kUnitSlots))) break;
      for (int i = t.lane; i < (int)(sizeof(LaPass) / 4); i += 32)
        reinterpret_cast<uint32_t*>(&d->a)[i] = reinterpret_cast<const uint32_t*>(&a)[i];
      if (t.lane == 0) {
        d->un = un, d->h0 = h0, d->planes = work.exact[pass] ? kPlanes : 1;
        d->begins = a.reverse ? un.last : un.first, d->ends = ends;
      }
    } else if (!(ok = t.wait_free(kUnitFree + n % kUnitSlots, n / kUnitSlots))) {
      break;
    }
    if (t.lane == 0) d->chunks = chunks;
    t.arrive(kUnit + n % kUnitSlots);
    ++n;
    if (!left) break;
    const LaPass& a = d->a;
    const int8_t* map = work.map[pass];
    const CUtensorMap *tq = &maps.m[map[0]], *tk = &maps.m[map[1]], *tv = &maps.m[map[2]];
    const int qh = h0 / a.q_div, kh = h0 / a.k_div, vh = h0 / a.v_div;  // (two heads: v_div is 1)
    const bool two = PAIR || a.PV > 64, q = !a.states_only;
    const bool dots = PL > 1 && a.dots != nullptr;
    const CUtensorMap* td = &maps.m[map[3]];
    const int dh = dots ? h0 / a.dot_div : 0;
    const uint32_t bytes = ((q ? 2 : 1) * (NT / 64) + (two ? 2 : 1)) * kAtomBytes;
    const bool reverse = a.reverse;
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
      if (!(ok = t.wait_free(kFree + s, use))) break;
      if (t.lane == 0) {
        uint64_t* bar = &t.bars[kFull + s];
        uint8_t* to = t.smem + s * L::kStage;
        const int tok = (int)un.t0 + (reverse ? chunks - 1 - c : c) * kC;
        mbar_expect_tx(bar, bytes);
#pragma unroll
        for (int i = 0; i < NT / 64; ++i) tma_load_3d(to + L::kK + i * kAtomBytes, tk, 64 * i, kh, tok, bar);
        if (q) {
#pragma unroll
          for (int i = 0; i < NT / 64; ++i) tma_load_3d(to + L::kQ + i * kAtomBytes, tq, 64 * i, qh, tok, bar);
        }
        tma_load_3d(to + L::kV, tv, 0, vh, tok, bar);
        if (two) tma_load_3d(to + L::kV + kAtomBytes, tv, PAIR ? 0 : 64, PAIR ? vh + 1 : vh, tok, bar);
      }
      __syncwarp();
      if (++s == L::kStages) s = 0, ++use;
      if (PL > 1 && dots) {
        const int slot = dot & 1;
        if (!(ok = t.wait_free(kDotFree + slot, dot >> 1))) break;
        if (t.lane == 0) {
          uint64_t* bar = &t.bars[kDotFull + slot];
          uint8_t* to = t.smem + L::kDot + slot * 2 * kAtomBytes;
          const int tok = (int)un.t0 + (reverse ? chunks - 1 - c : c) * kC;
          mbar_expect_tx(bar, (two ? 2 : 1) * kAtomBytes);
          tma_load_3d(to, td, 0, dh, tok, bar);
          if (two) tma_load_3d(to + kAtomBytes, td, 64, dh, tok, bar);
        }
        __syncwarp();
        ++dot;
      }
    }
  }
  // What was issued lands before the CTA ends, whichever role a wait ran out in (at once in a list
  // that was worked through).  The last use of stage d that was loaded is `use`, or the one before
#pragma unroll 1
  for (int d = 0; d < L::kStages; ++d) {
    const int n = use - (d >= s);
    if (n >= 0) wait_polls(smem_u32(&t.bars[kFull + d]), (uint32_t)n & 1u, kDrainPolls);
  }
  if (PL > 1)
#pragma unroll 1
    for (int d = max(0, dot - 2); d < dot; ++d)
      wait_polls(smem_u32(&t.bars[kDotFull + (d & 1)]), (uint32_t)(d >> 1) & 1u, kDrainPolls);
}

// dS = (upd o value)^T key, plane by plane.
template <int NT, bool PAIR, int PL>
__device__ __forceinline__ void ds_role(const Cta& t) {
  using L = TcSmem<NT, PAIR, PL>;
  const Issue mma(t);
  constexpr uint32_t id_ds = idesc_bf16(128, NT, 0, 1);
  bool ok = true;
  int s = 0, use = 0, g = 0, m = 0;  // m: planes so far
  Units at(t, L::kUnits);
#pragma unroll 1
  while (ok && at.next())
#pragma unroll 1
  for (int c = 0; c < at.d->chunks; ++c, ++g) {
    if (!(ok = t.wait(kReady + s, use)) || !(ok = t.wait(kDsFree, g))) break;  // (the unit's first: S is loaded)
    const uint64_t k_mn = mma.at(mma.mn_major, s * L::kStage + L::kK);
#pragma unroll 1
    for (int p = 0; p < kPlanes; ++p, ++m) {
      const int slot = m & 1;
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
  mma.drain(kDrain);
}

// S1 = query key^T, a block ahead; Yi^T = S query^T and Ya^T = value^T P^T.
template <int NT, bool PAIR, int PL>
__device__ __forceinline__ void y_role(const Cta& t, int withhold) {
  using L = TcSmem<NT, PAIR, PL>;
  const Issue mma(t);
  constexpr uint32_t id_s1 = idesc_bf16(64, kC, 0, 0), id_yi = idesc_bf16(128, kC, 0, 0),
                     id_ya = idesc_bf16(128, PAIR ? 2 * kC : kC, 1, 0);
  constexpr int sp_slots = PAIR ? 1 : 2;
  Units at(t, L::kUnits), ahead(t, L::kUnits);  // of Y, and of S1 (this one gives no slot back)
  bool ok = true;
  int s = 0, use = 0, s1 = 0, s1use = 0, m = 0;  // stages of Y and of S1; m: planes of S so far
  int left = 0, left1 = 0, planes = 1;           // blocks left of either's unit
#pragma unroll 1
  for (int g = -1;; ++g) {
    while (left1 == 0) {
      if (!(ok = ahead.peek())) break;
      left1 = ahead.d->chunks;
    }
    if (!ok) break;
    if (left1 > 0) {
      // A whole block's tiles as they landed.  Where the sequence ends inside the block, its keys
      // past the end are another's until they are zeroed, and a reverse pass's mask (j >= i)
      // keeps them: a NaN of theirs would meet the zeroed values in Ya, and 0 * NaN is NaN
      const int bar = ahead.d->rows(ahead.d->chunks - left1) < kC ? kReady : kFull;
      --left1;
      if (!(ok = t.wait(bar + s1, s1use)) || !(ok = t.wait_free(kS1Free, g + 1))) break;
      tc_fence_after();
      if (mma.leader) {
        const uint64_t q = mma.at(mma.k_major, s1 * L::kStage + L::kQ), k = mma.at(mma.k_major, s1 * L::kStage + L::kK);
#pragma unroll 1
        for (int kk = 0; kk < NT / 16; ++kk)
          umma_f16(t.tmem + kColS1, q + Issue::koff(kk), k + Issue::koff(kk), id_s1, kk > 0);
      }
      __syncwarp();
      if (!withhold) mma.commit(kS1Full);
      if (++s1 == L::kStages) s1 = 0, ++s1use;
    }
    if (g < 0) continue;
    while (left == 0) {
      if (!(ok = at.next())) break;
      left = at.d->chunks, planes = PL > 1 ? at.d->planes : 1;
    }
    if (!ok) break;  // the end of the list, or a wait that gave up
    --left;
    if (!(ok = t.wait_free(kYFree, g))) break;
    const uint64_t q = mma.at(mma.k_major, s * L::kStage + L::kQ);
    // Ya goes between the planes of S: the third plane's slot is free once the first is done
#pragma unroll 1
    for (int p = 0; p < planes; ++p, ++m) {
      const int slot = m % sp_slots;
      if (!(ok = t.wait(kSpFull + slot, m / sp_slots))) break;
      tc_fence_after();
      if (mma.leader) {
        const uint32_t sp = t.tmem + (slot ? kColSp1 : kColSp0);
#pragma unroll 1
        for (int kk = 0; kk < NT / 16; ++kk)
          umma_f16_ta(t.tmem + kColYi, sp + kk * 8, q + Issue::koff(kk), id_yi, p > 0 || kk > 0);
      }
      __syncwarp();
      mma.commit(kSpFree + slot);
      if (p) continue;
      if (!(ok = t.wait(kReady + s, use)) || !(ok = t.wait(kPFull + (g & 1), g >> 1))) break;
      tc_fence_after();
      if (mma.leader) {
        const uint64_t v_mn = mma.at(mma.mn_major, s * L::kStage + L::kV);
#pragma unroll 1
        for (int k = 0; k < planes; ++k) {
          const uint64_t pm = mma.at(mma.k_major, L::kP + ((g & 1) * L::kPTiles + k) * kAtomBytes);
#pragma unroll 1
          for (int kk = 0; kk < kC / 16; ++kk)
            umma_f16(t.tmem + kColYa, v_mn + kk * 128, pm + kk * 2, id_ya, k > 0 || kk > 0);
        }
      }
      __syncwarp();
      mma.commit(kPFree + (g & 1));
    }
    if (!ok) break;
    mma.commit(kYFull);
    mma.commit(kFree + s);  // (S1 of this block was done before its P)
    if (++s == L::kStages) s = 0, ++use;
  }
  mma.drain(kDrain + 1);
}

// One head: lane l takes tokens 2 l, 2 l + 1 of each block.  Two: half a warp each, 4 tokens a lane.
template <int NT, bool PAIR, int PL>
__device__ __forceinline__ void gate_role(const Cta& t) {
  using L = TcSmem<NT, PAIR, PL>;
  constexpr int kLanes = 32 / L::kHeads, kTok = kC / kLanes;
  const int which = PAIR ? t.lane >> 4 : 0, l = t.lane & (kLanes - 1), i0 = kTok * l;
  Units at(t, L::kUnits);
  int g = 0;
#pragma unroll 1
  while (at.next()) {
    const LaPass& a = at.d->a;
    const bool reverse = a.reverse;
    const float sr = reverse ? 1.f : a.scale, su = reverse ? a.scale : 1.f;
    const float* from = a.log_decay + at.d->h0 + which;
    const int64_t pitch = a.per_token ? a.H : 0;
    double total = 0.0;
    float x[kTok];
    auto load = [&](int c) {
      if (c >= at.d->chunks) return;
      const int64_t tok = at.d->token(c) + i0;
      const int left = at.d->rows(c) - i0;
#pragma unroll
      for (int j = 0; j < kTok; ++j) x[j] = j < left ? from[(tok + j) * pitch] : 0.f;
    };
    load(0);
#pragma unroll 1
    for (int c = 0; c < at.d->chunks; ++c, ++g) {
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
      const int slot = g % kGateSlots;
      if (!t.wait_free(kGFree + slot, g / kGateSlots)) return;
      Gate* to = reinterpret_cast<Gate*>(t.smem + L::kGate) + slot * L::kHeads + which;
#pragma unroll
      for (int j = 0; j < kTok; ++j) {
        const double cc = before + sum[j];
        float hi, lo;
        const float from_start = exp2_split(cc, hi, lo);
        // signed, so that the decay between i and j is 2^(c_i - c_j) either way.  In one number
        // where P is rounded to bf16: sums of up to 64 x 150 are held to 2^-11, so a difference is
        // off by 2^-10 and a factor by 7e-4 at most (in a block whose tokens nearly all forget; 2e-5 where
        // sums stay within 512), and P's own rounding by up to 2^-8, 39e-4
        const float sign = reverse ? -1.f : 1.f;
        to->chi[i0 + j] = sign * (PL > 1 ? hi : hi + lo);
        if (PL > 1) to->clo[i0 + j] = sign * lo;
        const float to_end = exp2_split(end - cc, hi, lo);
        to->row[i0 + j] = (reverse ? to_end : from_start) * sr;
        to->upd[i0 + j] = (reverse ? from_start : to_end) * su;
      }
      if (l == 0) {
        float hi, lo;
        to->decay = exp2_split(end, hi, lo);
      }
      total += end;
      t.arrive(kGFull + slot);
    }
    if (a.states_only && l == 0) {
      float hi, lo;
      a.window_decay[(int64_t)at.d->un.window * a.H + at.d->h0 + which] = exp2_split(total, hi, lo);
    }
  }
}

// S1 -> P.  Warp q holds rows 16 q .. 16 q + 15 of S1 (lanes 0 .. 15 of its quarter of tensor
// memory: a product of 64 rows puts 16 in each quarter).
template <int NT, bool PAIR, int PL>
__device__ __forceinline__ void mask_role(const Cta& t) {
  using L = TcSmem<NT, PAIR, PL>;
  const int q = threadIdx.x / 32 & 3;
  const int gr = t.lane >> 2, gc = (t.lane & 3) * 2;
  const int i0 = 16 * q + gr;
  const uint32_t lanes = (uint32_t)(32 * q) << 16;
  Units at(t, L::kUnits);
  uint8_t* P = t.smem + L::kP;
  auto put = [&](uint8_t* tile, int i, int j, uint32_t v) {
    *reinterpret_cast<uint32_t*>(tile + sw128_off(i, j >> 3) + (j & 7) * 2) = v;
  };
  int g = 0;
#pragma unroll 1
  while (at.next()) {
    const LaPass& a = at.d->a;
    const bool reverse = a.reverse, states = a.states_only;
    const float scale = a.scale;
    const int planes = PL > 1 ? at.d->planes : 1;
    // the pairs of column tiles with any j in reach; the others are zero (written anyway for the
    // first two blocks of a unit: another unit's direction may have filled them)
    const int b0 = reverse ? q : 0, b1 = reverse ? 4 : q + 1;
    // j <= i (reverse: j >= i) is sign * (i - j) >= 0, for the thread's rows i0, i0 + 8 and columns j, j + 1
    const int sign = reverse ? -1 : 1;
#pragma unroll 1
    for (int c = 0; c < at.d->chunks; ++c, ++g) {
      const int slot = g % kGateSlots;
      if (!t.wait(kGFull + slot, g / kGateSlots)) return;
      if (!states) {
        const Gate* gate = reinterpret_cast<const Gate*>(t.smem + L::kGate) + slot * L::kHeads;
        if (!t.wait(kS1Full, g) || !t.wait_free(kPFree + (g & 1), g >> 1)) return;
        tc_fence_after();
        const int from = c < 2 ? 0 : b0, to = c < 2 ? 4 : b1;
        uint8_t* tiles = P + (g & 1) * L::kPTiles * kAtomBytes;
        // the next columns are on their way while these are worked on; S1 is free before the last
        uint32_t r[8], next[8];
        tmem_ld_16x256_x2(t.tmem + lanes + kColS1 + 16 * from, r);
        tmem_ld_wait8(r);
#pragma unroll 1
        for (int b = from; b < to; ++b) {
          if (b + 1 < to) tmem_ld_16x256_x2(t.tmem + lanes + kColS1 + 16 * (b + 1), next);
          if (b + 1 == to) {
            tc_fence_before();
            t.arrive(kS1Free);
          }
#pragma unroll
          for (int hh = 0; hh < L::kHeads; ++hh) {
            const float hi0 = gate[hh].chi[i0], hi1 = gate[hh].chi[i0 + 8];
            const float lo0 = PL > 1 ? gate[hh].clo[i0] : 0.f, lo1 = PL > 1 ? gate[hh].clo[i0 + 8] : 0.f;
#pragma unroll
            for (int nn = 0; nn < 2; ++nn) {
              const int j = 16 * b + 8 * nn + gc;
              const float2 hj = *reinterpret_cast<const float2*>(&gate[hh].chi[j]);
              const float2 lj = PL > 1 ? *reinterpret_cast<const float2*>(&gate[hh].clo[j]) : make_float2(0.f, 0.f);
              float v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float d = (e >> 1 ? hi1 : hi0) - (e & 1 ? hj.y : hj.x);
                if (PL > 1) d += (e >> 1 ? lo1 : lo0) - (e & 1 ? lj.y : lj.x);
                const bool in = sign * (i0 - j) + sign * (8 * (e >> 1) - (e & 1)) >= 0;
                v[e] = in ? __uint_as_float(r[4 * nn + e]) * scale * ex2(d) : 0.f;
              }
#pragma unroll
              for (int p = 0; p < PL; ++p) {
                if (p >= planes) break;
                const uint32_t x = bf16x2(v[0], v[1]), y = bf16x2(v[2], v[3]);
                uint8_t* tile = tiles + (PAIR ? hh : p) * kAtomBytes;
                put(tile, i0, j, x);
                put(tile, i0 + 8, j, y);
                v[0] -= bf16_lo(x), v[1] -= bf16_hi(x), v[2] -= bf16_lo(y), v[3] -= bf16_hi(y);
              }
            }
          }
          if (b + 1 < to) {
            tmem_ld_wait8(next);
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i] = next[i];
          }
        }
        fence_proxy_async();
        t.arrive(kPFull + (g & 1));
      }
      t.arrive(kGFree + slot);
    }
  }
}

// value -> the planes of upd o value in tensor memory, transposed on the way.  Warp w makes rows
// 32 (w % 4) .. and half of the block's tokens.
template <int NT, bool PAIR, int PL>
__device__ __forceinline__ void decay_role(const Cta& t) {
  using L = TcSmem<NT, PAIR, PL>;
  const int w = threadIdx.x / 32 - kDecayWarp, q = w & 3, half = w >> 2, lane = t.lane;
  const int head = PAIR ? q >> 1 : 0;
  const uint32_t uv = t.tmem + ((uint32_t)(32 * q) << 16) + kColUv + 16 * half;
  Units at(t, L::kUnits);
  int s = 0, use = 0, g = 0, m = 0;  // m: planes so far
#pragma unroll 1
  while (at.next()) {
    const bool active = (PAIR ? 32 * q & 63 : 32 * q) < at.d->a.PV;
#pragma unroll 1
    for (int c = 0; c < at.d->chunks; ++c, ++g) {
      const int slot = g % kGateSlots, rows = at.d->rows(c);
      uint8_t* tiles = t.smem + s * L::kStage;
      if (!t.wait(kFull + s, use)) return;
      if (rows < kC) {
        // the sequence ends inside the block: what follows is another's, and 0 * NaN is NaN.  A
        // row of key and value is 8 pieces of 16 bytes in each of up to 4 atoms
        constexpr int kAtoms = NT / 64 + 2;
#pragma unroll 1
        for (int i = rows + w; i < kC; i += 8)
          if (lane < 8 * kAtoms)
            *reinterpret_cast<uint4*>(tiles + L::kK + (lane >> 3) * kAtomBytes + i * 128 + (lane & 7) * 16) =
                make_uint4(0, 0, 0, 0);
        fence_proxy_async();
      }
      t.arrive(kReady + s);
      if (rows < kC && !t.wait(kReady + s, use)) return;
      if (++s == L::kStages) s = 0, ++use;
      if (!t.wait(kGFull + slot, g / kGateSlots)) return;
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
            for (int k = 0; k < 4; ++k) {
              x[hf][4 * kk + k][0] = bf16_lo(v[k]) * (k < 2 ? ua.x : ub.x);
              x[hf][4 * kk + k][1] = bf16_hi(v[k]) * (k < 2 ? ua.y : ub.y);
            }
          }
        }
      }
      t.arrive(kGFree + slot);
#pragma unroll 1
      for (int p = 0; p < kPlanes; ++p, ++m) {
        const int us = m & 1;
        if (!t.wait_free(kUvFree + us, m >> 1)) return;
        tc_fence_after();
        if (active) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              v[i] = bf16x2(x[hf][i][0], x[hf][i][1]);
              if (p + 1 < kPlanes) x[hf][i][0] -= bf16_lo(v[i]), x[hf][i][1] -= bf16_hi(v[i]);
            }
            tmem_st_16x128_x4(uv + ((uint32_t)(16 * hf) << 16) + 32 * us, v);
          }
          tmem_st_wait();
        }
        tc_fence_before();
        t.arrive(kUvFull + us);
      }
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
__device__ __forceinline__ void move_state(uint32_t ds, const StateAt& at, int lane, int row0, int n0, int rows,
                                           int cols) {
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
// S in registers: warp w (of 8) holds rows 32 (w % 4) .. and half of the columns.  Step c = -1 of a
// unit takes the start state the way the others take dS, from the same columns, so that there
// is one piece of code for what follows either.
template <int NT, bool PAIR, int PL>
__device__ __forceinline__ void state_role(const Cta& t) {
  using L = TcSmem<NT, PAIR, PL>;
  constexpr int NC = NT / 2, sp_slots = PAIR ? 1 : 2;  // columns of a thread
  const int w = threadIdx.x / 32 - kStateWarp, q = w & 3, half = w >> 2;
  const int head = PAIR ? q >> 1 : 0;
  const int row0 = PAIR ? 32 * q & 63 : 32 * q;  // the warp's first row of the head
  const int n0 = half * NC;
  const uint32_t lanes = (uint32_t)(32 * q) << 16;
  const uint32_t ds = t.tmem + lanes + kColDs + n0;  // the thread's part of dS
  Units at(t, L::kUnits);
  float S[NC];
  int g = 0, m = 0;  // blocks and planes so far
#pragma unroll 1
  while (at.next()) {
    const LaPass& a = at.d->a;
    const int h = at.d->h0 + head, planes = PL > 1 ? at.d->planes : 1;
    const bool states = a.states_only;
    const int64_t state_at = ((int64_t)at.d->un.seq * a.H + h) * a.NK * a.PV;
    auto window_at = [&](float* base, int64_t win) {
      return StateAt{base + (win * a.H + h) * a.PV * a.NK, (int64_t)a.NK, 1};
    };
    {
      StateAt from{nullptr, a.NK, 1};
      if (!at.d->begins) {
        if (!states) from = window_at(a.carry, at.d->un.window);
      } else if (a.start) {
        from = StateAt{const_cast<float*>(a.start) + state_at, a.sr, a.sc};
      }
      move_state<NC, false>(ds, from, t.lane, row0, n0, from.base ? a.PV : 0, a.NK);
#pragma unroll
      for (int n = 0; n < NC; ++n) S[n] = 0.f;
    }
#pragma unroll 1
    for (int c = -1; c < at.d->chunks; ++c) {
      float dec = 0.f;
      if (c >= 0) {
        if (!t.wait(kGFull + g % kGateSlots, g / kGateSlots)) return;
        dec = (reinterpret_cast<const Gate*>(t.smem + L::kGate) + (g % kGateSlots) * L::kHeads + head)->decay;
        if (!t.wait(kDsFull, g)) return;
      }
      const bool more = c + 1 < at.d->chunks, out = more && !states;
      // The next step's first plane goes out as S is made, and of three the second with it; the
      // third follows when the first one's slot is free again.
      const bool three = PL > 1 && planes > 1;
      const int slot = m % sp_slots, slot2 = (m + 1) % sp_slots;
      if (out && !t.wait_free(kSpFree + slot, m / sp_slots)) return;
      if (PL > 1 && out && three && !t.wait_free(kSpFree + slot2, (m + 1) / sp_slots)) return;
      tc_fence_after();
      const uint32_t sp = t.tmem + lanes + (slot ? kColSp1 : kColSp0) + half * (NC / 2);
      const uint32_t sp2 = t.tmem + lanes + (slot2 ? kColSp1 : kColSp0) + half * (NC / 2);
#pragma unroll
      for (int b = 0; b < NC / 16; ++b) {
        uint32_t d[16], v[8];
        tmem_ld16(ds + 16 * b, d);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) S[16 * b + i] = fmaf(S[16 * b + i], dec, __uint_as_float(d[i]));
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = bf16x2(S[16 * b + 2 * i], S[16 * b + 2 * i + 1]);
        if (out) tmem_st8(sp + 8 * b, v);
        if (PL > 1 && out && three) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            v[i] = bf16x2(S[16 * b + 2 * i] - bf16_lo(v[i]), S[16 * b + 2 * i + 1] - bf16_hi(v[i]));
          tmem_st8(sp2 + 8 * b, v);
        }
      }
      if (out) tmem_st_wait();
      // Copies that are wanted: of the windows' states (forward, after a window's last block;
      // reverse, before it), and of the unit's last one.
      const int bl = a.reverse ? at.d->chunks - 2 - c : c;
      const bool dump = a.dump && bl >= 0 && (bl == at.d->chunks - 1 || (bl + 1) * kC % a.window == 0);
      const bool last = !more && (states || (a.last && at.d->ends));
      if (dump || last) {
#pragma unroll
        for (int b = 0; b < NC / 16; ++b) {
          uint32_t v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(S[16 * b + i]);
          tmem_st16(ds + 16 * b, v);
        }
        tmem_st_wait();
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          if (!(k ? last : dump)) continue;
          StateAt to = window_at(k ? a.carry : a.dump, at.d->un.window + (k ? 0 : bl * kC / a.window));
          if (k && !states) to = StateAt{a.last + state_at, a.sr, a.sc};
          move_state<NC, true>(ds, to, t.lane, row0, n0, a.PV, a.NK);
        }
      }
      tc_fence_before();
      if (out) {
        t.arrive(kSpFull + slot);
        if (PL > 1 && three) t.arrive(kSpFull + slot2);
        m += PL > 1 && three ? 2 : 1;
      }
      if (more) t.arrive(kDsFree);
      if (c >= 0) {
        t.arrive(kGFree + g % kGateSlots);
        ++g;
      }
      if (PL > 1 && out && three) {  // what the first two leave
        const int sl = m % sp_slots;
        if (!t.wait_free(kSpFree + sl, m / sp_slots)) return;
        tc_fence_after();
        const uint32_t to = t.tmem + lanes + (sl ? kColSp1 : kColSp0) + half * (NC / 2);
#pragma unroll
        for (int b = 0; b < NC / 16; ++b) {
          uint32_t v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            // made anew: kept from above, the remainders would not fit the registers
            asm volatile("" : "+f"(S[16 * b + 2 * i]), "+f"(S[16 * b + 2 * i + 1]));
            float x = S[16 * b + 2 * i], y = S[16 * b + 2 * i + 1];
            v[i] = bf16x2(x, y);
            x -= bf16_lo(v[i]), y -= bf16_hi(v[i]);
            v[i] = bf16x2(x, y);
            v[i] = bf16x2(x - bf16_lo(v[i]), y - bf16_hi(v[i]));
          }
          tmem_st8(to + 8 * b, v);
        }
        tmem_st_wait();
        tc_fence_before();
        t.arrive(kSpFull + sl);
        ++m;
      }
    }
  }
}

// Yi, Ya -> out: warp q writes rows 32 q .., 16 tokens at a time.  Tensor memory is read in the
// layout of mma.sync's accumulators (registers are pairs of tokens of one row), turned by
// transposing stores to shared memory, and written from there in 16-byte pieces (single 2-byte
// stores took 16 cycles each, 5 of the 9 thousand that a block then had).
template <int NT, bool PAIR, int PL, bool F32>
__device__ __forceinline__ void out_role(const Cta& t) {
  using L = TcSmem<NT, PAIR, PL>;
  const int q = threadIdx.x / 32 & 3;
  const int head = PAIR ? q >> 1 : 0;
  const int row0 = PAIR ? 32 * q & 63 : 32 * q;  // the warp's first row of the head
  const uint32_t lanes = (uint32_t)(32 * q) << 16;
  uint8_t* stage = t.smem + L::kOut + q * kOutBytes;
  float* sums = reinterpret_cast<float*>(t.smem + L::kSum + q * kSumBytes);
  const int gr = t.lane >> 2, gc = (t.lane & 3) * 2;
  Units walk(t, L::kUnits);
  int g = 0, dot = 0;
#pragma unroll 1
  while (walk.next()) {
  const LaPass& a = walk.d->a;
  const int h = walk.d->h0 + head;
  const bool active = row0 < a.PV;
  const bool dots = PL > 1 && a.dot != nullptr;
  const int PV = a.PV, chunks = walk.d->chunks;
  const int64_t pitch = (int64_t)a.H * PV;
  const bool out_f32 = F32 && a.out_f32;
#pragma unroll 1
  for (int c = 0; c < chunks; ++c, ++g) {
    const float* rowf = (reinterpret_cast<const Gate*>(t.smem + L::kGate) + (g % kGateSlots) * L::kHeads + head)->row;
    if (!t.wait(kGFull + g % kGateSlots, g / kGateSlots) || !t.wait(kYFull, g)) return;
    tc_fence_after();
    const int64_t tok = walk.d->token(c);
    const int rows = walk.d->rows(c);
    const int64_t at = tok * pitch + (int64_t)h * PV + row0;
    uint8_t* dot_tile = t.smem + L::kDot + (dot & 1) * 2 * kAtomBytes + (row0 >> 6) * kAtomBytes;
    if (dots && !t.wait(kDotFull + (dot & 1), dot >> 1)) return;
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
      if (!out_f32) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint8_t* to = stage + (16 * b + 8 * (t.lane >> 4) + (t.lane & 7)) * kOutPitch + 32 * hf +
                              16 * ((t.lane >> 3) & 1);
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
          if (16 * b + i < rows && row0 + p < PV) *reinterpret_cast<float4*>(to + i * pitch + p) = v;
        }
        __syncwarp();
      }
      if (dots && active) {  // sums over the warp's rows of out * dot, for the decay's gradient
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t v[4];
          const int i = 16 * b + 8 * (t.lane >> 4) + (t.lane & 7), p = (row0 & 63) + 16 * hf + 8 * ((t.lane >> 3) & 1);
          const uint8_t* from = dot_tile + sw128_off(i, p >> 3);
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
        *reinterpret_cast<float4*>(sums + (b * 32 + t.lane) * 4) = make_float4(sum[0], sum[1], sum[2], sum[3]);
      }
    }
    if (dots) {
      t.arrive(kDotFree + (dot & 1));
      ++dot;
    }
    if (dots && active) {
      // lane 4 r + l of step b has the rows r, r + 8, .. of tokens 16 b + 2 l, + 1, + 8, + 9
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int i = t.lane + 32 * k, b = i >> 4, l = (i & 7) >> 1, e = (i & 1) + 2 * ((i >> 3) & 1);
        float sum = 0.f;
#pragma unroll
        for (int r = 0; r < 8; ++r) sum += sums[(b * 32 + 4 * r + l) * 4 + e];
        if (i < rows) a.dots[((int64_t)q * a.tokens + tok + i) * a.H + h] = sum;
      }
    }
    t.arrive(kGFree + g % kGateSlots);
    if (!active || out_f32) continue;
    __syncwarp();
    __nv_bfloat16* to = static_cast<__nv_bfloat16*>(a.out) + at;
#pragma unroll 4
    for (int k = 0; k < 8; ++k) {
      const int i = 8 * k + gr, p = (t.lane & 3) * 8;
      const uint4 v = *reinterpret_cast<const uint4*>(stage + i * kOutPitch + p * 2);
      if (i < rows && row0 + p < PV) *reinterpret_cast<uint4*>(to + i * pitch + p) = v;
    }
    __syncwarp();
  }
  }
}

// Grid: a CTA per SM at most.  The list: units of a pass times heads or pairs of heads, heads fastest.
template <int NT, bool PAIR, int PL, bool F32>
__global__ void __launch_bounds__(kThreadsTc, 1)
    la_tc_kernel(const __grid_constant__ TcMaps maps, const __grid_constant__ TcWork work, unsigned int* status,
                 uint32_t polls, int withhold) {
  using L = TcSmem<NT, PAIR, PL>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  const int warp = threadIdx.x >> 5;
  const bool states = work.pass[0].states_only;
  Cta t;
  t.smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // (an offset, so that accesses stay known as shared)
  t.bars = reinterpret_cast<uint64_t*>(t.smem + L::kBar);
  t.abort_flag = reinterpret_cast<volatile int*>(t.smem + L::kFlag);
  t.polls = polls;
  t.lane = threadIdx.x & 31;
  if (warp == 0) {
    tmem_alloc(&s_tmem, kTmem);
    tmem_relinquish();
  }
  if (threadIdx.x >= 32 && threadIdx.x < 32 + kBars) {
    const int i = threadIdx.x - 32;
    int n = 1;
    if (i == kS1Free || (i >= kPFull && i < kPFree) || i == kYFree || (i >= kDotFree && i < kDrain)) n = 4;
    if ((i >= kReady && i < kFree) || (i >= kUvFull && i < kUvFree)) n = 8;
    if (i == kDsFree || (i >= kSpFull && i < kSpFree)) n = 8;
    if (i >= kFree && i < kS1Full) n = states ? 1 : 2;
    if (i >= kGFree && i < kUnit) n = states ? 20 : 24;
    if (i >= kUnitFree && i < kDotFull) n = states ? 22 : 27;  // every warp but the load warp
    mbar_init(&t.bars[i], n);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x == 0) *t.abort_flag = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  t.tmem = s_tmem;

  // Registers: 896 threads start with 72 each (64512); the warpgroups' shares after the split,
  // 128 x (40 + 56 + 2 x 64 + 2 x 104 + 72) = 64512, are what the launch holds.
  if (warp < kMaskWarp) {
    set_regs_dec<40>();
    if (warp == kLoadWarp) {
      load_role<NT, PAIR, PL>(t, work, maps);
    } else if (warp == kGateWarp) {
      gate_role<NT, PAIR, PL>(t);
    } else if (warp == kDsWarp) {
      ds_role<NT, PAIR, PL>(t);
    } else if (!states) {
      y_role<NT, PAIR, PL>(t, withhold);
    }
  } else if (warp < kDecayWarp) {
    set_regs_dec<56>();
    mask_role<NT, PAIR, PL>(t);
  } else if (warp < kStateWarp) {
    set_regs_dec<64>();
    decay_role<NT, PAIR, PL>(t);
  } else if (warp < kOutWarp) {
    set_regs_inc<104>();
    state_role<NT, PAIR, PL>(t);
  } else if (!states) {
    out_role<NT, PAIR, PL, F32>(t);
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

template <int NT, bool PAIR, int PL, bool F32>
cudaError_t launch_one(const TcMaps& maps, const TcWork& work, cudaStream_t st) {
  auto* fn = la_tc_kernel<NT, PAIR, PL, F32>;
  using L = TcSmem<NT, PAIR, PL>;
  static_assert(L::kBytes <= 227 * 1024, "tiles must fit the SM's shared memory");
  static_assert(kBars + 32 <= kThreadsTc, "a thread per barrier");
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
  if (e != cudaSuccess) return e;
  // a poll takes 1 us (2000 cycles) at most: the bound in polls is within that of the wait limit
  const uint32_t polls = (uint32_t)std::min<long long>(std::max<long long>(device_wait_limit() / 2000, 1), 1u << 22);
  fn<<<(unsigned)std::min(work.total, device_sm_count()), kThreadsTc, L::kBytes, st>>>(
      maps, work, device_status_word(), polls, device_withhold() & 4);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

bool la_tc_supports(const LaPass& p) { return p.tokens > 0 && p.NK % 8 == 0 && p.PV % 8 == 0; }

bool la_tc_pairs(const LaPass& p) {
  return p.PV <= 64 && p.H % 2 == 0 && p.q_div % 2 == 0 && p.k_div % 2 == 0 && p.v_div == 1;
}

cudaError_t launch_la_tc(const LaPass* p, int passes, cudaStream_t st) {
  bool exact = false, f32 = false, pair = passes == 1 && la_tc_pairs(p[0]), narrow = true;
  for (int i = 0; i < passes; ++i) {
    exact |= p[i].dots != nullptr;
    f32 |= p[i].out_f32 != 0;
    narrow &= p[i].NK <= 64;
  }
  pair &= !exact && !f32;
  TcWork work{};
  TcMaps maps;
  const void* bases[4] = {};  // an operand that passes share has one map
  int dims[4] = {}, counts[4] = {}, made = 0;
  work.passes = passes;
  int64_t total = 0;
  for (int i = 0; i < 2 * passes; ++i) {
    const LaPass& q = p[i % passes];
    work.first[i] = (int)std::min<int64_t>(total, INT32_MAX);
    total += (i < passes ? q.whole : la_units(q) - q.whole) * (pair ? q.H / 2 : q.H);
  }
  for (int i = 0; i < passes; ++i) {
    work.pass[i] = p[i];
    work.exact[i] = p[i].dots != nullptr;
    const void* operand[4] = {p[i].query, p[i].key, p[i].value, p[i].dot};
    const int dim[4] = {p[i].NK, p[i].NK, p[i].PV, p[i].PV};
    const int heads[4] = {p[i].q_heads, p[i].k_heads, p[i].v_heads, p[i].dot_heads};
    for (int o = 0; o < (p[i].dots ? 4 : 3); ++o) {
      int k = 0;
      while (k < made && (bases[k] != operand[o] || dims[k] != dim[o] || counts[k] != heads[o])) ++k;
      if (k == made) {
        if (made == 4 || (operand[o] && !make_map(&maps.m[k], operand[o], dim[o], heads[o], p[i].tokens)))
          return cudaErrorInvalidValue;
        bases[made] = operand[o], dims[made] = dim[o], counts[made] = heads[o];
        ++made;
      }
      work.map[i][o] = (int8_t)k;
    }
  }
  if (total > (1ll << 31) - 1) return cudaErrorInvalidConfiguration;
  if (total == 0) return cudaSuccess;
  work.total = (int)total;
  // A packed batch's windows are of 1 to `window` tokens: whoever is free takes the next (which CTA
  // works on a unit does not change its result).  A dense batch's units are alike.
  work.next = p[0].next ? p[0].next + (p[0].states_only ? 1 : 0) : nullptr;
  if (narrow) {
    if (exact) return f32 ? launch_one<64, false, kPlanes, true>(maps, work, st)
                          : launch_one<64, false, kPlanes, false>(maps, work, st);
    if (f32) return launch_one<64, false, 1, true>(maps, work, st);
    return pair ? launch_one<64, true, 1, false>(maps, work, st) : launch_one<64, false, 1, false>(maps, work, st);
  }
  if (exact) return f32 ? launch_one<128, false, kPlanes, true>(maps, work, st)
                        : launch_one<128, false, kPlanes, false>(maps, work, st);
  if (f32) return launch_one<128, false, 1, true>(maps, work, st);
  return pair ? launch_one<128, true, 1, false>(maps, work, st) : launch_one<128, false, 1, false>(maps, work, st);
}

}  // namespace ssd
