// Decayed linear attention over a packed pass, bf16 inputs: one cooperative
// launch for the piece states, their decayed sums, and the output of every
// row.  With a = exp(log_decay[h]) and S the state entering a tile of up to
// 128 rows (row i of the tile, its segment starting at row s(i) of it):
//
//     o_i = sum_{s(i) <= j <= i} a^(i-j) (q_i . k_j) v_j  +  a^(i-s(i)+1) S^T q_i
//     S  <- a^n S + sum_j a^(n-1-j) k_j v_j^T                       (n rows)
//
// The work is cut as span_output's is (k_span_output.cu): one run of tiles per
// SM from a host-built list; a piece is the part of a segment-head (a view, or
// a branch longer than a tile) inside a run.  Two phases:
//
//   1. Every CTA runs over K and V of its pieces and keeps the pieces' own
//      states, S <- a^n S + K^T V' from S = 0 with V' = a^(n-1-j) v_j: the state
//      before each tile goes to a table (16 KiB a tile and head), the one
//      after the piece to a slot that other CTAs read.
//   2. Once every CTA has counted itself a CTA sums the slots that a piece's start
//      state needs by Horner's rule, S <- a^rows S + piece, and runs the tiles:
//      the state entering tile t of a piece is a^(128 t) (start) + (table).
//
// So K^T V, with its scaled operand, is not in the second phase's chain, which
// is bound by the latency of its hand-offs.  Keeping it there (the first
// phase then only for pieces that others need, the running state carried from
// tile to tile as span_output does) took 5,300 cycles a tile and 198 us for a
// pass of four requests, against 120.
//
// Measured, 16 heads: 7,796 rows (a view of 7,400 and 8 branches) 26.7 us with
// the inputs in L2 and 28.8 us cold; 43,684 rows of four requests 120 us;
// 208,830 rows of sixteen 509 us; 64 branches from a kept state 14.4 us (16.4
// cold).  Large passes are bound by DRAM: K and V are read once for each phase
// and the table is written and read, 679 MB for four requests where the call's
// own inputs and outputs are 359 MB, at 5.8 TB/s (85 % of what a copy reaches);
// the chains would take about as long, 1.0 us a tile in phase 1 and 1.6 in
// phase 2.  Phase 1 is bound by shared memory: 176 KB go in and out a tile (K and
// V, V read and written three times as wide, the operands read), 1,400 cycles
// of the 1,850 that its products take one behind the other; the output warps'
// help with V' (16 warps instead of 8) changed nothing.  Small passes are bound by
// latency: launch, their tiles through phase 1, the grid-wide counter, their tiles
// through phase 2.
//
// The runs are cut to equal numbers of tiles, whatever they are: with the tiles
// that have a phase-1 part weighted 2 : 1 against packed branches, sixteen requests
// took 565 us, with 5 : 4 524, with 4 : 5 539, with 1 : 1 514.
//
// Where the decay enters:
//   scores   in fp32, as P leaves tensor memory to become the bf16 operand of
//            P V: a row's factors fall by a from each column to the one
//            before (running products of a^4, at most eight factors deep,
//            from a power at the block's last column); in the 32 x 32 blocks on
//            the diagonal of a head with a < 1/16, where those would start above
//            1 by more than fp32 holds, products of a from the diagonal down.
//   Q S      a row factor, which no rounding to bf16 should see: Q S has its own
//            accumulator, and the output warps add a^(i-s(i)+1) times it to P V.
//   K^T V    by scaling V, fp32, as a sum of three bf16 numbers (24 bits: exactly
//            the fp32 product), side by side as one operand of 192 columns.  The
//            state is kept to fp32 accuracy that way; V' rounded to bf16 once
//            would leave it 2e-3 off, twice 3e-6.  (A factor on the tensor
//            memory side is not possible: the rows j are the summed dimension.)
//
// 19 warps:
//   warp 0      producer: K, V tiles of phase 1, then Q, K, V tiles and table
//               entries, by TMA and bulk copies.
//   warp 1      front issuer: phase 1, K^T V'; then per tile P = Q K^T.
//   warp 2      O issuer: P V, then Q S.
//   warps 3-10  phase 1: V' (16 bytes of V at a time; rows past the tile become
//               zero).  Then P, two warps per TMEM lane quarter, one per
//               64-column half; V's rows past the tile, infinities and NaNs
//               become zero first (see add_nonfinite).
//   warps 11-18 phase 1: the piece states, 16 columns of one state row per
//               thread.  Then S, staged in bf16, and O, 32 columns of one row
//               per thread.
#include "decay_math.cuh"
#include "span_tiles.cuh"
#include "spanla_internal.h"
#include "tc_ptx.cuh"

namespace spanla {
namespace {

constexpr int kThreads = 32 * (3 + 8 + 8);
constexpr int kGroupThreads = 32 * 8;                      // state and output
constexpr int kConvWarps = 8;                              // scaling and conversion
constexpr int kConvThreads = 32 * kConvWarps;
constexpr int kStateWarp0 = 3 + kConvWarps;                // first state/output warp
constexpr int kStages = 3;
constexpr int kSetupLoads = kFirstLoads < kStages ? kFirstLoads : kStages;   // loads on fresh stages
constexpr int kParts = 3;                                  // bf16 parts of V'
constexpr uint32_t kRowTileBytes = kTileRows * 128;        // 128 rows x 128 B
constexpr uint32_t kStageBytes = 3 * kRowTileBytes;        // Q K V
constexpr uint32_t kStateTileBytes = kHeadDim * 128;       // 64 rows x 128 B (bf16)
// An S operand: S in bf16 in its first 8 KB; O of two lane quarters on its way
// out in the second 8 KB (quarters 0, 1 in operand 0; 2, 3 in operand 1).
constexpr uint32_t kSOpBytes = 2 * kStateTileBytes;
constexpr uint32_t kOQuarterBytes = kOutStoreRows * 128;
static_assert(2 * kOQuarterBytes == kStateTileBytes, "two quarters of O staging per S operand");
constexpr int kP1Slots = 16;
constexpr int kSegSlots = 4;   // tiles whose segment starts are kept for the output warps
constexpr int kBadSlots = 8;   // tiles whose marks are (made before P(i): five tiles could be open)
// log2 a of a steep head: below it a^-31, the factor of a diagonal block's
// last column in its first row (a masked one), could pass the fp32 range.
constexpr float kSteepLog2 = -4.f;
constexpr uint32_t kTmemCols = 512;
// TMEM columns: P buffers (128 each), O and Q S buffers (64 each); in phase 1
// two K^T V' buffers of 192.
constexpr uint32_t kColP0 = 0, kColP1 = 128, kColO0 = 256, kColO1 = 320, kColQS0 = 384, kColQS1 = 448;
constexpr uint32_t kColsState = kParts * kHeadDim, kColD0 = 0, kColD1 = kColsState;
static_assert(2 * kColsState <= kTmemCols, "two K^T V' buffers");
constexpr uint32_t kNamedStateBar = 1;

struct DecaySmem {
  static constexpr uint32_t kStage0 = 0;
  static constexpr uint32_t kK = 0, kV = kRowTileBytes, kQ = 2 * kRowTileBytes;
  static constexpr uint32_t kS = kStages * kStageBytes;
  // The stages' table entries (phase 2).  In phase 1, which uses neither
  // those nor the S operands and Q, two V' buffers: buffer 0 here, buffer 1 in
  // the last stage's Q and the S operands, which lie together.
  static constexpr uint32_t kTable = kS + 2 * kSOpBytes;
  static constexpr uint32_t kVs0 = kTable, kVs1 = kS - kRowTileBytes;
  static_assert(kStages * kStateFloats * 4 == kParts * kRowTileBytes && 2 * kSOpBytes == (kParts - 1) * kRowTileBytes,
                "the V' buffers' places");
  static_assert(kQ + kRowTileBytes == kStageBytes, "the last stage's Q ends where the S operands begin");
  static constexpr uint32_t kBar = kTable + kStages * kStateFloats * 4;
  // Barriers; the pairs are used by alternate tiles.  Empty takes two
  // arrivals per use (both issuers read a tile's stage; the front issuer
  // arrives twice on a phase-1 stage), OReady two (the MMAs' completion and
  // the issuing thread, behind which the segment starts that the conversion
  // warps wrote are visible).
  static constexpr int kFull = 0, kEmpty = kStages, kPReady = 2 * kStages, kPDone = kPReady + 2, kOReady = kPReady + 4,
                       kOFree = kPReady + 6, kSSmem = kPReady + 8, kP1Ready = kPReady + 10, kP1Free = kPReady + 12,
                       kPFree = kPReady + 14, kVReady = kPReady + 16, kVFree = kPReady + 18, kP1Done = kPReady + 20,
                       kNumBars = kPReady + 21;
  static constexpr uint32_t kTmemSlot = kBar + 8 * kNumBars;
  static constexpr uint32_t kP1 = (kTmemSlot + 4 + 15) & ~15u;
  static constexpr uint32_t kSeg = kP1 + sizeof(DecayPiece) * kP1Slots;   // first row of each row's segment
  static constexpr uint32_t kBad = kSeg + kSegSlots * kTileRows;        // 1 + the tile whose V held an inf or NaN
  static constexpr uint32_t kBytes = kBad + 4 * kBadSlots;
  static constexpr uint32_t kRequest = kBytes + 1024;
};
static_assert(DecaySmem::kRequest <= 227 * 1024, "shared memory budget");

struct DecayParams {
  const CtaHead* heads;
  const DecayTile* work;
  const uint8_t* bounds;
  const float* log_decay;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const float* stateA;
  float* ws;
  float* table;           // states before the tiles of the pieces (thread-major, see table_at)
  float2* ws_factor;      // a^rows of each slot's piece, as a Factor
  float* final_out;
  __nv_bfloat16* out;
  unsigned* err;
  const DecayPiece* p1;
  unsigned* counter;
  unsigned target;
  int H;
  int n_p1_ctas;
};

// The parts of a tile record each role reads.
struct Start {   // rows and flags, the start state, the final state and the table's entries
  int32_t row0, nrows, head, flags, stateA, stateB, a_n, b_n, final_idx, slot;
};
__device__ __forceinline__ Start load_start(const DecayTile* p) {
  const int4 a = __ldg(reinterpret_cast<const int4*>(p));
  const int4 b = __ldg(reinterpret_cast<const int4*>(p) + 1);
  const int2 c = __ldg(reinterpret_cast<const int2*>(p) + 4);
  return Start{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y};
}
struct Mask {    // rows and segment starts (conversion)
  int32_t nrows, head, flags, bound0;
  uint4 inl;
  __device__ __forceinline__ int nbound() const { return flags >> kDecayBoundShift; }
};
__device__ __forceinline__ Mask load_mask4(const DecayTile* p) {
  const int4 a = __ldg(reinterpret_cast<const int4*>(p));
  const uint4 d = __ldg(reinterpret_cast<const uint4*>(p) + 3);
  return Mask{a.y, a.z, a.w, __ldg(&p->bound0), d};
}

// True when one of two bf16 is infinite or NaN (its exponent bits all set).
__device__ __forceinline__ bool nonfinite2(uint32_t w) { return ((w & 0x7fff7fffu) + 0x00800080u) & 0x80008000u; }
__device__ __forceinline__ bool nonfinite_lo(uint32_t w) { return (w & 0x7f80u) == 0x7f80u; }
__device__ __forceinline__ bool nonfinite_hi(uint32_t w) { return (w & 0x7f800000u) == 0x7f800000u; }

// (out of line: a few calls a piece)
__device__ __noinline__ Factor factor_of(float ld, float n) { return decay_factor(ld, n); }

// A tile's P V ran without the infinite and NaN values of V (they stand as 0
// in shared memory: 0 times one of them, in a masked place, would be NaN).
// Their terms a^(i-j) (q_i . k_j) v_jc, for the rows that see them: added to
// 32 columns of row i = `row` of the tile where the output has them already
// (whatever it holds there, one such term makes it infinite or NaN).
__device__ __noinline__ void add_nonfinite(const DecayParams& prm, int64_t row0, int row, int seg_start, int head, int col,
                                           float l2) {
  const int64_t stride = static_cast<int64_t>(prm.H) * kHeadDim;
  const int64_t at = row0 * stride + static_cast<int64_t>(head) * kHeadDim;
  uint32_t* out = reinterpret_cast<uint32_t*>(prm.out + at + row * stride + col);
  for (int j = seg_start; j <= row; ++j) {
    const uint32_t* v = reinterpret_cast<const uint32_t*>(prm.v + at + j * stride + col);
    bool any = false;
    for (int c = 0; c < 16; ++c) any |= nonfinite2(v[c]);
    if (!any) continue;
    float score = 0.f;
    for (int e = 0; e < kHeadDim; ++e)
      score = fmaf(__bfloat162float(prm.q[at + row * stride + e]), __bfloat162float(prm.k[at + j * stride + e]), score);
    score *= decay_pow(l2, static_cast<float>(row - j));
    for (int c = 0; c < 16; ++c) {
      if (!nonfinite2(v[c])) continue;
      const uint32_t o = __ldcg(out + c);
      float lo = __uint_as_float(o << 16), hi = __uint_as_float(o & 0xffff0000u);
      if (nonfinite_lo(v[c])) lo += score * __uint_as_float(v[c] << 16);
      if (nonfinite_hi(v[c])) hi += score * __uint_as_float(v[c] & 0xffff0000u);
      out[c] = pack_bf16x2(lo, hi);
    }
  }
}

// Two fp32 numbers (24 bits) as sums of three bf16 each (8 bits), packed:
// cut off 16 bits, then the rest's, exactly.
__device__ __forceinline__ void split3(uint64_t x, uint32_t (&part)[kParts]) {
  const uint64_t minus = f32x2(-1.f, -1.f);
#pragma unroll
  for (int p = 0; p < kParts; ++p) {
    float lo, hi;
    f32x2_split(x, lo, hi);
    part[p] = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
    if (p + 1 < kParts)
      x = fma_f32x2(f32x2(__uint_as_float(__float_as_uint(lo) & 0xffff0000u), __uint_as_float(__float_as_uint(hi) & 0xffff0000u)),
                    minus, x);
  }
}

// The infinite and NaN ones among 16 products sum_j a^(rows-1-j) k_jd v_jc (c
// from col on), once more from the definition: an infinity in K or V met parts of
// V' that are 0 or a remainder of itself, and made NaN where the sum is infinite.
__device__ __noinline__ void redo_products(const DecayParams& prm, int64_t row0, int rows, int head, int d, int col, float l2,
                                           float* x) {
  const int64_t stride = static_cast<int64_t>(prm.H) * kHeadDim;
  const int64_t at = row0 * stride + static_cast<int64_t>(head) * kHeadDim;
  float sum[16];
#pragma unroll
  for (int c = 0; c < 16; ++c) sum[c] = 0.f;
#pragma unroll 4
  for (int j = 0; j < rows; ++j) {
    const float f = decay_pow(l2, static_cast<float>(rows - 1 - j)) * __bfloat162float(prm.k[at + j * stride + d]);
    const uint32_t* v = reinterpret_cast<const uint32_t*>(prm.v + at + j * stride + col);
#pragma unroll
    for (int c = 0; c < 16; c += 2) {
      const uint32_t w = v[c / 2];
      sum[c] = fmaf(f, __uint_as_float(w << 16), sum[c]);
      sum[c + 1] = fmaf(f, __uint_as_float(w & 0xffff0000u), sum[c + 1]);
    }
  }
#pragma unroll
  for (int c = 0; c < 16; ++c)
    if (!isfinite(x[c])) x[c] = sum[c];
}
// Zeros in place of the infinite and NaN ones of eight values of V.
__device__ __noinline__ void clear_nonfinite(uint8_t* src) {
  uint32_t* v = reinterpret_cast<uint32_t*>(src);
  for (int e = 0; e < 4; ++e) v[e] &= (nonfinite_lo(v[e]) ? 0u : 0xffffu) | (nonfinite_hi(v[e]) ? 0u : 0xffff0000u);
}

__global__ void __launch_bounds__(kThreads, 1)
span_decay_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                  const __grid_constant__ DecayParams prm) {
  using L = DecaySmem;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const int H = prm.H;
  unsigned* err = prm.err;

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  auto bar = [&](int slot) { return base + L::kBar + 8u * slot; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kTmemSlot);

  const int4* hd = reinterpret_cast<const int4*>(prm.heads + blockIdx.x);
  const int4 h0 = __ldg(hd), h1 = __ldg(hd + 1);
  const int i_begin = h0.x, n = h0.y, p1_begin = h0.z, n_p1 = h0.w;
  const int n1 = h1.x;                                   // phase-1 tiles
  const bool counted = h1.z != 0;                        // others wait for this CTA's slots
  // Loads issued during the set-up: phase 1's, or else the run's.
  const int n_first = min(n1 > 0 ? n1 : h1.y, kSetupLoads);
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(L::kFull + s), 1);
      mbar_init(bar(L::kEmpty + s), 2);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(L::kPReady + b), 1);
      mbar_init(bar(L::kPDone + b), kConvThreads);
      mbar_init(bar(L::kOReady + b), 2);
      mbar_init(bar(L::kPFree + b), 1);
      mbar_init(bar(L::kOFree + b), kGroupThreads);
      mbar_init(bar(L::kSSmem + b), kGroupThreads);
      mbar_init(bar(L::kP1Ready + b), 1);
      mbar_init(bar(L::kP1Free + b), kGroupThreads);
      mbar_init(bar(L::kVReady + b), kConvThreads);
      mbar_init(bar(L::kVFree + b), 1);
    }
    mbar_init(bar(L::kP1Done), kGroupThreads);
    for (int s = 0; s < kBadSlots; ++s) reinterpret_cast<int*>(smem + L::kBad)[s] = 0;
    fence_mbar_init();
    const int4 f0 = __ldg(hd + 2), f1 = __ldg(hd + 3);
    const int fr[2 * kFirstLoads] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
#pragma unroll
    for (int u = 0; u < kSetupLoads; ++u) {
      if (u < n_first) {   // (phase-1 tiles, or a run's when there are none)
        const uint32_t st = base + L::kStage0 + u * kStageBytes;
        mbar_arrive_expect_tx(bar(L::kFull + u), u < n1 ? 2 * kRowTileBytes : kStageBytes);
        if (u >= n1) tma_load_3d(st + L::kQ, &tm_q, bar(L::kFull + u), 0, fr[2 * u], fr[2 * u + 1]);
        tma_load_3d(st + L::kK, &tm_k, bar(L::kFull + u), 0, fr[2 * u], fr[2 * u + 1]);
        tma_load_3d(st + L::kV, &tm_v, bar(L::kFull + u), 0, fr[2 * u], fr[2 * u + 1]);
      }
    }
    tma_prefetch_desc(&tm_o);
  }

  const DecayTile* list = prm.work + i_begin;
  const DecayPiece* p1 = prm.p1 + p1_begin;
  DecayPiece* p1s = reinterpret_cast<DecayPiece*>(smem + L::kP1);
  if (warp == 2) {   // idle until the set-up completes: stages the phase-1 pieces
    for (int j = lane; j < n_p1 && j < kP1Slots; j += 32) p1s[j] = p1[j];
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  auto p1_of = [&](int j) { return j < kP1Slots ? p1s[j] : p1[j]; };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      bool ok = true;
      int u = 0;   // load index: phase-1 tiles, then the run's tiles
      for (int j = 0; j < n_p1 && ok; ++j) {
        const DecayPiece sd = p1_of(j);
        for (int r = 0; r < sd.len && ok; r += kTileRows, ++u) {
          if (u < n_first) continue;   // issued during the set-up
          const int s = u % kStages;
          if (!wait_or_flag(bar(L::kEmpty + s), ((u / kStages) & 1) ^ 1, err, kErrTimeoutMma)) { ok = false; break; }
          const uint32_t st = base + L::kStage0 + s * kStageBytes;
          mbar_arrive_expect_tx(bar(L::kFull + s), 2 * kRowTileBytes);
          tma_load_3d(st + L::kK, &tm_k, bar(L::kFull + s), 0, sd.row0 + r, sd.head);
          tma_load_3d(st + L::kV, &tm_v, bar(L::kFull + s), 0, sd.row0 + r, sd.head);
        }
      }
      bool p1_over = n_p1 == 0;   // phase 1's V' buffers are free and its table is written
      auto wait_p1 = [&]() {
        if (!p1_over) ok = wait_or_flag(bar(L::kP1Done), 0, err, kErrTimeoutMma);
        p1_over = true;
      };
      int t = 0;   // tile of its piece
      int4 nxt = n > 0 ? __ldg(reinterpret_cast<const int4*>(list)) : int4{};   // row0, nrows, head, flags
      int nxt_table0 = n > 0 ? __ldg(&list->table0) : 0;
      for (int i = 0; i < n && ok; ++i, ++u) {
        const int4 h = nxt;
        const int table0 = nxt_table0;
        if (i + 1 < n) {
          nxt = __ldg(reinterpret_cast<const int4*>(list + i + 1));
          nxt_table0 = __ldg(&list[i + 1].table0);
        }
        t = (h.w & kTileFirst) ? 0 : t + 1;
        if (u < n_first) continue;
        const int s = u % kStages;
        if (!wait_or_flag(bar(L::kEmpty + s), ((u / kStages) & 1) ^ 1, err, kErrTimeoutMma)) { ok = false; break; }
        const uint32_t st = base + L::kStage0 + s * kStageBytes;
        mbar_arrive_expect_tx(bar(L::kFull + s), kStageBytes + (t > 0 ? kStateFloats * 4 : 0));
        tma_load_3d(st + L::kK, &tm_k, bar(L::kFull + s), 0, h.x, h.z);
        tma_load_3d(st + L::kV, &tm_v, bar(L::kFull + s), 0, h.x, h.z);
        if (s == kStages - 1) wait_p1();
        tma_load_3d(st + L::kQ, &tm_q, bar(L::kFull + s), 0, h.x, h.z);
        if (t > 0) {
          wait_p1();
          bulk_copy_g2s(base + L::kTable + s * (kStateFloats * 4),
                        prm.table + (static_cast<int64_t>(table0) + t - 1) * kStateFloats, kStateFloats * 4,
                        bar(L::kFull + s));
        }
      }
      // Wait (bounded) for the last loads to land before the CTA can exit.
      for (int w = (u > kStages ? u - kStages : 0); w < u; ++w)
        mbar_wait_bounded(bar(L::kFull + w % kStages), (w / kStages) & 1, ok ? kWaitLimitNs : 1000000ull);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ front issuer
    constexpr uint32_t id_qk = idesc_bf16_f32(128, 128, 0, 0);
    constexpr uint32_t id_kv = idesc_bf16_f32(128, kColsState, 1, 1);
    bool ok = true;
    int u = 0;
    // Phase 1: [K | K]^T [V'_0 V'_1 V'_2] of each tile of the pieces.  (Both
    // 64-wide M atoms read the K tile: leading byte offset 0; TMEM lanes
    // 64..127 get a second copy of rows 0..63.)
    for (int j = 0; j < n_p1 && ok; ++j) {
      const DecayPiece sd = p1_of(j);
      for (int r = 0; r < sd.len; r += kTileRows, ++u) {
        const int s = u % kStages, b = u & 1;
        ok = wait_or_flag(bar(L::kFull + s), (u / kStages) & 1, err, kErrTimeoutTma);
        if (!__all_sync(0xffffffffu, ok)) break;
        const uint32_t st = base + L::kStage0 + s * kStageBytes;
        if (sd.len - r < kTileRows) {
          // K rows past the piece may hold anything, even NaN: zeros.
          uint8_t* krow = smem + (st + L::kK - base);
          for (int q = (sd.len - r) * 8 + lane; q < kTileRows * 8; q += 32)
            *reinterpret_cast<uint4*>(krow + q * 16) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();   // (lane 0 issues the product)
        }
        ok = wait_or_flag(bar(L::kVReady + b), (u >> 1) & 1, err, kErrTimeoutMma);
        if (ok && u >= 2) ok = wait_or_flag(bar(L::kP1Free + b), ((u - 2) >> 1) & 1, err, kErrTimeoutMma);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after_sync();
        if (lane == 0) {
          const uint64_t dk = smem_desc_sw128(st + L::kK, 0, 1024);
          const uint64_t dv = smem_desc_sw128(base + (b ? L::kVs1 : L::kVs0), kRowTileBytes, 1024);
#pragma unroll
          for (int kk = 0; kk < kTileRows / 16; ++kk)   // (addresses in units of 16 bytes)
            mma_bf16(tmem + (b ? kColD1 : kColD0), dk + kk * (2048 / 16), dv + kk * (2048 / 16), id_kv, kk > 0 ? 1u : 0u);
          mma_commit(bar(L::kP1Ready + b));
          mma_commit(bar(L::kVFree + b));
          mma_commit(bar(L::kEmpty + s));
          mma_commit(bar(L::kEmpty + s));
        }
        __syncwarp();
      }
    }
    // The run's tiles take the columns once phase 1 has been read out.
    ok = __all_sync(0xffffffffu, ok);
    if (ok && n_p1 > 0) ok = wait_or_flag(bar(L::kP1Done), 0, err, kErrTimeoutMma);
    ok = __all_sync(0xffffffffu, ok);
    for (int i = 0; i < n && ok; ++i, ++u) {
      const int s = u % kStages, b = i & 1;
      ok = wait_or_flag(bar(L::kFull + s), (u / kStages) & 1, err, kErrTimeoutTma);
      // P buffer b is free once P V of tile i-2 has completed.
      if (ok && i >= 2) ok = wait_or_flag(bar(L::kPFree + b), ((i - 2) >> 1) & 1, err, kErrTimeoutMma);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after_sync();
      if (lane == 0) {
        const uint32_t st = base + L::kStage0 + s * kStageBytes;
        const uint64_t dq = smem_desc_sw128(st + L::kQ, 16, 1024), dk = smem_desc_sw128(st + L::kK, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < kHeadDim / 16; ++kk)
          mma_bf16(tmem + (b ? kColP1 : kColP0), dq + kk * 2, dk + kk * 2, id_qk, kk > 0 ? 1u : 0u);
        mma_commit(bar(L::kPReady + b));
        mma_commit(bar(L::kEmpty + s));
      }
      __syncwarp();
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ O issuer
    constexpr uint32_t id_n64_b_mn = idesc_bf16_f32(128, 64, 0, 1);
    int flags = n > 0 ? __ldg(&list->flags) : 0;
    for (int i = 0; i < n; ++i) {
      const bool has_state = !(flags & kTileFirst) || (flags & kTileHasInit);
      if (i + 1 < n) flags = __ldg(&list[i + 1].flags);
      const int u = n1 + i;
      const int s = u % kStages, b = i & 1;
      const uint32_t st = base + L::kStage0 + s * kStageBytes;
      // P(i) is bf16 in TMEM, and O(i-2) and its Q S have been read: P V.
      bool ok = wait_or_flag(bar(L::kPDone + b), (i >> 1) & 1, err, kErrTimeoutMma);
      if (ok && i >= 2) ok = wait_or_flag(bar(L::kOFree + b), ((i - 2) >> 1) & 1, err, kErrTimeoutMma);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after_sync();
      if (lane == 0) {
        const uint32_t colP = tmem + (b ? kColP1 : kColP0);
        const uint64_t dv = smem_desc_sw128(st + L::kV, kRowTileBytes, 1024);
        // keys 0..63 of P in columns 0..31, keys 64..127 in columns 64..95
#pragma unroll
        for (int kk = 0; kk < kTileRows / 16; ++kk)
          mma_bf16_tmem_a(tmem + (b ? kColO1 : kColO0), colP + (kk < 4 ? kk * 8 : 64 + (kk - 4) * 8),
                          dv + kk * (2048 / 16), id_n64_b_mn, kk > 0 ? 1u : 0u);
        mma_commit(bar(L::kPFree + b));
      }
      __syncwarp();
      // S(i) staged: Q S.
      if (!__all_sync(0xffffffffu, wait_or_flag(bar(L::kSSmem + b), (i >> 1) & 1, err, kErrTimeoutMma))) break;
      tc_fence_after_sync();
      if (lane == 0) {
        if (has_state) {
          const uint64_t dq = smem_desc_sw128(st + L::kQ, 16, 1024);
          const uint64_t ds = smem_desc_sw128(base + L::kS + b * kSOpBytes, kStateTileBytes, 1024);
#pragma unroll
          for (int kk = 0; kk < kHeadDim / 16; ++kk)
            mma_bf16(tmem + (b ? kColQS1 : kColQS0), dq + kk * 2, ds + kk * (2048 / 16), id_n64_b_mn, kk > 0 ? 1u : 0u);
        }
        mma_commit(bar(L::kOReady + b));
        mma_commit(bar(L::kEmpty + s));
        mbar_arrive(bar(L::kOReady + b));
      }
      __syncwarp();
    }
  } else if (warp < 3 + kConvWarps) {
    // ------------------------------------------------------------ scaling and conversion
    const int ct = tid - 3 * 32;
    const int quarter = warp & 3;                 // TMEM lane quarter of this warp
    const int half = (warp - 3) >> 2;             // 64-column half of P this warp converts
    const int row = quarter * 32 + lane;          // tile row = TMEM lane
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t my16 = L::kV + ct * 16;   // this thread's 16-byte pieces of a V tile: every 4 KB from here
    constexpr int kPieces = kTileRows * 8 / kConvThreads;
    constexpr uint32_t kPieceStep = kConvThreads * 16;
    auto piece_row = [&](int w) { return (ct >> 3) + (kConvThreads / 8) * w; };   // (whatever the swizzle)
    bool ok = true;
    int u = 0;
    // Phase 1: V' of each tile: row r times a^(rows - 1 - r), zero past them.
    for (int j = 0; j < n_p1 && ok; ++j) {
      const DecayPiece sd = p1_of(j);
      const float l2 = decay_log2(load_log_decay(prm.log_decay, sd.head));
      for (int r0 = 0; r0 < sd.len; r0 += kTileRows, ++u) {
        const int rows = min(sd.len - r0, kTileRows);
        ok = wait_or_flag(bar(L::kFull + u % kStages), (u / kStages) & 1, err, kErrTimeoutTma);
        if (ok && u >= 2) ok = wait_or_flag(bar(L::kVFree + (u & 1)), ((u - 2) >> 1) & 1, err, kErrTimeoutMma);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint8_t* src = smem + L::kStage0 + (u % kStages) * kStageBytes + my16;
        uint8_t* dst = smem + ((u & 1) ? L::kVs1 : L::kVs0) + ct * 16;
#pragma unroll 4
        for (int w = 0; w < kPieces; ++w) {
          const int r = piece_row(w);
          const uint4 x4 = r < rows ? *reinterpret_cast<const uint4*>(src + kPieceStep * w) : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w};
          const float f = decay_pow_fast(l2, static_cast<float>(max(rows - 1 - r, 0)));
          uint4 part[kParts];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t b2[kParts];
            split3(mul_f32x2(f32x2(__uint_as_float(x[e] << 16), __uint_as_float(x[e] & 0xffff0000u)), f32x2(f, f)), b2);
#pragma unroll
            for (int p = 0; p < kParts; ++p) reinterpret_cast<uint32_t*>(&part[p])[e] = b2[p];
          }
#pragma unroll
          for (int p = 0; p < kParts; ++p)
            *reinterpret_cast<uint4*>(dst + p * kRowTileBytes + kPieceStep * w) = part[p];
        }
        fence_proxy_async_smem();
        mbar_arrive(bar(L::kVReady + (u & 1)));
      }
    }
    Mask nxt = n > 0 ? load_mask4(list) : Mask{};
    int head = -1;
    float l2 = 0.f;
    for (int i = 0; i < n && ok; ++i, ++u) {
      const Mask r = nxt;
      if (r.head != head) {   // (a load whose address is itself on its way would hold up every tile)
        head = r.head;
        l2 = decay_log2(load_log_decay(prm.log_decay, head));
      }
      if (i + 1 < n) nxt = load_mask4(list + i + 1);
      const int b = i & 1;
      if (!__all_sync(0xffffffffu, wait_or_flag(bar(L::kFull + u % kStages), (u / kStages) & 1, err, kErrTimeoutTma))) break;
      // V's rows past the tile, its infinities and NaNs become zero (0 times
      // one of those, in a masked place, would be NaN); the latter mark the tile.
      {
        uint8_t* src = smem + L::kStage0 + (u % kStages) * kStageBytes + my16;
        uint32_t bad = 0;
        uint4 x[kPieces];
#pragma unroll
        for (int w = 0; w < kPieces; ++w) x[w] = *reinterpret_cast<const uint4*>(src + kPieceStep * w);
#pragma unroll
        for (int w = 0; w < kPieces; ++w)
          bad |= (nonfinite2(x[w].x) | nonfinite2(x[w].y) | nonfinite2(x[w].z) | nonfinite2(x[w].w)) << w;
        if (bad != 0 || r.nrows < kTileRows) {
          for (int w = 0; w < kPieces; ++w) {
            if (piece_row(w) >= r.nrows) {
              *reinterpret_cast<uint4*>(src + kPieceStep * w) = make_uint4(0u, 0u, 0u, 0u);
            } else if ((bad >> w) & 1) {
              clear_nonfinite(src + kPieceStep * w);
              reinterpret_cast<int*>(smem + L::kBad)[i % kBadSlots] = i + 1;
            }
          }
          fence_proxy_async_smem();
        }
      }

      int seg_start = 0;
      const int nbound = r.nbound();
      if (nbound > 1) {
        const int nb = nbound < kInlineBounds ? nbound : kInlineBounds;
        for (int q = 1; q < nb; ++q) {
          const int sb = inline_bound(r.inl, q);
          if (sb <= row) seg_start = sb;
        }
        for (int q = kInlineBounds; q < nbound; ++q) {
          const int sb = prm.bounds[r.bound0 + q];
          if (sb <= row) seg_start = sb;
        }
      }
      const int hi_col = row < r.nrows ? row : -1;   // last kept column of this row
      if (!__all_sync(0xffffffffu, wait_or_flag(bar(L::kPReady + b), (i >> 1) & 1, err, kErrTimeoutMma)))
        break;
      tc_fence_after_sync();
      // The output warps read it once O(i) is ready.  The slot's last reader,
      // O(i-4), is behind: P(i) was issued after P V of tile i-2 completed, which
      // was issued once O(i-4)'s accumulators had been read (kOFree), behind the
      // read of the slot.
      if (half == 0) smem[L::kSeg + (i % kSegSlots) * kTileRows + row] = static_cast<uint8_t>(seg_start);
      const uint32_t colP = (b ? kColP1 : kColP0) + half * 64;
      // Two 32-column chunks in turn; chunk q's bf16 pairs go to columns
      // 16q .. 16q + 15 of the half, over scores already read.
#pragma unroll 1
      for (int q = 0; q < 2; ++q) {
        const int c0 = half * 64 + 32 * q;
        uint32_t pk[16];
        if (__all_sync(0xffffffffu, c0 > hi_col || c0 + 31 < seg_start)) {
#pragma unroll
          for (int c = 0; c < 16; ++c) pk[c] = 0u;
        } else {
          uint32_t r0[32];
          tmem_ld_32cols(tmem + lane_base + colP + 32 * q, r0);
          tmem_ld_wait();
          // Kept columns of this row: c0 + lo .. c0 + hi.
          const int lo = seg_start - c0, hi = hi_col - c0;
          const bool all_kept = __all_sync(0xffffffffu, lo <= 0 && hi >= 31);
          if (c0 == quarter * 32 && l2 < kSteepLog2) {
            // On the diagonal of a steep head: from the row's own column down.
            const float a1 = decay_pow_fast(l2, 1.f);
            float w = 1.f;
#pragma unroll
            for (int c = 31; c >= 0; --c) {
              w = c < lane ? w * a1 : 1.f;
              r0[c] = __float_as_uint(__uint_as_float(r0[c]) * w);
            }
          } else {
            // a^(row - column), from the last column down, two pairs at a time.
            const float step = decay_pow_fast(l2, 4.f);
            const uint64_t step2 = f32x2(step, step);
            uint64_t w[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
              w[e] = f32x2(decay_pow_fast(l2, static_cast<float>(row - (c0 + 28 + 2 * e))),
                           decay_pow_fast(l2, static_cast<float>(row - (c0 + 29 + 2 * e))));
#pragma unroll
            for (int c = 28; c >= 0; c -= 4)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float x0, x1;
                f32x2_split(mul_f32x2(f32x2(__uint_as_float(r0[c + 2 * e]), __uint_as_float(r0[c + 2 * e + 1])), w[e]), x0, x1);
                r0[c + 2 * e] = __float_as_uint(x0);
                r0[c + 2 * e + 1] = __float_as_uint(x1);
                w[e] = mul_f32x2(w[e], step2);
              }
          }
          if (!all_kept) {
            const uint32_t kept = (hi >= 31 ? ~0u : hi < 0 ? 0u : (2u << hi) - 1u) & (lo <= 0 ? ~0u : lo > 31 ? 0u : ~0u << lo);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!(kept & (1u << c))) r0[c] = 0u;
          }
          // Rounded to bf16, as the state is for Q S (stage_state_slice): the operand
          // type of the inputs, and the undecayed pass's way.  Each adds up to 2^-8 of
          // a term; the output is off by 0.0023 of its norm, of which its own rounding
          // is 0.0017.
#pragma unroll
          for (int c = 0; c < 16; ++c) pk[c] = pack_bf16x2(__uint_as_float(r0[2 * c]), __uint_as_float(r0[2 * c + 1]));
        }
        tmem_st_16cols(tmem + lane_base + colP + 16 * q, pk);
      }
      tmem_st_wait();
      tc_fence_before_sync();
      mbar_arrive(bar(L::kPDone + b));
    }
  } else {
    // ------------------------------------------------------------ state and output
    const int quarter = warp & 3;                 // TMEM lane quarter of this warp
    const int pi = (warp - kStateWarp0) >> 2;     // which of the quarter's two warps
    const int row = quarter * 32 + lane;          // tile row = TMEM lane
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    // State work: lanes 0..63 and their copy in lanes 64..127 hold state rows
    // d = row & 63; the lower copy handles columns 0..31, the upper 32..63,
    // and the quarter's two warps take 16 of those each.
    const int d = row & 63, sh = row >> 6;
    const int col0 = 32 * sh + 16 * pi;
    bool ok = true;
    // The table and the slots hold a state as this group's threads hold it:
    // float4 c of thread g at c * 256 + g, so that each writes and reads whole
    // lines.
    const int g = tid - kStateWarp0 * 32;
    auto table_at = [&](int64_t entry) { return reinterpret_cast<float4*>(prm.table + entry * kStateFloats) + g; };

    // Phase 1: S <- a^n S + K^T V' over the tiles of each piece.  (Tile by
    // tile, in fp32 rounded to nearest, which the tensor core's long sums are
    // not.)  Then this CTA counts itself.
    if (n_p1 > 0) {
      int u = 0;
      for (int j = 0; j < n_p1 && ok; ++j) {
        const DecayPiece sd = p1_of(j);
        const float ld = load_log_decay(prm.log_decay, sd.head);
        const Factor f_tile = factor_of(ld, static_cast<float>(kTileRows));
        float s[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = 0.f;
        int t = 0;
        for (int r = 0; r < sd.len; r += kTileRows, ++u, ++t) {
          const int b = u & 1;
          ok = __all_sync(0xffffffffu, wait_or_flag(bar(L::kP1Ready + b), (u >> 1) & 1, err, kErrTimeoutMma));
          if (!ok) break;
          tc_fence_after_sync();
          // the parts' products, smallest first
          const uint32_t at = tmem + lane_base + (b ? kColD1 : kColD0) + col0;
          uint32_t x[16], y[16];
          tmem_ld_16cols(at + 2 * kHeadDim, x);
          tmem_ld_16cols(at + kHeadDim, y);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) + __uint_as_float(y[e]));
          tmem_ld_16cols(at, y);
          tmem_ld_wait();
          tc_fence_before_sync();
          mbar_arrive(bar(L::kP1Free + b));
          float bad = 0.f;   // NaN if a product is infinite or NaN
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            x[e] = __float_as_uint(__uint_as_float(x[e]) + __uint_as_float(y[e]));
            bad = fmaf(__uint_as_float(x[e]), 0.f, bad);
          }
          if (bad != 0.f) {
            float z[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) z[e] = __uint_as_float(x[e]);
            redo_products(prm, sd.row0 + r, min(sd.len - r, kTileRows), sd.head, d, col0, decay_log2(ld), z);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(z[e]);
          }
          const Factor f = sd.len - r >= kTileRows ? f_tile : factor_of(ld, static_cast<float>(sd.len - r));
#pragma unroll
          for (int e = 0; e < 16; ++e) s[e] = f.step(s[e], __uint_as_float(x[e]));
          if (t < sd.n_table) {
            float4* p = table_at(static_cast<int64_t>(sd.table0) + t);
#pragma unroll
            for (int c = 0; c < 4; ++c) p[kGroupThreads * c] = make_float4(s[4 * c], s[4 * c + 1], s[4 * c + 2], s[4 * c + 3]);
          }
        }
        if (!ok) break;
        if (sd.slot >= 0) {
          float4* p = reinterpret_cast<float4*>(prm.ws + static_cast<int64_t>(sd.slot) * kStateFloats) + g;
#pragma unroll
          for (int c = 0; c < 4; ++c) p[kGroupThreads * c] = make_float4(s[4 * c], s[4 * c + 1], s[4 * c + 2], s[4 * c + 3]);
          if (g == 0) {
            const Factor f = factor_of(ld, static_cast<float>(sd.len));
            prm.ws_factor[sd.slot] = make_float2(f.hi, f.lo);
          }
        }
      }
      // (the producer reads the table by bulk copies, other CTAs the slots)
      asm volatile("fence.proxy.async;" ::: "memory");
      __threadfence();
      mbar_arrive(bar(L::kP1Done));
      named_barrier_sync(kNamedStateBar, kGroupThreads);   // (also for the slots' decays, which one thread writes)
      if (counted && g == 0) atomicAdd(prm.counter, 1u);
    }
    // Phase 2.  s_run is the start state of the piece at hand (row d, columns
    // col0 ..).  tag_run names it, tag_op the start state each S operand holds;
    // -1: none (see k_span_output.cu).
    const int64_t slice = static_cast<int64_t>(d) * kHeadDim + col0;
    float s_run[16];
    int64_t tag_run = -1, tag_op0 = -1, tag_op1 = -1;
    auto carry_tag = [&](int view, int head) -> int64_t {
      return (static_cast<int64_t>(1) << 62) | (static_cast<int64_t>(view) << 16) | head;
    };
    auto start_tag = [&](const Start& r) -> int64_t {
      if (!(r.flags & kTileFirst) || !(r.flags & kTileHasInit)) return -1;
      if (r.flags & kTileCarry) return carry_tag(r.final_idx, r.head);
      if (r.b_n > 0) return static_cast<int64_t>(1) << 61;   // (only the first piece of a CTA's run has earlier ones)
      return (static_cast<int64_t>(r.stateA) << 16) | r.head;   // (a_n goes by stateA)
    };
    // Wait (bounded) until every CTA whose slots others read has counted
    // itself, once, before the first read of such a slot.  (Each warp for
    // itself: a warp whose waits ran out has left the loop.)
    bool synced = prm.n_p1_ctas == 0;
    auto grid_sync = [&]() {
      if (synced) return;
      synced = true;
      if (lane == 0) {
        const unsigned long long t0 = global_timer_ns();
        while (ld_acquire_gpu(prm.counter) != prm.target) {
          if (global_timer_ns() - t0 > kWaitLimitNs) {
            atomicOr(err, kErrTimeoutMma);
            break;
          }
          __nanosleep(64);
        }
      }
      __syncwarp();
    };
    // This thread's slice of a state in the usual layout.
    auto load_row = [&](const float* p) {
      const float4* p4 = reinterpret_cast<const float4*>(p + slice);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float4 x = __ldcg(p4 + c);
        s_run[4 * c] = x.x; s_run[4 * c + 1] = x.y; s_run[4 * c + 2] = x.z; s_run[4 * c + 3] = x.w;
      }
    };
    // s_run <- a^rows s_run + slot k.
    auto add_slot = [&](int k) {
      const float2 f2 = __ldcg(prm.ws_factor + k);
      const Factor f{f2.x, f2.y};
      const float4* p = reinterpret_cast<const float4*>(prm.ws + static_cast<int64_t>(k) * kStateFloats) + g;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float4 x = __ldcg(p + kGroupThreads * c);
        s_run[4 * c] = f.step(s_run[4 * c], x.x);
        s_run[4 * c + 1] = f.step(s_run[4 * c + 1], x.y);
        s_run[4 * c + 2] = f.step(s_run[4 * c + 2], x.z);
        s_run[4 * c + 3] = f.step(s_run[4 * c + 3], x.w);
      }
    };
    // s_run becomes the start state of the piece of tile `r`: zero, the final
    // state this CTA computed (carry), the one it holds already, or term A (a
    // kept state, or the parent view-head's pieces) and term B (the segment's
    // earlier pieces) by Horner's rule.
    auto start_piece = [&](const Start& r) {
      const int64_t tag = start_tag(r);
      if (tag >= 0 && tag == tag_run) return;
      tag_run = tag;
#pragma unroll
      for (int e = 0; e < 16; ++e) s_run[e] = 0.f;
      if (tag < 0) return;
      if (r.flags & kTileCarry) {   // (a long branch ran in between: as this thread wrote it)
        load_row(prm.final_out + (static_cast<int64_t>(r.final_idx) * H + r.head) * kStateFloats);
        return;
      }
      const bool kept = prm.final_out == nullptr;
      if (r.b_n > 0 || !kept) grid_sync();
      if (kept) load_row(prm.stateA + (static_cast<int64_t>(r.stateA) * H + r.head) * kStateFloats);
      else
#pragma unroll 2
        for (int k = 0; k < r.a_n; ++k) add_slot(r.stateA + k);
#pragma unroll 2
      for (int k = 0; k < r.b_n; ++k) add_slot(r.stateB + k);
    };
    // A view-head's final state: its last piece's start state decayed over the
    // piece, plus the piece's own state.
    auto final_state = [&](const Start& r) {
      add_slot(r.slot);
      store_slice(prm.final_out + (static_cast<int64_t>(r.final_idx) * H + r.head) * kStateFloats + slice, s_run);
      tag_run = carry_tag(r.final_idx, r.head);
    };
    // S(i) -> S operand i & 1, unless it holds that start state already: the
    // start state for a piece's first tile, else a^rows times it plus the
    // table's entry in the tile's stage, `rows` rows into the piece.  The
    // operand was last read by Q S of tile i-2, whose completion o_work(i-2)
    // saw.  (The stage is released behind Q S, so behind this.)
    auto stage = [&](int i, const Start& r, float l2, int rows) -> bool {
      uint8_t* op = smem + L::kS + (i & 1) * kSOpBytes;
      if (r.flags & kTileFirst) {
        const int64_t tag = start_tag(r);
        const int64_t held = (i & 1) ? tag_op1 : tag_op0;
        if (tag >= 0 && tag != held) {
          stage_state_slice(op, d, col0, s_run);
          if (i & 1) tag_op1 = tag; else tag_op0 = tag;
        }
      } else {
        if (i & 1) tag_op1 = -1; else tag_op0 = -1;
        const int u = n1 + i;
        if (!__all_sync(0xffffffffu, wait_or_flag(bar(L::kFull + u % kStages), (u / kStages) & 1, err, kErrTimeoutTma)))
          return false;
        const float f = decay_pow_fast(l2, static_cast<float>(rows));
        const float4* x = reinterpret_cast<const float4*>(smem + L::kTable + (u % kStages) * (kStateFloats * 4)) + g;
        float y[16];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float4 xc = x[kGroupThreads * c];
          y[4 * c] = fmaf(f, s_run[4 * c], xc.x);
          y[4 * c + 1] = fmaf(f, s_run[4 * c + 1], xc.y);
          y[4 * c + 2] = fmaf(f, s_run[4 * c + 2], xc.z);
          y[4 * c + 3] = fmaf(f, s_run[4 * c + 3], xc.w);
        }
        stage_state_slice(op, d, col0, y);
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(L::kSSmem + (i & 1)));
      return true;
    };

    // O(i) = P V + a^(i-s(i)+1) Q S -> global (rows of the tile only), through
    // this warp's O staging when its 32 rows all lie in the tile (one TMA
    // store), else row by row.
    bool o_pending = false;   // this warp's last TMA store may still read its staging
    auto o_work = [&](int i, const Start& r, float l2) -> bool {
      const int b = i & 1;
      if (!__all_sync(0xffffffffu, wait_or_flag(bar(L::kOReady + b), (i >> 1) & 1, err, kErrTimeoutMma))) return false;
      tc_fence_after_sync();
      const uint32_t colO = b ? kColO1 : kColO0;
      const bool whole = (quarter + 1) * 32 <= r.nrows;
      const bool has_state = !(r.flags & kTileFirst) || (r.flags & kTileHasInit);
      uint8_t* ob = smem + L::kS + (quarter >> 1) * kSOpBytes + kStateTileBytes + (quarter & 1) * kOQuarterBytes +
                    pi * (kOQuarterBytes / 2);
      if (whole && o_pending) {
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
      }
      uint4* dst = reinterpret_cast<uint4*>(
          prm.out + ((static_cast<int64_t>(r.row0) + row) * H + r.head) * kHeadDim + 32 * pi);
      const bool store = row < r.nrows;
      const int seg_start = smem[L::kSeg + (i % kSegSlots) * kTileRows + row];
      const bool bad = reinterpret_cast<const int*>(smem + L::kBad)[i % kBadSlots] == i + 1;
      const float f = decay_pow_fast(l2, static_cast<float>(row - seg_start + 1));
      uint32_t pk[16];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t r0[16];
        tmem_ld_16cols(tmem + lane_base + colO + 32 * pi + 16 * hf, r0);
        if (has_state) {
          uint32_t r1[16];
          tmem_ld_16cols(tmem + lane_base + (b ? kColQS1 : kColQS0) + 32 * pi + 16 * hf, r1);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) r0[e] = __float_as_uint(fmaf(f, __uint_as_float(r1[e]), __uint_as_float(r0[e])));
        } else {
          tmem_ld_wait();
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          pk[8 * hf + e] = pack_bf16x2(__uint_as_float(r0[2 * e]), __uint_as_float(r0[2 * e + 1]));
      }
      tc_fence_before_sync();
      mbar_arrive(bar(L::kOFree + b));
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint4 v4 = make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        if (whole)
          *reinterpret_cast<uint4*>(ob + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) = v4;
        else if (store)
          dst[c] = v4;
      }
      if (whole) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(&tm_o, smem_addr(ob), 32 * pi, r.row0 + quarter * 32, r.head);
          bulk_commit_group();
        }
        o_pending = true;
      }
      if (bad) {
        if (lane == 0) bulk_wait_all();
        __syncwarp();
        if (store) add_nonfinite(prm, r.row0, row, seg_start, r.head, 32 * pi, l2);
      }
      return true;
    };

    // (A warp whose bounded wait ran out leaves the loop: no barrier in it waits
    // for warps.)
    if (n > 0 && ok) {
      Start cur = load_start(list);
      Start nxt = n > 1 ? load_start(list + 1) : Start{};
      float l2 = decay_log2(load_log_decay(prm.log_decay, cur.head));
      int rows = 0;   // rows of the piece before the tile to stage
      start_piece(cur);
      ok = stage(0, cur, l2, 0);
      for (int i = 0; i < n && ok; ++i) {
        float l2_next = l2;
        if (cur.flags & kTileFinalOut) final_state(cur);
        if (i + 1 < n) {
          // S(i+1) first: the O issuer needs it right after P V of tile i+1.
          rows += cur.nrows;
          if (cur.flags & kTileLast) {
            if (nxt.head != cur.head) l2_next = decay_log2(load_log_decay(prm.log_decay, nxt.head));
            rows = 0;
            start_piece(nxt);
          }
          if (!stage(i + 1, nxt, l2_next, rows)) break;
        }
        ok = o_work(i, cur, l2);
        cur = nxt;
        l2 = l2_next;
        if (i + 2 < n) nxt = load_start(list + i + 2);
      }
    }
    if (lane == 0) bulk_wait_all();   // the last O stores have completed
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace

cudaError_t launch_span_decay(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                              const CUtensorMap& tm_o, const SpanDecayArgs& a, cudaStream_t stream) {
  if (a.grid <= 0) return cudaSuccess;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = set_smem_limit_once(span_decay_kernel, DecaySmem::kRequest, done);
  if (e != cudaSuccess) return e;
  DecayParams p{};
  p.heads = a.heads;
  p.work = a.work;
  p.bounds = a.bounds;
  p.log_decay = a.log_decay;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k = static_cast<const __nv_bfloat16*>(a.k);
  p.v = static_cast<const __nv_bfloat16*>(a.v);
  p.stateA = a.stateA;
  p.ws = a.ws;
  p.table = a.table;
  p.ws_factor = a.ws_factor;
  p.final_out = a.final_out;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.err = a.err;
  p.p1 = a.p1;
  p.counter = a.counter;
  p.target = a.target;
  p.H = a.H;
  p.n_p1_ctas = a.n_p1_ctas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = DecaySmem::kRequest;
  cfg.stream = stream;
  // CTAs wait on one another when some have phase-1 pieces: then all of them
  // must be resident at once.
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.n_p1_ctas > 0 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, span_decay_kernel, tm_q, tm_k, tm_v, tm_o, p);
}

}  // namespace spanla
