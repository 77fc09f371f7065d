// Softmax attention of a few new rows of each sequence (the next token, some
// drafted ones) over the paged cache: row heads r * group + g of one sequence and
// key head, at most 16 of them, against all of the sequence's cached rows.
//
// Bound by memory: every cached row and head is read once, 256 bytes of bf16 or
// 130 of e4m3, for 256 multiply-adds a row head.  So the cached rows are cut into
// units of 8 KB (32 rows of bf16, 64 of e4m3), numbered through all sequences, key
// heads and rows, and every warp of the card gets the same number of consecutive
// units, whatever the lengths: a warp finds its first unit by the sequences'
// running sums, and streams its units through a ring of its own, filled by TMA (its
// lane 0), without waiting for other warps.  The lengths are device memory: every
// CTA sums them up for itself.
//
// A unit: S = Q K^T (m16n8k16, the row heads as M), running maximum m and sum l of
// each row head in registers, O += P V.  bf16 pages: P enters as two bf16 parts
// (hi + lo, 2^-16 of it), the M = 16 products being free beside the loads.  e4m3
// pages: q, K and V enter as fp16 (K and V exactly, q scaled by a power of two
// for its row, then all but its least elements), the rows' powers of two go onto
// the scores and the weights in fp32; the weights w_j = p_j 2^(e_j) have a running
// maximum 2^M of their own and enter 2^15 times over it, so that fp16 holds them to
// 2^-11 of each, or 2^-40 of the largest.  Products that add to the same sums stand
// apart in the code: one behind the other they would wait for each other.
//
// A warp's first and last items may go on in other warps.  Those parts (m, M, l,
// O) meet in shared memory for the warps of a CTA and then, for the items that go
// over several CTAs, in the join kernel, which starts behind this one.
//
// Measured (with the join, one call behind the other): 128 tokens of up to 18,000
// rows over bf16 pages, 8 key heads of 4, 222 us, 6.8 TB/s, as fast as a copy; 61
// over e4m3 pages, 16 heads, 117 us, 5.4 TB/s (a warp takes 790 instructions for
// 64 rows of e4m3, and the chains of eleven warps leave half of the SM's issue slots
// empty).  One token of one sequence, 7,401 rows, 16 heads, 11.4 us, of which the
// data are 4.5: the lengths are there after 1.0, the first unit's data after 2.9,
// the last unit is done after 7.4, the warps' parts are one after 8.5, and the join
// begins after 9.5 and takes 2.
#include <algorithm>
#include <type_traits>

#include "paged_join.cuh"

namespace spanla {
namespace {

// kTwo: up to 16 row heads, as 8 and 8 (else up to 8, and the products' second half is empty).
template <bool kE4m3, bool kTwo>
struct Cfg {
  static constexpr int kUnit = kE4m3 ? 64 : 32;                // cached rows
  // e4m3 pages keep a warp busier for its bytes (conversions): as many warps as fit beside their rings.  (61 tokens:
  // 8 warps 126 us, 10 132, 11 119.  bf16 pages, 128 tokens: 8 warps 231 us, 10 239, 11 242; three units in flight a warp
  // instead of two: 245.)
  static constexpr int kWarps = kE4m3 && !kTwo ? 11 : 8;
  static constexpr int kStages = 2;
  static constexpr int kRows = kTwo ? 16 : 8;                  // row heads of a part in shared memory
  static constexpr int kSlot = kRows * kSlotStride + 3 * kM;   // its floats
  static constexpr uint32_t kRow = kE4m3 ? 64 : 128;           // bytes
  static constexpr uint32_t kHalf = kUnit * kRow;              // K or V of a unit
  static constexpr uint32_t kStage = 2 * kHalf;
  static constexpr uint32_t kRing = kStages * kStage;          // of a warp
  static constexpr uint32_t kScales = kWarps * kRing;          // 2 x kUnit bytes a stage
  static constexpr uint32_t kFactors = kScales + (kE4m3 ? kWarps * kStages * 2 * kUnit : 0);   // of a unit's rows, 8 bytes
  static constexpr uint32_t kHead = kFactors + (kE4m3 ? kWarps * kUnit * 8 : 0);
  static constexpr uint32_t kSum = kHead + kWarps * kSlot * 4;
  static constexpr uint32_t kLen = kSum + (kStepSeqs + 1) * 8;
  static constexpr uint32_t kRow0 = kLen + kStepSeqs * 4;
  static constexpr uint32_t kCount = kRow0 + kStepSeqs * 4;
  static constexpr uint32_t kInfo = kCount + kStepSeqs;        // 8 bytes a stage: the rows that are there
  static constexpr uint32_t kScan = kInfo + kWarps * kStages * 8;
  static constexpr uint32_t kBar = kScan + kWarps * 8;
  static constexpr uint32_t kOpen = kBar + kWarps * kStages * 8;   // Open of each warp, and one more
  static constexpr uint32_t kRedo = (kOpen + (kWarps + 1) * 24 + 15) & ~15u;   // StepRedo of each warp
  static constexpr uint32_t kBytes = kRedo + kWarps * 16;
  static constexpr uint32_t kRequest = kBytes + 1024;
  static_assert(kRequest <= 227 * 1024 && kRing >= kSlot * 4 && kInfo % 8 == 0 && kSum % 16 == 0 && kHead % 16 == 0, "shared memory");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// Two sums at once, two products.  (One by one 118.4 us instead of 115.5 for 61 tokens over e4m3 pages.)
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(f32x2(x, y)), "l"(f32x2(a, b)));
  f32x2_split(d, x, y);
}
__device__ __forceinline__ void mul2(float& x, float& y, float a, float b) { f32x2_split(mul_f32x2(f32x2(x, y), f32x2(a, b)), x, y); }

template <bool kHalfFloat>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (kHalfFloat)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2, int c3,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "l"(policy)
      : "memory");
}

// Where a warp is in the numbered units.
struct At {
  int s, h;            // sequence (of this launch), key head
  int32_t blk, units;  // unit of the item, units of the item
};

// An item of several parts, by the warp in which it begins (or the CTA's first one).
struct Open {
  int64_t begin;       // its first unit
  int32_t units, s, h; // units 0: none
};

// Output of a row head: elements d, d + 1.
__device__ __forceinline__ void store_pair(const PagedAttn& p, int64_t at, int d, float x, float y) {
  *reinterpret_cast<uint32_t*>(p.out + at * kHeadDim + d) = pack_bf16x2(x, y);
}

// kWhole: the CTAs take whole items, there is no workspace, and no join kernel behind.
template <bool kE4m3, bool kTwo, bool kWhole>
__global__ void __launch_bounds__(Cfg<kE4m3, kTwo>::kWarps * 32, 1)
paged_step_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ KvArgs a,
                  const __grid_constant__ PagedAttn p, int s0, int ns, bool behind, float* ws) {
  using C = Cfg<kE4m3, kTwo>;
  constexpr int kW = C::kWarps, kS = C::kStages, kUnit = C::kUnit, kN = kUnit / 8, kR = kTwo ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  int64_t* sum = reinterpret_cast<int64_t*>(smem + C::kSum);
  int32_t* s_len = reinterpret_cast<int32_t*>(smem + C::kLen);
  int32_t* s_row0 = reinterpret_cast<int32_t*>(smem + C::kRow0);
  uint8_t* s_count = smem + C::kCount;
  auto bar = [&](int stage) { return base + C::kBar + 8u * (warp * kS + stage); };
  auto units_of = [](int32_t len) { return max(1, (len + kUnit - 1) / kUnit); };

  if (lane == 0) {
    for (int i = 0; i < kS; ++i) mbar_init(bar(i), 1);
    fence_mbar_init();
    if (warp == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
  }
  // Behind the call's chunk kernel, which has waited for what comes before the call, and works on other sequences: no wait
  // but one CTA's at the end, as what comes behind waits for this grid alone.
  if (!behind) griddep_wait();
  griddep_launch_dependents();
  // ---------------------------------------------------------------- the sequences' running sums of units
  {
    const int per = (ns + kW * 32 - 1) / (kW * 32), b = min(ns, tid * per), e = min(ns, b + per);
    bool bad = false;
    int64_t mine = 0;
    for (int s = b; s < e; ++s) {
      const SeqRows r = seq_rows(a, s0 + s, &bad);
      const bool here = r.n > 0 && static_cast<int64_t>(r.n) * p.group <= kM;
      s_len[s] = r.len;
      s_row0[s] = static_cast<int32_t>(r.row0);
      s_count[s] = here ? static_cast<uint8_t>(r.n) : 0;
      sum[s] = mine;
      mine += here ? static_cast<int64_t>(units_of(r.len)) * a.heads : 0;
    }
    if (bad) atomicOr(a.err, kErrSequence);
    int64_t upto = mine;
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += x;
    }
    int64_t* scan = reinterpret_cast<int64_t*>(smem + C::kScan);
    if (lane == 31) scan[warp] = upto;
    __syncthreads();
    int64_t before = upto - mine;
    for (int w = 0; w < warp; ++w) before += scan[w];
    for (int s = b; s < e; ++s) sum[s] += before;
    if (tid == kW * 32 - 1) sum[ns] = before + mine;
    __syncthreads();
  }
  // ---------------------------------------------------------------- this warp's units
  // nw warps are at work, each has a unit at least: the first `more` have each + 1 of them, the others `each`.
  struct Shares {
    int64_t nw, each, more;
  };
  auto shares = [&]() -> Shares {   // (twice, and not in registers meanwhile)
    const int64_t U = *const_cast<volatile int64_t*>(sum + ns), nw = max(static_cast<int64_t>(1), min(static_cast<int64_t>(gridDim.x) * kW, U));
    const int64_t each = quotient(U, nw);
    return {nw, each, U - each * nw};
  };
  const Shares sh = shares();
  auto locate = [&](int64_t x, At& at) {
    int l = 0, r = ns;   // the last sequence that starts at x or before
    while (r - l > 1) {
      const int mid = (l + r) >> 1;
      if (sum[mid] <= x) l = mid;
      else r = mid;
    }
    at.s = l;
    at.units = units_of(s_len[l]);
    const int64_t in = x - sum[l];
    at.h = static_cast<int>(quotient(in, at.units));
    at.blk = static_cast<int32_t>(in - static_cast<int64_t>(at.h) * at.units);
  };
  const int64_t edge_w = min(sh.nw, static_cast<int64_t>(blockIdx.x) * kW + min(lane, kW));
  int64_t edge = sh.each * edge_w + min(edge_w, sh.more);               // lane w: the first unit of the CTA's warp w
  auto edge_of = [&](int w) { return __shfl_sync(0xffffffffu, edge, w); };
  if (kWhole) {
    // Items of a few units each: a CTA takes those that begin in its share, whole, and shares them out to its warps
    // (the first ones, where there are fewer units than warps).
    At at{};
    if (edge < sum[ns]) {
      locate(edge, at);
      edge -= at.blk;
    }
    const int64_t b = edge_of(0), n = edge_of(kW) - b, w = max(static_cast<int64_t>(1), min(static_cast<int64_t>(kW), n));
    const int64_t per = quotient(n, w), rest = n - per * w, i = min(static_cast<int64_t>(lane), w);
    edge = b + per * i + min(i, rest);
  }
  const int64_t lo = edge_of(warp), hi = edge_of(warp + 1);
  auto advance = [&](At& at) {
    if (++at.blk < at.units) return;
    at.blk = 0;
    if (++at.h < a.heads) return;
    at.h = 0;
    do ++at.s;
    while (at.s < ns && sum[at.s + 1] == sum[at.s]);
    at.units = at.s < ns ? units_of(s_len[at.s]) : 1;
  };

  const uint32_t ring = base + warp * C::kRing;
  uint8_t* ring_p = smem + warp * C::kRing;
  uint64_t* info = reinterpret_cast<uint64_t*>(smem + C::kInfo) + warp * kS;
  float* factors = reinterpret_cast<float*>(smem + C::kFactors) + warp * kUnit * 2;
  uint8_t* scales = smem + C::kScales + warp * kS * 2 * kUnit;
  // A part that began in an earlier warp stands in the head slot, one that goes on in later ones in the ring, which is
  // done by then.
  auto slot_of = [&](int w, bool head) {
    return head ? reinterpret_cast<float*>(smem + C::kHead) + w * C::kSlot : reinterpret_cast<float*>(smem + w * C::kRing);
  };
  constexpr int kStats = C::kRows * kSlotStride;   // in a slot in shared memory: m, M and l behind O

  // ---------------------------------------------------------------- loads
  constexpr uint64_t kAll = kUnit == 64 ? ~0ull : (1ull << (kUnit & 63)) - 1ull;
  const uint64_t policy = l2_evict_first_policy();
  const int32_t box = min(a.page_rows, kUnit), copies = kUnit / box;   // copies: pages of a unit, at most 4
  int win_s = -1, win0 = 0;
  int32_t win = -1;        // lane i: page win0 + i of sequence win_s
  auto issue = [&](const At& at, int stage) {
    const int32_t len = s_len[at.s];
    const int32_t n_pages = (len + a.page_rows - 1) >> a.page_shift;
    const int32_t first = (at.blk * kUnit) >> a.page_shift;
    if (at.s != win_s || first < win0 || first + copies > win0 + 32) {
      win_s = at.s;
      win0 = first;
      win = first + lane < n_pages ? page_at(a, s0 + at.s, first + lane) : 0;
      if (win < 0) atomicOr(a.err, kErrPage);
    }
    const int32_t page = __shfl_sync(0xffffffffu, win, (first - win0 + lane) & 31);
    const bool mine = lane < copies && first + lane < n_pages && page >= 0;
    const uint32_t which = __ballot_sync(0xffffffffu, mine);
    if (lane == 0) {
      uint64_t there = kAll;
      if (which != (1u << copies) - 1u) {
        there = 0;
        for (int c = 0; c < copies; ++c)
          if ((which >> c) & 1u) there |= (box == 64 ? ~0ull : (1ull << box) - 1ull) << (c * box);
      }
      info[stage] = there;
      const uint32_t bytes = __popc(which) * box * (2 * C::kRow + (kE4m3 ? 2 : 0));
      if (bytes == 0) mbar_arrive(bar(stage));
      else mbar_arrive_expect_tx(bar(stage), bytes);
    }
    __syncwarp();
    if (mine) {
      const int32_t row = (at.blk * kUnit) & (a.page_rows - 1);
      const uint32_t st = ring + stage * C::kStage + lane * box * C::kRow;
      tma_load_4d(st, &tm_k, bar(stage), 0, row, at.h, page, policy);
      tma_load_4d(st + C::kHalf, &tm_v, bar(stage), 0, row, at.h, page, policy);
      if (kE4m3) {
        const int64_t from = page * a.scale_page_stride + at.h * a.scale_head_stride + row;
        const uint32_t to = smem_addr(scales) + stage * 2 * kUnit + lane * box;
        bulk_copy_g2s(to, a.k_scale + from, box, bar(stage));
        bulk_copy_g2s(to + kUnit, a.v_scale + from, box, bar(stage));
      }
    }
    __syncwarp();
  };

  Open* open = reinterpret_cast<Open*>(smem + C::kOpen);
  // Row heads of whole items whose O came out infinite or NaN though the sum of weights is finite are looked at once more,
  // without the rows that they do not see: by the join kernel, which finds them by their marks, or, where there is none, by
  // this warp.  (A call here costs the loop over the units registers: 61 tokens over e4m3 pages 119.7 us instead of 117.7.)
  StepRedo* redo = reinterpret_cast<StepRedo*>(smem + C::kRedo) + warp;
  if (lane == 0) {
    if (!kWhole) *redo = {INT64_MAX, -1};
    open[warp].units = 0;
    if (warp == 0) open[kW].units = 0;
  }
  At prod{}, cons{};
  int64_t issued = lo;
  if (lo < hi) {
    locate(lo, cons);
    prod = cons;
    for (int i = 0; i < kS && issued < hi; ++i, ++issued) {
      issue(prod, i);
      advance(prod);
    }
  }

  // ---------------------------------------------------------------- units
  uint32_t qa[4][4];                  // Q fragments of the item
  float qc[kR];                       // what turns a score of row g, g + 8 into powers of two
  float o[8][4], m[kR], M[kR], l[kR];
  int32_t seen[kR];                   // rows that row heads g, g + 8 see
  int32_t first_hidden = 0;           // rows before it are seen by every row head
  bool ok = true, started_before = false;
  int64_t done = lo;
  bool new_item = true;
  int stage = 0;
  uint32_t phase = 0;
  while (done < hi) {
    const int32_t len = s_len[cons.s];
    const int n = s_count[cons.s];
    if (new_item) {
      started_before = cons.blk > 0;
      const int mh = n * p.group;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (i >= kR) {   // (rows 8 .. 15 of the products are none)
#pragma unroll
          for (int c = 0; c < 4; ++c) qa[c][i] = qa[c][2 + i] = 0u;
          continue;
        }
        const int row = g + 8 * i, r = row / p.group;
        const bool live = row < mh;
        seen[i] = live ? len - n + r + 1 : 0;
        m[i] = M[i] = -INFINITY;
        l[i] = 0.f;
        const __nv_bfloat16* src = p.q + (s_row0[cons.s] + static_cast<int64_t>(live ? r : 0)) * p.q_row_stride +
                                   (cons.h * p.group + (live ? row % p.group : 0)) * kHeadDim;
        if (kE4m3) {
          // Elements 16 t .. 16 t + 15; the row by a power of two so that its largest is in [2^14, 2^15).
          uint32_t w[8] = {};
          if (live) {
            const uint4 x = *reinterpret_cast<const uint4*>(src + 16 * t), y = *reinterpret_cast<const uint4*>(src + 16 * t + 8);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w, w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
          }
          uint32_t top = 0;
#pragma unroll
          for (int c = 0; c < 8; ++c) top = max(top, max(w[c] & 0x7fffu, (w[c] >> 16) & 0x7fffu));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int e = max(1, min(254, static_cast<int>(top >> 7)));    // biased exponent of the largest
          // 2^(14 + 127 - e) as two factors, 2^(128 - e) and 2^13
          const float f0 = __uint_as_float(static_cast<uint32_t>(255 - e) << 23), f1 = 8192.f;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float x[4];
#pragma unroll
            for (int d = 0; d < 2; ++d) {
              x[2 * d] = __uint_as_float(w[2 * c + d] << 16) * f0 * f1;
              x[2 * d + 1] = __uint_as_float(w[2 * c + d] & 0xffff0000u) * f0 * f1;
            }
            qa[c][i] = half2_of(x[0], x[1]);
            qa[c][2 + i] = half2_of(x[2], x[3]);
          }
          qc[i] = p.q_unit * __uint_as_float(static_cast<uint32_t>(e) << 23);   // (and p.k_unit goes to the keys' factors)
        } else {
          qc[i] = p.scale * 1.4426950408889634f;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            qa[c][i] = live ? *reinterpret_cast<const uint32_t*>(src + 16 * c + 2 * t) : 0u;
            qa[c][2 + i] = live ? *reinterpret_cast<const uint32_t*>(src + 16 * c + 8 + 2 * t) : 0u;
          }
        }
      }
      first_hidden = len - n + 1;
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
      new_item = false;
    }
    if (!mbar_wait_bounded(bar(stage), phase, kWaitLimitNs)) {
      atomicOr(a.err, kErrTimeoutTma);
      ok = false;
    }
    if (!__all_sync(0xffffffffu, ok)) {
      ok = false;
      break;
    }
    const uint32_t st = ring + stage * C::kStage;
    const uint32_t vt = st + C::kHalf;
    const int32_t j0 = cons.blk * kUnit;
    const int32_t left = len - j0;                              // rows of the unit that exist
    const uint64_t exist = info[stage] & (left >= kUnit ? kAll : left <= 0 ? 0ull : (1ull << left) - 1ull);
    const bool whole = exist == kAll;
    if (!whole) {
      // What does not exist may hold anything; its weight is 0, and 0 times NaN is NaN.
      for (int row = lane; row < kUnit; row += 32)
        if (!((exist >> row) & 1ull)) {
          uint4* v = reinterpret_cast<uint4*>(ring_p + stage * C::kStage + C::kHalf + row * C::kRow);
#pragma unroll
          for (int c = 0; c < static_cast<int>(C::kRow / 16); ++c) v[c] = make_uint4(0u, 0u, 0u, 0u);
        }
      fence_proxy_async_smem();   // (the next load of this stage comes behind it)
    }
    if (kE4m3) {
      // (what a row's powers of two do: the score's factor, the weight's logarithm; of the two rows that a lane has of a
      // block of 8, side by side: rows 0 3, 1 2, 4 7, 5 6)
#pragma unroll
      for (int k = 0; k < kUnit / 32; ++k) {
        const uint8_t* sc = scales + stage * 2 * kUnit + lane + 32 * k;
        const uint32_t v = sc[kUnit];
        const int in4 = lane & 3, second = in4 >> 1;
        float* to = factors + ((lane + 32 * k) >> 3) * 16 + (((lane >> 2) & 1) * 2 + (second ? 3 - in4 : in4)) * 4 + second;
        to[0] = scale_of(sc[0]) * p.k_unit;
        to[2] = v == 255 ? NAN : static_cast<float>(static_cast<int>(v) - 127);
      }
    }
    __syncwarp();

    // S: x[i][0..1] of row head g, [2..3] of g + 8, cached rows col(i, 0), col(i, 1) of the unit.
    float x[kN][4];
#pragma unroll
    for (int i = 0; i < kN; ++i) x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
    // Column n of a block of 8 is (e4m3) cached row (n & 1 ? 3 - (t & 1) : t & 1) + 4 (t >> 1), t = n >> 1: with the
    // 64-byte swizzle no two lanes' reads of K or V then meet in a bank.
    const int f0 = kE4m3 ? (t & 1) + 4 * (t >> 1) : 2 * t, f1 = kE4m3 ? 3 - (t & 1) + 4 * (t >> 1) : 2 * t + 1;
    if (kE4m3) {
      const uint32_t in8 = ((g & 1) ? 3 - ((g >> 1) & 1) : (g >> 1) & 1) + 4 * (g >> 2);
      const uint32_t at0 = st + in8 * 64 + ((t ^ ((in8 >> 1) & 3)) << 4);
#pragma unroll
      for (int half = 0; half < kN / 4; ++half) {
        uint32_t w[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3])
                       : "r"(at0 + (4 * half + i) * 512) : "memory");
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t b0, b1;
            half2_of_e4m3(w[i][c], b0, b1);
            mma16816<true>(x[4 * half + i], qa[c], b0, b1);
          }
        }
      }
    } else {
      const uint32_t at0 = st + (lane & 7) * 128;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t b[kN][4];
#pragma unroll
        for (int i = 0; i < kN; ++i) ldsm4(at0 + i * 1024 + (((4 * c + (lane >> 3)) ^ (lane & 7)) << 4), b[i]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int i = 0; i < kN; ++i) mma16816<false>(x[i], qa[2 * c + k], b[i][2 * k], b[i][2 * k + 1]);
        }
      }
    }
    // z: e4m3: the score with log2 of V's power of two, whose maximum is M.
    const bool two = kTwo && n * p.group > 8;   // (else row heads g + 8 are none)
    float z[kN][4];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      if (r == 1 && !two) break;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        if (!kE4m3) {
          mul2(x[i][2 * r], x[i][2 * r + 1], qc[r], qc[r]);
        } else {
          float4 sc = *reinterpret_cast<const float4*>(factors + i * 16 + t * 4);
          mul2(sc.x, sc.y, qc[r], qc[r]);   // (first, as a score may be an fp32 number that it is not without K's power)
          mul2(x[i][2 * r], x[i][2 * r + 1], sc.x, sc.y);
          z[i][2 * r] = x[i][2 * r], z[i][2 * r + 1] = x[i][2 * r + 1];
          add2(z[i][2 * r], z[i][2 * r + 1], sc.z, sc.w);
        }
      }
    }
    if (!whole || j0 + kUnit > first_hidden) {
#pragma unroll
      for (int r = 0; r < kR; ++r) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int in = i * 8 + (c ? f1 : f0);
            if (!((exist >> in) & 1ull) || j0 + in >= seen[r]) x[i][2 * r + c] = z[i][2 * r + c] = -INFINITY;
          }
        }
      }
    }
    // Running maxima.
    float top[kR], wtop[kR];
    bool raised = false;
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      top[r] = m[r], wtop[r] = M[r];
      if (r == 1 && !two) break;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        top[r] = fmaxf(top[r], fmaxf(x[i][2 * r], x[i][2 * r + 1]));
        if (kE4m3) wtop[r] = fmaxf(wtop[r], fmaxf(z[i][2 * r], z[i][2 * r + 1]));
      }
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], d));
        if (kE4m3) wtop[r] = fmaxf(wtop[r], __shfl_xor_sync(0xffffffffu, wtop[r], d));
      }
      if (!kE4m3) wtop[r] = top[r];
      raised |= top[r] != m[r] || wtop[r] != M[r];
    }
    if (__any_sync(0xffffffffu, raised)) {
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        l[r] *= rescale(m[r], top[r]);
        const float f = rescale(M[r], wtop[r]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          o[j][2 * r] *= f;
          o[j][2 * r + 1] *= f;
        }
        m[r] = top[r];
        M[r] = wtop[r];
      }
    }
    // Weights and O, 16 cached rows at a time.
    float bm[kR], bM[kR], sum0[kR], sum1[kR];   // (less m, less M and 15 more)
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      bm[r] = m[r] == -INFINITY ? 0.f : -m[r];
      bM[r] = 15.f - (M[r] == -INFINITY ? 0.f : M[r]);
      sum0[r] = sum1[r] = 0.f;
    }
#pragma unroll
    for (int ks = 0; ks < kN / 2; ++ks) {
      uint32_t hi_p[4] = {0u, 0u, 0u, 0u}, lo_p[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        if (r == 1 && !two) break;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int i = 2 * ks + half;
          add2(x[i][2 * r], x[i][2 * r + 1], bm[r], bm[r]);
          const float p0 = ex2(x[i][2 * r]), p1 = ex2(x[i][2 * r + 1]);
          add2(sum0[r], sum1[r], p0, p1);
          if (kE4m3) {
            add2(z[i][2 * r], z[i][2 * r + 1], bM[r], bM[r]);
            hi_p[2 * half + r] = half2_of(ex2(z[i][2 * r]), ex2(z[i][2 * r + 1]));
          } else {
            const uint32_t h = pack_bf16x2(p0, p1);
            hi_p[2 * half + r] = h;
            lo_p[2 * half + r] = pack_bf16x2(p0 - __uint_as_float(h << 16), p1 - __uint_as_float(h & 0xffff0000u));
          }
        }
      }
      if (kE4m3) {
        // O's columns: block j, column n is element 8 n + j, so that a lane reads 8 neighbours of each of its rows.
        uint32_t v[4][2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t in8 = (k & 1) ? f1 : f0;
          asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[k][0]), "=r"(v[k][1])
                       : "r"(vt + (16 * ks + 8 * (k >> 1) + in8) * 64 + (((g >> 1) ^ ((in8 >> 1) & 3)) << 4) + (g & 1) * 8) : "memory");
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {   // blocks 2 j, 2 j + 1: two bytes of each row
          const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;
          uint32_t b0[2], b1[2];
          half2_of_e4m3(__byte_perm(v[0][j >> 1], v[1][j >> 1], sel), b0[0], b0[1]);
          half2_of_e4m3(__byte_perm(v[2][j >> 1], v[3][j >> 1], sel), b1[0], b1[1]);
          mma16816<true>(o[2 * j], hi_p, b0[0], b1[0]);
          mma16816<true>(o[2 * j + 1], hi_p, b0[1], b1[1]);
        }
      } else {
        uint32_t b[4][4];
        const uint32_t at0 = vt + (16 * ks + (lane & 15)) * 128;
#pragma unroll
        for (int j = 0; j < 4; ++j) ldsm4_trans(at0 + (((2 * j + (lane >> 4)) ^ (lane & 7)) << 4), b[j]);
#pragma unroll
        for (int j = 0; j < 8; ++j) mma16816<false>(o[j], hi_p, b[j >> 1][2 * (j & 1)], b[j >> 1][2 * (j & 1) + 1]);
#pragma unroll
        for (int j = 0; j < 8; ++j) mma16816<false>(o[j], lo_p, b[j >> 1][2 * (j & 1)], b[j >> 1][2 * (j & 1) + 1]);
      }
    }
#pragma unroll
    for (int r = 0; r < kR; ++r) l[r] += sum0[r] + sum1[r];
    __syncwarp();
    ++done;
    if (issued < hi) {
      issue(prod, stage);
      advance(prod);
      ++issued;
    }
    if (++stage == kS) stage = 0, phase ^= 1u;
    const bool item_done = cons.blk == cons.units - 1;
    if (item_done || done == hi) {
      // ------------------------------------------------------------ the end of an item, or of this warp's part of it
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      }
      const int mh = n * p.group;
      if (item_done && !started_before) {
        uint32_t which = 0;
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          const int row = g + 8 * r;
          bool wild = false;
          if (row < mh) {
            const OutFactor f = out_factor<kE4m3>(m[r], M[r], l[r]);
            const int64_t at = (s_row0[cons.s] + static_cast<int64_t>(row / p.group)) * p.heads + cons.h * p.group + row % p.group;
            float y[16];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              y[j] = l[r] == 0.f ? 0.f : f(o[j][2 * r]);
              y[8 + j] = l[r] == 0.f ? 0.f : f(o[j][2 * r + 1]);
              wild |= !(fabsf(y[j]) <= 3.4e38f) || !(fabsf(y[8 + j]) <= 3.4e38f);
            }
            wild &= l[r] == l[r];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if (kE4m3) store_pair(p, at, 16 * t + 2 * j, y[2 * j], y[2 * j + 1]);
              else store_pair(p, at, 8 * j + 2 * t, y[j], y[8 + j]);
            }
            if (p.lse != nullptr && t == 0) p.lse[at] = log_sum(m[r], l[r]);
            if (!kWhole && wild) {   // (the lanes' elements that they have just stored)
              uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + at * kHeadDim);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                uint32_t* two = dst + (kE4m3 ? 8 * t + j : 4 * j + t);
                *two = marked(*two);
              }
              const int64_t it = static_cast<int64_t>(s0 + cons.s) * a.heads + cons.h;
              *redo = {min(redo->first, it), it};
            }
          }
          if (kWhole) {
            const uint32_t b = __ballot_sync(0xffffffffu, wild);
            for (int i = 0; b != 0 && i < 8; ++i)
              if ((b >> (4 * i)) & 15u) which |= 1u << (i + 8 * r);
          }
        }
        if (kWhole && which != 0) redo_rows<kE4m3>(a, p, which, s0 + cons.s, cons.h, s_row0[cons.s], 0, len - n + 1);
      } else {
        // (what began before the CTA is warp 0's to tell of: open[kW] where it ends in warp 0, as another may begin there)
        if (lane == 0 && (item_done ? warp == 0 : warp == 0 || !started_before))
          open[item_done ? kW : warp] = {done - 1 - cons.blk, cons.units, cons.s, cons.h};
        float* slot = slot_of(warp, started_before);
        if (!started_before) __syncwarp();   // (the ring's last reads are done)
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          const int row = g + 8 * r;
          float* to = slot + row * kSlotStride;
          if (kE4m3) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<float4*>(to + 16 * t + 4 * j) =
                  j < 2 ? make_float4(o[4 * j][2 * r], o[4 * j + 1][2 * r], o[4 * j + 2][2 * r], o[4 * j + 3][2 * r])
                        : make_float4(o[4 * j - 8][2 * r + 1], o[4 * j - 7][2 * r + 1], o[4 * j - 6][2 * r + 1], o[4 * j - 5][2 * r + 1]);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) *reinterpret_cast<float2*>(to + 8 * j + 2 * t) = make_float2(o[j][2 * r], o[j][2 * r + 1]);
          }
          if (t == 0) {
            slot[kStats + row] = m[r];
            slot[kStats + kM + row] = M[r];
            slot[kStats + 2 * kM + row] = l[r];
          }
        }
      }
      new_item = true;
    }
    if (done < hi) advance(cons);
  }
  if (!ok) {   // wait (a little) for the loads in flight before the CTA can leave
    for (int64_t u = done; u < issued; ++u) {
      mbar_wait_bounded(bar(stage), phase, 1000000ull);
      if (++stage == kS) stage = 0, phase ^= 1u;
    }
  }
  ok = __syncthreads_and(ok);

  // ---------------------------------------------------------------- items of several parts
  // All warps share the row heads of all of them, two at a time: half a warp each, first its lanes the parts, then four
  // elements of O; two such pairs side by side where a warp has more than one, as each is a chain of shuffles.
  // (By the warps that had some of the item, one by one: 24 x 4 tokens 32.4 us instead of 30.8, of which CTAs with many
  // short sequences took 6 here; 131,072 rows 20.4 instead of 18.4.)
  float* ws_part = ws + static_cast<int64_t>(blockIdx.x) * kStepWsFloats;
  StepJoin join{};   // what the join kernel finds of this CTA: the item that begins here and goes on, if there is one
  if (ok) {
    const int half = lane >> 4, sub = lane & 15;
    const int64_t cta_lo = edge_of(0), cta_hi = edge_of(kW);
    const Open my_open = open[min(lane, kW)];   // lane k: the k-th one and its pairs
    const int my_pairs = lane <= kW && my_open.units != 0 ? (s_count[my_open.s] * p.group + 1) >> 1 : 0;
    int upto = my_pairs;
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += x;
    }
    const int each_warp = (__shfl_sync(0xffffffffu, upto, kW) + kW - 1) / kW, from = each_warp * warp, to = from + each_warp;
    if (tid <= kW && my_open.units != 0) {
      const int64_t ie = my_open.begin + my_open.units;
      if (my_open.begin >= cta_lo && ie > cta_hi) {
        const int64_t x = ie - 1;   // its last unit, and the warp that has it
        const Shares sh = shares();
        const int64_t wide = sh.more * (sh.each + 1);
        const int64_t w = x < wide ? quotient(x, sh.each + 1) : sh.more + quotient(x - wide, sh.each);
        join = {static_cast<int32_t>(w / kW) - static_cast<int32_t>(blockIdx.x) + 1, s0 + my_open.s, my_open.h, s_count[my_open.s],
                s_len[my_open.s], s_row0[my_open.s], {}};
      }
    }
    uint32_t items = __ballot_sync(0xffffffffu, my_pairs > 0 && upto > from && upto - my_pairs < to);
#pragma unroll 1
    for (; items != 0; items &= items - 1) {
      const int k = __ffs(items) - 1;
      const Open it = open[k];
      const int before = __shfl_sync(0xffffffffu, upto - my_pairs, k);
      const int64_t ib = it.begin, ie = ib + it.units;
      const int w0 = k == kW ? 0 : k;   // the first and the last warp of the CTA with some of it
      const int w1 = max(w0, __popc(__ballot_sync(0xffffffffu, lane > 0 && lane < kW && edge < min(ie, cta_hi))));
      const int parts = w1 - w0 + 1;
      const bool complete = ib >= cta_lo && ie <= cta_hi;
      const bool w0_head = edge_of(w0) > ib;      // (the later ones have it in their head slots)
      const int n = s_count[it.s], mh = n * p.group;
      float* out_slot = ws_part + (ib < cta_lo ? 0 : kSlotFloats);
      const float* mine = slot_of(w0 + min(sub, parts - 1), min(sub, parts - 1) > 0 || w0_head);
      const int end = min(to - before, (mh + 1) >> 1);
      uint32_t which = 0;
      auto join_pairs = [&](auto at_once, int i) {   // from pair i on
        constexpr int kAtOnce = decltype(at_once)::value;
        int row[kAtOnce];
        float jm[kAtOnce], jM[kAtOnce], jl[kAtOnce], f[kAtOnce];
        float4 jo[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          row[u] = min(2 * (i + u) + half, mh - 1);
          jm[u] = sub < parts ? mine[kStats + row[u]] : -INFINITY;
          jM[u] = sub < parts ? mine[kStats + kM + row[u]] : -INFINITY;
          jl[u] = sub < parts ? mine[kStats + 2 * kM + row[u]] : 0.f;
          jo[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float pm[kAtOnce], pM[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) pm[u] = jm[u], pM[u] = jM[u];
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) {
#pragma unroll
          for (int u = 0; u < kAtOnce; ++u) {
            jm[u] = fmaxf(jm[u], __shfl_xor_sync(0xffffffffu, jm[u], d));
            if (kE4m3) jM[u] = fmaxf(jM[u], __shfl_xor_sync(0xffffffffu, jM[u], d));
          }
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          if (!kE4m3) jM[u] = jm[u];   // (the same, over bf16 pages)
          f[u] = rescale(pM[u], jM[u]);
          jl[u] *= rescale(pm[u], jm[u]);
        }
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) {
#pragma unroll
          for (int u = 0; u < kAtOnce; ++u) jl[u] += __shfl_xor_sync(0xffffffffu, jl[u], d);
        }
#pragma unroll 2
        for (int w = 0; w < parts; ++w) {
          const float* slot = slot_of(w0 + w, w > 0 || w0_head) + 4 * sub;
#pragma unroll
          for (int u = 0; u < kAtOnce; ++u) {
            const float4 y = *reinterpret_cast<const float4*>(slot + row[u] * kSlotStride);
            const float fw = __shfl_sync(0xffffffffu, f[u], w, 16);
            jo[u].x = fmaf(fw, y.x, jo[u].x), jo[u].y = fmaf(fw, y.y, jo[u].y);
            jo[u].z = fmaf(fw, y.z, jo[u].z), jo[u].w = fmaf(fw, y.w, jo[u].w);
          }
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          const bool in = i + u < end && 2 * (i + u) + half < mh;
          bool wild = false;
          if (complete) {
            const int r = row[u] / p.group;
            const int64_t o_at = (s_row0[it.s] + static_cast<int64_t>(r)) * p.heads + it.h * p.group + row[u] - r * p.group;
            const OutFactor of = out_factor<kE4m3>(jm[u], jM[u], jl[u]);
            const float y[4] = {of(jo[u].x), of(jo[u].y), of(jo[u].z), of(jo[u].w)};
#pragma unroll
            for (int c = 0; c < 4; ++c) wild |= !(fabsf(y[c]) <= 3.4e38f);
            wild &= in && jl[u] == jl[u] && jl[u] != 0.f;
            if (in) {
              *reinterpret_cast<uint2*>(p.out + o_at * kHeadDim + 4 * sub) =
                  jl[u] == 0.f ? make_uint2(0u, 0u) : make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
              if (p.lse != nullptr && sub == 0) p.lse[o_at] = log_sum(jm[u], jl[u]);
              if (!kWhole && wild) {
                uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + o_at * kHeadDim + 4 * sub);
                dst[0] = marked(dst[0]), dst[1] = marked(dst[1]);
                const int64_t ri = static_cast<int64_t>(s0 + it.s) * a.heads + it.h;
                *redo = {min(redo->first, ri), max(redo->last, ri)};
              }
            }
          } else if (in) {
            *reinterpret_cast<float4*>(out_slot + row[u] * kSlotStride + 4 * sub) = jo[u];
            if (sub == 0) {
              out_slot[kM * kSlotStride + row[u]] = jm[u];
              out_slot[kM * kSlotStride + kM + row[u]] = jM[u];
              out_slot[kM * kSlotStride + 2 * kM + row[u]] = jl[u];
            }
          }
          const uint32_t bits = kWhole ? __ballot_sync(0xffffffffu, wild) : 0u;
          which |= ((bits & 0xffffu) ? 1u : 0u) << (2 * (i + u)) | ((bits >> 16) ? 2u : 0u) << (2 * (i + u));
        }
      };
      int i = max(from - before, 0);
      if (end - i == 1) {
        join_pairs(std::integral_constant<int, 1>(), i);
      } else {
#pragma unroll 1
        for (; i < end; i += 2) join_pairs(std::integral_constant<int, 2>(), i);
      }
      if (kWhole && which != 0) redo_rows<kE4m3>(a, p, which, s0 + it.s, it.h, s_row0[it.s], 0, s_len[it.s] - n + 1);
    }
  }
  // (warp 0's lanes have the records: the one that has the item writes, or lane 0)
  if (warp == 0 && !kWhole) {
    const uint32_t goes_on = __ballot_sync(0xffffffffu, join.parts > 0);
    if (goes_on != 0 ? join.parts > 0 : lane == 0) *reinterpret_cast<StepJoin*>(ws_part + 2 * kSlotFloats) = join;
  }
  if (!kWhole) {
    StepRedo* to = reinterpret_cast<StepRedo*>(ws_part + 2 * kSlotFloats + sizeof(StepJoin) / 4);
    __syncwarp();
    if (lane == 0) {
      to[warp] = ok ? *redo : StepRedo{INT64_MAX, -1};   // (not ok: a wait ran out, and there are items without any result)
      if (warp + kW < kStepMostWarps) to[warp + kW] = {INT64_MAX, -1};
    }
  }
  if (behind && blockIdx.x == 0) griddep_wait();
}

template <bool kE4m3, int kJoinSlices>
__global__ void __launch_bounds__(kJoinRows * kJoinSlices * 16, 1024 / (kJoinRows * kJoinSlices * 16))
paged_join_kernel(const __grid_constant__ KvArgs a, const __grid_constant__ PagedAttn p, const float* ws) {
  griddep_launch_dependents();
  griddep_wait();
  if (blockIdx.y == gridDim.y - 1) redo_step_items<kE4m3>(a, p, ws);
  else join_step_parts<kE4m3, kJoinSlices>(a, p, ws, static_cast<int>(gridDim.x), static_cast<int>(blockIdx.y));
}

template <bool kE4m3, bool kTwo, bool kWhole>
cudaError_t launch(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const KvArgs& a, const PagedAttn& p, int s0, int ns, int grid,
                   bool behind, float* ws, cudaStream_t stream) {
  using C = Cfg<kE4m3, kTwo>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = set_smem_limit_once(paged_step_kernel<kE4m3, kTwo, kWhole>, C::kRequest, done);
  if (e != cudaSuccess) return e;
  return launch_behind(paged_step_kernel<kE4m3, kTwo, kWhole>, dim3(grid), C::kWarps * 32, C::kRequest, stream, tm_k, tm_v, a, p, s0, ns,
                       behind, ws);
}

}  // namespace

static_assert(kStepWsFloats * 4 >= 2 * kSlotFloats * 4 + sizeof(StepJoin) + kStepMostWarps * sizeof(StepRedo) &&
                  Cfg<true, false>::kWarps <= kStepMostWarps && 2 * Cfg<false, false>::kWarps >= kStepMostWarps,
              "workspace of a CTA");

int paged_step_unit(bool e4m3) { return e4m3 ? Cfg<true, false>::kUnit : Cfg<false, false>::kUnit; }

int paged_step_grid(int64_t most_units, int num_sms) {
  constexpr int64_t w = Cfg<false, false>::kWarps;   // (the least that a CTA has)
  return static_cast<int>(std::min<int64_t>(std::min(num_sms, kStepMaxGrid), (most_units + w - 1) / w));
}

// At most 8 row heads where the call says so (max_rows): the products' second half, and its exponentials, are left out.
// (61 tokens over e4m3 pages, 16 heads: 117.5 us then, by the kernel for 16 row heads 133; 128 tokens over bf16 pages, four heads
// a key head: 221 and 223.)
cudaError_t launch_paged_step(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const KvArgs& a, const PagedAttn& p, int s0, int ns,
                              int grid, bool e4m3, bool whole_items, bool behind, float* ws, cudaStream_t stream) {
  const bool two = a.max_rows * p.group > 8;
  auto* run = whole_items ? (e4m3 ? (two ? launch<true, true, true> : launch<true, false, true>)
                                  : (two ? launch<false, true, true> : launch<false, false, true>))
                          : (e4m3 ? (two ? launch<true, true, false> : launch<true, false, false>)
                                  : (two ? launch<false, true, false> : launch<false, false, false>));
  return run(tm_k, tm_v, a, p, s0, ns, grid, behind, ws, stream);
}

cudaError_t launch_paged_join(const KvArgs& a, const PagedAttn& p, int grid, bool e4m3, const float* ws, cudaStream_t stream) {
  const int64_t most = std::min<int64_t>(kM, a.max_rows * p.group);   // row heads
  const dim3 ctas(grid, static_cast<unsigned>((most + kJoinRows - 1) / kJoinRows + 1));
  // Items over four CTAs and more: twice the threads, as a thread then has several parts; but where the call has long
  // chunks too (and its step kernel perhaps nothing), the bigger launch costs more.  (131,072 rows, up to 90 parts: 18.4 us,
  // by twice the threads 17.7; 24 x 4 tokens, up to 6 parts: 30.5 and 31.9; a chunk of 512: 34.9 and 35.8.)
  const bool many = static_cast<int64_t>(a.seqs) * a.heads * 4 <= grid && a.max_rows * p.group <= kM;
  auto* kernel = many ? (e4m3 ? paged_join_kernel<true, 8> : paged_join_kernel<false, 8>)
                      : (e4m3 ? paged_join_kernel<true, 4> : paged_join_kernel<false, 4>);
  return launch_behind(kernel, ctas, many ? 512 : 256, 0, stream, a, p, ws);
}

}  // namespace spanla
