// Softmax attention of a few new rows of each sequence (the next token, some
// drafted ones) over the paged cache: row heads r * group + g of one sequence and
// key head, at most 16 of them, against all of the sequence's cached rows.
//
// Bound by memory: every cached row and head is read once, 256 bytes of bf16 or
// 130 of e4m3, for 256 multiply-adds a row head.  So the cached rows are cut into
// units of 32, numbered through all sequences, key heads and rows, and every warp
// of the card gets the same number of consecutive units, whatever the lengths: a
// warp finds its first unit by the sequences' running sums, and streams its units
// through a ring of its own, filled by TMA (its lane 0), without waiting for other
// warps.  The lengths are device memory: every CTA sums them up for itself.
//
// A unit: S = Q K^T (m16n8k16, the row heads as M), running maximum m and sum l of
// each row head in registers, O += P V.  bf16 pages: P enters as two bf16 parts
// (hi + lo, 2^-17 of it), the M = 16 products being free beside the loads.  e4m3
// pages: q, K and V enter as fp16 (K and V exactly, q scaled by a power of two
// for its row, then all but its least elements), the rows' powers of two go onto
// the scores and the weights in fp32; the weights w_j = p_j 2^(e_j) have a running
// maximum 2^M of their own and enter 2^15 times over it, so that fp16 holds them to
// 2^-11 of each, or 2^-40 of the largest.
//
// A warp's first and last items may go on in other warps.  Those parts (m, M, l,
// O) meet in shared memory for the warps of a CTA and then, for the items that go
// over several CTAs, in the join kernel, which starts behind this one.
#include <algorithm>

#include "paged.cuh"

namespace spanla {
namespace {

constexpr int kUnit = kStepUnit;          // cached rows
constexpr int kM = kStepHeads;            // row heads
constexpr int kSlotStride = 72;           // floats from row head to row head of a part (72: no bank conflicts)

// A part of an item: [16][72] floats of O, then m, M, l of 16 row heads.
constexpr int kSlotFloats = kM * kSlotStride + 3 * kM;

template <bool kE4m3>
struct Cfg {
  static constexpr int kWarps = kE4m3 ? 12 : 8;
  static constexpr int kStages = kE4m3 ? 3 : 2;
  static constexpr uint32_t kRow = kE4m3 ? 64 : 128;           // bytes
  static constexpr uint32_t kHalf = kUnit * kRow;              // K or V of a unit
  static constexpr uint32_t kStage = 2 * kHalf;
  static constexpr uint32_t kRing = kStages * kStage;          // of a warp
  static constexpr uint32_t kScales = kWarps * kRing;          // 2 x 32 bytes a stage
  static constexpr uint32_t kFactors = kScales + (kE4m3 ? kWarps * kStages * 2 * kUnit : 0);   // of a unit's rows, 8 bytes
  static constexpr uint32_t kHead = kFactors + (kE4m3 ? kWarps * kUnit * 8 : 0);
  static constexpr uint32_t kSum = kHead + kWarps * kSlotFloats * 4;
  static constexpr uint32_t kLen = kSum + (kStepSeqs + 1) * 8;
  static constexpr uint32_t kRow0 = kLen + kStepSeqs * 4;
  static constexpr uint32_t kCount = kRow0 + kStepSeqs * 4;
  static constexpr uint32_t kInfo = kCount + kStepSeqs;
  static constexpr uint32_t kScan = kInfo + kWarps * kStages * 4;
  static constexpr uint32_t kBar = (kScan + kWarps * 8 + 7) / 8 * 8;
  static constexpr uint32_t kBytes = kBar + kWarps * kStages * 8;
  static constexpr uint32_t kRequest = kBytes + 1024;
  static_assert(kRequest <= 227 * 1024 && kRing >= kSlotFloats * 4, "shared memory budget");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

template <bool kHalfFloat>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (kHalfFloat)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
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

__device__ __forceinline__ int32_t units_of(int32_t len) { return max(1, (len + kUnit - 1) / kUnit); }

// Output of row head m of an item, elements d0 .. d0 + 1.
__device__ __forceinline__ void store_pair(const PagedAttn& p, int64_t at, int d, float x, float y) {
  *reinterpret_cast<uint32_t*>(p.out + at * kHeadDim + d) = pack_bf16x2(x, y);
}

// The weights of a row head are relative to 2^m, its O to 2^(M - 15) (bf16 pages: 2^m): o = O 2^(M - 15 - m) / l.
template <bool kE4m3>
__device__ __forceinline__ float out_factor(float m, float M, float l) {
  return l == 0.f ? 0.f : (kE4m3 ? ex2(M - m - 15.f) : 1.f) / l;
}
__device__ __forceinline__ float log_sum(float m, float l) { return l == 0.f ? -INFINITY : fmaf(m, 0.6931471805599453f, logf(l)); }

// 2^(from - to), 0 where nothing is relative to `from`.
__device__ __forceinline__ float rescale(float from, float to) { return from == to ? 1.f : from == -INFINITY ? 0.f : ex2(from - to); }

// Row heads of an item whose O came out infinite or NaN though the sum of weights is finite: once more from the
// cache, without the rows that they do not see (and without O's parts, whose infinities may cancel).
template <bool kE4m3>
__device__ __forceinline__ void redo_rows(const KvArgs& a, const PagedAttn& p, uint32_t which, int s, int64_t row0, int n, int32_t len,
                                          int h) {
  while (which != 0) {
    const int m = __ffs(which) - 1;
    which &= which - 1;
    const int r = m / p.group;
    attend_row<kE4m3>(a, p, s, row0 + r, h * p.group + m % p.group, max(0, len - n + r + 1));
  }
}

template <bool kE4m3>
__global__ void __launch_bounds__(Cfg<kE4m3>::kWarps * 32, 1)
paged_step_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ KvArgs a,
                  const __grid_constant__ PagedAttn p, int s0, int ns, float* __restrict__ ws) {
  using C = Cfg<kE4m3>;
  constexpr int kW = C::kWarps, kS = C::kStages;
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

  if (lane == 0) {
    for (int i = 0; i < kS; ++i) mbar_init(bar(i), 1);
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  griddep_launch_dependents();   // (the next kernels of the call wait for this grid's end, or need not)
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
    int64_t* scan = reinterpret_cast<int64_t*>(smem + (C::kScan + 7) / 8 * 8);
    if (lane == 31) scan[warp] = upto;
    __syncthreads();
    int64_t before = upto - mine;
    for (int w = 0; w < warp; ++w) before += scan[w];
    for (int s = b; s < e; ++s) sum[s] += before;
    if (tid == kW * 32 - 1) sum[ns] = before + mine;
    __syncthreads();
  }
  const int64_t U = sum[ns];
  // ---------------------------------------------------------------- this warp's units
  const int64_t nw = min(static_cast<int64_t>(gridDim.x) * kW, U);     // warps at work: each has a unit at least
  auto begin_of = [&](int64_t w) { return w >= nw ? U : U * w / nw; };
  const int64_t edge = begin_of(static_cast<int64_t>(blockIdx.x) * kW + min(lane, kW));   // lane w: of the CTA's warp w
  auto edge_of = [&](int w) { return __shfl_sync(0xffffffffu, edge, w); };
  const int64_t lo = edge_of(warp), hi = edge_of(warp + 1), cta_lo = edge_of(0), cta_hi = edge_of(kW);
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
    at.h = static_cast<int>(in / at.units);
    at.blk = static_cast<int32_t>(in - static_cast<int64_t>(at.h) * at.units);
  };
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
  uint32_t* info = reinterpret_cast<uint32_t*>(smem + C::kInfo) + warp * kS;
  float2* factors = reinterpret_cast<float2*>(smem + C::kFactors) + warp * kUnit;
  uint8_t* scales = smem + C::kScales + warp * kS * 2 * kUnit;
  float* head_slot = reinterpret_cast<float*>(smem + C::kHead) + warp * kSlotFloats;
  float* tail_slot = reinterpret_cast<float*>(ring_p);   // once the ring is done
  auto slot_of = [&](int w, bool head) {
    return head ? reinterpret_cast<float*>(smem + C::kHead) + w * kSlotFloats : reinterpret_cast<float*>(smem + w * C::kRing);
  };

  // ---------------------------------------------------------------- loads
  const uint64_t policy = l2_evict_first_policy();
  int win_s = -1, win0 = 0;
  int32_t win = -1;        // lane i: page win0 + i of sequence win_s
  auto issue = [&](const At& at, int stage) {
    const int32_t len = s_len[at.s];
    const int32_t n_pages = (len + a.page_rows - 1) >> a.page_shift;
    const int32_t first = (at.blk * kUnit) >> a.page_shift;       // (16-row pages: first and first + 1, first even)
    if (at.s != win_s || first < win0 || first >= win0 + 32) {
      win_s = at.s;
      win0 = first;
      win = first + lane < n_pages ? a.table[(s0 + at.s) * a.table_stride + first + lane] : 0;
      if (win < 0 || win >= a.pages) {
        atomicOr(a.err, kErrPage);
        win = -1;
      }
    }
    const bool two = a.page_rows < kUnit;
    const int32_t p0 = __shfl_sync(0xffffffffu, win, first - win0), p1 = __shfl_sync(0xffffffffu, win, (first - win0 + 1) & 31);
    const bool has0 = first < n_pages && p0 >= 0, has1 = two ? first + 1 < n_pages && p1 >= 0 : has0;
    if (lane == 0) {
      info[stage] = (has0 ? 0xffffu : 0u) | (has1 ? 0xffff0000u : 0u);
      const uint32_t st = ring + stage * C::kStage;
      const int32_t rows = two ? 16 : kUnit;
      const int copies = (has0 ? 1 : 0) + (two && has1 ? 1 : 0);
      const uint32_t bytes = copies * rows * (2 * C::kRow + (kE4m3 ? 2 : 0));
      if (bytes == 0) {
        mbar_arrive(bar(stage));
      } else {
        mbar_arrive_expect_tx(bar(stage), bytes);
        for (int c = 0; c < (two ? 2 : 1); ++c) {
          if (!(c == 0 ? has0 : has1)) continue;
          const int32_t page = c == 0 ? p0 : p1, row = two ? 0 : (at.blk * kUnit) & (a.page_rows - 1);
          tma_load_4d(st + c * 16 * C::kRow, &tm_k, bar(stage), 0, row, at.h, page, policy);
          tma_load_4d(st + C::kHalf + c * 16 * C::kRow, &tm_v, bar(stage), 0, row, at.h, page, policy);
          if (kE4m3) {
            const int64_t from = page * a.scale_page_stride + at.h * a.scale_head_stride + row;
            const uint32_t to = smem_addr(scales) + stage * 2 * kUnit + c * 16;
            bulk_copy_g2s(to, a.k_scale + from, rows, bar(stage));
            bulk_copy_g2s(to + kUnit, a.v_scale + from, rows, bar(stage));
          }
        }
      }
    }
    __syncwarp();
  };

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
  const float c2 = p.scale * 1.4426950408889634f;
  uint32_t qa[4][4];                  // Q fragments of the item
  float qc[2] = {c2, c2};             // what turns a score of row g, g + 8 into powers of two
  float o[8][4], m[2], M[2], l[2];
  int32_t seen[2];                    // rows that row heads g, g + 8 see
  int32_t first_hidden = 0;           // rows before it are seen by every row head
  bool ok = true, started_before = false;
  int64_t done = lo;
  bool new_item = true;
  while (done < hi) {
    const int stage = static_cast<int>((done - lo) % kS);
    const int32_t len = s_len[cons.s];
    const int n = s_count[cons.s];
    if (new_item) {
      started_before = cons.blk > 0;
      const int mh = n * p.group;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
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
          qc[i] = c2 * (1.f / 16384.f) * __uint_as_float(static_cast<uint32_t>(e) << 23);
        } else {
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
    if (!mbar_wait_bounded(bar(stage), static_cast<uint32_t>((done - lo) / kS) & 1u, kWaitLimitNs)) {
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
    const uint32_t pages_ok = info[stage];
    const int32_t left = len - j0;                              // rows of the unit that exist
    const bool whole = left >= kUnit && pages_ok == 0xffffffffu;
    uint32_t exist = pages_ok & (left >= kUnit ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u);
    if (!whole && !((exist >> lane) & 1u)) {
      // What does not exist may hold anything; its weight is 0, and 0 times NaN is NaN.
      uint4* row = reinterpret_cast<uint4*>(ring_p + stage * C::kStage + C::kHalf + lane * C::kRow);
#pragma unroll
      for (int c = 0; c < static_cast<int>(C::kRow / 16); ++c) row[c] = make_uint4(0u, 0u, 0u, 0u);
      fence_proxy_async_smem();   // (the next load of this stage comes behind it)
    }
    __syncwarp();

    // S: x[i][0..1] of row head g, [2..3] of g + 8, cached rows col(i, 0), col(i, 1) of the unit.
    float x[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
      if (kE4m3) {
        // Column n of a block of 8 is cached row (n & 1 ? 3 - (t & 1) : t & 1) + 4 (t >> 1), t = n >> 1: with the
        // 64-byte swizzle no two lanes' reads of K or V then meet in a bank.
        const uint32_t row = i * 8 + ((g & 1) ? 3 - ((g >> 1) & 1) : (g >> 1) & 1) + 4 * (g >> 2);
        uint32_t w[4];
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(st + row * 64 + ((t ^ ((row >> 1) & 3)) << 4)) : "memory");
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t b0, b1;
          half2_of_e4m3(w[c], b0, b1);
          mma16816<true>(x[i], qa[c], b0, b1);
        }
      } else {
        const uint32_t row = i * 8 + (lane & 7);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t b[4];
          ldsm4(st + row * 128 + (((4 * c + (lane >> 3)) ^ (lane & 7)) << 4), b);
          mma16816<false>(x[i], qa[2 * c], b[0], b[1]);
          mma16816<false>(x[i], qa[2 * c + 1], b[2], b[3]);
        }
      }
    }
    if (kE4m3) {
      // (what a row's powers of two do: the score's factor, the weight's logarithm)
      const uint8_t* sc = scales + stage * 2 * kUnit + lane;
      const uint32_t v = sc[kUnit];
      factors[lane] = make_float2(scale_of(sc[0]), v == 255 ? NAN : static_cast<float>(static_cast<int>(v) - 127));
      __syncwarp();
    }
    const int f0 = kE4m3 ? (t & 1) + 4 * (t >> 1) : 2 * t, f1 = kE4m3 ? 3 - (t & 1) + 4 * (t >> 1) : 2 * t + 1;
    // z: e4m3: the score with log2 of V's power of two, whose maximum is M + 15.
    const bool two = n * p.group > 8;   // (else row heads g + 8 are none)
    float z[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c >= 2 && !two) continue;
        if (kE4m3) {
          const float2 sc = factors[i * 8 + ((c & 1) ? f1 : f0)];
          x[i][c] = x[i][c] * qc[c >> 1] * sc.x;
          z[i][c] = x[i][c] + sc.y;
        } else {
          x[i][c] *= c2;
        }
      }
    }
    if (!whole || j0 + kUnit > first_hidden) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int in = i * 8 + ((c & 1) ? f1 : f0);
          if (!((exist >> in) & 1u) || j0 + in >= seen[c >> 1]) x[i][c] = z[i][c] = -INFINITY;
        }
      }
    }
    // Running maxima.
    float top[2] = {m[0], m[1]}, wtop[2] = {M[0], M[1]};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (i == 1 && !two) continue;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        top[i] = fmaxf(top[i], fmaxf(x[k][2 * i], x[k][2 * i + 1]));
        if (kE4m3) wtop[i] = fmaxf(wtop[i], fmaxf(z[k][2 * i], z[k][2 * i + 1]));
      }
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], d));
        if (kE4m3) wtop[i] = fmaxf(wtop[i], __shfl_xor_sync(0xffffffffu, wtop[i], d));
      }
      if (!kE4m3) wtop[i] = top[i];
    }
    if (__any_sync(0xffffffffu, top[0] != m[0] || top[1] != m[1] || wtop[0] != M[0] || wtop[1] != M[1])) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[i] *= rescale(m[i], top[i]);
        const float f = rescale(M[i], wtop[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          o[j][2 * i] *= f;
          o[j][2 * i + 1] *= f;
        }
        m[i] = top[i];
        M[i] = wtop[i];
      }
    }
    // Weights and O.
    const float b0 = m[0] == -INFINITY ? 0.f : m[0], b1 = m[1] == -INFINITY ? 0.f : m[1];
    const float B0 = (M[0] == -INFINITY ? 0.f : M[0]) - 15.f, B1 = (M[1] == -INFINITY ? 0.f : M[1]) - 15.f;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      uint32_t hi_p[4], lo_p[4];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int i = 2 * ks + half;
        float w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          w[c] = 0.f;
          if (c >= 2 && !two) continue;
          const float pw = ex2(x[i][c] - (c < 2 ? b0 : b1));
          l[c >> 1] += pw;
          w[c] = kE4m3 ? ex2(z[i][c] - (c < 2 ? B0 : B1)) : pw;
        }
        if (kE4m3) {
          hi_p[2 * half] = half2_of(w[0], w[1]);
          hi_p[2 * half + 1] = half2_of(w[2], w[3]);
        } else {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            hi_p[2 * half + r] = pack_bf16x2(w[2 * r], w[2 * r + 1]);
            lo_p[2 * half + r] = pack_bf16x2(w[2 * r] - __uint_as_float(hi_p[2 * half + r] << 16),
                                             w[2 * r + 1] - __uint_as_float(hi_p[2 * half + r] & 0xffff0000u));
          }
        }
      }
      if (kE4m3) {
        // O's columns: block j, column n is element 8 n + j, so that a lane reads 8 neighbours of each of its rows.
        uint32_t v[4][2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t row = 16 * ks + 8 * (k >> 1) + ((k & 1) ? f1 : f0);
          asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[k][0]), "=r"(v[k][1])
                       : "r"(vt + row * 64 + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + (g & 1) * 8) : "memory");
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {   // blocks 2 j, 2 j + 1: two bytes of each row
          const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;
          const uint32_t y0 = __byte_perm(v[0][j >> 1], v[1][j >> 1], sel), y1 = __byte_perm(v[2][j >> 1], v[3][j >> 1], sel);
          uint32_t b0[2], b1[2];
          half2_of_e4m3(y0, b0[0], b0[1]);
          half2_of_e4m3(y1, b1[0], b1[1]);
          mma16816<true>(o[2 * j], hi_p, b0[0], b1[0]);
          mma16816<true>(o[2 * j + 1], hi_p, b0[1], b1[1]);
        }
      } else {
        const uint32_t row = 16 * ks + (lane & 15);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t b[4];
          ldsm4_trans(vt + row * 128 + (((2 * j + (lane >> 4)) ^ (lane & 7)) << 4), b);
          mma16816<false>(o[2 * j], hi_p, b[0], b[1]);
          mma16816<false>(o[2 * j], lo_p, b[0], b[1]);
          mma16816<false>(o[2 * j + 1], hi_p, b[2], b[3]);
          mma16816<false>(o[2 * j + 1], lo_p, b[2], b[3]);
        }
      }
    }
    __syncwarp();
    ++done;
    if (issued < hi) {
      issue(prod, stage);
      advance(prod);
      ++issued;
    }
    const bool item_done = cons.blk == cons.units - 1;
    if (item_done || done == hi) {
      // ------------------------------------------------------------ the end of an item, or of this warp's part of it
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      }
      const int mh = n * p.group;
      if (item_done && !started_before) {
        bool wild[2] = {false, false};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = g + 8 * i;
          if (row >= mh) continue;
          const float f = out_factor<kE4m3>(m[i], M[i], l[i]);
          const int64_t at = (s_row0[cons.s] + static_cast<int64_t>(row / p.group)) * p.heads + cons.h * p.group + row % p.group;
          float y[16];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            y[j] = l[i] == 0.f ? 0.f : o[j][2 * i] * f;
            y[8 + j] = l[i] == 0.f ? 0.f : o[j][2 * i + 1] * f;
            wild[i] |= !(fabsf(y[j]) <= 3.4e38f) || !(fabsf(y[8 + j]) <= 3.4e38f);
          }
          wild[i] &= l[i] == l[i];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (kE4m3) store_pair(p, at, 16 * t + 2 * j, y[2 * j], y[2 * j + 1]);
            else store_pair(p, at, 8 * j + 2 * t, y[j], y[8 + j]);
          }
          if (p.lse != nullptr && t == 0) p.lse[at] = log_sum(m[i], l[i]);
        }
        uint32_t which = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t b = __ballot_sync(0xffffffffu, wild[i]);
          for (int r = 0; b != 0 && r < 8; ++r)
            if ((b >> (4 * r)) & 15u) which |= 1u << (r + 8 * i);
        }
        if (which != 0) {
          __syncwarp();
          redo_rows<kE4m3>(a, p, which, s0 + cons.s, s_row0[cons.s], n, len, cons.h);
        }
      } else {
        float* slot = started_before ? head_slot : tail_slot;
        if (!started_before) __syncwarp();   // (the ring's last reads are done)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = g + 8 * i;
          float* to = slot + row * kSlotStride;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (kE4m3) {
              to[16 * t + j] = o[j][2 * i];
              to[16 * t + 8 + j] = o[j][2 * i + 1];
            } else {
              *reinterpret_cast<float2*>(to + 8 * j + 2 * t) = make_float2(o[j][2 * i], o[j][2 * i + 1]);
            }
          }
          if (t == 0) {
            slot[kM * kSlotStride + row] = m[i];
            slot[kM * kSlotStride + kM + row] = M[i];
            slot[kM * kSlotStride + 2 * kM + row] = l[i];
          }
        }
      }
      new_item = true;
    }
    if (done < hi) advance(cons);
  }
  if (!ok) {   // wait (a little) for the loads in flight before the CTA can leave
    for (int64_t u = done; u < issued; ++u) mbar_wait_bounded(bar(static_cast<int>((u - lo) % kS)), static_cast<uint32_t>((u - lo) / kS) & 1u, 1000000ull);
  }
  ok = __syncthreads_and(ok);

  // ---------------------------------------------------------------- items over several warps of this CTA
  // `cons` is the last item of the warp's units; its first one it finds again.  The warps that have some of an item
  // share its row heads.
  float* ws_part = ws + static_cast<int64_t>(blockIdx.x) * kStepWsFloats;
  if (ok && lo < hi) {
    At first{};
    locate(lo, first);
    const bool same = first.s == cons.s && first.h == cons.h;
#pragma unroll 1
    for (int what = 0; what < (same ? 1 : 2); ++what) {
      const At& at = what == 0 ? first : cons;
      const int64_t ib = what == 0 ? lo - first.blk : hi - 1 - cons.blk, ie = ib + at.units;
      if (ib >= lo && ie <= hi) continue;
      int w0 = warp, w1 = warp;   // the first and the last warp of the CTA with some of it
      while (w0 > 0 && edge_of(w0) > ib) --w0;
      while (w1 < kW - 1 && edge_of(w1 + 1) < min(ie, cta_hi)) ++w1;
      const int parts = w1 - w0 + 1;
      const bool complete = ib >= cta_lo && ie <= cta_hi;
      const bool w0_head = edge_of(w0) > ib;      // (the later ones have it in their head slots)
      const int n = s_count[at.s], mh = n * p.group;
      float* out_slot = ws_part + (ib < cta_lo ? 0 : kSlotFloats);
      const float* mine = slot_of(w0 + min(lane, parts - 1), min(lane, parts - 1) > 0 || w0_head) + kM * kSlotStride;
      uint32_t which = 0;
      for (int row = warp - w0; row < mh; row += parts) {
        const float pm = lane < parts ? mine[row] : -INFINITY, pM = lane < parts ? mine[kM + row] : -INFINITY;
        float jm = pm, jM = pM;
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) {
          jm = fmaxf(jm, __shfl_xor_sync(0xffffffffu, jm, d));
          jM = fmaxf(jM, __shfl_xor_sync(0xffffffffu, jM, d));
        }
        jm = __shfl_sync(0xffffffffu, jm, 0), jM = __shfl_sync(0xffffffffu, jM, 0);
        const float f = rescale(pM, jM);
        float jl = lane < parts ? mine[2 * kM + row] * rescale(pm, jm) : 0.f;
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) jl += __shfl_xor_sync(0xffffffffu, jl, d);
        jl = __shfl_sync(0xffffffffu, jl, 0);
        float2 jo = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int w = 0; w < parts; ++w) {
          const float2 part =
              *reinterpret_cast<const float2*>(slot_of(w0 + w, w > 0 || w0_head) + row * kSlotStride + 2 * lane);
          const float fw = __shfl_sync(0xffffffffu, f, w);
          jo.x = fmaf(fw, part.x, jo.x), jo.y = fmaf(fw, part.y, jo.y);
        }
        if (complete) {
          const int64_t o_at = (s_row0[at.s] + static_cast<int64_t>(row / p.group)) * p.heads + at.h * p.group + row % p.group;
          const float of = out_factor<kE4m3>(jm, jM, jl);
          const float y0 = jl == 0.f ? 0.f : jo.x * of, y1 = jl == 0.f ? 0.f : jo.y * of;
          store_pair(p, o_at, 2 * lane, y0, y1);
          if (p.lse != nullptr && lane == 0) p.lse[o_at] = log_sum(jm, jl);
          if (__any_sync(0xffffffffu, (!(fabsf(y0) <= 3.4e38f) || !(fabsf(y1) <= 3.4e38f)) && jl == jl)) which |= 1u << row;
        } else {
          *reinterpret_cast<float2*>(out_slot + row * kSlotStride + 2 * lane) = jo;
          if (lane == 0) {
            out_slot[kM * kSlotStride + row] = jm;
            out_slot[kM * kSlotStride + kM + row] = jM;
            out_slot[kM * kSlotStride + 2 * kM + row] = jl;
          }
        }
      }
      if (which != 0) {
        __syncwarp();
        redo_rows<kE4m3>(a, p, which, s0 + at.s, s_row0[at.s], n, s_len[at.s], at.h);
      }
    }
  }
  // What the join kernel finds of this CTA: the item that begins here and goes on, if there is one.
  if (tid == 0 && gridDim.x > 1) {
    StepJoin j{};
    if (ok && cta_lo < cta_hi) {
      At at{};
      locate(cta_hi - 1, at);
      const int64_t ib = cta_hi - 1 - at.blk, ie = ib + at.units;
      if (ib >= cta_lo && ie > cta_hi) {
        const int64_t last_warp = (ie * nw - 1) / U;   // of the last unit, ie - 1
        j.parts = static_cast<int32_t>(last_warp / kW) - static_cast<int32_t>(blockIdx.x) + 1;
        j.s = s0 + at.s;
        j.h = at.h;
        j.n = s_count[at.s];
        j.len = s_len[at.s];
        j.row0 = s_row0[at.s];
      }
    }
    *reinterpret_cast<StepJoin*>(ws_part + 2 * kSlotFloats) = j;
  }
}

// One CTA for each CTA of the step kernel: the item that begins in it and goes on, from the parts of this and the next
// CTAs.  16 groups of 16 lanes: first a group has a row head, its lanes the parts' maxima and sums; then a group has a
// row head and every so manieth part, its lanes four elements of O each.
constexpr int kJoinThreads = 256, kJoinEach = kStepMaxGrid / 16;

template <bool kE4m3>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ KvArgs a, const __grid_constant__ PagedAttn p,
                                                                  const float* __restrict__ ws) {
  __shared__ float4 so[16][16];
  __shared__ float factor[kM][kStepMaxGrid];
  __shared__ float total[kM][3];
  __shared__ uint32_t wild;
  griddep_launch_dependents();
  griddep_wait();
  const float* mine = ws + static_cast<int64_t>(blockIdx.x) * kStepWsFloats;
  const StepJoin j = *reinterpret_cast<const StepJoin*>(mine + 2 * kSlotFloats);
  if (j.parts == 0) return;
  const int tid = threadIdx.x, grp = tid >> 4, sub = tid & 15;
  const int mh = j.n * p.group;
  auto part_of = [&](int i) { return mine + static_cast<int64_t>(i) * kStepWsFloats + (i == 0 ? kSlotFloats : 0); };
  if (tid == 0) wild = 0;
  {
    float pm[kJoinEach], pM[kJoinEach], pl[kJoinEach], m = -INFINITY, M = -INFINITY, l = 0.f;
#pragma unroll
    for (int k = 0; k < kJoinEach; ++k) {
      const int i = sub + 16 * k;
      const bool in = i < j.parts && grp < mh;
      const float* st = part_of(in ? i : 0) + kM * kSlotStride + (in ? grp : 0);
      pm[k] = in ? st[0] : -INFINITY, pM[k] = in ? st[kM] : -INFINITY, pl[k] = in ? st[2 * kM] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kJoinEach; ++k) m = fmaxf(m, pm[k]), M = fmaxf(M, pM[k]);
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) {
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    }
#pragma unroll
    for (int k = 0; k < kJoinEach; ++k) {
      l += pl[k] * rescale(pm[k], m);
      if (sub + 16 * k < j.parts) factor[grp][sub + 16 * k] = rescale(pM[k], M);
    }
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    if (sub == 0) total[grp][0] = m, total[grp][1] = M, total[grp][2] = l;
  }
  __syncthreads();
  int rows = 1;
  while (rows < mh) rows <<= 1;
  const int row = grp & (rows - 1), slices = 16 / rows;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (row < mh) {
#pragma unroll 8
    for (int i = grp / rows; i < j.parts; i += slices) {
      const float4 x = *reinterpret_cast<const float4*>(part_of(i) + row * kSlotStride + 4 * sub);
      const float f = factor[row][i];
      o.x = fmaf(f, x.x, o.x), o.y = fmaf(f, x.y, o.y), o.z = fmaf(f, x.z, o.z), o.w = fmaf(f, x.w, o.w);
    }
  }
  so[grp][sub] = o;
  __syncthreads();
  if (grp < rows && row < mh) {
    for (int i = 1; i < slices; ++i) {
      const float4 x = so[grp + i * rows][sub];
      o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
    }
    const float m = total[row][0], M = total[row][1], l = total[row][2], f = out_factor<kE4m3>(m, M, l);
    const int64_t at = (j.row0 + static_cast<int64_t>(row / p.group)) * p.heads + j.h * p.group + row % p.group;
    const float y[4] = {o.x * f, o.y * f, o.z * f, o.w * f};
    bool w = false;
#pragma unroll
    for (int c = 0; c < 4; ++c) w |= !(fabsf(y[c]) <= 3.4e38f);
    if (w && l == l && l != 0.f) atomicOr(&wild, 1u << row);
    store_pair(p, at, 4 * sub, l == 0.f ? 0.f : y[0], l == 0.f ? 0.f : y[1]);
    store_pair(p, at, 4 * sub + 2, l == 0.f ? 0.f : y[2], l == 0.f ? 0.f : y[3]);
    if (p.lse != nullptr && sub == 0) p.lse[at] = log_sum(m, l);
  }
  __syncthreads();
  if (wild != 0 && tid < 32) redo_rows<kE4m3>(a, p, wild, j.s, j.row0, j.n, j.len, j.h);
}

template <bool kE4m3>
cudaError_t launch(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const KvArgs& a, const PagedAttn& p, int s0, int ns, int grid,
                   float* ws, cudaStream_t stream) {
  using C = Cfg<kE4m3>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = set_smem_limit_once(paged_step_kernel<kE4m3>, C::kRequest, done);
  if (e != cudaSuccess) return e;
  paged_step_kernel<kE4m3><<<grid, C::kWarps * 32, C::kRequest, stream>>>(tm_k, tm_v, a, p, s0, ns, ws);
  return cudaGetLastError();
}

}  // namespace

static_assert(kStepWsFloats * 4 >= 2 * kSlotFloats * 4 + sizeof(StepJoin), "workspace of a CTA");

int paged_step_grid(int64_t most_units, bool e4m3, int num_sms) {
  const int64_t w = e4m3 ? Cfg<true>::kWarps : Cfg<false>::kWarps;
  return static_cast<int>(std::min<int64_t>(std::min(num_sms, kStepMaxGrid), (most_units + w - 1) / w));
}

cudaError_t launch_paged_step(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const KvArgs& a, const PagedAttn& p, int s0, int ns,
                              int grid, bool e4m3, float* ws, cudaStream_t stream) {
  return e4m3 ? launch<true>(tm_k, tm_v, a, p, s0, ns, grid, ws, stream) : launch<false>(tm_k, tm_v, a, p, s0, ns, grid, ws, stream);
}

cudaError_t launch_paged_join(const KvArgs& a, const PagedAttn& p, int grid, bool e4m3, const float* ws, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return e4m3 ? cudaLaunchKernelEx(&cfg, paged_join_kernel<true>, a, p, ws) : cudaLaunchKernelEx(&cfg, paged_join_kernel<false>, a, p, ws);
}

}  // namespace spanla
