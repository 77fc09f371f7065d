// The paged cache of keys and values on the device: where a sequence's rows
// stand, and e4m3 rows with a power of two each.
//
// Page tables, lengths and row offsets are device memory that a host check
// cannot see, so each kernel checks what it reads of them: a sequence whose
// offsets or length are out of range is skipped, a page out of range is not
// touched, and either sets a bit of the device error word (span_la_check).
#pragma once

#include <utility>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "spanla_internal.h"
#include "tc_ptx.cuh"

namespace spanla {

// A sequence's part of a call: packed rows [row0, row0 + n), whose last one is
// row len - 1 of the sequence.  n = 0 where there is nothing to do (or it is
// out of range: then *bad is set).
struct SeqRows {
  int64_t row0;
  int32_t n, len;
};

__device__ __forceinline__ SeqRows rows_between(const KvArgs& a, int64_t b, int64_t e, int32_t len, bool* bad) {
  const bool wrong = b < 0 || e < b || e > a.rows || e - b > a.max_rows || len < 0 || len > a.capacity;
  if (wrong) *bad = true;
  return {b, wrong ? 0 : static_cast<int32_t>(e - b), wrong ? 0 : len};
}

__device__ __forceinline__ SeqRows seq_rows(const KvArgs& a, int s, bool* bad) {
  return rows_between(a, a.row_cu != nullptr ? a.row_cu[s] : s, a.row_cu != nullptr ? a.row_cu[s + 1] : s + 1, a.seq_len[s], bad);
}

// The sequence whose rows hold packed row t, or -1.
__device__ __forceinline__ int seq_of_row(const KvArgs& a, int64_t t) {
  if (a.row_cu == nullptr) return t < a.seqs ? static_cast<int>(t) : -1;
  int lo = 0, hi = a.seqs + 1;   // the first offset above t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a.row_cu[mid] <= t) lo = mid + 1;
    else hi = mid;
  }
  return lo >= 1 && lo <= a.seqs ? lo - 1 : -1;
}

// Entry i of sequence s in the table as a page of the arrays, or -1 (out of range).
__device__ __forceinline__ int32_t page_at(const KvArgs& a, int s, int32_t i) {
  const int32_t p = a.table[s * a.table_stride + i];
  return p < 0 || p >= a.pages ? -1 : a.copied > 0 ? s * a.copied + i : p;
}

// The page of row `pos` (0 <= pos < len) of sequence s, or -1.
__device__ __forceinline__ int32_t page_of(const KvArgs& a, int s, int32_t pos) { return page_at(a, s, pos >> a.page_shift); }

// Every sequence's offsets and length, by the threads of one CTA.
__device__ __forceinline__ void check_sequences(const KvArgs& a) {
  bool bad = false;
  for (int s = threadIdx.x; s < a.seqs; s += blockDim.x) seq_rows(a, s, &bad);
  if (bad) atomicOr(a.err, kErrSequence);
}

// A launch whose CTAs may come up while the kernel before it in the stream still runs; they wait for its end
// (griddep_wait) before they touch memory.  Calls one behind the other then do not wait for each other's launch.  What
// such a kernel reads may be written while it is up, so it reads nothing by __restrict__ const pointers or __ldg: the
// compiler may take those reads past the wait.
template <typename... Params, typename... Args>
inline cudaError_t launch_behind(void (*kernel)(Params...), dim3 grid, int threads, uint32_t smem, cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// a / b, quickly where both fit 32 bits.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

// 2^(code - 127); 255 is NaN.
__device__ __forceinline__ float scale_of(uint32_t code) {
  return __uint_as_float(code == 0 ? 0x00400000u : code == 255 ? 0x7fffffffu : code << 23);
}

// Two e4m3 values (the low byte first) as fp32; exact.
__device__ __forceinline__ float2 from_e4m3x2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
  return __half22float2(__half2(h));
}

// Four e4m3 values as two pairs of fp16.
__device__ __forceinline__ void half2_of_e4m3(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(four));
}

// Eight elements of a cached row, as they lie and as fp32.
template <bool kE4m3>
struct EightOf;
template <>
struct EightOf<false> {
  uint4 w;
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    w = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at);
  }
  __device__ __forceinline__ void get(float, float (&x)[8]) const {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) x[2 * c] = __uint_as_float(v[c] << 16), x[2 * c + 1] = __uint_as_float(v[c] & 0xffff0000u);
  }
  __device__ __forceinline__ bool finite() const {   // (0x0080 carried into a half's sign bit: its exponent was all ones)
    auto carry = [](uint32_t v) { return (v & 0x7f807f80u) + 0x00800080u; };
    return ((carry(w.x) | carry(w.y) | carry(w.z) | carry(w.w)) & 0x80008000u) == 0;
  }
};
template <>
struct EightOf<true> {
  uint2 w;
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(base) + at);
  }
  __device__ __forceinline__ void get(float scale, float (&x)[8]) const {
    const uint32_t v[2] = {w.x, w.y};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float2 y = from_e4m3x2((v[c >> 1] >> (16 * (c & 1))) & 0xffffu);
      x[2 * c] = y.x * scale, x[2 * c + 1] = y.y * scale;
    }
  }
  __device__ __forceinline__ bool finite() const {   // (0x7f is NaN)
    return ((((w.x & 0x7f7f7f7fu) + 0x01010101u) | ((w.y & 0x7f7f7f7fu) + 0x01010101u)) & 0x80808080u) == 0;
  }
};

__device__ __forceinline__ bool bf16_finite(uint32_t bits) { return (bits & 0x7f80u) != 0x7f80u; }

// What elements to be found again by the join kernel hold till then: a NaN that no rounding gives.  (A row whose scores are
// NaN is NaN, and stays so.)
constexpr uint32_t kRedoMark = 0x7f81u;
__device__ __forceinline__ bool has_mark(uint32_t two) { return (two & 0xffffu) == kRedoMark || two >> 16 == kRedoMark; }
__device__ __forceinline__ uint32_t marked(uint32_t two) {
  return (bf16_finite(two) ? two & 0xffffu : kRedoMark) | (bf16_finite(two >> 16) ? two & 0xffff0000u : kRedoMark << 16);
}

// q . k of a row head, whose eight lanes have eight elements each.
template <bool kE4m3>
__device__ __forceinline__ float dot64(const EightOf<false>& q, const EightOf<kE4m3>& k, float k_scale) {
  float x[8], y[8], sum = 0.f;
  q.get(1.f, x);
  k.get(k_scale, y);
#pragma unroll
  for (int c = 0; c < 8; ++c) sum = fmaf(x[c], y[c], sum);
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  return sum;
}

// Elements of o that came out infinite or NaN, once more, by one warp.  The kernels multiply rows that a row does not see
// by weights of 0, and 0 times an infinity or a NaN is NaN; weights that are no fp32 number any more, or sums past one, end
// there too.  This touches only what a row sees.  `which` names row heads base + i (i a bit) of the rows from packed row
// row0 on, of which row r sees the first seen0 + r rows of sequence s; their o has been stored, by any lanes of the warp (or
// before a barrier), and only what is not finite in it is stored again.  Four row heads at a time, eight lanes each, eight
// elements a lane.
//
// First, what is not finite in the rows of V that they see, and has a score above -infinity: the sum of that is the answer,
// however small its weight.  (The first 17 to 32 such rows are looked for once for all row heads, 16 rows at a time, more of
// them by each four; most calls end here.)  Where there is none, the rest:
//
//   l' = l e^(m - m') + sum w,   o' = o l e^(m - m') / l' + sum w / l' v,   w = e^(x - m')
//
// in fp32: a mean at every step, which passes fp32 no more than V does.
template <bool kE4m3>
__device__ __noinline__ void redo_rows(const KvArgs& a, const PagedAttn& p, uint32_t which, int s, int kvh, int64_t row0, int base,
                                       int32_t seen0) {
  constexpr int kAtOnce = 4, kScan = 16;   // (a page holds a multiple of both)
  const int lane = threadIdx.x & 31, part = lane & 7;
  auto scale_at = [&](const uint8_t* scales, int32_t page, int32_t in) {
    return kE4m3 ? scale_of(scales[page * a.scale_page_stride + kvh * a.scale_head_stride + in]) : 1.f;
  };
  // Of the 16 rows from j on, those below `end` with anything in V that is not finite (bits).
  auto scan = [&](int32_t page, int32_t j, int32_t end) {
    const int32_t in = (j & (a.page_rows - 1)) + (lane >> 3);
    EightOf<kE4m3> v[kScan / 4];
#pragma unroll
    for (int i = 0; i < kScan / 4; ++i) v[i].load(a.v, page * a.page_stride + kvh * a.head_stride + 8 * part + (in + 4 * i) * a.row_stride);
    uint32_t rows = 0;
#pragma unroll
    for (int i = 0; i < kScan / 4; ++i) {
      const bool found = !v[i].finite() || (kE4m3 && !(scale_at(a.v_scale, page, in + 4 * i) < INFINITY));
      const uint32_t b = __ballot_sync(0xffffffffu, found && j + (lane >> 3) + 4 * i < end);
#pragma unroll
      for (int g = 0; g < 4; ++g) rows |= (b >> (8 * g)) & 0xffu ? 1u << (4 * i + g) : 0u;
    }
    return rows;
  };
  int listed = 0;              // lane i has the i-th such row
  int32_t list = 0, next = 0;  // rows before `next` have been looked at
  const int32_t last = which != 0 ? max(0, seen0 + (base + 31 - __clz(which)) / p.group) : 0;   // rows that any of them sees
  for (int32_t page = -1; next < last && listed <= 32 - kScan; next += kScan) {
    if ((next & (a.page_rows - 1)) == 0) {
      page = page_of(a, s, next);
      if (page < 0) atomicOr(a.err, kErrPage);
    }
    if (page < 0) continue;
    for (uint32_t rows = scan(page, next, last); rows != 0; rows &= rows - 1, ++listed)
      if (lane == listed) list = next + __ffs(rows) - 1;
  }
  while (which != 0) {
    int mine = -1;   // lanes 8 g .. 8 g + 7 have the g-th of them
    for (int g = 0; g < 4 && which != 0; ++g) {
      if (g == lane >> 3) mine = __ffs(which) - 1;
      which &= which - 1;
    }
    const int rr = base + max(mine, 0), r = rr / p.group, head = kvh * p.group + rr % p.group;
    const int32_t seen = mine < 0 ? 0 : max(0, seen0 + r);
    uint32_t* out = reinterpret_cast<uint32_t*>(p.out + ((row0 + r) * p.heads + head) * kHeadDim + 8 * part);
    uint32_t wanted = 0;   // elements to be found
    __syncwarp();          // (what lanes of this warp have stored)
    if (mine >= 0) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        wanted |= (bf16_finite(out[c]) ? 0u : 1u << (2 * c)) | (bf16_finite(out[c] >> 16) ? 0u : 2u << (2 * c));
    }
    int32_t most = seen;   // rows to look at
#pragma unroll
    for (int d = 8; d < 32; d <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
    EightOf<false> q;
    q.load(p.q, (row0 + r) * p.q_row_stride + head * kHeadDim + 8 * part);
    float o[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) o[c] = 0.f;
    // ------------------------------------------------------------ what is not finite
    uint32_t met = 0;
    int32_t page = -1;
    auto look_at = [&](int32_t j, int32_t of_page) {
      const int32_t in = j & (a.page_rows - 1);
      const int64_t at = of_page * a.page_stride + kvh * a.head_stride + in * a.row_stride + 8 * part;
      EightOf<kE4m3> kk, vv;
      kk.load(a.k, at);
      vv.load(a.v, at);
      const float x = dot64<kE4m3>(q, kk, scale_at(a.k_scale, of_page, in)) * p.scale;
      if (j >= seen || x == -INFINITY) return;
      float y[8];
      vv.get(scale_at(a.v_scale, of_page, in), y);
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (!(fabsf(y[c]) < INFINITY)) o[c] += y[c], met |= 1u << c;
    };
    for (int i = 0; i < listed; ++i) {
      const int32_t j = __shfl_sync(0xffffffffu, list, i);
      look_at(j, page_of(a, s, j));
    }
    for (int32_t j0 = next; j0 < most; j0 += kScan) {
      if (j0 == next || (j0 & (a.page_rows - 1)) == 0) {
        page = page_of(a, s, j0);
        if (page < 0) atomicOr(a.err, kErrPage);
        bool open = false;   // some element is not NaN yet
#pragma unroll
        for (int c = 0; c < 8; ++c) open |= ((wanted >> c) & 1u) && o[c] == o[c];
        if (!__any_sync(0xffffffffu, open)) break;
      }
      if (page < 0) continue;
      for (uint32_t rows = scan(page, j0, most); rows != 0; rows &= rows - 1) look_at(j0 + __ffs(rows) - 1, page);
    }
    __syncwarp();
    auto store = [&](uint32_t which_ones) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t take = (which_ones >> (2 * c)) & 3u, two = pack_bf16x2(o[2 * c], o[2 * c + 1]);
        if (take != 0) out[c] = take == 3u ? two : take == 1u ? (out[c] & 0xffff0000u) | (two & 0xffffu) : (out[c] & 0xffffu) | (two & 0xffff0000u);
      }
    };
    store(wanted & met);
    wanted &= ~met;
    if (!__any_sync(0xffffffffu, wanted != 0)) continue;
    // ------------------------------------------------------------ what is
    float m = -INFINITY, l = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) o[c] = 0.f;
    for (int32_t j = 0; j < most; j += kAtOnce) {
      if ((j & (a.page_rows - 1)) == 0) {
        page = page_of(a, s, j);
        if (__all_sync(0xffffffffu, wanted == 0 || l != l)) break;   // (NaN scores)
      }
      if (page < 0) continue;
      EightOf<kE4m3> kk[kAtOnce], vv[kAtOnce];
      const int64_t at = page * a.page_stride + kvh * a.head_stride + 8 * part;
      auto in_page = [&](int i) { return (j + i < most ? j + i : j) & (a.page_rows - 1); };   // (no row that nobody sees)
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) kk[i].load(a.k, at + in_page(i) * a.row_stride), vv[i].load(a.v, at + in_page(i) * a.row_stride);
      float w[kAtOnce], top = m;
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        w[i] = dot64<kE4m3>(q, kk[i], scale_at(a.k_scale, page, in_page(i))) * p.scale;
        if (j + i >= seen) w[i] = -INFINITY;
        top = fmaxf(top, w[i]);
      }
      const float old = m == top ? l : m == -INFINITY ? 0.f : l * expf(m - top);
      float sum = old;
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        w[i] = w[i] == -INFINITY ? 0.f : expf(w[i] - top);
        sum += w[i];
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum, keep = old * inv;
      m = top, l = sum;
#pragma unroll
      for (int c = 0; c < 8; ++c) o[c] *= keep;
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const float f = w[i] * inv;
        float v[8];
        vv[i].get(scale_at(a.v_scale, page, in_page(i)), v);
        if (f != 0.f) {   // (what has no weight may hold anything)
#pragma unroll
          for (int c = 0; c < 8; ++c) o[c] = fmaf(f, v[c], o[c]);
        }
      }
    }
    store(wanted);
  }
}

}  // namespace spanla
