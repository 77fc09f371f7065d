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
// Row elements 2 * lane, 2 * lane + 1 of row `pos` of the cache, given its page.
template <bool kE4m3>
__device__ __forceinline__ float2 cached_pair(const KvArgs& a, const void* base, const uint8_t* scale, int32_t page, int32_t pos,
                                              int head, int lane) {
  const int32_t r = pos & (a.page_rows - 1);
  const int64_t at = page * a.page_stride + head * a.head_stride + r * a.row_stride + 2 * lane;
  if (kE4m3) {
    const float2 x = from_e4m3x2(*reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(base) + at));
    const float e = scale_of(scale[page * a.scale_page_stride + head * a.scale_head_stride + r]);
    return make_float2(x.x * e, x.y * e);
  }
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(static_cast<const __nv_bfloat16*>(base) + at));
}

// Softmax attention of one packed row t and query head by one warp, in fp32
// throughout: the row of sequence s that sees its first `seen` rows.  The other
// kernels send a row here whose products came out infinite or NaN though its sum of
// weights is finite: they multiply rows that the row does not see by 0, this does
// not touch them.  (0.38 us a cached row, four of them at a time, latency: a token over
// 7,401 rows whose V is infinite somewhere 2.8 ms instead of 12 us.)
template <bool kE4m3>
__device__ __noinline__ void attend_row(const KvArgs& a, const PagedAttn& p, int s, int64_t t, int head, int32_t seen) {
  constexpr int kAtOnce = 4;
  const int lane = threadIdx.x & 31, kvh = head / p.group;
  const float2 q = __bfloat1622float2(
      *reinterpret_cast<const __nv_bfloat162*>(p.q + t * p.q_row_stride + head * kHeadDim + 2 * lane));
  float m = -INFINITY, l = 0.f;
  float2 o = make_float2(0.f, 0.f);
  bool bad = false;
  for (int32_t j0 = 0; j0 < seen; j0 += kAtOnce) {   // (a page holds a multiple of kAtOnce rows)
    const int32_t page = page_of(a, s, j0);
    if (page < 0) {
      bad = true;
      continue;
    }
    const int n = min(kAtOnce, seen - j0);
    float2 v[kAtOnce];
    float x[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      v[i] = make_float2(0.f, 0.f), x[i] = 0.f;
      if (i >= n) continue;
      const float2 k = cached_pair<kE4m3>(a, a.k, a.k_scale, page, j0 + i, kvh, lane);
      v[i] = cached_pair<kE4m3>(a, a.v, a.v_scale, page, j0 + i, kvh, lane);
      x[i] = q.x * k.x + q.y * k.y;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], d);
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (i >= n) break;
      const float y = x[i] * p.scale;
      if (y == -INFINITY) continue;   // weight 0
      const float m_new = y > m || y != y ? y : m;
      const float old = m == m_new ? 1.f : m == -INFINITY ? 0.f : expf(m - m_new), w = expf(y - m_new);
      l = l * old + w;
      o.x = (old == 0.f ? 0.f : o.x * old) + w * v[i].x;
      o.y = (old == 0.f ? 0.f : o.y * old) + w * v[i].y;
      m = m_new;
    }
  }
  if (bad && lane == 0) atomicOr(a.err, kErrPage);
  const bool none = l == 0.f;
  const int64_t at = t * p.heads + head;
  *reinterpret_cast<uint32_t*>(p.out + at * kHeadDim + 2 * lane) = none ? 0u : pack_bf16x2(o.x / l, o.y / l);
  if (p.lse != nullptr && lane == 0) p.lse[at] = none ? -INFINITY : m + logf(l);
}

}  // namespace spanla
