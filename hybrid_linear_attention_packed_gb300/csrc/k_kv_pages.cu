// Packed rows of keys and values into the paged cache, quantised on the way,
// and back.  Both are bound by memory.
//
// A row and head of e4m3 pages is held as y = x / 2^e rounded to e4m3 with the
// least e >= -126 at which its largest finite magnitude is at most 448 2^e.  (A
// floating-point grid is as fine at any scale, so a power of two loses nothing
// to the exact quotient, and y 2^e is a bf16 number: reading back rounds
// nothing.)  e is at most 119: beyond 448 2^119 = 1.75 2^127 magnitudes come out as
// that, as the next value of the grid is not an fp32 number.  Infinite and NaN
// elements are held as NaN.
//
// A CTA of 8 warps takes 32 packed rows; each warp one head of K or V of 16 of them
// at a time, 8 lanes a row (16 bytes of bf16 a lane), 4 rows at once, all 16 in
// flight.  Consecutive rows of one head are neighbours in a page, and their powers
// of two go out as one store.  (All 32 rows at once: twice the registers and half
// the warps, 45 us for four prompts of fp32 rows where 16 took 40, before launches
// overlapped.)  Few rows are bound
// by the reads that find their places, one behind the other: lengths, then the
// page; the rows themselves are on their way meanwhile.  Measured: four prompts of
// fp32 rows (20,576 rows, 16 heads) into e4m3 pages 36.6 us, 5.8 TB/s (35.3 one call
// behind the other); sixteen views
// (87,648 rows) out of bf16 pages 109.5 us, 6.6 TB/s; eight tokens written 2.7 us.
#include <algorithm>

#include "paged.cuh"

namespace spanla {
namespace {

constexpr int kRows = 32, kWarps = 8, kSteps = 4;
constexpr int64_t kBlocks = 4864;   // 32 for each of 152 SMs

struct Places {            // of a CTA's rows: element offset of head 0 in the pages (-1: none), byte offset in the scales
  int64_t at[kRows], scale_at[kRows];
};

// The sequence of a row near row t0 of a warp's 32 rows: all lanes look for t0's together (32 offsets at a time), then
// each goes on to its own, which mostly is the same.
__device__ __forceinline__ int find_seq(const KvArgs& a, int64_t t0) {
  const int lane = threadIdx.x & 31;
  const int64_t t = t0 + lane;
  int lo = 0, n = a.seqs + 1;
  while (n > 1) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const int upto = __popc(__ballot_sync(0xffffffffu, at < lo + n && a.row_cu[min(at, a.seqs)] <= t0));
    const int from = max(upto - 1, 0) * step;
    n = min(step, n - from);
    lo += from;
  }
  for (int i = 0; i < 4; ++i) {
    if (lo >= a.seqs) return -1;
    if (a.row_cu[lo + 1] > t) return lo;   // (a.row_cu[lo] > t: the caller sees that)
    ++lo;
  }
  return seq_of_row(a, t);
}

// The sequence of a warp's row t0 + lane, or -1, and its part of the call.  Up to 31 sequences by one read of all
// offsets and lengths, each lane's own; more of them by a search.
__device__ __forceinline__ int find_rows(const KvArgs& a, int64_t t0, SeqRows* r) {
  const int lane = threadIdx.x & 31;
  const int64_t t = t0 + lane;
  bool bad = false;
  if (a.row_cu == nullptr || a.seqs > 31) {
    const int s = a.row_cu == nullptr ? (t < a.seqs ? static_cast<int>(t) : -1) : find_seq(a, t0);
    if (s >= 0 && t < a.rows) *r = seq_rows(a, s, &bad);
    return s >= 0 && t < a.rows ? s : -1;
  }
  const int32_t cu = a.row_cu[min(lane, a.seqs)], len = a.seq_len[min(lane, a.seqs - 1)];
  int s = -1;
  for (int i = 0; i < a.seqs; ++i)
    if (__shfl_sync(0xffffffffu, cu, i) <= t) s = i;
  const int64_t b = __shfl_sync(0xffffffffu, cu, max(s, 0)), e = __shfl_sync(0xffffffffu, cu, max(s, 0) + 1);
  const int32_t n = __shfl_sync(0xffffffffu, len, max(s, 0));
  *r = rows_between(a, b, e, n, &bad);
  return t < a.rows ? s : -1;
}

__device__ __forceinline__ void find_places(const KvArgs& a, Places& pl) {
  if (threadIdx.x < kRows) {
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kRows, t = t0 + threadIdx.x;
    int64_t at = -1, scale_at = 0;
    SeqRows r{};
    const int s = find_rows(a, t0, &r);
    if (s >= 0) {
      const int64_t pos = r.len - (r.n - (t - r.row0));   // (negative: the sequence is shorter than its packed rows)
      if (t >= r.row0 && t - r.row0 < r.n && pos >= 0) {
        const int32_t page = page_of(a, s, static_cast<int32_t>(pos));
        if (page < 0) {
          atomicOr(a.err, kErrPage);
        } else {
          const int32_t in = static_cast<int32_t>(pos) & (a.page_rows - 1);
          at = page * a.page_stride + in * a.row_stride;
          scale_at = page * a.scale_page_stride + in;
        }
      }
    }
    pl.at[threadIdx.x] = at;
    pl.scale_at[threadIdx.x] = scale_at;
  }
  if (blockIdx.x == 0 && blockIdx.y == 0) check_sequences(a);
  __syncthreads();
}

// 8 elements as they lie in memory, and as fp32.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p), b = *(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void store(float* p) const { reinterpret_cast<float4*>(p)[0] = a, reinterpret_cast<float4*>(p)[1] = b; }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&x)[8]) { a = make_float4(x[0], x[1], x[2], x[3]), b = make_float4(x[4], x[5], x[6], x[7]); }
};
template <>
struct Eight<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = a; }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    a = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  }
};
// One type into another: rounded once, the same type as it is.
template <typename To, typename From>
__device__ __forceinline__ void convert(const Eight<From>& x, Eight<To>& y) {
  float f[8];
  x.get(f);
  y.set(f);
}
template <typename T>
__device__ __forceinline__ void convert(const Eight<T>& x, Eight<T>& y) {
  y = x;
}

// max(a, |b|, |c|), NaN if one of them is.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
  return d;
}

__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

// Units u: 16 of the rows (u & 1: the second 16), K or V (u & 2), head u / 4; a CTA's warps take every so manieth one.
template <typename T, bool kE4m3>
__global__ void __launch_bounds__(kWarps * 32) kv_write_kernel(const __grid_constant__ KvArgs a, const __grid_constant__ KvRows in) {
  __shared__ Places pl;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, sub = lane & 7;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kRows;
  Eight<T> x[kSteps];
  auto load = [&](int unit) {   // (rows of no sequence too: their places are not known yet)
    const T* src = static_cast<const T*>((unit & 2) ? in.v : in.k) + (unit >> 2) * kHeadDim + sub * 8;
    const int64_t stride = (unit & 2) ? in.v_row_stride : in.k_row_stride;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int64_t t = t0 + 16 * (unit & 1) + 4 * i + (lane >> 3);
      x[i] = Eight<T>{};
      if (t < a.rows) x[i].load(src + t * stride);
    }
  };
  const int first = blockIdx.y * kWarps + (threadIdx.x >> 5);
  if (first < 4 * a.heads) load(first);
  find_places(a, pl);
  for (int unit = first; unit < 4 * a.heads; unit += gridDim.y * kWarps) {
    const int head = unit >> 2, half = 16 * (unit & 1);
    const bool is_v = unit & 2;
    if (unit != first) load(unit);
    uint32_t code = 0;   // row `half + lane`'s power of two, lanes 0 .. 15
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int r = half + 4 * i + (lane >> 3);
      const int64_t at = pl.at[r] + head * a.head_stride + sub * 8;
      if (kE4m3) {
        float f[8];
        x[i].get(f);
        // The largest magnitude, NaN if there is one; where it is not finite, that of the finite ones (and NaN for the
        // others).
        float big = max3_abs(0.f, f[0], f[1]);
#pragma unroll
        for (int c = 2; c < 8; c += 2) big = max3_abs(big, f[c], f[c + 1]);
        uint32_t top = __float_as_uint(big);
        if (__any_sync(0xffffffffu, !finite(big))) {
          top = 0;   // (magnitudes as bits order like numbers)
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            if (finite(f[c])) top = max(top, __float_as_uint(f[c]) & 0x7fffffffu);
            else f[c] = NAN;
          }
        }
#pragma unroll
        for (int d = 4; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        // top = m 2^E, 1 <= m < 2: at most 448 2^e = 1.75 2^(8 + e) from e = E - 8 on, or E - 7 where m > 1.75.
        const int e = min(119, max(-126, static_cast<int>(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0)));
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        const uint32_t mine = __shfl_sync(0xffffffffu, static_cast<uint32_t>(e + 127), (lane & 3) * 8);
        if ((lane >> 2) == i) code = mine;
        if (pl.at[r] >= 0) {
          uint32_t w[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float y0, y1;
            f32x2_split(mul_f32x2(f32x2(f[2 * c], f[2 * c + 1]), f32x2(inv, inv)), y0, y1);
            w[c] = __nv_cvt_float2_to_fp8x2(make_float2(y0, y1), __NV_SATFINITE, __NV_E4M3);
          }
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? a.v : a.k) + at) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
        }
      } else if (pl.at[r] >= 0) {
        Eight<__nv_bfloat16> y;
        convert(x[i], y);
        y.store(static_cast<__nv_bfloat16*>(is_v ? a.v : a.k) + at);
      }
    }
    if (kE4m3 && lane < 16 && pl.at[half + lane] >= 0)
      (is_v ? a.v_scale : a.k_scale)[pl.scale_at[half + lane] + head * a.scale_head_stride] = static_cast<uint8_t>(code);
  }
}

template <typename T, bool kE4m3>
__global__ void __launch_bounds__(kWarps * 32) kv_read_kernel(const __grid_constant__ KvArgs a, const __grid_constant__ KvRows to) {
  __shared__ Places pl;
  griddep_wait();
  griddep_launch_dependents();
  find_places(a, pl);
  const int lane = threadIdx.x & 31, sub = lane & 7;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kRows;
  for (int unit = blockIdx.y * kWarps + (threadIdx.x >> 5); unit < 4 * a.heads; unit += gridDim.y * kWarps) {
    const int head = unit >> 2, half = 16 * (unit & 1);
    const bool is_v = unit & 2;
    T* dst = static_cast<T*>(is_v ? to.v : to.k) + head * kHeadDim + sub * 8;
    const int64_t stride = is_v ? to.v_row_stride : to.k_row_stride;
    if (kE4m3) {
      uint2 raw[kSteps];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int r = half + 4 * i + (lane >> 3);
        raw[i] = make_uint2(0u, 0u);
        if (pl.at[r] >= 0)
          raw[i] = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(is_v ? a.v : a.k) + pl.at[r] + head * a.head_stride + sub * 8);
      }
      const float scale =
          pl.at[half + (lane & 15)] >= 0 ? scale_of((is_v ? a.v_scale : a.k_scale)[pl.scale_at[half + (lane & 15)] + head * a.scale_head_stride]) : 0.f;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int r = half + 4 * i + (lane >> 3);
        const float e = __shfl_sync(0xffffffffu, scale, r - half);
        const uint32_t w[2] = {raw[i].x, raw[i].y};
        float f[8];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float2 y = from_e4m3x2((w[c >> 1] >> (16 * (c & 1))) & 0xffffu);
          f[2 * c] = y.x * e, f[2 * c + 1] = y.y * e;
        }
        Eight<T> y;
        y.set(f);
        if (pl.at[r] >= 0) y.store(dst + (t0 + r) * stride);
      }
    } else {
      Eight<__nv_bfloat16> x[kSteps];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int r = half + 4 * i + (lane >> 3);
        if (pl.at[r] >= 0) x[i].load(static_cast<const __nv_bfloat16*>(is_v ? a.v : a.k) + pl.at[r] + head * a.head_stride + sub * 8);
      }
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int r = half + 4 * i + (lane >> 3);
        Eight<T> y;
        convert(x[i], y);
        if (pl.at[r] >= 0) y.store(dst + (t0 + r) * stride);
      }
    }
  }
}

// A warp: 16 rows of one page and head, of K or V.  Bound by memory (65 bytes in, 128 out, a row and head) and, as small
// as it is, by its launch: 20,048 rows of 4 key heads 10 us from cold caches.
__global__ void __launch_bounds__(kWarps * 32) kv_expand_kernel(const __grid_constant__ KvArgs a, const __grid_constant__ KvArgs to,
                                                                int group) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, sub = lane & 7, per_page = a.page_rows / 16;
  // (sequence, page, head, K or V, 16 rows): the last varies fastest
  int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int r0 = 16 * static_cast<int>(u % per_page);
  u /= per_page;
  const bool is_v = u & 1;
  u >>= 1;
  const int head = static_cast<int>(u % a.heads);
  u /= a.heads;
  const int32_t i = static_cast<int32_t>(u % to.copied);
  const int s = static_cast<int>(u / to.copied);
  if (s >= a.seqs) return;
  bool bad = false;
  const SeqRows r = seq_rows(a, s, &bad);
  if (static_cast<int64_t>(r.n) * group <= kStepHeads || static_cast<int64_t>(i) * a.page_rows + r0 >= r.len) return;
  const int32_t page = page_at(a, s, i);
  if (page < 0) return;   // (the chunk kernel says so)
  const int64_t from = page * a.page_stride + head * a.head_stride + sub * 8;
  uint2 raw[kSteps];
#pragma unroll
  for (int k = 0; k < kSteps; ++k)
    raw[k] = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(is_v ? a.v : a.k) + from + (r0 + 4 * k + (lane >> 3)) * a.row_stride);
  const float scale = scale_of((is_v ? a.v_scale : a.k_scale)[page * a.scale_page_stride + head * a.scale_head_stride + r0 + (lane & 15)]);
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_v ? to.v : to.k) + (static_cast<int64_t>(s) * to.copied + i) * to.page_stride +
                       head * to.head_stride + sub * 8;
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int row = 4 * k + (lane >> 3);
    const float e = __shfl_sync(0xffffffffu, scale, row);
    const uint32_t w[2] = {raw[k].x, raw[k].y};
    float f[8];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float2 y = from_e4m3x2((w[c >> 1] >> (16 * (c & 1))) & 0xffffu);
      f[2 * c] = y.x * e, f[2 * c + 1] = y.y * e;
    }
    Eight<__nv_bfloat16> y;
    y.set(f);
    y.store(dst + (r0 + row) * to.row_stride);
  }
}

template <typename Kernel>
cudaError_t launch(Kernel kernel, const KvArgs& a, const KvRows& x, cudaStream_t stream) {
  // A CTA takes several heads of its rows where there are CTAs enough: finding the rows' places takes as long as copying a
  // few heads.  (In a graph, all heads, with 32 CTAs an SM, one head a warp: sixteen views out of bf16 pages 111.6, 109.1
  // and 110.5 us, out of e4m3 pages 88.4, 86.4 and 85.0; one view 8.8, 7.1, 7.1; four prompts written 44.0, 35.3, 35.2.)
  const int64_t blocks = (a.rows + kRows - 1) / kRows;
  const int64_t eights = (4 * a.heads + kWarps - 1) / kWarps;
  const int64_t turns = std::max<int64_t>(1, eights * blocks / kBlocks), split = (eights + turns - 1) / turns;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(split));
  return launch_behind(kernel, grid, kWarps * 32, 0, stream, a, x);
}

}  // namespace

cudaError_t launch_kv_write(const KvArgs& a, const KvRows& x, bool e4m3, bool f32, cudaStream_t stream) {
  if (f32) return launch(e4m3 ? kv_write_kernel<float, true> : kv_write_kernel<float, false>, a, x, stream);
  return launch(e4m3 ? kv_write_kernel<__nv_bfloat16, true> : kv_write_kernel<__nv_bfloat16, false>, a, x, stream);
}

cudaError_t launch_kv_expand(const KvArgs& a, const KvArgs& to, int group, cudaStream_t stream) {
  const int64_t warps = static_cast<int64_t>(a.seqs) * to.copied * a.heads * 2 * (a.page_rows / 16);
  return launch_behind(kv_expand_kernel, dim3(static_cast<unsigned>((warps + kWarps - 1) / kWarps)), kWarps * 32, 0, stream, a, to, group);
}

cudaError_t launch_kv_read(const KvArgs& a, const KvRows& x, bool e4m3, bool f32, cudaStream_t stream) {
  if (f32) return launch(e4m3 ? kv_read_kernel<float, true> : kv_read_kernel<float, false>, a, x, stream);
  return launch(e4m3 ? kv_read_kernel<__nv_bfloat16, true> : kv_read_kernel<__nv_bfloat16, false>, a, x, stream);
}

}  // namespace spanla
