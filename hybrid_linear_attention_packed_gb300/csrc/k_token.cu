// Single-token kernels: the decayed recurrence for one new row of each
// sequence, and the preparation of queries and keys (RMS norm of each head,
// then the position rotation).  Both are bound by memory.
#include <cuda_bf16.h>

#include "decay_math.cuh"
#include "spanla_internal.h"
#include "tc_ptx.cuh"

namespace spanla {
namespace {

// ------------------------------------------------------------------ step
// One CTA of 128 threads per (token, head): S <- a S + k v^T, o = S^T q.
// Thread (ir, jg) holds rows ir + 8 u (u = 0..7), columns 4 jg .. 4 jg + 3, so
// that all 16 KiB of the state are in flight at once and every warp load or
// store covers two whole rows.  Bound by the state's way in and out, 32 KiB a
// token and head: 1,024 tokens of 16 heads take 82.6 us (bf16), 6.6 TB/s; one
// token takes a launch, 2 us.
constexpr int kStepThreads = 128;

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 a = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xffff0000u), __uint_as_float(a.y << 16),
                     __uint_as_float(a.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float* p, const float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float4 x) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
}

// kSlots: indices carried in the launch's own parameters (0: row t uses state t).
template <int kSlots>
struct StepIndex {
  int32_t at[kSlots];
  __device__ __forceinline__ int32_t of(int64_t t) const { return at[t]; }
};
template <>
struct StepIndex<0> {
  __device__ __forceinline__ int64_t of(int64_t t) const { return t; }
};

template <typename T, int kSlots>
__global__ void __launch_bounds__(kStepThreads)
decay_step_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                  const float* __restrict__ log_decay, float* __restrict__ states, T* __restrict__ out, int H,
                  const __grid_constant__ StepIndex<kSlots> index) {
  __shared__ float sq[kHeadDim], sk[kHeadDim];
  __shared__ float4 part[kStepThreads / 32][16];
  const int64_t t = blockIdx.x / H;
  const int h = blockIdx.x % H;
  const int64_t slot = index.of(t);
  if (slot < 0) return;   // a row of padding: the whole CTA leaves
  const int tid = threadIdx.x, jg = tid & 15, ir = tid >> 4;
  float* S = states + (slot * H + h) * kStateFloats + ir * kHeadDim + 4 * jg;
  float4 s[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) s[u] = *reinterpret_cast<const float4*>(S + 8 * u * kHeadDim);
  const int64_t row = (t * H + h) * kHeadDim;
  if (tid < kHeadDim) {
    sq[tid] = to_float(q[row + tid]);
    sk[tid] = to_float(k[row + tid]);
  }
  const float4 x = load4(v + row + 4 * jg);
  const Factor g = log_decay != nullptr ? decay_factor(load_log_decay(log_decay, h), 1.f) : kNoDecay;
  __syncthreads();
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const float ki = sk[ir + 8 * u], qi = sq[ir + 8 * u];
    float4 y;
    y.x = g.step(s[u].x, ki * x.x);
    y.y = g.step(s[u].y, ki * x.y);
    y.z = g.step(s[u].z, ki * x.z);
    y.w = g.step(s[u].w, ki * x.w);
    *reinterpret_cast<float4*>(S + 8 * u * kHeadDim) = y;
    o.x = fmaf(qi, y.x, o.x);
    o.y = fmaf(qi, y.y, o.y);
    o.z = fmaf(qi, y.z, o.z);
    o.w = fmaf(qi, y.w, o.w);
  }
  o.x += __shfl_xor_sync(0xffffffffu, o.x, 16);
  o.y += __shfl_xor_sync(0xffffffffu, o.y, 16);
  o.z += __shfl_xor_sync(0xffffffffu, o.z, 16);
  o.w += __shfl_xor_sync(0xffffffffu, o.w, 16);
  if ((tid & 31) < 16) part[tid >> 5][jg] = o;
  __syncthreads();
  if (tid < 16) {
    float4 y = part[0][tid];
#pragma unroll
    for (int w = 1; w < kStepThreads / 32; ++w) {
      const float4 z = part[w][tid];
      y.x += z.x; y.y += z.y; y.z += z.z; y.w += z.w;
    }
    store4(out + row + 4 * tid, y);
  }
}

template <typename T, int kSlots>
cudaError_t step_chunk(const StepArgs& a, int64_t t0, int64_t n, cudaStream_t stream) {
  StepIndex<kSlots> index{};
  if constexpr (kSlots > 0)
    for (int64_t i = 0; i < n; ++i) index.at[i] = a.index[t0 + i];
  const int64_t at = t0 * a.H * kHeadDim;
  decay_step_kernel<T, kSlots><<<static_cast<unsigned>(n * a.H), kStepThreads, 0, stream>>>(
      static_cast<const T*>(a.q) + at, static_cast<const T*>(a.k) + at, static_cast<const T*>(a.v) + at, a.log_decay,
      kSlots > 0 ? a.states : a.states + t0 * a.H * kStateFloats, static_cast<T*>(a.out) + at, a.H, index);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ norm and rotation
// One warp per row.  A lane holds 16 bytes of a head (kVec values; kLanes
// lanes a head), so a warp step covers 4 (bf16) or 2 (fp32) heads; two steps
// of each side are in flight.  Bound by memory: 43,758 rows of 16 + 16 heads in
// fp32 take 110.6 us (6.5 TB/s); 7,829 rows in bf16, 1.6 warps for every one that
// fits, 16.5 us cold (3.9 TB/s, issue slots 54 % busy).
//
// The angle of position p and frequency f (in turns, f / 2 pi) is p f mod 1.
// f is held as a 64-bit binary fraction F, so that the low 64 bits of p F are
// the angle to p times F's own error (2^-63 at most), below 2^-32 of a turn at any
// position; its top 32 bits count.  What is left of it beside the nearest quarter
// turn goes to sincospi, as fp32: 24 bits of at most an eighth of a turn, to
// 2^-28.  (The whole angle as fp32 was off by 2^-26.)  The row's angles are
// computed once, one per lane, for all heads.
//
// (y_a, y_b) = r (w_a x_a, w_b x_b) rotated by (c, s): each lane keeps its
// dimensions' own factors c w and their partners' -+ s w, so that an element
// costs two products and a multiply-add besides the sum of squares, two
// elements at a time (f32x2).  Where the partner is:
//   kWhole  pairs (i, i + 32): a lane loads 8 bytes of each half of the head,
//           so that pairs meet in it
//   kPart   pairs (i, i + r/2) of r < 64 rotated dimensions: 16 bytes a lane,
//           partners from another lane by shuffles
//   kNext   pairs (2 i, 2 i + 1): 16 bytes a lane
enum RopePairs { kWhole, kPart, kNext };
constexpr int kRopeWarps = 4;
// CTAs on an SM: 32 warps of 64 registers, with two steps of each side in
// flight.  For 7,829 rows of 16 + 16 heads (bf16) 16.6 us; 18.4 us with four
// steps, or with 24 warps.  A warp that runs on to further rows, loading the
// next one's first steps ahead, took 24 us.
constexpr int kRopeCtas = 8;

template <typename T>
struct Lane16;   // 16 bytes of a row as pairs of fp32
template <>
struct Lane16<float> {
  static constexpr int kVec = 4;
  static __device__ __forceinline__ void unpack(const uint4& a, uint64_t (&x)[2]) {
    x[0] = f32x2(__uint_as_float(a.x), __uint_as_float(a.y));
    x[1] = f32x2(__uint_as_float(a.z), __uint_as_float(a.w));
  }
  static __device__ __forceinline__ uint4 pack(const uint64_t (&x)[2]) {
    float a, b, c, d;
    f32x2_split(x[0], a, b);
    f32x2_split(x[1], c, d);
    return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
  }
};
template <>
struct Lane16<__nv_bfloat16> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ void unpack(const uint4& a, uint64_t (&x)[4]) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = f32x2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ uint4 pack(const uint64_t (&x)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      f32x2_split(x[i], lo, hi);
      w[i] = pack_bf16x2(lo, hi);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Two neighbouring weights (of an even index).
__device__ __forceinline__ float2 load_weights(const void* p, bool f32, int at) {
  if (p == nullptr) return make_float2(1.f, 1.f);
  if (f32) return __ldg(reinterpret_cast<const float2*>(static_cast<const float*>(p) + at));
  const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p) + at));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

template <typename T, RopePairs kPairs>
__global__ void __launch_bounds__(32 * kRopeWarps, kRopeCtas)
qk_norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  using L = Lane16<T>;
  constexpr int kVec = L::kVec, kHalfVec = kVec / 2;
  constexpr int kLanes = kHeadDim / kVec;      // lanes a head
  constexpr int kHeads = 32 / kLanes;          // heads a warp step
  constexpr int kSteps = 2;                    // steps in flight, of each side
  __shared__ float2 table[kRopeWarps][kHeadDim / 2];   // cos, sin of the row's angles
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRopeWarps + warp;
  if (t >= a.rows) return;                     // (warps do not wait for one another)
  const int pos = __ldg(a.positions + t);
  if (pos < 0) return;                         // a row in no sequence
  const int half = a.rotary >> 1;
  const int l = lane % kLanes, sub = lane / kLanes;
  // This lane's values: kVec of them from d0 on, or (kWhole) kHalfVec from d0
  // and from d0 + 32 on.
  const int d0 = kPairs == kWhole ? l * kHalfVec : l * kVec;

  auto load = [&](const T* row, int heads, int step) -> uint4 {
    const int head = step * kHeads + sub;
    if (head >= heads) return make_uint4(0u, 0u, 0u, 0u);
    const T* p = row + head * kHeadDim + d0;
    if (kPairs != kWhole) return *reinterpret_cast<const uint4*>(p);
    const uint2 lo = *reinterpret_cast<const uint2*>(p), hi = *reinterpret_cast<const uint2*>(p + kHeadDim / 2);
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
  };
  const T* row_q = static_cast<const T*>(a.q.in) + t * a.q.in_stride;
  const T* row_k = static_cast<const T*>(a.k.in) + t * a.k.in_stride;
  uint4 raw_q[kSteps], raw_k[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) raw_q[i] = load(row_q, a.q.heads, i);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) raw_k[i] = load(row_k, a.k.heads, i);

  if (lane < half) {
    const uint64_t turn = a.freq[lane] * static_cast<uint64_t>(pos);
    const uint32_t angle = static_cast<uint32_t>(turn >> 32);
    const uint32_t quarters = (angle + 0x20000000u) >> 30;
    const float x = static_cast<float>(static_cast<int32_t>(angle - (quarters << 30))) * 0x1p-31f;   // half turns
    float c, s;
    sincospif(x, &s, &c);
    if (quarters & 1) {   // a quarter turn further: (c, s) -> (-s, c)
      const float c0 = c;
      c = -s;
      s = c0;
    }
    if (quarters & 2) {
      c = -c;
      s = -s;
    }
    table[warp][lane] = make_float2(c, s);
  }
  __syncwarp();
  const bool rotated = kPairs == kWhole || d0 < a.rotary;
  const bool upper = kPairs == kPart && d0 >= half;
  // kPart: the lane with the partners, and their first dimension.
  const int away = kPairs == kPart && rotated ? (upper ? -half : half) : 0;
  const int partner = lane + away / kVec;

  auto run_side = [&](const RopeArgs::Side& side, const T* row, uint4 (&raw)[kSteps]) {
    uint64_t own[kHalfVec], other[kHalfVec];   // by pairs of values
    auto factors = [&](int w0) {
#pragma unroll
      for (int e = 0; e < kVec; e += 2) {
        if (kPairs == kNext) {
          const float2 w = load_weights(side.weight, a.weight_f32, w0 + d0 + e);
          const float2 cs = rotated ? table[warp][(d0 + e) >> 1] : make_float2(1.f, 0.f);
          own[e / 2] = f32x2(cs.x * w.x, cs.x * w.y);
          other[e / 2] = f32x2(-cs.y * w.y, cs.y * w.x);
        } else {
          const bool second = kPairs == kWhole ? e >= kHalfVec : upper;
          const int d = kPairs == kWhole ? d0 + e % kHalfVec + (second ? kHeadDim / 2 : 0) : d0 + e;
          const int pd = kPairs == kWhole ? (second ? d - kHeadDim / 2 : d + kHeadDim / 2) : d + away;
          const float2 w = load_weights(side.weight, a.weight_f32, w0 + d), pw = load_weights(side.weight, a.weight_f32, w0 + pd);
          const int f = second ? pd : d;
          const float2 cs0 = rotated ? table[warp][f] : make_float2(1.f, 0.f);
          const float2 cs1 = rotated ? table[warp][f + 1] : make_float2(1.f, 0.f);
          own[e / 2] = f32x2(cs0.x * w.x, cs1.x * w.y);
          other[e / 2] = second ? f32x2(cs0.y * pw.x, cs1.y * pw.y) : f32x2(-cs0.y * pw.x, -cs1.y * pw.y);
        }
      }
    };
    if (side.w_stride == 0) factors(0);
    T* out = static_cast<T*>(side.out) + t * side.out_stride;
    const int heads = side.heads;
    const int steps = (heads + kHeads - 1) / kHeads;
    for (int s0 = 0; s0 < steps; s0 += kSteps) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        if (s0 + i >= steps) break;
        const int head = (s0 + i) * kHeads + sub;
        if (side.w_stride != 0) factors((head < heads ? head : 0) * side.w_stride);
        const uint4 mine = raw[i];
        raw[i] = load(row, heads, s0 + i + kSteps);
        uint64_t x[kHalfVec], z[kHalfVec];
        L::unpack(mine, x);
        if (kPairs == kPart) {
          const uint4 theirs = make_uint4(__shfl_sync(0xffffffffu, mine.x, partner), __shfl_sync(0xffffffffu, mine.y, partner),
                                          __shfl_sync(0xffffffffu, mine.z, partner), __shfl_sync(0xffffffffu, mine.w, partner));
          L::unpack(theirs, z);
        } else {
#pragma unroll
          for (int e = 0; e < kHalfVec; ++e) {
            if (kPairs == kWhole) {
              z[e] = x[(e + kHalfVec / 2) % kHalfVec];
            } else {
              float lo, hi;
              f32x2_split(x[e], lo, hi);
              z[e] = f32x2(hi, lo);
            }
          }
        }
        uint64_t ss2 = mul_f32x2(x[0], x[0]);
#pragma unroll
        for (int e = 1; e < kHalfVec; ++e) ss2 = fma_f32x2(x[e], x[e], ss2);
        float ss, hi;
        f32x2_split(ss2, ss, hi);
        ss += hi;
#pragma unroll
        for (int m = kLanes / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        const float r = rsqrtf(fmaf(ss, 1.f / kHeadDim, a.eps));
        const uint64_t r2 = f32x2(r, r);
#pragma unroll
        for (int e = 0; e < kHalfVec; ++e) {
          uint64_t y = mul_f32x2(x[e], own[e]);
          if (rotated) y = fma_f32x2(z[e], other[e], y);   // (a partner's infinity stays out of dimensions that have none)
          x[e] = mul_f32x2(y, r2);
        }
        if (head < heads) {
          const uint4 y = L::pack(x);
          T* p = out + head * kHeadDim + d0;
          if (kPairs == kWhole) {
            *reinterpret_cast<uint2*>(p) = make_uint2(y.x, y.y);
            *reinterpret_cast<uint2*>(p + kHeadDim / 2) = make_uint2(y.z, y.w);
          } else {
            *reinterpret_cast<uint4*>(p) = y;
          }
        }
      }
    }
  };
  run_side(a.q, row_q, raw_q);
  run_side(a.k, row_k, raw_k);
}

template <typename T>
void run_rope(const RopeArgs& a, bool interleaved, unsigned grid, cudaStream_t stream) {
  if (interleaved) qk_norm_rope_kernel<T, kNext><<<grid, 32 * kRopeWarps, 0, stream>>>(a);
  else if (a.rotary == kHeadDim) qk_norm_rope_kernel<T, kWhole><<<grid, 32 * kRopeWarps, 0, stream>>>(a);
  else qk_norm_rope_kernel<T, kPart><<<grid, 32 * kRopeWarps, 0, stream>>>(a);
}

}  // namespace

cudaError_t launch_decay_step(const StepArgs& a, cudaStream_t stream) {
  // The indices ride in the launch's parameters, so that the host array is
  // read during the call only and nothing is copied; a longer batch takes a
  // launch per kStepMostSlots rows.
  for (int64_t t0 = 0; t0 < a.n;) {
    const int64_t most = a.index != nullptr ? kStepMostSlots : (INT64_C(1) << 30) / a.H;
    const int64_t n = a.n - t0 < most ? a.n - t0 : most;
    cudaError_t e;
    if (a.index == nullptr) {
      e = a.f32 ? step_chunk<float, 0>(a, t0, n, stream) : step_chunk<__nv_bfloat16, 0>(a, t0, n, stream);
    } else if (n <= kStepFewSlots) {
      e = a.f32 ? step_chunk<float, kStepFewSlots>(a, t0, n, stream)
                : step_chunk<__nv_bfloat16, kStepFewSlots>(a, t0, n, stream);
    } else if (n <= kStepManySlots) {
      e = a.f32 ? step_chunk<float, kStepManySlots>(a, t0, n, stream)
                : step_chunk<__nv_bfloat16, kStepManySlots>(a, t0, n, stream);
    } else {
      e = a.f32 ? step_chunk<float, kStepMostSlots>(a, t0, n, stream)
                : step_chunk<__nv_bfloat16, kStepMostSlots>(a, t0, n, stream);
    }
    if (e != cudaSuccess) return e;
    t0 += n;
  }
  return cudaSuccess;
}

cudaError_t launch_qk_norm_rope(const RopeArgs& a, bool f32, bool interleaved, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((a.rows + kRopeWarps - 1) / kRopeWarps);
  if (f32) run_rope<float>(a, interleaved, grid, stream);
  else run_rope<__nv_bfloat16>(a, interleaved, grid, stream);
  return cudaGetLastError();
}

}  // namespace spanla
