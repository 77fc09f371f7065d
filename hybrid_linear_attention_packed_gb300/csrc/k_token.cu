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
// store covers two whole rows.
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
  const Factor g = log_decay != nullptr ? decay_factor(load_log_decay(log_decay, h), 1.f) : Factor{1.f, 0.f};
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
// lanes a head), so a warp step covers 256 (bf16) or 128 (fp32) values, all
// its loads in flight before the first is used.
//
// The angle of position p and frequency f (in turns, f / 2 pi) is p f mod 1.
// f is held as a 64-bit binary fraction F, so that the low 64 bits of p F are
// the angle exactly, whatever the position; its top 32 bits go to
// sincospi.  The row's angles are computed once, one per lane, for all heads.
constexpr int kRopeWarps = 4;

template <typename T>
struct Lane16;   // 16 bytes of a row
template <>
struct Lane16<float> {
  static constexpr int kVec = 4;
  static __device__ __forceinline__ void unpack(const uint4& a, float* x) {
    x[0] = __uint_as_float(a.x); x[1] = __uint_as_float(a.y); x[2] = __uint_as_float(a.z); x[3] = __uint_as_float(a.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <>
struct Lane16<__nv_bfloat16> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ void unpack(const uint4& a, float* x) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  }
};

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(32 * kRopeWarps)
qk_norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  using L = Lane16<T>;
  constexpr int kVec = L::kVec;
  constexpr int kLanes = kHeadDim / kVec;      // lanes a head
  constexpr int kHeads = 32 / kLanes;          // heads a warp step
  constexpr int kSteps = 4;                    // steps in flight
  __shared__ float2 table[kRopeWarps][32];     // cos, sin of the row's angles
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRopeWarps + warp;
  if (t >= a.rows) return;                     // (warps do not wait for one another)
  const int pos = __ldg(a.positions + t);
  if (pos < 0) return;                         // a row in no sequence
  const int half = a.rotary >> 1;
  const int l = lane % kLanes, sub = lane / kLanes;
  const int q_steps = (a.q.heads + kHeads - 1) / kHeads, k_steps = (a.k.heads + kHeads - 1) / kHeads;
  const int steps = q_steps + k_steps;

  uint4 raw[kSteps];
  auto load = [&](int s, uint4& x) {
    const bool is_q = s < q_steps;
    const RopeArgs::Side& side = is_q ? a.q : a.k;
    const int head = (is_q ? s : s - q_steps) * kHeads + sub;
    x = make_uint4(0u, 0u, 0u, 0u);
    if (s < steps && head < side.heads)
      x = *reinterpret_cast<const uint4*>(static_cast<const T*>(side.in) + t * side.in_stride + head * kHeadDim + l * kVec);
  };
#pragma unroll
  for (int i = 0; i < kSteps; ++i) load(i, raw[i]);

  if (lane < half) {
    const uint64_t turn = a.freq[lane] * static_cast<uint64_t>(pos);
    const float x = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f;   // half turns: 2^-31
    float c, s;
    sincospif(x, &s, &c);
    table[warp][lane] = make_float2(c, s);
  }
  __syncwarp();
  // This lane's angles: kVec / 2 neighbouring pairs, or kVec dimensions of
  // one half of the rotated part.
  const int d0 = l * kVec;
  const bool rotated = d0 < a.rotary;
  const bool upper = d0 >= half;
  const int partner = lane + (rotated ? (upper ? -(half / kVec) : half / kVec) : 0);
  float c[kVec], s[kVec];
#pragma unroll
  for (int e = 0; e < kVec; ++e) {
    const int f = kInterleaved ? (d0 + e) >> 1 : (upper ? d0 - half : d0) + e;
    const float2 cs = rotated ? table[warp][f] : make_float2(1.f, 0.f);
    c[e] = cs.x;
    s[e] = kInterleaved ? cs.y : (upper ? cs.y : -cs.y);
  }

  for (int s0 = 0; s0 < steps; s0 += kSteps) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int st = s0 + i;
      if (st >= steps) break;
      const bool is_q = st < q_steps;
      const RopeArgs::Side& side = is_q ? a.q : a.k;
      const int head = (is_q ? st : st - q_steps) * kHeads + sub;
      float x[kVec];
      L::unpack(raw[i], x);
      load(st + kSteps, raw[i]);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < kVec; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int m = kLanes / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
      const float r = 1.f / sqrtf(ss * (1.f / kHeadDim) + a.eps);
      const int wo = (head < side.heads ? head : 0) * side.w_stride + d0;
      if (side.weight == nullptr) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) x[e] *= r;
      } else if (a.weight_f32) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) x[e] *= r * __ldg(static_cast<const float*>(side.weight) + wo + e);
      } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e)
          x[e] *= r * __bfloat162float(static_cast<const __nv_bfloat16*>(side.weight)[wo + e]);
      }
      float y[kVec];
      if (kInterleaved) {
#pragma unroll
        for (int e = 0; e < kVec; e += 2) {
          y[e] = x[e] * c[e] - x[e + 1] * s[e];
          y[e + 1] = x[e + 1] * c[e] + x[e] * s[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const float other = __shfl_sync(0xffffffffu, x[e], partner);
          y[e] = rotated ? fmaf(other, s[e], x[e] * c[e]) : x[e];
        }
      }
      if (head < side.heads)
        *reinterpret_cast<uint4*>(static_cast<T*>(side.out) + t * side.out_stride + head * kHeadDim + d0) = L::pack(y);
    }
  }
}

}  // namespace

cudaError_t launch_decay_step(const StepArgs& a, cudaStream_t stream) {
  // The indices ride in the launch's parameters (up to 4 KB), so that the
  // host array is read during the call only and nothing is copied; a longer
  // batch takes a launch per kStepMostSlots rows.
  for (int64_t t0 = 0; t0 < a.n;) {
    const int64_t most = a.index != nullptr ? kStepMostSlots : (INT64_C(1) << 30) / a.H;
    const int64_t n = a.n - t0 < most ? a.n - t0 : most;
    cudaError_t e;
    if (a.index == nullptr) {
      e = a.f32 ? step_chunk<float, 0>(a, t0, n, stream) : step_chunk<__nv_bfloat16, 0>(a, t0, n, stream);
    } else if (n <= kStepFewSlots) {
      e = a.f32 ? step_chunk<float, kStepFewSlots>(a, t0, n, stream)
                : step_chunk<__nv_bfloat16, kStepFewSlots>(a, t0, n, stream);
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
  if (f32) {
    if (interleaved) qk_norm_rope_kernel<float, true><<<grid, 32 * kRopeWarps, 0, stream>>>(a);
    else qk_norm_rope_kernel<float, false><<<grid, 32 * kRopeWarps, 0, stream>>>(a);
  } else {
    if (interleaved) qk_norm_rope_kernel<__nv_bfloat16, true><<<grid, 32 * kRopeWarps, 0, stream>>>(a);
    else qk_norm_rope_kernel<__nv_bfloat16, false><<<grid, 32 * kRopeWarps, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace spanla
