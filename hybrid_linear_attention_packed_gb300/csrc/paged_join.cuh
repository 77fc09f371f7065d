// What the step kernel's parts of items look like, and how they are joined: by a
// kernel of its own, or by some CTAs of the chunk kernel's join.
#pragma once

#include "paged.cuh"

namespace spanla {

constexpr int kM = kStepHeads;            // row heads of an item, at most
constexpr int kSlotStride = 72;           // floats from row head to row head of a part (72: no bank conflicts)

// A part of an item: [kM][72] floats of O, then m, M, l of kM row heads.
constexpr int kSlotFloats = kM * kSlotStride + 3 * kM;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The weights of a row head are relative to 2^m, its O to 2^(M - 15) (bf16 pages: 2^m): o = O 2^(M - 15 - m) / l.
// In two factors, 2^-15 / l and 2^(M - m), as their product need not be an fp32 number where V is small.
struct OutFactor {
  float a, b;
  __device__ __forceinline__ float operator()(float o) const { return o * a * b; }
};
template <bool kE4m3>
__device__ __forceinline__ OutFactor out_factor(float m, float M, float l) {
  if (l == 0.f) return {0.f, 0.f};
  return {(kE4m3 ? 0x1p-15f : 1.f) / l, kE4m3 ? exp2f(M - m) : 1.f};
}
__device__ __forceinline__ float log_sum(float m, float l) { return l == 0.f ? -INFINITY : fmaf(m, 0.6931471805599453f, logf(l)); }

// 2^(from - to), 0 where nothing is relative to `from`.
__device__ __forceinline__ float rescale(float from, float to) { return from == to ? 1.f : from == -INFINITY ? 0.f : ex2(from - to); }

// A CTA: the row heads that a CTA of the step kernel has marked, in items of its own.  (On CTAs of their own, and not
// beside a join, whose latency counts: one token 12.6 us then, instead of 11.4.)
template <bool kE4m3>
__device__ __forceinline__ void redo_step_items(const KvArgs& a, const PagedAttn& p, const float* ws) {
  const StepRedo* marks = reinterpret_cast<const StepRedo*>(ws + static_cast<int64_t>(blockIdx.x) * kStepWsFloats + 2 * kSlotFloats +
                                                            sizeof(StepJoin) / 4);
  StepRedo x = marks[threadIdx.x & (kStepMostWarps - 1)];
#pragma unroll
  for (int d = kStepMostWarps / 2; d > 0; d >>= 1) {
    x.first = min(x.first, static_cast<int64_t>(__shfl_xor_sync(0xffffffffu, x.first, d)));
    x.last = max(x.last, static_cast<int64_t>(__shfl_xor_sync(0xffffffffu, x.last, d)));
  }
  const int lane = threadIdx.x & 31;
  if (x.last < 0) return;   // (first is no item then)
  for (int64_t it = x.first + (threadIdx.x >> 5); it <= x.last; it += blockDim.x >> 5) {
    const int s = static_cast<int>(it / a.heads), h = static_cast<int>(it % a.heads);
    bool bad = false;
    const SeqRows r = seq_rows(a, s, &bad);
    const int64_t mh = static_cast<int64_t>(r.n) * p.group;
    if (mh > kM) continue;
    uint32_t which = 0;
    for (int i = 0; i < kM; i += 4) {
      const int row = i + (lane >> 3);
      bool mark = false;
      if (row < mh) {
        const uint4 o = *reinterpret_cast<const uint4*>(p.out + ((r.row0 + row / p.group) * p.heads + h * p.group + row % p.group) * kHeadDim +
                                                        8 * (lane & 7));
        mark = has_mark(o.x) || has_mark(o.y) || has_mark(o.z) || has_mark(o.w);
      }
      const uint32_t lanes = __ballot_sync(0xffffffffu, mark);
      for (int g = 0; g < 4; ++g)
        if ((lanes >> (8 * g)) & 0xffu) which |= 1u << (i + g);
    }
    if (which != 0) redo_rows<kE4m3>(a, p, which, s, h, r.row0, 0, r.len - r.n + 1);
  }
}

// CTA (c, y): row heads 4 y .. 4 y + 3 of the item that begins in CTA c of the step kernel and goes on, from the parts of
// it and the next CTAs.  Groups of 16 lanes: group (row, slice) has every kJoinSlices-th part of a row head, a lane four
// elements of O; the row heads' maxima and sums are one group's, a lane a part.  What most items need is asked for before
// the record is there that says what they need (the workspace holds all of it, whether or not it is of this item): the
// kernel is three reads one behind the other else, and little more.
constexpr int kJoinEach = kStepMaxGrid / 16, kJoinRows = 4, kJoinAhead = 2;

template <bool kE4m3, int kJoinSlices>
__device__ __forceinline__ void join_step_parts(const KvArgs& a, const PagedAttn& p, const float* ws, int grid, int y) {
  __shared__ float4 so[kJoinRows * kJoinSlices][16];
  __shared__ float factor[kJoinRows][kStepMaxGrid];
  __shared__ float total[kJoinRows][3];
  __shared__ uint32_t wild;
  const float* mine = ws + static_cast<int64_t>(blockIdx.x) * kStepWsFloats;
  const int tid = threadIdx.x, grp = tid >> 4, sub = tid & 15, last = static_cast<int>(grid - 1 - blockIdx.x);
  const int row4 = grp & (kJoinRows - 1), row = kJoinRows * y + row4, slice = grp / kJoinRows;
  auto part_of = [&](int i) { return mine + static_cast<int64_t>(i) * kStepWsFloats + (i == 0 ? kSlotFloats : 0); };
  const StepJoin j = *reinterpret_cast<const StepJoin*>(mine + 2 * kSlotFloats);
  float pm[kJoinEach], pM[kJoinEach], pl[kJoinEach];
  {
    const float* st = part_of(min(sub, last)) + kM * kSlotStride + row;
    pm[0] = st[0], pM[0] = st[kM], pl[0] = st[2 * kM];
  }
  float4 ahead[kJoinAhead];
#pragma unroll
  for (int k = 0; k < kJoinAhead; ++k)
    ahead[k] = *reinterpret_cast<const float4*>(part_of(min(slice + kJoinSlices * k, last)) + row * kSlotStride + 4 * sub);
  const int mh = j.n * p.group;
  if (j.parts == 0 || kJoinRows * y >= mh) return;
  if (tid == 0) wild = 0;
  static_assert(kJoinRows * 16 % 32 == 0, "whole warps have slice 0, as the shuffles below need");
  if (slice == 0) {
    float m = -INFINITY, M = -INFINITY, l = 0.f;
#pragma unroll
    for (int k = 0; k < kJoinEach; ++k) {
      const int i = sub + 16 * k;
      if (i >= j.parts) {
        pm[k] = pM[k] = -INFINITY, pl[k] = 0.f;
      } else if (k > 0) {
        const float* st = part_of(i) + kM * kSlotStride + row;
        pm[k] = st[0], pM[k] = st[kM], pl[k] = st[2 * kM];
      }
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
      if (16 * k >= j.parts) break;
      l += pl[k] * rescale(pm[k], m);
      factor[row4][sub + 16 * k] = rescale(pM[k], M);
    }
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    if (sub == 0) total[row4][0] = m, total[row4][1] = M, total[row4][2] = l;
  }
  __syncthreads();
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float4& x, float f) {
    o.x = fmaf(f, x.x, o.x), o.y = fmaf(f, x.y, o.y), o.z = fmaf(f, x.z, o.z), o.w = fmaf(f, x.w, o.w);
  };
  if (row < mh) {
#pragma unroll
    for (int k = 0; k < kJoinAhead; ++k)
      if (slice + kJoinSlices * k < j.parts) add(ahead[k], factor[row4][slice + kJoinSlices * k]);
#pragma unroll 8
    for (int i = slice + kJoinSlices * kJoinAhead; i < j.parts; i += kJoinSlices)
      add(*reinterpret_cast<const float4*>(part_of(i) + row * kSlotStride + 4 * sub), factor[row4][i]);
  }
  so[grp][sub] = o;
  __syncthreads();
  if (slice == 0 && row < mh) {
#pragma unroll
    for (int i = 1; i < kJoinSlices; ++i) add(so[grp + i * kJoinRows][sub], 1.f);
    const float m = total[row4][0], M = total[row4][1], l = total[row4][2];
    const OutFactor f = out_factor<kE4m3>(m, M, l);
    const int64_t at = (j.row0 + static_cast<int64_t>(row / p.group)) * p.heads + j.h * p.group + row % p.group;
    const float y[4] = {f(o.x), f(o.y), f(o.z), f(o.w)};
    bool w = false;
#pragma unroll
    for (int c = 0; c < 4; ++c) w |= !(fabsf(y[c]) <= 3.4e38f);
    if (w && l == l && l != 0.f) atomicOr(&wild, 1u << row);
    *reinterpret_cast<uint2*>(p.out + at * kHeadDim + 4 * sub) =
        l == 0.f ? make_uint2(0u, 0u) : make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
    if (p.lse != nullptr && sub == 0) p.lse[at] = log_sum(m, l);
  }
  __syncthreads();
  if (wild != 0 && tid < 32) redo_rows<kE4m3>(a, p, wild, j.s, j.h, j.row0, 0, j.len - j.n + 1);
}

}  // namespace spanla
