// Device pieces of the span kernels.  k_span_output.cu and k_span_decay.cu
// share waits that flag their timeouts, inline segment starts, state slices to
// global memory and to the shared-memory S operand, and the counter's load; the
// parts of a WorkTile that each role reads are k_span_output.cu's
// (k_span_decay.cu's DecayTile has its own).
#pragma once

#include "spanla_internal.h"
#include "tc_ptx.cuh"

namespace spanla {

__device__ __forceinline__ bool wait_or_flag(uint32_t bar, uint32_t parity, unsigned* err,
                                             unsigned code) {
  if (mbar_wait_bounded(bar, parity, kWaitLimitNs)) return true;
  atomicOr(err, code);
  return false;
}

// The parts of a tile record each role reads (fewer registers per role).
struct TileHead {     // row0, nrows, head, flags
  int32_t row0, nrows, head, flags;
};
struct TileState {    // ... and the start-state recipe
  int32_t row0, nrows, head, flags, stateA, stateB, a_n, b_n, final_idx;
};
struct TileMask {     // rows and segment starts (P conversion)
  int32_t nrows, bound0, nbound;
  uint4 inl;
};

__device__ __forceinline__ TileHead load_head(const WorkTile* p) {
  const int4 a = __ldg(reinterpret_cast<const int4*>(p));
  return TileHead{a.x, a.y, a.z, a.w};
}

__device__ __forceinline__ TileState load_state(const WorkTile* p) {
  const int4 a = __ldg(reinterpret_cast<const int4*>(p));
  const int4 b = __ldg(reinterpret_cast<const int4*>(p) + 1);
  const int32_t f = __ldg(&p->final_idx);
  return TileState{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, f};
}

__device__ __forceinline__ TileMask load_mask(const WorkTile* p) {
  const int4 c = __ldg(reinterpret_cast<const int4*>(p) + 2);
  const uint4 d = __ldg(reinterpret_cast<const uint4*>(p) + 3);
  return TileMask{__ldg(&p->nrows), c.y, c.z, d};
}

__device__ __forceinline__ int inline_bound(const uint4& v, int q) {
  const uint32_t w = q < 4 ? v.x : q < 8 ? v.y : q < 12 ? v.z : v.w;
  return static_cast<int>((w >> (8 * (q & 3))) & 0xffu);
}

// Write 16 state values (columns col0 ..) of row d, rounded to bf16, into
// the MN-major S operand ([d][64 e], 128-byte swizzle).  (The state itself
// stays fp32; only its product with Q takes the rounded copy, whose entries
// are off by less than 2^-9 of their value, as q, k and v are.)
__device__ __forceinline__ void stage_state_slice(uint8_t* s_op, int d, int col0, const float* x) {
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    uint32_t b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) b[u] = pack_bf16x2(x[8 * g + 2 * u], x[8 * g + 2 * u + 1]);
    *reinterpret_cast<uint4*>(s_op + sw128_offset(d, col0 + 8 * g)) = make_uint4(b[0], b[1], b[2], b[3]);
  }
}

// 16 fp32 values (one thread's slice of a state row) to global memory.
__device__ __forceinline__ void store_slice(float* dst, const float* x) {
  float4* d4 = reinterpret_cast<float4*>(dst);
#pragma unroll
  for (int c = 0; c < 4; ++c) d4[c] = make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
}

__device__ __forceinline__ unsigned ld_acquire_gpu(const unsigned* p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

}  // namespace spanla
