// Decayed linear attention by the recurrence itself, on CUDA cores:
//
//     S_t = a S_{t-1} + k_t v_t^T        o_t = S_t^T q_t        (a = exp(log_decay[h]))
//
// over pieces of rows of one segment (a view or a branch) and one head.  Three
// launches: the local state of every piece that a later piece or a branch
// needs, a scan that turns those into the state entering each piece (and each
// view's final state), and the output of every piece from its start state.
//
// The recurrence needs 3 * 4096 operations a row and head for the output
// (k_i v_j, a S + that, q_i S) and 2 * 4096 for a piece state, all in fp32:
// results are exact to fp32 roundings.  It is bound by the fp32 pipe, not by
// memory (1 KB a row and head in fp32).
//
// One CTA of 64 threads per (piece, head): thread (rg, cg) holds the 8 x 8
// block of S at rows 8 rg, columns 8 cg in registers, so that a row costs it
// 8 values of q and of k and 8 of v from shared memory for 192 operations.
// Partial outputs are added over the 8 row groups: 4 inside a warp by
// shuffles (each lane keeps 2 columns), 2 across the warps through shared
// memory.  Rows come in chunks of 16 by 16-byte asynchronous copies, one
// chunk ahead.
#include <cuda_bf16.h>

#include "decay_math.cuh"
#include "spanla_internal.h"
#include "tc_ptx.cuh"

namespace spanla {
namespace {

constexpr int kThreads = 64;
constexpr int kRows = 16;    // rows of a chunk

template <typename T>
struct Row8;   // 8 consecutive values of a row in shared memory, as fp32
template <>
struct Row8<float> {
  static __device__ __forceinline__ void get(const float* p, float* x) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};
template <>
struct Row8<__nv_bfloat16> {
  static __device__ __forceinline__ void get(const __nv_bfloat16* p, float* x) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void store_out(float* p, float a, float b) {
  *reinterpret_cast<float2*>(p) = make_float2(a, b);
}
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float a, float b) {
  *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(a, b);
}

template <typename T, bool kOut>
struct Smem {
  T row[2][kOut ? 3 : 2][kRows][kHeadDim];   // K, V (and Q) of two chunks
  float part[kOut ? 2 : 1][kOut ? kRows : 1][kHeadDim];   // a warp's partial outputs
};

template <typename T, bool kOut>
__global__ void __launch_bounds__(kThreads)
recur_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
             const RecurUnit* __restrict__ units, int H, const float* __restrict__ log_decay,
             const float* __restrict__ stateA, float* __restrict__ ws, T* __restrict__ out) {
  __shared__ __align__(16) Smem<T, kOut> sm;
  const int h = blockIdx.x % H;
  const RecurUnit u = units[blockIdx.x / H];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rg = tid >> 3, cg = tid & 7;
  const float ld = load_log_decay(log_decay, h);
  // a is rounded, which a state that remembers 1 / (1 - a) rows would collect
  // that often: every chunk's end makes up for its rows.
  const Factor f1 = decay_factor(ld, 1.f);
  const float a = f1.hi;
  const float eps = f1.lo != 0.f ? f1.lo / f1.hi : 0.f;

  const int64_t stride = static_cast<int64_t>(H) * kHeadDim;
  const int64_t base = static_cast<int64_t>(u.row0) * stride + static_cast<int64_t>(h) * kHeadDim;
  constexpr int kVec = 16 / sizeof(T);              // values of one copy
  constexpr int kPerRow = kHeadDim / kVec;
  auto load = [&](int r0, int b) {
    const int n = min(kRows, u.len - r0);
    for (int c = tid; c < n * kPerRow; c += kThreads) {
      const int r = c / kPerRow, x = (c % kPerRow) * kVec;
      const int64_t at = base + (r0 + r) * stride + x;
      cp_async16(smem_addr(&sm.row[b][0][r][x]), k + at);
      cp_async16(smem_addr(&sm.row[b][1][r][x]), v + at);
      if (kOut) cp_async16(smem_addr(&sm.row[b][kOut ? 2 : 0][r][x]), q + at);
    }
  };
  load(0, 0);
  cp_async_commit();

  float S[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) S[i][j] = 0.f;
  if (kOut) {
    // Start state: the scanned prefix of the segment's earlier rows, plus the
    // parent view's final state decayed over them.
    const int64_t slice = static_cast<int64_t>(8 * rg) * kHeadDim + 8 * cg;
    if (u.parent >= 0) {
      const float f = decay_pow(decay_log2(ld), static_cast<float>(u.before));
      const float* p = stateA + (static_cast<int64_t>(u.parent) * H + h) * kStateFloats + slice;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        Row8<float>::get(p + i * kHeadDim, S[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) S[i][j] *= f;
      }
    }
    if (u.slot >= 0) {
      const float* p = ws + (static_cast<int64_t>(u.slot) * H + h) * kStateFloats + slice;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float x[8];
        Row8<float>::get(p + i * kHeadDim, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) S[i][j] += x[j];
      }
    }
  }

  int b = 0;
  for (int r0 = 0; r0 < u.len; r0 += kRows, b ^= 1) {
    const int n = min(kRows, u.len - r0);
    if (r0 + kRows < u.len) load(r0 + kRows, b ^ 1);
    cp_async_commit();
    cp_async_wait<1>();
    __syncthreads();
    for (int r = 0; r < n; ++r) {
      float kr[8], vr[8];
      Row8<T>::get(&sm.row[b][0][r][8 * rg], kr);
      Row8<T>::get(&sm.row[b][1][r][8 * cg], vr);
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) S[i][j] = fmaf(a, S[i][j], kr[i] * vr[j]);
      if (kOut) {
        float qr[8], o[8];
        Row8<T>::get(&sm.row[b][kOut ? 2 : 0][r][8 * rg], qr);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = qr[0] * S[0][j];
#pragma unroll
        for (int i = 1; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = fmaf(qr[i], S[i][j], o[j]);
        // Add over the warp's 4 row groups (lane bits 3 and 4), each step
        // keeping half of the columns.
        const bool up4 = lane & 16, up3 = lane & 8;
        float x[4], y[2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float give = up4 ? o[j] : o[4 + j];
          x[j] = (up4 ? o[4 + j] : o[j]) + __shfl_xor_sync(0xffffffffu, give, 16);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float give = up3 ? x[j] : x[2 + j];
          y[j] = (up3 ? x[2 + j] : x[j]) + __shfl_xor_sync(0xffffffffu, give, 8);
        }
        *reinterpret_cast<float2*>(&sm.part[kOut ? warp : 0][kOut ? r : 0][8 * cg + (up4 ? 4 : 0) + (up3 ? 2 : 0)]) =
            make_float2(y[0], y[1]);
      }
    }
    const float back = eps * static_cast<float>(n);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) S[i][j] = fmaf(back, S[i][j], S[i][j]);
    __syncthreads();
    if (kOut) {
      for (int c = tid; c < n * (kHeadDim / 2); c += kThreads) {
        const int r = c / (kHeadDim / 2), x = 2 * (c % (kHeadDim / 2));
        store_out(out + base + (r0 + r) * stride + x, sm.part[0][kOut ? r : 0][x] + sm.part[kOut ? 1 : 0][kOut ? r : 0][x],
                  sm.part[0][kOut ? r : 0][x + 1] + sm.part[kOut ? 1 : 0][kOut ? r : 0][x + 1]);
      }
      // (The next chunk's partial outputs are written behind its barrier.)
    }
  }
  if (!kOut) {
    float* p = ws + (static_cast<int64_t>(u.slot) * H + h) * kStateFloats + static_cast<int64_t>(8 * rg) * kHeadDim + 8 * cg;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      *reinterpret_cast<float4*>(p + i * kHeadDim) = make_float4(S[i][0], S[i][1], S[i][2], S[i][3]);
      *reinterpret_cast<float4*>(p + i * kHeadDim + 4) = make_float4(S[i][4], S[i][5], S[i][6], S[i][7]);
    }
  }
}

// The piece states of each segment-head, in order, become the states entering
// the pieces (in place), and their total the view's final state:
// run <- a^len run + piece.  256 threads take one float4 of a quarter of a
// state each, 8 slots of loads ahead.
constexpr int kScanThreads = 256;
constexpr int kScanParts = kStateFloats / (4 * kScanThreads);
constexpr int kAhead = 8;

__global__ void __launch_bounds__(kScanThreads)
recur_scan_kernel(const RecurScan* __restrict__ scan, int H, int piece, const float* __restrict__ log_decay,
                  float* __restrict__ ws, float* __restrict__ final_out) {
  const int part = blockIdx.x % kScanParts;
  const int64_t rest = blockIdx.x / kScanParts;
  const int h = static_cast<int>(rest % H);
  const RecurScan sd = scan[rest / H];
  const int off = (part * kScanThreads + threadIdx.x) * 4;
  const float ld = load_log_decay(log_decay, h);
  const Factor f = decay_factor(ld, static_cast<float>(piece));
  const Factor f_last = decay_factor(ld, static_cast<float>(sd.last_len));
  float* p = ws + (static_cast<int64_t>(sd.slot0) * H + h) * kStateFloats + off;
  const int64_t stride = static_cast<int64_t>(H) * kStateFloats;
  const int n_read = sd.final_idx >= 0 ? sd.nslots : sd.nslots - 1;   // a branch's last piece has no state of its own
  float4 run = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c0 = 0; c0 < sd.nslots; c0 += kAhead) {
    float4 x[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (c0 + j < n_read) x[j] = *reinterpret_cast<const float4*>(p + (c0 + j) * stride);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int c = c0 + j;
      if (c < sd.nslots) *reinterpret_cast<float4*>(p + c * stride) = run;
      if (c < n_read) {
        const Factor g = c + 1 < sd.nslots ? f : f_last;
        run.x = g.step(run.x, x[j].x);
        run.y = g.step(run.y, x[j].y);
        run.z = g.step(run.z, x[j].z);
        run.w = g.step(run.w, x[j].w);
      }
    }
  }
  if (sd.final_idx >= 0)
    *reinterpret_cast<float4*>(final_out + (static_cast<int64_t>(sd.final_idx) * H + h) * kStateFloats + off) = run;
}

template <typename T>
cudaError_t recur_state(const RecurArgs& a, cudaStream_t stream) {
  recur_kernel<T, false><<<static_cast<unsigned>(a.n_state * a.H), kThreads, 0, stream>>>(
      nullptr, static_cast<const T*>(a.k), static_cast<const T*>(a.v), a.state_units, a.H, a.log_decay, nullptr, a.ws,
      nullptr);
  return cudaGetLastError();
}

template <typename T>
cudaError_t recur_output(const RecurArgs& a, cudaStream_t stream) {
  recur_kernel<T, true><<<static_cast<unsigned>(a.n_out * a.H), kThreads, 0, stream>>>(
      static_cast<const T*>(a.q), static_cast<const T*>(a.k), static_cast<const T*>(a.v), a.out_units, a.H, a.log_decay,
      a.stateA, a.ws, static_cast<T*>(a.out));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_recur_state(const RecurArgs& a, cudaStream_t stream) {
  if (a.n_state <= 0) return cudaSuccess;
  return a.f32 ? recur_state<float>(a, stream) : recur_state<__nv_bfloat16>(a, stream);
}

cudaError_t launch_recur_scan(const RecurArgs& a, cudaStream_t stream) {
  if (a.n_scan <= 0) return cudaSuccess;
  recur_scan_kernel<<<static_cast<unsigned>(a.n_scan * a.H * kScanParts), kScanThreads, 0, stream>>>(
      a.scan, a.H, a.piece, a.log_decay, a.ws, a.final_out);
  return cudaGetLastError();
}

cudaError_t launch_recur_output(const RecurArgs& a, cudaStream_t stream) {
  if (a.n_out <= 0) return cudaSuccess;
  return a.f32 ? recur_output<float>(a, stream) : recur_output<__nv_bfloat16>(a, stream);
}

}  // namespace spanla
