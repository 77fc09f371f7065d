// Decayed linear attention for fp32 inputs, on CUDA cores:
//
//     S_t = a S_{t-1} + k_t v_t^T        o_t = S_t^T q_t        (a = exp(log_decay[h]))
//
// over pieces of rows of one segment (a view or a branch) and one head.  Three
// launches: the local state of every piece that a later piece or a branch
// needs, a scan that turns those into the state entering each piece (and each
// view's final state), and the output of every piece from its start state.
// Every product and sum is fp32.
//
// Rows come in chunks of 16.  A piece state adds a^(n-1-r) k_r v_r^T to a^n S
// over a chunk of n rows: 4096 multiply-adds a row and head.  An output chunk
// keeps S_r / a^(r+1) instead of S_r, so that the update is one multiply-add
// for each element, k_r / a^(r+1) times v_r, and the output another, a^(r+1)
// times at the end: 8192 a row and head, where the recurrence as written takes
// 12288.  A head with a < e^-1.5, for which a^-16 could leave the fp32 range,
// takes it as written.
//
// One warp per (piece, head): thread (rg, cg) holds rows 16 rg .. and columns
// 4 cg .. and 32 + 4 cg .. of S, 16 x 8, in registers, so that a row costs it 16
// values each of k and q and 8 of v from shared memory for 256 multiply-adds, two
// rows of S at a time (f32x2).  Partial outputs are added over the 4 row groups
// by shuffles (each lane keeps 2 columns).  Rows come by 16-byte asynchronous
// copies, one chunk ahead, and k and v of a row from shared memory while the row
// before it is multiplied.
//
// Bound by the fp32 pipe, not by memory (1 KB a row and head): 7,796 rows of 16
// heads take 91 us (30 us the piece states, 13 the scan, 60 the outputs, their
// ends overlapped), the pipe 52 % busy with the 8 warps that the registers
// of the states leave room for.  With 8 x 8 blocks, two warps a piece and 16 on an
// SM, the loads and sums around the multiply-adds took a third more
// instructions: 111 us, 99 with this block at the same pieces.  Outputs
// interleaved with the update (102), two rows unrolled (106): slower.
#include "decay_math.cuh"
#include "spanla_internal.h"
#include "tc_ptx.cuh"

namespace spanla {
namespace {

constexpr int kThreads = 32;
constexpr int kPairs = 8;      // pairs of rows of S a thread holds
constexpr float kSteepLogDecay = -1.5f;
constexpr int kRows = 16;    // rows of a chunk: eight CTAs' buffers fill the shared memory

// 16 consecutive values as eight pairs.
__device__ __forceinline__ void get_pairs(const float* p, uint64_t (&x)[kPairs]) {
#pragma unroll
  for (int i = 0; i < kPairs; i += 2) {
    const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(p + 2 * i);
    x[i] = a.x; x[i + 1] = a.y;
  }
}
// Columns 4 cg .. 4 cg + 3 of a row and the same of its second half.
__device__ __forceinline__ void get8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + kHeadDim / 2);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
// The same of a state in global memory, from L2: the launch before wrote it, and
// this one may have started during it, so that it is not read-only data.
__device__ __forceinline__ void get8_state(const float* p, float (&x)[8]) {
  const float4 a = __ldcg(reinterpret_cast<const float4*>(p)), b = __ldcg(reinterpret_cast<const float4*>(p + kHeadDim / 2));
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <bool kOut>
struct Smem {
  float row[2][kOut ? 3 : 2][kRows][kHeadDim];            // K, V (and Q) of two chunks
  float up[kRows + 1], down[kRows + 1];                   // a^m and a^-m
};

template <bool kOut>
__global__ void __launch_bounds__(kThreads, kRecurUnitsPerSm)
recur_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
             const RecurUnit* __restrict__ units, int H, const float* __restrict__ log_decay,
             const float* stateA, float* ws, float* __restrict__ out) {
  __shared__ __align__(16) Smem<kOut> sm;
  griddep_launch_dependents();   // (the next launch waits for this one's end before it reads)
  const int h = blockIdx.x % H;
  const RecurUnit u = units[blockIdx.x / H];
  const int tid = threadIdx.x;
  const int rg = tid >> 3, cg = tid & 7;
  const float ld = load_log_decay(log_decay, h);
  const float l2 = decay_log2(ld);
  const Factor f_chunk = decay_factor(ld, static_cast<float>(kRows));   // a^n of a whole chunk
  const bool steep = kOut && ld < kSteepLogDecay;
  const float a1 = decay_pow(l2, 1.f);
  if (tid <= kRows) {   // (read behind the first chunk's barrier)
    sm.up[tid] = decay_pow(l2, static_cast<float>(tid));
    sm.down[tid] = decay_pow(l2, -static_cast<float>(tid));
  }

  const int64_t stride = static_cast<int64_t>(H) * kHeadDim;
  const int64_t base = static_cast<int64_t>(u.row0) * stride + static_cast<int64_t>(h) * kHeadDim;
  constexpr int kPerRow = kHeadDim / 4;             // 16-byte copies of a row
  auto load = [&](int r0, int b) {
    const int n = min(kRows, u.len - r0);
    for (int c = tid; c < n * kPerRow; c += kThreads) {
      const int r = c / kPerRow, x = (c % kPerRow) * 4;
      const int64_t at = base + (r0 + r) * stride + x;
      cp_async16(smem_addr(&sm.row[b][0][r][x]), k + at);
      cp_async16(smem_addr(&sm.row[b][1][r][x]), v + at);
      if (kOut) cp_async16(smem_addr(&sm.row[b][kOut ? 2 : 0][r][x]), q + at);
    }
  };
  load(0, 0);
  cp_async_commit();

  uint64_t S[kPairs][8];   // pairs of rows, 8 columns
#pragma unroll
  for (int i = 0; i < kPairs; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) S[i][j] = 0;
  if (kOut) {
    griddep_wait();   // start states from the scan
    // Start state: the scanned prefix of the segment's earlier rows, plus the
    // parent view's final state decayed over them.
    const int64_t slice = static_cast<int64_t>(2 * kPairs * rg) * kHeadDim + 4 * cg;
    auto add = [&](const float* p, float f) {
      const uint64_t f2 = f32x2(f, f);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        float x[8], y[8];
        get8_state(p + 2 * i * kHeadDim, x);
        get8_state(p + (2 * i + 1) * kHeadDim, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) S[i][j] = fma_f32x2(f32x2(x[j], y[j]), f2, S[i][j]);
      }
    };
    if (u.parent >= 0)
      add(stateA + (static_cast<int64_t>(u.parent) * H + h) * kStateFloats + slice, decay_pow(l2, static_cast<float>(u.before)));
    if (u.slot >= 0) add(ws + (static_cast<int64_t>(u.slot) * H + h) * kStateFloats + slice, 1.f);
  }

  auto decay_state = [&](const Factor f) {
    const uint64_t hi = f32x2(f.hi, f.hi), lo = f32x2(f.lo, f.lo);
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) S[i][j] = fma_f32x2(hi, S[i][j], mul_f32x2(lo, S[i][j]));
  };
  int b = 0;
  for (int r0 = 0; r0 < u.len; r0 += kRows, b ^= 1) {
    const int n = min(kRows, u.len - r0);
    if (r0 + kRows < u.len) load(r0 + kRows, b ^ 1);
    cp_async_commit();
    cp_async_wait<1>();
    __syncwarp();
    const Factor fn = n == kRows ? f_chunk : decay_factor(ld, static_cast<float>(n));
    if (!kOut) decay_state(fn);
    uint64_t kr[kPairs];
    float vr[8], w;
    auto fetch = [&](int r) {
      get_pairs(&sm.row[b][0][r][2 * kPairs * rg], kr);
      get8(&sm.row[b][1][r][4 * cg], vr);
      w = kOut ? sm.down[r + 1] : sm.up[max(n - 1 - r, 0)];
    };
    fetch(0);
    for (int r = 0; r < n; ++r) {
      uint64_t qr[kPairs];
      if (kOut) get_pairs(&sm.row[b][kOut ? 2 : 0][r][2 * kPairs * rg], qr);
      if (steep) {
        const uint64_t a2 = f32x2(a1, a1);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint64_t v2 = f32x2(vr[j], vr[j]);
#pragma unroll
          for (int i = 0; i < kPairs; ++i) S[i][j] = fma_f32x2(a2, S[i][j], mul_f32x2(kr[i], v2));
        }
      } else {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) kr[i] = mul_f32x2(kr[i], f32x2(w, w));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint64_t v2 = f32x2(vr[j], vr[j]);
#pragma unroll
          for (int i = 0; i < kPairs; ++i) S[i][j] = fma_f32x2(kr[i], v2, S[i][j]);
        }
      }
      fetch(min(r + 1, kRows - 1));
      if (kOut) {
        uint64_t o2[8];
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) o2[j] = i == 0 ? mul_f32x2(qr[0], S[0][j]) : fma_f32x2(qr[i], S[i][j], o2[j]);
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float lo, hi;
          f32x2_split(o2[j], lo, hi);
          o[j] = lo + hi;
        }
        // Add over the 4 row groups (lane bits 3 and 4), each step keeping half
        // of the columns.
        const bool up4 = tid & 16, up3 = tid & 8;
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
        const float f = steep ? 1.f : sm.up[r + 1];
        *reinterpret_cast<float2*>(out + base + (r0 + r) * stride + 4 * cg + (up4 ? kHeadDim / 2 : 0) + (up3 ? 2 : 0)) =
            make_float2(y[0] * f, y[1] * f);
      }
    }
    if (kOut && !steep) decay_state(fn);
    __syncwarp();
  }
  if (!kOut) {
    float* p = ws + (static_cast<int64_t>(u.slot) * H + h) * kStateFloats + static_cast<int64_t>(2 * kPairs * rg) * kHeadDim + 4 * cg;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      float x[8], y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f32x2_split(S[i][j], x[j], y[j]);
      float* p0 = p + 2 * i * kHeadDim;
      float* p1 = p0 + kHeadDim;
      *reinterpret_cast<float4*>(p0) = make_float4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<float4*>(p0 + kHeadDim / 2) = make_float4(x[4], x[5], x[6], x[7]);
      *reinterpret_cast<float4*>(p1) = make_float4(y[0], y[1], y[2], y[3]);
      *reinterpret_cast<float4*>(p1 + kHeadDim / 2) = make_float4(y[4], y[5], y[6], y[7]);
    }
  }
}

// The piece states of each segment-head, in order, become the states entering
// the pieces (in place), and their total the view's final state:
// run <- a^len run + piece.  One element a thread, so that a pass of few
// segments still has a state's 4096 chains times its heads in flight, 16 slots
// of loads ahead.  (A float4 a thread, 8 slots ahead: 25 us where this takes
// 10, for 58 slots of 16 heads.)
constexpr int kScanThreads = 256;
constexpr int kScanParts = kStateFloats / kScanThreads;
constexpr int kAhead = 16;

__global__ void __launch_bounds__(kScanThreads)
recur_scan_kernel(const RecurScan* __restrict__ scan, int H, int piece, const float* __restrict__ log_decay,
                  float* __restrict__ ws, float* __restrict__ final_out) {
  griddep_launch_dependents();
  const int part = blockIdx.x % kScanParts;
  const int64_t rest = blockIdx.x / kScanParts;
  const int h = static_cast<int>(rest % H);
  const RecurScan sd = scan[rest / H];
  const int off = part * kScanThreads + threadIdx.x;
  const float ld = load_log_decay(log_decay, h);
  const Factor f = decay_factor(ld, static_cast<float>(piece));
  const Factor f_last = decay_factor(ld, static_cast<float>(sd.last_len));
  float* p = ws + (static_cast<int64_t>(sd.slot0) * H + h) * kStateFloats + off;
  const int64_t stride = static_cast<int64_t>(H) * kStateFloats;
  const int n_read = sd.final_idx >= 0 ? sd.nslots : sd.nslots - 1;   // a branch's last piece has no state of its own
  griddep_wait();   // piece states
  float run = 0.f;
  for (int c0 = 0; c0 < sd.nslots; c0 += kAhead) {
    float x[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (c0 + j < n_read) x[j] = __ldcg(p + (c0 + j) * stride);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int c = c0 + j;
      if (c < sd.nslots) __stcg(p + c * stride, run);
      if (c < n_read) run = (c + 1 < sd.nslots ? f : f_last).step(run, x[j]);
    }
  }
  if (sd.final_idx >= 0) final_out[(static_cast<int64_t>(sd.final_idx) * H + h) * kStateFloats + off] = run;
}

// A launch whose set-up may overlap the end of the kernel before it (`after`:
// there is one in this call).
template <typename... Args>
cudaError_t launch(void (*kernel)(Args...), int64_t grid, int threads, bool after, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_recur_state(const RecurArgs& a, cudaStream_t stream) {
  if (a.n_state <= 0) return cudaSuccess;
  return launch(recur_kernel<false>, a.n_state * a.H, kThreads, false, stream, static_cast<const float*>(nullptr), a.k,
                a.v, a.state_units, a.H, a.log_decay, static_cast<const float*>(nullptr), a.ws, static_cast<float*>(nullptr));
}

cudaError_t launch_recur_scan(const RecurArgs& a, cudaStream_t stream) {
  if (a.n_scan <= 0) return cudaSuccess;
  return launch(recur_scan_kernel, a.n_scan * a.H * kScanParts, kScanThreads, a.n_state > 0, stream, a.scan, a.H, a.piece,
                a.log_decay, a.ws, a.final_out);
}

cudaError_t launch_recur_output(const RecurArgs& a, cudaStream_t stream) {
  if (a.n_out <= 0) return cudaSuccess;
  return launch(recur_kernel<true>, a.n_out * a.H, kThreads, a.n_scan > 0, stream, a.q, a.k, a.v, a.out_units, a.H,
                a.log_decay, a.stateA, a.ws, a.out);
}

}  // namespace spanla
