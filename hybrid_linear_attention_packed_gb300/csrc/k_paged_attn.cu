// Softmax attention of packed rows over the paged cache of keys and values.
#include "paged.cuh"

namespace spanla {
namespace {

constexpr int kRowWarps = 4;

template <bool kE4m3>
__global__ void __launch_bounds__(kRowWarps * 32) paged_rows_kernel(const __grid_constant__ KvArgs a,
                                                                    const __grid_constant__ PagedAttn p) {
  if (blockIdx.x == 0 && blockIdx.y == 0) check_sequences(a);
  const int64_t t = blockIdx.x;
  const int s = seq_of_row(a, t);
  if (s < 0) return;
  bool bad = false;
  const SeqRows r = seq_rows(a, s, &bad);
  const int64_t i = t - r.row0;
  if (i < 0 || i >= r.n || static_cast<int64_t>(r.n) * p.group <= kStepHeads) return;
  const int32_t seen = max(0, static_cast<int32_t>(r.len - r.n + i + 1));
  const int head = blockIdx.y * kRowWarps + (threadIdx.x >> 5);
  if (head < p.heads) attend_row<kE4m3>(a, p, s, t, head, seen);
}

}  // namespace

cudaError_t launch_paged_rows(const KvArgs& a, const PagedAttn& p, bool e4m3, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.rows), (p.heads + kRowWarps - 1) / kRowWarps);
  (e4m3 ? paged_rows_kernel<true> : paged_rows_kernel<false>)<<<grid, kRowWarps * 32, 0, stream>>>(a, p);
  return cudaGetLastError();
}

}  // namespace spanla
