// Softmax attention of chunks of new rows (more than 16 row heads of a sequence
// and key head) over the paged cache, on the tensor cores (tcgen05).
//
// An item is up to two tiles of 128 row heads of one sequence and key head: rows
// r of the sequence and the `group` query heads of the key head, as row head
// r * group + g, so that grouped heads share the cached rows as consecutive rows
// do.  Per block of 128 cached rows, each tile has
//
//     S = Q K^T                 (M128 N128 K64, fp32 in tensor memory)
//     P = 2^(scale' (S - m))    (bf16, in tensor memory columns of its own)
//     O += P V                  (M128 N64 K128, A = P, in tensor memory over the item's blocks)
//
// with a reference maximum m, raised (and O scaled) only when a row's maximum
// exceeds it by a factor of 2^8 of its weights.  Every row head belongs to one
// thread, which takes its 128 scores into registers at once: the next S is on its
// way while the exponentials are computed, and the other tile's work fills what
// is left.  (Columns of a tile: S 128, P 64, O 64; two tiles are all 512.)
//
// The blocks of all items are numbered through, and every CTA (one an SM) gets
// the same number of consecutive ones, whatever the lengths, which are device
// memory.  An item that goes over several CTAs leaves its parts (m, l, O) in the
// workspace for the join kernel, which starts behind this one.
//
// Measured: 2,048 rows behind 18,000 of 4 key heads of 4, bf16 pages, 169 us, 0.49
// of cuBLAS's rate; 512 rows behind 7,400 of 16 heads 33 us with the launches beside
// it.  A block of two tiles takes 2,450 cycles, of which the products are 1,790: the
// rest is softmax (without exponentials and maxima 131 us) and hand-offs between
// the warps, of which each waits for the one before (without products 161 us).
//
// 12 warps, 16 for e4m3 pages:
//   0      loads, by TMA: Q of each item, K and V of each block, page by page
//   1, 2   issue the products, S and P V
//   3      bf16 pages: zeroes V rows that do not exist (0 times what lies there may be NaN)
//   4-7    softmax of tile 0, a thread a row head; 8-11 of tile 1
//   12-15  e4m3 pages: K and V as they were loaded into bf16 tiles, a thread a row, times its power of two (exact)
#include <algorithm>

#include "paged_join.cuh"

namespace spanla {
namespace {

constexpr uint32_t kTileBytes = kTileRows * 128;      // 128 rows of 64 bf16
constexpr uint32_t kStageBytes = 2 * kTileBytes;      // K, V
constexpr uint32_t kRawBytes = 2 * kTileRows * 64;    // of e4m3
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColP = 128, kColO = 192, kTileCols = 256;
constexpr int kPartFloats = kChunkPartFloats;         // of a tile: O [16][128][4], then m and l of 128 row heads

template <bool kE4m3>
struct Cfg {
  static constexpr int kThreads = kE4m3 ? 512 : 384;
  static constexpr int kStages = kE4m3 ? 3 : 4;
  static constexpr int kRaw = kE4m3 ? 2 : 0;
  // Registers of a thread, by warps of four: they add up to what the block is launched with, for which the compiler has to
  // give a thread kRegsLaunch (paged_chunk_registers, and the build, see that it did: with fewer, a warp would wait for its
  // share for ever).
  static constexpr int kRegsLaunch = kE4m3 ? 128 : 168;
  static constexpr int kRegsFew = 56, kRegsConvert = 88, kRegsSoftmax = kE4m3 ? 184 : 224;
  static_assert((kRegsFew + 2 * kRegsSoftmax + (kE4m3 ? kRegsConvert : 0)) * 128 <= kRegsLaunch * kThreads, "registers");
  static constexpr uint32_t kQ = 0;                                   // [2 buffers][2 tiles]
  static constexpr uint32_t kStage0 = 4 * kTileBytes;
  static constexpr uint32_t kRaw0 = kStage0 + kStages * kStageBytes;
  static constexpr uint32_t kScale0 = kRaw0 + kRaw * kRawBytes;       // [raw stage][K, V][128]
  static constexpr uint32_t kSum = kScale0 + kRaw * 2 * kTileRows;
  static constexpr uint32_t kLen = kSum + (kStepSeqs + 1) * 8;
  static constexpr uint32_t kRow0 = kLen + kStepSeqs * 4;
  static constexpr uint32_t kCount = kRow0 + kStepSeqs * 4;
  static constexpr uint32_t kScan = kCount + kStepSeqs * 4;
  static constexpr uint32_t kBar = kScan + 16 * 8;
  // barriers
  static constexpr int kFull = 0, kReady = kFull + (kE4m3 ? kRaw : kStages), kEmpty = kReady + kStages, kRawEmpty = kEmpty + kStages,
                       kQFull = kRawEmpty + kRaw, kQFree = kQFull + 2, kSReady = kQFree + 2, kSFree = kSReady + 2, kPReady = kSFree + 2,
                       kPvDone = kPReady + 2, kNumBars = kPvDone + 2;
  static constexpr uint32_t kInfo = kBar + 8 * kNumBars;              // pages of a block that are there: bit i, rows 16 i ..
  static constexpr uint32_t kMissing = kInfo + 4 * (kStages + kRaw);
  static constexpr uint32_t kTmemSlot = kMissing + 4;
  static constexpr uint32_t kRedo = (kTmemSlot + 16 + 15) & ~15u;      // ChunkRedo of each softmax warp
  static constexpr uint32_t kBytes = kRedo + kChunkSoftmaxWarps * sizeof(ChunkRedo);
  static constexpr uint32_t kRequest = kBytes + 1024;
  static_assert(kRequest <= 227 * 1024, "shared memory budget");
};

__device__ __forceinline__ bool wait_or_flag(uint32_t bar, uint32_t parity, unsigned* err, unsigned code) {
  if (mbar_wait_bounded(bar, parity, kWaitLimitNs)) return true;
  atomicOr(err, code);
  return false;
}

template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.ftz.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// Rows of a sequence in an item (both tiles), and blocks of 128 cached rows of item b of a sequence of n new rows: as
// many as its last row sees.
__device__ __forceinline__ int32_t blocks_of(int32_t len, int32_t n, int32_t b, int32_t rows) {
  return max(1, (len - n + min(n, (b + 1) * rows) + kTileRows - 1) >> 7);
}

// sum over i < n of floor((a i + b) / m), a, b >= 0 (Euclid's steps), in 32 bits where they are enough.
template <typename T>
__device__ __forceinline__ int64_t floor_sum(T n, T m, T a, T b) {
  int64_t sum = 0;
  while (n > 0) {
    if (a >= m) sum += static_cast<int64_t>(n) * (n - 1) / 2 * (a / m), a %= m;
    if (b >= m) sum += static_cast<int64_t>(n) * (b / m), b %= m;
    const T last = a * n + b;
    if (last < m) break;
    n = last / m;
    b = last % m;
    const T x = m;
    m = a, a = x;
  }
  return sum;
}

// Blocks of the items before item b (b up to their number).
__device__ __forceinline__ int64_t blocks_before(int32_t len, int32_t n, int32_t b, int32_t rows) {
  const int32_t items = (n + rows - 1) / rows, full = min(b, items - 1), first = len - n;   // full: items of `rows` rows
  const int32_t one = min(full, max(0, kTileRows - first) / rows);                          // those of one block
  const int64_t start = static_cast<int64_t>(first) + static_cast<int64_t>(one + 1) * rows + kTileRows - 1;
  const uint32_t more = static_cast<uint32_t>(full - one);
  int64_t sum = one;
  if (more > 0) {
    if (more < (1u << 20) && start < (int64_t(1) << 31))
      sum += floor_sum<uint32_t>(more, kTileRows, rows, static_cast<uint32_t>(start));
    else
      sum += floor_sum<uint64_t>(more, kTileRows, rows, static_cast<uint64_t>(start));
  }
  if (b == items) sum += blocks_of(len, n, items - 1, rows);
  return sum;
}

// An item counts as so many blocks more than it has: what its start and end cost a CTA that goes from one item to the
// next (512 rows behind 7,400, 16 heads: the CTAs with two items took 5 us longer than the others, of 26).
constexpr int32_t kItemBlocks = 3;

// A run of blocks [j0, j1) of one item, and the units it counts for.
struct Run {
  int s, h;
  int32_t b, j0, j1, blocks;
  int64_t units;
};

// kWhole: no item goes over several CTAs, there is no workspace, and no join kernel behind.
template <bool kE4m3, bool kWhole>
__global__ void __launch_bounds__(Cfg<kE4m3>::kThreads, 1)
paged_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ KvArgs a, const __grid_constant__ PagedAttn p, int s0, int ns, float* ws) {
  using C = Cfg<kE4m3>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int64_t* sum = reinterpret_cast<int64_t*>(smem + C::kSum);
  int32_t* s_len = reinterpret_cast<int32_t*>(smem + C::kLen);
  int32_t* s_row0 = reinterpret_cast<int32_t*>(smem + C::kRow0);
  int32_t* s_n = reinterpret_cast<int32_t*>(smem + C::kCount);
  volatile uint32_t* info = reinterpret_cast<volatile uint32_t*>(smem + C::kInfo);
  volatile uint32_t* some_missing = reinterpret_cast<volatile uint32_t*>(smem + C::kMissing);   // some block lacks pages
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kTmemSlot);
  auto bar = [&](int slot) { return base + C::kBar + 8u * slot; };
  const int32_t tile_rows = kTileRows / p.group, item_rows = 2 * tile_rows;

  if (tid == 0) {
    for (int i = 0; i < (kE4m3 ? C::kRaw : C::kStages); ++i) mbar_init(bar(C::kFull + i), 1);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(bar(C::kReady + i), kE4m3 ? 4 : 1);
      mbar_init(bar(C::kEmpty + i), 1);
    }
    for (int i = 0; i < C::kRaw; ++i) mbar_init(bar(C::kRawEmpty + i), 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::kQFull + i), 1);
      mbar_init(bar(C::kQFree + i), 1);
      mbar_init(bar(C::kSReady + i), 1);
      mbar_init(bar(C::kSFree + i), 128);
      mbar_init(bar(C::kPReady + i), 128);
      mbar_init(bar(C::kPvDone + i), 1);
    }
    fence_mbar_init();
    *some_missing = 0;
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  griddep_wait();                // (what comes before the call)
  griddep_launch_dependents();   // (the step kernel reads nothing of this one; what comes behind it waits for both)
  // ---------------------------------------------------------------- the sequences' running sums of blocks
  {
    const int per = (ns + C::kThreads - 1) / C::kThreads, b = min(ns, tid * per), e = min(ns, b + per);
    bool bad = false;
    int64_t mine = 0;
    for (int s = b; s < e; ++s) {
      const SeqRows r = seq_rows(a, s0 + s, &bad);
      const bool here = static_cast<int64_t>(r.n) * p.group > kStepHeads;
      s_len[s] = r.len;
      s_row0[s] = static_cast<int32_t>(r.row0);
      s_n[s] = here ? r.n : 0;
      sum[s] = mine;
      const int32_t items = (r.n + item_rows - 1) / item_rows;
      mine += here ? (blocks_before(r.len, r.n, items, item_rows) + static_cast<int64_t>(items) * kItemBlocks) * a.heads : 0;
    }
    if (bad) atomicOr(a.err, kErrSequence);
    int64_t upto = mine;
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += x;
    }
    int64_t* scan = reinterpret_cast<int64_t*>(smem + C::kScan);
    if (lane == 31) scan[warp] = upto;
    __syncthreads();
    int64_t before = upto - mine;
    for (int w = 0; w < warp; ++w) before += scan[w];
    for (int s = b; s < e; ++s) sum[s] += before;
    if (tid == C::kThreads - 1) sum[ns] = before + mine;
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
  }
  const uint32_t tmem = *tmem_slot;
  const int64_t U = sum[ns];
  // nw CTAs are at work, each has a unit at least: the first `more` have each + 1 of them, the others `each`.
  const int64_t nw = max(static_cast<int64_t>(1), min(static_cast<int64_t>(gridDim.x), U));
  const int64_t each = quotient(U, nw), more = U - each * nw;
  auto edge_of = [&](int64_t c) { return each * min(c, nw) + min(min(c, nw), more); };
  const int64_t lo = edge_of(blockIdx.x), hi = edge_of(blockIdx.x + 1);
  // The run of blocks that unit `lo` begins (every warp finds it for itself).
  Run first{};
  int64_t left = hi - lo;
  // The run from unit `off` of the item on: its blocks are the units behind the first kItemBlocks.
  auto take = [&](Run& r, int64_t off) {
    r.blocks = blocks_of(s_len[r.s], s_n[r.s], r.b, item_rows);
    r.units = static_cast<int64_t>(r.blocks) + kItemBlocks - off;
    if (!kWhole) r.units = min(r.units, left);
    r.j0 = static_cast<int32_t>(max(static_cast<int64_t>(0), off - kItemBlocks));
    r.j1 = static_cast<int32_t>(max(static_cast<int64_t>(r.j0), off + r.units - kItemBlocks));
    if (r.j1 == r.j0) left = 0;   // (the CTA's units end before the item's blocks begin)
  };
  if (lo < hi) {
    int l = 0, r = ns;   // the last sequence that starts at lo or before
    while (r - l > 1) {
      const int mid = (l + r) >> 1;
      if (sum[mid] <= lo) l = mid;
      else r = mid;
    }
    first.s = l;
    const int32_t len = s_len[l], n = s_n[l], items = (n + item_rows - 1) / item_rows;
    const int64_t a_head = quotient(sum[l + 1] - sum[l], a.heads), in = lo - sum[l];
    first.h = static_cast<int>(quotient(in, a_head));
    const int64_t rest = in - first.h * a_head;
    int32_t at = 0, count = items;   // the last item that starts at `rest` or before, 32 at a time
    int64_t begin = 0;
    while (count > 1) {
      const int32_t step = (count + 31) / 32, mine = at + lane * step;
      const int64_t b = mine < at + count ? blocks_before(len, n, mine, item_rows) + static_cast<int64_t>(mine) * kItemBlocks : INT64_MAX;
      const int upto = max(__popc(__ballot_sync(0xffffffffu, b <= rest)) - 1, 0);
      begin = __shfl_sync(0xffffffffu, b, upto);
      const int32_t from = upto * step;
      count = min(step, count - from);
      at += from;
    }
    first.b = at;
    take(first, rest - begin);
  }
  auto next_run = [&](Run& r, int64_t& left) {
    left -= r.units;
    if (left <= 0) return;
    if ((r.b + 1) * static_cast<int64_t>(item_rows) < s_n[r.s]) {
      ++r.b;
    } else {
      r.b = 0;
      if (++r.h == a.heads) {
        r.h = 0;
        do ++r.s;
        while (sum[r.s + 1] == sum[r.s]);
      }
    }
    take(r, 0);
  };
  // Rows of tile x of a run's item.
  auto rows_of = [&](const Run& r, int x) { return max(0, min(tile_rows, s_n[r.s] - r.b * item_rows - x * tile_rows)); };

  // Whole items: a CTA takes those that begin in its units.
  if (kWhole && left > 0 && first.units < first.blocks + kItemBlocks) next_run(first, left);

  Run r = first;
  if (warp < 4) {
    regs_dec<C::kRegsFew>();
    if (warp == 0) {
      // ------------------------------------------------------------ loads
      constexpr int kRing = kE4m3 ? C::kRaw : C::kStages;
      bool ok = true;
      int g = 0, item = 0;
      const int32_t box = min(a.page_rows, kTileRows), copies = kTileRows / box;   // copies: pages of a block, at most 8
      for (; left > 0 && ok; next_run(r, left), ++item) {
        const int qb = item & 1;
        const int32_t len = s_len[r.s], n_pages = (len + a.page_rows - 1) >> a.page_shift;
        if (!__all_sync(0xffffffffu, wait_or_flag(bar(C::kQFree + qb), ((item >> 1) & 1) ^ 1, a.err, kErrTimeoutMma))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          const int tiles = rows_of(r, 1) > 0 ? 2 : 1;
          mbar_arrive_expect_tx(bar(C::kQFull + qb), tiles * tile_rows * p.group * 128);
          for (int x = 0; x < tiles; ++x)
            tma_load_3d(base + C::kQ + (2 * qb + x) * kTileBytes, &tm_q, bar(C::kQFull + qb), 0, r.h * p.group,
                        s_row0[r.s] + r.b * item_rows + x * tile_rows);
        }
        int win0 = -64;
        int32_t win = -1;   // lane i: page win0 + i of the sequence
        for (int32_t j = r.j0; j < r.j1 && ok; ++j, ++g) {
          const int st = g % kRing;
          if (!__all_sync(0xffffffffu, wait_or_flag(bar((kE4m3 ? C::kRawEmpty : C::kEmpty) + st), ((g / kRing) & 1) ^ 1, a.err, kErrTimeoutMma))) {
            ok = false;
            break;
          }
          const int32_t page0 = (j * kTileRows) >> a.page_shift;
          if (page0 < win0 || page0 + copies > win0 + 32) {
            win0 = page0;
            win = page0 + lane < n_pages ? page_at(a, s0 + r.s, page0 + lane) : 0;
            if (win < 0) atomicOr(a.err, kErrPage);
          }
          const int32_t page = __shfl_sync(0xffffffffu, win, (page0 - win0 + lane) & 31);
          const bool mine = lane < copies && page0 + lane < n_pages && page >= 0;
          const uint32_t which = __ballot_sync(0xffffffffu, mine);
          if (lane == 0) {
            uint32_t there = 0;   // 16 rows a bit
            for (int c = 0; c < copies; ++c)
              if ((which >> c) & 1u) there |= ((1u << (box / 16)) - 1u) << (c * (box / 16));
            info[st] = there;
            if (there != 0xffu) *some_missing = 1;
            const uint32_t bytes = __popc(which) * box * (kE4m3 ? 130u : 256u);
            if (bytes != 0) mbar_arrive_expect_tx(bar(C::kFull + st), bytes);
            else mbar_arrive(bar(C::kFull + st));
          }
          __syncwarp();
          if (mine) {
            const int32_t row = (j * kTileRows) & (a.page_rows - 1);   // (0 but in pages of 256 rows)
            const uint32_t to = kE4m3 ? base + C::kRaw0 + st * kRawBytes : base + C::kStage0 + st * kStageBytes;
            constexpr uint32_t kRow = kE4m3 ? 64 : 128;
            tma_load_4d(to + lane * box * kRow, &tm_k, bar(C::kFull + st), 0, row, r.h, page);
            tma_load_4d(to + kTileRows * kRow + lane * box * kRow, &tm_v, bar(C::kFull + st), 0, row, r.h, page);
            if (kE4m3) {
              const int64_t from = page * a.scale_page_stride + r.h * a.scale_head_stride + row;
              const uint32_t sc = base + C::kScale0 + st * 2 * kTileRows + lane * box;
              bulk_copy_g2s(sc, a.k_scale + from, box, bar(C::kFull + st));
              bulk_copy_g2s(sc + kTileRows, a.v_scale + from, box, bar(C::kFull + st));
            }
          }
          __syncwarp();
        }
      }
      // Wait (bounded) for the loads in flight before the CTA can exit.
      for (int u = max(0, g - kRing); u < g; ++u)
        mbar_wait_bounded(bar(C::kFull + u % kRing), (u / kRing) & 1, ok ? kWaitLimitNs : 1000000ull);
    } else if (warp == 3) {
      // ------------------------------------------------------------ V rows that do not exist; the join kernel's record
      bool ok = true;
      int g = 0;
      ChunkJoin join{};
      for (; left > 0 && ok; next_run(r, left)) {
        const int32_t len = s_len[r.s];
        if (!kE4m3) {
          for (int32_t j = r.j0; j < r.j1; ++j, ++g) {
            const int st = g % C::kStages;
            if (!__all_sync(0xffffffffu, wait_or_flag(bar(C::kFull + st), (g / C::kStages) & 1, a.err, kErrTimeoutTma))) {
              ok = false;
              break;
            }
            const uint32_t there = info[st];
            const int32_t rows = len - j * kTileRows;
            if (rows < kTileRows || there != 0xffu) {
              uint8_t* v = smem + C::kStage0 + st * kStageBytes + kTileBytes;
              for (int i = lane; i < kTileRows * 8; i += 32)
                if ((i >> 3) >= rows || !((there >> (i >> 7)) & 1u)) *reinterpret_cast<uint4*>(v + i * 16) = make_uint4(0u, 0u, 0u, 0u);
              fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::kReady + st));
          }
        }
        if (r.j0 == 0 && r.j1 < r.blocks) {
          const int64_t u = hi + (r.blocks - r.j1) - 1;   // the item's last unit, and the CTA that has it
          const int64_t c = u < more * (each + 1) ? quotient(u, each + 1) : more + quotient(u - more * (each + 1), each);
          join.parts = static_cast<int32_t>(c) - static_cast<int32_t>(blockIdx.x) + 1;
          join.s = s0 + r.s;
          join.h = r.h;
          join.first = r.b * item_rows;
          join.n = s_n[r.s];
          join.len = len;
          join.row0 = s_row0[r.s];
        }
      }
      if (lane == 0 && !kWhole) {
        if (!ok) join.parts = 0;
        *reinterpret_cast<ChunkJoin*>(ws + blockIdx.x * kChunkWsFloats + 4 * kPartFloats) = join;
      }
    } else if (lane == 0) {
      // ------------------------------------------------------------ products, issued by one lane: S by warp 1, P V by warp 2
      // Apart, because the S that a softmax warp needs next may be issued as soon as it has taken the last one, while
      // the P V in between waits for its exponentials: with both from one warp in turn, S came 650 cycles late.  (The
      // loops are unrolled and the descriptors' low words counted up; built for each product, on a scheduler shared
      // with busy warps, the issue took twice as long as the products.)
      constexpr uint32_t id_qk = idesc_bf16_f32(128, 128, 0, 0), id_pv = idesc_bf16_f32(128, 64, 0, 1);
      bool ok = true;
      int st = 0, item = 0;
      uint32_t use = 0, gx[2] = {0, 0};      // use: of the ring, st: its stage; gx: blocks of each tile
      if (warp == 1) {
        const uint64_t d_q = smem_desc_sw128(base + C::kQ, 16, 1024), d_k = smem_desc_sw128(base + C::kStage0, 16, 1024);
        const uint32_t b_k = bar(kE4m3 ? C::kReady : C::kFull);
        for (; left > 0 && ok; next_run(r, left), ++item) {
          const int qb = item & 1, tiles = rows_of(r, 1) > 0 ? 2 : 1;
          ok = wait_or_flag(bar(C::kQFull + qb), (item >> 1) & 1, a.err, kErrTimeoutTma);
          const uint64_t q = d_q + qb * (2 * kTileBytes >> 4);
          for (int32_t j = r.j0; j < r.j1 && ok; ++j) {
            ok = wait_or_flag(b_k + 8 * st, use & 1, a.err, kErrTimeoutTma);
            const uint64_t k = d_k + st * (kStageBytes >> 4);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (x >= tiles || !ok) break;
              if (gx[x] > 0) ok = wait_or_flag(bar(C::kSFree + x), (gx[x] - 1) & 1, a.err, kErrTimeoutMma);
              if (!ok) break;
              tc_fence_after_sync();
#pragma unroll
              for (int kk = 0; kk < kHeadDim / 16; ++kk)
                mma_bf16(tmem + x * kTileCols, q + x * (kTileBytes >> 4) + kk * 2, k + kk * 2, id_qk, kk > 0 ? 1u : 0u);
              mma_commit(bar(C::kSReady + x));
              ++gx[x];
            }
            if (ok && j == r.j1 - 1) mma_commit(bar(C::kQFree + qb));
            if (++st == C::kStages) st = 0, ++use;
          }
        }
      } else {
        const uint64_t d_v = smem_desc_sw128(base + C::kStage0 + kTileBytes, kTileBytes, 1024);
        for (; left > 0 && ok; next_run(r, left)) {
          const int tiles = rows_of(r, 1) > 0 ? 2 : 1;
          for (int32_t j = r.j0; j < r.j1 && ok; ++j) {
            ok = wait_or_flag(bar(C::kReady + st), use & 1, a.err, kErrTimeoutTma);
            const uint64_t v = d_v + st * (kStageBytes >> 4);
            const uint32_t more = j > r.j0 ? 1u : 0u;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (x >= tiles || !ok) break;
              ok = wait_or_flag(bar(C::kPReady + x), gx[x] & 1, a.err, kErrTimeoutMma);
              if (!ok) break;
              tc_fence_after_sync();
#pragma unroll
              for (int kk = 0; kk < kTileRows / 16; ++kk)
                mma_bf16_tmem_a(tmem + x * kTileCols + kColO, tmem + x * kTileCols + kColP + kk * 8, v + kk * (2048 >> 4), id_pv,
                                kk > 0 ? 1u : more);
              mma_commit(bar(C::kPvDone + x));
              ++gx[x];
            }
            if (ok) mma_commit(bar(C::kEmpty + st));   // (S of the block is done: P came of it)
            if (++st == C::kStages) st = 0, ++use;
          }
        }
      }
    }
  } else if (warp < 12) {
    // -------------------------------------------------------------- softmax of tile x
    regs_inc<C::kRegsSoftmax>();
    const int x = (warp - 4) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t ts = tmem + x * kTileCols + (static_cast<uint32_t>(quarter * 32) << 16);
    const float c2 = p.scale * 1.4426950408889634f;
    const float raise_margin = fminf(8.f / c2, 1e37f);
    const int my_row = row / p.group, my_head = row % p.group;
    ChunkRedo* redo = reinterpret_cast<ChunkRedo*>(smem + C::kRedo) + (warp - 4);
    if (!kWhole && lane == 0) redo->some = 0;
    __syncwarp();
    bool ok = true;
    int g = 0, gx = 0;
    for (; left > 0 && ok; next_run(r, left)) {
      const int32_t rows = rows_of(r, x);
      if (rows == 0) {
        g += r.j1 - r.j0;
        continue;
      }
      const bool live = my_row < rows;
      const int32_t len = s_len[r.s], n = s_n[r.s], in_seq = r.b * item_rows + x * tile_rows + my_row;
      const int32_t seen = live ? max(0, len - n + in_seq + 1) : INT32_MAX;   // (who is no row head has nothing to mask)
      float m_ref = -INFINITY, l = 0.f;
      for (int32_t j = r.j0; j < r.j1; ++j, ++g, ++gx) {
        const int st = g % C::kStages;
        if (!__all_sync(0xffffffffu, wait_or_flag(bar(C::kSReady + x), gx & 1, a.err, kErrTimeoutMma))) {
          ok = false;
          break;
        }
        uint32_t there = 0xffu;
        if (__any_sync(0xffffffffu, *some_missing != 0)) {   // (set before the block's loads were issued)
          if (!__all_sync(0xffffffffu, wait_or_flag(bar((kE4m3 ? C::kReady : C::kFull) + st), (g / C::kStages) & 1, a.err, kErrTimeoutTma))) {
            ok = false;
            break;
          }
          there = info[kE4m3 ? C::kRaw + st : st];
        }
        tc_fence_after_sync();
        float sc[128];
        {
          uint32_t(&sr)[128] = reinterpret_cast<uint32_t(&)[128]>(sc);
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld_32cols(ts + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(sr + 32 * c));
          tmem_ld_wait();
        }
        tc_fence_before_sync();
        mbar_arrive(bar(C::kSFree + x));   // (by every thread: a warp barrier and one arrival took longer)
        const int32_t hi_col = seen - j * kTileRows;      // columns before it are seen
        if (!__all_sync(0xffffffffu, hi_col >= kTileRows && there == 0xffu)) {
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c >= hi_col || !((there >> (c / 16)) & 1u)) sc[c] = -INFINITY;
        }
        float mx4[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) mx4[c] = fmaxf(sc[2 * c], sc[2 * c + 1]);
#pragma unroll
        for (int c = 8; c < 128; c += 2) mx4[(c >> 1) & 3] = max3(mx4[(c >> 1) & 3], sc[c], sc[c + 1]);
        const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        if (j == r.j0) {
          m_ref = mx;   // (O starts with this block)
        } else if (__any_sync(0xffffffffu, mx > m_ref + raise_margin)) {
          if (!__all_sync(0xffffffffu, wait_or_flag(bar(C::kPvDone + x), (gx - 1) & 1, a.err, kErrTimeoutMma))) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const float m_new = mx > m_ref + raise_margin ? mx : m_ref;   // (by the row alone, not by its neighbours)
          const float f = m_new == m_ref ? 1.f : ex2((m_ref - m_new) * c2);   // 0 where m_ref = -inf
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            uint32_t o[16];
            tmem_ld_16cols(ts + kColO + 16 * h, o);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
            tmem_st_16cols(ts + kColO + 16 * h, o);
          }
          l *= f;
          m_ref = m_new;
        }
        // (a reference that the scale takes to -infinity is none: its scores' weights are then 0, a NaN's NaN)
        const float neg = m_ref * c2 == -INFINITY ? 0.f : -m_ref * c2;
        const uint64_t cc = f32x2(c2, c2), nn = f32x2(neg, neg);
        uint64_t acc[2] = {f32x2(0.f, 0.f), f32x2(0.f, 0.f)};
        uint32_t pk[2][32];
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          float y0, y1;
          f32x2_split(fma_f32x2(f32x2(sc[2 * c], sc[2 * c + 1]), cc, nn), y0, y1);
          y0 = ex2(y0), y1 = ex2(y1);
          acc[c & 1] = add_f32x2(acc[c & 1], f32x2(y0, y1));
          pk[c >> 5][c & 31] = pack_bf16x2(y0, y1);
        }
        if (gx > 0) {   // P's last reader
          if (!__all_sync(0xffffffffu, wait_or_flag(bar(C::kPvDone + x), (gx - 1) & 1, a.err, kErrTimeoutMma))) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
        }
        tmem_st_32cols(ts + kColP, pk[0]);
        tmem_st_32cols(ts + kColP + 32, pk[1]);
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(bar(C::kPReady + x));
        float a0, a1, b0, b1;
        f32x2_split(acc[0], a0, a1);
        f32x2_split(acc[1], b0, b1);
        l += (a0 + b0) + (a1 + b1);
      }
      if (!ok) break;
      // ------------------------------------------------------------ the end of the item, or of this CTA's part
      if (!__all_sync(0xffffffffu, wait_or_flag(bar(C::kPvDone + x), (gx - 1) & 1, a.err, kErrTimeoutMma))) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const float m2 = m_ref == -INFINITY ? -INFINITY : m_ref * c2;
      if (m2 == INFINITY) l = NAN;   // (the greatest score is infinite, or the scale took it there)
      const bool complete = r.j0 == 0 && r.j1 == r.blocks;
      const int64_t at = (s_row0[r.s] + static_cast<int64_t>(in_seq)) * p.heads + r.h * p.group + my_head;
      float* part = ws + blockIdx.x * kChunkWsFloats + (2 * (r.j0 > 0 ? 0 : 1) + x) * kPartFloats;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      bool wild = false;
      uint32_t o[2][32];
      tmem_ld_32cols(ts + kColO, o[0]);
      tmem_ld_32cols(ts + kColO + 32, o[1]);
      tmem_ld_wait();
      tc_fence_before_sync();
      if (live && complete) {
        uint4* dst = reinterpret_cast<uint4*>(p.out + at * kHeadDim);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t pk[4];
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const float y0 = __uint_as_float(o[c >> 2][8 * (c & 3) + 2 * d]) * inv, y1 = __uint_as_float(o[c >> 2][8 * (c & 3) + 2 * d + 1]) * inv;
            wild |= !(fabsf(y0) <= 3.4e38f) || !(fabsf(y1) <= 3.4e38f);
            pk[d] = l == 0.f ? 0u : pack_bf16x2(y0, y1);
          }
          dst[c] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
        if (p.lse != nullptr) p.lse[at] = l == 0.f ? -INFINITY : fmaf(m2, 0.6931471805599453f, logf(l));
      } else if (live) {
        float4* dst = reinterpret_cast<float4*>(part) + row;   // four elements of all row heads, then the next four
#pragma unroll
        for (int c = 0; c < 16; ++c)
          dst[c * kTileRows] = make_float4(__uint_as_float(o[c >> 3][4 * (c & 7)]), __uint_as_float(o[c >> 3][4 * (c & 7) + 1]),
                               __uint_as_float(o[c >> 3][4 * (c & 7) + 2]), __uint_as_float(o[c >> 3][4 * (c & 7) + 3]));
        part[kTileRows * kHeadDim + row] = m2;
        part[kTileRows * kHeadDim + kTileRows + row] = l;
      }
      // Rows whose O came out infinite or NaN though the sum of weights is finite are looked at once more, without the rows
      // that they do not see: by the join kernel, which finds them by their marks.  (Here it would cost the loop over the
      // blocks registers, 2,048 rows 183 us instead of 175; and, over a long cache, take longer than the CTA's other warps
      // wait for this one.)  By this warp where there is no join, over at most 512 rows.
      wild &= l == l && l != 0.f;
      if (!kWhole && wild) {
        if (redo->some == 0) redo->s = s0 + r.s, redo->h = r.h, redo->b = r.b;
        redo->last_s = s0 + r.s, redo->last_h = r.h, redo->last_b = r.b;
        redo->some = 1;
        uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + at * kHeadDim);
#pragma unroll 1
        for (int c = 0; c < kHeadDim / 2; ++c) dst[c] = marked(dst[c]);
      }
      if (kWhole) {
        const uint32_t which = __ballot_sync(0xffffffffu, wild);
        if (which != 0)
          redo_rows<kE4m3>(a, p, which, s0 + r.s, r.h, s_row0[r.s] + static_cast<int64_t>(in_seq - my_row), quarter * 32,
                           len - n + in_seq - my_row + 1);
      }
    }
    if (!kWhole) {
      __syncwarp();
      if (lane == 0) {
        if (!ok) redo->some = 0;   // (a wait ran out: there are items without any result)
        reinterpret_cast<ChunkRedo*>(ws + blockIdx.x * kChunkWsFloats + 4 * kPartFloats + 8)[warp - 4] = *redo;
      }
    }
  } else {
    // -------------------------------------------------------------- e4m3 rows into bf16 tiles
    regs_dec<C::kRegsConvert>();
    if (kE4m3) {
      const int row = tid - 384;
      bool ok = true;
      int g = 0;
      for (; left > 0 && ok; next_run(r, left)) {
        const int32_t len = s_len[r.s];
        for (int32_t j = r.j0; j < r.j1; ++j, ++g) {
          const int rs = g % max(1, C::kRaw), st = g % C::kStages;
          bool w = wait_or_flag(bar(C::kFull + rs), (g / max(1, C::kRaw)) & 1, a.err, kErrTimeoutTma);
          if (w) w = wait_or_flag(bar(C::kEmpty + st), ((g / C::kStages) & 1) ^ 1, a.err, kErrTimeoutMma);
          if (!__all_sync(0xffffffffu, w)) {
            ok = false;
            break;
          }
          const uint32_t there = info[rs];
          const bool exists = j * kTileRows + row < len && ((there >> (row / 16)) & 1u);
          if (row == 0) info[C::kRaw + st] = there;
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            const uint8_t* from = smem + C::kRaw0 + rs * kRawBytes + kv * kTileRows * 64 + row * 64;
            uint8_t* to = smem + C::kStage0 + st * kStageBytes + kv * kTileBytes + row * 128;
            if (!exists) {
#pragma unroll
              for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(to + c * 16) = make_uint4(0u, 0u, 0u, 0u);
              continue;
            }
            const float e = scale_of(smem[C::kScale0 + (rs * 2 + kv) * kTileRows + row]);
            const uint64_t ee = f32x2(e, e);
            uint4 in[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) in[c] = *reinterpret_cast<const uint4*>(from + ((c ^ ((row >> 1) & 3)) << 4));
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t w[4] = {in[c].x, in[c].y, in[c].z, in[c].w};
              uint32_t out[8];
#pragma unroll
              for (int d = 0; d < 4; ++d) {
                uint32_t h[2];
                half2_of_e4m3(w[d], h[0], h[1]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
                  float v0, v1;
                  f32x2_split(mul_f32x2(f32x2(v.x, v.y), ee), v0, v1);
                  out[2 * d + i] = pack_bf16x2(v0, v1);
                }
              }
              *reinterpret_cast<uint4*>(to + (((2 * c) ^ (row & 7)) << 4)) = make_uint4(out[0], out[1], out[2], out[3]);
              *reinterpret_cast<uint4*>(to + (((2 * c + 1) ^ (row & 7)) << 4)) = make_uint4(out[4], out[5], out[6], out[7]);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(C::kRawEmpty + rs));
            mbar_arrive(bar(C::kReady + st));
          }
        }
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

// CTA (c, y): 32 row heads (y & 3) of tile y >> 2 of the item that begins in CTA c of the chunk kernel and goes on, from
// the parts of it and the next CTAs.  A lane has a row head, warp w eight elements of O, and the maxima and sums of every
// eighth part.  What an item of two parts needs is asked for before the record is there that says how many there are.
constexpr int kChunkJoinThreads = 256, kJoinWarps = kChunkJoinThreads / 32;

// A warp: the rows that a softmax warp (x, quarter) has marked, in items from the first to the last that it names.
template <bool kE4m3>
__device__ __forceinline__ void redo_chunk_items(const KvArgs& a, const PagedAttn& p, const ChunkRedo& redo, int x, int quarter) {
  const int lane = threadIdx.x & 31;
  const int32_t tile_rows = kTileRows / p.group;
  int32_t h = redo.h, b = redo.b;
  for (int32_t s = redo.s; s <= redo.last_s; ++s, h = b = 0) {
    bool bad = false;
    const SeqRows r = seq_rows(a, s, &bad);
    if (static_cast<int64_t>(r.n) * p.group <= kStepHeads) continue;
    const int32_t items = (r.n + 2 * tile_rows - 1) / (2 * tile_rows);
    const int32_t last_h = s == redo.last_s ? redo.last_h : a.heads - 1;
    for (; h <= last_h; ++h, b = 0) {
      const int32_t last_b = s == redo.last_s && h == last_h ? redo.last_b : items - 1;
      for (; b <= last_b; ++b) {
        const int32_t first = (2 * b + x) * tile_rows;
        uint32_t which = 0;
        for (int i = 0; i < 32; i += 4) {
          const int row = quarter * 32 + i + (lane >> 3), in = first + row / p.group;
          bool mark = false;
          if (row / p.group < tile_rows && in < r.n) {
            const uint4 o =
                *reinterpret_cast<const uint4*>(p.out + ((r.row0 + in) * p.heads + h * p.group + row % p.group) * kHeadDim + 8 * (lane & 7));
            mark = has_mark(o.x) || has_mark(o.y) || has_mark(o.z) || has_mark(o.w);
          }
          const uint32_t lanes = __ballot_sync(0xffffffffu, mark);
          for (int g = 0; g < 4; ++g)
            if ((lanes >> (8 * g)) & 0xffu) which |= 1u << (i + g);
        }
        if (which != 0) redo_rows<kE4m3>(a, p, which, s, h, r.row0 + first, quarter * 32, r.len - r.n + first + 1);
      }
    }
  }
}

// CTAs (c, 8 ..): the step kernel's parts (of `step_grid` CTAs), where it has some of the same call, and the row heads that it
// has marked; the last ones: those that the chunk kernel has marked.
template <bool kE4m3, bool kStepE4m3>
__global__ void __launch_bounds__(kChunkJoinThreads, 4)
chunk_join_kernel(const __grid_constant__ KvArgs a, const __grid_constant__ PagedAttn p, const float* ws, const __grid_constant__ KvArgs step,
                  const float* step_ws, int step_grid) {
  __shared__ float factor[kStepMaxGrid][32];
  __shared__ float best[kJoinWarps][32], sums[kJoinWarps][32];
  __shared__ uint32_t wild;
  griddep_launch_dependents();
  griddep_wait();
  const float* mine = ws + blockIdx.x * kChunkWsFloats;
  if (blockIdx.y >= 8) {
    const int y = static_cast<int>(blockIdx.y) - 8, steps = kM / kJoinRows;
    if (blockIdx.y == gridDim.y - 1) {
      const int w = static_cast<int>(threadIdx.x) >> 5;   // a warp for each softmax warp
      static_assert(kJoinWarps == kChunkSoftmaxWarps, "warps");
      const ChunkRedo* redo = reinterpret_cast<const ChunkRedo*>(mine + 4 * kPartFloats + 8) + w;
      if (redo->some != 0) redo_chunk_items<kE4m3>(a, p, *redo, w >> 2, w & 3);
    } else if (static_cast<int>(blockIdx.x) < step_grid) {
      if (y < steps) join_step_parts<kStepE4m3, kChunkJoinThreads / 16 / kJoinRows>(step, p, step_ws, step_grid, y);
      else redo_step_items<kStepE4m3>(step, p, step_ws);
    }
    return;
  }
  const int x = blockIdx.y >> 2, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = (blockIdx.y & 3) * 32 + lane;
  const int last = static_cast<int>(gridDim.x - 1 - blockIdx.x);
  auto part_of = [&](int i) { return mine + i * kChunkWsFloats + (2 * (i == 0 ? 1 : 0) + x) * kPartFloats; };
  auto four = [&](int i, int c) { return reinterpret_cast<const float4*>(part_of(i))[(2 * warp + c) * kTileRows + row]; };
  const ChunkJoin j = *reinterpret_cast<const ChunkJoin*>(mine + 4 * kPartFloats);
  float m0, l0;
  {
    const float* st = part_of(min(warp, last)) + kTileRows * kHeadDim + row;
    m0 = st[0], l0 = st[kTileRows];
  }
  float4 ahead[kJoinAhead][2];
#pragma unroll
  for (int i = 0; i < kJoinAhead; ++i) ahead[i][0] = four(min(i, last), 0), ahead[i][1] = four(min(i, last), 1);
  const int32_t tile_rows = kTileRows / p.group, in = j.first + x * tile_rows + row / p.group;
  const bool live = j.parts > 0 && row / p.group < tile_rows && in < j.n;
  if (threadIdx.x == 0) wild = 0;
  if (!__syncthreads_or(live)) return;
  float m = warp < j.parts ? m0 : -INFINITY, l = 0.f;
  for (int i = warp + kJoinWarps; i < j.parts; i += kJoinWarps) m = fmaxf(m, part_of(i)[kTileRows * kHeadDim + row]);
  best[warp][lane] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, best[w][lane]);
  for (int i = warp; i < j.parts; i += kJoinWarps) {
    const float* st = part_of(i) + kTileRows * kHeadDim + row;
    const float pm = i == warp ? m0 : st[0], pl = i == warp ? l0 : st[kTileRows];
    const float f = pm == m ? 1.f : pm == -INFINITY ? 0.f : ex2(pm - m);
    factor[i][lane] = f;
    l += pl * f;
  }
  sums[warp][lane] = l;
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) l += sums[w][lane];
  if (live) {
    float o[8] = {};
    auto add = [&](const float4& y, int c, float f) {
      o[4 * c] = fmaf(f, y.x, o[4 * c]), o[4 * c + 1] = fmaf(f, y.y, o[4 * c + 1]);
      o[4 * c + 2] = fmaf(f, y.z, o[4 * c + 2]), o[4 * c + 3] = fmaf(f, y.w, o[4 * c + 3]);
    };
#pragma unroll
    for (int i = 0; i < kJoinAhead; ++i) add(ahead[i][0], 0, factor[i][lane]), add(ahead[i][1], 1, factor[i][lane]);   // (two at least)
#pragma unroll 4
    for (int i = kJoinAhead; i < j.parts; ++i) add(four(i, 0), 0, factor[i][lane]), add(four(i, 1), 1, factor[i][lane]);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t at = (j.row0 + static_cast<int64_t>(in)) * p.heads + j.h * p.group + row % p.group;
    bool w = false;
    uint32_t pk[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float y0 = o[2 * c] * inv, y1 = o[2 * c + 1] * inv;
      w |= !(fabsf(y0) <= 3.4e38f) || !(fabsf(y1) <= 3.4e38f);
      pk[c] = l == 0.f ? 0u : pack_bf16x2(y0, y1);
    }
    *reinterpret_cast<uint4*>(p.out + at * kHeadDim + 8 * warp) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
    if (p.lse != nullptr && warp == 0) p.lse[at] = l == 0.f ? -INFINITY : fmaf(m, 0.6931471805599453f, logf(l));
    if (w && l == l && l != 0.f) atomicOr(&wild, 1u << lane);
  }
  __syncthreads();
  const uint32_t which = wild & (0xfu << (4 * warp));   // the row heads that are done over, four a warp
  const int32_t first = j.first + x * tile_rows;
  if (which != 0)
    redo_rows<kE4m3>(a, p, which, j.s, j.h, j.row0 + static_cast<int64_t>(first), (blockIdx.y & 3) * 32, j.len - j.n + first + 1);
}

template <bool kE4m3, bool kWhole>
cudaError_t launch(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const KvArgs& a, const PagedAttn& p, int s0,
                   int ns, int grid, float* ws, cudaStream_t stream) {
  using C = Cfg<kE4m3>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = set_smem_limit_once(paged_chunk_kernel<kE4m3, kWhole>, C::kRequest, done);
  if (e != cudaSuccess) return e;
  return launch_behind(paged_chunk_kernel<kE4m3, kWhole>, dim3(grid), C::kThreads, C::kRequest, stream, tm_q, tm_k, tm_v, a, p, s0, ns, ws);
}

}  // namespace

cudaError_t paged_chunk_registers(int* built, int* needed) {
  static std::atomic<int> found{0};   // built, less what is needed, plus 1024 (0: not asked yet); the scarcest kernel's
  int least = found.load(std::memory_order_relaxed);
  if (least == 0) {
    cudaFuncAttributes attr[4];
    cudaError_t e = cudaFuncGetAttributes(&attr[0], paged_chunk_kernel<false, false>);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&attr[1], paged_chunk_kernel<false, true>);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&attr[2], paged_chunk_kernel<true, false>);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&attr[3], paged_chunk_kernel<true, true>);
    if (e != cudaSuccess) return e;
    least = 1024 + std::min(std::min(attr[0].numRegs, attr[1].numRegs) - Cfg<false>::kRegsLaunch,
                            std::min(attr[2].numRegs, attr[3].numRegs) - Cfg<true>::kRegsLaunch);
    found.store(least, std::memory_order_relaxed);
  }
  *needed = Cfg<false>::kRegsLaunch;
  *built = *needed + least - 1024;
  return cudaSuccess;
}

cudaError_t launch_paged_chunk(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const KvArgs& a,
                               const PagedAttn& p, int s0, int ns, int grid, bool e4m3, bool whole_items, float* ws, cudaStream_t stream) {
  if (whole_items) return (e4m3 ? launch<true, true> : launch<false, true>)(tm_q, tm_k, tm_v, a, p, s0, ns, grid, ws, stream);
  return (e4m3 ? launch<true, false> : launch<false, false>)(tm_q, tm_k, tm_v, a, p, s0, ns, grid, ws, stream);
}

cudaError_t launch_chunk_join(const KvArgs& a, const PagedAttn& p, int grid, bool e4m3, const float* ws, const KvArgs& step, int step_grid,
                              bool step_e4m3, const float* step_ws, cudaStream_t stream) {
  auto* kernel = e4m3 ? chunk_join_kernel<true, true> : step_e4m3 ? chunk_join_kernel<false, true> : chunk_join_kernel<false, false>;
  return launch_behind(kernel, dim3(grid, step_grid > 0 ? 8 + kM / kJoinRows + 2 : 8 + 1), kChunkJoinThreads, 0, stream, a, p, ws, step, step_ws,
                       step_grid);
}

}  // namespace spanla
