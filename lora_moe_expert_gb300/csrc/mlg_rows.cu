// mlg_rows.cu -- rows into expert order and back: the stable sort of the flat
// (token, slot) rows by cell, the row copies into that order, the weighted sum
// back to tokens, and its gradient.
#include <algorithm>
#include <mutex>

#include "mlg_launch.cuh"

namespace mlg {
namespace {

constexpr size_t kSortSmem = 200 * 1024;
constexpr int kCopyThreads = 256;
constexpr int kGradThreads = 256, kGradBatch = 4;
// One launch sorts and copies: what one CTA compares, and all of them.
constexpr int kSmallGroup = 8, kSmallSlots = 2048, kSmallWork = 1 << 19, kSmallCells = 4096;

// ---------------------------------------------------------------- the sort
//
// The slots are cut into consecutive pieces, one per warp:
//   1. each warp reads its piece (up to kSteps steps of 32 slots at a time),
//      finds the equal cells of each step and counts them, one lane for each
//      cell, into its own histogram of cells + 1 bins (the last holds the slots
//      of no cell);
//   2. prefix over the warps and the cells: where each (cell, warp) begins;
//   3. each warp walks its piece in order, a step at a time, equal cells of a
//      step by lane, so equal cells keep their order.
// One cluster of up to 16 CTAs does it in one launch: CTA totals go to the peers
// through distributed shared memory, no global scratch is needed.  What it costs
// is latency and, on so few SMs, the steps' votes and the scattered stores of
// src (which mlg_dispatch leaves to its copy): 163840 slots of 512 cells 18 us,
// 32768 8 us.  Counting and ranking on 64 SMs in two launches more, with a scratch,
// gained 2 us of 124 in a dispatch of 163840 slots and lost 1.6 of 20 in one of
// 32744.  With many cells few warps have room for a histogram, and the CTAs shrink
// with them: 163840 slots of 4096 cells 64 us, of 24576 (one warp a CTA) 827.
struct SortParams {
  const int32_t *indices, *row_adapter;
  int32_t *offsets, *src, *pos;
  int32_t n_slots, top_k, n_experts, n_adapters, cells;
  int32_t warps;    // W
  int32_t cluster;  // C
  int32_t piece;    // slots per warp, a multiple of 32
  int32_t all_src;  // 0: write src only for the slots of no cell
  int32_t bits;     // of a bin
};

__device__ __forceinline__ uint32_t ld_dsmem_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// The bins of N slots i0, i0 + stride, ...: a slot's cell, or `cells` when it has
// none; cells + 1 from hi on.  The loads are all under way before any is used.
template <int N>
__device__ __forceinline__ void slot_bins(const SortParams &p, int64_t i0, int stride, int64_t hi,
                                          int (&bin)[N]) {
  int e[N], s[N];
#pragma unroll
  for (int k = 0; k < N; ++k)
    e[k] = i0 + k * stride < hi ? p.indices[i0 + k * stride] : -1;
  if (p.row_adapter) {
#pragma unroll
    for (int k = 0; k < N; ++k)
      s[k] = i0 + k * stride < hi
                 ? p.row_adapter[static_cast<int>(i0 + k * stride) / p.top_k]
                 : -1;
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) s[k] = 0;
  }
  const uint32_t E = p.n_experts, A = p.row_adapter ? p.n_adapters : 1;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const bool ok = static_cast<uint32_t>(e[k]) < E && static_cast<uint32_t>(s[k]) < A;
    bin[k] = i0 + k * stride >= hi ? p.cells + 1 : ok ? s[k] * p.n_experts + e[k] : p.cells;
  }
}

constexpr int kSteps = 12;

// The lanes that hold the same value (a value per lane, `bits` bits): a vote
// per bit, which takes less than half of match.any's time.  All lanes call it.
__device__ __forceinline__ uint32_t same_lanes(uint32_t v, int bits) {
  uint32_t same = kFullWarp;
#pragma unroll 5
  for (int b = 0; b < bits; ++b, v >>= 1) {
    const uint32_t m = __ballot_sync(kFullWarp, (v & 1u) != 0);
    same &= m ^ ((v & 1u) - 1u);  // m of a set bit, ~m of a clear one
  }
  return same;
}

// The slots [i0, hi) of a warp, 32 a step, at most kSteps: into `steps` (32 a
// step) a slot's bin (bits 10 up), how many of the step's earlier lanes have it
// too (bits 5..9) and how many in all, less one (bits 0..4); -1 past the end.
// With `mine`, counts them into that histogram.  Loops, not unrolled code: the
// kernel runs once for a few steps, and instruction misses would cost more.
__device__ __forceinline__ void load_steps(const SortParams &p, int64_t i0, int64_t hi, int *steps,
                                           uint32_t *mine) {
  const int lane = threadIdx.x & 31;
  const int n = static_cast<int>(min(static_cast<int64_t>(kSteps), (hi - i0 + 31) / 32));
#pragma unroll 1
  for (int k0 = 0; k0 < n; k0 += 4) {
    int bin[4];
    slot_bins(p, i0 + k0 * 32 + lane, 32, hi, bin);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k0 + k < kSteps) steps[(k0 + k) * 32 + lane] = bin[k];
  }
#pragma unroll 1
  for (int k = 0; k < n; ++k) {
    const int bin = steps[k * 32 + lane];
    const uint32_t same = same_lanes(bin, p.bits);
    const int below = __popc(same & ((1u << lane) - 1u)), all = __popc(same);
    const bool in = bin <= p.cells;
    steps[k * 32 + lane] = in ? bin << 10 | below << 5 | (all - 1) : -1;
    if (mine && in && below == 0) mine[bin] += all;
    __syncwarp();
  }
}

// Ranks a warp's steps; `mine` holds where its next slot of each bin goes.
__device__ __forceinline__ void place_steps(const SortParams &p, int64_t i0, int64_t hi,
                                            const int *steps, uint32_t *mine) {
  const int lane = threadIdx.x & 31;
  const int n = static_cast<int>(min(static_cast<int64_t>(kSteps), (hi - i0 + 31) / 32));
#pragma unroll 1
  for (int k = 0; k < n; ++k) {
    const int step = steps[k * 32 + lane];
    const bool in = step >= 0;
    const int c = step >> 10, below = step >> 5 & 31;
    uint32_t at = in ? mine[c] : 0u;
    __syncwarp();
    if (in && below == 0) mine[c] = at + (step & 31) + 1;
    __syncwarp();
    if (in) {
      const int i = static_cast<int>(i0 + k * 32 + lane);
      at += below;
      if (p.all_src || c == p.cells) p.src[at] = i;
      p.pos[i] = c < p.cells ? static_cast<int32_t>(at) : -1;
    }
  }
}

// Exclusive prefix of a value per thread over the CTA; `carry` in: the sum of
// earlier calls, out: with this one's.  All threads call it.
__device__ __forceinline__ uint32_t cta_prefix(uint32_t v, uint32_t (&warp_total)[32],
                                               uint32_t &carry) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = static_cast<int>(blockDim.x) >> 5;
  uint32_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(kFullWarp, incl, o);
    if (lane >= o) incl += u;
  }
  __syncthreads();  // warp_total of the last call is read
  if (lane == 31) warp_total[warp] = incl;
  __syncthreads();
  const uint32_t t = lane < warps ? warp_total[lane] : 0u;
  const uint32_t before = __reduce_add_sync(kFullWarp, lane < warp ? t : 0u);
  const uint32_t out = carry + before + incl - v;
  carry += __reduce_add_sync(kFullWarp, t);
  return out;
}

__global__ void __launch_bounds__(1024) sort_kernel(const SortParams p) {
  extern __shared__ uint32_t smem[];
  __shared__ uint32_t warp_total[32];
  const int tid = threadIdx.x, threads = blockDim.x, warp = tid >> 5;
  const int bins = p.cells + 1, W = p.warps;
  const int rank = p.cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  uint32_t *hist = smem;                 // [W][bins]
  uint32_t *total = smem + W * bins;     // [bins], read by the peers
  int *steps = reinterpret_cast<int *>(total + bins) + warp * (kSteps * 32);
  for (int i = tid; i < W * bins; i += threads) hist[i] = 0;
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();  // dispatch_kernel counts on this order

  const int64_t lo = (static_cast<int64_t>(rank) * W + warp) * p.piece;
  const int64_t hi = min(lo + p.piece, static_cast<int64_t>(p.n_slots));
  uint32_t *mine = hist + warp * bins;
  for (int64_t i0 = lo; i0 < hi; i0 += kSteps * 32) load_steps(p, i0, hi, steps, mine);
  __syncthreads();

  for (int c = tid; c < bins; c += threads) {
    uint32_t all = 0;
#pragma unroll 8
    for (int w = 0; w < W; ++w) all += hist[w * bins + c];
    total[c] = all;
  }
  if (p.cluster > 1) cluster_sync(); else __syncthreads();

  uint32_t carry = 0;
  for (int base = 0; base < bins; base += threads) {
    const int c = base + tid;
    uint32_t before = 0, all = 0;
    if (c < bins) {
      if (p.cluster > 1) {
        const uint32_t a = smem_addr(total + c);
#pragma unroll 8
        for (int r = 0; r < p.cluster; ++r) {
          const uint32_t v = ld_dsmem_u32(map_to_rank(a, r));
          if (r < rank) before += v;
          all += v;
        }
      } else {
        all = total[c];
      }
    }
    const uint32_t begin = cta_prefix(all, warp_total, carry);
    if (c < bins) {
      if (rank == 0) p.offsets[c] = static_cast<int32_t>(begin);
      uint32_t run = begin + before;
#pragma unroll 8
      for (int w = 0; w < W; ++w) {
        const uint32_t v = hist[w * bins + c];
        hist[w * bins + c] = run;
        run += v;
      }
    }
  }
  __syncthreads();
  if (p.cluster > 1) cluster_arrive();  // this CTA has read its peers' totals

  for (int64_t i0 = lo; i0 < hi; i0 += kSteps * 32) {
    if (p.piece > kSteps * 32) load_steps(p, i0, hi, steps, nullptr);
    place_steps(p, i0, hi, steps, mine);
  }
  __syncwarp();
  if (p.cluster > 1) cluster_wait();  // no CTA leaves while a peer reads its totals
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Slots per warp, a multiple of 32, for `warps` warps in all.
int32_t piece_for(int32_t n_slots, int64_t warps) {
  return static_cast<int32_t>(
      std::max<int64_t>(ceil_div(ceil_div(n_slots, warps), 32) * 32, 32));
}

cudaError_t launch_sort(SortParams &p, cudaStream_t stream) {
  static std::once_flag once[64];
  static cudaError_t attr_err[64];
  int dev = 0;
  cudaGetDevice(&dev);
  std::call_once(once[dev & 63], [d = dev & 63] {
    attr_err[d] = cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kSortSmem));
    if (attr_err[d] == cudaSuccess)
      attr_err[d] = cudaFuncSetAttribute(sort_kernel,
                                         cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  if (attr_err[dev & 63] != cudaSuccess) return attr_err[dev & 63];
  const int64_t bins = p.cells + 1;
  p.warps = 32;
  auto bytes = [&] { return ((p.warps + 1) * bins + p.warps * kSteps * 32) * 4; };
  while (p.warps > 1 && bytes() > static_cast<int64_t>(kSortSmem)) p.warps /= 2;
  p.cluster = 1;
  while (p.cluster < 16 && static_cast<int64_t>(p.cluster) * p.warps * 64 < p.n_slots)
    p.cluster *= 2;
  p.piece = piece_for(p.n_slots, static_cast<int64_t>(p.cluster) * p.warps);
  return launch_early(sort_kernel, p.cluster, p.warps * 32, bytes(), p.cluster, stream, p);
}

// ---------------------------------------------------------------- row copies
struct RowParams {
  const uint8_t *x;        // dispatch: token rows; combine: sorted rows
  const uint8_t *dout;     // combine_backward: token rows
  uint8_t *out;            // dispatch: sorted rows; combine: token rows
  uint8_t *dy;             // combine_backward: sorted rows
  int32_t *src;            // dispatch: written for the rows of a cell
  const int32_t *pos, *rows_held;
  const float *weights;
  float *dweights;
  int64_t ld;              // token row stride in bytes
  int64_t row_bytes;       // sorted row stride in bytes
  int32_t n_tokens, n_slots, n_rows, top_k, pieces;  // pieces: 16-byte pieces a row
};

// Token and 16-byte piece of a flat piece number.
__device__ __forceinline__ void piece_of(const RowParams &p, int64_t id, int64_t &t, int64_t &off) {
  if (id <= 0xffffffffll) {
    const uint32_t q = static_cast<uint32_t>(id) / static_cast<uint32_t>(p.pieces);
    t = q;
    off = static_cast<int64_t>(static_cast<uint32_t>(id) - q * p.pieces) * 16;
  } else {
    t = id / p.pieces;
    off = (id - t * p.pieces) * 16;
  }
}

// One thread copies one 16-byte piece of a token's row to all its sorted rows, so
// x is read once however large top_k.  Bound by the stores: 16384 x top 10 rows
// of 2048 bf16, 738 MB, 109 us (100 % of the copy bandwidth).
__global__ void __launch_bounds__(kCopyThreads) dispatch_kernel(const RowParams p) {
  griddep_launch_dependents();
  int64_t t, off;
  piece_of(p, static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x, t, off);
  // x is read while the sort runs, which let this kernel start only after what
  // came before it had ended (from L2: no line that an earlier kernel left in L1).
  uint4 v = {};
  if (t < p.n_tokens) v = __ldcg(reinterpret_cast<const uint4 *>(p.x + t * p.ld + off));
  griddep_wait();
  if (t >= p.n_tokens) return;
  for (int k = 0; k < p.top_k; ++k) {
    const int64_t i = t * p.top_k + k;
    if (i >= p.n_slots) break;
    const int r = p.pos[i];
    if (r < 0) continue;
    *reinterpret_cast<uint4 *>(p.out + r * p.row_bytes + off) = v;
    if (off == 0) p.src[r] = static_cast<int32_t>(i);
  }
  for (int64_t r = *p.rows_held + t; r < p.n_slots; r += p.n_tokens)  // rows of no cell
    *reinterpret_cast<uint4 *>(p.out + r * p.row_bytes + off) = make_uint4(0, 0, 0, 0);
}

// Sort and copy of a small batch in one launch: a CTA per token finds its
// slots' rows by counting, over all slots, those of lower cells and the
// earlier ones of the same cell, so nothing waits for a sort.  One more CTA
// writes expert_offsets.  Every CTA reads all slots once for every 8 of its own:
// it pays while a second launch costs more.  Rows of 2048 bf16, this way and with
// a sort before: 64 x top 8 3.0 and 5.1 us, 256 x 8 6.1 and 6.5, 1024 x 8 22 and
// 10.7; 512 x top 1 3.2 and 4.4, 1024 x 1 5.9 and 5.0; 724 x 2 6.0 and 5.7;
// 128 x 16 9.7 and 7.2.
__global__ void __launch_bounds__(kCopyThreads) dispatch_small_kernel(const SortParams s,
                                                                      const RowParams p) {
  extern __shared__ uint32_t smem[];  // the last CTA's histogram
  constexpr int kGroup = kSmallGroup;  // slots counted at a time
  constexpr int kW = kCopyThreads / 32;
  __shared__ int part[kW][kGroup];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (static_cast<int>(blockIdx.x) == p.n_tokens) {
    const int bins = s.cells + 1;
    for (int c = tid; c < bins; c += kCopyThreads) smem[c] = 0;
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    for (int i = tid; i < s.n_slots; i += 4 * kCopyThreads) {
      int bin[4];
      slot_bins(s, i, kCopyThreads, s.n_slots, bin);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (bin[k] <= s.cells) atomicAdd(smem + bin[k], 1u);
    }
    __syncthreads();
    uint32_t carry = 0;
    for (int base = 0; base < bins; base += kCopyThreads) {
      const int c = base + tid;
      const uint32_t n = c < bins ? smem[c] : 0u;
      uint32_t incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(kFullWarp, incl, o);
        if (lane >= o) incl += v;
      }
      if (base > 0) __syncthreads();  // part is read
      if (lane == 31) part[warp][0] = static_cast<int>(incl);
      __syncthreads();
      const uint32_t w_total = lane < kW ? static_cast<uint32_t>(part[lane][0]) : 0u;
      const uint32_t w_before = __reduce_add_sync(kFullWarp, lane < warp ? w_total : 0u);
      if (c < bins) s.offsets[c] = static_cast<int32_t>(carry + w_before + incl - n);
      carry += __reduce_add_sync(kFullWarp, w_total);
    }
    return;
  }
  griddep_wait();
  griddep_launch_dependents();
  const int t = blockIdx.x;
  const uint8_t *row = p.x + t * p.ld;
  for (int k0 = 0; k0 < p.top_k; k0 += kGroup) {
    const int i0 = t * p.top_k + k0;
    const int n = min(kGroup, min(p.top_k - k0, p.n_slots - i0));
    if (n <= 0) break;
    int mine[kGroup], count[kGroup];
#pragma unroll
    for (int k = 0; k < kGroup; ++k) count[k] = 0;
    slot_bins(s, i0, 1, i0 + n, mine);
    for (int j0 = tid; j0 < s.n_slots; j0 += 2 * kCopyThreads) {
      int bin[2];  // past the end: above every cell
      slot_bins(s, j0, kCopyThreads, s.n_slots, bin);
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int k = 0; k < kGroup; ++k)  // below mine, or the same and earlier
          count[k] += bin[q] < mine[k] + (j0 + q * kCopyThreads < i0 + k ? 1 : 0) ? 1 : 0;
    }
    if (k0 > 0) __syncthreads();  // part is read
#pragma unroll
    for (int k = 0; k < kGroup; ++k) {
      const int sum = __reduce_add_sync(kFullWarp, count[k]);
      if (lane == 0) part[warp][k] = sum;
    }
    __syncthreads();
    int at[kGroup];
#pragma unroll
    for (int k = 0; k < kGroup; ++k) {
      at[k] = 0;
#pragma unroll
      for (int w = 0; w < kW; ++w) at[k] += part[w][k];
    }
    if (tid == 0)
#pragma unroll
      for (int k = 0; k < kGroup; ++k)
        if (k < n) {
          s.src[at[k]] = i0 + k;
          s.pos[i0 + k] = mine[k] < s.cells ? at[k] : -1;
        }
    for (int c = tid; c < p.pieces; c += kCopyThreads) {
      const uint4 v = *reinterpret_cast<const uint4 *>(row + c * 16);
#pragma unroll
      for (int k = 0; k < kGroup; ++k)
        if (k < n)
          *reinterpret_cast<uint4 *>(p.out + at[k] * p.row_bytes + c * 16) =
              mine[k] < s.cells ? v : make_uint4(0, 0, 0, 0);
    }
  }
}

// One thread sums one 16-byte piece of a token's rows, kBatch rows in flight
// (one after the other: 162 us).  Bound by HBM: 16384 x top 10 rows of 2048 bf16,
// 739 MB, 115 us, 95 % of the copy bandwidth.
template <typename T>
__global__ void __launch_bounds__(kCopyThreads) combine_kernel(const RowParams p) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int N = Piece<T>::kN, kBatch = 5;
  int64_t t, off;
  piece_of(p, static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x, t, off);
  if (t >= p.n_tokens) return;
  float acc[N] = {};
  const int64_t i0 = t * p.top_k;
  for (int k0 = 0; k0 < p.top_k; k0 += kBatch) {
    uint4 v[kBatch];
    float w[kBatch];
    bool there[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const bool in = k0 + k < p.top_k;
      const int64_t r = !in ? -1 : p.pos ? p.pos[i0 + k0 + k] : i0 + k0 + k;
      there[k] = r >= 0 && r < p.n_rows;
      w[k] = in && p.weights ? p.weights[i0 + k0 + k] : 1.0f;
      v[k] = make_uint4(0, 0, 0, 0);
      if (there[k]) v[k] = __ldcs(reinterpret_cast<const uint4 *>(p.x + r * p.row_bytes + off));
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (!there[k]) continue;
      float f[N];
      Piece<T>::load(v[k], f);
#pragma unroll
      for (int j = 0; j < N; ++j) acc[j] += w[k] * f[j];
    }
  }
  *reinterpret_cast<uint4 *>(p.out + t * p.ld + off) = Piece<T>::store(acc);
}

// One CTA per token, kGradBatch slots at a time: the pieces of dout are read
// once a batch, the rows of y are in flight together, and the dot products are
// summed over the CTA in a fixed order.  Bound by HBM: 4001 x top 8 rows of 2048
// bf16, 278 MB, 45 us, 91 % of the copy bandwidth.
template <typename T>
__global__ void __launch_bounds__(kGradThreads) combine_backward_kernel(const RowParams p) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int N = Piece<T>::kN;
  __shared__ float part[2][kGradThreads / 32][kGradBatch];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int threads = blockDim.x, warps = threads >> 5;
  const int64_t t = blockIdx.x;
  const uint8_t *dout = p.dout + t * p.ld;
  const int top_k = t < p.n_tokens ? p.top_k : 0;  // no tokens: one CTA, for the zeros
  for (int k0 = 0, turn = 0; k0 < top_k; k0 += kGradBatch, turn ^= 1) {
    const int64_t i0 = t * p.top_k + k0;
    int64_t at[kGradBatch];  // byte offset of the slot's row, negative: none
    float w[kGradBatch], dot[kGradBatch];
#pragma unroll
    for (int k = 0; k < kGradBatch; ++k) {
      const bool in = k0 + k < p.top_k;
      const int64_t r = !in ? -1 : p.pos ? p.pos[i0 + k] : i0 + k;
      at[k] = r >= 0 && r < p.n_rows ? r * p.row_bytes : -1;
      w[k] = in && p.weights ? p.weights[i0 + k] : 1.0f;
      dot[k] = 0.0f;
    }
    for (int c = tid; c < p.pieces; c += threads) {
      const uint4 dv = *reinterpret_cast<const uint4 *>(dout + c * 16);
      uint4 yv[kGradBatch];
      if (p.dweights) {
#pragma unroll
        for (int k = 0; k < kGradBatch; ++k) {
          yv[k] = make_uint4(0, 0, 0, 0);
          if (at[k] >= 0) yv[k] = __ldcs(reinterpret_cast<const uint4 *>(p.x + at[k] + c * 16));
        }
      }
      float d[N];
      Piece<T>::load(dv, d);
#pragma unroll
      for (int k = 0; k < kGradBatch; ++k) {
        if (at[k] < 0) continue;
        float f[N];
        if (p.dweights) {
          Piece<T>::load(yv[k], f);
#pragma unroll
          for (int j = 0; j < N; ++j) dot[k] += d[j] * f[j];
        }
#pragma unroll
        for (int j = 0; j < N; ++j) f[j] = w[k] * d[j];
        *reinterpret_cast<uint4 *>(p.dy + at[k] + c * 16) = Piece<T>::store(f);
      }
    }
    if (p.dweights) {
#pragma unroll
      for (int k = 0; k < kGradBatch; ++k) {
        const float sum = warp_sum(dot[k]);
        if (lane == 0) part[turn][warp][k] = sum;
      }
      if (warps > 1) __syncthreads(); else __syncwarp();
      if (tid < kGradBatch && k0 + tid < p.top_k) {
        float sum = 0.0f;
        for (int v = 0; v < warps; ++v) sum += part[turn][v][tid];
        p.dweights[i0 + tid] = sum;
      }
    }
  }
  if (p.rows_held)
    for (int64_t r = max(*p.rows_held, 0) + t; r < p.n_rows; r += gridDim.x)
      for (int c = tid; c < p.pieces; c += threads)
        *reinterpret_cast<uint4 *>(p.dy + r * p.row_bytes + c * 16) = make_uint4(0, 0, 0, 0);
}

mlg_status check_sort(int32_t n_slots, int32_t top_k, int32_t n_experts, const void *row_adapter,
                      int32_t n_adapters, int64_t *cells) {
  if (n_slots < 0 || top_k < 1 || n_experts < 0 || n_adapters < 1) return MLG_ERR_INVALID_ARG;
  *cells = static_cast<int64_t>(n_experts) * (row_adapter ? n_adapters : 1);
  return *cells > MLG_SORT_MAX_CELLS ? MLG_ERR_UNSUPPORTED : MLG_OK;
}

// Rows of `width` elements of `type` and their token rows' stride `ld`.
mlg_status check_rows(int32_t type, int32_t width, int64_t ld, int32_t top_k) {
  if (!known_type(type) || width < 1 || ld < width || top_k < 1) return MLG_ERR_INVALID_ARG;
  const int64_t n = 16 / static_cast<int64_t>(type_size(type));
  return width % n != 0 || ld % n != 0 ? MLG_ERR_UNSUPPORTED : MLG_OK;
}

SortParams sort_params(const int32_t *indices, const int32_t *row_adapter, int32_t *offsets,
                       int32_t *src, int32_t *pos, int32_t n_slots, int32_t top_k,
                       int32_t n_experts, int32_t n_adapters, int64_t cells) {
  SortParams p = {};
  p.indices = indices;
  p.row_adapter = row_adapter;
  p.offsets = offsets;
  p.src = src;
  p.pos = pos;
  p.n_slots = n_slots;
  p.top_k = top_k;
  p.n_experts = n_experts;
  p.n_adapters = n_adapters;
  p.cells = static_cast<int32_t>(cells);
  p.all_src = 1;
  p.bits = 1;
  while ((cells + 2) > (int64_t{1} << p.bits)) ++p.bits;  // bins 0..cells, and one past the end
  return p;
}

}  // namespace
}  // namespace mlg

extern "C" {

mlg_status mlg_sort_slots(const int32_t *indices, const int32_t *row_adapter,
                          int32_t *expert_offsets, int32_t *src, int32_t *pos, int32_t n_slots,
                          int32_t top_k, int32_t n_experts, int32_t n_adapters, void *stream) {
  using namespace mlg;
  int64_t cells = 0;
  const mlg_status st = check_sort(n_slots, top_k, n_experts, row_adapter, n_adapters, &cells);
  if (st != MLG_OK) return st;
  if (!expert_offsets || (n_slots > 0 && (!indices || !src || !pos))) return MLG_ERR_INVALID_ARG;
  SortParams p = sort_params(indices, row_adapter, expert_offsets, src, pos, n_slots, top_k,
                             n_experts, n_adapters, cells);
  return cuda_status(launch_sort(p, static_cast<cudaStream_t>(stream)));
}

mlg_status mlg_dispatch(const void *x, int32_t type, int64_t ld_x, const int32_t *indices,
                        const int32_t *row_adapter, int32_t *expert_offsets, int32_t *src,
                        int32_t *pos, void *x_rows, int32_t n_slots, int32_t width, int32_t top_k,
                        int32_t n_experts, int32_t n_adapters, void *stream) {
  using namespace mlg;
  int64_t cells = 0;
  mlg_status st = check_rows(type, width, ld_x, top_k);
  if (st != MLG_OK) return st;
  st = check_sort(n_slots, top_k, n_experts, row_adapter, n_adapters, &cells);
  if (st != MLG_OK) return st;
  if (!expert_offsets || (n_slots > 0 && (!x || !x_rows || !indices || !src || !pos)))
    return MLG_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(x_rows)) return MLG_ERR_UNSUPPORTED;
  SortParams sp = sort_params(indices, row_adapter, expert_offsets, src, pos, n_slots, top_k,
                              n_experts, n_adapters, cells);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (n_slots == 0) return cuda_status(launch_sort(sp, s));
  RowParams p = {};
  p.x = static_cast<const uint8_t *>(x);
  p.out = static_cast<uint8_t *>(x_rows);
  p.pos = pos;
  p.rows_held = expert_offsets + cells;
  p.src = src;
  p.ld = ld_x * type_size(type);
  p.row_bytes = static_cast<int64_t>(width) * type_size(type);
  p.pieces = static_cast<int32_t>(p.row_bytes / 16);
  p.n_tokens = (n_slots - 1) / top_k + 1;
  p.n_slots = n_slots;
  p.top_k = top_k;
  const int64_t compared = int64_t{n_slots} * ((top_k - 1) / kSmallGroup + 1);  // by a CTA
  if (compared <= kSmallSlots && compared * p.n_tokens <= kSmallWork && cells <= kSmallCells)
    return cuda_status(launch_early(dispatch_small_kernel, p.n_tokens + 1, kCopyThreads,
                                    (cells + 1) * sizeof(uint32_t), 1, s, sp, p));
  sp.all_src = 0;
  st = cuda_status(launch_sort(sp, s));
  if (st != MLG_OK) return st;
  const int64_t grid = (static_cast<int64_t>(p.n_tokens) * p.pieces + kCopyThreads - 1) /
                       kCopyThreads;
  if (grid > 0x7fffffff) return MLG_ERR_UNSUPPORTED;
  return cuda_status(launch_early(dispatch_kernel, grid, kCopyThreads, 0, 1, s, p));
}

mlg_status mlg_combine(const void *y_rows, int32_t type, const int32_t *pos, const float *weights,
                       void *out, int64_t ld_out, int32_t n_tokens, int32_t width, int32_t top_k,
                       int32_t n_rows, void *stream) {
  using namespace mlg;
  const mlg_status st = check_rows(type, width, ld_out, top_k);
  if (st != MLG_OK) return st;
  if (n_tokens < 0 || n_rows < 0) return MLG_ERR_INVALID_ARG;
  if (static_cast<int64_t>(n_tokens) * top_k > 0x7fffffff) return MLG_ERR_UNSUPPORTED;
  if (n_tokens == 0) return MLG_OK;
  if (!out || (n_rows > 0 && !y_rows)) return MLG_ERR_INVALID_ARG;
  if (!aligned16(y_rows) || !aligned16(out)) return MLG_ERR_UNSUPPORTED;
  RowParams p = {};
  p.x = static_cast<const uint8_t *>(y_rows);
  p.out = static_cast<uint8_t *>(out);
  p.pos = pos;
  p.weights = weights;
  p.ld = ld_out * type_size(type);
  p.row_bytes = static_cast<int64_t>(width) * type_size(type);
  p.pieces = static_cast<int32_t>(p.row_bytes / 16);
  p.n_tokens = n_tokens;
  p.n_rows = n_rows;
  p.top_k = top_k;
  const int64_t grid = (static_cast<int64_t>(n_tokens) * p.pieces + kCopyThreads - 1) /
                       kCopyThreads;
  if (grid > 0x7fffffff) return MLG_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(type == MLG_TYPE_BF16
                         ? launch_early(combine_kernel<__nv_bfloat16>, grid, kCopyThreads, 0, 1,
                                        s, p)
                         : launch_early(combine_kernel<float>, grid, kCopyThreads, 0, 1, s, p));
}

mlg_status mlg_combine_backward(const void *dout, int32_t type, int64_t ld_dout,
                                const void *y_rows, const int32_t *pos, const float *weights,
                                const int32_t *rows_held, void *dy_rows, float *dweights,
                                int32_t n_tokens, int32_t width, int32_t top_k, int32_t n_rows,
                                void *stream) {
  using namespace mlg;
  const mlg_status st = check_rows(type, width, ld_dout, top_k);
  if (st != MLG_OK) return st;
  if (n_tokens < 0 || n_rows < 0) return MLG_ERR_INVALID_ARG;
  if (static_cast<int64_t>(n_tokens) * top_k > 0x7fffffff) return MLG_ERR_UNSUPPORTED;
  if (n_tokens == 0 && (n_rows == 0 || !rows_held)) return MLG_OK;
  if ((n_tokens > 0 && !dout) || (n_rows > 0 && (!dy_rows || (dweights && !y_rows))))
    return MLG_ERR_INVALID_ARG;
  if (!aligned16(dout) || !aligned16(dy_rows) || (dweights && !aligned16(y_rows)))
    return MLG_ERR_UNSUPPORTED;
  RowParams p = {};
  p.x = static_cast<const uint8_t *>(y_rows);
  p.dout = static_cast<const uint8_t *>(dout);
  p.dy = static_cast<uint8_t *>(dy_rows);
  p.pos = pos;
  p.weights = weights;
  p.rows_held = rows_held;
  p.dweights = dweights;
  p.ld = ld_dout * type_size(type);
  p.row_bytes = static_cast<int64_t>(width) * type_size(type);
  p.pieces = static_cast<int32_t>(p.row_bytes / 16);
  p.n_tokens = n_tokens;
  p.n_rows = n_rows;
  p.top_k = top_k;
  // Two pieces a thread where the row has them.
  const int threads = std::min(kGradThreads, (p.pieces + 63) / 64 * 32);
  const int grid = std::max(n_tokens, 1);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(
      type == MLG_TYPE_BF16
          ? launch_early(combine_backward_kernel<__nv_bfloat16>, grid, threads, 0, 1, s, p)
          : launch_early(combine_backward_kernel<float>, grid, threads, 0, 1, s, p));
}

}  // extern "C"
