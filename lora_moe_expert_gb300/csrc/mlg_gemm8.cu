// mlg_gemm8.cu -- the expert product of expert-sorted rows in e4m3, with an
// fp32 scale for each 128 values of a row and each 128 x 128 block of a weight.
//
//     out[r, n] = sum_b sx[r, b] sw[e, n / 128, b] (sum_{k in b} x[r, k] w[e, n, k])
//
// The scale of a partial sum differs from row to row and from block to block,
// so it cannot go into the tensor core's accumulator: the 128-wide partial sums
// are taken out of TMEM and summed, scaled, in registers.  That fixes the tile:
// 128 rows x 256 columns of fp32 are half of an SM's registers.
//
// One CTA per SM, persistent over units (a tile of at most 128 rows of one
// expert, 256 output columns), dealt round-robin, the columns of a tile to
// neighbours (they share its x in L2, the tiles of an expert its weights):
//  * warp 1 fills a ring of stages: 128 k of x (boxes of 32 rows, as many as the
//    tile has) and of 256 weight rows, 128-byte swizzled TMA boxes;
//  * warp 0 issues tcgen05.mma (kind::f8f6f4, M 128, N 256 or twice 128, K 32), four
//    a stage, each stage into the other one of two TMEM accumulators;
//  * warps 4-11 (32 rows x 128 columns each) wait for an accumulator, read it in
//    pieces of 32 columns and add scale * piece (two columns an instruction);
//    at the end of a unit they round once and store as the GEMM with the fold
//    does: whole 32-row boxes by TMA, others row by row.  Warps without rows only
//    take part in the barriers, so a tile of few rows costs little but its bytes.
// What bounds it: weights of few rows come at 83 % of the copy bandwidth (512 rows of 128 experts,
// k 768, n 2048: 35.5 us); in full tiles the loads (48 KB a stage, 16 TB/s from L2 at most),
// the products and the sums take about as long as one another and overlap as far as two
// accumulators and the ring let them (30720 rows, k 2048, n 1536: 121 us, 1.6 PFLOP/s, without
// products or without sums 106; 163840 rows of 512 experts, k 512, n 2048: 260 us, 5.0 TB/s; dense
// 8192 x 4096 x 4096: 112 us, 2.4 PFLOP/s).
// Every wait is bounded; a timeout sets an error bit and the CTA drains its copies.
#include <cuda.h>

#include <mutex>

#include "mlg_launch.cuh"
#include "mlg_tiles.cuh"
#include "mlg_tmap.cuh"

namespace mlg {
namespace {

constexpr int kThreads8 = 384;
constexpr int kEpiWarps8 = 8;
constexpr int kTileM8 = 128, kTileN8 = 256, kBlockK8 = MLG_F8_BLOCK;
constexpr uint32_t kXBytes8 = kTileM8 * kBlockK8, kWBytes8 = kTileN8 * kBlockK8;
constexpr uint32_t kStageBytes8 = kXBytes8 + kWBytes8;
constexpr uint32_t kOutBox8 = 32 * 64;  // 32 rows x 32 bf16 columns, 64-byte swizzle
constexpr int kListed8 = 128;           // units of a CTA that are looked up before all else
constexpr uint32_t kSmemLimit8 = 227 * 1024 - 1024;
// Registers: 384 threads x 168 at launch = 128 x 40 + 256 x 232.
constexpr int kRegsFew = 40, kRegsMany = 232;
static_assert(128 * kRegsFew + 256 * kRegsMany <= kThreads8 * 168, "register split");

// Two plans.  STORES is for short sums over full tiles, whose time goes into the results as
// much as into the products: a stage less, four boxes of results under way in place of one,
// and a stage's product in two parts of 128 columns, each with its own barriers, so that
// the warps of the first part take it out of TMEM while the second is being computed.
// The other plan is for the rest: small tiles have few whole boxes and wait for weights, and in
// long sums a product of 256 columns (128 cycles) reads the tile of x once, not twice.
// STORES and the other, in us, 128 experts where nothing else is said: k 512, 163840 rows of 512
// experts 260 and 288; k 768, 30720 rows 77 and 80, 8192 42.2 and 42.3, 4096 39.4 and 39.3,
// 2048 37.9 and 37.3, 512 36.8 and 36.1, 8 7.4 and 7.1; k 1024, 30720 rows 73.9 and 74.2;
// k 2048, 30720 rows 125 and 120.
template <bool STORES>
struct Plan8 {
  static constexpr int kStages = STORES ? 3 : 4, kOutBoxes = STORES ? 4 : 1;
  static constexpr int kParts = STORES ? 2 : 1;
  static constexpr uint32_t kOffList =
      kStages * kStageBytes8 + kEpiWarps8 * kOutBoxes * kOutBox8;
  static constexpr uint32_t kOffTab = kOffList + kListed8 * 16;
  static_assert(kOffTab + (MLG_F8_MAX_EXPERTS + 1) * 4 + 1024 <= kSmemLimit8, "shared memory");
};

// Rows, columns and values of k are counted in 32 bits, up to a tile past the last one, and are
// coordinates of TMA boxes.
static_assert(MLG_F8_MAX_ROWS <= INT32_MAX / 2 + 1 && MLG_F8_MAX_WIDTH <= INT32_MAX / 2, "sizes");

static __device__ uint32_t g_gemm8_errors;
int g_gemm8_lose = 0;  // mlg_test_set_knob

struct Gemm8Params {
  const int32_t *offsets;
  const float *x_scales, *w_scales;
  uint8_t *out;
  int32_t k_in, n_out, n_experts, row_offset, row_end, win, tile_m;
  int32_t kb_count, nc_count, nb_count;  // blocks along k, 256-column chunks, blocks along n
  int32_t v8;                            // output rows 32-byte aligned
  uint32_t w_bytes;                      // what a stage waits for of the weights: kWBytes8
};

struct Ctl8 {
  uint64_t full[4], empty[4], acc_full[2][2], acc_empty[2][2], drain;
  uint32_t tmem_base;
  volatile int abort_flag;
  int warp_total[kThreads8 / 32];
};

__device__ __forceinline__ bool wait8(Ctl8 &ctl, uint64_t &bar, uint32_t parity) {
  return wait_or_abort(ctl, bar, parity, &g_gemm8_errors);
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *tmap, int32_t x, int32_t y,
                                            int32_t z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// kind::f8f6f4, both operands e4m3, fp32 accumulators, K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}
__device__ __forceinline__ void umma_e4m3_if(bool leader, uint32_t d_tmem, uint64_t a_desc,
                                             uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, l;\n\t"
      "setp.ne.b32 l, %5, 0;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@l tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(static_cast<uint32_t>(leader))
      : "memory");
}
__device__ __forceinline__ void umma_commit_if(bool leader, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred l;\n\t"
      "setp.ne.b32 l, %1, 0;\n\t"
      "@l tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          bar),
      "r"(static_cast<uint32_t>(leader))
      : "memory");
}

// 32 lanes x 32 consecutive columns; complete after tmem_wait_ld().
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
      "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// (a.x, a.y) += s * (lo, hi)
__device__ __forceinline__ void fma2(uint64_t &a, uint32_t lo, uint32_t hi, uint64_t s) {
  asm("{\n\t.reg .b64 v;\n\t"
      "mov.b64 v, {%1, %2};\n\t"
      "fma.rn.f32x2 %0, v, %3, %0;\n\t}"
      : "+l"(a)
      : "r"(lo), "r"(hi), "l"(s));
}
__device__ __forceinline__ uint32_t round_pair(uint64_t a) {
  return pack_bf16x2(__uint_as_float(static_cast<uint32_t>(a)),
                     __uint_as_float(static_cast<uint32_t>(a >> 32)));
}

// All but the last N of this thread's bulk stores have been read from shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void store_v4(void *p, const uint32_t *v) {
  asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}
// One whole 32-byte sector (address 32-byte aligned).
__device__ __forceinline__ void store_v8(void *p, const uint32_t *v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

struct alignas(16) Unit8 {
  int e, r0, r1, n0;
};

__device__ __forceinline__ Unit8 unit_of(const Gemm8Params &p, const int *tile_start, int u) {
  const int t = u / p.nc_count;
  const TileInfo ti = tile_info(p, tile_start, p.n_experts, t);
  return Unit8{ti.e, ti.r0, ti.r1, (u - t * p.nc_count) * kTileN8};
}

// A CTA's unit i, of its list where that is so long.
__device__ __forceinline__ Unit8 unit_at(const Gemm8Params &p, const int *tile_start,
                                         const Unit8 *list, int i) {
  return i < kListed8 ? list[i] : unit_of(p, tile_start, blockIdx.x + i * gridDim.x);
}

template <bool STORES>
__global__ void __launch_bounds__(kThreads8, 1)
    gemm8_kernel(const __grid_constant__ CUtensorMap tmap_x,
                 const __grid_constant__ CUtensorMap tmap_w,
                 const __grid_constant__ CUtensorMap tmap_out, const Gemm8Params p) {
  constexpr int kStages8 = Plan8<STORES>::kStages, kOutBoxes8 = Plan8<STORES>::kOutBoxes;
  constexpr int kParts8 = Plan8<STORES>::kParts, kPartN8 = kTileN8 / kParts8;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Ctl8 ctl;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int *tile_start = reinterpret_cast<int *>(smem + Plan8<STORES>::kOffTab);  // [n_experts + 1]

  if (tid == 0) {
    for (int s = 0; s < kStages8; ++s) {
      mbar_init(smem_addr(&ctl.full[s]), 1);
      mbar_init(smem_addr(&ctl.empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b)
      for (int h = 0; h < kParts8; ++h) {
        mbar_init(smem_addr(&ctl.acc_full[b][h]), 1);
        mbar_init(smem_addr(&ctl.acc_empty[b][h]), kEpiWarps8 / kParts8);
      }
    mbar_init(smem_addr(&ctl.drain), 1);
    ctl.abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmap_x);
    prefetch_tmap(&tmap_w);
    prefetch_tmap(&tmap_out);
  }
  __syncthreads();
  if (warp == 0) {
    tmem_alloc(smem_addr(&ctl.tmem_base), 512);
    tmem_relinquish();
  }
  griddep_wait();
  griddep_launch_dependents();

  // tile_start: exclusive prefix over the experts' tiles
  int carry = 0;
  for (int base = 0; base < p.n_experts; base += kThreads8) {
    const int e = base + tid;
    const int n = e < p.n_experts ? span_tiles(p, span_lo(p, e), span_hi(p, e)) : 0;
    int incl = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(kFullWarp, incl, d);
      if (lane >= d) incl += v;
    }
    if (lane == 31) ctl.warp_total[warp] = incl;
    __syncthreads();
    int before = carry;
    for (int w = 0; w < kThreads8 / 32; ++w) {
      if (w < warp) before += ctl.warp_total[w];
      carry += ctl.warp_total[w];
    }
    if (e < p.n_experts) tile_start[e] = before + incl - n;
    __syncthreads();
  }
  if (tid == 0) tile_start[p.n_experts] = carry;
  __syncthreads();
  const int units = tile_start[p.n_experts] * p.nc_count, G = static_cast<int>(gridDim.x);
  Unit8 *list = reinterpret_cast<Unit8 *>(smem + Plan8<STORES>::kOffList);
  if (tid < kListed8 && static_cast<int>(blockIdx.x) + tid * G < units)
    list[tid] = unit_of(p, tile_start, blockIdx.x + tid * G);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem_base, ring = smem_addr(smem);
  const int kbs = p.kb_count;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew));
    if (warp == 0) {
      // ============================================================ MMA issuer
      // The whole warp goes along in uniform control flow, and the instructions are one
      // lane's by their predicate: addresses and descriptors stay in uniform registers.
      // (Issued from a branch of one lane, an MMA of 256 columns takes 149 cycles with its
      // commits, elected anew each time 131, of which the product is 128; one of 128
      // columns 115 or, so, little more than its 64.)
      const bool leader = elect_one();
      const uint64_t desc = umma_desc_sw128(ring);
      uint32_t it = 0;
      for (int u = blockIdx.x; u < units; u += G) {
        const int n0 = u % p.nc_count * kTileN8;
        for (int kb = 0; kb < kbs; ++kb, ++it) {
          const int st = it % kStages8, b = it & 1;
          const uint64_t ad = desc + st * (kStageBytes8 >> 4), bd = ad + (kXBytes8 >> 4);
          const int steps = min(4, (p.k_in - kb * kBlockK8 + 31) / 32);
          bool ready = wait8(ctl, ctl.full[st], (it / kStages8) & 1);
#pragma unroll
          for (int h = 0; h < kParts8; ++h) {
            ready = ready && wait8(ctl, ctl.acc_empty[b][h], ((it >> 1) & 1) ^ 1);
            if (!__all_sync(kFullWarp, ready)) goto mma_done;
            tc_fence_after();
            const int cols = min(kPartN8, (p.n_out - n0 - h * kPartN8 + 15) / 16 * 16);
            if (cols > 0) {
              // d: all of TMEM is this CTA's, so its columns begin at 0
              const uint32_t idesc = idesc_e4m3(kTileM8, cols), d = b * kTileN8 + h * kPartN8;
              const uint64_t w = bd + h * (kPartN8 * kBlockK8 >> 4);
              umma_e4m3_if(leader, d, ad, w, idesc, 0);
              if (steps > 1) umma_e4m3_if(leader, d, ad + 2, w + 2, idesc, 1);
              if (steps > 2) umma_e4m3_if(leader, d, ad + 4, w + 4, idesc, 1);
              if (steps > 3) umma_e4m3_if(leader, d, ad + 6, w + 6, idesc, 1);
            }
            umma_commit_if(leader, smem_addr(&ctl.acc_full[b][h]));
          }
          umma_commit_if(leader, smem_addr(&ctl.empty[st]));
        }
      }
    mma_done:
      umma_commit_if(leader, smem_addr(&ctl.drain));
      mbar_wait_bounded(smem_addr(&ctl.drain), 0);
    } else if (warp == 1 && lane == 0) {
      // ============================================================ ring fill
      uint32_t it = 0;
      for (int u = blockIdx.x, i = 0; u < units; u += G, ++i) {
        const Unit8 m = unit_at(p, tile_start, list, i);
        const int boxes = (m.r1 - m.r0 + 31) / 32;
        for (int kb = 0; kb < kbs; ++kb, ++it) {
          const int st = it % kStages8;
          if (!wait8(ctl, ctl.empty[st], ((it / kStages8) & 1) ^ 1)) goto fill_done;
          const uint32_t full = smem_addr(&ctl.full[st]), xs = ring + st * kStageBytes8;
          mbar_arrive_expect_tx(full, p.w_bytes + boxes * 32 * kBlockK8);
          tma_load_3d(xs + kXBytes8, &tmap_w, kb * kBlockK8, m.n0, m.e, full);
          for (int b = 0; b < boxes; ++b)
            tma_load_2d(xs + b * 32 * kBlockK8, &tmap_x, kb * kBlockK8, m.r0 + 32 * b, full);
        }
      }
    fill_done:
      // what was asked for and never used: let it land
      const uint64_t t0 = global_timer_ns();
      for (uint32_t k = 0; k < kStages8 && k < it; ++k) {
        const uint32_t j = it - 1 - k;
        mbar_wait_until(smem_addr(&ctl.full[j % kStages8]), (j / kStages8) & 1, t0);
      }
    }
    __syncwarp();
  } else {
    // ================================================================ epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMany));
    const int ew = warp - 4, quarter = warp & 3, half = ew >> 2, part = half * kParts8 / 2;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * 128;
    uint8_t *stages = smem + kStages8 * kStageBytes8 + ew * kOutBoxes8 * kOutBox8;
    uint32_t it = 0;
    // The two scales of the next block of k, asked for a block ahead (the next unit's
    // first too): each is a trip to L2 or HBM.
    const float *sx = nullptr, *sw = nullptr;
    float next_x = 0.0f, next_w = 0.0f;
    auto ask_first = [&](int i) {
      const Unit8 m = unit_at(p, tile_start, list, i);
      const int block = min((m.n0 >> 7) + half, p.nb_count - 1);
      sx = p.x_scales + int64_t{min(m.r0 + quarter * 32 + lane, m.r1 - 1)} * kbs;
      sw = p.w_scales + (int64_t{m.e} * p.nb_count + block) * kbs;
      next_x = __ldg(sx), next_w = __ldg(sw);
    };
    if (static_cast<int>(blockIdx.x) < units) ask_first(0);
    for (int u = blockIdx.x, i = 0; u < units; u += G, ++i) {
      const Unit8 m = unit_at(p, tile_start, list, i);
      const int row = m.r0 + quarter * 32 + lane, col0 = m.n0 + half * 128;
      const bool valid = row < m.r1;
      const bool busy = m.r0 + quarter * 32 < m.r1 && col0 < p.n_out;
      if (!busy) {
        for (int kb = 0; kb < kbs; ++kb, ++it) {
          const int b = it & 1;
          if (!wait8(ctl, ctl.acc_full[b][part], (it >> 1) & 1)) goto epi_done;
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&ctl.acc_empty[b][part]));
        }
        if (u + G < units) ask_first(i + 1);
        continue;
      }
      uint64_t acc[64];
#pragma unroll
      for (int c = 0; c < 64; ++c) acc[c] = 0;
      for (int kb = 0; kb < kbs; ++kb, ++it) {
        const int b = it & 1;
        const float s = next_x * next_w;
        uint64_t s2;
        asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "f"(s));
        if (kb + 1 < kbs)
          next_x = __ldg(++sx), next_w = __ldg(++sw);
        else if (u + G < units)
          ask_first(i + 1);
        if (!wait8(ctl, ctl.acc_full[b][part], (it >> 1) & 1)) goto epi_done;
        tc_fence_after();
        uint32_t v[2][32];
        tmem_ld32(lane_addr + b * 256, v[0]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c < 3) tmem_ld32(lane_addr + b * 256 + (c + 1) * 32, v[(c + 1) & 1]);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            fma2(acc[c * 16 + i], v[c & 1][2 * i], v[c & 1][2 * i + 1], s2);
          if (c < 3) tmem_wait_ld();
          if (c == 2) {  // the last piece is in registers
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&ctl.acc_empty[b][part]));
          }
        }
      }
      uint32_t packed[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) packed[i] = round_pair(acc[i]);
      if (m.r0 + quarter * 32 + 32 <= m.r1) {  // whole boxes; TMA clips columns past n_out
#pragma unroll
        for (int bx = 0; bx < 4; ++bx) {
          if (col0 + bx * 32 >= p.n_out) break;
          if (lane == 0) bulk_wait_read<kOutBoxes8 - 1>();  // the last box of this buffer has left
          __syncwarp();
          uint8_t *stage = stages + bx % kOutBoxes8 * kOutBox8;
#pragma unroll
          for (int cc = 0; cc < 4; ++cc)
            *reinterpret_cast<uint4 *>(stage + lane * 64 + ((cc ^ ((lane >> 1) & 3)) << 4)) =
                make_uint4(packed[bx * 16 + 4 * cc], packed[bx * 16 + 4 * cc + 1],
                           packed[bx * 16 + 4 * cc + 2], packed[bx * 16 + 4 * cc + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tmap_out, col0 + bx * 32, m.r0 + quarter * 32, smem_addr(stage));
            bulk_commit();
          }
        }
        // Empty groups for the boxes that n_out cuts off: the wait counts groups, and a buffer's
        // last box is past the newest kOutBoxes8 - 1 only if every unit leaves as many as buffers.
        if (kOutBoxes8 > 1 && lane == 0)
          for (int c = col0 + 96; c >= p.n_out; c -= 32) bulk_commit();
      } else if (valid) {
        uint8_t *to = p.out + (int64_t{row} * p.n_out + col0) * 2;
        if (p.v8) {
#pragma unroll
          for (int cc = 0; cc < 8; ++cc)
            if (col0 + 16 * cc < p.n_out) store_v8(to + cc * 32, packed + 8 * cc);
        } else {
#pragma unroll
          for (int cc = 0; cc < 16; ++cc)
            if (col0 + 8 * cc < p.n_out) store_v4(to + cc * 16, packed + 4 * cc);
        }
      }
    }
  epi_done:
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ host side
// A map of `rank` dimensions, the innermost adjacent, strides in bytes.
bool encode8(CUtensorMap *map, CUtensorMapDataType type, int rank, const void *base,
             const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box,
             CUtensorMapSwizzle swizzle) {
  const cuuint32_t ones[3] = {1, 1, 1};
  return encode_fn()(map, type, static_cast<cuuint32_t>(rank), const_cast<void *>(base), dims,
                     strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// At most `units` units.
template <bool STORES>
cudaError_t launch_gemm8(const Gemm8Params &p, int64_t units, const CUtensorMap &tmap_x,
                         const CUtensorMap &tmap_w, const CUtensorMap &tmap_out, cudaStream_t s) {
  static std::once_flag once[64];
  static cudaError_t attr_err[64];
  int dev = 0;
  cudaGetDevice(&dev);
  std::call_once(once[dev & 63], [d = dev & 63] {
    attr_err[d] = cudaFuncSetAttribute(reinterpret_cast<const void *>(gemm8_kernel<STORES>),
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kSmemLimit8));
  });
  if (attr_err[dev & 63] != cudaSuccess) return attr_err[dev & 63];
  const uint32_t smem = Plan8<STORES>::kOffTab + (p.n_experts + 1) * 4 + 1024;
  int64_t grid = sm_count();
  if (grid > units) grid = units;
  return launch_early(gemm8_kernel<STORES>, grid, kThreads8, smem, 1, s, tmap_x, tmap_w, tmap_out,
                      p);
}

}  // namespace

void gemm8_set_lose(int on) { g_gemm8_lose = on; }

uint32_t gemm8_read_errors(bool clear) {
  uint32_t v = 0;
  cudaMemcpyFromSymbol(&v, g_gemm8_errors, sizeof v);
  if (clear) {
    const uint32_t z = 0;
    cudaMemcpyToSymbol(g_gemm8_errors, &z, sizeof z);
  }
  return v;
}

}  // namespace mlg

extern "C" mlg_status mlg_grouped_gemm_f8(const mlg_f8 *x, const float *x_scales,
                                          const int32_t *expert_offsets, const mlg_f8 *w,
                                          const float *w_scales, mlg_bf16 *out, int32_t n_rows,
                                          int32_t k_in, int32_t n_out, int32_t n_experts,
                                          void *stream) {
  using namespace mlg;
  if (n_rows < 0 || k_in < 1 || n_out < 1 || n_experts < 0 || (!expert_offsets && n_experts != 1))
    return MLG_ERR_INVALID_ARG;
  if (k_in % 16 != 0 || n_out % 8 != 0 || n_experts > MLG_F8_MAX_EXPERTS ||
      n_rows > MLG_F8_MAX_ROWS || k_in > MLG_F8_MAX_WIDTH || n_out > MLG_F8_MAX_WIDTH)
    return MLG_ERR_UNSUPPORTED;
  if (n_rows == 0 || n_experts == 0) return MLG_OK;
  if (!x || !x_scales || !w || !w_scales || !out) return MLG_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w) || !aligned16(out) || !aligned4(x_scales) ||
      !aligned4(w_scales) || !aligned4(expert_offsets))
    return MLG_ERR_UNSUPPORTED;
  Gemm8Params p = {};
  p.offsets = expert_offsets;
  p.x_scales = x_scales;
  p.w_scales = w_scales;
  p.out = reinterpret_cast<uint8_t *>(out);
  p.k_in = k_in;
  p.n_out = n_out;
  p.n_experts = n_experts;
  p.row_end = n_rows;
  p.win = n_rows;
  p.tile_m = kTileM8;
  p.kb_count = (k_in + kBlockK8 - 1) / kBlockK8;
  p.nc_count = (n_out + kTileN8 - 1) / kTileN8;
  p.nb_count = (n_out + kBlockK8 - 1) / kBlockK8;
  p.v8 = (n_out % 16 == 0 && (reinterpret_cast<uintptr_t>(out) & 31u) == 0) ? 1 : 0;
  p.w_bytes = kWBytes8 + (g_gemm8_lose ? 16 : 0);
  if (encode_fn() == nullptr) return MLG_ERR_CUDA;
  CUtensorMap tmap_x, tmap_w, tmap_out;
  const cuuint64_t k = static_cast<cuuint64_t>(k_in), n = static_cast<cuuint64_t>(n_out);
  const cuuint64_t rows = static_cast<cuuint64_t>(n_rows);
  const cuuint64_t xd[2] = {k, rows}, xs[1] = {k};
  const cuuint64_t wd[3] = {k, n, static_cast<cuuint64_t>(n_experts)}, ws[2] = {k, k * n};
  const cuuint64_t od[2] = {n, rows}, os[1] = {n * 2};
  const cuuint32_t xb[2] = {kBlockK8, 32}, wb[3] = {kBlockK8, kTileN8, 1}, ob[2] = {32, 32};
  if (!encode8(&tmap_x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, x, xd, xs, xb,
               CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode8(&tmap_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, w, wd, ws, wb,
               CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode8(&tmap_out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, out, od, os, ob,
               CU_TENSOR_MAP_SWIZZLE_64B))
    return MLG_ERR_CUDA;

  const int64_t most = ((int64_t{n_rows} + kTileM8 - 1) / kTileM8 + n_experts) * p.nc_count;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // 32 rows an expert: from there on tiles have whole boxes of results (see Plan8)
  const bool stores = p.kb_count <= 8 && n_rows / 32 >= n_experts;
  return cuda_status(stores ? launch_gemm8<true>(p, most, tmap_x, tmap_w, tmap_out, s)
                            : launch_gemm8<false>(p, most, tmap_x, tmap_w, tmap_out, s));
}
