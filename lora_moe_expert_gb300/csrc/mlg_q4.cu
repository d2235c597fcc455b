// mlg_q4.cu -- the decode-side product of gathered rows with 4-bit expert
// weights:  out[r, n] = sum_k x[r / top_k, k] * scale * (code - zero).
//
// Every weight is read once for all the rows of its expert, so a decode batch
// is bound by the codes' HBM traffic until an expert has some twenty rows.
//
//  * A job is an expert with up to 8 * NT of its rows; a tile is 32 output
//    features of a job.  A team of WK warps shares a tile, each warp with a run
//    of its 128-wide slices of k, and a round is a tile for every team of a CTA.
//    The CTAs (persistent, one per SM) take equal, contiguous runs of the
//    rounds, so a CTA meets one or two experts and stages their x rows in
//    shared memory once.  The jobs are counted on the device from `indices`
//    (no host copy).
//  * A warp's codes stream through a ring of its own (TMA boxes
//    of 32 rows x 128 codes) that runs on into the next tile and the next job,
//    so the stream does not stop there; a tile's scales and zero points are
//    one contiguous block and come in likewise, a ring per team.  The partial
//    sums of a tile meet in shared memory and are added in warp order.
//  * The product is mma.sync m16n8k16 with the weights as the M operand and 8
//    rows as N.  Four bits become bf16 exactly: in a 16-bit field whose other
//    bits are masked out, code << s (s = 0 or 4) is the subnormal bf16
//    code * 2^(s - 133), and one fused multiply-add by 2^(127 - s) gives
//    (code - zero) / 64.  The sum of a group is scaled in fp32, so a weight is
//    never rounded.  A word gives its eight codes as pairs (i, i + 4); x is
//    staged in that order, so neither side is shuffled in the loop.
//    (tcgen05.mma takes ~71 ns however small its N, which for 128 x 16 weights
//    is a third of the rate at which HBM delivers them.)
//
// Measured: 64 x top 8 rows, k 768, n 2048, groups of 32 with zero points (121
// MB, four rows an expert) 31 us, 57 % of the copy bandwidth; 256 x top 8 rows, k
// 2048, n 768, groups of 128 (108 MB, sixteen rows an expert) 43 us, 37 %; one
// token's 8 experts of that shape (6.5 MB) 6.4 us.  The stream alone (no
// products) runs at the copy bandwidth; what bounds the larger batches is the
// decoding and the products, at half the issue rate with four warps a
// scheduler (registers and the staged x leave room for no more), tensor pipe
// 41 % busy; one token is bound by the chain of counting the rows, the first
// boxes' round trip and the joining.  A CTA's first product comes 4 us after
// its start, a later job's 2 us after the last one's.
#include <cuda.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "mlg_launch.cuh"
#include "mlg_tmap.cuh"

namespace mlg {
namespace {

constexpr int kWarps = 16;                  // 12 and 24 measured slower
constexpr int kThreads = kWarps * 32;
constexpr int kTileN = 32;                  // output features per tile
constexpr int kDepth = 2;                   // ring stages per warp
constexpr int kScaleDepth = 2;              // ring stages per team
constexpr int kSlice = 4;                   // 32-wide chunks of k per slice
constexpr int kStage = kTileN * 16 * kSlice;  // bytes of a slice of a tile's codes
constexpr int kMaxNT = 3;                   // blocks of 8 rows per job
constexpr int kCached = 4;                  // slots per thread kept in registers
constexpr size_t kSmemMax = 230400;         // 227 KB less the static arrays

static __device__ uint32_t g_q4_errors;
int g_lose = 0;  // mlg_test_set_knob

struct Q4Params {
  const uint8_t *x;  // bf16 rows
  const int32_t *indices;
  const uint16_t *scales;
  const uint8_t *zeros;
  uint8_t *out;  // bf16 rows
  int32_t n_slots, k_in, n_out, top_k, n_experts;
  int32_t cap;              // rows per job, 8 * NT
  int32_t wk, teams;        // warps per tile, teams of them (powers of two)
  int32_t teams_log;
  int32_t tiles_per_job;    // ceil(n_out / 32)
  int32_t rounds_per_job;   // ceil(tiles_per_job / teams)
  int32_t part;             // slices of k per warp
  int32_t x_stride;         // bytes per staged row of x; 0: x is not staged
  uint32_t s_stage;         // bytes of a scale ring's stage
  uint32_t off_red, off_x, off_scale, off_jobs;
  uint32_t expect;          // bytes that a stage waits for: kStage, or more than come (test hook)
};

// D = A * B (+ D): m16n8k16, no side effects, so the compiler may schedule it.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1, bool fresh) {
  if (fresh)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// An 8 x 8 matrix of 16-bit values (row lane / 4, columns 2 (lane % 4) and the next) transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ void team_sync(int team, int wk) {
  if (wk == 1)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(wk * 32) : "memory");
}

// team_sync, and whether `any` holds for one of the team's threads.
__device__ __forceinline__ bool team_any(int team, int wk, bool any) {
  if (wk == 1) return __any_sync(kFullWarp, any);
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "bar.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(team + 1), "r"(wk * 32), "r"(any ? 1u : 0u)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// Codes h and h + 4 (h = 0 or 1) of a word as (code - zero) / 64 in bf16;
// z2 = -zero / 64 in both halves.  The multipliers are 2^127 and 2^123.
__device__ __forceinline__ uint32_t weights2(uint32_t w, int h, uint32_t z2) {
  return fma_bf16x2(w & (h ? 0x00f000f0u : 0x000f000fu), h ? 0x7d007d00u : 0x7f007f00u, z2);
}
// -zero / 64 of the zero point in the low four bits of each half.
__device__ __forceinline__ uint32_t minus_zero(uint32_t z) {
  return fma_bf16x2(z & 0x000f000fu, 0xff00ff00u, 0u);
}

// The same value in every lane, known to be so by the compiler.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(kFullWarp, v, 0); }

// The expert of a job at or after expert e's first; first_job: jobs before each
// expert (exclusive prefix, n_experts + 1 entries).
__device__ __forceinline__ int job_expert(const int32_t *first_job, int e, int job) {
  while (first_job[e + 1] <= job) ++e;
  return uniform(e);
}

// The CTA's tiles: of job `first` from `lo0` on, up to job `last`'s `hi1`.
struct Run {
  int first, last, lo0, hi1, tiles_per_job;
  __device__ __forceinline__ int lo(int job) const { return job == first ? lo0 : 0; }
  __device__ __forceinline__ int hi(int job) const { return job == last ? hi1 : tiles_per_job; }
};

// 16 bytes of x as values 0 4 1 5 2 6 3 7.
__device__ __forceinline__ uint4 x_piece(const uint8_t *at) {
  const uint4 v = *reinterpret_cast<const uint4 *>(at);
  return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                    __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
}

// A slice of a tile for NB blocks of 8 rows, added to sum (in units of 1 / 64).
// GC: chunks per group; sz: this lane's scale (high half) and -zero / 64 (low
// half, all 8 where there are no ZEROS) for each group; load_b(n, j): the
// operand of rows block n, chunk j.
template <int GC, int NB, bool ZEROS, class LoadB>
__device__ __forceinline__ void slice_mma(const uint8_t *stage, const uint32_t (&sz)[kSlice / GC],
                                          LoadB load_b, float (&sum)[2][NB][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const uint8_t *row = stage + g * 64 + c * 4;
  const int swz = (g >> 1) & 3;  // the 64-byte swizzle: piece j at j ^ swz
  float d[2][NB][4];
#pragma unroll
  for (int j = 0; j < kSlice; ++j) {
    uint4 b[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) b[n] = load_b(n, j);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = *reinterpret_cast<const uint32_t *>(row + i * 512 + ((j ^ swz) << 4));
    // Rows g + 16 m and g + 16 m + 8 are lanes 2 m and 2 m + 1 of the quad.  Both
    // m before the products: twice as many of those are then independent.
    uint32_t sc2[2][2], zp2[2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const uint32_t own = sz[j / GC];
      sc2[m][0] = __shfl_sync(kFullWarp, own, (lane & ~3) | (2 * m));
      sc2[m][1] = __shfl_sync(kFullWarp, own, (lane & ~3) | (2 * m + 1));
      zp2[m][0] = ZEROS ? __byte_perm(sc2[m][0], 0, 0x1010) : 0xbe00be00u;
      zp2[m][1] = ZEROS ? __byte_perm(sc2[m][1], 0, 0x1010) : 0xbe00be00u;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t a[2][4];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const uint32_t w0 = w[m * 2] >> (8 * h), w1 = w[m * 2 + 1] >> (8 * h);
        a[m][0] = weights2(w0, 0, zp2[m][0]);
        a[m][1] = weights2(w1, 0, zp2[m][1]);
        a[m][2] = weights2(w0, 1, zp2[m][0]);
        a[m][3] = weights2(w1, 1, zp2[m][1]);
      }
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int m = 0; m < 2; ++m)
          mma(d[m][n], a[m], h ? b[n].z : b[n].x, h ? b[n].w : b[n].y, j % GC == 0 && h == 0);
    }
    if (j % GC == GC - 1) {  // the group ends
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const float f0 = ZEROS ? bf16hi_to_f32(sc2[m][0]) : __uint_as_float(sc2[m][0]);
        const float f1 = ZEROS ? bf16hi_to_f32(sc2[m][1]) : __uint_as_float(sc2[m][1]);
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          sum[m][n][0] += f0 * d[m][n][0];
          sum[m][n][1] += f0 * d[m][n][1];
          sum[m][n][2] += f1 * d[m][n][2];
          sum[m][n][3] += f1 * d[m][n][3];
        }
      }
    }
  }
}

// Where the streams are: a warp's codes, one stage per slice, fetched one slice
// ahead, and its team's scales and zero points, one stage per tile.
static_assert(kDepth == 2, "the other stage is the one to fetch");
struct Stream {
  const Q4Params &p;
  const CUtensorMap *map;
  const int32_t *jobs;
  const Run &run;
  uint64_t *s_bars;          // the team's, one per stage
  uint32_t bars, ring;       // the warp's barriers and stages
  uint64_t policy;           // of the codes in L2: they are read once
  int team, slice0, slice1;  // the warp's slices [slice0, slice1)
  int groups;                // per weight row
  // the team's next tile and the next whose scales load; `left`: tiles left to
  // the team in that job (0: none is left at all)
  int job, e, tile, left, code_row, s_job, s_e, s_tile, s_left;
  int64_t s_row;             // weight row s_tile begins at
  uint32_t s_put, s_ring;    // `s_put`: the scale stage to fill next

  // The team's next tile from (j, t) on, j's expert, and how many tiles it has
  // in that job.
  __device__ __forceinline__ int settle(int &j, int &ex, int &t) const {
    while (j <= run.last && t >= run.hi(j)) {
      ++j;
      t = run.lo(j) + team;
    }
    if (j > run.last) return 0;
    ex = job_expert(jobs, ex, j);
    return (run.hi(j) - t + p.teams - 1) >> p.teams_log;
  }
  __device__ __forceinline__ void aim_codes() {
    left = settle(job, e, tile);
    code_row = e * p.n_out + tile * kTileN;
  }
  __device__ __forceinline__ void next_tile() {
    tile += p.teams;
    code_row += p.teams * kTileN;
    if (--left <= 0) aim_codes();
  }
  __device__ __forceinline__ void aim_scales() {
    s_left = settle(s_job, s_e, s_tile);
    s_row = static_cast<int64_t>(s_e) * p.n_out + s_tile * kTileN;
  }
  // A slice of the codes from weight row `row` on (zeros past k_in), by one lane.
  __device__ __forceinline__ void fetch(uint32_t stage, int slice, int row) const {
    const uint32_t bar = bars + stage * 8;
    mbar_arrive_expect_tx(bar, p.expect);
    tma_load_2d_hint(ring + stage * kStage, map, slice * (16 * kSlice), row, bar, policy);
  }
  // The next tile's scales and zero points, copied by one warp of the team
  // (`me`): 16 and 8 bytes a copy, the alignment that every tile has.
  __device__ __forceinline__ void fetch_scales(bool me) {
    if (s_left == 0) return;
    if (me) {
      const int lane = threadIdx.x & 31, rows = min(kTileN, p.n_out - s_tile * kTileN);
      const uint32_t to = s_ring + s_put * p.s_stage;
      const uint8_t *s = reinterpret_cast<const uint8_t *>(p.scales + s_row * groups);
      for (int i = lane * 16; i < rows * groups * 2; i += 512) cp_async_16(to + i, s + i, 16);
      if (p.zeros) {
        const uint8_t *z = p.zeros + s_row * groups;
        const uint32_t zt = to + kTileN * groups * 2;
        for (int i = lane * 8; i < rows * groups; i += 256)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(zt + i), "l"(z + i)
                       : "memory");
      }
      cp_async_arrive_noinc(smem_addr(s_bars + s_put));
    }
    s_put = (s_put + 1) & (kScaleDepth - 1);
    s_tile += p.teams;
    s_row += p.teams * kTileN;
    if (--s_left == 0) aim_scales();
  }
};

// Before a warp whose waits ran out returns: its copies have landed, or a wait for
// them ran out as well, so that none reaches shared memory that is another CTA's
// by then.  Which of the two phases a barrier is in is asked of the barrier (to
// keep that at hand costs the loop 1 us of 43); a stage that nothing was asked for
// waits in vain, once, until the limit.
__device__ __forceinline__ void drain(uint32_t bars) {
#pragma unroll 1
  for (int i = 0; i < kDepth; ++i)
    mbar_wait_bounded(bars + i * 8, mbar_try_wait(bars + i * 8, 0) ? 1u : 0u);
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// What a warp carries from job to job.
struct Flow {
  const uint8_t *ring;        // its ring
  const uint8_t *s_ring;      // its team's scales
  const uint8_t *x;           // staged rows
  float4 *red;                // its team's partial sums
  uint32_t take, phase;       // the stage to use next, and its barrier's phase
  uint32_t s_take, s_phase;
  int scale_turn;             // the warp that copies scales next
  // A wait ran out, of this lane or, from the next joining on, of another in the
  // team: nothing more is fetched or stored, and no wait waits.
  bool dead;

  __device__ __forceinline__ void wait(uint32_t bar, uint32_t parity) {
    if (!dead && !mbar_wait_bounded(bar, parity)) {
      atomicOr(&g_q4_errors, kErrWaitTimeout);
      dead = true;
    }
  }
};

// The tiles [lo, hi) of a job with NB blocks of rows; STAGED: x in shared
// memory, else (k_in too long for that) from L2.
template <int GC, int NB, bool ZEROS, bool STAGED>
__device__ __forceinline__ void run_job(const Q4Params &p, Stream &st, Flow &f,
                                        const int32_t *rows, int n_rows, int e, int lo, int hi,
                                        int team, int wk) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int WK = p.wk;
  const uint8_t *xr[NB];  // this lane's row of each block, at its piece
  bool there[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    there[n] = n * 8 + g < n_rows;
    if (STAGED)
      xr[n] = f.x + (n * 8 + g) * p.x_stride + c * 16;
    else
      xr[n] = p.x + (there[n] ? static_cast<int64_t>(rows[n * 8 + g] / p.top_k) * p.k_in * 2 : 0) +
              c * 16;
  }

  int row = e * p.n_out + (lo + team) * kTileN;
  for (int tile = lo + team; tile < hi; tile += p.teams, row += p.teams * kTileN) {
    float sum[2][NB][4] = {};
    st.next_tile();
    const bool more = st.left > 0;
    f.wait(smem_addr(st.s_bars + f.s_take), f.s_phase);
    const uint8_t *sc = f.s_ring + f.s_take * p.s_stage;
    const uint8_t *zc = sc + kTileN * st.groups * 2;
    const int own_row = (c * 8 + g) * st.groups;
#pragma unroll 1
    for (int s = st.slice0; s < st.slice1; ++s) {
      // Weight row 8 c + g (g = lane / 4, c = lane % 4), this slice's groups
      // (past k_in the last one again: codes and x are zeros there).
      uint32_t sz[kSlice / GC];
      const int first = s * (kSlice / GC), last = st.groups - 1 - first;
      const uint16_t *s_at = reinterpret_cast<const uint16_t *>(sc) + own_row + first;
#pragma unroll
      for (int i = 0; i < kSlice / GC; ++i) {
        const int k = GC == kSlice ? 0 : min(i, last);
        sz[i] = static_cast<uint32_t>(s_at[k]) << 16;
        if (ZEROS) sz[i] |= minus_zero(zc[own_row + first + k]);
      }
      const bool last_slice = s + 1 == st.slice1;
      if (lane == 0 && (!last_slice || more) && !f.dead)
        st.fetch(f.take ^ 1u, last_slice ? st.slice0 : s + 1, last_slice ? st.code_row : row);
      f.wait(st.bars + f.take * 8, f.phase);
      slice_mma<GC, NB, ZEROS>(f.ring + f.take * kStage, sz, [&](int n, int j) {
        if (STAGED) return *reinterpret_cast<const uint4 *>(xr[n] + s * 256 + j * 64);
        return there[n] && (s * 4 + j) * 32 < p.k_in ? x_piece(xr[n] + s * 256 + j * 64)
                                                     : make_uint4(0, 0, 0, 0);
      }, sum);
      __syncwarp();  // the stage may be refilled
      f.take ^= 1u;
      f.phase ^= f.take ^ 1u;
    }

    // Unit u (16 features x 8 rows) is added up by warp u % WK (a power of two).
    float4 *red = f.red + lane;
    if (WK > 1) {
#pragma unroll
      for (int u = 0; u < 2 * NB; ++u)
        red[(wk * 2 * NB + u) * 32] = make_float4(sum[u & 1][u >> 1][0], sum[u & 1][u >> 1][1],
                                                  sum[u & 1][u >> 1][2], sum[u & 1][u >> 1][3]);
    }
    f.dead = team_any(team, WK, f.dead);
    if (!f.dead) st.fetch_scales(f.scale_turn == wk);  // the stage just used is free
    f.scale_turn = f.scale_turn + 1 == WK ? 0 : f.scale_turn + 1;
    f.s_take = (f.s_take + 1) & (kScaleDepth - 1);
    f.s_phase ^= f.s_take == 0 ? 1u : 0u;
#pragma unroll
    for (int u = 0; u < 2 * NB; ++u) {
      if ((u & (WK - 1)) != wk) continue;
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = WK > 1 ? 0.0f : sum[u & 1][u >> 1][i];
      if (WK > 1) {
#pragma unroll 4
        for (int w = 0; w < WK; ++w) {
          const float4 o = red[(w * 2 * NB + u) * 32];
          v[0] += o.x;
          v[1] += o.y;
          v[2] += o.z;
          v[3] += o.w;
        }
      }
      // features x rows -> a lane with two features of one row
      const uint32_t lo2 = transpose8x8(pack_bf16x2(64.0f * v[0], 64.0f * v[1]));
      const uint32_t hi2 = transpose8x8(pack_bf16x2(64.0f * v[2], 64.0f * v[3]));
      const int r = (u >> 1) * 8 + g, n = tile * kTileN + (u & 1) * 16 + c * 2;
      if (r < n_rows && !f.dead) {
        uint8_t *o = p.out + (static_cast<int64_t>(rows[r]) * p.n_out + n) * 2;
        if (n < p.n_out) *reinterpret_cast<uint32_t *>(o) = lo2;
        if (n + 8 < p.n_out) *reinterpret_cast<uint32_t *>(o + 16) = hi2;
      }
    }
    if (WK > 1) team_sync(team, WK);  // the partial sums are read
  }
}

template <int GC, int NT, bool ZEROS>
__global__ void __launch_bounds__(kThreads, 1)
    q4_kernel(const Q4Params p, const __grid_constant__ CUtensorMap map) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ uint64_t bars[kWarps][kDepth];
  __shared__ uint64_t s_bars[kWarps][kScaleDepth];
  __shared__ int32_t rows[8 * NT];  // the job's flat rows
  __shared__ int32_t warp_n[kCached * kWarps];
  __shared__ int32_t jobs_n[kWarps];
  __shared__ int32_t first_e;  // the expert of this CTA's first job
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  const int E = p.n_experts, WK = p.wk;
  const int team = warp / WK, wk = warp - team * WK;
  constexpr int cap = 8 * NT;
  int32_t *jobs = reinterpret_cast<int32_t *>(smem + p.off_jobs);  // [E + 1]
  for (int e = tid; e <= E; e += kThreads) jobs[e] = 0;
  if (lane < kDepth) mbar_init(smem_addr(&bars[warp][lane]), 1);
  if (lane < kScaleDepth) mbar_init(smem_addr(&s_bars[warp][lane]), 32);
  if (tid == 0) prefetch_tmap(&map);
  fence_mbar_init();
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();

  // ---- rows per expert, then jobs before each expert
  int slot_e[kCached];  // the experts of this thread's first slots, -1 past the end
  if (p.indices) {
#pragma unroll
    for (int q = 0; q < kCached; ++q)
      slot_e[q] = q * kThreads + tid < p.n_slots ? p.indices[q * kThreads + tid] : -1;
#pragma unroll
    for (int q = 0; q < kCached; ++q)
      if (slot_e[q] >= 0 && slot_e[q] < E) atomicAdd(jobs + slot_e[q], 1);
    for (int i = kCached * kThreads + tid; i < p.n_slots; i += kThreads) {
      const int e = p.indices[i];
      if (e >= 0 && e < E) atomicAdd(jobs + e, 1);
    }
  } else if (tid == 0 && E > 0) {
    jobs[0] = p.n_slots;
  }
  __syncthreads();
  const int per = (E + kThreads - 1) / kThreads;
  const int e_lo = min(tid * per, E), e_hi = min(e_lo + per, E);
  int mine = 0;
  for (int e = e_lo; e < e_hi; ++e) mine += (jobs[e] + cap - 1) / cap;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFullWarp, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) jobs_n[warp] = incl;
  __syncthreads();
  const int w_n = lane < kWarps ? jobs_n[lane] : 0;
  int before = incl - mine + __reduce_add_sync(kFullWarp, lane < warp ? w_n : 0);
  const uint32_t total = uniform(__reduce_add_sync(kFullWarp, w_n));
  // This CTA's run of the rounds (their number fits 31 bits).
  const uint32_t rpj = p.rounds_per_job, all = total * rpj, cta = blockIdx.x;
  const uint32_t each = all / gridDim.x, more = all - each * gridDim.x;
  const uint32_t begin = cta * each + min(cta, more), end = begin + each + (cta < more ? 1 : 0);
  const int first_job = static_cast<int>(begin / rpj);
  for (int e = e_lo; e < e_hi; ++e) {
    const int n = (jobs[e] + cap - 1) / cap;
    jobs[e] = before;
    if (first_job >= before && first_job < before + n) first_e = e;
    before += n;
  }
  if (tid == 0) jobs[E] = static_cast<int32_t>(total);
  __syncthreads();

  if (begin < end) {
    Run run;
    run.first = first_job;
    run.last = (end - 1) / rpj;
    run.lo0 = (begin - run.first * rpj) * p.teams;
    run.hi1 = min(static_cast<int>(end - run.last * rpj) * p.teams, p.tiles_per_job);
    run.tiles_per_job = p.tiles_per_job;
    const int slices = (p.k_in + 32 * kSlice - 1) / (32 * kSlice);
    const uint8_t *ring = smem + warp * (kDepth * kStage);
    const uint8_t *s_ring = smem + p.off_scale + team * kScaleDepth * p.s_stage;
    Stream st = {p, &map, jobs, run, s_bars[team], smem_addr(bars[warp]), smem_addr(ring),
                 l2_evict_first(), team, min(wk * p.part, slices), min((wk + 1) * p.part, slices),
                 p.k_in / (32 * GC)};
    int e = first_e;
    st.job = st.s_job = run.first;
    st.e = st.s_e = e;
    st.tile = st.s_tile = run.lo0 + team;
    st.s_put = 0;
    st.s_ring = smem_addr(s_ring);
    st.aim_codes();
    if (lane == 0 && st.left > 0 && st.slice0 < st.slice1) st.fetch(0, st.slice0, st.code_row);
    st.aim_scales();
#pragma unroll 1
    for (int i = 0; i < kScaleDepth; ++i) st.fetch_scales(wk == 0);
    Flow f = {ring, s_ring, smem + p.off_x,
              reinterpret_cast<float4 *>(smem + p.off_red) + team * WK * (p.cap / 4) * 32};
    f.take = f.phase = f.s_take = f.s_phase = 0;
    f.scale_turn = 0;
    f.dead = false;

    for (int job = run.first; job <= run.last; ++job) {
      e = job_expert(jobs, e, job);
      const int skip = (job - jobs[e]) * p.cap;  // rows of the expert's earlier jobs
      int n_rows;
      __syncthreads();  // the last job's rows are no longer read
      if (!p.indices) {
        n_rows = min(p.cap, p.n_slots - skip);
        if (tid < n_rows) rows[tid] = skip + tid;
      } else {  // the expert's rows, in order, from `skip` on
        int found = 0;
        for (int i0 = 0; i0 < p.n_slots; i0 += kCached * kThreads) {
          if (i0 > 0) __syncthreads();  // warp_n is read
          uint32_t hit[kCached];
#pragma unroll
          for (int q = 0; q < kCached; ++q) {
            const int i = i0 + q * kThreads + tid;
            const int v = i0 == 0 ? slot_e[q] : i < p.n_slots ? p.indices[i] : -1;
            hit[q] = __ballot_sync(kFullWarp, v == e);
            if (lane == 0) warp_n[q * kWarps + warp] = __popc(hit[q]);
          }
          __syncthreads();
#pragma unroll
          for (int q = 0; q < kCached; ++q) {  // rows found before this warp's, in slot order
            if (hit[q] == 0) continue;
            int n = 0;
            for (int w = lane; w < q * kWarps + warp; w += 32) n += warp_n[w];
            const int at = found - skip + __reduce_add_sync(kFullWarp, n) +
                           __popc(hit[q] & ((1u << lane) - 1u));
            if ((hit[q] >> lane & 1u) && at >= 0 && at < p.cap)
              rows[at] = i0 + q * kThreads + tid;
          }
          int n = 0;
          for (int w = lane; w < kCached * kWarps; w += 32) n += warp_n[w];
          found += __reduce_add_sync(kFullWarp, n);
        }
        n_rows = min(found - skip, p.cap);
      }
      n_rows = uniform(n_rows);
      __syncthreads();
      if (p.x_stride > 0) {
        // x into shared memory, zeros past k_in up to a whole slice
        const int per_row = slices * 16, pieces = p.k_in / 8;
        constexpr int kLoads = 8;
        for (int r = warp; r < n_rows; r += kWarps) {
          const uint8_t *from = p.x + static_cast<int64_t>(rows[r] / p.top_k) * p.k_in * 2;
          uint8_t *to = smem + p.off_x + r * p.x_stride;
          for (int q0 = lane; q0 < per_row; q0 += kLoads * 32) {
            uint4 v[kLoads];
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
              v[k] = make_uint4(0, 0, 0, 0);
              if (q0 + k * 32 < pieces) v[k] = x_piece(from + (q0 + k * 32) * 16);
            }
#pragma unroll
            for (int k = 0; k < kLoads; ++k)
              if (q0 + k * 32 < per_row) *reinterpret_cast<uint4 *>(to + (q0 + k * 32) * 16) = v[k];
          }
        }
        __syncthreads();
      }
      const int lo = run.lo(job), hi = run.hi(job);
      // All jobs take NT blocks of rows, the short ones too: a second variant of
      // the loop costs its cold instructions (256 x 8 rows: 49 us with three).
      if (NT == 1 && p.x_stride == 0)
        run_job<GC, NT, ZEROS, false>(p, st, f, rows, n_rows, e, lo, hi, team, wk);
      else
        run_job<GC, NT, ZEROS, true>(p, st, f, rows, n_rows, e, lo, hi, team, wk);
    }
    if (f.dead) drain(smem_addr(bars[warp]));
  }

  // ---- rows of no expert
  if (p.indices || E == 0)
    for (int64_t i = blockIdx.x; i < p.n_slots; i += gridDim.x) {
      const int e = p.indices ? p.indices[i] : 0;
      if (e >= 0 && e < E) continue;
      for (int q = tid; q < p.n_out / 8; q += kThreads)
        *reinterpret_cast<uint4 *>(p.out + (i * p.n_out + q * 8) * 2) = make_uint4(0, 0, 0, 0);
    }
}

// Shared memory of a launch with rows capped at 8 * nt; sets the offsets.
size_t layout(Q4Params &p, int nt, bool staged) {
  p.cap = 8 * nt;
  const int slices = (p.k_in + 32 * kSlice - 1) / (32 * kSlice);
  // A row's stride is an odd number of 64-byte halves, so that the 16-byte
  // pieces of two rows, which a quarter warp reads at once, hit all banks.
  p.x_stride = staged ? slices * 256 + 64 : 0;
  const size_t ring = static_cast<size_t>(kWarps) * kDepth * kStage;
  const size_t red = static_cast<size_t>(kWarps) * nt * 1024;  // partial sums
  p.off_red = static_cast<uint32_t>(ring);
  p.off_x = static_cast<uint32_t>(ring + red);
  p.off_scale = static_cast<uint32_t>(p.off_x + static_cast<size_t>(p.cap) * p.x_stride);
  p.off_jobs = p.off_scale + p.teams * kScaleDepth * p.s_stage;
  return p.off_jobs + (static_cast<size_t>(p.n_experts) + 1) * 4;
}

template <int GC, int NT, bool ZEROS>
cudaError_t launch(const Q4Params &p, const CUtensorMap &map, int grid, size_t smem,
                   cudaStream_t s) {
  static std::once_flag once[64];
  static cudaError_t attr_err[64];
  int dev = 0;
  cudaGetDevice(&dev);
  std::call_once(once[dev & 63], [d = dev & 63] {
    attr_err[d] = cudaFuncSetAttribute(q4_kernel<GC, NT, ZEROS>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kSmemMax));
  });
  if (attr_err[dev & 63] != cudaSuccess) return attr_err[dev & 63];
  return launch_early(q4_kernel<GC, NT, ZEROS>, grid, kThreads, smem, 1, s, p, map);
}

template <int GC, bool ZEROS>
cudaError_t launch_nt(const Q4Params &p, const CUtensorMap &map, int grid, size_t smem,
                      cudaStream_t s) {
  return p.cap == 8    ? launch<GC, 1, ZEROS>(p, map, grid, smem, s)
         : p.cap == 16 ? launch<GC, 2, ZEROS>(p, map, grid, smem, s)
                       : launch<GC, 3, ZEROS>(p, map, grid, smem, s);
}

template <bool ZEROS>
cudaError_t launch_group(const Q4Params &p, int group, const CUtensorMap &map, int grid,
                         size_t smem, cudaStream_t s) {
  return group == 32   ? launch_nt<1, ZEROS>(p, map, grid, smem, s)
         : group == 64 ? launch_nt<2, ZEROS>(p, map, grid, smem, s)
                       : launch_nt<4, ZEROS>(p, map, grid, smem, s);
}

}  // namespace

void q4_set_lose(int on) { g_lose = on; }

uint32_t q4_read_errors(bool clear) {
  uint32_t v = 0;
  cudaMemcpyFromSymbol(&v, g_q4_errors, sizeof v);
  if (clear) {
    const uint32_t z = 0;
    cudaMemcpyToSymbol(g_q4_errors, &z, sizeof z);
  }
  return v;
}

}  // namespace mlg

extern "C" mlg_status mlg_gather_q4(const mlg_bf16 *x, const int32_t *indices,
                                    const uint8_t *codes, const mlg_bf16 *scales,
                                    const uint8_t *zeros, mlg_bf16 *out, int32_t n_slots,
                                    int32_t k_in, int32_t n_out, int32_t top_k,
                                    int32_t n_experts, int32_t group, void *stream) {
  using namespace mlg;
  if (n_slots < 0 || k_in < 1 || n_out < 1 || top_k < 1 || n_experts < 0)
    return MLG_ERR_INVALID_ARG;
  if (group != 32 && group != 64 && group != 128) return MLG_ERR_UNSUPPORTED;
  if (k_in % group != 0 || n_out % 8 != 0 || n_experts > MLG_Q4_MAX_EXPERTS ||
      k_in / group > MLG_Q4_MAX_GROUPS)
    return MLG_ERR_UNSUPPORTED;
  if (n_slots == 0) return MLG_OK;
  if (!out || (n_experts > 0 && (!x || !codes || !scales))) return MLG_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(out) || !aligned16(scales) ||
      !aligned16(zeros))
    return MLG_ERR_UNSUPPORTED;
  Q4Params p = {};
  p.x = reinterpret_cast<const uint8_t *>(x);
  p.indices = indices;
  p.scales = scales;
  p.zeros = zeros;
  p.out = reinterpret_cast<uint8_t *>(out);
  p.n_slots = n_slots;
  p.k_in = k_in;
  p.n_out = n_out;
  p.top_k = top_k;
  p.n_experts = n_experts;
  p.expect = kStage + (g_lose ? 16 : 0);
  p.tiles_per_job = (n_out + kTileN - 1) / kTileN;
  const double mean = static_cast<double>(n_slots) / std::max(1, n_experts);
  const int64_t hit = std::min<int64_t>(n_slots, n_experts);
  const int sms = sm_count(), slices = (k_in + 32 * kSlice - 1) / (32 * kSlice);
  // The tiles of all jobs are numbered in 31 bits (jobs: at most one per row).
  if (static_cast<int64_t>(n_slots) * p.tiles_per_job > 0x7fffffff ||
      static_cast<int64_t>(n_experts) * n_out > 0x7fffffff)
    return MLG_ERR_UNSUPPORTED;
  p.s_stage = (kTileN * (k_in / group) * 3 + 15) / 16 * 16;
  // Teams of wk warps.  Returns what the busiest CTA's rounds cost in slices, a
  // round being a warp's slices and the joining of the sums.  (Teams of 1, 2,
  // 4, 8 warps: 64 x 8 rows of the down projection, one block of rows, 33, 34,
  // 44, 53 us; 256 x 8 rows of gate/up, three blocks, 54, 46, 43, 50 us.)
  auto team_up = [&](int wk, int nt) {
    p.wk = wk;
    p.teams = kWarps / wk;
    p.teams_log = 0;
    while ((1 << p.teams_log) < p.teams) ++p.teams_log;
    p.part = (slices + wk - 1) / wk;
    p.rounds_per_job = (p.tiles_per_job + p.teams - 1) / p.teams;
    const double join = nt == 1 ? 1.7 : nt == 2 ? 1.0 : 0.7;
    const int64_t jobs = hit * std::max<int64_t>(1, (n_slots / std::max<int64_t>(hit, 1) + 8 * nt - 1) / (8 * nt));
    return ((jobs * p.rounds_per_job + sms - 1) / sms) * (p.part + join);
  };
  // Rows per job: what an expert gets on average and two deviations more, so
  // that few experts need their codes twice; as far as their x fits.  The
  // cheapest teams that fit; without staging (k_in too long for 8 rows) x
  // comes from L2.
  int nt = 1;
  while (nt < kMaxNT && 8 * nt < mean + 2 * std::sqrt(mean)) ++nt;
  size_t smem = 0;
  for (int staged = 1;; --nt) {
    if (nt == 0) {
      if (staged == 0) return MLG_ERR_UNSUPPORTED;
      staged = 0;
      nt = 1;
    }
    int best = 0;
    double least = 0;
    for (int wk = 1; wk <= kWarps; wk *= 2) {
      const double cost = team_up(wk, nt);
      if (layout(p, nt, staged != 0) <= kSmemMax && (best == 0 || cost < least))
        least = cost, best = wk;
    }
    if (best == 0) continue;
    team_up(best, nt);
    smem = layout(p, nt, staged != 0);
    break;
  }
  const int64_t most = (hit + n_slots / p.cap) * p.rounds_per_job;  // rounds, at most
  const int grid = static_cast<int>(std::min<int64_t>(sms, std::max<int64_t>(most, 1)));
  // The codes as rows of bytes; a box is one stage of a warp, in the 64-byte
  // swizzle that keeps the loads of eight rows' words on different banks.
  CUtensorMap map = {};
  if (n_experts > 0) {
    EncodeTiledFn enc = encode_fn();
    if (enc == nullptr) return MLG_ERR_CUDA;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(k_in / 2),
                                static_cast<cuuint64_t>(n_experts) * n_out};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(k_in / 2)};
    const cuuint32_t box[2] = {16 * kSlice, kTileN}, step[2] = {1, 1};
    if (enc(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(codes), dims, strides,
            box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return MLG_ERR_UNSUPPORTED;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(zeros ? launch_group<true>(p, group, map, grid, smem, s)
                           : launch_group<false>(p, group, map, grid, smem, s));
}
