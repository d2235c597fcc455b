// mlg_q4.cu -- the decode-side product of gathered rows with 4-bit expert
// weights:  out[r, n] = sum_k x[r / top_k, k] * scale * (code - zero).
//
// Every weight is read once for all the rows of its expert, so a decode batch
// is bound by the codes' HBM traffic until an expert has some twenty rows.
//
//  * A job is an expert with up to 8 * NT of its rows; a tile is 32 output
//    features of a job.  The CTAs (persistent, one per SM) take equal,
//    contiguous runs of the tiles, so a CTA meets one or two experts.  The
//    jobs are counted on the device from `indices` (no host copy).
//  * WK warps share a tile, each with its own part of k (up to 128 wide).  A
//    warp's part of the job's x rows stays in its registers, as tensor-core
//    operands, over all the tiles of the job; its codes stream through a ring
//    of its own (TMA boxes of 32 rows x 128 codes) that runs on into the next
//    job, so the stream does not stop there.  The partial sums of a tile meet in
//    shared memory, added in warp order by one warp for every 16 features x 8
//    rows, in turn.
//  * The product is mma.sync m16n8k16 with the weights as the M operand and 8
//    rows as N.  Four bits become bf16 exactly: 0x4300 | code is 128 + code,
//    less 128 + zero in one packed subtraction, an integer of -15..15.  The
//    sum of a group is scaled in fp32, so a weight is never rounded.  A word
//    gives its eight codes as pairs (i, i + 4); x is loaded in that order, so
//    neither side is shuffled in the loop.  (tcgen05.mma takes ~71 ns however
//    small its N, which for 128 x 16 weights is a third of the rate at which
//    HBM delivers them; mma.sync keeps pace.)
#include <cuda.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "mlg_launch.cuh"

namespace mlg {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kTileN = 32;                  // output features per tile
constexpr int kDepth = 4;                   // ring stages per warp
constexpr int kStage = kTileN * 64;         // bytes: 32 rows x up to 128 codes
constexpr int kMaxNT = 3;                   // blocks of 8 rows per job
constexpr size_t kSmemMax = 230400;         // 227 KB less the static arrays

static __device__ uint32_t g_q4_errors;

struct Q4Params {
  const uint8_t *x;  // bf16 rows
  const int32_t *indices;
  const uint16_t *scales;
  const uint8_t *zeros;
  uint8_t *out;  // bf16 rows
  int32_t n_slots, k_in, n_out, top_k, n_experts;
  int32_t cap;              // rows per job, 8 * NT
  int32_t wk;               // warps per tile
  int32_t tiles_per_job;    // ceil(n_out / 32)
  int32_t part;             // 32-wide chunks of k per warp
  uint32_t off_red, off_jobs;
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

// Codes i and i + 4 of a word as bf16 integers less their zero point
// (magic = 128 in both halves, z2 = 128 + zero).  The magic number comes in a
// register: as a constant it would cost a second logic instruction.
__device__ __forceinline__ uint32_t weights2(uint32_t w, int i, uint32_t magic, uint32_t z2) {
  uint32_t q;
  asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(q) : "r"(w >> (4 * i)), "r"(magic));
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&q),
                                   *reinterpret_cast<const __nv_bfloat162 *>(&z2));
  return *reinterpret_cast<const uint32_t *>(&d);
}

// The same value in every lane, known to be so by the compiler.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(kFullWarp, v, 0); }

// Jobs before expert e (exclusive prefix, n_experts + 1 entries) -> the expert of a job.
__device__ __forceinline__ int job_expert(const int32_t *first_job, int n_experts, int job) {
  int lo = 0, hi = n_experts - 1;  // largest e with first_job[e] <= job
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first_job[mid] <= job) lo = mid; else hi = mid - 1;
  }
  return lo;
}

struct Run {  // the CTA's tiles [begin, end) over all jobs
  int64_t begin, end;
  int tiles_per_job;
  __device__ __forceinline__ int first_job() const { return static_cast<int>(begin / tiles_per_job); }
  __device__ __forceinline__ int last_job() const {
    return static_cast<int>((end - 1) / tiles_per_job);
  }
  __device__ __forceinline__ int lo(int job) const {
    const int64_t t = begin - static_cast<int64_t>(job) * tiles_per_job;
    return t > 0 ? static_cast<int>(t) : 0;
  }
  __device__ __forceinline__ int hi(int job) const {
    const int64_t t = end - static_cast<int64_t>(job) * tiles_per_job;
    return t < tiles_per_job ? static_cast<int>(t) : tiles_per_job;
  }
};

// Up to 128 of a tile's k for NB blocks of 8 rows, added to sum; GC: chunks
// per group, b: the x rows' operands of these chunks (zeros past the part).
template <int GC, int NB>
__device__ __forceinline__ void slice_mma(const uint8_t *stage, const uint4 (&b)[NB][4],
                                          uint32_t magic, const uint32_t (&sz)[4 / GC],
                                          float (&sum)[2][NB][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const uint8_t *row = stage + g * 64 + c * 4;
  const int swz = (g >> 1) & 3;
  float d[2][NB][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = *reinterpret_cast<const uint32_t *>(row + i * 512 + ((j ^ swz) << 4));
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      // scale (high half) and zero point (low half) of rows g + 16 m and
      // g + 16 m + 8, which lanes 2 m and 2 m + 1 of the quad hold
      const uint32_t own = sz[j / GC];
      const uint32_t s0 = __shfl_sync(kFullWarp, own, (lane & ~3) | (2 * m));
      const uint32_t s1 = __shfl_sync(kFullWarp, own, (lane & ~3) | (2 * m + 1));
      const uint32_t z0 = __byte_perm(s0, 0, 0x1010), z1 = __byte_perm(s1, 0, 0x1010);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t a[4] = {
            weights2(w[m * 2], 2 * h, magic, z0), weights2(w[m * 2 + 1], 2 * h, magic, z1),
            weights2(w[m * 2], 2 * h + 1, magic, z0), weights2(w[m * 2 + 1], 2 * h + 1, magic, z1)};
#pragma unroll
        for (int n = 0; n < NB; ++n)
          mma(d[m][n], a, h ? b[n][j].z : b[n][j].x, h ? b[n][j].w : b[n][j].y,
              j % GC == 0 && h == 0);
      }
      if (j % GC == GC - 1) {  // the group ends
        const float f0 = bf16hi_to_f32(s0), f1 = bf16hi_to_f32(s1);
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

// A lane's scales and zero points of a stage, as they are in memory: those of
// row 8 c + g of the tile (g = lane / 4, c = lane % 4), for the stage's groups.
template <int GC>
struct Raw {
  uint16_t s[4 / GC];
  uint8_t z[4 / GC];
};

// A warp's stream of codes and scales, one stage per (tile, 128 of its part).
template <int GC>
struct Stream {
  const Q4Params &p;
  const CUtensorMap *map;
  const int32_t *jobs;
  const Run &run;
  uint64_t *bars;  // the warp's, one per stage
  int job_end, team, teams, chunk0, chunk1;  // the warp's chunks [chunk0, chunk1)
  int groups;                                // per weight row
  // the next stage to fetch and the next whose scales load; `left`: tiles left
  // to the team in that job (0: the stream has ended)
  int job, tile, chunk, left, code_row, s_job, s_tile, s_chunk, s_left;
  const uint16_t *scale_at;  // this lane's row
  uint32_t put, ring;        // `put`: the stage to fill next

  // The team's next tile from (j, t) on and how many it has in that job.
  __device__ __forceinline__ int settle(int &j, int &t) const {
    while (j < job_end && t >= run.hi(j)) {
      ++j;
      t = run.lo(j) + team;
    }
    return j < job_end && chunk0 < chunk1 ? (run.hi(j) - t + teams - 1) / teams : 0;
  }
  __device__ __forceinline__ void aim_codes() {
    left = settle(job, tile);
    if (left > 0)
      code_row = uniform(job_expert(jobs, p.n_experts, job)) * p.n_out + tile * kTileN;
  }
  __device__ __forceinline__ void aim_scales() {
    if (s_left == 0) s_left = settle(s_job, s_tile);
    if (s_left == 0) return;
    const int e = uniform(job_expert(jobs, p.n_experts, s_job)), n0 = s_tile * kTileN;
    const int lane = threadIdx.x & 31;  // rows past n_out read the last one
    const int n = min(n0 + (lane & 3) * 8 + (lane >> 2), p.n_out - 1);
    scale_at = p.scales + (static_cast<int64_t>(e) * p.n_out + n) * groups;
  }
  // The codes of the next stage (nothing past k_in: TMA writes zeros there).
  __device__ __forceinline__ void fetch() {
    if (left == 0) return;
    if ((threadIdx.x & 31) == 0) {
      const uint32_t bar = smem_addr(bars + put);
      mbar_arrive_expect_tx(bar, kStage);
      tma_load_2d(ring + put * kStage, map, chunk * 16, code_row, bar);
    }
    put = (put + 1) & (kDepth - 1);
    chunk += 4;
    if (chunk < chunk1) return;
    chunk = chunk0;
    tile += teams;
    code_row += teams * kTileN;
    if (--left == 0) aim_codes();
  }
  // Loads the next stage's scales and zero points; nothing waits for them here.
  __device__ __forceinline__ void scales(Raw<GC> &raw) {
    if (s_left == 0) return;
    const int first = s_chunk / GC;
    const uint16_t *at = scale_at + first;
#pragma unroll
    for (int i = 0; i < 4 / GC; ++i)
      raw.s[i] = GC == 4 || first + i < groups ? at[i] : static_cast<uint16_t>(0);
    if (p.zeros) {
      const uint8_t *z = p.zeros + (at - p.scales);
#pragma unroll
      for (int i = 0; i < 4 / GC; ++i)
        raw.z[i] = GC == 4 || first + i < groups ? z[i] : static_cast<uint8_t>(0);
    }
    s_chunk += 4;
    if (s_chunk < chunk1) return;
    s_chunk = chunk0;
    s_tile += teams;
    if (--s_left > 0 && s_tile * kTileN + kTileN <= p.n_out)
      scale_at += teams * kTileN * groups;
    else
      aim_scales();
  }
};

// What a warp carries from job to job.
template <int GC>
struct Flow {
  const uint8_t *ring;     // its ring
  float4 *red;             // its team's partial sums, the first of two buffers
  uint32_t take, phase;    // the stage to use next, and its barrier's phase
  int it;                  // tiles done, which alternates the buffers
  uint32_t magic;
  bool dead;               // a wait ran out: wait no more
  Raw<GC> raw;             // of the next stage
};

// x of a row's 16-byte piece, as values 0 4 1 5 2 6 3 7.
__device__ __forceinline__ uint4 x_piece(const uint8_t *at) {
  const uint4 v = *reinterpret_cast<const uint4 *>(at);
  return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                    __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
}

// The tiles [lo, hi) of a job with NB blocks of rows.  R: 128-wide pieces of k
// whose x stays in registers (the warp's part); 0: any number, x from L2.
template <int GC, int NB, int R>
__device__ __forceinline__ void run_job(const Q4Params &p, Stream<GC> &st, Flow<GC> &f,
                                        const int32_t *rows, int n_rows, int lo, int hi, int team,
                                        int wk) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int WK = p.wk;
  constexpr int kR = R > 0 ? R : 1;
  const uint8_t *xr[NB];  // this lane's row of each block, at its piece of the warp's part
  uint4 b[kR][NB][4];
  auto load_x = [&](uint4 (&to)[NB][4], int chunk) {
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        to[n][j] = n * 8 + g < n_rows && chunk + j < st.chunk1 ? x_piece(xr[n] + (chunk + j) * 64)
                                                               : make_uint4(0, 0, 0, 0);
  };
#pragma unroll
  for (int n = 0; n < NB; ++n)
    xr[n] = p.x + (n * 8 + g < n_rows
                       ? static_cast<int64_t>(rows[n * 8 + g] / p.top_k) * p.k_in * 2 + c * 16
                       : 0);
  if (R > 0)
#pragma unroll
    for (int r = 0; r < kR; ++r) load_x(b[r], st.chunk0 + r * 4);

  for (int tile = lo + team; tile < hi; tile += st.teams) {
    float sum[2][NB][4] = {};
    auto slice = [&](const uint4 (&bb)[NB][4]) {
      uint32_t sz[4 / GC];  // scale (high half) and 128 + zero (low half)
#pragma unroll
      for (int i = 0; i < 4 / GC; ++i) {
        sz[i] = __byte_perm(f.raw.s[i], 0x43080000u, 0x1076);
        if (p.zeros) sz[i] = (sz[i] & 0xfffffff0u) | (f.raw.z[i] & 15u);
      }
      st.fetch();
      st.scales(f.raw);
      if (!f.dead && !mbar_wait_bounded(smem_addr(st.bars + f.take), f.phase)) {
        atomicOr(&g_q4_errors, kErrWaitTimeout);
        f.dead = true;
      }
      slice_mma<GC, NB>(f.ring + f.take * kStage, bb, f.magic, sz, sum);
      __syncwarp();  // the stage may be refilled
      f.take = (f.take + 1) & (kDepth - 1);
      f.phase ^= f.take == 0 ? 1u : 0u;
    };
    if (R > 0) {
#pragma unroll
      for (int r = 0; r < kR; ++r)
        if (st.chunk0 + r * 4 < st.chunk1) slice(b[r]);
    } else {
      for (int k = st.chunk0; k < st.chunk1; k += 4) {
        load_x(b[0], k);
        slice(b[0]);
      }
    }

    // Unit u (16 features x 8 rows) is added up by one warp, in warp order.
    float4 *red = f.red + (f.it & 1) * (kWarps * (p.cap / 4) * 32) + lane;
#pragma unroll
    for (int u = 0; u < 2 * NB; ++u)
      red[(wk * 2 * NB + u) * 32] = make_float4(sum[u & 1][u >> 1][0], sum[u & 1][u >> 1][1],
                                                sum[u & 1][u >> 1][2], sum[u & 1][u >> 1][3]);
    team_sync(team, WK);
    // units go round the warps: tile `it` starts at warp it * 2 NB
    for (int u = (wk - f.it * 2 * NB) & (WK - 1); u < 2 * NB; u += WK) {
      float v[4] = {};
      for (int w = 0; w < WK; ++w) {
        const float4 o = red[(w * 2 * NB + u) * 32];
        v[0] += o.x;
        v[1] += o.y;
        v[2] += o.z;
        v[3] += o.w;
      }
      // features x rows -> a lane with two features of one row
      const uint32_t lo2 = transpose8x8(pack_bf16x2(v[0], v[1]));
      const uint32_t hi2 = transpose8x8(pack_bf16x2(v[2], v[3]));
      const int r = (u >> 1) * 8 + g, n = tile * kTileN + (u & 1) * 16 + c * 2;
      if (r < n_rows) {
        uint8_t *o = p.out + (static_cast<int64_t>(rows[r]) * p.n_out + n) * 2;
        if (n < p.n_out) *reinterpret_cast<uint32_t *>(o) = lo2;
        if (n + 8 < p.n_out) *reinterpret_cast<uint32_t *>(o + 16) = hi2;
      }
    }
    ++f.it;
  }
}

template <int GC>
__global__ void __launch_bounds__(kThreads, 1)
    q4_kernel(const Q4Params p, const __grid_constant__ CUtensorMap map) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ uint64_t bars[kWarps][kDepth];
  __shared__ int32_t rows[8 * kMaxNT];   // the job's flat rows
  __shared__ int32_t warp_n[kWarps];
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  const int E = p.n_experts, WK = p.wk;
  const int team = warp / WK, wk = warp & (WK - 1);
  int32_t *jobs = reinterpret_cast<int32_t *>(smem + p.off_jobs);  // [E + 1]
  for (int e = tid; e <= E; e += kThreads) jobs[e] = 0;
  if (lane < kDepth) mbar_init(smem_addr(&bars[warp][lane]), 1);
  if (tid == 0) prefetch_tmap(&map);
  fence_mbar_init();
  __syncthreads();
  griddep_wait();

  // ---- rows per expert, then jobs before each expert
  if (p.indices) {
    for (int i = tid; i < p.n_slots; i += kThreads) {
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
  for (int e = e_lo; e < e_hi; ++e) mine += (jobs[e] + p.cap - 1) / p.cap;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFullWarp, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_n[warp] = incl;
  __syncthreads();
  int before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int n = warp_n[w];
    if (w < warp) before += n;
    total += n;
  }
  for (int e = e_lo; e < e_hi; ++e) {
    const int n = (jobs[e] + p.cap - 1) / p.cap;
    jobs[e] = before;
    before += n;
  }
  if (tid == 0) jobs[E] = total;
  total = uniform(total);
  __syncthreads();

  Run run;
  run.tiles_per_job = p.tiles_per_job;
  const int64_t tiles = static_cast<int64_t>(total) * p.tiles_per_job;
  run.begin = tiles * blockIdx.x / gridDim.x;
  run.end = tiles * (blockIdx.x + 1) / gridDim.x;

  if (run.begin < run.end) {
    const int chunks = p.k_in / 32, teams = kWarps / WK;
    const int job0 = run.first_job(), job_end = run.last_job() + 1;
    const uint8_t *ring = smem + warp * (kDepth * kStage);
    Stream<GC> st = {p, &map, jobs, run, bars[warp], job_end, team, teams,
                     min(wk * p.part, chunks), min((wk + 1) * p.part, chunks), chunks / GC};
    st.job = st.s_job = job0;
    st.tile = st.s_tile = run.lo(job0) + team;
    st.chunk = st.s_chunk = st.chunk0;
    st.left = st.s_left = 0;
    st.put = 0;
    st.ring = smem_addr(ring);
    st.aim_codes();
    st.aim_scales();
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) st.fetch();
    Flow<GC> f = {ring, reinterpret_cast<float4 *>(smem + p.off_red) + team * WK * (p.cap / 4) * 32};
    f.take = f.phase = 0;
    f.it = 0;
    f.dead = false;
    asm volatile("mov.b32 %0, 0x43004300;" : "=r"(f.magic));
    st.scales(f.raw);

    for (int job = job0; job < job_end; ++job) {
      const int e = uniform(job_expert(jobs, E, job));
      const int skip = (job - jobs[e]) * p.cap;  // rows of the expert's earlier jobs
      int n_rows;
      __syncthreads();  // the last job's rows are no longer read
      if (!p.indices) {
        n_rows = min(p.cap, p.n_slots - skip);
        if (tid < n_rows) rows[tid] = skip + tid;
      } else {  // the expert's rows, in order, from `skip` on
        const int piece = ((p.n_slots + kWarps - 1) / kWarps + 31) & ~31;
        const int a = warp * piece, z = min(a + piece, p.n_slots);
        int n = 0;
        for (int i = a; i < z; i += 32)
          n += __popc(__ballot_sync(kFullWarp, i + lane < z && p.indices[i + lane] == e));
        if (lane == 0) warp_n[warp] = n;
        __syncthreads();
        int at = -skip, all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const int v = warp_n[w];
          if (w < warp) at += v;
          all += v;
        }
        n_rows = min(all - skip, p.cap);
        for (int i = a; n > 0 && i < z; i += 32) {
          const bool hit = i + lane < z && p.indices[i + lane] == e;
          const uint32_t m = __ballot_sync(kFullWarp, hit);
          const int r = at + __popc(m & ((1u << lane) - 1u));
          if (hit && r >= 0 && r < p.cap) rows[r] = i + lane;
          at += __popc(m);
        }
      }
      n_rows = uniform(n_rows);
      __syncthreads();
      const int lo = run.lo(job), hi = run.hi(job);
      // x in registers for parts of k up to 128 (three times that for 8 rows)
      if (p.part > 12 || (p.part > 4 && n_rows > 8)) {
        if (n_rows <= 8)
          run_job<GC, 1, 0>(p, st, f, rows, n_rows, lo, hi, team, wk);
        else
          run_job<GC, 2, 0>(p, st, f, rows, n_rows, lo, hi, team, wk);
      } else if (p.part > 4) {
        run_job<GC, 1, 3>(p, st, f, rows, n_rows, lo, hi, team, wk);
      } else if (n_rows <= 8) {
        run_job<GC, 1, 1>(p, st, f, rows, n_rows, lo, hi, team, wk);
      } else if (GC < 4 || n_rows <= 16) {
        run_job<GC, 2, 1>(p, st, f, rows, n_rows, lo, hi, team, wk);
      } else {
        run_job<GC, 3, 1>(p, st, f, rows, n_rows, lo, hi, team, wk);
      }
    }
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
size_t layout(Q4Params &p, int nt) {
  p.cap = 8 * nt;
  const size_t ring = static_cast<size_t>(kWarps) * kDepth * kStage;
  const size_t red = static_cast<size_t>(kWarps) * nt * 1024 * 2;  // partial sums, two buffers
  p.off_red = static_cast<uint32_t>(ring);
  p.off_jobs = static_cast<uint32_t>(ring + red);
  return ring + red + (static_cast<size_t>(p.n_experts) + 1) * 4;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

template <int GC>
cudaError_t launch(const Q4Params &p, const CUtensorMap &map, int grid, size_t smem,
                   cudaStream_t s) {
  static std::once_flag once[64];
  static cudaError_t attr_err[64];
  int dev = 0;
  cudaGetDevice(&dev);
  std::call_once(once[dev & 63], [d = dev & 63] {
    attr_err[d] = cudaFuncSetAttribute(q4_kernel<GC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kSmemMax));
  });
  if (attr_err[dev & 63] != cudaSuccess) return attr_err[dev & 63];
  return launch_early(q4_kernel<GC>, grid, kThreads, smem, 1, s, p, map);
}

}  // namespace

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
  if (k_in % group != 0 || n_out % 8 != 0 || n_experts > MLG_Q4_MAX_EXPERTS)
    return MLG_ERR_UNSUPPORTED;
  if (n_slots == 0) return MLG_OK;
  if (!out || (n_experts > 0 && (!x || !codes || !scales))) return MLG_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(scales) & 1u) != 0)
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
  p.tiles_per_job = (n_out + kTileN - 1) / kTileN;
  // Rows per job: what an expert gets on average and two deviations more, so
  // that few experts need their codes twice.  Three blocks only with one
  // group per 128 codes and k up to 2048 (registers).
  const double mean = static_cast<double>(n_slots) / std::max(1, n_experts);
  const int64_t hit = std::min<int64_t>(n_slots, n_experts);
  const int sms = sm_count(), chunks = k_in / 32;
  int nt = 1;
  const int most_nt = group == 128 && chunks <= 4 * kWarps ? kMaxNT : 2;
  while (nt < most_nt && 8 * nt < mean + 2 * std::sqrt(mean)) ++nt;
  if (chunks > 4 * kWarps && chunks <= 12 * kWarps && mean <= 8) nt = 1;
  // Warps per tile: enough to keep a warp's part of k within 128, and more
  // where there are too few tiles for every team of every SM.
  p.wk = 1;
  const int gc = group / 32;
  while (p.wk < kWarps && p.wk * gc < chunks &&
         (p.wk * 4 < chunks || hit * p.tiles_per_job * p.wk < sms * kWarps))
    p.wk *= 2;
  // A part is whole groups, so that a group's sum stays in one warp.
  p.part = (chunks / gc + p.wk - 1) / p.wk * gc;
  size_t smem = layout(p, nt);
  while (nt > 1 && smem > kSmemMax) smem = layout(p, --nt);
  const int64_t most = std::max<int64_t>(hit * p.tiles_per_job, 1);
  const int grid = static_cast<int>(std::min<int64_t>(sms, most));
  // The codes as rows of bytes; a box is one stage of a warp, in the 64-byte
  // swizzle that keeps the loads of eight rows' words on different banks.
  CUtensorMap map = {};
  if (n_experts > 0) {
    EncodeTiledFn enc = encode_fn();
    if (enc == nullptr) return MLG_ERR_CUDA;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(k_in / 2),
                                static_cast<cuuint64_t>(n_experts) * n_out};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(k_in / 2)};
    const cuuint32_t box[2] = {64, kTileN}, step[2] = {1, 1};
    if (dims[1] > 0x7fffffffu) return MLG_ERR_UNSUPPORTED;
    if (enc(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(codes), dims, strides,
            box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return MLG_ERR_UNSUPPORTED;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(group == 32   ? launch<1>(p, map, grid, smem, s)
                     : group == 64 ? launch<2>(p, map, grid, smem, s)
                                   : launch<4>(p, map, grid, smem, s));
}
