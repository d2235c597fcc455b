// mlg_q4.cu -- the decode-side product of gathered rows with 4-bit expert
// weights:  out[r, n] = sum_k x[r / top_k, k] * scale * (code - zero).
//
// Every weight is read once for all the rows of its expert, so a decode batch
// is bound by the codes' HBM traffic until an expert has some twenty rows.
//
//  * A job is an expert with up to 8 * NT of its rows; a tile is 32 output
//    features of a job.  The CTAs (persistent, one per SM) take equal,
//    contiguous runs of the tiles, so a CTA meets one or two experts and
//    stages their x rows in shared memory once.  The jobs are counted on the
//    device from `indices` (no host copy).
//  * WK warps share a tile, each taking every WK-th 128-wide slice of k; each
//    warp streams its codes through a ring of its own (cp.async, D slices
//    deep), which runs on into the next tile and the next expert, so the
//    stream does not stop at their boundaries.
//  * The product is mma.sync m16n8k16 with the weights as the M operand and 8
//    rows as N.  Four bits become bf16 exactly: 0x4300 | code is 128 + code,
//    less 128 + zero in one packed subtraction, an integer of -15..15.  The
//    sum of a group is scaled in fp32, so a weight is never rounded.  A word
//    gives its eight codes as pairs (i, i + 4); x is staged with its values in
//    that order, so neither side is shuffled in the loop.  (tcgen05.mma takes
//    ~71 ns however small its N, which for 128 x 16 weights is a third of the
//    rate at which HBM delivers them; mma.sync keeps pace.)
#include <algorithm>
#include <mutex>

#include "mlg_launch.cuh"

namespace mlg {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kTileN = 32;                  // output features per tile
constexpr int kDepth = 3;                   // ring stages per warp
constexpr int kStage = kTileN * 64;         // bytes: 32 rows x 128 codes
constexpr int kMaxNT = 3;                   // blocks of 8 rows per job
constexpr size_t kSmemMax = 231424;         // 227 KB less the static arrays

struct Q4Params {
  const uint8_t *x;  // bf16 rows
  const int32_t *indices;
  const uint8_t *codes;
  const uint16_t *scales;
  const uint8_t *zeros;
  uint8_t *out;  // bf16 rows
  int32_t n_slots, k_in, n_out, top_k, n_experts;
  int32_t cap;              // rows per job, 8 * NT
  int32_t wk;               // warps per tile
  int32_t tiles_per_job;    // ceil(n_out / 32)
  int32_t slices;           // ceil(k_in / 128)
  int32_t chunk;            // slices of x staged at a time, a multiple of wk
  int32_t x_stride;         // bytes per staged row
  uint32_t off_ring, off_red, off_jobs;
};

// D = A * B + C with a fresh D (C may be zeros).
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint32_t lds_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds_u128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}

__device__ __forceinline__ void team_sync(int team, int wk) {
  asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(wk * 32) : "memory");
}

// Codes i and i + 4 of a word as bf16 integers less their zero point
// (z2 = 128 + zero in both halves).
__device__ __forceinline__ uint32_t weights2(uint32_t w, int i, uint32_t z2) {
  const uint32_t q = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&q),
                                   *reinterpret_cast<const __nv_bfloat162 *>(&z2));
  return *reinterpret_cast<const uint32_t *>(&d);
}

// Where a warp is in the CTA's run of tiles: tile `tile` of job `job` (tiles
// numbered within the job), slice `slice` of its k.
struct Cursor {
  int job, tile, slice;
};

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

// One slice of a tile, for NB blocks of 8 rows; GC: 32-code chunks per group.
// d: the running sums of the current group, sum: the scaled sums.
template <int GC, int NB>
__device__ __forceinline__ void slice_mma(uint32_t stage, uint32_t xa, int x_stride, int chunks,
                                          const uint32_t (&sz)[4], float (&sum)[2][kMaxNT][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const uint32_t row = stage + g * 64 + c * 4;
  const uint32_t swz = (g >> 1) & 3;
  float d[2][NB][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j >= chunks) break;
    uint4 b[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) b[n] = lds_u128(xa + n * 8 * x_stride + j * 64);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const uint32_t w0 = lds_u32(row + (m * 2) * 512 + ((j ^ swz) << 4));
      const uint32_t w1 = lds_u32(row + (m * 2 + 1) * 512 + ((j ^ swz) << 4));
      // scale (high half) and zero point (low half) of rows g + 16 m, g + 16 m + 8
      uint32_t s0 = sz[m * 2], s1 = sz[m * 2 + 1];
      if (GC < 4) {  // lane c of the quad holds group c (of 4) or c & 1 (of 2)
        const int from = (lane & ~3) | (j / GC);
        s0 = __shfl_sync(kFullWarp, s0, from);
        s1 = __shfl_sync(kFullWarp, s1, from);
      }
      const uint32_t z0 = __byte_perm(s0, 0, 0x1010), z1 = __byte_perm(s1, 0, 0x1010);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t a[4] = {weights2(w0, 2 * h, z0), weights2(w1, 2 * h, z1),
                               weights2(w0, 2 * h + 1, z0), weights2(w1, 2 * h + 1, z1)};
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const uint32_t b0 = h ? b[n].z : b[n].x, b1 = h ? b[n].w : b[n].y;
          if (j % GC == 0 && h == 0)
            mma_first(d[m][n], a, b0, b1);
          else
            mma_bf16_16816(d[m][n], a[0], a[1], a[2], a[3], b0, b1);
        }
      }
      if (j % GC == GC - 1 || j == chunks - 1) {  // the group ends
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

template <int GC>
__global__ void __launch_bounds__(kThreads, 1) q4_kernel(const Q4Params p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int32_t rows[8 * kMaxNT];   // the job's flat rows
  __shared__ int32_t warp_n[kWarps];
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int E = p.n_experts, WK = p.wk, teams = kWarps / WK;
  const int team = warp / WK, wk = warp % WK;
  int32_t *jobs = reinterpret_cast<int32_t *>(smem + p.off_jobs);  // [E + 1]
  for (int e = tid; e <= E; e += kThreads) jobs[e] = 0;
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
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += warp_n[w];
    total += warp_n[w];
  }
  for (int e = e_lo; e < e_hi; ++e) {
    const int n = (jobs[e] + p.cap - 1) / p.cap;
    jobs[e] = before;
    before += n;
  }
  if (tid == 0) jobs[E] = total;
  __syncthreads();

  Run run;
  run.tiles_per_job = p.tiles_per_job;
  const int64_t tiles = static_cast<int64_t>(total) * p.tiles_per_job;
  run.begin = tiles * blockIdx.x / gridDim.x;
  run.end = tiles * (blockIdx.x + 1) / gridDim.x;

  const uint32_t ring = smem_addr(smem + p.off_ring) + warp * (kDepth * kStage);
  const int64_t row_codes = p.k_in / 2;
  const int chunks_all = p.k_in / 32;
  const int groups = chunks_all / GC;  // per weight row

  if (run.begin < run.end) {
    const int job_end = run.last_job() + 1;
    // First tile of this warp's team from `job` on; slice = its first, job = job_end at the end.
    auto settle = [&](Cursor &u) {
      while (u.job < job_end && u.tile >= run.hi(u.job)) {
        ++u.job;
        u.tile = run.lo(u.job) + team;
      }
      if (wk >= p.slices) u.job = job_end;
    };
    auto advance = [&](Cursor &u) {
      u.slice += WK;
      if (u.slice < p.slices) return;
      u.slice = wk;
      u.tile += teams;
      settle(u);
    };
    Cursor fetch = {run.first_job(), run.lo(run.first_job()) + team, wk};
    settle(fetch);
    Cursor next = fetch;  // the slice whose scales load next
    int fetch_job = -1, fetch_e = 0, next_job = -1, next_e = 0, put = 0;

    auto issue = [&]() {  // codes of `fetch` into ring stage `put`
      if (fetch.job < job_end) {
        if (fetch.job != fetch_job) {
          fetch_job = fetch.job;
          fetch_e = job_expert(jobs, E, fetch_job);
        }
        const uint8_t *base = p.codes + static_cast<int64_t>(fetch_e) * p.n_out * row_codes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = i * 8 + g;
          const int n = min(fetch.tile * kTileN + r, p.n_out - 1);
          const bool in = fetch.slice * 4 + c < chunks_all;
          cp_async_16(ring + put * kStage + r * 64 + ((c ^ ((r >> 1) & 3)) << 4),
                      base + n * row_codes + (in ? fetch.slice * 64 + c * 16 : 0), in ? 16 : 0);
        }
        advance(fetch);
      }
      cp_async_commit();
      put = put + 1 == kDepth ? 0 : put + 1;
    };
    // scale (high half) and 128 + zero (low half) of four weight rows, group
    // c (or its like) of the slice
    auto scales = [&](uint32_t (&sz)[4]) {
      if (next.job >= job_end) return;
      if (next.job != next_job) {
        next_job = next.job;
        next_e = job_expert(jobs, E, next_job);
      }
      const int group = min(next.slice * (4 / GC) + (GC == 1 ? c : GC == 2 ? (c & 1) : 0),
                            groups - 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = min(next.tile * kTileN + i * 8 + g, p.n_out - 1);
        const int64_t at = (static_cast<int64_t>(next_e) * p.n_out + n) * groups + group;
        const uint32_t z = p.zeros ? p.zeros[at] : 8u;
        sz[i] = (static_cast<uint32_t>(p.scales[at]) << 16) | 0x4300u | (z & 15u);
      }
      advance(next);
    };

#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) issue();
    uint32_t sz[4] = {}, sz_next[4] = {};
    scales(sz_next);
    int take = 0;
    const uint32_t xs = smem_addr(smem);

    for (int job = run.first_job(); job < job_end; ++job) {
      const int lo = run.lo(job), hi = run.hi(job);
      const int e = job_expert(jobs, E, job);
      const int skip = (job - jobs[e]) * p.cap;  // rows of the expert's earlier jobs
      int n_rows = 0;
      for (int t0 = lo; t0 < hi; t0 += teams) {
        const int tile = t0 + team;
        float sum[2][kMaxNT][4] = {};
        for (int k0 = 0; k0 < p.slices; k0 += p.chunk) {
          if (t0 == lo || p.chunk < p.slices) {
            __syncthreads();  // the staged rows are no longer read
            if (t0 == lo && k0 == 0) {
              // the job's rows: the expert's, in order, from `skip` on
              if (!p.indices) {
                n_rows = min(p.cap, p.n_slots - skip);
                if (tid < n_rows) rows[tid] = skip + tid;
              } else {
                const int piece = ((p.n_slots + kWarps - 1) / kWarps + 31) & ~31;
                const int a = warp * piece, z = min(a + piece, p.n_slots);
                int n = 0;
                for (int i = a; i < z; i += 32)
                  n += __popc(__ballot_sync(kFullWarp, i + lane < z && p.indices[i + lane] == e));
                if (lane == 0) warp_n[warp] = n;
                __syncthreads();
                int at = -skip, all = 0;
                for (int w = 0; w < kWarps; ++w) {
                  if (w < warp) at += warp_n[w];
                  all += warp_n[w];
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
              __syncthreads();
            }
            // x rows, each 16-byte piece as values 0 4 1 5 2 6 3 7
            const int pieces = (min(p.chunk, p.slices - k0) * 128 + k0 * 128 > p.k_in
                                    ? p.k_in - k0 * 128
                                    : min(p.chunk, p.slices - k0) * 128) / 8;
            for (int i = tid; i < n_rows * pieces; i += kThreads) {
              const int r = i / pieces, q = i - r * pieces;
              const uint4 v = *reinterpret_cast<const uint4 *>(
                  p.x + (static_cast<int64_t>(rows[r] / p.top_k) * p.k_in + k0 * 128 + q * 8) * 2);
              *reinterpret_cast<uint4 *>(smem + r * p.x_stride + q * 16) =
                  make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                             __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
            }
            __syncthreads();
          }
          if (tile >= hi) continue;
          const int k1 = min(k0 + p.chunk, p.slices);
          for (int s = k0 + wk; s < k1; s += WK) {
#pragma unroll
            for (int i = 0; i < 4; ++i) sz[i] = sz_next[i];
            issue();
            scales(sz_next);
            cp_async_wait_group<kDepth - 1>();
            __syncwarp();
            const uint32_t stage = ring + take * kStage;
            const uint32_t xa = xs + g * p.x_stride + (s - k0) * 256 + c * 16;
            const int n = min(4, chunks_all - s * 4);
            if (n_rows > 16)
              slice_mma<GC, 3>(stage, xa, p.x_stride, n, sz, sum);
            else if (n_rows > 8)
              slice_mma<GC, 2>(stage, xa, p.x_stride, n, sz, sum);
            else
              slice_mma<GC, 1>(stage, xa, p.x_stride, n, sz, sum);
            __syncwarp();  // the stage may be refilled
            take = take + 1 == kDepth ? 0 : take + 1;
          }
        }
        if (tile >= hi) continue;

        // ---- the tile's warps add up in warp order; the first rounds and stores
        const int blocks = (n_rows + 7) >> 3;
        float4 *red = reinterpret_cast<float4 *>(smem + p.off_red) +
                      static_cast<int64_t>(team) * (WK - 1) * (p.cap / 8) * 64;
        if (wk > 0) {
          float4 *mine_red = red + (wk - 1) * (p.cap / 8) * 64;
#pragma unroll
          for (int n = 0; n < kMaxNT; ++n)
            if (n < blocks) {
#pragma unroll
              for (int m = 0; m < 2; ++m)
                mine_red[(n * 2 + m) * 32 + lane] =
                    make_float4(sum[m][n][0], sum[m][n][1], sum[m][n][2], sum[m][n][3]);
            }
        }
        team_sync(team, WK);
        if (wk == 0) {
#pragma unroll
          for (int n = 0; n < kMaxNT; ++n)
            if (n < blocks) {
              for (int w = 0; w < WK - 1; ++w)
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                  const float4 v = red[(w * (p.cap / 8) + n) * 64 + m * 32 + lane];
                  sum[m][n][0] += v.x;
                  sum[m][n][1] += v.y;
                  sum[m][n][2] += v.z;
                  sum[m][n][3] += v.w;
                }
            }
          __syncwarp();
          // features x rows -> rows of 32 features in shared memory, then 16-byte stores
          __nv_bfloat16 *t = reinterpret_cast<__nv_bfloat16 *>(red);
#pragma unroll
          for (int n = 0; n < kMaxNT; ++n)
            if (n < blocks) {
#pragma unroll
              for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  t[(n * 8 + c * 2 + (i & 1)) * 32 + m * 16 + (i >> 1) * 8 + g] =
                      __float2bfloat16_rn(sum[m][n][i]);
            }
          __syncwarp();
          for (int i = lane; i < n_rows * 4; i += 32) {
            const int r = i >> 2, n = tile * kTileN + (i & 3) * 8;
            if (n < p.n_out)
              *reinterpret_cast<uint4 *>(p.out + (static_cast<int64_t>(rows[r]) * p.n_out + n) * 2) =
                  reinterpret_cast<const uint4 *>(t)[i];
          }
        }
        team_sync(team, WK);
      }
    }
    cp_async_wait_group<0>();
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
  const size_t jobs = (static_cast<size_t>(p.n_experts) + 1) * 4;
  const size_t ring = static_cast<size_t>(kWarps) * kDepth * kStage;
  // partial sums of all but the first warp of each tile (which reuses them to store)
  const size_t red = static_cast<size_t>(kWarps / p.wk) * (p.wk - 1) * nt * 1024;
  const size_t fixed = (jobs + 127) / 128 * 128 + ring + red;
  if (fixed >= kSmemMax) return kSmemMax + 1;
  // slices of x that fit beside them, in steps of wk; a row's stride is an odd
  // number of 64-byte halves, so that eight rows' pieces hit all banks
  p.chunk = (p.slices + p.wk - 1) / p.wk * p.wk;
  while (p.chunk > p.wk && fixed + static_cast<size_t>(p.cap) * (p.chunk * 256 + 64) > kSmemMax)
    p.chunk -= p.wk;
  p.x_stride = p.chunk * 256 + 64;
  const size_t x = (static_cast<size_t>(p.cap) * p.x_stride + 127) / 128 * 128;
  p.off_ring = static_cast<uint32_t>(x);
  p.off_red = static_cast<uint32_t>(x + ring);
  p.off_jobs = static_cast<uint32_t>(x + ring + red);
  return x + fixed;
}

template <int GC>
cudaError_t launch(const Q4Params &p, int grid, size_t smem, cudaStream_t s) {
  static std::once_flag once[64];
  static cudaError_t attr_err[64];
  int dev = 0;
  cudaGetDevice(&dev);
  std::call_once(once[dev & 63], [d = dev & 63] {
    attr_err[d] = cudaFuncSetAttribute(q4_kernel<GC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kSmemMax));
  });
  if (attr_err[dev & 63] != cudaSuccess) return attr_err[dev & 63];
  return launch_early(q4_kernel<GC>, grid, kThreads, smem, 1, s, p);
}

}  // namespace
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
  p.codes = codes;
  p.scales = scales;
  p.zeros = zeros;
  p.out = reinterpret_cast<uint8_t *>(out);
  p.n_slots = n_slots;
  p.k_in = k_in;
  p.n_out = n_out;
  p.top_k = top_k;
  p.n_experts = n_experts;
  p.tiles_per_job = (n_out + kTileN - 1) / kTileN;
  p.slices = (k_in + 127) / 128;
  // Rows per job: what an expert gets on average and two deviations more, so
  // that few experts need their codes twice.
  const double mean = static_cast<double>(n_slots) / std::max(1, n_experts);
  int nt = 1;
  while (nt < kMaxNT && 8 * nt < mean && (8 * nt - mean) * (8 * nt - mean) < 4 * mean) ++nt;
  // Warps per tile: few where there are tiles for every team of every SM.
  const int64_t hit = std::min<int64_t>(n_slots, n_experts);
  const int64_t per_sm = hit * p.tiles_per_job / sm_count();
  p.wk = per_sm >= 8 ? 2 : per_sm >= 4 ? 4 : per_sm >= 2 ? 8 : 16;
  size_t smem = layout(p, nt);
  while (nt > 1 && smem > kSmemMax) smem = layout(p, --nt);
  const int64_t most = std::max<int64_t>(hit * p.tiles_per_job, 1);
  const int grid = static_cast<int>(std::min<int64_t>(sm_count(), most));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(group == 32   ? launch<1>(p, grid, smem, s)
                     : group == 64 ? launch<2>(p, grid, smem, s)
                                   : launch<4>(p, grid, smem, s));
}
