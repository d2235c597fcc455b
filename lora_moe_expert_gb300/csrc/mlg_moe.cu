// mlg_moe.cu -- a whole MoE layer for a few tokens: the router's choice, then
// two kernels that stream the chosen experts' weights once.
//
// HBM bounds it: 3 hidden inter weights an expert, a handful of rows each, so the
// weights' rows are the M of the warp-wide products (m16n8k16) and the tokens the
// N.  A CTA has four warps of 16 weight rows each and four that feed them; two
// CTAs share an SM.  The feeders ask for 64 weight rows (256 bytes each, by TMA) and
// the rows of up to 16 of the expert's tokens (gathered by their index) a stage,
// ahead into a ring that goes on from one unit to the next: nothing is waited for
// but the data.  An expert of more tokens is taken again for those (from L2).
//  * gate and up: a unit is an expert and 32 channels, 32 gate rows beside the 32
//    up rows of the same channels, so that a lane ends with a channel's gate and up
//    and writes silu(gate) * up.  Units go round-robin over the CTAs.
//  * down: a CTA has 64 output channels and a share of the experts; it adds
//    weight * row for each into fp32 sums of all tokens in shared memory, and the
//    CTAs of a cluster (one share of the experts each) add theirs up in rank order.
//    Its weights do not depend on the kernel before it, so the first stages are
//    under way before that has ended.
// 8-bit weights become fp16 in registers, exactly, by the one instruction there is
// for two of them (to bf16 it takes five), and the tokens' rows fp16 times a power of two
// for each 128 values, exactly too but for what is 2^-29 below the largest; both scales go
// into the block's fp32 sum.  act has 16 bits a value (pack_act): with bf16 weights the second
// kernel takes it as the sum of two bf16 numbers, twice the products.
// Measured, 8 of 128 experts of 2048 x 768: bf16 1 token 21 us (3.6 TB/s; the choice and the starts
// of three dependent launches are 8 of them), 4 tokens 51 (5.4), 16 125 (6.2), 64 183 (6.5);
// in 8 bits 19, 16 tokens 77 (5.0) and 64 125, where the conversion beside the products is
// what bounds it (issue slots half busy).
// Every wait is bounded; a timeout sets an error bit and the CTA stops: what it has not
// summed becomes NaN, through act and the cluster's sums, in every output it belongs to.
#include <cuda.h>
#include <cuda_fp16.h>

#include <mutex>

#include "mlg_launch.cuh"
#include "mlg_tiles.cuh"
#include "mlg_tmap.cuh"

namespace mlg {
namespace {

constexpr int kMoeWarps = 4, kGatherWarps = 3;
constexpr int kMoeThreads = (kMoeWarps + 1 + kGatherWarps) * 32;
constexpr int kMoeRows = 16 * kMoeWarps;         // weight rows of a unit
constexpr uint32_t kMoeWBytes = kMoeRows * 256;  // of a stage: two boxes of 128 bytes a row
constexpr int kMoeMaxStages = 8;
constexpr int kMoeTokens = 16;                   // of an expert that a unit takes
// A stage's fp32 factors with 8-bit weights, for each of its two blocks of k: of the
// tokens' columns, and the scales of the weight rows, 8 at a time (two of each warp).
constexpr int kFactors = 2 * (kMoeTokens + 2 * kMoeWarps);
constexpr int kMoeMaxCluster = 8;
constexpr int64_t kMoePrefetch = 24 << 20;
constexpr uint32_t kMoeSmem = 227 * 1024 / 2 - 1024 - 512;  // a CTA's, two a multiprocessor

// What a stage holds along k: 128 bytes of a weight row are kBoxK values; the
// tokens' rows are boxes of 64 bf16 values, kXBoxes a stage.
template <bool F8>
struct MoeStage {
  static constexpr int kBoxK = F8 ? 128 : 64, kK = 2 * kBoxK, kXBoxes = kK / 64;
  static constexpr uint32_t kXBytes = kXBoxes * 8 * 128;  // of 8 tokens
};

static __device__ uint32_t g_moe_errors;
int g_moe_lose = 0;  // mlg_test_set_knob

struct MoeParams {
  const int32_t *indices;
  const float *weights;
  const float *scales;     // of 8-bit weights
  const __nv_bfloat16 *x;  // the tokens' rows: hidden states, then act
  const uint8_t *w_down;
  uint16_t *act;           // pack_act()'s, 8 channels a group
  __nv_bfloat16 *out;
  int32_t n_tokens, top_k, n_experts, hidden, inter;
  int32_t k, n, slices, k_steps, k_blocks;  // of this kernel's weights: values a row, rows, ...
  int32_t unit_tokens, stages, joined;  // joined: k is whole boxes
  int32_t log_parts;                    // a hit's k is 2^log_parts units of the second kernel
  uint32_t w_bytes;      // what a stage waits for of the weights: kMoeWBytes
  uint32_t rest_offset;  // of the second summands of act's rows, bf16 weights
  uint32_t stage_bytes, off_acc, off_mask, off_hits, off_slots, off_tokens, off_weights, off_ids,
      off_base, off_factors;
};

struct MoeCtl {
  uint64_t full[kMoeMaxStages], empty[kMoeMaxStages];
  int warp_total[kMoeWarps];
  int n_hits;
  volatile int abort_flag;
};

__device__ __forceinline__ bool wait_moe(MoeCtl &ctl, uint64_t &bar, uint32_t parity) {
  return wait_or_abort(ctl, bar, parity, &g_moe_errors);
}

__device__ __forceinline__ void tma_load_3d_moe(uint32_t dst, const void *tmap, int32_t x,
                                                int32_t y, int32_t z, uint32_t bar, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(pol)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d_moe(uint32_t dst, const void *tmap, int32_t x,
                                                int32_t y, int32_t z, int32_t w, uint32_t bar,
                                                uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar), "l"(pol)
      : "memory");
}
// 4-byte global -> shared copy; zeros where src_bytes is 0.
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void *src, uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(src_bytes)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void lds_v2(uint32_t addr, uint32_t &a, uint32_t &b) {
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr) : "memory");
}
// Four e4m3 codes as fp16 values, exactly.
__device__ __forceinline__ void e4m3_to_f16x2(uint32_t v, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}
// Products, m16n8k16, that the compiler may move (they touch registers alone).
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(0x80008000u));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(bf16hi_to_f32(w)), "f"(bf16lo_to_f32(w)));
  return r;
}

// 8 of the 128 bf16 values of a row, of which 16 adjacent lanes hold 8 each, to
// fp16 times a power of two that brings the largest of the 128 to [2^14, 2^15): exact
// down to 2^-29 of the largest, and what is below is off by at most 2^-39 of it.
// Returns the power's inverse.  (A block with an infinity or NaN keeps them.)
__device__ __forceinline__ float to_scaled_f16(uint4 &v) {
  uint32_t *w = reinterpret_cast<uint32_t *>(&v);
  uint32_t m = 0;  // the largest magnitude's bits, an integer maximum
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = max(m, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kFullWarp, m, o));
  const uint32_t field = min(268u - (m >> 7), 254u);  // of the power, a bf16 and an fp32 exponent
  const uint32_t power = field << 7 | field << 23;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = bf16x2_to_f16x2(mul_bf16x2(w[i], power));
  return __uint_as_float(field == 254 ? 0x00400000u : (254u - field) << 23);
}

// What the first kernel leaves for the second, 16 bits a value: 8 channels share a power of
// two, that brings the largest's exponent e to 14, and are fp16 times it, of which the last
// bit is not the value's but bit g of e: 10 bits of a value, rounded, the layer's error 1.03 times
// that of rounding its results alone (a value in bf16, of 8 bits: 1.4 times, and 8 to 10 % faster for
// one token and for 43 of 97 experts in bf16, 2 % in 8 bits).  e = 255, where one of the 8 is
// not finite, makes them all NaN.  The 8 values are those of the lanes that differ in g = lane / 4.
__device__ __forceinline__ uint16_t pack_act(float v, int g) {
  uint32_t m = __float_as_uint(v) & 0x7fffffffu;
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) m = max(m, __shfl_xor_sync(kFullWarp, m, o));
  const uint32_t e = max(m >> 23, 16u);
  // to 10 bits, to nearest: so many of the fp32 number, which fp16 then holds
  const float f = v * __uint_as_float((268u - e) << 23);  // below 2^15
  const uint32_t ten = (__float_as_uint(f) + 0x1fffu + (__float_as_uint(f) >> 14 & 1)) & ~0x3fffu;
  const uint32_t h = __half_as_ushort(__float2half_rn(__uint_as_float(ten)));
  return static_cast<uint16_t>((h & 0xfffeu) | (e >> g & 1));
}
// Their e, and the 8 values as fp16 times 2^(141 - e).
__device__ __forceinline__ uint32_t unpack_act(uint4 &v) {
  uint32_t *w = reinterpret_cast<uint32_t *>(&v), e = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e |= (w[i] & 0x10001u) << (2 * i);  // channel 2 i's bit at 2 i, the other's at 16 + 2 i
    w[i] &= 0xfffefffeu;
  }
  return (e | e >> 15) & 0xffu;
}
// To fp16 times a power of two for each 128 values, of which 16 adjacent lanes hold 8 each.
// Returns the power's inverse.
__device__ __forceinline__ float act_to_f16(uint4 &v) {
  const uint32_t e = unpack_act(v);
  uint32_t most = e;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(kFullWarp, most, o));
  // 2^(e - most) in two fp16 factors: the first a normal number, the second down to 2^-24,
  // and 0 from there on, where the values would be less than half of fp16's least number
  const uint32_t down = most - e, one = min(down, 14u), two = min(down - one, 25u);
  const uint32_t f1 = (15u - one) << 10, f2 = two <= 14 ? (15u - two) << 10 : (1u << 24) >> two;
  uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{\n\t.reg .b32 t;\n\tmul.rn.f16x2 t, %1, %2;\n\tmul.rn.f16x2 %0, t, %3;\n\t}"
        : "=r"(w[i])
        : "r"(w[i]), "r"(f1 | f1 << 16), "r"(f2 | f2 << 16));
  return __uint_as_float(most == 255 ? 0x7fc00000u : (max(most, 15u) - 14) << 23);
}
// To two bf16 numbers each, whose sum is the value: its first 8 bits and the others.
__device__ __forceinline__ void act_to_bf16(uint4 &v, uint4 &rest) {
  const uint32_t e = unpack_act(v);
  const float power = __uint_as_float(e == 255 ? 0x7fc00000u : (max(e, 14u) - 14) << 23);
  uint32_t *w = reinterpret_cast<uint32_t *>(&v), *r = reinterpret_cast<uint32_t *>(&rest);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 f = __half22float2(*reinterpret_cast<const __half2 *>(w + i));
    f = __fmul2_rn(f, make_float2(power, power));
    const uint32_t a = __float_as_uint(f.x), b = __float_as_uint(f.y);
    w[i] = __byte_perm(a, b, 0x7632);
    const float c = f.x - __uint_as_float(a & 0xffff0000u);
    const float d = f.y - __uint_as_float(b & 0xffff0000u);
    r[i] = __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x7632);
  }
}

// The experts that were chosen, each with its rows by token, up to kMoeTokens a hit:
// hits[i] = (expert, first row << 8 | rows), and for the rows slots[], tokens[] and
// weights[].  Up to 32 slots one warp compares them (the experts in the order of the slots;
// the other way takes 1 us longer).  More: a token chooses an expert once at most, so a
// bit a token says it all, in whatever order the bits come (the experts in the order of
// their ids).  mask: zeros; ids, base: scratch.
struct Hits {
  unsigned long long *mask;  // [n_experts]
  int2 *hits;
  uint16_t *slots, *tokens, *ids, *base;
  float *weights;
};
template <bool DOWN>
__device__ void find_hits(const MoeParams &p, MoeCtl &ctl, const Hits &o) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_slots = p.n_tokens * p.top_k, E = p.n_experts;
  if (n_slots <= 32 && p.n_tokens <= p.unit_tokens) {
    if (warp == 0) {
      const int mine = lane < n_slots ? __ldcg(p.indices + lane) : -1;
      const float w = DOWN && lane < n_slots ? __ldcg(p.weights + lane) : 0.0f;
      const bool there = mine >= 0 && mine < E;
      const unsigned same = __match_any_sync(kFullWarp, there ? mine : -1 - lane);
      const unsigned before = (1u << lane) - 1;
      const bool leads = there && (same & before) == 0;
      const unsigned leaders = __ballot_sync(kFullWarp, leads);
      const int n = __popc(same);
      int base = leads ? n : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(kFullWarp, base, d);
        if (lane >= d) base += v;
      }
      base -= leads ? n : 0;
      const int at = __shfl_sync(kFullWarp, base, __ffs(same) - 1) + __popc(same & before);
      if (leads) o.hits[__popc(leaders & before)] = make_int2(mine, base << 8 | n);
      if (there) {
        o.slots[at] = static_cast<uint16_t>(lane);
        o.tokens[at] = static_cast<uint16_t>(lane / p.top_k);
        if (DOWN) o.weights[at] = w;
      }
      if (lane == 0) ctl.n_hits = __popc(leaders);
    }
    __syncthreads();
    return;
  }
  // the first slot of every thread stays in registers: mostly there are no others
  const int first = tid < n_slots ? __ldcg(p.indices + tid) : -1;
  const float first_w = DOWN && tid < n_slots ? __ldcg(p.weights + tid) : 0.0f;
  for (int s = tid; s < n_slots; s += kMoeThreads) {
    const int e = s == tid ? first : __ldcg(p.indices + s);
    const bool there = e >= 0 && e < E;
    o.ids[s] = there ? static_cast<uint16_t>(e) : 0xffffu;
    if (there) atomicOr(o.mask + e, 1ull << (s / p.top_k));
  }
  __syncthreads();
  constexpr int kScan = kMoeWarps * 32;
  const int share = (E + kScan - 1) / kScan;  // experts a thread, one after the other
  int own = 0, incl = 0;                      // hits << 16 | rows
  if (tid < kScan) {
    for (int i = 0; i < share; ++i) {
      const int e = tid * share + i;
      const int n = e < E ? __popcll(o.mask[e]) : 0;
      own += (n + p.unit_tokens - 1) / p.unit_tokens << 16 | n;
    }
    incl = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(kFullWarp, incl, d);
      if (lane >= d) incl += v;
    }
    if (lane == 31) ctl.warp_total[warp] = incl;
  }
  __syncthreads();
  if (tid < kScan) {
    int at = incl - own;
    for (int w = 0; w < warp; ++w) at += ctl.warp_total[w];
    for (int i = 0; i < share; ++i) {
      const int e = tid * share + i;
      const int n = e < E ? __popcll(o.mask[e]) : 0;
      if (n == 0) continue;
      o.base[e] = static_cast<uint16_t>(at & 0xffff);
      for (int c = 0; c < n; c += p.unit_tokens) {
        const int some = min(n - c, p.unit_tokens);
        o.hits[at >> 16] = make_int2(e, (at & 0xffff) << 8 | some);
        at += (1 << 16) + some;
      }
    }
    if (tid == kScan - 1) ctl.n_hits = at >> 16;
  }
  __syncthreads();
  for (int s = tid; s < n_slots; s += kMoeThreads) {
    const int e = o.ids[s], t = s / p.top_k;
    if (e == 0xffff) continue;
    const int at = o.base[e] + __popcll(o.mask[e] & ((1ull << t) - 1));
    o.slots[at] = static_cast<uint16_t>(s);
    o.tokens[at] = static_cast<uint16_t>(t);
    if (DOWN) o.weights[at] = s == tid ? first_w : __ldcg(p.weights + s);
  }
  __syncthreads();
}

// A unit: a hit, a slice (64 weight rows) and a range of k in stages.
struct MoeUnit {
  int hit, slice, k0, k1;
};
// This CTA's unit i.
template <bool DOWN>
__device__ __forceinline__ bool unit_at(const MoeParams &p, int n_hits, int i, MoeUnit &u) {
  if (DOWN) {  // the cluster's slice, this rank's share of the hits or of their parts
    const int n = cluster_ctarank() + i * cluster_size();
    u.hit = n >> p.log_parts;
    const int part = n - (u.hit << p.log_parts);
    u.slice = cluster_id_x();
    u.k0 = part * p.k_steps >> p.log_parts, u.k1 = (part + 1) * p.k_steps >> p.log_parts;
    return u.hit < n_hits;
  }
  const int n = blockIdx.x + i * gridDim.x;
  u.hit = n / p.slices;
  u.slice = n - u.hit * p.slices;
  u.k0 = 0, u.k1 = p.k_steps;
  return u.hit < n_hits;
}

// One stage's products of a warp's 16 rows with J blocks of 8 tokens (the columns
// past an expert's tokens hold whatever is there: no column reaches another).
// Everything is unrolled without a branch, so that the loads and conversions of
// the whole stage run ahead of the products that wait for one another.
//   ws, xs  this lane's weight row for ldmatrix and the stage's tokens' rows
//   next    bytes from one box of the weight rows to the other
//   factors the stage's, of 8-bit weights
//   rest    bytes from the tokens' rows to the second summands of theirs (REST)
template <bool F8, int J, int NB, bool REST>
__device__ __forceinline__ void stage_products(float (&acc)[4][NB][4],
                                               uint32_t ws, uint32_t xs, uint32_t next,
                                               uint32_t rest, const float *factors, int warp) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, sub = lane >> 3, r8 = lane & 7;
  constexpr uint32_t kXBytes = MoeStage<F8>::kXBytes;
  if (F8) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // a block of 128
      float part[2][J][4];         // two sums, so that half as many products wait in line
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) part[q][j][c] = 0.0f;
      uint32_t a[4][4], x[8][J][2];
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)  // 32 values of k: two 16-byte pieces a row
        ldmatrix_x4(ws + h * next + (((2 * kk + (sub >> 1)) ^ r8) << 4), a[kk]);
#pragma unroll
      for (int k16 = 0; k16 < 8; ++k16)
#pragma unroll
        for (int j = 0; j < J; ++j)
          lds_v2(xs + j * kXBytes + (2 * h + (k16 >> 2)) * 1024 + g * 128 +
                     (((2 * (k16 & 3) + (t >> 1)) ^ g) << 4) + (t & 1) * 8,
                 x[k16][j][0], x[k16][j][1]);
#pragma unroll
      for (int k16 = 0; k16 < 8; ++k16) {
        const int kk = k16 >> 1, q = k16 & 1;
        uint32_t b[4];  // rows g, g + 8: values 4t, 4t+1; the same: 4t+2, 4t+3
        e4m3_to_f16x2(a[kk][2 * q], b[0], b[2]);
        e4m3_to_f16x2(a[kk][2 * q + 1], b[1], b[3]);
#pragma unroll
        for (int j = 0; j < J; ++j) mma_f16_16816(part[q][j], b, x[k16][j][0], x[k16][j][1]);
      }
      const float *f = factors + h * (kFactors / 2);
      const float2 scale = *reinterpret_cast<const float2 *>(f + kMoeTokens + 2 * warp);
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const float2 xp = *reinterpret_cast<const float2 *>(f + j * 8 + 2 * t);
        acc[0][j][0] += scale.x * xp.x * (part[0][j][0] + part[1][j][0]);
        acc[0][j][1] += scale.x * xp.y * (part[0][j][1] + part[1][j][1]);
        acc[0][j][2] += scale.y * xp.x * (part[0][j][2] + part[1][j][2]);
        acc[0][j][3] += scale.y * xp.y * (part[0][j][3] + part[1][j][3]);
      }
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t a[4][4], b[2][J][4];
#pragma unroll
      for (int k16 = 0; k16 < 4; ++k16)
        ldmatrix_x4(ws + h * next + (((2 * k16 + (sub >> 1)) ^ r8) << 4), a[k16]);
#pragma unroll
      for (int pair = 0; pair < 2; ++pair)  // 32 values of k
#pragma unroll
        for (int j = 0; j < J; ++j)
          ldmatrix_x4(xs + j * kXBytes + h * 1024 + r8 * 128 + (((4 * pair + sub) ^ r8) << 4),
                      b[pair][j]);
#pragma unroll
      for (int pair = 0; pair < 2; ++pair)
#pragma unroll
        for (int j = 0; j < J; ++j) {
          // four sums: the products that wait for one another are four a stage
          mma_16816(acc[2 * pair][j], a[2 * pair], b[pair][j][0], b[pair][j][1]);
          mma_16816(acc[2 * pair + 1][j], a[2 * pair + 1], b[pair][j][2], b[pair][j][3]);
        }
      if constexpr (REST) {
#pragma unroll
        for (int pair = 0; pair < 2; ++pair)
#pragma unroll
          for (int j = 0; j < J; ++j) {
            ldmatrix_x4(xs + rest + j * kXBytes + h * 1024 + r8 * 128 +
                            (((4 * pair + sub) ^ r8) << 4),
                        b[pair][j]);
            mma_16816(acc[2 * pair][j], a[2 * pair], b[pair][j][0], b[pair][j][1]);
            mma_16816(acc[2 * pair + 1][j], a[2 * pair + 1], b[pair][j][2], b[pair][j][3]);
          }
      }
    }
  }
}

// F8: 8-bit weights.  DOWN: the second kernel.  NB: blocks of 8 tokens of a unit.
template <bool F8, bool DOWN, int NB>
__global__ void __launch_bounds__(kMoeThreads, 2)
    moe_kernel(const __grid_constant__ CUtensorMap tmap_w, const MoeParams p) {
  using Stage = MoeStage<F8>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ MoeCtl ctl;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Hits found = {reinterpret_cast<unsigned long long *>(smem + p.off_mask),
                      reinterpret_cast<int2 *>(smem + p.off_hits),
                      reinterpret_cast<uint16_t *>(smem + p.off_slots),
                      reinterpret_cast<uint16_t *>(smem + p.off_tokens),
                      reinterpret_cast<uint16_t *>(smem + p.off_ids),
                      reinterpret_cast<uint16_t *>(smem + p.off_base),
                      reinterpret_cast<float *>(smem + p.off_weights)};
  const int2 *hits = found.hits;
  float *factors = reinterpret_cast<float *>(smem + p.off_factors);  // [stages][kFactors], F8
  float *sums = reinterpret_cast<float *>(smem + p.off_acc);       // [tokens][64], DOWN
  // A stage's weights: [box][64 rows][128 bytes], or the gates' two boxes and the ups'.
  constexpr int kLoadRows = DOWN ? kMoeRows : kMoeRows / 2;
  constexpr uint32_t kNextBox = kLoadRows * 128;

  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(smem_addr(&ctl.full[s]), 1 + 32);  // the weights' bytes, a warp of the rows' ones
      mbar_init(smem_addr(&ctl.empty[s]), kMoeWarps);
    }
    ctl.abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmap_w);
  }
  if (DOWN)
    for (int i = tid; i < p.n_tokens * kMoeRows; i += kMoeThreads) sums[i] = 0.0f;
  for (int e = tid; e < p.n_experts; e += kMoeThreads) found.mask[e] = 0;
  __syncthreads();
  if (!DOWN) {
    griddep_wait();
    griddep_launch_dependents();
  }
  // In the second kernel the choice, like the weights, was complete before the
  // first kernel let this one start; only `act` has to be waited for.
  find_hits<DOWN>(p, ctl, found);
  const int n_hits = ctl.n_hits;
  const uint32_t ring = smem_addr(smem);

  if (warp == kMoeWarps) {
    if (lane == 0) {
      // ============================================================ the weights
      const uint64_t policy = l2_evict_first();
      uint32_t it = 0;
      MoeUnit u;
      for (int i = 0; unit_at<DOWN>(p, n_hits, i, u); ++i) {
        const int e = hits[u.hit].x;
        for (int ks = u.k0; ks < u.k1; ++ks, ++it) {
          const int st = it % p.stages;
          if (!wait_moe(ctl, ctl.empty[st], ((it / p.stages) & 1) ^ 1)) goto fed;
          const uint32_t full = smem_addr(&ctl.full[st]), to = ring + st * p.stage_bytes;
          mbar_arrive_expect_tx(full, p.w_bytes);
#pragma unroll
          for (int v = 0; v < (DOWN ? 1 : 2); ++v) {  // the gates' rows, the ups'
            const int row = u.slice * kLoadRows + v * p.inter;
            const uint32_t at = to + v * 2 * kNextBox;
            if (p.joined) {
              tma_load_4d_moe(at, &tmap_w, 0, row, 2 * ks, e, full, policy);
            } else {
              tma_load_3d_moe(at, &tmap_w, ks * Stage::kK, row, e, full, policy);
              tma_load_3d_moe(at + kNextBox, &tmap_w, ks * Stage::kK + Stage::kBoxK, row, e, full,
                              policy);
            }
          }
        }
      }
      if (!DOWN) {
        // HBM would idle until the second kernel's CTAs are there: what each of them asks
        // for first goes to L2 meanwhile (an expert of each rank of a cluster), up to 24 MB
        // (one token, 8 experts of 2048 x 2048: 36.0 us, without that limit 38.9, without
        // prefetch 36.5; of 2048 x 768 21.1, 20.8 and 22.2).
        const int slices = (p.hidden + kMoeRows - 1) / kMoeRows, size = F8 ? 1 : 2;
        const int64_t most = kMoePrefetch / (int64_t{kMoeRows} * p.inter * size);
        const int first = static_cast<int>(
            min(int64_t{min(n_hits, kMoeMaxCluster)} * slices, most));
        for (int n = blockIdx.x; n < first; n += gridDim.x) {
          const int row = n % slices * kMoeRows, rows = min(kMoeRows, p.hidden - row);
          const int64_t at = (int64_t{hits[n / slices].x} * p.hidden + row) * p.inter * size;
          prefetch_l2(p.w_down + at, static_cast<uint32_t>(rows * p.inter * size));
        }
      }
    fed:
      const uint64_t t0 = global_timer_ns();
      for (uint32_t k = 0; k < static_cast<uint32_t>(p.stages) && k < it; ++k) {
        const uint32_t j = it - 1 - k;  // nothing is under way when the CTA ends
        mbar_wait_until(smem_addr(&ctl.full[j % p.stages]), (j / p.stages) & 1, t0);
      }
    }
    __syncwarp();
  } else if (warp > kMoeWarps) {
    // ============================================================== the tokens' rows
    // Gathered by 16-byte copies into the places that swizzled boxes would have, 16
    // or 32 lanes a row.  (As TMA gathers of four rows, at some 40 ns each a
    // multiprocessor, they took longer than the weights.)
    if (DOWN) {
      griddep_wait();
      griddep_launch_dependents();
    }
    // The warps take turns, a stage each; no more of them than stages, so that a warp's
    // last stage is at most one round of the ring away from its next (a wait by parity
    // cannot tell two rounds from none).  With 8-bit weights the rows become fp16 here, and
    // act's two bf16 summands with bf16 weights, in place, once their copies are there: a
    // warp asks for its next stage first where that is free already.
    constexpr bool kConvert = F8 || DOWN;
    constexpr int kLanes = Stage::kK / 8, kAtOnce = 32 / kLanes;
    const int turn = warp - kMoeWarps - 1, turns = min(kGatherWarps, p.stages);
    const int c = lane % kLanes, j0 = lane / kLanes;
    const uint16_t *source = DOWN ? found.slots : found.tokens;
    uint32_t it = 0, last = 0;
    MoeUnit u;
    int last_n = -1;  // the stage whose copies are under way, and its rows
    auto place = [&](uint32_t i, int j) {
      return (i % p.stages) * p.stage_bytes + kMoeWBytes + (j >> 3) * Stage::kXBytes +
             (c >> 3) * 1024 + (j & 7) * 128 + (((c & 7) ^ (j & 7)) << 4);
    };
    auto convert = [&](uint32_t i, int n) {
      if (!F8) {  // each lane its own copies
        for (int j = j0; j < n; j += kAtOnce) {
          uint4 *at = reinterpret_cast<uint4 *>(smem + place(i, j)), v = *at, rest;
          act_to_bf16(v, rest);
          *at = v;
          at[p.rest_offset / 16] = rest;
        }
        mbar_arrive(smem_addr(&ctl.full[i % p.stages]));
        return;
      }
      float *to = factors + (i % p.stages) * kFactors + (c >> 4) * (kFactors / 2);
      for (int j = 0; j < n; j += 4) {  // each lane its own copies, four rows' at once
        uint4 v[4] = {};
        float power[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (j + q < n) v[q] = *reinterpret_cast<const uint4 *>(smem + place(i, j + q));
#pragma unroll
        for (int q = 0; q < 4; ++q) power[q] = DOWN ? act_to_f16(v[q]) : to_scaled_f16(v[q]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (j + q >= n) break;
          *reinterpret_cast<uint4 *>(smem + place(i, j + q)) = v[q];
          if (c % 16 == 0) to[j + q] = power[q];
        }
      }
      mbar_arrive(smem_addr(&ctl.full[i % p.stages]));
    };
    for (int i = 0; unit_at<DOWN>(p, n_hits, i, u); ++i) {
      const int2 h = hits[u.hit];
      const int n = h.y & 0xff;
      const uint16_t *r = source + (h.y >> 8);
      for (int ks = u.k0; ks < u.k1; ++ks, ++it) {
        if (static_cast<int>(it % turns) != turn) continue;  // (never for one past the turns)
        const int st = it % p.stages;
        const uint32_t parity = ((it / p.stages) & 1) ^ 1;
        if (kConvert && last_n >= 0 &&  // (the lanes go the same way)
            !__all_sync(kFullWarp, mbar_test_wait(smem_addr(&ctl.empty[st]), parity))) {
          cp_async_wait_group<0>();
          convert(last, last_n);
          last_n = -1;
        }
        if (!wait_moe(ctl, ctl.empty[st], parity)) goto gathered;
        const int k = ks * Stage::kK + c * 8;
        for (int j = j0; j < n; j += kAtOnce) {
          const __nv_bfloat16 *src = p.x + int64_t{r[j]} * p.k + (k < p.k ? k : 0);
          cp_async_16(ring + place(it, j), src, k < p.k ? 16u : 0u);
        }
        if (!kConvert) {
          cp_async_arrive_noinc(smem_addr(&ctl.full[st]));
          continue;
        }
        if (F8 && lane < 4 * kMoeWarps) {  // the scales: late they would be if asked for by who needs them
          const int b = lane / (2 * kMoeWarps), q = lane % (2 * kMoeWarps), block = 2 * ks + b;
          const int row = DOWN ? u.slice * kMoeRows + q * 8
                               : u.slice * kLoadRows + (q >> 1) * 8 + (q & 1) * p.inter;
          const int blocks = (p.n + MLG_F8_BLOCK - 1) / MLG_F8_BLOCK;
          const bool there = block < p.k_blocks;
          const float *src = p.scales + (int64_t{h.x} * blocks + min(row / MLG_F8_BLOCK, blocks - 1)) *
                                            p.k_blocks + (there ? block : 0);
          cp_async_4(smem_addr(factors + st * kFactors + b * (kFactors / 2) + kMoeTokens + q), src,
                     there ? 4u : 0u);
        }
        cp_async_commit();
        if (last_n >= 0) {
          cp_async_wait_group<1>();
          convert(last, last_n);
        }
        last = it, last_n = n;
      }
    }
    if (last_n >= 0) {
      cp_async_wait_group<0>();
      convert(last, last_n);
    }
  gathered:
    cp_async_wait_group<0>();
    __syncwarp();
  } else {
    // ================================================================ the products
    const int g = lane >> 2, t = lane & 3;
    // this lane's row of the matrices that ldmatrix takes: weights in the order
    // (rows 0-7, 8-15) x (k 0-7, 8-15); rows 8-15 are the up rows in the first kernel
    const int sub = lane >> 3, r8 = lane & 7;
    const uint32_t w_row = DOWN ? (warp * 16 + (sub & 1) * 8 + r8) * 128
                                : (sub & 1) * 2 * kNextBox + (warp * 8 + r8) * 128;
    const int n_lo = DOWN ? warp * 16 : warp * 8;  // the first of this warp's rows
    uint32_t it = 0;
    MoeUnit u;
    bool whole = true;  // until a wait runs out: nothing is waited for from then on
    for (int i = 0; unit_at<DOWN>(p, n_hits, i, u); ++i) {
      const int2 h = hits[u.hit];
      const int n = h.y & 0xff, first = h.y >> 8;
      float acc[4][NB][4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[q][j][c] = 0.0f;
      for (int ks = whole ? u.k0 : u.k1; ks < u.k1; ++ks, ++it) {
        const int st = it % p.stages;
        if (!wait_moe(ctl, ctl.full[st], (it / p.stages) & 1)) {
          whole = false;
          break;
        }
        const uint32_t ws = ring + st * p.stage_bytes + w_row;
        const uint32_t xs = ring + st * p.stage_bytes + kMoeWBytes;
        const float *f = factors + st * kFactors;
        if (NB == 1 || n <= 8)
          stage_products<F8, 1, NB, DOWN && !F8>(acc, ws, xs, kNextBox, p.rest_offset, f, warp);
        else
          stage_products<F8, NB, NB, DOWN && !F8>(acc, ws, xs, kNextBox, p.rest_offset, f, warp);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&ctl.empty[st]));
      }
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          acc[0][j][c] = whole ? (acc[0][j][c] + acc[1][j][c]) + (acc[2][j][c] + acc[3][j][c])
                               : __uint_as_float(0x7fc00000u);
      // acc[0][j][c]: row g (c < 2) or g + 8, token column 8 j + 2 t + (c & 1)
      if (!DOWN) {
        const int channel = u.slice * kLoadRows + n_lo + g;
        if (channel < p.inter) {
#pragma unroll
          for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int col = 8 * j + 2 * t + c;
              const float gate = acc[0][j][c], up = acc[0][j][2 + c];
              const uint16_t v = pack_act(gate / (1.0f + expf(-gate)) * up, g);  // (all lanes)
              if (col < n) p.act[int64_t{found.slots[first + col]} * p.inter + channel] = v;
            }
        }
      } else {
        // this warp's rows are its own, and a column is one token's: no two lanes meet
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int col = 8 * j + 2 * t + c;
            if (col >= n) continue;
            const float w = found.weights[first + col];
            float *to = sums + found.tokens[first + col] * kMoeRows + n_lo + g;
            to[0] += w * acc[0][j][c];
            to[8] += w * acc[0][j][2 + c];
          }
        __syncwarp();
      }
    }
    __syncwarp();
  }
  if (!DOWN) return;
  cluster_sync();
  // Every rank adds up a share of the tokens, over the ranks in their order.
  const int ranks = cluster_size(), rank = cluster_ctarank();
  const int quads = p.n_tokens * (kMoeRows / 4);
  for (int q = rank * kMoeThreads + tid; q < quads; q += ranks * kMoeThreads) {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int c = 0; c < ranks; ++c) {
      const float4 o = ld_dsmem_f4(map_to_rank(smem_addr(sums) + q * 16, c));
      v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
    }
    const int token = q / (kMoeRows / 4);
    const int col = cluster_id_x() * kMoeRows + q % (kMoeRows / 4) * 4;
    if (col < p.hidden)
      *reinterpret_cast<uint2 *>(p.out + int64_t{token} * p.hidden + col) =
          make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  }
  cluster_sync();
}

// ------------------------------------------------------------------ host side
// Weights [experts, n, k]: boxes of `rows` rows x 128 bytes of one expert, and where
// k is whole boxes, pairs of them (the boxes along k are a dimension of their own).
bool map_weights(CUtensorMap *map, const void *w, bool f8, bool joined, int64_t k, int64_t n,
                 int64_t experts, uint32_t rows) {
  const cuuint64_t size = f8 ? 1 : 2, in_box = 128 / size, K = static_cast<cuuint64_t>(k),
                   N = static_cast<cuuint64_t>(n), E = static_cast<cuuint64_t>(experts);
  const cuuint64_t dims[4] = {joined ? in_box : K, N, joined ? K / in_box : E, E};
  const cuuint64_t strides[3] = {K * size, joined ? 128 : K * N * size, K * N * size};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(in_box), rows, joined ? 2u : 1u, 1};
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return encode_fn()(map, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                     joined ? 4 : 3, const_cast<void *>(w), dims, strides, box, ones,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

using MoeKernel = void (*)(CUtensorMap, MoeParams);
template <bool F8, bool DOWN>
MoeKernel moe_kernel_of(int unit_tokens) {
  return unit_tokens <= 8 ? moe_kernel<F8, DOWN, 1> : moe_kernel<F8, DOWN, 2>;
}

cudaError_t allow_moe_smem() {
  static std::once_flag once[64];
  static cudaError_t err[64];
  int dev = 0;
  cudaGetDevice(&dev);
  std::call_once(once[dev & 63], [d = dev & 63] {
    cudaError_t e = cudaSuccess;
    for (int n : {8, kMoeTokens})
      for (MoeKernel k : {moe_kernel_of<false, false>(n), moe_kernel_of<false, true>(n),
                          moe_kernel_of<true, false>(n), moe_kernel_of<true, true>(n)})
        if (e == cudaSuccess) e = allow_smem(k, kMoeSmem);
    err[d] = e;
  });
  return err[dev & 63];
}

uint32_t up16(uint32_t v) { return (v + 15) / 16 * 16; }

// Lays out a CTA's shared memory: as many stages as there is room for (two and more: the
// tables take 57 KB at most).
uint32_t plan_moe(MoeParams &p, bool f8, bool down) {
  const uint32_t slots = p.n_tokens * p.top_k, experts = p.n_experts;
  const uint32_t most = (slots < experts ? slots : experts) + slots / p.unit_tokens;  // hits
  uint32_t off = 0;
  auto take = [&](uint32_t bytes) {
    const uint32_t at = off;
    off += up16(bytes);
    return at;
  };
  p.off_acc = take(down ? p.n_tokens * kMoeRows * 4 : 0);
  p.off_mask = take(experts * 8);
  p.off_hits = take(most * 8);
  p.off_slots = take(slots * 2);
  p.off_tokens = take(slots * 2);
  p.off_ids = take(slots * 2);
  p.off_weights = take(down ? slots * 4 : 0);
  p.off_base = take(experts * 2);
  p.off_factors = take(f8 ? kMoeMaxStages * kFactors * 4 : 0);
  p.rest_offset =
      p.unit_tokens / 8 * (f8 ? MoeStage<true>::kXBytes : MoeStage<false>::kXBytes);
  p.stage_bytes = kMoeWBytes + (down && !f8 ? 2 : 1) * p.rest_offset;
  p.stages = static_cast<int32_t>((kMoeSmem - 1024 - off) / p.stage_bytes);
  if (p.stages > kMoeMaxStages) p.stages = kMoeMaxStages;
  const uint32_t ring = p.stages * p.stage_bytes;  // first, on its boundary of 1024
  for (uint32_t *o : {&p.off_acc, &p.off_mask, &p.off_hits, &p.off_slots, &p.off_tokens, &p.off_ids,
                      &p.off_weights, &p.off_base, &p.off_factors})
    *o += ring;
  return ring + off + 1024;
}

// Ranks of a cluster of the second kernel, which share its hits, and p.log_parts.
//  * 8, that both CTAs of a multiprocessor have work (16 tokens, 8 of 128 experts of 2048 x 768 in
//    8 bits: 77.7 us, with 4 ranks 95.3), but no more CTAs than find a place at once (one
//    token, 8 experts of 6144 x 1024, bf16: 51.7 us with 2 ranks, 57.0 with 4).
//  * Half of them where so many, or most of them, find a place beside the first kernel's, and
//    are there when it ends, and twice as many do not: one token, 8 experts of 2048 x 768 in
//    8 bits 18.9 us, with 8 ranks 22.5; 2 tokens, 4 experts of 2048 x 768 18.6 and 22.6; 8 of
//    2816 x 640 in bf16 22.6 and 26.7.  Where all find a place in the end it may lose some: 8 of
//    2048 x 768 in bf16 20.9 and 20.4, 2 tokens 21.3 and 20.0, 8 of 2048 x 512 16.5 and 16.0.
//  * Few hits may not come out even, so the ranks share a hit's k too, two stages and more a
//    part (one token, 2 experts of 4096 x 8192, bf16 64.5 us, whole 71.7, in 8 bits 42.4 and
//    51.7).  Many come out even enough (43 tokens, 6 of 97 experts 61.9 us, in parts 63.1).
int ranks_of(MoeParams &p, int64_t hits, int64_t up_grid) {
  const int64_t places = 2 * sm_count(), left = places - up_grid;
  const auto most_fit = [&](int ranks) { return 4 * left >= 3 * int64_t{ranks} * p.slices; };
  int ranks = kMoeMaxCluster;
  while (ranks > 1 && int64_t{ranks} * p.slices > places) ranks /= 2;
  if (ranks > 2 && !most_fit(ranks) && most_fit(ranks / 2)) ranks /= 2;
  int64_t least = INT64_MAX;  // stages of the rank that has the most
  for (int log = 0; log == 0 || (hits <= 2 * kMoeMaxCluster && p.k_steps >> log >= 2); ++log) {
    const int64_t stages =
        ((hits << log) + ranks - 1) / ranks * ((p.k_steps + (1 << log) - 1) >> log);
    if (stages < least) least = stages, p.log_parts = log;
    if (1 << log >= ranks) break;
  }
  return ranks;
}

mlg_status moe_layer(const void *logits, int32_t logits_type, int64_t ld_logits, const mlg_bf16 *x,
                     const void *w_gate_up, const float *gate_up_scales, const void *w_down,
                     const float *down_scales, bool f8, int32_t *indices, float *weights,
                     mlg_bf16 *act, mlg_bf16 *out, int32_t n_tokens, int32_t hidden, int32_t inter,
                     int32_t n_experts, int32_t top_k, int32_t renormalize, cudaStream_t stream) {
  if (n_tokens < 0 || hidden < 1 || inter < 1 || n_experts < 1 || top_k < 1 ||
      !known_type(logits_type) || ld_logits < n_experts)
    return MLG_ERR_INVALID_ARG;
  const int32_t whole = f8 ? 16 : 8;
  if (n_tokens > MLG_MOE_MAX_TOKENS || hidden % whole != 0 || inter % whole != 0 ||
      hidden > MLG_MOE_MAX_WIDTH || inter > MLG_MOE_MAX_WIDTH || n_experts > MLG_ROUTE_MAX_EXPERTS || top_k > MLG_ROUTE_MAX_TOP_K)
    return MLG_ERR_UNSUPPORTED;
  if (n_tokens == 0) return MLG_OK;
  if (!x || !w_gate_up || !w_down || !act || !out || !logits || !indices || !weights ||
      (f8 && (!gate_up_scales || !down_scales)))
    return MLG_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w_gate_up) || !aligned16(w_down) || !aligned16(act) ||
      !aligned16(out) || !aligned4(indices) || !aligned4(weights) || !aligned4(gate_up_scales) ||
      !aligned4(down_scales) || (reinterpret_cast<uintptr_t>(logits) & (type_size(logits_type) - 1)) != 0)
    return MLG_ERR_UNSUPPORTED;
  if (encode_fn() == nullptr) return MLG_ERR_CUDA;
  cudaError_t err = allow_moe_smem();
  if (err != cudaSuccess) return cuda_status(err);

  MoeParams up = {}, down = {};
  up.indices = indices, up.weights = weights;
  up.act = reinterpret_cast<uint16_t *>(act), up.out = reinterpret_cast<__nv_bfloat16 *>(out);
  up.n_tokens = n_tokens, up.top_k = top_k, up.n_experts = n_experts;
  up.hidden = hidden, up.inter = inter;
  down = up;
  up.scales = gate_up_scales, down.scales = down_scales;
  up.x = reinterpret_cast<const __nv_bfloat16 *>(x);
  down.x = reinterpret_cast<const __nv_bfloat16 *>(act);
  up.w_down = static_cast<const uint8_t *>(w_down);
  up.k = hidden, up.n = 2 * inter, up.slices = (inter + kMoeRows / 2 - 1) / (kMoeRows / 2);
  down.k = inter, down.n = hidden, down.slices = (hidden + kMoeRows - 1) / kMoeRows;
  // Tokens that a unit takes: 8 where an expert seldom has more, which leaves more of the
  // shared memory to the stages (64 tokens in 8 bits, 4 an expert: 126 us, with 16 143).
  const int64_t slots = int64_t{n_tokens} * top_k;
  const int32_t unit_tokens = n_tokens <= 8 || slots <= 6 * int64_t{n_experts} ? 8 : kMoeTokens;
  for (MoeParams *q : {&up, &down}) {
    const int32_t stage_k = f8 ? MoeStage<true>::kK : MoeStage<false>::kK;
    q->k_steps = (q->k + stage_k - 1) / stage_k;
    q->k_blocks = (q->k + MLG_F8_BLOCK - 1) / MLG_F8_BLOCK;
    q->joined = q->k % (stage_k / 2) == 0;
    q->unit_tokens = unit_tokens;
    q->w_bytes = kMoeWBytes + (g_moe_lose ? 16 : 0);
  }
  const uint32_t up_smem = plan_moe(up, f8, false), down_smem = plan_moe(down, f8, true);
  const int64_t experts = slots < n_experts ? slots : n_experts;
  const int64_t hits = experts + (n_tokens <= unit_tokens ? 0 : slots / unit_tokens);  // at most

  CUtensorMap up_w, down_w;
  if (!map_weights(&up_w, w_gate_up, f8, up.joined, up.k, up.n, n_experts, kMoeRows / 2) ||
      !map_weights(&down_w, w_down, f8, down.joined, down.k, down.n, n_experts, kMoeRows))
    return MLG_ERR_CUDA;

  const mlg_status st = mlg_route_topk(logits, logits_type, ld_logits, indices, weights, n_tokens,
                                       n_experts, top_k, renormalize, stream);
  if (st != MLG_OK) return st;
  int64_t grid = hits * up.slices;
  if (grid > 2 * sm_count()) grid = 2 * sm_count();
  MoeKernel k = f8 ? moe_kernel_of<true, false>(unit_tokens) : moe_kernel_of<false, false>(unit_tokens);
  err = launch_early(k, grid, kMoeThreads, up_smem, 1, stream, up_w, up);
  if (err != cudaSuccess) return cuda_status(err);
  const int cluster = ranks_of(down, hits, grid);
  k = f8 ? moe_kernel_of<true, true>(unit_tokens) : moe_kernel_of<false, true>(unit_tokens);
  return cuda_status(launch_early(k, int64_t{down.slices} * cluster, kMoeThreads, down_smem,
                                  cluster, stream, down_w, down));
}

}  // namespace

void moe_set_lose(int on) { g_moe_lose = on; }

uint32_t moe_read_errors(bool clear) {
  uint32_t v = 0;
  cudaMemcpyFromSymbol(&v, g_moe_errors, sizeof v);
  if (clear) {
    const uint32_t z = 0;
    cudaMemcpyToSymbol(g_moe_errors, &z, sizeof z);
  }
  return v;
}

}  // namespace mlg

extern "C" {

mlg_status mlg_moe_layer(const void *logits, int32_t logits_type, int64_t ld_logits,
                         const mlg_bf16 *x, const mlg_bf16 *w_gate_up, const mlg_bf16 *w_down,
                         int32_t *indices, float *weights, mlg_bf16 *act, mlg_bf16 *out,
                         int32_t n_tokens, int32_t hidden, int32_t inter, int32_t n_experts,
                         int32_t top_k, int32_t renormalize, void *stream) {
  return mlg::moe_layer(logits, logits_type, ld_logits, x, w_gate_up, nullptr, w_down, nullptr,
                        false, indices, weights, act, out, n_tokens, hidden, inter, n_experts,
                        top_k, renormalize, static_cast<cudaStream_t>(stream));
}

mlg_status mlg_moe_layer_f8(const void *logits, int32_t logits_type, int64_t ld_logits,
                            const mlg_bf16 *x, const mlg_f8 *w_gate_up,
                            const float *gate_up_scales, const mlg_f8 *w_down,
                            const float *down_scales, int32_t *indices, float *weights,
                            mlg_bf16 *act, mlg_bf16 *out, int32_t n_tokens, int32_t hidden,
                            int32_t inter, int32_t n_experts, int32_t top_k, int32_t renormalize,
                            void *stream) {
  return mlg::moe_layer(logits, logits_type, ld_logits, x, w_gate_up, gate_up_scales, w_down,
                        down_scales, true, indices, weights, act, out, n_tokens, hidden, inter,
                        n_experts, top_k, renormalize, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
