// mlg_norm.cu -- the norms around a block with its gate, residual sum and
// scales, and their gradients.
//
// HBM bounds both: every row is read once, by whole warps of threads that hold 16
// bytes of each of the row's arrays (more beyond 1024 such pieces).  A thread copies
// its pieces of the rows to come into shared memory places of its own (cp.async, a
// few rows ahead: no barrier, no registers) and reads them from there as often as
// it needs them.  The norm of out needs out whole, so a row takes two sums one
// after the other: over a warp by shuffles, over a row's warps through shared memory
// with one barrier (the slots alternate, so that the next sum's barrier is the one
// that frees them).  A CTA walks over rows and keeps the weights in registers; in
// the gradient it keeps the weights' gradients of its rows there too and leaves them
// as one partial row, which a second, small kernel sums over the CTAs in their
// order: no atomics, the same bits every time.
// Measured, 16384 rows of 2048 bf16: forward with a gate a channel and both norms 59 us (5.7
// TB/s), the gradient with all its outputs 89 us (6.0 TB/s), 3 of them the second kernel's;
// with loads to registers in place of the rows ahead 71 and 152.  64 rows take 2.6 us.  In
// fp32 116 us (5.8 TB/s) and 169 (6.4).  The widest rows leave room for one of them ahead or
// none, and the gradient's registers spill (2048 x 16384 bf16: 86 us, 3.9 TB/s, and 163, 3.3).
#include <cmath>
#include <mutex>

#include "mlg_launch.cuh"

namespace mlg {
namespace {

constexpr int kNormThreads = 512;      // of a CTA, about; two of them a multiprocessor
// The gradient's, one a multiprocessor: with 8 values a thread 80 registers, with more 128.
constexpr int kNormGradThreads = 768;
constexpr int norm_grad_threads(int values) { return values <= 8 ? kNormGradThreads : 512; }
constexpr int kNormMaxWarps = 32;
// A group of two warps and more has a named barrier of its own, 1 to 15.
static_assert(kNormThreads / 64 <= 15 && kNormGradThreads / 64 <= 15, "named barriers");
constexpr uint32_t kNormRing = 200 * 1024;  // a multiprocessor's shared memory for rows to come
constexpr int kNormMaxAhead = 4;

struct NormParams {
  const void *x, *y, *gate, *w_post, *w_pre;
  void *out, *z;
  int64_t ld_x, ld_y, ld_gate, ld_out, ld_z;
  const void *dout, *dz;
  void *dx, *dy, *dgate;
  int64_t ld_dout, ld_dz, ld_dx, ld_dy, ld_dgate;
  float *partial;
  int32_t n_rows, width, gate_width, tpr;  // tpr: threads a row
  int32_t ahead;                           // rows whose copies are under way
  float residual_scale, branch_scale, eps;
};

// 16 bytes of a row as pairs of fp32 values: two of them an instruction.
template <typename T>
struct Pairs {
  static constexpr int kN = Piece<T>::kN / 2;
  float2 v[kN];
  Pairs() = default;
  __device__ __forceinline__ explicit Pairs(const uint4 &raw) {
    float f[2 * kN];
    Piece<T>::load(raw, f);
#pragma unroll
    for (int k = 0; k < kN; ++k) v[k] = make_float2(f[2 * k], f[2 * k + 1]);
  }
  __device__ __forceinline__ uint4 rounded() const {
    float f[2 * kN];
#pragma unroll
    for (int k = 0; k < kN; ++k) f[2 * k] = v[k].x, f[2 * k + 1] = v[k].y;
    return Piece<T>::store(f);
  }
};
__device__ __forceinline__ float2 operator*(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// Sums of up to four values over a row's threads, in a fixed order.
struct RowSum {
  float4 (*slots)[kNormMaxWarps];  // [2][warps of a CTA]
  int tpr, group, parity;
  __device__ __forceinline__ float4 operator()(float4 v) {
    // Over a warp, four sums at once: two steps halve the values that a lane has to
    // do with, then lane l holds value l & 3 of its eighth.
    const int lane = threadIdx.x & 31;
    const bool odd = lane & 1, high = lane & 2;
    float a = (odd ? v.y : v.x) + __shfl_xor_sync(kFullWarp, odd ? v.x : v.y, 1);
    float b = (odd ? v.w : v.z) + __shfl_xor_sync(kFullWarp, odd ? v.z : v.w, 1);
    a = (high ? b : a) + __shfl_xor_sync(kFullWarp, high ? a : b, 2);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) a += __shfl_xor_sync(kFullWarp, a, o);
    float4 *s = slots[parity] + group * (tpr >> 5);
    parity ^= 1;
    if (lane < 4) reinterpret_cast<float *>(s + (threadIdx.x >> 5) - group * (tpr >> 5))[lane] = a;
    if (tpr == 32)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(tpr) : "memory");
    const int warps = tpr >> 5;
    v = s[0];
#pragma unroll 4
    for (int w = 1; w < warps; ++w) {
      const float4 o = s[w];
      v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
    }
    return v;
  }
  // One value, in the same order (the same bits beside others or alone).
  __device__ __forceinline__ float one(float v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) v += __shfl_xor_sync(kFullWarp, v, o);
    if (tpr == 32) return v;
    float4 *s = slots[parity] + group * (tpr >> 5);
    parity ^= 1;
    const int warps = tpr >> 5;
    if ((threadIdx.x & 31) == 0) s[(threadIdx.x >> 5) - group * warps].x = v;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(tpr) : "memory");
    v = s[0].x;
#pragma unroll 4
    for (int w = 1; w < warps; ++w) v += s[w].x;
    return v;
  }
};

// The pieces of the rows to come: [row][array][piece][thread], 16 bytes each.
template <int ARRAYS, int P>
struct Ahead {
  uint4 *ring;
  int rows, slot;
  __device__ __forceinline__ uint4 *place(int k, int array, int piece) const {
    return ring + ((k * ARRAYS + array) * P + piece) * blockDim.x + threadIdx.x;
  }
  __device__ __forceinline__ int before() const { return slot > 0 ? slot - 1 : rows - 1; }
  __device__ __forceinline__ void next() { slot = slot + 1 < rows ? slot + 1 : 0; }
  __device__ __forceinline__ uint4 get(int array, int piece) const {
    return *place(slot, array, piece);
  }
  // Waits for the oldest of `rows` groups.
  __device__ __forceinline__ void wait() const {
    switch (rows) {
      case 1: cp_async_wait_group<0>(); break;
      case 2: cp_async_wait_group<1>(); break;
      case 3: cp_async_wait_group<2>(); break;
      default: cp_async_wait_group<3>(); break;
    }
  }
};

template <typename T>
__device__ __forceinline__ uint4 load_piece(const void *p, int64_t ld, int64_t r, int col) {
  return *reinterpret_cast<const uint4 *>(static_cast<const T *>(p) + r * ld + col);
}
template <typename T>
__device__ __forceinline__ void store_piece(void *p, int64_t ld, int64_t r, int col, uint4 v) {
  *reinterpret_cast<uint4 *>(static_cast<T *>(p) + r * ld + col) = v;
}

// A row's weight, kept in registers where a thread has 8 values of it.
template <typename T, int P>
struct Weight {
  static constexpr bool kKept = 2 * Pairs<T>::kN * P <= 8;
  const void *from;
  uint4 kept[P];
  __device__ __forceinline__ Weight(const void *w, const int (&col)[P], const bool (&in)[P])
      : from(w) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      kept[i] = make_uint4(0, 0, 0, 0);
      if (kKept && w && in[i]) kept[i] = load_piece<T>(w, 0, 0, col[i]);
    }
  }
  __device__ __forceinline__ Pairs<T> get(int i, int col) const {
    return Pairs<T>(kKept ? kept[i] : __ldg(reinterpret_cast<const uint4 *>(
                                          static_cast<const T *>(from) + col)));
  }
};

// P: 16-byte pieces of a row that a thread holds.  ALL: both norms are there.
template <typename T, int P, bool ALL>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const NormParams p) {
  using V = Pairs<T>;
  extern __shared__ uint4 ring[];
  __shared__ float4 slots[2][kNormMaxWarps];
  griddep_wait();
  griddep_launch_dependents();
  const int tpr = p.tpr, group = threadIdx.x / tpr, lane = threadIdx.x - group * tpr;
  const int groups = blockDim.x / tpr;
  const bool y = ALL || p.y, w_post = ALL || p.w_post, w_pre = ALL || p.w_pre;
  const bool full = p.gate && p.gate_width != 1;
  RowSum sum{slots, tpr, group, 0};
  int col[P];
  bool in[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    col[i] = (i * tpr + lane) * 2 * V::kN;
    in[i] = col[i] < p.width;
  }
  const Weight<T, P> post(p.w_post, col, in), pre(p.w_pre, col, in);
  const float inv_width = 1.0f / static_cast<float>(p.width);
  const int64_t first = int64_t{blockIdx.x} * groups + group, step = int64_t{gridDim.x} * groups;
  Ahead<3, P> rows{ring, p.ahead, 0};  // x, y, gate
  auto fetch = [&](int64_t r, int k) {
    if (r < p.n_rows)
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (!in[i]) continue;
        auto copy = [&](int array, const void *from, int64_t ld) {
          cp_async_16(smem_addr(rows.place(k, array, i)),
                      static_cast<const T *>(from) + r * ld + col[i], 16);
        };
        copy(0, p.x, p.ld_x);
        if (y) copy(1, p.y, p.ld_y);
        if (full) copy(2, p.gate, p.ld_gate);
      }
    cp_async_commit();
  };
  for (int k = 0; k < p.ahead - 1; ++k) fetch(first + k * step, k);
  for (int64_t r = first; r < p.n_rows; r += step, rows.next()) {
    fetch(r + (p.ahead - 1) * step, rows.before());
    float scale = p.branch_scale;  // of the branch, where the gate is not one a channel
    if (p.gate && !full) scale *= to_f32(static_cast<const T *>(p.gate)[r * p.ld_gate]);
    rows.wait();
    float rstd = 1.0f;
    if (w_post) {
      float2 s = both(0.0f);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (!in[i]) continue;
        const V v(rows.get(1, i));
#pragma unroll
        for (int k = 0; k < V::kN; ++k) s = fma2(v.v[k], v.v[k], s);
      }
      rstd = rsqrtf(sum.one(s.x + s.y) * inv_width + p.eps);
    }
    float2 s = both(0.0f);
    uint4 stored[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (!in[i]) continue;
      V u(rows.get(0, i));
#pragma unroll
      for (int k = 0; k < V::kN; ++k) u.v[k] = u.v[k] * both(p.residual_scale);
      if (y) {
        V v(rows.get(1, i));
        if (w_post) {
          const V w = post.get(i, col[i]);
#pragma unroll
          for (int k = 0; k < V::kN; ++k) v.v[k] = v.v[k] * both(rstd) * w.v[k];
        }
        if (full) {
          const V c(rows.get(2, i));
#pragma unroll
          for (int k = 0; k < V::kN; ++k) v.v[k] = v.v[k] * c.v[k];
        }
#pragma unroll
        for (int k = 0; k < V::kN; ++k) u.v[k] = fma2(both(scale), v.v[k], u.v[k]);
      }
      stored[i] = u.rounded();
      if (p.out) store_piece<T>(p.out, p.ld_out, r, col[i], stored[i]);
      u = V(stored[i]);  // out as it is stored
#pragma unroll
      for (int k = 0; k < V::kN; ++k) s = fma2(u.v[k], u.v[k], s);
    }
    if (!w_pre) continue;
    const float rstd_out = rsqrtf(sum.one(s.x + s.y) * inv_width + p.eps);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (!in[i]) continue;
      V u(stored[i]);
      const V w = pre.get(i, col[i]);
#pragma unroll
      for (int k = 0; k < V::kN; ++k) u.v[k] = u.v[k] * both(rstd_out) * w.v[k];
      store_piece<T>(p.z, p.ld_z, r, col[i], u.rounded());
    }
  }
  cp_async_wait_group<0>();
}

// ALL: everything that can be left out is there (but the gate, of whichever width).
template <typename T, int P, bool ALL>
__global__ void __launch_bounds__(norm_grad_threads(2 * Pairs<T>::kN * P), 1)
    norm_grad_kernel(const NormParams p) {
  using V = Pairs<T>;
  constexpr int N = 2 * V::kN;
  extern __shared__ uint4 ring[];
  __shared__ float4 slots[2][kNormMaxWarps];
  griddep_wait();
  griddep_launch_dependents();
  const int tpr = p.tpr, group = threadIdx.x / tpr, lane = threadIdx.x - group * tpr;
  const int groups = blockDim.x / tpr;
  const bool y = ALL || p.y, w_post = ALL || p.w_post, w_pre = ALL || p.w_pre;
  const bool dout = ALL || p.dout, dx = ALL || p.dx, dy = ALL || p.dy;
  const bool full = p.gate && p.gate_width != 1, sum_gate = p.dgate && !full;
  RowSum sum{slots, tpr, group, 0};
  V dpost[P], dpre[P];
  int col[P];
  bool in[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    col[i] = (i * tpr + lane) * N;
    in[i] = col[i] < p.width;
#pragma unroll
    for (int k = 0; k < V::kN; ++k) dpost[i].v[k] = dpre[i].v[k] = both(0.0f);
  }
  const Weight<T, P> post(p.w_post, col, in), pre(p.w_pre, col, in);
  const float inv_width = 1.0f / static_cast<float>(p.width);
  const int64_t first = int64_t{blockIdx.x} * groups + group, step = int64_t{gridDim.x} * groups;
  enum { kDout, kDz, kOut, kY, kGate, kArrays };
  Ahead<kArrays, P> rows{ring, p.ahead, 0};
  auto fetch = [&](int64_t r, int k) {
    if (r < p.n_rows)
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (!in[i]) continue;
        auto copy = [&](int array, const void *from, int64_t ld) {
          cp_async_16(smem_addr(rows.place(k, array, i)),
                      static_cast<const T *>(from) + r * ld + col[i], 16);
        };
        if (dout) copy(kDout, p.dout, p.ld_dout);
        if (w_pre) copy(kDz, p.dz, p.ld_dz), copy(kOut, p.out, p.ld_out);
        if (y) copy(kY, p.y, p.ld_y);
        if (full) copy(kGate, p.gate, p.ld_gate);
      }
    cp_async_commit();
  };
  for (int k = 0; k < p.ahead - 1; ++k) fetch(first + k * step, k);
  for (int64_t r = first; r < p.n_rows; r += step, rows.next()) {
    fetch(r + (p.ahead - 1) * step, rows.before());
    float scale = p.branch_scale;
    if (p.gate && !full) scale *= to_f32(static_cast<const T *>(p.gate)[r * p.ld_gate]);
    rows.wait();
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);  // out^2, dz w_pre out, y^2
    if (w_pre || w_post) {
      float2 s0 = both(0.0f), s1 = s0, s2 = s0;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (!in[i]) continue;
        if (w_pre) {
          const V a(rows.get(kOut, i)), b(rows.get(kDz, i)), w = pre.get(i, col[i]);
#pragma unroll
          for (int k = 0; k < V::kN; ++k) {
            s0 = fma2(a.v[k], a.v[k], s0);
            s1 = fma2(a.v[k], b.v[k] * w.v[k], s1);
          }
        }
        if (w_post) {
          const V v(rows.get(kY, i));
#pragma unroll
          for (int k = 0; k < V::kN; ++k) s2 = fma2(v.v[k], v.v[k], s2);
        }
      }
      s = sum(make_float4(s0.x + s0.y, s1.x + s1.y, s2.x + s2.y, 0.0f));
    }
    const float ru = rsqrtf(s.x * inv_width + p.eps);
    // of out / rms(out), which is of the size of 1 whatever out's: 1 / rms^3, of out itself, leaves
    // fp32's range from an rms of 1e14 on, and with eps 0 below 1e-13
    const float cu = -(ru * inv_width * (ru * s.y));
    const float ry = w_post ? rsqrtf(s.z * inv_width + p.eps) : 1.0f;
    V d[P];
    float2 t0 = both(0.0f), t1 = t0;  // dn w_post y, and d n for a gate a row
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (!in[i]) continue;
      if (dout) {
        d[i] = V(rows.get(kDout, i));
      } else {
#pragma unroll
        for (int k = 0; k < V::kN; ++k) d[i].v[k] = both(0.0f);
      }
      if (w_pre) {
        const V a(rows.get(kOut, i)), b(rows.get(kDz, i)), w = pre.get(i, col[i]);
#pragma unroll
        for (int k = 0; k < V::kN; ++k) {
          const float2 unit = a.v[k] * both(ru);
          d[i].v[k] = fma2(both(ru), b.v[k] * w.v[k], fma2(both(cu), unit, d[i].v[k]));
          dpre[i].v[k] = fma2(b.v[k], unit, dpre[i].v[k]);
        }
      }
      if (dx) {
        V v;
#pragma unroll
        for (int k = 0; k < V::kN; ++k) v.v[k] = d[i].v[k] * both(p.residual_scale);
        store_piece<T>(p.dx, p.ld_dx, r, col[i], v.rounded());
      }
      if (!y) continue;
      V n(rows.get(kY, i)), w;  // y / rms(y)
      if (w_post) {
        w = post.get(i, col[i]);
#pragma unroll
        for (int k = 0; k < V::kN; ++k) n.v[k] = n.v[k] * both(ry);
      }
      if (full) {
#pragma unroll
        for (int k = 0; k < V::kN; ++k) d[i].v[k] = d[i].v[k] * both(p.branch_scale);
        if (ALL || p.dgate) {
          V dg;
#pragma unroll
          for (int k = 0; k < V::kN; ++k)
            dg.v[k] = d[i].v[k] * (w_post ? n.v[k] * w.v[k] : n.v[k]);
          store_piece<T>(p.dgate, p.ld_dgate, r, col[i], dg.rounded());
        }
        const V c(rows.get(kGate, i));
#pragma unroll
        for (int k = 0; k < V::kN; ++k) d[i].v[k] = d[i].v[k] * c.v[k];
      } else {
        if (sum_gate)
#pragma unroll
          for (int k = 0; k < V::kN; ++k)
            t1 = fma2(d[i].v[k], w_post ? n.v[k] * w.v[k] : n.v[k], t1);
#pragma unroll
        for (int k = 0; k < V::kN; ++k) d[i].v[k] = d[i].v[k] * both(scale);
      }
      if (w_post)
#pragma unroll
        for (int k = 0; k < V::kN; ++k) {
          dpost[i].v[k] = fma2(d[i].v[k], n.v[k], dpost[i].v[k]);
          d[i].v[k] = d[i].v[k] * w.v[k];
          t0 = fma2(d[i].v[k], n.v[k], t0);
        }
    }
    if (!y) continue;
    float t = 0.0f;
    if (sum_gate) {
      s = sum(make_float4(t0.x + t0.y, t1.x + t1.y, 0.0f, 0.0f));
      t = s.x;
      if (lane == 0)
        put(static_cast<T *>(p.dgate) + r * p.ld_dgate, p.branch_scale * s.y);
    } else if (w_post) {
      t = sum.one(t0.x + t0.y);
    }
    if (!dy) continue;
    const float cy = -(t * inv_width);  // of y / rms(y), like t
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (!in[i]) continue;
      if (w_post) {
        const V v(rows.get(kY, i));
#pragma unroll
        for (int k = 0; k < V::kN; ++k)
          d[i].v[k] = both(ry) * fma2(both(cy), v.v[k] * both(ry), d[i].v[k]);
      }
      store_piece<T>(p.dy, p.ld_dy, r, col[i], d[i].rounded());
    }
  }
  cp_async_wait_group<0>();
  if (!p.partial) return;
  // This CTA's sums: [post, pre][width].  With more than one group they meet in shared
  // memory, where the rows were, in the groups' order.
  float *row = p.partial + int64_t{blockIdx.x} * 2 * p.width;
  if (groups > 1) {
    float *shared = reinterpret_cast<float *>(ring);
    const int span = P * tpr * N;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int k = 0; k < V::kN; ++k) {
        float *to = shared + group * 2 * span + col[i] + 2 * k;
        *reinterpret_cast<float2 *>(to) = dpost[i].v[k];
        *reinterpret_cast<float2 *>(to + span) = dpre[i].v[k];
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.width; i += blockDim.x) {
      const int which = i >= p.width, c = i - which * p.width;
      float v = 0.0f;
      for (int q = 0; q < groups; ++q) v += shared[(q * 2 + which) * span + c];
      row[i] = v;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if (!in[i]) continue;
#pragma unroll
    for (int k = 0; k < V::kN; k += 2) {
      *reinterpret_cast<float4 *>(row + col[i] + 2 * k) = make_float4(
          dpost[i].v[k].x, dpost[i].v[k].y, dpost[i].v[k + 1].x, dpost[i].v[k + 1].y);
      *reinterpret_cast<float4 *>(row + p.width + col[i] + 2 * k) = make_float4(
          dpre[i].v[k].x, dpre[i].v[k].y, dpre[i].v[k + 1].x, dpre[i].v[k + 1].y);
    }
  }
}

// dw[c] = sum over the CTAs' partial rows: 32 columns a CTA, 16 warps that share
// the rows and add up in order.
constexpr int kWeightWarps = 16;
__global__ void __launch_bounds__(kWeightWarps * 32)
    norm_weights_kernel(const float *partial, int n_partial, int width, float *dw_post,
                        float *dw_pre) {
  __shared__ float part[kWeightWarps][32];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane;  // of [post, pre][width]
  float v = 0.0f;
  if (i < 2 * width)
#pragma unroll 8
    for (int r = warp; r < n_partial; r += kWeightWarps) v += partial[int64_t{r} * 2 * width + i];
  part[warp][lane] = v;
  __syncthreads();
  if (warp != 0 || i >= 2 * width) return;
  for (int w = 1; w < kWeightWarps; ++w) v += part[w][lane];
  float *to = i < width ? dw_post : dw_pre;
  if (to) to[i < width ? i : i - width] = v;
}

// How a kernel is laid out: threads a row (whole warps, one piece a thread as far as
// they go), pieces a thread, rows a CTA, CTAs, rows ahead.
struct Shape {
  int tpr, pieces, groups, grid, ahead;
  size_t smem;
};
// A thread has 8 values of a row, in CTAs of up to `threads` threads; more where that does
// not hold a row, in CTAs of up to 512.  `arrays` are copied ahead; at most `most` CTAs,
// `per_sm` a multiprocessor.
Shape shape_of(int32_t width, size_t size, int32_t n_rows, int arrays, int threads, int per_sm,
               int most) {
  const int whole = static_cast<int>(width * size / 16);
  Shape s = {};
  s.pieces = static_cast<int>(size / 2);
  if (s.pieces * threads < whole) {
    threads = 512;
    while (s.pieces * threads < whole) s.pieces *= 2;
  }
  s.tpr = ((whole + s.pieces - 1) / s.pieces + 31) / 32 * 32;
  s.groups = threads / s.tpr;
  // few rows: spread over the multiprocessors
  const int64_t spread = (int64_t{n_rows} + sm_count() - 1) / sm_count();
  if (s.groups > spread) s.groups = static_cast<int>(spread);
  const int64_t ctas = (int64_t{n_rows} + s.groups - 1) / s.groups;
  s.grid = static_cast<int>(ctas < most ? ctas : most);
  const size_t row = size_t{16} * arrays * s.pieces * s.tpr * s.groups;
  s.ahead = static_cast<int>(kNormRing / per_sm / row);
  if (s.ahead > kNormMaxAhead) s.ahead = kNormMaxAhead;
  if (s.ahead < 1) s.ahead = 1;
  s.smem = row * s.ahead;
  return s;
}

// Rows of `type`: 16-byte aligned, whole pieces.
bool rows_fit(const void *p, int64_t ld, int32_t type) {
  return p == nullptr || (aligned16(p) && ld % (16 / static_cast<int64_t>(type_size(type))) == 0);
}

mlg_status check_norm(int32_t type, int32_t n_rows, int32_t width, const void *gate,
                      int32_t gate_width, float eps) {
  if (n_rows < 0 || width < 1 || !known_type(type) || !(eps >= 0.0f)) return MLG_ERR_INVALID_ARG;
  if (gate && gate_width != 1 && gate_width != width) return MLG_ERR_INVALID_ARG;
  const int64_t bytes = int64_t{width} * static_cast<int64_t>(type_size(type));
  if (bytes > MLG_NORM_MAX_BYTES || bytes % 16 != 0) return MLG_ERR_UNSUPPORTED;
  return MLG_OK;
}

// A gate of one number a row needs its element's alignment alone.
bool gate_fits(const void *p, int64_t ld, int32_t gate_width, int32_t type) {
  if (gate_width != 1) return rows_fit(p, ld, type);
  return (reinterpret_cast<uintptr_t>(p) & (type_size(type) - 1)) == 0;
}

using NormKernel = void (*)(NormParams);

template <bool ALL>
NormKernel norm_of(int32_t type, int pieces) {
  if (type == MLG_TYPE_BF16)
    return pieces == 1   ? norm_kernel<__nv_bfloat16, 1, ALL>
           : pieces == 2 ? norm_kernel<__nv_bfloat16, 2, ALL>
                         : norm_kernel<__nv_bfloat16, 4, ALL>;
  return pieces == 2 ? norm_kernel<float, 2, ALL> : norm_kernel<float, 4, ALL>;
}
template <bool ALL>
NormKernel norm_grad_of(int32_t type, int pieces) {
  if (type == MLG_TYPE_BF16)
    return pieces == 1   ? norm_grad_kernel<__nv_bfloat16, 1, ALL>
           : pieces == 2 ? norm_grad_kernel<__nv_bfloat16, 2, ALL>
                         : norm_grad_kernel<__nv_bfloat16, 4, ALL>;
  return pieces == 2 ? norm_grad_kernel<float, 2, ALL> : norm_grad_kernel<float, 4, ALL>;
}

cudaError_t allow_norm_smem() {
  static std::once_flag once[64];
  static cudaError_t err[64];
  int dev = 0;
  cudaGetDevice(&dev);
  std::call_once(once[dev & 63], [d = dev & 63] {
    cudaError_t e = cudaSuccess;
    for (int32_t type : {MLG_TYPE_BF16, MLG_TYPE_F32})
      for (int pieces : {1, 2, 4})
        for (NormKernel k : {norm_of<true>(type, pieces), norm_of<false>(type, pieces),
                             norm_grad_of<true>(type, pieces), norm_grad_of<false>(type, pieces)})
          if (e == cudaSuccess) e = allow_smem(k, kNormRing);
    err[d] = e;
  });
  return err[dev & 63];
}

}  // namespace
}  // namespace mlg

extern "C" {

mlg_status mlg_block_norm(const void *x, int32_t type, int64_t ld_x, const void *y, int64_t ld_y,
                          const void *gate, int64_t ld_gate, const void *w_post,
                          const void *w_pre, void *out, int64_t ld_out, void *z, int64_t ld_z,
                          int32_t n_rows, int32_t width, int32_t gate_width, float residual_scale,
                          float branch_scale, float eps, void *stream) {
  using namespace mlg;
  if (!y) gate = w_post = nullptr;
  const mlg_status st = check_norm(type, n_rows, width, gate, gate_width, eps);
  if (st != MLG_OK) return st;
  if (n_rows == 0) return MLG_OK;
  if (!x || (!out && !w_pre) || (!z != !w_pre)) return MLG_ERR_INVALID_ARG;
  if (ld_x < width || (y && ld_y < width) || (gate && ld_gate < gate_width) ||
      (out && ld_out < width) || (z && ld_z < width))
    return MLG_ERR_INVALID_ARG;
  if (!rows_fit(x, ld_x, type) || !rows_fit(y, ld_y, type) || !rows_fit(out, ld_out, type) ||
      !rows_fit(z, ld_z, type) || !rows_fit(w_post, 0, type) || !rows_fit(w_pre, 0, type) ||
      !gate_fits(gate, ld_gate, gate_width, type))
    return MLG_ERR_UNSUPPORTED;
  cudaError_t err = allow_norm_smem();
  if (err != cudaSuccess) return cuda_status(err);
  const Shape shape = shape_of(width, type_size(type), n_rows, 3, kNormThreads, 2, 2 * sm_count());
  NormParams p = {};
  p.x = x, p.ld_x = ld_x, p.y = y, p.ld_y = ld_y, p.gate = gate, p.ld_gate = ld_gate;
  p.w_post = w_post, p.w_pre = w_pre;
  p.out = out, p.ld_out = ld_out, p.z = z, p.ld_z = ld_z;
  p.n_rows = n_rows, p.width = width, p.gate_width = gate_width;
  p.tpr = shape.tpr, p.ahead = shape.ahead;
  p.residual_scale = residual_scale, p.branch_scale = branch_scale, p.eps = eps;
  const bool all = y && w_post && w_pre;
  return cuda_status(launch_early(all ? norm_of<true>(type, shape.pieces)
                                      : norm_of<false>(type, shape.pieces), shape.grid,
                                  shape.tpr * shape.groups, shape.smem, 1,
                                  static_cast<cudaStream_t>(stream), p));
}

mlg_status mlg_block_norm_backward(
    const void *dout, int32_t type, int64_t ld_dout, const void *dz, int64_t ld_dz,
    const void *out, int64_t ld_out, const void *y, int64_t ld_y, const void *gate,
    int64_t ld_gate, const void *w_post, const void *w_pre, void *dx, int64_t ld_dx, void *dy,
    int64_t ld_dy, void *dgate, int64_t ld_dgate, float *dw_post, float *dw_pre, float *partial,
    int32_t n_rows, int32_t width, int32_t gate_width, float residual_scale, float branch_scale,
    float eps, void *stream) {
  using namespace mlg;
  if (n_rows != 0) {  // (an empty batch's rows have no addresses)
    if (!y && (dy || dgate || dw_post)) return MLG_ERR_INVALID_ARG;
    if (!y) gate = w_post = nullptr;
    if ((dgate && !gate) || (dw_post && !w_post) || (dw_pre && !w_pre)) return MLG_ERR_INVALID_ARG;
  }
  const mlg_status st = check_norm(type, n_rows, width, gate, gate_width, eps);
  if (st != MLG_OK) return st;
  const bool weights = dw_post || dw_pre;
  if (weights && !partial) return MLG_ERR_INVALID_ARG;
  if (weights && (!aligned16(partial) || !aligned4(dw_post) || !aligned4(dw_pre)))
    return MLG_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int64_t grid = 0;
  if (n_rows > 0) {
    if ((w_pre && (!dz || !out)) || (!dx && !dy && !dgate && !weights)) return MLG_ERR_INVALID_ARG;
    if (!w_pre) dz = out = nullptr;
    if ((dout && ld_dout < width) || (dz && ld_dz < width) || (out && ld_out < width) ||
        (y && ld_y < width) || (gate && ld_gate < gate_width) || (dx && ld_dx < width) ||
        (dy && ld_dy < width) || (dgate && ld_dgate < gate_width))
      return MLG_ERR_INVALID_ARG;
    if (!rows_fit(dout, ld_dout, type) || !rows_fit(dz, ld_dz, type) ||
        !rows_fit(out, ld_out, type) || !rows_fit(y, ld_y, type) ||
        !rows_fit(w_post, 0, type) || !rows_fit(w_pre, 0, type) || !rows_fit(dx, ld_dx, type) ||
        !rows_fit(dy, ld_dy, type) || !gate_fits(gate, ld_gate, gate_width, type) ||
        !gate_fits(dgate, ld_dgate, gate_width, type))
      return MLG_ERR_UNSUPPORTED;
    cudaError_t err = allow_norm_smem();
    if (err != cudaSuccess) return cuda_status(err);
    const int most = sm_count() < MLG_NORM_PARTIALS ? sm_count() : MLG_NORM_PARTIALS;
    Shape shape = shape_of(width, type_size(type), n_rows, 5, kNormGradThreads, 1, most);
    const size_t sums =
        size_t{2} * shape.tpr * shape.groups * shape.pieces * (16 / type_size(type)) * 4;
    if (shape.groups > 1 && shape.smem < sums) shape.smem = sums;
    grid = shape.grid;
    NormParams p = {};
    p.dout = dout, p.ld_dout = ld_dout, p.dz = dz, p.ld_dz = ld_dz;
    p.out = const_cast<void *>(out), p.ld_out = ld_out;
    p.y = y, p.ld_y = ld_y, p.gate = gate, p.ld_gate = ld_gate;
    p.w_post = w_post, p.w_pre = w_pre;
    p.dx = dx, p.ld_dx = ld_dx, p.dy = dy, p.ld_dy = ld_dy, p.dgate = dgate, p.ld_dgate = ld_dgate;
    p.partial = weights ? partial : nullptr;
    p.n_rows = n_rows, p.width = width, p.gate_width = gate_width;
    p.tpr = shape.tpr, p.ahead = shape.ahead;
    p.residual_scale = residual_scale, p.branch_scale = branch_scale, p.eps = eps;
    const bool all = dout && y && w_post && w_pre && dx && dy && (dgate || gate_width == 1 || !gate);
    err = launch_early(all ? norm_grad_of<true>(type, shape.pieces)
                           : norm_grad_of<false>(type, shape.pieces), grid, shape.tpr * shape.groups, shape.smem,
                       1, s, p);
    if (err != cudaSuccess || !weights) return cuda_status(err);
  }
  if (!weights) return MLG_OK;
  return cuda_status(launch_early(norm_weights_kernel, (2 * int64_t{width} + 31) / 32,
                                  kWeightWarps * 32, 0, 1, s,
                                  static_cast<const float *>(partial), static_cast<int>(grid),
                                  static_cast<int>(width), dw_post, dw_pre));
}

}  // extern "C"
