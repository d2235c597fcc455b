// mlg_rows8.cu -- rows to e4m3 with an fp32 scale for each 128 values, and the
// gated activation between an expert's two projections with the same output.
//
// HBM bounds both: a token's row is read once, quantised once and written to
// the rows of all its slots (top_k 8: 9 bytes out for every 2 in), so that there
// is no bf16 copy in expert order.  A group of lanes holds a block (8 lanes of
// 16 bf16 values, 16 of 8 fp32), so its largest value is three or four shuffles.
// The groups take the blocks of all rows one after the other, whatever a row's width,
// and ask for their next block before they compute.
// Measured: 4096 tokens of 2048 bf16 values to 8 rows each 15.1 us (5.7 TB/s), a warp a row
// 16.6; the activation of 32768 rows of 768 26.6 us (4.8 TB/s), of 8191 of 784 with its bf16
// copy 10.6 (4.3 TB/s).
#include <cuda_fp8.h>

#include "mlg_launch.cuh"

namespace mlg {
namespace {

constexpr int kWarps8 = 8;  // of a CTA
// CTAs a multiprocessor: twice what finds a place there (48 and 64 registers a thread).  Rows
// of 4096 tokens of 2048 to 8 places each 15.1 us, with 5 17.0, with 16 15.3; the activation of
// 8191 rows of 784 10.5 us, with 4 11.7, with 16 12.4.
constexpr int kRowsCtas8 = 10, kSwigluCtas8 = 8;
constexpr float kE4m3Max = 448.0f;
constexpr float kLeastScale = 1.17549435e-38f;  // 2^-126

struct Rows8Params {
  const void *x;
  int64_t ld_x, rows;
  const int32_t *pos;
  void *act;
  uint8_t *q;
  float *scales;
  int32_t width, top_k, n_rows, blocks;
};

// The scale of the block that this lane's group holds, v N of its values (0
// where the row has ended).  The quotient is the nearest one, as in quantise().
template <int N>
__device__ __forceinline__ float block_scale(const float (&v)[N]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) m = fmaxf(m, fabsf(v[i]));  // a NaN is passed over
#pragma unroll
  for (int o = MLG_F8_BLOCK / N / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullWarp, m, o));
  constexpr float kOver = 1.0f / kE4m3Max;
  const float q = m * kOver;
  const float s = fmaf(fmaf(-q, kE4m3Max, m), kOver, q);
  return m < INFINITY ? fmaxf(s, kLeastScale) : m;
}

// N codes, four a word.  The quotients are the nearest ones, so that a code depends on
// nothing but its value and its scale: with the nearest reciprocal y of the scale, q = x y
// corrected by its exact remainder, q - (q scale - x) y, is the nearest (Markstein 1990),
// as long as the remainder needs no bits below 2^-149, which scales from 2^-60 on see to
// (what is below 2^-11 of them becomes 0 whatever its quotient's last bit).
template <int N>
__device__ __forceinline__ void quantise(const float (&v)[N], float scale, uint32_t (&w)[N / 4]) {
  float2 q[N / 2];
  if (scale >= 0x1p-60f) {
    const float inverse = __frcp_rn(scale);
    const float2 y = both(inverse), minus_y = both(-inverse), s = both(scale);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float2 x = make_float2(v[2 * i], v[2 * i + 1]);
      q[i] = __fmul2_rn(x, y);
      // (x - q scale in its place would make +0 of -0)
      q[i] = __ffma2_rn(__ffma2_rn(q[i], s, make_float2(-x.x, -x.y)), minus_y, q[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
      q[i] = make_float2(__fdiv_rn(v[2 * i], scale), __fdiv_rn(v[2 * i + 1], scale));
  }
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(q[2 * i], __NV_SATFINITE, __NV_E4M3) |
           __nv_cvt_float2_to_fp8x2(q[2 * i + 1], __NV_SATFINITE, __NV_E4M3) << 16;
}

template <int N>
__device__ __forceinline__ void store_codes(uint8_t *p, const uint32_t (&w)[N / 4]) {
  if constexpr (N == 16)
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else
    *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
}

// 32 bytes of a row.
struct Raw8 {
  uint4 v[2];
  template <typename T>
  __device__ __forceinline__ void values(float (&f)[2 * Piece<T>::kN]) const {
    constexpr int N = Piece<T>::kN;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float some[N];
      Piece<T>::load(v[h], some);
#pragma unroll
      for (int i = 0; i < N; ++i) f[h * N + i] = some[i];
    }
  }
};

// A group's walk over the blocks of all rows: its block now, and the step to the next.
template <int N>
struct Walk {
  static constexpr int kLanes = MLG_F8_BLOCK / N, kGroups = kWarps8 * 32 / kLanes;
  int64_t row, row_step;
  int block, block_step, blocks, width;
  __device__ __forceinline__ explicit Walk(const Rows8Params &p)
      : blocks(p.blocks), width(p.width) {
    // (the grid is a few CTAs a multiprocessor: 32 bits)
    const uint32_t unit = blockIdx.x * kGroups + threadIdx.x / kLanes, n = p.blocks;
    const uint32_t step = gridDim.x * kGroups;
    row = unit / n;
    block = static_cast<int>(unit % n);
    row_step = step / n;
    block_step = static_cast<int>(step % n);
  }
  __device__ __forceinline__ void next() {
    row += row_step;
    block += block_step;
    if (block >= blocks) block -= blocks, ++row;
  }
  __device__ __forceinline__ int col() const {
    return block * MLG_F8_BLOCK + (threadIdx.x & (kLanes - 1)) * N;
  }
  __device__ __forceinline__ bool in(int64_t rows) const { return row < rows && col() < width; }
  // This lane's 32 bytes of the block, from column `from` on.
  template <typename T>
  __device__ __forceinline__ Raw8 load(const Rows8Params &p, int from) const {
    Raw8 raw = {};
    if (in(p.rows)) {
      const uint4 *at = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.x) +
                                                        row * p.ld_x + from + col());
      raw.v[0] = __ldg(at), raw.v[1] = __ldg(at + 1);
    }
    return raw;
  }
};

template <typename T>
__global__ void __launch_bounds__(kWarps8 * 32) rows8_kernel(const Rows8Params p) {
  constexpr int N = 2 * Piece<T>::kN, kLanes = MLG_F8_BLOCK / N;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int in_group = lane & (kLanes - 1);
  Walk<N> at(p);
  Raw8 raw = at.template load<T>(p, 0);
  // A lane's slot of the token, the next unit's asked for a unit ahead like its values.
  auto ask = [&](const Walk<N> &w, int j) {
    int r = -1;
    if (w.row < p.rows && in_group < p.top_k - j) {
      const int64_t slot = w.row * p.top_k + j + in_group;
      r = p.pos ? __ldg(p.pos + slot) : static_cast<int>(slot);
    }
    return r;
  };
  int mine = ask(at, 0);
  // the lanes of a warp stay together: they shuffle
  while (__any_sync(kFullWarp, at.row < p.rows)) {
    Walk<N> next = at;
    next.next();
    const Raw8 next_raw = next.template load<T>(p, 0);
    const int next_mine = ask(next, 0);
    float v[N];
    raw.template values<T>(v);
    const float scale = block_scale(v);
    uint32_t w[N / 4];
    quantise(v, scale, w);
    const bool in = at.in(p.rows);
    for (int64_t base = 0; base < p.top_k; base += kLanes) {
      if (base > 0) mine = ask(at, static_cast<int>(base));
      const int n = min(kLanes, p.top_k - static_cast<int>(base));
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        const int64_t r = __shfl_sync(kFullWarp, mine, j, kLanes);
        if (!in || r < 0 || r >= p.n_rows) continue;
        store_codes<N>(p.q + r * p.width + at.col(), w);
        if (in_group == 0) p.scales[r * p.blocks + at.block] = scale;
      }
    }
    at = next;
    raw = next_raw;
    mine = next_mine;
  }
}

// Two gates' silu: g / (1 + 2^t), t = -g log2(e) as the sum of its fp32 value and what that
// leaves out, r: 2^t = 2^hi (1 + r ln 2).  Beyond +-128 the power is 0 or infinite.  The
// denominator is taken 2^-8 times, exactly: as it is its reciprocal is below 2^-126 from
// g = -87.34 on, and rcp.approx gives 0 there, up to -88.72 too soon.
__device__ __forceinline__ float2 silu2(float2 g) {
  constexpr float kLog2e = 1.44269504f, kLog2eRest = 1.92596299e-8f, kLn2 = 0.693147181f;
  const float2 x = make_float2(fminf(fmaxf(-g.x, -128.0f), 128.0f),
                               fminf(fmaxf(-g.y, -128.0f), 128.0f));
  const float2 t = __fmul2_rn(x, both(kLog2e));
  float2 r = __ffma2_rn(x, both(kLog2e), make_float2(-t.x, -t.y));
  r = __ffma2_rn(x, both(kLog2eRest), r);
  float2 e, i;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  // an infinite power stays one: its correction is at most 1 + 2^-17
  constexpr float kLess = 0x1p-8f;
  e = __fadd2_rn(__fmul2_rn(e, __ffma2_rn(r, both(kLess * kLn2), both(kLess))), both(kLess));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(i.x) : "f"(e.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(i.y) : "f"(e.y));
  return __fmul2_rn(g, __fmul2_rn(i, both(kLess)));
}

template <typename T>
__global__ void __launch_bounds__(kWarps8 * 32) swiglu8_kernel(const Rows8Params p) {
  constexpr int N = 2 * Piece<T>::kN, kLanes = MLG_F8_BLOCK / N;
  griddep_wait();
  griddep_launch_dependents();
  Walk<N> at(p);
  Raw8 gate_raw = at.template load<T>(p, 0), up_raw = at.template load<T>(p, p.width);
  while (__any_sync(kFullWarp, at.row < p.rows)) {
    Walk<N> next = at;
    next.next();
    const Raw8 next_gate = next.template load<T>(p, 0);
    const Raw8 next_up = next.template load<T>(p, p.width);
    float gate[N], v[N];
    gate_raw.template values<T>(gate);
    up_raw.template values<T>(v);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float2 a = __fmul2_rn(silu2(make_float2(gate[2 * i], gate[2 * i + 1])),
                                  make_float2(v[2 * i], v[2 * i + 1]));
      v[2 * i] = a.x, v[2 * i + 1] = a.y;
    }
    const bool in = at.in(p.rows);
    if (p.act && in) {
      uint4 *to = reinterpret_cast<uint4 *>(static_cast<T *>(p.act) + at.row * p.width + at.col());
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float some[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) some[i] = v[h * (N / 2) + i];
        to[h] = Piece<T>::store(some);
      }
    }
    if (p.q) {
      const float scale = block_scale(v);
      uint32_t w[N / 4];
      quantise(v, scale, w);
      if (in) {
        store_codes<N>(p.q + at.row * p.width + at.col(), w);
        if ((threadIdx.x & (kLanes - 1)) == 0) p.scales[at.row * p.blocks + at.block] = scale;
      }
    }
    at = next;
    gate_raw = next_gate, up_raw = next_up;
  }
}

// CTAs for `rows` rows, at most `per_sm` a multiprocessor.
cudaError_t launch_rows(void (*k)(Rows8Params), int64_t rows, int64_t piece, int per_sm,
                        Rows8Params p, cudaStream_t s) {
  p.blocks = (p.width - 1) / MLG_F8_BLOCK + 1;
  p.rows = rows;
  const int64_t per_cta = kWarps8 * 32 * 2 * piece / MLG_F8_BLOCK;
  int64_t grid = (rows * p.blocks + per_cta - 1) / per_cta;
  if (grid > per_sm * sm_count()) grid = per_sm * sm_count();
  return launch_early(k, grid, kWarps8 * 32, 0, 1, s, p);
}

}  // namespace
}  // namespace mlg

extern "C" {

mlg_status mlg_rows_f8(const void *x, int32_t type, int64_t ld_x, const int32_t *pos, mlg_f8 *q,
                       float *scales, int32_t n_tokens, int32_t width, int32_t top_k,
                       int32_t n_rows, void *stream) {
  using namespace mlg;
  if (n_tokens < 0 || width < 1 || top_k < 1 || n_rows < 0 || !known_type(type) || ld_x < width)
    return MLG_ERR_INVALID_ARG;
  const int64_t piece = 16 / static_cast<int64_t>(type_size(type));
  if (width % 16 != 0 || ld_x % piece != 0 || int64_t{n_tokens} * top_k > INT32_MAX)
    return MLG_ERR_UNSUPPORTED;
  if (n_tokens == 0) return MLG_OK;
  if (!x || !q || !scales) return MLG_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(q) || !aligned4(scales) || !aligned4(pos))
    return MLG_ERR_UNSUPPORTED;
  Rows8Params p = {};
  p.x = x;
  p.ld_x = ld_x;
  p.pos = pos;
  p.q = reinterpret_cast<uint8_t *>(q);
  p.scales = scales;
  p.width = width;
  p.top_k = top_k;
  p.n_rows = n_rows;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(launch_rows(
      type == MLG_TYPE_BF16 ? rows8_kernel<__nv_bfloat16> : rows8_kernel<float>, n_tokens, piece,
      kRowsCtas8, p, s));
}

mlg_status mlg_swiglu_f8(const void *gate_up, int32_t type, int64_t ld, void *act, mlg_f8 *q,
                         float *scales, int32_t n_rows, int32_t inter, void *stream) {
  using namespace mlg;
  if (n_rows < 0 || inter < 1 || !known_type(type) || ld < 2 * int64_t{inter})
    return MLG_ERR_INVALID_ARG;
  const int64_t piece = 16 / static_cast<int64_t>(type_size(type));
  if (inter % 16 != 0 || ld % piece != 0) return MLG_ERR_UNSUPPORTED;
  if (n_rows == 0) return MLG_OK;
  if (!gate_up || (!q != !scales) || (!q && !act)) return MLG_ERR_INVALID_ARG;
  if (!aligned16(gate_up) || !aligned16(act) || !aligned16(q) || !aligned4(scales))
    return MLG_ERR_UNSUPPORTED;
  Rows8Params p = {};
  p.x = gate_up;
  p.ld_x = ld;
  p.act = act;
  p.q = reinterpret_cast<uint8_t *>(q);
  p.scales = scales;
  p.width = inter;
  p.n_rows = n_rows;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(launch_rows(type == MLG_TYPE_BF16 ? swiglu8_kernel<__nv_bfloat16>
                                                       : swiglu8_kernel<float>,
                                 n_rows, piece, kSwigluCtas8, p, s));
}

}  // extern "C"
