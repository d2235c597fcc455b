// mlg_q4.cu -- the decode-side product of gathered rows with 4-bit expert
// weights:  out[r, n] = sum_k x[r / top_k, k] * scale * (code - zero).
//
// One warp per output element; a lane takes eight codes (one word) at a time.
#include "mlg_launch.cuh"

namespace mlg {
namespace {

constexpr int kWarps = 8;

struct Q4Params {
  const uint8_t *x;  // bf16 rows
  const int32_t *indices;
  const uint8_t *codes;
  const __nv_bfloat16 *scales;
  const uint8_t *zeros;
  __nv_bfloat16 *out;
  int32_t n_slots, k_in, n_out, top_k, n_experts, group, n_tiles;
};

__global__ void __launch_bounds__(kWarps * 32) q4_kernel(const Q4Params p) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.x / p.n_tiles;
  const int n = (blockIdx.x % p.n_tiles) * kWarps + (threadIdx.x >> 5);
  if (n >= p.n_out) return;
  const int e = p.indices ? p.indices[r] : 0;
  float sum = 0.0f;
  if (e >= 0 && e < p.n_experts) {
    const int64_t row = static_cast<int64_t>(e) * p.n_out + n;
    const uint32_t *codes = reinterpret_cast<const uint32_t *>(p.codes + row * (p.k_in / 2));
    const int64_t groups = row * (p.k_in / p.group);
    const uint4 *x = reinterpret_cast<const uint4 *>(p.x + static_cast<int64_t>(r / p.top_k) *
                                                               p.k_in * 2);
    for (int i = lane; i < p.k_in / 8; i += 32) {
      const int64_t g = groups + i * 8 / p.group;
      const float zero = p.zeros ? static_cast<float>(p.zeros[g]) : 8.0f;
      const uint32_t c = codes[i];
      float f[8], part = 0.0f;
      Piece<__nv_bfloat16>::load(x[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        part += f[j] * (static_cast<float>((c >> (4 * j)) & 15u) - zero);
      sum += part * __bfloat162float(p.scales[g]);
    }
    sum = warp_sum(sum);
  }
  if (lane == 0) p.out[static_cast<int64_t>(r) * p.n_out + n] = __float2bfloat16_rn(sum);
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
  if (k_in % group != 0 || n_out % 8 != 0) return MLG_ERR_UNSUPPORTED;
  if (n_slots == 0) return MLG_OK;
  if (!out || (n_experts > 0 && (!x || !codes || !scales))) return MLG_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(scales) & 1u) != 0)
    return MLG_ERR_UNSUPPORTED;
  Q4Params p = {};
  p.x = reinterpret_cast<const uint8_t *>(x);
  p.indices = indices;
  p.codes = codes;
  p.scales = reinterpret_cast<const __nv_bfloat16 *>(scales);
  p.zeros = zeros;
  p.out = reinterpret_cast<__nv_bfloat16 *>(out);
  p.n_slots = n_slots;
  p.k_in = k_in;
  p.n_out = n_out;
  p.top_k = top_k;
  p.n_experts = n_experts;
  p.group = group;
  p.n_tiles = (n_out + kWarps - 1) / kWarps;
  const int64_t grid = static_cast<int64_t>(n_slots) * p.n_tiles;
  if (grid > 0x7fffffff) return MLG_ERR_UNSUPPORTED;
  return cuda_status(launch_early(q4_kernel, grid, kWarps * 32, 0, 1,
                                  static_cast<cudaStream_t>(stream), p));
}
