// mlg_launch.cuh -- launch helper and small device helpers shared by the
// kernels around the fold (router, row order, 4-bit product).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "mlg.h"
#include "mlg_internal.h"
#include "mlg_ptx.cuh"

namespace mlg {

constexpr uint32_t kFullWarp = 0xffffffffu;

// Launch with early start (programmatic dependent launch): the kernel may
// become resident while the preceding one runs.  It calls griddep_wait() before
// it touches memory, and griddep_launch_dependents() only then: what comes next
// may read early (the decode folds their tables and pairs) what any kernel before
// this one wrote.  A kernel that is only ever launched behind one of these may
// read before its wait, and release its successor, what the one before does not
// write (dispatch_kernel).  cluster > 1 adds a cluster dimension.
template <typename... A>
cudaError_t launch_early(void (*kernel)(A...), int64_t grid, int threads, size_t smem, int cluster,
                         cudaStream_t stream, const std::remove_cv_t<A> &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Lets a kernel have up to `bytes` of dynamic shared memory, and all of a multiprocessor's for
// its CTAs (left to itself the driver may keep so much for L1 that one CTA fits where two would).
template <typename K>
cudaError_t allow_smem(K kernel, uint32_t bytes) {
  const void *f = reinterpret_cast<const void *>(kernel);
  const cudaError_t err = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(bytes));
  if (err != cudaSuccess) return err;
  return cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout,
                              cudaSharedmemCarveoutMaxShared);
}

inline size_t type_size(int32_t type) { return type == MLG_TYPE_BF16 ? 2 : 4; }
inline bool known_type(int32_t type) { return type == MLG_TYPE_BF16 || type == MLG_TYPE_F32; }

// 16 bytes of a row as fp32 values, and back with one rounding each.
template <typename T>
struct Piece;
template <>
struct Piece<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void load(const uint4 &v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16lo_to_f32(w[i]);
      f[2 * i + 1] = bf16hi_to_f32(w[i]);
    }
  }
  static __device__ __forceinline__ uint4 store(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct Piece<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void load(const uint4 &v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 store(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullWarp, v, o);
  return v;
}

// Waits until the phase is complete, false once the CTA has given up (ctl.abort_flag); a wait past
// kWaitLimitNs sets that and an error bit.
template <class Ctl>
__device__ __forceinline__ bool wait_or_abort(Ctl &ctl, uint64_t &bar, uint32_t parity,
                                              uint32_t *errors) {
  const uint32_t a = smem_addr(&bar);
  if (mbar_try_wait(a, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
    if (mbar_try_wait(a, parity)) return true;
    if (ctl.abort_flag) return false;
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      atomicOr(errors, kErrWaitTimeout);
      ctl.abort_flag = 1;
      return false;
    }
  }
}

// A number as a pair of fp32 operands.
__device__ __forceinline__ float2 both(float f) { return make_float2(f, f); }

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }

}  // namespace mlg
