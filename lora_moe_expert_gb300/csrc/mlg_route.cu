// mlg_route.cu -- the router: top_k experts of each token with their softmax
// weights, and the weights' gradient.
//
// One warp owns a token and keeps its logits in registers as unsigned keys that
// order as the logits do, so a choice is a warp-wide integer maximum over each
// lane's best key (redux).  fp32 keys fill 32 bits: a second reduction finds the
// lowest id that holds the maximum, and the lane that held it looks for its next
// best when its second is gone too.  bf16 keys leave room for the id in the same
// word: one reduction, all keys different.  There a lane knows its three best,
// and the winner moves up its next: no search, no branch.  Only a lane that three
// were chosen of has to look for a fourth (the largest below its third key k, as
// keys below k are the largest key - k, mod 2^32: one fused add-and-maximum a
// value), and only if that would have been chosen the slower loop, which searches
// as it goes, begins anew.  That loop alone serves top_k above 24, where it is
// the usual end (16384 x 256, top 32: 14.5 us against 15.2; top 24 11.5, 10.7).
//
// Instructions bound it, half of them on the integer pipe: 16384 tokens x 512 bf16
// logits, top 10, take 8.3 us (16.8 MB, 30 % of the copy bandwidth; the searching
// loop alone 9.0, keys and ids apart 33), fp32 15 us; 64 x 128, top 8, 1.5 us,
// which is the launch.
//
// The gradient reads and writes each logit once, one warp a token, everything
// in registers: 4099 x 97 fp32 logits 2.0 us (3.5 MB), launch and one round trip.
#include <cfloat>

#include "mlg_launch.cuh"

namespace mlg {
namespace {

constexpr int kWarps = 8;  // a CTA's at most
constexpr int kFastTopK = 24;

struct RouteParams {
  const void *logits;
  int64_t ld_logits;
  int32_t *indices;
  float *weights;
  const float *dweights;
  void *dlogits;
  int64_t ld_dlogits;
  int32_t n_tokens, n_experts, top_k, renormalize;
};

// Order-preserving key of a logit: 0 for one that cannot be chosen (-inf,
// NaN), +inf as the largest finite value, -0 as +0 (they compare equal).
__device__ __forceinline__ uint32_t logit_key(float v) {
  const uint32_t b = __float_as_uint(fminf(v, FLT_MAX) + 0.0f);
  const uint32_t turned = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
  return v > -INFINITY ? turned : 0u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

template <int VPL>
__global__ void __launch_bounds__(kWarps * 32) route_topk_kernel(const RouteParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= p.n_tokens) return;
  __shared__ uint2 chosen[kWarps][MLG_ROUTE_MAX_TOP_K];
  const float *row = static_cast<const float *>(p.logits) + t * p.ld_logits;
  float logit[VPL];  // all loads under way before any is used
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    logit[i] = i * 32 + lane < p.n_experts ? row[i * 32 + lane] : -INFINITY;
  uint32_t key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) key[i] = logit_key(logit[i]);
  uint32_t best = 0, second = 0;  // the lane's two best, at steps `at` and `at2`
  int at = 0, at2 = 0;            // at2 -1: not known
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    if (key[i] > best) {
      second = best, at2 = at;
      best = key[i], at = i;
    } else if (key[i] > second) {
      second = key[i], at2 = i;
    }
  }

  const uint32_t top = __reduce_max_sync(kFullWarp, best);
  const float m = key_logit(top);
  float total = 0.0f;
  if (!p.renormalize) {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (key[i]) total += expf(key_logit(key[i]) - m);
    total = warp_sum(total);
  }

  // Key 0, once all are gone, is told after the rounds.
  uint2 *choices = chosen[threadIdx.x >> 5];  // id and key
  for (int j = 0; j < p.top_k; ++j) {
    const uint32_t k = __reduce_max_sync(kFullWarp, best);
    const uint32_t mine = best == k ? static_cast<uint32_t>(at * 32 + lane) : 0xffffffffu;
    const uint32_t e = __reduce_min_sync(kFullWarp, mine);
    const bool won = mine == e;  // one lane
    if (won) choices[j] = make_uint2(e, k);
    const int gone = at;
    if (won) best = second, at = at2, at2 = -1, second = 0;
    if (won && at < 0) {  // what comes after (k, gone) in its order
      best = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if ((key[i] < k || (key[i] == k && i > gone)) && key[i] > best) best = key[i], at = i;
    }
    __syncwarp();
  }
  const uint2 mine = lane < p.top_k ? choices[lane] : make_uint2(0, 0);  // choice `lane`
  const int my_id = mine.y ? static_cast<int>(mine.x) : -1;
  const float w = my_id >= 0 ? expf(key_logit(mine.y) - m) : 0.0f;
  if (p.renormalize) total = warp_sum(w);
  if (lane < p.top_k) {
    const int64_t o = static_cast<int64_t>(t) * p.top_k + lane;
    p.indices[o] = my_id;
    p.weights[o] = my_id >= 0 ? w / total : 0.0f;
  }
}

// bf16 logits, two a word: lane l holds experts 64 i + 2 l and the next (h = 1).
// A key is value (bits 15..30) | 15 - i (6..9) | 31 - l (1..5) | 1 - h (0), in
// the order of the ids, with a lane's own number left out of its local keys and
// put into what it offers.  PAIRS: word loads; FULL: n_experts = 64 WPL.
template <int WPL, bool PAIRS, bool FULL>
__global__ void __launch_bounds__(kWarps * 32) route_topk_bf16_kernel(const RouteParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= p.n_tokens) return;
  constexpr uint32_t kMasked = 0x007fu;  // the 16-bit key of -inf
  __shared__ uint32_t chosen[kWarps][MLG_ROUTE_MAX_TOP_K];
  const uint16_t *row = static_cast<const uint16_t *>(p.logits) + t * p.ld_logits;
  uint32_t key[2 * WPL], best = 0, second = 0, third = 0;  // the lane's
#pragma unroll
  for (int i = 0; i < WPL; ++i) {
    const int e = i * 64 + lane * 2;
    uint32_t w = 0xff80ff80u;
    if (PAIRS) {
      if (FULL || e < p.n_experts) w = *reinterpret_cast<const uint32_t *>(row + e);
    } else {
      if (e < p.n_experts) w = (w & 0xffff0000u) | row[e];
      if (e + 1 < p.n_experts) w = (w & 0xffffu) | static_cast<uint32_t>(row[e + 1]) << 16;
    }
    // NaN becomes -inf and -0 becomes +0; then the sign bit of positive and
    // all bits of negative values turn
    const __nv_bfloat162 inf2 = __halves2bfloat162(__ushort_as_bfloat16(0xff80),
                                                   __ushort_as_bfloat16(0xff80));
    const __nv_bfloat162 zero2 = __halves2bfloat162(__ushort_as_bfloat16(0),
                                                    __ushort_as_bfloat16(0));
    const __nv_bfloat162 v =
        __hadd2(__hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&w), inf2), zero2);
    w = *reinterpret_cast<const uint32_t *>(&v);
    w ^= (__hlt2_mask(v, zero2) & 0x7fff7fffu) | 0x80008000u;
    key[2 * i] = ((w << 15) & 0x7fff8000u) | static_cast<uint32_t>((15 - i) << 6 | 1);
    key[2 * i + 1] = ((w >> 1) & 0x7fff8000u) | static_cast<uint32_t>((15 - i) << 6);
    const uint32_t hi = max(key[2 * i], key[2 * i + 1]), lo = min(key[2 * i], key[2 * i + 1]);
    third = max(max(third, min(best, lo)), min(second, hi));
    second = max(max(second, lo), min(best, hi));
    best = max(best, hi);
  }
  const uint32_t own = static_cast<uint32_t>(31 - lane) << 1;
  auto value = [](uint32_t k16) {  // of a 16-bit key; +inf as the largest finite
    const uint32_t h = (k16 & 0x8000u) ? (k16 & 0x7fffu) : (~k16 & 0xffffu);
    return fminf(__uint_as_float(h << 16), FLT_MAX);
  };
  const uint32_t top = __reduce_max_sync(kFullWarp, best | own) >> 15;
  const float m = value(top);
  float total = 0.0f;
  if (!p.renormalize) {
#pragma unroll
    for (int i = 0; i < 2 * WPL; ++i)
      if ((key[i] >> 15) > kMasked) total += expf(value(key[i] >> 15) - m);
    total = warp_sum(total);
  }
  // Every round has one winner, as the offers of two lanes differ; what cannot be
  // chosen comes last and is told after.
  uint32_t *choices = chosen[threadIdx.x >> 5];
  bool done = false;
  if (p.top_k <= kFastTopK || WPL == 1) {
    // A lane offers its three best.  One that all three were chosen of looks
    // whether it has a fourth above the last choice: then the other loop.
    uint32_t s1 = best | own, s2 = second | own, s3 = WPL > 1 ? third | own : 0u, k = 0;
#pragma unroll 2
    for (int j = 0; j < p.top_k; ++j) {
      k = __reduce_max_sync(kFullWarp, s1);
      const bool won = s1 == k;
      if (won) choices[j] = k;
      s1 = won ? s2 : s1;
      s2 = won ? s3 : s2;
      s3 = won ? 0u : s3;
    }
    done = true;
    if (WPL > 1 && __any_sync(kFullWarp, s1 == 0)) {
      uint32_t fourth = 0;
#pragma unroll
      for (int i = 0; i < 2 * WPL; ++i) fourth = max(fourth, key[i] - third);
      fourth = fourth > 0x7fffffffu ? (fourth + third) | own : 0u;
      done = !__any_sync(kFullWarp, s1 == 0 && fourth > k);
    }
  }
  if (!done) {  // second 0: not known
    __syncwarp();  // the choices above are written before these, by whichever lanes
    for (int j = 0; j < p.top_k; ++j) {
      const uint32_t offer = best | own;
      const uint32_t k = __reduce_max_sync(kFullWarp, offer);
      const bool won = offer == k;
      if (won) choices[j] = k;
      uint32_t next = won ? second : best;
      if (next == 0 && won) {
#pragma unroll
        for (int i = 0; i < 2 * WPL; ++i) next = max(next, key[i] - best);
        next = next > 0x7fffffffu ? next + best : 0u;
      }
      second = won ? 0u : second;
      best = next;
      __syncwarp();
    }
  }
  __syncwarp();
  uint32_t mine = lane < p.top_k ? choices[lane] : 0u;  // choice `lane`
  if (mine <= (kMasked << 15 | 0x7fffu)) mine = 0;
  const float w = mine ? expf(value(mine >> 15) - m) : 0.0f;
  if (p.renormalize) total = warp_sum(w);
  if (lane < p.top_k) {
    const int64_t o = static_cast<int64_t>(t) * p.top_k + lane;
    const uint32_t inv = ~mine;  // ids count down in a key
    p.indices[o] = mine ? static_cast<int>((inv >> 6 & 15u) << 6 | (inv >> 1 & 31u) << 1 | (inv & 1u))
                        : -1;
    p.weights[o] = mine ? w / total : 0.0f;
  }
}

// One warp per token: every element -p_e * s (s = sum of weight * dweight over
// the chosen; 0 for all when renormalized), then the chosen ones again with
// their own term.  Lane l holds elements 32 PER i + PER l and the next PER - 1
// (PER 2: bf16 rows on 4-byte boundaries).
template <typename T, int PER, int STEPS>
__global__ void __launch_bounds__(kWarps * 32) route_backward_kernel(const RouteParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, E = p.n_experts;
  const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= p.n_tokens) return;
  const T *row = static_cast<const T *>(p.logits) + t * p.ld_logits;
  T *out = static_cast<T *>(p.dlogits) + t * p.ld_dlogits;
  float v[STEPS][PER];
  if (!p.renormalize) {
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int e = (i * 32 + lane) * PER;
      if (PER == 2) {
        const uint32_t w = e < E ? *reinterpret_cast<const uint32_t *>(row + e) : 0xff80ff80u;
        v[i][0] = bf16lo_to_f32(w);
        v[i][PER - 1] = bf16hi_to_f32(w);
      } else {
        v[i][0] = e < E ? to_f32(row[e]) : -INFINITY;
      }
    }
  }
  int id = -1;
  float w = 0.0f, dw = 0.0f;
  if (lane < p.top_k) {
    const int64_t o = static_cast<int64_t>(t) * p.top_k + lane;
    id = p.indices[o];
    w = p.weights[o];
    dw = p.dweights[o];
    if (id < 0 || id >= E) id = -1;
  }
  const float wdw = id >= 0 ? w * dw : 0.0f;
  const float s = warp_sum(wdw);
  if (p.renormalize) {
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
#pragma unroll
      for (int h = 0; h < PER; ++h) v[i][h] = 0.0f;
  } else {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
#pragma unroll
      for (int h = 0; h < PER; ++h) {
        v[i][h] = v[i][h] > -INFINITY ? fminf(v[i][h], FLT_MAX) : -INFINITY;  // NaN: -inf
        top = max(top, logit_key(v[i][h]));
      }
    top = __reduce_max_sync(kFullWarp, top);
    const float m = top ? key_logit(top) : 0.0f;
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
#pragma unroll
      for (int h = 0; h < PER; ++h) {
        v[i][h] = expf(v[i][h] - m);  // 0 for -inf
        z += v[i][h];
      }
    z = warp_sum(z);
    const float c = z > 0.0f ? -s / z : 0.0f;
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
#pragma unroll
      for (int h = 0; h < PER; ++h) v[i][h] *= c;
  }
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int e = (i * 32 + lane) * PER;
    if (e >= E) continue;
    if (PER == 2)
      *reinterpret_cast<uint32_t *>(out + e) = pack_bf16x2(v[i][0], v[i][PER - 1]);
    else
      put(out + e, v[i][0]);
  }
  __syncwarp();  // the chosen after all
  if (id >= 0) put(out + id, wdw - w * s);
}

// One warp a token, 8 of them a CTA where a token is so little work that the
// launching of CTAs shows (16384 x 128 bf16, top 8: 4.8 us, 5.4 with 4), else 4,
// which end more evenly (16384 x 512 fp32, top 10: 15.2 us, 15.7 with 8).
cudaError_t launch_tokens(void (*k)(RouteParams), const RouteParams &p, cudaStream_t s) {
  const int warps = p.n_experts <= 128 ? kWarps : kWarps / 2;
  return launch_early(k, (int64_t{p.n_tokens} + warps - 1) / warps, warps * 32, 0, 1, s, p);
}

cudaError_t launch_topk_f32(const RouteParams &p, cudaStream_t s) {
  const int E = p.n_experts;
  void (*k)(RouteParams) = E <= 32    ? route_topk_kernel<1>
                           : E <= 64  ? route_topk_kernel<2>
                           : E <= 128 ? route_topk_kernel<4>
                           : E <= 256 ? route_topk_kernel<8>
                           : E <= 512 ? route_topk_kernel<16>
                                      : route_topk_kernel<32>;
  return launch_tokens(k, p, s);
}

template <bool PAIRS>
cudaError_t launch_topk_bf16(const RouteParams &p, cudaStream_t s) {
  const int E = p.n_experts;
  void (*k)(RouteParams) = E <= 64    ? route_topk_bf16_kernel<1, PAIRS, false>
                           : E <= 128 ? route_topk_bf16_kernel<2, PAIRS, false>
                           : E <= 256 ? route_topk_bf16_kernel<4, PAIRS, false>
                           : E <= 512 ? route_topk_bf16_kernel<8, PAIRS, false>
                                      : route_topk_bf16_kernel<16, PAIRS, false>;
  if (PAIRS)  // no lane has less than its share
    switch (E) {
      case 64: k = route_topk_bf16_kernel<1, PAIRS, PAIRS>; break;
      case 128: k = route_topk_bf16_kernel<2, PAIRS, PAIRS>; break;
      case 256: k = route_topk_bf16_kernel<4, PAIRS, PAIRS>; break;
      case 512: k = route_topk_bf16_kernel<8, PAIRS, PAIRS>; break;
      case 1024: k = route_topk_bf16_kernel<16, PAIRS, PAIRS>; break;
    }
  return launch_tokens(k, p, s);
}

template <typename T, int PER>
cudaError_t launch_backward(const RouteParams &p, cudaStream_t s) {
  const int steps = (p.n_experts + 32 * PER - 1) / (32 * PER);
  void (*k)(RouteParams) = steps <= 1   ? route_backward_kernel<T, PER, 1>
                           : steps <= 2 ? route_backward_kernel<T, PER, 2>
                           : steps <= 4 ? route_backward_kernel<T, PER, 4>
                           : steps <= 8 ? route_backward_kernel<T, PER, 8>
                           : steps <= 16 ? route_backward_kernel<T, PER, 16>
                                         : route_backward_kernel<T, PER, 32 / PER>;
  return launch_tokens(k, p, s);
}

mlg_status check(int32_t type, int32_t n_tokens, int32_t n_experts, int32_t top_k) {
  if (n_tokens < 0 || n_experts < 1 || top_k < 1 || !known_type(type)) return MLG_ERR_INVALID_ARG;
  if (n_experts > MLG_ROUTE_MAX_EXPERTS || top_k > MLG_ROUTE_MAX_TOP_K)
    return MLG_ERR_UNSUPPORTED;
  return MLG_OK;
}

bool element_aligned(const void *p, int32_t type) {
  return (reinterpret_cast<uintptr_t>(p) & (type_size(type) - 1)) == 0;
}

}  // namespace
}  // namespace mlg

extern "C" {

mlg_status mlg_route_topk(const void *logits, int32_t logits_type, int64_t ld_logits,
                          int32_t *indices, float *weights, int32_t n_tokens, int32_t n_experts,
                          int32_t top_k, int32_t renormalize, void *stream) {
  using namespace mlg;
  const mlg_status st = check(logits_type, n_tokens, n_experts, top_k);
  if (st != MLG_OK) return st;
  if (ld_logits < n_experts) return MLG_ERR_INVALID_ARG;
  if (n_tokens == 0) return MLG_OK;
  if (!logits || !indices || !weights) return MLG_ERR_INVALID_ARG;
  if (!element_aligned(logits, logits_type)) return MLG_ERR_UNSUPPORTED;
  RouteParams p = {};
  p.logits = logits;
  p.ld_logits = ld_logits;
  p.indices = indices;
  p.weights = weights;
  p.n_tokens = n_tokens;
  p.n_experts = n_experts;
  p.top_k = top_k;
  p.renormalize = renormalize != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (logits_type == MLG_TYPE_F32) return cuda_status(launch_topk_f32(p, s));
  // Two bf16 a load where every row begins on a 4-byte boundary and ends on one.
  const bool pairs = n_experts % 2 == 0 && ld_logits % 2 == 0 &&
                     (reinterpret_cast<uintptr_t>(logits) & 3u) == 0;
  return cuda_status(pairs ? launch_topk_bf16<true>(p, s) : launch_topk_bf16<false>(p, s));
}

mlg_status mlg_route_topk_backward(const void *logits, int32_t logits_type, int64_t ld_logits,
                                   const int32_t *indices, const float *weights,
                                   const float *dweights, void *dlogits, int64_t ld_dlogits,
                                   int32_t n_tokens, int32_t n_experts, int32_t top_k,
                                   int32_t renormalize, void *stream) {
  using namespace mlg;
  const mlg_status st = check(logits_type, n_tokens, n_experts, top_k);
  if (st != MLG_OK) return st;
  if (ld_dlogits < n_experts || (!renormalize && ld_logits < n_experts))
    return MLG_ERR_INVALID_ARG;
  if (n_tokens == 0) return MLG_OK;
  if (!indices || !weights || !dweights || !dlogits || (!renormalize && !logits))
    return MLG_ERR_INVALID_ARG;
  if (!element_aligned(dlogits, logits_type) ||
      (!renormalize && !element_aligned(logits, logits_type)))
    return MLG_ERR_UNSUPPORTED;
  RouteParams p = {};
  p.logits = logits;
  p.ld_logits = ld_logits;
  p.indices = const_cast<int32_t *>(indices);
  p.weights = const_cast<float *>(weights);
  p.dweights = dweights;
  p.dlogits = dlogits;
  p.ld_dlogits = ld_dlogits;
  p.n_tokens = n_tokens;
  p.n_experts = n_experts;
  p.top_k = top_k;
  p.renormalize = renormalize != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (logits_type == MLG_TYPE_F32) return cuda_status(launch_backward<float, 1>(p, s));
  const bool pairs = n_experts % 2 == 0 && ld_dlogits % 2 == 0 &&
                     (reinterpret_cast<uintptr_t>(dlogits) & 3u) == 0 &&
                     (renormalize || (ld_logits % 2 == 0 &&
                                      (reinterpret_cast<uintptr_t>(logits) & 3u) == 0));
  return cuda_status(pairs ? launch_backward<__nv_bfloat16, 2>(p, s)
                           : launch_backward<__nv_bfloat16, 1>(p, s));
}

}  // extern "C"
