// int8.cu -- the product of 8-bit integers with one scale for each token and each channel:
//   out[t, n] = bf16( sum_k a[t, k] w[n, k] * a_scales[t] * w_scales[n] )
// The sums are exact int32 (|sum| <= 127^2 K < 2^31); each is converted to fp32, multiplied by
// the two scales and rounded once.  The rows' codes come from nvfp4_int8_quantize or
// moe_nvfp4_pre_norm_int8 (norm.cu).
#include "dense.cuh"

namespace nvfp4 {
namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <bool LOSE>
int product(const int8_t *a, const float *a_scales, const int8_t *w, const float *w_scales,
            int64_t T, int64_t N, int64_t K, __nv_bfloat16 *out, int32_t *error_flag,
            cudaStream_t stream) {
  if (T < 0 || N <= 0 || K <= 0) return NVFP4_EINVAL;
  if (K % 16 || N % 8 || K > 32768 || N > (1 << 24) || T >= (int64_t(1) << 30) ||
      T > (int64_t(1) << 44) / N)
    return NVFP4_ESHAPE;
  if (!w || !w_scales || !aligned16(w) || !aligned16(w_scales) ||
      (reinterpret_cast<uintptr_t>(error_flag) & 3))
    return NVFP4_EINVAL;
  if (LOSE && (T == 0 || !error_flag)) return NVFP4_EINVAL;
  if (T == 0) return NVFP4_OK;
  if (!a || !a_scales || !out || !aligned16(a) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(a_scales) & 3))
    return NVFP4_EINVAL;
  DenseArgs p = {};
  p.K = K, p.out = out, p.ld = N, p.flag = error_flag;
  if (dense_use_pair(T, N)) {
    p.M = T, p.N = N, p.m_scale = a_scales, p.n_scale = w_scales;
    CUtensorMap to;
    if (int st = out_map(&to, out, T, N, N)) return st;
    return launch_pair<kS8, false, false, kEpiScale, 0, LOSE>(p, {a, w}, to, to, to, stream);
  }
  p.M = N, p.N = T, p.m_scale = w_scales, p.n_scale = a_scales;
  return launch_split_n<kS8, false, kEpiScale, 0, LOSE>(p, {w, a}, stream);
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" int nvfp4_int8_matmul(const int8_t *a, const float *a_scales, const int8_t *w,
                                 const float *w_scales, int64_t T, int64_t N, int64_t K,
                                 __nv_bfloat16 *out, int32_t *error_flag, cudaStream_t stream) {
  return product<false>(a, a_scales, w, w_scales, T, N, K, out, error_flag, stream);
}

extern "C" int nvfp4_selftest_int8_matmul_timeout(const int8_t *a, const float *a_scales,
                                                  const int8_t *w, const float *w_scales,
                                                  int64_t T, int64_t N, int64_t K,
                                                  __nv_bfloat16 *out, int32_t *error_flag,
                                                  cudaStream_t stream) {
  return product<true>(a, a_scales, w, w_scales, T, N, K, out, error_flag, stream);
}
