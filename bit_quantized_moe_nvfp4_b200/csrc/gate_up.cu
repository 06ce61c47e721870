// gate_up.cu -- the gated projection of a feed-forward block and its gradients, BF16:
//   [g | u] = x w_gu^T,   h = act(g) u                       (one kernel; sums stay in TMEM)
//   dg = dh u act'(g),    du = dh act(g)                     (elementwise, into the workspace)
//   dx = [dg | du] w_gu,  dw_gu = [dg | du]^T x              (two products)
// The gradients' operands are used as they lie in memory (MN-major tensor-core operands).
// dg and du are rounded to bf16, the type the tensor cores take; everything before and after
// that is fp32 with one rounding.  The second rounding costs dx and dw_gu 0.0023 of their 2-norm
// against 0.0017 for the result's own alone; two bf16 terms for each of dg and du would save it at
// twice the products' time.
#include "dense.cuh"

namespace nvfp4 {
namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// act(z) and act'(z).  GELU: with s = 1 / (1 + exp(-2 v)), act = z s and its slope is
// s (1 + 2 z (1 - s) v'); the smaller of s and 1 - s is the quotient e / (1 + e), not a difference.
// From |z| = 11 on it is 0 in fp32 and so is its product; there z is held at 32, lest z v'
// overflow beside it.
template <int ACT>
__device__ __forceinline__ void act_grad(float z, float &a, float &da) {
  if (ACT == NVFP4_ACT_SILU) {
    const float s = 1.f / (1.f + expf(-z));
    a = z * s;
    da = s * fmaf(z, 1.f - s, 1.f);
  } else {
    const float v = gelu_v(z), e = expf(-2.f * fabsf(v));
    const float big = 1.f / (1.f + e), small = e * big;
    const float s = z < 0.f ? small : big, rest = z < 0.f ? big : small;
    const float zc = fminf(fmaxf(z, -32.f), 32.f);
    const float dv = kGeluA * fmaf(3.f * kGeluB, zc * zc, 1.f);
    a = z * s;
    da = s * fmaf(2.f * zc * rest, dv, 1.f);
  }
}

// One thread takes 8 columns of a row: 16-byte loads of g, u and dh, 16-byte stores of dg, du.
// Bound by HBM: 4096 x 2048 moves 84 MB in 16 us (5.2 TB/s).
template <int ACT>
__global__ void __launch_bounds__(256) gate_grad_kernel(const __nv_bfloat16 *gu,
                                                        const __nv_bfloat16 *dh,
                                                        __nv_bfloat16 *dgu, int64_t T, int I) {
  const int nv = I / 8;
  const int64_t total = T * nv;
  pdl_launch_dependents();
  pdl_wait();
  for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < total;
       e += (int64_t)gridDim.x * blockDim.x) {
    const int64_t t = e / nv;
    const int c = (int)(e - t * nv);
    const uint4 *row = reinterpret_cast<const uint4 *>(gu + t * 2 * I);
    const uint4 gv = ld_stream(row + c), uv = ld_stream(row + nv + c);
    const uint4 dv = ld_stream(reinterpret_cast<const uint4 *>(dh) + e);
    const uint32_t g[4] = {gv.x, gv.y, gv.z, gv.w}, u[4] = {uv.x, uv.y, uv.z, uv.w};
    const uint32_t d[4] = {dv.x, dv.y, dv.z, dv.w};
    uint32_t og[4], ou[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float a0, s0, a1, s1;
      act_grad<ACT>(bf16_lo(g[k]), a0, s0);
      act_grad<ACT>(bf16_hi(g[k]), a1, s1);
      const float d0 = bf16_lo(d[k]), d1 = bf16_hi(d[k]);
      // the slope first: it is at most 1.13, so nothing overflows that the result does not
      og[k] = pack_bf16x2(d0 * (bf16_lo(u[k]) * s0), d1 * (bf16_hi(u[k]) * s1));
      ou[k] = pack_bf16x2(d0 * a0, d1 * a1);
    }
    uint4 *o = reinterpret_cast<uint4 *>(dgu + t * 2 * I);
    o[c] = make_uint4(og[0], og[1], og[2], og[3]);
    o[nv + c] = make_uint4(ou[0], ou[1], ou[2], ou[3]);
  }
}

template <int ACT, bool LOSE = false>
int forward(const __nv_bfloat16 *x, const __nv_bfloat16 *w_gu, int64_t T, int64_t H, int64_t I,
            __nv_bfloat16 *h, __nv_bfloat16 *gu, int32_t *flag, cudaStream_t s) {
  DenseArgs p = {};
  p.K = H, p.half = I, p.out = h, p.gu = gu, p.ld = I, p.flag = flag;
  if (dense_use_pair(T, 2 * I)) {
    p.M = T, p.N = I, p.save_gu = gu != nullptr;
    CUtensorMap th, tg, tu;
    if (int st = out_map(&th, h, T, I, I)) return st;
    tg = tu = th;
    if (gu) {   // the two halves of a row are tensors of their own, so a tile ends with its half
      if (int st = out_map(&tg, gu, T, I, 2 * I)) return st;
      if (int st = out_map(&tu, gu + I, T, I, 2 * I)) return st;
    }
    return launch_pair<kBf16, false, false, kEpiGate, ACT, LOSE>(p, {x, w_gu}, th, tg, tu, s);
  }
  p.M = I, p.N = T;
  return launch_split_n<kBf16, false, kEpiGate, ACT, LOSE>(p, {w_gu, x}, s);
}

int check(int64_t T, int64_t H, int64_t I, int act) {
  if (T < 0 || H <= 0 || I <= 0 || (act != NVFP4_ACT_SILU && act != NVFP4_ACT_GELU))
    return NVFP4_EINVAL;
  if (H % 8 || I % 8 || H > 65536 || I > 65536 || T >= (int64_t(1) << 30) ||
      T > (int64_t(1) << 44) / std::max(H, 2 * I))
    return NVFP4_ESHAPE;
  return NVFP4_OK;
}

int check_forward(const __nv_bfloat16 *x, const __nv_bfloat16 *w_gu, int64_t T, int64_t H,
                  int64_t I, int act, const __nv_bfloat16 *h, const __nv_bfloat16 *gu,
                  const int32_t *error_flag) {
  if (int st = check(T, H, I, act)) return st;
  if (!w_gu || !aligned16(w_gu) || (reinterpret_cast<uintptr_t>(error_flag) & 3))
    return NVFP4_EINVAL;
  if (T > 0 && (!x || !h || !aligned16(x) || !aligned16(h) || !aligned16(gu)))
    return NVFP4_EINVAL;
  return NVFP4_OK;
}

int zero(void *p, size_t bytes, cudaStream_t s) {
  const cudaError_t e = cudaMemsetAsync(p, 0, bytes, s);
  if (e == cudaSuccess) return NVFP4_OK;
  set_last_cuda_error(e);
  return NVFP4_ECUDA;
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" int moe_nvfp4_gate_up(const __nv_bfloat16 *x, const __nv_bfloat16 *w_gu, int64_t T,
                                 int64_t H, int64_t I, int act, __nv_bfloat16 *h,
                                 __nv_bfloat16 *gu, int32_t *error_flag, cudaStream_t stream) {
  if (int st = check_forward(x, w_gu, T, H, I, act, h, gu, error_flag)) return st;
  if (T == 0) return NVFP4_OK;
  return act == NVFP4_ACT_SILU ? forward<NVFP4_ACT_SILU>(x, w_gu, T, H, I, h, gu, error_flag, stream)
                               : forward<NVFP4_ACT_GELU>(x, w_gu, T, H, I, h, gu, error_flag, stream);
}

extern "C" int nvfp4_selftest_gate_up_timeout(const __nv_bfloat16 *x, const __nv_bfloat16 *w_gu,
                                              int64_t T, int64_t H, int64_t I, __nv_bfloat16 *h,
                                              __nv_bfloat16 *gu, int32_t *error_flag,
                                              cudaStream_t stream) {
  if (int st = check_forward(x, w_gu, T, H, I, NVFP4_ACT_SILU, h, gu, error_flag)) return st;
  if (T == 0 || !error_flag) return NVFP4_EINVAL;
  return forward<NVFP4_ACT_SILU, true>(x, w_gu, T, H, I, h, gu, error_flag, stream);
}

extern "C" size_t moe_nvfp4_gate_up_backward_workspace_size(int64_t T, int64_t I) {
  if (T <= 0 || I <= 0) return 0;
  return align256((size_t)T * 2 * (size_t)I * 2);
}

extern "C" int moe_nvfp4_gate_up_backward(const __nv_bfloat16 *dh, const __nv_bfloat16 *x,
                                          const __nv_bfloat16 *w_gu, const __nv_bfloat16 *gu,
                                          int64_t T, int64_t H, int64_t I, int act,
                                          __nv_bfloat16 *dx, __nv_bfloat16 *dw_gu,
                                          void *workspace, size_t ws_bytes, int32_t *error_flag,
                                          cudaStream_t stream) {
  if (int st = check(T, H, I, act)) return st;
  if ((!dx && !dw_gu && T > 0) || !aligned16(dx) || !aligned16(dw_gu) ||
      (reinterpret_cast<uintptr_t>(error_flag) & 3))
    return NVFP4_EINVAL;
  if (T == 0) return dw_gu ? zero(dw_gu, (size_t)(2 * I) * (size_t)H * 2, stream) : NVFP4_OK;
  if (!dh || !gu || !aligned16(dh) || !aligned16(gu) || (dx && (!w_gu || !aligned16(w_gu))) ||
      (dw_gu && (!x || !aligned16(x))))
    return NVFP4_EINVAL;
  if (!workspace || !aligned16(workspace) ||
      ws_bytes < moe_nvfp4_gate_up_backward_workspace_size(T, I))
    return NVFP4_EWORKSPACE;
  __nv_bfloat16 *dgu = static_cast<__nv_bfloat16 *>(workspace);
  const int64_t blocks = std::min<int64_t>(ceil_div(T * (I / 8), 256), (int64_t)num_sms() * 8);
  const dim3 grid((unsigned)blocks), block(256);
  if (int st = act == NVFP4_ACT_SILU
                   ? launch_pdl(gate_grad_kernel<NVFP4_ACT_SILU>, grid, block, 0, stream, gu, dh,
                                dgu, T, (int)I)
                   : launch_pdl(gate_grad_kernel<NVFP4_ACT_GELU>, grid, block, 0, stream, gu, dh,
                                dgu, T, (int)I))
    return st;
  CUtensorMap to;
  if (dx) {   // [T, H] = dgu [T, 2I] w_gu [2I, H]
    DenseArgs p = {};
    p.K = 2 * I, p.out = dx, p.ld = H, p.flag = error_flag;
    if (dense_use_pair(T, H)) {
      p.M = T, p.N = H;
      if (int st = out_map(&to, dx, T, H, H)) return st;
      if (int st = launch_pair<kBf16, false, true, kEpiStore, 0>(p, {dgu, w_gu}, to, to, to, stream))
        return st;
    } else {
      p.M = H, p.N = T;
      if (int st = launch_split_n<kBf16, true, kEpiStore, 0>(p, {w_gu, dgu}, stream))
        return st;
    }
  }
  if (dw_gu) {   // [2I, H] = dgu^T [2I, T] x [T, H]
    DenseArgs p = {};
    p.M = 2 * I, p.N = H, p.K = T, p.out = dw_gu, p.ld = H, p.flag = error_flag;
    if (dense_use_pair(2 * I, H)) {
      if (int st = out_map(&to, dw_gu, 2 * I, H, H)) return st;
      return launch_pair<kBf16, true, true, kEpiStore, 0>(p, {dgu, x}, to, to, to, stream);
    }
    return launch_split<kBf16, true, true, kEpiStore, 0, 64, true>(p, {dgu, x}, stream);
  }
  return NVFP4_OK;
}
