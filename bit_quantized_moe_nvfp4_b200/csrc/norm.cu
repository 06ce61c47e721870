// norm.cu -- root-mean-square norms before and after a block, fused with the block's gate and
// the residual sum, their gradients, and rows rounded to 8-bit integers.
//
// For a row x of H values, with r = rsqrt(mean(x^2) + eps) and n = r x:
//   before a block   y    = w n                      (bf16, or 8-bit codes and one scale)
//   after it         out  = a residual + g (w n)     next = w2 out rsqrt(mean(out^2) + eps)
// Gradients, with dn = d g w (d the gradient of the result, g = 1 where there is no gate):
//   dx = r (dn - n mean(dn n)),  dw = sum over rows of d g n,  dg = d w n summed over the
//   axes g is broadcast along,  d residual = a d.
// With x in registers, mean(dn n) = r sum(dn x) / H, so both sums of a row come from one
// pass over it and are reduced together.
//
// Every kernel here is bound by HBM: a row is read once into registers (16-byte loads) and
// each output is written once.  A row of at most 1024 values belongs to a warp (no barrier);
// a longer one to a CTA.  All statistics and sums are fp32; each result is rounded once.
// next is taken from the unrounded out, and codes from the unrounded y.
#include <algorithm>
#include <type_traits>

#include "moe.cuh"

namespace nvfp4 {
namespace {

constexpr int64_t kMaxH = 32768;   // 4 vectors of 8 values for each of 1024 threads
constexpr int kWarpRowVecs = 128;  // rows of up to 128 vectors (1024 values) take a warp
constexpr int kWarps = 8;          // warps of a CTA whose warps take a row each

enum { kPre = 0, kPreInt8 = 1, kPost = 2, kPostNext = 3, kQuant = 4 };

struct NormParams {
  const __nv_bfloat16 *x;         // [T, H]
  const __nv_bfloat16 *w;         // [H]
  const __nv_bfloat16 *residual;  // [T, H]
  const __nv_bfloat16 *gate;      // null, or strides gt (0 or gh ? H : 1) and gh (0 or 1)
  const __nv_bfloat16 *w_next;    // [H]
  __nv_bfloat16 *out;             // [T, H]
  __nv_bfloat16 *next;            // [T, H]
  int8_t *codes;                  // [T, H]
  float *scales;                  // [T]
  int64_t T, gt;
  int H, gh;
  float eps, a;
};

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
  f[4] = bf16_lo(v.z), f[5] = bf16_hi(v.z), f[6] = bf16_lo(v.w), f[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

struct Sum {
  static __device__ __forceinline__ float op(float a, float b) { return a + b; }
};
struct Max {
  static __device__ __forceinline__ float op(float a, float b) { return fmaxf(a, b); }
};

// Reduce N values over the threads that share a row: a warp, or the CTA through `buf`
// ([2][32][N]; the half alternates with `turn`, so one barrier a reduction is enough).
template <bool WARP, typename Op, int N>
__device__ __forceinline__ void reduce_row(float (&v)[N], float *buf, int &turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = Op::op(v[k], __shfl_xor_sync(0xFFFFFFFFu, v[k], o));
  if (WARP) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  float *b = buf + turn * 32 * N;
  turn ^= 1;
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) b[warp * N + k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    float s = b[k];
    for (int w = 1; w < nw; ++w) s = Op::op(s, b[w * N + k]);
    v[k] = s;
  }
}

// Codes of 8 values: the integers nearest to 127 y / amax, ties to even.  For bf16 y both
// 127 y and the distance of the quotient from a tie are exact to far below an fp32 ulp
// (|p / q - (k + 1/2)| >= 1 / (2 q) for q < 2^8), so the fp32 quotient rounds as the real
// one does.  `pre` is a power of two that keeps 127 y finite.
__device__ __forceinline__ uint2 codes8(const float (&y)[8], float pre, float amax) {
  uint32_t q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float v = amax > 0.f ? __fdiv_rn(y[j] * pre * 127.f, amax) : 0.f;
    q[j] = (uint32_t)(uint8_t)(int8_t)__float2int_rn(fminf(fmaxf(v, -127.f), 127.f));
  }
  return make_uint2(q[0] | q[1] << 8 | q[2] << 16 | q[3] << 24,
                    q[4] | q[5] << 8 | q[6] << 16 | q[7] << 24);
}

// MAXT: most threads of a CTA.  0 is a warp for each row, in CTAs of kWarps.
template <int MAXT>
constexpr int max_threads() {
  return MAXT ? MAXT : kWarps * 32;
}

template <int VPT, int MAXT, int MODE>
__global__ void __launch_bounds__(max_threads<MAXT>()) norm_kernel(NormParams p) {
  constexpr bool WARP = MAXT == 0;
  __shared__ float buf[2 * 32];
  const int tpr = WARP ? 32 : blockDim.x;             // threads of a row
  const int me = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int nvec = p.H / 8;
  const int64_t step = (int64_t)gridDim.x * (WARP ? blockDim.x / 32 : 1);
  const float inv_h = 1.f / (float)p.H;
  int turn = 0;
  pdl_launch_dependents();
  pdl_wait();
  for (int64_t t = WARP ? (int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5)
                        : (int64_t)blockIdx.x;
       t < p.T; t += step) {
    uint4 xv[VPT], rv[VPT];
    float ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = me + i * tpr;
      xv[i] = rv[i] = make_uint4(0, 0, 0, 0);
      if (c < nvec) {
        xv[i] = ldg_stream(reinterpret_cast<const uint4 *>(p.x + t * p.H) + c);
        if (MODE == kPost || MODE == kPostNext)
          rv[i] = ldg_stream(reinterpret_cast<const uint4 *>(p.residual + t * p.H) + c);
      }
    }
    if (MODE == kQuant) {
      float am[1] = {0.f};
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float f[8];
        unpack8(xv[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) am[0] = fmaxf(am[0], fabsf(f[j]));
      }
      reduce_row<WARP, Max>(am, buf, turn);
      const float pre = am[0] > 1e30f ? 0x1p-64f : 1.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = me + i * tpr;
        float f[8];
        unpack8(xv[i], f);
        if (c < nvec)
          reinterpret_cast<uint2 *>(p.codes + t * p.H)[c] = codes8(f, pre, am[0] * pre);
      }
      if (me == 0) p.scales[t] = am[0] > 0.f ? __fdiv_rn(am[0], 127.f) : 1.f;
      continue;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float f[8];
      unpack8(xv[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss[0] = fmaf(f[j], f[j], ss[0]);
    }
    reduce_row<WARP, Sum>(ss, buf, turn);
    const float r = rsqrtf(fmaf(ss[0], inv_h, p.eps));
    if (MODE == kPre || MODE == kPreInt8) {
      float am[1] = {0.f};
      float y[VPT][8];
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = me + i * tpr;
        float w[8];
        unpack8(xv[i], y[i]);
        unpack8(c < nvec ? __ldg(reinterpret_cast<const uint4 *>(p.w) + c)
                         : make_uint4(0, 0, 0, 0), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          y[i][j] = y[i][j] * r * w[j];
          if (MODE == kPreInt8) am[0] = fmaxf(am[0], fabsf(y[i][j]));
        }
        if (MODE == kPre && c < nvec)
          reinterpret_cast<uint4 *>(p.out + t * p.H)[c] = pack8(y[i]);
      }
      if (MODE == kPreInt8) {
        reduce_row<WARP, Max>(am, buf, turn);
        const float pre = am[0] > 1e30f ? 0x1p-64f : 1.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int c = me + i * tpr;
          if (c < nvec)
            reinterpret_cast<uint2 *>(p.codes + t * p.H)[c] = codes8(y[i], pre, am[0] * pre);
        }
        if (me == 0) p.scales[t] = am[0] > 0.f ? __fdiv_rn(am[0], 127.f) : 1.f;
      }
    } else {
      float o[VPT][8];
      float s2[1] = {0.f};
      const __nv_bfloat16 *grow = p.gate ? p.gate + t * p.gt : nullptr;
      const float g1 = (grow && !p.gh) ? __bfloat162float(*grow) : 1.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = me + i * tpr;
        const bool in = c < nvec;
        float w[8], q[8], g[8];
        unpack8(xv[i], o[i]);
        unpack8(rv[i], q);
        unpack8(in ? __ldg(reinterpret_cast<const uint4 *>(p.w) + c) : make_uint4(0, 0, 0, 0), w);
        if (p.gh && in) {
          unpack8(__ldg(reinterpret_cast<const uint4 *>(grow) + c), g);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) g[j] = g1;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          o[i][j] = fmaf(g[j], o[i][j] * r * w[j], p.a * q[j]);
          if (MODE == kPostNext) s2[0] = fmaf(in ? o[i][j] : 0.f, o[i][j], s2[0]);
        }
        if (in) reinterpret_cast<uint4 *>(p.out + t * p.H)[c] = pack8(o[i]);
      }
      if (MODE == kPostNext) {
        reduce_row<WARP, Sum>(s2, buf, turn);
        const float r2 = rsqrtf(fmaf(s2[0], inv_h, p.eps));
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int c = me + i * tpr;
          if (c >= nvec) continue;
          float w[8];
          unpack8(__ldg(reinterpret_cast<const uint4 *>(p.w_next) + c), w);
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] *= o[i][j] * r2;
          reinterpret_cast<uint4 *>(p.next + t * p.H)[c] = pack8(w);
        }
      }
    }
  }
}

// ------------------------------------------------------------------ gradients
struct NormGradParams {
  const __nv_bfloat16 *d;      // [T, H]  gradient of the result
  const __nv_bfloat16 *x;      // [T, H]
  const __nv_bfloat16 *w;      // [H]
  const __nv_bfloat16 *gate;   // as in NormParams
  const __nv_bfloat16 *dskip;  // [T, H] added to dx, or null
  __nv_bfloat16 *dx;           // [T, H]
  __nv_bfloat16 *dres;         // [T, H] a * d, or null
  __nv_bfloat16 *dgate_el;     // [T, H] or [T, 1] gate gradient, or null
  float *part_w;               // [P, H] sums over a CTA's rows
  float *part_g;               // [P, H] of the channel gate's gradient, or [P] of a single one's
  int64_t T, gt;
  int H, gh;
  int sum_g;                   // 0: none, 1: [P, H] (gate [1, H]), 2: [P] (gate [1, 1])
  float eps, a;
};

template <int VPT, int MAXT>
__global__ void __launch_bounds__(max_threads<MAXT>()) norm_grad_kernel(NormGradParams p) {
  constexpr bool WARP = MAXT == 0;
  __shared__ float buf[2 * 32 * 2];
  extern __shared__ float acc_s[];   // WARP: [2][H] sums of the CTA's warps
  const int tpr = WARP ? 32 : blockDim.x;
  const int me = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int nvec = p.H / 8;
  const int64_t step = (int64_t)gridDim.x * (WARP ? blockDim.x / 32 : 1);
  const float inv_h = 1.f / (float)p.H;
  int turn = 0;
  float aw[VPT][8], ag[VPT][8], a1 = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) aw[i][j] = ag[i][j] = 0.f;
  pdl_launch_dependents();
  pdl_wait();
  for (int64_t t = WARP ? (int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5)
                        : (int64_t)blockIdx.x;
       t < p.T; t += step) {
    uint4 xv[VPT], dv[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = me + i * tpr;
      xv[i] = dv[i] = make_uint4(0, 0, 0, 0);
      if (c < nvec) {
        xv[i] = ldg_stream(reinterpret_cast<const uint4 *>(p.x + t * p.H) + c);
        dv[i] = ldg_stream(reinterpret_cast<const uint4 *>(p.d + t * p.H) + c);
      }
    }
    const __nv_bfloat16 *grow = p.gate ? p.gate + t * p.gt : nullptr;
    const float g1 = (grow && !p.gh) ? __bfloat162float(*grow) : 1.f;
    // s[0] = sum x^2, s[1] = sum d w x (times the gate where it has a value for each channel)
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = me + i * tpr;
      if (c >= nvec) continue;
      float x[8], d[8], w[8];
      unpack8(xv[i], x);
      unpack8(dv[i], d);
      unpack8(__ldg(reinterpret_cast<const uint4 *>(p.w) + c), w);
      if (p.gh) {
        float g[8];
        unpack8(__ldg(reinterpret_cast<const uint4 *>(grow) + c), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] *= g[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[0] = fmaf(x[j], x[j], s[0]);
        s[1] = fmaf(d[j] * w[j], x[j], s[1]);
      }
    }
    reduce_row<WARP, Sum>(s, buf, turn);
    const float r = rsqrtf(fmaf(s[0], inv_h, p.eps));
    const float m = r * s[1] * inv_h * g1;   // mean(dn n)
    if (grow && !p.gh) {
      if (p.sum_g == 2)
        a1 += r * s[1];
      else if (me == 0 && p.dgate_el)
        p.dgate_el[t] = __float2bfloat16_rn(r * s[1]);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = me + i * tpr;
      if (c >= nvec) continue;
      float x[8], d[8], w[8], g[8], o[8], e[8];
      unpack8(xv[i], x);
      unpack8(dv[i], d);
      unpack8(__ldg(reinterpret_cast<const uint4 *>(p.w) + c), w);
      if (p.gh) {
        unpack8(__ldg(reinterpret_cast<const uint4 *>(grow) + c), g);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = g1;
      }
      if (p.dskip) {
        unpack8(ldg_stream(reinterpret_cast<const uint4 *>(p.dskip + t * p.H) + c), o);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = x[j] * r;
        e[j] = d[j] * w[j] * n;
        aw[i][j] = fmaf(d[j] * g[j], n, aw[i][j]);
        if (p.sum_g == 1) ag[i][j] += e[j];
        o[j] += r * (d[j] * g[j] * w[j] - n * m);
      }
      reinterpret_cast<uint4 *>(p.dx + t * p.H)[c] = pack8(o);
      if (p.gh && p.dgate_el) reinterpret_cast<uint4 *>(p.dgate_el + t * p.H)[c] = pack8(e);
      if (p.dres) {
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] *= p.a;
        reinterpret_cast<uint4 *>(p.dres + t * p.H)[c] = pack8(d);
      }
    }
  }
  // this CTA's sums, always in the same order
  if (WARP) {
    const int warp = threadIdx.x >> 5;
    for (int w = 0; w < (int)(blockDim.x / 32); ++w) {
      if (warp == w) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int c = me + i * 32;
          if (c >= nvec) continue;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            acc_s[c * 8 + j] = w ? acc_s[c * 8 + j] + aw[i][j] : aw[i][j];
            if (p.sum_g == 1)
              acc_s[p.H + c * 8 + j] = w ? acc_s[p.H + c * 8 + j] + ag[i][j] : ag[i][j];
          }
        }
        if (me == 0) buf[0] = w ? buf[0] + a1 : a1;
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < p.H; c += blockDim.x) {
      p.part_w[(int64_t)blockIdx.x * p.H + c] = acc_s[c];
      if (p.sum_g == 1) p.part_g[(int64_t)blockIdx.x * p.H + c] = acc_s[p.H + c];
    }
    if (p.sum_g == 2 && threadIdx.x == 0) p.part_g[blockIdx.x] = buf[0];
  } else {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = me + i * tpr;
      if (c >= nvec) continue;
      float4 *o = reinterpret_cast<float4 *>(p.part_w + (int64_t)blockIdx.x * p.H + c * 8);
      o[0] = make_float4(aw[i][0], aw[i][1], aw[i][2], aw[i][3]);
      o[1] = make_float4(aw[i][4], aw[i][5], aw[i][6], aw[i][7]);
      if (p.sum_g == 1) {
        o = reinterpret_cast<float4 *>(p.part_g + (int64_t)blockIdx.x * p.H + c * 8);
        o[0] = make_float4(ag[i][0], ag[i][1], ag[i][2], ag[i][3]);
        o[1] = make_float4(ag[i][4], ag[i][5], ag[i][6], ag[i][7]);
      }
    }
    if (p.sum_g == 2 && threadIdx.x == 0) p.part_g[blockIdx.x] = a1;
  }
}

// Column sums of the CTAs' partial sums: 32 columns by 8 slices of the P rows a CTA, the
// slices added in order.  blockIdx.y 0: dweight, 1: the channel gate's gradient; the
// gradient of a single gate is one more column sum, of [P, 1].
__global__ void __launch_bounds__(256) norm_grad_sum_kernel(const float *part_w,
                                                            const float *part_g, int P, int H,
                                                            int gcols, __nv_bfloat16 *dw,
                                                            __nv_bfloat16 *dg) {
  __shared__ float s[8][32];
  const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
  const float *part = blockIdx.y ? part_g : part_w;
  __nv_bfloat16 *out = blockIdx.y ? dg : dw;
  const int cols = blockIdx.y ? gcols : H;
  const int c = blockIdx.x * 32 + lane;
  pdl_wait();
  float v = 0.f;
  if (c < cols) {
#pragma unroll 4
    for (int i = q; i < P; i += 8) v += part[(int64_t)i * cols + c];
  }
  s[q][lane] = v;
  __syncthreads();
  if (q == 0 && c < cols) {
#pragma unroll
    for (int k = 1; k < 8; ++k) v += s[k][lane];
    out[c] = __float2bfloat16_rn(v);
  }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// How a row of nvec vectors is spread over threads: a warp for short rows, else a CTA of
// ceil(nvec / vpt) threads, at most 256 of them where enough rows run at a time and the row
// fits (more registers for a thread), else at most 1024.
struct RowShape {
  int vpt, threads, maxt;
};
RowShape row_shape(int nvec, bool few_rows) {
  if (nvec <= kWarpRowVecs) return {(nvec + 31) / 32, kWarps * 32, 0};
  const int maxt = few_rows || nvec > 4 * 256 ? 1024 : 256;
  const int vpt = (nvec + maxt - 1) / maxt;
  return {vpt, (int)(ceil_div((nvec + vpt - 1) / vpt, 32) * 32), maxt};
}

// f(std::integral_constant<VPT>, std::integral_constant<MAXT>) for a row shape
template <typename F>
int with_shape(const RowShape &rs, F f) {
  auto vpt = [&](auto maxt) {
    switch (rs.vpt) {
      case 1: return f(std::integral_constant<int, 1>(), maxt);
      case 2: return f(std::integral_constant<int, 2>(), maxt);
      case 3: return f(std::integral_constant<int, 3>(), maxt);
      default: return f(std::integral_constant<int, 4>(), maxt);
    }
  };
  if (rs.maxt == 0) return vpt(std::integral_constant<int, 0>());
  if (rs.maxt == 256) return vpt(std::integral_constant<int, 256>());
  return vpt(std::integral_constant<int, 1024>());
}

template <int MODE>
int launch_norm(const NormParams &p, cudaStream_t s) {
  const RowShape rs = row_shape(p.H / 8, p.T < num_sms());
  const int64_t ctas = rs.maxt ? p.T : ceil_div(p.T, kWarps);
  const dim3 grid((unsigned)std::min<int64_t>(ctas, (int64_t)1 << 30));
  return with_shape(rs, [&](auto vpt, auto maxt) {
    return launch_pdl(norm_kernel<vpt(), maxt(), MODE>, grid, dim3(rs.threads), 0, s, p);
  });
}

constexpr int kGradCtasPerSm = 2;
int grad_ctas(int64_t T, int64_t H) {
  const int64_t per = H / 8 <= kWarpRowVecs ? kWarps : 1;
  return (int)std::max<int64_t>(
      1, std::min<int64_t>(ceil_div(T, per), (int64_t)num_sms() * kGradCtasPerSm));
}
size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

int run_grad(NormGradParams &p, __nv_bfloat16 *dw, __nv_bfloat16 *dg_sum, void *ws,
             cudaStream_t s) {
  const int P = grad_ctas(p.T, p.H);
  p.part_w = static_cast<float *>(ws);
  p.part_g = reinterpret_cast<float *>(static_cast<char *>(ws) + align256((size_t)P * p.H * 4));
  const RowShape rs = row_shape(p.H / 8, p.T < num_sms());
  const size_t smem = rs.maxt ? 0 : (size_t)p.H * 8;   // at most 8 KB
  const int st = with_shape(rs, [&](auto vpt, auto maxt) {
    return launch_pdl(norm_grad_kernel<vpt(), maxt()>, dim3(P), dim3(rs.threads), smem, s, p);
  });
  if (st) return st;
  const dim3 grid((unsigned)ceil_div(p.H, 32), p.sum_g ? 2 : 1);
  return launch_pdl(norm_grad_sum_kernel, grid, dim3(256), 0, s, (const float *)p.part_w,
                    (const float *)p.part_g, P, p.H, p.sum_g == 2 ? 1 : p.H, dw, dg_sum);
}

int zero(void *p, size_t bytes, cudaStream_t s) {
  const cudaError_t e = cudaMemsetAsync(p, 0, bytes, s);
  if (e == cudaSuccess) return NVFP4_OK;
  set_last_cuda_error(e);
  return NVFP4_ECUDA;
}

// Checks every norm call shares.  Pointers of T-row arrays may be null when T is 0.
int check_rows(int64_t T, int64_t H, float eps) {
  if (T < 0 || H <= 0 || !(eps > 0.f) || !(eps < 1e30f)) return NVFP4_EINVAL;
  if (H % 8 || H > kMaxH || T > (int64_t(1) << 40) / H) return NVFP4_ESHAPE;
  return NVFP4_OK;
}
int check_gate(const __nv_bfloat16 *gate, int64_t T, int64_t H, int64_t gate_rows,
               int64_t gate_cols, NormParams *p) {
  p->gate = nullptr;
  p->gt = 0;
  p->gh = 0;
  if (!gate && !gate_rows && !gate_cols) return NVFP4_OK;
  if ((gate_rows != 1 && gate_rows != T) || (gate_cols != 1 && gate_cols != H) ||
      (!gate && gate_rows > 0))
    return NVFP4_EINVAL;
  if (reinterpret_cast<uintptr_t>(gate) & (gate_cols == H ? 15 : 1)) return NVFP4_EINVAL;
  p->gate = gate;
  p->gh = gate_cols == H ? 1 : 0;   // H >= 8, so one column is never H
  p->gt = gate_rows == 1 ? 0 : gate_cols;
  return NVFP4_OK;
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" int moe_nvfp4_pre_norm(const __nv_bfloat16 *x, const __nv_bfloat16 *weight, int64_t T,
                                  int64_t H, float eps, __nv_bfloat16 *out,
                                  cudaStream_t stream) {
  if (int st = check_rows(T, H, eps)) return st;
  if (!weight || !aligned16(weight)) return NVFP4_EINVAL;
  if (T == 0) return NVFP4_OK;
  if (!x || !out || !aligned16(x) || !aligned16(out)) return NVFP4_EINVAL;
  NormParams p = {};
  p.x = x, p.w = weight, p.out = out, p.T = T, p.H = (int)H, p.eps = eps;
  return launch_norm<kPre>(p, stream);
}

extern "C" int moe_nvfp4_pre_norm_int8(const __nv_bfloat16 *x, const __nv_bfloat16 *weight,
                                       int64_t T, int64_t H, float eps, int8_t *codes,
                                       float *scales, cudaStream_t stream) {
  if (int st = check_rows(T, H, eps)) return st;
  if (H % 16) return NVFP4_ESHAPE;
  if (!weight || !aligned16(weight)) return NVFP4_EINVAL;
  if (T == 0) return NVFP4_OK;
  if (!x || !codes || !scales || !aligned16(x) || !aligned16(codes) ||
      (reinterpret_cast<uintptr_t>(scales) & 3))
    return NVFP4_EINVAL;
  NormParams p = {};
  p.x = x, p.w = weight, p.codes = codes, p.scales = scales, p.T = T, p.H = (int)H, p.eps = eps;
  return launch_norm<kPreInt8>(p, stream);
}

extern "C" int nvfp4_int8_quantize(const __nv_bfloat16 *x, int64_t rows, int64_t cols,
                                   int8_t *codes, float *scales, cudaStream_t stream) {
  if (rows < 0 || cols <= 0) return NVFP4_EINVAL;
  if (cols % 16 || cols > kMaxH || rows > (int64_t(1) << 40) / cols) return NVFP4_ESHAPE;
  if (rows == 0) return NVFP4_OK;
  if (!x || !codes || !scales || !aligned16(x) || !aligned16(codes) ||
      (reinterpret_cast<uintptr_t>(scales) & 3))
    return NVFP4_EINVAL;
  NormParams p = {};
  p.x = x, p.codes = codes, p.scales = scales, p.T = rows, p.H = (int)cols;
  return launch_norm<kQuant>(p, stream);
}

extern "C" int moe_nvfp4_post_norm(const __nv_bfloat16 *y, const __nv_bfloat16 *weight,
                                   const __nv_bfloat16 *residual, const __nv_bfloat16 *gate,
                                   int64_t T, int64_t H, int64_t gate_rows, int64_t gate_cols,
                                   float eps, float residual_scale,
                                   const __nv_bfloat16 *next_weight, __nv_bfloat16 *out,
                                   __nv_bfloat16 *next, cudaStream_t stream) {
  if (int st = check_rows(T, H, eps)) return st;
  NormParams p = {};
  if (int st = check_gate(gate, T, H, gate_rows, gate_cols, &p)) return st;
  if (!weight || !aligned16(weight) || !aligned16(next_weight)) return NVFP4_EINVAL;
  if (T == 0) return NVFP4_OK;
  if (!y || !residual || !out || !aligned16(y) || !aligned16(residual) || !aligned16(out) ||
      (next_weight != nullptr) != (next != nullptr) || !aligned16(next))
    return NVFP4_EINVAL;
  p.x = y, p.w = weight, p.residual = residual, p.w_next = next_weight, p.out = out;
  p.next = next, p.T = T, p.H = (int)H, p.eps = eps, p.a = residual_scale;
  return next ? launch_norm<kPostNext>(p, stream) : launch_norm<kPost>(p, stream);
}

extern "C" size_t moe_nvfp4_norm_backward_workspace_size(int64_t T, int64_t H) {
  if (T < 0 || H <= 0) return 0;
  return 2 * align256((size_t)grad_ctas(T, H) * (size_t)H * 4);
}

extern "C" int moe_nvfp4_pre_norm_backward(const __nv_bfloat16 *dy, const __nv_bfloat16 *x,
                                           const __nv_bfloat16 *weight,
                                           const __nv_bfloat16 *dskip, int64_t T, int64_t H,
                                           float eps, __nv_bfloat16 *dx, __nv_bfloat16 *dweight,
                                           void *workspace, size_t ws_bytes,
                                           cudaStream_t stream) {
  if (int st = check_rows(T, H, eps)) return st;
  if (!weight || !dweight || !aligned16(weight) || !aligned16(dweight)) return NVFP4_EINVAL;
  if (T == 0) return zero(dweight, (size_t)H * 2, stream);
  if (!dy || !x || !dx || !aligned16(dy) || !aligned16(x) || !aligned16(dx) || !aligned16(dskip))
    return NVFP4_EINVAL;
  if (!workspace || !aligned16(workspace) ||
      ws_bytes < moe_nvfp4_norm_backward_workspace_size(T, H))
    return NVFP4_EWORKSPACE;
  NormGradParams p = {};
  p.d = dy, p.x = x, p.w = weight, p.dskip = dskip, p.dx = dx, p.T = T, p.H = (int)H;
  p.eps = eps;
  return run_grad(p, dweight, nullptr, workspace, stream);
}

extern "C" int moe_nvfp4_post_norm_backward(
    const __nv_bfloat16 *dout, const __nv_bfloat16 *y, const __nv_bfloat16 *weight,
    const __nv_bfloat16 *gate, int64_t T, int64_t H, int64_t gate_rows, int64_t gate_cols,
    float eps, float residual_scale, __nv_bfloat16 *dy, __nv_bfloat16 *dweight,
    __nv_bfloat16 *dgate, __nv_bfloat16 *dresidual, void *workspace, size_t ws_bytes,
    cudaStream_t stream) {
  if (int st = check_rows(T, H, eps)) return st;
  NormParams g = {};
  if (int st = check_gate(gate, T, H, gate_rows, gate_cols, &g)) return st;
  if (!weight || !dweight || !aligned16(weight) || !aligned16(dweight)) return NVFP4_EINVAL;
  if ((reinterpret_cast<uintptr_t>(dgate) & (gate_cols == H ? 15 : 1)) ||
      (gate && gate_rows == 1 && !dgate) || (!gate && dgate))
    return NVFP4_EINVAL;
  if (T == 0) {
    if (int st = zero(dweight, (size_t)H * 2, stream)) return st;
    return gate_rows == 1 ? zero(dgate, (size_t)gate_cols * 2, stream) : NVFP4_OK;
  }
  if (!dout || !y || !dy || (gate && !dgate) || !aligned16(dout) || !aligned16(y) ||
      !aligned16(dy) || !aligned16(dresidual))
    return NVFP4_EINVAL;
  if (!workspace || !aligned16(workspace) ||
      ws_bytes < moe_nvfp4_norm_backward_workspace_size(T, H))
    return NVFP4_EWORKSPACE;
  NormGradParams p = {};
  p.d = dout, p.x = y, p.w = weight, p.gate = g.gate, p.dx = dy, p.dres = dresidual;
  p.T = T, p.gt = g.gt, p.gh = g.gh, p.H = (int)H, p.eps = eps, p.a = residual_scale;
  p.sum_g = gate && gate_rows == 1 ? (gate_cols == H ? 1 : 2) : 0;
  p.dgate_el = gate && gate_rows != 1 ? dgate : nullptr;
  return run_grad(p, dweight, p.sum_g ? dgate : nullptr, workspace, stream);
}
