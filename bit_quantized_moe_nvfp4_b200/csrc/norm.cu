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
// A row is read once and each output written once.  A row of at most 1536 values belongs to a
// warp (no barrier); a longer one to a CTA.  CTAs are persistent.  Each thread copies the 16-byte
// vectors that it will itself need of its rows into shared memory (cp.async).  Where two rows of
// all arrays fit the CTA's share of shared memory that is done a row ahead, so loads stay in
// flight through the reductions and stores of the present row, without registers or barriers for
// it: with one or two arrays up to 24576 values a row.  With three (dskip, or a gate for each
// value) only some widths have the room; neither 1032 nor 6144 does, and a row's loads start when
// the row before has left its slots.
// Long rows of one and two arrays are bound by HBM.  Captured in a graph: post_norm with next,
// 16384 x 6144 and a channel gate, 137 us (805 MB, 5.9 TB/s); pre_norm 4096 x 6144, 17.7 us
// (101 MB, 5.7 TB/s); gradients 4096 x 6144, with the 6 to 7 us of their column sums: no gate 41,
// token gate 42 (201 MB, 4.8 TB/s), channel gate 50 (two CTAs an SM), full gate 56 (302 MB),
// pre_norm's 36, with dskip 41.  The quantizer is near its issue limit (4096 x 6144, 15.5 us, 75
// MB, issue slots 75% busy); short rows wait for memory (gradients with dskip of 8191 x 1032: 18
// us for 68 MB, issue slots 46% busy, nothing in flight ahead).
// All statistics and sums are fp32; each result is rounded once.  next is taken from the
// unrounded out, and codes from the unrounded y.
#include <algorithm>
#include <type_traits>

#include "moe.cuh"

namespace nvfp4 {
namespace {

constexpr int64_t kMaxH = 32768;   // 4 vectors of 8 values for each of 1024 threads
constexpr int kWarpRowVecs = 192;  // rows of up to 192 vectors (1536 values) take a warp
constexpr int kWarps = 8;          // warps of a CTA whose warps take a row each

enum { kPre = 0, kPreInt8 = 1, kPost = 2, kPostNext = 3, kQuant = 4 };

struct NormParams {
  const __nv_bfloat16 *w;         // [H]
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

// Pairs of fp32 values: one instruction for both (fma, mul, add .f32x2), rounded as two.
__device__ __forceinline__ uint64_t f2_bits(float2 a) {
  return (uint64_t)__float_as_uint(a.x) | (uint64_t)__float_as_uint(a.y) << 32;
}
__device__ __forceinline__ float2 f2_from(uint64_t v) {
  return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)), "l"(f2_bits(c)));
  return f2_from(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
  return f2_from(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
  return f2_from(r);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// 8 bf16 values <-> 4 pairs of fp32
__device__ __forceinline__ void unpack8(uint4 v, float2 (&f)[4]) {
  f[0] = make_float2(bf16_lo(v.x), bf16_hi(v.x)), f[1] = make_float2(bf16_lo(v.y), bf16_hi(v.y));
  f[2] = make_float2(bf16_lo(v.z), bf16_hi(v.z)), f[3] = make_float2(bf16_lo(v.w), bf16_hi(v.w));
}
__device__ __forceinline__ uint4 pack8(const float2 (&f)[4]) {
  return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y),
                    pack_bf16x2(f[2].x, f[2].y), pack_bf16x2(f[3].x, f[3].y));
}
// Weights and gates too are read by ordinary loads: the kernel before may write them while this
// one is already resident, and of one row an output may be the gate's tensor.
__device__ __forceinline__ uint4 ld8(const __nv_bfloat16 *p, int c) {
  return reinterpret_cast<const uint4 *>(p)[c];
}
__device__ __forceinline__ void stg8(__nv_bfloat16 *p, int c, const float2 (&f)[4]) {
  reinterpret_cast<uint4 *>(p)[c] = pack8(f);
}

struct Sum {
  static __device__ __forceinline__ float op(float a, float b) { return a + b; }
};
// The larger of two magnitudes.  Without a sign bit floats are ordered as their bits are, with
// infinity and then NaN above all numbers: a row's NaN reaches its maximum.
struct Max {
  static __device__ __forceinline__ float op(float a, float b) {
    return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
  }
};
__device__ __forceinline__ float magnitude(float v) {
  return __uint_as_float(__float_as_uint(v) & 0x7FFFFFFFu);
}

// Reduce N values over the threads that share a row: a warp, or the CTA through `buf`
// ([2][N][32]; the half alternates with `turn`, so one barrier a reduction is enough).  Both
// operations have 0 for the warps that a CTA lacks (a maximum is one of magnitudes).
template <bool WARP, typename Op, int N>
__device__ __forceinline__ void reduce_row(float (&v)[N], float *buf, int &turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = Op::op(v[k], __shfl_xor_sync(0xFFFFFFFFu, v[k], o));
  if (WARP) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = (int)(blockDim.x + 127) >> 7;
  float *b = buf + turn * 32 * N;
  turn ^= 1;
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) b[k * 32 + warp] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    float s = 0.f;
    for (int w = 0; w < nw; ++w) {
      const float4 q = reinterpret_cast<const float4 *>(b + k * 32)[w];
      s = Op::op(s, Op::op(Op::op(q.x, q.y), Op::op(q.z, q.w)));
    }
    v[k] = s;
  }
}
// Before the first reduction of a CTA: the places of warps that it lacks.
template <bool WARP, int N>
__device__ __forceinline__ void clear_reduce(float (&buf)[N]) {
  if constexpr (!WARP) {
    for (int k = threadIdx.x; k < N; k += blockDim.x) buf[k] = 0.f;
    __syncthreads();
  }
}

// Codes of 8 values: the integers nearest to 127 y / amax, ties to even, without a division
// for each.  With inv = fl(127 / amax), v = fl(y inv) is off by at most 2^-23 relative; adding
// 1.5 2^23 rounds it to the integer, whose low byte is then the code.
// BF16: where y and amax are bf16 values, a quotient of 127 p / q with p, q < 2^8 (their
// significands) and a power of two is either a tie (k + 1/2, at most 9 bits) or at least 2^-16
// relative away from one.  So v rounded to 18 significant bits (in its bit pattern) first is the
// tie itself where there is one and stays on its side otherwise, and the code is the real
// quotient's.  Other values can lie next to a tie, where that step would move them onto it: they
// are rounded once, as they are.
template <bool BF16>
__device__ __forceinline__ uint32_t code_bits(float v) {
  if (BF16) v = __uint_as_float((__float_as_uint(v) + 32u) & ~63u);
  return __float_as_uint(v + 12582912.f);
}
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
template <bool BF16>
__device__ __forceinline__ uint2 codes8(const float2 (&y)[4], float inv) {
  uint32_t q[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 v = mul2(y[j], both(inv));
    q[2 * j] = code_bits<BF16>(v.x);
    q[2 * j + 1] = code_bits<BF16>(v.y);
  }
  return make_uint2(low_bytes(q[0], q[1], q[2], q[3]), low_bytes(q[4], q[5], q[6], q[7]));
}
// Power of two that brings a row of this amax to where 127 / amax neither overflows nor
// underflows, that quotient, and the scale of the row.
__device__ __forceinline__ float code_range(float amax) {
  return amax > 0x1p60f ? 0x1p-64f : amax < 0x1p-60f ? 0x1p+76f : 1.f;
}
__device__ __forceinline__ float code_inverse(float amax, float pre) {
  return amax > 0.f ? __fdiv_rn(127.f, amax * pre) : 0.f;
}
// NaN for a row with NaN or an infinity, whose codes (integers) cannot say so.
__device__ __forceinline__ float code_scale(float amax) {
  if (!(amax < __int_as_float(0x7F800000))) return __int_as_float(0x7FC00000);
  return amax > 0.f ? __fdiv_rn(amax, 127.f) : 1.f;
}

// CTAs that an SM holds: registers and shared memory are shared out for so many.  Of 256
// threads three, against two or four: post_norm with next of 16384 x 6144, 140 us against 161
// and 144; gradients of 4096 x 6144, 45 us against 52 (with a channel gate's column sums in
// registers too, or four vectors a thread, two fit).  Gradients of short rows: the fewer CTAs
// the fewer partial sums to add (forward and backward of 8191 x 1032: 30.7 us with 2 CTAs of 8
// warps, 33.3 with 4 of 4).
constexpr int row_ctas(int maxt) { return maxt == 1024 ? 1 : 3; }
constexpr int grad_row_ctas(int maxt, int vpt, bool sum_g) {
  if (maxt == 1024) return 1;
  if (!maxt) return vpt <= 2 && !sum_g ? 3 : 2;
  return vpt == 1 ? 4 : vpt == 4 || (vpt == 3 && sum_g) ? 2 : 3;
}

// MAXT: most threads of a CTA.  0 is a warp for each row, in CTAs of kWarps.
template <int MAXT>
constexpr int max_threads() {
  return MAXT ? MAXT : kWarps * 32;
}

// ------------------------------------------------------------------ rows ahead
// Rows in flight for each CTA or warp.  Two against four: 4096 x 2048 post_norm with next 14.8 us
// against 16.5 (more CTAs fit), longer rows the same; one: 18.4.
constexpr int kMaxStages = 2;
constexpr int kMaxArrays = 3;

// The row arrays a kernel streams (bf16, H values a row).
struct RowArrays {
  const __nv_bfloat16 *p[kMaxArrays];
  int n, stages;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Wait until at most `pending` of this thread's copy groups are in flight.
__device__ __forceinline__ void cp_async_wait(int pending) {
  static_assert(kMaxStages <= 2, "one case for each number of groups that may be pending");
  if (pending == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// A thread's own slots: [stage][array][i] vectors, `pitch` bytes (16 a thread) apart.
template <int VPT>
struct RowFeed {
  const RowArrays &a;
  uint32_t base;
  int me, tpr, nvec, pitch;
  int64_t T, row_bytes;

  __device__ __forceinline__ uint32_t stage_at(int stage) const {
    return base + (uint32_t)(stage * a.n * VPT * pitch);
  }
  __device__ __forceinline__ bool in(int i) const { return me + i * tpr < nvec; }
  __device__ __forceinline__ void fetch(int64_t t, uint32_t at) const {
    if (t < T) {
      const int64_t off = t * row_bytes + me * 16;
#pragma unroll
      for (int k = 0; k < kMaxArrays; ++k) {
        if (k >= a.n) break;
        const char *src = reinterpret_cast<const char *>(a.p[k]) + off;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
          if (in(i)) cp_async16(at + (k * VPT + i) * pitch, src + i * tpr * 16);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // Vector i of array `arr` (only where in(i)).
  __device__ __forceinline__ uint4 get(uint32_t at, int arr, int i) const {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at + (arr * VPT + i) * pitch)
                 : "memory");
    return v;
  }
};

extern __shared__ __align__(16) unsigned char dyn_smem[];

template <int VPT, int MAXT>
__device__ __forceinline__ RowFeed<VPT> make_feed(const RowArrays &a, int64_t T, int64_t H) {
  const int tpr = MAXT ? blockDim.x : 32;
  return {a, (uint32_t)__cvta_generic_to_shared(dyn_smem) + threadIdx.x * 16,
          (int)(MAXT ? threadIdx.x : threadIdx.x & 31), tpr, (int)(H / 8), (int)blockDim.x * 16,
          T, H * 2};
}

template <int VPT, int MAXT, int MODE>
__global__ void __launch_bounds__(max_threads<MAXT>(), row_ctas(MAXT))
    norm_kernel(const __grid_constant__ NormParams p, const __grid_constant__ RowArrays rows) {
  constexpr bool WARP = MAXT == 0;
  __shared__ __align__(16) float buf[2 * 32];
  const RowFeed<VPT> feed = make_feed<VPT, MAXT>(rows, p.T, p.H);
  const int me = feed.me, tpr = feed.tpr;
  const int64_t step = (int64_t)gridDim.x * (WARP ? kWarps : 1);
  const int64_t t0 =
      WARP ? (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  const float inv_h = 1.f / (float)p.H;
  int turn = 0, stage = 0;
  clear_reduce<WARP>(buf);
  pdl_launch_dependents();
  pdl_wait();
  for (int k = 0; k < rows.stages; ++k) feed.fetch(t0 + k * step, feed.stage_at(k));
  for (int64_t t = t0; t < p.T; t += step) {
    cp_async_wait(rows.stages - 1);
    const uint32_t at = feed.stage_at(stage);
    float r = 1.f;
    if constexpr (MODE != kQuant) {
      float2 sq = both(0.f);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if (!feed.in(i)) continue;
        float2 x[4];
        unpack8(feed.get(at, 0, i), x);
#pragma unroll
        for (int j = 0; j < 4; ++j) sq = fma2(x[j], x[j], sq);
      }
      float ss[1] = {sq.x + sq.y};
      reduce_row<WARP, Sum>(ss, buf, turn);
      r = rsqrtf(fmaf(ss[0], inv_h, p.eps));
    }
    if constexpr (MODE == kPre) {
      __nv_bfloat16 *out = p.out + t * p.H;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if (!feed.in(i)) continue;
        const int c = me + i * tpr;
        float2 y[4], w[4];
        unpack8(feed.get(at, 0, i), y);
        unpack8(ld8(p.w, c), w);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = mul2(mul2(y[j], both(r)), w[j]);
        stg8(out, c, y);
      }
    } else if constexpr (MODE == kPreInt8 || MODE == kQuant) {
      float am[1] = {0.f};
      uint4 xv[MODE == kQuant ? VPT : 1];
      float2 y[MODE == kPreInt8 ? VPT : 1][4];
      if constexpr (MODE == kPreInt8) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          if (!feed.in(i)) continue;
          float2 w[4];
          unpack8(feed.get(at, 0, i), y[i]);
          unpack8(ld8(p.w, me + i * tpr), w);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            y[i][j] = mul2(mul2(y[i][j], both(r)), w[j]);
            am[0] = Max::op(am[0], Max::op(magnitude(y[i][j].x), magnitude(y[i][j].y)));
          }
        }
      } else {   // the largest of two bf16 at a time, exact
        __nv_bfloat162 m = __float2bfloat162_rn(0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          if (!feed.in(i)) continue;
          xv[i] = feed.get(at, 0, i);
          const uint32_t u[4] = {xv[i].x, xv[i].y, xv[i].z, xv[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&u[j])));
        }
        am[0] = Max::op(magnitude(__low2float(m)), magnitude(__high2float(m)));
      }
      reduce_row<WARP, Max>(am, buf, turn);
      const float pre = code_range(am[0]), inv = code_inverse(am[0], pre);
      uint2 *out = reinterpret_cast<uint2 *>(p.codes + t * p.H);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if (!feed.in(i)) continue;
        const int k = MODE == kPreInt8 ? i : 0;
        if (MODE == kQuant) unpack8(xv[MODE == kQuant ? i : 0], y[k]);
        if (pre != 1.f)
#pragma unroll
          for (int j = 0; j < 4; ++j) y[k][j] = mul2(y[k][j], both(pre));
        out[me + i * tpr] = codes8<MODE == kQuant>(y[k], inv);
      }
      if (me == 0) p.scales[t] = code_scale(am[0]);
    } else {
      float2 o[VPT][4];
      float2 sq = both(0.f);
      const float g1 = (p.gate && !p.gh) ? __bfloat162float(p.gate[t * p.gt]) : 1.f;
      const float rg = p.gh ? r : r * g1;   // a row's single gate goes with its norm
      __nv_bfloat16 *out = p.out + t * p.H;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if (!feed.in(i)) continue;
        const int c = me + i * tpr;
        float2 w[4], q[4];
        unpack8(feed.get(at, 0, i), o[i]);
        unpack8(feed.get(at, 1, i), q);
        unpack8(ld8(p.w, c), w);
        if (p.gh) {   // a gate for each value is a third row array
          float2 g[4];
          unpack8(p.gt ? feed.get(at, 2, i) : ld8(p.gate, c), g);
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = mul2(w[j], g[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          o[i][j] = fma2(mul2(o[i][j], both(rg)), w[j], mul2(both(p.a), q[j]));
          if (MODE == kPostNext) sq = fma2(o[i][j], o[i][j], sq);
        }
        stg8(out, c, o[i]);
      }
      if constexpr (MODE == kPostNext) {
        float s2[1] = {sq.x + sq.y};
        reduce_row<WARP, Sum>(s2, buf, turn);
        const float r2 = rsqrtf(fmaf(s2[0], inv_h, p.eps));
        out = p.next + t * p.H;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          if (!feed.in(i)) continue;
          const int c = me + i * tpr;
          float2 w[4];
          unpack8(ld8(p.w_next, c), w);
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = mul2(w[j], mul2(o[i][j], both(r2)));
          stg8(out, c, w);
        }
      }
    }
    feed.fetch(t + rows.stages * step, at);   // this thread has used its slots
    stage = stage + 1 == rows.stages ? 0 : stage + 1;
  }
}

// ------------------------------------------------------------------ gradients
struct NormGradParams {
  const __nv_bfloat16 *w;      // [H]
  const __nv_bfloat16 *gate;   // as in NormParams
  __nv_bfloat16 *dx;           // [T, H]
  __nv_bfloat16 *dres;         // [T, H] a * d, or null
  __nv_bfloat16 *dgate_el;     // [T, H] or [T, 1] gate gradient, or null
  float *part_w;               // [P, H] sums over a CTA's rows
  float *part_g;               // [P, H] of the channel gate's gradient, or [P] of a single one's
  int64_t T, gt;               // gt, gh: as in NormParams
  int H, gh;
  int sum_g;                   // 0: none, 1: [P, H] (gate [1, H]), 2: [P] (gate [1, 1])
  int skip;                    // the third row array is dskip
  float eps, a;
};

// What the gate is: none, one for a row ([T, 1], [1, 1]), one for a channel ([1, H]: its
// gradient is a column sum), one for each value.
enum { kNoGate = 0, kRowGate = 1, kChannelGate = 2, kFullGate = 3 };

// Row arrays: x, the gradient of the result, then dskip and the gate where there are any.
template <int VPT, int MAXT, int GATE>
__global__ void __launch_bounds__(max_threads<MAXT>(), grad_row_ctas(MAXT, VPT, GATE == kChannelGate))
    norm_grad_kernel(const __grid_constant__ NormGradParams p,
                     const __grid_constant__ RowArrays rows) {
  constexpr bool WARP = MAXT == 0, SUMG = GATE == kChannelGate;
  __shared__ __align__(16) float buf[2 * 32 * 2];
  const RowFeed<VPT> feed = make_feed<VPT, MAXT>(rows, p.T, p.H);
  const int me = feed.me, tpr = feed.tpr, nvec = feed.nvec;
  const int64_t step = (int64_t)gridDim.x * (WARP ? kWarps : 1);
  const int64_t t0 =
      WARP ? (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  const float inv_h = 1.f / (float)p.H;
  int turn = 0, stage = 0;
  clear_reduce<WARP>(buf);
  float2 aw[VPT][4], ag[SUMG ? VPT : 1][4];
  float a1 = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      aw[i][j] = both(0.f);
      if (SUMG) ag[i][j] = both(0.f);
    }
  pdl_launch_dependents();
  pdl_wait();
  for (int k = 0; k < rows.stages; ++k) feed.fetch(t0 + k * step, feed.stage_at(k));
  for (int64_t t = t0; t < p.T; t += step) {
    cp_async_wait(rows.stages - 1);
    const uint32_t at = feed.stage_at(stage);
    // read before the reduction: its gradient may be written over it after
    const float g1 = GATE == kRowGate ? __bfloat162float(p.gate[t * p.gt]) : 1.f;
    // sums of x^2, and of d w x (times the gate where it has a value for each channel)
    float2 sx = both(0.f), sd = both(0.f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (!feed.in(i)) continue;
      const int c = me + i * tpr;
      float2 x[4], d[4], w[4];
      unpack8(feed.get(at, 0, i), x);
      unpack8(feed.get(at, 1, i), d);
      unpack8(ld8(p.w, c), w);
      if (GATE >= kChannelGate) {
        float2 g[4];
        unpack8(GATE == kFullGate ? feed.get(at, 2, i) : ld8(p.gate, c), g);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = mul2(w[j], g[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sx = fma2(x[j], x[j], sx);
        sd = fma2(mul2(d[j], w[j]), x[j], sd);
      }
    }
    float s[2] = {sx.x + sx.y, sd.x + sd.y};
    reduce_row<WARP, Sum>(s, buf, turn);
    const float r = rsqrtf(fmaf(s[0], inv_h, p.eps));
    const float rg = r * g1;
    // dx = r dn - r mean(dn n) n; both terms carry the row's single gate, the second in x rg.
    // No product here holds r^2 alone, which leaves fp32 at the smallest eps.
    const float rm = r * (r * s[1] * inv_h);
    if (GATE == kRowGate) {
      if (p.sum_g == 2)
        a1 += r * s[1];
      else if (me == 0)
        p.dgate_el[t] = __float2bfloat16_rn(r * s[1]);
    }
    const int64_t row = t * p.H;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (!feed.in(i)) continue;
      const int c = me + i * tpr;
      float2 x[4], d[4], w[4], o[4];
      unpack8(feed.get(at, 0, i), x);   // read again: registers hold the column sums
      unpack8(feed.get(at, 1, i), d);
      unpack8(ld8(p.w, c), w);
      float2 g[4];   // before the stores: of one row, any output may be the gate's tensor
      if (GATE >= kChannelGate)
        unpack8(GATE == kFullGate ? feed.get(at, 2, i) : ld8(p.gate, c), g);
      if (p.dres) {
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = mul2(d[j], both(p.a));
        stg8(p.dres + row, c, o);
      }
      float2 n[4];   // x r, and the row's single gate (dweight = sum d g n)
#pragma unroll
      for (int j = 0; j < 4; ++j) n[j] = mul2(x[j], both(rg));
      if (GATE >= kChannelGate) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 dw = mul2(d[j], w[j]);
          d[j] = mul2(d[j], g[j]);
          if (SUMG) ag[i][j] = fma2(dw, n[j], ag[i][j]);
          if (GATE == kFullGate) o[j] = mul2(dw, n[j]);
        }
        if (GATE == kFullGate) stg8(p.dgate_el + row, c, o);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) aw[i][j] = fma2(d[j], n[j], aw[i][j]);
      if (p.skip) {
        unpack8(feed.get(at, 2, i), o);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = fma2(mul2(d[j], w[j]), both(rg), o[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = mul2(mul2(d[j], w[j]), both(rg));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = fma2(n[j], both(-rm), o[j]);
      stg8(p.dx + row, c, o);
    }
    feed.fetch(t + rows.stages * step, at);
    stage = stage + 1 == rows.stages ? 0 : stage + 1;
  }
  // this CTA's sums, always in the same order
  if (WARP) {
    // each warp's sums as [i][j][lane] pairs in the slots, which are empty now, then their total
    constexpr int kPart = VPT * 4 * 32;   // pairs of one warp
    float2 *acc = reinterpret_cast<float2 *>(dyn_smem);
    const int warp = threadIdx.x >> 5;
    cp_async_wait(0);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[warp * kPart + (i * 4 + j) * 32 + me] = aw[i][j];
        if (SUMG) acc[(kWarps + warp) * kPart + (i * 4 + j) * 32 + me] = ag[i][j];
      }
    if (me == 0) buf[warp] = a1;
    __syncthreads();
    for (int e = threadIdx.x; e < kPart; e += blockDim.x) {
      const int at = ((e >> 7) * 32 + (e & 31)) * 8 + ((e >> 5) & 3) * 2;   // column of the pair
      if (at >= p.H) continue;
#pragma unroll
      for (int k = 0; k < (SUMG ? 2 : 1); ++k) {
        float2 v = acc[k * kWarps * kPart + e];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) v = add2(v, acc[(k * kWarps + w) * kPart + e]);
        *reinterpret_cast<float2 *>((k ? p.part_g : p.part_w) + (int64_t)blockIdx.x * p.H + at) = v;
      }
    }
    if (p.sum_g == 2 && threadIdx.x == 0) {
      float v = buf[0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) v += buf[w];
      p.part_g[blockIdx.x] = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = me + i * tpr;
      if (c >= nvec) continue;
      float4 *o = reinterpret_cast<float4 *>(p.part_w + (int64_t)blockIdx.x * p.H + c * 8);
      o[0] = make_float4(aw[i][0].x, aw[i][0].y, aw[i][1].x, aw[i][1].y);
      o[1] = make_float4(aw[i][2].x, aw[i][2].y, aw[i][3].x, aw[i][3].y);
      if (SUMG) {
        o = reinterpret_cast<float4 *>(p.part_g + (int64_t)blockIdx.x * p.H + c * 8);
        o[0] = make_float4(ag[i][0].x, ag[i][0].y, ag[i][1].x, ag[i][1].y);
        o[1] = make_float4(ag[i][2].x, ag[i][2].y, ag[i][3].x, ag[i][3].y);
      }
    }
    if (p.sum_g == 2 && threadIdx.x == 0) p.part_g[blockIdx.x] = a1;
  }
}

// Column sums of the CTAs' partial sums: 32 columns (16-byte loads of 4) by 128 slices of the
// P rows a CTA, so that a thread's few loads are all in flight at once; the slices are added
// in order.  blockIdx.y 0: dweight, 1: the channel gate's gradient, or in one CTA that of a
// single gate (gcols 1): the sum of P values.
__global__ void __launch_bounds__(1024) norm_grad_sum_kernel(const float *part_w,
                                                             const float *part_g, int P, int H,
                                                             int gcols, __nv_bfloat16 *dw,
                                                             __nv_bfloat16 *dg) {
  __shared__ float s[128][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool single = blockIdx.y && gcols == 1;
  if (single && blockIdx.x) return;
  const float *part = blockIdx.y ? part_g : part_w;
  pdl_wait();
  if (single) {
    float v = 0.f;
    for (int i = threadIdx.x; i < P; i += 1024) v += part[i];
    s[warp][lane] = v;
    __syncthreads();
    v = 0.f;
    if (warp == 0)
      for (int k = 0; k < 32; ++k) v += s[k][lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (threadIdx.x == 0) dg[0] = __float2bfloat16_rn(v);
    return;
  }
  const int q = threadIdx.x >> 3, c = blockIdx.x * 32 + (threadIdx.x & 7) * 4;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < H) {
#pragma unroll 8
    for (int i = q; i < P; i += 128) {
      const float4 x = *reinterpret_cast<const float4 *>(part + (int64_t)i * H + c);
      v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
    }
  }
  float *at = &s[q][(threadIdx.x & 7) * 4];
  at[0] = v.x, at[1] = v.y, at[2] = v.z, at[3] = v.w;
  __syncthreads();
  float t = s[lane][warp];   // warp w adds the 128 slices of column w
#pragma unroll
  for (int k = 1; k < 4; ++k) t += s[lane + 32 * k][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
  const int col = blockIdx.x * 32 + warp;
  if (lane == 0 && col < H) (blockIdx.y ? dg : dw)[col] = __float2bfloat16_rn(t);
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
  if (rs.maxt == 0) {
    const std::integral_constant<int, 0> warp;
    if (rs.vpt == 5) return f(std::integral_constant<int, 5>(), warp);
    if (rs.vpt == 6) return f(std::integral_constant<int, 6>(), warp);
    return vpt(warp);
  }
  if (rs.maxt == 256) return vpt(std::integral_constant<int, 256>());
  return vpt(std::integral_constant<int, 1024>());
}

// How many rows ahead a CTA fetches: what fits its share of an SM's shared memory when
// `ctas` of them share it, at most kMaxStages.
size_t plan_rows(RowArrays *rows, const RowShape &rs, int ctas) {
  const size_t stage = (size_t)rows->n * rs.vpt * rs.threads * 16;
  const size_t budget = 208 * 1024 / ctas;
  rows->stages = (int)std::max<size_t>(1, std::min<size_t>(kMaxStages, budget / stage));
  return stage * rows->stages;
}

template <int MODE>
int launch_norm(const NormParams &p, RowArrays rows, cudaStream_t s) {
  const RowShape rs = row_shape(p.H / 8, p.T < num_sms());
  const int64_t ctas = rs.maxt ? p.T : ceil_div(p.T, kWarps);
  const size_t smem = plan_rows(&rows, rs, row_ctas(rs.maxt));
  return with_shape(rs, [&](auto vpt, auto maxt) {
    auto k = norm_kernel<vpt(), maxt(), MODE>;
    const int nb = resident_blocks(k, rs.threads, smem);
    if (nb <= 0) return (int)NVFP4_ECUDA;
    const dim3 grid((unsigned)std::min<int64_t>(ctas, (int64_t)num_sms() * nb));
    return launch_pdl(k, grid, dim3(rs.threads), smem, s, p, rows);
  });
}

// Most CTAs of a gradient: their partial sums of H values stay within about 8 MB (three CTAs
// an SM at least), so that writing and adding them is small beside the rows.
int grad_ctas(int64_t T, int64_t H) {
  const int64_t per = H / 8 <= kWarpRowVecs ? kWarps : 1;
  const int64_t most = std::min<int64_t>(8, std::max<int64_t>(3, (2 << 20) / H / num_sms()));
  return (int)std::max<int64_t>(1, std::min<int64_t>(ceil_div(T, per), num_sms() * most));
}
size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

int run_grad(NormGradParams &p, RowArrays rows, __nv_bfloat16 *dw, __nv_bfloat16 *dg_sum,
             void *ws, cudaStream_t s) {
  const int most = grad_ctas(p.T, p.H);
  int P = most;
  p.part_w = static_cast<float *>(ws);
  p.part_g = reinterpret_cast<float *>(static_cast<char *>(ws) + align256((size_t)most * p.H * 4));
  const RowShape rs = row_shape(p.H / 8, p.T < num_sms());
  size_t smem = plan_rows(&rows, rs, grad_row_ctas(rs.maxt, rs.vpt, p.sum_g == 1));
  if (!rs.maxt)   // the warps' sums of dweight, and of a channel gate's gradient
    smem = std::max(smem, (size_t)(p.sum_g == 1 ? 2 : 1) * kWarps * rs.vpt * 4 * 32 * 8);
  auto launch = [&](auto k) {
    const int nb = resident_blocks(k, rs.threads, smem);
    if (nb <= 0) return (int)NVFP4_ECUDA;
    P = std::min(most, num_sms() * nb);
    return launch_pdl(k, dim3(P), dim3(rs.threads), smem, s, p, rows);
  };
  const int st = with_shape(rs, [&](auto vpt, auto maxt) {
    if (!p.gate) return launch(norm_grad_kernel<vpt(), maxt(), kNoGate>);
    if (!p.gh) return launch(norm_grad_kernel<vpt(), maxt(), kRowGate>);
    if (!p.gt) return launch(norm_grad_kernel<vpt(), maxt(), kChannelGate>);
    return launch(norm_grad_kernel<vpt(), maxt(), kFullGate>);
  });
  if (st) return st;
  const dim3 grid((unsigned)ceil_div(p.H, 32), p.sum_g ? 2 : 1);
  return launch_pdl(norm_grad_sum_kernel, grid, dim3(1024), 0, s, (const float *)p.part_w,
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
  p.w = weight, p.out = out, p.T = T, p.H = (int)H, p.eps = eps;
  return launch_norm<kPre>(p, {{x}, 1}, stream);
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
  p.w = weight, p.codes = codes, p.scales = scales, p.T = T, p.H = (int)H, p.eps = eps;
  return launch_norm<kPreInt8>(p, {{x}, 1}, stream);
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
  p.codes = codes, p.scales = scales, p.T = rows, p.H = (int)cols;
  return launch_norm<kQuant>(p, {{x}, 1}, stream);
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
  p.w = weight, p.w_next = next_weight, p.out = out;
  p.next = next, p.T = T, p.H = (int)H, p.eps = eps, p.a = residual_scale;
  const RowArrays rows = {{y, residual, gate}, p.gh && p.gt ? 3 : 2};
  return next ? launch_norm<kPostNext>(p, rows, stream) : launch_norm<kPost>(p, rows, stream);
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
  p.w = weight, p.dx = dx, p.T = T, p.H = (int)H, p.eps = eps, p.skip = dskip != nullptr;
  return run_grad(p, {{x, dy, dskip}, dskip ? 3 : 2}, dweight, nullptr, workspace, stream);
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
  p.w = weight, p.gate = g.gate, p.dx = dy, p.dres = dresidual;
  p.T = T, p.gt = g.gt, p.gh = g.gh, p.H = (int)H, p.eps = eps, p.a = residual_scale;
  p.sum_g = gate && gate_rows == 1 ? (gate_cols == H ? 1 : 2) : 0;
  p.dgate_el = gate && gate_rows != 1 ? dgate : nullptr;
  return run_grad(p, {{y, dout, gate}, p.gh && p.gt ? 3 : 2}, dweight, p.sum_g ? dgate : nullptr,
                  workspace, stream);
}
