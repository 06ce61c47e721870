// dense.cuh -- dense tensor-core products D = A B^T (tcgen05, sm_100a) with the epilogues of
// the 8-bit product (int8.cu) and of the gated projection and its gradients (gate_up.cu).
//
// Operands are 16-bit floats (fp32 sums) or 8-bit integers (exact int32 sums).  Each comes by
// TMA into a ring of 128-byte-swizzled stages, K-major ([rows, K], as weights and activations
// lie in memory) or, for 16-bit types, MN-major ([K, rows]: the transposed operands of the
// gradients, so nothing is ever transposed in memory).  What lies outside a tensor reads as
// zero, so no size has to be a multiple of a tile.  Two kernels:
//
//  * dense_pair_kernel, large products: pairs of CTAs (cta_group::2) each take 256 x 256
//    tiles.  Every CTA holds 128 rows of A and 128 rows of B a stage, so the pair reads half
//    the shared memory per flop that two single CTAs would.  Tiles are handed out in a fixed
//    order; two TMEM accumulators let the epilogue of a tile run under the next one's MMAs.
//    Bound by the tensor pipe and the power limit: 4096 x 4096 x 6144 bf16 with the gate 140 us
//    (1,475 TFLOP/s, pipe 85% active), 8-bit 4096 x 6144 x 6144 96 us (3,220), both in a captured
//    graph of a few milliseconds; 161 and 110 us in a loop of a second, where the power limit
//    holds the clock at 1.36 and 1.44 GHz of 1.965.
//  * dense_split_kernel, few tokens or small matrices: 128 x NT tiles of one CTA, the sum
//    over K split over the CTAs of a cluster so that every SM streams its share of the
//    weights.  Partial tiles meet in shared memory: each CTA adds its slice of the tile over
//    the cluster's CTAs in rank order (the result does not depend on timing) and stores it.
//    Bound by the stream of weights at few tokens (1 x 4096 x 6144 bf16: 11.2 us for 50 MB),
//    by the parts' way between the SMs at 64 (1.5 to 2 us of 10 at 64 x 4096 x 6144, 8-bit).
//
// Every wait is bounded.  One that gives up ORs bit 1 into the caller's error flag, nothing is
// issued or re-armed behind it, and what it was waiting for comes out as NaN: a lost tile shows
// without a flag too.  (LOSE: the selftest kernels, which leave out loads and wait 2 ms.)
#pragma once
#include <algorithm>

#include "moe.cuh"
#include "tcgen05.cuh"

namespace nvfp4 {

enum DenseKind { kBf16 = 0, kS8 = 1 };
enum DenseEpi { kEpiStore = 0, kEpiScale = 1, kEpiGate = 2 };

// act(z): SiLU, or GELU by its tanh form, in which (1 + tanh v) / 2 = 1 / (1 + exp(-2 v)): one
// quotient, as exact for negative z as for positive (1 + tanh v cancels there: 0.6% off at
// z = -4.25, 35% at -5).
constexpr float kGeluA = 0.7978845608028654f;    // v = A (z + B z^3), A = sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;
__device__ __forceinline__ float gelu_v(float z) { return kGeluA * fmaf(kGeluB * z * z, z, z); }
template <int ACT>
__device__ __forceinline__ float gate_act(float z) {
  if (ACT == NVFP4_ACT_SILU) return silu_f32(z);
  return z / (1.f + expf(-2.f * gelu_v(z)));
}

struct DenseArgs {
  // Logical product: D[m, n] = sum_k A[m, k] B[n, k].  pair kernel: D rows are the output's
  // rows.  split kernel: D rows are the output's columns, unless ROWS.
  int64_t M, N, K;
  int64_t half;                // kEpiGate: I, the rows of the gate half of w_gu
  const float *m_scale;        // kEpiScale: scale of each D row (ordinary loads: the kernel before
                               //            may write them while this one is already resident)
  const float *n_scale;        //            scale of each D column
  __nv_bfloat16 *out;          // split kernel: output, `ld` elements a row
  __nv_bfloat16 *gu;           // split kernel, kEpiGate: [cols, 2 half] pre-activations, or null
  int64_t ld;
  int save_gu;                 // pair kernel, kEpiGate: tensor maps g / u are set
  int32_t *flag;               // error bits, or null
  int m_tiles, n_tiles;
  int whole, cut, items;       // pair kernel: see item_at
};

// Bounded wait of one CTA; after any of its waits has given up, later ones return at once.
struct CtaWait {
  int *abort;
  int32_t *flag;
  uint64_t limit_ns;
  __device__ __forceinline__ bool operator()(uint64_t *bar, uint32_t parity) const {
    if (mbar_try_wait(bar, parity)) return true;
    if (*(volatile int *)abort) return false;
    if (mbar_wait(bar, parity, limit_ns)) return true;
    *(volatile int *)abort = 1;
    report_timeout(flag);
    return false;
  }
  // The same for a converged warp: one answer for all lanes.
  __device__ __forceinline__ bool warp(uint64_t *bar, uint32_t parity) const {
    return __all_sync(0xFFFFFFFFu, (*this)(bar, parity));
  }
};

// One lane of a converged warp, always the same one.  The issuing warps run their loops with
// all lanes and elect one around each group of tensor or copy instructions: those take their
// operands from the warp's uniform registers, and from inside a divergent branch each of them
// needs its operands moved there one at a time (the 256 x 256 tiles ran 12% slower so).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}

template <bool LOSE>
constexpr uint64_t wait_limit() {
  return LOSE ? 2000000ull : kWaitLimitNs;
}
// What a lost value is: two bf16 NaN, an fp32 NaN, and in the int32 sums (|sum| <= 2^29) the
// lowest value.
constexpr uint32_t kLostBf16x2 = 0x7FFF7FFFu, kLostF32 = 0x7FFFFFFFu, kLostS32 = 0x80000000u;

// ------------------------------------------------------------------ pairs of CTAs
constexpr int kPS = 6;                              // stages
constexpr uint32_t kPHalf = 128 * 128;              // A or B part of a stage, one CTA
constexpr uint32_t kPStage = 2 * kPHalf;
constexpr uint32_t kPOut = kPS * kPStage;           // 4 warps x 2 buffers of 32 rows x 128 B
constexpr uint32_t kPBars = kPOut + 4 * 2 * 4096;
constexpr uint32_t kPMisc = kPBars + 8 * (2 * kPS + 4);
constexpr uint32_t kPSmem = kPMisc + 16 + 1024;
constexpr int kPThreads = 192;                      // producer, MMA, 4 epilogue warps
static_assert(kPSmem <= 227 * 1024, "shared memory budget");

// What work item `i` is.  The first p.whole items are whole tiles, one after another to each
// pair; the tiles that are left, too few to keep all pairs busy, are cut into `cut` items of
// 256 / cut columns each (launch_pair), so the last round is that much shorter.
struct PairItem {
  int mt, nt, part, width;   // tile, part of it, columns of the part
};
__device__ __forceinline__ void tile_at(int i, int m_tiles, int n_tiles, int &mt, int &nt);
__device__ __forceinline__ PairItem item_at(int i, const DenseArgs &p) {
  PairItem t = {0, 0, 0, 256};
  int tile = i;
  if (i >= p.whole) {
    t.part = (i - p.whole) % p.cut;
    t.width = 256 / p.cut;
    tile = p.whole + (i - p.whole) / p.cut;
  }
  tile_at(tile, p.m_tiles, p.n_tiles, t.mt, t.nt);
  return t;
}

// Tile `i` of m_tiles x n_tiles, in groups of 16 rows of tiles, so that the tiles in flight at
// one time share A and B tiles in L2 (groups of 8: 3% slower in a loop at 4096 x 6144 x 4096).
constexpr int kGroupM = 16;
__device__ __forceinline__ void tile_at(int i, int m_tiles, int n_tiles, int &mt, int &nt) {
  const int per = kGroupM * n_tiles, g = i / per, r = i % per;
  const int rows = min(kGroupM, m_tiles - g * kGroupM);
  mt = g * kGroupM + r % rows;
  nt = r / rows;
}

// One 128-byte-wide chunk (64 bf16 columns) of a warp's 32 rows: packed values -> swizzled
// staging buffer -> TMA store (rows and columns outside the tensor are not written).
__device__ __forceinline__ void store_chunk(const uint32_t (&v)[32], unsigned char *buf, int lane,
                                            const CUtensorMap *map, int x, int y, bool inside) {
  if (lane == 0) bulk_wait_group_read<1>();   // the store before the last has left this buffer
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<uint4 *>(buf + lane * 128 + ((c ^ (lane & 7)) << 4)) =
        make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (inside) tma_store_2d(map, x, y, buf);
    bulk_commit_group();
  }
}

template <int KIND, bool AMN, bool BMN, int EPI, int ACT, bool LOSE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPThreads, 1)
    dense_pair_kernel(const __grid_constant__ CUtensorMap map_a,
                      const __grid_constant__ CUtensorMap map_b,
                      const __grid_constant__ CUtensorMap map_out,
                      const __grid_constant__ CUtensorMap map_g,
                      const __grid_constant__ CUtensorMap map_u, DenseArgs p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  //   full[s]      (leader's) both CTAs' tiles of stage s have landed
  //   freeb[s]     the MMAs reading stage s are done (commit, to both CTAs)
  //   accfull[b]   accumulator b holds a finished tile (commit, to both CTAs)
  //   accempty[b]  (leader's) the 8 epilogue warps have read accumulator b
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + kPBars);
  uint64_t *freeb = full + kPS;
  uint64_t *accfull = freeb + kPS;
  uint64_t *accempty = accfull + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + kPMisc);
  int *abort = reinterpret_cast<int *>(smem + kPMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();

  if (threadIdx.x == 0) {
    *abort = 0;
    for (int s = 0; s < kPS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&freeb[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accfull[b], 1);
      mbar_init(&accempty[b], 8);
    }
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // the peer's barriers exist before anything arrives on them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();

  const CtaWait wait{abort, p.flag, wait_limit<LOSE>()};
  const int total = p.items, pairs = (int)gridDim.x / 2;
  const int first = (int)blockIdx.x / 2;
  constexpr int kElems = KIND == kS8 ? 128 : 64;   // K elements of a stage
  const int kblocks = (int)((p.K + kElems - 1) / kElems);

  if (warp == 0) {
    int kg = 0;
    bool ok = true;
    const uint32_t full0 = map_rank(smem_u32(full), 0);
    for (int i = first; ok && i < total; i += pairs) {
      const PairItem it = item_at(i, p);
      const int m0 = it.mt * 256 + rank * 128;
      const int hw = it.width / 2;   // this CTA's half of the item's B rows
      const int n0 = EPI == kEpiGate ? (int)(rank * p.half) + it.nt * 128 + it.part * hw
                                     : it.nt * 256 + it.part * it.width + rank * hw;
      for (int kb = 0; kb < kblocks; ++kb, ++kg) {
        const int s = kg % kPS;
        if (kg >= kPS) ok = wait.warp(&freeb[s], ((kg / kPS) - 1) & 1);
        if (!ok) break;
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * (kPHalf + hw * 128));
          const uint32_t bar = full0 + s * 8;
          unsigned char *A = smem + s * kPStage, *B = A + kPHalf;
          const int k0 = kb * kElems;
          if (LOSE && rank == 1 && i != first && kb == 0) {
            // the peer's part of a pair's second tile never lands
          } else if (AMN) {
            tma_load_2d_pair(A, &map_a, m0, k0, bar);
            tma_load_2d_pair(A + kPHalf / 2, &map_a, m0 + 64, k0, bar);
          } else {
            tma_load_2d_pair(A, &map_a, k0, m0, bar);
          }
          if (LOSE && rank == 1 && i != first && kb == 0) {
          } else if (BMN) {
            tma_load_2d_pair(B, &map_b, n0, k0, bar);
            if (hw > 64) tma_load_2d_pair(B + kPHalf / 2, &map_b, n0 + 64, k0, bar);
          } else {
            tma_load_2d_pair(B, &map_b, k0, n0, bar);
            if (hw > 64) tma_load_2d_pair(B + kPHalf / 2, &map_b, k0, n0 + 64, bar);
          }
        }
        __syncwarp();
      }
    }
    // the leader sees both CTAs' copies land; the peer stays until then (cluster_sync)
    if (rank == 0)
      for (int t = max(0, kg - kPS); t < kg; ++t)
        mbar_wait(&full[t % kPS], (t / kPS) & 1, wait_limit<LOSE>());
  } else if (warp == 1) {
    if (rank == 0) {
      int kg = 0, tc = 0;
      bool ok = true;
      for (int i = first; i < total; i += pairs, ++tc) {
        const int acc = tc & 1;
        if (tc >= 2 && !wait.warp(&accempty[acc], ((tc >> 1) - 1) & 1)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + acc * 256;
        const int width = item_at(i, p).width;
        const uint32_t idesc =
            (KIND == kS8 ? idesc_s8_s32(256, width) : idesc_bf16_f32(256, width)) |
            (AMN ? kIdescMnMajorA : 0) | (BMN ? kIdescMnMajorB : 0);
        for (int kb = 0; kb < kblocks; ++kb, ++kg) {
          const int s = kg % kPS;
          ok = wait.warp(&full[s], (kg / kPS) & 1);
          if (!ok) break;   // nothing is committed: the others give up in their turn
          tc_fence_after();
          if (elect_one()) {
            const uint32_t a = smem_u32(smem + s * kPStage);
            const uint64_t da = AMN ? smem_desc_mn_sw128(a, kPHalf / 2) : smem_desc_sw128(a);
            const uint64_t db = BMN ? smem_desc_mn_sw128(a + kPHalf, kPHalf / 2)
                                    : smem_desc_sw128(a + kPHalf);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              // 32 bytes along the rows (K-major), or 16 K rows of 128 bytes (MN-major)
              const uint64_t ak = da + (AMN ? 128 : 2) * kk, bk = db + (BMN ? 128 : 2) * kk;
              if (KIND == kS8)
                umma_s8_pair(d, ak, bk, idesc, kb > 0 || kk > 0);
              else
                umma_bf16_pair(d, ak, bk, idesc, kb > 0 || kk > 0);
            }
            umma_commit_pair(&freeb[s]);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (elect_one()) umma_commit_pair(&accfull[acc]);
        __syncwarp();
      }
    }
  } else {
    const int q = warp & 3;
    unsigned char *buf = smem + kPOut + (warp - 2) * 8192;
    int tc = 0, nst = 0;
    bool lost = false;   // stays: the barriers' phases mean nothing behind a lost tile
    for (int i = first; i < total; i += pairs, ++tc) {
      const PairItem it = item_at(i, p);
      const int hw = it.width / 2;
      const int acc = tc & 1;
      lost = lost || !wait.warp(&accfull[acc], (tc >> 1) & 1);
      tc_fence_after();
      const uint32_t tb = tmem_base + acc * 256 + ((uint32_t)(q * 32) << 16);
      const int row0 = it.mt * 256 + rank * 128 + q * 32;
      const bool rows_in = row0 < p.M;
      if (lost) {
        uint32_t bad[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) bad[k] = kLostBf16x2;
        const int cols = EPI == kEpiGate ? hw : it.width;
        for (int c = 0; c < cols / 64; ++c) {
          const int x = it.nt * (EPI == kEpiGate ? 128 : 256) + it.part * cols + c * 64;
          const bool in = rows_in && x < p.N;
          store_chunk(bad, buf + (nst++ & 1) * 4096, lane, &map_out, x, row0, in);
          if (EPI == kEpiGate && p.save_gu) {
            store_chunk(bad, buf + (nst++ & 1) * 4096, lane, &map_g, x, row0, in);
            store_chunk(bad, buf + (nst++ & 1) * 4096, lane, &map_u, x, row0, in);
          }
        }
        continue;
      }
      if (EPI == kEpiGate) {
        // the first half of the columns is the gate, the second the up projection of the
        // same columns of h
        for (int c = 0; c < hw / 64; ++c) {
          const int x = it.nt * 128 + it.part * hw + c * 64;
          uint32_t hp[32], gp[32], up[32];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t g[32], u[32];
            tmem_ld32(tb + c * 64 + hf * 32, g);
            tmem_ld32(tb + hw + c * 64 + hf * 32, u);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float g0 = __uint_as_float(g[2 * k]), g1 = __uint_as_float(g[2 * k + 1]);
              const float u0 = __uint_as_float(u[2 * k]), u1 = __uint_as_float(u[2 * k + 1]);
              hp[hf * 16 + k] = pack_bf16x2(gate_act<ACT>(g0) * u0, gate_act<ACT>(g1) * u1);
              gp[hf * 16 + k] = pack_bf16x2(g0, g1);
              up[hf * 16 + k] = pack_bf16x2(u0, u1);
            }
          }
          const bool in = rows_in && x < p.N;
          store_chunk(hp, buf + (nst++ & 1) * 4096, lane, &map_out, x, row0, in);
          if (p.save_gu) {
            store_chunk(gp, buf + (nst++ & 1) * 4096, lane, &map_g, x, row0, in);
            store_chunk(up, buf + (nst++ & 1) * 4096, lane, &map_u, x, row0, in);
          }
        }
      } else {
        const int row = row0 + lane;
        const float ms = (EPI == kEpiScale && row < p.M) ? p.m_scale[row] : 0.f;
        for (int c = 0; c < it.width / 64; ++c) {
          const int x = it.nt * 256 + it.part * it.width + c * 64;
          uint32_t o[32];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t v[32];
            tmem_ld32(tb + c * 64 + hf * 32, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              float f[4];
              if (EPI == kEpiScale) {
                const int col = x + hf * 32 + k * 4;
                const float4 ns = col < p.N ? *reinterpret_cast<const float4 *>(p.n_scale + col)
                                            : make_float4(0.f, 0.f, 0.f, 0.f);
                f[0] = (float)(int)v[4 * k] * ms * ns.x;
                f[1] = (float)(int)v[4 * k + 1] * ms * ns.y;
                f[2] = (float)(int)v[4 * k + 2] * ms * ns.z;
                f[3] = (float)(int)v[4 * k + 3] * ms * ns.w;
              } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = __uint_as_float(v[4 * k + j]);
              }
              o[hf * 16 + 2 * k] = pack_bf16x2(f[0], f[1]);
              o[hf * 16 + 2 * k + 1] = pack_bf16x2(f[2], f[3]);
            }
          }
          store_chunk(o, buf + (nst++ & 1) * 4096, lane, &map_out, x, row0, rows_in && x < p.N);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_rank(smem_u32(&accempty[acc]), 0));
    }
    if (lane == 0) bulk_wait_group_all();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  pdl_launch_dependents();
  cluster_sync();   // the leader's MMAs read the peer's shared memory until here
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
  cluster_sync();   // both CTAs are there for the deallocation
}

// ------------------------------------------------------------------ K split over a cluster
constexpr int kSThreads = 256;   // producer, MMA; all 8 warps read TMEM, add and store
constexpr int kMaxSplit = 8;     // CTAs of a cluster (the portable limit)
template <int NT, bool ROWS>   // ROWS: the result is row-major in D (out[m][n])
struct SplitShape {
  static constexpr int kStages = NT == 64 ? 4 : 5;
  static constexpr uint32_t kA = 128 * 128, kB = NT * 128, kStage = kA + kB;
  // partial tile, fp32 or int32, in the ring: [NT][128], or [128][NT + 4] (ROWS)
  static constexpr int kPitch = ROWS ? NT + 4 : 128;
  static constexpr uint32_t kTile = (ROWS ? 128 : NT) * kPitch * 4;
  static constexpr uint32_t kBars = kStages * kStage;
  static constexpr uint32_t kMisc = kBars + 8 * (2 * kStages + 1);
  static constexpr uint32_t kSmem = kMisc + 16 + 1024;
  static constexpr uint32_t kTmemCols = NT < 32 ? 32 : NT;
  static_assert(kTile <= kStages * kStage, "the partial tile fits the ring");
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs an SM (1 KB reserved for each)");
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 pack4(float4 v) {
  return make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

template <int KIND, bool AMN, bool BMN, int EPI, int ACT, int NT, bool ROWS, bool LOSE>
__global__ void __launch_bounds__(kSThreads, 2)
    dense_split_kernel(const __grid_constant__ CUtensorMap map_a,
                       const __grid_constant__ CUtensorMap map_b, DenseArgs p) {
  using S = SplitShape<NT, ROWS>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + S::kBars);
  uint64_t *freeb = full + S::kStages;
  uint64_t *accfull = freeb + S::kStages;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + S::kMisc);
  int *abort = reinterpret_cast<int *>(smem + S::kMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank(), nr = (int)cluster_size();

  const CtaWait wait{abort, p.flag, wait_limit<LOSE>()};
  constexpr int kElems = KIND == kS8 ? 128 : 64;
  const int kblocks = (int)((p.K + kElems - 1) / kElems);
  const int kb0 = (int)((int64_t)rank * kblocks / nr), kb1 = (int)((int64_t)(rank + 1) * kblocks / nr);
  const int tile = (int)blockIdx.x / nr, mt = tile % p.m_tiles, nt = tile / p.m_tiles;
  constexpr int kTileM = EPI == kEpiGate ? 64 : 128;   // output columns (D rows) of a tile
  const int m0 = mt * kTileM, n0 = nt * NT;

  if (warp == 0) {
    if (lane == 0) {
      *abort = 0;
      for (int s = 0; s < S::kStages; ++s) {
        mbar_init(&full[s], 1);
        mbar_init(&freeb[s], 1);
      }
      mbar_init(accfull, 1);
      mbar_init_fence();
    }
    __syncwarp();
    asm volatile("bar.arrive 1, %0;" ::"n"(kSThreads) : "memory");   // barriers are ready
    // The first ring of weights is asked into L2 while the kernel before may still run (8-bit
    // 1 x 6144 x 4096 with its quantizer 9.8 -> 9.3 us, bf16 1 x 2048 x 2048 with the gate 5.5 ->
    // 4.9; alone the same).  A hint: the loads themselves come after pdl_wait, and L2 is where
    // any write of that kernel meets them, so nothing older can be read.
    if (!ROWS && elect_one()) {
      for (int kb = kb0; kb < min(kb1, kb0 + S::kStages); ++kb) {
        const int k0 = kb * kElems;
        if (EPI == kEpiGate) {
          tma_prefetch_2d(&map_a, k0, m0);
          tma_prefetch_2d(&map_a, k0, (int)p.half + m0);
        } else if (AMN) {
          tma_prefetch_2d(&map_a, m0, k0);
          tma_prefetch_2d(&map_a, m0 + 64, k0);
        } else {
          tma_prefetch_2d(&map_a, k0, m0);
        }
      }
    }
    __syncwarp();
  } else {
    if (warp == 1) tmem_alloc(tmem_slot, S::kTmemCols);
    tc_fence_before();
    asm volatile("bar.sync 1, %0;" ::"n"(kSThreads) : "memory");
    tc_fence_after();
  }
  pdl_launch_dependents();
  pdl_wait();

  if (warp == 0) {
    int i = 0;
    for (int kb = kb0; kb < kb1; ++kb, ++i) {
      const int s = i % S::kStages;
      if (i >= S::kStages && !wait.warp(&freeb[s], ((i / S::kStages) - 1) & 1)) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(&full[s], S::kStage);
        unsigned char *A = smem + s * S::kStage, *B = A + S::kA;
        const int k0 = kb * kElems;
        if (LOSE && rank == 0 && i == 0) {
          // the first CTA's first weights never land
        } else if (EPI == kEpiGate) {   // 64 gate rows, then the matching 64 up rows
          tma_load_2d(A, &map_a, k0, m0, &full[s]);
          tma_load_2d(A + S::kA / 2, &map_a, k0, (int)p.half + m0, &full[s]);
        } else if (AMN) {
          tma_load_2d(A, &map_a, m0, k0, &full[s]);
          tma_load_2d(A + S::kA / 2, &map_a, m0 + 64, k0, &full[s]);
        } else {
          tma_load_2d(A, &map_a, k0, m0, &full[s]);
        }
        if (BMN) {
#pragma unroll
          for (int j = 0; j < NT / 64; ++j)
            tma_load_2d(B + j * 8192, &map_b, n0 + 64 * j, k0, &full[s]);
        } else {
          tma_load_2d(B, &map_b, k0, n0, &full[s]);
        }
      }
      __syncwarp();
    }
    // every copy lands before the ring is used again or the CTA exits
    for (int t = max(0, i - S::kStages); t < i; ++t)
      mbar_wait(&full[t % S::kStages], (t / S::kStages) & 1, wait_limit<LOSE>());
  } else if (warp == 1) {
    const uint32_t tmem_base = *tmem_slot;
    constexpr uint32_t idesc = (KIND == kS8 ? idesc_s8_s32(128, NT) : idesc_bf16_f32(128, NT)) |
                               (AMN ? kIdescMnMajorA : 0) | (BMN ? kIdescMnMajorB : 0);
    bool ok = true;
    for (int i = 0; i < kb1 - kb0; ++i) {
      const int s = i % S::kStages;
      ok = wait.warp(&full[s], (i / S::kStages) & 1);
      if (!ok) break;   // nothing is committed: the others give up in their turn
      tc_fence_after();
      if (elect_one()) {
        const uint32_t a = smem_u32(smem + s * S::kStage);
        const uint64_t da = AMN ? smem_desc_mn_sw128(a, S::kA / 2) : smem_desc_sw128(a);
        const uint64_t db =
            BMN ? smem_desc_mn_sw128(a + S::kA, 8192) : smem_desc_sw128(a + S::kA);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t ak = da + (AMN ? 128 : 2) * kk, bk = db + (BMN ? 128 : 2) * kk;
          if (KIND == kS8)
            umma_s8(tmem_base, ak, bk, idesc, i > 0 || kk > 0);
          else
            umma_bf16(tmem_base, ak, bk, idesc, i > 0 || kk > 0);
        }
        umma_commit(&freeb[s]);
      }
      __syncwarp();
    }
    if (ok && elect_one()) umma_commit(accfull);
  }
  __syncwarp();
  // every thread of the CTA waits for the tile: the ring is free and may hold partial sums
  wait(accfull, 0);
  __syncthreads();   // the producer's copies have landed too
  const bool lost = *(volatile int *)abort;   // a wait of this CTA gave up: its part is not there
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  uint32_t *red = reinterpret_cast<uint32_t *>(smem);
  const int ncols = (int)min((int64_t)NT, p.N - n0);   // D columns inside the result
  {   // two warps for each quarter of the TMEM lanes, 16 columns at a time in turn
    const int row = (warp & 3) * 32 + lane;
    const uint32_t tb = tmem_base + ((uint32_t)((warp & 3) * 32) << 16);
#pragma unroll 1
    for (int c = (warp >> 2) * 16; c < ncols; c += 32) {
      uint32_t v[16];
      tmem_ld16(tb + c, v);
      if (lost)
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = KIND == kS8 ? kLostS32 : kLostF32;
      if (ROWS) {
#pragma unroll
        for (int k = 0; k < 16; k += 4)
          *reinterpret_cast<uint4 *>(red + row * S::kPitch + c + k) =
              make_uint4(v[k], v[k + 1], v[k + 2], v[k + 3]);
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) red[(c + k) * S::kPitch + row] = v[k];
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, S::kTmemCols);
  }
  cluster_sync();
  // Add the cluster's partial tiles: four neighbouring values a thread, this CTA's share.
  uint32_t peer[kMaxSplit];
#pragma unroll
  for (int r = 0; r < kMaxSplit; ++r) peer[r] = map_rank(smem_u32(red), r < nr ? r : 0);
  auto sum_at = [&](int at) {   // `at`: index of the first of four elements of the tile
    float4 w[kMaxSplit];
#pragma unroll
    for (int r = 0; r < kMaxSplit; ++r)   // all loads first
      w[r] = r < nr ? ld_cluster_f4(peer[r] + at * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
    float4 v = w[0];
    if (KIND == kS8) {   // an absent part is 0 in either type
      int a[4] = {0, 0, 0, 0};
      bool gone = false;
#pragma unroll
      for (int r = 0; r < kMaxSplit; ++r) {
        gone = gone || __float_as_uint(w[r].x) == kLostS32;
        a[0] += __float_as_int(w[r].x), a[1] += __float_as_int(w[r].y);
        a[2] += __float_as_int(w[r].z), a[3] += __float_as_int(w[r].w);
      }
      v = make_float4((float)a[0], (float)a[1], (float)a[2], (float)a[3]);
      if (gone) v.x = v.y = v.z = v.w = __uint_as_float(kLostF32);
    } else {
#pragma unroll
      for (int r = 1; r < kMaxSplit; ++r)
        v.x += w[r].x, v.y += w[r].y, v.z += w[r].z, v.w += w[r].w;
    }
    return v;
  };
  // M and N are multiples of 8, so four neighbours are all inside or all outside
  if (ROWS) {
    const int quads = 128 * (NT / 4);
    const int e0 = (int)((int64_t)quads * rank / nr), e1 = (int)((int64_t)quads * (rank + 1) / nr);
    for (int e = e0 + (int)threadIdx.x; e < e1; e += kSThreads) {
      const int m = e / (NT / 4), n = e % (NT / 4) * 4;
      if (m0 + m < p.M && n0 + n < p.N)
        *reinterpret_cast<uint2 *>(p.out + (int64_t)(m0 + m) * p.ld + n0 + n) =
            pack4(sum_at(m * S::kPitch + n));
    }
  } else {
    const int quads = ncols * (kTileM / 4);
    const int e0 = (int)((int64_t)quads * rank / nr), e1 = (int)((int64_t)quads * (rank + 1) / nr);
    for (int e = e0 + (int)threadIdx.x; e < e1; e += kSThreads) {
      const int n = e / (kTileM / 4), m = e % (kTileM / 4) * 4;
      if (m0 + m >= p.M) continue;
      float4 v = sum_at(n * S::kPitch + m);
      const int64_t row = n0 + n;
      if (EPI == kEpiGate) {
        const float4 u = sum_at(n * S::kPitch + 64 + m);
        if (p.gu) {
          __nv_bfloat16 *o = p.gu + row * 2 * p.half + m0 + m;
          *reinterpret_cast<uint2 *>(o) = pack4(v);
          *reinterpret_cast<uint2 *>(o + p.half) = pack4(u);
        }
        v.x = gate_act<ACT>(v.x) * u.x, v.y = gate_act<ACT>(v.y) * u.y;
        v.z = gate_act<ACT>(v.z) * u.z, v.w = gate_act<ACT>(v.w) * u.w;
      } else if (EPI == kEpiScale) {
        const float ts = p.n_scale[row];
        const float4 ms = *reinterpret_cast<const float4 *>(p.m_scale + m0 + m);
        v.x = v.x * ts * ms.x, v.y = v.y * ts * ms.y;
        v.z = v.z * ts * ms.z, v.w = v.w * ts * ms.w;
      }
      *reinterpret_cast<uint2 *>(p.out + row * p.ld + m0 + m) = pack4(v);
    }
  }
  cluster_sync();   // no CTA leaves while another still reads its partial tile
}

// ------------------------------------------------------------------ host side
// Tensor map of a 16- or 8-bit operand: K-major [rows, K] (boxes of box_rows rows by 128
// bytes), or MN-major [K, rows] (boxes of 64 K rows by 64 values).
inline int operand_map(CUtensorMap *m, int kind, bool mn, const void *base, int64_t rows,
                       int64_t K, int box_rows) {
  const CUtensorMapDataType t =
      kind == kS8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int bytes = kind == kS8 ? 1 : 2;
  int st = mn ? make_map(m, t, bytes, base, (uint64_t)rows, (uint64_t)K, 64, 64,
                         CU_TENSOR_MAP_SWIZZLE_128B)
              : make_map(m, t, bytes, base, (uint64_t)K, (uint64_t)rows, 128 / bytes,
                         (uint32_t)box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
  if (st) set_last_cuda_error(cudaErrorInvalidValue);
  return st;
}
// Tensor map of an output: `cols` bf16 of rows `ld` elements apart, boxes of 32 rows x 64.
inline int out_map(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t ld) {
  int st = make_map_pitch(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, (uint64_t)cols,
                          (uint64_t)rows, (uint64_t)ld * 2, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B);
  if (st) set_last_cuda_error(cudaErrorInvalidValue);
  return st;
}

// Whether a [rows, cols] result goes to the pair kernel: more than 128 rows (half a tile) and
// tiles enough that, cut in half, they occupy five of eight CTA pairs.  Measured with K = 6144:
// 24 tiles, 8-bit 256 x 6144: pairs 17 us, split 20; 128 x 6144: pairs 17, split 15; 16 tiles,
// 8-bit 512 x 2048 x 2048: pairs 9 us, split 8.
inline bool dense_use_pair(int64_t rows, int64_t cols) {
  return rows > 128 && ceil_div(rows, 256) * ceil_div(cols, 256) * 16 >= num_sms() / 2 * 5;
}

// Where the operands lie: A [M, K] (or [K, M]) and B [N, K] (or [K, N]).
struct DenseOperands {
  const void *a, *b;
};

template <int KIND, bool AMN, bool BMN, int EPI, int ACT, bool LOSE = false>
int launch_pair(DenseArgs p, DenseOperands o, const CUtensorMap &out, const CUtensorMap &g,
                const CUtensorMap &u, cudaStream_t s) {
  CUtensorMap ta, tb;
  const int64_t brows = EPI == kEpiGate ? 2 * p.half : p.N;
  if (int st = operand_map(&ta, KIND, AMN, o.a, p.M, p.K, 128)) return st;
  if (int st = operand_map(&tb, KIND, BMN, o.b, brows, p.K, 64)) return st;
  p.m_tiles = (int)ceil_div(p.M, 256);
  p.n_tiles = (int)ceil_div(p.N, EPI == kEpiGate ? 128 : 256);
  auto k = dense_pair_kernel<KIND, AMN, BMN, EPI, ACT, LOSE>;
  if (resident_blocks(k, kPThreads, kPSmem) < 0) return NVFP4_ECUDA;
  const int total = p.m_tiles * p.n_tiles, slots = num_sms() / 2;
  const int left = total % slots;
  p.cut = left && left * 2 <= slots ? 2 : 1;
  p.whole = total - left;
  p.items = p.whole + left * p.cut;
  const int pairs = std::min(p.items, slots);
  return launch_pdl(k, dim3(2 * pairs), dim3(kPThreads), kPSmem, s, ta, tb, out, g, u, p);
}

// A kernel of the split kernel's block size whose residency stands for it: the occupancy
// queries answer one block an SM for kernels that allocate TMEM, whatever they allocate (two
// run: the split kernel's columns are at most 64 of 512).
static __global__ void __launch_bounds__(kSThreads, 2) split_shape_kernel() {}

// Over how many CTAs the sum over K is split: as many as keep all clusters resident at once
// (a second round of clusters costs a whole pass: 8-bit 1 x 6144 x 6144, 48 tiles, 12 us with
// clusters of 5 of which 56 fit, 16 us with 6 of which 45 fit), one in sixteen left free for
// the kernel before, which may still be running.  0 after a CUDA error.
inline int split_count(int64_t tiles, int64_t kblocks, size_t smem) {
  if (resident_blocks(split_shape_kernel, kSThreads, smem) <= 0) return 0;
  for (int nr = (int)std::min<int64_t>(kMaxSplit, kblocks); nr > 1; --nr) {
    const int fit = resident_clusters_fn(reinterpret_cast<const void *>(split_shape_kernel),
                                         kSThreads, smem, nr);
    if (fit < 0) return 0;
    if (tiles * 16 <= (int64_t)fit * 15) return nr;
  }
  return 1;
}

template <int KIND, bool AMN, bool BMN, int EPI, int ACT, int NT, bool ROWS = false,
          bool LOSE = false>
int launch_split(DenseArgs p, DenseOperands o, cudaStream_t s) {
  using S = SplitShape<NT, ROWS>;
  CUtensorMap ta, tb;
  const int64_t arows = EPI == kEpiGate ? 2 * p.half : p.M;
  if (int st = operand_map(&ta, KIND, AMN, o.a, arows, p.K, EPI == kEpiGate ? 64 : 128)) return st;
  if (int st = operand_map(&tb, KIND, BMN, o.b, p.N, p.K, NT)) return st;
  p.m_tiles = (int)ceil_div(p.M, EPI == kEpiGate ? 64 : 128);
  p.n_tiles = (int)ceil_div(p.N, NT);
  auto k = dense_split_kernel<KIND, AMN, BMN, EPI, ACT, NT, ROWS, LOSE>;
  if (resident_blocks(k, kSThreads, S::kSmem) <= 0) return NVFP4_ECUDA;
  const int64_t tiles = (int64_t)p.m_tiles * p.n_tiles;
  const int64_t kblocks = ceil_div(p.K, KIND == kS8 ? 128 : 64);
  const int nr = split_count(tiles, kblocks, S::kSmem);
  if (nr <= 0) return NVFP4_ECUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * nr));
  cfg.blockDim = dim3(kSThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = nr;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, ta, tb, p);
  if (e != cudaSuccess) {
    set_last_cuda_error(e);
    return NVFP4_ECUDA;
  }
  return NVFP4_OK;
}

// The split kernel with the smallest column tile that holds N columns, at most 64: at 128 the
// partial tiles' way through the cluster costs more than the second read of A it saves (8-bit
// 128 x 4096 x 1024 with its quantizer: 9.8 us against 11.7; it won by 8% at 192..256 x 6144
// x 4096).
template <int KIND, bool AMN, int EPI, int ACT, bool LOSE = false>
int launch_split_n(const DenseArgs &p, DenseOperands o, cudaStream_t s) {
  if (p.N <= 16) return launch_split<KIND, AMN, false, EPI, ACT, 16, false, LOSE>(p, o, s);
  if (p.N <= 32) return launch_split<KIND, AMN, false, EPI, ACT, 32, false, LOSE>(p, o, s);
  return launch_split<KIND, AMN, false, EPI, ACT, 64, false, LOSE>(p, o, s);
}

}  // namespace nvfp4
