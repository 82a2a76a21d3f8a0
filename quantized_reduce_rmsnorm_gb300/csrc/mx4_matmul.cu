// mx4_matmul.cu -- product of two microscaled 4-bit tensors (mx4.cuh):
//   out[t, n] = sum_k x[t, k] * w[n, k],  binary32 accumulation, rounded once.
//
// tcgen05.mma kind::mxf4 multiplies e2m1 codes and applies the blocks' e8m0
// scales itself.  The tile's 128 rows are output features (w) and its columns
// are tokens (x): one token costs 16 columns, not 128 rows, and the
// accumulator's lanes are neighbouring features, so a warp stores neighbouring
// elements of a row of `out`.  One warp keeps a ring of TMA copies ahead (codes
// through tensor maps with the 128-byte swizzle, 256 elements of k a stage;
// scale tiles as they lie), one thread moves the scales to the tensor core's
// memory and issues the products, four warps bring the result out.  (Issued under
// `lane == 0` and not under an elected lane, 8192 x 8192 x 8192 took 374 us instead
// of 262, before any other step.)
#include <cuda.h>

#include <algorithm>

#include "block.h"
#include "mx4.cuh"

namespace fc {
namespace {

constexpr int kM = 128;          // features of a tile
constexpr int kStageK = 256;     // elements of k a stage: 128 bytes of codes a row
constexpr int kThreads = 192;    // warps 0-3: result; 4: copies; 5: products
constexpr int kMostParts = 8;    // of k, in one cluster
constexpr int kErrCuda = 2;      // FC_ERR_CUDA

template <int BN>
struct Tile {
  static constexpr int kStages = BN >= 128 ? 3 : BN >= 32 ? 4 : 5;  // two CTAs an SM
  static constexpr int kABytes = kM * 128, kBBytes = BN * 128;
  static constexpr int kSfBytes = 1024;               // 128 rows, 256 elements of k
  static constexpr int kStageBytes = kABytes + kBBytes + 2 * kSfBytes;
  static constexpr int kSmem = kStages * kStageBytes + 1024 + 256;
  // columns of the tensor core's memory: the accumulator, then each stage's scales
  static constexpr int kSfCols = 16;
  static constexpr int kColsUsed = BN + kStages * kSfCols;
  static constexpr int kCols = kColsUsed <= 128 ? 128 : 256;
};

struct Job {
  const uint8_t* x_scales;
  const uint8_t* w_scales;
  void* out;
  int32_t* status;
  int64_t rows, features;
  int64_t wait;     // cycles
  int H, KT;        // elements and scale tiles of k
  int out_f32;
};

// ------------------------------------------------------------- tcgen05 ----
__device__ __forceinline__ void tmem_alloc(uint32_t* where, int cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(where)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t at, int cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols));
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// Arrives on bar when all tcgen05 work that this thread issued is done.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_u32(bar))
               : "memory");
}
// 32 rows of 16 bytes (512 neighbouring bytes) to four columns of the first 32
// lanes, and again to the other three groups of 32 lanes.
__device__ __forceinline__ void tc_copy_scales(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}
__device__ __forceinline__ void tc_mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                            uint32_t sfa, uint32_t sfb, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(static_cast<uint32_t>(acc))
      : "memory");
}
// 16 neighbouring columns of this warp's 32 lanes.
__device__ __forceinline__ void tc_load16(uint32_t tmem, uint32_t v[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, "
      "[%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(tmem));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// One lane of a converged warp.  The tcgen05 and TMA instructions are issued
// under this predicate and not under `lane == 0`: the compiler knows it to be
// uniform, and their operands then need no loop over the lanes.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// Shared-memory matrix descriptors: rows of 128 bytes with the 128-byte
// swizzle, 1024 bytes from one group of eight rows to the next; and rows of 16
// bytes without a swizzle, 128 bytes from group to group.
__device__ __forceinline__ uint64_t desc_codes(uint32_t smem) {
  return static_cast<uint64_t>((smem & 0x3FFFF) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_scales(uint32_t smem) {
  return static_cast<uint64_t>((smem & 0x3FFFF) >> 4) | (1ull << 16) | (8ull << 32) | (1ull << 46);
}
// Instruction descriptor: e2m1 by e2m1, both along k, e8m0 scales, M rows, N
// columns; sf: which half (0 or 2) of a scale word's four bytes.
__device__ __forceinline__ uint32_t idesc_mxf4(int M, int N, uint32_t sf) {
  return (sf << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>(M >> 4) << 24) | (sf << 29);
}

__device__ __forceinline__ void store_out(const Job& j, int64_t t, int f, float v) {
  if (j.out_f32)
    static_cast<float*>(j.out)[t * j.features + f] = v;
  else
    static_cast<__nv_bfloat16*>(j.out)[t * j.features + f] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      ::"r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

// ------------------------------------------------ few tokens: k in parts --
// With few tokens the weights' bytes count and there are fewer tiles than SMs:
// the CTAs of a cluster take the parts of k of one tile, leave their sums in
// their shared memory, and each adds up a slice of the features over the parts,
// in order (no atomics: the same bits every time).  Bound by the weights' bytes:
// one token by 8192 x 8192, weights that are not in L2, 8.5 us, 4.2 TB/s (floor 5.3 us;
// one CTA a tile 11.5); what is left is a launch, the first copies' latency and the join.
__device__ __forceinline__ float4 ld_cluster(uint32_t at) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}

template <int BN>
__global__ void __launch_bounds__(kThreads)
    k_mx4_matmul(const Job j, const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x) {
  using T = Tile<BN>;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sa = base;                                    // [stage][128 rows][128 bytes]
  uint8_t* sb = sa + T::kStages * T::kABytes;            // [stage][BN rows][128 bytes]
  uint8_t* ssa = sb + T::kStages * T::kBBytes;           // [stage][1024]
  uint8_t* ssb = ssa + T::kStages * T::kSfBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(ssb + T::kStages * T::kSfBytes);
  uint64_t* empty = full + T::kStages;
  uint64_t* done = empty + T::kStages;       // the accumulator holds this part's sums
  uint64_t* ended = done + 1;                // all copies and products issued have ended
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(ended + 1);
  volatile uint32_t* failed = tmem_at + 1;
  float* part = reinterpret_cast<float*>(base);          // [BN][128] sums, when the stages are done with
  static_assert(BN * kM * 4 <= T::kStages * T::kStageBytes, "the sums fit where the stages were");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * kM;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * BN;
  const int parts = gridDim.z, part_id = blockIdx.z;     // a cluster is the parts of a tile
  const int stages_k = (j.H + kStageK - 1) / kStageK;
  const int i0 = stages_k * part_id / parts, i1 = stages_k * (part_id + 1) / parts;

  if (threadIdx.x == 0) {
    for (int s = 0; s < T::kStages; ++s) mbar_init(full + s, 1), mbar_init(empty + s, 1);
    mbar_init(done, 1), mbar_init(ended, 2);
    *failed = 0;
    mbar_init_fence();
  }
  // taken before the next kernel may start, so that all of this grid's CTAs have theirs
  if (warp == 5) tmem_alloc(tmem_at, T::kCols);
  if (warp == 4 && elect_one())
    for (int i = i0; i < i1 && i < i0 + T::kStages; ++i) {
      tma_prefetch_2d(&map_w, i * 128, n0);
      prefetch_l2(j.w_scales + (static_cast<int64_t>(blockIdx.x) * j.KT + 2 * i) * 512, j.KT - 2 * i >= 2 ? 1024 : 512);
    }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  pdl_begin();

  if (warp == 4) {
    if (elect_one()) {
      int s = 0, used = 0;
      uint32_t phase = 1;  // a first pass over the stages waits for nothing
      for (int i = i0; i < i1; ++i) {
        if (!mbar_wait_for(empty + s, phase, j.wait)) {
          *failed = 1;
          break;
        }
        const uint32_t sf = j.KT - 2 * i >= 2 ? 1024u : 512u;  // the last stage may hold one scale tile of k
        mbar_expect_tx(full + s, T::kABytes + T::kBBytes + 2 * sf);
        tma_load_2d(sa + s * T::kABytes, &map_w, i * 128, n0, full + s);
        bulk_load(ssa + s * T::kSfBytes, j.w_scales + (static_cast<int64_t>(blockIdx.x) * j.KT + 2 * i) * 512, sf,
                  full + s);
        tma_load_2d(sb + s * T::kBBytes, &map_x, i * 128, static_cast<int>(t0), full + s);
        bulk_load(ssb + s * T::kSfBytes, j.x_scales + (t0 / 128 * j.KT + 2 * i) * 512, sf, full + s);
        used = min(used + 1, T::kStages);
        if (++s == T::kStages) s = 0, phase ^= 1;
      }
      // the last copies land before the CTA ends, also where the products gave up on them
      for (int q = 0; q < used; ++q) {
        if (--s < 0) s = T::kStages - 1, phase ^= 1;
        mbar_wait_bounded(full + s, phase ^ 1);
      }
      mbar_arrive(ended);
    }
  } else if (warp == 5) {
    if (elect_one()) {
      int s = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int i = i0; i < i1; ++i) {
        if (!mbar_wait_for(full + s, phase, j.wait)) {
          *failed = 1;
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sf = tmem + BN + s * T::kSfCols;
        const int halves = j.KT - 2 * i >= 2 ? 2 : 1;  // scale tiles of k in this stage
        for (int q = 0; q < halves; ++q) {
          tc_copy_scales(sf + 4 * q, desc_scales(smem_u32(ssa + s * T::kSfBytes + q * 512)));
          tc_copy_scales(sf + 8 + 4 * q, desc_scales(smem_u32(ssb + s * T::kSfBytes + q * 512)));
        }
        const uint64_t da = desc_codes(smem_u32(sa + s * T::kABytes));
        const uint64_t db = desc_codes(smem_u32(sb + s * T::kBBytes));
        const int steps = min(4, (j.H - i * kStageK + 63) / 64);
#pragma unroll
        for (int k = 0; k < 4; ++k)  // 64 elements: 32 bytes further along the row
          if (k < steps)
            tc_mma_mxf4(tmem, da + 2 * k, db + 2 * k, idesc_mxf4(kM, BN, (k & 1) * 2), sf + 4 * (k >> 1),
                        sf + 8 + 4 * (k >> 1), i > i0 || k > 0);
        tc_commit(empty + s);
        if (++s == T::kStages) s = 0, phase ^= 1;
      }
      if (ok) tc_commit(done);
      tc_commit(ended);
      mbar_wait_bounded(ended, 0);  // before the memory that they use goes
    }
  } else {
    const bool there = __all_sync(kFull, mbar_wait_for(done, 0, j.wait));
    if (!there) {
      *failed = 1;
      mbar_wait_bounded(ended, 0);
    }
    tc_fence_after();
    __syncwarp();
    const int f = warp * 32 + lane;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(BN), j.rows - t0));
    const uint32_t mine = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    for (int c = 0; c < tokens; c += 16) {
      uint32_t v[16];
      tc_load16(mine + c, v);
      if (parts > 1) {
        // a part without its sums makes NaN of the tile
#pragma unroll
        for (int i = 0; i < 16; ++i) part[(c + i) * kM + f] = __uint_as_float(there ? v[i] : 0x7FC00000u);
      } else if (n0 + f < j.features && there) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (c + i < tokens) store_out(j, t0 + c + i, n0 + f, __uint_as_float(v[i]));
      }
    }
    tc_fence_before();
  }
  __syncwarp();
  if (parts > 1) {
    cluster_sync_all();  // every part's sums are in its shared memory
    const int tokens = static_cast<int>(min(static_cast<int64_t>(BN), j.rows - t0));
    const int shift = 5 - (31 - __clz(parts));  // log2 of the slice's groups of four features
    for (int k = threadIdx.x; k < tokens << shift; k += kThreads) {
      const int t = k >> shift, f = ((part_id << shift) + (k & ((1 << shift) - 1))) * 4;
      const float* p = part + t * kM + f;
      float4 v[kMostParts], s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int r = 0; r < kMostParts; ++r)
        if (r < parts) v[r] = ld_cluster(cluster_addr(p, r));
#pragma unroll
      for (int r = 0; r < kMostParts; ++r)
        if (r < parts) s.x += v[r].x, s.y += v[r].y, s.z += v[r].z, s.w += v[r].w;
      if (n0 + f < j.features) {  // a multiple of 16: all four or none
        const int64_t at = (t0 + t) * j.features + n0 + f;
        if (j.out_f32)
          *reinterpret_cast<float4*>(static_cast<float*>(j.out) + at) = s;
        else
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(j.out) + at) =
              make_uint2(pack_bf2(s.x, s.y), pack_bf2(s.z, s.w));
      }
    }
    __syncwarp();
    cluster_sync_all();  // no part's memory goes before the others have read it
  } else {
    __syncthreads();
  }
  if (threadIdx.x == 0 && *failed && j.status) *j.status = kErrCuda;
  if (warp == 5) {
    __syncwarp();
    tc_fence_after();
    tmem_free(tmem, T::kCols);
  }
}

// ------------------------------------------------- many tokens: persistent --
// A pair of CTAs (two SMs) takes tile after tile of 256 features by 256 tokens: each
// CTA stages 128 features and 128 tokens, and one thread of the first issues
// products of both (cta_group::2), which read the tokens' codes from both CTAs'
// shared memory and leave each CTA its 128 features by all 256 tokens.  A pair
// loads a third less than two CTAs with tiles of their own: 35 KB a stage and CTA
// (8192 x 8192 x 8192: 162 us against 170, with four stages of the five 169; with the
// scales' moves between the products 160 us, with the waits of mbar_wait_for 153, 7.2
// PFLOP/s, the tensor pipe active for four fifths of it).  An instruction takes 64
// elements of k; those of 96 that this chip has, at half as much again, are not used.  Copies run
// ahead into the next tile; the eight result warps take the accumulator into
// registers (each 32 features by 128 tokens) and hand it back, so that the
// next tile's products start while they round, stage and store this one's, each
// warp by itself: 16 tokens at a time to shared memory, and from there by bulk
// tensor stores.  bf16 leaves the tensor memory as 16 x 8 fragments, whose transposed
// store makes rows of features (4096 tokens, 8192 features, 1024 elements, in tiles of one
// CTA: 20.4 us against 23.1 with a store for each element; pairs of CTAs 24.2, their loss
// where k is short).
template <bool OUT32>
struct Wide {
  static constexpr int kTile = 256;     // features and tokens of a pair's tile
  static constexpr int kHalf = 128;     // of one CTA
  static constexpr int kStages = 5, kBufs = 2;  // of copies, of results
  static constexpr int kThreads = 320;  // warps 0-7: result; 8: copies; 9: products
  static constexpr int kCodeBytes = kHalf * 128, kSfBytes = 1024;
  static constexpr int kStageBytes = 2 * kCodeBytes + 3 * kSfBytes;
  static constexpr int kOutBytes = OUT32 ? 2048 : 1024;  // of a result warp: 32 features by 16 tokens, kBufs times
  static constexpr int kSmem = kStages * kStageBytes + 8 * kBufs * kOutBytes + 1024 + 256;
  static constexpr int kSfCols = 24;    // [half of k] features; [half of k][128 tokens]
  static constexpr int kCols = 512;     // the accumulator's 256, then each stage's scales
  static_assert(kTile + kStages * kSfCols <= kCols && kSmem <= 227 * 1024, "fits");
};

// The same as above for a pair of CTAs.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* where, int cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(where)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tmem_free_pair(uint32_t at, int cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols));
}
// Arrives on bar of both CTAs.
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
// Each CTA's shared memory to its own tensor memory.
__device__ __forceinline__ void tc_copy_scales_pair(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}
__device__ __forceinline__ void tc_mma_mxf4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                                 uint32_t sfb, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(static_cast<uint32_t>(acc))
      : "memory");
}
// Into this CTA's shared memory, counted on a barrier of the pair (a cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// Arrives on bar of this CTA alone.
__device__ __forceinline__ void tc_commit_own(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

template <int N>  // N * 32 neighbouring columns of this warp's 32 lanes
__device__ __forceinline__ void tc_load_all(uint32_t tmem, uint32_t (&v)[N * 32]) {
#pragma unroll
  for (int b = 0; b < N; ++b) {
    uint32_t* r = v + b * 32;
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(tmem + b * 32));
  }
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// N * 64 neighbouring columns of 16 lanes (0 or 16 on from tmem's), as fragments of
// 16 lanes by 8 columns: thread l has lane l / 4, columns 2 (l % 4) and the next, in
// the first two of a fragment's four registers, and lane l / 4 + 8 in the others.
template <int N>
__device__ __forceinline__ void tc_load_fragments(uint32_t tmem, uint32_t (&v)[N * 32]) {
#pragma unroll
  for (int b = 0; b < N; ++b) {
    uint32_t* r = v + b * 32;
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, "
        "[%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(tmem + b * 64));
  }
}
// Four 8 x 8 matrices of 16-bit elements to shared memory, transposed: thread l's
// register m holds row l / 4, columns 2 (l % 4) and the next of matrix m; `row` is
// where column l % 8 of matrix l / 8 goes.
__device__ __forceinline__ void store_transposed(uint32_t row, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(row), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int x, int y, const void* src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x),
               "r"(y), "r"(smem_u32(src))
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

template <bool OUT32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Wide<OUT32>::kThreads, 1)
    k_mx4_matmul_wide(const Job j, const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                      const __grid_constant__ CUtensorMap map_wsf, const __grid_constant__ CUtensorMap map_xsf,
                      const __grid_constant__ CUtensorMap map_out) {
  using T = Wide<OUT32>;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sa = base;                               // [stage] 128 features' codes
  uint8_t* sb = sa + T::kStages * T::kCodeBytes;    // [stage] 128 tokens' codes
  uint8_t* ssa = sb + T::kStages * T::kCodeBytes;   // [stage] this CTA's features' scales
  uint8_t* ssb = ssa + T::kStages * T::kSfBytes;    // [stage][2] all 256 tokens' scales
  uint8_t* so = ssb + 2 * T::kStages * T::kSfBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(so + 8 * T::kBufs * T::kOutBytes);  // the first CTA's: both CTAs' copies
  uint64_t* empty = full + T::kStages;
  uint64_t* acc_full = empty + T::kStages;   // the accumulator holds a tile
  uint64_t* acc_free = acc_full + 1;         // the first CTA's: it is in both CTAs' result warps' registers
  uint64_t* ended = acc_free + 1;            // the first CTA's: all products issued have ended
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(ended + 1);
  volatile uint32_t* failed = tmem_at + 1;   // a role of either CTA gave up
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x & 1, pairs = gridDim.x >> 1;
  const int stages_k = (j.H + kStageK - 1) / kStageK;
  const int tiles_n = static_cast<int>((j.features + T::kTile - 1) / T::kTile);
  const int tiles = tiles_n * static_cast<int>((j.rows + T::kTile - 1) / T::kTile);

  if (threadIdx.x == 0) {
    for (int s = 0; s < T::kStages; ++s) mbar_init(full + s, 1), mbar_init(empty + s, 1);
    mbar_init(acc_full, 1);
    mbar_init(acc_free, 16), mbar_init(ended, 1);
    *failed = 0;
    mbar_init_fence();
  }
  if (warp == 9) tmem_alloc_pair(tmem_at, T::kCols);
  tc_fence_before();
  __syncwarp();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  const uint32_t peer_failed = cluster_addr(const_cast<const uint32_t*>(failed), rank ^ 1);
  auto give_up = [&] {
    *failed = 1;
    asm volatile("st.shared::cluster.u32 [%0], 1;" ::"r"(peer_failed) : "memory");
  };
  pdl_begin();

  if (warp == 8) {
    if (elect_one()) {
      int s = 0;
      uint32_t phase = 1;  // a first pass over the stages waits for nothing
      bool ok = true;
      for (int tile = blockIdx.x >> 1; tile < tiles && ok; tile += pairs) {
        const int nt = tile % tiles_n * 2, tt = tile / tiles_n * 2;  // in steps of 128
        for (int i = 0; i < stages_k; ++i) {
          if (!mbar_wait_for(empty + s, phase, j.wait)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_expect_tx(full + s, 2 * T::kStageBytes);
          const uint32_t bar = cluster_addr(full + s, 0);
          // what lies past the end of a tensor reads as 0; a stage's second scale tile of k
          // may be the next row's first, and is not used then
          tma_load_2d_pair(sa + s * T::kCodeBytes, &map_w, i * 128, (nt + rank) * 128, bar);
          tma_load_2d_pair(sb + s * T::kCodeBytes, &map_x, i * 128, (tt + rank) * 128, bar);
          tma_load_2d_pair(ssa + s * T::kSfBytes, &map_wsf, 0, ((nt + rank) * j.KT + 2 * i) * 4, bar);
          tma_load_2d_pair(ssb + 2 * s * T::kSfBytes, &map_xsf, 0, (tt * j.KT + 2 * i) * 4, bar);
          tma_load_2d_pair(ssb + (2 * s + 1) * T::kSfBytes, &map_xsf, 0, ((tt + 1) * j.KT + 2 * i) * 4, bar);
          if (++s == T::kStages) s = 0, phase ^= 1;
        }
      }
      if (!ok) give_up();
    }
  } else if (warp == 9) {
    if (rank == 0 && elect_one()) {
      int s = 0;
      uint32_t phase = 0, acc_phase = 1;
      bool ok = true;
      for (int tile = blockIdx.x >> 1; tile < tiles && ok; tile += pairs) {
        if (!mbar_wait_for(acc_free, acc_phase, j.wait)) {
          ok = false;
          break;
        }
        acc_phase ^= 1;
        // Scales of 128 elements of k go to the tensor core's memory while the products
        // before them run: the second half's behind the stage's first product, the
        // next stage's first half's before its last.
        auto copy_scales = [&](int st, int q) {
          const uint32_t sf = tmem + T::kTile + st * T::kSfCols;
          tc_copy_scales_pair(sf + 4 * q, desc_scales(smem_u32(ssa + st * T::kSfBytes + q * 512)));
          for (int r = 0; r < 2; ++r)
            tc_copy_scales_pair(sf + 8 + 4 * (2 * q + r), desc_scales(smem_u32(ssb + (2 * st + r) * T::kSfBytes + q * 512)));
        };
        auto ready = [&](int st, uint32_t ph) {  // the stage's copies have landed
          ok = mbar_wait_for(full + st, ph, j.wait);
          tc_fence_after();
          return ok;
        };
        if (!ready(s, phase)) break;
        copy_scales(s, 0);
        for (int i = 0; i < stages_k; ++i) {
          const uint32_t sf = tmem + T::kTile + s * T::kSfCols;
          const uint64_t da = desc_codes(smem_u32(sa + s * T::kCodeBytes));
          const uint64_t db = desc_codes(smem_u32(sb + s * T::kCodeBytes));
          const int steps = min(4, (j.H - i * kStageK + 63) / 64);
          auto product = [&](int k) {
            if (k < steps)
              tc_mma_mxf4_pair(tmem, da + 2 * k, db + 2 * k, idesc_mxf4(T::kTile, T::kTile, (k & 1) * 2),
                               sf + 4 * (k >> 1), sf + 8 + 8 * (k >> 1), i > 0 || k > 0);
          };
          product(0);
          if (j.KT - 2 * i >= 2) copy_scales(s, 1);  // the last stage may hold one scale tile of k
          product(1);
          product(2);
          const int s1 = s + 1 == T::kStages ? 0 : s + 1;
          const uint32_t phase1 = s1 == 0 ? phase ^ 1 : phase;
          if (i + 1 < stages_k) {
            if (!ready(s1, phase1)) break;
            copy_scales(s1, 0);
          }
          product(3);
          tc_commit_pair(empty + s);
          s = s1, phase = phase1;
        }
        if (ok) tc_commit_pair(acc_full);
      }
      if (!ok) give_up();
      tc_commit_own(ended);
      mbar_wait_bounded(ended, 0);  // before the memory that they use goes
    }
  } else {
    constexpr int kCols = T::kTile / 2;
    const int half = warp >> 2;
    uint8_t* buf0 = so + warp * T::kBufs * T::kOutBytes;
    int turn = 0;
    const uint32_t freed = cluster_addr(acc_free, 0);
    uint32_t phase = 0;
    for (int tile = blockIdx.x >> 1; tile < tiles; tile += pairs) {
      const bool there = mbar_wait_for(acc_full, phase, j.wait);
      phase ^= 1;
      if (__any_sync(kFull, !there || *failed)) {
        give_up();
        break;
      }
      tc_fence_after();
      const uint32_t mine = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + half * kCols;
      uint32_t v[OUT32 ? kCols : kCols / 2], u[kCols / 2];  // bf16: lanes 0-15 in v, 16-31 in u
      if constexpr (OUT32) {
        tc_load_all<kCols / 32>(mine, v);
      } else {
        tc_load_fragments<kCols / 64>(mine, v);
        tc_load_fragments<kCols / 64>(mine + (16u << 16), u);
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
      }
      tc_fence_before();
      if (lane == 0) mbar_arrive_cluster(freed);
      const int n0 = tile % tiles_n * T::kTile + rank * T::kHalf + (warp & 3) * 32;
      const int64_t t0 = static_cast<int64_t>(tile / tiles_n) * T::kTile + half * kCols;
      if (n0 >= j.features) continue;
#pragma unroll
      for (int c = 0; c < kCols; c += 16) {
        if (t0 + c >= j.rows) break;
        uint8_t* buf = buf0 + turn * T::kOutBytes;
        turn = turn + 1 == T::kBufs ? 0 : turn + 1;
        // the buffer's last store has read it
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(T::kBufs - 1) : "memory");
        __syncwarp();
        if constexpr (OUT32) {
#pragma unroll
          for (int i = 0; i < 16; ++i) reinterpret_cast<uint32_t*>(buf)[i * 32 + lane] = v[c + i];
        } else {
          // 16 tokens of 64 bytes, 16-byte groups in the order of the 64-byte swizzle
          // (group g of row t at g ^ (t / 2 % 4)): eight rows' groups hit all banks once
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int t = h * 8 + (lane & 7), k = (c / 8 + h) * 4;
            const uint32_t row = smem_u32(buf) + t * 64 + (((lane >> 3) ^ (t >> 1 & 3)) * 16);
            auto pk = [](uint32_t lo, uint32_t hi) { return pack_bf2(__uint_as_float(lo), __uint_as_float(hi)); };
            store_transposed(row, pk(v[k], v[k + 1]), pk(v[k + 2], v[k + 3]), pk(u[k], u[k + 1]), pk(u[k + 2], u[k + 3]));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tma_store_2d(&map_out, n0, static_cast<int>(t0 + c), buf);
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncwarp();
  cluster_sync_all();  // neither CTA ends while the other's products or barriers use its memory
  if (*failed) {
    // Copies may be in flight that neither CTA can wait for: the second CTA's count on
    // the first's barriers, and the CTAs may have given up at different stages.  No more
    // are issued; they have the time of a wait to land in.
    const long long t0 = clock64();
    while (clock64() - t0 < 1ll << 31) __nanosleep(10000);
    __syncwarp();
    cluster_sync_all();
  }
  if (threadIdx.x == 0 && *failed && j.status) *j.status = kErrCuda;
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    tmem_free_pair(tmem, T::kCols);
  }
}

// ------------------------------------------------------------- launch ----
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// Codes [rows, H / 2 bytes] in boxes of 128 bytes by box_rows rows; bytes and
// rows past the end read as 0.
cudaError_t codes_map(CUtensorMap* m, const void* codes, int64_t rows, int H, int box_rows) {
  const EncodeFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(H / 2), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(H / 2)};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t step[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

// out [rows, features] in boxes of 32 features by 16 tokens (bf16: 64-byte swizzle);
// what lies past the end is not written.
cudaError_t out_map(CUtensorMap* m, const Mx4MatmulArgs& a) {
  const EncodeFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.features), static_cast<cuuint64_t>(a.rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(a.features) * (a.out_f32 ? 4 : 2)};
  const cuuint32_t box[2] = {32, 16}, step[2] = {1, 1};
  return fn(m, a.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.out, dims, strides,
            box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, a.out_f32 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

// Scale tiles as rows of 128 bytes, two neighbouring tiles (1024 bytes) a box.
cudaError_t scales_map(CUtensorMap* m, const uint8_t* scales, int64_t rows, int KT) {
  const EncodeFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {128, static_cast<cuuint64_t>((rows + 127) / 128) * KT * 4};
  const cuuint64_t strides[1] = {128};
  const cuuint32_t box[2] = {128, 8}, step[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(scales), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

template <bool OUT32>
cudaError_t launch_wide(const Mx4MatmulArgs& a, const Job& j, cudaStream_t st) {
  using T = Wide<OUT32>;
  auto* kern = k_mx4_matmul_wide<OUT32>;
  if (cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), T::kSmem)) return e;
  CUtensorMap mw, mx, mws, mxs, mo;
  if (cudaError_t e = codes_map(&mw, a.w_codes, a.features, a.H, T::kHalf)) return e;
  if (cudaError_t e = codes_map(&mx, a.x_codes, a.rows, a.H, T::kHalf)) return e;
  if (cudaError_t e = scales_map(&mws, a.w_scales, a.features, j.KT)) return e;
  if (cudaError_t e = scales_map(&mxs, a.x_scales, a.rows, j.KT)) return e;
  if (cudaError_t e = out_map(&mo, a)) return e;
  const int64_t tiles = ((a.features + T::kTile - 1) / T::kTile) * ((a.rows + T::kTile - 1) / T::kTile);
  const int64_t pairs = std::min<int64_t>(tiles, num_sms() / 2);
  return launch_pdl(kern, dim3(static_cast<unsigned>(2 * pairs)), dim3(T::kThreads), T::kSmem, st, j, mw, mx, mws, mxs,
                    mo);
}

template <int BN>
cudaError_t launch(const Mx4MatmulArgs& a, const Job& j, int parts, cudaStream_t st) {
  auto* kern = k_mx4_matmul<BN>;
  if (cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), Tile<BN>::kSmem)) return e;
  CUtensorMap mw, mx;
  if (cudaError_t e = codes_map(&mw, a.w_codes, a.features, a.H, kM)) return e;
  if (cudaError_t e = codes_map(&mx, a.x_codes, a.rows, a.H, BN)) return e;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = static_cast<unsigned>(parts);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.features + kM - 1) / kM), static_cast<unsigned>((a.rows + BN - 1) / BN),
                     static_cast<unsigned>(parts));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Tile<BN>::kSmem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, j, mw, mx);
}

}  // namespace

cudaError_t launch_mx4_matmul(const Mx4MatmulArgs& a, cudaStream_t st) {
  const Job j{a.x_scales, a.w_scales, a.out, a.status, a.rows, a.features, wait_cycles,
              a.H, static_cast<int>(mx4_tiles_k(a.H)), a.out_f32 ? 1 : 0};
  // The kernel that cuts k holds two CTAs an SM.  Its parts: as many as keep all
  // CTAs resident at once, at least four stages each (us, inputs changing from call to
  // call, 1 / 2 / 4 / 8 parts: 1 token 8192 x 8192 11.5 / 10.1 / 8.5 / 11.6, 64 tokens 4096
  // x 4096 8.8 / 8.3 / 6.3 / 7.7 at two stages a part).  Above 128 tokens, and where k
  // is not cut, the persistent kernel's wider tile wins (512 tokens 8192 x 8192 16.9
  // against 20.5, 2048 tokens 4096 x 4096 17.1 against 25.9); with k cut it does not (512
  // tokens 2048 x 8192: 15.0 against 12.2).
  const int64_t stages = (a.H + kStageK - 1) / kStageK;
  const int bn = a.rows <= 16 ? 16 : a.rows <= 32 ? 32 : a.rows <= 64 ? 64 : 128;
  const int64_t tiles = ((a.features + kM - 1) / kM) * ((a.rows + bn - 1) / bn);
  int parts = 1;
  while (parts < kMostParts && parts * 8 <= stages && tiles * parts * 2 <= 2 * num_sms()) parts *= 2;
  if (a.rows > 128 && parts == 1)
    return a.out_f32 ? launch_wide<true>(a, j, st) : launch_wide<false>(a, j, st);
  if (bn == 16) return launch<16>(a, j, parts, st);
  if (bn == 32) return launch<32>(a, j, parts, st);
  if (bn == 64) return launch<64>(a, j, parts, st);
  return launch<128>(a, j, parts, st);
}

}  // namespace fc
