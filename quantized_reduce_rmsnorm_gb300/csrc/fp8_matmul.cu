// fp8_matmul.cu -- product of two tensors in 8-bit floating point with a scale for each
// block of 128 elements of k (fp8.cuh):
//   out[t, n] = sum over blocks b of sx[t, b] * sw[n / 128, b] * sum over k in b of x[t, k] * w[n, k]
//
// tcgen05.mma kind::f8f6f4 multiplies the codes: a block's sum is a product of its own
// in tensor memory (binary32), which the result warps read, multiply with the two scales
// (their product rounded once) and add to sums in their registers, while the tensor core
// is at the next block.  Scales are any binary32 numbers, so the tensor core's own
// scaling, by powers of two, is not used.
#include <algorithm>

#include "block.h"
#include "tc.cuh"

namespace fc {
namespace {

constexpr int kK = 128;          // elements of k of a block, a stage: 128 bytes of codes a row
constexpr int kMostParts = 8;    // of k, in one cluster
constexpr int kErrCuda = 2;      // FC_ERR_CUDA

struct Job {
  const float* x_scales;
  const float* w_scales;
  void* out;
  int32_t* status;
  int64_t rows, features;
  int64_t wait;     // cycles
  int KB;           // blocks of k
  int out_f32;
};

// ------------------------------------------------ few tokens: k in parts --
// With few tokens the weights' bytes count.  The tile's 128 rows are features of one
// block of the weight's, its columns are tokens: one token costs 16 columns, not 128
// rows.  The CTAs of a cluster take the parts of k of one tile, leave their sums in their
// shared memory, and each adds up a slice of the features over the parts, in order (no
// atomics: the same bits every time).  The products of the tokens' scales and the
// features' come a batch of blocks at a time, so that their loads wait together and not
// block by block.  Bound by the weights' bytes and a launch's start and join: one token by
// 8192 x 8192 12.5 us, 5.4 TB/s (floor 9.9 us); 64 tokens 15.7, the result warps' time.
template <int BN>
struct Tile {
  static constexpr int kM = 128, kThreads = 192;  // warps 0-3: result; 4: copies; 5: products
  static constexpr int kStages = BN >= 64 ? 4 : BN >= 32 ? 5 : 6;  // two CTAs an SM
  static constexpr int kABytes = kM * kK, kBBytes = BN * kK;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kBufs = 4;  // block sums in tensor memory
  static constexpr int kCols = BN * kBufs;
  static constexpr int kBatch = 16;  // blocks
  static constexpr int kFactors = kBatch * BN;       // of a batch, for all tokens; two batches
  static constexpr int kSmem = kStages * kStageBytes + 2 * kFactors * 4 + 1024 + 256;
  static_assert(2 * kCols <= 512 && 2 * (kSmem + 1024) <= 228 * 1024, "two CTAs an SM");
};

template <int BN>
__global__ void __launch_bounds__(Tile<BN>::kThreads, 2)
    k_fp8_matmul(const Job j, const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x) {
  using T = Tile<BN>;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sa = base;                                    // [stage][128 rows][128 bytes]
  uint8_t* sb = sa + T::kStages * T::kABytes;            // [stage][BN rows][128 bytes]
  float* factors = reinterpret_cast<float*>(sb + T::kStages * T::kBBytes);  // [2][block of the batch][token]
  uint64_t* full = reinterpret_cast<uint64_t*>(factors + 2 * T::kFactors);
  uint64_t* empty = full + T::kStages;
  uint64_t* acc_full = empty + T::kStages;   // [buffer] holds a block's sums
  uint64_t* acc_free = acc_full + T::kBufs;
  uint64_t* ended = acc_free + T::kBufs;     // all copies and products issued have ended
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(ended + 1);
  volatile uint32_t* failed = tmem_at + 1;
  float* part = reinterpret_cast<float*>(base);          // [BN][128] sums, when the stages are done with
  static_assert(BN * T::kM * 4 <= T::kStages * T::kStageBytes, "the sums fit where the stages were");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * T::kM;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * BN;
  const int parts = gridDim.z, part_id = blockIdx.z;     // a cluster is the parts of a tile
  const int i0 = j.KB * part_id / parts, i1 = j.KB * (part_id + 1) / parts;

  if (threadIdx.x == 0) {
    for (int s = 0; s < T::kStages; ++s) mbar_init(full + s, 1), mbar_init(empty + s, 1);
    for (int b = 0; b < T::kBufs; ++b) mbar_init(acc_full + b, 1), mbar_init(acc_free + b, 4);
    mbar_init(ended, 2);
    *failed = 0;
    mbar_init_fence();
  }
  // taken before the next kernel may start, so that all of this grid's CTAs have theirs
  if (warp == 5) tmem_alloc(tmem_at, T::kCols);
  if (warp == 4 && elect_one())
    for (int i = i0; i < i1 && i < i0 + T::kStages; ++i) tma_prefetch_2d(&map_w, i * kK, n0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  pdl_begin();

  float2 acc[BN / 2];
  bool there = true;
  if (warp == 4) {
    if (elect_one()) {
      int s = 0, used = 0;
      uint32_t phase = 1;  // a first pass over the stages waits for nothing
      for (int i = i0; i < i1; ++i) {
        if (!mbar_wait_for(empty + s, phase, j.wait)) {
          *failed = 1;
          break;
        }
        mbar_expect_tx(full + s, T::kStageBytes);
        tma_load_2d(sa + s * T::kABytes, &map_w, i * kK, n0, full + s);
        tma_load_2d(sb + s * T::kBBytes, &map_x, i * kK, static_cast<int>(t0), full + s);
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
      int s = 0, b = 0;
      uint32_t phase = 0, acc_phase = 1;
      for (int i = i0; i < i1; ++i) {
        if (!mbar_wait_for(full + s, phase, j.wait) || !mbar_wait_for(acc_free + b, acc_phase, j.wait)) {
          *failed = 1;
          break;
        }
        tc_fence_after();
        const uint64_t da = desc_along_k(smem_u32(sa + s * T::kABytes));
        const uint64_t db = desc_along_k(smem_u32(sb + s * T::kBBytes));
#pragma unroll
        for (int k = 0; k < 4; ++k)  // 32 elements
          tc_mma_e4m3(tmem + b * BN, da + 2 * k, db + 2 * k, idesc_e4m3(T::kM, BN), k > 0);
        tc_commit(empty + s);
        tc_commit(acc_full + b);
        if (++s == T::kStages) s = 0, phase ^= 1;
        if (++b == T::kBufs) b = 0, acc_phase ^= 1;
      }
      tc_commit(ended);
      mbar_wait_bounded(ended, 0);  // before the memory that they use goes
    }
  } else {
    // a thread's factors of a batch: those of token e / kBatch, block e % kBatch, for e = its
    // index and every 128th after it
    constexpr int kPer = T::kFactors / 128;
    const float* sw = j.w_scales + static_cast<int64_t>(blockIdx.x) * j.KB;
    const float* sx = j.x_scales + t0 * j.KB;
    float next[kPer];
    auto fetch = [&](int first) {
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const int e = q * 128 + threadIdx.x, t = e / T::kBatch, i = first + e % T::kBatch;
        next[q] = i < i1 && t0 + t < j.rows ? sx[static_cast<int64_t>(t) * j.KB + i] * sw[i] : 0.0f;
      }
    };
    fetch(i0);
#pragma unroll
    for (int c = 0; c < BN / 2; ++c) acc[c] = make_float2(0.0f, 0.0f);
    auto sum = [&](int c) { return c & 1 ? acc[c / 2].y : acc[c / 2].x; };
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    int b = 0;
    uint32_t phase = 0;
    for (int i = i0; i < i1; ++i) {
      const int in = (i - i0) % T::kBatch;
      float* batch = factors + ((i - i0) / T::kBatch & 1) * T::kFactors;
      if (in == 0) {
        // whoever is still at the batch before this one does not read this half
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
          const int e = q * 128 + threadIdx.x;
          batch[e % T::kBatch * BN + e / T::kBatch] = next[q];
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (i + T::kBatch < i1) fetch(i + T::kBatch);
      }
      const float* mine = batch + in * BN;
      // a wait that runs out ends the tile: the ones after it do not wait
      there = __all_sync(kFull, mbar_wait_for(acc_full + b, phase, there ? j.wait : 0) && there);
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < BN; c += 16) {
        uint32_t v[16];
        tc_load16(lanes + b * BN + c, v);
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
          const float4 f = *reinterpret_cast<const float4*>(mine + c + k);
          float2* a = acc + (c + k) / 2;
          a[0] = pfma(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), make_float2(f.x, f.y), a[0]);
          a[1] = pfma(make_float2(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3])), make_float2(f.z, f.w), a[1]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_free + b);
      if (++b == T::kBufs) b = 0, phase ^= 1;
    }
    if (!there) {
      *failed = 1;
      mbar_wait_bounded(ended, 0);
    }
    const int f = warp * 32 + lane;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(BN), j.rows - t0));
    if (parts > 1) {
      // a part without its sums makes NaN of the tile
#pragma unroll
      for (int c = 0; c < BN; ++c)
        if (c < tokens) part[c * T::kM + f] = there ? sum(c) : __uint_as_float(0x7FC00000u);
    } else if (n0 + f < j.features && there) {
#pragma unroll
      for (int c = 0; c < BN; ++c)
        if (c < tokens) {
          const int64_t at = (t0 + c) * j.features + n0 + f;
          if (j.out_f32)
            static_cast<float*>(j.out)[at] = sum(c);
          else
            static_cast<__nv_bfloat16*>(j.out)[at] = __float2bfloat16_rn(sum(c));
        }
    }
  }
  __syncwarp();
  if (parts > 1) {
    cluster_sync_all();  // every part's sums are in its shared memory
    const int tokens = static_cast<int>(min(static_cast<int64_t>(BN), j.rows - t0));
    const int shift = 5 - (31 - __clz(parts));  // log2 of the slice's groups of four features
    for (int k = threadIdx.x; k < tokens << shift; k += T::kThreads) {
      const int t = k >> shift, f = ((part_id << shift) + (k & ((1 << shift) - 1))) * 4;
      const float* p = part + t * T::kM + f;
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
// A pair of CTAs (two SMs) takes tile after tile of 256 tokens by 256 features: each CTA
// stages 128 tokens and 128 features, and one thread of the first issues products of
// both (cta_group::2), which leave each CTA its 128 tokens by all 256 features.  Two
// block sums fit the tensor memory: the tensor core fills one while the eight result
// warps, each 32 tokens by 128 features (one block of the weight's), empty the other:
// a thread has one token, so one factor, the product of the token's and the features'
// scales, serves all 128 of its sums.
// Bound by the turns of the two buffers: 8192 x 8192 x 8192 396 to 417 us, 2.7 PFLOP/s
// (floor 288); the same products summed in tensor memory, read once a tile, take 327.  A
// block takes about 780 cycles, of which the products 540: handing a buffer over
// and back costs as much again as emptying it.  Steps: scales loaded where they are used
// 1213; a block ahead, with 16 columns of sums on their way 945; buffers handed back
// without a release to the whole cluster, which waits for every load and store of the
// thread, 443; the products' warp asking for the copies before the buffer 405.  Not kept:
// halves of 128 features with four buffers (418; the products alone are as fast), sixteen
// result warps (470), warps that make the factors in shared memory (442), scales eight
// blocks ahead by asynchronous copies (466), more registers for the result warps by
// setmaxnreg and 32 columns on their way (437 to 550), one CTA a tile (461).
template <bool OUT32>
struct Wide {
  static constexpr int kTile = 256, kHalf = 128;
  static constexpr int kStages = 6, kBufs = 2;
  static constexpr int kThreads = 320;  // warps 0-7: result; 8: copies; 9: products
  static constexpr int kCodeBytes = kHalf * kK, kStageBytes = 2 * kCodeBytes;
  static constexpr int kOutBytes = 4096;  // of a result warp: 32 tokens by 128 bytes
  static constexpr int kOutCols = OUT32 ? 32 : 64;
  static constexpr int kSmem = kStages * kStageBytes + 8 * kOutBytes + 1024 + 256;
  static constexpr int kCols = kBufs * kTile;
  static_assert(kCols <= 512 && kSmem <= 227 * 1024, "fits");
};

template <bool OUT32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Wide<OUT32>::kThreads, 1)
    k_fp8_matmul_wide(const Job j, const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                      const __grid_constant__ CUtensorMap map_out) {
  using T = Wide<OUT32>;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sa = base;                               // [stage] 128 tokens' codes
  uint8_t* sb = sa + T::kStages * T::kCodeBytes;    // [stage] 128 features' codes
  uint8_t* so = sb + T::kStages * T::kCodeBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(so + 8 * T::kOutBytes);  // the first CTA's: both CTAs' copies
  uint64_t* empty = full + T::kStages;
  uint64_t* acc_full = empty + T::kStages;      // [buffer] holds a block's sums
  uint64_t* acc_free = acc_full + T::kBufs;     // the first CTA's: both CTAs' result warps have read it
  uint64_t* ended = acc_free + T::kBufs;        // the first CTA's: all products issued have ended
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(ended + 1);
  volatile uint32_t* failed = tmem_at + 1;      // a role of either CTA gave up
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x & 1, pairs = gridDim.x >> 1;
  const int tiles_n = static_cast<int>((j.features + T::kTile - 1) / T::kTile);
  const int tiles_m = static_cast<int>((j.rows + T::kTile - 1) / T::kTile);
  const int tiles = tiles_n * tiles_m;

  if (threadIdx.x == 0) {
    for (int s = 0; s < T::kStages; ++s) mbar_init(full + s, 1), mbar_init(empty + s, 1);
    for (int b = 0; b < T::kBufs; ++b) mbar_init(acc_full + b, 1), mbar_init(acc_free + b, 16);
    mbar_init(ended, 1);
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
        const int2 at = grouped_tile(tile, tiles_m, tiles_n);
        for (int i = 0; i < j.KB; ++i) {
          if (!mbar_wait_for(empty + s, phase, j.wait)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_expect_tx(full + s, 2 * T::kStageBytes);
          const uint32_t bar = cluster_addr(full + s, 0);
          // what lies past the end of a tensor reads as 0
          tma_load_2d_pair(sa + s * T::kCodeBytes, &map_x, i * kK, at.x * T::kTile + rank * T::kHalf, bar);
          tma_load_2d_pair(sb + s * T::kCodeBytes, &map_w, i * kK, at.y * T::kTile + rank * T::kHalf, bar);
          if (++s == T::kStages) s = 0, phase ^= 1;
        }
      }
      if (!ok) give_up();
    }
  } else if (warp == 9) {
    if (rank == 0 && elect_one()) {
      int s = 0, b = 0;
      uint32_t phase = 0, acc_phase = 1;
      bool ok = true;
      for (int tile = blockIdx.x >> 1; tile < tiles && ok; tile += pairs)
        for (int i = 0; i < j.KB; ++i) {
          const uint64_t da = desc_along_k(smem_u32(sa + s * T::kCodeBytes));
          const uint64_t db = desc_along_k(smem_u32(sb + s * T::kCodeBytes));
          if (!mbar_wait_for(full + s, phase, j.wait) || !mbar_wait_for(acc_free + b, acc_phase, j.wait)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 4; ++k)  // 32 elements
            tc_mma_e4m3_pair(tmem + b * T::kTile, da + 2 * k, db + 2 * k, idesc_e4m3(T::kTile, T::kTile), k > 0);
          tc_commit_pair(acc_full + b);
          tc_commit_pair(empty + s);
          if (++s == T::kStages) s = 0, phase ^= 1;
          if (++b == T::kBufs) b = 0, acc_phase ^= 1;
        }
      if (!ok) give_up();
      tc_commit_own(ended);
      mbar_wait_bounded(ended, 0);  // before the memory that they use goes
    }
  } else {
    const int half = warp >> 2;
    uint8_t* buf = so + warp * T::kOutBytes;
    int b = 0;
    uint32_t phase = 0;
    bool there = true;
    const uint32_t freed = cluster_addr(acc_free, 0);
    for (int tile = blockIdx.x >> 1; tile < tiles && there; tile += pairs) {
      const int2 at = grouped_tile(tile, tiles_m, tiles_n);
      const int64_t row0 = static_cast<int64_t>(at.x) * T::kTile + rank * T::kHalf + (warp & 3) * 32;
      const int col0 = at.y * T::kTile + half * T::kHalf;
      // past the ends any scale serves: the sums there are 0 and are not stored
      const float* sx = j.x_scales + min(row0 + lane, j.rows - 1) * j.KB;
      const float* sw = j.w_scales + min(static_cast<int64_t>(col0 / kK), (j.features - 1) / kK) * j.KB;
      // the two scales of the next block are on their way while this one's sums are added
      float fx = sx[0], fw = sw[0];
      float2 acc[T::kHalf / 2];
#pragma unroll
      for (int c = 0; c < T::kHalf / 2; ++c) acc[c] = make_float2(0.0f, 0.0f);
      for (int i = 0; i < j.KB; ++i) {
        const float2 f = dup2(fx * fw);
        if (i + 1 < j.KB) fx = sx[i + 1], fw = sw[i + 1];
        there = mbar_wait_for(acc_full + b, phase, j.wait);
        if (__any_sync(kFull, !there)) {
          there = false;
          give_up();
          break;
        }
        tc_fence_after();
        const uint32_t mine = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + b * T::kTile + half * T::kHalf;
        // 16 columns at a time, the next 16 on their way
        uint32_t v[2][16];
        tc_load16_start(mine, v[0]);
        tc_load16_wait(v[0]);
#pragma unroll
        for (int c = 0; c < T::kHalf / 16; ++c) {
          if (c + 1 < T::kHalf / 16) tc_load16_start(mine + 16 * (c + 1), v[(c + 1) & 1]);
          const uint32_t* u = v[c & 1];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            acc[8 * c + k] = pfma(make_float2(__uint_as_float(u[2 * k]), __uint_as_float(u[2 * k + 1])), f, acc[8 * c + k]);
          if (c + 1 < T::kHalf / 16) tc_load16_wait(v[(c + 1) & 1]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(freed + 8 * b);
        if (++b == T::kBufs) b = 0, phase ^= 1;
      }
      if (!there || row0 >= j.rows) continue;
#pragma unroll
      for (int c = 0; c < T::kHalf; c += T::kOutCols) {
        if (col0 + c >= j.features) break;
        // the buffer's last store has read it
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
        // a row of 128 bytes a lane, 16-byte groups in the order of the 128-byte swizzle
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          uint4 w;
          if constexpr (OUT32) {
            const float2 p = acc[c / 2 + 2 * g], q = acc[c / 2 + 2 * g + 1];
            w = make_uint4(__float_as_uint(p.x), __float_as_uint(p.y), __float_as_uint(q.x), __float_as_uint(q.y));
          } else {
            const float2* p = acc + c / 2 + 4 * g;
            w = make_uint4(pack_bf2(p[0].x, p[0].y), pack_bf2(p[1].x, p[1].y), pack_bf2(p[2].x, p[2].y),
                           pack_bf2(p[3].x, p[3].y));
          }
          *reinterpret_cast<uint4*>(buf + lane * 128 + ((g ^ (lane & 7)) * 16)) = w;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tma_store_2d(&map_out, col0 + c, static_cast<int>(row0), buf);
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncwarp();
  cluster_sync_all();  // neither CTA ends while the other's products or barriers use its memory
  if (*failed) {
    // Copies may be in flight that neither CTA can wait for (mx4_matmul.cu): no more are
    // issued, and they have the time of a wait to land in.
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
// Codes [rows, H] in boxes of 128 by box_rows.
cudaError_t codes_map(CUtensorMap* m, const void* codes, int64_t rows, int H, int box_rows) {
  return matrix_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, codes, rows, H, box_rows, kK, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

template <bool OUT32>
cudaError_t launch_wide(const Fp8MatmulArgs& a, const Job& j, cudaStream_t st) {
  using T = Wide<OUT32>;
  auto* kern = k_fp8_matmul_wide<OUT32>;
  if (cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), T::kSmem)) return e;
  CUtensorMap mx, mw, mo;
  if (cudaError_t e = codes_map(&mx, a.x_codes, a.rows, a.H, T::kHalf)) return e;
  if (cudaError_t e = codes_map(&mw, a.w_codes, a.features, a.H, T::kHalf)) return e;
  if (cudaError_t e = matrix_map(&mo, OUT32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                                 OUT32 ? 4 : 2, a.out, a.rows, a.features, 32, T::kOutCols, CU_TENSOR_MAP_SWIZZLE_128B,
                                 CU_TENSOR_MAP_L2_PROMOTION_NONE))
    return e;
  const int64_t tiles = ((a.features + T::kTile - 1) / T::kTile) * ((a.rows + T::kTile - 1) / T::kTile);
  const int64_t pairs = std::min<int64_t>(tiles, num_sms() / 2);
  return launch_pdl(kern, dim3(static_cast<unsigned>(2 * pairs)), dim3(T::kThreads), T::kSmem, st, j, mx, mw, mo);
}

template <int BN>
cudaError_t launch(const Fp8MatmulArgs& a, const Job& j, int parts, cudaStream_t st) {
  using T = Tile<BN>;
  auto* kern = k_fp8_matmul<BN>;
  if (cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), T::kSmem)) return e;
  CUtensorMap mw, mx;
  if (cudaError_t e = codes_map(&mw, a.w_codes, a.features, a.H, T::kM)) return e;
  if (cudaError_t e = codes_map(&mx, a.x_codes, a.rows, a.H, BN)) return e;
  return launch_parts(kern,
                      dim3(static_cast<unsigned>((a.features + T::kM - 1) / T::kM),
                           static_cast<unsigned>((a.rows + BN - 1) / BN), static_cast<unsigned>(parts)),
                      T::kThreads, T::kSmem, st, j, mw, mx);
}

}  // namespace

cudaError_t launch_fp8_matmul(const Fp8MatmulArgs& a, cudaStream_t st) {
  const Job j{a.x_scales, a.w_scales, a.out, a.status, a.rows, a.features, wait_cycles,
              (a.H + kK - 1) / kK, a.out_f32 ? 1 : 0};
  // Sizes are features x hidden.  Few tokens, in tiles of at most 64 (128 tokens 8192 x 8192: 23.3 us, in one tile of 128
  // 26.2): a thread of that kernel has a feature, so each token's factor is a load, and
  // the weights are read once for each tile of tokens.  k is cut into as many parts, of
  // four blocks at least, as keep two CTAs an SM; eight parts of 64 tokens only where there
  // is then one, for their join (us, 1 / 2 / 4 / 8 parts: 1 token 8192 x 8192 16.8 / 14.8 /
  // 12.5 / 15.6, 16 tokens 1024 x 8192 14.7 / 9.3 / 6.3 / 4.7, 64 tokens 4096 x 4096 15.6 /
  // 10.8 / 9.0 / 10.1).  Above 128 tokens, and where k is not cut, the persistent kernel
  // (us, it / few tokens: 300 tokens 4096 x 4096 17.3 / 21.0, 128 tokens 8192 x 8192 29.4 /
  // 23.3; with k cut 200 tokens 4096 x 4096 17.1 / 14.1, 512 tokens 2048 x 8192 29.1 / 22.7).
  const int bn = a.rows <= 16 ? 16 : a.rows <= 32 ? 32 : 64;
  const int64_t tiles = ((a.features + 127) / 128) * ((a.rows + bn - 1) / bn);
  int parts = 1;
  while (parts < kMostParts && parts * 8 <= j.KB && tiles * parts * 2 <= (bn == 64 && parts == 4 ? 1 : 2) * num_sms())
    parts *= 2;
  if (a.rows > 128 && parts == 1)
    return a.out_f32 ? launch_wide<true>(a, j, st) : launch_wide<false>(a, j, st);
  if (bn == 16) return launch<16>(a, j, parts, st);
  if (bn == 32) return launch<32>(a, j, parts, st);
  return launch<64>(a, j, parts, st);
}

}  // namespace fc
