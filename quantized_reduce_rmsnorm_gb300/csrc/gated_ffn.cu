// gated_ffn.cu -- the gated feed-forward block's first half and its gradient, in bf16:
//   g = x w_gate^T,  u = x w_up^T,  out = bf16(act(g) * u)
//   dg = dout * u * act'(g),  du = dout * act(g)
//   dx = dg w_gate + du w_up,  dw_gate = dg^T x,  dw_up = du^T x
// x [rows, H], weights [features, H], out, g and u [rows, features]; act is SiLU, z
// sigmoid(z), or GELU by its tanh form, z sigmoid(2 sqrt(2 / pi) (z + 0.044715 z^3)).
//
// All products are tcgen05.mma kind::f16 with binary32 sums in tensor memory; each result
// is rounded once.  Both projections share a tile's copies of x, and their sums meet in
// the thread that has a token's row of both, so g and u leave the chip only where the
// caller keeps them (in bf16, for the gradient).  dg and du go to the tensor core in bf16, by
// the workspace.  In large products one bf16 number stands for each: its rounding, at most
// 2^-8 of a term, is no more than a result's own, and independent from term to term.  In
// small ones (gated_ffn_terms), where more products cost little, and where the caller asks for
// it, each is the sum of two bf16 numbers, 16 bits of it.
// Sizes below are tokens x features x hidden, or features x hidden after the tokens.
#include <algorithm>

#include "block.h"
#include "tc.cuh"

namespace fc {
namespace {

constexpr int kK = 64;           // elements of k a stage: 128 bytes of a row
constexpr int kMostParts = 8;    // of k, in one cluster
constexpr int kErrCuda = 2;      // FC_ERR_CUDA

// sigmoid(z): the hardware's exponential and reciprocal, a few units of 2^-22; 0 below
// about -88.
__device__ __forceinline__ float sigmoid(float z) { return rcp_approx(1.0f + __expf(-z)); }
constexpr float kGeluScale = 1.5957691216f, kGeluCube = 0.044715f;  // 2 sqrt(2 / pi)
template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if (ACT == kSilu) return z * sigmoid(z);
  return z * sigmoid(kGeluScale * __fmaf_rn(kGeluCube * z * z, z, z));
}
// The activation and its slope s + z p' s (1 - s), s = sigmoid(p(z)).
template <int ACT>
__device__ __forceinline__ float2 activate_slope(float z) {
  const float zz = z * z;
  const float p = ACT == kSilu ? z : kGeluScale * __fmaf_rn(kGeluCube * zz, z, z);
  const float dp = ACT == kSilu ? 1.0f : kGeluScale * __fmaf_rn(3.0f * kGeluCube, zz, 1.0f);
  const float s = sigmoid(p), a = z * s, t = 1.0f - s;
  // far out s or 1 - s is 0, and what it multiplies may be past binary32; an infinite z has no
  // slope (infinity times 0)
  return make_float2(a, s == 0.0f || t == 0.0f ? __fmaf_rn(z, 0.0f, s) : __fmaf_rn(a, dp * t, s));
}

// ------------------------------------------------ few tokens: k in parts --
// With few tokens the weights' bytes count.  The tile's 128 rows are 64 features of the
// gate and the same 64 of the other projection, its columns are tokens: one token costs
// 16 columns, not 128 rows.  The CTAs of a cluster take the parts of k of one tile and
// leave their sums in their shared memory, where the two projections of a feature meet;
// each adds up a slice of the features over the parts, in order (no atomics).  Bound by the
// weights' bytes: one token by 8192 x 8192 41.6 us, 6.5 TB/s (0.95 of the measured copy rate).
struct FewJob {
  void* out;
  void* gate;
  void* up;
  int32_t* status;
  int64_t rows, features;
  int64_t wait;     // cycles
  int H;
};

template <int BN>
struct Few {
  static constexpr int kM = 128, kFeatures = 64, kThreads = 192;  // warps 0-3: result; 4: copies; 5: products
  static constexpr int kStages = BN >= 128 ? 3 : BN >= 64 ? 4 : BN >= 32 ? 5 : 6;  // two CTAs an SM
  static constexpr int kABytes = kM * 128, kBBytes = BN * 128;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kCols = BN < 32 ? 32 : BN;
  static constexpr int kSmem = kStages * kStageBytes + 1024 + 256;
  static_assert(2 * kCols <= 512 && 2 * (kSmem + 1024) <= 228 * 1024, "two CTAs an SM");
};

template <int BN, int ACT>
__global__ void __launch_bounds__(Few<BN>::kThreads, 2)
    k_gated_ffn(const FewJob j, const __grid_constant__ CUtensorMap map_gate, const __grid_constant__ CUtensorMap map_up,
                const __grid_constant__ CUtensorMap map_x) {
  using T = Few<BN>;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sa = base;                                    // [stage][64 rows of the gate, 64 of the other][128 bytes]
  uint8_t* sb = sa + T::kStages * T::kABytes;            // [stage][BN rows][128 bytes]
  uint64_t* full = reinterpret_cast<uint64_t*>(sb + T::kStages * T::kBBytes);
  uint64_t* empty = full + T::kStages;
  uint64_t* done = empty + T::kStages;       // the accumulator holds this part's sums
  uint64_t* ended = done + 1;                // all copies and products issued have ended
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(ended + 1);
  volatile uint32_t* failed = tmem_at + 1;
  float* part = reinterpret_cast<float*>(base);          // [BN][128] sums, when the stages are done with
  static_assert(BN * T::kM * 4 <= T::kStages * T::kStageBytes, "the sums fit where the stages were");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * T::kFeatures;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * BN;
  const int parts = gridDim.z, part_id = blockIdx.z;     // a cluster is the parts of a tile
  const int stages_k = (j.H + kK - 1) / kK;
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
      tma_prefetch_2d(&map_gate, i * kK, n0);
      tma_prefetch_2d(&map_up, i * kK, n0);
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
        mbar_expect_tx(full + s, T::kStageBytes);
        tma_load_2d(sa + s * T::kABytes, &map_gate, i * kK, n0, full + s);
        tma_load_2d(sa + s * T::kABytes + T::kABytes / 2, &map_up, i * kK, n0, full + s);
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
        const uint64_t da = desc_along_k(smem_u32(sa + s * T::kABytes));
        const uint64_t db = desc_along_k(smem_u32(sb + s * T::kBBytes));
#pragma unroll
        for (int k = 0; k < 4; ++k)  // 16 elements
          tc_mma_bf16(tmem, da + 2 * k, db + 2 * k, idesc_bf16(T::kM, BN, false, false), i > i0 || k > 0);
        tc_commit(empty + s);
        if (++s == T::kStages) s = 0, phase ^= 1;
      }
      if (ok) tc_commit(done);
      tc_commit(ended);
      mbar_wait_bounded(ended, 0);  // before the memory that they use goes
    }
  } else {
    const bool there = __all_sync(kFull, mbar_wait_for(done, 0, j.wait));
    if (!there) *failed = 1;
    mbar_wait_bounded(ended, 0);  // the sums go where the copies went
    tc_fence_after();
    __syncwarp();
    const int f = warp * 32 + lane;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(BN), j.rows - t0));
    for (int c = 0; c < tokens; c += 16) {
      uint32_t v[16];
      tc_load16(tmem + (static_cast<uint32_t>(warp * 32) << 16) + c, v);
      // a part without its sums makes NaN of the tile
#pragma unroll
      for (int i = 0; i < 16; ++i) part[(c + i) * T::kM + f] = __uint_as_float(there ? v[i] : 0x7FC00000u);
    }
    tc_fence_before();
  }
  __syncwarp();
  cluster_sync_all();  // every part's sums are in its shared memory
  const int tokens = static_cast<int>(min(static_cast<int64_t>(BN), j.rows - t0));
  const int shift = 4 - (31 - __clz(parts));  // log2 of the slice's groups of four features
  for (int k = threadIdx.x; k < tokens << shift; k += T::kThreads) {
    const int t = k >> shift, f = ((part_id << shift) + (k & ((1 << shift) - 1))) * 4;
    const float* p = part + t * T::kM + f;
    float4 v[kMostParts], w[kMostParts], g = make_float4(0.0f, 0.0f, 0.0f, 0.0f), u = g;
#pragma unroll
    for (int r = 0; r < kMostParts; ++r)
      if (r < parts) v[r] = ld_cluster(cluster_addr(p, r)), w[r] = ld_cluster(cluster_addr(p + T::kFeatures, r));
#pragma unroll
    for (int r = 0; r < kMostParts; ++r)
      if (r < parts) {
        g.x += v[r].x, g.y += v[r].y, g.z += v[r].z, g.w += v[r].w;
        u.x += w[r].x, u.y += w[r].y, u.z += w[r].z, u.w += w[r].w;
      }
    if (n0 + f < j.features) {  // a multiple of 16: all four or none
      const int64_t at = (t0 + t) * j.features + n0 + f;
      auto put = [&](void* to, float a, float b, float c, float d) {
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(to) + at) = make_uint2(pack_bf2(a, b), pack_bf2(c, d));
      };
      put(j.out, activate<ACT>(g.x) * u.x, activate<ACT>(g.y) * u.y, activate<ACT>(g.z) * u.z, activate<ACT>(g.w) * u.w);
      if (j.gate) {
        put(j.gate, g.x, g.y, g.z, g.w);
        put(j.up, u.x, u.y, u.z, u.w);
      }
    }
  }
  __syncwarp();
  cluster_sync_all();  // no part's memory goes before the others have read it
  if (threadIdx.x == 0 && *failed && j.status) *j.status = kErrCuda;
  if (warp == 5) {
    __syncwarp();
    tc_fence_after();
    tmem_free(tmem, T::kCols);
  }
}

// ------------------------------------------------- many tokens: persistent --
// A pair of CTAs (two SMs) takes tile after tile of 256 rows by 256 columns: each CTA stages
// 128 rows of A and 128 of B, and one thread of the first issues products of both
// (cta_group::2), which leave each CTA its 128 rows by all 256 columns.  Two accumulators:
// the eight result warps, each 32 rows by half the columns, round, stage and store one
// tile while the products of the next run.
//
// An operand lies along k (its rows are the matrix's rows) or across it (its rows are the
// matrix's columns, read as they lie).  The forward pass:
//   A = x, B = the gate's weight (the first CTA's half) and the other's (the second's), both
//   along k: 256 tokens by 128 features of both.
// The gradient, in one launch, so that its products share the pairs out evenly:
//   dx: A = dg, then du, along k; B = w_gate, then w_up, across;
//   dw_gate, then dw_up: A = dg, or du, across k; B = x across k;
// both once more with the second terms of dg and du where there are any.
// A pair's tiles of dx come first; pairs that have one more of them than others have
// `ahead` tiles of the weights fewer, as many as take the time of one of dx.
//
// Bound by the products: 4096 tokens by 8192 x 8192 forward 606 to 645 us, 1.7 to 1.8 PFLOP/s
// (0.9 or more of the measured burst rate, the rate of long runs under the power limit),
// the tensor pipe active 87 % of the time at 2048 x 4096 x 4096, where the last of 3.4 turns
// of the tiles leaves pairs idle; the gradient of 4096 x 8192 x 4096 650 to 711 us, of which
// the factors' kernel is 50, the tensor pipe active 94 % of the products' time (two launches
// with tiles in turn: 698; 777 x 4112 x 2064 70 us against 49).
enum Pass { kForward, kBackward };

struct Job {
  int32_t* status;
  int64_t rows, features;
  int64_t wait;        // cycles
  int H;
  int keep;            // forward: g and u are kept
  int tiles_first;     // forward: all tiles; backward: those of dx
  int tiles_weights;   // backward: those of both weights
  int ahead;
  int terms;           // backward: of dg and du
};

// The tile of a pair's turn `step`; false: it has no more.
struct Tile {
  int m, n;       // in tiles of the output
  int k_stages;
  int weights;    // backward: 0 dx, 1 dw_gate, 2 dw_up
};

struct Wide {
  static constexpr int kTile = 256, kHalf = 128;
  static constexpr int kStages = 6, kBufs = 2;
  static constexpr int kThreads = 320;  // warps 0-7: result; 8: copies; 9: products
  static constexpr int kPartBytes = kHalf * 128, kStageBytes = 2 * kPartBytes;
  static constexpr int kOutBytes = 4096;  // of a result warp: 32 rows by 64 columns
  static constexpr int kSmem = kStages * kStageBytes + 8 * kOutBytes + 1024 + 256;
  static constexpr int kCols = kBufs * kTile;
  static_assert(kCols <= 512 && kSmem <= 227 * 1024, "fits");
};

// Matrices: forward 0 x, 1 w_gate, 2 w_up; backward 0 dg, 1 du, 2 and 3 their second terms, 4
// w_gate, 5 w_up, 6 x.  Outputs: forward out, g, u; backward dx, dw_gate, dw_up.
struct Maps {
  CUtensorMap in[7], out[3];
};

template <int PASS>
__device__ __forceinline__ bool tile_of(const Job& j, int pair, int pairs, int step, Tile& t) {
  constexpr int kTileN = PASS == kForward ? Wide::kHalf : Wide::kTile;
  const int tiles_t = static_cast<int>((j.rows + Wide::kTile - 1) / Wide::kTile);  // of tokens
  int tile = pair + step * pairs;
  if (PASS == kForward || tile < j.tiles_first) {
    if (PASS == kForward && tile >= j.tiles_first) return false;
    const int cols = PASS == kForward ? static_cast<int>(j.features) : j.H;
    const int2 at = grouped_tile(tile, tiles_t, (cols + kTileN - 1) / kTileN);
    const int k = PASS == kForward ? (j.H + kK - 1) / kK : j.terms * 2 * ((static_cast<int>(j.features) + kK - 1) / kK);
    t = Tile{at.x, at.y, k, 0};
    return true;
  }
  const int extra = j.tiles_first % pairs;  // pairs with one more tile of dx
  step -= j.tiles_first / pairs + (pair < extra);
  if (pair >= extra) {
    tile = step * (pairs - extra) + pair - extra;
    if (step >= j.ahead) tile = j.ahead * (pairs - extra) + (step - j.ahead) * pairs + pair - extra;
  } else {
    tile = j.ahead * (pairs - extra) + step * pairs + pair + pairs - extra;
  }
  if (tile >= j.tiles_weights) return false;
  const int one = j.tiles_weights / 2, second = tile >= one;
  const int tiles_m = (static_cast<int>(j.features) + Wide::kTile - 1) / Wide::kTile;
  const int2 at = grouped_tile(tile - second * one, tiles_m, (j.H + Wide::kTile - 1) / Wide::kTile);
  t = Tile{at.x, at.y, j.terms * static_cast<int>((j.rows + kK - 1) / kK), 1 + second};
  return true;
}

template <int PASS, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Wide::kThreads, 1)
    k_gated_wide(const Job j, const __grid_constant__ Maps maps) {
  using T = Wide;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sa = base;                               // [stage] 128 rows of A
  uint8_t* sb = sa + T::kStages * T::kPartBytes;    // [stage] 128 of B
  uint8_t* so = sb + T::kStages * T::kPartBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(so + 8 * T::kOutBytes);  // the first CTA's: both CTAs' copies
  uint64_t* empty = full + T::kStages;
  uint64_t* acc_full = empty + T::kStages;      // [buffer] holds a tile
  uint64_t* acc_free = acc_full + T::kBufs;     // the first CTA's: both CTAs' result warps have read it
  uint64_t* ended = acc_free + T::kBufs;        // the first CTA's: all products issued have ended
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(ended + 1);
  volatile uint32_t* failed = tmem_at + 1;      // a role of either CTA gave up
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x & 1, pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;
  Tile t;

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
      for (int step = 0; ok && tile_of<PASS>(j, pair, pairs, step, t); ++step) {
        const int a0 = t.m * T::kTile + rank * T::kHalf;
        const int b0 = PASS == kForward ? t.n * T::kHalf : t.n * T::kTile + rank * T::kHalf;
        // backward: k in runs, of dg, of du (dx alone) and of their second terms
        const int run = PASS == kForward ? 0 : t.k_stages / (t.weights ? j.terms : 2 * j.terms);
        int which = PASS == kBackward && t.weights ? t.weights - 1 : 0, in_run = 0;
        for (int i = 0; i < t.k_stages; ++i) {
          if (!mbar_wait_for(empty + s, phase, j.wait)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_expect_tx(full + s, 2 * T::kStageBytes);
          const uint32_t bar = cluster_addr(full + s, 0);
          uint8_t* da = sa + s * T::kPartBytes;
          uint8_t* db = sb + s * T::kPartBytes;
          // what lies past the end of a tensor reads as 0
          if constexpr (PASS == kForward) {
            tma_load_2d_pair(da, maps.in, i * kK, a0, bar);
            tma_load_2d_pair(db, maps.in + 1 + rank, i * kK, b0, bar);
          } else {
            const int k = in_run * kK;
            const CUtensorMap* ma = maps.in + which;
            const CUtensorMap* mb = maps.in + (t.weights ? 6 : 4 + (which & 1));
            if (++in_run == run) in_run = 0, which += t.weights ? 2 : 1;
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // 64 rows of an operand each
              const int row = a0 + 64 * h;
              tma_load_2d_pair(da + h * (T::kPartBytes / 2), ma, t.weights ? row : k, t.weights ? k : row, bar);
              tma_load_2d_pair(db + h * (T::kPartBytes / 2), mb, b0 + 64 * h, k, bar);
            }
          }
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
      for (int step = 0; ok && tile_of<PASS>(j, pair, pairs, step, t); ++step) {
        if (!mbar_wait_for(acc_free + b, acc_phase, j.wait)) {
          ok = false;
          break;
        }
        const bool across = PASS == kBackward && t.weights;  // A's; B's is the pass's
        const uint32_t idesc = idesc_bf16(T::kTile, T::kTile, across, PASS == kBackward);
        const uint32_t step_a = across ? 128 : 2, step_b = PASS == kBackward ? 128 : 2;
        for (int i = 0; i < t.k_stages; ++i) {
          if (!mbar_wait_for(full + s, phase, j.wait)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = smem_u32(sa + s * T::kPartBytes), bb = smem_u32(sb + s * T::kPartBytes);
          const uint64_t da = across ? desc_across_k(a, T::kPartBytes / 2) : desc_along_k(a);
          const uint64_t db = PASS == kBackward ? desc_across_k(bb, T::kPartBytes / 2) : desc_along_k(bb);
#pragma unroll
          for (int k = 0; k < 4; ++k)  // 16 elements
            tc_mma_bf16_pair(tmem + b * T::kTile, da + step_a * k, db + step_b * k, idesc, i > 0 || k > 0);
          tc_commit_pair(empty + s);
          if (++s == T::kStages) s = 0, phase ^= 1;
        }
        if (ok) tc_commit_pair(acc_full + b);
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
    // 32 columns of the lane's row, packed, as 16-byte groups 4 q and on of its 128 bytes in
    // the order of the 128-byte swizzle
    auto put = [&](int q, const uint32_t (&w)[16]) {
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<uint4*>(buf + lane * 128 + (((4 * q + g) ^ (lane & 7)) * 16)) =
            make_uint4(w[4 * g], w[4 * g + 1], w[4 * g + 2], w[4 * g + 3]);
    };
    auto wait_stored = [&] {  // the buffer's last store has read it
      if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      __syncwarp();
    };
    auto store = [&](const CUtensorMap* map, int col, int64_t row) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tma_store_2d(map, col, static_cast<int>(row), buf);
    };
    auto release = [&] {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_addr(acc_free + b, 0));
    };
    auto pack = [](uint32_t lo, uint32_t hi) { return pack_bf2(__uint_as_float(lo), __uint_as_float(hi)); };
    for (int step = 0; tile_of<PASS>(j, pair, pairs, step, t); ++step) {
      const bool there = mbar_wait_for(acc_full + b, phase, j.wait);
      if (__any_sync(kFull, !there || *failed)) {
        give_up();
        break;
      }
      tc_fence_after();
      const uint32_t mine = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + b * T::kTile;
      const int64_t row0 = static_cast<int64_t>(t.m) * T::kTile + rank * T::kHalf + (warp & 3) * 32;
      if constexpr (PASS == kForward) {
        const int col0 = t.n * T::kHalf + half * 64;
        const bool on = row0 < j.rows && col0 < j.features;
        uint32_t pg[2][16], pu[2][16];
        wait_stored();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t g[32], u[32], w[16];
          tc_load_all<1>(mine + half * 64 + q * 32, g);
          tc_load_all<1>(mine + T::kHalf + half * 64 + q * 32, u);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            pg[q][i] = pack(g[2 * i], g[2 * i + 1]), pu[q][i] = pack(u[2 * i], u[2 * i + 1]);
            w[i] = pack_bf2(activate<ACT>(__uint_as_float(g[2 * i])) * __uint_as_float(u[2 * i]),
                            activate<ACT>(__uint_as_float(g[2 * i + 1])) * __uint_as_float(u[2 * i + 1]));
          }
          put(q, w);
        }
        release();
        if (on) store(maps.out, col0, row0);
        if (j.keep) {
          wait_stored();
          put(0, pg[0]), put(1, pg[1]);
          if (on) store(maps.out + 1, col0, row0);
          wait_stored();
          put(0, pu[0]), put(1, pu[1]);
          if (on) store(maps.out + 2, col0, row0);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int col0 = t.n * T::kTile + half * T::kHalf + c * 64;
          wait_stored();
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t v[32], w[16];
            tc_load_all<1>(mine + half * T::kHalf + c * 64 + q * 32, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = pack(v[2 * i], v[2 * i + 1]);
            put(q, w);
          }
          if (c == 1) release();
          if (row0 < (t.weights ? j.features : j.rows) && col0 < j.H) store(maps.out + t.weights, col0, row0);
        }
      }
      if (++b == T::kBufs) b = 0, phase ^= 1;
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

// ------------------------------------- gradient of few tokens: k in parts --
// dx of few tokens: again the weights' bytes count.  The tile's 128 rows are columns
// of the weights (read across k, as they lie), its columns tokens: the first terms of dg and
// du, then as many columns of the second terms, whose products cost no more bytes.  The
// cluster's CTAs take the parts of k, which runs over the gate's features and then over the
// other's, and join their sums as above.  The whole gradient of 64 tokens, 4096 x 4096: 37.8
// us, of which the bytes of the weights and their gradients take 20 (with every product in
// the kernel of many tokens, and one term, 43.9).
struct FewDxJob {
  void* dx;
  int32_t* status;
  int64_t rows;
  int64_t wait;     // cycles
  int H;
  int run;          // stages of k of one weight
};

template <int BN>
struct FewDx {
  static constexpr int kM = 128, kThreads = 192;  // warps 0-3: result; 4: copies; 5: products
  static constexpr int kN = 2 * BN;
  static constexpr int kPerSm = BN >= 128 ? 1 : 2;  // CTAs
  static constexpr int kStages = BN >= 128 ? 4 : BN >= 64 ? 3 : BN >= 32 ? 4 : 5;
  static constexpr int kABytes = kM * 128, kBBytes = kN * 128;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kSmem = kStages * kStageBytes + 1024 + 256;
  static_assert(kPerSm * kN <= 512 && kPerSm * (kSmem + 1024) <= 228 * 1024, "fits");
};

template <int BN>
__global__ void __launch_bounds__(FewDx<BN>::kThreads, FewDx<BN>::kPerSm)
    k_gated_dx(const FewDxJob j, const __grid_constant__ Maps maps) {
  using T = FewDx<BN>;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sa = base;                                    // [stage][two blocks of 64 columns][64 k][128 bytes]
  uint8_t* sb = sa + T::kStages * T::kABytes;            // [stage][first terms, second terms][BN rows][128 bytes]
  uint64_t* full = reinterpret_cast<uint64_t*>(sb + T::kStages * T::kBBytes);
  uint64_t* empty = full + T::kStages;
  uint64_t* done = empty + T::kStages;       // the accumulator holds this part's sums
  uint64_t* ended = done + 1;                // all copies and products issued have ended
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(ended + 1);
  volatile uint32_t* failed = tmem_at + 1;
  float* part = reinterpret_cast<float*>(base);          // [BN][128] sums, when the stages are done with
  static_assert(BN * T::kM * 4 <= T::kStages * T::kStageBytes, "the sums fit where the stages were");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * T::kM;
  const int parts = gridDim.z, part_id = blockIdx.z;     // a cluster is the parts of a tile
  const int i0 = 2 * j.run * part_id / parts, i1 = 2 * j.run * (part_id + 1) / parts;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * BN;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(BN), j.rows - t0));

  if (threadIdx.x == 0) {
    for (int s = 0; s < T::kStages; ++s) mbar_init(full + s, 1), mbar_init(empty + s, 1);
    mbar_init(done, 1), mbar_init(ended, 2);
    *failed = 0;
    mbar_init_fence();
  }
  // taken before the next kernel may start, so that all of this grid's CTAs have theirs
  if (warp == 5) tmem_alloc(tmem_at, T::kN);
  if (warp == 4 && elect_one())
    for (int i = i0; i < i1 && i < i0 + T::kStages; ++i) {
      const CUtensorMap* w = maps.in + 4 + (i >= j.run);
      const int k = (i >= j.run ? i - j.run : i) * kK;
      tma_prefetch_2d(w, n0, k);
      tma_prefetch_2d(w, n0 + 64, k);
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
        const int which = i >= j.run, k = (i - which * j.run) * kK;
        mbar_expect_tx(full + s, T::kStageBytes);
        tma_load_2d(sa + s * T::kABytes, maps.in + 4 + which, n0, k, full + s);
        tma_load_2d(sa + s * T::kABytes + T::kABytes / 2, maps.in + 4 + which, n0 + 64, k, full + s);
        tma_load_2d(sb + s * T::kBBytes, maps.in + which, k, static_cast<int>(t0), full + s);
        tma_load_2d(sb + s * T::kBBytes + T::kBBytes / 2, maps.in + 2 + which, k, static_cast<int>(t0), full + s);
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
        const uint64_t da = desc_across_k(smem_u32(sa + s * T::kABytes), T::kABytes / 2);
        const uint64_t db = desc_along_k(smem_u32(sb + s * T::kBBytes));
#pragma unroll
        for (int k = 0; k < 4; ++k)  // 16 elements
          tc_mma_bf16(tmem, da + 128 * k, db + 2 * k, idesc_bf16(T::kM, T::kN, true, false), i > i0 || k > 0);
        tc_commit(empty + s);
        if (++s == T::kStages) s = 0, phase ^= 1;
      }
      if (ok) tc_commit(done);
      tc_commit(ended);
      mbar_wait_bounded(ended, 0);  // before the memory that they use goes
    }
  } else {
    const bool there = __all_sync(kFull, mbar_wait_for(done, 0, j.wait));
    if (!there) *failed = 1;
    mbar_wait_bounded(ended, 0);  // the sums go where the copies went
    tc_fence_after();
    __syncwarp();
    const uint32_t mine = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    for (int c = 0; c < tokens; c += 16) {
      uint32_t v[16], u[16];
      tc_load16(mine + c, v);
      tc_load16(mine + BN + c, u);
      // a part without its sums makes NaN of the tile
#pragma unroll
      for (int i = 0; i < 16; ++i)
        part[(c + i) * T::kM + warp * 32 + lane] =
            there ? __uint_as_float(v[i]) + __uint_as_float(u[i]) : __uint_as_float(0x7FC00000u);
    }
    tc_fence_before();
  }
  __syncwarp();
  cluster_sync_all();  // every part's sums are in its shared memory
  const int shift = 5 - (31 - __clz(parts));  // log2 of the slice's groups of four columns
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
    if (n0 + f < j.H)  // a multiple of 16: all four or none
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(j.dx) + (t0 + t) * j.H + n0 + f) =
          make_uint2(pack_bf2(s.x, s.y), pack_bf2(s.z, s.w));
  }
  __syncwarp();
  cluster_sync_all();  // no part's memory goes before the others have read it
  if (threadIdx.x == 0 && *failed && j.status) *j.status = kErrCuda;
  if (warp == 5) {
    __syncwarp();
    tc_fence_after();
    tmem_free(tmem, T::kN);
  }
}

// --------------------------------------------------- gradient's factors ---
// v less its rounding r; 0 where r is not finite.
__device__ __forceinline__ float2 rest(float2 v, float2 r) {
  auto one = [](float a, float b) { return fabsf(b) < __uint_as_float(0x7F800000u) ? a - b : 0.0f; };
  return make_float2(one(v.x, r.x), one(v.y, r.y));
}

// dg and du of 16 neighbouring elements a thread.  Bound by memory: three tensors in, two out,
// 2048 x 4096 13.2 us, 6.4 TB/s.
template <int ACT, int TERMS>
__global__ void __launch_bounds__(256)
    k_gated_factors(const void* gate, const void* up, const void* dout, int64_t pieces, void* dg, void* du, void* dg2,
                    void* du2) {
  pdl_begin();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= pieces) return;
  const Raw<false, 16> g = load_raw<false, 16>(gate, i * 16), u = load_raw<false, 16>(up, i * 16),
                       d = load_raw<false, 16>(dout, i * 16);
  float2 a[8], b[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 z = pair<false, 16>(g, k), o = pair<false, 16>(d, k);
    const float2 x = activate_slope<ACT>(z.x), y = activate_slope<ACT>(z.y);
    a[k] = pmul(pmul(o, pair<false, 16>(u, k)), make_float2(x.y, y.y));
    b[k] = pmul(o, make_float2(x.x, y.x));
  }
  const Raw<false, 16> ra = pack_raw<false, 16>(a), rb = pack_raw<false, 16>(b);
  store_raw<false, 16>(dg, i * 16, ra);
  store_raw<false, 16>(du, i * 16, rb);
  if constexpr (TERMS == 2) {  // what the rounding left; of an infinity or a NaN nothing more
#pragma unroll
    for (int k = 0; k < 8; ++k) a[k] = rest(a[k], pair<false, 16>(ra, k)), b[k] = rest(b[k], pair<false, 16>(rb, k));
    store_raw<false, 16>(dg2, i * 16, pack_raw<false, 16>(a));
    store_raw<false, 16>(du2, i * 16, pack_raw<false, 16>(b));
  }
}

// ------------------------------------------------------------- launch ----
// A bf16 matrix in boxes of 64 columns (128 bytes, swizzled) by box_rows rows.
cudaError_t bf16_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int box_rows) {
  return matrix_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p, rows, cols, box_rows, 64, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

template <int PASS, int ACT>
cudaError_t launch_wide(Job j, const Maps& maps, cudaStream_t st) {
  auto* kern = k_gated_wide<PASS, ACT>;
  if (cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), Wide::kSmem)) return e;
  const int pairs = std::min(j.tiles_first + j.tiles_weights, num_sms() / 2);
  // as many tiles of the weights as take the time of one of dx, by their stages of k and
  // about eight that a tile takes besides
  const int64_t k_in = j.terms * 2 * ((j.features + kK - 1) / kK) + 8, k_weights = j.terms * ((j.rows + kK - 1) / kK) + 8;
  j.ahead = static_cast<int>((k_in + k_weights / 2) / k_weights);
  return launch_pdl(kern, dim3(static_cast<unsigned>(2 * pairs)), dim3(Wide::kThreads), Wide::kSmem, st, j, maps);
}

template <int BN>
cudaError_t launch_few_dx(const GatedFfnGradArgs& a, Maps m, cudaStream_t st) {
  using T = FewDx<BN>;
  if (cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(k_gated_dx<BN>), T::kSmem)) return e;
  auto* ws = static_cast<__nv_bfloat16*>(a.ws);
  for (int k = 0; k < 4; ++k)
    if (cudaError_t e = bf16_map(m.in + k, ws + k * a.rows * a.features, a.rows, a.features, BN)) return e;
  const int run = static_cast<int>((a.features + kK - 1) / kK);
  const int64_t tiles_h = (a.H + T::kM - 1) / T::kM, tiles_t = (a.rows + BN - 1) / BN;
  int parts = 1;
  while (parts < kMostParts && parts * 8 <= 2 * run && tiles_h * tiles_t * parts * 2 <= T::kPerSm * num_sms()) parts *= 2;
  const FewDxJob j{a.dx, a.status, a.rows, wait_cycles, a.H, run};
  return launch_parts(k_gated_dx<BN>,
                      dim3(static_cast<unsigned>(tiles_h), static_cast<unsigned>(tiles_t), static_cast<unsigned>(parts)),
                      T::kThreads, T::kSmem, st, j, m);
}

int wide_tiles(int64_t rows, int64_t cols, int of_cols) {
  return static_cast<int>((rows + Wide::kTile - 1) / Wide::kTile * ((cols + of_cols - 1) / of_cols));
}

template <int BN>
cudaError_t launch_few(const GatedFfnArgs& a, int parts, cudaStream_t st) {
  using T = Few<BN>;
  auto* kern = a.activation == kSilu ? k_gated_ffn<BN, kSilu> : k_gated_ffn<BN, kGeluTanh>;
  if (cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), T::kSmem)) return e;
  CUtensorMap mg, mu, mx;
  if (cudaError_t e = bf16_map(&mg, a.w_gate, a.features, a.H, T::kFeatures)) return e;
  if (cudaError_t e = bf16_map(&mu, a.w_up, a.features, a.H, T::kFeatures)) return e;
  if (cudaError_t e = bf16_map(&mx, a.x, a.rows, a.H, BN)) return e;
  const FewJob j{a.out, a.gate, a.up, a.status, a.rows, a.features, wait_cycles, a.H};
  return launch_parts(kern,
                      dim3(static_cast<unsigned>((a.features + T::kFeatures - 1) / T::kFeatures),
                           static_cast<unsigned>((a.rows + BN - 1) / BN), static_cast<unsigned>(parts)),
                      T::kThreads, T::kSmem, st, j, mg, mu, mx);
}

}  // namespace

cudaError_t launch_gated_ffn(const GatedFfnArgs& a, cudaStream_t st) {
  // A tile of 128 tokens where k is then cut in four at most: the join of eight parts takes
  // longer than reading the weights twice (us, tiles of 128 / 64 tokens: 200 x 1024 x 4096
  // 16.3 / 11.2; 200 x 4096 x 4096 21.6 / 24.9; 100 x 4096 x 4096 17.8 / 19.3).
  const bool small = (a.features + 63) / 64 * ((a.rows + 127) / 128) * 4 <= num_sms();
  const int bn = a.rows <= 16 ? 16 : a.rows <= 32 ? 32 : a.rows <= 64 || small ? 64 : 128;
  const int64_t stages = (a.H + kK - 1) / kK;
  const int64_t tiles = ((a.features + 63) / 64) * ((a.rows + bn - 1) / bn);
  // k in as many parts, of four stages at least, as keep two CTAs an SM, as for the 8-bit
  // product (us, 1 / 2 / 4 / 8 parts: 1 token 8192 x 8192 47.1 / 41.6 / 43.4 / 46.3, 1 token
  // 4096 x 4096 16.9 / 14.8 / 12.6 / 15.7, 64 tokens 2048 x 4096 21.8 / 14.0 / 11.5 / 12.8).
  // Above 128 tokens, and where k is not cut, the persistent kernel (us, it / few tokens: 333
  // tokens 4112 x 2064 16.0 / 23.6; with k cut 200 tokens 4096 x 4096 23.3 / 21.0, 512 tokens
  // 2048 x 4096 22.7 / 19.9).
  int parts = 1;
  while (parts < kMostParts && parts * 8 <= stages && tiles * parts * 2 <= (bn == 64 && parts == 4 ? 1 : 2) * num_sms())
    parts *= 2;
  if (a.rows > 128 && parts == 1) {
    Maps m{};
    if (cudaError_t e = bf16_map(m.in, a.x, a.rows, a.H, Wide::kHalf)) return e;
    if (cudaError_t e = bf16_map(m.in + 1, a.w_gate, a.features, a.H, Wide::kHalf)) return e;
    if (cudaError_t e = bf16_map(m.in + 2, a.w_up, a.features, a.H, Wide::kHalf)) return e;
    if (cudaError_t e = bf16_map(m.out, a.out, a.rows, a.features, 32)) return e;
    if (a.gate) {
      if (cudaError_t e = bf16_map(m.out + 1, a.gate, a.rows, a.features, 32)) return e;
      if (cudaError_t e = bf16_map(m.out + 2, a.up, a.rows, a.features, 32)) return e;
    }
    const Job j{a.status, a.rows, a.features, wait_cycles, a.H, a.gate != nullptr,
                wide_tiles(a.rows, a.features, Wide::kHalf), 0, 0, 1};
    return a.activation == kSilu ? launch_wide<kForward, kSilu>(j, m, st) : launch_wide<kForward, kGeluTanh>(j, m, st);
  }
  if (bn == 16) return launch_few<16>(a, parts, st);
  if (bn == 32) return launch_few<32>(a, parts, st);
  if (bn == 64) return launch_few<64>(a, parts, st);
  return launch_few<128>(a, parts, st);
}

cudaError_t launch_gated_ffn_grad(const GatedFfnGradArgs& a, cudaStream_t st) {
  const int64_t n = a.rows * a.features;
  const int terms = a.terms;
  auto* ws = static_cast<__nv_bfloat16*>(a.ws);  // [term][dg, du][rows, features]
  auto* factors = terms == 2 ? a.activation == kSilu ? k_gated_factors<kSilu, 2> : k_gated_factors<kGeluTanh, 2>
                             : a.activation == kSilu ? k_gated_factors<kSilu, 1> : k_gated_factors<kGeluTanh, 1>;
  if (cudaError_t e = launch_pdl(factors, dim3(static_cast<unsigned>((n / 16 + 255) / 256)), dim3(256), 0, st, a.gate,
                                 a.up, a.dout, n / 16, static_cast<void*>(ws), static_cast<void*>(ws + n),
                                 static_cast<void*>(ws + 2 * n), static_cast<void*>(ws + 3 * n)))
    return e;
  Maps m{};
  for (int k = 0; k < 2 * terms; ++k)
    if (cudaError_t e = bf16_map(m.in + k, ws + k * n, a.rows, a.features, 64)) return e;
  if (cudaError_t e = bf16_map(m.in + 4, a.w_gate, a.features, a.H, 64)) return e;
  if (cudaError_t e = bf16_map(m.in + 5, a.w_up, a.features, a.H, 64)) return e;
  if (cudaError_t e = bf16_map(m.in + 6, a.x, a.rows, a.H, 64)) return e;
  bool wide_dx = a.dx != nullptr;
  // dx with k in parts, where k is long enough to pay for a launch of its own (us, two terms
  // either way, in parts / with the weights' products: 64 x 4096 x 4096 37.8 / 76.6, 128 x 8192 x
  // 4096 76 / 153, 64 x 496 x 4096 14.8 / 16.3, 64 x 384 x 1024 13.2 / 12.3, 128 x 256 x 4096 16.2 /
  // 11.5): of up to 128 tokens, and of more where tiles of 128 leave SMs idle and k is long
  // beside the tokens (140 x 3696 x 4096 53 / 72, 300 x 1024 x 512 17.8 / 23.7, 500 x 1024 x 512
  // 26.8 / 24.9).  That kernel takes two terms and no other number of them: with one, above
  // 2^19 factors, dx is made with the weights' products, which is faster next to the border
  // where there are columns enough (us, one term in one launch / two in parts: 140 x 3792 x
  // 4096 42.5 / 54.2) and slower where there are few (129 x 4112 x 1024 42.6 / 28.1, 300 x
  // 4112 x 512 44.5 / 26.4): a caller who asks for two terms gets the second figures.
  const int64_t tiles = (a.H + 127) / 128 * ((a.rows + 127) / 128);
  const bool long_k = a.features >= kFewDxFeatures && a.features >= 3 * a.rows && tiles * 2 <= num_sms();
  if (a.dx && (a.rows <= kFewDx ? a.features >= kFewDxFeatures : terms == 2 && long_k)) {
    if (cudaError_t e = a.rows <= 16   ? launch_few_dx<16>(a, m, st)
                        : a.rows <= 32 ? launch_few_dx<32>(a, m, st)
                        : a.rows <= 64 ? launch_few_dx<64>(a, m, st)
                                       : launch_few_dx<128>(a, m, st))
      return e;
    wide_dx = false;
    if (!a.dw_gate) return cudaSuccess;
  }
  if (wide_dx)
    if (cudaError_t e = bf16_map(m.out, a.dx, a.rows, a.H, 32)) return e;
  if (a.dw_gate) {
    if (cudaError_t e = bf16_map(m.out + 1, a.dw_gate, a.features, a.H, 32)) return e;
    if (cudaError_t e = bf16_map(m.out + 2, a.dw_up, a.features, a.H, 32)) return e;
  }
  const Job j{a.status, a.rows, a.features, wait_cycles, a.H, 0, wide_dx ? wide_tiles(a.rows, a.H, Wide::kTile) : 0,
              a.dw_gate ? 2 * wide_tiles(a.features, a.H, Wide::kTile) : 0, 0, terms};
  return launch_wide<kBackward, kSilu>(j, m, st);
}

}  // namespace fc
