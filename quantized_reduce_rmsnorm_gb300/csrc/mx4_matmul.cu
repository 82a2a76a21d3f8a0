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
// memory and issues the products, four warps bring the result out.
#include <cuda.h>

#include "block.h"
#include "mx4.cuh"

namespace fc {
namespace {

constexpr int kM = 128;          // features of a tile
constexpr int kStageK = 256;     // elements of k a stage: 128 bytes of codes a row
constexpr int kThreads = 192;    // warps 0-3: result; 4: copies; 5: products
constexpr int kErrCuda = 2;      // FC_ERR_CUDA

template <int BN>
struct Tile {
  static constexpr int kStages = BN >= 256 ? 4 : BN >= 128 ? 6 : 5;
  static constexpr int kSfbTiles = BN > 128 ? 2 : 1;  // 128-row scale tiles of the tokens
  static constexpr int kABytes = kM * 128, kBBytes = BN * 128;
  static constexpr int kSfBytes = 1024;               // 128 rows, 256 elements of k
  static constexpr int kStageBytes = kABytes + kBBytes + kSfBytes * (1 + kSfbTiles);
  static constexpr int kSmem = kStages * kStageBytes + 1024 + 256;
  // columns of the tensor core's memory: the accumulator, then each stage's scales
  static constexpr int kSfCols = 8 * (1 + kSfbTiles);
  static constexpr int kColsUsed = BN + kStages * kSfCols;
  static constexpr int kCols = kColsUsed <= 128 ? 128 : kColsUsed <= 256 ? 256 : 512;
};

struct Job {
  const uint8_t* x_scales;
  const uint8_t* w_scales;
  void* out;
  int32_t* status;
  int64_t rows, features;
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

// Shared-memory matrix descriptors: rows of 128 bytes with the 128-byte
// swizzle, 1024 bytes from one group of eight rows to the next; and rows of 16
// bytes without a swizzle, 128 bytes from group to group.
__device__ __forceinline__ uint64_t desc_codes(uint32_t smem) {
  return static_cast<uint64_t>((smem & 0x3FFFF) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_scales(uint32_t smem) {
  return static_cast<uint64_t>((smem & 0x3FFFF) >> 4) | (1ull << 16) | (8ull << 32) | (1ull << 46);
}
// Instruction descriptor: e2m1 by e2m1, both along k, e8m0 scales, N columns,
// 128 rows; sf: which half (0 or 2) of a scale word's four bytes.
__device__ __forceinline__ uint32_t idesc_mxf4(int N, uint32_t sf) {
  return (sf << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>(kM >> 4) << 24) | (sf << 29);
}

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      ::"r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
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
  uint8_t* ssb = ssa + T::kStages * T::kSfBytes;         // [stage][tiles][1024]
  uint64_t* full = reinterpret_cast<uint64_t*>(ssb + T::kStages * T::kSfBytes * T::kSfbTiles);
  uint64_t* empty = full + T::kStages;
  uint64_t* done = empty + T::kStages;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(done + 1);
  volatile uint32_t* failed = tmem_at + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * kM;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * BN;
  const int stages_k = (j.H + kStageK - 1) / kStageK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < T::kStages; ++s) mbar_init(full + s, 1), mbar_init(empty + s, 1);
    mbar_init(done, 1);
    *failed = 0;
    mbar_init_fence();
  }
  // taken before the next kernel may start, so that all of this grid's CTAs have theirs
  if (warp == 5) tmem_alloc(tmem_at, T::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  pdl_begin();

  if (warp == 4) {
    if (lane == 0) {
      int i = 0;
      for (; i < stages_k; ++i) {
        const int s = i % T::kStages, n = i / T::kStages;
        if (n > 0 && !mbar_wait_bounded(empty + s, (n - 1) & 1)) {
          *failed = 1;
          break;
        }
        // the last stage may hold one scale tile of k, not two
        const uint32_t sf = j.KT - 2 * i >= 2 ? 1024u : 512u;
        int sfb_tiles = 1;
        if (T::kSfbTiles == 2 && t0 + 128 < j.rows) sfb_tiles = 2;
        mbar_expect_tx(full + s, T::kABytes + T::kBBytes + sf * (1 + sfb_tiles));
        tma_load_2d(sa + s * T::kABytes, &map_w, i * 128, n0, full + s);
        tma_load_2d(sb + s * T::kBBytes, &map_x, i * 128, static_cast<int>(t0), full + s);
        bulk_load(ssa + s * T::kSfBytes, j.w_scales + (static_cast<int64_t>(blockIdx.x) * j.KT + 2 * i) * 512,
                  sf, full + s);
        for (int q = 0; q < sfb_tiles; ++q)
          bulk_load(ssb + (s * T::kSfbTiles + q) * T::kSfBytes,
                    j.x_scales + ((t0 / 128 + q) * j.KT + 2 * i) * 512, sf, full + s);
      }
      // after a failure: the copies in flight land before the CTA ends
      if (i < stages_k)
        for (int q = max(0, i - T::kStages); q < i; ++q)
          mbar_wait_bounded(full + q % T::kStages, (q / T::kStages) & 1);
    }
  } else if (warp == 5) {
    if (lane == 0) {
      for (int i = 0; i < stages_k; ++i) {
        const int s = i % T::kStages, n = i / T::kStages;
        if (!mbar_wait_bounded(full + s, n & 1)) {
          *failed = 1;
          break;
        }
        tc_fence_after();
        const uint32_t sf = tmem + BN + s * T::kSfCols;
        const int halves = j.KT - 2 * i >= 2 ? 2 : 1;  // scale tiles of k in this stage
        for (int q = 0; q < halves; ++q) {
          tc_copy_scales(sf + 4 * q, desc_scales(smem_u32(ssa + s * T::kSfBytes + q * 512)));
          for (int r = 0; r < T::kSfbTiles; ++r)  // columns: [half of k][token tile]
            tc_copy_scales(sf + 8 + 4 * (q * T::kSfbTiles + r),
                           desc_scales(smem_u32(ssb + (s * T::kSfbTiles + r) * T::kSfBytes + q * 512)));
        }
        const uint64_t da = desc_codes(smem_u32(sa + s * T::kABytes));
        const uint64_t db = desc_codes(smem_u32(sb + s * T::kBBytes));
        const int steps = min(4, (j.H - i * kStageK + 63) / 64);
        for (int k = 0; k < steps; ++k) {  // 64 elements: 32 bytes further along the row
          const int q = k >> 1;
          tc_mma_mxf4(tmem, da + 2 * k, db + 2 * k, idesc_mxf4(BN, (k & 1) * 2), sf + 4 * q,
                      sf + 8 + 4 * q * T::kSfbTiles, i > 0 || k > 0);
        }
        tc_commit(empty + s);
      }
      tc_commit(done);
    }
  } else {
    if (!mbar_wait_bounded(done, 0)) *failed = 1;
    tc_fence_after();
    __syncwarp();
    if (!*failed) {
      const int64_t f = n0 + warp * 32 + lane;
      for (int c = 0; c < BN && t0 + c < j.rows; c += 16) {
        uint32_t v[16];
        tc_load16(tmem + (static_cast<uint32_t>(warp * 32) << 16) + c, v);
        if (f < j.features) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int64_t t = t0 + c + i;
            if (t >= j.rows) break;
            if (j.out_f32)
              static_cast<float*>(j.out)[t * j.features + f] = __uint_as_float(v[i]);
            else
              static_cast<__nv_bfloat16*>(j.out)[t * j.features + f] = __float2bfloat16_rn(__uint_as_float(v[i]));
          }
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (threadIdx.x == 0 && *failed && j.status) *j.status = kErrCuda;
  if (warp == 5) {
    __syncwarp();
    tc_fence_after();
    tmem_free(tmem, T::kCols);
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

template <int BN>
cudaError_t launch(const Mx4MatmulArgs& a, const Job& j, cudaStream_t st) {
  auto* kern = k_mx4_matmul<BN>;
  if (cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), Tile<BN>::kSmem)) return e;
  CUtensorMap mw, mx;
  if (cudaError_t e = codes_map(&mw, a.w_codes, a.features, a.H, kM)) return e;
  if (cudaError_t e = codes_map(&mx, a.x_codes, a.rows, a.H, BN)) return e;
  const dim3 grid(static_cast<unsigned>((a.features + kM - 1) / kM), static_cast<unsigned>((a.rows + BN - 1) / BN));
  return launch_pdl(kern, grid, dim3(kThreads), Tile<BN>::kSmem, st, j, mw, mx);
}

}  // namespace

cudaError_t launch_mx4_matmul(const Mx4MatmulArgs& a, cudaStream_t st) {
  const Job j{a.x_scales, a.w_scales, a.out, a.status, a.rows, a.features, a.H,
              static_cast<int>(mx4_tiles_k(a.H)), a.out_f32 ? 1 : 0};
  if (a.rows <= 16) return launch<16>(a, j, st);
  if (a.rows <= 32) return launch<32>(a, j, st);
  if (a.rows <= 64) return launch<64>(a, j, st);
  if (a.rows <= 128) return launch<128>(a, j, st);
  return launch<256>(a, j, st);
}

}  // namespace fc
