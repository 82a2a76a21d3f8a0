// grad_rows.cuh -- what the gradients of the norms share: rows in columns of a CTA's
// threads, sums over a cluster's memory, and the join of the CTAs' sums over rows.
#pragma once

#include "mx4.cuh"

namespace fc {

// A thread has W columns, in groups of 16 bytes, the live threads side by side: no bank
// conflicts where the row is in shared memory.
template <bool F32, int W>
struct Cols {
  static constexpr int kPer = F32 ? 4 : 8;  // columns of a group
  static constexpr int kGroups = W / kPer;
  // first column of group j of thread t, `live` threads in all
  static __device__ __forceinline__ int at(int j, int t, int live) { return (j * live + t) * kPer; }
};

template <bool F32, int W>
struct RawCols {
  uint4 g[Cols<F32, W>::kGroups];
};
// The thread's columns of a row (or of a weight), from shared or global memory.
template <bool F32, int W>
__device__ __forceinline__ RawCols<F32, W> load_cols(const void* row, int t, int live) {
  constexpr int es = F32 ? 4 : 2;
  RawCols<F32, W> r;
#pragma unroll
  for (int j = 0; j < Cols<F32, W>::kGroups; ++j)
    r.g[j] = *reinterpret_cast<const uint4*>(static_cast<const char*>(row) + Cols<F32, W>::at(j, t, live) * es);
  return r;
}
// Columns 2i and 2i + 1 of them.
template <bool F32, int W>
__device__ __forceinline__ float2 pair(const RawCols<F32, W>& r, int i) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(r.g);
  if constexpr (F32) return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  return make_float2(bf_lo(w[i]), bf_hi(w[i]));
}
template <bool F32, int W>
__device__ __forceinline__ void store_cols(void* row, int t, int live, const float2 f[W / 2]) {
  constexpr int es = F32 ? 4 : 2, kPairs = Cols<F32, W>::kPer / 2;
#pragma unroll
  for (int j = 0; j < Cols<F32, W>::kGroups; ++j) {
    const float2* v = f + j * kPairs;
    uint4 w;
    if constexpr (F32)
      w = make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
    else
      w = make_uint4(pack_bf2(v[0].x, v[0].y), pack_bf2(v[1].x, v[1].y), pack_bf2(v[2].x, v[2].y),
                     pack_bf2(v[3].x, v[3].y));
    st128(static_cast<char*>(row) + Cols<F32, W>::at(j, t, live) * es, w);
  }
}
// The same columns of a row of fp32 sums.
template <bool F32, int W>
__device__ __forceinline__ void store_sums(float* row, int t, int live, const float2 f[W / 2]) {
  constexpr int kPer = Cols<F32, W>::kPer;
#pragma unroll
  for (int k = 0; k < W / 4; ++k) {  // four columns at a time
    const int at = Cols<F32, W>::at(4 * k / kPer, t, live) + 4 * k % kPer;
    *reinterpret_cast<float4*>(row + at) = make_float4(f[2 * k].x, f[2 * k].y, f[2 * k + 1].x, f[2 * k + 1].y);
  }
}

// A float to another CTA of the cluster; the rows of its memory in which a row's sums meet,
// one float for each warp of each CTA, an odd number of 16-byte groups a row: no bank conflicts.
__device__ __forceinline__ void st_cluster(uint32_t at, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}
template <int CL>
struct Red {
  static constexpr int kEntries = CL == 1 ? 32 : 64, kStride = kEntries + 4;
};

constexpr int kSumWarps = 16, kSumCols = 64, kSumBatch = 10;
// Adds n rows of sums, columns col and col + 1 (64 columns a CTA, a lane has two), 16
// warps over the addends, in a fixed order.  true: this thread (of the first warp) has
// the sums of its columns in s.
__device__ __forceinline__ bool column_sums(const float* src, int n, int H, int col, float2 (&red)[kSumWarps][32],
                                            float2& s) {
  const int l = threadIdx.x & 31, w = threadIdx.x >> 5;
  const float2 zero = make_float2(0.0f, 0.0f);
  s = zero;
  if (col < H)
    for (int i0 = w; i0 < n; i0 += kSumWarps * kSumBatch) {  // loads that do not wait for one another
      float2 v[kSumBatch];
#pragma unroll
      for (int k = 0; k < kSumBatch; ++k) {
        const int i = i0 + k * kSumWarps;
        v[k] = i < n ? *reinterpret_cast<const float2*>(src + static_cast<int64_t>(i) * H + col) : zero;
      }
#pragma unroll
      for (int k = 0; k < kSumBatch; ++k) s = padd(s, v[k]);
    }
  red[w][l] = s;
  __syncthreads();
  if (w != 0 || col >= H) return false;
#pragma unroll
  for (int i = 1; i < kSumWarps; ++i) s = padd(s, red[i][l]);
  return true;
}

}  // namespace fc
