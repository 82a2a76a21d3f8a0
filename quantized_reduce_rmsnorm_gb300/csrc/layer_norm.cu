// layer_norm.cu -- residual add and layer norm, one pass over the rows:
//   h = T(x + r)            (h = x without a residual)
//   m = mean(h),  inv = 1 / sqrt(mean((h - m)^2) + eps)
//   y = T((h - m) * inv * weight + bias)
// T is the rows' type (bf16 or fp32).  h is rounded once, where it is stored, and y is
// the norm of the h that is stored.  Everything else is binary32.
//
// The variance is that of values about the mean, never a difference of two large
// sums: a row in registers is summed twice.  The first sum's rounding leaves m off by a
// few steps of the mean; the second sum takes the values' distances to it along with
// their squares, and their mean, d, corrects both: the row's mean is m + d and its
// variance mean((h - m)^2) - d^2, where d^2 is far below the first term's rounding unless
// the row is all but constant.
//
// Bound by memory: x and r in, h and y out.  As in block_norm.cu a CTA holds a row in
// registers, rows that fit one warp take one each, weights come from L1 where they are
// used, and rows start for L2 before a CTA takes them.  Measured on GB300, inputs changing
// from call to call: 8192 x 8192 bf16 with a residual 78.4 us, 6.8 TB/s (all of the measured
// copy rate), without 51.3 (0.77: issue and two block sums a row); 1037 x 5120 fp32 with
// 15.5, without 11.1; one row of 4096 3.0, the host's launch.
#include <algorithm>

#include "block.h"
#include "mx4.cuh"

namespace fc {
namespace {

// Sums of two values over the row's threads (red: 64 floats of its own).
__device__ __forceinline__ float2 row_sum2(float2 v, float* red, bool one_warp) {
  v.x = warp_sum(v.x), v.y = warp_sum(v.y);
  if (one_warp) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v.x, red[32 + (threadIdx.x >> 5)] = v.y;
  __syncthreads();
  const int n = (blockDim.x + 31) >> 5, l = threadIdx.x & 31;
  return make_float2(warp_sum(l < n ? red[l] : 0.0f), warp_sum(l < n ? red[32 + l] : 0.0f));
}

// One row, by its team: TEAM one warp, else the CTA.  hr: the thread's columns of x.
template <bool F32, int W, bool TEAM>
__device__ __forceinline__ void norm_row(const LayerNormArgs& a, Raw<F32, W> hr, int64_t row, int e, bool live,
                                         float (&red)[3][32]) {
  const int64_t at = row * a.H + e;
  const float inv_n = 1.0f / static_cast<float>(a.H);
  float2 ss = make_float2(0.0f, 0.0f);
  if (live) {
    if (a.res_in) {
      const Raw<F32, W> rr = load_raw<F32, W>(a.res_in, at);
      float2 u[W / 2];
#pragma unroll
      for (int i = 0; i < W / 2; ++i) u[i] = padd(pair<F32, W>(hr, i), pair<F32, W>(rr, i));
      hr = pack_raw<F32, W>(u);
      store_raw<F32, W>(a.res_out, at, hr);
    }
#pragma unroll
    for (int i = 0; i < W / 2; ++i) ss = padd(ss, pair<F32, W>(hr, i));
  }
  const float mean = row_sum(ss.x + ss.y, red[0], TEAM) * inv_n;
  float2 s1 = make_float2(0.0f, 0.0f), s2 = s1;
  const float2 minus = dup2(-mean);
  if (live)
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
      const float2 c = padd(pair<F32, W>(hr, i), minus);
      s1 = padd(s1, c);
      s2 = pfma(c, c, s2);
    }
  const float2 s = row_sum2(make_float2(s1.x + s1.y, s2.x + s2.y), red[1], TEAM);
  const float d = s.x * inv_n;
  const float var = __fmaf_rn(-d, d, s.y * inv_n);
  const float inv = inv_sqrt((var < 0.0f ? 0.0f : var) + a.eps);  // NaN stays
  if (a.stats && e == 0) *reinterpret_cast<float2*>(a.stats + 2 * row) = make_float2(mean + d, inv);
  if (!live) return;
  const float2 vi = dup2(inv), shift = dup2(-d * inv);
  float2 u[W / 2];
#pragma unroll
  for (int i = 0; i < W / 2; ++i) u[i] = pfma(padd(pair<F32, W>(hr, i), minus), vi, shift);
  if (a.weight && a.bias) {
    const Raw<F32, W> w = load_weight<F32, W>(a.weight, e), b = load_weight<F32, W>(a.bias, e);
#pragma unroll
    for (int i = 0; i < W / 2; ++i) u[i] = pfma(u[i], pair<F32, W>(w, i), pair<F32, W>(b, i));
  } else if (a.weight) {
    const Raw<F32, W> w = load_weight<F32, W>(a.weight, e);
#pragma unroll
    for (int i = 0; i < W / 2; ++i) u[i] = pmul(u[i], pair<F32, W>(w, i));
  } else if (a.bias) {
    const Raw<F32, W> b = load_weight<F32, W>(a.bias, e);
#pragma unroll
    for (int i = 0; i < W / 2; ++i) u[i] = padd(u[i], pair<F32, W>(b, i));
  }
  store_raw<F32, W>(a.y, at, pack_raw<F32, W>(u));
}

// TEAM: one warp a row, four rows a CTA; else one row a CTA.  W: columns of a thread.
template <bool F32, int W, bool TEAM, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) k_layer_norm(const LayerNormArgs a) {
  __shared__ float red[3][32];
  pdl_begin();
  const uint32_t row = TEAM ? blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
  const int e = (TEAM ? threadIdx.x & 31 : threadIdx.x) * W;
  if (row >= a.rows) return;  // TEAM only: a whole warp
  const bool live = e < a.H;
  if (!TEAM && threadIdx.x == 0 && row + a.ahead < a.rows) {
    const uint32_t bytes = a.H * (F32 ? 4 : 2);
    const int64_t off = static_cast<int64_t>(row + a.ahead) * bytes;
    prefetch_l2(static_cast<const char*>(a.x) + off, bytes);
    if (a.res_in) prefetch_l2(static_cast<const char*>(a.res_in) + off, bytes);
  }
  Raw<F32, W> hr;
  if (live) hr = load_raw<F32, W>(a.x, static_cast<int64_t>(row) * a.H + e);
  norm_row<F32, W, TEAM>(a, hr, row, e, live, red);
}

// A CTA takes row after row, without a residual: the next row's loads are on their way while
// this one is summed (with a residual the four streams fill the memory's time as they are).
template <bool F32, int W, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) k_layer_norm_rows(const LayerNormArgs a) {
  __shared__ float red[3][32];
  pdl_begin();
  const int e = threadIdx.x * W;
  const bool live = e < a.H;
  Raw<F32, W> next;
  if (live) next = load_raw<F32, W>(a.x, static_cast<int64_t>(blockIdx.x) * a.H + e);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const Raw<F32, W> hr = next;
    if (live && row + gridDim.x < a.rows) next = load_raw<F32, W>(a.x, (row + gridDim.x) * a.H + e);
    norm_row<F32, W, false>(a, hr, row, e, live, red);
  }
}

// MINB: CTAs an SM with a residual, of one row each; ROWS: without one, of rows in turn.
template <bool F32, int W, int MAXT, int MINB, int ROWS>
cudaError_t launch_rows(const LayerNormArgs& a, cudaStream_t st) {
  const int threads = (a.H / W + 31) / 32 * 32;
  if (a.res_in)
    return launch_pdl(k_layer_norm<F32, W, false, MAXT, MINB>, dim3(static_cast<unsigned>(a.rows)), dim3(threads), 0, st, a);
  auto* kern = k_layer_norm_rows<F32, W, MAXT, ROWS>;
  const int occ = occupancy_memo(reinterpret_cast<const void*>(kern), threads, 0, 1, [&] {
    int v = 0;
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&v, kern, threads, 0);
    return v;
  });
  const int64_t ctas = std::min<int64_t>(a.rows, static_cast<int64_t>(num_sms()) * std::max(occ, 1));
  return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(threads), 0, st, a);
}
template <bool F32, int W>
cudaError_t launch_teams(const LayerNormArgs& a, cudaStream_t st) {
  return launch_pdl(k_layer_norm<F32, W, true, 128, 1>, dim3(static_cast<unsigned>((a.rows + 3) / 4)), dim3(128), 0, st,
                    a);
}

}  // namespace

cudaError_t launch_layer_norm(bool f32, LayerNormArgs a, cudaStream_t st) {
  a.ahead = num_sms();
  // CTAs an SM with a residual, one row each (us, two / three, bf16 rows of 8192: 300 5.7 /
  // 6.4, 600 9.5 / 10.7, 8192 78.4 / 79.1; fp32, two / three, 1037 rows of 5120 15.9 / 15.5),
  // and without one, rows in turn (two / three CTAs: 300 3.5 / 4.7, 8192 53.7 / 56.1 with
  // the steps of then; one row a CTA 58.3).
  if (!f32) {
    if (a.H <= 512) return launch_teams<false, 16>(a, st);
    return a.H > 8192 ? launch_rows<false, 16, 1024, 1, 1>(a, st) : launch_rows<false, 16, 512, 2, 2>(a, st);
  }
  if (a.H <= 256) return launch_teams<true, 8>(a, st);
  if (a.H <= 5120) return launch_rows<true, 8, 640, 3, 2>(a, st);
  return a.H <= 8192 ? launch_rows<true, 8, 1024, 1, 1>(a, st) : launch_rows<true, 16, 1024, 1, 1>(a, st);
}

}  // namespace fc
