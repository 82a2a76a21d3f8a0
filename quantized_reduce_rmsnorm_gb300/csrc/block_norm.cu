// block_norm.cu -- the norms before and after a block with its gate and
// residual scale, one pass over the rows:
//   u = x                          or  (x * inv_x) * post_weight
//   h = T(alpha * r + beta * (gate * u))
//   y = T((h * inv_h) * pre_weight), inv = 1 / sqrt(mean of squares + eps)
// T is the rows' type (bf16 or fp32).  h is rounded once, where it is stored,
// and y is the norm of the h that is stored: the same as the norm run alone on
// the residual stream.  Everything else is binary32.
//
// Bound by memory: x and r in, h and y out.  One CTA holds one row in
// registers (16 neighbouring elements a thread, so a warp's loads and stores
// cover 1 KB), and each row is read once.  Rows of at most 512 elements take
// one warp each.  The quantised y (mx4.cuh) leaves from the registers that
// hold it.
#include "block.h"
#include "mx4.cuh"

namespace fc {
namespace {

// Sum over the row's threads: one warp, or the CTA (red: 32 floats of its own
// for each of a row's sums, so that one barrier serves).
__device__ __forceinline__ float row_sum(float v, float* red, bool one_warp) {
  v = warp_sum(v);
  if (one_warp) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const int n = (blockDim.x + 31) >> 5, l = threadIdx.x & 31;
  return warp_sum(l < n ? red[l] : 0.0f);
}

__device__ __forceinline__ float inv_rms_rn(float ss, int H, float eps) {
  return __frsqrt_rn(__fadd_rn(__fdiv_rn(ss, static_cast<float>(H)), eps));
}

// TEAM: one warp a row, blockDim.x / 32 rows a CTA; else one row a CTA.
template <bool F32, bool TEAM, int MAXT>
__global__ void __launch_bounds__(MAXT) k_block_norm(const BlockNormArgs a) {
  __shared__ float red[2][32];
  pdl_begin();
  const int64_t row = TEAM ? static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5) : blockIdx.x;
  const int t = TEAM ? threadIdx.x & 31 : threadIdx.x;
  const int e = t * 16;
  if (row >= a.rows) return;  // TEAM only: a whole warp
  const bool live = e < a.H;
  const int64_t at = row * a.H + e;
  Raw16<F32> xr, rr, gr, w1, w2;
  if (live) {
    xr = load_raw16<F32>(a.x, at);
    if (a.res_in) rr = load_raw16<F32>(a.res_in, at);
    if (a.gate) gr = load_weight16<F32>(a.gate, row / a.gate_seg * a.H + e);
    if (a.post_w) w1 = load_weight16<F32>(a.post_w, e);
    if (a.pre_w) w2 = load_weight16<F32>(a.pre_w, e);
  }
  float u[16] = {};
  if (live) unpack_raw<F32>(xr, u);
  if (a.post_w) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = __fmaf_rn(u[i], u[i], ss);
    const float inv = inv_rms_rn(row_sum(ss, red[0], TEAM), a.H, a.eps_post);
    if (live) {
      float w[16];
      unpack_raw<F32>(w1, w);
#pragma unroll
      for (int i = 0; i < 16; ++i) u[i] = u[i] * inv * w[i];
    }
  }
  Raw16<F32> hr;
  if (live) {
    float g[16], r[16];
    if (a.gate) {
      unpack_raw<F32>(gr, g);
#pragma unroll
      for (int i = 0; i < 16; ++i) u[i] *= g[i];
    }
    if (a.res_in) {
      unpack_raw<F32>(rr, r);
#pragma unroll
      for (int i = 0; i < 16; ++i) u[i] = __fmaf_rn(a.beta, u[i], a.alpha * r[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) u[i] *= a.beta;
    }
    hr = pack_raw<F32>(u);
    store_raw16<F32>(a.res_out, at, hr);
    unpack_raw<F32>(hr, u);
  }
  if (!a.pre_w) return;
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) ss = __fmaf_rn(u[i], u[i], ss);
  const float inv = inv_rms_rn(row_sum(ss, red[1], TEAM), a.H, a.eps_pre);
  Raw16<F32> yr;
  uint32_t m = 0;
  if (live) {
    float w[16];
    unpack_raw<F32>(w2, w);
#pragma unroll
    for (int i = 0; i < 16; ++i) u[i] = u[i] * inv * w[i];
    yr = pack_raw<F32>(u);
    if (a.y) store_raw16<F32>(a.y, at, yr);
    unpack_raw<F32>(yr, u);  // what is quantised is y as it is stored
    m = absmax_raw<F32>(yr);
  }
  if (a.y_codes) {
    const int KT = static_cast<int>(mx4_tiles_k(a.H));
    mx4_store16(u, m, live, (t & 7) == 0 && live, static_cast<uint8_t*>(a.y_codes) + at / 2,
                a.y_scales + mx4_scale_word(row, min(t >> 3, KT - 1), KT));
  }
}

}  // namespace

cudaError_t launch_block_norm(bool f32, const BlockNormArgs& a, cudaStream_t st) {
  if (a.H <= 512) {
    const dim3 grid(static_cast<unsigned>((a.rows + 3) / 4));
    return f32 ? launch_pdl(k_block_norm<true, true, 128>, grid, dim3(128), 0, st, a)
               : launch_pdl(k_block_norm<false, true, 128>, grid, dim3(128), 0, st, a);
  }
  const dim3 grid(static_cast<unsigned>(a.rows));
  const dim3 block(static_cast<unsigned>((a.H / 16 + 31) / 32 * 32));
  if (block.x <= 512)
    return f32 ? launch_pdl(k_block_norm<true, false, 512>, grid, block, 0, st, a)
               : launch_pdl(k_block_norm<false, false, 512>, grid, block, 0, st, a);
  return f32 ? launch_pdl(k_block_norm<true, false, 1024>, grid, block, 0, st, a)
             : launch_pdl(k_block_norm<false, false, 1024>, grid, block, 0, st, a);
}

}  // namespace fc
