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
// registers (32 neighbouring bytes a thread, so a warp's loads and stores
// cover 1 KB), and each row is read once.  Rows that fit one warp take one each.
// The weights come where they are used, from L1: fewer registers, more rows in
// flight, which is what a row's two sums are hidden behind; and rows start for L2
// before a CTA takes them.  The quantised y (mx4.cuh) leaves from the registers that
// hold it.  Measured on GB300, inputs changing from call to call: 8192 x
// 8192 bf16, both norms and eight gates, 83.2 us, 6.5 TB/s (0.95 of the measured copy
// rate; without rows sent for 89.0, with twice as far ahead 84.5); 4096 x 8192 fp32 89.5
// us; one row of 4096 1.9 us in a graph.
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

// TEAM: one warp a row, four rows a CTA; else one row a CTA.  W: columns of a
// thread, 32 bytes of them or (fp32 rows above 8192) 64.
template <bool F32, int W, bool TEAM, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) k_block_norm(const BlockNormArgs a) {
  __shared__ float red[2][32];
  pdl_begin();
  const uint32_t row = TEAM ? blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
  const int t = TEAM ? threadIdx.x & 31 : threadIdx.x;
  const int e = t * W;
  if (row >= a.rows) return;  // TEAM only: a whole warp
  const bool live = e < a.H;
  const int64_t at = static_cast<int64_t>(row) * a.H + e;
  const float inv_n = 1.0f / static_cast<float>(a.H);
  // The row that the CTAs of the next turn or so will take starts on its way to L2
  // (`ahead` rows on, the SMs' number; whole rows are multiples of 32 bytes).
  if (!TEAM && threadIdx.x == 0 && row + a.ahead < a.rows) {
    const uint32_t bytes = a.H * (F32 ? 4 : 2);
    const int64_t off = static_cast<int64_t>(row + a.ahead) * bytes;
    prefetch_l2(static_cast<const char*>(a.x) + off, bytes);
    if (a.res_in) prefetch_l2(static_cast<const char*>(a.res_in) + off, bytes);
    if (a.gate && a.gate_seg == 1) prefetch_l2(static_cast<const char*>(a.gate) + off, bytes);
  }
  Raw<F32, W> xr, rr, gr;
  if (live) {
    xr = load_raw<F32, W>(a.x, at);
    if (a.res_in) rr = load_raw<F32, W>(a.res_in, at);
    if (a.gate)
      gr = load_weight<F32, W>(a.gate, static_cast<int64_t>(row / static_cast<uint32_t>(a.gate_seg)) * a.H + e);
  }
  const float2 zero = make_float2(0.0f, 0.0f);
  float inv = 1.0f;
  if (a.post_w) {
    float2 ss = zero;
    if (live)
#pragma unroll
      for (int i = 0; i < W / 2; ++i) ss = pfma(pair<F32, W>(xr, i), pair<F32, W>(xr, i), ss);
    inv = inv_sqrt(row_sum(ss.x + ss.y, red[0], TEAM) * inv_n + a.eps_post);
  }
  Raw<F32, W> hr;
  float2 ss = zero;
  if (live) {
    float2 u[W / 2];
#pragma unroll
    for (int i = 0; i < W / 2; ++i) u[i] = pmul(pair<F32, W>(xr, i), dup2(inv));
    if (a.post_w) {
      const Raw<F32, W> w = load_weight<F32, W>(a.post_w, e);
#pragma unroll
      for (int i = 0; i < W / 2; ++i) u[i] = pmul(u[i], pair<F32, W>(w, i));
    }
    if (a.gate)
#pragma unroll
      for (int i = 0; i < W / 2; ++i) u[i] = pmul(u[i], pair<F32, W>(gr, i));
    // block_scale last: with the inverse root alone it may be past binary32
    if (a.res_in) {
#pragma unroll
      for (int i = 0; i < W / 2; ++i) u[i] = pfma(u[i], dup2(a.beta), pmul(pair<F32, W>(rr, i), dup2(a.alpha)));
    } else {
#pragma unroll
      for (int i = 0; i < W / 2; ++i) u[i] = pmul(u[i], dup2(a.beta));
    }
    hr = pack_raw<F32, W>(u);
    store_raw<F32, W>(a.res_out, at, hr);
#pragma unroll
    for (int i = 0; i < W / 2; ++i) ss = pfma(pair<F32, W>(hr, i), pair<F32, W>(hr, i), ss);
  }
  if (!a.pre_w) return;
  inv = inv_sqrt(row_sum(ss.x + ss.y, red[1], TEAM) * inv_n + a.eps_pre);
  Raw<F32, W> yr;
  if (live) {
    const Raw<F32, W> w = load_weight<F32, W>(a.pre_w, e);
    float2 u[W / 2];
#pragma unroll
    for (int i = 0; i < W / 2; ++i) u[i] = pmul(pmul(pair<F32, W>(hr, i), dup2(inv)), pair<F32, W>(w, i));
    yr = pack_raw<F32, W>(u);
    if (a.y) store_raw<F32, W>(a.y, at, yr);
  }
  if (a.y_codes) {  // what is quantised is y as it is stored
    float v[W] = {};
    uint32_t m = 0;
    if (live) {
      m = absmax_raw<F32, W>(yr);
      unpack_raw<F32, W>(yr, v);
    }
    const int KT = static_cast<int>(mx4_tiles_k(a.H));
    mx4_store<W>(v, m, live, live && t % (128 / W) == 0, static_cast<uint8_t*>(a.y_codes) + at / 2,
                 a.y_scales + mx4_scale_word(row, min(e / 128, KT - 1), KT));
  }
}

template <bool F32, int W, int MAXT, int MINB>
cudaError_t launch_rows(const BlockNormArgs& a, cudaStream_t st) {
  return launch_pdl(k_block_norm<F32, W, false, MAXT, MINB>, dim3(static_cast<unsigned>(a.rows)),
                    dim3(static_cast<unsigned>((a.H / W + 31) / 32 * 32)), 0, st, a);
}
// Turns of the whole GPU that the rows take.
template <bool F32, int W, int MAXT, int MINB>
int64_t turns(const BlockNormArgs& a) {
  auto* kern = k_block_norm<F32, W, false, MAXT, MINB>;
  const int threads = (a.H / W + 31) / 32 * 32;
  const int occ = occupancy_memo(reinterpret_cast<const void*>(kern), threads, 0, 1, [&] {
    int v = 0;
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&v, kern, threads, 0);
    return v;
  });
  const int64_t slots = static_cast<int64_t>(num_sms()) * (occ > 0 ? occ : 1);
  return (a.rows + slots - 1) / slots;
}
template <bool F32, int W>
cudaError_t launch_teams(const BlockNormArgs& a, cudaStream_t st) {
  return launch_pdl(k_block_norm<F32, W, true, 128, 1>, dim3(static_cast<unsigned>((a.rows + 3) / 4)), dim3(128), 0, st,
                    a);
}

}  // namespace

cudaError_t launch_block_norm(bool f32, BlockNormArgs a, cudaStream_t st) {
  a.ahead = num_sms();
  // Registers for three CTAs of 512 threads an SM spill a little: they are taken where
  // the rows then go in fewer turns of the whole GPU (us, inputs changing from call to
  // call, three / two CTAs, rows of 8192: 300 7.2 / 6.1, 456 8.3 / 10.3, 600 12.1 / 11.3,
  // 2048 25.8 / 26.0, 8192 83.2 / 85.8).  fp32 rows up to 5120: CTAs of up to 640 threads,
  // two an SM (1037 x 5120, a gate a row, 19.6 us; held to three they spill, 23.8); wider
  // ones have an SM to themselves, which costs the narrower of them: 1037 rows of 5120,
  // 5136, 6144, 7168, one gate, 17.2, 20.6, 23.3, 25.6 us; 4096 rows of 6144 72.9 us, 0.82
  // of the copy rate, of 8192 89.5, 0.89.
  if (!f32) {
    if (a.H <= 512) return launch_teams<false, 16>(a, st);
    if (a.H > 8192) return launch_rows<false, 16, 1024, 1>(a, st);
    return turns<false, 16, 512, 3>(a) < turns<false, 16, 512, 2>(a) ? launch_rows<false, 16, 512, 3>(a, st)
                                                                     : launch_rows<false, 16, 512, 2>(a, st);
  }
  if (a.H <= 256) return launch_teams<true, 8>(a, st);
  if (a.H <= 5120) return launch_rows<true, 8, 640, 2>(a, st);
  return a.H <= 8192 ? launch_rows<true, 8, 1024, 1>(a, st) : launch_rows<true, 16, 1024, 1>(a, st);
}

}  // namespace fc
