// block_norm_grad.cu -- gradient of block_norm.cu.  With hh = h * inv_h,
// xh = x * inv_x, u = xh * post_weight (or x), for one row:
//   dn   = dy * pre_weight
//   dh'  = dh + inv_h * (dn - hh * mean(dn * hh))
//   dres = alpha * dh'            du = beta * gate * dh'
//   dx   = inv_x * (e - xh * mean(e * xh)), e = du * post_weight   (or du)
// and over rows:
//   dpre_weight  = sum dy * hh    dpost_weight = sum du * xh
//   dgate        = beta * sum over the rows that share the gate row of dh' * u
// x and h are what the forward pass read and kept; the inverse root mean
// squares are computed again from them (that reads nothing more).
//
// Bound by memory: four rows in, two out.  The sums over rows stay on chip:
// a CTA takes one run of neighbouring rows (within one gate row's rows) and
// adds its columns up in shared memory, each thread its own 16 columns, so
// there is no atomic and the order of every sum is fixed.  A CTA writes its sums
// once, to the workspace, and a second kernel adds the CTAs' sums in order.
#include <algorithm>

#include "block.h"
#include "mx4.cuh"

namespace fc {
namespace {

// Sums over the row's threads of N values at once; red: N * 32 floats.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* red) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  const int n = blockDim.x >> 5, l = threadIdx.x & 31;
  if (l == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) red[i * 32 + (threadIdx.x >> 5)] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(l < n ? red[i * 32 + l] : 0.0f);
}

// A thread's 16 running column sums of one kind, in shared memory as four
// planes of float4 (lanes 16 bytes apart: no bank conflict).
__device__ __forceinline__ void acc_add(float4* acc, const float v[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float4 s = acc[j * blockDim.x + threadIdx.x];
    s.x += v[4 * j], s.y += v[4 * j + 1], s.z += v[4 * j + 2], s.w += v[4 * j + 3];
    acc[j * blockDim.x + threadIdx.x] = s;
  }
}
__device__ __forceinline__ void acc_take(float4* acc, float v[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 s = acc[j * blockDim.x + threadIdx.x];
    v[4 * j] = s.x, v[4 * j + 1] = s.y, v[4 * j + 2] = s.z, v[4 * j + 3] = s.w;
    acc[j * blockDim.x + threadIdx.x] = make_float4(0, 0, 0, 0);
  }
}

// How the rows are cut: `segs` runs of seg_rows rows that share a gate row,
// each into `cuts` pieces; piece i of the segs * cuts is CTA i, i + grid, ...
struct GradPlan {
  int64_t segs, seg_rows;
  int cuts, grid;
  bool gate_direct;   // a gate row for every row: its gradient is written row by row
  bool gate_final;    // one piece per gate row: its sum is final
};

struct GradJob {
  BlockNormGradArgs a;
  GradPlan p;
  float* ws_pre;      // [grid, H] sums of the CTAs
  float* ws_post;
  float* ws_gate;     // [segs * cuts, H]
};

template <bool F32, int MAXT>
__global__ void __launch_bounds__(MAXT) k_block_norm_grad(const GradJob job) {
  extern __shared__ float4 acc[];
  // a row's three sums and one more, each its own floats; neighbouring rows take
  // turns, so a row's first barrier frees what the row before it read
  __shared__ float red[2][4 * 32];
  int turn = 0;
  const BlockNormGradArgs& a = job.a;
  const GradPlan& p = job.p;
  pdl_begin();
  const int e = threadIdx.x * 16;
  const bool live = e < a.H;
  const bool w_pre = a.dpre_w != nullptr, w_post = a.dpost_w != nullptr;
  const bool g_sum = a.dgate != nullptr && !p.gate_direct;
  float4* acc_pre = acc;
  float4* acc_post = acc + 4 * blockDim.x;
  float4* acc_gate = acc + 8 * blockDim.x;
#pragma unroll
  for (int j = 0; j < 12; ++j) acc[j * blockDim.x + threadIdx.x] = make_float4(0, 0, 0, 0);
  const float inv_n = 1.0f / static_cast<float>(a.H);
  float w1[16], w2[16];
  {
    Raw16<F32> r{};
    if (live && a.post_w) r = load_weight16<F32>(a.post_w, e);
    unpack_raw<F32>(r, w1);
    if (live && a.pre_w) r = load_weight16<F32>(a.pre_w, e);
    unpack_raw<F32>(r, w2);
  }
  for (int64_t piece = blockIdx.x; piece < p.segs * p.cuts; piece += gridDim.x) {
    const int64_t seg = piece / p.cuts, cut = piece - seg * p.cuts;
    const int64_t r0 = seg * p.seg_rows + p.seg_rows * cut / p.cuts;
    const int64_t r1 = seg * p.seg_rows + p.seg_rows * (cut + 1) / p.cuts;
    for (int64_t row = r0; row < r1; ++row) {
      const int64_t at = row * a.H + e;
      float x[16] = {}, h[16] = {}, dy[16] = {}, dh[16] = {}, g[16];
      if (live) {
        unpack_raw<F32>(load_raw16<F32>(a.x, at), x);
        if (a.dy) {
          unpack_raw<F32>(load_raw16<F32>(a.h, at), h);
          unpack_raw<F32>(load_raw16<F32>(a.dy, at), dy);
        }
        if (a.dh) unpack_raw<F32>(load_raw16<F32>(a.dh, at), dh);
        if (a.gate)
          unpack_raw<F32>(load_weight16<F32>(a.gate, (p.gate_direct ? row : seg) * a.H + e), g);
      }
      float s[3] = {0, 0, 0};
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[0] = __fmaf_rn(h[i], h[i], s[0]);
        s[1] = __fmaf_rn(dy[i] * w2[i], h[i], s[1]);
        s[2] = __fmaf_rn(x[i], x[i], s[2]);
      }
      turn ^= 1;
      row_sums<3>(s, red[turn]);
      if (a.dy) {
        const float inv = __frsqrt_rn(__fadd_rn(s[0] * inv_n, a.eps_pre));
        const float c = inv * inv * s[1] * inv_n;  // mean(dn * hh) * inv_h
        float t[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float hh = h[i] * inv;
          dh[i] += __fmaf_rn(inv, dy[i] * w2[i], -(hh * c));
          t[i] = dy[i] * hh;
        }
        if (w_pre) acc_add(acc_pre, t);
      }
      if (live && a.dres) {
        float t[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) t[i] = a.alpha * dh[i];
        store_raw16<F32>(a.dres, at, pack_raw<F32>(t));
      }
      const float inv_x = a.post_w ? __frsqrt_rn(__fadd_rn(s[2] * inv_n, a.eps_post)) : 1.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        dh[i] *= a.beta;  // now the gradient of gate * u
        x[i] *= inv_x;    // now xh (x where there is no norm)
      }
      if (a.gate) {
        float t[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) t[i] = dh[i] * (a.post_w ? x[i] * w1[i] : x[i]);
        if (g_sum) acc_add(acc_gate, t);
        if (live && a.dgate && p.gate_direct) store_raw16<F32>(a.dgate, at, pack_raw<F32>(t));
#pragma unroll
        for (int i = 0; i < 16; ++i) dh[i] = live ? dh[i] * g[i] : 0.0f;  // now du
      }
      if (a.post_w) {
        float t[16], q[1] = {0};
#pragma unroll
        for (int i = 0; i < 16; ++i) t[i] = dh[i] * x[i];
        if (w_post) acc_add(acc_post, t);
#pragma unroll
        for (int i = 0; i < 16; ++i) q[0] = __fmaf_rn(t[i], w1[i], q[0]);
        row_sums<1>(q, red[turn] + 96);
        const float c = q[0] * inv_n;
#pragma unroll
        for (int i = 0; i < 16; ++i) dh[i] = inv_x * __fmaf_rn(dh[i], w1[i], -(x[i] * c));
      }
      if (live) store_raw16<F32>(a.dx, at, pack_raw<F32>(dh));
    }
    if (g_sum) {
      float t[16];
      acc_take(acc_gate, t);
      if (live) {
        if (p.gate_final)
          store_raw16<F32>(a.dgate, seg * a.H + e, pack_raw<F32>(t));
        else
          store_raw16<true>(job.ws_gate, piece * a.H + e, pack_raw<true>(t));
      }
    }
  }
  float t[16];
  if (w_pre) {
    acc_take(acc_pre, t);
    if (live) store_raw16<true>(job.ws_pre, static_cast<int64_t>(blockIdx.x) * a.H + e, pack_raw<true>(t));
  }
  if (w_post) {
    acc_take(acc_post, t);
    if (live) store_raw16<true>(job.ws_post, static_cast<int64_t>(blockIdx.x) * a.H + e, pack_raw<true>(t));
  }
}

// Adds the CTAs' sums: 32 columns a CTA, eight warps over the addends, in a
// fixed order.  blockIdx.y: 0 the norm before, 1 the norm after, 2 + s gate row s.
template <bool F32>
__global__ void __launch_bounds__(256) k_block_norm_grad_sum(const GradJob job) {
  __shared__ float red[8][32];
  pdl_begin();
  const int H = job.a.H, col = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
  for (int64_t y = blockIdx.y;; y += gridDim.y) {
    const float* src;
    int n;
    if (y == 0) {
      src = job.a.dpre_w ? job.ws_pre : nullptr, n = job.p.grid;
    } else if (y == 1) {
      src = job.a.dpost_w ? job.ws_post : nullptr, n = job.p.grid;
    } else {
      if (!job.ws_gate || y - 2 >= job.p.segs) return;
      src = job.ws_gate + (y - 2) * job.p.cuts * H, n = job.p.cuts;
    }
    if (!src) continue;
    float s = 0.0f;
    if (col < H)
      for (int i = w; i < n; i += 8) s += src[static_cast<int64_t>(i) * H + col];
    red[w][threadIdx.x & 31] = s;
    __syncthreads();
    if (w == 0 && col < H) {
#pragma unroll
      for (int i = 1; i < 8; ++i) s += red[i][threadIdx.x];
      if (y == 0)
        job.a.dpre_w[col] = s;
      else if (y == 1)
        job.a.dpost_w[col] = s;
      else if (F32)
        static_cast<float*>(job.a.dgate)[(y - 2) * H + col] = s;
      else
        static_cast<__nv_bfloat16*>(job.a.dgate)[(y - 2) * H + col] = __float2bfloat16_rn(s);
    }
    __syncthreads();
  }
}

template <bool F32, int MAXT>
cudaError_t launch(GradJob& job, int threads, cudaStream_t st) {
  auto* kern = k_block_norm_grad<F32, MAXT>;
  const int smem = threads * 12 * static_cast<int>(sizeof(float4));
  if (cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), smem)) return e;
  const int occ = occupancy_memo(reinterpret_cast<const void*>(kern), threads, smem, 1, [&] {
    int v = 0;
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&v, kern, threads, smem);
    return v;
  });
  if (occ < 1) return cudaErrorInvalidConfiguration;
  const BlockNormGradArgs& a = job.a;
  GradPlan& p = job.p;
  const int64_t most = std::min<int64_t>(kNormGradMaxCtas, static_cast<int64_t>(num_sms()) * occ);
  p.gate_direct = a.gate && a.gate_rows == a.rows;
  p.segs = a.gate && !p.gate_direct ? a.gate_rows : 1;
  p.seg_rows = a.rows / p.segs;
  // one piece a CTA where there are fewer gate rows than CTAs, else one piece a gate row
  p.cuts = static_cast<int>(std::max<int64_t>(1, std::min(most / p.segs, p.seg_rows)));
  p.gate_final = p.cuts == 1;
  p.grid = static_cast<int>(std::min(most, p.segs * p.cuts));
  const int64_t H = a.H;
  job.ws_pre = a.ws;
  job.ws_post = a.ws + p.grid * H;
  const bool sum_gate = a.dgate && !p.gate_direct && !p.gate_final;
  job.ws_gate = sum_gate ? a.ws + 2 * p.grid * H : nullptr;
  if (cudaError_t e = launch_pdl(kern, dim3(p.grid), dim3(threads), smem, st, job)) return e;
  if (!a.dpre_w && !a.dpost_w && !sum_gate) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>((H + 31) / 32),
                  static_cast<unsigned>(std::min<int64_t>(65535, 2 + (sum_gate ? p.segs : 0))));
  return launch_pdl(k_block_norm_grad_sum<F32>, grid, dim3(256), 0, st, job);
}

}  // namespace

cudaError_t launch_block_norm_grad(bool f32, const BlockNormGradArgs& a, cudaStream_t st) {
  GradJob job{};
  job.a = a;
  const int threads = (a.H / 16 + 31) / 32 * 32;
  if (threads <= 512) return f32 ? launch<true, 512>(job, threads, st) : launch<false, 512>(job, threads, st);
  return f32 ? launch<true, 1024>(job, threads, st) : launch<false, 1024>(job, threads, st);
}

}  // namespace fc
