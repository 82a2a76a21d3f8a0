// layer_norm_grad.cu -- gradient of layer_norm.cu.  With n = (h - mean) * inv and a = dy *
// weight, for one row:
//   dx = dh + inv * (a - mean(a) - n * mean(a * n))
// and over rows: dweight = sum dy * n, dbias = sum dy.  h is the residual stream that
// was normed, mean and inv are what the forward pass kept of the row, dh (or none) is the
// gradient that reaches h by itself; dx is that of x and of the residual alike.
//
// Bound by memory: three rows in, one out.  As in block_norm_grad.cu a CTA takes a run of
// neighbouring rows, staged in shared memory by bulk copies a few rows ahead; a row's
// two sums meet at one barrier, its stage is free again there, and the sums over rows
// stay in registers, each thread its own columns: no atomics, every order fixed.  A CTA
// writes its sums once, and a second kernel adds the CTAs' in order.  Rows too wide for
// one CTA's registers are cut over a cluster, whose CTAs exchange the row's sums.
// Measured on GB300 with everything asked for: 8192 x 5120 bf16 58.1 us, 5.8 TB/s (0.85
// of the measured copy rate), of which the second kernel is about 5; fp32 102, 6.6 TB/s (0.97).
#include <algorithm>

#include "block.h"
#include "grad_rows.cuh"

namespace fc {
namespace {

constexpr int kErrCuda = 2;  // FC_ERR_CUDA
constexpr int kMostStages = 4;

struct GradJob {
  LayerNormGradArgs a;
  float* ws_w;        // [teams, H] sums of the teams
  float* ws_b;
  int teams;
  uint32_t late;      // not 0: every copy counts as late
};

// Sums of two values over the CTA, or the CL CTAs of the cluster, each thread ending
// with both, in the same order everywhere.  A warp folds them onto one another: lanes
// 0-15 end with the first, 16-31 with the second.  red: 2 rows of Red<CL>::kStride.
template <int CL>
__device__ __forceinline__ void row_sums2(float (&v)[2], float* red) {
  using R = Red<CL>;
  const int l = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool hi = l & 16;
  float s = (hi ? v[1] : v[0]) + __shfl_xor_sync(kFull, hi ? v[0] : v[1], 16);
#pragma unroll
  for (int m = 8; m >= 1; m >>= 1) s += __shfl_xor_sync(kFull, s, m);
  float* mine = red + (l >> 4) * R::kStride;
  if constexpr (CL == 1) {
    if ((l & 15) == 0) mine[warp] = s;
    __syncthreads();
  } else {
    // a value's lanes each tell one CTA of the cluster (its rank is the block's)
    const int at = static_cast<int>(blockIdx.x % CL) * (blockDim.x >> 5) + warp;
    if ((l & 15) < CL) st_cluster(cluster_addr(mine + at, l & 15), s);
    __syncwarp();
    cluster_sync_all();
  }
  const float* part = mine + (l & 15) * (R::kEntries / 16);
  s = 0.0f;
#pragma unroll
  for (int k = 0; k < R::kEntries / 32; ++k) {
    const float2 p = *reinterpret_cast<const float2*>(part + 2 * k);
    s += p.x + p.y;
  }
#pragma unroll
  for (int m = 8; m >= 1; m >>= 1) s += __shfl_xor_sync(kFull, s, m);
  v[0] = __shfl_sync(kFull, s, 0);
  v[1] = __shfl_sync(kFull, s, 16);
}

// CL: CTAs of a cluster, a team, that share a row's columns.
template <bool F32, int W, int CL, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) k_layer_norm_grad(const GradJob job, int stages) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(16) float red[2][2 * Red<CL>::kStride];  // neighbouring rows take turns
  __shared__ uint64_t full[kMostStages];
  __shared__ volatile uint32_t late[2];  // not 0: a copy did not land in time, by turns as red
  constexpr int es = F32 ? 4 : 2, kP = W / 2;
  const LayerNormGradArgs& a = job.a;
  const int t = threadIdx.x, H = a.H;
  const int team = blockIdx.x / CL, teams = job.teams, rank = blockIdx.x % CL;
  const int col0 = CL == 1 ? 0 : H / 16 * rank / CL * 16;
  const int cols = CL == 1 ? H : H / 16 * (rank + 1) / CL * 16 - col0;
  const int live = cols / W, row_bytes = cols * es;          // of this CTA
  const int stride = H * es, shift = CL == 1 ? 0 : col0 * es;  // of a row in memory
  const bool on = t < live;
  const int slots = a.dh ? 3 : 2;  // of a stage: h, dy, dh
  if (t == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(full + s, 1);
    late[0] = late[1] = job.late;
    mbar_init_fence();
  }
  for (int i = t; i < 2 * 2 * Red<CL>::kStride; i += blockDim.x) red[0][i] = 0.0f;
  __syncwarp();
  if constexpr (CL == 1)
    __syncthreads();
  else
    cluster_sync_all();
  pdl_begin();

  // rows of this team: neighbours, the first teams one more where they do not divide
  const int rows = static_cast<int>(a.rows), per = rows / teams, more = rows % teams;
  const int r0 = team * per + min(team, more), r1 = r0 + per + (team < more);
  const char* from = nullptr;  // lane k of the first warp copies tensor k
  if (t == 0) from = static_cast<const char*>(a.h) + shift;
  if (t == 1) from = static_cast<const char*>(a.dy) + shift;
  if (t == 2) from = static_cast<const char*>(a.dh) + shift;
  auto stage_row = [&](int row, int st) {  // the first warp
    // unsigned: a few rows ahead of the last may be past 2^31 - 1.  (777 rows of 2064 fp32 7.9 us;
    // with the row counted from the CTA's first 8.7, with the sum taken apart 8.5.)
    if (static_cast<uint32_t>(row) >= static_cast<uint32_t>(r1)) return;
    if (t == 0) {
      fence_proxy_async_smem();
      mbar_expect_tx(full + st, slots * row_bytes);
    }
    __syncwarp();
    if (t < slots)
      bulk_load(ring + (st * slots + t) * row_bytes, from + static_cast<int64_t>(row) * stride, row_bytes, full + st);
  };
  if (t < 32)
    for (int k = 0; k < stages; ++k) stage_row(r0 + k, k);

  const float inv_n = 1.0f / static_cast<float>(H);
  const float2 zero = make_float2(0.0f, 0.0f);
  float2 acc_w[kP], acc_b[kP];
  RawCols<F32, W> w{};
  if (on && a.weight) w = load_cols<F32, W>(static_cast<const char*>(a.weight) + shift, t, live);
#pragma unroll
  for (int i = 0; i < kP; ++i) acc_w[i] = acc_b[i] = zero;
  const float2* stats = reinterpret_cast<const float2*>(a.stats);
  float2 next = r0 < r1 ? stats[r0] : zero;
  int s = 0;
  uint32_t phase = 0;
  bool stop = false;
  int row = r0;
  for (; row < r1; ++row) {
    const float2 st = next;
    if (row + 1 < r1) next = stats[row + 1];
    const uint8_t* src = ring + s * slots * row_bytes;
    const int turn = (row - r0) & 1;
    if (!mbar_wait_bounded(full + s, phase)) {
      if constexpr (CL == 1)
        late[turn] = 1;
      else
        for (int c = 0; c < CL; ++c) st_cluster(cluster_addr(const_cast<const uint32_t*>(late + turn), c), 1.0f);
    }
    const float2 vi = dup2(st.y), vm = dup2(-st.x);
    RawCols<F32, W> h, dy, dh{};
    float r[2] = {};
    if (on) {
      h = load_cols<F32, W>(src, t, live);
      dy = load_cols<F32, W>(src + row_bytes, t, live);
      if (a.dh) dh = load_cols<F32, W>(src + 2 * row_bytes, t, live);
      float2 s0 = zero, s1 = zero;
#pragma unroll
      for (int i = 0; i < kP; ++i) {
        const float2 n = pmul(padd(pair<F32, W>(h, i), vm), vi);
        float2 e = pair<F32, W>(dy, i);
        acc_b[i] = padd(acc_b[i], e);
        acc_w[i] = pfma(e, n, acc_w[i]);
        if (a.weight) e = pmul(e, pair<F32, W>(w, i));
        s0 = padd(s0, e);
        s1 = pfma(e, n, s1);
      }
      r[0] = s0.x + s0.y, r[1] = s1.x + s1.y;
    }
    row_sums2<CL>(r, red[turn]);
    if (late[turn]) {  // set at the start, or before this row's barrier: all read the same
      stop = true;
      break;
    }
    if (t < 32) stage_row(static_cast<int>(static_cast<uint32_t>(row) + stages), s);
    if (++s == stages) s = 0, phase ^= 1;
    if (!on) continue;
    const float2 m0 = dup2(-(r[0] * inv_n)), m1 = dup2(-(r[1] * inv_n));
    float2 o[kP];
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const float2 n = pmul(padd(pair<F32, W>(h, i), vm), vi);
      float2 e = pair<F32, W>(dy, i);
      if (a.weight) e = pmul(e, pair<F32, W>(w, i));
      o[i] = pfma(pfma(m1, n, padd(e, m0)), vi, pair<F32, W>(dh, i));
    }
    store_cols<F32, W>(static_cast<char*>(a.dx) + static_cast<int64_t>(row) * stride + shift, t, live, o);
  }
  if (on && !stop) {
    if (a.dweight) store_sums<F32, W>(job.ws_w + static_cast<int64_t>(team) * H + col0, t, live, acc_w);
    if (a.dbias) store_sums<F32, W>(job.ws_b + static_cast<int64_t>(team) * H + col0, t, live, acc_b);
  }
  if (stop && t == 0) {  // a copy never landed: say so, and let those in flight land
    if (a.status) *a.status = kErrCuda;
    for (int i = row; i < r1 && i - row < stages; ++i) mbar_wait_bounded(full + (i - r0) % stages, ((i - r0) / stages) & 1);
  }
  if constexpr (CL > 1) {  // no CTA's memory goes while another may write to it
    __syncwarp();
    cluster_sync_all();
  }
}

// Adds the teams' sums.  blockIdx.y: 0 the weight's, 1 the bias's.
__global__ void __launch_bounds__(kSumWarps * 32) k_layer_norm_grad_sum(const GradJob job) {
  __shared__ float2 red[kSumWarps][32];
  pdl_begin();
  const int col = blockIdx.x * kSumCols + 2 * (threadIdx.x & 31);
  float* out = blockIdx.y == 0 ? job.a.dweight : job.a.dbias;
  if (!out) return;
  float2 s;
  if (!column_sums(blockIdx.y == 0 ? job.ws_w : job.ws_b, job.teams, job.a.H, col, red, s)) return;
  out[col] = s.x, out[col + 1] = s.y;  // 4-byte aligned
}

template <bool F32, int W, int CL, int MAXT, int MINB>
cudaError_t launch_staged(GradJob& job, int threads, int stages, int smem, cudaStream_t st) {
  auto* kern = k_layer_norm_grad<F32, W, CL, MAXT, MINB>;
  const void* fn = reinterpret_cast<const void*>(kern);
  if (cudaError_t e = raise_smem_limit(fn, smem)) return e;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = CL;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CL);
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = CL == 1 ? 1 : 2;
  // teams that the GPU holds at once
  const int held = occupancy_memo(fn, threads, smem, CL, [&] {
    int v = 0;
    if (CL == 1) {
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&v, kern, threads, smem);
      return v * num_sms();
    }
    cfg.attrs = at + 1, cfg.numAttrs = 1;
    cudaOccupancyMaxActiveClusters(&v, kern, &cfg);
    cfg.attrs = at, cfg.numAttrs = 2;
    return v;
  });
  if (held < 1) return cudaErrorInvalidConfiguration;
  job.teams = static_cast<int>(std::min<int64_t>(std::min(held, kNormGradMaxCtas), job.a.rows));
  job.ws_w = job.a.ws;
  job.ws_b = job.a.ws + static_cast<int64_t>(job.teams) * job.a.H;
  cfg.gridDim = dim3(static_cast<unsigned>(job.teams * CL));
  return cudaLaunchKernelEx(&cfg, kern, static_cast<const GradJob&>(job), stages);
}

template <bool F32>
cudaError_t launch_grad(GradJob& job, cudaStream_t st) {
  const LayerNormGradArgs& a = job.a;
  constexpr int kMost = 220 * 1024;
  // A CTA's columns in a team of CL (the widest), its threads at eight columns each, the bytes
  // of a stage, and the stages that fit.
  auto cols = [&](int CL) { return (a.H / 16 + CL - 1) / CL * 16; };
  auto threads = [&](int CL) { return (cols(CL) / 8 + 31) / 32 * 32; };
  auto stage = [&](int CL) { return (a.dh ? 3 : 2) * cols(CL) * (F32 ? 4 : 2); };
  auto stages = [&](int CL) { return std::min(kMostStages, kMost / stage(CL)); };  // two at least
  // Eight columns a thread, and one CTA an SM of more than 320 threads: two of up to 640, at 48
  // registers a thread, spill (us, one / two, 8192 rows of 5120 bf16 58.2 / 82.9, 777 of
  // 2064 fp32 without dh 10.0 / 15.4, inputs from memory: where they are in L2 it is 7.9); 16
  // columns a thread are no faster (58.3, 12.2) and leave 777 rows fewer warps; four stages,
  // eight take 60.4.  Rows above 8192 columns take a cluster.
  const int n = stages(1);
  if (threads(1) <= 640) return launch_staged<F32, 8, 1, 640, 1>(job, threads(1), n, n * stage(1), st);
  if (threads(1) <= 1024) return launch_staged<F32, 8, 1, 1024, 1>(job, threads(1), n, n * stage(1), st);
  return launch_staged<F32, 8, 2, 1024, 1>(job, threads(2), stages(2), stages(2) * stage(2), st);
}

}  // namespace

cudaError_t launch_layer_norm_grad(bool f32, const LayerNormGradArgs& a, cudaStream_t st) {
  GradJob job{};
  job.a = a;
  job.late = wait_cycles <= 0;
  if (cudaError_t e = f32 ? launch_grad<true>(job, st) : launch_grad<false>(job, st)) return e;
  if (!a.dweight && !a.dbias) return cudaSuccess;
  return launch_pdl(k_layer_norm_grad_sum, dim3(static_cast<unsigned>((a.H + kSumCols - 1) / kSumCols), 2),
                    dim3(kSumWarps * 32), 0, st, job);
}

}  // namespace fc
