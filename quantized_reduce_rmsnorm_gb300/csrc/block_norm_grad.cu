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
// adds its columns up in registers, each thread its own, so there is no atomic
// and the order of every sum is fixed.  A CTA writes its sums once, to the
// workspace, and a second kernel adds the CTAs' sums in order.
// Measured on GB300, 8192 x 5120 bf16 with everything asked for: 84.8 us, 5.9 TB/s
// (0.88 of the measured copy rate), of which the second kernel is about 4; rows
// straight to registers with two barriers a row took 233.
#include <algorithm>

#include "block.h"
#include "grad_rows.cuh"

namespace fc {
namespace {

constexpr int kErrCuda = 2;  // FC_ERR_CUDA

// How the rows are cut: `segs` runs of seg_rows rows that share a gate row,
// each into `cuts` pieces; piece i of the segs * cuts is CTA i, i + grid, ...
struct GradPlan {
  int64_t segs, seg_rows;
  int cuts, grid;
  int cut_rows, cut_more;  // rows of a piece; the first cut_more of a run have one more
  bool gate_direct;   // a gate row for every row: its gradient is written row by row
  bool gate_final;    // one piece per gate row: its sum is final
};

struct GradJob {
  BlockNormGradArgs a;
  GradPlan p;
  float* ws_pre;      // [grid, H] sums of the CTAs
  float* ws_post;
  float* ws_gate;     // [segs * cuts, H]
  uint32_t late;      // not 0: every copy counts as late
};

// The rows are staged in shared memory by bulk copies, a few rows ahead, and all of
// a row's sums are taken at once.  With a = dy * pre_weight, gw = beta * gate *
// post_weight (one factor a column) and k = inv_h^2 * mean(a * h):
//   dh' = dh + inv_h * (a - k * h)
//   sum(e * x) = sum gw x dh + inv_h * (sum gw x a - k * sum gw x h)
// so the six sums h^2, a h, x^2, gw x dh, gw x a and gw x h, which need nothing of
// the row before them, give every factor of the row: one barrier a row, and the
// row goes from shared memory to registers once.  Its stage is free again at
// that barrier.  With r = sum over rows of inv_x * dh' * x (one column), dgate =
// beta * post_weight * r and, for a gate that the piece's rows share,
// dpost_weight = beta * gate * r: one running sum serves both.  It and
// dpre_weight's are in registers.  A thread has W columns, in groups of 16
// bytes, the live threads side by side: no bank conflicts.  Rows too wide for one
// CTA's registers are cut over the CTAs of a cluster, which exchange each row's
// sums through distributed shared memory.
// Sums of eight values over the CTA, or the CL CTAs of the cluster, each thread
// ending with all eight, in the same order everywhere.  Within a warp the values are
// folded onto one another (lanes give away the half that the other lanes keep), so
// that eight sums take 9 shuffles and not 40; lane l ends with value l / 4.
// red: 8 rows of Red<CL>::kStride floats (an odd number of 16-byte groups: no bank
// conflicts), one for each warp of each CTA, those past them 0.
template <int CL>
__device__ __forceinline__ void row_sums8(float (&v)[8], float* red) {
  using R = Red<CL>;
  const int l = threadIdx.x & 31;
#pragma unroll
  for (int m = 16, n = 4; m >= 4; m >>= 1, n >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const bool hi = l & m;
      const float keep = hi ? v[i + n] : v[i], give = hi ? v[i] : v[i + n];
      v[i] = keep + __shfl_xor_sync(kFull, give, m);
    }
  float s = v[0];
  s += __shfl_xor_sync(kFull, s, 2);
  s += __shfl_xor_sync(kFull, s, 1);
  float* mine = red + (l >> 2) * R::kStride;
  const int warp = threadIdx.x >> 5;
  if constexpr (CL == 1) {
    if ((l & 3) == 0) mine[warp] = s;
    __syncthreads();
  } else {
    // a value's four lanes each tell one CTA of the cluster (its rank is the block's)
    const int at = static_cast<int>(blockIdx.x % CL) * (blockDim.x >> 5) + warp;
    if ((l & 3) < CL) st_cluster(cluster_addr(mine + at, l & 3), s);
    __syncwarp();
    cluster_sync_all();
  }
  const float* part = mine + (l & 3) * (R::kEntries / 4);
#pragma unroll
  for (int k = 0; k < R::kEntries / 32; ++k) {
    const float4 a = *reinterpret_cast<const float4*>(part + 8 * k);
    const float4 b = *reinterpret_cast<const float4*>(part + 8 * k + 4);
    const float sum = ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w));
    s = k == 0 ? sum : s + sum;
  }
  s += __shfl_xor_sync(kFull, s, 2);
  s += __shfl_xor_sync(kFull, s, 1);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __shfl_sync(kFull, s, i * 4);
}

constexpr int kMostStages = 4;

// TOKEN: a gate row for every row, staged with the row.  CL: CTAs of a cluster, a
// team, that share a row's columns.
template <bool F32, bool TOKEN, int W, int CL, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) k_block_norm_grad_staged(const GradJob job, int stages) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(16) float red[2][8 * Red<CL>::kStride];  // neighbouring rows take turns
  __shared__ uint64_t full[kMostStages];
  __shared__ volatile uint32_t late[2];  // not 0: a copy did not land in time, by turns as red
  __shared__ struct { int piece, row, end, stage, count; } next;
  constexpr int es = F32 ? 4 : 2, kP = W / 2;
  const BlockNormGradArgs& a = job.a;
  const GradPlan& p = job.p;
  const int t = threadIdx.x, H = a.H;
  // this CTA's columns: runs of 16, shared out over the team
  const int team = blockIdx.x / CL, teams = gridDim.x / CL, rank = blockIdx.x % CL;
  const int col0 = CL == 1 ? 0 : H / 16 * rank / CL * 16;
  const int cols = CL == 1 ? H : H / 16 * (rank + 1) / CL * 16 - col0;
  const int live = cols / W, row_bytes = cols * es;          // of this CTA
  const int stride = H * es, shift = CL == 1 ? 0 : col0 * es;  // of a row in memory
  const bool on = t < live;
  const bool pre = a.dy != nullptr, post = a.post_w != nullptr;
  // slots of a stage: x, h, dy, dh, gate row; absent tensors take none
  const int slot_h = 1, slot_dy = 2, slot_dh = pre ? 3 : 1, slot_g = slot_dh + (a.dh ? 1 : 0);
  const int slots = slot_g + (TOKEN ? 1 : 0);
  float4* acc_post = reinterpret_cast<float4*>(ring + static_cast<size_t>(stages) * slots * row_bytes);
  if (t == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(full + s, 1);
    late[0] = late[1] = job.late;
    mbar_init_fence();
  }
  for (int i = t; i < 2 * 8 * Red<CL>::kStride; i += blockDim.x) red[0][i] = 0.0f;
  for (int j = 0; j < W / 4; ++j) acc_post[j * blockDim.x + t] = make_float4(0, 0, 0, 0);
  __syncwarp();
  if constexpr (CL == 1)
    __syncthreads();
  else
    cluster_sync_all();
  pdl_begin();

  const int pieces = static_cast<int>(p.segs) * p.cuts;  // at most the rows
  auto piece_rows = [&](int piece, int& r0, int& r1) {
    const int seg = piece / p.cuts, cut = piece - seg * p.cuts;
    r0 = seg * static_cast<int>(p.seg_rows) + cut * p.cut_rows + min(cut, p.cut_more);
    r1 = r0 + p.cut_rows + (cut < p.cut_more);
  };
  // Stages the next row (the first warp): each of a row's tensors is one lane's
  // copy.  `next` keeps the place out of the registers.
  const char* from = nullptr;
  {
    int k = 0;
    auto slot = [&](bool there, const void* base) {
      if (there && t == k++) from = static_cast<const char*>(base) + shift;
    };
    slot(true, a.x), slot(pre, a.h), slot(pre, a.dy), slot(a.dh != nullptr, a.dh), slot(TOKEN, a.gate);
  }
  auto stage_next = [&] {
    const int piece = next.piece, row = next.row, st = next.stage;
    __syncwarp();
    if (piece >= pieces) return;
    if (t == 0) {
      fence_proxy_async_smem();
      mbar_expect_tx(full + st, slots * row_bytes);
      ++next.count;
      next.stage = st + 1 == stages ? 0 : st + 1;
      next.row = row + 1;
      if (row + 1 == next.end) {
        next.piece = piece + teams;
        if (next.piece < pieces) piece_rows(next.piece, next.row, next.end);
      }
    }
    __syncwarp();
    if (t < slots)
      bulk_load(ring + (st * slots + t) * row_bytes, from + static_cast<int64_t>(row) * stride, row_bytes, full + st);
  };
  if (t < 32) {
    if (t == 0) {
      next.piece = team;
      next.count = next.stage = 0;
      if (next.piece < pieces) piece_rows(next.piece, next.row, next.end);
    }
    __syncwarp();
    for (int k = 0; k < stages; ++k) stage_next();
  }

  const float inv_n = 1.0f / static_cast<float>(H);
  const float2 zero = make_float2(0.0f, 0.0f);
  float2 gw[kP], acc_pre[kP], acc_r[kP];
  RawCols<F32, W> w2{};
  if (on && a.pre_w) w2 = load_cols<F32, W>(static_cast<const char*>(a.pre_w) + shift, t, live);
#pragma unroll
  for (int i = 0; i < kP; ++i) acc_pre[i] = acc_r[i] = zero;
  int count = 0, s = 0;  // rows done; the row's stage
  uint32_t phase = 0;
  bool stop = false;
  for (int piece = team; piece < pieces && !stop; piece += teams) {
    int r0, r1;
    piece_rows(piece, r0, r1);
    const int64_t seg_off = static_cast<int64_t>(piece / p.cuts) * stride + shift;  // its gate row
#pragma unroll
    for (int i = 0; i < kP; ++i) gw[i] = dup2(a.beta);
    if (on && post) {
      const RawCols<F32, W> w = load_cols<F32, W>(static_cast<const char*>(a.post_w) + shift, t, live);
#pragma unroll
      for (int i = 0; i < kP; ++i) gw[i] = pmul(gw[i], pair<F32, W>(w, i));
    }
    if (on && !TOKEN && a.gate) {
      const RawCols<F32, W> w = load_cols<F32, W>(static_cast<const char*>(a.gate) + seg_off, t, live);
#pragma unroll
      for (int i = 0; i < kP; ++i) gw[i] = pmul(gw[i], pair<F32, W>(w, i));
    }
    for (int row = r0; row < r1; ++row, ++count) {
      const int64_t off = static_cast<int64_t>(row) * stride + shift;
      const uint8_t* src = ring + s * slots * row_bytes;
      if (!mbar_wait_bounded(full + s, phase)) {
        if constexpr (CL == 1)
          late[count & 1] = 1;
        else
          for (int c = 0; c < CL; ++c) st_cluster(cluster_addr(const_cast<const uint32_t*>(late + (count & 1)), c), 1.0f);
      }
      RawCols<F32, W> x, h{}, dy{}, dh{}, g;
      float r[8] = {};
      if (on) {
        x = load_cols<F32, W>(src, t, live);
        if (pre) h = load_cols<F32, W>(src + slot_h * row_bytes, t, live);
        if (pre) dy = load_cols<F32, W>(src + slot_dy * row_bytes, t, live);
        if (a.dh) dh = load_cols<F32, W>(src + slot_dh * row_bytes, t, live);
        if (TOKEN) g = load_cols<F32, W>(src + slot_g * row_bytes, t, live);
        float2 s0 = zero, s1 = zero, s2 = zero, s3 = zero, s4 = zero, s5 = zero;
#pragma unroll
        for (int i = 0; i < kP; ++i) {
          const float2 xi = pair<F32, W>(x, i), hi = pair<F32, W>(h, i), ai = pmul(pair<F32, W>(dy, i), pair<F32, W>(w2, i));
          float2 gx = pmul(gw[i], xi);
          if (TOKEN) gx = pmul(gx, pair<F32, W>(g, i));
          s0 = pfma(hi, hi, s0);
          s1 = pfma(ai, hi, s1);
          s2 = pfma(xi, xi, s2);
          s3 = pfma(gx, pair<F32, W>(dh, i), s3);
          s4 = pfma(gx, ai, s4);
          s5 = pfma(gx, hi, s5);
        }
        r[0] = s0.x + s0.y, r[1] = s1.x + s1.y, r[2] = s2.x + s2.y;
        r[3] = s3.x + s3.y, r[4] = s4.x + s4.y, r[5] = s5.x + s5.y;
      }
      row_sums8<CL>(r, red[count & 1]);
      if (late[count & 1]) {  // set at the start, or before this row's barrier: all read the same
        stop = true;
        break;
      }
      if (t < 32) stage_next();
      if (++s == stages) s = 0, phase ^= 1;
      const float inv = pre ? inv_sqrt(__fadd_rn(r[0] * inv_n, a.eps_pre)) : 0.0f;
      // Each inverse root multiplies the sum with one h (x) before the next does, and the
      // third the row's values: nothing here is the square or the cube of an inverse root,
      // which for rows near 0 with a small eps is past binary32 where the gradient is not.
      const float k = inv * (inv * (r[1] * inv_n));
      const float inv_x = post ? inv_sqrt(__fadd_rn(r[2] * inv_n, a.eps_post)) : 1.0f;
      const float c = inv_x * (inv_x * (__fmaf_rn(inv, __fmaf_rn(-k, r[5], r[4]), r[3]) * inv_n));
      if (!on) continue;
      const float2 vi = dup2(inv), vk = dup2(-k), vx = dup2(inv_x), vc = dup2(-c);
      float2 d[kP], o[kP];
#pragma unroll
      for (int i = 0; i < kP; ++i) {
        const float2 hi = pair<F32, W>(h, i), e = pair<F32, W>(dy, i);
        acc_pre[i] = pfma(pmul(e, vi), hi, acc_pre[i]);
        d[i] = pfma(vi, pfma(vk, hi, pmul(e, pair<F32, W>(w2, i))), pair<F32, W>(dh, i));
      }
      if (a.dres) {
#pragma unroll
        for (int i = 0; i < kP; ++i) o[i] = pmul(d[i], dup2(a.alpha));
        store_cols<F32, W>(static_cast<char*>(a.dres) + off, t, live, o);
      }
      if (TOKEN) {
        // dgate row = beta * post_weight * dh' * xh; what remains is as without a gate
        if (a.dgate) {
#pragma unroll
          for (int i = 0; i < kP; ++i) o[i] = pmul(pmul(gw[i], vx), pmul(d[i], pair<F32, W>(x, i)));
          store_cols<F32, W>(static_cast<char*>(a.dgate) + off, t, live, o);
        }
#pragma unroll
        for (int i = 0; i < kP; ++i) d[i] = pmul(d[i], pair<F32, W>(g, i));
      }
#pragma unroll
      for (int i = 0; i < kP; ++i) {
        const float2 xi = pair<F32, W>(x, i);
        acc_r[i] = pfma(pmul(d[i], xi), vx, acc_r[i]);
        o[i] = pmul(d[i], gw[i]);
        if (post) o[i] = pmul(pfma(vc, xi, o[i]), vx);
      }
      store_cols<F32, W>(static_cast<char*>(a.dx) + off, t, live, o);
    }
    if (on && !stop) {
      float2 o[kP];
      if (a.dgate && !TOKEN) {
#pragma unroll
        for (int i = 0; i < kP; ++i) o[i] = pmul(acc_r[i], dup2(a.beta));
        if (post) {
          const RawCols<F32, W> w = load_cols<F32, W>(static_cast<const char*>(a.post_w) + shift, t, live);
#pragma unroll
          for (int i = 0; i < kP; ++i) o[i] = pmul(o[i], pair<F32, W>(w, i));
        }
        if (p.gate_final)
          store_cols<F32, W>(static_cast<char*>(a.dgate) + seg_off, t, live, o);
        else
          store_sums<F32, W>(job.ws_gate + static_cast<int64_t>(piece) * H + col0, t, live, o);
      }
      if (a.dpost_w) {
#pragma unroll
        for (int i = 0; i < kP; ++i) o[i] = pmul(acc_r[i], dup2(a.beta));
        if (!TOKEN && a.gate) {
          const RawCols<F32, W> w = load_cols<F32, W>(static_cast<const char*>(a.gate) + seg_off, t, live);
#pragma unroll
          for (int i = 0; i < kP; ++i) o[i] = pmul(o[i], pair<F32, W>(w, i));
        }
#pragma unroll
        for (int j = 0; j < W / 4; ++j) {
          float4 x = acc_post[j * blockDim.x + t];
          x.x += o[2 * j].x, x.y += o[2 * j].y, x.z += o[2 * j + 1].x, x.w += o[2 * j + 1].y;
          acc_post[j * blockDim.x + t] = x;
        }
      }
#pragma unroll
      for (int i = 0; i < kP; ++i) acc_r[i] = zero;
    }
  }
  if (on && !stop) {
    if (a.dpre_w) store_sums<F32, W>(job.ws_pre + static_cast<int64_t>(team) * H + col0, t, live, acc_pre);
    if (a.dpost_w) {
      float2 o[kP];
#pragma unroll
      for (int j = 0; j < W / 4; ++j) {
        const float4 x = acc_post[j * blockDim.x + t];
        o[2 * j] = make_float2(x.x, x.y), o[2 * j + 1] = make_float2(x.z, x.w);
      }
      store_sums<F32, W>(job.ws_post + static_cast<int64_t>(team) * H + col0, t, live, o);
    }
  }
  if (stop && t == 0) {  // a copy never landed: say so, and let those in flight land
    if (a.status) *a.status = kErrCuda;
    for (int i = count; i < next.count; ++i) mbar_wait_bounded(full + i % stages, (i / stages) & 1);
  }
  if constexpr (CL > 1) {  // no CTA's memory goes while another may write to it
    __syncwarp();
    cluster_sync_all();
  }
}

// Adds the CTAs' sums.  blockIdx.y: 0 the norm before, 1 the norm after, 2 +
// s gate row s (segs is below kNormGradMaxCtas where their sums are in pieces).
template <bool F32>
__global__ void __launch_bounds__(kSumWarps * 32) k_block_norm_grad_sum(const GradJob job) {
  __shared__ float2 red[kSumWarps][32];
  pdl_begin();
  const int H = job.a.H, y = blockIdx.y;
  const int col = blockIdx.x * kSumCols + 2 * (threadIdx.x & 31);
  const float* src = y == 0 ? job.ws_pre : y == 1 ? job.ws_post : job.ws_gate + (y - 2) * static_cast<int64_t>(job.p.cuts) * H;
  const int n = y < 2 ? job.p.grid : job.p.cuts;
  if ((y == 0 && !job.a.dpre_w) || (y == 1 && !job.a.dpost_w)) return;
  float2 s;
  if (!column_sums(src, n, H, col, red, s)) return;
  if (y < 2) {  // 4-byte aligned
    float* out = (y == 0 ? job.a.dpre_w : job.a.dpost_w) + col;
    out[0] = s.x, out[1] = s.y;
  } else if (F32) {
    *reinterpret_cast<float2*>(static_cast<float*>(job.a.dgate) + static_cast<int64_t>(y - 2) * H + col) = s;
  } else {
    *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(job.a.dgate) + static_cast<int64_t>(y - 2) * H + col) =
        pack_bf2(s.x, s.y);
  }
}

// Cuts the rows for `most` CTAs and lays the workspace out.
void plan(GradJob& job, int64_t most) {
  const BlockNormGradArgs& a = job.a;
  GradPlan& p = job.p;
  p.gate_direct = a.gate && a.gate_rows == a.rows;
  p.segs = a.gate && !p.gate_direct ? a.gate_rows : 1;
  p.seg_rows = a.rows / p.segs;
  // One piece a CTA where there are fewer gate rows than CTAs, else one piece a gate
  // row.  A count of gate rows just above the CTAs, or half of them, leaves many idle
  // (us, rows of 5120 bf16, 152 CTAs, 50 rows a gate row, by gate rows: 76 57.4, 77 77.3,
  // 152 79.9, 153 149.1, 304 150.4).
  p.cuts = static_cast<int>(std::max<int64_t>(1, std::min(most / p.segs, p.seg_rows)));
  p.cut_rows = static_cast<int>(p.seg_rows / p.cuts);
  p.cut_more = static_cast<int>(p.seg_rows % p.cuts);
  p.gate_final = p.cuts == 1;
  p.grid = static_cast<int>(std::min(most, p.segs * p.cuts));
  job.ws_pre = a.ws;
  job.ws_post = a.ws + static_cast<int64_t>(p.grid) * a.H;
  job.ws_gate = a.dgate && !p.gate_direct && !p.gate_final ? a.ws + 2 * static_cast<int64_t>(p.grid) * a.H : nullptr;
}

template <bool F32, bool TOKEN, int W, int CL, int MAXT, int MINB>
cudaError_t launch_staged(GradJob& job, int threads, int stages, int smem, cudaStream_t st) {
  auto* kern = k_block_norm_grad_staged<F32, TOKEN, W, CL, MAXT, MINB>;
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
  plan(job, std::min(held, kNormGradMaxCtas));
  cfg.gridDim = dim3(static_cast<unsigned>(job.p.grid * CL));
  return cudaLaunchKernelEx(&cfg, kern, static_cast<const GradJob&>(job), stages);
}

template <bool F32, bool TOKEN>
cudaError_t launch_grad(GradJob& job, cudaStream_t st) {
  const BlockNormGradArgs& a = job.a;
  const int slots = 1 + (a.dy ? 2 : 0) + (a.dh ? 1 : 0) + (TOKEN ? 1 : 0);
  constexpr int kMost = 220 * 1024;
  // A CTA's columns in a team of CL (the widest), its threads at W columns each, the
  // stages that fit where `ctas` CTAs share an SM's memory, and what they take.
  auto cols = [&](int CL) { return (a.H / 16 + CL - 1) / CL * 16; };
  auto threads = [&](int W, int CL) { return (cols(CL) / W + 31) / 32 * 32; };
  auto stage = [&](int CL) { return slots * cols(CL) * (F32 ? 4 : 2); };
  auto stages = [&](int W, int CL, int ctas) {
    return std::min(kMostStages, (kMost / ctas - threads(W, CL) * W * 4) / stage(CL));
  };
  auto smem = [&](int W, int CL, int n) { return n * stage(CL) + threads(W, CL) * W * 4; };
  // Two CTAs an SM where both have two stages, else one with as many as fit.  Eight
  // columns a thread keep a row's warps many; 16 fit bf16 rows that would need
  // more than 80 registers in two CTAs (8192 rows of 4096: 72.0 us, with eight 75.3;
  // not for a few rows, 300: 13.4 against 10.8, and not with a gate row for every
  // row, 102.8 against 88.3) or more than 64 in one (4096 rows of 8192: 70.8 us, with
  // eight 109.7).  Wider rows take a cluster (1024 rows of 16384 bf16 56.5 us, in one
  // CTA of 1024 threads 94.3; 1024 of 8192 fp32 52.7, in one 61.4; 600 of 12288 fp32
  // 53.0).  fp32 rows of 2064 and wider in two CTAs spill 88 bytes a thread, with a gate
  // row for every row 172: 2048 rows of 2560 with one each 44.1 us, 0.56 of the copy rate.
  if (const int n = stages(8, 1, 2); n >= 2) {
    const int t = threads(8, 1);
    if (t <= 256) return launch_staged<F32, TOKEN, 8, 1, 256, 2>(job, t, n, smem(8, 1, n), st);
    if (t <= 384) return launch_staged<F32, TOKEN, 8, 1, 384, 2>(job, t, n, smem(8, 1, n), st);
    if constexpr (!F32 && !TOKEN)
      if (threads(16, 1) <= 256 && a.rows > 8 * num_sms())
        return launch_staged<F32, TOKEN, 16, 1, 256, 2>(job, threads(16, 1), n, smem(16, 1, n), st);
  }
  if (threads(8, 1) <= 640) {
    const int n = stages(8, 1, 1);
    return launch_staged<F32, TOKEN, 8, 1, 640, 1>(job, threads(8, 1), n, smem(8, 1, n), st);
  }
  if constexpr (!F32) {
    if (threads(16, 1) <= 512) {
      const int n = stages(16, 1, 1);
      return launch_staged<F32, TOKEN, 16, 1, 512, 1>(job, threads(16, 1), n, smem(16, 1, n), st);
    }
    const int n = stages(16, 2, 1);  // at most 8192 columns a CTA
    return launch_staged<F32, TOKEN, 16, 2, 512, 1>(job, threads(16, 2), n, smem(16, 2, n), st);
  } else {
    if (threads(8, 2) <= 640) {
      const int n = stages(8, 2, 1);
      return launch_staged<F32, TOKEN, 8, 2, 640, 1>(job, threads(8, 2), n, smem(8, 2, n), st);
    }
    const int n = stages(8, 4, 1);  // at most 4096 columns a CTA
    return launch_staged<F32, TOKEN, 8, 4, 512, 1>(job, threads(8, 4), n, smem(8, 4, n), st);
  }
}

}  // namespace

cudaError_t launch_block_norm_grad(bool f32, const BlockNormGradArgs& a, cudaStream_t st) {
  GradJob job{};
  job.a = a;
  job.late = wait_cycles <= 0;
  const bool token = a.gate && a.gate_rows == a.rows;
  if (cudaError_t e = f32 ? token ? launch_grad<true, true>(job, st) : launch_grad<true, false>(job, st)
                          : token ? launch_grad<false, true>(job, st)
                                  : launch_grad<false, false>(job, st))
    return e;
  const bool sum_gate = job.ws_gate != nullptr;
  if (!a.dpre_w && !a.dpost_w && !sum_gate) return cudaSuccess;
  const dim3 grid((a.H + kSumCols - 1) / kSumCols, static_cast<unsigned>(2 + (sum_gate ? job.p.segs : 0)));
  return f32 ? launch_pdl(k_block_norm_grad_sum<true>, grid, dim3(kSumWarps * 32), 0, st, job)
             : launch_pdl(k_block_norm_grad_sum<false>, grid, dim3(kSumWarps * 32), 0, st, job);
}

}  // namespace fc
