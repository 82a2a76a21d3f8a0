// fp8.cu -- quantisation of bf16 or fp32 rows to 8-bit floating point with a scale for each
// block of 128, or of 128 by 128, and back (fp8.cuh).
//
// Bound by memory: 2 (bf16) or 4 bytes read and 1.03 written per element, and the
// reverse.  A lane takes 16 elements (one or two 256-bit loads, 16 bytes of codes), eight
// lanes a block's part of one row.  A weight's block is one CTA's.  Measured on GB300, 8192 x
// 8192: bf16 to eight bits 30.2 us, 6.7 TB/s (0.98 of the measured copy rate), back 30.6; fp32
// 48.3 and 49.2; a bf16 weight 41.8 (0.71: a CTA loads its one block, meets at a barrier and
// encodes it with nothing more on its way).
#include "block.h"
#include "fp8.cuh"

namespace fc {
namespace {

constexpr int kThreads = 128;
constexpr int kBlocks = kThreads / 8;  // blocks (of one row) of a CTA's turn

template <bool F32, int kTurns>  // turns whose loads are in flight together
__global__ void __launch_bounds__(kThreads)
    k_fp8_quantize(const void* x, uint32_t blocks, int H, uint32_t KB, uint8_t* codes, float* scales) {
  pdl_begin();
  const int sub = threadIdx.x & 7;
  Raw<F32, 16> r[kTurns];
  int64_t at[kTurns];
  bool live[kTurns];
  const uint32_t b0 = blockIdx.x * (kTurns * kBlocks) + (threadIdx.x >> 3);
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const uint32_t b = b0 + i * kBlocks;
    const uint32_t row = b / KB, kb = b - row * KB;
    const int e = kb * 128 + sub * 16;
    live[i] = b < blocks && e < H;
    at[i] = static_cast<int64_t>(row) * H + e;
    if (live[i]) r[i] = load_raw<F32, 16>(x, at[i]);
  }
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    uint32_t m = live[i] ? absmax_raw<F32, 16>(r[i]) : 0u;
#pragma unroll
    for (int k = 1; k < 8; k <<= 1) m = max(m, __shfl_xor_sync(kFull, m, k));
    if (!live[i]) continue;
    const float s = fp8_scale(m);
    st128(codes + at[i], fp8_encode16<F32>(r[i], s));
    if (sub == 0) scales[b0 + i * kBlocks] = s;
  }
}

// One block of 128 by 128 a CTA: 256 threads, four 16-element pieces of a row each.
template <bool F32>
__global__ void __launch_bounds__(256)
    k_fp8_quantize_square(const void* x, int64_t rows, int H, uint32_t KB, uint8_t* codes, float* scales) {
  __shared__ uint32_t red[8];
  pdl_begin();
  const uint32_t rb = blockIdx.x / KB, kb = blockIdx.x - rb * KB;
  const int e = kb * 128 + (threadIdx.x & 7) * 16;
  const int64_t row0 = static_cast<int64_t>(rb) * 128 + (threadIdx.x >> 3);
  Raw<F32, 16> r[4];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (row0 + 32 * i < rows && e < H) {
      r[i] = load_raw<F32, 16>(x, (row0 + 32 * i) * H + e);
      m = max(m, absmax_raw<F32, 16>(r[i]));
    }
  m = __reduce_max_sync(kFull, m);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, red[i]);
  const float s = fp8_scale(m);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (row0 + 32 * i < rows && e < H) st128(codes + (row0 + 32 * i) * H + e, fp8_encode16<F32>(r[i], s));
  if (threadIdx.x == 0) scales[blockIdx.x] = s;
}

// shift: 0, or 7 for blocks of 128 rows.
template <bool F32, int kTurns>
__global__ void __launch_bounds__(kThreads)
    k_fp8_dequantize(const uint8_t* codes, const float* scales, uint32_t blocks, int H, uint32_t KB, int shift, void* out) {
  pdl_begin();
  const int sub = threadIdx.x & 7;
  uint4 c[kTurns];
  float s[kTurns];
  int64_t at[kTurns];
  bool live[kTurns];
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const uint32_t b = (blockIdx.x * kTurns + i) * kBlocks + (threadIdx.x >> 3);
    const uint32_t row = b / KB, kb = b - row * KB;
    const int e = kb * 128 + sub * 16;
    live[i] = b < blocks && e < H;
    at[i] = static_cast<int64_t>(row) * H + e;
    if (live[i]) {
      c[i] = ld128_stream(codes + at[i]);
      s[i] = scales[static_cast<int64_t>(row >> shift) * KB + kb];
    }
  }
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    if (!live[i]) continue;
    float2 v[8];
    fp8_decode16(c[i], s[i], v);
    store_raw<F32, 16>(out, at[i], pack_raw<F32, 16>(v));
  }
}

template <int kTurns>
dim3 grid_for(uint32_t blocks) {
  return dim3((blocks + kBlocks * kTurns - 1) / (kBlocks * kTurns));
}
// bf16: three turns a lane where there are CTAs enough, one where more of them start sooner
// (us, one / three turns, quantising: 1024 x 8192 5.5 / 6.3, 2048 x 8192 9.4 / 9.2, 8192 x
// 8192 34.1 / 30.2; back 1024 5.3 / 5.4, 8192 33.8 / 30.6).  fp32 has twice the bytes in
// flight: one turn (8192 x 8192 48.3 / 48.7, back 49.2).
bool many(bool f32, uint32_t blocks) { return !f32 && blocks >= 1u << 17; }

}  // namespace

cudaError_t launch_fp8_quantize(bool f32, bool square, const void* x, int64_t rows, int H, void* codes, float* scales,
                                cudaStream_t st) {
  const uint32_t KB = static_cast<uint32_t>((H + 127) / 128);
  auto* c = static_cast<uint8_t*>(codes);
  if (square)
    return launch_pdl(f32 ? k_fp8_quantize_square<true> : k_fp8_quantize_square<false>,
                      dim3(static_cast<uint32_t>((rows + 127) / 128) * KB), dim3(256), 0, st, x, rows, H, KB, c, scales);
  const uint32_t blocks = static_cast<uint32_t>(rows * KB);  // below 2^31: the caller's check
  if (many(f32, blocks))
    return launch_pdl(k_fp8_quantize<false, 3>, grid_for<3>(blocks), dim3(kThreads), 0, st, x, blocks, H, KB, c, scales);
  return launch_pdl(f32 ? k_fp8_quantize<true, 1> : k_fp8_quantize<false, 1>, grid_for<1>(blocks), dim3(kThreads), 0, st,
                    x, blocks, H, KB, c, scales);
}

cudaError_t launch_fp8_dequantize(bool f32, bool square, const void* codes, const float* scales, int64_t rows, int H,
                                  void* out, cudaStream_t st) {
  const uint32_t KB = static_cast<uint32_t>((H + 127) / 128);
  const uint32_t blocks = static_cast<uint32_t>(rows * KB);
  const int shift = square ? 7 : 0;
  auto* c = static_cast<const uint8_t*>(codes);
  if (many(f32, blocks))
    return launch_pdl(k_fp8_dequantize<false, 3>, grid_for<3>(blocks), dim3(kThreads), 0, st, c, scales, blocks, H, KB,
                      shift, out);
  return launch_pdl(f32 ? k_fp8_dequantize<true, 1> : k_fp8_dequantize<false, 1>, grid_for<1>(blocks), dim3(kThreads),
                    0, st, c, scales, blocks, H, KB, shift, out);
}

}  // namespace fc
