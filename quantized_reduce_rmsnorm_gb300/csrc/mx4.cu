// mx4.cu -- quantisation of bf16 or fp32 rows to microscaled 4-bit floating
// point and back (format and scale layout: mx4.cuh).
//
// Bound by memory: 2 (bf16) or 4 bytes read and 0.53 written per element, and
// the reverse.  A lane takes 16 elements (one or two 256-bit loads, 8 bytes of
// codes); eight lanes make one word of four scales, so every scale is written
// once, in words, with the bytes past a row's end set to 0.  Measured on GB300, 8192
// x 8192 bf16: to four bits 26.3 us (6.5 TB/s, 0.95 of the measured copy rate; with
// one load in flight 34.2), back 26.4 us; 8192 x 8192 fp32 43.8 and 44.8 us.
#include "block.h"
#include "mx4.cuh"

namespace fc {
namespace {

constexpr int kThreads = 128;
constexpr int kWords = kThreads / 8;  // scale words of a CTA's turn

template <bool F32, int kTurns>  // turns whose loads are in flight together
__global__ void __launch_bounds__(kThreads)
    k_mx4_quantize(const void* x, uint32_t words, int H, uint32_t KT, uint8_t* codes, uint8_t* scales) {
  pdl_begin();
  const int sub = threadIdx.x & 7;
  Raw<F32, 16> r[kTurns];
  int64_t at[kTurns], sw[kTurns];
  bool live[kTurns], word[kTurns];
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const uint32_t w = (blockIdx.x * kTurns + i) * kWords + (threadIdx.x >> 3);
    const uint32_t row = w / KT, kt = w - row * KT;
    const int e = kt * 128 + sub * 16;
    word[i] = w < words;
    live[i] = word[i] && e < H;
    at[i] = static_cast<int64_t>(row) * H + e;
    sw[i] = mx4_scale_word(row, kt, KT);
    if (live[i]) r[i] = load_raw<F32, 16>(x, at[i]);
  }
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    float v[16] = {};
    uint32_t m = 0;
    if (live[i]) {
      m = absmax_raw<F32, 16>(r[i]);
      unpack_raw<F32, 16>(r[i], v);
    }
    mx4_store<16>(v, m, live[i], word[i] && sub == 0, codes + at[i] / 2, scales + sw[i]);
  }
}

template <bool F32, int kTurns>  // turns whose loads are in flight together
__global__ void __launch_bounds__(kThreads)
    k_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, uint32_t words, int H, uint32_t KT, void* out) {
  pdl_begin();
  const int sub = threadIdx.x & 7;
  uint2 c[kTurns];
  uint32_t byte[kTurns];
  int64_t at[kTurns];
  bool live[kTurns];
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const uint32_t w = (blockIdx.x * kTurns + i) * kWords + (threadIdx.x >> 3);
    const uint32_t row = w / KT, kt = w - row * KT;
    const int e = kt * 128 + sub * 16;
    live[i] = w < words && e < H;
    at[i] = static_cast<int64_t>(row) * H + e;
    if (live[i]) {
      c[i] = ld64_stream(codes + at[i] / 2);
      byte[i] = scales[mx4_scale_word(row, kt, KT) + (sub >> 1)];
    }
  }
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    if (!live[i]) continue;
    const float s = mx4_scale(byte[i]);
    float v[16];
    mx4_decode8(c[i].x, s, v);
    mx4_decode8(c[i].y, s, v + 8);
    float2 p[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) p[k] = make_float2(v[2 * k], v[2 * k + 1]);
    store_raw<F32, 16>(out, at[i], pack_raw<F32, 16>(p));
  }
}

template <int kTurns>
dim3 grid_for(uint32_t words) {
  return dim3((words + kWords * kTurns - 1) / (kWords * kTurns));
}
// Three turns a lane where there are CTAs enough, one where more of them start
// sooner (us, one / three turns, bf16 to four bits: 512 x 8192 2.9 / 3.3, 1024 x 8192
// 4.9 / 3.9, 8192 x 8192 34.2 / 26.4).  Reading back to fp32 writes eight bytes for
// each it reads: one turn (1024 x 8192 6.0 / 7.7, 8192 x 8192 44.8 / 45.7).
bool many(uint32_t words) { return words >= 3u << 14; }

}  // namespace

cudaError_t launch_mx4_quantize(bool f32, const void* x, int64_t rows, int H, void* codes,
                                uint8_t* scales, cudaStream_t st) {
  const uint32_t KT = static_cast<uint32_t>(mx4_tiles_k(H));
  const uint32_t words = static_cast<uint32_t>(rows * KT);  // below 2^31: the caller's check
  auto* c = static_cast<uint8_t*>(codes);
  if (many(words))
    return launch_pdl(f32 ? k_mx4_quantize<true, 3> : k_mx4_quantize<false, 3>, grid_for<3>(words), dim3(kThreads), 0,
                      st, x, words, H, KT, c, scales);
  return launch_pdl(f32 ? k_mx4_quantize<true, 1> : k_mx4_quantize<false, 1>, grid_for<1>(words), dim3(kThreads), 0,
                    st, x, words, H, KT, c, scales);
}

cudaError_t launch_mx4_dequantize(bool f32, const void* codes, const uint8_t* scales, int64_t rows,
                                  int H, void* out, cudaStream_t st) {
  const uint32_t KT = static_cast<uint32_t>(mx4_tiles_k(H));
  const uint32_t words = static_cast<uint32_t>(rows * KT);  // below 2^31: the caller's check
  auto* c = static_cast<const uint8_t*>(codes);
  if (f32)
    return launch_pdl(k_mx4_dequantize<true, 1>, grid_for<1>(words), dim3(kThreads), 0, st, c, scales, words, H, KT, out);
  if (many(words))
    return launch_pdl(k_mx4_dequantize<false, 3>, grid_for<3>(words), dim3(kThreads), 0, st, c, scales, words, H, KT, out);
  return launch_pdl(k_mx4_dequantize<false, 1>, grid_for<1>(words), dim3(kThreads), 0, st, c, scales, words, H, KT, out);
}

}  // namespace fc
