// mx4.cu -- quantisation of bf16 or fp32 rows to microscaled 4-bit floating
// point and back (format and scale layout: mx4.cuh).
//
// Bound by memory: 2 (bf16) or 4 bytes read and 0.53 written per element, and
// the reverse.  A lane takes 16 elements (one or two 256-bit loads, 8 bytes of
// codes); eight lanes make one word of four scales, so every scale is written
// once, in words, with the bytes past a row's end set to 0.
#include "block.h"
#include "mx4.cuh"

namespace fc {
namespace {

constexpr int kThreads = 256;

template <bool F32>
__global__ void __launch_bounds__(kThreads)
    k_mx4_quantize(const void* x, int64_t words, int H, int KT, uint8_t* codes, uint8_t* scales) {
  pdl_begin();
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 8);
  // a warp's four words are handled together: every lane makes as many turns
  const int sub = threadIdx.x & 7;
  for (int64_t w0 = static_cast<int64_t>(blockIdx.x) * (kThreads / 8) + (threadIdx.x >> 5) * 4;
       w0 < words; w0 += step) {
    const int64_t w = w0 + ((threadIdx.x >> 3) & 3);
    const bool word = w < words;
    const int64_t row = word ? w / KT : 0;
    const int kt = static_cast<int>(w - row * KT);
    const int e = kt * 128 + sub * 16;
    const bool live = word && e < H;
    const int64_t at = row * H + e;
    float v[16] = {};
    uint32_t m = 0;
    if (live) {
      const Raw16<F32> r = load_raw16<F32>(x, at);
      m = absmax_raw<F32>(r);
      unpack_raw<F32>(r, v);
    }
    mx4_store16(v, m, live, word && sub == 0, codes + at / 2,
                scales + (word ? mx4_scale_word(row, kt, KT) : 0));
  }
}

template <bool F32>
__global__ void __launch_bounds__(kThreads)
    k_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t words, int H, int KT,
                     void* out) {
  pdl_begin();
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 8);
  const int sub = threadIdx.x & 7;
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / 8) + (threadIdx.x >> 3);
       w < words; w += step) {
    const int64_t row = w / KT;
    const int kt = static_cast<int>(w - row * KT);
    const int e = kt * 128 + sub * 16;
    if (e >= H) continue;
    const int64_t at = row * H + e;
    const uint2 c = ld64_stream(codes + at / 2);
    const float s = mx4_scale(scales[mx4_scale_word(row, kt, KT) + (sub >> 1)]);
    float v[16];
    mx4_decode8(c.x, s, v);
    mx4_decode8(c.y, s, v + 8);
    store_raw16<F32>(out, at, pack_raw<F32>(v));
  }
}

unsigned grid_for(int64_t words) {
  const int64_t want = (words + kThreads / 8 - 1) / (kThreads / 8);
  return static_cast<unsigned>(want < (1 << 30) ? want : (1 << 30));
}

}  // namespace

cudaError_t launch_mx4_quantize(bool f32, const void* x, int64_t rows, int H, void* codes,
                                uint8_t* scales, cudaStream_t st) {
  const int KT = static_cast<int>(mx4_tiles_k(H));
  const int64_t words = rows * KT;
  auto* c = static_cast<uint8_t*>(codes);
  return f32 ? launch_pdl(k_mx4_quantize<true>, dim3(grid_for(words)), dim3(kThreads), 0, st, x, words, H,
                          KT, c, scales)
             : launch_pdl(k_mx4_quantize<false>, dim3(grid_for(words)), dim3(kThreads), 0, st, x, words, H,
                          KT, c, scales);
}

cudaError_t launch_mx4_dequantize(bool f32, const void* codes, const uint8_t* scales, int64_t rows,
                                  int H, void* out, cudaStream_t st) {
  const int KT = static_cast<int>(mx4_tiles_k(H));
  const int64_t words = rows * KT;
  auto* c = static_cast<const uint8_t*>(codes);
  return f32 ? launch_pdl(k_mx4_dequantize<true>, dim3(grid_for(words)), dim3(kThreads), 0, st, c, scales,
                          words, H, KT, out)
             : launch_pdl(k_mx4_dequantize<false>, dim3(grid_for(words)), dim3(kThreads), 0, st, c, scales,
                          words, H, KT, out);
}

}  // namespace fc
