// block.h -- launch interface between the C ABI (api.cu) and the kernels that
// stand around the fused boundary: the norms of a block with its gate and
// residual scale (block_norm.cu), their gradient (block_norm_grad.cu),
// microscaled 4-bit quantisation (mx4.cu) and the product of microscaled
// tensors (mx4_matmul.cu); and of those that a feed-forward block adds: layer norm
// and its gradient (layer_norm.cu, layer_norm_grad.cu), 8-bit floating point and its
// product (fp8.cu, fp8_matmul.cu), the gated feed-forward and its gradient (gated_ffn.cu).
#pragma once

#include "internal.h"

namespace fc {

// A row of `hidden` elements is held in the registers of one CTA: at most
// 1024 threads of 16 elements each.
constexpr int kBlockNormMaxHidden = 16384;

// Clock cycles after which the product gives up waiting for a copy or a product and
// reports FC_ERR_CUDA: 2^31, about a second.  Read at a launch.  The gradient's rows have
// the whole 2^31 whatever it is (a limit of their own, polled for, makes 8192 x 5120 87.4
// us instead of 85.3), but with 0 they all count as late.  Waits that let work in
// flight end before the memory it uses goes always have the whole 2^31.
extern int64_t wait_cycles;

struct BlockNormArgs {
  const void* x;
  const void* res_in;
  void* res_out;
  void* y;              // NULL: not written
  void* y_codes;        // NULL: not quantised
  uint8_t* y_scales;
  const void* post_w;   // NULL: the block's output is not normed
  const void* gate;     // NULL: none
  const void* pre_w;    // NULL: no y
  int64_t rows;
  int64_t gate_seg;     // neighbouring rows that share one row of gate
  int H;
  int ahead;            // set at the launch
  float alpha, beta;    // residual scale, block scale
  float eps_post, eps_pre;
};
cudaError_t launch_block_norm(bool f32, BlockNormArgs a, cudaStream_t st);

// CTAs of the gradient kernel at most (152 SMs, up to 4 on each); its
// workspace is sized by this and not by the device, so that a caller can ask
// for it without a GPU.
constexpr int kNormGradMaxCtas = 608;

struct BlockNormGradArgs {
  const void* x;
  const void* h;
  const void* dy;       // NULL: no gradient through y
  const void* dh;       // NULL: no gradient through residual_out
  const void* post_w;
  const void* gate;
  const void* pre_w;
  void* dx;
  void* dres;           // NULL: not wanted
  void* dgate;          // NULL: not wanted; so for the two below
  float* dpost_w;
  float* dpre_w;
  float* ws;
  int32_t* status;      // NULL, or word 0 set to FC_ERR_CUDA if a staged row never lands
  int64_t rows;
  int64_t gate_rows;
  int H;
  float alpha, beta;
  float eps_post, eps_pre;
};
cudaError_t launch_block_norm_grad(bool f32, const BlockNormGradArgs& a, cudaStream_t st);

struct LayerNormArgs {
  const void* x;
  const void* res_in;   // NULL: h is x, and not written
  void* res_out;
  void* y;
  const void* weight;   // NULL: ones
  const void* bias;     // NULL: none
  float* stats;         // NULL, or [rows][2]: mean and inverse deviation
  int64_t rows;
  int H;
  int ahead;            // set at the launch
  float eps;
};
cudaError_t launch_layer_norm(bool f32, LayerNormArgs a, cudaStream_t st);

struct LayerNormGradArgs {
  const void* h;
  const float* stats;
  const void* dy;
  const void* dh;       // NULL: none
  const void* weight;   // NULL: ones
  void* dx;
  float* dweight;       // NULL: not wanted
  float* dbias;         // NULL: not wanted
  float* ws;
  int32_t* status;      // NULL, or word 0 set to FC_ERR_CUDA if a staged row never lands
  int64_t rows;
  int H;
};
cudaError_t launch_layer_norm_grad(bool f32, const LayerNormGradArgs& a, cudaStream_t st);

cudaError_t launch_mx4_quantize(bool f32, const void* x, int64_t rows, int H, void* codes,
                                uint8_t* scales, cudaStream_t st);
cudaError_t launch_mx4_dequantize(bool f32, const void* codes, const uint8_t* scales, int64_t rows,
                                  int H, void* out, cudaStream_t st);

struct Mx4MatmulArgs {
  const void* x_codes;
  const uint8_t* x_scales;
  const void* w_codes;
  const uint8_t* w_scales;
  void* out;
  int32_t* status;      // NULL, or word 0 set to FC_ERR_CUDA if a bounded wait ran out
  int64_t rows;         // tokens
  int64_t features;
  int H;
  bool out_f32;
};
cudaError_t launch_mx4_matmul(const Mx4MatmulArgs& a, cudaStream_t st);

// 8-bit floating point with a scale for each block of 128 (square: of 128 by 128).
cudaError_t launch_fp8_quantize(bool f32, bool square, const void* x, int64_t rows, int H, void* codes, float* scales,
                                cudaStream_t st);
cudaError_t launch_fp8_dequantize(bool f32, bool square, const void* codes, const float* scales, int64_t rows, int H,
                                  void* out, cudaStream_t st);

struct Fp8MatmulArgs {
  const void* x_codes;
  const float* x_scales;  // [rows, ceil(H / 128)]
  const void* w_codes;
  const float* w_scales;  // [ceil(features / 128), ceil(H / 128)]
  void* out;
  int32_t* status;        // NULL, or word 0 set to FC_ERR_CUDA if a bounded wait ran out
  int64_t rows;           // tokens
  int64_t features;
  int H;
  bool out_f32;
};
cudaError_t launch_fp8_matmul(const Fp8MatmulArgs& a, cudaStream_t st);

enum Activation : int { kSilu = 0, kGeluTanh = 1 };

struct GatedFfnArgs {
  const void* x;          // [rows, H]
  const void* w_gate;     // [features, H]
  const void* w_up;
  void* out;              // [rows, features]
  void* gate;             // NULL: not kept
  void* up;
  int32_t* status;
  int64_t rows;
  int64_t features;
  int H;
  int activation;
};
cudaError_t launch_gated_ffn(const GatedFfnArgs& a, cudaStream_t st);

// Tokens up to which, and features from which on, the kernel of few tokens makes dx.
constexpr int64_t kFewDx = 128, kFewDxFeatures = 512;
// bf16 numbers that stand for each of the gradient's factors dg and du, and that the
// workspace holds, where the caller leaves it to the sizes.  With one the results are off by
// 1.41 times what their own rounding leaves (root mean square: the factors' roundings are
// as large as it and independent of it, so the squares add up), with two by that alone.  Two
// for few tokens, whose gradients the weights' bytes bound, and up to 2^19 factors, where
// they cost 5 to 12 us (us, one / two numbers, tokens x features x hidden next to the border:
// 1024 x 528 x 1024 13.0 / 18.2, 2048 x 272 x 1024 17.3 / 26.4, 140 x 3792 x 4096 42.5 / 54.2;
// further up 1024 x 1040 x 1024 18.4 / 28.2, 777 x 4112 x 2064 48.9 / 89.0, 4096 x 8192 x 4096
// 650 / 1312).
constexpr int64_t kTwoTermFactors = 1 << 19;
constexpr int gated_ffn_terms(int64_t rows, int64_t features) {
  return rows <= kFewDx || rows * features <= kTwoTermFactors ? 2 : 1;
}

struct GatedFfnGradArgs {
  const void* x;
  const void* w_gate;
  const void* w_up;
  const void* gate;
  const void* up;
  const void* dout;       // [rows, features]
  void* dx;               // NULL: not wanted; so for the weights' two
  void* dw_gate;
  void* dw_up;
  void* ws;               // [terms][2][rows, features] bf16
  int32_t* status;
  int64_t rows;
  int64_t features;
  int H;
  int activation;
  int terms;              // gated_ffn_terms, or 2
};
cudaError_t launch_gated_ffn_grad(const GatedFfnGradArgs& a, cudaStream_t st);

}  // namespace fc
