// block.h -- launch interface between the C ABI (api.cu) and the kernels that
// stand around the fused boundary: the norms of a block with its gate and
// residual scale (block_norm.cu), their gradient (block_norm_grad.cu),
// microscaled 4-bit quantisation (mx4.cu) and the product of microscaled
// tensors (mx4_matmul.cu).
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

}  // namespace fc
