// mx4.cuh -- microscaled 4-bit floating point (MXFP4) device helpers.
//
// A block is 32 neighbouring elements of a row.  With m the largest |x| of
// the block and e = floor(log2 m) - 2 (the exponent of the largest e2m1
// value, 6 = 1.5 * 2^2, is 2), the block's scale is 2^e, stored as the byte
// e + 127 (e8m0), and each element's code is x / 2^e rounded to the nearest
// e2m1 value (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign), ties to the even code,
// saturating at 6.  Scaling by a power of two is exact in binary32 (values
// that it makes subnormal are far below 0.25 and round to 0 either way), so a
// code is one rounding of its element.  e is held at -127 or above: a block
// of zeros, and one whose m is below 2^-125, has the byte 0.  A block with an
// infinity or a NaN gets the byte 0xFF, which stands for NaN.
//
// Scales lie in tiles of 128 rows by 4 blocks (512 bytes), tile (r / 128,
// k / 4) at ((r / 128) * ceil(hidden / 128) + k / 4) * 512, and in it row r,
// block k at (r % 32) * 16 + (r / 32 % 4) * 4 + k % 4: the order in which the
// tensor core wants 128 rows' scales in its memory (32 lanes of 16 bytes), so
// a tile goes there with one copy of 512 neighbouring bytes.
#pragma once

#include "device.cuh"

namespace fc {

__host__ __device__ __forceinline__ int64_t mx4_tiles_k(int H) { return (H + 127) / 128; }
// Byte offset of the four scales of row r, blocks 4 * kt .. 4 * kt + 3.
__device__ __forceinline__ int64_t mx4_scale_word(int64_t r, int64_t kt, int64_t KT) {
  return ((r >> 7) * KT + kt) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

// The largest |v| of a block is found on bits: as unsigned numbers the bit patterns
// of non-negative floats order as the floats do, infinity and NaN above all.

// e8m0 byte of a block whose largest |v| has these bits.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t amax_bits) {
  const int E = static_cast<int>(amax_bits >> 23);
  return E == 255 ? 255u : static_cast<uint32_t>(max(E - 2, 0));
}
// 2^-e of that byte (for the NaN byte any factor serves: the scale decides).
__device__ __forceinline__ float mx4_inv_scale(uint32_t byte) {
  return __uint_as_float((254u - min(byte, 252u)) << 23);
}
// 2^e; the byte 0 is 2^-127, a subnormal.
__device__ __forceinline__ float mx4_scale(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7FC00000u)
                      : byte == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}

// Eight floats -> eight e2m1 codes, element 2i in the low nibble of byte i.
__device__ __forceinline__ uint32_t mx4_encode8(const float* v, float inv) {
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = __fmul_rn(v[i], inv);
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}"
      : "=r"(r)
      : "f"(s[0]), "f"(s[1]), "f"(s[2]), "f"(s[3]), "f"(s[4]), "f"(s[5]), "f"(s[6]), "f"(s[7]));
  return r;
}
// Eight codes -> eight floats, times the block's scale.
__device__ __forceinline__ void mx4_decode8(uint32_t w, float scale, float* v) {
  uint32_t h[4];
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}"
        : "=f"(lo), "=f"(hi)
        : "r"(h[i]));
    v[2 * i] = __fmul_rn(lo, scale);
    v[2 * i + 1] = __fmul_rn(hi, scale);
  }
}

// One warp's share of a quantisation: every lane holds W (8 or 16) elements, 32 / W
// neighbouring lanes a block, 128 / W of them one scale word (`live`: the lane's
// elements are inside the row).  Writes the lane's codes and, by the lane with
// `word` (the first of the word's), the word of four scale bytes (0 past the row's
// end).  amax_bits is that of the lane's elements, 0 for a lane that is not live.
template <int W>
__device__ __forceinline__ void mx4_store(const float* v, uint32_t amax_bits, bool live, bool word, uint8_t* codes,
                                          uint8_t* scales) {
  uint32_t m = max(amax_bits, __shfl_xor_sync(kFull, amax_bits, 1));
  if constexpr (W == 8) m = max(m, __shfl_xor_sync(kFull, m, 2));
  const uint32_t byte = live ? mx4_scale_byte(m) : 0u;
  if (live) {
    const float inv = mx4_inv_scale(byte);
    if constexpr (W == 8) {
      *reinterpret_cast<uint32_t*>(codes) = mx4_encode8(v, inv);
    } else {
      uint2 c;
      c.x = mx4_encode8(v, inv);
      c.y = mx4_encode8(v + 8, inv);
      *reinterpret_cast<uint2*>(codes) = c;
    }
  }
  constexpr int kBlock = 32 / W;  // lanes
  uint32_t w = byte | (__shfl_down_sync(kFull, byte, kBlock) << 8);
  w |= __shfl_down_sync(kFull, w, 2 * kBlock) << 16;
  if (word) *reinterpret_cast<uint32_t*>(scales) = w;
}

// 1 / sqrt(v): the hardware's approximation (relative error about 2^-22) and one
// step of Newton's method, which squares the error; what is left is its
// rounding, below 2^-22.  0, infinity and NaN give what the approximation does.
__device__ __forceinline__ float inv_sqrt(float v) {
  const float y = rsqrtf(v);
  const float e = __fmaf_rn(-v * y, y, 1.0f);  // 1 - v y^2
  const float r = __fmaf_rn(0.5f * y, e, y);
  return v > 0.0f && v < __uint_as_float(0x7F800000u) ? r : y;
}

// ------------------------------------------------ rows of bf16 or fp32 --
// W neighbouring elements of a row tensor in 256-bit pieces (coherent loads: an
// output may be the input's own memory).
template <bool F32, int W>
struct Raw {
  static constexpr int kPieces = W * (F32 ? 4 : 2) / 32;
  V8 v[kPieces];
};
template <bool F32, int W>
__device__ __forceinline__ Raw<F32, W> load_raw(const void* base, int64_t elem) {
  Raw<F32, W> r;
  const char* p = static_cast<const char*>(base) + elem * (F32 ? 4 : 2);
#pragma unroll
  for (int i = 0; i < r.kPieces; ++i) r.v[i] = ld256_coherent(p + 32 * i);
  return r;
}
// Weights and gates, which every row re-reads.
template <bool F32, int W>
__device__ __forceinline__ Raw<F32, W> load_weight(const void* base, int64_t elem) {
  Raw<F32, W> r;
  const char* p = static_cast<const char*>(base) + elem * (F32 ? 4 : 2);
#pragma unroll
  for (int i = 0; i < r.kPieces; ++i) r.v[i] = ld256_keep(p + 32 * i);
  return r;
}
// Elements 2i and 2i + 1.
template <bool F32, int W>
__device__ __forceinline__ float2 pair(const Raw<F32, W>& r, int i) {
  if constexpr (F32)
    return make_float2(__uint_as_float(r.v[i / 4].w[2 * i % 8]), __uint_as_float(r.v[i / 4].w[2 * i % 8 + 1]));
  else
    return make_float2(bf_lo(r.v[i / 8].w[i % 8]), bf_hi(r.v[i / 8].w[i % 8]));
}
// Rounds W floats to the row type (bf16: to nearest even; fp32: as they are).
template <bool F32, int W>
__device__ __forceinline__ Raw<F32, W> pack_raw(const float2* f) {
  Raw<F32, W> r;
#pragma unroll
  for (int i = 0; i < W / 2; ++i) {
    if constexpr (F32) {
      r.v[i / 4].w[2 * i % 8] = __float_as_uint(f[i].x);
      r.v[i / 4].w[2 * i % 8 + 1] = __float_as_uint(f[i].y);
    } else {
      r.v[i / 8].w[i % 8] = pack_bf2(f[i].x, f[i].y);
    }
  }
  return r;
}
template <bool F32, int W>
__device__ __forceinline__ void store_raw(void* base, int64_t elem, const Raw<F32, W>& r) {
  char* p = static_cast<char*>(base) + elem * (F32 ? 4 : 2);
#pragma unroll
  for (int i = 0; i < r.kPieces; ++i) st256(p + 32 * i, r.v[i]);
}
// Largest |element| as bits: bf16 without unpacking.
template <bool F32, int W>
__device__ __forceinline__ uint32_t absmax_raw(const Raw<F32, W>& r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < r.kPieces; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k)
      m = F32 ? max(m, r.v[i].w[k] & 0x7FFFFFFFu) : __vmaxu2(m, r.v[i].w[k] & 0x7FFF7FFFu);
  return F32 ? m : max(m << 16, m & 0xFFFF0000u);
}
template <bool F32, int W>
__device__ __forceinline__ void unpack_raw(const Raw<F32, W>& r, float* f) {
#pragma unroll
  for (int i = 0; i < W / 2; ++i) {
    const float2 p = pair<F32, W>(r, i);
    f[2 * i] = p.x, f[2 * i + 1] = p.y;
  }
}

// ------------------------------------------------------------ bounded waits --
// Waits for phase `parity` of the barrier for at most about `cycles` clock cycles;
// false: not complete by then.  One loop, its tries suspended for at most a part of the
// limit.  Measured (us): 64 tokens by 4096 x 4096 6.3, with a loop of polls for short limits
// beside it 7.0, with a first try before the clock is read 6.3 (16 tokens 5.5 against 5.1);
// 8192 x 8192 x 8192 153, with tries of the hardware's own length 160, polled for 162.
__device__ __forceinline__ bool mbar_wait_for(uint64_t* bar, uint32_t parity, int64_t cycles) {
  const long long t0 = clock64();
  uint32_t ok;
  do {
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(static_cast<uint32_t>(cycles >> 11))  // ns
        : "memory");
  } while (!ok && clock64() - t0 < cycles);
  return ok != 0;
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// ------------------------------------------------------- thread-block clusters --
// Barrier of all CTAs of the cluster (whole, converged warps), and the cluster
// address of a CTA's shared memory.
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
}  // namespace fc
