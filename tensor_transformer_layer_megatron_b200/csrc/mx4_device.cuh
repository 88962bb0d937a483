// Microscaled 4-bit floating point: the block formats, shared by the quantisers (mx4.cu) and the
// products' fused epilogues (gemm_mx4.cu).
//
// An element is e2m1 (1 sign, 2 exponent, 1 mantissa bit): +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}. Blocks
// run along the summed axis. MXFP4 (OCP Microscaling Formats v1.0): 32 elements share 2^e, held
// as the byte e + 127, e = floor(log2 amax) - 2. NVFP4: 16 elements share an e4m3 scale
// s = e4m3(amax / (6 f)), and the tensor a factor f.
//
// Every rounding decision is the one exact arithmetic takes: x 2^-e is exact in fp32, and so is
// x / f for a power of two f; x / (f s) is a correctly rounded quotient, which can meet a border
// between two elements (at most 3 significant bits) only where the exact quotient does: x / f
// and border * s (at most 7 bits) differ by at least one unit in the 24th bit of x / f, more
// than half a unit of the quotient.
#pragma once
#include <cuda_fp16.h>

#include "mgt_device.cuh"

namespace mgt {

constexpr int kMxfp4 = 0;
constexpr int kNvfp4 = 1;

// Let the next kernel of the stream, where it was launched programmatically, start as soon as every
// CTA of this one has come here. It still waits for this kernel's results (grid_dependency_wait);
// what it does before is its set-up, and in the products with few rows the fetch of weights into
// L2. Each kernel that calls this waits for its own predecessor, so results stay ordered along the
// stream.
__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <int FMT>
struct Mx4Fmt {
  static constexpr int kBlock = FMT == kMxfp4 ? 32 : 16;  // elements that share a scale
  static constexpr int kTileCols = 4 * kBlock;            // columns of one 512-byte scale tile
};

// Byte offset of the scale of row r, block b in an operand of leading dimension ld: tiles of
// 128 rows by 4 blocks, in a tile 16 (r % 32) + 4 (r % 128 / 32) + b % 4. That is the order in
// which tcgen05.cp (32x128b, four warps) fills four tensor-memory columns.
template <int FMT>
__device__ __forceinline__ long long mx4_scale_off(long long r, int b, long long ld) {
  return ((r >> 7) * (ld / Mx4Fmt<FMT>::kTileCols) + (b >> 2)) * 512 + 16 * (r & 31) +
         4 * ((r >> 5) & 3) + (b & 3);
}

// The fp32 value of a scale byte (without the tensor's factor).
template <int FMT>
__device__ __forceinline__ float mx4_scale_value(uint32_t byte) {
  if constexpr (FMT == kMxfp4) {
    if (byte == 255u) return __uint_as_float(0x7fc00000u);
    return __uint_as_float(byte ? byte << 23 : 0x00400000u);  // 2^-127 is subnormal
  } else {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)byte));
    return __half2float(__ushort_as_half((unsigned short)(h2 & 0xffffu)));
  }
}

// Tensor factor as the quantisers use it. Below 2^-100 the factor times a scale could be subnormal,
// and below 2^-128 its reciprocal is no fp32 number: such a factor is `tiny`, f and inv are those of
// 2^64 times it, and what it divides has to be multiplied by 2^64 first (mx4_lift, or in a patch by
// quantize_patch).
constexpr float kLift = 1.8446744e19f;  // 2^64
struct Mx4Factor {
  float f, inv;
  bool tiny;
};
template <int FMT>
__device__ __forceinline__ Mx4Factor mx4_factor(const float* factor) {
  Mx4Factor t = {1.f, 1.f, false};
  if (FMT == kNvfp4 && factor) {
    t.f = factor[1];
    t.tiny = t.f < 7.8886091e-31f;
    if (t.tiny) t.f *= kLift;
    t.inv = 1.0f / t.f;
  }
  return t;
}
// Values for a tiny factor: times 2^64; those beyond 4096 f saturate wherever they lie and are cut off
// there, infinities and NaN stay.
template <int N>
__device__ __forceinline__ void mx4_lift(float (&v)[N], const Mx4Factor& f) {
  const float most = 4096.0f * f.f;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (fabsf(v[i]) <= 3.4028234e38f) v[i] = fminf(fmaxf(v[i] * kLift, -most), most);
}

// What a block's elements are multiplied by, and the byte that stands for its scale.
struct Mx4Block {
  float inv;      // mxfp4: 2^-e. nvfp4: 1 / (f s), within two units in the last place
  float fs;       // nvfp4: f s
  uint32_t byte;  // mxfp4: e + 127 (255 = NaN). nvfp4: e4m3 (0x7f = NaN)
  uint32_t mask;  // codes are ANDed with it: 0 for a block without a usable scale
  bool wide;      // nvfp4: x / (f s) may leave fp32's range
};

// From the largest |x| of the block as fp32 bits (NaN above infinity above every number). A
// block that holds an infinity or a NaN gets the scale NaN and zero codes.
template <int FMT>
__device__ __forceinline__ Mx4Block mx4_block(uint32_t amax_bits, const Mx4Factor& f) {
  Mx4Block q;
  if constexpr (FMT == kMxfp4) {
    const int eb = (int)(amax_bits >> 23);  // floor(log2 amax) + 127; 0 for subnormals
    const bool bad = eb == 255;
    q.byte = bad ? 255u : (uint32_t)max(eb - 2, 0);
    q.inv = bad ? 0.f : __uint_as_float((254u - q.byte) << 23);
    q.mask = bad ? 0u : 0xffffffffu;
    q.fs = 0.f;
    q.wide = false;
  } else {
    // t = amax / (6 f): the quotient by 6 from its rounded reciprocal and one residual, correctly
    // rounded (see mx4_scaled)
    constexpr float kSixth = 1.0f / 6.0f;
    const float u = fminf(__uint_as_float(amax_bits) * f.inv, 3.4028234e38f);
    const float y = u * kSixth;
    const float t = fmaf(fmaf(-y, 6.0f, u), kSixth, y);
    uint16_t e;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(e) : "f"(0.f), "f"(t));
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(e));
    const float s = __half2float(__ushort_as_half((unsigned short)(h2 & 0xffffu)));
    const bool bad = amax_bits >= 0x7f800000u;
    q.byte = bad ? 0x7fu : (uint32_t)(e & 0xffu);
    q.mask = (bad || s == 0.f) ? 0u : 0xffffffffu;
    q.fs = f.f * s;
    q.inv = q.mask ? f.inv * rcp_approx(s) : 0.f;
    q.wide = t > 896.0f;
  }
  return q;
}

// The scaled element. nvfp4: x / (f s) by a product with the reciprocal and one residual
// correction (P. Markstein, Computation of elementary functions on the IBM RISC System/6000
// processor, 1990): the residual is exact, so the value that the last step rounds is within
// 2^-45 of the quotient, which is far less than an unequal quotient's distance from a border.
template <int FMT>
__device__ __forceinline__ float mx4_scaled(float x, const Mx4Block& q) {
  const float y = x * q.inv;
  if constexpr (FMT == kMxfp4) return y;
  return fmaf(fmaf(-y, q.fs, x), q.inv, y);
}
// The same for a block whose quotients may overflow (a kept factor far too small: they saturate):
// first x / f, clamped to fp32's range, then by s.
__device__ __forceinline__ float mx4_scaled_wide(float x, uint32_t byte, float inv_f) {
  return fmaxf(fminf(x * inv_f, 3.4028234e38f), -3.4028234e38f) /
         mx4_scale_value<kNvfp4>(byte);
}

// Two fp32 values to two codes in the low byte (lo in its low half).
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{ .reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tcvt.u32.u8 %0, b; }"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r;
}

// Eight fp32 values to eight e2m1 codes (round to nearest, ties to even, saturating at 6), the
// first in the low four bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{ .reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3}; }"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

template <int FMT>
__device__ __forceinline__ uint32_t mx4_codes8(const float (&x)[8], const Mx4Block& q,
                                               const Mx4Factor& f) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = mx4_scaled<FMT>(x[i], q);
  if (FMT == kNvfp4 && q.wide) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = mx4_scaled_wide(x[i], q.byte, f.inv);
  }
  return e2m1x8(v) & q.mask;
}

// Eight e2m1 codes to fp32.
__device__ __forceinline__ void e2m1x8_values(uint32_t w, float (&v)[8]) {
  uint32_t h[4];
  asm("{ .reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3; }"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
// Larger of two pairs of 16-bit values.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// z cut off at +-most (a positive number); NaN stays NaN.
__device__ __forceinline__ float cut_off(float z, float most) {
  float r;
  asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(z), "f"(most));
  return r;
}

// Activation of a gated block and its derivative. ACT: 0 silu, 1 gelu (erf), 2 gelu (tanh). A
// block's scale follows its largest value, so a value counts by its relative error however small
// it is: Phi(z) = erfc(-z / sqrt 2) / 2 and (1 + tanh y) / 2 = 1 / (1 + e^-2y) keep it in the
// negative tail, where 1 + erf and 1 + tanh cancel.
template <int ACT>
__device__ __forceinline__ void gate_and_grad(float z, float& h, float& dh) {
  if constexpr (ACT == 0) {
    // sigmoid(z) = 2^-7 / (2^-7 + 2^-7 e^-z): the special-function unit's reciprocal is zero where
    // its argument passes 2^126, which 1 + e^-z does at z = -87.3, where z sigmoid(z) is a normal
    // number yet (down to -91.8); the scaled sum does at -92.2. Relative error about 2^-21 + |z| 2^-24
    // (the exponent's product, ex2.approx, rcp.approx), far below the 2^-3 of an element; a larger shift
    // would cost bits of the exponent near z = 0. With expf and an IEEE division, within 2^-22, the
    // backward of 2048 x 11008 took 91 us instead of 76.
    const float s = 0x1p-7f * rcp_approx(0x1p-7f + ex2_approx(fmaf(z, -1.4426950408889634f, -7.0f)));
    h = z * s;
    dh = s * fmaf(z, 1.0f - s, 1.0f);
  } else if constexpr (ACT == 1) {
    const float c = 0.5f * erfcf(z * -0.7071067811865476f);
    h = z * c;
    dh = fmaf(z * 0.3989422804014327f, expf(-0.5f * z * z), c);
  } else {
    const float k = 0.7978845608028654f;  // sqrt(2 / pi)
    // At |z| = 64, s is 0 or 1 to every bit and dh is s. What they are made of is taken there beyond,
    // where z^2 and z^3 would overflow and make NaN of 0 * inf (a NaN stays one). The quarter: 1 + e^-2y
    // overflows at -2y = 88.7, where z s is a normal number yet (up to 89.6).
    const float b = cut_off(z, 64.0f), b2 = b * b;
    const float s =
        0.25f * (1.0f / (0.25f + expf(fmaf(-2.0f * k * b, fmaf(0.044715f, b2, 1.0f), -1.3862944f))));
    h = z * s;
    dh = s * fmaf(b * (1.0f - s), 2.0f * k * fmaf(0.134145f, b2, 1.0f), 1.0f);
  }
}

}  // namespace mgt
