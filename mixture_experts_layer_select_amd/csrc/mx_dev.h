// Device code of the microscaled 4-bit format (OCP MXFP4: E2M1 elements, one
// E8M0 scale per 32 of a row), shared by its kernels. Internal to libmoe.so.
//
// A block's scale is 2^e with e = floor(log2(amax)) - 2, so its largest
// element lands in [4, 8) and is held as 4 or 6; e is clamped to the format's
// -127..127 (byte e + 127). A code is the nearest E2M1 value of v / 2^e, ties
// to the even code, saturating at 6: dividing by a power of two is exact and
// v_cvt_scalef32_pk_fp4_f32 rounds this way (checked value by value, ties
// included), so every code is exact. An all-zero block has byte 127; a block
// with a NaN or an infinity has byte 255 (NaN in E8M0) and codes 0.
#pragma once

#include "ffn_dev.h"

namespace moe {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kMxBlock = 32;
constexpr uint32_t kMxNan = 255;

// scale byte of a block from the bits of its largest |v| (integer maximum:
// a NaN's bits are above an infinity's, which are above every number's)
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
    const int biased = (int)(amax_bits >> 23);  // 0 for denormals: below 2^-126, the clamp's side
    const uint32_t b = (uint32_t)max(biased - 2, 0);
    return biased == 255 ? kMxNan : amax_bits == 0 ? 127u : b;
}
// 2^-e of a scale byte (0..252 from mx_scale_byte); 0 for the NaN byte
__device__ __forceinline__ float mx_inverse(uint32_t byte) {
    return byte == kMxNan ? 0.0f : __uint_as_float((254u - byte) << 23);
}
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// eight values times inv = 2^-e -> eight codes, the first in the low nibble
__device__ __forceinline__ uint32_t mx_pack8(const float* v, float inv) {
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0] * inv, v[1] * inv, 1.0f, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2] * inv, v[3] * inv, 1.0f, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4] * inv, v[5] * inv, 1.0f, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6] * inv, v[7] * inv, 1.0f, 3);
    return inv == 0.0f ? 0u : r;
}

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_max_u32(uint32_t v) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xf, 0xf, false);
    return o > v ? o : v;
}

// The codes of this lane's eight values of a block that lies in four
// neighbouring lanes (aligned to 4, all of them active), and the block's scale byte.
__device__ __forceinline__ uint32_t mx_quantise8(const float* v, uint32_t& byte) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]));
    m = dpp_max_u32<0xb1>(m);  // lane ^ 1
    m = dpp_max_u32<0x4e>(m);  // lane ^ 2
    byte = mx_scale_byte(m);
    return mx_pack8(v, mx_inverse(byte));
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
// two fp32 -> packed bf16, round to nearest even (v_cvt_pk_bf16_f32)
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

// D += A B with both operands E2M1 (format 4): lane (l31, hi) holds row l31's
// codes k = 32 hi + [0, 32) of A, and the same of B's column l31, each with
// that block's scale byte; it receives D[8 (r / 4) + 4 hi + r % 4][l31].
// kByte picks the byte of the scale registers. 32x32x64 rather than 16x16x128:
// with register operands the former reached 6.8 PFLOP/s on random codes at one
// wave per SIMD, the latter 4.8 (8.1 and 5.1 on zeros).
template <int kByteA, int kByteB>
__device__ __forceinline__ f32x16 mfma_fp4(u32x4 a, u32x4 b, f32x16 c, uint32_t sa, uint32_t sb) {
    const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, kByteA, (int)sa, kByteB, (int)sb);
}

// a large kernel's lambdas are otherwise left as calls with their captures in memory
#define MX_INLINE __attribute__((always_inline))

// The workgroup barrier of the load ring: this wave's LDS reads are done and no
// memory access moves across it at compile time, but loads stay in flight.
__device__ __forceinline__ void mx_barrier() {
    asm volatile("" ::: "memory");
    barrier_only();
    asm volatile("" ::: "memory");
}

}  // namespace
}  // namespace moe
