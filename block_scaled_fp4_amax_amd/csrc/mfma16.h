// mfma16.h -- decoding E2M1 codes to the 16-bit operands of gfx950's matrix
// instructions (device only).
//
// MXFP4 decodes to bf16: +-G[m] 2^k has at most two significant bits and bf16
// has binary32's exponents, so it is exact.  NVFP4 and AMD-FP4 decode to FP16:
// G[m] d has at most six significant bits, and FP16 has a packed multiply where
// bf16 has none.  To stay within FP16's range, d is decoded as d / 2^kShift
// (2^8 for E4M3, 2^4 for UE5M3): the products' magnitudes are then 0 or within
// [2^-18, 10.5] (E4M3) and [2^-22, 43008] (UE5M3) and multiples of 2^-24, so they
// are exact; the caller multiplies its sums by kUnshift.
#pragma once

#include "fp4q_device.h"

namespace fp4q {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// BIAS: 0 (MXFP4), 7 (E4M3) or 15 (UE5M3)
template <int BIAS>
struct Dec {
    static constexpr bool kBf16 = BIAS == 0;
    static constexpr int kBlock = BIAS == 0 ? 32 : 16;
    static constexpr float kUnshift = BIAS == 0 ? 1.0f : BIAS == 7 ? 256.0f : 16.0f;

    // A scale byte as the decoders below take it: 2^k in binary32 (MXFP4; the
    // conversions read the exponent alone, so byte 0 is 2^-127, and byte 0xFF gives
    // NaN) or d / 2^kShift twice in FP16.
    static __device__ __forceinline__ uint32_t scale(uint32_t byte)
    {
        if constexpr (BIAS == 0) return byte << 23;
        // E4M3's fields shifted into FP16's read as d 2^-8, subnormals included
        if constexpr (BIAS == 7) return byte * 0x00800080u;
        // UE5M3's largest exponent is FP16's infinity: through binary32, whose
        // fields at bias 15 read as d 2^-112 (subnormals included)
        const float d = __uint_as_float(byte << 20) * 0x1p108f;
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(d, d));
    }

    // The two codes of byte B of w, times the scale.
    template <int B>
    static __device__ __forceinline__ uint32_t pair(uint32_t w, uint32_t s)
    {
        if constexpr (BIAS == 0) {
            return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, __uint_as_float(s), B));
        } else {
            const f16x2_t g = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, B));
            return __builtin_bit_cast(uint32_t, g * __builtin_bit_cast(f16x2_t, s));
        }
    }

    // The eight codes of w, in order.
    static __device__ __forceinline__ uint4 octet(uint32_t w, uint32_t s)
    {
        return make_uint4(pair<0>(w, s), pair<1>(w, s), pair<2>(w, s), pair<3>(w, s));
    }

    // Two binary32 values rounded to the operands' type.
    static __device__ __forceinline__ uint32_t round2(float a, float b)
    {
        if constexpr (BIAS == 0) {
            const bf16x2_t v = {(__bf16)a, (__bf16)b};
            return __builtin_bit_cast(uint32_t, v);
        } else {
            const f16x2_t v = {(_Float16)a, (_Float16)b};
            return __builtin_bit_cast(uint32_t, v);
        }
    }

    // What round2 has left of them, rounded too.
    static __device__ __forceinline__ uint32_t rest2(float a, float b, uint32_t rounded)
    {
        if constexpr (BIAS == 0) {
            return round2(a - __uint_as_float(rounded << 16), b - __uint_as_float(rounded & 0xFFFF0000u));
        } else {
            const f16x2_t v = __builtin_bit_cast(f16x2_t, rounded);
            return round2(a - (float)v[0], b - (float)v[1]);
        }
    }

    static constexpr uint32_t kOnes = BIAS == 0 ? 0x3F803F80u : 0x3C003C00u;

    // C += A B with A [16 rows x 32], B [32 x 16 columns]: lane l holds A's row
    // l % 16 and B's column l % 16 at places 8 (l / 16) .. + 7 of the summed
    // axis, and C's column l % 16 at rows 4 (l / 16) .. + 3.
    static __device__ __forceinline__ f32x4_t mfma(uint4 a, uint4 b, f32x4_t c)
    {
        if constexpr (BIAS == 0)
            return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                           c, 0, 0, 0);
        else
            return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b),
                                                          c, 0, 0, 0);
    }
};

// Decoding to bf16 for every format, for products whose other operand needs
// binary32's exponents (activations and gradients of any size): G[m] d has at
// most six significant bits, so the upper halves of the binary32 products are the
// bf16 values.
template <int BIAS>
struct DecBf16 {
    // 2^k (MXFP4) or d in binary32: a byte's fields shifted to binary32's read as
    // d 2^(BIAS - 127), subnormals included
    static __device__ __forceinline__ float scale(uint32_t byte)
    {
        if constexpr (BIAS == 0) return __uint_as_float(byte << 23);
        return __uint_as_float(byte << 20) * (BIAS == 7 ? 0x1p120f : 0x1p112f);
    }

    template <int B>
    static __device__ __forceinline__ uint32_t pair(uint32_t w, float s)
    {
        if constexpr (BIAS == 0) return Dec<0>::pair<B>(w, __float_as_uint(s));
        const auto g = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, B);
        return __builtin_amdgcn_perm(__float_as_uint(g[1] * s), __float_as_uint(g[0] * s), 0x07060302u);
    }

    static __device__ __forceinline__ uint4 octet(uint32_t w, float s)
    {
        return make_uint4(pair<0>(w, s), pair<1>(w, s), pair<2>(w, s), pair<3>(w, s));
    }
};

}  // namespace fp4q
