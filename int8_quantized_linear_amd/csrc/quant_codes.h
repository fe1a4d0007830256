// quant_codes.h -- int8 and fp8 (E4M3) codes of fp32 values, shared by the row quantizers.
#pragma once

#include "ql_internal.h"

namespace ql {

// rint(x / s) clamped to [-127, 127], as (code + 128) in the byte `sel` of `acc`.
// x / s is taken as q0 = RN(x * y), r = x - q0 * s (exact, one fma), RN(q0 + r * y) with
// y = RN(1 / s) divided once per row: Markstein's theorem on division through a correctly
// rounded reciprocal makes that the correctly rounded quotient (a zero may change sign,
// which no code sees), so the code is the one the IEEE quotient gives, at three
// operations instead of a full division.
__device__ inline uint32_t code_u8_biased(float x, float s, float y, uint32_t sel, uint32_t acc) {
    const float q0 = __fmul_rn(x, y);
    const float r = fmaf(-q0, s, x);
    const float q = rintf(fmaf(r, y, q0));
    const float c = __builtin_amdgcn_fmed3f(q, -127.0f, 127.0f) + 128.0f;
    return __builtin_amdgcn_cvt_pk_u8_f32(c, sel, acc);
}

// E int8 codes of v with scale s and y = 1 / s correctly rounded; q is aligned to E bytes.
template <int E>
__device__ inline void store_codes_i8(int8_t* q, const float* v, float s, float y) {
    uint32_t w[E / 4];
#pragma unroll
    for (int j = 0; j < E / 4; ++j) {
        uint32_t b = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            b = code_u8_biased(v[4 * j + i], s, y, i, b);
        w[j] = b ^ 0x80808080u;   // code + 128 -> two's complement code
    }
    if constexpr (E == 8)
        *reinterpret_cast<u32x2*>(q) = u32x2{w[0], w[1]};
    else
        *reinterpret_cast<uint32_t*>(q) = w[0];
}

// fp8 (OCP E4M3) codes: the correctly rounded quotient (as code_u8_biased), kept within
// +-448 (it cannot pass it: s = absmax / 448), then v_cvt_pk_fp8_f32, which rounds to
// nearest even into E4M3 (gfx950 converts to the OCP format).
template <int E>
__device__ inline void store_codes_e4m3(uint8_t* q, const float* v, float s, float y) {
    uint32_t w[E / 4];
#pragma unroll
    for (int j = 0; j < E / 4; ++j) {
        float t[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = v[4 * j + i];
            const float q0 = __fmul_rn(x, y);
            const float r = fmaf(-q0, s, x);
            // s > 0, so the quotient has x's sign; the refinement alone would turn
            // x = -0 into +0 (r = +0 + -0), and fp8 keeps the sign of zero.
            t[i] = __builtin_amdgcn_fmed3f(copysignf(fmaf(r, y, q0), x), -448.0f, 448.0f);
        }
        int b = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], 0, false);
        b = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], b, true);
        w[j] = (uint32_t)b;
    }
    if constexpr (E == 16)
        *reinterpret_cast<u32x4*>(q) = u32x4{w[0], w[1], w[2], w[3]};
    else if constexpr (E == 8)
        *reinterpret_cast<u32x2*>(q) = u32x2{w[0], w[1]};
    else
        *reinterpret_cast<uint32_t*>(q) = w[0];
}

}  // namespace ql
