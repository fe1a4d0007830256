// kv4.hip -- rows of K and V quantized into a paged 4-bit cache, and rows read back from it.
//
// Per token, head and group of G values, from the group's minimum and maximum:
//   low = fp16(min), scale = max(fp16((max - low) / 15), 2^-24),
//   code = clamp(round((x - low) / scale), 0, 15),  x ~ scale * code + low
// The codes are taken with the stored fp16 scale and low, as the int4 weights' are, so a value
// read back is the nearest one that the stored pair can give. Rounding is half to even, the
// quotient the correctly rounded one.
#include "kv4.h"

namespace ql {
namespace {

constexpr int KT = 256;   // threads per workgroup

template <bool F16>
__device__ inline float load1(const void* p, int64_t i) {
    if constexpr (F16)
        return (float)reinterpret_cast<const _Float16*>(p)[i];
    else
        return reinterpret_cast<const float*>(p)[i];
}

// fp16 of a float, kept within fp16's finite range.
__device__ inline _Float16 to_f16_sat(float v) {
    return (_Float16)__builtin_amdgcn_fmed3f(v, -65504.0f, 65504.0f);
}

__device__ inline void group_params(float lo, float hi, _Float16& s16, _Float16& lo16) {
    lo16 = to_f16_sat(lo);
    s16 = to_f16_sat(fmaxf((hi - (float)lo16) / 15.0f, 0.0f));
    const _Float16 least = (_Float16)5.9604644775390625e-08f;   // 2^-24
    s16 = s16 > least ? s16 : least;
}

__device__ inline uint32_t code4(float x, float s, float lo) {
    return (uint32_t)__builtin_amdgcn_fmed3f(rintf((x - lo) / s), 0.0f, 15.0f);
}

// One thread per (row, head, group): min and max, then the codes of its G values.
template <int D, int G, bool F16>
__global__ __launch_bounds__(KT) void kv4_append_kernel(const void* __restrict__ k, const void* __restrict__ v,
                                                        int64_t k_stride, int64_t v_stride, int rows, Kv4Cache c,
                                                        Kv4Batch b) {
    using L = Kv4Layout<D, G>;
    const int P = 1 << c.page_log2;
    const int64_t id = (int64_t)blockIdx.x * KT + threadIdx.x;
    const int g = (int)(id % L::NG);
    const int64_t rh = id / L::NG;
    const int head = (int)(rh % c.heads);
    if (rh / c.heads >= rows)
        return;
    const int row = (int)(rh / c.heads);
    const int seq = kv4_seq(b, row);
    const int len = kv4_len(b, c, seq), pos = kv4_pos(b, seq, len, row);
    if (pos < 0 || pos >= len)
        return;
    uint8_t* page = kv4_page(b, c, seq, pos, head);
    const int slot = pos & (P - 1);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const void* x = which ? v : k;
        const int64_t base = row * (which ? v_stride : k_stride) + (int64_t)head * D + g * G;
        float lo = INFINITY, hi = -INFINITY;
        for (int i = 0; i < G; ++i) {
            const float t = load1<F16>(x, base + i);
            lo = fminf(lo, t);
            hi = fmaxf(hi, t);
        }
        _Float16 s16, lo16;
        group_params(lo, hi, s16, lo16);
        const float s = (float)s16, l = (float)lo16;
        reinterpret_cast<_Float16*>(page + (which ? L::v_scale(P, g) : L::k_scale(P, g)))[slot] = s16;
        reinterpret_cast<_Float16*>(page + (which ? L::v_low(P, g) : L::k_low(P, g)))[slot] = lo16;
        if (which == 0) {
            uint32_t* to = reinterpret_cast<uint32_t*>(page + L::k_codes(slot));
            for (int w = 0; w < G / 8; ++w) {
                const int d = g * G + 8 * w;
                uint32_t word = 0;
                for (int e = 0; e < 8; ++e)
                    word |= code4(load1<F16>(x, base + 8 * w + e), s, l) << (16 * (e & 1) + 4 * (e >> 1));
                to[((d % 32) / 8) * (D / 32) + d / 32] = word;
            }
        } else {
            // quads with their low half in this group; a group of 32 holds half of each quad
            // of its 64-wide chunk, one byte (d, d + 1)
            uint8_t* to = page + L::v_codes(P, slot / 8);
            for (int w = 0; w < G / 2; ++w) {
                const int d = g * G + 2 * w;
                const uint32_t byte = code4(load1<F16>(x, base + 2 * w), s, l) |
                                      code4(load1<F16>(x, base + 2 * w + 1), s, l) << 4;
                const int quad = (d / 64) * 16 + (d % 32) / 2;
                to[quad * 16 + (slot % 8) * 2 + (d % 64) / 32] = (uint8_t)byte;
            }
        }
    }
}

// One thread per (row, head, 8 values) of K and of V.
template <int D, int G, bool F16>
__global__ __launch_bounds__(KT) void kv4_read_kernel(Kv4Cache c, Kv4Batch b, int rows, void* __restrict__ k_out,
                                                      void* __restrict__ v_out) {
    using L = Kv4Layout<D, G>;
    const int P = 1 << c.page_log2;
    const int64_t id = (int64_t)blockIdx.x * KT + threadIdx.x;
    const int d0 = (int)(id % (D / 8)) * 8;
    const int64_t rh = id / (D / 8);
    const int head = (int)(rh % c.heads);
    if (rh / c.heads >= rows)
        return;
    const int row = (int)(rh / c.heads);
    const int seq = kv4_seq(b, row);
    const int len = kv4_len(b, c, seq), pos = kv4_pos(b, seq, len, row);
    float kx[8] = {}, vx[8] = {};
    if (pos >= 0 && pos < len) {
        const uint8_t* page = kv4_page(b, c, seq, pos, head);
        const int slot = pos & (P - 1), g = d0 / G;
        const uint32_t kw = reinterpret_cast<const uint32_t*>(page + L::k_codes(slot))[((d0 % 32) / 8) * (D / 32) + d0 / 32];
        const float ks = (float)reinterpret_cast<const _Float16*>(page + L::k_scale(P, g))[slot];
        const float kl = (float)reinterpret_cast<const _Float16*>(page + L::k_low(P, g))[slot];
        const float vs = (float)reinterpret_cast<const _Float16*>(page + L::v_scale(P, g))[slot];
        const float vl = (float)reinterpret_cast<const _Float16*>(page + L::v_low(P, g))[slot];
        const uint8_t* vb = page + L::v_codes(P, slot / 8);
        for (int e = 0; e < 8; ++e) {
            const int d = d0 + e, quad = (d / 64) * 16 + (d % 32) / 2;
            kx[e] = fmaf(ks, (float)((kw >> (16 * (e & 1) + 4 * (e >> 1))) & 15), kl);
            vx[e] = fmaf(vs, (float)((vb[quad * 16 + (slot % 8) * 2 + (d % 64) / 32] >> (4 * (d & 1))) & 15), vl);
        }
    }
    const int64_t at = rh * D + d0;
    for (int e = 0; e < 8; ++e)
        if constexpr (F16) {
            reinterpret_cast<_Float16*>(k_out)[at + e] = (_Float16)kx[e];
            reinterpret_cast<_Float16*>(v_out)[at + e] = (_Float16)vx[e];
        } else {
            reinterpret_cast<float*>(k_out)[at + e] = kx[e];
            reinterpret_cast<float*>(v_out)[at + e] = vx[e];
        }
}

}  // namespace

ql_status launch_kv4_append(const void* k, const void* v, bool f16, int64_t k_stride, int64_t v_stride, int64_t rows,
                            const Kv4Cache& c, int D, int G, const Kv4Batch& b, hipStream_t stream) {
    return kv4_dispatch(D, G, [&](auto d, auto g) {
        constexpr int DD = decltype(d)::value, GG = decltype(g)::value;
        const int64_t n = rows * c.heads * (DD / GG);
        const dim3 grid((uint32_t)((n + KT - 1) / KT));
        if (f16)
            kv4_append_kernel<DD, GG, true><<<grid, KT, 0, stream>>>(k, v, k_stride, v_stride, (int)rows, c, b);
        else
            kv4_append_kernel<DD, GG, false><<<grid, KT, 0, stream>>>(k, v, k_stride, v_stride, (int)rows, c, b);
        return launch_status();
    });
}

ql_status launch_kv4_read(const Kv4Cache& c, int D, int G, const Kv4Batch& b, int64_t rows, void* k_out, void* v_out,
                          bool f16, hipStream_t stream) {
    return kv4_dispatch(D, G, [&](auto d, auto g) {
        constexpr int DD = decltype(d)::value, GG = decltype(g)::value;
        const int64_t n = rows * c.heads * (DD / 8);
        const dim3 grid((uint32_t)((n + KT - 1) / KT));
        if (f16)
            kv4_read_kernel<DD, GG, true><<<grid, KT, 0, stream>>>(c, b, (int)rows, k_out, v_out);
        else
            kv4_read_kernel<DD, GG, false><<<grid, KT, 0, stream>>>(c, b, (int)rows, k_out, v_out);
        return launch_status();
    });
}

}  // namespace ql
