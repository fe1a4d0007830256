// norm.hip -- root-mean-square norm with the residual's addition, written as 8-bit codes with
// one scale per row: the activations of the next W8A8 or fp8 layer.
//
//   h = residual + x;  y = h / sqrt(mean(h^2) + eps) * gamma;  y ~ scale * code
//
// The row's factor r = 1 / sqrt(mean(h^2) + eps) is common to every y of the row, so it cancels
// in y / (max|y| / 127): the codes are those of t = h * gamma with s = max|t| / 127, and r
// enters the row's scale only, scale = s * r. The codes therefore need one rounding each for h,
// t, s and t / s, whatever the order in which the squares are summed, and the kernel needs one
// reduction (the maximum and the sum of squares together) and one pass over the row. (The squares
// and their sum are fp32.)
//
// Bound by memory: every value is read and written once. 2048 rows of 11008 (fp16 x and residual,
// in and out, int8 codes: 158 MB) take 36 us, 4.4 TB/s, where a large copy reaches 5.0; 2048 of
// 4096 15.2 us from cold memory, 11 us where the caches hold part of it; one row of 4096 3.0 us,
// a launch and the row's one chain of load, reduction and store.
#include "quant_codes.h"

namespace ql {
namespace {

constexpr int NT = 256;   // threads per workgroup, one workgroup per row

// 8 values from fp16 or fp32 memory, as fp32.
template <bool F16>
__device__ inline void load8(float (&v)[8], const void* p, int64_t i) {
    if constexpr (F16) {
        const f16x8 h = *reinterpret_cast<const f16x8*>(reinterpret_cast<const _Float16*>(p) + i);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = (float)h[j];
    } else {
        const f32x4* f = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(p) + i);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = f[j / 4][j % 4];
    }
}

enum { R_NONE = 0, R_F16 = 1, R_F32 = 2 };

// One workgroup per row of K = 8 * nch values. NC > 0: rows of up to NT * NC chunks of 8 stay in
// registers. Short rows get a smaller NC, which leaves the CUs room for more of them: 8192 rows of
// 1024 take 14.7 us with NC = 1 and 22.3 with 8, 2048 of 4096 15.2 with 2 and 15.6 with 8. (4 for
// rows up to 8192 lost: 2048 of 8192 29.5, with 8 27.0. So did loading all chunks before the first
// store, which doubles the registers: 2048 of 16384 52.5, chunk by chunk 47.5.) NC == 0: longer rows
// are read twice (the statistics, then h and the codes): 2048 rows of 16384 take 64 us so. A chunk of h
// is written by the thread that has read it, and in the second pass only, so that res_out may be
// the residual or x itself.
template <bool XF16, int RES, bool E4M3, int NC>
__global__ __launch_bounds__(NT) void rms_norm_quant_kernel(const void* x, const void* residual,
                                                            const float* __restrict__ gamma, float eps, int64_t K,
                                                            void* res_out, int8_t* __restrict__ q,
                                                            float* __restrict__ scale) {
    constexpr float QMAX = E4M3 ? 448.0f : 127.0f;
    __shared__ float red[2 * (NT / WAVE)];
    const int64_t row = blockIdx.x, base = row * K;
    const int nch = (int)(K / 8);
    float amax = 0.0f, sum = 0.0f;

    // h of one chunk, and t = h * gamma in its place; the statistics take both.
    auto chunk = [&](int ch, float (&t)[8], bool write) {
        float h[8], g[8];
        load8<XF16>(h, x, base + (int64_t)ch * 8);
        load8<false>(g, gamma, (int64_t)ch * 8);
        if constexpr (RES != R_NONE) {
            float r[8];
            load8<RES == R_F16>(r, residual, base + (int64_t)ch * 8);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                h[j] += r[j];
            if (write)
                store8<RES == R_F16>(res_out, base + (int64_t)ch * 8, h);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            sum = fmaf(h[j], h[j], sum);
            t[j] = h[j] * g[j];
            amax = fmaxf(amax, fabsf(t[j]));
        }
    };
    auto codes = [&](int ch, const float (&t)[8], float s, float y) {
        if constexpr (E4M3)
            store_codes_e4m3<8>(reinterpret_cast<uint8_t*>(q) + base + (int64_t)ch * 8, t, s, y);
        else
            store_codes_i8<8>(q + base + (int64_t)ch * 8, t, s, y);
    };
    // Both statistics over the workgroup; s and the row's scale.
    auto finish = [&]() {
#pragma unroll
        for (int o = WAVE / 2; o > 0; o >>= 1) {
            amax = fmaxf(amax, __shfl_xor(amax, o, WAVE));
            sum += __shfl_xor(sum, o, WAVE);
        }
        const int w = threadIdx.x / WAVE;
        if ((threadIdx.x & (WAVE - 1)) == 0) {
            red[2 * w] = amax;
            red[2 * w + 1] = sum;
        }
        __syncthreads();
        amax = red[0];
        sum = red[1];
#pragma unroll
        for (int i = 1; i < NT / WAVE; ++i) {
            amax = fmaxf(amax, red[2 * i]);
            sum += red[2 * i + 1];
        }
        const float s = fmaxf(amax, 1e-10f) / QMAX;
        if (threadIdx.x == 0)
            scale[row] = s * (1.0f / sqrtf(sum / (float)K + eps));
        return s;
    };

    if constexpr (NC > 0) {
        float t[NC][8];
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if ((int)threadIdx.x + i * NT < nch)
                chunk(threadIdx.x + i * NT, t[i], true);
        const float s = finish();
        const float y = 1.0f / s;
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if ((int)threadIdx.x + i * NT < nch)
                codes(threadIdx.x + i * NT, t[i], s, y);
    } else {
        float t[8];
        for (int ch = threadIdx.x; ch < nch; ch += NT)
            chunk(ch, t, false);
        const float s = finish();
        const float y = 1.0f / s;
        for (int ch = threadIdx.x; ch < nch; ch += NT) {
            chunk(ch, t, true);
            codes(ch, t, s, y);
        }
    }
}

template <bool XF16, int RES, bool E4M3>
void launch_typed(const void* x, const void* residual, const float* gamma, float eps, int64_t M, int64_t K,
                  void* res_out, int8_t* q, float* scale, hipStream_t stream) {
    const int64_t nch = K / 8;
    constexpr int64_t MOST = (int64_t)1 << 22;   // rows of a launch: its threads stay below 2^32
    auto go = [&](auto kernel) {
        auto at = [&](auto* p, int64_t i) { return p ? reinterpret_cast<decltype(p)>((uintptr_t)p + i) : nullptr; };
        for (int64_t m = 0; m < M; m += MOST)
            kernel<<<dim3((uint32_t)(M - m < MOST ? M - m : MOST)), dim3(NT), 0, stream>>>(
                at(x, m * K * (XF16 ? 2 : 4)), at(residual, m * K * (RES == R_F16 ? 2 : 4)), gamma, eps, K,
                at(res_out, m * K * (RES == R_F16 ? 2 : 4)), q + m * K, scale + m);
    };
    if (nch <= NT)
        go(rms_norm_quant_kernel<XF16, RES, E4M3, 1>);
    else if (nch <= 2 * NT)
        go(rms_norm_quant_kernel<XF16, RES, E4M3, 2>);
    else if (nch <= 8 * NT)
        go(rms_norm_quant_kernel<XF16, RES, E4M3, 8>);
    else
        go(rms_norm_quant_kernel<XF16, RES, E4M3, 0>);
}

}  // namespace

ql_status launch_rms_norm_quant(const void* x, bool x_f16, const void* residual, bool res_f16, const float* gamma,
                                float eps, int64_t M, int64_t K, void* res_out, void* q, bool e4m3, float* scale,
                                hipStream_t stream) {
    auto by_codes = [&](auto xt, auto rt) {
        constexpr bool XF16 = decltype(xt)::value;
        constexpr int RES = decltype(rt)::value;
        int8_t* codes = reinterpret_cast<int8_t*>(q);
        if (e4m3)
            launch_typed<XF16, RES, true>(x, residual, gamma, eps, M, K, res_out, codes, scale, stream);
        else
            launch_typed<XF16, RES, false>(x, residual, gamma, eps, M, K, res_out, codes, scale, stream);
    };
    auto by_residual = [&](auto xt) {
        if (!residual)
            by_codes(xt, std::integral_constant<int, R_NONE>{});
        else if (res_f16)
            by_codes(xt, std::integral_constant<int, R_F16>{});
        else
            by_codes(xt, std::integral_constant<int, R_F32>{});
    };
    if (x_f16)
        by_residual(std::true_type{});
    else
        by_residual(std::false_type{});
    return launch_status();
}

}  // namespace ql
