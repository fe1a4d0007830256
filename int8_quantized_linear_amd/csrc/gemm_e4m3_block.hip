// gemm_e4m3_block.hip -- the layer on E4M3 codes with a scale for each block of 128:
//
//   y[m,n] = act(sum_b xs[b,m] ws[n/128,b] sum_{k in block b} xq[m,k] wq[n,k] + bias[n])
//
// The inner sums run on the fp8 matrix cores, from zero for each block; the block's sum is then
// added to the output's fp32 sum with its scales, one multiply-add an output and block.
#include "e4m3_block.h"

namespace ql {
namespace {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));

__device__ inline i32x8 cat(i32x4 lo, i32x4 hi) { return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7); }

struct BlockGemm {
    const uint8_t* xq;
    const float* xs;
    const uint8_t* wq;
    const float* ws;
    const float* bias;
    void* y;
    int rows, N, K, act;   // rows of this launch
    int64_t M;             // rows of xs
};

template <bool F16>
__device__ inline float activated(float v, int act) {
    return act == ACT_GELU ? activation<ACT_GELU, F16>(v) : act == ACT_SILU ? activation<ACT_SILU, F16>(v) : v;
}

// Few rows: bound by the read of W. A workgroup owns 16 output columns and 16 MB rows; its SW waves
// take the blocks of K in turn (neighbouring waves read neighbouring 128 bytes of W's rows). A wave
// copies its blocks (16 rows of W, the rows of X, X's scales) straight into its own ring of S slots
// in LDS, S - 1 blocks ahead, and needs no barrier until its sums are joined with the others'.
// W is the first operand, so a lane's sums belong to one row m (lane & 15) and four columns
// (4 (lane >> 4) + i): one scale of X a lane, one of W for all.
template <int MB, int SW, int S, bool YF16>
__global__ __launch_bounds__(64 * SW) void gemm_block_few_kernel(BlockGemm g) {
    constexpr int W_BYTES = 16 * QB, X_BYTES = MB * 16 * QB, SLOT = W_BYTES + X_BYTES + 256;
    constexpr int COPIES = 2 + 2 * MB + 1;
    __shared__ __attribute__((aligned(1024))) int8_t smem[SW * S * SLOT];
    static_assert(SW * MB * 1024 <= SW * S * SLOT, "the joined sums fit the ring");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16 * MB;
    const int nkb = (g.K + QB - 1) / QB;
    int8_t* ring = smem + wave * S * SLOT;

    const __amdgpu_buffer_rsrc_t rw = buffer_of(g.wq + (int64_t)n0 * g.K, min(g.N - n0, 16) * g.K);
    const __amdgpu_buffer_rsrc_t rx = buffer_of(g.xq + (int64_t)m0 * g.K, min(g.rows - m0, 16 * MB) * g.K);
    const int row = lane >> 3, c0 = copy_chunk128(lane, 0), c1 = copy_chunk128(lane, 1);
    const int far = 0x40000000;
    // Block b of K into a slot; blocks past the end, and the upper half of a last block of 64,
    // come as zeros.
    auto copy = [&](int b, int slot) {
        int8_t* to = ring + slot * SLOT;
        const int left = g.K - b * QB;   // of this block
        const int cut0 = 16 * c0 < left ? 0 : far, cut1 = 16 * c1 < left ? 0 : far;
        const int o0 = row * g.K + 16 * c0 + b * QB, o1 = row * g.K + 16 * c1 + b * QB;
        buffer_to_lds16<2>(rw, o0 | cut0, 0, to);
        buffer_to_lds16<2>(rw, (o1 + 8 * g.K) | cut1, 0, to + 1024);
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            buffer_to_lds16(rx, (o0 + 16 * i * g.K) | cut0, 0, to + W_BYTES + 2048 * i);
            buffer_to_lds16(rx, (o1 + (16 * i + 8) * g.K) | cut1, 0, to + W_BYTES + 2048 * i + 1024);
        }
        global_to_lds4(g.xs + (int64_t)min(b, nkb - 1) * g.M + min(m0 + lane, g.rows - 1), to + W_BYTES + X_BYTES);
    };

    f32x4 acc[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
        acc[i] = f32x4{0, 0, 0, 0};
    // W's scales of this wave's blocks, 64 of them at a time, one a lane
    const float* wrow = g.ws + (int64_t)(n0 / QB) * nkb;
    auto scales_from = [&](int j) { return wrow[min(wave + SW * (j + lane), nkb - 1)]; };
    float wsc = scales_from(0);
#pragma unroll
    for (int s = 0; s < S - 1; ++s)
        copy(wave + SW * s, s);
    asm volatile("" : "+v"(wsc));   // waited for here, behind the first copies, and not in the loop

    const int r = lane & 15, q = lane >> 4;
    const int f0 = r * QB + ((q ^ swizzle128(r)) << 4), f1 = r * QB + (((q + 4) ^ swizzle128(r)) << 4);
    const int nj = (nkb - wave + SW - 1) / SW;
    int slot = 0;
    for (int j = 0; j < nj; ++j) {
        const int8_t* at = ring + slot * SLOT;
        copy(wave + SW * (j + S - 1), slot == 0 ? S - 1 : slot - 1);
        if (j > 0 && (j & 63) == 0) {
            wsc = scales_from(j);
            asm volatile("" : "+v"(wsc));
        }
        __builtin_amdgcn_s_waitcnt(wait_vm((S - 1) * COPIES));
        __builtin_amdgcn_sched_barrier(0);
        const float w1 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wsc), j & 63));
        const i32x8 a = cat(*reinterpret_cast<const i32x4*>(at + f0), *reinterpret_cast<const i32x4*>(at + f1));
        i32x8 x[MB];
        float sc[MB];
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            const int8_t* p = at + W_BYTES + 2048 * i;
            x[i] = cat(*reinterpret_cast<const i32x4*>(p + f0), *reinterpret_cast<const i32x4*>(p + f1));
            sc[i] = *reinterpret_cast<const float*>(at + W_BYTES + X_BYTES + 4 * (16 * i + r));
        }
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            const f32x4 zero{0, 0, 0, 0};
            const f32x4 p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, x[i], zero, 0, 0, 0, 0, 0, 0);
            const float s = sc[i] * w1;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[i][e] = fmaf(s, p[e], acc[i][e]);
        }
        // the slot's reads are done before it is filled again
        __builtin_amdgcn_s_waitcnt(WAIT_LDS);
        __builtin_amdgcn_sched_barrier(0);
        slot = slot + 1 == S ? 0 : slot + 1;
    }
    __builtin_amdgcn_s_waitcnt(wait_vm(0));
    __syncthreads();
    f32x4* red = reinterpret_cast<f32x4*>(smem);
#pragma unroll
    for (int i = 0; i < MB; ++i)
        red[(wave * MB + i) * 64 + lane] = acc[i];
    __syncthreads();
    using OutT = typename std::conditional<YF16, _Float16, float>::type;
    using Out4 = OutT __attribute__((ext_vector_type(4)));
    for (int i = wave; i < MB; i += SW) {
        f32x4 t = red[i * 64 + lane];
#pragma unroll
        for (int w = 1; w < SW; ++w)
            t += red[(w * MB + i) * 64 + lane];
        const int m = m0 + 16 * i + r, n = n0 + 4 * q;
        if (m >= g.rows)
            continue;
        Out4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[e] = (OutT)activated<YF16>(t[e] + (g.bias != nullptr && n + e < g.N ? g.bias[n + e] : 0.0f), g.act);
        OutT* to = reinterpret_cast<OutT*>(g.y) + (int64_t)m * g.N + n;
        if ((g.N & 3) == 0) {
            if (n < g.N)
                *reinterpret_cast<Out4*>(to) = o;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < g.N)
                    to[e] = o[e];
        }
    }
}

template <bool YF16>
void launch_few(const BlockGemm& g, hipStream_t stream) {
    const uint32_t nx = (uint32_t)((g.N + 15) / 16);
    // rows in launches whose grid stays within 65535 in y
    auto go = [&](auto kernel, int sw, int rows) {
        const int64_t most = (int64_t)rows * 65535;
        for (int64_t m = 0; m < g.M; m += most) {
            BlockGemm p = g;
            p.xq += m * g.K;
            p.xs += m;
            p.y = reinterpret_cast<int8_t*>(g.y) + m * g.N * (YF16 ? 2 : 4);
            p.rows = (int)(g.M - m < most ? g.M - m : most);
            kernel<<<dim3(nx, (uint32_t)((p.rows + rows - 1) / rows)), dim3(64 * sw), 0, stream>>>(p);
        }
    };
    if (g.M <= 16)
        go(gemm_block_few_kernel<1, 8, 4, YF16>, 8, 16);
    else
        go(gemm_block_few_kernel<2, 8, 3, YF16>, 8, 32);
}

}  // namespace

ql_status launch_gemm_e4m3_block(const uint8_t* xq, const float* x_scale, const uint8_t* wq, const float* w_scale,
                                 const float* bias, int act, void* y, bool y_f16, int64_t M, int64_t N, int64_t K,
                                 hipStream_t stream) {
    const BlockGemm g{xq, x_scale, wq, w_scale, bias, y, 0, (int)N, (int)K, act, M};
    if (y_f16)
        launch_few<true>(g, stream);
    else
        launch_few<false>(g, stream);
    return launch_status();
}

}  // namespace ql
