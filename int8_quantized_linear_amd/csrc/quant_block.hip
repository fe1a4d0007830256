// quant_block.hip -- E4M3 codes with a scale for each block of 128: activations (one row's 128
// values a block) and weights (128 x 128 a block).
//
//   a = max |v| over the block,  s = max(a, 1e-10) / 448,  code = e4m3(clamp(v / s, -448, 448))
//
// Each value is read once and its code written once; both are bound by memory. 2048 x 11008 values of fp16
// take 15 us, 4.5 TB/s, of fp32 21 us, 5.5 TB/s; 11008 x 4096 weights 49 us from cold memory, 4.6 TB/s (a
// large copy reaches 4.95).
#include "e4m3_block.h"
#include "quant_codes.h"

namespace ql {
namespace {

constexpr int NT = 256;

template <int CTRL>
__device__ inline float max_dpp(float v) {
    return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true)));
}

// Maximum over L = 8 or 16 neighbouring lanes, in every one of them.
template <int L>
__device__ inline float max_of(float v) {
    v = max_dpp<0xB1>(v);    // within pairs, fours,
    v = max_dpp<0x4E>(v);
    v = max_dpp<0x141>(v);   // eights (mirrored)
    return L == 16 ? max_dpp<0x140>(v) : v;
}

template <bool F16, int V>
__device__ inline void load_values(float (&v)[V], const void* p, int64_t i) {
    if constexpr (F16) {
        const f16x8* h = reinterpret_cast<const f16x8*>(reinterpret_cast<const _Float16*>(p) + i);
#pragma unroll
        for (int j = 0; j < V; ++j)
            v[j] = (float)h[j / 8][j % 8];
    } else {
        const f32x4* f = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(p) + i);
#pragma unroll
        for (int j = 0; j < V; ++j)
            v[j] = f[j / 4][j % 4];
    }
}

template <int V>
__device__ inline float absmax(const float (&v)[V]) {
    float a = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j)
        a = fmaxf(a, fabsf(v[j]));
    return a;
}

// A workgroup takes 16 rows and RB blocks of K, so that the 16 scales of a block leave as one 64-byte
// piece; 16 lanes a row. A lane has 32 bytes of x at a time: 16 values of fp16 (with 8 values, whose codes
// leave 8 bytes a lane, 2048 x 11008 took 16.7 us, now 15.1), 8 of fp32.
constexpr int RB = 4;
template <bool F16>
__global__ __launch_bounds__(NT) void quant_rows_block_kernel(const void* __restrict__ x, int64_t M, int64_t K,
                                                              int nkb, int64_t first, uint8_t* __restrict__ xq,
                                                              float* __restrict__ xs) {
    constexpr int V = F16 ? 16 : 8, L = QB / V, STEP = 16 / L;   // lanes of a block, blocks at a time
    const int kgroups = (nkb + RB - 1) / RB;
    const int64_t wg = first + blockIdx.x;
    const int64_t m = wg / kgroups * 16 + threadIdx.x / 16;
    const int b0 = (int)(wg % kgroups) * RB + threadIdx.x % 16 / L, l = threadIdx.x % L;
    if (m >= M)
        return;
    float v[RB / STEP][V];
#pragma unroll
    for (int i = 0; i < RB / STEP; ++i) {
        const int64_t k = (int64_t)(b0 + i * STEP) * QB + V * l;
        if (k < K) {
            load_values<F16>(v[i], x, m * K + k);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                v[i][j] = 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < RB / STEP; ++i) {
        const int b = b0 + i * STEP;
        const int64_t k = (int64_t)b * QB + V * l;
        const float s = fmaxf(max_of<L>(absmax(v[i])), 1e-10f) / 448.0f;
        if (k < K)
            store_codes_e4m3<V>(xq + m * K + k, v[i], s, 1.0f / s);
        if (l == 0 && b < nkb)
            xs[b * M + m] = s;
    }
}

// A workgroup takes one block of 128 x 128: 16 lanes a row, eight rows a thread.
__global__ __launch_bounds__(NT) void quant_weight_block_kernel(const float* __restrict__ w, int64_t N, int64_t K,
                                                                int64_t nnb, int64_t nkb, int64_t first,
                                                                uint8_t* __restrict__ wq, float* __restrict__ ws) {
    __shared__ float red[NT / WAVE];
    const int64_t wg = first + blockIdx.x;
    const int64_t kb = wg % nkb, nb = wg / nkb % nnb, e = wg / nkb / nnb;
    const int64_t k = kb * QB + 8 * (threadIdx.x % 16), n0 = nb * QB + threadIdx.x / 16;
    w += e * N * K;
    wq += e * N * K;
    float v[8][8], a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (n0 + 16 * i < N && k < K) {
            load_values<false>(v[i], w, (n0 + 16 * i) * K + k);
            a = fmaxf(a, absmax(v[i]));
        }
    }
#pragma unroll
    for (int o = WAVE / 2; o > 0; o >>= 1)
        a = fmaxf(a, __shfl_xor(a, o, WAVE));
    if (threadIdx.x % WAVE == 0)
        red[threadIdx.x / WAVE] = a;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / WAVE; ++i)
        a = fmaxf(a, red[i]);
    const float s = fmaxf(a, 1e-10f) / 448.0f, y = 1.0f / s;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (n0 + 16 * i < N && k < K)
            store_codes_e4m3<8>(wq + (n0 + 16 * i) * K + k, v[i], s, y);
    if (threadIdx.x == 0)
        ws[wg] = s;
}

constexpr int64_t MOST = (int64_t)1 << 23;   // workgroups of a launch: its threads stay below 2^32

}  // namespace

ql_status launch_quant_rows_block_e4m3(const void* x, bool x_f16, int64_t M, int64_t K, uint8_t* xq, float* x_scale,
                                       hipStream_t stream) {
    const int nkb = (int)e4m3_blocks(K);
    const int64_t wgs = (M + 15) / 16 * ((nkb + RB - 1) / RB);
    for (int64_t f = 0; f < wgs; f += MOST) {
        const dim3 grid((uint32_t)(wgs - f < MOST ? wgs - f : MOST));
        if (x_f16)
            quant_rows_block_kernel<true><<<grid, dim3(NT), 0, stream>>>(x, M, K, nkb, f, xq, x_scale);
        else
            quant_rows_block_kernel<false><<<grid, dim3(NT), 0, stream>>>(x, M, K, nkb, f, xq, x_scale);
    }
    return launch_status();
}

ql_status launch_quant_weight_block_e4m3(const float* w, int64_t E, int64_t N, int64_t K, uint8_t* wq, float* w_scale,
                                         hipStream_t stream) {
    const int64_t nnb = e4m3_blocks(N), nkb = e4m3_blocks(K), wgs = E * nnb * nkb;
    for (int64_t f = 0; f < wgs; f += MOST)
        quant_weight_block_kernel<<<dim3((uint32_t)(wgs - f < MOST ? wgs - f : MOST)), dim3(NT), 0, stream>>>(
            w, N, K, nnb, nkb, f, wq, w_scale);
    return launch_status();
}

}  // namespace ql
