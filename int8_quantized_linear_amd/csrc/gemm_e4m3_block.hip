// gemm_e4m3_block.hip -- the layer on E4M3 codes with a scale for each block of 128:
//
//   y[m,n] = act(sum_b xs[b,m] ws[n/128,b] sum_{k in block b} xq[m,k] wq[n,k] + bias[n])
//
// The inner sums run on the fp8 matrix cores, from zero for each block; the block's sum is then
// added to the output's fp32 sum with its scales, one multiply-add an output and block.
//
// The fp8 matrix cores cut each product to a multiple of 2^(E - 13), E the largest exponent sum in its group of 8
// (tests/test_gpu_fp8.py shows it): fewer bits than fp32, and a choice. fp32 outputs are 1.5e-5 to 3e-5 of their
// norm off; fp16 outputs 2.10e-4 instead of the 2.08e-4 of their own rounding, a tenth of them by one step. The fp16 matrix
// cores take the codes exactly (fp32 outputs 7e-8 to 1.1e-7 off), at half the rate and a conversion of every operand.
// us with fp8 / fp16 matrix cores: 1 x 11008 x 4096 12.1 / 12.3, 32 x 4096 x 11008 14.7 / 15.0, 64 x 4096 x 4096 7.3 / 8.0,
// 128 x 4096 x 4096 10.1 / 11.4, 512 x 4096 x 4096 22.1 / 28.8, 1024 x 4096 x 4096 30 / 36 and 2048 x 11008 x 4096 106 / 202
// (fp32 outputs; the best tiles of each). All kernels keep to one arithmetic, which gemm_e4m3_per_channel has too, so
// that the precision does not depend on the number of rows.
//
// Few rows are bound by the read of W (1 x 11008 x 4096: 8.9 us, 5.1 TB/s). Between, by what a CU's copies bring and
// how many CUs have a tile (333 x 4001 x 2112: 12.6 us). Many rows, 2048 x 11008 x 4096: 92 us, 2010 TFLOP/s, where a
// library product of 8192 x 8192 x 8192 on such codes without block scales reaches 2910. Its 464 tiles are 1.81 of two
// rounds, at the library's rate 70 us; the matrix cores are busy for 56% of a busy CU's cycles, at 2.1 GHz. us with work left
// out in copies made for timing: matrix instructions, barriers and outputs alone 67, with the multiply-adds for the
// scales 72, all but the reads of LDS 81, all but the copies 76, all but the multiply-adds 83. So the copies and reads beside
// the matrix instructions cost more than the multiply-adds.
#include "e4m3_block.h"
#include "gemm_w8a8_tile.h"

namespace ql {
namespace {

struct BlockGemm {
    const uint8_t* xq;
    const float* xs;
    const uint8_t* wq;
    const float* ws;
    const float* bias;
    void* y;
    int rows, N, K, act;
    int64_t M;   // rows too, for products past 2^31
};

template <bool F16>
__device__ inline float activated(float v, int act) {
    return act == ACT_GELU ? activation<ACT_GELU, F16>(v) : act == ACT_SILU ? activation<ACT_SILU, F16>(v) : v;
}

// Few rows: bound by the read of W. A workgroup owns 16 NB output columns and 16 MB rows; its SW waves
// take the blocks of K in turn (neighbouring waves read neighbouring 128 bytes of W's rows). A wave
// copies its blocks (16 NB rows of W, the rows of X, X's scales) straight into its own ring of S slots
// in LDS, S - 1 blocks ahead, and needs no barrier until its sums are joined with the others'.
// W is the first operand, so a lane's sums belong to one row m (lane & 15) and four columns
// (4 (lane >> 4) + i): one scale of X a lane, one of W for all.
// ONCE: one group of rows, so that W is read once and loaded non-temporally, also where K is no multiple of 128
// and a line holds codes of two blocks; several groups read W again, and keep it. us from cold memory,
// non-temporal / kept: 1 x 11008 x 4096 12.1 / 13.0, 1 x 11008 x 4160 12.4 / 12.9, 32 x 11008 x 2112 10.7 / 11.0,
// 1 x 4096 x 2112 4.5 / 4.5 (one group); 64 x 4096 x 4096 8.7 / 7.3, 64 x 4096 x 2112 8.5 / 6.7, 300 x 70 x 2176
// 5.9 / 4.2, 150 x 2000 x 8192 19.6 / 17.4, 600 x 700 x 1024 6.9 / 6.2 (2 to 19 groups).
template <int NB, int MB, int SW, int S, bool YF16, bool ONCE>
__global__ __launch_bounds__(64 * SW) void gemm_block_few_kernel(BlockGemm g) {
    constexpr int W_BYTES = NB * 16 * QB, X_BYTES = MB * 16 * QB, SLOT = W_BYTES + X_BYTES + 256;
    constexpr int COPIES = 2 * NB + 2 * MB + 1;
    __shared__ __attribute__((aligned(1024))) int8_t smem[SW * S * SLOT];
    static_assert(SW * NB * MB * 1024 <= SW * S * SLOT, "the joined sums fit the ring");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16 * NB, m0 = blockIdx.y * 16 * MB;
    const int nkb = (g.K + QB - 1) / QB;
    int8_t* ring = smem + wave * S * SLOT;

    const __amdgpu_buffer_rsrc_t rw = buffer_of(g.wq + (int64_t)n0 * g.K, min(g.N - n0, 16 * NB) * g.K);
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
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            buffer_to_lds16<ONCE ? 2 : 0>(rw, (o0 + 16 * i * g.K) | cut0, 0, to + 2048 * i);
            buffer_to_lds16<ONCE ? 2 : 0>(rw, (o1 + (16 * i + 8) * g.K) | cut1, 0, to + 2048 * i + 1024);
        }
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            buffer_to_lds16(rx, (o0 + 16 * i * g.K) | cut0, 0, to + W_BYTES + 2048 * i);
            buffer_to_lds16(rx, (o1 + (16 * i + 8) * g.K) | cut1, 0, to + W_BYTES + 2048 * i + 1024);
        }
        global_to_lds4(g.xs + (int64_t)min(b, nkb - 1) * g.M + min(m0 + lane, g.rows - 1), to + W_BYTES + X_BYTES);
    };

    f32x4 acc[NB][MB];
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < MB; ++i)
            acc[j][i] = f32x4{0, 0, 0, 0};
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
        i32x8 a[NB], x[MB];
#pragma unroll
        for (int i = 0; i < NB; ++i)
            a[i] = cat8(*reinterpret_cast<const i32x4*>(at + 2048 * i + f0), *reinterpret_cast<const i32x4*>(at + 2048 * i + f1));
        float sc[MB];
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            const int8_t* p = at + W_BYTES + 2048 * i;
            x[i] = cat8(*reinterpret_cast<const i32x4*>(p + f0), *reinterpret_cast<const i32x4*>(p + f1));
            sc[i] = *reinterpret_cast<const float*>(at + W_BYTES + X_BYTES + 4 * (16 * i + r));
        }
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            const float s = sc[i] * w1;
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const f32x4 zero{0, 0, 0, 0};
                const f32x4 p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[n], x[i], zero, 0, 0, 0, 0, 0, 0);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[n][i][e] = fmaf(s, p[e], acc[n][i][e]);
            }
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
    for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < MB; ++i)
            red[(wave * NB * MB + j * MB + i) * 64 + lane] = acc[j][i];
    __syncthreads();
    using OutT = typename std::conditional<YF16, _Float16, float>::type;
    using Out4 = OutT __attribute__((ext_vector_type(4)));
    for (int b = wave; b < NB * MB; b += SW) {
        f32x4 t = red[b * 64 + lane];
#pragma unroll
        for (int w = 1; w < SW; ++w)
            t += red[(w * NB * MB + b) * 64 + lane];
        const int m = m0 + 16 * (b % MB) + r, n = n0 + 16 * (b / MB) + 4 * q;
        if (m >= g.rows)
            continue;
        Out4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[e] = (OutT)activated<YF16>(t[e] + (g.bias != nullptr && n + e < g.N ? g.bias[n + e] : 0.0f), g.act);
        OutT* to = reinterpret_cast<OutT*>(g.y) + (int64_t)m * g.N + n;
        if (n + 4 <= g.N) {
            typedef Out4 __attribute__((aligned(2))) Piece;   // rows start at any element
            *reinterpret_cast<Piece*>(to) = o;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < g.N)
                    to[e] = o[e];
        }
    }
}

// Rows between: tiles of 64 x 64 on four waves, 32 x 32 each, up to three workgroups a CU. A stage is a block
// of K, copied straight into a ring of S stages that the waves share; one barrier a stage shows that all
// copies of it have landed and that all waves have read the one before, whose place is then filled. X's
// scales come into registers, one a lane. Outputs leave through LDS in whole 16-byte pieces of a row.
//
// Bound by the copies into LDS. us from warm memory, with work left out in copies made for timing:
//                              whole        no products  no LDS reads  neither      no reads, L1  no copies
//   512 x 4096 x 4096 / 8192   18.8 / 32.7  16.2 / 28.2  17.4 / 29.3   15.6 / 27.8  16.1 / 26.4   12.7 / 19.4
// (L1: every stage copies the first block.) 32 stages of two workgroups a CU are 13.9 us, 75 GB/s a CU; the copies
// alone take 12.1 of them (87 GB/s), and 4.9 us are launch, first loads and outputs. Lines in L1 bring no more than 102
// GB/s a CU, so neither L2 nor memory is the limit. The LDS is active for 24% of the cycles (bank conflicts 2% of those), the
// matrix cores for 23%. So what counts is how many bytes the
// busiest CU copies: us for 64 x 64, 64 x 128, 128 x 64 of this kernel and 128 x 128 below
//   333 x 4001 x 2112  12.6 14.6 13.8 14.8      512 x 4096 x 4096   18.8 22.0 21.0 20.3
//   256 x 4096 x 4096  14.6 21.0 20.1 19.7      1024 x 4096 x 4096  33.7 30.7 30.5 24.3
// (a fourth stage changed nothing).
// Reading the next stage's operands from LDS under this one's products changed nothing.
template <bool YF16>
__global__ __launch_bounds__(256) void gemm_block_mid_kernel(BlockGemm g) {
    constexpr int S = 3, TILE = 64, X_BYTES = TILE * QB, STAGE = 2 * TILE * QB;
    constexpr int NC = 2 * TILE / 32, COPIES = NC + 1;   // of a wave
    using OutT = typename std::conditional<YF16, _Float16, float>::type;
    using Out4 = OutT __attribute__((ext_vector_type(4)));
    constexpr int PITCH = TILE * (int)sizeof(OutT) + 16;
    static_assert(TILE * PITCH <= S * STAGE, "the outputs fit the ring");
    __shared__ __attribute__((aligned(1024))) int8_t smem[S * STAGE];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave & 1, wn = wave >> 1, lr = lane & 31, lh = lane >> 5;
    // tiles of the same columns of W one after another on one XCD
    const int tiles_m = (g.rows + TILE - 1) / TILE, tile = xcd_remap(blockIdx.x, gridDim.x);
    const int m0 = tile % tiles_m * TILE, n0 = tile / tiles_m * TILE;
    const int K = g.K, nkb = (K + QB - 1) / QB, far = 0x40000000;

    const __amdgpu_buffer_rsrc_t rw = buffer_of(g.wq + (int64_t)n0 * K, min(g.N - n0, TILE) * K);
    const __amdgpu_buffer_rsrc_t rx = buffer_of(g.xq + (int64_t)m0 * K, min(g.rows - m0, TILE) * K);
    // wave w copies the groups of 8 rows w, w + 4, ... of X's rows and then W's
    const int row = 8 * wave + (lane >> 3), chunk = (lane & 7) ^ (lane >> 3) ^ (wave & 1);
    auto fetch = [&](int b, int slot, float& xs) {
        int8_t* to = smem + slot * STAGE + 1024 * wave;
        const int at = row * K + 16 * chunk + b * QB, cut = 16 * chunk < K - b * QB ? 0 : far;   // past K: zeros
#pragma unroll
        for (int i = 0; i < NC; ++i)
            buffer_to_lds16(i < 2 ? rx : rw, (at + 32 * (i & 1) * K) | cut, 0, to + 4096 * i);
        xs = g.xs[(int64_t)min(b, nkb - 1) * g.M + min(m0 + 32 * wm + lr, g.rows - 1)];
        asm volatile("" ::: "memory");   // no load may sink past the waits that count it
    };
    const float* wrow = g.ws + (int64_t)(n0 / QB) * nkb;
    auto scales_from = [&](int b) { return wrow[min(b + lane, nkb - 1)]; };
    float wsc = scales_from(0);
    asm volatile("" : "+v"(wsc));

    f32x16 acc{};
    float xs[S];
#pragma unroll
    for (int s = 0; s < S - 1; ++s)
        fetch(s, s, xs[s]);
    int at[4];   // of 16 bytes k in a fragment's row
#pragma unroll
    for (int k = 0; k < 4; ++k)
        at[k] = lr * QB + (((2 * k + lh) ^ swizzle128(lr)) << 4);
    // in rounds of S stages, the last one filled up with zeros
    for (int b0 = 0; b0 < nkb; b0 += S) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int b = b0 + s;
            __builtin_amdgcn_s_waitcnt(wait_vm((S - 2) * COPIES) & WAIT_LDS);
            barrier_no_fence();
            if (b > 0 && (b & 63) == 0) {
                wsc = scales_from(b);
                asm volatile("" : "+v"(wsc));
            }
            fetch(b + S - 1, (s + S - 1) % S, xs[(s + S - 1) % S]);
            __builtin_amdgcn_sched_barrier(0);
            const int8_t *xp = smem + s * STAGE + 32 * wm * QB, *wp = smem + s * STAGE + X_BYTES + 32 * wn * QB;
            i32x8 x[2], w[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                w[k] = cat8(*reinterpret_cast<const i32x4*>(wp + at[2 * k]), *reinterpret_cast<const i32x4*>(wp + at[2 * k + 1]));
                x[k] = cat8(*reinterpret_cast<const i32x4*>(xp + at[2 * k]), *reinterpret_cast<const i32x4*>(xp + at[2 * k + 1]));
            }
            f32x16 p{};
#pragma unroll
            for (int k = 0; k < 2; ++k)
                p = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w[k], x[k], p, 0, 0, 0, 0, 0, 0);
            const float sc = xs[s] * __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wsc), b & 63));
#pragma unroll
            for (int e = 0; e < 16; ++e)
                acc[e] = fmaf(sc, p[e], acc[e]);
        }
    }
    __builtin_amdgcn_s_waitcnt(wait_vm(0) & WAIT_LDS);
    barrier_no_fence();
    // element e of a lane is row lr, column 8 (e / 4) + 4 lh + e % 4
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int c = 32 * wn + 8 * q + 4 * lh;
        Out4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[e] = (OutT)activated<YF16>(acc[4 * q + e] + (g.bias != nullptr ? g.bias[min(n0 + c + e, g.N - 1)] : 0.0f), g.act);
        *reinterpret_cast<Out4*>(smem + (32 * wm + lr) * PITCH + c * (int)sizeof(OutT)) = o;
    }
    __syncthreads();
    constexpr int VEC = 16 / sizeof(OutT), PIECES = TILE / VEC;
    for (int i = threadIdx.x; i < TILE * PIECES; i += 256) {
        const int m = m0 + i / PIECES, n = n0 + i % PIECES * VEC;
        const u32x4 v = *reinterpret_cast<const u32x4*>(smem + i / PIECES * PITCH + i % PIECES * 16);
        OutT* to = reinterpret_cast<OutT*>(g.y) + (int64_t)m * g.N + n;
        if (m < g.rows && n + VEC <= g.N) {
            typedef u32x4 __attribute__((aligned(2))) Piece;   // rows start at any element
            *reinterpret_cast<Piece*>(to) = v;
        } else if (m < g.rows) {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (n + e < g.N)
                    to[e] = reinterpret_cast<const OutT*>(&v)[e];
        }
    }
}

// Many rows: the tiles of gemm_w8a8_tile.h with block scales, 256 x 192 first and then, on the columns
// they leave, 128 x BNS. Workgroup b takes big tile b and then small tile b.
struct BlockPlan {
    int tiles_m_big, nbig, tiles_m_small, nsmall, n_small0;
};

template <int YMODE, int BNS>
__global__ __launch_bounds__(64 * NWAVES, 1) void gemm_block_tile_kernel(BlockGemm g, BlockPlan plan) {
    __shared__ __attribute__((aligned(1024))) int8_t smem[RING_BYTES + SCALE_BYTES];
    const int bid = blockIdx.x, M = (int)g.M;
    const int8_t* A = reinterpret_cast<const int8_t*>(g.xq);
    const int8_t* B = reinterpret_cast<const int8_t*>(g.wq);
    const EpiArgs none{nullptr, nullptr, nullptr, 0};
    if (bid < plan.nbig) {
        const int tile = xcd_remap(bid, plan.nbig);
        const int tn = tile / plan.tiles_m_big, tm = tile - tn * plan.tiles_m_big;
        gemm_tile_pp<256, 192, YMODE, EL_E4M3_BLOCK>(A, g.xs, B, g.ws, g.bias, g.y, M, g.N, g.K, tm * 256, tn * 192, g.act,
                                                     none, smem);
        if (bid >= plan.nsmall)
            return;
        __builtin_amdgcn_s_waitcnt(WAIT_LDS);   // the epilogue has read all it needs from LDS
        barrier_no_fence();
    }
    if (bid < plan.nsmall) {
        const int tile = xcd_remap(bid, plan.nsmall);
        const int tn = tile / plan.tiles_m_small, tm = tile - tn * plan.tiles_m_small;
        gemm_tile_ks<BNS, YMODE, EL_E4M3_BLOCK>(A, g.xs, B, g.ws, g.bias, g.y, M, g.N, g.K, tm * 128,
                                                plan.n_small0 + tn * BNS, g.act, none, smem);
    }
}

// The kernels to choose from: few-row kernels with NB x 16 columns and MB x 16 rows a workgroup, tiles, and
// the kernel between. A call takes rounds of as many workgroups as the chip holds at once, each about a + b * blocks
// of K us long; the least product is chosen. a and b are fits to times on MI355X of 60 shapes. At 250 others (M 1-4096,
// N 192-14336, K 256-14336, from cold memory) the choice takes 3.1% longer than the best in the geometric mean,
// at 202 up to 5%, at 14 up to 10%, at most 48% (32 x 192 x 5120 1x2 7.6 us, 1x1 5.2). Some of both sides, us from cold
// memory (chosen first):
//   1 x 11008 x 4096     2x1 12.1, 1x1 12.9            64 x 4096 x 4096    2x2 7.4, 2x1 9.4, 64x64 14.5
//   32 x 11008 x 4096    4x2 14.5, 2x2 16.6            128 x 4096 x 4096   2x4 10.2, 4x2 10.7, 64x64 14.8
//   96 x 11008 x 4096    64x64 23.2, 128x128 25.8      256 x 4096 x 4096   64x64 15.6, 2x4 18.3, 128x128 19.3
//   512 x 4096 x 4096    64x64 21.9, 128x128 23.5      150 x 2000 x 8192   2x4 17.1, 4x2 15.0
//   333 x 11008 x 4096   128x192 30.5, 256x192 42.2    1024 x 11008 x 4096 256x192 48.2, 128x192 61.7
//   1024 x 4096 x 4096   128x128 26.3, 128x192 30.0    4096 x 4096 x 4096  mixed 79.2, 256x192 82.0
struct Choice {
    int nb, mb, waves, slots;   // few-row kernels; 0: tiles
    int rows, cols;             // of a workgroup
    int per_cu;
    float a, b;
};
constexpr Choice CHOICES[] = {
    {1, 1, 8, 2, 16, 16, 2, 1.4f, 0.13f},  {2, 1, 4, 3, 16, 32, 2, 2.0f, 0.20f},   {1, 2, 8, 2, 32, 16, 1, 1.8f, 0.12f},
    {2, 2, 8, 2, 32, 32, 1, 3.1f, 0.152f}, {4, 2, 4, 3, 32, 64, 1, 3.8f, 0.224f},  {2, 4, 4, 2, 64, 32, 1, 3.45f, 0.217f},
    {0, 0, 0, 0, 128, 128, 1, 5.0f, 0.56f}, {0, 0, 0, 0, 128, 192, 1, 7.4f, 0.65f}, {0, 0, 0, 0, 256, 192, 1, 7.0f, 1.0f},
};
constexpr int FEW = 6, SMALL128 = 6, SMALL192 = 7, BIG = 8, MIXED = 9, MID = 10;
// gemm_block_mid_kernel with one workgroup a CU, and with two
constexpr Choice MID_ONE{0, 0, 0, 0, 64, 64, 1, 4.7f, 0.31f}, MID_TWO{0, 0, 0, 0, 64, 64, 2, 5.5f, 0.404f};

struct Chosen {
    int kernel;       // index into CHOICES; MIXED: whole rounds of big tiles, then 128 x 192; or MID
    int big_panels;   // columns of big tiles
};

Chosen choose(int64_t M, int64_t N, int64_t K) {
    const int64_t kb = e4m3_blocks(K);
    const auto cdiv = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    const auto tiles = [&](const Choice& c, int64_t n) { return cdiv(M, c.rows) * cdiv(n, c.cols); };
    const auto cost = [&](const Choice& c, int64_t wgs) { return (float)cdiv(wgs, c.per_cu * cu_count()) * (c.a + c.b * kb); };
    Chosen best{0, 0};
    float least = cost(CHOICES[0], tiles(CHOICES[0], N));
    for (int i = 1; i <= BIG; ++i) {
        if (i < FEW && CHOICES[i].rows > 16 && CHOICES[i].rows >= 2 * cdiv(M, 16) * 16)
            continue;   // half of its rows or more would be empty
        const float t = cost(CHOICES[i], tiles(CHOICES[i], N));
        if (t < least) {
            least = t;
            best.kernel = i;
        }
    }
    const int64_t mid = tiles(MID_ONE, N);
    const float mid_cost = cost(MID_ONE, mid) < cost(MID_TWO, mid) ? cost(MID_ONE, mid) : cost(MID_TWO, mid);
    if (mid_cost < least) {
        least = mid_cost;
        best.kernel = MID;
    }
    // whole rounds of big tiles, and small ones for the columns that would make a last, short round
    const int64_t big = tiles(CHOICES[BIG], N), panels = big / cu_count() * cu_count() / cdiv(M, 256);
    if (best.kernel == BIG && panels > 0 && panels < cdiv(N, 192)) {
        const float t = cost(CHOICES[BIG], panels * cdiv(M, 256)) + cost(CHOICES[SMALL192], tiles(CHOICES[SMALL192], N - panels * 192));
        if (t < least)
            best = {MIXED, (int)panels};
    }
    if (best.kernel == BIG)
        best.big_panels = (int)cdiv(N, 192);
    return best;
}

template <bool YF16>
void launch_few(const BlockGemm& g, int c, hipStream_t stream) {
    // (The rule takes tiles long before the groups of rows pass the grid's 65535 in y: tests/test_block_grids.py.)
    auto go = [&](auto kernel, auto several) {
        const Choice& k = CHOICES[c];
        const dim3 grid((uint32_t)((g.N + k.cols - 1) / k.cols), (uint32_t)((g.rows + k.rows - 1) / k.rows));
        (g.rows <= k.rows ? kernel : several)<<<grid, dim3(64 * k.waves), 0, stream>>>(g);
    };
    auto of = [&](auto i) {
        constexpr Choice k = CHOICES[decltype(i)::value];
        if (c == decltype(i)::value)
            go(gemm_block_few_kernel<k.nb, k.mb, k.waves, k.slots, YF16, true>,
               gemm_block_few_kernel<k.nb, k.mb, k.waves, k.slots, YF16, false>);
    };
    of(std::integral_constant<int, 0>{});
    of(std::integral_constant<int, 1>{});
    of(std::integral_constant<int, 2>{});
    of(std::integral_constant<int, 3>{});
    of(std::integral_constant<int, 4>{});
    of(std::integral_constant<int, 5>{});
}

template <bool YF16>
void launch_mid(const BlockGemm& g, hipStream_t stream) {
    const int64_t tiles = (g.M + 63) / 64 * ((g.N + 63) / 64);
    gemm_block_mid_kernel<YF16><<<dim3((uint32_t)tiles), dim3(256), 0, stream>>>(g);
}

template <int YMODE>
void launch_tiles(const BlockGemm& g, const Chosen& c, hipStream_t stream) {
    const int64_t small = c.kernel == SMALL128 ? 128 : 192;
    BlockPlan p{};
    p.tiles_m_big = (int)((g.M + 255) / 256);
    p.tiles_m_small = (int)((g.M + 127) / 128);
    p.nbig = p.tiles_m_big * c.big_panels;
    p.n_small0 = c.big_panels * 192;
    p.nsmall = g.N <= p.n_small0 ? 0 : (int)(p.tiles_m_small * ((g.N - p.n_small0 + small - 1) / small));
    const dim3 grid((uint32_t)(p.nbig > p.nsmall ? p.nbig : p.nsmall)), nt(64 * NWAVES);
    if (small == 128)
        gemm_block_tile_kernel<YMODE, 128><<<grid, nt, 0, stream>>>(g, p);
    else
        gemm_block_tile_kernel<YMODE, 192><<<grid, nt, 0, stream>>>(g, p);
}

}  // namespace

extern "C" int ql_gemm_e4m3_block_kernel(int64_t M, int64_t N, int64_t K) { return choose(M, N, K).kernel; }

ql_status launch_gemm_e4m3_block(const uint8_t* xq, const float* x_scale, const uint8_t* wq, const float* w_scale,
                                 const float* bias, int act, void* y, bool y_f16, int64_t M, int64_t N, int64_t K,
                                 hipStream_t stream) {
    const BlockGemm g{xq, x_scale, wq, w_scale, bias, y, (int)M, (int)N, (int)K, act, M};
    const Chosen c = choose(M, N, K);
    if (c.kernel == MID)
        (y_f16 ? launch_mid<true> : launch_mid<false>)(g, stream);
    else if (c.kernel < FEW)
        (y_f16 ? launch_few<true> : launch_few<false>)(g, c.kernel, stream);
    else
        (y_f16 ? launch_tiles<Y_F16> : launch_tiles<Y_F32>)(g, c, stream);
    return launch_status();
}

}  // namespace ql
