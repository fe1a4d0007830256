// gemm_w8a8.hip -- W8A8 GEMM on gfx950 int8 MFMA with int32 accumulation and a fused
// dequantization + bias epilogue.
//
//   acc[m,n] = sum_k xq[m,k] * wq[k,n]                 (int32, exact)
//   y[m,n]   = float(acc) * x_scale[m] * w_scale[n] + bias[n]
//
// hotelren.com "量化算法的本质", "W8A8矩阵乘法": Y = (x_scale*X) @ (w_scale*W) + bias with
// X [M,K] row-major int8 and W [K,N] column-major int8, i.e. both operands K-contiguous.
// quant67.com ch.17 §四: int32 accumulators, scales and bias applied in the epilogue
// while the tile is still in registers (no int32 round trip through memory).
// 2048ai.net INT8 Llama-2-7B write-up §5.3: the K loop double-buffers tiles in on-chip
// memory; here that is LDS, filled while the matrix cores work on the other buffer.
//
// A workgroup of 8 waves (two per SIMD) computes a 256 x 256 output tile on
// v_mfma_i32_32x32x32_i8. K advances 128 bytes per stage through LDS buffers filled by
// direct buffer -> LDS copies (no register staging), whole 128-byte row pieces. The tile
// size is set by L2 -> CU bandwidth: a tile moves (BM + BN) bytes per k for BM * BN
// multiply-adds. The two 4-wave groups alternate between MFMA phases (with the copies
// spread between the MFMAs) and phases of LDS fragment reads, so a SIMD's MFMA stream
// never waits behind its own LDS reads. When the last round of 256 x 256 tiles would leave CUs idle, its N
// panels run as 128 x 256 or 128 x 192 tiles whose K is split between the two groups; a single
// partial round of big tiles runs as 256 x 192 tiles where those put more CUs to work; when
// no round of big tiles fills the chip, every tile is small, as 128 x 128 tiles where those
// make at most one round. K % 128 == 64 runs a last stage whose upper half reads zeros.
#include "gemm_w8a8_tile.h"

namespace ql {
namespace {

// Tiles: `nbig` 256 x BNB tiles (BNB = 256, or 192 when the big tiles make one partial round
// and nothing else) cover the first `nbig / tiles_m` N-panels and `nsmall` 128 x BNS tiles
// (BNS = 256, 192, or 128 when every tile is small) the remaining columns; workgroup b takes
// big tile b, then small tile b (or the small tile first, when staggered).
// With 256 CUs, whole rounds of big tiles keep every CU busy and the leftover panels run
// as half-height tiles in a shorter final round. Within each kind, tiles are dealt to
// XCDs so that an XCD's tiles are consecutive and share W panels (column-major order).
// `stagger` != 0: the workgroups b < nsmall with (b & stagger) != 0 run their half tile first
// and their big tile after it (below).
struct TilePlan {
    int tiles_m_big, nbig, tiles_m_small, nsmall, n_small0, bn_small, bn_big, stagger;
};

template <int YMODE, int ELEM, int BNS, int BNB>
__global__ __launch_bounds__(64 * NWAVES, 1) void gemm_w8a8_kernel(
    const int8_t* __restrict__ A, const float* __restrict__ xs, const int8_t* __restrict__ B,
    const float* __restrict__ ws, const float* __restrict__ bias, void* __restrict__ Y, int M,
    int N, int K, int act, EpiArgs epi, TilePlan plan) {
    __shared__ __attribute__((aligned(1024))) int8_t smem[RING_BYTES + SCALE_BYTES];
    const int bid = blockIdx.x;
    // Staggered order: when every CU runs one big tile and then a half tile, all big tiles
    // finish together and their epilogues store the whole big-tile output (32 MiB at the
    // 2048 x 11008 layer) at once, with the matrix cores idle everywhere. Half of each XCD's
    // workgroups (bit 3 of b: workgroups are dealt to the XCDs round-robin) instead run the
    // half tile first, so half of that burst overlaps the other workgroups' K loops. The
    // tiles and their sums are unchanged.
    if ((bid & plan.stagger) != 0 && bid < plan.nsmall && bid < plan.nbig) {
        {
            const int tile = xcd_remap(bid, plan.nsmall);
            const int tn = tile / plan.tiles_m_small, tm = tile - tn * plan.tiles_m_small;
            gemm_tile_ks<BNS, YMODE, ELEM>(A, xs, B, ws, bias, Y, M, N, K, tm * 128, plan.n_small0 + tn * BNS, act,
                                          epi, smem);
        }
        // the half tile's epilogue has read all it needs from LDS
        __builtin_amdgcn_s_waitcnt(vmcnt_le(63) & ~(0xF << 8));   // lgkmcnt(0)
        barrier_no_fence();
        const int tile = xcd_remap(bid, plan.nbig);
        const int tn = tile / plan.tiles_m_big, tm = tile - tn * plan.tiles_m_big;
        gemm_tile_pp<256, BNB, YMODE, ELEM>(A, xs, B, ws, bias, Y, M, N, K, tm * 256, tn * BNB, act, epi, smem);
        return;
    }
    if (bid < plan.nbig) {
        const int tile = xcd_remap(bid, plan.nbig);
        const int tn = tile / plan.tiles_m_big, tm = tile - tn * plan.tiles_m_big;
        gemm_tile_pp<256, BNB, YMODE, ELEM>(A, xs, B, ws, bias, Y, M, N, K, tm * 256, tn * BNB, act, epi, smem);
        if (bid >= plan.nsmall)
            return;
        // The big tile's epilogue has read all it needs from LDS (its stores may still be in
        // flight): the half tile may refill the LDS.
        __builtin_amdgcn_s_waitcnt(vmcnt_le(63) & ~(0xF << 8));   // lgkmcnt(0)
        barrier_no_fence();
    }
    if (bid < plan.nsmall) {
        const int tile = xcd_remap(bid, plan.nsmall);
        const int tn = tile / plan.tiles_m_small, tm = tile - tn * plan.tiles_m_small;
        gemm_tile_ks<BNS, YMODE, ELEM>(A, xs, B, ws, bias, Y, M, N, K, tm * 128, plan.n_small0 + tn * BNS, act, epi,
                                      smem);
    }
}

TilePlan plan_tiles(int64_t M, int64_t N) {
    TilePlan p{};
    const int tm = (int)((M + 255) / 256), tn = (int)((N + 255) / 256);
    const int total = tm * tn, cus = cu_count();
    int small_panels = 0;
    if (M <= 128 || 2 * total <= cus) {
        // every tile is half height: with at most half the CUs' worth of big tiles, half
        // tiles (K split between the two wave groups) put twice as many CUs to work
        small_panels = tn;
    } else if (total > cus) {
        const int left = total % cus;           // tiles of the last, partial round
        if (left > 0 && left <= cus / 2)
            small_panels = (left + tm - 1) / tm;
    }
    p.tiles_m_big = tm;
    p.nbig = (tn - small_panels) * tm;
    p.tiles_m_small = (int)((M + 127) / 128);
    p.nsmall = small_panels * p.tiles_m_small;
    p.n_small0 = (tn - small_panels) * 256;
    p.bn_small = 256;
    p.bn_big = 256;
    return p;
}

// 256 x 192 big tiles when the 256 x 256 ones make one partial round and no small tiles follow
// (between half and all of the CUs), and the narrower tiles put more CUs to work, still in one
// round: each does three quarters of a big tile's work. Measured at K = 4096 (us, 256 x 256 /
// 256 x 192; the same int32 sums and outputs): M = 768, N = 11008 (129 / 174 tiles) 43.5 /
// 36.9; M = 1024, N = 11008 46.0 / 43.1; M = 768, N = 14336 44.9 / 42.1; M = 1280, N = 8192
// 43.8 / 40.4; M = 768, N = 11008, K = 11008 95.9 / 85.4.
int big_tiles_192(const TilePlan& p, int64_t N) { return p.tiles_m_big * (int)((N + 191) / 192); }

bool use_big_192(const TilePlan& p, int64_t N) {
    const int n = big_tiles_192(p, N);
    return p.nsmall == 0 && p.nbig > 0 && p.nbig < cu_count() && n > p.nbig && n <= cu_count();
}

TilePlan plan_big_192(TilePlan p, int64_t N) {
    p.nbig = big_tiles_192(p, N);
    p.bn_big = 192;
    return p;
}

// The 64 x 64 kernel (gemm_w8a8_mid.hip) takes the shapes where the tile plan puts at most
// half of the CUs to work and its own tiles make at most two rounds. Measured at K = 4096
// (us, tile plan against 64 x 64 tiles): N = 4096: M = 256 24.3 / 13.5, M = 512 25.5 / 17.2,
// M = 768 27.3 / 28.4; N = 11008: M = 129 26.7 / 27.0, M = 256 27.6 / 29.1; at M = 256,
// N = 4096 also K = 11008 53.7 / 30.6 and K = 14336 66.4 / 38.4.
// 128 x 128 small tiles instead of 128 x 256 when every tile is small and the 128 x 128 tiles
// make at most one round: twice the workgroups on the same two-group split-K schedule.
// Measured at K = 4096 (us, 128 x 256 / 128 x 128): N = 4096: M = 600 30.4 / 21.9, M = 768
// 31.5 / 23.0, M = 1024 31.2 / 23.1; N = 11008: M = 129 29.4 / 21.5, M = 256 34.0 / 24.1;
// N = 14336, M = 256 35.1 / 25.6; N = 4096, M = 1024, K = 11008 74.1 / 53.4; M = 768,
// K = 14336 92.7 / 65.9. Past one round it loses (M = 1536, N = 4096: 32.4 / 43.3; M = 384,
// N = 11008, 258 tiles: 32.6 / 34.6).
bool use_quarter_tiles(const TilePlan& p, int64_t N) {
    return p.nbig == 0 && (int64_t)p.tiles_m_small * ((N + 127) / 128) <= cu_count();
}

TilePlan quarter_plan(TilePlan p, int64_t N) {
    p.nsmall = p.tiles_m_small * (int)((N + 127) / 128);
    p.bn_small = 128;
    return p;
}

// Small tiles 192 columns wide where they make more workgroups than 256-wide ones and still
// at most one round: the small tiles run together, so the widest sets their time, and a CU's
// operand bytes per tile fall by a sixth. Measured at K = 4096 (us, 128 x 256 / 128 x 192; the
// same int32 sums and outputs): M = 2048, N = 11008 (256 big tiles, then 176 / 240 small)
// 86.6 / 84.0; M = 384, N = 11008 27.9 / 24.3; M = 512, N = 11008 30.6 / 27.4; M = 384,
// N = 14336 31.2 / 27.2; M = 600, N = 9000 30.8 / 27.6; M = 1025, N = 4096 28.6 / 24.7;
// M = 1536, N = 11008 78.6 / 74.4; M = 3072, N = 11008 132.9 / 128.2; M = 512, N = 11008,
// K = 11008 66.2 / 60.2.
int small_tiles_192(const TilePlan& p, int64_t N) {
    return p.tiles_m_small * (int)((N - p.n_small0 + 191) / 192);
}

bool use_192_tiles(const TilePlan& p, int64_t N) {
    const int n = small_tiles_192(p, N);
    return p.nsmall > 0 && n > p.nsmall && n <= cu_count();
}

TilePlan plan_192(TilePlan p, int64_t N) {
    p.nsmall = small_tiles_192(p, N);
    p.bn_small = 192;
    return p;
}

bool use_mid_tiles(const TilePlan& p, int64_t M, int64_t N) {
    const int wgs = p.nbig > p.nsmall ? p.nbig : p.nsmall;
    const int64_t mid = ((M + 63) / 64) * ((N + 63) / 64);
    return 2 * wgs <= cu_count() && mid <= 2 * (int64_t)cu_count();
}

}  // namespace

ql_status launch_gemm_w8a8(const int8_t* xq, const float* x_scale, const int8_t* wq,
                           const float* w_scale, const float* bias, void* y, int y_mode, int act,
                           const float* x_zero, const int32_t* colsum, int64_t M, int64_t N,
                           int64_t K, hipStream_t stream, bool e4m3, const float* out_scale,
                           int out_scale_n) {
    if (M == 0 || N == 0)
        return QL_OK;
    TilePlan plan = plan_tiles(M, N);
    if (use_mid_tiles(plan, M, N)) {
        // the tile plan would leave most CUs idle: 64 x 64 tiles instead
        return launch_gemm_w8a8_mid(xq, x_scale, wq, w_scale, bias, y, y_mode, act, x_zero, colsum, out_scale,
                                    out_scale_n, M, N, K, stream, e4m3);
    }
    if (use_quarter_tiles(plan, N))
        plan = quarter_plan(plan, N);
    else if (use_192_tiles(plan, N))
        plan = plan_192(plan, N);
    else if (use_big_192(plan, N))
        plan = plan_big_192(plan, N);
    // One round of big tiles followed by half tiles on the same workgroups: stagger the order
    // on half of them. Measured at K = 4096 (us, all big-first / staggered; the same outputs):
    // M = 2048, N = 11008 83.1 / 80.6 and 82.9 / 80.3; N = 10000 82.4 / 81.4; N = 8704 76.7 /
    // 74.7; M = 1792, N = 11008 81.6 / 81.1; M = 2048, N = 9000 77.2 / 77.5; at K = 11008
    // 192.5 / 191.0. With two rounds of big tiles (M = 3072, N = 11008) staggering delayed the
    // first round (123.8 / 124.9), so it is not used there.
    plan.stagger = plan.nsmall > 0 && plan.nbig <= cu_count() ? 8 : 0;
    // Workgroup b runs big tile b (b < nbig) and then half tile b (b < nsmall), or the two the
    // other way round when staggered, so the half tiles need no dispatch of their own and
    // each tile's first copies overlap the previous tile's last stores.
    const dim3 grid((unsigned)(plan.nbig > plan.nsmall ? plan.nbig : plan.nsmall)), block(64 * NWAVES);
    const int m = (int)M, n = (int)N, k = (int)K;
#define QL_LAUNCH_ONE(MODE, EL, BNS, BNB)                                                                \
    hipLaunchKernelGGL((gemm_w8a8_kernel<MODE, EL, BNS, BNB>), grid, block, 0, stream, xq, x_scale, wq, w_scale, \
                       bias, y, m, n, k, act, (EpiArgs{x_zero, colsum, out_scale, out_scale_n}), plan)
#define QL_LAUNCH(MODE, EL)                                                                              \
    do {                                                                                                 \
        if (plan.bn_big == 192)                                                                          \
            QL_LAUNCH_ONE(MODE, EL, 256, 192);                                                           \
        else if (plan.bn_small == 128)                                                                   \
            QL_LAUNCH_ONE(MODE, EL, 128, 256);                                                           \
        else if (plan.bn_small == 192)                                                                   \
            QL_LAUNCH_ONE(MODE, EL, 192, 256);                                                           \
        else                                                                                             \
            QL_LAUNCH_ONE(MODE, EL, 256, 256);                                                           \
    } while (0)
    if (e4m3) {
        if (y_mode == Y_F32)
            QL_LAUNCH(Y_F32, EL_E4M3);
        else
            QL_LAUNCH(Y_F16, EL_E4M3);
        return launch_status();
    }
    switch (y_mode) {
    case Y_I8:
        QL_LAUNCH(Y_I8, EL_I8);
        break;
    case Y_F32:
        QL_LAUNCH(Y_F32, EL_I8);
        break;
    case Y_F16:
        QL_LAUNCH(Y_F16, EL_I8);
        break;
    default:
        QL_LAUNCH(Y_I32, EL_I8);
        break;
    }
#undef QL_LAUNCH
#undef QL_LAUNCH_ONE
    return launch_status();
}

}  // namespace ql
