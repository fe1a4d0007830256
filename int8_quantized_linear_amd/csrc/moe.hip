// moe.hip -- a mixture-of-experts layer for a few tokens, its weights in E4M3 codes with a scale for
// each block of 128 x 128.
//
//   p       = softmax(logits[t]); e_1 .. e_k its largest, equal ones by the lower number first
//   h_j     = p_j silu(W1[e_j] x) * (W3[e_j] x)         (p_j over their sum, if renormalized)
//   out[t]  = sum_j W2[e_j] h_j
//
// Bound by the read of the chosen experts' codes: a token's products are 2 operations a code. Two
// kernels: the gated products of every (token, expert) pair into the workspace, and the sums over
// the experts. Codes become fp16 (first kernel, beside x) or bf16 (second kernel) exactly, the
// products run on the matrix cores with fp32 sums from zero for each block of 128, and the block's
// scale is applied in fp32. h is kept as two bf16 terms (16 bits of significand, fp32's range): one
// rounding of relative size 2^-17 that its products see.
//
// A wave reads codes through its own ring in LDS, copied there directly and several blocks ahead;
// the other operand's few rows come from L2 into registers, as far ahead. The order of every sum is
// fixed, whatever the other tokens are.
#include "e4m3_block.h"

namespace ql {
namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int NW = 8;            // waves of a workgroup
constexpr int NT = NW * WAVE;

// Workgroup barrier that leaves copies into LDS in flight (__syncthreads would wait for them); LDS
// operations before it are done.
__device__ inline void barrier_lds() {
    __builtin_amdgcn_s_waitcnt(WAIT_LDS);
    asm volatile("s_barrier" ::: "memory");
}

// ------------------------------------------------------------------------------- the router
//
// logits[t][e] = sum_k x[t][k] w[e][k], 16 experts and 16 tokens a workgroup, its waves taking every
// 16th step of 32 k.

constexpr int RW = 16;   // waves
constexpr int RU = 4;    // steps of a wave in flight

__global__ __launch_bounds__(RW* WAVE) void moe_router_kernel(const _Float16* __restrict__ x,
                                                              const _Float16* __restrict__ w, float* __restrict__ logits,
                                                              int64_t T, int E, int K) {
    __shared__ f32x4 red[RW][WAVE];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, q = lane >> 4;
    const int e0 = blockIdx.x * 16;
    const int64_t t0 = (int64_t)blockIdx.y * 16;
    const _Float16* wp = w + (int64_t)min(e0 + r, E - 1) * K + 8 * q;
    const _Float16* xp = x + min(t0 + r, T - 1) * K + 8 * q;
    f32x4 acc{0, 0, 0, 0};
    const int steps = K / 32;
    for (int s = wave; s < steps; s += RU * RW) {
        f16x8 a[RU], b[RU];
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            const int at = 32 * min(s + u * RW, steps - 1);
            a[u] = *reinterpret_cast<const f16x8*>(wp + at);
            b[u] = *reinterpret_cast<const f16x8*>(xp + at);
        }
#pragma unroll
        for (int u = 0; u < RU; ++u)
            if (s + u * RW < steps)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[u], b[u], acc, 0, 0, 0);
    }
    red[wave][lane] = acc;
    __syncthreads();
    // element i of lane l is expert 4 q + i, token r
    if (wave < 4) {
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < RW; ++v)
            sum += red[v][lane][wave];
        const int e = e0 + 4 * q + wave;
        if (e < E && t0 + r < T)
            logits[(t0 + r) * E + e] = sum;
    }
}

// -------------------------------------------------------------------------------- the routes
//
// Every workgroup of the first kernel works the routes out for itself from the logits (it would
// wait as long for another to do it). Pairs (expert, token) are numbered expert by expert, tokens
// in order.

struct Routes {
    unsigned long long tokens[MOE_EXPERTS];   // bit t: token t takes the expert
    uint16_t base[MOE_EXPERTS];               // first pair of an expert
    uint16_t act[MOE_EXPERTS];                // experts that some token takes
    uint16_t id[MOE_TOKENS][MOE_TOP_K];       // of a token, MOE_EXPERTS for none
    float p[MOE_TOKENS][MOE_TOP_K];
    float pair_p[MOE_TOKENS * MOE_TOP_K];
    uint16_t pair_token[MOE_TOKENS * MOE_TOP_K];
    uint32_t part[NW];
    int nact;
};

// The workspace: the routes as the second kernel needs them, then h's two terms, [pairs][I] each.
struct MoeSpace {
    int nact;
    int pad[3];
    struct {
        uint16_t expert, base, count, pad;
    } act[MOE_EXPERTS];
    uint16_t pair_token[MOE_TOKENS * MOE_TOP_K];
};

struct Moe {
    MoeLayer l;
    int T;           // tokens of this launch
    MoeSpace* space;
    __bf16 *hi, *lo;
};

template <class F>
__device__ inline float row16(float v, F f) {
    auto step = [&](auto ctrl) {
        v = f(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, 0xF, 0xF, true)));
    };
    step(std::integral_constant<int, 0x128>{});   // rotations by 8, 4, 2 and 1 of 16 lanes
    step(std::integral_constant<int, 0x124>{});
    step(std::integral_constant<int, 0x122>{});
    step(std::integral_constant<int, 0x121>{});
    return v;
}

__device__ inline int row16_min(int v) {
    auto step = [&](auto ctrl) {
        v = min(v, __builtin_amdgcn_update_dpp(0, v, decltype(ctrl)::value, 0xF, 0xF, true));
    };
    step(std::integral_constant<int, 0x128>{});
    step(std::integral_constant<int, 0x124>{});
    step(std::integral_constant<int, 0x122>{});
    step(std::integral_constant<int, 0x121>{});
    return v;
}

// 16 lanes a token, R logits a lane: top_k rounds of the largest that is left. NaN is never taken,
// nor is -infinity.
template <int R>
__device__ inline void make_routes(Routes& rt, const Moe& g) {
    const int tid = threadIdx.x, E = g.l.E, k = g.l.top_k;
    for (int e = tid; e < MOE_EXPERTS; e += NT)
        rt.tokens[e] = 0;
    __syncthreads();
    const int l = tid & 15;
    for (int t0 = 0; t0 < g.T; t0 += NT / 16) {
        const int t = t0 + tid / 16;
        const float* row = g.l.logits + (int64_t)min(t, g.T - 1) * E;
        float v[R];
        float top = -INFINITY;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            v[r] = 16 * r + l < E ? row[16 * r + l] : -INFINITY;
            top = fmaxf(top, v[r]);
        }
        top = row16(top, [](float a, float b) { return fmaxf(a, b); });
        const float from = top == -INFINITY ? 0.0f : top;
        float all = 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r)
            all += v[r] == v[r] ? __expf(v[r] - from) : 0.0f;
        all = row16(all, [](float a, float b) { return a + b; });
        float chosen = 0.0f, mine = 0.0f;
        int my_id = MOE_EXPERTS;
        for (int j = 0; j < k; ++j) {
            float best = -INFINITY;
#pragma unroll
            for (int r = 0; r < R; ++r)
                best = fmaxf(best, v[r]);
            best = row16(best, [](float a, float b) { return fmaxf(a, b); });
            int at = MOE_EXPERTS;
#pragma unroll
            for (int r = R - 1; r >= 0; --r)
                at = v[r] == best ? 16 * r + l : at;
            at = row16_min(at);
            at = best == -INFINITY ? MOE_EXPERTS : at;
            const float p = best == -INFINITY ? 0.0f : __expf(best - from);
            chosen += p;
            if (l == j) {
                mine = p;
                my_id = at;
            }
#pragma unroll
            for (int r = 0; r < R; ++r)
                v[r] = 16 * r + l == at ? -INFINITY : v[r];
        }
        if (t < g.T && l < k) {
            rt.id[t][l] = (uint16_t)my_id;
            rt.p[t][l] = mine / (g.l.renormalize ? chosen : all);
            if (my_id < MOE_EXPERTS)
                atomicOr(&rt.tokens[my_id], 1ull << t);
        }
    }
    __syncthreads();
    // experts in use, and their first pairs: a running sum over the experts, one a thread
    static_assert(NT == MOE_EXPERTS, "one expert a thread");
    const unsigned long long m = rt.tokens[tid];
    const uint32_t own = (uint32_t)__popcll(m) << 16 | (m != 0);
    uint32_t sum = own;
#pragma unroll
    for (int o = 1; o < WAVE; o <<= 1) {
        const uint32_t up = __shfl_up(sum, o, WAVE);
        sum += (tid & 63) >= o ? up : 0;
    }
    if ((tid & 63) == 63)
        rt.part[tid >> 6] = sum;
    __syncthreads();
    sum -= own;
    uint32_t total = 0;
    for (int w = 0; w < NW; ++w) {
        total += rt.part[w];
        sum += w < tid >> 6 ? rt.part[w] : 0;
    }
    rt.base[tid] = (uint16_t)(sum >> 16);
    if (m != 0)
        rt.act[sum & 0xFFFF] = (uint16_t)tid;
    if (tid == 0)
        rt.nact = (int)(total & 0xFFFF);
    __syncthreads();
    for (int i = tid; i < g.T * k; i += NT) {
        const int t = i / k, e = rt.id[t][i % k];
        if (e < MOE_EXPERTS) {
            const int at = rt.base[e] + __popcll(rt.tokens[e] & ((1ull << t) - 1));
            rt.pair_token[at] = (uint16_t)t;
            rt.pair_p[at] = rt.p[t][i % k];
        }
    }
    __syncthreads();
}

// 8 codes (two words) as fp16 or bf16, exactly.
__device__ inline f16x8 codes_f16(int w0, int w1) {
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.0f, false);
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.0f, true);
    const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.0f, false);
    const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.0f, true);
    return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ inline bf16x8 codes_bf16(int w0, int w1) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// ------------------------------------------------------------------------ the gated products
//
// A task is an expert in use and 16 columns of h: 16 rows of W1 and 16 of W3 against the expert's
// tokens (TILES tiles of 16). A workgroup takes every gridDim-th task; its waves split K, wave w
// taking the blocks w, w + 8, ... of every task. The wave's items (task, block) make one sequence, so
// the next task's first copies are in flight while a task's sums are joined. W is the first
// operand: a lane's sums belong to one token (lane & 15) and four columns of h.

template <int TILES>
constexpr int UP_DEPTH = TILES == 4 ? 2 : 3;

template <int TILES, int R>
__global__ __launch_bounds__(NT) void moe_up_kernel(Moe g) {
    constexpr int S = UP_DEPTH<TILES>, SLOT = 4096 + 256, BATCH = 5 + 4 * TILES;
    __shared__ Routes rt;
    __shared__ __attribute__((aligned(1024))) int8_t rings[NW * S * SLOT];
    __shared__ f32x4 red[NW][TILES][2][WAVE];
    make_routes<R>(rt, g);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4;
    const int K = g.l.K, I = g.l.I, nact = __builtin_amdgcn_readfirstlane(rt.nact);
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0)
            g.space->nact = nact;
        for (int i = threadIdx.x; i < nact; i += NT) {
            const int e = rt.act[i];
            g.space->act[i] = {(uint16_t)e, rt.base[e], (uint16_t)__popcll(rt.tokens[e]), 0};
        }
        for (int i = threadIdx.x; i < g.T * g.l.top_k; i += NT)
            g.space->pair_token[i] = rt.pair_token[i];
    }
    const int nkb = (K + QB - 1) / QB, cols = I / 16, tasks = nact * cols;
    const int J = (nkb + NW - 1) / NW;                       // a wave's blocks of a task
    const int first = blockIdx.x, G = gridDim.x;
    const int mine = first < tasks ? (tasks - first + G - 1) / G : 0;
    const int items = mine * J;
    if (items == 0)
        return;

    int8_t* ring = rings + wave * S * SLOT;
    const int64_t blocks13 = e4m3_blocks(2 * (int64_t)I);
    const __amdgpu_buffer_rsrc_t rx = buffer_of(g.l.x, g.T * K * 2);
    const int row = lane >> 3, c0 = copy_chunk128(lane, 0), c1 = copy_chunk128(lane, 1);
    const int far = 0x40000000;

    // the item that is fetched next
    struct {
        int task, j;
        __amdgpu_buffer_rsrc_t gate, up;
        const float* scale;
        int xoff[TILES];
    } nx;
    auto enter = [&](int task) {
        nx.task = task;
        nx.j = 0;
        const int a = min(task, tasks - 1);
        const int e = __builtin_amdgcn_readfirstlane(rt.act[a / cols]), i0 = (a % cols) * 16;
        const int size = task < tasks ? 16 * K : 0;
        const uint8_t* w = g.l.w13 + ((int64_t)e * 2 * I + i0) * K;
        nx.gate = buffer_of(w, size);
        nx.up = buffer_of(w + (int64_t)I * K, size);
        nx.scale = g.l.s13 + (e * blocks13 + (i0 + (lane < 32 ? 0 : I)) / QB) * nkb;
        const int base = rt.base[e], count = __popcll(rt.tokens[e]);
#pragma unroll
        for (int i = 0; i < TILES; ++i)   // columns past the tokens repeat the last one
            nx.xoff[i] = (rt.pair_token[base + min(16 * i + r, count - 1)] * K + 16 * q) * 2;
    };
    i32x4 xv[S][TILES][4];
    auto fetch = [&](int slot, i32x4 (&x)[TILES][4]) {
        int8_t* to = ring + slot * SLOT;
        const int b = wave + NW * nx.j, left = K - b * QB;
        const int cut0 = 16 * c0 < left ? 0 : far, cut1 = 16 * c1 < left ? 0 : far;
        const int o0 = row * K + 16 * c0 + b * QB, o1 = (row + 8) * K + 16 * c1 + b * QB;
        buffer_to_lds16<2>(nx.gate, o0 | cut0, 0, to);
        buffer_to_lds16<2>(nx.gate, o1 | cut1, 0, to + 1024);
        buffer_to_lds16<2>(nx.up, o0 | cut0, 0, to + 2048);
        buffer_to_lds16<2>(nx.up, o1 | cut1, 0, to + 3072);
        global_to_lds4(nx.scale + min(b, nkb - 1), to + 4096);
        // past K the codes are zeros, and x anything finite
        const int bx = min(b, nkb - 1) * QB, half = left > 64 ? 128 : 0;
#pragma unroll
        for (int i = 0; i < TILES; ++i)
#pragma unroll
            for (int f = 0; f < 4; ++f)
                x[i][f] = __builtin_amdgcn_raw_buffer_load_b128(rx, nx.xoff[i] + 16 * (f & 1) + (f >> 1) * half, 2 * bx, 0);
        asm volatile("" ::: "memory");   // no load may sink past the waits that count it
        if (++nx.j == J)
            enter(nx.task + G);
    };

    f32x4 acc[TILES][2];
    auto clear = [&]() {
#pragma unroll
        for (int i = 0; i < TILES; ++i)
            acc[i][0] = acc[i][1] = f32x4{0, 0, 0, 0};
    };
    clear();
    enter(first);
#pragma unroll
    for (int s = 0; s < S - 1; ++s)
        fetch(s, xv[s]);
    int task = first, j = 0;
    const int f0 = r * QB + ((q ^ swizzle128(r)) << 4), f1 = r * QB + (((q + 4) ^ swizzle128(r)) << 4);
    // in rounds of S items, the last one filled up with zeros (a branch out of the middle would make
    // the compiler wait for all loads in every round)
    for (int it = 0; it < items; it += S) {
#pragma unroll
        for (int u = 0; u < S; ++u) {
            fetch((u + S - 1) % S, xv[(u + S - 1) % S]);
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(wait_vm((S - 1) * BATCH));
            __builtin_amdgcn_sched_barrier(0);
            const int8_t* at = ring + u * SLOT;
            const i32x4 g0 = *reinterpret_cast<const i32x4*>(at + f0), g1 = *reinterpret_cast<const i32x4*>(at + f1);
            const i32x4 u0 = *reinterpret_cast<const i32x4*>(at + 2048 + f0);
            const i32x4 u1 = *reinterpret_cast<const i32x4*>(at + 2048 + f1);
            const float sg = *reinterpret_cast<const float*>(at + 4096);
            const float su = *reinterpret_cast<const float*>(at + 4096 + 128);
            const f16x8 ga[4] = {codes_f16(g0[0], g0[1]), codes_f16(g0[2], g0[3]), codes_f16(g1[0], g1[1]), codes_f16(g1[2], g1[3])};
            const f16x8 ua[4] = {codes_f16(u0[0], u0[1]), codes_f16(u0[2], u0[3]), codes_f16(u1[0], u1[1]), codes_f16(u1[2], u1[3])};
#pragma unroll
            for (int i = 0; i < TILES; ++i) {
                f32x4 pg{0, 0, 0, 0}, pu{0, 0, 0, 0};
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    const f16x8 b = __builtin_bit_cast(f16x8, xv[u][i][f]);
                    pg = __builtin_amdgcn_mfma_f32_16x16x32_f16(ga[f], b, pg, 0, 0, 0);
                    pu = __builtin_amdgcn_mfma_f32_16x16x32_f16(ua[f], b, pu, 0, 0, 0);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    acc[i][0][e] = fmaf(sg, pg[e], acc[i][0][e]);
                    acc[i][1][e] = fmaf(su, pu[e], acc[i][1][e]);
                }
            }
            __builtin_amdgcn_s_waitcnt(WAIT_LDS);   // the slot's reads are done before it is filled again
            __builtin_amdgcn_sched_barrier(0);
            if (++j == J && task < tasks) {
                // the task's sums of all waves, joined by one wave a tile
#pragma unroll
                for (int i = 0; i < TILES; ++i) {
                    red[wave][i][0][lane] = acc[i][0];
                    red[wave][i][1][lane] = acc[i][1];
                }
                clear();
                barrier_lds();
                const int e = rt.act[task / cols], i0 = (task % cols) * 16;
                const int pair = 16 * wave + r, count = __popcll(rt.tokens[e]);
                if (wave < TILES && 16 * wave < count) {
                    f32x4 gs = red[0][wave][0][lane], us = red[0][wave][1][lane];
#pragma unroll
                    for (int w = 1; w < NW; ++w) {
                        gs += red[w][wave][0][lane];
                        us += red[w][wave][1][lane];
                    }
                    if (pair < count) {
                        const int at_pair = rt.base[e] + pair;
                        const float p = rt.pair_p[at_pair];
                        bf16x4 hi, lo;
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            const float h = p * activation<ACT_SILU>(gs[n]) * us[n];
                            hi[n] = (__bf16)h;
                            lo[n] = (__bf16)(h - (float)hi[n]);
                        }
                        const int64_t to = (int64_t)at_pair * I + i0 + 4 * q;
                        *reinterpret_cast<bf16x4*>(g.hi + to) = hi;
                        *reinterpret_cast<bf16x4*>(g.lo + to) = lo;
                    }
                }
                barrier_lds();
                j = 0;
                task += G;
            }
        }
    }
    __builtin_amdgcn_s_waitcnt(wait_vm(0));
}

// --------------------------------------------------------------------- the sums over experts
//
// A workgroup owns 16 columns of the output. Block b of expert e is wave (e * blocks + b) % 8's: a
// wave's blocks of an expert lie 8 apart (neighbouring waves read neighbouring 128 bytes), the waves
// have about as many blocks each, and which wave adds what to a token's sums does not depend on the
// other tokens' experts. A wave adds an expert's products to its own sums [token][16] in LDS, and the
// waves' sums are added at the end.

template <int TILES>
__global__ __launch_bounds__(NT) void moe_down_kernel(Moe g) {
    constexpr int S = TILES == 1 ? 4 : 3, SLOT = 2048 + 256, TOK = 16 * TILES;
    constexpr int BATCH = 3 + 8;
    __shared__ __attribute__((aligned(1024))) int8_t rings[NW * S * SLOT];
    __shared__ float sums[NW][TOK][16];
    __shared__ __attribute__((aligned(8))) uint16_t act[MOE_EXPERTS][4];   // expert, first pair, pairs
    __shared__ __attribute__((aligned(4))) uint16_t pair_token[TOK * MOE_TOP_K];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4;
    const int K = g.l.K, I = g.l.I, n0 = blockIdx.x * 16;
    const int nact = __builtin_amdgcn_readfirstlane(g.space->nact);
    for (int i = threadIdx.x; i < nact; i += NT)
        *reinterpret_cast<u32x2*>(act[i]) = *reinterpret_cast<const u32x2*>(&g.space->act[i]);
    for (int i = threadIdx.x; i < (g.T * g.l.top_k + 1) / 2; i += NT)
        reinterpret_cast<uint32_t*>(pair_token)[i] = reinterpret_cast<const uint32_t*>(g.space->pair_token)[i];
    for (int i = threadIdx.x; i < NW * TOK * 4; i += NT)
        reinterpret_cast<f32x4*>(sums)[i] = f32x4{0, 0, 0, 0};
    __syncthreads();
    const int nib = (I + QB - 1) / QB;

    int8_t* ring = rings + wave * S * SLOT;
    const int64_t blocks2 = e4m3_blocks(K);
    const int pairs = g.T * g.l.top_k;
    const __amdgpu_buffer_rsrc_t rh = buffer_of(g.hi, pairs * I * 2), rl = buffer_of(g.lo, pairs * I * 2);
    const int row = lane >> 3, c0 = copy_chunk128(lane, 0), c1 = copy_chunk128(lane, 1);
    const int far = 0x40000000;
    auto pair_offset = [&](int s, int tile) {   // columns past the pairs repeat the last one
        const int base = act[s][1], count = act[s][2];
        return ((base + min(16 * tile + r, count - 1)) * I + 16 * q) * 2;
    };
    // the wave's first block of the next expert in use, from number s on, that has one; s == nact
    // at the end
    auto next = [&](int& s, int& b) {
        for (; s < nact; ++s) {
            b = (wave - __builtin_amdgcn_readfirstlane(act[s][0]) * nib) & (NW - 1);
            if (b < nib)
                return;
        }
        b = 0;
    };
    struct {
        int s, b;   // what is fetched next
        __amdgpu_buffer_rsrc_t w;
        const float* scale;
        int hoff;
    } nx;
    auto enter = [&]() {
        next(nx.s, nx.b);
        const int a = min(nx.s, nact - 1);
        const int e = __builtin_amdgcn_readfirstlane(act[a][0]);
        nx.w = buffer_of(g.l.w2 + ((int64_t)e * K + n0) * I, nx.s < nact ? 16 * I : 0);
        nx.scale = g.l.s2 + (e * blocks2 + n0 / QB) * nib;
        nx.hoff = pair_offset(a, 0);
    };
    i32x4 hv[S][2][4];
    auto load_h = [&](i32x4 (&h)[2][4], int off, int b) {
        const int half = I - b * QB > 64 ? 128 : 0;   // past I the codes are zeros, and h anything finite
#pragma unroll
        for (int f = 0; f < 4; ++f) {
            h[0][f] = __builtin_amdgcn_raw_buffer_load_b128(rh, off + 16 * (f & 1) + (f >> 1) * half, 2 * b * QB, 0);
            h[1][f] = __builtin_amdgcn_raw_buffer_load_b128(rl, off + 16 * (f & 1) + (f >> 1) * half, 2 * b * QB, 0);
        }
    };
    auto fetch = [&](int slot, i32x4 (&h)[2][4]) {
        int8_t* to = ring + slot * SLOT;
        const int left = I - nx.b * QB;
        const int cut0 = 16 * c0 < left ? 0 : far, cut1 = 16 * c1 < left ? 0 : far;
        const int o0 = row * I + 16 * c0 + nx.b * QB, o1 = (row + 8) * I + 16 * c1 + nx.b * QB;
        buffer_to_lds16<2>(nx.w, o0 | cut0, 0, to);
        buffer_to_lds16<2>(nx.w, o1 | cut1, 0, to + 1024);
        global_to_lds4(nx.scale + nx.b, to + 2048);
        load_h(h, nx.hoff, nx.b);
        asm volatile("" ::: "memory");   // no load may sink past the waits that count it
        nx.b += NW;
        if (nx.b >= nib) {
            ++nx.s;
            enter();
        }
    };

    f32x4 acc[TILES];
#pragma unroll
    for (int i = 0; i < TILES; ++i)
        acc[i] = f32x4{0, 0, 0, 0};
    int s = 0, b = 0;
    if (nact > 0)
        next(s, b);
    if (s < nact) {
        nx.s = 0;
        enter();
#pragma unroll
        for (int i = 0; i < S - 1; ++i)
            fetch(i, hv[i]);
        const int f0 = r * QB + ((q ^ swizzle128(r)) << 4), f1 = r * QB + (((q + 4) ^ swizzle128(r)) << 4);
        while (s < nact) {   // in rounds, as in the first kernel
#pragma unroll
            for (int u = 0; u < S; ++u) {
                fetch((u + S - 1) % S, hv[(u + S - 1) % S]);
                __builtin_amdgcn_sched_barrier(0);
                __builtin_amdgcn_s_waitcnt(wait_vm((S - 1) * BATCH));
                __builtin_amdgcn_sched_barrier(0);
                const int8_t* at = ring + u * SLOT;
                const i32x4 w0 = *reinterpret_cast<const i32x4*>(at + f0), w1 = *reinterpret_cast<const i32x4*>(at + f1);
                const float sc = *reinterpret_cast<const float*>(at + 2048);
                const bf16x8 a[4] = {codes_bf16(w0[0], w0[1]), codes_bf16(w0[2], w0[3]), codes_bf16(w1[0], w1[1]),
                                     codes_bf16(w1[2], w1[3])};
                auto product = [&](const i32x4 (&h)[2][4], f32x4& to) {
                    f32x4 ph{0, 0, 0, 0}, pl{0, 0, 0, 0};
#pragma unroll
                    for (int f = 0; f < 4; ++f) {
                        ph = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[f], __builtin_bit_cast(bf16x8, h[0][f]), ph, 0, 0, 0);
                        pl = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[f], __builtin_bit_cast(bf16x8, h[1][f]), pl, 0, 0, 0);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        to[e] = fmaf(sc, ph[e] + pl[e], to[e]);
                };
                product(hv[u], acc[0]);
                const int count = __builtin_amdgcn_readfirstlane(act[min(s, nact - 1)][2]);
#pragma unroll
                for (int i = 1; i < TILES; ++i) {
                    if (16 * i < count) {
                        i32x4 more[2][4];
                        load_h(more, pair_offset(min(s, nact - 1), i), b);
                        product(more, acc[i]);
                    }
                }
                __builtin_amdgcn_s_waitcnt(WAIT_LDS);   // the slot's reads are done before it is filled again
                __builtin_amdgcn_sched_barrier(0);
                b += NW;
                if (b >= nib && s < nact) {
                    // leave the expert: a token's four sums lie together, and no two pairs of an
                    // expert share a token
                    const int base = act[s][1];
#pragma unroll
                    for (int i = 0; i < TILES; ++i) {
                        if (16 * i + r < count) {
                            f32x4* to = reinterpret_cast<f32x4*>(&sums[wave][pair_token[base + 16 * i + r]][4 * q]);
                            *to += acc[i];
                        }
                        acc[i] = f32x4{0, 0, 0, 0};
                    }
                    ++s;
                    next(s, b);
                }
            }
        }
        __builtin_amdgcn_s_waitcnt(wait_vm(0));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < g.T * 16; i += NT) {
        const int t = i / 16, n = i % 16;
        float v = sums[0][t][n];
#pragma unroll
        for (int w = 1; w < NW; ++w)
            v += sums[w][t][n];
        const int64_t at = (int64_t)t * K + n0 + n;
        if (g.l.out_f16)
            reinterpret_cast<_Float16*>(g.l.out)[at] = (_Float16)v;
        else
            reinterpret_cast<float*>(g.l.out)[at] = v;
    }
}

template <int TILES>
void launch_up(const Moe& g, uint32_t grid, hipStream_t stream) {
    const dim3 wgs(grid), nt(NT);
    if (g.l.E <= 64)
        moe_up_kernel<TILES, 4><<<wgs, nt, 0, stream>>>(g);
    else if (g.l.E <= 128)
        moe_up_kernel<TILES, 8><<<wgs, nt, 0, stream>>>(g);
    else
        moe_up_kernel<TILES, 32><<<wgs, nt, 0, stream>>>(g);
}

}  // namespace

int64_t moe_workspace(int64_t T, int top_k, int I) {
    const int64_t t = T < MOE_TOKENS ? T : MOE_TOKENS;
    return (int64_t)sizeof(MoeSpace) + t * top_k * I * 4;
}

ql_status launch_moe_router(const void* x, const void* w, float* logits, int64_t T, int64_t E, int64_t K,
                            hipStream_t stream) {
    const _Float16* xp = reinterpret_cast<const _Float16*>(x);
    constexpr int64_t MOST = 16 * 65535;   // tokens of a launch: its grid stays within bounds
    for (int64_t t = 0; t < T; t += MOST) {
        const int64_t n = T - t < MOST ? T - t : MOST;
        moe_router_kernel<<<dim3((uint32_t)((E + 15) / 16), (uint32_t)((n + 15) / 16)), dim3(RW * WAVE), 0, stream>>>(
            xp + t * K, reinterpret_cast<const _Float16*>(w), logits + t * E, n, (int)E, (int)K);
    }
    return launch_status();
}

ql_status launch_moe_e4m3_block(const MoeLayer& l, hipStream_t stream) {
    for (int64_t t = 0; t < l.T; t += MOE_TOKENS) {
        Moe g{};
        g.l = l;
        g.T = (int)(l.T - t < MOE_TOKENS ? l.T - t : MOE_TOKENS);
        g.l.x += t * l.K;
        g.l.logits += t * l.E;
        g.l.out = reinterpret_cast<int8_t*>(l.out) + t * l.K * (l.out_f16 ? 2 : 4);
        g.space = reinterpret_cast<MoeSpace*>(l.ws);
        g.hi = reinterpret_cast<__bf16*>(l.ws + sizeof(MoeSpace));
        g.lo = g.hi + (int64_t)g.T * l.top_k * l.I;
        const int64_t most = (int64_t)(l.E < g.T * l.top_k ? l.E : g.T * l.top_k) * (l.I / 16);
        const uint32_t grid = (uint32_t)(most < cu_count() ? most : cu_count());
        const dim3 down((uint32_t)(l.K / 16)), nt(NT);
        if (g.T <= 16) {
            launch_up<1>(g, grid, stream);
            moe_down_kernel<1><<<down, nt, 0, stream>>>(g);
        } else if (g.T <= 32) {
            launch_up<2>(g, grid, stream);
            moe_down_kernel<2><<<down, nt, 0, stream>>>(g);
        } else {
            launch_up<4>(g, grid, stream);
            moe_down_kernel<4><<<down, nt, 0, stream>>>(g);
        }
    }
    return launch_status();
}

}  // namespace ql
