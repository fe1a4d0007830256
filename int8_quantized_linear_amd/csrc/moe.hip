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
// scale is applied in fp32. h is kept as two bf16 terms for fp16 outputs (16 bits of significand with
// fp32's range: one rounding of relative size 2^-17 that its products see), three for fp32 outputs
// (2^-25; the outputs are then 4e-7 of their norm from 64 bits).
//
// Two pairs of kernels. Where experts have few tokens, a wave copies the blocks of 128 that it takes
// straight into its own ring in LDS, one block ahead, has the other operand's few rows in registers, and
// needs no barrier until the waves' sums are joined. Where they have many, the tokens' operand goes
// through LDS once for eight waves and the codes through registers. launch_experts has the rule. The
// order of every sum is the same in both, whatever the other tokens are.
//
// 5 tokens of 8 large experts (2 of them each, K 4096, I 7168): 99 us, 5.35 TB/s of codes; 64 tokens of 64
// experts (6 each, K 2048, I 1408): 125 us, 4.4 TB/s; one token of 64 (8, K 2048, I 1536): 27 us, of which
// about 13 are the two kernels' fixed part: launch, the routes, a first load's latency, the join.
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
// in order, and cut into units of one expert and up to 16 pairs, the columns of a matrix instruction
// (all of them, and up to 32 in the second kernel, where experts have many).

constexpr int DOWN_COLS = 32;   // output columns of a workgroup of the second kernel
constexpr int DOWN_WIDE_UNIT = 32;   // pairs of a unit there where experts have many
constexpr int MOE_PAIRS = MOE_TOKENS * MOE_TOP_K;
constexpr int MOE_UNITS = MOE_EXPERTS + MOE_PAIRS / 16;   // at most: all experts, each with a last, short unit

struct alignas(8) MoeUnit {
    uint16_t expert, base, count, pad;   // its first pair, its pairs
};

struct Routes {
    MoeUnit units[MOE_UNITS];
    float pair_p[MOE_PAIRS];
    uint8_t pair_token[MOE_PAIRS];
    int nunits;
};
// what only make_routes needs
struct RouteScratch {
    unsigned long long tokens[MOE_EXPERTS];   // bit t: token t takes the expert
    uint16_t base[MOE_EXPERTS];               // first pair of an expert
    uint16_t id[MOE_TOKENS][MOE_TOP_K];       // of a token, MOE_EXPERTS for none
    float p[MOE_TOKENS][MOE_TOP_K];
    uint32_t part[NW];
    __attribute__((aligned(16))) float row[NW][WAVE];   // a wave's token's logits
};

// The workspace: the routes as the second kernel needs them, arrivals at each slice of output columns,
// h's terms ([pairs][I] each), and the parts' sums of the output.
constexpr int MOE_SLICES = 131072 / DOWN_COLS;
struct MoeSpace {
    int nunits;
    int pad[3];
    MoeUnit units[MOE_UNITS];
    uint8_t pair_token[MOE_PAIRS];
    uint32_t arrived[MOE_SLICES];
};

struct Moe {
    MoeLayer l;
    int T;           // tokens of this launch
    int parts;       // workgroups that share a slice of output columns in the second kernel
    MoeSpace* space;
    __bf16* h;       // TERMS planes
    float* sums;     // [parts][T][K]
};

template <int CTRL, class T>
__device__ inline T dpp(T v) {
    return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

// f over the 16 lanes of a row, in every one of them (rotations by 8, 4, 2 and 1 lanes).
template <class T, class F>
__device__ inline T row16(T v, F f) {
    v = f(v, dpp<0x128>(v));
    v = f(v, dpp<0x124>(v));
    v = f(v, dpp<0x122>(v));
    return f(v, dpp<0x121>(v));
}

// Running sum over a wave's lanes, each lane's own included.
__device__ inline uint32_t wave_scan(uint32_t v) {
    auto add = [&](auto ctrl, auto rows) {
        v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, decltype(rows)::value, 0xF, false);
    };
    using std::integral_constant;
    add(integral_constant<int, 0x111>{}, integral_constant<int, 0xF>{});   // shifts by 1, 2, 4 and 8 in rows of 16
    add(integral_constant<int, 0x112>{}, integral_constant<int, 0xF>{});
    add(integral_constant<int, 0x114>{}, integral_constant<int, 0xF>{});
    add(integral_constant<int, 0x118>{}, integral_constant<int, 0xF>{});
    add(integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{});   // lane 15 and 47 to the next row
    add(integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{});   // lane 31 to the upper rows
    return v;
}

// The experts of at most NW tokens, a wave a token and an expert a lane: each logit's rank is the number
// of logits that are larger, of equal ones the lower experts first. One round whatever top_k is: 1 token,
// 64 experts and top_k 8 take the kernel 8.3 us, with the rounds of search_experts 9.6.
__device__ inline void rank_experts(RouteScratch& rs, const Moe& g) {
    const int lane = threadIdx.x & 63, t = threadIdx.x >> 6, E = g.l.E, k = g.l.top_k;
    if (t >= g.T)
        return;
    float* row = rs.row[t];
    const float x = lane < E ? g.l.logits[(int64_t)t * E + lane] : -INFINITY;
    const float v = x == x ? x : -INFINITY;
    row[lane] = v;
    asm volatile("" ::: "memory");   // the wave's LDS operations complete in order
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < (E + 3) / 4; ++j) {
        const f32x4 other = reinterpret_cast<const f32x4*>(row)[j];
#pragma unroll
        for (int n = 0; n < 4; ++n)
            rank += other[n] > v ? 1 : 0;
    }
    // equal logits share a rank: told apart where it matters
    bool equal = false;
    for (int n = 0; n < k; ++n)
        equal = equal || __popcll(__ballot(rank == n && v > -INFINITY)) > 1;
    if (equal)
        for (int j = 0; j < E; ++j)
            rank += row[j] == v && j < lane ? 1 : 0;
    const unsigned long long first = __ballot(rank == 0 && v > -INFINITY);
    const float from = first != 0 ? __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), __builtin_ctzll(first))) : 0.0f;
    const float p = __expf(v - from);
    const bool chosen = rank < k && v > -INFINITY;
    // added in search_experts' order: a token's result is the same among few tokens and among many
    float sum = 0.0f;
    if (g.l.renormalize) {
        for (int n = 0; n < k; ++n) {
            const unsigned long long at = __ballot(rank == n && chosen);
            sum += at != 0 ? __int_as_float(__builtin_amdgcn_readlane(__float_as_int(p), __builtin_ctzll(at))) : 0.0f;
        }
    } else {
        row[lane] = p;
        asm volatile("" ::: "memory");
        for (int n = 0; n < WAVE; n += 16)
            sum += row[n + (lane & 15)];
        sum = row16(sum, [](float a, float b) { return a + b; });
    }
    if (chosen) {
        rs.id[t][rank] = (uint16_t)lane;
        rs.p[t][rank] = p / sum;
        atomicOr(&rs.tokens[lane], 1ull << t);
    }
    const int taken = __popcll(__ballot(chosen));
    if (lane >= taken && lane < k)
        rs.id[t][lane] = MOE_EXPERTS;
}

// The same for any number of tokens: 16 lanes a token, R logits a lane, and top_k rounds of the largest that is
// left. NaN is never taken, nor is -infinity.
template <int R>
__device__ inline void search_experts(RouteScratch& rs, const Moe& g) {
    const int tid = threadIdx.x, E = g.l.E, k = g.l.top_k, l = tid & 15;
    const auto larger = [](float a, float b) { return fmaxf(a, b); };
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
        top = row16(top, larger);
        const float from = top == -INFINITY ? 0.0f : top;
        float all = 0.0f;
        if (!g.l.renormalize) {
#pragma unroll
            for (int r = 0; r < R; ++r)
                all += v[r] == v[r] ? __expf(v[r] - from) : 0.0f;
            all = row16(all, [](float a, float b) { return a + b; });
        }
        float chosen = 0.0f, mine = 0.0f;
        int my_id = MOE_EXPERTS;
        for (int j = 0; j < k; ++j) {
            float best = -INFINITY;
#pragma unroll
            for (int r = 0; r < R; ++r)
                best = fmaxf(best, v[r]);
            best = row16(best, larger);
            int at = MOE_EXPERTS;
#pragma unroll
            for (int r = R - 1; r >= 0; --r)
                at = v[r] == best ? 16 * r + l : at;
            at = row16(at, [](int a, int b) { return min(a, b); });
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
            rs.id[t][l] = (uint16_t)my_id;
            rs.p[t][l] = mine / (g.l.renormalize ? chosen : all);
            if (my_id < MOE_EXPERTS)
                atomicOr(&rs.tokens[my_id], 1ull << t);
        }
    }
}

// At most 16 R experts.
template <int R, int UNIT, int DOWN_UNIT>
__device__ inline void make_routes(Routes& rt, RouteScratch& rs, const Moe& g) {
    const int tid = threadIdx.x, k = g.l.top_k;
    rs.tokens[tid] = 0;
    __syncthreads();
    if (R == 4 && g.T <= NW)
        rank_experts(rs, g);
    else
        search_experts<R>(rs, g);
    __syncthreads();
    // the experts' first pairs and units: a running sum over the experts, one a thread, of pairs, units
    // of DOWN_UNIT and units of UNIT in one number
    static_assert(NT == MOE_EXPERTS, "one expert a thread");
    const int pairs = __popcll(rs.tokens[tid]);
    const uint32_t own = (uint32_t)pairs << 20 | (uint32_t)((pairs + DOWN_UNIT - 1) / DOWN_UNIT) << 10 |
                         (uint32_t)((pairs + UNIT - 1) / UNIT);
    uint32_t sum = wave_scan(own);
    if ((tid & 63) == 63)
        rs.part[tid >> 6] = sum;
    __syncthreads();
    sum -= own;
    uint32_t total = 0;
    for (int w = 0; w < NW; ++w) {
        total += rs.part[w];
        sum += w < tid >> 6 ? rs.part[w] : 0;
    }
    const int base = (int)(sum >> 20);
    rs.base[tid] = (uint16_t)base;
    for (int i = 0; UNIT * i < pairs; ++i)
        rt.units[(sum & 1023) + i] = {(uint16_t)tid, (uint16_t)(base + UNIT * i), (uint16_t)min(UNIT, pairs - UNIT * i), 0};
    if (tid == 0)
        rt.nunits = (int)(total & 1023);
    if (blockIdx.x == 0) {
        for (int i = 0; DOWN_UNIT * i < pairs; ++i)
            g.space->units[(sum >> 10 & 1023) + i] = {(uint16_t)tid, (uint16_t)(base + DOWN_UNIT * i),
                                                      (uint16_t)min(DOWN_UNIT, pairs - DOWN_UNIT * i), 0};
        if (tid == 0)
            g.space->nunits = (int)(total >> 10 & 1023);
    }
    __syncthreads();
    for (int i = tid; i < g.T * k; i += NT) {
        const int t = i / k, e = rs.id[t][i % k];
        if (e < MOE_EXPERTS) {
            const int at = rs.base[e] + __popcll(rs.tokens[e] & ((1ull << t) - 1));
            rt.pair_token[at] = (uint8_t)t;
            rt.pair_p[at] = rs.p[t][i % k];
        }
    }
    __syncthreads();
}

// What the second kernel needs beside the units; by one workgroup.
__device__ inline void publish_routes(const Routes& rt, const Moe& g) {
    if (blockIdx.x != 0)
        return;
    for (int i = threadIdx.x; i < g.T * g.l.top_k; i += NT)
        g.space->pair_token[i] = rt.pair_token[i];
    for (int i = threadIdx.x; i < g.l.K / DOWN_COLS; i += NT)
        g.space->arrived[i] = 0;
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

// Four columns of a pair's h = p silu(gate) up, in TERMS bf16 terms.
template <int TERMS>
__device__ inline void write_h(const Moe& g, int pair, int col, float p, f32x4 gate, f32x4 up) {
    float h[4];
#pragma unroll
    for (int c = 0; c < 4; ++c)
        h[c] = p * activation<ACT_SILU>(gate[c]) * up[c];
#pragma unroll
    for (int k = 0; k < TERMS; ++k) {
        bf16x4 v;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            v[c] = (__bf16)h[c];
            h[c] -= (float)v[c];
        }
        *reinterpret_cast<bf16x4*>(g.h + ((int64_t)k * g.T * g.l.top_k + pair) * g.l.I + col) = v;
    }
}

// Four columns of a token's result.
__device__ inline void write_out(const Moe& g, int t, int col, f32x4 v) {
    typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
    const int64_t at = (int64_t)t * g.l.K + col;
    if (g.l.out_f16)
        *reinterpret_cast<f16x4*>(reinterpret_cast<_Float16*>(g.l.out) + at) =
            f16x4{(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
    else
        *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(g.l.out) + at) = v;
}

// The parts' sums go past the XCDs' caches, as the parts may be on different ones: stores and loads of
// device scope (sc1), the stores done before the arrival is counted. Whoever counts the last arrival
// adds the parts in order. Nobody waits for another.
constexpr int DEVICE = 16;

__device__ inline bool last_to_arrive(const Moe& g, int slice, int parts, int& last) {
    __builtin_amdgcn_s_waitcnt(wait_vm(0));
    __syncthreads();
    if (threadIdx.x == 0)
        last = __hip_atomic_fetch_add(&g.space->arrived[slice], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
               (uint32_t)parts - 1;
    __syncthreads();
    return last != 0;
}

__device__ inline f32x4 part_sums(const Moe& g, int part, int t, int col) {
    const __amdgpu_buffer_rsrc_t from = buffer_of(g.sums + (int64_t)part * g.T * g.l.K, g.T * g.l.K * 4);
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(from, (t * g.l.K + col) * 4, 0, DEVICE));
}

// ------------------------------------------------------------------------ the gated products
//
// A task is a unit and 16 columns of h: 16 rows of W1 and 16 of W3 against the unit's tokens. A workgroup
// takes every gridDim-th task; its waves split K, wave w taking the blocks w, w + 8, ... of every task. The
// wave's items (task, block) make one sequence, so the next task's first loads are in flight while a task's
// sums are joined. Codes go through the wave's ring of S slots in LDS; the tokens' rows of x come from L2
// into registers, as far ahead. W is the first operand: a lane's sums belong to one token (lane & 15) and
// four columns of h.

// (Two slots; with three, one token of 64 experts takes 29.6 us instead of 27.3, 64 tokens 126 instead of
// 127: eight waves have enough loads under way, and more start later.)
constexpr int UP_S = 2, UP_SLOT = 4096 + 256;

// (One LDS variable a kernel: with several the compiler tells the copies into them apart and waits for
// those into the rings, all of them, before any read of a ring.)
struct UpShared {
    int8_t rings[NW * UP_S * UP_SLOT];   // RouteScratch before the copies start
    f32x4 red[NW][2][WAVE];
    Routes rt;
};

template <int R, int TERMS, bool WHOLE>
__global__ __launch_bounds__(NT) void moe_up_kernel(Moe g) {
    constexpr int S = UP_S, COPIES = 5 + 4;
    __shared__ __attribute__((aligned(1024))) UpShared sh;
    static_assert(sizeof(RouteScratch) <= sizeof(sh.rings), "the routes are made before the rings are used");
    Routes& rt = sh.rt;
    auto& red = sh.red;
    make_routes<R, 16, 16>(rt, *reinterpret_cast<RouteScratch*>(sh.rings), g);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4;
    const int K = g.l.K, I = g.l.I, nunits = __builtin_amdgcn_readfirstlane(rt.nunits);
    publish_routes(rt, g);
    const int nkb = (K + QB - 1) / QB, cols = I / 16, tasks = nunits * cols;
    const int J = (nkb + NW - 1) / NW;                       // a wave's blocks of a task
    const int first = blockIdx.x, G = gridDim.x;
    if (first >= tasks)
        return;

    int8_t* ring = sh.rings + wave * S * UP_SLOT;
    const int64_t blocks13 = e4m3_blocks(2 * (int64_t)I);
    const __amdgpu_buffer_rsrc_t rx = buffer_of(g.l.x, g.T * K * 2);
    const int row = lane >> 3, c0 = copy_chunk128(lane, 0), c1 = copy_chunk128(lane, 1);
    const int far = 0x40000000;

    // the item that is fetched next
    struct {
        int task, j;
        __amdgpu_buffer_rsrc_t gate, up;
        const float* scale;
        int xoff;
    } nx;
    auto enter = [&](int task) {
        nx.task = task;
        nx.j = 0;
        const int a = min(task, tasks - 1), i0 = (a % cols) * 16;
        const MoeUnit u = rt.units[a / cols];
        const int e = __builtin_amdgcn_readfirstlane(u.expert);
        const int size = task < tasks ? 16 * K : 0;
        const uint8_t* w = g.l.w13 + ((int64_t)e * 2 * I + i0) * K;
        nx.gate = buffer_of(w, size);
        nx.up = buffer_of(w + (int64_t)I * K, size);
        nx.scale = g.l.s13 + (e * blocks13 + (i0 + (lane < 32 ? 0 : I)) / QB) * nkb;
        // columns past the tokens repeat the last one
        nx.xoff = (rt.pair_token[u.base + min(r, u.count - 1)] * K + 16 * q) * 2;
    };
    auto fetch = [&](int slot, i32x4 (&x)[4]) {
        int8_t* to = ring + slot * UP_SLOT;
        const int b = wave + NW * nx.j, left = K - b * QB;   // blocks past the end come as zeros
        const int cut0 = 16 * c0 < left ? 0 : far, cut1 = 16 * c1 < left ? 0 : far;
        const int o0 = row * K + 16 * c0 + b * QB, o1 = (row + 8) * K + 16 * c1 + b * QB;
        buffer_to_lds16<WHOLE ? 2 : 0>(nx.gate, o0 | cut0, 0, to);
        buffer_to_lds16<WHOLE ? 2 : 0>(nx.gate, o1 | cut1, 0, to + 1024);
        buffer_to_lds16<WHOLE ? 2 : 0>(nx.up, o0 | cut0, 0, to + 2048);
        buffer_to_lds16<WHOLE ? 2 : 0>(nx.up, o1 | cut1, 0, to + 3 * 1024);
        global_to_lds4(nx.scale + min(b, nkb - 1), to + 4096);
        // past K the codes are zeros, and x anything finite
        const int bx = min(b, nkb - 1) * QB, half = left > 64 ? 128 : 0;
#pragma unroll
        for (int f = 0; f < 4; ++f)
            x[f] = __builtin_amdgcn_raw_buffer_load_b128(rx, nx.xoff + 16 * (f & 1) + (f >> 1) * half, 2 * bx, 0);
        asm volatile("" ::: "memory");   // no load may sink past the waits that count it
        if (++nx.j == J)
            enter(nx.task + G);
    };

    f32x4 acc[2];
    auto clear = [&]() { acc[0] = acc[1] = f32x4{0, 0, 0, 0}; };
    clear();
    i32x4 xv[S][4];
    enter(first);
#pragma unroll
    for (int s = 0; s < S - 1; ++s)
        fetch(s, xv[s]);
    const int f0 = r * QB + ((q ^ swizzle128(r)) << 4), f1 = r * QB + (((q + 4) ^ swizzle128(r)) << 4);
    const int items = ((tasks - first + G - 1) / G) * J;
    int task = first, j = 0;
    // in rounds of S items, the last one filled up with zeros
    for (int it = 0; it < items; it += S) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            fetch((s + S - 1) % S, xv[(s + S - 1) % S]);
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(wait_vm((S - 1) * COPIES));
            __builtin_amdgcn_sched_barrier(0);
            const int8_t* at = ring + s * UP_SLOT;
            const i32x4 g0 = *reinterpret_cast<const i32x4*>(at + f0), g1 = *reinterpret_cast<const i32x4*>(at + f1);
            const i32x4 u0 = *reinterpret_cast<const i32x4*>(at + 2048 + f0);
            const i32x4 u1 = *reinterpret_cast<const i32x4*>(at + 2048 + f1);
            const float sg = *reinterpret_cast<const float*>(at + 4096);
            const float su = *reinterpret_cast<const float*>(at + 4096 + 128);
            const f16x8 ga[4] = {codes_f16(g0[0], g0[1]), codes_f16(g0[2], g0[3]), codes_f16(g1[0], g1[1]), codes_f16(g1[2], g1[3])};
            const f16x8 ua[4] = {codes_f16(u0[0], u0[1]), codes_f16(u0[2], u0[3]), codes_f16(u1[0], u1[1]), codes_f16(u1[2], u1[3])};
            f32x4 pg{0, 0, 0, 0}, pu{0, 0, 0, 0};
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const f16x8 x = __builtin_bit_cast(f16x8, xv[s][f]);
                pg = __builtin_amdgcn_mfma_f32_16x16x32_f16(ga[f], x, pg, 0, 0, 0);
                pu = __builtin_amdgcn_mfma_f32_16x16x32_f16(ua[f], x, pu, 0, 0, 0);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                acc[0][e] = fmaf(sg, pg[e], acc[0][e]);
                acc[1][e] = fmaf(su, pu[e], acc[1][e]);
            }
            __builtin_amdgcn_s_waitcnt(WAIT_LDS);   // the slot's reads are done before it is filled again
            __builtin_amdgcn_sched_barrier(0);
            if (++j == J && task < tasks) {
                // the task's sums of all waves, joined by one
                red[wave][0][lane] = acc[0];
                red[wave][1][lane] = acc[1];
                clear();
                barrier_lds();
                if (wave == 0) {
                    const MoeUnit u = rt.units[task / cols];
                    f32x4 gs = red[0][0][lane], us = red[0][1][lane];
#pragma unroll
                    for (int w = 1; w < NW; ++w) {
                        gs += red[w][0][lane];
                        us += red[w][1][lane];
                    }
                    if (r < u.count)
                        write_h<TERMS>(g, u.base + r, (task % cols) * 16 + 4 * q, rt.pair_p[u.base + r], gs, us);
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
// A workgroup owns 32 columns of the output and one of `parts` shares of I. Block b of expert e is
// number (e * blocks + b) % (parts * 8)'s, part by part and wave by wave: neighbouring waves read
// neighbouring 128 bytes, all have about as many blocks, and who adds what to a token's sums does not
// depend on the other tokens' experts. A wave's blocks of all units make one sequence. Codes go through
// its ring of S slots in LDS; h's few rows come from L2 into registers, as far ahead (in LDS they would
// take twice the codes' space). A wave adds a unit's products to its own sums [token][32] in LDS; the
// waves' sums are added at the end, and the parts' by the workgroup that comes last.

constexpr int DOWN_S = 2, DOWN_SLOT = DOWN_COLS * QB + 256;

template <int TOKENS>
struct DownShared {
    int8_t rings[NW * DOWN_S * DOWN_SLOT];
    float sums[NW][TOKENS][DOWN_COLS];
    MoeUnit units[MOE_UNITS];
    uint8_t pair_token[TOKENS * MOE_TOP_K];
    int last;
};

template <int TERMS, int TOKENS, bool WHOLE>
__global__ __launch_bounds__(NT) void moe_down_kernel(Moe g) {
    constexpr int COPIES = DOWN_COLS / 8 + 1 + TERMS * 4;
    constexpr int S = DOWN_S;
    __shared__ __attribute__((aligned(1024))) DownShared<TOKENS> sh;
    auto& sums = sh.sums;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4;
    const int slices = g.l.K / DOWN_COLS, slice = blockIdx.x % slices, part = blockIdx.x / slices;
    const int K = g.l.K, I = g.l.I, n0 = slice * DOWN_COLS;
    const int units_load = g.space->nunits;
    // (as many units as there can be, so that the loads do not wait for the number)
    const int most = g.T * g.l.top_k < MOE_UNITS ? g.T * g.l.top_k : MOE_UNITS;
    for (int i = threadIdx.x; i < most; i += NT)
        *reinterpret_cast<u32x2*>(&sh.units[i]) = *reinterpret_cast<const u32x2*>(&g.space->units[i]);
    for (int i = threadIdx.x; 4 * i < g.T * g.l.top_k; i += NT)
        reinterpret_cast<uint32_t*>(sh.pair_token)[i] = reinterpret_cast<const uint32_t*>(g.space->pair_token)[i];
    for (int i = threadIdx.x; i < NW * TOKENS * DOWN_COLS / 4; i += NT)
        reinterpret_cast<f32x4*>(sums)[i] = f32x4{0, 0, 0, 0};
    const int nunits = __builtin_amdgcn_readfirstlane(units_load);
    __syncthreads();
    const int nib = (I + QB - 1) / QB, share = part * NW + wave, shares = g.parts * NW;

    int8_t* ring = sh.rings + wave * S * DOWN_SLOT;
    const int64_t blocks2 = e4m3_blocks(K);
    const int plane = g.T * g.l.top_k * I * 2;
    __amdgpu_buffer_rsrc_t rh[TERMS];
#pragma unroll
    for (int k = 0; k < TERMS; ++k)
        rh[k] = buffer_of(reinterpret_cast<const int8_t*>(g.h) + (int64_t)k * plane, plane);
    const int row = lane >> 3, c0 = copy_chunk128(lane, 0), c1 = copy_chunk128(lane, 1);
    const int far = 0x40000000;

    // What is fetched next: block b of the unit that lane `at` of the window holds. A window is 64
    // units, one a lane, and `have` says in which of them the wave has a block.
    struct {
        int window, at, b, hoff;
        unsigned long long have;
        int expert, pairs, first;   // of the lane's unit: base and count << 16, the wave's first block
        __amdgpu_buffer_rsrc_t w;
        const float* scale;
    } nx;
    auto open_window = [&](int w) {
        nx.window = w;
        const int n = min(w + lane, nunits - 1);
        const MoeUnit u = sh.units[n];
        nx.expert = u.expert;
        nx.pairs = u.base | u.count << 16;
        nx.first = (share - u.expert * nib) & (shares - 1);
        nx.have = __ballot(w + lane < nunits && nx.first < nib);
    };
    auto enter = [&]() {   // the next unit that has a block, if any is left
        while (nx.have == 0 && nx.window + 64 < nunits)
            open_window(nx.window + 64);
        if (nx.have == 0) {
            nx.at = -1;
            nx.w = buffer_of(g.l.w2, 0);
            return;
        }
        nx.at = __builtin_ctzll(nx.have);
        nx.have &= nx.have - 1;
        nx.b = __builtin_amdgcn_readlane(nx.first, nx.at);
        const int e = __builtin_amdgcn_readlane(nx.expert, nx.at), pairs = __builtin_amdgcn_readlane(nx.pairs, nx.at);
        nx.w = buffer_of(g.l.w2 + ((int64_t)e * K + n0) * I, DOWN_COLS * I);
        nx.scale = g.l.s2 + (e * blocks2 + n0 / QB) * nib;
        // columns past the unit's pairs repeat the last one
        nx.hoff = (((pairs & 0xFFFF) + min(r, (pairs >> 16) - 1)) * I + 16 * q) * 2;
    };
    // an item's unit as pairs above, with bit 31 where it is the wave's last block of the unit; -1 past
    // the end
    auto fetch = [&](int slot, i32x4 (&h)[TERMS][4]) {
        int8_t* to = ring + slot * DOWN_SLOT;
        const int left = I - nx.b * QB;
        const int cut0 = 16 * c0 < left ? 0 : far, cut1 = 16 * c1 < left ? 0 : far;
        const int o0 = row * I + 16 * c0 + nx.b * QB, o1 = (row + 8) * I + 16 * c1 + nx.b * QB;
#pragma unroll
        for (int i = 0; i < DOWN_COLS / 16; ++i) {
            buffer_to_lds16<WHOLE ? 2 : 0>(nx.w, (o0 + 16 * i * I) | cut0, 0, to + 2048 * i);
            buffer_to_lds16<WHOLE ? 2 : 0>(nx.w, (o1 + 16 * i * I) | cut1, 0, to + 2048 * i + 1024);
        }
        global_to_lds4(nx.scale + nx.b, to + DOWN_COLS * QB);
        const int half = left > 64 ? 128 : 0;   // past I the codes are zeros, and h anything finite
#pragma unroll
        for (int k = 0; k < TERMS; ++k)
#pragma unroll
            for (int f = 0; f < 4; ++f)
                h[k][f] = __builtin_amdgcn_raw_buffer_load_b128(rh[k], nx.hoff + 16 * (f & 1) + (f >> 1) * half, 2 * nx.b * QB, 0);
        asm volatile("" ::: "memory");   // no load may sink past the waits that count it
        if (nx.at < 0)
            return -1;
        int info = __builtin_amdgcn_readlane(nx.pairs, nx.at);
        nx.b += shares;
        if (nx.b >= nib) {
            info |= (int)0x80000000;
            nx.b = 0;
            enter();
        }
        return info;
    };

    f32x4 acc[DOWN_COLS / 16];
#pragma unroll
    for (int i = 0; i < DOWN_COLS / 16; ++i)
        acc[i] = f32x4{0, 0, 0, 0};
    if (nunits > 0) {
        i32x4 hv[S][TERMS][4];
        int info[S];
        nx.scale = g.l.s2;
        nx.b = nx.hoff = 0;
        open_window(0);
        enter();
#pragma unroll
        for (int i = 0; i < S - 1; ++i)
            info[i] = fetch(i, hv[i]);
        const int f0 = r * QB + ((q ^ swizzle128(r)) << 4), f1 = r * QB + (((q + 4) ^ swizzle128(r)) << 4);
        // in rounds of S items, the last one filled up with zeros
        while (info[0] != -1) {
#pragma unroll
            for (int u = 0; u < S; ++u) {
                info[(u + S - 1) % S] = fetch((u + S - 1) % S, hv[(u + S - 1) % S]);
                __builtin_amdgcn_sched_barrier(0);
                __builtin_amdgcn_s_waitcnt(wait_vm((S - 1) * COPIES));
                __builtin_amdgcn_sched_barrier(0);
                const int8_t* at = ring + u * DOWN_SLOT;
                const float sc = *reinterpret_cast<const float*>(at + DOWN_COLS * QB);
#pragma unroll
                for (int i = 0; i < DOWN_COLS / 16; ++i) {
                    const i32x4 w0 = *reinterpret_cast<const i32x4*>(at + 2048 * i + f0);
                    const i32x4 w1 = *reinterpret_cast<const i32x4*>(at + 2048 * i + f1);
                    const bf16x8 a[4] = {codes_bf16(w0[0], w0[1]), codes_bf16(w0[2], w0[3]), codes_bf16(w1[0], w1[1]),
                                         codes_bf16(w1[2], w1[3])};
                    f32x4 p[TERMS];
#pragma unroll
                    for (int k = 0; k < TERMS; ++k) {
                        p[k] = f32x4{0, 0, 0, 0};
#pragma unroll
                        for (int f = 0; f < 4; ++f)
                            p[k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[f], __builtin_bit_cast(bf16x8, hv[u][k][f]), p[k],
                                                                           0, 0, 0);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float v = p[TERMS - 1][e];
#pragma unroll
                        for (int k = TERMS - 2; k >= 0; --k)
                            v += p[k][e];
                        acc[i][e] = fmaf(sc, v, acc[i][e]);
                    }
                }
                __builtin_amdgcn_s_waitcnt(WAIT_LDS);   // the slot's reads are done before it is filled again
                __builtin_amdgcn_sched_barrier(0);
                if (info[u] < -1) {
                    // leave the unit: a token's four sums lie together, and no two pairs of a unit share a
                    // token
                    const int base = info[u] & 0xFFFF, count = info[u] >> 16 & 0x7FFF;
                    if (r < count) {
                        float* to = sums[wave][sh.pair_token[base + r]] + 4 * q;
#pragma unroll
                        for (int i = 0; i < DOWN_COLS / 16; ++i)
                            *reinterpret_cast<f32x4*>(to + 16 * i) += acc[i];
                    }
#pragma unroll
                    for (int i = 0; i < DOWN_COLS / 16; ++i)
                        acc[i] = f32x4{0, 0, 0, 0};
                }
            }
        }
        __builtin_amdgcn_s_waitcnt(wait_vm(0));
    }
    __syncthreads();
    // four columns of a token a thread
    constexpr int C4 = DOWN_COLS / 4;
    auto joined = [&](int i) {
        f32x4 v[NW];
#pragma unroll
        for (int w = 0; w < NW; ++w)
            v[w] = *reinterpret_cast<const f32x4*>(&sums[w][i / C4][i % C4 * 4]);
        return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    };
    if (g.parts == 1) {
        for (int i = threadIdx.x; i < g.T * C4; i += NT)
            write_out(g, i / C4, n0 + i % C4 * 4, joined(i));
        return;
    }
    const __amdgpu_buffer_rsrc_t mine = buffer_of(g.sums + (int64_t)part * g.T * K, g.T * K * 4);
    for (int i = threadIdx.x; i < g.T * C4; i += NT)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, joined(i)), mine,
                                               ((i / C4) * K + n0 + i % C4 * 4) * 4, 0, DEVICE);
    if (!last_to_arrive(g, slice, g.parts, sh.last))
        return;
    for (int i = threadIdx.x; i < g.T * C4; i += NT) {
        f32x4 v{0, 0, 0, 0};
        for (int p = 0; p < g.parts; ++p)
            v += part_sums(g, p, i / C4, n0 + i % C4 * 4);
        write_out(g, i / C4, n0 + i % C4 * 4, v);
    }
}

// ------------------------------------------------------------------- experts with many tokens
//
// The same two products where an expert has many tokens: the tokens' operand (x, or h's terms) then
// outweighs the codes in what comes from L2, so it goes through an LDS ring that a workgroup's eight
// waves share, and each wave has 16 columns of the output for itself, its codes loaded into registers.
// One barrier a block of 128: it shows that all waves' copies of this block have landed and that all
// have read the one before, whose slot is then filled. Sums are made in the order of the kernels
// above, so a token's result does not depend on which ones are taken: share by share of the blocks,
// each share's sum from zero, and the shares' sums added as there.

constexpr int WIDE_COLS = 16 * NW;   // columns of a workgroup: one block's scale serves them all

// 16 rows of 128 codes into registers, whole lines a load (half lines, as the matrix instructions take
// them, cost the first kernel 126 us where these take 100 at 64 tokens of 8 experts, K 4096, I 7168):
// lane l has a chunk of row l / 8 and of row l / 8 + 8. They change lanes in a few KB of LDS.
__device__ inline void load_codes(i32x4* w, __amdgpu_buffer_rsrc_t rows, int stride, int k, int left) {
    const int lane = threadIdx.x & 63, c0 = copy_chunk128(lane, 0), c1 = copy_chunk128(lane, 1), far = 0x40000000;
    const int o0 = 16 * c0 < left ? (lane >> 3) * stride + 16 * c0 + k : far;
    const int o1 = 16 * c1 < left ? ((lane >> 3) + 8) * stride + 16 * c1 + k : far;
    if (whole_lines(stride)) {
        w[0] = __builtin_amdgcn_raw_buffer_load_b128(rows, o0, 0, 2);
        w[1] = __builtin_amdgcn_raw_buffer_load_b128(rows, o1, 0, 2);
    } else {
        w[0] = __builtin_amdgcn_raw_buffer_load_b128(rows, o0, 0, 0);
        w[1] = __builtin_amdgcn_raw_buffer_load_b128(rows, o1, 0, 0);
    }
}

// What lane (r, q) multiplies: bytes 16 q + 64 j of row r. (A wave's LDS operations complete in order.)
__device__ inline void turn_codes(int8_t* lds, const i32x4* w, i32x4 (&out)[2]) {
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    i32x4* at = reinterpret_cast<i32x4*>(lds);
    at[lane] = w[0];
    at[WAVE + lane] = w[1];
    asm volatile("" ::: "memory");
    out[0] = at[8 * r + (q ^ swizzle128(r))];
    out[1] = at[8 * r + ((q + 4) ^ swizzle128(r))];
    asm volatile("" ::: "memory");
}

// The gated products. A task is an expert and 128 columns of h; a unit is all of its pairs.
// (Three stages of the ring instead of four, and 64 columns with two workgroups a CU: 64 tokens, 4 of 16
// experts, K and I 2048, 63.5 and 67.0 us instead of 62.5.)
constexpr int UPW_S = 4, UPW_TILES = MOE_TOKENS / 16, UPW_SLOT = MOE_TOKENS * 2 * QB;

struct UpWideShared {
    int8_t ring[UPW_S * UPW_SLOT];   // RouteScratch before the copies start
    int8_t turn[NW][4096];
    Routes rt;
};

template <int R, int TERMS>
__global__ __launch_bounds__(NT) void moe_up_wide_kernel(Moe g) {
    constexpr int S = UPW_S, TILES = UPW_TILES, X = UPW_TILES * 4 / NW, COPIES = X + 4 + 1;
    __shared__ __attribute__((aligned(1024))) UpWideShared sh;
    static_assert(sizeof(RouteScratch) <= sizeof(sh.ring), "the routes are made before the ring is used");
    Routes& rt = sh.rt;
    make_routes<R, MOE_TOKENS, DOWN_WIDE_UNIT>(rt, *reinterpret_cast<RouteScratch*>(sh.ring), g);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4;
    const int K = g.l.K, I = g.l.I, nunits = __builtin_amdgcn_readfirstlane(rt.nunits);
    publish_routes(rt, g);
    const int nkb = (K + QB - 1) / QB, slabs = (I + WIDE_COLS - 1) / WIDE_COLS, tasks = nunits * slabs;
    const int G = gridDim.x, first = blockIdx.x;
    if (first >= tasks)
        return;
    const int far = 0x40000000;
    const int64_t blocks13 = e4m3_blocks(2 * I);
    const __amdgpu_buffer_rsrc_t rx = buffer_of(g.l.x, g.T * K * 2);
    const int xrow = 4 * wave + (lane >> 4), xchunk = (lane & 15) ^ (xrow & 15);   // of a copy of 4 rows

    // a task's blocks share by share: w, w + NW, ..., as the waves of the narrow kernel have them
    const auto next_block = [&](int b) {
        const int share = b & (NW - 1);
        return b + NW < nkb ? b + NW : share + 1 < min(nkb, NW) ? share + 1 : 0;
    };

    struct {
        int task, b;
        __amdgpu_buffer_rsrc_t gate, up;
        const float* scale;
        int xoff[X];
    } nx;
    auto enter = [&](int task) {
        nx.task = task;
        nx.b = 0;
        const int a = min(task, tasks - 1), i0 = (a % slabs) * WIDE_COLS + 16 * wave;
        const MoeUnit u = rt.units[a / slabs];
        const int e = __builtin_amdgcn_readfirstlane(u.expert);
        const int size = task < tasks && i0 < I ? 16 * K : 0;
        const uint8_t* w = g.l.w13 + ((int64_t)e * 2 * I + min(i0, I - 16)) * K;
        nx.gate = buffer_of(w, size);
        nx.up = buffer_of(w + (int64_t)I * K, size);
        nx.scale = g.l.s13 + (e * blocks13 + (min(i0, I - 16) + (lane < 32 ? 0 : I)) / QB) * nkb;
#pragma unroll
        for (int i = 0; i < X; ++i) {
            const int n = xrow + 4 * NW * i;
            nx.xoff[i] = n < u.count && task < tasks ? rt.pair_token[u.base + min(n, u.count - 1)] * K * 2 + 16 * xchunk : far;
        }
    };
    auto fetch = [&](int slot, i32x4 (&w)[4], float& scale) {
        int8_t* to = sh.ring + slot * UPW_SLOT + 1024 * wave;
        const int left = K - nx.b * QB, cut = 8 * xchunk < left ? 0 : far;   // zeros past K, and past the tokens
#pragma unroll
        for (int i = 0; i < X; ++i)
            buffer_to_lds16<0>(rx, (nx.xoff[i] + 2 * QB * nx.b) | cut, 0, to + 1024 * NW * i);
        load_codes(w, nx.gate, K, nx.b * QB, left);
        load_codes(w + 2, nx.up, K, nx.b * QB, left);
        scale = nx.scale[nx.b];
        asm volatile("" ::: "memory");   // no load may sink past the waits that count it
        nx.b = next_block(nx.b);
        if (nx.b == 0)
            enter(nx.task + G);
    };

    f32x4 acc[TILES][2], sum[TILES][2];
    auto clear = [&](f32x4 (&v)[TILES][2]) {
#pragma unroll
        for (int i = 0; i < TILES; ++i)
            v[i][0] = v[i][1] = f32x4{0, 0, 0, 0};
    };
    clear(acc);
    clear(sum);
    i32x4 wv[S][4];
    float sv[S];
    enter(first);
#pragma unroll
    for (int s = 0; s < S - 1; ++s)
        fetch(s, wv[s], sv[s]);
    int at[4];   // of a fragment in a tile's rows
#pragma unroll
    for (int f = 0; f < 4; ++f)
        at[f] = r * 2 * QB + 16 * ((8 * (f >> 1) + 2 * q + (f & 1)) ^ r);
    const int items = ((tasks - first + G - 1) / G) * nkb;
    int task = first, blk = 0, count = rt.units[task / slabs].count;
    for (int it = 0; it < items; it += S) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            __builtin_amdgcn_s_waitcnt(wait_vm((S - 2) * COPIES));
            barrier_lds();
            fetch((s + S - 1) % S, wv[(s + S - 1) % S], sv[(s + S - 1) % S]);
            __builtin_amdgcn_sched_barrier(0);
            const int8_t* xs = sh.ring + s * UPW_SLOT;
            i32x4 wg[2], wu[2];
            turn_codes(sh.turn[wave], wv[s], wg);
            turn_codes(sh.turn[wave] + 2048, wv[s] + 2, wu);
            const f16x8 ga[4] = {codes_f16(wg[0][0], wg[0][1]), codes_f16(wg[0][2], wg[0][3]), codes_f16(wg[1][0], wg[1][1]),
                                 codes_f16(wg[1][2], wg[1][3])};
            const f16x8 ua[4] = {codes_f16(wu[0][0], wu[0][1]), codes_f16(wu[0][2], wu[0][3]), codes_f16(wu[1][0], wu[1][1]),
                                 codes_f16(wu[1][2], wu[1][3])};
            const float sg = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sv[s]), 0));
            const float su = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sv[s]), 32));
#pragma unroll
            for (int i = 0; i < TILES; ++i) {
                if (16 * i < count) {
                    f32x4 pg{0, 0, 0, 0}, pu{0, 0, 0, 0};
#pragma unroll
                    for (int f = 0; f < 4; ++f) {
                        const f16x8 x = *reinterpret_cast<const f16x8*>(xs + 16 * 2 * QB * i + at[f]);
                        pg = __builtin_amdgcn_mfma_f32_16x16x32_f16(ga[f], x, pg, 0, 0, 0);
                        pu = __builtin_amdgcn_mfma_f32_16x16x32_f16(ua[f], x, pu, 0, 0, 0);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        acc[i][0][e] = fmaf(sg, pg[e], acc[i][0][e]);
                        acc[i][1][e] = fmaf(su, pu[e], acc[i][1][e]);
                    }
                }
            }
            if (blk + NW >= nkb) {   // the share's last block
#pragma unroll
                for (int i = 0; i < TILES; ++i) {
                    sum[i][0] += acc[i][0];
                    sum[i][1] += acc[i][1];
                }
                clear(acc);
            }
            blk = next_block(blk);
            if (blk == 0) {
                const int i0 = (task % slabs) * WIDE_COLS + 16 * wave;
                if (task < tasks && i0 < I) {
                    const MoeUnit u = rt.units[task / slabs];
#pragma unroll
                    for (int i = 0; i < TILES; ++i) {
                        const int n = 16 * i + r;
                        if (n < u.count)
                            write_h<TERMS>(g, u.base + n, i0 + 4 * q, rt.pair_p[u.base + n], sum[i][0], sum[i][1]);
                    }
                }
                clear(sum);
                task += G;
                count = rt.units[min(task, tasks - 1) / slabs].count;
            }
        }
    }
    __builtin_amdgcn_s_waitcnt(wait_vm(0));
}

// The sums over experts. A workgroup owns 128 columns of the output and two neighbouring shares of I
// of the narrow kernel's parts * NW: first all blocks of the one, then of the other, each into its own
// sums in LDS.
constexpr int DOWN_WIDE_TILES = DOWN_WIDE_UNIT / 16, WIDE_PARTS = NW / 2;   // workgroups for one of the narrow kernel's parts

template <int TERMS>
struct DownWideShared {
    static constexpr int S = TERMS == 2 ? 4 : 3, SLOT = TERMS * DOWN_WIDE_UNIT * 2 * QB;
    int8_t ring[S * SLOT];
    int8_t turn[NW][2048];
    float sums[2][MOE_TOKENS][WIDE_COLS + 4];   // rows 16 bytes apart in the banks
    MoeUnit units[MOE_UNITS];
    uint8_t pair_token[MOE_PAIRS];
    int last;
};

template <int TERMS>
__global__ __launch_bounds__(NT) void moe_down_wide_kernel(Moe g) {
    constexpr int S = DownWideShared<TERMS>::S, SLOT = DownWideShared<TERMS>::SLOT, COPIES = TERMS + 2 + 1;
    constexpr int TILES = DOWN_WIDE_TILES, PLANE = DOWN_WIDE_UNIT * 2 * QB;
    __shared__ __attribute__((aligned(1024))) DownWideShared<TERMS> sh;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4;
    const int K = g.l.K, I = g.l.I, slices = (K + WIDE_COLS - 1) / WIDE_COLS;
    const int slice = blockIdx.x % slices, part = blockIdx.x / slices, n0 = slice * WIDE_COLS, col = n0 + 16 * wave;
    const int units_load = g.space->nunits;
    const int most = min(g.T * g.l.top_k, MOE_UNITS);
    for (int i = threadIdx.x; i < most; i += NT)
        *reinterpret_cast<u32x2*>(&sh.units[i]) = *reinterpret_cast<const u32x2*>(&g.space->units[i]);
    for (int i = threadIdx.x; 4 * i < g.T * g.l.top_k; i += NT)
        reinterpret_cast<uint32_t*>(sh.pair_token)[i] = reinterpret_cast<const uint32_t*>(g.space->pair_token)[i];
    for (int i = threadIdx.x; i < (int)(sizeof(sh.sums) / 16); i += NT)
        reinterpret_cast<f32x4*>(sh.sums)[i] = f32x4{0, 0, 0, 0};
    const int nunits = __builtin_amdgcn_readfirstlane(units_load);
    __syncthreads();
    const int nib = (I + QB - 1) / QB, shares = g.parts * NW, far = 0x40000000;
    const int64_t blocks2 = e4m3_blocks(K);
    const int plane = g.T * g.l.top_k * I * 2;
    const __amdgpu_buffer_rsrc_t rh = buffer_of(g.h, TERMS * plane);
    const int hrow = 4 * wave + (lane >> 4), hchunk = (lane & 15) ^ (hrow & 15);

    // What is fetched next, as in the narrow kernel, for share 2 part + turn.
    struct {
        int turn, window, at, b, hoff;
        unsigned long long have;
        int expert, pairs, first;
        __amdgpu_buffer_rsrc_t w, scale;
    } nx;
    auto open_window = [&](int w) {
        nx.window = w;
        const MoeUnit u = sh.units[min(w + lane, nunits - 1)];
        nx.expert = u.expert;
        nx.pairs = u.base | u.count << 16;
        nx.first = (2 * part + nx.turn - u.expert * nib) & (shares - 1);
        nx.have = __ballot(w + lane < nunits && nx.first < nib);
    };
    auto enter = [&]() {
        while (nx.have == 0) {
            if (nx.window + 64 < nunits) {
                open_window(nx.window + 64);
            } else if (nx.turn == 0) {
                nx.turn = 1;
                open_window(0);
            } else {
                nx.at = -1;
                nx.w = nx.scale = buffer_of(g.l.w2, 0);
                nx.hoff = far;
                return;
            }
        }
        nx.at = __builtin_ctzll(nx.have);
        nx.have &= nx.have - 1;
        nx.b = __builtin_amdgcn_readlane(nx.first, nx.at);
        const int e = __builtin_amdgcn_readlane(nx.expert, nx.at), pairs = __builtin_amdgcn_readlane(nx.pairs, nx.at);
        nx.w = buffer_of(g.l.w2 + ((int64_t)e * K + min(col, K - 16)) * I, col < K ? 16 * I : 0);
        nx.scale = buffer_of(g.l.s2 + (e * blocks2 + slice) * nib, nib * 4);
        nx.hoff = hrow < pairs >> 16 ? ((pairs & 0xFFFF) + hrow) * I * 2 + 16 * hchunk : far;
    };
    // as the narrow kernel's, with bit 30 for the second share
    auto fetch = [&](int slot, i32x4 (&w)[2], float& scale) {
        int8_t* to = sh.ring + slot * SLOT + 1024 * wave;
        const int left = I - nx.b * QB, cut = 8 * hchunk < left ? 0 : far;
#pragma unroll
        for (int k = 0; k < TERMS; ++k)
            buffer_to_lds16<0>(rh, (nx.hoff + 2 * QB * nx.b) | cut, k * plane, to + PLANE * k);
        load_codes(w, nx.w, I, nx.b * QB, left);
        scale = __int_as_float(__builtin_amdgcn_raw_buffer_load_b32(nx.scale, 4 * nx.b, 0, 0));
        asm volatile("" ::: "memory");
        if (nx.at < 0)
            return -1;
        int info = __builtin_amdgcn_readlane(nx.pairs, nx.at) | nx.turn << 30;
        nx.b += shares;
        if (nx.b >= nib) {
            info |= (int)0x80000000;
            nx.b = 0;
            enter();
        }
        return info;
    };

    f32x4 acc[TILES];
    auto clear = [&]() {
#pragma unroll
        for (int i = 0; i < TILES; ++i)
            acc[i] = f32x4{0, 0, 0, 0};
    };
    clear();
    if (nunits > 0) {
        i32x4 wv[S][2];
        float sv[S];
        int info[S];
        nx.turn = nx.b = 0;
        open_window(0);
        enter();
#pragma unroll
        for (int i = 0; i < S - 1; ++i)
            info[i] = fetch(i, wv[i], sv[i]);
        int at[4];
#pragma unroll
        for (int f = 0; f < 4; ++f)
            at[f] = r * 2 * QB + 16 * ((8 * (f >> 1) + 2 * q + (f & 1)) ^ r);
        while (info[0] != -1) {
#pragma unroll
            for (int u = 0; u < S; ++u) {
                __builtin_amdgcn_s_waitcnt(wait_vm((S - 2) * COPIES));
                barrier_lds();
                info[(u + S - 1) % S] = fetch((u + S - 1) % S, wv[(u + S - 1) % S], sv[(u + S - 1) % S]);
                __builtin_amdgcn_sched_barrier(0);
                const int8_t* hs = sh.ring + u * SLOT;
                i32x4 w[2];
                turn_codes(sh.turn[wave], wv[u], w);
                const bf16x8 a[4] = {codes_bf16(w[0][0], w[0][1]), codes_bf16(w[0][2], w[0][3]), codes_bf16(w[1][0], w[1][1]),
                                     codes_bf16(w[1][2], w[1][3])};
                const int base = info[u] & 0xFFFF, count = info[u] >> 16 & 0x7F;
#pragma unroll
                for (int i = 0; i < TILES; ++i) {
                    if (16 * i < count) {
                        f32x4 p[TERMS];
#pragma unroll
                        for (int k = 0; k < TERMS; ++k) {
                            p[k] = f32x4{0, 0, 0, 0};
#pragma unroll
                            for (int f = 0; f < 4; ++f)
                                p[k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                    a[f], *reinterpret_cast<const bf16x8*>(hs + PLANE * k + 16 * 2 * QB * i + at[f]), p[k], 0, 0, 0);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float v = p[TERMS - 1][e];
#pragma unroll
                            for (int k = TERMS - 2; k >= 0; --k)
                                v += p[k][e];
                            acc[i][e] = fmaf(sv[u], v, acc[i][e]);
                        }
                    }
                }
                if (info[u] < -1) {
                    auto& sums = sh.sums[info[u] >> 30 & 1];
#pragma unroll
                    for (int i = 0; i < TILES; ++i)
                        if (16 * i + r < count)
                            *reinterpret_cast<f32x4*>(&sums[sh.pair_token[base + 16 * i + r]][16 * wave + 4 * q]) += acc[i];
                    clear();
                }
            }
        }
        __builtin_amdgcn_s_waitcnt(wait_vm(0));
    }
    __syncthreads();
    constexpr int C4 = WIDE_COLS / 4;
    const int parts = g.parts * WIDE_PARTS, psize = g.T * K * 4;
    const __amdgpu_buffer_rsrc_t mine = buffer_of(g.sums + (int64_t)part * g.T * K, psize);
    for (int i = threadIdx.x; i < g.T * C4; i += NT) {
        const int c = n0 + i % C4 * 4;
        const float *a = &sh.sums[0][i / C4][i % C4 * 4], *b = &sh.sums[1][i / C4][i % C4 * 4];
        const f32x4 v = *reinterpret_cast<const f32x4*>(a) + *reinterpret_cast<const f32x4*>(b);
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), mine, c < K ? (i / C4 * K + c) * 4 : far, 0,
                                               DEVICE);
    }
    if (!last_to_arrive(g, slice, parts, sh.last))
        return;
    for (int i = threadIdx.x; i < g.T * C4; i += NT) {
        const int c = n0 + i % C4 * 4;
        if (c >= K)
            continue;
        f32x4 v{0, 0, 0, 0};
#pragma unroll 4
        for (int p = 0; p < parts; p += WIDE_PARTS) {
            f32x4 w[WIDE_PARTS];
#pragma unroll
            for (int k = 0; k < WIDE_PARTS; ++k)
                w[k] = part_sums(g, p + k, i / C4, c);
            v += (w[0] + w[1]) + (w[2] + w[3]);
        }
        write_out(g, i / C4, c, v);
    }
}

template <int TERMS>
void launch_wide(const Moe& g, hipStream_t stream) {
    const int64_t pairs = g.T * g.l.top_k, most = (pairs < g.l.E ? pairs : g.l.E) * ((g.l.I + WIDE_COLS - 1) / WIDE_COLS);
    const dim3 up((uint32_t)(most < cu_count() ? most : cu_count())), nt(NT);
    if (g.l.E <= 64)
        moe_up_wide_kernel<4, TERMS><<<up, nt, 0, stream>>>(g);
    else   // at most 128: a launch has 1024 pairs, and an expert 8 on average
        moe_up_wide_kernel<8, TERMS><<<up, nt, 0, stream>>>(g);
    const dim3 down((uint32_t)((g.l.K + WIDE_COLS - 1) / WIDE_COLS * g.parts * WIDE_PARTS));
    moe_down_wide_kernel<TERMS><<<down, nt, 0, stream>>>(g);
}

template <int TERMS>
void launch_narrow(const Moe& g, hipStream_t stream) {
    const int64_t most = (int64_t)(g.T * g.l.top_k < MOE_UNITS ? g.T * g.l.top_k : MOE_UNITS) * (g.l.I / 16);
    const dim3 up((uint32_t)(most < cu_count() ? most : cu_count())), nt(NT);
    // (Over 128 experts 32 logits a lane: a call with next to nothing to read, K = I = 64 and top_k 8, takes at 64, 128, 256
    // and 512 experts 15.0, 15.4, 18.8 and 19.5 us for one token, 20.7, 21.2, 33.1 and 39.2 for 64. 64 tokens of 256
    // experts with K 2048, I 768 take 187 us of these kernels, codes at 5.6 and 5.6 TB/s.)
    auto launch_up = [&](auto kernel, auto halves) { (whole_lines(g.l.K) ? kernel : halves)<<<up, nt, 0, stream>>>(g); };
    if (g.l.E <= 64)
        launch_up(moe_up_kernel<4, TERMS, true>, moe_up_kernel<4, TERMS, false>);
    else if (g.l.E <= 128)
        launch_up(moe_up_kernel<8, TERMS, true>, moe_up_kernel<8, TERMS, false>);
    else
        launch_up(moe_up_kernel<32, TERMS, true>, moe_up_kernel<32, TERMS, false>);
    const dim3 down((uint32_t)(g.l.K / DOWN_COLS * g.parts));
    auto launch_down = [&](auto kernel, auto halves) { (whole_lines(g.l.I) ? kernel : halves)<<<down, nt, 0, stream>>>(g); };
    if (g.T <= 16)
        launch_down(moe_down_kernel<TERMS, 16, true>, moe_down_kernel<TERMS, 16, false>);
    else if (g.T <= 32)
        launch_down(moe_down_kernel<TERMS, 32, true>, moe_down_kernel<TERMS, 32, false>);
    else
        launch_down(moe_down_kernel<TERMS, 64, true>, moe_down_kernel<TERMS, 64, false>);
}

template <int TERMS>
void launch_experts(const Moe& g, hipStream_t stream) {
    // Wide where an expert has 8 tokens on average, its tasks of 128 columns occupy most CUs and there are
    // enough codes to make up for its longer start and join. Narrow / wide, us, at T, E, top_k, K, I:
    //   64 8 2 4096 7168  232.7 / 159.9    12 4 4 4096 7168   88.0 / 78.0    5 8 2 4096 7168   102.6 / 130.0
    //   64 8 2 2048 3200   68.8 / 60.3     64 8 2 2048 2560   58.4 / 56.1    20 4 2 2048 4096   33.5 / 41.0
    //   64 16 2 4096 2048  91.2 / 95.1     64 32 8 4096 1024 143.2 / 105.2   64 16 2 1024 2048  41.1 / 49.7
    //   64 64 6 2048 1408 125.2 / 126.4    64 60 8 1984 1344 135.2 / 132.4   32 64 8 2048 1408 110.1 / 119.0
    const int64_t tasks = (int64_t)g.l.E * ((g.l.I + WIDE_COLS - 1) / WIDE_COLS);
    if (g.T * g.l.top_k >= 8 * g.l.E && 4 * tasks >= 3 * cu_count() && (int64_t)g.l.E * g.l.K * g.l.I >= 40 << 20)
        launch_wide<TERMS>(g, stream);
    else
        launch_narrow<TERMS>(g, stream);
}

// Workgroups that share a slice of output columns, so that the slices of narrow layers fill the chip's
// 256 CUs, once. Filling half / all of them / twice as many workgroups, the layer's us at T, E, top_k, K, I:
// 1 64 8 2048 1536 28.2 / 27.3 / 30.5, 5 8 2 4096 7168 119 / 100 / 104, 64 64 6 2048 1408 151 / 127 / 133.
// (A rule on K alone: the order of a token's sums must not depend on the batch, nor on the card.)
int parts_of(int K) {
    int p = 1;
    while (p < 8 && 2 * p * (K / DOWN_COLS) <= 256)
        p *= 2;
    return p;
}

}  // namespace

int64_t moe_workspace(int64_t T, int top_k, int K, int I) {
    const int64_t t = T < MOE_TOKENS ? T : MOE_TOKENS;
    return (int64_t)sizeof(MoeSpace) + t * K * 4 * parts_of(K) * WIDE_PARTS + t * top_k * I * 6;
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
        g.parts = parts_of(l.K);
        g.l.x += t * l.K;
        g.l.logits += t * l.E;
        g.l.out = reinterpret_cast<int8_t*>(l.out) + t * l.K * (l.out_f16 ? 2 : 4);
        g.space = reinterpret_cast<MoeSpace*>(l.ws);
        g.sums = reinterpret_cast<float*>(l.ws + sizeof(MoeSpace));
        g.h = reinterpret_cast<__bf16*>(g.sums + (int64_t)g.parts * WIDE_PARTS * g.T * l.K);
        if (l.out_f16)
            launch_experts<2>(g, stream);
        else
            launch_experts<3>(g, stream);
    }
    return launch_status();
}

}  // namespace ql
