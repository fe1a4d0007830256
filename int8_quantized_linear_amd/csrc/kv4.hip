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

constexpr int KT = 256, KW = KT / WAVE;   // threads and waves per workgroup

// 8 neighbouring values as they lie in memory (fp16 or fp32), and as fp32.
template <bool F16>
struct Eight {
    u32x4 w[F16 ? 1 : 2];
    __device__ inline void load(const void* p, int64_t i) {
        const u32x4* s = reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(p) + i * (F16 ? 2 : 4));
#pragma unroll
        for (int j = 0; j < (F16 ? 1 : 2); ++j)
            w[j] = __builtin_nontemporal_load(&s[j]);   // read once (prompts of 8850 rows 53 -> 47 us)
    }
    __device__ inline void get(float (&v)[8]) const {
        if constexpr (F16) {
            const f16x8 h = __builtin_bit_cast(f16x8, w[0]);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = (float)h[e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = __uint_as_float(w[e / 4][e % 4]);
        }
    }
};

// +inf as fp32's largest number, whose scale and code saturate as the definition has it (the
// refined quotients below make NaN of infinite ones).
constexpr float FINITE = 3.402823466e38f;
__device__ inline float to_finite(float v) { return v > FINITE ? FINITE : v; }

// fp16 of a float, kept within fp16's finite range.
__device__ inline _Float16 to_f16_sat(float v) {
    return (_Float16)__builtin_amdgcn_fmed3f(v, -65504.0f, 65504.0f);
}

// Minimum and maximum over the N = 4, 8 or 16 lanes that share a group, on the vector unit alone:
// neighbours, pairs, then the mirror images of 8 and of 16 lanes.
template <int CTRL>
__device__ inline void fold(float& lo, float& hi) {
    const float a = __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(lo), CTRL, 0xF, 0xF, true));
    const float b = __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(hi), CTRL, 0xF, 0xF, true));
    lo = fminf(lo, a);
    hi = fmaxf(hi, b);
}
template <int N>
__device__ inline void group_range(float& lo, float& hi) {
    fold<0xB1>(lo, hi);   // lane ^ 1
    fold<0x4E>(lo, hi);   // lane ^ 2
    if constexpr (N >= 8)
        fold<0x141>(lo, hi);   // 7 - lane
    if constexpr (N >= 16)
        fold<0x140>(lo, hi);   // 15 - lane
}

// a / 15 and 1 / s for an fp16 s, correctly rounded: through RN(1 / 15) with one correction, and
// one step from v_rcp_f32 (within one unit in the last place).
__device__ inline float fifteenth(float a) {
    constexpr float r = 1.0f / 15.0f;
    const float q0 = __fmul_rn(a, r);
    return fmaf(fmaf(-q0, 15.0f, a), r, q0);
}
__device__ inline float reciprocal_f16(float s) {
    const float y = __builtin_amdgcn_rcpf(s);
    return fmaf(fmaf(-s, y, 1.0f), y, y);
}

// clamp(round(a / s), 0, 15) with y = 1 / s correctly rounded: a / s as RN(q0 + (a - q0 s) y),
// q0 = RN(a y), the correctly rounded quotient (Markstein) where nothing underflows; where
// something does, a / s is below 2^-80 and the code 0 on either path. Clamping first changes no
// code (the bounds are integers), and adding 1.5 2^23 rounds half to even into the low bits:
// the result is the code + ROUNDED.
constexpr float ROUND = 12582912.0f;
constexpr uint32_t ROUNDED = 0x4B400000u;
__device__ inline uint32_t code4(float a, float s, float y) {
    const float q0 = __fmul_rn(a, y);
    const float q = fmaf(fmaf(-q0, s, a), y, q0);
    return __float_as_uint(__fadd_rn(__builtin_amdgcn_fmed3f(q, 0.0f, 15.0f), ROUND));
}

// Place of code e in a word: K's pairs of neighbours meet in the halves, V's bytes hold pairs.
constexpr int k_shift(int e) { return 16 * (e & 1) + 4 * (e >> 1); }
constexpr int v_shift(int e) { return 4 * e; }

// Eight codes in one word; the sum of the shifted ROUNDED wraps to a constant, taken off first.
template <bool K>
__device__ inline uint32_t codes8(const float (&x)[8], float low, float s, float y) {
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        w -= ROUNDED << (K ? k_shift(e) : v_shift(e));
#pragma unroll
    for (int e = 0; e < 8; ++e)
        w += code4(x[e] - low, s, y) << (K ? k_shift(e) : v_shift(e));
    return w;
}

// A wave takes the runs of up to 8 rows that start among its `per` rows: rows of one sequence
// whose positions lie in one aligned group of 8 (a unit of V's layout, inside one page), for the
// heads of its group, the next head's rows in flight while one is written. Lanes of D / 8 take a
// token, 8 values each, so that a lane's K codes are one word, and G / 8 lanes share a scale.
// V's codes of a full run are gathered through LDS into the 16-byte units of 8 tokens; a part of
// a run writes its tokens' 16 bits, so that its neighbours keep theirs. Bound by memory where rows
// are many: 8850 fp16 rows of 32 heads of 128 in groups of 128 (183 MB) take 45 us, 4.1 TB/s, where
// a large copy reaches 5.0; 32 rows of 8 heads 4.2 us, the chain from the batch's lists over the
// block table to a row.
template <int D, int G, bool F16>
__global__ __launch_bounds__(KT) void kv4_append_kernel(const void* __restrict__ k, const void* __restrict__ v,
                                                        int64_t k_stride, int64_t v_stride, int rows, int per,
                                                        int head_groups, Kv4Cache c, Kv4Batch b) {
    using L = Kv4Layout<D, G>;
    constexpr int LPT = D / 8, TPP = WAVE / LPT, PASSES = 8 / TPP;
    __shared__ __attribute__((aligned(16))) uint16_t units[KW][D / 4][8];
    const int P = 1 << c.page_log2, lane = threadIdx.x & (WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int head0 = blockIdx.x % head_groups;
    const int r0 = (int)(blockIdx.x / head_groups * KW + wave) * per;

    // lane i < per looks at row r0 + i: does a run start there?
    int seq = 0, pos = -1, n = 0;
    if (lane < per && r0 + lane < rows) {
        const int row = r0 + lane;
        seq = kv4_seq(b, row);
        const int len = kv4_len(b, c, seq), end = b.starts[seq + 1];
        pos = kv4_pos(b, seq, len, row);
        if (pos >= 0 && pos < len && ((pos & 7) == 0 || row == b.starts[seq]))
            n = min(min(8 - (pos & 7), end - row), rows - row);
    }
    uint64_t runs = __ballot(n > 0);
    while (runs) {
        const int i = __builtin_ctzll(runs);
        runs &= runs - 1;
        const int rseq = __builtin_amdgcn_readlane(seq, i), rpos = __builtin_amdgcn_readlane(pos, i);
        const int rn = __builtin_amdgcn_readlane(n, i);
        const int slot0 = rpos & (P - 1) & ~7, t0 = rpos & 7;   // the run is tokens t0 .. t0 + rn - 1 of 8
        const int d0 = (lane % LPT) * 8, g = d0 / G;
        Eight<F16> next[2][PASSES];
        auto load = [&](int head) {
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                const int t = p * TPP + lane / LPT - t0;
                if (t >= 0 && t < rn) {
                    const int64_t row = r0 + i + t;
                    next[0][p].load(k, row * k_stride + head * D + d0);
                    next[1][p].load(v, row * v_stride + head * D + d0);
                }
            }
        };
        const int cnt = (c.heads + head_groups - 1) / head_groups, h0 = head0 * cnt, h1 = min(h0 + cnt, c.heads);
        if (h0 >= h1)
            return;
        load(h0);
        uint8_t* page = kv4_page(b, c, rseq, rpos, h0);
        for (int head = h0; head < h1; ++head) {
            Eight<F16> raw[2][PASSES];
#pragma unroll
            for (int p = 0; p < PASSES; ++p)
                raw[0][p] = next[0][p], raw[1][p] = next[1][p];
            if (head + 1 < h1)
                load(head + 1);
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                const int tok = p * TPP + lane / LPT, slot = slot0 + tok;
                const bool on = tok >= t0 && tok < t0 + rn;
#pragma unroll
                for (int which = 0; which < 2; ++which) {
                    float x[8];
                    raw[which][p].get(x);
                    float lo = x[0], hi = x[0];
#pragma unroll
                    for (int e = 1; e < 8; ++e) {
                        lo = fminf(lo, x[e]);
                        hi = fmaxf(hi, x[e]);
                    }
                    group_range<G / 8>(lo, hi);
                    if (__any(hi > FINITE)) {
                        hi = to_finite(hi);
                        lo = to_finite(lo);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            x[e] = to_finite(x[e]);
                    }
                    const _Float16 lo16 = to_f16_sat(lo);
                    const float lf = (float)lo16;
                    const _Float16 least = (_Float16)5.9604644775390625e-08f;   // 2^-24
                    _Float16 s16 = to_f16_sat(fmaxf(fifteenth(hi - lf), 0.0f));
                    s16 = s16 > least ? s16 : least;
                    const float s = (float)s16, y = reciprocal_f16(s);
                    if (on && lane % (G / 8) == 0) {
                        reinterpret_cast<_Float16*>(page + (which ? L::v_scale(P, g) : L::k_scale(P, g)))[slot] = s16;
                        reinterpret_cast<_Float16*>(page + (which ? L::v_low(P, g) : L::k_low(P, g)))[slot] = lo16;
                    }
                    if (which == 0) {
                        const uint32_t w = codes8<true>(x, lf, s, y);
                        if (on)
                            reinterpret_cast<uint32_t*>(page + L::k_codes(slot))[((d0 % 32) / 8) * (D / 32) + d0 / 32] = w;
                    } else {
                        // bytes of d pairs, of 4 quads; the other half of each is 32 values away,
                        // in lane ^ 4: either lane completes two quads
                        const uint32_t w = codes8<false>(x, lf, s, y);
                        const uint32_t z = __shfl_xor(w, 4, WAVE);
                        const bool up = lane & 4;
                        const uint32_t a = up ? z >> 16 : w, h = up ? w >> 16 : z;
                        const uint32_t two = (a & 0xFF) | (h & 0xFF) << 8 | (a & 0xFF00) << 8 | (h & 0xFF00) << 16;
                        const int quad = d0 / 64 * 16 + d0 % 32 / 2 + (up ? 2 : 0);
                        if (rn == 8) {
                            units[wave][quad][tok] = (uint16_t)two;
                            units[wave][quad + 1][tok] = (uint16_t)(two >> 16);
                        } else if (on) {
                            uint16_t* to = reinterpret_cast<uint16_t*>(page + L::v_codes(P, slot / 8)) + slot % 8;
                            to[quad * 8] = (uint16_t)two;
                            to[quad * 8 + 8] = (uint16_t)(two >> 16);
                        }
                    }
                }
            }
            if (rn == 8) {
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
                if (lane < D / 4)
                    *reinterpret_cast<u32x4*>(page + L::v_codes(P, slot0 / 8) + lane * 16) =
                        *reinterpret_cast<const u32x4*>(units[wave][lane]);
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
            }
            page += c.head_bytes;
        }
    }
}

// Values d .. of two chunks c and c + 1, held as halves (0, 32) of c in the even lanes and of c + 1
// in the odd ones (4 lanes on): the even chunk's halves from both lanes, then the odd chunk's.
__device__ inline void trade_store(_Float16* to, const float (&v)[2][8], bool odd) {
    f16x8 h[2];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        h[0][e] = (_Float16)v[0][e], h[1][e] = (_Float16)v[1][e];
    const u32x4 give = __builtin_bit_cast(u32x4, odd ? h[0] : h[1]);
    u32x4 got;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        got[e] = (uint32_t)__shfl_xor((int)give[e], 4, WAVE);
    const u32x4 own = __builtin_bit_cast(u32x4, odd ? h[1] : h[0]);
    __builtin_nontemporal_store(odd ? got : own, reinterpret_cast<u32x4*>(to));
    __builtin_nontemporal_store(odd ? own : got, reinterpret_cast<u32x4*>(to + 64));
}

// Lanes of D / 16 take a row, 16 values of K and of V each: d = 64 c + 8 kg + 0 .. 7 and 32 more,
// which are two neighbouring words of K and the 4 quads 4 kg .. 4 kg + 3 of V's chunk c. A wave
// has 1024 / D neighbouring rows, so that V's units of 8 tokens are read whole, and goes through
// the heads of its group. Bound by memory: 8850 rows of 32 heads of 128 in groups of 128 to fp16
// (183 MB) take 30 us, 6.2 TB/s, the cache's part of it still held by the caches of the chip.
template <int D, int G, bool F16>
__global__ __launch_bounds__(KT) void kv4_read_kernel(Kv4Cache c, Kv4Batch b, int rows, int head_groups,
                                                      void* __restrict__ k_out, void* __restrict__ v_out) {
    using L = Kv4Layout<D, G>;
    constexpr int LPR = D / 16, RPW = WAVE / LPR;
    const int P = 1 << c.page_log2, lane = threadIdx.x & (WAVE - 1);
    const int row = (int)(blockIdx.x / head_groups * KW + threadIdx.x / WAVE) * RPW + lane / LPR;
    if (row >= rows)
        return;
    const int head0 = blockIdx.x % head_groups, ch = lane % LPR / 4, kg = lane % 4, d0 = ch * 64 + kg * 8;
    const int seq = kv4_seq(b, row);
    const int len = kv4_len(b, c, seq), pos = kv4_pos(b, seq, len, row);
    const bool on = pos >= 0 && pos < len;
    const int cnt = (c.heads + head_groups - 1) / head_groups, h0 = head0 * cnt, h1 = min(h0 + cnt, c.heads);
    const uint8_t* page = on ? kv4_page(b, c, seq, pos, h0) : nullptr;
    const int slot = pos & (P - 1);
    const int k_at = L::k_codes(slot) + (kg * (D / 32) + 2 * ch) * 4;
    const int v_at = L::v_codes(P, slot / 8) + (ch * 16 + kg * 4) * 16 + slot % 8 * 2;
    for (int head = h0; head < h1; ++head) {
        float kx[2][8] = {}, vx[2][8] = {};
        if (on) {
            const u32x2 kw = *reinterpret_cast<const u32x2*>(page + k_at);
            const uint16_t* vq = reinterpret_cast<const uint16_t*>(page + v_at);
            const uint32_t q[4] = {vq[0], vq[8], vq[16], vq[24]};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int g = (d0 + 32 * h) / G;
                const float ks = (float)reinterpret_cast<const _Float16*>(page + L::k_scale(P, g))[slot];
                const float kl = (float)reinterpret_cast<const _Float16*>(page + L::k_low(P, g))[slot];
                const float vs = (float)reinterpret_cast<const _Float16*>(page + L::v_scale(P, g))[slot];
                const float vl = (float)reinterpret_cast<const _Float16*>(page + L::v_low(P, g))[slot];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    kx[h][e] = fmaf(ks, (float)((kw[h] >> k_shift(e)) & 15), kl);
                    vx[h][e] = fmaf(vs, (float)((q[e / 2] >> (8 * h + 4 * (e & 1))) & 15), vl);
                }
            }
        }
        const int64_t at = ((int64_t)row * c.heads + head) * D;
        if constexpr (F16 && D >= 128) {
            // 32 values (64 bytes) of a row in each half and 4 lanes: lanes of neighbouring chunks
            // trade halves, so that 8 lanes write 128 bytes together, past the caches. (Left dirty
            // in them, the 100 MB of 24600 rows of 8 heads hold up the next kernel: 49 us a write
            // and a read of these sizes, 36 like this.)
            const bool odd = ch & 1;
            const int64_t even_at = at + (ch & ~1) * 64 + kg * 8 + (odd ? 32 : 0);
            trade_store(reinterpret_cast<_Float16*>(k_out) + even_at, kx, odd);
            trade_store(reinterpret_cast<_Float16*>(v_out) + even_at, vx, odd);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                store8<F16>(k_out, at + d0 + 32 * h, kx[h]);
                store8<F16>(v_out, at + d0 + 32 * h, vx[h]);
            }
        }
        page += c.head_bytes;
    }
}

// Groups of heads, each a workgroup's loop: as many as make FILL workgroups.
constexpr int64_t FILL = 2048;
inline int groups_of_heads(int64_t blocks, int heads) {
    const int64_t n = (FILL + blocks - 1) / blocks;
    return n < heads ? (int)n : heads;
}

}  // namespace

ql_status launch_kv4_append(const void* k, const void* v, bool f16, int64_t k_stride, int64_t v_stride, int64_t rows,
                            const Kv4Cache& c, int D, int G, const Kv4Batch& b, hipStream_t stream) {
    return kv4_dispatch(D, G, [&](auto d, auto g) {
        constexpr int DD = decltype(d)::value, GG = decltype(g)::value;
        // runs of 8 rows a wave for prompts, single rows where sequences bring few (8 heads of 128:
        // 32 x 1 row 4.2 us by single rows, 14.5 us by eights; 128 x 4 4.9 and 6.1; 128 x 8 8.0 and
        // 6.3; 8850 rows of 32 heads 117 and 47 us)
        const int per = rows > 4 * (int64_t)b.batch ? 8 : 1;
        const int64_t blocks = (rows + per * KW - 1) / (per * KW);
        const int hg = groups_of_heads(blocks, c.heads);
        const dim3 grid((uint32_t)(blocks * hg));
        if (f16)
            kv4_append_kernel<DD, GG, true><<<grid, KT, 0, stream>>>(k, v, k_stride, v_stride, (int)rows, per, hg, c, b);
        else
            kv4_append_kernel<DD, GG, false><<<grid, KT, 0, stream>>>(k, v, k_stride, v_stride, (int)rows, per, hg, c, b);
        return launch_status();
    });
}

ql_status launch_kv4_read(const Kv4Cache& c, int D, int G, const Kv4Batch& b, int64_t rows, void* k_out, void* v_out,
                          bool f16, hipStream_t stream) {
    return kv4_dispatch(D, G, [&](auto d, auto g) {
        constexpr int DD = decltype(d)::value, GG = decltype(g)::value;
        constexpr int per = KW * (1024 / DD);
        const int64_t blocks = (rows + per - 1) / per;
        const int hg = groups_of_heads(blocks, c.heads);
        const dim3 grid((uint32_t)(blocks * hg));
        if (f16)
            kv4_read_kernel<DD, GG, true><<<grid, KT, 0, stream>>>(c, b, (int)rows, hg, k_out, v_out);
        else
            kv4_read_kernel<DD, GG, false><<<grid, KT, 0, stream>>>(c, b, (int)rows, hg, k_out, v_out);
        return launch_status();
    });
}

}  // namespace ql
