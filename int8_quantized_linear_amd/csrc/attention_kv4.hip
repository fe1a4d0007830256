// attention_kv4.hip -- causal attention over the paged 4-bit K/V cache.
//
//   o = sum_j softmax_j(scale * q . k_j) v_j   over the positions j that the row sees,
//   max(0, p - window + 1) <= j <= p for a row at position p (from 0 without a window)
//
// in one pass with a running maximum and sum. A row that sees nothing gives zeros.
//
// Decode kernel (few rows of a sequence): bound by reading the cache. The rows of one sequence
// that share a kv head, (row, head) pairs in order, make tiles of 16 columns. A workgroup of four
// waves takes one tile and one stretch of the sequence; each wave steps through every fourth
// block of 32 tokens on its own (no barrier in the loop), and the four partial results are
// joined through LDS at the end, the stretches' by a second kernel.
//   S^T = K Q^T   16x16x32 fp16: rows are tokens, columns the tile's rows. K's codes enter as
//                 fp16 integers (the masked nibbles are fp16 subnormals c 2^-24 or 16 c 2^-24,
//                 which the matrix cores take exactly; q's slots carry the 1/16, and a power of
//                 two where q is small enough to lose bits by it), one product
//                 for each group of G values, and scale and low are applied to the fp32 product:
//                 s_t sum_d c q_d + low_t sum_d q_d.
//   O^T = V^T P^T the products' layout hands each lane the weights of 8 consecutive tokens for
//                 one column, which is the layout of the next product's operand: P never
//                 crosses lanes. V becomes fp16 values scale * code + low (one rounding), since
//                 its scales lie along the summed axis; folding them into P would tie P's fp16
//                 range to V's magnitude. P enters as two fp16 terms (22 bits): V's rounding and
//                 the output's are the only ones to fp16. With one term the error against 64
//                 bits is 1.6 times the output's own rounding, with two 1.33 times, and with V's
//                 codes and scales kept apart as well 1.0 times, but for long sums, whose two parts
//                 cancel (4 times at 131072 tokens). The second term costs the decode kernel 4 to
//                 7% (517 positions 9.95 -> 10.3 us, 131072 40.0 -> 42.3 us), 15% where the chip is
//                 full (165 -> 190 us), the prompt kernel 13%.
// The running maximum is raised only when a score exceeds it by 2^8 (weights up to 2^14, sums
// in fp32), so most steps have neither a reduction across lanes nor a rescaling of O.
// 64 tokens of 8 x 8 heads of 128 over 8192 to 16384 positions (902 MB in groups of 64) take 172 to
// 187 us by the card, 4.8 to 5.2 TB/s; where they take 177, the same copies without the arithmetic
// take 143.
#include <algorithm>

#include "kv4.h"

namespace ql {
namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

constexpr int AT = 256, AW = AT / WAVE;   // threads and waves of a decode workgroup
constexpr int TB = 32;                    // tokens of a step
constexpr float M_NONE = -3.402823466e38f;   // running maximum before the first score, fp32's least
constexpr float P_SHIFT = 6.0f;           // weights are 2^(score - max + P_SHIFT)
constexpr float M_SLACK = 8.0f;           // and may exceed 2^P_SHIFT by 2^M_SLACK before a rescale

__device__ inline f16x2 as_f16x2(uint32_t w) { return __builtin_bit_cast(f16x2, w); }
__device__ inline uint32_t as_u32(f16x2 h) { return __builtin_bit_cast(uint32_t, h); }

// The page table is not written while a kernel runs: scalar loads.
__device__ inline uint32_t table_entry(const int32_t* p) {
    return (uint32_t)*(const __attribute__((address_space(4))) int32_t*)(uintptr_t)p;
}

// Rows that one workgroup handles and the positions that they see.
struct RowTile {
    int first;       // position of the sequence's row 0
    int rows;        // the sequence's rows
    int begin, end;  // positions that any of the tile's rows sees
    int all_begin, all_end;   // positions that all of them see
};

__device__ inline RowTile row_tile(const Kv4Batch& b, const Kv4Cache& c, int seq, int tile, int per, int R, int window) {
    RowTile t;
    const int len = kv4_len(b, c, seq);
    const int64_t rows = (int64_t)b.starts[seq + 1] - b.starts[seq];   // whatever the starts are
    t.rows = rows < 0 ? 0 : rows > b.rows ? b.rows : (int)rows;
    t.first = len - t.rows;
    const int i0 = tile * per / R, i1 = min((tile * per + per - 1) / R, t.rows - 1);
    t.end = max(0, t.first + i1 + 1);
    t.all_end = max(0, t.first + i0 + 1);
    const int seen = max(i0, -t.first);   // the first row with a position
    t.begin = window ? max(0, t.first + seen + 1 - window) : 0;
    t.all_begin = window ? max(0, t.end - window) : 0;
    return t;
}

// Row i of a sequence in the call's rows, or a number outside them (unsigned: also below 0) where
// the caller's starts lead there.
__device__ inline uint32_t row_of(const Kv4Batch& b, int seq, int i) { return (uint32_t)b.starts[seq] + (uint32_t)i; }

// Tokens of one split: the launch's stretch, or more where the splits would not reach the end.
// Positions are below 2^31; sums of them and of stretches are unsigned, below 2^32.
__device__ inline uint32_t split_tokens(const RowTile& t, uint32_t stretch, int nsplit) {
    const int base = t.begin & ~(TB - 1);
    const uint32_t need = ((uint32_t)(t.end - base) + nsplit - 1) / nsplit;
    return max(stretch, (need + TB * AW - 1) & ~(uint32_t)(TB * AW - 1));
}

struct Split {
    int n;              // splits
    uint32_t stretch;   // tokens of each at the launch's max_len
    int tiles;          // row tiles a sequence and kv head at the launch's max_q
};

typedef __attribute__((address_space(3))) void* lds_ptr;

// s_waitcnt immediate: at most n vector-memory operations pending (gfx9 encoding: vmcnt in
// bits 3:0 and 15:14, the other counters not waited for)
constexpr int vmcnt_le(int n) { return (n & 0xF) | (0x7 << 4) | (0xF << 8) | (((n >> 4) & 3) << 14); }

// 16 bytes per lane from memory straight into LDS: lane l's land at l * 16 past the wave-uniform
// LDS address. Device pass only (in the host pass the builtin makes clang drop the kernel's
// launch stub).
__device__ inline void lds_copy16(const void* g, void* lds) {
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_global_load_lds(g, (lds_ptr)lds, 16, 0, 2);   // nt: read once
#endif
}

// Reads from LDS that the compiler does not see as such: it would make each wait for every copy in
// flight (the copies write LDS too). The reads and their wait are one block; what orders them
// behind the copies of their slot is the caller's wait for those, and what orders a later copy
// into the slot behind them is the wait in the block.
__device__ inline uint32_t lds_addr(const void* p) { return (uint32_t)(uintptr_t)(lds_ptr)p; }

template <int O0, int O1>
__device__ inline void lds_read(uint32_t at, u32x2& a, u32x2& b) {
    asm volatile("ds_read_b64 %0, %2 offset:%3\n\tds_read_b64 %1, %2 offset:%4\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(a), "=&v"(b)
                 : "v"(at), "n"(O0), "n"(O1));
}
template <int O0, int O1>
__device__ inline void lds_read(uint32_t at, u32x4& a, u32x4& b) {
    asm volatile("ds_read_b128 %0, %2 offset:%3\n\tds_read_b128 %1, %2 offset:%4\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(a), "=&v"(b)
                 : "v"(at), "n"(O0), "n"(O1));
}
template <int O0, int O1, int O2, int O3>
__device__ inline void lds_read(uint32_t at, u32x4& a, u32x4& b, u32x4& c, u32x4& d) {
    asm volatile(
        "ds_read_b128 %0, %4 offset:%5\n\tds_read_b128 %1, %4 offset:%6\n\tds_read_b128 %2, %4 offset:%7\n\t"
        "ds_read_b128 %3, %4 offset:%8\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(a), "=&v"(b), "=&v"(c), "=&v"(d)
        : "v"(at), "n"(O0), "n"(O1), "n"(O2), "n"(O3));
}

// A block's cache data in LDS, copied straight from memory (16 bytes a lane, lane l's at 16 l of
// each 1024-byte copy). K's codes, V's codes and each array of scales or lows of 32 tokens are
// contiguous in a page, so all copies are linear; with pages of 16 tokens their upper halves come
// from a second page. K's 16-byte chunks of token T are rotated by T / 8 places within the
// token's row, so that the operands' reads (tokens 8 x + 0 .. 3 at once) meet no bank twice.
template <int D, int G, bool BIG>
struct Ring {
    using L = Kv4Layout<D, G>;
    static constexpr int NG = D / G, KC = D / 64, PC = (NG + 3) / 4, COPIES = 2 * KC + PC;
    static constexpr int K_AT = 0, V_AT = 16 * D, P_AT = 32 * D, BYTES = 32 * D + 256 * NG;
    const int32_t* table;
    const uint8_t* data;   // the head's part of page 0
    int64_t page_bytes;
    int pages, log2p, last;
    int k_src[KC], v_src, p_src[PC];   // this lane's byte offsets in a page, without the slot's part
    bool k_hi, p_hi;                   // the lane's bytes come from the second page

    __device__ inline Ring(const Kv4Batch& b, const Kv4Cache& c, int seq, int head, int end) {
        table = b.table + (int64_t)seq * b.width;
        data = c.data + head * c.head_bytes;
        page_bytes = c.heads * c.head_bytes;
        pages = c.pages;
        log2p = c.page_log2;
        last = end - 1;
        const int lane = threadIdx.x & (WAVE - 1), P = 1 << log2p;
        constexpr int CPT = D / 32;   // 16-byte chunks of a token's K row
        for (int i = 0; i < KC; ++i) {
            const int at = i * 64 + lane, tok = at / CPT, part = at % CPT;
            const int src = CPT == 4 || CPT == 8 ? (part & ~3) | ((part - tok / 8) & 3) : part;
            k_src[i] = (BIG ? tok : tok & 15) * (D / 2) + src * 16;
        }
        // which page: D = 64 has both in one copy, larger rows a page in half the copies
        k_hi = !BIG && D == 64 && lane >= 32;
        v_src = L::v_codes(P, 0) + lane * 16 - (k_hi ? 512 : 0);
        const int part = lane & 3;
        p_hi = !BIG && part >= 2;
        for (int i = 0; i < PC; ++i) {
            const int seg = min(i * 16 + lane / 4, 4 * NG - 1);   // ks, kl of each group, then vs, vl
            p_src[i] = (seg < 2 * NG ? L::k_scale(P, 0) : L::v_scale(P, 0)) + (seg % (2 * NG)) * 2 * P + (BIG ? part : part & 1) * 16;
        }
    }
    __device__ inline uint32_t page_of(int pos) const {
        const uint32_t p = table_entry(table + (min(pos, last) >> log2p));
        return p < (uint32_t)pages ? p : (uint32_t)pages - 1;
    }
    // Starts the copies of the block at t0, whose pages are a (and b, of its second 16 tokens).
    __device__ inline void copy(uint8_t* slot, int t0, uint32_t a, uint32_t b) const {
        const int in = t0 & ((1 << log2p) - 1);   // first token's place in the page
        const uint8_t* pa = data + (int64_t)a * page_bytes;
        const uint8_t* pb = BIG ? pa : data + (int64_t)b * page_bytes;
#pragma unroll
        for (int i = 0; i < KC; ++i) {
            const uint8_t* base = BIG ? pa : D == 64 ? (k_hi ? pb : pa) : i < KC / 2 ? pa : pb;
            lds_copy16(base + (in * (D / 2) + k_src[i]), slot + K_AT + 1024 * i);
        }
#pragma unroll
        for (int i = 0; i < KC; ++i) {
            const uint8_t* base = BIG ? pa : D == 64 ? (k_hi ? pb : pa) : i < KC / 2 ? pa : pb;
            const int i0 = BIG || D == 64 || i < KC / 2 ? i : i - KC / 2;
            lds_copy16(base + (in * (D / 2) + v_src + 1024 * i0), slot + V_AT + 1024 * i);
        }
        const uint8_t* pp = p_hi ? pb : pa;
#pragma unroll
        for (int i = 0; i < PC; ++i)
            if (NG % 4 == 0 || (int)(threadIdx.x & (WAVE - 1)) < 16 * NG)
                lds_copy16(pp + (2 * in + p_src[i]), slot + P_AT + 1024 * i);
    }
    // LDS addresses, past the slot's, of lane (m, kg)'s operand words: K's of token 8 (m / 4) + m % 4
    // (+ 4) and d = 32 i + 8 kg .., V's of tokens 8 kg .. 8 kg + 7 and quad m, and those 8 tokens'
    // scales and lows.
    static __device__ inline uint32_t k_at() {
        const int lane = threadIdx.x & (WAVE - 1), m = lane & 15, kg = lane >> 4, x = m >> 2;
        const int chunk = D == 64 ? 0 : ((D / 128) * kg & ~3) | (((D / 128) * kg + x) & 3);   // D = 256: see k_words
        return K_AT + (x * 8 + (m & 3)) * (D / 2) + (D == 64 ? kg * 8 : chunk * 16);
    }
    static __device__ inline uint32_t v_at() {
        const int lane = threadIdx.x & (WAVE - 1), m = lane & 15, kg = lane >> 4;
        return V_AT + kg * 4 * D + m * 16;
    }
    static __device__ inline uint32_t p_at() { return P_AT + ((threadIdx.x & (WAVE - 1)) >> 4) * 16; }
    // K's words of both halves of the block.
    static __device__ inline void k_words(uint32_t (&w)[2][D / 32], uint32_t at) {
        if constexpr (D == 64) {
            u32x2 x, y;
            lds_read<0, 4 * (D / 2)>(at, x, y);
            w[0][0] = x[0], w[0][1] = x[1], w[1][0] = y[0], w[1][1] = y[1];
        } else {
            // D = 256: the lane's second chunk is one place on, in the same 64 bytes, so the
            // places wrap where x + 2 kg is odd and 3
#pragma unroll
            for (int c = 0; c < D / 128; ++c) {
                const int lane = threadIdx.x & (WAVE - 1), kg = lane >> 4, q = (lane & 15) >> 2;
                const int place = ((D / 128) * kg + q) & 3;
                const uint32_t to = at + (c ? (place == 3 ? -48 : 16) : 0);
                u32x4 x, y;
                lds_read<0, 4 * (D / 2)>(to, x, y);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[0][4 * c + j] = x[j], w[1][4 * c + j] = y[j];
            }
        }
    }
    static __device__ inline void v_words(u32x4 (&w)[D / 64], uint32_t at) {
        if constexpr (D == 64)
            lds_read<0, 0>(at, w[0], w[0]);
        else if constexpr (D == 128)
            lds_read<0, 256>(at, w[0], w[1]);
        else
            lds_read<0, 256, 512, 768>(at, w[0], w[1], w[2], w[3]);
    }
    // Scales and lows of all groups, K's (0) or V's (1).
    template <int WHICH, int GI = 0>
    static __device__ inline void params(u32x4 (&sc)[NG], u32x4 (&low)[NG], uint32_t at) {
        constexpr int O = (WHICH * NG + GI) * 128;
        if constexpr (GI + 1 < NG) {
            lds_read<O, O + 64, O + 128, O + 192>(at, sc[GI], low[GI], sc[GI + 1], low[GI + 1]);
            if constexpr (GI + 2 < NG)
                params<WHICH, GI + 2>(sc, low, at);
        } else {
            lds_read<O, O + 64>(at, sc[GI], low[GI]);
        }
    }
};

// fp16 subnormals of 8 codes, slots in d order: (0, 1) c, (2, 3) 16 c, (4, 5) c, (6, 7) 16 c.
__device__ inline f16x8 codes_raw(uint32_t w) {
    const uint32_t h = w >> 8;
    const u32x4 r = {w & 0x000F000Fu, w & 0x00F000F0u, h & 0x000F000Fu, h & 0x00F000F0u};
    return __builtin_bit_cast(f16x8, r);
}

// Constants of the masks in registers: (w & mask) | 1024 is then one v_and_or_b32 (an instruction
// with three operands takes no literal).
struct Masks {
    uint32_t even, odd, k1024;
    __device__ inline Masks() {
        asm("s_mov_b32 %0, 0x000F000F" : "=s"(even));
        asm("s_mov_b32 %0, 0x00F000F0" : "=s"(odd));
        asm("v_mov_b32 %0, 0x64006400" : "=v"(k1024));
    }
};

// Codes of nibble JJ of each half as fp16 integers: 1024 + c (or 1024 + 16 c) is exact.
template <int JJ>
__device__ inline f16x2 codes_int(uint32_t w, const Masks& mk) {
    const uint32_t h = JJ & 2 ? w >> 8 : w;
    if constexpr (JJ & 1)
        return as_f16x2((h & mk.odd) | mk.k1024) * (f16x2){(_Float16)0.0625f, (_Float16)0.0625f} -
               (f16x2){(_Float16)64.0f, (_Float16)64.0f};
    else
        return as_f16x2((h & mk.even) | mk.k1024) - (f16x2){(_Float16)1024.0f, (_Float16)1024.0f};
}

// v as two fp16 terms: hi rounded to nearest, lo = fp16(v - hi). The factor -1 is kept from the
// compiler's sight so that each difference and its rounding stay one mixed-precision instruction on
// the packed hi; written as a subtraction, hi is converted twice and back once.
__device__ inline void two_terms(const float (&v)[8], f16x8& hi, f16x8& lo) {
    u32x4 h, l;
    float minus = -1.f;
    asm("" : "+s"(minus));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f16x2 a{(_Float16)v[2 * e], (_Float16)v[2 * e + 1]};
        h[e] = as_u32(a);
        asm("" : "+v"(h[e]));
        a = as_f16x2(h[e]);
        l[e] = as_u32(f16x2{(_Float16)fmaf((float)a[0], minus, v[2 * e]),
                            (_Float16)fmaf((float)a[1], minus, v[2 * e + 1])});
    }
    hi = __builtin_bit_cast(f16x8, h);
    lo = __builtin_bit_cast(f16x8, l);
}

// Q's operand of one column, lane kg's d = 32 i + 8 kg + 0 .. 7, from q at `src` (zeros if !ok), and
// for each group the sum of q over it: both 2^e times as large, the operand times `sign`, its slots
// 2, 3, 6 and 7 divided by 16 for codes that stand 16 times as high, the sums times sign 2^-24.
// Returns e. The division rounds to 2^-24, which costs q below 2^-10 bits. Beside others of 1/4 and
// more that is of the order of the fp32 sums' own rounding, and e is 0; a wave with a lane whose q are
// all smaller brings the largest |q| of each column to 2^14 (by 2^30 at most, with which the smallest
// fp16 number is 64). Done in every wave, that took 0.25 us of a call, the look for it 0.1.
template <int D, int G>
__device__ inline int q_column(const _Float16* src, bool ok, float sign, f16x8 (&q)[D / 32], float (&qsum)[D / G]) {
    f16x8 big = {};
#pragma unroll
    for (int g = 0; g < D / G; ++g)
        qsum[g] = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        f16x8 x = {};
        if (ok)
            x = *reinterpret_cast<const f16x8*>(src + 32 * i);
        big = __builtin_elementwise_max(big, __builtin_elementwise_abs(x));
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            s += (float)x[e];
        q[i] = x;
        qsum[i / (G / 32)] += s;
    }
#pragma unroll
    for (int g = 0; g < D / G; ++g) {
        qsum[g] += __shfl_xor(qsum[g], 16, WAVE);
        qsum[g] += __shfl_xor(qsum[g], 32, WAVE);
        qsum[g] *= sign * 5.9604644775390625e-08f;   // 2^-24
    }
    const f16x4 four = __builtin_elementwise_max(__builtin_shufflevector(big, big, 0, 1, 2, 3),
                                                 __builtin_shufflevector(big, big, 4, 5, 6, 7));
    const f16x2 two = __builtin_elementwise_max(__builtin_shufflevector(four, four, 0, 1),
                                                __builtin_shufflevector(four, four, 2, 3));
    float top = fmaxf((float)two[0], (float)two[1]);
    int e = 0;
    if (__any(ok && top < 0.25f)) {
        top = fmaxf(top, __shfl_xor(top, 16, WAVE));
        top = fmaxf(top, __shfl_xor(top, 32, WAVE));
        e = min(max(127 + 14 - (int)(__float_as_uint(top) >> 23), 0), 30);
        const _Float16 a = (_Float16)ldexpf(1.0f, e / 2), b = (_Float16)ldexpf(1.0f, e - e / 2);
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            q[i] = q[i] * (f16x8){a, a, a, a, a, a, a, a} * (f16x8){b, b, b, b, b, b, b, b};
#pragma unroll
        for (int g = 0; g < D / G; ++g)
            qsum[g] = ldexpf(qsum[g], e);
    }
    const _Float16 one = (_Float16)sign, part = (_Float16)(sign * 0.0625f);
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
        q[i] *= (f16x8){one, one, part, part, one, one, part, part};
    return e;
}

// What a score's sums are multiplied by for the softmax in base 2: the codes' 2^-24 and q's 2^e
// taken out. Not 0, so that a hidden score, -inf, keeps its weight of 0 with a scale of 0 too (what
// the bound makes of a smaller scale is still below 2^-50), and not so large that a product (a sum
// is below 2^20) passes fp32: at 1e30, sums that differ in fp32 are far enough apart for a weight of 0.
__device__ inline float to_base2(float scale, int e) {
    return __builtin_amdgcn_fmed3f(ldexpf(fabsf(scale) * 1.44269504088896f, 24 - e), 1e-30f, 1e30f);
}

// A weight, 2^(s kappa - m + P_SHIFT), `shift` the last two. Past 2^22 or so a maximum m is rounded by
// enough that the exact product lies far above it or below: all weights of a row pass fp16, or
// vanish. With CARE the product is rounded as the maximum is.
template <bool CARE>
__device__ inline float weight(float s, float kappa, float m, float shift) {
    if constexpr (CARE) {
#pragma clang fp contract(off)
        const float product = s * kappa;
        return __builtin_amdgcn_exp2f(fminf(product - m, M_SLACK) + P_SHIFT);
    } else {
        return __builtin_amdgcn_exp2f(fmaf(s, kappa, shift));
    }
}

// V's operand for nibble JJ of chunk words w: one d of 8 tokens, scale * code + low in fp16. A stored
// pair goes up to 15 * 65504 + 65504, past fp16 (fp32 rows that large, and pairs of rows near 65504
// whose rounding passes it by up to 32), and an infinite value times another row's weight of 0 is
// NaN. Operands are taken as they are at first; CARE makes them 1 / 16 of every value, which holds
// all that a pair can stand for, low / 16 and the value rounded to multiples of 2^-24 at least.
//
// Steps without CARE leave a sum that is not finite wherever a value or a weight passed fp16, and a
// sum of weights below 2^P_SHIFT where they vanished (the largest is 2^P_SHIFT and more). Such rows
// are gone through again with CARE, and no others pay for it.
template <int JJ, bool CARE>
__device__ inline f16x8 v_values(u32x4 w, u32x4 s, u32x4 l, const Masks& mk) {
    const f16x2 part = {(_Float16)0.0625f, (_Float16)0.0625f};
    u32x4 r;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        f16x2 c = codes_int<JJ>(w[p], mk), low = as_f16x2(l[p]);
        if constexpr (CARE)
            c *= part, low *= part;
        r[p] = as_u32(__builtin_elementwise_fma(c, as_f16x2(s[p]), low));
    }
    return __builtin_bit_cast(f16x8, r);
}
constexpr float CARE_UNIT = 16.0f;

// Whether a column's sums of values are infinite or NaN, or its weights' sum is not what a row that
// has a maximum must have. `sum` is the column's, the same in its lanes.
template <int N, int M>
__device__ inline bool needs_care(const f32x4 (&o)[N][M], const float (&sum)[N], const float (&m)[N]) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < N; ++i)
        bad |= m[i] != M_NONE && !(sum[i] > 32.0f);   // half of 2^P_SHIFT, past all roundings
    float z[4] = {};   // four chains
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < M; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                z[r] = fmaf(o[i][j][r], 0.0f, z[r]);
    return __any(bad || (z[0] + z[1]) + (z[2] + z[3]) != 0.0f);
}

__device__ inline float half_of(u32x4 w, int i) { return (float)as_f16x2(w[i / 2])[i & 1]; }

// Ring slots of a wave: one in use, the other filling. Two let four workgroups of a CU (two of
// D = 256) share its 160 KB of LDS.
constexpr int SLOTS = 2;

template <int D, int G, bool BIG, int NQ>
__global__ __launch_bounds__(AT, NQ == 1 && D <= 128 && G * 2 >= D ? 3 : D == 256 && G == 32 ? 1 : 2) void attention_kv4_decode_kernel(
    Kv4Attn a, Kv4Cache c, Kv4Batch b, Split sp) {
    using RG = Ring<D, G, BIG>;
    constexpr int NG = D / G, NI = D / 32, NC = D / 64, PER = 16 * NQ;
    // the ring, and after the loop the waves' partial results in its place
    constexpr int RING = AW * SLOTS * RG::BYTES, PART = AW * 16 * (D + 4) * 4;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[RING > PART ? RING : PART];
    __shared__ float stats[AW][16][2];
    float(*part)[16][D + 4] = reinterpret_cast<float(*)[16][D + 4]>(lds);
    const int R = a.q_heads / c.heads;
    int id = blockIdx.x;
    const int head = id % c.heads;
    id /= c.heads;
    const int seq = id % b.batch;
    id /= b.batch;
    const int split = id % sp.n;
    const int tile0 = id / sp.n;
    const int lane = threadIdx.x & (WAVE - 1), n = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const Masks mk;
    const float sign = a.scale < 0.0f ? -1.0f : a.scale > 0.0f ? 1.0f : 0.0f;

    for (int tile = tile0;; tile += sp.tiles) {
        const RowTile t = row_tile(b, c, seq, tile, PER, R, a.window);
        if (tile * PER >= t.rows * R)
            return;
        const uint32_t end = t.end, stretch = split_tokens(t, sp.stretch, sp.n);
        const uint32_t from = (uint32_t)(t.begin & ~(TB - 1)) + split * stretch;
        const uint32_t to = from < end ? from + min(stretch, end - from) : from;
        // a split's maximum and sum for one (row, head), behind all splits' sums of values
        auto split_stats = [&](int64_t at) {
            return a.ws + ((int64_t)sp.n * a.rows * a.q_heads * D + (at * sp.n + split) * 2);
        };
        if (split > 0 && from >= end) {
            // no tokens: a sum of 0, whose values nobody reads
            for (int idx = tile * PER + threadIdx.x; idx < min(tile * PER + PER, t.rows * R); idx += AT) {
                const uint32_t row = row_of(b, seq, idx / R);
                if (row < (uint32_t)a.rows) {
                    float* st = split_stats((int64_t)row * a.q_heads + head * R + idx % R);
                    st[0] = M_NONE, st[1] = 0.0f;
                }
            }
            continue;
        }

        const RG ring(b, c, seq, head, t.end);
        uint8_t* slots = lds + wave * (SLOTS * RG::BYTES);
        const uint32_t k_at = lds_addr(slots) + RG::k_at(), v_at = lds_addr(slots) + RG::v_at(),
                       p_at = lds_addr(slots) + RG::p_at();
        uint32_t t0;               // the block in use
        uint32_t pa = 0, pb = 0;   // pages of the block to be copied next
        auto pages = [&](uint32_t pos) {
            if (pos < to) {
                pa = ring.page_of(pos);
                pb = BIG ? pa : ring.page_of(pos + 16);
            }
        };
        auto begin = [&] {
            t0 = from + wave * TB;
#pragma unroll
            for (int i = 0; i < SLOTS; ++i) {
                pages(t0 + i * AW * TB);
                if (t0 + i * AW * TB < to)
                    ring.copy(slots + i * RG::BYTES, t0 + i * AW * TB, pa, pb);
            }
            pages(t0 + SLOTS * AW * TB);
        };
        __syncthreads();   // the last tile's partial results have been read
        begin();

        // Q's operand: column n of each row tile
        f16x8 q[NQ][NI];
        float qsum[NQ][NG], kappa[NQ];
        int rbeg[NQ], rend[NQ];
#pragma unroll
        for (int u = 0; u < NQ; ++u) {
            const int idx = tile * PER + u * 16 + n, i = idx / R;
            const uint32_t row = row_of(b, seq, i);
            const bool ok = i < t.rows && row < (uint32_t)a.rows;
            rend[u] = ok ? max(0, t.first + i + 1) : 0;
            rbeg[u] = a.window ? max(0, rend[u] - a.window) : 0;
            const _Float16* src = a.q + (int64_t)(ok ? row : 0) * a.q_stride + (int64_t)(head * R + idx % R) * D + kg * 8;
            kappa[u] = to_base2(a.scale, q_column<D, G>(src, ok, sign, q[u], qsum[u]));
        }

        f32x4 o[NQ][D / 16], l[NQ];
        float m[NQ];
        const _Float16 one = (_Float16)1.0f;
        const f16x8 ones = {one, one, one, one, one, one, one, one};

        auto step = [&](uint32_t at, auto care) {
            constexpr bool CARE = decltype(care)::value;
            const bool edge = t0 < (uint32_t)t.all_begin || t0 + TB > (uint32_t)t.all_end;   // some row does not see all of it
            f32x4 s[NQ][2];
            uint32_t kw[2][NI];
            u32x4 sc[NG], low[NG];
            RG::k_words(kw, k_at + at);
            RG::template params<0>(sc, low, p_at + at);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    f32x4 acc[NQ];
#pragma unroll
                    for (int u = 0; u < NQ; ++u)
                        acc[u] = f32x4{0, 0, 0, 0};
#pragma unroll
                    for (int i = g * (G / 32); i < (g + 1) * (G / 32); ++i) {
                        const f16x8 kc = codes_raw(kw[h][i]);
#pragma unroll
                        for (int u = 0; u < NQ; ++u)
                            acc[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kc, q[u][i], acc[u], 0, 0, 0);
                    }
#pragma unroll
                    for (int u = 0; u < NQ; ++u)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            s[u][h][r] = fmaf(half_of(low[g], 4 * h + r), qsum[u][g], g ? s[u][h][r] : 0.0f);
                            s[u][h][r] = fmaf(half_of(sc[g], 4 * h + r), acc[u][r], s[u][h][r]);
                        }
                }
            }
            if (edge) {
                // a score below all others at every scale: its weight is exactly 0
                int tb = t0;
                asm volatile("" : "+s"(tb));   // a branch, not selects in every step
#pragma unroll
                for (int u = 0; u < NQ; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int j = tb + kg * 8 + 4 * h + r;
                            s[u][h][r] = j >= rbeg[u] && j < rend[u] ? s[u][h][r] : -INFINITY;
                        }
            }
            f16x8 p[NQ], pl[NQ];
#pragma unroll
            for (int u = 0; u < NQ; ++u) {
                float top = s[u][0][0];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        top = fmaxf(top, s[u][h][r]);
                top *= kappa[u];
                if (__any(top > m[u] + M_SLACK)) {
                    top = fmaxf(top, __shfl_xor(top, 16, WAVE));
                    top = fmaxf(top, __shfl_xor(top, 32, WAVE));
                    const float mn = fmaxf(m[u], top);
                    const float f = __builtin_amdgcn_exp2f(m[u] - mn);
                    m[u] = mn;
                    l[u][0] *= f;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
                        o[u][i] *= f;
                }
                // before a row's first score, 0 in place of the maximum: masked weights stay 0
                const float shift = m[u] > M_NONE ? P_SHIFT - m[u] : 0.0f;
                float w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    w[e] = weight<CARE>(s[u][e / 4][e % 4], kappa[u], m[u], shift);
                two_terms(w, p[u], pl[u]);
                l[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, p[u], l[u], 0, 0, 0);
                l[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, pl[u], l[u], 0, 0, 0);
            }
            u32x4 vs[NG], vl[NG], vw[NC];
            RG::v_words(vw, v_at + at);
            RG::template params<1>(vs, vl, p_at + at);
            if (edge && (t0 < (uint32_t)t.begin || t0 + TB > end)) {
                // what lies at positions that no row sees may be anything: a weight of 0 must
                // not meet an infinite or NaN value
                int tb = t0;
                asm volatile("" : "+s"(tb));
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int j = tb + kg * 8 + 2 * w;
                    const uint32_t keep = (j >= t.begin && j < t.end ? 0xFFFFu : 0u) |
                                          (j + 1 >= t.begin && j + 1 < t.end ? 0xFFFF0000u : 0u);
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        vs[g][w] &= keep;
                        vl[g][w] &= keep;
                    }
                }
            }
#pragma unroll
            for (int ch = 0; ch < NC; ++ch) {
                const int g0 = 64 * ch / G, g1 = (64 * ch + 32) / G;
                const f16x8 vv[4] = {
                    v_values<0, CARE>(vw[ch], vs[g0], vl[g0], mk), v_values<1, CARE>(vw[ch], vs[g0], vl[g0], mk),
                    v_values<2, CARE>(vw[ch], vs[g1], vl[g1], mk), v_values<3, CARE>(vw[ch], vs[g1], vl[g1], mk)};
                // the second terms after all first ones: a product that waits for the one before
                // it on the same sum would stall
                auto add = [&](const f16x8(&w)[NQ]) {
#pragma unroll
                    for (int jj = 0; jj < 4; ++jj)
#pragma unroll
                        for (int u = 0; u < NQ; ++u)
                            o[u][4 * ch + jj] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vv[jj], w[u], o[u][4 * ch + jj], 0, 0, 0);
                };
                add(p);
                add(pl);
            }
        };

        auto walk = [&](auto care) {
#pragma unroll
            for (int u = 0; u < NQ; ++u) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    o[u][i] = f32x4{0, 0, 0, 0};
                l[u] = f32x4{0, 0, 0, 0};
                m[u] = M_NONE;
            }
            for (uint32_t at = 0; t0 < to; t0 += AW * TB) {
                // the block's copies have landed when only the younger slots' are pending
                if (t0 + (SLOTS - 1) * AW * TB < to)
                    __builtin_amdgcn_s_waitcnt(vmcnt_le((SLOTS - 1) * RG::COPIES));
                else
                    __builtin_amdgcn_s_waitcnt(vmcnt_le(0));
                __builtin_amdgcn_sched_barrier(0);
                step(at, care);
                __builtin_amdgcn_sched_barrier(0);
                if (t0 + SLOTS * AW * TB < to)
                    ring.copy(slots + at, t0 + SLOTS * AW * TB, pa, pb);
                pages(t0 + (SLOTS + 1) * AW * TB);
                at = at + RG::BYTES == SLOTS * RG::BYTES ? 0 : at + RG::BYTES;
            }
        };
        walk(std::false_type{});
        float unit = 1.0f, sums[NQ];   // unit: of the wave's sums of values
#pragma unroll
        for (int u = 0; u < NQ; ++u)
            sums[u] = l[u][0];
        if (needs_care(o, sums, m)) {
            begin();   // the last copies have landed and been read
            walk(std::true_type{});
            unit = CARE_UNIT;
        }

        // join the waves: each brings its O to the largest maximum
#pragma unroll
        for (int u = 0; u < NQ; ++u) {
            __syncthreads();
            if (kg == 0) {
                stats[wave][n][0] = m[u];
                stats[wave][n][1] = l[u][0];
            }
            __syncthreads();
            float top = stats[0][n][0];
#pragma unroll
            for (int w = 1; w < AW; ++w)
                top = fmaxf(top, stats[w][n][0]);
            const float f = __builtin_amdgcn_exp2f(m[u] - top) * unit;
#pragma unroll
            for (int ch = 0; ch < NC; ++ch)
#pragma unroll
                for (int jj = 0; jj < 4; ++jj)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        part[wave][n][ch * 64 + (jj >> 1) * 32 + kg * 8 + 2 * r + (jj & 1)] = o[u][4 * ch + jj][r] * f;
            __syncthreads();
            constexpr int E = D / 16;   // values of one thread: row tid / 16, E neighbouring d
            const int rr = threadIdx.x / 16, d0 = (threadIdx.x % 16) * E;
            const int idx = tile * PER + u * 16 + rr, i = idx / R;
            const uint32_t row = row_of(b, seq, i);
            if (i < t.rows && row < (uint32_t)a.rows) {
                float mx = stats[0][rr][0], sum = 0.0f, v[E];
#pragma unroll
                for (int w = 1; w < AW; ++w)
                    mx = fmaxf(mx, stats[w][rr][0]);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    v[e] = 0.0f;
#pragma unroll
                for (int w = 0; w < AW; ++w) {
                    sum += stats[w][rr][1] * __builtin_amdgcn_exp2f(stats[w][rr][0] - mx);
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        v[e] += part[w][rr][d0 + e];
                }
                const int64_t at = (int64_t)row * a.q_heads + head * R + idx % R;
                if (sp.n == 1) {
                    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        a.out[at * D + d0 + e] = (_Float16)(v[e] * inv);
                } else {
                    float* ws = a.ws + ((int64_t)split * a.rows * a.q_heads + at) * D + d0;
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        ws[e] = v[e];
                    if (threadIdx.x % 16 == 0)
                        split_stats(at)[0] = mx, split_stats(at)[1] = sum;
                }
            }
        }
    }
}

// Joins the splits of one (row, head): v = sum_s 2^(m_s - max) v_s over l = sum_s 2^(m_s - max) l_s.
// Two launches' latencies (a split's statistics, then its values) are most of it, so nothing
// else is looked up: splits without tokens have left l = 0. One workgroup for many splits of few
// rows, one wave for a few splits of many (both kernels together, by workgroups and by waves: 1 row
// of 32 heads in 64 splits 41.9 and 43.0 us, 2 rows in 32 splits 18.5 and 19.4, 4 rows in 16 splits
// 18.0 and 18.0, 65 rows of 28 heads in 3 splits 16.7 and 15.7 us). The join of 33 rows of 32 heads in
// 2 splits takes 4.5 us.
constexpr int MAX_SPLITS = 256;

template <int D, int WAVES>
__global__ __launch_bounds__(AT) void attention_kv4_join_kernel(const float* __restrict__ ws, _Float16* __restrict__ out,
                                                                int64_t all, int n) {
    constexpr int LANES = D / 4, PARTS = WAVES * WAVE / LANES, ROWS = AW / WAVES;
    static_assert(PARTS >= 1, "a row's waves hold its values");
    __shared__ float weight[ROWS][WAVES * WAVE], red[AW][2];
    __shared__ f32x4 part[ROWS][PARTS][LANES];
    const int group = threadIdx.x / (WAVES * WAVE), tid = threadIdx.x % (WAVES * WAVE);
    for (int64_t first = (int64_t)blockIdx.x * ROWS; first < all; first += (int64_t)gridDim.x * ROWS) {
        const int64_t at = first + group;
        const float* st = ws + (int64_t)n * all * D + at * n * 2;
        float m = M_NONE, l = 0.0f;
        if (at < all && tid < n) {
            m = st[2 * tid];
            l = st[2 * tid + 1];
        }
        float top = m;
#pragma unroll
        for (int o = WAVE / 2; o > 0; o >>= 1)
            top = fmaxf(top, __shfl_xor(top, o, WAVE));
        if ((tid & (WAVE - 1)) == 0)
            red[threadIdx.x / WAVE][0] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
            top = fmaxf(top, red[group * WAVES + w][0]);
        const float f = l > 0.0f ? __builtin_amdgcn_exp2f(m - top) : 0.0f;
        weight[group][tid] = f;
        float sum = l * f;
#pragma unroll
        for (int o = WAVE / 2; o > 0; o >>= 1)
            sum += __shfl_xor(sum, o, WAVE);
        if ((tid & (WAVE - 1)) == 0)
            red[threadIdx.x / WAVE][1] = sum;
        __syncthreads();
        sum = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
            sum += red[group * WAVES + w][1];
        const int d4 = tid % LANES, p = tid / LANES;
        f32x4 v = {0, 0, 0, 0};
        if (at < all) {
            const float* src = ws + at * D + 4 * d4;
#pragma unroll 4
            for (int s = p; s < n; s += PARTS) {
                const float w = weight[group][s];
                if (w != 0.0f)   // a split without tokens wrote no values
                    v += *reinterpret_cast<const f32x4*>(src + s * all * D) * w;
            }
        }
        part[group][p][d4] = v;
        __syncthreads();
        if (p == 0 && at < all) {
#pragma unroll
            for (int k = 1; k < PARTS; ++k)
                v += part[group][k][d4];
            const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
            _Float16* to = out + at * D + 4 * d4;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                to[e] = (_Float16)(v[e] * inv);
        }
        __syncthreads();   // the shared arrays have been read
    }
}

// Prompt kernel (many rows of a sequence): bound by the matrix cores and the softmax beside them.
// A workgroup of eight waves takes 128 NQ (row, head) pairs, 16 NQ a wave, and steps through the
// tokens in blocks of PB that all its waves share: each thread turns its part of the block's
// codes into operands once, in LDS, in 16-byte units (8 d of a token for K, 8 tokens of one d for
// V, neighbouring lanes' units side by side). As in the decode kernel K's operand is its codes
// and V's its values. A score is
//   sum_g s_tg (sum_{d in g} c q_d) + sum_g low_tg (sum_{d in g} q_d):
// the second sum is a product over groups, taken on the matrix cores too and exactly, with low in
// two bf16 terms (11 bits) and the sums of q in three (24 bits): 6 of the 8 slots of a group, so
// that one product serves 4 groups. A score then costs one fused multiply-add a group.
//
// A block has two phases, products (P V of the block before, then S) and vector work (softmax,
// the operands of the block after next, loads of the one after that). Each SIMD holds a wave of
// either half of the workgroup, and the halves run one phase apart, with a barrier at each
// phase's end: one wave's products run beside the other's vector work. What block j's operands
// overwrite has then been read: K's of block j - 3 (three buffers), V's of j - 4 (four). 2048 rows of
// 8 x 4 heads of 128 after 2048 positions take 180 to 212 us by the card, 575 TFLOP/s of the formula's
// products at 180, or 860 with those of P's second term (a library product of 8192 x 8192 x 8192 reaches
// 1216). Pages of less than a block look each part's page up (4 x 1024 rows of 1024: 77.4 us from pages
// of 16, 76.2 of 64). D = 64, D = 256 in groups of 32 and D = 128 in groups of 32 with two blocks a wave keep
// 2 to 12 registers in scratch, none of them touched in the loop over the blocks.
constexpr int PT = 512;   // threads
constexpr int prompt_block(int D) { return D == 256 ? 32 : 64; }   // tokens of a block: 126 KB of LDS

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Workgroup barrier for LDS alone: loads into registers stay in flight across it.
__device__ inline void phase_end() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// The leading 8 bits of v, a bf16 value.
__device__ inline float bf16_part(float v) { return __uint_as_float(__float_as_uint(v) & 0xFFFF0000u); }
// Six bf16 values and two zeros as an operand's 8 slots.
__device__ inline bf16x8 bf16_terms(float a, float b, float c, float d, float e, float f) {
    auto two = [](float x, float y) { return __float_as_uint(x) >> 16 | (__float_as_uint(y) & 0xFFFF0000u); };
    return __builtin_bit_cast(bf16x8, (u32x4){two(a, b), two(c, d), two(e, f), 0u});
}

// Two workgroups of a CU for D = 64, whose LDS has room for them: 128 registers.
template <int D, int G, bool BIG, int NQ>
__global__ __launch_bounds__(PT, D == 64 ? 4 : 2) void attention_kv4_prompt_kernel(Kv4Attn a, Kv4Cache c, Kv4Batch b, int tiles) {
    using L = Kv4Layout<D, G>;
    constexpr int PB = prompt_block(D), XT = PB / 16, NI = D / 32, NG = D / G, NL = (NG + 3) / 4, PER = 128 * NQ;
    constexpr int PARTS = D * PB / 16;   // threads' parts of a block
    static_assert(PARTS <= PT, "one part a thread");
    __shared__ __attribute__((aligned(16))) f16x8 kt[3][D / 8][PB], vt[4][PB / 8][D];
    __shared__ __attribute__((aligned(16))) u32x4 lowt[3][NG][PB];   // low's terms
    __shared__ __attribute__((aligned(16))) _Float16 sct[3][NG][PB];
    __shared__ int again;   // some wave's columns need care
    const int R = a.q_heads / c.heads, P = 1 << c.page_log2;
    const int tid = threadIdx.x, lane = tid & (WAVE - 1), n = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
    int id = blockIdx.x;
    const int head = id % c.heads;
    id /= c.heads;
    const int seq = id % b.batch;
    // the sequence's last tiles see most: they start first
    const int tile0 = tiles - 1 - id / b.batch;
    const Masks mk;
    const float sign = a.scale < 0.0f ? -1.0f : a.scale > 0.0f ? 1.0f : 0.0f;

    // The thread's part of a block: of K two words, d = 32 (2 j + z) + 8 kgk .., of one token; of V
    // two d, 64 (quad / 16) + 32 half + 2 (quad % 16) + 0, 1, of 8 tokens.
    const int tok = tid % PB, kgk = tid / PB & 3, j = tid / PB >> 2;
    const int place = (tok & ~31) | (tok & 4) << 2 | (tok & 24) >> 1 | (tok & 3);   // its row of the products
    const int quad = tid % (D / 4), half = tid / (D / 4) & 1, t8 = tid / (D / 2);
    const bool mine = PARTS == PT || tid < PARTS;

    for (int tile = tile0;; tile += tiles) {
        const RowTile t = row_tile(b, c, seq, tile, PER, R, a.window);
        if (tile * PER >= t.rows * R)
            return;
        const int from = t.begin & ~(PB - 1), nb = ((uint32_t)(t.end - from) + PB - 1) / PB;

        f16x8 q[NQ][NI];
        bf16x8 ql[NQ][NL];   // lane (n, kg): the terms of the sum of q over group kg (+ 4)
        float kappa[NQ];
        int rbeg[NQ], rend[NQ];
#pragma unroll
        for (int u = 0; u < NQ; ++u) {
            const int idx = tile * PER + (wave * NQ + u) * 16 + n, i = idx / R;
            const uint32_t row = row_of(b, seq, i);
            const bool ok = i < t.rows && row < (uint32_t)a.rows;
            rend[u] = ok ? max(0, t.first + i + 1) : 0;
            rbeg[u] = a.window ? max(0, rend[u] - a.window) : 0;
            const _Float16* src = a.q + (int64_t)(ok ? row : 0) * a.q_stride + (int64_t)(head * R + idx % R) * D + kg * 8;
            float qsum[NG];
            kappa[u] = to_base2(a.scale, q_column<D, G>(src, ok, sign, q[u], qsum));
#pragma unroll
            for (int y = 0; y < NL; ++y) {
                float own = 0.0f;
#pragma unroll
                for (int g = 4 * y; g < NG && g < 4 * y + 4; ++g)
                    own = kg == g - 4 * y ? qsum[g] : own;
                const float q1 = bf16_part(own), q2 = bf16_part(own - q1), q3 = own - q1 - q2;
                ql[u][y] = bf16_terms(q1, q2, q3, q1, q2, q3);
            }
        }
        // positions that all of the wave's rows see
        const int w0 = tile * PER + wave * 16 * NQ, wl = min(w0 + 16 * NQ - 1, t.rows * R - 1);
        const int w_all_end = max(0, t.first + w0 / R + 1);
        const int w_all_begin = a.window ? max(0, max(0, t.first + wl / R + 1) - a.window) : 0;

        f32x4 o[NQ][D / 16];
        f16x8 p[NQ][XT / 2], pl[NQ][XT / 2];
        float m[NQ], l[NQ];   // l: the lane's tokens' part of the weights' sum

        u32x2 kw;
        _Float16 ks[2], kl[2];
        u32x4 vw, vs, vl;
        const int32_t* table = b.table + (int64_t)seq * b.width;
        auto page = [&](int pos, auto uniform) {
            const int32_t* e = table + (min(pos, t.end - 1) >> c.page_log2);
            uint32_t pg = decltype(uniform)::value ? table_entry(e) : (uint32_t)*e;
            pg = pg < (uint32_t)c.pages ? pg : (uint32_t)c.pages - 1;
            return c.data + ((int64_t)pg * c.heads + head) * c.head_bytes;
        };
        // BIG: the block lies in one page
        auto load = [&](int i) {
            const int t0 = from + i * PB, in = t0 & (P - 1);
            if (mine) {
                const uint8_t* pk = BIG ? page(t0, std::true_type{}) : page(t0 + tok, std::false_type{});
                const int slot = BIG ? in + tok : (t0 + tok) & (P - 1);
                kw = *reinterpret_cast<const u32x2*>(pk + (L::k_codes(slot) + (kgk * NI + 2 * j) * 4));
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const int g = (2 * j + z) * 32 / G;
                    ks[z] = *reinterpret_cast<const _Float16*>(pk + (L::k_scale(P, g) + 2 * slot));
                    kl[z] = *reinterpret_cast<const _Float16*>(pk + (L::k_low(P, g) + 2 * slot));
                }
                const uint8_t* pv = BIG ? pk : page(t0 + 8 * t8, std::false_type{});
                const int vslot = BIG ? in + 8 * t8 : (t0 + 8 * t8) & (P - 1);
                vw = *reinterpret_cast<const u32x4*>(pv + (L::v_codes(P, vslot / 8) + quad * 16));
                const int g = (quad / 16 * 64 + half * 32) / G;
                vs = *reinterpret_cast<const u32x4*>(pv + (L::v_scale(P, g) + 2 * vslot));
                vl = *reinterpret_cast<const u32x4*>(pv + (L::v_low(P, g) + 2 * vslot));
            }
        };
        auto put = [&](int i, int kb, int vb, auto care) {
            constexpr bool CARE = decltype(care)::value;
            const int t0 = from + i * PB;
            if (mine) {
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    kt[kb][(2 * j + z) * 4 + kgk][place] = codes_raw(kw[z]);
                    const int g = (2 * j + z) * 32 / G;
                    if (kgk == 0 && (2 * j + z) * 32 % G == 0) {   // one thread a token and group
                        sct[kb][g][tok] = ks[z];
                        const float low = (float)kl[z], l1 = bf16_part(low), l2 = low - l1;
                        lowt[kb][g][place] = __builtin_bit_cast(u32x4, bf16_terms(l1, l1, l1, l2, l2, l2));
                    }
                }
                if (t0 < t.begin || (uint32_t)t0 + PB > (uint32_t)t.end) {
                    // what lies at positions that no row sees may be anything
                    int tb = t0 + 8 * t8;
                    asm volatile("" : "+v"(tb));   // a branch, not selects in every block
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int x = tb + 2 * w;
                        const uint32_t keep = (x >= t.begin && x < t.end ? 0xFFFFu : 0u) |
                                              (x + 1 >= t.begin && x + 1 < t.end ? 0xFFFF0000u : 0u);
                        vs[w] &= keep;
                        vl[w] &= keep;
                    }
                }
                u32x4 w = vw;
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    w[x] >>= 8 * half;
                f16x8* to = &vt[vb][t8][quad / 16 * 64 + half * 32 + quad % 16 * 2];
                to[0] = v_values<0, CARE>(w, vs, vl, mk);
                to[1] = v_values<1, CARE>(w, vs, vl, mk);
            }
        };
        // The operands of the next rows of products are read while the present ones run; the
        // scheduling barriers keep more of them from piling up in registers.
        struct Keys {
            f16x8 k[NI];
            bf16x8 low[NL];
            f16x4 sc[NG];
        };
        auto keys = [&](int kb, int x) {
            Keys f;
#pragma unroll
            for (int y = 0; y < NL; ++y)   // lanes past the last group meet q's zeros
                f.low[y] = __builtin_bit_cast(bf16x8, lowt[kb][min(4 * y + kg, NG - 1)][16 * x + n]);
#pragma unroll
            for (int i = 0; i < NI; ++i)
                f.k[i] = kt[kb][4 * i + kg][16 * x + n];
#pragma unroll
            for (int g = 0; g < NG; ++g)   // scales of tokens 32 (x / 2) + 8 kg + 4 (x % 2) + r
                f.sc[g] = *reinterpret_cast<const f16x4*>(&sct[kb][g][(x >> 1) * 32 + kg * 8 + (x & 1) * 4]);
            return f;
        };
        auto scores = [&](f32x4(&s)[NQ][XT], int kb) {
            Keys f = keys(kb, 0);
#pragma unroll
            for (int x = 0; x < XT; ++x) {
                __builtin_amdgcn_sched_barrier(0);
                Keys next = f;
                if (x + 1 < XT)
                    next = keys(kb, x + 1);
#pragma unroll
                for (int u = 0; u < NQ; ++u)
                    s[u][x] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int y = 0; y < NL; ++y)
#pragma unroll
                    for (int u = 0; u < NQ; ++u)
                        s[u][x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.low[y], ql[u][y], s[u][x], 0, 0, 0);
                f32x4 acc[NG][NQ];
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int i = g * (G / 32); i < (g + 1) * (G / 32); ++i)
#pragma unroll
                        for (int u = 0; u < NQ; ++u)
                            acc[g][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                                f.k[i], q[u][i], i == g * (G / 32) ? f32x4{0, 0, 0, 0} : acc[g][u], 0, 0, 0);
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int u = 0; u < NQ; ++u)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            s[u][x][r] = fmaf((float)f.sc[g][r], acc[g][u][r], s[u][x][r]);
                f = next;
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        auto softmax = [&](f32x4(&s)[NQ][XT], int i, auto care) {
            constexpr bool CARE = decltype(care)::value;
            const int t0 = from + i * PB;
            if (t0 < w_all_begin || (uint32_t)t0 + PB > (uint32_t)w_all_end) {
                int tb = t0;
                asm volatile("" : "+s"(tb));
#pragma unroll
                for (int u = 0; u < NQ; ++u)
#pragma unroll
                    for (int x = 0; x < XT; ++x)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int at = tb + (x >> 1) * 32 + kg * 8 + (x & 1) * 4 + r;
                            s[u][x][r] = at >= rbeg[u] && at < rend[u] ? s[u][x][r] : -INFINITY;
                        }
            }
#pragma unroll
            for (int u = 0; u < NQ; ++u) {
                float top = s[u][0][0];
#pragma unroll
                for (int x = 0; x < XT; ++x)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        top = fmaxf(top, s[u][x][r]);
                top *= kappa[u];
                if (__any(top > m[u] + M_SLACK)) {
                    top = fmaxf(top, __shfl_xor(top, 16, WAVE));
                    top = fmaxf(top, __shfl_xor(top, 32, WAVE));
                    const float mn = fmaxf(m[u], top);
                    const float f = __builtin_amdgcn_exp2f(m[u] - mn);
                    m[u] = mn;
                    l[u] *= f;
#pragma unroll
                    for (int x = 0; x < D / 16; ++x)
                        o[u][x] *= f;
                }
                const float shift = m[u] > M_NONE ? P_SHIFT - m[u] : 0.0f;
#pragma unroll
                for (int y = 0; y < XT / 2; ++y) {
                    float w[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        w[e] = weight<CARE>(s[u][2 * y + e / 4][e % 4], kappa[u], m[u], shift);
                    l[u] += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
                    two_terms(w, p[u][y], pl[u][y]);
                }
            }
            // the weights are done in this phase, not where they are used
#pragma unroll
            for (int u = 0; u < NQ; ++u)
#pragma unroll
                for (int y = 0; y < XT / 2; ++y)
                    asm volatile("" : "+v"(p[u][y]), "+v"(pl[u][y]));
        };
        auto values = [&](int vb) {
            constexpr int STEP = 2;   // of D / 16
            f16x8 f[STEP][XT / 2];
            auto read = [&](f16x8(&to)[STEP][XT / 2], int x0) {
#pragma unroll
                for (int x = 0; x < STEP; ++x)
#pragma unroll
                    for (int y = 0; y < XT / 2; ++y)
                        to[x][y] = vt[vb][4 * y + kg][16 * (x0 + x) + n];
            };
            read(f, 0);
#pragma unroll
            for (int x0 = 0; x0 < D / 16; x0 += STEP) {
                __builtin_amdgcn_sched_barrier(0);
                f16x8 next[STEP][XT / 2];
                if (x0 + STEP < D / 16)
                    read(next, x0 + STEP);
                auto add = [&](const f16x8(&w)[NQ][XT / 2]) {
#pragma unroll
                    for (int y = 0; y < XT / 2; ++y)
#pragma unroll
                        for (int x = 0; x < STEP; ++x)
#pragma unroll
                            for (int u = 0; u < NQ; ++u)
                                o[u][x0 + x] =
                                    __builtin_amdgcn_mfma_f32_16x16x32_f16(f[x][y], w[u][y], o[u][x0 + x], 0, 0, 0);
                };
                add(p);
                add(pl);
#pragma unroll
                for (int x = 0; x < STEP; ++x)
#pragma unroll
                    for (int y = 0; y < XT / 2; ++y)
                        f[x][y] = next[x][y];
            }
            __builtin_amdgcn_sched_barrier(0);
        };

        auto walk = [&](auto care) {
#pragma unroll
            for (int u = 0; u < NQ; ++u) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    o[u][i] = f32x4{0, 0, 0, 0};
                l[u] = 0.0f;
                m[u] = M_NONE;
            }
            if (nb == 0)
                return;
            load(0);
            put(0, 0, 0, care);
            if (nb > 1) {
                load(1);
                put(1, 1, 1, care);
            }
            if (nb > 2)
                load(2);
            phase_end();
            if (wave >= 4)
                phase_end();   // the second half runs one phase behind
            int kb = 0;        // i % 3
#pragma clang loop unroll(disable)
            for (int i = 0; i < nb; ++i) {
                f32x4 s[NQ][XT];
                __builtin_amdgcn_s_setprio(1);
                if (i > 0)
                    values((i - 1) & 3);
                scores(s, kb);
                __builtin_amdgcn_s_setprio(0);
                phase_end();
                softmax(s, i, care);
                if (i + 2 < nb) {
                    put(i + 2, kb == 0 ? 2 : kb - 1, (i + 2) & 3, care);
                    if (i + 3 < nb)
                        load(i + 3);
                }
                phase_end();
                kb = kb == 2 ? 0 : kb + 1;
            }
            values((nb - 1) & 3);
            if (wave < 4)
                phase_end();
        };
        __syncthreads();   // the last tile's blocks have been read, and its `again`
        if (tid == 0)
            again = 0;
        float unit = 1.0f;   // of the sums of values
        walk(std::false_type{});
        if (nb > 0) {
            // the operands are shared, so all waves go again (a barrier at least lies between the
            // walk's start and its end)
            float sums[NQ];
#pragma unroll
            for (int u = 0; u < NQ; ++u) {
                sums[u] = l[u] + __shfl_xor(l[u], 16, WAVE);
                sums[u] += __shfl_xor(sums[u], 32, WAVE);
            }
            if (needs_care(o, sums, m) && lane == 0)
                again = 1;
            __syncthreads();
            if (__builtin_amdgcn_readfirstlane(again)) {
                walk(std::true_type{});
                unit = CARE_UNIT;
            }
        }

#pragma unroll
        for (int u = 0; u < NQ; ++u) {
            const int idx = tile * PER + (wave * NQ + u) * 16 + n, i = idx / R;
            const uint32_t row = row_of(b, seq, i);
            float sum = l[u] + __shfl_xor(l[u], 16, WAVE);
            sum += __shfl_xor(sum, 32, WAVE);
            if (i < t.rows && row < (uint32_t)a.rows) {
                const float inv = sum > 0.0f ? unit / sum : 0.0f;
                _Float16* to = a.out + ((int64_t)row * a.q_heads + head * R + idx % R) * D;
                // o's tile x, register r: d = 16 x + 4 kg + r
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    f16x4 h;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        h[r] = (_Float16)(o[u][x][r] * inv);
                    *reinterpret_cast<f16x4*>(to + 16 * x + 4 * kg) = h;
                }
            }
        }
    }
}

// Workgroups that a call's splits make: two on each CU. In us, 8 x 4 heads, with 256, 512, 768, 1024:
// 1 x 65536 tokens, D = 64 22.2, 19.8, 20.9, 21.2; D = 128 28.0, 26.9, 29.1, 32.6; D = 256 41.9, 43.3,
// 49.1, 54.2 (in groups of 32, one workgroup a CU: 52.9, 63.7, 76.4, 83.3); 33 x 4100 and shorter, D = 64
// 30.4, 26.3, 24.7, 23.1; D = 128 40.0, 35.2, 34.4, 34.4; D = 256 62.4, 57.7, 63.6, 61.4; 8 x 5 rows over
// 8192, D = 128 33.1, 31.5, 37.9, 38.8.
constexpr int64_t FILL = 512;
constexpr int64_t MAX_GROUPS = (int64_t)1 << 22;   // of a launch (threads stay below 2^32); the kernels loop

// Blocks of 16 (row, head) pairs that each wave of the prompt kernel takes, or 0 for the decode
// kernel. Costs in cycles a token of the longest length, as measured on 8 kv heads with 1 and 4 query heads each:
// a round of prompt workgroups, which each hold a CU and are not split over the length, and a decode
// tile of 32 pairs as a share of the whole chip. Rows see `mean` of the longest length on average;
// decode tiles and prompt workgroups past the first round make use of that, a first round lasts as
// long as its longest. In us, one block a wave, two, decode (8 x 4 heads, D = 128): 1 x 2048 rows of 2048
// positions 81, 98, 99; 1 x 2048 of 4096 191, 186, 213; 4 x 1024 of 1024 94, 74, 122; 1 x 512 of 8192
// 237, 332, 146; 16 x 64 of 2048 69, 95, 70. D = 64 in blocks of two gained nowhere, D = 256 has
// registers for one only. The rule counts max_q rows of max_len positions in every sequence: in a
// batch that mixes prompts with single tokens it takes the single tokens for prompts.
inline int prompt_blocks(int64_t pairs, int64_t heads, int D, int max_q, int max_len, int window) {
    const double one = D == 64 ? 30.0 : D == 128 ? 76.0 : 100.0, two = 106.0;
    const double first = D == 64 ? 13.5 : 0.0;   // two workgroups share a CU: a round alone costs more
    const double tile = D == 64 ? 0.043 : D == 128 ? 0.086 : 0.164;
    const double longest = window > 0 ? std::min(max_len, window) : max_len;
    const double mean = std::min(max_len - 0.5 * std::min(max_q, max_len), longest) / longest;
    const auto cost = [&](double round, int64_t per) {
        const int64_t workgroups = heads * ((pairs + per - 1) / per);
        return first + round * std::max(1.0, mean * (double)((workgroups + 255) / 256));
    };
    const double decode = mean * tile * (double)(heads * ((pairs + 31) / 32));
    const double of_one = cost(one, 128), of_two = D == 128 ? cost(two, 256) : of_one;
    return decode <= std::min(of_one, of_two) ? 0 : of_two < of_one ? 2 : 1;
}

// Rows of a decode tile: 16, or 32 where a sequence has more and two tiles' O and Q fit in the
// registers of two waves a SIMD. In us, in tiles of 32 and of 16: 8 x 5 rows of 8 x 4 heads over 8192
// tokens, D = 64 22.7, 24.6; D = 128 31.4, 34.5; D = 256 139, 56; one sequence of 8 rows over 32768,
// which are few tiles either way, D = 128 29.5, 26.8.
inline int rows_per_tile(int64_t pairs, int D) { return pairs <= 16 || D == 256 ? 16 : 32; }

// Splits: two workgroups of four waves a CU fill the chip, so that many in all, each with at
// least 256 tokens, and at most what the second kernel joins. Up to 640 tokens stay whole: the
// join costs what 256 tokens do (32 heads of 128, 512 tokens 9.4 us whole, 10.3 us in halves; 768
// tokens 11.6 and 10.9; 1024 tokens 13.8 us whole, 11.1 us in quarters).
Split plan(int q_heads, int kv_heads, int D, int batch, int max_q, int max_len, int window) {
    const int64_t pairs = (int64_t)max_q * (q_heads / kv_heads);
    constexpr int64_t unit = TB * AW;
    if (window > 0)   // the positions that a sequence's rows see together
        max_len = (int)std::min<int64_t>(max_len, (int64_t)window + max_q);
    Split s;
    const int per = rows_per_tile(pairs, D);
    const int64_t heads = (int64_t)batch * kv_heads;   // at most MAX_GROUPS
    s.tiles = (int)std::min((pairs + per - 1) / per, std::max<int64_t>(1, MAX_GROUPS / std::max<int64_t>(1, heads)));
    const int64_t base = heads * s.tiles;
    int64_t want = base > 0 ? (FILL + base - 1) / base : 1;
    want = want < MAX_SPLITS ? want : MAX_SPLITS;
    int64_t stretch = max_len <= 5 * unit ? max_len : (max_len + want - 1) / want;
    stretch = stretch < 2 * unit ? 2 * unit : (stretch + unit - 1) / unit * unit;
    s.stretch = (uint32_t)stretch;
    s.n = (int)((max_len + stretch - 1) / stretch);
    return s;
}

}  // namespace

int64_t attention_kv4_workspace(int64_t rows, int q_heads, int kv_heads, int D, int batch, int max_q, int max_len,
                                int window) {
    max_q = (int)std::min<int64_t>(max_q, std::max<int64_t>(rows, 1));
    if (prompt_blocks((int64_t)max_q * (q_heads / kv_heads), (int64_t)batch * kv_heads, D, max_q, max_len, window))
        return 0;
    const Split s = plan(q_heads, kv_heads, D, batch, max_q, max_len, window);
    return s.n == 1 ? 0 : s.n * rows * q_heads * (D + 2);
}

extern "C" int ql_attention_kv4_kernel(int64_t rows, int q_heads, int kv_heads, int D, int batch, int max_q, int max_len,
                                       int window) {
    max_q = (int)std::min<int64_t>(max_q, std::max<int64_t>(rows, 1));
    return prompt_blocks((int64_t)max_q * (q_heads / kv_heads), (int64_t)batch * kv_heads, D, max_q, max_len, window);
}

ql_status launch_attention_kv4(const Kv4Attn& a, const Kv4Cache& c, int D, int G, const Kv4Batch& b,
                               hipStream_t stream) {
    const int max_q = std::min(a.max_q, a.rows);
    const int64_t pairs = (int64_t)max_q * (a.q_heads / c.heads);
    const int nq = prompt_blocks(pairs, (int64_t)b.batch * c.heads, D, max_q, a.max_len, a.window);
    if (nq)
        return kv4_dispatch(D, G, [&](auto d, auto g) {
            constexpr int DD = decltype(d)::value, GG = decltype(g)::value;
            const int64_t heads = (int64_t)c.heads * b.batch, rows = 128 * nq;
            const int tiles = (int)std::min((pairs + rows - 1) / rows, std::max<int64_t>(1, MAX_GROUPS / heads));
            const dim3 grid((uint32_t)(heads * tiles));
            const bool big = (1 << c.page_log2) >= prompt_block(DD);
            auto go = [&](auto kernel) { kernel<<<grid, PT, 0, stream>>>(a, c, b, tiles); };
            if (nq == 1) {
                if (big)
                    go(attention_kv4_prompt_kernel<DD, GG, true, 1>);
                else
                    go(attention_kv4_prompt_kernel<DD, GG, false, 1>);
            } else if constexpr (DD == 128) {
                if (big)
                    go(attention_kv4_prompt_kernel<DD, GG, true, 2>);
                else
                    go(attention_kv4_prompt_kernel<DD, GG, false, 2>);
            }
            return launch_status();
        });
    const int per = rows_per_tile(pairs, D);
    const Split sp = plan(a.q_heads, c.heads, D, b.batch, max_q, a.max_len, a.window);
    return kv4_dispatch(D, G, [&](auto d, auto g) {
        constexpr int DD = decltype(d)::value, GG = decltype(g)::value;
        const dim3 grid((uint32_t)((int64_t)c.heads * b.batch * sp.n * sp.tiles));
        auto go = [&](auto kernel) { kernel<<<grid, AT, 0, stream>>>(a, c, b, sp); };
        if (per == 16) {
            if (c.page_log2 >= 5)
                go(attention_kv4_decode_kernel<DD, GG, true, 1>);
            else
                go(attention_kv4_decode_kernel<DD, GG, false, 1>);
        } else if constexpr (DD < 256) {
            if (c.page_log2 >= 5)
                go(attention_kv4_decode_kernel<DD, GG, true, 2>);
            else
                go(attention_kv4_decode_kernel<DD, GG, false, 2>);
        }
        if (sp.n > 1) {
            const int64_t all = (int64_t)a.rows * a.q_heads, most = MAX_GROUPS;
            if (sp.n > 16)
                attention_kv4_join_kernel<DD, AW>
                    <<<dim3((uint32_t)std::min(all, most)), AT, 0, stream>>>(a.ws, a.out, all, sp.n);
            else
                attention_kv4_join_kernel<DD, 1>
                    <<<dim3((uint32_t)std::min((all + AW - 1) / AW, most)), AT, 0, stream>>>(a.ws, a.out, all, sp.n);
        }
        return launch_status();
    });
}

}  // namespace ql
