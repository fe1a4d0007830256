// kv4.h -- layout of the paged 4-bit K/V cache and the rows of a batch, shared by the kernels
// that write, read and attend over it.
//
// A page holds P tokens (a power of two, 16 or more) of one kv head as P * (D + 8 D / G) bytes:
//   K codes   [P][4][D / 32] words: word (kg, i) of a token holds d = 32 i + 8 kg + e, e = 0..7,
//             element e in bits [b, b + 3], b = 16 (e & 1) + 4 (e >> 1)
//   K scales  [D / G][2][P] fp16: for each group of G values the tokens' scales, then lows
//   V codes   [P / 8][D / 4][8] 16-bit: for each token quad n of chunk c holds
//             d = 64 c + 2 n + {0, 1, 32, 33} in bits 0, 4, 8 and 12
//   V scales  as K's
// and a value is scale * code + low. The order is the one the matrix cores' operands want:
// masking a 32-bit word with 0x000F000F (0x00F000F0; the same after a shift by 8) leaves a pair
// of neighbouring k slots as fp16 integers, for K two neighbouring d of one token, for V one d of
// two neighbouring tokens, and a lane's words of one operand are contiguous.
#pragma once

#include "ql_internal.h"

namespace ql {

// The batch: sequence b has the rows starts[b] .. starts[b + 1] of `rows`, its last positions.
struct Kv4Batch {
    const int32_t* table;    // [batch][width] page numbers
    const int32_t* lens;     // [batch] lengths, the rows included
    const int32_t* starts;   // [batch + 1]
    int batch, width, rows;
};

struct Kv4Cache {
    uint8_t* data;
    int64_t head_bytes;   // bytes of one page and head
    int pages, heads, page_log2;
};

// Length of a sequence, kept within what its row of the table can hold.
__device__ inline int kv4_len(const Kv4Batch& b, const Kv4Cache& c, int seq) {
    const int64_t room = (int64_t)b.width << c.page_log2;
    const int n = b.lens[seq];
    return n < 0 ? 0 : n > room ? (int)room : n;
}

// Sequence of a row: the last one that starts at or before it.
__device__ inline int kv4_seq(const Kv4Batch& b, int row) {
    int lo = 0, hi = b.batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (b.starts[mid] <= row)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Position of a row in its sequence; negative where the sequence is shorter than its rows.
__device__ inline int kv4_pos(const Kv4Batch& b, int seq, int len, int row) {
    return len - (b.starts[seq + 1] - row);
}

// Page of position `pos` (0 <= pos < kv4_len): its base address for one head. Numbers outside
// the cache are taken as its last page, so that no access leaves the array.
__device__ inline uint8_t* kv4_page(const Kv4Batch& b, const Kv4Cache& c, int seq, int pos, int head) {
    uint32_t p = (uint32_t)b.table[(int64_t)seq * b.width + (pos >> c.page_log2)];
    p = p < (uint32_t)c.pages ? p : (uint32_t)c.pages - 1;
    return c.data + ((int64_t)p * c.heads + head) * c.head_bytes;
}

// Byte offsets in a page of P tokens.
template <int D, int G>
struct Kv4Layout {
    static constexpr int NG = D / G;
    static __host__ __device__ inline int64_t bytes(int P) { return (int64_t)P * (D + 8 * NG); }
    static __device__ inline int k_codes(int slot) { return slot * (D / 2); }
    static __device__ inline int k_scale(int P, int g) { return P * (D / 2) + g * 4 * P; }
    static __device__ inline int k_low(int P, int g) { return k_scale(P, g) + 2 * P; }
    static __device__ inline int v_codes(int P, int t8) { return P * (D / 2 + 4 * NG) + t8 * (4 * D); }
    static __device__ inline int v_scale(int P, int g) { return P * (D + 4 * NG) + g * 4 * P; }
    static __device__ inline int v_low(int P, int g) { return v_scale(P, g) + 2 * P; }
};

// Calls f with the head size and group as compile-time numbers; QL_ERR_SHAPE for others.
template <class F>
inline ql_status kv4_dispatch(int D, int G, F f) {
    auto by_group = [&](auto d) {
        constexpr int DD = decltype(d)::value;
        switch (G) {
        case 32:
            return f(d, std::integral_constant<int, 32>{});
        case 64:
            return f(d, std::integral_constant<int, 64>{});
        case 128:
            if constexpr (DD >= 128)
                return f(d, std::integral_constant<int, 128>{});
        }
        return QL_ERR_SHAPE;
    };
    switch (D) {
    case 64:
        return by_group(std::integral_constant<int, 64>{});
    case 128:
        return by_group(std::integral_constant<int, 128>{});
    case 256:
        return by_group(std::integral_constant<int, 256>{});
    }
    return QL_ERR_SHAPE;
}

ql_status launch_kv4_append(const void* k, const void* v, bool f16, int64_t k_stride, int64_t v_stride, int64_t rows,
                            const Kv4Cache& c, int D, int G, const Kv4Batch& b, hipStream_t stream);
ql_status launch_kv4_read(const Kv4Cache& c, int D, int G, const Kv4Batch& b, int64_t rows, void* k_out, void* v_out,
                          bool f16, hipStream_t stream);

// Causal attention of `rows` query rows over the cache.
struct Kv4Attn {
    const _Float16* q;   // row r, head h at q + r * q_stride + h * D
    int64_t q_stride;
    _Float16* out;       // [rows][q_heads][D]
    int rows, q_heads;
    int max_q, max_len;  // sizes of the launch; any true sizes give the same results
    float scale;
    int window;          // 0: none
    float* ws;           // split partials
    int64_t ws_floats;
};
// Floats of workspace that launch_attention_kv4 uses for these sizes.
int64_t attention_kv4_workspace(int64_t rows, int q_heads, int kv_heads, int D, int batch, int max_q, int max_len,
                                int window);
// Kernel of launch_attention_kv4 for these sizes: 0 decode, 1 or 2 prompt with as many blocks of 16
// (row, head) pairs a wave. For tests; not part of the interface.
extern "C" int ql_attention_kv4_kernel(int64_t rows, int q_heads, int kv_heads, int D, int batch, int max_q, int max_len,
                                       int window);
ql_status launch_attention_kv4(const Kv4Attn& a, const Kv4Cache& c, int D, int G, const Kv4Batch& b,
                               hipStream_t stream);

}  // namespace ql
