// attention_kv4.hip -- causal attention over the paged 4-bit K/V cache.
//
//   o = sum_j softmax_j(scale * q . k_j) v_j   over the positions j that the row sees,
//   max(0, p - window + 1) <= j <= p for a row at position p (from 0 without a window)
//
// in one pass with a running maximum and sum. A row that sees nothing gives zeros.
#include "kv4.h"

namespace ql {
namespace {

constexpr int AT = 256;   // threads per workgroup, tokens per step

template <int D, int G>
__global__ __launch_bounds__(AT) void attention_kv4_row_kernel(Kv4Attn a, Kv4Cache c, Kv4Batch b) {
    using L = Kv4Layout<D, G>;
    constexpr int PARTS = AT / D;   // parts of a step's tokens, each summed by D threads
    __shared__ float qs[D], prob[AT], red[AT / WAVE], part[AT];
    const int P = 1 << c.page_log2, tid = threadIdx.x;
    const int row = blockIdx.x / a.q_heads, qh = blockIdx.x % a.q_heads;
    const int head = qh / (a.q_heads / c.heads);
    const int seq = kv4_seq(b, row), len = kv4_len(b, c, seq), pos = kv4_pos(b, seq, len, row);
    const int end = pos >= len ? 0 : pos + 1;
    const int begin = a.window && end > a.window ? end - a.window : 0;

    if (tid < D)
        qs[tid] = (float)a.q[row * a.q_stride + (int64_t)qh * D + tid];
    __syncthreads();
    float m = -INFINITY, sum = 0.0f, acc = 0.0f;
    for (int j0 = begin; j0 < end; j0 += AT) {
        const int j = j0 + tid;
        float s = -INFINITY;
        if (j < end) {
            const uint8_t* page = kv4_page(b, c, seq, j, head);
            const int slot = j & (P - 1);
            const uint32_t* kw = reinterpret_cast<const uint32_t*>(page + L::k_codes(slot));
            float dot = 0.0f;
            for (int g = 0; g < L::NG; ++g) {
                float qc = 0.0f, q1 = 0.0f;
                for (int d = g * G; d < g * G + G; d += 8) {
                    const uint32_t w = kw[((d % 32) / 8) * (D / 32) + d / 32];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        qc = fmaf(qs[d + e], (float)((w >> (16 * (e & 1) + 4 * (e >> 1))) & 15), qc);
                        q1 += qs[d + e];
                    }
                }
                dot = fmaf((float)reinterpret_cast<const _Float16*>(page + L::k_scale(P, g))[slot], qc, dot);
                dot = fmaf((float)reinterpret_cast<const _Float16*>(page + L::k_low(P, g))[slot], q1, dot);
            }
            s = dot * a.scale;
        }
        float top = s;
        for (int o = WAVE / 2; o > 0; o >>= 1)
            top = fmaxf(top, __shfl_xor(top, o, WAVE));
        __syncthreads();
        if ((tid & (WAVE - 1)) == 0)
            red[tid / WAVE] = top;
        __syncthreads();
        float mn = m;
        for (int i = 0; i < AT / WAVE; ++i)
            mn = fmaxf(mn, red[i]);
        const float keep = __expf(m - mn);   // 0 at the first step (m = -inf, mn finite)
        prob[tid] = __expf(s - mn);
        m = mn;
        __syncthreads();
        sum *= keep;
        acc *= keep;
        const int d = tid % D, n = min(AT, end - j0);
        const int g = d / G, quad = (d / 64) * 16 + (d % 32) / 2;
        for (int i = 0; i < n; ++i)
            sum += prob[i];
        for (int i = tid / D; i < n; i += PARTS) {
            const uint8_t* page = kv4_page(b, c, seq, j0 + i, head);
            const int slot = (j0 + i) & (P - 1);
            const uint32_t byte = page[L::v_codes(P, slot / 8) + quad * 16 + (slot % 8) * 2 + (d % 64) / 32];
            const float vs = (float)reinterpret_cast<const _Float16*>(page + L::v_scale(P, g))[slot];
            const float vl = (float)reinterpret_cast<const _Float16*>(page + L::v_low(P, g))[slot];
            acc = fmaf(prob[i], fmaf(vs, (float)((byte >> (4 * (d & 1))) & 15), vl), acc);
        }
    }
    part[tid] = acc;
    __syncthreads();
    if (tid < D) {
        for (int i = 1; i < PARTS; ++i)
            acc += part[i * D + tid];
        a.out[(int64_t)blockIdx.x * D + tid] = (_Float16)(end > begin ? acc / sum : 0.0f);
    }
}

}  // namespace

int64_t attention_kv4_workspace(int64_t, int, int, int, int, int, int) { return 0; }

ql_status launch_attention_kv4(const Kv4Attn& a, const Kv4Cache& c, int D, int G, const Kv4Batch& b,
                               hipStream_t stream) {
    return kv4_dispatch(D, G, [&](auto d, auto g) {
        constexpr int DD = decltype(d)::value, GG = decltype(g)::value;
        attention_kv4_row_kernel<DD, GG><<<dim3((uint32_t)(a.rows * a.q_heads)), AT, 0, stream>>>(a, c, b);
        return launch_status();
    });
}

}  // namespace ql
