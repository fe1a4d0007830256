// e4m3_block.h -- E4M3 codes with a scale for each block of 128: what the quantizers, the product
// and the mixture-of-experts layer share.
//
//   activations  codes [M][K], scales [blocks of K][M]: a block's scales of neighbouring rows are
//                contiguous, as a tile of rows reads them
//   weights      codes [N][K], scales [blocks of N][blocks of K], one for 128 x 128 codes
//
// The last block of K or N may be short.
#pragma once

#include "ql_internal.h"

namespace ql {

constexpr int QB = 128;   // values of a block

__host__ __device__ inline int64_t e4m3_blocks(int64_t n) { return (n + QB - 1) / QB; }

typedef __attribute__((address_space(3))) void* lds_addr;

// 16 bytes per lane from a buffer straight into LDS: lane l's bytes land at l * 16 past the
// wave-uniform LDS address; lanes whose offset is past the descriptor's size bring zeros. AUX 2:
// data that is read once (non-temporal).
template <int AUX = 0>
__device__ inline void buffer_to_lds16(__amdgpu_buffer_rsrc_t r, int voff, int soff, int8_t* lds) {
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_addr)lds, 16, voff, soff, 0, AUX);
#endif
}

// 4 bytes per lane from global memory straight into LDS, lane l's at l * 4.
__device__ inline void global_to_lds4(const void* g, int8_t* lds) {
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_global_load_lds(g, (lds_addr)lds, 4, 0, 0);
#endif
}

__device__ inline __amdgpu_buffer_rsrc_t buffer_of(const void* p, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00020000);
}

// The experts' codes are loaded non-temporally (AUX 2) where their rows are whole lines of 128 bytes. Else a
// line holds codes of two blocks, and is worth keeping until the second is read. The layer, us, non-temporal /
// kept, at T, E, top_k, K, I: 64 64 6 2048 1408 120.4 / 126.7, 5 8 2 4096 7168 94.6 / 101.1 (whole lines);
// 64 60 6 1984 1344 129.3 / 126.3, 5 8 2 4160 7232 114.7 / 112.6 (halves); 8 60 4 2048 1344 57.4 / 59.2 and with
// each kernel by its own rows 53.4. The few-row product has another rule, stated at it; the tiles read W
// once for every tile of rows, and keep it.
inline __host__ __device__ bool whole_lines(int row_bytes) { return row_bytes % 128 == 0; }

// s_waitcnt immediates: at most n vector-memory operations pending, LDS operations left alone;
// and no LDS operation pending, vector memory left alone.
constexpr int wait_vm(int n) { return (n & 0xF) | (0x7 << 4) | (0xF << 8) | (((n >> 4) & 3) << 14); }
constexpr int WAIT_LDS = wait_vm(63) & ~(0xF << 8);

// In LDS, chunk c (16 bytes) of a 128-byte row r lies at chunk position c ^ swizzle128(r), so that
// the rows that one fragment read touches fall into distinct banks.
__device__ inline int swizzle128(int r) { return (r & 7) ^ ((r >> 3) & 1); }

// Lane l's chunk in a copy of 8 rows x 128 bytes to LDS, for rows that start at a multiple of 16
// (half 0) or 8 past one (half 1).
__device__ inline int copy_chunk128(int lane, int half) { return (lane & 7) ^ ((lane >> 3) & 7) ^ half; }

ql_status launch_quant_rows_block_e4m3(const void* x, bool x_f16, int64_t M, int64_t K, uint8_t* xq, float* x_scale,
                                       hipStream_t stream);
ql_status launch_quant_weight_block_e4m3(const float* w, int64_t E, int64_t N, int64_t K, uint8_t* wq, float* w_scale,
                                         hipStream_t stream);
ql_status launch_gemm_e4m3_block(const uint8_t* xq, const float* x_scale, const uint8_t* wq, const float* w_scale,
                                 const float* bias, int act, void* y, bool y_f16, int64_t M, int64_t N, int64_t K,
                                 hipStream_t stream);

// Kernel of launch_gemm_e4m3_block for these sizes, by its number there. For tests; not part of the interface.
extern "C" int ql_gemm_e4m3_block_kernel(int64_t M, int64_t N, int64_t K);

// A mixture-of-experts layer; see moe_e4m3_block in ql.h.
struct MoeLayer {
    const _Float16* x;      // [T][K]
    const float* logits;    // [T][E]
    const uint8_t* w13;     // [E][2 I][K]
    const float* s13;
    const uint8_t* w2;      // [E][K][I]
    const float* s2;
    void* out;              // [T][K]
    int8_t* ws;
    int64_t T;
    int E, top_k, K, I;
    bool renormalize, out_f16;
};
constexpr int MOE_TOKENS = 64;     // of a launch
constexpr int MOE_EXPERTS = 512;   // at most
constexpr int MOE_TOP_K = 16;      // at most
int64_t moe_workspace(int64_t T, int top_k, int K, int I);
ql_status launch_moe_router(const void* x, const void* w, float* logits, int64_t T, int64_t E, int64_t K,
                            hipStream_t stream);
ql_status launch_moe_e4m3_block(const MoeLayer& l, hipStream_t stream);

}  // namespace ql
