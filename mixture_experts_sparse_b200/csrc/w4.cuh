// 4-bit weights with group scales: layout and decoding (internal header).
//
// A row of K weights is cut into blocks of 128, 64 bytes each (the last block is
// padded with zero weights).  Word 4 t + j (t, j = 0..3) of a block holds its
// weights k = 32 j + 8 t .. + 7, as q + 8 in 4 bits: k + 2 i in bits 4 i, k + 2 i + 1
// in bits 16 + 4 i.  So (a) the 16 bytes that lane t of a quad loads give, word
// by word, the A fragments of m16n8k16 for 32 consecutive k -- a group scale
// never cuts a fragment, and the matching B fragment is 16 consecutive bytes of
// the token's row; (b) one shift, one logic operation and one subtraction
// decode an adjacent pair.
// Scales are bf16, [matrix][group][row]: the scales of a tile's rows are adjacent.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kW4Block = 128;        // weights per block
constexpr int kW4BlockBytes = 64;

inline int64_t w4_blocks(int64_t k) { return (k + kW4Block - 1) / kW4Block; }
inline int64_t w4_row_bytes(int64_t k) { return w4_blocks(k) * kW4BlockBytes; }

struct W4Mat {            // one weight matrix per expert: [N][rows][K]
    const uint8_t* q;     // [N][rows][w4_row_bytes(K)]
    const uint16_t* s;    // [N][groups][rows] bf16
};

// Weights 2 p and 2 p + 1 of the word's eight as a bf16 pair: 128 + (q + 8) is
// exact in bf16 (0x4300 is 128, whose last place is 1), and so is the difference.
__device__ __forceinline__ uint32_t w4_pair(uint32_t w, int p) {
    uint32_t u;   // (w >> 4 p & mask) | magic in one operation (two immediates would make it two)
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(u) : "r"(w >> (4 * p)), "r"(0x000F000Fu), "r"(0x43004300u));
    const uint32_t c = 0x43084308u;   // 136, 136
    __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u), *reinterpret_cast<const __nv_bfloat162*>(&c));
    return *reinterpret_cast<uint32_t*>(&r);
}

struct W4FfnArgs {
    int act; int N; int d; int d_ff; int group; int64_t R_cap;
    const __nv_bfloat16* xe; const int32_t* offsets;
    W4Mat w1, w3, w2;
    const __nv_bfloat16* b1; const __nv_bfloat16* b3; const __nv_bfloat16* b2;
    __nv_bfloat16* h;      // [R_cap, d_ff]
    __nv_bfloat16* h_lo;   // [R_cap, d_ff]: what h's rounding left (few rows)
    __nv_bfloat16* ye;     // [R_cap, d]
    float* part;           // w4_part_bytes(): sums of tiles that CTAs share
    int32_t* count;        // [2][kW4Counters], zero between calls
    WsHeader* hdr;
};
int w4_gemv_ctas(int sms);
int64_t w4_part_bytes();
cudaError_t launch_w4_quantize(int64_t mats, int64_t rows, int64_t k, int group, int dtype, const void* w, uint8_t* q,
                               uint16_t* scale, cudaStream_t s);
cudaError_t launch_w4_dequantize(int64_t mats, int64_t rows, int64_t k, int group, int dtype, const uint8_t* q,
                                 const uint16_t* scale, void* w, cudaStream_t s);
cudaError_t launch_w4_ffn(const W4FfnArgs& a, cudaStream_t s);

}  // namespace moe
