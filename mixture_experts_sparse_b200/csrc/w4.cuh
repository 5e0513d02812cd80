// 4-bit weights with group scales: layout (internal header).
//
// A row of K weights is cut into blocks of 128, 64 bytes each (the last block is
// padded with zero weights).  Word 4 t + j (t, j = 0..3) of a block holds its
// weights k = 32 j + 8 t .. + 7, as q + 8 in 4 bits: k + 2 i in bits 4 i, k + 2 i + 1
// in bits 16 + 4 i.  So (a) the 16 bytes that lane t of a quad loads give, word
// by word, the A fragments of m16n8k32 for 32 consecutive k, and a group scale
// never cuts a fragment; (b) the even and the odd nibbles of a word, as the upper
// halves of four bytes each, are 16 q in two's complement after one exclusive or;
// (c) one logic operation on the word, or on it shifted by 8, gives an adjacent pair as fp16.
// Scales are bf16, [matrix][group][row]: the scales of a tile's rows are adjacent.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kW4Block = 128;        // weights per block
constexpr int kW4BlockBytes = 64;
constexpr int kW4Counters = 512;     // arrival counters of a few-row launch, one per CTA

inline int64_t w4_blocks(int64_t k) { return (k + kW4Block - 1) / kW4Block; }
inline int64_t w4_row_bytes(int64_t k) { return w4_blocks(k) * kW4BlockBytes; }

struct W4Mat {            // one weight matrix per expert: [N][rows][K]
    const uint8_t* q;     // [N][rows][w4_row_bytes(K)]
    const uint16_t* s;    // [N][groups][rows] bf16
};

// Rows of activations for the few-row kernels: blocks of 64 or 128 values as 16-bit
// integers X = rint(v / unit) with their own unit, max |v| / 32512, held as two
// signed bytes, X = 256 hi + lo.  64 values are 128 bytes, hi then lo; 64 bytes
// are the B fragments of two k-steps: for t, j = 0..3, 0..1 the eight values k =
// 32 j + 8 t .. + 7 at 16 t + 8 j, in the order 0 4 1 5 2 6 3 7 of the words'
// nibbles.  Rows are padded to 256 values; units are fp32 [R][padded / 64] (a block of
// 128 has its unit twice), divided by 16 (the weights' bytes are 16 q) and by 2^12 (range).  A block that holds a
// NaN or infinity has unit NaN; a block whose largest magnitude is below 2^-100 counts as 0.
constexpr int kW4ActBlock = 64;
inline __host__ __device__ int64_t w4_padded(int64_t k) { return (k + 255) / 256 * 256; }

struct W4FfnArgs {
    int act; int N; int d; int d_ff; int group; int64_t R_cap;
    const __nv_bfloat16* xe; const int32_t* offsets;
    W4Mat w1, w3, w2;
    const __nv_bfloat16* b1; const __nv_bfloat16* b3; const __nv_bfloat16* b2;
    uint8_t* xq;           // [R_cap][w4_padded(d)] x 2 bytes: xe as integers
    float* xu;             // [R_cap][w4_padded(d) / 64]: their units
    uint8_t* hq;           // [R_cap][w4_padded(d_ff)] x 2 bytes: H
    float* hu;
    void* h;               // many rows: H as fp16 [R_cap, d_ff]; x as fp16 is in xq, exponents in xu and hu
    int8_t* wexp;          // [N, d_ff] twice and [N, d]: the weight rows' exponents
    int32_t* top;          // [4][N]
    __nv_bfloat16* ye;     // [R_cap, d]
    float* part;           // w4_part_bytes(): sums of tiles that CTAs share
    int32_t* count;        // [2][kW4Counters], cleared by every call
    WsHeader* hdr;
};
int w4_gemv_ctas(int sms);
int64_t w4_part_bytes();
cudaError_t launch_w4_quantize(int64_t mats, int64_t rows, int64_t k, int group, int dtype, const void* w, uint8_t* q,
                               uint16_t* scale, cudaStream_t s);
cudaError_t launch_w4_dequantize(int64_t mats, int64_t rows, int64_t k, int group, int dtype, const uint8_t* q,
                                 const uint16_t* scale, void* w, cudaStream_t s);
cudaError_t launch_w4_ffn(const W4FfnArgs& a, cudaStream_t s);      // chooses by the rows per expert
cudaError_t launch_w4_ffn_tc(const W4FfnArgs& a, cudaStream_t s);   // many rows (w4_tc.cu)

}  // namespace moe
