// 4-bit quantisation of weight matrices with a scale per group of G weights of a
// row, and back.
//   scale = bf16(max |w| / 7),  q = rint(w / scale) in [-7, 7],  value = q scale.
// Both are decided exactly, whatever a quotient in fp32 rounds to, so the result is
// that of real arithmetic with ties to even.  For q: r = rint(w / s) from an
// approximate quotient is at most one off, and the residual w - r s is exact in one
// fma (r s has 12 bits, and what is left of w is a multiple of its last place and
// below s); r is right iff |w - r s| < s / 2, and only the lanes' 8 weights for which
// that fails, ties among them, take the long way.  A group of zeros has scale 0; a
// group with an infinity or NaN has scale NaN and stands for NaN as a whole.
//
// Bound by HBM: one read of the weights, half a byte plus 2 / G written each; with a
// division per weight the kernel was bound by its instructions (172 us for 117 M
// bf16 weights, where their bytes take 46).  A lane owns eight consecutive weights
// (one word of the packed row), sixteen lanes a block of 128; several blocks are in
// flight per lane.
#include "w4.cuh"

namespace moe {
namespace {

constexpr int kQuantThreads = 256;
constexpr int kQuantRows = kQuantThreads / 16;   // one row per 16 lanes
constexpr int kQuantBlocks = 4;                  // consecutive 128-blocks per lane

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
    v[0] = bf16lo(a.x); v[1] = bf16hi(a.x); v[2] = bf16lo(a.y); v[3] = bf16hi(a.y);
    v[4] = bf16lo(a.z); v[5] = bf16hi(a.z); v[6] = bf16lo(a.w); v[7] = bf16hi(a.w);
}

// max |w| / 7 to bf16, nearest even, of the real quotient
__device__ __forceinline__ uint16_t group_scale(uint32_t max_bits) {
    if (max_bits >= 0x7F800000u) return 0x7FC0u;
    const float m = __uint_as_float(max_bits), t = m / 7.f;
    const uint32_t b = __float_as_uint(t);
    if ((b & 0xFFFFu) == 0x8000u) {   // the fp32 quotient is a tie: the residual says where the real one lies
        const float r = fmaf(-t, 7.f, m);
        return (uint16_t)((b >> 16) + (r > 0.f ? 1u : (r < 0.f ? 0u : (b >> 16) & 1u)));
    }
    return __bfloat16_as_ushort(__float2bfloat16_rn(t));
}

// r = rint(t) of an approximate quotient t of w / s, put right and clamped
__device__ __forceinline__ float settle(float w, float s, float r) {
    const float d = fmaf(-r, s, w), a = fabsf(d), h = 0.5f * s;
    if (a > h || (a == h && ((int)r & 1))) r += copysignf(1.f, d);
    return fminf(fmaxf(r, -7.f), 7.f);
}

// A word of eight weights with scale s (finite, not 0), m their group's largest magnitude.
__device__ __forceinline__ uint32_t quant8(const float (&v)[8], float s, float m) {
    constexpr float kRound = 12582912.f;   // 1.5 2^23: adding it rounds to an integer, ties to even
    const float inv = __fdividef(1.f, s);
    float r[8], worst = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        r[j] = fmaf(v[j], inv, kRound) - kRound;
        worst = fmaxf(worst, fabsf(fmaf(-r[j], s, v[j])));
    }
    if (worst >= 0.5f * s) {   // a tie among the eight, or one that the quotient's error moved
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = settle(v[j], s, r[j]);
    }
    // tiny scales: the reciprocal flushes, and the scale's own rounding can take m / s past 7.5
    if (s < 1e-36f || m > 7.5f * s) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = settle(v[j], s, fabsf(v[j] / s) < 100.f ? rintf(v[j] / s) : copysignf(7.f, v[j]));
    }
    // weight 2 p + odd in bits 4 p + 16 odd: from the top, sixteen times what is there plus the next code,
    // each with kRound's bits, whose sum over the places is taken off at the end
    uint32_t word = 0, off = 0;
#pragma unroll
    for (int n = 7; n >= 0; --n) {
        const int j = n < 4 ? 2 * n : 2 * (n - 4) + 1;
        word = word * 16u + __float_as_uint(r[j] + (kRound + 8.f));
        off = off * 16u + 0x4B400000u;
    }
    return word - off;
}

template <typename T, int G>
__global__ void __launch_bounds__(kQuantThreads)
w4_quantize_kernel(const T* __restrict__ w, uint8_t* __restrict__ q, uint16_t* __restrict__ scale, int64_t all_rows,
                   int64_t rows, int k) {
    const int l = threadIdx.x & 15;
    const int64_t r = (int64_t)blockIdx.x * kQuantRows + (threadIdx.x >> 4);   // row of all matrices
    const int b0 = blockIdx.y * kQuantBlocks, nb = (k + kW4Block - 1) / kW4Block, ng = (k + G - 1) / G;
    pdl_wait();
    pdl_launch();
    const bool live = r < all_rows;
    const T* src = w + r * k + 8 * l;
    float v[kQuantBlocks][8];
#pragma unroll
    for (int i = 0; i < kQuantBlocks; ++i) {
        const int k0 = (b0 + i) * kW4Block;
        if (live && k0 + 8 * l < k) {
            load8(src + k0, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        }
    }
    const int64_t mat = r / rows, row = r - mat * rows;
#pragma unroll
    for (int i = 0; i < kQuantBlocks; ++i) {
        // the group's largest magnitude, compared as bits: NaN above infinity above all numbers
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = G / 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const int b = b0 + i;
        if (!live || b >= nb) continue;
        const uint16_t sb = group_scale(m);
        const float s = __uint_as_float((uint32_t)sb << 16);
        const bool zero = m >= 0x7F800000u || s == 0.f;
        const uint32_t word = zero ? 0x88888888u : quant8(v[i], s, __uint_as_float(m));
        *reinterpret_cast<uint32_t*>(q + r * ((int64_t)nb * kW4BlockBytes) + b * kW4BlockBytes +
                                     4 * (4 * (l & 3) + (l >> 2))) = word;
        const int g = (b * kW4Block + 8 * l) / G;
        if ((8 * l) % G == 0 && g < ng) scale[(mat * ng + g) * rows + row] = sb;
    }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&v)[8]) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&v)[8]) {
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                   pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
}

template <typename T, int G>
__global__ void __launch_bounds__(kQuantThreads)
w4_dequantize_kernel(const uint8_t* __restrict__ q, const uint16_t* __restrict__ scale, T* __restrict__ w,
                     int64_t all_rows, int64_t rows, int k) {
    const int l = threadIdx.x & 15;
    const int64_t r = (int64_t)blockIdx.x * kQuantRows + (threadIdx.x >> 4);
    const int b0 = blockIdx.y * kQuantBlocks, nb = (k + kW4Block - 1) / kW4Block, ng = (k + G - 1) / G;
    pdl_wait();
    pdl_launch();
    if (r >= all_rows) return;
    const int64_t mat = r / rows, row = r - mat * rows;
    uint32_t word[kQuantBlocks];
    uint16_t sb[kQuantBlocks];
#pragma unroll
    for (int i = 0; i < kQuantBlocks; ++i) {
        const int b = b0 + i, k0 = b * kW4Block + 8 * l;
        word[i] = 0;
        sb[i] = 0;
        if (k0 < k) {
            word[i] = __ldcs(reinterpret_cast<const uint32_t*>(q + r * ((int64_t)nb * kW4BlockBytes) + b * kW4BlockBytes +
                                                               4 * (4 * (l & 3) + (l >> 2))));
            sb[i] = __ldg(scale + (mat * ng + k0 / G) * rows + row);
        }
    }
#pragma unroll
    for (int i = 0; i < kQuantBlocks; ++i) {
        const int k0 = (b0 + i) * kW4Block + 8 * l;
        if (k0 >= k) continue;
        const float s = __uint_as_float((uint32_t)sb[i] << 16);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = (float)((int)((word[i] >> (4 * (j >> 1) + 16 * (j & 1))) & 15u) - 8) * s;
        store8(w + r * k + k0, v);
    }
}

template <typename T, int G>
cudaError_t run(bool back, int64_t mats, int64_t rows, int64_t k, const void* w, uint8_t* q, uint16_t* scale,
                cudaStream_t s) {
    const int64_t all = mats * rows;
    const dim3 grid((unsigned)((all + kQuantRows - 1) / kQuantRows),
                    (unsigned)((w4_blocks(k) + kQuantBlocks - 1) / kQuantBlocks));
    if (back)
        return launch_k(w4_dequantize_kernel<T, G>, grid, dim3(kQuantThreads), 0, s, 1, static_cast<const uint8_t*>(q),
                        static_cast<const uint16_t*>(scale), static_cast<T*>(const_cast<void*>(w)), all, rows, (int)k);
    return launch_k(w4_quantize_kernel<T, G>, grid, dim3(kQuantThreads), 0, s, 1, static_cast<const T*>(w), q, scale,
                    all, rows, (int)k);
}

template <typename T>
cudaError_t run_group(bool back, int64_t mats, int64_t rows, int64_t k, int group, const void* w, uint8_t* q,
                      uint16_t* scale, cudaStream_t s) {
    if (mats == 0 || rows == 0) return cudaSuccess;
    if (group == 32) return run<T, 32>(back, mats, rows, k, w, q, scale, s);
    if (group == 64) return run<T, 64>(back, mats, rows, k, w, q, scale, s);
    return run<T, 128>(back, mats, rows, k, w, q, scale, s);
}

}  // namespace

cudaError_t launch_w4_quantize(int64_t mats, int64_t rows, int64_t k, int group, int dtype, const void* w, uint8_t* q,
                               uint16_t* scale, cudaStream_t s) {
    return dtype == MOE_BF16 ? run_group<__nv_bfloat16>(false, mats, rows, k, group, w, q, scale, s)
                             : run_group<float>(false, mats, rows, k, group, w, q, scale, s);
}

cudaError_t launch_w4_dequantize(int64_t mats, int64_t rows, int64_t k, int group, int dtype, const uint8_t* q,
                                 const uint16_t* scale, void* w, cudaStream_t s) {
    uint8_t* qq = const_cast<uint8_t*>(q);
    uint16_t* ss = const_cast<uint16_t*>(scale);
    return dtype == MOE_BF16 ? run_group<__nv_bfloat16>(true, mats, rows, k, group, w, qq, ss, s)
                             : run_group<float>(true, mats, rows, k, group, w, qq, ss, s);
}

}  // namespace moe
