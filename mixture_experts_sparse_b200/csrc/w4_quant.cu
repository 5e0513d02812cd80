// 4-bit quantisation of weight matrices with a scale per group of G weights of a
// row, and back.
//   scale = bf16(max |w| / 7),  q = rint(w / scale) in [-7, 7],  value = q scale.
// Both are decided exactly, whatever a quotient in fp32 rounds to, so the result is
// that of real arithmetic with ties to even.  Of fp32 weights: r = rint(w / s) from an
// approximate quotient is at most one off, and the residual w - r s is exact in one fma
// (r s has 12 bits, and what is left of w is a multiple of its last place and below
// s); r is right iff |w - r s| < s / 2, and only lanes where that fails for one of
// their eight weights, ties among them, take the long way.  bf16 weights leave room
// between a tie and the next quotient, so rounding twice decides them.  A group of zeros
// has scale 0; a group with an infinity or NaN has scale NaN and stands for NaN as a whole.
//
// Bound by HBM in principle: one read of the weights, half a byte plus 2 / G written
// each.  117 M bf16 weights take 74 us (46 at the copy rate) and 50 back; with a
// division per weight the kernel was bound by its instructions and took 172.  A lane
// owns eight consecutive weights (one word of the packed row), sixteen lanes a block of
// 128; several blocks are in flight per lane.
#include "w4.cuh"

namespace moe {
namespace {

constexpr int kQuantThreads = 256;
constexpr int kQuantRows = kQuantThreads / 16;   // one row per 16 lanes
// Consecutive 128-blocks per lane: 64 bytes of weights in flight.  117 M bf16 weights there and
// back take 130 / 111 / 120 / 111 us at 2 / 4 / 6 / 8 blocks, 5.2 M fp32 ones 15.7 / 19.1 at 2 / 4.
template <typename T> constexpr int kBlocksOf = 8 / (int)sizeof(T);

// eight weights as they lie in memory, their values and their largest magnitude's bits
// (compared as integers: NaN above infinity above all numbers)
template <typename T> struct Eight;
template <> struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void load(const float* p) {
        a = __ldcs(reinterpret_cast<const float4*>(p));
        b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void values(float (&v)[8]) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
    template <int Lanes>
    __device__ __forceinline__ uint32_t largest() const {   // over the Lanes lanes of a group
        float v[8];
        values(v);
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = Lanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        return m;
    }
};
template <> struct Eight<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void values(float (&v)[8]) const {
        v[0] = bf16lo(a.x); v[1] = bf16hi(a.x); v[2] = bf16lo(a.y); v[3] = bf16hi(a.y);
        v[4] = bf16lo(a.z); v[5] = bf16hi(a.z); v[6] = bf16lo(a.w); v[7] = bf16hi(a.w);
    }
    template <int Lanes>
    __device__ __forceinline__ uint32_t largest() const {
        constexpr uint32_t kAbs = 0x7FFF7FFFu;
        uint32_t m = __vmaxu2(__vmaxu2(a.x & kAbs, a.y & kAbs), __vmaxu2(a.z & kAbs, a.w & kAbs));
        m = max(m & 0xFFFFu, m >> 16) << 16;
#pragma unroll
        for (int o = Lanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        return m;
    }
};

// max |w| / 7 to bf16, nearest even, of the real quotient.  Of a bf16 weight, whose eight
// bits are never seven times the nine of a tie but at least 2^-12 away, the fp32 product
// with 1 / 7 decides.
template <typename T>
__device__ __forceinline__ uint16_t group_scale(uint32_t max_bits) {
    if (max_bits >= 0x7F800000u) return 0x7FC0u;
    const float m = __uint_as_float(max_bits);
    if (sizeof(T) == 2 && m > 1e-30f) return __bfloat16_as_ushort(__float2bfloat16_rn(m * (1.f / 7.f)));
    const float t = m / 7.f;
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
template <typename T>
__device__ __forceinline__ uint32_t quant8(const float (&v)[8], float s, float m) {
    constexpr float kRound = 12582912.f;   // 1.5 2^23: adding it rounds to an integer, ties to even
    const float inv = __fdividef(1.f, s);
    float r[8];
    if (sizeof(T) == 2) {
        // w and s have eight bits each, so w / s is k + 1/2 or at least 2^-10 from it: to multiples
        // of 2^-12 first (1.5 2^11), which puts a tie back in its place and moves nothing else across
        constexpr float kSnap = 1.5f * 2048.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = fmaf(v[j], inv, kSnap) - kSnap;
    } else {
        float worst = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            r[j] = fmaf(v[j], inv, kRound) - kRound;
            worst = fmaxf(worst, fabsf(fmaf(-r[j], s, v[j])));
        }
        if (worst >= 0.5f * s) {   // a tie among the eight, or one that the quotient's error moved
#pragma unroll
            for (int j = 0; j < 8; ++j) r[j] = settle(v[j], s, r[j]);
        }
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

// the matrix of row r; the 64-bit division costs as much as a block of weights
__device__ __forceinline__ int64_t matrix_of(int64_t r, int64_t rows, int64_t all_rows) {
    return all_rows <= 0xFFFFFFFFll ? (int64_t)((uint32_t)r / (uint32_t)rows) : r / rows;
}

template <typename T, int G>
__global__ void __launch_bounds__(kQuantThreads)
w4_quantize_kernel(const T* __restrict__ w, uint8_t* __restrict__ q, uint16_t* __restrict__ scale, int64_t all_rows,
                   int64_t rows, int k) {
    constexpr int kQuantBlocks = kBlocksOf<T>;
    const int l = threadIdx.x & 15;
    const int64_t r = (int64_t)blockIdx.x * kQuantRows + (threadIdx.x >> 4);   // row of all matrices
    const int b0 = blockIdx.y * kQuantBlocks, nb = (k + kW4Block - 1) / kW4Block, ng = (k + G - 1) / G;
    pdl_wait();
    pdl_launch();
    const bool live = r < all_rows;
    const T* src = w + r * k + 8 * l;
    Eight<T> raw[kQuantBlocks];
#pragma unroll
    for (int i = 0; i < kQuantBlocks; ++i) {
        const int k0 = (b0 + i) * kW4Block;
        if (live && k0 + 8 * l < k) raw[i].load(src + k0);
        else raw[i].zero();
    }
    const int64_t mat = matrix_of(r, rows, all_rows), row = r - mat * rows;
    uint8_t* dst = q + (r * nb + b0) * kW4BlockBytes + 4 * (4 * (l & 3) + (l >> 2));
    const int g0 = b0 * (kW4Block / G) + 8 * l / G;
    uint16_t* sc = scale + (mat * ng + g0) * rows + row;
#pragma unroll
    for (int i = 0; i < kQuantBlocks; ++i) {
        const uint32_t m = raw[i].template largest<G / 8>();
        if (!live || b0 + i >= nb) continue;
        const uint16_t sb = group_scale<T>(m);
        const float s = __uint_as_float((uint32_t)sb << 16);
        float v[8];
        raw[i].values(v);
        const uint32_t word =
            m >= 0x7F800000u || s == 0.f ? 0x88888888u : quant8<T>(v, s, __uint_as_float(m));
        *reinterpret_cast<uint32_t*>(dst + i * kW4BlockBytes) = word;
        if ((8 * l) % G == 0 && g0 + i * (kW4Block / G) < ng) sc[(int64_t)i * (kW4Block / G) * rows] = sb;
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
    constexpr int kQuantBlocks = kBlocksOf<T>;
    const int l = threadIdx.x & 15;
    const int64_t r = (int64_t)blockIdx.x * kQuantRows + (threadIdx.x >> 4);
    const int b0 = blockIdx.y * kQuantBlocks, nb = (k + kW4Block - 1) / kW4Block, ng = (k + G - 1) / G;
    pdl_wait();
    pdl_launch();
    if (r >= all_rows) return;
    const int64_t mat = matrix_of(r, rows, all_rows), row = r - mat * rows;
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
    constexpr int kQuantBlocks = kBlocksOf<T>;
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
