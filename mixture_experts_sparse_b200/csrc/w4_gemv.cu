// Expert FFN on 4-bit weights for few rows per expert: matrix-vector work, bound
// by the one read of the weights of every expert that has rows.
//
//   stage 1: H = relu(x W1^T + b1), or silu(x W1^T + b1) * (x W3^T + b3)
//   stage 2: y = H W2^T + b2              W[o][k] = q[o][k] s[o][k / G]
//
// A warp holds 16 output features and streams their packed rows from global
// memory into registers, a block of 128 weights per row and step, D steps ahead;
// the 16 bytes of a lane are, word by word, the A fragments of mma.sync m16n8k16
// (w4.cuh), decoded to bf16 exactly as integers.  The tokens are the 8 columns,
// so a tile is fed at one instruction per 2048 weights and eight tokens; what
// bounds the loop is decoding (11 operations per 8 weights), still below the
// rate at which HBM delivers them.  (A 128-row tcgen05 tile would be decoded
// through shared memory or TMEM for the same few columns.)  The integer products
// of a group are exact in the fp32 accumulator; the group's scale multiplies the
// sum, once per row and group, in fp32.
// The warps of a CTA take interleaved blocks of K and add their sums in order
// through shared memory: no atomics, the same bits each time.
// H keeps two bf16 parts, its rounding and the remainder (16 bits): the second
// product costs one more mma per fragment, of which there are few, and the
// output then has one rounding that matters.
#include "w4.cuh"

namespace moe {
namespace {

constexpr int kGemvWarps = 8;
constexpr int kGemvThreads = 32 * kGemvWarps;

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ldg_stream(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

struct GemvParams {
    const int32_t* offsets; int N; int64_t R_cap;
    int m_dim;                    // output features
    int k_dim;
    W4Mat wa, wb;                 // wb: W3 (SwiGLU stage 1)
    const __nv_bfloat16* bias_a; const __nv_bfloat16* bias_b;
    const __nv_bfloat16* x; const __nv_bfloat16* x_lo;   // [R, k_dim]
    __nv_bfloat16* out; __nv_bfloat16* out_lo;           // [R, m_dim]
};

enum { W4_RELU = 0, W4_SWIGLU = 1, W4_OUT = 2 };

// MATS: weight matrices (2: SwiGLU).  One step: 16 rows x 128 weights of each.
template <int MATS>
struct Step {
    uint4 w[MATS][2];        // rows g and g + 8, this lane's 16 bytes
    uint16_t s[MATS][2];     // scales of the group that holds word `t` of the block
};

template <int MATS, int G>
__device__ __forceinline__ void load_step(Step<MATS>& st, const uint8_t* const (&q)[MATS], const uint16_t* const (&s)[MATS],
                                          int64_t pitch, int m_dim, int kb, int nb, int ng, int t) {
    if (kb < nb) {
        const int g = min(kb * (kW4Block / G) + t * (kW4Block / G) / 4, ng - 1);   // past the last group: zero weights
#pragma unroll
        for (int i = 0; i < MATS; ++i) {
            st.w[i][0] = ldg_stream(q[i] + kb * kW4BlockBytes);
            st.w[i][1] = ldg_stream(q[i] + 8 * pitch + kb * kW4BlockBytes);
            st.s[i][0] = __ldg(s[i] + (int64_t)g * m_dim);
            st.s[i][1] = __ldg(s[i] + (int64_t)g * m_dim + 8);
        }
    }
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int j) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; }

// Rows [row0, row0 + n) of x times 16 features: acc += this warp's blocks of K.
template <int EPI, int G, int NT>
__device__ __forceinline__ void gemv_unit(const GemvParams& p, int e, int m0, int64_t row0, int n, float* s_red) {
    constexpr int MATS = EPI == W4_SWIGLU ? 2 : 1;
    constexpr bool HILO = EPI == W4_OUT;
    constexpr int D = NT == 1 ? (MATS == 2 ? 4 : 6) : 3;   // steps in flight
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int nb = (p.k_dim + kW4Block - 1) / kW4Block, ng = (p.k_dim + G - 1) / G;
    const int64_t pitch = (int64_t)nb * kW4BlockBytes;
    const uint8_t* q[MATS];
    const uint16_t* s[MATS];
#pragma unroll
    for (int i = 0; i < MATS; ++i) {
        const W4Mat& m = i == 0 ? p.wa : p.wb;
        q[i] = m.q + ((int64_t)e * p.m_dim + m0 + g) * pitch + 16 * t;
        s[i] = m.s + (int64_t)e * ng * p.m_dim + m0 + g;
    }
    float acc[MATS][NT][4];
#pragma unroll
    for (int i = 0; i < MATS; ++i)
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][c][j] = 0.f;
    Step<MATS> ring[D];
#pragma unroll
    for (int i = 0; i < D; ++i) load_step<MATS, G>(ring[i], q, s, pitch, p.m_dim, warp + i * kGemvWarps, nb, ng, t);
    const __nv_bfloat16* xr = p.x + (row0 + g) * p.k_dim + 8 * t;
    const __nv_bfloat16* xl = HILO ? p.x_lo + (row0 + g) * p.k_dim + 8 * t : nullptr;
    for (int base = warp; base < nb; base += D * kGemvWarps) {
#pragma unroll
        for (int i = 0; i < D; ++i) {
            const int kb = base + i * kGemvWarps;
            if (kb < nb) {
                Step<MATS>& st = ring[i];
                float part[MATS][NT][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if ((j * (kW4Block / G)) % 4 == 0) {   // word j starts a group
#pragma unroll
                        for (int m = 0; m < MATS; ++m)
#pragma unroll
                            for (int c = 0; c < NT; ++c)
#pragma unroll
                                for (int r = 0; r < 4; ++r) part[m][c][r] = 0.f;
                    }
                    const int k0 = kb * kW4Block + 32 * j;
                    uint4 b[NT], bl[HILO ? NT : 1];
#pragma unroll
                    for (int c = 0; c < NT; ++c) {
                        const bool ok = 8 * c + g < n && k0 + 8 * t < p.k_dim;
                        b[c] = ok ? __ldg(reinterpret_cast<const uint4*>(xr + (int64_t)8 * c * p.k_dim + k0))
                                  : make_uint4(0, 0, 0, 0);
                        if (HILO)
                            bl[c] = ok ? __ldg(reinterpret_cast<const uint4*>(xl + (int64_t)8 * c * p.k_dim + k0))
                                       : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int m = 0; m < MATS; ++m) {
                        const uint32_t w0 = word_of(st.w[m][0], j), w1 = word_of(st.w[m][1], j);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t a0 = w4_pair(w0, 2 * h), a1 = w4_pair(w1, 2 * h);
                            const uint32_t a2 = w4_pair(w0, 2 * h + 1), a3 = w4_pair(w1, 2 * h + 1);
#pragma unroll
                            for (int c = 0; c < NT; ++c) {
                                mma16816(part[m][c], a0, a1, a2, a3, h ? b[c].z : b[c].x, h ? b[c].w : b[c].y);
                                if (HILO)
                                    mma16816(part[m][c], a0, a1, a2, a3, h ? bl[c].z : bl[c].x, h ? bl[c].w : bl[c].y);
                            }
                        }
                    }
                    if (((j + 1) * (kW4Block / G)) % 4 == 0) {   // word j ends a group
#pragma unroll
                        for (int m = 0; m < MATS; ++m) {
                            uint32_t u0 = st.s[m][0], u1 = st.s[m][1];
                            if (G < kW4Block) {   // the lane of the quad that loaded this group's scale
                                u0 = __shfl_sync(0xffffffffu, u0, (lane & ~3) | j);
                                u1 = __shfl_sync(0xffffffffu, u1, (lane & ~3) | j);
                            }
                            const float f0 = __uint_as_float(u0 << 16), f1 = __uint_as_float(u1 << 16);
#pragma unroll
                            for (int c = 0; c < NT; ++c) {
                                acc[m][c][0] = fmaf(part[m][c][0], f0, acc[m][c][0]);
                                acc[m][c][1] = fmaf(part[m][c][1], f0, acc[m][c][1]);
                                acc[m][c][2] = fmaf(part[m][c][2], f1, acc[m][c][2]);
                                acc[m][c][3] = fmaf(part[m][c][3], f1, acc[m][c][3]);
                            }
                        }
                    }
                }
                load_step<MATS, G>(st, q, s, pitch, p.m_dim, kb + D * kGemvWarps, nb, ng, t);
            }
        }
    }
    // warps in order: s_red[warp][matrix][column][feature]
    constexpr int TILE = 16 * 8 * NT;
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                s_red[(warp * MATS + m) * TILE + (8 * c + 2 * t + (r & 1)) * 16 + g + 8 * (r >> 1)] = acc[m][c][r];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * n; i += kGemvThreads) {
        const int col = i >> 4, f = i & 15, feat = m0 + f;
        float v[MATS];
#pragma unroll
        for (int m = 0; m < MATS; ++m) {
            v[m] = 0.f;
#pragma unroll
            for (int w = 0; w < kGemvWarps; ++w) v[m] += s_red[(w * MATS + m) * TILE + col * 16 + f];
        }
        const __nv_bfloat16* ba = p.bias_a ? p.bias_a + (int64_t)e * p.m_dim + feat : nullptr;
        if (ba) v[0] += __bfloat162float(*ba);
        float o = v[0];
        if (EPI == W4_RELU) o = o < 0.f ? 0.f : o;   // NaN stays
        if (EPI == W4_SWIGLU) {
            if (p.bias_b) v[MATS - 1] += __bfloat162float(p.bias_b[(int64_t)e * p.m_dim + feat]);
            o = o / (1.f + fast_exp2(-o * kLog2e)) * v[MATS - 1];
        }
        const __nv_bfloat16 hi = __float2bfloat16_rn(o);
        p.out[(row0 + col) * p.m_dim + feat] = hi;
        if (EPI != W4_OUT) p.out_lo[(row0 + col) * p.m_dim + feat] = __float2bfloat16_rn(o - __bfloat162float(hi));
    }
    __syncthreads();
}

template <int EPI, int G>
__global__ void __launch_bounds__(kGemvThreads, 2)
w4_gemv_kernel(const GemvParams p) {
    constexpr int MATS = EPI == W4_SWIGLU ? 2 : 1;
    __shared__ float s_red[kGemvWarps * MATS * 16 * 16];
    __shared__ int s_row[129], s_exp[128], s_live;
    const int tid = threadIdx.x;
    if (EPI != W4_OUT) {
        pdl_wait();
        pdl_launch();
    }
    // Stage 2 starts while stage 1 drains: the offsets are inputs of both, so they
    // are read before the wait.
    for (int i = tid; i <= p.N; i += kGemvThreads) {
        const int64_t v = p.offsets[i];
        s_row[i] = (int)(v < 0 ? 0 : (v > p.R_cap ? p.R_cap : v));
    }
    __syncthreads();
    if (tid == 0) {
        int c = 0;
        for (int e = 0; e < p.N; ++e)
            if (s_row[e + 1] > s_row[e]) s_exp[c++] = e;
        s_live = c;
    }
    __syncthreads();
    if (EPI == W4_OUT) {
        pdl_wait();
        pdl_launch();
    }
    const int tiles = p.m_dim / 16;
    const int64_t units = (int64_t)s_live * tiles;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int e = s_exp[u / tiles], m0 = (int)(u % tiles) * 16;
        const int r1 = s_row[e + 1];
        for (int r = s_row[e]; r < r1;) {
            const int left = r1 - r;
            if (left <= 8) {
                gemv_unit<EPI, G, 1>(p, e, m0, r, left, s_red);
                r += 8;
            } else {
                gemv_unit<EPI, G, 2>(p, e, m0, r, min(left, 16), s_red);
                r += 16;
            }
        }
    }
}

template <int EPI>
cudaError_t run_gemv(const GemvParams& p, int group, int sms, cudaStream_t s) {
    const dim3 grid((unsigned)(2 * sms)), block(kGemvThreads);
    if (group == 32) return launch_k(w4_gemv_kernel<EPI, 32>, grid, block, 0, s, 1, p);
    if (group == 64) return launch_k(w4_gemv_kernel<EPI, 64>, grid, block, 0, s, 1, p);
    return launch_k(w4_gemv_kernel<EPI, 128>, grid, block, 0, s, 1, p);
}

}  // namespace

cudaError_t launch_w4_ffn(const W4FfnArgs& a, cudaStream_t s) {
    int sms = 0;
    cudaError_t err = device_sm_count(&sms);
    if (err != cudaSuccess) return err;
    GemvParams p{};
    p.offsets = a.offsets;
    p.N = a.N;
    p.R_cap = a.R_cap;
    p.m_dim = a.d_ff;
    p.k_dim = a.d;
    p.wa = a.w1;
    p.wb = a.w3;
    p.bias_a = a.b1;
    p.bias_b = a.b3;
    p.x = a.xe;
    p.out = a.h;
    p.out_lo = a.h_lo;
    err = a.act == MOE_SWIGLU ? run_gemv<W4_SWIGLU>(p, a.group, sms, s) : run_gemv<W4_RELU>(p, a.group, sms, s);
    if (err != cudaSuccess) return err;
    p.m_dim = a.d;
    p.k_dim = a.d_ff;
    p.wa = a.w2;
    p.bias_a = a.b2;
    p.bias_b = nullptr;
    p.x = a.h;
    p.x_lo = a.h_lo;
    p.out = a.ye;
    p.out_lo = nullptr;
    return run_gemv<W4_OUT>(p, a.group, sms, s);
}

}  // namespace moe
