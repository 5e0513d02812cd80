// Load-balancing loss, per-expert counts and router z-loss over the sequences of
// a padded batch, and their gradient with respect to the router logits.
//
// Tokens t of sequence s (rows [seqs[s], seqs[s+1])), mask m_t in {0, 1},
// p_t = softmax(h_t), lse_t = log sum_e exp h_te, n_s = sum m_t, n = sum_s n_s,
// S' = sequences with n_s > 0:
//   counts[s][e] = #{(t, r) : m_t = 1, idx[t][r] = e},  f = counts / (k n_s),
//   P[s][e] = (1 / n_s) sum_t m_t p_te,
//   loss[0] = alpha N / S' sum_s sum_e f P,   loss[1] = z_coef / n sum_t m_t lse_t^2.
// With one sequence, no mask and k = 1 loss[0] is the layer's own alpha N sum f P
// ("From Switch Transformer to GLaM", Load balancing); counting all k choices
// is that rule for top-k gates.  f is a count and has no gradient (CMU 10-423
// Lecture 16, section 4.2), so with upstream gradients g0, g1
//   dL/dh_tj = m_t p_tj (a_sj - sum_i p_ti a_si + g1 2 z_coef lse_t / n),
//   a_sj = g0 alpha N f_sj / (S' n_s).
//
// Both passes are bound by HBM: the forward reads the logits and choices once,
// the backward reads the logits again (the loss of the whole batch comes before
// any gradient) and writes the gradient.  A row is held by L lanes, 4 C values
// each, so the softmax needs log2 L shuffles and no shared memory.
//
// Forward: a CTA owns a tile of consecutive tokens and walks the sequences that
// cut it.  The share of (tile b, sequence s) goes to slot b + s of the
// workspace: both indexes only grow along the tokens, so no two shares meet,
// and a reducer finds its sequence's shares without a list.  Sums of p run in
// fp32 over a lane's own tokens, then in fixed order (warp tree, warps, tiles in
// fp64); counts are integers.  Nothing depends on the order of arrival.
#include <math_constants.h>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kBalThreads = 256;
constexpr int kBalWarps = kBalThreads / 32;

// e^z for z <= 0 to about an ulp: z log2 e in two parts, 2^hi in one MUFU and
// the low part to first order.  Below -120 the result is 0 (fp32 underflow);
// NaN stays NaN.
__device__ __forceinline__ float exp_neg(float z) {
    z = z < -120.f ? -120.f : z;
    const float t = z * kLog2e;
    const float r = fmaf(z, 1.9259629911e-8f, fmaf(z, kLog2e, -t));   // log2 e - fp32(log2 e)
    const float y = fast_exp2(t);
    return fmaf(y * 0.69314718056f, r, y);
}

// L lanes share a row, lane l holds 4 C columns: VEC, four consecutive ones at
// 4 (l + L c); otherwise l + L j (any alignment, coalesced).
template <int L, int C, bool VEC>
__device__ __forceinline__ int col_of(int l, int c, int i) {
    return VEC ? 4 * (l + L * c) + i : l + L * (4 * c + i);
}

template <typename T> struct Quad;
template <> struct Quad<float> {
    using type = float4;
    static __device__ __forceinline__ void unpack(const float4& q, float* v) {
        v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    }
    static __device__ __forceinline__ float4 pack(const float* v) { return make_float4(v[0], v[1], v[2], v[3]); }
};
template <> struct Quad<__nv_bfloat16> {
    using type = uint2;
    static __device__ __forceinline__ void unpack(const uint2& q, float* v) {
        v[0] = bf16lo(q.x); v[1] = bf16hi(q.x); v[2] = bf16lo(q.y); v[3] = bf16hi(q.y);
    }
    static __device__ __forceinline__ uint2 pack(const float* v) {
        return make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    }
};

// This lane's columns of one row; columns past N are -inf.  ok = false: no load.
template <typename T, int L, int C, bool VEC>
__device__ __forceinline__ void load_row(const T* row, int l, int N, bool ok, float (&v)[4 * C]) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (VEC) {   // N is a multiple of 4 here
            if (ok && col_of<L, C, VEC>(l, c, 0) < N)
                Quad<T>::unpack(__ldg(reinterpret_cast<const typename Quad<T>::type*>(row) + l + L * c), v + 4 * c);
            else
                v[4 * c] = v[4 * c + 1] = v[4 * c + 2] = v[4 * c + 3] = -CUDART_INF_F;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = col_of<L, C, VEC>(l, c, i);
                v[4 * c + i] = ok && e < N ? Elem<T>::to_f(row[e]) : -CUDART_INF_F;
            }
        }
    }
}

// v <- softmax over the row, lse.  A row without a finite logit has p = 0 and
// lse = 0 (it adds nothing to either loss); NaN and +inf make the row NaN.
template <int L, int C>
__device__ __forceinline__ void softmax_row(float (&v)[4 * C], float& lse) {
    float m = v[0];
#pragma unroll
    for (int j = 1; j < 4 * C; ++j) m = fmaxf(m, v[j]);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float m0 = m == -CUDART_INF_F ? 0.f : m;
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 4 * C; ++j) {
        v[j] = exp_neg(v[j] - m0);
        s += v[j];
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float inv = s == 0.f ? 0.f : 1.f / s;
    lse = s == 0.f ? 0.f : m0 + logf(s);
#pragma unroll
    for (int j = 0; j < 4 * C; ++j) v[j] *= inv;
}

__device__ __forceinline__ int64_t bound(int64_t v, int64_t T) { return v < 0 ? 0 : (v > T ? T : v); }

// first row of sequence s; without offsets the batch is one sequence
__device__ __forceinline__ int64_t seq_at(const int32_t* seqs, int s, int64_t T) {
    return seqs ? bound(__ldg(seqs + s), T) : (s == 0 ? 0 : T);
}

// the last sequence that starts at or before row t (0 when none does)
__device__ __forceinline__ int first_seq(const int32_t* seqs, int S, int64_t t, int64_t T) {
    int lo = 0, hi = S;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (seq_at(seqs, mid, T) <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <typename T, int L, int C, bool VEC>
__global__ void __launch_bounds__(kBalThreads)
balance_tile_kernel(const BalanceArgs a) {
    constexpr int G = 32 / L;              // rows a warp holds at once
    constexpr int U = C == 1 ? 4 : 2;      // row loads in flight per lane
    __shared__ float s_p[kBalWarps][4 * C * L];
    __shared__ int s_cnt[kBalWarps][4 * C * L];
    __shared__ double s_z[kBalWarps];
    __shared__ int s_n[kBalWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, l = lane % L, g = lane / L;
    const int N = a.N;
    const T* h = reinterpret_cast<const T*>(a.h);
    for (int j = lane; j < 4 * C * L; j += 32) s_cnt[warp][j] = 0;
    pdl_wait();
    pdl_launch();
    const int64_t t0 = (int64_t)blockIdx.x * a.tile, t1 = min(a.T, t0 + a.tile);
    for (int s = first_seq(a.seqs, a.S, t0, a.T); s < a.S; ++s) {
        const int64_t q0 = seq_at(a.seqs, s, a.T);
        if (q0 >= t1) break;
        const int64_t p0 = max(t0, q0), p1 = min(t1, seq_at(a.seqs, s + 1, a.T));
        if (p0 >= p1) continue;   // an empty sequence, or one that ends before the tile
        float acc[4 * C];
#pragma unroll
        for (int j = 0; j < 4 * C; ++j) acc[j] = 0.f;
        double z = 0.0;
        int n = 0;
        for (int64_t b = p0 + warp * G; b < p1; b += (int64_t)kBalWarps * G * U) {
            float v[U][4 * C];
            bool ok[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t t = b + (int64_t)u * kBalWarps * G + g;
                ok[u] = t < p1;
                load_row<T, L, C, VEC>(h + t * a.ld, l, N, ok[u], v[u]);
                ok[u] = ok[u] && (!a.mask || __ldg(a.mask + t) != 0);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float lse;
                softmax_row<L, C>(v[u], lse);
                if (ok[u]) {
#pragma unroll
                    for (int j = 0; j < 4 * C; ++j) acc[j] += v[u][j];
                    z += (double)lse * (double)lse;
                    ++n;
                }
            }
        }
        for (int64_t t = p0 + tid; t < p1; t += kBalThreads) {
            if (a.mask && __ldg(a.mask + t) == 0) continue;
            for (int r = 0; r < a.k; ++r) {
                const int e = __ldg(a.idx + t * a.k + r);
                if ((unsigned)e < (unsigned)N) atomicAdd(&s_cnt[warp][e], 1);
            }
        }
        // the warp's rows, then the warps in order
#pragma unroll
        for (int o = L; o < 32; o <<= 1) {
#pragma unroll
            for (int j = 0; j < 4 * C; ++j) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
            z += __shfl_xor_sync(0xffffffffu, z, o);
            n += __shfl_xor_sync(0xffffffffu, n, o);
        }
        if (g == 0) {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) s_p[warp][col_of<L, C, VEC>(l, c, i)] = acc[4 * c + i];
        }
        if (lane == 0) {
            s_z[warp] = z;
            s_n[warp] = n;
        }
        __syncthreads();
        const int64_t slot = (int64_t)blockIdx.x + s;
        for (int e = tid; e < N; e += kBalThreads) {
            double p = 0.0;
            int c = 0;
#pragma unroll
            for (int w = 0; w < kBalWarps; ++w) {
                p += (double)s_p[w][e];
                c += s_cnt[w][e];
                s_cnt[w][e] = 0;
            }
            a.slot_p[slot * N + e] = (float)p;
            a.slot_c[slot * N + e] = c;
        }
        if (tid == 0) {
            double zs = 0.0;
            int ns = 0;
            for (int w = 0; w < kBalWarps; ++w) {
                zs += s_z[w];
                ns += s_n[w];
            }
            a.slot_z[slot] = zs;
            a.slot_n[slot] = ns;
        }
        __syncthreads();
    }
}

// One CTA per sequence (grid-stride): its shares in tile order, then the CTA that
// finishes last adds the sequences' terms in sequence order.
constexpr int kBalSumThreads = 512;

__global__ void __launch_bounds__(kBalSumThreads)
balance_sum_kernel(const BalanceArgs a) {
    __shared__ double s_p[kBalSumThreads];
    __shared__ int s_c[kBalSumThreads];
    __shared__ double s_red[kBalSumThreads / 32];
    __shared__ int s_n[kBalSumThreads / 32];
    __shared__ int s_last;
    const int tid = threadIdx.x, N = a.N;
    const int ways = kBalSumThreads / N;   // threads per expert (N <= 512)
    const int e = tid % N, way = tid / N;
    pdl_wait();
    pdl_launch();
    for (int s = blockIdx.x; s < a.S; s += gridDim.x) {
        const int64_t q0 = seq_at(a.seqs, s, a.T), q1 = seq_at(a.seqs, s + 1, a.T);
        const int64_t b0 = q0 / a.tile, b1 = q1 > q0 ? (q1 - 1) / a.tile + 1 : b0;
        double p = 0.0;
        int c = 0;
        if (way < ways) {
#pragma unroll 8
            for (int64_t b = b0 + way; b < b1; b += ways) {
                p += (double)a.slot_p[(b + s) * N + e];
                c += a.slot_c[(b + s) * N + e];
            }
        }
        s_p[tid] = p;
        s_c[tid] = c;
        __syncthreads();
        int n = 0;
        double z = 0.0;
        for (int64_t b = b0 + tid; b < b1; b += kBalSumThreads) {
            n += a.slot_n[b + s];
            z += a.slot_z[b + s];
        }
        // n and z over the block, in fixed order
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            n += __shfl_xor_sync(0xffffffffu, n, o);
            z += __shfl_xor_sync(0xffffffffu, z, o);
        }
        if ((tid & 31) == 0) {
            s_n[tid >> 5] = n;
            s_red[tid >> 5] = z;
        }
        __syncthreads();
        n = 0;
        z = 0.0;
        for (int w = 0; w < kBalSumThreads / 32; ++w) {
            n += s_n[w];
            z += s_red[w];
        }
        double term = 0.0;
        if (tid < N) {
            for (int w = 1; w < ways; ++w) {
                p += s_p[tid + w * N];
                c += s_c[tid + w * N];
            }
            const double P = n > 0 ? p / (double)n : 0.0;
            if (a.P) a.P[(int64_t)s * N + tid] = (float)P;
            a.counts[(int64_t)s * N + tid] = c;
            term = n > 0 ? P * (double)c / ((double)a.k * (double)n) : 0.0;
        }
        __syncthreads();
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(0xffffffffu, term, o);
        if ((tid & 31) == 0) s_red[tid >> 5] = term;
        __syncthreads();
        if (tid == 0) {
            double t = 0.0;
            for (int w = 0; w < kBalSumThreads / 32; ++w) t += s_red[w];
            a.seq_term[s] = t;
            a.seq_z[s] = z;
            a.tokens[s] = n;
        }
        __syncthreads();
    }
    if (tid == 0) {
        __threadfence();
        s_last = atomicAdd(a.ticket, 1) == (int)gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    if (tid < 32) {
        double t = 0.0, z = 0.0;
        int n = 0, used = 0;
        for (int s = tid; s < a.S; s += 32) {
            t += __ldcg(a.seq_term + s);
            z += __ldcg(a.seq_z + s);
            const int ns = __ldcg(a.tokens + s);
            n += ns;
            used += ns > 0;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            t += __shfl_xor_sync(0xffffffffu, t, o);
            z += __shfl_xor_sync(0xffffffffu, z, o);
            n += __shfl_xor_sync(0xffffffffu, n, o);
            used += __shfl_xor_sync(0xffffffffu, used, o);
        }
        if (tid == 0) {
            a.loss[0] = (float)((double)a.alpha * N * t / (used > 0 ? used : 1));
            a.loss[1] = (float)((double)a.z_coef * z / (n > 0 ? n : 1));
            a.tokens[a.S] = n;
            a.tokens[a.S + 1] = used;
            *a.ticket = 0;
        }
    }
}

template <typename T, int L, int C, bool VEC>
__global__ void __launch_bounds__(kBalThreads)
balance_grad_kernel(const BalanceArgs a) {
    constexpr int G = 32 / L;
    constexpr int U = C == 1 ? 4 : 2;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, l = lane % L, g = lane / L;
    const int N = a.N;
    const T* h = reinterpret_cast<const T*>(a.h);
    T* dh = reinterpret_cast<T*>(a.dh);
    pdl_wait();
    pdl_launch();
    const int64_t t0 = (int64_t)blockIdx.x * a.tile, t1 = min(a.T, t0 + a.tile);
    const int total = __ldg(a.tokens + a.S), used = __ldg(a.tokens + a.S + 1);
    const float g0 = a.dloss ? __ldg(a.dloss) : 1.f, g1 = a.dloss ? __ldg(a.dloss + 1) : 1.f;
    const float zc = (float)((double)g1 * 2.0 * a.z_coef / (total > 0 ? total : 1));
    for (int s = first_seq(a.seqs, a.S, t0, a.T); s < a.S; ++s) {
        const int64_t q0 = seq_at(a.seqs, s, a.T);
        if (q0 >= t1) break;
        const int64_t p0 = max(t0, q0), p1 = min(t1, seq_at(a.seqs, s + 1, a.T));
        if (p0 >= p1) continue;
        const int ns = __ldg(a.tokens + s);
        const double w = ns > 0 && used > 0 ? (double)g0 * a.alpha * N / ((double)used * ns) / ((double)a.k * ns) : 0.0;
        float av[4 * C];
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = col_of<L, C, VEC>(l, c, i);
                av[4 * c + i] = e < N ? (float)(w * (double)__ldg(a.counts + (int64_t)s * N + e)) : 0.f;
            }
        for (int64_t b = p0 + warp * G; b < p1; b += (int64_t)kBalWarps * G * U) {
            float v[U][4 * C];
            bool in[U], ok[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t t = b + (int64_t)u * kBalWarps * G + g;
                in[u] = t < p1;
                load_row<T, L, C, VEC>(h + t * a.ld, l, N, in[u], v[u]);
                ok[u] = in[u] && (!a.mask || __ldg(a.mask + t) != 0);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t t = b + (int64_t)u * kBalWarps * G + g;
                float lse;
                softmax_row<L, C>(v[u], lse);
                float dot = 0.f;
#pragma unroll
                for (int j = 0; j < 4 * C; ++j) dot = fmaf(v[u][j], av[j], dot);
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
                const float shift = fmaf(zc, lse, -dot);
                if (!in[u] || (!ok[u] && a.accumulate)) continue;
                T* row = dh + t * a.dld;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    float d[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        d[i] = ok[u] ? v[u][4 * c + i] * (av[4 * c + i] + shift) : 0.f;
                    if (VEC) {
                        if (col_of<L, C, VEC>(l, c, 0) < N) {
                            auto* q = reinterpret_cast<typename Quad<T>::type*>(row) + l + L * c;
                            if (a.accumulate) {
                                float o[4];
                                Quad<T>::unpack(*q, o);
#pragma unroll
                                for (int i = 0; i < 4; ++i) d[i] += o[i];
                            }
                            *q = Quad<T>::pack(d);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int e = col_of<L, C, VEC>(l, c, i);
                            if (e < N) row[e] = Elem<T>::from_f(a.accumulate ? Elem<T>::to_f(row[e]) + d[i] : d[i]);
                        }
                    }
                }
            }
        }
    }
}

template <typename T, int L, int C, bool VEC>
cudaError_t launch_shape(const BalanceArgs& a, bool grad, unsigned tiles, cudaStream_t s) {
    return grad ? launch_k(balance_grad_kernel<T, L, C, VEC>, dim3(tiles), dim3(kBalThreads), 0, s, 1, a)
                : launch_k(balance_tile_kernel<T, L, C, VEC>, dim3(tiles), dim3(kBalThreads), 0, s, 1, a);
}

template <typename T, bool VEC>
cudaError_t launch_typed(const BalanceArgs& a, bool grad, unsigned tiles, cudaStream_t s) {
    if (a.N <= 4) return launch_shape<T, 1, 1, VEC>(a, grad, tiles, s);
    if (a.N <= 8) return launch_shape<T, 2, 1, VEC>(a, grad, tiles, s);
    if (a.N <= 16) return launch_shape<T, 4, 1, VEC>(a, grad, tiles, s);
    if (a.N <= 32) return launch_shape<T, 8, 1, VEC>(a, grad, tiles, s);
    if (a.N <= 64) return launch_shape<T, 16, 1, VEC>(a, grad, tiles, s);
    if (a.N <= 128) return launch_shape<T, 32, 1, VEC>(a, grad, tiles, s);
    if (a.N <= 256) return launch_shape<T, 32, 2, VEC>(a, grad, tiles, s);
    return launch_shape<T, 32, 4, VEC>(a, grad, tiles, s);
}

cudaError_t launch_any(const BalanceArgs& a, bool grad, unsigned tiles, cudaStream_t s) {
    // four columns per access need aligned rows and no ragged last quad
    const bool vec = a.N % 4 == 0 && a.ld % 4 == 0 && (!grad || a.dld % 4 == 0);
    if (a.dtype == MOE_BF16)
        return vec ? launch_typed<__nv_bfloat16, true>(a, grad, tiles, s)
                   : launch_typed<__nv_bfloat16, false>(a, grad, tiles, s);
    return vec ? launch_typed<float, true>(a, grad, tiles, s) : launch_typed<float, false>(a, grad, tiles, s);
}

}  // namespace

// Tokens per CTA of the forward: 296 tiles (two per SM) while a tile stays
// between 64 tokens and the 4096 over which a lane may sum p in fp32.
int balance_tile(int64_t T) {
    int64_t t = (T + 295) / 296;
    return (int)(t < 64 ? 64 : (t > 4096 ? 4096 : t));
}
int64_t balance_slots(int64_t T, int S) {
    const int64_t tile = balance_tile(T);
    return (T + tile - 1) / tile + S;
}

cudaError_t launch_balance_loss(BalanceArgs a, cudaStream_t s) {
    a.tile = balance_tile(a.T);
    const unsigned tiles = (unsigned)((a.T + a.tile - 1) / a.tile);
    if (tiles > 0) {
        const cudaError_t err = launch_any(a, false, tiles, s);
        if (err != cudaSuccess) return err;
    }
    const unsigned grid = (unsigned)(a.S < 1024 ? a.S : 1024);
    return launch_k(balance_sum_kernel, dim3(grid), dim3(kBalSumThreads), 0, s, 1, a);
}

cudaError_t launch_balance_grad(BalanceArgs a, cudaStream_t s) {
    if (a.T <= 0) return cudaSuccess;
    int64_t t = (a.T + 148 * 8 - 1) / (148 * 8);
    a.tile = (int)(t < 64 ? 64 : t);
    return launch_any(a, true, (unsigned)((a.T + a.tile - 1) / a.tile), s);
}

}  // namespace moe
