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
// each, so the softmax needs log2 L shuffles and no shared memory; with up to 16
// values per lane the shuffles stay below a third of the instructions.  Rows are
// loaded a batch ahead, whatever sequence they belong to.  262144 rows of 256 fp32
// logits in 64 masked sequences, 8 choices each: forward 74 us (43 at the copy
// rate), gradient 92 (83).
//
// Forward: a CTA owns a tile of consecutive tokens and walks the sequences that
// cut it.  The share of (tile b, sequence s) goes to slot b + s of the
// workspace: both indexes only grow along the tokens, so no two shares meet,
// and a reducer finds its sequence's shares without a list.  Sums of p run in
// fp32 over a lane's own tokens, then in fixed order (warp, warps, tiles in
// fp64); counts are integers.  Nothing depends on the order of arrival.
#include <math_constants.h>

#include <type_traits>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kBalThreads = 256;
constexpr int kBalWarps = kBalThreads / 32;
constexpr int kBalPerSm = 2;   // resident CTAs (with 3, which leaves 80 registers and spills: 201 us for 196)

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

// The rows of a warp's batch: U rows of 4 C values per lane, G = 32 / L rows side by side.
template <int C> constexpr int kRowsAhead = C == 1 ? 4 : (C == 2 ? 2 : 1);

template <typename T, int L, int C, bool VEC>
struct Batch {
    static constexpr int U = kRowsAhead<C>, G = 32 / L, kRows = U * G * kBalWarps;   // rows of the CTA
    float v[U][4 * C];
    int m[U];   // mask of a row in the tile, as loaded: a test here would wait for it
    static __device__ __forceinline__ int row(int b, int u, int warp, int g) { return b + (u * kBalWarps + warp) * G + g; }
    __device__ __forceinline__ void load(const BalanceArgs& a, int b, int t1, int warp, int l, int g) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = row(b, u, warp, g);
            const bool in = t < t1;
            m[u] = in && a.mask ? __ldg(a.mask + t) : 1;
            load_row<T, L, C, VEC>(reinterpret_cast<const T*>(a.h) + (int64_t)t * a.ld, l, a.N, in, v[u]);
        }
    }
};

// first row of sequence s; without offsets the batch is one sequence
__device__ __forceinline__ int seq_at(const BalanceArgs& a, int s) {
    const int T = (int)a.T;
    if (!a.seqs) return s == 0 ? 0 : T;
    const int v = __ldg(a.seqs + s);
    return v < 0 ? 0 : (v > T ? T : v);
}

// The last sequence that starts at or before row t (0 when none does), by a whole warp:
// 32 bounds at a time, so two dependent loads for up to 1024 sequences.
__device__ __forceinline__ int first_seq(const BalanceArgs& a, int t, int lane) {
    int lo = 0, n = a.S;   // it is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int s = lo + lane * step;
        const uint32_t le = __ballot_sync(0xffffffffu, lane * step < n && seq_at(a, s) <= t);
        const int last = le ? 31 - __clz(le) : 0;
        n = min(step, n - last * step);
        lo += last * step;
    }
    return lo;
}

// ---- sums over the tiles ------------------------------------------------------

template <int Ways> struct SumShared {
    double p[Ways][32];
    int c[Ways][32];
    double z;
    int n;
};

// Unit (sequence s, 32 experts): the shares of the sequence's tiles, Ways warps taking every
// Ways-th tile and warp 0 adding theirs in order.  Another warp adds the token counts and lse^2.
template <int Ways>
__device__ __forceinline__ void sum_unit(const BalanceArgs& a, int unit, SumShared<Ways>& sh) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, N = a.N, chunks = (N + 31) / 32;
    const int s = unit / chunks, e = (unit - s * chunks) * 32 + lane;
    const int q0 = seq_at(a, s), q1 = seq_at(a, s + 1);
    const int b0 = q0 / a.tile, b1 = q1 > q0 ? (q1 - 1) / a.tile + 1 : b0;
    double p = 0.0;
    int c = 0;
    if (e < N) {
#pragma unroll 8
        for (int b = b0 + warp; b < b1; b += Ways) {
            p += __ldcg(a.slot_p + (int64_t)(b + s) * N + e);
            c += __ldcg(a.slot_c + (int64_t)(b + s) * N + e);
        }
    }
    sh.p[warp][lane] = p;
    sh.c[warp][lane] = c;
    if (warp == Ways - 1) {
        double z = 0.0;
        int n = 0;
#pragma unroll 4
        for (int b = b0 + lane; b < b1; b += 32) {
            n += __ldcg(a.slot_n + b + s);
            z += __ldcg(a.slot_z + b + s);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            n += __shfl_xor_sync(0xffffffffu, n, o);
            z += __shfl_xor_sync(0xffffffffu, z, o);
        }
        if (lane == 0) {
            sh.n = n;
            sh.z = z;
        }
    }
    __syncthreads();
    if (warp == 0) {
        const int n = sh.n;
        p = 0.0;
        c = 0;
#pragma unroll
        for (int w = 0; w < Ways; ++w) {
            p += sh.p[w][lane];
            c += sh.c[w][lane];
        }
        double term = 0.0;
        if (e < N) {
            const double P = n > 0 ? p / (double)n : 0.0;
            if (a.P) a.P[(int64_t)s * N + e] = (float)P;
            a.counts[(int64_t)s * N + e] = c;
            term = n > 0 ? P * (double)c / ((double)a.k * (double)n) : 0.0;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(0xffffffffu, term, o);
        if (lane == 0) {
            a.seq_term[unit] = term;
            if (unit == s * chunks) {
                a.seq_z[s] = sh.z;
                a.tokens[s] = n;
            }
        }
    }
    __syncthreads();   // before the next unit's shares
}

// the units' terms in order, by one warp that sees them all
__device__ __forceinline__ void sum_losses(const BalanceArgs& a, int lane) {
    const int units = a.S * ((a.N + 31) / 32);
    double t = 0.0, z = 0.0;
    int n = 0, used = 0;
#pragma unroll 4
    for (int u = lane; u < units; u += 32) t += __ldcg(a.seq_term + u);
#pragma unroll 4
    for (int s = lane; s < a.S; s += 32) {
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
    if (lane == 0) {
        a.loss[0] = (float)((double)a.alpha * a.N * t / (used > 0 ? used : 1));
        a.loss[1] = (float)((double)a.z_coef * z / (n > 0 ? n : 1));
        a.tokens[a.S] = n;
        a.tokens[a.S + 1] = used;
    }
}

// Units over the grid; the CTA that finishes last adds their terms.
constexpr int kBalSumWays = 16;

__global__ void __launch_bounds__(32 * kBalSumWays)
balance_sum_kernel(const BalanceArgs a) {
    __shared__ SumShared<kBalSumWays> sh;
    const int lane = threadIdx.x & 31, units = a.S * ((a.N + 31) / 32);
    pdl_wait();
    pdl_launch();
    for (int u = blockIdx.x; u < units; u += gridDim.x) sum_unit<kBalSumWays>(a, u, sh);
    if (threadIdx.x >= 32) return;
    int last = 1;
    if (lane == 0 && gridDim.x > 1) {
        __threadfence();
        last = atomicAdd(a.ticket, 1) == (int)gridDim.x - 1;
        if (last) *a.ticket = 0;
    }
    if (!__shfl_sync(0xffffffffu, last, 0)) return;
    __threadfence();
    sum_losses(a, lane);
}

// ---- one pass over the tokens -------------------------------------------------

// W experts, padded.  A warp's sum of p: of its row groups in fp64, or (one group, L = 32) its lane's own.
template <int W, int L> struct TileShared {
    std::conditional_t<L == 32, float, double> p[kBalWarps][W];
    int cnt[kBalWarps][W];
    double z[kBalWarps];
    int n[kBalWarps];
};

// Sums of a lane's N columns over the row groups that lane bits O ... L tell apart.  A step halves the
// columns that a lane adds up (its partner takes the others); with one left the groups only add.
template <int L, int O, int N, int M, typename P>
__device__ __forceinline__ void fold(P (&p)[M], int lane, int& first, bool& writes) {
    if constexpr (O >= L) {
        const bool upper = lane & O;
        if constexpr (N > 1) {
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                const P give = upper ? p[j] : p[j + N / 2];
                p[j] = (upper ? p[j + N / 2] : p[j]) + __shfl_xor_sync(0xffffffffu, give, O);
            }
            first += upper ? N / 2 : 0;
        } else {
            p[0] += __shfl_xor_sync(0xffffffffu, p[0], O);
            writes = writes && !upper;
        }
        fold<L, O / 2, (N > 1 ? N / 2 : 1)>(p, lane, first, writes);
    }
}

// acc over a warp's 32 / L row groups, in fp64, into out by column: 16 columns over 8 groups take 14
// exchanges and not 48 (65536 rows of 64: 15.6 us for 16.7)
template <int L, int C, bool VEC, typename P>
__device__ __forceinline__ void sum_groups(const float (&acc)[4 * C], int lane, int l, P* out) {
    constexpr int G = 32 / L, N = 4 * C > G ? 4 * C / G : 1;   // columns a lane ends with
    P p[4 * C];
#pragma unroll
    for (int j = 0; j < 4 * C; ++j) p[j] = acc[j];
    int first = 0;
    bool writes = true;
    fold<L, 16, 4 * C>(p, lane, first, writes);
    if (writes) {
#pragma unroll
        for (int j = 0; j < N; ++j) out[col_of<L, C, VEC>(l, (first + j) / 4, (first + j) % 4)] = p[j];
    }
}

// FUSED: the tile that finishes last also sums, without a second launch (few tiles: one CTA
// per SM, and registers enough not to spill)
template <typename T, int L, int C, bool VEC, bool FUSED>
__global__ void __launch_bounds__(kBalThreads, FUSED ? 1 : kBalPerSm)
balance_tile_kernel(const BalanceArgs a) {
    using B = Batch<T, L, C, VEC>;
    constexpr int U = B::U;
    __shared__ TileShared<4 * C * L, L> sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, l = lane % L, g = lane / L;
    const int N = a.N;
    for (int j = lane; j < 4 * C * L; j += 32) sh.cnt[warp][j] = 0;
    __syncwarp();   // before any lane counts in them
    pdl_wait();
    if (!FUSED) pdl_launch();
    const int t0 = (int)blockIdx.x * a.tile, t1 = (int)min(a.T, (int64_t)t0 + a.tile);
    B next;
    next.load(a, t0, t1, warp, l, g);
    int s = first_seq(a, t0, lane), q0 = seq_at(a, s), q1 = seq_at(a, s + 1);
    float acc[4 * C];
    double z = 0.0;
    int n = 0;
#pragma unroll
    for (int j = 0; j < 4 * C; ++j) acc[j] = 0.f;

    // Choice j of the batch at b is that of row b + j / k; the first E per thread are loaded a batch
    // ahead (a sequence's choices all at its start, each behind the test of its mask, took a third of
    // the kernel's time; the shared-memory atomics themselves are free).
    constexpr int E = C == 4 ? 2 : 4;
    const uint32_t inv = 0xFFFFFFFFu / (uint32_t)a.k + 1u;   // j < 2^14: the quotient by k is one product
    auto row_of = [&](int b, int j) { return b + (a.k == 1 ? j : (int)__umulhi((uint32_t)j, inv)); };
    auto choice = [&](int b, int j, int& m) {
        const int t = row_of(b, j);
        const bool in = j < B::kRows * a.k && t < t1;
        m = in && a.mask ? __ldg(a.mask + t) : 1;
        return in ? __ldg(a.idx + (int64_t)b * a.k + j) : -1;
    };
    auto count = [&](int b, int j, int e, int m) {
        const int t = row_of(b, j);
        if ((unsigned)e < (unsigned)N && m != 0 && t >= q0 && t < q1) atomicAdd(&sh.cnt[warp][e], 1);
    };
    int ne[E], nm[E];
#pragma unroll
    for (int i = 0; i < E; ++i) ne[i] = choice(t0, tid + i * kBalThreads, nm[i]);
    // the share of sequence s: the warp's rows, then the warps in order
    auto flush = [&]() {
        if (max(t0, q0) >= min(t1, q1)) return;   // no row of it in the tile
#pragma unroll
        for (int o = L; o < 32; o <<= 1) {
            z += __shfl_xor_sync(0xffffffffu, z, o);
            n += __shfl_xor_sync(0xffffffffu, n, o);
        }
        sum_groups<L, C, VEC>(acc, lane, l, sh.p[warp]);
        if (lane == 0) {
            sh.z[warp] = z;
            sh.n[warp] = n;
        }
        __syncthreads();
        const int64_t slot = (int64_t)blockIdx.x + s;
        for (int e = tid; e < N; e += kBalThreads) {
            double p = 0.0;
            int c = 0;
#pragma unroll
            for (int w = 0; w < kBalWarps; ++w) {
                p += (double)sh.p[w][e];
                c += sh.cnt[w][e];
                sh.cnt[w][e] = 0;
            }
            a.slot_p[slot * N + e] = p;
            a.slot_c[slot * N + e] = c;
        }
        if (warp == kBalWarps - 1) {
            double zs = lane < kBalWarps ? sh.z[lane] : 0.0;
            int ns = lane < kBalWarps ? sh.n[lane] : 0;
#pragma unroll
            for (int o = kBalWarps / 2; o > 0; o >>= 1) {
                zs += __shfl_xor_sync(0xffffffffu, zs, o);
                ns += __shfl_xor_sync(0xffffffffu, ns, o);
            }
            if (lane == 0) {
                a.slot_z[slot] = zs;
                a.slot_n[slot] = ns;
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4 * C; ++j) acc[j] = 0.f;
        z = 0.0;
        n = 0;
    };

#pragma unroll 1
    for (int b = t0; b < t1; b += B::kRows) {
        B cur = next;
        int e[E], em[E];
        next.load(a, b + B::kRows, t1, warp, l, g);
#pragma unroll
        for (int i = 0; i < E; ++i) {
            e[i] = ne[i];
            em[i] = nm[i];
            ne[i] = choice(b + B::kRows, tid + i * kBalThreads, nm[i]);
        }
        float lse[U];
#pragma unroll
        for (int u = 0; u < U; ++u) softmax_row<L, C>(cur.v[u], lse[u]);
        for (;;) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int t = B::row(b, u, warp, g);
                if (cur.m[u] != 0 && t >= q0 && t < min(q1, t1)) {
#pragma unroll
                    for (int j = 0; j < 4 * C; ++j) acc[j] += cur.v[u][j];
                    z += (double)lse[u] * (double)lse[u];
                    ++n;
                }
            }
#pragma unroll
            for (int i = 0; i < E; ++i) count(b, tid + i * kBalThreads, e[i], em[i]);
#pragma unroll 4
            for (int j = tid + E * kBalThreads; j < B::kRows * a.k; j += kBalThreads) {
                int m;
                const int x = choice(b, j, m);
                count(b, j, x, m);
            }
            if (q1 >= min(b + B::kRows, t1) || s + 1 >= a.S) break;
            flush();
            ++s;
            q0 = q1;
            q1 = seq_at(a, s + 1);
        }
    }
    flush();

    if constexpr (FUSED) {
        __shared__ SumShared<kBalWarps> sum;
        __shared__ int s_last;
        int last = 1;
        if (gridDim.x > 1) {
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                s_last = atomicAdd(a.ticket, 1) == (int)gridDim.x - 1;
                if (s_last) *a.ticket = 0;
            }
            __syncthreads();
            last = s_last;
        }
        pdl_launch();
        if (!last) return;
        __threadfence();
        __syncthreads();
        for (int u = 0, units = a.S * ((N + 31) / 32); u < units; ++u) sum_unit<kBalWarps>(a, u, sum);
        if (warp == 0) sum_losses(a, lane);
    }
}

template <typename T, int L, int C, bool VEC>
__global__ void __launch_bounds__(kBalThreads, kBalPerSm)
balance_grad_kernel(const BalanceArgs a) {
    using B = Batch<T, L, C, VEC>;
    constexpr int U = B::U;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, l = lane % L, g = lane / L;
    const int N = a.N;
    T* dh = reinterpret_cast<T*>(a.dh);
    pdl_wait();
    pdl_launch();
    const int t0 = (int)blockIdx.x * a.tile, t1 = (int)min(a.T, (int64_t)t0 + a.tile);
    B next;
    next.load(a, t0, t1, warp, l, g);
    const int total = __ldg(a.tokens + a.S), used = __ldg(a.tokens + a.S + 1);
    const float g0 = a.dloss ? __ldg(a.dloss) : 1.f, g1 = a.dloss ? __ldg(a.dloss + 1) : 1.f;
    int s = first_seq(a, t0, lane), q0 = seq_at(a, s), q1 = seq_at(a, s + 1);
    const float zc = 2.f * a.z_coef * g1 / (float)max(total, 1);
    float av[4 * C];
    // a_s at this lane's columns; the two quotients apart, so that neither leaves fp32's range early
    auto coefs = [&]() {
        const int ns = __ldg(a.tokens + s);
        int c[4 * C];
#pragma unroll
        for (int j = 0; j < 4 * C; ++j) {
            const int e = col_of<L, C, VEC>(l, j / 4, j % 4);
            c[j] = e < N ? __ldg(a.counts + (int64_t)s * N + e) : 0;
        }
        const bool any = ns > 0 && used > 0;
        const float w = any ? g0 * a.alpha * (float)N / ((float)used * (float)ns) : 0.f;
        const float f = any ? 1.f / ((float)a.k * (float)ns) : 0.f;
#pragma unroll
        for (int j = 0; j < 4 * C; ++j) av[j] = w * ((float)c[j] * f);
    };
    coefs();
#pragma unroll 1
    for (int b = t0; b < t1; b += B::kRows) {
        B cur = next;
        next.load(a, b + B::kRows, t1, warp, l, g);
        float lse[U];
#pragma unroll
        for (int u = 0; u < U; ++u) softmax_row<L, C>(cur.v[u], lse[u]);
        for (;;) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int t = B::row(b, u, warp, g);
                float dot = 0.f;
#pragma unroll
                for (int j = 0; j < 4 * C; ++j) dot = fmaf(cur.v[u][j], av[j], dot);
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
                const float shift = fmaf(zc, lse[u], -dot);
                const bool ok = cur.m[u] != 0;
                if (t < q0 || t >= min(q1, t1) || (!ok && a.accumulate)) continue;
                T* row = dh + (int64_t)t * a.dld;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    float d[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        d[i] = ok ? cur.v[u][4 * c + i] * (av[4 * c + i] + shift) : 0.f;
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
            if (q1 >= min(b + B::kRows, t1) || s + 1 >= a.S) break;
            ++s;
            q0 = q1;
            q1 = seq_at(a, s + 1);
            coefs();
        }
    }
}

enum class BalPass { kForward, kFused, kGrad };

template <typename T, int L, int C, bool VEC>
cudaError_t launch_shape(const BalanceArgs& a, BalPass pass, unsigned tiles, cudaStream_t s) {
    if (pass == BalPass::kGrad)
        return launch_k(balance_grad_kernel<T, L, C, VEC>, dim3(tiles), dim3(kBalThreads), 0, s, 1, a);
    return pass == BalPass::kFused
               ? launch_k(balance_tile_kernel<T, L, C, VEC, true>, dim3(tiles), dim3(kBalThreads), 0, s, 1, a)
               : launch_k(balance_tile_kernel<T, L, C, VEC, false>, dim3(tiles), dim3(kBalThreads), 0, s, 1, a);
}

template <typename T, bool VEC>
cudaError_t launch_typed(const BalanceArgs& a, BalPass pass, unsigned tiles, cudaStream_t s) {
    if (a.N <= 4) return launch_shape<T, 1, 1, VEC>(a, pass, tiles, s);
    if (a.N <= 8) return launch_shape<T, 2, 1, VEC>(a, pass, tiles, s);
    if (a.N <= 16) return launch_shape<T, 4, 1, VEC>(a, pass, tiles, s);
    if (a.N <= 32) return launch_shape<T, 4, 2, VEC>(a, pass, tiles, s);
    if (a.N <= 64) return launch_shape<T, 4, 4, VEC>(a, pass, tiles, s);
    if (a.N <= 128) return launch_shape<T, 8, 4, VEC>(a, pass, tiles, s);
    if (a.N <= 256) return launch_shape<T, 16, 4, VEC>(a, pass, tiles, s);
    return launch_shape<T, 32, 4, VEC>(a, pass, tiles, s);
}

cudaError_t launch_any(const BalanceArgs& a, BalPass pass, unsigned tiles, cudaStream_t s) {
    // four columns per access need aligned rows and no ragged last quad
    const bool vec = a.N % 4 == 0 && a.ld % 4 == 0 && (pass != BalPass::kGrad || a.dld % 4 == 0);
    if (a.dtype == MOE_BF16)
        return vec ? launch_typed<__nv_bfloat16, true>(a, pass, tiles, s)
                   : launch_typed<__nv_bfloat16, false>(a, pass, tiles, s);
    return vec ? launch_typed<float, true>(a, pass, tiles, s) : launch_typed<float, false>(a, pass, tiles, s);
}

// rows of one batch of a CTA (Batch::kRows): 4096 values of rows padded to a power of two
int batch_rows(int N) {
    int np = 4;
    while (np < N) np *= 2;
    return 4096 / np;
}

}  // namespace

// Tokens per CTA of the forward: kBalPerSm tiles per SM while a tile stays between one
// batch and the 4096 over which a lane may sum p in fp32.
int balance_tile(int64_t T, int N) {
    const int64_t t = (T + 148 * kBalPerSm - 1) / (148 * kBalPerSm), lo = batch_rows(N);
    return (int)(t < lo ? lo : (t > 4096 ? 4096 : t));
}
int64_t balance_slots(int64_t T, int N, int S) {
    const int64_t tile = balance_tile(T, N);
    return (T + tile - 1) / tile + S;
}

cudaError_t launch_balance_loss(BalanceArgs a, cudaStream_t s) {
    a.tile = balance_tile(a.T, a.N);
    const int64_t tiles = (a.T + a.tile - 1) / a.tile, units = (int64_t)a.S * ((a.N + 31) / 32);
    // few tiles and units: one CTA adds them sooner than a second launch would (512 rows of 8: 6.4 us for 9.2)
    const bool fused = tiles > 0 && tiles <= 64 && units <= 4;
    if (tiles > 0) {
        const cudaError_t err = launch_any(a, fused ? BalPass::kFused : BalPass::kForward, (unsigned)tiles, s);
        if (err != cudaSuccess || fused) return err;
    }
    return launch_k(balance_sum_kernel, dim3((unsigned)(units < 1024 ? units : 1024)), dim3(32 * kBalSumWays), 0, s, 1, a);
}

cudaError_t launch_balance_grad(BalanceArgs a, cudaStream_t s) {
    if (a.T <= 0) return cudaSuccess;
    // a row per lane group at least, which spreads a small batch over the SMs
    const int64_t t = (a.T + 148 * 8 - 1) / (148 * 8), lo = a.N <= 16 ? batch_rows(a.N) / 4 : batch_rows(a.N);
    a.tile = (int)(t < lo ? lo : t);
    return launch_any(a, BalPass::kGrad, (unsigned)((a.T + a.tile - 1) / a.tile), s);
}

}  // namespace moe
