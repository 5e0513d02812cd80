// Expert FFN on 4-bit weights for many rows per expert, on tcgen05.
//
//   stage 1: H = relu(x W1^T + b1), or silu(x W1^T + b1) * (x W3^T + b3)
//   stage 2: y = H W2^T + b2              W[o][k] = q[o][k] s[o][k / G]
//
// The weights are the A operand: a tile is 128 weight rows by up to 192 tokens, or by
// up to 256 (see Shape), so each word is decoded once for all of them, and a thread that
// decodes owns one row.  Decoded words go straight into TMEM (tcgen05.st), from where tcgen05.mma
// reads A: through shared memory the operand would be written and read again
// beside the tokens' tiles, more than the 128 bytes a cycle shared memory has.
//
// Operands are fp16, because q s (three bits times a bf16 scale's eight) is exact in
// its eleven and not in bf16's eight; everything then accumulates over all of K in
// TMEM.  (bf16 integers as A, with every group's sum read back from TMEM and scaled
// in registers, took 0.98 ms where this, at the time, took 0.86: reading back was the
// bottleneck.)  fp16's range is met by powers of two, which round nothing:
//   weights: per row, so that its largest scale lies in [2^10, 2^12) -- exact for
//     scales down to 2^-27 of it;
//   x: per token, so that its largest value lies in [2^13, 2^15) -- exact for values
//     down to 2^-29 of it (bf16 has eight bits);
//   H: per token, from |u| <= (sum |x|) 8 max|s| and the biases, which no value
//     passes.  The bound is about 2^8 (SwiGLU: 2^16) above typical values, whose fp16
//     form has all its bits down to 2^-14 / 2^14 = 2^-28 of it; those give 2^-11, an
//     eighth of the rounding to bf16 that the layer on bf16 weights applies here.
// The epilogues undo the powers in fp32.  All exponents are even: half of a row's and half
// of a token's make a factor t = 2^((e + ex) / 2) that is always a normal number, and
// (sum t) t leaves fp32 only where the result itself does (the sum is 0 or 2^-48 ... 2^53,
// so sum t is subnormal or infinite only if sum t t is far below 2^-126 or above 2^128).
//
// Single-lane branches around TMA, MMA and commit use elect.sync in a warp-uniform
// loop: with `lane == 0` each such instruction took 45 cycles to issue, not 9.
// 256 rows for each of 8 experts, d_model 4096, d_ff 14336: 0.63 ms, 1.14 PFLOP/s; 1024
// tokens routed unevenly, inputs changing: 0.83 ms, 0.87 PFLOP/s.  With few tokens a tile (32
// rows an expert: 0.36 ms) a block's hand-overs between the roles bound it, not its MMAs.
//
// Roles (five warpgroups): warps 0 and 3 TMA of the tokens' rows, 1 MMA issue, 2 TMA
// of the packed rows and scales (they come from HBM and are asked for further ahead);
// warps 4-11 decode, the two groups a block each in turn; warps 12-19 write out, half of
// a tile's tokens a group (beside the next tile's MMAs, or see Shape).  SwiGLU puts
// a feature's W1 row on lane l < 16 and its W3 row on lane l + 16 of the same warp,
// so the gate and the value meet by a shuffle.
// Every wait is bounded; on expiry the kernel latches MOE_ERR_TIMEOUT, stops
// issuing, waits (bounded) for its copies and MMAs, frees TMEM and returns.
#include <cuda_fp16.h>

#include "tc_common.cuh"
#include "w4.cuh"

namespace moe {
using namespace tc;
namespace {

constexpr int kThreadsTc = 640;
constexpr int kBoxN = 64;                         // tokens per TMA box
constexpr int kBoxBytes = kBoxN * 128;            // ... by 64 of K
constexpr int kWBytes = 128 * 128;
constexpr int kSBytes = 2048;                     // scales of a stage: 2 boxes x 256 / G groups x 64 rows

// Tiles of up to 192 tokens, whose accumulator has a second one beside it in TMEM; or (WIDE) of up to
// 256, one accumulator, so that nothing accumulates while a tile is written out.  A step reads one
// stage of tokens, and its end (mdone) frees that stage and, with a block's last step, the block's A
// buffer: one commit for both.  Two stages of 128 of K kept 64 KB in flight for a wide tile, less
// than the loads' latency wants; five of 64 took 1024 tokens from 852 to 820 us.
template <bool WIDE>
struct Shape {
    static constexpr int N = WIDE ? 256 : 192;            // tokens of a tile
    static constexpr int PART = N / 2;                    // ... of a group of writing warps
    static constexpr int D = WIDE ? 1 : 2;                // accumulators
    static constexpr int A = 2;                           // blocks of decoded weights
    static constexpr uint32_t COL_D = 0, COL_A = D * N;   // TMEM columns
    static constexpr int WSTAGES = WIDE ? 3 : 4;          // packed rows and scales: 256 of K each
    static constexpr int U = WIDE ? 64 : 128;             // K of a stage of tokens, and of a step
    static constexpr int XSTAGES = WIDE ? 5 : 3;
    static constexpr int UPB = kW4Block / U;              // steps per block of 128
    static constexpr int RING = WIDE ? 20 : 6;            // a multiple of XSTAGES and A UPB
    static constexpr int XSUB = N / kBoxN * kBoxBytes;    // 64 of K
    static constexpr int XBYTES = U / 64 * XSUB;
    static constexpr int SMEM = WSTAGES * (kWBytes + kSBytes) + XSTAGES * XBYTES + 1024;
    static_assert(A == 2 && RING > XSTAGES && RING % XSTAGES == 0 && RING % (A * UPB) == 0, "the ring's indexes");
};
constexpr int kNanExp = 0x7FFF;                   // exponent of a row that holds a NaN or infinity

enum { W4_RELU = 0, W4_SWIGLU = 1, W4_OUT = 2 };

struct TcParams {
    const int32_t* offsets; int N; int64_t R_cap;
    int m_dim, k_dim;
    const __nv_bfloat16* bias_a; const __nv_bfloat16* bias_b;
    const int8_t* ea; const int8_t* eb;   // [N, m_dim] row exponents, -126 .. 116: scales were taken times 2^-e
    const int16_t* ex;                    // [R] exponents of the tokens' rows, -126 .. 126: x times 2^-ex
    const int16_t* lx;                    // stage 1: [R] sum |x| < 2^lx
    const int32_t* top;                   // stage 1: [4][N] largest scale and bias of W1, W3 (as float bits)
    int16_t* eh;                          // stage 1: [R] exponents of H
    void* out;                            // stage 1: H [R, m_dim] fp16, stage 2: y [R, m_dim] bf16
    int32_t* status;
    long long limit_ns;
};

__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Weights 2 p and 2 p + 1 of a word's eight, times the scale s2 (an fp16 pair), by the known
// way of joining integers to a float's low mantissa bits (for 4-bit experts: Kim, Henry, Fahim
// and Hassan Awadalla, "Who Says Elephants Can't Run", 2022): 0x6400 is 1024 in fp16, whose last place is 1, so nibbles in the low bits add to it
// exactly, and in bits 4-7 as sixteenfold; w8 = w >> 8 holds the odd pairs.
__device__ __forceinline__ uint32_t decode_pair(uint32_t w, uint32_t w8, int p, __half2 s2) {
    uint32_t u;   // one operation: written as two immediates it would be two
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(u) : "r"(p < 2 ? w : w8), "r"(p & 1 ? 0x00F000F0u : 0x000F000Fu), "r"(0x64006400u));
    __half2 q = *reinterpret_cast<const __half2*>(&u);
    if (p & 1) q = __hfma2(q, __half2half2(__ushort_as_half(0x2C00)), __half2half2(__ushort_as_half(0xD480)));   // / 16 - 72
    else q = __hsub2(q, __half2half2(__ushort_as_half(0x6408)));                                                 // - 1032
    q = __hmul2(q, s2);
    return *reinterpret_cast<const uint32_t*>(&q);
}

// 2^e, -126 <= e <= 127
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }
// the next even exponent, up
__device__ __forceinline__ int even(int e) { return (e + 1) & ~1; }
// exponent of a finite positive float's leading bit (0 and subnormals: -127)
__device__ __forceinline__ int exp_of(uint32_t bits) { return (int)(bits >> 23) - 127; }

// The exponent that brings a token's H to fp16 range: its bound's, less 15 (or 14).  A bound
// past 2^141 takes 126 too: H itself, in fp32, is below 2^128.
template <int EPI>
__device__ __forceinline__ int h_exponent(const int32_t* top, int N, int e, int lx) {
    // |u| < 2^lx 8 2^(exp(max scale) + 1), plus the bias
    auto side = [&](int m) {
        const int u = lx + 3 + exp_of(top[2 * m * N + e]) + 1, b = exp_of(top[(2 * m + 1) * N + e]) + 1;
        return max(u, b) + 1;
    };
    return even(min(max(side(0) + (EPI == W4_SWIGLU ? side(1) : 0) - 15, -126), 126));
}

template <bool WIDE>
struct SharedTc {
    uint64_t wfull[Shape<WIDE>::WSTAGES], wempty[Shape<WIDE>::WSTAGES];
    uint64_t xfull[Shape<WIDE>::XSTAGES];
    uint64_t afull[Shape<WIDE>::A];       // a block's weights are in TMEM
    uint64_t mdone[Shape<WIDE>::RING];    // a step's MMAs are done: its tokens and weights have been read
    uint64_t dfull[2], dempty[2];   // accumulators of a tile
    uint64_t done;
    uint32_t tmem;
    int abort, live;
    int row[129], exp[128], first[129];
    float scale[8][2][Shape<WIDE>::PART];      // per writing warp: the tokens' powers of two
};

struct Tile {
    int e, m0, row0, n;
};

// rows of an expert in equal chunks of at most `most`, a multiple of 16
__device__ __forceinline__ int chunk_rows(int n, int most) {
    const int chunks = (n + most - 1) / most;
    return ((n + chunks - 1) / chunks + 15) / 16 * 16;
}

template <bool WIDE>
__device__ __forceinline__ Tile tile_of(const SharedTc<WIDE>& sh, int u, int feats) {
    int lo = 0, hi = sh.live;   // first[lo] <= u < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sh.first[mid] <= u) lo = mid;
        else hi = mid;
    }
    const int e = sh.exp[lo], rows = sh.row[e + 1] - sh.row[e], local = u - sh.first[lo];
    const int per = chunk_rows(rows, Shape<WIDE>::N), chunks = (rows + per - 1) / per;
    Tile t;   // the chunks of a feature tile follow one another: its weights are in L2
    t.e = e;
    t.m0 = local / chunks * feats;
    t.row0 = sh.row[e] + local % chunks * per;
    t.n = min(per, sh.row[e + 1] - t.row0);
    return t;
}

template <int EPI, int G, bool WIDE>
__global__ void __launch_bounds__(kThreadsTc, 1)
w4_tc_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
             const __grid_constant__ CUtensorMap map_sa, const __grid_constant__ CUtensorMap map_sb,
             const __grid_constant__ CUtensorMap map_x, const TcParams p) {
    constexpr int MATS = EPI == W4_SWIGLU ? 2 : 1;
    constexpr int FEATS = 128 / MATS;
    constexpr int PER = kW4Block / G;   // groups per 128 of K
    using S = Shape<WIDE>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* smem_x = smem + S::WSTAGES * kWBytes;
    uint8_t* smem_s = smem_x + S::XSTAGES * S::XBYTES;
    __shared__ __align__(8) SharedTc<WIDE> sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < S::WSTAGES; ++s) {
            mbar_init(smem_u32(&sh.wfull[s]), 1);
            mbar_init(smem_u32(&sh.wempty[s]), 8);
        }
        for (int s = 0; s < S::XSTAGES; ++s) mbar_init(smem_u32(&sh.xfull[s]), 1);
        for (int i = 0; i < S::A; ++i) mbar_init(smem_u32(&sh.afull[i]), 4);
        for (int i = 0; i < S::RING; ++i) mbar_init(smem_u32(&sh.mdone[i]), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.dfull[i]), 1);
            mbar_init(smem_u32(&sh.dempty[i]), 8);
        }
        mbar_init(smem_u32(&sh.done), 1);
        sh.abort = 0;
        mbar_fence_init();
        prefetch_tmap(&map_a);
        prefetch_tmap(&map_x);
    }
    if (warp == 1) tmem_alloc(&sh.tmem, 512);
    pdl_wait();
    pdl_launch();
    for (int i = tid; i <= p.N; i += kThreadsTc) {
        const int64_t v = p.offsets[i];
        sh.row[i] = (int)(v < 0 ? 0 : (v > p.R_cap ? p.R_cap : v));
    }
    __syncthreads();
    const int tiles = (p.m_dim + FEATS - 1) / FEATS;
    if (warp == 3) {   // live experts and their first units: four experts a lane, a scan over the lanes
        int n[4], live = 0, units = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = 4 * lane + i, rows = e < p.N ? max(0, sh.row[e + 1] - sh.row[e]) : 0;
            const int per = chunk_rows(max(rows, 1), S::N);
            n[i] = (rows + per - 1) / per * tiles;
            live += n[i] > 0;
            units += n[i];
        }
        int l = live, u = units;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int lo = __shfl_up_sync(0xffffffffu, l, o), uo = __shfl_up_sync(0xffffffffu, u, o);
            if (lane >= o) {
                l += lo;
                u += uo;
            }
        }
        if (lane == 31) {
            sh.live = l;
            sh.first[l] = u;
        }
        l -= live;
        u -= units;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n[i] > 0) {
                sh.exp[l] = 4 * lane + i;
                sh.first[l++] = u;
                u += n[i];
            }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const int units = sh.first[sh.live];
    const int nb = (p.k_dim + kW4Block - 1) / kW4Block;   // blocks of 128
    const Waiter w{&sh.abort, p.status, p.limit_ns};

    if (warp < 4) {
        if (warp == 0 || warp == 3) {
            // ---------------- TMA: the tokens' rows (two warps, stages in turn) ----------------
            int xs = 0, r = 0, ahead = S::XSTAGES;   // r: the step that read stage xs last, once none is ahead
            uint32_t xph = 0, rph = 0, xused = 0;
            bool ok = true, mine = warp == 0;
            for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
                const Tile t = tile_of(sh, u, FEATS);
                const int boxes = (t.n + kBoxN - 1) / kBoxN;
                for (int k = 0; k < nb * kW4Block; k += S::U, mine = !mine) {
                    if (mine) {
                        if (ahead == 0) ok = __all_sync(0xffffffffu, wait_bar_soon(smem_u32(&sh.mdone[r]), rph, w));
                        if (!ok) break;
                        const uint32_t fb = smem_u32(&sh.xfull[xs]), dst = smem_u32(smem_x) + xs * S::XBYTES;
                        const int parts = S::U == 128 && k + 64 < p.k_dim ? 2 : 1;   // (a box past K: zeros, not used)
                        if (elect_one()) {
                            mbar_expect_tx(fb, parts * boxes * kBoxBytes);
                            for (int h = 0; h < parts; ++h)
                                for (int b = 0; b < boxes; ++b)
                                    tma_load_2d(dst + h * S::XSUB + b * kBoxBytes, &map_x, fb, k + h * 64, t.row0 + b * kBoxN);
                        }
                        __syncwarp();
                    }
                    if (ahead > 0) {
                        --ahead;
                    } else if (++r == S::RING) {
                        r = 0;
                        rph ^= 1u;
                    }
                    xused |= 1u << xs;
                    if (++xs == S::XSTAGES) {
                        xs = 0;
                        xph ^= 1u;
                    }
                }
            }
            // every load has landed before the CTA retires (each warp looks at all stages)
            for (int s = 0; s < S::XSTAGES; ++s)
                if (xused >> s & 1u) drain_bar(smem_u32(&sh.xfull[s]), s < xs ? xph : xph ^ 1u, p.limit_ns, p.status);
        } else if (warp == 2) {
            // ---------------- TMA: packed rows and scales ----------------
            int ws = 0;
            uint32_t wph = 0, wused = 0;
            bool ok = true;
            const int ng = (p.k_dim + G - 1) / G;
            for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
                const Tile t = tile_of(sh, u, FEATS);
                const int row = t.e * p.m_dim + t.m0;
                const bool second = MATS == 2 || t.m0 + 64 < p.m_dim;   // the upper 64 rows hold something
                for (int kb = 0; kb < nb; kb += 2) {
                    ok = __all_sync(0xffffffffu, wait_bar_soon(smem_u32(&sh.wempty[ws]), wph ^ 1u, w));
                    if (!ok) break;
                    constexpr int SB = 2 * PER * 128;   // one box of scales
                    const uint32_t fb = smem_u32(&sh.wfull[ws]), dst = smem_u32(smem) + ws * kWBytes;
                    const uint32_t sdst = smem_u32(smem_s) + ws * kSBytes;
                    if (elect_one()) {
                        mbar_expect_tx(fb, (second ? 2 : 1) * (kWBytes / 2 + SB));
                        tma_load_2d(dst, &map_a, fb, kb * kW4BlockBytes, row);
                        tma_load_2d(sdst, &map_sa, fb, t.m0, t.e * ng + kb * PER);
                        if (second) {
                            tma_load_2d(dst + kWBytes / 2, MATS == 2 ? &map_b : &map_a, fb, kb * kW4BlockBytes,
                                        MATS == 2 ? row : row + 64);
                            tma_load_2d(sdst + SB, MATS == 2 ? &map_sb : &map_sa, fb, MATS == 2 ? t.m0 : t.m0 + 64,
                                        t.e * ng + kb * PER);
                        }
                    }
                    __syncwarp();
                    wused |= 1u << ws;
                    if (++ws == S::WSTAGES) {
                        ws = 0;
                        wph ^= 1u;
                    }
                }
            }
            for (int s = 0; s < S::WSTAGES; ++s)
                if (wused >> s & 1u) drain_bar(smem_u32(&sh.wfull[s]), s < ws ? wph : wph ^ 1u, p.limit_ns, p.status);
        } else if (warp == 1) {
            // ---------------- MMA: one thread ----------------
            // Its own instructions bound the kernel, not what it waits for: one wait and one commit
            // a step, no predicates but at the end of K, the elected thread alone in the loop
            // (1024 tokens 852 -> 740 us; the predicates and votes alone were 46).
            uint32_t issued = 0;
            if (elect_one()) {
                int xs = 0, a = 0, d = 0, r = 0;
                uint32_t xph = 0, aph = 0, dph = 0;
                const uint64_t bd0 = umma_desc(smem_u32(smem_x));
                for (int u = blockIdx.x; u < units; u += gridDim.x) {
                    const Tile t = tile_of(sh, u, FEATS);
                    const uint32_t idesc = idesc_f16_f32(128, (t.n + 15) / 16 * 16), dd = tmem + S::COL_D + d * S::N;
                    bool ok = wait_bar_soon(smem_u32(&sh.dempty[d]), dph ^ 1u, w);
                    for (int kb = 0; kb < nb && ok; ++kb) {
#pragma unroll
                        for (int h = 0; h < S::UPB; ++h) {
                            const uint32_t xb = smem_u32(&sh.xfull[xs]);
                            ok = h == 0 ? wait_two(smem_u32(&sh.afull[a]), aph, xb, xph, w) : wait_bar_soon(xb, xph, w);
                            if (!ok) break;
                            tc_fence_after();
                            issued = 1;
                            const uint64_t bd = bd0 + (uint64_t)(xs * (S::XBYTES >> 4));
                            const uint32_t ad = tmem + S::COL_A + a * 64 + h * 32;
                            const int nk = (p.k_dim - kb * kW4Block - h * 64) / 16;   // K is a multiple of 16
                            auto mma = [&](int kk) {
                                umma_ts(dd, ad + 8 * kk, bd + (uint64_t)((kk / 4 * S::XSUB) >> 4) + 2 * (kk % 4), idesc,
                                        kk ? 1 : kb | h);
                            };
                            if (nk >= S::U / 16) {
#pragma unroll
                                for (int kk = 0; kk < S::U / 16; ++kk) mma(kk);
                            } else {   // the end of K
#pragma unroll
                                for (int kk = 0; kk < S::U / 16; ++kk)
                                    if (kk < nk) mma(kk);
                            }
                            umma_commit(smem_u32(&sh.mdone[r]));
                            if (++r == S::RING) r = 0;
                            if (++xs == S::XSTAGES) {
                                xs = 0;
                                xph ^= 1u;
                            }
                        }
                        if (++a == S::A) {
                            a = 0;
                            aph ^= 1u;
                        }
                    }
                    if (!ok) break;
                    umma_commit(smem_u32(&sh.dfull[d]));
                    if (++d == S::D) {
                        d = 0;
                        dph ^= 1u;
                    }
                }
                if (issued) umma_commit(smem_u32(&sh.done));
            }
            // every MMA has completed before TMEM is freed
            if (__any_sync(0xffffffffu, issued)) drain_bar(smem_u32(&sh.done), 0u, p.limit_ns, p.status);
        }
    } else if (warp < 12) {
        // ---------------- decode: lane = weight row ----------------
        // Two groups of four warps take blocks in turn, one for each A buffer, and
        // decode into registers before they wait for it: only the stores lie between
        // one MMA and the next but one.  (Each barrier operation costs a warp about
        // 130 cycles; halves of every block, twice as many of them, took 1280 cycles
        // a block.)
        const int quad = warp & 3;   // TMEM lane quadrant
        const int a = (warp - 4) >> 2;
        int step = a * S::UPB + S::UPB - 1;   // the one that frees buffer a next
        bool fresh = true;                    // nothing has read it yet
        // SwiGLU: lanes 0-15 hold 16 features of W1, lanes 16-31 the same of W3
        const int r = MATS == 2 ? (lane >> 4) * 64 + quad * 16 + (lane & 15) : quad * 32 + lane;
        // its scales in a stage: box, then 64 features a group
        const int soff = ((r >> 6) * (2 * PER * 64) + (r & 63)) * 2;
        const int8_t* exps = MATS == 2 && lane >= 16 ? p.eb : p.ea;
        const uint32_t dst = tmem + S::COL_A + a * 64 + ((uint32_t)(quad * 32) << 16);
        int ws = 0, turn = 0;
        uint32_t wph = 0, rph = 0;
        bool ok = true;
        for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
            const Tile t = tile_of(sh, u, FEATS);
            const int feat = t.m0 + (MATS == 2 ? r & 63 : r);
            const float down = pow2i(feat < p.m_dim ? -(int)exps[(int64_t)t.e * p.m_dim + feat] : 0);
            for (int kb = 0; kb < nb && ok; ++kb, turn ^= 1) {
                const bool mine = turn == a, last = kb % 2 == 1 || kb + 1 == nb;
                uint32_t v[64];
                if (mine) {
                    if (!(ok = __all_sync(0xffffffffu, wait_bar_soon(smem_u32(&sh.wfull[ws]), wph, w)))) break;
                    const uint8_t* src = smem + ws * kWBytes + r * 128;
                    const uint8_t* ssrc = smem_s + ws * kSBytes + kb % 2 * (PER * 128) + soff;
                    __half2 sc[PER];
#pragma unroll
                    for (int g = 0; g < PER; ++g)
                        sc[g] = __float2half2_rn(
                            __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(ssrc + g * 128) << 16) * down);
#pragma unroll
                    for (int t4 = 0; t4 < 4; ++t4) {
                        const uint4 q = *reinterpret_cast<const uint4*>(src + (((kb % 2 * 4 + t4) ^ (r & 7)) << 4));
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t word = j == 0 ? q.x : j == 1 ? q.y : j == 2 ? q.z : q.w;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                v[16 * j + 4 * t4 + i] = decode_pair(word, word >> 8, i, sc[j * PER / 4]);
                        }
                    }
                    __syncwarp();
                    if (lane == 0) {   // one of the stage's two blocks, or its only one
                        mbar_arrive(smem_u32(&sh.wempty[ws]));
                        if (last && kb % 2 == 0) mbar_arrive(smem_u32(&sh.wempty[ws]));
                    }
                }
                if (last && ++ws == S::WSTAGES) {
                    ws = 0;
                    wph ^= 1u;
                }
                if (!mine) continue;
                if (!fresh) {
                    if (!(ok = __all_sync(0xffffffffu, wait_bar_soon(smem_u32(&sh.mdone[step]), rph, w)))) break;
                    if ((step += 2 * S::UPB) >= S::RING) {
                        step -= S::RING;
                        rph ^= 1u;
                    }
                }
                fresh = false;
                tc_fence_after();
                tmem_st32(dst, v);
                tmem_st32(dst + 32, v + 32);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_relaxed(smem_u32(&sh.afull[a]));
            }
        }
    } else {
        // ---------------- write out: lane = weight row ----------------
        // two groups of four warps, half of the tile's tokens each (96, or 128 of a wide one)
        const int quad = warp & 3, c0 = (warp - 12) / 4 * S::PART;
        const int f = MATS == 2 ? quad * 16 + (lane & 15) : quad * 32 + lane;   // feature of the tile
        const bool low = lane < 16;
        const __nv_bfloat16* bias = MATS == 2 && !low ? p.bias_b : p.bias_a;
        const int8_t* exps = MATS == 2 && !low ? p.eb : p.ea;
        int d = 0;
        uint32_t dph = 0;
        bool ok = true;
        for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
            const Tile t = tile_of(sh, u, FEATS);
            const int feat = t.m0 + f;
            const bool in = feat < p.m_dim;
            const int n = t.n - c0;   // this group's tokens (may be none)
            const int64_t at = (int64_t)t.e * p.m_dim + feat;
            const float up = pow2i((in ? exps[at] : 0) / 2);
            const float b = in && bias ? __bfloat162float(bias[at]) : 0.f;
            // the powers of two of these tokens: half of x's, and H's
            float* s_x = sh.scale[warp - 12][0];
            float* s_h = sh.scale[warp - 12][1];
            for (int c = lane; c < n && c < S::PART; c += 32) {
                const int ex = p.ex[t.row0 + c0 + c];
                s_x[c] = ex == kNanExp ? __int_as_float(0x7FC00000) : pow2i(ex / 2);
                if (EPI != W4_OUT) {
                    const int eh = h_exponent<EPI>(p.top, p.N, t.e, p.lx[t.row0 + c0 + c]);
                    s_h[c] = pow2i(-eh);
                    if (t.m0 == 0 && quad == 0) p.eh[t.row0 + c0 + c] = (int16_t)(ex == kNanExp ? kNanExp : eh);
                }
            }
            __syncwarp();
            if (!(ok = __all_sync(0xffffffffu, wait_bar_soon(smem_u32(&sh.dfull[d]), dph, w)))) break;
            tc_fence_after();
            const uint32_t src = tmem + S::COL_D + d * S::N + c0 + ((uint32_t)(quad * 32) << 16);
#pragma unroll 1
            for (int cb = 0; cb < S::PART && cb < n; cb += 32) {
                uint32_t v[32];
                tmem_ld32(src + cb, v);
                tmem_wait_ld();
                const int64_t row = (int64_t)(t.row0 + c0 + cb) * p.m_dim + feat;
                if (EPI == W4_SWIGLU) {
                    // lanes < 16 finish the even tokens, their partners the odd ones
                    __half* dst = reinterpret_cast<__half*>(p.out) + row + (low ? 0 : p.m_dim);
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        const float t0 = up * s_x[cb + c], t1 = up * s_x[cb + c + 1];
                        const float v0 = fmaf(__uint_as_float(v[c]) * t0, t0, b);
                        const float v1 = fmaf(__uint_as_float(v[c + 1]) * t1, t1, b);
                        const float other = __shfl_xor_sync(0xffffffffu, low ? v1 : v0, 16);
                        const float gate = low ? v0 : other, val = low ? other : v1;
                        // e^-z -> inf for very negative z: the fast division gives the limit 0
                        const float o = __fdividef(gate, 1.f + fast_exp2(-gate * kLog2e)) * val;
                        if (in && cb + c + (low ? 0 : 1) < n)
                            dst[(int64_t)c * p.m_dim] = __float2half_rn(o * s_h[cb + c + (low ? 0 : 1)]);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const float tc = up * s_x[cb + c];
                        float o = fmaf(__uint_as_float(v[c]) * tc, tc, b);
                        if (EPI == W4_RELU) {
                            o = o < 0.f ? 0.f : o;   // NaN stays
                            if (in && cb + c < n)
                                (reinterpret_cast<__half*>(p.out) + row)[(int64_t)c * p.m_dim] = __float2half_rn(o * s_h[cb + c]);
                        } else if (in && cb + c < n) {
                            (reinterpret_cast<__nv_bfloat16*>(p.out) + row)[(int64_t)c * p.m_dim] = __float2bfloat16_rn(o);
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_relaxed(smem_u32(&sh.dempty[d]));
            if (++d == S::D) {
                d = 0;
                dph ^= 1u;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// x as fp16 rows, each times a power of two (one warp per row); clears `top`.
__global__ void __launch_bounds__(256)
w4_half_rows_kernel(const __nv_bfloat16* __restrict__ x, const int32_t* __restrict__ offsets, int N, int64_t R_cap,
                    int k_dim, __half* __restrict__ out, int16_t* __restrict__ ex, int16_t* __restrict__ lx,
                    int32_t* __restrict__ top) {
    pdl_wait();
    pdl_launch();
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < 4 * N; i += 256) top[i] = 0;
    const int64_t last = offsets[N], rows = last < 0 ? 0 : (last > R_cap ? R_cap : last);
    const int lane = threadIdx.x & 31;
    for (int64_t r = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; r < rows; r += (int64_t)gridDim.x * 8) {
        const uint4* src = reinterpret_cast<const uint4*>(x + r * k_dim);
        uint32_t m = 0;   // bf16 magnitudes of both halves, compared as 16-bit integers
#pragma unroll 8
        for (int i = lane; i < k_dim / 8; i += 32) {
            const uint4 q = __ldg(src + i);
            m = __vmaxu2(m, __vmaxu2(__vmaxu2(q.x & 0x7FFF7FFFu, q.y & 0x7FFF7FFFu), __vmaxu2(q.z & 0x7FFF7FFFu, q.w & 0x7FFF7FFFu)));
        }
        const uint32_t big = __reduce_max_sync(0xffffffffu, max(m >> 16, m & 0xFFFFu)) << 16;
        const bool finite = big < 0x7F800000u;
        const int e = even(max(exp_of(big) - 14, -112));
        const float down = finite ? pow2i(-e) : 0.f;
        if (lane == 0) ex[r] = (int16_t)(finite ? e : kNanExp);
        uint4* dst = reinterpret_cast<uint4*>(out + r * k_dim);
        float sum = 0.f;
#pragma unroll 8
        for (int i = lane; i < k_dim / 8; i += 32) {
            uint4 q = __ldg(src + i);
            if (!finite) q = make_uint4(0, 0, 0, 0);
            const uint32_t in[4] = {q.x, q.y, q.z, q.w};
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float a = bf16lo(in[k]) * down, b = bf16hi(in[k]) * down;
                sum += fabsf(a) + fabsf(b);
                const __half2 hh = __floats2half2_rn(a, b);
                o[k] = *reinterpret_cast<const uint32_t*>(&hh);
            }
            dst[i] = make_uint4(o[0], o[1], o[2], o[3]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) lx[r] = (int16_t)(e + exp_of(__float_as_uint(sum * 1.0625f)) + 1);   // its fp32 sum's error and more
    }
}

// Every weight row's exponent: its largest finite scale times 2^-e lies in [2^10, 2^12);
// and of W1, W3 the largest scale and bias of the expert.  A thread takes eight rows and a
// slice of the groups, eight loads in flight (a thread per row waited for one load after the
// other: 37 us for the d_model 4096 layer's 22 MB of scales).  Four slices of groups of 128,
// sixteen of shorter ones: 32 rows an expert of that layer, groups of 128, take 355 us with 4
// slices and 368 with 16, its ReLU form with groups of 32 314 and 294.
// It runs beside the conversion of x, whose launch follows the end of all earlier work: the
// weights' arrays are read and the exponents written before the wait, `top` only behind it.
struct ExpArgs {
    const uint16_t* s[3]; int8_t* e[3];
    const __nv_bfloat16* b[2];
    int rows[3], ng[3];
    const int32_t* offsets; int N;
    int32_t* top;
};
constexpr int kExpThreads = 256;
template <int SLICES> constexpr int kExpRows = kExpThreads / SLICES * 8;   // of a block
template <int SLICES>
__global__ void __launch_bounds__(kExpThreads)
w4_exponent_kernel(const ExpArgs a) {
    constexpr int LANES = kExpThreads / SLICES;
    __shared__ uint4 sh[SLICES][LANES];
    const int m = blockIdx.z, e = blockIdx.y, l = threadIdx.x % LANES, slice = threadIdx.x / LANES;
    const int rows = a.rows[m], row = blockIdx.x * kExpRows<SLICES> + 8 * l;   // rows are multiples of 16
    uint32_t bias = 0;
    uint32_t big[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const bool live = a.s[m] != nullptr && a.offsets[e + 1] > a.offsets[e] && blockIdx.x * kExpRows<SLICES> < rows;
    if (live) {
        uint32_t v[4] = {0, 0, 0, 0};
        // magnitudes of two scales as 16-bit integers; infinities and NaN count as 0
        auto take = [&](uint32_t (&v)[4], const uint4& q) {
            const uint32_t in[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t x = in[i] & 0x7FFF7FFFu;
                v[i] = __vmaxu2(v[i], x & __vcmpltu2(x, 0x7F807F80u));
            }
        };
        if (row < rows) {
            const uint16_t* s = a.s[m] + (int64_t)e * a.ng[m] * rows + row;
#pragma unroll 8
            for (int g = slice; g < a.ng[m]; g += SLICES) take(v, __ldg(reinterpret_cast<const uint4*>(s + (int64_t)g * rows)));
        }
        sh[slice][l] = make_uint4(v[0], v[1], v[2], v[3]);
        __syncthreads();
        if (slice == 0 && row < rows) {
#pragma unroll
            for (int i = 1; i < SLICES; ++i) take(v, sh[i][l]);
#pragma unroll
            for (int i = 0; i < 8; ++i) big[i] = i & 1 ? v[i / 2] & 0xFFFF0000u : v[i / 2] << 16;
            uint32_t out[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i) out[i / 4] |= (uint32_t)(even(max(exp_of(big[i]) - 11, -126)) & 255) << (8 * (i & 3));
            *reinterpret_cast<uint2*>(a.e[m] + (int64_t)e * rows + row) = make_uint2(out[0], out[1]);
            if (m < 2 && a.b[m]) {
                uint32_t b[4] = {0, 0, 0, 0};
                take(b, *reinterpret_cast<const uint4*>(a.b[m] + (int64_t)e * rows + row));
                b[0] = __vmaxu2(__vmaxu2(b[0], b[1]), __vmaxu2(b[2], b[3]));
                bias = max(b[0] >> 16, b[0] & 0xFFFFu) << 16;
            }
#pragma unroll
            for (int i = 1; i < 8; ++i) big[0] = max(big[0], big[i]);
        }
    }
    pdl_wait();
    pdl_launch();
    if (!live || m == 2 || threadIdx.x >= max(32, LANES)) return;   // whole warps with slice 0
    const uint32_t all = __reduce_max_sync(0xffffffffu, big[0]), b = __reduce_max_sync(0xffffffffu, bias);
    if (threadIdx.x % 32 == 0) {   // a maximum: the order of arrival does not matter
        atomicMax(a.top + 2 * m * a.N + e, (int32_t)all);
        atomicMax(a.top + (2 * m + 1) * a.N + e, (int32_t)b);
    }
}

template <int EPI, int G, bool WIDE>
cudaError_t run_tc_g(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& sa, const CUtensorMap& sb,
                     const CUtensorMap& x, const TcParams& p, int sms, cudaStream_t s) {
    auto kern = w4_tc_kernel<EPI, G, WIDE>;
    cudaError_t err = once_per_device(reinterpret_cast<const void*>(kern), [](const void* k) {
        return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<WIDE>::SMEM);
    });
    if (err != cudaSuccess) return err;
    return launch_k(kern, dim3((unsigned)sms), dim3(kThreadsTc), Shape<WIDE>::SMEM, s, 1, a, b, sa, sb, x, p);
}

// one matrix of a stage: its packed rows and its scales
struct Maps {
    CUtensorMap q, s;
    bool make(const W4Mat& w, int N, int rows, int k, int group) {
        return make_map_u8(&q, w.q, (int64_t)N * rows, w4_row_bytes(k), 64) &&
               make_map_u16(&s, w.s, (int64_t)N * ((k + group - 1) / group), rows, 64, 256 / group);
    }
};

template <int EPI, bool WIDE>
cudaError_t run_tc_w(const Maps& a, const Maps& b, const CUtensorMap& x, const TcParams& p, int group, int sms,
                     cudaStream_t s) {
    if (group == 32) return run_tc_g<EPI, 32, WIDE>(a.q, b.q, a.s, b.s, x, p, sms, s);
    if (group == 64) return run_tc_g<EPI, 64, WIDE>(a.q, b.q, a.s, b.s, x, p, sms, s);
    return run_tc_g<EPI, 128, WIDE>(a.q, b.q, a.s, b.s, x, p, sms, s);
}

template <int EPI>
cudaError_t run_tc(const Maps& a, const Maps& b, const CUtensorMap& x, const TcParams& p, int group, int sms,
                   cudaStream_t s) {
    // Wide tiles where they save one (500 rows of each of 8 experts, d_model 4096: 1.12 ms for 1.21);
    // else the overlapped write-out wins (192 rows: 472 us for 526, 384: 875 for 949).
    const int64_t rows = (p.R_cap + p.N - 1) / p.N;   // of an expert, on average
    const bool wide = (rows + Shape<true>::N - 1) / Shape<true>::N < (rows + Shape<false>::N - 1) / Shape<false>::N;
    return wide ? run_tc_w<EPI, true>(a, b, x, p, group, sms, s) : run_tc_w<EPI, false>(a, b, x, p, group, sms, s);
}

}  // namespace

cudaError_t launch_w4_ffn_tc(const W4FfnArgs& a, cudaStream_t s) {
    int sms = 0;
    cudaError_t err = device_sm_count(&sms);
    if (err != cudaSuccess) return err;
    Maps m1, m3, m2;
    CUtensorMap mx, mh;
    if (!m1.make(a.w1, a.N, a.d_ff, a.d, a.group) || !m2.make(a.w2, a.N, a.d, a.d_ff, a.group) ||
        !make_map_bf16(&mx, a.xq, a.R_cap, a.d, kBoxN) || !make_map_bf16(&mh, a.h, a.R_cap, a.d_ff, kBoxN))
        return cudaErrorInvalidValue;
    m3 = m1;
    const bool swiglu = a.act == MOE_SWIGLU;
    if (swiglu && !m3.make(a.w3, a.N, a.d_ff, a.d, a.group)) return cudaErrorInvalidValue;
    // exponents: x's and H's in the place of the few-row kernels' units, the weights' in their own
    int16_t* ex = reinterpret_cast<int16_t*>(a.xu);
    int16_t* lx = ex + a.R_cap;
    int16_t* eh = reinterpret_cast<int16_t*>(a.hu);
    int8_t* e1 = a.wexp;
    int8_t* e3 = e1 + (int64_t)a.N * a.d_ff;
    int8_t* e2 = e3 + (int64_t)a.N * a.d_ff;
    const int64_t rb = (a.R_cap + 7) / 8;
    err = launch_k(w4_half_rows_kernel, dim3((unsigned)(rb < 8 * sms ? rb : 8 * sms)), dim3(256), 0, s, 1, a.xe, a.offsets,
                   a.N, a.R_cap, a.d, reinterpret_cast<__half*>(a.xq), ex, lx, a.top);
    if (err != cudaSuccess) return err;
    ExpArgs ea{};
    const int ng1 = (a.d + a.group - 1) / a.group, ng2 = (a.d_ff + a.group - 1) / a.group;
    ea.s[0] = a.w1.s;
    ea.s[1] = swiglu ? a.w3.s : nullptr;
    ea.s[2] = a.w2.s;
    ea.e[0] = e1;
    ea.e[1] = e3;
    ea.e[2] = e2;
    ea.b[0] = a.b1;
    ea.b[1] = a.b3;
    ea.rows[0] = ea.rows[1] = a.d_ff;
    ea.rows[2] = a.d;
    ea.ng[0] = ea.ng[1] = ng1;
    ea.ng[2] = ng2;
    ea.offsets = a.offsets;
    ea.N = a.N;
    ea.top = a.top;
    const int most = a.d > a.d_ff ? a.d : a.d_ff;
    auto exponents = [&](auto kern, int rows) {
        return launch_k(kern, dim3((unsigned)((most + rows - 1) / rows), (unsigned)a.N, 3u), dim3(kExpThreads), 0, s, 1, ea);
    };
    err = a.group == 128 ? exponents(w4_exponent_kernel<4>, kExpRows<4>) : exponents(w4_exponent_kernel<16>, kExpRows<16>);
    if (err != cudaSuccess) return err;
    TcParams p{};
    p.offsets = a.offsets;
    p.N = a.N;
    p.R_cap = a.R_cap;
    p.status = &a.hdr->status;
    p.limit_ns = kWaitLimitNs;
    p.ea = e1;
    p.eb = e3;
    p.ex = ex;
    p.lx = lx;
    p.eh = eh;
    p.top = a.top;
    p.m_dim = a.d_ff;
    p.k_dim = a.d;
    p.bias_a = a.b1;
    p.bias_b = a.b3;
    p.out = a.h;
    err = a.act == MOE_SWIGLU ? run_tc<W4_SWIGLU>(m1, m3, mx, p, a.group, sms, s)
                              : run_tc<W4_RELU>(m1, m1, mx, p, a.group, sms, s);
    if (err != cudaSuccess) return err;
    p.m_dim = a.d;
    p.k_dim = a.d_ff;
    p.bias_a = a.b2;
    p.bias_b = nullptr;
    p.ea = e2;
    p.ex = eh;
    p.out = a.ye;
    return run_tc<W4_OUT>(m2, m2, mh, p, a.group, sms, s);
}

}  // namespace moe
