// Expert FFN on 4-bit weights for many rows per expert, on tcgen05.
//
//   stage 1: H = relu(x W1^T + b1), or silu(x W1^T + b1) * (x W3^T + b3)
//   stage 2: y = H W2^T + b2              W[o][k] = q[o][k] s[o][k / G]
//
// The weights are the A operand: a tile is 128 weight rows by up to 128 tokens, so
// each word is decoded once for 128 tokens, and a thread that decodes owns one
// row.  Decoded words are bf16 integers, exact, and go straight into TMEM
// (tcgen05.st), from where tcgen05.mma reads A: through shared memory the
// operand would be written and read again beside the tokens' tiles, more than the
// 128 bytes a cycle that shared memory has.  The scales do not enter the operands
// (q s has up to 12 significant bits, bf16 8): the products of one group
// accumulate in TMEM from zero, and a thread per weight row adds them, times the
// row's scale, to its fp32 sums in registers -- one fma per output and group.
// H is rounded to bf16 between the stages, as in the layer on bf16 weights.
//
// Roles (576 threads): warp 0 TMA (packed rows; the tokens' rows of x), warp 1 MMA
// issue and TMEM, warps 2-9 decode, warps 10-17 add up and write out.  TMEM: two
// partial accumulators of 128 columns, two A buffers of 64 (128 of K).  SwiGLU
// puts a feature's W1 row on lane l < 16 and its W3 row on lane l + 16 of the same
// warp, so the gate and the value meet by a shuffle.
// Every wait is bounded; on expiry the kernel latches MOE_ERR_TIMEOUT, stops
// issuing, waits (bounded) for its copies and MMAs, frees TMEM and returns.
#include "tc_common.cuh"
#include "w4.cuh"

namespace moe {
using namespace tc;
namespace {

constexpr int kThreadsTc = 576;
constexpr int kTileN = 128;                       // tokens of a tile
constexpr int kHalfN = kTileN / 2;                // ... of a group of four adding warps
constexpr int kBoxN = 32;                         // tokens per TMA box
constexpr int kWStages = 3;                       // packed rows: 256 of K each
constexpr int kXStages = 4;                       // tokens: 128 of K each
constexpr int kWBytes = 128 * 128;
constexpr int kXSub = kTileN * 128;               // 64 of K
constexpr int kXBytes = 2 * kXSub;
constexpr int kSmemTc = kWStages * kWBytes + kXStages * kXBytes + 1024;
constexpr uint32_t kColD = 0, kColA = 256;        // TMEM columns

enum { W4_RELU = 0, W4_SWIGLU = 1, W4_OUT = 2 };

struct TcParams {
    const int32_t* offsets; int N; int64_t R_cap;
    int m_dim, k_dim;
    const uint16_t* sa; const uint16_t* sb;
    const __nv_bfloat16* bias_a; const __nv_bfloat16* bias_b;
    __nv_bfloat16* out;           // [R, m_dim]
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
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
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

// Weights 2 p and 2 p + 1 of a word's eight as a bf16 pair of integers: 128 + (q + 8)
// is exact in bf16 (0x4300 is 128, whose last place is 1), and so is the difference.
__device__ __forceinline__ uint32_t decode_pair(uint32_t w, int p) {
    uint32_t u;   // one operation: written as two immediates it would be two
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(u) : "r"(w >> (4 * p)), "r"(0x000F000Fu), "r"(0x43004300u));
    const uint32_t c = 0x43084308u;   // 136, 136
    const __nv_bfloat162 r =
        __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u), *reinterpret_cast<const __nv_bfloat162*>(&c));
    return *reinterpret_cast<const uint32_t*>(&r);
}

struct SharedTc {
    uint64_t wfull[kWStages], wempty[kWStages], xfull[kXStages], xempty[kXStages];
    uint64_t afull[2], aempty[2], dfull[2], dempty[2], done;
    uint32_t tmem;
    int abort, live;
    int row[129], exp[128], first[129];
};

struct Tile {
    int e, m0, row0, n;
};

// rows of an expert in equal chunks of at most 128, a multiple of 16
__device__ __forceinline__ int chunk_rows(int n) {
    const int chunks = (n + kTileN - 1) / kTileN;
    return ((n + chunks - 1) / chunks + 15) / 16 * 16;
}

__device__ __forceinline__ Tile tile_of(const SharedTc& sh, int u, int feats) {
    int lo = 0, hi = sh.live;   // first[lo] <= u < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sh.first[mid] <= u) lo = mid;
        else hi = mid;
    }
    const int e = sh.exp[lo], rows = sh.row[e + 1] - sh.row[e], local = u - sh.first[lo];
    const int per = chunk_rows(rows), chunks = (rows + per - 1) / per;
    Tile t;   // the chunks of a feature tile follow one another: its weights are in L2
    t.e = e;
    t.m0 = local / chunks * feats;
    t.row0 = sh.row[e] + local % chunks * per;
    t.n = min(per, sh.row[e + 1] - t.row0);
    return t;
}

template <int EPI, int G>
__global__ void __launch_bounds__(kThreadsTc, 1)
w4_tc_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
             const __grid_constant__ CUtensorMap map_x, const TcParams p) {
    constexpr int MATS = EPI == W4_SWIGLU ? 2 : 1;
    constexpr int FEATS = 128 / MATS;
    constexpr int PER = kW4Block / G;   // groups per 128 of K
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* smem_x = smem + kWStages * kWBytes;
    __shared__ __align__(8) SharedTc sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < kWStages; ++s) {
            mbar_init(smem_u32(&sh.wfull[s]), 1);
            mbar_init(smem_u32(&sh.wempty[s]), 8);
        }
        for (int s = 0; s < kXStages; ++s) {
            mbar_init(smem_u32(&sh.xfull[s]), 1);
            mbar_init(smem_u32(&sh.xempty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.afull[i]), 4);
            mbar_init(smem_u32(&sh.aempty[i]), 1);
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
    if (warp == 2) {   // live experts and their first units: four experts a lane, a scan over the lanes
        int n[4], live = 0, units = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = 4 * lane + i, rows = e < p.N ? max(0, sh.row[e + 1] - sh.row[e]) : 0;
            n[i] = rows == 0 ? 0 : (rows + chunk_rows(rows) - 1) / chunk_rows(rows) * tiles;
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

    if (warp == 0) {
        // ---------------- TMA ----------------
        if (lane == 0) {
            int ws = 0, xs = 0;
            uint32_t wph = 0, xph = 0, wused = 0, xused = 0;
            bool ok = true;
            for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
                const Tile t = tile_of(sh, u, FEATS);
                const int row = t.e * p.m_dim + t.m0;
                const bool second = MATS == 2 || t.m0 + 64 < p.m_dim;   // the upper 64 rows hold something
                const int boxes = (t.n + kBoxN - 1) / kBoxN;
                for (int kb = 0; kb < nb; ++kb) {
                    if (kb % 2 == 0) {
                        if (!(ok = wait_bar(smem_u32(&sh.wempty[ws]), wph ^ 1u, w))) break;
                        const uint32_t fb = smem_u32(&sh.wfull[ws]), dst = smem_u32(smem + ws * kWBytes);
                        mbar_expect_tx(fb, second ? kWBytes : kWBytes / 2);
                        tma_load_2d(dst, &map_a, fb, kb * kW4BlockBytes, row);
                        if (second)
                            tma_load_2d(dst + kWBytes / 2, MATS == 2 ? &map_b : &map_a, fb, kb * kW4BlockBytes,
                                        MATS == 2 ? row : row + 64);
                        wused |= 1u << ws;
                        if (++ws == kWStages) {
                            ws = 0;
                            wph ^= 1u;
                        }
                    }
                    if (!(ok = wait_bar(smem_u32(&sh.xempty[xs]), xph ^ 1u, w))) break;
                    const uint32_t fb = smem_u32(&sh.xfull[xs]), dst = smem_u32(smem_x + xs * kXBytes);
                    const int halves = kb * kW4Block + 64 < p.k_dim ? 2 : 1;
                    mbar_expect_tx(fb, halves * boxes * kBoxN * 128);
                    for (int h = 0; h < halves; ++h)
                        for (int b = 0; b < boxes; ++b)
                            tma_load_2d(dst + h * kXSub + b * kBoxN * 128, &map_x, fb, kb * kW4Block + h * 64,
                                        t.row0 + b * kBoxN);
                    xused |= 1u << xs;
                    if (++xs == kXStages) {
                        xs = 0;
                        xph ^= 1u;
                    }
                }
            }
            // every load has landed before the CTA retires (normally long consumed)
            for (int s = 0; s < kWStages; ++s)
                if (wused >> s & 1u) drain_bar(smem_u32(&sh.wfull[s]), s < ws ? wph : wph ^ 1u, p.limit_ns, p.status);
            for (int s = 0; s < kXStages; ++s)
                if (xused >> s & 1u) drain_bar(smem_u32(&sh.xfull[s]), s < xs ? xph : xph ^ 1u, p.limit_ns, p.status);
        }
    } else if (warp == 1) {
        // ---------------- MMA ----------------
        if (lane == 0) {
            int xs = 0, a = 0, d = 0;
            uint32_t xph = 0, aph = 0, dph = 0;
            bool ok = true, issued = false;
            for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
                const Tile t = tile_of(sh, u, FEATS);
                const uint32_t idesc = idesc_bf16_f32(128, (t.n + 15) / 16 * 16);
                for (int kb = 0; kb < nb && ok; ++kb) {
                    ok = wait_bar(smem_u32(&sh.xfull[xs]), xph, w) && wait_bar(smem_u32(&sh.afull[a]), aph, w);
                    if (!ok) break;
                    const uint64_t bd = umma_desc(smem_u32(smem_x + xs * kXBytes));
                    const uint32_t ad = tmem + kColA + a * 64;
                    const int nk = min(8, (p.k_dim - kb * kW4Block) / 16);   // K is a multiple of 16
#pragma unroll
                    for (int gi = 0; gi < PER; ++gi) {
                        if (gi * (8 / PER) >= nk) break;
                        if (!(ok = wait_bar(smem_u32(&sh.dempty[d]), dph ^ 1u, w))) break;
                        tc_fence_after();
                        issued = true;
#pragma unroll
                        for (int kk = gi * (8 / PER); kk < (gi + 1) * (8 / PER); ++kk)
                            if (kk < nk)
                                umma_ts(tmem + kColD + d * 128, ad + 8 * kk, bd + (uint64_t)((kk / 4 * kXSub) >> 4) + 2 * (kk % 4),
                                        idesc, kk > gi * (8 / PER));
                        umma_commit(smem_u32(&sh.dfull[d]));
                        d ^= 1;
                        if (d == 0) dph ^= 1u;
                    }
                    if (!ok) break;
                    umma_commit(smem_u32(&sh.aempty[a]));
                    umma_commit(smem_u32(&sh.xempty[xs]));
                    a ^= 1;
                    if (a == 0) aph ^= 1u;
                    if (++xs == kXStages) {
                        xs = 0;
                        xph ^= 1u;
                    }
                }
            }
            if (issued) {   // every MMA has completed before TMEM is freed
                umma_commit(smem_u32(&sh.done));
                drain_bar(smem_u32(&sh.done), 0u, p.limit_ns, p.status);
            }
        }
    } else if (warp < 10) {
        // ---------------- decode: lane = weight row ----------------
        // two groups of four warps, one for each A buffer: they take blocks in turn
        const int quad = warp & 3;   // TMEM lane quadrant
        const int a = (warp - 2) >> 2;
        // SwiGLU: lanes 0-15 hold 16 features of W1, lanes 16-31 the same of W3
        const int r = MATS == 2 ? (lane >> 4) * 64 + quad * 16 + (lane & 15) : quad * 32 + lane;
        int ws = 0, turn = 0;
        uint32_t wph = 0, aph = 0;
        bool ok = true;
        for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
            for (int kb = 0; kb < nb && ok; ++kb, turn ^= 1) {
                if (kb % 2 == 0) ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&sh.wfull[ws]), wph, w));
                if (!ok) break;
                const bool mine = turn == a;
                uint4 q[4];
                if (mine) {
                    const uint8_t* src = smem + ws * kWBytes + r * 128;
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        q[t] = *reinterpret_cast<const uint4*>(src + (((kb % 2 * 4 + t) ^ (r & 7)) << 4));
                }
                if (kb % 2 == 1 || kb + 1 == nb) {   // both groups are done with the stage
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sh.wempty[ws]));
                    if (++ws == kWStages) {
                        ws = 0;
                        wph ^= 1u;
                    }
                }
                if (!mine) continue;
                if (!(ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&sh.aempty[a]), aph ^ 1u, w)))) break;
                aph ^= 1u;
                tc_fence_after();
                const uint32_t dst = tmem + kColA + a * 64 + ((uint32_t)(quad * 32) << 16);
#pragma unroll
                for (int half = 0; half < 2; ++half) {   // columns 32 half .. : words j = 2 half, 2 half + 1
                    uint32_t v[32];
#pragma unroll
                    for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const int j = 2 * half + jj;
                            const uint32_t word = j == 0 ? q[t].x : j == 1 ? q[t].y : j == 2 ? q[t].z : q[t].w;
#pragma unroll
                            for (int i = 0; i < 4; ++i) v[16 * jj + 4 * t + i] = decode_pair(word, i);
                        }
                    tmem_st32(dst + 32 * half, v);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.afull[a]));
            }
        }
    } else {
        // ---------------- add up and write out: lane = weight row ----------------
        // two groups of four warps, 64 of the tile's tokens each
        const int quad = warp & 3, c0 = (warp - 10) / 4 * kHalfN;
        const int f = MATS == 2 ? quad * 16 + (lane & 15) : quad * 32 + lane;   // feature of the tile
        const uint16_t* sc = MATS == 2 && lane >= 16 ? p.sb : p.sa;
        const __nv_bfloat16* bias = MATS == 2 && lane >= 16 ? p.bias_b : p.bias_a;
        const int ng = (p.k_dim + G - 1) / G;
        int d = 0;
        uint32_t dph = 0;
        bool ok = true;
        for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
            const Tile t = tile_of(sh, u, FEATS);
            const int feat = t.m0 + f;
            const bool in = feat < p.m_dim;
            const uint16_t* srow = sc + (int64_t)t.e * ng * p.m_dim + (in ? feat : 0);
            const int n = t.n - c0;   // this group's tokens (may be none)
            float acc[kHalfN];
#pragma unroll
            for (int c = 0; c < kHalfN; ++c) acc[c] = 0.f;
            uint16_t s0 = __ldg(srow), s1 = ng > 1 ? __ldg(srow + p.m_dim) : 0;
            for (int g = 0; g < ng; ++g) {
                const float s = __uint_as_float((uint32_t)s0 << 16);
                s0 = s1;
                s1 = g + 2 < ng ? __ldg(srow + (int64_t)(g + 2) * p.m_dim) : 0;   // two groups ahead
                if (!(ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&sh.dfull[d]), dph, w)))) break;
                tc_fence_after();
                const uint32_t src = tmem + kColD + d * 128 + c0 + ((uint32_t)(quad * 32) << 16);
#pragma unroll
                for (int c = 0; c < kHalfN / 16; ++c) {
                    if (16 * c < n) {
                        uint32_t v[16];
                        tmem_ld16(src + 16 * c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) acc[16 * c + i] = fmaf(__uint_as_float(v[i]), s, acc[16 * c + i]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.dempty[d]));
                d ^= 1;
                if (d == 0) dph ^= 1u;
            }
            if (!ok) break;
            const float b = in && bias ? __bfloat162float(bias[(int64_t)t.e * p.m_dim + feat]) : 0.f;
            __nv_bfloat16* dst = p.out + (int64_t)(t.row0 + c0) * p.m_dim + feat;
            if (EPI == W4_SWIGLU) {
                // lanes < 16 finish the even tokens, their partners the odd ones
#pragma unroll
                for (int c = 0; c < kHalfN; c += 2) {
                    if (c >= n) continue;   // (a break would put acc in local memory)
                    const float mine = lane < 16 ? acc[c] + b : acc[c + 1] + b, send = lane < 16 ? acc[c + 1] + b : acc[c] + b;
                    const float other = __shfl_xor_sync(0xffffffffu, send, 16);
                    const float gate = lane < 16 ? mine : other, up = lane < 16 ? other : mine;
                    const int col = c + (lane >> 4);
                    if (in && col < n)
                        dst[(int64_t)col * p.m_dim] =
                            __float2bfloat16_rn(gate / (1.f + fast_exp2(-gate * kLog2e)) * up);
                }
            } else {
#pragma unroll
                for (int c = 0; c < kHalfN; ++c) {
                    float o = acc[c] + b;
                    if (EPI == W4_RELU) o = o < 0.f ? 0.f : o;   // NaN stays
                    if (in && c < n) dst[(int64_t)c * p.m_dim] = __float2bfloat16_rn(o);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int EPI, int G>
cudaError_t run_tc_g(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& x, const TcParams& p, int sms,
                     cudaStream_t s) {
    auto kern = w4_tc_kernel<EPI, G>;
    cudaError_t err = once_per_device(reinterpret_cast<const void*>(kern), [](const void* k) {
        return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemTc);
    });
    if (err != cudaSuccess) return err;
    return launch_k(kern, dim3((unsigned)sms), dim3(kThreadsTc), kSmemTc, s, 1, a, b, x, p);
}

template <int EPI>
cudaError_t run_tc(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& x, const TcParams& p, int group, int sms,
                   cudaStream_t s) {
    if (group == 32) return run_tc_g<EPI, 32>(a, b, x, p, sms, s);
    if (group == 64) return run_tc_g<EPI, 64>(a, b, x, p, sms, s);
    return run_tc_g<EPI, 128>(a, b, x, p, sms, s);
}

}  // namespace

cudaError_t launch_w4_ffn_tc(const W4FfnArgs& a, cudaStream_t s) {
    int sms = 0;
    cudaError_t err = device_sm_count(&sms);
    if (err != cudaSuccess) return err;
    CUtensorMap m1, m3, m2, mx, mh;
    if (!make_map_u8(&m1, a.w1.q, (int64_t)a.N * a.d_ff, w4_row_bytes(a.d), 64) ||
        !make_map_u8(&m2, a.w2.q, (int64_t)a.N * a.d, w4_row_bytes(a.d_ff), 64) ||
        !make_map_bf16(&mx, a.xe, a.R_cap, a.d, kBoxN) || !make_map_bf16(&mh, a.h, a.R_cap, a.d_ff, kBoxN))
        return cudaErrorInvalidValue;
    m3 = m1;
    if (a.act == MOE_SWIGLU && !make_map_u8(&m3, a.w3.q, (int64_t)a.N * a.d_ff, w4_row_bytes(a.d), 64))
        return cudaErrorInvalidValue;
    TcParams p{};
    p.offsets = a.offsets;
    p.N = a.N;
    p.R_cap = a.R_cap;
    p.status = &a.hdr->status;
    p.limit_ns = kWaitLimitNs;
    p.m_dim = a.d_ff;
    p.k_dim = a.d;
    p.sa = a.w1.s;
    p.sb = a.w3.s;
    p.bias_a = a.b1;
    p.bias_b = a.b3;
    p.out = a.h;
    err = a.act == MOE_SWIGLU ? run_tc<W4_SWIGLU>(m1, m3, mx, p, a.group, sms, s)
                              : run_tc<W4_RELU>(m1, m1, mx, p, a.group, sms, s);
    if (err != cudaSuccess) return err;
    p.m_dim = a.d;
    p.k_dim = a.d_ff;
    p.sa = a.w2.s;
    p.bias_a = a.b2;
    p.bias_b = nullptr;
    p.out = a.ye;
    return run_tc<W4_OUT>(m2, m2, mh, p, a.group, sms, s);
}

}  // namespace moe
