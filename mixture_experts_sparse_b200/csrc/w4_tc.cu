// Expert FFN on 4-bit weights for many rows per expert, on tcgen05.
//
//   stage 1: H = relu(x W1^T + b1), or silu(x W1^T + b1) * (x W3^T + b3)
//   stage 2: y = H W2^T + b2              W[o][k] = q[o][k] s[o][k / G]
//
// The weights are the A operand: a tile is 128 weight rows by up to 192 tokens, so
// each word is decoded once for 192 tokens, and a thread that decodes owns one
// row.  Decoded words are bf16 integers, exact, and go straight into TMEM
// (tcgen05.st), from where tcgen05.mma reads A: through shared memory the
// operand would be written and read again beside the tokens' tiles, more than the
// 128 bytes a cycle that shared memory has.  The scales do not enter the operands
// (q s has up to 12 significant bits, bf16 8): the products of one group
// accumulate in TMEM from zero, and a thread per weight row adds them, times the
// row's scale, to its fp32 sums in registers -- one fma per output and group.
// H is rounded to bf16 between the stages, as in the layer on bf16 weights.
//
// Bound: the instructions around the MMAs.  A block of 128 rows x 128 of K is 860
// warp instructions to decode and, with 192 tokens, about 1100 to add up, for MMAs
// of 800 cycles; hence the wide tile (all 512 columns of TMEM: two partial
// accumulators of 192, two A buffers of 64), and 96 sums per adding thread, whose
// registers setmaxnreg takes from the other warps.  Single-lane branches around
// TMA, MMA and commit use elect.sync in a warp-uniform loop: with `lane == 0` each
// such instruction took 45 cycles to issue instead of 9.
//
// Roles (five warpgroups): warp 0 TMA of the tokens' rows, 1 MMA issue, 2 TMA of
// the packed rows and scales (they come from HBM and are asked for further ahead);
// warps 4-11 decode, in turns, one group per A buffer; warps 12-19 add up and
// write out, 96 tokens a group.  SwiGLU puts a feature's W1 row on lane l < 16 and
// its W3 row on lane l + 16 of the same warp, so the gate and the value meet by a
// shuffle.
// Every wait is bounded; on expiry the kernel latches MOE_ERR_TIMEOUT, stops
// issuing, waits (bounded) for its copies and MMAs, frees TMEM and returns.
#include "tc_common.cuh"
#include "w4.cuh"

namespace moe {
using namespace tc;
namespace {

constexpr int kAddGroups = 2;                     // warpgroups that add up
constexpr int kThreadsTc = 128 * (3 + kAddGroups);
constexpr int kTileN = 192;                       // tokens of a tile
constexpr int kPartN = kTileN / kAddGroups;       // ... of a group of adding warps
constexpr int kBoxN = 32;                         // tokens per TMA box
constexpr int kWStages = 4;                       // packed rows and scales: 256 of K each
constexpr int kXStages = 3;                       // tokens: 128 of K each
constexpr int kWBytes = 128 * 128;
constexpr int kXSub = kTileN * 128;               // 64 of K
constexpr int kXBytes = 2 * kXSub;
constexpr int kSBytes = 2048;                     // scales of a stage: 2 boxes x 256 / G groups x 64 rows
constexpr int kSmemTc = kWStages * (kWBytes + kSBytes) + kXStages * kXBytes + 1024;
constexpr uint32_t kColD = 0, kColA = 2 * kTileN; // TMEM columns
// Registers per thread: the launch's 640 x 96 are dealt out anew, 40 + 2 x 72 +
// 2 x 144 = 472 <= 5 x 96 per warpgroup lane.
constexpr int kRegsLaunch = 96, kRegsControl = 32, kRegsDecode = 64, kRegsAdd = 160;
static_assert(kRegsControl + 2 * kRegsDecode + kAddGroups * kRegsAdd <= (3 + kAddGroups) * kRegsLaunch, "register pool");
template <int R>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }

enum { W4_RELU = 0, W4_SWIGLU = 1, W4_OUT = 2 };

struct TcParams {
    const int32_t* offsets; int N; int64_t R_cap;
    int m_dim, k_dim;
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
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// two fp32 fused multiply-adds in one instruction
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

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
    uint64_t wfull[kWStages], wempty[kWStages], sempty[kWStages];   // wfull: rows and scales
    uint64_t xfull[kXStages], xempty[kXStages];
    uint64_t afull[2];              // a block's weights are in TMEM
    uint64_t mdone[2];              // its MMAs are done: A is free, (G = 128) its sums are there
    uint64_t dfull[2], dempty[2];   // partial accumulators; dfull: G < 128
    uint64_t done;
    uint32_t tmem;
    int abort, live;
    int row[129], exp[128], first[129];
};

struct Tile {
    int e, m0, row0, n;
};

// rows of an expert in equal chunks of at most 192, a multiple of 16
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
             const __grid_constant__ CUtensorMap map_sa, const __grid_constant__ CUtensorMap map_sb,
             const __grid_constant__ CUtensorMap map_x, const TcParams p) {
    constexpr int MATS = EPI == W4_SWIGLU ? 2 : 1;
    constexpr int FEATS = 128 / MATS;
    constexpr int PER = kW4Block / G;   // groups per 128 of K
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* smem_x = smem + kWStages * kWBytes;
    uint8_t* smem_s = smem_x + kXStages * kXBytes;
    __shared__ __align__(8) SharedTc sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < kWStages; ++s) {
            mbar_init(smem_u32(&sh.wfull[s]), 1);
            mbar_init(smem_u32(&sh.wempty[s]), 8);
            mbar_init(smem_u32(&sh.sempty[s]), 4 * kAddGroups);
        }
        for (int s = 0; s < kXStages; ++s) {
            mbar_init(smem_u32(&sh.xfull[s]), 1);
            mbar_init(smem_u32(&sh.xempty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.afull[i]), 8);
            mbar_init(smem_u32(&sh.mdone[i]), 1);
            mbar_init(smem_u32(&sh.dfull[i]), 1);
            mbar_init(smem_u32(&sh.dempty[i]), 4 * kAddGroups);
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

    if (warp < 4) {
        regs_dec<kRegsControl>();
        if (warp == 0) {
            // ---------------- TMA: the tokens' rows ----------------
            int xs = 0;
            uint32_t xph = 0, xused = 0;
            bool ok = true;
            for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
                const Tile t = tile_of(sh, u, FEATS);
                const int boxes = (t.n + kBoxN - 1) / kBoxN;
                for (int kb = 0; kb < nb; ++kb) {
                    ok = __all_sync(0xffffffffu, wait_bar_soon(smem_u32(&sh.xempty[xs]), xph ^ 1u, w));
                    if (!ok) break;
                    const uint32_t fb = smem_u32(&sh.xfull[xs]), dst = smem_u32(smem_x) + xs * kXBytes;
                    const int halves = kb * kW4Block + 64 < p.k_dim ? 2 : 1;
                    if (elect_one()) {
                        mbar_expect_tx(fb, halves * boxes * kBoxN * 128);
                        for (int h = 0; h < halves; ++h)
                            for (int b = 0; b < boxes; ++b)
                                tma_load_2d(dst + h * kXSub + b * kBoxN * 128, &map_x, fb, kb * kW4Block + h * 64,
                                            t.row0 + b * kBoxN);
                    }
                    __syncwarp();
                    xused |= 1u << xs;
                    if (++xs == kXStages) {
                        xs = 0;
                        xph ^= 1u;
                    }
                }
            }
            // every load has landed before the CTA retires
            for (int s = 0; s < kXStages; ++s)
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
                    ok = __all_sync(0xffffffffu, wait_bar_soon(smem_u32(&sh.wempty[ws]), wph ^ 1u, w) &&
                                                     wait_bar_soon(smem_u32(&sh.sempty[ws]), wph ^ 1u, w));
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
                    if (++ws == kWStages) {
                        ws = 0;
                        wph ^= 1u;
                    }
                }
            }
            for (int s = 0; s < kWStages; ++s)
                if (wused >> s & 1u) drain_bar(smem_u32(&sh.wfull[s]), s < ws ? wph : wph ^ 1u, p.limit_ns, p.status);
        } else if (warp == 1) {
            // ---------------- MMA ----------------
            int xs = 0, a = 0, d = 0;
            uint32_t xph = 0, aph = 0, dph = 0;
            bool ok = true, issued = false;
            const uint64_t bd0 = umma_desc(smem_u32(smem_x));
            for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
                const Tile t = tile_of(sh, u, FEATS);
                const uint32_t idesc = idesc_bf16_f32(128, (t.n + 15) / 16 * 16);
                for (int kb = 0; kb < nb && ok; ++kb) {
                    ok = __all_sync(0xffffffffu, wait_bar_soon(smem_u32(&sh.afull[a]), aph, w) &&
                                                     wait_bar_soon(smem_u32(&sh.xfull[xs]), xph, w));
                    if (!ok) break;
                    const uint64_t bd = bd0 + (uint64_t)(xs * (kXBytes >> 4));
                    const uint32_t ad = tmem + kColA + a * 64;
                    const int nk = min(8, (p.k_dim - kb * kW4Block) / 16);   // K is a multiple of 16
#pragma unroll
                    for (int gi = 0; gi < PER; ++gi) {
                        if (gi * (8 / PER) >= nk) break;
                        if (!(ok = __all_sync(0xffffffffu, wait_bar_soon(smem_u32(&sh.dempty[d]), dph ^ 1u, w)))) break;
                        tc_fence_after();
                        issued = true;
                        const uint32_t dd = tmem + kColD + d * kTileN;
                        if (elect_one()) {
#pragma unroll
                            for (int kk = gi * (8 / PER); kk < (gi + 1) * (8 / PER); ++kk)
                                if (kk < nk)
                                    umma_ts(dd, ad + 8 * kk, bd + (uint64_t)((kk / 4 * kXSub) >> 4) + 2 * (kk % 4), idesc,
                                            kk > gi * (8 / PER));
                            if (PER > 1) umma_commit(smem_u32(&sh.dfull[d]));
                            if (gi == PER - 1 || (gi + 1) * (8 / PER) >= nk) {
                                umma_commit(smem_u32(&sh.mdone[a]));
                                umma_commit(smem_u32(&sh.xempty[xs]));
                            }
                        }
                        __syncwarp();
                        d ^= 1;
                        if (d == 0) dph ^= 1u;
                    }
                    a ^= 1;
                    if (a == 0) aph ^= 1u;
                    if (++xs == kXStages) {
                        xs = 0;
                        xph ^= 1u;
                    }
                }
            }
            if (issued) {   // every MMA has completed before TMEM is freed
                if (elect_one()) umma_commit(smem_u32(&sh.done));
                __syncwarp();
                drain_bar(smem_u32(&sh.done), 0u, p.limit_ns, p.status);
            }
        }
    } else if (warp < 12) {
        // ---------------- decode: lane = weight row ----------------
        // two groups of four warps, half of every block each: the words t = 2 h, 2 h + 1,
        // columns 16 j + 8 h .. + 7.  They decode into registers before they wait for
        // the A buffer, so only the stores are between one MMA and the next but one.
        regs_dec<kRegsDecode>();
        const int quad = warp & 3;   // TMEM lane quadrant
        const int h = (warp - 4) >> 2;
        // SwiGLU: lanes 0-15 hold 16 features of W1, lanes 16-31 the same of W3
        const int r = MATS == 2 ? (lane >> 4) * 64 + quad * 16 + (lane & 15) : quad * 32 + lane;
        int ws = 0, a = 0;
        uint32_t wph = 0, aph = 0;
        bool ok = true;
        for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
            for (int kb = 0; kb < nb && ok; ++kb) {
                if (kb % 2 == 0) ok = __all_sync(0xffffffffu, wait_bar_soon(smem_u32(&sh.wfull[ws]), wph, w));
                if (!ok) break;
                const uint8_t* src = smem + ws * kWBytes + r * 128;
                uint32_t v[32];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const uint4 q = *reinterpret_cast<const uint4*>(src + (((kb % 2 * 4 + 2 * h + t) ^ (r & 7)) << 4));
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t word = j == 0 ? q.x : j == 1 ? q.y : j == 2 ? q.z : q.w;
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[8 * j + 4 * t + i] = decode_pair(word, i);
                    }
                }
                if (kb % 2 == 1 || kb + 1 == nb) {   // this warp is done with the stage
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sh.wempty[ws]));
                    if (++ws == kWStages) {
                        ws = 0;
                        wph ^= 1u;
                    }
                }
                if (!(ok = __all_sync(0xffffffffu, wait_bar_soon(smem_u32(&sh.mdone[a]), aph ^ 1u, w)))) break;
                tc_fence_after();
                const uint32_t dst = tmem + kColA + a * 64 + 8 * h + ((uint32_t)(quad * 32) << 16);
#pragma unroll
                for (int j = 0; j < 4; ++j) tmem_st8(dst + 16 * j, v + 8 * j);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.afull[a]));
                a ^= 1;
                if (a == 0) aph ^= 1u;
            }
        }
    } else {
        // ---------------- add up and write out: lane = weight row ----------------
        // two groups of four warps, 96 of the tile's tokens each
        regs_inc<kRegsAdd>();
        const int quad = warp & 3, c0 = (warp - 12) / 4 * kPartN;
        const int f = MATS == 2 ? quad * 16 + (lane & 15) : quad * 32 + lane;   // feature of the tile
        // its scales in a stage: box, then 64 features a group
        const int soff = (MATS == 2 ? (lane >> 4) * (2 * PER * 64) + f : f / 64 * (2 * PER * 64) + f % 64) * 2;
        const __nv_bfloat16* bias = MATS == 2 && lane >= 16 ? p.bias_b : p.bias_a;
        const int ng = (p.k_dim + G - 1) / G;
        int d = 0, ws = 0;
        uint32_t dph = 0, wph = 0;
        bool ok = true;
        for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
            const Tile t = tile_of(sh, u, FEATS);
            const int feat = t.m0 + f;
            const bool in = feat < p.m_dim;
            const int n = t.n - c0;   // this group's tokens (may be none)
            uint64_t acc2[kPartN / 2];   // pairs of fp32 sums (fma.rn.f32x2)
#pragma unroll
            for (int c = 0; c < kPartN / 2; ++c) acc2[c] = 0;
            for (int g = 0; g < ng; ++g) {
                const int gs = g % (2 * PER);   // group of the stage
                if (gs == 0 && !(ok = __all_sync(0xffffffffu, wait_bar_soon(smem_u32(&sh.wfull[ws]), wph, w)))) break;
                const float s = __uint_as_float(
                    (uint32_t)*reinterpret_cast<const uint16_t*>(smem_s + ws * kSBytes + gs * 128 + soff) << 16);
                if (gs == 2 * PER - 1 || g + 1 == ng) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sh.sempty[ws]));
                    if (++ws == kWStages) {
                        ws = 0;
                        wph ^= 1u;
                    }
                }
                ok = __all_sync(0xffffffffu, wait_bar_soon(smem_u32(PER > 1 ? &sh.dfull[d] : &sh.mdone[d]), dph, w));
                if (!ok) break;
                tc_fence_after();
                const uint32_t src = tmem + kColD + d * kTileN + c0 + ((uint32_t)(quad * 32) << 16);
                const uint64_t s2 = pack_f32x2(s, s);
                auto release = [&]() {   // this warp's last read of the buffer
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sh.dempty[d]));
                };
                if (n <= 0) release();
#pragma unroll
                for (int c = 0; c < kPartN / 32; ++c) {
                    if (32 * c < n) {
                        uint32_t v[32];
                        tmem_ld32(src + 32 * c, v);
                        tmem_wait_ld();
                        if (32 * (c + 1) >= n || c + 1 == kPartN / 32) release();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            acc2[16 * c + i] = fma_f32x2(pack_f32x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), s2,
                                                         acc2[16 * c + i]);
                    }
                }
                d ^= 1;
                if (d == 0) dph ^= 1u;
            }
            if (!ok) break;
            float acc[kPartN];
#pragma unroll
            for (int c = 0; c < kPartN / 2; ++c) unpack_f32x2(acc2[c], acc[2 * c], acc[2 * c + 1]);
            const float b = in && bias ? __bfloat162float(bias[(int64_t)t.e * p.m_dim + feat]) : 0.f;
            __nv_bfloat16* dst = p.out + (int64_t)(t.row0 + c0) * p.m_dim + feat;
            if (EPI == W4_SWIGLU) {
                // lanes < 16 finish the even tokens, their partners the odd ones
                const bool low = lane < 16;
                if (!low) dst += p.m_dim;
#pragma unroll
                for (int c = 0; c < kPartN; c += 2) {
                    if (c < n) {   // (a break would put acc in local memory)
                        const float mine = (low ? acc[c] : acc[c + 1]) + b, send = (low ? acc[c + 1] : acc[c]) + b;
                        const float other = __shfl_xor_sync(0xffffffffu, send, 16);
                        const float gate = low ? mine : other, up = low ? other : mine;
                        // e^-z -> inf for very negative z: the fast division gives the limit 0
                        const float o = __fdividef(gate, 1.f + fast_exp2(-gate * kLog2e)) * up;
                        if (in && (low || c + 1 < n)) *dst = __float2bfloat16_rn(o);
                        dst += 2 * p.m_dim;
                    }
                }
            } else {
#pragma unroll
                for (int c = 0; c < kPartN; ++c) {
                    if (c < n) {
                        float o = acc[c] + b;
                        if (EPI == W4_RELU) o = o < 0.f ? 0.f : o;   // NaN stays
                        if (in) *dst = __float2bfloat16_rn(o);
                        dst += p.m_dim;
                    }
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
cudaError_t run_tc_g(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& sa, const CUtensorMap& sb,
                     const CUtensorMap& x, const TcParams& p, int sms, cudaStream_t s) {
    auto kern = w4_tc_kernel<EPI, G>;
    cudaError_t err = once_per_device(reinterpret_cast<const void*>(kern), [](const void* k) {
        return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemTc);
    });
    if (err != cudaSuccess) return err;
    return launch_k(kern, dim3((unsigned)sms), dim3(kThreadsTc), kSmemTc, s, 1, a, b, sa, sb, x, p);
}

// one matrix of a stage: its packed rows and its scales
struct Maps {
    CUtensorMap q, s;
    bool make(const W4Mat& w, int N, int rows, int k, int group) {
        return make_map_u8(&q, w.q, (int64_t)N * rows, w4_row_bytes(k), 64) &&
               make_map_u16(&s, w.s, (int64_t)N * ((k + group - 1) / group), rows, 64, 256 / group);
    }
};

template <int EPI>
cudaError_t run_tc(const Maps& a, const Maps& b, const CUtensorMap& x, const TcParams& p, int group, int sms,
                   cudaStream_t s) {
    if (group == 32) return run_tc_g<EPI, 32>(a.q, b.q, a.s, b.s, x, p, sms, s);
    if (group == 64) return run_tc_g<EPI, 64>(a.q, b.q, a.s, b.s, x, p, sms, s);
    return run_tc_g<EPI, 128>(a.q, b.q, a.s, b.s, x, p, sms, s);
}

}  // namespace

cudaError_t launch_w4_ffn_tc(const W4FfnArgs& a, cudaStream_t s) {
    int sms = 0;
    cudaError_t err = device_sm_count(&sms);
    if (err != cudaSuccess) return err;
    Maps m1, m3, m2;
    CUtensorMap mx, mh;
    if (!m1.make(a.w1, a.N, a.d_ff, a.d, a.group) || !m2.make(a.w2, a.N, a.d, a.d_ff, a.group) ||
        !make_map_bf16(&mx, a.xe, a.R_cap, a.d, kBoxN) || !make_map_bf16(&mh, a.h, a.R_cap, a.d_ff, kBoxN))
        return cudaErrorInvalidValue;
    m3 = m1;
    if (a.act == MOE_SWIGLU && !m3.make(a.w3, a.N, a.d_ff, a.d, a.group)) return cudaErrorInvalidValue;
    TcParams p{};
    p.offsets = a.offsets;
    p.N = a.N;
    p.R_cap = a.R_cap;
    p.status = &a.hdr->status;
    p.limit_ns = kWaitLimitNs;
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
    p.out = a.ye;
    return run_tc<W4_OUT>(m2, m2, mh, p, a.group, sms, s);
}

}  // namespace moe
