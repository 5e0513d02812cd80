// Expert FFN on 4-bit weights for few rows per expert: bound by the one read of
// the weights of every expert that has rows.
//
//   stage 1: H = relu(x W1^T + b1), or silu(x W1^T + b1) * (x W3^T + b3)
//   stage 2: y = H W2^T + b2              W[o][k] = q[o][k] s[o][k / G]
//
// Decoding is what a matrix-vector kernel on 4-bit weights has to get out of the
// way: at the rate of HBM an SM receives about 46 weights a cycle and has 128
// lanes for everything.  Decoded to bf16 a weight costs 1.4 operations (a
// measured kernel stayed at 3.5 TB/s, bound by the integer pipe); as bytes of
// the integer mma.sync m16n8k32 it costs 3/8: one word gives two fragment
// registers by a shift and two logic operations.  So the rows of x (and H)
// are turned into integers, 16 bits per value in blocks of 64 with a unit each
// (w4.cuh), two columns of bytes per token.  Integer sums are exact; per block
// of 64 the two bytes' sums join in fp32 and the unit and the group's scale
// multiply them.  The rounding of x is below 2^-16 of its block's largest value,
// against 2^-9 of y's own rounding to bf16.
// tcgen05 with at most 16 tokens would decode the same words, into shared memory
// or TMEM, for a product that takes a few per cent of the time here.
//
// A CTA has four consumer warps and a producer warp.  Its tile is 128 weight rows
// (64 features of W1 and the same of W3 for SwiGLU) by up to 8 tokens, a
// pipeline stage 256 of K: the producer brings the packed rows with TMA
// (128-byte swizzle) and the tokens' rows and the group scales with cp.async
// into an mbarrier ring.  A consumer warp owns 32 weight rows as two m16 tiles;
// its 16-byte shared loads are, word by word, the A fragments.  Lane g of an mma
// row group reads tile row perm(g): rows 0 4 1 5 2 6 3 7, whose swizzled 16-byte
// chunks fall into different banks.
//
// CTAs take whole tiles, or equal ranges of the list of all tiles' stages.  A tile
// that such a cut divides is added up by the CTA that arrives last, from fp32 parts
// in the workspace, in K order: the result depends on where the cuts fall (on
// the number of tiles), not on the order of arrival.
#include "tc_common.cuh"
#include "w4.cuh"

namespace moe {
using namespace tc;
namespace {

constexpr int kWarps = 4;                        // consumer warps
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kRows = 32 * kWarps;               // weight rows of a tile
constexpr int kStageBlocks = 2;                  // 128-weight blocks of K per stage
constexpr int kStageK = kStageBlocks * kW4Block;
constexpr int kWBytes = kRows * kStageBlocks * kW4BlockBytes;   // 16 KB
constexpr int kOutPitch = kRows + 8;             // conflict-free accumulator writes
constexpr int kMaxStages = 8;
// 128 registers a thread: up to 12 bytes are spilled in stage 1 of ReLU with groups of 64 and in
// stage 2 of SwiGLU with groups of 64 and 128.
constexpr int kCtasPerSm = 3;
constexpr int kSmem = 72 * 1024;                 // of a CTA
constexpr int kBoxRows = 64, kBoxBytes = kBoxRows * 128;       // one TMA box of weights
constexpr int kMinSteps = 2;                     // stages per CTA at least, when they are dealt out
constexpr int kIdleSteps = 8;                    // see the plan
constexpr int kPartFloats = 8 * kRows;          // one fp32 part of a tile

// Rows per expert of the capacity, on average, up to which this kernel is used: at 12 it takes 261 us,
// at 16 279 and at 24 465, where w4_tc.cu takes 356 (d_model 4096, d_ff 14336, 8 SwiGLU experts with
// as many rows each).
constexpr int kFewRows = 16;

enum { W4_RELU = 0, W4_SWIGLU = 1, W4_OUT = 2 };

struct GemvParams {
    const int32_t* offsets; int N; int64_t R_cap;
    int m_dim;                    // output features
    int k_dim;
    const uint16_t* sa; const uint16_t* sb;              // scales (sb: W3)
    const __nv_bfloat16* bias_a; const __nv_bfloat16* bias_b;
    const uint8_t* x; const float* xu;                   // rows as integers, their units
    __nv_bfloat16* out;                                  // stage 2: [R, m_dim]
    uint8_t* hq; float* hu;                              // stage 1: H as integers
    float* part;                  // [CTAs][2][kPartFloats]
    int32_t* count;               // [CTAs] arrivals per shared tile, zero at the start
    int smem_bytes;               // dynamic shared memory of a CTA
    int32_t* status;
    long long limit_ns;
};

__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The first product of a block: c = kMagic + a b.  As bits of a float that is
// 1.5 2^23 + the sum, exact while the sum stays below 2^22 (up to 128 products of at
// most 128 x 128 are 2^21): the conversion to fp32 is one subtraction.
constexpr int kMagic = 0x4B400000;
__device__ __forceinline__ void mma_s8_first(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(kMagic));
}
constexpr float kMagicValue = 12582912.f;   // 1.5 2^23
// kMagicValue + 256 hi + lo, rounded once to fp32
__device__ __forceinline__ float joined(int hi, int lo) {
    return fmaf(__int_as_float(hi) - kMagicValue, 256.f, __int_as_float(lo));
}

// (w ^ 0x88888888) & 0xF0F0F0F0: the odd nibbles as bytes 16 q
__device__ __forceinline__ uint32_t odd_nibbles(uint32_t w) {
    uint32_t u;
    asm("lop3.b32 %0, %1, %2, %3, 0x28;" : "=r"(u) : "r"(w), "r"(0x88888888u), "r"(0xF0F0F0F0u));
    return u;
}

// Eight values of a row as integers: bytes hi and lo of rint(v inv), in fragment order.
__device__ __forceinline__ void to_bytes(const float (&v)[8], float inv, uint2& hi, uint2& lo) {
    uint32_t h[2] = {0, 0}, l[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int k = i / 4 * 2 + (i >> 1 & 1) + 4 * (i & 1);   // 0 4 1 5 2 6 3 7
        const int X = __float2int_rn(v[k] * inv), b = (X + 128 & 255) - 128;
        h[i / 4] |= (uint32_t)((X - b) >> 8 & 255) << (8 * (i & 3));
        l[i / 4] |= (uint32_t)(b & 255) << (8 * (i & 3));
    }
    hi = make_uint2(h[0], h[1]);
    lo = make_uint2(l[0], l[1]);
}
// Units carry a further 2^-12, which the sums' readers take back: kMagicValue times a unit
// and a block's sum (up to 128 x 8 values) stay finite for blocks up to bf16's and fp32's
// largest.  From 2^-95 down units are subnormal, with 18 bits left at 2^-100.
constexpr float kUnitDown = 1.f / 4096.f, kSumUp = 4096.f;
// the unit (over 16) and its reciprocal for a block's largest magnitude, given as bits
__device__ __forceinline__ void block_unit(uint32_t max_bits, float& unit16, float& inv) {
    const float m = __uint_as_float(max_bits);
    const bool finite = max_bits < 0x7F800000u, some = finite && m >= 7.8886e-31f;   // 2^-100
    inv = some ? 32512.f / m : 0.f;
    unit16 = some ? m * (kUnitDown / (16.f * 32512.f)) : (finite ? 0.f : __uint_as_float(0x7FC00000u));
}

// 16 bytes global -> shared; ok = false fills zeros
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
// arrive on the barrier when this thread's copies so far have landed
__device__ __forceinline__ void cp_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// plain loads, so that the compiler moves them ahead of the mma they feed
__device__ __forceinline__ uint4 lds16(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ float lds_bf16(const uint8_t* p) {
    return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(p) << 16);
}
__device__ __forceinline__ uint32_t word_of(const uint4& v, int j) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; }

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    int row[129];
    int exp[128];      // live experts
    int first[129];    // their first unit
    int live, cap, abort, last;
};

// The work of a launch: units (live expert, feature tile, row chunk), each of
// `steps` pipeline stages.  CTA b takes the units b, b + gridDim.x, ...; or (deal)
// the stages of all units form one list, cut into equal ranges, one per CTA.
struct Plan {
    int tiles, steps, chunk;   // feature tiles; stages per unit; rows per chunk
    int units;
    bool deal;
    int ctas, each, rest;      // deal: CTAs with a range; stages / ctas and what is left over
    __device__ int begin(int c) const {   // floor(stages c / ctas) in 32 bits (c, ctas < 2^10)
        return c >= ctas ? units * steps : each * c + rest * c / ctas;
    }
    __device__ int cta_of(int step) const {   // the CTA that holds this stage
        int c = (int)((float)step * ((float)ctas / (float)(units * steps)));
        while (begin(c) > step) --c;
        while (begin(c + 1) <= step) ++c;
        return c;
    }
};

struct Unit {
    int e, m0, row0, n;
};

__device__ __forceinline__ Unit unit_of(const Shared& sh, const Plan& pl, int u, int feats) {
    int lo = 0, hi = sh.live;   // first[lo] <= u < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sh.first[mid] <= u) lo = mid;
        else hi = mid;
    }
    const int e = sh.exp[lo], local = u - sh.first[lo];
    const int chunks = (sh.row[e + 1] - sh.row[e] + pl.chunk - 1) / pl.chunk;
    Unit t;   // the chunks of a feature tile follow one another: its weights are in L2
    t.e = e;
    t.m0 = local / chunks * feats;
    t.row0 = sh.row[e] + local % chunks * pl.chunk;
    t.n = min(pl.chunk, sh.row[e + 1] - t.row0);
    return t;
}

// A CTA's way through its work, segment by segment: stages [k0, k1) of unit u.
struct Walk {
    int u, k0, k1, left;   // deal: the stages after this segment
    __device__ void start(const Plan& pl) {
        k0 = 0;
        if (pl.deal) {
            const int b = pl.begin(blockIdx.x);
            left = pl.begin(blockIdx.x + 1) - b;
            u = b / pl.steps;
            k1 = b - u * pl.steps;   // next() goes on from here
            --u;
        } else {
            u = (int)blockIdx.x - (int)gridDim.x;
            k1 = pl.steps;
        }
    }
    __device__ bool next(const Plan& pl) {
        if (!pl.deal) {
            u += gridDim.x;
            return u < pl.units;
        }
        if (left == 0) return false;
        ++u;
        k0 = k1 == pl.steps ? 0 : k1;
        k1 = min(pl.steps, k0 + left);
        left -= k1 - k0;
        return true;
    }
};

template <int EPI, int G>
struct Shape {
    static constexpr int MATS = EPI == W4_SWIGLU ? 2 : 1;
    static constexpr int FEATS = kRows / MATS;                   // output features of a tile
    static constexpr int SGROUPS = kStageK / G;                  // groups per stage
    static constexpr int S_OFF = kWBytes;                        // scales, behind the weights
    static constexpr int U_OFF = S_OFF + SGROUPS * kRows * 2;    // units: 4 floats a token
};

// A launch's tiles hold up to `cap` (4 or 8) tokens, by its largest expert;
// fewer make the stages smaller and their number larger.
struct Ring {
    uint32_t base;      // shared address
    const uint8_t* ptr;
    int cap, x_off, stage, stages;
};

template <int EPI, int G>
__device__ __forceinline__ void produce(const GemvParams& p, const CUtensorMap* ma, const CUtensorMap* mb, Shared& sh,
                                        const Ring& rg, const Plan& pl, const Waiter& w) {
    using S = Shape<EPI, G>;
    const int lane = threadIdx.x & 31;
    const int ng = (p.k_dim + G - 1) / G;
    const int64_t padded = w4_padded(p.k_dim);
    // the rows of x, their units and the scales of stage ks of tile c
    auto rows_of = [&](const Unit& c, int ks, int st) {
        const int k0 = ks * kStageK;
        const uint32_t base = rg.base + st * rg.stage;
        // a token's 512 bytes: [block of 64][hi, lo][t][16], into [block][column][t][16]
        const uint32_t xd = base + rg.x_off + (lane >> 3) * (rg.cap * 128) + (lane >> 2 & 1) * 64 + (lane & 3) * 16;
        const uint8_t* xs = p.x + ((int64_t)c.row0 * padded + k0) * 2 + lane * 16;
        for (int v = 0; v < c.n; ++v) cp16(xd + v * 128, xs + v * padded * 2, true);
        if (lane < c.n)
            cp16(base + S::U_OFF + lane * 16, p.xu + ((int64_t)(c.row0 + lane) * padded + k0) / kW4ActBlock, true);
        // scales: 8 tile rows a lane
        constexpr int LANES = kRows / 8;
        const int r = lane % LANES * 8;       // tile row
        const uint16_t* sc = S::MATS == 2 && r >= S::FEATS ? p.sb : p.sa;
        const int f = c.m0 + (S::MATS == 2 ? r % S::FEATS : r);
#pragma unroll
        for (int i = 0; i < S::SGROUPS; i += 32 / LANES) {
            const int gi = i + lane / LANES, g = k0 / G + gi;
            const bool have = g < ng && f < p.m_dim;
            cp16(base + S::S_OFF + gi * kRows * 2 + r * 2, have ? sc + ((int64_t)c.e * ng + g) * p.m_dim + f : p.sa, have);
        }
        cp_arrive(smem_u32(&sh.full[st]));
    };
    Walk walk, late;                 // late: the first stages' rows, asked for after the wait
    walk.start(pl);
    late = walk;
    int pending = 0, stage = 0;
    bool waited = false, ok = true;
    auto catch_up = [&]() {
        pdl_wait();
        waited = true;
        for (int i = 0; i < pending && late.next(pl);) {
            const Unit t = unit_of(sh, pl, late.u, S::FEATS);
            for (int ks = late.k0; ks < late.k1 && i < pending; ++ks, ++i) rows_of(t, ks, i);
        }
    };
    uint32_t phase = 0, used = 0;
    while (ok && walk.next(pl)) {
        const Unit t = unit_of(sh, pl, walk.u, S::FEATS);
        constexpr int BOXES = kRows / kBoxRows, PER = BOXES / S::MATS;           // boxes of a matrix
        const int live = min(PER, (p.m_dim - t.m0 + kBoxRows - 1) / kBoxRows);   // those that hold something
        const int row = t.e * p.m_dim + t.m0;
        for (int ks = walk.k0; ks < walk.k1; ++ks) {
            if (!waited && pending == rg.stages) catch_up();   // the ring is full of weights
            ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&sh.empty[stage]), phase ^ 1u, w));
            if (!ok) break;
            if (lane == 0) {
                const uint32_t fb = smem_u32(&sh.full[stage]), base = rg.base + stage * rg.stage;
                mbar_expect_tx(fb, live * S::MATS * kBoxBytes);
#pragma unroll
                for (int b = 0; b < BOXES; ++b)
                    if (b % PER < live)
                        tma_load_2d(base + b * kBoxBytes, b < PER ? ma : mb, fb, ks * kStageBlocks * kW4BlockBytes,
                                    row + b % PER * kBoxRows);
            }
            __syncwarp();
            used |= 1u << stage;
            if (waited) rows_of(t, ks, stage);
            else ++pending;
            if (++stage == rg.stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
    }
    if (!waited) catch_up();
    // nothing of this warp's copies is in flight when the CTA ends
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!ok && lane == 0) {   // aborted: the weights asked for last have landed too
        for (int s = 0; s < rg.stages; ++s)
            if (used >> s & 1u)
                drain_bar(smem_u32(&sh.full[s]), s < stage ? phase : phase ^ 1u, p.limit_ns, p.status);
    }
    __syncwarp();
}

// This warp's part of stages [ks, stop) of one tile of up to 4 NT tokens: the sums
// into s_out[token][tile row].
template <int EPI, int G, int UB, int NT>
__device__ __forceinline__ void tile_sums(const GemvParams& p, Shared& sh, const Ring& rg, float* s_out, int ks, int stop,
                                          int& stage, uint32_t& phase, bool& dead, const Waiter& w) {
    using S = Shape<EPI, G>;
    constexpr int JOIN = (G < UB ? G : UB) / 32;   // words whose sums join at once
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int nb = (p.k_dim + kW4Block - 1) / kW4Block, ng = (p.k_dim + G - 1) / G;
    const int pg = (g >> 1) | ((g & 1) << 2);   // tile row of mma row g: 0 4 1 5 2 6 3 7
    // m16 tile i of this warp: SwiGLU, the same 16 features of either matrix; else 32 rows
    auto tile_row = [&](int i) { return S::MATS == 2 ? i * S::FEATS + 16 * warp : 32 * warp + 16 * i; };
    float acc[2][NT][2];   // [m16 tile][column block][row pg, pg + 8] of token 4 c + t
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int c = 0; c < NT; ++c) acc[i][c][0] = acc[i][c][1] = 0.f;
    for (; ks < stop; ++ks) {
        const int kb0 = ks * kStageBlocks;
        // after an abort the warp only keeps the barriers going
        if (!dead) dead = !__all_sync(0xffffffffu, wait_bar(smem_u32(&sh.full[stage]), phase, w));
        const uint8_t* base = rg.ptr + stage * rg.stage;
#pragma unroll
        for (int b = 0; b < kStageBlocks; ++b) {
            if (dead || kb0 + b >= nb) break;   // a block past K holds nothing
            uint4 wd[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    wd[i][h] = lds16(base + (tile_row(i) + 8 * h + pg) * 128 + (((4 * b + t) ^ pg) << 4));
            int part[2][NT][4];
            uint4 x[NT];   // a column that no token fills holds anything: it is not read back
#pragma unroll
            for (int j = 0; j < 4; ++j) {   // 32 values
                if (j % 2 == 0) {
                    if ((kb0 + b) * kW4Block + j * 32 >= p.k_dim) break;
#pragma unroll
                    for (int c = 0; c < NT; ++c)
                        x[c] = lds16(base + rg.x_off + ((2 * b + j / 2) * 2 * rg.cap + 8 * c + g) * 64 + t * 16);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t w0 = word_of(wd[i][0], j), w1 = word_of(wd[i][1], j);
                    const uint32_t a0 = odd_nibbles(w0 << 4), a1 = odd_nibbles(w1 << 4);
                    const uint32_t a2 = odd_nibbles(w0), a3 = odd_nibbles(w1);
#pragma unroll
                    for (int c = 0; c < NT; ++c) {
                        const uint32_t b0 = j % 2 ? x[c].z : x[c].x, b1 = j % 2 ? x[c].w : x[c].y;
                        if (j % JOIN == 0) mma_s8_first(part[i][c], a0, a1, a2, a3, b0, b1);
                        else mma_s8(part[i][c], a0, a1, a2, a3, b0, b1);
                    }
                }
                // the sums of JOIN x 32 values join: 256 hi + lo, times the unit and the scale
                const bool end = JOIN == 4 ? j == 3 || (j == 1 && (kb0 + b) * kW4Block + 64 >= p.k_dim) : (j + 1) % JOIN == 0;
                const int gi = b * (kW4Block / G) + j * (kW4Block / G) / 4;   // group of the stage
                if (!end || kb0 * (kW4Block / G) + gi >= ng) continue;        // (a last block shorter than 64)
#pragma unroll
                for (int c = 0; c < NT; ++c) {
                    const float un = *reinterpret_cast<const float*>(base + S::U_OFF + (4 * c + t) * 16 + (2 * b + j / 2) * 4);
                    const float off = -kMagicValue * un;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint8_t* sa = base + S::S_OFF + (gi * kRows + tile_row(i) + pg) * 2;
                        acc[i][c][0] = fmaf(fmaf(joined(part[i][c][0], part[i][c][1]), un, off), lds_bf16(sa), acc[i][c][0]);
                        acc[i][c][1] = fmaf(fmaf(joined(part[i][c][2], part[i][c][3]), un, off), lds_bf16(sa + 16), acc[i][c][1]);
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.empty[stage]));
        if (++stage == rg.stages) {
            stage = 0;
            phase ^= 1u;
        }
    }
    named_bar(1, kRows);   // the previous tile's values have been read
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
            for (int r = 0; r < 2; ++r) s_out[(4 * c + t) * kOutPitch + tile_row(i) + pg + 8 * r] = acc[i][c][r];
}

template <int EPI, int G, int UB>
__device__ __forceinline__ void consume(const GemvParams& p, Shared& sh, const Ring& rg, float* s_out, const Plan& pl,
                                        const Waiter& w) {
    using S = Shape<EPI, G>;
    const int tid = threadIdx.x;
    int stage = 0;
    uint32_t phase = 0;
    bool dead = false;
    Walk walk;
    walk.start(pl);
    while (walk.next(pl)) {
        const Unit un = unit_of(sh, pl, walk.u, S::FEATS);
        if (un.n <= 4) tile_sums<EPI, G, UB, 1>(p, sh, rg, s_out, walk.k0, walk.k1, stage, phase, dead, w);
        else tile_sums<EPI, G, UB, 2>(p, sh, rg, s_out, walk.k0, walk.k1, stage, phase, dead, w);
        named_bar(1, kRows);
        if (walk.k1 - walk.k0 < pl.steps) {   // other CTAs hold the rest of the tile's K
            const int u0 = walk.u * pl.steps;
            const int c0 = pl.cta_of(u0), c1 = pl.cta_of(u0 + pl.steps - 1);
            float* dst = p.part + ((int64_t)blockIdx.x * 2 + (walk.k0 > 0 ? 0 : 1)) * kPartFloats;
            for (int col = 0; col < un.n; ++col) __stcg(dst + col * kRows + tid, s_out[col * kOutPitch + tid]);
            named_bar(1, kRows);
            if (tid == 0) {   // the barrier orders the CTA's stores before this thread's fence
                __threadfence();
                const int before = atomicAdd(p.count + c0, 1);
                sh.last = before == c1 - c0;
                __threadfence();
            }
            named_bar(1, kRows);
            if (!sh.last) continue;
            for (int col = 0; col < un.n; ++col) {   // in K order, eight loads at a time
                const float* src = p.part + col * kRows + tid;
                float v = __ldcg(src + ((int64_t)c0 * 2 + 1) * kPartFloats);   // c0's part starts the tile: slot 1
                for (int c = c0 + 1; c <= c1; c += 8) {                        // the later ones start inside it: slot 0
                    float q[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) q[i] = c + i <= c1 ? __ldcg(src + (int64_t)(c + i) * 2 * kPartFloats) : 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) v += q[i];
                }
                s_out[col * kOutPitch + tid] = v;
            }
            named_bar(1, kRows);
        }
        // bias, activation: a thread per feature, the tokens dealt to the tile's MATS halves
        const int f = tid % S::FEATS, feat = un.m0 + f;
        const bool in = feat < p.m_dim;
        const int64_t bi = (int64_t)un.e * p.m_dim + feat;
        const float ba = in && p.bias_a ? __bfloat162float(p.bias_a[bi]) : 0.f;
        const float bb = S::MATS == 2 && in && p.bias_b ? __bfloat162float(p.bias_b[bi]) : 0.f;
        for (int col = tid / S::FEATS; col < un.n; col += S::MATS) {
            float o = fmaf(s_out[col * kOutPitch + f], kSumUp, ba);
            if (EPI == W4_OUT) {
                if (in) p.out[(int64_t)(un.row0 + col) * p.m_dim + feat] = __float2bfloat16_rn(o);
                continue;
            }
            if (EPI == W4_RELU) o = o < 0.f ? 0.f : o;   // NaN stays
            if (EPI == W4_SWIGLU)
                o = o / (1.f + fast_exp2(-o * kLog2e)) * fmaf(s_out[col * kOutPitch + S::FEATS + f], kSumUp, bb);
            s_out[col * kOutPitch + f] = in ? o : 0.f;
        }
        if (EPI == W4_OUT) continue;
        // H as integers: eight lanes per token and 64 features
        named_bar(1, kRows);
        constexpr int BLOCKS = S::FEATS / kW4ActBlock, HUB = EPI == W4_RELU && G == 128 ? 128 : 64;
        const int64_t padded = w4_padded(p.m_dim);
        for (int k0 = 0; k0 < un.n * BLOCKS; k0 += kRows / 8) {
            const int k = k0 + tid / 8, l = tid % 8;
            const int col = k / BLOCKS, blk = k % BLOCKS;
            const bool ok = k < un.n * BLOCKS && un.m0 + blk * kW4ActBlock < p.m_dim;
            float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (ok) {
                const float4* src = reinterpret_cast<const float4*>(s_out + col * kOutPitch + blk * kW4ActBlock + 8 * l);
                const float4 a = src[0], b = src[1];
                v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
                v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
            }
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
            for (int o = HUB / 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            float unit16, inv;
            block_unit(m, unit16, inv);
            uint2 hi, lo;
            to_bytes(v, inv, hi, lo);
            if (ok) {
                const int64_t at = (int64_t)(un.row0 + col) * padded + un.m0 + blk * kW4ActBlock;   // in values
                uint8_t* dst = p.hq + at * 2 + (l & 3) * 16 + (l >> 2) * 8;
                *reinterpret_cast<uint2*>(dst) = hi;
                *reinterpret_cast<uint2*>(dst + 64) = lo;
                if (l == 0) p.hu[at / kW4ActBlock] = unit16;
            }
        }
    }
}

// Rows of x as integers: eight lanes per 64 values, whose unit is that of their
// block of UB (64 or 128).  Clears both stages' counters, whatever the workspace held.
constexpr int kRowThreads = 256;
template <int UB>
__global__ void __launch_bounds__(kRowThreads)
w4_rows_kernel(const __nv_bfloat16* __restrict__ x, const int32_t* __restrict__ offsets, int N, int64_t R_cap, int k_dim,
               uint8_t* __restrict__ xq, float* __restrict__ xu, int32_t* __restrict__ count) {
    pdl_wait();
    pdl_launch();
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < 2 * kW4Counters; i += kRowThreads) count[i] = 0;
    const int64_t last = offsets[N], rows = last < 0 ? 0 : (last > R_cap ? R_cap : last);
    const int64_t padded = w4_padded(k_dim);
    const int blocks = (int)(padded / kW4ActBlock), l = threadIdx.x & 7;
    for (int64_t q0 = (int64_t)blockIdx.x * (kRowThreads / 8); q0 < rows * blocks; q0 += (int64_t)gridDim.x * (kRowThreads / 8)) {
        const int64_t q = q0 + threadIdx.x / 8, row = q / blocks;
        const int k = (int)(q - row * blocks) * kW4ActBlock + 8 * l;
        const bool ok = q < rows * blocks;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (ok && k < k_dim) {
            const uint4 a = *reinterpret_cast<const uint4*>(x + row * k_dim + k);
            v[0] = bf16lo(a.x); v[1] = bf16hi(a.x); v[2] = bf16lo(a.y); v[3] = bf16hi(a.y);
            v[4] = bf16lo(a.z); v[5] = bf16hi(a.z); v[6] = bf16lo(a.w); v[7] = bf16hi(a.w);
        }
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = UB / 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        float unit16, inv;
        block_unit(m, unit16, inv);
        uint2 hi, lo;
        to_bytes(v, inv, hi, lo);
        if (ok) {
            const int64_t at = row * padded + k - 8 * l;
            uint8_t* dst = xq + at * 2 + (l & 3) * 16 + (l >> 2) * 8;
            *reinterpret_cast<uint2*>(dst) = hi;
            *reinterpret_cast<uint2*>(dst + 64) = lo;
            if (l == 0) xu[at / kW4ActBlock] = unit16;
        }
    }
}

template <int EPI, int G, int UB>
__device__ __forceinline__ void run_tiles(const GemvParams& p, const CUtensorMap* ma, const CUtensorMap* mb, Shared& sh,
                                          uint8_t* smem) {
    using S = Shape<EPI, G>;
    const int tid = threadIdx.x;
    Plan pl;
    pl.tiles = (p.m_dim + S::FEATS - 1) / S::FEATS;
    pl.steps = (p.k_dim + kStageK - 1) / kStageK;
    if (tid < 32) {   // live experts and their first units: four experts a lane, a scan over the lanes
        int n[4], live = 0, units = 0, most = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = 4 * tid + i;
            n[i] = e < p.N ? max(0, sh.row[e + 1] - sh.row[e]) : 0;
            most = max(most, n[i]);
        }
        most = __reduce_max_sync(0xffffffffu, most);
        const int cap = most <= 4 ? 4 : 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            live += n[i] > 0;
            units += (n[i] + cap - 1) / cap * pl.tiles;
        }
        int l = live, u = units;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int lo = __shfl_up_sync(0xffffffffu, l, o), uo = __shfl_up_sync(0xffffffffu, u, o);
            if (tid >= o) {
                l += lo;
                u += uo;
            }
        }
        if (tid == 31) {
            sh.live = l;
            sh.first[l] = u;
            sh.cap = cap;
        }
        l -= live;
        u -= units;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n[i] > 0) {
                sh.exp[l] = 4 * tid + i;
                sh.first[l++] = u;
                u += (n[i] + cap - 1) / cap * pl.tiles;
            }
    }
    __syncthreads();
    Ring rg;
    rg.cap = sh.cap;
    rg.x_off = (S::U_OFF + rg.cap * 16 + 127) / 128 * 128;
    rg.stage = (rg.x_off + rg.cap * 2 * kStageK + 1023) / 1024 * 1024;
    rg.stages = min(kMaxStages, (p.smem_bytes - 1024 - rg.cap * kOutPitch * 4) / rg.stage);
    rg.base = smem_u32(smem);
    rg.ptr = smem;
    pl.chunk = rg.cap;
    pl.units = sh.first[sh.live];
    // Whole units leave CTAs idle in the last wave; dealing out stages costs the
    // shared tiles' parts.  The former while it idles less than kIdleSteps stages
    // per CTA: with 2 the 32 ReLU experts (16 stages, 0.42 of the CTAs idle) took
    // 59 us and not 52, the odd sizes 22.7 and not 21.7; one and sixteen tokens of
    // the d_model 4096 layer (16 and 56 stages) deal either way.
    const int grid = gridDim.x, over = pl.units % grid;
    pl.deal = over > 0 && (int64_t)(grid - over) * pl.steps > (int64_t)kIdleSteps * grid;
    pl.ctas = pl.deal ? min((pl.units * pl.steps + kMinSteps - 1) / kMinSteps, grid) : min(pl.units, grid);
    pl.each = pl.deal ? pl.units * pl.steps / pl.ctas : 0;
    pl.rest = pl.units * pl.steps - pl.each * pl.ctas;
    if ((int)blockIdx.x >= pl.ctas) {   // nothing to do
        pdl_wait();
        pdl_launch();
        return;
    }
    float* s_out = reinterpret_cast<float*>(smem + rg.stages * rg.stage);
    const Waiter w{&sh.abort, p.status, p.limit_ns};
    if (tid >= 32 * kWarps) {
        produce<EPI, G>(p, ma, mb, sh, rg, pl, w);
    } else {
        pdl_wait();
        pdl_launch();
        consume<EPI, G, UB>(p, sh, rg, s_out, pl, w);
    }
}

template <int EPI, int G, int UB>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
w4_gemv_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const GemvParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    __shared__ __align__(8) Shared sh;
    const int tid = threadIdx.x;
    if (tid == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(smem_u32(&sh.full[s]), 1 + 32);     // the TMA's expect and the producer lanes' copies
            mbar_init(smem_u32(&sh.empty[s]), kWarps);
        }
        sh.abort = 0;
        mbar_fence_init();
        prefetch_tmap(&map_a);
        prefetch_tmap(&map_b);
    }
    // A stage may start while its predecessor (the rows' conversion, stage 1) drains:
    // the offsets and the weights are inputs of the whole call, complete before
    // the conversion began, so they are read before the wait for the rows.
    for (int i = tid; i <= p.N; i += kThreads) {
        const int64_t v = p.offsets[i];
        sh.row[i] = (int)(v < 0 ? 0 : (v > p.R_cap ? p.R_cap : v));
    }
    __syncthreads();
    run_tiles<EPI, G, UB>(p, &map_a, &map_b, sh, smem);
}

// packed rows [rows][pitch] bytes: boxes of 64 rows x 128 bytes, 128-byte swizzle
bool make_map_w4(CUtensorMap* map, const void* q, int64_t rows, int64_t pitch) {
    return make_map_u8(map, q, rows, pitch, kBoxRows);
}

template <int EPI, int G, int UB>
cudaError_t run_gemv_g(const CUtensorMap& a, const CUtensorMap& b, GemvParams p, int sms, cudaStream_t s) {
    auto kern = w4_gemv_kernel<EPI, G, UB>;
    cudaError_t err = once_per_device(reinterpret_cast<const void*>(kern), [](const void* k) {
        return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    });
    if (err != cudaSuccess) return err;
    p.smem_bytes = kSmem;
    return launch_k(kern, dim3((unsigned)w4_gemv_ctas(sms)), dim3(kThreads), kSmem, s, 1, a, b, p);
}

// Groups of 128: one unit per 128 values and one join per group, except for the H
// of SwiGLU, whose tiles have 64 features.
template <int EPI, int UB128>
cudaError_t run_gemv(const CUtensorMap& a, const CUtensorMap& b, const GemvParams& p, int group, int sms, cudaStream_t s) {
    if (group == 32) return run_gemv_g<EPI, 32, 64>(a, b, p, sms, s);
    if (group == 64) return run_gemv_g<EPI, 64, 64>(a, b, p, sms, s);
    return run_gemv_g<EPI, 128, UB128>(a, b, p, sms, s);
}

}  // namespace

int w4_gemv_ctas(int sms) { return sms * kCtasPerSm < kW4Counters ? sms * kCtasPerSm : kW4Counters; }
int64_t w4_part_bytes() { return (int64_t)kW4Counters * 2 * kPartFloats * 4; }

cudaError_t launch_w4_ffn(const W4FfnArgs& a, cudaStream_t s) {
    if (a.R_cap > (int64_t)kFewRows * a.N) return launch_w4_ffn_tc(a, s);
    int sms = 0;
    cudaError_t err = device_sm_count(&sms);
    if (err != cudaSuccess) return err;
    CUtensorMap m1, m3, m2;
    if (!make_map_w4(&m1, a.w1.q, (int64_t)a.N * a.d_ff, w4_row_bytes(a.d)) ||
        !make_map_w4(&m2, a.w2.q, (int64_t)a.N * a.d, w4_row_bytes(a.d_ff)))
        return cudaErrorInvalidValue;
    m3 = m1;
    if (a.act == MOE_SWIGLU && !make_map_w4(&m3, a.w3.q, (int64_t)a.N * a.d_ff, w4_row_bytes(a.d)))
        return cudaErrorInvalidValue;
    GemvParams p{};
    p.offsets = a.offsets;
    p.N = a.N;
    p.R_cap = a.R_cap;
    p.part = a.part;
    p.status = &a.hdr->status;
    p.limit_ns = kWaitLimitNs;
    p.m_dim = a.d_ff;
    p.k_dim = a.d;
    p.sa = a.w1.s;
    p.sb = a.w3.s;
    p.bias_a = a.b1;
    p.bias_b = a.b3;
    p.x = a.xq;
    p.xu = a.xu;
    p.hq = a.hq;
    p.hu = a.hu;
    p.count = a.count;
    const int64_t row_blocks = (a.R_cap * (w4_padded(a.d) / kW4ActBlock) + kRowThreads / 8 - 1) / (kRowThreads / 8);
    err = launch_k(a.group == 128 ? w4_rows_kernel<128> : w4_rows_kernel<64>,
                   dim3((unsigned)(row_blocks < 8 * sms ? row_blocks : 8 * sms)), dim3(kRowThreads), 0, s, 1, a.xe, a.offsets,
                   a.N, a.R_cap, a.d, a.xq, a.xu, a.count);
    if (err != cudaSuccess) return err;
    err = a.act == MOE_SWIGLU ? run_gemv<W4_SWIGLU, 128>(m1, m3, p, a.group, sms, s)
                              : run_gemv<W4_RELU, 128>(m1, m3, p, a.group, sms, s);
    if (err != cudaSuccess) return err;
    p.m_dim = a.d;
    p.k_dim = a.d_ff;
    p.sa = a.w2.s;
    p.bias_a = a.b2;
    p.bias_b = nullptr;
    p.x = a.hq;
    p.xu = a.hu;
    p.out = a.ye;
    p.count = a.count + kW4Counters;
    return a.act == MOE_SWIGLU ? run_gemv<W4_OUT, 64>(m2, m2, p, a.group, sms, s)
                               : run_gemv<W4_OUT, 128>(m2, m2, p, a.group, sms, s);
}

}  // namespace moe
