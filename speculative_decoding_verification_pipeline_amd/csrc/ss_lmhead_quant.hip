// LM-head logits from 4-bit weights with group scales (gfx950 bf16 MFMA).
//
//   y[b, v] = sum_g s[v, g] ( sum_{k in g} (n[v, k] - z[v, g]) x[b, k] )
//
// What bounds it: the weight stream (V K / 2 bytes) while the rows are few, and
// beside it, at 64 rows, the vector ALU that widens nibbles, the matrix cores
// and the LDS reads of x.
//
//  * Widening costs two operations for two weights: byte j of a word times
//    2^3 + 2^15 puts its nibbles on the top mantissa bits of two bfloat16, and
//    under the exponent of 16 they read 16 + n, exactly. (Widening to s (n - z)
//    would round every weight to 8 bits.) The matrix cores sum (16 + n) x; the
//    scaled group is added in binary32, and
//      - sum_g s (16 + z) (sum_{k in g} x)
//    is a product over groups of its own, four groups per binary32 MFMA. Its sums
//    of x come from MFMAs against ones, each batch tile's made by one wave and
//    shared through LDS, so this part follows a set of four groups later: until
//    then the outputs carry sums of (16 + n) x and are rounded at their size, five
//    times that of the result for x around 0 and more where x has a mean. Of the
//    result's norm the error is 1.3e-7 to 3.3e-7 in groups of 128 and 2.5e-7 to
//    5.3e-7 in groups of 32, K = 256 to 8192, x ~ N(0, 1) (a binary32 matrix product
//    of the weights: 2.2e-7 to 1.5e-6; it is the better one at K = 1024, 8 rows,
//    groups of 32, 2.4e-7 against 3.7e-7); with x ~ N(1, 1) up to 7.6e-7 and 2.0e-6
//    (1.4e-7 to 1.5e-6). Taken off each group before it is scaled it would round
//    less, but every wave would need the sums of all its tiles of x: 12 MFMAs a step
//    for 9 at 64 rows.
//  * v_mfma_f32_16x16x32_bf16 with x as the A operand (batch rows) and W as B
//    (vocabulary rows as columns): a lane's accumulators then belong to the
//    vocabulary row whose weights it widens, so the scale is one value per lane
//    and row tile.
//  * Operands go from memory to LDS by global_load_lds_dwordx4, a stage of 128 BPS k
//    ahead, so the stream stays in flight without registers. Each of the two stages
//    is an LDS object of its own: the compiler then orders a read against the
//    copies into its own stage only, which the explicit wait has seen land. A
//    wave copies the weights it uses and its share of x. What lies behind K is
//    copied as zeros of x, so no block is special.
//  * Any assignment of k to MFMA slots is right as long as both operands share
//    it. A lane's 16 bytes are 32 weights of one row, its four words serve four
//    MFMAs: for groups of 128 as they are, for groups of 64 and 32 after
//    exchanging words between the lanes that hold the same row (permlane
//    swaps), so that no MFMA crosses a group.
//  * The row blocks left over beyond a multiple of the CUs, or all where they are
//    few, are cut along K between workgroups; the one that arrives last adds the
//    parts, in order.
//  * WAVES waves: RW row blocks of RT tiles by KW ranges of K, whose sums are
//    added in a fixed order through LDS.
#include <type_traits>
#include <utility>

#include "ss_device.h"
#include "ss_internal.h"

namespace ss {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int LQ_KB = 128;   // k per block: 16 bytes of weights per lane and row tile

#define LQ_LDS(x) ((__attribute__((address_space(3))) void*)(x))

constexpr int LQ_WAIT = 0x0070;  // s_waitcnt with vmcnt 0, lgkmcnt 0, expcnt free (gfx9 encoding)

// Word of eight nibbles -> eight bfloat16 16 + n, in order. mask and exponent come
// in vector registers: one v_and_or_b32 takes them, literals would take two
// operations.
struct LqWiden {
    uint32_t mask, exponent;
    __device__ __forceinline__ LqWiden() {
        asm("v_mov_b32 %0, 0x780078" : "=v"(mask));
        asm("v_mov_b32 %0, 0x41804180" : "=v"(exponent));
    }
    __device__ __forceinline__ bf16x8 operator()(uint32_t w) const {
        u32x4 r;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            r[j] = (__umul24(w >> 8 * j & 0xFFu, 0x8008u) & mask) | exponent;
        return __builtin_bit_cast(bf16x8, r);
    }
};

__device__ __forceinline__ void lq_swap32(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void lq_swap16(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

// Exchanges words between the lanes l, l ^ 16, l ^ 32, l ^ 48 (one row) so that
// MFMA i multiplies words of one group only.
template <int GROUP>
__device__ __forceinline__ u32x4 lq_regroup(u32x4 w) {
    uint32_t a = w[0], b = w[1], c = w[2], d = w[3];
    if (GROUP <= 64) {
        lq_swap32(a, c);
        lq_swap32(b, d);
    }
    if (GROUP <= 32) {
        lq_swap16(a, b);
        lq_swap16(c, d);
    }
    return u32x4{a, b, c, d};
}

// A stage holds BPS blocks of 128 k. A copy moves rows of 64 BPS bytes, 16 / BPS
// of them, consecutive lanes a row: memory requests are formed over consecutive
// lanes. With BPS = 2 a row of weights is a whole 128-byte line (K a multiple of
// 256), read once and not kept (non-temporal); with BPS = 1 its halves come a stage apart, and the
// line has to stay in L2 meanwhile. In LDS row r's 16-byte unit j lies at
// 64 BPS r + 16 (j ^ swizzle(r)). A read of 16 bytes a lane is served sixteen lanes
// at a time, and not sixteen in a row: rows 0 .. 3 and 12 .. 15 of one quarter
// with rows 4 .. 11 of the next. The swizzle spreads those over all banks, whatever
// unit each of the two quarters reads (bits 0 and 1 of r / 4 are b and c: c, b ^ c
// from the top; by r / 2 alone a seventh of the time went into conflicts).
//
// x of one 16-row tile and stage is four such tiles of 32 BPS k. MFMA i, quarter
// q of the wave reads the unit that lq_regroup gives it: unit 4 q + i of the
// block (128); 8 (i / 2) + i % 2 + 2 q', q' the bits of q reversed (64); 4 i + q
// (32). The lane's part of that is its offset, the step's part is added, or, in
// the bits the swizzle uses, goes in by xor.
template <int BPS>
__device__ __forceinline__ int lq_swizzle(int r) {
    const int c = r >> 3 & 1, bc = (r >> 2 & 1) ^ c;
    return BPS == 2 ? c << 2 | bc << 1 | (r >> 1 & 1) : bc << 1 | c;
}
template <int BPS>
__device__ __forceinline__ uint32_t lq_unit(int r, int j) {
    return r * 64 * BPS + ((j ^ lq_swizzle<BPS>(r)) << 4);
}
template <int GROUP, int BPS>
__device__ __forceinline__ uint32_t lq_lane_offset(int lane) {
    const int q = lane >> 4, r = lane & 15;
    if (GROUP == 32) return lq_unit<BPS>(r, q);
    if (BPS == 2) {
        if (GROUP == 64) return lq_unit<BPS>(r, (q & 1) * 4 + (q >> 1) * 2);
        return (q >> 1) * 2048 + lq_unit<BPS>(r, (q & 1) * 4);
    }
    if (GROUP == 64) return (q & 1) * 1024 + lq_unit<BPS>(r, q & 2);
    return q * 1024 + lq_unit<BPS>(r, 0);
}
template <int GROUP, int BPS>
constexpr int lq_step_offset(int i) {
    return GROUP == 128 ? 0 : GROUP == 64 || BPS == 2 ? (i >> 1) * 2048 : i * 1024;
}
template <int GROUP, int BPS>
constexpr int lq_step_xor(int i) {
    return GROUP == 128 ? i << 4 : GROUP == 64 ? (i & 1) << 4 : BPS == 2 ? (i & 1) << 6 : 0;
}

__device__ __forceinline__ u32x4 lq_at(const uint8_t* p) { return *reinterpret_cast<const u32x4*>(p); }

__device__ __forceinline__ floatx4 lq_mfma(bf16x8 x, bf16x8 w, floatx4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w, c, 0, 0, 0);
}

// Scale and zero point of one group of one vocabulary row, as loaded: those of
// groups behind the last one are 0.
struct LqRaw {
    uint32_t s, z;
};

__device__ __forceinline__ LqRaw lq_load(const QuantArgs& a, int v, int g, int n_groups) {
    LqRaw r = {0u, 8u};
    if (g < n_groups) {
        r.s = a.scales[(int64_t)v * n_groups + g];
        if (a.zeros) r.z = a.zeros[(int64_t)v * ((n_groups + 1) / 2) + (g >> 1)] >> (g & 1) * 4 & 15;
    }
    return r;
}

__device__ __forceinline__ float lq_scale(uint32_t bits, bool f16) {
    return f16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)bits) : __uint_as_float(bits << 16);
}

template <class F, int... I>
__device__ __forceinline__ void lq_each(F& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}

__device__ __forceinline__ uint64_t lq_pair(float lo, float hi) {
    return (uint64_t)__float_as_uint(hi) << 32 | __float_as_uint(lo);
}

__device__ const u32x4 lq_zero = {0u, 0u, 0u, 0u};

template <int GROUP, int NT, int RT, int KW, int WAVES, int BPS>
__global__ __launch_bounds__(WAVES* WAVE, 2) void k_lmhead_quant(QuantArgs a) {
    constexpr int RW = WAVES / KW;
    constexpr int ROWS = RW * RT * 16;           // vocabulary rows per workgroup
    constexpr int GPB = LQ_KB / GROUP;           // groups per block
    constexpr int PER = 4 / GPB;                 // MFMAs per group
    constexpr int GPS = GPB * BPS;               // groups per stage
    constexpr int SET = GPS < 4 ? 4 / GPS : 1;   // stages per set of four groups
    constexpr int SPS = GPS > 4 ? GPS / 4 : 1;   // sets per stage
    constexpr int XT = 4096 * BPS;               // bytes of a tile of x, of a tile of weights
    constexpr int WT_ = 1024 * BPS;
    constexpr int XB = KW * NT * XT;             // bytes of x, of weights per stage
    constexpr int WB = WAVES * RT * WT_;
    constexpr int XC = NT * KW * 4 * BPS / WAVES;  // copies of x per wave and stage
    __shared__ __attribute__((aligned(1024))) uint8_t b0[XB + WB];
    __shared__ __attribute__((aligned(1024))) uint8_t b1[XB + WB];
    __shared__ float s_sum[2 * SPS][KW][4][NT * 16];  // sums of x over a set's groups
    __shared__ float s_scale[WAVES][SPS][4][RT * 16];
    const int tid = threadIdx.x;
    const int lane = tid & (WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int rw = wave % RW, kw = wave / RW;
    const int r16 = lane & 15, quarter = lane >> 4;
    const int K = a.K, V = a.V;
    // the first workgroups take a part of K of one of the last row blocks each
    const bool part = (int)blockIdx.x < a.split_blocks * a.split;
    const int row_block = part ? a.whole_blocks + blockIdx.x / a.split : blockIdx.x - a.split_blocks * a.split;
    const int row0 = row_block * ROWS + rw * RT * 16;
    const int n_groups = (K + GROUP - 1) / GROUP;
    // stages of a range: whole sets where there are several ranges
    const int all = (K + LQ_KB * BPS - 1) / (LQ_KB * BPS);
    const int start = part ? blockIdx.x % a.split * a.split_stages : 0;
    const int own = part ? a.split_stages : all;
    const int stages = KW > 1 ? ((own + KW - 1) / KW + SET - 1) / SET * SET : min(own, all - start);
    const int first_stage = start + kw * stages;
    // Each workgroup starts at a set of its own, so that the rows that are read
    // at the same time are read at different places: rows a power of two apart
    // would otherwise meet in the same memory channels. A last, partial set
    // stays last.
    const int whole_sets = stages / SET;
    const int turn = (int)((blockIdx.x * 2654435761u >> 8) % (unsigned)max(whole_sets, 1));
    auto place = [&](int j) {
        int set = j / SET;
        if (set < whole_sets) {
            set += turn;
            set = set >= whole_sets ? set - whole_sets : set;
        }
        return set * SET + j % SET;
    };
    // Each wave takes the tiles of x in an order of its own: the first is the one
    // whose sums it makes.
    auto tile_of = [&](int n) { return (n + rw) % NT; };
    const bool f16 = a.scale_f16 != 0;
    const LqWiden widen;
    const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});

    // This lane's place in a copy, as an offset from an address that is the same
    // for the wave: a stage's copies then cost the vector ALU nothing.
    constexpr int LPR = 4 * BPS, RPC = 16 / BPS;  // lanes per row, rows per copy
    auto unit_of = [&](int row) { return (lane % LPR) ^ lq_swizzle<BPS>(row); };
    const uint8_t* wbase[RT];
    uint32_t woff[RT][BPS];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int first = min(row0 + t * 16, V - 1);
        wbase[t] = a.qweight + (int64_t)first * (K / 2);
#pragma unroll
        for (int c = 0; c < BPS; ++c) {
            const int row = c * RPC + lane / LPR;
            woff[t][c] = (uint32_t)(min(row0 + t * 16 + row, V - 1) - first) * (K / 2) + unit_of(row) * 16;
        }
    }
    // x: copy u of the stage is rows (u % BPS) RPC .. of segment (u / BPS) % 4 of
    // tile u / (4 BPS) % NT of range u / (4 BPS NT); a wave's XC copies follow
    // each other and stay within one tile.
    static_assert(XC * WAVES == NT * KW * 4 * BPS && 4 * BPS % XC == 0, "copies of x");
    const int xu = wave * XC;
    const int xtile = xu / (4 * BPS) % NT, xrange = xu / (4 * BPS * NT);
    const uint8_t* xbase = reinterpret_cast<const uint8_t*>(a.hidden);
    // lines that hold parts of two copies are kept for the second (K = 4160: 41.7 -> 39.2 us)
    const bool whole_lines = BPS == 2 && K % 256 == 0;
    uint32_t xoff[BPS];
#pragma unroll
    for (int c = 0; c < BPS; ++c) {
        const int row = c * RPC + lane / LPR;
        xoff[c] = (uint32_t)min(xtile * 16 + row, a.B - 1) * (uint32_t)K * 2 + unit_of(row) * 16;
    }
    // Copies of a stage, from addresses kept in bounds.
    auto copy = [&](uint8_t* buf, int j) {
        uint8_t* ws = buf + XB + wave * RT * WT_;
        const int at = place(j);
        const int kb = (first_stage + at) * BPS;
        if ((kb + BPS) * LQ_KB <= K) {
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int c = 0; c < BPS; ++c) {
                    const void* src = wbase[t] + (int64_t)kb * (LQ_KB / 2) + woff[t][c];
                    if (whole_lines) __builtin_amdgcn_global_load_lds(src, LQ_LDS(ws + t * WT_ + c * 1024), 16, 0, 2);
                    else __builtin_amdgcn_global_load_lds(src, LQ_LDS(ws + t * WT_ + c * 1024), 16, 0, 0);
                }
        } else {
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int c = 0; c < BPS; ++c) {
                    const int64_t k = (int64_t)kb * (LQ_KB / 2) + unit_of(c * RPC + lane / LPR) * 16;
                    const int64_t back = k > K / 2 - 16 ? k - (K / 2 - 16) : 0;
                    __builtin_amdgcn_global_load_lds(
                        (const void*)(wbase[t] + (int64_t)kb * (LQ_KB / 2) + woff[t][c] - back),
                        LQ_LDS(ws + t * WT_ + c * 1024), 16, 0, 0);
                }
        }
        const int k0 = (start + xrange * stages + at) * BPS * LQ_KB;
        uint8_t* xs = buf + xu * 1024;
#pragma unroll
        for (int i = 0; i < XC; ++i) {
            const int u = xu % (4 * BPS) + i;
            const int c = XC % BPS == 0 ? i % BPS : u % BPS;  // known ahead where a wave has several
            const uint32_t off = BPS == 2 && c ? xoff[BPS - 1] : xoff[0];
            const uint8_t* src = xbase + ((int64_t)k0 + u / BPS * 32 * BPS) * 2 + off;
            if (k0 + BPS * LQ_KB > K) {
                const int k = k0 + u / BPS * 32 * BPS + unit_of(c * RPC + lane / LPR) * 8;
                if (k >= K) src = reinterpret_cast<const uint8_t*>(&lq_zero);
            }
            __builtin_amdgcn_global_load_lds((const void*)src, LQ_LDS(xs + i * 1024), 16, 0, 0);
        }
    };

    floatx4 out[RT][NT];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n) out[t][n] = floatx4{0.f, 0.f, 0.f, 0.f};
    for (int i = tid; i < 2 * SPS * KW * 4 * NT * 16; i += WAVES * WAVE) (&s_sum[0][0][0][0])[i] = 0.f;

    // A lane loads scale and zero point of the one group of a set that its quarter
    // contributes to the product of the sums, a set ahead; the wave's lanes share
    // the scales through LDS.
    LqRaw next[SPS][RT];
    float c_now[SPS][RT], c_before[SPS][RT];
#pragma unroll
    for (int h = 0; h < SPS; ++h)
#pragma unroll
        for (int t = 0; t < RT; ++t) c_now[h][t] = 0.f;
    auto load_scales = [&](int j) {
#pragma unroll
        for (int h = 0; h < SPS; ++h)
#pragma unroll
            for (int t = 0; t < RT; ++t)
                next[h][t] = lq_load(a, min(row0 + t * 16 + r16, V - 1),
                                     (first_stage + place(j)) * GPS + h * 4 + quarter, n_groups);
    };
    // - s (16 + z) times the sums of x, of the sets before the one that begins at stage j
    auto add_sums = [&](int j, const float (&c)[SPS][RT]) {
#pragma unroll
        for (int h = 0; h < SPS; ++h) {
            const int slot = (SPS == 2 ? (j + 1) % 2 * 2 : (j / SET + 1) % 2) + h;
            float x[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) x[n] = s_sum[slot][kw][quarter][tile_of(n) * 16 + r16];
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    out[t][n] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[n], c[h][t], out[t][n], 0, 0, 0);
        }
    };

    // block h of a stage; g0: its first group's place in its set, slot: the set's sums
    auto block = [&](const uint8_t* buf, int slot, auto hc, auto gc) {
        constexpr int h = decltype(hc)::value, g0 = decltype(gc)::value;
        const uint32_t xs = kw * NT * XT + h * 4096 + lq_lane_offset<GROUP, BPS>(lane);
        const uint32_t ws = XB + wave * RT * WT_ + (lq_unit<BPS>(r16, quarter) ^ (h << 6));
        u32x4 w[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) w[t] = lq_at(buf + ws + t * WT_);
#pragma unroll
        for (int t = 0; t < RT; ++t) w[t] = lq_regroup<GROUP>(w[t]);
        const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
        floatx4 acc[RT][NT], sum = zero;
        // x of the next MFMA step is read while this one's is multiplied
        bf16x8 now[NT], then[NT];
        auto read_x = [&](int i, bf16x8 (&x)[NT]) {
            const uint8_t* at = buf + (xs ^ lq_step_xor<GROUP, BPS>(i)) + lq_step_offset<GROUP, BPS>(i);
#pragma unroll
            for (int n = 0; n < NT; ++n) x[n] = __builtin_bit_cast(bf16x8, lq_at(at + tile_of(n) * XT));
        };
        read_x(0, then);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int n = 0; n < NT; ++n) now[n] = then[n];
            if (i < 3) read_x(i + 1, then);
            __builtin_amdgcn_sched_barrier(0);
            const bool first = i % PER == 0;
            sum = lq_mfma(ones, now[0], first ? zero : sum);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const bf16x8 wv = widen(w[t][i]);
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[t][n] = lq_mfma(now[n], wv, first ? zero : acc[t][n]);
            }
            if (i % PER == PER - 1) {
                const int g = g0 + i / PER;
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const float scale = s_scale[wave][h % SPS][g][t * 16 + r16];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            out[t][n][q] = __builtin_fmaf(scale, acc[t][n][q], out[t][n][q]);
                }
                // every row of the product with ones is the sum of batch row r16
                if (rw < NT && quarter == 0) s_sum[slot][kw][g][tile_of(0) * 16 + r16] = sum[0];
            }
        }
    };

    load_scales(0);
    copy(b0, 0);
    constexpr int U = SET > 2 ? SET : 2;  // a multiple of the two stages and of a set
    for (int j0 = 0; j0 < stages; j0 += U) {
        auto stage = [&](auto uc) {
            constexpr int u = decltype(uc)::value;
            const int j = j0 + u;
            if (j >= stages) return;
            // this stage has landed for every wave, and the one before has been read
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(LQ_WAIT);
            // the builtins say nothing about memory: no access may cross them
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            uint8_t* const bufs[2] = {b0, b1};
            if (u % SET == 0) {
#pragma unroll
                for (int h = 0; h < SPS; ++h)
#pragma unroll
                    for (int t = 0; t < RT; ++t) {
                        c_before[h][t] = c_now[h][t];
                        const float scale = lq_scale(next[h][t].s, f16);
                        c_now[h][t] = -scale * (16.f + (float)next[h][t].z);
                        s_scale[wave][h][quarter][t * 16 + r16] = scale;
                    }
                if (j + SET < stages) load_scales(j + SET);
            }
            if (j + 1 < stages) copy(bufs[(u + 1) % 2], j + 1);
            const int slot = SPS == 2 ? j % 2 * 2 : j / SET % 2;
            auto one = [&](auto hc) {
                constexpr int h = decltype(hc)::value;
                constexpr int g = (u % SET * GPS + h * GPB) % 4;  // place of its first group
                block(bufs[u % 2], slot + h % SPS, hc, std::integral_constant<int, g>{});
            };
            lq_each(one, std::make_integer_sequence<int, BPS>{});
            if (u % SET == 0 && j > 0) add_sums(j, c_before);
        };
        lq_each(stage, std::make_integer_sequence<int, U>{});
    }
    __syncthreads();
    add_sums((stages + SET - 1) / SET * SET, c_now);

    if constexpr (KW > 1) {  // the ranges of K, added in order
        static_assert((KW - 1) * RW * RT * NT * 1024 <= XB + WB, "the ranges' sums fit a stage");
        floatx4* s_red = reinterpret_cast<floatx4*>(b0);
        __syncthreads();
        if (kw > 0) {
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    s_red[((((kw - 1) * RW + rw) * RT + t) * NT + n) * WAVE + lane] = out[t][n];
        }
        __syncthreads();
        if (kw == 0) {
#pragma unroll
            for (int k = 1; k < KW; ++k)
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        out[t][n] += s_red[((((k - 1) * RW + rw) * RT + t) * NT + n) * WAVE + lane];
        }
    }
    const bool holds = KW == 1 || kw == 0;  // the workgroup's sums
    if (part) {  // the parts of K, added in order by the workgroup that is last to leave its own
        __shared__ int s_last;
        constexpr int SUMS = RW * RT * NT * 2 * WAVE;  // pairs of sums per workgroup
        const int mine = rw * RT * NT * 2 * WAVE + lane;
        if (holds) {
            uint64_t* to = a.part + (int64_t)blockIdx.x * SUMS + mine;
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        __hip_atomic_store(to + ((t * NT + n) * 2 + h) * WAVE,
                                           lq_pair(out[t][n][2 * h], out[t][n][2 * h + 1]),
                                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (tid == 0) {
            int32_t* arrived = a.arrived + (row_block - a.whole_blocks) * QUANT_COUNTER;
            s_last = __hip_atomic_fetch_add(arrived, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                     a.split - 1;
            if (s_last) __hip_atomic_store(arrived, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        if (!s_last) return;
        if (holds) {
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int n = 0; n < NT; ++n) out[t][n] = floatx4{0.f, 0.f, 0.f, 0.f};
            const uint64_t* from = a.part + (int64_t)(blockIdx.x - blockIdx.x % a.split) * SUMS + mine;
            for (int p = 0; p < a.split; ++p, from += SUMS)
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint64_t v = __hip_atomic_load(from + ((t * NT + n) * 2 + h) * WAVE,
                                                                 __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                            out[t][n][2 * h] += __uint_as_float((uint32_t)v);
                            out[t][n][2 * h + 1] += __uint_as_float((uint32_t)(v >> 32));
                        }
        }
    }
    if (!holds) return;
    // a lane holds four batch rows of one vocabulary entry
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int v = row0 + t * 16 + r16;
        if (v >= V) continue;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int b = tile_of(n) * 16 + quarter * 4 + q;
                if (b >= a.B) continue;
                const int64_t at = (int64_t)b * a.out_stride + v;
                if (a.out_bf16) static_cast<__bf16*>(a.out)[at] = (__bf16)out[t][n][q];  // rounded once
                else static_cast<float*>(a.out)[at] = out[t][n][q];
            }
    }
}

// Where row blocks are left over beyond a multiple of the CUs, other CUs would wait for
// those that have one more. These blocks are cut along K, in as many parts as there
// are CUs for them. B = 8, V = 3000, K = 8192: 21.1 -> 10.3 us, B = 64: 35.8 -> 15.8;
// B = 64, V = 70000, K = 8192, groups of 128: 190 -> 128, B = 20, V = 67000, K = 4096:
// 61 -> 50, B = 13, V = 50257, K = 4160: 39 -> 37. Where not all whole blocks are
// resident, late ones fill the gaps by themselves (B = 24, V = 100000: 73, cut 74.5),
// unless there is one a CU. With more parts than CUs their sums cost more than they
// gain (B = 64, V = 11000, K = 4096, 516 parts: 31, uncut 22).
static QuantSplit quant_split(int blocks, int resident, int sets) {
    QuantSplit s = {blocks, 0, 1, 0};
    const int over = blocks % QUANT_CUS;
    const int rounds = blocks / QUANT_CUS;
    if (over == 0 || (resident > 1 && rounds > resident)) return s;
    for (int f = 2; f <= QUANT_SPLIT && f <= sets && f * over <= QUANT_CUS; ++f) {
        const int per = (sets + f - 1) / f;
        if ((sets + per - 1) / per == f)  // else a part would be empty
            s = {blocks - over, over, f, per};
    }
    return s;
}

// A choice of tiles: what its launch needs and what its parts' sums take.
template <int GROUP, int NT, int RT, int KW, int WAVES, int BPS>
struct QuantTiles {
    static constexpr int rows = WAVES / KW * RT * 16;
    static constexpr int part_bytes = rows * NT * 16 * 4;
    static constexpr int GPS = LQ_KB / GROUP * BPS, SET = (GPS < 4 ? 4 / GPS : 1) * KW;
    static constexpr int LDS = 2 * BPS * (KW * NT * 4096 + WAVES * RT * 1024);
    static QuantSplit split(int V, int K) {
        const int all = (K + LQ_KB * BPS - 1) / (LQ_KB * BPS);
        return quant_split((V + rows - 1) / rows, 160 * 1024 / LDS, (all + SET - 1) / SET);
    }
    static void launch(const QuantArgs& a, hipStream_t st, const LaunchEvents& le) {
        QuantArgs b = a;
        const QuantSplit s = split(a.V, a.K);
        b.whole_blocks = s.whole_blocks;
        b.split_blocks = s.split_blocks;
        b.split = s.split;
        b.split_stages = s.sets * SET;
        launch_k(le, 0, k_lmhead_quant<GROUP, NT, RT, KW, WAVES, BPS>,
                 dim3(b.whole_blocks + b.split_blocks * b.split), dim3(WAVES * WAVE), st, b);
    }
};

// ---------------------------------------------------------------------------
// one batch row: no matrix cores
//
// For a single token the weight stream is all there is: a wave reads QR_R whole
// rows side by side, 2048 k of each at a time, 32 consecutive k a lane, and dots
// its widened weights with x (v_dot2_f32_bf16: exact products, binary32 sums). x
// lies in LDS, swizzled as above, with the sum over every 32 k; waves meet at no
// barrier after it is there. A lane's 32 k are of one group, so scale and zero
// point are one value, and only the finished rows cross lanes.

constexpr int QR_NT = 256;
constexpr int QR_R = 4;        // rows per wave
constexpr int QR_K = WAVE * 32;
constexpr int QR_ROWS = QR_NT / WAVE * QR_R;
constexpr int QR_MOST_K = 24576;  // x and its sums stay within 64 KB of LDS

template <int GROUP>
__global__ __launch_bounds__(QR_NT) void k_quant_rows(QuantArgs a) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    extern __shared__ __attribute__((aligned(16))) uint8_t s_x[];  // [K] bfloat16, then sums
    const int K = a.K, V = a.V;
    float* s_sum = reinterpret_cast<float*>(s_x + (size_t)K * 2);  // [K / 32]
    const int tid = threadIdx.x;
    const int lane = tid & (WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int n_groups = (K + GROUP - 1) / GROUP;
    const int zero_pitch = (n_groups + 1) / 2;
    const int chunks = (K + QR_K - 1) / QR_K;
    const bool f16 = a.scale_f16 != 0;
    const int first = (blockIdx.x * (QR_NT / WAVE) + wave) * QR_R;

    struct Load {
        u32x4 w;
        uint32_t s, z;
    };
    auto load = [&](int c, Load (&l)[QR_R]) {
        const int k = c * QR_K + lane * 32;
        const bool on = k < K;
        const int g = k / GROUP;
#pragma unroll
        for (int r = 0; r < QR_R; ++r) {
            const int64_t row = min(first + r, V - 1);
            l[r].w = u32x4{0u, 0u, 0u, 0u};
            l[r].s = 0u;
            l[r].z = 0x88u;  // both nibbles: which one is chosen where it is used
            if (on) {
                l[r].w = __builtin_nontemporal_load(
                    reinterpret_cast<const u32x4*>(a.qweight + row * (K / 2) + (k >> 1)));
                l[r].s = a.scales[row * n_groups + g];
                if (a.zeros) l[r].z = a.zeros[row * zero_pitch + (g >> 1)];
            }
        }
    };
    Load now[QR_R], then[QR_R];
    load(0, then);

    // x: 16-byte unit u to the 64 bytes of the lane that uses it
    for (int u = tid; u < K / 8; u += QR_NT) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(a.hidden + u * 8);
        *reinterpret_cast<u32x4*>(s_x + (u >> 2) * 64 + (((u & 3) ^ (u >> 4 & 3)) << 4)) = v;
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            s += __uint_as_float(v[q] << 16) + __uint_as_float(v[q] & 0xFFFF0000u);
        // K is a multiple of 64: the four units of 32 k lie in four lanes of one quad
        s += __uint_as_float(dpp_mov<DPP_QUAD_X1>(__float_as_uint(s)));
        s += __uint_as_float(dpp_mov<DPP_QUAD_X2>(__float_as_uint(s)));
        if ((u & 3) == 0) s_sum[u >> 2] = s;
    }
    __syncthreads();

    const LqWiden widen;
    float acc[QR_R];
#pragma unroll
    for (int r = 0; r < QR_R; ++r) acc[r] = 0.f;
    for (int c = 0; c < chunks; ++c) {
#pragma unroll
        for (int r = 0; r < QR_R; ++r) now[r] = then[r];
        const int k = c * QR_K + lane * 32;
        if (c + 1 < chunks) load(c + 1, then);
        const int at = k < K ? k : 0;  // lanes behind K have scale 0
        u32x4 x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = lq_at(s_x + at * 2 + ((u ^ (at >> 7 & 3)) << 4));
        const float sum = s_sum[at >> 5];
        const int nibble = (k / GROUP & 1) * 4;
#pragma unroll
        for (int r = 0; r < QR_R; ++r) {
            float dot = 0.f;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const u32x4 w = __builtin_bit_cast(u32x4, widen(now[r].w[u]));
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t wq = w[q], xq = x[u][q];
                    dot = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, wq),
                                                          __builtin_bit_cast(bf16x2, xq), dot, false);
                }
            }
            const float z = -16.f - (float)(now[r].z >> nibble & 15u);
            acc[r] = __builtin_fmaf(lq_scale(now[r].s, f16), __builtin_fmaf(z, sum, dot), acc[r]);
        }
    }
    float mine = 0.f;  // lane r: row r
#pragma unroll
    for (int r = 0; r < QR_R; ++r) {
        const float sum = wave_allreduce32(acc[r], [](float x, float y) { return x + y; });
        if (lane == r) mine = sum;
    }
    const int v = first + lane;
    if (lane < QR_R && v < V) {
        if (a.out_bf16) static_cast<__bf16*>(a.out)[v] = (__bf16)mine;  // rounded once
        else static_cast<float*>(a.out)[v] = mine;
    }
}

template <int GROUP>
static void launch_rows_t(const QuantArgs& a, hipStream_t st, const LaunchEvents& le) {
    const size_t lds = (size_t)a.K * 2 + (size_t)(a.K / 32) * 4;
    const dim3 grid((a.V + QR_ROWS - 1) / QR_ROWS);
    if (le.start(0))
        hipExtLaunchKernelGGL((k_quant_rows<GROUP>), grid, dim3(QR_NT), lds, st, le.start(0),
                              le.stop(0), 0, a);
    else
        hipLaunchKernelGGL((k_quant_rows<GROUP>), grid, dim3(QR_NT), lds, st, a);
}

// Calls f with the tiles of B rows. Fewer, larger workgroups share a stage of x and
// widen a weight for more batch rows; where they are few, smaller ones, with K in
// two ranges where those are few as well. The borders are sizes V alone. Over K =
// 2048, 4096 and 8192, 13 sizes V from 8000 to 128256 and 13, 24 and 64 rows, each
// choice timed (without zero points), the one made here was the fastest or within a tenth of it but at
//  - 24 rows, V = 40000 and 50257: up to 12 % behind two ranges or two row tiles;
//  - 64 rows, groups of 128, V = 72000 and 100000, K <= 4096: 17 to 22 % behind 128
//    rows a workgroup (with 256, 282 and 391 blocks leave CUs idle in the last round);
//  - 64 rows, V = 20000, K = 8192: 10 to 17 % behind two ranges or 256 rows;
//  - 64 rows, V = 40000, K = 2048: 11 % behind 64 rows a workgroup.
template <int GROUP, class F>
static void quant_choose(int B, int V, F f) {
    if (B <= 16) {
        // K = 4096: V = 20000 14.0 us (one range: 17.9), V = 50257 31.0 (27.0)
        if (V <= 32768) f(QuantTiles<GROUP, 1, 1, 2, 8, 2>{});
        else f(QuantTiles<GROUP, 1, 1, 1, 4, 2>{});
    } else if (B <= 32) {
        // K = 4096, two ranges, one, two row tiles a wave: V = 32000 21.9 us, 26.1, 28.1;
        // V = 40000 28.5, 29.5, 30.5; V = 56000 36.7, 42.1, 36.4; V = 128256 86.2, 85.7, 74.0
        if (V <= 32768) f(QuantTiles<GROUP, 2, 1, 2, 8, 1>{});
        else if (V <= 53248) f(QuantTiles<GROUP, 2, 1, 1, 4, 2>{});
        else f(QuantTiles<GROUP, 2, 2, 1, 4, 2>{});
    } else if (V <= 16384) {
        // groups of 128: V = 16000, K = 4096: 21.1 us (one range: 27.5), V = 24000: 33.9 (32.3)
        f(QuantTiles<GROUP, 4, 1, 2, 8, 1>{});
    } else if (V <= 32768 || GROUP == 32) {
        // groups of 128, K = 4096: V = 32000 35.0 us (two row tiles a wave: 38.2), V = 50257
        // 51.5 (48.2). Groups of 32 end with every MFMA: with two row tiles their
        // accumulators do not fit.
        f(QuantTiles<GROUP, 4, 1, 1, 4, 1>{});
    } else if constexpr (GROUP >= 64) {
        // K = 4096: groups of 128, 256 rows a workgroup by whole lines: V = 64000 53.5 us (128
        // rows: 50.3), V = 128256 104.5 (107.9), V = 200000 176 (191); groups of 64 by half
        // lines, 128 rows: V = 128256 123 (64 rows: 150; 256 rows and whole lines were slower)
        if (GROUP == 64 || V <= 65536) f(QuantTiles<GROUP, 4, 2, 1, 4, 1>{});
        else if constexpr (GROUP == 128) f(QuantTiles<GROUP, 4, 2, 1, 8, 2>{});
    }
}

template <int GROUP>
static void launch_quant_g(const QuantArgs& a, hipStream_t st, const LaunchEvents& le) {
    // One row: whole rows by v_dot2, where at least four fifths of the lanes have k
    // to read: V = 128256, K = 4096, groups of 32: 59 us (matrix cores: 105), K = 8192,
    // groups of 128: 111 (127), V = 32000, K = 2048: 10.2 (14.1); K = 4160, of three
    // chunks the last nearly empty: 40 (36).
    const int chunks = (a.K + QR_K - 1) / QR_K;
    if (a.B == 1 && (int64_t)a.K * 5 >= (int64_t)chunks * QR_K * 4 && a.K <= QR_MOST_K)
        launch_rows_t<GROUP>(a, st, le);
    else
        quant_choose<GROUP>(a.B, a.V, [&](auto tiles) { tiles.launch(a, st, le); });
}

template <int GROUP>
static int64_t quant_part_bytes_g(int V, int K, int max_batch) {
    int64_t most = 0;
    for (const int B : {16, 32, 64}) {  // the last batch of each choice
        quant_choose<GROUP>(max_batch < B ? max_batch : B, V, [&](auto tiles) {
            const QuantSplit s = tiles.split(V, K);
            const int64_t n = (int64_t)s.split_blocks * s.split * tiles.part_bytes;
            if (n > most) most = n;
        });
    }
    return most;
}

int64_t quant_part_bytes(int V, int K, int max_batch) {
    const int64_t a = quant_part_bytes_g<32>(V, K, max_batch), b = quant_part_bytes_g<64>(V, K, max_batch);
    const int64_t c = quant_part_bytes_g<128>(V, K, max_batch);
    return a > b ? (a > c ? a : c) : (b > c ? b : c);
}

hipError_t launch_quant(const QuantArgs& a, hipStream_t st, const LaunchEvents& le) {
    if (a.group == 32) launch_quant_g<32>(a, st, le);
    else if (a.group == 64) launch_quant_g<64>(a, st, le);
    else launch_quant_g<128>(a, st, le);
    return hipGetLastError();
}

}  // namespace ss
