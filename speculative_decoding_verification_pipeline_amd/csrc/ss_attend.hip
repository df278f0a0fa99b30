// Attention over a cache held in 8 bits (ss_cache_attend).
//
// o = sum_j softmax_j(scale q k_j) v_j over the slots j that a token sees, where a slot's
// key and value are 8-bit floats q8 under a power of two 2^x for each block of slots and
// head. One pass over the slots with a running maximum and sum.
//
// A wave takes steps of 32 slots and 16 * MT rows, a row being a query head of a token:
// the query heads that share a head of the cache and the step's tokens stand in one
// product. It forms S^T = K Q^T and O^T = V^T P^T with v_mfma_f32_16x16x32, keys and
// values as the A operands, straight from the cache's pages in registers:
//  * S^T: a lane holds slot (lane & 15) of a tile of 16 and, with each load of 16 bytes,
//    two runs of 8 of its dimensions; which dimension a lane group's k index names is free
//    as long as Q is loaded by the same rule, so loads are 16 bytes and neighbouring lane
//    groups read neighbouring pieces.
//  * The result, four slots of one row a lane, is the B operand of the second product as it
//    is: its k index g * 8 + j names slot g * 4 + j of the first tile for j < 4 and
//    g * 4 + j - 4 of the second beyond. Nothing crosses lanes.
//  * V^T: a lane holds DP / 16 neighbouring dimensions of the 8 slots of its group, read as
//    they lie, and pairs slots with byte permutes after widening. The product's rows are
//    then dimensions (row * DP / 16 + tile), and a lane ends with 4 * DP / 16 neighbouring
//    entries of one row of the output.
// An 8-bit float is exact in float16 and bfloat16, so the scales never meet the operands: a
// key's is a factor on S, and a value's joins the weight's exponent,
//     p_j = 2^(s_j + x_j - R),   o = sum_j p_j q8_j / sum_j p_j 2^(-x_j),
// R the running reference of a row. Weights are rounded to float16 (11 bits, where bfloat16
// has 8): a reference is set to 2^8 below the largest exponent and kept until one passes
// 2^15, so a weight keeps its bits down to 2^-22 of the largest.
#include <limits.h>

#include "ss_device.h"
#include "ss_internal.h"

namespace ss {

constexpr int AT_STEP = 32;                   // slots of a wave's step
constexpr int AT_CUS = 256;
constexpr float AT_NONE = -3.0e38f;           // reference of a row that has seen nothing
constexpr float AT_SET = 8.0f;                // a reference is set so far below the largest exponent
constexpr float AT_MOST = 32768.0f;           // and moves when a lane's four weights sum up to more

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 h16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 h16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 b16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 b16x8 __attribute__((ext_vector_type(8)));
typedef const __attribute__((address_space(4))) int32_t* const_i32;  // what no kernel writes meanwhile

template <class T, class F>
__device__ __forceinline__ T as(F f) {
    static_assert(sizeof(T) == sizeof(F), "bits");
    return __builtin_bit_cast(T, f);
}

template <int N>
struct Words;
template <>
struct Words<1> { typedef uint32_t type; };
template <>
struct Words<2> { typedef u32x2 type; };
template <>
struct Words<4> { typedef u32x4 type; };

// Two 8-bit floats (the low or high pair of a word) widened exactly.
template <bool F16>
__device__ __forceinline__ uint32_t widen(uint32_t w, bool high) {
    if constexpr (F16)
        return high ? as<uint32_t>(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true))
                    : as<uint32_t>(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
    else
        return high ? as<uint32_t>(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true))
                    : as<uint32_t>(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
}

template <bool F16>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(as<h16x8>(a), as<h16x8>(b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as<b16x8>(a), as<b16x8>(b), c, 0, 0, 0);
}

// Rows of one request as this launch sees them.
struct AttendRow {
    int base;   // committed slots
    int count;  // tokens of the step
    int end;    // slots that any of them may see
};

__device__ __forceinline__ AttendRow attend_row(const Kv8Attend& a, int b) {
    AttendRow r;
    const int cap = a.g.max_blocks * a.g.page_size;
    r.base = ((const_i32)a.s.base)[b];
    r.count = a.s.counts ? min(max(((const_i32)a.s.counts)[b], 0), a.s.N) : a.s.N;
    if (r.base < 0 || r.base > cap || (a.s.reserved && ((const_i32)a.s.reserved)[b] == 0)) {
        r.base = 0;
        r.count = 0;
    }
    r.end = r.count ? (int)min((int64_t)r.base + r.count, (int64_t)cap) : 0;
    return r;
}

// A byte that all lanes read, as a scalar load of the word it lies in: a vector load would be
// waited for with the loads before it.
__device__ __forceinline__ uint32_t scale_byte(const uint8_t* at) {
    const uint64_t p = reinterpret_cast<uint64_t>(at);
    return (uint32_t)*(const_i32)(p & ~3ull) >> ((uint32_t)p % 4 * 8) & 0xffu;
}

// A scale byte, held to what ss_cache_write leaves: whatever a block holds that nothing was
// written to, its factors are finite and not 0, and masked slots stay masked.
__device__ __forceinline__ uint32_t clamp_scale(uint32_t x) {
    return min(max(x, (uint32_t)(127 + KV8_XMIN)), (uint32_t)(127 + KV8_XMAX));
}

// The keys or the values of 32 slots as they lie in the pages, and their two tiles' scales.
template <int DP>
struct AttendKeys {
    u32x4 k[2][DP / 64];
    uint32_t s[2];
    bool ok[2];  // whether a tile lies on a page
};
template <int DP>
struct AttendValues {
    typename Words<DP / 64>::type v[8];
    uint32_t s[2];
};

// Where a wave stands in its row: a step of two tiles after the other. The pages of the next
// step are looked up a step ahead.
struct AttendCursor {
    const_i32 table;
    int block, inner;  // table entry of the tile after the pages below, and its place there
    int tiles;         // tiles of a page
    int left;          // tiles from there up to the row's last
    int page[2], at[2];
};

__device__ __forceinline__ void attend_look(AttendCursor& c) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        c.page[t] = -1;
        c.at[t] = c.inner;
        if (c.left > 0) c.page[t] = c.table[c.block];
        --c.left;
        const bool over = ++c.inner == c.tiles;
        c.block += over ? 1 : 0;
        c.inner = over ? 0 : c.inner;
    }
}

// Two tiles' places in the planes and in their scales. One on no page is read where page 0
// lies, and then put out.
struct AttendPlace {
    int64_t at[2], scale[2];
    bool ok[2];
};

__device__ __forceinline__ AttendPlace attend_next(const Kv8Attend& a, AttendCursor& c, int h) {
    AttendPlace p;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        p.ok[t] = (unsigned)c.page[t] < (unsigned)a.g.num_pages;
        const int64_t page = p.ok[t] ? c.page[t] : 0;
        const int off = c.at[t] * 16;
        p.at[t] = page * a.g.page + off * a.g.slot + h * a.g.head;
        p.scale[t] = page * a.g.sc_page + (off >> a.g.block_bits) * a.g.sc_block + h * a.g.sc_head;
    }
    attend_look(c);
    return p;
}

// k_at: where this lane's pieces of 64 dimensions lie, those behind the head's last at the
// first: they meet zeros of Q.
template <int DP>
__device__ __forceinline__ void load_keys(const Kv8Attend& a, const AttendPlace& p,
                                          const uint32_t (&k_at)[DP / 64], AttendKeys<DP>& x) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const char* from = a.k.data + p.at[t];
#pragma unroll
        for (int c = 0; c < DP / 64; ++c) x.k[t][c] = *reinterpret_cast<const u32x4*>(from + k_at[c]);
        x.s[t] = scale_byte(a.k.scales + p.scale[t]);
        x.ok[t] = p.ok[t];
    }
}

template <int DP>
__device__ __forceinline__ void load_values(const Kv8Attend& a, const AttendPlace& p,
                                            const uint32_t (&v_at)[4], AttendValues<DP>& x) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const char* from = a.v.data + p.at[t];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x.v[t * 4 + j] = *reinterpret_cast<const typename Words<DP / 64>::type*>(from + v_at[j]);
        x.s[t] = scale_byte(a.v.scales + p.scale[t]);
    }
}

// Tiles on no page are zeros; their weights become 2^-inf.
template <int DP>
__device__ __forceinline__ void put_out(AttendKeys<DP>& k, AttendValues<DP>& v) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        if (k.ok[t]) continue;
#pragma unroll
        for (int c = 0; c < DP / 64; ++c) k.k[t][c] = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j) v.v[t * 4 + j] = {};
    }
}

// Scores of tiles on no page are 0, whatever the queries hold: zeros times what is not finite
// are NaN. Without a branch: behind one the compiler has read a product's accumulator in the
// next instruction, where it must wait for seven.
template <int MT>
__device__ __forceinline__ void put_out_scores(const bool (&ok)[2], f32x4 (&s)[2][MT]) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const uint32_t keep = ok[t] ? ~0u : 0u;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[t][m][i] = as<float>(as<uint32_t>((float)s[t][m][i]) & keep);
    }
}

// What a wave holds of its rows.
template <int DP, int MT>
struct AttendState {
    u32x4 q[MT][DP / 32];
    f32x4 o[MT][DP / 16];
    float l[MT];               // this lane's share of the sum
    float ref[MT];             // the same in the four lanes of a row
};

// The slots that a row sees of a lane's four from `at` on (behind the committed ones), a bit
// each: of a tree's nodes those in `up`, else those up to token n; `end` bounds all.
__device__ __forceinline__ uint32_t attend_sees(bool tree, unsigned long long up, int n, int at, int end) {
    const int below = min(max(-at, 0), 4);  // committed slots, seen by all
    uint32_t own;
    if (tree) own = at >= 64 ? 0 : at >= 0 ? (uint32_t)(up >> at) : (uint32_t)up << below;
    else own = (1u << min(max(n + 1 - at, 0), 4)) - 1;
    return (own | ((1u << below) - 1)) & ((1u << min(max(end - at, 0), 4)) - 1);
}

template <int DP>
__device__ __forceinline__ uint32_t word_of(const typename Words<DP / 64>::type& v, int w) {
    if constexpr (DP == 64) return v;
    else return v[w];
}

template <int DP>
__device__ __forceinline__ void set_word(typename Words<DP / 64>::type& v, int w, uint32_t to) {
    if constexpr (DP == 64) v = to;
    else v[w] = to;
}

// The word if the bit is set, else the other, without a condition a lane (masks of many of
// them took the scalar registers).
__device__ __forceinline__ uint32_t keep_if(uint32_t bits, int bit, uint32_t w, uint32_t other) {
    const uint32_t m = (uint32_t)((int32_t)(bits << (31 - bit)) >> 31);
    return (w & m) | (other & ~m);
}

// Puts out the scores of a step's slots that a row does not see. rel: this lane's first slot
// behind the committed ones; ok: tiles on a page; vis: those seen, bit 4 t + i slot i of tile t.
template <int MT>
__device__ __forceinline__ void attend_mask(const Kv8Attend& a, unsigned long long above, int first, int rows,
                                            int rel, int end, const bool (&ok)[2], f32x4 (&s)[2][MT],
                                            uint32_t (&vis)[MT]) {
    const int col = threadIdx.x & 15;
    const uint32_t on = (ok[0] ? 0xfu : 0u) | (ok[1] ? 0xf0u : 0u);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int n = (first + min(m * 16 + col, rows - 1)) / a.group;
        const unsigned long long up = (unsigned long long)(uint32_t)__shfl((int)(above >> 32), n & 63) << 32 |
                                      (uint32_t)__shfl((int)above, n & 63);
        vis[m] = (attend_sees(a.s.parents, up, n, rel, end) |
                  attend_sees(a.s.parents, up, n, rel + 16, end) << 4) & on;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                s[t][m][i] = as<float>(keep_if(vis[m], 4 * t + i, as<uint32_t>((float)s[t][m][i]), 0xff800000u));
    }
}

// S^T of one step.
template <int DP, int MT, bool F16>
__device__ __forceinline__ void attend_scores(const AttendKeys<DP>& x, const AttendState<DP, MT>& w,
                                              f32x4 (&s)[2][MT]) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int m = 0; m < MT; ++m) s[t][m] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int st = 0; st < DP / 32; ++st) {
            const u32x4 b = x.k[t][st / 2];
            const uint32_t w0 = b[st % 2 * 2], w1 = b[st % 2 * 2 + 1];
            const u32x4 k = {widen<F16>(w0, false), widen<F16>(w0, true), widen<F16>(w1, false),
                             widen<F16>(w1, true)};
#pragma unroll
            for (int m = 0; m < MT; ++m) s[t][m] = mfma<F16>(k, w.q[m][st], s[t][m]);
        }
    }
}

// What two tiles' scales come to: the factor on S with the softmax's scale, the exponent that
// a value's scale adds to its weight, and the factor that takes it off again.
struct AttendScales {
    float fk[2], xv[2], inv[2];
};

__device__ __forceinline__ AttendScales scales_of(const Kv8Attend& a, const uint32_t (&ks)[2],
                                                  const uint32_t (&vs)[2], const bool (&ok)[2]) {
    AttendScales x;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const uint32_t v = clamp_scale(vs[t]);
        x.fk[t] = as<float>(clamp_scale(ks[t]) << 23) * a.scale_log2;
        x.xv[t] = ok[t] ? (float)((int)v - 127) : -INFINITY;
        x.inv[t] = as<float>((254u - v) << 23);
    }
    return x;
}

// Weights of two tiles under the rows' references. A lane's sums, which the rows need anyway,
// tell whether a weight has passed 2^15; a row's reference then moves to its largest exponent
// less 8, and the weights are formed again. (Looking for the largest exponent at every step
// took a third of the vector instructions.)
template <int DP, int MT>
__device__ __forceinline__ void attend_weights(const AttendScales& x, const f32x4 (&s)[2][MT],
                                               AttendState<DP, MT>& w, u32x4 (&p)[MT]) {
    float sum[2][MT];
    auto form = [&] {
        float most = 0.0f;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const float c = x.xv[t] - w.ref[m];
                float e[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][m][i], x.fk[t], c));
                sum[t][m] = (e[0] + e[1]) + (e[2] + e[3]);
                most = fmaxf(most, sum[t][m]);
                p[m][2 * t] = as<uint32_t>(__builtin_convertvector((f32x2{e[0], e[1]}), h16x2));
                p[m][2 * t + 1] = as<uint32_t>(__builtin_convertvector((f32x2{e[2], e[3]}), h16x2));
            }
        }
        return most;
    };
    if (__any(form() > AT_MOST)) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float top = -INFINITY;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const float most = fmaxf(fmaxf(s[t][m][0], s[t][m][1]), fmaxf(s[t][m][2], s[t][m][3]));
                top = fmaxf(top, __builtin_fmaf(most, x.fk[t], x.xv[t]));
            }
            top = fmaxf(top, xor_lane_f<16>(top));
            top = fmaxf(top, xor_lane_f<32>(top)) - AT_SET;
            // rows below their reference keep it, bit by bit
            const float to = fmaxf(w.ref[m], top);
            const float f = __builtin_amdgcn_exp2f(w.ref[m] - to);
            w.ref[m] = to;
            w.l[m] *= f;
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) w.o[m][d] *= f;
        }
        form();
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < 2; ++t) w.l[m] = __builtin_fmaf(sum[t][m], x.inv[t], w.l[m]);
}

// A NaN among the values of one dimension reaches the rows that see it and no others: it is
// counted where it is seen, and taken out of the product. v: eight slots of a lane's, widened;
// vis: those that a row sees, bit by bit; o: the rows' sums of this dimension tile.
template <int MT>
__device__ __forceinline__ u32x4 take_nans(u32x4 v, const uint32_t (&vis)[MT], f32x4* (&o)[MT]) {
    u32x4 nan;
    uint32_t any = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        nan[j] = ((v[j] & 0x7fff7fffu) + 0x03ff03ffu) & 0x80008000u;
        any |= nan[j];
    }
    if (__any(any != 0)) {
        u32x4 hot;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            hot[j] = (nan[j] >> 15) * 0x3c00u;
            v[j] &= ~((nan[j] >> 15) * 0xffffu);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            u32x4 sees;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                sees[j] = (vis[m] >> (2 * j) & 1) * 0x3c00u | (vis[m] >> (2 * j + 1) & 1) * 0x3c000000u;
            const f32x4 n = mfma<true>(hot, sees, f32x4{0, 0, 0, 0});
#pragma unroll
            for (int i = 0; i < 4; ++i)  // n is 0 or at least 1
                (*o[m])[i] += n[i] * as<float>(as<uint32_t>((float)n[i]) ? 0x7fc00000u : 0u);
        }
    }
    return v;
}

// O^T of one step.
template <int DP, int MT, bool MASK>
__device__ __forceinline__ void attend_values(const AttendValues<DP>& x, const u32x4 (&p)[MT],
                                              const uint32_t (&vis)[MT], AttendState<DP, MT>& w) {
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) {
        uint32_t lo[8], hi[8];  // dimensions 0 and 1, 2 and 3 of the word
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            lo[j] = widen<true>(word_of<DP>(x.v[j], c), false);
            hi[j] = widen<true>(word_of<DP>(x.v[j], c), true);
        }
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            u32x4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t u0 = d < 2 ? lo[2 * j] : hi[2 * j], u1 = d < 2 ? lo[2 * j + 1] : hi[2 * j + 1];
                v[j] = __builtin_amdgcn_perm(u1, u0, d % 2 ? 0x07060302u : 0x05040100u);
            }
            if constexpr (MASK) {
                f32x4* o[MT];
#pragma unroll
                for (int m = 0; m < MT; ++m) o[m] = &w.o[m][c * 4 + d];
                v = take_nans<MT>(v, vis, o);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) w.o[m][c * 4 + d] = mfma<true>(v, p[m], w.o[m][c * 4 + d]);
        }
    }
}

// Which work a workgroup takes. All requests' slots that a head of the cache and a block of rows
// see, in units of UNIT, are one line, and a.shares workgroups take equal shares of it: the end of
// one request's slots, whole requests, the start of the next one's. So all are done at the same
// time, however uneven the contexts, and as many requests are cut as there are shares (64 requests
// of 4000 slots on average: 115 us, each request cut into workgroups of its own 147). With
// a.shares = 0 there are requests enough, and each is a workgroup's.
//
// Neighbouring workgroups, which run on different XCDs, take different heads of one share: they
// read the same pages at about the same time, and with eight heads an XCD's cache holds the
// pages of one. Later blocks of rows, which see more, come first.
struct AttendPiece {
    int h, first;         // head of the cache, first row
    int line, p;          // of heads and blocks of rows, and the share of it
    uint32_t share;       // its units
    uint32_t at, end;     // those of the line that it takes, from the present request on
    int b;                // the request
    uint32_t before, of;  // units of the requests before it, and its own
    int from, to;         // units of it that this share takes
    int c, n;             // the c-th of the n shares that it lies in
};

__device__ __forceinline__ int attend_see(const Kv8Attend& a, const AttendRow& row, int last) {
    if (a.s.parents || !row.count) return row.end;
    return (int)min((int64_t)row.end, (int64_t)row.base + last + 1);
}

// Units of UNIT slots that rows up to token `last` of a request see; one where they see none.
template <int UNIT>
__device__ __forceinline__ uint32_t attend_units(const Kv8Attend& a, int b, int last) {
    return max(((uint32_t)attend_see(a, attend_row(a, b), last) + UNIT - 1) / UNIT, 1u);
}

__device__ __forceinline__ void attend_part(AttendPiece& x) {
    x.from = (int)(x.at - x.before);
    x.to = (int)min(x.end - x.before, x.of);
    const uint32_t first = x.before / x.share;
    x.n = (int)((x.before + x.of - 1) / x.share - first) + 1;
    x.c = x.p - (int)first;
}

template <int ROWS>
__device__ __forceinline__ int attend_last(const Kv8Attend& a, int first) {
    return (min(a.s.N * a.group, first + ROWS) - 1) / a.group;
}

// False: nothing is left for this workgroup.
template <int UNIT, int ROWS>
__device__ __forceinline__ bool attend_share(const Kv8Attend& a, AttendPiece& x) {
    const int lane = threadIdx.x & (WAVE - 1);
    const int lines = a.g.heads * a.blocks;
    x.p = blockIdx.x / lines;
    x.line = blockIdx.x - x.p * lines;
    const int block = x.line / a.g.heads;
    x.h = x.line - block * a.g.heads;
    x.first = (a.blocks - 1 - block) * ROWS;
    x.c = x.from = 0;
    x.n = 1;
    x.at = x.before = 0;
    if (a.shares == 0) {
        x.b = x.p;
        x.to = INT_MAX / UNIT;
        x.of = x.end = x.share = 1;
        return true;
    }
    const int last = attend_last<ROWS>(a, x.first);
    // 32 bits hold the units of all: the host has seen to it
    uint32_t total = 0;
    for (int b0 = 0; b0 < a.s.B; b0 += WAVE)
        if (b0 + lane < a.s.B) total += attend_units<UNIT>(a, b0 + lane, last);
    total = (uint32_t)__builtin_amdgcn_readfirstlane(wave_sum_i((int)total));
    x.share = (total + a.shares - 1) / a.shares;
    x.at = x.p * x.share;
    if (x.at >= total) return false;
    x.end = min(x.at + x.share, total);
    for (int b0 = 0; b0 < a.s.B; b0 += WAVE) {
        const uint32_t u = b0 + lane < a.s.B ? attend_units<UNIT>(a, b0 + lane, last) : 0;
        const uint32_t to = x.before + (uint32_t)wave_incl_scan_i((int)u);
        const unsigned long long m = __ballot(x.at < to);
        if (m) {
            const int l = __builtin_ctzll(m);
            x.b = __builtin_amdgcn_readfirstlane(b0 + l);
            x.of = (uint32_t)__builtin_amdgcn_readlane((int)u, l);
            x.before = (uint32_t)__builtin_amdgcn_readlane((int)to, l) - x.of;
            attend_part(x);
            return true;
        }
        x.before = (uint32_t)__builtin_amdgcn_readlane((int)to, WAVE - 1);
    }
    return false;
}

// On to the next request of the share; false: it ends.
template <int UNIT, int ROWS>
__device__ __forceinline__ bool attend_on(const Kv8Attend& a, AttendPiece& x) {
    x.at = x.before + x.of;
    if (x.at >= x.end || ++x.b >= a.s.B) return false;
    x.before = x.at;
    x.of = (uint32_t)__builtin_amdgcn_readfirstlane(
        (int)attend_units<UNIT>(a, x.b, attend_last<ROWS>(a, x.first)));
    attend_part(x);
    return true;
}

// Where a line's share p leaves the sums of the request that it ends with (which = 1), or of the
// one that began before it (0).
__device__ __forceinline__ int attend_left(const Kv8Attend& a, const AttendPiece& x, int p, int which) {
    return (x.line * a.shares + p) * 2 + which;
}

// Values that other workgroups, on other XCDs, wrote in this launch or will read in it.
__device__ __forceinline__ void put(float* p, float a, float b) {
    __hip_atomic_store(reinterpret_cast<unsigned long long*>(p), as<unsigned long long>(f32x2{a, b}),
                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ f32x2 get(const float* p) {
    return as<f32x2>(__hip_atomic_load(reinterpret_cast<const unsigned long long*>(p), __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT));
}

// Two floats as the output's type.
template <bool F16>
__device__ __forceinline__ uint32_t narrow(float a, float b) {
    const f32x2 v = {a, b};
    if constexpr (F16) return as<uint32_t>(__builtin_convertvector(v, h16x2));
    else return as<uint32_t>(__builtin_convertvector(v, b16x2));
}

// A row of a head of the cache (a query head of a token) in the output.
struct AttendOut {
    uint16_t* to;
    int64_t lse;
};

__device__ __forceinline__ AttendOut attend_out(const Kv8Attend& a, int b, int h, int r) {
    const int n = r / a.group, head = h * a.group + r - n * a.group;
    return {a.out.data + b * a.out.row + n * a.out.token + head * a.out.head,
            ((int64_t)b * a.s.N + n) * a.q_heads + head};
}

// The factor on a row's sums: 0 where it has seen nothing, or scores of -inf alone.
__device__ __forceinline__ float attend_factor(float l, bool live) { return live && l != 0.0f ? 1.0f / l : 0.0f; }

__device__ __forceinline__ float attend_lse(float ref, float l, bool live) {
    return live ? (ref + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

// Two entries of a row; what a row that is not live has summed up may be anything.
template <bool F16>
__device__ __forceinline__ void put_pair(uint16_t* to, float a, float b, float f, bool live) {
    *reinterpret_cast<uint32_t*>(to) = live ? narrow<F16>(a * f, b * f) : 0u;
}

// Floats that a piece of `rows` rows leaves: references and sums, then their outputs.
constexpr int attend_slot(int dp, int rows) { return rows * (dp + 2); }

// Counts a piece that has left its sums. The one that counts last of a row adds them all, in
// their order, eight rows a wave at a time, a lane two neighbouring entries of each 128: whole
// lines a load, four pieces on their way at once. Of few rows the pieces are dealt out to the
// waves, which meet in LDS.
template <int DP, int ROWS, bool F16>
__device__ __forceinline__ void add_pieces(const Kv8Attend& a, const AttendPiece& pc, int rows, float* s_mem,
                                           const int* s_live) {
    constexpr int WAVES = 4;
    constexpr int PAIRS = 8 * DP / 128;  // of a lane's, over eight rows
    constexpr int ONCE = PAIRS >= 16 ? 2 : 4;
    const int b = pc.b, n = pc.n, h = pc.h, first = pc.first;
    const int tid = threadIdx.x;
    const int lane = tid & (WAVE - 1);
    const int wave = tid / WAVE;
    __shared__ int s_last;
    // what it left has reached the agent's point of coherence before it counts
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid == 0) {
        // a share begins one request at most that others go on with: its counter is the share's
        int32_t* arrived = a.arrived + (int64_t)(pc.line * a.shares + pc.p - pc.c) * KV8_COUNTER;
        s_last = __hip_atomic_fetch_add(arrived, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == n - 1;
        if (s_last) __hip_atomic_store(arrived, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (!s_last) return;
    auto left = [&](int i) {  // what the i-th piece has left
        return a.part + (int64_t)attend_left(a, pc, pc.p - pc.c + i, i == 0) * attend_slot(DP, ROWS);
    };
    const int groups = (rows + 7) / 8;
    const int share = groups == 1 ? WAVES : groups == 2 ? WAVES / 2 : 1;  // waves of a group
    const int sub = wave % share;
    auto row_of = [&](int k) { return (k * WAVE + lane) * 2 / DP; };
    for (int r0 = wave / share * 8; r0 < groups * 8; r0 += WAVES / share * 8) {
        const int mine = min(r0 + lane % 8, rows - 1);  // whose sums this lane has; of a wave's last rows any
        float ref = AT_NONE, l = 0.0f;
        f32x2 o[PAIRS];
#pragma unroll
        for (int k = 0; k < PAIRS; ++k) o[k] = f32x2{0.0f, 0.0f};
        for (int c0 = sub; c0 < n; c0 += ONCE * share) {
            f32x2 s[ONCE], v[ONCE][PAIRS];
#pragma unroll
            for (int i = 0; i < ONCE; ++i) {
                const float* p = left(min(c0 + i * share, n - 1));
                s[i] = get(p + mine * 2);
#pragma unroll
                for (int k = 0; k < PAIRS; ++k) v[i][k] = get(p + 2 * ROWS + r0 * DP + (k * WAVE + lane) * 2);
            }
            float to = ref;
#pragma unroll
            for (int i = 0; i < ONCE; ++i) to = fmaxf(to, s[i][0]);
            const float f = __builtin_amdgcn_exp2f(ref - to);
            ref = to;
            l *= f;
#pragma unroll
            for (int k = 0; k < PAIRS; ++k) o[k] *= __shfl(f, row_of(k));
#pragma unroll
            for (int i = 0; i < ONCE; ++i) {
                // behind the last piece nothing is added
                const float g = c0 + i * share < n ? __builtin_amdgcn_exp2f(s[i][0] - ref) : 0.0f;
                l = __builtin_fmaf(s[i][1], g, l);
#pragma unroll
                for (int k = 0; k < PAIRS; ++k) {
                    const float gk = __shfl(g, row_of(k));
                    o[k][0] = __builtin_fmaf(v[i][k][0], gk, o[k][0]);
                    o[k][1] = __builtin_fmaf(v[i][k][1], gk, o[k][1]);
                }
            }
        }
        if (share > 1) {  // one round for all waves
            float* s_o = s_mem + wave * 8 * DP;
            float* s_s = s_mem + WAVES * 8 * DP;
#pragma unroll
            for (int k = 0; k < PAIRS; ++k) *reinterpret_cast<f32x2*>(s_o + (k * WAVE + lane) * 2) = o[k];
            if (lane < 8) {
                s_s[(wave * 8 + lane) * 2] = ref;
                s_s[(wave * 8 + lane) * 2 + 1] = l;
            }
            __syncthreads();
            if (sub) continue;
            float to = ref;
            for (int i = 1; i < share; ++i) to = fmaxf(to, s_s[((wave + i) * 8 + lane % 8) * 2]);
            const float f = __builtin_amdgcn_exp2f(ref - to);
            ref = to;
            l *= f;
#pragma unroll
            for (int k = 0; k < PAIRS; ++k) o[k] *= __shfl(f, row_of(k));
            for (int i = 1; i < share; ++i) {
                const float* other = s_s + ((wave + i) * 8 + lane % 8) * 2;
                const float g = __builtin_amdgcn_exp2f(other[0] - ref);
                l = __builtin_fmaf(other[1], g, l);
#pragma unroll
                for (int k = 0; k < PAIRS; ++k) {
                    const f32x2 v = *reinterpret_cast<const f32x2*>(s_o + i * 8 * DP + (k * WAVE + lane) * 2);
                    const float gk = __shfl(g, row_of(k));
                    o[k][0] = __builtin_fmaf(v[0], gk, o[k][0]);
                    o[k][1] = __builtin_fmaf(v[1], gk, o[k][1]);
                }
            }
        }
        const bool live = s_live[mine] != 0;
        const float f = attend_factor(l, live);
        if (a.lse && lane < 8 && r0 + lane < rows)
            a.lse[attend_out(a, b, h, first + r0 + lane).lse] = attend_lse(ref, l, live);
#pragma unroll
        for (int k = 0; k < PAIRS; ++k) {
            const int r = r0 + row_of(k), e = (k * WAVE + lane) * 2 % DP;
            const float fk = __shfl(f, row_of(k));
            const bool on = __shfl((int)live, row_of(k));
            if (r < rows && e < a.g.dim)
                put_pair<F16>(attend_out(a, b, h, first + r).to + e, o[k][0], o[k][1], fk, on);
        }
    }
}

// For a loop over requests: what does not change from one to the next (addresses, sizes, lanes'
// places) is formed again for each, as if it did. Kept instead, it took 40 vector registers and
// a hundred spilled scalar ones.
struct ArgsAgain {
    const __attribute__((address_space(4))) Kv8Attend* p;
    int tid;
    __device__ __forceinline__ ArgsAgain()
        : p((const __attribute__((address_space(4))) Kv8Attend*)__builtin_amdgcn_kernarg_segment_ptr()),
          tid(threadIdx.x) {}
    __device__ __forceinline__ const Kv8Attend& args() {
        asm volatile("" : "+s"(p));
        asm volatile("" : "+v"(tid));
        return *(const Kv8Attend*)p;
    }
    __device__ __forceinline__ int thread() const { return tid; }
};

// Few rows: the four waves take a share's slots each a run of them, and meet in LDS. Keys and
// values go to registers straight from the pages: they are read once, and a step's 8 KB a wave,
// half of them on their way at any time, are what a CU needs at one wave a SIMD.
// What bounds it: HBM. 64 single tokens over uneven contexts of 4000 slots on average, 8 heads of
// 128: 113 to 115 us, 4.6 TB/s; even ones 102 us, 5.2 TB/s; one token over 131072 slots 61 us, 4.4 TB/s
// with its start and the addition of 32 pieces. Where requests are few and short it is a chain of
// loads: 9.4 us for four of 900 slots.
template <int DP, int MT, bool F16>
__global__ __launch_bounds__(256, DP == 256 ? 1 : MT == 2 || DP == 128 ? 2 : 3) void k_attend(Kv8Attend args) {
    constexpr int WAVES = 4;
    constexpr int DT = DP / 16;
    constexpr int SLOT = attend_slot(DP, MT * 16);
    constexpr int UNIT = AT_STEP * WAVES;
    __shared__ float s_o[WAVES][16][DP + 4];
    __shared__ float s_ref[WAVES][MT * 16], s_l[WAVES][MT * 16];
    __shared__ int s_live[MT * 16];
    AttendPiece pc;
    if (!attend_share<UNIT, MT * 16>(args, pc)) return;
    ArgsAgain again;
    do {
        const Kv8Attend& a = again.args();
        const int lane = again.thread() & (WAVE - 1);
        const int tid = again.thread();
        const int wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
        const int g = lane >> 4, col = lane & 15;
        const int h = pc.h, first = pc.first;
        const int rows = min(a.s.N * a.group - first, MT * 16);
        const AttendRow row = attend_row(a, pc.b);

        AttendState<DP, MT> w;
        unsigned long long rooted = 0;  // nodes that hang below the root
        if (a.s.parents) rooted = __ballot(tree_node(a.s.parents + (int64_t)pc.b * a.s.N, a.s.N).above != 0);
        uint32_t k_on = 0;  // the pieces of 64 dimensions that reach into the head's
#pragma unroll
        for (int c = 0; c < DP / 64; ++c) k_on |= (c * 64 + g * 16 < a.g.dim ? 1u : 0u) << c;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int r = first + min(m * 16 + col, rows - 1);
            const int n = r / a.group;
            w.l[m] = 0.0f;
            w.ref[m] = AT_NONE;
            const bool live = n < row.count && (!a.s.parents || (rooted >> (n & 63) & 1));
            if (wave == 0 && g == 0) s_live[m * 16 + col] = live;
            const uint16_t* q = a.q.data + pc.b * a.q.row + n * a.q.token +
                                (h * a.group + r - n * a.group) * a.q.head + g * 16;
#pragma unroll
            for (int st = 0; st < DP / 32; ++st) {
                w.q[m][st] = u32x4{0, 0, 0, 0};
                if (k_on >> (st / 2) & 1)
                    w.q[m][st] = *reinterpret_cast<const u32x4*>(q + st / 2 * 64 + st % 2 * 8);
            }
#pragma unroll
            for (int d = 0; d < DT; ++d) w.o[m][d] = f32x4{0, 0, 0, 0};
        }

        // the slots of this piece, and of this wave of it, in steps
        const int see = attend_see(a, row, (first + rows - 1) / a.group);
        int full = min(row.base, row.end);  // slots before it all rows see
        if (!a.s.parents && row.count) full = (int)min((int64_t)row.end, (int64_t)row.base + first / a.group + 1);
        const int steps = (int)(((int64_t)see + AT_STEP - 1) / AT_STEP);
        const int s0 = (int)min((int64_t)pc.from * WAVES, (int64_t)steps);
        const int s1 = (int)min((int64_t)pc.to * WAVES, (int64_t)steps);
        const int per = (s1 - s0 + WAVES - 1) / WAVES;
        const int from = min(s0 + wave * per, s1), to = min(from + per, s1);
        const int plain = max(min(to, full / AT_STEP), from);  // steps before it need no mask
        if (from < to) {
            AttendCursor at;
            at.table = (const_i32)(a.s.t.tables + (int64_t)pc.b * a.s.t.stride);
            at.tiles = a.g.page_size / 16;
            at.block = from * 2 / at.tiles;
            at.inner = from * 2 - at.block * at.tiles;
            at.left = (row.end + 15) / 16 - from * 2;
            uint32_t k_at[DP / 64], v_at[4];
#pragma unroll
            for (int c = 0; c < DP / 64; ++c)
                k_at[c] = (uint32_t)col * (uint32_t)a.g.slot + (k_on >> c & 1 ? c * 64 + g * 16 : 0);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v_at[j] = (uint32_t)(g * 4 + j) * (uint32_t)a.g.slot + (col * DT < a.g.dim ? col * DT : 0);
            AttendKeys<DP> k;
            AttendValues<DP> v;
            f32x4 e[2][MT];
            u32x4 p[MT];
            const uint32_t none[MT] = {};
            attend_look(at);
            AttendPlace place = attend_next(a, at, h);
            load_keys<DP>(a, place, k_at, k);
            // keys of the next step are on their way while this one's weights and values are
            // worked on, values while its scores are (a step's values loaded a step ahead as well,
            // into registers of their own: 1 to 3 % slower)
            for (int s = from; s < plain; ++s) {
                load_values<DP>(a, place, v_at, v);
                if (!(k.ok[0] && k.ok[1])) put_out<DP>(k, v);
                attend_scores<DP, MT, F16>(k, w, e);
                put_out_scores<MT>(k.ok, e);
                const uint32_t ks[2] = {k.s[0], k.s[1]};
                const bool ok[2] = {k.ok[0], k.ok[1]};
                place = attend_next(a, at, h);  // behind the last step: page 0
                load_keys<DP>(a, place, k_at, k);
                attend_weights<DP, MT>(scales_of(a, ks, v.s, ok), e, w, p);
                attend_values<DP, MT, false>(v, p, none, w);
            }
            unsigned long long above = 0;
            if (a.s.parents && plain < to)
                above = tree_node(a.s.parents + (int64_t)pc.b * a.s.N, a.s.N).above;
            // steps with slots that some row does not see
#pragma clang loop unroll(disable)
            for (int s = plain; s < to; ++s) {
                if (s > plain) {
                    place = attend_next(a, at, h);
                    load_keys<DP>(a, place, k_at, k);
                }
                load_values<DP>(a, place, v_at, v);
                if (!(k.ok[0] && k.ok[1])) put_out<DP>(k, v);
                attend_scores<DP, MT, F16>(k, w, e);
                const int rel = s * AT_STEP - row.base + g * 4, end = row.end - row.base;
                uint32_t vis[MT];
                attend_mask<MT>(a, above, first, rows, rel, end, k.ok, e, vis);
                // values behind the last token are not numbers to be multiplied by 0
                const uint32_t there = ((1u << min(max(end - rel, 0), 4)) - 1) |
                                       ((1u << min(max(end - rel - 16, 0), 4)) - 1) << 4;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
#pragma unroll
                    for (int c = 0; c < DP / 64; ++c)
                        set_word<DP>(v.v[j], c, keep_if(there, j, word_of<DP>(v.v[j], c), 0u));
                }
                attend_weights<DP, MT>(scales_of(a, k.s, v.s, k.ok), e, w, p);
                attend_values<DP, MT, true>(v, p, vis, w);
            }
        }

        // the waves' sums to one reference
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            w.l[m] += xor_lane_f<16>(w.l[m]);
            w.l[m] += xor_lane_f<32>(w.l[m]);
            if (g == 0) {
                s_ref[wave][m * 16 + col] = w.ref[m];
                s_l[wave][m * 16 + col] = w.l[m];
            }
        }
        // a thread adds pairs of entries of a row, neighbours' pairs side by side
        constexpr int PER_ROW = WAVES * 4;
        const int r16 = tid / PER_ROW, part = tid % PER_ROW;
        float* slot = a.part + (int64_t)attend_left(a, pc, pc.p, pc.c == 0) * SLOT;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            __syncthreads();
            float ref = s_ref[0][m * 16 + col];
#pragma unroll
            for (int v = 1; v < WAVES; ++v) ref = fmaxf(ref, s_ref[v][m * 16 + col]);
            const float f = __builtin_amdgcn_exp2f(w.ref[m] - ref);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int d = 0; d < DT; d += 4) {
                    const f32x4 v = {w.o[m][d][i] * f, w.o[m][d + 1][i] * f, w.o[m][d + 2][i] * f,
                                     w.o[m][d + 3][i] * f};
                    *reinterpret_cast<f32x4*>(&s_o[wave][col][(g * 4 + i) * DT + d]) = v;
                }
            __syncthreads();
            const int rr = m * 16 + r16;
            if (rr >= rows) continue;
            ref = s_ref[0][rr];
#pragma unroll
            for (int v = 1; v < WAVES; ++v) ref = fmaxf(ref, s_ref[v][rr]);
            float l = 0.0f;
#pragma unroll
            for (int v = 0; v < WAVES; ++v)
                l = __builtin_fmaf(s_l[v][rr], __builtin_amdgcn_exp2f(s_ref[v][rr] - ref), l);
            const bool live = s_live[rr] != 0;
            const AttendOut out = attend_out(a, pc.b, h, first + rr);
            const float to = attend_factor(l, live);
            if (part == 0) {
                if (pc.n > 1) put(slot + rr * 2, ref, l);
                else if (a.lse) a.lse[out.lse] = attend_lse(ref, l, live);
            }
#pragma unroll
            for (int k = 0; k < DP / 2 / PER_ROW; ++k) {
                const int e = (k * PER_ROW + part) * 2;
                f32x2 o = {0.0f, 0.0f};
#pragma unroll
                for (int v = 0; v < WAVES; ++v) o += *reinterpret_cast<const f32x2*>(&s_o[v][r16][e]);
                if (pc.n > 1) put(slot + 2 * MT * 16 + rr * DP + e, o[0], o[1]);
                else if (e < a.g.dim) put_pair<F16>(out.to + e, o[0], o[1], to, live);
            }
        }
        if (pc.n > 1) add_pieces<DP, MT * 16, F16>(a, pc, rows, &s_o[0][0][0], s_live);
        __syncthreads();  // LDS is read
    } while (attend_on<UNIT, MT * 16>(args, pc));
}

// ---------------------------------------------------------------------------
// Many rows: the waves of a workgroup take rows of their own, 16 * MT each, and share keys and
// values. Of a tile of 64 slots every wave widens 16 and leaves them in LDS as the operands'
// registers hold them: keys 16 bytes a lane, so that neither its writes nor the reads meet in a
// bank; values, of which a wave has half of an operand, 8 bytes at a stride of 16, whose writes
// do (4 % of a CU's cycles). Two tiles take turns: one is read while the next is left, with a
// barrier a tile; the one after that is on its way from memory meanwhile.
// What bounds it: no unit alone. Of a tile a wave of 32 rows has 64 matrix instructions and 248
// other vector ones (counted), and two waves a SIMD take 2.5 us for it. Vector instructions take
// 52 % of a SIMD's cycles, products 39 %, reading operands from LDS about as long as they, by
// their bytes; a wave waits for 28 % of its cycles. 2048 tokens behind 6144 slots, 32 heads of
// 128: 283 to 291 us, 826 to 850 TFLOP/s; 32 trees of 16 nodes over 2000 slots: 58 to 68 us by
// their lengths, with 25 MB of pieces left and read again beside 130 MB of pages. Scores of the next half tile formed
// between this one's weights, with a second barrier, took 299 us; a wave of higher priority while
// it multiplies 291.

constexpr int AT_TILE = 64;

template <int DP>
struct AttendTile {
    u32x4 k[4][DP / 32][WAVE];  // by tile of 16 slots and step of 32 dimensions
    u32x4 v[2][DP / 16][WAVE];  // by step of 32 slots and tile of 16 dimensions
    f32x4 x[4];                 // factor on S, exponent of the weights, its inverse
};

// A wave's 16 slots of the next tile, as they lie in the page.
template <int DP>
struct AttendRaw {
    u32x4 k[DP / 64];
    typename Words<DP / 64>::type v[4];
    uint32_t ks, vs;
    bool ok;
    int there;  // its slots up to the row's last
};

// Where a wave's 16 slots of a tile lie in its row.
struct AttendWalk {
    const_i32 table;
    int block, inner;        // table entry, tile of 16 within its page
    int tiles, over, ahead;  // tiles of a page; table entries and tiles from one tile of 64 to the next
    int left;                // slots from there up to the row's last
};

template <int DP>
__device__ __forceinline__ void load_raw(const Kv8Attend& a, AttendWalk& c, int h, const uint32_t (&k_at)[DP / 64],
                                         const uint32_t (&v_at)[4], AttendRaw<DP>& x) {
    int page = -1;
    if (c.left > 0) page = c.table[c.block];
    x.ok = (unsigned)page < (unsigned)a.g.num_pages;
    x.there = c.left;
    const int64_t p = x.ok ? page : 0;
    const int off = c.inner * 16;
    const int64_t at = p * a.g.page + off * a.g.slot + h * a.g.head;
    const int64_t sc = p * a.g.sc_page + (off >> a.g.block_bits) * a.g.sc_block + h * a.g.sc_head;
#pragma unroll
    for (int i = 0; i < DP / 64; ++i) x.k[i] = *reinterpret_cast<const u32x4*>(a.k.data + at + k_at[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        x.v[j] = *reinterpret_cast<const typename Words<DP / 64>::type*>(a.v.data + at + v_at[j]);
    x.ks = scale_byte(a.k.scales + sc);
    x.vs = scale_byte(a.v.scales + sc);
    c.left -= AT_TILE;
    c.block += c.over;
    c.inner += c.ahead;
    if (c.inner >= c.tiles) {
        c.inner -= c.tiles;
        ++c.block;
    }
}

// Widens them into the tile, as its wave-th 16.
template <int DP, bool F16>
__device__ __forceinline__ void leave_raw(const Kv8Attend& a, AttendRaw<DP>& x, int wave, AttendTile<DP>& t) {
    const int lane = threadIdx.x & (WAVE - 1);
    if (!x.ok || x.there < 16) {  // values behind the last token are not numbers to be multiplied by 0
        const int g = lane >> 4;
#pragma unroll
        for (int c = 0; c < DP / 64; ++c)
            if (!x.ok) x.k[c] = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (!x.ok || g * 4 + j >= x.there) x.v[j] = {};
    }
#pragma unroll
    for (int st = 0; st < DP / 32; ++st) {
        const uint32_t w0 = x.k[st / 2][st % 2 * 2], w1 = x.k[st / 2][st % 2 * 2 + 1];
        t.k[wave][st][lane] = u32x4{widen<F16>(w0, false), widen<F16>(w0, true), widen<F16>(w1, false),
                                    widen<F16>(w1, true)};
    }
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) {
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            lo[j] = widen<true>(word_of<DP>(x.v[j], c), false);
            hi[j] = widen<true>(word_of<DP>(x.v[j], c), true);
        }
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            u32x2 v;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t u0 = d < 2 ? lo[2 * j] : hi[2 * j], u1 = d < 2 ? lo[2 * j + 1] : hi[2 * j + 1];
                v[j] = __builtin_amdgcn_perm(u1, u0, d % 2 ? 0x07060302u : 0x05040100u);
            }
            reinterpret_cast<u32x2*>(&t.v[wave / 2][c * 4 + d][lane])[wave % 2] = v;
        }
    }
    if (lane == 0) {
        const uint32_t v = clamp_scale(x.vs);
        t.x[wave] = f32x4{as<float>(clamp_scale(x.ks) << 23) * a.scale_log2,
                          x.ok ? (float)((int)v - 127) : -INFINITY, as<float>((254u - v) << 23), 0.0f};
    }
}

// The half-th 32 slots of the tile in LDS. rel and end as attend_mask has them, for the wave's
// rows from `first` on.
template <int DP, int MT, bool F16, bool MASK>
__device__ __forceinline__ void attend_tile(const Kv8Attend& a, const AttendTile<DP>& t, int half, int rel,
                                            int end, unsigned long long above, int first, int rows,
                                            AttendState<DP, MT>& w) {
    const int lane = threadIdx.x & (WAVE - 1);
    f32x4 e[2][MT];
    u32x4 p[MT];
    AttendScales x;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const f32x4 v = t.x[half * 2 + k];
        x.fk[k] = v[0];
        x.xv[k] = v[1];
        x.inv[k] = v[2];
#pragma unroll
        for (int m = 0; m < MT; ++m) e[k][m] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int st = 0; st < DP / 32; ++st) {
            const u32x4 f = t.k[half * 2 + k][st][lane];
#pragma unroll
            for (int m = 0; m < MT; ++m) e[k][m] = mfma<F16>(f, w.q[m][st], e[k][m]);
        }
    }
    uint32_t vis[MT] = {};
    // the same in all lanes
    const bool ok[2] = {__builtin_amdgcn_readfirstlane(as<int>(x.xv[0])) != as<int>(-INFINITY),
                        __builtin_amdgcn_readfirstlane(as<int>(x.xv[1])) != as<int>(-INFINITY)};
    if constexpr (MASK) attend_mask<MT>(a, above, first, rows, rel, end, ok, e, vis);
    else put_out_scores<MT>(ok, e);
    attend_weights<DP, MT>(x, e, w, p);
#pragma unroll
    for (int d = 0; d < DP / 16; ++d) {
        u32x4 v = t.v[half][d][lane];
        if constexpr (MASK) {
            f32x4* o[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) o[m] = &w.o[m][d];
            v = take_nans<MT>(v, vis, o);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) w.o[m][d] = mfma<true>(v, p[m], w.o[m][d]);
    }
}

template <int DP, int MT, bool F16>
__global__ __launch_bounds__(256, 2) void k_attend_rows(Kv8Attend args) {
    constexpr int WAVES = 4;
    constexpr int DT = DP / 16;
    constexpr int ROWS = WAVES * MT * 16;
    constexpr int SLOT = attend_slot(DP, ROWS);
    union Shared {
        AttendTile<DP> t[2];
        float o[WAVES][16][DP + 4];
    };
    __shared__ Shared sh;
    __shared__ int s_live[ROWS];
    AttendPiece pc;
    if (!attend_share<AT_TILE, ROWS>(args, pc)) return;
    ArgsAgain again;
    do {
        const Kv8Attend& a = again.args();
        const int lane = again.thread() & (WAVE - 1);
        const int wave = __builtin_amdgcn_readfirstlane(again.thread() / WAVE);
        const int g = lane >> 4, col = lane & 15;
        const int h = pc.h, first = pc.first;
        const int rows = min(a.s.N * a.group - first, ROWS);
        const AttendRow row = attend_row(a, pc.b);

        const int mine = first + wave * MT * 16;                       // rows of this wave
        const int count = min(max(rows - wave * MT * 16, 0), MT * 16);
        unsigned long long above = 0, rooted = 0;
        if (a.s.parents) {
            above = tree_node(a.s.parents + (int64_t)pc.b * a.s.N, a.s.N).above;
            rooted = __ballot(above != 0);
        }
        AttendState<DP, MT> w;
        uint32_t lives = 0;  // of a lane's rows; in LDS for other lanes, which a barrier must divide
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int r = mine + min(m * 16 + col, max(count, 1) - 1);
            const int rc = min(r, first + rows - 1);
            const int n = rc / a.group;
            w.l[m] = 0.0f;
            w.ref[m] = AT_NONE;
            const bool live = n < row.count && (!a.s.parents || (rooted >> (n & 63) & 1));
            if (g == 0) s_live[wave * MT * 16 + m * 16 + col] = live;
            lives |= (live ? 1u : 0u) << m;
            const uint16_t* q = a.q.data + pc.b * a.q.row + n * a.q.token +
                                (h * a.group + rc - n * a.group) * a.q.head + g * 16;
#pragma unroll
            for (int st = 0; st < DP / 32; ++st) {
                w.q[m][st] = u32x4{0, 0, 0, 0};
                if (st / 2 * 64 + g * 16 < a.g.dim)
                    w.q[m][st] = *reinterpret_cast<const u32x4*>(q + st / 2 * 64 + st % 2 * 8);
            }
#pragma unroll
            for (int d = 0; d < DT; ++d) w.o[m][d] = f32x4{0, 0, 0, 0};
        }

        // tiles of this piece, and what this wave's rows see of them
        const int see = count ? attend_see(a, row, (mine + count - 1) / a.group) : 0;
        int full = min(row.base, row.end);
        if (!a.s.parents && row.count) full = (int)min((int64_t)row.end, (int64_t)row.base + first / a.group + 1);
        const int t0 = pc.from;
        const int most = attend_see(a, row, (first + rows - 1) / a.group);
        const int t1 = min(pc.to, (int)(((int64_t)most + AT_TILE - 1) / AT_TILE));
        const int t2 = max(min(full / AT_TILE, t1), t0);  // tiles before it need no mask
        if (t0 < t1) {
            AttendWalk at;
            at.table = (const_i32)(a.s.t.tables + (int64_t)pc.b * a.s.t.stride);
            at.tiles = a.g.page_size / 16;
            at.over = 4 / at.tiles;
            at.ahead = 4 - at.over * at.tiles;
            at.block = (t0 * 4 + wave) / at.tiles;
            at.inner = t0 * 4 + wave - at.block * at.tiles;
            at.left = row.end - (t0 * AT_TILE + wave * 16);
            uint32_t k_at[DP / 64], v_at[4];
#pragma unroll
            for (int c = 0; c < DP / 64; ++c)
                k_at[c] = (uint32_t)col * (uint32_t)a.g.slot + (c * 64 + g * 16 < a.g.dim ? c * 64 + g * 16 : 0);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v_at[j] = (uint32_t)(g * 4 + j) * (uint32_t)a.g.slot + (col * DT < a.g.dim ? col * DT : 0);
            AttendRaw<DP> raw;
            load_raw<DP>(a, at, h, k_at, v_at, raw);
            leave_raw<DP, F16>(a, raw, wave, sh.t[0]);
            load_raw<DP>(a, at, h, k_at, v_at, raw);
            auto next = [&](int i) {
                __syncthreads();
                if (i + 1 < t1) {
                    leave_raw<DP, F16>(a, raw, wave, sh.t[(i - t0 + 1) & 1]);
                    load_raw<DP>(a, at, h, k_at, v_at, raw);
                }
            };
            // tiles that all rows see
            for (int i = t0; i < t2; ++i) {
                next(i);
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    attend_tile<DP, MT, F16, false>(a, sh.t[(i - t0) & 1], k, 0, 0, 0, mine, count, w);
            }
            // those that some row does not see, of the step's own tokens or behind the last one: in a
            // loop of their own, or what they need is kept, in scratch memory, through the other
#pragma clang loop unroll(disable)
            for (int i = t2; i < t1; ++i) {
                next(i);
                const int s0 = i * AT_TILE;
#pragma clang loop unroll(disable)
                for (int k = 0; k < 2 && s0 + k * AT_STEP < see; ++k)
                    attend_tile<DP, MT, F16, true>(a, sh.t[(i - t0) & 1], k, s0 + k * AT_STEP - row.base + g * 4,
                                                      row.end - row.base, above, mine, count, w);
            }
        }

        float* slot = a.part + (int64_t)attend_left(a, pc, pc.p, pc.c == 0) * SLOT;
        if (pc.n > 1) __syncthreads();  // the tiles are read; what pieces leave goes through LDS, in whole lines
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            w.l[m] += xor_lane_f<16>(w.l[m]);
            w.l[m] += xor_lane_f<32>(w.l[m]);
            const int r0 = wave * MT * 16 + m * 16, rr = r0 + col;
            if (pc.n > 1) {
                if (g == 0 && rr < rows) put(slot + rr * 2, w.ref[m], w.l[m]);
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int d = 0; d < DT; d += 4)
                        *reinterpret_cast<f32x4*>(&sh.o[wave][col][(g * 4 + k) * DT + d]) =
                            f32x4{w.o[m][d][k], w.o[m][d + 1][k], w.o[m][d + 2][k], w.o[m][d + 3][k]};
                __builtin_amdgcn_wave_barrier();  // a wave's own part: its LDS operations stay in order
#pragma unroll
                for (int k = 0; k < DP / 8; ++k) {
                    const int r = (k * WAVE + lane) * 2 / DP, e = (k * WAVE + lane) * 2 % DP;
                    const f32x2 o = *reinterpret_cast<const f32x2*>(&sh.o[wave][r][e]);
                    if (r0 + r < rows) put(slot + 2 * ROWS + (r0 + r) * DP + e, o[0], o[1]);
                }
                __builtin_amdgcn_wave_barrier();
            } else if (rr < rows) {  // a lane has 4 * DT neighbouring entries of a row
                const bool live = lives >> m & 1;
                const float f = attend_factor(w.l[m], live);
                const AttendOut out = attend_out(a, pc.b, h, first + rr);
                if (a.lse && g == 0) a.lse[out.lse] = attend_lse(w.ref[m], w.l[m], live);
#pragma unroll
                for (int e = 0; e < 4 * DT; e += 8) {
                    if (g * 4 * DT + e >= a.g.dim) break;
                    u32x4 v;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int x = e + 2 * k;
                        v[k] = live ? narrow<F16>(w.o[m][x % DT][x / DT] * f, w.o[m][x % DT + 1][x / DT] * f) : 0u;
                    }
                    *reinterpret_cast<u32x4*>(out.to + g * 4 * DT + e) = v;
                }
            }
        }
        if (pc.n > 1) add_pieces<DP, ROWS, F16>(a, pc, rows, &sh.o[0][0][0], s_live);
        __syncthreads();  // LDS is read
    } while (attend_on<AT_TILE, ROWS>(args, pc));
}

// Into how many shares the slots of a head and block of rows are cut: as many as there are CUs
// (few rows: a workgroup a CU; twice as many took 60 -> 73 us for one request of 131072 slots and
// 115 -> 130 for 64 uneven ones of 4000, since more pages are read at a time) or twice that (many
// rows: two a CU; 32 trees of 64 rows over 2000 slots 81 -> 68 us), as far as what they leave has
// room: of blocks of 128 rows in heads of 128 283, so that several prompts, which are cut, run one
// workgroup a CU (8 of 512 tokens behind 512: 146 us, 354 TFLOP/s; 64 trees of 64 nodes and 8
// query heads a head: 633).
template <int ROWS>
static int64_t attend_grid(Kv8Attend& a, int dp, int workgroups) {
    a.blocks = (int)(((int64_t)a.s.N * a.group + ROWS - 1) / ROWS);
    const int64_t lines = (int64_t)a.g.heads * a.blocks;
    const int64_t most = KV8_PART_FLOATS / (2 * attend_slot(dp, ROWS));
    if (workgroups > most) workgroups = (int)most;
    a.shares = (int)(workgroups / lines);
    // whole requests where there are many, or where lines alone fill the card
    if (lines * a.s.B >= 4 * workgroups || a.s.B * ((int64_t)a.g.max_blocks * a.g.page_size / 64 + 1) > INT_MAX)
        a.shares = 0;
    return lines * (a.shares ? a.shares : a.s.B);
}

template <int DP, int MT, bool F16>
static hipError_t launch_few(Kv8Attend a, hipStream_t st) {
    const int64_t grid = attend_grid<MT * 16>(a, DP, AT_CUS);
    if (grid > INT_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_attend<DP, MT, F16>), dim3((unsigned)grid), dim3(256), 0, st, a);
    return hipGetLastError();
}

template <int DP, int MT, bool F16>
static hipError_t launch_many(Kv8Attend a, hipStream_t st) {
    const int64_t grid = attend_grid<MT * 64>(a, DP, 2 * AT_CUS);
    if (grid > INT_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_attend_rows<DP, MT, F16>), dim3((unsigned)grid), dim3(256), 0, st, a);
    return hipGetLastError();
}

// Up to 32 rows a wave takes them all, and heads above 128 always go that way: 32 requests of 8
// nodes and 4 query heads a head over 2000 slots take 50 us so and 57 where four waves share
// keys and values (16 nodes: 73 and 62); in heads of 256 16 nodes take 118 and 208, a prompt's
// 2048 tokens over 6144 slots, 16 query heads, 410 and 562. Above 64 rows a wave takes 32 of them; so it does
// not where workgroups of 128 rows leave CUs idle.
template <int DP, bool F16>
static hipError_t launch_attend_rows(const Kv8Attend& a, hipStream_t st) {
    const int64_t rows = (int64_t)a.s.N * a.group;
    if (rows <= 16) return launch_few<DP, 1, F16>(a, st);
    if (rows <= 32 || DP > 128) return launch_few<DP, 2, F16>(a, st);
    if constexpr (DP <= 128) {
        if (rows <= 64 || (rows + 127) / 128 * a.g.heads * a.s.B < AT_CUS) return launch_many<DP, 1, F16>(a, st);
        return launch_many<DP, 2, F16>(a, st);
    }
    return hipErrorInvalidValue;
}

template <bool F16>
static hipError_t launch_attend_dim(const Kv8Attend& a, hipStream_t st) {
    if (a.g.dim <= 64) return launch_attend_rows<64, F16>(a, st);
    if (a.g.dim <= 128) return launch_attend_rows<128, F16>(a, st);
    return launch_attend_rows<256, F16>(a, st);
}

hipError_t launch_kv8_attend(const Kv8Attend& a, ss_dtype dt, hipStream_t st) {
    return dt == SS_F16 ? launch_attend_dim<true>(a, st) : launch_attend_dim<false>(a, st);
}

}  // namespace ss
