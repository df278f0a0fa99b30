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
#include <stdlib.h>

#include "ss_device.h"
#include "ss_internal.h"

namespace ss {

constexpr int AT_STEP = 32;                   // slots of a wave's step
constexpr float AT_NONE = -3.0e38f;           // reference of a row that has seen nothing
constexpr float AT_SET = 8.0f, AT_MOST = 15.0f;

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

// Bytes of a word that are a NaN, as 0x80 each.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
    return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
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

// Weights of one step: s becomes them, under the rows' references, which may grow.
template <int DP, int MT>
__device__ __forceinline__ void attend_weights(const Kv8Attend& a, const uint32_t (&ks)[2],
                                               const uint32_t (&vs)[2], const bool (&ok)[2], const f32x4 (&s)[2][MT],
                                               AttendState<DP, MT>& w, u32x4 (&p)[MT]) {
    float fk[2], xv[2], inv[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const uint32_t v = clamp_scale(vs[t]);
        fk[t] = as<float>(clamp_scale(ks[t]) << 23) * a.scale_log2;
        xv[t] = ok[t] ? (float)((int)v - 127) : -INFINITY;
        inv[t] = as<float>((254u - v) << 23);
    }
    float top[MT];
    bool grows = false;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        top[m] = -INFINITY;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const float most = fmaxf(fmaxf(s[t][m][0], s[t][m][1]), fmaxf(s[t][m][2], s[t][m][3]));
            top[m] = fmaxf(top[m], __builtin_fmaf(most, fk[t], xv[t]));
        }
        grows |= top[m] > w.ref[m] + AT_MOST;
    }
    if (__any(grows)) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            top[m] = fmaxf(top[m], xor_lane_f<16>(top[m]));
            top[m] = fmaxf(top[m], xor_lane_f<32>(top[m]));
            if (top[m] > w.ref[m] + AT_MOST) {
                const float to = top[m] - AT_SET;
                const float f = __builtin_amdgcn_exp2f(w.ref[m] - to);
                w.ref[m] = to;
                w.l[m] *= f;
#pragma unroll
                for (int d = 0; d < DP / 16; ++d) w.o[m][d] *= f;
            }
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const float c = xv[t] - w.ref[m];
            float e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][m][i], fk[t], c));
            w.l[m] = __builtin_fmaf((e[0] + e[1]) + (e[2] + e[3]), inv[t], w.l[m]);
            p[m][2 * t] = as<uint32_t>(__builtin_convertvector((f32x2{e[0], e[1]}), h16x2));
            p[m][2 * t + 1] = as<uint32_t>(__builtin_convertvector((f32x2{e[2], e[3]}), h16x2));
        }
    }
}

// O^T of one step.
template <int DP, int MT>
__device__ __forceinline__ void attend_values(const AttendValues<DP>& x, const u32x4 (&p)[MT],
                                              AttendState<DP, MT>& w) {
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
#pragma unroll
            for (int m = 0; m < MT; ++m) w.o[m][c * 4 + d] = mfma<true>(v, p[m], w.o[m][c * 4 + d]);
        }
    }
}

// A NaN among the values reaches the rows that see it and no others: it is counted where it
// is seen, and taken out of the product.
template <int DP, int MT>
__device__ __forceinline__ void attend_nans(AttendValues<DP>& x, const uint32_t (&vis)[MT],
                                            AttendState<DP, MT>& w) {
    uint32_t any = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int c = 0; c < DP / 64; ++c) any |= nan_bytes(word_of<DP>(x.v[j], c));
    if (!__any(any != 0)) return;
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) {
        uint32_t nan[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t word = word_of<DP>(x.v[j], c);
            nan[j] = nan_bytes(word);
            set_word<DP>(x.v[j], c, word & ~((nan[j] >> 7) * 0xffu));
        }
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            u32x4 hot;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                hot[j] = ((nan[2 * j] >> (8 * d + 7)) & 1) * 0x3c00u |
                         ((nan[2 * j + 1] >> (8 * d + 7)) & 1) * 0x3c000000u;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                u32x4 sees;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sees[j] = (vis[m] >> (2 * j) & 1) * 0x3c00u | (vis[m] >> (2 * j + 1) & 1) * 0x3c000000u;
                const f32x4 n = mfma<true>(hot, sees, f32x4{0, 0, 0, 0});
#pragma unroll
                for (int i = 0; i < 4; ++i)  // n is 0 or at least 1
                    w.o[m][c * 4 + d][i] += n[i] * (as<float>(as<uint32_t>((float)n[i]) ? 0x7fc00000u : 0u));
            }
        }
    }
}

// Where workgroup `item` of a head and block of rows works: row b, piece c of its n. Rows
// are cut into pieces of equal size, about as many over all rows as a.pieces; every wave
// finds its own by itself.
struct AttendPiece {
    int b, c, n, units;  // units of UNIT slots of a piece
};

template <int UNIT>
__device__ __forceinline__ AttendPiece attend_piece(const Kv8Attend& a, int item) {
    if (a.pieces == 0) return {item, 0, 1, INT_MAX / UNIT};
    const int lane = threadIdx.x & (WAVE - 1);
    int total = 0;
    for (int b0 = 0; b0 < a.s.B; b0 += WAVE) {
        const int b = b0 + lane;
        if (b < a.s.B) total += max(1, (int)(((int64_t)attend_row(a, b).end + UNIT - 1) / UNIT));
    }
    total = wave_sum_i(total);
    const int units = (total + a.pieces - 1) / a.pieces;
    int before = 0;
    for (int b0 = 0; b0 < a.s.B; b0 += WAVE) {
        const int b = b0 + lane;
        int n = 0;
        if (b < a.s.B) {
            const int u = max(1, (int)(((int64_t)attend_row(a, b).end + UNIT - 1) / UNIT));
            n = (u + units - 1) / units;
        }
        const int to = before + wave_incl_scan_i(n);
        const unsigned long long m = __ballot(item < to);
        if (m) {
            const int l = __builtin_ctzll(m);
            const int nl = __shfl(n, l);
            return {b0 + l, item - (__shfl(to, l) - nl), nl, units};
        }
        before = __shfl(to, WAVE - 1);
    }
    return {-1, 0, 0, 0};
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

// Writes D neighbouring entries of a row of the output from entry d0 on.
template <int D, bool F16>
__device__ __forceinline__ void attend_out(const Kv8Attend& a, int b, int n, int head, int d0,
                                           const float* o, float f) {
    uint32_t r[D / 2];
#pragma unroll
    for (int i = 0; i < D / 2; ++i) {
        const f32x2 v = {o[2 * i] * f, o[2 * i + 1] * f};
        if constexpr (F16) r[i] = as<uint32_t>(__builtin_convertvector(v, h16x2));
        else r[i] = as<uint32_t>(__builtin_convertvector(v, b16x2));
    }
    uint16_t* to = a.out.data + b * a.out.row + n * a.out.token + head * a.out.head + d0;
    typedef typename Words<D / 2 < 4 ? D / 2 : 4>::type V;
#pragma unroll
    for (int i = 0; i < D / 2; i += sizeof(V) / 4) {
        V v;
        if constexpr (sizeof(V) == 4) {
            v = r[i];
        } else {
#pragma unroll
            for (unsigned k = 0; k < sizeof(V) / 4; ++k) v[k] = r[i + k];
        }
        *reinterpret_cast<V*>(to + 2 * i) = v;
    }
}

// A row's sums under one reference, of the entries that a thread has.
template <int PT>
struct AttendSum {
    float ref, l;
    float o[PT];
};

// Adds the waves' sums of row r (of the 16 from m on), which lie under the waves' largest
// reference.
template <int DP, int PT, int WAVES, class O, class S>
__device__ __forceinline__ AttendSum<PT> add_waves(const O& s_o, const S& s_ref, const S& s_l, int m, int r,
                                                   int part) {
    AttendSum<PT> s;
    s.ref = s_ref[0][m + r];
#pragma unroll
    for (int v = 1; v < WAVES; ++v) s.ref = fmaxf(s.ref, s_ref[v][m + r]);
    s.l = 0.0f;
#pragma unroll
    for (int d = 0; d < PT; ++d) s.o[d] = 0.0f;
#pragma unroll
    for (int v = 0; v < WAVES; ++v) {
        s.l = __builtin_fmaf(s_l[v][m + r], __builtin_amdgcn_exp2f(s_ref[v][m + r] - s.ref), s.l);
#pragma unroll
        for (int d = 0; d < PT; ++d) s.o[d] += s_o[v][r][part * PT + d];
    }
    return s;
}

// Row r of a head of the cache to the output: 0 where it has seen nothing, or scores of -inf
// alone.
template <int PT, bool F16>
__device__ __forceinline__ void attend_result(const Kv8Attend& a, AttendSum<PT> s, int b, int h, int r,
                                              int part, bool live) {
    const int n = r / a.group, head = h * a.group + r - n * a.group;
    if (!live) {
#pragma unroll
        for (int d = 0; d < PT; ++d) s.o[d] = 0.0f;
    }
    if (part * PT < a.g.dim)
        attend_out<PT, F16>(a, b, n, head, part * PT, s.o, live && s.l != 0.0f ? 1.0f / s.l : 0.0f);
    if (a.lse && part == 0)
        a.lse[((int64_t)b * a.s.N + n) * a.q_heads + head] =
            live ? (s.ref + log2f(s.l)) * 0.69314718055994531f : -INFINITY;
}

template <int DP, int MT, bool F16, int WAVES>
__global__ __launch_bounds__(WAVES* WAVE, DP == 256 || MT == 4 ? 1 : MT == 2 ? 2 : DP == 128 ? 3 : 4) void k_attend(Kv8Attend a) {
    constexpr int DT = DP / 16;
    constexpr int PT = DP / (WAVES * 4);      // entries of a row that a thread adds
    constexpr int SLOT = MT * 16 * (DP + 2);  // floats that a piece leaves
    __shared__ float s_o[WAVES][16][DP + 4];
    __shared__ float s_ref[WAVES][MT * 16], s_l[WAVES][MT * 16];
    __shared__ int s_live[MT * 16];
    __shared__ int s_last;
    const int tid = threadIdx.x;
    const int lane = tid & (WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int g = lane >> 4, col = lane & 15;
    const int items = a.s.B + a.pieces;
    const int item = blockIdx.x % items;
    const int y = blockIdx.x / items;
    const int h = y / a.blocks;
    const int first = (y - h * a.blocks) * (MT * 16);  // row of this block
    const int rows = min(a.s.N * a.group - first, MT * 16);
    AttendPiece pc = attend_piece<AT_STEP * WAVES>(a, item);
    pc.b = __builtin_amdgcn_readfirstlane(pc.b);
    pc.c = __builtin_amdgcn_readfirstlane(pc.c);
    pc.n = __builtin_amdgcn_readfirstlane(pc.n);
    pc.units = __builtin_amdgcn_readfirstlane(pc.units);
    if (pc.b < 0) return;
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
    int see = row.end;
    int full = min(row.base, row.end);  // slots before it all rows see
    if (!a.s.parents && row.count) {
        see = (int)min((int64_t)see, (int64_t)row.base + (first + rows - 1) / a.group + 1);
        full = (int)min((int64_t)row.end, (int64_t)row.base + first / a.group + 1);
    }
    const int steps = (int)(((int64_t)see + AT_STEP - 1) / AT_STEP);
    const int s0 = (int)min((int64_t)pc.c * pc.units * WAVES, (int64_t)steps);
    const int s1 = (int)min((int64_t)(pc.c + 1) * pc.units * WAVES, (int64_t)steps);
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
        attend_look(at);
        AttendPlace place = attend_next(a, at, h);
        load_keys<DP>(a, place, k_at, k);
        // keys of the next step are on their way while this one's weights and values are
        // worked on, values while its scores are
        for (int s = from; s < plain; ++s) {
            load_values<DP>(a, place, v_at, v);
            if (!(k.ok[0] && k.ok[1])) put_out<DP>(k, v);
            attend_scores<DP, MT, F16>(k, w, e);
            const uint32_t ks[2] = {k.s[0], k.s[1]};
            const bool ok[2] = {k.ok[0], k.ok[1]};
            place = attend_next(a, at, h);  // behind the last step: page 0
            load_keys<DP>(a, place, k_at, k);
            attend_weights<DP, MT>(a, ks, v.s, ok, e, w, p);
            attend_values<DP, MT>(v, p, w);
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
            uint32_t vis[MT];  // bit 4 t + i: slot i of this lane's in tile t is seen
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int n = (first + min(m * 16 + col, rows - 1)) / a.group;
                const unsigned long long up =
                    (unsigned long long)(uint32_t)__shfl((int)(above >> 32), n & 63) << 32 |
                    (uint32_t)__shfl((int)above, n & 63);
                vis[m] = attend_sees(a.s.parents, up, n, rel, end) |
                         attend_sees(a.s.parents, up, n, rel + 16, end) << 4;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        e[t][m][i] = as<float>(keep_if(vis[m], 4 * t + i, as<uint32_t>((float)e[t][m][i]), 0xff800000u));
            }
            // values behind the last token are not numbers to be multiplied by 0
            const uint32_t there = ((1u << min(max(end - rel, 0), 4)) - 1) |
                                   ((1u << min(max(end - rel - 16, 0), 4)) - 1) << 4;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
#pragma unroll
                for (int c = 0; c < DP / 64; ++c)
                    set_word<DP>(v.v[j], c, keep_if(there, j, word_of<DP>(v.v[j], c), 0u));
            }
            attend_weights<DP, MT>(a, k.s, v.s, k.ok, e, w, p);
            attend_nans<DP, MT>(v, vis, w);
            attend_values<DP, MT>(v, p, w);
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
    const int r16 = tid / (DP / PT), part = tid % (DP / PT);
    float* slot = a.part + (int64_t)blockIdx.x * SLOT;
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
        if (m * 16 + r16 >= rows) continue;
        AttendSum<PT> sum = add_waves<DP, PT, WAVES>(s_o, s_ref, s_l, m * 16, r16, part);
        const int rr = m * 16 + r16;
        if (pc.n > 1) {
            if (part == 0) put(slot + rr * 2, sum.ref, sum.l);
#pragma unroll
            for (int d = 0; d < PT; d += 2)
                put(slot + MT * 32 + rr * DP + part * PT + d, sum.o[d], sum.o[d + 1]);
        } else {
            attend_result<PT, F16>(a, sum, pc.b, h, first + rr, part, s_live[rr] != 0);
        }
    }
    if (pc.n <= 1) return;

    // the last piece of a row adds them all, in their order: a wave every WAVES-th of them
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid == 0) {
        int32_t* arrived = a.arrived + ((int64_t)y * a.s.B + pc.b) * KV8_COUNTER;
        s_last = __hip_atomic_fetch_add(arrived, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == pc.n - 1;
        if (s_last) __hip_atomic_store(arrived, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (!s_last) return;
    const float* all = a.part + (int64_t)(blockIdx.x - pc.c) * SLOT;  // pieces of a row follow each other
    for (int r0 = 0; r0 < rows; r0 += 8) {
        constexpr int ET = DP / 8;  // entries of a row that a lane adds
        const int r = lane / 8, e0 = lane % 8 * ET;
        const int rc = min(r0 + r, rows - 1);  // lanes behind the last row add it again
        AttendSum<ET> sum;
        sum.ref = AT_NONE;
        sum.l = 0.0f;
#pragma unroll
        for (int d = 0; d < ET; ++d) sum.o[d] = 0.0f;
        constexpr int AT_ONCE = 64 / ET < 4 ? 64 / ET : 4;
        for (int c0 = wave; c0 < pc.n; c0 += AT_ONCE * WAVES) {
            f32x2 s[AT_ONCE], v[AT_ONCE][ET / 2];
#pragma unroll
            for (int k = 0; k < AT_ONCE; ++k) {
                const float* p = all + (int64_t)min(c0 + k * WAVES, pc.n - 1) * SLOT;
                s[k] = get(p + rc * 2);
#pragma unroll
                for (int d = 0; d < ET / 2; ++d) v[k][d] = get(p + MT * 32 + rc * DP + e0 + 2 * d);
            }
            float ref = sum.ref;
#pragma unroll
            for (int k = 0; k < AT_ONCE; ++k) ref = fmaxf(ref, s[k][0]);
            const float f = __builtin_amdgcn_exp2f(sum.ref - ref);
            sum.ref = ref;
            sum.l *= f;
#pragma unroll
            for (int d = 0; d < ET; ++d) sum.o[d] *= f;
#pragma unroll
            for (int k = 0; k < AT_ONCE; ++k) {
                // behind the last piece nothing is added
                const float fk = c0 + k * WAVES < pc.n ? __builtin_amdgcn_exp2f(s[k][0] - ref) : 0.0f;
                sum.l = __builtin_fmaf(s[k][1], fk, sum.l);
#pragma unroll
                for (int d = 0; d < ET; ++d) sum.o[d] = __builtin_fmaf(v[k][d / 2][d % 2], fk, sum.o[d]);
            }
        }
        __syncthreads();  // the sums of the rows before are read
        if (lane % 8 == 0) {
            s_ref[wave][r] = sum.ref;
            s_l[wave][r] = sum.l;
        }
        __syncthreads();
        float ref = s_ref[0][r];
#pragma unroll
        for (int v = 1; v < WAVES; ++v) ref = fmaxf(ref, s_ref[v][r]);
        const float f = __builtin_amdgcn_exp2f(sum.ref - ref);
#pragma unroll
        for (int d = 0; d < ET; d += 4) {
            const f32x4 v = {sum.o[d] * f, sum.o[d + 1] * f, sum.o[d + 2] * f, sum.o[d + 3] * f};
            *reinterpret_cast<f32x4*>(&s_o[wave][r][e0 + d]) = v;
        }
        __syncthreads();
        if (r16 < 8 && r0 + r16 < rows)
            attend_result<PT, F16>(a, add_waves<DP, PT, WAVES>(s_o, s_ref, s_l, 0, r16, part), pc.b, h,
                                   first + r0 + r16, part, s_live[r0 + r16] != 0);
    }
}

// How many rows a workgroup takes, and into how many pieces rows are cut.
template <int DP, int MT, bool F16, int WAVES>
static hipError_t launch_attend(Kv8Attend a, hipStream_t st) {
    constexpr int64_t SLOT = MT * 16 * (DP + 2);
    a.blocks = (int)(((int64_t)a.s.N * a.group + MT * 16 - 1) / (MT * 16));
    const int64_t y = (int64_t)a.g.heads * a.blocks;
    // rows are cut where whole ones leave the card's CUs idle or uneven
    const int64_t most = KV8_PART_FLOATS / SLOT < KV8_SPLITS ? KV8_PART_FLOATS / SLOT : KV8_SPLITS;
    static const int target = getenv("AT_TARGET") ? atoi(getenv("AT_TARGET")) : 512;
    a.pieces = y * a.s.B <= most / 2 ? (int)((most / 2 < target ? most / 2 : target) / y) : 0;
    const int64_t grid = y * (a.s.B + a.pieces);
    if (grid > INT_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_attend<DP, MT, F16, WAVES>), dim3((unsigned)grid), dim3(WAVES * WAVE), 0, st, a);
    return hipGetLastError();
}

template <int DP, bool F16>
static hipError_t launch_attend_rows(const Kv8Attend& a, hipStream_t st) {
    const int64_t rows = (int64_t)a.s.N * a.group;
    if (rows <= 16) return launch_attend<DP, 1, F16, 4>(a, st);
    if (rows <= 32 || DP == 256) return launch_attend<DP, 2, F16, 4>(a, st);
    return launch_attend<DP, DP == 256 ? 2 : 4, F16, 4>(a, st);
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
