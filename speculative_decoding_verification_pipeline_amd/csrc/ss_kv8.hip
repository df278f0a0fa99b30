// Rotary positions, and a cache held in 8 bits: writing it and reading it back.
//
// A rotation turns pairs of a head's entries by their token's position: (u, v) becomes
// m (u cos a - v sin a, u sin a + v cos a), a = position * 2 pi * turns. The angle in turns
// is formed and reduced to [-1/2, 1/2] in binary64, so a far position loses nothing.
//
// An 8-bit cache holds a block of slots of one head as 8-bit floats under a power of two
// 2^x: the least with which the block's largest entry is at most 448. A power of two costs
// such a float no bit of its mantissa, and a block that grows is rounded again by a shift
// of its exponents, which loses only what falls below 2^-6.
//
// What bounds all three: HBM for prompts (each value read once and written once, 16 bytes a
// lane), latency for single tokens.
#include <limits.h>

#include "ss_device.h"
#include "ss_internal.h"
#include "ss_kv8.h"

namespace ss {

constexpr int KV_NT = 256;
constexpr int KV_UNIT = 16;         // entries of a head that a thread takes at once
constexpr int KV_UNITS = 4;         // units of a thread that stay in registers
constexpr int KV_PART_UNITS = 5;    // where a head of 256 has 17
constexpr int KV_SIN_BYTES = 32768; // sines and cosines held at once

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 h16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 b16x2 __attribute__((ext_vector_type(2)));

template <bool F16>
__device__ __forceinline__ f32x2 from16(uint32_t w) {
    if constexpr (F16) return __builtin_convertvector(__builtin_bit_cast(h16x2, w), f32x2);
    else return f32x2{__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)};
}

template <bool F16>
__device__ __forceinline__ uint32_t to16(float a, float b) {
    const f32x2 v = {a, b};
    if constexpr (F16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, h16x2));
    else return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, b16x2));
}

// Cosine and sine of a position's angle, times the magnitude.
__device__ __forceinline__ void turn(double position, double turns, double magnitude, double& c,
                                     double& s) {
    double t = position * turns;
    t -= rint(t);
    sincospi(t + t, &s, &c);
    c *= magnitude;
    s *= magnitude;
}

// Where the 16 entries of unit u of a head lie, as two runs of 8: of a rotation by halves,
// 8 first members of pairs and their seconds; else neighbours.
__device__ __forceinline__ void unit_at(const Rotary& r, bool turned, int u, int& lo, int& hi) {
    if (turned && !r.interleaved) {
        lo = u * 8;
        hi = r.dim / 2 + u * 8;
    } else {
        lo = u * KV_UNIT;
        hi = lo + 8;
    }
}

// A unit of a head whose rotated part 16 does not divide: two runs of entries, some of them
// no full 8, and the first `pairs` of lo's and hi's are pairs (of neighbours: the first
// 2 * pairs entries). By halves the pairs' units come first, the last of them short, then
// the entries behind them, which start where the rotated part ends.
struct PartUnit {
    int lo, hi, n_lo, n_hi, pairs;
};

__host__ __device__ __forceinline__ int part_units(int dim, int rot, bool interleaved) {
    return interleaved ? dim / KV_UNIT : (rot / 2 + 7) / 8 + (dim - rot + KV_UNIT - 1) / KV_UNIT;
}

__device__ __forceinline__ PartUnit part_unit(const Rotary& r, int dim, int u) {
    const int half = r.dim / 2, turned = (half + 7) / 8;
    if (r.interleaved) return {u * KV_UNIT, u * KV_UNIT + 8, 8, 8, min(max(half - u * 8, 0), 8)};
    if (u < turned) {
        const int n = min(half - u * 8, 8);
        return {u * 8, half + u * 8, n, n, n};
    }
    const int lo = r.dim + (u - turned) * KV_UNIT, hi = min(lo + 8, dim);
    return {lo, hi, hi - lo, min(dim - hi, 8), 0};
}

// A run of n <= 8 values, four at a time where `fours` says that all runs start and end at
// multiples of four, else one by one; those behind n are 0.
template <bool F16>
__device__ __forceinline__ void load_run(const uint16_t* from, int n, bool fours, float* x) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        u32x2 w = {0, 0};
        if (fours) {
            if (i < n) w = *reinterpret_cast<const u32x2*>(from + i);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + k < n) w[k / 2] |= (uint32_t)from[i + k] << (k % 2 * 16);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const f32x2 v = from16<F16>(w[k]);
            x[i + 2 * k] = v[0];
            x[i + 2 * k + 1] = v[1];
        }
    }
}

template <bool F16>
__device__ __forceinline__ void store_run(uint16_t* to, int n, bool fours, const float* x) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        const u32x2 w = {to16<F16>(x[i], x[i + 1]), to16<F16>(x[i + 2], x[i + 3])};
        if (fours) {
            if (i < n) *reinterpret_cast<u32x2*>(to + i) = w;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + k < n) to[i + k] = (uint16_t)(w[k / 2] >> (k % 2 * 16));
        }
    }
}

// The same of bytes, by words of four.
__device__ __forceinline__ void store_run8(char* to, int n, bool fours, uint32_t w0, uint32_t w1) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        const uint32_t w = i ? w1 : w0;
        if (fours) {
            if (i < n) *reinterpret_cast<uint32_t*>(to + i) = w;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + k < n) to[i + k] = (char)(w >> (k * 8));
        }
    }
}

// Turns a unit's 16 values by its 8 pairs' cosines and sines, or the first `pairs` of them.
template <class T>
__device__ __forceinline__ void turn_unit(bool interleaved, const T* c, const T* s, T x[16], int pairs = 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i >= pairs) break;
        const int p = interleaved ? 2 * i : i, q = interleaved ? 2 * i + 1 : i + 8;
        const T u = x[p], v = x[q];
        x[p] = fma(u, c[i], -(v * s[i]));
        x[q] = fma(u, s[i], v * c[i]);
    }
}

// ---------------------------------------------------------------------------
// rotation alone

// A workgroup takes `tokens` tokens and finds their sines once; then a thread takes units
// of all heads, queries' and keys' side by side. 4096 tokens of 40 heads of 128: 15.7 us, 5.3
// TB/s (HBM); one token 2.7 us, a chain of loads and the sines.
template <bool F16>
__global__ __launch_bounds__(KV_NT) void k_rotate(RotateArgs a, int tokens, int units) {
    extern __shared__ float s_turn[];  // [tokens][cosines, sines][dim / 2]
    const int tid = threadIdx.x;
    const int half = a.r.dim / 2;
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int64_t all = (int64_t)a.B * a.N;
    const int n = (int)min((int64_t)tokens, all - t0);
    const int per_head = a.head_dim / KV_UNIT;
    const int per_token = units * per_head;
    const int h0 = blockIdx.y * units;  // heads of this workgroup
    const int heads = min(a.q_heads + a.k_heads - h0, units);
    for (int i = tid; i < n * half; i += KV_NT) {
        const int t = i / half, f = i - t * half;
        double c, s;
        turn((double)a.positions[t0 + t], a.r.turns[f], a.r.magnitude, c, s);
        s_turn[t * a.r.dim + f] = (float)c;
        s_turn[t * a.r.dim + half + f] = (float)s;
    }
    __syncthreads();
    for (int i = tid; i < n * per_token; i += KV_NT) {
        const int t = i / per_token, j = i - t * per_token;
        const int hh = j / per_head, u = j - hh * per_head;
        if (hh >= heads) continue;
        const bool keys = h0 + hh >= a.q_heads;
        const int h = keys ? h0 + hh - a.q_heads : h0 + hh;
        const Heads& from = keys ? a.k : a.q;
        const Heads& to = keys ? a.k_out : a.q_out;
        const int b = (int)((t0 + t) / a.N), tok = (int)((t0 + t) - (int64_t)b * a.N);
        const bool turned = u * KV_UNIT < a.r.dim;
        int lo, hi;
        unit_at(a.r, turned, u, lo, hi);
        const uint16_t* p = from.data + b * from.row + tok * from.token + h * from.head;
        uint16_t* q = to.data + b * to.row + tok * to.token + h * to.head;
        const u32x4 w0 = *reinterpret_cast<const u32x4*>(p + lo), w1 = *reinterpret_cast<const u32x4*>(p + hi);
        u32x4 r0 = w0, r1 = w1;
        if (turned) {
            float x[16], c[8], s[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const f32x2 v0 = from16<F16>(w0[k]), v1 = from16<F16>(w1[k]);
                x[2 * k] = v0[0];
                x[2 * k + 1] = v0[1];
                x[8 + 2 * k] = v1[0];
                x[9 + 2 * k] = v1[1];
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                c[k] = s_turn[t * a.r.dim + u * 8 + k];
                s[k] = s_turn[t * a.r.dim + half + u * 8 + k];
            }
            turn_unit<float>(a.r.interleaved, c, s, x);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                r0[k] = to16<F16>(x[2 * k], x[2 * k + 1]);
                r1[k] = to16<F16>(x[8 + 2 * k], x[9 + 2 * k]);
            }
        }
        *reinterpret_cast<u32x4*>(q + lo) = r0;
        *reinterpret_cast<u32x4*>(q + hi) = r1;
    }
}

// The same for any sizes, strides and alignment: a thread takes one pair of a token, or one
// entry behind them, over all heads, 2 bytes at a time. 4096 tokens of 40 heads of 80, 20 of
// them turned: 33 us (11.9 turned whole, by the kernel above; its bytes take 10.7); one token
// 15 us, its heads one after the other.
template <bool F16>
__global__ __launch_bounds__(KV_NT) void k_rotate_any(RotateArgs a) {
    const int half = a.r.dim / 2;
    const int per_token = half + a.head_dim - a.r.dim;
    const int64_t i = (int64_t)blockIdx.x * KV_NT + threadIdx.x;
    if (i >= (int64_t)a.B * a.N * per_token) return;
    const int64_t t = i / per_token;
    const int f = (int)(i - t * per_token);
    const int b = (int)(t / a.N), tok = (int)(t - (int64_t)b * a.N);
    const bool pair = f < half;
    const int lo = !pair ? f + half : a.r.interleaved ? 2 * f : f;
    const int hi = a.r.interleaved ? lo + 1 : lo + half;
    double cd = 0, sd = 0;
    if (pair) turn((double)a.positions[t], a.r.turns[f], a.r.magnitude, cd, sd);
    const float c = (float)cd, s = (float)sd;
    for (int hh = 0; hh < a.q_heads + a.k_heads; ++hh) {
        const bool keys = hh >= a.q_heads;
        const int h = keys ? hh - a.q_heads : hh;
        const Heads& from = keys ? a.k : a.q;
        const Heads& to = keys ? a.k_out : a.q_out;
        const uint16_t* p = from.data + b * from.row + tok * from.token + h * from.head;
        uint16_t* q = to.data + b * to.row + tok * to.token + h * to.head;
        if (!pair) {
            q[lo] = p[lo];
            continue;
        }
        const f32x2 v = from16<F16>((uint32_t)p[lo] | (uint32_t)p[hi] << 16);
        const uint32_t r = to16<F16>(__builtin_fmaf(v[0], c, -(v[1] * s)), __builtin_fmaf(v[0], s, v[1] * c));
        q[lo] = (uint16_t)r;
        q[hi] = (uint16_t)(r >> 16);
    }
}

// ---------------------------------------------------------------------------
// writing

struct StepRow {
    int64_t base;
    int count;
};

__device__ __forceinline__ StepRow step_row(const Kv8Geo& g, const Kv8Step& s, int b) {
    StepRow r;
    r.base = s.base[b];
    r.count = s.counts ? min(max(s.counts[b], 0), s.N) : s.N;
    if (r.base < 0 || r.base > (int64_t)g.max_blocks * g.page_size || (s.reserved && s.reserved[b] == 0)) {
        r.base = 0;
        r.count = 0;
    }
    return r;
}

// The nearest binary32 towards 0, its last bit set where bits were lost: what is rounded
// from it to fewer bits is as if rounded from the binary64.
__device__ __forceinline__ float to_odd(double d) {
    const float f = (float)d;
    uint32_t b = __float_as_uint(f);
    if ((double)f != d && !(b & 1)) b += fabs((double)f) > fabs(d) ? -1 : 1;
    return __uint_as_float(b);
}

// The least whole x with amax <= 448 * 2^x = 1.75 * 2^(x + 8), within the scale's range.
__device__ __forceinline__ int scale_of(uint32_t amax) {
    const int e = (int)(amax >> 23) - 127;
    const int x = e - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(x, KV8_XMIN), KV8_XMAX);
}

// Four values under 2^-x as 8-bit floats: beyond 448 the largest, infinities a NaN.
__device__ __forceinline__ uint32_t to8(const float* x, float f) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = x[i] * f;
        v[i] = v[i] > 448.0f ? 448.0f : v[i] < -448.0f ? -448.0f : v[i];
        if ((__float_as_uint(x[i]) & 0x7f800000u) == 0x7f800000u) v[i] = NAN;
    }
    uint32_t w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    return __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], w, true);
}

struct WritePlan {
    int units;        // of a turned head
    int blocks;       // of a row's slots that a step can touch
    int heads;        // of the cache that a workgroup takes
    int parts;        // workgroups for the heads of a block
    int q_tokens;     // that a workgroup turns
    int q_chunks;
};

// Grid (plan, B): for each block of slots its keys' parts, its values' parts, then the
// queries. A workgroup holds its block's values, up to 16384, in registers: it finds the
// largest, then the scale, and writes. Two uneven prompts of 3000 tokens on average, 32 query
// heads and 8 of the cache: 36 to 40 us, 3.5 TB/s, where the rotation alone reaches 5.3: the
// queries' loads are issued behind binary64 sines and a barrier. One token 6 us, 48 trees of 16
// nodes 11.4, chains of loads, the tree's depths and the sines.
// PART: 16 does not divide the rotated part. Of a rotation by halves the runs of a unit then
// start where no 16 bytes do, and are read and written 8 (keys in 8 bits 4) at a time where
// pairs come in fours, else entry by entry; still a unit's thread reads what it writes, so
// queries may be turned where they lie. Two prompts of 3000 tokens on average, 32 query heads
// and 8 of the cache of 80, written and their ends read: 38 us turned whole, 43 turned by halves
// in 40 entries (38 in neighbours), 86 in 20, entry by entry.
template <bool F16, bool PART>
__global__ __launch_bounds__(KV_NT) void k_kv8_write(Kv8Write a, WritePlan p) {
    constexpr int UNITS = PART ? KV_PART_UNITS : KV_UNITS;
    __shared__ __align__(16) char s_mem[KV_SIN_BYTES];
    __shared__ uint32_t s_amax[64];
    __shared__ int s_depth[WAVE];
    const int tid = threadIdx.x;
    const int b = blockIdx.y;
    const int half = a.r.turns ? a.r.dim / 2 : 0;
    const StepRow row = step_row(a.g, a.s, b);
    const int kv = p.blocks * p.parts;
    const bool keys = (int)blockIdx.x < kv;
    const bool queries = (int)blockIdx.x >= 2 * kv;
    if (a.r.turns && a.s.parents && !a.positions && (keys || queries)) {
        const TreeNode t = tree_node(a.s.parents + (int64_t)b * a.s.N, a.s.N);
        if (tid < WAVE) s_depth[tid] = t.depth;
        __syncthreads();
    }
    auto position = [&](int i) -> double {
        if (a.positions) return (double)a.positions[(int64_t)b * a.s.N + i];
        return (double)(row.base + (a.s.parents ? s_depth[i] : i));
    };
    const bool in_runs = PART && !a.r.interleaved, fours = half % 4 == 0;

    if (queries) {
        const int per_head = p.units;
        float* turns = reinterpret_cast<float*>(s_mem);
        const int i0 = ((int)blockIdx.x - 2 * kv) * p.q_tokens;
        const int n = min(p.q_tokens, a.s.N - i0);
        const int live = min(max(row.count - i0, 0), n);
        for (int i = tid; i < live * half; i += KV_NT) {
            const int t = i / half, f = i - t * half;
            double c, s;
            turn(position(i0 + t), a.r.turns[f], a.r.magnitude, c, s);
            turns[t * a.r.dim + f] = (float)c;
            turns[t * a.r.dim + half + f] = (float)s;
        }
        __syncthreads();
        const int per_token = a.q_heads * per_head;
        for (int i = tid; i < n * per_token; i += KV_NT) {
            const int t = i / per_token, j = i - t * per_token;
            const int h = j / per_head, u = j - h * per_head;
            const uint16_t* from = a.q.data + b * a.q.row + (i0 + t) * a.q.token + h * a.q.head;
            uint16_t* to = a.q_out.data + b * a.q_out.row + (i0 + t) * a.q_out.token + h * a.q_out.head;
            int pairs = u * KV_UNIT < a.r.dim ? 8 : 0;
            if constexpr (PART) {
                const PartUnit at = part_unit(a.r, a.g.dim, u);
                pairs = at.pairs;
                if (in_runs) {
                    float x[16] = {}, c[8], s[8];
                    if (t < live) {
                        load_run<F16>(from + at.lo, at.n_lo, fours, x);
                        load_run<F16>(from + at.hi, at.n_hi, fours, x + 8);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            c[k] = k < pairs ? turns[t * a.r.dim + u * 8 + k] : 0.0f;
                            s[k] = k < pairs ? turns[t * a.r.dim + half + u * 8 + k] : 0.0f;
                        }
                        turn_unit<float>(false, c, s, x, pairs);
                    }
                    store_run<F16>(to + at.lo, at.n_lo, fours, x);
                    store_run<F16>(to + at.hi, at.n_hi, fours, x + 8);
                    continue;
                }
            }
            int lo, hi;
            unit_at(a.r, pairs != 0, u, lo, hi);
            u32x4 r0 = {0, 0, 0, 0}, r1 = {0, 0, 0, 0};
            if (t < live) {
                r0 = *reinterpret_cast<const u32x4*>(from + lo);
                r1 = *reinterpret_cast<const u32x4*>(from + hi);
                if (pairs) {
                    float x[16], c[8], s[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const f32x2 v0 = from16<F16>(r0[k]), v1 = from16<F16>(r1[k]);
                        x[2 * k] = v0[0];
                        x[2 * k + 1] = v0[1];
                        x[8 + 2 * k] = v1[0];
                        x[9 + 2 * k] = v1[1];
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const bool on = !PART || k < pairs;
                        c[k] = on ? turns[t * a.r.dim + u * 8 + k] : 0.0f;
                        s[k] = on ? turns[t * a.r.dim + half + u * 8 + k] : 0.0f;
                    }
                    turn_unit<float>(a.r.interleaved, c, s, x, PART ? pairs : 8);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        r0[k] = to16<F16>(x[2 * k], x[2 * k + 1]);
                        r1[k] = to16<F16>(x[8 + 2 * k], x[9 + 2 * k]);
                    }
                }
            }
            *reinterpret_cast<u32x4*>(to + lo) = r0;
            *reinterpret_cast<u32x4*>(to + hi) = r1;
        }
        return;
    }

    // the block's slots that this step writes
    const int task = keys ? blockIdx.x : (int)blockIdx.x - kv;
    const int jb = task / p.parts, h0 = (task - jb * p.parts) * p.heads;
    const int heads = min(p.heads, a.g.heads - h0);
    const int64_t j0 = (row.base / a.g.block + jb) * a.g.block;  // the block's first slot
    const int64_t end = min(row.base + row.count, (int64_t)a.g.max_blocks * a.g.page_size);
    const int lo_t = (int)max(row.base - j0, (int64_t)0);  // below the block's size
    const int hi_t = (int)max(min(end - j0, (int64_t)a.g.block), (int64_t)0);
    if (lo_t >= hi_t) return;
    const int page = a.s.t.tables[b * a.s.t.stride + j0 / a.g.page_size];
    if ((unsigned)page >= (unsigned)a.g.num_pages) return;
    if (a.s.t.ref[page] > 1) return;
    const int slot0 = (int)(j0 % a.g.page_size);
    const Kv8Plane plane = keys ? a.k : a.v;
    const Heads& src = keys ? a.keys : a.values;
    char* to = plane.data + page * a.g.page + slot0 * a.g.slot;
    uint8_t* scales = plane.scales + page * a.g.sc_page + slot0 / a.g.block * a.g.sc_block;
    if (tid < heads) s_amax[tid] = 0;

    const bool turns = keys && a.r.turns;
    const bool runs = in_runs && keys;  // PART: there is a rotation
    const int per_head = turns ? p.units : a.g.dim / KV_UNIT;
    const int per_slot = heads * per_head;
    const int tokens = hi_t - lo_t;
    const int total = tokens * per_slot;
    const int i0 = (int)(j0 + lo_t - row.base);  // the step's token in slot lo_t
    u32x4 w[UNITS][2];
    float x[UNITS][16];
    int tok[UNITS], hd[UNITS], un[UNITS];
#pragma unroll
    for (int k = 0; k < UNITS; ++k) {
        const int i = tid + k * KV_NT;
        tok[k] = i / per_slot;
        const int j = i - tok[k] * per_slot;
        hd[k] = j / per_head;
        un[k] = j - hd[k] * per_head;
        if (i < total) {
            const uint16_t* from = src.data + b * src.row + (i0 + tok[k]) * src.token +
                                   (h0 + hd[k]) * src.head;
            if constexpr (PART) {
                if (runs) {
                    const PartUnit at = part_unit(a.r, a.g.dim, un[k]);
                    load_run<F16>(from + at.lo, at.n_lo, fours, x[k]);
                    load_run<F16>(from + at.hi, at.n_hi, fours, x[k] + 8);
                    continue;
                }
            }
            int lo, hi;
            unit_at(a.r, turns && un[k] * KV_UNIT < a.r.dim, un[k], lo, hi);
            w[k][0] = *reinterpret_cast<const u32x4*>(from + lo);
            w[k][1] = *reinterpret_cast<const u32x4*>(from + hi);
        } else {
            tok[k] = INT_MAX;
        }
    }
#pragma unroll
    for (int k = 0; k < UNITS; ++k) {
        if (PART && runs) continue;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const f32x2 v0 = from16<F16>(w[k][0][c]), v1 = from16<F16>(w[k][1][c]);
            x[k][2 * c] = v0[0];
            x[k][2 * c + 1] = v0[1];
            x[k][8 + 2 * c] = v1[0];
            x[k][9 + 2 * c] = v1[1];
        }
    }
    if (turns) {
        double* s_turn = reinterpret_cast<double*>(s_mem);
        const int most = KV_SIN_BYTES / 8 / a.r.dim;  // tokens whose sines are held at once
        for (int t0 = 0; t0 < tokens; t0 += most) {
            const int n = min(most, tokens - t0);
            __syncthreads();
            for (int i = tid; i < n * half; i += KV_NT) {
                const int t = i / half, f = i - t * half;
                double c, s;
                turn(position(i0 + t0 + t), a.r.turns[f], a.r.magnitude, c, s);
                s_turn[t * a.r.dim + f] = c;
                s_turn[t * a.r.dim + half + f] = s;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < UNITS; ++k) {
                int pairs = un[k] * KV_UNIT < a.r.dim ? 8 : 0;
                if constexpr (PART) pairs = part_unit(a.r, a.g.dim, un[k]).pairs;
                if (tok[k] < t0 || tok[k] >= t0 + n || !pairs) continue;
                const double* at = s_turn + (tok[k] - t0) * a.r.dim + un[k] * 8;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (PART && i >= pairs) break;
                    const double c = at[i], s = at[half + i];
                    const int p0 = i, q0 = i + 8, p1 = 2 * i, q1 = 2 * i + 1;
                    if (a.r.interleaved) {
                        const double u = x[k][p1], v = x[k][q1];
                        x[k][p1] = to_odd(fma(u, c, -(v * s)));
                        x[k][q1] = to_odd(fma(u, s, v * c));
                    } else {
                        const double u = x[k][p0], v = x[k][q0];
                        x[k][p0] = to_odd(fma(u, c, -(v * s)));
                        x[k][q0] = to_odd(fma(u, s, v * c));
                    }
                }
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < UNITS; ++k) {
        if (tok[k] == INT_MAX) continue;
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t bits = __float_as_uint(x[k][i]) & 0x7fffffffu;
            most = max(most, bits < 0x7f800000u ? bits : 0u);
        }
        atomicMax(&s_amax[hd[k]], most);
    }
    __syncthreads();
    // slots that the block holds before the step's: the scale may grow, never shrink
#pragma unroll
    for (int k = 0; k < UNITS; ++k) {
        if (tok[k] == INT_MAX) continue;
        int e = scale_of(s_amax[hd[k]]);
        if (lo_t > 0) e = max(e, (int)scales[(h0 + hd[k]) * a.g.sc_head] - 127);
        e = min(max(e, KV8_XMIN), KV8_XMAX);
        const float f = __uint_as_float((uint32_t)(127 - e) << 23);
        char* at = to + (lo_t + tok[k]) * a.g.slot + (h0 + hd[k]) * a.g.head;
        const u32x2 v0 = {to8(x[k], f), to8(x[k] + 4, f)}, v1 = {to8(x[k] + 8, f), to8(x[k] + 12, f)};
        if constexpr (PART) {
            if (runs) {
                const PartUnit u = part_unit(a.r, a.g.dim, un[k]);
                store_run8(at + u.lo, u.n_lo, fours, v0[0], v0[1]);
                store_run8(at + u.hi, u.n_hi, fours, v1[0], v1[1]);
                continue;
            }
        }
        int lo, hi;
        unit_at(a.r, turns && un[k] * KV_UNIT < a.r.dim, un[k], lo, hi);
        *reinterpret_cast<u32x2*>(at + lo) = v0;
        *reinterpret_cast<u32x2*>(at + hi) = v1;
    }
    const int held_head = a.g.dim / KV_UNIT, held_slot = heads * held_head;
    for (int i = tid; i < lo_t * held_slot; i += KV_NT) {
        const int t = i / held_slot, j = i - t * held_slot;
        const int h = j / held_head, u = j - h * held_head;
        const int was = (int)scales[(h0 + h) * a.g.sc_head] - 127;
        const int e = scale_of(s_amax[h]);
        if (e <= was) continue;
        u32x4* at = reinterpret_cast<u32x4*>(to + t * a.g.slot + (h0 + h) * a.g.head + u * KV_UNIT);
        *at = kv8_shift(*at, was - e);
    }
    __syncthreads();  // every thread has its block's old scales
    if (tid < heads) {
        uint8_t* at = scales + (h0 + tid) * a.g.sc_head;
        int e = scale_of(s_amax[tid]);
        if (lo_t > 0) e = max(e, (int)*at - 127);
        *at = (uint8_t)(min(max(e, KV8_XMIN), KV8_XMAX) + 127);
    }
}

// ---------------------------------------------------------------------------
// reading

// Grid (units of a row's slots, B, planes): 16 bytes a thread. 8000 slots of 8 heads of 128 to
// bfloat16: 11 us, 4.5 TB/s (HBM).
template <bool F16>
__global__ __launch_bounds__(KV_NT) void k_kv8_read(Kv8Read a) {
    const int b = blockIdx.y, z = blockIdx.z;
    const int per_head = a.g.dim / KV_UNIT;
    const int per_slot = a.g.heads * per_head;
    const int64_t i = (int64_t)blockIdx.x * KV_NT + threadIdx.x;
    const int n = (int)(i / per_slot);
    if (n >= a.N) return;
    const int j = (int)(i - (int64_t)n * per_slot);
    const int h = j / per_head, u = j - h * per_head;
    const int count = a.counts ? a.counts[b] : a.N;
    const int64_t slot = (a.start ? (int64_t)a.start[b] : 0) + n;
    u32x4 r[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    if (n < count && slot >= 0 && slot < (int64_t)a.g.max_blocks * a.g.page_size) {
        const unsigned block = (unsigned)slot / (unsigned)a.g.page_size;
        const int in = (int)((unsigned)slot - block * (unsigned)a.g.page_size);
        const int page = a.t.tables[b * a.t.stride + block];
        if ((unsigned)page < (unsigned)a.g.num_pages) {
            const u32x4 w = *reinterpret_cast<const u32x4*>(a.p[z].data + page * a.g.page + in * a.g.slot +
                                                            h * a.g.head + u * KV_UNIT);
            const int s = a.p[z].scales[page * a.g.sc_page + in / a.g.block * a.g.sc_block + h * a.g.sc_head];
            const float f = __uint_as_float((uint32_t)min(max(s, 127 + KV8_XMIN), 127 + KV8_XMAX) << 23);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const f32x2 v0 = __builtin_amdgcn_cvt_pk_f32_fp8(w[k], false);
                const f32x2 v1 = __builtin_amdgcn_cvt_pk_f32_fp8(w[k], true);
                r[k / 2][k % 2 * 2] = to16<F16>(v0[0] * f, v0[1] * f);
                r[k / 2][k % 2 * 2 + 1] = to16<F16>(v1[0] * f, v1[1] * f);
            }
        }
    }
    uint16_t* to = a.out[z].data + b * a.out[z].row + n * a.out[z].token + h * a.out[z].head + u * KV_UNIT;
    reinterpret_cast<u32x4*>(to)[0] = r[0];
    reinterpret_cast<u32x4*>(to)[1] = r[1];
}

// ---------------------------------------------------------------------------

hipError_t launch_rotate(const RotateArgs& a, ss_dtype dt, hipStream_t st) {
    const int64_t all = (int64_t)a.B * a.N;
    if (!a.vectors) {
        const int64_t n = all * (a.head_dim - a.r.dim / 2);
        const int64_t grid = (n + KV_NT - 1) / KV_NT;
        if (grid > INT_MAX) return hipErrorInvalidValue;
        if (dt == SS_F16) hipLaunchKernelGGL(k_rotate_any<true>, dim3((unsigned)grid), dim3(KV_NT), 0, st, a);
        else hipLaunchKernelGGL(k_rotate_any<false>, dim3((unsigned)grid), dim3(KV_NT), 0, st, a);
        return hipGetLastError();
    }
    // four units a thread where there are tokens enough for the card, else one
    const int heads = a.q_heads + a.k_heads;
    const int64_t per_token = (int64_t)heads * (a.head_dim / KV_UNIT);
    int tokens = 1;
    while (tokens < 8 && per_token * tokens * 2 <= 4 * KV_NT && all >= (int64_t)tokens * 2 * 512) tokens *= 2;
    int units = heads;  // heads of a workgroup
    if (all < 512) units = KV_NT / (a.head_dim / KV_UNIT);
    if (units > heads) units = heads;
    if (units < 1) units = 1;
    const dim3 grid((unsigned)((all + tokens - 1) / tokens), (unsigned)((heads + units - 1) / units));
    const size_t lds = (size_t)tokens * a.r.dim * sizeof(float);
    if (dt == SS_F16) hipLaunchKernelGGL(k_rotate<true>, grid, dim3(KV_NT), lds, st, a, tokens, units);
    else hipLaunchKernelGGL(k_rotate<false>, grid, dim3(KV_NT), lds, st, a, tokens, units);
    return hipGetLastError();
}

hipError_t launch_kv8_write(const Kv8Write& a, ss_dtype dt, hipStream_t st) {
    const bool part = a.r.turns && a.r.dim % KV_UNIT;
    const int per_head = part ? part_units(a.g.dim, a.r.dim, a.r.interleaved) : a.g.dim / KV_UNIT;
    WritePlan p;
    p.units = per_head;
    p.blocks = (int)(((int64_t)a.g.block + a.s.N - 2) / a.g.block) + 1;
    // at least 1: block <= 64, dim <= 256, so 16 units a head, 17 where a part's last one is short
    p.heads = (part ? KV_PART_UNITS : KV_UNITS) * KV_NT / (a.g.block * per_head);
    if (p.heads > a.g.heads) p.heads = a.g.heads;
    if (p.heads > 64) p.heads = 64;
    p.parts = (a.g.heads + p.heads - 1) / p.heads;
    p.q_tokens = p.q_chunks = 0;
    if (a.q_heads) {
        p.q_tokens = 4 * KV_NT / (a.q_heads * per_head);
        if (p.q_tokens > 16) p.q_tokens = 16;
        if (p.q_tokens < 1) p.q_tokens = 1;
        p.q_chunks = (a.s.N + p.q_tokens - 1) / p.q_tokens;
    }
    const int64_t grid = 2ll * p.blocks * p.parts + p.q_chunks;
    if (grid > INT_MAX) return hipErrorInvalidValue;
    const dim3 g((unsigned)grid, a.s.B);
    if (dt == SS_F16 && part) hipLaunchKernelGGL((k_kv8_write<true, true>), g, dim3(KV_NT), 0, st, a, p);
    else if (part) hipLaunchKernelGGL((k_kv8_write<false, true>), g, dim3(KV_NT), 0, st, a, p);
    else if (dt == SS_F16) hipLaunchKernelGGL((k_kv8_write<true, false>), g, dim3(KV_NT), 0, st, a, p);
    else hipLaunchKernelGGL((k_kv8_write<false, false>), g, dim3(KV_NT), 0, st, a, p);
    return hipGetLastError();
}

hipError_t launch_kv8_read(const Kv8Read& a, ss_dtype dt, hipStream_t st) {
    const int64_t n = (int64_t)a.N * a.g.heads * (a.g.dim / KV_UNIT);
    const int64_t grid = (n + KV_NT - 1) / KV_NT;
    if (grid > INT_MAX) return hipErrorInvalidValue;
    const dim3 g((unsigned)grid, a.B, a.planes);
    if (dt == SS_F16) hipLaunchKernelGGL(k_kv8_read<true>, g, dim3(KV_NT), 0, st, a);
    else hipLaunchKernelGGL(k_kv8_read<false>, g, dim3(KV_NT), 0, st, a);
    return hipGetLastError();
}

}  // namespace ss
