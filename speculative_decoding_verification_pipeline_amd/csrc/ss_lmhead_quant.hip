// LM-head logits from 4-bit weights with group scales (gfx950 bf16 MFMA).
//
//   y[b, v] = sum_g s[v, g] ( sum_{k in g} (n[v, k] - z[v, g]) x[b, k] )
//
// What bounds it: the weight stream (V K / 2 bytes) while the rows are few, and
// beside it the vector ALU that widens nibbles for the matrix cores.
//
//  * Widening costs one operation per weight: a nibble shifted into the top of
//    a bfloat16 mantissa under the exponent of 16 is the number 16 + n exactly,
//    two at a time (nibbles j and j + 4 of a word share the mask), and no
//    product is rounded: the matrix cores multiply by 16 + n, and the group's
//    accumulators start from -(16 + z) sum_k x[b, k] instead of 0. Scales are
//    applied to the finished group in binary32. (Widening to s (n - z) would
//    round every weight to 8 bits.)
//  * v_mfma_f32_16x16x32_bf16, W as the A operand: a wave owns RT tiles of 16
//    vocabulary rows and NT tiles of 16 batch rows; widened weights are used NT
//    times. Weights go from memory straight to the registers of the one wave
//    that uses them: a lane loads 16 bytes (32 weights) of its row at a time,
//    one chunk ahead.
//  * Any assignment of k to MFMA slots is right as long as both operands share
//    it. A lane's four words serve four MFMAs; for groups of 128 as they are,
//    for groups of 64 and 32 after exchanging words between the lanes that hold
//    the same row (permlane swaps), so that no MFMA crosses a group.
//  * x is staged in LDS once per workgroup and chunk, in the order in which the
//    MFMAs read it (each operand read is 1 KB of consecutive LDS), with the
//    sums over each group.
//  * 8 waves: RW row blocks by KW splits of K. The splits are added in a fixed
//    order through LDS.
#include "ss_device.h"
#include "ss_internal.h"

namespace ss {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float floatx4u __attribute__((ext_vector_type(4), aligned(4)));

constexpr int LQ_NT = 512;
constexpr int LQ_WAVES = LQ_NT / WAVE;
constexpr int LQ_KB = 128;      // k per block: one 16-byte load per lane and row tile
constexpr int LQ_STEP = 4;      // blocks per wave and chunk

// Half-word masks and the exponent of 16 in bfloat16.
constexpr uint32_t LQ_MASK = 0x00780078u;
constexpr uint32_t LQ_BASE = 0x41804180u;

// Word of eight nibbles -> eight bfloat16 16 + n, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ bf16x8 lq_widen(uint32_t w) {
    u32x4 r;
    r[0] = ((w << 3) & LQ_MASK) | LQ_BASE;
    r[1] = ((w >> 1) & LQ_MASK) | LQ_BASE;
    r[2] = ((w >> 5) & LQ_MASK) | LQ_BASE;
    r[3] = ((w >> 9) & LQ_MASK) | LQ_BASE;
    return __builtin_bit_cast(bf16x8, r);
}

// The same order for eight consecutive bfloat16 of x.
__device__ __forceinline__ u32x4 lq_order(u32x4 x) {
    u32x4 r;
    r[0] = (x[0] & 0xFFFFu) | (x[2] << 16);
    r[1] = (x[0] >> 16) | (x[2] & 0xFFFF0000u);
    r[2] = (x[1] & 0xFFFFu) | (x[3] << 16);
    r[3] = (x[1] >> 16) | (x[3] & 0xFFFF0000u);
    return r;
}

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
__device__ __forceinline__ void lq_regroup(u32x4& w) {
    uint32_t a = w[0], b = w[1], c = w[2], d = w[3];
    if (GROUP <= 64) {
        lq_swap32(a, c);
        lq_swap32(b, d);
    }
    if (GROUP <= 32) {
        lq_swap16(a, b);
        lq_swap16(c, d);
    }
    w[0] = a;
    w[1] = b;
    w[2] = c;
    w[3] = d;
}

// Where the unit e (eight k) of a block lies after lq_regroup: MFMA * 4 + lane quarter.
template <int GROUP>
__device__ __forceinline__ int lq_slot(int e) {
    if (GROUP == 32) return e;                                  // MFMA e / 4, quarter e % 4
    if (GROUP == 64) {
        const int t = (e & 7) >> 1;                             // 16 k each: quarters 0 2 1 3
        return ((e >> 3) * 2 + (e & 1)) * 4 + ((t & 1) << 1 | t >> 1);
    }
    return (e & 3) * 4 + (e >> 2);                              // MFMA e % 4, quarter e / 4
}

__device__ __forceinline__ float lq_scale(uint16_t bits, int f16) {
    return f16 ? (float)__builtin_bit_cast(_Float16, bits) : __uint_as_float((uint32_t)bits << 16);
}

template <int GROUP, int NT, int RT, int KW>
__global__ __launch_bounds__(LQ_NT) void k_lmhead_quant(QuantArgs a) {
    constexpr int RW = LQ_WAVES / KW;
    constexpr int ROWS = RW * RT * 16;           // vocabulary rows per workgroup
    constexpr int CB = LQ_STEP * KW;             // blocks per chunk
    constexpr int GPB = LQ_KB / GROUP;           // groups per block
    constexpr int MPG = 4 / GPB;                 // MFMAs per group
    __shared__ __attribute__((aligned(16))) u32x4 s_x[CB * 4 * NT * WAVE];
    __shared__ float s_sum[CB * GPB * NT * 16];
    __shared__ __attribute__((aligned(16))) float s_scale[CB * GPB * ROWS];
    __shared__ __attribute__((aligned(16))) float s_zero[CB * GPB * ROWS];
    const int tid = threadIdx.x;
    const int lane = tid & (WAVE - 1);
    const int wave = tid / WAVE;
    const int rw = wave % RW, kw = wave / RW;
    const int r16 = lane & 15, quarter = lane >> 4;
    const int K = a.K, V = a.V;
    const int row0 = blockIdx.x * ROWS + rw * RT * 16;
    const int nb = (K + LQ_KB - 1) / LQ_KB;
    const int n_groups = (K + GROUP - 1) / GROUP;

    const uint8_t* wrow[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t)
        wrow[t] = a.qweight + (int64_t)min(row0 + t * 16 + r16, V - 1) * (K / 2) + quarter * 16;
    // block j of this wave's share of the chunk that starts at block c0
    auto load_w = [&](int c0, u32x4 w[RT][LQ_STEP]) {
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int j = 0; j < LQ_STEP; ++j) {
                const int kb = c0 + kw * LQ_STEP + j;
                u32x4 v = {0u, 0u, 0u, 0u};
                if (kb * LQ_KB + quarter * 32 < K)
                    v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(wrow[t] + kb * (LQ_KB / 2)));
                w[t][j] = v;
            }
    };

    floatx4 out[RT][NT];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n) out[t][n] = floatx4{0.f, 0.f, 0.f, 0.f};

    u32x4 w[RT][LQ_STEP];
    load_w(0, w);
    for (int c0 = 0; c0 < nb; c0 += CB) {
        __syncthreads();
        // x: a thread takes 32 k of one batch row (a wave: 16 rows, one block)
        for (int i = wave; i < CB * NT; i += LQ_WAVES) {
            const int kb = i / NT, nt = i % NT;
            const int b = nt * 16 + r16;
            const int k0 = (c0 + kb) * LQ_KB + quarter * 32;
            u32x4 v[4];
            const bool on = b < a.B && k0 < K;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = on ? *reinterpret_cast<const u32x4*>(a.hidden + (int64_t)b * K + k0 + e * 8)
                          : u32x4{0u, 0u, 0u, 0u};
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    s += __uint_as_float(v[e][q] << 16) + __uint_as_float(v[e][q] & 0xFFFF0000u);
                const int slot = lq_slot<GROUP>(quarter * 4 + e);
                s_x[((kb * 4 + (slot >> 2)) * NT + nt) * WAVE + (slot & 3) * 16 + r16] = lq_order(v[e]);
            }
            if (GROUP >= 64) s += __shfl_xor(s, 16);
            if (GROUP >= 128) s += __shfl_xor(s, 32);
            if ((quarter & (GROUP / 32 - 1)) == 0)
                s_sum[((kb * GPB + quarter / (GROUP / 32)) * NT + nt) * 16 + r16] = s;
        }
        // scales and zero points of the workgroup's rows, the chunk's groups
        for (int i = tid; i < ROWS * CB * GPB; i += LQ_NT) {
            const int g = i % (CB * GPB), r = i / (CB * GPB);
            const int gg = c0 * GPB + g;
            const int v = min((int)blockIdx.x * ROWS + r, V - 1);
            float s = 0.f, z = 8.f;
            if (gg < n_groups) {
                s = lq_scale(a.scales[(int64_t)v * n_groups + gg], a.scale_f16);
                if (a.zeros)
                    z = (float)(a.zeros[(int64_t)v * ((n_groups + 1) / 2) + (gg >> 1)] >> (gg & 1) * 4 & 15);
            }
            s_scale[g * ROWS + r] = s;
            s_zero[g * ROWS + r] = -(16.f + z);
        }
        __syncthreads();
        u32x4 next[RT][LQ_STEP];
        load_w(c0 + CB, next);
#pragma unroll
        for (int j = 0; j < LQ_STEP; ++j) {
            const int kb = kw * LQ_STEP + j;
#pragma unroll
            for (int t = 0; t < RT; ++t) lq_regroup<GROUP>(w[t][j]);
#pragma unroll
            for (int g = 0; g < GPB; ++g) {
                floatx4 acc[RT][NT], sc[RT];
                float sum[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) sum[n] = s_sum[((kb * GPB + g) * NT + n) * 16 + r16];
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const int at = (kb * GPB + g) * ROWS + (rw * RT + t) * 16 + quarter * 4;
                    const floatx4 z = *reinterpret_cast<const floatx4*>(&s_zero[at]);
                    sc[t] = *reinterpret_cast<const floatx4*>(&s_scale[at]);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int q = 0; q < 4; ++q) acc[t][n][q] = z[q] * sum[n];
                }
#pragma unroll
                for (int m = 0; m < MPG; ++m) {
                    const int i = g * MPG + m;
                    bf16x8 x[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        x[n] = __builtin_bit_cast(bf16x8, s_x[((kb * 4 + i) * NT + n) * WAVE + lane]);
#pragma unroll
                    for (int t = 0; t < RT; ++t) {
                        const bf16x8 wv = lq_widen(w[t][j][i]);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            acc[t][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, x[n], acc[t][n], 0, 0, 0);
                    }
                }
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            out[t][n][q] = __builtin_fmaf(sc[t][q], acc[t][n][q], out[t][n][q]);
            }
        }
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int j = 0; j < LQ_STEP; ++j) w[t][j] = next[t][j];
    }

    if (KW > 1) {  // the splits of K, added in order
        floatx4* s_red = reinterpret_cast<floatx4*>(s_x);
        static_assert(KW == 1 || (KW - 1) * RW * RT <= CB * 4, "the splits' sums fit the x stage");
        __syncthreads();
        if (kw > 0) {
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    s_red[((((kw - 1) * RW + rw) * RT + t) * NT + n) * WAVE + lane] = out[t][n];
        }
        __syncthreads();
        if (kw > 0) return;
#pragma unroll
        for (int k = 1; k < KW; ++k)
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    out[t][n] += s_red[((((k - 1) * RW + rw) * RT + t) * NT + n) * WAVE + lane];
    }
    // a lane holds four consecutive vocabulary entries of one batch row
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int b = n * 16 + r16;
        if (b >= a.B) continue;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const int v = row0 + t * 16 + quarter * 4;
            if (v >= V) continue;
            const int64_t at = (int64_t)b * a.out_stride + v;
            if (a.out_bf16) {
                __bf16* o = static_cast<__bf16*>(a.out) + at;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (v + q < V) o[q] = (__bf16)out[t][n][q];  // rounded once, to nearest even
            } else {
                float* o = static_cast<float*>(a.out) + at;
                if (v + 4 <= V) *reinterpret_cast<floatx4u*>(o) = out[t][n];
                else
                    for (int q = 0; q < 4; ++q)
                        if (v + q < V) o[q] = out[t][n][q];
            }
        }
    }
}

template <int GROUP, int NT, int RT, int KW>
static void launch_quant_t(const QuantArgs& a, hipStream_t st, const LaunchEvents& le) {
    constexpr int rows = LQ_WAVES / KW * RT * 16;
    launch_k(le, 0, k_lmhead_quant<GROUP, NT, RT, KW>, dim3((a.V + rows - 1) / rows), dim3(LQ_NT), st, a);
}

template <int GROUP>
static void launch_quant_g(const QuantArgs& a, hipStream_t st, const LaunchEvents& le) {
    if (a.B <= 16) launch_quant_t<GROUP, 1, 2, 2>(a, st, le);
    else if (a.B <= 32) launch_quant_t<GROUP, 2, 2, 2>(a, st, le);
    else launch_quant_t<GROUP, 4, 2, 1>(a, st, le);
}

hipError_t launch_quant(const QuantArgs& a, hipStream_t st, const LaunchEvents& le) {
    if (a.group == 32) launch_quant_g<32>(a, st, le);
    else if (a.group == 64) launch_quant_g<64>(a, st, le);
    else launch_quant_g<128>(a, st, le);
    return hipGetLastError();
}

}  // namespace ss
