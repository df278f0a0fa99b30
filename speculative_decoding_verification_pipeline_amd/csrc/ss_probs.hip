// Verification of a draft against probability rows with the caller's uniforms.
//
//   accept draft j     iff  u_j q_j(d_j) < p_j(d_j)            (j = 0, 1, ... until one fails)
//   r(v) = max(0, p(v) - q(v))   at the first rejected position,
//          max(0, p(v))          at the position behind the last draft
//   token = the lowest v with  r(0) + ... + r(v)  >  u_G (r(0) + ... + r(V-1))
//
// Products, differences and sums are binary64: u q of two binary32 values is
// exact there, so the accept test rounds nothing; p - q rounds once, at 2^-53.
//
// What bounds it: the one row (two with draft rows) that a request draws from;
// every other row costs a gather per draft. One workgroup per request would
// read a row at one CU's rate, so a row is cut into chunks of 2048 entries, one
// workgroup each, that first repeat the (few) accept tests to learn which row
// it is. A second launch scans the chunks' sums, finds the chunk the draw lies
// in and searches it. The kernel boundary is the only synchronisation.
#include <limits.h>

#include "ss_device.h"
#include "ss_internal.h"

#pragma clang fp contract(off)

namespace ss {

constexpr int PV_NT = 256;
constexpr int PV_EPT = 8;                   // entries per thread
constexpr int PV_CHUNK = PV_NT * PV_EPT;
static_assert(PV_CHUNK == WT, "the workspace holds one sum per wave tile");
constexpr int PV_WAVES = PV_NT / WAVE;

// Eight consecutive entries as they are stored: rows start at any element, so
// the vectors claim an element's alignment only (unaligned 16-byte loads are
// served in one instruction).
template <class T>
struct Raw8;
template <>
struct Raw8<float> {
    typedef float v4 __attribute__((ext_vector_type(4), aligned(4)));
    v4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const v4*>(p);
        b = *reinterpret_cast<const v4*>(p + 4);
    }
    __device__ __forceinline__ double at(int i) const { return (double)(i < 4 ? a[i] : b[i - 4]); }
};
struct Bf16 {
    uint16_t bits;
};
template <>
struct Raw8<Bf16> {
    typedef uint16_t v8 __attribute__((ext_vector_type(8), aligned(2)));
    v8 a;
    __device__ __forceinline__ void load(const Bf16* p) { a = *reinterpret_cast<const v8*>(p); }
    __device__ __forceinline__ double at(int i) const {
        return (double)__uint_as_float((uint32_t)a[i] << 16);
    }
};
template <>
struct Raw8<_Float16> {
    typedef _Float16 v8 __attribute__((ext_vector_type(8), aligned(2)));
    v8 a;
    __device__ __forceinline__ void load(const _Float16* p) { a = *reinterpret_cast<const v8*>(p); }
    __device__ __forceinline__ double at(int i) const { return (double)(float)a[i]; }
};

__device__ __forceinline__ double to_f64(float x) { return (double)x; }
__device__ __forceinline__ double to_f64(Bf16 x) {
    return (double)__uint_as_float((uint32_t)x.bits << 16);
}
__device__ __forceinline__ double to_f64(_Float16 x) { return (double)(float)x; }

// The rows a request draws from.
template <class T>
struct ProbsRow {
    const T* p;
    const T* q;   // the draft row of a rejected position, else null
    int hot;      // the rejected token of a one-hot draft, else -1
    int acc;      // accepted drafts
};

// Every wave makes the accept tests of its request, lane j draft j (G <= 63).
template <class T>
__device__ __forceinline__ ProbsRow<T> probs_row(const ProbsArgs& a, int b) {
    const int lane = threadIdx.x & (WAVE - 1);
    const T* target = static_cast<const T*>(a.target) + (int64_t)b * (a.G + 1) * a.target_stride;
    const T* draft = a.draft ? static_cast<const T*>(a.draft) + (int64_t)b * a.G * a.draft_stride
                             : nullptr;
    int n = a.G;
    if (a.draft_len) {
        n = a.draft_len[b];
        n = n < 0 ? 0 : n > a.G ? a.G : n;
    }
    bool ok = false;
    int d = -1;
    if (lane < n) {
        d = a.draft_tokens[(int64_t)b * a.G + lane];
        if (d >= 0 && d < a.V) {
            const double u = (double)a.uniforms[(int64_t)b * (a.G + 1) + lane];
            const double p = to_f64(target[lane * a.target_stride + d]);
            const double q = draft ? to_f64(draft[lane * a.draft_stride + d]) : 1.0;
            ok = u * q < p;
        }
    }
    const unsigned long long m = __ballot(ok);
    ProbsRow<T> r;
    r.acc = ~m ? __builtin_ctzll(~m) : WAVE;  // lanes from n on are 0: acc <= n
    const bool rejected = r.acc < n;
    r.p = target + r.acc * a.target_stride;
    r.q = rejected && draft ? draft + r.acc * a.draft_stride : nullptr;
    r.hot = rejected && !draft ? __shfl(d, r.acc) : -1;
    return r;
}

// Residual (x) and target mass (p) of the thread's entries v0 .. v0 + 7.
// fmax takes a NaN entry for 0, and a negative one as well.
template <class T>
__device__ __forceinline__ void probs_entries(const ProbsRow<T>& r, int v0, int V, double x[PV_EPT],
                                              double p[PV_EPT]) {
    if (v0 + PV_EPT <= V) {
        Raw8<T> rp, rq;
        rp.load(r.p + v0);
        if (r.q) rq.load(r.q + v0);
#pragma unroll
        for (int i = 0; i < PV_EPT; ++i) {
            p[i] = fmax(rp.at(i), 0.0);
            x[i] = r.q ? fmax(rp.at(i) - rq.at(i), 0.0) : p[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < PV_EPT; ++i) {
            p[i] = x[i] = 0.0;
            if (v0 + i < V) {
                const double pv = to_f64(r.p[v0 + i]);
                p[i] = fmax(pv, 0.0);
                x[i] = r.q ? fmax(pv - to_f64(r.q[v0 + i]), 0.0) : p[i];
            }
        }
    }
    if (r.hot >= 0) {
#pragma unroll
        for (int i = 0; i < PV_EPT; ++i)
            if (v0 + i == r.hot) x[i] = 0.0;
    }
}

template <class T>
__global__ __launch_bounds__(PV_NT) void k_probs_mass(ProbsArgs a) {
    __shared__ double2 s_part[PV_WAVES];
    const int b = blockIdx.y;
    const int wave = threadIdx.x / WAVE;
    const ProbsRow<T> r = probs_row<T>(a, b);
    double x[PV_EPT], p[PV_EPT];
    probs_entries(r, blockIdx.x * PV_CHUNK + threadIdx.x * PV_EPT, a.V, x, p);
    double sx = 0.0, sp = 0.0;
#pragma unroll
    for (int i = 0; i < PV_EPT; ++i) {
        sx += x[i];
        sp += p[i];
    }
    sx = wave_sum_d(sx);
    sp = wave_sum_d(sp);
    if ((threadIdx.x & (WAVE - 1)) == 0) s_part[wave] = make_double2(sx, sp);
    __syncthreads();
    if (threadIdx.x == 0) {
        double2 t = s_part[0];
#pragma unroll
        for (int w = 1; w < PV_WAVES; ++w) {
            t.x += s_part[w].x;
            t.y += s_part[w].y;
        }
        a.part[(int64_t)b * a.n_chunks + blockIdx.x] = t;
    }
}

template <class T>
__global__ __launch_bounds__(PV_NT) void k_probs_draw(ProbsArgs a) {
    __shared__ double s_wave[PV_WAVES];
    __shared__ int s_first[PV_WAVES], s_last[PV_WAVES];
    const int b = blockIdx.x;
    const int tid = threadIdx.x;
    const int lane = tid & (WAVE - 1);
    const int wave = tid / WAVE;
    const ProbsRow<T> r = probs_row<T>(a, b);
    // the chunk of the draw, found by every wave: two chunks per lane (V <= 262144: 128 chunks)
    const double2* part = a.part + (int64_t)b * a.n_chunks;
    double2 c0 = make_double2(0.0, 0.0), c1 = c0;
    if (2 * lane < a.n_chunks) c0 = part[2 * lane];
    if (2 * lane + 1 < a.n_chunks) c1 = part[2 * lane + 1];
    double incl = wave_incl_scan_d(c0.x + c1.x);
    double total = __shfl(incl, WAVE - 1);
    const bool whole = !(total > 0.0);  // p <= q everywhere: draw from p itself
    double m0 = c0.x, m1 = c1.x;
    if (whole) {
        m0 = c0.y;
        m1 = c1.y;
        incl = wave_incl_scan_d(m0 + m1);
        total = __shfl(incl, WAVE - 1);
    }
    int token = -1;
    if (total > 0.0) {
        const double goal = (double)a.uniforms[(int64_t)b * (a.G + 1) + a.G] * total;
        double before = __shfl_up(incl, 1);
        if (lane == 0) before = 0.0;
        // chunk 2 lane ends at before + m0, chunk 2 lane + 1 at incl
        const unsigned long long hit = __ballot(incl > goal && m0 + m1 > 0.0);
        int chunk;
        double base;
        if (hit) {
            const int l = __builtin_ctzll(hit);
            const double lb = __shfl(before, l), l0 = __shfl(m0, l), l1 = __shfl(m1, l);
            const bool second = !(l0 > 0.0 && lb + l0 > goal) && l1 > 0.0;
            chunk = 2 * l + (second ? 1 : 0);
            base = second ? lb + l0 : lb;
        } else {  // a uniform outside [0, 1): the last entry with mass
            const int l = WAVE - 1 - __builtin_clzll(__ballot(m0 + m1 > 0.0));
            chunk = 2 * l + (__shfl(m1, l) > 0.0 ? 1 : 0);
            base = 0.0;
        }
        double x[PV_EPT], p[PV_EPT];
        const int v0 = chunk * PV_CHUNK + tid * PV_EPT;
        probs_entries(r, v0, a.V, x, p);
        double own = 0.0;
#pragma unroll
        for (int i = 0; i < PV_EPT; ++i) {
            if (whole) x[i] = p[i];
            own += x[i];
        }
        const double scan = wave_incl_scan_d(own);
        if (lane == WAVE - 1) s_wave[wave] = scan;
        __syncthreads();
        double cum = base;
        for (int w = 0; w < wave; ++w) cum += s_wave[w];
        const double prev = __shfl_up(scan, 1);
        if (lane > 0) cum += prev;
        int first = INT_MAX, last = -1;
#pragma unroll
        for (int i = 0; i < PV_EPT; ++i) {
            cum += x[i];
            if (x[i] > 0.0) {
                last = v0 + i;
                if (hit && first == INT_MAX && cum > goal) first = v0 + i;
            }
        }
        const unsigned long long mf = __ballot(first != INT_MAX), ml = __ballot(last >= 0);
        first = mf ? __shfl(first, __builtin_ctzll(mf)) : INT_MAX;
        last = ml ? __shfl(last, WAVE - 1 - __builtin_clzll(ml)) : -1;
        if (lane == 0) {
            s_first[wave] = first;
            s_last[wave] = last;
        }
        __syncthreads();
        // The chunk's sums round differently here than in its total, so a goal
        // within rounding of the chunk's end may find none: its last entry then.
        first = INT_MAX;
#pragma unroll
        for (int w = 0; w < PV_WAVES; ++w) {
            first = min(first, s_first[w]);
            last = max(last, s_last[w]);
        }
        token = first != INT_MAX ? first : last;
    }
    if (tid <= a.G) {
        const int t = tid < r.acc ? a.draft_tokens[(int64_t)b * a.G + tid]
                                  : tid == r.acc ? token : -1;
        a.out_tokens[(int64_t)b * (a.G + 1) + tid] = t;
    }
    if (tid == 0) a.out_num_accepted[b] = r.acc;
    if (a.seq_tokens && wave == 0) {  // G + 1 <= 64: one wave appends
        const int len = a.seq_len[b];
        const int room = len < 0 || len > a.seq_capacity ? 0 : a.seq_capacity - len;
        const int n = min(r.acc + 1, room);
        if (lane < n)
            a.seq_tokens[(int64_t)b * a.seq_stride + len + lane] =
                lane < r.acc ? a.draft_tokens[(int64_t)b * a.G + lane] : token;
        if (lane == 0 && n > 0) a.seq_len[b] = len + n;
    }
}

template <class T>
static void launch_probs_t(const ProbsArgs& a, hipStream_t st, const LaunchEvents& le) {
    launch_k(le, 0, k_probs_mass<T>, dim3(a.n_chunks, a.B), dim3(PV_NT), st, a);
    launch_k(le, 1, k_probs_draw<T>, dim3(a.B), dim3(PV_NT), st, a);
}

hipError_t launch_probs(const ProbsArgs& a, ss_dtype dt, hipStream_t st, const LaunchEvents& le) {
    if (dt == SS_F32) launch_probs_t<float>(a, st, le);
    else if (dt == SS_BF16) launch_probs_t<Bf16>(a, st, le);
    else launch_probs_t<_Float16>(a, st, le);
    return hipGetLastError();
}

}  // namespace ss
