// Verification of a draft against probability rows with the caller's uniforms.
//
//   accept draft j     iff  u_j q_j(d_j) < p_j(d_j)            (j = 0, 1, ... until one fails)
//   r(v) = max(0, p(v) - q(v))   at the first rejected position,
//          max(0, p(v))          at the position behind the last draft, and where
//                                the first has no mass
//   token = the lowest v with  r(0) + ... + r(v)  >  u_G (r(0) + ... + r(V-1))
//
// Products, differences and sums are binary64: u q of two binary32 values is
// exact there, so the accept test rounds nothing; p - q rounds once, at 2^-53.
//
// What bounds it: the one row (two with draft rows) that a request draws from;
// every other row costs a gather per draft. One workgroup per request would
// read a row at one CU's rate, so a row is cut into chunks of 2048 entries,
// PER of them a workgroup, that first repeats the (few) accept tests to learn
// which row it is. The chunks' sums go to the workspace; the workgroup that
// arrives last at its request's counter has them all, finds the chunk the draw
// lies in and searches it, and sets the counter back to 0. (As two launches the
// draw waited for the slowest request and cost 3 us more on the host.)
// Which workgroup draws is open, what it computes is not: it sums in order.
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
    __device__ __forceinline__ float at(int i) const { return i < 4 ? a[i] : b[i - 4]; }
};
struct Bf16 {
    uint16_t bits;
};
template <>
struct Raw8<Bf16> {
    typedef uint16_t v8 __attribute__((ext_vector_type(8), aligned(2)));
    v8 a;
    __device__ __forceinline__ void load(const Bf16* p) { a = *reinterpret_cast<const v8*>(p); }
    __device__ __forceinline__ float at(int i) const { return __uint_as_float((uint32_t)a[i] << 16); }
};
template <>
struct Raw8<_Float16> {
    typedef _Float16 v8 __attribute__((ext_vector_type(8), aligned(2)));
    v8 a;
    __device__ __forceinline__ void load(const _Float16* p) { a = *reinterpret_cast<const v8*>(p); }
    __device__ __forceinline__ float at(int i) const { return (float)a[i]; }
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(Bf16 x) { return __uint_as_float((uint32_t)x.bits << 16); }
__device__ __forceinline__ float to_f32(_Float16 x) { return (float)x; }

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
            const double p = to_f32(target[lane * a.target_stride + d]);
            const double q = draft ? to_f32(draft[lane * a.draft_stride + d]) : 1.0;
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

// The thread's entries v0 .. v0 + 7, where all of them lie in the row.
template <class T>
__device__ __forceinline__ void probs_load(const ProbsRow<T>& r, int v0, int V, Raw8<T>& rp, Raw8<T>& rq) {
    if (v0 + PV_EPT <= V) {
        rp.load(r.p + v0);
        if (r.q) rq.load(r.q + v0);
    }
}

// Their residual; those of a row's end are loaded here. max(0, p - q) is formed
// as p - min(p, q): the comparison in binary32 is exact, and binary64, a quarter
// of its rate, only subtracts. A negative or NaN p counts as 0, and a NaN q
// leaves nothing.
__device__ __forceinline__ double residual(float p, float q) {
    const float a = fmaxf(p, 0.0f);
    return (double)a - (double)fminf(a, q);
}
template <class T>
__device__ __forceinline__ void probs_entries(const ProbsRow<T>& r, int v0, int V, const Raw8<T>& rp,
                                              const Raw8<T>& rq, double x[PV_EPT]) {
    if (v0 + PV_EPT <= V) {
#pragma unroll
        for (int i = 0; i < PV_EPT; ++i)
            x[i] = r.q ? residual(rp.at(i), rq.at(i)) : (double)fmaxf(rp.at(i), 0.0f);
    } else {
#pragma unroll
        for (int i = 0; i < PV_EPT; ++i) {
            x[i] = 0.0;
            if (v0 + i < V) x[i] = residual(to_f32(r.p[v0 + i]), r.q ? to_f32(r.q[v0 + i]) : 0.0f);
        }
    }
    if (r.hot >= 0) {
#pragma unroll
        for (int i = 0; i < PV_EPT; ++i)
            if (v0 + i == r.hot) x[i] = 0.0;
    }
}

// Sums cross from the workgroups that made them to the one that draws, on another
// XCD and behind another L2. They are stored and loaded at agent scope, past the
// caches that are not shared, and a wait for the stores stands before the count:
// a release would order the same, and write back the whole L2 for it, 20 us with
// a thousand workgroups.
__device__ __forceinline__ void put_sum(double* p, double v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ double get_sum(const double* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <class T, int PER>
__global__ __launch_bounds__(PV_NT) void k_probs(ProbsArgs a) {
    __shared__ double s_part[PER][PV_WAVES];
    __shared__ double s_chunk[MAX_WT];
    __shared__ double s_wave[PV_WAVES];
    __shared__ int s_first[PV_WAVES], s_last[PV_WAVES];
    __shared__ int s_draws;
    const int b = blockIdx.y;
    const int tid = threadIdx.x;
    const int lane = tid & (WAVE - 1);
    const int wave = tid / WAVE;
    ProbsRow<T> r = probs_row<T>(a, b);
    double* part = a.part + (int64_t)b * a.n_chunks;
    {
        Raw8<T> rp[PER], rq[PER];  // every chunk's loads in flight together
        const int c0 = blockIdx.x * PER;
#pragma unroll
        for (int k = 0; k < PER; ++k) probs_load(r, (c0 + k) * PV_CHUNK + tid * PV_EPT, a.V, rp[k], rq[k]);
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            double x[PV_EPT];
            probs_entries(r, (c0 + k) * PV_CHUNK + tid * PV_EPT, a.V, rp[k], rq[k], x);
            double sum = 0.0;
#pragma unroll
            for (int i = 0; i < PV_EPT; ++i) sum += x[i];
            sum = wave_sum_d(sum);
            if (lane == 0) s_part[k][wave] = sum;
        }
    }
    __syncthreads();
    if (wave == 0) {  // lane k: chunk k of this workgroup
        const int c = blockIdx.x * PER + lane;
        if (lane < PER && c < a.n_chunks) {
            double t = s_part[lane][0];
#pragma unroll
            for (int w = 1; w < PV_WAVES; ++w) t += s_part[lane][w];
            put_sum(part + c, t);
        }
        // the wave's sums have reached the agent's point of coherence before its count does
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        if (lane == 0) {
            int32_t* arrived = a.arrived + b * PROBS_COUNTER;
            const int before = __hip_atomic_fetch_add(arrived, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            s_draws = before == (int)gridDim.x - 1;
            if (s_draws) __hip_atomic_store(arrived, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    __syncthreads();
    if (!s_draws) return;
    // the chunk of the draw, found by every wave: two chunks per lane (V <= 262144: 128 chunks)
    double m0 = 2 * lane < a.n_chunks ? get_sum(part + 2 * lane) : 0.0;
    double m1 = 2 * lane + 1 < a.n_chunks ? get_sum(part + 2 * lane + 1) : 0.0;
    double incl = wave_incl_scan_d(m0 + m1);
    double total = __shfl(incl, WAVE - 1);
    if (!(total > 0.0) && (r.q || r.hot >= 0)) {
        // p <= q everywhere (rounded rows, or one that p alone fills): the draw is
        // from p itself, whose sums this workgroup makes, a chunk a wave
        r.q = nullptr;
        r.hot = -1;
        for (int c = wave; c < a.n_chunks; c += PV_WAVES) {
            double sum = 0.0;
            for (int i = lane * PV_EPT; i < PV_CHUNK; i += WAVE * PV_EPT) {
                Raw8<T> rp, rq;
                double x[PV_EPT];
                probs_load(r, c * PV_CHUNK + i, a.V, rp, rq);
                probs_entries(r, c * PV_CHUNK + i, a.V, rp, rq, x);
#pragma unroll
                for (int k = 0; k < PV_EPT; ++k) sum += x[k];
            }
            sum = wave_sum_d(sum);
            if (lane == 0) s_chunk[c] = sum;
        }
        __syncthreads();
        m0 = 2 * lane < a.n_chunks ? s_chunk[2 * lane] : 0.0;
        m1 = 2 * lane + 1 < a.n_chunks ? s_chunk[2 * lane + 1] : 0.0;
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
        double x[PV_EPT];
        const int v0 = chunk * PV_CHUNK + tid * PV_EPT;
        Raw8<T> rp, rq;
        probs_load(r, v0, a.V, rp, rq);
        probs_entries(r, v0, a.V, rp, rq, x);
        double own = 0.0;
#pragma unroll
        for (int i = 0; i < PV_EPT; ++i) own += x[i];
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

template <class T, int PER>
static void launch_probs_p(const ProbsArgs& a, hipStream_t st, const LaunchEvents& le) {
    launch_k(le, 0, k_probs<T, PER>, dim3((a.n_chunks + PER - 1) / PER, a.B), dim3(PV_NT), st, a);
}

template <class T>
static void launch_probs_t(const ProbsArgs& a, hipStream_t st, const LaunchEvents& le) {
    // A chunk a workgroup up to two workgroups a CU. Measured over 16 to 2016 chunks with
    // draft rows in f32 and bf16 and without, G = 4: 16 chunks 5.7 us (two a workgroup:
    // 6.2), 256 5.8 (6.2), 504 6.3 (6.4), 600 6.5 (6.4), 800 6.9 (6.7), 1200 7.5 (7.0),
    // 1512 8.8 (7.4), 2016 10.1 (8.4); [64, 7, 152064] bf16, 4800: 17.5 (12.5, four 12.8).
    if ((int64_t)a.n_chunks * a.B <= 512) launch_probs_p<T, 1>(a, st, le);
    else launch_probs_p<T, 2>(a, st, le);
}

hipError_t launch_probs(const ProbsArgs& a, ss_dtype dt, hipStream_t st, const LaunchEvents& le) {
    if (dt == SS_F32) launch_probs_t<float>(a, st, le);
    else if (dt == SS_BF16) launch_probs_t<Bf16>(a, st, le);
    else launch_probs_t<_Float16>(a, st, le);
    return hipGetLastError();
}

}  // namespace ss
