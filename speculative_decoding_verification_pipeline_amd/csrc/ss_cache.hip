// Pages of a key/value cache: reserve, fork, commit, truncate, copy.
//
// A cache is num_planes equal arrays (a layer's keys, a layer's values, ...) of
// num_pages pages of page_size slots; a slot of a plane is `heads` pieces of
// piece_bytes. A page number names the same page of every plane. A request's
// block table lists its pages; ref[page] counts the tables that hold it, and a
// page is free iff its count is 0.
//
// Nothing here depends on the order in which workgroups run: counts change by
// integer atomics only, a free page is named by its rank among the free pages
// in ascending order, and every launch reads either what no workgroup of that
// launch writes or entries that it alone owns; a commit's table is written by the
// workgroup that finds, at its row's counter, that the others have read it, and
// counts of pages that others hold as well are lowered by the one that finds, at
// the call's counter, that every row is settled.
//
// What bounds it: the copying is bound by HBM (each byte read once and written
// once, 16 bytes per lane and as many loads in flight as rows are moved); the
// table work is a few dependent loads, so it is bound by latency and kept to
// one or two launches.
#include <limits.h>

#include "ss_device.h"
#include "ss_internal.h"
#include "ss_kv8.h"

namespace ss {

constexpr int CA_NT = 256;
constexpr int CA_WAVES = CA_NT / WAVE;
constexpr int CA_REF_EPT = CACHE_REF_CHUNK / CA_NT;  // counts per thread of a free-page chunk
constexpr int CA_UNROLL = 8;
constexpr int CA_RUNS = 5;       // blocks of 16 slots that 63 neighbouring slots touch
static_assert(CA_REF_EPT == 16, "four vector loads of counts per thread");
constexpr int CACHE_COMPARED = 1024;  // pairs that every copying workgroup compares itself

typedef int int4u __attribute__((ext_vector_type(4), aligned(4)));

// Compiler vectors: of HIP's uint4, a class, the arrays below went to scratch memory
// (copying 100 pages of 2 MB 93.5 -> 86.4 us, a commit of 64 rows in 32 layers 26.2 ->
// 21.2 us with its reserve).
template <int VEC>
struct CacheVec;
template <>
struct CacheVec<16> { typedef uint32_t type __attribute__((ext_vector_type(4))); };
template <>
struct CacheVec<4> { typedef uint32_t type; };
template <>
struct CacheVec<1> { typedef uint8_t type; };

__device__ __forceinline__ bool page_ok(int page, int num_pages) {
    return (unsigned)page < (unsigned)num_pages;
}

// Copies the first n slots of a page of one plane. Pieces that follow each
// other in memory on both sides (g.joined) are one run per head.
template <int VEC>
__device__ __forceinline__ void copy_slots(const CacheCopy& g, const char* __restrict__ src,
                                           char* __restrict__ dst, int n) {
    typedef typename CacheVec<VEC>::type V;
    const unsigned run = g.joined ? (unsigned)n * g.units : (unsigned)g.units;
    const unsigned outer = g.joined ? (unsigned)g.heads : (unsigned)(g.heads * n);
    const unsigned total = outer * run;
    for (unsigned u0 = threadIdx.x; u0 < total; u0 += CA_NT * 4) {
        V v[4];
        int64_t to[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const unsigned u = u0 + k * CA_NT;
            if (u < total) {
                unsigned o = 0, c = u;
                if (outer > 1) {
                    o = u / run;
                    c = u - o * run;
                }
                unsigned h = o, s = 0;
                if (!g.joined) {
                    h = o / (unsigned)n;
                    s = o - h * (unsigned)n;
                }
                to[k] = h * g.dst_head + s * g.dst_slot + (int64_t)c * VEC;
                v[k] = *reinterpret_cast<const V*>(src + h * g.src_head + s * g.src_slot +
                                                   (int64_t)c * VEC);
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (u0 + k * CA_NT < total) *reinterpret_cast<V*>(dst + to[k]) = v[k];
    }
}

// Copies the scales of the first n blocks of a page of one plane.
__device__ __forceinline__ void copy_scales(const ScaleCopy& g, const uint8_t* __restrict__ src,
                                            uint8_t* __restrict__ dst, int n) {
    for (int i = threadIdx.x; i < n * g.heads; i += CA_NT) {
        const int k = i / g.heads, h = i - k * g.heads;
        dst[k * g.dst_block + h * g.dst_head] = src[k * g.src_block + h * g.src_head];
    }
}

// ---------------------------------------------------------------------------
// reserve

// First launch. Workgroups 0 .. n_chunks - 1 list the free pages of their chunk
// of counts in ascending order; the others take one request per wave: which
// entries of its table need a fresh page (marks: rank among them, else -1),
// and the page whose slots have to be carried over.
__global__ __launch_bounds__(CA_NT) void k_cache_plan(CacheReserve a) {
    const int tid = threadIdx.x;
    const int lane = tid & (WAVE - 1);
    if ((int)blockIdx.x < a.n_chunks) {
        __shared__ RedT<CA_NT> red;
        const int p0 = blockIdx.x * CACHE_REF_CHUNK + tid * CA_REF_EPT;
        int free_mask = 0;
        if (p0 + CA_REF_EPT <= a.num_pages) {
            int4u v[CA_REF_EPT / 4];
#pragma unroll
            for (int i = 0; i < CA_REF_EPT / 4; ++i) v[i] = reinterpret_cast<const int4u*>(a.t.ref + p0)[i];
#pragma unroll
            for (int i = 0; i < CA_REF_EPT; ++i)
                if (v[i / 4][i % 4] == 0) free_mask |= 1 << i;
        } else {
            for (int i = 0; i < CA_REF_EPT; ++i)
                if (p0 + i < a.num_pages && a.t.ref[p0 + i] == 0) free_mask |= 1 << i;
        }
        int total;
        int at = block_excl_scan_i<CA_NT>(__popc(free_mask), red, total);
        int32_t* out = a.ws.free_ids + (int64_t)blockIdx.x * CACHE_REF_CHUNK;
#pragma unroll
        for (int i = 0; i < CA_REF_EPT; ++i)
            if (free_mask >> i & 1) out[at++] = p0 + i;
        if (tid == 0) a.ws.free_cnt[blockIdx.x] = total;
        return;
    }
    const int b = ((int)blockIdx.x - a.n_chunks) * CA_WAVES + tid / WAVE;
    if (b >= a.B) return;
    const int64_t base = a.base[b];
    const int64_t add = a.add[b];
    const int32_t* tab = a.t.tables + (int64_t)b * a.t.stride;
    int32_t* mark = a.ws.mark + (int64_t)b * a.max_blocks;
    int need = 0, carry = -1;
    if (base < 0 || add < 0 || (add > 0 && base + add > (int64_t)a.max_blocks * a.page_size)) {
        need = -1;  // refused
    } else if (add > 0) {
        const int lo = (int)((unsigned)base / (unsigned)a.page_size);
        const int hi = (int)((unsigned)(base + add + a.page_size - 1) / (unsigned)a.page_size);
        for (int i0 = lo; i0 < hi; i0 += WAVE) {
            const int i = i0 + lane;
            bool take = false;
            int page = -1;
            bool shared = false;
            if (i < hi) {
                page = tab[i];
                const bool held = page_ok(page, a.num_pages);
                shared = held && a.t.ref[page] > 1;
                take = !held || shared;
            }
            const unsigned long long m = __ballot(take);
            if (i < hi)
                mark[i] = take ? need + __popcll(m & ((1ull << lane) - 1)) : -1;
            need += __popcll(m);
            if (i0 == lo && (unsigned)base % (unsigned)a.page_size) carry = __shfl(shared ? page : -1, 0);
        }
    }
    if (lane == 0) {
        a.ws.need[b] = need;
        a.ws.carry[b] = carry;
    }
}

// Second launch, grid (1 + planes, B): workgroup (0, b) hands request b its
// pages, the others copy the slots before `base` of a shared last page, one
// plane each. Every workgroup finds by itself where its request's pages start
// in the list of free pages.
template <int VEC>
__global__ __launch_bounds__(CA_NT) void k_cache_take(CacheReserve a, CacheCopy g, ScaleCopy sc) {
    __shared__ RedT<CA_NT> red;
    __shared__ int s_end[CACHE_MAX_CHUNKS];  // free pages up to and including each chunk
    const int tid = threadIdx.x;
    const int b = blockIdx.y;
    const int need = a.ws.need[b];
    const int carry = a.ws.carry[b];
    if (blockIdx.x > 0 && carry < 0) return;
    // pages asked for by the requests before b
    int before = 0;
    for (int i = tid; i < b; i += CA_NT) before += max(a.ws.need[i], 0);
    int total;
    block_excl_scan_i<CA_NT>(before, red, before);
    int n_free = 0;
    for (int c0 = 0; c0 < a.n_chunks; c0 += CA_NT) {
        const int c = c0 + tid;
        const int v = c < a.n_chunks ? a.ws.free_cnt[c] : 0;
        const int ex = block_excl_scan_i<CA_NT>(v, red, total);
        if (c < a.n_chunks) s_end[c] = n_free + ex + v;
        n_free += total;
    }
    __syncthreads();
    // need and before stay below 2^31: B * max_blocks does
    const bool ok = need >= 0 && before + need <= n_free;
    auto fresh = [&](int rank) {  // the free page of this rank
        int l = 0, r = a.n_chunks - 1;
        while (l < r) {
            const int m = (l + r) >> 1;
            if (s_end[m] > rank) r = m;
            else l = m + 1;
        }
        return a.ws.free_ids[(int64_t)l * CACHE_REF_CHUNK + rank - (l ? s_end[l - 1] : 0)];
    };
    if (blockIdx.x > 0) {
        if (!ok) return;
        const int plane = blockIdx.x - 1;
        char* p = g.dst_planes[plane];
        const int to = fresh(before);
        const int slots = (int)((unsigned)a.base[b] % (unsigned)a.page_size);
        copy_slots<VEC>(g, p + carry * g.src_page, p + to * g.dst_page, slots);
        if (sc.src_planes) {
            uint8_t* q = sc.dst_planes[plane];
            copy_scales(sc, q + carry * sc.src_page, q + to * sc.dst_page,
                        (slots + sc.block - 1) / sc.block);
        }
        return;
    }
    if (tid == 0 && a.out_ok) a.out_ok[b] = ok ? 1 : 0;
    if (!ok || need == 0) return;
    // not negative, and base + add < 2^31: so k_cache_plan has left it
    const unsigned base = a.base[b], page_size = a.page_size;
    const int lo = (int)(base / page_size);
    const int hi = (int)((base + a.add[b] + page_size - 1) / page_size);
    int32_t* tab = a.t.tables + (int64_t)b * a.t.stride;
    const int32_t* mark = a.ws.mark + (int64_t)b * a.max_blocks;
    for (int i = lo + tid; i < hi; i += CA_NT) {
        if (mark[i] < 0) continue;
        const int old = tab[i];
        const int page = fresh(before + mark[i]);
        if (page_ok(old, a.num_pages)) atomicSub(&a.t.ref[old], 1);
        atomicAdd(&a.t.ref[page], 1);
        tab[i] = page;
    }
}

// ---------------------------------------------------------------------------
// release: the entries from `first` on leave the table of one row, drop gives
// each page back

template <class Drop>
__device__ __forceinline__ void release_from(const CacheTables& t, int num_pages, int max_blocks,
                                             int row, int first, Drop drop) {
    int32_t* tab = t.tables + (int64_t)row * t.stride;
    for (int i = first + threadIdx.x; i < max_blocks; i += CA_NT) {
        // a row listed twice is released once: only one exchange sees the page
        if (tab[i] == -1) continue;
        const int page = atomicExch(&tab[i], -1);
        if (page_ok(page, num_pages)) drop(page);
    }
}

__global__ __launch_bounds__(CA_NT) void k_cache_truncate(CacheTruncate a) {
    const int i = blockIdx.x;
    const int row = a.rows ? a.rows[i] : i;
    if ((unsigned)row >= (unsigned)a.t.rows) return;
    const int keep = a.new_len ? max(a.new_len[i], 0) : 0;
    const unsigned first = ((unsigned)keep + a.page_size - 1) / (unsigned)a.page_size;
    if (first < (unsigned)a.max_blocks)
        release_from(a.t, a.num_pages, a.max_blocks, row, (int)first,
                     [&](int page) { atomicSub(&a.t.ref[page], 1); });
    if (threadIdx.x == 0) atomicMin(&a.t.len[row], keep);
}

// ---------------------------------------------------------------------------
// fork

__global__ __launch_bounds__(CA_NT) void k_cache_fork(CacheFork a) {
    const int i = blockIdx.x;
    const int tid = threadIdx.x;
    const int src = a.src[i], dst = a.dst[i];
    bool bad = (unsigned)src >= (unsigned)a.t.rows || (unsigned)dst >= (unsigned)a.t.rows;
    // a destination named twice, or a source as well, is refused
    for (int k = tid; k < a.n; k += CA_NT)
        if (a.src[k] == dst || (k != i && a.dst[k] == dst)) bad = true;
    bad = __syncthreads_or(bad);
    if (tid == 0 && a.out_ok) a.out_ok[i] = bad ? 0 : 1;
    if (bad) return;
    const int len = a.t.len[src];
    const unsigned held = len > 0 ? ((unsigned)len + a.page_size - 1) / (unsigned)a.page_size : 0;
    const int32_t* from = a.t.tables + (int64_t)src * a.t.stride;
    int32_t* to = a.t.tables + (int64_t)dst * a.t.stride;
    for (int k = tid; k < a.max_blocks; k += CA_NT) {
        const int old = to[k];
        int page = (unsigned)k < held ? from[k] : -1;
        if (!page_ok(page, a.num_pages)) page = -1;
        if (page >= 0) atomicAdd(&a.t.ref[page], 1);
        if (page_ok(old, a.num_pages)) atomicSub(&a.t.ref[old], 1);
        to[k] = page;
    }
    if (tid == 0) a.t.len[dst] = len;
}

// ---------------------------------------------------------------------------
// commit

// Whether request b's step can be committed, for every wave of a workgroup: the
// reserve's verdict, where the caller passes it, is not 0; node indices ascend from
// at least 1 and stay below N (so a row moves towards the front only, and no row is
// overwritten before it is read); and every slot that is kept or moved lies on a
// page that the table names and no other entry holds: a row whose reserve was
// refused neither grows over pages it never got nor writes to ones it shares.
// Lane i gets row i's offsets and the counts of the pages that it looked up, which
// the caller compares, so that loads of data go out beside those of the counts.
// Slots stay below 2^31, so they are divided as 32-bit numbers.
struct CommitRow {
    bool ok;           // but for the counts
    int acc;
    int len;           // base + 1 + acc
    int64_t src, dst;  // page * src_page + slot * src_slot of lane i's move
    int64_t src_scale, dst_scale;  // of a scaled cache: where the blocks' scales lie
    int dst_in;        // and the slot moved to within its block
    bool moves;
    int kept, moved;   // counts: of the kept slots' pages, of the page moved from
};

template <bool SCALED>
__device__ __forceinline__ CommitRow commit_row(const CacheCommit& a, const CacheCopy& g,
                                                const ScaleCopy& sc, int b) {
    const int lane = threadIdx.x & (WAVE - 1);
    CommitRow r;
    // what does not depend on anything is loaded together
    r.acc = a.num_accepted[b];
    const int64_t base = a.base[b];
    const int reserved = a.reserved ? a.reserved[b] : 1;
    int node = 0, prev = 0;
    if (a.nodes && lane < a.N) {
        const int32_t* nodes = a.nodes + (int64_t)b * a.nodes_stride;
        node = nodes[lane];
        prev = lane ? nodes[lane - 1] : 0;
    }
    r.src = r.dst = r.src_scale = r.dst_scale = 0;
    r.dst_in = 0;
    r.moves = false;
    r.len = r.kept = r.moved = 0;
    const int64_t room = (int64_t)a.max_blocks * a.page_size;
    r.ok = base >= 0 && r.acc >= 0 && base + 1 + r.acc <= room && (!a.nodes || r.acc < a.N) &&
           reserved != 0;
    if (!r.ok) return r;
    r.len = (int)base + 1 + r.acc;
    const int32_t* tab = a.t.tables + (int64_t)b * a.t.stride;
    const unsigned page_size = a.page_size;
    const unsigned first = (unsigned)base / page_size + lane;
    const unsigned last = ((unsigned)base + r.acc) / page_size;
    int kept = -1, sp = -1, dp = -1;
    bool bad = false;
    if (first <= last) {
        kept = tab[first];
        bad = !page_ok(kept, a.num_pages);
    }
    if (a.nodes && lane < r.acc) {
        if (node <= prev || node >= a.N || base + node >= room) {
            bad = true;
        } else if (node != lane + 1) {
            const unsigned s = (unsigned)base + node, d = (unsigned)base + 1 + lane;
            sp = tab[s / page_size];
            dp = tab[d / page_size];
            if (!page_ok(sp, a.num_pages) || !page_ok(dp, a.num_pages)) {
                bad = true;
            } else {
                r.src = sp * g.src_page + (s % page_size) * g.src_slot;
                r.dst = dp * g.dst_page + (d % page_size) * g.dst_slot;
                if constexpr (SCALED) {
                    const unsigned block = sc.block;
                    r.src_scale = sp * sc.src_page + s % page_size / block * sc.src_block;
                    r.dst_scale = dp * sc.dst_page + d % page_size / block * sc.dst_block;
                    r.dst_in = (int)(d % block);
                }
                r.moves = true;
            }
        }
    }
    if (first <= last && !bad) r.kept = a.t.ref[kept];
    if (r.moves) r.moved = a.t.ref[sp];
    for (unsigned i = first + WAVE; i <= last; i += WAVE) {  // more pages than lanes
        const int page = tab[i];
        const bool held = page_ok(page, a.num_pages);
        bad |= !held;
        if (held) r.kept = max(r.kept, a.t.ref[page]);
    }
    r.ok = __ballot(bad) == 0;
    return r;
}

// Grid (units / 256, B); without nodes (1, B). A lane owns one vector of one head
// of one plane and moves it for every accepted node in order, eight loads at a
// time: a slot written here is read by no later node (their sources lie further
// back). The first eight go out before the counts have come (their addresses are
// good whatever the verdict), nothing is stored before. The workgroup that is the
// last of its row to have read the table and the length (which may be the base)
// writes them: the new length, and the pages behind it given back. It reads
// nothing that the others write.
//
// Counts of pages that others hold as well stay as they were until every row's
// workgroups have compared them: their releases are listed, and the workgroup that
// settles its row last of all takes the list off the counts. (A page that nobody
// else holds is given back at once: no other row looks at it.) Rows are counted in
// groups, and groups by the row that is last of its own: one counter takes 11 ns a
// row (a linear commit of 4096 rows: 50.7 us, in groups 11.1; without a count 7.4).
//
// settle: counts one more, and `left` entries with it, at a counter of `all`;
// whether it is the last, and then the entries of all. The last sets it back to 0.
__device__ __forceinline__ bool settle(unsigned long long* counter, int all, unsigned& left) {
    const unsigned long long one = (unsigned long long)left << 32 | 1;
    const unsigned long long c =
        __hip_atomic_fetch_add(counter, one, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + one;
    if ((unsigned)c != (unsigned)all) return false;
    __hip_atomic_store(counter, 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    left = (unsigned)(c >> 32);
    return true;
}

// The moves of a scaled cache. A workgroup takes whole heads of planes, a lane one vector of
// a head, so that nobody else reads or writes the head's scales; they are written when
// all of them are read. The slots that move fill blocks one after the other; a block's
// scale becomes the largest that its slots had: the moved ones' and, where it holds slots
// before them, its own. Slots of a smaller scale are rounded again to it.
__device__ __forceinline__ void move_scaled(const CacheCommit& a, const CacheCopy& g, const ScaleCopy& sc,
                                            const CommitRow& r, unsigned long long moves,
                                            uint8_t (*s_scale)[CA_RUNS]) {
    const int tid = threadIdx.x;
    const int here = CA_NT / sc.piece;  // heads of this workgroup
    const int hh = tid / sc.piece, u = tid - hh * sc.piece;
    const unsigned head = blockIdx.x * (unsigned)here + hh;
    const unsigned plane = head / (unsigned)sc.heads, h = head - plane * sc.heads;
    const bool on = hh < here && plane < (unsigned)a.num_planes;
    char* p = nullptr;
    uint8_t* q = nullptr;
    if (on) {
        p = g.dst_planes[plane] + h * g.dst_head + u * 16;
        q = sc.dst_planes[plane] + h * sc.dst_head;
    }
    int runs = 0;
    for (int i0 = __builtin_ctzll(moves); i0 < r.acc; ++runs) {
        const int64_t to = __shfl(r.dst_scale, i0);
        const int in = __shfl(r.dst_in, i0);
        const int n = min(r.acc - i0, sc.block - in);  // slots of this block
        int own = 0, most = 0;
        if (on) {
            if (in > 0) most = own = q[to];
        }
        for (int k = 0; k < n; ++k) {
            const int64_t from = __shfl(r.src_scale, i0 + k);
            if (on) most = max(most, (int)q[from]);
        }
        if (on && u == 0) s_scale[hh][runs] = (uint8_t)most;
        const int64_t first = __shfl(r.dst, i0) - in * g.dst_slot;
        if (on && own < most) {
            for (int k = 0; k < in; ++k) {
                kv8x16* at = reinterpret_cast<kv8x16*>(p + first + k * g.dst_slot);
                *at = kv8_shift(*at, own - most);
            }
        }
        for (int k0 = 0; k0 < n; k0 += CA_UNROLL) {
            kv8x16 v[CA_UNROLL];
            int by[CA_UNROLL];
#pragma unroll
            for (int k = 0; k < CA_UNROLL; ++k) {
                const int64_t at = __shfl(r.src, i0 + k0 + k), x = __shfl(r.src_scale, i0 + k0 + k);
                if (on && k0 + k < n) {
                    v[k] = *reinterpret_cast<const kv8x16*>(p + at);
                    by[k] = (int)q[x] - most;
                }
            }
#pragma unroll
            for (int k = 0; k < CA_UNROLL; ++k) {
                const int64_t at = __shfl(r.dst, i0 + k0 + k);
                if (on && k0 + k < n)
                    *reinterpret_cast<kv8x16*>(p + at) = by[k] < 0 ? kv8_shift(v[k], by[k]) : v[k];
            }
        }
        i0 += n;
    }
    __syncthreads();
    runs = 0;
    for (int i0 = __builtin_ctzll(moves); i0 < r.acc; ++runs) {
        const int64_t to = __shfl(r.dst_scale, i0);
        const int in = __shfl(r.dst_in, i0);
        if (on && u == 0) q[to] = s_scale[hh][runs];
        i0 += min(r.acc - i0, sc.block - in);
    }
}

template <int VEC, bool SCALED>
__global__ __launch_bounds__(CA_NT) void k_cache_commit(CacheCommit a, CacheCopy g, ScaleCopy sc) {
    typedef typename CacheVec<VEC>::type V;
    __shared__ int s_settles, s_left;
    const int b = blockIdx.y;
    const int tid = threadIdx.x;
    const unsigned per_plane = (unsigned)g.heads * g.units;
    const unsigned u = blockIdx.x * CA_NT + tid;
    const unsigned plane = u / per_plane;
    const bool on = plane < (unsigned)a.num_planes;
    char* p = on ? g.dst_planes[plane] : nullptr;
    CommitRow r = commit_row<SCALED>(a, g, sc, b);
    const unsigned long long moves = r.ok ? __ballot(r.moves) : 0;
    int i0 = moves ? __builtin_ctzll(moves) : r.acc;
    V v[CA_UNROLL];
    auto load = [&] {
#pragma unroll
        for (int k = 0; k < CA_UNROLL; ++k) {
            const int64_t s = __shfl(r.src, i0 + k);
            if (on && i0 + k < r.acc) v[k] = *reinterpret_cast<const V*>(p + s);
        }
    };
    if (moves && !SCALED) {
        const unsigned w = u - plane * per_plane;
        const unsigned h = w / g.units;
        if (on) p += h * g.dst_head + (int64_t)(w - h * g.units) * VEC;
        load();
    }
    r.ok = r.ok && __ballot(max(r.kept, r.moved) > 1) == 0;
    // every wave has its loads before the workgroup is counted
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    int32_t* arrived = a.arrived + b * CACHE_COUNTER;
    int before = 0;
    if (tid == 0) before = __hip_atomic_fetch_add(arrived, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if constexpr (SCALED) {
        __shared__ uint8_t s_scale[CA_NT][CA_RUNS];  // of a workgroup's heads and the blocks they fill
        if (moves && r.ok) move_scaled(a, g, sc, r, moves, s_scale);
    } else if (moves && r.ok) {
        for (;;) {
#pragma unroll
            for (int k = 0; k < CA_UNROLL; ++k) {
                const int64_t d = __shfl(r.dst, i0 + k);
                if (on && i0 + k < r.acc) *reinterpret_cast<V*>(p + d) = v[k];
            }
            i0 += CA_UNROLL;
            if (i0 >= r.acc) break;
            load();
        }
    }
    if (tid == 0) {
        s_settles = before == (int)gridDim.x - 1;
        if (s_settles) __hip_atomic_store(arrived, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (!s_settles) return;
    if (tid == 0 && a.out_ok) a.out_ok[b] = r.ok ? 1 : 0;
    if (tid == 0 && r.ok) a.t.len[b] = r.len;
    if (!a.release) return;
    if (tid == 0) s_left = 0;
    __syncthreads();
    if (r.ok)
        release_from(a.t, a.num_pages, a.max_blocks, b,
                     (int)(((unsigned)r.len + a.page_size - 1) / (unsigned)a.page_size), [&](int page) {
                         if (a.t.ref[page] > 1) {
                             const int at = __hip_atomic_fetch_add(a.n_left, 1, __ATOMIC_RELAXED,
                                                                   __HIP_MEMORY_SCOPE_AGENT);
                             __hip_atomic_store(a.left + at, page, __ATOMIC_RELAXED,
                                                __HIP_MEMORY_SCOPE_AGENT);
                             atomicAdd(&s_left, 1);
                             // the entry has reached the agent's point of coherence before it counts
                             asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                         } else {
                             atomicSub(&a.t.ref[page], 1);
                         }
                     });
    __syncthreads();
    if (tid == 0) {  // the entries of the list if this row is the last of all, else -1
        const int group = b / a.group, groups = (a.B + a.group - 1) / a.group;
        unsigned left = s_left;
        bool last = settle(a.settled + (1 + group) * (CACHE_COUNTER / 2),
                           min(a.group, a.B - group * a.group), left);
        if (last && groups > 1) last = settle(a.settled, groups, left);
        s_left = last ? (int)left : -1;
    }
    __syncthreads();
    const int n = s_left;
    if (n <= 0) return;
    for (int i = tid; i < n; i += CA_NT)
        atomicSub(&a.t.ref[__hip_atomic_load(a.left + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)], 1);
    if (tid == 0) __hip_atomic_store(a.n_left, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ---------------------------------------------------------------------------
// copy: page src[i] of one cache to page dst[i] of another or the same

// Whether pair i is refused: out of range, a destination named twice, or (within
// one cache) one that is also a source. first, step: the pairs this lane compares.
__device__ __forceinline__ bool pair_bad(const CachePages& a, int i, int first, int step) {
    const int src = a.src[i], dst = a.dst[i];
    bool bad = !page_ok(src, a.src_pages) || !page_ok(dst, a.dst_pages);
    for (int k = first; k < a.n; k += step)
        if ((a.same && a.src[k] == dst) || (k != i && a.dst[k] == dst)) bad = true;
    return bad;
}

// One wave per pair, for calls of many pairs.
__global__ __launch_bounds__(CA_NT) void k_cache_pairs(CachePages a) {
    const int i = blockIdx.x * CA_WAVES + threadIdx.x / WAVE;
    const int lane = threadIdx.x & (WAVE - 1);
    if (i >= a.n) return;
    const bool ok = __ballot(pair_bad(a, i, lane, WAVE)) == 0;
    if (lane == 0) a.pair_ok[i] = ok ? 1 : 0;
}

// Grid (pairs, planes): a plane's pages side by side (planes side by side took 2 %
// longer). Few pairs are compared by every workgroup that copies: one launch
// instead of two.
template <int VEC, bool COMPARE>
__global__ __launch_bounds__(CA_NT) void k_cache_copy(CachePages a, CacheCopy g, ScaleCopy sc) {
    const int i = blockIdx.x;
    const int plane = blockIdx.y;
    const bool ok = COMPARE ? !__syncthreads_or(pair_bad(a, i, threadIdx.x, CA_NT)) : a.pair_ok[i] != 0;
    if (plane == 0 && threadIdx.x == 0 && a.out_ok) a.out_ok[i] = ok ? 1 : 0;
    if (!ok) return;
    copy_slots<VEC>(g, g.src_planes[plane] + a.src[i] * g.src_page,
                    g.dst_planes[plane] + a.dst[i] * g.dst_page, a.page_size);
    if (sc.src_planes)
        copy_scales(sc, sc.src_planes[plane] + a.src[i] * sc.src_page,
                    sc.dst_planes[plane] + a.dst[i] * sc.dst_page, a.page_size / sc.block);
}

// ---------------------------------------------------------------------------

hipError_t launch_cache_reserve(const CacheReserve& a, const CacheCopy& g, const ScaleCopy& sc,
                                hipStream_t st) {
    const int nb = a.n_chunks + (a.B + CA_WAVES - 1) / CA_WAVES;
    hipLaunchKernelGGL(k_cache_plan, dim3(nb), dim3(CA_NT), 0, st, a);
    const dim3 grid(1 + a.num_planes, a.B);
    if (g.vec == 16) hipLaunchKernelGGL(k_cache_take<16>, grid, dim3(CA_NT), 0, st, a, g, sc);
    else if (g.vec == 4) hipLaunchKernelGGL(k_cache_take<4>, grid, dim3(CA_NT), 0, st, a, g, sc);
    else hipLaunchKernelGGL(k_cache_take<1>, grid, dim3(CA_NT), 0, st, a, g, sc);
    return hipGetLastError();
}

hipError_t launch_cache_truncate(const CacheTruncate& a, hipStream_t st) {
    hipLaunchKernelGGL(k_cache_truncate, dim3(a.n), dim3(CA_NT), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_cache_fork(const CacheFork& a, hipStream_t st) {
    hipLaunchKernelGGL(k_cache_fork, dim3(a.n), dim3(CA_NT), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_cache_commit(const CacheCommit& a, const CacheCopy& g, const ScaleCopy& sc,
                               hipStream_t st) {
    if (a.nodes && sc.src_planes) {
        const int here = CA_NT / sc.piece;
        const int64_t heads = (int64_t)a.num_planes * sc.heads;
        const dim3 grid((unsigned)((heads + here - 1) / here), a.B);
        hipLaunchKernelGGL((k_cache_commit<16, true>), grid, dim3(CA_NT), 0, st, a, g, sc);
        return hipGetLastError();
    }
    const int64_t units = a.nodes ? (int64_t)a.num_planes * g.heads * g.units : 1;
    const dim3 grid((unsigned)((units + CA_NT - 1) / CA_NT), a.B);
    if (g.vec == 16) hipLaunchKernelGGL((k_cache_commit<16, false>), grid, dim3(CA_NT), 0, st, a, g, sc);
    else if (g.vec == 4) hipLaunchKernelGGL((k_cache_commit<4, false>), grid, dim3(CA_NT), 0, st, a, g, sc);
    else hipLaunchKernelGGL((k_cache_commit<1, false>), grid, dim3(CA_NT), 0, st, a, g, sc);
    return hipGetLastError();
}

template <int VEC>
static void launch_cache_copy_v(const CachePages& a, const CacheCopy& g, const ScaleCopy& sc,
                                hipStream_t st) {
    const dim3 grid(a.n, a.num_planes);
    if (a.n <= CACHE_COMPARED) {
        hipLaunchKernelGGL((k_cache_copy<VEC, true>), grid, dim3(CA_NT), 0, st, a, g, sc);
    } else {
        hipLaunchKernelGGL(k_cache_pairs, dim3((a.n + CA_WAVES - 1) / CA_WAVES), dim3(CA_NT), 0, st, a);
        hipLaunchKernelGGL((k_cache_copy<VEC, false>), grid, dim3(CA_NT), 0, st, a, g, sc);
    }
}

hipError_t launch_cache_copy(const CachePages& a, const CacheCopy& g, const ScaleCopy& sc,
                             hipStream_t st) {
    if (g.vec == 16) launch_cache_copy_v<16>(a, g, sc, st);
    else if (g.vec == 4) launch_cache_copy_v<4>(a, g, sc, st);
    else launch_cache_copy_v<1>(a, g, sc, st);
    return hipGetLastError();
}

}  // namespace ss
