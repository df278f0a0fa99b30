// Host side of the page cache: handle lifetime, argument checks, launches.
// Nothing here allocates or synchronises after create.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstring>
#include <new>

#include "ss_device_guard.h"
#include "ss_internal.h"

struct ss_cache {
    ss_cache_config cfg;
    void* ws_base;
    int64_t ws_bytes;
    char** planes;      // device copy of the plane pointers
    ss::CacheWork ws;
    uint64_t low_bits;  // of every plane address and stride: what vectors are aligned
    int n_chunks;
};

namespace {

constexpr int64_t kAlign = 256;
constexpr int64_t align_up(int64_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool bad_config(const ss_cache_config* c) {
    if (c->device < 0 || c->num_planes < 1 || c->num_planes > 4096 || c->num_pages < 1 ||
        c->num_pages > ss::CACHE_MAX_PAGES || c->page_size < 1 || c->page_size > 65536 ||
        c->heads < 1 || c->heads > 65536 || c->piece_bytes < 1 || c->max_batch < 1 ||
        c->max_batch > 65535 || c->max_blocks < 1 || c->max_blocks > (1 << 24))
        return true;
    if ((int64_t)c->max_batch * c->max_blocks > INT32_MAX) return true;
    if ((int64_t)c->max_blocks * c->page_size > INT32_MAX) return true;  // lengths are 32 bits
    if ((int64_t)c->heads * c->piece_bytes > (1 << 24)) return true;
    if ((int64_t)c->num_planes * c->heads * c->piece_bytes > INT32_MAX) return true;
    if ((int64_t)c->page_size * c->heads * c->piece_bytes > INT32_MAX) return true;
    // Every piece of a plane has bytes of its own: the strides, sorted, each
    // span what lies within them.
    struct Dim {
        int64_t stride, count;
    };
    Dim d[3] = {{c->page_stride, c->num_pages}, {c->slot_stride, c->page_size},
                {c->head_stride, c->heads}};
    for (int i = 0; i < 3; ++i) {
        if (d[i].count == 1) d[i].stride = 0;  // never stepped: any stride does
        else if (d[i].stride < 1 || d[i].stride > (INT64_MAX >> 24)) return true;
    }
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            if (d[j].stride > d[j + 1].stride) {
                const Dim t = d[j];
                d[j] = d[j + 1];
                d[j + 1] = t;
            }
    int64_t span = c->piece_bytes;
    for (int i = 0; i < 3; ++i) {
        if (d[i].count == 1) continue;
        if (d[i].stride < span) return true;
        span += d[i].stride * (d[i].count - 1);
    }
    return false;
}

// The copy between two caches of one shape: heads that lie next to each other
// in a slot on both sides are one piece, and so on, to the widest vector that
// every address allows.
ss::CacheCopy copy_of(const ss_cache* src, const ss_cache* dst) {
    const ss_cache_config &s = src->cfg, &d = dst->cfg;
    ss::CacheCopy g;
    std::memset(&g, 0, sizeof(g));
    g.src_planes = src->planes;
    g.dst_planes = dst->planes;
    g.src_page = s.page_stride;
    g.src_slot = s.slot_stride;
    g.src_head = s.head_stride;
    g.dst_page = d.page_stride;
    g.dst_slot = d.slot_stride;
    g.dst_head = d.head_stride;
    g.heads = s.heads;
    int piece = s.piece_bytes;
    if (g.heads > 1 && g.src_head == piece && g.dst_head == piece) {
        piece *= g.heads;
        g.heads = 1;
    }
    const uint64_t low = src->low_bits | dst->low_bits;
    g.vec = low % 16 == 0 ? 16 : low % 4 == 0 ? 4 : 1;
    g.units = piece / g.vec;
    g.joined = s.page_size == 1 || (g.src_slot == piece && g.dst_slot == piece);
    return g;
}

ss_status check_tables(const ss_cache* c, const ss_block_tables* t) {
    if (!c || !t || !t->tables || !t->ref || !t->len) return SS_ERR_INVALID_ARG;
    if (t->rows < 1 || t->rows > c->cfg.max_batch || t->stride < c->cfg.max_blocks)
        return SS_ERR_INVALID_ARG;
    if (!aligned4(t->tables) || !aligned4(t->ref) || !aligned4(t->len)) return SS_ERR_INVALID_ARG;
    return SS_OK;
}

ss::CacheTables tables_of(const ss_block_tables* t) {
    return {t->tables, t->stride, t->rows, t->ref, t->len};
}

}  // namespace

extern "C" {

ss_status ss_cache_create(const ss_cache_config* cfg, void* const* planes, ss_cache** out) {
    if (!cfg || !planes || !out) return SS_ERR_INVALID_ARG;
    *out = nullptr;
    if (bad_config(cfg)) return SS_ERR_INVALID_ARG;
    uint64_t low = (uint64_t)cfg->piece_bytes;
    if (cfg->num_pages > 1) low |= (uint64_t)cfg->page_stride;
    if (cfg->page_size > 1) low |= (uint64_t)cfg->slot_stride;
    if (cfg->heads > 1) low |= (uint64_t)cfg->head_stride;
    for (int i = 0; i < cfg->num_planes; ++i) {
        if (!planes[i]) return SS_ERR_INVALID_ARG;
        low |= (uint64_t)reinterpret_cast<uintptr_t>(planes[i]);
        // a plane named twice would be moved twice, by workgroups that do not wait
        for (int j = 0; j < i; ++j)
            if (planes[j] == planes[i]) return SS_ERR_INVALID_ARG;
    }
    int ndev = 0;
    if (hipGetDeviceCount(&ndev) != hipSuccess || cfg->device >= ndev) return SS_ERR_HIP;
    ss::DeviceGuard guard(cfg->device);
    if (!guard.ok) return SS_ERR_HIP;
    ss_cache* c = new (std::nothrow) ss_cache();
    if (!c) return SS_ERR_OUT_OF_MEMORY;
    c->cfg = *cfg;
    c->low_bits = low;
    c->n_chunks = (cfg->num_pages + ss::CACHE_REF_CHUNK - 1) / ss::CACHE_REF_CHUNK;
    int64_t off = 0;
    auto take = [&off](int64_t bytes) {
        const int64_t o = off;
        off = align_up(off + bytes);
        return o;
    };
    // the plane pointers and the counters of 0, filled by one copy
    const int64_t o_planes = take((int64_t)cfg->num_planes * sizeof(char*));
    const int64_t o_arrived =
        take(((int64_t)cfg->max_batch + 1 + ss::CACHE_GROUPS + 1) * ss::CACHE_COUNTER * 4);
    const int64_t filled = off;
    const int64_t o_ids = take((int64_t)c->n_chunks * ss::CACHE_REF_CHUNK * 4);
    const int64_t o_cnt = take((int64_t)c->n_chunks * 4);
    const int64_t o_need = take((int64_t)cfg->max_batch * 4);
    const int64_t o_carry = take((int64_t)cfg->max_batch * 4);
    const int64_t o_mark = take((int64_t)cfg->max_batch * cfg->max_blocks * 4);
    const int64_t o_pair = take((int64_t)cfg->num_pages * 4);
    c->ws_bytes = off;
    if (hipMalloc(&c->ws_base, (size_t)off) != hipSuccess) {
        (void)hipGetLastError();
        delete c;
        return SS_ERR_OUT_OF_MEMORY;
    }
    char* b = static_cast<char*>(c->ws_base);
    c->planes = reinterpret_cast<char**>(b + o_planes);
    c->ws.free_ids = reinterpret_cast<int32_t*>(b + o_ids);
    c->ws.free_cnt = reinterpret_cast<int32_t*>(b + o_cnt);
    c->ws.need = reinterpret_cast<int32_t*>(b + o_need);
    c->ws.carry = reinterpret_cast<int32_t*>(b + o_carry);
    c->ws.mark = reinterpret_cast<int32_t*>(b + o_mark);
    c->ws.pair_ok = reinterpret_cast<int32_t*>(b + o_pair);
    c->ws.arrived = reinterpret_cast<int32_t*>(b + o_arrived);
    int32_t* settled = c->ws.arrived + (int64_t)cfg->max_batch * ss::CACHE_COUNTER;
    c->ws.settled = reinterpret_cast<unsigned long long*>(settled);
    c->ws.n_left = settled + (1 + ss::CACHE_GROUPS) * ss::CACHE_COUNTER;
    char* h = new (std::nothrow) char[(size_t)filled]();
    if (!h) {
        (void)hipFree(c->ws_base);
        delete c;
        return SS_ERR_OUT_OF_MEMORY;
    }
    std::memcpy(h + o_planes, planes, (size_t)cfg->num_planes * sizeof(char*));
    const bool ok = hipMemcpy(b, h, (size_t)filled, hipMemcpyHostToDevice) == hipSuccess;
    delete[] h;
    if (!ok) {
        (void)hipFree(c->ws_base);
        delete c;
        return SS_ERR_HIP;
    }
    *out = c;
    return SS_OK;
}

void ss_cache_destroy(ss_cache* c) {
    if (!c) return;
    ss::DeviceGuard guard(c->cfg.device);
    (void)hipFree(c->ws_base);
    delete c;
}

int64_t ss_cache_workspace_bytes(const ss_cache* c) { return c ? c->ws_bytes : 0; }

ss_status ss_cache_reserve(ss_cache* c, const ss_block_tables* t, const int32_t* base,
                           const int32_t* add, int32_t B, int32_t* out_ok, void* stream) {
    ss_status st = check_tables(c, t);
    if (st != SS_OK) return st;
    if (B < 0 || B > t->rows) return SS_ERR_INVALID_ARG;
    if (B == 0) return SS_OK;
    if (!add) return SS_ERR_INVALID_ARG;
    ss::CacheReserve a;
    std::memset(&a, 0, sizeof(a));
    a.t = tables_of(t);
    a.ws = c->ws;
    a.base = base ? base : t->len;
    a.add = add;
    a.B = B;
    a.out_ok = out_ok;
    a.num_pages = c->cfg.num_pages;
    a.num_planes = c->cfg.num_planes;
    a.page_size = c->cfg.page_size;
    a.max_blocks = c->cfg.max_blocks;
    a.n_chunks = c->n_chunks;
    ss::DeviceGuard guard(c->cfg.device);
    if (!guard.ok) return SS_ERR_HIP;
    return ss::launch_cache_reserve(a, copy_of(c, c), static_cast<hipStream_t>(stream)) == hipSuccess
               ? SS_OK
               : SS_ERR_HIP;
}

ss_status ss_cache_fork(ss_cache* c, const ss_block_tables* t, const int32_t* src,
                        const int32_t* dst, int32_t n, int32_t* out_ok, void* stream) {
    ss_status st = check_tables(c, t);
    if (st != SS_OK) return st;
    if (n < 0 || n > t->rows) return SS_ERR_INVALID_ARG;
    if (n == 0) return SS_OK;
    if (!src || !dst) return SS_ERR_INVALID_ARG;
    ss::CacheFork a;
    std::memset(&a, 0, sizeof(a));
    a.t = tables_of(t);
    a.src = src;
    a.dst = dst;
    a.n = n;
    a.out_ok = out_ok;
    a.num_pages = c->cfg.num_pages;
    a.page_size = c->cfg.page_size;
    a.max_blocks = c->cfg.max_blocks;
    ss::DeviceGuard guard(c->cfg.device);
    if (!guard.ok) return SS_ERR_HIP;
    return ss::launch_cache_fork(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SS_OK
                                                                                    : SS_ERR_HIP;
}

ss_status ss_cache_commit(ss_cache* c, const ss_block_tables* t, const int32_t* base,
                          const int32_t* nodes, int64_t nodes_stride, int32_t N,
                          const int32_t* num_accepted, int32_t B, int32_t release,
                          int32_t* out_ok, void* stream) {
    return ss_cache_commit_reserved(c, t, base, nodes, nodes_stride, N, num_accepted, B, release,
                                    nullptr, out_ok, stream);
}

ss_status ss_cache_commit_reserved(ss_cache* c, const ss_block_tables* t, const int32_t* base,
                                   const int32_t* nodes, int64_t nodes_stride, int32_t N,
                                   const int32_t* num_accepted, int32_t B, int32_t release,
                                   const int32_t* reserved, int32_t* out_ok, void* stream) {
    ss_status st = check_tables(c, t);
    if (st != SS_OK) return st;
    if (B < 0 || B > t->rows) return SS_ERR_INVALID_ARG;
    if (B == 0) return SS_OK;
    if (!num_accepted) return SS_ERR_INVALID_ARG;
    if (nodes && (N < 1 || N > 64 || nodes_stride < N)) return SS_ERR_INVALID_ARG;
    ss::CacheCommit a;
    std::memset(&a, 0, sizeof(a));
    a.t = tables_of(t);
    a.base = base ? base : t->len;
    a.num_accepted = num_accepted;
    a.nodes = nodes;
    a.nodes_stride = nodes_stride;
    a.N = N;
    a.B = B;
    a.release = release != 0;
    a.reserved = reserved;
    a.arrived = c->ws.arrived;
    a.settled = c->ws.settled;
    a.n_left = c->ws.n_left;
    a.left = c->ws.mark;
    // about as many groups as rows in one, from 32 rows on: 65535 rows in 256 of 256
    a.group = 32;
    while (a.group * a.group < B) a.group *= 2;
    a.out_ok = out_ok;
    a.num_pages = c->cfg.num_pages;
    a.num_planes = c->cfg.num_planes;
    a.page_size = c->cfg.page_size;
    a.max_blocks = c->cfg.max_blocks;
    ss::DeviceGuard guard(c->cfg.device);
    if (!guard.ok) return SS_ERR_HIP;
    return ss::launch_cache_commit(a, copy_of(c, c), static_cast<hipStream_t>(stream)) == hipSuccess
               ? SS_OK
               : SS_ERR_HIP;
}

ss_status ss_cache_truncate(ss_cache* c, const ss_block_tables* t, const int32_t* rows,
                            const int32_t* new_len, int32_t n, void* stream) {
    ss_status st = check_tables(c, t);
    if (st != SS_OK) return st;
    if (n < 0 || n > t->rows) return SS_ERR_INVALID_ARG;
    if (n == 0) return SS_OK;
    ss::CacheTruncate a;
    std::memset(&a, 0, sizeof(a));
    a.t = tables_of(t);
    a.rows = rows;
    a.new_len = new_len;
    a.n = n;
    a.num_pages = c->cfg.num_pages;
    a.page_size = c->cfg.page_size;
    a.max_blocks = c->cfg.max_blocks;
    ss::DeviceGuard guard(c->cfg.device);
    if (!guard.ok) return SS_ERR_HIP;
    return ss::launch_cache_truncate(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SS_OK
                                                                                        : SS_ERR_HIP;
}

ss_status ss_cache_copy_pages(ss_cache* src_cache, const int32_t* src, ss_cache* dst_cache,
                              const int32_t* dst, int32_t n, int32_t* out_ok, void* stream) {
    if (!src_cache || !dst_cache) return SS_ERR_INVALID_ARG;
    const ss_cache_config &s = src_cache->cfg, &d = dst_cache->cfg;
    if (s.device != d.device || s.num_planes != d.num_planes || s.page_size != d.page_size ||
        s.heads != d.heads || s.piece_bytes != d.piece_bytes)
        return SS_ERR_INVALID_ARG;
    if (n < 0 || n > d.num_pages || n > 65535) return SS_ERR_INVALID_ARG;
    if (n == 0) return SS_OK;
    if (!src || !dst) return SS_ERR_INVALID_ARG;
    ss::CachePages a;
    std::memset(&a, 0, sizeof(a));
    a.src = src;
    a.dst = dst;
    a.n = n;
    a.same = src_cache == dst_cache;
    a.src_pages = s.num_pages;
    a.dst_pages = d.num_pages;
    a.num_planes = s.num_planes;
    a.page_size = s.page_size;
    a.pair_ok = dst_cache->ws.pair_ok;
    a.out_ok = out_ok;
    ss::DeviceGuard guard(d.device);
    if (!guard.ok) return SS_ERR_HIP;
    return ss::launch_cache_copy(a, copy_of(src_cache, dst_cache),
                                 static_cast<hipStream_t>(stream)) == hipSuccess
               ? SS_OK
               : SS_ERR_HIP;
}

}  // extern "C"
