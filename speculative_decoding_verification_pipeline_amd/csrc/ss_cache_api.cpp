// Host side of the page cache: handle lifetime, argument checks, launches.
// Nothing here allocates or synchronises after create.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstring>
#include <initializer_list>
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
    // a scaled cache (scales.block 0: it has none)
    ss_cache_scales scales;
    uint8_t** scale_planes;   // device copy of the scales' pointers
    ss::Kv8Plane* planes8;    // host copies of both, by plane
    float* part;              // what attention's pieces leave, and their counters
    int32_t* pieces;
};

namespace {

constexpr int64_t kAlign = 256;
constexpr int64_t align_up(int64_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

struct Dim {
    int64_t stride, count;
};

// Whether pieces of these strides share bytes: the strides, sorted, each span what lies
// within them.
bool overlap(const Dim (&dims)[3], int64_t piece) {
    Dim d[3] = {dims[0], dims[1], dims[2]};
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
    int64_t span = piece;
    for (int i = 0; i < 3; ++i) {
        if (d[i].count == 1) continue;
        if (d[i].stride < span) return true;
        span += d[i].stride * (d[i].count - 1);
    }
    return false;
}

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
    const Dim d[3] = {{c->page_stride, c->num_pages}, {c->slot_stride, c->page_size},
                      {c->head_stride, c->heads}};
    return overlap(d, c->piece_bytes);
}

// The scales of a cache: a byte for each block of slots and head.
bool bad_scales(const ss_cache_config* c, const ss_cache_scales* s) {
    if ((s->block != 16 && s->block != 32 && s->block != 64) || c->page_size % s->block) return true;
    const Dim d[3] = {{s->page_stride, c->num_pages}, {s->block_stride, c->page_size / s->block},
                      {s->head_stride, c->heads}};
    return overlap(d, 1);
}

// What the kernels of a scaled cache serve: heads in vectors of 16 bytes, tiles of 16 slots
// within a page, offsets within a page in 32 bits.
bool unserved_scaled(const ss_cache_config* c, uint64_t low) {
    if (c->piece_bytes % 16 || c->piece_bytes > 256 || c->page_size % 16 || low % 16) return true;
    const int64_t slots = c->page_size > 1 ? c->slot_stride * (c->page_size - 1) : 0;
    const int64_t heads = c->heads > 1 ? c->head_stride * (c->heads - 1) : 0;
    return slots > INT32_MAX || heads > INT32_MAX || slots + heads + 256 > INT32_MAX;
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

ss::ScaleCopy scales_of(const ss_cache* src, const ss_cache* dst) {
    ss::ScaleCopy g;
    std::memset(&g, 0, sizeof(g));
    if (!src->scales.block) return g;
    g.src_planes = src->scale_planes;
    g.dst_planes = dst->scale_planes;
    g.src_page = src->scales.page_stride;
    g.src_block = src->scales.block_stride;
    g.src_head = src->scales.head_stride;
    g.dst_page = dst->scales.page_stride;
    g.dst_block = dst->scales.block_stride;
    g.dst_head = dst->scales.head_stride;
    g.block = src->scales.block;
    g.heads = src->cfg.heads;
    g.piece = src->cfg.piece_bytes / 16;
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

ss::Kv8Geo geo_of(const ss_cache* c) {
    ss::Kv8Geo g;
    std::memset(&g, 0, sizeof(g));
    // a dimension of one entry is never stepped, whatever its stride
    g.page = c->cfg.num_pages > 1 ? c->cfg.page_stride : 0;
    g.slot = c->cfg.page_size > 1 ? c->cfg.slot_stride : 0;
    g.head = c->cfg.heads > 1 ? c->cfg.head_stride : 0;
    g.sc_page = c->cfg.num_pages > 1 ? c->scales.page_stride : 0;
    g.sc_block = c->scales.block_stride;
    g.sc_head = c->cfg.heads > 1 ? c->scales.head_stride : 0;
    g.page_size = c->cfg.page_size;
    g.block = c->scales.block;
    g.block_bits = c->scales.block == 16 ? 4 : c->scales.block == 32 ? 5 : 6;
    g.heads = c->cfg.heads;
    g.dim = c->cfg.piece_bytes;
    g.num_pages = c->cfg.num_pages;
    g.max_blocks = c->cfg.max_blocks;
    return g;
}

bool bad_dtype(ss_dtype dt) { return dt != SS_BF16 && dt != SS_F16; }

// Checks of an array of heads: bytes that pieces of 16 need, or single entries.
ss_status check_heads(const ss_heads* h, bool pieces) {
    if (!h || !h->data) return SS_ERR_INVALID_ARG;
    const uintptr_t p = reinterpret_cast<uintptr_t>(h->data);
    if (p & 1) return SS_ERR_INVALID_ARG;
    if (pieces && (p % 16 || h->row_stride % 8 || h->token_stride % 8 || h->head_stride % 8))
        return SS_ERR_UNSUPPORTED;
    return SS_OK;
}

ss::Heads heads_of(const ss_heads* h) {
    if (!h) return {nullptr, 0, 0, 0};
    return {static_cast<uint16_t*>(h->data), h->row_stride, h->token_stride, h->head_stride};
}

bool bad_rotary(const ss_rotary* r, int head_dim) {
    return !r->turns || (reinterpret_cast<uintptr_t>(r->turns) & 7) || r->dim < 2 || r->dim % 2 ||
           r->dim > head_dim;
}

ss::Rotary rotary_of(const ss_rotary* r) {
    if (!r) return {nullptr, 0, 0, 1.0};
    return {r->turns, r->dim, r->interleaved != 0, r->magnitude};
}

// What every call on a scaled cache checks; B = 0 is the caller's to answer.
ss_status check_scaled(const ss_cache* c, const ss_block_tables* t, int32_t B, int32_t N,
                       int32_t k_plane, int32_t v_plane, ss_dtype dt) {
    const ss_status st = check_tables(c, t);
    if (st != SS_OK) return st;
    if (!c->scales.block || bad_dtype(dt)) return SS_ERR_INVALID_ARG;
    if (k_plane < 0 || k_plane >= c->cfg.num_planes || v_plane < 0 || v_plane >= c->cfg.num_planes ||
        k_plane == v_plane)
        return SS_ERR_INVALID_ARG;
    if (B < 0 || B > t->rows || N < 1 || N > (int64_t)c->cfg.max_blocks * c->cfg.page_size)
        return SS_ERR_INVALID_ARG;
    return SS_OK;
}

ss_status check_step(const ss_cache_step* s) {
    if (s->parents && s->N > 64) return SS_ERR_INVALID_ARG;
    for (const void* p : {(const void*)s->base, (const void*)s->counts, (const void*)s->parents,
                          (const void*)s->reserved})
        if (!aligned4(p)) return SS_ERR_INVALID_ARG;
    return SS_OK;
}

ss::Kv8Step step_of(const ss_block_tables* t, const ss_cache_step* s) {
    return {tables_of(t), s->B, s->N, s->base ? s->base : t->len, s->counts, s->parents, s->reserved};
}

ss_status create(const ss_cache_config* cfg, void* const* planes, uint8_t* const* scales,
                 const ss_cache_scales* layout, ss_cache** out) {
    if (!cfg || !planes || !out) return SS_ERR_INVALID_ARG;
    *out = nullptr;
    if (bad_config(cfg)) return SS_ERR_INVALID_ARG;
    if (layout && bad_scales(cfg, layout)) return SS_ERR_INVALID_ARG;
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
        if (!layout) continue;
        if (!scales[i]) return SS_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (scales[j] == scales[i]) return SS_ERR_INVALID_ARG;
    }
    if (layout && unserved_scaled(cfg, low)) return SS_ERR_UNSUPPORTED;
    int ndev = 0;
    if (hipGetDeviceCount(&ndev) != hipSuccess || cfg->device >= ndev) return SS_ERR_HIP;
    ss::DeviceGuard guard(cfg->device);
    if (!guard.ok) return SS_ERR_HIP;
    ss_cache* c = new (std::nothrow) ss_cache();
    if (!c) return SS_ERR_OUT_OF_MEMORY;
    c->cfg = *cfg;
    if (layout) {
        c->scales = *layout;
        c->planes8 = new (std::nothrow) ss::Kv8Plane[cfg->num_planes];
        if (!c->planes8) {
            delete c;
            return SS_ERR_OUT_OF_MEMORY;
        }
        for (int i = 0; i < cfg->num_planes; ++i)
            c->planes8[i] = {static_cast<char*>(planes[i]), scales[i]};
    }
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
    const int64_t o_scales = take(layout ? (int64_t)cfg->num_planes * sizeof(uint8_t*) : 0);
    const int64_t o_pieces = take(layout ? (int64_t)ss::KV8_SPLITS * ss::KV8_COUNTER * 4 : 0);
    const int64_t filled = off;
    const int64_t o_ids = take((int64_t)c->n_chunks * ss::CACHE_REF_CHUNK * 4);
    const int64_t o_cnt = take((int64_t)c->n_chunks * 4);
    const int64_t o_need = take((int64_t)cfg->max_batch * 4);
    const int64_t o_carry = take((int64_t)cfg->max_batch * 4);
    const int64_t o_mark = take((int64_t)cfg->max_batch * cfg->max_blocks * 4);
    const int64_t o_pair = take((int64_t)cfg->num_pages * 4);
    const int64_t o_part = take(layout ? ss::KV8_PART_FLOATS * 4 : 0);
    c->ws_bytes = off;
    if (hipMalloc(&c->ws_base, (size_t)off) != hipSuccess) {
        (void)hipGetLastError();
        delete[] c->planes8;
        delete c;
        return SS_ERR_OUT_OF_MEMORY;
    }
    char* b = static_cast<char*>(c->ws_base);
    c->planes = reinterpret_cast<char**>(b + o_planes);
    c->scale_planes = reinterpret_cast<uint8_t**>(b + o_scales);
    c->pieces = reinterpret_cast<int32_t*>(b + o_pieces);
    c->part = reinterpret_cast<float*>(b + o_part);
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
        delete[] c->planes8;
        delete c;
        return SS_ERR_OUT_OF_MEMORY;
    }
    std::memcpy(h + o_planes, planes, (size_t)cfg->num_planes * sizeof(char*));
    if (layout) std::memcpy(h + o_scales, scales, (size_t)cfg->num_planes * sizeof(uint8_t*));
    const bool ok = hipMemcpy(b, h, (size_t)filled, hipMemcpyHostToDevice) == hipSuccess;
    delete[] h;
    if (!ok) {
        (void)hipFree(c->ws_base);
        delete[] c->planes8;
        delete c;
        return SS_ERR_HIP;
    }
    *out = c;
    return SS_OK;
}

}  // namespace

extern "C" {

ss_status ss_cache_create(const ss_cache_config* cfg, void* const* planes, ss_cache** out) {
    return create(cfg, planes, nullptr, nullptr, out);
}

ss_status ss_cache_create_scaled(const ss_cache_config* cfg, void* const* planes,
                                 uint8_t* const* scales, const ss_cache_scales* layout,
                                 ss_cache** out) {
    if (!scales || !layout) return SS_ERR_INVALID_ARG;
    return create(cfg, planes, scales, layout, out);
}

void ss_cache_destroy(ss_cache* c) {
    if (!c) return;
    ss::DeviceGuard guard(c->cfg.device);
    (void)hipFree(c->ws_base);
    delete[] c->planes8;
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
    return ss::launch_cache_reserve(a, copy_of(c, c), scales_of(c, c), static_cast<hipStream_t>(stream)) == hipSuccess
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
    return ss::launch_cache_commit(a, copy_of(c, c), scales_of(c, c), static_cast<hipStream_t>(stream)) == hipSuccess
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
        s.heads != d.heads || s.piece_bytes != d.piece_bytes ||
        src_cache->scales.block != dst_cache->scales.block)
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
    return ss::launch_cache_copy(a, copy_of(src_cache, dst_cache), scales_of(src_cache, dst_cache),
                                 static_cast<hipStream_t>(stream)) == hipSuccess
               ? SS_OK
               : SS_ERR_HIP;
}

ss_status ss_rotate(int32_t device, const ss_rotary* rotary, ss_dtype dtype, int32_t B, int32_t N,
                    int32_t head_dim, const int32_t* positions, const ss_heads* queries,
                    const ss_heads* out_queries, int32_t q_heads, const ss_heads* keys,
                    const ss_heads* out_keys, int32_t k_heads, void* stream) {
    if (!rotary || bad_dtype(dtype) || B < 0 || N < 0 || (int64_t)B * N > INT32_MAX) return SS_ERR_INVALID_ARG;
    if (head_dim < 1 || head_dim > 65536 || q_heads < 0 || k_heads < 0 || q_heads > 65536 ||
        k_heads > 65536 || q_heads + k_heads < 1 || q_heads + k_heads > 65536)
        return SS_ERR_INVALID_ARG;
    if (bad_rotary(rotary, head_dim)) return SS_ERR_INVALID_ARG;
    if (B == 0 || N == 0) return SS_OK;
    if (!positions || !aligned4(positions)) return SS_ERR_INVALID_ARG;
    ss::RotateArgs a;
    std::memset(&a, 0, sizeof(a));
    bool pieces = head_dim % 16 == 0 && head_dim <= 256 && rotary->dim % 16 == 0;
    const ss_heads* all[4] = {queries, out_queries, keys, out_keys};
    for (int i = 0; i < 4; ++i) {
        if (!(i < 2 ? q_heads : k_heads)) continue;
        const ss_status st = check_heads(all[i], false);
        if (st != SS_OK) return st;
        if (check_heads(all[i], true) != SS_OK) pieces = false;
    }
    a.r = rotary_of(rotary);
    a.positions = positions;
    a.B = B;
    a.N = N;
    a.head_dim = head_dim;
    a.q_heads = q_heads;
    a.k_heads = k_heads;
    if (q_heads) {
        a.q = heads_of(queries);
        a.q_out = heads_of(out_queries);
    }
    if (k_heads) {
        a.k = heads_of(keys);
        a.k_out = heads_of(out_keys);
    }
    a.vectors = pieces;
    ss::DeviceGuard guard(device);
    if (!guard.ok) return SS_ERR_HIP;
    return ss::launch_rotate(a, dtype, static_cast<hipStream_t>(stream)) == hipSuccess ? SS_OK
                                                                                       : SS_ERR_HIP;
}

ss_status ss_cache_write(ss_cache* c, const ss_block_tables* t, const ss_cache_step* step,
                         int32_t k_plane, int32_t v_plane, ss_dtype dtype, const ss_heads* keys,
                         const ss_heads* values, const ss_rotary* rotary,
                         const int32_t* positions, const ss_heads* queries,
                         const ss_heads* out_queries, int32_t q_heads, void* stream) {
    if (!step) return SS_ERR_INVALID_ARG;
    ss_status st = check_scaled(c, t, step->B, step->N, k_plane, v_plane, dtype);
    if (st != SS_OK) return st;
    st = check_step(step);
    if (st != SS_OK) return st;
    if (q_heads < 0 || q_heads > 65536 || (q_heads && !rotary) || !aligned4(positions))
        return SS_ERR_INVALID_ARG;
    if (rotary && bad_rotary(rotary, c->cfg.piece_bytes)) return SS_ERR_INVALID_ARG;
    if (step->B == 0) return SS_OK;
    for (const ss_heads* h : {keys, values, queries, out_queries}) {
        if (!q_heads && (h == queries || h == out_queries)) continue;
        st = check_heads(h, true);
        if (st != SS_OK) return st;
    }
    // a rotated part is a multiple of 16, or divides the head (a half, a quarter of it)
    if (rotary && rotary->dim % 16 && c->cfg.piece_bytes % rotary->dim) return SS_ERR_UNSUPPORTED;
    ss::Kv8Write a;
    std::memset(&a, 0, sizeof(a));
    a.g = geo_of(c);
    a.s = step_of(t, step);
    a.k = c->planes8[k_plane];
    a.v = c->planes8[v_plane];
    a.keys = heads_of(keys);
    a.values = heads_of(values);
    if (q_heads) {
        a.q = heads_of(queries);
        a.q_out = heads_of(out_queries);
    }
    a.q_heads = q_heads;
    a.r = rotary_of(rotary);
    a.positions = positions;
    ss::DeviceGuard guard(c->cfg.device);
    if (!guard.ok) return SS_ERR_HIP;
    return ss::launch_kv8_write(a, dtype, static_cast<hipStream_t>(stream)) == hipSuccess ? SS_OK
                                                                                          : SS_ERR_HIP;
}

ss_status ss_cache_read(ss_cache* c, const ss_block_tables* t, const int32_t* start,
                        const int32_t* counts, int32_t B, int32_t N, int32_t k_plane,
                        int32_t v_plane, ss_dtype dtype, const ss_heads* out_keys,
                        const ss_heads* out_values, void* stream) {
    ss_status st = check_scaled(c, t, B, N, k_plane, v_plane, dtype);
    if (st != SS_OK) return st;
    if (!aligned4(start) || !aligned4(counts)) return SS_ERR_INVALID_ARG;
    if (B == 0 || (!out_keys && !out_values)) return SS_OK;
    ss::Kv8Read a;
    std::memset(&a, 0, sizeof(a));
    a.g = geo_of(c);
    a.t = tables_of(t);
    const ss_heads* out[2] = {out_keys, out_values};
    for (int i = 0; i < 2; ++i) {
        if (!out[i]) continue;
        st = check_heads(out[i], true);
        if (st != SS_OK) return st;
        a.p[a.planes] = c->planes8[i ? v_plane : k_plane];
        a.out[a.planes++] = heads_of(out[i]);
    }
    a.start = start;
    a.counts = counts;
    a.B = B;
    a.N = N;
    ss::DeviceGuard guard(c->cfg.device);
    if (!guard.ok) return SS_ERR_HIP;
    return ss::launch_kv8_read(a, dtype, static_cast<hipStream_t>(stream)) == hipSuccess ? SS_OK
                                                                                         : SS_ERR_HIP;
}

ss_status ss_cache_attend(ss_cache* c, const ss_block_tables* t, const ss_cache_step* step,
                          int32_t k_plane, int32_t v_plane, ss_dtype dtype,
                          const ss_heads* queries, const ss_heads* out, int32_t q_heads,
                          float scale, float* out_lse, void* stream) {
    if (!step) return SS_ERR_INVALID_ARG;
    ss_status st = check_scaled(c, t, step->B, step->N, k_plane, v_plane, dtype);
    if (st != SS_OK) return st;
    st = check_step(step);
    if (st != SS_OK) return st;
    if (q_heads < 1 || q_heads > 65536 || q_heads % c->cfg.heads || !aligned4(out_lse)) return SS_ERR_INVALID_ARG;
    // rows and a block of 128 of them behind the last are counted in 32 bits
    if ((int64_t)step->N * (q_heads / c->cfg.heads) > INT32_MAX - 128) return SS_ERR_INVALID_ARG;
    // times a block's scale, 2^-60 to 2^60, neither 0 nor an infinity, which masked or zero scores
    // would turn into a NaN
    if (!(scale >= 0x1p-60f && scale <= 0x1p60f)) return SS_ERR_INVALID_ARG;
    if (step->B == 0) return SS_OK;
    for (const ss_heads* h : {queries, out}) {
        st = check_heads(h, true);
        if (st != SS_OK) return st;
    }
    ss::Kv8Attend a;
    std::memset(&a, 0, sizeof(a));
    a.g = geo_of(c);
    a.s = step_of(t, step);
    a.k = c->planes8[k_plane];
    a.v = c->planes8[v_plane];
    a.q = heads_of(queries);
    a.out = heads_of(out);
    a.lse = out_lse;
    a.q_heads = q_heads;
    a.group = q_heads / c->cfg.heads;
    a.scale_log2 = scale * 1.44269504088896341f;
    a.part = c->part;
    a.arrived = c->pieces;
    ss::DeviceGuard guard(c->cfg.device);
    if (!guard.ok) return SS_ERR_HIP;
    return ss::launch_kv8_attend(a, dtype, static_cast<hipStream_t>(stream)) == hipSuccess ? SS_OK
                                                                                           : SS_ERR_HIP;
}

}  // extern "C"
