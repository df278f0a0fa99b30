// Internal structures shared by the host side of the library and its kernels.
#pragma once

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ss_sampler.h"

namespace ss {

// Stage-1 summary of one 2048-entry wave tile of one row (32 bytes).
//  * Candidates are written as keys (z, id), unsorted, in cand[row][wave tile].
//  * Every finite entry of the wave tile that is not a candidate has
//    z <= zbeta; zbeta = -inf when every finite entry is a candidate.
struct WaveStat {
    float m;        // max processed logit x' (-inf if none is finite)
    int argmax;     // greedy rows: lowest id attaining m; -1 otherwise
    float zbeta;    // RN(beta / T) of the cut beta in x' (x' < beta, window; x' <= beta, count)
    int ncand;      // candidates written (<= WCAP)
    int nfinite;    // finite processed logits
    int flags;      // WS_OVF, WS_SUM, WS_APX
    float zmin;     // smallest z among the candidates (+inf: none)
    float zm;       // RN(m / T), the z of the maximum (T > 0)
    double s;       // WS_SUM / WS_APX: a mass relative to exp(zm)
    double sc;      // the candidates' mass relative to exp(zm) (binary32 terms)
};
static_assert(sizeof(WaveStat) == 48, "WaveStat layout");

// The window held more than WCAP entries: the candidates are the head of the
// wave tile by count instead.
constexpr int WS_OVF = 1;
// s holds the wave tile's whole mass, exact (count-cut tiles of rows top-k may
// not cut).
constexpr int WS_SUM = 2;
// s holds the mass of the wave tile's non-candidates, relative to RN(m / T) and
// approximate (window-cut tiles of rows top-k may not cut).
constexpr int WS_APX = 4;
// Neither flag: the tile holds more finite entries than the row's top-k, so the
// row is cut by top-k and the mass outside the candidates is not summed (the
// merge bounds what a top-k set deeper than the pool can miss by count).
// With WS_SUM: the tile's non-candidates' mass is also binned by z (Workspace::bins).
constexpr int WS_BIN = 8;
// Bins of a WS_BIN tile: BIN_S per unit of z on the absolute grid floor(-z BIN_S),
// NBIN of them from the one holding the tile's zbeta down; the last also holds
// everything deeper.
constexpr int BIN_S = 32;
constexpr int NBIN = 256;

// What the row finaliser knows about one row's filtered distribution.
// kept(v) <=> key64(z_v, v) >= kappa and (min_p <= 0 or exp(z_v - zmax) >= min_p),
// pi(v) = kept(v) ? exp(z_v - zmax) / W : 0.
struct RowInfo {
    unsigned long long kappa;
    double W;
    float zmax;
    float min_p;
    int n_kept;
    int token;      // sampled token (ss_sample and the bonus row), greedy token for T = 0
    int argmax;     // lowest id among the maxima of x'
    int path;       // 0 tile candidates, 1 whole-row fallback
    int pad[2];
};
static_assert(sizeof(RowInfo) == 48, "RowInfo layout");

// Per-row view of the caller's parameters, as device pointers (host-built;
// every pointer but mask is valid: absent parameters point at defaults).
struct ParamPtrs {
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    const float* rep;
    const float* freq;
    const float* pres;
    const int32_t* hist_ids;
    const int32_t* hist_len;
    int32_t hist_stride;
    const int32_t* bias_ids;
    const float* bias_vals;
    const int32_t* bias_len;
    int32_t bias_stride;
    const uint32_t* mask;
    int32_t mask_stride;
    const int32_t* request_ids;
    const int32_t* positions;
    uint64_t seed;
};

struct Workspace {
    WaveStat* wstats;        // [max_rows * n_wt]
    unsigned long long* cand;  // [max_rows * n_wt * WCAP]  candidate keys per wave tile
    RowInfo* rowinfo;        // [max_rows]
    int32_t* row_accept;     // [max_rows]: spec decision per draft row
    double2* resid_tile;     // [max_batch * n_tiles]: residual / target mass per tile
    float* scratch_z;        // [max_rows * V] fallback rows
    float* bins;             // [max_batch * n_wt * NBIN] WS_BIN tiles' masses by z, or null
    int32_t* tree_path;      // [max_rows * tree_dmax]: tokens from the root to each tree node
    int32_t* tree_depth;     // [max_rows]: depth of each tree node (-1: unreachable)
    int32_t* tree_next;      // [max_rows]: accepted child of each tree node (-1: none)
    int tree_dmax;           // path stride (the deepest path a tree of the handle can have)
    int n_tiles;             // 8192-entry workgroup tiles per row
    int n_wt;                // wave tiles per row (WPT per workgroup tile)
    int V;
};

struct SampleArgs {
    const void* logits;
    int64_t row_stride;
    int B;
    int V;
    ParamPtrs p;
    int32_t* out_tokens;
    float* dbg_processed;
    int32_t* dbg_topk;
    int32_t dbg_topk_stride;
    int32_t* dbg_kept;
    float* dbg_probs;
    int32_t* dbg_path;
    Workspace ws;
};

struct SpecArgs {
    const void* target;
    int64_t row_stride;
    const float* draft_probs;  // null: greedy draft, q one-hot at the draft token
    int64_t draft_stride;
    const int32_t* draft_tokens;
    int B;
    int G;
    int V;
    ParamPtrs p;
    int32_t* out_tokens;
    int32_t* out_num_accepted;
    int32_t* seq_tokens;       // null: no append to the request sequences
    int64_t seq_stride;
    int32_t seq_capacity;
    int32_t* seq_len;
    Workspace ws;
};

struct TreeArgs {
    const void* target;        // [B * N] rows: row b * N + n after the path root -> n
    int64_t row_stride;
    const int32_t* parents;    // [B, N]
    const int32_t* tokens;     // [B, N]
    int B;
    int N;
    int V;
    ParamPtrs p;
    int32_t* out_tokens;       // [B, N]
    int32_t* out_nodes;        // [B, N]
    int32_t* out_num_accepted; // [B]
    Workspace ws;
};

// Per (batch row, LM-head vocabulary tile) summary left by the processed
// epilogue: the tile's LM_NC largest keys (z', id) in key order, the next one
// (every other entry of the tile is at most it), the mass below the tile
// maximum, the best Gumbel score and the count of finite entries.
constexpr int LM_NC = 4;
struct LmTileStat {
    unsigned long long key[LM_NC];  // descending; 0 = none
    unsigned long long rest;        // 0 = none
    float mass;                     // sum of exp(z' - z'(key[0])) over the finite entries
    float best_s;                   // the largest z' + g (T > 0) or x' (T = 0)
    int best_i;                     // its id (the lowest among equals), INT_MAX if none
    int nfinite;
    float zmin;                     // the least finite z' (+inf if none)
    int pad;
};
static_assert(sizeof(LmTileStat) == 64, "LmTileStat layout");

// The kept set of an open LM-head row, fixed by the whole-row selection, and
// the best (z' + g, id) key its chunks have found (0 = none yet).
struct LmCut {
    unsigned long long kP;    // kept: key64(z', v) >= kP ...
    unsigned long long best;  // mono32(z' + g) << 32 | ~id, the maximum over the chunks
    float zmax;               // ... and, with min_p > 0, exp(z' - zmax) >= min_p
    float mp;
    float zlo;                // the row's least finite z'
    int total;                // its finite entries
};
static_assert(sizeof(LmCut) == 32, "LmCut layout");

struct LmheadArgs {
    const uint16_t* hidden;
    const uint16_t* weight;
    int B;
    int K;
    int V;
    const float* temperature;
    const int32_t* request_ids;
    const int32_t* positions;
    uint64_t seed;
    int32_t* out_tokens;
    float* debug_logits;
    float2* partials;        // [64 * n_vtiles] (score, id bits)
    int n_vtiles;
    // the per-request pipeline in the epilogue (ss_lmhead_sample_params)
    ParamPtrs p;
    LmTileStat* stats;       // [64 * n_vtiles]
    int32_t* unres;          // [64]: rows the candidates could not resolve
    LmCut* cut;              // [64]: their kept sets and best keys
    float* zmat;             // [64 * V]: z' of those rows, formed again
    int32_t* dbg_path;       // [B] or null: 0 candidates, 1 whole row, 2 no filter or greedy
};

// Verification against probability rows with the caller's uniforms. Counters
// stand this many integers apart: in one line they would be counted one by one.
constexpr int PROBS_COUNTER = 64;
struct ProbsArgs {
    const void* target;        // [B * (G + 1)] rows
    int64_t target_stride;
    const void* draft;         // [B * G] rows, or null: one-hot drafts
    int64_t draft_stride;
    const int32_t* draft_tokens;
    const int32_t* draft_len;  // [B] or null: G drafts each
    const float* uniforms;     // [B, G + 1]
    int B;
    int G;
    int V;
    int32_t* out_tokens;
    int32_t* out_num_accepted;
    int32_t* seq_tokens;       // null: no append to the request sequences
    int64_t seq_stride;
    int32_t seq_capacity;
    int32_t* seq_len;
    double* part;              // [B * n_chunks]: residual mass per 2048-entry chunk
    int n_chunks;
    int32_t* arrived;          // [B * PROBS_COUNTER]: workgroups of each request that have left their sums; 0
                               //      between calls
};

// LM-head logits from 4-bit weights.
struct QuantArgs {
    const uint16_t* hidden;    // [B, K] bfloat16
    const uint8_t* qweight;    // [V, K / 2]
    const uint16_t* scales;    // [V, ceil(K / group)]
    const uint8_t* zeros;      // [V, ceil(groups / 2)], or null: 8
    int scale_f16;
    int group;
    int B;
    int K;
    int V;
    void* out;
    int out_bf16;
    int64_t out_stride;
    // row blocks whose K is cut in parts, behind the whole ones (set by the launch)
    int whole_blocks, split_blocks, split, split_stages;
    uint64_t* part;            // [quant_part_bytes]: the parts' sums
    int32_t* arrived;          // [QUANT_CUS * QUANT_COUNTER]: parts of each row block that have left
                               //   their sums; 0 between calls
};
constexpr int QUANT_CUS = 256;
constexpr int QUANT_COUNTER = 64;  // integers between counters
constexpr int QUANT_SPLIT = 8;     // parts of a row block at most; of all, one a CU
struct QuantSplit {
    int whole_blocks, split_blocks, split, sets;
};

// ---------------------------------------------------------------------------
// page cache

constexpr int CACHE_REF_CHUNK = 4096;   // page counts listed by one workgroup
constexpr int CACHE_MAX_CHUNKS = 1024;
constexpr int CACHE_COUNTER = 64;       // integers between counters: in one line they would be
                                        //   counted one by one
constexpr int CACHE_GROUPS = 256;       // groups of rows whose settling is counted apart
constexpr int CACHE_MAX_PAGES = CACHE_REF_CHUNK * CACHE_MAX_CHUNKS;

struct CacheTables {
    int32_t* tables;  // [rows, stride]
    int64_t stride;
    int32_t rows;
    int32_t* ref;     // [num_pages]
    int32_t* len;     // [rows]
};

// How slots of one cache are copied to slots of another (or the same): strides
// in bytes, a piece of one head is `units` vectors of `vec` bytes.
struct CacheCopy {
    const char* const* src_planes;  // device array
    char* const* dst_planes;
    int64_t src_page, src_slot, src_head;
    int64_t dst_page, dst_slot, dst_head;
    int heads;
    int units;
    int vec;
    int joined;  // consecutive slots of a head follow each other on both sides
};

// The scales of a cache held in 8 bits, both sides of a copy (src null: it has none).
struct ScaleCopy {
    const uint8_t* const* src_planes;  // device array
    uint8_t* const* dst_planes;
    int64_t src_page, src_block, src_head;  // bytes
    int64_t dst_page, dst_block, dst_head;
    int block;   // slots that share a scale
    int heads;
    int piece;   // vectors of 16 bytes of a slot's head
};

struct CacheWork {
    int32_t* free_ids;  // [chunks * CACHE_REF_CHUNK]: free pages, ascending within a chunk
    int32_t* free_cnt;  // [chunks]
    int32_t* need;      // [max_batch]: fresh pages a request needs, -1 refused
    int32_t* carry;     // [max_batch]: shared page whose first slots move along, or -1
    int32_t* mark;      // [max_batch * max_blocks]; in a commit: pages that rows left and others hold
    int32_t* pair_ok;   // [num_pages]
    int32_t* arrived;   // [max_batch * CACHE_COUNTER]: workgroups of each row that have read its
                        //   table; 0 between calls
    unsigned long long* settled;  // [1 + CACHE_GROUPS], CACHE_COUNTER integers apart: groups of a
                        //   commit, and rows of each group, that are settled (low half) and the
                        //   entries that they left (high half); 0 between calls
    int32_t* n_left;    // places taken in the list in mark; 0 between calls
};

struct CacheReserve {
    CacheTables t;
    CacheWork ws;
    const int32_t* base;
    const int32_t* add;
    int B;
    int32_t* out_ok;
    int num_pages, num_planes, page_size, max_blocks, n_chunks;
};

struct CacheTruncate {
    CacheTables t;
    const int32_t* rows;     // null: 0 .. n - 1
    const int32_t* new_len;  // null: 0
    int n;
    int num_pages, page_size, max_blocks;
};

struct CacheFork {
    CacheTables t;
    const int32_t* src;
    const int32_t* dst;
    int n;
    int32_t* out_ok;
    int num_pages, page_size, max_blocks;
};

struct CacheCommit {
    CacheTables t;
    const int32_t* base;
    const int32_t* num_accepted;
    const int32_t* nodes;    // null: a linear draft, nothing moves
    int64_t nodes_stride;
    int N;
    int B;
    int release;
    const int32_t* reserved;  // [B] or null: the reserve's verdicts
    int32_t* arrived;
    unsigned long long* settled;
    int32_t* n_left;
    int32_t* left;
    int group;               // rows per group of the counters in settled
    int32_t* out_ok;
    int num_pages, num_planes, page_size, max_blocks;
};

struct CachePages {
    const int32_t* src;
    const int32_t* dst;
    int n;
    int same;
    int src_pages, dst_pages;
    int num_planes, page_size;
    int32_t* pair_ok;
    int32_t* out_ok;
};

// ---------------------------------------------------------------------------
// a cache held in 8 bits

constexpr int KV8_XMIN = -60, KV8_XMAX = 60;  // exponents of a block's scale

// One plane of a scaled cache with its scales, all strides in bytes.
struct Kv8Plane {
    char* data;
    uint8_t* scales;
};

struct Kv8Geo {
    int64_t page, slot, head;      // of the planes
    int64_t sc_page, sc_block, sc_head;
    int page_size, block, block_bits, heads, dim;  // a block has 2^block_bits slots
    int num_pages, max_blocks;
};

// A step's tokens (ss_cache_step with what the handle knows).
struct Kv8Step {
    CacheTables t;
    int B, N;
    const int32_t* base;
    const int32_t* counts;
    const int32_t* parents;
    const int32_t* reserved;
};

struct Heads {  // strides in elements
    uint16_t* data;
    int64_t row, token, head;
};

struct Rotary {
    const double* turns;
    int dim;
    int interleaved;
    double magnitude;
};

struct RotateArgs {
    Rotary r;
    const int32_t* positions;
    int B, N, head_dim, q_heads, k_heads;
    Heads q, q_out, k, k_out;
    int vectors;  // pieces of 16 bytes; else single entries
};

struct Kv8Write {
    Kv8Geo g;
    Kv8Step s;
    Kv8Plane k, v;
    Heads keys, values, q, q_out;
    int q_heads;      // 0: no queries
    Rotary r;         // turns null: keys stay
    const int32_t* positions;
};

struct Kv8Read {
    Kv8Geo g;
    CacheTables t;
    Kv8Plane p[2];
    Heads out[2];
    int planes;
    const int32_t* start;
    const int32_t* counts;
    int B, N;
};

// Attention: a workgroup takes a share of the requests' slots, for one head of the cache and a
// block of rows (query heads of tokens). What it sums up of requests that others go on with
// lies in `part`.
struct Kv8Attend {
    Kv8Geo g;
    Kv8Step s;
    Kv8Plane k, v;
    Heads q, out;
    float* lse;
    int q_heads;
    int group;        // query heads per head of the cache
    int blocks;       // blocks of rows of one request and head
    int shares;       // that the slots of a head and block of rows over all requests are cut
                      //   into; 0: none is cut
    float scale_log2; // scale * log2(e)
    float* part;
    int32_t* arrived;
};

constexpr int KV8_COUNTER = 64;       // integers between counters
constexpr int KV8_SPLITS = 1024;      // shares, over heads and blocks of rows, at most
constexpr int64_t KV8_PART_FLOATS = 9 << 20;  // what shares leave, at most

// Optional timing events of a call (see ss_sampler_set_launch_events): launch
// k is bracketed by ev[2k] (its start) and ev[2k + 1] (its end), recorded by
// the dispatch itself.
struct LaunchEvents {
    hipEvent_t ev[16];
    int n;
    hipEvent_t start(int k) const { return 2 * k + 1 < n ? ev[2 * k] : nullptr; }
    hipEvent_t stop(int k) const { return 2 * k + 1 < n ? ev[2 * k + 1] : nullptr; }
};

// Launches kernel k of a call, with its timing events when they are set.
template <class F, class... A>
inline void launch_k(const LaunchEvents& le, int k, F kernel, dim3 grid, dim3 block,
                     hipStream_t st, A... args) {
    if (le.start(k))
        hipExtLaunchKernelGGL(kernel, grid, block, 0, st, le.start(k), le.stop(k), 0, args...);
    else
        hipLaunchKernelGGL(kernel, grid, block, 0, st, args...);
}

hipError_t launch_sample(const SampleArgs& a, ss_dtype dt, hipStream_t st, const LaunchEvents& le);
hipError_t launch_spec(const SpecArgs& a, ss_dtype dt, hipStream_t st, const LaunchEvents& le);
hipError_t launch_tree(const TreeArgs& a, ss_dtype dt, hipStream_t st, const LaunchEvents& le);
hipError_t launch_lmhead(const LmheadArgs& a, hipStream_t st, const LaunchEvents& le);
hipError_t launch_lmhead_params(const LmheadArgs& a, hipStream_t st, const LaunchEvents& le);
hipError_t launch_probs(const ProbsArgs& a, ss_dtype dt, hipStream_t st, const LaunchEvents& le);
hipError_t launch_quant(const QuantArgs& a, hipStream_t st, const LaunchEvents& le);
// what the parts' sums of any call with these limits take
int64_t quant_part_bytes(int V, int K, int max_batch);
hipError_t launch_cache_reserve(const CacheReserve& a, const CacheCopy& g, const ScaleCopy& sc,
                                hipStream_t st);
hipError_t launch_cache_truncate(const CacheTruncate& a, hipStream_t st);
hipError_t launch_cache_fork(const CacheFork& a, hipStream_t st);
hipError_t launch_cache_commit(const CacheCommit& a, const CacheCopy& g, const ScaleCopy& sc,
                                hipStream_t st);
hipError_t launch_cache_copy(const CachePages& a, const CacheCopy& g, const ScaleCopy& sc,
                                hipStream_t st);
hipError_t launch_rotate(const RotateArgs& a, ss_dtype dt, hipStream_t st);
hipError_t launch_kv8_write(const Kv8Write& a, ss_dtype dt, hipStream_t st);
hipError_t launch_kv8_read(const Kv8Read& a, ss_dtype dt, hipStream_t st);
hipError_t launch_kv8_attend(const Kv8Attend& a, ss_dtype dt, hipStream_t st);
// the row kernels of ss_lmhead_sample_params (in the row-kernel source)
void launch_lm_merge(const LmheadArgs& a, hipStream_t st, const LaunchEvents& le, int k);
void launch_lm_slow(const LmheadArgs& a, hipStream_t st, const LaunchEvents& le, int k);
void launch_lm_gumbel(const LmheadArgs& a, hipStream_t st, const LaunchEvents& le, int k);

}  // namespace ss
