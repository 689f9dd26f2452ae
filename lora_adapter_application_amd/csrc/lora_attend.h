// lora_attend.h -- launch interface between the host side (lora_attend.cpp) and the kernels
// between a layer's projections: head norms with rotary positions (lora_norm.hip), the paged
// cache (lora_cache.hip) and attention over it (lora_attend.hip); and the index arithmetic that
// the kernels share with the host's checks.  Not installed; not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lora_layer.h"

namespace lora {

// ---------------------------------------------------------------------------
// head norms with rotary positions

struct NormArgs {
    RotaryArgs rot;
    const void *weight[kMaxGroup];   // [head_dim] or null (1)
    float eps;
};
hipError_t launch_norm_rotary(bool bf16, bool vec, const NormArgs &a, hipStream_t st);

// ---------------------------------------------------------------------------
// the cache
//
// Tokens are held in blocks of 32 of one key-value head, a block's keys, values and scales
// together, in the order in which the attention's matrix instructions take them:
//
//     keys    [dim / 8][32 tokens][8 dims]      a lane's 8 inputs of q . k stand together
//     values  [4][dim][8 tokens]                a lane's 8 inputs of p . v stand together
//     scales  [32] of the keys, [32] of the values (8 bits only), float
//
// with dim padded to 64, 96, 128 or 256; padding stays zero.  A page holds
// [kv_heads][page_size / 32] blocks.
constexpr int kBlock = 32;

enum CacheKind : int32_t { kCacheNative = 0, kCacheFp8 = 1, kCacheInt8 = 2 };

__host__ __device__ inline int padded_dim(int d) { return d <= 64 ? 64 : d <= 96 ? 96 : d <= 128 ? 128 : 256; }
__host__ __device__ inline int key_at(int tok, int d) { return ((d >> 3) * kBlock + tok) * 8 + (d & 7); }
__host__ __device__ inline int value_at(int dp, int tok, int d) { return ((tok >> 3) * dp + d) * 8 + (tok & 7); }

struct CacheView {
    char *base;
    int32_t kind;
    int32_t kv_heads, head_dim, dp;
    int32_t page_shift;              // page_size = 1 << page_shift, at least kBlock
    int32_t pages;
    int32_t elem;                    // bytes of a held element
    int32_t half;                    // bytes of a block's keys, and of its values
    int32_t block;                   // bytes of a block
};

__host__ __device__ inline int64_t cache_block(const CacheView &c, int page, int head, int block_in_page)
{
    return (((int64_t)page * c.kv_heads + head) * (1 << (c.page_shift - 5)) + block_in_page) * c.block;
}

struct CacheArgs {
    CacheView c;
    const void *k_in, *v_in;         // store: [T][kv_heads * head_dim]
    void *k_out, *v_out;             // load
    const int32_t *slots;            // [T]
    int32_t T;
    uint32_t *flags;
};
hipError_t launch_cache_store(bool bf16, const CacheArgs &a, hipStream_t st);
hipError_t launch_cache_load(bool bf16, const CacheArgs &a, hipStream_t st);

// ---------------------------------------------------------------------------
// attention
//
// Work is cut in tiles: up to R rows (a row is a query head of a new token, the heads of one
// key-value head counted on through the tokens) of one request over its own pages, or of the
// requests of one prefix over the prefix's pages.  Two lists of tiles, each for its kernel:
// narrow tiles of 16 rows, whose four waves share the tokens, and wide ones of 128 rows, whose
// four waves share the rows.  A tile's tokens are cut in units; the units of a list, key-value
// head by key-value head, are dealt to its workers (workgroups) in equal runs.  A worker that
// holds a tile whole writes the result; else parts (maximum, sum, weighted values) are kept and
// joined afterwards.
constexpr int kNarrowRows = 16, kNarrowUnit = 128;
constexpr int kWideRows = 128, kWideUnit = 64;
// A request of more rows than this (of one key-value head) goes by itself over its prefix:
// its tiles are as wide as the shared ones, so sharing would save nothing and cost the parts.
constexpr int kShareRows = 32;
// Workers are the workgroups of 256 threads that the chip's 256 CUs hold at once: as many of a
// kernel on a CU as its registers and LDS leave room for.
constexpr int kAttendCus = 256, kAttendWorkers = 4 * kAttendCus;   // at most
constexpr int kAttendPerCu(int elem, int kind, int dp)             // narrow tiles
{
    return dp > 128 ? (elem == 4 && kind == 0 ? 1 : 2) : dp > 96 ? (elem == 4 && kind == 0 ? 2 : 3)
         : dp > 64 && kind == 0 ? 3 : 4;
}

struct alignas(16) AttendTile {
    int32_t seq;                 // request, or prefix if `shared`
    int32_t shared;              // rows come from the list of the prefix's tokens
    int32_t token0;              // first new token of the request, or of the prefix in its list
    int32_t row0, rows;          // the tile's rows of the request or prefix
    int32_t pre_len;             // tokens of the prefix it reads by itself, before its own
    int32_t len, q_len;          // own tokens held, new tokens (shared: the prefix's length, 0)
    int32_t unit0, units;        // units before the tile, and its own, of one key-value head
    int32_t kept;                // its number among the tiles whose parts are always kept, or -1
    int32_t prefix;              // prefix whose shared tiles hold the other part, or -1
    int32_t pre_row;             // the row of the list of all such tokens at which this tile starts
    int32_t pre_seq;             // prefix read by itself (pre_len > 0)
    int32_t pad[2];
};

struct AttendList {
    int32_t tiles, units, kept;
    int32_t run;                 // units a worker takes
};

// What the plan leaves for the launches.
struct AttendPlan {
    AttendList list[2];          // narrow, wide
    int32_t bad;                 // the batch does not fit what the host was told: no work
    int32_t pad[7];
};

// A prefix's first shared tile.
struct PrefixTile { int32_t list, tile; };

struct AttendBatch {
    const int32_t *q_start, *lengths, *pages;
    const int32_t *prefix_seqs, *prefix_lengths, *prefix_pages;
    int32_t n_tokens, n_seqs, n_prefixes;
    int32_t max_pages, prefix_max_pages;
    int32_t max_queries;
    int32_t group;               // query heads of a key-value head
    int32_t kv_heads;
    int32_t page_shift;
    int32_t wide;                // wide tiles may be used
    int32_t workers[2];          // of the lists' kernels
    int32_t units_fit;           // no batch of these sizes has more than 2^29 units
    uint32_t group_mul, group_shift;   // x / group is (x + the high word of x group_mul) >> group_shift
    int32_t simple;              // planned by each launch for itself (simple_batch)
    // workspace, all written by the plan
    AttendPlan *plan;
    AttendTile *tiles[2];
    int32_t cap[2];              // tiles a list can hold
    int32_t kept_cap[2];         // kept tiles a list can hold
    int32_t *start[2];           // [workers] tile at which a worker starts
    int32_t *list_before;        // [n_seqs + 1] listed tokens (of requests that share) before a request
    int32_t *listed;             // [n_tokens] those tokens
    PrefixTile *prefix_tile;     // [n_prefixes]
    uint32_t *flags;
};

__host__ __device__ inline int clamp_to(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// What the arrays say of request i.
struct Request { int32_t start, end, length; };
__host__ __device__ inline Request request_words(const AttendBatch &b, int i)
{
    return {b.q_start ? b.q_start[i] : i, b.q_start ? b.q_start[i + 1] : i + 1, b.lengths[i]};
}

// The new tokens first..end of a request, and whether the starts are in order.
struct Queries { int32_t first, count; bool bad; };
__host__ __device__ inline Queries queries_of(const AttendBatch &b, const Request &r)
{
    const int first = clamp_to(r.start, 0, b.n_tokens), end = clamp_to(r.end, first, b.n_tokens);
    const int most = end - first < b.max_queries ? end - first : b.max_queries;
    return {first, most, r.start != first || r.end != end || most != end - first};
}

// A length bounded by what a row of the table of pages can name.
__host__ __device__ inline int held_of(int n, int max_pages, int page_shift, bool *bad)
{
    const int64_t most = (int64_t)max_pages << page_shift;
    const int fit = most < n ? (int)most : n;
    *bad |= n < 0 || fit != n;
    return fit < 0 ? 0 : fit;
}

// The prefix whose requests include i, or -1.
__host__ __device__ inline int prefix_of(const AttendBatch &b, int i)
{
    int lo = 0, hi = b.n_prefixes;           // the last p with prefix_seqs[p] <= i
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (b.prefix_seqs[mid] <= i)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo < b.n_prefixes && b.prefix_seqs[lo] <= i && i < b.prefix_seqs[lo + 1] ? lo : -1;
}

// One request, or one prefix with the requests that share it: its tiles.
struct AttendEntity {
    int32_t seq, shared;         // request, or prefix
    int32_t list, tiles;         // 0 narrow, 1 wide
    int32_t keeps;               // its tiles' parts are always kept
    int32_t token0, rows;
    int32_t len, q_len;
    int32_t pre_len, pre_seq;    // prefix read by itself
    int32_t prefix;              // prefix that the shared tiles read for it, or -1
    int32_t listed;              // tokens it adds to the list of that prefix
};

__host__ __device__ inline int units_for(int64_t tokens, int unit) { return (int)((tokens + unit - 1) / unit); }
// total / workers rounded up, for workers a multiple of 256 and total below 2^39, by a division of 32 bits
__host__ __device__ inline int32_t worker_run(int64_t total, int workers)
{
    const uint32_t k = (uint32_t)workers >> 8;
    return (int32_t)(((uint32_t)((total + 255) >> 8) + k - 1) / k);
}
__host__ __device__ inline int list_rows(int l) { return l ? kWideRows : kNarrowRows; }
__host__ __device__ inline int list_unit(int l) { return l ? kWideUnit : kNarrowUnit; }
__host__ __device__ inline int share_rows(int group) { return group > kShareRows ? group : kShareRows; }

__host__ __device__ inline AttendEntity request_of(const AttendBatch &b, int i, const Request &r, bool *bad)
{
    AttendEntity t{};
    const Queries q = queries_of(b, r);
    *bad |= q.bad;
    t.seq = i;
    t.len = held_of(r.length, b.max_pages, b.page_shift, bad);
    t.prefix = -1;
    t.pre_seq = -1;
    if (!q.count)
        return t;
    t.token0 = q.first;
    t.q_len = q.count;
    t.rows = q.count * b.group;
    const int p = prefix_of(b, i);
    const int pre = p < 0 ? 0 : held_of(b.prefix_lengths[p], b.prefix_max_pages, b.page_shift, bad);
    t.keeps = pre > 0 && t.rows <= share_rows(b.group);
    t.list = b.wide && t.rows > kShareRows;
    t.tiles = units_for(t.rows, list_rows(t.list));
    t.pre_len = t.keeps ? 0 : pre;
    t.pre_seq = p;
    t.prefix = t.keeps ? p : -1;
    t.listed = t.keeps ? q.count : 0;
    return t;
}

// The shared tiles of prefix p, whose requests list `listed` tokens from list0 on.
__host__ __device__ inline AttendEntity prefix_of_batch(const AttendBatch &b, int p, int list0, int listed, bool *bad)
{
    AttendEntity t{};
    t.seq = p;
    t.shared = 1;
    t.prefix = t.pre_seq = -1;
    t.len = held_of(b.prefix_lengths[p], b.prefix_max_pages, b.page_shift, bad);
    if (t.len <= 0 || listed <= 0)
        return t;
    t.token0 = list0;
    t.rows = listed * b.group;
    t.keeps = 1;
    t.list = b.wide && t.rows > kShareRows;
    t.tiles = units_for(t.rows, list_rows(t.list));
    return t;
}

// Batches that need no plan kernel: one new token a request, no prefixes, and requests whose rows
// are one narrow tile each, so few that a workgroup sums their units itself.
constexpr int kSimpleSeqs = 256;
inline bool simple_batch(const AttendBatch &b)
{
    return !b.q_start && !b.n_prefixes && b.n_seqs <= kSimpleSeqs && b.group <= kNarrowRows;
}
__host__ __device__ inline AttendTile simple_tile(int seq, int len, int group, int unit0)
{
    AttendTile t{};
    t.seq = t.token0 = seq;
    t.rows = group;
    t.len = len;
    t.q_len = 1;
    t.unit0 = unit0;
    t.units = len > 0 ? units_for(len, kNarrowUnit) : 1;
    t.kept = t.prefix = t.pre_seq = -1;
    return t;
}

// x / group for 0 <= x < 2^31, and the numbers that it takes.
__host__ __device__ inline int32_t over_group(const AttendBatch &b, int32_t x)
{
    return (int32_t)(((uint32_t)(((uint64_t)(uint32_t)x * b.group_mul) >> 32) + (uint32_t)x) >> b.group_shift);
}
inline void set_group(AttendBatch &b, int32_t group)
{
    b.group = group;
    b.group_shift = 0;
    while ((1u << b.group_shift) < (uint32_t)group)
        ++b.group_shift;
    b.group_mul = (uint32_t)((((1ull << b.group_shift) - group) << 32) / group + 1);
}

// Tile j of an entity; `list0`: where the list of tokens that share has the request's first.
__host__ __device__ inline AttendTile tile_of(const AttendBatch &b, const AttendEntity &e, int j, int list0)
{
    const int R = list_rows(e.list), unit = list_unit(e.list);
    AttendTile t{};
    t.seq = e.seq;
    t.shared = e.shared;
    t.token0 = e.token0;
    t.row0 = j * R;
    t.rows = e.rows - t.row0 < R ? e.rows - t.row0 : R;
    t.len = e.len;
    t.q_len = e.q_len;
    t.pre_len = e.pre_len;
    t.pre_seq = e.pre_seq;
    t.prefix = e.prefix;
    t.pre_row = e.prefix >= 0 ? list0 * b.group + t.row0 : 0;
    if (e.shared) {
        t.units = units_for(e.len, unit);
    } else {
        // its prefix where it reads that by itself, and its own tokens up to the last one
        // that its last row sees
        const int last = over_group(b, t.row0 + t.rows - 1);
        const int seen = e.len - e.q_len + last + 1;
        t.units = units_for(e.pre_len, unit) + units_for(seen < 0 ? 0 : seen, unit);
        if (t.units < 1)
            t.units = 1;                                   // a row that sees nothing is written too
    }
    return t;
}

// Whether a batch may be worked on: no token claimed twice, by requests (`tokens` new ones in all) or by
// prefixes (`listed`), no more than 2^29 units, and then, as the capacities are made, every list
// within its own (count: tiles of the lists, kept tiles, ...).
__host__ __device__ inline bool attend_fits(const AttendBatch &b, unsigned long long tokens, unsigned long long listed,
                                            unsigned long long units, const int32_t *count)
{
    return tokens <= (unsigned long long)b.n_tokens && listed <= (unsigned long long)b.n_tokens && units <= 1ull << 29 &&
           count[0] <= b.cap[0] && count[1] <= b.cap[1] && count[2] <= b.kept_cap[0] && count[3] <= b.kept_cap[1];
}

// Where worker w keeps its part of a tile of key-value head `head`: a kept tile's parts follow
// those of the tiles before it; of the others a worker has at most two, the one that starts
// before its run and the one that ends behind it.
__host__ __device__ inline int64_t part_slot(const AttendList &l, int workers, int head, const AttendTile &t, int w)
{
    if (t.kept >= 0)
        return 2ll * workers + (int64_t)head * l.kept + t.kept + w;
    const int64_t at = (int64_t)head * l.units + t.unit0;
    return 2ll * w + (at < (int64_t)w * l.run ? 0 : 1);
}
__host__ __device__ inline int64_t part_slots(int workers, int kept_cap, int kv_heads)
{
    return 3ll * workers + (int64_t)kept_cap * kv_heads;
}
__host__ __device__ inline int first_worker(const AttendList &l, int head, const AttendTile &t)
{
    return (int)(((int64_t)head * l.units + t.unit0) / l.run);
}
__host__ __device__ inline int last_worker(const AttendList &l, int head, const AttendTile &t)
{
    return (int)(((int64_t)head * l.units + t.unit0 + t.units - 1) / l.run);
}

// What the host allocates for a batch of which it knows the sizes only: tiles of each list, and
// those whose parts are always kept.
inline void attend_capacity(int64_t n_tokens, int64_t n_seqs, int64_t n_prefixes, int64_t max_queries,
                            int64_t group, bool wide, int64_t cap[2], int64_t kept[2])
{
    const int64_t seqs = n_seqs < n_tokens ? n_seqs : n_tokens;      // requests with new tokens
    const int64_t rows = n_tokens * group, most = max_queries * group;
    const int64_t limit = share_rows((int)group), per = most < limit ? most : limit;
    for (int l = 0; l < 2; ++l) {
        cap[l] = kept[l] = 0;
        const int64_t R = list_rows(l);
        if (l ? !wide || most <= kShareRows : false)
            continue;
        // every request may end in a tile that is not full
        const bool all = l || !wide;                                  // else those of few rows only
        cap[l] = all ? seqs + rows / R : seqs * (((most < kShareRows ? most : kShareRows) + R - 1) / R);
        if (n_prefixes && (l ? group > kShareRows : true))
            kept[l] = seqs * ((per + R - 1) / R);
    }
    if (!n_prefixes)
        return;
    const int64_t tokens = n_seqs * (per / group), listed = (n_tokens < tokens ? n_tokens : tokens) * group;
    const int64_t narrow = n_prefixes * (wide ? kShareRows / kNarrowRows : 1) + (wide ? 0 : listed / kNarrowRows);
    cap[0] += narrow;
    kept[0] += narrow;
    if (wide) {
        cap[1] += n_prefixes + listed / kWideRows;
        kept[1] += n_prefixes + listed / kWideRows;
    }
}

// What follows from the sizes that the host knows: what the lists can hold, and how the batch is
// planned.  False: more tiles than are numbered.
inline bool size_batch(AttendBatch &b)
{
    if (!b.q_start)                      // one new token a request, whatever the caller says of the most
        b.max_queries = 1;
    int64_t cap[2], kept[2];
    attend_capacity(b.n_tokens, b.n_seqs, b.n_prefixes, b.max_queries, b.group, b.wide != 0, cap, kept);
    for (int l = 0; l < 2; ++l) {
        if (cap[l] * b.kv_heads * 8 > INT32_MAX / 2 || kept[l] > INT32_MAX / 2)
            return false;
        b.cap[l] = (int32_t)cap[l];
        b.kept_cap[l] = (int32_t)kept[l];
    }
    // most tiles times most units of one
    const double most = ((double)b.max_pages + b.prefix_max_pages) * (1 << b.page_shift) / kWideUnit + 2;
    b.units_fit = (double)(cap[0] + cap[1]) * most < (double)(1 << 29);
    b.simple = simple_batch(b) && b.units_fit;               // their sum takes 32 bits
    return true;
}

struct AttendArgs {
    AttendBatch b;
    CacheView c;
    const void *q;               // [T][heads * head_dim]
    void *y;
    float *parts[2];             // [slots][R][dp] weighted values, then
    float *sums[2];              // [slots][R][2] maximum and sum
    float scale;                 // of q . k, times log2(e)
};
hipError_t launch_attend_plan(const AttendBatch &b, hipStream_t st);
hipError_t launch_attend(bool bf16, const AttendArgs &a, hipStream_t st);

}  // namespace lora
