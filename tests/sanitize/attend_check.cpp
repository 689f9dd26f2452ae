// attend_check.cpp -- the host side of lora_attend.cpp and the index arithmetic that its kernels
// share with it (csrc/lora_attend.h) under AddressSanitizer and UndefinedBehaviorSanitizer,
// without a GPU: the plan of many batches formed serially with the kernels' own functions, in
// order and out of order, its tiles, workers and parts checked against what the host allocates;
// the order of the cache; and every refusal that needs no device.  The kernels' launch functions
// are stubs that must not be reached.  Built and run by tests/test_attend_sanitizers.py.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <limits>
#include <random>
#include <set>
#include <utility>
#include <vector>

#include "lora_mi355x.h"
#include "../../lora_adapter_application_amd/csrc/lora_attend.h"

static int failures = 0;
static const char *current = "";

namespace lora {
static hipError_t reached()
{
    std::printf("FAIL a launch was reached\n");
    ++failures;
    return hipErrorNotSupported;
}
hipError_t launch_plan(const int32_t *, int32_t, int32_t, const PlanBuffers &, hipStream_t,
                       const LaunchTiming *) { return reached(); }
hipError_t launch_shrink(bool, const ShrinkArgs &, const SlotMeta &, hipStream_t, const LaunchTiming &)
{ return reached(); }
hipError_t launch_expand(bool, const ExpandArgs &, const SlotMeta &, hipStream_t, const LaunchTiming &)
{ return reached(); }
hipError_t launch_fused(const FusedArgs &, const SlotMeta &, hipStream_t, const LaunchTiming &)
{ return reached(); }
hipError_t launch_slot_finalize(bool, const FinalizeBatch &, hipStream_t) { return reached(); }
hipError_t launch_saved(bool, const SavedArgs &, hipStream_t, const LaunchTiming &) { return reached(); }
hipError_t scratch_address(int, void **) { return reached(); }
hipError_t xcd_dispatch_check(int, hipStream_t, bool *) { return reached(); }
hipError_t launch_norm_rotary(bool, bool, const NormArgs &, hipStream_t) { return reached(); }
hipError_t launch_cache_store(bool, const CacheArgs &, hipStream_t) { return reached(); }
hipError_t launch_cache_load(bool, const CacheArgs &, hipStream_t) { return reached(); }
hipError_t launch_attend_plan(const AttendBatch &, hipStream_t) { return reached(); }
hipError_t launch_attend(bool, const AttendArgs &, hipStream_t) { return reached(); }
}  // namespace lora

using namespace lora;

#define CHECK(cond)                                                        \
    do {                                                                   \
        if (!(cond)) {                                                     \
            std::printf("FAIL %s: %s (line %d)\n", current, #cond, __LINE__); \
            if (++failures > 20)                                           \
                std::exit(1);                                              \
        }                                                                  \
    } while (0)

struct Batch {
    AttendBatch b{};
    std::vector<int32_t> q_start, lengths, pages, seqs, pre_lengths, pre_pages;
    void link(bool with_start)
    {
        b.q_start = with_start ? q_start.data() : nullptr;
        b.lengths = lengths.data();
        b.prefix_seqs = seqs.data();
        b.prefix_lengths = pre_lengths.data();
        int64_t cap[2], kept[2];
        attend_capacity(b.n_tokens, b.n_seqs, b.n_prefixes, b.max_queries, b.group, b.wide != 0, cap, kept);
        for (int l = 0; l < 2; ++l) {
            b.cap[l] = (int32_t)cap[l];
            b.kept_cap[l] = (int32_t)kept[l];
        }
    }
};

// The plan kernel's steps one after the other.  `ordered`: the batch is a proper one.
static void check_plan(const Batch &in, bool ordered)
{
    const AttendBatch &b = in.b;
    const int N = b.n_seqs + b.n_prefixes;
    std::vector<AttendEntity> ent(N);
    std::vector<int64_t> list_before(b.n_seqs + 1), tiles_before[2], kept_before[2];
    std::vector<int> listed;
    int64_t tiles[2] = {}, kept[2] = {}, list = 0;
    bool bad = false;
    for (int i = 0; i < N; ++i) {
        if (i < b.n_seqs) {
            list_before[i] = list;
            ent[i] = request_of(b, i, request_words(b, i), &bad);
            CHECK(ent[i].listed <= share_rows(b.group) / b.group);
            for (int j = 0; j < ent[i].listed; ++j) {
                CHECK(ent[i].token0 + j >= 0 && ent[i].token0 + j < b.n_tokens);
                listed.push_back(ent[i].token0 + j);
            }
            list += ent[i].listed;
            if (i + 1 == b.n_seqs)
                list_before[b.n_seqs] = list;
        } else {
            const int p = i - b.n_seqs;
            const int lo = clamp_to(b.prefix_seqs[p], 0, b.n_seqs), hi = clamp_to(b.prefix_seqs[p + 1], lo, b.n_seqs);
            bad |= b.prefix_seqs[p] < 0 || b.prefix_seqs[p + 1] < b.prefix_seqs[p] || b.prefix_seqs[p + 1] > b.n_seqs;
            ent[i] = prefix_of_batch(b, p, (int)list_before[lo], (int)(list_before[hi] - list_before[lo]), &bad);
        }
        for (int l = 0; l < 2; ++l) {
            tiles_before[l].push_back(tiles[l]);
            kept_before[l].push_back(kept[l]);
        }
        tiles[ent[i].list] += ent[i].tiles;
        kept[ent[i].list] += ent[i].keeps ? ent[i].tiles : 0;
    }
    unsigned long long claimed = 0, shared = 0, all_units = 0;
    for (int i = 0; i < N; ++i) {
        (i < b.n_seqs ? claimed : shared) += ent[i].rows / b.group;
        for (int j = 0; j < ent[i].tiles; ++j)
            all_units += tile_of(b, ent[i], j, 0).units;
    }
    const int32_t count[4] = {(int32_t)tiles[0], (int32_t)tiles[1], (int32_t)kept[0], (int32_t)kept[1]};
    const bool fits = attend_fits(b, claimed, shared, all_units, count);
    if (ordered) {
        CHECK(!bad);
        CHECK(fits);
    } else if (!fits) {
        // nothing but tokens claimed twice and units without end is refused
        CHECK(bad);
        CHECK(claimed > (unsigned long long)b.n_tokens || shared > (unsigned long long)b.n_tokens || all_units > 1ull << 29);
        return;
    }
    std::vector<int> rows_done((size_t)b.n_tokens * b.group, 0);
    AttendList lists[2];
    std::vector<AttendTile> all[2];
    for (int l = 0; l < 2; ++l) {
        int64_t units = 0;
        for (int i = 0; i < N; ++i) {
            if (ent[i].list != l)
                continue;
            int list0 = 0;
            if (i < b.n_seqs && ent[i].prefix >= 0)
                list0 = (int)list_before[i];
            for (int j = 0; j < ent[i].tiles; ++j) {
                AttendTile t = tile_of(b, ent[i], j, list0);
                CHECK((int64_t)all[l].size() == tiles_before[l][i] + j);
                t.kept = ent[i].keeps ? (int32_t)kept_before[l][i] + j : -1;
                CHECK(t.rows >= 1 && t.rows <= list_rows(l) && t.units >= 1);
                t.unit0 = (int32_t)units;
                units += t.units;
                all[l].push_back(t);
            }
        }
        CHECK(units <= 1 << 29);
        lists[l] = {(int32_t)all[l].size(), (int32_t)units, (int32_t)kept[l],
                    std::max(1, worker_run(units * b.kv_heads, b.workers[l]))};
    }
    for (int l = 0; l < 2; ++l) {
        const AttendList &L = lists[l];
        std::set<int64_t> used;
        const int64_t slots = part_slots(b.workers[l], b.kept_cap[l], b.kv_heads);
        int64_t total = 0;
        for (int h = 0; h < b.kv_heads; ++h)
            for (const AttendTile &t : all[l]) {
                const int w0 = first_worker(L, h, t), w1 = last_worker(L, h, t);
                CHECK(w0 >= 0 && w0 <= w1 && w1 < b.workers[l]);
                const int64_t at = (int64_t)h * L.units + t.unit0;
                for (int w = w0; w <= w1; ++w) {
                    const int64_t a = std::max(at, (int64_t)w * L.run), e = std::min(at + t.units, (int64_t)(w + 1) * L.run);
                    CHECK(a < e);
                    total += e - a;
                    if (t.kept < 0 && w0 == w1)
                        continue;                            // written whole
                    const int64_t s = part_slot(L, b.workers[l], h, t, w);
                    CHECK(s >= 0 && s < slots);
                    CHECK(used.insert(s).second);
                }
                for (int r = 0; r < t.rows; ++r) {
                    const int row = t.row0 + r, tok = t.token0 + row / b.group;
                    if (t.shared) {
                        CHECK(tok < (int)listed.size());
                        continue;
                    }
                    CHECK(tok >= 0 && tok < b.n_tokens);
                    if (!h)
                        ++rows_done[(size_t)tok * b.group + row % b.group];
                    if (t.prefix >= 0 && !h) {               // the row of the shared tile is the same token's
                        const AttendEntity &p = ent[b.n_seqs + t.prefix];
                        const int lo = clamp_to(b.prefix_seqs[t.prefix], 0, b.n_seqs);
                        const int pr = t.pre_row - (int)list_before[lo] * b.group + r, PR = list_rows(p.list);
                        CHECK(pr >= 0);
                        CHECK(pr / PR < p.tiles);
                        const AttendTile &s = all[p.list][tiles_before[p.list][b.n_seqs + t.prefix] + pr / PR];
                        CHECK(s.shared && s.seq == t.prefix && pr % PR < s.rows && s.row0 + pr % PR == pr);
                        CHECK(listed[s.token0 + pr / b.group] == tok && pr % b.group == row % b.group);
                    }
                }
                // tokens stay inside of what the tables can name
                CHECK(t.len >= 0 && (int64_t)t.len <= (int64_t)(t.shared ? b.prefix_max_pages : b.max_pages) << b.page_shift);
                CHECK(t.pre_len >= 0 && (int64_t)t.pre_len <= (int64_t)b.prefix_max_pages << b.page_shift);
                if (t.pre_len)
                    CHECK(t.pre_seq >= 0 && t.pre_seq < b.n_prefixes);
            }
        CHECK(total == (int64_t)L.units * b.kv_heads);
    }
    if (ordered)
        for (int i = 0; i < b.n_seqs; ++i) {
            const int q0 = b.q_start ? b.q_start[i] : i, q1 = b.q_start ? b.q_start[i + 1] : i + 1;
            for (int t = q0; t < q1; ++t)
                for (int r = 0; r < b.group; ++r)
                    CHECK(rows_done[(size_t)t * b.group + r] == 1);
        }
}

static void plans()
{
    std::mt19937 rng(7);
    auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
    const int groups[] = {1, 2, 3, 5, 7, 8, 16, 17, 32, 40, 64};
    for (int round = 0; round < 1500; ++round) {
        current = "plan";
        Batch x;
        AttendBatch &b = x.b;
        set_group(b, groups[pick(0, 10)]);
        b.kv_heads = pick(1, 9);
        b.page_shift = pick(5, 8);
        b.wide = pick(0, 1);
        for (int &w : b.workers)
            w = kAttendCus * pick(1, kAttendWorkers / kAttendCus);
        b.n_seqs = pick(1, round % 7 ? 40 : 700);
        b.n_prefixes = pick(0, 2) ? pick(0, 6) : 0;
        b.max_pages = pick(0, 12);
        b.prefix_max_pages = pick(0, 30);
        const int most = pick(0, 1) ? 1 : pick(1, 90);
        b.max_queries = most;
        const bool start = most > 1 || pick(0, 1);
        x.q_start.push_back(start ? pick(0, 3) : 0);
        for (int i = 0; i < b.n_seqs; ++i) {
            x.q_start.push_back(x.q_start.back() + (start ? pick(0, most) : 1));
            x.lengths.push_back(pick(0, b.max_pages << b.page_shift));
        }
        b.n_tokens = x.q_start.back() + pick(0, 3);
        x.seqs.push_back(pick(0, b.n_seqs));
        for (int p = 0; p < b.n_prefixes; ++p) {
            x.seqs.push_back(pick(x.seqs.back(), b.n_seqs));
            x.pre_lengths.push_back(pick(0, 3) ? pick(0, b.prefix_max_pages << b.page_shift) : 0);
        }
        if (!b.n_tokens)
            continue;
        x.link(start);
        check_plan(x, true);
        // anything at all in the arrays
        current = "plan of a batch out of order";
        Batch y = x;
        const int wild[] = {-2147483647 - 1, -1000, -1, 0, 1, 2, 5, 1000, b.n_tokens, b.n_seqs, 2147483647};
        for (auto *v : {&y.q_start, &y.lengths, &y.seqs, &y.pre_lengths})
            for (auto &e : *v)
                if (!pick(0, 3))
                    e = wild[pick(0, 10)];
        y.link(start);
        check_plan(y, false);
    }
}

static void division()
{
    current = "a worker's run";
    std::mt19937_64 big(5);
    for (int k = 0; k < 20000; ++k) {
        const int64_t total = (int64_t)(big() >> (25 + k % 39));
        const int workers = kAttendCus * (1 + k % 4);
        CHECK(worker_run(total, workers) == (total + workers - 1) / workers);
    }
    current = "division by the heads of a key-value head";
    AttendBatch b{};
    std::mt19937 rng(3);
    for (int g = 1; g <= 1024; ++g) {
        set_group(b, g);
        for (int k = 0; k < 2000; ++k) {
            const int32_t x = k < 1000 ? k : k < 1500 ? (int32_t)(rng() >> 1) : (int32_t)(rng() >> 1) / g * g - k % 2;
            if (x >= 0)
                CHECK(over_group(b, x) == x / g);
        }
        for (int64_t x : {2147483647ll, 2147483646ll, 2147483647ll / g * g, 2147483647ll / g * g - 1})
            CHECK(over_group(b, (int32_t)x) == x / g);
    }
}

static void layout()
{
    current = "cache layout";
    const int dims[] = {8, 24, 64, 80, 96, 104, 128, 136, 256};
    for (int kind = 0; kind < 3; ++kind)
        for (int d : dims) {
            CacheView c{};
            c.kv_heads = 3;
            c.head_dim = d;
            c.dp = padded_dim(d);
            CHECK(c.dp >= d);
            c.page_shift = 6;
            c.elem = kind ? 1 : 2;
            c.half = kBlock * c.dp * c.elem;
            c.block = 2 * c.half + (kind ? 256 : 0);
            CHECK(c.block % 16 == 0);
            std::set<int> k, v;
            for (int t = 0; t < kBlock; ++t)
                for (int i = 0; i < d; ++i) {
                    const int a = key_at(t, i), e = value_at(c.dp, t, i);
                    CHECK(a >= 0 && a < kBlock * c.dp && k.insert(a).second);
                    CHECK(e >= 0 && e < kBlock * c.dp && v.insert(e).second);
                }
            std::set<int64_t> blocks;
            for (int p = 0; p < 4; ++p)
                for (int h = 0; h < 3; ++h)
                    for (int i = 0; i < 2; ++i) {
                        const int64_t at = cache_block(c, p, h, i);
                        CHECK(at >= 0 && at + c.block <= cache_block(c, 4, 0, 0) && blocks.insert(at / c.block).second);
                    }
        }
    CacheView c{};
    c.kv_heads = 64;
    c.page_shift = 5;
    c.block = 1 << 15;
    CHECK(cache_block(c, (1 << 26) - 1, 63, 0) == (((1ll << 26) - 1) * 64 + 63) * (1ll << 15));
}

static void expect(int got, int want, const char *what)
{
    if (got != want) {
        std::printf("FAIL %s: status %d, expected %d\n", what, got, want);
        ++failures;
    }
}

int main()
{
    plans();
    division();
    layout();
    const int bad = LORA_ERR_INVALID_ARGUMENT;
    lora_rotary rot;
    std::memset(&rot, 0, sizeof rot);
    lora_attend_batch batch;
    std::memset(&batch, 0, sizeof batch);
    lora_cache *cache = (lora_cache *)&batch;
    const int32_t mod = 0;
    expect(lora_norm_rotary_group(nullptr, &rot, 1, &mod, nullptr, nullptr, 1e-6, nullptr, nullptr, 0, nullptr), bad, "norm");
    expect(lora_cache_create(nullptr, &cache, 0, 1, 64, 64, 1), bad, "create");
    if (cache) {
        std::printf("FAIL a refused create left a handle\n");
        ++failures;
    }
    expect(lora_cache_create(nullptr, nullptr, 0, 1, 64, 64, 1), bad, "create without out");
    expect(lora_cache_destroy(nullptr, nullptr), bad, "destroy");
    expect(lora_cache_store(nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr), bad, "store");
    expect(lora_cache_load(nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr), bad, "load");
    expect(lora_attend_prepare(nullptr, nullptr, 1, &batch, nullptr), bad, "prepare");
    expect(lora_attend(nullptr, nullptr, nullptr, nullptr, 1.0, nullptr), bad, "attend");
    std::printf("failures: %d\n", failures);
    return failures != 0;
}
