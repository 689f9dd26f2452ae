// attend_sizes_check.cpp -- what the host decides for a batch of attention from its sizes alone
// (size_batch of csrc/lora_attend.h): whether its launches plan it for themselves, and room for
// every tile that the arrays can name.  Built and run by tests/test_attend_sizes.py.
#include <cstdio>
#include <initializer_list>

#include "../../lora_adapter_application_amd/csrc/lora_attend.h"

using namespace lora;

static int failures = 0;

#define CHECK(cond, ...)                                                      \
    do {                                                                      \
        if (!(cond)) {                                                        \
            std::printf("FAIL %s (line %d):", #cond, __LINE__);               \
            std::printf(__VA_ARGS__);                                         \
            std::printf("\n");                                                \
            ++failures;                                                       \
        }                                                                     \
    } while (0)

static AttendBatch sized(int seqs, int tokens, int queries, int group, bool wide, bool starts, int prefixes,
                         int max_pages = 4, int page_shift = 6)
{
    static const int32_t some[2] = {0, 0};
    AttendBatch b{};
    b.q_start = starts ? some : nullptr;
    b.n_seqs = seqs;
    b.n_tokens = tokens;
    b.n_prefixes = prefixes;
    b.max_queries = queries < tokens ? queries : tokens;
    b.kv_heads = 2;
    b.page_shift = page_shift;
    b.max_pages = max_pages;
    b.prefix_max_pages = prefixes ? 4 : 0;
    b.wide = wide;
    set_group(b, group);
    CHECK(size_batch(b), " %d requests", seqs);
    return b;
}

// Without starts a request has one new token, whatever the caller says of the most.
static void one_token_each()
{
    for (int wide = 0; wide < 2; ++wide)
        for (int prefixes : {0, 3})
            for (int seqs : {1, 64, 256, 300})
                for (int group : {1, 4, 16, 17, 40})
                    for (int queries : {1, 2, 64, 512}) {
                        const AttendBatch b = sized(seqs, seqs + 300, queries, group, wide, false, prefixes);
                        const AttendBatch one = sized(seqs, seqs + 300, 1, group, wide, false, prefixes);
                        CHECK(b.max_queries == 1, " %d", b.max_queries);
                        for (int l = 0; l < 2; ++l) {
                            CHECK(b.cap[l] == one.cap[l], " list %d: %d, %d", l, b.cap[l], one.cap[l]);
                            CHECK(b.kept_cap[l] == one.kept_cap[l], " list %d: %d, %d", l, b.kept_cap[l], one.kept_cap[l]);
                        }
                        if (b.simple)
                            CHECK(!b.cap[1], " %d requests, group %d, at most %d: %d wide tiles without a plan", seqs, group,
                                  queries, b.cap[1]);
                    }
}

// A launch that plans a batch for itself sums its units in 32 bits: only where no lengths that the
// table can name have more.
static void units_of_simple_batches()
{
    for (int seqs : {1, 31, 32, 200, 256})
        for (int page_shift : {5, 10, 20, 30})
            for (int pages : {1, 8, 2048, 1 << 21, 1 << 26}) {
                const AttendBatch b = sized(seqs, seqs, 1, 1, true, false, 0, pages, page_shift);
                const int64_t most = (int64_t)pages << page_shift;
                bool bad = false;
                const int held = held_of(INT32_MAX, pages, page_shift, &bad);
                CHECK(held == (most < INT32_MAX ? most : INT32_MAX), " %d", held);
                if (b.simple)
                    CHECK(seqs * (int64_t)simple_tile(0, held, 1, 0).units <= 1 << 29, " %d requests of %d tokens", seqs, held);
                if (most < (1ll << 33) / seqs)
                    CHECK(b.simple, " %d requests of %lld tokens", seqs, (long long)most);
            }
}

int main()
{
    one_token_each();
    units_of_simple_batches();
    std::printf("failures: %d\n", failures);
    return failures != 0;
}
