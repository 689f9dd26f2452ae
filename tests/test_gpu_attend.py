"""Attention over the paged cache (lora_attend) on the GPU against the formula in 64 bits."""
import math

import pytest
import torch

from attend_util import Requests, check_rows
from gpu_util import log
from layer_util import TORCH
from lora_adapter_application_amd import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load_library()


def attended(r, scale=None, flags=0):
    scale = r.dim ** -0.5 if scale is None else scale
    S, cache = r.make()
    S.flags()
    y = torch.full_like(r.q, 7.0).cuda()
    before = y.clone()
    batch, q = r.batch(), r.q.cuda()
    S.attend_prepare(cache, r.heads, batch)
    S.attend(cache, q, y, scale)
    torch.cuda.synchronize()
    assert S.flags() == flags
    cache.close()
    S.close()
    return y, before, scale


# dtype, kind, heads, kv_heads, head_dim, page, queries, lengths, prefixes
CASES = [
    # one request, lengths around the pieces that the work is cut in
    *[("bf16", "native", 4, 2, 128, 64, [1], [n], []) for n in (1, 2, 31, 32, 33, 127, 128, 129, 400)],
    ("bf16", "native", 8, 8, 128, 32, [1], [3000], []),
    # head layouts: none, few, uneven and all heads on one key-value head
    ("bf16", "native", 32, 32, 64, 64, [1] * 3, [100, 1, 257], []),
    ("bf16", "native", 15, 5, 96, 128, [1] * 3, [100, 1, 257], []),
    ("bf16", "native", 14, 2, 80, 32, [1] * 3, [100, 1, 257], []),
    ("bf16", "native", 16, 1, 256, 64, [1] * 3, [100, 1, 257], []),
    ("bf16", "native", 64, 1, 128, 64, [1] * 5, [100, 1, 257, 60, 5], [(0, 4, 130)]),
    ("bf16", "native", 40, 2, 136, 256, [1] * 2, [300, 7], []),
    ("bf16", "native", 3, 3, 8, 32, [1] * 2, [300, 7], []),
    # 8 bits
    ("bf16", "fp8", 8, 2, 128, 64, [1] * 4, [1, 64, 200, 333], [(0, 3, 77)]),
    ("bf16", "int8", 8, 2, 128, 64, [1] * 4, [1, 64, 200, 333], [(0, 3, 77)]),
    ("bf16", "fp8", 6, 2, 80, 32, [3, 1, 17], [30, 64, 99], [(1, 3, 40)]),
    ("bf16", "int8", 6, 2, 96, 32, [3, 1, 17], [30, 64, 99], [(1, 3, 40)]),
    ("bf16", "fp8", 4, 4, 256, 128, [1, 2], [30, 129], []),
    ("bf16", "int8", 4, 4, 64, 128, [1, 2], [30, 129], []),
    ("fp32", "fp8", 4, 2, 64, 32, [1, 2], [30, 129], [(0, 2, 33)]),
    ("fp32", "int8", 4, 2, 128, 32, [1, 2], [30, 129], [(0, 2, 33)]),
    # fp32
    ("fp32", "native", 12, 4, 80, 32, [1, 40, 5, 0, 9], [333, 40, 5, 10, 70], [(0, 2, 97), (2, 5, 31)]),
    ("fp32", "native", 6, 2, 256, 64, [1, 3], [200, 3], []),
    ("fp32", "native", 64, 1, 64, 64, [1, 3], [200, 3], [(0, 2, 50)]),
    # several new tokens: their rows see different tokens, some none
    ("bf16", "native", 4, 2, 128, 64, [5], [5], []),
    ("bf16", "native", 4, 1, 128, 64, [70, 33, 1, 130], [70, 200, 40, 131], []),
    ("bf16", "native", 8, 1, 64, 32, [300], [300], []),
    ("bf16", "native", 2, 2, 96, 32, [300, 17], [450, 17], [(0, 2, 64)]),
    ("bf16", "native", 8, 2, 128, 64, [4, 9, 2], [2, 0, 1], []),           # more new tokens than held
    ("bf16", "native", 8, 2, 128, 64, [4, 40, 2], [2, 0, 1], [(0, 2, 9)]),
    ("bf16", "int8", 8, 2, 128, 64, [4, 40, 2], [2, 0, 1], [(0, 2, 9)]),
    # requests of nothing, prefixes of nothing and of no request
    ("bf16", "native", 4, 2, 64, 32, [1, 1, 0, 1], [0, 40, 12, 0], [(0, 1, 0), (1, 1, 50), (1, 3, 20)]),
    ("bf16", "native", 4, 2, 64, 32, [0, 0], [5, 6], [(0, 2, 20)]),
    # shared prefixes: few rows, one tile, many tiles
    ("bf16", "native", 8, 8, 128, 64, [1] * 9, [33] * 9, [(2, 9, 300)]),
    ("bf16", "native", 16, 2, 128, 64, [1] * 40, list(range(1, 41)), [(0, 17, 1000), (17, 18, 65), (18, 39, 64)]),
    ("bf16", "fp8", 16, 2, 128, 64, [1] * 40, list(range(1, 41)), [(0, 17, 1000), (17, 18, 65), (18, 39, 64)]),
    ("bf16", "int8", 16, 2, 64, 64, [1, 2, 3] * 20, [50] * 60, [(0, 50, 513)]),
    ("bf16", "native", 10, 2, 80, 32, [2, 90, 1, 6, 7] * 4, [101] * 20, [(0, 3, 150), (3, 20, 33)]),
    # tiles of many rows in 8 bits and of every width, parts of long ones
    ("bf16", "fp8", 8, 1, 256, 64, [100, 3], [200, 30], [(0, 2, 100)]),
    ("bf16", "int8", 8, 1, 96, 32, [100, 3], [200, 30], [(0, 2, 100)]),
    ("bf16", "fp8", 16, 2, 64, 128, [100, 3, 33], [100, 30, 40], [(0, 2, 100)]),
    ("bf16", "native", 8, 1, 256, 32, [100, 3], [200, 30], [(0, 2, 100)]),
    ("bf16", "native", 8, 1, 128, 64, [700], [1500], [(0, 1, 900)]),
    ("bf16", "int8", 8, 1, 128, 32, [200], [1500], [(0, 1, 900)]),
    # many tiles of few rows: several key-value heads are joined together
    ("bf16", "native", 5, 5, 64, 32, [1] * 300, [i % 70 for i in range(300)], [(3, 290, 140)]),
    ("bf16", "fp8", 6, 3, 128, 32, [1] * 400, [i % 50 for i in range(400)], [(0, 400, 300)]),
    # more requests than a workgroup has threads, than the plan keeps in LDS
    ("bf16", "native", 2, 1, 64, 32, [1] * 1300, [1 + i % 9 for i in range(1300)], [(0, 700, 40), (700, 1290, 33)]),
    ("bf16", "int8", 2, 1, 64, 32, [1, 0, 2] * 900, [2 + i % 9 for i in range(2700)], [(0, 1200, 40), (1200, 2600, 33)]),
    # more work than workers
    ("bf16", "native", 32, 32, 64, 32, [1] * 70, [5 * i + 1 for i in range(70)], [(10, 60, 200)]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c[:6]) + f"-{len(c[6])}x{max(c[6])}-{max(c[7])}")
def test_against_64_bits(case):
    log(f"case attend {case}")
    r = Requests(len(str(case)), *case)
    y, before, scale = attended(r)
    log(f"  worst error / bound {check_rows(r, y, scale, before, str(case[:6])):.3f}")


def test_rows_of_no_request_stay():
    r = Requests(3, "bf16", "native", 4, 2, 64, 32, [2, 0, 1], [40, 3, 9], lead=3, tail=5)
    y, before, scale = attended(r)
    check_rows(r, y, scale, before, "lead and tail")


@pytest.mark.parametrize("dtype,heads,kv_heads,lengths", [
    ("bf16", 4, 2, [40, 3, 9, 0, 100, 7, 7]),
    ("bf16", 16, 1, [5000]),
    ("fp32", 3, 3, [0]),
    ("bf16", 8, 8, [11 * i % 400 for i in range(255)]),
    ("fp32", 5, 5, [7 * i % 90 for i in range(256)]),
    ("bf16", 2, 1, [7 * i % 90 for i in range(257)]),        # more than a launch plans by itself
    ("bf16", 17, 1, [40, 300]),                              # rows of more than one tile
])
def test_one_token_a_request_without_starts(dtype, heads, kv_heads, lengths):
    r = Requests(4, dtype, "native", heads, kv_heads, 64, 32, [1] * len(lengths), lengths, q_start=False, tail=2)
    y, before, scale = attended(r)
    check_rows(r, y, scale, before, "no q_start")


def test_lengths_out_of_range_without_starts():
    r = Requests(18, "bf16", "native", 4, 2, 64, 32, [1] * 6, [40, 3, 64, 9, 100, 7], q_start=False)
    S, cache = r.make()
    q, b = r.q.cuda(), r.batch()
    y, good = torch.full_like(q, 7.0), torch.full_like(q, 7.0)
    S.attend_prepare(cache, r.heads, b)
    S.attend(cache, q, good)
    assert S.flags() == 0
    for value in (2 ** 31 - 1, -2 ** 31):
        b.lengths[1] = value
        S.attend(cache, q, y)
        assert S.flags() == binding.LORA_FLAG_ATTEND_BATCH
        assert torch.equal(y[[0, 2, 3, 4, 5]], good[[0, 2, 3, 4, 5]])


@pytest.mark.parametrize("kind", ["native", "fp8", "int8"])
@pytest.mark.parametrize("offset", [1, 4])
def test_addresses_off_16_bytes(kind, offset):
    r = Requests(5, "bf16", kind, 4, 2, 80, 32, [1, 40, 3], [64, 40, 9], [(0, 2, 40)])
    S, cache = r.make()
    whole_q = torch.zeros(r.q.numel() + 8, dtype=r.q.dtype, device="cuda")
    whole_y = torch.full_like(whole_q, 7.0)
    q = whole_q[offset:offset + r.q.numel()].view_as(r.q)
    y = whole_y[offset:offset + r.q.numel()].view_as(r.q)
    q.copy_(r.q)
    S.attend_prepare(cache, r.heads, r.batch())
    S.attend(cache, q, y)
    check_rows(r, y, 80 ** -0.5, y, "off 16 bytes")
    rest = torch.cat((whole_y[:offset], whole_y[offset + r.q.numel():]))
    assert bool((rest == 7).all())


def test_large_scores_and_scale():
    """Scores of hundreds: one token takes all; the maximum moves far from block to block."""
    for spread, dtype in ((8.0, "bf16"), (3.0, "fp32")):
        r = Requests(6, dtype, "native", 4, 2, 64, 32, [1, 30], [700, 90], [(0, 2, 100)], spread=spread)
        scale = 0.5
        y, before, _ = attended(r, scale)
        check_rows(r, y, scale, before, f"spread {spread}")


def test_infinities_and_nans_stay_with_the_rows_that_see_them():
    """A key or value that is not finite changes the rows that see its token and no other; what
    those get is what the formula gives."""
    for dtype in ("bf16", "fp32"):
        for queries, length, pre in (([40], 70, 0), ([3], 40, 50), ([100], 100, 33), ([1], 40, 0)):
            n = queries[0]
            r = Requests(8, dtype, "native", 4, 2, 64, 32, queries, [length], [(0, 1, pre)] if pre else [])
            clean, _, scale = attended(r)
            at = r.slots_of(r.table[0], length)
            hit = max(length - n, length - 2) if n > 1 else length - 1       # token of the last new ones
            for what, change in (("value inf", lambda: r.v[at[hit], 0].__setitem__(5, math.inf)),
                                 ("value -inf", lambda: r.v[at[hit], 0].__setitem__(5, -math.inf)),
                                 ("value nan", lambda: r.v[at[hit], 0].__setitem__(5, math.nan)),
                                 ("key nan", lambda: r.k[at[hit], 0].__setitem__(5, math.nan))):
                saved = r.k.clone(), r.v.clone()
                change()
                y, _, _ = attended(r)
                r.k, r.v = saved
                got, ok = y.cpu().view(n, 2, 2, 64), clean.cpu().view(n, 2, 2, 64)
                first = hit - (length - n)                   # new token that sees it first
                assert torch.equal(got[:first], ok[:first]), (what, n)
                assert torch.equal(got[:, 1], ok[:, 1]), (what, n)
                seen = got[first:, 0]
                if what == "key nan":
                    assert torch.isnan(seen).all()
                    continue
                rest = [d for d in range(64) if d != 5]
                assert torch.equal(seen[..., rest], ok[first:, 0][..., rest]), (what, n)
                hot = seen[..., 5].float()
                assert {"value inf": (hot == math.inf), "value -inf": (hot == -math.inf),
                        "value nan": torch.isnan(hot)}[what].all(), (what, n)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("queries,length,pre", [([1], 300, 0), ([2], 200, 70), ([40], 300, 0), ([90], 200, 70)])
def test_infinite_values_that_every_row_sees(dtype, queries, length, pre):
    """In blocks without hidden tokens: an infinity makes its dim that of every row, both signs and a
    NaN make it NaN, no other dim changes."""
    r = Requests(19, dtype, "native", 4, 2, 64, 32, queries, [length], [(0, 1, pre)] if pre else [])
    clean, _, _ = attended(r)
    at = r.slots_of(r.prefix_table[0], pre) if pre else r.slots_of(r.table[0], 64)
    r.v[at[3], 0, 5], r.v[at[9], 0, 6] = math.inf, -math.inf
    r.v[at[3], 0, 7], r.v[at[40], 0, 7] = math.inf, -math.inf
    r.v[at[50], 0, 8] = math.nan
    y, _, _ = attended(r)
    got, ok = y.cpu().view(-1, 2, 2, 64).float(), clean.cpu().view(-1, 2, 2, 64).float()
    assert torch.equal(got[:, 1], ok[:, 1])
    rest = [d for d in range(64) if d not in (5, 6, 7, 8)]
    assert torch.equal(got[:, 0][..., rest], ok[:, 0][..., rest])
    assert (got[:, 0, :, 5] == math.inf).all() and (got[:, 0, :, 6] == -math.inf).all()
    assert torch.isnan(got[:, 0, :, 7:9]).all()


@pytest.mark.parametrize("kind", ["fp8", "int8"])
def test_a_coded_head_with_a_nan(kind):
    r = Requests(9, "bf16", kind, 4, 2, 64, 32, [40], [70])
    clean, _, _ = attended(r)
    at = r.slots_of(r.table[0], 70)
    r.v[at[50], 1, 3] = math.inf
    y, _, _ = attended(r)
    got, ok = y.cpu().view(40, 2, 2, 64), clean.cpu().view(40, 2, 2, 64)
    assert torch.equal(got[:20], ok[:20]) and torch.equal(got[:, 0], ok[:, 0])
    assert torch.isnan(got[20:, 1]).all()


def test_scores_without_a_largest_are_nan():
    """Every score of a row -inf: 0 / 0, as the formula says; not the zeros of a row that sees nothing."""
    r = Requests(10, "fp32", "native", 2, 2, 64, 32, [1, 1], [3, 3])
    r.q[0] = r.q[0].abs() + 1
    r.k[r.slots_of(r.table[0], 3)] = -math.inf
    y, _, _ = attended(r)
    assert torch.isnan(y[0]).all() and torch.isfinite(y[1]).all()


def test_equal_calls_give_equal_bits_and_graphs_replay():
    r = Requests(11, "bf16", "fp8", 16, 2, 128, 64, [1] * 40 + [70], list(range(1, 41)) + [90],
                 [(0, 17, 1000), (17, 30, 65)])
    S, cache = r.make()
    batch, q = r.batch(), r.q.cuda()
    y = torch.empty_like(q)
    S.attend_prepare(cache, r.heads, batch)
    S.attend(cache, q, y)
    torch.cuda.synchronize()
    eager = y.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        S.attend_prepare(cache, r.heads, batch)
        S.attend(cache, q, y)
    small = Requests(12, "bf16", "fp8", 16, 2, 128, 64, [1, 2], [3, 9], [(0, 1, 5)])
    sq, sy = small.q.cuda(), torch.empty_like(small.q).cuda()
    for k in range(3):
        y.fill_(1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager)
        # a smaller batch in between uses the same workspace
        S.attend_prepare(cache, 16, small.batch())
        S.attend(cache, sq, sy)
        torch.cuda.synchronize()
    # the graph reads the arrays as they are at the replay
    batch.lengths.copy_(torch.tensor([(i + 2) // 2 for i in range(40)] + [80], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    S.attend_prepare(cache, r.heads, batch)
    z = torch.empty_like(q)
    S.attend(cache, q, z)
    torch.cuda.synchronize()
    assert torch.equal(y, z) and not torch.equal(y, eager)
    assert S.flags() == 0


def test_another_stream():
    r = Requests(13, "bf16", "int8", 8, 2, 128, 64, [1] * 5, [100, 1, 257, 60, 5], [(0, 4, 130)])
    S, cache = r.make()
    q, batch = r.q.cuda(), r.batch()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = torch.full_like(q, 7.0)
    torch.cuda.synchronize()
    S.attend_prepare(cache, r.heads, batch, stream=s)
    S.attend(cache, q, y, stream=s)
    s.synchronize()
    check_rows(r, y, 128 ** -0.5, y, "another stream")


def test_arrays_out_of_range_are_clamped_and_flagged():
    """What the plan's tests on the CPU show to stay inside its bounds, on the device: lengths past
    the table, starts past the batch, bounds past the requests, pages past the cache."""
    r = Requests(14, "bf16", "native", 4, 2, 64, 32, [1] * 6, [40, 3, 64, 9, 100, 7], [(0, 3, 33)])
    S, cache = r.make()
    q = r.q.cuda()
    big, low = 2 ** 31 - 1, -2 ** 31
    for change, flag, same in (
            (lambda b: b.lengths.__setitem__(1, big), binding.LORA_FLAG_ATTEND_BATCH, [0, 2, 3, 4, 5]),
            (lambda b: b.lengths.__setitem__(1, low), binding.LORA_FLAG_ATTEND_BATCH, [0, 2, 3, 4, 5]),
            (lambda b: b.q_start.__setitem__(6, big), binding.LORA_FLAG_ATTEND_BATCH, [0, 1, 2, 3, 4, 5]),
            (lambda b: b.q_start.__setitem__(6, low), binding.LORA_FLAG_ATTEND_BATCH, [0, 1, 2, 3, 4]),
            (lambda b: b.q_start.__setitem__(3, 4), binding.LORA_FLAG_ATTEND_BATCH, [0, 1, 2, 4, 5]),   # two of at most one
            (lambda b: b.q_start.__setitem__(1, 6), binding.LORA_FLAG_ATTEND_BATCH, [0, 2, 3, 4, 5]),
            (lambda b: b.prefix_seqs.__setitem__(1, 1000), binding.LORA_FLAG_ATTEND_BATCH, [0, 1, 2]),
            (lambda b: b.prefix_lengths.__setitem__(0, big), binding.LORA_FLAG_ATTEND_BATCH, [3, 4, 5]),
            (lambda b: b.pages.__setitem__((4, 1), r.pages), binding.LORA_FLAG_CACHE_PAGE, [0, 1, 2, 3, 5]),
            (lambda b: b.pages.__setitem__((4, 1), low), binding.LORA_FLAG_CACHE_PAGE, [0, 1, 2, 3, 5])):
        b = r.batch()
        y = torch.full_like(q, 7.0)
        S.attend_prepare(cache, r.heads, b)
        S.attend(cache, q, y)
        good = y.clone()
        assert S.flags() == 0
        change(b)
        S.attend_prepare(cache, r.heads, b)
        S.attend(cache, q, y)
        assert S.flags() == flag
        assert torch.equal(y[same], good[same])


def test_refusals():
    r = Requests(15, "bf16", "native", 4, 2, 64, 32, [1] * 3, [40, 3, 64])
    S, cache = r.make()
    q, y, b = r.q.cuda(), torch.empty_like(r.q).cuda(), r.batch()
    E, N = binding.LORA_ERR_INVALID_ARGUMENT, binding.LORA_ERR_NO_PLAN

    def refused(status, fn, *args, **kw):
        with pytest.raises(binding.LoraError) as e:
            fn(*args, **kw)
        assert e.value.status == status, e.value

    refused(N, S.attend, cache, q, y)
    refused(E, S.attend_prepare, cache, 5, b)
    refused(E, S.attend_prepare, cache, 0, b)
    refused(binding.LORA_ERR_TOO_MANY_TOKENS, S.attend_prepare, cache, 4, b, S.max_tokens + 1)
    refused(E, S.attend_prepare, cache, 4, b, -1)
    S.attend_prepare(cache, 4, b)
    S.attend(cache, q, y)
    refused(E, S.attend, cache, q, y, 0.0)
    refused(E, S.attend, cache, q, y, -1.0)
    refused(E, S.attend, cache, q, y, math.nan)
    refused(E, S.attend, cache, q, q)
    other = S.cache(2, 96, 2, 32)
    with pytest.raises((binding.LoraError, ValueError)):
        S.attend(other, q, y)
    pages = S.cache(2, 64, 2, 64)
    refused(E, S.attend, pages, q, y)
    gone = cache.handle
    T = binding.Slots(1, 1, [(64, 64)], "bf16", 64)
    refused(E, binding.lora_attend, T.ctx, gone, q, y, 1.0)      # another pool's cache
    with pytest.raises(ValueError):
        binding.AttendBatch(b.lengths, b.pages[:2])
    with pytest.raises(ValueError):
        binding.AttendBatch(b.lengths.long(), b.pages)
    with pytest.raises(ValueError):
        binding.AttendBatch(b.lengths, b.pages.t())
    # a capture that lacks its prepare, and one whose workspace would have to grow
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        q.add_(0)
        refused(N, S.attend, cache, q, y)
    S.attend_prepare(cache, 4, b)
    S.attend(cache, q, y)
    with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=s):
        S.attend_prepare(cache, 4, b)
        S.attend(cache, q, y)
    refused(N, S.attend, cache, q, y)                            # the prepare has not run
    S.attend_prepare(cache, 4, b)
    S.attend(cache, q, y)
    torch.cuda.synchronize()
    T.close()


def test_a_capture_cannot_grow_the_workspace():
    r = Requests(16, "bf16", "native", 4, 2, 64, 32, [1] * 3, [40, 3, 64])
    S, cache = r.make()
    q, y, b = r.q.cuda(), torch.empty_like(r.q).cuda(), r.batch()
    s = torch.cuda.Stream()
    with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=s):
        q.add_(0)
        with pytest.raises(binding.LoraError) as e:
            S.attend_prepare(cache, 4, b)
        assert e.value.status == binding.LORA_ERR_INVALID_ARGUMENT and "before the capture" in str(e.value)


def test_empty_batches():
    r = Requests(17, "bf16", "native", 4, 2, 64, 32, [1] * 3, [40, 3, 64])
    S, cache = r.make()
    q, y = r.q.cuda(), torch.full_like(r.q, 7.0).cuda()
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    S.attend_prepare(cache, 4, binding.AttendBatch(none, none.view(0, 1)), n_tokens=3)
    S.attend(cache, q, y)
    torch.cuda.synchronize()
    assert bool((y == 7).all())


def test_more_workgroups_than_a_row_of_a_grid_holds():
    """2^19 requests of one token and a long last one, on 33 key-value heads: the last tiles' parts
    are joined by workgroups past 2^24.  Two pages hold the tokens of all requests."""
    n, kv_heads, group, dim, page, pages = (1 << 19) + 1, 33, 9, 8, 32768, 32
    heads = kv_heads * group
    S = binding.Slots(1, 1, [(64, 64)], "bf16", n)
    cache = S.cache(kv_heads, dim, 2, page)
    gen = torch.Generator().manual_seed(5)
    k = torch.zeros(4096, kv_heads * dim, dtype=torch.bfloat16).cuda()
    total = torch.zeros(kv_heads * dim, dtype=torch.float64)
    first = None
    for at in range(0, 2 * page, 4096):                      # a page around 1, the other around 5
        v = (torch.randn(4096, kv_heads * dim, generator=gen) + (1 if at < page else 5)).bfloat16()
        total += v.double().sum(0)
        first = v[0] if first is None else first
        S.cache_store(cache, k, v.cuda(), torch.arange(at, at + 4096, dtype=torch.int32).cuda())
    lengths = torch.ones(n, dtype=torch.int32)
    lengths[-1] = page * pages
    table = torch.zeros(n, pages, dtype=torch.int32, device="cuda")
    table[:, pages // 2:] = 1
    q = torch.zeros(n, heads * dim, dtype=torch.bfloat16, device="cuda")
    y = torch.full_like(q, 7.0)
    S.attend_prepare(cache, heads, binding.AttendBatch(lengths.cuda(), table))
    S.attend(cache, q, y)
    torch.cuda.synchronize()
    assert S.flags() == 0
    spread = first.view(kv_heads, 1, dim).expand(-1, group, -1).reshape(-1).cuda()
    assert torch.equal(y[:-1], spread.expand(n - 1, -1))
    # Equal weights, so the mean of the pages.  The weights are 1 and their sum is exact.  A wave adds
    # 2^18 of the values with a rounding each, of 2^-24 of the sum of their sizes at most (3.1 on
    # average): 2^-6 x 3.1 < 2^-4 of the mean, which is then rounded to bf16.
    want = (total / (2 * page)).view(kv_heads, 1, dim).expand(-1, group, -1).reshape(-1)
    bound = 2.0 ** -8 * want.abs() + 2.0 ** -4
    assert ((y[-1].double().cpu() - want).abs() <= bound).all()
    cache.close()
    S.close()


def test_a_bound_call_without_a_plan_of_its_own():
    r = Requests(31, "bf16", "native", 4, 2, 64, 64, [1] * 5, [100, 1, 257, 60, 5], [])
    S, cache = r.make()
    batch, q = r.batch(), r.q.cuda()
    y, z = torch.empty_like(q), torch.empty_like(q)
    first = S.bind_attend(cache, 4, q, y, batch)
    second = S.bind_attend(cache, 4, q, z, batch, prepare=False)
    fewer = S.bind_attend(cache, 4, q[:2], z[:2], batch, prepare=False)
    first()
    second()
    torch.cuda.synchronize()
    assert torch.equal(y, z)
    with pytest.raises(ValueError):
        fewer()
    with pytest.raises(ValueError):
        S.attend(cache, q[:2], z[:2])
    cache.close()
    S.close()
