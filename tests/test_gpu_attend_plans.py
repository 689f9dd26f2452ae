"""Batches of attention after each other on one ctx: each by its own plan."""
import pytest
import torch

from attend_util import Requests, check_rows
from gpu_util import log
from lora_adapter_application_amd import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load_library()


def cache_of(S, r):
    cache = S.cache(r.kv, r.dim, r.pages, r.page, r.kind)
    r.fill(S, cache)
    return cache


@pytest.mark.parametrize("requests,heads,kv_heads", [(64, 2, 2), (200, 16, 2), (300, 4, 1), (3, 1, 1)])
@pytest.mark.parametrize("queries", [2, 64, 512])
def test_single_tokens_without_starts_whatever_the_most_new_tokens(requests, heads, kv_heads, queries):
    """Behind a batch of prompts, whose plan has wide tiles."""
    log(f"case {requests} requests, {heads} heads on {kv_heads}, at most {queries}")
    prompts = Requests(41, "bf16", "native", heads, kv_heads, 64, 32, [100, 70, 3], [200, 70, 9], [(0, 2, 90)])
    r = Requests(42, "bf16", "native", heads, kv_heads, 64, 32, [1] * requests, [7 * i % 90 for i in range(requests)],
                 q_start=False, tail=400)
    S = binding.Slots(1, 1, [(64, 64)], "bf16", 4096)
    many, few = cache_of(S, prompts), cache_of(S, r)
    pq = prompts.q.cuda()
    py = torch.full_like(pq, 7.0)
    S.attend_prepare(many, heads, prompts.batch())
    S.attend(many, pq, py)
    torch.cuda.synchronize()
    b, q = r.batch(), r.q.cuda()
    b.max_queries = queries
    y = torch.full_like(q, 7.0)
    before = y.clone()
    S.attend_prepare(few, heads, b)
    S.attend(few, q, y)
    torch.cuda.synchronize()
    assert S.flags() == 0
    log(f"  worst error / bound {check_rows(r, y, 64 ** -0.5, before, 'single tokens'):.3f}")
    S.close()


def test_more_tokens_than_a_plan_counts():
    """256 requests that name one page over and over, 2^39 tokens in all: no work, and the flag."""
    n, page, pages = 256, 32768, 65536
    S = binding.Slots(1, 1, [(64, 64)], "bf16", 4096)
    cache = S.cache(1, 8, 1, page, "fp8")
    table = torch.zeros(n, pages, dtype=torch.int32, device="cuda")
    q = torch.ones(n, 8, dtype=torch.bfloat16, device="cuda")
    y = torch.full_like(q, 7.0)
    S.attend_prepare(cache, 1, binding.AttendBatch(torch.full((n,), 2 ** 31 - 1, dtype=torch.int32, device="cuda"), table))
    S.attend(cache, q, y)
    torch.cuda.synchronize()
    assert S.flags() == binding.LORA_FLAG_ATTEND_BATCH
    assert bool((y == 7).all())
    S.close()


def test_the_longest_request():
    """2^31 - 1 tokens, a page over and over: whole blocks are counted up to there.  Equal weights, so
    the mean of the page, whose last token is counted once less."""
    page, pages = 32768, 65536
    S = binding.Slots(1, 1, [(64, 64)], "bf16", page)
    cache = S.cache(1, 8, 1, page, "fp8")
    gen = torch.Generator().manual_seed(6)
    v = torch.randint(1, 8, (page, 8), generator=gen)
    v[:, 0] = 7                                               # a scale of 2^-6 throughout
    S.cache_store(cache, torch.zeros(page, 8).bfloat16().cuda(), v.bfloat16().cuda(),
                  torch.arange(page, dtype=torch.int32).cuda())
    table = torch.zeros(1, pages, dtype=torch.int32, device="cuda")
    q = torch.ones(1, 8, dtype=torch.bfloat16, device="cuda")
    y = torch.full_like(q, 7.0)
    S.attend_prepare(cache, 1, binding.AttendBatch(torch.full((1,), 2 ** 31 - 1, dtype=torch.int32, device="cuda"), table))
    S.attend(cache, q, y)
    torch.cuda.synchronize()
    assert S.flags() == 0
    # The codes of 1..7 in units of 2^-6 are whole numbers, exact.  A wave has 2^31 / 4096 = 2^19 tokens
    # at most of sums up to 7 times that, a lane a fourth of the tokens: both exact in fp32.  The parts'
    # sums are rounded about a thousand times, 2^-24 each.
    want = v.double().mean(0)
    bound = want * (2.0 ** -8 + 2 * 2.0 ** -14 + 2.0 ** -30)
    assert ((y[0].double().cpu() - want).abs() <= bound).all(), (y, want)
    S.close()


def test_a_replayed_graph_leaves_the_eager_plan():
    """prepare, replays of graphs with prepares of other batches, then the layers of the eager step."""
    shapes = [([1] * 40 + [70], list(range(1, 41)) + [90], [(0, 17, 1000), (17, 30, 65)]),
              ([100, 1, 3], [150, 9, 40], [(0, 2, 300)]),
              ([1] * 300, [7 * i % 90 for i in range(300)], [(5, 200, 130)])]
    batches = [Requests(51 + k, "bf16", "fp8", 16, 2, 128, 64, *shape) for k, shape in enumerate(shapes)]
    S = binding.Slots(1, 1, [(64, 64)], "bf16", 4096)
    caches = [cache_of(S, r) for r in batches]
    given = [r.batch() for r in batches]
    q = [r.q.cuda() for r in batches]
    y = [torch.full_like(v, 7.0) for v in q]
    eager = []
    for k in range(3):
        S.attend_prepare(caches[k], 16, given[k])
        S.attend(caches[k], q[k], y[k])
        torch.cuda.synchronize()
        check_rows(batches[k], y[k], 128 ** -0.5, y[k], f"batch {k}")
        eager.append(y[k].clone())
    graphs, s = [], torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for k in range(3):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            S.attend_prepare(caches[k], 16, given[k])
            S.attend(caches[k], q[k], y[k])
    z = [torch.empty_like(v) for v in q]
    for a in range(3):
        S.attend_prepare(caches[a], 16, given[a])
        for b in range(3):
            y[b].fill_(1.0)
            graphs[b].replay()
            z[a].fill_(1.0)
            S.attend(caches[a], q[a], z[a])
            torch.cuda.synchronize()
            assert torch.equal(z[a], eager[a]), (a, b)
            assert torch.equal(y[b], eager[b]), (a, b)
    assert S.flags() == 0
    S.close()


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("fp32", 256)])
@pytest.mark.parametrize("planned", ["native", "fp8"])
def test_layers_of_other_kinds_under_one_plan(dtype, dim, planned):
    shape = (4, 2, dim, 32, [1, 40, 3], [500, 90, 41], [(0, 2, 300)])
    layers = [Requests(61, dtype, kind, *shape) for kind in ("native", "fp8", "int8")]
    S = binding.Slots(1, 1, [(64, 64)], dtype, 4096)
    caches = [cache_of(S, r) for r in layers]
    S.attend_prepare(caches[0 if planned == "native" else 1], 4, layers[0].batch())
    q = layers[0].q.cuda()
    for r, cache in zip(layers, caches):
        y = torch.full_like(q, 7.0)
        before = y.clone()
        S.attend(cache, q, y)
        torch.cuda.synchronize()
        check_rows(r, y, dim ** -0.5, before, r.kind)
    assert S.flags() == 0
    S.close()


def test_bound_calls_after_close():
    r = Requests(62, "bf16", "native", 4, 2, 64, 32, [1] * 3, [40, 3, 64])
    S, cache = r.make()
    q, y, b = r.q.cuda(), torch.empty_like(r.q).cuda(), r.batch()
    k, slots = torch.zeros(3, 128, dtype=torch.bfloat16, device="cuda"), torch.arange(3, dtype=torch.int32, device="cuda")
    calls = [S.bind_cache_store(cache, k, k, slots), S.bind_cache_load(cache, slots, k, k.clone()),
             S.bind_attend(cache, 4, q, y, b), S.bind_attend(cache, 4, q, y, b, prepare=False)]
    for call in calls:
        call()
    torch.cuda.synchronize()
    for close in (cache.close, S.close):
        close()
        for call in calls:
            with pytest.raises(binding.LoraError) as e:
                call()
            assert e.value.status == binding.LORA_ERR_INVALID_ARGUMENT
