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
