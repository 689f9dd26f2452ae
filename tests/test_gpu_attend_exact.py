"""Attention on inputs whose exact result shows the bits of the weights."""
import copy
import math

import pytest
import torch

from attend_util import Requests
from gpu_util import log
from layer_util import HALF_STEP, U32
from lora_adapter_application_amd import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load_library()


SCALE = math.log(2.0)                                         # scores are q . k in powers of two


def attended(r):
    S, cache = r.make()
    S.flags()
    q = r.q.cuda()
    y = torch.full_like(q, 7.0)
    S.attend_prepare(cache, r.heads, r.batch())
    S.attend(cache, q, y, SCALE)
    torch.cuda.synchronize()
    assert S.flags() == 0
    S.close()
    return y.cpu()


WEIGHTS = [
    # queries, lengths, prefixes: blocks that all rows see whole, in part, of a shared prefix
    ([1], [160], []),
    ([1], [147], []),
    ([5, 3], [150, 140], []),
    ([1, 1, 2], [2, 3, 2], [(0, 2, 160), (2, 3, 150)]),
]


@pytest.mark.parametrize("batch", WEIGHTS, ids=str)
@pytest.mark.parametrize("kind", ["native", "fp8", "int8"])
def test_bits_of_the_weights_of_few_rows(kind, batch):
    """Up to 32 rows of a key-value head take their weights in two parts.  Dim d has the value 1 at token
    d + 1, whose weight p is 2^-a, and -round(p) at token 0, whose weight is 1: what is left of the sum
    is the rounding of p, next to nothing, and the result's own rounding is of that.

    The bound, of the sum of the weighted values' sizes: 2^-15 for the parts (the first cut off at 2^-7, the second
    rounded by 2^-8 of that; 2^-16 where the first is rounded), 2^-19 for scores under 2^3 with few roundings and
    their exponentials, 2 u a token and 64 u for the sums and the join."""
    log(f"case weights {kind} {batch}")
    queries, lengths, prefixes = batch
    r = Requests(7, "bf16", kind, 4, 2, 128, 32, queries, lengths, prefixes)
    r.k[r.used] = r.v[r.used] = 0
    a = (37 * torch.arange(1, 129) % 251 + 1).double() / 32   # 1/32 .. 251/32, 8 bits
    near = (2.0 ** -a).to(torch.bfloat16)
    for row, length in ([(r.prefix_table[p], prefixes[p][2]) for p in range(len(prefixes))] if prefixes
                        else list(zip(r.table, lengths))):
        at = r.slots_of(row, length)
        r.v[at[0]] = -near
        for d in range(128):
            r.k[at[d + 1], :, 0] = -a[d].to(torch.bfloat16)
            r.v[at[d + 1], :, d] = 1
    r.q.view(r.tokens, 4, 128)[..., 0] = 1
    r.q.view(r.tokens, 4, 128)[..., 1:] = 0
    got, (want, _) = attended(r).double(), r.attended(SCALE)
    sizes = copy.copy(r)
    sizes.v = r.v.abs()
    whole = sizes.attended(SCALE)[0]
    rows = r.own_rows()
    n = max(lengths) + max([p[2] for p in prefixes] + [0])
    bound = whole * ((2.0 ** -15 if kind == "native" else 2.0 ** -16) + 2.0 ** -19 + (2 * n + 64) * U32)
    bound = (bound + HALF_STEP[torch.bfloat16] * (want.abs() + bound))[rows]
    err = (got - want).abs()[rows]
    assert bool((err <= bound).all()), f"{int((err > bound).sum())} of {err.numel()}, worst {(err / bound).max():.1f}"
    # weights of one part would be off by more than that in many dims
    p = 2.0 ** -a
    off = (p - near.double()).abs() / (n - 128 + p.sum())
    assert (off > bound[0].view(4, 128)[0]).double().mean() > 0.25


@pytest.mark.parametrize("score", [0.0, -1.5, -20.0, -100.0, -120.0])
@pytest.mark.parametrize("length", [256, 230])
def test_infinite_values_under_weights_of_few_bits(length, score):
    """A weight that one part holds, however small it is: the other part of it is not 0 times infinity."""
    r = Requests(8, "bf16", "native", 2, 1, 64, 32, [1, 2], [length, length], [])
    r.k[r.used] = 0
    r.q.view(r.tokens, 2, 64)[..., 0] = 1
    for row in r.table:
        at = r.slots_of(row, length)
        r.k[at[40], 0, 0] = score
        r.v[at[40], 0, 3], r.v[at[40], 0, 4] = math.inf, -math.inf
    got = attended(r).view(r.tokens, 2, 64).float()
    assert (got[..., 3] == math.inf).all() and (got[..., 4] == -math.inf).all()
    got[..., 3:5] = 0
    assert torch.isfinite(got).all()
