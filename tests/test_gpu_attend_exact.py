"""Attention on inputs whose exact result shows each single token and the bits of the weights."""
import copy
import math

import pytest
import torch

from attend_util import Requests
from gpu_util import log
from layer_util import HALF_STEP, TORCH, U32
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


# A value that 8 bits hold with a scale that is a power of two.
UNIT = {"native": 1.0, "fp8": 448 / 512, "int8": 127 / 128}


def selection(seed, *case):
    """A batch whose rows each see one dim of the keys, of which a token has 0 or one unit: the scores
    are 0 or over 2^8 powers of two apart, so weights are 1 or 0 without an error.  Values are -1, 0 or
    1 units."""
    r = Requests(seed, *case)
    unit = UNIT[r.kind]
    k = torch.randint(0, 2, r.k.shape, generator=r.gen).to(r.k.dtype) * unit
    v = torch.randint(-1, 2, r.v.shape, generator=r.gen).to(r.v.dtype) * unit
    k[..., 0] = v[..., 0] = unit                              # the head's largest
    r.k[r.used], r.v[r.used] = k[r.used], v[r.used]
    r.dims = torch.randint(0, r.dim, (r.tokens, r.heads), generator=r.gen)
    r.q.zero_()
    r.q.view(r.tokens, r.heads, r.dim).scatter_(2, r.dims[..., None], 512.0)
    return r


def selected(r):
    """The mean of the values of the tokens that a row sees and selects (of all, if it selects none),
    in 64 bits, and how many tokens those are."""
    out = torch.zeros(r.tokens, r.heads, r.dim, dtype=torch.float64)
    count = torch.ones(r.tokens, r.heads, 1, dtype=torch.float64)
    group = r.heads // r.kv
    for i, (n, length) in enumerate(zip(r.queries, r.lengths)):
        p, at, pre = r.prefix_of(i), r.slots_of(r.table[i], length), 0
        if p >= 0:
            pre = r.prefixes[p][2]
            at = torch.cat((r.slots_of(r.prefix_table[p], pre), at))
        t = torch.arange(r.starts[i], r.starts[i + 1])
        sees = pre + (length - n + torch.arange(n) + 1).clamp_min(0)
        visible = torch.arange(len(at))[None, :] < sees[:, None]
        for h in range(r.heads):
            bits = (r.k[at, h // group].double() > 0)[:, r.dims[t, h]].t() & visible
            bits = torch.where(bits.any(1, keepdim=True), bits, visible).double()
            count[t, h] = bits.sum(1, keepdim=True).clamp_min(1)
            out[t, h] = bits @ r.v[at, h // group].double() / count[t, h]
    return out.view(r.q.shape), count.expand(out.shape).reshape(r.q.shape)


LONG = [
    # requests of many rows over a prefix by themselves and their own tokens: wide tiles
    *[("bf16", kind, 8, 1, dim, 64, [200], [1500], [(0, 1, 900)])
      for kind in ("native", "fp8", "int8") for dim in (64, 96, 128, 256)],
    ("bf16", "native", 8, 2, 128, 32, [700, 3, 90], [1500, 3, 2000], [(0, 1, 900), (1, 3, 1333)]),
    ("bf16", "int8", 8, 2, 128, 32, [700, 3, 90], [1500, 3, 2000], [(0, 1, 900), (1, 3, 1333)]),
    # a prefix of many requests: wide tiles over it, narrow ones over their own tokens
    *[("bf16", kind, 4, 2, dim, 32, [1] * 40, [17 * i % 701 for i in range(40)], [(0, 39, 2300)])
      for kind in ("native", "fp8", "int8") for dim in (64, 96, 128, 256)],
    # narrow tiles alone
    *[("bf16", kind, 8, 2, 128, 64, [1, 1, 2], [5000, 77, 1234], [(1, 3, 800)]) for kind in ("native", "fp8", "int8")],
    ("bf16", "native", 16, 1, 256, 256, [1, 1], [3000, 40], []),
    *[("fp32", kind, 4, 2, 64, 32, [90, 1], [700, 900], [(0, 1, 300)]) for kind in ("native", "fp8", "int8")],
]


@pytest.mark.parametrize("case", LONG, ids=lambda c: "-".join(str(v) for v in c[:6]) + f"-{len(c[6])}x{max(c[6])}")
def test_each_token_counts_once(case):
    """Sums of whole numbers of units, exact in fp32, over a whole number of tokens: reciprocal, product
    and the rounding of the result are all that is between the kernel and the mean.  A token of n left out
    or counted twice moves a sum by a unit, 1 / n of the mean's unit, and the bound is 2^-8 of a mean
    that is about a unit over the root of n."""
    log(f"case selection {case}")
    r = selection(len(str(case)), *case)
    got, (want, count) = attended(r).double(), selected(r)
    rows = r.own_rows()
    bound = want.abs() * (HALF_STEP[TORCH[r.dtype]] * (1 + 4 * U32) + 4 * U32)
    if r.dtype == "bf16" and r.kind == "native":
        # Second parts of weights are 2^-40 of values up to 1, and adding them may round the running sum, which
        # the tokens counted so far bound, by 2^-23 of it for each block of 32 tokens, over the count.
        most = max(r.lengths) + max([p[2] for p in r.prefixes] + [0])
        bound += 2.0 ** -39 + (most / 32 + 8) * 2.0 ** -23
    err, bound = (got - want).abs()[rows], bound[rows]
    assert bool((err <= bound).all()), f"{int((err > bound).sum())} of {err.numel()}, worst {err.max():.3e}"
    # a unit more or less in a sum is out of bounds in most dims (dim 0 has a unit everywhere)
    assert bool(((bound < UNIT[r.kind] / count[rows]).double().mean(-1) > 0.5).all())


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
