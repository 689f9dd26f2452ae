"""Batches with infinities in every row, through each kind of kernel: the base and gated
products give what the formula gives, in bounded time."""
import time

import pytest
import torch

from gpu_util import log
from lora_adapter_application_amd import binding
from layer_util import TORCH, act64, levels, random_weight

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load_library()


def load(S, module, w, group):
    q, s, z = w
    S.load_base(module, q.cuda(), s.cuda(), None if z is None else z.cuda(), group)


def formula(x, w, d_in, group):
    """sum_k x W with the rules of infinities and NaN: in 64 bits, the terms that are not
    finite counted by kind (a product over all inputs would need no more, but a matrix product
    need not multiply what it multiplies by 0)."""
    d, s, _ = levels(w, d_in, group)
    full = (d * s).cuda()
    x = x.double().cuda()
    finite = torch.where(x.isfinite(), x, torch.zeros_like(x))
    y = finite @ full.t().contiguous()
    count = lambda a, b: a.double() @ b.double().t().contiguous() > 0  # noqa: E731
    inf = float("inf")
    plus = count(x == inf, full > 0) | count(x == -inf, full < 0)
    minus = count(x == inf, full < 0) | count(x == -inf, full > 0)
    nan = count(x.isnan(), torch.ones_like(full)) | count(x.isinf(), full == 0) | (plus & minus)
    y[plus] = inf
    y[minus] = -inf
    y[nan] = float("nan")
    return y


def spoil(x, gen, kinds):
    """One row after the other: an infinity; two alike; two opposite; a NaN; none of them."""
    tokens, d_in = x.shape
    at = lambda: int(torch.randint(d_in, (1,), generator=gen))  # noqa: E731
    for t in range(tokens):
        kind = kinds[t % len(kinds)]
        if kind == "one":
            x[t, at()] = float("inf")
        elif kind == "minus":
            x[t, at()] = float("-inf")
        elif kind == "two":
            x[t, at()] = float("inf")
            x[t, at()] = float("inf")
        elif kind == "opposite":
            x[t, at()] = float("inf")
            x[t, at()] = float("-inf")
        elif kind == "last":
            x[t, d_in - 1] = float("inf")
        elif kind == "nan":
            x[t, at()] = float("nan")
        elif kind == "large":      # the finite inputs beside an infinity are too large to skip
            x[t, at()] = float("inf")
            x[t, at()] = 2.0 ** 70
    return x


KINDS = ["one", "minus", "two", "opposite", "last", "nan", "large", "none"]
SIZES = [("bf16", 3, 264), ("bf16", 16, 8200), ("bf16", 40, 264), ("bf16", 129, 2056), ("bf16", 257, 2056),
         ("bf16", 513, 2056), ("bf16", 1025, 2056), ("bf16", 2049, 2056), ("bf16", 2700, 2056),
         ("fp32", 3, 264), ("fp32", 37, 264), ("fp32", 17, 8200), ("fp32", 129, 8200)]


@pytest.mark.parametrize("d_in,group,zero", [(392, 128, True), (264, 32, False), (520, 64, True)])
@pytest.mark.parametrize("dtype,tokens,n", SIZES)
def test_infinities_in_every_row(dtype, tokens, n, d_in, group, zero):
    log("case", dtype, tokens, n, d_in, group, zero)
    gen = torch.Generator().manual_seed(tokens + group)
    w = random_weight(gen, n, d_in, group, zero)
    x = spoil(torch.randn(tokens, d_in, generator=gen).to(TORCH[dtype]), gen, KINDS)
    with binding.Slots(1, 1, [(d_in, n)], dtype, tokens) as S:
        load(S, 0, w, group)
        y = torch.empty(tokens, n, dtype=TORCH[dtype], device="cuda")
        S.base(x.cuda(), y, 0)
        want = formula(x, w, d_in, group)
        assert torch.equal(y.isnan(), want.isnan())
        assert torch.equal(y.isinf(), want.isinf())
        inf = want.isinf()
        assert torch.equal(y.double()[inf], want[inf])


@pytest.mark.parametrize("dtype,tokens,n", [("bf16", 3, 264), ("bf16", 40, 264), ("bf16", 129, 4104),
                                            ("bf16", 257, 4104), ("bf16", 449, 4104), ("bf16", 1025, 4104),
                                            ("fp32", 3, 264), ("fp32", 17, 8200), ("fp32", 65, 8200)])
def test_infinities_in_every_row_of_a_gated_product(dtype, tokens, n):
    log("case", dtype, tokens, n)
    d_in, group = 264, 64
    gen = torch.Generator().manual_seed(tokens)
    w = [random_weight(gen, n, d_in, group, True) for _ in range(2)]
    x = spoil(torch.randn(tokens, d_in, generator=gen).to(TORCH[dtype]), gen, KINDS)
    with binding.Slots(1, 1, [(d_in, n)] * 2, dtype, tokens) as S:
        for i in (0, 1):
            load(S, i, w[i], group)
        y = torch.empty(tokens, n, dtype=TORCH[dtype], device="cuda")
        S.base_gated(0, 1, x.cuda(), y)
        g, u = (formula(x, m, d_in, group) for m in w)
        # a row whose 2^70 fell on its infinity has products of 2^140, past the type's 2^128: the
        # rounding to the type makes them infinite
        want = (act64(g, "silu") * u).float().to(TORCH[dtype]).double()
        assert torch.equal(y.isnan(), want.isnan())
        assert torch.equal(y.isinf(), want.isinf())
        inf = want.isinf()
        assert torch.equal(y.double()[inf], want[inf])


def test_scales_that_are_infinite_or_large_beside_infinities():
    """Where scales do not let the finite inputs be skipped, every term counts."""
    d_in, n, tokens = 256, 32, 5
    gen = torch.Generator().manual_seed(3)
    for dtype in ("bf16", "fp32"):
        q, s, z = random_weight(gen, n, d_in, 128, True)
        s[1, 1] = float("inf")
        s[2, 0] = -float("inf")
        s[3, 1] = float("nan")
        s[4, 0] = 2.0 ** 100
        x = torch.randn(tokens, d_in, generator=gen).to(TORCH[dtype])
        x[:, 3] = float("inf")
        x[1, 200] = float("-inf")
        d, sc, _ = levels((q, s, z), d_in, 128)
        want = (x.double()[:, None, :] * (d * sc)[None]).sum(2)
        with binding.Slots(1, 1, [(d_in, n)], dtype, tokens) as S:
            load(S, 0, (q, s, z), 128)
            y = torch.empty(tokens, n, dtype=TORCH[dtype], device="cuda")
            S.base(x.cuda(), y, 0)
            y = y.cpu().double()
        assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y.isinf(), want.isinf())
        assert torch.equal(y[want.isinf()], want[want.isinf()])


def test_an_infinity_in_every_row_takes_bounded_time():
    """1024 tokens of 4096 -> 4096: whole sums by single threads took 170 times a finite batch,
    a scan of the rows takes some 17 times."""
    tokens, d_in, n = 1024, 4096, 4096
    gen = torch.Generator().manual_seed(3)
    w = random_weight(gen, n, d_in, 128, True)
    x = torch.randn(tokens, d_in, generator=gen).bfloat16().cuda()
    with binding.Slots(1, 1, [(d_in, n)], "bf16", tokens) as S:
        load(S, 0, w, 128)
        y = torch.empty(tokens, n, dtype=torch.bfloat16, device="cuda")

        def best():
            times = []
            for _ in range(4):
                torch.cuda.synchronize()
                t0 = time.perf_counter()
                for _ in range(5):
                    S.base(x, y, 0)
                torch.cuda.synchronize()
                times.append(time.perf_counter() - t0)
            return min(times)
        finite = best()
        x[:, d_in // 2] = float("inf")
        infinite = best()
        log("finite %.0f us, infinite %.0f us" % (finite * 2e5, infinite * 2e5))
        assert infinite <= 60 * finite
