"""The gated feed-forward on 4-bit weights (lora_base_gated) on the GPU against its formula
in 64 bits."""
import pytest
import torch

from gpu_util import log
from lora_adapter_application_amd import binding
from layer_util import (HALF_STEP, TORCH, U32, act64, base_sum, check_within, guarded,
                        integer_weight, random_weight)

pytestmark = pytest.mark.gpu

# The largest slope of each activation (silu 1.0998, gelu 1.1290, its tanh form 1.1290)
# and of its size over that of its argument (1).
SLOPE = 1.13


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load_library()


def expected(x, wg, wu, bias, add, d_in, group, kind):
    """act(g) u in 64 bits and the bound of its error: that of the two sums (with a step
    for each of bias and add) through the product, eight steps of 32 bits of the activation
    relative to |g|, one of the product, and the rounding of the result."""
    (g, eg), (u, eu) = (base_sum(x, w, d_in, group) for w in (wg, wu))
    for k, extra in enumerate((bias, add)):
        if extra[0] is not None:
            g = g + extra[0].double()
            eg = eg + U32 * (g.abs() + extra[0].double().abs())
        if extra[1] is not None:
            u = u + extra[1].double()
            eu = eu + U32 * (u.abs() + extra[1].double().abs())
    a = act64(g, kind)
    ea = SLOPE * eg + 8 * U32 * g.abs()
    want = a * u
    bound = ea * u.abs() + a.abs() * eu + ea * eu + U32 * want.abs()
    return want, bound + HALF_STEP[x.dtype] * (want.abs() + bound)


CASES = [
    # dtype, tokens, d_in, d_out, group, zero, bias, gate_add, up_add, activation
    ("bf16", 1, 4096, 264, 128, True, False, False, False, "silu"),
    ("bf16", 1, 8, 8, 0, True, True, True, True, "gelu"),
    ("bf16", 7, 1000, 136, 32, False, True, False, True, "gelu_tanh"),
    ("bf16", 16, 512, 40, 64, True, False, True, False, "silu"),
    ("bf16", 17, 640, 520, 128, True, False, True, True, "silu"),
    ("bf16", 33, 2056, 72, 256, True, True, True, True, "gelu"),
    ("bf16", 65, 392, 1032, 32, True, False, False, False, "silu"),
    ("bf16", 257, 1024, 264, 128, False, False, True, True, "gelu_tanh"),
    ("bf16", 600, 264, 776, 64, True, True, False, False, "silu"),
    ("fp32", 1, 1000, 264, 32, True, True, True, True, "silu"),
    ("fp32", 40, 640, 72, 128, True, False, False, True, "gelu"),
    ("fp32", 130, 264, 136, 0, False, False, True, False, "gelu_tanh"),
]


@pytest.mark.parametrize("dtype,tokens,d_in,d_out,group,zero,bias,gadd,uadd,act", CASES)
def test_gated(dtype, tokens, d_in, d_out, group, zero, bias, gadd, uadd, act):
    log("case", dtype, tokens, d_in, d_out, group, act)
    gen = torch.Generator().manual_seed(tokens + d_in)
    w = [random_weight(gen, d_out, d_in, group, zero) for _ in range(2)]
    dt = TORCH[dtype]
    val = lambda *s: torch.randn(*s, generator=gen).to(dt)  # noqa: E731
    x = val(tokens, d_in)
    b = [val(d_out) if bias else None for _ in range(2)]
    a = [val(tokens, d_out) if use else None for use in (gadd, uadd)]
    with binding.Slots(1, 1, [(d_in, d_out)] * 2, dtype, tokens) as S:
        for i, (q, s, z) in enumerate(w):
            S.load_base(i, q.cuda(), s.cuda(), None if z is None else z.cuda(), group,
                        None if b[i] is None else b[i].cuda())
        y, intact = guarded(tokens, d_out, dt)
        ad = [None if t is None else t.cuda() for t in a]
        S.base_gated(0, 1, x.cuda(), y, ad[0], ad[1], act)
        want, bound = expected(x, w[0], w[1], b, a, d_in, group, act)
        log("  worst error / bound %.3f" % check_within(y, want, bound, "gated"))
        intact()
        # y may be either of the two updates
        for k in (0, 1):
            if ad[k] is None:
                continue
            into = [None if t is None else t.clone() for t in ad]
            S.base_gated(0, 1, x.cuda(), into[k], into[0], into[1], act)
            assert torch.equal(into[k], y)
        # the same module on both sides
        S.base_gated(1, 1, x.cuda(), y, None, None, act)
        want, bound = expected(x, w[1], w[1], [b[1], b[1]], [None, None], d_in, group, act)
        check_within(y, want, bound, "one module twice")


# One case for each way the library multiplies.
WAYS = [("bf16", 9, 8200), ("bf16", 129, 4104), ("bf16", 257, 4104), ("bf16", 449, 4104),
        ("bf16", 1025, 4104),
        ("fp32", 9, 8200), ("fp32", 17, 8200), ("fp32", 65, 8200)]


@pytest.mark.parametrize("group,zero", [(0, True), (128, False), (64, True), (64, False),
                                        (32, True), (32, False)])
@pytest.mark.parametrize("dtype,tokens,d_out", WAYS)
def test_every_way(dtype, tokens, d_out, group, zero):
    d_in = 264
    log("case", dtype, tokens, d_out, group, zero)
    gen = torch.Generator().manual_seed(tokens + group)
    w = [random_weight(gen, d_out, d_in, group, zero) for _ in range(2)]
    x = torch.randn(tokens, d_in, generator=gen).to(TORCH[dtype])
    a = [torch.randn(tokens, d_out, generator=gen).to(TORCH[dtype]) for _ in range(2)]
    with binding.Slots(1, 1, [(d_in, d_out)] * 2, dtype, tokens) as S:
        for i, (q, s, z) in enumerate(w):
            S.load_base(i, q.cuda(), s.cuda(), None if z is None else z.cuda(), group)
        y, intact = guarded(tokens, d_out, TORCH[dtype])
        S.base_gated(0, 1, x.cuda(), y, a[0].cuda(), a[1].cuda())
        want, bound = expected(x, w[0], w[1], [None] * 2, a, d_in, group, "silu")
        check_within(y, want, bound, "gated")
        intact()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("tokens", [1, 80])
def test_activations_far_from_zero(act, tokens):
    """Arguments from -80 to 80, and infinities: no overflow turns into a NaN that the
    formula does not have."""
    d = 128
    gen = torch.Generator().manual_seed(9)
    w = [integer_weight(gen, d, d, 128, True) for _ in range(2)]
    x = torch.zeros(tokens, d).bfloat16()
    ga = torch.linspace(-80, 80, d).repeat(tokens, 1).bfloat16()
    ua = torch.full((tokens, d), 3.0).bfloat16()
    ga[0, 0], ga[0, 1], ga[0, 2] = float("inf"), float("nan"), float("-inf")
    with binding.Slots(1, 1, [(d, d)] * 2, "bf16", tokens) as S:
        for i, (q, s, z) in enumerate(w):
            S.load_base(i, q.cuda(), s.cuda(), z.cuda(), 128)
        y = torch.empty(tokens, d, dtype=torch.bfloat16, device="cuda")
        S.base_gated(0, 1, x.cuda(), y, ga.cuda(), ua.cuda(), act)
    y = y.cpu().double()
    assert y[0, 0] == float("inf") and y[0, 1].isnan() and y[0, 2].isnan()
    g = ga.double()
    want = act64(g, act) * 3
    fine = torch.ones(tokens, d, dtype=torch.bool)
    fine[0, :3] = False
    bound = 3 * 8 * U32 * g.abs() + 2.0 ** -8 * want.abs() + 2.0 ** -133
    assert bool(((y - want).abs() <= bound)[fine].all())


def test_nonfinite_rows():
    d_in, n, tokens = 264, 24, 6
    gen = torch.Generator().manual_seed(5)
    w = [random_weight(gen, n, d_in, 64, True) for _ in range(2)]
    x = torch.randn(tokens, d_in, generator=gen).bfloat16()
    x[1, 3] = float("inf")
    x[2, 100] = float("nan")
    with binding.Slots(1, 1, [(d_in, n)] * 2, "bf16", tokens) as S:
        for i, (q, s, z) in enumerate(w):
            S.load_base(i, q.cuda(), s.cuda(), z.cuda(), 64)
        y = torch.empty(tokens, n, dtype=torch.bfloat16, device="cuda")
        S.base_gated(0, 1, x.cuda(), y)
    y = y.cpu()
    sums = []
    for q, s, z in w:
        v = torch.stack((q & 15, q >> 4), 2).view(n, d_in).double()
        of = torch.arange(d_in) // 64
        full = (v - z.double()[:, of]) * s.double()[:, of]
        sums.append((x.double()[:, None, :] * full[None]).sum(2))
    want = act64(sums[0], "silu") * sums[1]
    assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y.isinf(), want.isinf())
    keep = [0, 3, 4, 5]
    ref, bound = expected(x[keep], w[0], w[1], [None] * 2, [None] * 2, d_in, 64, "silu")
    check_within(y[keep], ref, bound, "finite rows")


def test_refusals():
    gen = torch.Generator().manual_seed(4)
    mods = [(256, 64), (256, 64), (256, 72), (256, 64), (256, 64)]
    w = [random_weight(gen, n, k, 128, True) for k, n in mods]
    x = torch.randn(8, 256, generator=gen).bfloat16().cuda()
    y = torch.full((8, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    E = binding
    with binding.Slots(1, 1, mods, "bf16", 8) as S:
        def refused(want, call, text=""):
            with pytest.raises(binding.LoraError) as e:
                call()
            assert e.value.status == want and text in str(e.value), str(e.value)
        gated = lambda g, u, **kw: binding.lora_base_gated(S.ctx, g, u, kw.pop("x", x),  # noqa: E731
                                                           kw.pop("y", y), **kw)
        for i, (q, s, z) in enumerate(w[:4]):
            if i == 3:
                q, s, z = random_weight(gen, 64, 256, 32, True)
            S.load_base(i, q.cuda(), s.cuda(), z.cuda(), 32 if i == 3 else 128)
        refused(E.LORA_ERR_BAD_MODULE, lambda: gated(0, 5))
        refused(E.LORA_ERR_BAD_MODULE, lambda: gated(-1, 0))
        refused(E.LORA_ERR_INVALID_ARGUMENT, lambda: gated(0, 4), "no base weight")
        refused(E.LORA_ERR_INVALID_ARGUMENT, lambda: gated(0, 2), "shapes")
        refused(E.LORA_ERR_INVALID_ARGUMENT, lambda: gated(0, 3), "group storage")
        refused(E.LORA_ERR_INVALID_ARGUMENT, lambda: gated(0, 1, activation=3), "activation")
        refused(E.LORA_ERR_INVALID_ARGUMENT, lambda: gated(0, 1, y=None), "NULL")
        refused(E.LORA_ERR_INVALID_ARGUMENT, lambda: gated(0, 1, n_tokens=-2))
        refused(E.LORA_ERR_TOO_MANY_TOKENS, lambda: gated(0, 1, n_tokens=9))
        whole = torch.full((9, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        refused(E.LORA_ERR_INVALID_ARGUMENT, lambda: gated(0, 1, y=whole[:8], up_add=whole[1:]), "overlaps")
        refused(E.LORA_ERR_INVALID_ARGUMENT,
                lambda: gated(0, 1, y=x.view(-1)[:512].view(8, 64)), "overlaps")
        with pytest.raises(ValueError):
            S.base_gated(0, 1, x, y, activation="relu")
        S.base_gated(0, 1, x, y, n_tokens=0)
        torch.cuda.synchronize()
        assert bool((y == 5).all()) and bool((whole == 5).all())
