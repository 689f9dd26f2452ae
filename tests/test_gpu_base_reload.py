"""Captured base products and gated products after reloads of their weights: what the header
says a replay sees, at sizes that take each kind of kernel."""
import pytest
import torch

from gpu_util import log
from lora_adapter_application_amd import binding
from layer_util import TORCH, act64, base_sum, integer_weight, levels

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load_library()


def load(S, module, w, group):
    q, s, z = w
    S.load_base(module, q.cuda(), s.cuda(), None if z is None else z.cuda(), group)


def capture(call):
    """A graph of one call, and the stream it was captured on."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    torch.cuda.synchronize()
    return g


# few tokens, split (32 x 32, 64 x 128, 64 x 384), tiles; fp32 few tokens, tiles
SIZES = [("bf16", 3, 264), ("bf16", 40, 264), ("bf16", 513, 2056), ("bf16", 2049, 2056),
         ("bf16", 2700, 2056), ("fp32", 37, 264), ("fp32", 17, 8200), ("fp32", 129, 8200)]


@pytest.mark.parametrize("group", [128, 64, 32])
@pytest.mark.parametrize("dtype,tokens,n", SIZES)
def test_replay_after_a_reload_with_or_without_zero_points(dtype, tokens, n, group):
    """group_size and the presence of a bias are as before, zero points come and go: exact
    integers, so a replay that took another zero point than the loaded one shows."""
    log("case", dtype, tokens, n, group)
    d_in = 392
    gen = torch.Generator().manual_seed(tokens + group)
    ws = [integer_weight(gen, n, d_in, group, zero) for zero in (False, True, False, True)]
    x = torch.randint(-3, 4, (tokens, d_in), generator=gen).to(TORCH[dtype])
    xd = x.cuda()
    wants = []
    for w in ws:
        d, s, _ = levels(w, d_in, group)
        wants.append((xd.double() @ (d * s).cuda().t().contiguous()).float().to(TORCH[dtype]))
    for first in (0, 1):
        with binding.Slots(1, 1, [(d_in, n)], dtype, tokens) as S:
            load(S, 0, ws[first], group)
            S.sync_loads()
            y = torch.zeros(tokens, n, dtype=TORCH[dtype], device="cuda")
            g = capture(lambda: S.base(xd, y, 0))
            for i in (first, 1 - first, 2 + first, 3 - first):
                load(S, 0, ws[i], group)
                S.sync_loads()
                for _ in range(2):
                    y.zero_()
                    torch.cuda.synchronize()
                    g.replay()
                    torch.cuda.synchronize()
                    eager = torch.empty_like(y)
                    S.base(xd, eager, 0)
                    assert torch.equal(eager, wants[i]), ("eager", first, i)
                    assert torch.equal(y, wants[i]), ("replay", first, i)


@pytest.mark.parametrize("dtype,tokens,n", [("bf16", 3, 264), ("bf16", 40, 264), ("bf16", 257, 4104),
                                            ("bf16", 449, 4104), ("bf16", 1025, 4104),
                                            ("fp32", 17, 8200), ("fp32", 65, 8200)])
def test_gated_replay_after_a_reload_with_or_without_zero_points(dtype, tokens, n):
    """Gate's, up's or both modules' zero points come and go.  x and the weights are small
    integers and up's scale is 1, so u is exact; g is 0 or far above 0 (gate_add), where silu
    is 0 or within 2 steps of 32 bits of g: a wrong zero point is off by a whole x."""
    log("case", dtype, tokens, n)
    d_in, group = 264, 128
    gen = torch.Generator().manual_seed(tokens)
    ws = []
    for zero in (False, True):
        for _ in range(2):
            q, s, z = integer_weight(gen, n, d_in, group, zero)
            ws.append((q, torch.ones_like(s), z))
    none, some = ws[:2], ws[2:]
    x = torch.randint(0, 2, (tokens, d_in), generator=gen).to(TORCH[dtype])
    add = torch.full((tokens, n), 8192.0, dtype=TORCH[dtype])
    xd, ad = x.cuda(), add.cuda()

    def want(wg, wu):
        g, u = (xd.double() @ (lambda d, s, z: (d * s))(*levels(w, d_in, group)).cuda().t().contiguous()
                for w in (wg, wu))
        return act64(g + 8192.0, "silu") * u
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    with binding.Slots(1, 1, [(d_in, n)] * 2, dtype, tokens) as S:
        for first in (none, some):
            for i in (0, 1):
                load(S, i, first[i], group)
            S.sync_loads()
            y = torch.zeros(tokens, n, dtype=TORCH[dtype], device="cuda")
            graph = capture(lambda: S.base_gated(0, 1, xd, y, ad, None))
            for wg, wu in ((some[0], none[1]), (none[0], some[1]), (some[0], some[1]), (none[0], none[1])):
                load(S, 0, wg, group)
                load(S, 1, wu, group)
                S.sync_loads()
                eager = torch.empty_like(y)
                S.base_gated(0, 1, xd, eager, ad, None)
                y.zero_()
                torch.cuda.synchronize()
                graph.replay()
                torch.cuda.synchronize()
                w = want(wg, wu)
                # silu's few steps, the product, and the rounding
                bound = (4 * 2.0 ** -24 + half) * 1.01 * w.abs()
                for name, got in (("eager", eager), ("replay", y)):
                    assert bool(((got.double() - w).abs() <= bound).all()), name
                assert torch.equal(eager, y)


def test_group_of_modules_with_and_without_zero_points():
    """Modules of one call keep to their own zero points, also after they change."""
    d_in, tokens, outs = 392, 300, [264, 520, 136]
    gen = torch.Generator().manual_seed(11)
    x = torch.randint(-3, 4, (tokens, d_in), generator=gen).bfloat16()
    xd = x.cuda()
    with binding.Slots(1, 1, [(d_in, n) for n in outs], "bf16", tokens) as S:
        y = [torch.zeros(tokens, n, dtype=torch.bfloat16, device="cuda") for n in outs]
        g = None
        for pattern in ((False, False, False), (True, False, True), (False, True, False)):
            w = [integer_weight(gen, n, d_in, 64, zero) for n, zero in zip(outs, pattern)]
            for i in range(3):
                load(S, i, w[i], 64)
            S.sync_loads()
            if g is None:
                g = capture(lambda: S.base_group([0, 1, 2], [xd] * 3, y))
            for t in y:
                t.zero_()
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            eager = [torch.empty_like(t) for t in y]
            S.base_group([0, 1, 2], [xd] * 3, eager)
            for i in range(3):
                want = base_sum(x, w[i], d_in, 64)[0].float().bfloat16()
                assert torch.equal(eager[i].cpu(), want), ("eager", pattern, i)
                assert torch.equal(y[i].cpu(), want), ("replay", pattern, i)


@pytest.mark.parametrize("tokens", [3, 40, 700])
def test_replay_after_a_reload_in_another_group_size_and_back(tokens):
    """Weights in groups of 128, captured; then others in groups of 32, with more scales and
    a bias; then again groups of 128 without a bias, as at the capture: the replay sees them."""
    d_in, n = 392, 264
    gen = torch.Generator().manual_seed(tokens)
    x = torch.randint(-3, 4, (tokens, d_in), generator=gen).bfloat16()
    xd = x.cuda()
    bias = torch.randint(-3, 4, (n,), generator=gen).bfloat16()
    with binding.Slots(1, 1, [(d_in, n)], "bf16", tokens) as S:
        y = torch.zeros(tokens, n, dtype=torch.bfloat16, device="cuda")
        graph = None
        for group in (128, 32, 256, 64, 128):
            w = integer_weight(gen, n, d_in, group, True)
            b = bias if group == 32 else None
            S.load_base(0, *(t.cuda() for t in w), group, None if b is None else b.cuda())
            S.sync_loads()
            if graph is None:
                graph = capture(lambda: S.base(xd, y, 0))
            want = base_sum(x, w, d_in, group)[0] + (0 if b is None else b.double())
            want = want.float().bfloat16()
            eager = torch.empty_like(y)
            S.base(xd, eager, 0)
            assert torch.equal(eager.cpu(), want), group
            if group < 128:
                continue
            y.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y.cpu(), want), group
