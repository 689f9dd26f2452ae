"""Every kernel that the rule on tokens, columns and alignment chooses for the base and the
gated products, with each kind of scale storage, with and without zero points, exact on
integers: the sizes and addresses that the other files leave out."""
import pytest
import torch

from gpu_util import log
from lora_adapter_application_amd import binding
from layer_util import HALF_STEP, TORCH, U32, guarded, integer_weight, levels

pytestmark = pytest.mark.gpu

STORAGE = [(0, True), (0, False), (128, True), (128, False), (64, True), (64, False), (32, True), (32, False)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load_library()


def load(S, module, w, group):
    q, s, z = w
    S.load_base(module, q.cuda(), s.cuda(), None if z is None else z.cuda(), group)


def product(x, w, d_in, group):
    d, s, _ = levels(w, d_in, group)
    return x.cuda().double() @ (d * s).cuda().t().contiguous()


# dtype, tokens, columns, elements that x, add and y lie off a 16-byte boundary
BASE = [("bf16", 1, 264, 0), ("bf16", 2, 8200, 0), ("bf16", 9, 8200, 3), ("bf16", 16, 264, 1),
        ("bf16", 17, 264, 0), ("bf16", 40, 264, 0),              # split, 32 x 32
        ("bf16", 129, 2056, 0),                                  # split, 32 x 64
        ("bf16", 17, 264, 1), ("bf16", 64, 2056, 7),             # two token blocks
        ("bf16", 65, 264, 1), ("bf16", 200, 2056, 3),            # tiles through registers
        ("fp32", 1, 264, 1), ("fp32", 9, 8200, 3), ("fp32", 16, 264, 2),
        ("fp32", 17, 264, 0), ("fp32", 40, 264, 1),              # two token blocks
        ("fp32", 17, 8200, 1), ("fp32", 129, 8200, 3)]           # tiles, K halved; tiles


@pytest.mark.parametrize("group,zero", STORAGE)
@pytest.mark.parametrize("dtype,tokens,n,off", BASE)
def test_base(dtype, tokens, n, off, group, zero):
    d_in = 520 if group else 1000
    log("case", dtype, tokens, n, off, group, zero)
    dt = TORCH[dtype]
    gen = torch.Generator().manual_seed(tokens + group + off)
    w = integer_weight(gen, n, d_in, group, zero)
    x = torch.randint(-4, 5, (tokens, d_in), generator=gen).to(dt)
    a = torch.randint(-4, 5, (tokens, n), generator=gen).to(dt)
    with binding.Slots(1, 1, [(d_in, n)], dtype, tokens) as S:
        load(S, 0, w, group)
        xs, _ = guarded(tokens, d_in, dt, off)
        add, _ = guarded(tokens, n, dt, off)
        y, intact = guarded(tokens, n, dt, off)
        xs.copy_(x)
        add.copy_(a)
        S.base(xs, y, 0, add)
        want = product(x, w, d_in, group) + a.cuda().double()
        assert torch.equal(y, want.float().to(dt))
        intact()


GATED = [("bf16", 1, 264, 0), ("bf16", 5, 8200, 1), ("bf16", 9, 8200, 0), ("bf16", 16, 264, 3),
         ("bf16", 17, 264, 0), ("bf16", 40, 2056, 0), ("bf16", 100, 2056, 0),      # split, 32 x 64
         ("bf16", 17, 264, 1), ("bf16", 40, 2056, 3), ("bf16", 64, 264, 7),        # two token blocks
         ("bf16", 65, 264, 1), ("bf16", 200, 2056, 3),                             # tiles through registers
         ("fp32", 1, 264, 1), ("fp32", 9, 8200, 0), ("fp32", 16, 264, 2),
         ("fp32", 17, 264, 0), ("fp32", 40, 264, 1),                               # two token blocks
         ("fp32", 17, 8200, 3), ("fp32", 65, 8200, 1)]                             # tiles, K halved; tiles


@pytest.mark.parametrize("group,zero", STORAGE)
@pytest.mark.parametrize("dtype,tokens,n,off", GATED)
def test_gated(dtype, tokens, n, off, group, zero):
    """8192 added to gate's sums makes silu the identity (exp(-g) is far below a step of 1):
    y is a product of two exact numbers, rounded to 32 bits and to the type."""
    d_in = 264
    log("case", dtype, tokens, n, off, group, zero)
    dt = TORCH[dtype]
    gen = torch.Generator().manual_seed(tokens + group + off)
    w = [integer_weight(gen, n, d_in, group, zero) for _ in range(2)]
    x = torch.randint(-1, 2, (tokens, d_in), generator=gen).to(dt)
    u_add = torch.randint(-4, 5, (tokens, n), generator=gen).to(dt)
    with binding.Slots(1, 1, [(d_in, n)] * 2, dtype, tokens) as S:
        for i in (0, 1):
            load(S, i, w[i], group)
        xs, _ = guarded(tokens, d_in, dt, off)
        ga, _ = guarded(tokens, n, dt, off)
        ua, _ = guarded(tokens, n, dt, off)
        y, intact = guarded(tokens, n, dt, off)
        xs.copy_(x)
        ga.fill_(8192)
        ua.copy_(u_add)
        S.base_gated(0, 1, xs, y, ga, ua)
        g = product(x, w[0], d_in, group) + 8192
        u = product(x, w[1], d_in, group) + u_add.cuda().double()
        want = g * u
        # at most 264 * 15 below 8192: exp(-g) is 0
        assert bool((g > 200).all())
        bound = (U32 + HALF_STEP[dt] * (1 + U32)) * want.abs()
        assert bool(((y.double() - want).abs() <= bound).all())
        intact()
