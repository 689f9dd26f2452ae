"""Accuracy of the fp32 base products on inputs with a mean, where sums of x (16 + q) grow with
the number of inputs: the relative 2-norm error stays within 16 roundings (2^-24) of the
formula in 64 bits, the limit that zero-mean inputs are held to."""
import pytest
import torch

from gpu_util import log
from lora_adapter_application_amd import binding
from layer_util import U32, levels, random_weight

pytestmark = pytest.mark.gpu
LIMIT = 16 * U32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load_library()


def inputs(kind, gen, tokens, d_in):
    x = torch.randn(tokens, d_in, generator=gen)
    if kind == "narrow":
        return 1 + 0.1 * x
    if kind == "positive":
        return x.abs()
    if kind == "outlier":
        x[:, 5] *= 100
    return x


def load(S, module, w, group):
    q, s, z = w
    S.load_base(module, q.cuda(), s.cuda(), None if z is None else z.cuda(), group)


def product(x, w, d_in, group):
    d, s, _ = levels(w, d_in, group)
    return x.double().cuda() @ (d * s).cuda().t().contiguous()


# few tokens (four column blocks a workgroup, one), two token blocks, tiles with K halved, tiles
@pytest.mark.parametrize("tokens,n", [(1, 8200), (16, 8200), (3, 264), (24, 264), (40, 264),
                                      (64, 4096), (130, 4104), (300, 8200)])
@pytest.mark.parametrize("d_in,group,zero", [(4096, 128, False), (4096, 128, True), (2056, 0, False),
                                             (2048, 64, False), (1000, 32, False)])
def test_products_of_inputs_with_a_mean(tokens, n, d_in, group, zero):
    gen = torch.Generator().manual_seed(tokens + d_in)
    w = random_weight(gen, n, d_in, group, zero)
    with binding.Slots(1, 1, [(d_in, n)], "fp32", tokens) as S:
        load(S, 0, w, group)
        for kind in ("zero mean", "narrow", "positive", "outlier"):
            x = inputs(kind, gen, tokens, d_in)
            y = torch.empty(tokens, n, device="cuda")
            S.base(x.cuda(), y, 0)
            want = product(x, w, d_in, group)
            rel = ((y.double() - want).norm() / want.norm()).item()
            log("case", tokens, n, d_in, group, zero, kind, "%.2e" % rel)
            assert rel <= LIMIT, (kind, rel)


@pytest.mark.parametrize("tokens,n", [(1, 8200), (16, 8200), (3, 264), (24, 264), (130, 4104)])
@pytest.mark.parametrize("d_in,group", [(4096, 128), (2048, 64), (1000, 32)])
def test_gated_products_of_inputs_with_a_mean(tokens, n, d_in, group):
    """A gate whose weights are all 0, and 64 added to it: y = 64 u to within 2^-80."""
    gen = torch.Generator().manual_seed(tokens + d_in)
    up = random_weight(gen, n, d_in, group, False)
    gate = (torch.full_like(up[0], 0x88), up[1], None)
    with binding.Slots(1, 1, [(d_in, n)] * 2, "fp32", tokens) as S:
        load(S, 0, gate, group)
        load(S, 1, up, group)
        add = torch.full((tokens, n), 64.0, device="cuda")
        for kind in ("zero mean", "narrow", "positive"):
            x = inputs(kind, gen, tokens, d_in)
            y = torch.empty(tokens, n, device="cuda")
            S.base_gated(0, 1, x.cuda(), y, add)
            want = 64 * product(x, up, d_in, group)
            rel = ((y.double() - want).norm() / want.norm()).item()
            log("case", tokens, n, d_in, group, kind, "%.2e" % rel)
            assert rel <= LIMIT, (kind, rel)
