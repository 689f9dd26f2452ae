"""More than 2^24 tokens in a call, past what one row of a grid of workgroups of a token each holds."""
import pytest
import torch

from layer_util import HALF_STEP, U32
from lora_adapter_application_amd import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load_library()


def test_more_than_2_to_the_24_tokens():
    """Heads of 8 of which a pair turns by a quarter a position: whole numbers and signs, and for the
    norm of the rest of the head the formula."""
    n, dim = (1 << 24) + 5, 8
    S = binding.Slots(1, 1, [(8, dim)], "bf16", n)
    rot = binding.lora_rotary_init(dim, 2, "half")
    rot.turns[0] = 0.25
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randint(-8, 9, (n, dim), generator=gen, device="cuda", dtype=torch.int32).to(torch.bfloat16)
    x[:, 7] = 8                                               # no row without a length
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    y = torch.full_like(x, 77.0)
    S.norm_rotary_group(rot, [0], [x], [y], pos, None, 0.0)
    part = 1 << 22
    for at in range(0, n, part):                              # in parts: 64 bits of all would be 1 GiB a copy
        z = x[at:at + part].double()
        z = z / z.square().mean(1, keepdim=True).sqrt()
        a, b = z[:, 0].clone(), z[:, 1].clone()
        quarter = pos[at:at + part] % 4
        z[:, 0] = torch.where(quarter == 0, a, torch.where(quarter == 1, -b, torch.where(quarter == 2, -a, b)))
        z[:, 1] = torch.where(quarter == 0, b, torch.where(quarter == 1, a, torch.where(quarter == 2, -b, -a)))
        # rounded once, of what is off by some 16 roundings in fp32 (cosines of quarters are exact)
        err = (y[at:at + part].double() - z).abs()
        assert bool((err <= z.abs() * (HALF_STEP[torch.bfloat16] + 32 * U32)).all()), at
    S.close()


def test_more_than_2_to_the_24_positions():
    """The same turn without the norm: whole numbers and signs, exact."""
    n, dim = (1 << 24) + 5, 8
    S = binding.Slots(1, 1, [(8, dim)], "bf16", n)
    rot = binding.lora_rotary_init(dim, 2, "half")
    rot.turns[0] = 0.25
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randint(-8, 9, (n, dim), generator=gen, device="cuda", dtype=torch.int32).to(torch.bfloat16)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    y = torch.full_like(x, 77.0)
    S.rotary_group(rot, [0], [x], [y], pos)
    a, b, quarter = x[:, 0], x[:, 1], pos % 4
    assert torch.equal(y[:, 0], torch.where(quarter == 0, a, torch.where(quarter == 1, -b, torch.where(quarter == 2, -a, b))))
    assert torch.equal(y[:, 1], torch.where(quarter == 0, b, torch.where(quarter == 1, a, torch.where(quarter == 2, -b, -a))))
    assert torch.equal(y[:, 2:], x[:, 2:])
    S.close()
