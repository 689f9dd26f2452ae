"""Rotary positions (lora_rotary_group) on the GPU against the formula in 64 bits."""
import math

import pytest
import torch

from gpu_util import log
from lora_adapter_application_amd import binding
from layer_util import HALF_STEP, TORCH, check_within, guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load_library()


def rotated(x, rot, positions):
    """The formula, with the turns of `rot`, in 64 bits: (result, bound of its error).

    An angle is off by 2^-52 of its turns (its product in double); cosine and sine in fp32
    by 2^-22 for bf16 data (the fraction of a turn, at most 1/2, is rounded to fp32 and
    times 2 pi, and the functions and the factor round three times) and by 2^-23 for fp32
    data; the two products and their sum round three times."""
    turns = torch.tensor(list(rot.turns)[:rot.rotary_dim // 2], dtype=torch.float64)
    t = positions.double()[:, None] * turns
    w = 2 * math.pi * (t - t.round())[:, None, :]
    h = x.double().view(x.shape[0], -1, rot.head_dim)
    rd, half = rot.rotary_dim, rot.rotary_dim // 2
    out, size = h.clone(), torch.zeros_like(h)
    i, j = (slice(0, half), slice(half, rd)) if rot.layout == 0 else (slice(0, rd, 2), slice(1, rd, 2))
    a, b = h[..., i], h[..., j]
    out[..., i] = rot.amplitude * (a * w.cos() - b * w.sin())
    out[..., j] = rot.amplitude * (b * w.cos() + a * w.sin())
    size[..., i] = size[..., j] = rot.amplitude * (a.abs() + b.abs())
    trig = (2.0 ** -20 if x.dtype == torch.bfloat16 else 2.0 ** -23) + 3 * 2.0 ** -24
    far = 2.0 ** -52 * 2 * math.pi * t.abs().max().item()
    bound = size * (trig + far)
    out, bound = out.reshape(x.shape), bound.reshape(x.shape)
    return out, bound + HALF_STEP[x.dtype] * (out.abs() + bound)


SETTINGS = [
    # dtype, tokens, heads, head_dim, rotary_dim, layout, scaling, span
    ("bf16", 1, [32, 32], 128, 128, "half", "none", 2048),
    ("bf16", 3, [64, 8], 128, 128, "half", "yarn", 131072),
    ("bf16", 257, [5, 1, 2], 128, 128, "interleaved", "banded", 131072),
    ("bf16", 64, [7, 3], 80, 32, "half", "linear", 65536),
    ("bf16", 33, [12], 80, 20, "half", "none", 4096),          # a pair at a time
    ("bf16", 33, [12], 80, 20, "interleaved", "none", 4096),
    ("bf16", 40, [9, 2], 96, 64, "interleaved", "linear", 1 << 20),
    ("bf16", 2100, [3, 1], 64, 64, "half", "none", 1 << 30),
    ("bf16", 17, [4], 256, 256, "half", "none", 100),
    ("bf16", 17, [2], 320, 256, "interleaved", "none", 100),
    ("bf16", 5, [4], 4, 2, "half", "none", 100),
    ("fp32", 1, [1], 2, 2, "interleaved", "none", 100),
    ("fp32", 130, [6, 2], 64, 64, "half", "yarn", 1 << 20),
    ("fp32", 65, [12, 4], 80, 20, "interleaved", "linear", 65536),
    ("fp32", 65, [12, 4], 80, 18, "half", "banded", 1 << 30),
]
SCALING = {"none": {}, "linear": dict(factor=4.0),
           "yarn": dict(factor=8.0, original_positions=16384),
           "banded": dict(factor=8.0, original_positions=8192, low_factor=1.0, high_factor=4.0)}


@pytest.mark.parametrize("dtype,tokens,heads,head_dim,rotary_dim,layout,scaling,span", SETTINGS)
def test_rotation(dtype, tokens, heads, head_dim, rotary_dim, layout, scaling, span):
    """Out of place, in place, off a 16-byte boundary: the same bits, inside the bound, and
    nothing but the rows written; the elements past rotary_dim are copied exactly."""
    log("case", dtype, tokens, heads, head_dim, rotary_dim, layout, scaling)
    gen = torch.Generator().manual_seed(tokens + head_dim)
    dt = TORCH[dtype]
    rot = binding.lora_rotary_init(head_dim, rotary_dim, layout, scaling=scaling, **SCALING[scaling])
    widths = [h * head_dim for h in heads]
    # modules are multiples of 8 wide: narrow heads come in groups
    widths = [-(-w // 8) * 8 if w % 8 else w for w in widths]
    x = [torch.randn(tokens, w, generator=gen).to(dt) for w in widths]
    pos = torch.randint(span, (tokens,), generator=gen, dtype=torch.int32)
    pos[0] = span - 1
    if tokens > 2:
        pos[1], pos[2] = 0, -5
    with binding.Slots(1, 1, [(8, w) for w in widths], dtype, tokens) as S:
        mods = list(range(len(widths)))
        xd = [t.cuda() for t in x]
        y = [guarded(tokens, w, dt) for w in widths]
        S.rotary_group(rot, mods, xd, [t for t, _ in y], pos.cuda())
        for i in mods:
            want, bound = rotated(x[i], rot, pos)
            check_within(y[i][0], want, bound, f"module {i}")
            y[i][1]()
            assert torch.equal(xd[i].cpu(), x[i])
            rest = y[i][0].cpu().view(tokens, -1, head_dim)[..., rotary_dim:]
            assert torch.equal(rest, x[i].view(tokens, -1, head_dim)[..., rotary_dim:])
        for off in (0, 1):
            z = [guarded(tokens, w, dt, off) for w in widths]
            for i in mods:
                z[i][0].copy_(x[i])
            S.rotary_group(rot, mods, [t for t, _ in z], [t for t, _ in z], pos.cuda())
            for i in mods:
                assert torch.equal(z[i][0], y[i][0]), (off, i)
                z[i][1]()


def test_farthest_positions_keep_their_angle():
    rot = binding.lora_rotary_init(128)
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, -(2 ** 24) - 1], dtype=torch.int32)
    x = torch.randn(4, 256, generator=torch.Generator().manual_seed(1))
    with binding.Slots(1, 1, [(8, 256)], "fp32", 4) as S:
        y = torch.empty(4, 256, device="cuda")
        S.rotary_group(rot, [0], [x.cuda()], [y], pos.cuda())
        want, bound = rotated(x, rot, pos)
        check_within(y, want, bound, "far")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_negative_positions_are_the_inverse_and_the_gradient(layout):
    """R(-p) R(p) = amplitude^2, and the gradient of sum(g * R(p) x) in x is R(-p) g, against
    the formula's and against differences."""
    rot = binding.lora_rotary_init(64, 48, layout, scaling="yarn", factor=4.0, original_positions=512)
    gen = torch.Generator().manual_seed(2)
    t, w = 9, 128
    x, g = torch.randn(t, w, generator=gen), torch.randn(t, w, generator=gen)
    pos = torch.randint(-3000, 3000, (t,), generator=gen, dtype=torch.int32)
    with binding.Slots(1, 1, [(8, w)], "fp32", t) as S:
        def turn(v, p):
            y = torch.empty(t, w, device="cuda")
            S.rotary_group(rot, [0], [v.float().cuda()], [y], p.cuda())
            return y.cpu()
        back = turn(turn(x, pos), -pos).view(t, -1, 64)
        a2 = float(rot.amplitude) ** 2
        want = x.view(t, -1, 64).clone()
        want[..., :48] *= a2
        # two rotations of values below 5.2 * 1.2^2, each step off by 2^-21
        assert (back - want).abs().max() < 2 * 2.0 ** -21 * 10
        grad = turn(g, -pos)
        xr = x.double().requires_grad_()
        out, _ = rotated_graph(xr, rot, pos)
        formula, = torch.autograd.grad((out * g.double()).sum(), xr)
        assert (grad - formula).abs().max() < 2.0 ** -20 * 8
        # differences of the kernel itself: it is linear, so a wide step costs no accuracy
        for row, col in ((0, 0), (3, 47), (5, 63), (8, 100), (2, 24)):
            d = torch.zeros(t, w)
            d[row, col] = 1.0
            diff = ((turn(x + d, pos).double() - turn(x - d, pos).double()) / 2 * g.double()).sum()
            assert abs(diff - grad[row, col]) < 2.0 ** -20 * 64


def rotated_graph(x, rot, positions):
    turns = torch.tensor(list(rot.turns)[:rot.rotary_dim // 2], dtype=torch.float64)
    w = (2 * math.pi * positions.double()[:, None] * turns)[:, None, :]
    h = x.view(x.shape[0], -1, rot.head_dim)
    rd, half = rot.rotary_dim, rot.rotary_dim // 2
    if rot.layout == 0:
        a, b = h[..., :half], h[..., half:rd]
    else:
        a, b = h[..., 0:rd:2], h[..., 1:rd:2]
    p = rot.amplitude * (a * w.cos() - b * w.sin())
    q = rot.amplitude * (b * w.cos() + a * w.sin())
    turned = torch.cat((p, q), 2) if rot.layout == 0 else torch.stack((p, q), 3).flatten(2)
    return torch.cat((turned, h[..., rd:]), 2).reshape(x.shape), None


def test_infinities_stay_in_their_pairs_and_no_rows_behind_the_batch_change():
    rot = binding.lora_rotary_init(128)
    x = torch.randn(4, 128, generator=torch.Generator().manual_seed(3)).bfloat16()
    x[1, 5] = float("inf")
    x[2, 70] = float("nan")
    pos = torch.tensor([1, 2, 3, 4], dtype=torch.int32)
    with binding.Slots(1, 1, [(8, 128)], "bf16", 4) as S:
        y = torch.full((4, 128), 9.0, dtype=torch.bfloat16, device="cuda")
        S.rotary_group(rot, [0], [x.cuda()], [y], pos.cuda(), n_tokens=3)
        y = y.cpu()
    assert bool((y[3] == 9).all())
    bad = ~torch.isfinite(y[:3])
    want = torch.zeros(3, 128, dtype=torch.bool)
    want[1, 5] = want[1, 69] = want[2, 6] = want[2, 70] = True
    assert torch.equal(bad, want)


def test_graph_replays_read_the_positions_of_the_replay():
    rot = binding.lora_rotary_init(64, scaling="linear", factor=2.0)
    gen = torch.Generator().manual_seed(4)
    t = 50
    x = torch.randn(t, 512, generator=gen).bfloat16().cuda()
    pos = torch.zeros(t, dtype=torch.int32, device="cuda")
    with binding.Slots(1, 1, [(8, 512)], "bf16", t) as S:
        y, e = torch.empty_like(x), torch.empty_like(x)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            S.rotary_group(rot, [0], [x], [y], pos)
        for k in range(4):
            pos.copy_(torch.randint(10000, (t,), generator=gen, dtype=torch.int32))
            x.normal_()
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            S.rotary_group(rot, [0], [x], [e], pos)
            torch.cuda.synchronize()
            assert torch.equal(y, e), k


def test_refusals():
    rot = binding.lora_rotary_init(64)
    x = torch.randn(4, 128).bfloat16().cuda()
    y = torch.full((4, 128), 2.0, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    E = binding
    with binding.Slots(1, 1, [(8, 128), (8, 96)], "bf16", 4) as S:
        def refused(want, call, text=""):
            with pytest.raises(binding.LoraError) as e:
                call()
            assert e.value.status == want and text in str(e.value), str(e.value)
        ctx = S.ctx
        refused(E.LORA_ERR_BAD_MODULE, lambda: binding.lora_rotary_group(ctx, rot, [2], [x], [y], pos))
        refused(E.LORA_ERR_INVALID_ARGUMENT,
                lambda: binding.lora_rotary_group(ctx, rot, [1], [x], [y], pos), "whole heads")
        refused(E.LORA_ERR_TOO_MANY_TOKENS,
                lambda: binding.lora_rotary_group(ctx, rot, [0], [x], [y],
                                                  torch.zeros(5, dtype=torch.int32, device="cuda")))
        refused(E.LORA_ERR_INVALID_ARGUMENT,
                lambda: binding.lora_rotary_group(ctx, binding.Rotary(), [0], [x], [y], pos), "rotary")
        bad = binding.lora_rotary_init(64)
        bad.rotary_dim = 300
        refused(E.LORA_ERR_INVALID_ARGUMENT,
                lambda: binding.lora_rotary_group(ctx, bad, [0], [x], [y], pos), "rotary")
        refused(E.LORA_ERR_INVALID_ARGUMENT,
                lambda: binding.lora_rotary_group(ctx, rot, [0, 0], [x, x], [y, y], pos))
        whole = torch.full((6, 128), 2.0, dtype=torch.bfloat16, device="cuda")
        refused(E.LORA_ERR_INVALID_ARGUMENT,
                lambda: S.rotary_group(rot, [0], [whole[:4]], [whole[1:5]], pos), "overlaps")
        refused(E.LORA_ERR_INVALID_ARGUMENT,
                lambda: S.rotary_group(rot, [0, 0], [whole[:2], x], [y, whole[1:3]], pos, n_tokens=2),
                "overlaps")
        with pytest.raises(ValueError):
            S.rotary_group(rot, [0], [x], [y], pos.long())
        with pytest.raises(ValueError):
            S.rotary_group(rot, [0], [x[:2]], [y], pos)
        S.rotary_group(rot, [0], [x], [y], pos, n_tokens=0)
        torch.cuda.synchronize()
        assert bool((y == 2).all()) and bool((whole == 2).all())
        S.rotary_group(rot, [0], [x], [y], pos)       # position 0 turns nothing
        assert torch.equal(x, y)
