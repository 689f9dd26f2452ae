"""Head norms with rotary positions (lora_norm_rotary_group) on the GPU against the formula in
64 bits."""
import math

import pytest
import torch

from gpu_util import log
from layer_util import HALF_STEP, TORCH, U32, check_within, guarded
from lora_adapter_application_amd import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load_library()


def normed(x, weight, eps, rot, positions):
    """(result, bound of its error) in 64 bits.

    The sum of squares of d values rounds at most d + 6 times (u = 2^-24 each), the mean, eps,
    root and reciprocal five times more, of which the root halves what is before it; the
    products with the factor and the weight round twice.  Angle, cosine and sine are off by what
    the rotary positions' own test derives: 2^-20 of a value for bf16 data and 2^-23 for fp32, and
    2^-52 of the largest turns; the two products and their sum round three times."""
    h = x.double().view(x.shape[0], -1, rot.head_dim)
    z = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    if weight is not None:
        z = z * weight.double()
    turns = torch.tensor(list(rot.turns)[:rot.rotary_dim // 2], dtype=torch.float64)
    t = positions.double()[:, None] * turns
    w = 2 * math.pi * (t - t.round())[:, None, :]
    rd, half = rot.rotary_dim, rot.rotary_dim // 2
    out, size = z.clone(), z.abs()
    i, j = (slice(0, half), slice(half, rd)) if rot.layout == 0 else (slice(0, rd, 2), slice(1, rd, 2))
    a, b = z[..., i], z[..., j]
    out[..., i] = rot.amplitude * (a * w.cos() - b * w.sin())
    out[..., j] = rot.amplitude * (b * w.cos() + a * w.sin())
    size[..., i] = size[..., j] = rot.amplitude * (a.abs() + b.abs())
    trig = (2.0 ** -20 if x.dtype == torch.bfloat16 else 2.0 ** -23) + 3 * U32
    far = 2.0 ** -52 * 2 * math.pi * t.abs().max().item()
    bound = size * (trig + far + ((rot.head_dim + 6) / 2 + 8) * U32)
    out, bound = out.reshape(x.shape), bound.reshape(x.shape)
    return out, bound + HALF_STEP[x.dtype] * (out.abs() + bound)


SETTINGS = [
    # dtype, tokens, heads, head_dim, rotary_dim, layout, scaling, span
    ("bf16", 1, [64, 8], 128, 128, "half", "none", 2048),
    ("bf16", 3, [32, 32], 128, 128, "half", "yarn", 131072),
    ("bf16", 257, [5, 1, 2], 128, 128, "interleaved", "banded", 131072),
    ("bf16", 64, [7, 3], 80, 32, "half", "linear", 65536),
    ("bf16", 33, [12], 80, 20, "half", "none", 4096),          # a pair at a time
    ("bf16", 33, [12], 80, 20, "interleaved", "none", 4096),
    ("bf16", 40, [9, 2], 96, 64, "interleaved", "linear", 1 << 20),
    ("bf16", 2100, [3, 1], 64, 64, "half", "none", 1 << 30),
    ("bf16", 17, [4], 256, 256, "half", "none", 100),
    ("bf16", 17, [4], 256, 16, "half", "none", 100),
    ("bf16", 17, [2], 512, 256, "interleaved", "none", 100),
    ("bf16", 17, [2], 512, 2, "interleaved", "none", 100),
    ("bf16", 17, [2], 320, 250, "half", "none", 100),
    ("bf16", 5, [4], 4, 2, "half", "none", 100),
    ("fp32", 1, [1], 8, 2, "interleaved", "none", 100),
    ("fp32", 130, [6, 2], 64, 64, "half", "yarn", 1 << 20),
    ("fp32", 130, [6, 2], 80, 20, "interleaved", "linear", 1 << 20),
    ("fp32", 9, [2], 512, 256, "half", "none", 1 << 20),
    ("fp32", 9, [2], 512, 200, "interleaved", "none", 1 << 20),
    ("fp32", 9, [3], 90, 90, "half", "none", 1 << 20),
]


def rotary(head_dim, rotary_dim, layout, scaling):
    kw = {} if scaling == "none" else {"factor": 8.0}
    if scaling in ("yarn", "banded"):
        kw["original_positions"] = 4096
    return binding.lora_rotary_init(head_dim, rotary_dim, layout, scaling=scaling, **kw)


@pytest.mark.parametrize("s", SETTINGS, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("where", ["apart", "in place", "off 16 bytes"])
def test_against_64_bits(s, where):
    dtype, tokens, heads, head_dim, rotary_dim, layout, scaling, span = s
    if where == "off 16 bytes" and tokens > 300:
        tokens = 300
    if any(h * head_dim % 8 for h in heads):
        heads = [h * 8 for h in heads]
    log(f"case norm {s} {where}")
    gen = torch.Generator().manual_seed(tokens + head_dim)
    t = TORCH[dtype]
    rot = rotary(head_dim, rotary_dim, layout, scaling)
    S = binding.Slots(1, 1, [(8, h * head_dim) for h in heads], dtype, tokens)
    off = 1 if where == "off 16 bytes" else 0
    x = [(torch.randn(tokens, h * head_dim, generator=gen) * 10 ** (k - 1)).to(t) for k, h in enumerate(heads)]
    weight = [(1 + torch.randn(head_dim, generator=gen)).to(t) if k != 1 else None for k in range(len(heads))]
    pos = torch.randint(-span, span, (tokens,), generator=gen, dtype=torch.int32)
    xd, intact = zip(*[guarded(tokens, v.shape[1], t, off) for v in x])
    for a, b in zip(xd, x):
        a.copy_(b)
    if where == "in place":
        y, more = xd, intact
    else:
        y, more = zip(*[guarded(tokens, v.shape[1], t, off) for v in x])
    wd = [None if w is None else w.cuda() for w in weight]
    S.norm_rotary_group(rot, list(range(len(heads))), xd, y, pos.cuda(), wd, 1e-5)
    torch.cuda.synchronize()
    worst = 0
    for k, v in enumerate(x):
        want, bound = normed(v, weight[k], float(torch.tensor(1e-5)), rot, pos)
        worst = max(worst, check_within(y[k], want, bound, f"member {k}"))
        if where != "in place":
            assert torch.equal(xd[k].cpu(), v)
    for f in (*intact, *more):
        f()
    log(f"  worst error / bound {worst:.3f}")
    S.close()


def test_odd_values():
    """Zeros stay zeros, a head with a NaN or infinity touches no other head."""
    rot = rotary(64, 64, "half", "none")
    S = binding.Slots(1, 1, [(8, 256)], "bf16", 8)
    x = torch.randn(5, 256, dtype=torch.float32).bfloat16().cuda()
    x[1, 64:128] = 0
    clean, y = torch.empty_like(x), torch.empty_like(x)
    pos = torch.arange(5, dtype=torch.int32).cuda()
    S.norm_rotary_group(rot, [0], [x], [clean], pos)
    assert bool((clean[1, 64:128] == 0).all())
    x[2, 70], x[3, 130] = math.nan, math.inf
    S.norm_rotary_group(rot, [0], [x], [y], pos)
    torch.cuda.synchronize()
    assert torch.isnan(y[2, 64:128]).all() and torch.isnan(y[3, 128:192]).any()
    for r, c in ((2, slice(64, 128)), (3, slice(128, 192))):
        y[r, c] = clean[r, c]
    assert torch.equal(y, clean)
    S.norm_rotary_group(rot, [0], [x], [y], pos, eps=0.0)        # zero heads without eps: 0 / 0
    assert torch.isnan(y[1, 64:128]).all()
    S.close()


def test_graph_replays_and_no_tokens():
    rot = rotary(128, 128, "half", "none")
    S = binding.Slots(1, 1, [(8, 512), (8, 128)], "bf16", 64)
    x = [torch.randn(64, 512).bfloat16().cuda(), torch.randn(64, 128).bfloat16().cuda()]
    y = [torch.empty_like(v) for v in x]
    w = [torch.rand(128).bfloat16().cuda()] * 2
    pos = torch.arange(64, dtype=torch.int32).cuda()
    S.norm_rotary_group(rot, [0, 1], x, y, pos, w)
    torch.cuda.synchronize()
    eager = [v.clone() for v in y]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        S.norm_rotary_group(rot, [0, 1], x, y, pos, w)
    for _ in range(3):
        for v in y:
            v.fill_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(y, eager))
        S.norm_rotary_group(rot, [0, 1], x, y, pos, w, n_tokens=0)
        assert all(torch.equal(a, b) for a, b in zip(y, eager))
    S.close()


def test_refusals():
    rot = rotary(128, 128, "half", "none")
    S = binding.Slots(1, 1, [(8, 512), (8, 96)], "bf16", 64)
    x = torch.zeros(4, 512, dtype=torch.bfloat16, device="cuda")
    y, w = torch.empty_like(x), torch.ones(128, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    E = binding.LORA_ERR_INVALID_ARGUMENT

    def refused(status, *args, **kw):
        with pytest.raises(binding.LoraError) as e:
            binding.lora_norm_rotary_group(S.ctx, *args, **kw)
        assert e.value.status == status, e.value

    refused(E, rot, [0], [x], [y], pos, eps=-1.0)
    refused(E, rot, [0], [x], [y], pos, eps=math.nan)
    refused(E, rot, [0], [x], [y], pos, eps=1e300)
    refused(E, rot, [1], [x], [y], pos)                       # no whole heads
    refused(E, rot, [0, 0], [x, x], [y, y], pos)
    refused(E, rot, [0], [x], [y], pos, [y.view(-1)[:128]])   # y overlaps the weight
    refused(E, binding.Rotary(), [0], [x], [y], pos)
    refused(binding.LORA_ERR_BAD_MODULE, rot, [2], [x], [y], pos)
    refused(binding.LORA_ERR_TOO_MANY_TOKENS, rot, [0], [x], [y],
            torch.zeros(65, dtype=torch.int32, device="cuda"))
    T = binding.Slots(1, 1, [(8, 1024)], "bf16", 64)
    with pytest.raises(binding.LoraError):
        binding.lora_norm_rotary_group(T.ctx, rotary(1024, 64, "half", "none"), [0], [x], [y], pos)
    with pytest.raises(ValueError):
        S.norm_rotary_group(rot, [0], [x], [y], pos, [w.float()])
    with pytest.raises(ValueError):
        S.norm_rotary_group(rot, [0], [x], [y], pos, [w[:64]])
    with pytest.raises(ValueError):
        S.norm_rotary_group(rot, [0], [x], [y], pos, [w, w])
    T.close()
    S.close()
