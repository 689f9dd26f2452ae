"""The 4-bit base product (lora_base_load, lora_base, lora_base_group) on the GPU against
its formula in 64 bits."""
import pytest
import torch

from gpu_util import log
from lora_adapter_application_amd import binding
from layer_util import (HALF_STEP, TORCH, base_sum, check_within, groups_of, guarded,
                        integer_weight, random_weight)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load_library()


def make(dtype, tokens, d_in, outs, group, zero, bias, add, seed, integers=False):
    gen = torch.Generator().manual_seed(seed)
    draw = integer_weight if integers else random_weight
    w = [draw(gen, n, d_in, group, zero) for n in outs]
    if integers:
        val = lambda *s: torch.randint(-4, 5, s, generator=gen).to(TORCH[dtype])  # noqa: E731
    else:
        val = lambda *s: torch.randn(*s, generator=gen).to(TORCH[dtype])  # noqa: E731
    x = [val(tokens, d_in) for _ in outs]
    b = [val(n) if bias else None for n in outs]
    a = [val(tokens, n) if add else None for n in outs]
    return w, x, b, a


def load_all(S, w, group, bias):
    for i, ((q, s, z), b) in enumerate(zip(w, bias)):
        S.load_base(i, q.cuda(), s.cuda(), None if z is None else z.cuda(), group,
                    None if b is None else b.cuda())


def dev(ts):
    return [None if t is None else t.cuda() for t in ts]


EXACT = [
    # dtype, tokens, d_in, outs, group, zero, bias, add
    ("bf16", 1, 8, [8], 0, True, False, False),
    ("bf16", 1, 4096, [256, 24], 128, True, True, False),
    ("bf16", 2, 136, [40], 32, True, False, True),
    ("bf16", 15, 1000, [264, 8], 64, False, True, True),
    ("bf16", 16, 128, [16], 128, True, False, False),
    ("bf16", 17, 256, [72], 256, True, True, False),
    ("bf16", 32, 1160, [88], 0, True, False, True),
    ("bf16", 33, 1160, [88], 128, False, False, False),
    ("bf16", 64, 640, [520], 32, True, True, True),
    ("bf16", 65, 2056, [136], 128, True, False, False),
    ("bf16", 130, 512, [1032, 264], 64, True, True, False),
    ("bf16", 300, 392, [776], 128, True, True, True),
    ("bf16", 1025, 264, [280], 384, True, False, False),
    ("fp32", 1, 8, [8], 32, True, True, True),
    ("fp32", 3, 1000, [264], 32, True, False, False),
    ("fp32", 37, 1032, [40, 8], 64, False, True, False),
    ("fp32", 129, 640, [152], 128, True, False, True),
    ("fp32", 300, 264, [280], 0, True, True, True),
]


@pytest.mark.parametrize("dtype,tokens,d_in,outs,group,zero,bias,add", EXACT)
def test_integers_are_exact(dtype, tokens, d_in, outs, group, zero, bias, add):
    """Integer inputs and power-of-two scales: every 32-bit sum is exact, so the result is
    the formula's, rounded once, bit for bit, and no memory around the rows is touched."""
    log("case", dtype, tokens, d_in, outs, group)
    w, x, b, a = make(dtype, tokens, d_in, outs, group, zero, bias, add, 17 + tokens + d_in, True)
    with binding.Slots(1, 1, [(d_in, n) for n in outs], dtype, tokens) as S:
        load_all(S, w, group, b)
        ys = [guarded(tokens, n, TORCH[dtype]) for n in outs]
        S.base_group(list(range(len(outs))), dev(x), [y for y, _ in ys], dev(a))
        torch.cuda.synchronize()
        for i, (y, intact) in enumerate(ys):
            want, _ = base_sum(x[i], w[i], d_in, group)
            # the largest partial sum, in units of the smallest scale 1/4, fits 24 bits
            assert 4 * x[i].double().abs().sum(1).max() * 31 < 2 ** 24
            for extra in (b[i], a[i]):
                if extra is not None:
                    want = want + extra.double()
            assert torch.equal(y.cpu(), want.float().to(TORCH[dtype])), (i, dtype, tokens)
            intact()


# One case for each way the library multiplies (by tokens, columns and alignment), each
# with one, two and four groups a block of 128 inputs, with and without zero points.
WAYS = [
    # dtype, tokens, d_out: what takes it
    ("bf16", 3, 8200),       # few tokens, four column blocks a workgroup
    ("bf16", 16, 8200),
    ("bf16", 129, 2056),     # split, 32 x 64
    ("bf16", 257, 2056),     # split, 32 x 128
    ("bf16", 513, 2056),     # split, 64 x 128
    ("bf16", 1025, 2056),    # split, 64 x 256
    ("bf16", 2049, 2056),    # split, 64 x 384
    ("bf16", 2689, 2056),    # tiles
    ("fp32", 5, 8200),       # few tokens, four column blocks a workgroup
    ("fp32", 17, 8200),      # tiles, K halved
    ("fp32", 129, 8200),     # tiles
]


@pytest.mark.parametrize("group,zero", [(0, True), (128, False), (64, True), (64, False),
                                        (32, True), (32, False)])
@pytest.mark.parametrize("dtype,tokens,d_out", WAYS)
def test_every_way_is_exact_on_integers(dtype, tokens, d_out, group, zero):
    d_in = 520 if group else 1000
    log("case", dtype, tokens, d_out, group, zero)
    w, x, b, a = make(dtype, tokens, d_in, [d_out], group, zero, True, True, tokens + group, True)
    with binding.Slots(1, 1, [(d_in, d_out)], dtype, tokens) as S:
        load_all(S, w, group, b)
        y, intact = guarded(tokens, d_out, TORCH[dtype])
        S.base(x[0].cuda(), y, 0, a[0].cuda())
        # the 64-bit sums on the device, where they are quick
        v = torch.stack((w[0][0] & 15, w[0][0] >> 4), 2).view(d_out, d_in).double()
        of = torch.arange(d_in) // (group or d_in)
        z = 8.0 if w[0][2] is None else w[0][2].double()[:, of]
        full = ((v - z) * w[0][1].double()[:, of]).cuda()
        want = x[0].cuda().double() @ full.t().contiguous() + b[0].cuda().double() + a[0].cuda().double()
        assert torch.equal(y, want.float().to(TORCH[dtype]))
        intact()


@pytest.mark.parametrize("tokens", [20, 64, 65, 200])
def test_unaligned_rows_are_exact_on_integers(tokens):
    for group, zero, d_in in ((128, True, 520), (64, False, 392), (32, True, 264)):
        w, x, _, _ = make("bf16", tokens, d_in, [264], group, zero, False, False, tokens, True)
        with binding.Slots(1, 1, [(d_in, 264)], "bf16", tokens) as S:
            load_all(S, w, group, [None])
            xs, _ = guarded(tokens, d_in, torch.bfloat16, 1)
            xs.copy_(x[0])
            y, intact = guarded(tokens, 264, torch.bfloat16, 5)
            S.base(xs, y, 0)
            want, _ = base_sum(x[0], w[0], d_in, group)
            assert torch.equal(y.cpu(), want.float().bfloat16()), (group, zero)
            intact()


@pytest.mark.parametrize("tokens,n", [(40, 2056), (600, 2056), (2100, 2056), (2700, 2056)])
def test_nonfinite_rows_in_large_batches(tokens, n):
    """A NaN row, an infinity at the end of a row, and a batch of NaN: quick, and the rows
    beside them keep their bits."""
    d_in = 520
    w, x, _, a = make("bf16", tokens, d_in, [n], 128, True, False, True, 7, True)
    with binding.Slots(1, 1, [(d_in, n)], "bf16", tokens) as S:
        load_all(S, w, 128, [None])
        clean = torch.empty(tokens, n, dtype=torch.bfloat16, device="cuda")
        S.base(x[0].cuda(), clean, 0, a[0].cuda())
        bad = x[0].clone()
        bad[3, 0] = float("nan")
        bad[tokens - 1, d_in - 1] = float("inf")
        y = a[0].cuda()
        S.base(bad.cuda(), y, 0, y)
        keep = torch.ones(tokens, dtype=torch.bool)
        keep[3] = keep[tokens - 1] = False
        assert torch.equal(y[keep.cuda()], clean[keep.cuda()])
        assert bool(y[3].isnan().all())
        d = (w[0][0][:, -1] >> 4).double() - w[0][2][:, -1].double()    # the last input's weights
        last = y[tokens - 1].cpu()
        assert torch.equal(last.isnan(), d == 0)
        assert bool((last[d > 0] == float("inf")).all()) and bool((last[d < 0] == float("-inf")).all())
        bad[:] = float("nan")
        S.base(bad.cuda(), y, 0)
        assert bool(y.isnan().all())


def test_scales_of_a_bf16_pool():
    """16 significant bits of a float32 scale, to nearest; the largest stays finite, and an
    infinite or NaN scale acts as one."""
    s = torch.tensor([1 + 2.0 ** -15, 1 + 2.0 ** -16 + 2.0 ** -20, torch.finfo(torch.float32).max,
                      float("inf"), float("nan"), -0.75, 0.0, 2.0 ** -100]).view(8, 1)
    q = torch.full((8, 8), 0x99, dtype=torch.uint8)            # 9 - 8 = 1
    x = torch.zeros(1, 16).bfloat16()
    x[0, 0] = 1.0
    with binding.Slots(1, 1, [(16, 8)], "bf16", 1) as S:
        S.load_base(0, q.cuda(), s.cuda(), None, 0)
        add = torch.full((1, 8), -1.0).bfloat16().cuda()       # 1 + 2^-15 - 1 needs the kept bits
        y = torch.empty(1, 8, dtype=torch.bfloat16, device="cuda")
        S.base(x.cuda(), y, 0, add)
        y = y.cpu()[0]
    assert y[0] == 2.0 ** -15 and y[1] == 2.0 ** -15
    assert y[2].double() >= 3.3e38 or y[2] == float("inf")     # bf16 of the largest float32
    assert y[3] == float("inf") or y[3].isnan()                # inf * 0 of the other inputs
    assert y[4].isnan() and y[5] == -1.75 and y[6] == -1.0 and y[7] == -1.0


CLOSE = [
    ("bf16", 1, 4096, [4096], 128, True, False, False),
    ("bf16", 5, 11008, [264], 128, True, True, True),
    ("bf16", 24, 5120, [1024, 72], 64, False, False, True),
    ("bf16", 48, 2048, [520], 32, True, True, False),
    ("bf16", 100, 1000, [1032], 0, True, False, False),
    ("bf16", 520, 4096, [392], 128, True, False, True),
    ("fp32", 1, 4096, [520], 128, True, True, False),
    ("fp32", 20, 1000, [264], 32, True, False, True),
    ("fp32", 150, 2056, [136], 64, True, True, True),
]


@pytest.mark.parametrize("dtype,tokens,d_in,outs,group,zero,bias,add", CLOSE)
def test_random_values_within_the_derived_bound(dtype, tokens, d_in, outs, group, zero, bias, add):
    log("case", dtype, tokens, d_in, outs, group)
    w, x, b, a = make(dtype, tokens, d_in, outs, group, zero, bias, add, 91 + tokens + d_in)
    with binding.Slots(1, 1, [(d_in, n) for n in outs], dtype, tokens) as S:
        load_all(S, w, group, b)
        y = [torch.empty(tokens, n, dtype=TORCH[dtype], device="cuda") for n in outs]
        S.base_group(list(range(len(outs))), dev(x), y, dev(a))
        torch.cuda.synchronize()
        for i, n in enumerate(outs):
            want, bound = base_sum(x[i], w[i], d_in, group)
            for extra in (b[i], a[i]):
                if extra is not None:
                    want = want + extra.double()
                    bound = bound + 2.0 ** -24 * (want.abs() + extra.double().abs())
            bound = bound + HALF_STEP[TORCH[dtype]] * (want.abs() + bound)
            worst = check_within(y[i], want, bound, f"module {i}")
            # the bound is a worst case: independent roundings stay far inside it
            rel = ((y[i].cpu().double() - want).norm() / want.norm()).item()
            log("  worst error / bound %.3f, relative 2-norm %.2e" % (worst, rel))
            assert rel <= HALF_STEP[TORCH[dtype]] * (1 if dtype == "bf16" else 16)


@pytest.mark.parametrize("dtype,tokens", [("bf16", 1), ("bf16", 21), ("bf16", 200), ("fp32", 1),
                                          ("fp32", 40)])
def test_infinities_and_nans_give_what_the_formula_gives(dtype, tokens):
    d_in, n = 264, 40
    w, x, _, _ = make(dtype, tokens, d_in, [n], 64, True, False, False, 5)
    x = x[0]
    big = torch.finfo(TORCH[dtype]).max
    x[0, 3] = float("inf")
    if tokens > 1:
        x[1, 250] = float("-inf")
        x[2, 7] = float("nan")
        x[3, 9], x[3, 200] = float("inf"), float("inf")
        x[4, :] = 0
        x[4, 100] = big / 8          # 31 x overflows, (q - zero) * scale * x does not
        x[tokens - 1, 0] = -big / 8
    with binding.Slots(1, 1, [(d_in, n)], dtype, tokens) as S:
        load_all(S, w, 64, [None])
        y = torch.empty(tokens, n, dtype=TORCH[dtype], device="cuda")
        S.base(x.cuda(), y, 0)
        y = y.cpu()
    q, s, z = w[0]
    v = torch.stack((q & 15, q >> 4), 2).view(n, d_in).double()
    of = torch.arange(d_in) // 64
    full = (v - z.double()[:, of]) * s.double()[:, of]
    want = (x.double()[:, None, :] * full[None]).sum(2)
    assert torch.equal(y.isnan(), want.isnan())
    assert torch.equal(y.isinf(), want.isinf())
    inf = want.isinf()
    assert torch.equal(y.double()[inf], want[inf])
    fine = torch.isfinite(want)
    m = (x.double().abs().nan_to_num(0, 0)[:, None, :] * full.abs()[None]).sum(2)
    bound = HALF_STEP[TORCH[dtype]] * want[fine].abs() + 2 * 264 * 2.0 ** -24 * m[fine] * 64
    assert bool(((y.double()[fine] - want[fine]).abs() <= bound).all())


@pytest.mark.parametrize("dtype,tokens", [("bf16", 3), ("bf16", 70), ("bf16", 300), ("fp32", 5)])
def test_any_alignment_of_the_rows(dtype, tokens):
    """x, add and y off a 16-byte boundary: every alignment inside the derived bound.  (The
    kernels that alignment chooses between add the same products in other orders, so their
    32-bit sums may differ; each is within steps * 2^-24 * m of the exact sum, base_sum.)"""
    d_in, n = 520, 72
    w, x, b, a = make(dtype, tokens, d_in, [n], 128, True, True, True, 8)
    want, bound = base_sum(x[0], w[0], d_in, 128)
    for extra in (b[0], a[0]):
        want = want + extra.double()
        bound = bound + 2.0 ** -24 * (want.abs() + extra.double().abs())
    bound = bound + HALF_STEP[TORCH[dtype]] * (want.abs() + bound)
    with binding.Slots(1, 1, [(d_in, n)], dtype, tokens) as S:
        load_all(S, w, 128, b)
        for off in (0, 1, 2, 3, 8):
            xs, _ = guarded(tokens, d_in, TORCH[dtype], off)
            as_, _ = guarded(tokens, n, TORCH[dtype], off)
            ys, intact = guarded(tokens, n, TORCH[dtype], off)
            xs.copy_(x[0])
            as_.copy_(a[0])
            S.base(xs, ys, 0, as_)
            check_within(ys, want, bound, f"offset {off}")
            intact()


def test_group_equals_singles_and_add_in_place():
    tokens, d_in, outs = 19, 640, [264, 40, 8, 136]
    groups = [32, 128, 64, 0]                 # three kinds of scale storage in one call
    gen = torch.Generator().manual_seed(3)
    w = [random_weight(gen, n, d_in, g, True) for n, g in zip(outs, groups)]
    x = torch.randn(tokens, d_in, generator=gen).bfloat16().cuda()
    r = [torch.randn(tokens, n, generator=gen).bfloat16().cuda() for n in outs]
    with binding.Slots(1, 1, [(d_in, n) for n in outs], "bf16", tokens) as S:
        for i, (q, s, z) in enumerate(w):
            S.load_base(i, q.cuda(), s.cuda(), z.cuda(), groups[i])
        one = [torch.empty_like(t) for t in r]
        for i in range(4):
            S.base(x, one[i], i, r[i])
        order = [2, 0, 3, 1, 0]               # a module twice, with its own y
        many = [r[i].clone() for i in order]
        S.base_group(order, [x] * 5, many, many)        # add is y itself
        plain = [torch.empty_like(t) for t in r]
        S.base_group([0, 1, 2, 3], [x] * 4, plain, [r[0], None, r[2], None])
        for i, y in zip(order, many):
            assert torch.equal(y, one[i])
        assert torch.equal(plain[0], one[0]) and torch.equal(plain[2], one[2])
        # a batch of fewer tokens leaves the rows behind it
        y = torch.full((tokens, outs[0]), 3.0, dtype=torch.bfloat16, device="cuda")
        S.base(x, y, 0, r[0], n_tokens=5)
        want, bound = base_sum(x[:5].cpu(), w[0], d_in, groups[0])
        want = want + r[0][:5].cpu().double()
        check_within(y[:5], want, bound + 2.0 ** -7 * (want.abs() + bound), "five tokens")
        assert bool((y[5:] == 3).all())
        S.base(x, y, 0, n_tokens=0)
        assert bool((y[5:] == 3).all())


@pytest.mark.parametrize("source", ["pinned", "device", "staged"])
def test_sources_of_a_load(source):
    """Pinned host memory (through the stage in many pieces: a rank-1 pool holds a small
    one), device memory, and device memory off a 4-byte boundary give the same weights."""
    d_in, n, tokens = 2056, 1032, 3
    w, x, b, _ = make("bf16", tokens, d_in, [n], 32, True, True, False, 12)
    q, s, z = w[0]
    keep = []

    def place(t):
        if source == "pinned":
            t = t.pin_memory()
        elif source == "device":
            t = t.cuda()
        else:
            whole = torch.empty(t.numel() * t.element_size() + 64, dtype=torch.uint8, device="cuda")
            off = 2 if t.dtype == torch.bfloat16 else 4 if t.dtype == torch.float32 else 1
            v = whole[off:off + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
            v.copy_(t)
            t = v
        keep.append(t)
        return t
    with binding.Slots(1, 1, [(d_in, n)], "bf16", tokens) as S:
        S.load_base(0, place(q), place(s), place(z), 32, place(b[0]))
        y = torch.empty(tokens, n, dtype=torch.bfloat16, device="cuda")
        S.base(x[0].cuda(), y, 0)
        want, bound = base_sum(x[0], w[0], d_in, 32)
        want = want + b[0].double()
        check_within(y, want, bound + 2.0 ** -8 * (want.abs() + bound) + 2.0 ** -22, source)


def test_reload_waits_for_products_in_flight_and_products_for_the_load():
    """Loads over a weight in use, without host synchronisation: each product sees the
    weight of its own time, also one that runs on another stream."""
    tokens, d_in, n = 700, 2048, 1024
    gen = torch.Generator().manual_seed(1)
    x = torch.randint(-3, 4, (tokens, d_in), generator=gen).bfloat16().cuda()
    ws = [integer_weight(gen, n, d_in, g, True) for g in (128, 32, 64)]
    ds = [[t.cuda() for t in w] for w in ws]
    want = [base_sum(x.cpu(), w, d_in, g)[0].float().bfloat16() for w, g in zip(ws, (128, 32, 64))]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with binding.Slots(1, 1, [(d_in, n)], "bf16", tokens) as S:
        ys = [torch.empty(tokens, n, dtype=torch.bfloat16, device="cuda") for _ in range(9)]
        torch.cuda.synchronize()
        for i, y in enumerate(ys):
            q, s, z = ds[i % 3]
            # the C call, which does not wait for the host's streams
            binding._check(binding.load_library().lora_base_load(
                S.ctx, 0, q.data_ptr(), s.data_ptr(), z.data_ptr(), (128, 32, 64)[i % 3], None), S.ctx)
            S.base(x, y, 0, stream=side if i % 2 else None)
        torch.cuda.synchronize()
        for i, y in enumerate(ys):
            assert torch.equal(y.cpu(), want[i % 3]), i


def test_captured_product_replays_with_reloaded_weights():
    tokens, d_in, n = 40, 512, 264
    gen = torch.Generator().manual_seed(2)
    ws = [integer_weight(gen, n, d_in, 128, True) for _ in range(2)]
    xs = [torch.randint(-3, 4, (tokens, d_in), generator=gen).bfloat16().cuda() for _ in range(3)]
    x = xs[0].clone()
    with binding.Slots(1, 1, [(d_in, n)], "bf16", tokens) as S:
        load = lambda w: S.load_base(0, w[0].cuda(), w[1].cuda(), w[2].cuda(), 128)  # noqa: E731
        load(ws[0])
        y = torch.zeros(tokens, n, dtype=torch.bfloat16, device="cuda")
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            s.wait_stream(torch.cuda.default_stream())
        g = torch.cuda.CUDAGraph()
        # a load is pending: the first captured launch refuses
        with pytest.raises(binding.LoraError) as e:
            with torch.cuda.graph(g, stream=s):
                S.base(x, y, 0)
        assert "lora_sync_loads" in str(e.value)
        S.sync_loads()
        pinned = [t.pin_memory() for t in ws[1]]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            S.base(x, y, 0)
            with pytest.raises(binding.LoraError):
                # the C call alone: the binding would wait for the capturing stream
                binding._check(binding.load_library().lora_base_load(
                    S.ctx, 0, *[t.data_ptr() for t in pinned], 128, None), S.ctx)
        torch.cuda.synchronize()
        for w in (ws[0], ws[1], ws[0]):
            load(w)
            S.sync_loads()
            for xi in xs:
                x.copy_(xi)
                torch.cuda.synchronize()
                g.replay()
                torch.cuda.synchronize()
                eager = torch.empty_like(y)
                S.base(x, eager, 0)
                want = base_sum(xi.cpu(), w, d_in, 128)[0].float().bfloat16()
                assert torch.equal(y.cpu(), want) and torch.equal(eager.cpu(), want)


def test_refusals():
    """Every refused call leaves y as it was."""
    gen = torch.Generator().manual_seed(4)
    w = random_weight(gen, 64, 256, 128, True)
    q, s, z = (t.cuda() for t in w)
    x = torch.randn(8, 256, generator=gen).bfloat16().cuda()
    y = torch.full((8, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    E = binding
    with binding.Slots(1, 1, [(256, 64), (256, 64)], "bf16", 8) as S:
        lib, ctx = binding.load_library(), S.ctx

        def refused(want, call, text=""):
            with pytest.raises(binding.LoraError) as e:
                call()
            assert e.value.status == want and text in str(e.value), str(e.value)

        refused(E.LORA_ERR_INVALID_ARGUMENT, lambda: S.base(x, y, 0), "no base weight")
        refused(E.LORA_ERR_BAD_MODULE, lambda: binding.lora_base_load(ctx, 2, q, s, z, 128))
        refused(E.LORA_ERR_BAD_MODULE, lambda: binding.lora_base(ctx, x, y, -1))
        for g in (-1, 16, 48, 96, 200):
            refused(E.LORA_ERR_INVALID_ARGUMENT, lambda: binding.lora_base_load(ctx, 0, q, s, z, g),
                    "group_size")
        refused(E.LORA_ERR_INVALID_ARGUMENT, lambda: binding.lora_base_load(ctx, 0, None, s, z, 128))
        refused(E.LORA_ERR_INVALID_ARGUMENT, lambda: binding.lora_base_load(ctx, 0, q, None, z, 128))
        refused(E.LORA_ERR_HOST_NOT_PINNED,
                lambda: binding.lora_base_load(ctx, 0, w[0], s, z, 128))
        S.load_base(0, q, s, z, 128)
        refused(E.LORA_ERR_INVALID_ARGUMENT, lambda: binding.lora_base(ctx, None, y, 0, n_tokens=8))
        refused(E.LORA_ERR_INVALID_ARGUMENT, lambda: binding.lora_base(ctx, x, None, 0))
        refused(E.LORA_ERR_INVALID_ARGUMENT, lambda: binding.lora_base(ctx, x, y, 0, n_tokens=-1))
        refused(E.LORA_ERR_TOO_MANY_TOKENS, lambda: binding.lora_base(ctx, x, y, 0, n_tokens=9))
        refused(E.LORA_ERR_INVALID_ARGUMENT, lambda: S.base_group([0, 1], [x, x], [y, y.clone()]),
                "no base weight")
        S.load_base(1, q, s, z, 128)
        refused(E.LORA_ERR_INVALID_ARGUMENT, lambda: S.base_group([0, 1], [x, x], [y, y]))
        refused(E.LORA_ERR_INVALID_ARGUMENT,
                lambda: binding._check(lib.lora_base_group(ctx, 0, None, None, None, None, 1, None), ctx))
        wide = torch.full((17, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        refused(E.LORA_ERR_INVALID_ARGUMENT,
                lambda: S.base_group([0, 1], [x, x], [wide[:8], wide[7:15]]), "overlaps")
        refused(E.LORA_ERR_INVALID_ARGUMENT, lambda: S.base(x, wide[:8], 0, wide[1:9]), "overlaps")
        refused(E.LORA_ERR_INVALID_ARGUMENT,
                lambda: S.base_group([0, 1], [x, x], [wide[:8], y], [None, wide[:8]]), "overlaps")
        # rows of y inside x
        flat = torch.zeros(8 * 256 + 512, dtype=torch.bfloat16, device="cuda")
        refused(E.LORA_ERR_INVALID_ARGUMENT,
                lambda: S.base(flat[:2048].view(8, 256), flat[2040:2040 + 512].view(8, 64), 0), "overlaps")
        with pytest.raises(ValueError):
            S.base(x.float(), y, 0)
        with pytest.raises(ValueError):
            S.base(x, y[:4], 0)
        with pytest.raises(ValueError):
            S.load_base(0, q[:, :100].contiguous(), s, z, 128)
        with pytest.raises(ValueError):
            S.load_base(0, q, s.double(), z, 128)
        assert lib.lora_base_group(None, 1, None, None, None, None, 1, None) == E.LORA_ERR_INVALID_ARGUMENT
        torch.cuda.synchronize()
        assert bool((y == 5).all()) and bool((wide == 5).all())
        S.base(x, y, 0)
        want, bound = base_sum(x.cpu(), w, 256, 128)
        check_within(y, want, bound + 2.0 ** -8 * (want.abs() + bound), "after refusals")


def test_same_bits_on_every_run_and_on_two_streams():
    tokens, d_in, n = 65, 4096, 520
    w, x, _, _ = make("bf16", tokens, d_in, [n], 128, True, False, False, 6)
    with binding.Slots(1, 1, [(d_in, n)], "bf16", tokens) as S:
        load_all(S, w, 128, [None])
        xd = x[0].cuda()
        y0 = torch.empty(tokens, n, dtype=torch.bfloat16, device="cuda")
        S.base(xd, y0, 0)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        ys = [torch.empty_like(y0) for _ in range(8)]
        torch.cuda.synchronize()
        for i, y in enumerate(ys):
            S.base(xd, y, 0, stream=streams[i % 2])
        torch.cuda.synchronize()
        assert all(torch.equal(y, y0) for y in ys)


def test_group_counts():
    assert groups_of(1000, 32) == 32 and groups_of(1000, 0) == 1
