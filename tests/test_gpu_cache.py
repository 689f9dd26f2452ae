"""The paged cache (lora_cache_store, lora_cache_load) on the GPU: what is read back, bit for
bit, against codes formed in 64 bits."""
import math

import pytest
import torch

from attend_util import coded, read_back
from gpu_util import log
from layer_util import TORCH
from lora_adapter_application_amd import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load_library()


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


def same(got, want):
    """Equal bits, where any NaN is as good as another."""
    got, want = got.cpu(), want.cpu()
    nan = torch.isnan(want)
    return torch.equal(torch.isnan(got), nan) and torch.equal(bits(got[~nan]), bits(want[~nan]))


def slot_lists(gen, pages, page, tokens, how):
    total = pages * page
    if how == "scattered":
        return torch.randperm(total, generator=gen)[:tokens]
    if how == "run":                          # one request from somewhere in a page on
        order = torch.randperm(pages, generator=gen)
        s = torch.arange(tokens) + 5
        return order[s // page] * page + s % page
    # ragged requests, each from its own place in a page, some padding between them
    out, order, at = [], torch.randperm(pages, generator=gen).tolist(), 0
    while sum(len(o) for o in out) < tokens:
        first = int(torch.randint(page, (1,), generator=gen))
        n = int(torch.randint(1, page + 9, (1,), generator=gen))
        need = -(-(first + n) // page)
        s = torch.arange(first, first + n)
        out.append(torch.tensor(order[at:at + need])[s // page] * page + s % page)
        out.append(torch.tensor([-1, -2 ** 31][:int(torch.randint(3, (1,), generator=gen))], dtype=torch.int64))
        at += need
    return torch.cat(out)[:tokens]


@pytest.mark.parametrize("dtype,kind,kv_heads,head_dim,page,tokens,how", [
    ("bf16", "native", 8, 128, 64, 1, "scattered"),
    ("bf16", "native", 1, 8, 32, 100, "scattered"),
    ("bf16", "native", 3, 80, 32, 333, "run"),
    ("bf16", "native", 8, 128, 64, 500, "ragged"),
    ("bf16", "native", 2, 256, 256, 500, "ragged"),
    ("bf16", "native", 5, 64, 32, 200, "ragged"),
    ("bf16", "fp8", 8, 128, 64, 1, "scattered"),
    ("bf16", "fp8", 8, 128, 64, 500, "ragged"),
    ("bf16", "fp8", 3, 80, 32, 333, "run"),
    ("bf16", "fp8", 2, 256, 128, 77, "scattered"),
    ("bf16", "fp8", 1, 24, 32, 64, "run"),
    ("bf16", "int8", 8, 128, 64, 500, "ragged"),
    ("bf16", "int8", 3, 96, 32, 333, "run"),
    ("bf16", "int8", 33, 64, 32, 130, "scattered"),
    ("bf16", "int8", 2, 200, 128, 77, "ragged"),
    ("fp32", "native", 4, 80, 32, 150, "ragged"),
    ("fp32", "native", 2, 256, 64, 150, "run"),
    ("fp32", "fp8", 4, 128, 32, 150, "ragged"),
    ("fp32", "int8", 4, 104, 32, 150, "ragged"),
    ("fp32", "int8", 1, 256, 64, 3, "scattered"),
])
@pytest.mark.parametrize("offset", [0, 1])
def test_read_back(dtype, kind, kv_heads, head_dim, page, tokens, how, offset):
    log(f"case cache {dtype} {kind} {kv_heads} {head_dim} {page} {tokens} {how} {offset}")
    gen = torch.Generator().manual_seed(head_dim + tokens)
    t, pages = TORCH[dtype], 2 * (tokens // page + 1) + tokens // 8 + 2
    S = binding.Slots(1, 1, [(64, 64)], dtype, max(tokens, 64))
    cache = S.cache(kv_heads, head_dim, pages, page, kind)
    slots = slot_lists(gen, pages, page, tokens, how)
    k, v = (torch.randn(tokens, kv_heads, head_dim, generator=gen).to(t) for _ in range(2))
    k[0, 0] = 0                                             # a head of zeros
    v[-1, -1] *= 1e30                                       # and far sizes
    k[-1, 0] *= 1e-35
    place = lambda x: torch.cat((torch.zeros(offset, dtype=t), x.reshape(-1))).cuda()[offset:].view(x.shape)  # noqa: E731
    S.cache_store(cache, place(k), place(v), slots.to(torch.int32).cuda())
    back = torch.full((offset + 2 * k.numel() + 64,), 7.0, dtype=t, device="cuda")
    n = k.numel()
    kb, vb = back[offset:offset + n].view(k.shape), back[offset + n:offset + 2 * n].view(k.shape)
    S.cache_load(cache, slots.to(torch.int32).cuda(), kb, vb)
    torch.cuda.synchronize()
    live = slots >= 0
    assert same(kb[live.cuda()], read_back(k, kind)[live])
    assert same(vb[live.cuda()], read_back(v, kind)[live])
    assert bool((kb[~live.cuda()] == 7).all()) and bool((vb[~live.cuda()] == 7).all())
    assert bool((back[:offset] == 7).all()) and bool((back[offset + 2 * n:] == 7).all())
    # every other slot is still zero
    rest = torch.ones(pages * page, dtype=torch.bool)
    rest[slots[live]] = False
    other = rest.nonzero().view(-1).to(torch.int32).cuda()
    for part in other.split(S.max_tokens):
        a = torch.full((part.numel(), kv_heads, head_dim), 7.0, dtype=t, device="cuda")
        b = a.clone()
        S.cache_load(cache, part, a, b)
        assert bool((a == 0).all()) and bool((b == 0).all())
    # stored over, and what was beside it stays
    S.cache_store(cache, place(v)[:1], place(k)[:1], slots[:1].to(torch.int32).cuda())
    S.cache_load(cache, slots.to(torch.int32).cuda(), kb, vb)
    if live[0]:
        assert same(kb[:1], read_back(v, kind)[:1]) and same(vb[:1], read_back(k, kind)[:1])
    assert same(kb[1:][live[1:].cuda()], read_back(k, kind)[1:][live[1:]])
    assert S.flags() == 0
    cache.close()
    S.close()


@pytest.mark.parametrize("kind", ["fp8", "int8"])
def test_ties_and_borders(kind):
    """Heads whose quotients are ties, of every pair of a value and a largest value with 8 significant
    bits; the smallest codes of fp8."""
    top = torch.arange(128, 256, dtype=torch.float32)
    rows = []
    for sign in (1.0, -1.0):
        for shift in range(19):
            x = torch.arange(128, 256, dtype=torch.float32)[None, :] * 2.0 ** -shift * sign
            rows.append(torch.where(x.abs() > top[:, None], torch.zeros(()), x).repeat(1, 2))
    x = torch.cat(rows)
    big = top.repeat(len(rows))
    x[:, -1] = big                                          # the largest value of the head
    x = x.bfloat16()[:, None, :].contiguous()               # [tokens][1][256]
    levels = coded(x, kind)[0]
    assert len(levels.unique()) == (253 if kind == "fp8" else 255)
    S = binding.Slots(1, 1, [(64, 64)], "bf16", x.shape[0])
    cache = S.cache(1, 256, -(-x.shape[0] // 64), 64, kind)
    slots = torch.arange(x.shape[0], dtype=torch.int32).cuda()
    a, b = torch.empty_like(x).cuda(), torch.empty_like(x).cuda()
    S.cache_store(cache, x.cuda(), (-x).cuda(), slots)
    S.cache_load(cache, slots, a, b)
    assert torch.equal(a.cpu(), read_back(x, kind)) and torch.equal(b.cpu(), read_back(-x, kind))
    S.close()


@pytest.mark.parametrize("kind", ["native", "fp8", "int8"])
def test_infinities_and_nans(kind):
    x = torch.randn(40, 2, 64).bfloat16()
    x[3, 0, 5], x[3, 1, 6], x[20, 1, 63], x[21, 0, 0] = math.nan, math.inf, -math.inf, -math.nan
    S = binding.Slots(1, 1, [(64, 64)], "bf16", 64)
    cache = S.cache(2, 64, 2, 32, kind)
    slots = torch.arange(40, dtype=torch.int32).cuda()
    a, b = torch.empty_like(x).cuda(), torch.empty_like(x).cuda()
    S.cache_store(cache, x.cuda(), x.cuda(), slots)
    S.cache_load(cache, slots, a, b)
    want = read_back(x, kind)
    if kind != "native":
        assert all(torch.isnan(want[t, h]).all() for t, h in ((3, 0), (3, 1), (20, 1), (21, 0)))
    assert same(a, want) and same(b, want)
    S.close()


def test_slots_past_the_cache_and_refusals():
    S = binding.Slots(1, 1, [(64, 64)], "bf16", 64)
    cache = S.cache(2, 64, 2, 32)
    k = torch.randn(6, 2, 64).bfloat16().cuda()
    v = -k
    slots = torch.tensor([0, 64, 63, 2 ** 31 - 1, -1, 65], dtype=torch.int32).cuda()
    S.cache_store(cache, k, v, slots)
    assert S.flags() == binding.LORA_FLAG_CACHE_SLOT
    a, b = torch.full_like(k, 7.0), torch.full_like(k, 7.0)
    S.cache_load(cache, slots, a, b)
    assert S.flags() == binding.LORA_FLAG_CACHE_SLOT
    live = [0, 2]
    assert torch.equal(a[live], k[live]) and torch.equal(b[live], v[live])
    assert bool((a[[1, 3, 4, 5]] == 7).all()) and bool((b[[1, 3, 4, 5]] == 7).all())
    S.cache_store(cache, k, v, slots, n_tokens=0)
    E = binding.LORA_ERR_INVALID_ARGUMENT

    def refused(status, fn, *args, **kw):
        with pytest.raises(binding.LoraError) as e:
            fn(*args, **kw)
        assert e.value.status == status, e.value

    for kw in (dict(kv_heads=0), dict(kv_heads=1025), dict(head_dim=0), dict(head_dim=12), dict(head_dim=264),
               dict(page_size=16), dict(page_size=48), dict(page_size=0), dict(page_size=-32), dict(pages=0),
               dict(pages=2 ** 26), dict(kind=3), dict(kind=-1)):
        refused(E, binding.lora_cache_create, S.ctx,
                **{**dict(kv_heads=2, head_dim=64, pages=2, page_size=32), **kw})
    refused(binding.LORA_ERR_OUT_OF_MEMORY, S.cache, 1024, 256, 2 ** 25, 32)
    assert S.flags() == 0
    with pytest.raises(ValueError):
        S.cache(2, 64, 2, 32, "int4")
    refused(binding.LORA_ERR_TOO_MANY_TOKENS, binding.lora_cache_store, S.ctx, cache.handle, k, v,
            torch.zeros(65, dtype=torch.int32, device="cuda"))
    refused(E, binding.lora_cache_store, S.ctx, S.ctx, k, v, slots)
    refused(E, binding.lora_cache_load, S.ctx, cache.handle, slots, a, a)
    refused(E, binding.lora_cache_store, S.ctx, cache.handle, k, v, slots, n_tokens=-1)
    with pytest.raises(ValueError):
        S.cache_store(cache, k.float(), v, slots)
    with pytest.raises(ValueError):
        S.cache_store(cache, k[:5], v, slots)
    with pytest.raises(ValueError):
        S.cache_store(cache, k, v, slots.long())
    s = torch.cuda.Stream()
    with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=s):
        S.cache_store(cache, k, v, slots)
        refused(E, S.cache, 2, 64, 2, 32)
        refused(E, binding.lora_cache_destroy, S.ctx, cache.handle)
    handle = cache.handle
    cache.close()
    refused(E, binding.lora_cache_destroy, S.ctx, handle)
    refused(E, binding.lora_cache_store, S.ctx, handle, k, v, slots)
    S.close()


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes: its last pages are their own."""
    S = binding.Slots(1, 1, [(64, 64)], "bf16", 64)
    pages = 2 ** 33 // (32 * 8 * 128 * 2 * 2) + 3
    cache = S.cache(8, 128, pages, 32)
    k, v = torch.randn(64, 8, 128).bfloat16().cuda(), torch.randn(64, 8, 128).bfloat16().cuda()
    slots = (torch.arange(64) * (pages // 64) * 32 + torch.arange(64) % 32).to(torch.int32).cuda()
    slots[63] = pages * 32 - 1
    S.cache_store(cache, k, v, slots)
    a, b = torch.empty_like(k), torch.empty_like(v)
    S.cache_load(cache, slots, a, b)
    assert torch.equal(a, k) and torch.equal(b, v)
    # attention over them
    batch = binding.AttendBatch(torch.tensor([32 * 64], dtype=torch.int32).cuda(),
                                (slots // 32)[None].contiguous())
    one = torch.full((1, 8 * 128), 0.0, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(one)
    S.attend_prepare(cache, 8, batch)
    S.attend(cache, one, y)                    # q = 0: the mean of all values, zeros but for the 64
    want = v.double().sum(0).view(1, -1) / 2048
    assert bool(((y.double() - want).abs() <= 2.0 ** -7 * v.double().abs().sum(0).view(1, -1) / 2048).all())
    cache.close()
    S.close()
