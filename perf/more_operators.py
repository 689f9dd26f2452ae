"""Cases and plain forms of the operators between a layer's projections: norms and positions of
queries and keys, the paged cache of keys and values, and attention over it.

``norm``    an RMS norm of each head of one or more projections and the rotary turn of the
            normed head, in one pass (``lora_norm_rotary_group``)
``cache``   a batch's keys and values written into pages, in the ctx's type or in 8 bits, and
            read back (``lora_cache_store``, ``lora_cache_load``)
``attend``  attention of a batch's new tokens over their requests' pages and, for the requests
            of an adapter that share a prefix, over the prefix's pages, which are read once
            for all of them (``lora_attend_prepare``, ``lora_attend``)

In 8 bits a head of a token is held as codes and one float32 scale: fp8 (e4m3) codes of
x / scale with scale = max|x| / 448, int8 codes with scale = max|x| / 127, each rounded to
the nearest, ties to even.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_TOP = {"fp8": 448.0, "int8": 127.0}


def listed():
    qwen = {"dtype": "bf16", "heads": 64, "kv_heads": 8, "head_dim": 128}
    llama = {"dtype": "bf16", "heads": 32, "kv_heads": 32, "head_dim": 128}
    return [
        # q and k of one request's token in a Qwen-32B layer
        {"name": "norm 1 token", "op": "norm", "dtype": "bf16", "tokens": 1, "heads": "64+8",
         "head_dim": 128, "rotary_dim": 128, "layout": "half", "scaling": "none", "span": 2048},
        # a decode batch of the same layer far into long contexts
        {"name": "norm 512 tokens", "op": "norm", "dtype": "bf16", "tokens": 512, "heads": "64+8",
         "head_dim": 128, "rotary_dim": 128, "layout": "half", "scaling": "yarn", "span": 131072},
        # q and k of the Llama-7B-shaped prefill batch
        {"name": "norm 32556 tokens", "op": "norm", "dtype": "bf16", "tokens": 32556,
         "heads": "32+32", "head_dim": 128, "rotary_dim": 128, "layout": "half",
         "scaling": "none", "span": 2048},
        # a checking run in float32: a quarter of each head turns, in neighbouring pairs
        {"name": "norm fp32 part", "op": "norm", "dtype": "fp32", "tokens": 1021, "heads": "12+4",
         "head_dim": 80, "rotary_dim": 20, "layout": "interleaved", "scaling": "linear",
         "span": 65536},
        # one new token for each request of a Qwen-32B decode batch
        {"name": "cache fp8 512 tokens", "op": "cache", "dtype": "bf16", "cache": "fp8",
         "kv_heads": 8, "head_dim": 128, "page": 64, "requests": 512, "each": 1},
        # prompts of ragged lengths
        {"name": "cache int8 prompts", "op": "cache", "dtype": "bf16", "cache": "int8",
         "kv_heads": 8, "head_dim": 128, "page": 128, "requests": 29, "each": 2048},
        # prompts of a Llama-7B layer, held as they are
        {"name": "cache bf16 prompts", "op": "cache", "dtype": "bf16", "cache": "native",
         "kv_heads": 32, "head_dim": 128, "page": 32, "requests": 24, "each": 1024},
        # one token of one request through a Llama-7B layer
        dict(llama, name="attend 1 token", op="attend", cache="native", page=64, requests=1,
             queries=1, own=2047, prefixes=0, prefix=0),
        # a Llama-7B decode batch, 8 adapters with a system prompt of their own
        dict(llama, name="attend fp8 256 requests", op="attend", cache="fp8", page=64,
             requests=256, queries=1, own=2048, prefixes=8, prefix=1024),
        # a Qwen-32B decode batch behind 16 long documents
        dict(qwen, name="attend int8 512 requests", op="attend", cache="int8", page=128,
             requests=512, queries=1, own=1024, prefixes=16, prefix=16384),
        # questions of several hundred tokens about one document
        dict(qwen, name="attend prompts", op="attend", cache="native", page=64, requests=16,
             queries=1024, own=1024, prefixes=1, prefix=4096),
        # a checking run in float32 on odd sizes
        {"name": "attend fp32 ragged", "op": "attend", "dtype": "fp32", "heads": 12, "kv_heads": 4,
         "head_dim": 80, "cache": "native", "page": 32, "requests": 13, "queries": 40, "own": 333,
         "prefixes": 2, "prefix": 97},
    ]


def _spread(rng, low, high):
    """A whole number whose logarithm is uniform."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm", "cache", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    head_dim = rng.choice([64, 80, 96, 128, 128, 128, 256])
    if op == "norm":
        rotary_dim = head_dim if rng.random() < 0.6 else 2 * rng.randint(4, head_dim // 2)
        heads = [rng.randint(1, 64), rng.randint(1, 32)][:rng.choice([1, 2, 2])]
        most = 32556 * 64 * 128 // (sum(heads) * head_dim) // (2 if dtype == "fp32" else 1)
        tokens = _spread(rng, 1, min(32556, most))
        return {"op": op, "dtype": dtype, "tokens": tokens, "heads": "+".join(map(str, heads)),
                "head_dim": head_dim, "rotary_dim": rotary_dim,
                "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["none", "linear", "yarn", "banded"]),
                "span": _spread(rng, 64, 1 << 20)}
    case = {"op": op, "dtype": dtype, "cache": rng.choice(["native", "fp8", "int8"]),
            "kv_heads": rng.choice([1, 2, 4, 8, 8, 16, 32]), "head_dim": head_dim,
            "page": rng.choice([32, 64, 64, 128, 256])}
    if op == "cache":
        case.update(requests=_spread(rng, 1, 512), each=rng.choice([1, _spread(rng, 1, 4096)]))
        most = max(work(c)["bytes"] for c in listed() if c["op"] == "cache")
        while work(case)["bytes"] > most:
            case["each" if case["each"] > 1 else "requests"] //= 2
        return case
    case["heads"] = case["kv_heads"] * rng.choice([1, 1, 2, 4, 5, 8])
    while case["heads"] > 64:
        case["heads"] //= 2
        case["kv_heads"] //= 2
    case["requests"] = _spread(rng, 1, 512)
    prefixes = min(case["requests"], rng.choice([0, 1, rng.randint(2, 16)]))
    case.update(queries=rng.choice([1, 1, _spread(rng, 2, 1024)]),
                own=_spread(rng, 1, 8192), prefixes=prefixes,
                prefix=_spread(rng, 1, 16384) if prefixes else 0)
    case["own"] = max(case["own"], case["queries"])
    most = [work(c) for c in listed() if c["op"] == "attend" and c["dtype"] == "bf16"]
    flops = max(w["flops"] for w in most) // (16 if dtype == "fp32" else 1)
    size = max(w["bytes"] for w in most)
    while work(case)["flops"] > flops or work(case)["bytes"] > size:
        if case["requests"] > 16:
            case["requests"] //= 2
        elif case["queries"] > 8:
            case["queries"] //= 2
        else:
            case["own"], case["prefix"] = max(1, case["own"] // 2, case["queries"]), case["prefix"] // 2
            case["prefixes"] = case["prefixes"] if case["prefix"] else 0
    return case


def _sizes(text):
    return [int(v) for v in text.split("+")]


def _ragged(count, low, high, salt):
    """`count` lengths of the range, the same for the same arguments, the longest among them."""
    rng = random.Random(salt * 1000003 + count * 8191 + high)
    return [high] + [rng.randint(low, high) for _ in range(count - 1)]


def _requests(case):
    """New tokens, and tokens in the request's own pages (the new ones among them), by request;
    the first and one past the last request of each prefix."""
    n = case["requests"]
    queries = [1] * n if case["queries"] == 1 else _ragged(n, 1, case["queries"], 1)
    lengths = [max(q, o) for q, o in zip(queries, _ragged(n, 1, case["own"], 2))]
    p = case["prefixes"]
    bounds = [n * i // p for i in range(p + 1)] if p else []
    return queries, lengths, bounds


# ---------------------------------------------------------------------------
# inputs

def _rotary_settings(case):
    """What a model's configuration says of its rotary positions."""
    s = {"head_dim": case["head_dim"], "rotary_dim": case["rotary_dim"], "layout": case["layout"],
         "base": 10000.0, "scaling": case["scaling"]}
    if case["scaling"] != "none":
        s["factor"] = 8.0
    if case["scaling"] in ("yarn", "banded"):
        s["original_positions"] = 16384
    if case["scaling"] == "yarn":
        s.update(beta_fast=32.0, beta_slow=1.0)
    if case["scaling"] == "banded":
        s.update(low_factor=1.0, high_factor=4.0)
    return s


def _keys(gen, tokens, case):
    """Keys or values of one projection: unit variance, a few channels three times as large."""
    gain = torch.ones(case["kv_heads"], case["head_dim"], device="cuda")
    gain[:, torch.randint(case["head_dim"], (4,), generator=gen, device="cuda")] = 3
    x = torch.randn(tokens, case["kv_heads"], case["head_dim"], generator=gen, device="cuda")
    return (x * gain).to(_TYPES[case["dtype"]])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": case}
    if case["op"] == "norm":
        widths = [h * case["head_dim"] for h in _sizes(case["heads"])]
        dtype = _TYPES[case["dtype"]]
        state.update(
            settings=_rotary_settings(case), eps=1e-6,
            x=[(3 * torch.randn(case["tokens"], w, generator=gen, device="cuda")).to(dtype) for w in widths],
            weight=[(1 + 0.2 * torch.randn(case["head_dim"], generator=gen, device="cuda")).to(dtype)
                    for _ in widths],
            positions=torch.randint(case["span"], (case["tokens"],), generator=gen, device="cuda",
                                    dtype=torch.int32))
    elif case["op"] == "cache":
        _prepare_cache(state, gen)
    else:
        _prepare_attend(state, gen)
    if own:
        _prepare_own(state)
    return state


def _paged(gen, lengths, page):
    """Pages in random order for each of the lengths: int32 [len(lengths)][most pages]."""
    counts = [-(-n // page) for n in lengths]
    order = torch.randperm(sum(counts), generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(len(lengths), max(counts + [1]), dtype=torch.int32, device="cuda")
    which = torch.arange(table.shape[1], device="cuda")[None] < torch.tensor(counts, device="cuda")[:, None]
    table[which] = order
    return table


def _slots(table, row, first, end, page):
    """Where tokens first..end-1 of a row of the table are held."""
    at = torch.arange(first, end, device="cuda")
    return table[row, at // page].long() * page + at % page


def _prepare_cache(state, gen):
    """Each request's tokens follow some that its pages hold already."""
    case = state["case"]
    n, page = case["requests"], case["page"]
    each = [1] * n if case["each"] == 1 else _ragged(n, 1, case["each"], 3)
    before = torch.randint(2048 if case["each"] == 1 else page, (n,), generator=gen, device="cuda").tolist()
    table = _paged(gen, [b + e for b, e in zip(before, each)], page)
    state["slots"] = torch.cat([_slots(table, i, before[i], before[i] + each[i], page)
                                for i in range(n)]).to(torch.int32)
    state["pages"] = sum(-(-(b + e) // page) for b, e in zip(before, each))
    state["k"], state["v"] = (_keys(gen, sum(each), case) for _ in range(2))


def _prepare_attend(state, gen):
    case = state["case"]
    queries, lengths, bounds = _requests(case)
    n, p, page = case["requests"], case["prefixes"], case["page"]
    every = _paged(gen, lengths + [case["prefix"]] * p, page)
    state["pages"] = sum(-(-v // page) for v in lengths + [case["prefix"]] * p)
    state["table"] = every[:n].contiguous()
    state["prefix_table"] = every[n:].contiguous()
    state["k"], state["v"] = (_keys(gen, state["pages"] * page, case) for _ in range(2))
    state["q"] = torch.randn(sum(queries), case["heads"] * case["head_dim"], generator=gen,
                             device="cuda").to(_TYPES[case["dtype"]])
    starts = [0]
    for q in queries:
        starts.append(starts[-1] + q)
    state.update(starts=starts, lengths=lengths, bounds=bounds,
                 scale=1 / math.sqrt(case["head_dim"]))
    if not own:
        state["k"], state["v"] = _held(state["k"], case["cache"]), _held(state["v"], case["cache"])


def _prepare_own(state):
    """The slot pool, the cache with what it holds, the output buffers, and the call, as a
    serving program sets them up once."""
    from lora_adapter_application_amd import binding
    case = state["case"]
    device = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    if case["op"] == "norm":
        slots = binding.Slots(1, 1, [(64, x.shape[1]) for x in state["x"]], case["dtype"], case["tokens"])
        state["y"] = [torch.empty_like(x) for x in state["x"]]
        rotary = binding.lora_rotary_init(**state["settings"])
        state["call"] = slots.bind_norm_rotary(rotary, list(range(len(state["x"]))), state["x"], state["y"],
                                               state["positions"], state["weight"], state["eps"])
        return
    tokens = (state["slots"] if case["op"] == "cache" else state["q"]).shape[0]
    slots = binding.Slots(1, 1, [(64, 64)], case["dtype"], max(tokens, 8192))
    cache = slots.cache(case["kv_heads"], case["head_dim"], state["pages"], case["page"], case["cache"])
    state["cache"] = cache
    if case["op"] == "cache":
        state["y"] = [torch.empty_like(state["k"]), torch.empty_like(state["v"])]
        store = slots.bind_cache_store(cache, state["k"], state["v"], state["slots"])
        load = slots.bind_cache_load(cache, state["slots"], *state["y"])

        def call():
            store()
            load()
        state["call"] = call
        return
    held = state["pages"] * case["page"]
    for first in range(0, held, 8192):
        at = torch.arange(first, min(first + 8192, held), dtype=torch.int32, device="cuda")
        slots.cache_store(cache, state["k"][first:first + 8192], state["v"][first:first + 8192], at)
    torch.cuda.synchronize()
    del state["k"], state["v"]
    state["y"] = torch.empty_like(state["q"])
    batch = binding.AttendBatch(device(state["lengths"]), state["table"],
                                None if case["queries"] == 1 else device(state["starts"]), case["queries"])
    if case["prefixes"]:
        batch.share(device(state["bounds"]), device([case["prefix"]] * case["prefixes"]),
                    state["prefix_table"])
    state["call"] = slots.bind_attend(cache, case["heads"], state["q"], state["y"], batch, state["scale"])


# ---------------------------------------------------------------------------
# plain forms

def _held(x, kind):
    """x as the cache holds it: (values or codes, scale of each head of a token or None).  The
    quotients next to a border need 64 bits."""
    if kind == "native":
        return x, None
    high = x.float().abs().amax(-1, keepdim=True)
    scale = torch.div(high, torch.full_like(high, _TOP[kind]))
    codes = torch.empty(x.shape, dtype=torch.float8_e4m3fn if kind == "fp8" else torch.int8, device=x.device)
    for first in range(0, x.shape[0], 65536):
        part = slice(first, first + 65536)
        ratio = x[part].double() * _TOP[kind] / high[part].double()
        codes[part] = _e4m3(ratio) if kind == "fp8" else ratio.round().to(torch.int8)
    return codes, scale


def _e4m3(v):
    """The nearest fp8 value: 3 bits behind the leading one, steps of 2^-9 below 2^-6."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return ((v / step).round() * step).float().to(torch.float8_e4m3fn)


def _value(held, which=slice(None)):
    codes, scale = held
    return codes[which].float() if scale is None else codes[which].float() * scale[which]


def _frequencies(s, device):
    """Radians per position of each pair, and the factor on cosine and sine."""
    dim = s["rotary_dim"]
    f = s["base"] ** (-torch.arange(0, dim, 2, device=device, dtype=torch.float64) / dim)
    if s["scaling"] == "linear":
        return f / s["factor"], 1.0
    if s["scaling"] == "yarn":
        where = lambda turns: (dim * math.log(s["original_positions"] / (turns * 2 * math.pi))  # noqa: E731
                               / (2 * math.log(s["base"])))
        low = max(math.floor(where(s["beta_fast"])), 0)
        high = min(math.ceil(where(s["beta_slow"])), dim - 1)
        ramp = ((torch.arange(dim // 2, device=device, dtype=torch.float64) - low)
                / max(high - low, 0.001)).clamp(0, 1)
        return f / s["factor"] * ramp + f * (1 - ramp), 0.1 * math.log(s["factor"]) + 1
    if s["scaling"] == "banded":
        turns = s["original_positions"] * f / (2 * math.pi)
        keep = ((turns - s["low_factor"]) / (s["high_factor"] - s["low_factor"])).clamp(0, 1)
        return f / s["factor"] * (1 - keep) + f * keep, 1.0
    return f, 1.0


def _normed_rotated(x, weight, eps, settings, positions):
    dim, half = settings["rotary_dim"], settings["rotary_dim"] // 2
    f, factor = _frequencies(settings, x.device)
    angle = positions.double()[:, None, None] * f
    c, s = (angle.cos() * factor).float(), (angle.sin() * factor).float()
    h = x.view(x.shape[0], -1, settings["head_dim"]).float()
    h = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * weight.float()
    a, rest = h[..., :dim], h[..., dim:]
    if settings["layout"] == "half":
        a1, a2 = a[..., :half], a[..., half:]
        r = torch.cat((a1 * c - a2 * s, a2 * c + a1 * s), 2)
    else:
        a1, a2 = a[..., 0::2], a[..., 1::2]
        r = torch.stack((a1 * c - a2 * s, a2 * c + a1 * s), 3).flatten(2)
    return torch.cat((r, rest), 2).to(x.dtype).view(x.shape)


def _attended(state):
    """Request by request, the scores over the shared prefix formed for all of its requests."""
    case = state["case"]
    kv, dim, page = case["kv_heads"], case["head_dim"], case["page"]
    q = state["q"].float().view(-1, kv, case["heads"] // kv, dim)
    y = torch.empty_like(q)

    def part(table, row, length):          # [kv_heads][length][head_dim] of keys and of values
        at = _slots(table, row, 0, length, page)
        return _value(state["k"], at).transpose(0, 1), _value(state["v"], at).transpose(0, 1)

    def scores(q, k):                      # [kv_heads][tokens][heads of a kv head][length]
        s = q.transpose(0, 1).reshape(kv, -1, dim) @ k.transpose(1, 2).contiguous() * state["scale"]
        return s.view(kv, q.shape[0], q.shape[2], k.shape[1])

    groups = list(zip(state["bounds"], state["bounds"][1:])) or [(0, case["requests"])]
    for p, (first, end) in enumerate(groups):
        shared = None
        if case["prefixes"]:
            pk, pv = part(state["prefix_table"], p, case["prefix"])
            shared = scores(q[state["starts"][first]:state["starts"][end]], pk)
        for i in range(first, end):
            t0, t1, length = state["starts"][i], state["starts"][i + 1], state["lengths"][i]
            k, v = part(state["table"], i, length)
            s = scores(q[t0:t1], k)
            seen = (torch.arange(length, device=q.device)[None, :]
                    <= torch.arange(length - (t1 - t0), length, device=q.device)[:, None])
            s = s.masked_fill(~seen[None, :, None, :], -math.inf)
            if shared is not None:
                base = state["starts"][first]
                s = torch.cat((shared[:, t0 - base:t1 - base], s), 3)
                v = torch.cat((pv, v), 1)
            w = torch.exp(s - s.amax(3, keepdim=True))
            w = w / w.sum(3, keepdim=True)
            o = w.view(kv, -1, w.shape[3]) @ v
            y[t0:t1] = o.view(kv, t1 - t0, -1, dim).transpose(0, 1)
    return y.view(state["q"].shape).to(state["q"].dtype)


def run(state):
    if own:
        state["call"]()
        return state["y"]
    case = state["case"]
    if case["op"] == "norm":
        return [_normed_rotated(x, w, state["eps"], state["settings"], state["positions"])
                for x, w in zip(state["x"], state["weight"])]
    if case["op"] == "cache":
        return [_value(_held(x, case["cache"])).to(x.dtype) for x in (state["k"], state["v"])]
    return _attended(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    size = {"bf16": 2, "fp32": 4}[case["dtype"]]
    dim = case["head_dim"]
    if case["op"] == "norm":
        n = case["tokens"] * sum(_sizes(case["heads"]))
        return {"bytes": n * dim * 2 * size + 4 * case["tokens"],
                "flops": n * (4 * dim + 3 * case["rotary_dim"])}
    held = dim * size if case["cache"] == "native" else dim + 4     # of a token's head
    if case["op"] == "cache":
        n = case["requests"]
        tokens = n if case["each"] == 1 else sum(_ragged(n, 1, case["each"], 3))
        heads = 2 * tokens * case["kv_heads"]
        return {"bytes": heads * (2 * dim * size + 2 * held) + 8 * tokens, "flops": 4 * heads * dim}
    queries, lengths, _ = _requests(case)
    shared = case["prefix"] if case["prefixes"] else 0
    seen = sum(q * (shared + n - q) + q * (q + 1) // 2 for q, n in zip(queries, lengths))
    tokens = sum(lengths) + case["prefixes"] * shared
    return {"bytes": 2 * tokens * case["kv_heads"] * held + 2 * sum(queries) * case["heads"] * dim * size,
            "flops": 4 * seen * case["heads"] * dim}


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_normed(x, weight, eps, settings, positions):
    """Each head over its root mean square, its pairs as complex numbers times
    factor * exp(i position frequency)."""
    dim, kind = settings["rotary_dim"], settings["scaling"]
    rates, factor = [], 1.0
    for p in range(dim // 2):
        rate = settings["base"] ** (-2.0 * p / dim)
        slow = rate / settings.get("factor", 1.0)
        if kind == "linear":
            rate = slow
        elif kind == "yarn":
            factor = 1 + math.log(settings["factor"]) / 10
            pair = lambda turns: dim / 2 * (math.log(settings["original_positions"])  # noqa: E731
                                            - math.log(2 * math.pi * turns)) / math.log(settings["base"])
            first = max(0, math.floor(pair(settings["beta_fast"])))
            last = min(dim - 1, math.ceil(pair(settings["beta_slow"])))
            share = min(1.0, max(0.0, (p - first) / max(0.001, last - first)))
            rate = slow * share + rate * (1 - share)
        elif kind == "banded":
            length = 2 * math.pi / rate
            if length > settings["original_positions"] / settings["low_factor"]:
                rate = slow
            elif length >= settings["original_positions"] / settings["high_factor"]:
                share = ((settings["original_positions"] / length - settings["low_factor"])
                         / (settings["high_factor"] - settings["low_factor"]))
                rate = slow * (1 - share) + rate * share
        rates.append(rate)
    angle = torch.outer(positions.double(), torch.tensor(rates, dtype=torch.float64, device=x.device))
    turn = torch.polar(torch.full_like(angle, factor), angle)[:, None, :]
    out = x.double().reshape(x.shape[0], -1, settings["head_dim"])
    out = out * torch.rsqrt(out.square().mean(-1, keepdim=True) + eps) * weight.double()
    if settings["layout"] == "half":
        first, second = slice(0, dim // 2), slice(dim // 2, dim)
    else:
        first, second = slice(0, dim, 2), slice(1, dim, 2)
    z = torch.complex(out[..., first].contiguous(), out[..., second].contiguous()) * turn
    out[..., first], out[..., second] = z.real, z.imag
    return out.reshape(x.shape)


def _exact_held(x, kind):
    if kind == "native":
        return x.double()
    x = x.double()
    high = x.abs().amax(-1, keepdim=True)
    unit = high / _TOP[kind]
    level = x * _TOP[kind] / high                  # ties stay ties
    if kind == "int8":
        return torch.round(level) * unit
    # the values from zero up: 8 in steps of 2^-9, then 8 between each two powers of two
    values = [i / 512 for i in range(8)] + [(8 + i) * 2.0 ** (e - 3) for e in range(-6, 9) for i in range(8)]
    values = torch.tensor(values[:127], dtype=torch.float64, device=x.device)
    middle = (values[1:] + values[:-1]) / 2
    below, above = torch.bucketize(level.abs(), middle), torch.bucketize(level.abs(), middle, right=True)
    return values[torch.where(below % 2 == 0, below, above)] * level.sign() * unit


def _exact_attended(state, held_k, held_v):
    """Every request by itself over the whole of its context, one key-value head at a time."""
    case = state["case"]
    kv, dim, page = case["kv_heads"], case["head_dim"], case["page"]
    group = case["heads"] // kv
    q = state["q"].double().view(-1, kv, group, dim)
    out = torch.empty_like(q)
    owner = {}
    for p in range(case["prefixes"]):
        for i in range(state["bounds"][p], state["bounds"][p + 1]):
            owner[i] = p
    for i in range(case["requests"]):
        t0, t1 = state["starts"][i], state["starts"][i + 1]
        at = _slots(state["table"], i, 0, state["lengths"][i], page)
        if i in owner:
            at = torch.cat((_slots(state["prefix_table"], owner[i], 0, case["prefix"], page), at))
        last = torch.arange(at.numel() - (t1 - t0), at.numel(), device=at.device)
        hidden = torch.arange(at.numel(), device=at.device)[None, :] > last[:, None]
        hidden = hidden.repeat_interleave(group, 0)
        for h in range(kv):
            k, v = held_k(at, h), held_v(at, h)
            logit = torch.mm(q[t0:t1, h].reshape(-1, dim), k.t().contiguous()).mul_(state["scale"])
            logit[hidden] = -math.inf
            out[t0:t1, h] = torch.mm(torch.softmax(logit, 1), v).view(t1 - t0, group, dim)
    return out.view(state["q"].shape)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        state = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "norm":
        return [_exact_normed(x, w, state["eps"], state["settings"], state["positions"])
                for x, w in zip(state["x"], state["weight"])]
    if case["op"] == "cache":
        return [_exact_held(x, case["cache"]) for x in (state["k"], state["v"])]

    def reader(held):
        codes, scale = held
        return lambda at, h: (codes[at, h].double() if scale is None
                              else codes[at, h].double() * scale[at, h].double())
    return _exact_attended(state, reader(state["k"]), reader(state["v"]))
