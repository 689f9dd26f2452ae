"""Plain forms in 64 bits of the paged cache and of attention over it, with the bounds that the
tests hold the kernels to, and batches for them."""
from __future__ import annotations

import math

import torch

from lora_adapter_application_amd import binding
from layer_util import HALF_STEP, TORCH, U32

TOP = {"fp8": 448.0, "int8": 127.0}


def e4m3_values():
    """The values of an 8-bit float with 4 exponent and 3 mantissa bits, from zero up."""
    v = [i / 512 for i in range(8)] + [(8 + i) * 2.0 ** (e - 3) for e in range(-6, 9) for i in range(8)]
    return torch.tensor(v[:127], dtype=torch.float64)


def coded(x, kind):
    """(codes as their values in 64 bits, scale in fp32) of heads x [..., head_dim]: the quotient in 64
    bits, which holds it to a tie or far from one."""
    x = x.double()
    high = x.abs().amax(-1, keepdim=True)
    odd = ~torch.isfinite(high)
    high = torch.where(odd, torch.ones_like(high), high).clamp_min(2.0 ** -100)
    level = x * TOP[kind] / high
    if kind == "int8":
        codes = torch.round(level) + 0.0                      # whole numbers have one zero
    else:
        values = e4m3_values()
        middle = (values[1:] + values[:-1]) / 2
        below, above = torch.bucketize(level.abs(), middle), torch.bucketize(level.abs(), middle, right=True)
        codes = values[torch.where(below % 2 == 0, below, above).clamp_max(126)] * level.sign()
    scale = (high.float() / TOP[kind])
    scale = torch.where(odd, torch.full_like(scale, math.nan), scale)
    return torch.where(odd, torch.zeros_like(codes), codes), scale


def held(x, kind):
    """x as the cache holds it, in 64 bits."""
    if kind == "native":
        return x.double()
    codes, scale = coded(x, kind)
    return codes * scale.double()


def read_back(x, kind):
    """What a load of stored x gives, bit for bit."""
    if kind == "native":
        return x
    codes, scale = coded(x, kind)
    return (codes.float() * scale).to(x.dtype)


class Requests:
    """A batch: queries and lengths by request, prefixes as (first request, end, length)."""

    def __init__(self, seed, dtype, kind, heads, kv_heads, head_dim, page, queries, lengths, prefixes=(),
                 lead=0, tail=0, poison=True, spread=1.0, q_start=True):
        self.gen = torch.Generator().manual_seed(seed)
        self.dtype, self.kind, self.heads, self.kv, self.dim, self.page = dtype, kind, heads, kv_heads, head_dim, page
        self.queries, self.lengths, self.prefixes = list(queries), list(lengths), list(prefixes)
        n = len(self.queries)
        self.starts = [lead]
        for q in self.queries:
            self.starts.append(self.starts[-1] + q)
        self.tokens = self.starts[-1] + tail
        self.q_start = q_start
        every = self.lengths + [p[2] for p in self.prefixes]
        counts = [-(-v // page) for v in every]
        self.pages = sum(counts) + 2                          # two that no request has
        order = torch.randperm(self.pages, generator=self.gen).to(torch.int32)
        rows, at = [], 0
        for c in counts:
            rows.append(order[at:at + c])
            at += c
        width = max([1] + counts[:n])
        self.table = torch.zeros(n, width, dtype=torch.int32)
        for i in range(n):
            self.table[i, :counts[i]] = rows[i]
        width = max([1] + counts[n:])
        self.prefix_table = torch.zeros(len(self.prefixes), width, dtype=torch.int32)
        for p in range(len(self.prefixes)):
            self.prefix_table[p, :counts[n + p]] = rows[n + p]
        slots = self.pages * page
        make = lambda: (torch.randn(slots, kv_heads, head_dim, generator=self.gen) * spread).to(TORCH[dtype])  # noqa: E731
        self.k, self.v = make(), make()
        self.used = torch.zeros(slots, dtype=torch.bool)
        for row, length in zip(rows, every):
            s = torch.arange(length)
            self.used[row[s // page].long() * page + s % page] = True
        if poison:                                            # slots of no token may hold anything
            self.k[~self.used] = math.nan
            self.v[~self.used] = math.inf
        self.q = torch.randn(self.tokens, heads * head_dim, generator=self.gen).to(TORCH[dtype])

    def slots_of(self, row, length):
        s = torch.arange(length)
        return row[s // self.page].long() * self.page + s % self.page

    def prefix_of(self, i):
        for p, (a, b, length) in enumerate(self.prefixes):
            if a <= i < b:
                return p
        return -1

    def batch(self):
        d = lambda t: torch.as_tensor(t, dtype=torch.int32).cuda()  # noqa: E731
        b = binding.AttendBatch(d(self.lengths), d(self.table), d(self.starts) if self.q_start else None,
                                max([1] + self.queries), self.tokens)
        if self.prefixes:
            b.share(d([p[0] for p in self.prefixes] + [self.prefixes[-1][1]]), d([p[2] for p in self.prefixes]),
                    d(self.prefix_table))
        return b

    def fill(self, S, cache):
        """Store every slot of the cache."""
        for first in range(0, self.k.shape[0], S.max_tokens):
            part = slice(first, min(first + S.max_tokens, self.k.shape[0]))
            at = torch.arange(part.start, part.stop, dtype=torch.int32).cuda()
            S.cache_store(cache, self.k[part].cuda(), self.v[part].cuda(), at)
        torch.cuda.synchronize()

    def make(self):
        S = binding.Slots(1, 1, [(64, 64)], self.dtype, max(self.tokens, 4096))
        cache = S.cache(self.kv, self.dim, self.pages, self.page, self.kind)
        self.fill(S, cache)
        return S, cache

    def attended(self, scale):
        """(result, bound of its error) in 64 bits; rows of no request are NaN in the result.

        Of a score, the products of a row (exact in fp32 for bf16 and codes) are summed with an
        error of at most 2u = 2^-23 of the sum of their sizes each, u = 2^-24, scaled twice with u
        each, and its exponential is off by as much as the score itself, by 2^-21 for the function and its
        argument, and by u of the argument's size (under 2^7 in the tests).  Weights of a bf16
        ctx are rounded once (2^-8), a code's scale twice (2u); the weighted sum adds 2u per token,
        as does the sum below it, and their parts are joined with few roundings (2^-20 in all)."""
        bf16 = self.dtype == "bf16"
        out = torch.full((self.tokens, self.kv, self.heads // self.kv, self.dim), math.nan, dtype=torch.float64)
        bound = torch.zeros_like(out)
        q = self.q.double().view(out.shape)
        kh, vh = held(self.k, self.kind), held(self.v, self.kind)
        for i, (n, length) in enumerate(zip(self.queries, self.lengths)):
            p = self.prefix_of(i)
            at = self.slots_of(self.table[i], length)
            pre = 0
            if p >= 0:
                pre = self.prefixes[p][2]
                at = torch.cat((self.slots_of(self.prefix_table[p], pre), at))
            k, v = kh[at], vh[at]
            for j in range(n):
                sees = pre + max(0, length - n + j + 1)
                t = self.starts[i] + j
                if not sees:
                    out[t] = 0
                    continue
                kk, vv = k[:sees].transpose(0, 1), v[:sees].transpose(0, 1)      # [kv][sees][dim]
                s = q[t] @ kk.transpose(1, 2) * scale
                size = q[t].abs() @ kk.abs().transpose(1, 2) * scale
                w = torch.softmax(s, -1)
                out[t] = w @ vv
                rel = (self.dim + 4) * 2 * U32 * size.amax(-1, keepdim=True)
                rel = 2 * rel + 2.0 ** -16 + (2.0 ** -8 if bf16 else 0) + (2 * sees + 64) * 2 * U32
                bound[t] = (w @ vv.abs()) * rel
        out, bound = out.view(self.q.shape), bound.view(self.q.shape)
        return out, bound + HALF_STEP[TORCH[self.dtype]] * (out.abs() + bound)

    def own_rows(self):
        rows = torch.zeros(self.tokens, dtype=torch.bool)
        for a, b in zip(self.starts, self.starts[1:]):
            rows[a:b] = True
        return rows


def check_rows(r, got, scale, before, what):
    """Rows of requests within their bound, the others as they were."""
    want, bound = r.attended(scale)
    rows = r.own_rows()
    got = got.cpu()
    assert torch.equal(got[~rows].view(torch.int16 if r.dtype == "bf16" else torch.int32),
                       before.cpu()[~rows].view(torch.int16 if r.dtype == "bf16" else torch.int32)), \
        f"{what}: a row of no request changed"
    g, w, b = got[rows].double(), want[rows], bound[rows]
    assert torch.isfinite(g).all(), f"{what}: not finite"
    err = (g - w).abs()
    assert bool((err <= b).all()), f"{what}: worst error / bound {(err / b.clamp_min(1e-300)).max():.3f}"
    return (err / b.clamp_min(1e-300)).max().item() if err.numel() else 0.0
