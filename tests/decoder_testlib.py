"""Plain 64-bit forms of the decoder-block operators, and paged batches to run them on."""
from __future__ import annotations

import math

import torch

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def step(dtype) -> float:
    """Half a step of `dtype` relative to the value: what one rounding may be off."""
    return torch.finfo(dtype).eps / 2


def tiny(dtype) -> float:
    """Half a step of the subnormal numbers of `dtype`."""
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2


def rope_table(length, rot, device="cpu", base=10000.0):
    inv = base ** (-torch.arange(0, rot, 2, device=device, dtype=torch.float64) / max(rot, 1))
    a = torch.arange(length, device=device, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def turn64(x, table_rows, interleaved, back=False):
    """The rotation (or its transpose) of the first rot elements of x [..., d] in 64 bits;
    table_rows [..., rot] broadcasts over x's leading axes."""
    rot = table_rows.shape[-1]
    cos, sin = table_rows.double().chunk(2, -1)
    if back:
        sin = -sin
    y = x.double().clone()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        xa, xb = x[..., a].double(), x[..., b].double()
        y[..., a] = xa * cos[..., i] - xb * sin[..., i]
        y[..., b] = xb * cos[..., i] + xa * sin[..., i]
    return y


def norm_rope64(x, w, rows, eps, interleaved):
    """(y, size): size bounds the magnitudes that the rotation adds up for each element."""
    x = x.double()
    n = x * (x.square().mean(-1, keepdim=True) + eps).rsqrt() * w.double()
    size = n.abs().amax(-1, keepdim=True).expand_as(n)
    return (n if rows is None else turn64(n, rows, interleaved)), size


def norm_rope_grad64(g, x, w, rows, eps, interleaved):
    x, g, w = x.double(), g.double(), w.double()
    if rows is not None:
        g = turn64(g, rows, interleaved, back=True)
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    u = g * w
    dx = r * (u - x * r * (u * x * r).mean(-1, keepdim=True))
    return dx, (g * x * r).flatten(0, -2).sum(0), (g * x * r).abs().flatten(0, -2).sum(0), r


class Batch:
    """Sequences over a paged cache. new/total: tokens of each; the cache's unused places hold
    `fill`, pages are handed out in a random order, `lead` and `behind` rows belong to nobody."""

    def __init__(self, new, total, Hkv, d, page, dtype, seed=0, device="cuda", token_major=False, fill=math.nan,
                 spare=3, wide=None, lead=0, behind=0):
        g = torch.Generator().manual_seed(seed)
        self.new, self.total, self.page, self.Hkv, self.d, self.dtype = list(new), list(total), page, Hkv, d, dtype
        B, held = len(new), [-(-t // page) for t in total]
        pages = sum(held) + spare
        order = torch.randperm(pages, generator=g).int()
        width = max(held + [0]) if wide is None else wide
        table = torch.full((B, width), -7, dtype=torch.int32)  # entries that must not be read
        at = 0
        for b, n in enumerate(held):
            table[b, :n] = order[at:at + n]
            at += n
        cu = [lead]
        for n in new:
            cu.append(cu[-1] + n)
        self.T = cu[-1] + behind
        self.cu = cu
        shape = (pages, page, Hkv, d) if token_major else (pages, Hkv, page, d)
        k, v = (torch.full(shape, fill, dtype=dtype) for _ in range(2))
        if token_major:
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        self.keys, self.values = [], []
        for b, t in enumerate(total):
            kk = torch.randn(Hkv, t, d, generator=g).to(dtype)
            vv = torch.randn(Hkv, t, d, generator=g).to(dtype)
            self.keys.append(kk.to(device))
            self.values.append(vv.to(device))
            for i in range(held[b]):
                n = min(page, t - i * page)
                k[table[b, i], :, :n] = kk[:, i * page:i * page + n]
                v[table[b, i], :, :n] = vv[:, i * page:i * page + n]
        keep = (lambda x: x.transpose(1, 2).contiguous().to(device).transpose(1, 2)) if token_major else (
            lambda x: x.to(device))
        self.k_pages, self.v_pages = keep(k), keep(v)
        self.block_table = table.to(device)
        self.cu_seqlens = torch.tensor(cu, dtype=torch.int32, device=device)
        self.seq_lens = torch.tensor(total, dtype=torch.int32, device=device)
        self.max_q = max(list(new) + [1])
        self.g = g

    def rows(self, H, std=1.0, device="cuda"):
        return (torch.randn(self.T, H, self.d, generator=self.g) * std).to(self.dtype).to(device)

    def cached(self, b):
        """Sequence b's keys and values as the pages hold them, [Hkv, total, d] each."""
        used = self.block_table[b, :-(-self.total[b] // self.page)].long()
        return tuple(x[used].transpose(0, 1).flatten(1, 2)[:, :self.total[b]] for x in (self.k_pages, self.v_pages))


def attend64(batch: Batch, q, scale, causal, keys=None, values=None):
    """O, L and how far each may be off: for every sequence's rows, in 64 bits.

    A kernel may round each probability to the type of the inputs (one half step u relative to it,
    plus a subnormal half step where it is tiny), sums in 32 bits, and rounds O. A score's sum of
    d products in 32 bits, each step off by at most 2^-22 of the sum of magnitudes (a tensor core
    truncates what it aligns), is off by e <= d 2^-22 scale max_j sum |q||k_j|; so is L, and each
    probability by a factor 1 + 2e at most (numerator and sum)."""
    T, Hq, d = q.shape
    u, sub = step(q.dtype), tiny(q.dtype)
    O = torch.zeros(T, Hq, d, dtype=torch.float64, device=q.device)
    L = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=q.device)
    tol_o, tol_l = torch.zeros_like(O), torch.zeros_like(L)
    group = Hq // batch.Hkv
    for b, (n, t) in enumerate(zip(batch.new, batch.total)):
        if n == 0:
            continue
        rows = slice(batch.cu[b], batch.cu[b] + n)
        if t == 0:
            continue
        kk = (batch.keys[b] if keys is None else keys[b]).double().repeat_interleave(group, 0)
        vv = (batch.values[b] if values is None else values[b]).double().repeat_interleave(group, 0)
        x = q[rows].double().transpose(0, 1)
        s = scale * x @ kk.transpose(1, 2)
        seen = torch.ones(n, t, dtype=torch.bool, device=q.device)
        if causal:
            last = torch.arange(n, device=q.device) + t - n
            seen = torch.arange(t, device=q.device)[None] <= last[:, None]
        s = s.masked_fill(~seen, -math.inf)
        some = seen.any(1)
        lse = torch.logsumexp(s, -1)
        p = torch.exp(s - lse.masked_fill(~some, 0.0)[..., None])
        e = d * 2.0 ** -22 * scale * (x.abs() @ kk.abs().transpose(1, 2)).amax(-1)
        O[rows] = (p @ vv).transpose(0, 1)
        L[rows] = lse.transpose(0, 1)
        weight = (u + 2 * e)[..., None] * (p @ vv.abs()) + 2 * sub * vv.abs().sum(1, keepdim=True)
        tol_o[rows] = weight.transpose(0, 1) + u * O[rows].abs() + sub + 2.0 ** -18 * weight.transpose(0, 1)
        tol_l[rows] = (e + 2.0 ** -18 + 2.0 ** -22 * lse.abs().masked_fill(~some, 0.0)).transpose(0, 1)
    return O, L, tol_o, tol_l
