"""Paged batches held in 8 bits, and plain 64-bit forms of the operators of a compact cache."""
from __future__ import annotations

import math

import torch

from tests import decoder_testlib as lib

E4M3 = torch.float8_e4m3fn
LEAST = 2.0 ** -100
HALF8 = torch.finfo(E4M3).eps / 2   # half a step of E4M3 relative to the value
TINY8 = 2.0 ** -10                  # half a step of its subnormal numbers


def power(x):
    """The smallest power of two >= x (fp64 tensor), at least LEAST."""
    x = x.double().clamp(min=LEAST)
    m, e = torch.frexp(x)  # x = m 2^e, m in [1/2, 1)
    return ((e.long() - (m == 0.5).long() + 1023) << 52).view(torch.float64)


def put8(pages, index, codes):
    """pages[index] = codes for E4M3 tensors."""
    pages.view(torch.uint8)[index] = codes.view(torch.uint8)


class Batch8(lib.Batch):
    """lib.Batch whose cache is E4M3 with a scale for each page and head: `k_scale`, `v_scale`. Places that
    hold no token keep NaN; `spread`: how much the pages' magnitudes differ (powers of e); `odd`: scales
    that are no powers of two."""

    def __init__(self, *a, spread=1.0, odd=False, seed=0, **kw):
        super().__init__(*a, seed=seed, **kw)
        g = torch.Generator().manual_seed(seed + 1)
        pages, Hkv, page, d = self.k_pages.shape
        dev = self.k_pages.device
        for name in ("k", "v"):
            x = getattr(self, name + "_pages")
            size = (spread * torch.randn(pages, Hkv, 1, 1, generator=g)).exp().to(dev)
            x64 = x.double() * size
            top = torch.nan_to_num(x64.abs(), nan=0.0).amax((2, 3))
            scale = power(top / 448.0)
            if odd:
                scale = scale * (1 + torch.rand(pages, Hkv, generator=g).to(dev).double())
            scale = scale.float()
            codes = torch.empty_strided(x.shape, x.stride(), dtype=torch.uint8, device=dev)
            codes.copy_((x64 / scale[..., None, None].double()).float().to(E4M3).view(torch.uint8))
            setattr(self, name + "_pages", codes.view(E4M3))
            setattr(self, name + "_scale", scale.contiguous())
        self.decode()

    def decode(self):
        """keys and values of each sequence as the cache holds them, in 64 bits."""
        self.keys, self.values, self.codes, self.vscales = [], [], [], []
        for b, t in enumerate(self.total):
            used = self.block_table[b, :-(-t // self.page)].long()
            for out, pages, scale in ((self.keys, self.k_pages, self.k_scale), (self.values, self.v_pages, self.v_scale)):
                x = pages.view(torch.uint8)[used].view(E4M3).double() * scale[used][..., None, None].double()
                out.append(x.transpose(0, 1).flatten(1, 2)[:, :t])
            self.vscales.append(self.v_scale[used].double())


def attend64(b, q, scale, causal):
    """O, L and how far each may be off, from b.keys and b.values (64 bits).

    As in decoder_testlib.attend64, with P held in 11 bits whatever q's type: u = 2^-11 relative to each P.
    Small ones are cut off, at half a step of E5M2's subnormal numbers (2^-17) in P' = P v_scale / (largest
    v_scale) 2^11, at half a step of fp16's (2^-25) in 2^7 of it with more rows: either way by less than
    2^-28 (largest v_scale) times the code. (Each row's sum is at least 1 in P's unit.)"""
    u16 = torch.finfo(torch.float16).eps / 2
    T, Hq, d = q.shape
    u, sub = lib.step(q.dtype), lib.tiny(q.dtype)
    O = torch.zeros(T, Hq, d, dtype=torch.float64, device=q.device)
    L = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=q.device)
    tol_o, tol_l = torch.zeros_like(O), torch.zeros_like(L)
    group = Hq // b.Hkv
    for i, (n, t) in enumerate(zip(b.new, b.total)):
        if n == 0 or t == 0:
            continue
        rows = slice(b.cu[i], b.cu[i] + n)
        kk, vv = (x[i].repeat_interleave(group, 0) for x in (b.keys, b.values))
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
        unit = b.vscales[i].repeat_interleave(b.page, 0)[:t].T[..., None]
        codes = torch.where(unit > 0, b.values[i] / unit, 0.0).abs().sum(1, keepdim=True)
        small = (2.0 ** -28 * b.vscales[i].amax(0)[:, None, None] * codes).repeat_interleave(group, 0)
        weight = (u16 + 2 * e)[..., None] * (p @ vv.abs()) + small
        tol_o[rows] = weight.transpose(0, 1) + u * O[rows].abs() + sub + 2.0 ** -18 * weight.transpose(0, 1) + (
            2.0 ** -19 * (p @ vv.abs()).transpose(0, 1))
        tol_l[rows] = (e + 2.0 ** -18 + 2.0 ** -22 * lse.abs().masked_fill(~some, 0.0)).transpose(0, 1)
    return O, L, tol_o, tol_l
