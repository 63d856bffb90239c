"""The operators of a compact cache, as cases that can be measured: a paged cache of keys and values
held in 8 bits (E4M3) with one scale for each page and head, and the eviction of what little
attention has fallen on.

  append  new keys and values into the 8-bit cache, the keys rotated by position on the way
  attend  attention of new tokens (single ones, drafts, a chunk of a prompt) over the 8-bit cache
  weigh   the attention weight that new tokens give to every cached token of each key head, added
          to what earlier tokens gave it (8-bit or 16-bit cache)
  evict   each key head's cache cut to a budget of tokens: the most recent ones and those of the
          highest weight stay, moved together in order (8-bit or 16-bit cache)

`own = False` computes them in elementary torch operations in 32 bits; `own = True` calls the
package's operators on the same state.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
BASE = 10000.0
MOST = 448.0           # of E4M3
LEAST_SCALE = 2.0 ** -100


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one user's next token, a short conversation: latency alone
        dict(name="attend one sequence", op="attend", B=1, Hq=32, Hkv=8, d=128, page=16, new=1, new_hi=1,
             ctx=1000, ctx_hi=1000, lens=1, causal=True, dtype="bf16"),
        # a server's batch of ragged conversations, one token each, small pages: memory speed
        dict(name="attend ragged batch", op="attend", B=64, Hq=32, Hkv=8, d=128, page=16, new=1, new_hi=1,
             ctx=200, ctx_hi=8191, lens=2, causal=True, dtype="bf16"),
        # drafts of a few tokens to check, d = 64, every query head with its own keys
        dict(name="attend drafts d64", op="attend", B=24, Hq=12, Hkv=12, d=64, page=64, new=2, new_hi=7,
             ctx=1, ctx_hi=4097, lens=4, causal=True, dtype="fp16"),
        # a chunk of a long prompt over what the cache holds of it: arithmetic
        dict(name="attend chunk of a long prompt", op="attend", B=1, Hq=16, Hkv=2, d=128, page=64, new=2048,
             new_hi=2048, ctx=30720, ctx_hi=30720, lens=6, causal=True, dtype="bf16"),
        # one token of each of 64 sequences into the cache
        dict(name="append one token each", op="append", B=64, Hkv=8, d=128, page=16, new=1, new_hi=1,
             ctx=0, ctx_hi=8191, lens=7, rot=128, interleaved=False, dtype="bf16"),
        # ragged prompt chunks into the cache, half of each head rotated
        dict(name="append ragged chunks", op="append", B=9, Hkv=8, d=128, page=64, new=1, new_hi=8192,
             ctx=0, ctx_hi=5000, lens=8, rot=64, interleaved=True, dtype="fp16"),
        # after a decoding step of a ragged batch: every cached key's weight grows by the new tokens'
        dict(name="weigh single tokens", op="weigh", B=64, Hq=32, Hkv=8, d=128, page=16, new=1, new_hi=1,
             ctx=200, ctx_hi=8191, lens=9, causal=True, held8=True, dtype="bf16"),
        # after long prompts: the weight that their last 33 tokens give, 16-bit cache, d = 64
        dict(name="weigh the last tokens of prompts", op="weigh", B=5, Hq=12, Hkv=12, d=64, page=64, new=33,
             new_hi=33, ctx=4000, ctx_hi=16000, lens=10, causal=True, held8=False, dtype="fp16"),
        # all tokens of a chunk of a long prompt: arithmetic
        dict(name="weigh a chunk", op="weigh", B=1, Hq=16, Hkv=2, d=128, page=64, new=2048, new_hi=2048,
             ctx=30720, ctx_hi=30720, lens=6, causal=True, held8=True, dtype="bf16"),
        # one conversation that has outgrown its budget: latency
        dict(name="evict from one sequence", op="evict", B=1, Hkv=8, d=128, page=16, ctx=1500, ctx_hi=1500, lens=11,
             budget=1024, recent=100, held8=True, dtype="bf16"),
        # long documents cut by half, 8-bit cache
        dict(name="evict from long contexts", op="evict", B=8, Hkv=8, d=128, page=16, ctx=30000, ctx_hi=32768,
             lens=12, budget=16384, recent=1000, held8=True, dtype="bf16"),
        # a ragged batch, some within the budget already, 16-bit cache, d = 64
        dict(name="evict from a ragged batch", op="evict", B=33, Hkv=12, d=64, page=64, ctx=1, ctx_hi=5000, lens=13,
             budget=777, recent=128, held8=False, dtype="fp16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "weigh", "weigh", "evict"])
    d = rng.choice([64, 128])
    Hkv, page = rng.choice([1, 2, 3, 4, 8]), rng.choice([16, 32, 64, 128, 256])
    case = dict(op=op, d=d, Hkv=Hkv, page=page, lens=rng.randint(0, 1 << 20), dtype=rng.choice(["bf16", "fp16"]))
    if op == "append":
        B = _log_int(rng, 1, 128)
        hi = _log_int(rng, 1, max(1, 32768 // B))
        case.update(B=B, new=rng.randint(0, hi), new_hi=hi, ctx=0, ctx_hi=_log_int(rng, 1, 8192),
                    rot=rng.choice([d, d // 2, 16]), interleaved=rng.random() < 0.5)
        return case
    if op == "evict":
        B = _log_int(rng, 1, 128)
        ctx_hi = _log_int(rng, 1, max(2, min(32768, 2_000_000 // (B * Hkv))))
        budget = _log_int(rng, 1, max(1, ctx_hi * 3 // 4))
        case.update(B=B, ctx=rng.randint(0, ctx_hi), ctx_hi=ctx_hi, budget=budget, recent=rng.randint(0, budget),
                    held8=rng.random() < 0.6)
        return case
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    if rng.random() < 0.5:  # single tokens and drafts
        B = _log_int(rng, 1, 128)
        new, new_hi = rng.choice([(1, 1), (1, 1), (0, 3), (1, 8)])
        longest = max(2, min(32768, 2_000_000 // (B * Hkv)))
    else:  # chunks
        B = rng.randint(1, 4)
        new_hi = _log_int(rng, 9, 1024)
        new = rng.randint(1, new_hi)
        longest = max(2, min(16384, 400_000_000 // (B * Hq * new_hi)))
    ctx_hi = _log_int(rng, 1, longest)
    case.update(B=B, Hq=Hq, new=new, new_hi=new_hi, ctx=rng.randint(0, ctx_hi), ctx_hi=ctx_hi,
                causal=rng.random() < 0.8)
    if op == "weigh":
        case.update(held8=rng.random() < 0.6)
    return case


def _lengths(case):
    """New tokens and cached tokens of each sequence: the case's alone, the same for every seed."""
    r = random.Random(case["lens"])
    new = [r.randint(case["new"], case["new_hi"]) if "new" in case else 0 for _ in range(case["B"])]
    ctx = [r.randint(case["ctx"], case["ctx_hi"]) for _ in range(case["B"])]
    if "new" in case and sum(new) == 0:
        new[0] = 1
    if "new" not in case and sum(ctx) == 0:
        ctx[0] = 1
    return new, ctx


def work(case):
    d, Hkv = case["d"], case["Hkv"]
    new, ctx = _lengths(case)
    total = [n + c for n, c in zip(new, ctx)]
    wide = 1 if case.get("held8", True) else 2  # bytes of a cached element
    pages = sum(-(-t // case["page"]) for t in total)
    if case["op"] == "append":
        pages = sum(-(-t // case["page"]) - c // case["page"] for c, t in zip(ctx, total))
    scales = pages * Hkv * (4 if wide == 1 else 0)
    if case["op"] == "append":
        rows = sum(new) * Hkv
        return {"bytes": 2 * rows * d * 3 + sum(new) * case["rot"] * 4 + 2 * scales, "flops": rows * d * 8}
    if case["op"] == "evict":
        cut = [t for t in total if t > case["budget"]]
        moved = len(cut) * case["budget"] * Hkv
        kept = case["B"] * Hkv * case["budget"]
        return {"bytes": sum(cut) * Hkv * 4 + 4 * moved * d * wide + 4 * moved + 4 * kept, "flops": 4 * sum(cut) * Hkv}
    pairs = sum(n * c + n * (n + 1) // 2 if case["causal"] else n * t for n, c, t in zip(new, ctx, total))
    keys = sum(t for n, t in zip(new, total) if n)
    rows = sum(new) * case["Hq"]
    if case["op"] == "weigh":
        return {"bytes": keys * Hkv * (d * wide + 8) + rows * (2 * d + 4) + scales, "flops": 2 * pairs * case["Hq"] * d}
    return {"bytes": 2 * keys * Hkv * d + 2 * rows * d * 2 + 4 * rows + 2 * scales, "flops": 4 * pairs * case["Hq"] * d}


# ------------------------------------------------------------------------------------- inputs
def _table(length, rot, device):
    """cos then sin of each position's rot/2 angles, 32 bits from angles in 64."""
    inv = BASE ** (-torch.arange(0, rot, 2, device=device, dtype=torch.float64) / rot)
    angle = torch.arange(length, device=device, dtype=torch.float64)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], dim=1).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dtype, d, Hkv, page = TYPES[case["dtype"]], case["d"], case["Hkv"], case["page"]
    eight = case["op"] in ("attend", "append") or case["held8"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=dtype)

    s = {"case": case}
    new, ctx = _lengths(case)
    total = [n + c for n, c in zip(new, ctx)]
    held = [-(-t // page) for t in total]
    wide, pages = max(1, max(held)), sum(held) + 3
    order = torch.randperm(pages, generator=g, device=dev).int()
    # sequence b's pages are the next of a random order; the table's unused entries are 0
    starts = torch.tensor([sum(held[:b]) for b in range(len(held))], device=dev)
    at = torch.arange(wide, device=dev)
    inside = at[None, :] < torch.tensor(held, device=dev)[:, None]
    s["block_table"] = torch.where(inside, order[(starts[:, None] + at).clamp(max=pages - 1)], 0).int().contiguous()
    s["cu_seqlens"] = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], device=dev, dtype=torch.int32)
    s["seq_lens"] = torch.tensor(total, device=dev, dtype=torch.int32)
    s["max_q"], s["T"] = max(1, max(new)), sum(new)
    for name in ("k", "v"):
        x = normal(pages, Hkv, page, d)
        if eight:  # pages whose values differ in size, as those of different tokens do
            x = x.float() * (0.5 * torch.randn(pages, Hkv, 1, 1, generator=g, device=dev)).exp()
            scale = _power(x.abs().amax((2, 3)) / MOST)
            s[name + "_scale"] = scale.contiguous()
            x = (x / scale[..., None, None]).to(torch.float8_e4m3fn)
        s[name + "_pages"] = x.contiguous()
    if case["op"] == "append":
        rows = normal(s["T"], 3 * Hkv * d)  # the fused projection's output
        s["k"] = rows[:, Hkv * d:2 * Hkv * d].unflatten(-1, (Hkv, d))
        s["v"] = rows[:, 2 * Hkv * d:].unflatten(-1, (Hkv, d))
        s["rope"] = _table(max(total), case["rot"], dev)
        return s
    if case["op"] != "attend":  # what earlier tokens gave: few large weights, some none at all
        w = torch.randn(pages, Hkv, page, generator=g, device=dev).mul(2).exp()
        s["weights"] = w * (torch.rand(pages, Hkv, page, generator=g, device=dev) > 0.05)
    if case["op"] != "evict":
        s["q"] = normal(s["T"], case["Hq"], d)
    if case["op"] == "weigh":
        s["lse"] = _padded(s, False)[0]
    return s


# ----------------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    return {"attend": _attend, "append": _append, "weigh": _weigh, "evict": _evict}[op](s)


def _own(s, op):
    import exact_attention_forward_02_gb300 as fa

    c = s["case"]
    if op == "append":
        fa.paged_append_fp8(s["k"], s["v"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["block_table"],
                            s["cu_seqlens"], s["seq_lens"], rope=s["rope"], interleaved=c["interleaved"])
        return s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]
    if op == "attend":
        return fa.attention_paged_fp8(s["q"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"],
                                      s["block_table"], s["cu_seqlens"], s["seq_lens"], s["max_q"],
                                      causal=c["causal"])
    if op == "weigh":
        fa.paged_key_weights(s["q"], s["lse"], s["k_pages"], s["weights"], s["block_table"], s["cu_seqlens"],
                             s["seq_lens"], s["max_q"], causal=c["causal"], k_scale=s.get("k_scale"))
        return s["weights"]
    kept, lens = fa.paged_evict(s["k_pages"], s["v_pages"], s["weights"], s["block_table"], s["seq_lens"],
                                c["budget"], c["recent"], k_scale=s.get("k_scale"), v_scale=s.get("v_scale"))
    return kept, lens, s["weights"], s["k_pages"], s["v_pages"], s.get("k_scale"), s.get("v_scale")


def _power(x):
    """The smallest power of two that is not below x (and not below LEAST_SCALE)."""
    mantissa, exponent = torch.frexp(x.clamp(min=LEAST_SCALE))  # mantissa in [1/2, 1)
    return torch.ldexp(torch.ones_like(x), exponent - (mantissa == 0.5).int())


def _bytes(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _values(x, scale):
    """A cache's values in 32 bits."""
    return x.float() if scale is None else x.float() * scale[..., None, None]


def _rows(s):
    """The sequence and the position in it of each of the T new tokens."""
    cu, lens = s["cu_seqlens"].long(), s["seq_lens"].long()
    t = torch.arange(s["T"], device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    return b, t - cu[b], lens[b] - cu[b + 1] + t


def _padded(s, values):
    """L of every row of q, and the weights exp(score - L) of its keys, [B, Hkv, Hq / Hkv, max_q, keys],
    or with `values` the rows' outputs."""
    c, q = s["case"], s["q"]
    T, Hq, d = q.shape
    Hkv, page = c["Hkv"], c["page"]
    table, lens = s["block_table"].long(), s["seq_lens"].long()
    B, wide = table.shape
    b, i, pos = _rows(s)
    # queries padded to [B, max_q, Hq, d], keys and values of every page in order, 32 bits
    padded = torch.zeros(B, s["max_q"], Hq, d, device=q.device)
    padded[b, i] = q.float()
    last = torch.full((B, s["max_q"]), -1, device=q.device)
    last[b, i] = pos if c["causal"] else lens[b] - 1
    padded = padded.view(B, s["max_q"], Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, d)
    keys = _values(s["k_pages"], s.get("k_scale"))[table].permute(0, 2, 1, 3, 4).reshape(B, Hkv, wide * page, d)
    scores = torch.matmul(padded, keys.transpose(2, 3)) * (1.0 / math.sqrt(d))
    scores = scores.view(B, Hkv, Hq // Hkv, s["max_q"], wide * page)
    seen = torch.arange(wide * page, device=q.device) <= last[:, None, None, :, None]
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    weight = torch.exp(scores - top)
    total = weight.sum(-1, keepdim=True)
    lse = (top + total.log()).permute(0, 3, 1, 2, 4).reshape(B, s["max_q"], Hq)[b, i]
    if not values:
        return lse.contiguous(), scores, seen
    held = _values(s["v_pages"], s.get("v_scale"))[table].permute(0, 2, 1, 3, 4).reshape(B, Hkv, wide * page, d)
    out = torch.matmul(weight.view(B, Hkv, -1, wide * page), held).view(B, Hkv, Hq // Hkv, s["max_q"], d)
    out = torch.where(total > 0, out / total, 0.0).permute(0, 3, 1, 2, 4).reshape(B, s["max_q"], Hq, d)
    return out[b, i].to(q.dtype), lse


def _attend(s):
    return _padded(s, True)


def _weigh(s):
    c, q = s["case"], s["q"]
    Hkv, page = c["Hkv"], c["page"]
    table, lens, cu = s["block_table"].long(), s["seq_lens"].long(), s["cu_seqlens"].long()
    B, wide = table.shape
    b, i, _ = _rows(s)
    _, scores, seen = _padded(s, False)
    lse = torch.full((B, s["max_q"], q.shape[1]), math.inf, device=q.device)
    lse[b, i] = s["lse"]
    lse = lse.view(B, s["max_q"], Hkv, -1).permute(0, 2, 3, 1)[..., None]
    gained = torch.where(seen, torch.exp(scores - lse), 0.0).sum((2, 3)).view(B, Hkv, wide, page)
    at = torch.arange(wide * page, device=q.device).view(wide, page)
    new = (cu[1:] - cu[:-1])[:, None, None, None]
    first = lens[:, None, None, None] - new
    before = torch.where(at < first, s["weights"][table].transpose(1, 2), 0.0)
    held = (at < lens[:, None, None, None]) & (new > 0)
    to_b, to_h, to_p, to_s = torch.nonzero(held.expand(B, Hkv, wide, page), as_tuple=True)
    s["weights"][table[to_b, to_p], to_h, to_s] = (before + gained)[to_b, to_h, to_p, to_s]
    return s["weights"]


def _turn(x, cos, sin, interleaved):
    """Rotates the first rot elements of the last axis of x; cos and sin: [..., rot/2]."""
    half = cos.shape[-1]
    head, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = head[..., :half], head[..., half:]
        head = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([head, rest], dim=-1)


def _append(s):
    c, table, page = s["case"], s["block_table"].long(), s["case"]["page"]
    b, _, pos = _rows(s)
    first = (s["seq_lens"] - s["cu_seqlens"][1:] + s["cu_seqlens"][:-1]).long()
    at, slot = table[b, pos // page], pos % page
    cos, sin = s["rope"][pos][:, None, :].chunk(2, dim=-1)
    # a page's first new slot: all before it is kept, in the page's scale
    held = torch.full((s["k_pages"].shape[0],), page, device=table.device)
    held[at] = torch.where(pos // page == first[b] // page, first[b] % page, 0)
    for name, x in (("k", _turn(s["k"].float(), cos, sin, c["interleaved"])), ("v", s["v"].float())):
        pages, scale = s[name + "_pages"], s[name + "_scale"]
        top = torch.zeros_like(scale).index_reduce_(0, at, x.abs().amax(-1), "amax")
        wanted = _power(top / MOST)
        now = torch.where(held[:, None] == 0, wanted, torch.where(held[:, None] < page, torch.maximum(scale, wanted), scale))
        # codes held under a smaller scale are rounded anew
        grown = torch.nonzero((now > scale) & (held[:, None] > 0), as_tuple=True)
        old = _bytes(pages)[grown].view(torch.float8_e4m3fn)
        again = (old.float() * (scale[grown] / now[grown])[:, None, None]).to(torch.float8_e4m3fn)
        keep = torch.arange(page, device=table.device)[None, :, None] < held[grown[0]][:, None, None]
        _bytes(pages)[grown] = torch.where(keep, _bytes(again), _bytes(old))
        _bytes(pages)[at, :, slot] = _bytes((x / now[at][..., None]).to(torch.float8_e4m3fn))
        scale.copy_(now)
    return s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]


def _evict(s):
    c, page, budget, recent = s["case"], s["case"]["page"], s["case"]["budget"], s["case"]["recent"]
    table, lens, Hkv = s["block_table"].long(), s["seq_lens"].long(), s["case"]["Hkv"]
    B, wide = table.shape
    at = torch.arange(wide * page, device=table.device)
    w = s["weights"][table].transpose(1, 2).reshape(B, Hkv, wide * page)
    length = lens[:, None, None]
    score = torch.where(at < length - recent, w, torch.where(at < length, math.inf, -math.inf))
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, at.expand_as(order).contiguous())
    cut = (length > budget).expand(B, Hkv, 1)
    stays = (at < length) & (~cut | (rank < budget))
    place = torch.where(stays & (stays.cumsum(-1) <= budget), stays.cumsum(-1) - 1, budget)
    kept = torch.full((B, Hkv, budget + 1), -1, device=table.device, dtype=torch.long)
    kept = kept.scatter_(-1, place, at.expand(B, Hkv, -1).contiguous())[..., :budget].contiguous()
    # the rows that move: [entries] of sequence, head, place
    b, h, to = torch.nonzero((kept >= 0) & cut, as_tuple=True)
    from_at = kept[b, h, to]
    from_page, from_slot = table[b, from_at // page], from_at % page
    to_page, to_slot = table[b, to // page], to % page
    s["weights"][to_page, h, to_slot] = s["weights"][from_page, h, from_slot]
    for name in ("k", "v"):
        pages, scale = s[name + "_pages"], s.get(name + "_scale")
        rows = _bytes(pages)[from_page, h, from_slot]
        if scale is not None:  # a page's scale becomes the largest of those that its rows came from
            came = scale[from_page, h]
            flat = torch.zeros(scale.numel(), device=scale.device).index_reduce_(0, to_page * Hkv + h, came, "amax")
            ratio = came / flat[to_page * Hkv + h]
            rows = _bytes((rows.view(torch.float8_e4m3fn).float() * ratio[:, None]).to(torch.float8_e4m3fn))
            scale.copy_(torch.where(flat > 0, flat, scale.flatten()).view_as(scale))
        _bytes(pages)[to_page, h, to_slot] = rows
    return (kept.int(), torch.minimum(lens, torch.tensor(budget, device=lens.device)).int(), s["weights"],
            s["k_pages"], s["v_pages"], s.get("k_scale"), s.get("v_scale"))


# --------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The operators' definitions in 64 bits, sequence by sequence and head by head."""
    if case["op"] == "evict":
        if sum(_lengths(case)[1]) * case["Hkv"] > 3_000_000:
            return None
    s = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "weigh": _exact_weigh, "evict": _exact_evict}[case["op"]](s)


def _sequence(s, name, b, length):
    """The first `length` rows of sequence b's keys or values, [Hkv, length, d] in 64 bits."""
    used = s["block_table"][b, :-(-length // s["case"]["page"])].long()
    x = _bytes(s[name + "_pages"])[used]
    if name + "_scale" in s:
        x = x.view(torch.float8_e4m3fn).double() * s[name + "_scale"][used].double()[..., None, None]
    return x.double().transpose(0, 1).flatten(1, 2)[:, :length]


def _scores(s, b, q, n, before, h, k):
    c = s["case"]
    x = q[:, h].double() @ k[h * c["Hkv"] // c["Hq"]].T / math.sqrt(c["d"])
    if c["causal"]:
        x += torch.full_like(x, -math.inf).triu(before + 1)
    return x


def _exact_attend(s):
    c = s["case"]
    out, lse, t0 = [], [], 0
    for b, (n, before) in enumerate(zip(*_lengths(c))):
        q = s["q"][t0:t0 + n]
        t0 += n
        o = torch.empty(n, c["Hq"], c["d"], device=q.device, dtype=torch.float64)
        m = torch.empty(n, c["Hq"], device=q.device, dtype=torch.float64)
        if n:
            k, v = _sequence(s, "k", b, n + before), _sequence(s, "v", b, n + before)
        for h in range(c["Hq"] if n else 0):
            x = _scores(s, b, q, n, before, h, k)
            m[:, h] = torch.logsumexp(x, -1)
            o[:, h] = torch.exp(x - m[:, h, None]) @ v[h * c["Hkv"] // c["Hq"]]
        out.append(o)
        lse.append(m)
    return torch.cat(out), torch.cat(lse)


def _exact_weigh(s):
    c, page = s["case"], s["case"]["page"]
    weights, t0 = s["weights"].double(), 0
    for b, (n, before) in enumerate(zip(*_lengths(c))):
        if not n:
            continue
        q, length = s["q"][t0:t0 + n], n + before
        k = _sequence(s, "k", b, length)
        gained = torch.zeros(c["Hkv"], length, device=k.device, dtype=torch.float64)
        for h in range(c["Hq"]):
            x = _scores(s, b, q, n, before, h, k)
            gained[h * c["Hkv"] // c["Hq"]] += torch.exp(x - s["lse"][t0:t0 + n, h, None].double()).sum(0)
        t0 += n
        pos = torch.arange(length, device=k.device)
        where, slot = s["block_table"][b].long()[pos // page], pos % page
        old = weights[where, :, slot] * (pos < before)[:, None]
        weights[where, :, slot] = old + gained.T
    return weights


def _round8(x):
    """x (at most 448 in size) rounded to the nearest E4M3 number, ties to an even last bit."""
    step = torch.exp2(torch.frexp(x.abs().clamp(min=2.0 ** -6))[1].double() - 4)
    return torch.round(x / step) * step


def _power64(x):
    p = torch.exp2(torch.ceil(torch.log2(x.clamp(min=LEAST_SCALE))))
    p = torch.where(p / 2 >= x, p / 2, p)  # a logarithm that came out a little high, or low
    return torch.where(p < x, p * 2, p).clamp(min=LEAST_SCALE)


def _exact_append(s):
    c, page = s["case"], s["case"]["page"]
    half, t = c["rot"] // 2, 0
    out = {name: (s[name + "_pages"].double(), s[name + "_scale"].double()) for name in ("k", "v")}
    for b, (n, before) in enumerate(zip(*_lengths(c))):
        if not n:
            continue
        at = s["rope"][before:before + n].double()[:, None, :]
        turn = torch.complex(at[..., :half].contiguous(), at[..., half:].contiguous())
        k, v = s["k"][t:t + n].double(), s["v"][t:t + n].double()
        t += n
        first = slice(0, c["rot"], 2) if c["interleaved"] else slice(0, half)
        second = slice(1, c["rot"], 2) if c["interleaved"] else slice(half, c["rot"])
        z = torch.complex(k[..., first].contiguous(), k[..., second].contiguous()) * turn
        k[..., first], k[..., second] = z.real, z.imag
        for name, x in (("k", k), ("v", v)):
            pages, scale = out[name]
            # whole pages of rows: zeros stand for the slots before the first new one and behind the last
            lead, tail = before % page, -(before + n) % page
            x = torch.nn.functional.pad(x, (0, 0, 0, 0, lead, tail)).unflatten(0, (-1, page)).transpose(1, 2)
            used = s["block_table"][b, before // page:before // page + x.shape[0]].long()
            now = _power64(x.abs().amax((2, 3)) / MOST)
            if lead:
                now[0] = torch.maximum(now[0], scale[used[0]])
            old = pages[used[0], :, :lead] * (scale[used[0]] / now[0])[:, None, None]
            pos = torch.arange(lead, lead + n, device=x.device)
            pages[used[pos // page], :, pos % page] = _round8(x / now[..., None, None])[pos // page, :, pos % page]
            pages[used[0], :, :lead] = _round8(old)
            scale[used] = now
    return out["k"][0], out["v"][0], out["k"][1], out["v"][1]


def _exact_evict(s):
    c, page, budget = s["case"], s["case"]["page"], s["case"]["budget"]
    weights = s["weights"].double()
    caches = [s[n + "_pages"].double() for n in ("k", "v")]
    scales = [s[n + "_scale"].double() if n + "_scale" in s else None for n in ("k", "v")]
    kept = torch.full((c["B"], c["Hkv"], budget), -1, dtype=torch.int32, device=weights.device)
    lens = s["seq_lens"].clone()
    for b, length in enumerate(s["seq_lens"].tolist()):
        pos = torch.arange(length, device=weights.device)
        if length <= budget:
            kept[b, :, :length] = pos.int()
            continue
        lens[b] = budget
        where, slot = s["block_table"][b].long()[pos // page], pos % page
        old = weights[where, :, slot]  # [length, Hkv]
        to = torch.arange(budget, device=weights.device)
        for h in range(c["Hkv"]):
            early = old[:length - c["recent"], h]
            need = budget - c["recent"]
            stays = torch.ones(length, dtype=torch.bool, device=weights.device)
            if need < early.numel():
                border = torch.topk(early, need).values[-1] if need else torch.tensor(math.inf, device=early.device)
                above, same = early > border, early == border
                stays[:early.numel()] = above | (same & (same.cumsum(0) <= need - above.sum()))
            src = torch.nonzero(stays).flatten()
            kept[b, h] = src.int()
            weights[where[to], h, slot[to]] = old[src, h]
            for i, cache in enumerate(caches):
                rows = cache[where[src], h, slot[src]]
                if scales[i] is not None:
                    came = scales[i][where[src], h]
                    groups = torch.nn.functional.pad(came, (0, -budget % page)).view(-1, page).amax(1)
                    rows = _round8(rows * (came / groups[to // page])[:, None])
                    scales[i][where[to[::page]], h] = groups
                cache[where[to], h, slot[to]] = rows
    return (kept, lens, weights, *caches, *scales)
