"""The serving and position operators of this package, as cases that can be measured.

Four paths of a decoder block around the attention kernels, each on the inputs that a user's
program has in hand:

  attend       attention of new tokens (a chunk of a prompt, or one token of each sequence) over
               a paged cache of keys and values
  append       new keys and values into the paged cache, the keys rotated by position on the way
  rotate       RMS norm of every query and key head and the position rotation, one pass
  rotate_grad  the gradients of that pass, those of the norm weights among them

`own = False` computes them in elementary torch operations in 32 bits; `own = True` calls the
package's operators on the same state.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6
BASE = 10000.0


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one user's next token, a short conversation: latency alone
        dict(name="decode one sequence", op="attend", B=1, Hq=32, Hkv=8, d=128, page=16, new=1, new_hi=1,
             ctx=1000, ctx_hi=1000, lens=1, causal=True, dtype="bf16"),
        # a server's batch of ragged conversations, one token each, small pages
        dict(name="decode ragged batch", op="attend", B=64, Hq=32, Hkv=8, d=128, page=16, new=1, new_hi=1,
             ctx=200, ctx_hi=8191, lens=2, causal=True, dtype="bf16"),
        # few long documents, one token each: the cache is read once, at full memory speed
        dict(name="decode long contexts", op="attend", B=8, Hq=16, Hkv=8, d=128, page=128, new=1, new_hi=1,
             ctx=30000, ctx_hi=32768, lens=3, causal=True, dtype="fp16"),
        # drafts of a few tokens to check, d = 64, every query head with its own keys
        dict(name="decode drafts d64", op="attend", B=24, Hq=12, Hkv=12, d=64, page=64, new=2, new_hi=7,
             ctx=1, ctx_hi=4097, lens=4, causal=True, dtype="fp16"),
        # prompts of 1000 queries against an encoder's 4097 states, no mask
        dict(name="cross attention d64", op="attend", B=4, Hq=12, Hkv=12, d=64, page=32, new=1000, new_hi=1000,
             ctx=3097, ctx_hi=3097, lens=5, causal=False, dtype="fp16"),
        # a chunk of a long prompt over what the cache holds of it
        dict(name="chunk of a long prompt", op="attend", B=1, Hq=16, Hkv=2, d=128, page=64, new=2048, new_hi=2048,
             ctx=30720, ctx_hi=30720, lens=6, causal=True, dtype="bf16"),
        # one token of each of 64 sequences into the cache
        dict(name="append one token each", op="append", B=64, Hkv=8, d=128, page=16, new=1, new_hi=1,
             ctx=0, ctx_hi=8191, lens=7, rot=128, interleaved=False, dtype="bf16"),
        # ragged prompt chunks into the cache, half of each head rotated
        dict(name="append ragged chunks", op="append", B=9, Hkv=8, d=128, page=64, new=1, new_hi=8192,
             ctx=0, ctx_hi=5000, lens=8, rot=64, interleaved=True, dtype="fp16"),
        # the heads of a decoding batch, from the fused projection's rows
        dict(name="rotate decoding batch", op="rotate", B=1, N=64, Hq=32, Hkv=8, d=128, rot=128,
             interleaved=False, dtype="bf16"),
        # the heads of a training batch of two sequences of 8192
        dict(name="rotate training batch", op="rotate", B=2, N=8192, Hq=32, Hkv=8, d=128, rot=128,
             interleaved=False, dtype="bf16"),
        # the same batch's gradients
        dict(name="rotate gradients", op="rotate_grad", B=2, N=8192, Hq=32, Hkv=8, d=128, rot=128,
             interleaved=False, dtype="bf16"),
        # gradients of a small odd batch, d = 64, interleaved pairs
        dict(name="rotate gradients d64", op="rotate_grad", B=3, N=333, Hq=12, Hkv=12, d=64, rot=32,
             interleaved=True, dtype="fp16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "rotate", "rotate_grad"])
    d = rng.choice([64, 128])
    case = dict(op=op, d=d, dtype=rng.choice(["bf16", "fp16"]))
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    if op in ("rotate", "rotate_grad"):
        B, Hkv = rng.randint(1, 4), rng.choice([1, 2, 3, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 3, 4])
        N = _log_int(rng, 1, max(2, 16384 // B))
        case.update(B=B, N=N, Hq=Hq, Hkv=Hkv, rot=rng.choice([d, d, d // 2, 16]), interleaved=rng.random() < 0.5)
        return case
    page = rng.choice([16, 32, 64, 128, 256])
    case.update(Hkv=Hkv, page=page, lens=rng.randint(0, 1 << 20))
    if op == "append":
        B = _log_int(rng, 1, 128)
        hi = _log_int(rng, 1, max(1, 32768 // B))
        case.update(B=B, new=rng.randint(0, hi), new_hi=hi, ctx=0, ctx_hi=_log_int(rng, 1, 8192),
                    rot=rng.choice([d, d // 2, 16]), interleaved=rng.random() < 0.5)
        return case
    Hq = Hkv * group
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
    return case


def _lengths(case):
    """New tokens and cached tokens of each sequence: the case's alone, the same for every seed."""
    r = random.Random(case["lens"])
    new = [r.randint(case["new"], case["new_hi"]) for _ in range(case["B"])]
    ctx = [r.randint(case["ctx"], case["ctx_hi"]) for _ in range(case["B"])]
    if sum(new) == 0:
        new[0] = 1
    return new, ctx


def work(case):
    d, Hkv = case["d"], case["Hkv"]
    if case["op"] in ("rotate", "rotate_grad"):
        rows = case["B"] * case["N"] * (case["Hq"] + Hkv)
        tensors = 3 if case["op"] == "rotate_grad" else 2
        table = case["B"] * case["N"] * case["rot"] * 4
        return {"bytes": tensors * rows * d * 2 + table, "flops": rows * d * (16 if tensors == 3 else 8)}
    new, ctx = _lengths(case)
    if case["op"] == "append":
        rows = sum(new) * Hkv
        return {"bytes": 4 * rows * d * 2 + sum(new) * case["rot"] * 4, "flops": rows * case["rot"] * 3}
    total = [n + c for n, c in zip(new, ctx)]
    pairs = sum(n * c + n * (n + 1) // 2 if case["causal"] else n * t for n, c, t in zip(new, ctx, total))
    keys = sum(t for n, t in zip(new, total) if n)
    return {"bytes": (2 * keys * Hkv * d + 2 * sum(new) * case["Hq"] * d) * 2 + 4 * sum(new) * case["Hq"],
            "flops": 4 * pairs * case["Hq"] * d}


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
    dtype, d, Hkv = TYPES[case["dtype"]], case["d"], case["Hkv"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=dtype)

    s = {"case": case}
    if case["op"] in ("rotate", "rotate_grad"):
        B, N, Hq = case["B"], case["N"], case["Hq"]
        rows = normal(B, N, (Hq + 2 * Hkv) * d)  # the fused projection's output
        s["q"] = rows[..., :Hq * d].unflatten(-1, (Hq, d))
        s["k"] = rows[..., Hq * d:(Hq + Hkv) * d].unflatten(-1, (Hkv, d))
        s["wq"], s["wk"] = 1 + 0.1 * normal(d), 1 + 0.1 * normal(d)
        s["rope"] = _table(N + 1000, case["rot"], dev)
        first = torch.randint(0, 1000, (B, 1), generator=g, device=dev)
        s["positions"] = (first + torch.arange(N, device=dev)).int()
        if case["op"] == "rotate_grad":
            s["dq"], s["dk"] = normal(B, N, Hq, d), normal(B, N, Hkv, d)
        return s
    new, ctx = _lengths(case)
    page = case["page"]
    total = [n + c for n, c in zip(new, ctx)]
    wide = max(1, max(-(-t // page) for t in total))
    pages = sum(-(-t // page) for t in total) + 3
    order = torch.randperm(pages, generator=g, device=dev).int()
    # sequence b's pages are the next of a random order; the table's unused entries are 0
    starts = torch.tensor([sum(-(-t // page) for t in total[:b]) for b in range(len(total))], device=dev)
    held = torch.tensor([-(-t // page) for t in total], device=dev)
    at = torch.arange(wide, device=dev)
    inside = at[None, :] < held[:, None]
    s["block_table"] = torch.where(inside, order[(starts[:, None] + at).clamp(max=pages - 1)], 0).int().contiguous()
    s["cu_seqlens"] = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], device=dev, dtype=torch.int32)
    s["seq_lens"] = torch.tensor(total, device=dev, dtype=torch.int32)
    s["max_q"], s["T"] = max(new), sum(new)
    s["k_pages"], s["v_pages"] = normal(pages, Hkv, page, d), normal(pages, Hkv, page, d)
    if case["op"] == "append":
        rows = normal(s["T"], 3 * Hkv * d)
        s["k"] = rows[:, Hkv * d:2 * Hkv * d].unflatten(-1, (Hkv, d))
        s["v"] = rows[:, 2 * Hkv * d:].unflatten(-1, (Hkv, d))
        s["rope"] = _table(max(total), case["rot"], dev)
    else:
        s["q"] = normal(s["T"], case["Hq"], d)
    return s


# ----------------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    if op == "attend":
        return _attend(s)
    if op == "append":
        return _append(s)
    return _rotate(s) if op == "rotate" else _rotate_grad(s)


def _own(s, op):
    import exact_attention_forward_02_gb300 as fa

    c = s["case"]
    if op == "attend":
        return fa.attention_paged(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["cu_seqlens"],
                                  s["seq_lens"], s["max_q"], causal=c["causal"])
    if op == "append":
        fa.paged_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["block_table"], s["cu_seqlens"],
                        s["seq_lens"], rope=s["rope"], interleaved=c["interleaved"])
        return s["k_pages"], s["v_pages"]
    if op == "rotate":
        return fa.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["rope"], positions=s["positions"], eps=EPS,
                               interleaved=c["interleaved"])
    return fa.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], s["rope"],
                                    positions=s["positions"], eps=EPS, interleaved=c["interleaved"])


def _rows(s):
    """The sequence and the position in it of each of the T new tokens."""
    cu, lens = s["cu_seqlens"].long(), s["seq_lens"].long()
    t = torch.arange(s["T"], device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    return b, t - cu[b], lens[b] - cu[b + 1] + t


def _attend(s):
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
    keys = s["k_pages"][table].permute(0, 2, 1, 3, 4).reshape(B, Hkv, wide * page, d).float()
    values = s["v_pages"][table].permute(0, 2, 1, 3, 4).reshape(B, Hkv, wide * page, d).float()
    scores = torch.matmul(padded, keys.transpose(2, 3)) * (1.0 / math.sqrt(d))
    scores = scores.view(B, Hkv, Hq // Hkv, s["max_q"], wide * page)
    seen = torch.arange(wide * page, device=q.device) <= last[:, None, None, :, None]
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    weight = torch.exp(scores - top)
    total = weight.sum(-1, keepdim=True)
    out = torch.matmul(weight.view(B, Hkv, -1, wide * page), values).view(B, Hkv, Hq // Hkv, s["max_q"], d)
    out = torch.where(total > 0, out / total, 0.0).permute(0, 3, 1, 2, 4).reshape(B, s["max_q"], Hq, d)
    lse = (top + total.log()).permute(0, 3, 1, 2, 4).reshape(B, s["max_q"], Hq)
    return out[b, i].to(q.dtype), lse[b, i]


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
    c, table = s["case"], s["block_table"].long()
    b, _, pos = _rows(s)
    cos, sin = s["rope"][pos][:, None, :].chunk(2, dim=-1)
    at, slot = table[b, pos // c["page"]], pos % c["page"]
    s["k_pages"][at, :, slot] = _turn(s["k"].float(), cos, sin, c["interleaved"]).to(s["k"].dtype)
    s["v_pages"][at, :, slot] = s["v"]
    return s["k_pages"], s["v_pages"]


def _rotate(s):
    cos, sin = s["rope"][s["positions"].long()][:, :, None, :].chunk(2, dim=-1)
    turned = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        y = x.float()
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.float()
        turned.append(_turn(y, cos, sin, s["case"]["interleaved"]).to(x.dtype))
    return tuple(turned)


def _rotate_grad(s):
    cos, sin = s["rope"][s["positions"].long()][:, :, None, :].chunk(2, dim=-1)
    grads, weights = [], []
    for g, x, w in ((s["dq"], s["q"], s["wq"]), (s["dk"], s["k"], s["wk"])):
        y = x.float()
        r = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
        y = y * r
        g = _turn(g.float(), cos, -sin, s["case"]["interleaved"])  # the rotation's transpose
        weights.append((g * y).sum((0, 1, 2)))
        g = g * w.float()
        grads.append((r * (g - y * (g * y).mean(-1, keepdim=True))).to(x.dtype))
    return (*grads, *weights)


# --------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The operators' definitions in 64 bits, sequence by sequence and pair by pair."""
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(s)
    if case["op"] == "append":
        return _exact_append(s)
    half = case["rot"] // 2
    at = s["rope"].double()[s["positions"].long()][:, :, None, :]
    turn = torch.complex(at[..., :half].contiguous(), at[..., half:].contiguous())
    out = []
    for name in ("q", "k"):
        x, w = s[name].double(), s["w" + name].double()
        norm = (x.pow(2).sum(-1, keepdim=True) / case["d"] + EPS).sqrt()
        if case["op"] == "rotate":
            out.append(_exact_turn(x / norm * w, turn, case))
            continue
        g = _exact_turn(s["d" + name].double(), turn.conj(), case)
        unit = x / norm
        inner = (g * w * unit).sum(-1, keepdim=True) / case["d"]
        out.append(((g * w - unit * inner) / norm, torch.einsum("bnhd,bnhd->d", g, unit)))
    return tuple(out) if case["op"] == "rotate" else (out[0][0], out[1][0], out[0][1], out[1][1])


def _exact_turn(x, turn, case):
    """Pairs of elements as complex numbers, times turn."""
    half = case["rot"] // 2
    first = slice(0, case["rot"], 2) if case["interleaved"] else slice(0, half)
    second = slice(1, case["rot"], 2) if case["interleaved"] else slice(half, case["rot"])
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_attend(s):
    c = s["case"]
    new, ctx = _lengths(c)
    out, lse, t0 = [], [], 0
    for b, (n, before) in enumerate(zip(new, ctx)):
        length = n + before
        used = s["block_table"][b, :-(-length // c["page"])].long()
        k = s["k_pages"][used].transpose(0, 1).flatten(1, 2)[:, :length].double()
        v = s["v_pages"][used].transpose(0, 1).flatten(1, 2)[:, :length].double()
        q = s["q"][t0:t0 + n].double()
        t0 += n
        o, m = torch.empty_like(q), torch.empty(n, c["Hq"], device=q.device, dtype=torch.float64)
        for h in range(c["Hq"] if n else 0):
            x = q[:, h] @ k[h * c["Hkv"] // c["Hq"]].T / math.sqrt(c["d"])
            if c["causal"]:
                x += torch.full_like(x, -math.inf).triu(before + 1)
            m[:, h] = torch.logsumexp(x, -1)
            o[:, h] = torch.exp(x - m[:, h, None]) @ v[h * c["Hkv"] // c["Hq"]]
        out.append(o)
        lse.append(m)
    return torch.cat(out), torch.cat(lse)


def _exact_append(s):
    c = s["case"]
    new, ctx = _lengths(c)
    keys, values, t, half = s["k_pages"].double(), s["v_pages"].double(), 0, c["rot"] // 2
    for b, (n, before) in enumerate(zip(new, ctx)):
        at = s["rope"][before:before + n].double()[:, None, :]
        turn = torch.complex(at[..., :half].contiguous(), at[..., half:].contiguous())
        pos = torch.arange(before, before + n, device=keys.device)
        where, slot = s["block_table"][b].long()[pos // c["page"]], pos % c["page"]
        keys[where, :, slot] = _exact_turn(s["k"][t:t + n].double(), turn, c)
        values[where, :, slot] = s["v"][t:t + n].double()
        t += n
    return keys, values
