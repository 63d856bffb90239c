"""fa_paged_key_weights and fa_paged_evict against their definitions in 64 bits."""
import math

import pytest
import torch

from tests import compact_testlib as c8
from tests import decoder_testlib as lib
from tests.test_paged_gpu import SHAPES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_forward_02_gb300 as fa
    fa.fa_clear_status()
    yield fa
    assert fa.fa_last_status() == 0


def batch(held8, *a, **kw):
    return (c8.Batch8 if held8 else lib.Batch)(*a, **kw)


def weights_for(b, seed=0):
    g = torch.Generator().manual_seed(seed + 100)
    pages, Hkv, page, _ = b.k_pages.shape
    return torch.randn(pages, Hkv, page, generator=g).mul(2).exp().cuda()


def weigh64(b, q, lse, w, scale, causal):
    """The weights after a call and how far each may be off: a score's 32-bit sum is off by at most
    e = d 2^-22 scale sum |q||k| (see decoder_testlib.attend64), its exponent in base 2 by 2^-22 of its terms, the
    exponential by 2^-21 and a sum of n terms by n/2 2^-23 of them at most (here: 2^-17). Exponentials below the
    smallest normal number, 2^-126, may be flushed to zero, one for every row."""
    w = w.double().clone()
    tol = torch.zeros_like(w)
    group = q.shape[1] // b.Hkv
    for i, (n, t) in enumerate(zip(b.new, b.total)):
        if n == 0 or t == 0:
            continue
        rows = slice(b.cu[i], b.cu[i] + n)
        kk = b.keys[i].double().repeat_interleave(group, 0)
        x = q[rows].double().transpose(0, 1)
        s = scale * x @ kk.transpose(1, 2)
        seen = torch.ones(n, t, dtype=torch.bool, device=q.device)
        if causal:
            seen = torch.arange(t, device=q.device)[None] <= (torch.arange(n, device=q.device) + t - n)[:, None]
        L = lse[rows].double().transpose(0, 1)[..., None]
        p = torch.where(seen, torch.exp(s - L.masked_fill(torch.isinf(L), 0.0)), 0.0)
        e = b.d * 2.0 ** -22 * scale * (x.abs() @ kk.abs().transpose(1, 2))
        off = p * (2 * e + 2.0 ** -17 + 2.0 ** -20 * (s.abs() + L.abs().masked_fill(torch.isinf(L), 0.0)))
        gain, off = (y.view(b.Hkv, group, n, t).sum((1, 2)) for y in (p, off))
        pos = torch.arange(t, device=q.device)
        at, slot = b.block_table[i].long()[pos // b.page], pos % b.page
        old = w[at, :, slot] * (pos < t - n)[:, None]
        w[at, :, slot] = old + gain.T
        tol[at, :, slot] = off.T + 2.0 ** -23 * (old + gain.T) + n * group * 2.0 ** -126
    return w, tol


def check_weigh(fa, b, q, causal, scale=None, lse=None, **kw):
    scale = 1 / math.sqrt(b.d) if scale is None else scale
    if lse is None:
        lse = (c8.attend64 if hasattr(b, "k_scale") else lib.attend64)(b, q, scale, causal)[1].float()
    w = weights_for(b)
    # a new token's place may hold anything
    for i, (n, t) in enumerate(zip(b.new, b.total)):
        pos = torch.arange(max(t - n, 0), t, device="cuda")
        w[b.block_table[i].long()[pos // b.page], :, pos % b.page] = math.nan
    want, tol = weigh64(b, q, lse, torch.nan_to_num(w), scale, causal)
    untouched = (want == torch.nan_to_num(w).double()) & (tol == 0)
    before = w.clone()
    fa.paged_key_weights(q, lse, b.k_pages, w, b.block_table, b.cu_seqlens, b.seq_lens, b.max_q, causal=causal,
                         scale=scale, k_scale=getattr(b, "k_scale", None), **kw)
    assert fa.fa_last_status() == 0
    assert torch.equal(w[untouched].view(torch.int32), before[untouched].view(torch.int32))
    err = (w.double() - want).abs()[~untouched]
    assert (err <= tol[~untouched]).all(), ((err - tol[~untouched]).max(), err.max())
    return w


@pytest.mark.parametrize("held8", [False, True])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,total,Hq,Hkv,d,page", SHAPES)
def test_key_weights(fa, new, total, Hq, Hkv, d, page, causal, held8):
    dtype = torch.bfloat16 if (Hq + len(new)) % 2 else torch.float16
    b = batch(held8, new, total, Hkv, d, page, dtype, seed=Hq, token_major=page == 64, lead=2, behind=3)
    check_weigh(fa, b, b.rows(Hq), causal)


@pytest.mark.parametrize("held8", [False, True])
@pytest.mark.parametrize("B", [33, 257, 700])
def test_key_weights_of_many_sequences(fa, B, held8):
    new = [(0, 1, 1, 3, 0)[i % 5] for i in range(B)]
    b = batch(held8, new, [n + (i * 53) % 400 for i, n in enumerate(new)], 2, 64, 16, torch.bfloat16, seed=B, lead=1)
    check_weigh(fa, b, b.rows(4), True)
    new = [(0, 40, 1)[i % 3] for i in range(B)]
    b = batch(held8, new, [n + (i * 37) % 90 for i, n in enumerate(new)], 1, 128, 8, torch.float16, seed=B)
    b.max_q = 1  # longer chunks than the caller knew of
    check_weigh(fa, b, b.rows(8), True)


@pytest.mark.parametrize("held8", [False, True])
def test_key_weights_of_sharp_scores_and_other_scales(fa, held8):
    b = batch(held8, [1, 200, 6], [900, 1200, 6], 2, 128, 16, torch.bfloat16, seed=3)
    q = b.rows(8, std=4.0)
    check_weigh(fa, b, q, True)
    check_weigh(fa, b, q, False, scale=0.0)
    check_weigh(fa, b, q, True, scale=1e-3)


@pytest.mark.parametrize("held8", [False, True])
@pytest.mark.parametrize("d,Hkv,group", [(128, 4, 32), (64, 3, 4), (128, 2, 16), (64, 2, 100)])
def test_key_weights_units_of_one_and_two_tiles(fa, d, Hkv, group, held8):
    """Ragged sequences whose last 256 keys are one tile of 128 or two, in long runs and in turn, for rows of each
    form: the loads of the two tiles then run far apart."""
    total = [(90, 100, 300, 20, 1000, 513, 640, 130)[i % 8] + i for i in range(60)] + [120] * 40 + [700] * 30 + [60] * 30
    b = batch(held8, [1] * len(total), total, Hkv, d, 16, torch.bfloat16, seed=d + group)
    check_weigh(fa, b, b.rows(Hkv * group), True)


def test_key_weights_sum_to_the_rows(fa):
    """What the attention returns is what the weights want: each row gives 1 in all."""
    b = c8.Batch8([1, 70, 0], [3000, 500, 40], 2, 128, 32, torch.bfloat16, seed=9)
    q = b.rows(8)
    _, lse = fa.attention_paged_fp8(q, b.k_pages, b.v_pages, b.k_scale, b.v_scale, b.block_table, b.cu_seqlens,
                                    b.seq_lens, b.max_q)
    w = torch.zeros(b.k_pages.shape[:3], device="cuda")
    fa.paged_key_weights(q, lse, b.k_pages, w, b.block_table, b.cu_seqlens, b.seq_lens, b.max_q, k_scale=b.k_scale)
    for i, n in enumerate(b.new):
        mine = w[b.block_table[i, :-(-b.total[i] // b.page)].long()].double().sum((0, 2))
        assert ((mine - 4.0 * n).abs() <= 1e-4 * max(n, 1)).all()


def test_key_weights_over_what_nobody_sees(fa):
    """NaN in the rest of the last page (the batches here fill it with NaN), in rows of q that belong to
    nobody, and in rows that see no key."""
    for held8 in (False, True):
        b = batch(held8, [5, 40], [2, 30], 2, 64, 16, torch.float16, seed=4, lead=3, behind=2)
        q = b.rows(6)
        lse = (c8.attend64 if held8 else lib.attend64)(b, q, 0.125, True)[1].float()
        dirty = q.clone()
        dirty[:3] = dirty[-2:] = math.nan
        dead = torch.isinf(lse)
        dirty[dead] = math.nan
        a = weights_for(b)
        c = a.clone()
        for x, w in ((q, a), (dirty, c)):
            fa.paged_key_weights(x, lse, b.k_pages, w, b.block_table, b.cu_seqlens, b.seq_lens, b.max_q,
                                 k_scale=getattr(b, "k_scale", None))
        assert torch.equal(a, c) and torch.isfinite(a).all()
        assert fa.fa_last_status() == 0


def test_key_weights_reports_and_passes_over(fa):
    b = lib.Batch([1, 3, 2], [40, 300, 9], 2, 64, 16, torch.float16)
    q = b.rows(4)
    lse = lib.attend64(b, q, 0.125, True)[1].float()
    want = weights_for(b)
    fa.paged_key_weights(q, lse, b.k_pages, want, b.block_table, b.cu_seqlens, b.seq_lens, b.max_q)
    for change in ("rows", "page", "width"):
        w, table, cu = weights_for(b), b.block_table.clone(), b.cu_seqlens.clone()
        if change == "rows":
            cu[3] = 99
            skipped = b.block_table[2, :1].long()
        elif change == "page":
            table[1, 3] = 10 ** 6
            skipped = b.block_table[1, 3:4].long()
        else:
            table = table[:, :5].contiguous()
            skipped = b.block_table[1, 5:19].long()
        fa.paged_key_weights(q, lse, b.k_pages, w, table, cu, b.seq_lens, b.max_q)
        assert fa.fa_last_status() == fa.FA_ERR_RANGE
        fa.fa_clear_status()
        assert torch.equal(w[skipped], weights_for(b)[skipped])
        if change == "page":
            others = torch.ones(w.shape[0], dtype=torch.bool)
            others[skipped.cpu()] = False
            assert torch.equal(w[others.cuda()], want[others.cuda()])


# ------------------------------------------------------------------------------------ eviction
def evict64(b, w, budget, recent):
    """kept, lengths, and what the cache and the weights hold afterwards (values in 64 bits, and how far each
    may be off): position by position."""
    held8 = hasattr(b, "k_scale")
    scales = {n: getattr(b, n + "_scale").double().clone() for n in "kv"} if held8 else None
    raw = {n: getattr(b, n + "_pages").double() for n in "kv"}
    w = w.clone()
    kept = torch.full((len(b.total), b.Hkv, budget), -1, dtype=torch.int32)
    lens = [min(t, budget) for t in b.total]
    for i, t in enumerate(b.total):
        if t <= budget:
            kept[i, :, :t] = torch.arange(t, dtype=torch.int32)
            continue
        pos = torch.arange(t)
        at, slot = b.block_table[i].long().cpu()[pos // b.page], pos % b.page
        for h in range(b.Hkv):
            x = w[at, h, slot].cpu()
            key = torch.where(torch.isnan(x), math.inf, x.double())
            nan = torch.isnan(x)
            order = sorted(range(t - recent), key=lambda j: (not bool(nan[j]), -float(key[j]), j))
            keep = torch.tensor(sorted(order[:budget - recent]) + list(range(t - recent, t)), dtype=torch.long)
            kept[i, h] = keep.int()
            to = torch.arange(budget)
            w[at[to], h, slot[to]] = w[at[keep], h, slot[keep]]
            for n in "kv":
                rows = raw[n][at[keep], h, slot[keep]]
                if held8:
                    came = scales[n][at[keep], h]
                    now = torch.nn.functional.pad(came, (0, -budget % b.page)).view(-1, b.page).amax(1)
                    rows = (rows * (came / now[to // b.page])[:, None]).float().to(c8.E4M3).double()
                    scales[n][at[to[::b.page]], h] = now
                raw[n][at[to], h, slot[to]] = rows
    return kept, lens, w, raw, scales


def check_evict(fa, b, w, budget, recent, **kw):
    want_kept, want_lens, want_w, raw, scales = evict64(b, w, budget, recent)
    held8 = scales is not None
    kept, lens = fa.paged_evict(b.k_pages, b.v_pages, w, b.block_table, b.seq_lens, budget, recent,
                                k_scale=getattr(b, "k_scale", None), v_scale=getattr(b, "v_scale", None), **kw)
    assert fa.fa_last_status() == 0
    assert torch.equal(kept.cpu(), want_kept) and lens.tolist() == want_lens
    assert torch.equal(torch.nan_to_num(w, nan=-7.0), torch.nan_to_num(want_w, nan=-7.0))
    for n in "kv":
        got = getattr(b, n + "_pages").double()
        assert torch.equal(torch.nan_to_num(got, nan=1e9), torch.nan_to_num(raw[n], nan=1e9))
        if held8:
            assert torch.equal(getattr(b, n + "_scale").double(), scales[n])
    return kept, lens


EVICTIONS = [
    # total, Hkv, d, page, budget, recent
    ([1], 1, 64, 8, 1, 0),
    ([2], 2, 128, 8, 1, 0),
    ([2], 2, 128, 8, 1, 1),
    ([40, 17, 0, 16], 3, 64, 16, 16, 5),
    ([100, 300, 99], 2, 128, 16, 99, 0),
    ([1000, 31, 33], 1, 128, 32, 32, 32),
    ([777, 2049, 5], 4, 64, 64, 500, 77),
    ([1500], 8, 128, 128, 1024, 100),
    ([1400, 400], 2, 64, 384, 385, 1),
    ([3000, 2900], 2, 128, 1024, 2500, 2000),
    ([5000], 12, 128, 16, 4999, 10),
    ([9000, 1, 8999], 1, 64, 32, 123, 60),
]


@pytest.mark.parametrize("held8", [False, True])
@pytest.mark.parametrize("total,Hkv,d,page,budget,recent", EVICTIONS)
def test_evict(fa, total, Hkv, d, page, budget, recent, held8):
    dtype = torch.bfloat16 if Hkv % 2 else torch.float16
    kw = dict(spread=2.0) if held8 else {}
    b = batch(held8, [0] * len(total), total, Hkv, d, page, dtype, seed=budget, token_major=page == 64, **kw)
    check_evict(fa, b, weights_for(b, budget), budget, recent)


@pytest.mark.parametrize("held8", [False, True])
def test_evict_ties_zeros_and_what_is_not_finite(fa, held8):
    for kind in range(6):
        b = batch(held8, [0, 0], [700, 513], 2, 64, 16, torch.float16, seed=kind)
        w = weights_for(b, kind)
        if kind == 0:
            w.fill_(0.25)
        elif kind == 1:
            w.copy_((w * 2).round().clamp(max=3))
        elif kind == 2:
            w.zero_()
            w[:, :, ::2] = -0.0
        elif kind == 3:
            w[:, :, 1::5] = math.nan
            w[:, :, 2::5] = math.inf
        elif kind == 4:
            w[:, :, ::3] = -math.inf
            w.neg_()
        else:
            w.mul_(1e-40)  # subnormal
        check_evict(fa, b, w, 300, 40)


def test_evict_many_tokens(fa):
    """More weights than a block keeps in shared memory."""
    b = lib.Batch([0], [45000], 1, 64, 128, torch.bfloat16, seed=1)
    check_evict(fa, b, weights_for(b), 30000, 4000)
    b = c8.Batch8([0], [45000], 1, 64, 16, torch.bfloat16, seed=2)
    w = weights_for(b)
    w = (w * 8).round() / 8  # many ties
    check_evict(fa, b, w, 20001, 0)


def test_evict_in_place_lengths_streams_and_graphs(fa):
    def make():
        b = c8.Batch8([0, 0, 0], [700, 513, 90], 4, 128, 16, torch.bfloat16, seed=5, spread=1.0)
        return b, weights_for(b)
    b, w = make()
    check_evict(fa, b, w, 200, 30)
    side = torch.cuda.Stream()
    c, x = make()
    ws = torch.empty(fa.fa_paged_evict_workspace_bytes(3, 4, 200, True), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    kept, lens = fa.paged_evict(c.k_pages, c.v_pages, x, c.block_table, c.seq_lens, 200, 30, k_scale=c.k_scale,
                                v_scale=c.v_scale, new_lens=c.seq_lens, workspace=ws, stream=side)
    side.synchronize()
    assert lens.data_ptr() == c.seq_lens.data_ptr() and c.seq_lens.tolist() == [200, 200, 90]
    for n in ("k_pages", "v_pages"):
        assert torch.equal(getattr(b, n).view(torch.uint8), getattr(c, n).view(torch.uint8))
    # captured, replayed with other lengths: the second replay has nothing to do
    c, x = make()
    kept = torch.empty(3, 4, 200, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.paged_evict(c.k_pages, c.v_pages, x, c.block_table, c.seq_lens, 200, 30, k_scale=c.k_scale,
                       v_scale=c.v_scale, new_lens=c.seq_lens, kept=kept)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(x, w) and c.seq_lens.tolist() == [200, 200, 90]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(x, w) and torch.equal(kept[0, 0], torch.arange(200, device="cuda").int())


@pytest.mark.parametrize("held8", [False, True])
def test_evict_many_heads_with_lengths_in_place(fa, held8):
    """More heads than run at once: the last ones still see the lengths that new_lens overwrites."""
    b = batch(held8, [0] * 12, [90 + i for i in range(12)], 64, 64, 16, torch.float16, seed=8)
    kept, _ = check_evict(fa, b, weights_for(b, 8), 70, 9, new_lens=b.seq_lens)
    assert int(kept[:, :, -1].min()) == 89


def test_evict_reports_bad_pages(fa):
    b = lib.Batch([0], [300], 1, 64, 16, torch.float16, seed=6)
    w = weights_for(b)
    b.block_table[0, 2] = -5
    before = b.k_pages.clone()
    kept, lens = fa.paged_evict(b.k_pages, b.v_pages, w, b.block_table, b.seq_lens, 100, 10)
    assert fa.fa_last_status() == fa.FA_ERR_RANGE
    fa.fa_clear_status()
    assert lens.tolist() == [100] and not ((kept >= 32) & (kept < 48)).any()
    pages = b.block_table[0].long()
    assert torch.equal(torch.nan_to_num(b.k_pages[pages[7:]].float()), torch.nan_to_num(before[pages[7:]].float()))


def test_prompt_then_tokens_with_eviction(fa):
    """As a server would use them together: a prompt into the 8-bit cache, its weights, eviction, then tokens
    that attend to what was kept, against the same steps in 64 bits over what the cache holds."""
    Hq, Hkv, d, page, n, budget, recent = 8, 2, 64, 16, 500, 200, 50
    pages = 40
    g = torch.Generator().manual_seed(3)
    table = torch.randperm(pages, generator=g)[:36].int().cuda().view(1, 36)
    kp, vp = (torch.zeros(pages, Hkv, page, d, dtype=torch.uint8, device="cuda").view(c8.E4M3) for _ in range(2))
    ks, vs = (torch.ones(pages, Hkv, device="cuda") for _ in range(2))
    w = torch.full((pages, Hkv, page), math.nan, device="cuda")
    make = lambda t, h: torch.randn(t, h, d, generator=g).bfloat16().cuda()  # noqa: E731
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    q = make(n, Hq)
    fa.paged_append_fp8(make(n, Hkv), make(n, Hkv), kp, vp, ks, vs, table, cu, lens)
    _, lse = fa.attention_paged_fp8(q, kp, vp, ks, vs, table, cu, lens, n)
    fa.paged_key_weights(q, lse, kp, w, table, cu, lens, n, k_scale=ks)
    used = table[0, :32].long()
    values = lambda p, s: (p.view(torch.uint8)[used].view(c8.E4M3).double() * s[used].double()[..., None, None]  # noqa: E731
                           ).transpose(0, 1).flatten(1, 2)
    k0, v0 = values(kp, ks), values(vp, vs)
    kept, lens = fa.paged_evict(kp, vp, w, table, lens, budget, recent, k_scale=ks, v_scale=vs)
    k1, v1 = values(kp, ks), values(vp, vs)
    for h in range(Hkv):  # the kept rows moved, under scales that may have grown: half a step of E4M3 at most
        for x0, x1 in ((k0, k1), (v0, v1)):
            a, c = x0[h][kept[0, h].long()], x1[h, :budget]
            assert ((a - c).abs() <= c8.HALF8 * a.abs() + 2.0 ** -10).all()
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for step in range(3):
        lens = lens + 1
        q, k, v = make(1, Hq), make(1, Hkv), make(1, Hkv)
        fa.paged_append_fp8(k, v, kp, vp, ks, vs, table, cu, lens)
        out, lse = fa.attention_paged_fp8(q, kp, vp, ks, vs, table, cu, lens, 1)
        fa.paged_key_weights(q, lse, kp, w, table, cu, lens, 1, k_scale=ks)
        t = budget + step + 1
        kk, vv = (values(p, s)[:, :t].repeat_interleave(Hq // Hkv, 0) for p, s in ((kp, ks), (vp, vs)))
        s = (q[0].double()[:, None] @ kk.transpose(1, 2))[:, 0] / math.sqrt(d)
        want = (s.softmax(-1)[:, None] @ vv)[:, 0]
        assert ((out[0].double() - want).abs() <= 2.0 ** -7 * vv.abs().amax((1, 2))[:, None]).all()
    assert fa.fa_last_status() == 0 and torch.isfinite(w[table[0, :13].long()][:12]).all()


def test_evict_from_a_cache_without_pages(fa):
    """Every page is bad: nothing is looked at or moved, all weights count the same."""
    empty = torch.empty(0, 3, 16, 64, dtype=torch.float16, device="cuda")
    w = torch.empty(0, 3, 16, device="cuda")
    table = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    lens = torch.tensor([20, 3], dtype=torch.int32, device="cuda")
    kept, now = fa.paged_evict(empty, empty.clone(), w, table, lens, 4, 1)
    torch.cuda.synchronize()
    assert fa.fa_last_status() == fa.FA_ERR_RANGE
    fa.fa_clear_status()
    assert kept[0].tolist() == [[0, 1, 2, 19]] * 3 and kept[1].tolist() == [[0, 1, 2, -1]] * 3
    assert now.tolist() == [4, 3]


def test_calls_that_autograd_would_record_are_refused(fa):
    def grad(x):
        return x.clone().requires_grad_()

    b = c8.Batch8([2, 1], [20, 3], 2, 64, 16, torch.float16, seed=9)
    q, w = b.rows(4), torch.zeros(b.k_pages.shape[0], 2, 16, device="cuda")
    table = (b.block_table, b.cu_seqlens, b.seq_lens)
    _, L = fa.attention_paged_fp8(q, b.k_pages, b.v_pages, b.k_scale, b.v_scale, *table, 2)
    before = w.clone()
    with torch.enable_grad():
        with pytest.raises(ValueError, match="autograd"):
            fa.attention_paged_fp8(grad(q), b.k_pages, b.v_pages, b.k_scale, b.v_scale, *table, 2)
        with pytest.raises(ValueError, match="autograd"):
            fa.paged_append_fp8(grad(b.rows(2)), b.rows(2), b.k_pages, b.v_pages, b.k_scale, b.v_scale, *table)
        with pytest.raises(ValueError, match="autograd"):
            fa.paged_key_weights(q, grad(L), b.k_pages, w, *table, 2, k_scale=b.k_scale)
        with pytest.raises(ValueError, match="autograd"):
            fa.paged_evict(b.k_pages, b.v_pages, grad(w), b.block_table, b.seq_lens, 2, 1, k_scale=b.k_scale,
                           v_scale=b.v_scale)
    assert torch.equal(w, before)
    with torch.no_grad():
        fa.paged_key_weights(grad(q), grad(L), b.k_pages, w, *table, 2, k_scale=b.k_scale)
    assert not torch.equal(w, before)
