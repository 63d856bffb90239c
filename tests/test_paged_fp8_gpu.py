"""fa_paged_append_fp8 and fa_fwd_paged_fp8 against their definitions in 64 bits."""
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


def attend(fa, b, q, causal, **kw):
    return fa.attention_paged_fp8(q, b.k_pages, b.v_pages, b.k_scale, b.v_scale, b.block_table, b.cu_seqlens,
                                  b.seq_lens, b.max_q, causal=causal, **kw)


def check(fa, b, q, causal, scale=None, **kw):
    scale = 1 / math.sqrt(b.d) if scale is None else scale
    O = torch.full_like(q, 99.0) if "out" not in kw else kw.pop("out")
    L = torch.full(q.shape[:2], 99.0, device="cuda")
    attend(fa, b, q, causal, scale=scale, out=O, lse=L, **kw)
    want_o, want_l, tol_o, tol_l = c8.attend64(b, q, scale, causal)
    assert fa.fa_last_status() == 0
    mine = slice(b.cu[0], b.cu[-1])
    err = (O.double() - want_o).abs()[mine]
    assert (err <= tol_o[mine]).all(), ((err - tol_o[mine]).max(), err.max())
    dead = torch.isinf(want_l[mine])
    assert torch.equal(torch.isinf(L[mine]) & (L[mine] < 0), dead)
    assert not O[mine][dead].any()
    el = (L.double() - want_l).abs()[mine][~dead]
    assert (el <= tol_l[mine][~dead]).all(), el.max()
    for x in (O, L):  # rows of no sequence
        assert (x[:b.cu[0]] == 99).all() and (x[b.cu[-1]:] == 99).all()
    return O, L


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,total,Hq,Hkv,d,page", SHAPES)
def test_attention(fa, new, total, Hq, Hkv, d, page, causal):
    dtype = torch.bfloat16 if (Hq + len(new)) % 2 else torch.float16
    b = c8.Batch8(new, total, Hkv, d, page, dtype, seed=Hq, token_major=page == 64, lead=2, behind=3)
    check(fa, b, b.rows(Hq), causal)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("page", [8, 16, 64, 128, 384])
@pytest.mark.parametrize("d", [64, 128])
def test_types_pages_and_scales(fa, d, page, dtype):
    """Pages whose scales differ by much, scales that are no powers of two, sharp scores."""
    new, total = [1, 200, 6, 1], [900, 1200, 6, 2000]
    b = c8.Batch8(new, total, 2, d, page, lib.DTYPES[dtype], seed=3, spread=3.0)
    check(fa, b, b.rows(8, std=0.3), True)
    b = c8.Batch8(new, total, 2, d, page, lib.DTYPES[dtype], seed=4, spread=1.0, odd=True)
    q = b.rows(8, std=3.0)
    check(fa, b, q, True)
    check(fa, b, q, False, scale=0.0)
    b.max_q = 1  # a batch with longer chunks than the caller knew of
    check(fa, b, q, True, scale=1e-3)


@pytest.mark.parametrize("B", [33, 257, 700])
def test_many_sequences_some_without_tokens(fa, B):
    new = [(0, 1, 1, 3, 0)[i % 5] for i in range(B)]
    b = c8.Batch8(new, [n + (i * 53) % 400 for i, n in enumerate(new)], 2, 64, 16, torch.bfloat16, seed=B, lead=1)
    check(fa, b, b.rows(4), True)
    new = [(0, 40, 1)[i % 3] for i in range(B)]
    b = c8.Batch8(new, [n + (i * 37) % 90 for i, n in enumerate(new)], 1, 128, 16, torch.float16, seed=B)
    check(fa, b, b.rows(8), True)


def test_pages_of_zeros_and_all_codes(fa):
    """Scales of 0 for pages that hold zeros, and every finite code of E4M3 in keys and values."""
    b = c8.Batch8([1, 130], [1300, 1300], 2, 128, 32, torch.float16, seed=5)
    codes = torch.arange(256, device="cuda", dtype=torch.uint8)
    codes = codes[(codes & 127) != 127]
    for pages in (b.k_pages, b.v_pages):
        at = torch.randint(0, codes.numel(), pages.shape, generator=b.g).cuda()
        pages.view(torch.uint8).copy_(codes[at])
    first = b.block_table[:, :2].flatten().long()
    for pages, scale in ((b.k_pages, b.k_scale), (b.v_pages, b.v_scale)):
        scale.fill_(2.0 ** -7)
        pages.view(torch.uint8)[first] = 0
        scale[first] = 0.0
    b.decode()
    check(fa, b, b.rows(4), True)
    b.v_scale[:] = 0.0
    b.v_pages.view(torch.uint8)[:] = 0
    b.decode()
    O, _ = check(fa, b, b.rows(4), True)
    assert not O.any()


def test_large_and_small_scales(fa):
    """Values near the ends of bf16's range."""
    for factor in (2.0 ** 60, 2.0 ** -60):
        b = c8.Batch8([1, 140], [700, 300], 1, 64, 16, torch.bfloat16, seed=6)
        b.v_scale *= factor
        b.decode()
        check(fa, b, b.rows(4), True)


def test_results_do_not_change_and_streams(fa):
    b = c8.Batch8([1] * 20 + [300], [5000] * 20 + [3000], 4, 128, 16, torch.bfloat16, seed=7)
    q = b.rows(16)
    want = attend(fa, b, q, True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got = attend(fa, b, q, True, stream=side)
        side.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_captured_and_replayed_with_other_lengths(fa):
    b = c8.Batch8([1, 1, 1], [2000, 1500, 10], 2, 128, 16, torch.float16, seed=8)
    q = b.rows(8)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    attend(fa, b, q, True, out=out, lse=lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attend(fa, b, q, True, out=out, lse=lse)
    b.total = [17, 1499, 1]
    b.seq_lens.copy_(torch.tensor(b.total))
    graph.replay()
    torch.cuda.synchronize()
    b.decode()
    O, L, tol_o, tol_l = c8.attend64(b, q, 1 / math.sqrt(128), True)
    assert ((out.double() - O).abs() <= tol_o).all() and ((lse.double() - L).abs() <= tol_l).all()


# ------------------------------------------------------------------------------------- append
def check_append(fa, b, k, v, table=None, interleaved=False, skipped=lambda i, pos: False):
    """The pages after a call: scales as defined, every element within half a step of E4M3."""
    before = {n: (getattr(b, n + "_pages").double(), getattr(b, n + "_scale").double()) for n in "kv"}
    raw = {n: getattr(b, n + "_pages").view(torch.uint8).clone() for n in "kv"}
    fa.paged_append_fp8(k, v, b.k_pages, b.v_pages, b.k_scale, b.v_scale, b.block_table, b.cu_seqlens, b.seq_lens,
                        rope=table, interleaved=interleaved)
    torch.cuda.synchronize()
    touched = {n: torch.zeros(b.k_pages.shape[:3], dtype=torch.bool, device="cuda") for n in "kv"}
    for i, (n, t) in enumerate(zip(b.new, b.total)):
        rows = slice(b.cu[i], b.cu[i] + n)
        for name, x in (("k", k), ("v", v)):
            x = x[rows].double()
            size = x.abs()
            pos = torch.arange(t - n, t, device="cuda")
            if name == "k" and table is not None:
                inside = pos.clamp(min=0, max=table.shape[0] - 1)
                x = lib.turn64(x, table[inside][:, None], interleaved)
                size = size.amax(-1, keepdim=True).expand_as(x) * 2
            pages, scale = getattr(b, name + "_pages"), getattr(b, name + "_scale")
            for j in range(max(t - n, 0) // b.page, -(-t // b.page)):
                here = [y for y in range(n) if pos[y] // b.page == j and pos[y] >= 0 and not skipped(i, int(pos[y]))]
                if not here:
                    continue
                at = int(b.block_table[i, j])
                slots = pos[here] % b.page
                lead = max(0, t - n - j * b.page)
                new, s_old, s = x[here], before[name][1][at], scale[at].double()
                top = torch.where(torch.isfinite(new), new.abs(), 0.0).amax((0, 2))
                wide = 2.0 ** -21  # two products and a sum in fp32
                lo, hi = c8.power(top * (1 - wide) / 448), c8.power(top * (1 + wide) / 448)
                if lead:
                    lo, hi = torch.maximum(lo, s_old), torch.maximum(hi, s_old)
                assert ((s == lo) | (s == hi)).all()
                got = pages[at].view(torch.uint8)[:, slots].view(c8.E4M3).double().transpose(0, 1) * s[:, None]
                tol = c8.HALF8 * new.abs() * (1 + 2.0 ** -20) + c8.TINY8 * s[:, None] + wide * size[here]
                fine = torch.isfinite(new)
                assert torch.isnan(got[~fine]).all()
                assert ((got - new).abs() <= tol)[fine].all()
                if name == "v" and fine.all():  # nothing but one rounding: the very codes
                    want = (new / s[:, None]).float().to(c8.E4M3)
                    assert torch.equal(pages[at].view(torch.uint8)[:, slots].transpose(0, 1), want.view(torch.uint8))
                touched[name][at][:, slots] = True
                if lead:
                    old = before[name][0][at][:, :lead] * s_old[:, None, None]
                    got = pages[at].view(torch.uint8)[:, :lead].view(c8.E4M3).double() * s[:, None, None]
                    grown = s > s_old
                    assert torch.equal(pages[at].view(torch.uint8)[~grown][:, :lead], raw[name][at][~grown][:, :lead])
                    tol = c8.HALF8 * old.abs() * (1 + 2.0 ** -20) + c8.TINY8 * s[:, None, None]
                    some = torch.isfinite(old) & grown[:, None, None]
                    assert ((got - old).abs() <= tol)[some].all()
                    touched[name][at][grown, :lead] = True
    for n in "kv":  # everything else is as it was
        now = getattr(b, n + "_pages").view(torch.uint8)
        assert torch.equal(now[~touched[n]], raw[n][~touched[n]])
        quiet = ~touched[n].any(2)
        assert torch.equal(getattr(b, n + "_scale").double()[quiet], before[n][1][quiet])


APPENDS = [
    # new, total, Hkv, d, page
    ([1], [1], 1, 64, 8),
    ([1], [17], 3, 128, 16),
    ([5], [5], 2, 64, 16),
    ([1, 0, 3, 40], [50, 7, 3, 90], 2, 128, 16),
    ([1] * 70, [1 + (37 * i) % 211 for i in range(70)], 2, 64, 32),
    ([300, 1, 129], [700, 129, 129], 2, 128, 64),
    ([600], [900], 1, 128, 256),
    ([1000, 3], [1400, 770], 1, 64, 384),
    ([1300], [1300], 2, 128, 1024),
    ([5, 40], [2, 30], 2, 64, 16),   # fewer cached than new: leading rows have no place
]


@pytest.mark.parametrize("new,total,Hkv,d,page", APPENDS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append(fa, new, total, Hkv, d, page, dtype):
    b = c8.Batch8(new, total, Hkv, d, page, lib.DTYPES[dtype], seed=page, spread=2.0, lead=1, behind=2,
                  token_major=page == 32)
    fused = b.rows(3 * Hkv, std=1.0)
    k, v = fused[:, Hkv:2 * Hkv], fused[:, 2 * Hkv:]
    check_append(fa, b, k, v)
    short = any(n > t for n, t in zip(new, total))
    assert fa.fa_last_status() == (fa.FA_ERR_RANGE if short else 0)
    fa.fa_clear_status()
    for rot, interleaved in ((d, False), (d // 2, True), (16, False), (d, True)):
        table = lib.rope_table(max(total) + 3, rot, "cuda")
        b = c8.Batch8(new, total, Hkv, d, page, lib.DTYPES[dtype], seed=page + rot, spread=2.0)
        check_append(fa, b, b.rows(Hkv), b.rows(Hkv, std=5.0), table, interleaved)
        assert fa.fa_last_status() == (fa.FA_ERR_RANGE if short else 0)
        fa.fa_clear_status()


def test_append_of_zeros_and_of_what_is_not_finite(fa):
    b = c8.Batch8([20, 20], [20, 40], 2, 64, 16, torch.bfloat16, seed=1)
    k, v = b.rows(2), b.rows(2)
    k[3] = 0.0
    v[20:40] = 0.0
    v[5, 1, 7], v[6, 0, 3], k[22, 0, 9], k[23, 1, 1] = math.inf, math.nan, -math.inf, 3e38
    check_append(fa, b, k, v)


def test_append_skips_and_reports(fa):
    """Bad pages, positions behind the table, rows outside the packed tokens."""
    b = c8.Batch8([30, 30, 30], [60, 90, 30], 2, 64, 16, torch.float16, seed=2)
    k, v = b.rows(2), b.rows(2)
    table = lib.rope_table(70, 64, "cuda")
    check_append(fa, b, k, v, table, skipped=lambda i, pos: pos >= 70)
    assert fa.fa_last_status() == fa.FA_ERR_RANGE
    fa.fa_clear_status()
    for change in ("page", "width", "rows"):
        b = c8.Batch8([30, 30, 30], [60, 90, 30], 2, 64, 16, torch.float16, seed=2)
        if change == "page":
            bad = int(b.block_table[1, 4])
            b.block_table[1, 4] = 10 ** 6
            raw = b.k_pages.view(torch.uint8).clone()
            fa.paged_append_fp8(k, v, b.k_pages, b.v_pages, b.k_scale, b.v_scale, b.block_table, b.cu_seqlens, b.seq_lens)
            assert torch.equal(b.k_pages.view(torch.uint8)[bad], raw[bad])
        elif change == "width":
            b.block_table = b.block_table[:, :5].contiguous()
            fa.paged_append_fp8(k, v, b.k_pages, b.v_pages, b.k_scale, b.v_scale, b.block_table, b.cu_seqlens, b.seq_lens)
        else:
            b.cu_seqlens[3] = 99
            raw = b.v_pages.view(torch.uint8).clone()
            fa.paged_append_fp8(k, v, b.k_pages, b.v_pages, b.k_scale, b.v_scale, b.block_table, b.cu_seqlens, b.seq_lens)
            mine = b.block_table[2, :2].long()
            assert torch.equal(b.v_pages.view(torch.uint8)[mine], raw[mine])
        assert fa.fa_last_status() == fa.FA_ERR_RANGE
        fa.fa_clear_status()


def test_append_then_attend_token_by_token(fa):
    """A prompt, then single tokens: the cache that grows gives the attention of what it holds, and the
    pages' scales grow as their tokens do."""
    Hq, Hkv, d, page, n = 8, 2, 128, 16, 70
    pages = 8
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(0)).int().cuda().view(1, pages)
    kp, vp = (torch.zeros(pages, Hkv, page, d, dtype=torch.uint8, device="cuda").view(c8.E4M3) for _ in range(2))
    ks, vs = (torch.full((pages, Hkv), math.nan, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(1)
    size = torch.linspace(0.1, 4, n)[:, None, None]
    k, v = ((torch.randn(n, Hkv, d, generator=g) * size).bfloat16().cuda() for _ in range(2))
    q = torch.randn(n, Hq, d, generator=g).bfloat16().cuda()
    at, outs = 0, []
    for step in [37] + [1] * 33:
        cu = torch.tensor([0, step], dtype=torch.int32, device="cuda")
        lens = torch.tensor([at + step], dtype=torch.int32, device="cuda")
        rows = slice(at, at + step)
        fa.paged_append_fp8(k[rows], v[rows], kp, vp, ks, vs, table, cu, lens)
        outs.append(fa.attention_paged_fp8(q[rows], kp, vp, ks, vs, table, cu, lens, step)[0])
        at += step
    got = torch.cat(outs).double()
    kk, vv = (x.double().transpose(0, 1).repeat_interleave(Hq // Hkv, 0) for x in (k, v))
    s = (q.double().transpose(0, 1) @ kk.transpose(1, 2)) / math.sqrt(d)
    s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), -math.inf)
    want = (s.softmax(-1) @ vv).transpose(0, 1)
    # keys and values off by 2^-4 of themselves at most (2^-5.5 on average): far below the outputs' size
    assert float((got - want).norm() / want.norm()) < 0.06
