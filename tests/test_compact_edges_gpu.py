"""The operators of a compact cache where their callers may put things: cache and rows as views of larger tensors,
places past 32 bits, whole chains in a graph, calls at the same time on two streams. Every case is held
against the same call on plain copies, bit by bit (the kernels' order of sums does not depend on strides)."""
import pytest
import torch

from tests import compact_testlib as c8
from tests import decoder_testlib as lib

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_forward_02_gb300 as fa
    fa.fa_clear_status()
    return fa


def raw(x):
    return x.view(torch.uint8) if x.dtype == E4M3 else x.view(torch.int32) if x.dtype == torch.float32 else x.view(torch.int16)


def state(b, held8):
    """A copy of the batch's cache, with weights."""
    s = {n: getattr(b, n).clone(memory_format=torch.preserve_format) for n in
         ("k_pages", "v_pages") + (("k_scale", "v_scale") if held8 else ())}
    g = torch.Generator().manual_seed(11)
    s["w"] = torch.rand(b.k_pages.shape[0], b.Hkv, b.page, generator=g).cuda()
    return s


def chain(fa, b, s, q, k, v, budget, recent, **kw):
    """Append, attend, weigh, evict: what a step of a server does."""
    ids = (b.block_table, b.cu_seqlens, b.seq_lens)
    if "k_scale" in s:
        scales = (s["k_scale"], s["v_scale"])
        fa.paged_append_fp8(k, v, s["k_pages"], s["v_pages"], *scales, *ids, **kw)
        O, L = fa.attention_paged_fp8(q, s["k_pages"], s["v_pages"], *scales, *ids, b.max_q, **kw)
        fa.paged_key_weights(q, L, s["k_pages"], s["w"], *ids, b.max_q, k_scale=scales[0], **kw)
        kept, now = fa.paged_evict(s["k_pages"], s["v_pages"], s["w"], b.block_table, b.seq_lens, budget, recent,
                                   k_scale=scales[0], v_scale=scales[1], **kw)
    else:
        fa.paged_append(k, v, s["k_pages"], s["v_pages"], *ids, **kw)
        O, L = fa.attention_paged(q, s["k_pages"], s["v_pages"], *ids, b.max_q, **kw)
        fa.paged_key_weights(q, L, s["k_pages"], s["w"], *ids, b.max_q, **kw)
        kept, now = fa.paged_evict(s["k_pages"], s["v_pages"], s["w"], b.block_table, b.seq_lens, budget, recent, **kw)
    return O, L, kept, now


def same(x, y):
    return all(torch.equal(raw(i), raw(j)) if i.dtype != torch.int32 else torch.equal(i, j) for i, j in zip(x, y))


def make(held8, new=(1, 5, 40), total=(1200, 700, 90), Hkv=2, d=128, page=16, seed=3, **kw):
    return (c8.Batch8 if held8 else lib.Batch)(list(new), list(total), Hkv, d, page, torch.bfloat16, seed=seed, **kw)


@pytest.mark.parametrize("held8", [False, True])
@pytest.mark.parametrize("new", [(1, 1, 1), (1, 5, 40), (300, 1, 20)])
def test_cache_and_rows_as_views(fa, held8, new):
    """K and V side by side in one pool, rows of a fused projection."""
    total = [1200, 700, 90]
    b = make(held8, new, total)
    T, Hq, Hkv, d = b.T, 8, b.Hkv, 128
    fused = (torch.randn(T, Hq + 2 * Hkv, d, generator=b.g)).bfloat16().cuda()
    q, k, v = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    s = state(b, held8)
    want = chain(fa, b, s, q.contiguous(), k.contiguous(), v.contiguous(), 400, 30)
    x = state(b, held8)
    pool = torch.zeros(b.k_pages.shape[0], 3, Hkv, b.page, d, dtype=torch.uint8 if held8 else torch.bfloat16, device="cuda")
    for i, n in ((0, "k_pages"), (2, "v_pages")):
        pool[:, i] = x[n].view(torch.uint8) if held8 else x[n]
        x[n] = pool[:, i].view(E4M3) if held8 else pool[:, i]
    got = chain(fa, b, x, q, k, v, 400, 30)
    assert fa.fa_last_status() == 0
    assert same(want, got) and all(torch.equal(raw(s[n].contiguous()), raw(x[n].contiguous())) for n in s)
    assert not pool[:, 1].any()


@pytest.mark.parametrize("held8", [False, True])
def test_pages_past_32_bits(fa, held8):
    """The same pages at the far end of a cache of more than 2^32 bytes (and elements) each for K and V."""
    b = make(held8, (1, 5, 40), (1200, 700, 90), page=128)
    q, k, v = b.rows(8), b.rows(2), b.rows(2)
    s = state(b, held8)
    want = chain(fa, b, s, q, k, v, 400, 30)
    pages, per = b.k_pages.shape[0], b.Hkv * b.page * 128
    far = (1 << 32) // per + 1
    x = state(b, held8)
    for n in list(x):
        big = torch.empty(far + pages, *x[n].shape[1:], dtype=torch.uint8 if x[n].dtype == E4M3 else x[n].dtype, device="cuda")
        big[far:] = x[n].view(big.dtype)
        x[n] = big.view(x[n].dtype)
    b.block_table = torch.where(b.block_table >= 0, b.block_table + far, b.block_table)
    got = chain(fa, b, x, q, k, v, 400, 30)
    assert fa.fa_last_status() == 0
    assert same(want, got) and all(torch.equal(raw(s[n].contiguous()), raw(x[n][far:].contiguous())) for n in s)


@pytest.mark.parametrize("held8", [False, True])
def test_a_chain_in_a_graph(fa, held8):
    b = make(held8)
    q, k, v = b.rows(8), b.rows(2), b.rows(2)
    first = state(b, held8)
    s = {n: x.clone() for n, x in first.items()}
    want = chain(fa, b, s, q, k, v, 400, 30)
    x = {n: y.clone() for n, y in first.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(fa, b, x, q, k, v, 400, 30)
    for _ in range(2):
        for n in x:
            raw(x[n]).copy_(raw(first[n]))
        graph.replay()
        torch.cuda.synchronize()
        assert same(want, got) and all(torch.equal(raw(s[n]), raw(x[n])) for n in s)


@pytest.mark.parametrize("held8", [False, True])
def test_two_chains_at_the_same_time(fa, held8):
    """Two batches on two streams, each with workspaces of its own, several times over."""
    jobs = []
    for seed, new in ((3, (1, 5, 40)), (4, (1, 1, 1))):
        b = make(held8, new, (5000, 3000, 2000), Hkv=4, seed=seed)
        q, k, v = b.rows(16), b.rows(4), b.rows(4)
        s = state(b, held8)
        first = {n: x.clone() for n, x in s.items()}
        jobs.append((b, q, k, v, first, s, chain(fa, b, s, q, k, v, 1000, 100), torch.cuda.Stream()))
    for _ in range(3):
        ran = []
        copies = [{n: x.clone() for n, x in j[4].items()} for j in jobs]
        torch.cuda.synchronize()
        for (b, q, k, v, _, _, _, stream), x in zip(jobs, copies):
            with torch.cuda.stream(stream):
                ran.append(chain(fa, b, x, q, k, v, 1000, 100))
        torch.cuda.synchronize()
        for j, x, got in zip(jobs, copies, ran):
            assert same(j[6], got) and all(torch.equal(raw(j[5][n]), raw(x[n])) for n in x)
    assert fa.fa_last_status() == 0


@pytest.mark.parametrize("held8", [False, True])
def test_what_lies_behind_the_sequences_is_not_seen(fa, held8):
    """Other numbers in every place and row that belongs to nobody: the same results, and those stay as they were."""
    b = make(held8, lead=2, behind=3)
    q, k, v = b.rows(8), b.rows(2), b.rows(2)
    s, x = state(b, held8), state(b, held8)
    mine = torch.zeros(b.k_pages.shape[0], b.page, dtype=torch.bool, device="cuda")
    for i, t in enumerate(b.total):
        pos = torch.arange(t)
        mine[b.block_table[i].long().cpu()[pos // b.page], pos % b.page] = True
    junk = torch.randint(0, 256, x["k_pages"].view(torch.uint8).shape, generator=b.g, dtype=torch.uint8).cuda()
    for n in ("k_pages", "v_pages"):
        bytes_ = x[n].view(torch.uint8)
        bytes_.copy_(torch.where(mine[:, None, :, None], bytes_, junk))
    x["w"] = torch.where(mine[:, None], x["w"], torch.full_like(x["w"], float("nan")))
    before = {n: x[n].view(torch.uint8).clone() for n in ("k_pages", "v_pages", "w")}
    want, got = chain(fa, b, s, q, k, v, 400, 30), chain(fa, b, x, q, k, v, 400, 30)
    rows = slice(b.cu[0], b.cu[-1])
    assert fa.fa_last_status() == 0
    assert same([y[rows] for y in want[:2]], [y[rows] for y in got[:2]]) and same(want[2:], got[2:])
    for n, y in before.items():
        now = x[n].view(torch.uint8)
        there = mine[:, None, :, None].expand_as(now) if n != "w" else mine[:, None, :, None].expand(
            *x["w"].shape, 4).flatten(2)
        assert torch.equal(now[~there], y[~there])
