"""The operators of a compact cache on arrays that are not as they should be: what is passed over is reported, nothing is
read or written outside what belongs to the call, and the rest comes out as without it."""
import pytest
import torch

from tests import compact_testlib as c8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_forward_02_gb300 as fa
    fa.fa_clear_status()
    return fa


def status(fa):
    torch.cuda.synchronize()
    s = fa.fa_last_status()
    fa.fa_clear_status()
    return s


def held(s):
    """What pages and heads hold, as whole numbers: [pages, Hkv, bytes of K, of V and of both scales]."""
    k, v = (s[n].view(torch.uint8).flatten(2) for n in ("k_pages", "v_pages"))
    scales = [s[n].view(torch.uint8).view(*s[n].shape, 4) for n in ("k_scale", "v_scale")]
    return torch.cat([k, v, *scales], 2)


CACHE = ("k_pages", "v_pages", "k_scale", "v_scale")


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("cu,lens", [
    ([0, 900, 1000, 0, 10], [900, 100, 40, 10]),      # the search ends at a sequence that lies further on
    ([0, 10, 700, 650, 990, 1000], [30, 700, 5, 400, 10]),
    ([500, 400, 300, 200, 900], [60, 60, 60, 700]),
    ([0, 1000, -7, 1000, 1 << 30, 1000], [1000, 9, 1000, 9, 9]),
])
def test_append_with_offsets_that_decrease(fa, cu, lens, page):
    T, Hkv, d = 1000, 2, 64
    b = c8.Batch8([0] * len(lens), lens, Hkv, d, page, torch.bfloat16, seed=page, spare=2)
    k, v = (torch.randn(T, Hkv, d, generator=b.g).bfloat16().cuda() for _ in range(2))
    before = {n: getattr(b, n).clone() for n in CACHE}
    offsets = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    got = {n: x.clone() for n, x in before.items()}
    fa.paged_append_fp8(k, v, *(got[n] for n in CACHE), b.block_table, offsets(cu), b.seq_lens)
    assert status(fa) == fa.FA_ERR_RANGE
    may = torch.zeros(got["k_pages"].shape[0], dtype=torch.bool, device="cuda")
    for i, n in enumerate(lens):
        if not 0 <= cu[i] < cu[i + 1] <= T:
            continue
        want = {m: x.clone() for m, x in before.items()}  # its own tokens alone, under offsets as they should be
        fa.paged_append_fp8(k, v, *(want[m] for m in CACHE), b.block_table[i:i + 1], offsets(cu[i:i + 2]), b.seq_lens[i:i + 1])
        assert status(fa) in (0, fa.FA_ERR_RANGE)  # (tokens before position 0)
        mine = b.block_table[i, :-(-n // page)].long()
        may[mine] = True
        x, y, old = held(got)[mine], held(want)[mine], held(before)[mine]
        # K and V of a page and head are units of their own: written whole, or passed over
        half = x.shape[2] // 2 - 4
        for part in (list(range(half)) + list(range(2 * half, 2 * half + 4)),
                     list(range(half, 2 * half)) + list(range(2 * half + 4, 2 * half + 8))):
            assert ((x[..., part] == y[..., part]).all(-1) | (x[..., part] == old[..., part]).all(-1)).all()
    assert torch.equal(held(got)[~may], held(before)[~may])


# total, budget, recent; with 45000 tokens and recent = budget no weight is looked at
@pytest.mark.parametrize("total,budget,recent", [(300, 100, 40), (300, 100, 100), (300, 100, 0), (45000, 100, 100),
                                                 (45000, 100, 30)])
@pytest.mark.parametrize("where", ["to", "between", "last"])
def test_eviction_reports_every_bad_page(fa, total, budget, recent, where):
    """A bad entry among the places that rows move to, among tokens that go, among the last ones: always reported, and
    what has no source or no place stays as it was."""
    page, Hkv = 16, 2
    b = c8.Batch8([0], [total], Hkv, 64, page, torch.float16, seed=total + recent, spread=1.0)
    w = torch.rand(b.k_pages.shape[0], Hkv, page, generator=b.g).cuda()
    at = {"to": 2, "between": 10, "last": (total - 1) // page}[where]
    was = int(b.block_table[0, at])
    b.block_table[0, at] = -1 if recent else b.k_pages.shape[0]
    before = {n: getattr(b, n).clone() for n in CACHE}
    before["w"] = w.clone()
    kept, lens = fa.paged_evict(b.k_pages, b.v_pages, w, b.block_table, b.seq_lens, budget, recent, k_scale=b.k_scale,
                                v_scale=b.v_scale)
    assert status(fa) == fa.FA_ERR_RANGE and lens.tolist() == [budget]
    kept, pages = kept[0].cpu().long(), b.block_table[0].cpu().long()
    assert (kept[:, 1:] > kept[:, :-1]).all() and (kept[:, budget - recent:] == torch.arange(total - recent, total)).all()
    now = {n: getattr(b, n) for n in CACHE}
    assert torch.equal(held(now)[was], held(before)[was]) and torch.equal(w[was], before["w"][was])
    for h in range(Hkv):
        for j, i in enumerate(kept[h].tolist()):
            to, src = int(pages[j // page]), int(pages[i // page])
            if j // page == at:
                continue  # no place
            moved = before["w"][src, h, i % page] if i // page != at else before["w"][to, h, j % page]
            assert w[to, h, j % page] == moved


def test_eviction_with_a_length_at_the_end_of_32_bits(fa):
    """A corrupt length over a table that covers 2^31 keys (all of its pages outside a cache without pages): cut, reported,
    and the steps over the positions stay within 32 bits."""
    empty = torch.empty(0, 1, 1 << 27, 64, dtype=torch.float16, device="cuda")
    table = torch.zeros(1, 16, dtype=torch.int32, device="cuda")
    lens = torch.tensor([0x7fffffff], dtype=torch.int32, device="cuda")
    kept, now = fa.paged_evict(empty, empty.clone(), torch.empty(0, 1, 1 << 27, device="cuda"), table, lens, 5, 2)
    assert status(fa) == fa.FA_ERR_RANGE
    assert kept[0, 0].tolist() == [0, 1, 2, 0x7fff0000 - 2, 0x7fff0000 - 1] and now.tolist() == [5]
