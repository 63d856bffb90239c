"""Scales of 8-bit pages in an eviction: pages of zeros (scale 0, whatever their bytes), pages larger than the tokens that a
block looks at in one go."""
import pytest
import torch

from tests import compact_testlib as c8
from tests.test_evict_gpu import check_evict, fa, weights_for  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page,budget,recent", [(16, 200, 30), (64, 333, 0), (8, 100, 100)])
def test_pages_of_zeros(fa, page, budget, recent):  # noqa: F811
    """A row from a page with scale 0 is a row of zeros afterwards too, also where all of a page's rows are."""
    b = c8.Batch8([0, 0], [900, 600], 2, 64, page, torch.bfloat16, seed=page, spread=1.0)
    w = weights_for(b, page)
    for i, t in enumerate(b.total):
        pages = b.block_table[i, :-(-t // page)].long()
        for s, every in ((b.k_scale, 3), (b.v_scale, 2)):
            s[pages[::every], 0] = 0.0
        w[pages[2::5], 1] = 100.0  # whole runs of what stays come from pages of zeros
        b.k_scale[pages[2::5], 1] = 0.0
    old = {n: (getattr(b, n + "_pages").clone(), getattr(b, n + "_scale").clone()) for n in "kv"}
    kept, _ = fa.paged_evict(b.k_pages, b.v_pages, w, b.block_table, b.seq_lens, budget, recent, k_scale=b.k_scale,
                             v_scale=b.v_scale)
    assert fa.fa_last_status() == 0
    zeros = 0
    for i in range(2):
        table, to = b.block_table[i].long(), torch.arange(budget, device="cuda")
        for h in range(2):
            src = kept[i, h].long()
            for n in "kv":
                codes, scale = old[n]
                came = scale[table[src // page], h].double()
                want = codes.view(torch.uint8)[table[src // page], h, src % page].view(c8.E4M3).double() * came[:, None]
                now = torch.nn.functional.pad(came, (0, -budget % page)).view(-1, page).amax(1)
                scale = getattr(b, n + "_scale")[table[to[::page] // page], h].double()
                assert torch.equal(scale, now)
                zeros += int((now == 0).sum())
                got = getattr(b, n + "_pages").view(torch.uint8)[table[to // page], h, to % page].view(c8.E4M3).double()
                unit = scale[to // page][:, None]
                assert ((got * unit - want).abs() <= c8.HALF8 * want.abs() + c8.TINY8 * unit).all()
    assert zeros or page == 64


@pytest.mark.parametrize("page,total,budget,recent", [(16384, 40000, 20000, 1000), (8192, 20000, 9000, 9000),
                                                      (12288, 30000, 29999, 5)])
def test_large_pages(fa, page, total, budget, recent):  # noqa: F811
    b = c8.Batch8([0], [total], 1, 64, page, torch.bfloat16, seed=page, spread=2.0)
    check_evict(fa, b, weights_for(b), budget, recent)
