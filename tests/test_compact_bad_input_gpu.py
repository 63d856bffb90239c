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
