"""Places of a compact cache that only pages past 32 bits have, against the same call over a small cache."""
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


@pytest.mark.parametrize("group,new", [(1, 2), (8, 4)])
def test_key_weights_of_a_page_of_more_than_2_to_the_31(fa, group, new):
    """17 heads of a page of 2^27 tokens: the last head's weights begin 2^31 places into the page. (The keys are a view whose
    heads lie closer than a page is long: only its first tokens are in use.)"""
    Hkv, page, far, total, d = 17, 512, 1 << 27, 300, 64
    b = c8.Batch8([new], [total], Hkv, d, page, torch.bfloat16, seed=group, spare=0)
    q = b.rows(Hkv * group)
    ids = (b.cu_seqlens, b.seq_lens)
    _, lse = fa.attention_paged_fp8(q, b.k_pages, b.v_pages, b.k_scale, b.v_scale, b.block_table, *ids, new)
    want = torch.rand(1, Hkv, page, generator=b.g).cuda()
    big = torch.empty(1, Hkv, far, device="cuda")
    big[:, :, :page] = want
    fa.paged_key_weights(q, lse, b.k_pages, want, b.block_table, *ids, new, k_scale=b.k_scale)
    memory = torch.empty(far * d + Hkv * page * d, dtype=torch.uint8, device="cuda")
    keys = memory.as_strided((1, Hkv, far, d), (memory.numel(), page * d, d, 1))
    keys[:, :, :page] = b.k_pages.view(torch.uint8)
    fa.paged_key_weights(q, lse, keys.view(c8.E4M3), big, b.block_table, *ids, new, k_scale=b.k_scale)
    assert fa.fa_last_status() == 0
    assert torch.equal(big[:, :, :page], want)
