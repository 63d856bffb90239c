"""The ends of ranges of the operators of a compact cache that the host looks at (fake pointers, no CUDA call)."""
import pytest
import torch

import exact_attention_forward_02_gb300 as fa
from tests.test_compact_cpu import weigh
from tests.test_decoder_cpu import cache, heads


@pytest.mark.parametrize("Hkv,code", [(64, "FA_ERR_SHAPE"), (63, "FA_ERR_NULL")])
def test_weights_of_a_page_stay_below_2_to_the_32(Hkv, code):
    """64 heads of 2^26 tokens are refused; 63 pass that check and come to the next one."""
    rc = weigh(kv=cache(Hkv=Hkv, page=1 << 26), q=heads(H=Hkv), L=None)
    assert rc == getattr(fa, code), fa.strerror(rc)


def test_eviction_from_a_cache_without_heads_is_refused():
    """The lengths that it would return would be anything: nothing is launched for such a cache."""
    pages = torch.zeros(3, 0, 16, 64, dtype=torch.float16)
    table, lens = torch.zeros(2, 1, dtype=torch.int32), torch.tensor([9, 3], dtype=torch.int32)
    with pytest.raises(ValueError, match="heads"):
        fa.paged_evict(pages, pages.clone(), torch.zeros(3, 0, 16), table, lens, 4, 1)
