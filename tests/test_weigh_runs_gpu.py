"""The key weights of batches in which the second warpgroup of a block pauses: units of two key tiles, then runs of units of
one, whose rows differ much, so that what belongs to other rows would show."""
import pytest
import torch

from tests.test_evict_gpu import batch, check_weigh, fa, weights_for  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("held8", [False, True])
@pytest.mark.parametrize("d,Hkv,group,new", [(64, 2, 1, 1), (128, 2, 4, 3), (64, 1, 16, 1), (128, 1, 8, 20)])
def test_pauses_of_the_second_warpgroup(fa, held8, d, Hkv, group, new):  # noqa: F811
    total = [new + (230 if i % 14 < 1 + i // 14 % 3 else 30 + i % 90) for i in range(1400)]
    b = batch(held8, [new] * len(total), total, Hkv, d, 32, torch.bfloat16, seed=d + group)
    q = b.rows(Hkv * group) * (0.25 + 3 * torch.rand(b.T, 1, 1, generator=b.g).cuda()).bfloat16()
    first = check_weigh(fa, b, q, True)
    _, lse = (fa.attention_paged_fp8(q, b.k_pages, b.v_pages, b.k_scale, b.v_scale, b.block_table, b.cu_seqlens,
                                     b.seq_lens, b.max_q) if held8 else
              fa.attention_paged(q, b.k_pages, b.v_pages, b.block_table, b.cu_seqlens, b.seq_lens, b.max_q))
    runs = []
    for _ in range(8):
        w = weights_for(b)
        fa.paged_key_weights(q, lse, b.k_pages, w, b.block_table, b.cu_seqlens, b.seq_lens, b.max_q,
                             k_scale=getattr(b, "k_scale", None))
        runs.append(w)
    assert all(torch.equal(w, runs[0]) for w in runs[1:]) and first.shape == runs[0].shape
