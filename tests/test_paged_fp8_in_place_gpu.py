"""Attention over an 8-bit cache in forms that the library's contract allows: its output over the queries themselves, queries
that all heads share (strides of zero), two sequences with the same pages in front."""
import pytest
import torch

from tests import compact_testlib as c8

pytestmark = pytest.mark.gpu
FORMS = [  # new, total, Hq, Hkv, d: single tokens whole and cut, drafts, many rows, chunks
    ([1], [9000], 32, 8, 128), ([1] * 40, [2000] * 40, 8, 2, 64), ([3, 1, 2], [5000, 700, 400], 8, 2, 128),
    ([30, 1], [5000, 4000], 4, 4, 64), ([300, 40, 0], [3000, 500, 9], 4, 2, 64), ([2000], [2500], 6, 2, 128),
]


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_forward_02_gb300 as fa
    fa.fa_clear_status()
    return fa


def attend(fa, b, q, **kw):
    got = fa.attention_paged_fp8(q, b.k_pages, b.v_pages, b.k_scale, b.v_scale, b.block_table, b.cu_seqlens, b.seq_lens,
                                 b.max_q, **kw)
    assert fa.fa_last_status() == 0
    return got


@pytest.mark.parametrize("new,total,Hq,Hkv,d", FORMS)
def test_output_over_the_queries(fa, new, total, Hq, Hkv, d):
    b = c8.Batch8(new, total, Hkv, d, 16, torch.bfloat16, seed=d)
    q = b.rows(Hq)
    want = attend(fa, b, q)
    for _ in range(5):
        x = q.clone()
        O, L = attend(fa, b, x, out=x)
        assert O.data_ptr() == x.data_ptr() and torch.equal(O, want[0]) and torch.equal(L, want[1])


@pytest.mark.parametrize("new,total,Hq,Hkv,d", FORMS)
def test_queries_that_heads_share(fa, new, total, Hq, Hkv, d):
    b = c8.Batch8(new, total, Hkv, d, 16, torch.float16, seed=d)
    q = b.rows(1).expand(-1, Hq, -1)
    got, want = attend(fa, b, q), attend(fa, b, q.contiguous())
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("new", [1, 3, 50])
def test_pages_that_sequences_share(fa, new):
    """A common beginning: the second sequence's table names the first one's pages for its first 320 tokens; new tokens go
    to pages of their own."""
    b = c8.Batch8([new, new], [700, 500], 2, 64, 16, torch.bfloat16, seed=new)
    b.block_table[1, :20] = b.block_table[0, :20]
    b.decode()
    k, v, q = b.rows(2), b.rows(2), b.rows(8)
    shared = b.block_table[0, :20].long()
    before = [x.view(torch.uint8)[shared].clone() for x in (b.k_pages, b.v_pages, b.k_scale, b.v_scale)]
    fa.paged_append_fp8(k, v, b.k_pages, b.v_pages, b.k_scale, b.v_scale, b.block_table, b.cu_seqlens, b.seq_lens)
    assert all(torch.equal(x.view(torch.uint8)[shared], y) for x, y in zip((b.k_pages, b.v_pages, b.k_scale, b.v_scale), before))
    b.decode()
    O, L = attend(fa, b, q)
    want, lse, tol_o, tol_l = c8.attend64(b, q, 0.125, True)
    assert ((O.double() - want).abs() <= tol_o).all() and ((L.double() - lse).abs() <= tol_l).all()
