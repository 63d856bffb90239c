"""The decoder-block operators at the edges of what they accept."""
import math
import os
import subprocess
import sys

import pytest
import torch

from tests import decoder_testlib as lib

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_forward_02_gb300 as fa
    fa.fa_clear_status()
    yield fa
    assert fa.fa_last_status() == 0


def attend(fa, b, q, causal, **kw):
    return fa.attention_paged(q, b.k_pages, b.v_pages, b.block_table, b.cu_seqlens, b.seq_lens, b.max_q,
                              causal=causal, **kw)


def bits(x):
    return x.contiguous().view({2: torch.int16, 4: torch.int32}[x.element_size()])


# ---------------------------------------------------------------- scores that are not finite
# new, total, Hq, Hkv, d, page, table width: whole items with and without units, one sequence in parts,
# items over several SMs' ranges; single tokens and drafts (SPLIT, 4 to 1 copies of a row), chunks (PAIR)
KINDS = [
    ([1], [40], 8, 2, 128, 16, None),
    ([1, 3, 2], [300, 3, 512], 4, 1, 64, 16, None),
    ([1] * 200, [1 + (37 * i) % 300 for i in range(200)], 4, 2, 64, 32, None),
    ([1], [1001], 32, 8, 128, 16, None),
    ([1, 1, 1, 1], [3000, 20, 400, 2100], 8, 2, 64, 16, None),
    ([7, 9], [5000, 700], 6, 1, 128, 64, None),
    ([20], [9000], 4, 1, 128, 64, None),
    ([60, 1], [200, 2000], 4, 2, 128, 16, 200),
    ([300, 40], [300, 500], 4, 2, 64, 64, None),
    ([300], [6000], 4, 1, 128, 64, None),
    ([257, 100], [3000, 100], 6, 2, 64, 16, None),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,total,Hq,Hkv,d,page,wide", KINDS)
def test_a_nan_query_gives_nan_and_nothing_else_changes(fa, new, total, Hq, Hkv, d, page, wide, causal):
    """As in the dense kernels: a row whose scores are NaN is NaN in O and in L, whatever way its keys
    are shared out; O = 0 and L = -inf are for rows that see no key."""
    b = lib.Batch(new, total, Hkv, d, page, torch.bfloat16, seed=7, wide=wide)
    q = b.rows(Hq)
    want = attend(fa, b, q, causal)
    g = torch.Generator().manual_seed(3)
    hit = (torch.rand(q.shape[:2], generator=g) < 0.3).cuda()
    hit[0, 0] = hit[-1, -1] = True
    bad = q.clone()
    bad[hit] = math.nan
    one = torch.rand(q.shape[:2], generator=g).cuda() < 0.5   # one element of the row alone
    bad[hit & one] = q[hit & one]
    bad[hit & one, d // 2] = math.nan
    O, L = attend(fa, b, bad, causal)
    assert torch.isnan(O[hit]).all() and torch.isnan(L[hit]).all()
    assert torch.equal(O[~hit], want[0][~hit]) and torch.equal(L[~hit], want[1][~hit])


def test_rows_without_a_key_are_zero_whatever_the_query_holds(fa):
    """More new tokens than cached ones: the leading rows see nothing. Of an item in several parts, too."""
    for new, total, Hq in (([5, 700], [2, 300], 3), ([1, 2], [0, 1], 4), ([250], [180], 1), ([120], [100], 2)):
        b = lib.Batch(new, total, 1, 64, 16, torch.float16, seed=2, wide=300)
        q = b.rows(Hq)
        dead = torch.cat([torch.arange(n) < n - t for n, t in zip(new, total)]).cuda()
        q[:, 0] = math.nan
        O, L = attend(fa, b, q, True)
        assert not O[dead].any() and (L[dead] == -math.inf).all()
        assert torch.isnan(O[~dead][:, 0]).all() and torch.isnan(L[~dead][:, 0]).all()
        assert torch.isfinite(O[~dead][:, 1:]).all() and torch.isfinite(L[~dead][:, 1:]).all()


@pytest.mark.parametrize("new,total,Hq,Hkv,d,page,wide", KINDS)
def test_scores_past_32_bits_are_not_the_result_of_no_key(fa, new, total, Hq, Hkv, d, page, wide):
    """q.k beyond fp32: no weights can be had, so O is NaN; below -fp32's largest L rounds to -inf."""
    b = lib.Batch(new, total, Hkv, d, page, torch.bfloat16, seed=7, wide=wide)
    for x in (b.k_pages, b.v_pages):
        x.abs_().add_(0.5)
    q = b.rows(Hq)
    want = attend(fa, b, q, True)
    bad = q.clone()
    bad[0, 0], bad[-1, -1] = 3e38, -3e38
    O, L = attend(fa, b, bad, True)
    assert torch.isnan(O[0, 0]).all() and not L[0, 0] == -math.inf
    if q.shape[0] * q.shape[1] > 1:
        assert torch.isnan(O[-1, -1]).all() and not torch.isfinite(L[-1, -1])
    same = torch.ones(q.shape[:2], dtype=torch.bool, device="cuda")
    same[0, 0] = same[-1, -1] = False
    assert torch.equal(O[same], want[0][same]) and torch.equal(L[same], want[1][same])


# ------------------------------------------------------------------- tokens without a position
@pytest.mark.parametrize("d,Hq,Hk", [(64, 2, 1), (128, 3, 2), (64, 1, 1)])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
def test_padding_rows_add_nothing_to_the_weights_gradients(fa, d, Hq, Hk, eps):
    """Rows whose position is outside the table may hold anything, zeros with eps = 0 too."""
    N = 11
    g = torch.Generator().manual_seed(0)
    q, k, gq, gk = (torch.randn(1, N, H, d, generator=g).bfloat16().cuda() for H in (Hq, Hk, Hq, Hk))
    wq, wk = ((1 + 0.1 * torch.randn(d, generator=g)).bfloat16().cuda() for _ in range(2))
    table = lib.rope_table(20, d).cuda()
    pos = torch.tensor([[3, -1, 0, 20, 5, 6, 7, -9, 8, 9, 1000]], dtype=torch.int32).cuda()
    good = (pos[0] >= 0) & (pos[0] < 20)
    zeroed = [x.clone() for x in (gq, gk)]
    for x in zeroed:
        x[:, ~good] = 0
    clean = fa.qk_norm_rope_backward(*zeroed, q, k, wq, wk, table, pos, eps)
    for fill in (math.nan, math.inf, -math.inf, 0.0, 3e38):
        for x in (q, k, gq, gk):
            x[:, ~good] = fill
        out = [torch.full_like(x, 7.0) for x in (q, k)]
        got = fa.qk_norm_rope_backward(gq, gk, q, k, wq, wk, table, pos, eps, dq=out[0], dk=out[1])
        assert fa.fa_last_status() == fa.FA_ERR_RANGE
        fa.fa_clear_status()
        for x, y in zip(got[2:], clean[2:]):
            assert torch.isfinite(x).all() and torch.equal(x, y)
        for x, y in zip(got[:2], clean[:2]):
            assert torch.equal(x[:, good], y[:, good]) and (x[:, ~good] == 7).all()


def test_more_tokens_than_the_table_has_rows_are_refused(fa):
    """Without positions token n takes row n: the host knows that some have none."""
    q, w = torch.randn(2, 9, 2, 64).half().cuda(), torch.ones(64).half().cuda()
    table = lib.rope_table(8, 64).cuda()
    for call in (lambda: fa.qk_norm_rope(q, q, w, w, table), lambda: fa.qk_norm_rope_backward(q, q, q, q, w, w, table)):
        with pytest.raises(fa.FAError) as e:
            call()
        assert e.value.code == fa.FA_ERR_RANGE
    fa.qk_norm_rope(q[:, :8], q[:, :8], w, w, table)
    assert fa.fa_last_status() == 0


def test_a_table_without_rows_is_a_table(fa):
    """Every position is outside of it: reported, nothing written; no unrotated results."""
    empty = torch.zeros(0, 64, device="cuda")
    q, w = torch.randn(1, 3, 2, 64).half().cuda(), torch.ones(64).half().cuda()
    pos = torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    out = [torch.full_like(q, 7.0) for _ in range(2)]
    fa.qk_norm_rope(q, q, w, w, empty, pos, q_out=out[0], k_out=out[1])
    assert fa.fa_last_status() == fa.FA_ERR_RANGE
    fa.fa_clear_status()
    grads = fa.qk_norm_rope_backward(q, q, q, q, w, w, empty, pos, dq=out[0], dk=out[1])
    assert fa.fa_last_status() == fa.FA_ERR_RANGE
    fa.fa_clear_status()
    assert all((x == 7).all() for x in out) and not grads[2].any() and not grads[3].any()
    b = lib.Batch([1, 2], [5, 20], 2, 64, 16, torch.float16, fill=5.0)
    k, before = b.rows(2), b.k_pages.clone()
    fa.paged_append(k, k, b.k_pages, b.v_pages, b.block_table, b.cu_seqlens, b.seq_lens, rope=empty)
    assert fa.fa_last_status() == fa.FA_ERR_RANGE
    fa.fa_clear_status()
    assert torch.equal(b.k_pages, before)
    none = q[:, :0]
    fa.qk_norm_rope(none, none, w, w, empty, pos[:, :0])  # no tokens: nothing to report
    assert fa.fa_last_status() == 0


# ---------------------------------------------------------- elements that the rotation leaves out
SPECIAL = [math.inf, -math.inf, math.nan, -0.0, 0.0, 65504.0, -1.0]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("d,rot", [(64, 16), (64, 48), (128, 64), (128, 112)])
def test_elements_behind_the_rotation_are_copied(fa, d, rot, interleaved, dtype):
    """Bit by bit, whatever stands beside them."""
    b = lib.Batch([40, 1, 7], [40, 90, 30], 3, d, 16, lib.DTYPES[dtype], fill=5.0)
    k, v = b.rows(3), b.rows(3)
    g = torch.Generator().manual_seed(1)
    rest = k[..., rot:]
    pick = torch.randint(0, 2 * len(SPECIAL), rest.shape, generator=g).cuda()
    values = torch.tensor(SPECIAL, dtype=torch.float32).to(k.dtype).cuda()
    rest.copy_(torch.where(pick < len(SPECIAL), values[pick.clamp(max=len(SPECIAL) - 1)], rest))
    fa.paged_append(k, v, b.k_pages, b.v_pages, b.block_table, b.cu_seqlens, b.seq_lens,
                    rope=lib.rope_table(100, rot).cuda(), interleaved=interleaved)
    assert fa.fa_last_status() == 0
    for i, n in enumerate(b.new):
        got = b.cached(i)[0][:, b.total[i] - n:].transpose(0, 1)
        rows = k[b.cu[i]:b.cu[i] + n]
        assert torch.equal(bits(got[..., rot:]), bits(rows[..., rot:]))
        assert torch.isfinite(got[..., :rot]).all()


@pytest.mark.parametrize("interleaved", [True, False])
def test_gradients_behind_the_rotation_stay_in_their_places(fa, interleaved):
    """An infinite gradient of one element that is not rotated: the weights' gradients of its neighbours
    do not see it (u = g w couples the elements of dx, not those of dw)."""
    d, rot = 64, 16
    x, g = (torch.randn(1, 5, 2, d).bfloat16().cuda() for _ in range(2))
    w = torch.ones(d).bfloat16().cuda()
    table, none = lib.rope_table(5, rot).cuda(), x[:, :, :0]
    clean = fa.qk_norm_rope_backward(g, none, x, none, w, w, table, interleaved=interleaved)[2]
    g[0, 2, 1, 41] = math.inf
    got = fa.qk_norm_rope_backward(g, none, x, none, w, w, table, interleaved=interleaved)[2]
    keep = torch.arange(d) != 41
    assert not torch.isfinite(got[41]) and torch.equal(got[keep], clean[keep])


# ------------------------------------------------------------------------- rows of no sequence
@pytest.mark.parametrize("cu,fine", [
    ([0, 2, 5, 9], (0, 1)), ([-1, 2, 5, 7], (1, 2)), ([0, 9, 9, 9], ()), ([-5, -2, 0, 7], (2,)),
    ([0, 2, 5, 7], (0, 1, 2)),
    # decreasing
    ([0, -4, 5, 7], (2,)), ([0, 5, 2, 7], (0, 2)), ([0, 2, 8, 7], (0,)), ([3, 2, 5, 7], (1, 2)), ([7, 5, 2, 0], ())])
@pytest.mark.parametrize("d", [64, 128])
def test_append_passes_over_rows_outside_the_packed_tokens(fa, cu, fine, d):
    """cu_seqlens that leave [0, T] or decrease: as in the attention such a sequence is passed over and
    reported. Nothing is written but a sequence's own tokens in their own places; where no offset
    decreases, all of the others' are."""
    b = lib.Batch([2, 3, 2], [40, 300, 9], 2, d, 16, torch.float16, fill=5.0, wide=25)
    b.block_table[b.block_table < 0] = b.k_pages.shape[0] - 1  # entries behind a sequence: nobody's page
    k, was = b.rows(2), (b.k_pages.clone(), b.v_pages.clone())
    b.cu_seqlens.copy_(torch.tensor(cu, dtype=torch.int32))
    fa.paged_append(k, k, b.k_pages, b.v_pages, b.block_table, b.cu_seqlens, b.seq_lens)
    assert fa.fa_last_status() == (0 if len(fine) == 3 else fa.FA_ERR_RANGE)
    fa.fa_clear_status()
    for pages, before in zip((b.k_pages, b.v_pages), was):
        full = before.clone()
        for i in fine:
            for t in range(cu[i], cu[i + 1]):
                pos = b.total[i] - (cu[i + 1] - t)
                full[b.block_table[i, pos // 16].long(), :, pos % 16] = k[t]
        if cu == sorted(cu):
            assert torch.equal(pages, full)
        assert ((pages == before) | (pages == full)).all()


def test_append_finds_a_bad_offset_among_many(fa):
    """The offsets of 3000 sequences, one of them past the rows."""
    new = [1] * 3000
    b = lib.Batch(new, [1 + i % 20 for i in range(3000)], 1, 64, 16, torch.float16, fill=5.0)
    k = b.rows(1)
    for at in (0, 1500, 3000):
        before, good = b.k_pages.clone(), b.cu_seqlens.clone()
        b.cu_seqlens[at] = 3001
        fa.paged_append(k, k, b.k_pages, b.v_pages, b.block_table, b.cu_seqlens, b.seq_lens)
        assert fa.fa_last_status() == fa.FA_ERR_RANGE
        fa.fa_clear_status()
        full = before.clone()
        at_pos = torch.tensor(b.total, device="cuda") - 1
        full[b.block_table.long().gather(1, (at_pos // 16)[:, None])[:, 0], :, at_pos % 16] = k
        assert ((b.k_pages == before) | (b.k_pages == full)).all()
        b.cu_seqlens.copy_(good)
        fa.paged_append(k, k, b.k_pages, b.v_pages, b.block_table, b.cu_seqlens, b.seq_lens)
        assert fa.fa_last_status() == 0 and torch.equal(b.k_pages, full)
        b.k_pages.copy_(before)


# ---------------------------------------------------------------------- the manner of the calls
def test_inputs_that_require_gradients_are_refused_where_they_would_be_lost(fa):
    """The calls are not recorded by autograd: an input that requires a gradient must come without
    grad mode (or detached), so that its gradient is not lost unseen."""
    q, w = torch.randn(1, 3, 2, 64).half().cuda(), torch.ones(64).half().cuda()
    b = lib.Batch([2, 1], [20, 3], 2, 64, 16, torch.float16)
    rows = b.rows(4)
    table = (b.block_table, b.cu_seqlens, b.seq_lens)
    calls = [lambda x: fa.qk_norm_rope(x(q), q, w, w), lambda x: fa.qk_norm_rope(q, q, w, x(w)),
             lambda x: fa.attention_paged(x(rows), b.k_pages, b.v_pages, *table, 2),
             lambda x: fa.attention_paged(rows, b.k_pages, x(b.v_pages), *table, 2),
             lambda x: fa.paged_append(x(rows[:, :2]), rows[:, :2], b.k_pages, b.v_pages, *table)]
    for call in calls:
        with pytest.raises(ValueError, match="grad"):
            call(lambda t: t.detach().clone().requires_grad_())
        call(lambda t: t)
        with torch.no_grad():
            call(lambda t: t.detach().requires_grad_())
        with torch.inference_mode():
            call(lambda t: t)
    leaf = w.clone().requires_grad_()   # gradients from the call that computes them
    assert fa.qk_norm_rope_backward(q, q, q, q, leaf, leaf)[2].shape == (64,)


def test_an_allocation_that_fails_raises_torch_s_own_error(fa):
    """Out of memory is torch.cuda.OutOfMemoryError, which a server catches."""
    q, w = torch.randn(1, 1, 8, 128).half().cuda(), torch.ones(128).half().cuda()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (64 << 20)) / total)
    try:
        big = q.expand(1, 1 << 18, 8, 128)  # 512 MB of outputs
        with pytest.raises(torch.cuda.OutOfMemoryError):
            fa.qk_norm_rope(big, big, w, w)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert fa.qk_norm_rope(q, q, w, w)[0].shape == q.shape


def test_a_first_call_inside_a_capture():
    """A process whose first call of each operator is captured."""
    code = """
import torch
from tests import decoder_testlib as lib
import exact_attention_forward_02_gb300 as fa
b = lib.Batch([1, 1, 1], [3000, 900, 50], 2, 128, 16, torch.bfloat16, seed=1)
q, k = b.rows(8), b.rows(2)
w = torch.ones(128).bfloat16().cuda()
table = lib.rope_table(3000, 128).cuda()
pos = (b.seq_lens - 1)[None].contiguous()
torch.cuda.synchronize()
def step():
    x, y = fa.qk_norm_rope(q[None], k[None], w, w, table, pos)
    back = fa.qk_norm_rope_backward(x, y, q[None], k[None], w, w, table, pos)
    fa.paged_append(y[0], k, b.k_pages, b.v_pages, b.block_table, b.cu_seqlens, b.seq_lens)
    return (*back, *fa.attention_paged(x[0], b.k_pages, b.v_pages, b.block_table, b.cu_seqlens, b.seq_lens, 1))
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = step()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(got, step()))
assert fa.fa_last_status() == 0
print("captured first")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


def test_rows_past_the_range_of_the_sum_of_squares(fa):
    """As the header says: a mean square beyond fp32 gives zeros, zeros with eps = 0 give NaN; other rows
    are what they are without them."""
    q = torch.randn(1, 6, 2, 64).bfloat16().cuda()
    w, table = torch.ones(64).bfloat16().cuda(), lib.rope_table(6, 64).cuda()
    for eps in (1e-6, 0.0):
        want = fa.qk_norm_rope(q, q, w, w, table, eps=eps)[0]
        x = q.clone()
        x[0, 1], x[0, 4, 0] = 3e38, 0
        y = fa.qk_norm_rope(x, x, w, w, table, eps=eps)[0]
        assert not y[0, 1].any()
        assert torch.isnan(y[0, 4, 0]).all() if eps == 0 else not y[0, 4, 0].any()
        assert torch.equal(y[0, [0, 2, 3, 5]], want[0, [0, 2, 3, 5]]) and torch.equal(y[0, 4, 1], want[0, 4, 1])


@pytest.mark.parametrize("B,new,total,Hkv,d", [(1, 27000, 40000, 8, 128), (100, 20, 16640, 8, 64)])
def test_long_items_under_the_smallest_wait_limit(fa, B, new, total, Hkv, d):
    """Several items a block, each of a hundred tiles and more: a wait for a whole item is not a step of the
    pipeline, which the limit is for. (Sequences share their pages, as those of a common prefix do.)"""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    q = torch.randn(B * new, Hkv, d, generator=g, device="cuda", dtype=torch.bfloat16)
    k, v = (torch.randn(total // 64, Hkv, 64, d, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    table = torch.arange(total // 64, dtype=torch.int32, device="cuda").repeat(B, 1)
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * new
    lens = torch.full((B,), total, dtype=torch.int32, device="cuda")
    want = fa.attention_paged(q, k, v, table, cu, lens, 4096)
    torch.cuda.synchronize()
    try:
        assert fa.fa_set_wait_limit_us(100) == fa.FA_OK
        got = fa.attention_paged(q, k, v, table, cu, lens, 4096)
    finally:
        fa.fa_set_wait_limit_us(fa.FA_WAIT_LIMIT_DEFAULT_US)
    assert fa.fa_last_status() == 0
    assert torch.isfinite(want[0]).all() and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
