"""fa_paged_append and fa_fwd_paged against their definitions in 64 bits."""
import math

import pytest
import torch

from tests import decoder_testlib as lib

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
    return fa.attention_paged(q, b.k_pages, b.v_pages, b.block_table, b.cu_seqlens, b.seq_lens, b.max_q,
                              causal=causal, **kw)


def check(fa, b, q, causal, scale=None, **kw):
    scale = 1 / math.sqrt(b.d) if scale is None else scale
    O = torch.full_like(q, 99.0) if "out" not in kw else kw.pop("out")
    L = torch.full(q.shape[:2], 99.0, device="cuda")
    attend(fa, b, q, causal, scale=scale, out=O, lse=L, **kw)
    want_o, want_l, tol_o, tol_l = lib.attend64(b, q, scale, causal)
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


# new tokens and totals of the sequences; Hq, Hkv, d, page
SHAPES = [
    ([1], [1], 1, 1, 64, 8),
    ([1], [17], 8, 1, 128, 16),
    ([1, 1, 1], [127, 128, 129], 8, 8, 64, 16),
    ([1, 0, 1, 1], [300, 50, 0, 1000], 32, 8, 128, 16),
    ([1] * 9, [5, 64, 200, 511, 512, 513, 1, 2, 1500], 12, 4, 128, 64),
    ([3, 1, 8, 0, 5], [3, 700, 8, 9, 130], 10, 2, 64, 32),
    ([1, 2], [4097, 2], 5, 1, 128, 128),
    ([16, 33], [16, 200], 7, 7, 128, 256),
    ([100, 1, 257], [100, 1, 1000], 6, 2, 64, 16),
    ([128, 129, 127], [500, 129, 3000], 8, 1, 128, 64),
    ([1000], [1000], 4, 4, 128, 32),
    ([5, 700], [2, 300], 3, 1, 64, 8),            # fewer cached than new: leading rows see nothing
    ([1, 1], [9000, 20], 128, 1, 128, 384),
    ([2, 300], [2000, 301], 96, 1, 64, 64),
    ([7] * 40, list(range(7, 407, 10)), 16, 8, 64, 16),
    ([1] * 200, [1 + (37 * i) % 211 for i in range(200)], 4, 4, 64, 32),
    ([2048, 1], [2500, 5000], 16, 2, 128, 64),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,total,Hq,Hkv,d,page", SHAPES)
def test_attention(fa, new, total, Hq, Hkv, d, page, causal):
    dtype = torch.bfloat16 if (Hq + len(new)) % 2 else torch.float16
    b = lib.Batch(new, total, Hkv, d, page, dtype, seed=Hq, token_major=page == 64, lead=2, behind=3)
    check(fa, b, b.rows(Hq), causal)


@pytest.mark.parametrize("B", [31, 32, 33, 255, 256, 257, 700])
def test_many_sequences_some_without_tokens(fa, B):
    """The share of each SM is found from the lengths by one warp or by the whole block."""
    new = [(0, 1, 1, 3, 0)[i % 5] for i in range(B)]
    total = [n + (i * 53) % 400 for i, n in enumerate(new)]
    b = lib.Batch(new, total, 2, 64, 16, torch.bfloat16, seed=B, lead=1)
    check(fa, b, b.rows(4), True)
    new = [(0, 40, 1)[i % 3] for i in range(B)]
    b = lib.Batch(new, [n + (i * 37) % 90 for i, n in enumerate(new)], 1, 64, 16, torch.float16, seed=B)
    check(fa, b, b.rows(8), True)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
def test_types_and_sharp_scores(fa, d, dtype):
    """Scores spread over tens: the running maximum moves often and by much."""
    b = lib.Batch([1, 200, 6], [900, 1200, 6], 2, d, 16, lib.DTYPES[dtype], seed=3)
    q = b.rows(8, std=6.0)
    check(fa, b, q, True)
    check(fa, b, q, False, scale=0.0)   # all weights the same
    check(fa, b, q, True, scale=1e-3)


def test_descending_and_ascending_scores(fa):
    """Keys whose scores grow along the sequence (every tile moves the maximum), then fall."""
    for sign in (1.0, -1.0):
        b = lib.Batch([1, 130], [1300, 1300], 1, 128, 32, torch.bfloat16, seed=5)
        q = b.rows(4)
        for i, keys in enumerate(b.keys):
            t = torch.arange(1300, device="cuda") * (sign * 0.05)
            unit = q[b.cu[i]].float().mean(0)
            keys.copy_((keys.float() * 0.1 + t[None, :, None] * (unit / unit.norm())).to(keys.dtype))
            for j in range(b.block_table.shape[1]):
                n = min(32, 1300 - 32 * j)
                if n > 0:
                    b.k_pages[b.block_table[i, j].long(), :, :n] = keys[:, 32 * j:32 * j + n]
        check(fa, b, q, True)


def test_strided_queries_and_outputs(fa):
    """q as a slice of a fused projection, O head-major."""
    b = lib.Batch([4, 90], [60, 300], 2, 64, 16, torch.bfloat16)
    fused = b.rows(6 + 2 * 2)
    out = torch.full((6, b.T, 64), 99.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    check(fa, b, fused[:, :6], True, out=out)


def test_output_over_the_queries(fa):
    b = lib.Batch([3, 1, 200, 1], [3, 900, 700, 4000], 2, 128, 16, torch.float16)
    for rows in (b.rows(8), b.rows(12)[:, 4:]):
        want = attend(fa, b, rows, True)
        got = attend(fa, b, rows, True, out=rows)
        assert got[0] is rows or got[0].data_ptr() == rows.data_ptr()
        assert torch.equal(rows, want[0]) and torch.equal(got[1], want[1])


def test_rows_outside_the_packed_tokens_are_passed_over(fa):
    """cu_seqlens that decrease, or run past T: those sequences are skipped and reported."""
    b = lib.Batch([2, 3, 2], [40, 300, 9], 2, 64, 16, torch.float16)
    q = b.rows(4)
    want = attend(fa, b, q, True)
    out = torch.full_like(q, 7.0)
    b.cu_seqlens[3] = 9                    # the last sequence would end behind T = 7
    attend(fa, b, q, True, out=out)
    assert fa.fa_last_status() == fa.FA_ERR_RANGE
    fa.fa_clear_status()
    assert torch.equal(out[:5], want[0][:5]) and (out[5:] == 7).all()
    b.cu_seqlens[3], b.cu_seqlens[1] = 7, -4
    out.fill_(7.0)
    attend(fa, b, q, True, out=out)
    assert fa.fa_last_status() == fa.FA_ERR_RANGE
    fa.fa_clear_status()
    assert torch.equal(out[5:], want[0][5:]) and (out[:5] == 7).all()
    b.cu_seqlens[1], b.seq_lens[0] = 2, -5  # no keys at all
    got = attend(fa, b, q, True)
    assert not got[0][:2].any() and torch.isinf(got[1][:2]).all() and torch.equal(got[0][2:], want[0][2:])


def test_results_do_not_change_from_run_to_run(fa):
    b = lib.Batch([1] * 5 + [70], [3000, 20, 400, 1, 700, 2000], 4, 128, 16, torch.bfloat16)
    q = b.rows(16)
    first = attend(fa, b, q, True)
    for _ in range(3):
        again = attend(fa, b, q, True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("new,total,Hq,Hkv,d", [
    ([200], [1500], 4, 2, 64), ([70, 300], [80, 500], 4, 2, 128), ([9, 0, 40], [400, 100, 41], 6, 1, 64),
    ([500], [512], 8, 1, 128), ([129], [129], 1, 1, 64)])
def test_small_batches_shared_out_without_units(fa, new, total, Hq, Hkv, d):
    """One sequence, or whole items: every max_q, too small ones too."""
    b = lib.Batch(new, total, Hkv, d, 16, torch.bfloat16, seed=d)
    q = b.rows(Hq)
    for b.max_q in (1, 3, 30, 64, 300, 5000):
        check(fa, b, q, True)
        check(fa, b, q, False)


def test_max_q_is_a_hint(fa):
    """A batch with more new tokens than max_q says, and one with far fewer, are still right."""
    b = lib.Batch([150, 1, 40], [600, 300, 41], 2, 64, 32, torch.float16)
    q = b.rows(8)
    for hint in (1, 4, 1000):
        b.max_q = hint
        check(fa, b, q, True)


def test_many_pieces_of_one_row(fa):
    """One sequence and one key head: every SM takes a part of the same rows."""
    b = lib.Batch([1], [70000], 1, 128, 128, torch.bfloat16)
    check(fa, b, b.rows(8), True)
    b = lib.Batch([9], [50000], 1, 64, 16, torch.float16)
    check(fa, b, b.rows(2), True)
    b = lib.Batch([64], [30000], 1, 128, 64, torch.bfloat16)
    check(fa, b, b.rows(8), True)


def test_offsets_past_32_bits(fa):
    """Pages whose elements lie more than 2^31 elements behind the cache's start."""
    Hkv, d, page, far = 2, 128, 64, 140_000
    big = torch.empty(2, far, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    b = lib.Batch([2, 1], [150, 64], Hkv, d, page, torch.bfloat16)
    moved = b.block_table.clone()
    for i in range(2):
        for j in range(-(-b.total[i] // page)):
            old = int(b.block_table[i, j])
            moved[i, j] = far - 1 - old
            big[0, far - 1 - old], big[1, far - 1 - old] = b.k_pages[old], b.v_pages[old]
    b.block_table, b.k_pages, b.v_pages = moved, big[0], big[1]
    assert moved.max() * Hkv * page * d > 2 ** 31
    check(fa, b, b.rows(4), True)
    k, v = b.rows(Hkv), b.rows(Hkv)
    fa.paged_append(k, v, b.k_pages, b.v_pages, b.block_table, b.cu_seqlens, b.seq_lens)
    assert torch.equal(b.cached(0)[0][:, -2:], k[:2].transpose(0, 1))
    assert torch.equal(b.cached(1)[1][:, -1:], v[2:].transpose(0, 1))


def test_a_page_outside_the_cache_is_reported(fa):
    """Reads as zeros: the other sequences are as if nothing had been."""
    b = lib.Batch([1, 1, 60], [40, 90, 300], 2, 64, 16, torch.float16, wide=30)
    q = b.rows(4)
    want = attend(fa, b, q, True)
    for bad in (-1, b.k_pages.shape[0], 2 ** 31 - 1, -2 ** 31):
        kept = b.block_table[1, 2].item()
        b.block_table[1, 2] = bad
        got = attend(fa, b, q, True)
        assert fa.fa_last_status() == fa.FA_ERR_RANGE
        fa.fa_clear_status()
        b.block_table[1, 2] = kept
        for x, y in zip(got, want):
            assert torch.equal(x[0], y[0]) and torch.equal(x[2:], y[2:]) and torch.isfinite(x).all()


def test_a_length_past_the_table_is_cut_and_reported(fa):
    b = lib.Batch([1, 1], [64, 20], 1, 64, 16, torch.float16)
    q = b.rows(2)
    want = attend(fa, b, q, False)
    b.seq_lens[0] = 65
    got = attend(fa, b, q, False)
    assert fa.fa_last_status() == fa.FA_ERR_RANGE
    fa.fa_clear_status()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------------------------ append
@pytest.mark.parametrize("new,total,Hkv,d,page,rot,inter,dtype", [
    ([1], [1], 1, 64, 8, 64, False, "bf16"),
    ([1] * 64, [1 + 13 * i for i in range(64)], 8, 128, 16, 128, False, "bf16"),
    ([0, 5, 0, 0, 130, 1], [9, 5, 0, 3, 500, 77], 3, 64, 16, 32, True, "fp16"),
    ([700, 300], [700, 4000], 2, 128, 64, 64, False, "fp16"),
    ([33], [2000], 5, 128, 128, 16, True, "bf16"),
    ([12, 1, 40], [12, 900, 41], 4, 64, 32, 0, False, "bf16"),
    ([2] * 1100, [2 + i % 9 for i in range(1100)], 1, 64, 16, 48, False, "fp16"),
])
def test_append(fa, new, total, Hkv, d, page, rot, inter, dtype):
    dt = lib.DTYPES[dtype]
    b = lib.Batch(new, total, Hkv, d, page, dt, token_major=page == 64, fill=5.0, lead=1, behind=2)
    fused = b.rows(3 * Hkv)
    k, v = fused[:, Hkv:2 * Hkv], fused[:, 2 * Hkv:]
    table = lib.rope_table(max(total), rot).cuda() if rot else None
    want_k, want_v = b.k_pages.double(), b.v_pages.clone()
    for i, (n, t) in enumerate(zip(new, total)):
        rows = slice(b.cu[i], b.cu[i] + n)
        at = torch.arange(t - n, t, device="cuda")
        kk = k[rows].double()
        if rot:
            kk = lib.turn64(kk, table[at][:, None], inter)
        where = b.block_table[i].long()[at // page] if n else at
        want_k[where, :, at % page] = kk
        want_v[where, :, at % page] = v[rows]
    fa.paged_append(k, v, b.k_pages, b.v_pages, b.block_table, b.cu_seqlens, b.seq_lens, rope=table,
                    interleaved=inter)
    assert fa.fa_last_status() == 0
    assert torch.equal(b.v_pages, want_v)
    # two products and a sum in 32 bits of elements below `size`, rounded once
    size = k.double().abs().max()
    tol = lib.step(dt) * want_k.abs() + lib.tiny(dt) + 8 * 2.0 ** -24 * size
    assert ((b.k_pages.double() - want_k).abs() <= tol).all()


def test_append_skips_what_has_no_place(fa):
    b = lib.Batch([3, 2, 1], [3, 40, 20], 1, 64, 16, torch.float16, fill=5.0)
    b.seq_lens[0] = 2                    # its first token stands at -1
    b.seq_lens[1] = 49                   # past the table's three pages
    b.block_table[2, 1] = b.k_pages.shape[0]
    k, before = b.rows(1), b.k_pages.clone()
    fa.paged_append(k, k, b.k_pages, b.v_pages, b.block_table, b.cu_seqlens, b.seq_lens)
    assert fa.fa_last_status() == fa.FA_ERR_RANGE
    fa.fa_clear_status()
    before[b.block_table[0, 0].long(), :, :2] = k[1:3].transpose(0, 1)
    before[b.block_table[1, 2].long(), :, 15] = k[3]  # position 47
    assert torch.equal(b.k_pages, before)
    table = lib.rope_table(30, 64).cuda()             # shorter than the sequence
    kept = b.k_pages.clone()
    b.seq_lens[0], b.seq_lens[1] = 3, 40
    b.block_table[2, 1] = b.block_table[2, 0]
    fa.paged_append(k[3:], k[3:], b.k_pages, b.v_pages, b.block_table[1:].contiguous(),
                    (b.cu_seqlens[1:] - 3).contiguous(), b.seq_lens[1:].contiguous(), rope=table)
    assert fa.fa_last_status() == fa.FA_ERR_RANGE
    fa.fa_clear_status()
    assert torch.equal(b.k_pages[b.block_table[1, 2].long()], kept[b.block_table[1, 2].long()])


# ------------------------------------------------------------------------- run together
def test_norm_rotation_append_and_attention_of_a_growing_cache(fa):
    """A prompt chunk, then single tokens, of three sequences: norm and rotation of the heads in
    place, keys and values appended, attention over the cache; against dense 64-bit attention on
    what the cache holds. The captured step is replayed with the lengths of each token."""
    dtype, Hq, Hkv, d, page, steps = torch.bfloat16, 8, 2, 64, 16, 4
    chunk = [37, 5, 150]
    b = lib.Batch(chunk, [c + steps for c in chunk], Hkv, d, page, dtype)
    b.k_pages.fill_(math.nan), b.v_pages.fill_(math.nan)
    table = lib.rope_table(max(b.total), d).cuda()
    wq, wk = ((1 + 0.1 * torch.randn(d)).to(dtype).cuda() for _ in range(2))

    def step(rows, positions, cu, lens, most):
        q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
        q, k = fa.qk_norm_rope(q[None], k[None], wq, wk, table, positions)
        fa.paged_append(k[0], v, b.k_pages, b.v_pages, b.block_table, cu, lens)
        return q[0], *fa.attention_paged(q[0], b.k_pages, b.v_pages, b.block_table, cu, lens, most)

    def expect(q, O, L, new, total):
        b.new, b.total, b.cu = new, total, [sum(new[:i]) for i in range(4)]
        held = [b.cached(i) for i in range(3)]
        want_o, want_l, tol_o, tol_l = lib.attend64(b, q, 1 / math.sqrt(d), True, [x[0] for x in held],
                                                    [x[1] for x in held])
        assert ((O.double() - want_o).abs() <= tol_o).all() and ((L.double() - want_l).abs() <= tol_l).all()

    rows = torch.randn(sum(chunk), Hq + 2 * Hkv, d).to(dtype).cuda()
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in chunk]).cuda()[None]
    lens = torch.tensor(chunk, dtype=torch.int32).cuda()
    expect(*step(rows, pos, b.cu_seqlens, lens, max(chunk)), chunk, chunk)
    # the keys that the cache holds are the normed, rotated ones
    k64 = lib.norm_rope64(rows[:37, Hq:Hq + Hkv], wk, table[:37, None], 1e-6, False)[0]
    assert (b.cached(0)[0].transpose(0, 1).double() - k64).abs().max() <= lib.step(dtype) * k64.abs().max() * 1.01

    one, cu1 = rows[:3].clone(), torch.arange(4, dtype=torch.int32).cuda()
    step(one, lens[None].clone(), cu1, lens + 1, 1)  # the plain call, before it is captured
    graph, at, now = torch.cuda.CUDAGraph(), lens[None].clone(), lens + 1
    with torch.cuda.graph(graph):
        q, O, L = step(one, at, cu1, now, 1)
    for i in range(steps):
        one.copy_(torch.randn_like(one))
        at.copy_(lens[None] + i)
        now.copy_(lens + i + 1)
        graph.replay()
        torch.cuda.synchronize()
        expect(q, O, L, [1, 1, 1], [c + i + 1 for c in chunk])


def test_training_step_through_norm_attention_and_back(fa):
    """norm + rotation -> fa_fwd -> fa_bwd -> their gradients, against autograd in 64 bits."""
    B, N, H, d, dtype = 2, 200, 3, 64, torch.float16
    torch.manual_seed(0)
    fused = torch.randn(B, N, 3 * H * d).to(dtype).cuda()
    q, k, v = (x.unflatten(-1, (H, d)) for x in fused.chunk(3, -1))
    wq, wk = ((1 + 0.1 * torch.randn(d)).to(dtype).cuda() for _ in range(2))
    table = lib.rope_table(N, d).cuda()
    dense = [torch.empty(B, H, N, d, dtype=dtype, device="cuda") for _ in range(2)]
    fa.qk_norm_rope(q, k, wq, wk, table, q_out=dense[0].transpose(1, 2), k_out=dense[1].transpose(1, 2))
    vd = v.transpose(1, 2).contiguous()
    O, L = fa.attention(*dense, vd, causal=True)
    dO = torch.randn_like(O)
    grads = [torch.empty_like(O) for _ in range(3)]
    ws = torch.empty(fa.fa_bwd_workspace_bytes(B, H, N, N, d), dtype=torch.uint8, device="cuda")
    rc = fa.fa_bwd(dense[0].data_ptr(), dense[1].data_ptr(), vd.data_ptr(), O.data_ptr(), dO.data_ptr(), L.data_ptr(),
                   *(g.data_ptr() for g in grads), B, H, N, N, d, 1 / math.sqrt(d), True, fa.FA_F16, ws.data_ptr(),
                   ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(grads[0].transpose(1, 2), grads[1].transpose(1, 2), q, k, wq, wk,
                                                table)
    leaves = [x.double().requires_grad_() for x in (q, k, v, wq, wk)]
    y = [lib.norm_rope64(x, w, table[None, :, None], 1e-6, False)[0].transpose(1, 2)
         for x, w in ((leaves[0], leaves[3]), (leaves[1], leaves[4]))]
    s = (y[0] @ y[1].transpose(2, 3) / math.sqrt(d)).masked_fill(
        torch.ones(N, N, dtype=torch.bool, device="cuda").triu(1), -math.inf)
    (torch.softmax(s, -1) @ leaves[2].transpose(1, 2)).backward(dO.double())
    # four roundings to fp16 on the way (heads, P, dS, dQ and dK), each half a step of values of the
    # gradients' own size; a row's sums average them, so eight half steps of the largest bound each
    for got, leaf in ((dq, leaves[0]), (dk, leaves[1]), (grads[2].transpose(1, 2), leaves[2])):
        assert (got.double() - leaf.grad).abs().max() <= 8 * lib.step(dtype) * leaf.grad.abs().max()
    # each of the weights' sums adds B N H terms that carry those errors
    for got, leaf, go, x, w in ((dwq, leaves[3], grads[0], q, wq), (dwk, leaves[4], grads[1], k, wk)):
        mag = lib.norm_rope_grad64(go.transpose(1, 2), x, w, table[None, :, None], 1e-6, False)[2]
        assert ((got.double() - leaf.grad).abs() <= 8 * lib.step(dtype) * mag.max()).all()


def test_calls_on_another_stream_and_side_by_side(fa):
    """Two streams at once, each with its own workspace."""
    batches = [lib.Batch([1, 1, 20], [2000 + 300 * i, 50, 90], 2, 64, 16, torch.float16, seed=i) for i in range(2)]
    qs = [b.rows(8) for b in batches]
    want = [attend(fa, b, q, True) for b, q in zip(batches, qs)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i in range(2):
            got[i] = attend(fa, batches[i], qs[i], True, stream=streams[i])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    assert fa.fa_last_status() == 0


def test_captured_calls_replayed_with_other_lengths(fa):
    """Graphs of split single tokens and of chunks, each with the workspace its capture took; replayed
    in turn and at once with lengths that change between replays."""
    batches = [lib.Batch([1, 1, 1], [3000, 900, 50], 2, 128, 16, torch.bfloat16, seed=1),
               lib.Batch([300, 40], [2500, 700], 2, 64, 64, torch.float16, seed=2)]
    qs = [b.rows(8) for b in batches]
    for b, q in zip(batches, qs):
        attend(fa, b, q, True)  # the plain call, before it is captured
    graphs, outs = [], []
    for b, q in zip(batches, qs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(attend(fa, b, q, True))
    streams = [torch.cuda.Stream() for _ in range(2)]
    lengths = [b.seq_lens.clone() for b in batches]
    for cut in (0, 37, 400, 1):
        want = []
        for b, q, n in zip(batches, qs, lengths):
            b.seq_lens.copy_((n - cut).clamp(min=1))
            want.append(attend(fa, b, q, True))
        for o in outs:
            o[0].fill_(5.0), o[1].fill_(5.0)
        torch.cuda.synchronize()
        for _ in range(3):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        assert fa.fa_last_status() == 0
        for o, w in zip(outs, want):
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
