"""The package's build and its tensor-level calls at the edges of what they accept, without a GPU."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

import exact_attention_forward_02_gb300 as fa
from tests import decoder_testlib as lib


def _run(code, cwd):
    return subprocess.run([sys.executable, "-c", code], cwd=cwd, capture_output=True, text=True, timeout=120,
                          env={**os.environ, "PYTHONPATH": "", "FA_LIBRARY": "release"})


@pytest.fixture
def bare(tmp_path):
    """The package with its C library and without the module over libtorch."""
    pkg = tmp_path / "exact_attention_forward_02_gb300"
    pkg.mkdir()
    for name in ("__init__.py", "build.py"):
        shutil.copy(os.path.join(fa.PKG, name), pkg / name)
    os.symlink(fa.LIB_PATH, pkg / "libfa.so")
    return tmp_path


def test_the_c_library_s_binding_needs_no_torch(bare):
    r = _run("""
import sys
sys.modules["torch"] = None
import exact_attention_forward_02_gb300 as fa
assert fa.fa_fwd(None, None, None, None, None, 1, 1, 8, 8, 64, 1.0, 0, 0, None) == fa.FA_ERR_NULL
assert fa.fa_paged_append(None, None, None, 1, 1, None, None, None, 1, None, 0, None) == fa.FA_ERR_NULL
try:
    fa.attention_paged(None, None, None, None, None, None, 1)
except ImportError as e:
    print("said:", e)
""", bare)
    assert r.returncode == 0 and "_fa_torch.so" in r.stdout and "not built" in r.stdout, r.stderr


BUILDER = "import exact_attention_forward_02_gb300.build as b\n"


def test_the_build_leaves_the_calls_out_where_there_is_no_torch(bare):
    r = _run("import sys; sys.modules['torch'] = None\n" + BUILDER + "assert b.build_many([]) == []", bare)
    assert r.returncode == 0 and "no CUDA build of torch" in r.stderr, r.stderr


def test_the_build_leaves_the_calls_out_where_torch_has_no_cuda(bare):
    (bare / "torch" / "lib").mkdir(parents=True)
    (bare / "torch" / "__init__.py").write_text("")
    r = _run(BUILDER + "assert b.torch_root() is None and b.build_many([]) == []", bare)
    assert r.returncode == 0 and "no CUDA build of torch" in r.stderr, r.stderr


def test_the_calls_are_built_again_for_another_torch(bare):
    lib = bare / "torch" / "lib"
    lib.mkdir(parents=True)
    (lib / "libtorch_cuda.so").write_text("")
    (bare / "torch" / "__init__.py").write_text("")
    version = bare / "torch" / "version.py"
    version.write_text("__version__ = '1'")
    r = _run(BUILDER + f"""
import os
root = b.torch_root()
assert os.path.realpath(root) == os.path.realpath({str(bare / 'torch')!r})
b.TORCH_DEPS = [b.__file__]
assert b._calls_stale(root)                       # no module
open(b.TORCH_LIB, "w").close()
assert b._calls_stale(root)                       # one of an unknown torch
os.makedirs(os.path.dirname(b.TORCH_STAMP))
open(b.TORCH_STAMP, "w").write(b.torch_version(root))
assert not b._calls_stale(root)
open({str(version)!r}, "w").write("__version__ = '2'")
assert b._calls_stale(root)
""", bare)
    assert r.returncode == 0, r.stderr


P = 1 << 20  # 16-byte aligned, not null, never touched


def heads(H=4, token=256, head=64):
    return fa.fa_heads(P, 0, token, head, H)


def test_a_table_shorter_than_the_tokens_is_refused_without_positions():
    def norm(N, length, positions, rot=64, B=1):
        return fa.fa_qk_norm_rope(heads(), heads(), heads(), heads(), B, N, 64, P, P, 1e-6,
                                  fa.fa_rope(P, length, rot, 0), positions, fa.FA_F16, None)

    def backward(N, length, positions):
        return fa.fa_qk_norm_rope_bwd(*(heads() for _ in range(6)), P, P, 1, N, 64, P, P, 1e-6,
                                      fa.fa_rope(P, length, 64, 0), positions, fa.FA_F16, P, 1 << 30, None)

    for call in (norm, backward):
        assert call(9, 8, None) == fa.FA_ERR_RANGE
        assert call(1, 0, None) == fa.FA_ERR_RANGE
    assert norm(0, 0, None) == fa.FA_OK and norm(9, 8, None, B=0) == fa.FA_OK


def test_a_table_as_long_as_the_tokens_is_not_refused():
    if torch.cuda.is_available():
        pytest.skip("a GPU would be given the pointers of this test")
    for args in (dict(N=8, length=8, positions=None), dict(N=9, length=8, positions=P),
                 dict(N=9, length=8, positions=None, rot=0)):
        rot = args.pop("rot", 64)
        rc = fa.fa_qk_norm_rope(heads(), heads(), heads(), heads(), 1, args["N"], 64, P, P, 1e-6,
                                fa.fa_rope(P, args["length"], rot, 0), args["positions"], fa.FA_F16, None)
        assert rc in (fa.FA_ERR_CUDA, fa.FA_ERR_DEVICE)  # past the checks, and no device here


def test_flags_that_have_no_truth_value_are_refused():
    """An argument whose bool() raises: a TypeError, before anything else is looked at."""
    b = lib.Batch([2, 1], [20, 3], 2, 64, 16, torch.float16, device="cpu", fill=0.0)
    q, k = b.rows(4, device="cpu"), b.rows(2, device="cpu")
    table, two = (b.block_table, b.cu_seqlens, b.seq_lens), torch.zeros(2)
    x, w = torch.zeros(1, 5, 2, 64).half(), torch.zeros(64).half()
    for call in (lambda: fa.attention_paged(q, b.k_pages, b.v_pages, *table, 2, causal=two),
                 lambda: fa.paged_append(k, k, b.k_pages, b.v_pages, *table, interleaved=two),
                 lambda: fa.qk_norm_rope(x, x, w, w, interleaved=two),
                 lambda: fa.qk_norm_rope_backward(x, x, x, x, w, w, interleaved=two)):
        with pytest.raises(TypeError, match="truth value"):
            call()


@pytest.mark.parametrize("B", [(1 << 30) + 1, 0x7ffffff0, 0x7ffffffe, 0x7fffffff])
def test_more_sequences_than_the_kernels_can_count_are_refused(B):
    """Rounding B up to whole warps' and blocks' shares would pass 32 bits on the device."""
    kv = fa.fa_paged_kv(P, P, 16384, 1024, 64, 8, 16, 4, 64)
    assert fa.fa_paged_append(kv, heads(), heads(), B, 8, P, P, P, 4, None, 1, None) == fa.FA_ERR_SHAPE
    assert fa.fa_fwd_paged(kv, heads(8), heads(8), P, B, 8, 4, P, P, P, 4, 0.125, 1, 1, P, 1 << 40,
                           None) == fa.FA_ERR_SHAPE
