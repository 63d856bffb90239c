"""The package's build and its tensor-level calls at the edges of what they accept, without a GPU."""
import os
import shutil
import subprocess
import sys

import pytest

import exact_attention_forward_02_gb300 as fa


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
