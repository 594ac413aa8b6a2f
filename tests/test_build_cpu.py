"""The build and the import around the helpers' extension module, which belongs to
one version of torch: the library and every scan stand without it."""
import os
import subprocess
import sys

import pytest

from selective_state_space_chunked_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    assert build.up_to_date()


def imports(change):
    body = f"""
import warnings
from selective_state_space_chunked_gb300 import build
{change}
with warnings.catch_warnings(record=True) as w:
    warnings.simplefilter("always")
    from selective_state_space_chunked_gb300 import binding as lr
said = [str(x.message) for x in w if issubclass(x.category, RuntimeWarning)]
assert lr.lr_version() > 0 and lr.lr_host_sync is not None
args = [None] * 10
declines = lr._lrtorch.decay_attn(*args) is None and lr._lrtorch.decay_attn_step(*args) is None
assert declines and lr._lrtorch.group_norm_act(*args[:8]) is None
print(len(said))
"""
    r = subprocess.run([sys.executable, "-c", body], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return int(r.stdout)


def test_the_import_stands_without_the_module(tmp_path):
    assert imports("") == 0
    assert imports("build.TORCH_MODULE = '/nonexistent/_lrtorch.so'") == 1
    bad = tmp_path / "_lrtorch.so"
    bad.write_text("not a shared object")
    assert imports(f"build.TORCH_MODULE = {str(bad)!r}") == 1


def test_a_module_of_another_torch_is_neither_used_nor_up_to_date(tmp_path, monkeypatch):
    other = tmp_path / "version"
    other.write_text("1.0.0")
    assert imports(f"build.TORCH_VERSION = {str(other)!r}") == 1
    monkeypatch.setattr(build, "TORCH_VERSION", str(other))
    assert not build.up_to_date()
    monkeypatch.setattr(build, "TORCH_VERSION", str(tmp_path / "none"))
    assert not build.up_to_date()


def test_a_build_that_fails_at_the_module_leaves_the_library_and_no_older_module(tmp_path, monkeypatch):
    import torch
    for name in ("LIB_PATH", "TORCH_MODULE", "TORCH_VERSION"):
        monkeypatch.setattr(build, name, str(tmp_path / name))
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path))
    (tmp_path / "TORCH_MODULE").write_text("the last build's")
    (tmp_path / "TORCH_VERSION").write_text(torch.__version__)
    assert build.torch_module_matches()

    def run(cmd, **kw):   # every CUDA file compiles and links, the module does not
        return subprocess.CompletedProcess(cmd, 1 if cmd[0] == "g++" else 0, "", "no")
    monkeypatch.setattr(build.subprocess, "run", run)
    with pytest.raises(RuntimeError):
        build.build(force=True)
    assert (tmp_path / "LIB_PATH").exists() and not build.torch_module_matches()
