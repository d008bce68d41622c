"""The build of the C library and of the torch binding, apart from one another."""
import importlib.util
import os
import subprocess
import sys

import pytest

from libbuild import ROOT, build_and_import

build_and_import()
BUILD = os.path.join(ROOT, "paged_kv_cache_208_gb300", "build.py")


@pytest.fixture
def builder(tmp_path):
    """build.py with its outputs and sources in a folder of their own: one C++ file, no kernels."""
    spec = importlib.util.spec_from_file_location("_pkv_build_alone", BUILD)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    (csrc / "one.cpp").write_text('extern "C" int one() { return 1; }\n')
    mod.CSRC, mod.OBJ_DIR = str(csrc), str(tmp_path / "obj")
    mod.LIB, mod.BINDING = str(tmp_path / "libpkv.so"), str(tmp_path / "_pkv_torch.so")
    return mod


def test_a_binding_that_does_not_compile_leaves_the_library(builder):
    def fails():
        raise RuntimeError("g++ failed on the binding")

    builder._compile_binding = fails
    with pytest.raises(RuntimeError, match="the binding"):
        builder.build(force=True)
    assert os.path.exists(builder.LIB) and not os.path.exists(builder.BINDING)


def test_the_library_is_built_without_torch(tmp_path):
    """Where there is no torch there is nothing to bind to, and nvcc is enough."""
    code = f"""
import importlib.util, os, sys
sys.modules["torch"] = None
spec = importlib.util.spec_from_file_location("b", {BUILD!r})
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
t = {str(tmp_path)!r}
os.mkdir(t + "/csrc")
open(t + "/csrc/one.cpp", "w").write("int one() {{ return 1; }}")
b.CSRC, b.OBJ_DIR, b.LIB, b.BINDING = t + "/csrc", t + "/obj", t + "/l.so", t + "/b.so"
b.build(force=True)
assert os.path.exists(b.LIB) and not os.path.exists(b.BINDING)
b.build()
"""
    subprocess.run([sys.executable, "-c", code], check=True)


def test_a_binding_of_another_torch_is_stale(builder):
    os.makedirs(builder.OBJ_DIR)
    for path in (builder.LIB, builder.BINDING):
        open(path, "w").close()
    builder._note_binding()
    assert not builder._stale()
    was = builder._torch_version
    builder._torch_version = lambda: was() + ".other"
    assert builder._stale()


def test_the_package_works_without_the_binding():
    """The older calls need libpkv.so alone; those of the binding say what is missing."""
    code = """
import sys
sys.modules["paged_kv_cache_208_gb300._pkv_torch"] = None
import paged_kv_cache_208_gb300 as pkv
assert pkv.xxh64(b"") == 0xEF46DB3751D8E999
assert pkv.BlockManager(4, 8).take(2) == [0, 1]
for call, n in ((pkv.kv_store_fp8, 8), (pkv.kv_gather_fp8, 7), (pkv.paged_decode_attn_fp8, 9),
                (pkv.paged_decode_attn_weights, 7), (pkv.kv_evict, 9)):
    try:
        call(*[None] * n)
    except ImportError as e:
        assert "_pkv_torch.so" in str(e) and "build.py" in str(e), e
    else:
        raise AssertionError(call.__name__)
"""
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)
