"""The build on the host, with a compiler that only notes what it is asked for."""

import os
import subprocess
import sys
import time

import pytest

import moe_decode_layer_bf16_gb300 as m
from moe_decode_layer_bf16_gb300 import build as b


@pytest.fixture
def made(monkeypatch, tmp_path):
    """Names of the files that the last build made; a file in `fails` does not compile."""
    names, fails, clock = [], set(), [time.time()]

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        names.append(os.path.basename(out))
        if names[-1] in fails:
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        with open(out, "w"):
            pass
        clock[0] += 10  # (files of one moment cannot be told apart)
        os.utime(out, (clock[0], clock[0]))
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(b, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libmoe_decode.so"))
    monkeypatch.setattr(b, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(b, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(b.subprocess, "run", run)

    def build():
        names.clear()
        b.build()
        return sorted(names)

    build.fails, build.names = fails, names
    return build


OBJECTS = sorted(s[:-3] + ".o" for s in b.SOURCES)


def test_everything_once(made):
    assert made() == sorted([*OBJECTS, "calls.o", "libmoe_decode.so", "_calls.so"])
    assert made() == []


def test_the_library_without_torch(made, monkeypatch):
    monkeypatch.setattr(b, "_torch_root", lambda: None)
    assert made() == sorted([*OBJECTS, "libmoe_decode.so"])


def test_the_library_where_the_extension_does_not_compile(made):
    made.fails.add("calls.o")
    with pytest.raises(RuntimeError, match="no such header"):
        made()
    assert "libmoe_decode.so" in made.names and os.path.exists(b.LIB)


def test_another_torch_another_extension(made, monkeypatch):
    made()
    key = b._calls_key()
    monkeypatch.setattr(b, "_calls_key", lambda: key + "newer")
    assert made() == ["_calls.so", "calls.o"]
    assert made() == []


def test_the_key_names_torch_and_python():
    import torch
    assert torch.__version__ in b._calls_key() and sys.version in b._calls_key()


def test_package_and_library_without_torch():
    """Importing the package, its build and the loaded library take no torch."""
    code = ("import sys; sys.modules['torch'] = None\n"
            "import moe_decode_layer_bf16_gb300 as m\n"
            "from moe_decode_layer_bf16_gb300 import build\n"
            "assert build._torch_root() is None and m.lib().kv_cache_append and 'fp8_linear' in dir(m)\n"
            "try:\n    m.fp8_linear\nexcept ImportError:\n    print('needs torch')\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(m.__file__)))
    if not os.path.exists(m.LIB_PATH):
        b.build()
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "needs torch", r.stderr


def test_names_of_the_attention_module():
    from moe_decode_layer_bf16_gb300 import attention
    for name in m._ATTENTION:
        assert getattr(m, name) is getattr(attention, name)
    with pytest.raises(AttributeError, match="no_such_name"):
        m.no_such_name
    code = "import moe_decode_layer_bf16_gb300 as m; assert m.attention.fp8_linear is m.fp8_linear"
    root = os.path.dirname(os.path.dirname(os.path.abspath(m.__file__)))
    subprocess.run([sys.executable, "-c", code], cwd=root, check=True)
    star = {}
    exec("from moe_decode_layer_bf16_gb300 import *", star)
    assert {*m._ATTENTION, "MoeDecodeLayer", "moe_decode_layer", "MOE_OK"} <= set(star)
