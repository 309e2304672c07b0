"""Host-side rules of the attention sublayer's operators (no GPU)."""

import contextlib
import ctypes
import itertools
import os
import re
import subprocess

import pytest
import torch

import moe_decode_layer_bf16_gb300 as m
from moe_decode_layer_bf16_gb300 import attention as att


@pytest.fixture(scope="module", autouse=True)
def library():
    if not os.path.exists(m.LIB_PATH):
        from moe_decode_layer_bf16_gb300 import build
        build.build()


CSRC = os.path.join(os.path.dirname(m.__file__), "csrc")


def compiled(tmp_path, name, source):
    """A shared library of host code that includes the sources' headers."""
    src, out = tmp_path / (name + ".cpp"), tmp_path / (name + ".so")
    src.write_text(source)
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-shared", "-fPIC", "-I" + CSRC, "-o", str(out),
                    str(src)], check=True)
    return ctypes.CDLL(str(out))


def test_rows_of_a_step_that_do_not_fit(tmp_path):
    """Every pair of ends, those whose difference passes 31 bits among them."""
    L = compiled(tmp_path, "rows", '#include "step_rows.h"\n'
                 'extern "C" int ok(int a, int b, int t) { return moe::step_rows_ok(a, b, t); }\n')
    lo, hi = -2 ** 31, 2 ** 31 - 1
    ends = [lo, lo + 1, -(1 << 24), -2, -1, 0, 1, 2, 5, 6, 7, 1 << 24, (1 << 24) + 1, 1 << 30, hi - 1, hi]
    for total in (0, 1, 6, 1 << 24):
        for start, stop in itertools.product(ends, ends):
            assert bool(L.ok(start, stop, total)) == (0 <= start <= stop <= total), (start, stop, total)


def test_attention_decode_stays_on_the_stream_it_is_given(monkeypatch):
    """Everything of a step, `rotate` and a new output among it, runs with that stream current."""
    current, seen = [None], []

    @contextlib.contextmanager
    def stream(s):
        before, current[0] = current[0], s
        yield
        current[0] = before

    def note(what):
        return lambda *args, stream=None, **kw: seen.append((what, current[0] if stream is None else stream))

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(att, "moe_workspace_init", lambda ws: None)
    for name in ("fp8_linear", "kv_cache_append", "decode_attention"):
        monkeypatch.setattr(att, name, note(name))
    empty = torch.empty

    def allocate(*args, **kw):
        seen.append(("empty", current[0]))
        return empty(*args, **kw)

    layer = m.AttentionDecode(128, 2, 1, 64, dict.fromkeys(("qkv", "qkv_s", "o", "o_s")),
                              m.Fp8KvCache(2, 1, 64, 16, device="cpu"), max_tokens=2, rotate=note("rotate"))
    monkeypatch.setattr(torch, "empty", allocate)
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    for s in (None, torch.Stream(device="cpu")):
        seen.clear()
        layer(x, None, None, None, stream=s)
        assert [w for w, _ in seen] == ["empty", "fp8_linear", "rotate", "kv_cache_append", "decode_attention", "fp8_linear"]
        assert all(at is s for _, at in seen)
    assert current == [None]


def test_a_setting_is_made_once_on_each_device(tmp_path):
    """The second device of a process gets its own, and a failure is not kept."""
    L = compiled(tmp_path, "devices", '#include "per_device.h"\n'
                 "static moe::OncePerDevice once;\n"
                 'extern "C" int set(int dev, int rc, int* calls) { return once(dev, [&] { ++*calls; return rc; }); }\n')
    calls = ctypes.c_int(0)

    def made(dev, rc=0):
        before = calls.value
        return L.set(dev, rc, ctypes.byref(calls)), calls.value - before

    assert made(0) == (0, 1) and made(0) == (0, 0)
    assert made(1) == (0, 1) and made(1) == (0, 0) and made(0) == (0, 0)
    assert made(2, 7) == (7, 1) and made(2, 7) == (7, 1) and made(2) == (0, 1) and made(2) == (0, 0)
    assert made(63) == (0, 1) and made(63) == (0, 0)
    for dev in (-1, 64, 1000):  # not kept: asked for each time
        assert made(dev) == (0, 1) and made(dev) == (0, 1)


def test_no_kernel_keeps_its_shared_memory_limit_for_the_process():
    """cudaFuncSetAttribute acts on the current device: behind a static of the process it
    would leave the next device without."""
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            text = " ".join(f.read().split())
        assert not re.search(r"static[^;]*cudaFuncSetAttribute", text), name


def test_attention_of_more_items_than_can_be_counted_is_refused():
    fake = ctypes.c_void_p(0x10000)
    L = m.lib()

    def call(B, total, heads, kv_heads):
        c = att._Cache(0x10000, 0x10000, 0x10000, 0x10000, 8, kv_heads, 64, 64)
        return L.decode_attention(c, fake, heads * 64, heads, fake, 4, fake, fake, B, total, 1, 0.1, 0.0, 0, None, fake,
                                  None, None, 0, None)  # (no workspace: refused, where nothing refuses before)

    assert call(1 << 20, 1 << 20, 1024, 1024) == m.MOE_ERR_UNSUPPORTED
    assert call(700000, 700000, 1024, 1024) == m.MOE_ERR_UNSUPPORTED
    for ok in ((600000, 600000, 1024, 1024), (1, 1 << 20, 1024, 1024), (1 << 20, 1, 1024, 1024), (4, 93000, 128, 8),
               (1, 1 << 24, 127, 1)):
        assert call(*ok) == m.MOE_ERR_INVALID_ARG, ok


def test_batches_without_sequences_or_tokens_are_no_ops():
    """Arrays of no elements have no address."""
    L, fake, big = m.lib(), ctypes.c_void_p(0x10000), 1 << 40
    c = att._Cache(0x10000, 0x10000, 0x10000, 0x10000, 8, 2, 64, 64)
    for B, total, width in ((0, 0, 0), (0, 0, 4), (2, 0, 4), (2, 0, 0), (0, 3, 4)):
        assert L.kv_cache_append(c, None, 128, None, 128, None, width, None, None, B, total, 1, fake, big, None) == m.MOE_OK
        assert L.decode_attention(c, None, 256, 4, None, width, None, None, B, total, 1, 0.1, 0.0, 0, None, None, None, fake,
                                  big, None) == m.MOE_OK
    for B, total, width in ((-1, 0, 4), (0, -1, 4), (0, 0, -1)):
        assert L.kv_cache_append(c, None, 128, None, 128, None, width, None, None, B, total, 1, fake, big,
                                 None) == m.MOE_ERR_INVALID_ARG
    for width in (0, 4):  # with tokens, everything is wanted
        assert L.kv_cache_append(c, fake, 128, fake, 128, None if width else fake, width, fake, fake, 2, 3, 1, fake, big,
                                 None) == m.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("n", [0, 1, 2])
def test_attention_decode_of_a_few_tokens_or_none(monkeypatch, n):
    shapes = []
    monkeypatch.setattr(att, "moe_workspace_init", lambda ws: None)
    monkeypatch.setattr(att, "fp8_linear", lambda x, w, w_s, out, ws, **kw: shapes.append((tuple(x.shape), tuple(out.shape))))
    for name in ("kv_cache_append", "decode_attention"):
        monkeypatch.setattr(att, name, lambda *args, **kw: None)
    layer = m.AttentionDecode(128, 2, 1, 64, dict.fromkeys(("qkv", "qkv_s", "o", "o_s")),
                              m.Fp8KvCache(2, 1, 64, 16, device="cpu"), max_tokens=2)
    y = layer(torch.zeros((n, 128), dtype=torch.bfloat16), None, None, None)
    assert tuple(y.shape) == (n, 128) and shapes == [((n, 128), (n, 256)), ((n, 128), (n, 128))]


def test_an_argument_without_a_truth_value_raises_its_own_error():
    x, w = torch.zeros((1, 128), dtype=torch.bfloat16), torch.zeros((128, 128), dtype=torch.uint8)
    args = (x, w, torch.zeros((1, 1)), torch.zeros((1, 128)), torch.zeros(1 << 20, dtype=torch.uint8))
    with pytest.raises(RuntimeError, match="ambiguous"):
        m.fp8_linear(*args, e8m0=torch.zeros(2))
    with pytest.raises(ValueError, match="CUDA"):  # and what has one is looked at further
        m.fp8_linear(*args, e8m0=torch.ones(1))
