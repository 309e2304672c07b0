"""Host-side rules of the attention sublayer's operators (no GPU)."""

import ctypes
import itertools
import os
import subprocess

import pytest

import moe_decode_layer_bf16_gb300 as m

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
