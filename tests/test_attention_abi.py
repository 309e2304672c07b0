"""The attention sublayer's entry points on the host: bad arguments are refused
before anything is enqueued (no GPU), by the binding and by the library; and the
oracle against direct evaluations."""

import ctypes
import os

import numpy as np
import pytest
import torch

import moe_decode_layer_bf16_gb300 as m
from moe_decode_layer_bf16_gb300 import attention as att
from tests.fixtures_attention import Batch, bf16_values, e4m3_decode, orc, weights


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(m.LIB_PATH):
        from moe_decode_layer_bf16_gb300 import build
        build.build()
    return m.lib()


FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10004)
BIG = 1 << 40


# ---------------------------------------------------------------- library
def test_linear_sizes(L):
    # codes, scales and the partial sums grow with the shape; any N, K in steps of 16
    assert m.fp8_linear_workspace_size(1, 9216, 7168) > m.fp8_block_gemm_workspace_size(1, 9216, 7168) > 0
    assert m.fp8_linear_workspace_size(256, 9216, 7168) > 256 * 7168
    assert m.fp8_linear_workspace_size(1, 1, 16) > 0
    for M, N, K, code in [(4, 128, 100, m.MOE_ERR_UNSUPPORTED), (4, 0, 128, m.MOE_ERR_INVALID_ARG),
                          (-1, 128, 128, m.MOE_ERR_INVALID_ARG), (4, 128, 0, m.MOE_ERR_INVALID_ARG),
                          (4, 128, (1 << 17) + 16, m.MOE_ERR_UNSUPPORTED), (4, (1 << 20) + 1, 128, m.MOE_ERR_UNSUPPORTED),
                          ((1 << 20) + 1, 128, 128, m.MOE_ERR_UNSUPPORTED)]:
        for f in (m.fp8_linear_workspace_size, m.fp8_block_gemm_workspace_size):
            with pytest.raises(m.MoeError) as e:
                f(M, N, K)
            assert e.value.status == code


def test_linear_refusals(L):
    def call(x=FAKE, ldx=512, w=FAKE, ws=FAKE, M=4, N=128, K=512, out=FAKE, work=FAKE, size=BIG):
        return L.fp8_linear(x, ldx, w, ws, M, N, K, 0, out, 0, work, size, None)

    assert call(M=0) == m.MOE_OK
    for kw in (dict(x=None), dict(w=None), dict(ws=None), dict(out=None), dict(work=None), dict(x=ODD), dict(w=ODD),
               dict(out=ODD), dict(work=ODD), dict(ldx=511), dict(ldx=516)):
        assert call(**kw) == m.MOE_ERR_INVALID_ARG, kw
    assert call(K=520, ldx=520) == m.MOE_ERR_UNSUPPORTED
    need = m.fp8_linear_workspace_size(4, 128, 512)
    assert call(size=need - 1) == m.MOE_ERR_WORKSPACE_TOO_SMALL

    def gemm(c=FAKE, s=FAKE, w=FAKE, ws=FAKE, out=FAKE, work=FAKE, size=BIG, M=4):
        return L.fp8_block_gemm(c, s, w, ws, M, 128, 512, out, 1, work, size, None)

    assert gemm(M=0) == m.MOE_OK
    for kw in (dict(c=None), dict(s=None), dict(w=None), dict(ws=None), dict(out=None), dict(work=None), dict(c=ODD),
               dict(s=ODD), dict(w=ODD), dict(out=ODD)):
        assert gemm(**kw) == m.MOE_ERR_INVALID_ARG, kw
    assert gemm(size=m.fp8_block_gemm_workspace_size(4, 128, 512) - 1) == m.MOE_ERR_WORKSPACE_TOO_SMALL

    def quant(x=FAKE, ldx=512, M=4, K=512, c=FAKE, s=FAKE):
        return L.fp8_quant_rows(x, ldx, M, K, 0, c, s, None)

    assert quant(M=0) == m.MOE_OK
    for kw in (dict(x=None), dict(c=None), dict(s=None), dict(x=ODD), dict(c=ODD), dict(s=ODD), dict(ldx=256)):
        assert quant(**kw) == m.MOE_ERR_INVALID_ARG, kw
    assert quant(K=500) == m.MOE_ERR_UNSUPPORTED


def cache(k=0x10000, v=0x10000, ks=0x10000, vs=0x10000, pages=8, heads=2, page=64, dim=128):
    return att._Cache(k, v, ks, vs, pages, heads, page, dim)


BAD_CACHES = [(dict(k=0), m.MOE_ERR_INVALID_ARG), (dict(v=0), m.MOE_ERR_INVALID_ARG), (dict(ks=0), m.MOE_ERR_INVALID_ARG),
              (dict(vs=0), m.MOE_ERR_INVALID_ARG), (dict(k=0x10008), m.MOE_ERR_INVALID_ARG),
              (dict(pages=0), m.MOE_ERR_INVALID_ARG), (dict(heads=0), m.MOE_ERR_INVALID_ARG),
              (dict(page=48), m.MOE_ERR_UNSUPPORTED), (dict(page=256), m.MOE_ERR_UNSUPPORTED),
              (dict(dim=96), m.MOE_ERR_UNSUPPORTED), (dict(heads=1025), m.MOE_ERR_UNSUPPORTED),
              (dict(pages=1 << 30, heads=4), m.MOE_ERR_UNSUPPORTED)]


def test_append_refusals(L):
    def call(c=None, k=FAKE, ks=256, v=FAKE, vs=256, table=FAKE, width=4, q=FAKE, lens=FAKE, B=2, total=3, new=2,
             ws=FAKE, size=BIG):
        return L.kv_cache_append(cache() if c is None else c, k, ks, v, vs, table, width, q, lens, B, total, new, ws,
                                 size, None)

    assert call(B=0) == m.MOE_OK and call(total=0) == m.MOE_OK
    for kw, code in BAD_CACHES:
        assert call(c=cache(**kw)) == code, kw
    for kw in (dict(k=None), dict(v=None), dict(k=ODD), dict(ks=255), dict(vs=260), dict(table=None), dict(q=None),
               dict(lens=None), dict(width=0), dict(B=-1), dict(total=-1), dict(new=0), dict(ws=None), dict(ws=ODD)):
        assert call(**kw) == m.MOE_ERR_INVALID_ARG, kw
    assert call(width=1 << 25) == m.MOE_ERR_UNSUPPORTED
    assert call(size=m.kv_cache_workspace_size() - 1) == m.MOE_ERR_WORKSPACE_TOO_SMALL
    assert L.kv_cache_append(None, FAKE, 256, FAKE, 256, FAKE, 4, FAKE, FAKE, 2, 3, 2, FAKE, BIG, None) == m.MOE_ERR_INVALID_ARG


def test_attention_refusals(L):
    def call(c=None, q=FAKE, qs=512, heads=4, table=FAKE, width=4, start=FAKE, lens=FAKE, B=2, total=3, new=2,
             scale=0.1, cap=0.0, window=0, out=FAKE, ws=FAKE, size=BIG):
        return L.decode_attention(cache() if c is None else c, q, qs, heads, table, width, start, lens, B, total, new,
                                  scale, cap, window, None, out, None, ws, size, None)

    assert call(B=0) == m.MOE_OK and call(total=0) == m.MOE_OK
    for kw, code in BAD_CACHES:
        assert call(c=cache(**kw)) == code, kw
    for kw in (dict(q=None), dict(q=ODD), dict(qs=500), dict(table=None), dict(start=None), dict(lens=None),
               dict(width=0), dict(new=0), dict(out=None), dict(out=ODD), dict(ws=None), dict(ws=ODD),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(cap=-1.0), dict(cap=float("inf")),
               dict(window=-1), dict(heads=0)):
        assert call(**kw) == m.MOE_ERR_INVALID_ARG, kw
    for kw in (dict(heads=3, qs=384), dict(heads=4098, qs=4098 * 128), dict(width=1 << 25), dict(total=1 << 25)):
        assert call(**kw) == m.MOE_ERR_UNSUPPORTED, kw
    need = m.decode_attention_workspace_size(4, 2, 128, 2)
    assert call(size=need - 1) == m.MOE_ERR_WORKSPACE_TOO_SMALL
    with pytest.raises(m.MoeError):
        m.decode_attention_workspace_size(5, 2, 128, 1)


# ---------------------------------------------------------------- binding
def test_binding_refuses_what_is_not_as_documented(L):
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    w, ws = torch.zeros((128, 256), dtype=torch.uint8), torch.zeros((1, 2))
    out, work = torch.zeros((4, 128), dtype=torch.bfloat16), torch.zeros(1 << 20, dtype=torch.uint8)
    for bad, what in [((x.float(), w, ws, out, work), "x"), ((x, w.float(), ws, out, work), "w"),
                      ((x, w, ws.double(), out, work), "w_s"), ((x, w, torch.zeros((2, 2)), out, work), "w_s"),
                      ((x, w, ws, out.half(), work), "out"), ((x, w, ws, torch.zeros((4, 129)), work), "out"),
                      ((x[:, :128], w, ws, out, work), "x"), ((x.t().contiguous().t(), w, ws, out, work), "x"),
                      ((x, w.t().contiguous().t(), ws, out, work), "w"), ((x[0], w, ws, out, work), "x")]:
        with pytest.raises(ValueError, match=what):
            m.fp8_linear(*bad)
    with pytest.raises(ValueError, match="CUDA"):  # all as it should be, but not on a GPU
        m.fp8_linear(x, w, ws, out, work)
    with pytest.raises(ValueError, match="CUDA"):
        m.fp8_quant_rows(x, torch.zeros((4, 256), dtype=torch.uint8), torch.zeros((2, 4)))
    with pytest.raises(ValueError, match="scales"):
        m.fp8_quant_rows(x, torch.zeros((4, 256), dtype=torch.uint8), torch.zeros((4, 2)))
    with pytest.raises(ValueError, match="CUDA"):
        m.fp8_block_gemm(torch.zeros((4, 256), dtype=torch.uint8), torch.zeros((2, 4)), w, ws, out, work)

    kc, sc = torch.zeros((8, 2, 16, 64), dtype=torch.uint8), torch.zeros((8, 2))
    table, start = torch.zeros((2, 4), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    lens = torch.zeros(2, dtype=torch.int32)
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16)
    good = [k, k, kc, kc, sc, sc, table, start, lens, 2, work]
    for i, bad, what in [(0, k.float(), "k"), (1, k[:2], "v"), (2, kc.float(), "k_cache"), (3, kc[:7], "v_cache"),
                         (4, sc.double(), "k_scale"), (5, sc[:7], "v_scale"), (6, table.long(), "page_table"),
                         (6, table[:1], "page_table"), (7, start[:2], "q_start"), (8, lens.long(), "lens"),
                         (0, k.transpose(1, 2).contiguous().transpose(1, 2), "k")]:
        args = list(good)
        args[i] = bad
        with pytest.raises(ValueError, match=what):
            m.kv_cache_append(*args)
    with pytest.raises(ValueError, match="CUDA"):
        m.kv_cache_append(*good)
    good = dict(q=q, k_cache=kc, v_cache=kc, k_scale=sc, v_scale=sc, page_table=table, q_start=start, lens=lens,
                max_new=2, out=torch.zeros_like(q), workspace=work)
    for name, bad in [("q", q.float()), ("q", q[:, :, :32]), ("out", q[:2]), ("lse", torch.zeros((3, 3))),
                      ("slopes", torch.zeros(3)), ("k_cache", kc[0]), ("lens", lens[None])]:
        with pytest.raises(ValueError, match=name):
            m.decode_attention(**{**good, name: bad})
    with pytest.raises(ValueError, match="CUDA"):
        m.decode_attention(**good)


# ---------------------------------------------------------------- the oracle itself
def test_oracle_linear_is_the_product_of_the_dequantised_matrices():
    rng = np.random.default_rng(0)
    x = bf16_values(rng, (5, 272))
    w, s = weights(rng, 130, 272)
    codes, scales = orc.quant_rows(x, False)
    out, mag = orc.block_gemm(codes, scales, w, s)
    xd = e4m3_decode(codes) * np.repeat(scales.T, 128, 1)[:, :272]
    wd = e4m3_decode(w) * np.repeat(np.repeat(s, 128, 0), 128, 1)[:130, :272].astype(np.float64)
    assert np.allclose(out, xd @ wd.T, rtol=1e-12, atol=0) and (mag >= np.abs(out) * (1 - 1e-12)).all()
    # the codes stand for x to half an E4M3 step, or half the smallest step of its group
    step = np.repeat(scales.T, 128, 1)[:, :272].astype(np.float64)
    assert (np.abs(xd - x) <= np.maximum(np.abs(x) * 2.0 ** -4, step * 2.0 ** -10) * (1 + 1e-6)).all()


def test_oracle_append_then_read_back():
    rng = np.random.default_rng(1)
    b = Batch(rng, [0, 0], [0, 0], 2, 64, 16)
    cache = {"k": np.full((6, 2, 16, 64), 0x7F, np.uint8), "v": np.full((6, 2, 16, 64), 0x7F, np.uint8),
             "k_scale": np.full((6, 2), np.nan, np.float32), "v_scale": np.full((6, 2), np.nan, np.float32)}
    table = np.array([[4, 1, 3], [0, 5, 2]], np.int32)
    values = bf16_values(rng, (2, 40, 2, 64))
    values[:, 20:] *= 7.0  # louder tokens: the second block's scale grows as they come
    done = 0
    for step in (3, 14, 1, 6, 16):
        new = values[:, done:done + step].reshape(2 * step, 2, 64)
        done += step
        orc.append(new, new, cache, table, [0, step, 2 * step], [done, done])
    for s in range(2):
        pg, at = table[s, np.arange(40) // 16], np.arange(40) % 16
        got = e4m3_decode(cache["k"][pg, :, at]) * cache["k_scale"][pg][:, :, None].astype(np.float64)
        scale = cache["k_scale"][pg][:, :, None].astype(np.float64)
        # one rounding as the token came, a second where a grown scale made its code subnormal
        tol = np.maximum(np.abs(values[s]) * 2.0 ** -4, scale * 2.0 ** -9)
        assert (np.abs(got - values[s]) <= tol).all()
    assert b.total == 0


def test_oracle_attention_against_a_direct_softmax():
    rng = np.random.default_rng(2)
    b = Batch(rng, [37, 0, 5], [2, 1, 3], 2, 64, 16)
    q = bf16_values(rng, (b.total, 6, 64))
    out, lse, _, _ = orc.attention(q, b.cache, b.table, b.q_start, b.lens, 0.125, window=9)
    k = e4m3_decode(b.cache["k"][b.table[0, :3], 1].reshape(48, 64)[:37]) * np.repeat(b.cache["k_scale"][b.table[0, :3], 1], 16)[:37, None]
    v = e4m3_decode(b.cache["v"][b.table[0, :3], 1].reshape(48, 64)[:37]) * np.repeat(b.cache["v_scale"][b.table[0, :3], 1], 16)[:37, None]
    s = 0.125 * (k[27:36] @ q[0, 4].astype(np.float64))  # row 0 is at position 35 and sees 27 .. 35
    p = np.exp(s)
    assert np.allclose(out[0, 4], p @ v[27:36] / p.sum(), rtol=1e-9) and np.isclose(lse[0, 4], np.log(p.sum()))
    assert (out[2] == 0).all() and np.isneginf(lse[2]).all()  # the empty sequence's row
    assert np.isfinite(out).all()
