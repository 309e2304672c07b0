"""A prompt's operators on the host: bad arguments are refused before anything is
enqueued (no GPU), by the binding and by the library."""

import ctypes
import os

import pytest
import torch

import moe_decode_layer_bf16_gb300 as m


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(m.LIB_PATH):
        from moe_decode_layer_bf16_gb300 import build
        build.build()
    return m.lib()


FAKE = ctypes.c_void_p(0x10000)
OTHER = ctypes.c_void_p(0x20000)
ODD = ctypes.c_void_p(0x10004)
BIG = 1 << 40


# ---------------------------------------------------------------- library
def test_norm_refusals(L):
    def call(x=FAKE, ldx=256, r=FAKE, ldr=256, g=FAKE, M=4, H=256, eps=1e-6, c=FAKE, s=FAKE, out=None, ro=OTHER):
        return L.rmsnorm_residual_fp8(x, ldx, r, ldr, g, M, H, eps, 0, c, s, out, ro, None)

    assert call(M=0) == m.MOE_OK
    for kw in (dict(r=None), dict(g=None), dict(c=None), dict(s=None), dict(ro=None), dict(x=ODD), dict(r=ODD), dict(g=ODD),
               dict(c=ODD), dict(s=ODD), dict(out=ODD), dict(ro=ODD), dict(ldx=255), dict(ldx=260), dict(ldr=128),
               dict(M=-1), dict(H=0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
               dict(ro=FAKE, ldr=264)):  # in place, with rows that are not where the output's are
        assert call(**kw) == m.MOE_ERR_INVALID_ARG, kw
    for kw in (dict(H=248, ldx=248, ldr=248), dict(H=16400, ldx=16400, ldr=16400), dict(M=(1 << 20) + 1)):
        assert call(**kw) == m.MOE_ERR_UNSUPPORTED, kw


def test_pages_refusals(L):
    need = m.kv_cache_workspace_size()

    def extend(t=FAKE, width=4, lens=FAKE, new=FAKE, B=2, stack=FAKE, cap=8, state=FAKE, page=64, pages=8, q=FAKE, lo=FAKE,
               fo=FAKE, pos=FAKE, slots=FAKE, rows=16, ws=FAKE, size=BIG):
        return L.kv_pages_extend(t, width, lens, new, B, stack, cap, state, page, pages, q, lo, fo, pos, slots, rows, ws, size,
                                 None)

    def release(t=FAKE, width=4, lens=FAKE, done=FAKE, B=2, stack=FAKE, cap=8, state=FAKE, page=64, pages=8, lo=FAKE, fo=FAKE,
                ws=FAKE, size=BIG):
        return L.kv_pages_release(t, width, lens, done, B, stack, cap, state, page, pages, lo, fo, ws, size, None)

    shared = [dict(t=None), dict(lens=None), dict(stack=None), dict(state=None), dict(lo=None), dict(fo=None), dict(ws=None),
              dict(ws=ODD), dict(width=0), dict(width=-1), dict(B=-1), dict(cap=-1), dict(pages=0), dict(page=0)]
    for call, more in ((extend, [dict(new=None), dict(q=None), dict(pos=None), dict(slots=None), dict(rows=-1)]),
                       (release, [dict(done=None)])):
        for kw in shared + more:
            assert call(**kw) == m.MOE_ERR_INVALID_ARG, kw
        for kw in (dict(page=48), dict(page=256), dict(width=1 << 25), dict(B=(1 << 20) + 1)):
            assert call(**kw) == m.MOE_ERR_UNSUPPORTED, kw
        assert call(size=need - 1) == m.MOE_ERR_WORKSPACE_TOO_SMALL
    assert extend(rows=(1 << 24) + 1) == m.MOE_ERR_UNSUPPORTED


def test_prompt_attention_refusals(L):
    def call(q=FAKE, qs=512, k=FAKE, ks=256, v=FAKE, vs=256, heads=4, hk=2, d=128, start=FAKE, B=2, total=9, scale=0.1,
             cap=0.0, window=0, out=FAKE, ws=FAKE, size=BIG):
        return L.prompt_attention(q, qs, k, ks, v, vs, heads, hk, d, start, B, total, scale, cap, window, None, out, None, ws,
                                  size, None)

    assert call(B=0) == m.MOE_OK and call(total=0) == m.MOE_OK
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(qs=504), dict(qs=516),
               dict(ks=248), dict(vs=260), dict(start=None), dict(out=None), dict(out=ODD), dict(ws=None), dict(ws=ODD),
               dict(B=-1), dict(total=-1), dict(heads=0), dict(hk=0), dict(d=0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(cap=-1.0), dict(cap=float("inf")), dict(window=-1)):
        assert call(**kw) == m.MOE_ERR_INVALID_ARG, kw
    for kw in (dict(d=96), dict(heads=3), dict(heads=4098, qs=4098 * 128), dict(hk=2000, heads=2000), dict(B=(1 << 20) + 1),
               dict(total=(1 << 24) + 1), dict(total=1 << 24, heads=256, qs=256 * 128)):
        assert call(**kw) == m.MOE_ERR_UNSUPPORTED, kw
    assert call(size=m.prompt_attention_workspace_size() - 1) == m.MOE_ERR_WORKSPACE_TOO_SMALL


# ---------------------------------------------------------------- binding
def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_binding_refuses_norm(L):
    good = dict(residual=bf(5, 256), gain=bf(256), codes=torch.zeros((5, 256), dtype=torch.uint8), scales=torch.zeros((2, 8)),
                residual_out=bf(5, 256), eps=1e-6)
    for name, bad in (("residual", bf(5, 256).float()), ("residual", bf(256)), ("gain", bf(255)), ("codes", bf(5, 256)),
                      ("codes", torch.zeros((5, 255), dtype=torch.uint8)), ("scales", torch.zeros((2, 5))),
                      ("scales", torch.zeros((2, 8), dtype=torch.float64)), ("residual_out", bf(5, 512)[:, :256]),
                      ("x", bf(4, 256)), ("x", bf(256, 5).t()), ("out", bf(5, 256).half())):
        with pytest.raises(ValueError, match=name):
            m.rmsnorm_residual_fp8(**{**good, name: bad})
    with pytest.raises(ValueError, match="CUDA"):
        m.rmsnorm_residual_fp8(**good)


def test_binding_refuses_pages(L):
    ws = torch.zeros(4096, dtype=torch.uint8)
    good = dict(page_table=i32(3, 4), lens=i32(3), free_pages=i32(9), free_state=i32(2), page_size=16, num_pages=9,
                lens_out=i32(3), free_out=i32(2), workspace=ws)
    ext = dict(new=i32(3), q_start=i32(4), positions=i32(7), slots=torch.zeros(7, dtype=torch.int64))
    rel = dict(done=torch.zeros(3, dtype=torch.bool))
    shared = [("page_table", i32(3)), ("page_table", i32(4, 3).t()), ("lens", i32(4)), ("lens", i32(3).long()),
              ("free_pages", i32(3, 3)), ("free_state", i32(1)), ("lens_out", i32(2)), ("free_out", i32(3))]
    for f, more, own in ((m.kv_pages_extend, ext, [("new", i32(2)), ("q_start", i32(3)), ("positions", i32(7, 1)),
                                                   ("slots", i32(7)), ("slots", torch.zeros(6, dtype=torch.int64))]),
                         (m.kv_pages_release, rel, [("done", torch.zeros(3)), ("done", torch.zeros(2, dtype=torch.bool))])):
        for name, bad in shared + own:
            with pytest.raises(ValueError, match=name):
                f(**{**good, **more, name: bad})
        with pytest.raises(ValueError, match="CUDA"):
            f(**good, **more)


def test_binding_refuses_prompt_attention(L):
    good = dict(q=bf(9, 4, 64), k=bf(9, 2, 64), v=bf(9, 2, 64), q_start=i32(3), out=bf(9, 4, 64),
                workspace=torch.zeros(4096, dtype=torch.uint8))
    for name, bad in (("q", bf(9, 256)), ("q", bf(9, 4, 64).float()), ("k", bf(8, 2, 64)), ("k", bf(9, 2, 128)),
                      ("v", bf(9, 1, 64)), ("v", bf(9, 64, 2).transpose(1, 2)), ("q_start", i32(0)), ("q_start", i32(3).long()),
                      ("out", bf(9, 4, 64).half()), ("out", bf(9, 64, 4).transpose(1, 2)), ("lse", torch.zeros((9, 3))),
                      ("slopes", torch.zeros(2))):
        with pytest.raises(ValueError, match=name):
            m.prompt_attention(**{**good, name: bad})
    with pytest.raises(ValueError, match="CUDA"):
        m.prompt_attention(**good)


def test_names_of_the_prompt_module():
    from moe_decode_layer_bf16_gb300 import prompt
    for name in m._PROMPT:
        assert getattr(m, name) is getattr(prompt, name) and name in dir(m)
    star = {}
    exec("from moe_decode_layer_bf16_gb300 import *", star)
    assert set(m._PROMPT) <= set(star)


def test_attention_prompt_takes_no_more_tokens_than_it_has_room_for(monkeypatch):
    from moe_decode_layer_bf16_gb300 import attention, prompt
    monkeypatch.setattr(attention, "moe_workspace_init", lambda ws: None)
    monkeypatch.setattr(prompt, "moe_workspace_init", lambda ws: None)
    decode = m.AttentionDecode(128, 2, 1, 64, dict.fromkeys(("qkv", "qkv_s", "o", "o_s")),
                               m.Fp8KvCache(2, 1, 64, 16, device="cpu"), max_tokens=2)
    layer = m.AttentionPrompt(decode, max_tokens=8)
    with pytest.raises(ValueError, match="at most 8"):
        layer(bf(9, 128), None, None, None, 9)
