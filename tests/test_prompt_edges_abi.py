"""A prompt's operators on the host: what is refused beside the plain calls' refusals
(no GPU)."""

import os

import pytest
import torch

import moe_decode_layer_bf16_gb300 as m
from tests.test_prompt_abi import BIG, FAKE, ODD, bf, i32


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(m.LIB_PATH):
        from moe_decode_layer_bf16_gb300 import build
        build.build()
    return m.lib()


def test_prompt_attention_checked_refusals(L):
    def call(q=FAKE, start=FAKE, lens=FAKE, B=2, total=9, out=FAKE, ws=FAKE, size=BIG, d=128, cap=0.0):
        return L.prompt_attention_checked(q, 512, FAKE, 256, FAKE, 256, 4, 2, d, start, lens, B, total, 0.1, cap, 0, None, out,
                                          None, ws, size, None)

    for lens in (None, FAKE):
        assert call(lens=lens, B=0) == m.MOE_OK and call(lens=lens, total=0) == m.MOE_OK
        for kw in (dict(q=None), dict(start=None), dict(out=ODD), dict(ws=None), dict(B=-1), dict(cap=-1.0)):
            assert call(lens=lens, **kw) == m.MOE_ERR_INVALID_ARG, kw
        assert call(lens=lens, d=96) == m.MOE_ERR_UNSUPPORTED
        assert call(lens=lens, size=m.prompt_attention_workspace_size() - 1) == m.MOE_ERR_WORKSPACE_TOO_SMALL


def test_binding_refuses_lens(L):
    good = dict(q=bf(9, 4, 64), k=bf(9, 2, 64), v=bf(9, 2, 64), q_start=i32(3), out=bf(9, 4, 64),
                workspace=torch.zeros(4096, dtype=torch.uint8))
    for bad in (i32(3), i32(2, 1), i32(2).long(), i32(4)[::2]):
        with pytest.raises(ValueError, match="lens"):
            m.prompt_attention(**good, lens=bad)
    with pytest.raises(ValueError, match="CUDA"):
        m.prompt_attention(**good, lens=i32(2))
