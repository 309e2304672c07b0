"""A prompt's operators on the GPU where their documentation allows more than a fresh
allocation, one kernel or one kind of batch: against the oracle, or bit for bit against
the ordinary call."""

import numpy as np
import pytest
import torch

import moe_decode_layer_bf16_gb300 as m
from tests.test_gpu_prompt import DEV, dev, host, packed, run_prompt, workspace

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- where results lie
@pytest.mark.parametrize("at", [0, 8, 16, 24])  # bf16 values from the allocation's start
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_results_at_any_16_bytes(D, at):
    rng = np.random.default_rng(40)
    t, v, start = packed(rng, [150, 3], 6, 2, D, before=1, after=2)
    want = run_prompt(t, start)[0]
    n = want.size
    room = torch.full((n + 64,), 7.0, dtype=torch.bfloat16, device=DEV)
    out, ws = room[at:at + n].view(want.shape), workspace()
    assert out.data_ptr() % 32 == 2 * at % 32
    m.prompt_attention(*t, dev(start), out, ws)
    assert m.moe_device_status(ws) == m.MOE_OK and np.array_equal(host(out), want)
    assert bool((room[:at] == 7).all()) and bool((room[at + n:] == 7).all())
