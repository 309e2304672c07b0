"""A prompt's operators on the GPU where their documentation allows more than a fresh
allocation, one kernel or one kind of batch: against the oracle, or bit for bit against
the ordinary call."""

import numpy as np
import pytest
import torch

import moe_decode_layer_bf16_gb300 as m
from oracle import prompt_oracle as orc
from tests.fixtures_attention import bf16, bf16_values
from tests.test_gpu_prompt import DEV, dev, host, layers, packed, run_prompt, tolerance, workspace

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


# ---------------------------------------------------------------- waits that give up
@pytest.mark.parametrize("D,G", [(64, 2), (128, 5)])
def test_prompt_gives_up_as_a_whole(D, G):
    """With an earlier call's time-out still in the status word no wait lasts longer than some
    milliseconds, which an item of this document does: whatever has been reached by then, the
    call ends, says so, leaves the rows of no prompt and the workspace as they were, and the
    next call is right."""
    g = torch.Generator(device=DEV)
    g.manual_seed(41)
    n = 200000
    qkv = torch.randn((n + 2, G + 2, D), generator=g, device=DEV).to(torch.bfloat16)
    out, ws = torch.full((n + 2, G, D), 7.0, dtype=torch.bfloat16, device=DEV), workspace()
    ws.view(torch.int32)[0] = m.MOE_ERR_DEVICE_TIMEOUT
    start = dev(np.array([1, n + 1], np.int32))
    m.prompt_attention(qkv[:, :G], qkv[:, G:G + 1], qkv[:, G + 1:], start, out, ws)
    assert m.moe_device_status(ws) == m.MOE_ERR_DEVICE_TIMEOUT and not ws.any()
    assert bool((out[0] == 7).all()) and bool((out[n + 1] == 7).all())
    t, v, start = packed(np.random.default_rng(42), [300, 40], 6, 2, D)
    got, want = run_prompt(t, start, ws=ws), run_prompt(t, start)
    assert got[2] == m.MOE_OK and np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


# ---------------------------------------------------------------- what a row depends on
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,hk", [(7, 1), (1, 3), (40, 1)])
@pytest.mark.parametrize("kw", [dict(), dict(softcap=25.0), dict(window=90)])
def test_prompt_with_another_end(D, G, hk, kw):
    """The rows of a prompt's start are the same bit for bit whatever follows them, and a head's
    whatever the other heads hold: the running maximum of loud rows moves while that of the
    quiet ones, a warp's other rows, stays."""
    rng = np.random.default_rng(43)
    n, same = 500, 311
    t, v, start = packed(rng, [n], G * hk, hk, D)
    q, k, val = (x.clone() for x in t)
    k[:] *= torch.linspace(0.2, 3.0, n, device=DEV).to(torch.bfloat16)[:, None, None]  # (scores grow along the rows)
    first = run_prompt((q, k, val), start, **kw)
    q[same:] *= 30.0
    k[same:] *= -2.0
    if G > 1:
        q[:, 1::2] *= 16.0
    after = run_prompt((q, k, val), start, **kw)
    heads = slice(0, None, 2) if G > 1 else slice(None)
    assert first[2] == after[2] == m.MOE_OK
    assert np.array_equal(first[0][:same, heads], after[0][:same, heads]) and np.array_equal(first[1][:same, heads], after[1][:same, heads])
    alone = run_prompt([x[:same] for x in (q, k, val)], np.array([0, same], np.int32), **kw)
    assert np.array_equal(alone[0], after[0][:same]) and np.array_equal(alone[1], after[1][:same])


# ---------------------------------------------------------------- caps
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sm_scale", [1e9, -1e9, 3e38])
@pytest.mark.parametrize("softcap", [1e-30, 1e-38])
def test_prompt_caps_far_below_the_scale(D, sm_scale, softcap):
    """Scores within 1e-30 of zero, some of them zero itself: every row is the mean of what it
    sees, as with queries of zeros."""
    rng = np.random.default_rng(44)
    t, v, start = packed(rng, [200, 9], 4, 2, D)
    q = t[0].clone()
    q[50:90] = 0.0
    q[120, 1] = 0.0
    out, lse, status = run_prompt((q, t[1], t[2]), start, sm_scale, softcap=softcap)
    ref = orc.attention(np.zeros_like(v[0]), v[1], v[2], start, 1.0)
    t_out, t_lse = tolerance(ref, D, 200)
    assert status == m.MOE_OK and (np.abs(out - ref[0]) <= t_out).all() and (np.abs(lse - ref[1]) <= t_lse).all()


# ---------------------------------------------------------------- sequences that go on
@pytest.mark.parametrize("n", [5, 45])  # (prompts are looked at 32 at a time)
def test_prompts_that_go_on_are_left_out(n):
    rng = np.random.default_rng(45)
    rows = rng.integers(0, 60, n)
    t, v, start = packed(rng, rows.tolist(), 4, 2, 64)
    want = run_prompt(t, start)
    exact = np.where(rows > 0, rows, rng.integers(0, 9, n)).astype(np.int32)  # (what has no rows may hold anything)
    same = run_prompt(t, start, lens=dev(exact))
    assert same[2] == m.MOE_OK and np.array_equal(same[0], want[0]) and np.array_equal(same[1], want[1])
    on = (rng.random(n) < 0.4) & (rows > 0)
    on[rows.argmax()] = True
    for lens in (exact + 7 * on, np.where(on, exact - 1, exact), np.where(on, -2 ** 31, exact)):
        out, lse, status = run_prompt(t, start, lens=dev(lens.astype(np.int32)))
        gone = np.repeat(on, rows)
        assert status == m.MOE_ERR_INVALID_ARG
        assert (out[gone] == 7).all() and (lse[gone] == 7).all()
        assert np.array_equal(out[~gone], want[0][~gone]) and np.array_equal(lse[~gone], want[1][~gone])


def test_attention_prompt_reports_a_sequence_that_goes_on():
    """A step of new prompts and of one sequence that holds more than the step's rows."""
    rng = np.random.default_rng(46)
    hidden = 128
    cache, att, prompt, pages = layers(rng, hidden, 2, 1, 64, 16, 3, 6, 60)
    new = [np.array(x, np.int32) for x in ([0, 20, 0], [30, 1, 9])]
    x = bf16(bf16_values(rng, (40, hidden))).to(DEV)
    pages.extend(dev(new[0]))
    prompt(x[:20], pages.page_table, pages.q_start, pages.lens, 20)
    assert prompt.status() == m.MOE_OK  # (sequences without rows are left alone)
    pages.extend(dev(new[1]))
    out = prompt(x, pages.page_table, pages.q_start, pages.lens, 30)
    assert prompt.status() == m.MOE_ERR_INVALID_ARG
    alone = m.KvPages(cache, 2, 6, 60)
    alone.extend(dev(np.array([30, 9], np.int32)))
    rows = list(range(30)) + list(range(31, 40))
    want = prompt(x[rows].contiguous(), alone.page_table, alone.q_start, alone.lens, 30)
    assert prompt.status() == m.MOE_OK
    # (the projections' cells are the same for 39 and 40 rows)
    assert torch.equal(out[rows], want)


# ---------------------------------------------------------------- pages
def test_pages_report_who_was_not_served():
    """More rows than the step has room for, and a sequence that outgrows its table."""
    cache = m.Fp8KvCache(40, 1, 64, 16)
    p = m.KvPages(cache, 3, 4, max_rows=50)
    assert p.status() == m.MOE_OK
    for new, lens, status in (([20, 10, 20], [20, 10, 20], m.MOE_OK), ([30, 21, 0], [50, 10, 20], m.MOE_ERR_INVALID_ARG),
                              ([1, 1, 45], [51, 11, 20], m.MOE_ERR_INVALID_ARG), ([0, 1, 1], [51, 12, 21], m.MOE_OK)):
        p.extend(dev(np.array(new, np.int32)))
        assert host(p.lens).tolist() == lens and int(p.q_start[-1]) <= 50
        assert p.status() == status and p.status() == m.MOE_OK
    p.release(torch.ones(3, dtype=torch.bool, device=DEV))
    assert p.status() == m.MOE_OK and host(p.free).tolist() == [40, 0]
