"""A prompt's operators on the GPU where their documentation allows more than a fresh
allocation, one kernel or one kind of batch: against the oracle, or bit for bit against
the ordinary call."""

import math

import numpy as np
import pytest
import torch

import moe_decode_layer_bf16_gb300 as m
from oracle import prompt_oracle as orc
from oracle.moe_oracle import e4m3_decode
from tests.fixtures_attention import bf16, bf16_values
from tests.test_gpu_prompt import (DEV, check_norm, check_prompt, dev, host, layers, packed, run_prompt, tolerance,
                                   workspace)

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


# ---------------------------------------------------------------- infinities and NaN under caps and biases
MODS = [dict(softcap=20.0), dict(slopes=True), dict(softcap=5.0, slopes=True, window=60)]


def options(kw, heads):
    kw = dict(kw)
    if kw.pop("slopes", False):
        kw["slopes"] = np.exp2(-8.0 * np.arange(1, heads + 1) / heads).astype(np.float32)
    return kw


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kw", MODS)
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_prompt_bad_values_under_caps_and_biases(D, kw, bad):
    rng = np.random.default_rng(47)
    H, hk = 4, 2
    kw = options(kw, H)
    t, v, start = packed(rng, [300, 200], H, hk, D)
    ref = orc.attention(*v, start, 1 / math.sqrt(D), **kw)
    t_out, t_lse = tolerance(ref, D, 300, kw.get("softcap"))
    at, window = [(0, 0, 5), (140, 1, 63), (299, 0, 7), (300, 1, 9), (431, 0, 40)], kw.get("window", 0)
    for r, h, c in at:
        t[2][r, h, c] = bad
    out, lse, status = run_prompt(t, start, **kw)
    assert status == m.MOE_OK and (np.abs(lse - ref[1]) <= t_lse).all()
    hit = np.zeros(out.shape, bool)
    for r, h, c in at:
        end = 300 if r < 300 else 500
        hit[r:min(end, r + window) if window else end, 2 * h:2 * h + 2, c] = True
    assert not np.isfinite(out[hit]).any() and (np.abs(out - ref[0]) <= t_out)[~hit].all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kw", MODS)
def test_prompt_bad_keys_and_queries_under_caps_and_biases(D, kw):
    """A NaN in a key or a query as without caps.  An infinity in a query's row: scores of plus or
    minus the cap, as the formula says; without a cap NaN."""
    rng = np.random.default_rng(48)
    H, hk = 4, 2
    kw = options(kw, H)
    cap, window = kw.get("softcap"), kw.get("window", 0)
    t, v, start = packed(rng, [300, 200], H, hk, D)
    v[0][17, 0, 0] = v[0][333, 2, 1] = np.inf
    t[0][17, 0, 0] = t[0][333, 2, 1] = float("inf")
    with np.errstate(invalid="ignore"):
        ref = orc.attention(*v, start, 1 / math.sqrt(D), **kw)
    scores = [x.copy() for x in ref]
    for a in scores[3:]:  # (such rows' scores are the cap's size, and nothing is lost on the way to it)
        a[17, 0], a[333, 2] = (0.0 if a is scores[3] else cap or 0.0), (0.0 if a is scores[3] else cap or 0.0)
    if "slopes" in kw and cap:
        for r, h, i in ((17, 0, 17), (333, 2, 33)):
            scores[4][r, h] = cap + kw["slopes"][h] * min(i, (window or 1000) - 1)
    t_out, t_lse = tolerance(scores, D, 300, cap)
    t[1][140, 1, 3] = float("nan")
    t[1][420, 0, 90 % D] = float("nan")
    t[0][499, 3, D - 1] = float("nan")
    out, lse, status = run_prompt(t, start, **kw)
    hit = np.zeros(lse.shape, bool)
    hit[140:min(300, 140 + window) if window else 300, 2:] = True
    hit[420:min(500, 420 + window) if window else 500, :2] = True
    hit[499, 3] = True
    if not cap:
        hit[17, 0] = hit[333, 2] = True
    assert status == m.MOE_OK and np.isnan(out[hit]).all() and np.isnan(lse[hit]).all()
    assert (np.abs(out - ref[0]) <= t_out)[~hit].all() and (np.abs(lse - ref[1]) <= t_lse)[~hit].all()


# ---------------------------------------------------------------- batches
def test_prompt_of_many_heads_and_many_empty_prompts():
    rng = np.random.default_rng(49)
    check_prompt(rng, [3, 130], 2048, 1024, 64)
    check_prompt(rng, [2, 1], 4096, 1, 128)
    lens = np.zeros(3000, int)
    lens[[0, 31, 32, 700, 1999, 2999]] = [5, 140, 1, 300, 64, 9]
    check_prompt(rng, lens.tolist(), 6, 2, 64, before=3, after=1)


# ---------------------------------------------------------------- norm
@pytest.mark.parametrize("M,H", [(305, 1024), (999, 656), (304, 1024), (400, 512), (311, 256), (5000, 16), (700, 2048)])
@pytest.mark.parametrize("kw", [dict(x=True, out=True), dict(e8m0=True, extra=8)])
def test_norm_widths_of_many_rows(M, H, kw):
    rng = np.random.default_rng(M * H)
    kw = dict(kw)
    x = bf16_values(rng, (M, H)) if kw.pop("x", False) else None
    check_norm(bf16_values(rng, (M, H), 2.0), bf16(1 + 0.1 * rng.standard_normal(H)).float().numpy(), x, **kw)


@pytest.mark.parametrize("M", [3, 400])
@pytest.mark.parametrize("e8m0", [False, True])
def test_norm_gains_of_any_size(M, e8m0):
    """Groups of columns whose scales lie from 2^-112 to 2^104: the quotient by way of a reciprocal
    has factors of its own at both ends."""
    rng = np.random.default_rng(50)
    H = 1280
    gain = np.repeat(np.exp2([-100.0, -95.0, -90.0, -60.0, 0.0, 60.0, 92.0, 101.0, 110.0, 0.0]), 128)
    gain = bf16(gain * (1 + 0.1 * rng.standard_normal(H))).float().numpy()
    check_norm(bf16_values(rng, (M, H), 2.0), gain, e8m0=e8m0, out=True)


# ---------------------------------------------------------------- the sublayer
def test_attention_prompt_rotates_by_positions():
    """Position encodings by the positions that extend gives, in the prompts and in the steps after them."""
    rng = np.random.default_rng(51)
    hidden, heads, hk, D, lens = 256, 4, 2, 64, [33, 1, 20]
    state = {}

    def rotate(q, k):
        at = state["pages"].positions[:q.shape[0]].float()
        angle = at[:, None] * torch.exp2(-torch.arange(D // 2, device=DEV).float() / 4)[None]
        cos, sin = angle.cos()[:, None], angle.sin()[:, None]
        for x in (q, k):
            a, b = x[..., :D // 2].float(), x[..., D // 2:].float()
            x.copy_(torch.cat([a * cos - b * sin, a * sin + b * cos], -1))

    total = sum(lens)
    cache, att, prompt, pages = layers(rng, hidden, heads, hk, D, 16, 3, 4, total, rotate=rotate)
    state["pages"] = pages
    x = bf16(bf16_values(rng, (total, hidden))).to(DEV)
    pages.extend(dev(np.array(lens, np.int32)))
    assert host(pages.positions).tolist() == [i for n in lens for i in range(n)]
    y = prompt(x, pages.page_table, pages.q_start, pages.lens, max(lens))
    w, ws = att.weights, workspace(att.workspace.numel())
    qkv, mixed, want = (torch.empty(s, dtype=torch.bfloat16, device=DEV) for s in ((total, heads + 2 * hk, D), (total, heads, D), (total, hidden)))
    m.fp8_linear(x, w["qkv"], w["qkv_s"], qkv.flatten(1), ws)
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + hk], qkv[:, heads + hk:]
    plain = k.clone()
    rotate(q, k)
    assert not torch.equal(plain, k)
    m.prompt_attention(q, k, v, pages.q_start, mixed, ws)
    m.fp8_linear(mixed.flatten(1), w["o"], w["o_s"], want, ws)
    assert torch.equal(y, want)
    # the cache holds the rotated keys: half a step of E4M3, 2^-4 of a normal value, 2^-10 scales below 2^-6
    table, codes, scales = host(pages.page_table), e4m3_decode(host(cache.k)), host(cache.k_scale).astype(np.float64)
    for b, n in enumerate(lens):
        lo = int(sum(lens[:b]))
        for i in range(n):
            page, at = int(table[b, i // 16]), i % 16
            held, sc, want_k = codes[page, :, at], scales[page][:, None], host(k[lo + i])
            assert (np.abs(held * sc - want_k) <= np.maximum(np.abs(want_k) * 2.0 ** -4, sc * 2.0 ** -10)).all()
    # a step of a token each: the same by single calls, whose queries and keys are rotated by the new positions
    pages.extend(torch.ones(3, dtype=torch.int32, device=DEV))
    assert host(pages.positions)[:4].tolist() == [*lens, -1]
    last = x[:3].contiguous()
    out = att(last, pages.page_table, pages.q_start, pages.lens)
    step, attended, got = (torch.empty(s, dtype=torch.bfloat16, device=DEV) for s in ((3, heads + 2 * hk, D), (3, heads, D), (3, hidden)))
    m.fp8_linear(last, w["qkv"], w["qkv_s"], step.flatten(1), ws)
    rotate(step[:, :heads], step[:, heads:heads + hk])
    m.decode_attention(step[:, :heads], cache.k, cache.v, cache.k_scale, cache.v_scale, pages.page_table, pages.q_start, pages.lens, 1,
                       attended, ws)
    m.fp8_linear(attended.flatten(1), w["o"], w["o_s"], got, ws)
    assert torch.equal(out, got)
    assert (att.status(), prompt.status(), pages.status()) == (m.MOE_OK,) * 3


def test_attention_prompt_of_no_tokens():
    rng = np.random.default_rng(52)
    cache, att, prompt, pages = layers(rng, 128, 2, 1, 64, 16, 2, 4, 8)
    pages.extend(torch.zeros(2, dtype=torch.int32, device=DEV))
    x = torch.zeros((0, 128), dtype=torch.bfloat16, device=DEV)
    quantised = torch.zeros((0, 128), dtype=torch.uint8, device=DEV), torch.zeros((1, 0), device=DEV)
    for rows in (x, quantised):
        assert prompt(rows, pages.page_table, pages.q_start, pages.lens, 1).shape == (0, 128)
    assert prompt.status() == pages.status() == m.MOE_OK
