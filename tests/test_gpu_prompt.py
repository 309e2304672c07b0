"""A prompt's operators on the GPU against the oracle (oracle/prompt_oracle.py): whole
numbers and the new residual exactly, computed values within tolerances that count
their roundings."""

import importlib.util
import math
import os

import numpy as np
import pytest
import torch

import moe_decode_layer_bf16_gb300 as m
from oracle import prompt_oracle as orc
from oracle.moe_oracle import e4m3_decode
from tests.fixtures_attention import BF16, F32, bf16, bf16_values, weights

pytestmark = pytest.mark.gpu
DEV = "cuda"


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64) if t.dtype == torch.bfloat16 else t.detach().cpu().numpy()


def workspace(n=None):
    return torch.zeros(n or m.prompt_attention_workspace_size(), dtype=torch.uint8, device=DEV)


def spaced(x, extra):
    """x as rows of a wider matrix whose other columns are NaN."""
    wide = torch.full((x.shape[0], x.shape[1] + extra), float("nan"), dtype=x.dtype, device=DEV)
    wide[:, 8:8 + x.shape[1]] = x
    return wide[:, 8:8 + x.shape[1]]


# ---------------------------------------------------------------- pages (bad values first: they must not fault)
def paged(rng, lens, page, width, spare):
    """A table whose sequences hold their pages, and a stack of `spare` more."""
    held = [-(-n // page) if n > 0 else 0 for n in lens]
    total = sum(held) + spare
    order = rng.permutation(total).astype(np.int32)
    table = np.full((len(lens), width), -1, np.int32)
    at = spare
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    stack = np.full(total, -1, np.int32)
    stack[:spare] = order[:spare]
    return table, stack, total


def run_extend(table, lens, new, stack, state, page, pages, rows, in_place=False, ws=None):
    t = {"table": dev(table), "lens": dev(np.array(lens, np.int32)), "new": dev(np.array(new, np.int32)), "stack": dev(stack),
         "state": dev(np.array(state, np.int32))}
    B = len(lens)
    lens_out = t["lens"] if in_place else torch.full((B,), -9, dtype=torch.int32, device=DEV)
    state_out = t["state"] if in_place else torch.full((2,), -9, dtype=torch.int32, device=DEV)
    q = torch.full((B + 1,), -9, dtype=torch.int32, device=DEV)
    pos = torch.full((rows,), -9, dtype=torch.int32, device=DEV)
    slots = torch.full((rows,), -9, dtype=torch.int64, device=DEV)
    ws = workspace() if ws is None else ws
    m.kv_pages_extend(t["table"], t["lens"], t["new"], t["stack"], t["state"], page, pages, q, lens_out, state_out, pos, slots,
                      ws)
    status = m.moe_device_status(ws)
    assert not ws.any(), "the workspace is left as it was found"
    assert np.array_equal(host(t["stack"]), stack)
    return [host(x) for x in (t["table"], q, lens_out, state_out, pos, slots)], status


def check_extend(table, lens, new, stack, state, page, pages, rows, **kw):
    got, status = run_extend(table, lens, new, stack, state, page, pages, rows, **kw)
    want = orc.extend(table, lens, new, stack, state, page, pages, rows)
    for name, g, w in zip(("table", "q_start", "lens", "state", "positions", "slots"), got, want):
        assert np.array_equal(g, w), (name, np.argwhere(g != w)[:5])
    assert (status == m.MOE_OK) == want[-1] and status in (m.MOE_OK, m.MOE_ERR_INVALID_ARG)


@pytest.mark.parametrize("what", ["length", "new", "too_long", "page_on_stack", "page_in_table", "state", "state_negative",
                                  "rows"])
def test_extend_bad_values(what):
    rng = np.random.default_rng(1)
    lens, new, page = [5, 16, 40, 3], [20, 3, 0, 9], 16
    table, stack, pages = paged(rng, lens, page, 4, 6)
    state, rows = [6, 0], 40
    if what == "length":
        lens[1] = -3
    elif what == "new":
        new[2] = -2 ** 31
    elif what == "too_long":
        new[0] = 60
    elif what == "page_on_stack":
        stack[5] = pages
    elif what == "page_in_table":
        table[3, 0] = -7
    elif what == "state":
        state[0] = len(stack) + 1
    elif what == "state_negative":
        state[0] = -1
    elif what == "rows":
        rows = 25
    check_extend(table, lens, new, stack, state, page, pages, rows)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("B,hi,t", [(1, 0, 1), (1, 1, 200), (5, 300, 3), (64, 5000, 1), (300, 90, 140), (1025, 40, 2),
                                    (2500, 70, 1)])
@pytest.mark.parametrize("spare", [0.0, 0.6, 1.0])
def test_extend(page, B, hi, t, spare):
    rng = np.random.default_rng(B + page)
    lens, new = rng.integers(0, hi + 1, B).tolist(), rng.integers(0, t + 1, B).tolist()
    width = max(-(-(n + k) // page) for n, k in zip(lens, new)) + 1
    need = sum(-(-(n + k) // page) - -(-n // page) for n, k in zip(lens, new))
    table, stack, pages = paged(rng, lens, page, width, math.ceil(need * spare))
    check_extend(table, lens, new, stack, [math.ceil(need * spare), 5], page, max(pages, 1), sum(new) + 7,
                 in_place=B % 2 == 0)


def test_extend_of_nothing():
    check_extend(np.zeros((0, 3), np.int32), [], [], np.arange(4, dtype=np.int32), [4, 0], 16, 4, 5)
    check_extend(np.full((2, 3), -1, np.int32), [0, 7], [0, 0], np.zeros(0, np.int32), [0, 0], 16, 4, 0)


@pytest.mark.parametrize("what", ["length", "page", "state", "full"])
def test_release_bad_values(what):
    rng = np.random.default_rng(2)
    lens, page = [5, 16, 40, 3], 16
    table, stack, pages = paged(rng, lens, page, 4, 2)
    state = [2, 0]
    if what == "length":
        lens[2] = 65
    elif what == "page":
        table[0, 0] = pages + 3
    elif what == "state":
        state[0] = -5
    elif what == "full":
        state[0] = len(stack) - 4
    check_release(table, lens, [True, False, True, True], stack, state, page, pages)


def check_release(table, lens, done, stack, state, page, pages, in_place=False):
    t, s = dev(table), dev(stack)
    n, f = dev(np.array(lens, np.int32)), dev(np.array(state, np.int32))
    lens_out = n if in_place else torch.full_like(n, -9)
    state_out = f if in_place else torch.full_like(f, -9)
    ws = workspace()
    m.kv_pages_release(t, n, dev(np.array(done)), s, f, page, pages, lens_out, state_out, ws)
    status = m.moe_device_status(ws)
    want = orc.release(table, lens, done, stack, state, page, pages)
    for name, g, w in zip(("stack", "lens", "state"), (s, lens_out, state_out), want):
        assert np.array_equal(host(g), w), name
    assert np.array_equal(host(t), table) and not ws.any()
    assert (status == m.MOE_OK) == want[-1]


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("B,hi,share", [(1, 1, 1.0), (1, 900, 1.0), (7, 300, 0.5), (64, 9000, 0.1), (500, 3000, 0.9),
                                        (1500, 100, 0.4), (3, 50, 0.0)])
def test_release(page, B, hi, share):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, hi + 1, B).tolist()
    table, stack, pages = paged(rng, lens, page, max(1, -(-hi // page)), 3)
    check_release(table, lens, rng.random(B) < share, stack, [3, 9], page, pages, in_place=B % 2 == 1)


def test_pages_come_and_go():
    """Steps of a batch in place: no page is held twice, and all come back."""
    rng = np.random.default_rng(3)
    cache = m.Fp8KvCache(60, 1, 64, 16)
    p = m.KvPages(cache, 9, 10, max_rows=200)
    for step in range(12):
        p.extend(dev(rng.integers(0, 30, 9).astype(np.int32)))
        lens, table, free = host(p.lens), host(p.page_table), host(p.free)
        held = [int(x) for b in range(9) for x in table[b, :-(-int(lens[b]) // 16)]]
        on_stack = host(p.free_pages)[:free[0]].tolist()
        assert sorted(held + on_stack) == list(range(60))
        p.release(dev(rng.random(9) < 0.3))
    p.release(torch.ones(9, dtype=torch.bool, device=DEV))
    m.moe_device_status(p.workspace)  # (a sequence may have outgrown its table)
    assert host(p.free).tolist() == [60, 0] and sorted(host(p.free_pages).tolist()) == list(range(60))


def test_pages_captured_and_replayed():
    rng = np.random.default_rng(4)
    cache = m.Fp8KvCache(64, 1, 64, 16)
    p = m.KvPages(cache, 4, 16, max_rows=8)
    new = torch.ones(4, dtype=torch.int32, device=DEV)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        p.extend(new)
    torch.cuda.synchronize()
    want = np.zeros(4, np.int32)
    for _ in range(20):
        t = rng.integers(0, 3, 4).astype(np.int32)
        new.copy_(dev(t))
        graph.replay()
        want += t
        assert np.array_equal(host(p.lens), want) and host(p.q_start).tolist() == np.concatenate([[0], np.cumsum(t)]).tolist()


# ---------------------------------------------------------------- norm
def run_norm(r, gain, x=None, out=False, e8m0=False, eps=1e-6, extra=0, in_place=False):
    M, H = r.shape
    rt, xt = bf16(r).to(DEV), None if x is None else bf16(x).to(DEV)
    if extra:
        rt, xt = spaced(rt, extra), None if xt is None else spaced(xt, extra + 16)
    codes = torch.full((M, H), 0x55, dtype=torch.uint8, device=DEV)
    scales = torch.full((-(-H // 128), M + 3 & -4), -7.0, device=DEV)
    ro = rt if in_place else torch.empty((M, H), dtype=torch.bfloat16, device=DEV)
    o = torch.empty((M, H), dtype=torch.bfloat16, device=DEV) if out else None
    m.rmsnorm_residual_fp8(rt, bf16(gain).to(DEV), codes, scales, ro, eps, x=xt, out=o, e8m0=e8m0)
    assert bool((scales[:, M:] == -7.0).all())  # left as they were
    return host(ro), host(codes), host(scales)[:, :M].astype(np.float64), None if o is None else host(o)


def check_norm(r, gain, x=None, e8m0=False, eps=1e-6, **kw):
    """The sum of squares is off by at most 32 + 10 + 2 roundings of half an fp32 step of
    itself (a thread's values, two reductions over lanes, the squares), its inverse root by
    half of that and 4 more, y by 2 more: under 2^-18 in all."""
    M, H = r.shape
    new, y, amax = orc.norm(r, gain, eps, x)
    ro, codes, scales, out = run_norm(r, gain, x, e8m0=e8m0, eps=eps, **kw)
    assert np.array_equal(ro, new)
    e = 2.0 ** -18
    if out is not None:
        assert (np.abs(out - y) <= (BF16 * (1 + e) + e) * np.abs(y)).all()
    if e8m0:
        lo, hi = (np.exp2(np.ceil(np.log2(np.where(amax > 0, amax, 1.0) * f))) for f in (1 - e, 1 + e))
        assert ((scales == lo) | (scales == hi)).all()
    else:
        assert (np.abs(scales - np.where(amax > 0, amax, 1.0)) <= (e + 2 * F32) * scales).all()
    s = np.repeat(scales.T, 128, axis=1)[:, :H]
    q = y / s
    # half a step of E4M3: 2^-4 of a normal value, 2^-10 below 2^-6
    assert (np.abs(e4m3_decode(codes) - q) <= np.maximum(np.abs(q) * 2.0 ** -4, 2.0 ** -10) * (1 + 2.0 ** -10) + 2 * e * np.abs(q)).all()


@pytest.mark.parametrize("M,H", [(1, 16), (1, 128), (3, 144), (1, 7168), (5, 7168), (2, 8192), (1, 8208), (4, 16384), (37, 2064),
                                 (310, 128), (400, 7168), (306, 1040), (305, 9008), (1021, 272)])
@pytest.mark.parametrize("kw", [dict(), dict(x=True, out=True, extra=40), dict(x=True, e8m0=True, in_place=True),
                                dict(out=True, e8m0=True, extra=8)])
def test_norm(M, H, kw):
    rng = np.random.default_rng(M + H)
    kw = dict(kw)
    loud = np.where(rng.random(H) > 0.98, 16.0, 1.0)
    r = bf16_values(rng, (M, H), 3.0) * loud
    x = bf16_values(rng, (M, H)) if kw.pop("x", False) else None
    check_norm(bf16(r).float().numpy(), bf16(1 + 0.1 * rng.standard_normal(H)).float().numpy(), x, **kw)


def test_norm_is_the_two_calls_but_for_one_rounding():
    """rmsnorm_residual and then fp8_quant_rows, whose input is rounded to bf16 in between."""
    rng = np.random.default_rng(7)
    M, H = 64, 7168
    r, x, gain = bf16_values(rng, (M, H), 2.0), bf16_values(rng, (M, H)), bf16(1 + 0.1 * rng.standard_normal(H)).float().numpy()
    ro, codes, scales, out = run_norm(r, gain, x, out=True)
    o2, r2 = (torch.empty((M, H), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    m.rmsnorm_residual(bf16(r).to(DEV), bf16(gain).to(DEV), o2, r2, 1e-6, x=bf16(x).to(DEV))
    assert np.array_equal(ro, host(r2))
    # the means are summed in another order: 2^-18 apart, at most one bf16 step where that crosses a border
    assert (np.abs(out - host(o2)) <= 2 * BF16 * np.abs(out)).all() and (out != host(o2)).mean() < 1e-3
    c2, s2 = torch.empty((M, H), dtype=torch.uint8, device=DEV), torch.empty((H // 128, M), device=DEV)
    m.fp8_quant_rows(o2, c2, s2)
    a = e4m3_decode(codes) * np.repeat(scales.T, 128, 1)
    b = e4m3_decode(host(c2)) * np.repeat(host(s2).T, 128, 1)
    # a code's half step twice, and the bf16 rounding of the value and of the scale
    big = np.repeat(scales.T, 128, 1)
    assert (np.abs(a - b) <= np.maximum(np.abs(b) * 2.0 ** -3, big * 2.0 ** -9) + 3 * BF16 * np.abs(b) + 3 * BF16 * big).all()


def test_norm_of_zeros_and_of_values_that_are_none():
    rng = np.random.default_rng(8)
    M, H = 6, 400
    r = bf16_values(rng, (M, H))
    r[1] = 0.0
    r[2, 5], r[3, 399] = np.nan, np.inf
    gain = np.ones(H, np.float32)
    ro, codes, scales, out = run_norm(r, gain, out=True)
    assert (codes[1] & 0x7F == 0).all() and (scales[:, 1] == 1.0).all()
    assert np.isnan(out[2]).all() and (codes[2] & 0x7F == 0x7F).all()
    assert np.isnan(out[3, 399]) and (out[3, :399] == 0).all()  # (the mean is infinite)
    good = [0, 4, 5]
    alone = run_norm(r[good], gain, out=True)
    assert np.array_equal(codes[good], alone[1]) and np.array_equal(scales[:, good], alone[2]) and np.array_equal(out[good], alone[3])


def test_norm_far_rows():
    """Rows more than 2^31 elements from the first."""
    M, H, step = 3, 256, (1 << 30) + 8
    wide = torch.empty(2 * step + H, dtype=torch.bfloat16, device=DEV)
    r = wide.as_strided((M, H), (step, 1))
    v = torch.randn((M, H), device=DEV).to(torch.bfloat16)
    r.copy_(v)
    outs = []
    for t in (r, v):
        codes, scales = torch.empty((M, H), dtype=torch.uint8, device=DEV), torch.zeros((2, 4), device=DEV)
        ro = torch.empty_like(v)
        m.rmsnorm_residual_fp8(t, torch.ones(H, dtype=torch.bfloat16, device=DEV), codes, scales, ro, 1e-6)
        outs.append((codes, scales, ro))
    assert all(torch.equal(a, b) for a, b in zip(*outs))


# ---------------------------------------------------------------- prompt attention
def packed(rng, lens, heads, hk, D, before=0, after=0, poison=True):
    """q, k, v as columns of one matrix (on the GPU), and their values; rows of no prompt are NaN."""
    total = before + sum(lens) + after
    qkv = bf16_values(rng, (total, heads + 2 * hk, D))
    qkv[:, :heads] *= 2.0
    if poison:
        qkv[:before] = np.nan
        qkv[total - after:] = np.nan
    t = bf16(qkv).to(DEV)
    start = (before + np.concatenate([[0], np.cumsum(lens)])).astype(np.int32)
    return (t[:, :heads], t[:, heads:heads + hk], t[:, heads + hk:]), (qkv[:, :heads], qkv[:, heads:heads + hk], qkv[:, heads + hk:]), start


def run_prompt(t, start, sm_scale=None, ws=None, lse=True, **kw):
    total, H, D = t[0].shape
    out = torch.full((total, H, D), 7.0, dtype=torch.bfloat16, device=DEV)
    ls = torch.full((total, H), 7.0, device=DEV) if lse else None
    ws = workspace() if ws is None else ws
    if kw.get("slopes") is not None:
        kw["slopes"] = dev(kw["slopes"])
    m.prompt_attention(*t, dev(start), out, ws, lse=ls, sm_scale=sm_scale, **kw)
    status = m.moe_device_status(ws)
    assert not ws.any(), "the workspace is left as it was found"
    return host(out), None if ls is None else host(ls), status


def tolerance(ref, D, n, softcap=0.0):
    """A score: exact products, each of the D additions off by at most a step (2 F32) of
    sum |q k|; scaling, bias and change to base 2 by 8 roundings of the scores' size; a cap by
    2^-20 of the capped score (its polynomial or quotient 2^-21, two products).  A weight:
    twice that (its own and the sum's), the exponential's 2^-22 twice, its rounding to bf16.
    Sums over tokens: a step for each group of 16 in the products, n / 4 + 16 additions of the
    row's sum."""
    out, lse, mag, unit, big = ref
    e = 2 * F32 * D * unit + 8 * F32 * (unit + big) + (2.0 ** -20 * big if softcap else 0.0)
    sums = (n / 4 + 16) * F32
    w = 2 * e + 2.0 ** -21 + BF16 + sums + 2 * F32 * (n / 16 + 8)
    t_out = w[..., None] * mag
    return t_out + BF16 * (np.abs(out) + t_out), e + 2.0 ** -22 + sums + 4 * F32 * np.abs(lse)


def check_prompt(rng, lens, heads, hk, D, before=0, after=0, sm_scale=None, **kw):
    t, v, start = packed(rng, lens, heads, hk, D, before, after)
    out, lse, status = run_prompt(t, start, sm_scale, **kw)
    assert status == m.MOE_OK
    ref = orc.attention(*v, start, 1 / math.sqrt(D) if sm_scale is None else sm_scale, **kw)
    t_out, t_lse = tolerance(ref, D, max(lens), kw.get("softcap"))
    rows = slice(int(start[0]), int(start[-1]))
    d, dl = np.abs(out - ref[0])[rows], np.abs(lse - ref[1])[rows]
    assert (d <= t_out[rows]).all(), (np.argwhere(d > t_out[rows])[:4], (d / t_out[rows]).max())
    assert (dl <= t_lse[rows]).all(), (np.argwhere(dl > t_lse[rows])[:4], (dl / t_lse[rows]).max())
    for a in (out, lse):
        assert (a[:rows.start] == 7).all() and (a[rows.stop:] == 7).all()


@pytest.mark.parametrize("start", [[0, 5, 3, 20], [0, 9, 4, 9, 9, 20], [0, 20] * 40, [0, 40, 20, 20], [-4, 5, 9, 20], [0, 5, 2 ** 31 - 1, 20], [0, 5, 9, 21],
                                   [-2 ** 31, 2 ** 31 - 1, 9, 20]])
def test_prompt_bad_starts(start):
    """Prompts that do not lie among the rows are left out and reported."""
    rng = np.random.default_rng(10)
    t, v, _ = packed(rng, [20], 2, 1, 64)
    out, lse, status = run_prompt(t, np.array(start, np.int32))
    assert status == m.MOE_ERR_INVALID_ARG
    held, end = np.zeros(20, bool), 0
    for a, b in zip(start[:-1], start[1:]):
        if 0 <= a <= b <= 20 and a >= end:  # (nor does one start before an earlier one ends)
            ref = orc.attention(*v, [a, b], 1 / 8)
            assert (np.abs(out - ref[0]) <= tolerance(ref, 64, 20)[0])[a:b].all()
            held[a:b], end = True, b
    assert (out[~held] == 7).all() and (lse[~held] == 7).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,heads,hk", [([1], 1, 1), ([2, 1, 0, 3], 3, 1), ([127, 128, 129], 1, 1), ([640], 16, 16),
                                           ([513, 257], 2, 2), ([255, 0, 256, 1, 300], 5, 1), ([33], 56, 8), ([90, 300], 14, 2),
                                           ([70, 130], 24, 2), ([40, 3], 40, 1), ([9, 130], 97, 1), ([5], 300, 1),
                                           ([1100], 7, 1), ([1025], 1, 1)])
def test_prompt(D, lens, heads, hk):
    check_prompt(np.random.default_rng(sum(lens) + heads), lens, heads, hk, D, before=5, after=9)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kw", [dict(window=1), dict(window=2), dict(window=127), dict(window=128), dict(window=129),
                                dict(window=300), dict(window=2 ** 31 - 1), dict(softcap=30.0), dict(softcap=2.0),
                                dict(softcap=1e-3), dict(softcap=3e38), dict(slopes=True), dict(softcap=20.0, slopes=True, window=65),
                                dict(sm_scale=-0.2), dict(sm_scale=0.0), dict(sm_scale=1e-35), dict(sm_scale=3.0)])
def test_prompt_options(D, kw):
    kw = dict(kw)
    if kw.pop("slopes", False):
        kw["slopes"] = np.exp2(-8.0 * np.arange(1, 7) / 6).astype(np.float32)
    check_prompt(np.random.default_rng(11), [390, 17, 700], 6, 2, D, **kw)


def test_prompt_of_many():
    """More prompts than are looked at together, and more items than CTAs."""
    rng = np.random.default_rng(12)
    check_prompt(rng, rng.integers(0, 90, 77).tolist(), 4, 2, 64)
    check_prompt(rng, [1] * 500, 2, 2, 128)


@pytest.mark.parametrize("window", [0, 60])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_prompt_bad_values_reach_the_rows_that_see_them(window, bad):
    rng = np.random.default_rng(13)
    lens, H, hk, D = [300, 200], 4, 2, 64
    t, v, start = packed(rng, lens, H, hk, D)
    ref = orc.attention(*v, start, 1 / 8, window=window)
    t_out, t_lse = tolerance(ref, D, 300)
    at = [(0, 0, 5), (140, 1, 63), (299, 0, 7), (300, 1, 9), (431, 0, 40)]  # (row, kv head, column)
    for r, h, c in at:
        t[2][r, h, c] = bad
    out, lse, status = run_prompt(t, start, window=window)
    assert status == m.MOE_OK and (np.abs(lse - ref[1]) <= t_lse).all()
    hit = np.zeros(out.shape, bool)
    for r, h, c in at:
        end = 300 if r < 300 else 500
        hit[r:min(end, r + window) if window else end, 2 * h:2 * h + 2, c] = True
    assert not np.isfinite(out[hit]).any() and (np.abs(out - ref[0]) <= t_out)[~hit].all()
    if np.isinf(bad):
        assert (out[hit] == bad).mean() > 0.9  # (NaN where the weight is below what bf16 holds)


@pytest.mark.parametrize("window", [0, 60])
def test_prompt_bad_keys_and_queries(window):
    rng = np.random.default_rng(14)
    lens, H, hk, D = [300, 200], 4, 2, 128
    t, v, start = packed(rng, lens, H, hk, D)
    ref = orc.attention(*v, start, 1 / math.sqrt(D), window=window)
    t_out, t_lse = tolerance(ref, D, 300)
    t[1][140, 1, 3] = float("nan")
    t[1][420, 0, 90] = float("nan")
    t[0][17, 0, 0] = float("inf")
    t[0][499, 3, 127] = float("nan")
    out, lse, status = run_prompt(t, start, window=window)
    hit = np.zeros(lse.shape, bool)
    hit[140:min(300, 140 + window) if window else 300, 2:] = True
    hit[420:min(500, 420 + window) if window else 500, :2] = True
    hit[17, 0] = hit[499, 3] = True
    assert status == m.MOE_OK and np.isnan(out[hit]).all() and np.isnan(lse[hit]).all()
    assert (np.abs(out - ref[0]) <= t_out)[~hit].all() and (np.abs(lse - ref[1]) <= t_lse)[~hit].all()


def test_prompt_all_values_bad():
    rng = np.random.default_rng(15)
    t, v, start = packed(rng, [260, 100], 4, 1, 128)
    t[2][:260] = float("nan")
    out, lse, status = run_prompt(t, start)
    ref = orc.attention(*v, start, 1 / math.sqrt(128))
    assert np.isnan(out[:260]).all() and (np.abs(out - ref[0]) <= tolerance(ref, 128, 260)[0])[260:].all()


def test_prompt_far_scores():
    """Scores of hundreds, rising along the row: the maximum in use has to follow."""
    rng = np.random.default_rng(16)
    n, D = 700, 64
    t, v, start = packed(rng, [n], 2, 1, D)
    ramp = np.linspace(0.1, 30.0, n).astype(np.float32)
    for turn in (ramp, ramp[::-1].copy()):
        k = bf16(np.abs(v[1]) * turn[:, None, None]).to(DEV)
        q = bf16(np.abs(v[0])).to(DEV)
        out, lse, status = run_prompt((q, k, t[2]), start)
        ref = orc.attention(host(q), host(k), v[2], start, 1 / 8)
        t_out, t_lse = tolerance(ref, D, n)
        assert status == m.MOE_OK and (np.abs(out - ref[0]) <= t_out).all() and (np.abs(lse - ref[1]) <= t_lse).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,hk", [(7, 2), (1, 4), (16, 1)])
def test_prompt_rows_that_see_themselves(D, G, hk):
    """With a window of one token a row's result is its value, bit for bit; in most key tiles
    of an item some rows see nothing, so that the maximum in use is moved in the midst of it.
    Many times over: what one warp rescales while products run shows now and then only."""
    rng = np.random.default_rng(24)
    t, v, start = packed(rng, [1748, 1, 633, 300], G * hk, hk, D)
    want = t[2].repeat_interleave(G, 1)
    out, ws, s = torch.empty_like(want), workspace(), dev(start)
    for _ in range(400):
        out.zero_()
        m.prompt_attention(*t, s, out, ws, window=1)
        assert torch.equal(out, want)
    assert m.moe_device_status(ws) == m.MOE_OK


def test_prompt_strides_and_no_lse():
    """Queries, keys and values of matrices of their own, with gaps of their own; far rows."""
    rng = np.random.default_rng(17)
    t, v, start = packed(rng, [200], 6, 2, 64, poison=False)
    apart = [spaced(x.reshape(200, -1), e).unflatten(1, x.shape[1:]) for x, e in zip(t, (8, 24, 1000))]
    a, lse, _ = run_prompt(t, start)
    b, none, status = run_prompt(apart, start, lse=False)
    assert status == m.MOE_OK and none is None and np.array_equal(a, b)
    step = 11_000_000  # elements: the last row lies 2.2e9 from the first
    wide = torch.empty(199 * step + 128, dtype=torch.bfloat16, device=DEV)
    k = wide.as_strided((200, 2, 64), (step, 64, 1))
    k.copy_(t[1])
    c, _, _ = run_prompt((t[0], k, t[2]), start)
    d, _, _ = run_prompt((t[0], t[1], k), start)
    e, _, _ = run_prompt((t[0], t[1], t[1]), start)
    assert np.array_equal(a, c) and np.array_equal(d, e)
    f, _, _ = run_prompt((k, t[1], t[2]), start)
    g, _, _ = run_prompt((t[1], t[1], t[2]), start)
    assert np.array_equal(f, g)


@pytest.mark.parametrize("D,n,window", [(128, 70001, 0), (64, 150000, 40000)])
def test_prompt_of_a_long_document(D, n, window):
    """Some rows of it, among them the first and the last, in float64."""
    g = torch.Generator(device=DEV)
    g.manual_seed(23)
    qkv = torch.randn((n, 4, D), generator=g, device=DEV).to(torch.bfloat16)
    q, k, v = qkv[:, :2], qkv[:, 2:3], qkv[:, 3:]
    out, lse, ws = torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty((n, 2), device=DEV), workspace()
    m.prompt_attention(q, k, v, dev(np.array([0, n], np.int32)), out, ws, lse=lse, window=window)
    assert m.moe_device_status(ws) == m.MOE_OK
    for row in (0, 1, 127, 128, 40000, 40001, n // 2 + 77, n - 129, n - 1):
        first = max(0, row - window + 1) if window else 0
        K, V, Q = (x.double() for x in (k[first:row + 1, 0], v[first:row + 1, 0], q[row]))
        s = Q @ K.t() / math.sqrt(D)
        p = torch.softmax(s, dim=1)
        ref = [x.cpu().numpy() for x in (p @ V, torch.logsumexp(s, dim=1), p @ V.abs(), ((Q.abs() @ K.abs().t()) / math.sqrt(D)).amax(dim=1),
                                         s.abs().amax(dim=1))]
        t_out, t_lse = tolerance(ref, D, row + 1 - first)
        assert (np.abs(host(out[row]) - ref[0]) <= t_out).all() and (np.abs(host(lse[row]) - ref[1]) <= t_lse).all(), row


def test_prompt_is_the_same_each_time():
    rng = np.random.default_rng(18)
    t, v, start = packed(rng, rng.integers(1, 400, 20).tolist(), 14, 2, 128)
    first = run_prompt(t, start)
    ws = workspace()
    for _ in range(5):
        again = run_prompt(t, start, ws=ws)
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


@pytest.mark.parametrize("G", [3, 7, 100])
def test_what_was_there_before_does_not_matter(G):
    """Tiles of whole tokens leave rows over, which hold what an earlier call left there."""
    rng = np.random.default_rng(22)
    t, v, start = packed(rng, [700, 50], G, 1, 128)
    full, _, all_rows = packed(rng, [2048], 16, 16, 128)
    got = []
    for scale in (0.0, 1e4, float("nan")):
        run_prompt([full[0] * scale, full[1], full[2]], all_rows)
        got.append(run_prompt(t, start))
    for out, lse, _ in got[1:]:
        assert np.array_equal(out, got[0][0]) and np.array_equal(lse, got[0][1])


def test_prompts_alone_are_the_prompts_together():
    """A prompt's rows do not depend on what it is packed with."""
    rng = np.random.default_rng(19)
    lens = [130, 7, 260]
    t, v, start = packed(rng, lens, 7, 1, 64)
    out, lse, _ = run_prompt(t, start)
    for b, n in enumerate(lens):
        rows = slice(int(start[b]), int(start[b + 1]))
        alone = run_prompt([x[rows] for x in t], np.array([0, n], np.int32))
        assert np.array_equal(out[rows], alone[0]) and np.array_equal(lse[rows], alone[1])


def test_prompt_on_streams_and_in_graphs():
    """Two streams with a workspace each, and two graphs that share one, replayed in turn."""
    rng = np.random.default_rng(20)
    cases = []
    for lens, H, hk, D in (([300, 40], 14, 2, 128), ([700], 4, 4, 64)):
        t, v, start = packed(rng, lens, H, hk, D)
        want = run_prompt(t, start)[0]
        out = torch.zeros(t[0].shape, dtype=torch.bfloat16, device=DEV)
        cases.append((t, dev(start), out, want, torch.cuda.Stream(), workspace()))
    torch.cuda.synchronize()
    for _ in range(3):
        for t, start, out, want, stream, ws in cases:
            m.prompt_attention(*t, start, out, ws, stream=stream)
    torch.cuda.synchronize()
    for t, start, out, want, stream, ws in cases:
        assert np.array_equal(host(out), want)
        out.zero_()
    torch.cuda.synchronize()
    side, shared, graphs = torch.cuda.Stream(), workspace(), []
    for t, start, out, want, stream, ws in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
            m.prompt_attention(*t, start, out, shared)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for t, start, out, want, stream, ws in cases:
        assert np.array_equal(host(out), want)
    assert m.moe_device_status(shared) == m.MOE_OK


def test_prompt_empty():
    t, v, start = packed(np.random.default_rng(21), [4], 2, 1, 64)
    for s in ([4, 4], [0], [2, 2, 2]):
        out, lse, status = run_prompt(t, np.array(s, np.int32))
        assert status == m.MOE_OK and (out == 7).all()
    ws = workspace()
    z = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    m.prompt_attention(z, z, z, dev(np.array([0, 0], np.int32)), z, ws)
    assert m.moe_device_status(ws) == m.MOE_OK


# ---------------------------------------------------------------- together
def layers(rng, hidden, heads, hk, D, page, batch, width, total, **kw):
    w, s = weights(rng, (heads + 2 * hk) * D, hidden)
    o, os_ = weights(rng, hidden, heads * D)
    cache = m.Fp8KvCache(batch * width, hk, D, page)
    att = m.AttentionDecode(hidden, heads, hk, D, {"qkv": dev(w), "qkv_s": dev(s), "o": dev(o), "o_s": dev(os_)}, cache, total, **kw)
    return cache, att, m.AttentionPrompt(att, total), m.KvPages(cache, batch, width, total)


@pytest.mark.parametrize("D,kw", [(64, {}), (128, dict(window=40, softcap=50.0))])
def test_a_prompts_way(D, kw):
    """Pages, norm, sublayer and a decode step after it, against the calls one by one and
    against attention over the cache, which holds the same keys and values in FP8."""
    rng = np.random.default_rng(30)
    hidden, heads, hk, page, lens = 256, 6, 2, 16, [50, 1, 33]
    total = sum(lens)
    cache, att, prompt, pages = layers(rng, hidden, heads, hk, D, page, 3, 6, total, max_new=50, **kw)
    r = bf16(bf16_values(rng, (total, hidden))).to(DEV)
    gain = torch.ones(hidden, dtype=torch.bfloat16, device=DEV)
    codes, scales = torch.empty((total, hidden), dtype=torch.uint8, device=DEV), torch.empty((2, total + 3 & -4), device=DEV)
    ro, normed = torch.empty_like(r), torch.empty_like(r)
    m.rmsnorm_residual_fp8(r, gain, codes, scales, ro, 1e-6, out=normed)
    pages.extend(dev(np.array(lens, np.int32)))
    y = prompt((codes, scales), pages.page_table, pages.q_start, pages.lens, max(lens))
    # the same by single calls
    w = att.weights
    qkv = torch.empty((total, heads + 2 * hk, D), dtype=torch.bfloat16, device=DEV)
    ws = workspace(att.workspace.numel())
    m.fp8_block_gemm(codes, scales, w["qkv"], w["qkv_s"], qkv.flatten(1), ws)
    mixed = torch.empty((total, heads, D), dtype=torch.bfloat16, device=DEV)
    m.prompt_attention(qkv[:, :heads], qkv[:, heads:heads + hk], qkv[:, heads + hk:], pages.q_start, mixed, ws, **kw)
    want = torch.empty((total, hidden), dtype=torch.bfloat16, device=DEV)
    m.fp8_linear(mixed.flatten(1), w["o"], w["o_s"], want, ws)
    assert torch.equal(y, want)
    ref = orc.attention(*(host(x) for x in (qkv[:, :heads], qkv[:, heads:heads + hk], qkv[:, heads + hk:])), host(pages.q_start),
                        1 / math.sqrt(D), **kw)
    assert (np.abs(host(mixed) - ref[0]) <= tolerance(ref, D, 50, kw.get("softcap"))[0]).all()
    # bf16 input: the other projection, near the same
    z = prompt(normed, pages.page_table, pages.q_start, pages.lens, max(lens))
    assert ((z - y).float().norm() / y.float().norm()).item() < 0.1  # (two quantisations of 2^-4 a value)
    # a step of one token each: the lengths go on, and the cache holds the prompts
    before = pages.lens.clone()
    pages.extend(torch.ones(3, dtype=torch.int32, device=DEV))
    x = bf16(bf16_values(rng, (3, hidden))).to(DEV)
    out = att(x, pages.page_table, pages.q_start, pages.lens)
    assert bool(torch.isfinite(out).all()) and torch.equal(pages.lens, before + 1)
    assert host(pages.positions)[:4].tolist() == [50, 1, 33, -1]
    assert (att.status(), prompt.status(), m.moe_device_status(pages.workspace)) == (m.MOE_OK,) * 3


def test_attention_prompt_on_a_stream_and_in_a_graph():
    rng = np.random.default_rng(31)
    cache, att, prompt, pages = layers(rng, 128, 2, 1, 64, 16, 2, 4, 40)
    x = bf16(bf16_values(rng, (40, 128))).to(DEV)
    pages.extend(dev(np.array([30, 10], np.int32)))
    want = prompt(x, pages.page_table, pages.q_start, pages.lens, 30)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = prompt(x, pages.page_table, pages.q_start, pages.lens, 30, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out, g = torch.zeros_like(want), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        prompt(x, pages.page_table, pages.q_start, pages.lens, 30, out=out)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_prompt_block_example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "prompt_block.py")
    spec = importlib.util.spec_from_file_location("prompt_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    x = mod.main(["--prompts", "40", "1", "17", "--steps", "3"])
    assert bool(torch.isfinite(x).all())
