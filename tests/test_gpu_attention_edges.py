"""The attention sublayer's operators at the ends of their range on the GPU, against
the float64 oracle (oracle/attention_oracle.py)."""

import math

import numpy as np
import pytest
import torch

import moe_decode_layer_bf16_gb300 as m
from tests.fixtures_attention import BF16, F16, F32, Batch, bf16, bf16_values, orc, weights
from tests.test_gpu_attention import assert_cache, dev, f64, run_attention, workspace

pytestmark = pytest.mark.gpu
DEV = "cuda"


def largest_value(b):
    """Of the batch's V, NaN aside."""
    v = orc.e4m3_decode(b.cache["v"]) * b.cache["v_scale"].astype(np.float64)[:, :, None, None]
    return float(np.nanmax(np.abs(v), initial=0.0))


def tolerance(ref, D, count, vmax, score=0.0):
    """(for out, for lse) of ref = oracle's (out, lse, mag, unit).

    A score: q's f16 values are within 2^-39 of the row's largest (times sum |k|), the
    products are exact, each of the D / 16 steps of 16 products takes two fp32 roundings of
    sum |q k|, and the scales, the bias, the change to base 2, the cap's products and the
    difference from the maximum 16 more; `score` is what the caller adds (the tanh).  A
    weight: its score's error and the sum's, the exponential's 2^-22 twice, one rounding to
    f16, and the floor of f16's subnormals, 2^-25 in units of 2^-15 of the largest weight.
    Sums over the tokens and the pieces: an fp32 rounding for each group of 16 tokens, and
    at most 300 pieces.  Then the output's rounding (2^-134: half a subnormal step)."""
    out, lse, mag, unit = ref
    e = 2.0 ** -39 * unit[..., 1] + (D / 8 + 16) * F32 * unit[..., 0] + score
    sums = (count / 16 + 300) * F32
    t = (2 * e + 2.0 ** -21 + F16 + sums)[..., None] * mag + count * 2.0 ** -40 * vmax
    t = t + BF16 * (np.abs(out) + t) + 2.0 ** -134
    return t, e + 2.0 ** -21 + sums + 4 * F32 * np.abs(np.where(np.isfinite(lse), lse, 0.0))


def check(b, q, got, lse, sm, score=0.0, rows=None, **kw):
    """The oracle's values; where it has no number, neither has the kernel."""
    ref = orc.attention(q, b.cache, b.table, b.q_start, b.lens, sm, **kw)
    t_out, t_lse = tolerance(ref, b.D, int(max(b.lens.max(), 1)), largest_value(b), score)
    rows = slice(None) if rows is None else rows
    nan = np.isnan(ref[0])[rows]
    assert np.array_equal(np.isnan(got[rows]), nan)
    off = np.abs(got - ref[0])[rows]
    assert ((off <= t_out[rows]) | nan).all(), float(np.nanmax(off - t_out[rows]))
    if lse is not None:
        same = (lse == ref[1]) | (np.isnan(lse) & np.isnan(ref[1]))  # (both -inf)
        with np.errstate(invalid="ignore"):
            assert (same | (np.abs(lse - ref[1]) <= t_lse))[rows].all()


# ---------------------------------------------------------------- blocks of zeros
TINY = np.float32(2.0 ** -126)  # the scale that the append gives a block of zeros


@pytest.mark.parametrize("D,hk,G,page", [(64, 2, 2, 16), (128, 1, 4, 64), (128, 2, 12, 32), (64, 1, 9, 128)])
def test_values_of_zeros_give_zeros(D, hk, G, page):
    """All V zero, written by the append: out is zero exactly, lse as ever."""
    rng = np.random.default_rng(50)
    lens = [5, 40, 300, 1, 2000]
    b = Batch(rng, lens, lens, hk, D, page)
    t = b.tensors(DEV)
    ws = workspace()
    k = bf16_values(rng, (b.total, hk, D))
    m.kv_cache_append(bf16(k).to(DEV), torch.zeros((b.total, hk, D), dtype=torch.bfloat16, device=DEV), t["k"], t["v"],
                      t["k_scale"], t["v_scale"], t["table"], t["q_start"], t["lens"], 2000, ws)
    b.cache = {n: t[n].cpu().numpy() for n in b.cache}
    assert (b.cache["v_scale"][b.table[b.table >= 0]] == TINY).all()
    b.q_start, b.total, b.news = np.arange(6, dtype=np.int32), 5, [1] * 5
    t["q_start"] = dev(b.q_start)
    q = bf16_values(rng, (5, hk * G, D))
    got, lse, status = run_attention(b, q, hk * G, tensors=t)
    assert status == m.MOE_OK
    assert (got == 0).all()
    check(b, q, got, lse, 1 / math.sqrt(D))


@pytest.mark.parametrize("where", ["first", "last", "every other", "middle", "all but one", "a warp's start"])
@pytest.mark.parametrize("D,hk,G,page", [(64, 2, 2, 16), (128, 1, 7, 64), (128, 2, 12, 32)])
def test_blocks_of_zeros_among_others(where, D, hk, G, page):
    rng = np.random.default_rng(51)
    b = Batch(rng, [9000, 700, 64, 90], [1, 2, 1, 1], hk, D, page)
    for s in range(4):
        n = -(-int(b.lens[s]) // page)
        at = {"first": [0], "last": [n - 1], "every other": range(0, n, 2), "middle": range(n // 3, n // 2 + 1),
              "all but one": [i for i in range(n) if i != n // 2], "a warp's start": range(0, n, 5)}[where]
        for i in at:
            b.cache["v"][b.table[s, i]] &= 0x80  # zeros of either sign
            b.cache["v_scale"][b.table[s, i]] = TINY
    q = bf16_values(rng, (b.total, hk * G, D))
    got, lse, status = run_attention(b, q, hk * G)
    assert status == m.MOE_OK
    check(b, q, got, lse, 1 / math.sqrt(D))


@pytest.mark.parametrize("D,hk,G,page", [(64, 2, 2, 16), (128, 1, 7, 64), (128, 2, 12, 32)])
@pytest.mark.parametrize("spread", [0, 8, 20])
def test_values_of_the_smallest_scales(D, hk, G, page, spread):
    """V scales from 2^-126 up: small, but values like any others."""
    rng = np.random.default_rng(52)
    b = Batch(rng, [3000, 33, 150], [1, 2, 1], hk, D, page)
    shape = b.cache["v_scale"].shape
    b.cache["v_scale"] = np.where(np.isnan(b.cache["v_scale"]), np.nan,
                                  np.exp2(-126 + np.round(rng.uniform(0, spread, shape)))).astype(np.float32)
    q = bf16_values(rng, (b.total, hk * G, D))
    got, lse, status = run_attention(b, q, hk * G)
    assert status == m.MOE_OK
    check(b, q, got, lse, 1 / math.sqrt(D))


# ---------------------------------------------------------------- row numbers of every size
def wild_rows(b):
    """Sequences 1 to 3 of five get rows that are none: their ends are the largest and the
    smallest int32, whose differences wrap to small numbers."""
    b.q_start = np.array([0, 5, 2 ** 31 - 1, -2 ** 31, 5, 6], np.int32)
    b.total = 6
    return b


def test_append_row_numbers_whose_difference_wraps():
    rng = np.random.default_rng(60)
    b = wild_rows(Batch(rng, [70, 40, 33, 20, 9], [5, 1, 1, 1, 1], 2, 64, 32))
    k, v = (bf16_values(rng, (6, 2, 64)) for _ in range(2))
    want = {n: a.copy() for n, a in b.cache.items()}
    orc.append(k, v, want, b.table, [0, 5, 5, 5, 5, 6], b.lens)
    t = b.tensors(DEV)
    ws = workspace(m.kv_cache_workspace_size())
    m.kv_cache_append(bf16(k).to(DEV), bf16(v).to(DEV), t["k"], t["v"], t["k_scale"], t["v_scale"], t["table"],
                      t["q_start"], t["lens"], 5, ws)
    assert m.moe_device_status(ws) == m.MOE_ERR_INVALID_ARG
    assert_cache(t, want)


def test_attention_row_numbers_whose_difference_wraps():
    rng = np.random.default_rng(61)
    b = wild_rows(Batch(rng, [70, 40, 33, 20, 9], [5, 1, 1, 1, 1], 2, 64, 32))
    q = bf16_values(rng, (6, 4, 64))
    got, lse, status = run_attention(b, q, 4)
    assert status == m.MOE_ERR_INVALID_ARG
    b.q_start = np.array([0, 5, 5, 5, 5, 6], np.int32)
    check(b, q, got, lse, 0.125)


# ---------------------------------------------------------------- streams
@pytest.mark.parametrize("handle", [False, True])
def test_attention_decode_on_a_side_stream_with_rotated_keys(handle):
    """The side stream is busy as the step is called: what of it ran elsewhere would read
    and write the projection before it is there."""
    rng = np.random.default_rng(62)
    hidden, heads, hk, D, page = 384, 6, 2, 64, 16
    (qkv, qkv_s), (o, o_s) = weights(rng, (heads + 2 * hk) * D, hidden), weights(rng, hidden, heads * D)
    wt = {"qkv": dev(qkv), "qkv_s": dev(qkv_s), "o": dev(o), "o_s": dev(o_s)}
    side, at = torch.cuda.Stream(), []

    def rotate(q, k):
        at.append(torch.cuda.current_stream().cuda_stream)
        q.mul_(-2)
        k.mul_(0.5)

    table = dev(np.array([[3, 1], [0, 7]], np.int32))
    start, lens = dev(np.array([0, 3, 5], np.int32)), dev(np.array([3, 2], np.int32))
    xs = [bf16(bf16_values(rng, (5, hidden))).to(DEV) for _ in range(4)]
    both, busy = [], torch.randn((8192, 8192), device=DEV, dtype=torch.bfloat16)
    for stream in (None, side):
        att = m.AttentionDecode(hidden, heads, hk, D, wt, m.Fp8KvCache(8, hk, D, page), max_tokens=6, max_new=3,
                                rotate=rotate)
        ys = []
        torch.cuda.synchronize()
        for x in xs:
            if stream is not None:
                with torch.cuda.stream(stream):
                    torch.mm(busy, busy)
            ys.append(att(x, table, start, lens, stream=stream.cuda_stream if stream and handle else stream))
        torch.cuda.synchronize()
        assert att.status() == m.MOE_OK
        both.append(ys)
    assert at == [torch.cuda.current_stream().cuda_stream] * 4 + [side.cuda_stream] * 4
    for a, b in zip(*both):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- windows
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 3, 2 ** 30, 2 ** 30 - 1])
def test_windows_beyond_every_length(window):
    """No window at all, also for a sequence with more new rows than tokens."""
    rng = np.random.default_rng(53)
    b = Batch(rng, [1, 300, 40, 2], [4, 2, 40, 5], 2, 64, 16)
    q = bf16_values(rng, (b.total, 4, 64))
    got, lse, status = run_attention(b, q, 4, window=window)
    assert status == m.MOE_OK
    check(b, q, got, lse, 0.125)


# ---------------------------------------------------------------- work beyond 2^31 units
def test_more_work_than_a_31_bit_count():
    """A long chunk behind a long context: 32768 tiles of 32 tokens, 8192 groups of 16
    rows, 8 heads.  The table names 64 pages over and over, so a few rows are checked
    against a direct softmax over the pages with their multiplicities."""
    hk, G, D, page, pages, n, new = 8, 16, 64, 128, 64, 1 << 20, 8192
    heads = hk * G
    assert (n // 32 + 2) * (new * G // 16) * hk > 2 ** 31 - 1
    g = torch.Generator(device=DEV)
    g.manual_seed(58)
    cache = [torch.randn((pages, hk, page, D), generator=g, device=DEV).to(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.exp2(torch.randint(-2, 3, (pages, hk), generator=g, device=DEV).float()) for _ in range(2)]
    table = torch.arange(n // page, device=DEV, dtype=torch.int32).remainder(pages)[None].contiguous()
    q = torch.randn((new, heads, D), generator=g, device=DEV).to(torch.bfloat16)
    out = torch.full((new, heads, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full((new, heads), float("nan"), device=DEV)
    ws = workspace(m.decode_attention_workspace_size(heads, hk, D, new))
    m.decode_attention(q, *cache, *scales, table, dev(np.array([0, new], np.int32)), dev(np.array([n], np.int32)), new,
                       out, ws, lse=lse)
    assert m.moe_device_status(ws) == m.MOE_OK
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    assert int(ws[4:1024].sum()) == 0
    for i, h in ((0, 0), (1, 127), (4095, 16), (4096, 64), (8000, 77), (8191, 127), (8191, 0)):
        kv = h // G
        k, v = ((c[:, kv].float() * s[:, kv, None, None]).double().reshape(-1, D) for c, s in zip(cache, scales))
        seen = n - new + i + 1
        times = torch.full((pages * page,), seen // (pages * page), device=DEV, dtype=torch.float64)
        times[:seen % (pages * page)] += 1
        s = k @ q[i, h].double() / math.sqrt(D)
        p = torch.exp(s - s.max()) * times
        want, mag = p @ v / p.sum(), p @ v.abs() / p.sum()
        ref = [x.cpu().numpy() for x in (want, s.max() + p.sum().log(), mag,
                                         torch.stack([(k.abs() @ q[i, h].double().abs()).max(),
                                                      q[i, h].abs().max().double() * k.abs().sum(1).max()]) / math.sqrt(D))]
        t_out, t_lse = tolerance(ref, D, n, float(v.abs().max()))
        assert (np.abs(f64(out[i, h]) - ref[0]) <= t_out).all(), (i, h)
        assert abs(float(lse[i, h]) - float(ref[1])) <= t_lse, (i, h)


def test_rows_that_too_many_sequences_count_as_theirs():
    """Numbers of rows that no batch can have are reported, and nothing is written."""
    total, hk, D = 1 << 20, 8, 64
    cache = m.Fp8KvCache(4, hk, D, 16)
    start = dev(np.array([0, total] * 3000 + [0], np.int32))
    lens = torch.zeros(6000, dtype=torch.int32, device=DEV)
    table = torch.zeros((6000, 1), dtype=torch.int32, device=DEV)
    q = torch.zeros((total, hk, D), dtype=torch.bfloat16, device=DEV)
    out = torch.full_like(q, 3.0)
    ws = workspace(m.decode_attention_workspace_size(hk, hk, D, 1 << 20))
    m.decode_attention(q, cache.k, cache.v, cache.k_scale, cache.v_scale, table, start, lens, 1 << 20, out, ws)
    assert m.moe_device_status(ws) == m.MOE_ERR_INVALID_ARG
    assert bool((out == 3.0).all()) and int(ws[4:1024].sum()) == 0


# ---------------------------------------------------------------- NaN behind a mask
@pytest.mark.parametrize("window", [0, 6, 40, 2000])
@pytest.mark.parametrize("lens,news", [([7, 64, 500, 130, 33], [7, 4, 5, 40, 33]), ([9000, 2500, 40], [5, 3, 2])])
@pytest.mark.parametrize("D,hk,G,page", [(64, 2, 2, 16), (128, 1, 2, 64), (128, 2, 6, 32), (64, 1, 5, 128)])
def test_nan_values_reach_only_the_rows_that_see_them(window, lens, news, D, hk, G, page):
    """A NaN in a token's V or K reaches the rows that see the token, and no other: not
    those before it, nor those whose window has passed it."""
    rng = np.random.default_rng(54)
    b = Batch(rng, lens, news, hk, D, page)
    for s, (n, new) in enumerate(zip(lens, news)):
        edges = rng.integers(max(0, n - new - 8), n, 4).tolist()
        if 0 < window < n - new:
            edges += rng.integers(n - new - window, n - window + 4, 3).tolist()
        for i, pos in enumerate(edges):
            b.cache["v"][b.table[s, pos // page], i % hk, pos % page, rng.integers(0, D, 3)] = (0x7F, 0xFF, 0x7F)
        pos = n - 2
        b.cache["k"][b.table[s, pos // page], 0, pos % page, 5] = 0x7F
    q = bf16_values(rng, (b.total, hk * G, D))
    ref = orc.attention(q, b.cache, b.table, b.q_start, b.lens, 1 / math.sqrt(D), window=window)[0]
    assert np.isnan(ref).any() and np.isfinite(ref).any()
    ws = workspace(m.decode_attention_workspace_size(hk * G, hk, D, b.max_new))
    got, lse, status = run_attention(b, q, hk * G, ws=ws, window=window)
    assert status == m.MOE_OK
    check(b, q, got, lse, 1 / math.sqrt(D), window=window)
    again = run_attention(b, q, hk * G, ws=ws, window=window)[0]
    assert np.array_equal(got, again, equal_nan=True)


# ---------------------------------------------------------------- caps
@pytest.mark.parametrize("cap", [1e-40, 1e-3, 0.5, 255.0, 257.0, 4096.0, 1e6, 1e20, 3e38])
@pytest.mark.parametrize("D,hk,G", [(64, 2, 2), (128, 1, 12)])
def test_caps_of_every_size(cap, D, hk, G):
    """A cap far above the scores changes nothing, one far below flattens them."""
    rng = np.random.default_rng(55)
    b = Batch(rng, [300, 40, 7], [1, 2, 3], hk, D, 32)
    q = bf16_values(rng, (b.total, hk * G, D), 4.0)
    q[2] = 0.0  # scores of zero
    sm = 1 / math.sqrt(D)
    cap = float(np.float32(cap))
    got, lse, status = run_attention(b, q, hk * G, softcap=cap)
    assert status == m.MOE_OK
    # the tanh is off by 2^-22 of the cap, and above 256 by at most 2^-20 of the score
    unit = orc.attention(q, b.cache, b.table, b.q_start, b.lens, sm, cap)[3][..., 0]
    check(b, q, got, lse, sm, score=2.0 ** -22 * cap if cap <= 256 else 2.0 ** -20 * unit, softcap=cap)


# ---------------------------------------------------------------- batches without tokens
def test_batches_without_sequences_or_tokens():
    hk, D, page = 2, 64, 16
    cache = m.Fp8KvCache(3, hk, D, page)
    c = (cache.k, cache.v, cache.k_scale, cache.v_scale)
    ws = workspace(1 << 20)

    def ints(*a):
        return torch.tensor(a, dtype=torch.int32, device=DEV)

    for B, width in ((0, 4), (0, 0), (2, 4)):
        table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
        start, lens = ints(*[0] * (B + 1)), ints(*[0] * B)
        kv = torch.empty((0, hk, D), dtype=torch.bfloat16, device=DEV)
        m.kv_cache_append(kv, kv, *c, table, start, lens, 1, ws)
        q = torch.empty((0, 4, D), dtype=torch.bfloat16, device=DEV)
        m.decode_attention(q, *c, table, start, lens, 1, torch.empty_like(q), ws,
                           lse=torch.empty((0, 4), device=DEV))
    assert m.moe_device_status(ws) == m.MOE_OK


def test_attention_decode_of_no_tokens():
    rng = np.random.default_rng(59)
    hidden, heads, hk, D, page = 256, 4, 2, 64, 16
    (qkv, qkv_s), (o, o_s) = weights(rng, (heads + 2 * hk) * D, hidden), weights(rng, hidden, heads * D)
    att = m.AttentionDecode(hidden, heads, hk, D, {"qkv": dev(qkv), "qkv_s": dev(qkv_s), "o": dev(o), "o_s": dev(o_s)},
                            m.Fp8KvCache(4, hk, D, page), max_tokens=2)
    table = dev(np.array([[0, 1], [2, 3]], np.int32))
    x = torch.empty((0, hidden), dtype=torch.bfloat16, device=DEV)
    y = att(x, table, dev(np.array([0, 0, 0], np.int32)), dev(np.array([3, 0], np.int32)))
    assert tuple(y.shape) == (0, hidden) and att.status() == m.MOE_OK


# ---------------------------------------------------------------- prompts
@pytest.mark.parametrize("kw", [dict(), dict(window=1), dict(window=50), dict(softcap=20.0, slopes=True, window=97)])
@pytest.mark.parametrize("lens,news", [([300], [300]), ([500, 90, 40], [129, 64, 40]), ([1300], [47])])
@pytest.mark.parametrize("D,hk,G,page", [(64, 2, 1, 16), (128, 1, 3, 64), (64, 1, 5, 128), (128, 2, 8, 32)])
def test_a_prompts_chunk(kw, lens, news, D, hk, G, page):
    """Many new tokens of a sequence: many groups of rows, with the diagonal across their tiles."""
    rng = np.random.default_rng(56)
    b = Batch(rng, lens, news, hk, D, page)
    kw = dict(kw)
    if kw.get("slopes"):
        kw["slopes"] = np.exp2(-8.0 * np.arange(1, hk * G + 1) / (hk * G)).astype(np.float32)
    q = bf16_values(rng, (b.total, hk * G, D))
    sm = 1 / math.sqrt(D)
    got, lse, status = run_attention(b, q, hk * G, **kw)
    assert status == m.MOE_OK
    check(b, q, got, lse, sm, score=2.0 ** -22 * kw.get("softcap", 0.0), **kw)


def test_a_prompt_in_chunks_is_the_prompt_at_once():
    rng = np.random.default_rng(57)
    hk, G, D, page, n = 2, 4, 128, 64, 700
    b = Batch(rng, [n], [n], hk, D, page)
    q = bf16_values(rng, (n, hk * G, D))
    whole, lse, _ = run_attention(b, q, hk * G)
    vmax, t = largest_value(b), b.tensors(DEV)
    done, got, got_lse = 0, [], []
    for step in (1, 130, 64, 255, 250):
        part = Batch.__new__(Batch)
        part.__dict__ = dict(b.__dict__, total=step, news=[step], lens=np.array([done + step], np.int32),
                             q_start=np.array([0, step], np.int32))
        o, l, status = run_attention(part, q[done:done + step], hk * G,
                                     tensors={**t, "lens": dev(part.lens), "q_start": dev(part.q_start)})
        assert status == m.MOE_OK
        got.append(o)
        got_lse.append(l)
        done += step
    ref = orc.attention(q, b.cache, b.table, b.q_start, b.lens, 1 / math.sqrt(D))
    t_out, t_lse = tolerance(ref, D, n, vmax)
    for o, l in ((whole, lse), (np.concatenate(got), np.concatenate(got_lse))):
        assert (np.abs(o - ref[0]) <= t_out).all() and (np.abs(l - ref[1]) <= t_lse).all()
