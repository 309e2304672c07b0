"""The attention sublayer's operators on the GPU against the float64 oracle
(oracle/attention_oracle.py): codes, scales and cache contents exactly, sums
within tolerances that count their roundings (tests/fixtures_attention.py)."""

import math

import numpy as np
import pytest
import torch

import moe_decode_layer_bf16_gb300 as m
from tests.fixtures_attention import Batch, attention_tolerance, bf16, bf16_values, linear_tolerance, orc, weights

pytestmark = pytest.mark.gpu
DEV = "cuda"


def workspace(nbytes=64 << 20):
    return torch.zeros(nbytes, dtype=torch.uint8, device=DEV)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64) if t.dtype == torch.bfloat16 else t.detach().cpu().numpy()


def strided(x: torch.Tensor, extra: int) -> torch.Tensor:
    """x (on the GPU) as rows of a wider matrix whose other columns are NaN."""
    wide = torch.full((x.shape[0], x.shape[1] + extra), float("nan"), dtype=x.dtype, device=DEV)
    wide[:, 8:8 + x.shape[1]] = x.to(DEV)
    return wide[:, 8:8 + x.shape[1]]


# ---------------------------------------------------------------- append (bad values first: they must not fault)
def make_append(rng, lens, news, hk, D, page, **kw):
    """Sequences whose new tokens are still to be written."""
    b = Batch(rng, lens, news, hk, D, page, **kw)
    k = bf16_values(rng, (b.total, hk, D), 2.0)
    v = bf16_values(rng, (b.total, hk, D), 0.5)
    loud = np.exp2(np.round(rng.uniform(-3, 5, (b.total, 1, 1)))).astype(np.float32)
    return b, k * loud, v * loud


def run_append(b, k, v, stride_extra=0, ws=None, max_new=None):
    t = b.tensors(DEV)
    ws = workspace(m.kv_cache_workspace_size()) if ws is None else ws
    row = b.hk * b.D
    kk, vv = (strided(bf16(a.reshape(b.total, row)), stride_extra).unflatten(1, (b.hk, b.D)) if stride_extra
              else bf16(a).to(DEV) for a in (k, v))
    m.kv_cache_append(kk, vv, t["k"], t["v"], t["k_scale"], t["v_scale"], t["table"], t["q_start"], t["lens"],
                      b.max_new if max_new is None else max_new, ws)
    status = m.moe_device_status(ws)
    return t, status


def assert_cache(t, want):
    for name in ("k", "v"):
        got, ref = t[name].cpu().numpy(), want[name]
        nan = ((got & 0x7F) == 0x7F) & ((ref & 0x7F) == 0x7F)
        zero = ((got & 0x7F) == 0) & ((ref & 0x7F) == 0)  # (either sign)
        bad = (got != ref) & ~nan & ~zero
        assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[:4])
        assert np.array_equal(t[name + "_scale"].cpu().numpy(), want[name + "_scale"], equal_nan=True), name


@pytest.mark.parametrize("what", ["page", "page_negative", "length", "length_negative", "start", "shorter"])
def test_append_bad_batches_are_reported_and_left_out(what):
    rng = np.random.default_rng(5)
    b, k, v = make_append(rng, [70, 40, 33], [5, 20, 1], 2, 64, 32)
    want = {n: a.copy() for n, a in b.cache.items()}
    ok = Batch.__new__(Batch)
    ok.__dict__ = dict(b.__dict__)
    lens, start = b.lens.copy(), b.q_start.copy()
    if what == "page":
        b.table[1, 1] = b.pages
    elif what == "page_negative":
        b.table[1, 1] = -7
    elif what == "length":
        b.lens = np.array([70, b.width * 32 + 1, 33], np.int32)
    elif what == "length_negative":
        b.lens = np.array([70, -3, 33], np.int32)
    elif what == "start":
        b.q_start = np.array([0, 5, 1 << 20, 26], np.int32)
    elif what == "shorter":
        b.lens = np.array([70, 19, 33], np.int32)  # fewer tokens than new ones
    t, status = run_append(b, k, v)
    assert status == m.MOE_ERR_INVALID_ARG
    # the first sequence is written as ever; the second is not (but for its good block)
    n_ok = [0, 5, 5, 5]
    orc.append(k, v, want, b.table, n_ok, lens)
    if what.startswith("page"):  # its tokens 20 .. 31 lie in block 0, which is in range
        first = dict(want)
        orc.append(k, v, first, b.table, [5, 5, 17, 17], np.array([0, 32, 0]))
    if what != "start":
        orc.append(k, v, want, b.table, [25, 25, 25, 26], lens)
    assert_cache(t, want)
    assert start[-1] == b.total


CASES = [
    ([1], [1], 1, 64, 16), ([17], [1], 2, 64, 16), ([16], [1], 2, 128, 16), ([64, 65, 63], [1, 1, 1], 3, 128, 64),
    ([100, 0, 7, 250], [100, 0, 7, 13], 2, 128, 64), ([129, 128, 127], [3, 128, 126], 1, 128, 128),
    ([33, 300], [2, 257], 2, 64, 32), ([128, 140], [128, 70], 1, 64, 128), ([5, 1000], [5, 700], 8, 128, 32),
]


@pytest.mark.parametrize("lens,news,hk,D,page", CASES)
@pytest.mark.parametrize("extra", [0, 24])
def test_append(lens, news, hk, D, page, extra):
    rng = np.random.default_rng(len(lens) * 1000 + D + page)
    b, k, v = make_append(rng, lens, news, hk, D, page)
    want = {n: a.copy() for n, a in b.cache.items()}
    orc.append(k, v, want, b.table, b.q_start, b.lens)
    t, status = run_append(b, k, v, extra)
    assert status == m.MOE_OK
    assert_cache(t, want)


def test_append_token_by_token_grows_the_scale():
    rng = np.random.default_rng(3)
    b, k, v = make_append(rng, [40, 40], [40, 40], 2, 128, 16)
    cache = {n: a.copy() for n, a in b.cache.items()}
    t = b.tensors(DEV)
    ws = workspace(m.kv_cache_workspace_size())
    for i in range(40):
        kk, vv = (np.stack([a[i], a[40 + i]]) for a in (k, v))
        lens, start = np.array([i + 1, i + 1], np.int32), np.array([0, 1, 2], np.int32)
        orc.append(kk, vv, cache, b.table, start, lens)
        m.kv_cache_append(bf16(kk).to(DEV), bf16(vv).to(DEV), t["k"], t["v"], t["k_scale"], t["v_scale"], t["table"],
                          dev(start), dev(lens), 1, ws)
    assert m.moe_device_status(ws) == m.MOE_OK
    assert_cache(t, cache)


def test_append_zeros_tiny_huge_and_non_finite_values():
    rng = np.random.default_rng(4)
    b, k, v = make_append(rng, [3, 20, 18, 16, 16], [3, 20, 1, 16, 16], 2, 64, 16)
    k[0:3] = 0.0                         # a block of zeros: the smallest scale
    v[0:3] = 2.0 ** -130                 # subnormal in float32
    k[3:23] *= 2.0 ** 100
    v[5, 0, 3], v[6, 1, 7], v[7, 0, 1] = np.inf, -np.inf, np.nan
    k[24:40] = 0.0
    k[30, :, 0] = 448.0 * 2.0 ** -9      # amax / 448 a power of two exactly
    k[40:56] = np.nan
    want = {n: a.copy() for n, a in b.cache.items()}
    orc.append(k, v, want, b.table, b.q_start, b.lens)
    t, status = run_append(b, k, v)
    assert status == m.MOE_OK
    assert_cache(t, want)


def test_append_into_a_cache_whose_scales_are_no_powers_of_two():
    rng = np.random.default_rng(6)
    b, k, v = make_append(rng, [20, 9], [3, 4], 2, 64, 32)
    for n in ("k_scale", "v_scale"):
        b.cache[n] = (b.cache[n] * np.float32(1.37) * np.float32(64)).astype(np.float32)  # large: they stay
    want = {n: a.copy() for n, a in b.cache.items()}
    orc.append(k, v, want, b.table, b.q_start, b.lens)
    t, status = run_append(b, k, v)
    assert status == m.MOE_OK
    assert_cache(t, want)


# ---------------------------------------------------------------- attention
def run_attention(b, q, heads, ws=None, q_tensor=None, lse=True, stream=None, tensors=None, **kw):
    t = b.tensors(DEV) if tensors is None else tensors
    ws = workspace(m.decode_attention_workspace_size(heads, b.hk, b.D, b.max_new)) if ws is None else ws
    qt = bf16(q).to(DEV) if q_tensor is None else q_tensor
    out = torch.full((b.total, heads, b.D), float("nan"), dtype=torch.bfloat16, device=DEV)
    ls = torch.full((b.total, heads), float("nan"), dtype=torch.float32, device=DEV) if lse else None
    if kw.get("slopes") is not None:
        kw["slopes"] = dev(kw["slopes"])
    m.decode_attention(qt, t["k"], t["v"], t["k_scale"], t["v_scale"], t["table"], t["q_start"], t["lens"], b.max_new,
                       out, ws, lse=ls, stream=stream, **kw)
    status = m.moe_device_status(ws)
    assert int(ws[4:1024].sum()) == 0  # the counters are left at zero
    return f64(out), None if ls is None else f64(ls), status


def assert_attention(b, q, heads, got, got_lse, sm_scale, softcap=0.0, window=0, slopes=None, rows=None):
    out, lse, mag, unit = orc.attention(q, b.cache, b.table, b.q_start, b.lens, sm_scale, softcap, window, slopes)
    t_out, t_lse = attention_tolerance(out, lse, mag, unit, b.D, int(max(b.lens.max(), 1)))
    cap = 2.0 ** -22 * softcap  # the tanh's own error, in every score
    t_out = t_out + 2 * cap * mag[..., :]
    rows = slice(None) if rows is None else rows
    empty = np.isneginf(lse)
    with np.errstate(invalid="ignore"):
        assert (np.abs(got - out) <= t_out)[rows].all(), float(np.nanmax((np.abs(got - out) - t_out)[rows]))
        if got_lse is not None:
            assert np.array_equal(np.isneginf(got_lse)[rows], empty[rows])
            ok = (np.abs(got_lse - lse) <= t_lse + cap) | empty
            assert ok[rows].all()


@pytest.mark.parametrize("what", ["page", "page_negative", "length", "length_negative", "start", "descending"])
def test_attention_bad_batches_are_reported(what):
    rng = np.random.default_rng(15)
    b = Batch(rng, [70, 140, 33], [1, 2, 1], 2, 64, 32)
    q = bf16_values(rng, (b.total, 4, 64))
    t = b.tensors(DEV)
    if what == "page":
        t["table"][1, 2] = b.pages
    elif what == "page_negative":
        t["table"][1, 2] = -1
    elif what == "length":
        t["lens"][1] = b.width * 32 + 1
    elif what == "length_negative":
        t["lens"][1] = -1
    elif what == "start":
        t["q_start"][2] = 1 << 28
    elif what == "descending":
        t["q_start"][1] = 100
    got, lse, status = run_attention(b, q, 4, tensors=t)
    assert status == m.MOE_ERR_INVALID_ARG
    if what not in ("start", "descending"):  # the other sequences are not touched by it
        assert_attention(b, q, 4, got, lse, 0.125, rows=[0, 3])
    if what.startswith("page"):  # the page's 32 tokens are masked
        ref = Batch.__new__(Batch)
        ref.__dict__ = dict(b.__dict__)
        ref.cache = {n: a.copy() for n, a in b.cache.items()}
        pg = b.table[1, 2]
        keep = [i for i in range(140) if not 64 <= i < 96]
        for h in range(4):
            for i in range(2):
                at = np.array([j for j in keep if j <= 138 + i])
                kk = orc.e4m3_decode(b.cache["k"][b.table[1, at // 32], h // 2, at % 32]) * b.cache["k_scale"][b.table[1, at // 32], h // 2][:, None]
                vv = orc.e4m3_decode(b.cache["v"][b.table[1, at // 32], h // 2, at % 32]) * b.cache["v_scale"][b.table[1, at // 32], h // 2][:, None]
                s = 0.125 * (kk @ q[1 + i, h].astype(np.float64))
                p = np.exp(s - s.max())
                want, size = p @ vv / p.sum(), p @ np.abs(vv) / p.sum()
                assert (np.abs(got[1 + i, h] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * size).all()
        assert pg >= 0


LENS = {
    "one token": ([1], [1]),
    "around a tile": ([31, 32, 33, 63, 64, 65], [1] * 6),
    "empty slots": ([0, 40, 0, 0], [1, 1, 1, 1]),
    "no rows": ([50, 20, 90], [1, 0, 2]),
    "several new": ([4, 130, 9, 300], [4, 3, 9, 5]),
    "more new than tokens": ([2, 60], [4, 1]),
    "long": ([5000], [1]),
    "uneven": ([1, 2500, 17, 700, 3, 129], [1, 2, 1, 1, 3, 1]),
}


@pytest.mark.parametrize("lens", LENS.values(), ids=LENS.keys())
@pytest.mark.parametrize("hk,G,D,page", [(1, 1, 64, 16), (2, 7, 128, 64), (1, 8, 128, 32), (3, 5, 64, 128), (2, 2, 128, 16),
                                         (1, 16, 64, 64), (1, 12, 128, 128)])
def test_attention(lens, hk, G, D, page):
    rng = np.random.default_rng(hk * 100 + G * 10 + page)
    b = Batch(rng, lens[0], lens[1], hk, D, page)
    heads = hk * G
    q = bf16_values(rng, (b.total, heads, D), 1.5)
    sm = 1 / math.sqrt(D)
    got, lse, status = run_attention(b, q, heads)
    assert status == m.MOE_OK
    assert_attention(b, q, heads, got, lse, sm)


@pytest.mark.parametrize("kw", [dict(window=1), dict(window=33), dict(window=100), dict(softcap=5.0), dict(slopes=True),
                                dict(window=70, softcap=20.0, slopes=True), dict(sm_scale=-0.3), dict(sm_scale=0.0)])
@pytest.mark.parametrize("hk,G,D,page,news", [(2, 4, 128, 64, 1), (1, 3, 64, 16, 4), (1, 12, 128, 32, 2)])
def test_attention_masks_caps_and_biases(kw, hk, G, D, page, news):
    rng = np.random.default_rng(21)
    b = Batch(rng, [5, 400, 64, 1, 0, 129], [min(news, 5), news, news, 1, 1, news], hk, D, page)
    heads = hk * G
    q = bf16_values(rng, (b.total, heads, D), 2.0)
    kw = dict(kw)
    if kw.get("slopes"):
        kw["slopes"] = np.exp2(-8.0 * np.arange(1, heads + 1) / heads).astype(np.float32)
    sm = kw.pop("sm_scale", 1 / math.sqrt(D))
    got, lse, status = run_attention(b, q, heads, sm_scale=sm, **kw)
    assert status == m.MOE_OK
    assert_attention(b, q, heads, got, lse, sm, **kw)


def test_attention_below_the_window_pages_may_be_gone():
    rng = np.random.default_rng(22)
    b = Batch(rng, [300, 170], [2, 1], 2, 64, 16)
    q = bf16_values(rng, (b.total, 4, 64))
    out, lse, mag, unit = orc.attention(q, b.cache, b.table, b.q_start, b.lens, 0.125, window=40)
    t = b.tensors(DEV)
    t["table"][0, :16] = -1    # tokens 0 .. 255; the rows see 259 .. 299
    t["table"][1, :8] = 1 << 30
    got, got_lse, status = run_attention(b, q, 4, tensors=t, window=40)
    assert status == m.MOE_OK
    t_out, t_lse = attention_tolerance(out, lse, mag, unit, 64, 300)
    assert (np.abs(got - out) <= t_out).all() and (np.abs(got_lse - lse) <= t_lse).all()


def test_attention_extreme_scales_and_scores():
    rng = np.random.default_rng(23)
    b = Batch(rng, [200, 90], [1, 2], 2, 128, 32, spread=0.0)
    b.cache["v_scale"] *= np.exp2(np.round(rng.uniform(-12, 12, b.cache["v_scale"].shape))).astype(np.float32)
    q = bf16_values(rng, (b.total, 8, 128), 30.0)  # one token takes nearly all the weight
    q[1] = 0.0                                      # a row of zeros: every token alike
    q[2] *= 2.0 ** -60
    got, lse, status = run_attention(b, q, 8)
    assert status == m.MOE_OK
    assert_attention(b, q, 8, got, lse, 1 / math.sqrt(128))


def test_attention_non_finite_rows_stay_alone():
    rng = np.random.default_rng(24)
    b = Batch(rng, [100, 60], [3, 1], 1, 128, 64)
    q = bf16_values(rng, (b.total, 4, 128))
    q[1, 2, 5], q[3, 0, 7] = np.inf, np.nan
    got, lse, status = run_attention(b, q, 4)
    assert status == m.MOE_OK
    assert np.isnan(got[1, 2]).all() and np.isnan(got[3, 0]).all() and np.isnan(lse[1, 2]) and np.isnan(lse[3, 0])
    q[1, 2, 5], q[3, 0, 7] = 0, 0
    out, ref, mag, unit = orc.attention(q, b.cache, b.table, b.q_start, b.lens, 1 / math.sqrt(128))
    t_out, t_lse = attention_tolerance(out, ref, mag, unit, 128, 100)
    fine = np.ones((b.total, 4), bool)
    fine[1, 2] = fine[3, 0] = False
    assert (np.abs(got - out) <= t_out)[fine].all() and (np.abs(lse - ref) <= t_lse)[fine].all()


def test_attention_many_sequences():
    # more sequences than threads add up, most of them short, some without rows
    rng = np.random.default_rng(25)
    n = 700
    lens = rng.integers(0, 40, n).tolist()
    lens[13], lens[600] = 900, 333
    news = rng.integers(0, 3, n).tolist()
    b = Batch(rng, lens, news, 1, 64, 16)
    q = bf16_values(rng, (b.total, 2, 64))
    got, lse, status = run_attention(b, q, 2)
    assert status == m.MOE_OK
    assert_attention(b, q, 2, got, lse, 0.125)


def test_attention_strided_queries_no_lse_and_repeats():
    rng = np.random.default_rng(26)
    b = Batch(rng, [3000, 500, 64], [2, 1, 4], 2, 128, 64)
    q = bf16_values(rng, (b.total, 14, 128))
    qt = strided(bf16(q.reshape(b.total, -1)), 512).unflatten(1, (14, 128))
    assert not qt.is_contiguous()
    ws = workspace(m.decode_attention_workspace_size(14, 2, 128, 4))
    first = run_attention(b, q, 14, ws=ws, q_tensor=qt)
    assert_attention(b, q, 14, first[0], first[1], 1 / math.sqrt(128))
    for _ in range(5):  # the same bits every time, with and without lse
        again = run_attention(b, q, 14, ws=ws, lse=False)
        assert np.array_equal(first[0], again[0])


def test_cache_beyond_four_gigabytes():
    # page numbers whose byte offsets pass 32 bits
    pages, hk, page, D = 36000, 8, 128, 128
    rng = np.random.default_rng(27)
    kc, vc = (torch.full((pages, hk, page, D), 0x7F, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.full((pages, hk), float("nan"), device=DEV) for _ in range(2))
    assert kc.numel() > 1 << 32
    lens, table = [200, 130], np.array([[pages - 1, 33000], [35999 - 40, 34567]], np.int32)
    new = np.array([0, 200, 330], np.int32)
    k, v = bf16_values(rng, (330, hk, D)), bf16_values(rng, (330, hk, D))
    ws = workspace(8 << 20)
    tt, st, ln = dev(table), dev(new), dev(np.array(lens, np.int32))
    m.kv_cache_append(bf16(k).to(DEV), bf16(v).to(DEV), kc, vc, ks, vs, tt, st, ln, 200, ws)
    small = {n: np.zeros((4, hk, page, D), np.uint8) for n in ("k", "v")}
    small |= {n + "_scale": np.zeros((4, hk), np.float32) for n in ("k", "v")}
    orc.append(k, v, small, np.array([[0, 1], [2, 3]]), new, lens)
    ids = torch.from_numpy(table.reshape(-1).astype(np.int64)).to(DEV)
    for n, codes, scale in (("k", kc, ks), ("v", vc, vs)):
        assert np.array_equal(scale[ids].cpu().numpy(), small[n + "_scale"])
        got = codes[ids].cpu().numpy()
        for i, (b, blk) in enumerate([(0, 0), (0, 1), (1, 0), (1, 1)]):
            held = min(lens[b] - blk * page, page)
            assert ((got[i, :, :held] == small[n][i, :, :held]) | ((got[i, :, :held] & 0x7F) == 0)).all()
    q = bf16_values(rng, (2, 8, D))
    out = torch.empty((2, 8, D), dtype=torch.bfloat16, device=DEV)
    m.decode_attention(bf16(q).to(DEV), kc, vc, ks, vs, tt, dev(np.array([0, 1, 2], np.int32)), ln, 1, out, ws)
    assert m.moe_device_status(ws) == m.MOE_OK
    ref, lse, mag, unit = orc.attention(q, small, np.array([[0, 1], [2, 3]]), [0, 1, 2], lens, 1 / math.sqrt(D))
    t_out, _ = attention_tolerance(ref, lse, mag, unit, D, 200)
    assert (np.abs(f64(out) - ref) <= t_out).all()


# ---------------------------------------------------------------- linear
@pytest.mark.parametrize("M,K", [(1, 16), (3, 128), (5, 144), (37, 1552), (130, 7168), (300, 272)])
@pytest.mark.parametrize("e8m0", [False, True])
@pytest.mark.parametrize("extra", [0, 40])
def test_quant_rows_exact(M, K, e8m0, extra):
    rng = np.random.default_rng(M + K)
    x = bf16_values(rng, (M, K)) * np.exp2(np.round(rng.uniform(-20, 20, (M, 1)))).astype(np.float32)
    x[0, : K // 2] = 0.0
    x[-1] = 0.0
    if M > 2:
        x[1] = np.float32(2.0 ** -120) * np.round(x[1] * 4)  # scales whose reciprocals are no normal numbers
        x[2] *= np.float32(2.0 ** 100)
    t = strided(bf16(x), extra) if extra else bf16(x).to(DEV)
    codes = torch.full((M, K), 0x7F, dtype=torch.uint8, device=DEV)
    scales = torch.full((-(-K // 128), (M + 3) // 4 * 4), float("nan"), device=DEV)
    m.fp8_quant_rows(t, codes, scales, e8m0=e8m0)
    ref_c, ref_s = orc.quant_rows(f64(bf16(x)), e8m0)
    got = codes.cpu().numpy()
    assert np.array_equal(scales[:, :M].cpu().numpy(), ref_s)
    assert ((got == ref_c) | (((got | ref_c) & 0x7F) == 0)).all()


def test_quant_rows_every_pair_of_significands():
    # x and amax are bf16: all 128 x 128 pairs, x over 12 binades below amax
    sig = (1 + np.arange(128) / 128).astype(np.float32)
    rows = []
    for e in range(12):
        r = np.zeros((128, 256), np.float32)
        r[:, :128] = sig[None, :] * np.float32(2.0 ** -e)
        r[:, 127] = np.where(sig * 2 > r[:, :127].max(axis=1), sig * 2, 4 * sig)  # the row's amax: each significand once
        r[:, 128:] = r[:, :128]
        rows.append(r)
    x = np.concatenate(rows)
    codes = torch.empty(x.shape, dtype=torch.uint8, device=DEV)
    scales = torch.empty((2, x.shape[0]), device=DEV)
    m.fp8_quant_rows(bf16(x).to(DEV), codes, scales)
    ref_c, ref_s = orc.quant_rows(x, False)
    assert np.array_equal(scales.cpu().numpy(), ref_s) and np.array_equal(codes.cpu().numpy(), ref_c)


SHAPES = [(1, 1, 16), (1, 9216 // 8, 7168), (2, 129, 272), (7, 128, 128), (8, 1000, 528), (9, 257, 4096), (16, 640, 144),
          (17, 300, 1552), (32, 130, 48), (33, 1001, 1552), (64, 128, 2048), (65, 96, 784), (128, 15, 7168), (129, 512, 256),
          (130, 257, 1040), (256, 1000, 2064), (300, 8, 512), (513, 2049, 272), (1000, 136, 144)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("e8m0,f32", [(False, False), (False, True), (True, True)])
def test_linear(M, N, K, e8m0, f32):
    rng = np.random.default_rng(M * 7 + N + K)
    x = bf16_values(rng, (M, K)) * np.where(rng.random(K) > 0.98, 20, 1).astype(np.float32)
    x[M // 2] = 0.0
    w, s = weights(rng, N, K, e8m0)
    out = torch.full((M, N), float("nan"), dtype=torch.float32 if f32 else torch.bfloat16, device=DEV)
    ws = workspace(m.fp8_linear_workspace_size(M, N, K))
    t = strided(bf16(x), 16) if N % 2 else bf16(x).to(DEV)
    m.fp8_linear(t, dev(w), dev(s), out, ws, e8m0=e8m0)
    assert m.moe_device_status(ws) == m.MOE_OK and int(ws[4:1024].sum()) == 0
    codes, scales = orc.quant_rows(f64(bf16(x)), e8m0)
    ref, mag = orc.block_gemm(codes, scales, w, s)
    err, tol = np.abs(f64(out) - ref), linear_tolerance(ref, mag, K, f32)
    assert (err <= tol).all(), float((err - tol).max())


# whole waves of tiles with a remainder, and tiles cut along K, in both arrangements
@pytest.mark.parametrize("M,N,K", [(3, 19500, 1040), (20, 19457, 528), (12, 700, 3600), (150, 301, 6016), (260, 70, 5136),
                                   (2000, 2500, 4112)])
@pytest.mark.parametrize("f32", [False, True])
def test_linear_waves_and_pieces(M, N, K, f32):
    test_linear(M, N, K, False, f32)


@pytest.mark.parametrize("M,N,K", [(1, 1152, 7168), (13, 260, 1040), (40, 1001, 1552), (200, 700, 2064)])
def test_linear_is_its_two_parts_and_repeats(M, N, K):
    rng = np.random.default_rng(M)
    x, (w, s) = bf16(bf16_values(rng, (M, K))).to(DEV), weights(rng, N, K)
    w, s = dev(w), dev(s)
    ws = workspace()
    codes = torch.empty((M, K), dtype=torch.uint8, device=DEV)
    scales = torch.empty((-(-K // 128), (M + 3) // 4 * 4), device=DEV)
    a, b, c = (torch.empty((M, N), dtype=torch.float32, device=DEV) for _ in range(3))
    m.fp8_quant_rows(x, codes, scales)
    m.fp8_block_gemm(codes, scales, w, s, a, ws)
    m.fp8_linear(x, w, s, b, ws)
    assert torch.equal(a, b)
    for _ in range(5):
        m.fp8_linear(x, w, s, c.zero_(), ws)
        assert torch.equal(a, c)
    # codes and scales of a float8 tensor's own type are taken as well
    m.fp8_block_gemm(codes.view(torch.float8_e4m3fn), scales, w.view(torch.float8_e4m3fn), s, c.zero_(), ws)
    assert torch.equal(a, c)


@pytest.mark.parametrize("M", [4, 40, 150])
def test_linear_non_finite_rows_stay_alone(M):
    rng = np.random.default_rng(M)
    N, K = 200, 512
    x = bf16_values(rng, (M, K))
    w, s = weights(rng, N, K)
    ref, mag = orc.block_gemm(*orc.quant_rows(x, False), w, s)
    x[1, 5], x[M - 1, 300] = np.inf, np.nan
    out = torch.empty((M, N), dtype=torch.float32, device=DEV)
    ws = workspace(m.fp8_linear_workspace_size(M, N, K))
    m.fp8_linear(bf16(x).to(DEV), dev(w), dev(s), out, ws)
    got = f64(out)
    assert not np.isfinite(got[1]).any() and np.isnan(got[M - 1]).all()
    rest = [i for i in range(M) if i not in (1, M - 1)]
    assert (np.abs(got - ref) <= linear_tolerance(ref, mag, K, True))[rest].all()


# ---------------------------------------------------------------- together
def test_streams_graph_and_one_workspace():
    """The three operators on a side stream with one workspace, then captured and
    replayed on new inputs."""
    rng = np.random.default_rng(31)
    hk, G, D, page, hidden = 2, 3, 64, 16, 256
    heads = hk * G
    rows = (heads + 2 * hk) * D
    w, s = weights(rng, rows, hidden)
    b = Batch(rng, [33, 70, 1, 0], [1, 1, 1, 1], hk, D, page)
    x = bf16_values(rng, (b.total, hidden))
    t = b.tensors(DEV)
    ws = workspace()
    wt, st = dev(w), dev(s)
    xt = bf16(x).to(DEV)
    qkv = torch.empty((b.total, rows), dtype=torch.bfloat16, device=DEV)
    out = torch.empty((b.total, heads, D), dtype=torch.bfloat16, device=DEV)
    t["lens"][3] = 1  # (the batch's last slot: one token, written by this step)
    free = sorted(set(range(b.pages)) - set(b.table[b.table >= 0].tolist()))  # (no page is written by two sequences)
    t["table"][3, 0] = free.pop()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step(stream=None):
        m.fp8_linear(xt, wt, st, qkv, ws, stream=stream)
        v = qkv.unflatten(1, (heads + 2 * hk, D))
        m.kv_cache_append(v[:, heads:heads + hk], v[:, heads + hk:], t["k"], t["v"], t["k_scale"], t["v_scale"], t["table"],
                          t["q_start"], t["lens"], 1, ws, stream=stream)
        m.decode_attention(v[:, :heads], t["k"], t["v"], t["k_scale"], t["v_scale"], t["table"], t["q_start"], t["lens"],
                           1, out, ws, stream=stream)

    def want(x):
        cache = {n: t[n].cpu().numpy() for n in ("k", "v", "k_scale", "v_scale")}
        ref = f64(qkv).reshape(b.total, heads + 2 * hk, D)
        lin, mag = orc.block_gemm(*orc.quant_rows(x, False), w, s)
        assert (np.abs(f64(qkv) - lin) <= linear_tolerance(lin, mag, hidden, False)).all()
        lens, table = t["lens"].cpu().numpy(), t["table"].cpu().numpy()
        for n, lo in (("k", heads), ("v", heads + hk)):  # the newest token of each sequence is what was written
            for i, L in enumerate(lens):
                pg, at = table[i, (L - 1) // page], (L - 1) % page
                got = orc.e4m3_decode(cache[n][pg, :, at]) * cache[n + "_scale"][pg][:, None]
                x_ = ref[i, lo:lo + hk]
                assert (np.abs(got - x_) <= np.maximum(np.abs(x_) * 2.0 ** -4, cache[n + "_scale"][pg][:, None] * 2.0 ** -10)).all()
        o, lse, mg, unit = orc.attention(ref[:, :heads], cache, table, b.q_start, lens, 1 / math.sqrt(D))
        assert (np.abs(f64(out) - o) <= attention_tolerance(o, lse, mg, unit, D, 70)[0]).all()

    step(side)
    side.synchronize()
    want(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step()
    for seed in (1, 2):
        x2 = bf16_values(np.random.default_rng(seed), (b.total, hidden))
        xt.copy_(bf16(x2))
        t["lens"] += 1  # the next token of every sequence: read by the graph as it stands
        for i, L in enumerate(t["lens"].tolist()):
            if (L - 1) % page == 0 and t["table"][i, (L - 1) // page] < 0:
                t["table"][i, (L - 1) // page] = free.pop()
        graph.replay()
        torch.cuda.synchronize()
        want(x2)
    assert m.moe_device_status(ws) == m.MOE_OK


@pytest.mark.parametrize("D,G", [(128, 4), (64, 12)])
def test_lengths_written_by_the_kernel_before(D, G):
    """The attention starts while the kernel before it runs and may look at the lengths
    early; what counts is what that kernel leaves there.  Here it is a quantisation
    whose last row of codes is the lengths, other ones each time."""
    rng = np.random.default_rng(43)
    hk, page, rows = 2, 32, 20000
    both = np.array([[300, 5, 832], [64, 777, 3]], np.int32)
    b = Batch(rng, [832, 832, 832], [1, 1, 1], hk, D, page)
    t = b.tensors(DEV)
    q = bf16(bf16_values(rng, (3, hk * G, D))).to(DEV)
    ws = workspace()
    x = []
    for lens in both:
        last = np.zeros(16, np.uint8)
        last[:12] = np.frombuffer(lens.tobytes(), np.uint8)
        last[15] = 0x7E  # 448: the scale is 1, and the codes are the values' own
        v = np.zeros((rows, 16))
        v[-1] = orc.e4m3_decode(last)
        x.append(bf16(v).to(DEV))
    codes = torch.zeros((rows, 16), dtype=torch.uint8, device=DEV)
    scales = torch.empty((1, (rows + 3) // 4 * 4), dtype=torch.float32, device=DEV)
    lens = codes[-1].view(torch.int32)[:3]

    def attend(lens, out):
        m.decode_attention(q, t["k"], t["v"], t["k_scale"], t["v_scale"], t["table"], t["q_start"], lens, 1, out, ws)

    want = [torch.empty_like(q) for _ in both]
    for n, o in zip(both, want):
        attend(torch.from_numpy(n).to(DEV), o)
    got = [torch.empty_like(q) for _ in range(40)]
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        m.fp8_quant_rows(x[i % 2], codes, scales)
        attend(lens, o)
    torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])
    for i, o in enumerate(got):
        assert torch.equal(o, want[i % 2]), i
    assert m.moe_device_status(ws) == m.MOE_OK


def test_attention_decode_is_its_parts():
    rng = np.random.default_rng(41)
    hidden, heads, hk, D, page = 384, 6, 2, 64, 16
    rows = (heads + 2 * hk) * D
    (qkv, qkv_s), (o, o_s) = weights(rng, rows, hidden), weights(rng, hidden, heads * D)
    wt = {"qkv": dev(qkv), "qkv_s": dev(qkv_s), "o": dev(o), "o_s": dev(o_s)}
    cache = m.Fp8KvCache(8, hk, D, page)
    turned = []
    att = m.AttentionDecode(hidden, heads, hk, D, wt, cache, max_tokens=6, max_new=3, window=20,
                            rotate=lambda q, k: turned.append((q.mul_(-1).shape, k.shape)))
    table = dev(np.array([[3, 1], [0, 7]], np.int32))
    x = bf16(bf16_values(rng, (5, hidden))).to(DEV)
    start, lens = dev(np.array([0, 3, 5], np.int32)), dev(np.array([3, 2], np.int32))
    y = att(x, table, start, lens)
    assert att.status() == m.MOE_OK and turned == [((5, heads, D), (5, hk, D))]
    # the same with the functions, from the cache that the step left
    ws = workspace()
    p = torch.empty((5, rows), dtype=torch.bfloat16, device=DEV)
    m.fp8_linear(x, wt["qkv"], wt["qkv_s"], p, ws)
    q = -p.view(5, -1, D)[:, :heads]
    mixed, want = torch.empty_like(q), torch.empty_like(y)
    m.decode_attention(q, cache.k, cache.v, cache.k_scale, cache.v_scale, table, start, lens, 3, mixed, ws, window=20)
    m.fp8_linear(mixed.view(5, -1), wt["o"], wt["o_s"], want, ws)
    assert torch.equal(y, want)
    with pytest.raises(ValueError, match="at most 6"):
        att(x.repeat(2, 1), table, start, lens)


def test_decode_block_example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_block.py")
    spec = importlib.util.spec_from_file_location("decode_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    y = mod.main(["--steps", "3", "--batch", "3", "--prompt", "5"])
    assert torch.isfinite(y.float()).all()
