"""CPU oracle of the attention sublayer's operators (test infrastructure only):
the FP8 block-scaled linear layer, the FP8 paged cache's writer and attention
over the cache, from their definitions in include/moe_decode.h, in float64.

Where a definition rounds (scales and quotients to float32, codes to E4M3), so
does the oracle; everything else is float64.  Loops over sequences, blocks and
heads: small cases only.
"""

from __future__ import annotations

import numpy as np

from . import moe_oracle
from .moe_oracle import e4m3_decode, pow2_round_up

BLOCK = 128
QMAX = np.float32(448.0)
TINY_SCALE = np.float32(2.0 ** -126)


def e4m3_encode(v) -> np.ndarray:
    """E4M3 codes of float32 values; a NaN becomes the code 0x7f."""
    v = np.asarray(v, np.float32)
    nan = np.isnan(v)
    return np.where(nan, np.uint8(0x7F), moe_oracle.e4m3_encode(np.where(nan, np.float32(0), v)))


def quant_rows(x: np.ndarray, e8m0: bool):
    """(codes uint8 [M, K], scales float32 [ceil(K / 128), M]) of bf16 values x."""
    x = np.asarray(x, np.float32)
    M, K = x.shape
    codes = np.zeros((M, K), np.uint8)
    scales = np.zeros((-(-K // BLOCK), M), np.float32)
    for b, k0 in enumerate(range(0, K, BLOCK)):
        g = x[:, k0:k0 + BLOCK]
        amax = np.abs(g).max(axis=1)
        with np.errstate(invalid="ignore"):
            s = (amax / QMAX).astype(np.float32)
        if e8m0:
            s = pow2_round_up(np.maximum(s, TINY_SCALE))
        s = np.where(amax == 0, np.float32(1), s).astype(np.float32)
        with np.errstate(invalid="ignore", over="ignore"):
            codes[:, k0:k0 + BLOCK] = e4m3_encode((g / s[:, None]).astype(np.float32))
        scales[b] = s
    return codes, scales


def block_gemm(codes, scales, w, w_s):
    """(out, sum of the terms' magnitudes), both float64 [M, N]."""
    M, K = codes.shape
    N = w.shape[0]
    a, b = e4m3_decode(codes), e4m3_decode(w)
    out, mag = np.zeros((M, N)), np.zeros((M, N))
    rows = np.arange(N) // BLOCK
    for kb, k0 in enumerate(range(0, K, BLOCK)):
        ab, bb = a[:, k0:k0 + BLOCK], b[:, k0:k0 + BLOCK]
        s = np.outer(scales[kb, :M].astype(np.float64), w_s[rows, kb].astype(np.float64))
        out += (ab @ bb.T) * s
        mag += (np.abs(ab) @ np.abs(bb).T) * s
    return out, mag


def block_scale(amax: np.ndarray) -> np.ndarray:
    """Scale of a cache block: the power of two at or above amax / 448, at least 2^-126."""
    return pow2_round_up(np.maximum((np.asarray(amax, np.float32) / QMAX).astype(np.float32), TINY_SCALE))


def append(k, v, cache, page_table, q_start, lens):
    """Writes the new tokens into `cache` (dict of numpy arrays k, v, k_scale,
    v_scale) in place."""
    page = cache["k"].shape[2]
    for b, n_all in enumerate(lens):
        start, n = int(q_start[b]), int(q_start[b + 1] - q_start[b])
        if n == 0:
            continue
        for blk in range((n_all - n) // page, (n_all - 1) // page + 1):
            lo, hi = max(blk * page, n_all - n), min((blk + 1) * page, n_all)
            held, pg = lo - blk * page, int(page_table[b, blk])
            for name, x in (("k", k), ("v", v)):
                codes, scale = cache[name][pg], cache[name + "_scale"][pg]  # [heads, page, dim], [heads]
                new = np.asarray(x[start + lo - (n_all - n):start + hi - (n_all - n)], np.float32).transpose(1, 0, 2)
                fin = np.where(np.isfinite(new), np.abs(new), 0.0)
                s = block_scale(fin.max(axis=(1, 2)))
                if held:
                    s = np.maximum(s, scale).astype(np.float32)
                    old = e4m3_decode(codes[:, :held]) * (scale.astype(np.float64) / s)[:, None, None]
                    keep = (s == scale)[:, None, None]
                    codes[:, :held] = np.where(keep, codes[:, :held], e4m3_encode(old.astype(np.float32)))
                with np.errstate(invalid="ignore", over="ignore"):
                    codes[:, held:held + hi - lo] = e4m3_encode((new / s[:, None, None]).astype(np.float32))
                scale[:] = s


def attention(q, cache, page_table, q_start, lens, sm_scale, softcap=0.0, window=0, slopes=None):
    """(out, lse, magnitude sum_j p_j |v_j|, largest score error unit) in float64.

    The last is, for each row, |sm_scale| times the max over its tokens of sum_d |q_d k_d|
    and of max|q| sum_d |k_d|: what the roundings of a score are relative to."""
    total, H, D = q.shape
    hk, page = cache["k"].shape[1], cache["k"].shape[2]
    G = H // hk
    out, lse = np.zeros((total, H, D)), np.full((total, H), -np.inf)
    mag, unit = np.zeros((total, H, D)), np.zeros((total, H, 2))
    q = np.asarray(q, np.float64)
    for b, n_all in enumerate(lens):
        start, n = int(q_start[b]), int(q_start[b + 1] - q_start[b])
        for i in range(n):
            pos = int(n_all) - n + i
            first = max(0, pos - window + 1) if window > 0 else 0
            at = np.arange(first, min(pos, int(n_all) - 1) + 1)
            if at.size == 0:
                continue
            pg = page_table[b, at // page]
            for h in range(H):
                kv = h // G
                kk = e4m3_decode(cache["k"][pg, kv, at % page]) * cache["k_scale"][pg, kv].astype(np.float64)[:, None]
                vv = e4m3_decode(cache["v"][pg, kv, at % page]) * cache["v_scale"][pg, kv].astype(np.float64)[:, None]
                row = q[start + i, h]
                s = sm_scale * (kk @ row)
                unit[start + i, h] = abs(sm_scale) * np.array([(np.abs(kk) @ np.abs(row)).max(),
                                                          np.abs(row).max() * np.abs(kk).sum(axis=1).max()])
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                if slopes is not None:
                    s = s + float(slopes[h]) * (at - pos)
                m = s.max()
                p = np.exp(s - m)
                L = p.sum()
                out[start + i, h] = (p / L) @ vv
                mag[start + i, h] = (p / L) @ np.abs(vv)
                lse[start + i, h] = m + np.log(L)
    return out, lse, mag, unit
