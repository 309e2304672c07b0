"""Test-side inputs of the attention sublayer's operators, as numpy arrays and
their torch copies, and the tolerances of their outputs.

Tolerances count roundings: half a step is eps / 2 relative (bf16 2^-8, f16
2^-11, fp32 2^-24).
"""

from __future__ import annotations

import numpy as np
import torch

from oracle import attention_oracle as orc
from oracle.moe_oracle import e4m3_decode

BF16, F16, F32 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24


def bf16(a) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def bf16_values(rng, shape, scale=1.0) -> np.ndarray:
    """Normal values that are exact in bf16 (float32 array)."""
    return bf16(rng.standard_normal(shape).astype(np.float32) * scale).float().numpy()


def weights(rng, N, K, e8m0=False):
    """E4M3 codes of every finite value and block scales."""
    w = rng.integers(0, 256, (N, K), dtype=np.uint8)
    w[(w & 0x7F) == 0x7F] ^= 1
    s = np.exp2(rng.uniform(-12, -8, (-(-N // 128), -(-K // 128)))).astype(np.float32)
    if e8m0:
        s = np.exp2(np.round(np.log2(s))).astype(np.float32)
    return w, s


def linear_tolerance(out, mag, K, f32):
    """Every product of two codes is exact.  Each of the K additions, and the
    product of the two scales with a block's sum (three roundings), is off by at
    most half an fp32 step of the sum of magnitudes; then the output's rounding."""
    tol = (K + 3) * F32 * mag
    return tol + (F32 if f32 else BF16) * (np.abs(out) + tol)


class Batch:
    """Sequences of given lengths (new tokens included) in a paged cache whose
    other contents are poison: NaN codes in every slot that no sequence holds,
    NaN scales for unused pages."""

    def __init__(self, rng, lens, news, hk, D, page, poison=True, spread=4.0):
        self.lens = np.array(lens, np.int32)
        self.news = list(news)
        self.hk, self.D, self.page = hk, D, page
        self.q_start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.total = int(self.q_start[-1])
        pages_of = [-(-n // page) for n in lens]
        self.width = max(1, max(pages_of))
        self.pages = sum(pages_of) + 3
        order = rng.permutation(self.pages)
        self.table = np.full((len(lens), self.width), -1, np.int32)
        at = 0
        for b, n in enumerate(pages_of):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (self.pages, hk, page, D)
        self.cache = {}
        for name in ("k", "v"):
            codes = rng.integers(0, 256, shape, dtype=np.uint8)
            codes[(codes & 0x7F) == 0x7F] ^= 1
            # unit-sized values with a loudness of their own for each block
            scale = np.exp2(np.round(rng.uniform(-8 - spread / 2, -8 + spread / 2, shape[:2]))).astype(np.float32)
            if poison:
                held = np.zeros((self.pages, page), bool)
                for b, n in enumerate(lens):
                    for i in range(n):
                        held[self.table[b, i // page], i % page] = True
                codes.transpose(0, 2, 1, 3)[~held] = 0x7F
                scale[~held.any(axis=1)] = np.nan
            self.cache[name], self.cache[name + "_scale"] = codes, scale

    def tensors(self, device):
        t = {k: torch.from_numpy(v.copy()).to(device) for k, v in self.cache.items()}
        t["table"] = torch.from_numpy(self.table).to(device)
        t["lens"] = torch.from_numpy(self.lens).to(device)
        t["q_start"] = torch.from_numpy(self.q_start).to(device)
        return t

    @property
    def max_new(self):
        return max(1, max(self.news))


def attention_tolerance(out, lse, mag, unit, D, count):
    """(for out, for lse).

    A score: the split of q is off by at most 2^-21 of the row's largest value
    (times sum |k|); the products are exact, their D / 32 * 2 sums of 32 and the
    joining and scaling of the two parts are at most D / 16 + 6 fp32 roundings of
    sum |q k|; the bias, the cap and the change to base 2 are 6 more of the
    score's own size, which sum |q k| bounds.  A weight: twice the score's error
    (its own and the sum's), the exponential's 2^-22, one rounding to f16, and its
    floor: weights below 2^-29 of the largest lose bits, at most 2^-39 each.  Sums over
    the tokens and the pieces: an fp32 rounding for each 16-token group (and at
    most 300 pieces).  The tanh: 2^-22 of the cap, which `unit` does not bound, so
    callers add it."""
    e = 2.0 ** -21 * unit[..., 1] + (D / 16 + 12) * F32 * unit[..., 0]
    sums = (count / 16 + 300) * F32
    w = 2 * e + 2.0 ** -21 + F16 + sums
    t_out = w[..., None] * mag + count * 2.0 ** -39 * np.abs(mag).max(initial=0.0)
    t_out = t_out + BF16 * (np.abs(out) + t_out)
    t_lse = e + 2.0 ** -21 + sums + 4 * F32 * np.abs(np.where(np.isfinite(lse), lse, 0.0))
    return t_out, t_lse


__all__ = ["Batch", "attention_tolerance", "bf16", "bf16_values", "e4m3_decode", "linear_tolerance", "orc", "weights"]
