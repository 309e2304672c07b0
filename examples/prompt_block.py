"""Prompts through one decoder block, then a token at a time: pages of the cache given on the
GPU, the residual norm with FP8 output, the attention sublayer over whole prompts, then
decode steps of the same sequences captured in a CUDA graph, and the pages taken back.

    python examples/prompt_block.py
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import moe_decode_layer_bf16_gb300 as moe  # noqa: E402
from decode_block import attention_weights  # noqa: E402
from moe_decode_layer_bf16_gb300 import synth  # noqa: E402


class Boundary:
    """residual += x; its norm as FP8 rows for up to max_tokens tokens."""

    def __init__(self, hidden, max_tokens, eps=1e-6):
        self.gain, self.eps = torch.ones(hidden, dtype=torch.bfloat16, device="cuda"), eps
        self.codes = torch.empty((max_tokens, hidden), dtype=torch.uint8, device="cuda")
        self.scales = torch.empty(-(-hidden // 128) * (max_tokens + 3 & -4), dtype=torch.float32, device="cuda")

    def __call__(self, residual, x=None):
        n, hidden = residual.shape
        codes, groups, n4 = self.codes[:n], -(-hidden // 128), n + 3 & -4
        scales = self.scales[:groups * n4].view(groups, n4)
        moe.rmsnorm_residual_fp8(residual, self.gain, codes, scales, residual, self.eps, x=x)
        return codes, scales


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--prompts", type=int, nargs="+", default=[70, 5, 129, 1])
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args(argv)
    hidden, heads, kv_heads, dim, page = 512, 8, 2, 64, 16
    torch.manual_seed(0)
    batch, total, longest = len(a.prompts), sum(a.prompts), max(a.prompts)
    width = -(-(longest + a.steps + 2) // page)
    cache = moe.Fp8KvCache(batch * width, kv_heads, dim, page)
    pages = moe.KvPages(cache, batch, width, max_rows=total)
    decode = moe.AttentionDecode(hidden, heads, kv_heads, dim, attention_weights(hidden, heads, kv_heads, dim), cache, batch)
    prompt = moe.AttentionPrompt(decode, total)
    boundary = Boundary(hidden, total)

    _, residual = synth.make_tokens(total, hidden, device="cuda")
    pages.extend(torch.tensor(a.prompts, dtype=torch.int32, device="cuda"))
    y = prompt(boundary(residual), pages.page_table, pages.q_start, pages.lens, longest)

    # the last token of each prompt goes on
    last = pages.q_start[1:].long() - 1
    x, residual = y[last].contiguous(), residual[last].contiguous()
    one = torch.ones(batch, dtype=torch.int32, device="cuda")
    normed = torch.empty_like(x)

    def step():
        pages.extend(one)
        moe.rmsnorm_residual(residual, boundary.gain, normed, residual, boundary.eps, x=x)
        decode(normed, pages.page_table, pages.q_start, pages.lens, out=x)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(a.steps):
        graph.replay()
    lens = pages.lens.tolist()
    pages.release(pages.lens > 0)
    status = (decode.status(), prompt.status(), pages.status())
    assert status == (moe.MOE_OK,) * 3, status
    assert lens == [n + a.steps + 1 for n in a.prompts], lens
    print(f"prompts of {a.prompts} tokens and {a.steps + 1} steps: {lens} tokens; {int(pages.free[0])} pages free again; "
          f"|x| {x.float().abs().mean().item():.4f}")
    return x


if __name__ == "__main__":
    main()
