"""One decoder block, a token at a time: the attention sublayer over an FP8 paged
cache, the layer boundary, and the MoE layer, captured once in a CUDA graph and
replayed for each step.

    python examples/decode_block.py                # a small block
    python examples/decode_block.py --dsv3         # DeepSeek-V3-shaped MoE layer, 56 query and 8 kv heads of 128
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_decode_layer_bf16_gb300 as moe  # noqa: E402
from moe_decode_layer_bf16_gb300 import synth  # noqa: E402
from moe_decode_layer_bf16_gb300.dims import DSV3, TINY  # noqa: E402


def attention_weights(hidden, heads, kv_heads, head_dim, seed=0, device="cuda"):
    """Random projections, quantised for each 128 x 128 block."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def draw(rows, cols):
        return synth.fp8_blocks(torch.randn((rows, cols), generator=g, device=device) / cols ** 0.5, False)

    qkv, qkv_s = draw((heads + 2 * kv_heads) * head_dim, hidden)
    o, o_s = draw(hidden, heads * head_dim)
    return {"qkv": qkv, "qkv_s": qkv_s, "o": o, "o_s": o_s}


class Block:
    """Attention and MoE sublayers of one decoder block for `batch` sequences."""

    def __init__(self, dims, heads, kv_heads, head_dim, batch, max_len, page_size=64, max_new=1):
        H, self.batch, pages = dims.hidden, batch, -(-max_len // page_size)
        self.cache = moe.Fp8KvCache(batch * pages, kv_heads, head_dim, page_size)
        tokens = batch * max_new
        self.attention = moe.AttentionDecode(H, heads, kv_heads, head_dim, attention_weights(H, heads, kv_heads, head_dim),
                                             self.cache, tokens, max_new=max_new)
        self.layer = moe.MoeDecodeLayer(dims, synth.make_layer(dims, device="cuda"), max_tokens=tokens)
        self.gain = torch.ones(H, dtype=torch.bfloat16, device="cuda")
        self.page_table = torch.randperm(batch * pages, device="cuda").to(torch.int32).view(batch, pages)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.eps = dims.rms_eps

    def step(self, x, residual, q_start):
        """x, residual bf16 [tokens, hidden]; the tokens of each sequence as q_start
        says.  Advances the sequences' lengths."""
        self.lens += q_start[1:] - q_start[:-1]
        a = self.attention(x, self.page_table, q_start, self.lens)
        y, r = torch.empty_like(x), torch.empty_like(residual)
        moe.rmsnorm_residual(residual, self.gain, y, r, self.eps, x=a)
        return self.layer(y, r)


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--dsv3", action="store_true")
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=8, help="tokens of each prompt, taken in one step")
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args(argv)
    dims, heads, kv_heads, head_dim = (DSV3, 56, 8, 128) if a.dsv3 else (TINY, 8, 2, 64)
    torch.manual_seed(0)
    block = Block(dims, heads, kv_heads, head_dim, a.batch, a.prompt + a.steps + 2, max_new=a.prompt)
    n = a.batch * a.prompt
    x, residual = synth.make_tokens(n, dims.hidden, device="cuda")
    start = torch.arange(a.batch + 1, dtype=torch.int32, device="cuda")
    y, r = block.step(x, residual, start * a.prompt)

    # each step takes the block's output of the last token as the next one's input
    x, residual = y[a.prompt - 1::a.prompt].clone(), r[a.prompt - 1::a.prompt].clone()
    y, r = block.step(x, residual, start)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        y, r = block.step(x, residual, start)
    torch.cuda.synchronize()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(a.steps):
        graph.replay()
        x.copy_(y)
        residual.copy_(r)
    end.record()
    torch.cuda.synchronize()
    status = (block.attention.status(), block.layer.status())
    assert status == (moe.MOE_OK, moe.MOE_OK), status
    print(f"{a.steps} steps of {a.batch} sequences, now {block.lens.tolist()} tokens: "
          f"{begin.elapsed_time(end) / a.steps * 1e3:.1f} us a step; |y| {y.float().abs().mean().item():.4f}")
    return y


if __name__ == "__main__":
    main()
