"""Cases of the attention sublayer's operators: the FP8 block-scaled linear layer (`linear`), writing new keys and values
into the FP8 paged cache (`append`), and attention of a step's tokens over that cache (`attend`).

Each operator has a plain form (elementary torch operations in float32, rounded once at the end) and, with `own`, the
library's calls. `exact` gives the same outputs from the definitions in float64."""

import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
BLOCK = 128  # columns of an activation group, side of a weight scale block
TINY_SCALE = 2.0 ** -126  # scale of a cache block that holds only zeros


# ---------------------------------------------------------------- cases
def listed():
    # 56 query heads of 128 make the DeepSeek-V3-shaped layer's hidden size of 7168; with 8 key/value heads the fused
    # query, key and value projection has (56 + 2 * 8) * 128 = 9216 rows.
    return [
        # one token of one conversation through the query/key/value projection: a weight stream, latency counts
        {"name": "linear, one token", "op": "linear", "m": 1, "k": 7168, "n": 9216, "e8m0": False},
        # eight conversations through the output projection
        {"name": "linear, 8 tokens", "op": "linear", "m": 8, "k": 7168, "n": 7168, "e8m0": False},
        # a small projection whose last scale block is partial in both directions, and an odd number of tokens
        {"name": "linear, ragged", "op": "linear", "m": 37, "k": 1552, "n": 1001, "e8m0": True},
        # a verify batch of 64 conversations with 4 tokens each
        {"name": "linear, verify batch", "op": "linear", "m": 256, "k": 7168, "n": 9216, "e8m0": False},
        # a prompt's chunk: compute bound
        {"name": "linear, prompt chunk", "op": "linear", "m": 4096, "k": 7168, "n": 9216, "e8m0": False},
        # each of 64 conversations stores its newest token
        {"name": "append, a token each", "op": "append", "b": 64, "new": 1, "kv_heads": 8, "dim": 128, "page": 64,
         "len_min": 1, "len_max": 2048},
        # four prompts' chunks of uneven length are stored, each behind what its conversation holds
        {"name": "append, prompt chunks", "op": "append", "b": 4, "new": 2048, "kv_heads": 8, "dim": 128, "page": 64,
         "len_min": 2100, "len_max": 5000},
        # one conversation a page or so beyond its start: latency counts
        {"name": "attend, short", "op": "attend", "b": 1, "new": 1, "heads": 56, "kv_heads": 8, "dim": 128, "page": 64,
         "len_min": 777, "len_max": 777, "pad": 0, "softcap": 0.0, "window": 0, "slopes": False},
        # a serving batch of uneven conversations, with the empty slots of a captured batch size
        {"name": "attend, serving batch", "op": "attend", "b": 64, "new": 1, "heads": 56, "kv_heads": 8, "dim": 128,
         "page": 64, "len_min": 300, "len_max": 16384, "pad": 3, "softcap": 0.0, "window": 0, "slopes": False},
        # one conversation over a long document: the work of one row is split over the whole GPU
        {"name": "attend, long document", "op": "attend", "b": 1, "new": 1, "heads": 64, "kv_heads": 8, "dim": 128,
         "page": 64, "len_min": 131001, "len_max": 131001, "pad": 0, "softcap": 0.0, "window": 0, "slopes": False},
        # verification of drafted tokens: 4 rows a conversation, causal among themselves, small pages
        {"name": "attend, verify 4 tokens", "op": "attend", "b": 16, "new": 4, "heads": 56, "kv_heads": 8, "dim": 128,
         "page": 32, "len_min": 5, "len_max": 8200, "pad": 1, "softcap": 0.0, "window": 0, "slopes": False},
        # small heads with capped scores, a sliding window and a distance bias, over the smallest pages
        {"name": "attend, capped and windowed", "op": "attend", "b": 48, "new": 1, "heads": 32, "kv_heads": 16, "dim": 64,
         "page": 16, "len_min": 17, "len_max": 6000, "pad": 0, "softcap": 30.0, "window": 2049, "slopes": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "append", "attend", "attend"])
    if op == "linear":
        m = _log(rng, 1, 4096)
        k = 16 * _log(rng, 8, 7168 // 16)
        return {"op": op, "m": m, "k": k, "n": _log(rng, 64, 9216), "e8m0": rng.random() < 0.3}
    dim = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        new = _log(rng, 1, 2048)
        b = _log(rng, 1, max(1, min(64, 8192 // new)))
        lo = _log(rng, new, new + 1000)
        return {"op": op, "b": b, "new": new, "kv_heads": rng.choice([1, 2, 3, 4, 8]), "dim": dim, "page": page,
                "len_min": lo, "len_max": _log(rng, lo, lo + 3000)}
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8, 12, 16])
    new = rng.choice([1, 1, 1, 2, 3, 4, 5, 8])
    b = _log(rng, 1, 64)
    hi = _log(rng, new + 1, min(131072, 262144 // b))
    lo = _log(rng, max(1, new), hi)
    return {"op": op, "b": b, "new": new, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "len_min": lo,
            "len_max": hi, "pad": rng.choice([0, 0, 1, 2]) if b > 4 else 0, "softcap": rng.choice([0.0, 0.0, 30.0, 50.0]),
            "window": rng.choice([0, 0, 0, _log(rng, 1, hi)]), "slopes": rng.random() < 0.3}


def _lens(case):
    """Lengths of the sequences (new tokens included): spread over the logarithm of their range, the first the longest;
    the last `pad` ones are the empty slots of a captured batch."""
    lo, hi, b = case["len_min"], case["len_max"], case["b"]
    got = [int(round(lo * (hi / lo) ** (1.0 - (0.6180339887 * i) % 1.0))) for i in range(b)]
    return [0 if i >= b - case.get("pad", 0) else n for i, n in enumerate(got)]


def _news(case, lens):
    """New tokens of each sequence. Prompt chunks are uneven; a step's tokens are as many for every slot."""
    if case["op"] == "append" and case["new"] > 1:
        return [max(1, min(n, case["new"] - (37 * i) % max(1, case["new"] // 2))) for i, n in enumerate(lens)]
    return [case["new"]] * len(lens)


# ---------------------------------------------------------------- inputs
def _pow2_ceil(v):
    """The smallest power of two that is at least v (float32, v >= 0), and at least TINY_SCALE."""
    m, _ = torch.frexp(v)  # v = m * 2^e: v / m is 2^e without rounding
    p = torch.where(m == 0.5, v, v / m)
    return torch.where(v > TINY_SCALE, p, torch.full_like(v, TINY_SCALE))


def _over_max(amax):
    """amax / 448, rounded once: a division by a plain number may become a product with its rounded reciprocal."""
    return amax / torch.full_like(amax, E4M3_MAX)


def _to_e4m3(v):
    return v.clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)


def _blocks(a, side):
    return (a + side - 1) // side


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    if case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        # normalised activations with a few loud channels, as a residual stream has them
        x = torch.randn((m, k), generator=g, device=DEV)
        loud = torch.rand((k,), generator=g, device=DEV)
        x = (x * torch.where(loud > 0.99, 20.0, 1.0)).to(torch.bfloat16)
        # weights of fan-in variance, quantised for each block of 128 x 128
        w = torch.randn((n, k), generator=g, device=DEV) / math.sqrt(k)
        nb, kb = _blocks(n, BLOCK), _blocks(k, BLOCK)
        pad = torch.nn.functional.pad(w, (0, kb * BLOCK - k, 0, nb * BLOCK - n)).view(nb, BLOCK, kb, BLOCK)
        w_s = _over_max(pad.abs().amax(dim=(1, 3)))
        if case["e8m0"]:
            w_s = _pow2_ceil(w_s)
        w = _to_e4m3((pad / w_s[:, None, :, None]).view(nb * BLOCK, kb * BLOCK)[:n, :k]).view(torch.uint8).contiguous()
        return {"op": "linear", "e8m0": case["e8m0"], "x": x, "w": w, "w_s": w_s.contiguous(),
                "out": torch.empty((m, n), dtype=torch.bfloat16, device=DEV),
                "workspace": torch.zeros((64 << 20,), dtype=torch.uint8, device=DEV)}
    lens = _lens(case)
    news = _news(case, lens)
    b, hk, d, page = case["b"], case["kv_heads"], case["dim"], case["page"]
    pages_of = [_blocks(n, page) for n in lens]
    width, total = max(1, max(pages_of)), sum(pages_of) + 1
    # pages in the order an allocator leaves them: any; unused table entries are -1
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    first = torch.tensor([sum(pages_of[:i]) for i in range(b)], device=DEV)
    col = torch.arange(width, device=DEV)
    held = col[None, :] < torch.tensor(pages_of, device=DEV)[:, None]
    table = torch.where(held, order[torch.where(held, first[:, None] + col, 0)], -1).to(torch.int32).contiguous()
    sums = [sum(news[:i]) for i in range(b + 1)]
    s = {"op": case["op"], "page": page, "max_new": max(news), "table": table,
         "lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
         "q_start": torch.tensor(sums, dtype=torch.int32, device=DEV),
         "workspace": torch.zeros((64 << 20,), dtype=torch.uint8, device=DEV)}

    def cache():
        # keys and values of unit size with a loudness of their own for each page and head
        v = torch.randn((total, hk, page, d), generator=g, device=DEV)
        v *= torch.exp2(2.0 * torch.rand((total, hk, 1, 1), generator=g, device=DEV) - 1.0)
        sc = _pow2_ceil(_over_max(v.abs().amax(dim=(2, 3))))
        return _to_e4m3(v.div_(sc[:, :, None, None])).view(torch.uint8), sc

    s["k_cache"], s["k_scale"] = cache()
    s["v_cache"], s["v_scale"] = cache()
    if case["op"] == "append":
        # keys and values as the fused projection leaves them: columns of a wider matrix
        qkv = torch.randn((sums[-1], 3 * hk, d), generator=g, device=DEV)
        qkv = (qkv * torch.exp2(3.0 * torch.rand((sums[-1], 1, 1), generator=g, device=DEV))).to(torch.bfloat16)
        s["k"], s["v"] = qkv[:, hk:2 * hk], qkv[:, 2 * hk:]
        return s
    h = case["heads"]
    s["q"] = torch.randn((sums[-1], h, d), generator=g, device=DEV).mul_(2.0).to(torch.bfloat16)
    s["sm_scale"] = 1.0 / math.sqrt(d)
    s["softcap"], s["window"] = case["softcap"], case["window"]
    s["slopes"] = None
    if case["slopes"]:
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, h + 1, device=DEV, dtype=torch.float32) / h)
    s["out"] = torch.empty((sums[-1], h, d), dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.empty((sums[-1], h), dtype=torch.float32, device=DEV)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        return _own(s)
    return {"linear": _linear, "append": _append, "attend": _attend}[s["op"]](s)


def _own(s):
    import moe_decode_layer_bf16_gb300 as moe
    if s["op"] == "linear":
        moe.fp8_linear(s["x"], s["w"], s["w_s"], s["out"], s["workspace"], e8m0=s["e8m0"])
        return s["out"]
    if s["op"] == "append":
        moe.kv_cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                            s["q_start"], s["lens"], s["max_new"], s["workspace"])
        return _cache_outputs(s)
    moe.decode_attention(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["q_start"],
                         s["lens"], s["max_new"], s["out"], s["workspace"], lse=s["lse"], sm_scale=s["sm_scale"],
                         softcap=s["softcap"], window=s["window"], slopes=s["slopes"])
    return {"out": s["out"], "lse": s["lse"]}


def _cache_outputs(s):
    return {"k": s["k_cache"].view(E4M3), "v": s["v_cache"].view(E4M3), "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _linear(s):
    x, w, w_s = s["x"].float(), s["w"], s["w_s"]
    m, k = x.shape
    n = w.shape[0]
    kb = w_s.shape[1]
    xg = torch.nn.functional.pad(x, (0, kb * BLOCK - k)).view(m, kb, BLOCK)
    amax = xg.abs().amax(dim=2, keepdim=True)
    sc = _over_max(amax)
    if s["e8m0"]:
        sc = _pow2_ceil(sc)
    sc = torch.where(amax == 0, torch.ones_like(sc), sc)
    xd = (_to_e4m3(xg / sc).float() * sc).view(m, kb * BLOCK)[:, :k]
    ws = w_s.repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
    wd = w.view(E4M3).float() * ws
    return (xd @ wd.t()).to(torch.bfloat16)


def _tokens(s, count):
    """For each new token: its sequence and its position in the sequence."""
    at = torch.arange(count, device=DEV)
    start, lens = s["q_start"].long(), s["lens"].long()
    seq = torch.searchsorted(start[1:], at, right=True)
    pos = lens[seq] - (start[seq + 1] - start[seq]) + at - start[seq]
    return seq, pos


def _append(s):
    page, table = s["page"], s["table"].long()
    count, hk, d = s["k"].shape
    b = table.shape[0]
    start, lens = s["q_start"].long(), s["lens"].long()
    seq, pos = _tokens(s, count)
    before = lens - (start[1:] - start[:-1])
    block0 = before // page
    nb = (s["max_new"] + page - 1) // page + 1
    used = (lens - 1) // page - block0  # last touched block of the sequence, from its first
    j = torch.minimum(torch.arange(nb, device=DEV)[None, :], used[:, None])
    ids = table.gather(1, block0[:, None] + j)  # [b, nb]; past the last touched block it is named again
    fresh = (before % page == 0)[:, None]
    tok_block = seq * nb + pos // page - block0[seq]
    old_slots = torch.arange(page, device=DEV)[None, :] < (before % page)[:, None]  # [b, page]
    tok_page, tok_slot = table[seq, pos // page], pos % page
    for x, codes, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        x = x.float()
        amax = torch.zeros((b * nb, hk), device=DEV)
        amax.scatter_reduce_(0, tok_block[:, None].expand(-1, hk), x.abs().amax(dim=2), "amax")
        new = _pow2_ceil(_over_max(amax)).view(b, nb, hk)
        old = scale[ids[:, 0]]
        grown = torch.where(fresh, new[:, 0], torch.maximum(new[:, 0], old))
        new = torch.cat([grown[:, None], new[:, 1:]], dim=1).gather(1, j[:, :, None].expand(-1, -1, hk))
        # what the first block held before keeps its values: its codes are written anew in the grown scale
        held = codes[ids[:, 0]].view(E4M3).float()  # [b, hk, page, d]
        again = _to_e4m3(held * (old / grown)[:, :, None, None]).view(torch.uint8)
        keep = old_slots[:, None, :, None]
        codes[ids[:, 0]] = torch.where(keep, again, codes[ids[:, 0]])
        scale[ids.reshape(-1)] = new.reshape(-1, hk)
        q = _to_e4m3(x / new.view(b * nb, hk)[tok_block][:, :, None]).view(torch.uint8)
        codes[tok_page, :, tok_slot] = q
    return _cache_outputs(s)


def _attend(s):
    page, table = s["page"], s["table"].long()
    b, width = table.shape
    q = s["q"]
    count, h, d = q.shape
    hk, t = s["k_cache"].shape[1], s["max_new"]
    length = width * page
    seq, pos = _tokens(s, count)
    row = torch.arange(count, device=DEV) - s["q_start"].long()[seq]
    qp = torch.zeros((b, t, h, d), device=DEV)
    qp[seq, row] = q.float()
    qp = qp.view(b, t, hk, h // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, (h // hk) * t, d)
    ids = table.clamp(min=0)

    def gathered(codes, scale):
        v = codes[ids].view(E4M3).float() * scale[ids][:, :, :, None, None]
        return v.transpose(1, 2).reshape(b, hk, length, d)

    sc = (qp @ gathered(s["k_cache"], s["k_scale"]).transpose(2, 3)).mul_(s["sm_scale"]).view(b, hk, h // hk, t, length)
    if s["softcap"]:
        sc = torch.tanh(sc / s["softcap"]).mul_(s["softcap"])
    start, lens = s["q_start"].long(), s["lens"].long()
    at = torch.arange(length, device=DEV)
    here = (lens - (start[1:] - start[:-1]))[:, None] + torch.arange(t, device=DEV)  # [b, t] positions of the rows
    if s["slopes"] is not None:
        far = (at[None, None, :] - here[:, :, None]).float()
        sc = sc + s["slopes"].view(1, hk, h // hk, 1, 1) * far[:, None, None]
    seen = (at[None, None, :] <= here[:, :, None]) & (at[None, None, :] < lens[:, None, None])
    if s["window"]:
        seen &= at[None, None, :] > here[:, :, None] - s["window"]
    sc = sc.masked_fill_(~seen[:, None, None], float("-inf"))
    top = sc.amax(dim=-1, keepdim=True)
    p = sc.sub_(torch.where(top == float("-inf"), 0.0, top)).exp_()
    total = p.sum(dim=-1, keepdim=True)
    out = p.view(b, hk, -1, length) @ gathered(s["v_cache"], s["v_scale"])
    out = out.view(b, hk, h // hk, t, d) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log()).squeeze(-1)
    out = out.permute(0, 3, 1, 2, 4).reshape(b, t, h, d)[seq, row]
    return {"out": out.to(torch.bfloat16), "lse": lse.permute(0, 3, 1, 2).reshape(b, t, h)[seq, row]}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        return {"bytes": 2 * m * k + n * k + 4 * _blocks(n, BLOCK) * _blocks(k, BLOCK) + 2 * m * n, "flops": 2 * m * k * n}
    lens = _lens(case)
    news = _news(case, lens)
    hk, d, page = case["kv_heads"], case["dim"], case["page"]
    if case["op"] == "append":
        # the new rows read (bf16) and written (one byte a value), and the touched blocks' scales
        touched = sum((n - 1) // page - (n - t) // page + 1 for n, t in zip(lens, news))
        return {"bytes": 2 * hk * (sum(news) * d * 3 + touched * 8), "flops": 4 * hk * sum(news) * d}
    h, window = case["heads"], case["window"]
    read = pairs = 0
    for n, t in zip(lens, news):
        rows = [n - t + i + 1 for i in range(t) if n - t + i >= 0]
        rows = [min(r, window) if window else r for r in rows]
        pairs += sum(rows)
        read += min(n, window + t - 1) if window else n
    return {"bytes": read * hk * (2 * d + 8 / page) + sum(news) * h * (4 * d + 4), "flops": 4 * pairs * h * d}


# ---------------------------------------------------------------- the definitions in float64
def _e4m3_64(v):
    """The nearest E4M3 values (ties to even, saturating) of float64 values."""
    _, e = torch.frexp(v.abs().clamp(min=2.0 ** -20))
    step = (((e - 1).clamp(min=-6) - 3 + 1023).long() << 52).view(torch.float64)  # 2^(exponent - 3), from its bits
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _scale_64(amax, pow2):
    """The float32 scale of a group, as float64. An E8M0 scale is the power of two at or above amax / 448: the bits
    of the quotient with any mantissa carried into the exponent."""
    s = (amax / E4M3_MAX).float()
    if pow2:
        bits = s.clamp(min=TINY_SCALE).contiguous().view(torch.int32)
        s = ((bits + 0x7FFFFF) & 0x7F800000).view(torch.float32)
    return s.double()


def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "append": _exact_append, "attend": _exact_attend}[case["op"]](case, s)


def _exact_linear(case, s):
    x, w = s["x"].double(), s["w"].view(E4M3).float().double()
    out = torch.zeros((case["m"], case["n"]), dtype=torch.float64, device=DEV)
    row_block = torch.arange(case["n"], device=DEV) // BLOCK
    for b, k0 in enumerate(range(0, case["k"], BLOCK)):
        xb = x[:, k0:k0 + BLOCK]
        amax = xb.abs().amax(dim=1, keepdim=True)
        sc = torch.where(amax == 0, 1.0, _scale_64(amax, case["e8m0"]))
        # the quotient is a float32 by definition: at x = 10.5 s, say, a longer one falls beside the tie
        out += (_e4m3_64((xb / sc).float().double()) * sc) @ (w[:, k0:k0 + BLOCK] * s["w_s"][row_block, b].double()[:, None]).t()
    return out


def _exact_append(case, s):
    lens = _lens(case)
    news = _news(case, lens)
    page, table, done, got = case["page"], s["table"].tolist(), 0, {}
    for name in ("k", "v"):
        got[name] = s[name + "_cache"].view(E4M3).float().double()
        got[name + "_scale"] = s[name + "_scale"].double()
    for i, (n, t) in enumerate(zip(lens, news)):
        for blk in range((n - t) // page, (n - 1) // page + 1):
            lo, hi = max(blk * page, n - t), min((blk + 1) * page, n)
            where, a = table[i][blk], done - (n - t)
            for name in ("k", "v"):
                new = s[name][a + lo:a + hi].double().transpose(0, 1)  # [heads, tokens, dim]
                sc = _scale_64(new.abs().amax(dim=(1, 2)), True)
                codes, scale = got[name][where], got[name + "_scale"][where]
                if lo > blk * page:
                    sc = torch.maximum(sc, scale)
                    kept = codes[:, :lo - blk * page] * scale[:, None, None]
                    codes[:, :lo - blk * page] = _e4m3_64(kept / sc[:, None, None])
                codes[:, lo - blk * page:hi - blk * page] = _e4m3_64(new / sc[:, None, None])
                scale.copy_(sc)
        done += t
    return {"k": got["k"], "v": got["v"], "k_scale": got["k_scale"], "v_scale": got["v_scale"]}


def _exact_attend(case, s):
    lens = _lens(case)
    news = _news(case, lens)
    h, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    table = s["table"].long()
    outs, lses, done = [], [], 0
    for i, (n, t) in enumerate(zip(lens, news)):
        q = s["q"][done:done + t].double()
        done += t
        if n == 0:
            outs.append(torch.zeros((t, h, d), dtype=torch.float64, device=DEV))
            lses.append(torch.full((t, h), float("-inf"), dtype=torch.float64, device=DEV))
            continue
        ids = table[i, :_blocks(n, page)]

        def rows(name):
            v = s[name + "_cache"][ids].view(E4M3).float().double() * s[name + "_scale"][ids].double()[:, :, None, None]
            v = v.transpose(0, 1).reshape(hk, -1, d)[:, :n]
            return v.repeat_interleave(h // hk, 0)  # [h, n, d]

        sc = torch.einsum("thd,hnd->htn", q, rows("k")) / math.sqrt(d)
        if case["softcap"]:
            sc = case["softcap"] * torch.tanh(sc / case["softcap"])
        gap = torch.arange(n, device=DEV)[None, :] - (n - t + torch.arange(t, device=DEV))[:, None]  # key minus row
        if case["slopes"]:
            sc = sc + torch.exp2(-8.0 * torch.arange(1, h + 1, device=DEV).double() / h)[:, None, None] * gap
        sc = sc.masked_fill(gap > 0, float("-inf"))
        if case["window"]:
            sc = sc.masked_fill(gap <= -case["window"], float("-inf"))
        lse = torch.logsumexp(sc, dim=2)
        p = torch.exp(sc - torch.where(torch.isinf(lse), 0.0, lse)[:, :, None])
        outs.append(torch.einsum("htn,hnd->thd", p, rows("v")))
        lses.append(lse.t())
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
