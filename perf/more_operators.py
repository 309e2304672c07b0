"""Cases of the operators that a prompt meets on its way through the attention sublayer: the residual's addition and RMSNorm
with FP8 output (`norm`), pages of the cache given to a step's tokens and taken back (`extend`, `release`), and causal
attention over packed prompts (`prompt`).

Each operator has a plain form (elementary torch operations in float32, rounded once at the end) and, with `own`, the
library's calls. `exact` gives the computed outputs from the definitions in float64."""

import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
GROUP = 128  # columns that share a scale
EPS = 1e-6


# ---------------------------------------------------------------- cases
def listed():
    # 56 query heads of 128 on 8 key/value heads belong to the DeepSeek-V3-shaped layer's hidden size of 7168.
    return [
        # the boundary before one token's projections: latency counts
        {"name": "norm, one token", "op": "norm", "m": 1, "h": 7168, "x": True, "out": False, "e8m0": False, "gap": 0},
        # a small odd batch at the model's entry (nothing to add yet), the last group partial, the bf16 rows wanted too
        {"name": "norm, ragged", "op": "norm", "m": 37, "h": 2064, "x": False, "out": True, "e8m0": True, "gap": 48},
        # a prompt's chunk: a stream of bytes
        {"name": "norm, prompt chunk", "op": "norm", "m": 8192, "h": 7168, "x": True, "out": False, "e8m0": False, "gap": 0},
        # each of 64 conversations gets room for its next token, with rows of a captured batch to spare
        {"name": "extend, a token each", "op": "extend", "b": 64, "page": 64, "len_min": 1, "len_max": 16384, "new_min": 1,
         "new_max": 1, "spare": 4, "want": 1.5, "fresh": False},
        # new prompts among running conversations on small pages, with too few pages for the last ones
        {"name": "extend, prompts", "op": "extend", "b": 300, "page": 16, "len_min": 1, "len_max": 3000, "new_min": 1,
         "new_max": 4096, "spare": 100, "want": 0.9, "fresh": True},
        # a few of 64 conversations have ended
        {"name": "release, a few", "op": "release", "b": 64, "page": 64, "len_min": 1, "len_max": 16384, "done": 0.1},
        # most of a large batch of long conversations has ended, on small pages
        {"name": "release, most", "op": "release", "b": 500, "page": 16, "len_min": 100, "len_max": 8000, "done": 0.8},
        # one short question: latency counts
        {"name": "prompt, one short", "op": "prompt", "b": 1, "len_min": 33, "len_max": 33, "pad": 0, "heads": 56, "kv_heads": 8,
         "dim": 128, "softcap": 0.0, "window": 0, "slopes": False},
        # prompts of a serving step, packed, with the empty slots of a captured batch size
        {"name": "prompt, serving mix", "op": "prompt", "b": 16, "len_min": 20, "len_max": 2048, "pad": 2, "heads": 56,
         "kv_heads": 8, "dim": 128, "softcap": 0.0, "window": 0, "slopes": False},
        # a long document: compute bound
        {"name": "prompt, long document", "op": "prompt", "b": 1, "len_min": 8192, "len_max": 8192, "pad": 0, "heads": 56,
         "kv_heads": 8, "dim": 128, "softcap": 0.0, "window": 0, "slopes": False},
        # a key/value head for each query head, three uneven prompts
        {"name": "prompt, heads of their own", "op": "prompt", "b": 3, "len_min": 701, "len_max": 2999, "pad": 0, "heads": 16,
         "kv_heads": 16, "dim": 128, "softcap": 0.0, "window": 0, "slopes": False},
        # small heads with capped scores, a sliding window and a distance bias
        {"name": "prompt, capped and windowed", "op": "prompt", "b": 6, "len_min": 97, "len_max": 4001, "pad": 0, "heads": 32,
         "kv_heads": 16, "dim": 64, "softcap": 30.0, "window": 1025, "slopes": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "extend", "release", "prompt", "prompt", "prompt"])
    if op == "norm":
        return {"op": op, "m": _log(rng, 1, 8192), "h": 16 * _log(rng, 4, 7168 // 16), "x": rng.random() < 0.7,
                "out": rng.random() < 0.3, "e8m0": rng.random() < 0.3, "gap": rng.choice([0, 0, 8, 2048])}
    page = rng.choice([16, 32, 64, 128])
    lo = _log(rng, 1, 1000)
    if op == "release":
        return {"op": op, "b": _log(rng, 1, 500), "page": page, "len_min": lo, "len_max": _log(rng, lo, 8000),
                "done": rng.choice([0.02, 0.3, 0.8])}
    if op == "extend":
        new = _log(rng, 1, 500)
        return {"op": op, "b": _log(rng, 1, 300), "page": page, "len_min": lo, "len_max": _log(rng, lo, 3000),
                "new_min": new if rng.random() < 0.5 else 1, "new_max": new, "spare": rng.choice([0, 1, 64]),
                "want": rng.choice([0.5, 1.0, 1.5]), "fresh": rng.random() < 0.5}
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    b = _log(rng, 1, 64)
    # the plain form holds every score of the longest prompt for each prompt and head
    hi = _log(rng, 2, min(8192, int(math.sqrt(3.7e9 / (b * heads)))))
    return {"op": op, "b": b, "len_min": _log(rng, 1, hi), "len_max": hi, "pad": rng.choice([0, 0, 1, 2]) if b > 4 else 0,
            "heads": heads, "kv_heads": kv_heads, "dim": rng.choice([64, 128, 128]), "softcap": rng.choice([0.0, 0.0, 30.0, 50.0]),
            "window": rng.choice([0, 0, 0, _log(rng, 1, hi)]), "slopes": rng.random() < 0.25}


def _spread(lo, hi, n, turn=0.6180339887):
    """n lengths spread over the logarithm of their range, the first the longest."""
    return [int(round(lo * (hi / lo) ** (1.0 - (turn * i) % 1.0))) for i in range(n)]


def _lens(case):
    """Tokens of each conversation: none in the empty slots at a captured batch's end (`pad`), nor in each third one where
    some are new (`fresh`)."""
    got = _spread(case["len_min"], case["len_max"], case["b"])
    return [0 if i >= case["b"] - case.get("pad", 0) or (case.get("fresh") and i % 3 == 2) else n for i, n in enumerate(got)]


def _news(case):
    return _spread(case["new_min"], case["new_max"], case["b"], 0.4142135623)


def _up(a, side):
    return (a + side - 1) // side


def _done(case):
    """Which conversations have ended: the same share of them everywhere in the batch, one at least."""
    return [i == 0 or (0.7548776662 * i) % 1.0 < case["done"] for i in range(case["b"])]


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op = case["op"]
    if op == "norm":
        m, h = case["m"], case["h"]

        def rows(loudness):
            # rows of a residual stream with a few loud channels; with a gap, columns of a wider matrix
            v = torch.randn((m, h + case["gap"]), generator=g, device=DEV) * loudness
            v[:, :h] *= torch.where(torch.rand((h,), generator=g, device=DEV) > 0.99, 20.0, 1.0)
            return v.to(torch.bfloat16)[:, :h]

        s = {"op": op, "e8m0": case["e8m0"], "residual": rows(4.0), "x": rows(1.0) if case["x"] else None,
             "gain": (1.0 + 0.1 * torch.randn((h,), generator=g, device=DEV)).to(torch.bfloat16),
             "residual_out": torch.empty((m, h), dtype=torch.bfloat16, device=DEV),
             "codes": torch.empty((m, h), dtype=torch.uint8, device=DEV),
             "scales": torch.empty((_up(h, GROUP), m + 3 & -4), dtype=torch.float32, device=DEV), "out": None}
        if case["out"]:
            s["out"] = torch.empty((m, h), dtype=torch.bfloat16, device=DEV)
        return s
    lens = _lens(case)
    b = case["b"]

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)

    if op == "prompt":
        h, hk, d = case["heads"], case["kv_heads"], case["dim"]
        total = sum(lens)
        # queries, keys and values as the fused projection leaves them: columns of one matrix
        qkv = torch.randn((total, h + 2 * hk, d), generator=g, device=DEV)
        qkv[:, :h] *= 2.0
        qkv = qkv.to(torch.bfloat16)
        slopes = None
        if case["slopes"]:
            slopes = torch.exp2(-8.0 * torch.arange(1, h + 1, device=DEV, dtype=torch.float32) / h)
        return {"op": op, "q": qkv[:, :h], "k": qkv[:, h:h + hk], "v": qkv[:, h + hk:], "longest": max(lens),
                "q_start": ints([sum(lens[:i]) for i in range(b + 1)]), "sm_scale": 1.0 / math.sqrt(d),
                "softcap": case["softcap"], "window": case["window"], "slopes": slopes,
                "out": torch.empty((total, h, d), dtype=torch.bfloat16, device=DEV),
                "lse": torch.empty((total, h), dtype=torch.float32, device=DEV),
                "workspace": torch.zeros((1 << 20,), dtype=torch.uint8, device=DEV)}
    page = case["page"]
    held = [_up(n, page) for n in lens]
    # pages in the order an allocator leaves them: any; table entries past a conversation's pages are -1
    if op == "extend":
        news = _news(case)
        need = sum(_up(n + t, page) - p for n, t, p in zip(lens, news, held))
        free = max(1, int(need * case["want"]))
        width = max(_up(n + t, page) for n, t in zip(lens, news))
        cap = sum(held) + free
    else:
        news, free, width = None, 7, max(held)
        cap = sum(held) + free
    order = torch.randperm(cap, generator=g, device=DEV).to(torch.int32)
    first = torch.tensor([sum(held[:i]) for i in range(b)], device=DEV)
    col = torch.arange(width, device=DEV)
    have = col[None, :] < torch.tensor(held, device=DEV)[:, None]
    table = torch.where(have, order[free:][torch.where(have, first[:, None] + col, 0)], -1).to(torch.int32).contiguous()
    stack = torch.full((cap,), -1, dtype=torch.int32, device=DEV)
    stack[:free] = order[:free]
    s = {"op": op, "page": page, "num_pages": cap, "table": table, "lens": ints(lens), "free_pages": stack,
         "free_state": ints([free, 0]), "free_out": ints([0, 0]), "lens_out": ints([0] * b),
         "workspace": torch.zeros((1 << 20,), dtype=torch.uint8, device=DEV)}
    if op == "extend":
        rows = sum(news) + case["spare"]
        s["new"] = ints(news)
        s["q_start"] = ints([0] * (b + 1))
        s["positions"] = torch.empty((rows,), dtype=torch.int32, device=DEV)
        s["slots"] = torch.empty((rows,), dtype=torch.int64, device=DEV)
    else:
        s["done"] = torch.tensor(_done(case), device=DEV)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        return _own(s)
    return {"norm": _norm, "extend": _extend, "release": _release, "prompt": _prompt}[s["op"]](s)


def _own(s):
    import moe_decode_layer_bf16_gb300 as moe
    if s["op"] == "norm":
        moe.rmsnorm_residual_fp8(s["residual"], s["gain"], s["codes"], s["scales"], s["residual_out"], EPS, x=s["x"],
                                 out=s["out"], e8m0=s["e8m0"])
        return _norm_outputs(s)
    if s["op"] == "extend":
        moe.kv_pages_extend(s["table"], s["lens"], s["new"], s["free_pages"], s["free_state"], s["page"], s["num_pages"],
                            s["q_start"], s["lens_out"], s["free_out"], s["positions"], s["slots"], s["workspace"])
        return {n: s[n] for n in ("table", "q_start", "lens_out", "free_out", "positions", "slots")}
    if s["op"] == "release":
        moe.kv_pages_release(s["table"], s["lens"], s["done"], s["free_pages"], s["free_state"], s["page"], s["num_pages"],
                             s["lens_out"], s["free_out"], s["workspace"])
        return {n: s[n] for n in ("free_pages", "lens_out", "free_out")}
    moe.prompt_attention(s["q"], s["k"], s["v"], s["q_start"], s["out"], s["workspace"], lse=s["lse"],
                         sm_scale=s["sm_scale"], softcap=s["softcap"], window=s["window"], slopes=s["slopes"])
    return {"out": s["out"], "lse": s["lse"]}


def _norm_outputs(s):
    return {"residual_out": s["residual_out"], "codes": s["codes"].view(E4M3), "scales": s["scales"][:, :s["codes"].shape[0]],
            "out": s["out"]}


def _pow2_ceil(v):
    """The smallest power of two that is at least v (float32, v > 0)."""
    m, _ = torch.frexp(v)  # v = m * 2^e: v / m is 2^e without rounding
    return torch.where(m == 0.5, v, v / m)


def _norm(s):
    r = s["residual"].float()
    if s["x"] is not None:
        r = s["x"].float() + r
    r = r.to(torch.bfloat16)
    s["residual_out"].copy_(r)
    r = r.float()
    m, h = r.shape
    y = r * torch.rsqrt((r * r).mean(dim=1, keepdim=True) + EPS) * s["gain"].float()
    groups = _up(h, GROUP)
    yg = torch.nn.functional.pad(y, (0, groups * GROUP - h)).view(m, groups, GROUP)
    amax = yg.abs().amax(dim=2)
    # (a division by a plain number may become a product with its rounded reciprocal)
    sc = amax / torch.full_like(amax, E4M3_MAX)
    if s["e8m0"]:
        sc = _pow2_ceil(sc)
    sc = torch.where(amax == 0, torch.ones_like(sc), sc)
    codes = (yg / sc[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3).view(torch.uint8)
    s["codes"].copy_(codes.view(m, groups * GROUP)[:, :h])
    s["scales"][:, :m] = sc.t()
    if s["out"] is not None:
        s["out"].copy_(y)
    return _norm_outputs(s)


def _extend(s):
    lens, new, page, table = s["lens"].long(), s["new"].long(), s["page"], s["table"]
    b, width = table.shape
    count = s["free_state"][0].long()
    held = (lens + page - 1) // page
    need = (lens + new + page - 1) // page - held
    upto = need.cumsum(0)
    fits = (need == 0) | (upto <= count)
    got, n = torch.where(fits, need, 0), torch.where(fits, new, 0)
    # the pages of the stack's top first, in the order of the conversations and of their tokens
    j = torch.arange(width, device=DEV)[None, :] - held[:, None]
    at = (count - 1 - (upto - need)[:, None] - j).clamp(0, s["free_pages"].shape[0] - 1)
    table.copy_(torch.where((j >= 0) & (j < got[:, None]), s["free_pages"][at], table))
    s["q_start"].zero_()
    s["q_start"][1:] = n.cumsum(0)
    s["lens_out"].copy_(lens + n)
    s["free_out"].copy_(torch.stack([count - got.sum(), need.sum() - got.sum()]))
    start = s["q_start"].long()
    row = torch.arange(s["slots"].shape[0], device=DEV)
    seq = torch.searchsorted(start[1:], row, right=True)
    live = seq < b
    seq = seq.clamp(max=b - 1)
    pos = lens[seq] + row - start[seq]
    where = table[seq, (pos // page).clamp(max=width - 1)].long()
    s["positions"].copy_(torch.where(live, pos, -1))
    s["slots"].copy_(torch.where(live, where * page + pos % page, -1))
    return {n: s[n] for n in ("table", "q_start", "lens_out", "free_out", "positions", "slots")}


def _release(s):
    lens, done, page, table = s["lens"].long(), s["done"], s["page"], s["table"]
    count, cap = s["free_state"][0].long(), s["free_pages"].shape[0]
    n = torch.where(done, (lens + page - 1) // page, 0)
    upto = n.cumsum(0)
    col = torch.arange(table.shape[1], device=DEV)[None, :]
    to = torch.where(col < n[:, None], count + (upto - n)[:, None] + col, cap)
    stack = torch.cat([s["free_pages"], s["free_pages"][:1]])
    stack[to.reshape(-1)] = table.reshape(-1)  # (entries that stay with their conversation fall behind the stack's end)
    s["free_pages"].copy_(stack[:cap])
    s["lens_out"].copy_(torch.where(done, 0, lens))
    s["free_out"].copy_(torch.stack([count + n.sum(), torch.zeros_like(count)]))
    return {n: s[n] for n in ("free_pages", "lens_out", "free_out")}


def _prompt(s):
    q, k, v, t = s["q"], s["k"], s["v"], s["longest"]
    total, h, d = q.shape
    hk = k.shape[1]
    start = s["q_start"].long()
    b = start.shape[0] - 1
    row = torch.arange(total, device=DEV)
    seq = torch.searchsorted(start[1:], row, right=True)
    pos = row - start[seq]

    def padded(x):
        p = torch.zeros((b, t, x.shape[1], d), device=DEV)
        p[seq, pos] = x.float()
        return p.transpose(1, 2)  # [b, heads, t, d]

    group = h // hk
    qp = padded(q).reshape(b, hk, group * t, d)
    sc = (qp @ padded(k).transpose(2, 3)).mul_(s["sm_scale"]).view(b, hk, group, t, t)
    if s["softcap"]:
        sc = sc.div_(s["softcap"]).tanh_().mul_(s["softcap"])
    at = torch.arange(t, device=DEV)
    gap = at[None, :] - at[:, None]  # key minus row
    if s["slopes"] is not None:
        sc += s["slopes"].view(1, hk, group, 1, 1) * gap.float()
    seen = gap <= 0
    if s["window"]:
        seen = seen & (gap > -s["window"])
    sc = sc.masked_fill_(~seen, float("-inf"))
    top = sc.amax(dim=-1, keepdim=True)
    p = sc.sub_(top).exp_()
    sums = p.sum(dim=-1, keepdim=True)
    out = (p.view(b, hk, group * t, t) @ padded(v)).view(b, hk, group, t, d) / sums
    lse = (top + sums.log()).squeeze(-1)
    s["out"].copy_(out.permute(0, 3, 1, 2, 4).reshape(b, t, h, d)[seq, pos])
    s["lse"].copy_(lse.permute(0, 3, 1, 2).reshape(b, t, h)[seq, pos])
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "norm":
        m, h = case["m"], case["h"]
        return {"bytes": m * h * (5 + 2 * case["x"] + 2 * case["out"]) + 2 * h + 4 * m * _up(h, GROUP), "flops": 8 * m * h}
    lens = _lens(case)
    b = case["b"]
    if case["op"] == "prompt":
        h, hk, d, w = case["heads"], case["kv_heads"], case["dim"], case["window"]
        pairs = 0
        for n in lens:
            m = min(n, w) if w else n  # rows up to the m-th see all before them, the others as many as the window holds
            pairs += m * (m + 1) // 2 + (n - m) * m
        return {"bytes": sum(lens) * (4 * h * d + 4 * hk * d + 4 * h) + 4 * (b + 1), "flops": 4 * pairs * h * d}
    page = case["page"]
    held = [_up(n, page) for n in lens]
    if case["op"] == "release":
        pages = sum(p for p, d in zip(held, _done(case)) if d)
        return {"bytes": 8 * pages + 9 * b + 16, "flops": 0}
    news = _news(case)
    needs = [_up(n + t, page) - p for n, t, p in zip(lens, news, held)]
    left = max(1, int(sum(needs) * case["want"]))
    pages, upto = 0, 0
    for need in needs:
        upto += need
        pages += need if upto <= left else 0
    # the rows of the step, and those to spare, are written whether they are given to a conversation or not
    return {"bytes": 8 * pages + 16 * b + 20 + 12 * (sum(news) + case["spare"]), "flops": 0}


# ---------------------------------------------------------------- the definitions in float64
def exact(case, seed):
    if case["op"] in ("extend", "release"):
        return None  # whole numbers
    s = prepare(case, seed)
    return _exact_norm(case, s) if case["op"] == "norm" else _exact_prompt(case, s)


def _exact_norm(case, s):
    r = s["residual"].double()
    if s["x"] is not None:
        r = r + s["x"].double()
    r = r.float().bfloat16().double()  # the new residual is held in bf16 by definition, from a float32 sum
    mean = (r * r).sum(dim=1, keepdim=True) / case["h"]
    y = r / torch.sqrt(mean + EPS) * s["gain"].double()
    codes, scales = torch.zeros_like(y), []
    for c in range(0, case["h"], GROUP):
        amax = y[:, c:c + GROUP].abs().amax(dim=1)
        sc = amax / E4M3_MAX
        if case["e8m0"]:
            sc = torch.exp2(torch.ceil(torch.log2(sc)))
        sc = torch.where(amax == 0, 1.0, sc)
        # what the codes stand for, unrounded: quotients of products of bf16 values often lie on the border of two codes,
        # where the last bit of any arithmetic decides
        codes[:, c:c + GROUP] = y[:, c:c + GROUP] / sc[:, None]
        scales.append(sc)
    return {"residual_out": r, "codes": codes, "scales": torch.stack(scales), "out": y if case["out"] else None}


def _exact_prompt(case, s):
    h, hk = case["heads"], case["kv_heads"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for n in _lens(case):
        if n == 0:
            continue
        back = torch.arange(n, device=DEV)[:, None] - torch.arange(n, device=DEV)[None, :]  # row minus key
        hidden = back < 0
        if case["window"]:
            hidden |= back >= case["window"]
        for i in range(h):
            q, k, v = (s[x][at:at + n, j].double() for x, j in (("q", i), ("k", i * hk // h), ("v", i * hk // h)))
            sc = q @ k.t() / math.sqrt(case["dim"])
            if case["softcap"]:
                sc = case["softcap"] * torch.tanh(sc / case["softcap"])
            if case["slopes"]:
                sc = sc - s["slopes"][i].double() * back
            sc = sc.masked_fill(hidden, float("-inf"))
            lse[at:at + n, i] = torch.logsumexp(sc, dim=1)
            out[at:at + n, i] = torch.softmax(sc, dim=1) @ v
        at += n
    return {"out": out, "lse": lse}
