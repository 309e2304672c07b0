"""Oracle of a prompt's operators (test infrastructure only): residual RMSNorm with
FP8 output, pages given and taken back, causal attention of packed prompts; numpy,
float64 where something is computed."""

from __future__ import annotations

import numpy as np

from oracle.moe_oracle import bf16_round

QMAX = 448.0


def norm(residual, gain, eps, x=None):
    """(new residual, y, scales of amax / 448): residual, x float32 arrays of bf16 values."""
    r = np.asarray(residual, np.float32)
    if x is not None:
        r = (np.asarray(x, np.float32) + r).astype(np.float32)
    r = bf16_round(r).astype(np.float64)
    y = r / np.sqrt((r * r).mean(axis=1, keepdims=True) + eps) * np.asarray(gain, np.float64)
    M, H = y.shape
    amax = np.zeros((-(-H // 128), M))
    for g in range(amax.shape[0]):
        amax[g] = np.abs(y[:, 128 * g:128 * g + 128]).max(axis=1)
    return r, y, amax / QMAX


def extend(table, lens, new, stack, state, page, num_pages, rows):
    """(table, q_start, lens, state, positions, slots, whether all values fit)."""
    table, out_lens = table.copy(), [int(n) for n in lens]
    B, width = table.shape
    ok = 0 <= state[0] <= len(stack)
    count = int(state[0]) if ok else 0
    positions, slots = np.full(rows, -1, np.int32), np.full(rows, -1, np.int64)
    q_start, asked_pages, asked_rows, got, at = [0], 0, 0, 0, 0
    for b in range(B):
        n, t = int(lens[b]), int(new[b])
        if n < 0 or t < 0 or n + t > width * page:
            ok = False
            q_start.append(at)
            continue
        held = -(-n // page)
        need = -(-(n + t) // page) - held
        asked_pages += need
        asked_rows += t
        room = t == 0 or asked_rows <= rows
        ok &= room
        if not room or (need and asked_pages > count):
            q_start.append(at)
            continue
        for j in range(need):
            table[b, held + j] = stack[count - 1 - got]
            ok &= 0 <= table[b, held + j] < num_pages
            got += 1
        for i in range(t):
            p = int(table[b, (n + i) // page])
            positions[at] = n + i
            if 0 <= p < num_pages:
                slots[at] = p * page + (n + i) % page
            else:
                ok = False
            at += 1
        out_lens[b] = n + t
        q_start.append(at)
    return (table, np.array(q_start, np.int32), np.array(out_lens, np.int32),
            np.array([state[0] - got, asked_pages - got], np.int32), positions, slots, ok)


def release(table, lens, done, stack, state, page, num_pages):
    """(stack, lens, state, whether all values fit)."""
    stack, out_lens, ok = stack.copy(), np.array(lens, np.int32), True
    pages = []
    gone = []
    for b, n in enumerate(lens):
        if not done[b]:
            continue
        if n < 0 or n > table.shape[1] * page:
            ok = False
            continue
        gone.append(b)
        pages += [int(p) for p in table[b, :-(-int(n) // page)]]
    if state[0] < 0 or state[0] > len(stack) or len(pages) > len(stack) - state[0]:
        return stack, out_lens, np.array([state[0], 0], np.int32), False
    ok &= all(0 <= p < num_pages for p in pages)
    stack[state[0]:state[0] + len(pages)] = pages
    out_lens[gone] = 0
    return stack, out_lens, np.array([state[0] + len(pages), 0], np.int32), ok


def attention(q, k, v, q_start, sm_scale, softcap=0.0, window=0, slopes=None):
    """(out, lse, sum_j p_j |v_j|, |sm_scale| max_j sum_d |q_d k_d|, largest |score|) of the
    rows of the prompts, float64; zeros elsewhere."""
    total, H, D = q.shape
    G = H // k.shape[1]
    out, mag = np.zeros((total, H, D)), np.zeros((total, H, D))
    lse, unit, big = np.zeros((total, H)), np.zeros((total, H)), np.zeros((total, H))
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    for b in range(len(q_start) - 1):
        rows = slice(int(q_start[b]), int(q_start[b + 1]))
        n = rows.stop - rows.start
        if n <= 0:
            continue
        gap = np.arange(n)[None, :] - np.arange(n)[:, None]
        hidden = gap > 0
        if window > 0:
            hidden |= gap <= -window
        for h in range(H):
            Q, K, V = q[rows, h], k[rows, h // G], v[rows, h // G]
            s = sm_scale * (Q @ K.T)
            unit[rows, h] = np.where(hidden, 0.0, abs(sm_scale) * (np.abs(Q) @ np.abs(K).T)).max(axis=1)
            if softcap:
                s = softcap * np.tanh(s / softcap)
            if slopes is not None:
                s = s + float(slopes[h]) * gap
            big[rows, h] = np.where(hidden, 0.0, np.abs(s)).max(axis=1)
            s = np.where(hidden, -np.inf, s)
            m = s.max(axis=1, keepdims=True)
            p = np.exp(s - m)
            L = p.sum(axis=1, keepdims=True)
            out[rows, h] = (p / L) @ V
            mag[rows, h] = (p / L) @ np.abs(V)
            lse[rows, h] = (m + np.log(L))[:, 0]
    return out, lse, mag, unit, big
