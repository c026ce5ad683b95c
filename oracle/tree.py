"""Plain 64-bit definitions of the tree-drafting operations (numpy, slow):
rotary positions in general form, the masks, walk and commit of a tree of
drafts, its attention over KV_full, and log probabilities of tokens.  Shares
no code with the CUDA path."""
from __future__ import annotations

import math

import numpy as np


def rotary_frequencies(theta, rot_dim, factor=1.0, original_len=0, low_turns=0.0, high_turns=0.0) -> np.ndarray:
    """Radians per position of each pair."""
    f = np.array([theta ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)], dtype=np.float64)
    if factor == 1.0:
        return f
    if original_len == 0:
        return f / factor
    g = np.clip((original_len * f / (2 * math.pi) - low_turns) / (high_turns - low_turns), 0.0, 1.0)
    return f * (g + (1.0 - g) / factor)


def rotary(x, pos, freqs, interleaved=False, amplitude=1.0) -> np.ndarray:
    """x [m][heads][d], pos [m]; the first 2 * len(freqs) channels rotated."""
    y = np.array(x, dtype=np.float64)
    n = len(freqs)
    ang = np.asarray(pos, dtype=np.float64)[:, None] * freqs[None]
    c, s = amplitude * np.cos(ang)[:, None], amplitude * np.sin(ang)[:, None]
    i0 = np.arange(n) * 2 if interleaved else np.arange(n)
    i1 = i0 + 1 if interleaved else i0 + n
    a, b = np.array(y[..., i0]), np.array(y[..., i1])
    y[..., i0], y[..., i1] = a * c - b * s, b * c + a * s
    return y


def tree_plan(parent, seq_len):
    """One request: (mask list of ints, positions, whether something was
    wrong).  Absent nodes: mask 0, position -1."""
    n = len(parent)
    base = seq_len - n
    masks, pos, bad = [], [], base < 0
    for i, p in enumerate(parent):
        p = int(p)
        if base < 0:
            masks.append(0)
        elif p < -1:
            masks.append(0)
        elif p >= i or (p >= 0 and masks[p] == 0):
            masks.append(0)
            bad = True
        else:
            masks.append((1 << i) | (masks[p] if p >= 0 else 0))
        pos.append(base + bin(masks[-1]).count("1") - 1 if masks[-1] else -1)
    return masks, pos, bad


def tree_accept(parent, tokens, verified):
    """One request: (accept_len, path, emitted), lists of their own length."""
    if int(parent[0]) != -1:
        return -1, [], []
    path = [0]
    while True:
        cur = path[-1]
        nxt = [j for j in range(cur + 1, len(parent)) if parent[j] == cur and tokens[j] == verified[cur]]
        if not nxt:
            break
        path.append(nxt[0])
    return len(path) - 1, path, [int(tokens[j]) for j in path[1:]] + [int(verified[path[-1]])]


def tree_attn(q, k, v, masks, scale):
    """One request: q [n_q][Hq][D], k / v [L][Hkv][D] in 64 bits.  Returns
    (out, spread, score_err): spread[..c] = sum_t p_t |v_tc|, score_err[i][h] =
    max_t sum_c |q_c k_tc| * scale, which error bounds are made of."""
    n_q, hq, d = q.shape
    L, hkv = k.shape[0], k.shape[1]
    base = L - n_q
    out, spread, serr = np.zeros((n_q, hq, d)), np.zeros((n_q, hq, d)), np.zeros((n_q, hq))
    for i in range(n_q):
        m = int(masks[i])
        if m == 0:
            continue
        seen = [t for t in range(L) if t < base or (m >> (t - base)) & 1]
        for h in range(hq):
            kk, vv = k[seen, h // (hq // hkv)], v[seen, h // (hq // hkv)]
            if not len(seen):
                continue
            s = kk @ q[i, h] * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            out[i, h], spread[i, h] = p @ vv, p @ np.abs(vv)
            serr[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * scale
    return out, spread, serr


def token_logprobs(x, ids, tau, k):
    """One row of logits in 64 bits: (log p of ids, entropy, top ids, top log p)."""
    x = np.asarray(x, dtype=np.float64)
    if np.isnan(x).any() or (x == np.inf).any():
        nan = float("nan")
        return [nan if 0 <= i < len(x) else 0.0 for i in ids], nan, [-1] * k, [nan] * k
    if (x == -np.inf).all():
        return [-np.inf if 0 <= i < len(x) else 0.0 for i in ids], 0.0, [-1] * k, [-np.inf] * k
    y = (x - x.max()) / tau
    c = int((y == 0).sum())
    log_s = math.log(c) + math.log1p(np.exp(y[y < 0]).sum() / c)
    lp = y - log_s
    p = np.exp(lp)
    ent = float(-(p[p > 0] * lp[p > 0]).sum())
    order = sorted(range(len(x)), key=lambda j: (-x[j], j)) if k else []
    top = [j for j in order if x[j] > -np.inf][:k]
    return ([lp[i] if 0 <= i < len(x) else 0.0 for i in ids], ent, top + [-1] * (k - len(top)),
            [lp[j] for j in top] + [-np.inf] * (k - len(top)))
