"""Plain 64-bit forms of the operators on committed tokens and drafts (include/gdnreplay.h gdn_replay_advance,
gdnlayer.h gdn_conv_advance, gdnattn.h gdn_attn_chunk, gdndraft.h), written from their definitions, and the
bounds of their tests.  numpy on the CPU."""
from __future__ import annotations

import numpy as np


def advance(S, q, k, v, g, beta, scale):
    """S [H, dv, dk], q, k [n, Hk, dk], v [n, H, dv], g, beta [n, H].  Returns out [n, H, dv], the state after the
    last token, and what the bounds need: the largest norm of a state's row on the way (with the update's), and the most that
    steps' errors of 1 add up to, max_t e_t with e_t = alpha_t e_{t-1} + 1."""
    H = S.shape[0]
    rep = H // k.shape[1]
    out, norm, e, eff = [], np.sqrt((S * S).sum(-1)).max(), np.zeros(H), 1.0
    for t in range(len(q)):
        kt, qt = (np.repeat(x[t], rep, 0) for x in (k, q))
        a = np.exp(g[t])
        S = a[:, None, None] * S
        w = beta[t][:, None] * (v[t] - np.einsum("hij,hj->hi", S, kt))
        S = S + w[:, :, None] * kt[:, None]
        out.append(np.einsum("hij,hj->hi", S, qt) * scale)
        norm = max(norm, np.sqrt((S * S).sum(-1)).max(), np.abs(v[t]).max())
        e = a * e + 1
        eff = max(eff, e.max())
    return np.array(out).reshape(len(q), H, S.shape[1]), S, norm, eff


def advance_bound(norm, eff, dk, chunked):
    """Bound on the absolute error of a state's element (an output's: times |q| scale).

    A step alpha S (I - beta k k^T) + beta v k^T does not lengthen a difference by more than alpha (|k| = 1 up to
    its rounding), so errors of steps add up to eff times the largest.  Token by token, a step's is that of two sums of dk
    products and a few roundings, each 2^-24 of the norms: (dk + 8) 2^-24 norm.  Chunked: the products of 64 tokens with
    S, with x and of E and MP take operands of three bf16 terms each, which are exact; left out of a product of two such
    operands are its parts of the third order, 2 * 2^-7 * 2^-14 of the norms, in E x, in (MP) x and in MP itself; the
    sums, rows of up to dk + 64 summands in fp32 (2^-23: added without rounding to nearest), lie on S's path and on
    the update's: 2^-18 + (dk + 64) 2^-22 of the norms, once per chunk and so at most once per step."""
    step = 2.0 ** -18 + (dk + 64) * 2.0 ** -22 if chunked else (dk + 8) * 2.0 ** -24
    return 1.01 * eff * step * norm + 1e-30


def conv(window, x, weight, bias, silu):
    """window [W - 1, D] (oldest first), x [n, D].  Returns y [n, D], the new window and sum_j |w_j x_j| + |bias|."""
    W, n = weight.shape[1], len(x)
    z = np.concatenate([window, x])
    y = np.zeros_like(x) + bias
    mag = np.abs(bias) + np.zeros_like(x)
    for j in range(W):
        y = y + z[j:j + n] * weight[:, j]
        mag = mag + np.abs(z[j:j + n] * weight[:, j])
    if silu:
        with np.errstate(over="ignore"):
            y = y / (1 + np.exp(-y))
    return y, z[n:], mag


def sample(tokens, parent, probs, draft, u, n):
    """One sequence: the accepted tokens' numbers, the next token and how near the draw or an accept came to a
    border (relative)."""
    if n == 0:
        return [], -1, 1.0
    V = probs.shape[-1]
    cur, path, near = 0, [0], 1.0
    r, m = np.maximum(probs[0], 0), 1.0
    for t in range(1, n):
        if parent[t] != cur or not m > 0:
            continue
        x = tokens[t]
        q = draft[cur] if draft is not None else (np.arange(V) == x) * 1.0
        a, b = u[t] * q[x] * m, r[x]
        if a != b:
            near = min(near, abs(a - b) / max(abs(a), abs(b)))
        if a < b:
            cur, r, m = t, np.maximum(probs[t], 0), 1.0
            path.append(t)
        else:
            if draft is None:
                m -= r[x]
                r = np.where(np.arange(V) == x, 0.0, r)
            else:
                r = np.maximum(r - m * q, 0)
                m = r.sum()
    if not r.sum() > 0:
        r = np.maximum(probs[cur], 0)
    s = np.cumsum(r)
    if not 0 < s[-1] < np.inf:
        return path, -1, near
    hit = np.flatnonzero(s > u[0] * s[-1])
    nxt = int(hit[0]) if len(hit) else int(np.flatnonzero(r > 0)[-1])
    d = np.abs(s - u[0] * s[-1])
    d = d[(d > 0) & (r > 0)]
    return path, nxt, min(near, d.min() / s[-1] if len(d) else 1.0)
