"""Plain 64-bit (numpy) and integer definitions of the paged serving step, for its tests."""
from __future__ import annotations

import numpy as np

PAGE = 128


def plan(n_cached, n_new, free_pages, table, n_tokens):
    """(table, cu, positions, slots, pages used), token by token."""
    table = table.copy()
    cu, pos, slots, used = [0], [], [], 0
    for b, (c, n) in enumerate(zip(n_cached, n_new)):
        for j in range(-(-c // PAGE), -(-(c + n) // PAGE)):
            table[b, j] = free_pages[used]
            used += 1
        for p in range(c, c + n):
            pos.append(p)
            slots.append(int(table[b, p // PAGE]) * PAGE + p % PAGE)
        cu.append(cu[-1] + n)
    pad = [-1] * (n_tokens - len(pos))
    return (table, np.array(cu, np.int32), np.array(pos + pad, np.int32), np.array(slots + pad, np.int32), used)


def rotate(x, positions, theta):
    """RoPE of x [T, heads, hd] at a position per token (interleaved pairs)."""
    hd = x.shape[-1]
    ang = positions.astype(np.float64)[:, None] * theta ** (-np.arange(0, hd, 2) / hd)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    a, b = x[..., 0::2], x[..., 1::2]
    out = np.empty(x.shape)
    out[..., 0::2] = a * c - b * s
    out[..., 1::2] = a * s + b * c
    return out


def attention(q, k, v, past):
    """q [n, n_q, hd] at positions past.. over k, v [past + n, n_kv, hd]; keys a query does not see do
    not enter its sums at all."""
    n, n_q, hd = q.shape
    r = n_q // k.shape[1]
    out = np.empty((n, n_q, hd))
    for i in range(n):
        m = past + i + 1
        for h in range(n_q):
            s = k[:m, h // r] @ q[i, h] / np.sqrt(hd)
            w = np.exp(s - s.max())
            out[i, h] = w @ v[:m, h // r] / w.sum()
    return out


def softmax(z, T):
    z = z.astype(np.float64) / T
    w = np.exp(z - z.max())
    return w / w.sum()


def verify(z, y, T, tokens, u, noise):
    """One sequence: (accepted, out tokens, margin).  margin is the smallest relative distance of any
    comparison on the way to the value it is compared with (an fp32 evaluation may differ only there)."""
    n = z.shape[0]
    out, margin = [-1] * n, np.inf
    for i in range(n):
        if T <= 0:
            out[i] = int(np.argmax(z[i]))
            if i < n - 1 and out[i] == tokens[i + 1]:
                continue
            return i, out, margin
        p = softmax(z[i], T)
        w = p
        if i < n - 1:
            d = int(tokens[i + 1])
            if y is None:
                q = np.zeros_like(p)
                if 0 <= d < len(p):
                    q[d] = 1.0
            else:
                q = softmax(y[i], T)
            if 0 <= d < len(p):
                lhs, rhs = u[i] * q[d], p[d]
                if lhs != rhs:
                    margin = min(margin, abs(lhs - rhs) / max(lhs, rhs))
                if lhs < rhs:
                    out[i] = d
                    continue
            w = np.maximum(p - q, 0.0)
            if w.sum() <= 0:
                w = p
        race = w / noise.astype(np.float64)
        out[i] = int(np.argmax(race))
        if len(race) > 1:
            top = np.sort(race)[-2:]
            margin = min(margin, (top[1] - top[0]) / top[1])
        return i, out, margin
    raise AssertionError("a sequence has at least one row")
