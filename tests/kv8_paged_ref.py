"""Plain 64-bit (numpy) and integer definitions of the 8-bit paged cache and of beam search, for their tests."""
from __future__ import annotations

import numpy as np

from tests.serving_ref import PAGE, rotate

# every E4M3 ("e4m3fn") value by its code: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7F is NaN
_c = np.arange(128)
_mag = np.where(_c >> 3 == 0, (_c & 7) * 2.0 ** -9, (1 + (_c & 7) / 8) * 2.0 ** ((_c >> 3) - 7.0))
_mag[127] = np.nan
E4M3 = np.concatenate([_mag, -_mag])


def encode(x):
    """E4M3 codes of x: to nearest, ties to the even code, saturating; NaN to 0x7F."""
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    hi = np.clip(np.searchsorted(_mag[:127], a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dh, dl = _mag[hi] - a, a - _mag[lo]
    with np.errstate(invalid="ignore"):
        code = np.where(a >= 448, 126, np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi))
    code = np.where(np.isnan(x), 127, code)
    return (code + 128 * np.signbit(x)).astype(np.uint8)


def row_scale(u):
    """The smallest 2^e, e in -100 .. 100, with u <= 448 * 2^e."""
    u = np.asarray(u, np.float64)
    e = np.full(u.shape, -100)
    for _ in range(200):
        e = np.where((u > 448 * 2.0 ** e) & (e < 100), e + 1, e)
    return 2.0 ** e


def k_bound(k):
    return np.max(np.abs(k[..., 0::2]) + np.abs(k[..., 1::2]), -1)


def append(k, v, positions, theta):
    """(rotated K, its scales, V, its scales): values before rounding, scales [T, n_kv]."""
    return rotate(k, positions, theta), row_scale(k_bound(k)), v, row_scale(np.max(np.abs(v), -1))


def rows(codes, scales, table_row, n):
    """Values [n, n_kv, hd] of positions 0 .. n-1 of a sequence."""
    pos = np.arange(n)
    page = table_row[pos // PAGE]
    return E4M3[codes[page, pos % PAGE]] * scales[page, :, pos % PAGE].astype(np.float64)[..., None]


def attend(q, k, v):
    """q [n_q, hd] over k, v [n, n_kv, hd]; zeros without keys."""
    n_q, hd = q.shape
    out = np.zeros((n_q, hd))
    if len(k) == 0:
        return out
    r = n_q // k.shape[1]
    for h in range(n_q):
        s = k[:, h // r] @ q[h] / np.sqrt(hd)
        w = np.exp(s - s.max())
        out[h] = w @ v[:, h // r] / w.sum()
    return out


def select(z, scores, finished, pad, n_out):
    """One request: [(score, beam, token)] of the n_out best; fewer candidates: (-inf, -1, -1).  Candidates of one beam
    differ by their logits, whatever a large score leaves of that in 64 bits."""
    found = []
    for w in range(len(scores)):
        if scores[w] == -np.inf:
            continue
        if finished is not None and finished[w]:
            found.append((float(scores[w]), w, 0.0, pad))
            continue
        x = z[w].astype(np.float64)
        live = np.nonzero(x > -np.inf)[0]
        if len(live) == 0:
            continue
        m = x[live].max()
        s = float(scores[w]) + ((x[live] - m) - np.log(np.sum(np.exp(x[live] - m))))
        order = np.argsort(-x[live], kind="stable")[:n_out]
        found += [(float(s[i]), w, -float(x[live[i]]), int(live[i])) for i in order]
    found.sort(key=lambda f: (-f[0], *f[1:]))
    found = [(s, w, t) for s, w, _, t in found[:n_out]]
    return found + [(-np.inf, -1, -1)] * (n_out - len(found))


def reorder(parents, n_cached, table, free, W, n_pages, table_out=None):
    """(n_cached_out, table_out, freed, pages taken, moves [(source, destination, rows)]); with too few free pages the
    entry is -1 and the move is left out."""
    B = len(parents)
    P = table.shape[1]
    out = (table if table_out is None else table_out).copy()
    n_out, freed, moves, taken = [], [], [], 0
    for b in range(B):
        n = [c if 0 <= c <= PAGE * P else 0 for c in n_cached[b * W:b * W + W]]
        par = [p if -1 <= p < W else -1 for p in parents[b]]
        old = table[b * W:b * W + W]
        kept = sorted({p for p in par if p >= 0})
        dead = []
        for j in range(P):
            stay = {int(old[p, j]) for p in kept if j * PAGE < n[p]}
            for p in range(W):
                page = int(old[p, j])
                if j * PAGE < n[p] and 0 <= page < n_pages and page not in stay and page not in dead:
                    dead.append(page)
        ends, ncopy = [], 0
        for w, p in enumerate(par):
            n_out.append(n[p] if p >= 0 else 0)
            if p < 0:
                continue
            for j in range(-(-n[p] // PAGE)):
                page = int(old[p, j])
                if j == n[p] // PAGE:
                    if page in ends:
                        src, page = page, -1
                        if ncopy < len(dead):
                            page = dead[ncopy]
                        else:
                            if taken < len(free):
                                page = int(free[taken])
                            taken += 1
                        ncopy += 1
                        if not 0 <= src < n_pages or not 0 <= page < n_pages:
                            page = -1
                        else:
                            moves.append((src, page, n[p] % PAGE))
                    else:
                        ends.append(page)
                out[b * W + w, j] = page
        freed += dead[ncopy:]
    return np.array(n_out, np.int32), out, freed, taken, moves
