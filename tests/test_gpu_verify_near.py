"""Draft verification where the draft's distribution is close to the target's: the remainder p - q is then a
small difference of nearly equal numbers, and its race is decided by digits that p and q alone do not hold."""
import numpy as np
import pytest

import llama_decoder_block_fwd_gb300 as L
from tests import serving_ref as R

pytestmark = pytest.mark.gpu

# Relative error of a probability: an exponent of at most 40 formed to 2^-24, ex2 2^-22, a sum in a tree of
# depth under 40, the quotient 2^-22.
PROB = 40 * 2.0 ** -24 + 2.0 ** -22 + 40 * 2.0 ** -24 + 2.0 ** -22


def _call(z, y, T, new, tokens, u, noise):
    import torch
    B, N, V = len(new), z.shape[0], z.shape[1]
    d = lambda a, t: None if a is None else torch.from_numpy(np.ascontiguousarray(a.astype(t))).cuda()
    n_acc, out = (torch.full((n,), -9, dtype=torch.int32, device="cuda") for n in (B, N))
    dims = L.dims_of(B, N, 128, 1, 1, 128, 128, 1e4, 1e-5)
    ws = torch.full((L.llama_workspace_bytes(L.OP_VERIFY_DRAFTS, dims, L.F32, vocab=V),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    L.llama_verify_drafts(d(z, np.float32), d(y, np.float32), T, d(np.concatenate([[0], np.cumsum(new)]), np.int32),
                          d(tokens, np.int32), d(u, np.float32), d(noise, np.float32), n_acc, out, ws)
    assert L.llama_get_device_status() == 0
    return n_acc.cpu().numpy(), out.cpu().numpy()


def _refused(B, V, off, seed):
    """B sequences of one draft each, which the target does not allow at all: it is turned down whatever its
    (small) weight in the draft model."""
    rng = np.random.default_rng(seed)
    z = (2.5 * rng.normal(size=(2 * B, V))).astype(np.float32)
    y = (z + off * rng.normal(size=z.shape)).astype(np.float32)
    tokens = rng.integers(0, V, 2 * B)
    z[np.arange(0, 2 * B, 2), tokens[1::2]] = -np.inf
    y[np.arange(0, 2 * B, 2), tokens[1::2]] = -12.0
    return z, y, tokens, np.full(2 * B, 0.5), rng.exponential(size=(B, V)).astype(np.float32)


def _winner(z, y, T, noise):
    """The remainder's winner in 64 bits and whether the stated error leaves no other.  The weight is p (1 - q / p),
    1 - q / p = -expm1(x0 - log R), x0 = (y - z - (max y - max z)) / T, R - 1 = sum p expm1(x0): as p - q, 64 bits
    would leave 2^-53 of p, which of a p near 1 is more than the others' whole remainders.  The weight has p's
    relative error, and x0 - log R is off by a share PROB of what x0 and R are made of where the remainder is
    small beside p, at the winner or at the token of the largest p / noise, by 2 PROB else."""
    z, y = z.astype(np.float64), y.astype(np.float64)
    p = R.softmax(z, T)
    with np.errstate(invalid="ignore"):
        x0 = np.where(p > 0, (y - z - (y.max() - z.max())) / T, 0.0)
    extra = np.exp((y[p == 0] - y.max()) / T).sum() / np.exp((z - z.max()) / T).sum()
    terms = p * np.expm1(x0)
    x = x0 - np.log1p(terms.sum() + extra)
    rest = np.maximum(-p * np.expm1(x), 0.0)
    score = rest / noise
    top = int(np.argmax(score))
    if rest[top] < p[top] / 128 or score[top] < (p / noise).max() / 2 ** 14:
        off = 2 * PROB * (np.abs(x0) + np.abs(terms).sum() + extra)
    else:
        off = 2 * PROB
    err = 2 * PROB * score + np.minimum(off, 1.0) * p / noise
    others = np.delete(score + err, top)
    return top, score[top] - err[top] > others.max()


@pytest.mark.parametrize("off", [1e-6, 1e-5, 1e-4, 1e-3, 0.02, 0.3])
@pytest.mark.parametrize("V,T,B", [(4000, 1.0, 150), (4001, 0.7, 40), (32000, 1.0, 60), (1000, 3.0, 700)])
def test_remainder_of_close_models(V, T, B, off):
    _check_remainders(*_refused(B, V, off, seed=int(V + 1e6 * off)), T)


@pytest.mark.parametrize("shift", [3.0, 0.7, -40.0])
def test_remainder_of_close_models_a_constant_apart(shift):
    z, y, tokens, u, noise = _refused(200, 3000, 0.0, seed=2)
    _check_remainders(z, y + np.float32(shift), tokens, u, noise, 1.0)         # the sums' rounding is all that differs


def _check_remainders(z, y, tokens, u, noise, T):
    B = len(noise)
    n_acc, out = _call(z, y, T, [2] * B, tokens, u, noise)
    assert (n_acc == 0).all()
    want = [_winner(z[2 * b], y[2 * b], T, noise[b].astype(np.float64)) for b in range(B)]
    clear = [b for b in range(B) if want[b][1]]
    assert len(clear) >= 0.9 * B
    wrong = [(b, want[b][0], int(out[2 * b])) for b in clear if out[2 * b] != want[b][0]]
    assert not wrong, f"{len(wrong)} of {len(clear)}: {wrong[:4]}"


@pytest.mark.parametrize("shift", [0.0, 1.0, -64.0])
def test_models_that_differ_by_a_constant(shift):
    """Logits that differ by a constant are one distribution: nothing remains, and the token is drawn from p."""
    B, V = 30, 3000
    rng = np.random.default_rng(3)
    z = (np.round(rng.normal(size=(2 * B, V)) * 2.5 * 1024) / 1024).astype(np.float32)
    tokens = rng.integers(0, V, 2 * B)
    z[np.arange(0, 2 * B, 2), tokens[1::2]] = -np.inf
    y, u, noise = z + np.float32(shift), np.full(2 * B, 0.5), rng.exponential(size=(B, V)).astype(np.float32)
    n_acc, out = _call(z, y, 1.0, [2] * B, tokens, u, noise)
    assert (n_acc == 0).all()
    for b in range(B):
        score = R.softmax(z[2 * b], 1.0) / noise[b].astype(np.float64)
        best = np.sort(score)[-2:]
        if best[1] > best[0] * (1 + 4 * PROB):
            assert out[2 * b] == int(np.argmax(score))


@pytest.mark.parametrize("T", [1.0, 0.3, 2.5])
@pytest.mark.parametrize("drafts", [True, False])
def test_drafts_of_weights_below_the_least_normal_number(T, drafts):
    """Whether u q < p does not depend on how small both are, nor u = 0 on how small p is."""
    B, V = 400, 50
    rng = np.random.default_rng(5)
    z = rng.normal(size=(2 * B, V)).astype(np.float32)
    y = rng.normal(size=(2 * B, V)).astype(np.float32)
    tokens, u = rng.integers(0, V, 2 * B), rng.random(2 * B).astype(np.float32)
    low = rng.uniform(60, 300, B).astype(np.float32) * np.float32(T)
    row, d = np.arange(0, 2 * B, 2), tokens[1::2]
    z[row, d], y[row, d] = -low, -low + T * rng.normal(size=B).astype(np.float32)
    u[row[::5]] = 0.0
    off = np.arange(0, B, 9)                                 # not allowed by the target, nor (some) by the draft
    z[row[off], d[off]] = rng.choice([-np.inf, np.finfo(np.float32).min], off.size)
    y[row[off[::2]], d[off[::2]]] = np.finfo(np.float32).min
    noise = rng.exponential(size=(B, V)).astype(np.float32)
    n_acc, _ = _call(z, y if drafts else None, T, [2] * B, tokens, u, noise)
    compared = 0
    for b in range(B):
        r = 2 * b
        want, _, margin = R.verify(z[r:r + 2], y[r:r + 2] if drafts else None, T, tokens[r:r + 2], u[r:r + 2], noise[b])
        # exponents of up to 440 (300 / ln 2) formed to 2^-24 on both sides, besides the rest
        if u[r] == 0 or margin > 2 * (440 * 2.0 ** -24 + PROB):
            compared += 1
            assert n_acc[b] == want, (b, float(low[b]), float(u[r]))
    assert compared > 0.95 * B


@pytest.mark.parametrize("gap", [8.0, 14.0, 18.0, 30.0])
@pytest.mark.parametrize("off", [1e-3, 0.3])
def test_remainder_beside_a_token_of_almost_all_weight(gap, off):
    """p and q of one token near 1: the rounding of its p - q is larger than the other tokens' p - q, so that
    their race alone would not tell whether the remainder is theirs or its."""
    B, V = 300, 60
    z, y, tokens, u, noise = _refused(B, V, off, seed=int(gap))
    peak = np.random.default_rng(1).integers(0, V, 2 * B)
    peak[tokens[1::2].repeat(2) == peak] += 1
    peak %= V
    r = np.arange(2 * B)
    z[r, peak] = y[r, peak] = gap + 6.0
    y[np.arange(0, 2 * B, 2), tokens[1::2]] = np.where(np.arange(B) % 2, -12.0, 2.0)   # the draft's share of q
    n_acc, out = _call(z, y, 1.0, [2] * B, tokens, u, noise)
    assert (n_acc == 0).all()
    want = [_winner(z[2 * b], y[2 * b], 1.0, noise[b].astype(np.float64)) for b in range(B)]
    clear = [b for b in range(B) if want[b][1]]
    assert len(clear) >= 0.5 * B
    wrong = [(b, want[b][0], int(out[2 * b])) for b in clear if out[2 * b] != want[b][0]]
    assert not wrong, f"{len(wrong)} of {len(clear)}: {wrong[:4]}"


def test_close_models_late_in_a_long_sequence():
    """The refused row lies behind the rows whose merged statistics are kept."""
    V, n, B = 2000, 70, 12
    rng = np.random.default_rng(9)
    z = (2.5 * rng.normal(size=(B * n, V))).astype(np.float32)
    y = (z + 1e-5 * rng.normal(size=z.shape)).astype(np.float32)
    tokens, u = rng.integers(0, V, B * n), np.full(B * n, 0.5)
    stop = rng.integers(30, n - 1, B)
    for b in range(B):
        row = b * n + stop[b]
        z[row, tokens[row + 1]], y[row, tokens[row + 1]] = -np.inf, -12.0
    noise = rng.exponential(size=(B, V)).astype(np.float32)
    n_acc, out = _call(z, y, 1.0, [n] * B, tokens, u, noise)
    assert n_acc.tolist() == stop.tolist()
    want = [_winner(z[b * n + stop[b]], y[b * n + stop[b]], 1.0, noise[b].astype(np.float64)) for b in range(B)]
    assert sum(w[1] for w in want) >= B - 1
    assert all(out[b * n + stop[b]] == w[0] for b, w in enumerate(want) if w[1])


def test_close_and_other_models_in_one_captured_call():
    """One graph, replayed with models that are close in some sequences and not in others, and with none of either;
    two such graphs in flight at once.  Replays of the same inputs agree."""
    import torch
    B, V = 90, 3000
    far, near = _refused(B, V, 0.5, seed=1), _refused(B, V, 1e-5, seed=2)
    dims = L.dims_of(B, 2 * B, 128, 1, 1, 128, 128, 1e4, 1e-5)
    cu = torch.arange(0, 2 * B + 1, 2, dtype=torch.int32, device="cuda")
    runs = []
    for _ in range(2):
        z, y = (torch.empty((2 * B, V), device="cuda") for _ in range(2))
        tokens, u = torch.empty(2 * B, dtype=torch.int32, device="cuda"), torch.full((2 * B,), 0.5, device="cuda")
        noise = torch.ones((B, V), device="cuda")
        z.normal_(), y.copy_(z), tokens.fill_(1)
        n_acc, out = (torch.full((n,), -9, dtype=torch.int32, device="cuda") for n in (B, 2 * B))
        ws = torch.empty(L.llama_workspace_bytes(L.OP_VERIFY_DRAFTS, dims, L.F32, vocab=V), dtype=torch.uint8, device="cuda")
        st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=st):
            L.llama_verify_drafts(z, y, 1.0, cu, tokens, u, noise, n_acc, out, ws)
        runs.append((z, y, tokens, noise, n_acc, out, st, g, ws))
    for turn in range(3):
        mixes = []
        for k, (z, y, tokens, noise, *_) in enumerate(runs):
            pick = np.arange(B) % 3 == turn if k == 0 else np.full(B, turn == 1)
            rows = pick.repeat(2)[:, None]
            mix = [np.where(r, a, b) for r, a, b in ((rows, near[0], far[0]), (rows, near[1], far[1]),
                                                     (rows[:, 0], near[2], far[2]), (pick[:, None], near[4], far[4]))]
            for dst, a in zip((z, y, tokens, noise), mix):
                dst.copy_(torch.from_numpy(np.ascontiguousarray(a)))
            mixes.append(mix)
        results = []
        for _ in range(3):
            torch.cuda.synchronize()
            for run in runs:
                with torch.cuda.stream(run[6]):
                    run[7].replay()
            torch.cuda.synchronize()
            results.append([(run[4].clone(), run[5].clone()) for run in runs])
        assert L.llama_get_device_status() == 0
        assert all(torch.equal(a, b) for again in results[1:] for x, w in zip(results[0], again) for a, b in zip(x, w))
        for (z, y, _, noise), (n_acc, out) in zip(mixes, results[0]):
            assert (n_acc == 0).all()
            out = out.cpu().numpy()
            for b in range(B):
                top, clear = _winner(z[2 * b], y[2 * b], 1.0, noise[b].astype(np.float64))
                assert not clear or out[2 * b] == top
