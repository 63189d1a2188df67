"""Beam selection on the GPU: scores and order to the error that the header states, rows where that error is largest, and very
many rows of whole vectors."""
import os
import re

import numpy as np
import pytest

from tests import kv8_paged_ref as R
from tests.test_gpu_beam import _select, _status

pytestmark = pytest.mark.gpu

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "llama_block.h")


def _stated(V):
    """The header's figure: the error of a score before out_scores rounds it.  It comes from: the exponent z - m, rounded, and its
    product with log2(e), 2.23 * 2^-24 of the distance, whose mean under the softmax is at most ln V (12.01 for 163840: 26.8);
    two exponentials of 2^-22 (8); 25 additions in a row (25), a product of 2^-24 among them; the logarithm (0.5): 60.3 * 2^-24.
    Each further 163840 logits are one more step of the join, an exponential, a product and a sum (6), and ln V grows."""
    text = " ".join(open(HEADER).read().replace("\n * ", " ").split())
    text = text[text.index("The n_out best continuations of each request"):text.index("int llama_beam_select(")]
    bits = re.search(r"scores good to (?:about )?2\^-(\d+)", text)
    more = re.search(r"2\^-(\d+) more for each 163840 beyond", text)
    return 2.0 ** -int(bits.group(1)) + (2.0 ** -int(more.group(1)) * -(-max(0, V - 163840) // 163840) if more else 0.0)


def _check(z, scores, K, got):
    """Every score within the stated error, every choice among those whose scores lie within twice it of the definition's, beams'
    own candidates in the order of their logits, none twice."""
    z, scores = z.astype(np.float32), scores.astype(np.float32)
    for b in range(len(scores)):
        eps = _stated(z.shape[-1])
        want = R.select(z[b], scores[b], None, 0, K)
        by = {}
        for w in range(z.shape[1]):
            by.update({(w, t): s for s, _, t in R.select(z[b, w:w + 1], scores[b, w:w + 1], None, 0, K)})
        par, tok, out = (g[b] for g in got)
        pairs = list(zip(par.tolist(), tok.tolist()))
        assert len(set(pairs)) == K
        for k, (s, w, t) in enumerate(want):
            mine = by[pairs[k]]                        # (a beam's K best hold all that it can give)
            assert abs(out[k] - mine) <= eps + 2.0 ** -24 * abs(mine), (b, k, out[k], mine, abs(out[k] - mine) / eps)
            assert abs(mine - s) <= 2 * eps, (b, k, pairs[k], (w, t))
        for w in range(z.shape[1]):
            mine = [t for p, t in pairs if p == w]
            order = np.lexsort((np.arange(z.shape[-1]), -z[b, w].astype(np.float64)))
            assert mine == order[:len(mine)].tolist()


@pytest.mark.parametrize("V", [1000, 32000, 128256, 163840])
@pytest.mark.parametrize("gap", [0.0, 3.0, 8.37, 9.6, 10.1, 11.77, 12.4])
def test_scores_of_one_peak_over_a_flat_row(V, gap):
    """Equal logits `gap` below one: the rounding of their exponent is the same for all."""
    W, K = 4, 6
    z = np.zeros((1, W, V))
    for w in range(W):
        z[0, w, 13 + 1000 * w % V] = gap * (1 + w / 97)
    got = _select(z, np.array([[-1.0, -1.5, -2.0, -0.25]]), None, 0, K)
    assert _status() == 0
    _check(z, np.array([[-1.0, -1.5, -2.0, -0.25]]), K, got)


@pytest.mark.parametrize("V,std", [(5000, 1.0), (128256, 2.5), (128256, 0.01), (128256, 6.0), (50257, 4.0), (1000003, 2.0)])
def test_scores_of_spread_rows(V, std):
    rng = np.random.default_rng(V)
    W, K = 8, 16
    z, scores = rng.normal(size=(2, W, V)) * std, -20 - 4 * rng.random((2, W))
    got = _select(z, scores, None, 0, K)
    assert _status() == 0
    _check(z, scores, K, got)


def test_scores_of_rising_blocks():
    """The maximum moves from batch to batch, so that the sums are carried over at each."""
    V, W, K = 163840, 2, 9
    x = np.arange(V) // 640 * (14.0 / 256) + np.random.default_rng(1).normal(size=(1, W, V)) * 0.1
    got = _select(x, np.array([[-3.0, -3.5]]), None, 0, K)
    assert _status() == 0
    _check(x, np.array([[-3.0, -3.5]]), K, got)


def test_very_many_rows_of_whole_vectors():
    """More rows than every CTA looks through, of two batches each, by bulk copies; some finished, some empty."""
    rng = np.random.default_rng(3)
    B, W, V, K = 825, 20, 5200, 5
    z = rng.standard_normal(size=(B, W, V), dtype=np.float32) * 2
    scores = -10 * rng.random((B, W))
    scores[rng.random((B, W)) < 0.2] = -np.inf
    finished = (rng.random((B, W)) < 0.2).astype(np.int32)
    scores[3], finished[4] = -np.inf, 1
    par, tok, out = _select(z, scores, finished, 2, K)
    assert _status() == 0
    eps = _stated(V)
    s32 = scores.astype(np.float32)
    for b in list(range(0, B, 23)) + [3, 4, B - 1]:
        want = R.select(z[b], s32[b], finished[b], 2, K)
        for k, (s, w, t) in enumerate(want):
            if s == -np.inf:
                assert (par[b, k], tok[b, k], out[b, k]) == (-1, -1, -np.inf)
            else:
                assert abs(out[b, k] - s) <= 3 * eps + 2.0 ** -24 * abs(s)        # (another within twice the error)
        near = [abs(x[0] - y[0]) <= 2 * eps for x, y in zip(want, want[1:]) if y[0] > -np.inf]
        if not any(near):
            # equal but where the K-th and the next are as near
            assert [(int(p), int(t)) for p, t in zip(par[b], tok[b])][:-1] == [(w, t) for _, w, t in want][:-1]
