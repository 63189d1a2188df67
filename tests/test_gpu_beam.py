"""Beam search on the GPU against its definitions (tests/kv8_paged_ref.py): the choice of the next beams, the cache that
follows them, and a search over the 8-bit paged cache with all its calls in a row."""
import numpy as np
import pytest

import llama_decoder_block_fwd_gb300 as L
from synth import BF16
from tests import kv8_paged_ref as R
from tests import serving_ref as S
from tests.helpers import assert_parity, to_f64

pytestmark = pytest.mark.gpu


def _dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def _i32(a):
    return _dev(np.asarray(a, dtype=np.int32))


def _status():
    return L.llama_get_device_status()


def _bdims(B, W):
    return L.dims_of(B, W, 128, 1, 1, 128, 128, 1e4, 1e-5)


# ------------------------------------------------------------------------------------------ select
def _select(z, scores, finished, pad, K, ld=None, shift=0):
    import torch
    B, W = scores.shape
    V = z.shape[-1]
    ld = V if ld is None else ld
    buf = torch.full((B * W * ld + shift + 8,), float("nan"), device="cuda")
    zt = buf[shift:shift + B * W * ld].view(B * W, ld)
    zt[:, :V] = _dev(z.reshape(B * W, V).astype(np.float32))
    par, tok = (torch.full((B, K), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    out = torch.full((B, K), 5.0, device="cuda")
    ws = torch.full((L.llama_workspace_bytes(L.OP_BEAM_SELECT, _bdims(B, W), L.F32, vocab=V),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    L.llama_beam_select(zt, _dev(scores.astype(np.float32)), None if finished is None else _i32(finished), pad, par, tok, out,
                        ws, vocab=V)
    return par.cpu().numpy(), tok.cpu().numpy(), out.cpu().numpy().astype(np.float64)


def _tol(V, s):
    """A score is rounded once (2^-24 of itself); the sum of exponentials is in fp32: 2^-21 of each term and 2^-24 for
    each of the additions in a row (at most V, and 1024 in the long run's partial sums)."""
    return 2.0 ** -24 * np.abs(s) + 2.0 ** -21 + min(V, 1024) * 2.0 ** -24


def _check_select(z, scores, finished, pad, K, got):
    z, scores = z.astype(np.float32), scores.astype(np.float32)
    for b in range(len(scores)):
        want = R.select(z[b], scores[b], None if finished is None else finished[b], pad, K)
        more = R.select(z[b], scores[b], None if finished is None else finished[b], pad, 2 * K + 2)
        by = {(w, t): s for s, w, t in more}
        prev = None
        for k, (s, w, t) in enumerate(want):
            par, tok, out = got[0][b, k], got[1][b, k], got[2][b, k]
            if s == -np.inf:
                assert (par, tok, out) == (-1, -1, -np.inf), (b, k)
                continue
            tol = _tol(z.shape[-1], s)
            assert abs(out - s) <= tol, (b, k, out, s)
            if (par, tok) != (w, t):     # another of (nearly) the same score, of another beam
                assert (par, tok) in by and abs(by[par, tok] - s) <= 2 * tol and by[par, tok] != s, (b, k, par, tok, w, t)
            assert (par, tok) != prev
            prev = (par, tok)


CASES = [(1, 1, 1, 1), (1, 1, 7, 20), (2, 4, 50, 8), (3, 3, 1000, 5), (1, 4, 32000, 4), (2, 8, 128256, 16), (5, 32, 333, 64),
         (1, 32, 4097, 64), (40, 2, 2000, 3), (1, 1, 128256, 64), (170, 3, 600, 6), (7, 5, 9000, 33), (1, 2, 300001, 2)]


@pytest.mark.parametrize("B,W,V,K", CASES)
@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 1), (64, 0)])
def test_select_matches_its_definition(B, W, V, K, pad, shift):
    rng = np.random.default_rng(V + K)
    z = rng.normal(size=(B, W, V)) * 2.5
    scores = -20 - 4 * rng.random((B, W))
    got = _select(z, scores, None, 0, K, ld=V + pad, shift=shift)
    _check_select(z, scores, None, 0, K, got)


def test_select_with_masked_tokens_finished_and_empty_beams():
    rng = np.random.default_rng(7)
    B, W, V, K = 9, 6, 700, 12
    z = rng.normal(size=(B, W, V)) * 3
    z[rng.random(z.shape) < 0.6] = -np.inf
    z[2, 1] = -np.inf                      # no candidate at all
    z[3] = -np.inf
    z[4, :, 5:] = -np.inf
    z[5, 0] = -3e38
    z[6, 2, :] = 3e38
    scores = -5 - 5 * rng.random((B, W))
    scores[1, 1:] = -np.inf
    scores[7] = -np.inf
    finished = (rng.random((B, W)) < 0.3).astype(np.int32)
    finished[0] = 1
    finished[7, 2] = 1                     # finished, and empty
    finished[8] = [0, 1, -1, 0, 1 << 30, 0]
    z[0] = np.nan                          # never read
    got = _select(z, scores, finished, 17, K)
    _check_select(np.where(np.isnan(z), 0.0, z), scores, finished, 17, K, got)


@pytest.mark.parametrize("V", [5, 1000, 40000, 128256])
def test_select_breaks_ties_by_beam_then_token(V):
    W, K = 4, 11
    z = np.zeros((3, W, V))
    z[1] = np.where(np.arange(V) % 3 == 1, 2.0, -1.0)
    z[2] = np.random.default_rng(V).integers(0, 3, size=(V,))      # the same row for every beam
    scores = np.full((3, W), -2.5)
    scores[0, 2] = -2.0
    got = _select(z, scores, None, 0, K)
    for b in range(3):
        want = R.select(z[b].astype(np.float32), scores[b], None, 0, K)
        assert [(int(p), int(t)) for p, t in zip(got[0][b], got[1][b])] == [(w, t) for _, w, t in want], b


def test_select_of_rising_and_falling_rows():
    """Every element beats those before it, or none does; the best all in one place."""
    B, W, V, K = 2, 3, 128256, 40
    x = np.linspace(-9, 9, V)
    z = np.stack([np.stack([x, x[::-1], np.roll(x, V // 2)]), np.stack([np.roll(x, 5), -np.abs(x), np.abs(x)])])
    scores = np.array([[-1.0, -1.25, -1.5], [-3.0, -2.0, -2.5]])
    got = _select(z, scores, None, 0, K)
    _check_select(z, scores, None, 0, K, got)


def test_select_of_sharp_and_far_logits():
    B, W, V, K = 4, 2, 5000, 6
    rng = np.random.default_rng(2)
    z = rng.normal(size=(B, W, V)) * np.array([1e-3, 1.0, 50.0, 1e4])[:, None, None] + np.array([0, 1e4, -1e5, 0])[:, None, None]
    scores = -1e3 * rng.random((B, W))
    scores[0] = [3e30, -3e30]
    got = _select(z, scores, None, 0, K)
    _check_select(z, scores, None, 0, K, got)


def test_select_of_very_many_rows():
    """More rows than every CTA looks through for the ones to read: none left out, finished and empty ones passed over."""
    rng = np.random.default_rng(9)
    B, W, V, K = 900, 20, 37, 5
    z = rng.normal(size=(B, W, V)) * 2
    scores = -10 * rng.random((B, W))
    scores[rng.random((B, W)) < 0.2] = -np.inf
    finished = (rng.random((B, W)) < 0.2).astype(np.int32)
    scores[3], finished[4], finished[5] = -np.inf, 1, 0
    got = _select(z, scores, finished, 2, K)
    some = list(range(0, B, 29)) + [3, 4, 5, B - 1]
    _check_select(z[some], scores[some], finished[some], 2, K, tuple(g[some] for g in got))


def test_select_gives_the_same_bits_again_and_for_equal_rows():
    rng = np.random.default_rng(11)
    row = rng.normal(size=128256) * 2.5
    z = np.broadcast_to(row, (3, 7, 128256))
    scores = np.full((3, 7), -4.0)
    a, b = _select(z, scores, None, 0, 9), _select(z, scores, None, 0, 9, ld=128260)
    for x, y in zip(a, b):
        np.testing.assert_array_equal(x, y)
    # equal beams: each token from every beam in turn
    np.testing.assert_array_equal(a[0][0], [0, 1, 2, 3, 4, 5, 6, 0, 1])
    assert len(set(a[2][0][:7].tolist())) == 1 and len(set(a[1][0][:7].tolist())) == 1


def test_select_captured_and_on_two_streams():
    import torch
    B, W, V, K = 2, 4, 32000, 8
    rng = np.random.default_rng(5)
    dims = _bdims(B, W)
    n = L.llama_workspace_bytes(L.OP_BEAM_SELECT, dims, L.F32, vocab=V)
    sets = []
    for i in range(2):
        t = dict(z=torch.empty(B * W, V, device="cuda"), s=torch.empty(B, W, device="cuda"),
                 par=torch.empty(B, K, dtype=torch.int32, device="cuda"), tok=torch.empty(B, K, dtype=torch.int32, device="cuda"),
                 out=torch.empty(B, K, device="cuda"), ws=torch.empty(n, dtype=torch.uint8, device="cuda"),
                 stream=torch.cuda.Stream())
        call = lambda t=t: L.llama_beam_select(t["z"], t["s"], None, 0, t["par"], t["tok"], t["out"], t["ws"])
        t["z"].zero_(), t["s"].zero_()
        call()
        torch.cuda.synchronize()
        t["g"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(t["g"], stream=t["stream"]):
            call()
        sets.append(t)
    for step in range(3):
        data = [(rng.normal(size=(B, W, V)) * 2, -9 * rng.random((B, W))) for _ in range(2)]
        for t, (z, s) in zip(sets, data):
            t["z"].copy_(_dev(z.reshape(B * W, V).astype(np.float32)))
            t["s"].copy_(_dev(s.astype(np.float32)))
        torch.cuda.synchronize()
        for t in sets:
            with torch.cuda.stream(t["stream"]):
                t["g"].replay()
        torch.cuda.synchronize()
        for t, (z, s) in zip(sets, data):
            _check_select(z, s, None, 0, K, (t["par"].cpu().numpy(), t["tok"].cpu().numpy(), t["out"].cpu().numpy().astype(float)))


# ----------------------------------------------------------------------------------------- reorder
class Beams:
    """Beams of B requests in shuffled pages: prompt pages shared, further full pages shared by some, open pages alone."""

    def __init__(self, B, W, lengths, n_kv=2, hd=64, layers=2, bits=8, seed=0, free=None, share=0.5, P=None):
        import torch
        rng = np.random.default_rng(seed)
        self.B, self.W = B, W
        self.n_cached = np.array([n for row in lengths for n in row], np.int32)
        cols = -(-self.n_cached // 128)
        self.P = int(max(cols.max() if len(cols) else 1, 1)) + 1 if P is None else P
        self.n_pages = int(cols.sum()) + B * W + 3
        ids = [int(x) for x in rng.permutation(self.n_pages)]
        self.table = np.full((B * W, self.P), -3, np.int32)
        for b in range(B):
            for w in range(W):
                s = b * W + w
                for j in range(cols[s]):
                    full = (j + 1) * 128 <= self.n_cached[s]
                    prev = [v for v in range(b * W, s) if (j + 1) * 128 <= self.n_cached[v]]
                    if full and prev and rng.random() < share:
                        self.table[s, j] = self.table[prev[rng.integers(len(prev))], j]
                    else:
                        self.table[s, j] = ids.pop()
        self.free = np.array(ids if free is None else ids[:free], np.int32)
        if bits == 8:
            kv = [rng.integers(0, 255, size=(layers, self.n_pages, 128, n_kv, hd)).astype(np.uint8) for _ in range(2)]
            sc = [rng.random(size=(layers, self.n_pages, n_kv, 128)).astype(np.float32) for _ in range(2)]
        else:
            kv = [rng.integers(-30000, 30000, size=(layers, self.n_pages, 128, n_kv, hd)).astype(np.int16) for _ in range(2)]
            sc = []
        self.kv, self.sc = kv, sc

    def run(self, parents, in_place=False, room=None, ws=None):
        import torch
        kv, sc = [_dev(x) for x in self.kv], [_dev(x) for x in self.sc]
        n, table = _i32(self.n_cached), _i32(self.table)
        n_out, out = (n, table) if in_place else (torch.full_like(n, -9), torch.full_like(table, -4))
        freed = torch.full((self.B * self.W * self.P if room is None else room,), -8, dtype=torch.int32, device="cuda")
        counts = torch.full((2,), -8, dtype=torch.int32, device="cuda")
        if ws is None:
            ws = torch.full((L.llama_workspace_bytes(L.OP_BEAM_REORDER_PAGED, _bdims(self.B, self.W), L.BF16,
                                                     kv_capacity=128 * self.P),), 0xFF, dtype=torch.uint8, device="cuda")
        L.llama_beam_reorder_paged(_i32(parents).view(self.B, self.W), n, n_out, table, out, _i32(self.free), self.n_pages, kv,
                                   sc, freed, counts, ws)
        return n_out, out, freed, counts, kv, sc

    def check(self, parents, got, in_place=False, room=None):
        n_out, out, freed, counts, kv, sc = got
        start = self.table if in_place else np.full_like(self.table, -4)
        wn, wt, wf, taken, moves = R.reorder(parents, self.n_cached, self.table, self.free, self.W, self.n_pages, start)
        np.testing.assert_array_equal(n_out.cpu().numpy(), wn)
        np.testing.assert_array_equal(out.cpu().numpy(), wt)
        assert counts.tolist() == [taken, len(wf)]
        f = freed.tolist()
        wf = wf[:len(f)]
        assert f == wf + [-8] * (len(f) - len(wf))
        kv2, sc2 = [x.copy() for x in self.kv], [x.copy() for x in self.sc]
        for src, dst, rows in moves:
            for x, y in zip(kv2, self.kv):
                x[:, dst, :rows] = y[:, src, :rows]
            for x, y in zip(sc2, self.sc):
                x[:, dst, :, :rows] = y[:, src, :, :rows]
        for got_, want in zip(kv + sc, kv2 + sc2):
            np.testing.assert_array_equal(got_.cpu().numpy(), want)


REORDERS = [
    ([[300, 300, 300, 300]], [[0, 0, 2, 1]]),
    ([[300] * 4], [[3, 3, 3, 3]]),                       # one beam takes all
    ([[300] * 4], [[0, 1, 2, 3]]),                       # nothing moves
    ([[256] * 4], [[1, 1, 0, 2]]),                       # no open page
    ([[127, 0, 0, 0]], [[0, 0, 0, 0]]),                  # a prompt forks: pages from the free list
    ([[0] * 3], [[0, 1, 1]]),
    ([[5] * 2, [129] * 2, [640] * 2], [[1, 1], [0, 0], [1, 0]]),
    ([[300, 200, 100, 400, 128, 1]], [[0, 0, 3, 1, 4, 4]]),   # finished beams of other lengths
    ([[700] * 8, [701] * 8], [[5, 5, 5, 2, 2, 0, 7, 7], [0] * 8]),
    ([[300] * 4, [200] * 4], [[-1, 2, -1, 2], [-1] * 4]),     # empty beams, a request that ends
    ([[1000]], [[0]]),
    ([[1300] * 32], [[(w * w) % 32 for w in range(32)]]),
    ([[128, 100, 128, 100]], [[1, 0, 1, 1]]),            # dead pages do not suffice
]


@pytest.mark.parametrize("case", range(len(REORDERS)))
@pytest.mark.parametrize("bits,n_kv,hd", [(8, 2, 64), (16, 1, 128), (8, 3, 4), (16, 1, 2)])
@pytest.mark.parametrize("in_place", [False, True])
def test_reorder_matches_its_definition(case, bits, n_kv, hd, in_place):
    lengths, parents = REORDERS[case]
    s = Beams(len(lengths), len(lengths[0]), lengths, n_kv, hd, bits=bits, seed=case)
    got = s.run(parents, in_place)
    assert _status() == 0
    s.check(parents, got, in_place)


def test_reorder_of_many_requests_and_long_rows():
    rng = np.random.default_rng(4)
    lengths = [[int(x)] * 4 for x in rng.integers(1, 900, size=300)]
    parents = rng.integers(-1, 4, size=(300, 4)).tolist()
    s = Beams(300, 4, lengths, 1, 16, layers=1, seed=4)
    s.check(parents, s.run(parents))
    assert _status() == 0
    s = Beams(2, 3, [[128 * 700 + 5] * 3, [128 * 300] * 3], 1, 4, layers=1, seed=5, share=0.9)    # more columns than a CTA has threads
    for parents in ([[2, 2, 0], [1, 1, 1]], [[0, 0, 0], [-1, -1, -1]]):
        s.check(parents, s.run(parents))
        assert _status() == 0


@pytest.mark.parametrize("bits,n_kv,hd", [(8, 3, 100), (16, 1, 150), (8, 8, 128), (16, 5, 128)])
@pytest.mark.parametrize("in_place", [False, True])
def test_reorder_of_long_runs_in_many_layers(bits, n_kv, hd, in_place):
    """Ranges that begin and end inside runs of many kilobytes, rows that are not whole vectors (300 bytes), scales beside them."""
    b = Beams(5, 4, [[229, 101, 355, 383], [127] * 4, [130, 1, 2, 200], [128, 256, 77, 77], [250] * 4], n_kv, hd, layers=7, bits=bits,
              seed=hd)
    parents = [[0, 0, 2, 3], [1, 1, 1, 1], [3, 0, 3, 3], [2, 0, 2, 1], [3, 2, 1, 0]]
    got = b.run(parents, in_place)
    assert _status() == 0
    b.check(parents, got, in_place)


def test_reorder_of_open_pages_that_beams_already_share():
    """Beams that start from one prompt with its open page in every row: each but the first gets its own."""
    s = Beams(1, 4, [[300] * 4], seed=2)
    s.table[:] = s.table[0]
    for parents in ([[0, 1, 2, 3]], [[3, 3, 1, 0]]):
        got = s.run(parents)
        assert _status() == 0
        s.check(parents, got)
        assert len(set(got[1][:, 2].tolist())) == 4


def test_reorder_without_pools_and_without_requests():
    import torch
    s = Beams(2, 4, [[300] * 4, [130] * 4], seed=3)
    s.kv, s.sc = [], []
    s.check([[0, 0, 1, 1], [2, 2, 2, 2]], s.run([[0, 0, 1, 1], [2, 2, 2, 2]]))
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    counts = torch.full((2,), -8, dtype=torch.int32, device="cuda")
    t = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    L.llama_beam_reorder_paged(torch.empty(0, 2, dtype=torch.int32, device="cuda"), e, e, t, t, e, 9, [], [], e, counts, None)
    assert _status() == 0 and counts.tolist() == [0, 0]


def test_reorder_latches_what_it_cannot_do():
    lengths, parents = [[300] * 4, [200] * 4], [[0, 0, 0, 0], [1, 1, 1, 1]]
    s = Beams(2, 4, [[300, 0, 0, 0], [200, 300, 300, 300]], seed=6, free=2)
    got = s.run(parents)                                  # three pages wanted, two there
    assert _status() == 1
    s.check(parents, got)
    assert got[1][3, 2] == -1
    s = Beams(2, 4, lengths, seed=6)
    got = s.run(parents, room=1)                          # more dead pages than room to list them
    assert _status() == 1
    s.check(parents, got, room=1)
    bad = [[0, 4, -2, 1], [1, 1, 0, 0]]                   # parents that are none
    got = s.run(bad)
    assert _status() == 1
    s.check(bad, got)
    s.n_cached[1], s.n_cached[6] = -1, 128 * s.P + 1      # lengths that cannot be
    got = s.run(parents)
    assert _status() == 1
    s.check(parents, got)
    s = Beams(2, 4, lengths, seed=6)
    s.table[0, 2], s.table[5, 0] = s.n_pages, -1          # pages outside the pool: an open one, a full one
    got = s.run(parents)
    assert _status() == 1
    s.check(parents, got)
    s = Beams(2, 4, lengths, seed=6)
    s.check(parents, s.run(parents))
    assert _status() == 0


# --------------------------------------------------------------------------- a search, all calls in a row
class Search:
    """A one-layer toy decoder whose K, V and q come from the token alone: what the search keeps per beam is exactly what the
    cache holds, so each step can be checked against the beams' own histories."""

    def __init__(self, B, W, n_q, n_kv, hd, V, prompts, seed=0):
        import torch
        rng = np.random.default_rng(seed)
        self.B, self.W, self.n_q, self.n_kv, self.hd, self.V = B, W, n_q, n_kv, hd, V
        self.qkv = _dev(rng.normal(size=(V, n_q + 2 * n_kv, hd)) * 1.5, torch.bfloat16)
        self.head = _dev(rng.normal(size=(n_q * hd, V)) * 0.15).float()
        self.prompts = [rng.integers(0, V, size=n).tolist() for n in prompts]
        self.P, self.n_pages = -(-(max(prompts) + 200) // 128), 40 * B * W
        dims = self.dims = L.dims_of(B * W, B * W, n_q * hd, n_q, n_kv, hd, 128, 1e4, 1e-5)
        self.one = L.dims_of(B * W, 1, n_q * hd, n_q, n_kv, hd, 128, 1e4, 1e-5)
        self.kc, self.vc = (torch.full((self.n_pages, 128, n_kv, hd), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.ks, self.vs = (torch.full((self.n_pages, n_kv, 128), float("nan"), device="cuda") for _ in range(2))
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
        T = B * W
        self.table, self.n = i32(T, self.P), i32(T)
        self.table.fill_(-1)
        self.cu, self.pos, self.slots, self.used, self.counts = i32(T + 1), i32(T), i32(T), i32(1), i32(2)
        self.par, self.tok, self.sc = i32(B, W), i32(B, W), torch.zeros(B, W, device="cuda")
        self.scores, self.freed = torch.full((B, W), -np.inf, device="cuda"), i32(T * self.P)
        self.scores[:, 0] = 0
        self.ones = i32(T)
        self.ones.fill_(1)
        self.free = list(range(self.n_pages))[::-1]
        self.free_t = i32(64)
        self.x = torch.zeros(T, n_q + 2 * n_kv, hd, dtype=torch.bfloat16, device="cuda")
        self.q, self.o = (torch.zeros(T, n_q, hd, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.logits = torch.zeros(T, V, device="cuda")
        byte = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")
        self.ws_a = byte(L.llama_workspace_bytes(L.OP_GQA_ATTENTION_DECODE_PAGED_KV8, self.one, L.BF16, kv_capacity=128 * self.P))
        self.ws_s = byte(L.llama_workspace_bytes(L.OP_BEAM_SELECT, _bdims(B, W), L.F32, vocab=V))
        self.ws_r = byte(L.llama_workspace_bytes(L.OP_BEAM_REORDER_PAGED, _bdims(B, W), L.BF16, kv_capacity=128 * self.P))

    def prefill(self):
        """The prompts into beam 0 of each request, its attention through pages read back to bf16."""
        import torch
        B, W, n_q, n_kv, hd = self.B, self.W, self.n_q, self.n_kv, self.hd
        T = sum(map(len, self.prompts))
        new = _i32([len(self.prompts[s // W]) if s % W == 0 else 0 for s in range(B * W)])
        cu, used = torch.zeros(B * W + 1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        pos, slots = (torch.zeros(T, dtype=torch.int32, device="cuda") for _ in range(2))
        free = _i32(self.free[::-1])
        L.llama_paged_plan(self.n, new, free, self.n_pages, self.table, cu, pos, slots, used)
        x = self.qkv[_i32([t for p in self.prompts for t in p]).long()]
        dims = L.dims_of(B * W, T, n_q * hd, n_q, n_kv, hd, 128, 1e4, 1e-5)
        q, o = torch.empty(T, n_q, hd, dtype=torch.bfloat16, device="cuda"), torch.empty(T, n_q, hd, dtype=torch.bfloat16, device="cuda")
        L.llama_rope_append_paged_kv8(dims, x[:, :n_q], x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:], pos, slots, q, self.kc, self.ks,
                                      self.vc, self.vs)
        pools = [torch.zeros(self.n_pages, 128, n_kv, hd, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        L.llama_kv_dequantize_paged(self.kc, self.ks, self.vc, self.vs, self.table, new, *pools)
        top = max(map(len, self.prompts)) - 1
        ws = torch.empty(L.llama_workspace_bytes(L.OP_GQA_ATTENTION_CHUNK_PAGED, dims, L.BF16, kv_capacity=top + 1), dtype=torch.uint8,
                         device="cuda")
        L.llama_gqa_attention_chunk_paged(dims, q, *pools, self.table, cu, self.n, top, o, ws)
        self.free = self.free[:len(self.free) - int(used)]
        self.n.copy_(new)
        last = cu[1:].long()[::W] - 1
        self.logits.zero_()
        self.logits[::W] = o[last].float().view(B, -1) @ self.head
        self.qkv_np = to_f64(self.qkv)
        out, qr, at = to_f64(o), to_f64(q), 0
        for b, p in enumerate(self.prompts):         # the chunk attention saw the cache's own values
            k, v = self.cached(b * W, p)
            for i in (0, len(p) // 2, len(p) - 1):
                assert_parity(out[at + i], R.attend(qr[at + i], k[:i + 1], v[:i + 1]), BF16, f"prompt {b}, token {i}")
            at += len(p)

    def cached(self, seq, tokens):
        """K and V values in the pages of a sequence, checked against its tokens: V exactly, K within half a code's step of
        the exact rotation (and 2^-18 of the pair for the fp32 rotation)."""
        row = self.table[seq].cpu().numpy()
        k, v = (R.rows(c.cpu().numpy(), x.cpu().numpy(), row, len(tokens)) for c, x in ((self.kc, self.ks), (self.vc, self.vs)))
        x = self.qkv_np[tokens]
        xk, xv = x[:, self.n_q:self.n_q + self.n_kv], x[:, self.n_q + self.n_kv:]
        kr, ks, xv, vs = R.append(xk, xv, np.arange(len(tokens)), 1e4)
        np.testing.assert_array_equal(v, R.E4M3[R.encode(xv / vs[..., None])] * vs[..., None])
        pair = np.repeat(np.abs(xk[..., 0::2]) + np.abs(xk[..., 1::2]), 2, axis=-1)
        assert np.all(np.abs(k - kr) <= np.maximum(2.0 ** -4 * np.abs(kr), 2.0 ** -10 * ks[..., None]) + 2.0 ** -18 * pair)
        return k, v

    def choose(self):
        L.llama_beam_select(self.logits, self.scores, None, 0, self.par, self.tok, self.sc, self.ws_s)
        L.llama_beam_reorder_paged(self.par, self.n, self.n, self.table, self.table, self.free_t, self.n_pages, [self.kc, self.vc],
                                   [self.ks, self.vs], self.freed, self.counts, self.ws_r)
        self.scores.copy_(self.sc)

    def extend(self, free):
        import torch
        n_q, n_kv = self.n_q, self.n_kv
        L.llama_paged_plan(self.n, self.ones, free, self.n_pages, self.table, self.cu, self.pos, self.slots, self.used)
        torch.index_select(self.qkv, 0, self.tok.view(-1), out=self.x)
        L.llama_rope_append_paged_kv8(self.dims, self.x[:, :n_q], self.x[:, n_q:n_q + n_kv], self.x[:, n_q + n_kv:], self.pos,
                                      self.slots, self.q, self.kc, self.ks, self.vc, self.vs)
        L.llama_gqa_attention_decode_paged_kv8(self.one, self.q, self.kc, self.ks, self.vc, self.vs, self.table, self.pos,
                                               128 * self.P - 1, self.o, self.ws_a)
        self.n.add_(self.ones)
        torch.mm(self.o.view(self.B * self.W, -1).float(), self.head, out=self.logits)

    def give_pages(self):
        n = self.free_t.numel()
        self.free_t.copy_(_i32(self.free[-n:][::-1]))

    def settle(self, used, freed=()):
        """The host's side of the free list: pages taken from its front, dead pages back."""
        self.free = self.free[:len(self.free) - used] + list(freed)


@pytest.mark.parametrize("captured", [False, True])
def test_beam_search_over_the_8_bit_cache(captured):
    import torch
    B, W, V = 2, 4, 300
    s = Search(B, W, 8, 2, 64, V, [130, 57], seed=1)
    s.prefill()
    beams = [[list(p) for _ in range(W)] for p in s.prompts]
    choose, extend = s.choose, lambda: s.extend(s.free_t)
    for step in range(90):
        if captured and step == 2:
            graphs, st = [torch.cuda.CUDAGraph() for _ in range(2)], torch.cuda.Stream()
            for g, call in zip(graphs, (choose, extend)):
                with torch.cuda.graph(g, stream=st):
                    call()
            choose, extend = graphs[0].replay, graphs[1].replay
        z, before = to_f64(s.logits).reshape(B, W, V), to_f64(s.scores)
        s.give_pages()
        choose()
        par, tok, sc = s.par.cpu().numpy(), s.tok.cpu().numpy(), to_f64(s.sc)
        _check_select(z, before, None, 0, W, (par, tok, sc))
        taken, dead = s.counts.tolist()
        s.settle(taken, s.freed[:dead].tolist())
        beams = [[beams[b][par[b, w]] + [int(tok[b, w])] for w in range(W)] for b in range(B)]
        s.give_pages()
        extend()
        s.settle(int(s.used))
        assert _status() == 0
        assert s.n.tolist() == [len(x) for r in beams for x in r]
        if step % 10 in (0, 7) or step < 3:
            out, q = to_f64(s.o), to_f64(s.q)
            for b in range(B):
                for w in range(W):
                    k, v = s.cached(b * W + w, beams[b][w])
                    assert_parity(out[b * W + w], R.attend(q[b * W + w], k, v), BF16, f"step {step}, request {b}, beam {w}")
        held = {p for r, n in zip(s.table.tolist(), s.n.tolist()) for p in r[:-(-n // 128)]}
        assert not held & set(s.free) and len(held) + len(s.free) == s.n_pages and len(set(s.free)) == len(s.free)


@pytest.mark.parametrize("captured", [False, True])
def test_beam_calls_behind_a_wait_on_another_stream(captured):
    """The calls before them have finished early, what they read comes late from another stream: it is waited for."""
    import torch
    rng = np.random.default_rng(31)
    B, W, V, P, n_pages = 3, 4, 9000, 3, 64
    late, first = (_dev(rng.normal(size=(B * W, V)).astype(np.float32)) for _ in range(2))
    scores = torch.zeros(B, W, device="cuda")
    z, zero = torch.zeros_like(late), torch.zeros(B, W, dtype=torch.int32, device="cuda")
    ws = torch.empty(L.llama_workspace_bytes(L.OP_BEAM_SELECT, _bdims(B, W), L.F32, vocab=V), dtype=torch.uint8, device="cuda")
    wr = torch.empty(L.llama_workspace_bytes(L.OP_BEAM_REORDER_PAGED, _bdims(B, W), L.F32, kv_capacity=128 * P),
                     dtype=torch.uint8, device="cuda")
    outs = [[torch.empty(B, W, dtype=t, device="cuda") for t in (torch.int32, torch.int32, torch.float32)] for _ in range(2)]
    n_cached = _i32([200] * (B * W))
    pages = np.full((B * W, P), -1, np.int32)
    for b in range(B):
        for w in range(W):
            pages[b * W + w, :2] = 8 * b, 8 * b + 1 + w
    table, free = _dev(pages), _i32(range(30, n_pages))
    late_parents, parents = _i32([[3, 3, 0, 1], [2, 2, 2, 2], [0, 1, 2, 3]]), zero.clone()
    pool = torch.zeros(n_pages, 128, 1, 16, dtype=torch.uint8, device="cuda")
    got = [(torch.empty_like(n_cached), torch.full_like(table, -7), torch.full_like(n_cached, -7), _i32([0, 0])) for _ in range(2)]
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def calls():
        side.wait_stream(torch.cuda.current_stream())
        L.llama_beam_select(first, scores, None, 0, *outs[0], ws)
        L.llama_beam_select(first, scores, None, 0, *outs[0], ws)
        with torch.cuda.stream(side):
            torch.cuda._sleep(1_000_000)
            z.copy_(late)
        torch.cuda.current_stream().wait_stream(side)
        L.llama_beam_select(z, scores, None, 0, *outs[1], ws)
        with torch.cuda.stream(side):
            torch.cuda._sleep(1_000_000)
            parents.copy_(late_parents)
        torch.cuda.current_stream().wait_stream(side)
        n, t, freed, counts = got[1]
        L.llama_beam_reorder_paged(parents, n_cached, n, table, t, free, n_pages, [pool], [], freed, counts, wr)

    torch.cuda.synchronize()
    with torch.cuda.stream(main):
        calls()
    torch.cuda.synchronize()
    want = [x.clone() for x in (*outs[1], *got[1])]
    _check_select(late.cpu().numpy().reshape(B, W, V), np.zeros((B, W)), None, 0, W,
                  (want[0].cpu().numpy(), want[1].cpu().numpy(), want[2].cpu().numpy().astype(np.float64)))
    assert want[6].tolist() == [0, 0]      # one copy and one dead page, three and three, none
    assert want[4].cpu().numpy()[:, :2].tolist() == [[0, 4], [0, 3], [0, 1], [0, 2], [8, 11], [8, 9], [8, 10], [8, 12],
                                                     [16, 17], [16, 18], [16, 19], [16, 20]]
    g = None
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=main):
            calls()
    for _ in range(5):
        z.zero_(), parents.zero_()
        for t in (*outs[1], *got[1]):
            t.fill_(-7)
        torch.cuda.synchronize()
        with torch.cuda.stream(main):
            g.replay() if captured else calls()
        torch.cuda.synchronize()
        assert _status() == 0
        for x, y in zip((*outs[1], *got[1]), want):
            assert torch.equal(x, y)
