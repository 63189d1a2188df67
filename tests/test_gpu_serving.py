"""The paged serving step on the GPU against its 64-bit definitions (tests/serving_ref.py): planning,
RoPE and the write into pages, attention of packed chunks, verification of drafts, and the four in a
row as a step uses them."""
import numpy as np
import pytest

import llama_decoder_block_fwd_gb300 as L
from tests import serving_ref as R
from tests.helpers import BF16_TOL, assert_parity, to_f64
from synth import BF16

pytestmark = pytest.mark.gpu
THETA = 5e5


def _dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def _i32(a):
    return _dev(np.asarray(a, dtype=np.int32).reshape(-1))


def _status():
    return L.llama_get_device_status()


# ------------------------------------------------------------------------------------------ plan
def _plan_inputs(cached, new, seed=0, extra=3):
    rng = np.random.default_rng(seed)
    have = [-(-c // 128) for c in cached]
    need = [-(-(c + n) // 128) for c, n in zip(cached, new)]
    P = max(need + [1]) + 1
    n_pages = sum(need) + extra
    ids = rng.permutation(n_pages).astype(np.int32)
    table = np.full((len(cached), P), -7, np.int32)
    k = 0
    for b, h in enumerate(have):
        table[b, :h] = ids[k:k + h]
        k += h
    return table, ids[k:], n_pages


def _run_plan(cached, new, free, n_pages, table, T):
    import torch
    t = dict(table=_dev(table), cu=torch.full((len(cached) + 1,), -9, dtype=torch.int32, device="cuda"),
             pos=torch.full((T,), -9, dtype=torch.int32, device="cuda"),
             slots=torch.full((T,), -9, dtype=torch.int32, device="cuda"),
             used=torch.full((1,), -9, dtype=torch.int32, device="cuda"))
    L.llama_paged_plan(_i32(cached), _i32(new), _i32(free), n_pages, t["table"], t["cu"], t["pos"], t["slots"],
                       t["used"])
    return t


PLANS = [([0], [1]), ([127], [2]), ([128], [1]), ([5, 0, 300, 128], [0, 0, 129, 128]), ([0, 0], [0, 0]),
         ([1000] * 5, [1, 5, 0, 700, 1]), (list(range(0, 7000, 7)), [b % 4 for b in range(1000)]),
         (list(range(8192)), [(b * 37) % 3 for b in range(8192)]), ([30720], [9000])]


@pytest.mark.parametrize("case", range(len(PLANS)))
@pytest.mark.parametrize("pad", [0, 37])
def test_plan_matches_its_definition(case, pad):
    cached, new = PLANS[case]
    table, free, n_pages = _plan_inputs(cached, new, seed=case)
    T = sum(new) + pad
    want = R.plan(cached, new, free, table, T)
    got = _run_plan(cached, new, free, n_pages, table, T)
    assert _status() == 0
    for name, w in zip(("table", "cu", "pos", "slots"), want):
        np.testing.assert_array_equal(got[name].cpu().numpy(), w, err_msg=name)
    assert int(got["used"]) == want[4]


def test_plan_with_no_sequences():
    import torch
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    cu, used = (torch.full((1,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    pos, slots = (torch.full((3,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    L.llama_paged_plan(e, e, e, 4, torch.empty(0, 2, dtype=torch.int32, device="cuda"), cu, pos, slots, used)
    assert _status() == 0
    assert cu.tolist() == [0] and used.tolist() == [0] and pos.tolist() == slots.tolist() == [-1] * 3


def test_plan_latches_what_it_cannot_plan():
    cached, new = [100, 0, 250], [60, 3, 10]
    table, free, n_pages = _plan_inputs(cached, new)
    T = sum(new)
    want = R.plan(cached, new, free, table, T)
    # a negative length: that sequence brings nothing, the others are planned
    got = _run_plan([100, -1, 250], new, free, n_pages, table, T)
    assert _status() == 1 and got["cu"].tolist() == [0, 60, 60, 70]
    got = _run_plan(cached, [60, 1 << 30, 10], free, n_pages, table, T)     # longer than its table row
    assert _status() == 1 and got["cu"].tolist() == [0, 60, 60, 70]
    # one page too few: the tokens that lack it get no slot
    got = _run_plan(cached, new, free[:want[4] - 1], n_pages, table, T)
    assert _status() == 1 and int(got["used"]) == want[4]
    lost = [s for s, w in zip(got["slots"].tolist(), want[3]) if s != w]
    assert lost and all(s == -1 for s in lost)
    # more tokens than rows
    got = _run_plan(cached, new, free, n_pages, table, T - 5)
    assert _status() == 1 and got["cu"].tolist() == [0, 60, 63, T - 5]
    np.testing.assert_array_equal(got["slots"].cpu().numpy(), want[3][:T - 5])
    # a page id outside the pool
    bad = table.copy()
    bad[2, 1] = n_pages
    got = _run_plan(cached, new, free, n_pages, bad, T)
    assert _status() == 1 and got["slots"].tolist()[63:69] == [-1] * 6
    got = _run_plan(cached, new, free, n_pages, table, T)                     # and the next call is clean
    assert _status() == 0


# ---------------------------------------------------------------------------------------- append
def _assert_rotated(got, x, positions, what):
    """bf16 of a cos - b sin: half a step of the result, plus what the angle is off by: its reduction
    (two constants, at most 6e-11 per turn) and the fp32 sine and cosine (2^-20 in all)."""
    ref = R.rotate(x, positions, THETA)
    pair = np.abs(x[..., 0::2]) + np.abs(x[..., 1::2])
    off = 2.0 ** -19 + positions.astype(np.float64)[:, None, None] * 1e-11
    tol = 2.0 ** -8 * np.abs(ref) + np.repeat(pair * off, 2, axis=-1)
    assert np.all(np.abs(got - ref) <= tol), (what, float(np.max(np.abs(got - ref) / tol)))


@pytest.mark.parametrize("T,n_q,n_kv,hd,first", [(1, 32, 8, 128, 0), (5, 8, 2, 64, 131), (300, 32, 8, 128, 131000),
                                                 (1000, 28, 4, 128, 8000), (7, 3, 3, 8, 40), (9, 5, 1, 256, 3),
                                                 (700, 2, 1, 72, 77), (2500, 8, 8, 64, 400000)])
@pytest.mark.parametrize("fused", [True, False])
def test_append_rotates_and_writes_pages(T, n_q, n_kv, hd, first, fused):
    import torch
    rng = np.random.default_rng(T)
    x = _dev(rng.normal(size=(T, n_q + 2 * n_kv, hd)), torch.bfloat16)
    parts = (x[:, :n_q], x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:])
    q, k, v = parts if fused else [p.contiguous() for p in parts]
    n_pages = -(-T // 128) + 4
    kp = _dev(rng.normal(size=(n_pages, 128, n_kv, hd)), torch.bfloat16)
    vp = _dev(rng.normal(size=(n_pages, 128, n_kv, hd)), torch.bfloat16)
    before = kp.clone(), vp.clone()
    positions = (first + np.arange(T)).astype(np.int32)
    slots = rng.permutation(n_pages * 128)[:T].astype(np.int32)
    dead = rng.random(T) < 0.2 if T > 1 else np.zeros(1, bool)
    slots[dead] = -1
    qo = torch.full((T, n_q, hd), 9.0, dtype=torch.bfloat16, device="cuda")
    dims = L.dims_of(1, T, 128, n_q, n_kv, hd, 128, THETA, 1e-5)
    L.llama_rope_append_paged(dims, q, k, v, _i32(positions), _i32(slots), qo, kp, vp)
    assert _status() == 0
    live = ~dead
    xh = to_f64(x)
    _assert_rotated(to_f64(qo)[live], xh[live, :n_q], positions[live], "q")
    assert (to_f64(qo)[dead] == 9.0).all()
    flat = to_f64(kp).reshape(-1, n_kv, hd)
    _assert_rotated(flat[slots[live]], xh[live, n_q:n_q + n_kv], positions[live], "k")
    flat_v = to_f64(vp).reshape(-1, n_kv, hd)
    np.testing.assert_array_equal(flat_v[slots[live]], xh[live, n_q + n_kv:])
    other = np.setdiff1d(np.arange(n_pages * 128), slots[live])
    np.testing.assert_array_equal(flat[other], to_f64(before[0]).reshape(-1, n_kv, hd)[other])
    np.testing.assert_array_equal(flat_v[other], to_f64(before[1]).reshape(-1, n_kv, hd)[other])


def test_append_in_place_and_by_halves():
    """q rotated in place, q alone and k/v alone give what one call gives."""
    import torch
    T, n_q, n_kv, hd = 33, 8, 2, 64
    rng = np.random.default_rng(8)
    q, k, v = (_dev(rng.normal(size=(T, h, hd)), torch.bfloat16) for h in (n_q, n_kv, n_kv))
    pos, slots = _i32(rng.integers(0, 5000, T)), _i32(rng.permutation(256)[:T])
    dims = L.dims_of(1, T, 128, n_q, n_kv, hd, 128, THETA, 1e-5)
    pools = [torch.zeros((2, 128, n_kv, hd), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    qo, alone, inplace = torch.empty_like(q), torch.empty_like(q), q.clone()
    L.llama_rope_append_paged(dims, q, k, v, pos, slots, qo, pools[0], pools[1])
    L.llama_rope_append_paged(dims, q, None, None, pos, slots, alone, None, None)
    L.llama_rope_append_paged(dims, None, k, v, pos, slots, None, pools[2], pools[3])
    L.llama_rope_append_paged(dims, inplace, None, None, pos, slots, inplace, None, None)
    assert _status() == 0
    assert torch.equal(qo, alone) and torch.equal(qo, inplace)
    assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])


def test_append_skips_rows_outside_the_pool():
    import torch
    T, n_kv, hd = 6, 2, 64
    k = torch.ones((T, n_kv, hd), dtype=torch.bfloat16, device="cuda")
    dims = L.dims_of(1, T, 128, 2, n_kv, hd, 128, THETA, 1e-5)
    for pos, slots, live in (([0] * 6, [0, 256, 5, 1 << 30, 7, -5], [0, 5, 7]),
                             ([0, -1, 1 << 24, 0, 0, 0], [1, 2, 3, 4, 5, 6], [1, 4, 5, 6])):
        kp, vp = (torch.zeros((2, 128, n_kv, hd), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        L.llama_rope_append_paged(dims, None, k, k, _i32(pos), _i32(slots), None, kp, vp)
        assert _status() == 1
        assert torch.nonzero(vp.view(-1, n_kv * hd).sum(-1)).flatten().tolist() == live


# ------------------------------------------------------------------------------------- attention
class Batch:
    """Sequences in pages scattered over a pool whose unused rows are NaN."""

    def __init__(self, cached, new, n_q, n_kv, hd, seed=0, pad=0, q_std=1.0):
        import torch
        rng = np.random.default_rng(seed)
        self.cached, self.new, self.heads = cached, new, (n_q, n_kv, hd)
        B, need = len(cached), [-(-(c + n) // 128) for c, n in zip(cached, new)]
        self.n_pages = sum(need) + 3
        ids = rng.permutation(self.n_pages).astype(np.int32)
        table = np.full((B, max(need + [1])), ids[-1], np.int32)
        self.kp = torch.full((self.n_pages, 128, n_kv, hd), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.vp = self.kp.clone()
        self.k, self.v, at = [], [], 0
        for b, (c, n) in enumerate(zip(cached, new)):
            pages = ids[at:at + need[b]]
            table[b, :need[b]] = pages
            at += need[b]
            kk = torch.from_numpy(rng.normal(size=(c + n, n_kv, hd)).astype(np.float32)).bfloat16()
            vv = torch.from_numpy(rng.normal(size=(c + n, n_kv, hd)).astype(np.float32)).bfloat16()
            self.k.append(kk)
            self.v.append(vv)
            if c + n:
                rows = torch.from_numpy((pages[:, None].astype(np.int64) * 128 + np.arange(128)).reshape(-1)[:c + n]).cuda()
                self.kp.view(-1, n_kv, hd)[rows] = kk.cuda()
                self.vp.view(-1, n_kv, hd)[rows] = vv.cuda()
        self.T = sum(new)
        self.q = torch.from_numpy((q_std * rng.normal(size=(self.T + pad, n_q, hd))).astype(np.float32)).bfloat16()
        if pad:
            self.q[self.T:] = float("nan")
        self.table, self.cu = table, np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.max_pos = max([c + n for c, n in zip(cached, new)] + [1]) - 1
        self.dims = L.dims_of(B, self.T + pad, 128, n_q, n_kv, hd, 128, THETA, 1e-5)

    def run(self, slack=0, stream=None):
        import torch
        o = torch.full(tuple(self.q.shape), 7.0, dtype=torch.bfloat16, device="cuda")
        ws = torch.full((L.llama_workspace_bytes(L.OP_GQA_ATTENTION_CHUNK_PAGED, self.dims, L.BF16,
                                                 kv_capacity=self.max_pos + 1 + slack),), 0xFF, dtype=torch.uint8,
                        device="cuda")
        table = self.table
        if slack:
            table = np.pad(table, ((0, 0), (0, -(-slack // 128))), constant_values=-1)
        L.llama_gqa_attention_chunk_paged(self.dims, self.q.cuda(), self.kp, self.vp, _dev(table), _i32(self.cu),
                                          _i32(self.cached), self.max_pos + slack, o, ws, stream)
        return o

    def check(self, o, every=1):
        n_q, n_kv, hd = self.heads
        got = to_f64(o)
        assert (got[self.T:] == 7.0).all()
        for b, (c, n) in enumerate(zip(self.cached, self.new)):
            if n == 0:
                continue
            lo = self.cu[b]
            rows = sorted({0, n - 1, *range(0, n, every)})
            k, v, q = (t.double().numpy() for t in (self.k[b], self.v[b], self.q[lo:lo + n]))
            ref = np.concatenate([R.attention(q[i:i + 1], k[:c + i + 1], v[:c + i + 1], c + i) for i in rows])
            assert_parity(got[lo + np.array(rows)], ref, BF16, f"seq {b}: {n} after {c}")


CHUNKS = [([0], [1], 4, 1, 64), ([0], [1], 32, 8, 128), ([5], [3], 8, 2, 128), ([127], [1], 8, 2, 64), ([127], [2], 8, 2, 64),
          ([128], [1], 8, 8, 128), ([200, 0, 1, 1000], [5, 1, 0, 3], 32, 8, 128), ([0, 0, 0], [0, 7, 0], 8, 2, 64),
          ([0], [129], 8, 2, 128), ([100], [300], 8, 2, 64), ([333], [777], 4, 4, 128), ([0, 40, 2000], [256, 33, 5], 32, 8, 128),
          ([77, 3], [100, 61], 28, 4, 128), ([400], [50], 6, 2, 64), ([50, 130], [9, 200], 16, 1, 64), ([60], [40], 128, 1, 128),
          ([10], [4], 100, 1, 64), ([5000], [1], 8, 1, 128), ([9000, 100], [2, 2], 8, 1, 64), ([0] * 40, list(range(40)), 8, 2, 64),
          ([0], [700], 1, 1, 64), ([130] * 3, [64, 65, 63], 2, 1, 128)]


@pytest.mark.parametrize("case", range(len(CHUNKS)))
def test_chunk_attention(case):
    cached, new, n_q, n_kv, hd = CHUNKS[case]
    b = Batch(cached, new, n_q, n_kv, hd, seed=case, pad=case % 3)
    o = b.run(slack=(0, 1, 4000)[case % 3])
    assert _status() == 0
    b.check(o, every=1 if b.T * (max(cached) + 300) * n_q < 1e6 else 37)


@pytest.mark.parametrize("n_q,n_kv,hd", [(32, 8, 128), (8, 8, 64)])
@pytest.mark.parametrize("kind", ["lone", "pairs", "both"])
def test_chunk_attention_many_units_per_sm(kind, n_q, n_kv, hd):
    """More work units than SMs, of many key tiles each: every CTA walks from unit to unit, between
    lone Q tiles and pairs."""
    rng = np.random.default_rng(len(kind))
    B = 40
    cached = [int(c) for c in rng.integers(0, 4000, B)]
    tile = 128 // (n_q // n_kv)
    few = [int(n) for n in rng.integers(1, min(tile, 6) + 1, B)]
    many = [int(n) for n in rng.integers(tile + 1, 3 * tile, B)]
    new = {"lone": few, "pairs": many, "both": [few[b] if b % 2 else many[b] for b in range(B)]}[kind]
    b = Batch(cached, new, n_q, n_kv, hd, seed=B)
    o = b.run()
    assert _status() == 0
    b.check(o, every=97)


def test_chunk_attention_long_and_mixed():
    """One long prompt chunk among short decodes, and sharp rows (scores of +-100)."""
    b = Batch([3000, 20, 7000, 1], [1, 1500, 4, 1], 32, 8, 128, seed=5, q_std=8.0)
    o = b.run()
    assert _status() == 0
    b.check(o, every=211)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("cached,new", [(0, 200), (150, 40), (700, 3)])
def test_chunk_attention_unseen_values_do_not_reach_a_query(cached, new, bad, hd):
    """A key and a value that are not finite reach exactly the queries that see them."""
    import torch
    b = Batch([cached], [new], 8, 2, hd, seed=3)
    at = cached + new // 2
    page, row = int(b.table[0, at // 128]), at % 128
    kp, vp = b.kp.clone(), b.vp.clone()
    clean = b.run()
    b.vp[page, row, 1, 5] = bad
    got = b.run()
    assert _status() == 0
    sees = slice(at - cached, None)
    same = torch.ones(clean.shape, dtype=torch.bool)
    same[sees, 4:, 5] = False
    same = same.cuda()
    assert torch.equal(got[same], clean[same])
    hit = got[~same].float()
    assert (torch.isnan(hit) if bad != bad else hit == bad).all()
    b.vp = vp
    b.kp[page, row, 0, 9] = bad
    got = b.run()
    assert torch.equal(got[:at - cached], clean[:at - cached]) and torch.equal(got[:, 4:], clean[:, 4:])
    b.kp = kp


@pytest.mark.parametrize("hd", [64, 128])
def test_chunk_attention_unseen_values_in_every_unit(hd):
    """Units follow each other on an SM, each with a value that is not finite in its last tiles."""
    import torch
    rng = np.random.default_rng(hd)
    new = [int(n) for n in rng.integers(129, 256, 250)]
    b = Batch([0] * len(new), new, 8, 8, hd, seed=4)
    clean = b.run()
    bad = torch.zeros(b.q.shape, dtype=torch.bool)
    for i, n in enumerate(new):
        at = int(rng.integers(0, n))
        b.vp[int(b.table[i, at // 128]), at % 128, :, i % hd] = float("inf")
        bad[b.cu[i] + at:b.cu[i + 1], :, i % hd] = True
    got = b.run()
    assert _status() == 0
    bad = bad.cuda()
    assert torch.equal(got[~bad], clean[~bad]) and bool((got[bad] == float("inf")).all())


@pytest.mark.parametrize("B,seed", [(1500, 0), (2600, 1)])
def test_chunk_attention_many_sequences(B, seed):
    """More sequences than the shapes that are kept on the chip, most of them without new tokens or short."""
    rng = np.random.default_rng(seed)
    cached = [int(c) for c in rng.integers(0, 200, B)]
    new = [int(n) for n in rng.integers(0, 4, B)]
    cached[B // 2], new[B // 2], new[-1] = 3000, 90, 5
    b = Batch(cached, new, 4, 2, 64, seed=seed)
    o = b.run()
    assert _status() == 0
    b.check(o, every=7)


@pytest.mark.parametrize("n_q,n_kv,hd", [(100, 1, 64), (128, 1, 128), (42, 2, 128), (5, 5, 64)])
def test_chunk_attention_head_layouts_over_many_units(n_q, n_kv, hd):
    rng = np.random.default_rng(n_q)
    cached, new = [int(c) for c in rng.integers(0, 1500, 24)], [int(n) for n in rng.integers(0, 60, 24)]
    b = Batch(cached, new, n_q, n_kv, hd, seed=n_q)
    o = b.run()
    assert _status() == 0
    b.check(o, every=19)


def test_chunk_attention_shares_pages_between_sequences():
    """Two sequences over one prefix: the first pages of both are the same pages."""
    b = Batch([384, 384], [5, 70], 8, 2, 128, seed=11)
    b.table[1, :3] = b.table[0, :3]
    b.k[1][:384], b.v[1][:384] = b.k[0][:384], b.v[0][:384]
    o = b.run()
    assert _status() == 0
    b.check(o)


def test_chunk_attention_reports_pages_outside_the_pool():
    for wrong in (-1, 1 << 20):
        b = Batch([300, 200], [4, 130], 8, 2, 64, seed=2)
        b.table[0, 1] = wrong
        o = b.run()
        assert _status() == 1
        b.cached[0], b.new[0] = 0, 0                                     # the other sequence is right
        got = to_f64(o)
        k, v, q = (t.double().numpy() for t in (b.k[1], b.v[1], b.q[4:]))
        assert_parity(got[4:], R.attention(q, k, v, 200), BF16, "seq 1")
    b = Batch([300], [4], 8, 2, 64)
    b.max_pos = 300                                                       # the last token is at 303
    b.run()
    assert _status() == 1
    b = Batch([300], [4], 8, 2, 64)
    assert _status() == 0
    b.check(b.run())


def test_pools_past_2_to_the_31_elements():
    """The last pages of pools of 2.4e9 elements: append writes them and attention reads them."""
    import torch
    n_pages, n_q, n_kv, hd, c, n = 18400, 32, 8, 128, 130, 5
    rng = np.random.default_rng(3)
    kp, vp = (torch.empty((n_pages, 128, n_kv, hd), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = np.array([[n_pages - 1, n_pages - 3]], np.int32)
    x = _dev(rng.normal(size=(c + n, n_q + 2 * n_kv, hd)), torch.bfloat16)
    pos = np.arange(c + n)
    slots = table[0, pos // 128].astype(np.int64) * 128 + pos % 128
    dims = L.dims_of(1, c + n, 128, n_q, n_kv, hd, 128, THETA, 1e-5)
    q = torch.empty((c + n, n_q, hd), dtype=torch.bfloat16, device="cuda")
    L.llama_rope_append_paged(dims, x[:, :n_q], x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:], _i32(pos), _i32(slots), q, kp, vp)
    dims = L.dims_of(1, n, 128, n_q, n_kv, hd, 128, THETA, 1e-5)
    o, q = torch.empty((n, n_q, hd), dtype=torch.bfloat16, device="cuda"), q[c:].contiguous()
    ws = torch.empty(L.llama_workspace_bytes(L.OP_GQA_ATTENTION_CHUNK_PAGED, dims, L.BF16, kv_capacity=c + n),
                     dtype=torch.uint8, device="cuda")
    L.llama_gqa_attention_chunk_paged(dims, q, kp, vp, _dev(table), _i32([0, n]), _i32([c]), c + n - 1, o, ws)
    assert _status() == 0
    at = torch.from_numpy(slots).cuda()
    k, v = to_f64(kp.view(-1, n_kv, hd)[at]), to_f64(vp.view(-1, n_kv, hd)[at])
    _assert_rotated(k, to_f64(x)[:, n_q:n_q + n_kv], pos, "k")
    assert np.array_equal(v, to_f64(x)[:, n_q + n_kv:])
    assert_parity(to_f64(o), R.attention(to_f64(q), k, v, c), BF16, "far pages")


def test_packed_rows_past_2_to_the_31_elements():
    """q and o of 2.2e9 elements: 540 sequences of 1000 tokens, 32 heads over one KV head."""
    import torch
    B, n, n_q, n_kv, hd = 540, 1000, 32, 1, 128
    gen = torch.Generator("cuda").manual_seed(1)
    kp, vp = (torch.randn((8 * B, 128, n_kv, hd), generator=gen, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.empty((B * n, n_q, hd), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    o = torch.full_like(q, 7.0)
    table = torch.arange(8 * B, dtype=torch.int32, device="cuda").view(B, 8)
    dims = L.dims_of(B, B * n, 128, n_q, n_kv, hd, 128, THETA, 1e-5)
    ws = torch.empty(L.llama_workspace_bytes(L.OP_GQA_ATTENTION_CHUNK_PAGED, dims, L.BF16, kv_capacity=n),
                     dtype=torch.uint8, device="cuda")
    cu = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
    L.llama_gqa_attention_chunk_paged(dims, q, kp, vp, table, cu, torch.zeros(B, dtype=torch.int32, device="cuda"), n - 1, o, ws)
    assert _status() == 0
    for b in (0, 270, B - 1):
        k, v = (to_f64(t[8 * b:8 * b + 8]).reshape(-1, n_kv, hd) for t in (kp, vp))
        for i in (0, 500, n - 1):
            ref = R.attention(to_f64(q[b * n + i:b * n + i + 1]), k[:i + 1], v[:i + 1], i)
            assert_parity(to_f64(o[b * n + i:b * n + i + 1]), ref, BF16, f"seq {b}, token {i}")


def test_calls_on_a_given_stream():
    """The stream argument, from outside any stream context."""
    import torch
    b = Batch([300, 7], [20, 3], 8, 2, 64, seed=31)
    want = b.run()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = b.run(stream=st)
    torch.cuda.synchronize()
    assert _status() == 0 and torch.equal(got, want)


def test_chunk_attention_agrees_with_the_decode_call():
    import torch
    b = Batch([900, 17, 2048], [1, 1, 1], 32, 8, 128, seed=21)
    o = b.run()
    dims = L.dims_of(3, 1, 128, 32, 8, 128, 128, THETA, 1e-5)
    ws = torch.empty(L.llama_workspace_bytes(L.OP_GQA_ATTENTION, dims, L.BF16, kv_capacity=b.max_pos + 1),
                     dtype=torch.uint8, device="cuda")
    one = torch.empty_like(o)
    L.llama_gqa_attention_decode_paged(dims, b.q.cuda(), b.kp, b.vp, _dev(b.table), _i32(b.cached), b.max_pos, one, ws)
    assert _status() == 0
    # each side is within the bar of the exact value, so the two are within twice the bar of each other
    assert_parity(to_f64(o).reshape(-1, 128), to_f64(one).reshape(-1, 128), BF16, tol=2 * BF16_TOL)


# ---------------------------------------------------------------------------------------- verify
def _verify(z, y, T, new, tokens, u, noise, strided=0):
    import torch
    B, N = len(new), len(tokens)
    pad = (lambda a: None if a is None else torch.nn.functional.pad(_dev(a), (0, strided), value=50.0)[:, :a.shape[1]])
    n_acc = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    out = torch.full((N,), -9, dtype=torch.int32, device="cuda")
    V = z.shape[1]
    dims = L.dims_of(B, max(N, 1), 128, 1, 1, 128, 128, THETA, 1e-5)
    ws = torch.full((L.llama_workspace_bytes(L.OP_VERIFY_DRAFTS, dims, L.F32, vocab=V),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    L.llama_verify_drafts(pad(z), pad(y), T, _i32(np.concatenate([[0], np.cumsum(new)])), _i32(tokens),
                          None if u is None else _dev(u), pad(noise), n_acc, out, ws)
    return n_acc.cpu().numpy(), out.cpu().numpy()


def _verify_inputs(new, V, seed, spread=2.5, off=0.6, pad=0):
    rng = np.random.default_rng(seed)
    N = sum(new) + pad
    z = (spread * rng.normal(size=(N, V))).astype(np.float32)
    y = (z + off * rng.normal(size=(N, V))).astype(np.float32)
    tokens = np.array([int(np.argmax(y[max(t - 1, 0)] - np.log(rng.exponential(size=V)))) for t in range(N)], np.int32)
    return z, y, tokens, rng.random(N).astype(np.float32), rng.exponential(size=(len(new), V)).astype(np.float32)


# A comparison is decided as in 64 bits unless its two sides are closer than this: an exponent of at
# most 40 formed to 2^-24 (40 * 2^-24 of the weight), ex2 2^-22, a sum of 2^17 terms in a tree of depth
# under 40 (40 * 2^-24), the quotient 2^-22, on both sides.
NEAR = 2 * (40 * 2.0 ** -24 + 2.0 ** -22 + 40 * 2.0 ** -24 + 2.0 ** -22)


def _check_verify(got, z, y, T, new, tokens, u, noise):
    n_acc, out = got
    at = 0
    for b, n in enumerate(new):
        if n == 0:
            assert n_acc[b] == 0
            continue
        w = R.verify(z[at:at + n], None if y is None else y[at:at + n], T, tokens[at:at + n], u[at:at + n], noise[b])
        if w[2] > NEAR:
            assert n_acc[b] == w[0] and out[at:at + n].tolist() == w[1], (b, n_acc[b], w, out[at:at + n])
        at += n
    assert (out[at:] == -9).all()


@pytest.mark.parametrize("V", [1, 2, 50, 8191, 8192, 8197, 32000, 128256])
@pytest.mark.parametrize("T", [0.0, 0.7, 1.0, 5.0])
@pytest.mark.parametrize("drafts", [True, False])
def test_verify_matches_its_definition(V, T, drafts):
    new = [1, 4, 0, 9, 2, 5] if V > 10000 else [1, 4, 0, 9, 2, 5] * 9
    z, y, tokens, u, noise = _verify_inputs(new, V, seed=V, pad=2)
    y = y if drafts else None
    for strided in (0, 3):
        got = _verify(z, y, T, new, tokens, u, noise, strided)
        assert _status() == 0
        _check_verify(got, z, y, T, new, tokens, u, noise)


def test_verify_masked_logits_and_equal_models():
    V, new = 1000, [3] * 16
    for low in (-np.inf, np.finfo(np.float32).min):
        z, y, tokens, u, noise = _verify_inputs(new, V, seed=4)
        rng = np.random.default_rng(1)
        z[rng.random(z.shape) < 0.6] = low
        y[rng.random(y.shape) < 0.3] = low
        z[:, 17], y[:, 17] = 1.0, 1.0
        z[5], y[5] = low, low
        z[5, 3], y[5, 3] = 0.5, -2.0                       # a single token left
        for T in (0.0, 0.8):
            got = _verify(z, y, T, new, tokens, u, noise)
            assert _status() == 0
            _check_verify(got, z, y, T, new, tokens, u, noise)
            got = _verify(z, None, T, new, tokens, u, noise)
            _check_verify(got, z, None, T, new, tokens, u, noise)
    z, y, tokens, u, noise = _verify_inputs(new, V, seed=6, off=0.0)      # equal models: every draft stands
    n_acc, out = _verify(z, y, 1.0, new, tokens, np.full_like(u, 0.99999994), noise)
    assert (n_acc == 2).all()
    z[:] = 0.0                                              # ties: the lowest id
    n_acc, out = _verify(z, None, 0.0, new, np.zeros_like(tokens), u, noise)
    assert (n_acc == 2).all() and (out == 0).all()
    noise[:] = 1.0
    n_acc, out = _verify(z, z, 1.0, new, tokens, u, noise)
    assert (n_acc == 2).all() and (out.reshape(-1, 3)[:, 2] == 0).all()


def test_verify_long_sequences_and_many():
    """More rows than the statistics that are kept on the chip, and more sequences than CTAs per cluster."""
    for new, V in (([70, 1, 33, 34, 40], 3000), ([2] * 700, 60)):
        z, y, tokens, u, noise = _verify_inputs(new, V, seed=8, off=0.02)
        for d in (y, None):
            got = _verify(z, d, 1.0, new, tokens, u, noise)
            assert _status() == 0
            _check_verify(got, z, d, 1.0, new, tokens, u, noise)
    new, tokens = [70, 1, 33, 34, 40], np.full(178, 7, np.int32)
    z, y, _, u, noise = _verify_inputs(new, 3000, seed=8)
    z[:, 7], y[:, 7] = 60.0, 60.0                           # no doubt: every draft stands, however many
    n_acc, out = _verify(z, y, 1.0, new, tokens, u, noise)
    assert n_acc.tolist() == [n - 1 for n in new] and (out == 7).all()
    z[50, 9], y[50, 9] = 200.0, 0.0                         # the 51st row wants another token
    n_acc, out = _verify(z, y, 1.0, new, tokens, u, noise)
    assert n_acc.tolist() == [50, 0, 32, 33, 39] and out[50] == 9 and (out[51:70] == -1).all() and (out[70:] == 7).all()


@pytest.mark.parametrize("V,new", [(128256, [5, 0, 3, 1, 4] * 7), (32003, [4, 1, 2, 0, 0, 9, 40, 3] * 4), (1000, [3] * 2500),
                                   (5000, [0] * 300 + [70, 1] * 30 + [0] * 5), (151936, [66])])
@pytest.mark.parametrize("T", [0.0, 0.8])
@pytest.mark.parametrize("drafts", [True, False])
def test_verify_large_batches(V, new, T, drafts):
    """Rows by the hundred, empty sequences in a row, vocabularies that end inside a part."""
    z, y, tokens, u, noise = _verify_inputs(new, V, seed=len(new), off=0.2, pad=1)
    y = y if drafts else None
    for strided in (0, 1):
        got = _verify(z, y, T, new, tokens, u, noise, strided)
        assert _status() == 0
        _check_verify(got, z, y, T, new, tokens, u, noise)


def test_verify_large_batch_with_nothing_remaining():
    """Equal models, a draft of weight 0 in both, in every sequence of a large batch."""
    V, new = 20000, [3] * 120
    z, y, tokens, u, noise = _verify_inputs(new, V, seed=15, off=0.0)
    tokens[1::3] = 40
    z[:, 40] = y[:, 40] = -np.inf
    got = _verify(z, y, 1.0, new, tokens, u, noise)
    assert _status() == 0 and (got[0] == 0).all()
    _check_verify(got, z, y, 1.0, new, tokens, u, noise)


def test_verify_large_batches_captured_and_on_two_streams():
    """Two calls in flight at once, each captured and replayed with other inputs."""
    import torch
    V, runs = 30011, []
    for seed, new in enumerate(([4] * 70, [2, 9, 0, 1] * 30)):
        z, y, tokens, u, noise = _verify_inputs(new, V, seed=20 + seed)
        t = [_dev(z), _dev(y), _i32(np.concatenate([[0], np.cumsum(new)])), _i32(tokens), _dev(u), _dev(noise)]
        n_acc, out = (torch.full((n,), -9, dtype=torch.int32, device="cuda") for n in (len(new), sum(new)))
        dims = L.dims_of(len(new), sum(new), 128, 1, 1, 128, 128, THETA, 1e-5)
        ws = torch.full((L.llama_workspace_bytes(L.OP_VERIFY_DRAFTS, dims, L.F32, vocab=V),), 0xFF, dtype=torch.uint8,
                        device="cuda")
        st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=st):
            L.llama_verify_drafts(t[0], t[1], 0.9, t[2], t[3], t[4], t[5], n_acc, out, ws)
        runs.append((new, t, n_acc, out, st, g, ws))
    for turn in range(3):
        inputs = []
        for seed, (new, t, _, _, _, _, _) in enumerate(runs):
            z, y, tokens, u, noise = _verify_inputs(new, V, seed=30 + 10 * turn + seed)
            for dst, a in zip((t[0], t[1], t[3], t[4], t[5]), (z, y, tokens, u, noise)):
                dst.copy_(torch.from_numpy(a))
            inputs.append((z, y, tokens, u, noise))
        torch.cuda.synchronize()
        for _, _, _, _, st, g, _ in runs:
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        assert _status() == 0
        for (new, _, n_acc, out, _, _, _), (z, y, tokens, u, noise) in zip(runs, inputs):
            _check_verify((n_acc.cpu().numpy(), out.cpu().numpy()), z, y, 0.9, new, tokens, u, noise)


def test_verify_extreme_temperatures():
    V, new = 500, [3] * 12
    z, y, tokens, u, noise = _verify_inputs(new, V, seed=12)
    z[:, ::3] = -np.inf
    flat = lambda a: np.where(np.isfinite(a), 0.0, -np.inf).astype(np.float32)
    for d in (y, None):
        got = _verify(z, d, float("inf"), new, tokens, u, noise)          # every token that is left alike
        assert _status() == 0
        _check_verify(got, flat(z), None if d is None else flat(d), 1.0, new, tokens, u, noise)
        for T in (1e-30, 1e-38, 1e-42):                                   # the argmax
            got = _verify(z, d, T, new, tokens, u, noise)
            assert _status() == 0
            _check_verify(got, z, d, T, new, tokens, u, noise)


def test_verify_draft_that_neither_model_allows():
    """Equal models, a draft of weight 0 in both: turned down with nothing in the remainder, so the new token is
    drawn from p."""
    V, new = 900, [2, 3]
    z, y, tokens, u, noise = _verify_inputs(new, V, seed=13, off=0.0)
    tokens[1] = tokens[3] = 40
    z[:, 40] = y[:, 40] = -np.inf
    got = _verify(z, y, 1.0, new, tokens, u, noise)
    assert _status() == 0 and got[0].tolist() == [0, 0] and 0 <= got[1][0] < V and got[1][0] != 40
    _check_verify(got, z, y, 1.0, new, tokens, u, noise)


def test_verify_uses_the_first_vocab_columns():
    import torch
    V, new = 700, [3, 1, 4]
    z, y, tokens, u, noise = _verify_inputs(new, V + 9, seed=17)
    tokens = np.minimum(tokens, V - 1)
    z[:, V:], noise[:, V:] = 50.0, 1e-9                      # what stands behind them would win
    n_acc, out = (torch.full((k,), -9, dtype=torch.int32, device="cuda") for k in (3, 8))
    dims = L.dims_of(3, 8, 128, 1, 1, 128, 128, THETA, 1e-5)
    ws = torch.empty(L.llama_workspace_bytes(L.OP_VERIFY_DRAFTS, dims, L.F32, vocab=V), dtype=torch.uint8, device="cuda")
    L.llama_verify_drafts(_dev(z), _dev(y), 1.0, _i32([0, 3, 4, 8]), _i32(tokens), _dev(u), _dev(noise), n_acc, out, ws,
                          vocab=V)
    assert _status() == 0
    _check_verify((n_acc.cpu().numpy(), out.cpu().numpy()), z[:, :V], y[:, :V], 1.0, new, tokens, u, noise[:, :V])


def test_verify_without_rows():
    n_acc, out = _verify(np.zeros((0, 5), np.float32), None, 1.0, [0, 0, 0], np.zeros(0, np.int32), np.zeros(0, np.float32),
                         np.ones((3, 5), np.float32))
    assert _status() == 0 and n_acc.tolist() == [0, 0, 0]


def test_verify_rejects_drafts_outside_the_vocabulary():
    V, new = 300, [3, 3]
    z, y, tokens, u, noise = _verify_inputs(new, V, seed=9)
    u[:] = 0.0
    for wrong in (-1, V, 1 << 30):
        tokens[4] = wrong
        n_acc, out = _verify(z, y, 1.0, new, tokens, u, noise)
        assert _status() == 1
        assert n_acc.tolist() == [2, 0] and out[4:].tolist() == [-1, -1] and 0 <= out[3] < V
        n_acc, out = _verify(z, None, 0.0, new, tokens, u, noise)
        assert _status() == 1 and n_acc[1] == 0


def test_verify_keeps_the_target_distribution():
    """Over many draws the first token of a step is distributed as p, whatever the draft proposes.  For
    N draws the count of a token is off by less than 6 sqrt(N p (1 - p)) + 1."""
    V, N = 8, 20000
    rng = np.random.default_rng(0)
    zr, yr = rng.normal(size=V) * 1.5, rng.normal(size=V) * 1.5
    p, q = R.softmax(zr, 1.0), R.softmax(yr, 1.0)
    new = [2] * N
    z = np.tile(zr.astype(np.float32), (2 * N, 1))
    y = np.tile(yr.astype(np.float32), (2 * N, 1))
    tokens = np.zeros(2 * N, np.int32)
    tokens[1::2] = rng.choice(V, size=N, p=q)
    n_acc, out = _verify(z, y, 1.0, new, tokens, rng.random(2 * N).astype(np.float32),
                         rng.exponential(size=(N, V)).astype(np.float32))
    first = np.bincount(out[0::2], minlength=V)
    assert np.all(np.abs(first - N * p) <= 6 * np.sqrt(N * p * (1 - p)) + 1)
    kept = np.minimum(p, q).sum()
    assert abs(n_acc.sum() - N * kept) <= 6 * np.sqrt(N * kept * (1 - kept)) + 1


# -------------------------------------------------------------------------------------- together
class Step:
    """One serving step over random projections: plan, append, attend, verify."""

    def __init__(self, cached, new, n_q=8, n_kv=2, hd=64, V=2000, room=None, seed=0):
        import torch
        rng = np.random.default_rng(seed)
        self.cached, self.new, self.V = cached, new, V
        self.n_q, self.n_kv, self.hd = n_q, n_kv, hd
        self.table0, self.free, self.n_pages = _plan_inputs(cached, new, seed)
        self.T = room or sum(new)
        f = lambda *s: _dev(rng.normal(size=s), torch.bfloat16)
        self.qkv = f(self.T, n_q + 2 * n_kv, hd)
        self.kp, self.vp = f(self.n_pages, 128, n_kv, hd), f(self.n_pages, 128, n_kv, hd)
        self.pools0 = self.kp.clone(), self.vp.clone()
        self.w_out = _dev(rng.normal(size=(n_q * hd, V)) * 0.2, torch.float32)
        self.tokens = _i32(rng.integers(0, V, self.T))
        self.u = _dev(rng.random(self.T).astype(np.float32))
        self.noise = _dev(rng.exponential(size=(len(cached), V)).astype(np.float32))
        i = lambda n: torch.full((n,), -9, dtype=torch.int32, device="cuda")
        B = len(cached)
        self.lens = _i32(cached), _i32(new)
        self.free_t, self.table = _i32(self.free), _dev(self.table0)
        self.cu, self.pos, self.slots, self.used = i(B + 1), i(self.T), i(self.T), i(1)
        self.q = torch.zeros((self.T, n_q, hd), dtype=torch.bfloat16, device="cuda")
        self.o = torch.zeros_like(self.q)
        self.n_acc, self.out = i(B), i(self.T)
        self.max_pos = max(c + n for c, n in zip(cached, new)) - 1
        self.dims = L.dims_of(B, self.T, 128, n_q, n_kv, hd, 128, THETA, 1e-5)
        byte = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")
        self.ws = byte(L.llama_workspace_bytes(L.OP_GQA_ATTENTION_CHUNK_PAGED, self.dims, L.BF16,
                                               kv_capacity=self.max_pos + 1))
        self.ws2 = byte(L.llama_workspace_bytes(L.OP_VERIFY_DRAFTS, self.dims, L.F32, vocab=V))
        self.logits = torch.empty((self.T, V), dtype=torch.float32, device="cuda")

    def run(self):
        import torch
        q, k, v = (self.qkv[:, a:b] for a, b in ((0, self.n_q), (self.n_q, self.n_q + self.n_kv),
                                                 (self.n_q + self.n_kv, self.n_q + 2 * self.n_kv)))
        L.llama_paged_plan(*self.lens, self.free_t, self.n_pages, self.table, self.cu, self.pos, self.slots, self.used)
        L.llama_rope_append_paged(self.dims, q, k, v, self.pos, self.slots, self.q, self.kp, self.vp)
        L.llama_gqa_attention_chunk_paged(self.dims, self.q, self.kp, self.vp, self.table, self.cu, self.lens[0],
                                          self.max_pos, self.o, self.ws)
        torch.matmul(self.o.view(self.T, -1).float(), self.w_out, out=self.logits)
        L.llama_verify_drafts(self.logits, None, 1.0, self.cu, self.tokens, self.u, self.noise, self.n_acc, self.out,
                              self.ws2)

    def check(self):
        table, cu, pos, slots, used = R.plan(self.cached, self.new, self.free, self.table0, self.T)
        np.testing.assert_array_equal(self.slots.cpu().numpy(), slots)
        np.testing.assert_array_equal(self.table.cpu().numpy(), table)
        n, x = int(cu[-1]), to_f64(self.qkv)
        kp, vp = (to_f64(p).reshape(-1, self.n_kv, self.hd) for p in self.pools0)
        at = slots[:n]
        # what the step stored (bf16) is what attention reads
        _assert_rotated(to_f64(self.kp).reshape(kp.shape)[at], x[:n, self.n_q:self.n_q + self.n_kv], pos[:n], "k")
        kp, vp = to_f64(self.kp).reshape(kp.shape), vp.copy()
        vp[at] = x[:n, self.n_q + self.n_kv:]
        qr, z, tok = to_f64(self.q), self.logits.cpu().numpy(), self.tokens.cpu().numpy()
        _assert_rotated(qr[:n], x[:n, :self.n_q], pos[:n], "q")
        n_acc, out = self.n_acc.cpu().numpy(), self.out.cpu().numpy()
        for b, (c, m) in enumerate(zip(self.cached, self.new)):
            if m == 0:
                continue
            lo = cu[b]
            rows = (table[b][np.arange(c + m) // 128].astype(np.int64) * 128 + np.arange(c + m) % 128)
            ref = R.attention(qr[lo:lo + m], kp[rows], vp[rows], c)
            assert_parity(to_f64(self.o)[lo:lo + m], ref, BF16, f"seq {b}")
            w = R.verify(z[lo:lo + m], None, 1.0, tok[lo:lo + m], self.u.cpu().numpy()[lo:lo + m],
                         self.noise[b].cpu().numpy())
            if w[2] > NEAR:
                assert n_acc[b] == w[0] and out[lo:lo + m].tolist() == w[1]


def test_serving_step():
    s = Step([300, 0, 127, 1000], [4, 60, 2, 1], seed=1)
    s.run()
    assert _status() == 0
    s.check()


def test_serving_step_captured_and_replayed_with_other_lengths():
    """The step captured once with room for more tokens, replayed after lengths and values changed; two
    graphs share the workspaces."""
    import torch
    s = Step([300, 20, 127], [4, 60, 2], room=90, seed=2)
    s.run()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    for turn, (cached, new) in enumerate((([300, 20, 127], [4, 60, 2]), ([299, 70, 100], [1, 1, 5]),
                                          ([40, 33, 120], [0, 30, 9]), ([128, 0, 1], [40, 46, 4]))):
        table, free, n_pages = _plan_inputs(cached, new, seed=turn)
        P, F = s.table0.shape[1], len(s.free)
        if table.shape[1] > P or n_pages > s.n_pages or sum(-(-(c + n) // 128) + 0 for c, n in zip(cached, new)) > s.n_pages:
            raise AssertionError("the replayed case must fit the captured one")
        full = np.full((len(cached), P), -7, np.int32)
        full[:, :table.shape[1]] = table
        taken = sum(-(-(c + n) // 128) - -(-c // 128) for c, n in zip(cached, new))
        free_full = np.zeros(F, np.int32)
        assert taken <= F
        free_full[:taken] = free[:taken]
        s.cached, s.new, s.table0, s.free = cached, new, full, free_full
        s.lens[0].copy_(_i32(cached))
        s.lens[1].copy_(_i32(new))
        s.free_t.copy_(_i32(free_full))
        s.table.copy_(_dev(full))
        s.pools0 = s.kp.clone(), s.vp.clone()
        s.qkv.copy_(_dev(np.random.default_rng(turn).normal(size=tuple(s.qkv.shape)), torch.bfloat16))
        graphs[turn % 2].replay()
        assert _status() == 0
        s.check()


def test_serving_steps_on_two_streams():
    import torch
    steps = [Step([700, 5], [5, 130], seed=3), Step([64, 2000, 1], [64, 3, 1], seed=4)]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, st in zip(steps, streams):
            with torch.cuda.stream(st):
                s.run()
    torch.cuda.synchronize()
    assert _status() == 0
    for s in steps:
        s.check()
