"""The 8-bit paged cache on the GPU against its 64-bit definitions (tests/kv8_paged_ref.py): rows written with a scale per
position and head, read back, and attended to."""
import numpy as np
import pytest

import llama_decoder_block_fwd_gb300 as L
from synth import BF16
from tests import kv8_paged_ref as R
from tests.helpers import assert_parity, to_f64

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


def _dims(B, S, n_q, n_kv, hd, theta=THETA):
    return L.dims_of(B, S, n_q * hd, n_q, n_kv, hd, 128, theta, 1e-5)


# ---------------------------------------------------------------------------------------- append
def _append(q, k, v, positions, slots, n_pages, fill=0x55, n_q=None):
    """Runs the call on a pool filled with a pattern: (q_out, k codes, k scales, v codes, v scales) as numpy."""
    import torch
    T, n_kv, hd = k.shape
    n_q = (q.shape[1] if q is not None else n_kv) if n_q is None else n_q
    codes = [torch.full((n_pages, 128, n_kv, hd), fill, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((n_pages, n_kv, 128), -7.0, device="cuda") for _ in range(2)]
    qo = None if q is None else torch.full((T, n_q, hd), -3.0, dtype=torch.bfloat16, device="cuda")
    L.llama_rope_append_paged_kv8(_dims(1, T, n_q, n_kv, hd), q, k, v, _i32(positions), _i32(slots), qo, codes[0],
                                  scales[0], codes[1], scales[1])
    return (None if qo is None else to_f64(qo), *[x.cpu().numpy() for p in zip(codes, scales) for x in p])


def _at(slots, codes, scales):
    page, row = np.asarray(slots) // 128, np.asarray(slots) % 128
    return codes[page, row], scales[page, :, row]


def _check_written(k, v, positions, got, slots):
    """Scales exactly; V's codes exactly (nothing but one rounding); K's within half a step of the exact
    rotation, plus what the fp32 rotation is off by (angle reduction 6e-11 a turn, sine and cosine 2^-20 in all)."""
    x, ks, y, vs = R.append(k, v, positions, THETA)
    _, kc, ksc, vc, vsc = got
    c, s = _at(slots, kc, ksc)
    np.testing.assert_array_equal(s, ks)
    pair = np.repeat(np.abs(k[..., 0::2]) + np.abs(k[..., 1::2]), 2, axis=-1)
    off = pair * (2.0 ** -19 + positions.astype(np.float64)[:, None, None] * 1e-11)
    tol = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * ks[..., None]) + off * (1 + 2.0 ** -4)
    assert np.all(np.abs(R.E4M3[c] * s[..., None] - x) <= tol)
    c, s = _at(slots, vc, vsc)
    np.testing.assert_array_equal(s, vs)
    np.testing.assert_array_equal(c, R.encode(y / vs[..., None]))


@pytest.mark.parametrize("T,n_q,n_kv,hd,first", [(1, 32, 8, 128, 0), (5, 8, 2, 64, 131), (300, 32, 8, 128, 131000),
                                                 (1000, 28, 4, 128, 8000), (7, 3, 3, 8, 40), (9, 5, 1, 256, 3),
                                                 (700, 2, 1, 72, 77), (2500, 8, 8, 64, 400000), (613, 6, 3, 24, 1),
                                                 (1300, 32, 8, 128, 12), (640, 4, 2, 200, 9)])
@pytest.mark.parametrize("fused", [True, False])
def test_append_writes_codes_and_scales(T, n_q, n_kv, hd, first, fused):
    import torch
    rng = np.random.default_rng(T + hd)
    x = rng.normal(size=(T, n_q + 2 * n_kv, hd)) * np.exp(rng.normal(size=(T, n_q + 2 * n_kv, 1)) * 3)
    x = _dev(x, torch.bfloat16)
    parts = (x[:, :n_q], x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:])
    q, k, v = parts if fused else [p.contiguous() for p in parts]
    n_pages = -(-T // 128) + 4
    positions = (first + np.arange(T)).astype(np.int32)
    slots = rng.permutation(n_pages * 128)[:T].astype(np.int32)
    got = _append(q, k, v, positions, slots, n_pages)
    assert _status() == 0
    _check_written(to_f64(k), to_f64(v), positions, got, slots)
    # q: half a bf16 step, and what the angle is off by
    ref = R.rotate(to_f64(q), positions, THETA)
    pair = np.repeat(np.abs(to_f64(q)[..., 0::2]) + np.abs(to_f64(q)[..., 1::2]), 2, axis=-1)
    tol = 2.0 ** -8 * np.abs(ref) + pair * (2.0 ** -19 + positions.astype(np.float64)[:, None, None] * 1e-11)
    assert np.all(np.abs(got[0] - ref) <= tol)
    # nothing else was written
    rest = np.setdiff1d(np.arange(n_pages * 128), slots)
    for codes, scales in ((got[1], got[2]), (got[3], got[4])):
        c, s = _at(rest, codes, scales)
        assert np.all(c == 0x55) and np.all(s == -7.0)
    # append only gives the same rows
    alone = _append(None, k, v, positions, slots, n_pages, n_q=n_q)
    for a, b in zip(alone[1:], got[1:]):
        np.testing.assert_array_equal(a, b)


def test_append_of_extreme_rows():
    """Zeros, single elements, both ends of a binade, subnormal and huge rows, infinities and NaN."""
    import torch
    hd, n_kv = 64, 1
    v = np.zeros((16, n_kv, hd))
    v[1, 0, 5] = 448.0
    v[2, 0, 5] = -450.0                  # above 448: the next scale
    v[3, 0] = 2.0 ** -130                # below the smallest scale's smallest code
    v[4, 0, :2] = 3.0e38, -1.0           # the largest scale saturates nothing below 448 * 2^100
    v[5, 0, 3] = np.inf
    v[6, 0, 3], v[6, 0, 4] = np.nan, 2.0
    v[7, 0] = 7.0 / 8 * 2.0 ** 3
    v[8, 0] = np.where(np.arange(hd) % 2, 1.0, 2.0 ** -9)
    v[9, 0] = -np.inf
    v[10, 0] = np.nan
    v[11, 0, 63] = -2.0 ** -100
    v[12, 0] = np.linspace(-500, 500, hd)
    v[13, 0, 0], v[13, 0, 1] = 1.76 * 2.0 ** 8, 1.75 * 2.0 ** 8
    t = _dev(v, torch.bfloat16)
    vf = to_f64(t)
    slots = np.arange(16)
    _, kc, ks, vc, vs = _append(None, t, t, np.zeros(16), slots, 1)
    assert _status() == 0
    u = np.fmax.reduce(np.abs(vf), -1)
    u = np.where(np.isnan(u), 0.0, u)
    want = R.row_scale(u)
    c, s = _at(slots, vc, vs)
    np.testing.assert_array_equal(s, want)
    with np.errstate(invalid="ignore"):
        ref = R.encode(vf / want[..., None])
    nan = np.isnan(vf)
    assert np.all((c[nan] & 0x7F) == 0x7F)
    np.testing.assert_array_equal(c[~nan], ref[~nan])
    # at position 0 a key is its own rotation: rows of finite values come out as for V, at K's scale
    fin = np.isfinite(vf).all((1, 2))
    kw = R.row_scale(R.k_bound(vf[fin]))
    c, s = _at(slots[fin], kc, ks)
    np.testing.assert_array_equal(s, kw)
    np.testing.assert_array_equal(R.E4M3[c], R.E4M3[R.encode(vf[fin] / kw[..., None])])
    assert _at([6], kc, ks)[1][0, 0] == R.row_scale(2.0)      # a pair that holds a NaN has no part in its row's scale


def test_append_skips_and_latches():
    import torch
    rng = np.random.default_rng(3)
    T, n_kv, hd, n_pages = 9, 2, 64, 2
    k = _dev(rng.normal(size=(T, n_kv, hd)), torch.bfloat16)
    q = _dev(rng.normal(size=(T, 4, hd)), torch.bfloat16)
    slots = np.array([3, -1, 200, 7, 256, 9, -1, 100, 50])
    pos = np.array([0, 1, 2, 3, 4, -5, 6, 1 << 24, 8])
    got = _append(q, k, k, pos, slots, n_pages)
    assert _status() == 1
    live = [0, 2, 3, 8]
    _check_written(to_f64(k)[live], to_f64(k)[live], pos[live], got, slots[live])
    assert np.all(got[0][[1, 4, 5, 6, 7]] == -3.0)
    rest = np.setdiff1d(np.arange(256), slots[live])
    assert np.all(_at(rest, got[1], got[2])[0] == 0x55)
    got = _append(q, k, k, np.arange(T), np.full(T, -1), n_pages)          # nothing to do is no error
    assert _status() == 0 and np.all(got[1] == 0x55)


@pytest.mark.parametrize("T,n_q,n_kv,hd", [(4003, 6, 3, 64), (3661, 4, 1, 128), (8191, 1, 1, 64)])
def test_append_of_many_tokens_some_skipped(T, n_q, n_kv, hd):
    import torch
    rng = np.random.default_rng(T)
    x = _dev(rng.normal(size=(T, n_q + 2 * n_kv, hd)) * np.exp(rng.normal(size=(T, n_q + 2 * n_kv, 1)) * 3), torch.bfloat16)
    q, k, v = x[:, :n_q], x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:]
    n_pages = -(-T // 128) + 1
    slots = rng.permutation(n_pages * 128)[:T].astype(np.int32)
    slots[rng.random(T) < 0.3] = -1
    slots[:9] = -1
    pos = rng.integers(0, 1 << 17, size=T).astype(np.int32)
    got = _append(q, k, v, pos, slots, n_pages)
    assert _status() == 0
    live = np.flatnonzero(slots >= 0)
    _check_written(to_f64(k)[live], to_f64(v)[live], pos[live], got, slots[live])
    assert np.all(got[0][slots < 0] == -3.0)
    ref = R.rotate(to_f64(q)[live], pos[live], THETA)
    pair = np.repeat(np.abs(to_f64(q)[live][..., 0::2]) + np.abs(to_f64(q)[live][..., 1::2]), 2, axis=-1)
    tol = 2.0 ** -8 * np.abs(ref) + pair * (2.0 ** -19 + pos[live].astype(np.float64)[:, None, None] * 1e-11)
    assert np.all(np.abs(got[0][live] - ref) <= tol)
    rest = np.setdiff1d(np.arange(n_pages * 128), slots)
    for codes, scales in ((got[1], got[2]), (got[3], got[4])):
        c, s = _at(rest, codes, scales)
        assert np.all(c == 0x55) and np.all(s == -7.0)


# -------------------------------------------------------------------------------------- read back
class Cache:
    """Random codes and scales of sequences of the given lengths in shuffled pages, NaN in every row that no
    sequence holds; shared: sequences whose first pages are sequence 0's."""

    def __init__(self, lengths, n_kv, hd, seed=0, spread=1.0, shared=(), general=False):
        rng = np.random.default_rng(seed)
        self.lengths, self.n_kv, self.hd = list(lengths), n_kv, hd
        pages = [-(-n // 128) for n in lengths]
        self.P = max(pages + [1]) + 1
        self.n_pages = sum(pages) + 3
        ids = list(rng.permutation(self.n_pages))
        self.table = np.full((len(lengths), self.P), -5, np.int32)
        for b, c in enumerate(pages):
            self.table[b, :c] = [ids.pop() for _ in range(c)]
            if b in shared:
                self.table[b, :min(c, pages[0]) - 1] = self.table[0, :min(c, pages[0]) - 1]
        self.codes = [np.full((self.n_pages, 128, n_kv, hd), 0x7F, np.uint8) for _ in range(2)]
        self.scales = [np.full((self.n_pages, n_kv, 128), np.nan, np.float32) for _ in range(2)]
        for b, n in enumerate(lengths):
            pos = np.arange(n)
            page, row = self.table[b, pos // 128], pos % 128
            for c, s in zip(self.codes, self.scales):
                x = rng.normal(size=(n, n_kv, hd)) * np.exp(spread * rng.normal(size=(n, n_kv, 1)))
                sc = R.row_scale(np.max(np.abs(x), -1))
                if general:
                    sc = (np.max(np.abs(x), -1) / 448).astype(np.float32).astype(np.float64)
                c[page, row] = R.encode(x / sc[..., None])
                s[page, :, row] = sc

    def dev(self):
        return [_dev(x) for p in zip(self.codes, self.scales) for x in p]

    def rows(self, b, n=None):
        n = self.lengths[b] if n is None else n
        return [R.rows(c, s, self.table[b], n) for c, s in zip(self.codes, self.scales)]


LENGTHS = [[1], [127, 128, 129], [0, 5, 0, 700], [3000], [640] * 7, [1, 2, 3, 1000, 0]]


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("n_kv,hd,general", [(8, 128, False), (2, 64, True), (1, 8, False), (3, 72, True), (1, 256, False)])
def test_dequantize_gives_the_values(lengths, n_kv, hd, general):
    import torch
    c = Cache(lengths, n_kv, hd, seed=hd + len(lengths), general=general)
    pools = [torch.full((c.n_pages, 128, n_kv, hd), -9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    L.llama_kv_dequantize_paged(*c.dev(), _dev(c.table), _i32(lengths), *pools)
    assert _status() == 0
    for codes, scales, pool in zip(c.codes, c.scales, pools):
        want = np.full(codes.shape, -9.0)
        for b, n in enumerate(lengths):
            pos = np.arange(n)
            page = c.table[b, pos // 128]
            x = (R.E4M3[codes[page, pos % 128]].astype(np.float32) * scales[page, :, pos % 128][..., None])   # one fp32 product
            want[page, pos % 128] = to_f64(torch.from_numpy(x).to(torch.bfloat16))
        np.testing.assert_array_equal(to_f64(pool), want)


def test_dequantize_latches_and_skips():
    import torch
    c = Cache([300, 300, 300], 2, 64)
    table, pools = c.table.copy(), [torch.zeros(c.n_pages, 128, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table[1, 1] = c.n_pages
    L.llama_kv_dequantize_paged(*c.dev(), _dev(table), _i32([300, 300, -1]), *pools)
    assert _status() == 1
    got = to_f64(pools[0])
    assert np.all(got[c.table[2, :3]] == 0) and np.all(got[c.table[1, 1]] == 0)
    for b, j, n in ((0, 0, 128), (0, 2, 44), (1, 0, 128), (1, 2, 44)):
        np.testing.assert_array_equal(got[c.table[b, j], :n], c.rows(b)[0][j * 128:j * 128 + n])
    for bad in (128 * c.P + 1, 2 ** 31 - 1, -2 ** 31):
        L.llama_kv_dequantize_paged(*c.dev(), _dev(c.table), _i32([bad, 0, 0]), *pools)
        assert _status() == 1
    wide = torch.full((1, 1 << 18), -1, dtype=torch.int32, device="cuda")       # room for more positions than there are
    L.llama_kv_dequantize_paged(*c.dev(), wide, _i32([2 ** 24 + 1]), *pools)
    assert _status() == 1
    L.llama_kv_dequantize_paged(*c.dev(), _dev(c.table), _i32([300, 300, 300]), *pools)
    assert _status() == 0


# -------------------------------------------------------------------------------------- attention
def _attend(c, q, seq_pos, table=None, max_pos=None, stream=None, ws=None, o=None):
    import torch
    B, n_q, hd = q.shape
    dims = _dims(B, 1, n_q, c.n_kv, hd)
    top = max(max(seq_pos), 0) if max_pos is None else max_pos
    o = torch.full((B, n_q, hd), 77.0, dtype=torch.bfloat16, device="cuda") if o is None else o
    ws = torch.full((L.llama_workspace_bytes(L.OP_GQA_ATTENTION_DECODE_PAGED_KV8, dims, L.BF16, kv_capacity=top + 1),), 0xFF,
                    dtype=torch.uint8, device="cuda") if ws is None else ws
    L.llama_gqa_attention_decode_paged_kv8(dims, q, *c.dev(), _dev(c.table if table is None else table), _i32(seq_pos), top, o,
                                           ws, stream)
    return o


def _queries(B, n_q, hd, seed, std=2.0):
    import torch
    return _dev(np.random.default_rng(seed).normal(size=(B, n_q, hd)) * std, torch.bfloat16)


def _check_attention(c, q, o, seqs=None):
    ref = np.stack([R.attend(to_f64(q)[b], *c.rows(b)) for b in (range(len(c.lengths)) if seqs is None else seqs)])
    got = to_f64(o) if seqs is None else to_f64(o)[list(seqs)]
    live = [i for i, b in enumerate(range(len(c.lengths)) if seqs is None else seqs) if c.lengths[b] > 0]
    dead = [i for i in range(len(ref)) if i not in live]
    assert np.all(got[dead] == 0)
    if live:
        assert_parity(got[live], ref[live], BF16, "attention over 8-bit pages")


HEADS = [(32, 8, 128), (8, 2, 64), (1, 1, 128), (6, 3, 64), (28, 4, 128), (16, 1, 128), (24, 1, 128), (40, 1, 64), (7, 7, 64),
         (12, 4, 128), (64, 2, 128), (3, 1, 64), (34, 2, 128), (10, 2, 128), (32, 2, 64), (18, 2, 64), (128, 1, 128), (320, 320, 128), (310, 310, 64)]


@pytest.mark.parametrize("n_q,n_kv,hd", HEADS)
@pytest.mark.parametrize("lengths", [[1], [128, 129, 1, 0, 640, 77], [2050, 5]])
def test_attention_matches_its_definition(n_q, n_kv, hd, lengths):
    c = Cache(lengths, n_kv, hd, seed=n_q)
    q = _queries(len(lengths), n_q, hd, 1)
    o = _attend(c, q, [n - 1 for n in lengths])
    assert _status() == 0
    _check_attention(c, q, o)


@pytest.mark.parametrize("spread,std", [(0.0, 0.3), (3.0, 2.0), (1.0, 12.0), (6.0, 0.01)])
def test_attention_of_flat_and_peaked_rows(spread, std):
    """Scales that differ by orders of magnitude within a tile, weights from even to one key's."""
    lengths = [1500, 300, 129]
    c = Cache(lengths, 2, 128, seed=5, spread=spread)
    q = _queries(3, 8, 128, 2, std)
    o = _attend(c, q, [n - 1 for n in lengths])
    assert _status() == 0
    _check_attention(c, q, o)


def test_attention_keeps_a_long_tail_beside_a_sink():
    """One key has most of the weight, tens of thousands the rest: their sum is not lost to the 8-bit weights."""
    import torch
    n, hd = 60000, 128
    c = Cache([n], 1, hd, seed=8, spread=0.0)
    rng = np.random.default_rng(1)
    q = np.zeros((1, 1, hd))
    q[0, 0, 0] = 4.0
    k = np.zeros((n, 1, hd))
    k[7, 0, 0] = np.log(40000.0) * np.sqrt(hd) / 4.0       # exp(score): 40000 against 60000 times 1
    v = np.abs(rng.normal(size=(n, 1, hd))) + 0.5
    v[7] = -1.0
    pos = np.arange(n)
    page, row = c.table[0, pos // 128], pos % 128
    for x, codes, scales in ((k, c.codes[0], c.scales[0]), (v, c.codes[1], c.scales[1])):
        s = R.row_scale(np.max(np.abs(x), -1))
        codes[page, row], scales[page, :, row] = R.encode(x / s[..., None]), s
    qd = _dev(q, torch.bfloat16)
    o = _attend(c, qd, [n - 1])
    assert _status() == 0
    _check_attention(c, qd, o)


def test_attention_with_general_scales_and_shared_pages():
    lengths = [1000, 900, 1000, 130]
    c = Cache(lengths, 4, 128, seed=9, general=True, shared=(1, 2))
    q = _queries(4, 28, 128, 3)
    o = _attend(c, q, [n - 1 for n in lengths], max_pos=5 + max(lengths))
    assert _status() == 0
    _check_attention(c, q, o)


def test_attention_of_heads_of_very_different_size():
    import torch
    lengths = [700]
    c = Cache(lengths, 1, 128, seed=4)
    q = np.random.default_rng(2).normal(size=(1, 16, 128)) * (10.0 ** np.linspace(-6, 1, 16))[None, :, None]
    q[0, 3] = 0.0
    q = _dev(q, torch.bfloat16)
    o = _attend(c, q, [699])
    assert _status() == 0
    _check_attention(c, q, o)


def test_attention_latches_bad_positions_and_pages():
    import torch
    lengths = [300, 300, 300, 300]
    c = Cache(lengths, 2, 128, seed=6)
    q = _queries(4, 8, 128, 6)
    table = c.table.copy()
    table[2, 1] = c.n_pages
    table[3, 0] = -1
    o = _attend(c, q, [299, 300, 299, 299], table=table, max_pos=299)
    assert _status() == 1
    assert torch.all(o[1] == 0)
    _check_attention(c, q, o, [0])
    o = _attend(c, q, [299, -2, 299, -1])
    assert _status() == 1 and torch.all(o[1] == 0) and torch.all(o[3] == 0)
    _check_attention(c, q, o, [0, 2])
    o = _attend(c, q, [299] * 4)
    assert _status() == 0
    _check_attention(c, q, o)


@pytest.mark.parametrize("B,hi", [(300, 40), (700, 300)])
def test_attention_of_many_sequences(B, hi):
    rng = np.random.default_rng(B)
    lengths = [int(x) for x in rng.integers(0, hi, size=B)]
    c = Cache(lengths, 2, 64, seed=B)
    q = _queries(B, 8, 64, B)
    o = _attend(c, q, [n - 1 for n in lengths], max_pos=hi)
    assert _status() == 0
    _check_attention(c, q, o)


def test_attention_of_a_long_sequence_beside_short_ones():
    lengths = [9, 70000, 0, 130]
    c = Cache(lengths, 2, 128, seed=2)
    q = _queries(4, 8, 128, 2)
    o = _attend(c, q, [n - 1 for n in lengths])
    assert _status() == 0
    _check_attention(c, q, o)


def test_attention_of_a_pool_past_2_31_bytes():
    """Page offsets past 32 bits: the pages in use are the last of a 2.3 GB pool."""
    import torch
    lengths = [300]
    c = Cache(lengths, 8, 128, seed=1)
    n_pages = 18000
    shift = n_pages - c.n_pages
    pools = []
    for codes, scales in zip(c.codes, c.scales):
        big = torch.empty(n_pages, 128, 8, 128, dtype=torch.uint8, device="cuda")
        big[shift:] = _dev(codes)
        sc = torch.empty(n_pages, 8, 128, device="cuda")
        sc[shift:] = _dev(scales)
        pools += [big, sc]
    q = _queries(1, 32, 128, 1)
    dims = _dims(1, 1, 32, 8, 128)
    o = torch.empty_like(q)
    ws = torch.empty(L.llama_workspace_bytes(L.OP_GQA_ATTENTION_DECODE_PAGED_KV8, dims, L.BF16, kv_capacity=300),
                     dtype=torch.uint8, device="cuda")
    table = _dev(np.where(c.table >= 0, c.table + shift, c.table).astype(np.int32))
    L.llama_gqa_attention_decode_paged_kv8(dims, q, *pools, table, _i32([299]), 299, o, ws)
    assert _status() == 0
    _check_attention(c, q, o)
    bf = [torch.zeros(n_pages, 128, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    L.llama_kv_dequantize_paged(*pools, table, _i32([300]), *bf)
    k = to_f64(bf[0][table[0, :3].long()]).reshape(-1, 8, 128)[:300]
    np.testing.assert_array_equal(k, c.rows(0)[0])
    x = _queries(1, 8, 128, 3)
    slot = int(table[0, 2]) * 128 + 44
    L.llama_rope_append_paged_kv8(_dims(1, 1, 32, 8, 128), None, x, x, _i32([0]), _i32([slot]), None, *pools)
    assert _status() == 0
    assert pools[3][slot // 128, 0, 44] == float(R.row_scale(np.max(np.abs(to_f64(x)[0, 0]))))


def test_attention_captured_and_replayed_beside_another_stream():
    """A captured call replays with other lengths, tables and queries, while a second one with a workspace of its own
    runs on another stream."""
    import torch
    lengths = [2000, 4, 500]
    c = Cache(lengths, 2, 128, seed=12)
    cache, table, q = c.dev(), _dev(c.table), _queries(3, 8, 128, 1)
    dims = _dims(3, 1, 8, 2, 128)
    n = L.llama_workspace_bytes(L.OP_GQA_ATTENTION_DECODE_PAGED_KV8, dims, L.BF16, kv_capacity=2000)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    pos = [_i32([1999, 0, 499]) for _ in range(2)]
    qs, o = [q.clone(), q.clone()], [torch.empty_like(q) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        L.llama_gqa_attention_decode_paged_kv8(dims, qs[i], *cache, table, pos[i], 1999, o[i], ws[i])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[i]):
            L.llama_gqa_attention_decode_paged_kv8(dims, qs[i], *cache, table, pos[i], 1999, o[i], ws[i])
        graphs.append(g)
    for step in range(4):
        now = [[1999 - 100 * step, step, 499 - step], [128 * step, 0, 130 + step]]
        for i in range(2):
            pos[i].copy_(_i32(now[i]))
            qs[i].copy_(_queries(3, 8, 128, 10 * step + i))
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
                graphs[i].replay()
        torch.cuda.synchronize()
        assert _status() == 0
        for i in range(2):
            for b in range(3):
                ref = R.attend(to_f64(qs[i])[b], *c.rows(b, now[i][b] + 1))
                assert_parity(to_f64(o[i])[b], ref, BF16, f"replay {step}, graph {i}, sequence {b}")


def test_calls_on_a_given_stream_and_twice_give_the_same_bits():
    """The stream argument is honoured (work queued behind a long wait on that stream alone), and repeated calls agree."""
    import torch
    lengths = [5000, 131, 0, 2600]
    c = Cache(lengths, 2, 128, seed=3)
    q = _queries(4, 8, 128, 5)
    want = _attend(c, q, [n - 1 for n in lengths])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):                      # the inputs made here, the call made there
        q2 = q.clone()
    o = torch.empty_like(q)
    s.synchronize()
    for stream in (s, s.cuda_stream):
        o.fill_(7.0)
        torch.cuda.synchronize()
        _attend(c, q2, [n - 1 for n in lengths], stream=stream, o=o)
        s.synchronize()
        assert torch.equal(o, want)
    pools = [torch.zeros(c.n_pages, 128, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cache, table, n = c.dev(), _dev(c.table), _i32(lengths)
    torch.cuda.synchronize()
    L.llama_kv_dequantize_paged(*cache, table, n, *pools, stream=s)
    s.synchronize()
    np.testing.assert_array_equal(to_f64(pools[1])[c.table[1, 0]], c.rows(1)[1][:128])
    x = _queries(3, 2, 128, 1)
    pos, slots = _i32([0, 1, 2]), _i32([0, 1, 2])
    torch.cuda.synchronize()
    L.llama_rope_append_paged_kv8(_dims(1, 3, 8, 2, 128), None, x, x, pos, slots, None, *cache, stream=s)
    s.synchronize()
    assert _status() == 0 and cache[3][0, 1, 2] == float(R.row_scale(np.max(np.abs(to_f64(x)[2, 1]))))


@pytest.mark.parametrize("captured", [False, True])
def test_attention_behind_a_wait_on_another_stream(captured):
    """The call before it has finished early, what it reads comes late from another stream: it is waited for."""
    import torch
    lengths = [900, 4, 300]
    c = Cache(lengths, 2, 128, seed=21)
    cache, table, late = c.dev(), _dev(c.table), _queries(3, 8, 128, 5)
    dims = _dims(3, 1, 8, 2, 128)
    ws = torch.empty(L.llama_workspace_bytes(L.OP_GQA_ATTENTION_DECODE_PAGED_KV8, dims, L.BF16, kv_capacity=900),
                     dtype=torch.uint8, device="cuda")
    late_pos, q, pos = _i32([899, 3, 299]), torch.zeros_like(late), _i32([0, 0, 0])
    o = [torch.zeros_like(late) for _ in range(2)]
    first, main, side = _queries(3, 8, 128, 6), torch.cuda.Stream(), torch.cuda.Stream()
    early = _i32([500, 1, 2])

    def calls():
        side.wait_stream(torch.cuda.current_stream())
        L.llama_gqa_attention_decode_paged_kv8(dims, first, *cache, table, early, 899, o[0], ws)
        with torch.cuda.stream(side):
            torch.cuda._sleep(1_000_000)
            q.copy_(late)
            pos.copy_(late_pos)
        torch.cuda.current_stream().wait_stream(side)
        L.llama_gqa_attention_decode_paged_kv8(dims, q, *cache, table, pos, 899, o[1], ws)

    torch.cuda.synchronize()
    with torch.cuda.stream(main):
        calls()
    torch.cuda.synchronize()
    want = o[1].clone()
    _check_attention(c, late, want)
    g = None
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=main):
            calls()
    for _ in range(5):
        q.zero_(), pos.zero_(), o[1].fill_(3.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(main):
            g.replay() if captured else calls()
        torch.cuda.synchronize()
        assert _status() == 0 and torch.equal(o[1], want)
