"""The calls of the 8-bit paged cache and of beam search on the host: bad arguments come back as status codes before anything
is launched, each limit from both sides, and what the binding refuses.  No GPU is used."""
import ctypes

import pytest

import llama_decoder_block_fwd_gb300 as L
from tests.test_serving_binding import meta, note  # noqa: F401  (note: a fixture)

torch = pytest.importorskip("torch")
FAKE = 0x10000          # aligned, never dereferenced
BIG = 1 << 62
OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = range(5)


def dims(**kw):
    base = dict(B=2, S=6, d_model=1024, n_q=8, n_kv=2, head_dim=128, d_ff=128, theta_base=1e4, eps=1e-5)
    base.update(kw)
    return L.dims_of(**base)


def append(d=None, **kw):
    d = dims() if d is None else d
    w, wk = d.n_q * d.head_dim, d.n_kv * d.head_dim
    a = dict(q=FAKE, qs=w, k=FAKE, ks=wk, v=FAKE, vs=wk, positions=FAKE, slots=FAKE, q_out=FAKE, kc=FAKE, ksc=FAKE, vc=FAKE,
             vsc=FAKE, n_pages=4)
    a.update(kw)
    return L.lib().llama_rope_append_paged_kv8(ctypes.byref(d), *a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(d=dims(S=0)), OK), (dict(q=None), INVALID), (dict(q_out=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(kc=None), INVALID), (dict(ksc=None), INVALID), (dict(vc=None), INVALID), (dict(vsc=None), INVALID),
    (dict(positions=None), INVALID), (dict(slots=None), INVALID), (dict(n_pages=0), INVALID), (dict(qs=1016), INVALID),
    (dict(ks=248), INVALID), (dict(vs=248), INVALID), (dict(d=dims(n_q=7)), INVALID), (dict(d=dims(B=-1)), INVALID),
    (dict(d=dims(theta_base=0.0)), INVALID), (dict(qs=1028, q_out=FAKE + 4096), ALIGNMENT), (dict(ks=260), ALIGNMENT), (dict(q=FAKE + 8), ALIGNMENT),
    (dict(kc=FAKE + 8), ALIGNMENT), (dict(vsc=FAKE + 4), ALIGNMENT), (dict(slots=FAKE + 2), ALIGNMENT),
    (dict(qs=1032), INVALID),                       # in place with a stride of its own
    (dict(d=dims(n_q=4096), slots=None), INVALID), (dict(d=dims(n_q=4098)), UNSUPPORTED),
    (dict(d=dims(head_dim=256), slots=None), INVALID), (dict(d=dims(head_dim=264)), UNSUPPORTED), (dict(d=dims(head_dim=12)), UNSUPPORTED),
    (dict(d=dims(S=2 ** 31 - 9), slots=None), INVALID), (dict(d=dims(S=2 ** 31 - 7)), UNSUPPORTED),
    (dict(n_pages=2 ** 24 - 1, slots=None), INVALID), (dict(n_pages=2 ** 24), UNSUPPORTED)])
def test_append_refuses(kw, want):
    assert append(**kw) == want


def dequant(d=None, **kw):
    d = dims(S=0) if d is None else d
    a = dict(kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, n_pages=9, table=FAKE, max_pages=4, n_pos=FAKE, kp=FAKE, vp=FAKE)
    a.update(kw)
    return L.lib().llama_kv_dequantize_paged(ctypes.byref(d), *a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(d=dims(B=0)), OK), (dict(d=dims(B=-1)), INVALID), (dict(d=dims(n_kv=0)), INVALID), (dict(n_pages=0), INVALID),
    (dict(max_pages=0), INVALID), *[({n: None}, INVALID) for n in ("kc", "ks", "vc", "vs", "table", "n_pos", "kp", "vp")],
    (dict(kc=FAKE + 8), ALIGNMENT), (dict(vp=FAKE + 8), ALIGNMENT), (dict(table=FAKE + 2), ALIGNMENT), (dict(d=dims(head_dim=12)), UNSUPPORTED),
    (dict(d=dims(B=65535), n_pos=None), INVALID), (dict(d=dims(B=65536)), UNSUPPORTED), (dict(d=dims(head_dim=264)), UNSUPPORTED),
    (dict(d=dims(n_q=4096, n_kv=4096), n_pos=None), INVALID), (dict(d=dims(n_q=4097, n_kv=4097)), UNSUPPORTED),
    (dict(n_pages=2 ** 24 - 1, n_pos=None), INVALID), (dict(n_pages=2 ** 24), UNSUPPORTED),
    (dict(max_pages=2 ** 31 - 1, n_pos=None), INVALID), (dict(max_pages=2 ** 31), UNSUPPORTED)])
def test_dequantize_refuses(kw, want):
    assert dequant(**kw) == want


def attend(d=None, **kw):
    d = dims(S=1) if d is None else d
    a = dict(q=FAKE, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, n_pages=9, table=FAKE, max_pages=4, seq_pos=FAKE, max_pos=500, o=FAKE, ws=FAKE,
             ws_bytes=BIG)
    a.update(kw)
    return L.lib().llama_gqa_attention_decode_paged_kv8(ctypes.byref(d), *a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(d=dims(S=1, B=0)), OK), (dict(d=dims(S=2)), INVALID), (dict(d=dims(S=1, n_q=7)), INVALID), (dict(n_pages=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(max_pos=-1), INVALID), (dict(max_pos=511, ws=None), WORKSPACE), (dict(max_pos=512), INVALID),
    (dict(max_pages=2 ** 18, max_pos=2 ** 24 - 1, ws=None), WORKSPACE), (dict(max_pages=2 ** 18, max_pos=2 ** 24), INVALID),
    *[({n: None}, INVALID) for n in ("q", "kc", "ks", "vc", "vs", "table", "seq_pos", "o")],
    (dict(q=FAKE + 8), ALIGNMENT), (dict(vs=FAKE + 4), ALIGNMENT), (dict(seq_pos=FAKE + 1), ALIGNMENT), (dict(ws=FAKE + 8), ALIGNMENT),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=8), WORKSPACE), (dict(d=dims(S=1, head_dim=96)), UNSUPPORTED),
    (dict(d=dims(S=1, head_dim=64), ws=None), WORKSPACE), (dict(d=dims(S=1, n_q=65536), ws=None), WORKSPACE),
    (dict(d=dims(S=1, n_q=65538)), UNSUPPORTED), (dict(d=dims(S=1, B=65535), ws=None), WORKSPACE), (dict(d=dims(S=1, B=65536)), UNSUPPORTED),
    (dict(d=dims(S=1, B=32767, n_q=512, n_kv=512), ws=None), WORKSPACE), (dict(d=dims(S=1, B=32768, n_q=512, n_kv=512)), UNSUPPORTED),
    (dict(n_pages=2 ** 24 - 1, ws=None), WORKSPACE), (dict(n_pages=2 ** 24), UNSUPPORTED),
    (dict(max_pages=2 ** 31 - 1, ws=None), WORKSPACE), (dict(max_pages=2 ** 31), UNSUPPORTED)])
def test_attention_refuses(kw, want):
    assert attend(**kw) == want


def select(**kw):
    a = dict(z=FAKE, B=2, W=4, V=100, ld=100, scores=FAKE, finished=FAKE, pad=0, K=8, par=FAKE, tok=FAKE, out=FAKE, ws=FAKE, ws_bytes=BIG)
    a.update(kw)
    return L.lib().llama_beam_select(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), OK), (dict(B=-1), INVALID), (dict(W=0), INVALID), (dict(K=0), INVALID), (dict(V=0, ld=0), INVALID), (dict(ld=99), INVALID),
    (dict(pad=-1), INVALID), (dict(pad=100), INVALID), (dict(pad=-1, finished=None, ws=None), WORKSPACE),
    *[({n: None}, INVALID) for n in ("z", "scores", "par", "tok", "out")], (dict(z=FAKE + 2), ALIGNMENT), (dict(finished=FAKE + 1), ALIGNMENT),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=8), WORKSPACE), (dict(ws=FAKE + 8), ALIGNMENT), (dict(W=32, ws=None), WORKSPACE),
    (dict(W=33), UNSUPPORTED), (dict(K=64, ws=None), WORKSPACE), (dict(K=65), UNSUPPORTED), (dict(B=2 ** 20 - 1, ws=None), WORKSPACE),
    (dict(B=2 ** 20), UNSUPPORTED), (dict(V=2 ** 30, ld=BIG, ws=None), WORKSPACE), (dict(V=2 ** 30 + 1, ld=BIG), INVALID)])
def test_select_refuses(kw, want):
    assert select(**kw) == want


def reorder(pools=((FAKE, 2, 1, 1024), (FAKE, 2, 8, 4)), **kw):
    records = None if pools is None else (L.PagePool * max(1, len(pools)))(*[L.PagePool(*p) for p in pools])
    a = dict(par=FAKE, B=2, W=4, n=FAKE, n_out=FAKE, table=FAKE, out=FAKE, max_pages=4, free=FAKE, n_free=3, n_pages=9,
             pools=records, n_pools=1 if pools is None else len(pools), freed=FAKE, room=5, counts=FAKE, ws=FAKE, ws_bytes=BIG)
    a.update(kw)
    return L.lib().llama_beam_reorder_paged(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), INVALID), (dict(W=0), INVALID), (dict(max_pages=0), INVALID), (dict(n_free=-1), INVALID), (dict(n_pages=0), INVALID),
    (dict(room=-1), INVALID), (dict(n_pools=-1), INVALID), *[({n: None}, INVALID) for n in ("par", "n", "n_out", "table", "out", "free", "freed", "counts", "pools")],
    (dict(free=None, n_free=0, ws=None), WORKSPACE), (dict(freed=None, room=0, ws=None), WORKSPACE), (dict(par=FAKE + 2), ALIGNMENT),
    (dict(counts=FAKE + 1), ALIGNMENT), (dict(ws=None), WORKSPACE), (dict(ws_bytes=8), WORKSPACE), (dict(ws=FAKE + 8), ALIGNMENT),
    (dict(W=32, ws=None), WORKSPACE), (dict(W=33), UNSUPPORTED), (dict(B=8192, ws=None), WORKSPACE), (dict(B=8193), UNSUPPORTED),
    (dict(n_pages=2 ** 24 - 1, ws=None), WORKSPACE), (dict(n_pages=2 ** 24), UNSUPPORTED), (dict(max_pages=2 ** 17, ws=None), WORKSPACE),
    (dict(max_pages=2 ** 17 + 1), UNSUPPORTED), (dict(n_free=2 ** 31 - 1, ws=None), WORKSPACE), (dict(n_free=2 ** 31), UNSUPPORTED),
    (dict(room=2 ** 31 - 1, ws=None), WORKSPACE), (dict(room=2 ** 31), UNSUPPORTED),
    (dict(pools=[(FAKE, 1, 1, 16)] * 8, ws=None), WORKSPACE), (dict(pools=[(FAKE, 1, 1, 16)] * 9), UNSUPPORTED),
    (dict(pools=[(None, 1, 1, 16)]), INVALID), (dict(pools=[(FAKE + 8, 1, 1, 16)]), ALIGNMENT), (dict(pools=[(FAKE, 0, 1, 16)]), INVALID),
    (dict(pools=[(FAKE, 1, 0, 16)]), INVALID), (dict(pools=[(FAKE, 1, 1, 0)]), INVALID), (dict(pools=[(FAKE, 1, 1, 6)]), INVALID),
    (dict(pools=[(FAKE, 1, 1, 2 ** 24)], ws=None), WORKSPACE), (dict(pools=[(FAKE, 1, 2, 2 ** 24)]), UNSUPPORTED),
    (dict(pools=[(FAKE, 1, 2 ** 40, 2 ** 40)]), UNSUPPORTED), (dict(pools=[(FAKE, 2 ** 23, 1, 16)], ws=None), WORKSPACE),
    (dict(pools=[(FAKE, 2 ** 24 + 1, 1, 4)]), UNSUPPORTED), (dict(pools=[(FAKE, 8, 2, 2 ** 23)], ws=None), WORKSPACE),
    (dict(pools=[(FAKE, 9, 2, 2 ** 23)]), UNSUPPORTED)])
def test_reorder_refuses(kw, want):
    assert reorder(**kw) == want


def test_workspace_sizes():
    n = lambda op, d, dt=L.BF16, **kw: L.llama_workspace_bytes(op, d, dt, **kw)
    a = n(L.OP_GQA_ATTENTION_DECODE_PAGED_KV8, dims(S=1), kv_capacity=501)
    assert a > 0 and attend(ws_bytes=a - 1) == WORKSPACE
    assert n(L.OP_GQA_ATTENTION_DECODE_PAGED_KV8, dims(S=1), L.F32, kv_capacity=501) == 0
    assert n(L.OP_GQA_ATTENTION_DECODE_PAGED_KV8, dims(S=1, head_dim=96), kv_capacity=501) == 0
    assert n(L.OP_GQA_ATTENTION_DECODE_PAGED_KV8, dims(S=1, n_kv=0), kv_capacity=501) == 0
    # bounded whatever the lengths
    assert n(L.OP_GQA_ATTENTION_DECODE_PAGED_KV8, dims(S=1, B=64, n_q=32, n_kv=8), kv_capacity=1 << 24) < 1 << 26
    s = n(L.OP_BEAM_SELECT, dims(S=4), L.F32, vocab=100)
    assert s > 0 and select(ws_bytes=s - 1) == WORKSPACE
    assert n(L.OP_BEAM_SELECT, dims(S=33), L.F32, vocab=100) == 0 and n(L.OP_BEAM_SELECT, dims(S=0), L.F32, vocab=100) == 0
    assert n(L.OP_BEAM_SELECT, dims(B=48, S=8), L.F32, vocab=128256) < 1 << 24
    r = n(L.OP_BEAM_REORDER_PAGED, dims(S=4), kv_capacity=512)
    assert r > 0 and reorder(ws_bytes=r - 1) == WORKSPACE
    assert n(L.OP_BEAM_REORDER_PAGED, dims(S=4), kv_capacity=0) == 0


# ---------------------------------------------------------------------------------------- binding
def i32(*s):
    return meta(*s, dtype=torch.int32)


def f32(*s):
    return meta(*s, dtype=torch.float32)


def cache(n_pages=9, n_kv=2, hd=64, dtype=torch.uint8):
    return [meta(n_pages, 128, n_kv, hd, dtype=dtype), f32(n_pages, n_kv, 128), meta(n_pages, 128, n_kv, hd, dtype=dtype), f32(n_pages, n_kv, 128)]


D = L.dims_of(2, 1, 128, 8, 2, 64, 128, 1e4, 1e-5)


def test_binding_hands_over_what_it_is_given(note):  # noqa: F811
    for dtype in (torch.uint8, torch.float8_e4m3fn):
        L.llama_gqa_attention_decode_paged_kv8(D, meta(2, 8, 64), *cache(dtype=dtype), i32(2, 4), i32(2), 500, meta(2, 8, 64), None)
    qkv = meta(6, 12, 64)
    L.llama_rope_append_paged_kv8(L.dims_of(2, 6, 128, 8, 2, 64, 128, 1e4, 1e-5), OnView(qkv, (6, 8, 64)), OnView(qkv, (6, 2, 64)),
                                  OnView(qkv, (6, 2, 64)), i32(6), i32(6), meta(6, 8, 64), *cache())
    L.llama_kv_dequantize_paged(*cache(), i32(2, 4), i32(2), meta(9, 128, 2, 64), meta(9, 128, 2, 64))
    L.llama_beam_select(f32(8, 100), f32(2, 4), None, 0, i32(2, 6), i32(2, 6), f32(2, 6), None)
    L.llama_beam_reorder_paged(i32(2, 4), i32(8), i32(8), i32(8, 5), i32(8, 5), i32(7), 9, [meta(3, 9, 128, 2, 64), meta(9, 128, 2, 64)],
                               [f32(3, 9, 2, 128), f32(9, 2, 128)], i32(20), i32(2), None)
    names = [n for n, _ in note.calls]
    assert names == ["llama_gqa_attention_decode_paged_kv8"] * 2 + ["llama_rope_append_paged_kv8", "llama_kv_dequantize_paged",
                                                                   "llama_beam_select", "llama_beam_reorder_paged"]
    a = [x[1] for x in note.calls]
    assert a[0][6:9] == (9, 0x7000, 4) and a[0][10] == 500
    assert a[2][1:7] == (0x7000, 12 * 64) * 3 and a[2][14] == 9
    assert a[3][5:8] == (9, 0x7000, 4)
    assert a[4][1:5] == (2, 4, 100, 100) and a[4][6] is None and a[4][8] == 6
    pools = [(p.n_layers, p.parts, p.row_bytes) for p in a[5][11]]
    assert pools == [(3, 1, 256), (1, 1, 256), (3, 2, 4), (1, 2, 4)] and a[5][7] == 5 and a[5][9:11] == (7, 9) and a[5][14] == 20


class OnView:
    """A view of some heads of a fused projection's output."""

    def __init__(self, t, shape):
        self.t, self.shape, self.dtype, self.is_cuda, self.device = t, torch.Size(shape), t.dtype, True, t.device

    def get_device(self):
        return 0

    def stride(self):
        return self.t.stride()

    def data_ptr(self):
        return 0x7000


@pytest.mark.parametrize("call", [
    lambda: L.llama_gqa_attention_decode_paged_kv8(D, meta(2, 8, 64), *cache(dtype=torch.int8), i32(2, 4), i32(2), 500, meta(2, 8, 64), None),
    lambda: L.llama_gqa_attention_decode_paged_kv8(D, meta(2, 8, 64), *cache(n_kv=3), i32(2, 4), i32(2), 500, meta(2, 8, 64), None),
    lambda: L.llama_gqa_attention_decode_paged_kv8(D, meta(2, 8, 64), *cache(), i32(2, 4), i32(3), 500, meta(2, 8, 64), None),
    lambda: L.llama_gqa_attention_decode_paged_kv8(D, meta(2, 8, 64), *cache(), i32(2, 4), i32(2), 500, meta(2, 8, 32), None),
    lambda: L.llama_kv_dequantize_paged(*cache(), i32(3, 4), i32(2), meta(9, 128, 2, 64), meta(9, 128, 2, 64)),
    lambda: L.llama_kv_dequantize_paged(*cache(), i32(2, 4), i32(2), meta(9, 128, 2, 64), meta(9, 128, 2, 64, dtype=torch.float16)),
    lambda: L.llama_beam_select(f32(7, 100), f32(2, 4), None, 0, i32(2, 6), i32(2, 6), f32(2, 6), None),
    lambda: L.llama_beam_select(f32(8, 100), f32(2, 4), i32(8), 0, i32(2, 6), i32(2, 6), f32(2, 6), None),
    lambda: L.llama_beam_select(f32(8, 100), f32(2, 4), None, 0, i32(2, 6), i32(2, 5), f32(2, 6), None),
    lambda: L.llama_beam_reorder_paged(i32(2, 4), i32(7), i32(8), i32(8, 5), i32(8, 5), i32(7), 9, [], [], i32(20), i32(2), None),
    lambda: L.llama_beam_reorder_paged(i32(2, 4), i32(8), i32(8), i32(8, 5), i32(8, 4), i32(7), 9, [], [], i32(20), i32(2), None),
    lambda: L.llama_beam_reorder_paged(i32(2, 4), i32(8), i32(8), i32(8, 5), i32(8, 5), i32(7), 9, [meta(8, 128, 2, 64)], [], i32(20), i32(2), None),
    lambda: L.llama_beam_reorder_paged(i32(2, 4), i32(8), i32(8), i32(8, 5), i32(8, 5), i32(7), 9, [], [f32(9, 128, 2)], i32(20), i32(2), None)])
def test_binding_refuses(note, call):  # noqa: F811
    with pytest.raises(ValueError):
        call()
    assert not note.calls
