"""The paged serving calls on the host: bad arguments are refused with a status code before anything
is launched, and the binding refuses tensors that the library would misread.  No GPU is used."""
import ctypes

import pytest

import llama_decoder_block_fwd_gb300 as L

FAKE = 0x10000          # aligned, never dereferenced: validation fails before any launch
BIG = 1 << 40
INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 4


def _dims(**kw):
    base = dict(B=2, S=6, d_model=1024, n_q=8, n_kv=2, head_dim=128, d_ff=128, theta_base=1e4, eps=1e-5)
    base.update(kw)
    return L.dims_of(**base)


def _plan(**kw):
    a = dict(n_cached=FAKE, n_new=FAKE, B=2, free=FAKE, n_free=3, n_pages=9, table=FAKE, max_pages=4, n_tokens=6,
             cu=FAKE, positions=FAKE, slots=FAKE, used=FAKE)
    a.update(kw)
    return L.lib().llama_paged_plan(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), INVALID), (dict(n_free=-1), INVALID), (dict(n_pages=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(n_tokens=-1), INVALID), (dict(B=8193), UNSUPPORTED), (dict(n_pages=1 << 24), UNSUPPORTED),
    (dict(max_pages=(1 << 17) + 1), UNSUPPORTED), (dict(n_tokens=1 << 31), UNSUPPORTED),
    (dict(n_cached=None), INVALID), (dict(n_new=None), INVALID), (dict(free=None), INVALID), (dict(table=None), INVALID),
    (dict(cu=None), INVALID), (dict(positions=None), INVALID), (dict(slots=None), INVALID), (dict(used=None), INVALID),
    (dict(slots=FAKE + 2), ALIGNMENT), (dict(table=FAKE + 1), ALIGNMENT)])
def test_plan_refuses(kw, want):
    assert _plan(**kw) == want


def _append(dims=None, **kw):
    a = dict(q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, positions=FAKE, slots=FAKE, q_out=FAKE + 4096, kp=FAKE,
             vp=FAKE, n_pages=4)
    a.update(kw)
    return L.lib().llama_rope_append_paged(ctypes.byref(dims or _dims()), *a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(dims=_dims(head_dim=100)), UNSUPPORTED), (dict(dims=_dims(n_kv=3)), INVALID), (dict(q=None), INVALID),
    (dict(q_out=None), INVALID), (dict(k=None), INVALID), (dict(vp=None), INVALID), (dict(qs=1016), INVALID),
    (dict(ks=248), INVALID), (dict(vs=8), INVALID), (dict(qs=1536, q_out=FAKE), INVALID), (dict(n_pages=0), INVALID),
    (dict(n_pages=1 << 24), UNSUPPORTED), (dict(positions=None), INVALID), (dict(slots=None), INVALID),
    (dict(qs=1028), ALIGNMENT), (dict(ks=260), ALIGNMENT), (dict(q=FAKE + 8), ALIGNMENT), (dict(kp=FAKE + 2), ALIGNMENT),
    (dict(slots=FAKE + 2), ALIGNMENT), (dict(dims=_dims(S=0)), 0),
    (dict(q=None, q_out=None, k=None, v=None, kp=None, vp=None), 0)])
def test_append_refuses(kw, want):
    assert _append(**kw) == want


def _chunk(dims=None, **kw):
    a = dict(q=FAKE, kp=FAKE, vp=FAKE, n_pages=8, table=FAKE, max_pages=4, cu=FAKE, cached=FAKE, max_pos=500, o=FAKE,
             ws=FAKE, ws_bytes=BIG)
    a.update(kw)
    return L.lib().llama_gqa_attention_chunk_paged(ctypes.byref(dims or _dims()), *a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(dims=_dims(n_kv=3)), INVALID), (dict(n_pages=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(max_pos=-1), INVALID), (dict(max_pos=512), INVALID), (dict(n_pages=1 << 24), UNSUPPORTED),
    (dict(dims=_dims(head_dim=96)), UNSUPPORTED), (dict(dims=_dims(n_q=129, n_kv=1)), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(kp=None), INVALID), (dict(vp=None), INVALID), (dict(table=None), INVALID),
    (dict(cu=None), INVALID), (dict(cached=None), INVALID), (dict(o=None), INVALID), (dict(q=FAKE + 8), ALIGNMENT),
    (dict(vp=FAKE + 2), ALIGNMENT), (dict(cu=FAKE + 2), ALIGNMENT), (dict(ws=None), WORKSPACE),
    (dict(ws_bytes=16), WORKSPACE), (dict(ws=FAKE + 4), ALIGNMENT), (dict(dims=_dims(B=0)), 0), (dict(dims=_dims(S=0)), 0)])
def test_chunk_attention_refuses(kw, want):
    assert _chunk(**kw) == want


def _verify(**kw):
    a = dict(z=FAKE, T=6, V=100, ld=100, y=FAKE, ldy=100, temp=1.0, cu=FAKE, B=2, tokens=FAKE, u=FAKE, noise=FAKE, ldn=100,
             n_acc=FAKE, out=FAKE, ws=FAKE, ws_bytes=BIG)
    a.update(kw)
    return L.lib().llama_verify_drafts(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(V=0), INVALID), (dict(ld=99), INVALID), (dict(ldy=99), INVALID),
    (dict(ldn=99), INVALID), (dict(temp=float("nan")), INVALID), (dict(T=1 << 31), UNSUPPORTED),
    (dict(T=1 << 20, V=1 << 30, ld=1 << 30, ldy=1 << 30, ldn=1 << 30), UNSUPPORTED), (dict(z=None), INVALID),
    (dict(cu=None), INVALID), (dict(tokens=None), INVALID), (dict(u=None), INVALID), (dict(noise=None), INVALID),
    (dict(n_acc=None), INVALID), (dict(out=None), INVALID), (dict(z=FAKE + 2), ALIGNMENT), (dict(u=FAKE + 1), ALIGNMENT),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=8), WORKSPACE), (dict(ws=FAKE + 4), ALIGNMENT), (dict(B=0), 0)])
def test_verify_refuses(kw, want):
    assert _verify(**kw) == want


def test_rows_times_sequences_are_no_limit():
    """B counts sequences and S packed rows: a large batch of many rows is refused for nothing but its arguments."""
    big = _dims(B=8192, S=1 << 20)
    assert _chunk(dims=big, ws=None) == WORKSPACE and _append(dims=big, slots=None) == INVALID
    assert L.llama_workspace_bytes(L.OP_GQA_ATTENTION_CHUNK_PAGED, big, L.BF16, kv_capacity=500) > 0
    assert _chunk(dims=_dims(B=-1)) == INVALID and _append(dims=_dims(B=-1)) == INVALID
    assert _plan(n_tokens=1 << 30) == UNSUPPORTED


def test_workspace_sizes():
    d = _dims()
    small = L.llama_workspace_bytes(L.OP_GQA_ATTENTION_CHUNK_PAGED, d, L.BF16, kv_capacity=500)
    assert small > 0
    assert L.llama_workspace_bytes(L.OP_GQA_ATTENTION_CHUNK_PAGED, d, L.F32, kv_capacity=500) == 0
    assert L.llama_workspace_bytes(L.OP_GQA_ATTENTION_CHUNK_PAGED, _dims(head_dim=96), L.BF16, kv_capacity=500) == 0
    assert _chunk(ws_bytes=small - 1) == WORKSPACE
    # the scratch is bounded whatever the lengths: a long prompt, a long cache, many sequences
    for dims, cap in ((_dims(B=1, S=65536, n_q=32, n_kv=8), 1 << 20), (_dims(B=1, S=1, n_q=32, n_kv=8), 1 << 24),
                      (_dims(B=512, S=512, n_q=32, n_kv=8), 1 << 17)):
        assert 0 < L.llama_workspace_bytes(L.OP_GQA_ATTENTION_CHUNK_PAGED, dims, L.BF16, kv_capacity=cap) < 1 << 30
    v = L.llama_workspace_bytes(L.OP_VERIFY_DRAFTS, _dims(S=6), L.F32, vocab=100)
    assert v > 0 and _verify(ws_bytes=v - 1) == WORKSPACE
    assert L.llama_workspace_bytes(L.OP_VERIFY_DRAFTS, _dims(S=0), L.F32, vocab=100) == 0


def test_binding_refuses_what_the_library_would_misread():
    torch = pytest.importorskip("torch")

    class Fake:                       # what the checks look at, without device memory
        def __init__(self, shape, dtype, strides, device=0):
            self.shape, self.dtype, self._st, self._dev = torch.Size(shape), dtype, strides, device
            self.is_cuda, self.device = device >= 0, f"cuda:{device}" if device >= 0 else "cpu"

        def stride(self):
            return self._st

        def get_device(self):
            return self._dev

        def is_contiguous(self):
            return self._st == tuple(torch.empty(self.shape, device="meta").stride())

        def dim(self):
            return len(self.shape)

        def data_ptr(self):
            return 0x1000

    from llama_decoder_block_fwd_gb300 import _arg, _heads, _matrix
    bf, f32 = torch.bfloat16, torch.float32
    assert _arg("f", "x", Fake((4, 3), f32, (3, 1)), f32, 0, (4, 3)) == 0x1000
    assert _arg("f", "x", None, f32, 0) is None and _arg("f", "x", 0x20, f32, 0) == 0x20
    for bad, what in ((Fake((4, 3), bf, (3, 1)), "float32"), (Fake((4, 3), f32, (6, 1)), "contiguous"),
                      (Fake((4, 2), f32, (2, 1)), "shape"), (Fake((4, 3), f32, (3, 1), 1), "current device"),
                      (Fake((4, 3), f32, (3, 1), -1), "CUDA tensor")):
        with pytest.raises(ValueError, match=what):
            _arg("f", "x", bad, f32, 0, (4, 3))
    view = lambda *a, **k: _heads("f", "q", Fake(*a, **k), bf, 0, 4, 2, 64)
    assert _heads("f", "q", None, bf, 0, 4, 2, 64) == (None, 0)
    assert view((4, 2, 64), bf, (512, 64, 1)) == (0x1000, 512)
    assert _heads("f", "q", Fake((1, 2, 64), bf, (0, 64, 1)), bf, 0, 1, 2, 64) == (0x1000, 128)
    assert _heads("f", "q", Fake((4, 1, 64), bf, (80, 5, 1)), bf, 0, 4, 1, 64) == (0x1000, 80)
    for bad in (((4, 2, 64), torch.float16, (512, 64, 1)), ((4, 2, 64), bf, (512, 32, 1)), ((4, 2, 64), bf, (512, 64, 2)),
                ((4, 3, 64), bf, (512, 64, 1))):
        with pytest.raises(ValueError):
            view(*bad)
    with pytest.raises(ValueError):
        view((4, 2, 64), bf, (512, 64, 1), device=1)
    mat = lambda *a, **k: _matrix("f", "z", Fake(*a, **k), f32, 0, 4, 10)
    assert mat((4, 12), f32, (16, 1)) == (0x1000, 16)
    assert _matrix("f", "z", Fake((1, 12), f32, (0, 1)), f32, 0, 1, 10) == (0x1000, 10)
    assert _matrix("f", "z", Fake((0, 12), f32, (0, 0)), f32, 0, 0, 10) == (0x1000, 10)    # no rows, no strides
    assert _heads("f", "q", Fake((0, 2, 64), bf, (0, 0, 0)), bf, 0, 0, 2, 64) == (0x1000, 128)
    for bad in (((4, 9), f32, (9, 1)), ((4, 12), f32, (16, 2)), ((3, 12), f32, (12, 1)), ((4, 12), bf, (12, 1)),
                ((48,), f32, (1,))):
        with pytest.raises(ValueError):
            mat(*bad)
