"""The limits that the header states for the paged serving calls, each from both sides: refused beyond, and at the
limit found fault with only for what is left out on purpose (so that nothing is launched).  No GPU is used."""
import ctypes

import pytest

import llama_decoder_block_fwd_gb300 as L

FAKE = 0x10000          # aligned, never dereferenced
BIG = 1 << 62
OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = range(5)


def dims(**kw):
    base = dict(B=2, S=6, d_model=1024, n_q=8, n_kv=2, head_dim=128, d_ff=128, theta_base=1e4, eps=1e-5)
    base.update(kw)
    return L.dims_of(**base)


def plan(**kw):         # without cu_new: INVALID once the sizes are accepted
    a = dict(n_cached=FAKE, n_new=FAKE, B=2, free=FAKE, n_free=3, n_pages=9, table=FAKE, max_pages=4, n_tokens=6,
             cu=None, positions=FAKE, slots=FAKE, used=FAKE)
    a.update(kw)
    return L.lib().llama_paged_plan(*a.values(), None)


@pytest.mark.parametrize("name,most", [("B", 8192), ("n_pages", 2 ** 24 - 1), ("max_pages", 2 ** 17),
                                       ("n_tokens", 2 ** 30 - 1), ("n_free", 2 ** 31 - 1)])
def test_plan(name, most):
    assert plan(**{name: most}) == INVALID and plan(**{name: most + 1}) == UNSUPPORTED


def append(d, **kw):    # without slots: INVALID once the sizes are accepted
    w, wk = d.n_q * d.head_dim, d.n_kv * d.head_dim
    a = dict(q=FAKE, qs=w, k=FAKE, ks=wk, v=FAKE, vs=wk, positions=FAKE, slots=None, q_out=FAKE, kp=FAKE, vp=FAKE, n_pages=4)
    a.update(kw)
    return L.lib().llama_rope_append_paged(ctypes.byref(d), *a.values(), None)


def test_append():
    for good, bad in ((dict(n_q=4096), dict(n_q=4098)), (dict(n_q=4096, n_kv=4096), dict(n_q=4097, n_kv=4097)),
                      (dict(S=2 ** 31 - 9), dict(S=2 ** 31 - 7)), (dict(head_dim=256), dict(head_dim=264)),
                      (dict(head_dim=8), dict(head_dim=12))):
        assert append(dims(**good)) == INVALID and append(dims(**bad)) == UNSUPPORTED, (good, bad)
    assert append(dims(), n_pages=2 ** 24 - 1) == INVALID and append(dims(), n_pages=2 ** 24) == UNSUPPORTED
    assert append(dims(), slots=FAKE, qs=1024 + 4, q_out=FAKE + 4096) == ALIGNMENT


def chunk(d, **kw):     # without a workspace: WORKSPACE once the rest is accepted
    a = dict(q=FAKE, kp=FAKE, vp=FAKE, n_pages=8, table=FAKE, max_pages=4, cu=FAKE, cached=FAKE, max_pos=500, o=FAKE,
             ws=None, ws_bytes=BIG)
    a.update(kw)
    return L.lib().llama_gqa_attention_chunk_paged(ctypes.byref(d), *a.values(), None)


def test_chunk_attention():
    for good, bad in ((dict(S=2 ** 30 - 1), dict(S=2 ** 30)), (dict(B=2 ** 23 - 1), dict(B=2 ** 23)),
                      (dict(n_q=65536, n_kv=512), dict(n_q=131072, n_kv=1024)), (dict(n_q=128, n_kv=1), dict(n_q=129, n_kv=1)),
                      # 128 heads per group: one token per Q tile, so S / 2 items per group
                      (dict(B=1, S=2 ** 27 - 2, n_q=512, n_kv=4), dict(B=2, S=2 ** 27 - 2, n_q=512, n_kv=4)),
                      (dict(head_dim=64), dict(head_dim=32))):
        assert chunk(dims(**good)) == WORKSPACE and chunk(dims(**bad)) == UNSUPPORTED, (good, bad)
    assert chunk(dims(), n_pages=2 ** 24 - 1) == WORKSPACE and chunk(dims(), n_pages=2 ** 24) == UNSUPPORTED
    assert chunk(dims(), max_pages=2 ** 31 - 1) == WORKSPACE and chunk(dims(), max_pages=2 ** 31) == UNSUPPORTED
    assert chunk(dims(), max_pos=511) == WORKSPACE and chunk(dims(), max_pos=512) == INVALID
    far = dict(max_pages=2 ** 18)
    assert chunk(dims(), max_pos=2 ** 24 - 1, **far) == WORKSPACE and chunk(dims(), max_pos=2 ** 24, **far) == INVALID


def verify(**kw):       # without a workspace: WORKSPACE once the rest is accepted
    a = dict(z=FAKE, T=6, V=100, ld=BIG, y=FAKE, ldy=BIG, temp=1.0, cu=FAKE, B=2, tokens=FAKE, u=FAKE, noise=FAKE, ldn=BIG,
             n_acc=FAKE, out=FAKE, ws=None, ws_bytes=BIG)
    a.update(kw)
    return L.lib().llama_verify_drafts(*a.values(), None)


def test_verify():
    assert verify(T=2 ** 29 - 1, V=1024) == WORKSPACE and verify(T=2 ** 29, V=1024) == UNSUPPORTED
    assert verify(T=2 ** 29 - 1, V=1025) == UNSUPPORTED
    assert verify(B=2 ** 27 - 1) == WORKSPACE and verify(B=2 ** 27) == UNSUPPORTED
    assert verify(V=2 ** 30) == WORKSPACE and verify(V=2 ** 30 + 1) == INVALID
