"""The chunk attention's own work-split code, compiled for the host (tests/chunk_units_host.cu): its divisions by
reciprocals, its cuts and its units, held to the invariants of tests/test_chunk_scheme.py.  No GPU is used."""
import ctypes
import os
import random
import subprocess

import pytest

from llama_decoder_block_fwd_gb300 import _build
from tests import test_chunk_scheme as scheme

HERE = os.path.dirname(os.path.abspath(__file__))
NONE = -2 ** 31                 # `part` of a unit that stores o
ULPS = [-2, -1, 0, 1, 2]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("units") / "units.so")
    subprocess.check_call([_build.nvcc(), *_build.ARCH, "-O1", "-std=c++17", "-Xcompiler", "-fPIC", "-shared",
                           "--expt-relaxed-constexpr", "-I", _build.CSRC, "-o", out, os.path.join(HERE, "chunk_units_host.cu")])
    return ctypes.CDLL(out)


def test_divisions(lib):
    r = random.Random(0)
    for ulps in ULPS:
        lib.host_ulps(ulps)
        for _ in range(20000):
            b = max(1, int(2 ** r.uniform(0, 21)))
            k = r.randrange(0, max(1, (1 << 22) // b))
            for a in (k * b, k * b + b - 1, max(0, k * b - 1), r.randrange(0, 1 << 22)):
                if a < 1 << 22:
                    assert lib.host_div_by(a, b) == a // b, (a, b, ulps)
    for _ in range(50000):
        b = max(1, int(2 ** r.uniform(0, 17)))
        k = r.randrange(0, max(1, (1 << 30) // b))
        for a in (k * b, min((1 << 30) - 1, k * b + b - 1), max(0, k * b - 1)):
            assert lib.host_div_inv(a, b) == a // b, (a, b)


def test_cuts(lib):
    """Chunks of at most C tiles, none of them empty, over the whole range of tiles and for every candidate."""
    out = (ctypes.c_int * 2)()
    r = random.Random(1)
    sizes = sorted({lib.host_candidate(w) for w in range(31)})
    assert sizes[:8] == [1, 2, 3, 4, 6, 8, 12, 16] and sizes[-1] == 1 << 15 and lib.host_candidate(31) > 1 << 17
    tiles = [*range(1, 300), *(r.randrange(300, 1 << 17) for _ in range(400)), (1 << 17) - 1, 1 << 17]
    for ulps in ULPS:
        lib.host_ulps(ulps)
        for C in [*sizes, lib.host_candidate(31)]:
            for nt in tiles:
                lib.host_cut(nt, C, out)
                nc, ct = out
                assert ct <= max(C, 1) and (nc - 1) * ct < nt <= nc * ct, (nt, C, nc, ct)
                assert (nc, ct) == scheme.cut(nt, C)


@pytest.mark.parametrize("seed", range(30))
def test_every_tile_in_one_unit(lib, monkeypatch, seed):
    """The scheme's invariants with the kernel's units in place of the model's."""
    r = random.Random(100 + seed)
    lib.host_ulps(r.choice(ULPS))
    order = ("unit0", "lo", "n", "c", "np", "wp", "span", "nc", "ct", "cut_n", "part0", "split0")
    out = (ctypes.c_int * 12)()

    def cut(nt, C):
        lib.host_cut(nt, C, out)
        return out[0], out[1]

    def make_unit(s, u, ratio, n_kv):
        if not lib.host_unit(ratio, n_kv, (ctypes.c_int * 12)(*(s[k] for k in order)), u, out):
            return None
        g, t0, n0, n1, lone, row0, row1, part, end, pos_off, kv_len, clean = out
        assert end == s["lo"] + s["n"] and pos_off == s["c"] - s["lo"] and kv_len == s["c"] + s["n"]
        # tiles before `clean` are seen whole by the unit's first row, tile `clean` is not
        assert 128 * clean <= row1 + pos_off + 1 < 128 * (clean + 1)
        return g, t0, n0, n1, bool(lone), (row0, row1), None if part == NONE else part

    monkeypatch.setattr(scheme, "cut", cut)
    monkeypatch.setattr(scheme, "make_unit", make_unit)
    ratio, n_kv = r.choice([(1, 2), (4, 2), (8, 1), (3, 1), (7, 3), (100, 1), (128, 1)])
    B = r.randrange(1, 7)
    new = [r.choice([0, 1, r.randrange(1, 9), r.randrange(1, 400 // min(ratio, 8))]) for _ in range(B)]
    cached = [r.choice([0, r.randrange(0, 300), r.randrange(0, 3000)]) for _ in range(B)]
    items = sum(scheme.cdiv(n, 2 * (128 // ratio)) for n in new)
    for C in (1, 2, 3, 6, 12, lib.host_candidate(31)):
        scheme.check_split(cached, new, ratio, n_kv, C, r.choice([0, r.randrange(0, items + 2)]), 2)
        scheme.check_split(cached, new, ratio, n_kv, C, 0, 1)
