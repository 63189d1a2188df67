"""What the binding of the paged serving calls hands to the library, with a library that only takes notes: no GPU."""
import pytest

import llama_decoder_block_fwd_gb300 as L

torch = pytest.importorskip("torch")


class Note:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append((name, a)) or 0


class OnDevice:
    """A tensor's metadata (a meta tensor) as if it lived on a CUDA device."""

    def __init__(self, t, device=0):
        self.t, self.dev = t, device
        self.is_cuda, self.device = device >= 0, torch.device("cuda", device) if device >= 0 else torch.device("cpu")
        self.shape, self.dtype = t.shape, t.dtype

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.dev

    def data_ptr(self):
        return 0x7000


def meta(*shape, dtype=torch.bfloat16, device=0):
    return OnDevice(torch.empty(*shape, dtype=dtype, device="meta"), device)


@pytest.fixture
def note(monkeypatch):
    n = Note()
    monkeypatch.setattr(L, "_here", lambda stream: (n, torch, 0, 0))
    return n


def chunk(ws):
    i32 = torch.int32
    L.llama_gqa_attention_chunk_paged(L.dims_of(2, 6, 128, 8, 2, 64, 128, 1e4, 1e-5), meta(6, 8, 64), meta(9, 128, 2, 64),
                                      meta(9, 128, 2, 64), meta(2, 4, dtype=i32), meta(3, dtype=i32), meta(2, dtype=i32),
                                      500, meta(6, 8, 64), ws)


def verify(ws):
    i32, f32 = torch.int32, torch.float32
    L.llama_verify_drafts(meta(6, 50, dtype=f32), None, 1.0, meta(3, dtype=i32), meta(6, dtype=i32), meta(6, dtype=f32),
                          meta(2, 50, dtype=f32), meta(2, dtype=i32), meta(6, dtype=i32), ws)


def bytes_on(t, device=0):
    return OnDevice(t, device)


@pytest.mark.parametrize("call", [chunk, verify])
def test_workspace_is_one_piece_of_this_devices_memory(note, call):
    raw = torch.empty(4096, dtype=torch.uint8, device="meta")
    call(bytes_on(raw))
    call(bytes_on(torch.empty(1024, dtype=torch.float32, device="meta")))      # any type: bytes count
    call(None)                                                                  # the library says what it lacks
    at = {"llama_gqa_attention_chunk_paged": slice(11, 13), "llama_verify_drafts": slice(15, 17)}
    assert [a[at[name]] for name, a in note.calls] == [(0x7000, 4096), (0x7000, 4096), (None, 0)]
    # as many elements as it takes, but not that much memory: what lies behind it would be written
    for bad, what in ((bytes_on(torch.empty(1, dtype=torch.uint8, device="meta").expand(4096)), "contiguous"),
                      (bytes_on(raw[::2]), "contiguous"), (bytes_on(raw, 1), "current device"),
                      (bytes_on(raw, -1), "CUDA tensor")):
        with pytest.raises(ValueError, match=what):
            call(bad)
    assert len(note.calls) == 3
