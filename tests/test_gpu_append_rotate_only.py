"""RoPE at per-token positions without a pool: a row is rotated when its slot is not negative, whatever it is."""
import pytest

import llama_decoder_block_fwd_gb300 as L

pytestmark = pytest.mark.gpu


def test_rotate_only_takes_any_slot():
    import torch
    slots = [0, 7, 2 ** 31 - 129, 2 ** 31 - 128, 2 ** 31 - 1, -1, -2 ** 31]
    T, n_q, hd = len(slots), 2, 64
    gen = torch.Generator().manual_seed(1)
    q = torch.randn((T, n_q, hd), generator=gen).bfloat16().cuda()
    pos = torch.arange(40, 40 + T, dtype=torch.int32, device="cuda")
    dims = L.dims_of(1, T, 128, n_q, 1, hd, 128, 1e4, 1e-5)
    want, got = torch.full_like(q, 9.0), torch.full_like(q, 9.0)
    L.llama_rope_append_paged(dims, q, None, None, pos, torch.zeros(T, dtype=torch.int32, device="cuda"), want, None, None)
    L.llama_rope_append_paged(dims, q, None, None, pos, torch.tensor(slots, dtype=torch.int32, device="cuda"), got, None,
                              None)
    assert L.llama_get_device_status() == 0
    live = torch.tensor([s >= 0 for s in slots])
    assert torch.equal(got[live], want[live]) and bool((got[~live] == 9.0).all())
