"""A paged cache of more arrays than one reordering call takes: several calls on the same inputs, the last one in place."""
import numpy as np
import pytest

import llama_decoder_block_fwd_gb300 as L
from tests.test_gpu_beam import Beams, _bdims, _dev, _i32, _status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [8, 16])
def test_layers_in_pools_of_their_own(bits):
    import torch
    layers = 5
    b = Beams(3, 4, [[229, 101, 355, 383], [127] * 4, [130, 1, 2, 200]], 2, 64, layers=layers, bits=bits, seed=1)
    parents = [[0, 0, 2, 3], [1, 1, 1, 1], [3, 0, 3, 3]]
    kv, sc = [_dev(x) for x in b.kv], [_dev(x) for x in b.sc]
    n, table = _i32(b.n_cached), _i32(b.table)
    freed = torch.full((b.B * b.W * b.P,), -8, dtype=torch.int32, device="cuda")
    counts = torch.full((2,), -8, dtype=torch.int32, device="cuda")
    ws = torch.full((L.llama_workspace_bytes(L.OP_BEAM_REORDER_PAGED, _bdims(b.B, b.W), L.BF16, kv_capacity=128 * b.P),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    for layer in range(layers):
        last = layer == layers - 1
        n_out, out = (n, table) if last else (torch.full_like(n, -9), torch.full_like(table, -4))
        L.llama_beam_reorder_paged(_i32(parents).view(b.B, b.W), n, n_out, table, out, _i32(b.free), b.n_pages, [x[layer] for x in kv],
                                   [x[layer] for x in sc], freed, counts, ws)
        if not last:
            keep = out.cpu().numpy()
    assert _status() == 0
    b.check(parents, (n_out, out, freed, counts, kv, sc), in_place=True)
    held = keep != -4                                   # what the calls before it wrote is what it wrote
    np.testing.assert_array_equal(keep[held], out.cpu().numpy()[held])
