"""The tree attention writes nothing behind a workspace of the exact size, and needs no more for its results."""
import numpy as np
import pytest
import torch

import kpool_indexer_int8_b200 as kp
from tests.test_gpu_tree import CALL, case
from tests.test_gpu_tree_edges import device_args

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T,H,width", [(1, 2, 8, 3000), (5, 1, 16, 2000), (8, 6, 4, 1500), (4, 6, 10, 3000), (1, 8, 64, 2176),
                                         (6, 3, 64, 2176), (3, 13, 64, 4096), (30, 2, 64, 8192), (2, 64, 2, 40000)])
def test_nothing_behind_the_workspace_is_written(cuda, B, T, H, width):
    dims = kp.make_dims(H)
    lens = [width - 97 * (i % 7) for i in range(B)]
    c = case(np.random.default_rng(B + H + width), "int8", B, T, H, width, lens, [T] * B, n_rows=400)
    d = device_args(c, cuda, dims)
    n = d["workspace"].numel()
    guarded = torch.full((n + (1 << 25),), 0xA5, dtype=torch.uint8, device=cuda)
    d["workspace"] = guarded[:n]
    guarded[n - 256:n] = 0
    CALL["int8"](dims, **d)
    torch.cuda.synchronize()
    assert bool((guarded[n:] == 0xA5).all()) and not bool(guarded[n - 256:n].any())
    out, lse = torch.full_like(d["out"], 3.0), torch.full_like(d["lse"], 3.0)
    CALL["int8"](dims, **dict(d, out=out, lse=lse, workspace=torch.zeros(n + (1 << 25), dtype=torch.uint8, device=cuda)))
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), d["out"].view(torch.int16)) and torch.equal(lse, d["lse"])
