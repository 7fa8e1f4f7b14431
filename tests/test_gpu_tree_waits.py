"""A wait of the tree attention on its tensor cores gives up without a fault.

Every wait is a bounded poll. When one runs out, the CTA goes on without its later waits, but for the products still in
flight, sets bit 32 (one CTA a run) or 64 (pairs of CTAs) of the status word at the end of the workspace and
returns. The test has every wait give up at once through the library's test hook (nothing is left unset, faults or
traps), reads the status, and checks that the next calls are right."""
import numpy as np
import pytest
import torch

import kpool_indexer_int8_b200 as kp
from tests.test_gpu_tree import CALL, case, check
from tests.test_gpu_tree_edges import device_args

pytestmark = pytest.mark.gpu


# tiles of 16, 32, 64 and 128 query rows; one tile, several, and runs that are merged
@pytest.mark.parametrize("B,T,H,width,bit", [(1, 2, 8, 40, 32), (1, 2, 8, 3000, 32), (8, 6, 4, 700, 32), (4, 6, 10, 700, 32),
                                             (150, 6, 10, 150, 32), (1, 2, 64, 80, 32), (10, 8, 64, 700, 64), (2, 6, 40, 1500, 64)])
@pytest.mark.parametrize("fmt", ["int8", "fp4"])
def test_waits_give_up_with_a_status_and_no_fault(cuda, fmt, B, T, H, width, bit):
    dims = kp.make_dims(H)
    c = case(np.random.default_rng(B + H + width), fmt, B, T, H, width, [width] * B, [T] * B, n_rows=400)
    d = device_args(c, cuda, dims)
    status = d["workspace"][-256:-252].view(torch.int32)
    try:
        kp.glm_debug_tree_waits_give_up(True)
        CALL[fmt](dims, **d)
        torch.cuda.synchronize()
    finally:
        kp.glm_debug_tree_waits_give_up(False)
    assert int(status.item()) == bit
    status.zero_()
    for _ in range(2):
        CALL[fmt](dims, **d)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    check(c, d["out"], d["lse"])


def test_the_status_word_is_at_the_end_of_a_larger_workspace(cuda):
    # one workspace for calls of different shapes: their status words are one, and no call's partials lie over it
    big = case(np.random.default_rng(1), "int8", 2, 4, 64, 3000, [3000] * 2, [4] * 2, n_rows=400)
    small = case(np.random.default_rng(2), "int8", 1, 2, 8, 300, [300], [2], n_rows=400)
    b, s = device_args(big, cuda, kp.make_dims(64)), device_args(small, cuda, kp.make_dims(8))
    n = b["workspace"].numel()
    assert s["workspace"].numel() < n - 256
    for extra in (0, 100):                                        # (a size that is no multiple of 256 too)
        ws = torch.full((n + extra,), 0xFF, dtype=torch.uint8, device=cuda)
        status = ws[n - 256:n - 252].view(torch.int32)
        status.zero_()
        b["workspace"] = s["workspace"] = ws
        try:
            kp.glm_debug_tree_waits_give_up(True)
            CALL["int8"](kp.make_dims(8), **s)
            torch.cuda.synchronize()
        finally:
            kp.glm_debug_tree_waits_give_up(False)
        assert int(status.item()) == 32
        status.zero_()
        CALL["int8"](kp.make_dims(64), **b)
        CALL["int8"](kp.make_dims(8), **s)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        check(big, b["out"], b["lse"])
        check(small, s["out"], s["lse"])
