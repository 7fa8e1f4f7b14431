"""The tree attention (glm_tree_mla_decode, _fp8, _fp4) against its fp64 reference.

Outputs are poisoned first; every element must be written and lie within the error derived in
tests/tree_reference.py.
"""
import numpy as np
import pytest
import torch

import kpool_indexer_int8_b200 as kp
import oracle
import synth
from tests import tree_reference as R

pytestmark = pytest.mark.gpu

STORE = {"int8": oracle.store_int8, "fp8": oracle.store_fp8, "fp4": oracle.store_fp4}
CALL = {"int8": kp.glm_tree_mla_decode, "fp8": kp.glm_tree_mla_decode_fp8, "fp4": kp.glm_tree_mla_decode_fp4}
SM = float(np.float32(512 ** -0.5))


def make_rows(rng, n, fmt, outliers=0.02):
    x = rng.standard_normal((n, 512)).astype(np.float32)
    x[rng.random(n) < outliers] *= 8
    cache = np.zeros((n, R.ROW[fmt]), np.int8 if fmt == "int8" else np.uint8)
    if n:
        STORE[fmt](synth.f32_to_bf16_bits(x), np.arange(n, dtype=np.int64), cache)
    return cache


def tree_masks(rng, T):
    m = []
    for i in range(T):
        p = int(rng.integers(-1, i)) if i else -1
        m.append((m[p] if p >= 0 else 0) | (1 << i))
    return m


def as_int64(masks):
    return torch.tensor([[v - (1 << 64) if v >= 1 << 63 else v for v in row] for row in masks], dtype=torch.int64)


def bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16)


def case(rng, fmt, B, T, H, width, lens, n_tree, n_rows=3000, q_scale=1.0, holes=0.0):
    """Inputs on the host: random distinct rows, `holes` of the list's entries -1."""
    rows = np.full((B, max(width, 0)), -1, np.int32)
    for b in range(B):
        n = min(lens[b], width)
        rows[b, :n] = rng.choice(n_rows, size=n, replace=n > n_rows)
        if holes:
            rows[b, :n][rng.random(n) < holes] = -1
    return dict(fmt=fmt, cache=make_rows(rng, n_rows, fmt), draft=make_rows(rng, B * T, fmt), rows=rows,
                row_len=np.array(lens, np.int32), n_tree=np.array(n_tree, np.int32),
                masks=[tree_masks(rng, T) for _ in range(B)],
                q=synth.f32_to_bf16_bits((rng.standard_normal((B, T, H, 512)) * q_scale).astype(np.float32)))


def launch(c, dev, sm=SM, ws=None, out=None, lse=None, **kw):
    B, T, H = c["q"].shape[:3]
    dims = kp.make_dims(H)
    need = kp.glm_dsa_workspace_size(dims, kp.GLM_OP_TREE_MLA, B, select_k=T, width=c["rows"].shape[1])
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=dev) if ws is None else ws
    ws[need - 256:need].zero_()
    out = torch.full((B, T, H, 512), 7.0, dtype=torch.bfloat16, device=dev) if out is None else out
    lse = torch.full((B, T, H), 7.0, dtype=torch.float32, device=dev) if lse is None else lse
    CALL[c["fmt"]](dims, bf16(c["q"]).to(dev), torch.from_numpy(c["cache"]).to(dev), torch.from_numpy(c["rows"]).to(dev),
                   torch.from_numpy(c["draft"]).to(dev), as_int64(c["masks"]).to(dev), sm, out, ws, lse=lse,
                   row_len=torch.from_numpy(c["row_len"]).to(dev), n_tree=torch.from_numpy(c["n_tree"]).to(dev), **kw)
    torch.cuda.synchronize()
    assert int(ws[need - 256:need - 252].view(torch.int32).item()) == 0
    return out, lse


def check(c, out, lse, sm=SM):
    o = out.float().cpu().numpy().astype(np.float64)
    l = lse.cpu().numpy().astype(np.float64)
    q = synth.bf16_bits_to_f32(c["q"]).astype(np.float64)
    worst = 0.0
    for b, i, want, wl, tol, ltol in R.tree(q, c["cache"], c["rows"], c["row_len"], c["draft"], c["masks"], c["n_tree"],
                                            sm, c["fmt"]):
        err = np.abs(o[b, i] - want)
        assert (err <= tol).all(), (b, i, float((err / tol).max()), float(err.max()))
        if np.isneginf(wl).all():
            assert np.isneginf(l[b, i]).all() and not o[b, i].any()
        else:
            assert (np.abs(l[b, i] - wl) <= ltol).all(), (b, i, float((np.abs(l[b, i] - wl) / ltol).max()))
        worst = max(worst, float((err / tol).max()))
    return worst


@pytest.mark.parametrize("fmt", ["int8", "fp8", "fp4"])
@pytest.mark.parametrize("B,T,H,width,lens,n_tree", [
    (1, 1, 16, 80, [67], [1]),                       # one token, one tile and its own row
    (1, 4, 16, 80, [67], [4]),
    (1, 1, 1, 5, [1], [1]),                          # one head, one entry
    (2, 3, 8, 64, [64, 63], [3, 2]),                 # 24 query rows; a full tile, one short of it
    (1, 8, 64, 2176, [2051], [8]),                   # the selection of a long context
    (4, 13, 64, 4096, [7, 64, 1027, 4096], [13, 1, 5, 12]),
    (3, 64, 20, 200, [200, 0, 129], [64, 33, 0]),    # every node; no prefix; no tree
    (2, 5, 128, 130, [130, 65], [5, 4]),
    (5, 2, 3, 40, [40, 1, 2, 39, 0], [2, 2, 1, 0, 2]),
])
def test_tree_matches_reference(cuda, fmt, B, T, H, width, lens, n_tree):
    rng = np.random.default_rng(1000 * B + 100 * T + H + width)
    c = case(rng, fmt, B, T, H, width, lens, n_tree, holes=0.1 if width > 100 else 0.0)
    check(c, *launch(c, cuda))
