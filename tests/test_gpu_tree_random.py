"""Calls of the tree attention drawn at random: formats, shapes, lengths, holes, scales of both signs from 2^-126 to 2^100 of
the usual, queries of many sizes, the same row again and again, and unwritten drafts, against tests/tree_bounds.py."""
import numpy as np
import pytest

import synth
from tests import tree_bounds as B
from tests import tree_reference as R
from tests.test_gpu_tree import SM, case, launch
from tests.test_gpu_tree_edges import set_scale

pytestmark = pytest.mark.gpu


def draw(rng):
    fmt, heads = str(rng.choice(["int8", "fp8", "fp4"])), int(rng.choice([1, 2, 3, 8, 16, 20, 32, 64, 128]))
    many = rng.random() < 0.2
    nodes = int(rng.integers(1, 5 if many else (65 if rng.random() < 0.3 else 9)))
    batch = int(rng.integers(100, 300)) if many else int(rng.integers(1, 12))
    heads = min(heads, 16) if many else heads
    width = int(min(np.exp(rng.uniform(0, np.log(200 if many else 2000))), max(1, 3e7 / (batch * nodes * heads))))
    lens = [max(0, int(v)) for v in rng.integers(-2, width + 3, batch)]
    c = case(rng, fmt, batch, nodes, heads, width, lens, [int(v) for v in rng.integers(-1, nodes + 2, batch)], n_rows=700,
             q_scale=float(np.exp(rng.uniform(-6, 4))), holes=float(rng.choice([0, 0.1, 0.9])))
    sc = R.row_scales(c["cache"], np.arange(700), fmt)
    kind = rng.integers(0, 7)
    if kind == 1:                                                 # scales of many sizes and both signs, some zero
        sc = sc * 2.0 ** rng.uniform(-20, 20, 700) * rng.choice([1, -1, 0], 700, p=[0.9, 0.07, 0.03])
    elif kind == 2:                                               # a few far from the others
        sc[rng.integers(0, 700, 3)] = 2.0 ** rng.uniform(-100, 100, 3)
    elif kind == 3:                                               # all of them tiny
        sc = sc * 2.0 ** rng.uniform(-110, -60)
    elif kind == 4:                                               # in groups far apart
        sc = sc * 2.0 ** rng.choice([-126, -30, 0, 30, 60], 700)
    elif kind == 5:
        c["rows"] = np.where(c["rows"] >= 0, np.minimum(c["rows"], 3), -1).astype(np.int32)
    elif kind == 6:                                               # queries of many sizes
        q = synth.bf16_bits_to_f32(c["q"])
        c["q"] = synth.f32_to_bf16_bits(q * np.exp2(rng.integers(-60, 20, q.shape[:3] + (1,))).astype(np.float32))
    set_scale(c["cache"], np.arange(700), fmt, sc.astype(np.float32))
    if rng.random() < 0.5:                                        # drafts that nobody sees hold any bytes
        for b in range(batch):
            for j in range(nodes):
                if rng.random() < 0.3:
                    c["masks"][b] = [m & ~(1 << j) for m in c["masks"][b]]
                    c["draft"].view(np.uint8)[b * nodes + j] = rng.integers(0, 256, c["draft"].shape[1], dtype=np.uint8)
    return c


@pytest.mark.parametrize("seed", range(12))
def test_random_calls(cuda, seed):
    rng = np.random.default_rng(seed)
    for call in range(8):
        c = draw(rng)
        out, lse = launch(c, cuda)
        o, l = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
        q = synth.bf16_bits_to_f32(c["q"]).astype(np.float64)
        seqs = sorted({int(v) for v in rng.integers(0, len(q), 3)})
        for b, i, want, wl, tol, ltol in B.tree(c, SM, q, seqs):
            if not (np.abs(want) < 1e37).all() or not (np.abs(wl[np.isfinite(wl)]) < 1e30).all():
                continue                                          # (past fp32's or bf16's range)
            if np.isneginf(wl).all():
                assert np.isneginf(l[b, i]).all() and not o[b, i].any(), (call, b, i)
                continue
            # (a bf16 denormal is off by half its step of 2^-133 more, and one of fp32 beside it)
            assert (np.abs(o[b, i] - want) <= tol + 2.0 ** -133).all(), (call, b, i)
            assert (np.abs(l[b, i] - wl) <= ltol).all(), (call, b, i)
