"""The softmax weights of the tree attention: a node's output depends on the rows that it sees, each by what it weighs.

Rows that a node does not see, and rows that it sees but that weigh nothing, may have scales far above the others',
without an effect on its output. Errors allowed: those of tests/tree_bounds.py, from the rows seen alone."""
import numpy as np
import pytest

import synth
from tests import tree_bounds as B
from tests import tree_reference as R
from tests.test_gpu_tree import SM, STORE, case, launch
from tests.test_gpu_tree_edges import set_scale

pytestmark = pytest.mark.gpu

FLT_MAX = float(np.finfo(np.float32).max)

# (batch, nodes, heads, width): the kernels' tiles of 16, 32, 64 and 128 query rows, one run of keys or several
CUTS = [(2, 6, 4, 70), (8, 6, 4, 700), (4, 6, 10, 700), (150, 6, 10, 70), (2, 6, 40, 70), (2, 6, 40, 1500)]


def check(c, out, lse, nodes=None, sm=SM, bits=11):
    """The nodes (None: all) of a call's first two and last sequences against the bounds."""
    o, l = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    q = synth.bf16_bits_to_f32(c["q"]).astype(np.float64)
    for b, i, want, wl, tol, ltol in B.tree(c, sm, q, sorted({0, 1, len(q) - 1} & set(range(len(q)))), bits):
        if nodes is not None and i not in nodes:
            continue
        if np.isneginf(wl).all():
            assert np.isneginf(l[b, i]).all() and not o[b, i].any(), (b, i)
            continue
        err = np.abs(o[b, i] - want)
        assert (err <= tol).all(), (b, i, float((err / tol).max()), float(err.max()))
        assert (np.abs(l[b, i] - wl) <= ltol).all(), (b, i, float((np.abs(l[b, i] - wl) / ltol).max()))



@pytest.mark.parametrize("fmt", ["int8", "fp8", "fp4"])
@pytest.mark.parametrize("cut", CUTS)
def test_random_rows(cuda, fmt, cut):
    b, T, H, width = cut
    rng = np.random.default_rng(H + width)
    c = case(rng, fmt, b, T, H, width, [width - i % 60 for i in range(b)], [T - i % 3 for i in range(b)], n_rows=700, holes=0.05)
    check(c, *launch(c, cuda))


@pytest.mark.parametrize("fmt", ["int8", "fp8", "fp4"])
@pytest.mark.parametrize("cut", CUTS)
@pytest.mark.parametrize("value", [2.0 ** 16, 2.0 ** 30, 1e30, FLT_MAX])
def test_drafts_that_a_node_does_not_see(cuda, fmt, cut, value):
    # drafts 1 and 4 hold scales of any finite size; node 5 is padding of the tree, with no bit set anywhere
    b, T, H, width = cut
    rng = np.random.default_rng(H + width + 1)
    c = case(rng, fmt, b, T, H, width, [width - i % 60 for i in range(b)], [T] * b, n_rows=700)
    for s in range(b):
        set_scale(c["draft"], [s * T + 1, s * T + 4, s * T + 5], fmt, value)
    c["masks"] = [[0b000001, 0b000010, 0b000101, 0b001001, 0b011001, 0]] * b
    check(c, *launch(c, cuda), nodes=(0, 2, 3, 5))


@pytest.mark.parametrize("fmt", ["int8", "fp8", "fp4"])
@pytest.mark.parametrize("cut", CUTS)
@pytest.mark.parametrize("ratio", [2.0 ** 10, 2.0 ** 20, 2.0 ** 100])
@pytest.mark.parametrize("first", [True, False])
def test_rows_that_are_seen_and_weigh_nothing(cuda, fmt, cut, ratio, first):
    # a row of the list far above the others in scale and far below them in score, at the start or the middle of it
    b, T, H, width = cut
    rng = np.random.default_rng(H + width + 2)
    c = case(rng, fmt, b, T, H, width, [width] * b, [T] * b, n_rows=700)
    q = synth.bf16_bits_to_f32(c["q"]) + np.float32(0.5)          # (a positive sum over the dims, so that ...)
    c["q"] = synth.f32_to_bf16_bits(q)
    raw = c["cache"].view(np.uint8)
    raw[7, :288 if fmt == "fp4" else 512] = {"int8": 0x9C, "fp8": 0xFE, "fp4": 0xAA}[fmt]       # (... -100, -448, -1 give a low score)
    if fmt == "fp4":
        raw[7, 256:288] = 0x7E                                   # (block scales of 448)
    typical = float(np.median(R.row_scales(c["cache"], np.arange(700), fmt)))
    c["rows"][c["rows"] == 7] = 8
    c["rows"][:, 0 if first else width // 2] = 7
    set_scale(c["cache"], [7], fmt, typical * ratio)
    s = R.values(c["cache"], [7], fmt)[0] @ synth.bf16_bits_to_f32(c["q"]).astype(np.float64).reshape(-1, 512).T * SM
    assert s.max() < -150.0                                       # (far below any other row's)
    check(c, *launch(c, cuda))


@pytest.mark.parametrize("fmt", ["int8", "fp8", "fp4"])
@pytest.mark.parametrize("cut", CUTS)
@pytest.mark.parametrize("order", [1, -1])
def test_scales_and_scores_that_move_against_each_other(cuda, fmt, cut, order):
    # scales from 2^-12 to 2^6 of the usual along the list, queries so large that the scores move with them
    b, T, H, width = cut
    rng = np.random.default_rng(H + width + 3)
    c = case(rng, fmt, b, T, H, width, [width] * b, [T] * b, n_rows=700, q_scale=4.0)
    sc = R.row_scales(c["cache"], np.arange(700), fmt)
    set_scale(c["cache"], np.arange(700), fmt, (sc * 2.0 ** np.linspace(-12, 6, 700)).astype(np.float32))
    c["rows"] = np.sort(c["rows"], axis=1)[:, ::order].copy()
    check(c, *launch(c, cuda))


@pytest.mark.parametrize("fmt", ["int8", "fp8", "fp4"])
@pytest.mark.parametrize("H", [4, 20, 60, 80])
def test_a_long_tail_far_below_the_peaks(cuda, fmt, H):
    # 262,144 rows: in every 1,024 one row 12 to 20 nats above the others, which all weigh the same and alone hold
    # values in the upper dims; one of them in 63 with a scale eight times the others'
    n = 1 << 18
    x = np.zeros((64, 512), np.float32)
    x[0, :256] = 1.0
    x[1:, 256:] = 1.0 + np.arange(63)[:, None] / 64.0
    x[63] *= 8.0
    cache = np.zeros((64, R.ROW[fmt]), np.int8 if fmt == "int8" else np.uint8)
    STORE[fmt](synth.f32_to_bf16_bits(x), np.arange(64, dtype=np.int64), cache)
    rows = 1 + np.arange(n, dtype=np.int32) % 63
    rows[::1024] = 0
    gap = np.linspace(12.0, 20.0, H)
    q = np.zeros((1, 1, H, 512), np.float32)
    q[..., :256] = (gap / (256 * SM))[None, None, :, None]
    c = dict(fmt=fmt, cache=cache, draft=cache[:1], rows=rows[None], row_len=np.array([n], np.int32),
             n_tree=np.array([1], np.int32), masks=[[0]], q=synth.f32_to_bf16_bits(q))
    out, lse = launch(c, cuda)
    want, wl, tol, ltol = B.node(synth.bf16_bits_to_f32(c["q"])[0, 0].astype(np.float64), R.values(cache, np.arange(64), fmt),
                                 R.row_scales(cache, np.arange(64), fmt), SM, times=np.bincount(rows, minlength=64))
    err = np.abs(out[0, 0].float().cpu().numpy().astype(np.float64) - want)
    assert (err <= tol).all(), float((err / tol).max())
    assert (np.abs(lse[0, 0].cpu().numpy() - wl) <= ltol).all()


@pytest.mark.parametrize("fmt", ["int8", "fp8", "fp4"])
@pytest.mark.parametrize("cut", CUTS)
@pytest.mark.parametrize("value", [-2.0 ** 16, -1e30, -FLT_MAX, -np.inf, "bytes"])
def test_drafts_that_nobody_has_written(cuda, fmt, cut, value):
    # rows of a tree's unused places as they may lie in memory: scales of either sign, or any bytes
    b, T, H, width = cut
    rng = np.random.default_rng(H + width + 4)
    c = case(rng, fmt, b, T, H, width, [width - i % 60 for i in range(b)], [T] * b, n_rows=700)
    rows = [s * T + j for s in range(b) for j in (1, 4, 5)]
    if value == "bytes":
        c["draft"].view(np.uint8)[rows] = rng.integers(0, 256, (len(rows), c["draft"].shape[1]), dtype=np.uint8)
    else:
        set_scale(c["draft"], rows, fmt, value)
    c["masks"] = [[0b000001, 0, 0b000101, 0b001001, 0b001000, 0]] * b
    check(c, *launch(c, cuda))


@pytest.mark.parametrize("fmt", ["int8", "fp8", "fp4"])
@pytest.mark.parametrize("cut", CUTS)
@pytest.mark.parametrize("ratio", [1.0, 2.0 ** 20])
def test_rows_with_negative_scales(cuda, fmt, cut, ratio):
    # code times scale is what a row holds, whatever its sign; one of them far above the others and, seen, of no weight
    b, T, H, width = cut
    rng = np.random.default_rng(H + width + 5)
    c = case(rng, fmt, b, T, H, width, [width] * b, [T] * b, n_rows=700)
    sc = R.row_scales(c["cache"], np.arange(700), fmt)
    sc[rng.random(700) < 0.5] *= -1.0
    set_scale(c["cache"], np.arange(700), fmt, sc.astype(np.float32))
    c["q"] = synth.f32_to_bf16_bits(synth.bf16_bits_to_f32(c["q"]) + np.float32(0.5))
    c["cache"].view(np.uint8)[7, :288 if fmt == "fp4" else 512] = {"int8": 100, "fp8": 0x7E, "fp4": 0x22}[fmt]
    if fmt == "fp4":
        c["cache"].view(np.uint8)[7, 256:288] = 0x7E
    set_scale(c["cache"], [7], fmt, -float(np.median(np.abs(sc))) * 1024 * ratio)
    c["rows"][c["rows"] == 7] = 8
    c["rows"][:, width // 3] = 7
    check(c, *launch(c, cuda))


@pytest.mark.parametrize("fmt", ["int8", "fp8", "fp4"])
@pytest.mark.parametrize("b,T,H,width", [(2, 6, 4, 70), (1, 4, 16, 80), (1, 1, 16, 3000), (8, 1, 16, 700), (200, 1, 12, 90)])
def test_tiles_of_16_rows_weigh_with_22_bits(cuda, fmt, b, T, H, width):
    # rows in pairs of opposite codes, whose weights nearly cancel: what is left shows each weight's rounding
    rng = np.random.default_rng(H + width + 6)
    c = case(rng, fmt, b, T, H, width, [width] * b, [T] * b, n_rows=700, q_scale=0.01)
    x = rng.standard_normal((350, 512)).astype(np.float32)
    STORE[fmt](synth.f32_to_bf16_bits(np.concatenate([x, -x])), np.arange(700, dtype=np.int64), c["cache"])
    first = np.stack([rng.permutation(350)[np.arange(width // 2) % 350] for _ in range(b)])
    c["rows"] = np.ascontiguousarray(np.stack([first, first + 350], axis=2).reshape(b, -1)[:, rng.permutation(width // 2 * 2)]).astype(np.int32)
    c["row_len"][:] = width // 2 * 2
    c["masks"] = [[0] * T] * b
    check(c, *launch(c, cuda), bits=22)


@pytest.mark.parametrize("fmt", ["int8", "fp8", "fp4"])
@pytest.mark.parametrize("cut", CUTS)
@pytest.mark.parametrize("ratio", [2.0 ** 10, 2.0 ** 24, 2.0 ** 40, 2.0 ** 90])
@pytest.mark.parametrize("first", [True, False])
def test_a_row_that_weighs_everything(cuda, fmt, cut, ratio, first):
    # a row far above the others in scale and score: the output is that row, from the first tile on or after others
    b, T, H, width = cut
    rng = np.random.default_rng(H + width + 7)
    c = case(rng, fmt, b, T, H, width, [width] * b, [T] * b, n_rows=700)
    c["q"] = synth.f32_to_bf16_bits(synth.bf16_bits_to_f32(c["q"]) + np.float32(0.5))
    raw = c["cache"].view(np.uint8)
    raw[7, :256 if fmt == "fp4" else 512] = {"int8": 0x64, "fp8": 0x7E, "fp4": 0x22}[fmt]
    if fmt == "fp4":
        raw[7, 256:288] = 0x7E
    c["rows"][c["rows"] == 7] = 8
    c["rows"][:, 0 if first else width // 2] = 7
    set_scale(c["cache"], [7], fmt, float(np.median(R.row_scales(c["cache"], np.arange(700), fmt))) * ratio)
    row = R.values(c["cache"], [7], fmt)[0]
    s = synth.bf16_bits_to_f32(c["q"]).astype(np.float64) @ row * SM
    assert s.min() > 300.0                                        # (any other row's e^-150 and less beside it)
    out, lse = launch(c, cuda)
    o, l = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    # the output: 2^-11 of the weight, 2^-8 of bf16; lse: 520 half steps of the sum of |q c|, all of one sign but for q's
    assert (np.abs(o - row) <= 1.01 * (2.0 ** -8 + 2.0 ** -11) * np.abs(row)).all()
    mag = np.abs(synth.bf16_bits_to_f32(c["q"]).astype(np.float64)) @ np.abs(row) * SM
    assert (np.abs(l - s) <= 1.01 * (520 * R.U32 * mag + 8 * R.U32 * np.abs(s))).all()
