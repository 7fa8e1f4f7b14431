"""The tree attention where it can go wrong: every way a call is cut, rows that are not finite in masked
and in seen places, references that move in every tile, empty lists, long caches, graphs and streams.
Errors allowed: those derived in tests/tree_reference.py."""
import numpy as np
import pytest
import torch

import kpool_indexer_int8_b200 as kp
import synth
from tests import tree_reference as R
from tests.test_gpu_tree import CALL, SM, as_int64, bf16, case, check, launch, make_rows

pytestmark = pytest.mark.gpu

SCALE_AT = {"int8": 512, "fp8": 512, "fp4": 288}


def set_scale(cache, rows, fmt, value):
    at = SCALE_AT[fmt]
    v = np.broadcast_to(np.asarray(value, np.float32), (len(rows),))
    cache.view(np.uint8)[np.asarray(rows), at:at + 4] = np.ascontiguousarray(v).view(np.uint8).reshape(-1, 4)


def put_nan(cache, rows, fmt):
    """NaN in the rows: a code (E4M3), a block scale (4-bit rows), the row scale (int8)."""
    if fmt == "int8":
        set_scale(cache, rows, fmt, np.nan)
    else:
        cache[np.asarray(rows), 256 + 7 if fmt == "fp4" else 300] = 0xFF


# How a call is cut depends on its rows (nodes x heads), the batch and the width: small calls go 16 rows
# a CTA, 17 to 64 rows in one CTA a run, more in pairs of CTAs; one run or several a sequence.
@pytest.mark.parametrize("fmt", ["int8", "fp8", "fp4"])
@pytest.mark.parametrize("B,T,H,width,lens,n_tree", [
    (3, 7, 3, 70, [70, 64, 3], [7, 3, 1]),                        # 21 rows: two CTAs of 16 rows
    (3, 1, 16, 5000, [5000, 17, 64], [1, 1, 1]),                  # 16 rows, several runs
    (160, 2, 8, 70, [i % 71 for i in range(160)], [i % 3 for i in range(160)]),      # 16 rows, one run
    (8, 3, 8, 1500, [1500, 0, 64, 65, 63, 1, 800, 128], [3, 3, 1, 2, 0, 3, 3, 3]),   # 24 rows
    (150, 3, 8, 80, [(7 * i) % 81 for i in range(150)], [i % 4 for i in range(150)]),
    (4, 4, 16, 1500, [1500, 1, 64, 640], [4, 1, 4, 3]),           # 64 rows, several runs
    (150, 4, 16, 65, [i % 66 for i in range(150)], [i % 5 for i in range(150)]),     # 64 rows, one run
    (10, 8, 128, 200, [200, 0, 96, 95, 97, 192, 193, 1, 150, 40], [8, 8, 8, 7, 1, 2, 0, 8, 5, 8]),   # pairs, one run
    (2, 5, 64, 3000, [3000, 33], [5, 2]),                         # pairs, several runs, rows of the last not all there
    (1, 64, 2, 6000, [5999], [64]),                               # 128 rows, 64 nodes
])
def test_every_cut(cuda, fmt, B, T, H, width, lens, n_tree):
    rng = np.random.default_rng(B + 10 * T + 100 * H + width)
    c = case(rng, fmt, B, T, H, width, lens, n_tree, n_rows=700, holes=0.05)
    check(c, *launch(c, cuda))


def test_lists_of_very_different_lengths(cuda):
    # (more tiles than 32 waves: the run length is weighed against the lengths)
    rng = np.random.default_rng(3)
    c = case(rng, "fp4", 4, 1, 4, 80000, [80000, 5, 0, 9000], [1, 1, 1, 1], n_rows=500)
    check(c, *launch(c, cuda))


@pytest.mark.parametrize("fmt", ["int8", "fp8", "fp4"])
@pytest.mark.parametrize("H,width", [(4, 70), (4, 3000), (40, 70), (40, 3000)])
def test_rows_that_are_not_finite(cuda, fmt, H, width):
    # drafts 1 and 4 hold NaN, draft 2 an infinite scale: a node that sees one gives NaN, the others must not notice
    rng = np.random.default_rng(H + width)
    T = 6
    c = case(rng, fmt, 2, T, H, width, [width, width // 2], [T, T], n_rows=600)
    for b in range(2):
        put_nan(c["draft"], [b * T + 1, b * T + 4], fmt)
        set_scale(c["draft"], [b * T + 2], fmt, np.inf)
    masks = [0b000001, 0b000010, 0b000101, 0b001001, 0b011001, 0b101001]
    c["masks"] = [masks, masks]
    out, lse = launch(c, cuda)
    o, l = out.float().cpu().numpy(), lse.cpu().numpy()
    clean = dict(c, draft=c["draft"].copy(), masks=[[m if m & 0b010110 == 0 else 0b1 for m in masks]] * 2)
    bad = [i for i, m in enumerate(masks) if m & 0b010110]
    for i in bad:
        assert np.isnan(o[:, i]).all() and np.isnan(l[:, i]).all(), i
    good = [i for i in range(T) if i not in bad]
    assert np.isfinite(o[:, good]).all() and np.isfinite(l[:, good]).all()
    q = synth.bf16_bits_to_f32(c["q"]).astype(np.float64)
    for b, i, want, wl, tol, ltol in R.tree(q, c["cache"], c["rows"], c["row_len"], clean["draft"], clean["masks"],
                                            c["n_tree"], SM, fmt):
        if i in good:
            assert (np.abs(o[b, i] - want) <= tol).all() and (np.abs(l[b, i] - wl) <= ltol).all(), (b, i)


@pytest.mark.parametrize("fmt", ["int8", "fp8", "fp4"])
@pytest.mark.parametrize("H", [4, 40])
def test_a_nan_row_of_a_list_stays_in_its_sequence(cuda, fmt, H):
    rng = np.random.default_rng(H)
    c = case(rng, fmt, 3, 2, H, 300, [300, 300, 300], [2, 2, 2], n_rows=600)
    c["rows"][c["rows"] == 599] = 598
    c["rows"][1, 130] = 599
    put_nan(c["cache"], [599], fmt)
    out, lse = launch(c, cuda)
    assert np.isnan(out[1].float().cpu().numpy()).all() and np.isnan(lse[1].cpu().numpy()).all()
    for b in (0, 2):
        one = {k: v[b:b + 1] if isinstance(v, (np.ndarray, list)) and k not in ("cache", "draft") else v for k, v in c.items()}
        one["draft"] = c["draft"][2 * b:2 * b + 2]
        check(one, out[b:b + 1], lse[b:b + 1])


@pytest.mark.parametrize("fmt", ["int8", "fp8", "fp4"])
@pytest.mark.parametrize("H", [4, 20, 40])
@pytest.mark.parametrize("q_scale,order", [(40.0, 1), (40.0, -1), (1e-3, 1), (1e4, 1), (2.0 ** -100, 1)])
def test_references_move(cuda, fmt, H, q_scale, order):
    # scores that rise or fall along the list by far more than a reference may lag, and scores of nearly nothing
    rng = np.random.default_rng(int(H + abs(order)))
    c = case(rng, fmt, 2, 2, H, 900, [900, 450], [2, 2], n_rows=900, q_scale=q_scale)
    q = synth.bf16_bits_to_f32(c["q"]).astype(np.float64)
    v = R.values(c["cache"], np.arange(900), fmt)
    for b in range(2):
        n = c["row_len"][b]
        s = v[c["rows"][b, :n]] @ q[b, 0, 0]
        c["rows"][b, :n] = c["rows"][b, :n][np.argsort(order * s)]
    check(c, *launch(c, cuda))


@pytest.mark.parametrize("fmt", ["int8", "fp8", "fp4"])
@pytest.mark.parametrize("H", [4, 40])
@pytest.mark.parametrize("order", [1, -1])
def test_scales_of_many_sizes(cuda, fmt, H, order):
    # row scales from 2^-30 to 2^6 along the list, some zero: sigma follows the largest of them
    rng = np.random.default_rng(H)
    c = case(rng, fmt, 1, 3, H, 800, [800], [3], n_rows=800)
    c["rows"][0] = np.arange(800)
    e = np.sort(rng.uniform(-30, 6, 800))[::order]
    sc = (2.0 ** e).astype(np.float32) * np.float32(1e-3 if fmt == "fp4" else 1e-2)
    sc[rng.random(800) < 0.05] = 0.0
    set_scale(c["cache"], np.arange(800), fmt, sc)
    check(c, *launch(c, cuda))


@pytest.mark.parametrize("fmt", ["int8", "fp8", "fp4"])
@pytest.mark.parametrize("H", [4, 40])
def test_nothing_to_see(cuda, fmt, H):
    rng = np.random.default_rng(1)
    c = case(rng, fmt, 5, 3, H, 130, [130, 130, 0, 0, 7], [3, 0, 3, 3, -2])
    c["row_len"][3] = -4
    c["rows"][0] = -1                                    # a list of padding only
    c["rows"][1, 3] = 2 ** 31 - 1                        # (entries past the cache are padding too)
    c["masks"][0] = [0, 0b010, 0b111]                    # a node that sees nothing at all
    c["masks"][2] = [0b100, 0, -1]                       # bits past the tree's nodes mean nothing
    check(c, *launch(c, cuda))


@pytest.mark.parametrize("fmt", ["int8", "fp8", "fp4"])
def test_optional_arguments(cuda, fmt):
    rng = np.random.default_rng(2)
    c = case(rng, fmt, 2, 3, 8, 100, [100, 100], [3, 3])
    out, lse = launch(c, cuda)
    dims = kp.make_dims(8)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(cuda)                         # noqa: E731
    need = kp.glm_dsa_workspace_size(dims, kp.GLM_OP_TREE_MLA, 2, select_k=3, width=100)
    ws = torch.zeros(need, dtype=torch.uint8, device=cuda)
    bare = torch.full_like(out, 3.0)
    CALL[fmt](dims, bf16(c["q"]).to(cuda), t(c["cache"]), t(c["rows"]), t(c["draft"]), as_int64(c["masks"]).to(cuda), SM, bare,
              ws)
    assert torch.equal(bare.view(torch.int16), out.view(torch.int16))
    # no list at all
    need = kp.glm_dsa_workspace_size(dims, kp.GLM_OP_TREE_MLA, 2, select_k=3, width=0)
    e = dict(c, rows=np.zeros((2, 0), np.int32), row_len=np.zeros(2, np.int32))
    CALL[fmt](dims, bf16(c["q"]).to(cuda), t(c["cache"]), torch.zeros((2, 0), dtype=torch.int32, device=cuda), t(c["draft"]),
              as_int64(c["masks"]).to(cuda), SM, bare, ws, lse=lse)
    torch.cuda.synchronize()
    check(e, bare, lse)


@pytest.mark.parametrize("H", [16, 64])
def test_the_same_row_many_times(cuda, H):
    rng = np.random.default_rng(4)
    c = case(rng, "int8", 2, 2, H, 500, [500, 500], [2, 2])
    c["rows"][0] = 17
    c["rows"][1, ::2] = 5
    check(c, *launch(c, cuda))


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("H", [8, 64])
def test_rows_past_two_gigabytes(cuda, fmt, H):
    rng = np.random.default_rng(5)
    c = case(rng, fmt, 1, 2, H, 200, [200], [2], n_rows=300)
    n = (2 ** 31 // R.ROW[fmt]) + 2000
    kind = torch.int8 if fmt == "int8" else torch.uint8
    cache = torch.zeros((n, R.ROW[fmt]), dtype=kind, device=cuda)
    at = np.concatenate([np.arange(100), n - 200 + np.arange(200)])
    cache[torch.from_numpy(at).to(cuda)] = torch.from_numpy(c["cache"]).to(cuda)
    dims = kp.make_dims(H)
    need = kp.glm_dsa_workspace_size(dims, kp.GLM_OP_TREE_MLA, 1, select_k=2, width=200)
    ws = torch.zeros(need, dtype=torch.uint8, device=cuda)
    out = torch.full((1, 2, H, 512), 7.0, dtype=torch.bfloat16, device=cuda)
    lse = torch.full((1, 2, H), 7.0, dtype=torch.float32, device=cuda)
    rows = torch.from_numpy(at[c["rows"]].astype(np.int32)).to(cuda)
    CALL[fmt](dims, bf16(c["q"]).to(cuda), cache, rows, torch.from_numpy(c["draft"]).to(cuda), as_int64(c["masks"]).to(cuda), SM,
              out, ws, lse=lse)
    torch.cuda.synchronize()
    check(c, out, lse)


def device_args(c, dev, dims):
    B, T, H = c["q"].shape[:3]
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)                          # noqa: E731
    need = kp.glm_dsa_workspace_size(dims, kp.GLM_OP_TREE_MLA, B, select_k=T, width=c["rows"].shape[1])
    return dict(q=bf16(c["q"]).to(dev), cache=t(c["cache"]), rows=t(c["rows"]), draft=t(c["draft"]), mask=as_int64(c["masks"]).to(dev),
                sm_scale=SM, out=torch.full((B, T, H, 512), 7.0, dtype=torch.bfloat16, device=dev),
                workspace=torch.zeros(need, dtype=torch.uint8, device=dev),
                lse=torch.full((B, T, H), 7.0, dtype=torch.float32, device=dev), row_len=t(c["row_len"]), n_tree=t(c["n_tree"]))


@pytest.mark.parametrize("fmt", ["int8", "fp8", "fp4"])
@pytest.mark.parametrize("H", [16, 64])
def test_streams_and_graphs(cuda, fmt, H):
    # two calls at once on two streams, each captured too and replayed on new lengths: equal bits each time
    dims = kp.make_dims(H)
    rng = np.random.default_rng(6)
    cs = [case(rng, fmt, 2, 4, H, 1500, [1500, 700], [4, 3]) for _ in range(2)]
    ds = [device_args(c, cuda, dims) for c in cs]
    streams = [torch.cuda.Stream(cuda) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for d, s in zip(ds, streams):
            CALL[fmt](dims, **d, stream=s)
    torch.cuda.synchronize()
    for c, d in zip(cs, ds):
        check(c, d["out"], d["lse"])
    first = [d["out"].clone() for d in ds]
    graphs = []
    for d, s in zip(ds, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            CALL[fmt](dims, **d)
            CALL[fmt](dims, **d)
        graphs.append(g)
    for d in ds:
        d["out"].fill_(7.0)
        d["lse"].fill_(7.0)
    torch.cuda.synchronize()
    for g, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for d, f in zip(ds, first):
        assert torch.equal(d["out"].view(torch.int16), f.view(torch.int16))
    c = dict(cs[0], row_len=np.array([3, 1499], np.int32), n_tree=np.array([1, 4], np.int32))
    ds[0]["row_len"].copy_(torch.from_numpy(c["row_len"]))
    ds[0]["n_tree"].copy_(torch.from_numpy(c["n_tree"]))
    torch.cuda.synchronize()
    graphs[0].replay()
    torch.cuda.synchronize()
    check(c, ds[0]["out"], ds[0]["lse"])


def test_binding_refuses(cuda):
    dims = kp.make_dims(16)
    c = case(np.random.default_rng(7), "int8", 1, 2, 16, 70, [70], [2])
    good = device_args(c, cuda, dims)
    for name, bad in [("q", good["q"].float()), ("q", good["q"].cpu()), ("q", good["q"][..., ::2]), ("q", good["q"][:, :, :8]),
                      ("cache", good["cache"].view(torch.uint8)), ("cache", good["cache"][:, :304]), ("rows", good["rows"].long()),
                      ("rows", good["rows"][:, ::2]), ("draft", good["draft"][:1]), ("mask", good["mask"].int()),
                      ("mask", good["mask"][:, :1]), ("out", good["out"].float()), ("lse", good["lse"][..., :8]),
                      ("row_len", good["row_len"].long()), ("n_tree", good["n_tree"].repeat(2)),
                      ("workspace", good["workspace"][:-256])]:
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            CALL["int8"](dims, **dict(good, **{name: bad}))
    CALL["int8"](dims, **good)
    torch.cuda.synchronize()
    check(c, good["out"], good["lse"])


@pytest.mark.parametrize("fmt", ["int8", "fp8", "fp4"])
@pytest.mark.parametrize("H", [4, 40])
@pytest.mark.parametrize("top", [2.0 ** -126, 2.0 ** -140, 2.0 ** 100])
def test_scales_at_the_ends_of_fp32(cuda, fmt, H, top):
    # denormal scales lose bits as such (the rows are what they are), not in the sums
    rng = np.random.default_rng(H)
    c = case(rng, fmt, 1, 2, H, 200, [200], [2], n_rows=200)
    for name in ("cache", "draft"):
        n = len(c[name])
        set_scale(c[name], np.arange(n), fmt, (top * rng.uniform(0.25, 1.0, n)).astype(np.float32))
    sm = float(np.float32(2.0 ** -110 if top > 1 else SM))
    out, lse = launch(c, cuda, sm=sm)
    o = out.float().cpu().numpy().astype(np.float64)
    q = synth.bf16_bits_to_f32(c["q"]).astype(np.float64)
    for b, i, want, wl, tol, ltol in R.tree(q, c["cache"], c["rows"], c["row_len"], c["draft"], c["masks"], c["n_tree"], sm, fmt):
        # (a bf16 or fp32 denormal is off by half its step more)
        assert (np.abs(o[b, i] - want) <= tol + 2.0 ** -134 + 2.0 ** -148).all(), (b, i)
        assert (np.abs(lse[b, i].cpu().numpy() - wl) <= ltol).all(), (b, i)


@pytest.mark.parametrize("fmt", ["int8", "fp8", "fp4"])
@pytest.mark.parametrize("H", [4, 40])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_query_that_is_not_finite_stays_alone(cuda, fmt, H, value):
    rng = np.random.default_rng(8)
    c = case(rng, fmt, 2, 3, H, 300, [300, 200], [3, 3], n_rows=400)
    good = launch(c, cuda)
    q = bf16(c["q"]).clone()
    q[0, 1, H - 1, 77] = value
    bad = dict(c, q=q.view(torch.int16).numpy().view(np.uint16))
    out, lse = launch(bad, cuda)
    assert torch.isnan(out[0, 1, H - 1]).all() and torch.isnan(lse[0, 1, H - 1])
    out[0, 1, H - 1], lse[0, 1, H - 1] = good[0][0, 1, H - 1], good[1][0, 1, H - 1]
    check(c, out, lse)


@pytest.mark.parametrize("H", [4, 40])
def test_views_and_an_empty_cache(cuda, H):
    # tensors that start inside their storage, one that wants a gradient, and a cache of no rows
    dims = kp.make_dims(H)
    c = case(np.random.default_rng(9), "fp8", 2, 3, H, 100, [100, 50], [3, 2], n_rows=300)
    d = device_args(c, cuda, dims)
    inside = {k: torch.cat([v[:1], v])[1:] if isinstance(v, torch.Tensor) and k != "workspace" else v for k, v in d.items()}
    assert inside["q"].storage_offset() > 0 and inside["q"].is_contiguous()
    inside["q"].requires_grad_()
    CALL["fp8"](dims, **inside)
    torch.cuda.synchronize()
    check(c, inside["out"], inside["lse"])
    none = dict(c, rows=np.full((2, 100), -1, np.int32))
    d["rows"].fill_(-1)
    d["cache"] = d["cache"][:0]
    CALL["fp8"](dims, **d)
    torch.cuda.synchronize()
    check(none, d["out"], d["lse"])


def test_output_over_the_query_is_refused(cuda):
    dims = kp.make_dims(4)
    c = case(np.random.default_rng(10), "int8", 1, 2, 4, 70, [70], [2])
    d = device_args(c, cuda, dims)
    with pytest.raises(kp.GlmError):
        CALL["int8"](dims, **dict(d, out=d["q"]))


def test_the_widest_list(cuda):
    # 1,024 rows 1,024 times over: their softmax is that of the rows once, lse by log 1024 more
    rng = np.random.default_rng(11)
    n = 1 << 20
    c = case(rng, "int8", 1, 1, 2, 1024, [1024], [1], n_rows=1024)
    wide = dict(c, rows=np.tile(c["rows"], (1, 1024)), row_len=np.array([n], np.int32), masks=[[0]])
    out, lse = launch(wide, cuda)
    c["masks"] = [[0]]
    q = synth.bf16_bits_to_f32(c["q"]).astype(np.float64)
    (_, _, want, wl, tol, ltol), = R.tree(q, c["cache"], c["rows"], c["row_len"], c["draft"], c["masks"], c["n_tree"], SM, "int8")
    more = n / 8 * R.U32                                  # the sums of tests/tree_reference.py, over n rows
    v = R.values(c["cache"], c["rows"][0], "int8")
    s = (q[0, 0] @ v.T) * SM
    p = np.exp(s - wl[:, None])
    o, l = out[0, 0].float().cpu().numpy(), lse[0, 0].cpu().numpy()
    assert (np.abs(o - want) <= tol + more * (p @ np.abs(v))).all()
    assert (np.abs(l - (wl + np.log(1024))) <= ltol + more).all()


@pytest.mark.parametrize("B,T,H,width", [(20000, 1, 1, 3), (1, 64, 128, 90), (2, 64, 128, 700)])
def test_the_largest_batch_and_trees(cuda, B, T, H, width):
    rng = np.random.default_rng(12)
    c = case(rng, "fp4", B, T, H, width, [int(v) for v in rng.integers(0, width + 1, B)], [int(v) for v in rng.integers(0, T + 1, B)],
             n_rows=300)
    check(c, *launch(c, cuda))


@pytest.mark.parametrize("H,width", [(4, 300), (20, 3000), (64, 300), (64, 3000)])
def test_what_unused_nodes_hold_means_nothing(cuda, H, width):
    # queries, masks and drafted rows past a tree's nodes: NaN, infinities, bits everywhere
    rng = np.random.default_rng(13)
    c = case(rng, "fp8", 3, 5, H, width, [width, 10, 0], [3, 0, 1], n_rows=400)
    q = bf16(c["q"]).clone()
    for b, t in enumerate(c["n_tree"]):
        q[b, t:, ::2], q[b, t:, 1::2] = float("nan"), float("inf")
        c["masks"][b][t:] = [-1] * (5 - t)
        c["draft"][b * 5 + t:b * 5 + 5] = 0xFF
    c["q"] = q.view(torch.int16).numpy().view(np.uint16)
    out, lse = launch(c, cuda)
    plain = q.clone()
    plain[~torch.isfinite(plain)] = 0.0
    check(dict(c, q=plain.view(torch.int16).numpy().view(np.uint16)), out, lse)
