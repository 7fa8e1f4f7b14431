"""What the Python binding of the drafting entry points refuses, with a ValueError that names the tensor."""
import numpy as np
import pytest
import torch

import kpool_indexer_int8_b200 as kp
from tests.test_gpu_block_tables import commit_case
from tests.test_gpu_tree import CALL, case, check
from tests.test_gpu_tree_edges import device_args

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,other", [("fp8", 304), ("fp4", 528), ("int8", 304), ("fp4", 608)])
def test_rows_of_another_width_are_refused(cuda, fmt, other):
    # contiguous tensors of the right type, whose rows would be read shifted
    c = case(np.random.default_rng(1), fmt, 1, 2, 16, 70, [70], [2], n_rows=304 * 528 // 304)
    good = device_args(c, cuda, kp.make_dims(16))
    kind, row = good["cache"].dtype, good["cache"].shape[1]
    for name, n in (("cache", 528), ("draft", 2)):
        wrong = dict(good, **{name: torch.zeros((n, other), dtype=kind, device=cuda)})
        with pytest.raises(ValueError, match=f"rows of {row} bytes"):
            CALL[fmt](kp.make_dims(16), **wrong)
    # the same bytes in another shape, and a flat one
    for flat in (good["cache"].reshape(-1, other) if good["cache"].numel() % other == 0 else good["cache"].reshape(-1),
                 good["cache"].reshape(-1)):
        with pytest.raises(ValueError, match=f"rows of {row} bytes"):
            CALL[fmt](kp.make_dims(16), **dict(good, cache=flat))
    CALL[fmt](kp.make_dims(16), **dict(good, cache=good["cache"].reshape(16, -1, row)))    # rows in blocks
    torch.cuda.synchronize()
    check(c, good["out"], good["lse"])


@pytest.mark.parametrize("wrong", [3, None, "x", [1, 2], np.zeros((2, 2))])
def test_what_is_no_tensor_is_a_value_error(cuda, wrong):
    dims = kp.make_dims(16)
    c = case(np.random.default_rng(2), "int8", 1, 2, 16, 70, [70], [2])
    good = device_args(c, cuda, dims)
    for name in ("q", "cache", "rows", "draft", "mask", "out", "workspace"):
        if wrong is None and name in ("mask", "out"):
            continue                                            # (the library refuses these)
        with pytest.raises(ValueError, match=name):
            kp.glm_tree_mla_decode(dims, **dict(good, **{name: wrong}))
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device=cuda)                            # noqa: E731
    tables = dict(length=i(2), n_new=i(2), n_blocks=i(2), block_table=i(2, 4), free=i(9), n_free=i(1), block_size=16, pool_blocks=9,
                  slots=i(5).long(), q_seq=i(5), q_pos=i(5), len_out=i(2), n_blocks_out=i(2), cu_new=i(3), free_out=i(9),
                  n_free_out=i(1), slot_map=i(2, 64).long())
    for name in ("length", "block_table", "slots", "free", "slot_map"):
        if wrong is None and name == "slot_map":
            continue
        with pytest.raises(ValueError, match=name):
            kp.glm_block_tables(**dict(tables, **{name: wrong}))
    c = commit_case(np.random.default_rng(3), 2, 4, "int8", 4, 3)
    commit = {k: v if k == "n_nodes" else torch.from_numpy(np.ascontiguousarray(v)).to(cuda) for k, v in c.items()}
    for k in ("draft_k", "draft_gate", "k", "gate"):
        commit[k] = commit[k].view(torch.bfloat16)
    for name in ("draft", "path", "slots", "cache", "k"):
        if wrong is None and name == "k":
            continue
        with pytest.raises(ValueError, match=name):
            kp.glm_tree_commit(dims, **dict(commit, **{name: wrong}))


def test_tensors_of_another_rank_are_a_value_error(cuda):
    dims = kp.make_dims(16)
    c = case(np.random.default_rng(2), "int8", 1, 2, 16, 70, [70], [2])
    good = device_args(c, cuda, dims)
    for name in ("q", "cache", "rows", "draft"):
        with pytest.raises(ValueError, match=name):
            kp.glm_tree_mla_decode(dims, **dict(good, **{name: good[name].reshape(-1)}))
    c = commit_case(np.random.default_rng(3), 2, 4, "int8", 4, 3)
    commit = {k: v if k == "n_nodes" else torch.from_numpy(np.ascontiguousarray(v)).to(cuda) for k, v in c.items()}
    for k in ("draft_k", "draft_gate", "k", "gate"):
        commit[k] = commit[k].view(torch.bfloat16)
    for name in ("draft", "path", "cache", "k"):
        with pytest.raises(ValueError, match=name):
            kp.glm_tree_commit(dims, **dict(commit, **{name: commit[name].reshape(-1)}))


def test_the_checks_in_python_are_the_native_ones(cuda, monkeypatch):
    # without csrc/args.c: the same calls are taken and refused
    from tests import test_gpu_block_tables, test_gpu_tree_edges
    monkeypatch.setattr(kp, "_args", None)
    test_gpu_tree_edges.test_binding_refuses(cuda)
    test_gpu_tree_edges.test_views_and_an_empty_cache(cuda, 4)
    test_gpu_block_tables.run(cuda, test_gpu_block_tables.request_batch(np.random.default_rng(1), 5, 16, 90, 20, pads=True), 120, 130)
    test_gpu_block_tables.run_commit(cuda, commit_case(np.random.default_rng(2), 3, 5, "fp4", 5, 4))
