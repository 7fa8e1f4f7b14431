"""The drafting entry points reject bad arguments on the host, before any CUDA call (no GPU needed)."""
import ctypes as C

import pytest
import torch

kp = pytest.importorskip("kpool_indexer_int8_b200")

MIS8, MIS4 = C.c_void_p(0x10008), C.c_void_p(0x10002)


def P(i):
    """Distinct aligned addresses 16 MiB apart, never dereferenced."""
    return C.c_void_p((i + 1) << 24)


def tree_args(**kw):
    a = dict(dims=C.byref(kp.make_dims(64)), q=P(0), cache=P(1), n_rows=100, rows=P(2), row_len=None, width=80, draft=P(3),
             mask=P(4), n_tree=None, batch=1, n_nodes=4, sm=0.04, out=P(5), lse=None, ws=P(6), ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("fn", ["glm_tree_mla_decode", "glm_tree_mla_decode_fp8", "glm_tree_mla_decode_fp4"])
def test_tree_rejects_before_launch(fn):
    f = getattr(kp.lib, fn)
    bad = lambda rc, **kw: f(*tree_args(**kw)) == rc                       # noqa: E731
    inv = kp.GLM_ERR_INVALID_ARG
    assert bad(kp.GLM_ERR_UNSUPPORTED, dims=C.byref(kp.make_dims(64, qk_rope_head_dim=64)))
    assert bad(kp.GLM_ERR_UNSUPPORTED, dims=C.byref(kp.make_dims(129)))
    for kw in (dict(batch=-1), dict(n_nodes=0), dict(n_nodes=65), dict(width=-1), dict(width=(1 << 20) + 1),
               dict(batch=2000, n_nodes=40), dict(n_rows=-1), dict(sm=float("nan")), dict(q=None), dict(q=MIS8),
               dict(cache=None), dict(cache=MIS8), dict(rows=None), dict(rows=MIS4), dict(row_len=MIS4),
               dict(draft=None), dict(draft=MIS8), dict(mask=None), dict(mask=C.c_void_p(0x10004)), dict(n_tree=MIS4),
               dict(out=None), dict(out=MIS8), dict(lse=MIS4)):
        assert bad(inv, **kw), kw
    assert bad(kp.GLM_ERR_WORKSPACE, ws=None)
    assert bad(kp.GLM_ERR_WORKSPACE, ws=C.c_void_p(0x10010))
    need = kp.glm_dsa_workspace_size(kp.make_dims(64), kp.GLM_OP_TREE_MLA, 1, select_k=4, width=80)
    assert bad(kp.GLM_ERR_WORKSPACE, ws_bytes=need - 1)
    assert bad(kp.GLM_OK, batch=0, q=None, cache=None, rows=None, draft=None, mask=None, out=None, ws=None)


def test_tree_workspace_covers_every_smaller_call():
    for heads in (1, 16, 64, 128):
        d = kp.make_dims(heads)
        size = lambda b, t, w: kp.glm_dsa_workspace_size(d, kp.GLM_OP_TREE_MLA, b, select_k=t, width=w)   # noqa: E731
        for values, at in (((1, 2, 5, 33, 148, 149, 1000), lambda v: size(v, 64, 4096)),
                           ((1, 2, 3, 16, 63, 64), lambda v: size(3, v, 262144)),
                           ((0, 1, 64, 65, 4096, 262144, 1 << 20), lambda v: size(2, 8, v))):
            sizes = [at(v) for v in values]
            assert sizes == sorted(sizes), (heads, sizes)
    for b, t, w in ((-1, 4, 8), (1, 0, 8), (1, 65, 8), (1, 4, -1), (1, 4, (1 << 20) + 1), (2000, 64, 8)):
        with pytest.raises(kp.GlmError):
            kp.glm_dsa_workspace_size(kp.make_dims(64), kp.GLM_OP_TREE_MLA, b, select_k=t, width=w)


NAMES = ("len", "n_new", "n_blocks", "pad", "batch", "bs", "table", "ld_blocks", "free", "n_free", "free_cap", "pool",
         "slots", "q_seq", "q_pos", "n_cap", "slot_map", "ld_slot", "len_out", "n_blocks_out", "cu_new", "free_out",
         "n_free_out", "stream")


def tables_args(**kw):
    v = (P(0), P(1), P(2), P(3), 4, 256, P(4), 10, P(5), P(6), 100, 100, P(7), P(8), P(9), 20, P(10), 100, P(11), P(12),
         P(13), P(14), P(15), None)
    a = dict(zip(NAMES, v))
    a.update(kw)
    return tuple(a.values())


def test_block_tables_rejects_before_launch():
    f, inv = kp.lib.glm_block_tables, kp.GLM_ERR_INVALID_ARG
    for kw in (dict(batch=-1), dict(batch=8193), dict(bs=0), dict(bs=65537), dict(ld_blocks=-1), dict(ld_blocks=1 << 31),
               dict(free_cap=-1), dict(pool=-1), dict(pool=1 << 23, bs=256), dict(n_cap=-1), dict(n_cap=1 << 31),
               dict(ld_slot=-1)):
        assert f(*tables_args(**kw)) == inv, kw
    for name in ("len", "n_new", "n_blocks", "table", "free", "n_free", "slots", "q_seq", "q_pos", "len_out",
                 "n_blocks_out", "cu_new", "free_out", "n_free_out"):
        assert f(*tables_args(**{name: None})) == inv, name
        assert f(*tables_args(**{name: MIS4})) == inv, name
    assert f(*tables_args(slot_map=C.c_void_p(0x10004))) == inv
    # an output that is an input, or another output
    for a, b in (("len_out", "len"), ("n_blocks_out", "n_blocks"), ("free_out", "free"), ("n_free_out", "n_free"),
                 ("len_out", "n_blocks_out"), ("q_seq", "q_pos"), ("slots", "slot_map"), ("cu_new", "table")):
        args = dict(zip(NAMES, tables_args()))
        assert f(*tables_args(**{a: args[b]})) == inv, (a, b)
        if b != "n_free":                                            # (one word)
            assert f(*tables_args(**{a: C.c_void_p(args[b].value + 8)})) == inv, (a, b)   # a part of it


def commit_args(**kw):
    a = dict(dims=C.byref(kp.make_dims(64)), draft=P(0), fmt=kp.GLM_CACHE_INT8, path=P(1), batch=2, n_nodes=4, ld_path=4,
             slots=P(2), q_seq=P(3), q_pos=P(4), cu_new=P(5), n_cap=8, cache=P(6), n_rows=100, dk=P(7), dg=P(8), k=P(9),
             gate=P(10), ld_tokens=50, stream=None)
    a.update(kw)
    return tuple(a.values())


def test_commit_rejects_before_launch():
    f, inv = kp.lib.glm_tree_commit, kp.GLM_ERR_INVALID_ARG
    assert f(*commit_args(dims=C.byref(kp.make_dims(64, kv_lora_rank=576)))) == kp.GLM_ERR_UNSUPPORTED
    for kw in (dict(fmt=-1), dict(fmt=3), dict(batch=-1), dict(n_nodes=0), dict(n_nodes=65), dict(ld_path=-1),
               dict(n_cap=-1), dict(n_rows=-1), dict(ld_tokens=-1), dict(k=None), dict(dk=None), dict(gate=None),
               dict(dg=None), dict(draft=None), dict(draft=MIS8), dict(path=None), dict(path=MIS4), dict(slots=None),
               dict(slots=C.c_void_p(0x10004)), dict(q_seq=None), dict(q_pos=None), dict(cu_new=None), dict(cache=None),
               dict(cache=MIS8), dict(k=MIS8), dict(draft=P(6)), dict(cache=C.c_void_p(P(0).value + 528 * 7))):
        assert f(*commit_args(**kw)) == inv, kw
    assert f(*commit_args(n_cap=0, slots=None, draft=None)) == kp.GLM_OK
    assert f(*commit_args(batch=0)) == kp.GLM_OK


def test_binding_checks_types_and_shapes():
    # the checks of the binding come before the library is called: CPU tensors never reach it
    z = lambda *s, dt=torch.int32: torch.zeros(*s, dtype=dt)               # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        kp.glm_tree_mla_decode(kp.make_dims(64), z(1, 2, 64, 512, dt=torch.bfloat16), z(4, 528, dt=torch.int8), z(1, 8),
                               z(2, 528, dt=torch.int8), z(1, 2, dt=torch.int64), 0.04,
                               z(1, 2, 64, 512, dt=torch.bfloat16), z(16, dt=torch.uint8))
    with pytest.raises(ValueError, match="CUDA"):
        kp.glm_block_tables(z(2), z(2), z(2), z(2, 4), z(9), z(1), 256, 9, z(5, dt=torch.int64), z(5), z(5), z(2), z(2),
                            z(3), z(9), z(1))
    with pytest.raises(ValueError, match="CUDA"):
        kp.glm_tree_commit(kp.make_dims(64), z(8, 528, dt=torch.int8), z(2, 4), 4, z(5, dt=torch.int64), z(5), z(5), z(3),
                           z(9, 528, dt=torch.int8))
