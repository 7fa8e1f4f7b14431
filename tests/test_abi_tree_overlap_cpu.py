"""Calls of the drafting entry points whose outputs lie over their inputs, or over each other, are refused on the host:
their CTAs read what others write (no GPU needed)."""
import ctypes as C

import pytest

kp = pytest.importorskip("kpool_indexer_int8_b200")
from tests.test_abi_tree_cpu import P, commit_args, tree_args           # noqa: E402


def at(p, more):
    return C.c_void_p(p.value + more)


@pytest.mark.parametrize("src", ["dk", "dg"])
@pytest.mark.parametrize("dst", ["k", "gate"])
def test_commit_refuses_indexer_inputs_drafted_in_place(src, dst):
    # 2 requests of 4 nodes: 2,048 bytes of drafts; of 50 tokens: 25,600 bytes of k
    f, inv = kp.lib.glm_tree_commit, kp.GLM_ERR_INVALID_ARG
    base = {"k": P(9), "gate": P(10)}[dst]
    for more in (0, 256, 25600 - 256):
        assert f(*commit_args(**{src: at(base, more)})) == inv, more
    assert f(*commit_args(**{src: at(base, -2048 + 256)})) == inv


def test_commit_refuses_destinations_over_each_other():
    f, inv = kp.lib.glm_tree_commit, kp.GLM_ERR_INVALID_ARG
    assert f(*commit_args(k=P(10))) == inv
    assert f(*commit_args(gate=at(P(9), 25600 - 16))) == inv
    assert f(*commit_args(k=at(P(6), 528 * 99 // 16 * 16))) == inv
    assert f(*commit_args(gate=at(P(6), -16))) == inv


def test_tree_refuses_outputs_over_inputs():
    names = dict(q=P(0), cache=P(1), rows=P(2), draft=P(3), mask=P(4))
    for fn in ("glm_tree_mla_decode", "glm_tree_mla_decode_fp8", "glm_tree_mla_decode_fp4"):
        f = getattr(kp.lib, fn)
        for name, p in names.items():
            assert f(*tree_args(out=p)) == kp.GLM_ERR_INVALID_ARG, name
            assert f(*tree_args(lse=p)) == kp.GLM_ERR_INVALID_ARG, name
            assert f(*tree_args(ws=p)) == kp.GLM_ERR_INVALID_ARG, name
        assert f(*tree_args(out=P(6))) == kp.GLM_ERR_INVALID_ARG
        assert f(*tree_args(lse=at(P(5), 64))) == kp.GLM_ERR_INVALID_ARG
        assert f(*tree_args(row_len=P(5))) == kp.GLM_ERR_INVALID_ARG
        assert f(*tree_args(n_tree=at(P(6), 256))) == kp.GLM_ERR_INVALID_ARG
