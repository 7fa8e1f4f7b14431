"""Steps of speculative decoding as they are used: drafted rows stored, the tree's attention over them and the
context, slots for what was accepted from the block tables, the accepted drafts committed, and again on the
grown context, with requests that end and come in between. Against plain Python kept beside it."""
import numpy as np
import pytest
import torch

import kpool_indexer_int8_b200 as kp
import synth
from tests import tables_reference as TR
from tests import tree_reference as R
from tests.test_gpu_tree import CALL, SM, as_int64, bf16, tree_masks

pytestmark = pytest.mark.gpu

STORE = {"int8": kp.glm_kv_store_int8, "fp8": kp.glm_kv_store_fp8, "fp4": kp.glm_kv_store_fp4}


def accepted_path(rng, mask, n):
    """A root-to-node path of the tree (the nodes that node i sees, in order), at most n nodes, maybe none."""
    if n == 0 or rng.random() < 0.2:
        return []
    i = int(rng.integers(0, n))
    return [j for j in range(n) if (mask[i] >> j) & 1]


@pytest.mark.parametrize("fmt", ["int8", "fp8", "fp4"])
@pytest.mark.parametrize("H,T", [(16, 4), (64, 6)])
def test_steps(cuda, fmt, H, T):
    rng = np.random.default_rng(H)
    B, bs, pool_blocks, ld_blocks, ld = 5, 16, 60, 12, 180
    n_rows, row = pool_blocks * bs, R.ROW[fmt]
    kind = torch.int8 if fmt == "int8" else torch.uint8
    dims = kp.make_dims(H)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=cuda)                          # noqa: E731
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(cuda)                       # noqa: E731
    cache, draft = torch.zeros((n_rows, row), dtype=kind, device=cuda), torch.zeros((B * T, row), dtype=kind, device=cuda)
    keys = [torch.zeros((B, ld, 128), dtype=torch.bfloat16, device=cuda) for _ in range(2)]
    length, n_blocks, table, slot_map = i32(B), i32(B), i32(B, ld_blocks), torch.full((B, ld), -1, dtype=torch.int64, device=cuda)
    free, n_free = dev(rng.permutation(pool_blocks).astype(np.int32)), i32(1) + pool_blocks
    length2, n_blocks2, free2, n_free2 = i32(B), i32(B), i32(pool_blocks), i32(1)   # the outputs, the inputs of the next call
    slots = torch.zeros(B * 64, dtype=torch.int64, device=cuda)
    q_seq, q_pos, cu = i32(B * 64), i32(B * 64), i32(B + 1)
    ws = torch.zeros(kp.glm_dsa_workspace_size(dims, kp.GLM_OP_TREE_MLA, B, select_k=T, width=ld), dtype=torch.uint8, device=cuda)
    out, lse = torch.zeros((B, T, H, 512), dtype=torch.bfloat16, device=cuda), torch.zeros((B, T, H), device=cuda)
    every = torch.arange(B * T, dtype=torch.int64, device=cuda)
    # the plain side: each request's rows and keys in order, and the tables
    context, state = [[] for _ in range(B)], [[] for _ in range(B)]
    h = dict(length=np.zeros(B, np.int64), held=np.zeros(B, np.int64), table=np.zeros((B, ld_blocks), np.int32),
             free=free.cpu().numpy().copy(), n_free=pool_blocks, map=np.full((B, ld), -1, np.int64))

    def advance(n_new):
        """The block tables of both sides after n_new tokens a request (-1: it ends)."""
        nonlocal length, length2, n_blocks, n_blocks2, free, free2, n_free, n_free2
        kp.glm_block_tables(length, dev(n_new.astype(np.int32)), n_blocks, table, free, n_free, bs, pool_blocks, slots, q_seq, q_pos,
                            length2, n_blocks2, cu, free2, n_free2, slot_map=slot_map)
        length, length2, n_blocks, n_blocks2 = length2, length, n_blocks2, n_blocks
        free, free2, n_free, n_free2 = free2, free, n_free2, n_free
        w = TR.block_tables(h["length"], n_new, h["held"], None, h["table"], h["free"], h["n_free"], bs, pool_blocks, B * 64, ld,
                            h["map"], 0)
        h.update(length=w["len_out"], held=w["n_blocks_out"], table=w["table"], free=w["free_out"], n_free=int(w["n_free_out"][0]),
                 map=w["slot_map"])
        assert np.array_equal(slots.cpu().numpy(), w["slots"]) and np.array_equal(length.cpu().numpy(), w["len_out"])

    def prompt(b, n):
        """A request comes in with n tokens."""
        advance(np.where(np.arange(B) == b, n, 0))
        lat = torch.from_numpy(rng.standard_normal((n, 512)).astype(np.float32)).bfloat16().to(cuda)
        STORE[fmt](dims, lat, slots[:n], cache)
        context[b] = list(cache[slots[:n]].cpu().numpy())
        state[b] = [(np.zeros(128), np.zeros(128))] * n

    for b, n in enumerate([33, 1, 16, 90, 0]):
        if n:
            prompt(b, n)
    for step in range(6):
        n_tree = rng.integers(0, T + 1, B)
        masks = [tree_masks(rng, T) for _ in range(B)]
        q = synth.f32_to_bf16_bits(rng.standard_normal((B, T, H, 512)).astype(np.float32))
        STORE[fmt](dims, torch.from_numpy(rng.standard_normal((B * T, 512)).astype(np.float32)).bfloat16().to(cuda), every, draft)
        dk = [torch.from_numpy(rng.standard_normal((B, T, 128)).astype(np.float32)).bfloat16().to(cuda) for _ in range(2)]
        CALL[fmt](dims, bf16(q).to(cuda), cache, slot_map.int(), draft, as_int64(masks).to(cuda), SM, out, ws, lse=lse,
                  row_len=length, n_tree=dev(n_tree.astype(np.int32)))
        # the plain attention, over the contexts as they were put together
        hd = draft.cpu().numpy()
        flat = [r for c in context for r in c]
        plain = np.stack(flat) if flat else np.zeros((0, row), hd.dtype)
        at = np.concatenate([[0], np.cumsum([len(c) for c in context])])
        lists = np.full((B, ld), -1, np.int32)
        for b in range(B):
            lists[b, :len(context[b])] = np.arange(at[b], at[b + 1])
        o, l = out.float().cpu().numpy(), lse.cpu().numpy()
        for b, i, want, wl, tol, ltol in R.tree(synth.bf16_bits_to_f32(q).astype(np.float64), plain, lists,
                                                [len(c) for c in context], hd, masks, n_tree, SM, fmt):
            assert (np.abs(o[b, i] - want) <= tol).all(), (step, b, i)
            assert np.array_equal(l[b, i], wl) if np.isneginf(wl).all() else (np.abs(l[b, i] - wl) <= ltol).all(), (step, b, i)
        # what is accepted
        paths = [accepted_path(rng, masks[b], int(n_tree[b])) for b in range(B)]
        path = np.full((B, T), -1, np.int32)
        for b, p in enumerate(paths):
            path[b, :len(p)] = p
        advance(np.array([len(p) for p in paths]))
        kp.glm_tree_commit(dims, draft, dev(path), T, slots, q_seq, q_pos, cu, cache, draft_k=dk[0], draft_gate=dk[1], k=keys[0],
                           gate=keys[1])
        hk = [d.float().cpu().numpy() for d in dk]
        for b, p in enumerate(paths):
            context[b] += [hd[b * T + j] for j in p]
            state[b] += [(hk[0][b, j], hk[1][b, j]) for j in p]
            got = cache[torch.from_numpy(h["map"][b, :len(context[b])]).to(cuda)].cpu().numpy()
            assert np.array_equal(got, np.stack(context[b]) if context[b] else got[:0]), (step, b)
            for d in range(2):
                k = keys[d][b, :len(state[b])].float().cpu().numpy()
                new = [j for j, s in enumerate(state[b]) if np.any(s[d])]
                assert all(np.array_equal(k[j], state[b][j][d]) for j in new), (step, b)
        if step in (1, 3):                               # a request ends, another comes into its place
            b = step
            advance(np.where(np.arange(B) == b, -1, 0))
            context[b], state[b] = [], []
            keys[0][b].zero_()
            keys[1][b].zero_()
            prompt(b, int(rng.integers(1, 60)))
