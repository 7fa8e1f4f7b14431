"""glm_block_tables and glm_tree_commit against their plain Python definitions: whole numbers and
bytes, so every output must be equal, and what a call does not write must keep its poison."""
import numpy as np
import pytest
import torch

import kpool_indexer_int8_b200 as kp
from tests import tables_reference as R

pytestmark = pytest.mark.gpu

POISON = -77


def request_batch(rng, B, bs, max_len, new_hi, ended=0.0, idle=0.0, pads=False, spare=5, bad=0.0):
    length = rng.integers(0, max_len + 1, B)
    held = -(-length // bs) + rng.integers(0, 2, B)            # some hold a spare block
    n_new = rng.integers(1, new_hi + 1, B)
    n_new[rng.random(B) < idle] = 0
    n_new[rng.random(B) < ended] = -rng.integers(1, 9)
    pool = int(held.sum() + (-(-(length + np.maximum(n_new, 0)) // bs)).sum() + spare)
    ids = rng.permutation(pool).astype(np.int32)
    ld = int(max(held.max(initial=0), (-(-(length + np.maximum(n_new, 0)) // bs)).max(initial=0))) + 1
    table = np.full((B, ld), POISON, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = np.full(pool, POISON, np.int32)
    free[:pool - at] = ids[at:]
    if bad:
        hit = rng.random(table.shape) < bad
        table[hit & (table >= 0)] = rng.choice([-1, pool, 2 ** 31 - 1])
    return dict(length=length.astype(np.int32), n_new=n_new.astype(np.int32), n_blocks=held.astype(np.int32),
                pad=rng.integers(0, 6, B).astype(np.int32) if pads else None, table=table, free=free, n_free=pool - at,
                block_size=bs, pool_blocks=pool)


def run(dev, c, n_cap, ld_slot=None, n_free=None, stream=None):
    B = len(c["length"])
    t = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev)   # noqa: E731
    n_free = c["n_free"] if n_free is None else n_free
    smap = None if ld_slot is None else np.full((B, ld_slot), POISON, np.int64)
    want = R.block_tables(c["length"], c["n_new"], c["n_blocks"], c["pad"], c["table"], c["free"], n_free,
                          c["block_size"], c["pool_blocks"], n_cap, ld_slot, smap, POISON)
    full = lambda n, dt: torch.full((n,), POISON, dtype=dt, device=dev)                      # noqa: E731
    o = dict(slots=full(n_cap, torch.int64), q_seq=full(n_cap, torch.int32), q_pos=full(n_cap, torch.int32),
             len_out=full(B, torch.int32), n_blocks_out=full(B, torch.int32), cu_new=full(B + 1, torch.int32),
             free_out=full(len(c["free"]), torch.int32), n_free_out=full(1, torch.int32), table=t(c["table"]),
             slot_map=t(smap))
    args = (t(c["length"]), t(c["n_new"]), t(c["n_blocks"]), o["table"], t(c["free"]),
            torch.tensor([n_free], dtype=torch.int32, device=dev), c["block_size"], c["pool_blocks"], o["slots"],
            o["q_seq"], o["q_pos"], o["len_out"], o["n_blocks_out"], o["cu_new"], o["free_out"], o["n_free_out"])
    pad = t(c["pad"])
    for _ in range(2):                                      # the same inputs again: the same outputs
        kp.glm_block_tables(*args, pad=pad, slot_map=o["slot_map"], stream=stream)
    torch.cuda.synchronize()
    for name, w in want.items():
        if w is not None:
            g = o[name].cpu().numpy()
            assert np.array_equal(g, w), (name, np.nonzero(g != w)[0][:8], g[g != w][:8], np.asarray(w)[g != w][:8])
    return o


@pytest.mark.parametrize("B,bs,max_len,new_hi,kw", [
    (1, 256, 0, 1, {}), (1, 256, 255, 1, {}), (1, 256, 256, 1, dict(pads=True)), (8, 256, 262144, 1, {}),
    (3, 1, 40, 7, {}), (200, 64, 9000, 8, dict(ended=0.1, idle=0.1, pads=True)), (16, 256, 0, 5000, dict(pads=True)),
    (513, 16, 300, 40, dict(ended=0.3, idle=0.2)), (1025, 128, 1000, 3, dict(pads=True)), (31, 100, 777, 333, {}),
    (8192, 256, 600, 2, dict(ended=0.01)), (7, 65536, 200000, 70000, {}), (40, 32, 500, 20, dict(bad=0.1)),
])
@pytest.mark.parametrize("with_map", [True, False])
def test_block_tables_equal_the_definition(cuda, B, bs, max_len, new_hi, kw, with_map):
    rng = np.random.default_rng(B + bs + max_len)
    c = request_batch(rng, B, bs, max_len, new_hi, **kw)
    tok = int(np.maximum(c["n_new"], 0).sum())
    ld_slot = int((c["length"] + np.maximum(c["n_new"], 0)).max()) + 6 if with_map and B < 1000 else None
    run(cuda, c, tok + 3, ld_slot)


@pytest.mark.parametrize("short", [0, 1, 3, 10 ** 6])
def test_requests_that_do_not_fit_take_nothing(cuda, short):
    # the stack is `short` blocks too small, packed tokens and slot map too small for some
    rng = np.random.default_rng(5)
    c = request_batch(rng, 50, 16, 200, 60, ended=0.1, pads=True)
    tok = int(np.maximum(c["n_new"], 0).sum())
    need = int(np.maximum(-(-(c["length"] + np.maximum(c["n_new"], 0)) // 16) - c["n_blocks"], 0)[c["n_new"] >= 0].sum())
    run(cuda, c, tok, 300, n_free=max(0, need - short))
    run(cuda, c, tok - 200, 300)
    run(cuda, c, tok, 210)
    run(cuda, c, 0, 300)


def test_numbers_that_are_no_requests_are_refused(cuda):
    rng = np.random.default_rng(6)
    c = request_batch(rng, 12, 16, 100, 20, pads=True)
    c["length"][0] = -1
    c["n_blocks"][1] = -5
    c["n_blocks"][2] = c["table"].shape[1] + 1
    c["length"][3] = c["n_blocks"][3] * 16 + 1              # more tokens than its blocks hold
    c["pad"][4] = -2
    c["n_new"][5] = 2 ** 31 - 1                            # past n_cap, every later request too
    c["n_new"][6] = -2 ** 31
    c["n_blocks"][6] = 2 ** 31 - 1                         # ends: at most ld_blocks come back
    run(cuda, c, 400, 200)
    run(cuda, c, 400, None, n_free=-3)
    run(cuda, c, 400, None, n_free=2 ** 31 - 1)


def test_no_requests(cuda):
    rng = np.random.default_rng(7)
    c = request_batch(rng, 3, 16, 100, 20)
    c = dict(c, length=c["length"][:0], n_new=c["n_new"][:0], n_blocks=c["n_blocks"][:0], table=c["table"][:0])
    run(cuda, c, 5)


def commit_case(rng, B, T, fmt, ld_path, hi, n_rows=500, ld=40):
    row = 304 if fmt == "fp4" else 528
    kind = np.int8 if fmt == "int8" else np.uint8
    raw = lambda *s: rng.integers(-128, 128, s).astype(np.int8).view(kind)                   # noqa: E731
    n = rng.integers(0, min(hi, T, ld_path) + 1, B)
    path = np.full((B, ld_path), -1, np.int32)
    seq, pos, cu = [], [], [0]
    for b in range(B):
        path[b, :n[b]] = np.sort(rng.choice(T, n[b], replace=False))
        start = int(rng.integers(0, ld - n[b] + 1))
        seq += [b] * int(n[b])
        pos += list(range(start, start + int(n[b])))
        cu.append(cu[-1] + int(n[b]))
    seq, pos = np.array(seq + [-1] * 2, np.int32), np.array(pos + [-1] * 2, np.int32)
    slots = rng.permutation(n_rows)[:len(seq)].astype(np.int64)
    keys = lambda *s: rng.integers(-2 ** 15, 2 ** 15, s + (128,)).astype(np.int16)           # noqa: E731
    return dict(draft=raw(B * T, row), path=path, n_nodes=T, slots=slots, q_seq=seq, q_pos=pos, cu_new=np.array(cu, np.int32),
                cache=raw(n_rows, row), draft_k=keys(B, T), draft_gate=keys(B, T), k=keys(B, ld), gate=keys(B, ld))


def run_commit(dev, c, state=True):
    t = {k: torch.from_numpy(np.ascontiguousarray(v)).to(dev) for k, v in c.items() if k != "n_nodes"}
    for k in ("draft_k", "draft_gate", "k", "gate"):
        t[k] = t[k].view(torch.bfloat16) if state else None
    kp.glm_tree_commit(kp.make_dims(64), t["draft"], t["path"], c["n_nodes"], t["slots"], t["q_seq"], t["q_pos"],
                       t["cu_new"], t["cache"], draft_k=t["draft_k"], draft_gate=t["draft_gate"], k=t["k"], gate=t["gate"])
    torch.cuda.synchronize()
    w = {k: v.copy() if isinstance(v, np.ndarray) else v for k, v in c.items()}
    R.commit(w["draft"], w["path"], w["n_nodes"], w["slots"], w["q_seq"], w["q_pos"], w["cu_new"], w["cache"],
             w["draft_k"], w["draft_gate"], w["k"] if state else None, w["gate"])
    assert np.array_equal(t["cache"].cpu().numpy(), w["cache"])
    if state:
        assert np.array_equal(t["k"].view(torch.int16).cpu().numpy(), w["k"])
        assert np.array_equal(t["gate"].view(torch.int16).cpu().numpy(), w["gate"])


@pytest.mark.parametrize("fmt", ["int8", "fp8", "fp4"])
@pytest.mark.parametrize("B,T,ld_path,hi", [(1, 1, 1, 1), (1, 16, 16, 4), (64, 64, 12, 12), (5, 7, 9, 7), (3, 4, 0, 4)])
@pytest.mark.parametrize("state", [True, False])
def test_commit_equals_the_definition(cuda, fmt, B, T, ld_path, hi, state):
    run_commit(cuda, commit_case(np.random.default_rng(B * T + hi), B, T, fmt, ld_path, hi), state)


def test_commit_skips_what_is_out_of_range(cuda):
    c = commit_case(np.random.default_rng(9), 8, 16, "int8", 10, 8)
    n = len(c["slots"])
    c["slots"][[0, 3]] = [-1, 500]
    c["slots"][5] = 2 ** 40
    c["q_seq"][[1, 7]] = [8, -9]
    c["q_pos"][[2, 4, 6]] = [-1, 40, 2 ** 31 - 1]
    c["path"][2, 0], c["path"][3, 0], c["path"][4, 0] = 16, -4, 2 ** 31 - 1
    c["cu_new"][6] = n + 5                                    # a token before its request's first
    run_commit(cuda, c)
