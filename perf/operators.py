"""Cases and plain forms of the speculative-decoding operators over the latent cache.

Three operators that run one after the other in a serving step that drafts several tokens:

  tree    attention of a tree of drafted tokens over the cache rows of their sequence
          (glm_tree_mla_decode, _fp8, _fp4): node i of sequence b sees the rows of its sequence's
          index list and the drafted rows whose bit is set in its mask;
  tables  block tables, slots and slot maps from request lengths (glm_block_tables);
  commit  the accepted drafts' rows and indexer inputs copied to their slots (glm_tree_commit).

``run`` computes the plain form (elementary torch operations in fp32) unless ``own`` is set, when
it makes the library's calls. ``exact`` computes the definition in fp64 (whole numbers with numpy).
Sizes are those of the repository's workloads: 512-wide latents in 528-byte rows (304 for 4-bit
codes), 16 or 64 query heads (up to 128), index lists of 2,051 of 2,176 entries, contexts up to
262,144 tokens, cache blocks of 256 rows.
"""
import math
import random

import numpy as np
import torch

own = False

LATENT = 512
SM_SCALE = LATENT ** -0.5
FORMATS = ("int8", "fp8", "fp4")
ROW_BYTES = {"int8": 528, "fp8": 528, "fp4": 304}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def _tree(name, fmt, batch, nodes, heads, lo, hi, width, ragged=False):
    return dict(name=name, op="tree", fmt=fmt, batch=batch, nodes=nodes, heads=heads, lo=lo, hi=hi, width=width,
                ragged=ragged)


def _tables(name, batch, block, lo, hi, new_lo, new_hi, ended=0, pads=False):
    return dict(name=name, op="tables", batch=batch, block=block, lo=lo, hi=hi, new_lo=new_lo, new_hi=new_hi,
                ended=ended, pads=pads)


def _commit(name, fmt, batch, nodes, path_lo, path_hi, state):
    return dict(name=name, op="commit", fmt=fmt, batch=batch, nodes=nodes, path_lo=path_lo, path_hi=path_hi,
                state=state)


def listed():
    return [
        # a chain of four drafts over the tiny decode's list: the smallest call, where latency counts
        _tree("tree_tiny", "int8", 1, 4, 16, 67, 67, 80),
        # eight drafts over the 2,051 rows that the indexer selects from a long context
        _tree("tree_selected", "int8", 1, 8, 64, 2051, 2051, 2176),
        # eight sequences, sixteen drafts each, over selected FP8 rows
        _tree("tree_selected_batch_fp8", "fp8", 8, 16, 64, 2051, 2051, 2176),
        # short contexts of a mixed batch attended whole, trees of different sizes
        _tree("tree_short_ragged", "int8", 4, 13, 64, 7, 4096, 4096, ragged=True),
        # a single token over a long context of 4-bit rows, 16 heads of a rank: bound by the rows
        _tree("single_token_long_fp4", "fp4", 1, 1, 16, 262144, 262144, 262144),
        # eight drafts over a whole long context
        _tree("tree_long", "int8", 1, 8, 64, 262144, 262144, 262144),
        # the batched decode's eight contexts attended whole by sixteen drafts each: the largest call
        _tree("tree_long_batch", "int8", 8, 16, 64, 32768, 262144, 262144, ragged=True),
        # one decode token for each of the batched decode's sequences
        _tables("tables_decode", 8, 256, 32768, 262144, 1, 1),
        # after verification: one to eight accepted tokens each, some requests ended
        _tables("tables_accepted", 200, 64, 0, 9000, 0, 8, ended=9, pads=True),
        # admission of prompts: every slot of 16 new sequences
        _tables("tables_prompts", 16, 256, 0, 0, 1, 32768, pads=True),
        # four accepted tokens of one sequence
        _commit("commit_one", "int8", 1, 16, 4, 4, True),
        # up to twelve accepted tokens of each of 64 sequences, 4-bit rows
        _commit("commit_batch_fp4", "fp4", 64, 64, 0, 12, True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.random()
    if kind < 0.6:
        heads = rng.choice((1, 3, 8, 16, 20, 32, 40, 64, 64, 96, 128))
        nodes, batch = _log_int(rng, 1, 64), _log_int(rng, 1, 16)
        hi = _log_int(rng, 1, 262144)
        # no more work than the largest listed case
        while batch > 1 and (batch * nodes * heads * hi > 1.0e9 or batch * hi > 1.1e6):
            batch -= 1
        while nodes > 1 and batch * nodes * heads * hi > 1.0e9:
            nodes -= 1
        lo = hi if rng.random() < 0.3 else rng.randint(0, hi)
        return dict(op="tree", fmt=rng.choice(FORMATS), batch=batch, nodes=nodes, heads=heads, lo=lo, hi=hi,
                    width=hi + rng.choice((0, 0, 1, 13, 125)), ragged=rng.random() < 0.5)
    if kind < 0.85:
        batch = _log_int(rng, 1, 512)
        block = rng.choice((16, 64, 128, 256, 256))
        hi = _log_int(rng, 1, min(262144, 1500000 // batch))
        new_hi = _log_int(rng, 1, min(32768, 262144 // batch))
        return dict(op="tables", batch=batch, block=block, lo=rng.randint(0, hi), hi=hi,
                    new_lo=rng.randint(0, new_hi), new_hi=new_hi, ended=rng.choice((0, 0, 3, 7)),
                    pads=rng.random() < 0.5)
    nodes = _log_int(rng, 1, 64)
    path_hi = rng.randint(1, min(nodes, 16))
    return dict(op="commit", fmt=rng.choice(FORMATS), batch=_log_int(rng, 1, 128), nodes=nodes,
                path_lo=rng.randint(0, path_hi), path_hi=path_hi, state=rng.random() < 0.7)


def _spread(lo, hi, n, phase=0.0):
    """n whole numbers over [lo, hi], the first one hi: fixed by the case alone."""
    if n == 1 or lo == hi:
        return [hi] * n
    fr = [(phase + i * 0.6180339887498949) % 1.0 for i in range(n)]
    v = [lo + int(round((hi - lo) * f)) for f in fr]
    v[0] = hi
    return v


def _tree_sizes(c):
    lens = _spread(c["lo"], c["hi"], c["batch"], 0.3)
    nodes = _spread(max(1, c["nodes"] // 2), c["nodes"], c["batch"], 0.1) if c["ragged"] else [c["nodes"]] * c["batch"]
    return lens, nodes


def _tables_sizes(c):
    lens = _spread(c["lo"], c["hi"], c["batch"], 0.3)
    new = _spread(c["new_lo"], c["new_hi"], c["batch"], 0.7)
    if c["ended"]:
        new = [-1 if b % c["ended"] == c["ended"] - 1 else v for b, v in enumerate(new)]
    pads = [(0, 2, 3, 5)[b % 4] if c["pads"] else 0 for b in range(c["batch"])]
    return lens, new, pads


def _commit_sizes(c):
    return _spread(c["path_lo"], c["path_hi"], c["batch"], 0.2)


def work(case):
    c = case
    if c["op"] == "tree":
        lens, nodes = _tree_sizes(c)
        rb = ROW_BYTES[c["fmt"]]
        per_q = c["heads"] * (2 * 2 * LATENT + 4)            # q, out, lse
        by = sum(n * (rb + 4) + t * rb + t * (per_q + 8) + 8 for n, t in zip(lens, nodes))
        # drafted keys: half of the tree's pairs stand for the ancestors a node sees
        fl = sum(4 * LATENT * c["heads"] * t * (n + (t + 1) / 2) for n, t in zip(lens, nodes))
        return {"bytes": by, "flops": fl}
    if c["op"] == "tables":
        lens, new, pads = _tables_sizes(c)
        bs, B = c["block"], c["batch"]
        tok = sum(max(0, v) for v in new)
        held = [(n + bs - 1) // bs for n in lens]
        want = [(n + max(0, v) + bs - 1) // bs for n, v in zip(lens, new)]
        touched = sum(w - n // bs for w, n, v in zip(want, lens, new) if v > 0)
        back = sum(h for h, v in zip(held, new) if v < 0)
        return {"bytes": B * (16 + 12) + tok * 24 + touched * 8 + 8 * (_pool_blocks(c) - sum(held)) + 8 * back,
                "flops": 0}
    tok = sum(_commit_sizes(c))
    return {"bytes": tok * (2 * ROW_BYTES[c["fmt"]] + 16 + 4 + (1024 if c["state"] else 0)) + 4 * c["batch"], "flops": 0}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _latents(n, g):
    x = torch.randn(n, LATENT, device="cuda", generator=g)
    big = torch.rand(n, 1, device="cuda", generator=g) < 0.01       # outlier rows
    return torch.where(big, x * 8.0, x)


def _rows_of(x, fmt):
    """Cache rows (uint8) holding fp32 latents x in one of the three formats."""
    n = x.shape[0]
    amax = x.abs().amax(1, keepdim=True).clamp_min(1e-4)
    row = torch.zeros(n, ROW_BYTES[fmt], dtype=torch.uint8, device="cuda")
    if fmt == "int8":
        s = amax / 127.0
        row[:, :512] = (x / s).round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
        row[:, 512:516] = s.view(torch.uint8)
    elif fmt == "fp8":
        s = amax / 448.0
        row[:, :512] = (x / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        row[:, 512:516] = s.view(torch.uint8)
    else:
        s = amax / 2688.0
        b = x.view(n, 32, 16)
        e = (b.abs().amax(2) / (6.0 * s)).to(torch.float8_e4m3fn)
        d = (e.float() * s).unsqueeze(2)
        y = torch.where(d > 0, b / d, torch.zeros_like(b))
        edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
        code = torch.bucketize(y.abs(), edges).to(torch.uint8) | ((y < 0).to(torch.uint8) << 3)
        code = code.view(n, LATENT)
        row[:, :256] = code[:, 0::2] | (code[:, 1::2] << 4)
        row[:, 256:288] = e.view(torch.uint8)
        row[:, 288:292] = s.view(torch.uint8)
    return row


def _fill_cache(n_rows, fmt, g):
    cache = torch.empty(n_rows, ROW_BYTES[fmt], dtype=torch.uint8, device="cuda")
    for i in range(0, n_rows, 1 << 17):
        m = min(1 << 17, n_rows - i)
        cache[i:i + m] = _rows_of(_latents(m, g), fmt)
    return cache


def _as_kind(rows, fmt):
    return rows.view(torch.int8) if fmt == "int8" else rows


def _tree_mask(nodes, width, py):
    """Masks of a random tree: node i sees its ancestors and itself; unused nodes see nothing."""
    m = []
    for i in range(nodes):
        parent = i - 1 if py.random() < 0.6 else py.randint(-1, i - 1)
        m.append((m[parent] if parent >= 0 else 0) | (1 << i))
    m += [0] * (width - nodes)
    return [v - (1 << 64) if v >= 1 << 63 else v for v in m]


def _prepare_tree(c, seed):
    g, py = _gen(seed), random.Random(seed)
    B, T, H, W, fmt = c["batch"], c["nodes"], c["heads"], max(1, c["width"]), c["fmt"]
    lens, nodes = _tree_sizes(c)
    blocks = [(n + 255) // 256 for n in lens]
    pool = sum(blocks) + 3
    n_rows = pool * 256
    cache = _as_kind(_fill_cache(n_rows, fmt, g), fmt)
    rows = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
    perm = torch.randperm(pool, device="cuda", generator=g)
    at = 0
    for b, n in enumerate(lens):   # the context in block order, or (selected lists) its rows in any order
        r = (perm[at:at + blocks[b]].view(-1, 1) * 256 + torch.arange(256, device="cuda")).view(-1)[:n]
        if n <= 2176:
            r = r[torch.randperm(n, device="cuda", generator=g)]
        rows[b, :n] = r.to(torch.int32)
        at += blocks[b]
    st = dict(
        case=c, lens=lens, nodes=nodes, cache=cache, rows=rows,
        draft=_as_kind(_rows_of(_latents(B * T, g), fmt), fmt),
        q=torch.randn(B, T, H, LATENT, device="cuda", generator=g).to(torch.bfloat16),
        mask=torch.tensor([_tree_mask(n, T, py) for n in nodes], dtype=torch.int64, device="cuda"),
        row_len=torch.tensor(lens, dtype=torch.int32, device="cuda"),
        n_tree=torch.tensor(nodes, dtype=torch.int32, device="cuda"),
        out=torch.zeros(B, T, H, LATENT, dtype=torch.bfloat16, device="cuda"),
        lse=torch.zeros(B, T, H, dtype=torch.float32, device="cuda"))
    if own:
        import kpool_indexer_int8_b200 as kp
        st["dims"] = kp.make_dims(H)
        need = kp.glm_dsa_workspace_size(st["dims"], kp.GLM_OP_TREE_MLA, B, select_k=T, width=W)
        st["ws"] = torch.zeros(max(need, 1), dtype=torch.uint8, device="cuda")
    return st


def _pool_blocks(c):
    lens, new, _ = _tables_sizes(c)
    bs = c["block"]
    return sum((n + max(0, v) + bs - 1) // bs for n, v in zip(lens, new)) + 37


def _prepare_tables(c, seed):
    g = _gen(seed)
    B, bs = c["batch"], c["block"]
    lens, new, pads = _tables_sizes(c)
    held = [(n + bs - 1) // bs for n in lens]
    pool = _pool_blocks(c)
    ld_blocks = max((n + max(0, v) + bs - 1) // bs for n, v in zip(lens, new)) + 1
    ld_slot = max(p + n + max(0, v) for p, n, v in zip(pads, lens, new)) + 1
    n_cap = sum(max(0, v) for v in new) + 3
    perm = torch.randperm(pool, device="cuda", generator=g).to(torch.int32)
    table = torch.full((B, ld_blocks), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = perm[at:at + h]
        at += h
    n_free = pool - at
    free = torch.full((pool,), -1, dtype=torch.int32, device="cuda")
    free[:n_free] = perm[at:]
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(
        case=c, block=bs, pool=pool, table=table, free=free,
        length=torch.tensor(lens, **i32), n_new=torch.tensor(new, **i32), n_blocks=torch.tensor(held, **i32),
        pad=torch.tensor(pads, **i32), n_free=torch.tensor([n_free], **i32),
        slots=torch.full((n_cap,), -7, dtype=torch.int64, device="cuda"), q_seq=torch.full((n_cap,), -7, **i32),
        q_pos=torch.full((n_cap,), -7, **i32),
        slot_map=torch.full((B, ld_slot), -1, dtype=torch.int64, device="cuda"),
        len_out=torch.zeros(B, **i32), n_blocks_out=torch.zeros(B, **i32), cu_new=torch.zeros(B + 1, **i32),
        free_out=torch.full((pool,), -1, **i32), n_free_out=torch.zeros(1, **i32))


def _prepare_commit(c, seed):
    g, py = _gen(seed), random.Random(seed)
    B, T, fmt = c["batch"], c["nodes"], c["fmt"]
    sizes = _commit_sizes(c)
    n_cap = sum(sizes) + 2
    n_rows, ld = 16 * B + 4096, 80
    paths, q_seq, q_pos, cu = [], [], [], [0]
    for b, n in enumerate(sizes):
        paths.append(sorted(py.sample(range(T), n)) + [-1] * (T - n))
        start = py.randint(0, ld - n)
        q_seq += [b] * n
        q_pos += list(range(start, start + n))
        cu.append(cu[-1] + n)
    q_seq += [-1] * (n_cap - len(q_seq))
    q_pos += [-1] * (n_cap - len(q_pos))
    slots = torch.randperm(n_rows, device="cuda", generator=g)[:n_cap]
    slots[cu[-1]:] = -1
    i32 = dict(dtype=torch.int32, device="cuda")

    def keys(*shape):
        return torch.randn(*shape, 128, device="cuda", generator=g).to(torch.bfloat16)
    return dict(
        case=c, draft=_as_kind(_rows_of(_latents(B * T, g), fmt), fmt), cache=_as_kind(_fill_cache(n_rows, fmt, g), fmt),
        path=torch.tensor(paths, **i32), slots=slots, q_seq=torch.tensor(q_seq, **i32),
        q_pos=torch.tensor(q_pos, **i32), cu_new=torch.tensor(cu, **i32), nodes=T,
        draft_k=keys(B, T) if c["state"] else None, draft_gate=keys(B, T) if c["state"] else None,
        k=keys(B, ld) if c["state"] else None, gate=keys(B, ld) if c["state"] else None)


def prepare(case, seed):
    st = {"tree": _prepare_tree, "tables": _prepare_tables, "commit": _prepare_commit}[case["op"]](case, seed)
    if own and "dims" not in st:
        import kpool_indexer_int8_b200 as kp
        st["dims"] = kp.make_dims(64)
    return st


# ------------------------------------------------------------------------------------------------
# the plain forms
# ------------------------------------------------------------------------------------------------
def _dequant(rows, fmt):
    """fp32 values of cache rows."""
    r = rows.view(torch.uint8)
    if fmt == "fp4":
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=r.device)
        pair = r[:, :256]
        code = torch.stack((pair & 15, pair >> 4), 2).view(-1, LATENT).long()
        scale = r[:, 256:288].contiguous().view(torch.float8_e4m3fn).float().repeat_interleave(16, 1)
        return table[code] * scale * r[:, 288:292].contiguous().view(torch.float32)
    codes = r[:, :512].view(torch.int8) if fmt == "int8" else r[:, :512].view(torch.float8_e4m3fn)
    return codes.float() * r[:, 512:516].contiguous().view(torch.float32)


def _plain_tree(st):
    c = st["case"]
    T, H, fmt = c["nodes"], c["heads"], c["fmt"]
    st["out"].zero_()
    st["lse"].fill_(-math.inf)
    bits = torch.arange(T, device="cuda")
    for b, (n, t) in enumerate(zip(st["lens"], st["nodes"])):
        idx = st["rows"][b, :n].long()
        seen = (idx >= 0) & (idx < st["cache"].shape[0])
        keys = _dequant(torch.cat((st["cache"][idx.clamp(0, st["cache"].shape[0] - 1)], st["draft"][b * T:b * T + t])), fmt)
        tree = ((st["mask"][b, :t, None] >> bits[:t]) & 1) != 0                  # [t, t]
        ok = torch.cat((seen.expand(t, n), tree), 1)                             # [t, n + t]
        step = max(1, (1 << 28) // ((n + t) * H))
        for i in range(0, t, step):
            j = min(t, i + step)
            s = (st["q"][b, i:j].float().view(-1, LATENT) @ keys.T).view(j - i, H, n + t) * SM_SCALE
            s = torch.where(ok[i:j, None], s, -math.inf)
            m = s.amax(2, keepdim=True)
            m = torch.where(m == -math.inf, torch.zeros_like(m), m)
            p = torch.exp(s - m)
            l = p.sum(2, keepdim=True)
            o = (p.view(-1, n + t) @ keys).view(j - i, H, LATENT) / torch.where(l > 0, l, torch.ones_like(l))
            st["out"][b, i:j] = o.to(torch.bfloat16)
            st["lse"][b, i:j] = (m + torch.log(l)).squeeze(2)
    return st["out"], st["lse"]


def _plain_tables(st):
    bs, pool = st["block"], st["pool"]
    ln, new, held, pad = (st[k].long() for k in ("length", "n_new", "n_blocks", "pad"))
    table, free, n_free = st["table"], st["free"].long(), st["n_free"].long()
    B, ld_blocks = table.shape
    n_cap, ld_slot = st["slots"].shape[0], st["slot_map"].shape[1]
    add = new.clamp_min(0)
    cu = torch.cat((torch.zeros(1, dtype=torch.int64, device="cuda"), add.cumsum(0)))
    want = (ln + add + bs - 1) // bs
    good = (want <= ld_blocks) & (pad + ln + add <= ld_slot) & (cu[1:] <= n_cap) & (ln <= held * bs) & (new >= 0)
    need = torch.where(good, (want - held).clamp_min(0), torch.zeros_like(want))
    off = need.cumsum(0) - need
    granted = good & ((need == 0) | (off + need <= n_free))
    take = torch.where(granted, need, torch.zeros_like(need))
    taken = take.sum()
    ended = new < 0
    # new blocks of each granted request
    col = torch.arange(ld_blocks, device="cuda")
    j = col - held[:, None]
    fresh = granted[:, None] & (j >= 0) & (j < need[:, None])
    src = (n_free - 1 - off[:, None] - j).clamp(0, free.shape[0] - 1)
    table.copy_(torch.where(fresh, free[src], table.long()).to(torch.int32))
    # packed tokens
    i = torch.arange(n_cap, device="cuda")
    b = torch.searchsorted(cu[1:], i, right=True)
    real = b < B
    b = b.clamp_max(B - 1)
    real &= granted[b]
    pos = ln[b] + i - cu[b]
    blk = table.long()[b, (pos // bs).clamp(0, ld_blocks - 1)]
    slot = torch.where((blk >= 0) & (blk < pool), blk * bs + pos % bs, -1)
    none = torch.full_like(i, -1)
    st["slots"].copy_(torch.where(real, slot, none))
    st["q_seq"].copy_(torch.where(real, b, none).to(torch.int32))
    st["q_pos"].copy_(torch.where(real, pad[b] + pos, none).to(torch.int32))
    # the slot map (tokens that are not real write to a spare last entry)
    flat = torch.cat((st["slot_map"].view(-1), none[:1]))
    flat[torch.where(real, b * ld_slot + pad[b] + pos, B * ld_slot)] = slot
    st["slot_map"].view(-1).copy_(flat[:-1])
    st["cu_new"].copy_(cu.to(torch.int32))
    st["len_out"].copy_(torch.where(ended, 0, torch.where(granted, ln + add, ln)).to(torch.int32))
    st["n_blocks_out"].copy_(torch.where(ended, 0, held + take).to(torch.int32))
    # the free list: what is left of it, then the ended requests' blocks
    left = n_free - taken
    back = torch.where(ended, held, torch.zeros_like(held))
    roff = back.cumsum(0) - back
    spare = free.shape[0]
    dst = torch.where(ended[:, None] & (col < held[:, None]), left + roff[:, None] + col, spare).clamp_max(spare)
    fo = torch.cat((st["free_out"].long(), none[:1]))
    k = torch.arange(spare, device="cuda")
    fo[:-1] = torch.where(k < left, free, fo[:-1])
    fo[dst.view(-1)] = table.long().view(-1)
    st["free_out"].copy_(fo[:-1].to(torch.int32))
    st["n_free_out"].copy_((left + back.sum()).view(1).to(torch.int32))
    return _tables_outputs(st)


def _tables_outputs(st):
    return {k: st[k] for k in ("slots", "q_seq", "q_pos", "slot_map", "len_out", "n_blocks_out", "cu_new", "free_out",
                               "n_free_out", "table")}


def _plain_commit(st):
    B, T = st["path"].shape[0], st["nodes"]
    cache, n_rows = st["cache"], st["cache"].shape[0]
    i = torch.arange(st["slots"].shape[0], device="cuda")
    b = st["q_seq"].long()
    ok = (b >= 0) & (b < B)
    b = b.clamp(0, B - 1)
    j = i - st["cu_new"].long()[b]
    ok &= (j >= 0) & (j < st["path"].shape[1])
    node = st["path"].long()[b, j.clamp(0, st["path"].shape[1] - 1)]
    ok &= (node >= 0) & (node < T)
    node = node.clamp(0, T - 1)
    slot, pos = st["slots"], st["q_pos"].long()
    row_ok = ok & (slot >= 0) & (slot < n_rows)
    at = torch.where(row_ok, slot, 0)
    keep = at[:1] * 0                                          # padding rewrites row 0 with what row 0 gets
    src = torch.where(row_ok[:, None], st["draft"][b * T + node], cache[keep])
    zero = row_ok & (slot == 0)
    src = torch.where((~row_ok & zero.any())[:, None], st["draft"][(b * T + node)[zero.int().argmax()]], src)
    cache[at] = src
    if st["k"] is not None:
        ld = st["k"].shape[1]
        pos_ok = ok & (pos >= 0) & (pos < ld)
        for name in ("k", "gate"):
            flat = torch.cat((st[name].view(-1, 128), st[name].view(-1, 128)[:1]))
            flat[torch.where(pos_ok, b * ld + pos, B * ld)] = st["draft_" + name][b, node]
            st[name].view(-1, 128).copy_(flat[:-1])
    return _commit_outputs(st)


def _commit_outputs(st):
    return [st["cache"]] + ([st["k"], st["gate"]] if st["k"] is not None else [])


# ------------------------------------------------------------------------------------------------
# the library's calls
# ------------------------------------------------------------------------------------------------
def _own_tree(st):
    import kpool_indexer_int8_b200 as kp
    fn = {"int8": kp.glm_tree_mla_decode, "fp8": kp.glm_tree_mla_decode_fp8,
          "fp4": kp.glm_tree_mla_decode_fp4}[st["case"]["fmt"]]
    fn(st["dims"], st["q"], st["cache"], st["rows"], st["draft"], st["mask"], SM_SCALE, st["out"], st["ws"],
       lse=st["lse"], row_len=st["row_len"], n_tree=st["n_tree"])
    return st["out"], st["lse"]


def _own_tables(st):
    import kpool_indexer_int8_b200 as kp
    kp.glm_block_tables(st["length"], st["n_new"], st["n_blocks"], st["table"], st["free"], st["n_free"], st["block"],
                        st["pool"], st["slots"], st["q_seq"], st["q_pos"], st["len_out"], st["n_blocks_out"],
                        st["cu_new"], st["free_out"], st["n_free_out"], pad=st["pad"], slot_map=st["slot_map"])
    return _tables_outputs(st)


def _own_commit(st):
    import kpool_indexer_int8_b200 as kp
    kp.glm_tree_commit(st["dims"], st["draft"], st["path"], st["nodes"], st["slots"], st["q_seq"], st["q_pos"],
                       st["cu_new"], st["cache"], draft_k=st["draft_k"], draft_gate=st["draft_gate"], k=st["k"],
                       gate=st["gate"])
    return _commit_outputs(st)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"tree": _own_tree, "tables": _own_tables, "commit": _own_commit}[op](state)
    return {"tree": _plain_tree, "tables": _plain_tables, "commit": _plain_commit}[op](state)


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def _values64(rows, fmt):
    """What cache rows stand for, in fp64: code times scale (times block scale)."""
    raw = rows.view(torch.uint8)
    at = 288 if fmt == "fp4" else 512
    scale = raw[:, at:at + 4].contiguous().view(torch.float32).double()
    if fmt == "int8":
        return raw[:, :512].contiguous().view(torch.int8).double() * scale
    if fmt == "fp8":
        return raw[:, :512].contiguous().view(torch.float8_e4m3fn).double() * scale
    lut = torch.tensor([v * s for s in (1, -1) for v in E2M1], dtype=torch.float64, device=raw.device)
    val = torch.empty(raw.shape[0], LATENT, dtype=torch.float64, device=raw.device)
    val[:, 0::2] = lut[(raw[:, :256] & 0xF).int()]
    val[:, 1::2] = lut[(raw[:, :256] >> 4).int()]
    block = raw[:, 256:288].contiguous().view(torch.float8_e4m3fn).double()
    return (val.view(-1, 32, 16) * block[:, :, None]).view(-1, LATENT) * scale


def _exact_tree(c, seed):
    st = _prepare_tree(c, seed)
    B, T, H, fmt = c["batch"], c["nodes"], c["heads"], c["fmt"]
    out = torch.zeros(B, T, H, LATENT, dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, H), -math.inf, dtype=torch.float64, device="cuda")
    masks = st["mask"].cpu().numpy().astype(np.uint64)
    for b in range(B):
        t, n = st["nodes"][b], st["lens"][b]
        pre = _values64(st["cache"][st["rows"][b, :n].long()], fmt)
        dr = _values64(st["draft"][b * T:b * T + t], fmt)
        for i in range(t):
            see = [j for j in range(t) if (int(masks[b, i]) >> j) & 1]
            q = st["q"][b, i].double() * SM_SCALE
            s = torch.cat((q @ pre.T, q @ dr[see].T), 1)
            if s.shape[1] == 0:
                continue
            lse[b, i] = torch.logsumexp(s, 1)
            w = torch.exp(s - lse[b, i, :, None])
            out[b, i] = w[:, :n] @ pre + w[:, n:] @ dr[see]
    return out, lse


def _exact_tables(c, seed):
    st = _prepare_tables(c, seed)
    a = {k: v.cpu().numpy().astype(np.int64) for k, v in st.items() if isinstance(v, torch.Tensor)}
    bs, pool = c["block"], st["pool"]
    table, smap, fo = a["table"].copy(), a["slot_map"].copy(), a["free_out"].copy()
    n_cap = a["slots"].shape[0]
    slots, seq, posn = (np.full(n_cap, -1, np.int64) for _ in range(3))
    len_out, nb_out, cu = [], [], [0]
    top, asked, back = int(a["n_free"][0]), 0, []
    left = top
    for b in range(c["batch"]):
        n, add, held, pad = (int(a[k][b]) for k in ("length", "n_new", "n_blocks", "pad"))
        first = cu[-1]
        cu.append(first + max(0, add))
        if add < 0:
            back += [int(v) for v in table[b, :held]]
            len_out.append(0)
            nb_out.append(0)
            continue
        blocks = -(-(n + add) // bs)
        need = max(0, blocks - held)
        asked += need
        if need and asked > top:
            len_out.append(n)
            nb_out.append(held)
            continue
        for k in range(need):
            table[b, held + k] = a["free"][top - asked + need - 1 - k]
        left -= need
        p = np.arange(n, n + add)
        s = table[b, p // bs] * bs + p % bs
        slots[first:first + add], seq[first:first + add], posn[first:first + add] = s, b, pad + p
        smap[b, pad + p] = s
        len_out.append(n + add)
        nb_out.append(max(held, blocks))
    fo[:left] = a["free"][:left]
    fo[left:left + len(back)] = back
    res = dict(slots=slots, q_seq=seq, q_pos=posn, slot_map=smap, len_out=len_out, n_blocks_out=nb_out, cu_new=cu,
               free_out=fo, n_free_out=[left + len(back)], table=table)
    return {k: torch.as_tensor(np.asarray(v), device="cuda").to(st[k].dtype) for k, v in res.items()}


def _exact_commit(c, seed):
    st = _prepare_commit(c, seed)
    path, slots = st["path"].cpu().tolist(), st["slots"].cpu().tolist()
    seq, posn, cu = (st[k].cpu().tolist() for k in ("q_seq", "q_pos", "cu_new"))
    for i, b in enumerate(seq):
        if b < 0:
            continue
        node = path[b][i - cu[b]]
        st["cache"][slots[i]] = st["draft"][b * c["nodes"] + node]
        if c["state"]:
            st["k"][b, posn[i]] = st["draft_k"][b, node]
            st["gate"][b, posn[i]] = st["draft_gate"][b, node]
    return [st["cache"]] + ([st["k"].double(), st["gate"].double()] if c["state"] else [])


def exact(case, seed):
    return {"tree": _exact_tree, "tables": _exact_tables, "commit": _exact_commit}[case["op"]](case, seed)
