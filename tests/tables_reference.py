"""glm_block_tables and glm_tree_commit in plain Python, written from their definitions."""
import numpy as np

I32 = 2 ** 31 - 1


def block_tables(length, n_new, n_blocks, pad, table, free, n_free, block_size, pool_blocks, n_cap, ld_slot,
                 slot_map, poison):
    """Returns a dict of every output; entries that the call does not write keep `poison` (free_out) or
    their values (table, slot_map)."""
    B, ld_blocks = table.shape
    table = table.copy()
    slot_map = None if slot_map is None else slot_map.copy()
    n_free = min(max(int(n_free), 0), len(free))
    slots, seq, pos = np.full(n_cap, -1, np.int64), np.full(n_cap, -1, np.int32), np.full(n_cap, -1, np.int32)
    len_out, nb_out, cu, back = [], [], [0], []
    off = taken = 0
    for b in range(B):
        ln, nw, held = int(length[b]), int(n_new[b]), int(n_blocks[b])
        pd = 0 if pad is None else int(pad[b])
        first = cu[-1]
        cu.append(first + max(nw, 0))
        if nw < 0:
            back += [int(v) for v in table[b, :min(max(held, 0), ld_blocks)]]
            len_out.append(0)
            nb_out.append(0)
            continue
        sound = pd >= 0 and 0 <= held <= ld_blocks and 0 <= ln <= held * block_size
        want = -(-(ln + nw) // block_size) if ln + nw > 0 else 0
        ok = sound and want <= ld_blocks and cu[-1] <= n_cap and pd + ln + nw <= I32
        if slot_map is not None:
            ok = ok and pd + ln + nw <= ld_slot
        need = max(0, want - held) if ok else 0
        if ok and need > 0:
            ok = off + need <= n_free
            if ok:
                for j in range(need):
                    table[b, held + j] = free[n_free - 1 - off - j]
                taken = off + need
            off += need
        len_out.append(ln + nw if ok else ln)
        nb_out.append(held + need if ok else held)
        if not ok:
            continue
        for i in range(nw):
            t = ln + i
            blk = int(table[b, t // block_size])
            s = blk * block_size + t % block_size if 0 <= blk < pool_blocks else -1
            slots[first + i], seq[first + i], pos[first + i] = s, b, pd + t
            if slot_map is not None:
                slot_map[b, pd + t] = s
    left = n_free - taken
    out = np.full(len(free), poison, np.int32)
    out[:left] = free[:left]
    n = min(len(free), left + len(back))
    out[left:n] = back[:n - left]
    return dict(slots=slots, q_seq=seq, q_pos=pos, slot_map=slot_map, table=table, len_out=np.array(len_out, np.int32),
                n_blocks_out=np.array(nb_out, np.int32), cu_new=np.array([min(v, I32) for v in cu], np.int32),
                free_out=out, n_free_out=np.array([n], np.int32))


def commit(draft, path, n_nodes, slots, q_seq, q_pos, cu_new, cache, draft_k, draft_gate, k, gate):
    """In place on cache, k and gate (numpy)."""
    B = path.shape[0]
    for i in range(len(slots)):
        b = int(q_seq[i])
        if not 0 <= b < B:
            continue
        j = i - int(cu_new[b])
        node = int(path[b, j]) if 0 <= j < path.shape[1] else -1
        if not 0 <= node < n_nodes:
            continue
        if 0 <= slots[i] < cache.shape[0]:
            cache[slots[i]] = draft[b * n_nodes + node]
        if k is not None and 0 <= q_pos[i] < k.shape[1]:
            k[b, q_pos[i]] = draft_k[b, node]
            gate[b, q_pos[i]] = draft_gate[b, node]
