"""The tree attention in fp64 (numpy) and the error that its kernels are allowed.

Reference: for node i of sequence b and head h, over the rows that the node sees,
    s = sm_scale q . c,   out = sum softmax(s) c,   lse = log sum exp(s).

Allowed error, from the arithmetic of the kernels (u32 = 2^-24, half a step of fp32):
  * scores: 512 exact products summed in fp32 and four fp32 multiplications: at most
    ds = 520 u32 sum_d |sm_scale q_d c_d| (+ the fp32 exponent's argument, 4 u32 |s|, and 2 ulp of
    the exponential) for each visible row; a weight is off by 2 ds relative, lse by ds. The query as
    fp16, its largest magnitude in [2^14, 2^15), is exact but for elements below 2^-14, off by 2^-25:
    2^-39 of the largest, so 2^-39 max|q| sm_scale sum_d |c_d| more.
  * softmax weights: a kernel multiplies the codes with P' = 2^x scale_j 4 / sigma in fp16, where x <= 12
    is the score less a reference, and the output is sigma / 4 sum P' code / l. P' is off by 2^-11
    relative, or by 2^-25 once it is below 2^-14. l >= 1, since each reference was some score's when it
    was set, and sigma, a power of two, is at most twice the largest finite scale of the sequence's rows
    and drafts, seen or not: 2^-25 sigma / 4 <= 2^-26 max(scale), times |code_j|, on the output for
    each row.
  * the sums: one accumulation for 16 rows, off by a whole step, 2 u32 (the sums of weights take one
    addition for 64 rows); 80 more for the merged ranges: (n / 8 + 80) u32 relative.
  * the output rounded to bf16: 2^-8 relative.
"""
import numpy as np

import oracle

U32 = 2.0 ** -24
DEQUANT = {"int8": None, "fp8": oracle.dequant_rows_fp8, "fp4": oracle.dequant_rows_fp4}
ROW = {"int8": 528, "fp8": 528, "fp4": 304}


def values(cache, rows, fmt):
    """fp64 values [len(rows), 512] of cache rows."""
    rows = np.asarray(rows, np.int64)
    if len(rows) == 0:
        return np.zeros((0, 512))
    if fmt == "int8":
        raw = np.ascontiguousarray(cache[rows]).view(np.uint8)
        scale = np.ascontiguousarray(raw[:, 512:516]).view(np.float32).astype(np.float64)
        return raw[:, :512].view(np.int8).astype(np.float64) * scale
    return DEQUANT[fmt](cache, rows.astype(np.int32))


def row_scales(cache, rows, fmt):
    at = 288 if fmt == "fp4" else 512
    raw = np.ascontiguousarray(np.ascontiguousarray(cache[np.asarray(rows, np.int64)]).view(np.uint8)[:, at:at + 4])
    return raw.view(np.float32)[:, 0].astype(np.float64)


def node(q, c, scales, sm_scale, top=0.0):
    """(out [H, 512], lse [H], allowed error of out, of lse) of one node over the rows c it sees; top: the
    largest finite scale among the sequence's rows."""
    H = q.shape[0]
    n = c.shape[0]
    if n == 0:
        return np.zeros((H, 512)), np.full(H, -np.inf), np.zeros((H, 512)), np.zeros(H)
    s = (q @ c.T) * sm_scale
    m = s.max(1, keepdims=True)
    e = np.exp(s - m)
    l = e.sum(1, keepdims=True)
    p = e / l
    out = p @ c
    lse = (m + np.log(l))[:, 0]
    ds = 520 * U32 * abs(sm_scale) * (np.abs(q) @ np.abs(c).T) + 4 * U32 * np.abs(s)
    ds = ds + 2.0 ** -39 * abs(sm_scale) * np.abs(q).max(1, keepdims=True) * np.abs(c).sum(1)[None]
    big = ds.max(1) + 2.0 ** -22
    sums = (n / 8 + 80) * U32
    spread = p @ np.abs(c)
    codes = np.where(scales[:, None] > 0, np.abs(c) / np.where(scales > 0, scales, 1.0)[:, None], 2688.0)
    tol = (2.0 ** -8 * np.abs(out) + spread * (2.0 ** -11 + 2 * big + sums)[:, None]
           + 2.0 ** -26 * top * codes.sum(0)[None]) * 1.01 + 1e-30
    return out, lse, tol, (big + sums) * 1.01 + 4 * U32 * np.abs(lse)


def tree(q, cache, rows, row_len, draft, mask, n_tree, sm_scale, fmt, n_rows=None):
    """Every node of a batch: q fp64 [B, T, H, 512]; cache, draft uint8/int8 rows; masks as Python ints.
    Yields (b, i, out, lse, out_tol, lse_tol)."""
    B, T = q.shape[:2]
    n_rows = cache.shape[0] if n_rows is None else n_rows
    for b in range(B):
        t = min(max(int(n_tree[b]), 0), T)
        lst = rows[b][:min(max(int(row_len[b]), 0), rows.shape[1])]
        lst = lst[(lst >= 0) & (lst < n_rows)]
        pre, psc = values(cache, lst, fmt), row_scales(cache, lst, fmt)
        every = np.concatenate([psc, row_scales(draft, np.arange(b * T, b * T + t), fmt)])
        top = float(every[np.isfinite(every)].max(initial=0.0))
        for i in range(T):
            see = [b * T + j for j in range(t) if (int(mask[b][i]) >> j) & 1] if i < t else []
            if i >= t:
                yield (b, i) + node(q[b, i], np.zeros((0, 512)), np.zeros(0), sm_scale)
                continue
            c = np.concatenate([pre, values(draft, see, fmt)])
            sc = np.concatenate([psc, row_scales(draft, see, fmt)])
            yield (b, i) + node(q[b, i], c, sc, sm_scale, top)
