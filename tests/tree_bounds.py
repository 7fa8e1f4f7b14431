"""The tree attention in fp64 and the error that its kernels are allowed, from the rows that a node sees alone.

For node i and head h, over the visible rows: s = sm_scale q . c, p = softmax(s), out = sum p c, lse = log sum exp(s).
tests/tree_reference.py bounds the error with the largest scale of a sequence; this bound knows nothing of the
rows that a node does not see, and of a row that it sees only what the row weighs. u32 = 2^-24.

  * scores: s_j is off by ds_j = 520 u32 sum_d |sm_scale q_d c_jd| + 4 u32 |s_j| (512 products summed in fp32, four
    multiplications, the exponent's argument) + 2^-39 max|q| sm_scale sum_d |c_jd| (the query as fp16) + 2^-22 (2 ulp
    of the exponential). A weight is off by p_j (e^ds_j - 1), out by that on |c_j| and, through the sum of the
    weights, by sum_j p_j (e^ds_j - 1) on sum_j p_j |c_j|.
  * softmax weights: the codes are multiplied with P'_j = 2^G p_j scale_j / sigma in fp16, sigma a power of two below
    twice the largest p_j scale_j of the rows seen: off by 2^-11 relative (in tiles of 16 query rows a second fp16
    number holds the rest: by 2^-22), or by at most 2^-25 and by itself when it is below 2^-14, that is by min(p_j scale_j, FLUSH max_j p_j scale_j) |code_j| of the output, FLUSH = 2^(-24 - G).
    (Weights below 2^-120 of the largest may be 0: far below that.)
  * the sums: (n / 8 + 80) u32 relative, as in tests/tree_reference.py; the output as bf16: 2^-8 relative.
"""
import numpy as np

from tests.tree_reference import U32, row_scales, values

FLUSH = 2.0 ** -32                                     # G = 8


def node(q, c, scales, sm_scale, times=None, bits=11):
    """(out [H, 512], lse [H], allowed error of out, of lse) of a node over the rows c that it sees, each of them
    `times` times over (None: once); bits: of a softmax weight."""
    H, n = q.shape[0], c.shape[0]
    if n == 0:
        return np.zeros((H, 512)), np.full(H, -np.inf), np.zeros((H, 512)), np.zeros(H)
    times = np.ones(n) if times is None else np.asarray(times, np.float64)
    mag = np.abs(c)
    s = (q @ c.T) * sm_scale
    m = s.max(1, keepdims=True)
    one = np.exp(s - m)                                # the weight of one of a row's copies
    total = (one * times).sum(1, keepdims=True)
    one = one / total
    p = one * times
    out, lse = p @ c, (m + np.log(total))[:, 0]
    ds = 520 * U32 * abs(sm_scale) * (np.abs(q) @ mag.T) + 4 * U32 * np.abs(s) + 2.0 ** -22
    ds = ds + 2.0 ** -39 * abs(sm_scale) * np.abs(q).max(1, keepdims=True) * mag.sum(1)[None]
    dp = p * np.expm1(np.minimum(ds, 600.0))
    drift = dp.sum(1)
    sums = (times.sum() / 8 + 80) * U32
    spread = p @ mag
    scales = np.abs(scales)
    codes = np.where(scales[:, None] > 0, mag / np.where(scales > 0, scales, 1.0)[:, None], 0.0)
    w = one * scales[None]
    flush = (times * np.minimum(w, FLUSH * w.max(1, keepdims=True))) @ codes
    tol = (2.0 ** -8 * np.abs(out) + dp @ mag + spread * (2.0 ** -bits + drift + sums)[:, None] + flush) * 1.01 + 1e-30
    return out, lse, tol, (drift + sums) * 1.01 + 4 * U32 * np.abs(lse)


def tree(c, sm_scale, q, batch, bits=11):
    """Every node of the sequences `batch` of a case of tests/test_gpu_tree.py, as tests/tree_reference.py's tree; q: fp64.
    Drafts that nobody sees may hold anything."""
    T = q.shape[1]
    for b in batch:
        t = min(max(int(c["n_tree"][b]), 0), T)
        lst = c["rows"][b][:min(max(int(c["row_len"][b]), 0), c["rows"].shape[1])]
        lst = lst[(lst >= 0) & (lst < c["cache"].shape[0])]
        pre, psc = values(c["cache"], lst, c["fmt"]), row_scales(c["cache"], lst, c["fmt"])
        for i in range(T):
            if i >= t:
                yield (b, i) + node(q[b, i], np.zeros((0, 512)), np.zeros(0), sm_scale)
                continue
            see = [b * T + j for j in range(t) if (int(c["masks"][b][i]) >> j) & 1]
            yield (b, i) + node(q[b, i], np.concatenate([pre, values(c["draft"], see, c["fmt"])]),
                                np.concatenate([psc, row_scales(c["draft"], see, c["fmt"])]), sm_scale, bits=bits)
