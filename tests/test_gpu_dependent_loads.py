"""What a kernel of a programmatic-dependent chain reads of the kernels before it.

Every kernel of a step may start while the one before it still runs, and waits for it before it
reads what that one writes. The step is run again and again with its index lists poisoned before
each run: an attention CTA that took an index row from before the wait attends to the poison.
"""
import pytest
import torch

import kpool_indexer_int8_b200 as kp
import synth
from kpool_indexer_int8_b200 import pipeline as P
from synth import device as sdev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("chunk,fmt", [(300, "int8"), (300, "fp4"), (1, "int8")])
def test_step_reads_the_index_lists_of_its_own_run(cuda, chunk, fmt):
    # 300 queries: the many-query kernels (selection, expansion and attention in separate launches);
    # one query: the fused ones. The attention alone, on the lists that the step wrote, must agree.
    wl = synth.custom("dependent", (0,), (6000,), n_heads=64, select_k=128, out_width=515, chunk=chunk, seed=44)
    b = sdev.allocate_for(synth.generate(wl), cuda, fp4=fmt == "fp4")
    sdev.load(synth.generate(wl), b, build_prefix=True)
    attend = kp.glm_sparse_mla_decode_fp4 if fmt == "fp4" else kp.glm_sparse_mla_decode
    b.ws_step[-256:].zero_()
    alone = torch.empty_like(b.out)
    for it in range(60):
        for t in (b.topk, b.tok, b.rows):
            t.fill_(4242 - it)
        b.n_sel.fill_(it)
        b.out.fill_(3.0)
        P.run_step(b)
        torch.cuda.synchronize()
        attend(b.dims, b.q, b.cache, b.rows, b.sm_scale, alone, b.ws_mla, lse=b.lse)
        torch.cuda.synchronize()
        assert torch.equal(b.out, alone), (it, torch.nonzero((b.out != alone).flatten(1).any(1)).flatten()[:8].tolist())


def test_step_reads_the_pool_scales_of_its_own_run(cuda):
    # the INT8 indexer state: the scales of the pools that the step itself builds are poisoned before
    # each run, and the scores must be those of the separate calls
    wl = synth.custom("dependent_q8", (0, 0, 0), (6000, 64, 2048), n_heads=16, select_k=16, out_width=80, seed=45)
    b = sdev.allocate_for(synth.generate(wl), cuda, keep_scores=True, q8=True)
    sdev.load(synth.generate(wl), b, build_prefix=True)
    b.ws_step[-256:].zero_()
    P.run_stages(b)
    torch.cuda.synchronize()
    want, seen = b.scores.clone(), torch.isfinite(b.scores)
    for it in range(60):
        for s in range(len(wl.lens)):
            b.pooled_scales[s, int(b.pool_begin[s]):] = 1e6
        P.run_step(b)
        torch.cuda.synchronize()
        assert torch.equal(b.scores[seen], want[seen]), it
