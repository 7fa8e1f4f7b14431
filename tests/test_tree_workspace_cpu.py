"""How much workspace the tree attention asks for (no GPU needed): what its runs can fill, and for every smaller call."""
import random

import pytest

kp = pytest.importorskip("kpool_indexer_int8_b200")

PARTIAL = 512 * 4 + 8                     # bytes of a query row's partial: 512 fp32 numbers, a reference and a sum
SMS = 148


def size(heads, batch, nodes, width):
    return kp.glm_dsa_workspace_size(kp.make_dims(heads), kp.GLM_OP_TREE_MLA, batch, select_k=nodes, width=width)


@pytest.mark.parametrize("heads,batch,nodes,width,rows", [
    (16, 1, 1, 262144, SMS * 16),         # one token: a run of 16 rows for each SM
    (64, 1, 8, 2176, SMS * 64),           # one sequence: as many runs as pairs of SMs, 128 rows each
    (64, 1, 8, 262144, SMS * 64),
    (64, 8, 16, 2176, 2 * SMS * 64),      # several: twice as many, for lists of different lengths
    (64, 4, 13, 4096, 2 * SMS * 64),
    (64, 8, 16, 262144, 8 * SMS * 64),    # long ones: four waves of runs
    (16, 1, 4, 80, 64 * 3),               # a few tiles: each of them
])
def test_what_a_call_asks_for(heads, batch, nodes, width, rows):
    assert size(heads, batch, nodes, width) <= rows * PARTIAL + 3 * 256


def test_every_smaller_call_fits():
    rng = random.Random(1)
    log = lambda hi: int(round(hi ** rng.random()))                        # noqa: E731
    for _ in range(3000):
        heads, nodes = rng.randint(1, 128), log(64)
        batch, width = log(65535 // nodes), log(1 << 20) - 1
        small = size(heads, log(batch), log(nodes), rng.choice((width, log(width + 1) - 1, max(0, width - 64))))
        assert small <= size(heads, batch, nodes, width), (heads, batch, nodes, width)
