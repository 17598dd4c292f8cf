"""Drafted trees where the kernels change gear: tiles of few and of many rows
after one another in a CTA, batches for every cluster size of the verification,
probabilities of very different sizes."""
import numpy as np
import pytest
import torch

import synth
from parity import to_np
from test_drafts_gpu import D, DEV, check_tree, drafts, grow, i32, offsets, oracle_verify, run_verify
from test_kvcache_gpu import fill

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def coda():
    import gemm_epilogue_transformer_bf16_gb300 as c
    from gemm_epilogue_transformer_bf16_gb300 import _build
    _build.build()
    c.load()
    return c


@pytest.mark.parametrize("sizes", [(2, 20), (20, 2, 2, 2), (1, 9, 0, 17), (8, 9)], ids=str)
def test_tiles_of_few_and_many_rows_in_turn(coda, sizes):
    """Groups of eight heads: 8 to 160 rows, several items per CTA."""
    batch, n_q, n_kv = 420, 8, 1
    nodes = [sizes[i % len(sizes)] for i in range(batch)]
    lens = [n + (37 * i) % 300 for i, n in enumerate(nodes)]
    cache, table, kval, vval, vs = fill(coda, lens, 16, n_kv, True)
    trees = [grow(n, i) for i, n in enumerate(nodes)]
    Q = synth.randn_bf16((sum(nodes), n_q * D), 1.0, 21).to(DEV)
    ws = coda.workspace(coda.load().coda_attention_tree_nvfp4_workspace_size(sum(nodes), batch, n_q, n_kv, D))
    args = (Q, cache, table.to(DEV), i32(lens), offsets(nodes), n_q)
    out = coda.attention_tree_nvfp4(*args, parents=i32([p for t in trees for p in t]), ws=ws)
    assert coda.get_status(ws) == 0
    check_tree(out, to_np(Q), lens, nodes, trees, kval, vval, vs, n_q, n_kv, D ** -0.5)


@pytest.mark.parametrize("drawn", [True, False], ids=["drawn", "chosen"])
@pytest.mark.parametrize("batch", [1, 38, 39, 76, 77, 152, 153, 305, 700])
def test_verification_in_clusters_of_every_size(coda, batch, drawn):
    r = np.random.default_rng(batch)
    nodes = [int(n) for n in r.integers(0, 6, size=batch)]
    nodes[0] = 6
    case = drafts(nodes, 301, drawn, torch.float32 if batch % 2 else torch.bfloat16, batch)
    assert run_verify(coda, *case, 7) == oracle_verify(*case, 7)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("drawn", [True, False], ids=["drawn", "chosen"])
def test_verification_of_probabilities_of_all_sizes(coda, drawn, dtype):
    """From 1 down to below 2^-100 in one row (what is below 2^-60 is dropped: a
    sum of 9001 of them is off by 2^-46)."""
    for seed in range(4):
        case = drafts([4, 9, 1, 6], 9001, drawn, dtype, seed, peaked=14.0)
        assert run_verify(coda, *case, 10) == oracle_verify(*case, 10)
