"""Drafted trees and their verification where a kernel's steps meet: items of a
CTA that follow one another closely, values and scores of very different sizes,
rows that are no probabilities."""
import numpy as np
import pytest
import torch

import synth
from oracle import coda_oracle as O
from parity import to_np
from test_drafts_gpu import D, DEV, check_tree, grow, i32, offsets
from test_kvcache_gpu import fill

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def coda():
    import gemm_epilogue_transformer_bf16_gb300 as c
    from gemm_epilogue_transformer_bf16_gb300 import _build
    _build.build()
    c.load()
    return c


def test_many_rows_then_few_unit_by_unit(coda):
    """Sequences of one unit and of a tile of 128 rows and one of 8: the sums at the
    end of the first lie where the weights of the second go.  The same bits in
    every call."""
    batch, n_q, n_kv, n = 900, 8, 1, 17
    nodes, lens = [n] * batch, [n + (7 * i) % 40 for i in range(batch)]
    cache, table, kval, vval, vs = fill(coda, lens, 16, n_kv, True)
    trees = [grow(n, i) for i in range(batch)]
    Q = synth.randn_bf16((n * batch, n_q * D), 1.0, 22).to(DEV)
    ws = coda.workspace(coda.load().coda_attention_tree_nvfp4_workspace_size(n * batch, batch, n_q, n_kv, D))
    args = (Q, cache, table.to(DEV), i32(lens), offsets(nodes), n_q)
    parents = i32([p for t in trees for p in t])
    first = {k: t.clone() for k, t in coda.attention_tree_nvfp4(*args, parents=parents, ws=ws).items() if k in ("O", "lse")}
    for _ in range(30):
        out = coda.attention_tree_nvfp4(*args, parents=parents, ws=ws)
        assert all(torch.equal(out[k], first[k]) for k in first)
    assert coda.get_status(ws) == 0
    check_tree(first, to_np(Q), lens, nodes, trees, kval, vval, vs, n_q, n_kv, D ** -0.5)
