"""The serving block with drafted tokens, run as it is used: prompts, a tree per
sequence, verification, the accepted rows moved, and the next step on them; with
and without QK-norm.  Each stage is compared with the fp64 oracle on the stage's
actual inputs, so the tolerances are those of the single operators."""
import numpy as np
import pytest
import torch

import synth
from oracle import coda_oracle as O
from parity import assert_bf16, to_np
from test_attention_gpu import check_forward
from test_drafts_gpu import check_tree, grow, i32, offsets
from test_kvcache_gpu import check_decode

pytestmark = pytest.mark.gpu
DEV = "cuda"
D, PAGE, N_Q, N_KV, HIDDEN = 128, 16, 4, 2, 256


@pytest.fixture(scope="module")
def coda():
    import gemm_epilogue_transformer_bf16_gb300 as c
    from gemm_epilogue_transformer_bf16_gb300 import _build
    _build.build()
    c.load()
    return c


def make(norm):
    shape = synth.BlockShape(tokens=64, hidden=HIDDEN, n_q=N_Q, n_kv=N_KV, head_dim=D, inter=512, seq_len=128)
    t = synth.make_block(shape, seed=9)
    if not norm:
        t = {k: v for k, v in t.items() if k not in ("gamma_q", "gamma_k")}
    return shape, t, {k: v.to(DEV) for k, v in t.items()}


SCALING = dict(kind="linear", factor=2.0)


@pytest.mark.parametrize("norm,chain", [(True, False), (False, False), (False, True)])
def test_prompts_trees_verification_and_the_next_token(coda, monkeypatch, norm, chain):
    from gemm_epilogue_transformer_bf16_gb300 import block as B
    shape, t, d = make(norm)
    w = {k: v.double().numpy() for k, v in t.items()}
    rotary, pairing = (D, "interleaved") if norm else (64, "half")
    cache = coda.kv_cache_nvfp4(16, PAGE, N_KV)
    table = torch.randperm(16, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(2, 8)
    blk = B.ServingBlock(shape, d, cache, pairing=pairing, rotary_dim=rotary, scaling=None if norm else SCALING)
    ws = coda.workspace(blk.workspace_size(64, 64, 2))
    seen = {}

    def keep(name):
        real = getattr(B, name)

        def call(*a, **k):
            seen[name] = (a, k, real(*a, **k))
            return seen[name][2]
        monkeypatch.setattr(B, name, call)
    for name in ("attention", "attention_decode_nvfp4", "attention_tree_nvfp4", "rmsnorm_linear", "kv_append_rope_nvfp4"):
        keep(name)

    def slot(b, j):
        j = torch.as_tensor(j)
        return table[b][j // PAGE].long() * PAGE + j % PAGE

    def cached(lens):
        at = [slot(b, torch.arange(n)) for b, n in enumerate(lens)]
        r = [coda.kv_read_nvfp4(cache, a.to(torch.int32).to(DEV), dtype=torch.float32) for a in at]
        return ([to_np(x["K"]) for x in r], [to_np(x["V"]) for x in r],
                [to_np(cache["scale"])[a // PAGE, 1, :, a % PAGE] for a in at])

    def check_projection(x, pos):
        # without QK-norm: the projection's rows against the oracle, then the rotation of what it stored
        Y = seen["rmsnorm_linear"][2][0]
        X = to_np(x)
        r = 1 / np.sqrt((X * X).mean(axis=1) + shape.eps)
        assert_bf16(Y, r[:, None] * (X @ to_np(blk.Wqkv_f).T), "projection")
        f = O.rope_scaled_frequencies(shape.theta, rotary, "linear", 2.0)
        a = np.asarray(pos, dtype=np.float64)[:, None] * f
        _, k, out = seen["kv_append_rope_nvfp4"]
        for got, y, heads in ((out["Q"], Y[:, :N_Q * D], N_Q), (out.get("K"), Y[:, N_Q * D:(N_Q + N_KV) * D], N_KV)):
            if got is None:
                continue
            y = to_np(y).reshape(len(pos), heads, D)
            ref = O.rope_part(y, np.cos(a), np.sin(a), pairing).reshape(len(pos), -1)
            # two products and a sum of at most |pair| in fp32 with a table in fp32, then half a step of bf16
            off = 2.0 ** -8 * np.abs(ref) + 8 * 2.0 ** -24 * np.abs(y).max()
            assert np.all(np.abs(to_np(got) - ref) <= off * (1 + 2.0 ** -8))

    def check_rest(y, x, A, name):
        x1 = to_np(x) + to_np(A) @ w["Wo"].T
        assert_bf16(y, O.mlp_fwd(x1, w["Wg"], w["Wu"], w["Wd"], x1, w["gamma_mlp"], shape.eps)["y"], name)

    # prompts, with two rows of padding
    lens, pad = [30, 21], 2
    x = synth.randn_bf16((51 + pad, HIDDEN), 1.0, 30)
    pos = [j for n in lens for j in range(n)] + [0] * pad
    slots = torch.cat([slot(b, torch.arange(n)) for b, n in enumerate(lens)]).tolist() + [-1] * pad
    y = blk.prefill(x.to(DEV), i32(pos), i32(slots), offsets(lens), ws=ws)
    (Q, K, V, *_), _, out = seen["attention"]
    cu = np.concatenate([[0], np.cumsum(lens)])
    ref = O.attention_fwd(to_np(Q), to_np(K), to_np(V), cu, cu, N_Q, N_KV, D ** -0.5)
    check_forward(out, ref, {"Q": Q.cpu(), "K": K.cpu(), "V": V.cpu()}, cu, cu, N_Q, N_KV, D ** -0.5)
    check_rest(y, x, out["O"], "prefill")
    if not norm:
        check_projection(x, pos)
        # the cache holds the values of the separate append of these rows (its keys
        # are rounded to 4 bits from the fp32 rotation, not from what K holds of it)
        other = coda.kv_cache_nvfp4(16, PAGE, N_KV)
        coda.kv_append_nvfp4(K, V, i32(slots), other)
        every = torch.tensor([s for s in slots if s >= 0], device=DEV)
        for k in ("codes", "sf"):
            a, b = cache[k][:, 1], other[k][:, 1]
            assert torch.equal(a[every // PAGE, :, every % PAGE], b[every // PAGE, :, every % PAGE]), k

    for step, nodes in enumerate(([5, 9], [1, 17])):
        trees = [[i - 1 for i in range(n)] if chain else [-1 if i == 0 else p for i, p in enumerate(grow(n, n + step))]
                 for n in nodes]
        depth = []
        for tr in trees:
            here = []
            for p in tr:
                here.append(0 if p < 0 else here[p] + 1)
            depth.append(here)
        T = sum(nodes)
        x = synth.randn_bf16((T + pad, HIDDEN), 1.0, 50 + step)
        pos = [lens[b] + v for b in range(2) for v in depth[b]] + [0] * pad
        slots = torch.cat([slot(b, lens[b] + torch.arange(n)) for b, n in enumerate(nodes)]).tolist() + [-1] * pad
        parents = None if chain else i32([p for tr in trees for p in tr] + [0] * pad)
        full = [a + b for a, b in zip(lens, nodes)]
        y = blk.tree(x.to(DEV), i32(pos), i32(slots), offsets(nodes), table.to(DEV), i32(full), parents=parents, ws=ws)
        (Q, *_), _, out = seen["attention_tree_nvfp4"]
        check_tree({k: v[:T] for k, v in out.items()}, to_np(Q), full, nodes, trees, *cached(full), N_Q, N_KV, D ** -0.5)
        assert torch.all(out["O"][T:] == 0)
        check_rest(y, x, out["O"], "tree")
        if not norm:
            check_projection(x, pos)
        # drafts of which some are accepted: the target favours the first child of every node
        V = 97
        tokens = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(step))
        at = np.concatenate([[0], np.cumsum(nodes)])
        probs = torch.full((T, V), 1e-4)
        for b, tr in enumerate(trees):
            for i in range(nodes[b] - 1, 0, -1):
                if tr[i] >= 0:
                    probs[at[b] + tr[i], tokens[at[b] + i]] = 0.9
        u, un = torch.full((T,), 0.5), torch.tensor([0.25, 0.75])
        v = coda.verify_drafts(probs.to(DEV), i32(tokens.tolist()), offsets(nodes), u.to(DEV), un.to(DEV), max(nodes),
                               parents=None if chain else parents[:T], ws=ws)
        count, path = v["count"].tolist(), v["nodes"].cpu().numpy()
        kv_before = cached(full)
        new = blk.accept(table.to(DEV), i32(full), offsets(nodes), v["nodes"], v["count"], ws=ws).tolist()
        assert new == [n + 1 + c for n, c in zip(lens, count)] and (step or sum(count) > 0)
        kv_after = cached(new)
        for b in range(2):
            rows = list(range(lens[b])) + [lens[b] + int(i) for i in path[b][:count[b] + 1]]
            for before, after in zip(kv_before, kv_after):
                assert np.array_equal(before[b][rows], after[b])
        lens = new
    # one token more, on the rows as they lie now
    x = synth.randn_bf16((2, HIDDEN), 1.0, 70)
    at = i32([int(slot(b, lens[b])) for b in range(2)])
    full = [n + 1 for n in lens]
    y = blk.decode(x.to(DEV), i32(lens), at, table.to(DEV), i32(full), ws=ws)
    (Q, *_), _, out = seen["attention_decode_nvfp4"]
    check_decode(out, to_np(Q), full, *cached(full), N_Q, N_KV, D ** -0.5)
    check_rest(y, x, out["O"], "decode")
    if not norm:
        check_projection(x, lens)
    assert coda.get_status(ws) == 0


def test_a_chunk_behind_a_prefix_without_qk_norm(coda):
    """The cached keys' path: a chunk's output is that of the tree of the same
    tokens as a chain, to the roundings of both."""
    from gemm_epilogue_transformer_bf16_gb300.block import ServingBlock
    shape, _, d = make(False)
    cache = coda.kv_cache_nvfp4(4, PAGE, N_KV)
    blk = ServingBlock(shape, d, cache)
    x = synth.randn_bf16((40, HIDDEN), 1.0, 3).to(DEV)
    every = i32(list(range(40)))
    blk.prefill(x[:33], every[:33], every[:33], i32([0, 33]))
    chunk = blk.prefill(x[33:], every[33:], every[33:], i32([0, 7]), key_slots=every, cu_seqlens_k=i32([0, 40]))
    kept = {k: v.clone() for k, v in cache.items()}
    tree = blk.tree(x[33:], every[33:], every[33:], i32([0, 7]), i32([[0, 1, 2, 3]]), i32([40]))
    for k in cache:
        assert torch.equal(cache[k].nan_to_num() if cache[k].is_floating_point() else cache[k],
                           kept[k].nan_to_num() if kept[k].is_floating_point() else kept[k]), k
    # attention outputs off by 2^-8 of themselves and 2^-10 of the values' mean size
    # each; the projections behind them carry that on, beside their own 2^-8
    a, b = to_np(chunk), to_np(tree)
    assert np.linalg.norm(a - b) <= 4 * 2.0 ** -8 * np.linalg.norm(b)


def test_status_and_refusals(coda):
    from gemm_epilogue_transformer_bf16_gb300.block import ServingBlock
    shape, _, d = make(False)
    cache = coda.kv_cache_nvfp4(4, PAGE, N_KV)
    blk = ServingBlock(shape, d, cache)
    ws = coda.workspace(blk.workspace_size(6, 6, 2))
    x, tab = synth.randn_bf16((6, HIDDEN), 1.0, 3).to(DEV), i32([[0, 1], [2, 3]])
    good = dict(pos=i32([0, 1, 1, 0, 1, 2]), slots=i32([0, 1, 2, 32, 33, 34]), cu_seqlens=i32([0, 3, 6]), block_table=tab,
                seq_lens=i32([3, 3]), parents=i32([-1, 0, 0, -1, 0, 1]))
    want = blk.tree(x, **good)
    assert torch.equal(blk.tree(x, **good, ws=ws), want) and coda.get_status(ws) == 0
    for change, code in ((dict(parents=i32([-1, 0, 2, -1, 0, 1])), 11), (dict(pos=i32([0, 1, 128, 0, 1, 2])), 8),
                         (dict(slots=i32([0, 1, 64, 32, 33, 34])), 10), (dict(cu_seqlens=i32([0, 3, 7])), 9),
                         (dict(seq_lens=i32([3, 33])), 9), (dict(block_table=i32([[0, 1], [4, 3]])), 10)):
        blk.tree(x, **{**good, **change}, ws=ws)
        assert coda.get_status(ws) == code, change
        coda.reset_status(ws)
    assert torch.equal(blk.tree(x, **good, ws=ws), want) and coda.get_status(ws) == 0
    with pytest.raises(ValueError, match="gamma_q"):
        ServingBlock(shape, {**d, "gamma_q": torch.ones(D, device=DEV)}, cache)
    with pytest.raises(ValueError, match="rotary_dim"):
        ServingBlock(shape, make(True)[2], cache, rotary_dim=64)
    with pytest.raises(ValueError, match="RoPE"):
        ServingBlock(shape, d, cache, pairing="quarter").tree(x, **good)
