"""Drafted tokens over the 4-bit cache against the fp64 oracle: attention of
trees, verification, and the accepted rows' move.

Tolerances of the attention, from the kernel's roundings:

  scores  K' = e2m1 * e4m3 and Q (scaled by a power of two) are exact in f16
          up to f16's smallest step for Q elements far below the row's
          largest (2^-25 of it); 128 products summed in fp32 are off by at
          most 128 * 2^-24 of their absolute sum, and the fp32 factors and sums
          on the way to the exponent by 2^-22 of the terms that they add, which
          are at most the largest score and the logarithms of the values' row
          scales (a weight carries its value's row scale):
            e = scale (128 2^-24 sum|q k| + 128 2^-25 max|q| max|k|)
                + 2^-21 (max|s| + max|log rs|)
  O       weights times row scales are rounded to f16: half a step is 2^-11
          relative, or 2^-25 units where the largest weighted row scale that a
          row sees is at least one unit, times values of at most 2688; O is
          rounded to bf16 once (2^-8); a weight moves by exp(+-2e), and by 2^-21
          for exponentials and reciprocals; the sums over n keys add n 2^-24
          each.
  lse     off by e, n 2^-24, 2^-21, and 2^-22 (|lse| + 16) for the fp32
          logarithms and products.
"""
import numpy as np
import pytest
import torch

import synth
from oracle import coda_oracle as O
from parity import to_np
from test_kvcache_gpu import fill, oracle_rows

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = 128


@pytest.fixture(scope="module")
def coda():
    import gemm_epilogue_transformer_bf16_gb300 as c
    from gemm_epilogue_transformer_bf16_gb300 import _build
    _build.build()
    c.load()
    return c


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def offsets(nodes):
    return i32(np.concatenate([[0], np.cumsum(nodes)]).tolist())


def grow(n, seed):
    """Parents of n nodes, several of them without one among them."""
    r = np.random.default_rng(seed)
    return [-1 if i == 0 or r.random() < 0.05 else int(r.integers(max(0, i - 6), i)) for i in range(n)]


def check_tree(out, Q, lens, nodes, trees, kval, vval, vscale, n_q, n_kv, scale, at=0):
    got, lse = to_np(out["O"]), to_np(out["lse"])
    for b, (keys, n) in enumerate(zip(lens, nodes)):
        if n == 0:
            continue
        q = Q[at:at + n]
        ref = O.tree_attention_fwd(q, kval[b], vval[b], O.tree_sees(trees[b]), n_q, n_kv, scale)
        for h in range(n_q):
            kv = h // (n_q // n_kv)
            c = slice(h * D, (h + 1) * D)
            k = kval[b][:, kv * D:(kv + 1) * D]
            rs = vscale[b][:, kv].astype(np.float64)
            e = (scale * (D * 2.0 ** -24 * np.abs(q[:, c]) @ np.abs(k).T).max(axis=1)
                 + scale * D * 2.0 ** -25 * np.abs(q[:, c]).max(axis=1) * np.abs(k).max()
                 + 2.0 ** -21 * (ref["S"][:, h] + np.abs(np.log(rs)).max()))
            rel = np.expm1(2 * e) + 4 * keys * 2.0 ** -24 + 2.0 ** -20
            small = keys * 2.0 ** -25 * (ref["P"][:, h] * rs).max(axis=1) * 2688
            bound = ((2.0 ** -11 + rel)[:, None] * ref["A"][:, c] * (1 + 2.0 ** -8) + small[:, None]
                     + 2.0 ** -8 * np.abs(ref["O"][:, c]))
            err = np.abs(got[at:at + n, c] - ref["O"][:, c])
            assert np.all(err <= bound), (b, h, float((err - bound).max()), float(err.max()))
            off = np.abs(lse[at:at + n, h] - ref["lse"][:, h])
            assert np.all(off <= e + keys * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -22 * (np.abs(ref["lse"][:, h]) + 16)), (b, h)
        at += n


CASES = {
    # lens (nodes among them), nodes, page, n_q, n_kv, values of very different sizes, std of Q, chain
    "one_node": ([1], [1], 16, 2, 2, False, 1.0, True),
    "one_node_behind": ([40], [1], 16, 8, 1, True, 1.0, False),
    "only_the_tree": ([9, 17], [9, 17], 16, 4, 2, True, 1.0, False),
    "page_ends": ([16, 17, 31, 32, 33], [3, 2, 5, 16, 4], 16, 4, 2, False, 1.0, False),
    "unit_ends": ([127, 128, 129, 255, 257, 130], [3, 7, 2, 5, 9, 4], 64, 8, 1, True, 1.0, False),
    "tree_over_two_units": ([140, 300], [30, 60], 32, 8, 2, True, 1.0, False),
    "no_nodes_among": ([50, 5, 0, 300, 20], [0, 5, 0, 7, 0], 32, 6, 2, True, 1.0, False),
    "all_empty": ([40, 0], [0, 0], 16, 4, 4, False, 1.0, True),
    "wide_group": ([300, 77], [11, 5], 64, 40, 1, True, 1.0, False),
    "odd_group": ([513], [19], 128, 7, 1, True, 1.0, False),
    "rows_128": ([400], [16], 64, 8, 1, True, 1.0, True),
    "rows_129": ([400], [43], 64, 3, 1, True, 1.0, False),
    "rows_600": ([700, 100], [75, 10], 64, 8, 1, True, 1.0, False),
    "long_chain": ([500], [300], 64, 4, 2, False, 1.0, True),
    "largest_tree": ([300], [256], 16, 2, 1, True, 1.0, False),
    "split_over_ctas": ([9000, 300], [6, 3], 256, 8, 1, True, 1.0, False),
    "wide_and_split": ([5000], [40], 128, 16, 2, True, 1.0, False),
    "peaked": ([700, 190], [8, 5], 64, 8, 2, True, 60.0, False),
    "flat": ([700, 90], [8, 5], 64, 8, 2, True, 0.0, False),
    "tiny_q": ([300], [6], 64, 4, 1, False, 2.0 ** -40, False),
    "many": (list(range(8, 60)), [1 + i % 8 for i in range(52)], 16, 8, 8, False, 1.0, False),
    "more_than_threads": ([3 + (7 * i) % 41 for i in range(600)], [i % 3 for i in range(600)], 16, 2, 1, True, 1.0, False),
}


@pytest.mark.parametrize("name", CASES)
def test_tree_attention(coda, name):
    lens, nodes, page, n_q, n_kv, spread, std, chain = CASES[name]
    cache, table, kval, vval, vs = fill(coda, lens, page, n_kv, spread)
    trees = [[i - 1 for i in range(n)] if chain else grow(n, i) for i, n in enumerate(nodes)]
    T, pad = sum(nodes), 3
    wide = synth.randn_bf16((T + pad, n_q * D + 64), std, 99).to(DEV)
    Q = wide[:, 64:]                                     # columns of a wider tensor, rows behind the last sequence
    out = {"O": torch.full((T + pad, n_q * D), 5.0, dtype=torch.bfloat16, device=DEV),
           "lse": torch.full((T + pad, n_q), 5.0, device=DEV)}
    parents = None if chain else i32([p for t in trees for p in t] + [0] * pad)
    ws = coda.workspace(coda.load().coda_attention_tree_nvfp4_workspace_size(T + pad, len(lens), n_q, n_kv, D))
    got = coda.attention_tree_nvfp4(Q, cache, table.to(DEV), i32(lens), offsets(nodes), n_q, parents=parents, out=out, ws=ws)
    assert coda.get_status(ws) == 0
    assert torch.all(got["O"][T:] == 5) and torch.all(got["lse"][T:] == 5)
    check_tree(got, to_np(Q), lens, nodes, trees, kval, vval, vs, n_q, n_kv, D ** -0.5)
    again = coda.attention_tree_nvfp4(Q, cache, table.to(DEV), i32(lens), offsets(nodes), n_q, parents=parents)
    assert torch.equal(again["O"][:T], got["O"][:T]) and torch.equal(again["lse"][:T], got["lse"][:T])


def test_rising_scores(coda):
    """Every block of keys holds larger scores than those before it: the running
    maximum rises all the way."""
    n_q, n_kv, page, keys, n = 4, 1, 64, 1500, 5
    cache = coda.kv_cache_nvfp4(30, page, n_kv)
    K, V = synth.randn_bf16((keys, D), 1.0, 1).float(), synth.randn_bf16((keys, D), 1.0, 2).float()
    K[:, :64] = 0.02 * torch.arange(keys).unsqueeze(1)
    V *= torch.exp2(torch.arange(keys) * -0.02).unsqueeze(1)
    K, V = K.to(torch.bfloat16), V.to(torch.bfloat16)
    slots = torch.arange(keys, dtype=torch.int32)
    coda.kv_append_nvfp4(K.to(DEV), V.to(DEV), slots.to(DEV), cache)
    Q = synth.randn_bf16((n, n_q * D), 0.1, 3).float()
    Q.view(n, n_q, D)[..., :64] = 0.5
    Q = Q.to(torch.bfloat16)
    got = coda.attention_tree_nvfp4(Q.to(DEV), cache, torch.arange(30, dtype=torch.int32, device=DEV).view(1, 30), i32([keys]),
                                    offsets([n]), n_q)
    (_, _, _, kv), (_, _, sc, vv) = oracle_rows(K, 1), oracle_rows(V, 1)
    check_tree(got, to_np(Q), [keys], [n], [[i - 1 for i in range(n)]], [kv], [vv], [sc], n_q, n_kv, D ** -0.5)


def test_values_of_all_sizes_and_zero_rows(coda):
    """Values from 2^-60 to 2^60, rows of zeros where the weights are largest."""
    n_q, n_kv, page, keys, n = 4, 1, 64, 400, 6
    cache = coda.kv_cache_nvfp4(8, page, n_kv)
    K, V = synth.randn_bf16((keys, D), 1.0, 1), synth.randn_bf16((keys, D), 1.0, 2).float()
    for exponent in (-60, 60):
        v = V * 2.0 ** exponent
        v[::3] = 0
        v[128:256] = 0
        v = v.to(torch.bfloat16)
        coda.kv_append_nvfp4(K.to(DEV), v.to(DEV), torch.arange(keys, dtype=torch.int32, device=DEV), cache)
        Q = synth.randn_bf16((n, n_q * D), 1.0, 3)
        got = coda.attention_tree_nvfp4(Q.to(DEV), cache, torch.arange(8, dtype=torch.int32, device=DEV).view(1, 8),
                                        i32([keys]), offsets([n]), n_q)
        (_, _, _, kv), (_, _, sc, vv) = oracle_rows(K, 1), oracle_rows(v, 1)
        sc = np.where(np.abs(vv).max(axis=1, keepdims=True) == 0, 2.0 ** (exponent - 9.0), sc)    # a row of zeros has no size
        check_tree(got, to_np(Q), [keys], [n], [[i - 1 for i in range(n)]], [kv], [vv], [sc], n_q, n_kv, D ** -0.5)
    v.zero_()
    coda.kv_append_nvfp4(K.to(DEV), v.to(DEV), torch.arange(keys, dtype=torch.int32, device=DEV), cache)
    zero = coda.attention_tree_nvfp4(Q.to(DEV), cache, torch.arange(8, dtype=torch.int32, device=DEV).view(1, 8),
                                     i32([keys]), offsets([n]), n_q)
    assert torch.all(zero["O"] == 0) and torch.all((zero["lse"] - got["lse"]).abs() < 1e-4)


@pytest.mark.parametrize("n_q, n, sick", [(4, 9, 2), (16, 30, 7)])
def test_infinities_reach_only_the_nodes_that_see_them(coda, n_q, n, sick):
    """A drafted token with infinite values (or keys), and one with NaN scales:
    its descendants are not finite, the other nodes as without it."""
    n_kv, page, keys = 1, 32, 200
    cache, table, kval, vval, vs = fill(coda, [keys], page, n_kv, False)
    tree = [-1] + [0] * 8 + [1 + i % 8 for i in range(n - 9)]
    Q = synth.randn_bf16((n, n_q * D), 1.0, 5).to(DEV)
    call = lambda: coda.attention_tree_nvfp4(Q, cache, table.to(DEV), i32([keys]), offsets([n]), n_q, parents=i32(tree))
    want = call()
    at = keys - n + sick
    slot = i32([int(table[0, at // page]) * page + at % page])
    old = {k: t.clone() for k, t in cache.items()}
    sees = torch.from_numpy(O.tree_sees(tree)[:, sick])
    for what in ("V inf", "K inf", "V nan scale", "V nan blocks"):
        for k in cache:
            cache[k].copy_(old[k])
        x = torch.ones(1, D, dtype=torch.bfloat16, device=DEV)
        bad = x.clone()
        bad[0, 5] = float("inf")
        if what == "V nan scale":
            cache["scale"].view(-1, 2, page)[int(slot) // page, 1, int(slot) % page] = float("nan")
        elif what == "V nan blocks":
            cache["sf"].view(-1, 2, page, 8)[int(slot) // page, 1, int(slot) % page] = 0x7F
        else:
            coda.kv_append_nvfp4(bad if what == "K inf" else x, bad if what == "V inf" else x, slot, cache)
        got = call()
        finite = torch.isfinite(got["O"].float()).all(dim=1).cpu()
        assert torch.equal(finite, ~sees), what
        # A hidden value meets a weight of exactly 0, so nothing is added; but a
        # step of the product sums 16 keys in fp32 aligned to the largest operands,
        # and 2^-14 (f16's smallest exponent, which a zero has) times 2688 may be the
        # largest, so the other keys' terms may lose bits below 2^-25 of 2688 units
        # in a step: within the bound's term for the rounding of small weights.
        hidden = (~sees).to(DEV).unsqueeze(1)
        rest = {k: torch.where(hidden, got[k], want[k]) for k in ("O", "lse")}
        check_tree(rest, to_np(Q), [keys], [n], [tree], kval, vval, vs, n_q, n_kv, D ** -0.5)
        assert torch.equal(rest["lse"], want["lse"])


def test_bad_trees_lengths_and_pages_set_status(coda):
    n_q, n_kv, page, lens, nodes = 4, 2, 16, [40, 20, 33], [5, 4, 6]
    cache, table, kval, vval, vs = fill(coda, lens, page, n_kv, False)
    T = sum(nodes)
    Q = synth.randn_bf16((T, n_q * D), 1.0, 5)
    ws = coda.workspace(coda.load().coda_attention_tree_nvfp4_workspace_size(T, 3, n_q, n_kv, D))
    trees = [grow(n, 7 + n) for n in nodes]

    def run(tab=table, n=lens, cu=None, parents=trees):
        out = {"O": torch.full((T, n_q * D), 5.0, dtype=torch.bfloat16, device=DEV), "lse": torch.full((T, n_q), 5.0, device=DEV)}
        return coda.attention_tree_nvfp4(Q.to(DEV), cache, tab.to(DEV), i32(n), cu if cu is not None else offsets(nodes), n_q,
                                         parents=i32([p for t in parents for p in t]), out=out, ws=ws)

    def rest(out, but):
        for b in range(3):
            if b != but:
                check_tree(out, to_np(Q), [lens[b]], [nodes[b]], [trees[b]], [kval[b]], [vval[b]], [vs[b]], n_q, n_kv,
                           D ** -0.5, at=sum(nodes[:b]))
    # parents that are no earlier node: the node sees the prefix and itself
    for bad in (2, 3, 99, -2):
        other = [list(t) for t in trees]
        other[0][2] = bad
        out = run(parents=other)
        assert coda.get_status(ws) == 11                 # CODA_ERR_TREE_RANGE
        coda.reset_status(ws)
        rest(out, 0)
        other[0][2] = -1
        assert torch.equal(run(parents=other)["O"], out["O"]) and coda.get_status(ws) == 0
    # lengths below the tree or beyond the table
    for bad in (-1, 3, table.shape[1] * page + 1):
        out = run(n=[40, bad, 33])
        assert coda.get_status(ws) == 9                  # CODA_ERR_SEQLEN_RANGE
        coda.reset_status(ws)
        rest(out, 1)
        assert torch.all(out["O"][5:9] == 0) and torch.all(torch.isneginf(out["lse"][5:9]))
    # offsets that leave the tensor, or fall
    out = run(cu=i32([0, 5, 9, 200]))
    assert coda.get_status(ws) == 9
    coda.reset_status(ws)
    rest(out, 2)
    run(cu=i32([0, 9, 5, 15]))
    assert coda.get_status(ws) == 9
    coda.reset_status(ws)
    # pages outside the cache: their keys are left out
    for bad in (-1, cache["scale"].shape[0]):
        tab = table.clone()
        tab[0, 1] = bad                                  # keys 16 .. 31 of sequence 0
        out = run(tab=tab)
        assert coda.get_status(ws) == 10                 # CODA_ERR_PAGE_RANGE
        coda.reset_status(ws)
        keep = np.r_[0:16, 32:40]
        check_tree(out, to_np(Q), [24], [5], [trees[0]], [kval[0][keep]], [vval[0][keep]], [vs[0][keep]], n_q, n_kv, D ** -0.5)
        rest(out, 0)


def test_trees_too_large_get_zeros(coda):
    n_q, n_kv, page, lens, nodes = 2, 1, 64, [300, 40], [257, 5]
    cache, table, kval, vval, vs = fill(coda, lens, page, n_kv, False)
    Q = synth.randn_bf16((262, n_q * D), 1.0, 5)
    trees = [grow(n, n) for n in nodes]
    out = coda.attention_tree_nvfp4(Q.to(DEV), cache, table.to(DEV), i32(lens), offsets(nodes), n_q,
                                    parents=i32([p for t in trees for p in t]))
    assert coda.get_status(out["ws"]) == 11
    assert torch.all(out["O"][:257] == 0) and torch.all(torch.isneginf(out["lse"][:257]))
    check_tree(out, to_np(Q), lens[1:], nodes[1:], trees[1:], kval[1:], vval[1:], vs[1:], n_q, n_kv, D ** -0.5, at=257)


def test_one_node_is_single_token_attention(coda):
    """A tree of one node per sequence and attention_decode_nvfp4 agree within
    both kernels' bounds (each is held to them elsewhere)."""
    lens, n_q, n_kv = [5, 700, 129], 16, 2
    cache, table, *_ = fill(coda, lens, 64, n_kv, True)
    Q = synth.randn_bf16((3, n_q * D), 1.0, 5).to(DEV)
    a = coda.attention_decode_nvfp4(Q, cache, table.to(DEV), i32(lens), n_q)
    b = coda.attention_tree_nvfp4(Q, cache, table.to(DEV), i32(lens), offsets([1, 1, 1]), n_q)
    x, y = a["O"].float(), b["O"].float()
    assert float((x - y).norm() / x.norm()) < 2.0 ** -8 and torch.all((a["lse"] - b["lse"]).abs() < 1e-4)


def test_attention_offsets_beyond_32_bits(coda):
    n_q, n_kv, page = 8, 8, 256
    pages = (1 << 32) // (2 * n_kv * page * 64) + 40     # codes alone pass 4 GiB
    cache = {"codes": torch.zeros(pages, 2, n_kv, page, 64, dtype=torch.uint8, device=DEV),
             "sf": torch.zeros(pages, 2, n_kv, page, 8, dtype=torch.uint8, device=DEV),
             "scale": torch.zeros(pages, 2, n_kv, page, device=DEV)}
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32)
    j = torch.arange(300)
    slots = (table[0][j // page].long() * page + j % page).to(torch.int32)
    K, V = synth.randn_bf16((300, n_kv * D), 1.0, 1), synth.randn_bf16((300, n_kv * D), 1.0, 2)
    cs = coda.rope_table(1e4, 128, 300)
    coda.kv_append_rope_nvfp4(K.to(DEV), V.to(DEV), slots.to(DEV), cache, i32([0] * 300), cs)
    Q = synth.randn_bf16((3, n_q * D), 1.0, 5)
    out = coda.attention_tree_nvfp4(Q.to(DEV), cache, table.to(DEV), i32([300]), offsets([3]), n_q, parents=i32([-1, 0, 0]))
    (_, _, _, kv), (_, _, sc, vv) = oracle_rows(K, n_kv), oracle_rows(V, n_kv)
    check_tree(out, to_np(Q), [300], [3], [[-1, 0, 0]], [kv], [vv], [sc], n_q, n_kv, D ** -0.5)
    # the last node takes the place of the first draft
    new = coda.kv_accept_nvfp4(cache, table.to(DEV), i32([300]), offsets([3]), i32([[0, 2]]), i32([1]))["seq_lens"]
    back = coda.kv_read_nvfp4(cache, slots[-3:].to(DEV), dtype=torch.float32)["V"].cpu()
    assert new.tolist() == [299] and torch.equal(back, torch.from_numpy(vv[[297, 299, 299]]).float())


# --------------------------------------------------------------------------- verification

def drafts(nodes, V, drawn, dtype, seed, chain=False, peaked=3.0):
    """Probabilities, trees and tokens as a drafting model leaves them; random
    numbers with full fp32 fractions."""
    r = np.random.default_rng(seed)
    T = sum(nodes)
    z = r.normal(size=(T, V)) * peaked
    soft = lambda z: np.exp(z - z.max(axis=1, keepdims=True)) / np.exp(z - z.max(axis=1, keepdims=True)).sum(axis=1, keepdims=True)
    P = torch.from_numpy(soft(z)).to(dtype)
    Q = torch.from_numpy(soft(z + r.normal(size=(T, V)))).to(dtype)
    trees, tokens, at = [], np.zeros(T, dtype=np.int64), 0
    for n in nodes:
        t = [i - 1 if chain or i == 0 else int(r.integers(max(0, i - 4), i)) for i in range(n)]
        for i in range(1, n):
            q = Q[at + t[i]].double().numpy() if drawn else P[at + t[i]].double().numpy()
            tokens[at + i] = r.choice(V, p=q / q.sum())
        trees.append(t)
        at += n
    return P, Q if drawn else None, trees, tokens, r.random(T).astype(np.float32), r.random(len(nodes)).astype(np.float32)


def oracle_verify(P, Q, trees, tokens, u, un, width, at=0):
    count, nodes, text = [], [], []
    for b, t in enumerate(trees):
        n = len(t)
        if n == 0:
            path, words = [], []
        else:
            p, q = P[at:at + n].double().numpy(), Q[at:at + n].double().numpy() if Q is not None else None
            path, words = O.verify_drafts(p, tokens[at:at + n], t, u[at:at + n].astype(np.float64), float(un[b]), q, width)
        count.append(max(len(path) - 1, 0))
        nodes.append(path + [-1] * (width - len(path)))
        text.append(words + [-1] * (width - len(words)))
        at += n
    return count, nodes, text


def run_verify(coda, P, Q, trees, tokens, u, un, width, chain=False, ws=None):
    out = coda.verify_drafts(P.to(DEV), i32(tokens.tolist()), offsets([len(t) for t in trees]), torch.from_numpy(u).to(DEV),
                             torch.from_numpy(un).to(DEV), width, parents=None if chain else i32([p for t in trees for p in t]),
                             draft_probs=Q.to(DEV) if Q is not None else None, ws=ws)
    return tuple(out[k].tolist() for k in ("count", "nodes", "tokens"))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("drawn", [True, False], ids=["drawn", "chosen"])
@pytest.mark.parametrize("nodes, V, chain", [
    ([1], 1, True), ([1, 2, 3], 7, True), ([5, 0, 9, 1], 50, False), ([12] * 20, 33, False), ([40, 3], 1001, False),
    ([6] * 9, 4097, True), ([8, 8, 8, 30], 30011, False), ([5, 5], 128256, False)])
def test_verification(coda, nodes, V, chain, drawn, dtype):
    for seed in range(3):
        P, Q, trees, tokens, u, un = drafts(nodes, V, drawn, dtype, seed, chain)
        width = max(nodes) + 1
        ws = coda.workspace(coda.load().coda_verify_drafts_workspace_size(sum(nodes), len(nodes), V))
        got = run_verify(coda, P, Q, trees, tokens, u, un, width, chain, ws)
        assert coda.get_status(ws) == 0
        assert got == oracle_verify(P, Q, trees, tokens, u, un, width)


@pytest.mark.parametrize("drawn", [True, False], ids=["drawn", "chosen"])
def test_verification_of_many_children_and_the_same_token_twice(coda, drawn):
    """Stars of forty drafts: many refusals at one node, tokens drafted again."""
    V, n = 12, 41
    for seed in range(8):
        r = np.random.default_rng(seed)
        P, Q, _, _, u, un = drafts([n] * 3, V, drawn, torch.float32, seed, peaked=0.3)
        trees = [[-1] + [0] * (n - 1)] * 3
        tokens = r.integers(0, V, size=3 * n)
        u = (1 - 0.02 * r.random(3 * n)).astype(np.float32)          # nearly always refused
        assert run_verify(coda, P, Q, trees, tokens, u, un, 5) == oracle_verify(P, Q, trees, tokens, u, un, 5)


def test_verification_at_the_edges(coda):
    """Random numbers of 0 and just below 1, probabilities of 0 and 1, a walk
    that the width ends, nothing left to take."""
    one = float(np.nextafter(np.float32(1), np.float32(0)))
    V = 10
    P = torch.zeros(4, V)
    P[0, 3] = P[1, 9] = P[2, 0] = 1.0
    P[3, 2:4] = 0.5
    tokens, trees = np.array([0, 3, 9, 0]), [[-1, 0, 1, 2]]
    for un, last in ((0.0, 2), (one, 3), (0.5, 3), (0.49, 2)):
        for u in (0.0, one):
            got = run_verify(coda, P, None, trees, tokens, np.full(4, u, np.float32), np.array([un], np.float32), 6)
            assert got == ([3], [[0, 1, 2, 3, -1, -1]], [[3, 9, 0, last, -1, -1]])
    got = run_verify(coda, P, None, trees, tokens, np.zeros(4, np.float32), np.array([0.2], np.float32), 2)
    assert got == ([1], [[0, 1]], [[3, 9]])
    # the only token with a probability is refused: its own row decides; a row of zeros: -1
    got = run_verify(coda, P, P, [[-1, 0, -1, -1]], np.array([0, 5, 0, 0]), np.zeros(4, np.float32), np.zeros(1, np.float32), 2)
    assert got == ([0], [[0, -1]], [[3, -1]])
    got = run_verify(coda, P * 0, None, [[-1, 0, 1, 2]], tokens, np.zeros(4, np.float32), np.zeros(1, np.float32), 2)
    assert got == ([0], [[0, -1]], [[-1, -1]])
    bad = P.clone()
    bad[0] = torch.tensor([float("nan"), -1.0, float("-inf"), 0.0, float("inf"), 0.0, 0.0, 0.0, 0.0, 0.0])
    got = run_verify(coda, bad, None, [[-1, -1, -1, -1]], tokens, np.zeros(4, np.float32), np.array([0.9], np.float32), 2)
    assert got == ([0], [[0, -1]], [[4, -1]])


def test_verification_s_range_errors(coda):
    nodes, V = [5, 6, 4], 100
    P, Q, trees, tokens, u, un = drafts(nodes, V, True, torch.float32, 1)
    u[:] = 0
    ws = coda.workspace(coda.load().coda_verify_drafts_workspace_size(15, 3, V))
    want = oracle_verify(P, Q, trees, tokens, u, un, 7)
    for bad in (5, 9, -3):                               # never a child
        other = [list(t) for t in trees]
        other[1][2] = bad
        got = run_verify(coda, P, Q, other, tokens, u, un, 7, ws=ws)
        assert coda.get_status(ws) == 11
        coda.reset_status(ws)
        other[1][2] = -1
        assert got == oracle_verify(P, Q, other, tokens, u, un, 7)
    for bad in (-1, V, 1 << 30):
        x = tokens.copy()
        x[5 + 1] = bad
        got = run_verify(coda, P, Q, trees, x, u, un, 7, ws=ws)
        assert coda.get_status(ws) == 7                  # CODA_ERR_LABEL_RANGE
        coda.reset_status(ws)
        other = [trees[0], [-1, -1] + trees[1][2:], trees[2]]
        assert got == oracle_verify(P, Q, other, tokens, u, un, 7)
    x = i32(tokens.tolist())
    call = lambda cu: coda.verify_drafts(P.to(DEV), x, i32(cu), torch.from_numpy(u).to(DEV), torch.from_numpy(un).to(DEV), 7,
                                         parents=i32([p for t in trees for p in t]), draft_probs=Q.to(DEV), ws=ws)
    out = call([0, 5, 11, 99])
    assert coda.get_status(ws) == 9 and out["count"].tolist() == want[0][:2] + [0]
    assert out["nodes"].tolist()[:2] == want[1][:2] and out["tokens"].tolist()[2] == [-1] * 7
    coda.reset_status(ws)
    T = 1025                                             # a tree beyond the limit beside an ordinary one
    big = coda.verify_drafts(torch.rand(T + 2, 8, device=DEV), torch.zeros(T + 2, dtype=torch.int32, device=DEV), i32([0, T, T + 2]),
                             torch.zeros(T + 2, device=DEV), torch.zeros(2, device=DEV), 3, ws=ws)
    assert coda.get_status(ws) == 11 and big["count"].tolist() == [0, 1] and big["nodes"].tolist()[0] == [-1] * 3


# --------------------------------------------------------------------------- what stays

@pytest.mark.parametrize("page, n_kv, paths", [
    (16, 1, [[0, 1, 2]]), (16, 3, [[0, 2, 5], [0], [0, 1, 4, 5, 9, 12], []]), (32, 2, [[0] + list(range(3, 40, 2)), [0, 7]]),
    (256, 8, [[0, 3], [0, 1, 2, 9]])])
def test_accepted_rows_move(coda, page, n_kv, paths):
    nodes = [p[-1] + 3 if p else 0 for p in paths]
    lens = [n + 13 * (i + 1) for i, n in enumerate(nodes)]
    cache, table, *_ = fill(coda, lens, page, n_kv, True)
    want = {k: t.cpu().numpy().copy() for k, t in cache.items()}
    for b, path in enumerate(paths):
        src = [lens[b] - nodes[b] + i for i in path]
        dst = [lens[b] - nodes[b] + i for i in range(len(path))]
        for t in want.values():
            rows = [t[int(table[b, s // page]), :, :, s % page].copy() for s in src]
            for d, x in zip(dst, rows):
                t[int(table[b, d // page]), :, :, d % page] = x
    width = max(map(len, paths)) + 1
    ws = coda.workspace(256)
    new = coda.kv_accept_nvfp4(cache, table.to(DEV), i32(lens), offsets(nodes),
                               i32([p + [-1] * (width - len(p)) for p in paths]), i32([max(len(p) - 1, 0) for p in paths]), ws=ws)
    assert coda.get_status(ws) == 0
    assert new["seq_lens"].tolist() == [x - n + len(p) for x, n, p in zip(lens, nodes, paths)]
    for k in want:
        assert np.array_equal(cache[k].cpu().numpy(), want[k], equal_nan=k == "scale"), k


def test_bad_paths_move_nothing(coda):
    lens, nodes, page = [40, 30], [8, 6], 16
    cache, table, *_ = fill(coda, lens, page, 2, False)
    before = {k: t.clone() for k, t in cache.items()}
    ws = coda.workspace(256)

    def run(path, count, n=lens, tab=table):
        return coda.kv_accept_nvfp4(cache, tab.to(DEV), i32(n), offsets(nodes), i32([path, [0, -1, -1, -1]]), i32([count, 0]),
                                    ws=ws)["seq_lens"].tolist()
    same = lambda: all(torch.equal(cache[k].nan_to_num() if k == "scale" else cache[k],
                                   before[k].nan_to_num() if k == "scale" else before[k]) for k in cache)
    for path, count in (([0, 3, 2, -1], 2), ([1, 2, 3, -1], 2), ([0, 3, 3, -1], 2), ([0, 8, -1, -1], 1), ([0, 2, -1, -1], 2),
                        ([0, 1, 2, 3], 4), ([0, 1, 2, 3], 8), ([0, 1, 2, 3], -1)):
        assert run(path, count) == [32, 25] and coda.get_status(ws) == 11, (path, count)
        coda.reset_status(ws)
        assert same()
    for bad in (7, -1, 10 ** 6):
        assert run([0, 3, -1, -1], 1, n=[bad, 30]) == [0, 25] and coda.get_status(ws) == 9
        coda.reset_status(ws)
        assert same()
    tab = table.clone()
    tab[0, 2] = -1                                       # the tree's page
    assert run([0, 3, -1, -1], 1, tab=tab) == [34, 25] and coda.get_status(ws) == 10 and same()


# --------------------------------------------------------------------------- together

def test_a_step_in_a_graph(coda):
    """Append with rotation, attention, verification and the move as one captured
    graph: a replay on other inputs gives the eager calls' bits."""
    n_q, n_kv, page, V = 8, 2, 32, 500
    nodes, before = [6, 1, 9], [70, 0, 31]
    lens = [a + b for a, b in zip(nodes, before)]
    trees = [grow(n, n) for n in nodes]
    T, B = sum(nodes), len(nodes)
    cache, table, *_ = fill(coda, lens, page, n_kv, False)
    start = {k: t.clone() for k, t in cache.items()}
    local = [(b, before[b] + i) for b, n in enumerate(nodes) for i in range(n)]
    slots = i32([int(table[b, k // page]) * page + k % page for b, k in local])
    pos = i32([k for _, k in local])
    cs = coda.rope_table(1e4, 64, 200)
    par, cu, tab, n = i32([p for t in trees for p in t]), offsets(nodes), table.to(DEV), i32(lens)
    head = synth.randn_bf16((V, n_q * D), 0.05, 17).to(DEV)
    x = torch.zeros(T, (n_q + 2 * n_kv) * D, dtype=torch.bfloat16, device=DEV)
    tok, u, un = torch.zeros(T, dtype=torch.int32, device=DEV), torch.zeros(T, device=DEV), torch.zeros(B, device=DEV)
    ws = coda.workspace(max(coda.load().coda_attention_tree_nvfp4_workspace_size(T, B, n_q, n_kv, D),
                            coda.load().coda_verify_drafts_workspace_size(T, B, V)))

    def step():
        Q, K, Vv = x.split([n_q * D, n_kv * D, n_kv * D], dim=1)
        r = coda.kv_append_rope_nvfp4(K, Vv, slots, cache, pos, cs, Q=Q, n_q=n_q, ws=ws)
        a = coda.attention_tree_nvfp4(r["Q"], cache, tab, n, cu, n_q, parents=par, ws=ws)
        p = torch.softmax((a["O"] @ head.T).float(), dim=1)
        v = coda.verify_drafts(p, tok, cu, u, un, max(nodes), parents=par, ws=ws)
        return {**a, **v, **coda.kv_accept_nvfp4(cache, tab, n, cu, v["nodes"], v["count"], ws=ws)}

    def load(seed):
        g = torch.Generator().manual_seed(seed)
        x.copy_(synth.randn_bf16(tuple(x.shape), 1.0, seed))
        tok.copy_(torch.randint(0, V, (T,), generator=g))
        u.copy_(torch.rand(T, generator=g) * 1e-3)
        un.copy_(torch.rand(B, generator=g))
        for k in cache:
            cache[k].copy_(start[k])
    load(0)
    step()
    cap = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=cap):
        out = step()
    for seed in (1, 2):
        load(seed)
        g.replay()
        torch.cuda.synchronize()
        got = {k: t.clone() for k, t in {**out, **cache}.items()}
        load(seed)
        want = {**step(), **cache}
        torch.cuda.synchronize()
        for k in got:
            assert torch.equal(got[k].nan_to_num() if got[k].is_floating_point() else got[k],
                               want[k].nan_to_num() if got[k].is_floating_point() else want[k]), k
    assert coda.get_status(ws) == 0


def test_two_streams(coda):
    lens, nodes, n_q, n_kv = [300, 41, 2000], [7, 3, 20], 8, 2
    cache, table, *_ = fill(coda, lens, 64, n_kv, True)
    Q = synth.randn_bf16((30, n_q * D), 1.0, 5).to(DEV)
    P, q, trees, tokens, u, un = drafts(nodes, 3001, True, torch.float32, 4)
    par, cu, tab, n = i32([p for t in trees for p in t]), offsets(nodes), table.to(DEV), i32(lens)
    P, q, tokens, u, un = P.to(DEV), q.to(DEV), i32(tokens.tolist()), torch.from_numpy(u).to(DEV), torch.from_numpy(un).to(DEV)
    torch.cuda.synchronize()
    both = lambda s: (coda.attention_tree_nvfp4(Q, cache, tab, n, cu, n_q, parents=par, stream=s),
                      coda.verify_drafts(P, tokens, cu, u, un, 20, parents=par, draft_probs=q, stream=s))
    want = both(None)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [both(s) for _ in range(4) for s in side]
    torch.cuda.synchronize()
    for a, v in got:
        assert all(torch.equal(a[k], want[0][k]) for k in a) and all(torch.equal(v[k], want[1][k]) for k in v)


def test_binding_refuses_shapes(coda):
    cache = coda.kv_cache_nvfp4(2, 16, 2)
    q, tab, cu = torch.zeros(3, 4 * D, dtype=torch.bfloat16, device=DEV), i32([[0, 1]]), i32([0, 3])
    with pytest.raises(ValueError, match="block_table"):
        coda.attention_tree_nvfp4(q, cache, i32([[0, 1], [0, 1]]), i32([5]), cu, 4)
    with pytest.raises(ValueError, match="parents"):
        coda.attention_tree_nvfp4(q, cache, tab, i32([5]), cu, 4, parents=i32([-1, 0]))
    with pytest.raises(ValueError, match="seq_lens"):
        coda.attention_tree_nvfp4(q, cache, tab, i32([5, 5]), cu, 4)
    with pytest.raises(TypeError, match="cu_seqlens"):
        coda.attention_tree_nvfp4(q, cache, tab, i32([5]), cu.long(), 4)
    with pytest.raises(ValueError, match="too small"):
        coda.attention_tree_nvfp4(q, cache, tab, i32([5]), cu, 4, ws=torch.zeros(128, dtype=torch.uint8, device=DEV))
    P, u = torch.zeros(3, 10, device=DEV), torch.zeros(3, device=DEV)
    with pytest.raises(TypeError, match="probs"):
        coda.verify_drafts(P.half(), cu[:1], cu, u, u[:1], 2)
    with pytest.raises(TypeError, match="draft_probs"):
        coda.verify_drafts(P, i32([0, 0, 0]), cu, u, u[:1], 2, draft_probs=P.to(torch.bfloat16))
    with pytest.raises(ValueError, match="u_next"):
        coda.verify_drafts(P, i32([0, 0, 0]), cu, u, u, 2)
    with pytest.raises(coda.CodaError):
        coda.verify_drafts(P, i32([0, 0, 0]), cu, u, u[:1], 0)
    with pytest.raises(ValueError, match="nodes"):
        coda.kv_accept_nvfp4(cache, tab, i32([5]), cu, i32([0, 1]), i32([1]))
    lens = i32([5])
    with pytest.raises(coda.CodaError):                 # new lengths over the old ones
        coda.kv_accept_nvfp4(cache, tab, lens, cu, i32([[0, 1]]), i32([1]), out={"seq_lens": lens})
