"""Drafted trees and their verification where a kernel's steps meet: items of a
CTA that follow one another closely, values and scores of very different sizes,
rows that are no probabilities."""
import numpy as np
import pytest
import torch

import synth
from oracle import coda_oracle as O
from parity import to_np
from test_drafts_gpu import D, DEV, check_tree, drafts, grow, i32, offsets, oracle_verify, run_verify
from test_kvcache_gpu import fill, oracle_rows

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


def attend(coda, K, V, Q, lens, n, n_q, n_kv=1, page=64, seed=1):
    """Chains of n nodes behind rows K, V [sum(lens), n_kv * D], checked; K, V, Q as
    floats.  A row of zeros has no size."""
    K, V, Q = (x.to(torch.bfloat16) for x in (K, V, Q))
    need = [-(-x // page) for x in lens]
    cache = coda.kv_cache_nvfp4(sum(need), page, n_kv)
    order = torch.randperm(sum(need), generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    slots, at = [], 0
    for b, x in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        j = torch.arange(x)
        slots.append(table[b][j // page] * page + j.to(torch.int32) % page)
        at += need[b]
    ws = coda.workspace(coda.load().coda_attention_tree_nvfp4_workspace_size(n * len(lens), len(lens), n_q, n_kv, D))
    coda.kv_append_nvfp4(K.to(DEV), V.to(DEV), torch.cat(slots).to(DEV), cache, ws=ws)
    out = coda.attention_tree_nvfp4(Q.to(DEV), cache, table.to(DEV), i32(lens), offsets([n] * len(lens)), n_q, ws=ws)
    assert coda.get_status(ws) == 0
    (_, _, _, kv), (_, _, sc, vv) = oracle_rows(K, n_kv), oracle_rows(V, n_kv)
    sc = np.where(np.abs(vv).reshape(*sc.shape, D).max(axis=2) == 0, 2.0 ** -100, sc)
    cut = np.cumsum([0] + lens)
    part = lambda x: [x[a:b] for a, b in zip(cut, cut[1:])]
    check_tree(out, to_np(Q), lens, [n] * len(lens), [[i - 1 for i in range(n)]] * len(lens), part(kv), part(vv), part(sc), n_q,
               n_kv, D ** -0.5)


def sizes(batch, keys):
    """Sequences of about that length, one of them long enough to be cut."""
    return [keys + i % 7 for i in range(batch)] + ([40 * keys] if batch > 1 else [])


# sequences (a CTA has whole ones of many, and parts of one), exponents of the values
# before the last keys and in them, by how much their scores (base 2) lie above
JUMPS = [(-50, -50, 80), (0, -30, 125), (0, -30, 100), (-90, -90, 30), (-60, -60, 60), (-100, 15, 0), (-90, 20, -20), (30, -80, 95),
         (0, 0, 140), (0, 0, 300)]


@pytest.mark.parametrize("batch", [1, 330])
@pytest.mark.parametrize("before, behind, jump", JUMPS, ids=str)
def test_scores_that_jump_at_values_of_other_sizes(coda, batch, before, behind, jump):
    """The first weights against a reference are far too large, and what they add is
    taken back: the sums before them count as far as they did."""
    n_q, n = 4, 3
    lens = sizes(batch, 390)
    K, V = synth.randn_bf16((sum(lens), D), 0.5, 1).float(), synth.randn_bf16((sum(lens), D), 1.0, 2).float()
    Q = synth.randn_bf16((n * len(lens), n_q * D), 0.1, 3).float()
    Q.view(-1, n_q, D)[..., :64] = 1.0
    at = 0
    for x in lens:
        late = torch.arange(x) >= 0.7 * x
        late &= torch.arange(x) % 5 < 2
        V[at:at + x] *= torch.where(late, 2.0 ** behind, 2.0 ** before).unsqueeze(1)
        K[at:at + x, :64] = torch.where(late, jump * 0.6931 / (64 * D ** -0.5), 0.0).unsqueeze(1)
        at += x
    attend(coda, K, V, Q, lens, n, n_q)


def test_a_key_that_is_not_finite_stays_in_sums_that_pass_fp32(coda):
    n_q, n, page, keys, batch = 4, 3, 64, 390, 330
    lens = [keys] * batch
    cache, table, *_ = fill(coda, lens, page, 1, False)
    K, V = synth.randn_bf16((keys, D), 0.5, 1).float(), synth.randn_bf16((keys, D), 2.0 ** -60, 2)
    K[:, :64] = 0
    K[300:, :64] = 60 * 0.6931 / (64 * D ** -0.5)
    K = K.to(torch.bfloat16).to(DEV)
    j = torch.arange(keys)
    for b in range(batch):
        slots = table[b][j // page] * page + j.to(torch.int32) % page
        coda.kv_append_nvfp4(K, V.to(DEV), slots.to(DEV), cache)
        if b % 2:
            cache["scale"].view(-1, 2, page)[int(slots[5]) // page, b // 2 % 2, int(slots[5]) % page] = float("nan")
    Q = synth.randn_bf16((n * batch, n_q * D), 0.1, 3).float()
    Q.view(-1, n_q, D)[..., :64] = 1.0
    out = coda.attention_tree_nvfp4(Q.to(torch.bfloat16).to(DEV), cache, table.to(DEV), i32(lens), offsets([n] * batch), n_q)
    sick = (torch.arange(batch) % 2 == 1).repeat_interleave(n).to(DEV)
    assert torch.isnan(out["lse"][sick]).all() and torch.isnan(out["O"][sick].float()).all()
    assert torch.isfinite(out["lse"][~sick]).all() and torch.isfinite(out["O"][~sick].float()).all()


@pytest.mark.parametrize("first, lift", [(32, 1.0), (129, 1.0), (256, 1.0), (32, 20.0), (129, 30.0)])
@pytest.mark.parametrize("batch", [1, 330])
@pytest.mark.parametrize("sizes_of", [(-60,), (20, -60), (-60, 40), (0,)], ids=str)
def test_rows_of_zeros_have_no_say_in_the_units(coda, sizes_of, batch, first, lift):
    """Every sequence begins with value rows of zeros, has one in seven among the
    others and a few with the largest scores (by up to 85); sequences of small values
    follow those of large ones in a CTA."""
    n_q, n = 4, 3
    lens = sizes(batch, 390)
    K, V = synth.randn_bf16((sum(lens), D), 1.0, 1).float(), synth.randn_bf16((sum(lens), D), 1.0, 2).float()
    Q = synth.randn_bf16((n * len(lens), n_q * D), 0.1, 3).float()
    Q.view(-1, n_q, D)[..., :64] = 0.5
    at = 0
    for b, x in enumerate(lens):
        V[at:at + x] *= 2.0 ** sizes_of[b % len(sizes_of)]
        V[at:at + first] = 0
        V[at:at + x:7] = 0
        K[at:at + x:21, :64] += lift
        at += x
    attend(coda, K, V, Q, lens, n, n_q)


@pytest.mark.parametrize("std", [0.1, 3.0])
@pytest.mark.parametrize("batch", [1, 330])
def test_values_of_all_sizes_in_one_sequence(coda, batch, std):
    """Row by row from 2^-80 to 2^60, and zeros: the smallest count in the sum as far
    as their scores say."""
    n_q, n = 4, 3
    lens = sizes(batch, 390)
    r = np.random.default_rng(5)
    K, V = synth.randn_bf16((sum(lens), D), 1.0, 1).float(), synth.randn_bf16((sum(lens), D), 1.0, 2).float()
    Q = synth.randn_bf16((n * len(lens), n_q * D), std, 3).float()
    V *= torch.exp2(torch.from_numpy(r.integers(-80, 61, size=(sum(lens), 1))).float())
    V[::11] = 0
    attend(coda, K, V, Q, lens, n, n_q)


@pytest.mark.parametrize("batch", [1, 330])
@pytest.mark.parametrize("before, behind, jump", [(-100, 60, 0), (-100, 40, 5), (-90, 55, -10), (None, 60, 0), (-110, 100, 0),
                                                   (-40, 90, 3)], ids=str)
def test_large_values_behind_small_ones(coda, batch, before, behind, jump):
    """Scores of one size, values 2^100 times as large from some key on (None: zeros
    before them): a weight is infinite against the first reference though its share
    is no larger than the others'."""
    n_q, n = 4, 3
    lens = sizes(batch, 390)
    K, V = synth.randn_bf16((sum(lens), D), 0.5, 1).float(), synth.randn_bf16((sum(lens), D), 1.0, 2).float()
    Q = synth.randn_bf16((n * len(lens), n_q * D), 0.1, 3).float()
    Q.view(-1, n_q, D)[..., :64] = 1.0
    at = 0
    for x in lens:
        late = (torch.arange(x) >= 0.4 * x) & (torch.arange(x) % 3 < 2)
        V[at:at + x] *= torch.where(late, 2.0 ** behind, 0.0 if before is None else 2.0 ** before).unsqueeze(1)
        K[at:at + x, :64] = torch.where(late, jump * 0.6931 / (64 * D ** -0.5), 0.0).unsqueeze(1)
        at += x
    attend(coda, K, V, Q, lens, n, n_q)


@pytest.mark.parametrize("batch", [1, 330])
def test_weights_at_fp32_s_least(coda, batch):
    """Values of 2688 * 2^36 among rows of zeros, which count as rows of scale 2^-90:
    with scores that hardly differ every weight of theirs lies at 2^-126, just above
    or just below, and each is counted once."""
    n_q, n = 4, 3
    lens = sizes(batch, 390)
    K, V = synth.randn_bf16((sum(lens), D), 1.0, 1).float(), torch.zeros(sum(lens), D)
    V[::37] = 2688.0 * 2.0 ** 36 * torch.sign(synth.randn_bf16((len(V[::37]), D), 1.0, 2).float())
    attend(coda, K, V, synth.randn_bf16((n * len(lens), n_q * D), 2.0 ** -10, 3).float(), lens, n, n_q)


@pytest.mark.parametrize("group, n, batch, top", [(13, 30, 60, 170), (4, 2, 9, 1300), (8, 3, 200, 300), (2, 30, 60, 700)])
def test_values_about_fp32_s_range_apart(coda, group, n, batch, top):
    """Weights on either side of fp32's least, each counted once."""
    r = np.random.default_rng(group)
    lens = [int(x) for x in r.integers(n, top, size=batch)]
    T = sum(lens)
    K, V = synth.randn_bf16((T, D), 1.0, 1).float(), synth.randn_bf16((T, D), 1.0, 2).float()
    Q = synth.randn_bf16((n * batch, group * D), 1.0, 3).float()
    V *= torch.exp2(torch.from_numpy(r.integers(-80, 61, size=(T, 1))).float())
    V[torch.from_numpy(r.random(T) < 0.5)] = 0
    attend(coda, K, V, Q, lens, n, group, page=32)


# --------------------------------------------------------------------------- verification

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("drawn", [True, False], ids=["drawn", "chosen"])
def test_values_that_are_no_probabilities(coda, drawn, dtype):
    """Negative ones and NaN count as 0, those above 1 as 1, in the walk as in the
    sums; most of them at drafted tokens."""
    bad = torch.tensor([float("nan"), -0.25, -2.0, float("-inf"), 0.0, 1.5, float("inf")], dtype=dtype)
    clean = lambda x: x if x is None else x.float().nan_to_num(0.0, float("inf"), float("-inf")).clamp(0, 1)
    nodes, V = [9, 1, 14, 6] * 6, 23
    for seed in range(12):
        r = np.random.default_rng(seed)
        P, Q, trees, tokens, u, un = drafts(nodes, V, drawn, dtype, seed, peaked=1.0)
        at = 0
        for t in trees:
            for i, up in enumerate(t):
                for X in (P, Q):
                    if up >= 0 and X is not None and r.random() < 0.3:
                        X[at + up, tokens[at + i]] = bad[r.integers(5)]
                if r.random() < 0.1:
                    P[at + i, r.integers(V)] = bad[r.integers(7)]
                if Q is not None and r.random() < 0.1:
                    Q[at + i, r.integers(V)] = bad[r.integers(7)]
            at += len(t)
        got = run_verify(coda, P, Q, trees, tokens, u, un, 8)
        assert got == oracle_verify(clean(P), clean(Q), trees, tokens, u, un, 8)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("drawn", [True, False], ids=["drawn", "chosen"])
@pytest.mark.parametrize("copies", [1, 200])
def test_rows_that_sum_to_more_than_one(coda, copies, drawn, dtype):
    """Up to 16 they count as they are; from there on the sequence ends, with a status
    and without a next token, and the others are as without it."""
    r = np.random.default_rng(4)
    V = 5000
    for many, level in ((15, 1.0), (150, 0.1), (60, 0.25), (20, 0.75), (5000, 2.0 ** -9)):
        P = torch.zeros(4, V)
        for row in P:
            row[torch.from_numpy(r.permutation(V)[:many])] = level
        Q = torch.full((4, V), 1.0 / V) if drawn else None
        P, Q = P.repeat(copies, 1).to(dtype), Q.repeat(copies, 1).to(dtype) if drawn else None
        zero = [int(torch.nonzero(row == 0)[0]) if (row == 0).any() else 0 for row in P]
        tokens = np.array([0, zero[0], zero[0], zero[0]] * copies)            # refused, where there is anything to refuse
        trees = [[-1, 0, 0, 0]] * copies
        u, un = np.full(4 * copies, 0.9999, np.float32), r.random(copies).astype(np.float32)
        assert run_verify(coda, P, Q, trees, tokens, u, un, 3) == oracle_verify(P, Q, trees, tokens, u, un, 3), (many, level)
    for many, level in ((16, 1.0), (17, 1.0), (32, 1.0), (31, 1.0), (5000, 1.0), (33, 0.5), (4096, 2.0 ** -8)):
        P = torch.full((4, V), 0.0)
        P[:, :many] = level
        P[:, -1] = 2.0 ** -30                                                 # never drafted
        good = torch.softmax(torch.randn(4, V, generator=torch.Generator().manual_seed(1)) * 3, 1)
        P = torch.cat([good, P, good]).repeat(copies, 1).to(dtype)
        Q = torch.full((12 * copies, V), 1.0 / V).to(dtype) if drawn else None
        trees = [[-1, 0, 0, 0]] * 3 * copies
        tokens = np.array([0, V - 1, V - 2, V - 1] * 3 * copies)
        u, un = np.full(12 * copies, 0.9999, np.float32), r.random(3 * copies).astype(np.float32)
        ws = coda.workspace(256)
        count, path, out = run_verify(coda, P, Q, trees, tokens, u, un, 3, ws=ws)
        # (with drawn drafts the weights count, from which the refused child's q is gone)
        over = float((P[4].double() - (Q[4].double() if drawn else 0)).clamp(min=0).sum()) >= 16
        assert coda.get_status(ws) == (12 if over else 0)                     # CODA_ERR_PROBABILITY_RANGE
        want = oracle_verify(P, Q, trees, tokens, u, un, 3)
        for b in range(3 * copies):
            if over and b % 3 == 1:
                end = count[b]
                assert path[b] == want[1][b][:end + 1] + [-1] * (2 - end) and out[b] == want[2][b][:end] + [-1] * (3 - end)
            else:
                assert (count[b], path[b], out[b]) == tuple(x[b] for x in want), (many, level, b)


@pytest.mark.parametrize("drawn", [True, False], ids=["drawn", "chosen"])
def test_refusals_in_rows_that_sum_to_several(coda, drawn):
    for seed in range(10):
        P, Q, trees, tokens, u, un = drafts([9, 30, 5, 17] * 5, 97, drawn, torch.float32, seed, peaked=1.0)
        P = (P * (4.0 + seed)).clamp(max=1.0)
        u = (1 - 0.3 * u).astype(np.float32)
        assert run_verify(coda, P, Q, trees, tokens, u, un, 6) == oracle_verify(P, Q, trees, tokens, u, un, 6)


def test_the_next_token_at_an_exact_border(coda):
    """Weights of 2^-60 units about the border of u times a sum of more than 53 bits."""
    u = lambda n: n * 2.0 ** -60
    rows = [  # weights in units, u_next, the first x whose sum passes u_next times the sum
        ([2 ** 59, 2, 2 ** 59, 6], 0.5, 2),              # 2^59 + 4: not passed by 2^59 + 2
        ([2 ** 59, 4, 1, 2 ** 59, 3], 0.5, 2),           # 2^59 + 4: equal is not above
        ([2 ** 58, 1, 1, 2 ** 59, 2 ** 58, 6], 0.25, 3), # 2^58 + 2: equal again
        ([2 ** 58, 1, 2, 2 ** 59, 2 ** 58, 5], 0.25, 2),
        ([2 ** 59, 2 ** 58, 3, 1, 2 ** 58, 0], 0.75, 3), # 3 * 2^58 + 3: only its sum with 1 is above
        ([5, 1, 1, 1], 0.625, 1), ([5, 1, 1, 1], 0.5, 0), ([1, 2 ** 60], 2.0 ** -60, 1), ([1, 2 ** 60 - 2 ** 36], 2.0 ** -60, 0),
        ([1, 1], 2.0 ** -140, 0), ([0, 3], 0.0, 1)]
    for w, un, x in rows:
        total, c, first = sum(w), 0, None
        for i, n in enumerate(w):                        # in whole numbers
            c += n
            if first is None and c * 2 ** 140 > int(un * 2 ** 140) * total:
                first = i
        assert first == x
        P = torch.tensor([[u(n) for n in w]], dtype=torch.float64).float()
        assert [int(p * 2.0 ** 60) for p in P.double().tolist()[0]] == w
        got = run_verify(coda, P, None, [[-1]], np.array([0]), np.zeros(1, np.float32), np.array([un], np.float32), 1)
        assert got == ([0], [[0]], [[x]]), (w, un, got)
