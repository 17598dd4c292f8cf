"""CPU checks of the rotary and drafting operators: arguments refused on the
host before anything is enqueued, empty problems, and the oracle's own pins."""
import numpy as np
import pytest
import torch

import gemm_epilogue_transformer_bf16_gb300 as coda
from oracle import coda_oracle as O

FAKE = 1 << 20          # a 16-byte aligned non-null address (never dereferenced)
WS = 1 << 30


@pytest.fixture(scope="module")
def lib():
    from gemm_epilogue_transformer_bf16_gb300 import _build
    _build.build()
    return coda.load()


def table(lib, theta=1e4, rotary=64, max_pos=8, kind=2, factor=4.0, original=512.0, low=1.0, high=4.0, amplitude=1.0,
          cs=FAKE):
    return lib.coda_rope_table_scaled(theta, rotary, max_pos, kind, factor, original, low, high, amplitude, cs, None)


def rope(lib, X=FAKE, ldx=512, pos=FAKE, cs=FAKE, max_pos=8, rotary=64, pairing=0, Y=2 * FAKE, ldy=512, T=3, heads=4, d=128,
         ws=FAKE, ws_bytes=256, call="coda_rope"):
    return getattr(lib, call)(X, ldx, pos, cs, max_pos, rotary, pairing, Y, ldy, T, heads, d, ws, ws_bytes, None)


def rope_bwd(lib, **kw):
    return rope(lib, call="coda_rope_bwd", **kw)


def append(lib, Q=FAKE, ldq=512, K=FAKE, ldk=256, V=FAKE, ldv=256, slots=FAKE, pos=FAKE, cs=FAKE, max_pos=8, rotary=128,
           pairing=1, Qo=FAKE, Ko=None, T=5, codes=FAKE, sf=FAKE, scale=FAKE, pages=4, page=16, n_q=4, n_kv=2, d=128,
           ws=FAKE, ws_bytes=256):
    return lib.coda_kv_append_rope_nvfp4(Q, ldq, K, ldk, V, ldv, slots, pos, cs, max_pos, rotary, pairing, Qo, Ko, T, codes,
                                         sf, scale, pages, page, n_q, n_kv, d, ws, ws_bytes, None)


def tree(lib, Q=FAKE, ldq=512, codes=FAKE, sf=FAKE, scale=FAKE, pages=4, page=16, table=FAKE, max_pages=4, lens=FAKE,
         cu=FAKE, parents=None, T=9, batch=3, n_q=4, n_kv=2, d=128, sm=0.1, O=FAKE, lse=FAKE, ws=FAKE, ws_bytes=WS):
    return lib.coda_attention_tree_nvfp4(Q, ldq, codes, sf, scale, pages, page, table, max_pages, lens, cu, parents, T,
                                         batch, n_q, n_kv, d, sm, O, lse, ws, ws_bytes, None)


def verify(lib, P=FAKE, Q=None, dtype=1, V=100, tokens=FAKE, cu=FAKE, parents=None, u=FAKE, un=FAKE, T=9, batch=3, width=4,
           count=FAKE, nodes=FAKE, out=FAKE, ws=FAKE, ws_bytes=WS):
    return lib.coda_verify_drafts(P, Q, dtype, V, tokens, cu, parents, u, un, T, batch, width, count, nodes, out, ws,
                                  ws_bytes, None)


def accept(lib, codes=FAKE, sf=FAKE, scale=FAKE, pages=4, page=16, table=FAKE, max_pages=4, lens=FAKE, cu=FAKE, nodes=FAKE,
           width=4, count=FAKE, batch=3, n_kv=2, d=128, new=2 * FAKE, ws=FAKE, ws_bytes=256):
    return lib.coda_kv_accept_nvfp4(codes, sf, scale, pages, page, table, max_pages, lens, cu, nodes, width, count, batch,
                                    n_kv, d, new, ws, ws_bytes, None)


@pytest.mark.parametrize("call, change, code", [
    (table, dict(theta=0.0), 1), (table, dict(rotary=63), 1), (table, dict(max_pos=0), 1), (table, dict(kind=4), 1),
    (table, dict(factor=0.0), 1), (table, dict(high=1.0), 1), (table, dict(original=0.0), 1), (table, dict(cs=None), 1),
    (table, dict(amplitude=float("nan")), 1), (table, dict(kind=3, theta=1.0), 1), (table, dict(cs=FAKE + 4), 2),
    *[(c, d, e) for c in (rope, rope_bwd) for d, e in (
        (dict(X=None), 1), (dict(Y=None), 1), (dict(pos=None), 1), (dict(cs=None), 1), (dict(T=-1), 1), (dict(heads=0), 1),
        (dict(pairing=2), 1), (dict(ldx=504), 1), (dict(ldy=256), 1), (dict(max_pos=0), 1), (dict(rotary=0), 1),
        (dict(Y=FAKE, ldy=520), 1), (dict(rotary=24), 3), (dict(rotary=144), 3), (dict(d=64), 3), (dict(T=1 << 29), 3),
        (dict(X=FAKE + 2), 2), (dict(cs=FAKE + 8), 2), (dict(ldx=516), 2), (dict(ws=None), 4), (dict(ws_bytes=255), 4),
        (dict(T=0), 0))],
    (append, dict(K=None), 1), (append, dict(slots=None), 1), (append, dict(Q=None), 1), (append, dict(Qo=None), 1),
    (append, dict(pos=None), 1), (append, dict(T=-1), 1), (append, dict(n_q=-1), 1), (append, dict(ldq=384), 1),
    (append, dict(page=24), 3), (append, dict(rotary=100), 3), (append, dict(d=64), 3), (append, dict(T=1 << 29), 3),
    (append, dict(Ko=FAKE + 8), 2), (append, dict(ldv=260), 2), (append, dict(ws=None), 4), (append, dict(T=0), 0),
    (tree, dict(Q=None), 1), (tree, dict(table=None), 1), (tree, dict(lens=None), 1), (tree, dict(cu=None), 1),
    (tree, dict(O=None), 1), (tree, dict(lse=None), 1), (tree, dict(batch=-1), 1), (tree, dict(max_pages=-1), 1),
    (tree, dict(sm=0.0), 1), (tree, dict(sm=float("inf")), 1), (tree, dict(ldq=256), 1), (tree, dict(n_q=3), 3),
    (tree, dict(d=96), 3), (tree, dict(page=100), 3), (tree, dict(max_pages=1 << 28), 3), (tree, dict(Q=FAKE + 2), 2),
    (tree, dict(ldq=516), 2), (tree, dict(cu=FAKE + 1), 2), (tree, dict(parents=FAKE + 2), 2), (tree, dict(ws=None), 4),
    (tree, dict(ws_bytes=128), 4), (tree, dict(batch=0), 0), (tree, dict(T=0), 0),
    (verify, dict(P=None), 1), (verify, dict(tokens=None), 1), (verify, dict(cu=None), 1), (verify, dict(u=None), 1),
    (verify, dict(un=None), 1), (verify, dict(count=None), 1), (verify, dict(nodes=None), 1), (verify, dict(out=None), 1),
    (verify, dict(V=0), 1), (verify, dict(width=0), 1), (verify, dict(dtype=2), 1), (verify, dict(T=-1), 1),
    (verify, dict(V=1 << 30), 3), (verify, dict(P=FAKE + 4), 2), (verify, dict(Q=FAKE + 8), 2), (verify, dict(u=FAKE + 2), 2),
    (verify, dict(ws=None), 4), (verify, dict(batch=0), 0),
    (accept, dict(lens=None), 1), (accept, dict(cu=None), 1), (accept, dict(nodes=None), 1), (accept, dict(count=None), 1),
    (accept, dict(new=None), 1), (accept, dict(new=FAKE), 1), (accept, dict(table=None), 1), (accept, dict(width=0), 1),
    (accept, dict(batch=-1), 1), (accept, dict(page=8), 3), (accept, dict(max_pages=1 << 28), 3), (accept, dict(d=64), 3),
    (accept, dict(nodes=FAKE + 2), 2), (accept, dict(ws=None), 4), (accept, dict(batch=0), 0),
])
def test_refusals(lib, call, change, code):
    assert call(lib, **change) == code


def test_status_has_a_name():
    assert coda.status_string(11) == "CODA_ERR_TREE_RANGE"


def test_binding_refuses_host_tensors_and_scalings():
    x, i = torch.zeros(3, 256, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    cache = coda.kv_cache_nvfp4(2, 16, 2, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        coda.rope(x, i, torch.zeros(4, 64, 2), 2)
    with pytest.raises(ValueError, match="CUDA"):
        coda.kv_append_rope_nvfp4(x, x, i, cache, i, torch.zeros(4, 64, 2))
    with pytest.raises(ValueError, match="CUDA"):
        coda.attention_tree_nvfp4(x, cache, i.view(1, 3), i[:1], i[:2], 2)
    with pytest.raises(ValueError, match="CUDA"):
        coda.verify_drafts(torch.zeros(3, 10), i, i[:2], torch.zeros(3), torch.zeros(1), 2)
    with pytest.raises(ValueError, match="CUDA"):
        coda.kv_accept_nvfp4(cache, i.view(1, 3), i[:1], i[:2], i.view(1, 3), i[:1])
    out = torch.zeros(4, 32, 2)
    for bad in (dict(), dict(kind="other"), dict(kind="linear"), dict(kind="bands", factor=2.0),
                dict(kind="linear", factor=2.0, low=1.0)):
        with pytest.raises(ValueError, match="scaling"):
            coda.rope_table(1e4, 64, 4, out=out, scaling=bad)


# --------------------------------------------------------------------------- the oracle's own pins

def test_scaled_frequencies():
    f = O.rope_scaled_frequencies(1e4, 64)
    assert np.allclose(O.rope_scaled_frequencies(1e4, 64, "linear", factor=8.0), f / 8)
    turns = 512 * f / (2 * np.pi)
    b = O.rope_scaled_frequencies(1e4, 64, "bands", 8.0, 512.0, 1.0, 4.0)
    assert np.array_equal(b[turns > 4], f[turns > 4]) and np.allclose(b[turns < 1], f[turns < 1] / 8)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and np.all((b[mid] < f[mid]) & (b[mid] > f[mid] / 8))
    r = O.rope_scaled_frequencies(1e4, 64, "ramp", 8.0, 4096.0)
    assert r[0] == f[0] and np.isclose(r[-1], f[-1] / 8) and np.all(np.diff(r) < 0)


def test_rope_part_is_the_rotation_of_its_part():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(4, 3, 32))
    pos = np.array([0, 3, 100, 7])
    a = pos[:, None] * O.rope_scaled_frequencies(1e4, 16)
    for pairing in ("interleaved", "half"):
        y = O.rope_part(x, np.cos(a), np.sin(a), pairing)
        assert np.allclose(y[..., :16], O.rope(x[..., :16], pos, 1e4, pairing)) and np.array_equal(y[..., 16:], x[..., 16:])


def test_tree_attention_of_a_chain_is_causal():
    rng = np.random.default_rng(2)
    n_q, n_kv, d, n, keys = 4, 2, 8, 5, 12
    q, k, v = rng.normal(size=(n, n_q * d)), rng.normal(size=(keys, n_kv * d)), rng.normal(size=(keys, n_kv * d))
    got = O.tree_attention_fwd(q, k, v, O.tree_sees([-1, 0, 1, 2, 3]), n_q, n_kv, 0.3)
    want = O.attention_fwd(q, k, v, [0, n], [0, keys], n_q, n_kv, 0.3)
    assert np.allclose(got["O"], want["O"]) and np.allclose(got["lse"], want["lse"].T)
    # a branch sees what a chain of its ancestors sees
    t = O.tree_attention_fwd(q, k, v, O.tree_sees([-1, 0, 0, 2, 0]), n_q, n_kv, 0.3)
    pick = [0, 2, 3]
    rows = list(range(keys - n)) + [keys - n + i for i in pick]
    alone = O.attention_fwd(q[pick], k[rows], v[rows], [0, 3], [0, len(rows)], n_q, n_kv, 0.3)
    assert np.allclose(t["O"][3], alone["O"][2])


@pytest.mark.parametrize("drawn", [True, False])
def test_verified_tokens_are_distributed_as_the_target_s(drawn):
    """Two children of the root, all random numbers on a fine grid: the first
    token has the target's probabilities."""
    rng = np.random.default_rng(3)
    V, G = 4, 24
    p, q = rng.dirichlet(np.ones(V)), rng.dirichlet(np.ones(V))
    P = np.stack([p, p, p])
    got = np.zeros(V)
    grid = (np.arange(G) + 0.5) / G
    drafts = [((a, b), q[a] * q[b]) for a in range(V) for b in range(V)] if drawn else [((2, 0), 1.0)]
    for (a, b), weight in drafts:
        for u1 in grid:
            for u2 in grid:
                for un in grid:
                    _, text = O.verify_drafts(P, [0, a, b], [-1, 0, 0], [0.0, u1, u2], un, np.stack([q] * 3) if drawn else None)
                    got[text[0]] += weight / G ** 3
    assert np.all(np.abs(got - p) < 2.0 / G)


def test_verification_follows_the_tree():
    P = np.zeros((4, 3))
    P[0, 1] = P[2, 2] = P[1, 0] = P[3, 1] = 1.0
    assert O.verify_drafts(P, [0, 0, 1, 2], [-1, 0, 0, 2], [0.5] * 4, 0.3) == ([0, 2, 3], [1, 2, 1])
    assert O.verify_drafts(P, [0, 0, 1, 2], [-1, 0, 0, 2], [0.5] * 4, 0.3, width=2) == ([0, 2], [1, 2])
    assert O.verify_drafts(P, [0, 0, 1, 0], [-1, 0, 0, 2], [0.5] * 4, 0.3) == ([0, 2], [1, 2])
