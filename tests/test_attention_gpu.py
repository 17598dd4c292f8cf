"""Causal attention over packed sequences against the fp64 oracle.

Tolerances, from the kernel's roundings (half a step of bf16 is 2^-8
relative):

  O   each weight is rounded to bf16 before the second product, O once at the
      end: |err| <= 2^-8 sum_j p_ij |v_j| + 2^-8 |o|.  The scores are fp32 sums
      of 128 products, off by at most 128 * 2^-24 * scale * sum_d |q_d k_d| =:
      e (each partial sum rounds by half a step, 2^-24 relative); a score off
      by e moves its weight by a factor within exp(+-e), and the row's sum by
      as much, so the weights by exp(+-2e).  The SFU's 2^x is good to 2^-22
      and the sums over n keys to n 2^-24, in numerator and denominator.
  lse off by e, by the sum's n 2^-24, and by 2^-22 (|lse| + 16) for the
      maximum's product with the scale, the logarithm and their sum.
"""
import numpy as np
import pytest
import torch

import synth
from oracle import coda_oracle as O
from parity import to_np

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


def offsets(lens, first=0):
    return np.concatenate([[first], first + np.cumsum(lens)]).astype(np.int32)


def make(lq, lk, n_q, n_kv, front=0, pad=0, seed=0, std=1.0):
    """Packed inputs with `front` rows before the first sequence and `pad`
    behind the last."""
    cq = offsets(lq, front)
    ck = cq if lk is None else offsets(lk, front)
    Tq, Tk = int(cq[-1]) + pad, int(ck[-1]) + pad
    t = {"Q": synth.randn_bf16((Tq, n_q * D), std, seed), "K": synth.randn_bf16((Tk, n_kv * D), 1.0, seed + 1),
         "V": synth.randn_bf16((Tk, n_kv * D), 1.0, seed + 2)}
    return t, cq, ck, Tq, Tk


def score_error(t, cq, ck, n_q, n_kv, scale):
    """e of the module docstring, per query and head (largest over all keys)."""
    q, k = np.abs(to_np(t["Q"])), np.abs(to_np(t["K"]))
    e = np.zeros((n_q, q.shape[0]))
    for b in range(len(cq) - 1):
        for h in range(n_q):
            kv = h // (n_q // n_kv)
            prod = q[cq[b]:cq[b + 1], h * D:(h + 1) * D] @ k[ck[b]:ck[b + 1], kv * D:(kv + 1) * D].T
            if prod.size:
                e[h, cq[b]:cq[b + 1]] = prod.max(axis=1) * scale * D * 2.0 ** -24
    return e


def check_forward(out, ref, t, cq, ck, n_q, n_kv, scale):
    Tq = out["O"].shape[0]
    inside = np.zeros(Tq, bool)
    inside[cq[0]:cq[-1]] = True
    e = score_error(t, cq, ck, n_q, n_kv, scale)
    n = max(int((ck[1:] - ck[:-1]).max()), 1)
    rel = 2 * e + 2 * (n * 2.0 ** -24 + 2.0 ** -22)
    rel_o = np.repeat(rel.T, D, axis=1)
    got, want = to_np(out["O"]), ref["O"]
    bound = (2.0 ** -8 + 2 * rel_o) * ref["A"] + 2.0 ** -8 * np.abs(want)
    bad = (np.abs(got - want) > bound) & inside[:, None]
    assert not bad.any(), f"O: {bad.sum()} elements off, worst {np.abs(got - want)[inside].max()}"
    gl, wl = to_np(out["lse"])[:, inside], ref["lse"][:, inside]
    empty = np.isneginf(wl)
    assert np.array_equal(np.isneginf(gl), empty)
    lb = e[:, inside] + n * 2.0 ** -24 + 2.0 ** -22 * (np.abs(np.where(empty, 0, wl)) + 16)
    assert np.all(np.abs(np.where(empty, 0, gl) - np.where(empty, 0, wl)) <= lb), "lse"
    return inside


CASES = {
    # lq, lk (None: the same), n_q, n_kv, rows in front, rows behind
    "one_token": ([1], None, 2, 1, 0, 0),
    "one_block": ([128], None, 2, 1, 0, 0),
    "past_block": ([129], None, 1, 1, 0, 0),
    "two_tiles": ([255], None, 3, 1, 0, 0),
    "ragged": ([300, 1, 0, 129, 64], None, 4, 2, 3, 9),
    "odd_group": ([200, 57], None, 5, 1, 0, 1),
    "group_of_six": ([130, 3], None, 6, 1, 0, 0),
    "many_short": ([3, 7, 1, 16, 0, 9, 12, 2] * 5, None, 16, 2, 0, 7),
    "short_odd_group": ([2, 5, 1, 9], None, 7, 7, 0, 0),
    "prefix": ([70, 1, 200], [470, 333, 200], 8, 2, 0, 4),
    "prefix_short": ([1, 1, 2, 3], [129, 1, 64, 700], 16, 2, 0, 0),
    "rows_without_keys": ([300, 5, 9, 4], [100, 0, 9, 3], 4, 4, 0, 3),
    "long": ([2500], None, 4, 2, 0, 0),
}


@pytest.mark.parametrize("name", CASES)
def test_forward(coda, name):
    lq, lk, n_q, n_kv, front, pad = CASES[name]
    t, cq, ck, Tq, Tk = make(lq, lk, n_q, n_kv, front, pad, seed=len(name))
    d = {k: v.to(DEV) for k, v in t.items()}
    out = {"O": torch.full((Tq, n_q * D), 7.0, dtype=torch.bfloat16, device=DEV),
           "lse": torch.full((n_q, Tq), 7.0, device=DEV)}
    ws = coda.workspace(coda.load().coda_attention_workspace_size(Tq, Tk, len(lq), n_q, n_kv, D))
    coda.attention(d["Q"], d["K"], d["V"], torch.from_numpy(cq).to(DEV), n_q, n_kv,
                   cu_seqlens_k=None if lk is None else torch.from_numpy(ck).to(DEV), out=out, ws=ws)
    assert coda.get_status(ws) == 0
    scale = D ** -0.5
    ref = O.attention_fwd(to_np(t["Q"]), to_np(t["K"]), to_np(t["V"]), cq, ck, n_q, n_kv, scale)
    inside = check_forward(out, ref, t, cq, ck, n_q, n_kv, scale)
    # rows outside every sequence stay as they were
    assert torch.all(out["O"].cpu()[~torch.from_numpy(inside)] == 7) and torch.all(
        out["lse"].cpu()[:, ~torch.from_numpy(inside)] == 7)


def test_forward_columns_of_one_projection(coda):
    """Q, K, V as columns of one [T, (n_q + 2 n_kv) * 128] tensor give the same
    bits as separate tensors."""
    n_q, n_kv, cq = 4, 2, offsets([150, 20])
    T = int(cq[-1])
    qkv = synth.randn_bf16((T, (n_q + 2 * n_kv) * D), 1.0, 5).to(DEV)
    Q, K, V = qkv.split([n_q * D, n_kv * D, n_kv * D], dim=1)
    cu = torch.from_numpy(cq).to(DEV)
    a = coda.attention(Q, K, V, cu, n_q, n_kv)
    b = coda.attention(Q.contiguous(), K.contiguous(), V.contiguous(), cu, n_q, n_kv)
    assert torch.equal(a["O"], b["O"]) and torch.equal(a["lse"], b["lse"])


@pytest.mark.parametrize("std", [0.0, 8.0, 60.0])
def test_forward_flat_and_peaked_scores(coda, std):
    """All scores equal, scores that rise late in a row (the accumulator is
    rescaled), and rows that see one key almost alone."""
    n_q, n_kv, cq = 2, 1, offsets([700])
    t, _, _, Tq, _ = make([700], None, n_q, n_kv, seed=11, std=std)
    d = {k: v.to(DEV) for k, v in t.items()}
    out = coda.attention(d["Q"], d["K"], d["V"], torch.from_numpy(cq).to(DEV), n_q, n_kv)
    ref = O.attention_fwd(to_np(t["Q"]), to_np(t["K"]), to_np(t["V"]), cq, cq, n_q, n_kv, D ** -0.5)
    check_forward(out, ref, t, cq, cq, n_q, n_kv, D ** -0.5)


@pytest.mark.parametrize("lens", [[100, 60], [130, 140], [5, 9, 3]])
def test_forward_non_finite_rows_stay_in_their_sequence(coda, lens):
    """NaN and infinities in one sequence, and in rows behind the last one,
    leave the other sequences' bits alone."""
    n_q, n_kv, pad = 4, 2, 30
    t, cq, _, Tq, _ = make(lens, None, n_q, n_kv, 0, pad, seed=3)
    cu = torch.from_numpy(cq).to(DEV)
    d = {k: v.to(DEV) for k, v in t.items()}
    clean = coda.attention(d["Q"], d["K"], d["V"], cu, n_q, n_kv)
    for k, bad in (("Q", float("nan")), ("K", float("inf")), ("V", float("nan")), ("V", float("-inf"))):
        e = {n: v.clone() for n, v in d.items()}
        e[k][int(cq[1]):int(cq[2])] = bad
        e[k][int(cq[-1]):] = bad
        got = coda.attention(e["Q"], e["K"], e["V"], cu, n_q, n_kv)
        for lo, hi in [(int(cq[0]), int(cq[1]))] + [(int(a), int(b)) for a, b in zip(cq[2:-1], cq[3:])]:
            assert torch.equal(got["O"][lo:hi], clean["O"][lo:hi]), (k, bad)
            assert torch.equal(got["lse"][:, lo:hi], clean["lse"][:, lo:hi]), (k, bad)


def test_forward_bad_offsets_set_status(coda):
    n_q, n_kv = 2, 1
    t, _, _, Tq, Tk = make([64, 64], None, n_q, n_kv)
    d = {k: v.to(DEV) for k, v in t.items()}
    ws = coda.workspace(coda.load().coda_attention_workspace_size(Tq, Tk, 2, n_q, n_kv, D))
    for bad in ([0, 65, 64], [0, 64, 129], [-1, 64, 128]):
        out = {"O": torch.full((Tq, n_q * D), 7.0, dtype=torch.bfloat16, device=DEV),
               "lse": torch.full((n_q, Tq), 7.0, device=DEV)}
        coda.attention(d["Q"], d["K"], d["V"], torch.tensor(bad, dtype=torch.int32, device=DEV), n_q, n_kv, out=out,
                       ws=ws)
        assert coda.get_status(ws) == 9            # CODA_ERR_SEQLEN_RANGE
        assert torch.all(out["O"] == 7)            # nothing was computed
        coda.reset_status(ws)
    coda.attention(d["Q"], d["K"], d["V"], torch.tensor([0, 64, 128], dtype=torch.int32, device=DEV), n_q, n_kv, ws=ws)
    assert coda.get_status(ws) == 0
