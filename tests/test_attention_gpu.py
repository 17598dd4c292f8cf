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
    # more sequences, and more runs of rows, than the list builder's block has threads
    "many_sequences": ([(7 * i) % 5 for i in range(1500)], None, 2, 1, 1, 2),
    "many_prefixes": ([(3 * i) % 4 for i in range(1100)], [(5 * i) % 7 for i in range(1100)], 1, 1, 0, 0),
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


# few rows over many keys: the keys are cut into parts that a second kernel joins
SPLIT_CASES = {
    # lq, lk, n_q, n_kv, rows in front, rows behind
    "one_row": ([1], [9000], 8, 1, 0, 0),
    "rows_of_all_heads": ([16, 3], [5001, 130], 16, 2, 2, 5),
    "two_runs": ([130], [4097], 4, 2, 0, 0),
    "no_pairs": ([300, 1], [3000, 2561], 3, 3, 0, 1),
    "odd_group": ([40, 200, 0, 7], [6000, 100, 900, 1700], 7, 1, 1, 0),
    "one_sequence": ([2600], None, 2, 1, 0, 3),
    "rows_without_keys": ([600, 5], [300, 4000], 2, 2, 0, 0),
}


@pytest.mark.parametrize("name", SPLIT_CASES)
def test_forward_over_parts_of_the_keys(coda, name):
    lq, lk, n_q, n_kv, front, pad = SPLIT_CASES[name]
    t, cq, ck, Tq, Tk = make(lq, lk, n_q, n_kv, front, pad, seed=len(name))
    d = {k: v.to(DEV) for k, v in t.items()}
    kw = {} if lk is None else {"cu_seqlens_k": torch.from_numpy(ck).to(DEV)}
    ws = coda.workspace(coda.load().coda_attention_workspace_size(Tq, Tk, len(lq), n_q, n_kv, D))
    ws[256:].fill_(0xFF)                                  # what an earlier call may have left: NaN
    got = []
    for _ in range(2):
        out = {"O": torch.full((Tq, n_q * D), 7.0, dtype=torch.bfloat16, device=DEV),
               "lse": torch.full((n_q, Tq), 7.0, device=DEV)}
        got.append(coda.attention(d["Q"], d["K"], d["V"], torch.from_numpy(cq).to(DEV), n_q, n_kv, out=out, ws=ws, **kw))
    assert coda.get_status(ws) == 0
    assert all(torch.equal(got[0][k], got[1][k]) for k in out)
    scale = D ** -0.5
    ref = O.attention_fwd(to_np(t["Q"]), to_np(t["K"]), to_np(t["V"]), cq, ck, n_q, n_kv, scale)
    inside = check_forward(out, ref, t, cq, ck, n_q, n_kv, scale)
    assert torch.all(out["O"].cpu()[~torch.from_numpy(inside)] == 7) and torch.all(
        out["lse"].cpu()[:, ~torch.from_numpy(inside)] == 7)


def test_non_finite_rows_and_parts_of_the_keys(coda):
    """As in the calls that cut nothing: another sequence's numbers, and those
    behind the last, change no bit; a NaN in one part reaches the joined rows."""
    n_q, n_kv, pad = 4, 2, 30
    t, cq, ck, Tq, Tk = make([9, 7], [3001, 2500], n_q, n_kv, 0, pad, seed=3)
    cu, cuk = torch.from_numpy(cq).to(DEV), torch.from_numpy(ck).to(DEV)
    d = {k: v.to(DEV) for k, v in t.items()}
    clean = coda.attention(d["Q"], d["K"], d["V"], cu, n_q, n_kv, cu_seqlens_k=cuk)
    for k, c, bad in (("Q", cq, float("nan")), ("K", ck, float("inf")), ("V", ck, float("nan"))):
        e = {n: v.clone() for n, v in d.items()}
        e[k][int(c[1]):] = bad
        got = coda.attention(e["Q"], e["K"], e["V"], cu, n_q, n_kv, cu_seqlens_k=cuk)
        assert torch.equal(got["O"][:9], clean["O"][:9]) and torch.equal(got["lse"][:, :9], clean["lse"][:, :9]), k
    e = d["V"].clone()
    e[1500] = float("nan")
    got = coda.attention(d["Q"], d["K"], e, cu, n_q, n_kv, cu_seqlens_k=cuk)
    assert bool(torch.isnan(got["O"][:9].float()).all()) and torch.equal(got["O"][9:16], clean["O"][9:16])


def test_parts_of_the_keys_in_a_graph_with_other_lengths(coda):
    """A captured call cuts by the lengths of its replay, not by the capture's."""
    n_q, n_kv = 4, 1
    t, _, _, Tq, Tk = make([8, 8], [6000, 6000], n_q, n_kv, seed=5)
    d = {k: v.to(DEV) for k, v in t.items()}
    cu, ck = torch.tensor([0, 8, 16], dtype=torch.int32, device=DEV), torch.tensor([0, 40, 80], dtype=torch.int32, device=DEV)
    ws = coda.workspace(coda.load().coda_attention_workspace_size(Tq, Tk, 2, n_q, n_kv, D))

    def run(out=None):
        return coda.attention(d["Q"], d["K"], d["V"], cu, n_q, n_kv, cu_seqlens_k=ck, out=out, ws=ws)
    out = run()
    cap = torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=cap):
        run(out)
    for ends in ([0, 6000, 12000], [0, 9, 11009], [0, 0, 50], [0, 12000, 12000]):
        ck.copy_(torch.tensor(ends, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        want = run()
        torch.cuda.synchronize()
        assert torch.equal(out["O"], want["O"]) and torch.equal(out["lse"], want["lse"])
        ref = O.attention_fwd(to_np(t["Q"]), to_np(t["K"]), to_np(t["V"]), [0, 8, 16], ends, n_q, n_kv, D ** -0.5)
        check_forward(out, ref, t, np.array([0, 8, 16]), np.array(ends), n_q, n_kv, D ** -0.5)
    assert coda.get_status(ws) == 0


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


# --------------------------------------------------------------------------- backward
#
# Gradients, from the kernel's roundings.  p is recomputed as
# exp2(s c - lse2) from fp32 scores and the forward's lse: relative error
# u = exp(2 e') - 1, e' = e + |lse| 2^-22 + n 2^-24 + 2^-20.  For dV it is
# rounded to bf16 (2^-8).  dO.v is an fp32 sum of 128 products (far below the
# next term); D uses the forward's bf16 O, off by 2^-8 (|O| + sum p |v|) per
# element and so by 2^-8 t_i.  ds is rounded to bf16 (2^-8), the sums over
# n rows add n 2^-24, the outputs are rounded to bf16 once (2^-8).

def check_backward(got, r, t, cq, ck, n_q, n_kv, scale):
    e = score_error(t, cq, ck, n_q, n_kv, scale).max()
    lse = O.attention_fwd(to_np(t["Q"]), to_np(t["K"]), to_np(t["V"]), cq, ck, n_q, n_kv, scale)["lse"]
    top = np.abs(np.where(np.isfinite(lse), lse, 0)).max()
    n = max(int((ck[1:] - ck[:-1]).max()), int((cq[1:] - cq[:-1]).max()), 1) * (n_q // n_kv)
    u = np.expm1(2 * (e + top * 2.0 ** -22 + n * 2.0 ** -24 + 2.0 ** -20))
    h = 2.0 ** -8
    more = 1 + 4 * h                                       # products of the relative errors above
    bounds = {"dQ": more * ((h + n * 2.0 ** -24) * r["EQ"] + u * r["UQ"] + h * r["TQ"]) + h * np.abs(r["dQ"]),
              "dK": more * ((h + n * 2.0 ** -24) * r["EK"] + u * r["UK"] + h * r["TK"]) + h * np.abs(r["dK"]),
              "dV": more * (h + u + n * 2.0 ** -24) * r["EV"] + h * np.abs(r["dV"])}
    for name, b in bounds.items():
        cu = cq if name == "dQ" else ck
        rows = slice(int(cu[0]), int(cu[-1]))
        err = np.abs(to_np(got[name]) - r[name])[rows]
        assert np.all(err <= b[rows]), (name, float((err - b[rows]).max()), float(err.max()))
        ref = np.linalg.norm(r[name][rows])
        if ref > 0:
            assert np.linalg.norm(err) <= 1e-2 * ref, (name, float(np.linalg.norm(err) / ref))


def run_backward(coda, t, cq, ck, n_q, n_kv, same, fill=7.0):
    d = {k: v.to(DEV) for k, v in t.items()}
    cu = torch.from_numpy(cq).to(DEV)
    kw = {} if same else {"cu_seqlens_k": torch.from_numpy(ck).to(DEV)}
    f = coda.attention(d["Q"], d["K"], d["V"], cu, n_q, n_kv, **kw)
    out = {"dQ": torch.full_like(d["Q"], fill), "dK": torch.full_like(d["K"], fill), "dV": torch.full_like(d["V"], fill)}
    ws = coda.workspace(coda.load().coda_attention_bwd_workspace_size(d["Q"].shape[0], d["K"].shape[0], len(cq) - 1, n_q,
                                                                      n_kv, D))
    coda.attention_bwd(d["dO"], d["Q"], d["K"], d["V"], f["O"], f["lse"], cu, n_q, n_kv, out=out, ws=ws, **kw)
    assert coda.get_status(ws) == 0
    return out


BWD_CASES = {k: CASES[k] for k in CASES if k != "long"}
BWD_CASES["long"] = ([1100], None, 4, 2, 0, 0)
BWD_CASES["some_groups_cut"] = ([1500, 40, 200], None, 12, 1, 0, 3)
BWD_CASES["few_queries_cut"] = ([300, 1, 20], [290, 900, 20], 16, 2, 0, 0)
BWD_CASES["queries_missing"] = ([0, 40], [200, 60], 4, 2, 0, 5)


@pytest.mark.parametrize("name", BWD_CASES)
def test_backward(coda, name):
    lq, lk, n_q, n_kv, front, pad = BWD_CASES[name]
    t, cq, ck, Tq, Tk = make(lq, lk, n_q, n_kv, front, pad, seed=len(name))
    t["dO"] = synth.randn_bf16((Tq, n_q * D), 1.0, 77)
    out = run_backward(coda, t, cq, ck, n_q, n_kv, lk is None)
    ref = O.attention_bwd(to_np(t["dO"]), to_np(t["Q"]), to_np(t["K"]), to_np(t["V"]), cq, ck, n_q, n_kv, D ** -0.5)
    check_backward(out, ref, t, cq, ck, n_q, n_kv, D ** -0.5)
    for k, cu in (("dQ", cq), ("dK", ck), ("dV", ck)):     # rows outside every sequence stay as they were
        outside = np.ones(out[k].shape[0], bool)
        outside[cu[0]:cu[-1]] = False
        assert torch.all(out[k].cpu()[torch.from_numpy(outside)] == 7), k


@pytest.mark.parametrize("std", [0.0, 8.0])
def test_backward_flat_and_peaked_scores(coda, std):
    n_q, n_kv = 2, 1
    t, cq, _, Tq, _ = make([400, 30], None, n_q, n_kv, seed=11, std=std)
    t["dO"] = synth.randn_bf16((Tq, n_q * D), 1.0, 78)
    out = run_backward(coda, t, cq, cq, n_q, n_kv, True)
    ref = O.attention_bwd(to_np(t["dO"]), to_np(t["Q"]), to_np(t["K"]), to_np(t["V"]), cq, cq, n_q, n_kv, D ** -0.5)
    if std == 0.0:
        # all weights equal: dK = 0 exactly in the formula when Q = 0; the kernel's sums of zeros are zeros
        assert torch.all(out["dK"] == 0)
        ref["dK"][:] = 0
    check_backward(out, ref, t, cq, cq, n_q, n_kv, D ** -0.5)


def test_backward_against_differences(coda):
    """Directional differences of sum(O dO) in fp64 against the kernel's
    gradients.  The difference quotient's own error is O(step^2), 1e-8 here;
    the gradients are bf16, so their inner product with a unit direction is
    off by at most the Frobenius rule's 1e-2 of |gradient|."""
    n_q, n_kv = 2, 1
    t, cq, _, Tq, _ = make([150, 20], None, n_q, n_kv, seed=4)
    t["dO"] = synth.randn_bf16((Tq, n_q * D), 1.0, 79)
    out = run_backward(coda, t, cq, cq, n_q, n_kv, True)
    x = {k: to_np(v) for k, v in t.items()}
    rng = np.random.default_rng(1)
    for k in ("Q", "K", "V"):
        dirn = rng.normal(size=x[k].shape)
        dirn /= np.linalg.norm(dirn)
        f = []
        for sgn in (1, -1):
            y = dict(x, **{k: x[k] + sgn * 1e-4 * dirn})
            f.append(np.sum(O.attention_fwd(y["Q"], y["K"], y["V"], cq, cq, n_q, n_kv, D ** -0.5)["O"] * x["dO"]))
        g = to_np(out["d" + k])
        assert abs((f[0] - f[1]) / 2e-4 - np.sum(g * dirn)) <= 1e-2 * np.linalg.norm(g), k


@pytest.mark.parametrize("lens", [[100, 60], [130, 140], [5, 9, 3]])
def test_backward_non_finite_rows_stay_in_their_sequence(coda, lens):
    n_q, n_kv, pad = 4, 2, 30
    t, cq, _, Tq, _ = make(lens, None, n_q, n_kv, 0, pad, seed=3)
    t["dO"] = synth.randn_bf16((Tq, n_q * D), 1.0, 80)
    clean = run_backward(coda, t, cq, cq, n_q, n_kv, True)
    for k in ("Q", "K", "V", "dO"):
        for bad in (float("nan"), float("inf")):
            e = {n: v.clone() for n, v in t.items()}
            e[k][int(cq[1]):int(cq[2])] = bad
            e[k][int(cq[-1]):] = bad
            got = run_backward(coda, e, cq, cq, n_q, n_kv, True)
            for lo, hi in [(int(cq[0]), int(cq[1]))] + [(int(a), int(b)) for a, b in zip(cq[2:-1], cq[3:])]:
                for g in ("dQ", "dK", "dV"):
                    assert torch.equal(got[g][lo:hi], clean[g][lo:hi]), (k, bad, g)


def test_twice_gives_the_same_bits_and_so_does_a_graph(coda):
    n_q, n_kv = 6, 2
    t, cq, _, Tq, _ = make([500, 3, 260, 129], None, n_q, n_kv, seed=6)
    t["dO"] = synth.randn_bf16((Tq, n_q * D), 1.0, 81)
    d = {k: v.to(DEV) for k, v in t.items()}
    cu = torch.from_numpy(cq).to(DEV)
    lib = coda.load()
    ws = coda.workspace(max(lib.coda_attention_workspace_size(Tq, Tq, 4, n_q, n_kv, D),
                            lib.coda_attention_bwd_workspace_size(Tq, Tq, 4, n_q, n_kv, D)))

    def step(f, b):
        coda.attention(d["Q"], d["K"], d["V"], cu, n_q, n_kv, out=f, ws=ws)
        coda.attention_bwd(d["dO"], d["Q"], d["K"], d["V"], f["O"], f["lse"], cu, n_q, n_kv, out=b, ws=ws)

    def buffers():
        return ({"O": torch.zeros_like(d["Q"]), "lse": torch.zeros(n_q, Tq, device=DEV)},
                {"dQ": torch.zeros_like(d["Q"]), "dK": torch.zeros_like(d["K"]), "dV": torch.zeros_like(d["V"])})
    one, two, three = buffers(), buffers(), buffers()
    step(*one)
    step(*two)
    cap = torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cap):
        step(*three)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=cap):
        step(*three)
    for part in three:
        for v in part.values():
            v.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert coda.get_status(ws) == 0
    for a, b, c in zip(one, two, three):
        for k in a:
            assert torch.equal(a[k], b[k]) and torch.equal(a[k], c[k]), k


def test_on_another_stream(coda):
    """A call that names a stream allocates and runs there."""
    n_q, n_kv = 4, 2
    t, cq, _, Tq, _ = make([300, 41], None, n_q, n_kv, seed=8)
    d = {k: v.to(DEV) for k, v in t.items()}
    cu = torch.from_numpy(cq).to(DEV)
    want = coda.attention(d["Q"], d["K"], d["V"], cu, n_q, n_kv)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = coda.attention(d["Q"], d["K"], d["V"], cu, n_q, n_kv, stream=side)
    side.synchronize()
    assert torch.equal(got["O"], want["O"]) and torch.equal(got["lse"], want["lse"])


def test_own_scale_both_ways(coda):
    n_q, n_kv, scale = 4, 2, 0.3
    t, cq, _, Tq, _ = make([140, 9], None, n_q, n_kv, seed=9)
    t["dO"] = synth.randn_bf16((Tq, n_q * D), 1.0, 82)
    d = {k: v.to(DEV) for k, v in t.items()}
    cu = torch.from_numpy(cq).to(DEV)
    f = coda.attention(d["Q"], d["K"], d["V"], cu, n_q, n_kv, scale=scale)
    x = {k: to_np(v) for k, v in t.items()}
    check_forward(f, O.attention_fwd(x["Q"], x["K"], x["V"], cq, cq, n_q, n_kv, scale), t, cq, cq, n_q, n_kv, scale)
    g = coda.attention_bwd(d["dO"], d["Q"], d["K"], d["V"], f["O"], f["lse"], cu, n_q, n_kv, scale=scale)
    r = O.attention_bwd(x["dO"], x["Q"], x["K"], x["V"], cq, cq, n_q, n_kv, scale)
    check_backward(g, r, t, cq, cq, n_q, n_kv, scale)


def test_no_queries_or_no_keys_at_all(coda):
    n_q, n_kv = 4, 2

    def bf(rows, heads, v=1.0):
        return torch.full((rows, heads * D), v, dtype=torch.bfloat16, device=DEV)

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)
    # no keys: O = 0, lse = -inf, dQ = 0
    kw = {"cu_seqlens_k": i32([0, 0, 0])}
    f = coda.attention(bf(9, n_q), bf(0, n_kv), bf(0, n_kv), i32([0, 4, 9]), n_q, n_kv, **kw)
    assert torch.all(f["O"] == 0) and bool(torch.isneginf(f["lse"]).all())
    g = coda.attention_bwd(bf(9, n_q), bf(9, n_q), bf(0, n_kv), bf(0, n_kv), f["O"], f["lse"], i32([0, 4, 9]), n_q, n_kv, **kw)
    assert torch.all(g["dQ"] == 0) and g["dK"].shape == (0, n_kv * D)
    # no queries: dK = dV = 0
    kw = {"cu_seqlens_k": i32([0, 200, 209])}
    f = coda.attention(bf(0, n_q), bf(209, n_kv), bf(209, n_kv), i32([0, 0, 0]), n_q, n_kv, **kw)
    assert f["O"].shape == (0, n_q * D)
    g = coda.attention_bwd(bf(0, n_q), bf(0, n_q), bf(209, n_kv), bf(209, n_kv), f["O"], f["lse"], i32([0, 0, 0]), n_q, n_kv,
                           out={"dQ": bf(0, n_q), "dK": bf(209, n_kv, 7.0), "dV": bf(209, n_kv, 7.0)}, **kw)
    assert torch.all(g["dK"] == 0) and torch.all(g["dV"] == 0)
    # no sequences: nothing is written
    out = {"O": bf(5, n_q, 7.0), "lse": torch.full((n_q, 5), 7.0, device=DEV)}
    coda.attention(bf(5, n_q), bf(5, n_kv), bf(5, n_kv), i32([0]), n_q, n_kv, out=out)
    assert torch.all(out["O"] == 7) and torch.all(out["lse"] == 7)


def test_two_streams_with_a_workspace_each(coda):
    n_q, n_kv = 4, 2
    t, cq, _, Tq, _ = make([300, 41, 200], None, n_q, n_kv, seed=8)
    t["dO"] = synth.randn_bf16((Tq, n_q * D), 1.0, 83)
    d = {k: v.to(DEV) for k, v in t.items()}
    cu = torch.from_numpy(cq).to(DEV)
    f = coda.attention(d["Q"], d["K"], d["V"], cu, n_q, n_kv)
    want = coda.attention_bwd(d["dO"], d["Q"], d["K"], d["V"], f["O"], f["lse"], cu, n_q, n_kv)
    torch.cuda.synchronize()
    got = []
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        for _ in range(3):
            h = coda.attention(d["Q"], d["K"], d["V"], cu, n_q, n_kv, stream=s)
            got.append((h, coda.attention_bwd(d["dO"], d["Q"], d["K"], d["V"], h["O"], h["lse"], cu, n_q, n_kv, stream=s)))
    torch.cuda.synchronize()
    for h, g in got:
        assert torch.equal(h["O"], f["O"]) and torch.equal(h["lse"], f["lse"])
        for k in want:
            assert torch.equal(g[k], want[k]), k


def test_status_of_calls_that_make_their_own_workspace(coda):
    """Without `ws` the status word is read through the result; the outputs are
    the result's only items."""
    n_q, n_kv = 4, 2
    t, _, _, Tq, _ = make([64, 64], None, n_q, n_kv)
    d = {k: v.to(DEV) for k, v in t.items()}
    good, bad = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in ([0, 64, 128], [0, 64, 129]))
    f = coda.attention(d["Q"], d["K"], d["V"], good, n_q, n_kv)
    args = (d["Q"], d["Q"], d["K"], d["V"], f["O"], f["lse"])
    g = coda.attention_bwd(*args, good, n_q, n_kv)
    assert list(f) == ["O", "lse"] and list(g) == ["dQ", "dK", "dV"] and len(g.values()) == 3
    assert coda.get_status(f["ws"]) == 0 and coda.get_status(g["ws"]) == 0
    with pytest.raises(KeyError):
        f["dQ"]
    own = {k: torch.full_like(v, 7.0) for k, v in f.items()}
    h = coda.attention(d["Q"], d["K"], d["V"], bad, n_q, n_kv, out=own)
    assert coda.get_status(h["ws"]) == 9 and h["O"] is own["O"] and list(own) == ["O", "lse"]
    assert coda.get_status(coda.attention_bwd(*args, bad, n_q, n_kv)["ws"]) == 9
    cache = coda.kv_cache_nvfp4(2, 16, n_kv)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    for slot, code in ((31, 0), (32, 10)):
        a = coda.kv_append_nvfp4(d["K"][:1], d["V"][:1], i32([slot]), cache)
        r = coda.kv_read_nvfp4(a, i32([slot]))           # the returned cache is the cache
        assert list(a) == list(cache) and all(a[k] is cache[k] for k in cache) and list(r) == ["K", "V"]
        assert coda.get_status(a["ws"]) == code and coda.get_status(r["ws"]) == code
    for page, n, code in ((1, 16, 0), (2, 16, 10), (1, 17, 9)):
        o = coda.attention_decode_nvfp4(d["Q"][:1], cache, i32([[page]]), i32([n]), n_q)
        assert coda.get_status(o["ws"]) == code and list(o) == ["O", "lse"]


@pytest.mark.parametrize("lq, lk, n_q, n_kv", [
    ([150, 20], None, 4, 2),
    ([1500, 40, 200], None, 12, 1),                      # some key tiles' groups are cut
    ([300, 1, 20], [290, 900, 20], 16, 2),
])
def test_backward_columns_of_one_projection(coda, lq, lk, n_q, n_kv):
    """Q, K, V as columns of one projection's output (K and V of another one
    where the keys are longer), each with its own offset and row stride: the
    bits of separate tensors."""
    cq = offsets(lq)
    ck = cq if lk is None else offsets(lk)
    Tq, Tk = int(cq[-1]), int(ck[-1])
    if lk is None:
        wide = synth.randn_bf16((Tq, (n_q + 2 * n_kv + 1) * D), 1.0, 5).to(DEV)
        Q, K, V, _ = wide.split([n_q * D, n_kv * D, n_kv * D, D], dim=1)
        kw = {}
    else:
        _, Q = synth.randn_bf16((Tq, (1 + n_q) * D), 1.0, 5).to(DEV).split([D, n_q * D], dim=1)
        V, _, K, _ = synth.randn_bf16((Tk, (2 * n_kv + 3) * D), 1.0, 6).to(DEV).split([n_kv * D, D, n_kv * D, 2 * D], dim=1)
        kw = {"cu_seqlens_k": torch.from_numpy(ck).to(DEV)}
    dO = synth.randn_bf16((Tq, n_q * D), 1.0, 7).to(DEV)
    cu = torch.from_numpy(cq).to(DEV)
    got = []
    for q, k, v in ((Q, K, V), (Q.contiguous(), K.contiguous(), V.contiguous())):
        f = coda.attention(q, k, v, cu, n_q, n_kv, **kw)
        g = coda.attention_bwd(dO, q, k, v, f["O"], f["lse"], cu, n_q, n_kv, **kw)
        assert coda.get_status(g["ws"]) == 0
        got.append({**f, **g})
    for k in got[0]:
        assert torch.equal(got[0][k], got[1][k]), k


@pytest.mark.parametrize("rows, n_q, backward", [(8300, 32, True), (30000, 32, True), (263000, 2, False)])
def test_short_sequences_in_front_of_many_padding_rows(coda, rows, n_q, backward):
    """The work lists' bins are as wide as the tensors' rows ask for, so here
    runs of different lengths share bins; the rows behind hold NaN."""
    lens, n_kv = [700, 1, 260, 0, 129, 40, 385], 1
    t, cq, _, n, _ = make(lens, None, n_q, n_kv, seed=21)
    t["dO"] = synth.randn_bf16((n, n_q * D), 1.0, 22)
    d = {}
    for k, v in t.items():
        d[k] = torch.full((rows, v.shape[1]), float("nan"), dtype=torch.bfloat16, device=DEV)
        d[k][:n] = v.to(DEV)
    cu = torch.from_numpy(cq).to(DEV)
    out = {"O": torch.full((rows, n_q * D), 7.0, dtype=torch.bfloat16, device=DEV),
           "lse": torch.full((n_q, rows), 7.0, device=DEV)}
    f = coda.attention(d["Q"], d["K"], d["V"], cu, n_q, n_kv, out=out)
    assert coda.get_status(f["ws"]) == 0
    x = {k: to_np(v) for k, v in t.items()}
    ref = O.attention_fwd(x["Q"], x["K"], x["V"], cq, cq, n_q, n_kv, D ** -0.5)
    check_forward({"O": out["O"][:n], "lse": out["lse"][:, :n]}, ref, t, cq, cq, n_q, n_kv, D ** -0.5)
    assert torch.all(out["O"][n:] == 7) and torch.all(out["lse"][:, n:] == 7)
    if backward:
        grads = {"d" + k: torch.full_like(d[k], 7.0) for k in ("Q", "K", "V")}
        g = coda.attention_bwd(d["dO"], d["Q"], d["K"], d["V"], out["O"], out["lse"], cu, n_q, n_kv, out=grads)
        assert coda.get_status(g["ws"]) == 0
        r = O.attention_bwd(x["dO"], x["Q"], x["K"], x["V"], cq, cq, n_q, n_kv, D ** -0.5)
        check_backward({k: v[:n] for k, v in grads.items()}, r, t, cq, cq, n_q, n_kv, D ** -0.5)
        assert all(torch.all(v[n:] == 7) for v in grads.values())
