"""CPU checks of the attention operators: arguments refused on the host
before anything is enqueued, empty problems, workspace sizes, and the oracle's
own pins (against a direct evaluation and finite differences)."""
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


def fwd(lib, Q=FAKE, ldq=512, K=FAKE, ldk=256, V=FAKE, ldv=256, cu_q=FAKE, cu_k=None, n_seq=2, n_q=4, n_kv=2, d=128,
        scale=0.1, O=FAKE, lse=FAKE, Tq=64, Tk=64, ws=FAKE, ws_bytes=WS):
    return lib.coda_attention(Q, ldq, K, ldk, V, ldv, cu_q, cu_k, n_seq, n_q, n_kv, d, scale, O, lse, Tq, Tk, ws,
                              ws_bytes, None)


@pytest.mark.parametrize("change, code", [
    (dict(Q=None), 1), (dict(K=None), 1), (dict(V=None), 1), (dict(O=None), 1), (dict(lse=None), 1),
    (dict(cu_q=None), 1), (dict(Tq=-1), 1), (dict(Tk=-1), 1), (dict(n_seq=-1), 1), (dict(n_q=0), 1), (dict(n_kv=0), 1),
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(Tk=65), 1),                                   # other key rows need their own offsets
    (dict(ldq=504), 1), (dict(ldk=128), 1), (dict(ldv=248), 1),
    (dict(d=64), 3), (dict(n_q=5), 3), (dict(Tq=1 << 30, Tk=1 << 30), 3),
    (dict(Q=FAKE + 2), 2), (dict(O=FAKE + 8), 2), (dict(cu_q=FAKE + 2), 2), (dict(ldq=516), 2), (dict(ws=FAKE + 4), 2),
    (dict(ws=None), 4), (dict(ws_bytes=255), 4),
    (dict(Tq=0, Tk=0), 0), (dict(n_seq=0), 0),          # nothing to do
])
def test_forward_refusals(lib, change, code):
    assert fwd(lib, **change) == code


@pytest.mark.parametrize("call", ["forward", "backward"])
def test_key_tiles_are_counted_too(lib, call):
    """Few queries over many keys: the key tiles times the heads must fit 32
    bits as the query tiles do."""
    Tq, Tk, n_q = 64, (1 << 30) - 1, 65535
    if call == "forward":
        assert fwd(lib, Tq=Tq, Tk=Tk, cu_k=2 * FAKE, n_q=n_q, n_kv=1, ldq=n_q * 128) == 3
    else:
        assert lib.coda_attention_bwd(FAKE, FAKE, n_q * 128, FAKE, 128, FAKE, 128, FAKE, FAKE, FAKE, 2 * FAKE, 2, n_q, 1,
                                      128, 0.1, FAKE, FAKE, FAKE, Tq, Tk, FAKE, 1 << 60, None) == 3


def test_workspace_grows_with_rows_and_sequences(lib):
    w = lib.coda_attention_workspace_size
    assert w(8192, 8192, 4, 64, 8, 128) < 65536
    assert w(8192, 8192, 4096, 64, 8, 128) > w(8192, 8192, 4, 64, 8, 128)


def test_binding_refuses_host_tensors_and_shapes():
    q = torch.zeros(4, 256, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        coda.attention(q, q, q, cu, 2, 2)


def test_oracle_forward_pins():
    rng = np.random.default_rng(0)
    n_q, n_kv, d = 4, 2, 8
    cq, ck = [0, 3, 3, 7], [0, 5, 6, 8]
    Q, K, V = rng.normal(size=(7, n_q * d)), rng.normal(size=(8, n_kv * d)), rng.normal(size=(8, n_kv * d))
    r = O.attention_fwd(Q, K, V, cq, ck, n_q, n_kv, 0.3)
    for h in range(n_q):
        kv = h // 2
        for b in range(3):
            lq, lk = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
            for i in range(lq):
                seen = range(max(0, min(lk, i + lk - lq + 1)))
                w = [np.exp(0.3 * Q[cq[b] + i, h * d:(h + 1) * d] @ K[ck[b] + j, kv * d:(kv + 1) * d]) for j in seen]
                got = r["O"][cq[b] + i, h * d:(h + 1) * d]
                if not w:
                    assert np.all(got == 0) and np.isneginf(r["lse"][h, cq[b] + i])
                    continue
                want = sum(x * V[ck[b] + j, kv * d:(kv + 1) * d] for x, j in zip(w, seen)) / sum(w)
                assert np.allclose(got, want, rtol=1e-12, atol=1e-14)
                assert np.isclose(r["lse"][h, cq[b] + i], np.log(sum(w)), rtol=1e-12)
    # one key: its value, whatever the score
    one = O.attention_fwd(Q[:1], K[:1], V[:1], [0, 1], [0, 1], n_q, n_kv, 5.0)
    assert np.allclose(one["O"].reshape(n_q, d), np.repeat(V[:1].reshape(n_kv, d), 2, axis=0))


# --------------------------------------------------------------------------- the 4-bit cache

def append(lib, K=FAKE, ldk=256, V=FAKE, ldv=256, slots=FAKE, T=5, codes=FAKE, sf=FAKE, scale=FAKE, pages=4, page=16,
           n_kv=2, d=128, ws=FAKE, ws_bytes=256):
    return lib.coda_kv_append_nvfp4(K, ldk, V, ldv, slots, T, codes, sf, scale, pages, page, n_kv, d, ws, ws_bytes, None)


def read(lib, codes=FAKE, sf=FAKE, scale=FAKE, pages=4, page=16, slots=FAKE, T=5, n_kv=2, d=128, K=FAKE, V=FAKE,
         dtype=0, ws=FAKE, ws_bytes=256):
    return lib.coda_kv_read_nvfp4(codes, sf, scale, pages, page, slots, T, n_kv, d, K, V, dtype, ws, ws_bytes, None)


def decode(lib, Q=FAKE, ldq=512, codes=FAKE, sf=FAKE, scale=FAKE, pages=4, page=16, table=FAKE, max_pages=4, lens=FAKE,
           batch=3, n_q=4, n_kv=2, d=128, sm=0.1, O=FAKE, lse=FAKE, ws=FAKE, ws_bytes=WS):
    return lib.coda_attention_decode_nvfp4(Q, ldq, codes, sf, scale, pages, page, table, max_pages, lens, batch, n_q,
                                           n_kv, d, sm, O, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("call, change, code", [
    (append, dict(K=None), 1), (append, dict(slots=None), 1), (append, dict(codes=None), 1), (append, dict(T=-1), 1),
    (append, dict(ldk=128), 1), (append, dict(page=0), 1), (append, dict(page=24), 3), (append, dict(page=8), 3),
    (append, dict(pages=1 << 27), 3), (append, dict(d=64), 3), (append, dict(V=FAKE + 2), 2), (append, dict(ldv=260), 2),
    (append, dict(sf=FAKE + 8), 2), (append, dict(ws=None), 4), (append, dict(ws_bytes=128), 4), (append, dict(T=0), 0),
    (read, dict(K=None), 1), (read, dict(dtype=2), 1), (read, dict(slots=None), 1), (read, dict(page=48), 3),
    (read, dict(V=FAKE + 4), 2), (read, dict(ws=None), 4), (read, dict(T=0), 0),
    (decode, dict(Q=None), 1), (decode, dict(table=None), 1), (decode, dict(lens=None), 1), (decode, dict(O=None), 1),
    (decode, dict(batch=-1), 1), (decode, dict(max_pages=-1), 1), (decode, dict(sm=0.0), 1), (decode, dict(ldq=256), 1),
    (decode, dict(n_q=3), 3), (decode, dict(d=96), 3), (decode, dict(page=100), 3), (decode, dict(max_pages=1 << 28), 3),
    (decode, dict(Q=FAKE + 2), 2), (decode, dict(ldq=516), 2), (decode, dict(lens=FAKE + 1), 2),
    (decode, dict(ws=None), 4), (decode, dict(ws_bytes=4096), 4), (decode, dict(batch=0), 0),
])
def test_cache_refusals(lib, call, change, code):
    assert call(lib, **change) == code


def test_binding_refuses_host_caches_and_types():
    cache = coda.kv_cache_nvfp4(2, 16, 2, device="cpu")
    assert cache["codes"].shape == (2, 2, 2, 16, 64) and cache["sf"].shape == (2, 2, 2, 16, 8)
    x = torch.zeros(3, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        coda.kv_append_nvfp4(x, x, torch.zeros(3, dtype=torch.int32), cache)
    with pytest.raises(TypeError):
        coda.kv_read_nvfp4(cache, torch.zeros(3, dtype=torch.int32), dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        coda.kv_read_nvfp4(cache, torch.zeros(3, dtype=torch.int32))


# --------------------------------------------------------------------------- backward

def bwd(lib, dO=FAKE, Q=FAKE, ldq=512, K=FAKE, ldk=256, V=FAKE, ldv=256, O=FAKE, lse=FAKE, cu_q=FAKE, cu_k=None,
        n_seq=2, n_q=4, n_kv=2, d=128, scale=0.1, dQ=FAKE, dK=FAKE, dV=FAKE, Tq=64, Tk=64, ws=FAKE, ws_bytes=WS):
    return lib.coda_attention_bwd(dO, Q, ldq, K, ldk, V, ldv, O, lse, cu_q, cu_k, n_seq, n_q, n_kv, d, scale, dQ, dK, dV,
                                  Tq, Tk, ws, ws_bytes, None)


@pytest.mark.parametrize("change, code", [
    *[({n: None}, 1) for n in ("dO", "Q", "K", "V", "O", "lse", "cu_q", "dQ", "dK", "dV")],
    (dict(Tk=65), 1), (dict(scale=0.0), 1), (dict(ldq=256), 1), (dict(d=256), 3), (dict(n_q=3), 3),
    *[({n: FAKE + 2}, 2) for n in ("dO", "Q", "K", "V", "O", "dQ", "dK", "dV")], (dict(ldv=260), 2),
    (dict(ws=None), 4), (dict(ws_bytes=1024), 4), (dict(Tq=0, Tk=0), 0), (dict(n_seq=0), 0),
])
def test_backward_refusals(lib, change, code):
    assert bwd(lib, **change) == code


def test_oracle_backward_against_differences():
    rng = np.random.default_rng(2)
    n_q, n_kv, d = 4, 2, 4
    cq, ck = [0, 3, 5], [0, 5, 6]
    x = {"Q": rng.normal(size=(5, n_q * d)), "K": rng.normal(size=(6, n_kv * d)), "V": rng.normal(size=(6, n_kv * d))}
    dO = rng.normal(size=(5, n_q * d))
    r = O.attention_bwd(dO, x["Q"], x["K"], x["V"], cq, ck, n_q, n_kv, 0.4)
    for name in x:
        for i in np.ndindex(x[name].shape):
            f = []
            for s in (1, -1):
                y = {k: v.copy() for k, v in x.items()}
                y[name][i] += s * 1e-6
                f.append(np.sum(O.attention_fwd(y["Q"], y["K"], y["V"], cq, ck, n_q, n_kv, 0.4)["O"] * dO))
            assert abs((f[0] - f[1]) / 2e-6 - r["d" + name][i]) < 1e-7


# --------------------------------------------------------------------------- workspaces

@pytest.mark.parametrize("ws, error, match", [
    (torch.zeros(1, dtype=torch.uint8).expand(4096), ValueError, "contiguous"),     # one byte, said to be 4096
    (torch.zeros(8192, dtype=torch.uint8)[::2], ValueError, "contiguous"),
    (bytearray(4096), TypeError, "Tensor"),
    (torch.zeros(255, dtype=torch.uint8), ValueError, "too small"),
])
def test_workspace_must_be_memory_of_its_size(ws, error, match):
    """What the attention and cache calls take for their workspace, before
    anything is enqueued (device -1: the host, where the check alone runs)."""
    with pytest.raises(error, match=match):
        coda._scratch(ws, 256, -1, None)


def test_workspace_of_the_size_is_taken():
    ws = torch.zeros(4096, dtype=torch.uint8)
    assert coda._scratch(ws, 4096, -1, None) == (ws.data_ptr(), 4096, ws)


def test_results_name_the_workspace_of_their_call():
    """result["ws"] beside the items: the workspace a call made, or the one it
    was given when an earlier result is passed as its outputs."""
    a, b = torch.zeros(256, dtype=torch.uint8), torch.ones(256, dtype=torch.uint8)
    plain = {"O": 1, "lse": 2}
    assert coda._told(plain, a, a) is plain and "ws" not in plain
    made = coda._told(plain, None, a)
    assert made == plain and list(made.values()) == [1, 2] and made["ws"] is a and made.get("ws") is None
    assert coda._told(made, b, b) is made and made["ws"] is b
    assert coda._told(made, None, a)["ws"] is a and made["ws"] is b
    with pytest.raises(KeyError):
        made["K"]
