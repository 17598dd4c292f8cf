"""The block with its attention core, and its serving form over the 4-bit
cache, run together as they are used.  Each stage is compared with the fp64
oracle on the stage's actual inputs (the bf16 tensors the previous stage
stored), so the tolerances are those of the single operators."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import synth
from oracle import coda_oracle as O
from parity import assert_bf16, to_np
from test_attention_gpu import check_backward, check_forward, offsets
from test_kvcache_gpu import check_decode

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


def test_training_step(coda):
    from gemm_epilogue_transformer_bf16_gb300.block import AttentionBlock
    lens = [100, 1, 219]
    shape = synth.BlockShape(tokens=320, hidden=256, n_q=4, n_kv=2, head_dim=D, inter=512, seq_len=256)
    t = synth.make_block(shape, seed=5)
    cu = offsets(lens)
    t["pos"] = torch.cat([torch.arange(n) for n in lens]).to(torch.int32)
    d = {k: v.to(DEV) for k, v in t.items()}
    blk = AttentionBlock(shape, d, n_seq=len(lens))
    dcu = torch.from_numpy(cu).to(DEV)
    f = blk.forward(d["x0"], d["pos"], dcu)
    g = blk.backward(d["x0"], d["pos"], dcu, d["dx2"])
    assert coda.get_status(blk.ws) == 0
    cfg = dict(n_q=shape.n_q, n_kv=shape.n_kv, head_dim=D, theta=shape.theta, eps=shape.eps)
    scale = D ** -0.5
    qkv = {k: f[k].cpu() for k in ("Q", "K", "V")}
    # attention on the Q, K, V the projection stored
    ref = O.attention_fwd(*(to_np(qkv[k]) for k in ("Q", "K", "V")), cu, cu, shape.n_q, shape.n_kv, scale)
    check_forward({"O": f["A"], "lse": blk.att["lse"]}, ref, qkv, cu, cu, shape.n_q, shape.n_kv, scale)
    # its gradients on the dA the output projection's backward stored
    qkv["dO"] = g["dA"].cpu()
    refb = O.attention_bwd(to_np(g["dA"]), *(to_np(qkv[k]) for k in ("Q", "K", "V")), cu, cu, shape.n_q, shape.n_kv, scale)
    check_backward({k: g[k] for k in ("dQ", "dK", "dV")}, refb, qkv, cu, cu, shape.n_q, shape.n_kv, scale)
    # everything around it, on the A, dQ, dK, dV of the core
    o = {k: v.double().numpy() for k, v in t.items()}
    o.update(A=to_np(f["A"]), dQ=to_np(g["dQ"]), dK=to_np(g["dK"]), dV=to_np(g["dV"]))
    rf, rb = O.block_fwd(o, **cfg), O.block_bwd(o, **cfg)
    for k in ("Q", "K", "V", "x1", "x2"):
        assert_bf16(f[k], rf[k], k)
    for k in ("dx0", "dA", "dWqkv", "dWo", "dWg", "dWu", "dWd", "dgamma_attn", "dgamma_mlp"):
        assert_bf16(g[k], rb[k], k)
    with pytest.raises(ValueError, match="offsets"):
        blk.forward(d["x0"], d["pos"], dcu[:-1])


def test_training_step_twice_and_as_a_graph(coda):
    from gemm_epilogue_transformer_bf16_gb300.block import AttentionBlock
    lens = [130, 60, 66]
    shape = synth.BlockShape(tokens=256, hidden=256, n_q=4, n_kv=2, head_dim=D, inter=256, seq_len=256)
    t = synth.make_block(shape, seed=8)
    t["pos"] = torch.cat([torch.arange(n) for n in lens]).to(torch.int32)
    d = {k: v.to(DEV) for k, v in t.items()}
    dcu = torch.from_numpy(offsets(lens)).to(DEV)
    blk = AttentionBlock(shape, d, n_seq=3)
    want = {k: v.clone() for k, v in blk.step(d["x0"], d["pos"], dcu, d["dx2"]).items()}
    cap = torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cap):
        again = blk.step(d["x0"], d["pos"], dcu, d["dx2"])
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(want[k], again[k]), k
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=cap):
        out = blk.step(d["x0"], d["pos"], dcu, d["dx2"])
    for v in out.values():
        v.zero_()
    g.replay()
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(want[k], out[k]), k
    assert coda.get_status(blk.ws) == 0


def test_serving_prompts_chunks_and_single_tokens(coda):
    """Two prompts are prefilled, one of them in two chunks, then both decode
    three tokens: the attention output of every step against the oracle on the
    rows the cache holds, and the block's output against the oracle on that."""
    from gemm_epilogue_transformer_bf16_gb300 import block as B
    page, n_q, n_kv = 16, 4, 2
    shape = synth.BlockShape(tokens=64, hidden=256, n_q=n_q, n_kv=n_kv, head_dim=D, inter=512, seq_len=128)
    t = synth.make_block(shape, seed=9)
    d = {k: v.to(DEV) for k, v in t.items()}
    w = {k: v.double().numpy() for k, v in t.items()}
    cache = coda.kv_cache_nvfp4(16, page, n_kv)
    order = torch.randperm(16, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    table = order.view(2, 8)                                   # sequence b: 8 pages, 128 tokens
    blk = B.ServingBlock(shape, d, cache)
    seen = {}

    def keep(name):
        real = getattr(B, name)

        def call(*a, **k):
            seen[name] = (a, real(*a, **k))
            return seen[name][1]
        return real, call
    originals = {}
    for name in ("attention", "attention_decode_nvfp4"):
        originals[name], fake = keep(name)
        setattr(B, name, fake)

    def slot(b, j):
        j = torch.as_tensor(j)
        return table[b][j // page].long() * page + j % page

    def x_of(n, seed):
        return synth.randn_bf16((n, shape.hidden), 1.0, seed)

    def rest(x, A):
        # the output projection and the MLP on the attention output
        x1 = x + A @ w["Wo"].T
        return O.mlp_fwd(x1, w["Wg"], w["Wu"], w["Wd"], x1, w["gamma_mlp"], shape.eps)

    def check_rest(y, x, A, name):
        ref = rest(to_np(x), to_np(A))
        assert_bf16(y, ref["y"], name)

    try:
        # both prompts' first part: 30 and 21 new tokens, whole so far
        lens = [30, 21]
        x = x_of(51, 30)
        pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32)
        slots = torch.cat([slot(b, torch.arange(n)) for b, n in enumerate(lens)]).to(torch.int32)
        y = blk.prefill(x.to(DEV), pos.to(DEV), slots.to(DEV), torch.from_numpy(offsets(lens)).to(DEV))
        (Q, K, V, *_), out = seen["attention"]
        ref = O.attention_fwd(to_np(Q), to_np(K), to_np(V), offsets(lens), offsets(lens), n_q, n_kv, D ** -0.5)
        check_forward(out, ref, {"Q": Q.cpu(), "K": K.cpu(), "V": V.cpu()}, offsets(lens), offsets(lens), n_q, n_kv, D ** -0.5)
        check_rest(y, x, out["O"], "prefill")
        # a second chunk of the first prompt: 17 new tokens behind the cached 30
        x = x_of(17, 31)
        keys = slot(0, torch.arange(47)).to(torch.int32)
        y = blk.prefill(x.to(DEV), torch.arange(30, 47, dtype=torch.int32, device=DEV),
                        slot(0, torch.arange(30, 47)).to(torch.int32).to(DEV),
                        torch.tensor([0, 17], dtype=torch.int32, device=DEV), key_slots=keys.to(DEV),
                        cu_seqlens_k=torch.tensor([0, 47], dtype=torch.int32, device=DEV))
        (Q, K, V, *_), out = seen["attention"]
        assert torch.equal(K, coda.kv_read_nvfp4(cache, keys.to(DEV))["K"])
        cq, ck = offsets([17]), offsets([47])
        ref = O.attention_fwd(to_np(Q), to_np(K), to_np(V), cq, ck, n_q, n_kv, D ** -0.5)
        check_forward(out, ref, {"Q": Q.cpu(), "K": K.cpu(), "V": V.cpu()}, cq, ck, n_q, n_kv, D ** -0.5)
        check_rest(y, x, out["O"], "second chunk")
        lens = [47, 21]
        for step in range(3):
            x = x_of(2, 40 + step)
            new = torch.tensor([slot(b, lens[b]) for b in range(2)], dtype=torch.int32)
            pos = torch.tensor(lens, dtype=torch.int32)
            lens = [n + 1 for n in lens]
            y = blk.decode(x.to(DEV), pos.to(DEV), new.to(DEV), table.to(DEV),
                           torch.tensor(lens, dtype=torch.int32, device=DEV))
            (Q, *_), out = seen["attention_decode_nvfp4"]
            rows = [coda.kv_read_nvfp4(cache, slot(b, torch.arange(n)).to(torch.int32).to(DEV), dtype=torch.float32)
                    for b, n in enumerate(lens)]
            at = [slot(b, torch.arange(n)) for b, n in enumerate(lens)]
            scl = [to_np(cache["scale"])[a // page, 1, :, a % page] for a in at]
            check_decode(out, to_np(Q), lens, [to_np(r["K"]) for r in rows], [to_np(r["V"]) for r in rows], scl, n_q, n_kv,
                         D ** -0.5)
            check_rest(y, x, out["O"], f"decode {step}")
    finally:
        for name, real in originals.items():
            setattr(B, name, real)


def test_padded_training_batch_after_a_full_one(coda):
    """Rows behind the last sequence take no part in the attention, whatever an
    earlier step left there, and add to the weight gradients what their own dx2
    gives."""
    from gemm_epilogue_transformer_bf16_gb300.block import AttentionBlock
    shape = synth.BlockShape(tokens=256, hidden=256, n_q=4, n_kv=2, head_dim=D, inter=256, seq_len=256)
    t = synth.make_block(shape, seed=12)
    t["pos"] = (torch.arange(256) % 128).to(torch.int32)
    d = {k: v.to(DEV) for k, v in t.items()}
    cu = offsets([70, 100])
    blk, fresh = AttentionBlock(shape, d, n_seq=2), AttentionBlock(shape, d, n_seq=2)
    blk.step(d["x0"], d["pos"], torch.tensor([0, 128, 256], dtype=torch.int32, device=DEV), d["dx2"])
    dcu = torch.from_numpy(cu).to(DEV)
    f = blk.forward(d["x0"], d["pos"], dcu)
    g = blk.backward(d["x0"], d["pos"], dcu, d["dx2"])
    want = fresh.step(d["x0"], d["pos"], dcu, d["dx2"])
    for k in want:
        assert torch.equal(g[k], want[k]), k
    assert torch.all(f["A"][170:] == 0) and all(torch.all(g[k][170:] == 0) for k in ("dQ", "dK", "dV"))
    cfg = dict(n_q=4, n_kv=2, head_dim=D, theta=shape.theta, eps=shape.eps)
    o = {k: v.double().numpy() for k, v in t.items()}
    o.update(A=to_np(f["A"]), dQ=to_np(g["dQ"]), dK=to_np(g["dK"]), dV=to_np(g["dV"]))
    rf, rb = O.block_fwd(o, **cfg), O.block_bwd(o, **cfg)
    for k in ("x1", "x2"):
        assert_bf16(f[k], rf[k], k)
    for k in ("dx0", "dWqkv", "dWo", "dWg", "dWu", "dWd"):
        assert_bf16(g[k], rb[k], k)
    assert coda.get_status(blk.ws) == 0


def test_serving_reports_errors_and_pads(coda):
    from gemm_epilogue_transformer_bf16_gb300.block import ServingBlock
    shape = synth.BlockShape(tokens=64, hidden=256, n_q=4, n_kv=2, head_dim=D, inter=512, seq_len=128)
    d = {k: v.to(DEV) for k, v in synth.make_block(shape, seed=9).items()}
    cache = coda.kv_cache_nvfp4(4, 16, 2)
    blk = ServingBlock(shape, d, cache)
    ws = coda.workspace(blk.workspace_size(20, 20, 2))

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)
    x, pos = synth.randn_bf16((20, shape.hidden), 1.0, 3).to(DEV), i32(list(range(17)) + [0] * 3)
    cu = i32([0, 5, 17])
    y = blk.prefill(x, pos, i32(list(range(17)) + [-1] * 3), cu, ws=ws)      # three rows of padding
    again = blk.prefill(x, pos, i32(list(range(17)) + [-1] * 3), cu)
    assert coda.get_status(ws) == 0 and torch.equal(y, again) and bool(torch.isfinite(y.float()).all())
    blk.prefill(x, pos, i32(list(range(17)) + [64, -1, -1]), cu, ws=ws)
    assert coda.get_status(ws) == 10                     # CODA_ERR_PAGE_RANGE
    coda.reset_status(ws)
    blk.prefill(x, pos, i32([-1] * 20), i32([0, 5, 21]), ws=ws)
    assert coda.get_status(ws) == 9                      # CODA_ERR_SEQLEN_RANGE
    coda.reset_status(ws)
    one, p1, at, table = x[:2], i32([5, 12]), i32([-1, -1]), i32([[0], [0]])
    blk.decode(one, p1, at, table, i32([5, 16]), ws=ws)
    assert coda.get_status(ws) == 0
    blk.decode(one, p1, at, table, i32([5, 17]), ws=ws)
    assert coda.get_status(ws) == 9


def test_serving_workspace_holds_for_shorter_calls(coda):
    """workspace_size covers every call up to its counts: a few new tokens
    behind a long cached prefix need more room than many."""
    from gemm_epilogue_transformer_bf16_gb300.block import ServingBlock
    n_q, n_kv, keys = 4, 2, 2100
    shape = synth.BlockShape(tokens=64, hidden=256, n_q=n_q, n_kv=n_kv, head_dim=D, inter=512, seq_len=4096)
    d = {k: v.to(DEV) for k, v in synth.make_block(shape, seed=9).items()}
    cache = coda.kv_cache_nvfp4(2, 2048, n_kv)
    kv = synth.randn_bf16((keys, n_kv * D), 1.0, 4).to(DEV)
    slots = torch.arange(keys, dtype=torch.int32, device=DEV)
    coda.kv_append_nvfp4(kv, kv, slots, cache)
    blk = ServingBlock(shape, d, cache)
    ws = coda.workspace(blk.workspace_size(20000, 20000, 40))
    lib = coda.load()
    for t, n in ((1, 1), (3, 2), (40, 40), (700, 3), (2100, 1), (20000, 40)):
        assert lib.coda_attention_workspace_size(t, 20000, n, n_q, n_kv, D) <= ws.numel(), (t, n)
    for new in (1, 5, 200):
        x = synth.randn_bf16((new, shape.hidden), 1.0, 3).to(DEV)
        at = slots[keys - new:]
        y = blk.prefill(x, at, at, torch.tensor([0, new], dtype=torch.int32, device=DEV), key_slots=slots,
                        cu_seqlens_k=torch.tensor([0, keys], dtype=torch.int32, device=DEV), ws=ws)
        assert bool(torch.isfinite(y.float()).all())
    assert coda.get_status(ws) == 0


def test_serving_reports_positions(coda):
    """A position behind the rotation table shows in the caller's workspace, in
    both forms; the workspace serves the projections too."""
    from gemm_epilogue_transformer_bf16_gb300.block import ServingBlock
    shape = synth.BlockShape(tokens=64, hidden=256, n_q=4, n_kv=2, head_dim=D, inter=512, seq_len=128)
    d = {k: v.to(DEV) for k, v in synth.make_block(shape, seed=9).items()}
    blk = ServingBlock(shape, d, coda.kv_cache_nvfp4(4, 16, 2))

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)
    for rows in (1, 20):
        ws = coda.workspace(blk.workspace_size(rows, rows, rows))
        x, slots = synth.randn_bf16((rows, shape.hidden), 1.0, 3).to(DEV), i32(list(range(rows)))
        one = i32([[0], [1]] * (rows // 2) or [[0]])
        for last, code in ((127, 0), (128, 8), (-1, 8)):     # CODA_ERR_POSITION_RANGE
            pos = i32(list(range(rows - 1)) + [last])
            y = blk.prefill(x, pos, slots, i32([0, rows]), ws=ws)
            assert coda.get_status(ws) == code
            coda.reset_status(ws)
            z = blk.decode(x, pos, slots, one, i32([1] * rows), ws=ws)
            assert coda.get_status(ws) == code
            coda.reset_status(ws)
            if code == 0:                                    # the bits of calls that make their own
                assert torch.equal(y, blk.prefill(x, pos, slots, i32([0, rows])))
                assert torch.equal(z, blk.decode(x, pos, slots, one, i32([1] * rows)))


def test_without_programmatic_launch():
    """The runs above with programmatic dependent launch off (the switch is
    read once per process)."""
    e = dict(os.environ, CODA_PDL="0")
    here = os.path.abspath(__file__)
    r = subprocess.run([sys.executable, "-m", "pytest", here, "-x", "-q", "-m", "gpu", "-k", "training or serving"],
                       env=e, cwd=os.path.dirname(os.path.dirname(here)), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and " passed" in r.stdout, r.stdout[-3000:] + r.stderr[-2000:]
