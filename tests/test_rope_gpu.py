"""Rotary positions from tables, and the append to the 4-bit cache that rotates
on the way, against the fp64 oracle.

Tolerances.  A rotated element is x1 c - x2 s with both products and the sum
rounded to fp32 (3 * 2^-24 of |x1 c| + |x2 s|), then bf16 (2^-8 of the value).
Codes and scales of the cache are decisions: bit for bit those of the fp32
values that numpy computes in the same order.  A table entry is rounded to fp32
once (2^-24) and its angle in fp64 is off by 2^-50 of at most 10^6 (below
2^-29)."""
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


SCALINGS = [None, dict(kind="linear", factor=4.0), dict(kind="bands", factor=8.0, original=1024, low=1.0, high=4.0),
            dict(kind="ramp", factor=16.0, original=512, amplitude=1.25)]


@pytest.mark.parametrize("scaling", SCALINGS, ids=lambda s: s["kind"] if s else "plain")
@pytest.mark.parametrize("rotary, far", [(128, 70), (32, 5000), (96, 1)])
def test_table(coda, scaling, rotary, far):
    got = to_np(coda.rope_table(5e5, rotary, far, scaling=scaling))
    kw = dict(scaling or {})
    amp = kw.pop("amplitude", 1.0)
    a = np.arange(far)[:, None] * O.rope_scaled_frequencies(5e5, rotary, **kw)
    for i, f in enumerate((np.cos, np.sin)):
        assert np.all(np.abs(got[..., i] - amp * f(a)) <= amp * (2.0 ** -24 * np.abs(f(a)) + 2.0 ** -29))


def inputs(coda, T, heads, rotary, far, seed=0, pad=0):
    cs = coda.rope_table(1e4, rotary, far, scaling=SCALINGS[1])
    pos = torch.randint(0, far, (T,), generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    if T:
        pos[-1] = far - 1
    x = synth.randn_bf16((T, heads * D + pad), 1.0, seed + 1).to(DEV)[:, :heads * D]
    return x, pos.to(DEV), cs


def check_rotation(got, x, pos, cs, heads, pairing, back=False):
    x, t = to_np(x).reshape(-1, heads, D), to_np(cs)[to_np(pos).astype(int)]
    cos, sin = t[..., 0], t[..., 1] * (-1 if back else 1)
    want = O.rope_part(x, cos, sin, pairing)
    size = O.rope_part(np.abs(x), np.abs(cos), np.zeros_like(sin), pairing) + \
        np.abs(O.rope_part(np.abs(x), np.zeros_like(cos), np.abs(sin), pairing))
    bound = 3 * 2.0 ** -24 * size + 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -8)
    rotary = 2 * cos.shape[1]
    g = to_np(got).reshape(want.shape)
    assert np.all(np.abs(g - want)[..., :rotary] <= bound[..., :rotary])
    assert np.array_equal(g[..., rotary:], x[..., rotary:])


@pytest.mark.parametrize("pairing", ["interleaved", "half"])
@pytest.mark.parametrize("T, heads, rotary, pad", [(1, 1, 128, 0), (7, 3, 64, 0), (33, 13, 96, 64), (5, 72, 128, 8),
                                                   (130, 10, 16, 256), (0, 4, 128, 0)])
def test_rotation_and_gradient(coda, T, heads, rotary, pad, pairing):
    x, pos, cs = inputs(coda, T, heads, rotary, 300, pad=pad)
    ws = coda.workspace(256)
    y = coda.rope(x, pos, cs, heads, pairing=pairing, ws=ws)["Y"]
    dx = coda.rope_bwd(x, pos, cs, heads, pairing=pairing, ws=ws)["dX"]
    assert coda.get_status(ws) == 0
    check_rotation(y, x, pos, cs, heads, pairing)
    check_rotation(dx, x, pos, cs, heads, pairing, back=True)
    # in place, in the columns of a wider tensor
    z = x.clone() if not pad else torch.empty(T, heads * D + pad, dtype=x.dtype, device=DEV).copy_(
        torch.nn.functional.pad(x, (0, pad), value=7.0))[:, :heads * D]
    coda.rope(z, pos, cs, heads, pairing=pairing, out={"Y": z})
    assert torch.equal(z, y)


@pytest.mark.parametrize("pairing", ["interleaved", "half"])
def test_gradient_against_differences(coda, pairing):
    """<rope(x), g> is linear in x: its derivative along e is <rope(e), g> = <e, rope_bwd(g)>."""
    heads, T = 3, 4
    x, pos, cs = inputs(coda, T, heads, 64, 50)
    g = synth.randn_bf16((T, heads * D), 1.0, 9).to(DEV)
    dx = to_np(coda.rope_bwd(g, pos, cs, heads, pairing=pairing)["dX"])
    t = to_np(cs)[to_np(pos).astype(int)]
    f = lambda v: (O.rope_part(v.reshape(T, heads, D), t[..., 0], t[..., 1], pairing).reshape(T, -1) * to_np(g)).sum()
    base, h = to_np(x), 1e-3
    for i in [(0, 0), (1, 5), (2, 33), (3, 63), (0, 70), (2, 200), (3, 383)]:
        up, down = base.copy(), base.copy()
        up[i] += h
        down[i] -= h
        assert abs((f(up) - f(down)) / (2 * h) - dx[i]) <= 2.0 ** -8 * abs(dx[i]) + 1e-6


def test_positions_outside_the_table_are_clamped_and_told(coda):
    x, pos, cs = inputs(coda, 3, 2, 128, 10)
    ws = coda.workspace(256)
    bad = torch.tensor([-4, 10, 3], dtype=torch.int32, device=DEV)
    y = coda.rope(x, bad, cs, 2, ws=ws)["Y"]
    assert coda.get_status(ws) == 8                      # CODA_ERR_POSITION_RANGE
    assert torch.equal(y, coda.rope(x, bad.clamp(0, 9), cs, 2)["Y"])
    coda.reset_status(ws)
    cache = coda.kv_cache_nvfp4(1, 16, 2)
    coda.kv_append_rope_nvfp4(x, x, torch.arange(3, dtype=torch.int32, device=DEV), cache, bad, cs, ws=ws)
    assert coda.get_status(ws) == 8


def rotated_f32(x, pos, cs, heads, pairing):
    """The rotation in fp32, in the order that the kernel keeps."""
    x = x.float().cpu().numpy().reshape(-1, heads, D).copy()
    t = cs.cpu().numpy()[pos.cpu().numpy()][:, None]
    c, s = t[..., 0], t[..., 1]
    r = 2 * cs.shape[1]
    first, second = (np.s_[..., 0:r:2], np.s_[..., 1:r:2]) if pairing == "interleaved" else (np.s_[..., :r // 2], np.s_[..., r // 2:r])
    a, b = x[first].copy(), x[second].copy()
    x[first], x[second] = a * c - b * s, b * c + a * s
    assert x.dtype == np.float32
    return x


@pytest.mark.parametrize("pairing", ["interleaved", "half"])
@pytest.mark.parametrize("T, page, n_q, n_kv, rotary, packed, keep", [
    (1, 16, 2, 1, 128, False, True), (9, 16, 0, 3, 64, False, False), (130, 64, 12, 4, 96, True, True),
    (65, 256, 64, 8, 128, True, False), (20, 16, 5, 1, 48, False, True), (0, 16, 2, 1, 128, False, True)])
def test_append_rotates_on_the_way(coda, T, page, n_q, n_kv, rotary, packed, keep, pairing):
    qkv, pos, cs = inputs(coda, T, n_q + 2 * n_kv, rotary, 200)
    parts = qkv.split([n_q * D, n_kv * D, n_kv * D], dim=1)
    Q, K, V = parts if packed else (p.contiguous() for p in parts)
    pages = -(-T // page) + 2
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(3))[:T].to(torch.int32)
    if T > 4:
        slots[4] = -1                                    # rotated, not appended
    cache = coda.kv_cache_nvfp4(pages, page, n_kv)
    for t in cache.values():
        t.fill_(77)                                      # what no token names must stay
    ws = coda.workspace(256)
    out = coda.kv_append_rope_nvfp4(K, V, slots.to(DEV), cache, pos, cs, Q=Q if n_q else None, n_q=n_q, pairing=pairing,
                                    keep_k=keep, ws=ws)
    assert coda.get_status(ws) == 0 and set(out) == ({"Q"} if n_q else set()) | ({"K"} if keep else set())
    if n_q:
        assert torch.equal(out["Q"], coda.rope(Q, pos, cs, n_q, pairing=pairing)["Y"])
    if keep:
        assert torch.equal(out["K"], coda.rope(K, pos, cs, n_kv, pairing=pairing)["Y"])
    live = (slots >= 0).numpy()
    at = slots.numpy()[live]
    want = {n: t.clone().fill_(77).cpu().numpy() for n, t in cache.items()}
    for plane, x in enumerate((rotated_f32(K, pos, cs, n_kv, pairing), to_np(V).reshape(T, n_kv, D))):
        if not T:
            break
        codes, sf, s, _ = O.quantize_nvfp4_rows(x.reshape(T * n_kv, D).astype(np.float64))
        packed_codes = (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
        for name, part in (("codes", packed_codes.reshape(T, n_kv, 64)), ("sf", sf.reshape(T, n_kv, 8)),
                           ("scale", s.reshape(T, n_kv))):
            want[name][at // page, plane, :, at % page] = part[live]
    for name in want:
        assert np.array_equal(cache[name].cpu().numpy(), want[name]), name


def test_append_s_slots_outside_the_cache_set_status(coda):
    qkv, pos, cs = inputs(coda, 4, 3, 64, 20)
    K, V = qkv[:, D:2 * D], qkv[:, 2 * D:]
    cache, ws = coda.kv_cache_nvfp4(2, 16, 1), coda.workspace(256)
    slots = torch.tensor([3, 32, -1, 31], dtype=torch.int32, device=DEV)
    coda.kv_append_rope_nvfp4(K, V, slots, cache, pos, cs, ws=ws)
    assert coda.get_status(ws) == 10                     # CODA_ERR_PAGE_RANGE
    other = coda.kv_cache_nvfp4(2, 16, 1)
    good = torch.tensor([3, -1, -1, 31], dtype=torch.int32, device=DEV)
    coda.kv_append_rope_nvfp4(K, V, good, other, pos, cs)
    assert all(torch.equal(cache[n], other[n]) for n in other)


def test_no_rotation_is_the_plain_append(coda):
    """At position 0 the rotation is the identity: the codes of kv_append_nvfp4."""
    qkv, _, cs = inputs(coda, 40, 4, 128, 3)
    K, V = qkv[:, :2 * D].contiguous(), qkv[:, 2 * D:].contiguous()
    slots = torch.arange(40, dtype=torch.int32, device=DEV)
    a, b = coda.kv_cache_nvfp4(3, 16, 2), coda.kv_cache_nvfp4(3, 16, 2)
    coda.kv_append_rope_nvfp4(K, V, slots, a, torch.zeros_like(slots), cs, pairing="half")
    coda.kv_append_nvfp4(K, V, slots, b)
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_rotation_in_a_graph_beside_an_eager_one(coda):
    x, pos, cs = inputs(coda, 50, 6, 128, 100)
    want = coda.rope(x, pos, cs, 6)["Y"]
    back = coda.rope_bwd(x, pos, cs, 6)["dX"]
    out, ws = {"Y": torch.zeros_like(want)}, coda.workspace(256)
    grad = {"dX": torch.zeros_like(want)}
    cap = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=cap):
        coda.rope(x, pos, cs, 6, out=out, ws=ws)
        coda.rope_bwd(x, pos, cs, 6, out=grad, ws=ws)
    for _ in range(2):
        g.replay()
        side = coda.rope(x, pos, cs, 6)["Y"]
        torch.cuda.synchronize()
        assert torch.equal(out["Y"], want) and torch.equal(side, want) and torch.equal(grad["dX"], back)


def test_refusals(coda):
    x, pos, cs = inputs(coda, 4, 2, 64, 20)
    with pytest.raises(ValueError, match="X: expected"):
        coda.rope(x, pos, cs, 3)
    with pytest.raises(ValueError, match="pos"):
        coda.rope(x, pos[:3], cs, 2)
    with pytest.raises(TypeError, match="pos"):
        coda.rope(x, pos.long(), cs, 2)
    with pytest.raises(ValueError, match="cos_sin"):
        coda.rope(x, pos, cs[..., 0].contiguous(), 2)
    with pytest.raises(ValueError, match="pairing"):
        coda.rope(x, pos, cs, 2, pairing="other")
    with pytest.raises(ValueError, match="Y"):
        coda.rope(x, pos, cs, 2, out={"Y": x[:, :D]})
    with pytest.raises(coda.CodaError):                  # 24 rotated elements
        coda.rope(x, pos, coda.rope_table(1e4, 24, 20), 2)
    cache = coda.kv_cache_nvfp4(2, 16, 1)
    with pytest.raises(ValueError, match="both or none"):
        coda.kv_append_rope_nvfp4(x[:, :D], x[:, D:], pos, cache, pos, cs, Q=x)
    with pytest.raises(ValueError, match="slots"):
        coda.kv_append_rope_nvfp4(x[:, :D], x[:, D:], pos[:2], cache, pos, cs)
