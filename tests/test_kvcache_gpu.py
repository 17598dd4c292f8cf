"""The 4-bit key/value cache against the fp64 oracle: append (codes and scales
bit for bit), read back, and single-token attention over it.

Tolerances of the attention, from the kernel's roundings:

  scores  K' = e2m1 * e4m3 and Q (scaled by a power of two) are exact in f16
          up to f16's smallest step for Q elements far below the head's
          largest (2^-25 of it); 128 products summed in fp32 are off by at
          most 128 * 2^-24 of their absolute sum, three fp32 factors by
          2^-24 of the score each:
            e = scale (128 2^-24 sum|q k| + 128 2^-25 max|q| max|k|) + 2^-22 |s|
  O       weights times row scales are rounded to f16: half a step is 2^-11
          relative, or 2^-25 units where the largest weighted row scale is
          at least one unit (the kernel keeps it between 1 and 2^14), times
          values of at most 2688; O is rounded to bf16 once (2^-8); a weight moves by
          exp(+-2e); the sums over n keys add n 2^-24 each.
  lse     off by e, n 2^-24, and 2^-22 (|lse| + 16) for the fp32 logarithms
          and products.
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


def rows(T, n_kv, seed, spread=True):
    """bf16 rows of very different sizes, a zero row and a row of one element
    among them."""
    x = synth.randn_bf16((T, n_kv * D), 1.0, seed).float()
    if spread:
        g = torch.Generator().manual_seed(seed + 50)
        x *= torch.exp2(torch.randint(-12, 12, (T, 1), generator=g).float())
    x = x.to(torch.bfloat16)
    if T > 3:
        x[1] = 0
        x[2] = 0
        x[2, 5] = 3.0
    return x


def oracle_rows(x, n_kv):
    """codes [T, n_kv, 64], sf [T, n_kv, 8], scale [T, n_kv], values [T, n_kv*128]."""
    T = x.shape[0]
    codes, sf, s, vals = O.quantize_nvfp4_rows(to_np(x).reshape(T * n_kv, D))
    packed = (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    return (packed.reshape(T, n_kv, 64), sf.reshape(T, n_kv, 8), s.reshape(T, n_kv),
            (vals * s.astype(np.float64)[:, None]).reshape(T, n_kv * D))


@pytest.mark.parametrize("T, page, pages, n_kv", [(1, 16, 2, 1), (7, 16, 3, 3), (130, 64, 5, 2), (65, 256, 1, 8)])
def test_append_and_read(coda, T, page, pages, n_kv):
    K, V = rows(T, n_kv, 1), rows(T, n_kv, 2)
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(3))[:T].to(torch.int32)
    if T > 4:
        slots[4] = -1                                   # skipped
    cache = coda.kv_cache_nvfp4(pages, page, n_kv)
    for t in cache.values():
        t.fill_(77)                                     # what no token names must stay
    ws = coda.workspace(256)
    # rows as columns of one wider tensor
    kv = torch.cat([K, V], dim=1).to(DEV)
    k, v = kv.split([n_kv * D, n_kv * D], dim=1)
    coda.kv_append_nvfp4(k, v, slots.to(DEV), cache, ws=ws)
    assert coda.get_status(ws) == 0
    live = (slots >= 0).numpy()
    want = {n: t.clone().fill_(77).cpu().numpy() for n, t in cache.items()}
    at = slots.numpy()[live]
    for plane, x in enumerate((K, V)):
        for name, part in zip(("codes", "sf", "scale"), oracle_rows(x, n_kv)):
            want[name][at // page, plane, :, at % page] = part[live]
    for name in want:
        assert np.array_equal(cache[name].cpu().numpy(), want[name]), name
    back = coda.kv_read_nvfp4(cache, slots.to(DEV), dtype=torch.float32, ws=ws)
    half = coda.kv_read_nvfp4(cache, slots.to(DEV), ws=ws)
    assert coda.get_status(ws) == 0
    for n, x in (("K", K), ("V", V)):
        val = oracle_rows(x, n_kv)[3]
        val[~live] = 0
        f32 = torch.from_numpy(val).float()             # the exact product, rounded once
        assert torch.equal(back[n].cpu(), f32), n
        assert torch.equal(half[n].cpu(), f32.to(torch.bfloat16)), n


def test_slots_outside_the_cache_set_status(coda):
    n_kv, page, pages = 2, 16, 2
    K, V = rows(5, n_kv, 1).to(DEV), rows(5, n_kv, 2).to(DEV)
    cache = coda.kv_cache_nvfp4(pages, page, n_kv)
    ws = coda.workspace(256)
    slots = torch.tensor([0, 32, 5, -3, 31], dtype=torch.int32, device=DEV)
    coda.kv_append_nvfp4(K, V, slots, cache, ws=ws)
    assert coda.get_status(ws) == 10                     # CODA_ERR_PAGE_RANGE
    coda.reset_status(ws)
    good = torch.tensor([0, 5, 31], dtype=torch.int32, device=DEV)
    got = coda.kv_read_nvfp4(cache, good, dtype=torch.float32, ws=ws)["K"].cpu()
    assert torch.equal(got, torch.from_numpy(oracle_rows(K.cpu(), n_kv)[3][[0, 2, 4]]).float())
    assert coda.get_status(ws) == 0
    z = coda.kv_read_nvfp4(cache, slots, ws=ws)
    assert coda.get_status(ws) == 10 and torch.all(z["V"][[1, 3]] == 0)


def fill(coda, lens, page, n_kv, spread, seed=7):
    """A cache with the sequences' rows on shuffled pages, its table, and what
    the rows stand for (per sequence, [len, n_kv*128])."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((len(lens), max(need + [0]) + 1), 1 << 28, dtype=torch.int32)   # entries that must not be read
    cache = coda.kv_cache_nvfp4(pages, page, n_kv)
    cache["sf"].fill_(0x7F)                              # unwritten rows hold NaN scales
    cache["scale"].fill_(float("nan"))
    ks, vs, slots, at = [], [], [], 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        j = torch.arange(n)
        slots.append(table[b][(j // page)] * page + (j % page).to(torch.int32))
        ks.append(rows(n, n_kv, seed + 10 * b, False))
        vs.append(rows(n, n_kv, seed + 10 * b + 1, spread))
        at += need[b]
    if sum(lens):
        coda.kv_append_nvfp4(torch.cat(ks).to(DEV), torch.cat(vs).to(DEV), torch.cat(slots).to(torch.int32).to(DEV), cache)
    val = [[oracle_rows(x, n_kv)[3] if x.shape[0] else np.zeros((0, n_kv * D)) for x in part] for part in (ks, vs)]
    scl = [oracle_rows(x, n_kv)[2] if x.shape[0] else np.zeros((0, n_kv)) for x in vs]
    return cache, table, val[0], val[1], scl


def check_decode(out, Q, lens, kval, vval, vscale, n_q, n_kv, scale):
    cq = np.arange(len(lens) + 1)
    ck = np.concatenate([[0], np.cumsum(lens)]).astype(int)
    K, V = np.concatenate(kval), np.concatenate(vval)
    ref = O.attention_fwd(Q, K, V, cq, ck, n_q, n_kv, scale)
    got, lse = to_np(out["O"]), to_np(out["lse"])
    for b, n in enumerate(lens):
        for h in range(n_q):
            kv = h // (n_q // n_kv)
            c = slice(h * D, (h + 1) * D)
            if n == 0:
                assert np.all(got[b, c] == 0) and np.isneginf(lse[b, h])
                continue
            q, k = Q[b, c], K[ck[b]:ck[b + 1], kv * D:(kv + 1) * D]
            s = scale * (k @ q)
            e = (scale * (D * 2.0 ** -24 * np.abs(k) @ np.abs(q) + D * 2.0 ** -25 * np.abs(q).max() * np.abs(k).max())
                 + 2.0 ** -22 * np.abs(s)).max()
            p = np.exp(s - ref["lse"][h, b])
            rel = np.expm1(2 * e) + 4 * n * 2.0 ** -24 + 2.0 ** -20
            small = n * 2.0 ** -25 * (p * vscale[b][:, kv]).max() * 2688
            bound = (2.0 ** -11 + rel) * ref["A"][b, c] * (1 + 2.0 ** -8) + small + 2.0 ** -8 * np.abs(ref["O"][b, c])
            err = np.abs(got[b, c] - ref["O"][b, c])
            assert np.all(err <= bound), (b, h, float((err - bound).max()), float(err.max()))
            assert abs(lse[b, h] - ref["lse"][h, b]) <= e + n * 2.0 ** -24 + 2.0 ** -22 * (abs(ref["lse"][h, b]) + 16)


CASES = {
    # lens, page, n_q, n_kv, values of very different sizes, std of Q
    "one_token": ([1], 16, 2, 2, False, 1.0),
    "page_ends": ([16, 17, 31, 32, 33], 16, 4, 2, False, 1.0),
    "unit_ends": ([127, 128, 129, 255, 257], 64, 8, 1, True, 1.0),
    "empty_among": ([0, 5, 0, 300, 0], 32, 6, 2, True, 1.0),
    "all_empty": ([0, 0], 16, 4, 4, False, 1.0),
    "group_of_16": ([77, 400], 64, 32, 2, True, 1.0),
    "group_of_40": ([50, 290], 64, 40, 1, True, 1.0),
    "odd_group": ([513], 128, 7, 1, True, 1.0),
    "split_over_ctas": ([9000], 256, 8, 1, True, 1.0),
    "peaked": ([700, 90], 64, 8, 2, True, 60.0),
    "flat": ([700, 90], 64, 8, 2, True, 0.0),
    "tiny_q": ([300], 64, 4, 1, False, 2.0 ** -40),
    "many": (list(range(1, 60)), 16, 8, 8, False, 1.0),
    "more_than_threads": ([(7 * i) % 41 for i in range(400)], 16, 2, 1, True, 1.0),
}


@pytest.mark.parametrize("name", CASES)
def test_decode(coda, name):
    lens, page, n_q, n_kv, spread, std = CASES[name]
    cache, table, kval, vval, vs = fill(coda, lens, page, n_kv, spread)
    Q = synth.randn_bf16((len(lens), n_q * D), std, 99)
    ws = coda.workspace(coda.load().coda_attention_decode_nvfp4_workspace_size(len(lens), n_q, n_kv, D))
    out = coda.attention_decode_nvfp4(Q.to(DEV), cache, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                                      n_q, ws=ws)
    assert coda.get_status(ws) == 0
    check_decode(out, to_np(Q), lens, kval, vval, vs, n_q, n_kv, D ** -0.5)


def test_decode_bad_lengths_and_pages_set_status(coda):
    n_q, n_kv, page, lens = 4, 2, 16, [40, 20, 33]
    cache, table, kval, vval, vs = fill(coda, lens, page, n_kv, False)
    Q = synth.randn_bf16((3, n_q * D), 1.0, 5)
    ws = coda.workspace(coda.load().coda_attention_decode_nvfp4_workspace_size(3, n_q, n_kv, D))

    def run(tab, n):
        return coda.attention_decode_nvfp4(Q.to(DEV), cache, tab.to(DEV), torch.tensor(n, dtype=torch.int32, device=DEV),
                                           n_q, ws=ws)
    for bad in (-1, table.shape[1] * page + 1):
        out = run(table, [40, bad, 33])
        assert coda.get_status(ws) == 9                  # CODA_ERR_SEQLEN_RANGE
        coda.reset_status(ws)
        check_decode(out, to_np(Q), [40, 0, 33], [kval[0], kval[1][:0], kval[2]], [vval[0], vval[1][:0], vval[2]],
                     [vs[0], vs[1][:0], vs[2]], n_q, n_kv, D ** -0.5)
    for bad in (-1, cache["scale"].shape[0]):
        tab = table.clone()
        tab[0, 1] = bad                                  # keys 16 .. 31 of sequence 0 are left out
        out = run(tab, lens)
        assert coda.get_status(ws) == 10                 # CODA_ERR_PAGE_RANGE
        coda.reset_status(ws)
        keep = np.r_[0:16, 32:40]
        check_decode(out, to_np(Q), [24, 20, 33], [kval[0][keep], kval[1], kval[2]],
                     [vval[0][keep], vval[1], vval[2]], [vs[0][keep], vs[1], vs[2]], n_q, n_kv, D ** -0.5)


def test_decode_offsets_beyond_32_bits(coda):
    """Rows whose byte offsets pass 2^32: pages at the end of a large cache."""
    n_q, n_kv, page = 8, 8, 256
    pages = (1 << 32) // (2 * n_kv * page * 64) + 40     # codes alone pass 4 GiB
    cache = {"codes": torch.zeros(pages, 2, n_kv, page, 64, dtype=torch.uint8, device=DEV),
             "sf": torch.zeros(pages, 2, n_kv, page, 8, dtype=torch.uint8, device=DEV),
             "scale": torch.zeros(pages, 2, n_kv, page, device=DEV)}
    lens = [300]
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32)
    j = torch.arange(300)
    slots = (table[0][j // page].long() * page + j % page).to(torch.int32)
    K, V = rows(300, n_kv, 1, False), rows(300, n_kv, 2)
    coda.kv_append_nvfp4(K.to(DEV), V.to(DEV), slots.to(DEV), cache)
    Q = synth.randn_bf16((1, n_q * D), 1.0, 5)
    out = coda.attention_decode_nvfp4(Q.to(DEV), cache, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), n_q)
    back = coda.kv_read_nvfp4(cache, slots.to(DEV), dtype=torch.float32)
    (_, _, _, kv), (_, _, sc, vv) = oracle_rows(K, n_kv), oracle_rows(V, n_kv)
    assert torch.equal(back["K"].cpu(), torch.from_numpy(kv).float())
    check_decode(out, to_np(Q), lens, [kv], [vv], [sc], n_q, n_kv, D ** -0.5)


def test_decode_twice_gives_the_same_bits(coda):
    lens = [5000, 3, 700]
    cache, table, *_ = fill(coda, lens, 64, 2, True)
    Q = synth.randn_bf16((3, 8 * D), 1.0, 5).to(DEV)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    a = coda.attention_decode_nvfp4(Q, cache, table.to(DEV), n, 8)
    b = coda.attention_decode_nvfp4(Q, cache, table.to(DEV), n, 8)
    assert torch.equal(a["O"], b["O"]) and torch.equal(a["lse"], b["lse"])


def test_binding_refuses_shapes(coda):
    cache = coda.kv_cache_nvfp4(2, 16, 2)
    slots = torch.zeros(3, dtype=torch.int32, device=DEV)
    x = torch.zeros(3, 2 * D, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="cache sf"):
        coda.kv_read_nvfp4(dict(cache, sf=cache["sf"][:1]), slots)
    with pytest.raises(ValueError, match="slots"):
        coda.kv_append_nvfp4(x, x, slots[:2], cache)
    with pytest.raises(TypeError, match="slots"):
        coda.kv_append_nvfp4(x, x, slots.long(), cache)
    with pytest.raises(ValueError, match="K: expected"):
        coda.kv_append_nvfp4(x[:, :D], x, slots, cache)
    q = torch.zeros(3, 4 * D, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="block_table"):
        coda.attention_decode_nvfp4(q, cache, torch.zeros(2, 2, dtype=torch.int32, device=DEV), slots, 4)
    with pytest.raises(ValueError, match="workspace too small"):
        coda.attention_decode_nvfp4(q, cache, torch.zeros(3, 2, dtype=torch.int32, device=DEV), slots, 4,
                                    ws=coda.workspace(256))
    with pytest.raises(coda.CodaError):                 # 5 query heads over 2 key/value heads
        coda.attention_decode_nvfp4(torch.zeros(3, 5 * D, dtype=torch.bfloat16, device=DEV), cache,
                                    torch.zeros(3, 2, dtype=torch.int32, device=DEV), slots, 5)


def test_decode_in_a_graph_and_on_two_streams(coda):
    """A captured append and decode reads the lengths and pages of its replay;
    two streams with a workspace each give the bits of one; sequences may share
    pages."""
    lens, page, n_q, n_kv = [300, 41, 1000], 64, 8, 2
    cache, table, *_ = fill(coda, lens, page, n_kv, True)
    table[1, 0] = table[0, 0]                            # a shared first page
    tab, n = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    Q = synth.randn_bf16((3, n_q * D), 1.0, 5).to(DEV)
    K, V = rows(1, n_kv, 21).to(DEV), rows(1, n_kv, 22).to(DEV)
    slot = (tab[0, 4] * page + 44).reshape(1).to(torch.int32)      # sequence 0's token 300
    size = coda.load().coda_attention_decode_nvfp4_workspace_size(3, n_q, n_kv, D)
    ws = [coda.workspace(size) for _ in range(2)]
    before = coda.attention_decode_nvfp4(Q, cache, tab, n, n_q, ws=ws[0])
    out = {k: torch.zeros_like(v) for k, v in before.items()}
    cap = torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=cap):
        coda.kv_append_nvfp4(K, V, slot, cache, ws=ws[0])
        coda.attention_decode_nvfp4(Q, cache, tab, n, n_q, out=out, ws=ws[0])
    g.replay()                                           # the token is there, the lengths do not name it
    torch.cuda.synchronize()
    assert all(torch.equal(out[k], before[k]) for k in out)
    n[0] += 1
    g.replay()
    torch.cuda.synchronize()
    after = coda.attention_decode_nvfp4(Q, cache, tab, n, n_q, ws=ws[0])
    torch.cuda.synchronize()
    assert all(torch.equal(out[k], after[k]) for k in out) and not torch.equal(after["O"][0], before["O"][0])
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[coda.attention_decode_nvfp4(Q, cache, tab, n, n_q, ws=w, stream=s) for w, s in zip(ws, side)]
           for _ in range(5)]
    torch.cuda.synchronize()
    for pair in got:
        for one in pair:
            assert all(torch.equal(one[k], after[k]) for k in after)
    assert coda.get_status(ws[0]) == 0 and coda.get_status(ws[1]) == 0


def test_append_takes_the_quantiser_s_codes_of_any_number(coda):
    """Infinities, NaN, the smallest and largest numbers and zeros of both
    signs: the cached codes and row scales are quantize_nvfp4_rows' own."""
    n_kv = 2
    K = rows(8, n_kv, 3).float()
    K[0, 3], K[1, 130], K[2, :] = float("inf"), float("nan"), float("-inf")
    K[3, :] = torch.finfo(torch.bfloat16).max
    K[4, :] = 1e-40
    K[5, :] = -0.0
    K[6, ::2] = 2.0 ** -133
    K = K.to(torch.bfloat16).to(DEV)
    cache = coda.kv_cache_nvfp4(1, 16, n_kv)
    slots = torch.arange(8, dtype=torch.int32, device=DEV)
    coda.kv_append_nvfp4(K, K, slots, cache)
    codes, _, scale = coda.quantize_nvfp4_rows(K.view(8 * n_kv, D))
    for plane in range(2):
        got = cache["codes"][0, plane, :, :8].transpose(0, 1).reshape(8 * n_kv, 64)
        assert torch.equal(got, codes)
        sc = cache["scale"][0, plane, :, :8].transpose(0, 1).reshape(8 * n_kv)
        assert torch.equal(sc.view(torch.int32), scale.view(torch.int32))
    # a slot may be read twice
    twice = coda.kv_read_nvfp4(cache, slots[[3, 3, 7]], dtype=torch.float32)
    assert torch.equal(twice["K"][0], twice["K"][1]) and torch.equal(twice["K"][2], twice["V"][2])


def test_decode_non_finite_numbers_stay_in_their_sequence(coda):
    """NaN and infinities in one sequence's query, keys or values: the others
    keep their bits, and the sequence's own result is NaN."""
    lens, page, n_q, n_kv = [150, 700, 90], 32, 8, 2
    Q = synth.randn_bf16((3, n_q * D), 1.0, 5)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    cache, table, *_ = fill(coda, lens, page, n_kv, True)
    clean = coda.attention_decode_nvfp4(Q.to(DEV), cache, table.to(DEV), n, n_q)
    assert bool(torch.isfinite(clean["O"].float()).all())
    bad_q = Q.clone()
    bad_q[1, 5] = float("nan")
    got = coda.attention_decode_nvfp4(bad_q.to(DEV), cache, table.to(DEV), n, n_q)
    for k in got:
        assert torch.equal(got[k][[0, 2]], clean[k][[0, 2]]), k
    assert bool(torch.isnan(got["O"][1, :D].float()).all()) and bool(torch.isnan(got["lse"][1, 0]))
    # the other heads: those of the same key/value head may renew their units elsewhere
    assert torch.equal(got["O"][1, 4 * D:], clean["O"][1, 4 * D:])
    assert bool(torch.isfinite(got["O"][1, D:].float()).all())
    for plane, value in ((0, float("nan")), (0, float("inf")), (1, float("nan")), (1, float("inf"))):
        hurt = {k: v.clone() for k, v in cache.items()}
        hurt["scale"][int(table[1, 20]), plane, :, 7] = value           # key 647 of the second sequence
        got = coda.attention_decode_nvfp4(Q.to(DEV), hurt, table.to(DEV), n, n_q)
        for k in got:
            assert torch.equal(got[k][[0, 2]], clean[k][[0, 2]]), (plane, value, k)
        assert not bool(torch.isfinite(got["O"][1].float()).any()) or plane == 0


def test_decode_without_pages_and_with_an_own_scale(coda):
    n_q, n_kv = 4, 2
    Q = synth.randn_bf16((2, n_q * D), 1.0, 5)
    cache, table, kval, vval, vs = fill(coda, [40, 7], 16, n_kv, False)
    none = coda.attention_decode_nvfp4(Q.to(DEV), cache, torch.zeros(2, 0, dtype=torch.int32, device=DEV),
                                       torch.zeros(2, dtype=torch.int32, device=DEV), n_q)
    assert torch.all(none["O"] == 0) and bool(torch.isneginf(none["lse"]).all())
    out = coda.attention_decode_nvfp4(Q.to(DEV), cache, table.to(DEV),
                                      torch.tensor([40, 7], dtype=torch.int32, device=DEV), n_q, scale=0.3)
    check_decode(out, to_np(Q), [40, 7], kval, vval, vs, n_q, n_kv, 0.3)


def shared_rows(coda, K, V, lens, page, n_kv):
    """Sequences of `lens` tokens that all begin with the same rows K, V: as
    fill(), with the row scales of value rows that hold only zeros taken as 0
    (such a row adds nothing to O, so the bound has no use for its scale of 1)."""
    n = K.shape[0]
    pages = -(-n // page)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(4)).to(torch.int32)
    j = torch.arange(n)
    cache = coda.kv_cache_nvfp4(pages, page, n_kv)
    coda.kv_append_nvfp4(K.to(DEV), V.to(DEV), (order[j // page] * page + j % page).to(torch.int32).to(DEV), cache)
    kval, (vval, vs) = oracle_rows(K, n_kv)[3], (oracle_rows(V, n_kv)[i] for i in (3, 2))
    vs = np.where(np.abs(vval).reshape(n, n_kv, D).max(axis=2) > 0, vs, 0)
    return cache, order.repeat(len(lens), 1), [kval[:m] for m in lens], [vval[:m] for m in lens], [vs[:m] for m in lens]


def run_shared(coda, K, V, lens, page, Q, n_q, n_kv):
    cache, table, kval, vval, vs = shared_rows(coda, K, V, lens, page, n_kv)
    out = coda.attention_decode_nvfp4(Q.to(DEV), cache, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), n_q)
    check_decode(out, to_np(Q), lens, kval, vval, vs, n_q, n_kv, D ** -0.5)
    return out


@pytest.mark.parametrize("n_q, n_kv", [(8, 1), (16, 1), (4, 2)])
@pytest.mark.parametrize("std", [1.0, 1e-3, 1e-5, 1e-20])
def test_decode_value_rows_of_zeros(coda, std, n_q, n_kv):
    """Value rows of zeros (row scale 1) among small values, in front, in
    between, at the end, over whole units and with by far the largest weight:
    within the bound that rows without them meet."""
    base = synth.randn_bf16((1, D), 1.0, 31).float()
    K = synth.randn_bf16((700, n_kv * D), 0.3, 32)
    V = synth.randn_bf16((700, n_kv * D), std, 33)
    V[[0, 1, 39, 100, 159, 699]] = 0
    V[200:330] = 0
    K[100] = base.repeat(1, n_kv)[0].to(torch.bfloat16)
    lens = [1, 2, 40, 160, 331, 700] * 40
    Q = (base.repeat(len(lens), n_q) + 0.2 * synth.randn_bf16((len(lens), n_q * D), 1.0, 34).float()).to(torch.bfloat16)
    out = run_shared(coda, K, V, lens, 64, Q, n_q, n_kv)
    assert torch.all(out["O"][::6] == 0) and torch.all(out["O"][1::6] == 0) and bool(torch.isfinite(out["lse"]).all())


@pytest.mark.parametrize("n_q, n_kv", [(8, 1), (16, 1)])
@pytest.mark.parametrize("std", [1e-30, 1e-33, 1e-34, 1e-35])
def test_decode_smallest_values_behind_rising_scores(coda, std, n_q, n_kv):
    """Scores that rise late by 2^12 and more over values near the end of
    fp32's range: keys in front keep their small weights."""
    base = synth.randn_bf16((1, D), 1.0, 41).float()
    rise = torch.zeros(420, 1)
    rise[230:], rise[400:] = 0.73, 1.3                   # 2^12 and 2^21 at |base|^2 = 128
    K = (rise * base + 0.02 * synth.randn_bf16((420, D), 1.0, 42).float()).to(torch.bfloat16)
    V = synth.randn_bf16((420, D), std, 43)
    lens = [420, 380, 256, 131] * 100
    Q = (base.repeat(len(lens), n_q) + 0.1 * synth.randn_bf16((len(lens), n_q * D), 1.0, 44).float()).to(torch.bfloat16)
    run_shared(coda, K, V, lens, 64, Q, n_q, n_kv)
