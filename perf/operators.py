"""Workloads of the attention operators: causal attention over packed prompts
(forward, and forward + backward as a training step runs them), the 4-bit
key/value cache (append and read back) and single-token attention over it.

``own`` selects what ``run`` computes with: the plain form of each operator in
elementary torch operations, or the framework's own calls.  ``exact`` gives
the same outputs from the definitions in 64 bits.

Heads are 128 wide, as everywhere in the framework.  The key/value cache holds
NVFP4 rows: e2m1 codes (two per byte), an e4m3 scale per 16 elements and an
fp32 scale per row of 128; page p, plane 0 (keys) or 1 (values), kv head h,
offset o is row [p, plane, h, o] of its three tensors.
"""
import math
import random

import torch

own = False

D = 128
CHUNK_BYTES = 4 << 30   # score matrices held at once by the plain form


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # forward over prompts.  Many short requests (chat turns, scoring) in one call: launch latency counts
        dict(name="prompt_short", op="fwd", q="ragged:48:1:60:3", k="", n_q=16, n_kv=2, pad=13, packed=False),
        # one packed batch of very different requests, Q | K | V columns of one projection output, padded rows behind
        dict(name="prompt_ragged", op="fwd", q="1,17,300,1023,64,2047,129,0,777,1500", k="", n_q=32, n_kv=8, pad=70,
             packed=True),
        # the block's batch: 8192 tokens as four sequences of 2048, 64 + 8 heads
        dict(name="prompt_block", op="fwd", q="2048*4", k="", n_q=64, n_kv=8, pad=0, packed=False),
        # one long document
        dict(name="prompt_long", op="fwd", q="16384", k="", n_q=32, n_kv=8, pad=0, packed=False),
        # prompts continued from cached prefixes (a chunk of new tokens each, odd key lengths)
        dict(name="prompt_chunk", op="fwd", q="512,512,200,1", k="4096,1537,3801,2049", n_q=64, n_kv=8, pad=0,
             packed=False),
        # training step (forward + backward) on the block's batch
        dict(name="train_block", op="train", q="2048*4", k="", n_q=64, n_kv=8, pad=0, packed=False),
        # training step on packed documents of odd lengths, three query heads a kv head, padded rows behind
        dict(name="train_ragged", op="train", q="1,33,700,255,1911,128,480", k="", n_q=12, n_kv=4, pad=84,
             packed=False),
        # a prefilled prompt batch goes to the cache and is read back (prefix reuse)
        dict(name="cache_prompt", op="cache", tokens=8192, pages=768, page=64, n_kv=8),
        # one decode step's new tokens
        dict(name="cache_step", op="cache", tokens=61, pages=512, page=16, n_kv=8),
        # decode: one request, short context
        dict(name="decode_small", op="decode", lens="777", page=64, n_q=64, n_kv=8),
        # decode: a serving batch of mixed contexts, an empty one among them
        dict(name="decode_batch", op="decode", lens="0,ragged:127:1:8192:5", page=64, n_q=64, n_kv=8),
        # decode: few requests, very long contexts
        dict(name="decode_long", op="decode", lens="131072,100001,131071,98304", page=256, n_q=32, n_kv=8),
    ]


def draw(rng):
    most = max(_flops(c) for c in listed())
    kind = rng.choice(["fwd", "fwd", "train", "train", "cache", "decode", "decode"])
    n_kv = rng.choice([1, 2, 4, 8])
    n_q = n_kv * rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 16) if g * n_kv <= 64])
    if kind == "cache":
        page = rng.choice([16, 32, 64, 128, 256])
        tokens = _log(rng, 1, 8192)
        return dict(op="cache", tokens=tokens, pages=-(-tokens // page) + rng.randint(0, 64), page=page, n_kv=n_kv)
    if kind == "decode":
        batch = _log(rng, 1, 128)
        top = _log(rng, 1, min(131072, 1000000 // batch))
        return dict(op="decode", lens="ragged:%d:%d:%d:%d" % (batch, rng.randint(0, min(top, 3)), top,
                                                             rng.randrange(1 << 20)),
                    page=rng.choice([16, 32, 64, 128, 256]), n_q=n_q, n_kv=n_kv)
    while True:
        n = _log(rng, 1, 32)
        lq = [_log(rng, 1, 8192 // n) for _ in range(n)]
        chunk = kind == "fwd" and rng.random() < 0.4
        lk = [x + _log(rng, 1, 4096) - 1 for x in lq] if chunk else []
        case = dict(op=kind, q=",".join(map(str, lq)), k=",".join(map(str, lk)), n_q=n_q, n_kv=n_kv,
                    pad=rng.choice([0, 0, 1, 37, 200]), packed=not chunk and rng.random() < 0.3)
        if _flops(case) <= most:
            return case


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _lens(text):
    out = []
    for part in filter(None, text.split(",")):
        if part.startswith("ragged:"):
            n, lo, hi, seed = (int(x) for x in part[7:].split(":"))
            r = random.Random(seed)
            out += [r.randint(lo, hi) for _ in range(n)]
        elif "*" in part:
            v, n = part.split("*")
            out += [int(v)] * int(n)
        else:
            out.append(int(part))
    return out


def _pairs(lq, lk):
    """(query, key) pairs that the causal mask leaves."""
    total = 0
    for a, b in zip(lq, lk):
        first = b - a + 1                      # keys of query 0
        skip = max(0, min(a, 1 - first))       # queries without any key
        n = a - skip
        total += n * (first + skip) + n * (n - 1) // 2
    return total


def _flops(case):
    if case["op"] in ("fwd", "train"):
        lq = _lens(case["q"])
        return (4 if case["op"] == "fwd" else 14) * D * case["n_q"] * _pairs(lq, _lens(case["k"]) or lq)
    return 0


def work(case):
    """Bytes: each input read once, each output written once; flops: the
    products over the pairs that the mask leaves."""
    n_kv = case["n_kv"]
    if case["op"] == "cache":
        rows = 2 * case["tokens"] * n_kv
        return {"bytes": rows * (D * 2 + 76 + D * 4) + case["tokens"] * 4, "flops": 0}
    n_q = case["n_q"]
    if case["op"] == "decode":
        lens = _lens(case["lens"])
        return {"bytes": sum(lens) * n_kv * 152 + len(lens) * n_q * (D * 4 + 4), "flops": 4 * D * n_q * sum(lens)}
    tq = sum(_lens(case["q"]))
    tk = sum(_lens(case["k"])) if case["k"] else tq
    fwd = (2 * tq * n_q + 2 * tk * n_kv) * D * 2 + tq * n_q * 4
    back = (tq * n_q * 2 + 2 * tk * n_kv) * D * 2           # dO, dQ, dK, dV
    return {"bytes": fwd + (back if case["op"] == "train" else 0), "flops": _flops(case)}


# --------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _cu(lens):
    c = [0]
    for x in lens:
        c.append(c[-1] + x)
    return torch.tensor(c, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    n_kv = case["n_kv"]
    if case["op"] in ("fwd", "train"):
        # queries and keys leave per-head RMSNorm: unit entries; values are a projection's output
        lq = _lens(case["q"])
        lk = _lens(case["k"]) or lq
        tq, tk = sum(lq) + case["pad"], sum(lk) + (0 if case["k"] else case["pad"])
        n_q = case["n_q"]
        if case["packed"]:
            qkv = torch.randn(tq, (n_q + 2 * n_kv) * D, generator=g, device="cuda").to(torch.bfloat16)
            st["Q"], st["K"], st["V"] = qkv.split([n_q * D, n_kv * D, n_kv * D], dim=1)
        else:
            st["Q"] = torch.randn(tq, n_q * D, generator=g, device="cuda").to(torch.bfloat16)
            st["K"] = torch.randn(tk, n_kv * D, generator=g, device="cuda").to(torch.bfloat16)
            st["V"] = torch.randn(tk, n_kv * D, generator=g, device="cuda").to(torch.bfloat16)
        st["lq"], st["lk"] = lq, lk
        st["cu"] = _cu(lq)
        st["cu_k"] = _cu(lk) if case["k"] else None
        # rows behind the last sequence belong to the caller and stay zero
        st["out"] = {"O": torch.zeros(tq, n_q * D, dtype=torch.bfloat16, device="cuda"),
                     "lse": torch.zeros(n_q, tq, dtype=torch.float32, device="cuda")}
        if case["op"] == "train":
            st["dO"] = torch.randn(tq, n_q * D, generator=g, device="cuda").to(torch.bfloat16)
            st["grads"] = {"dQ": torch.zeros(tq, n_q * D, dtype=torch.bfloat16, device="cuda"),
                           "dK": torch.zeros(tk, n_kv * D, dtype=torch.bfloat16, device="cuda"),
                           "dV": torch.zeros(tk, n_kv * D, dtype=torch.bfloat16, device="cuda")}
        if own:
            import gemm_epilogue_transformer_bf16_gb300 as coda
            lib = coda.load()
            need = lib.coda_attention_workspace_size(tq, tk, len(lq), n_q, n_kv, D)
            if case["op"] == "train":
                need = max(need, lib.coda_attention_bwd_workspace_size(tq, tk, len(lq), n_q, n_kv, D))
            st["ws"] = coda.workspace(need)
        return st
    page = case["page"]
    if case["op"] == "cache":
        pages = case["pages"]
        t = case["tokens"]
        st["K"] = torch.randn(t, n_kv * D, generator=g, device="cuda").to(torch.bfloat16)
        spread = torch.exp(torch.randn(1, n_kv * D, generator=g, device="cuda"))
        st["V"] = (torch.randn(t, n_kv * D, generator=g, device="cuda") * spread).to(torch.bfloat16)
        st["slots"] = torch.randperm(pages * page, generator=g, device="cuda")[:t].to(torch.int32)
        st["cache"] = {"codes": torch.zeros(pages, 2, n_kv, page, D // 2, dtype=torch.uint8, device="cuda"),
                       "sf": torch.zeros(pages, 2, n_kv, page, D // 16, dtype=torch.uint8, device="cuda"),
                       "scale": torch.zeros(pages, 2, n_kv, page, dtype=torch.float32, device="cuda")}
        if own:
            import gemm_epilogue_transformer_bf16_gb300 as coda
            st["ws"] = coda.workspace(256)
        return st
    lens = _lens(case["lens"])
    need = [-(-x // page) for x in lens]
    pages = sum(need) + 3
    st["cache"] = {"codes": torch.empty(pages, 2, n_kv, page, D // 2, dtype=torch.uint8, device="cuda"),
                   "sf": torch.empty(pages, 2, n_kv, page, D // 16, dtype=torch.uint8, device="cuda"),
                   "scale": torch.empty(pages, 2, n_kv, page, dtype=torch.float32, device="cuda")}
    step = max(1, (1 << 26) // (2 * n_kv * page * D))
    for p in range(0, pages, step):
        x = torch.randn(min(step, pages - p), 2, n_kv, page, D, generator=g, device="cuda").to(torch.bfloat16)
        q, sf, sc = _quantise(x)
        for name, part in (("codes", q), ("sf", sf), ("scale", sc)):
            st["cache"][name][p:p + part.shape[0]] = part
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    st["table"] = table
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["host_lens"] = lens
    st["Q"] = torch.randn(len(lens), case["n_q"] * D, generator=g, device="cuda").to(torch.bfloat16)
    if own:
        import gemm_epilogue_transformer_bf16_gb300 as coda
        lib = coda.load()
        st["ws"] = coda.workspace(lib.coda_attention_decode_nvfp4_workspace_size(len(lens), case["n_q"], n_kv, D))
    return st


# --------------------------------------------------------------------------- plain forms

def _quantise(x):
    """NVFP4 rows of x [..., 128] (bf16): packed codes [..., 64], e4m3 block
    scales [..., 8] as bytes, fp32 row scales [...].  Every step is one fp32
    operation; e2m1 and e4m3 round to nearest, ties to even."""
    x = x.float()
    amax = x.abs().amax(-1)
    # tensor by tensor: a division by a Python number is a product with its rounded inverse
    s = torch.where(amax > 0, amax / torch.full_like(amax, 2688.0), torch.ones_like(amax))
    xb = x.unflatten(-1, (D // 16, 16))
    sf = (xb.abs().amax(-1) / (6.0 * s).unsqueeze(-1)).clamp(max=448.0).to(torch.float8_e4m3fn)
    denom = sf.float() * s.unsqueeze(-1)
    inv = (1.0 / denom).clamp(max=torch.finfo(torch.float32).max)
    a = (xb * inv.unsqueeze(-1)).abs()
    # halfway values go to the even code: (0.25, 0.75) are 0.5, 1 up, and so on
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = torch.where((denom == 0).unsqueeze(-1), torch.zeros_like(code), code)
    code = code | ((xb < 0) & (code > 0)).to(torch.uint8) << 3
    code = code.flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, sf.view(torch.uint8), s


def _values(codes, sf, scale, dtype):
    """What cache rows stand for: [..., 128] in `dtype`."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=dtype, device=codes.device)
    v = torch.stack((grid[(codes & 15).long()], grid[(codes >> 4).long()]), -1).flatten(-2)
    v = v.unflatten(-1, (D // 16, 16)) * sf.view(torch.float8_e4m3fn).to(dtype).unsqueeze(-1)
    return v.flatten(-2) * scale.to(dtype).unsqueeze(-1)


def _spans(st):
    q0 = k0 = 0
    for a, b in zip(st["lq"], st["lk"]):
        yield q0, a, k0, b
        q0, k0 = q0 + a, k0 + b


def _probabilities(q, k, scale, off):
    """q [h, g, a, D], k [h, b, D] fp32: masked softmax numerators' parts."""
    s = torch.matmul(q.flatten(1, 2), k.transpose(1, 2)).unflatten(1, q.shape[1:3]) * scale
    a, b = s.shape[-2:]
    i = torch.arange(a, device=q.device).unsqueeze(1)
    j = torch.arange(b, device=q.device).unsqueeze(0)
    s = s.masked_fill(j > i + off, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1)
    return p / torch.where(total == 0, torch.ones_like(total), total), lse


def _plain_prompt(st):
    case = st["case"]
    n_q, n_kv = case["n_q"], case["n_kv"]
    g = n_q // n_kv
    scale = 1.0 / math.sqrt(D)
    train = case["op"] == "train"
    out = {k: torch.zeros_like(v) for k, v in st["out"].items()}
    if train:
        out.update({k: torch.zeros_like(v) for k, v in st["grads"].items()})
    for q0, a, k0, b in _spans(st):
        if a == 0 or b == 0:
            out["lse"][:, q0:q0 + a] = -math.inf
            continue
        step = max(1, min(n_kv, CHUNK_BYTES // (4 * g * a * b)))
        for h in range(0, n_kv, step):
            e = min(n_kv, h + step)
            q = st["Q"][q0:q0 + a, h * g * D:e * g * D].float().view(a, e - h, g, D).permute(1, 2, 0, 3)
            k = st["K"][k0:k0 + b, h * D:e * D].float().view(b, e - h, D).transpose(0, 1)
            v = st["V"][k0:k0 + b, h * D:e * D].float().view(b, e - h, D).transpose(0, 1)
            p, lse = _probabilities(q, k, scale, b - a)
            o = torch.matmul(p.flatten(1, 2), v).unflatten(1, (g, a))
            out["O"][q0:q0 + a, h * g * D:e * g * D] = o.permute(2, 0, 1, 3).flatten(1).to(torch.bfloat16)
            out["lse"][h * g:e * g, q0:q0 + a] = lse.flatten(0, 1)
            if train:
                do = st["dO"][q0:q0 + a, h * g * D:e * g * D].float().view(a, e - h, g, D).permute(1, 2, 0, 3)
                dp = torch.matmul(do.flatten(1, 2), v.transpose(1, 2)).unflatten(1, (g, a))
                ds = p * (dp - (do * o).sum(-1, keepdim=True)) * scale
                dq = torch.matmul(ds.flatten(1, 2), k).unflatten(1, (g, a))
                dk = torch.matmul(ds.flatten(1, 2).transpose(1, 2), q.flatten(1, 2))
                dv = torch.matmul(p.flatten(1, 2).transpose(1, 2), do.flatten(1, 2))
                out["dQ"][q0:q0 + a, h * g * D:e * g * D] = dq.permute(2, 0, 1, 3).flatten(1).to(torch.bfloat16)
                out["dK"][k0:k0 + b, h * D:e * D] = dk.transpose(0, 1).flatten(1).to(torch.bfloat16)
                out["dV"][k0:k0 + b, h * D:e * D] = dv.transpose(0, 1).flatten(1).to(torch.bfloat16)
    return out


def _plain_cache(st):
    cache, slots = st["cache"], st["slots"].long()
    page, n_kv = st["case"]["page"], st["case"]["n_kv"]
    pg, off = slots // page, slots % page
    got = {}
    for plane, name in enumerate(("K", "V")):
        parts = _quantise(st[name].view(-1, n_kv, D))
        for key, part in zip(("codes", "sf", "scale"), parts):
            cache[key][pg, plane, :, off] = part
        got[name] = _values(cache["codes"][pg, plane, :, off], cache["sf"][pg, plane, :, off],
                            cache["scale"][pg, plane, :, off], torch.float32).flatten(1)
    return got


def _plain_decode(st):
    case, cache = st["case"], st["cache"]
    n_q, n_kv, page = case["n_q"], case["n_kv"], case["page"]
    g = n_q // n_kv
    batch, scale = len(st["host_lens"]), 1.0 / math.sqrt(D)
    O = torch.empty(batch, n_q * D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(batch, n_q, dtype=torch.float32, device="cuda")
    width = max(-(-max(st["host_lens"]) // page), 1)
    step = max(1, CHUNK_BYTES // (width * page * n_kv * D * 4))
    for b in range(0, batch, step):
        e = min(batch, b + step)
        t = st["table"][b:e, :width].long().clamp(min=0)
        kv = [_values(cache["codes"][t, i], cache["sf"][t, i], cache["scale"][t, i], torch.float32)
              .permute(0, 2, 1, 3, 4).flatten(2, 3) for i in (0, 1)]            # [b, h, keys, D]
        q = st["Q"][b:e].float().view(e - b, n_kv, g, D)
        s = torch.matmul(q, kv[0].transpose(2, 3)) * scale
        j = torch.arange(width * page, device="cuda")
        s = s.masked_fill(j >= st["lens"][b:e].view(-1, 1, 1, 1), -math.inf)
        m = s.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, torch.zeros_like(m), m)
        p = torch.exp(s - m)
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p, kv[1]) / torch.where(total == 0, torch.ones_like(total), total)
        O[b:e] = o.flatten(1).to(torch.bfloat16)
        lse[b:e] = (m + torch.log(total)).flatten(1)
    return {"O": O, "lse": lse}


# --------------------------------------------------------------------------- one pass

def run(st):
    case = st["case"]
    if not own:
        return {"fwd": _plain_prompt, "train": _plain_prompt, "cache": _plain_cache, "decode": _plain_decode}[case["op"]](st)
    import gemm_epilogue_transformer_bf16_gb300 as coda
    if case["op"] == "cache":
        coda.kv_append_nvfp4(st["K"], st["V"], st["slots"], st["cache"], ws=st["ws"])
        return coda.kv_read_nvfp4(st["cache"], st["slots"], dtype=torch.float32, ws=st["ws"])
    if case["op"] == "decode":
        return coda.attention_decode_nvfp4(st["Q"], st["cache"], st["table"], st["lens"], case["n_q"], ws=st["ws"])
    f = coda.attention(st["Q"], st["K"], st["V"], st["cu"], case["n_q"], case["n_kv"], cu_seqlens_k=st["cu_k"],
                       out=st["out"], ws=st["ws"])
    if case["op"] == "fwd":
        return f
    b = coda.attention_bwd(st["dO"], st["Q"], st["K"], st["V"], f["O"], f["lse"], st["cu"], case["n_q"], case["n_kv"],
                           out=st["grads"], ws=st["ws"])
    return {**f, **b}


# --------------------------------------------------------------------------- 64 bits

def _exact_head(q, k, v, scale):
    """One head from the definition: softmax over the visible keys."""
    a, b = q.shape[0], k.shape[0]
    seen = torch.ones(a, b, dtype=torch.bool, device=q.device).tril(b - a)
    w = torch.einsum("id,jd->ij", q, k).mul(scale).where(seen, torch.full((), -math.inf, dtype=q.dtype, device=q.device))
    lse = torch.logsumexp(w, 1)
    p = torch.exp(w - lse.clamp(min=-1e300).unsqueeze(1))
    return torch.einsum("ij,jd->id", p, v), lse


def _exact_prompt(case, st):
    if _flops(case) * (1 if case["op"] == "fwd" else 2) > 6e12:
        return None
    n_q, n_kv = case["n_q"], case["n_kv"]
    train = case["op"] == "train"
    out = {k: torch.zeros(v.shape, dtype=torch.float64, device="cuda")
           for k, v in {**st["out"], **(st["grads"] if train else {})}.items()}
    for q0, a, k0, b in _spans(st):
        for h in range(n_q):
            kv = h // (n_q // n_kv)
            cols, kcols = slice(h * D, h * D + D), slice(kv * D, kv * D + D)
            if a == 0:
                continue
            if b == 0:
                out["lse"][h, q0:q0 + a] = -math.inf
                continue
            x = [st["Q"][q0:q0 + a, cols].double(), st["K"][k0:k0 + b, kcols].double(), st["V"][k0:k0 + b, kcols].double()]
            for t in x:
                t.requires_grad_(train)
            o, lse = _exact_head(*x, 1.0 / math.sqrt(D))
            out["O"][q0:q0 + a, cols] = o.detach()
            out["lse"][h, q0:q0 + a] = lse.detach()
            if train:
                dq, dk, dv = torch.autograd.grad(o, x, st["dO"][q0:q0 + a, cols].double())
                out["dQ"][q0:q0 + a, cols] = dq
                out["dK"][k0:k0 + b, kcols] += dk
                out["dV"][k0:k0 + b, kcols] += dv
    return out


def _exact_rows(x):
    """The values NVFP4 rows of x [rows, 128] stand for.  The format's scales
    are fp32 and e4m3 numbers, so each is rounded to its own format here; the
    codes are the nearest grid points, the even one at a tie."""
    x = x.double()
    f32 = lambda t: t.float().double()
    big = x.abs().max(-1, keepdim=True).values
    s = f32(big / 2688.0)
    s = torch.where(big > 0, s, torch.ones_like(s))
    xb = x.view(x.shape[0], D // 16, 16)
    r = f32(xb.abs().max(-1, keepdim=True).values / f32(6.0 * s).unsqueeze(-1)).clamp(max=448.0)
    unit = torch.exp2(torch.floor(torch.log2(r.clamp(min=2.0 ** -6))) - 3)        # e4m3: three mantissa bits
    sf = torch.round(r / unit) * unit
    d = f32(sf * s.unsqueeze(-1))
    y = f32(xb * torch.where(d > 0, f32(1.0 / d), torch.zeros_like(d)))
    a = y.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    return (torch.sign(y) * torch.round(a / step) * step * sf * s.unsqueeze(-1)).view(x.shape)


def _exact_decode(case, st):
    cache, page = st["cache"], case["page"]
    n_q, n_kv = case["n_q"], case["n_kv"]
    O = torch.zeros(len(st["host_lens"]), n_q, D, dtype=torch.float64, device="cuda")
    lse = torch.full((len(st["host_lens"]), n_q), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["host_lens"]):
        if n == 0:
            continue
        pg = st["table"][b, :-(-n // page)].long()
        for kv in range(n_kv):
            k, v = (_values(cache["codes"][pg, i, kv], cache["sf"][pg, i, kv], cache["scale"][pg, i, kv],
                            torch.float64).flatten(0, 1)[:n] for i in (0, 1))
            hs = slice(kv * (n_q // n_kv), (kv + 1) * (n_q // n_kv))
            w = torch.einsum("hd,jd->hj", st["Q"][b].view(n_q, D)[hs].double(), k) / math.sqrt(D)
            lse[b, hs] = torch.logsumexp(w, 1)
            O[b, hs] = torch.einsum("hj,jd->hd", torch.softmax(w, 1), v)
    return {"O": O.flatten(1), "lse": lse}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "cache":
        return {n: _exact_rows(st[n].view(-1, D)).view(st[n].shape) for n in ("K", "V")}
    return _exact_decode(case, st) if case["op"] == "decode" else _exact_prompt(case, st)
