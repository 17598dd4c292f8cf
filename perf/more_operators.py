"""Workloads of the operators of a speculative decoding step over the 4-bit
key/value cache: rotary positions (forward, and forward + backward), the append
with the rotation on the way (and, behind it, the accepted nodes of a tree
moving to their places), attention of trees of drafted tokens, and their
verification against the target's probabilities.

``own`` selects what ``run`` computes with: the plain form of each operator in
elementary torch operations, or the framework's own calls.  ``exact`` gives
the same outputs from the definitions in 64 bits.

Heads are 128 wide, as everywhere in the framework.  Cache rows are NVFP4: e2m1
codes (two per byte), an e4m3 scale per 16 elements and an fp32 scale per row
of 128; page p, plane 0 (keys) or 1 (values), kv head h, offset o is row
[p, plane, h, o] of its three tensors.

A tree of sequence b is its run of tokens cu[b] .. cu[b + 1] - 1: node 0 is the
last committed token, whose keys are not in the cache before the step, the
others are drafted; parents[i] < i is the node that node i follows, -1 the
committed prefix.  Without parents the tokens are a chain.
"""
import math
import random

import torch

own = False

D = 128


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # training step of a block without per-head norms: queries and keys of 8192 tokens, 64 + 8 heads
        dict(name="rope_train", op="rope", tokens=8192, heads=72, rotary=128, pairing="half", back=True, far=2048,
             packed=False),
        # one decode step's tokens, half of each head rotated, far positions, columns of one projection output
        dict(name="rope_step", op="rope", tokens=61, heads=10, rotary=64, pairing="interleaved", back=False, far=131072,
             packed=True),
        # a prompt batch goes to the cache: Q and K rotated and kept for the prompts' own attention, K and V quantised
        dict(name="append_prompt", op="append", trees="2048*4", page=64, n_q=64, n_kv=8, rotary=128, pairing="half",
             keep_k=True, packed=True),
        # a decode step's trees: nodes appended, the accepted ones moved to the places behind the prefix
        dict(name="append_trees", op="append", trees="ragged:32:1:26:7", page=16, n_q=32, n_kv=8, rotary=64,
             pairing="interleaved", keep_k=False, packed=False),
        # one request, a chain of five drafts behind a short context: latency counts
        dict(name="tree_single", op="tree", lens="777", trees="6", chain=True, page=64, n_q=64, n_kv=8),
        # a serving batch of mixed contexts, chains of three drafts, one request without a prefix
        dict(name="tree_chains", op="tree", lens="0,ragged:63:1:8192:5", trees="4*64", chain=True, page=64, n_q=64, n_kv=8),
        # trees of very different sizes over mixed contexts
        dict(name="tree_ragged", op="tree", lens="ragged:24:60:6000:9", trees="ragged:24:1:64:3", chain=False, page=32,
             n_q=64, n_kv=8),
        # full trees over long contexts: the products count
        dict(name="tree_full", op="tree", lens="16384*8", trees="64*8", chain=False, page=128, n_q=32, n_kv=8),
        # two documents, small trees
        dict(name="tree_long", op="tree", lens="131055,100001", trees="16,11", chain=False, page=256, n_q=32, n_kv=8),
        # verification for one request, drafts sampled from a small model's probabilities
        dict(name="verify_one", op="verify", trees="8", chain=True, sampled=True, vocab=128256, dtype="float32"),
        # a serving batch of sampled chains
        dict(name="verify_chains", op="verify", trees="6*128", chain=True, sampled=True, vocab=128256, dtype="float32"),
        # trees of the most likely tokens (nothing sampled), bf16 probabilities, an odd vocabulary
        dict(name="verify_trees", op="verify", trees="ragged:48:1:40:11", chain=False, sampled=False, vocab=50257,
             dtype="bfloat16"),
    ]


def draw(rng):
    kind = rng.choice(["rope", "append", "tree", "tree", "tree", "verify", "verify"])
    n_kv = rng.choice([1, 2, 4, 8])
    n_q = n_kv * rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 16) if g * n_kv <= 64])
    rotary = rng.choice([32, 64, 96, 128, 128])
    pairing = rng.choice(["interleaved", "half"])
    if kind == "rope":
        return dict(op="rope", tokens=_log(rng, 1, 8192), heads=rng.choice([1, 3, 8, 10, 36, 72]), rotary=rotary,
                    pairing=pairing, back=rng.random() < 0.5, far=_log(rng, 64, 131072), packed=rng.random() < 0.5)
    if kind == "append":
        n = _log(rng, 1, 64)
        return dict(op="append", trees="ragged:%d:1:%d:%d" % (n, _log(rng, 1, min(256, 8192 // n)), rng.randrange(1 << 20)),
                    page=rng.choice([16, 32, 64, 128, 256]), n_q=n_q, n_kv=n_kv, rotary=rotary, pairing=pairing,
                    keep_k=rng.random() < 0.5, packed=rng.random() < 0.5)
    if kind == "tree":
        most = max(work(c)["flops"] for c in listed() if c["op"] == "tree")
        while True:
            n = _log(rng, 1, 64)
            top = _log(rng, 1, min(131072, 400000 // n))
            case = dict(op="tree", lens="ragged:%d:%d:%d:%d" % (n, rng.randint(0, min(top, 3)), top, rng.randrange(1 << 20)),
                        trees="ragged:%d:1:%d:%d" % (n, _log(rng, 1, 64), rng.randrange(1 << 20)), chain=rng.random() < 0.4,
                        page=rng.choice([16, 32, 64, 128, 256]), n_q=n_q, n_kv=n_kv)
            if work(case)["flops"] <= most:
                return case
    while True:
        chain = rng.random() < 0.5
        case = dict(op="verify", trees="ragged:%d:1:%d:%d" % (_log(rng, 1, 128), _log(rng, 1, 12 if chain else 48),
                                                             rng.randrange(1 << 20)),
                    chain=chain, sampled=rng.random() < 0.6, vocab=_log(rng, 1000, 160000),
                    dtype=rng.choice(["float32", "bfloat16"]))
        if sum(_lens(case["trees"])) * case["vocab"] <= 768 * 128256:
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


def _trees(case):
    """Parents of every node, tree by tree: a chain, or drafts that follow
    earlier nodes, the early ones more often."""
    r = random.Random(len(case["trees"]))
    out = []
    for n in _lens(case["trees"]):
        chain = case.get("chain", False)
        out.append([i - 1 if chain or i == 0 else int(i * r.random() ** 2) for i in range(n)])
    return out


def _depths(parents):
    d = []
    for p in parents:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def work(case):
    """Bytes: each input read once, each output written once; flops: the
    products over the pairs that the tree leaves."""
    if case["op"] == "rope":
        row = case["heads"] * D * 2
        return {"bytes": case["tokens"] * (row * 2 * (2 if case["back"] else 1) + 4 * case["rotary"] + 4), "flops": 0}
    nodes = _lens(case["trees"])
    if case["op"] == "append":
        t, n_kv = sum(nodes), case["n_kv"]
        rows = 2 * case["n_q"] + 2 * n_kv + (n_kv if case["keep_k"] else 0)
        back = 2 * n_kv * D * 4                                      # the read-back in fp32
        return {"bytes": t * (rows * D * 2 + 2 * n_kv * 76 + back + 4 * case["rotary"] + 8), "flops": 0}
    if case["op"] == "tree":
        lens, n_q, n_kv = _lens(case["lens"]), case["n_q"], case["n_kv"]
        pairs = sum(n * x + sum(d + 1 for d in _depths(t)) for n, x, t in zip(nodes, lens, _trees(case)))
        return {"bytes": (sum(lens) + sum(nodes)) * n_kv * 152 + sum(nodes) * n_q * (D * 4 + 4),
                "flops": 4 * D * n_q * pairs}
    # one row of the target's (and of the drafts') probabilities per request, and two values per node
    width = 4 if case["dtype"] == "float32" else 2
    rows = len(nodes) * (2 if case["sampled"] else 1)
    return {"bytes": rows * case["vocab"] * width + sum(nodes) * (2 * width + 12), "flops": 0}


# --------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cu(lens):
    c = [0]
    for x in lens:
        c.append(c[-1] + x)
    return _i32(c)


def _table(far, rotary):
    """cos | sin of every position and pair, angles in 64 bits."""
    a = torch.arange(far, device="cuda").double().unsqueeze(1)
    f = 500000.0 ** (-torch.arange(0, rotary, 2, device="cuda").double() / rotary)
    return torch.stack((torch.cos(a * f), torch.sin(a * f)), -1).float().contiguous()


def _rows(shape, g):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def _empty_cache(pages, n_kv, page):
    return {"codes": torch.zeros(pages, 2, n_kv, page, D // 2, dtype=torch.uint8, device="cuda"),
            "sf": torch.zeros(pages, 2, n_kv, page, D // 16, dtype=torch.uint8, device="cuda"),
            "scale": torch.zeros(pages, 2, n_kv, page, dtype=torch.float32, device="cuda")}


def _block_table(need, g):
    """Pages of every sequence, in no order."""
    order = torch.randperm(sum(need) + 3, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(need), max(need) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    if case["op"] == "rope":
        t, width = case["tokens"], case["heads"] * D
        wide = _rows((t, width + (256 if case["packed"] else 0)), g)
        st["X"] = wide[:, :width]
        if case["back"]:
            st["dY"] = _rows((t, width), g)
        st["cos_sin"] = _table(case["far"], case["rotary"])
        st["pos"] = torch.randint(0, case["far"], (t,), generator=g, device="cuda").to(torch.int32)
        if own:
            import gemm_epilogue_transformer_bf16_gb300 as coda
            st["ws"] = coda.workspace(256)
        return st
    trees = _trees(case)
    nodes = [len(t) for t in trees]
    total = sum(nodes)
    st["nodes"] = nodes
    st["cu"] = _cu(nodes)
    flat = [p for t in trees for p in t]
    if case["op"] == "append":
        n_q, n_kv, page = case["n_q"], case["n_kv"], case["page"]
        # keys in front of the trees: none for whole prompts, else a committed prefix
        r = random.Random(seed)
        before = [0 if case["keep_k"] else r.randint(0, 4 * page) for _ in nodes]
        lens = [a + b for a, b in zip(before, nodes)]
        st["table"] = _block_table([-(-x // page) for x in lens], g)
        st["lens"] = _i32(lens)
        owner = torch.repeat_interleave(torch.arange(len(nodes), device="cuda"), _i32(nodes).long())
        local = torch.arange(total, device="cuda") - st["cu"].long()[owner]
        at = local + _i32(before).long()[owner]
        st["slots"] = (st["table"][owner, at // page].long() * page + at % page).to(torch.int32)
        st["cache"] = _empty_cache(int(st["table"].max()) + 1, n_kv, page)
        st["cos_sin"] = _table(max(lens) + 1, case["rotary"])
        # a chain of prompts' tokens, or nodes at their depth behind the prefix
        where = [b + (i if case["keep_k"] else d) for t, b in zip(trees, before) for i, d in enumerate(_depths(t))]
        st["pos"] = _i32(where)
        cols = [n_q * D, n_kv * D, n_kv * D]
        if case["packed"]:
            st["Q"], st["K"], st["V"] = _rows((total, sum(cols)), g).split(cols, dim=1)
        else:
            st["Q"], st["K"], st["V"] = (_rows((total, c), g) for c in cols)
        # accepted nodes: the path from the root to some node (whole prompts: every token stays where it is)
        if not case["keep_k"]:
            paths = []
            for t in trees:
                i, path = r.randrange(len(t)), []
                while i >= 0:
                    path.append(i)
                    i = t[i]
                paths.append(path[::-1])
            width = max(len(p) for p in paths) + 1
            st["path"] = _i32([p + [-1] * (width - len(p)) for p in paths])
            st["count"] = _i32([len(p) - 1 for p in paths])
            st["paths"] = paths
        if own:
            import gemm_epilogue_transformer_bf16_gb300 as coda
            st["ws"] = coda.workspace(256)
        return st
    if case["op"] == "tree":
        n_q, n_kv, page = case["n_q"], case["n_kv"], case["page"]
        lens = [a + b for a, b in zip(_lens(case["lens"]), nodes)]
        table = _block_table([-(-x // page) for x in lens], g)
        pages = sum(-(-x // page) for x in lens) + 3
        st["cache"] = _empty_cache(pages, n_kv, page)
        step = max(1, (1 << 26) // (2 * n_kv * page * D))
        for p in range(0, pages, step):
            x = torch.randn(min(step, pages - p), 2, n_kv, page, D, generator=g, device="cuda").to(torch.bfloat16)
            for name, part in zip(("codes", "sf", "scale"), _quantise(x)):
                st["cache"][name][p:p + part.shape[0]] = part
        st["table"] = table
        st["lens"] = _i32(lens)
        st["host_lens"] = lens
        st["parents"] = None if case["chain"] else _i32(flat)
        st["trees"] = trees
        st["Q"] = _rows((total, n_q * D), g)
        st["out"] = {"O": torch.empty(total, n_q * D, dtype=torch.bfloat16, device="cuda"),
                     "lse": torch.empty(total, n_q, dtype=torch.float32, device="cuda")}
        if own:
            import gemm_epilogue_transformer_bf16_gb300 as coda
            need = coda.load().coda_attention_tree_nvfp4_workspace_size(total, len(lens), n_q, n_kv, D)
            st["ws"] = coda.workspace(need)
        return st
    # the target's probabilities after every node, and the drafts' where they were sampled
    vocab, dtype = case["vocab"], getattr(torch, case["dtype"])
    P = torch.empty(total, vocab, dtype=dtype, device="cuda")
    Q = torch.empty(total, vocab, dtype=dtype, device="cuda") if case["sampled"] else None
    kids = [[] for _ in range(total)]
    at = 0
    for t in trees:
        for i, p in enumerate(t):
            if p >= 0:
                kids[at + p].append(at + i)
        at += len(t)
    most = max(1, max(len(k) for k in kids))
    tokens = torch.zeros(total, dtype=torch.int64, device="cuda")
    step = max(1, (1 << 26) // vocab)
    for a in range(0, total, step):
        b = min(total, a + step)
        z = torch.randn(b - a, vocab, generator=g, device="cuda") * 3.0
        P[a:b] = torch.softmax(z, 1).to(dtype)
        z += torch.randn(b - a, vocab, generator=g, device="cuda") * 0.6
        q = torch.softmax(z, 1).to(dtype)
        if case["sampled"]:
            Q[a:b] = q
            pick = torch.multinomial(q.float(), most, replacement=True, generator=g)
        else:
            pick = torch.topk(z, most).indices
        to = [(c, i, j) for i in range(a, b) for j, c in enumerate(kids[i])]
        if to:
            to = torch.tensor(to, device="cuda")
            tokens[to[:, 0]] = pick[to[:, 1] - a, to[:, 2]]
    st["P"], st["draft_P"] = P, Q
    st["tokens"] = tokens.to(torch.int32)
    st["parents"] = None if case["chain"] else _i32(flat)
    st["trees"] = trees
    st["u"] = torch.rand(total, generator=g, device="cuda")
    st["u_next"] = torch.rand(len(nodes), generator=g, device="cuda")
    st["width"] = max(max(_depths(t)) for t in trees) + 1
    if own:
        import gemm_epilogue_transformer_bf16_gb300 as coda
        st["ws"] = coda.workspace(coda.load().coda_verify_drafts_workspace_size(total, len(nodes), vocab))
    return st


# --------------------------------------------------------------------------- plain forms

def _quantise(x):
    """NVFP4 rows of x [..., 128]: packed codes [..., 64], e4m3 block scales
    [..., 8] as bytes, fp32 row scales [...].  Every step is one fp32 operation;
    e2m1 and e4m3 round to nearest, ties to even."""
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


def _pairs(x, pairing):
    """The two elements of every rotated pair, and how to put them back."""
    if pairing == "half":
        return x.chunk(2, -1), lambda a, b: torch.cat((a, b), -1)
    return (x[..., 0::2], x[..., 1::2]), lambda a, b: torch.stack((a, b), -1).flatten(-2)


def _rotate(x, cos, sin, rotary, pairing):
    """x [T, heads, 128]; cos, sin [T, rotary / 2]; every step one operation."""
    (a, b), put = _pairs(x[..., :rotary], pairing)
    c, s = cos.unsqueeze(1), sin.unsqueeze(1)
    return torch.cat((put(a * c - b * s, b * c + a * s), x[..., rotary:]), -1)


def _plain_rope(st):
    case = st["case"]
    cos, sin = st["cos_sin"][st["pos"].long()].unbind(-1)
    out = {"Y": _rotate(st["X"].float().unflatten(1, (-1, D)), cos, sin, case["rotary"], case["pairing"])
           .flatten(1).to(torch.bfloat16)}
    if case["back"]:
        out["dX"] = _rotate(st["dY"].float().unflatten(1, (-1, D)), cos, -sin, case["rotary"], case["pairing"]) \
            .flatten(1).to(torch.bfloat16)
    return out


def _plain_append(st):
    case, cache, slots = st["case"], st["cache"], st["slots"].long()
    page, n_kv = case["page"], case["n_kv"]
    cos, sin = st["cos_sin"][st["pos"].long()].unbind(-1)
    turn = lambda x: _rotate(x.float().unflatten(1, (-1, D)), cos, sin, case["rotary"], case["pairing"])
    K = turn(st["K"])
    out = {"Q": turn(st["Q"]).flatten(1).to(torch.bfloat16)}
    if case["keep_k"]:
        out["K"] = K.flatten(1).to(torch.bfloat16)
    pg, off = slots // page, slots % page
    for plane, x in enumerate((K, st["V"].unflatten(1, (-1, D)))):
        for key, part in zip(("codes", "sf", "scale"), _quantise(x)):
            cache[key][pg, plane, :, off] = part
    if not case["keep_k"]:
        # the rows of every path, then into the places behind the prefix
        first, total = st["cu"].long()[:-1], slots.numel()
        keep = st["path"].long()
        ok = keep >= 0
        src = slots[(first.unsqueeze(1) + keep.clamp(min=0)).clamp(max=total - 1)]
        place = first.unsqueeze(1) + torch.arange(keep.shape[1], device="cuda")
        dst = slots[place.clamp(max=total - 1)]
        src, dst = src[ok], dst[ok]
        for t in cache.values():
            t[dst // page, :, :, dst % page] = t[src // page, :, :, src % page]
        nodes = st["cu"][1:] - st["cu"][:-1]
        out["seq_lens"] = st["lens"] - nodes + st["count"] + 1
    for plane, name in enumerate(("cache_K", "cache_V")):
        out[name] = _values(cache["codes"][pg, plane, :, off], cache["sf"][pg, plane, :, off],
                            cache["scale"][pg, plane, :, off], torch.float32).flatten(1)
    return out


def _seen(tree):
    """[n, n]: whether node i sees node j (itself and its ancestors)."""
    m = torch.zeros(len(tree), len(tree), dtype=torch.bool)
    for i, p in enumerate(tree):
        if p >= 0:
            m[i] = m[p]
        m[i, i] = True
    return m


def _plain_tree(st):
    case, cache = st["case"], st["cache"]
    n_q, n_kv, page = case["n_q"], case["n_kv"], case["page"]
    g, scale = n_q // n_kv, 1.0 / math.sqrt(D)
    O, lse = torch.empty_like(st["out"]["O"]), torch.empty_like(st["out"]["lse"])
    at = 0
    for b, (n, total) in enumerate(zip(st["nodes"], st["host_lens"])):
        pg = st["table"][b, :-(-total // page)].long()
        k, v = (_values(cache["codes"][pg, i], cache["sf"][pg, i], cache["scale"][pg, i], torch.float32)
                .transpose(0, 1).flatten(1, 2)[:, :total] for i in (0, 1))
        q = st["Q"][at:at + n].float().view(n, n_kv, g, D).permute(1, 2, 0, 3)
        s = torch.matmul(q.flatten(1, 2), k.transpose(1, 2)).unflatten(1, (g, n)) * scale
        s[..., total - n:].masked_fill_(~_seen(st["trees"][b]).cuda(), -math.inf)
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        l = p.sum(-1, keepdim=True)
        o = torch.matmul(p.flatten(1, 2), v).unflatten(1, (g, n)) / l
        O[at:at + n] = o.permute(2, 0, 1, 3).flatten(1).to(torch.bfloat16)
        lse[at:at + n] = (m + torch.log(l)).squeeze(-1).permute(2, 0, 1).flatten(1)
        at += n
    return {"O": O, "lse": lse}


def _plain_verify(st):
    """All requests side by side, node by node; w and its sums in 64 bits."""
    case, first = st["case"], st["cu"].long()[:-1]
    batch, total = len(st["nodes"]), st["tokens"].numel()
    nodes = st["cu"].long()[1:] - first
    parents = st["parents"]
    if parents is None:
        parents = torch.arange(total, device="cuda") - torch.repeat_interleave(first, nodes) - 1
    rows = torch.arange(batch, device="cuda")
    here = torch.zeros(batch, dtype=torch.int64, device="cuda")
    count = torch.zeros(batch, dtype=torch.int64, device="cuda")
    path = torch.full((batch, st["width"]), -1, dtype=torch.int32, device="cuda")
    out = path.clone()
    path[:, 0] = 0
    w, Z = st["P"][first].double(), torch.ones(batch, dtype=torch.float64, device="cuda")
    for i in range(1, max(st["nodes"])):
        row = (first + i).clamp(max=total - 1)
        child = (i < nodes) & (parents[row].long() == here)
        x = st["tokens"][row].long()
        wx = w[rows, x]
        q = st["draft_P"][first + here].double() if case["sampled"] else None
        qx = q[rows, x] if case["sampled"] else torch.ones_like(wx)
        take = child & (st["u"][row].double() * (qx * Z) < wx)
        drop = child & ~take
        if case["sampled"]:
            left = (w - Z.unsqueeze(1) * q).clamp(min=0)
            w = torch.where(drop.unsqueeze(1), left, w)
            Z = torch.where(drop, left.sum(1), Z)
        else:
            w[rows, x] = torch.where(drop, torch.zeros_like(wx), wx)
            Z = torch.where(drop, Z - wx, Z)
        w = torch.where(take.unsqueeze(1), st["P"][row].double(), w)
        Z = torch.where(take, torch.ones_like(Z), Z)
        out[rows[take], count[take]] = x[take].to(torch.int32)
        count = count + take.long()
        path[rows[take], count[take]] = i
        here = torch.where(take, torch.full_like(here, i), here)
    c = torch.cumsum(w, 1)
    nxt = (c <= st["u_next"].double().unsqueeze(1) * c[:, -1:]).sum(1)
    out[rows, count] = nxt.to(torch.int32)
    return {"count": count.to(torch.int32), "nodes": path, "tokens": out}


# --------------------------------------------------------------------------- one pass

def run(st):
    case = st["case"]
    if not own:
        return {"rope": _plain_rope, "append": _plain_append, "tree": _plain_tree, "verify": _plain_verify}[case["op"]](st)
    import gemm_epilogue_transformer_bf16_gb300 as coda
    ws = st["ws"]
    if case["op"] == "rope":
        out = {"Y": coda.rope(st["X"], st["pos"], st["cos_sin"], case["heads"], pairing=case["pairing"], ws=ws)["Y"]}
        if case["back"]:
            out["dX"] = coda.rope_bwd(st["dY"], st["pos"], st["cos_sin"], case["heads"], pairing=case["pairing"],
                                      ws=ws)["dX"]
        return out
    if case["op"] == "append":
        out = coda.kv_append_rope_nvfp4(st["K"], st["V"], st["slots"], st["cache"], st["pos"], st["cos_sin"], Q=st["Q"],
                                        n_q=case["n_q"], pairing=case["pairing"], keep_k=case["keep_k"], ws=ws)
        if not case["keep_k"]:
            out["seq_lens"] = coda.kv_accept_nvfp4(st["cache"], st["table"], st["lens"], st["cu"], st["path"], st["count"],
                                                   ws=ws)["seq_lens"]
        rows = coda.kv_read_nvfp4(st["cache"], st["slots"], dtype=torch.float32, ws=ws)
        return {**out, "cache_K": rows["K"], "cache_V": rows["V"]}
    if case["op"] == "tree":
        return coda.attention_tree_nvfp4(st["Q"], st["cache"], st["table"], st["lens"], st["cu"], case["n_q"],
                                         parents=st["parents"], out=st["out"], ws=ws)
    return coda.verify_drafts(st["P"], st["tokens"], st["cu"], st["u"], st["u_next"], st["width"], parents=st["parents"],
                              draft_probs=st["draft_P"], ws=ws)


# --------------------------------------------------------------------------- 64 bits

def _turn_exact(x, st, back=False):
    """Each pair as a complex number times exp(i angle) of the table."""
    case = st["case"]
    r = case["rotary"]
    x = x.double().unflatten(1, (-1, D)).clone()
    turn = torch.view_as_complex(st["cos_sin"].double())[st["pos"].long()].unsqueeze(1)
    if back:
        turn = turn.conj()
    if case["pairing"] == "half":
        first, second = slice(0, r // 2), slice(r // 2, r)
    else:
        first, second = slice(0, r, 2), slice(1, r, 2)
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
    x[..., first], x[..., second] = z.real, z.imag
    return x


def _exact_rows(x):
    """The values NVFP4 rows of x [rows, 128] stand for.  The format's scales
    are fp32 and e4m3 numbers, so each is rounded to its own format here; the
    codes are the nearest grid points, the even one at a tie."""
    f32 = lambda t: t.float().double()
    x = f32(x.double())
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


def _exact_append(case, st):
    K = _turn_exact(st["K"], st)
    out = {"Q": _turn_exact(st["Q"], st).flatten(1)}
    if case["keep_k"]:
        out["K"] = K.flatten(1)
    rows = {n: _exact_rows(x.reshape(-1, D)).view(x.shape[0], -1)
            for n, x in (("cache_K", K), ("cache_V", st["V"]))}
    if not case["keep_k"]:
        lens, first = [], 0
        for b, path in enumerate(st["paths"]):
            for to, i in enumerate(path):          # in order: a node's place is never behind it
                for x in rows.values():
                    x[first + to] = x[first + i]
            lens.append(int(st["lens"][b]) - st["nodes"][b] + len(path))
            first += st["nodes"][b]
        out["seq_lens"] = _i32(lens)
    return {**out, **rows}


def _exact_tree(case, st):
    cache, page, n_q, n_kv = st["cache"], case["page"], case["n_q"], case["n_kv"]
    total = st["Q"].shape[0]
    O = torch.zeros(total, n_q, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(total, n_q, dtype=torch.float64, device="cuda")
    at = 0
    for b, tree in enumerate(st["trees"]):
        n, keys = len(tree), st["host_lens"][b]
        pg = st["table"][b, :-(-keys // page)].long()
        hidden = torch.zeros(n, keys, dtype=torch.bool, device="cuda")
        for i in range(n):
            up, j = set(), i
            while j >= 0:
                up.add(j)
                j = tree[j]
            no = [keys - n + j for j in range(n) if j not in up]
            if no:
                hidden[i, torch.tensor(no, device="cuda")] = True
        for h in range(n_kv):
            k, v = (_values(cache["codes"][pg, i, h], cache["sf"][pg, i, h], cache["scale"][pg, i, h],
                            torch.float64).flatten(0, 1)[:keys] for i in (0, 1))
            hs = slice(h * (n_q // n_kv), (h + 1) * (n_q // n_kv))
            w = torch.einsum("ihd,jd->ihj", st["Q"][at:at + n].view(n, n_q, D)[:, hs].double(), k) / math.sqrt(D)
            w = torch.where(hidden.unsqueeze(1), torch.full((), -math.inf, dtype=torch.float64, device="cuda"), w)
            lse[at:at + n, hs] = torch.logsumexp(w, 2)
            O[at:at + n, hs] = torch.einsum("ihj,jd->ihd", torch.softmax(w, 2), v)
        at += n
    return {"O": O.flatten(1), "lse": lse}


def _exact_verify(case, st):
    """Request by request, as the definition reads."""
    width = st["width"]
    counts, paths, texts = [], [], []
    u, tokens, first = st["u"].tolist(), st["tokens"].tolist(), 0
    for b, tree in enumerate(st["trees"]):
        here, path, text = 0, [0], []
        while True:
            w, Z = st["P"][first + here].double(), 1.0
            went = False
            for i in (j for j, p in enumerate(tree) if p == here and j > here):
                x = tokens[first + i]
                q = st["draft_P"][first + here].double() if case["sampled"] else None
                if u[first + i] * ((float(q[x]) if case["sampled"] else 1.0) * Z) < float(w[x]):
                    here, went = i, True
                    path.append(i)
                    text.append(x)
                    break
                if case["sampled"]:
                    w = (w - Z * q).clamp(min=0)
                    Z = float(w.sum())
                else:
                    Z -= float(w[x])
                    w = w.clone()
                    w[x] = 0
            if not went:
                break
        c = torch.cumsum(w, 0)
        text.append(int((c <= float(st["u_next"][b].double()) * c[-1]).sum()))
        counts.append(len(path) - 1)
        paths.append(path + [-1] * (width - len(path)))
        texts.append(text + [-1] * (width - len(text)))
        first += len(tree)
    return {"count": _i32(counts), "nodes": _i32(paths), "tokens": _i32(texts)}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        out = {"Y": _turn_exact(st["X"], st).flatten(1)}
        if case["back"]:
            out["dX"] = _turn_exact(st["dY"], st, back=True).flatten(1)
        return out
    return {"append": _exact_append, "tree": _exact_tree, "verify": _exact_verify}[case["op"]](case, st)
