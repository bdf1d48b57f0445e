"""What is measured of the operators that check drafted tokens: attention of a
tree of drafted tokens over the paged key-value cache, copying and compacting
cache rows over all layers of a model, and the log probabilities of the head's
logits.

A tree: of a sequence's new tokens, token i has a parent before it or none
(-1).  It sees the keys cached before all of them, its ancestors and itself,
and stands at the position of the first new token plus its depth.  The cache is
that of qmm_kv.h: pages of page_size rows of each key-value head; sequence s
has its token j in row j % page_size of page table[s][j // page_size].
"""
import math
import random

import torch

own = False

DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}

# Head layouts: the 8B model's (4096 = 32 x 128, 8 key-value heads), the 1B
# model's (2048 = 32 x 64, 8), the 896-wide one's (14 x 64, 2), one with a
# head per key-value head, and one of wide heads.
HEADS = {"8b": (32, 8, 128), "1b": (32, 8, 64), "0.5b": (14, 2, 64), "one each": (32, 32, 128), "wide": (16, 8, 256)}


def listed():
    def tree(name, **k):
        base = dict(cap=0.0, window=0, slopes=False)
        base.update(k)
        return dict(name=name, op="tree", **base)

    def logprobs(name, **k):
        base = dict(given=1, top=0, scale=1.0, cap=0.0)
        base.update(k)
        return dict(name=name, op="logprobs", **base)

    return [
        # a few tokens drafted in a row at the start of a conversation with the smallest model: latency
        tree("tree, short chain", heads="0.5b", x="f32", cache="q8_0", seqs=1, new=5, branch=1, old=71, page=16),
        # one conversation, a full tree of drafts
        tree("tree, one conversation", heads="8b", x="f32", cache="q8_0", seqs=1, new=64, branch=9, old=7930, page=64),
        # few drafts at the end of a long document: the length is split
        tree("tree, one long", heads="8b", x="bf16", cache="f16", seqs=1, new=13, branch=3, old=130911, page=128),
        # a batch of image-and-text conversations with capped scores, a window, and wide heads
        tree("tree, window and cap", heads="wide", x="bf16", cache="bf16", seqs=12, new=26, branch=5, old=3100, page=32, cap=50.0, window=2048),
        # a full batch of long conversations, some drafts each: bandwidth against products
        tree("tree, full", heads="8b", x="f32", cache="q8_0", seqs=32, new=16, branch=4, old=12287, page=64),
        # the accepted path of one conversation's tree, all 32 layers: latency
        dict(name="keep, one path", op="keep", heads="8b", cache="f16", layers=32, seqs=1, old=1203, new=64, kept=5, page=64, sinks=2),
        # a batch of conversations each drops the middle of what it knows: bandwidth
        dict(name="keep, half of each", op="keep", heads="8b", cache="bf16", layers=16, seqs=8, old=0, new=4077, kept=1900, page=64, sinks=4),
        # one conversation forks: its last page is copied, 16 layers
        dict(name="copy, last page", op="copy", heads="1b", cache="f16", layers=16, pages=1, pool=6, page=32, whole=False),
        # conversations leave a shared batch with pages of their own
        dict(name="copy, many pages", op="copy", heads="8b", cache="f16", layers=32, pages=130, pool=300, page=32, whole=True),
        # a drawn token of one conversation and its alternatives: latency
        logprobs("log probabilities, one row", x="f32", rows=1, vocab=128256, top=20, scale=1.25),
        # the rows of a batch of drafted trees, each token's drafted children
        logprobs("log probabilities, drafts", x="f32", rows=257, vocab=128256, given=4, top=5),
        # a prompt scored whole, capped bf16 logits
        logprobs("log probabilities, prompt", x="bf16", rows=2048, vocab=151936, top=8, cap=30.0),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["tree", "tree", "tree", "keep", "copy", "logprobs", "logprobs"])
    if kind == "logprobs":
        vocab = _spread(rng, 1000, 260000)
        return dict(op="logprobs", x=rng.choice(["f32", "bf16"]), rows=_spread(rng, 1, min(2048, 2048 * 120000 // vocab)), vocab=vocab,
                    given=rng.choice([0, 1, 1, rng.randint(2, 16)]), top=rng.choice([0, 1, rng.randint(2, 20), rng.randint(21, 64)]),
                    scale=rng.choice([1.0, 1.0, 0.7, 1.6]), cap=rng.choice([0.0, 0.0, 30.0]))
    c = dict(op=kind, heads=rng.choice(sorted(HEADS)), cache=rng.choice(["q8_0", "f16", "bf16"]), page=rng.choice([16, 32, 48, 64, 128]))
    n_q, n_kv, dim = HEADS[c["heads"]]
    row = n_kv * dim * (4 if c["cache"] != "q8_0" else 14)  # bytes of a token's keys and values; Q8_0 ones are read back as fp32
    if kind == "copy":
        c["layers"] = rng.choice([4, 16, 24, 32])
        c["pages"] = _spread(rng, 1, max(1, min(130, 500_000_000 // (c["layers"] * row * c["page"]))))
        c.update(pool=2 * c["pages"] + rng.randint(0, c["pages"] + 2), whole=rng.random() < 0.5)
        return c
    if kind == "keep":
        c["layers"] = rng.choice([4, 16, 24, 32])
        c["seqs"] = _spread(rng, 1, 16)
        most = max(48, min(4077, 1_000_000_000 // (c["layers"] * row * c["seqs"])))
        c["new"] = _spread(rng, 16, most)
        c.update(old=rng.choice([0, rng.randint(1, min(300, most))]), sinks=rng.choice([0, 1, 4]))
        c["kept"] = max(c["sinks"] + 1, _spread(rng, 1, c["new"] // 2 - 4))
        return c
    c.update(x=rng.choice(["f32", "bf16"]), cap=rng.choice([0.0, 0.0, 30.0]), window=rng.choice([0, 0, 0, _spread(rng, 16, 4096)]),
             slopes=rng.random() < 0.2, seqs=_spread(rng, 1, 48), new=_spread(rng, 2, 100))
    c["branch"] = rng.randint(1, min(12, c["new"]))
    c["old"] = _spread(rng, 1, min(130000, 32 * 8000 * 1024 // (c["seqs"] * n_kv * dim), 15_000_000_000 // (c["new"] * c["seqs"] * n_q * dim) + 1))
    return c


def _uneven(most, n, least=1):
    """Lengths of a batch of n: uneven, down to a half of the longest."""
    return [max(least, most - int(most * ((i * 0.6180339887) % 1.0 * 0.5))) for i in range(n)]


def _trees(case, seed):
    """The parent of every new token, sequence by sequence: one of the `branch` places before it (none where that is before the first)."""
    r = random.Random(seed)
    return [[max(-1, i - 1 - r.randrange(case["branch"])) for i in range(n)] for n in _uneven(case["new"], case["seqs"])]


def _keeps(case, seed):
    """Indexes, among its new tokens, that each sequence keeps: the first few, and some of the second half."""
    r = random.Random(seed)
    out = []
    for n, k in zip(_uneven(case["new"], case["seqs"], 2 * case["kept"] + 8), _uneven(case["kept"], case["seqs"])):
        a = min(case["sinks"], k)
        out.append(list(range(a)) + sorted(r.sample(range(n // 2, n), min(k - a, n - n // 2))))
    return out


def _slopes(n_q, device):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / n_q) for h in range(n_q)], device=device)


def _q8_0_bytes(x):
    """Rows of fp32 values as Q8_0 blocks: d = amax / 127, codes rounded to the nearest, d stored as fp16."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    d = b.abs().amax(-1, keepdim=True) / 127.0
    codes = (b / d.clamp(min=1e-30)).round().clamp(-127, 127).to(torch.int8)
    return torch.cat([d.half().view(torch.uint8), codes.view(torch.uint8)], -1).reshape(*x.shape[:-1], -1)


def _rows(cache, pages):
    """The values that a cache array holds, as fp32."""
    if cache != "q8_0":
        return pages.float()
    b = pages.reshape(*pages.shape[:-1], -1, 34)
    d = b[..., :2].contiguous().view(torch.float16).float()
    return (b[..., 2:].contiguous().view(torch.int8).float() * d).flatten(-2)


def _pool(case, g, *shape):
    x = torch.randn(*shape, device="cuda", generator=g, dtype=torch.float32 if case["cache"] == "q8_0" else DTYPE[case["cache"]])
    return _q8_0_bytes(x) if case["cache"] == "q8_0" else x


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _pages(lens, page, g, spare=0):
    """A table of shuffled pages for sequences of these lengths, and how many pages there are."""
    width = -(-max(lens) // page)
    owned = torch.tensor([-(-n // page) for n in lens], device="cuda")
    n = int(owned.sum()) + spare
    order = torch.randperm(n, device="cuda", generator=g).to(torch.int32)
    at = (owned.cumsum(0) - owned)[:, None] + torch.arange(width, device="cuda")
    return torch.where(torch.arange(width, device="cuda") < owned[:, None], order[at.clamp(max=n - 1)], 0).contiguous(), n


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case}
    if case["op"] == "logprobs":
        # a head's logits: most of them noise, some tokens of each row likely
        N, V = case["rows"], case["vocab"]
        x = torch.randn(N, V, device="cuda", generator=g) * 2.5
        likely = (torch.randint(0, V, (N, 1), device="cuda", generator=g) + torch.arange(12, device="cuda") * (V // 12)) % V
        x.scatter_add_(1, likely, torch.rand(N, 12, device="cuda", generator=g) * 14)
        st["logits"] = x.to(DTYPE[case["x"]])
        st["tokens"] = torch.cat([likely, torch.randint(0, V, (N, 4), device="cuda", generator=g)], 1)[:, 16 - case["given"]:].to(torch.int32).contiguous()
        return st
    n_q, n_kv, dim = HEADS[case["heads"]]
    page = case["page"]
    st.update(n_q=n_q, n_kv=n_kv, dim=dim)
    if case["op"] == "copy":
        order = torch.randperm(case["pool"], device="cuda", generator=g).to(torch.int32)
        st["src"], st["dst"] = order[:case["pages"]].clone(), order[case["pages"]:2 * case["pages"]].clone()
        st["rows"] = None if case["whole"] else torch.randint(1, page + 1, (case["pages"],), device="cuda", generator=g, dtype=torch.int32)
        st["k"], st["v"] = (_pool(case, g, case["layers"], case["pool"], n_kv, page, dim) for _ in range(2))
        return st
    if case["op"] == "keep":
        keeps = _keeps(case, seed)
        first = [case["old"] // (1 + s % 3) for s in range(case["seqs"])]
        lens = [f + n for f, n in zip(first, _uneven(case["new"], case["seqs"], 2 * case["kept"] + 8))]
        st["table"], n_pages = _pages(lens, page, g)
        width = max(len(k) for k in keeps)
        st["first"], st["n_keep"] = _ints(first), _ints([len(k) for k in keeps])
        st["keep"] = _ints([[f + i for i in k] + [0] * (width - len(k)) for f, k in zip(first, keeps)])
        st["kv_len"] = _ints(lens)
        st["k"], st["v"] = (_pool(case, g, case["layers"], n_pages, n_kv, page, dim) for _ in range(2))
        return st
    parents = _trees(case, seed)
    new = [len(p) for p in parents]
    lens = [a + b for a, b in zip(new, _uneven(case["old"], case["seqs"]))]
    starts = [sum(new[:s]) for s in range(len(new) + 1)]
    st["table"], n_pages = _pages(lens, page, g, spare=2)
    st.update(N=starts[-1], new=max(new), kv=max(lens), q_start=_ints(starts), kv_len=_ints(lens), parents=_ints(sum(parents, [])))
    st["slopes"] = _slopes(n_q, "cuda") if case["slopes"] else None
    st["q"] = torch.randn(st["N"], n_q, dim, device="cuda", generator=g).to(DTYPE[case["x"]])
    st["k"], st["v"] = (_pool(case, g, n_pages, n_kv, page, dim) for _ in range(2))
    # the trees as a program that masks scores keeps them: who sees whom among the new tokens, and depths
    T = st["new"]
    sees = torch.zeros(case["seqs"], T, T, dtype=torch.bool)
    for s, p in enumerate(parents):
        for i, a in enumerate(p):
            if a >= 0:
                sees[s, i] = sees[s, a]
            sees[s, i, i] = True
    st["sees"] = sees.cuda()
    st["depth"] = st["sees"].sum(2) - 1
    return st


def run(st):
    case = st["case"]
    if own:
        return _run_own(st)
    return {"tree": _tree_plain, "keep": _keep_plain, "copy": _copy_plain, "logprobs": _logprobs_plain}[case["op"]](st)


def _run_own(st):
    import block_quantized_amd as Q
    case = st["case"]
    if case["op"] == "logprobs":
        lp = Q.logprobs(st["logits"], tokens=st["tokens"] if case["given"] else None, top=case["top"], scale=case["scale"], softcap=case["cap"])
        return [x for x in (lp.tokens, lp.entropy, lp.top_ids, lp.top) if x is not None]
    kind = {"q8_0": Q.QMM_Q8_0, "f16": Q.QMM_F16, "bf16": Q.QMM_BF16}[case["cache"]]
    if case["op"] == "tree":
        if "handle" not in st:  # what a program keeps over all layers of a step
            st["handle"] = Q.KVCache(st["k"], st["v"], kind, st["n_kv"], st["dim"], case["page"])
            st["batch"] = Q.KVBatch(st["q_start"], st["kv_len"], st["table"], st["N"], max_kv=st["kv"])
            st["tree"] = Q.KVTree(st["batch"], st["parents"], max_new=st["new"])
        return Q.attn(st["handle"], st["batch"], st["q"], softcap=case["cap"], window=case["window"], slopes=st["slopes"], tree=st["tree"])
    if "layers" not in st:
        st["layers"] = Q.KVLayers([Q.KVCache(k, v, kind, st["n_kv"], st["dim"], case["page"]) for k, v in zip(st["k"], st["v"])])
    out = []
    if case["op"] == "copy":
        Q.kv_copy(st["layers"], st["src"], st["dst"], rows=st["rows"])
    else:
        Q.kv_compact(st["layers"], st["table"], st["first"], st["keep"], st["n_keep"], kv_len=st["kv_len"])
        out = [st["kv_len"]]
    if case["cache"] != "q8_0":
        return out + [st["k"], st["v"]]
    rows = st["k"].numel() // st["k"].shape[-1]
    return out + [Q.dequantize(Q.QMM_Q8_0, c, rows, st["dim"]).view(*c.shape[:-1], st["dim"]) for c in (st["k"], st["v"])]


def _values(case, pools):
    return [_rows("q8_0", c) for c in pools] if case["cache"] == "q8_0" else list(pools)


def _copy_plain(st):
    src, dst = st["src"].long(), st["dst"].long()
    rows = torch.full_like(src, st["case"]["page"]) if st["rows"] is None else st["rows"]
    full = (torch.arange(st["case"]["page"], device="cuda") < rows[:, None])[:, None, :, None]  # pages, 1, rows, 1
    st["k"][:, dst] = torch.where(full, st["k"][:, src], st["k"][:, dst])
    st["v"][:, dst] = torch.where(full, st["v"][:, src], st["v"][:, dst])
    return _values(st["case"], (st["k"], st["v"]))


def _keep_plain(st):
    page, width = st["case"]["page"], st["keep"].shape[1]
    i = torch.arange(width, device="cuda")
    s, i = torch.nonzero(i < st["n_keep"][:, None], as_tuple=True)
    a, b = st["keep"][s, i].long(), st["first"][s].long() + i
    src, dst = st["table"][s, a // page].long(), st["table"][s, b // page].long()
    st["k"][:, dst, :, b % page] = st["k"][:, src, :, a % page]
    st["v"][:, dst, :, b % page] = st["v"][:, src, :, a % page]
    st["kv_len"].copy_(st["first"] + st["n_keep"])
    return [st["kv_len"]] + _values(st["case"], (st["k"], st["v"]))


def _logprobs_plain(st):
    case, raw = st["case"], st["logits"]
    x = raw.float()
    if case["cap"]:
        x = case["cap"] * torch.tanh(x / case["cap"])
    x = x * case["scale"]
    big = x.max(1, keepdim=True)
    x = x - big.values
    e = torch.exp(x).scatter_(1, big.indices, 0.0)  # the largest one's 1 stays out of the sum: where it is nearly all, the rest counts
    rest = e.sum(1, keepdim=True)
    out = []
    if case["given"]:
        out.append(torch.gather(x, 1, st["tokens"].long()) - torch.log1p(rest))
    out.append((torch.log1p(rest) - (e * x).sum(1, keepdim=True) / (1 + rest))[:, 0])
    if case["top"]:
        # the largest logits, equal ones by their index: one whole number for both
        bits = raw.float().add(0.0).view(torch.int32)  # (-0 + 0 is 0)
        key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * (1 << 32) + (case["vocab"] - 1 - torch.arange(case["vocab"], device="cuda"))
        ids = case["vocab"] - 1 - (torch.topk(key, case["top"], dim=1).values & 0xFFFFFFFF)
        out += [ids.int(), torch.gather(x, 1, ids) - torch.log1p(rest)]
    return out


def _tree_plain(st):
    case = st["case"]
    B, n_kv, dim, page = case["seqs"], st["n_kv"], st["dim"], case["page"]
    G, T = st["n_q"] // n_kv, st["new"]

    def dense(pages):  # B, n_kv, keys, dim
        return _rows(case["cache"], pages[st["table"].long()]).transpose(1, 2).reshape(B, n_kv, -1, dim)

    k, v = dense(st["k"]), dense(st["v"])
    L = k.shape[2]
    i = torch.arange(T, device="cuda")
    n = st["q_start"][1:] - st["q_start"][:-1]
    row = torch.where(i < n[:, None], st["q_start"][:-1, None] + i, st["N"])  # the row behind the last stands for none
    q = st["q"].float()[row.clamp(max=st["N"] - 1)]  # B, T, n_q, dim
    q = q.reshape(B, T, n_kv, G, dim).permute(0, 2, 3, 1, 4).reshape(B, n_kv, G * T, dim)
    s = (torch.matmul(q, k.transpose(2, 3)) * dim ** -0.5).view(B, n_kv, G, T, L)
    if case["cap"]:
        s = case["cap"] * torch.tanh(s / case["cap"])
    base = (st["kv_len"] - n)[:, None]
    at = torch.arange(L, device="cuda") - base  # B, L: among the new tokens, or below 0
    inside = at.clamp(0, T - 1)
    place = torch.where(at < 0, at, torch.gather(st["depth"], 1, inside))  # positions less the base's
    gap = st["depth"][:, :, None] - place[:, None]  # B, T, L
    if st["slopes"] is not None:
        s = s - st["slopes"].view(1, n_kv, G, 1, 1) * gap[:, None, None].abs()
    seen = (at < 0)[:, None] | torch.gather(st["sees"], 2, inside[:, None].expand(B, T, L))
    if case["window"]:
        seen = seen & (gap < case["window"])
    seen = (seen & (at < n[:, None])[:, None])[:, None, None]
    s = s.masked_fill(~seen, -math.inf)
    w = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e30))
    o = torch.matmul(w.view(B, n_kv, G * T, L), v) / w.sum(-1).clamp(min=1e-30).view(B, n_kv, G * T, 1)
    o = o.view(B, n_kv, G, T, dim).permute(0, 3, 1, 2, 4).reshape(B, T, st["n_q"], dim)
    out = torch.zeros(st["N"] + 1, st["n_q"], dim, device="cuda", dtype=DTYPE[case["x"]])
    out[row] = o.to(out.dtype)
    return out[:st["N"]]


def work(case):
    if case["op"] == "logprobs":
        x, small = 4 if case["x"] == "f32" else 2, case["rows"] * (8 * case["given"] + 4 + 8 * case["top"])
        return {"bytes": case["rows"] * case["vocab"] * x + small, "flops": 4 * case["rows"] * case["vocab"]}
    n_q, n_kv, dim = HEADS[case["heads"]]
    value = 34 / 32 if case["cache"] == "q8_0" else 2
    if case["op"] == "tree":
        new, old = _uneven(case["new"], case["seqs"]), _uneven(case["old"], case["seqs"])
        N, x = sum(new), 4 if case["x"] == "f32" else 2
        seen = [min(o, case["window"]) if case["window"] else o for o in old]
        mean = 1 + 2 * case["new"] / (case["branch"] + 1) / 2  # ancestors of a token, and itself
        return {"bytes": 2 * N * n_q * dim * x + 2 * sum(s + n for s, n in zip(seen, new)) * n_kv * dim * value,
                "flops": 4 * sum(n * (s + min(mean, n)) for s, n in zip(seen, new)) * n_q * dim}
    if case["op"] == "copy":
        tokens = case["pages"] * case["page"] * (1 if case["whole"] else 0.5)
        held = case["pool"] * case["page"]
    else:
        tokens = sum(max(0, k - min(case["sinks"], k)) for k in _uneven(case["kept"], case["seqs"]))
        lens = [case["old"] // (1 + s % 3) + n for s, n in enumerate(_uneven(case["new"], case["seqs"], 2 * case["kept"] + 8))]
        held = sum(-(-n // case["page"]) * case["page"] for n in lens)
    total = 2 * case["layers"] * tokens * n_kv * dim * value * 2 + 8 * case.get("pages", 0) + 4 * tokens * (case["op"] == "keep")
    if case["cache"] == "q8_0":  # the pages' values are read back as fp32
        total += 2 * case["layers"] * held * n_kv * dim * (value + 4)
    return {"bytes": total, "flops": 0}


def exact(case, seed):
    st = prepare(case, seed)
    return {"tree": _tree_exact, "keep": _moved_exact, "copy": _moved_exact, "logprobs": _logprobs_exact}[case["op"]](st)


def _values64(cache, pages):
    if cache != "q8_0":
        return pages.double()
    rows = pages.reshape(-1, 34)
    scale = rows[:, :2].clone().view(torch.float16).double()
    code = rows[:, 2:].double()
    code = code - 256 * (code > 127)
    return (scale * code).reshape(*pages.shape[:-1], -1)


def _moved_exact(st):
    case, page = st["case"], st["case"]["page"]
    moves, lens = [], []  # (page, row) that a row comes from, and where it goes
    if case["op"] == "copy":
        rows = [page] * case["pages"] if st["rows"] is None else st["rows"].tolist()
        for a, b, n in zip(st["src"].tolist(), st["dst"].tolist(), rows):
            moves += [(a, j, b, j) for j in range(n)]
    else:
        table, keep = st["table"].tolist(), st["keep"].tolist()
        for s, (f, n) in enumerate(zip(st["first"].tolist(), st["n_keep"].tolist())):
            moves += [(table[s][a // page], a % page, table[s][(f + i) // page], (f + i) % page) for i, a in enumerate(keep[s][:n])]
            lens.append(f + n)
    moves = torch.tensor(moves, device="cuda").T
    out = [_ints(lens)] if lens else []
    for c in ("k", "v"):
        pool = st[c].transpose(2, 3).contiguous()  # layers, pages, rows, heads, values
        flat = pool.view(pool.shape[0], -1, *pool.shape[3:])
        flat.index_copy_(1, moves[2] * page + moves[3], flat.index_select(1, moves[0] * page + moves[1]))
        out.append(_values64(case["cache"], pool.transpose(2, 3)))
    return out


def _logprobs_exact(st):
    case = st["case"]
    given, entropy, ids, top = [], [], [], []
    for part, tokens in zip(st["logits"].split(64), st["tokens"].long().split(64)):
        x = part.double()
        order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :case["top"]]
        if case["cap"]:
            x = torch.tanh(x / case["cap"]) * case["cap"]
        lp = torch.log_softmax(x * case["scale"], 1)
        given.append(lp.gather(1, tokens))
        entropy.append(-(lp.exp() * lp).sum(1))
        ids.append(order.int())
        top.append(lp.gather(1, order))
    out = [torch.cat(given)] if case["given"] else []
    out.append(torch.cat(entropy))
    return out + ([torch.cat(ids), torch.cat(top)] if case["top"] else [])


def _tree_exact(st):
    case, n_kv, dim = st["case"], st["n_kv"], st["dim"]
    G = st["n_q"] // n_kv
    starts, lens, parents = st["q_start"].tolist(), st["kv_len"].tolist(), st["parents"].tolist()
    out = torch.zeros(st["N"], st["n_q"], dim, dtype=torch.float64, device="cuda")
    for s, L in enumerate(lens):
        a, b = starts[s], starts[s + 1]
        o = L - (b - a)
        seen = torch.zeros(b - a, L, dtype=torch.bool)
        seen[:, :o] = True
        place = torch.arange(L)
        for i, p in enumerate(parents[a:b]):
            place[o + i] = o if p < 0 else place[o + p] + 1
            j = i
            while j >= 0:
                seen[i, o + j] = True
                j = parents[a + j]
        gap = (place[o:, None] - place[None]).cuda()
        seen = seen.cuda()
        if case["window"]:
            seen &= gap < case["window"]
        pages = st["table"][s, :-(-L // case["page"])].long()
        for h in range(n_kv):
            k, v = (_values64(case["cache"], st[c][pages, h]).reshape(-1, dim)[:L] for c in ("k", "v"))
            for g in range(G):
                head = h * G + g
                w = st["q"][a:b, head].double() @ k.T / math.sqrt(dim)
                if case["cap"]:
                    w = case["cap"] * torch.tanh(w / case["cap"])
                if st["slopes"] is not None:
                    w = w - float(st["slopes"][head]) * gap.abs()
                w = torch.softmax(torch.where(seen, w, -math.inf), 1)
                out[a:b, head] = w @ v
    return out
