"""What is measured of the key-value cache operators: appending rotated keys
and values to a paged cache (Q8_0, F16 or BF16 rows), and attention over such
a cache for single new tokens and for prompts.

The cache: two arrays of pages, keys and values.  A page holds, for each
key-value head, `page_size` rows of head_dim values one after another, each a
run of Q8_0 blocks (fp16 d, 32 int8 codes) or of 16-bit floats.  A batch is a
run of token rows: sequence s has rows q_start[s] .. q_start[s+1]-1, its cache
holds kv_len[s] tokens with these new ones at its end, and its token j lies in
row j % page_size of page table[s][j // page_size].
"""
import math

import torch

own = False

DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}

# Head layouts: the 8B model's (4096 = 32 x 128, 8 key-value heads), the 1B
# model's (2048 = 32 x 64, 8), the 896-wide one's (14 x 64, 2), one with a
# head per key-value head, and one of wide heads.
HEADS = {"8b": (32, 8, 128), "1b": (32, 8, 64), "0.5b": (14, 2, 64), "one each": (32, 32, 128), "wide": (16, 8, 256)}


def listed():
    def append(name, **k):
        return dict(name=name, op="append", **k)

    def attn(name, **k):
        base = dict(cap=0.0, window=0, slopes=False, prefix=0)
        base.update(k)
        return dict(name=name, op="attn", **base)

    return [
        # the next token of one conversation: latency alone
        append("append, one token", heads="8b", x="f32", cache="f16", seqs=1, new=1, old=1003, page=32, pairing="pairs", axes=1, rot=128),
        # a decode step of a batch of image-and-text conversations: three position axes
        append("append, 48 sequences", heads="one each", x="bf16", cache="bf16", seqs=48, new=1, old=2011, page=16, pairing="halves", axes=3, rot=128),
        # prompts of uneven lengths stored as Q8_0, half of each head rotated
        append("append, prompts", heads="8b", x="f32", cache="q8_0", seqs=5, new=1733, old=0, page=64, pairing="halves", axes=1, rot=64),
        # the first answers of a short conversation on the smallest model: latency
        attn("decode, short", heads="0.5b", x="f32", cache="q8_0", seqs=1, new=1, old=36, page=16),
        # one conversation at the end of a long context: the length is split
        attn("decode, one long", heads="8b", x="f32", cache="q8_0", seqs=1, new=1, old=130911, page=128),
        # one key-value head per head, a bias by distance
        attn("decode, slopes", heads="one each", x="f32", cache="bf16", seqs=13, new=1, old=1499, page=32, slopes=True),
        # wide heads with capped scores, uneven lengths
        attn("decode, capped", heads="wide", x="bf16", cache="f16", seqs=32, new=1, old=4095, page=64, cap=50.0),
        # a full batch of long conversations: bandwidth
        attn("decode, full", heads="8b", x="f32", cache="q8_0", seqs=64, new=1, old=16383, page=64),
        # a short question behind a cached document
        attn("prompt, behind a cache", heads="1b", x="f32", cache="q8_0", seqs=1, new=61, old=1940, page=16),
        # an ordinary prompt
        attn("prompt, 2048", heads="8b", x="f32", cache="q8_0", seqs=1, new=2048, old=0, page=64),
        # prompts of uneven lengths, each with an image first that all its tokens see; capped scores, a window
        attn("prompt, prefix and window", heads="8b", x="bf16", cache="bf16", seqs=4, new=2200, old=0, page=32, cap=30.0, window=1024, prefix=256),
        # a long document at once
        attn("prompt, long", heads="8b", x="bf16", cache="f16", seqs=1, new=8191, old=0, page=128),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    c = {"heads": rng.choice(sorted(HEADS)), "x": rng.choice(["f32", "bf16"]), "cache": rng.choice(["q8_0", "f16", "bf16"]),
         "page": rng.choice([16, 32, 48, 64, 128, 256])}
    n_q, n_kv, dim = HEADS[c["heads"]]
    kind = rng.choice(["append", "decode", "prompt"])
    if kind == "append":
        tokens = _spread(rng, 1, 6000)
        seqs = min(tokens, _spread(rng, 1, 64))
        axes = rng.choice([1, 1, 3])
        c.update(op="append", seqs=seqs, new=max(1, tokens // seqs), old=_spread(rng, 1, 4000) - 1,
                 pairing=rng.choice(["pairs", "halves"]), axes=axes, rot=rng.choice([dim, dim // 2]))
        return c
    c.update(op="attn", cap=rng.choice([0.0, 0.0, 30.0, 50.0]), window=rng.choice([0, 0, 0, _spread(rng, 16, 4096)]), slopes=rng.random() < 0.25, prefix=0)
    if kind == "decode":
        seqs = _spread(rng, 1, 64)
        keys = _spread(rng, 1, min(130000, 64 * 16384 * 1024 // (seqs * n_kv * dim)))
        c.update(seqs=seqs, new=1, old=keys - 1)
    else:
        new = _spread(rng, 2, 4000)
        seqs = rng.choice([1, 1, 2, 3])
        c.update(seqs=seqs, new=max(2, new // seqs), old=rng.choice([0, 0, _spread(rng, 1, 2000)]), prefix=rng.choice([0, 0, _spread(rng, 1, 600)]))
    return c


def _lengths(case):
    """New tokens and cached tokens of each sequence: a batch is uneven (down to a half of the longest)."""
    new, old = [], []
    for i in range(case["seqs"]):
        f = (i * 0.6180339887) % 1.0 * 0.5
        new.append(max(1, case["new"] - int(case["new"] * f)))
        old.append(case["old"] - int(case["old"] * f))
    return new, old


def _slopes(n_q, device):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / n_q) for h in range(n_q)], device=device)


def _q8_0_bytes(x):
    """Rows of fp32 values as Q8_0 blocks: d = amax / 127, codes round(x * (1 / d)) with halves away from 0, d stored as fp16."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    d = (amax.double() / torch.full_like(amax, 127, dtype=torch.float64)).float()
    inv = torch.where(d != 0, d.double().reciprocal().float(), torch.zeros_like(d))
    t = b * inv
    codes = (torch.sign(t).double() * torch.floor(t.double().abs() + 0.5)).clamp(-127, 127).to(torch.int8)
    out = torch.cat([d.half().view(torch.uint8), codes.view(torch.uint8)], -1)
    return out.reshape(*x.shape[:-1], -1)


def _rows(cache, pages):
    """The values that a cache array holds, as fp32."""
    if cache != "q8_0":
        return pages.float()
    b = pages.reshape(*pages.shape[:-1], -1, 34)
    d = b[..., :2].contiguous().view(torch.float16).float()
    return (b[..., 2:].contiguous().view(torch.int8).float() * d).flatten(-2)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n_q, n_kv, dim = HEADS[case["heads"]]
    page, cache = case["page"], case["cache"]
    new, old = _lengths(case)
    lens = [a + b for a, b in zip(new, old)]
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    N = starts[-1]
    width = -(-max(lens) // page)
    # an append touches the pages of its new tokens alone; the table's earlier entries name pages of others
    first = [o // page if case["op"] == "append" else 0 for o in old]
    owned = [-(-n // page) - f for n, f in zip(lens, first)]
    n_pages = sum(owned) + (2 if case["op"] == "attn" else 0)
    order = torch.randperm(n_pages, device="cuda", generator=g).to(torch.int32)
    table = torch.zeros(case["seqs"], width, dtype=torch.int32, device="cuda")
    at = 0
    for s in range(case["seqs"]):
        table[s, first[s]:first[s] + owned[s]] = order[at:at + owned[s]]
        at += owned[s]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, device="cuda", generator=g).to(dtype)

    def pool(spread):
        if case["op"] == "append":
            row = dim // 32 * 34 if cache == "q8_0" else dim
            return torch.zeros(n_pages, n_kv, page, row, device="cuda", dtype=torch.uint8 if cache == "q8_0" else DTYPE[cache])
        x = normal(n_pages, n_kv, page, dim) * spread
        return _q8_0_bytes(x) if cache == "q8_0" else x.to(DTYPE[cache])

    st = {"case": case, "n_q": n_q, "n_kv": n_kv, "dim": dim, "N": N, "new": max(new), "kv": max(lens),
          "q_start": torch.tensor(starts, dtype=torch.int32, device="cuda"),
          "kv_len": torch.tensor(lens, dtype=torch.int32, device="cuda"),
          "table": table, "k": pool(1.0), "v": pool(1.0), "q": normal(N, n_q, dim, dtype=DTYPE[case["x"]])}
    if case["op"] == "append":
        st["new_k"], st["new_v"] = (normal(N, n_kv, dim, dtype=DTYPE[case["x"]]) for _ in range(2))
        half = case["rot"] // 2
        st["freqs"] = 500000.0 ** (-2.0 * torch.arange(half, dtype=torch.float64, device="cuda") / case["rot"])
        st["pos"], st["sections"] = None, None
        if case["axes"] == 3:
            st["sections"] = [half - 2 * (half * 3 // 8), half * 3 // 8, half * 3 // 8]
            st["pos"] = torch.randint(0, max(lens), (3, N), generator=g, device="cuda", dtype=torch.int32)
    else:
        st["slopes"] = _slopes(n_q, "cuda") if case["slopes"] else None
        st["prefix"] = torch.tensor([min(case["prefix"], n) for n in lens], dtype=torch.int32, device="cuda") if case["prefix"] else None
    return st


def run(st):
    case = st["case"]
    if own:
        return _run_own(st)
    return _append_plain(st) if case["op"] == "append" else _attn_plain(st)


def _run_own(st):
    import block_quantized_amd as Q
    case = st["case"]
    if "handle" not in st:  # what a program keeps over all layers and steps
        kind = {"q8_0": Q.QMM_Q8_0, "f16": Q.QMM_F16, "bf16": Q.QMM_BF16}[case["cache"]]
        st["handle"] = Q.KVCache(st["k"], st["v"], kind, st["n_kv"], st["dim"], case["page"])
        st["batch"] = Q.KVBatch(st["q_start"], st["kv_len"], st["table"], st["N"], max_kv=st["kv"])
        if case["op"] == "append":
            pairing = Q.QMM_ROPE_PAIRS if case["pairing"] == "pairs" else Q.QMM_ROPE_HALVES
            st["rope"] = Q.Rope(st["freqs"], pairing, pos=st["pos"], sections=st["sections"])
    if case["op"] == "append":
        q = Q.kv_append(st["handle"], st["batch"], st["new_k"], st["new_v"], q=st["q"], rope=st["rope"])
        if case["cache"] != "q8_0":
            return q, st["k"], st["v"]
        rows = st["k"].numel() // st["k"].shape[-1]
        return [q] + [Q.dequantize(Q.QMM_Q8_0, c, rows, st["dim"]).view(*c.shape[:-1], st["dim"]) for c in (st["k"], st["v"])]
    return Q.attn(st["handle"], st["batch"], st["q"], scale=st["dim"] ** -0.5, softcap=case["cap"], window=case["window"],
                  slopes=st["slopes"], prefix=st["prefix"])


def _append_plain(st):
    case = st["case"]
    N, page, rot = st["N"], case["page"], case["rot"]
    t = torch.arange(N, device="cuda")
    seq = torch.searchsorted(st["q_start"][1:].contiguous(), t.int(), right=True)
    at = (st["kv_len"] - st["q_start"][1:])[seq] + t  # index in the sequence
    pos = at[None] if st["pos"] is None else st["pos"]
    axis = torch.zeros(rot // 2, dtype=torch.long, device="cuda")
    if st["sections"] is not None:
        i = torch.arange(rot // 2, device="cuda")
        axis = (i >= st["sections"][0]).long() + (i >= st["sections"][0] + st["sections"][1]).long()
    angle = pos.double()[axis].T * st["freqs"]
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]

    def turn(x):  # angles and products in 64 bits: the stored codes lie next to rounding borders
        y = x.double().clone()
        if case["pairing"] == "pairs":
            a, b = x[..., 0:rot:2].double(), x[..., 1:rot:2].double()
            y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
        else:
            a, b = x[..., :rot // 2].double(), x[..., rot // 2:rot].double()
            y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
        return y.float()

    where = st["table"][seq, at // page].long()
    for name, x in (("k", turn(st["new_k"])), ("v", st["new_v"].float())):
        st[name][where, :, at % page] = _q8_0_bytes(x) if case["cache"] == "q8_0" else x.to(DTYPE[case["cache"]])
    q = turn(st["q"]).to(DTYPE[case["x"]])
    if case["cache"] != "q8_0":
        return q, st["k"], st["v"]
    return [q, _rows("q8_0", st["k"]), _rows("q8_0", st["v"])]


def _attn_plain(st):
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
    p = (st["kv_len"] - n)[:, None] + i  # B, T
    j = torch.arange(L, device="cuda")
    gap = p[:, :, None] - j
    if st["slopes"] is not None:
        s = s - st["slopes"].view(1, n_kv, G, 1, 1) * gap.abs()[:, None, None]
    seen = gap >= 0
    if case["window"]:
        seen = seen & (gap < case["window"])
    if st["prefix"] is not None:
        seen = seen | (j < st["prefix"][:, None, None])
    seen = (seen & (j < st["kv_len"][:, None, None]))[:, None, None]
    s = s.masked_fill(~seen, -math.inf)
    w = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e30))
    o = torch.matmul(w.view(B, n_kv, G * T, L), v) / w.sum(-1).clamp(min=1e-30).view(B, n_kv, G * T, 1)
    o = o.view(B, n_kv, G, T, dim).permute(0, 3, 1, 2, 4).reshape(B, T, st["n_q"], dim)
    out = torch.zeros(st["N"] + 1, st["n_q"], dim, device="cuda", dtype=DTYPE[case["x"]])
    out[row] = o.to(out.dtype)
    return out[:st["N"]]


def _visible(case):
    """Pairs of a token and a key that it sees, and keys that any token sees, over all sequences."""
    pairs = keys = 0
    for n, o in zip(*_lengths(case)):
        first = o + n
        for p in range(o, o + n):
            lo = max(0, p - case["window"] + 1) if case["window"] else 0
            pre = min(case["prefix"], o + n)
            pairs += p + 1 - lo + (min(pre, lo) + max(0, pre - p - 1))
            first = min(first, lo)
        keys += o + n - first + min(min(case["prefix"], o + n), first)
    return pairs, keys


def work(case):
    n_q, n_kv, dim = HEADS[case["heads"]]
    new, _ = _lengths(case)
    N, x = sum(new), 4 if case["x"] == "f32" else 2
    value = 34 / 32 if case["cache"] == "q8_0" else 2
    if case["op"] == "append":
        total = N * dim * (2 * n_q * x + 2 * n_kv * (x + value))
        if case["cache"] == "q8_0":  # the pages' values are read back as fp32
            _, old = _lengths(case)
            rows = sum(-(-(a + b) // case["page"]) - b // case["page"] for a, b in zip(new, old)) * case["page"] * n_kv
            total += 2 * rows * dim * (value + 4)
        return {"bytes": total, "flops": N * (n_q + n_kv) * case["rot"] * 3}
    pairs, keys = _visible(case)
    return {"bytes": 2 * N * n_q * dim * x + 2 * keys * n_kv * dim * value, "flops": 4 * pairs * n_q * dim}


def exact(case, seed):
    st = prepare(case, seed)
    return _append_exact(st) if case["op"] == "append" else _attn_exact(st)


def _values64(cache, pages):
    if cache != "q8_0":
        return pages.double()
    rows = pages.reshape(-1, 34)
    scale = rows[:, :2].clone().view(torch.float16).double()
    code = rows[:, 2:].double()
    code = code - 256 * (code > 127)
    return (scale * code).reshape(*pages.shape[:-1], -1)


def _append_exact(st):
    case, rot, page = st["case"], st["case"]["rot"], st["case"]["page"]
    new, old = _lengths(case)
    at = torch.cat([torch.arange(o, o + n, dtype=torch.float64, device="cuda") for n, o in zip(new, old)])
    freq = torch.exp(torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") * (-math.log(500000.0) / rot))
    if st["sections"] is None:
        angle = torch.outer(at, freq)
    else:
        parts = torch.split(freq, st["sections"])
        angle = torch.cat([torch.outer(st["pos"][a].double(), f) for a, f in enumerate(parts)], 1)
    unit = torch.polar(torch.ones_like(angle), angle)[:, None]

    def turned(x):
        x = x.double()
        head, rest = x[..., :rot], x[..., rot:]
        if case["pairing"] == "pairs":
            z = torch.view_as_complex(head.reshape(*head.shape[:-1], -1, 2).contiguous()) * unit
            head = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(head[..., :rot // 2], head[..., rot // 2:]) * unit
            head = torch.cat([z.real, z.imag], -1)
        return torch.cat([head, rest], -1)

    def stored(x):
        if case["cache"] != "q8_0":
            return x
        b = x.float().double().reshape(*x.shape[:-1], -1, 32)  # a row is quantized from its fp32 values
        d = (b.abs().amax(-1, keepdim=True) / torch.tensor(127.0, dtype=torch.float64, device="cuda")).float()
        inv = (1.0 / d.double()).float().double()
        t = (b * inv).float().double()
        code = torch.where(t < 0, torch.ceil(t - 0.5), torch.floor(t + 0.5))
        return (torch.where(d > 0, code, 0.0) * d.half().double()).flatten(-2)

    def cache(x):
        out = torch.zeros(*st["k"].shape[:3], st["dim"], dtype=torch.float64, device="cuda")
        x, a = stored(x), 0
        for s, (n, o) in enumerate(zip(new, old)):
            j = torch.arange(o, o + n, device="cuda")
            out[st["table"][s].long()[j // page], :, j % page] = x[a:a + n]
            a += n
        return out

    return [turned(st["q"]), cache(turned(st["new_k"])), cache(st["new_v"].double())]


def _attn_exact(st):
    case, n_kv, dim = st["case"], st["n_kv"], st["dim"]
    G = st["n_q"] // n_kv
    new, old = _lengths(case)
    out = torch.zeros(st["N"], st["n_q"], dim, dtype=torch.float64, device="cuda")
    a = 0
    for s, (n, o) in enumerate(zip(new, old)):
        L = n + o
        pages = st["table"][s, :-(-L // case["page"])].long()
        p = torch.arange(o, L, device="cuda")
        j = torch.arange(L, device="cuda")
        seen = (j[None] <= p[:, None])
        if case["window"]:
            seen &= j[None] > p[:, None] - case["window"]
        if st["prefix"] is not None:
            seen |= (j < int(st["prefix"][s]))[None]
        for h in range(n_kv):
            k, v = (_values64(case["cache"], st[c][pages, h]).reshape(-1, dim)[:L] for c in ("k", "v"))
            for g in range(G):
                head = h * G + g
                w = st["q"][a:a + n, head].double() @ k.T / math.sqrt(dim)
                if case["cap"]:
                    w = case["cap"] * torch.tanh(w / case["cap"])
                if st["slopes"] is not None:
                    w = w - float(st["slopes"][head]) * (p[:, None] - j[None]).abs()
                w = torch.softmax(torch.where(seen, w, -math.inf), 1)
                out[a:a + n, head] = w @ v
        a += n
    return out
