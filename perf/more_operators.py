"""A decode loop's attention and choice of the next token, measured operator by operator.

append  rotary positions on queries and keys, keys and values written into a paged cache, in bf16 or as 8-bit
        rows with a scale each (Moe.kv_append); an 8-bit cache's rows are read back, as the values they stand for
read    rows of the cache as bf16 (Moe.kv_read)
attend  attention of one new token per sequence over the paged cache (Moe.kv_attend)
sample  temperature, min-p, top-k, top-p and the token that a given random number picks (Moe.sample)

`run` computes them with elementary torch operations, or with the library where `own` is true.
"""
import math

import torch

own = False

_DEV = "cuda"


def listed():
    return [
        # one new token of one sequence: queries and keys rotated, the cache extended
        {"name": "append one token", "op": "append", "seqs": 1, "rows": 1, "start": 1000, "q_heads": 16, "kv_heads": 8,
         "dim": 256, "page": 64, "rot": 256, "bits8": False},
        # one new token of each sequence of a batch, an 8-bit cache
        {"name": "append batch", "op": "append", "seqs": 64, "rows": 64, "start": 3000, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "page": 64, "rot": 128, "bits8": True},
        # a whole prompt, written in 8 bits and read back for the prompt's own attention
        {"name": "append prompt", "op": "append", "seqs": 1, "rows": 4096, "start": 0, "q_heads": 16, "kv_heads": 8,
         "dim": 256, "page": 64, "rot": 256, "bits8": True},
        # a long shared prefix taken out of the cache, ahead of a prompt's next chunk
        {"name": "read prefix", "op": "read", "seqs": 1, "rows": 32768, "kv_heads": 8, "dim": 128, "page": 64,
         "bits8": True},
        # rows of several sequences at odd sizes, a bf16 cache of short pages
        {"name": "read ragged", "op": "read", "seqs": 13, "rows": 1777, "kv_heads": 3, "dim": 80, "page": 16,
         "bits8": False},
        # one sequence, a context of 4096: latency
        {"name": "attend one sequence", "op": "attend", "seqs": 1, "length": 4096, "q_heads": 16, "kv_heads": 8,
         "dim": 256, "page": 64, "window": 0, "softcap": 0.0, "bits8": False, "even": True},
        # a batch in a layer with a sliding window
        {"name": "attend window", "op": "attend", "seqs": 64, "length": 8192, "q_heads": 16, "kv_heads": 8, "dim": 256,
         "page": 64, "window": 1024, "softcap": 0.0, "bits8": True, "even": False},
        # a batch of long sequences: the memory's rate
        {"name": "attend batch long", "op": "attend", "seqs": 32, "length": 32768, "q_heads": 32, "kv_heads": 4,
         "dim": 128, "page": 64, "window": 0, "softcap": 0.0, "bits8": True, "even": False},
        # odd sizes: three queries to a key, capped scores, empty sequences and sequences of one token
        {"name": "attend ragged", "op": "attend", "seqs": 23, "length": 1999, "q_heads": 9, "kv_heads": 3, "dim": 80,
         "page": 16, "window": 0, "softcap": 50.0, "bits8": False, "even": False},
        # the next token of one sequence
        {"name": "sample one row", "op": "sample", "rows": 1, "vocab": 262144, "pad": 0, "spread": 3.0},
        # a batch of sequences, each with filters of its own
        {"name": "sample batch", "op": "sample", "rows": 64, "vocab": 262144, "pad": 0, "spread": 3.0},
        # an odd vocabulary in padded rows
        {"name": "sample ragged", "op": "sample", "rows": 17, "vocab": 100003, "pad": 13, "spread": 2.0},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend", "sample", "sample"])
    kv, dim = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 64, 80, 96, 128, 128, 192, 256, 256])
    pages = {"kv_heads": kv, "dim": dim, "page": rng.choice([16, 32, 64, 128, 256]), "bits8": rng.random() < 0.5}
    if op == "append":
        decode = rng.random() < 0.5
        rows = _spread(rng, 1, 128 if decode else 4096)
        return {"op": op, "seqs": rows if decode else 1, "rows": rows, "start": _spread(rng, 1, 100000) if decode else 0,
                "q_heads": kv * rng.choice([1, 2, 3, 4]), "rot": rng.choice([0, dim, dim, 16 * (dim // 32)]), **pages}
    if op == "read":
        seqs = _spread(rng, 1, 64)
        return {"op": op, "seqs": seqs, "rows": max(seqs, _spread(rng, 1, 16384)), **pages}
    if op == "attend":
        while True:
            seqs, length, heads = _spread(rng, 1, 256), _spread(rng, 1, 65536), kv * rng.choice([1, 2, 3, 5, 8, 16])
            if seqs * length * dim * max(8 * kv * (1 if pages["bits8"] else 2), heads) <= 32 * 32768 * 128 * 32:
                return {"op": op, "seqs": seqs, "length": length, "q_heads": heads,
                        "window": rng.choice([0, 0, _spread(rng, 1, 4096)]), "softcap": rng.choice([0.0, 0.0, 50.0]),
                        "even": rng.random() < 0.3, **pages}
    return {"op": op, "rows": _spread(rng, 1, 64), "vocab": _spread(rng, 1000, 262144), "pad": rng.choice([0, 0, 5, 16]),
            "spread": rng.choice([2.0, 3.0, 4.0])}


# ------------------------------------------------------------------ inputs
def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=_DEV)


def _pool(g, st, n_pages):
    """Pages that hold rows of earlier steps: bell-shaped values, a few channels of the keys that stand out."""
    shape = (n_pages, st["kv_heads"], st["page"], st["dim"])
    for name in ("k", "v"):
        x = torch.empty(shape, dtype=torch.int8 if st["bits8"] else torch.bfloat16, device=_DEV)
        scales = torch.empty(shape[:3], dtype=torch.float32, device=_DEV) if st["bits8"] else None
        big = 1.0 + 4.0 * (torch.rand(st["dim"], generator=g, device=_DEV) > 0.97) if name == "k" else 1.0
        step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
        for a in range(0, n_pages, step):
            f = _randn(g, min(step, n_pages - a), *shape[1:]) * big
            if st["bits8"]:
                m = f.abs().amax(-1)
                x[a:a + step] = torch.round(f * (127.0 / m)[..., None]).to(torch.int8)
                scales[a:a + step] = m / 127.0
            else:
                x[a:a + step] = f.to(torch.bfloat16)
        st[name + "_pages"], st[name + "_scales"] = x, scales


def prepare(case, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(int(seed))
    st = dict(case)
    if case["op"] == "sample":
        T, V = case["rows"], case["vocab"]
        # most tokens are unlikely, a few hundred fit the text
        hot = 6.0 * (torch.rand((T, V + case["pad"]), generator=g, device=_DEV) < 300.0 / V)
        st["logits"] = (_randn(g, T, V + case["pad"]) * case["spread"] + hot)[:, :V]
        share = torch.rand((4, T), generator=g, device=_DEV)
        kind = torch.arange(T, device=_DEV) % 4  # the sequences' filters differ: top-k and top-p, top-p, min-p, top-k
        st["uniform"] = share[0]
        st["temperature"] = 0.6 + 0.6 * share[1]
        st["top_k"] = torch.where((kind == 0) | (kind == 3), (10.0 + 90.0 * share[2]).to(torch.int32), 0).to(torch.int32)
        st["top_p"] = torch.where(kind < 2, 0.8 + 0.19 * share[3], 1.0)
        st["min_p"] = torch.where(kind == 2, 0.02 + 0.1 * share[3], 0.0)
        st["tokens"] = torch.empty(T, dtype=torch.int32, device=_DEV)
        st["logprobs"] = torch.empty(T, dtype=torch.float32, device=_DEV)
        return st
    n, D, Hkv, page = case["seqs"], case["dim"], case["kv_heads"], case["page"]
    if case["op"] == "attend":
        L = case["length"]
        if case["even"]:
            lengths = torch.full((n,), L, device=_DEV)
        else:  # anything up to the longest, short ones too; a slot without a sequence, one that has just begun
            lengths = (L * torch.rand(n, generator=g, device=_DEV) ** 0.5).ceil().clamp(min=1)
            lengths[0] = L
            if n > 4:
                lengths[n // 2], lengths[n // 3] = 0, 1
        st["lengths"] = lengths.to(torch.int32)
        st["q"] = (_randn(g, n, case["q_heads"], D) * 1.5).to(torch.bfloat16)
        st["out"] = torch.empty_like(st["q"])
        st["scale"] = 1.0 / math.sqrt(D)
        last = L
    else:
        T, Hq = case["rows"], case.get("q_heads", 0)
        if case["op"] == "append" and n == T:  # a token each, at different places
            st["seq"] = torch.arange(n, device=_DEV, dtype=torch.int32)
            st["pos"] = (case["start"] * (1.0 - 0.5 * torch.rand(n, generator=g, device=_DEV))).to(torch.int32)
            last = case["start"] + 1
        else:  # runs of rows
            at = torch.arange(T, device=_DEV, dtype=torch.int32)
            st["seq"] = at % n
            st["pos"] = at // n + case.get("start", 0)
            last = (T + n - 1) // n + case.get("start", 0)
        if case["op"] == "append":
            # the projections' output: queries, keys and values of a token side by side
            st["qkv"] = _randn(g, T, (Hq + 2 * Hkv) * D).to(torch.bfloat16)
            st["q_out"] = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=_DEV)
            r = case["rot"]
            st["freq"] = 10000.0 ** (-torch.arange(0, r, 2, device=_DEV) / r) if r else None
        st["k_out"] = torch.empty((T, Hkv, D), dtype=torch.bfloat16, device=_DEV)
        st["v_out"] = torch.empty_like(st["k_out"])
    per = (last + page - 1) // page
    if case["op"] == "append" and n == st["rows"]:  # the pages that the tokens go to, and a few more
        pool = n + 3
        st["table"] = torch.zeros((n, per), dtype=torch.int32, device=_DEV)
        order = torch.randperm(pool, generator=g, device=_DEV)[:n].to(torch.int32)
        st["table"][st["seq"].long(), st["pos"].long() // page] = order
    else:
        pool = n * per + 3
        st["table"] = torch.randperm(pool, generator=g, device=_DEV)[:n * per].reshape(n, per).to(torch.int32)
    _pool(g, st, pool)
    return st


# ------------------------------------------------------------------ the plain forms
def _rotate(x, pos, freq, rot):
    """The first `rot` dimensions of heads x [T, H, D] turned by their rows' angles, in 32 bits."""
    f = x.float()
    if not rot:
        return f
    angle = pos.double()[:, None] * freq.double()
    c, s = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    a, b = f[..., :rot // 2], f[..., rot // 2:rot]
    return torch.cat([a * c - b * s, b * c + a * s, f[..., rot:]], -1)


def _split(st):
    """Queries, keys and values [T, heads, dim] of the rows, without a copy."""
    T, Hq, Hkv, D = st["rows"], st["q_heads"], st["kv_heads"], st["dim"]
    q, k, v = st["qkv"].split((Hq * D, Hkv * D, Hkv * D), 1)
    return q.unflatten(1, (Hq, D)), k.unflatten(1, (Hkv, D)), v.unflatten(1, (Hkv, D))


def _place(st):
    """Page and row in it of the state's rows."""
    pos = st["pos"].long()
    return st["table"][st["seq"].long(), pos // st["page"]].long(), pos % st["page"]


def _rows_of(st, name, page, row):
    """Rows [T, heads, dim] of the cache, in 32 bits."""
    x = st[name + "_pages"][page, :, row].float()
    return x * st[name + "_scales"][page, :, row][..., None] if st["bits8"] else x


def _append_plain(st):
    q, k, v = _split(st)
    page, row = _place(st)
    got = {"q": _rotate(q, st["pos"], st["freq"], st["rot"]).to(torch.bfloat16)}
    for name, x in (("k", _rotate(k, st["pos"], st["freq"], st["rot"])), ("v", v.float())):
        if st["bits8"]:
            m = x.abs().amax(-1, keepdim=True)
            st[name + "_pages"][page, :, row] = torch.where(m > 0, torch.round(x * 127.0 / m), 0.0).to(torch.int8)
            st[name + "_scales"][page, :, row] = m[..., 0] / 127.0
            got[name] = _rows_of(st, name, page, row).to(torch.bfloat16)
        else:
            st[name + "_pages"][page, :, row] = x.to(torch.bfloat16)
            got[name + "_pages"] = st[name + "_pages"]
    return got


def _read_plain(st):
    page, row = _place(st)
    return {name: _rows_of(st, name, page, row).to(torch.bfloat16) for name in ("k", "v")}


def _attend_plain(st):
    n, Hq, Hkv, D, page = st["seqs"], st["q_heads"], st["kv_heads"], st["dim"], st["page"]
    most = st["table"].shape[1] * page
    length, window = st["lengths"].long()[:, None], min(st["window"] or most, most)
    at = (length - window).clamp(min=0) + torch.arange(window, device=_DEV)  # the positions that a window spans
    seen = at < length
    at = at.clamp(max=most - 1)
    where = st["table"].gather(1, at // page).long(), at % page
    heads = []
    for name in ("k", "v"):  # [n, heads, positions, dim]
        x = st[name + "_pages"][where[0], :, where[1]].float()
        if st["bits8"]:
            x *= st[name + "_scales"][where[0], :, where[1]][..., None]
        heads.append(x.transpose(1, 2))
    q = st["q"].float().reshape(n, Hkv, Hq // Hkv, D)
    s = (q @ heads[0].transpose(2, 3)) * st["scale"]
    if st["softcap"]:
        s = st["softcap"] * torch.tanh(s / st["softcap"])
    s = torch.where(seen[:, None, None], s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m > -math.inf, m, 0.0))
    total = p.sum(-1, keepdim=True)
    o = (p @ heads[1]) / torch.where(total > 0, total, 1.0)
    return {"out": o.reshape(n, Hq, D).to(torch.bfloat16)}


def _sample_plain(st):
    l = st["logits"]
    T, V = l.shape
    t, p = st["temperature"].double()[:, None], st["top_p"].double()[:, None]
    best = l.double().amax(1, keepdim=True)
    keep = l.double() - best >= t * torch.log(st["min_p"].double()[:, None])
    w = torch.where(keep, torch.exp((l.double() - best) / t), 0.0)
    value, order = torch.sort(l, dim=1, descending=True, stable=True)  # ties: the lower id first
    w = w.gather(1, order)
    rank = torch.arange(V, device=_DEV)
    k = st["top_k"][:, None]
    w = torch.where((k <= 0) | (rank < k), w, 0.0)
    mass = w.cumsum(1)
    # a token stays while the mass before it is short of the share
    w = torch.where((p >= 1.0) | (mass - w < p * mass[:, -1:]) | (rank == 0), w, 0.0)
    w = torch.zeros_like(w).scatter_(1, order, w)
    mass = w.cumsum(1)
    over = (mass > st["uniform"].double()[:, None] * mass[:, -1:]) & (w > 0)
    token = torch.where(over, rank, V).amin(1)
    return {"tokens": token.to(torch.int32),
            "logprobs": torch.log(w.gather(1, token[:, None]) / mass[:, -1:])[:, 0].float()}


# ------------------------------------------------------------------ the framework's operators
_handle = []


def _moe():
    import bit_affine_quantized_gb300 as bq
    if not _handle:
        _handle.append(bq.Moe())
    return bq, _handle[0]


def _cache(bq, st):
    if "cache" not in st:  # a program keeps its cache's description
        st["cache"] = bq.make_kv_cache(st["k_pages"], st["v_pages"], st["table"], st["k_scales"], st["v_scales"])
    return st["cache"]


def _append_own(st):
    bq, moe = _moe()
    cache = _cache(bq, st)
    q, k, v = _split(st)
    moe.kv_append(k, v, st["pos"], cache, seqs=st["seq"], q=q, q_out=st["q_out"], inv_freq=st["freq"])
    if st["bits8"]:
        moe.kv_read(cache, st["pos"], st["k_out"], st["v_out"], seqs=st["seq"])
        return {"q": st["q_out"], "k": st["k_out"], "v": st["v_out"]}
    return {"q": st["q_out"], "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _read_own(st):
    bq, moe = _moe()
    moe.kv_read(_cache(bq, st), st["pos"], st["k_out"], st["v_out"], seqs=st["seq"])
    return {"k": st["k_out"], "v": st["v_out"]}


def _attend_own(st):
    bq, moe = _moe()
    cache = _cache(bq, st)
    if "ws" not in st:
        st["ws"] = torch.empty(moe.kv_attend_workspace_bytes(cache, st["q_heads"]), dtype=torch.uint8, device=_DEV)
    moe.kv_attend(st["q"], st["lengths"], cache, st["out"], st["ws"], scale=st["scale"], softcap=st["softcap"],
                  window=st["window"])
    return {"out": st["out"]}


def _sample_own(st):
    bq, moe = _moe()
    if "rules" not in st:
        st["rules"] = bq.make_sample_rules(st["uniform"], temperature=st["temperature"], top_k=st["top_k"],
                                           top_p=st["top_p"], min_p=st["min_p"])
    moe.sample(st["logits"], st["rows"], st["vocab"], st["rules"], st["tokens"], logprobs=st["logprobs"])
    return {"tokens": st["tokens"], "logprobs": st["logprobs"]}


def run(state):
    op = state["op"]
    if own:
        return {"append": _append_own, "read": _read_own, "attend": _attend_own, "sample": _sample_own}[op](state)
    return {"append": _append_plain, "read": _read_plain, "attend": _attend_plain, "sample": _sample_plain}[op](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "sample":
        T, V = case["rows"], case["vocab"]
        return {"bytes": 4 * T * V + 28 * T, "flops": 8 * T * V}
    Hkv, D = case["kv_heads"], case["dim"]
    row = 2 * Hkv * ((D + 4) if case["bits8"] else 2 * D)  # a position's keys and values in the cache
    if case["op"] == "attend":
        n, L, W = case["seqs"], case["length"], case["window"]
        mean = L if case["even"] or n == 1 else 2.0 * L / 3.0  # (of L sqrt(u), u uniform)
        if W and W < L:
            # E[min(W, L sqrt(u))]: the lengths' density is 2 x / L^2
            mean = W if case["even"] or n == 1 else W - W ** 3 / (3.0 * L * L)
        return {"bytes": int(n * mean * row) + 4 * n * case["q_heads"] * D,
                "flops": int(4 * n * mean * case["q_heads"] * D)}
    T = case["rows"]
    rows16 = 4 * T * Hkv * D  # keys and values in bf16
    if case["op"] == "read":
        return {"bytes": T * row + rows16 + 8 * T, "flops": 2 * T * Hkv * D}
    q = 4 * T * case["q_heads"] * D
    back = T * row + rows16 if case["bits8"] else 0  # read back
    return {"bytes": q + rows16 + T * row + 8 * T + back, "flops": 3 * T * (case["q_heads"] + Hkv) * case["rot"]}


# ------------------------------------------------------------------ the definitions in 64 bits
def _turned(st, x):
    """Complex numbers turn by their angle: exp(i a) (x_j + i x_(j + rot / 2))."""
    x = x.double()
    r = st["rot"]
    if r:
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=_DEV),
                           torch.outer(st["pos"].double(), st["freq"].double()))
        z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * turn.unsqueeze(1)
        x = torch.cat((z.real, z.imag, x[..., r:]), 2)
    return x


def _eighths(x):
    """What 8-bit codes with the row's scale keep of rows x."""
    step = torch.linalg.vector_norm(x, math.inf, dim=-1, keepdim=True) / 127
    return torch.round(x / torch.where(step > 0, step, 1.0)) * step


def _append_exact(st):
    q, k, v = _split(st)
    got = {"q": _turned(st, q)}
    for name, x in (("k", _turned(st, k)), ("v", v.double())):
        if st["bits8"]:
            got[name] = _eighths(x)
        else:
            pages = st[name + "_pages"].double()
            for t, (s, p) in enumerate(zip(st["seq"].tolist(), st["pos"].tolist())):
                pages[int(st["table"][s, p // st["page"]]), :, p % st["page"]] = x[t]
            got[name + "_pages"] = pages
    return got


def _read_exact(st):
    got = {}
    for name in ("k", "v"):
        pages = st[name + "_pages"].movedim(2, 1).flatten(0, 1)  # a row per place
        at = st["table"].long() * st["page"]
        at = at[st["seq"].long()].gather(1, (st["pos"].long() // st["page"])[:, None])[:, 0] + st["pos"] % st["page"]
        got[name] = pages.index_select(0, at).double()
        if st["bits8"]:
            got[name] *= st[name + "_scales"].movedim(2, 1).flatten(0, 1).index_select(0, at).double().unsqueeze(2)
    return got


def _attend_exact(st):
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=_DEV)
    for i, L in enumerate(st["lengths"].tolist()):
        a = max(0, L - st["window"]) if st["window"] else 0
        if L == a:
            continue
        at = torch.arange(a, L, device=_DEV)
        page = st["table"][i].long()[at // st["page"]]
        rows = []
        for name in ("k", "v"):
            x = st[name + "_pages"][page, :, at % st["page"]].double()
            if st["bits8"]:
                x = x * st[name + "_scales"][page, :, at % st["page"]].double().unsqueeze(-1)
            rows.append(x.repeat_interleave(st["q_heads"] // st["kv_heads"], 1))
        s = torch.einsum("hd,lhd->hl", st["q"][i].double(), rows[0]) * st["scale"]
        if st["softcap"]:
            s = torch.tanh(s / st["softcap"]) * st["softcap"]
        out[i] = torch.einsum("hl,lhd->hd", torch.softmax(s, 1), rows[1])
    return {"out": out}


def _sample_exact(st):
    logs = []
    for t in range(st["rows"]):
        l = st["logits"][t].double()
        z = l / st["temperature"][t].double()
        order = torch.argsort(l, descending=True, stable=True)
        prob = torch.softmax(z, 0)[order]
        n = prob.numel()
        if st["min_p"][t] > 0:
            n = int((prob >= st["min_p"][t].double() * prob[0]).sum())
        if st["top_k"][t] > 0:
            n = min(n, int(st["top_k"][t]))
        if st["top_p"][t] < 1:
            share = prob[:n].cumsum(0) / prob[:n].sum()
            n = min(n, int((share < st["top_p"][t].double()).sum()) + 1)
        ids = order[:n].sort().values
        log = torch.log_softmax(z[ids], 0)
        pick = int((log.exp().cumsum(0) <= st["uniform"][t].double()).sum())
        logs.append(log[min(pick, n - 1)])
    return {"tokens": None, "logprobs": torch.stack(logs)}


def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _append_exact, "read": _read_exact, "attend": _attend_exact, "sample": _sample_exact}[case["op"]](st)
