"""The batched way from the residual stream to the next token, measured operator by operator.

norm    residual addition, root-mean-square norm and 8-bit rows with a scale each (Moe.norm_quant)
qdense  8-bit rows times an 8-bit matrix, a scale per row and per output channel (Moe.qdense_forward)
logits  repetition, presence and frequency penalties, sparse biases, a grammar mask and the greedy
        token of the result (Moe.logits_process)

`run` computes them with elementary torch operations, or with the library where `own` is true.
"""
import math

import torch

own = False

EPS = 1e-6
_DEV = "cuda"


def listed():
    return [
        # one decode step: the block's output added, the norm before the next projection
        {"name": "norm one row", "op": "norm", "rows": 1, "width": 2816, "add": True, "weight": True, "rows16": False},
        # a whole prompt between two layers
        {"name": "norm prompt", "op": "norm", "rows": 4096, "width": 2816, "add": True, "weight": True, "rows16": False},
        # a ragged batch at another width; no residual to add, the bf16 rows wanted as well
        {"name": "norm ragged", "op": "norm", "rows": 777, "width": 1360, "add": False, "weight": False, "rows16": True},
        # an attention-like projection of one token
        {"name": "qdense one row", "op": "qdense", "rows": 1, "n": 4096, "k": 2816, "softcap": 0.0, "f32": False},
        # the head of one token: the whole vocabulary
        {"name": "qdense head one row", "op": "qdense", "rows": 1, "n": 262144, "k": 2816, "softcap": 30.0, "f32": True},
        # the head of a batch of sequences
        {"name": "qdense head batch", "op": "qdense", "rows": 24, "n": 262144, "k": 2816, "softcap": 30.0, "f32": True},
        # an output projection of a prefill chunk
        {"name": "qdense chunk", "op": "qdense", "rows": 128, "n": 2816, "k": 4096, "softcap": 0.0, "f32": False},
        # a projection of a whole prompt
        {"name": "qdense prompt", "op": "qdense", "rows": 4096, "n": 4096, "k": 2816, "softcap": 0.0, "f32": False},
        # odd numbers of rows and channels
        {"name": "qdense ragged", "op": "qdense", "rows": 333, "n": 1411, "k": 1072, "softcap": 0.0, "f32": True},
        # one sequence with a short history, free text
        {"name": "logits one row", "op": "logits", "rows": 1, "vocab": 262144, "pad": 0, "history": 300, "bias": 0,
         "mask": False},
        # a batch of sequences with everything on
        {"name": "logits batch", "op": "logits", "rows": 64, "vocab": 262144, "pad": 0, "history": 4096, "bias": 300,
         "mask": True},
        # an odd vocabulary in padded rows, long histories, a row whose grammar allows nothing
        {"name": "logits ragged", "op": "logits", "rows": 17, "vocab": 100003, "pad": 13, "history": 20000, "bias": 40,
         "mask": True},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "qdense", "qdense", "logits"])
    if op == "norm":
        while True:
            rows, width = _spread(rng, 1, 4096), 16 * _spread(rng, 4, 512)
            if rows * width <= 4096 * 2816:
                return {"op": op, "rows": rows, "width": width, "add": rng.random() < 0.7, "weight": rng.random() < 0.7,
                        "rows16": rng.random() < 0.5}
    if op == "qdense":
        while True:
            rows, n, k = _spread(rng, 1, 4096), _spread(rng, 17, 262144), 16 * _spread(rng, 4, 256)
            if rows * n * k <= 4096 * 4096 * 2816 and n * k <= 262144 * 2816 and rows * n <= 4096 * 4096:
                return {"op": op, "rows": rows, "n": n, "k": k, "softcap": rng.choice([0.0, 0.0, 30.0]),
                        "f32": rng.random() < 0.5}
    return {"op": op, "rows": _spread(rng, 1, 64), "vocab": _spread(rng, 1000, 262144), "pad": rng.choice([0, 0, 5, 16]),
            "history": _spread(rng, 1, 20000), "bias": rng.choice([0, 1, 40, 300]), "mask": rng.random() < 0.6}


# ------------------------------------------------------------------ inputs
def _codes(g, rows, k):
    """8-bit rows and their scales, of bell-shaped values: the largest of a row has the code 127 or -127."""
    q = torch.empty((rows, k), dtype=torch.int8, device=_DEV)
    s = torch.empty(rows, dtype=torch.float32, device=_DEV)
    step = max(1, (1 << 26) // k)
    for a in range(0, rows, step):
        v = torch.randn((min(step, rows - a), k), generator=g, device=_DEV)
        m = v.abs().amax(1, keepdim=True)
        q[a:a + step] = torch.round(v * (127.0 / m)).to(torch.int8)
        s[a:a + step] = m[:, 0] / 127.0
    return q, s


def prepare(case, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(int(seed))
    st = dict(case)
    if case["op"] == "norm":
        T, H = case["rows"], case["width"]
        # a residual stream: rows of different size, a few channels that stand out
        big = 1.0 + 20.0 * (torch.rand(H, generator=g, device=_DEV) > 0.995)
        size = torch.exp(torch.randn((T, 1), generator=g, device=_DEV))
        st["hidden"] = (torch.randn((T, H), generator=g, device=_DEV) * big * size).to(torch.bfloat16)
        st["y"] = (torch.randn((T, H), generator=g, device=_DEV) * size).to(torch.bfloat16) if case["add"] else None
        st["norm"] = (torch.rand(H, generator=g, device=_DEV) + 0.5).to(torch.bfloat16) if case["weight"] else None
        st["hidden_out"] = torch.empty_like(st["hidden"]) if case["add"] else None
        st["q"] = torch.empty((T, H), dtype=torch.int8, device=_DEV)
        st["scales"] = torch.empty(T, dtype=torch.float32, device=_DEV)
        st["x_out"] = torch.empty_like(st["hidden"]) if case["rows16"] else None
    elif case["op"] == "qdense":
        st["x"], st["x_scales"] = _codes(g, case["rows"], case["k"])
        st["w"], st["w_scales"] = _codes(g, case["n"], case["k"])
        st["w_scales"] *= (10.0 if case["softcap"] else 1.0) / math.sqrt(case["k"])
        st["out"] = torch.empty((case["rows"], case["n"]), dtype=torch.float32 if case["f32"] else torch.bfloat16,
                                device=_DEV)
    else:
        T, V, L = case["rows"], case["vocab"], case["history"]
        st["logits"] = (4.0 * torch.randn((T, V + case["pad"]), generator=g, device=_DEV))[:, :V]
        # text repeats itself: most of a history comes from a few hundred tokens
        few = torch.randint(0, V, (T, min(L, 400)), generator=g, device=_DEV)
        pick = torch.randint(0, few.shape[1], (T, L), generator=g, device=_DEV)
        rare = torch.randint(0, V, (T, L), generator=g, device=_DEV)
        st["history"] = torch.where(torch.rand((T, L), generator=g, device=_DEV) < 0.7, few.gather(1, pick),
                                    rare).to(torch.int32)
        share = torch.rand((2, T), generator=g, device=_DEV)
        st["history_len"] = (L * (1.0 - 0.5 * share[0])).ceil().to(torch.int32)
        st["prompt_len"] = (st["history_len"] * share[1]).to(torch.int32)
        st["repetition"] = 1.0 + 0.3 * torch.rand(T, generator=g, device=_DEV)
        st["presence"] = torch.rand(T, generator=g, device=_DEV)
        st["frequency"] = 0.5 * torch.rand(T, generator=g, device=_DEV)
        st["bias_ids"] = st["bias_values"] = st["bias_len"] = st["mask"] = None
        if case["bias"]:
            B = case["bias"]
            st["bias_ids"] = torch.randint(0, V, (T, B), generator=g, device=_DEV).to(torch.int32)
            st["bias_values"] = 5.0 * torch.randn((T, B), generator=g, device=_DEV)
            st["bias_len"] = torch.randint(0, B + 1, (T,), generator=g, device=_DEV).to(torch.int32)
        if case["mask"]:
            words = torch.randint(-(1 << 31), 1 << 31, (2, T, (V + 31) // 32), generator=g, device=_DEV)
            st["mask"] = (words[0] & words[1]).to(torch.int32)  # a quarter of the tokens allowed
            st["mask"][T // 2] = 0 if T > 1 else -1  # one sequence of a batch is at a dead end
        st["out"] = torch.empty((T, V), dtype=torch.float32, device=_DEV)
        st["tokens"] = torch.empty(T, dtype=torch.int32, device=_DEV)
    return st


# ------------------------------------------------------------------ the plain forms
def _norm_plain(st):
    h = st["hidden"]
    if st["y"] is not None:
        h = (h.float() + st["y"].float()).to(torch.bfloat16)
    f = h.float()
    u = f if st["norm"] is None else f * st["norm"].float()
    m = u.abs().amax(1, keepdim=True)
    r = 1.0 / torch.sqrt((f * f).mean(1, keepdim=True) + EPS)
    got = {"q": torch.where(m > 0, torch.round(u * 127.0 / m), 0.0).to(torch.int8), "scales": (m * r / 127.0)[:, 0]}
    if st["y"] is not None:
        got["hidden"] = h
    if st["rows16"]:
        got["x"] = (u * r).to(torch.bfloat16)
    return got


def _qdense_plain(st):
    v = (st["x"].float() @ st["w"].float().t()) * st["x_scales"][:, None] * st["w_scales"]
    if st["softcap"] > 0:
        v = st["softcap"] * torch.tanh(v / st["softcap"])
    return {"y": v if st["f32"] else v.to(torch.bfloat16)}


def _logits_plain(st):
    v = st["logits"]
    T, V = v.shape
    at = torch.arange(st["history"].shape[1], device=_DEV)
    ids = torch.where(at < st["history_len"][:, None], st["history"], V).long()  # V: a column that is dropped
    ones = torch.ones((), device=_DEV).expand(ids.shape)
    seen = torch.zeros((T, V + 1), device=_DEV).scatter_add_(1, ids, ones)[:, :V]
    made = torch.where(at >= st["prompt_len"][:, None], ids, V)
    count = torch.zeros((T, V + 1), device=_DEV).scatter_add_(1, made, ones)[:, :V]
    rep = st["repetition"][:, None]
    v = torch.where(seen > 0, torch.where(v > 0, v / rep, v * rep), v)
    v = v - st["frequency"][:, None] * count
    v = torch.where(count > 0, v - st["presence"][:, None], v)
    if st["bias_ids"] is not None:  # the last entry of a token counts
        B = st["bias_ids"].shape[1]
        j = torch.arange(B, device=_DEV)
        b = torch.where(j < st["bias_len"][:, None], st["bias_ids"], V).long()
        last = torch.full((T, V + 1), -1, device=_DEV).scatter_reduce_(1, b, j.expand(T, B), "amax")[:, :V]
        v = torch.where(last >= 0, v + st["bias_values"].gather(1, last.clamp(min=0)), v)
    if st["mask"] is not None:
        bits = (st["mask"][:, :, None] >> torch.arange(32, device=_DEV)) & 1
        v = torch.where(bits.reshape(T, -1)[:, :V] > 0, v, -math.inf)
    best = v.amax(1, keepdim=True)
    first = torch.where(v == best, torch.arange(V, device=_DEV), V).amin(1)
    return {"logits": v, "tokens": torch.where(best[:, 0] > -math.inf, first, -1).to(torch.int32)}


# ------------------------------------------------------------------ the framework's operators
_handle = []


def _moe():
    import bit_affine_quantized_gb300 as bq
    if not _handle:
        _handle.append(bq.Moe())
    return bq, _handle[0]


def _norm_own(st):
    _, moe = _moe()
    moe.norm_quant(st["hidden"], st["rows"], st["q"], st["scales"], y=st["y"], norm=st["norm"], eps=EPS,
                   hidden_out=st["hidden_out"], x_out=st["x_out"])
    got = {"q": st["q"], "scales": st["scales"]}
    if st["y"] is not None:
        got["hidden"] = st["hidden_out"]
    if st["rows16"]:
        got["x"] = st["x_out"]
    return got


def _qdense_own(st):
    bq, moe = _moe()
    if "weights" not in st:  # a program keeps its weights' description and the workspace
        st["weights"] = bq.make_qdense_weights(st["n"], st["k"], st["w"], st["w_scales"])
        st["ws"] = torch.empty(moe.qdense_workspace_bytes(st["weights"], st["rows"]), dtype=torch.uint8, device=_DEV)
    moe.qdense_forward(st["x"], st["x_scales"], st["rows"], st["weights"], st["ws"], softcap=st["softcap"],
                       **{"y32" if st["f32"] else "y": st["out"]})
    return {"y": st["out"]}


def _logits_own(st):
    bq, moe = _moe()
    if "rules" not in st:
        st["rules"] = bq.make_logit_rules(
            history=st["history"], history_len=st["history_len"], prompt_len=st["prompt_len"],
            repetition=st["repetition"], presence=st["presence"], frequency=st["frequency"], bias_ids=st["bias_ids"],
            bias_values=st["bias_values"], bias_len=st["bias_len"], mask=st["mask"])
    moe.logits_process(st["logits"], st["rows"], st["vocab"], st["rules"], out=st["out"], tokens=st["tokens"])
    return {"logits": st["out"], "tokens": st["tokens"]}


def run(state):
    op = state["op"]
    if own:
        return _norm_own(state) if op == "norm" else _qdense_own(state) if op == "qdense" else _logits_own(state)
    return _norm_plain(state) if op == "norm" else _qdense_plain(state) if op == "qdense" else _logits_plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    T = case["rows"]
    if case["op"] == "norm":
        H = case["width"]
        per = 2 + 1 + (4 if case["add"] else 0) + (2 if case["rows16"] else 0)
        return {"bytes": T * H * per + 4 * T + (2 * H if case["weight"] else 0), "flops": 6 * T * H}
    if case["op"] == "qdense":
        n, k = case["n"], case["k"]
        return {"bytes": n * k + T * k + 4 * (n + T) + T * n * (4 if case["f32"] else 2), "flops": 2 * T * n * k}
    V = case["vocab"]
    return {"bytes": T * V * 8 + 4 * T * case["history"] + 8 * T * case["bias"] + (T * V // 8 if case["mask"] else 0),
            "flops": 2 * T * V}


# ------------------------------------------------------------------ the definitions in 64 bits
def _norm_exact(st):
    h = st["hidden"].double()
    if st["y"] is not None:
        h = (h + st["y"].double()).to(torch.bfloat16).double()  # the stored residual stream is what is normed
    x = h / torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / h.shape[1] + EPS)
    if st["norm"] is not None:
        x = x * st["norm"].double()
    s = torch.linalg.vector_norm(x, math.inf, dim=1) / 127
    got = {"q": None, "scales": s}
    if st["y"] is not None:
        got["hidden"] = h
    if st["rows16"]:
        got["x"] = x
    return got


def _qdense_exact(st):
    x = st["x"].double() * st["x_scales"].double()[:, None]
    out = torch.empty((st["rows"], st["n"]), dtype=torch.float64, device=_DEV)
    for a in range(0, st["n"], 16384):
        b = slice(a, a + 16384)
        z = torch.einsum("tk,nk->tn", x, st["w"][b].double() * st["w_scales"][b].double()[:, None])
        out[:, b] = torch.tanh(z / st["softcap"]) * st["softcap"] if st["softcap"] > 0 else z
    return {"y": out}


def _logits_exact(st):
    rows = []
    for t in range(st["rows"]):
        v = st["logits"][t].double()
        V, n, p = v.numel(), int(st["history_len"][t]), int(st["prompt_len"][t])
        every = torch.bincount(st["history"][t, :n].long(), minlength=V)
        made = torch.bincount(st["history"][t, p:n].long(), minlength=V)
        r = st["repetition"][t].double()
        factor = torch.where(v > 0, 1 / r, r)
        v = v * torch.where(every > 0, factor, 1.0) - st["frequency"][t].double() * made
        v = v - st["presence"][t].double() * (made > 0)
        if st["bias_ids"] is not None:
            k = int(st["bias_len"][t])
            b = dict(zip(st["bias_ids"][t, :k].tolist(), st["bias_values"][t, :k].tolist()))
            if b:
                v[torch.tensor(list(b), device=_DEV)] += torch.tensor(list(b.values()), dtype=torch.float64, device=_DEV)
        if st["mask"] is not None:
            i = torch.arange(V, device=_DEV)
            v = v.masked_fill((st["mask"][t].long()[i // 32] >> (i % 32)) % 2 == 0, -math.inf)
        rows.append(v)
    return {"logits": torch.stack(rows), "tokens": None}


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _norm_exact, "qdense": _qdense_exact, "logits": _logits_exact}[case["op"]](st)
