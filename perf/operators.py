"""The measured cases of the operators that follow the short convolutions.

Behind the GDN conv: the gated delta rule as a varlen prefill ("gdn_prefill"),
as an update by one or a few tokens ("gdn_update") and as a speculative update
that keeps one state per draft ("gdn_spec"). Behind the CCA conv: the norms of
queries and keys with the position rotation and the write into the paged cache
("norm_rope"), and the attention of new tokens over that cache ("attn").

`run` computes each in elementary torch operations, or, where `own` is true, by
the library's entry points; `exact` computes it in 64 bits by other means.
"""
import math

import numpy as np
import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
CHUNK = 64          # tokens per step of the plain prefill
NORM_EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    gdn = {"hk": 16, "hv": 32, "dk": 128, "dv": 128}     # 8192 mixed channels
    nr = {"nq": 16, "nkv": 2, "hd": 128, "block": 16}
    at = {"nq": 16, "nkv": 4, "hd": 128, "block": 16}
    return [
        # one short prompt: the serial chain of a few chunks, latency alone
        {"name": "gdn_prefill_1x256", "op": "gdn_prefill", **gdn, "requests": 1, "tokens": 256,
         "even": True, "continued": False, "gates": "bf16"},
        # the mixed prefill batch of the conv benchmark: 8 ragged requests
        {"name": "gdn_prefill_8_ragged", "op": "gdn_prefill", **gdn, "requests": 8,
         "tokens": 8196, "even": False, "continued": True, "gates": "bf16"},
        # one long prompt: few independent chains, each as long as it gets
        {"name": "gdn_prefill_1x32768", "op": "gdn_prefill", **gdn, "requests": 1,
         "tokens": 32768, "even": True, "continued": False, "gates": "f32"},
        # a single user's decode step
        {"name": "gdn_update_1x1", "op": "gdn_update", **gdn, "requests": 1, "q": 1,
         "gates": "bf16"},
        # the decode batch of the conv benchmark
        {"name": "gdn_update_512x1", "op": "gdn_update", **gdn, "requests": 512, "q": 1,
         "gates": "bf16"},
        # the speculative batch of the conv benchmark: 4 drafts for each request
        {"name": "gdn_spec_128x4", "op": "gdn_spec", **gdn, "requests": 128, "q": 4,
         "gates": "bf16"},
        # a decode step's rows, then a batch of prompts with its decodes
        {"name": "norm_rope_17", "op": "norm_rope", **nr, "tokens": 17, "rot": 128,
         "interleaved": False, "k_out": False},
        {"name": "norm_rope_32768", "op": "norm_rope", **nr, "tokens": 32768, "rot": 64,
         "interleaved": False, "k_out": True},
        # one short conversation; a full decode batch; few very long ones; drafts
        {"name": "attn_1x300", "op": "attn", **at, "requests": 1, "q": 1, "longest": 300,
         "even": True},
        {"name": "attn_512_ragged", "op": "attn", **at, "requests": 512, "q": 1,
         "longest": 2048, "even": False},
        {"name": "attn_3x131071", "op": "attn", **at, "requests": 3, "q": 1,
         "longest": 131071, "even": True},
        {"name": "attn_64x4_drafts", "op": "attn", **at, "requests": 64, "q": 4,
         "longest": 8192, "even": False},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gdn_prefill", "gdn_update", "gdn_spec", "norm_rope", "attn"])
    if op.startswith("gdn"):
        hk = rng.choice([1, 2, 4, 8, 16])
        case = {"op": op, "hk": hk, "hv": hk * rng.choice([1, 2]), "dk": rng.choice([64, 128]),
                "dv": rng.choice([64, 128]), "gates": rng.choice(["bf16", "f32"])}
        if op == "gdn_prefill":
            tokens = _log_int(rng, 1, 32768)
            return {**case, "tokens": tokens, "requests": _log_int(rng, 1, min(tokens, 64)),
                    "even": rng.random() < 0.5, "continued": rng.random() < 0.5}
        if op == "gdn_update":
            q = rng.choice([1, 1, 2, 3, 4])
            return {**case, "requests": _log_int(rng, 1, 512 // q), "q": q}
        return {**case, "requests": _log_int(rng, 1, 128), "q": rng.randint(2, 4)}
    hd = rng.choice([64, 128, 256])
    nkv = rng.choice([1, 2, 4, 8])
    if op == "norm_rope":
        nkv = min(nkv, 512 // hd)
        return {"op": op, "nq": nkv * rng.choice([1, 4, 8]), "nkv": nkv, "hd": hd,
                "block": rng.choice([16, 64, 528]), "tokens": _log_int(rng, 1, 16384),
                "rot": rng.choice([hd, hd // 2]), "interleaved": rng.random() < 0.5,
                "k_out": rng.random() < 0.5}
    q = rng.choice([1, 1, 2, 5])
    requests = _log_int(rng, 1, 256)
    most = min(131072, 512 * 1024 * 512 // (requests * nkv * hd))
    return {"op": op, "nq": nkv * rng.choice([1, 4, 7, 16]), "nkv": nkv, "hd": hd,
            "block": rng.choice([16, 64, 528]), "requests": requests, "q": q,
            "longest": _log_int(rng, 8, most), "even": rng.random() < 0.5}


def _lengths(total, n, even, rng):
    """n lengths of at least one token with the given sum."""
    if even or n == 1:
        cuts = np.arange(1, n) * total // n
    else:
        cuts = np.sort(rng.choice(np.arange(1, total), n - 1, replace=False))
    return np.diff(np.concatenate([[0], cuts, [total]])).astype(np.int64)


def _cache_lengths(case, rng):
    """Cached tokens of each request, its q new ones among them."""
    n, top, q = case["requests"], case["longest"], case["q"]
    if case["even"]:
        return np.full(n, top, np.int64)
    return np.maximum(rng.integers(1, top + 1, n), q).astype(np.int64)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _randn(gen, *shape, dtype=BF16, scale=1.0):
    x = torch.empty(shape, dtype=dtype, device="cuda")
    return x.normal_(0.0, scale, generator=gen)


def _ints(values, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(values), device="cuda").to(dtype)


def _prepare_gdn(case, gen, rng):
    hk, hv, dk, dv = (case[n] for n in ("hk", "hv", "dk", "dv"))
    n = case["requests"]
    tokens = case["tokens"] if case["op"] == "gdn_prefill" else n * case["q"]
    # the conv's output rows [q | k | v], after its SiLU
    mixed = _randn(gen, tokens, 2 * hk * dk + hv * dv, dtype=F32)
    mixed = (mixed * torch.sigmoid(mixed)).to(BF16)
    gate = F32 if case["gates"] == "f32" else BF16
    # decay rates 1..16 and time steps 0.001..0.1, as such layers are initialised
    rate = torch.as_tensor(rng.uniform(1, 16, hv), device="cuda").to(F32)
    dt = torch.as_tensor(np.exp(rng.uniform(math.log(1e-3), math.log(0.1), hv)), device="cuda")
    spec = case["op"] == "gdn_spec"
    used = n * case["q"] if spec else n
    slots = rng.permutation(used + used // 4 + 1)[:used]
    s = {"case": case, "query": mixed[:, :hk * dk], "key": mixed[:, hk * dk:2 * hk * dk],
         "value": mixed[:, 2 * hk * dk:],
         "a": _randn(gen, tokens, hv, dtype=gate), "b": _randn(gen, tokens, hv, dtype=gate),
         "A_log": rate.log(), "dt_bias": torch.log(torch.expm1(dt)).to(F32),
         "out": torch.zeros(tokens, hv * dv, dtype=BF16, device="cuda"),
         "pool": _randn(gen, used + used // 4 + 1, hv, dv, dk, dtype=F32, scale=0.1),
         "slots": _ints(slots.reshape(n, -1) if spec else slots)}
    if spec:
        s["accepted"] = _ints(rng.integers(1, case["q"] + 1, n))
    if case["op"] == "gdn_prefill":
        lens = _lengths(tokens, n, case["even"], rng)
        starts = np.concatenate([[0], np.cumsum(lens)])
        has = rng.integers(0, 2, n) if case["continued"] else np.zeros(n, np.int64)
        # the host's plan of chunks: the rows of each (`tokens` = none), and of
        # each step the requests that still have one
        rows, steps = [], []
        for r in range(n):
            for i, t in enumerate(range(int(starts[r]), int(starts[r + 1]), CHUNK)):
                at = np.arange(t, t + CHUNK)
                rows.append(np.where(at < starts[r + 1], at, tokens))
                if i == len(steps):
                    steps.append(([], []))
                steps[i][0].append(r)
                steps[i][1].append(len(rows) - 1)
        s |= {"lens": lens, "qsl": _ints(starts), "has": _ints(has, torch.uint8),
              "rows": _ints(np.stack(rows), torch.int64),
              "steps": [(_ints(r, torch.int64), _ints(c, torch.int64)) for r, c in steps]}
    return s


def _prepare_norm_rope(case, gen, rng):
    nq, nkv, hd, tokens, block = (case[n] for n in ("nq", "nkv", "hd", "tokens", "block"))
    rows = _randn(gen, tokens, (nq + 2 * nkv) * hd)     # a CCA output row [q | k | v]
    blocks = -(-tokens // block) + 2
    slots = rng.permutation(blocks)[:, None] * block + np.arange(block)
    slots = slots.reshape(-1)[:tokens].copy()
    slots[rng.random(tokens) < 0.02] = -1               # rows that pad a captured batch
    top = 8192
    angle = torch.arange(top, dtype=F64, device="cuda")[:, None] * 1e6 ** (
        -torch.arange(0, case["rot"], 2, dtype=F64, device="cuda") / case["rot"])
    cache = lambda: _randn(gen, blocks, block, nkv, hd)
    return {"case": case, "query": rows[:, :nq * hd], "key": rows[:, nq * hd:(nq + nkv) * hd],
            "value": rows[:, (nq + nkv) * hd:],
            "q_weight": 1 + _randn(gen, hd, scale=0.1), "k_weight": 1 + _randn(gen, hd, scale=0.1),
            "table": torch.cat([angle.cos(), angle.sin()], 1).to(F32),
            "positions": _ints(rng.integers(0, top, tokens), torch.int64),
            "slots": _ints(slots, torch.int64), "k_cache": cache(), "v_cache": cache(),
            "q_out": torch.zeros(tokens, nq * hd, dtype=BF16, device="cuda"),
            "k_out": torch.zeros(tokens, nkv * hd, dtype=BF16, device="cuda")
            if case["k_out"] else None}


def _prepare_attn(case, gen, rng):
    nq, nkv, hd, block, q = (case[n] for n in ("nq", "nkv", "hd", "block", "q"))
    lens = _cache_lengths(case, rng)
    pages = -(-lens // block)
    order = rng.permutation(int(pages.sum()) + 3)
    table = np.zeros((len(lens), int(pages.max())), np.int64)
    at = 0
    for r, p in enumerate(pages):
        table[r, :p] = order[at:at + p]
        at += p
    cache = lambda: _randn(gen, len(order), block, nkv, hd)
    rows = len(lens) * q
    return {"case": case, "query": _randn(gen, rows, nq * hd), "k_cache": cache(),
            "v_cache": cache(), "table": _ints(table), "lens": _ints(lens),
            "longest": int(lens.max()),
            "out": torch.zeros(rows, nq * hd, dtype=BF16, device="cuda")}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    op = case["op"]
    return (_prepare_norm_rope if op == "norm_rope" else
            _prepare_attn if op == "attn" else _prepare_gdn)(case, gen, rng)


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _gates(s):
    """(log decay, beta) of each token and head, in 64 bits: a chunk's decays
    are differences of their running sum."""
    x = s["a"].to(F64) + s["dt_bias"].to(F64)
    soft = torch.where(x > 30, x, torch.log1p(torch.exp(torch.clamp(x, max=30))))
    return -torch.exp(s["A_log"].to(F64)) * soft, torch.sigmoid(s["b"].to(F64))


def _heads(x, heads, copies=1):
    """Rows (T, heads * d) as (T, heads * copies, d), each head repeated."""
    x = x.reshape(x.shape[0], heads, -1)
    return x if copies == 1 else x.repeat_interleave(copies, 1)


def _unit(x):
    x = x.to(F32)
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + NORM_EPS)


def _gdn_inputs(s):
    c = s["case"]
    copies = c["hv"] // c["hk"]
    return (_unit(_heads(s["query"], c["hk"], copies)) * c["dk"] ** -0.5,
            _unit(_heads(s["key"], c["hk"], copies)), _heads(s["value"], c["hv"]).to(F32))


def _plain_gdn_update(s):
    """Token by token: S = e^g S + u k^T with u = beta (v - e^g S k), o = S q."""
    c, n, q = s["case"], s["case"]["requests"], s["case"]["q"]
    spec = c["op"] == "gdn_spec"
    qs, ks, vs = (x.reshape(n, q, c["hv"], -1) for x in _gdn_inputs(s))
    g, beta = (x.to(F32).reshape(n, q, c["hv"], 1) for x in _gates(s))
    slots = s["slots"].long()
    first = slots.gather(1, s["accepted"].long()[:, None] - 1)[:, 0] if spec else slots
    S = s["pool"][first]
    outs, kept = [], []
    for t in range(q):
        S = S * torch.exp(g[:, t])[..., None]
        u = beta[:, t] * (vs[:, t] - (S @ ks[:, t, :, :, None])[..., 0])
        S = S + u[..., None] * ks[:, t, :, None]
        outs.append((S @ qs[:, t, :, :, None])[..., 0])
        kept.append(S)
    if spec:
        s["pool"][slots.reshape(-1)] = torch.stack(kept, 1).flatten(0, 1)
    else:
        s["pool"][slots] = S
    s["out"].copy_(torch.stack(outs, 1).reshape(n * q, -1))
    return {"out": s["out"], "state": s["pool"]}


def _plain_gdn_prefill(s):
    """Chunks of 64 tokens: within one, the updates u solve a triangular
    system that does not depend on the state; the state then passes through a
    request's chunks in turn. The forward substitution goes row by row."""
    c, rows = s["case"], s["rows"]
    pad = lambda x: torch.cat([x, x.new_zeros(1, *x.shape[1:])])[rows].transpose(1, 2)
    q, k, v = (pad(x).contiguous() for x in _gdn_inputs(s))          # (chunk, head, 64, d)
    g, beta = (pad(x[..., None])[..., 0] for x in _gates(s))         # (chunk, head, 64)
    G = g.cumsum(-1)
    beta = beta.to(F32)[..., None]
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=rows.device).tril()
    D = torch.where(lower, G[..., :, None] - G[..., None, :], -math.inf).exp().to(F32)
    eG, tail = G.exp().to(F32)[..., None], (G[..., -1:] - G).exp().to(F32)[..., None]
    kt = k.transpose(-1, -2).contiguous()
    A = beta * (D * (k @ kt)).tril(-1)
    P = D * (q @ kt)
    X = torch.cat([beta * v, beta * eG * k], -1)
    for t in range(1, CHUNK):
        X[:, :, t:t + 1] -= A[:, :, t:t + 1, :t] @ X[:, :, :t]
    Xv, Xk = X.split([c["dv"], c["dk"]], -1)
    qe, kd = q * eG, k * tail
    slots = s["slots"].long()
    S = torch.where(s["has"].bool()[:, None, None, None], s["pool"][slots], 0.0)
    O = torch.empty_like(v)
    for r, i in s["steps"]:
        St = S[r].transpose(-1, -2).contiguous()
        U = Xv[i] - Xk[i] @ St
        O[i] = qe[i] @ St + P[i] @ U
        S[r] = eG[i, :, -1:] * S[r] + U.transpose(-1, -2).contiguous() @ kd[i]
    s["pool"][slots] = S
    out = s["out"].new_empty(s["out"].shape[0] + 1, s["out"].shape[1])
    out[rows.reshape(-1)] = O.transpose(1, 2).reshape(rows.numel(), -1).to(BF16)
    s["out"].copy_(out[:-1])
    return {"out": s["out"], "state": s["pool"]}


def _rotate(x, s):
    """x (T, heads, hd) in 32 bits; the first `rot` values of a head turn."""
    c = s["case"]
    half = c["rot"] // 2
    cos, sin = s["table"][s["positions"]][:, None].split(half, -1)
    turn, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    if c["interleaved"]:
        x1, x2 = turn[..., 0::2], turn[..., 1::2]
    else:
        x1, x2 = turn[..., :half], turn[..., half:]
    pair = (x1 * cos - x2 * sin, x2 * cos + x1 * sin)
    turn = torch.stack(pair, -1).flatten(-2) if c["interleaved"] else torch.cat(pair, -1)
    return torch.cat([turn, rest], -1)


def _plain_norm_rope(s):
    c = s["case"]

    def one(x, heads, weight):
        x = _heads(x, heads).to(F32)
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + NORM_EPS) * weight.to(F32)
        return _rotate(x, s).to(BF16)
    q = one(s["query"], c["nq"], s["q_weight"])
    k = one(s["key"], c["nkv"], s["k_weight"])
    s["q_out"].copy_(q.flatten(1))
    if s["k_out"] is not None:
        s["k_out"].copy_(k.flatten(1))
    at = (s["slots"] >= 0).nonzero()[:, 0]
    for cache, rows in ((s["k_cache"], k), (s["v_cache"], _heads(s["value"], c["nkv"]))):
        cache.view(-1, c["nkv"], c["hd"])[s["slots"][at]] = rows[at]
    return {"q": s["q_out"], "k": s["k_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attn(s):
    c, n, q = s["case"], s["case"]["requests"], s["case"]["q"]
    nkv, hd, group = c["nkv"], c["hd"], c["nq"] // c["nkv"]
    k, v = (x[s["table"].long()].flatten(1, 2).transpose(1, 2).to(F32)
            for x in (s["k_cache"], s["v_cache"]))                   # (n, nkv, L, hd)
    Q = s["query"].to(F32).view(n, q, nkv, group, hd).permute(0, 2, 1, 3, 4)
    Q = Q.reshape(n, nkv, q * group, hd)
    score = (Q @ k.transpose(-1, -2).contiguous()) * hd ** -0.5
    last = s["lens"][:, None] - q + torch.arange(q, device=Q.device)  # newest visible position
    seen = torch.arange(k.shape[2], device=Q.device) <= last.repeat_interleave(group, 1)[..., None]
    score = torch.where(seen[:, None], score, -math.inf)
    top = score.max(-1, keepdim=True).values.clamp_min(-3e38)         # a row that sees nothing
    p = torch.exp(score - top)
    o = (p @ v) / p.sum(-1, keepdim=True).clamp_min(1e-30)
    o = o.view(n, nkv, q, group, hd).permute(0, 2, 1, 3, 4)
    s["out"].copy_(o.reshape(n * q, -1))
    return s["out"]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _own(s):
    import stateful_causal_short_amd as scs
    c = s["case"]
    op = c["op"]
    if op == "norm_rope":
        scs.sc_qk_norm_rope(s["query"], s["key"], s["value"], s["q_out"], s["k_out"],
                            s["q_weight"], s["k_weight"], s["table"], s["positions"],
                            s["slots"], s["k_cache"], s["v_cache"], head_dim=c["hd"],
                            eps=NORM_EPS, interleaved=c["interleaved"])
        return {"q": s["q_out"], "k": s["k_out"], "k_cache": s["k_cache"],
                "v_cache": s["v_cache"]}
    if op == "attn":
        scs.sc_paged_attn_decode(s["query"], s["out"], s["k_cache"], s["v_cache"], s["table"],
                                 s["lens"], q=c["q"], max_seq_len=s["longest"])
        return s["out"]
    args = [s[n] for n in ("query", "key", "value", "a", "b", "A_log", "dt_bias", "out", "pool")]
    if op == "gdn_prefill":
        scs.sc_gdn_prefill_varlen(*args, s["qsl"], s["slots"], s["has"])
    elif op == "gdn_update":
        scs.sc_gdn_update(*args, s["slots"], q=c["q"])
    else:
        scs.sc_gdn_update_spec(*args, s["slots"], s["accepted"], q=c["q"])
    return {"out": s["out"], "state": s["pool"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return (_plain_gdn_prefill if op == "gdn_prefill" else _plain_norm_rope
            if op == "norm_rope" else _plain_attn if op == "attn" else _plain_gdn_update)(state)


def work(case):
    op = case["op"]
    if op == "norm_rope":
        width, table = (case["nq"] + 2 * case["nkv"]) * case["hd"], 4 * case["rot"]
        written = width + (case["nkv"] * case["hd"] if case["k_out"] else 0)
        return {"bytes": case["tokens"] * (2 * width + 2 * written + 16)
                + min(case["tokens"], 8192) * table,
                "flops": case["tokens"] * (case["nq"] + case["nkv"]) * (4 * case["hd"] + 3 * case["rot"])}
    if op == "attn":
        rows = case["requests"] * case["q"] * case["nq"] * case["hd"]
        cached = case["requests"] * case["longest"] / (1 if case["even"] else 2)
        return {"bytes": cached * case["nkv"] * case["hd"] * 4 + rows * 4
                + cached / case["block"] * 4,
                "flops": 4 * cached * case["q"] * case["nq"] * case["hd"]}
    n, state = case["requests"], case["hv"] * case["dv"] * case["dk"]
    tokens = case["tokens"] if op == "gdn_prefill" else n * case["q"]
    gate = 4 if case["gates"] == "f32" else 2
    written = n * (case["q"] if op == "gdn_spec" else 1)
    read = 0 if op == "gdn_prefill" and not case["continued"] else n
    return {"bytes": tokens * 2 * (2 * case["hk"] * case["dk"] + 2 * case["hv"] * case["dv"]
                                   + case["hv"] * gate) + (read + written) * state * 4,
            "flops": 7 * tokens * state}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _exact_gdn(s):
    """The recurrence with the state as (DK, DV) and broadcast sums, every
    request a row of one batch that ends when its tokens do."""
    c = s["case"]
    per = c["hv"] // c["hk"]
    spec = c["op"] == "gdn_spec"
    lens = s["lens"] if "lens" in s else np.full(c["requests"], c["q"])
    starts = np.concatenate([[0], np.cumsum(lens)])
    a = s["a"].double() + s["dt_bias"].double()
    decay = torch.exp(-s["A_log"].double().exp() * torch.logaddexp(a, torch.zeros_like(a)))
    beta = 1 / (1 + torch.exp(-s["b"].double()))
    unit = lambda x: x / torch.sqrt(x.square().sum(2, keepdim=True) + NORM_EPS)
    q = unit(s["query"].double().unflatten(1, (c["hk"], c["dk"]))) / math.sqrt(c["dk"])
    k = unit(s["key"].double().unflatten(1, (c["hk"], c["dk"])))
    v = s["value"].double().unflatten(1, (c["hv"], c["dv"]))
    head = torch.arange(c["hv"], device=v.device) // per
    order = np.argsort(-lens, kind="stable")            # the longest first
    slots = s["slots"].long()[torch.as_tensor(order, device=v.device)]
    if spec:
        accepted = s["accepted"].long()[torch.as_tensor(order, device=v.device)]
        S = s["pool"].double()[slots[torch.arange(len(order), device=v.device), accepted - 1]]
    else:
        S = s["pool"].double()[slots]
    if "has" in s:
        S = S * s["has"].double()[torch.as_tensor(order, device=v.device)][:, None, None, None]
    S = S.transpose(2, 3).contiguous()
    out, pool = torch.zeros_like(v), s["pool"].double()
    first = torch.as_tensor(starts[order], device=v.device)
    active = [int((lens > t).sum()) for t in range(int(lens.max()))]
    for t, m in enumerate(active):
        at, A = first[:m] + t, S[:m]
        kt, qt = k[at][:, head], q[at][:, head]
        A.mul_(decay[at][..., None, None])
        miss = v[at] - (kt[:, :, None] @ A)[:, :, 0]
        A.add_(kt[..., None] * (beta[at][..., None] * miss)[:, :, None])
        out[at] = (qt[:, :, None] @ A)[:, :, 0]
        if spec:
            pool[slots[:, t]] = S.transpose(2, 3)
    if not spec:
        pool[slots] = S.transpose(2, 3)
    return {"out": out.flatten(1), "state": pool}


def _exact_norm_rope(s):
    """The rotation as a product of complex numbers."""
    c = s["case"]
    half = c["rot"] // 2
    row = s["table"].double()[s["positions"]]
    phase = torch.complex(row[:, :half], row[:, half:])[:, None]

    def one(x, heads, weight):
        x = x.double().unflatten(1, (heads, c["hd"]))
        x = x / torch.sqrt(x.square().sum(2, keepdim=True) / c["hd"] + NORM_EPS) * weight.double()
        turn = x[..., :c["rot"]]
        turn = turn.unflatten(2, (half, 2)) if c["interleaved"] else \
            turn.unflatten(2, (2, half)).transpose(2, 3)
        z = torch.view_as_real(torch.view_as_complex(turn.contiguous()) * phase)
        x[..., :c["rot"]] = z.flatten(2) if c["interleaved"] else z.transpose(2, 3).flatten(2)
        return x
    q, k = one(s["query"], c["nq"], s["q_weight"]), one(s["key"], c["nkv"], s["k_weight"])
    caches = [s["k_cache"].double(), s["v_cache"].double()]
    keep = s["slots"] >= 0
    block, at = s["slots"][keep] // c["block"], s["slots"][keep] % c["block"]
    caches[0][block, at] = k[keep]
    caches[1][block, at] = s["value"].double().unflatten(1, (c["nkv"], c["hd"]))[keep]
    return {"q": q.flatten(1), "k": None if s["k_out"] is None else k.flatten(1),
            "k_cache": caches[0], "v_cache": caches[1]}


def _exact_attn(s):
    """Request by request over its own tokens, one new token at a time."""
    c, q = s["case"], s["case"]["q"]
    group = c["nq"] // c["nkv"]
    out = torch.zeros(s["out"].shape, dtype=F64, device="cuda").unflatten(1, (c["nkv"], group, c["hd"]))
    query = s["query"].double().unflatten(1, (c["nkv"], group, c["hd"]))
    for r, n in enumerate(s["lens"].tolist()):
        pages = s["table"][r, :-(-n // c["block"])].long()
        k, v = (x[pages].flatten(0, 1)[:n].transpose(0, 1).double() for x in (s["k_cache"], s["v_cache"]))
        for j in range(q):
            m = n - q + 1 + j
            if m > 0:
                w = torch.softmax(query[r * q + j] @ k[:, :m].mT / math.sqrt(c["hd"]), -1)
                out[r * q + j] = w @ v[:, :m]
    return out.flatten(1)


def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_norm_rope if case["op"] == "norm_rope" else
            _exact_attn if case["op"] == "attn" else _exact_gdn)(s)
