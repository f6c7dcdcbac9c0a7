"""The measured cases of the quantised paged cache and of attention over shared prefixes.

The cache holds a head of a token as 8-bit floats (e4m3) with one power of two as
its scale. "store": the norms, rotation and quantising write of a prompt's rows, and
the requests' context read back as bf16 rows, as a step that continues prompts does;
"read": such a read alone; "attn_fp8": attention of new tokens over that cache;
"prefix": attention of requests that share the first pages of their caches, in
groups, over bf16 or quantised caches.

`run` computes each in elementary torch operations, or, where `own` is true, by
the library's entry points; `exact` computes it in 64 bits by other means.
"""
import math

import numpy as np
import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U8, E4M3 = torch.uint8, torch.float8_e4m3fn
NORM_EPS = 1e-6
POSITIONS = 65536


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    st = {"nq": 16, "nkv": 2, "hd": 128, "block": 16, "interleaved": False}
    at = {"nq": 16, "nkv": 4, "hd": 128, "block": 16}
    return [
        # the last tokens of one short prompt, behind what is cached of it
        {"name": "store_17_after_47", "op": "store", **st, "requests": 1, "tokens": 17,
         "before": 47, "even": True, "rot": 128},
        # a batch of whole prompts: the CCA benchmark's tokens
        {"name": "store_32768", "op": "store", **st, "requests": 64, "tokens": 32768,
         "before": 0, "even": False, "rot": 64},
        # the context of one short conversation, and of a few long ones, for their next chunk
        {"name": "read_1x300", "op": "read", **at, "requests": 1, "tokens": 300, "even": True},
        {"name": "read_8_ragged", "op": "read", **at, "requests": 8, "tokens": 262143,
         "even": False},
        # one short conversation; a full decode batch; few very long ones; drafts
        {"name": "attn_fp8_1x300", "op": "attn_fp8", **at, "requests": 1, "q": 1,
         "longest": 300, "even": True},
        {"name": "attn_fp8_512_ragged", "op": "attn_fp8", **at, "requests": 512, "q": 1,
         "longest": 2048, "even": False},
        {"name": "attn_fp8_3x131071", "op": "attn_fp8", **at, "requests": 3, "q": 1,
         "longest": 131071, "even": True},
        {"name": "attn_fp8_64x4_drafts", "op": "attn_fp8", **at, "requests": 64, "q": 4,
         "longest": 8192, "even": False},
        # a few users of one assistant, just begun: its instructions and short turns
        {"name": "prefix_8_on_1024", "op": "prefix", **at, "requests": 8, "q": 1, "groups": 1,
         "prefix": 1024, "own_len": 64, "fp8": False},
        # a full decode batch of questions on one long document
        {"name": "prefix_512_on_32768", "op": "prefix", **at, "requests": 512, "q": 1,
         "groups": 1, "prefix": 32768, "own_len": 500, "fp8": False},
        # drafts, over a quantised cache
        {"name": "prefix_64x4_on_16384_fp8", "op": "prefix", **at, "requests": 64, "q": 4,
         "groups": 1, "prefix": 16384, "own_len": 1000, "fp8": True},
        # several assistants' batches in one: uneven groups, prefixes of several lengths
        {"name": "prefix_10_groups", "op": "prefix", "nq": 32, "nkv": 4, "hd": 64, "block": 64,
         "requests": 201, "q": 1, "groups": 10, "prefix": 8192, "own_len": 333, "fp8": False},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "read", "attn_fp8", "prefix", "prefix"])
    hd = rng.choice([64, 128, 256])
    nkv = rng.choice([1, 2, 4, 8])
    case = {"op": op, "nq": nkv * rng.choice([1, 4, 7, 16]), "nkv": nkv, "hd": hd,
            "block": rng.choice([16, 64, 528])}
    if op == "store":
        nkv = min(nkv, 512 // hd)
        tokens = _log_int(rng, 1, 16384)
        return {**case, "nq": nkv * rng.choice([1, 4, 8]), "nkv": nkv, "tokens": tokens,
                "requests": _log_int(rng, 1, min(tokens, 64)), "before": rng.choice([0, 0, 100, 1000]),
                "even": rng.random() < 0.5, "rot": rng.choice([hd, hd // 2]),
                "interleaved": rng.random() < 0.5}
    if op == "read":
        tokens = _log_int(rng, 1, 262143 * 512 // (nkv * hd) if nkv * hd > 512 else 262143)
        return {**case, "tokens": tokens, "requests": _log_int(rng, 1, min(tokens, 64)),
                "even": rng.random() < 0.5}
    q = rng.choice([1, 1, 2, 5])
    if op == "attn_fp8":
        requests = _log_int(rng, 1, 256)
        most = min(131072, 512 * 1024 * 512 // (requests * nkv * hd))
        return {**case, "requests": requests, "q": q, "longest": _log_int(rng, 8, most),
                "even": rng.random() < 0.5}
    requests = _log_int(rng, 2, 512)
    groups = rng.choice([1, 1, 2, _log_int(rng, 1, min(requests, 40))])
    rows = groups * -(-requests // groups) * q * case["nq"]
    most = min(65536, 512 * 16 * 32768 * 128 // (rows * max(hd, 128) * 2),
               65536 * 4096 // (groups * nkv * hd))
    return {**case, "requests": requests, "q": q, "groups": groups,
            "prefix": case["block"] * max(1, _log_int(rng, 16, max(most, 16)) // case["block"]),
            "own_len": _log_int(rng, q, max(q, min(1000, 512 * 1024 * 512 // (requests * nkv * hd)))),
            "fp8": rng.random() < 0.5}


def _lengths(total, n, even, rng):
    """n lengths of at least one token with the given sum."""
    if even or n == 1:
        cuts = np.arange(1, n) * total // n
    else:
        cuts = np.sort(rng.choice(np.arange(1, total), n - 1, replace=False))
    return np.diff(np.concatenate([[0], cuts, [total]])).astype(np.int64)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _randn(gen, *shape, dtype=BF16, scale=1.0):
    x = torch.empty(shape, dtype=dtype, device="cuda")
    return x.normal_(0.0, scale, generator=gen)


def _ints(values, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(values), device="cuda").to(dtype)


def _starts(lens):
    return np.concatenate([[0], np.cumsum(lens)])


def _power(e):
    """2^e in 32 bits, from its bits (-126 <= e <= 127)."""
    return (e.to(torch.int32) + 127 << 23).view(F32)


def _quantise(x):
    """Heads (..., hd) as 8-bit codes and the bytes of their scales: the smallest
    power of two 2^(byte - 127) that brings the largest value to 448 or less."""
    x = x.to(F32)
    top = x.abs().amax(-1).view(torch.int32)         # 448 = 1.75 2^8: compare the mantissa
    byte = ((top + 0x1FFFFF >> 23) - 8).clamp(1, 254)
    return (x * _power(127 - byte)[..., None]).to(E4M3), byte.to(U8)


def _cache(gen, blocks, block, nkv, hd, fp8, spread=True):
    """A cache of `blocks` pages: bf16, or (codes, scales (blocks, nkv, block)).
    Tokens differ in size, as keys and values of a model do."""
    x = _randn(gen, blocks, block, nkv, hd)
    if spread:
        x *= torch.exp2(_randn(gen, blocks, block, nkv, 1))
    if not fp8:
        return x, None
    codes, scale = _quantise(x)
    return codes, scale.transpose(1, 2).contiguous().view(torch.float8_e8m0fnu)


def _pages(rng, lens, block, spare=3):
    """Block table rows for requests of these lengths, pages in random order."""
    need = -(-np.maximum(lens, 1) // block)
    order = rng.permutation(int(need.sum()) + spare)
    table = np.zeros((len(lens), int(need.max())), np.int64)
    at = 0
    for r, p in enumerate(need):
        table[r, :p] = order[at:at + p]
        at += p
    return table, len(order)


def _prepare_store(case, gen, rng):
    nq, nkv, hd, block, tokens = (case[n] for n in ("nq", "nkv", "hd", "block", "tokens"))
    new = _lengths(tokens, case["requests"], case["even"], rng)
    lens = new + case["before"]
    table, blocks = _pages(rng, lens, block)
    pos = np.concatenate([np.arange(n) + case["before"] for n in new])
    request = np.repeat(np.arange(len(new)), new)
    slots = table[request, pos // block] * block + pos % block
    rows = _randn(gen, tokens, (nq + 2 * nkv) * hd)     # CCA output rows [q | k | v]
    angle = torch.arange(POSITIONS, dtype=F64, device="cuda")[:, None] * 1e6 ** (
        -torch.arange(0, case["rot"], 2, dtype=F64, device="cuda") / case["rot"])
    (kc, ks), (vc, vs) = (_cache(gen, blocks, block, nkv, hd, True) for _ in range(2))
    total = int(lens.sum())
    return {"case": case, "query": rows[:, :nq * hd], "key": rows[:, nq * hd:(nq + nkv) * hd],
            "value": rows[:, (nq + nkv) * hd:],
            "q_weight": 1 + _randn(gen, hd, scale=0.1), "k_weight": 1 + _randn(gen, hd, scale=0.1),
            "turns": torch.cat([angle.cos(), angle.sin()], 1).to(F32),
            "positions": _ints(pos, torch.int64), "slots": _ints(slots, torch.int64),
            "k_cache": kc, "k_scale": ks, "v_cache": vc, "v_scale": vs, "table": _ints(table),
            "starts": _ints(_starts(lens)),
            "q_out": torch.zeros(tokens, nq * hd, dtype=BF16, device="cuda"),
            "k_rows": torch.zeros(total, nkv * hd, dtype=BF16, device="cuda"),
            "v_rows": torch.zeros(total, nkv * hd, dtype=BF16, device="cuda")}


def _prepare_read(case, gen, rng):
    nkv, hd, block = (case[n] for n in ("nkv", "hd", "block"))
    lens = _lengths(case["tokens"], case["requests"], case["even"], rng)
    table, blocks = _pages(rng, lens, block)
    (kc, ks), (vc, vs) = (_cache(gen, blocks, block, nkv, hd, True) for _ in range(2))
    return {"case": case, "k_cache": kc, "k_scale": ks, "v_cache": vc, "v_scale": vs,
            "table": _ints(table), "starts": _ints(_starts(lens)),
            "k_rows": torch.zeros(case["tokens"], nkv * hd, dtype=BF16, device="cuda"),
            "v_rows": torch.zeros(case["tokens"], nkv * hd, dtype=BF16, device="cuda")}


def _attn_state(case, gen, table, blocks, lens, fp8):
    nq, nkv, hd, block, q = (case[n] for n in ("nq", "nkv", "hd", "block", "q"))
    kc, ks = _cache(gen, blocks, block, nkv, hd, fp8, spread=False)
    vc, vs = _cache(gen, blocks, block, nkv, hd, fp8)
    rows = len(lens) * q
    return {"case": case, "query": _randn(gen, rows, nq * hd), "k_cache": kc, "k_scale": ks,
            "v_cache": vc, "v_scale": vs, "table": _ints(table), "lens": _ints(lens),
            "longest": int(lens.max()),
            "out": torch.zeros(rows, nq * hd, dtype=BF16, device="cuda")}


def _prepare_attn(case, gen, rng):
    n, top, q = case["requests"], case["longest"], case["q"]
    lens = np.full(n, top, np.int64) if case["even"] else \
        np.maximum(rng.integers(1, top + 1, n), q).astype(np.int64)
    table, blocks = _pages(rng, lens, case["block"])
    return _attn_state(case, gen, table, blocks, lens, True)


def _prepare_prefix(case, gen, rng):
    """Request r of group g has the group's pages first, then its own."""
    n, groups, block, q = (case[n] for n in ("requests", "groups", "block", "q"))
    top = case["prefix"] // block                    # pages of the longest prefix
    shared = np.maximum(1, top * rng.integers(1, 5, groups) // 4)
    shared[0] = top
    sizes = _lengths(n, groups, groups == 1, rng)
    mine = rng.integers(q, case["own_len"] + 1, n)
    pages, extra = -(-mine // block), -(-case["own_len"] // block)
    order = rng.permutation(int(shared.sum() + pages.sum()) + 3)
    table = np.zeros((n, top + extra), np.int64)
    group, at = np.repeat(np.arange(groups), sizes), int(shared.sum())
    first = _starts(shared)
    for r in range(n):
        s = shared[group[r]]
        table[r, :s] = order[first[group[r]]:first[group[r]] + s]
        table[r, s:s + pages[r]] = order[at:at + pages[r]]
        at += pages[r]
    s = _attn_state(case, gen, table, len(order), shared[group] * block + mine, case["fp8"])
    starts = _starts(sizes)
    # the host's plan: the requests of each group, padded (n: none), and each one's place in it
    member = np.minimum(starts[:-1, None] + np.arange(sizes.max()), n)
    member[member >= starts[1:, None]] = n
    return s | {"group_starts": _ints(starts), "prefix_lens": _ints(shared * block),
                "longest_prefix": case["prefix"] // block * block,
                "member": _ints(member, torch.int64), "group": _ints(group, torch.int64),
                "place": _ints(np.arange(n) - starts[group], torch.int64)}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    op = case["op"]
    return (_prepare_store if op == "store" else _prepare_read if op == "read" else
            _prepare_attn if op == "attn_fp8" else _prepare_prefix)(case, gen, rng)


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _values(s, name, pages):
    """Pages (...) of a cache in 32 bits, (..., block, nkv, hd)."""
    cache, scale = s[name + "_cache"], s[name + "_scale"]
    if scale is None:
        return cache[pages].to(F32)
    codes = cache.view(U8)[pages].view(E4M3).to(F32)
    power = _power(scale.view(U8)[pages].to(torch.int32) - 127)
    return codes * power.transpose(-1, -2)[..., None]


def _rotate(x, s):
    """x (T, heads, hd) in 32 bits; the first `rot` values of a head turn."""
    c = s["case"]
    half = c["rot"] // 2
    cos, sin = s["turns"][s["positions"]][:, None].split(half, -1)
    turn, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    if c["interleaved"]:
        x1, x2 = turn[..., 0::2], turn[..., 1::2]
    else:
        x1, x2 = turn[..., :half], turn[..., half:]
    pair = (x1 * cos - x2 * sin, x2 * cos + x1 * sin)
    turn = torch.stack(pair, -1).flatten(-2) if c["interleaved"] else torch.cat(pair, -1)
    return torch.cat([turn, rest], -1)


def _plain_read(s):
    """Row starts[r] + t is token t of request r."""
    c = s["case"]
    starts = s["starts"].long()
    row = torch.arange(s["k_rows"].shape[0], device=starts.device)
    r = torch.searchsorted(starts, row, right=True) - 1
    t = row - starts[r]
    page, at = s["table"].long()[r, t // c["block"]], t % c["block"]
    for name in ("k", "v"):
        codes = s[name + "_cache"].view(U8)[page, at].view(E4M3).to(F32)
        power = _power(s[name + "_scale"].view(U8)[page, :, at].to(torch.int32) - 127)
        s[name + "_rows"].copy_((codes * power[..., None]).flatten(1))
    return {"k": s["k_rows"], "v": s["v_rows"]}


def _plain_store(s):
    c = s["case"]

    def one(x, heads, weight):
        x = x.reshape(x.shape[0], heads, -1).to(F32)
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + NORM_EPS) * weight.to(F32)
        return _rotate(x, s)
    s["q_out"].copy_(one(s["query"], c["nq"], s["q_weight"]).flatten(1))
    page, at = s["slots"] // c["block"], s["slots"] % c["block"]
    rows = {"k": one(s["key"], c["nkv"], s["k_weight"]),
            "v": s["value"].reshape(c["tokens"], c["nkv"], -1)}
    for name, x in rows.items():
        codes, scale = _quantise(x)
        s[name + "_cache"].view(U8)[page, at] = codes.view(U8)
        s[name + "_scale"].view(U8)[page, :, at] = scale
    return {"q": s["q_out"], **_plain_read(s)}


def _rows(s):
    """Queries (n, nkv, q * group, hd) in 32 bits: the rows of a key/value head."""
    c = s["case"]
    x = s["query"].to(F32).view(-1, c["q"], c["nkv"], c["nq"] // c["nkv"], c["hd"])
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _part(Q, k, v, seen, scale):
    """(max, sum, weighted values) of rows Q (n, nkv, rows, hd) over tokens k, v
    (n, L, nkv, hd), those of which each row sees given as (n, rows or 1, L)."""
    k, v = (x.transpose(1, 2).contiguous() for x in (k, v))
    score = (Q @ k.transpose(-1, -2).contiguous()) * scale
    score = torch.where(seen[:, None], score, -math.inf)
    top = score.max(-1, keepdim=True).values.clamp_min(-3e38)
    p = torch.exp(score - top)
    return top, p.sum(-1, keepdim=True), p @ v


def _finish(s, o):
    c = s["case"]
    o = o.view(-1, c["nkv"], c["q"], c["nq"] // c["nkv"], c["hd"]).permute(0, 2, 1, 3, 4)
    s["out"].copy_(o.reshape(s["out"].shape))
    return s["out"]


def _limits(s):
    """The newest position that each row of a request sees, (n, q * group)."""
    c = s["case"]
    last = s["lens"][:, None] - c["q"] + torch.arange(c["q"], device=s["lens"].device)
    return last.repeat_interleave(c["nq"] // c["nkv"], 1)


def _plain_attn(s):
    k, v = (_values(s, name, s["table"].long()).flatten(1, 2) for name in ("k", "v"))
    seen = torch.arange(k.shape[1], device=k.device) <= _limits(s)[..., None]
    top, total, o = _part(_rows(s), k, v, seen, s["case"]["hd"] ** -0.5)
    return _finish(s, o / total.clamp_min(1e-30))


def _plain_prefix(s):
    """The rows of a group against its prefix, in one product; each request's
    against its own tokens; the two joined by their maxima."""
    c, table, scale = s["case"], s["table"].long(), s["case"]["hd"] ** -0.5
    Q, dev, block = _rows(s), s["table"].device, c["block"]
    shared = s["prefix_lens"].long()
    # (groups, nkv, members * rows, hd)
    Qg = torch.cat([Q, Q.new_zeros(1, *Q.shape[1:])])[s["member"]]
    Qg = Qg.transpose(1, 2).flatten(2, 3).contiguous()
    pages = table[s["group_starts"][:-1].long(), :s["longest_prefix"] // block]
    k, v = (_values(s, name, pages).flatten(1, 2) for name in ("k", "v"))
    seen = torch.arange(k.shape[1], device=dev) < shared[:, None, None]
    # each group's rows back to their requests
    m1, l1, o1 = (x.unflatten(2, (-1, Q.shape[2])).transpose(1, 2)[s["group"], s["place"]]
                  for x in _part(Qg, k, v, seen, scale))
    skip = shared[s["group"]]
    width = -(-c["own_len"] // block)
    pages = table.gather(1, (skip // block)[:, None] + torch.arange(width, device=dev))
    k, v = (_values(s, name, pages).flatten(1, 2) for name in ("k", "v"))
    seen = skip[:, None, None] + torch.arange(k.shape[1], device=dev) <= _limits(s)[..., None]
    m2, l2, o2 = _part(Q, k, v, seen, scale)
    m = torch.maximum(m1, m2)
    f1, f2 = torch.exp(m1 - m), torch.exp(m2 - m)
    return _finish(s, (o1 * f1 + o2 * f2) / (l1 * f1 + l2 * f2).clamp_min(1e-30))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _own(s):
    import stateful_causal_short_amd as scs
    c = s["case"]
    op = c["op"]
    if op in ("store", "read"):
        cache = [s[n] for n in ("k_cache", "k_scale", "v_cache", "v_scale")]
        if op == "store":
            scs.sc_qk_norm_rope_fp8(s["query"], s["key"], s["value"], s["q_out"], None,
                                    s["q_weight"], s["k_weight"], s["turns"], s["positions"],
                                    s["slots"], *cache, head_dim=c["hd"], eps=NORM_EPS,
                                    interleaved=c["interleaved"])
        scs.sc_paged_cache_read_fp8(*cache, s["k_rows"], s["v_rows"], s["table"], s["starts"])
        got = {"k": s["k_rows"], "v": s["v_rows"]}
        return got if op == "read" else {"q": s["q_out"], **got}
    if op == "attn_fp8":
        scs.sc_paged_attn_decode_fp8(s["query"], s["out"], s["k_cache"], s["k_scale"],
                                     s["v_cache"], s["v_scale"], s["table"], s["lens"],
                                     q=c["q"], max_seq_len=s["longest"])
        return s["out"]
    sizes = {"q": c["q"], "max_seq_len": s["longest"], "max_prefix_len": s["longest_prefix"]}
    where = s["table"], s["lens"], s["group_starts"], s["prefix_lens"]
    if c["fp8"]:
        scs.sc_paged_attn_prefix_fp8(s["query"], s["out"], s["k_cache"], s["k_scale"],
                                     s["v_cache"], s["v_scale"], *where, **sizes)
    else:
        scs.sc_paged_attn_prefix(s["query"], s["out"], s["k_cache"], s["v_cache"], *where, **sizes)
    return s["out"]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return (_plain_store if op == "store" else _plain_read if op == "read" else
            _plain_attn if op == "attn_fp8" else _plain_prefix)(state)


def work(case):
    op, nkv, hd = case["op"], case["nkv"], case["hd"]
    if op in ("store", "read"):
        back = case["tokens"] + (case["before"] * case["requests"] if op == "store" else 0)
        # read back: codes, scales and pages in, bf16 out
        got = {"bytes": 2 * back * nkv * (3 * hd + 1) + 4 * back / case["block"], "flops": 2 * back * nkv * hd}
        if op == "store":
            heads = case["nq"] + nkv
            got["bytes"] += case["tokens"] * (2 * (heads + nkv) * hd + 2 * case["nq"] * hd
                                              + 2 * nkv * (hd + 1) + 16 + 4 * case["rot"])
            got["flops"] += case["tokens"] * (heads * (4 * hd + 3 * case["rot"]) + 4 * nkv * hd)
        return got
    rows = case["requests"] * case["q"] * case["nq"] * hd
    token = nkv * (2 * (hd + 1) if op == "attn_fp8" or case["fp8"] else 4 * hd)
    if op == "attn_fp8":
        cached = case["requests"] * case["longest"] / (1 if case["even"] else 2)
        return {"bytes": cached * token + rows * 4 + cached / case["block"] * 4,
                "flops": 4 * cached * case["q"] * case["nq"] * hd}
    # a group's prefix is the longest for the first, 5/8 of it for the others on average
    mean = (1 + 5 / 8 * (case["groups"] - 1)) / case["groups"] * case["prefix"]
    mine = case["requests"] * case["own_len"] / 2
    tokens = case["groups"] * mean + mine
    return {"bytes": tokens * token + rows * 4 + tokens / case["block"] * 4,
            "flops": 4 * case["q"] * case["nq"] * hd * (case["requests"] * mean + mine)}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _two_to(e):
    """2^e in 64 bits."""
    return (e.to(torch.int64) + 1023 << 52).view(F64)


def _whole(s, name):
    """A cache's values in 64 bits, (blocks, block, nkv, hd)."""
    cache, scale = s[name + "_cache"], s[name + "_scale"]
    if scale is None:
        return cache.double()
    return cache.double() * _two_to(scale.view(U8).int() - 127).permute(0, 2, 1)[..., None]


def _held(x):
    """What the cache holds of heads x (..., hd) in 64 bits: x / 2^e to four
    significant bits, above 2^-9, ties to even."""
    top = x.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(top)                          # top = m 2^e, 1/2 <= m < 1
    e = torch.clamp(e - 9 + (m > 0.875).int(), -126, 127)
    y = x * _two_to(-e)
    step = _two_to(torch.clamp(torch.frexp(y)[1] - 4, min=-9))
    return torch.round(y / step) * step * _two_to(e)


def _exact_read(s, caches):
    c = s["case"]
    out = {"k": [], "v": []}
    for r, n in enumerate(s["starts"].diff().tolist()):
        pages = s["table"][r, :-(-n // c["block"])].long()
        for name, cache in caches.items():
            out[name].append(cache[pages].flatten(0, 1)[:n].flatten(1))
    return {name: torch.cat(rows) for name, rows in out.items()}


def _exact_store(s):
    """The rotation as a product of complex numbers."""
    c = s["case"]
    half = c["rot"] // 2
    row = s["turns"].double()[s["positions"]]
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
    caches = {"k": _whole(s, "k"), "v": _whole(s, "v")}
    block, at = s["slots"] // c["block"], s["slots"] % c["block"]
    caches["k"][block, at] = _held(one(s["key"], c["nkv"], s["k_weight"]))
    caches["v"][block, at] = _held(s["value"].double().unflatten(1, (c["nkv"], c["hd"])))
    return {"q": one(s["query"], c["nq"], s["q_weight"]).flatten(1), **_exact_read(s, caches)}


def _exact_attn(s):
    """Request by request over all of its own tokens, one new token at a time."""
    c, q = s["case"], s["case"]["q"]
    group = c["nq"] // c["nkv"]
    out = torch.zeros(s["out"].shape, dtype=F64, device="cuda").unflatten(1, (c["nkv"], group, c["hd"]))
    query = s["query"].double().unflatten(1, (c["nkv"], group, c["hd"]))
    caches = [_whole(s, "k"), _whole(s, "v")]
    for r, n in enumerate(s["lens"].tolist()):
        pages = s["table"][r, :-(-n // c["block"])].long()
        k, v = (x[pages].flatten(0, 1)[:n].transpose(0, 1).contiguous() for x in caches)
        for j in range(q):
            m = n - q + 1 + j
            if m > 0:
                w = torch.softmax(query[r * q + j] @ k[:, :m].mT / math.sqrt(c["hd"]), -1)
                out[r * q + j] = w @ v[:, :m]
    return out.flatten(1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "read":
        return _exact_read(s, {"k": _whole(s, "k"), "v": _whole(s, "v")})
    return _exact_store(s) if op == "store" else _exact_attn(s)
