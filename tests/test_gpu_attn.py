"""The head norms with rotation and cache write, and the attention over the
paged cache, on the GPU against plain forms in 64 bits on the CPU."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
F64, BF16 = torch.float64, torch.bfloat16


def scs():
    import stateful_causal_short_amd as m
    return m


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def i64(x):
    return torch.tensor(np.asarray(x), dtype=torch.int64, device="cuda")


def randn(g, *shape):
    return torch.randn(*shape, generator=g).to(BF16)


# ---------------------------------------------------------------------------
# norms, rotation, cache write
# ---------------------------------------------------------------------------
def norm_ref(x, w, table, pos, hd, eps, interleaved):
    """(rows, heads, hd) in 64 bits."""
    x = x.to(F64).unflatten(1, (-1, hd))
    x = x / torch.sqrt((x * x).mean(2, keepdim=True) + eps)
    if w is not None:
        x = x * w.to(F64)
    if table is None:
        return x
    rot = table.shape[1]
    half = rot // 2
    cos, sin = table.to(F64)[pos][:, None].split(half, 2)
    a = slice(0, rot, 2) if interleaved else slice(0, half)
    b = slice(1, rot, 2) if interleaved else slice(half, rot)
    y = x.clone()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def check_norm(got, want, hd, weight_max):
    """One bf16 rounding is half a step, 2^-8 of the value. Before it: the sum
    of squares, its root, two factors and the rotation's three operations, in
    fp32: under 16 roundings of 2^-24 of the pair's size, which is at most
    sqrt(2 hd) times the largest weight."""
    tol = 2.0 ** -8 * want.abs() + 16 * 2.0 ** -24 * math.sqrt(2 * hd) * weight_max
    off = (got.to(F64) - want).abs()
    assert bool((off <= tol).all()), float((off / tol).max())


NORMS = [  # nq, nkv, hd, rot, interleaved, table, weights, tokens, block, layout, k_out, in place
    (1, 1, 64, 64, False, "f32", True, 1, 16, "tokens", False, False),
    (4, 2, 128, 128, False, "bf16", True, 7, 48, "tokens", True, False),
    (4, 1, 128, 64, True, "f32", False, 33, 1, "heads", True, True),
    (6, 3, 64, 16, False, "f32", True, 19, 5, "joint", False, True),
    (16, 2, 256, 256, True, "bf16", True, 65, 16, "heads", True, False),
    (7, 7, 256, 8, False, "f32", True, 5, 16, "tokens", True, True),
    (3, 1, 128, 0, False, "f32", True, 21, 16, "none", True, True),
    (8, 8, 64, 48, False, "f32", False, 130, 528, "joint", True, False),
]


def caches(layout, blocks, block, nkv, hd, fill):
    """(k, v) cache tensors (blocks, block, nkv, hd) over three layouts."""
    if layout == "heads":
        t = [torch.full((blocks, nkv, block, hd), fill, dtype=BF16, device="cuda").transpose(1, 2)
             for _ in range(2)]
    elif layout == "joint":
        both = torch.full((blocks, 2, block, nkv, hd), fill, dtype=BF16, device="cuda")
        t = [both[:, 0], both[:, 1]]
    else:
        t = [torch.full((blocks, block, nkv, hd), fill, dtype=BF16, device="cuda")
             for _ in range(2)]
    return t


@pytest.mark.parametrize("case", NORMS, ids=[f"{c[0]}-{c[1]}-{c[2]}-rot{c[3]}-{c[9]}" for c in NORMS])
def test_qk_norm_rope(case):
    nq, nkv, hd, rot, inter, table_t, weights, T, block, layout, k_out, in_place = case
    print(f"[gpu] qk_norm {case}", flush=True)
    g = torch.Generator().manual_seed(T)
    width, pad = (nq + 2 * nkv) * hd, 4
    rows = randn(g, T + 2, width + pad)
    w = [randn(g, hd) for _ in range(2)] if weights else [None, None]
    wmax = max([1.0] + [float(x.abs().max()) for x in w if x is not None])
    table = None
    if rot:
        ang = torch.arange(50, dtype=F64)[:, None] * torch.rand(rot // 2, generator=g, dtype=F64)
        table = torch.cat([ang.cos(), ang.sin()], 1).to(torch.float32 if table_t == "f32" else BF16)
    rng = np.random.default_rng(T)
    pos = rng.integers(0, 50, T)
    pos_call = pos.copy()
    if T > 3:
        pos[1], pos_call[1] = 49, 10 ** 12          # clamped
        pos[2], pos_call[2] = 0, -5
    blocks = -(-T // block) + 2
    slots = rng.permutation(blocks * block)[:T]
    if T > 4:
        slots[3], slots[4] = -1, blocks * block     # not written
    d = rows.cuda()
    split = lambda x: (x[:T, :nq * hd], x[:T, nq * hd:(nq + nkv) * hd],
                       x[:T, (nq + nkv) * hd:width])
    q, k, v = split(d)
    kc, vc = caches(layout, blocks, block, nkv, hd, 3.5)
    cached = layout != "none"
    if in_place:
        qo, ko = q, (k if k_out else None)
    else:
        qo = torch.full((T + 1, nq * hd), 7.5, dtype=BF16, device="cuda")
        ko = torch.full((T + 1, nkv * hd), 7.5, dtype=BF16, device="cuda") if k_out else None
    scs().sc_qk_norm_rope(
        q, k, v if cached else None, qo, ko, *[None if x is None else x.cuda() for x in w],
        None if table is None else table.cuda(), None if table is None else i64(pos_call),
        i64(slots) if cached else None, kc if cached else None, vc if cached else None,
        head_dim=hd, eps=1e-5, interleaved=inter)
    hq, hk, hv = split(rows)
    want_q = norm_ref(hq, w[0], table, pos, hd, 1e-5, inter)
    want_k = norm_ref(hk, w[1], table, pos, hd, 1e-5, inter)
    check_norm(qo[:T].cpu().unflatten(1, (-1, hd)), want_q, hd, wmax)
    if k_out:
        check_norm(ko[:T].cpu().unflatten(1, (-1, hd)), want_k, hd, wmax)
    if not in_place:
        assert bool((qo[T:] == 7.5).all()) and torch.equal(d.cpu(), rows)
    else:
        out = d.cpu()
        assert torch.equal(out[T:], rows[T:]) and torch.equal(out[:, width:], rows[:, width:])
        assert torch.equal(out[:T, (nq + nkv) * hd:width], hv)
        if not k_out:
            assert torch.equal(out[:T, nq * hd:(nq + nkv) * hd], hk)
    kh, vh = kc.cpu(), vc.cpu()
    written = torch.zeros(blocks, block, dtype=torch.bool)
    if cached:
        for t in range(T):
            if 0 <= slots[t] < blocks * block:
                b, i = divmod(int(slots[t]), block)
                written[b, i] = True
                check_norm(kh[b, i], want_k[t], hd, wmax)
                assert torch.equal(vh[b, i].flatten(), hv[t])
    assert bool((kh[~written] == 3.5).all()) and bool((vh[~written] == 3.5).all())


def test_cache_rows_past_four_gigabytes():
    nkv, hd, block = 2, 128, 16
    blocks = 540_000                                   # 2.2e9 elements, 4.4 GB
    print("[gpu] far cache rows", flush=True)
    g = torch.Generator().manual_seed(1)
    cache = torch.empty(blocks, block, nkv, hd, dtype=BF16, device="cuda")
    other = torch.zeros_like(cache)
    n = 40
    x = randn(g, n, 4 * nkv * hd + 2 * nkv * hd).cuda()
    q, k, v = x[:, :1024], x[:, 1024:1280], x[:, 1280:]
    first = (blocks - 3) * block
    qo = torch.empty(n, 1024, dtype=BF16, device="cuda")
    scs().sc_qk_norm_rope(q, k, v, qo, None, None, None, None, None, i64(first + np.arange(n)),
                          cache, other, head_dim=hd)
    want = norm_ref(k.cpu(), None, None, None, hd, 1e-6, False)
    flat = cache.view(-1, nkv, hd)[first:first + n].cpu()
    check_norm(flat, want, hd, 1.0)
    assert torch.equal(other.view(-1, nkv * hd)[first:first + n], v)
    out = torch.empty(1, 1024, dtype=BF16, device="cuda")
    table = i32([[blocks - 3, blocks - 2, blocks - 1]])
    scs().sc_paged_attn_decode(qo[-1:], out, cache, other, table, i32([n]), max_seq_len=48)
    ref, tol = attn_ref(qo[-1:].cpu(), flat[None], v.cpu().view(1, n, nkv, hd), [n], 1, hd ** -0.5)
    check_attn(out.cpu(), ref, tol)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def attn_ref(q, k, v, lens, nq_tok, scale):
    """q (B * n, nq * hd); k, v: per request (L, nkv, hd). (want, tolerance).

    One bf16 rounding of the result is half a step, 2^-8 of it. Before it, all
    in fp32: a score rounds by sqrt(hd) 2^-24 |q||k| and its product with scale
    log2(e) and the difference from the maximum by 2^-23 of its size (which is
    at most |q||k| scale), four times that for the tail; a weight's relative
    error is the score's, and moves the mean by at most twice itself times
    max |v|; exp2 and the sums stay under 2^-20 of max |v|."""
    hd, nkv = k[0].shape[-1], k[0].shape[-2]
    B = len(lens)
    qq = q.to(F64).view(B, nq_tok, nkv, -1, hd)
    want, tol = torch.zeros(qq.shape, dtype=F64), torch.zeros(qq.shape, dtype=F64)
    for r in range(B):
        for j in range(nq_tok):
            n = lens[r] - nq_tok + 1 + j
            if n <= 0:
                continue
            kk, vv = (x[r][:n].to(F64).transpose(0, 1) for x in (k, v))   # (nkv, n, hd)
            s = qq[r, j] @ kk.transpose(1, 2) * scale
            want[r, j] = torch.softmax(s, -1) @ vv
            size = qq[r, j].norm(dim=-1).amax() * kk.norm(dim=-1).amax() * abs(scale)
            delta = 4 * float(size) * (math.sqrt(hd) * 2.0 ** -24 + 2 * 2.0 ** -23)
            tol[r, j] = 2.0 ** -8 * want[r, j].abs() + (2 * delta + 2.0 ** -20) * vv.abs().max()
    return want.flatten(2).flatten(0, 1), tol.flatten(2).flatten(0, 1)


def check_attn(got, want, tol):
    off = (got.to(F64) - want).abs()
    assert bool((off <= tol).all()), \
        f"{int((off > tol).sum())} of {off.numel()} values off, worst {float((off - tol).max()):.3g}"


def paged(g, lens, nkv, hd, block, layout, rng):
    """Random keys and values of each request, laid out in shuffled pages of a
    cache that holds NaN elsewhere (the rest of the last page included)."""
    pages = [-(-n // block) for n in lens]
    blocks = sum(pages) + 2
    kc, vc = caches(layout, blocks, block, nkv, hd, float("nan"))
    order = rng.permutation(blocks)
    table = np.full((len(lens), max(max(pages), 1)), 10 ** 9)      # behind the end: not read
    k = [randn(g, n, nkv, hd) for n in lens]
    v = [randn(g, n, nkv, hd) for n in lens]
    at = 0
    for r, p in enumerate(pages):
        table[r, :p] = order[at:at + p]
        for i in range(p):
            part = slice(i * block, min((i + 1) * block, lens[r]))
            n = part.stop - part.start
            kc[order[at + i], :n] = k[r][part].cuda()
            vc[order[at + i], :n] = v[r][part].cuda()
        at += p
    return kc, vc, table, k, v


ATTNS = [  # nq, nkv, hd, block, q, lens, layout, scale
    (1, 1, 64, 16, 1, [1], "tokens", None),
    (4, 1, 128, 16, 1, [0, 1, 15, 16, 17], "tokens", None),
    (8, 2, 128, 48, 1, [63, 64, 65, 300], "heads", 0.3),
    (14, 2, 64, 16, 3, [2, 3, 40, 0, 129], "joint", None),
    (5, 5, 256, 32, 2, [50, 1, 18], "heads", None),
    (20, 1, 128, 16, 1, [100, 33], "tokens", -0.2),
    (16, 4, 128, 528, 5, [1000, 4, 529, 531], "joint", None),
    (32, 2, 64, 64, 4, [700], "tokens", None),
    (16, 4, 128, 16, 1, [5000, 17, 0, 1234], "tokens", None),
    (2, 2, 256, 16, 1, [3001], "tokens", None),
]


@pytest.mark.parametrize("case", ATTNS, ids=[f"{c[0]}-{c[1]}-{c[2]}-q{c[4]}-{c[5][0]}" for c in ATTNS])
def test_paged_attention(case):
    nq, nkv, hd, block, q, lens, layout, scale = case
    print(f"[gpu] attn {case}", flush=True)
    g = torch.Generator().manual_seed(nq * 100 + q)
    rng = np.random.default_rng(len(lens))
    kc, vc, table, k, v = paged(g, lens, nkv, hd, block, layout, rng)
    B = len(lens)
    query = randn(g, B * q, nq * hd + 8) * 2
    out = torch.full((B * q + 1, nq * hd), 7.5, dtype=BF16, device="cuda")
    wide = i32(np.pad(table, ((0, 0), (0, 3))))
    call = dict(q=q, max_seq_len=max(max(lens), 1), scale=scale)
    scs().sc_paged_attn_decode(query.cuda()[:, :nq * hd], out, kc, vc,
                               wide[:, :table.shape[1]], i32(lens), **call)
    want, tol = attn_ref(query[:, :nq * hd], k, v, lens, q, hd ** -0.5 if scale is None else scale)
    got = out.cpu()
    check_attn(got[:-1], want, tol)
    assert bool((got[-1] == 7.5).all())
    for r, n in enumerate(lens):
        for j in range(q):
            if n - q + j < 0:
                assert bool((got[r * q + j] == 0).all()), "a row that sees nothing"
    again = torch.zeros_like(out)
    scs().sc_paged_attn_decode(query.cuda()[:, :nq * hd], again, kc, vc, i32(table), i32(lens),
                               **call)
    assert torch.equal(again[:-1], out[:-1])


MANY = [  # nq, nkv, hd, q, requests, lengths: more workgroups than the card holds at once
    (8, 4, 64, 1, 400, "some"),        # taken by falling length
    (4, 4, 64, 1, 512, "equal"),       # ... with all of them in one step
    (8, 4, 64, 1, 513, "some"),        # one more than are put in order
    (16, 4, 128, 2, 70, "long"),       # ... and with the length split
    (4, 2, 256, 1, 300, "one"),
]


@pytest.mark.parametrize("case", MANY, ids=[f"{c[1]}x{c[2]}-{c[4]}-{c[5]}" for c in MANY])
def test_paged_attention_many_requests(case):
    """Each request has its rows, whatever the order in which they are taken."""
    nq, nkv, hd, q, B, kind = case
    print(f"[gpu] attn many {case}", flush=True)
    g = torch.Generator().manual_seed(B)
    rng = np.random.default_rng(B)
    lens = {"some": rng.integers(0, 90, B), "equal": np.full(B, 33),
            "long": np.where(np.arange(B) % 9 == 4, rng.integers(2000, 3300, B),
                             rng.integers(0, 40, B)),
            "one": np.where(np.arange(B) == 250, 129, 1)}[kind].tolist()
    kc, vc, table, k, v = paged(g, lens, nkv, hd, 16, "tokens", rng)
    query = randn(g, B * q, nq * hd)
    out = torch.full((B * q + 1, nq * hd), 7.5, dtype=BF16, device="cuda")
    call = dict(q=q, max_seq_len=max(lens))
    scs().sc_paged_attn_decode(query.cuda(), out[:-1], kc, vc, i32(table), i32(lens), **call)
    want, tol = attn_ref(query, k, v, lens, q, hd ** -0.5)
    got = out.cpu()
    check_attn(got[:-1].view(B * q, nq, hd), want.view(B * q, nq, hd), tol.view(B * q, nq, hd))
    assert bool((got[-1] == 7.5).all())
    again = torch.zeros_like(out)
    scs().sc_paged_attn_decode(query.cuda(), again[:-1], kc, vc, i32(table), i32(lens), **call)
    assert torch.equal(again[:-1].cpu(), got[:-1])


def test_pages_outside_the_cache_hold_no_token():
    """A table entry outside the cache: its tokens are as if they were absent."""
    nq, nkv, hd, block = 4, 2, 64, 16
    print("[gpu] attn bad pages", flush=True)
    g = torch.Generator().manual_seed(3)
    rng = np.random.default_rng(3)
    lens = [70, 40]
    kc, vc, table, k, v = paged(g, lens, nkv, hd, block, "tokens", rng)
    bad = table.copy()
    bad[0, 1], bad[0, 3], bad[1, :] = -1, kc.shape[0], 2 ** 31 - 1
    query = randn(g, 2, nq * hd)
    out = torch.full((2, nq * hd), 7.5, dtype=BF16, device="cuda")
    scs().sc_paged_attn_decode(query.cuda(), out, kc, vc, i32(bad), i32(lens), max_seq_len=80)
    keep = [t for t in range(70) if t // block not in (1, 3)]
    want, tol = attn_ref(query[:1], [k[0][keep]], [v[0][keep]], [len(keep)], 1, hd ** -0.5)
    check_attn(out.cpu()[:1], want, tol)
    assert bool((out[1] == 0).all())


def test_lengths_are_clamped():
    nq, nkv, hd, block = 2, 1, 128, 16
    g = torch.Generator().manual_seed(4)
    print("[gpu] attn clamped lengths", flush=True)
    kc, vc, table, k, v = paged(g, [32, 20], nkv, hd, block, "tokens", np.random.default_rng(4))
    query = randn(g, 2, nq * hd)
    out = torch.zeros(2, nq * hd, dtype=BF16, device="cuda")
    scs().sc_paged_attn_decode(query.cuda(), out, kc, vc, i32(table), i32([2 ** 31 - 1, -7]),
                               max_seq_len=32)
    want, tol = attn_ref(query[:1], k, v, [32], 1, hd ** -0.5)
    check_attn(out.cpu()[:1], want, tol)
    assert bool((out[1] == 0).all())


def test_empty_calls():
    print("[gpu] attn empty calls", flush=True)
    S = scs()
    kc = torch.zeros(2, 16, 1, 64, dtype=BF16, device="cuda")
    out = torch.full((2, 64), 7.5, dtype=BF16, device="cuda")
    q = torch.ones(2, 64, dtype=BF16, device="cuda")
    none = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    S.sc_paged_attn_decode(q[:0], out[:0], kc, kc, none, i32([]), max_seq_len=64)
    S.sc_qk_norm_rope(q[:0], q[:0], q[:0], out[:0], None, None, None, None, None, i64([]), kc, kc,
                      head_dim=64)
    torch.cuda.synchronize()
    assert bool((out == 7.5).all()) and bool((kc == 0).all())
    S.sc_paged_attn_decode(q, out, kc, kc, none.new_zeros(2, 4), i32([0, 0]), max_seq_len=0)
    assert bool((out == 0).all())


@pytest.mark.parametrize("hd,value", [(64, float("nan")), (128, float("inf")), (256, float("-inf"))])
def test_later_drafts_do_not_reach_earlier_ones(hd, value):
    """A non-finite value row of draft j is in the results of drafts >= j alone."""
    nq, nkv, q, lens = 8, 2, 4, [37, 4, 64]
    print(f"[gpu] attn draft {value}", flush=True)
    g = torch.Generator().manual_seed(5)
    kc, vc, table, k, v = paged(g, lens, nkv, hd, 16, "tokens", np.random.default_rng(5))
    query = randn(g, 3 * q, nq * hd)
    args = (kc, vc, i32(table), i32(lens))
    clean = torch.zeros(3 * q, nq * hd, dtype=BF16, device="cuda")
    scs().sc_paged_attn_decode(query.cuda(), clean, *args, q=q, max_seq_len=64)
    for r, n in enumerate(lens):                     # draft 2, one value of each head
        t = n - q + 2
        vc[table[r, t // 16], t % 16, :, 5] = value
    out = torch.zeros_like(clean)
    scs().sc_paged_attn_decode(query.cuda(), out, *args, q=q, max_seq_len=64)
    a, b = (x.cpu().view(3, q, nq, hd) for x in (clean, out))
    assert torch.equal(a[:, :2], b[:, :2])
    hit = b[:, 2:, :, 5]
    assert bool(hit.isnan().all() if math.isnan(value) else (hit == value).all())
    rest = [i for i in range(hd) if i != 5]
    assert bool(b[:, 2:][..., rest].isfinite().all())
    off = (a[:, 2:][..., rest].float() - b[:, 2:][..., rest].float()).abs()
    assert float(off.max()) <= 2.0 ** -7 * float(a.float().abs().max())   # another order of sums


def test_graph_replays_and_own_workspace():
    nq, nkv, hd, block = 8, 2, 128, 16
    print("[gpu] attn graph", flush=True)
    g = torch.Generator().manual_seed(6)
    lens = [3000, 700]
    kc, vc, table, k, v = paged(g, lens, nkv, hd, block, "tokens", np.random.default_rng(6))
    S = scs()
    x = randn(g, 2, (nq + 2 * nkv) * hd).cuda()
    q, key, val = x[:, :nq * hd], x[:, nq * hd:(nq + nkv) * hd], x[:, (nq + nkv) * hd:]
    where = [int(table[r, (n - 1) // block]) * block + (n - 1) % block for r, n in enumerate(lens)]
    qo = torch.empty(2, nq * hd, dtype=BF16, device="cuda")
    out = torch.zeros_like(qo)
    tab, ln, sl = i32(table), i32(lens), i64(where)
    need = S.sc_paged_attn_workspace_bytes(2, max_seq_len=3000, num_q_heads=nq, num_kv_heads=nkv,
                                           head_dim=hd)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def step(w):
        S.sc_qk_norm_rope(q, key, val, qo, None, None, None, None, None, sl, kc, vc, head_dim=hd)
        S.sc_paged_attn_decode(qo, out, kc, vc, tab, ln, max_seq_len=3000, workspace=w)

    step(None)
    want = out.clone()
    k2, v2 = [t.clone() for t in k], [t.clone() for t in v]
    for r, n in enumerate(lens):
        k2[r][n - 1] = norm_ref(key[r:r + 1].cpu(), None, None, None, hd, 1e-6, False)[0].to(BF16)
        v2[r][n - 1] = val[r].cpu().view(nkv, hd)
    ref, tol = attn_ref(qo.cpu(), k2, v2, lens, 1, hd ** -0.5)
    check_attn(want.cpu(), ref, tol)
    graphs = []
    for w in (None, ws):
        gr = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(gr):
            step(w)
        graphs.append(gr)
    for gr in graphs * 2:
        out.zero_()
        step(None)
        out.zero_()
        torch.cuda.synchronize()
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    side = torch.cuda.Stream()
    out.zero_()
    torch.cuda.synchronize()
    S.sc_paged_attn_decode(qo, out, kc, vc, tab, ln, max_seq_len=3000, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    with pytest.raises(S.ScError):
        S.sc_paged_attn_decode(qo, out, kc, vc, tab, ln, max_seq_len=3000, workspace=ws[:need - 16])


def test_cca_then_norm_cache_and_attention():
    """The steps of such a layer together, for three decode steps: the CCA conv,
    norms with rotation into the cache, attention; the last two against 64 bits
    on what the step before gave."""
    import synthetic
    from tests._gpu import dev
    S = scs()
    nq, nkv, hd, block, n = 4, 2, 128, 16, 3
    print("[gpu] cca -> norm -> attention", flush=True)
    cc = synthetic.cca_case("attn_chain", synthetic.SEED_BASE + 91, nq=nq, nkv=nkv, hd=hd,
                            num_decodes=n, num_prefills=0, num_prefill_tokens=0, num_slots=8)
    g = torch.Generator().manual_seed(8)
    lens = [5, 30, 47]
    kc, vc, table, k, v = paged(g, [m + 3 for m in lens], nkv, hd, block, "joint",
                                np.random.default_rng(8))
    conv_state, delayed = dev(cc.conv_state), dev(cc.delayed_state)
    weights = [dev(x) for x in (cc.w_dw, cc.b_dw, cc.w_gr, cc.b_gr)]
    slots = i32([1, 4, 6])
    ang = torch.arange(64, dtype=F64)[:, None] * torch.rand(hd // 2, generator=g, dtype=F64)
    rope = torch.cat([ang.cos(), ang.sin()], 1).float()
    wq, wk = randn(g, hd), randn(g, hd)
    width = (nq + 2 * nkv) * hd
    for step in range(3):
        rows = torch.empty(n, width, dtype=BF16, device="cuda")
        raw = [randn(g, n, w).cuda() for w in (nq * hd, nkv * hd, nkv * hd // 2, nkv * hd // 2)]
        S.sc_cca_qk_conv(*raw, rows, *weights, None, conv_state, delayed, slots, None, None, None,
                         num_q_heads=nq, num_kv_heads=nkv, head_dim=hd, t0=cc.t0, t1=cc.t1)
        before = rows.cpu()
        q, key, val = rows[:, :nq * hd], rows[:, nq * hd:(nq + nkv) * hd], rows[:, (nq + nkv) * hd:]
        now = [m + step for m in lens]
        where = [int(table[r, m // block]) * block + m % block for r, m in enumerate(now)]
        S.sc_qk_norm_rope(q, key, val, q, None, wq.cuda(), wk.cuda(), rope.cuda(), i64(now),
                          i64(where), kc, vc, head_dim=hd)
        out = torch.empty(n, nq * hd, dtype=BF16, device="cuda")
        S.sc_paged_attn_decode(q, out, kc, vc, i32(table), i32([m + 1 for m in now]),
                               max_seq_len=64)
        hq, hk, hv = (before[:, a:b] for a, b in ((0, nq * hd), (nq * hd, (nq + nkv) * hd),
                                                  ((nq + nkv) * hd, width)))
        wmax = max(1.0, float(wq.abs().max()), float(wk.abs().max()))
        check_norm(q.cpu().unflatten(1, (-1, hd)), norm_ref(hq, wq, rope, now, hd, 1e-6, False), hd, wmax)
        new_k = norm_ref(hk, wk, rope, now, hd, 1e-6, False)
        for r, m in enumerate(now):
            got_k = kc[where[r] // block, where[r] % block].cpu()
            check_norm(got_k, new_k[r], hd, wmax)
            k[r][m], v[r][m] = got_k, hv[r].view(nkv, hd)
        want, tol = attn_ref(q.cpu(), k, v, [m + 1 for m in now], 1, hd ** -0.5)
        check_attn(out.cpu(), want, tol)
