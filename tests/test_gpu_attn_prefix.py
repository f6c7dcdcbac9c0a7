"""Attention over shared prefixes, on the GPU against a plain form in 64 bits on the
CPU that takes each request by itself."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests._fp8 import BF16, F64, U8, caches_fp8, put  # noqa: E402
from tests.test_gpu_attn import attn_ref, caches, check_attn, i32, i64, randn, scs  # noqa: E402

pytestmark = pytest.mark.gpu


def shared(g, sizes, prefixes, own, nkv, hd, block, layout, fp8, rng):
    """Caches of requests in groups: the first `prefixes[g]` tokens in shared blocks, a
    part of a block copied for each request, then own[r] tokens each. Requests
    with own[r] < 0 have a cache that ends -own[r] tokens before the prefix does.
    (caches, table, lens, values of the keys and of the values per request)."""
    lens, group = [], np.repeat(np.arange(len(sizes)), sizes)
    for r, gi in enumerate(group):
        lens.append(max(0, prefixes[gi] + own[r]))
    need = [-(-n // block) for n in lens]
    whole = [p // block for p in prefixes]
    blocks = sum(need) + sum(whole) + 2
    if fp8:
        c = caches_fp8(layout, blocks, block, nkv, hd)
    else:
        k, v = caches(layout, blocks, block, nkv, hd, float("nan"))
        c = [k, v]

    def write(which, b, x):
        if fp8:
            return put(c[2 * which], c[2 * which + 1], b, 0, x)
        c[which][b, :len(x)] = x.cuda()
        return x.to(F64)
    order = list(rng.permutation(blocks))
    table = np.full((len(lens), max(max(need), 1)), 10 ** 9)
    made = [[], []]
    made_prefix = []
    for gi, p in enumerate(prefixes):
        x = [randn(g, p, nkv, hd), randn(g, p, nkv, hd)]
        pages = [order.pop() for _ in range(whole[gi])]
        vals = [[write(w, pages[i], x[w][i * block:(i + 1) * block]) for i in range(whole[gi])]
                for w in range(2)]
        made_prefix.append((x, pages, vals))
    for r, gi in enumerate(group):
        x, pages, vals = made_prefix[gi]
        n, shared_pages = lens[r], min(whole[gi], lens[r] // block)
        table[r, :shared_pages] = pages[:shared_pages]
        rest = n - shared_pages * block
        fresh = [randn(g, max(0, n - prefixes[gi]), nkv, hd) for _ in range(2)]
        mine = [order.pop() for _ in range(-(-rest // block))]
        table[r, shared_pages:shared_pages + len(mine)] = mine
        for w in range(2):
            tail = torch.cat([x[w][shared_pages * block:min(n, prefixes[gi])], fresh[w]])
            got = vals[w][:shared_pages] + [write(w, b, tail[i * block:(i + 1) * block])
                                            for i, b in enumerate(mine)]
            made[w].append(torch.cat(got) if got else torch.zeros(0, nkv, hd, dtype=F64))
    return c, table, lens, made[0], made[1]


def ref(query, k, v, lens, q, scale):
    """attn_ref's values and tolerance, and for the weights over the prefix, each
    rounded to bf16 by half a step, 2^-8 of it, with their sum that of the rounded
    ones: sum p d (v - out) / sum p is at most 2^-8 times twice the largest value.
    Own tokens' weights over codes: 2^-16."""
    want, tol = attn_ref(query, k, v, lens, q, scale)
    top = max([float(x.abs().max()) for x in v if x.numel()] or [0.0])
    return want, tol + (2.0 ** -7 + 2.0 ** -16) * top


CASES = [  # nq, nkv, hd, block, q, group sizes, prefixes, own tokens (a range, or each), layout, scale
    (4, 1, 64, 16, 1, [3], [32], (1, 40), "tokens", None),
    (8, 2, 128, 16, 1, [2, 1], [33, 1], (1, 20), "tokens", None),
    (4, 4, 128, 48, 2, [5, 3], [100, 7], (2, 150), "joint", 0.2),
    (16, 4, 128, 16, 1, [20], [700], (1, 60), "heads", None),          # 80 rows
    (32, 4, 64, 64, 1, [40, 1, 30], [1000, 64, 333], (1, 99), "tokens", None),
    (14, 2, 128, 16, 5, [10], [129], (5, 30), "tokens", -0.1),         # 350 rows
    (6, 3, 256, 16, 1, [9], [200], (1, 70), "joint", None),
    (8, 1, 256, 32, 3, [12, 4], [65, 300], (3, 50), "tokens", None),   # 288 and 96 rows
    (2, 1, 64, 16, 1, [300], [50], (1, 5), "tokens", 0.0),             # 600 rows
    (4, 1, 128, 16, 1, [70], [5001], (1, 9), "tokens", None),          # split prefix
    (4, 2, 128, 528, 1, [3], [2000], (1, 1500), "tokens", None),       # own tokens split
    (1, 1, 64, 16, 1, [1] * 70, [17] * 70, (1, 3), "tokens", None),    # more groups than lanes
]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}-{c[1]}-{c[2]}-q{c[4]}-{c[5][0]}on{c[6][0]}" for c in CASES])
def test_shared_prefix(case, fp8):
    nq, nkv, hd, block, q, sizes, prefixes, own, layout, scale = case
    print(f"[gpu] prefix {case} {fp8}", flush=True)
    S = scs()
    g = torch.Generator().manual_seed(nq * 100 + sum(sizes))
    rng = np.random.default_rng(hd)
    B = sum(sizes)
    c, table, lens, k, v = shared(g, sizes, prefixes, rng.integers(own[0], own[1] + 1, B), nkv, hd,
                                  block, layout, fp8, rng)
    query = randn(g, B * q, nq * hd + 8)
    out = torch.full((B * q + 1, nq * hd), 7.5, dtype=BF16, device="cuda")
    starts = i32(np.concatenate([[0], np.cumsum(sizes)]))
    call = dict(q=q, max_seq_len=max(lens), max_prefix_len=max(prefixes))
    need = S.sc_paged_attn_prefix_workspace_bytes(B, num_groups=len(sizes), num_q_heads=nq,
                                                  num_kv_heads=nkv, head_dim=hd, **call)
    room = torch.full((need + 64,), 0xFF, dtype=U8, device="cuda")
    fn = S.sc_paged_attn_prefix_fp8 if fp8 else S.sc_paged_attn_prefix
    wide = i32(np.pad(table, ((0, 0), (0, 3))))
    fn(query.cuda()[:, :nq * hd], out, *c, wide[:, :table.shape[1]], i32(lens), starts,
       i32(prefixes), scale=scale, workspace=room[:need], **call)
    want, tol = ref(query[:, :nq * hd], k, v, lens, q, hd ** -0.5 if scale is None else scale)
    got = out.cpu()
    check_attn(got[:-1], want, tol)
    assert bool((got[-1] == 7.5).all()) and bool((room[need:] == 0xFF).all())
    again = torch.zeros_like(out)
    fn(query.cuda()[:, :nq * hd], again, *c, i32(table), i32(lens), starts, i32(prefixes),
       scale=scale, **call)
    assert torch.equal(again[:-1], out[:-1])


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_error_of_the_whole(fp8):
    """Over random data: the output's rounding, half a step at most and so 2^-8 / sqrt 3 in
    the mean square, and as much again from the weights', which are independent."""
    nq, nkv, hd, B = 16, 4, 128, 70
    print(f"[gpu] prefix error {fp8}", flush=True)
    g = torch.Generator().manual_seed(11)
    c, table, lens, k, v = shared(g, [B], [1500], np.full(B, 8), nkv, hd, 16, "tokens", fp8,
                                  np.random.default_rng(0))
    query = randn(g, B, nq * hd)
    out = torch.empty(B, nq * hd, dtype=BF16, device="cuda")
    fn = scs().sc_paged_attn_prefix_fp8 if fp8 else scs().sc_paged_attn_prefix
    fn(query.cuda(), out, *c, i32(table), i32(lens), i32([0, B]), i32([1500]), max_seq_len=1508,
       max_prefix_len=1500)
    want, _ = attn_ref(query, k, v, lens, 1, hd ** -0.5)
    rel = float((out.cpu().to(F64) - want).norm() / want.norm())
    assert rel <= 2.0 ** -8 * (2 / 3) ** 0.5, rel


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("q", [1, 3])
def test_requests_that_do_not_see_the_whole_prefix(q, fp8):
    """Empty and short requests in a group, in any place, requests of no group, groups of
    none, prefixes of no tokens and longer than all requests."""
    nq, nkv, hd, block = 8, 2, 128, 16
    print(f"[gpu] prefix short requests {q} {fp8}", flush=True)
    g = torch.Generator().manual_seed(q)
    rng = np.random.default_rng(q)
    sizes, prefixes = [4, 5, 3, 6], [40, 100, 16, 64]
    own = np.array([3, 9, 3, 4, -100, -60, 7, q - 1, -1, 5, 5, 5, -64, -64, -64, -64, -64, -64])
    c, table, lens, k, v = shared(g, sizes, prefixes, own, nkv, hd, block, "tokens", fp8, rng)
    B = sum(sizes)
    query = randn(g, B * q, nq * hd)
    want, tol = ref(query, k, v, lens, q, hd ** -0.5)
    fn = scs().sc_paged_attn_prefix_fp8 if fp8 else scs().sc_paged_attn_prefix
    for starts, given in (([0, 4, 9, 12, 18], prefixes),             # as they are
                          ([4, 4, 9, 12, 12], [99, 100, 16, 3]),     # the first and last in no group
                          ([0, 4, 9, 9, 9, 12], [0, 100, 5, 0, -7]), # no tokens, empty groups
                          ([0, 4, 9, 12, 18], [40, 10 ** 9, 16, 64]),   # beyond max_prefix_len
                          ([0], [])):
        out = torch.full((B * q, nq * hd), 7.5, dtype=BF16, device="cuda")
        fn(query.cuda(), out, *c, i32(table), i32(lens), i32(starts), i32(given), q=q, max_seq_len=max(lens),
           max_prefix_len=100)
        got = out.cpu()
        check_attn(got, want, tol)
        for r, n in enumerate(lens):
            for j in range(q):
                if n - q + j < 0:
                    assert bool((got[r * q + j] == 0).all())


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_bad_pages_in_a_prefix(fp8):
    """A block outside the cache holds no token of the prefix."""
    nq, nkv, hd, block, B = 8, 2, 64, 16, 6
    print(f"[gpu] prefix bad pages {fp8}", flush=True)
    g = torch.Generator().manual_seed(3)
    c, table, lens, k, v = shared(g, [B], [200], np.arange(1, 7) * 7, nkv, hd, block, "tokens", fp8,
                                  np.random.default_rng(3))
    bad = table.copy()
    bad[:, 1], bad[:, 5], bad[:, 11] = -1, c[0].shape[0], 2 ** 31 - 1
    keep = [[t for t in range(n) if t // block not in (1, 5, 11)] for n in lens]
    query = randn(g, B, nq * hd)
    out = torch.empty(B, nq * hd, dtype=BF16, device="cuda")
    fn = scs().sc_paged_attn_prefix_fp8 if fp8 else scs().sc_paged_attn_prefix
    fn(query.cuda(), out, *c, i32(bad), i32(lens), i32([0, B]), i32([200]), max_seq_len=max(lens),
       max_prefix_len=200)
    want, tol = ref(query, [x[s] for x, s in zip(k, keep)], [x[s] for x, s in zip(v, keep)],
                    [len(s) for s in keep], 1, hd ** -0.5)
    check_attn(out.cpu(), want, tol)


def test_infinities_in_a_prefix():
    """An infinite value in the prefix reaches its column of every row, a key with an
    infinity makes rows that score it plus infinity NaN and others not see it."""
    nq, nkv, hd, B, P = 2, 1, 64, 5, 64
    print("[gpu] prefix infinities", flush=True)
    g = torch.Generator().manual_seed(3)
    c, table, lens, k, v = shared(g, [B], [P], np.full(B, 3), nkv, hd, 16, "tokens", False,
                                  np.random.default_rng(3))
    query = randn(g, B, nq * hd)
    c[1][int(table[0, 1]), 5, 0, 9] = float("inf")
    c[0][int(table[0, 2]), 2, 0, 0] = float("inf")
    up = (query.view(B, nq, hd)[..., 0] > 0)
    out = torch.empty(B, nq * hd, dtype=BF16, device="cuda")
    scs().sc_paged_attn_prefix(query.cuda(), out, *c, i32(table), i32(lens), i32([0, B]), i32([P]),
                               max_seq_len=P + 3, max_prefix_len=P)
    got = out.cpu().view(B, nq, hd)
    assert bool(got[up].isnan().all())
    assert bool((got[~up][:, 9] == float("inf")).all())
    keep = [t for t in range(P + 3) if t != 34]
    want, tol = ref(query, [x[keep] for x in k], [x[keep] for x in v], [len(keep)] * B, 1, hd ** -0.5)
    rest = [i for i in range(hd) if i != 9]
    check_attn(got[~up][:, rest], want.view(B, nq, hd)[~up][:, rest], tol.view(B, nq, hd)[~up][:, rest])


def test_lowest_and_growing_scores():
    """Scores that rise from tile to tile by more and by less than what outputs are
    rescaled for, and scores near the lowest fp32 value."""
    hd, P, B = 64, 640, 4
    print("[gpu] prefix growing scores", flush=True)
    g = torch.Generator().manual_seed(6)
    steps = torch.linspace(-300, 300, P)[:, None] * (1 + torch.arange(P)[:, None] % 3)
    for key, first in ((steps, 1.0), (torch.full((P, 1), -2.0 ** 63), 2.0 ** 64)):
        k = torch.zeros(P + 16, 1, hd, dtype=BF16)
        k[:P, 0, :1] = key.to(BF16)
        if first > 1:
            k[P:, 0, 0] = -2.0 ** 63
        v = randn(g, P + 16, 1, hd)
        query = torch.zeros(B, hd, dtype=BF16)
        query[:, 0] = torch.tensor([first] * B)
        out = torch.empty(B, hd, dtype=BF16, device="cuda")
        scale = 1.29 if first > 1 else 0.11
        table = np.tile(np.arange(P // 16 + 1), (B, 1))
        scs().sc_paged_attn_prefix(query.cuda(), out, k.cuda().view(-1, 16, 1, hd),
                                   v.cuda().view(-1, 16, 1, hd), i32(table), i32([P + 1] * B), i32([0, B]),
                                   i32([P]), max_seq_len=P + 1, max_prefix_len=P, scale=scale)
        s = query.to(F64) @ k[:P + 1, 0].to(F64).T * scale
        want = torch.softmax(s, -1) @ v[:P + 1, 0].to(F64)
        # the rounded weights, 2^-7 of the largest value; the scores themselves, below 2^7 in
        # the first part, round by 2^-24 of that twice; equal in the second
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -7 + 2.0 ** -13) * float(v.float().abs().max())
        assert bool(((out.cpu().to(F64) - want).abs() <= tol).all())


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_captured_prefix(fp8):
    """Replays with other lengths, groups and prefixes give the eager results."""
    nq, nkv, hd, block = 8, 2, 128, 16
    print(f"[gpu] prefix graph {fp8}", flush=True)
    g = torch.Generator().manual_seed(8)
    sizes, prefixes = [30, 12], [600, 144]
    B = sum(sizes)
    c, table, lens, k, v = shared(g, sizes, prefixes, np.full(B, 40), nkv, hd, block, "tokens", fp8,
                                  np.random.default_rng(3))
    S = scs()
    fn = S.sc_paged_attn_prefix_fp8 if fp8 else S.sc_paged_attn_prefix
    table = i32(np.where(table > 10 ** 8, 0, table))
    query = randn(g, B, nq * hd).cuda()
    n, starts, pre = i32(lens), i32([0, 30, 42]), i32(prefixes)
    size = dict(max_seq_len=640, max_prefix_len=600)
    need = S.sc_paged_attn_prefix_workspace_bytes(B, num_groups=2, num_q_heads=nq, num_kv_heads=nkv,
                                                  head_dim=hd, **size)
    rooms = [torch.empty(need, dtype=U8, device="cuda") for _ in range(2)]
    outs = [torch.empty(B, nq * hd, dtype=BF16, device="cuda") for _ in range(2)]
    call = lambda o, w: fn(query, o, *c, table, n, starts, pre, workspace=w, **size)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(outs[0], rooms[0])
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for o, w in zip(outs, rooms):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(o, w)
    for i in range(4):
        query.copy_(randn(g, B, nq * hd))
        n.copy_(i32([max(0, x - 11 * i * (r % 5)) for r, x in enumerate(lens)]))
        starts.copy_(i32([[0, 30, 42], [0, 30, 30], [2, 30, 40], [0, 0, 0]][i]))
        pre.copy_(i32([[600, 144], [599, 0], [16, 144], [0, 0]][i]))
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.current_stream())
            graphs[1].replay()
        graphs[0].replay()
        torch.cuda.current_stream().wait_stream(side)
        eager = torch.empty_like(outs[0])
        call(eager, None)
        assert torch.equal(outs[0], eager) and torch.equal(outs[1], eager)
        want, tol = ref(query.cpu(), k, v, n.tolist(), 1, hd ** -0.5)
        check_attn(eager.cpu(), want, tol)
