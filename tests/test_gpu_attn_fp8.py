"""Attention over the quantised paged cache, on the GPU against a plain form in 64
bits on the CPU that reads the same codes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests._fp8 import BF16, F64, U8, caches_fp8, paged_fp8, put  # noqa: E402
from tests.test_gpu_attn import attn_ref, check_attn, i32, i64, randn, scs  # noqa: E402

pytestmark = pytest.mark.gpu


def ref(query, k, v, lens, q, scale):
    """attn_ref's values and tolerance, and for the weights in two bf16 parts: each
    rounds by half a step, 2^-8, so the second leaves 2^-16 of the weight, which
    moves the mean of the values by at most that times the largest."""
    want, tol = attn_ref(query, k, v, lens, q, scale)
    top = max([float(x.abs().max()) for x in v if x.numel()] or [0.0])
    return want, tol + 2.0 ** -16 * top


ATTNS = [  # nq, nkv, hd, block, q, lens, layout, scale
    (1, 1, 64, 16, 1, [1], "tokens", None),
    (4, 1, 128, 16, 1, [0, 1, 15, 16, 17], "tokens", None),
    (8, 2, 128, 48, 1, [31, 32, 33, 127, 128, 129, 300], "heads", 0.3),
    (14, 2, 64, 16, 3, [2, 3, 40, 0, 129], "joint", None),
    (5, 5, 256, 32, 2, [50, 1, 18], "heads", None),
    (20, 1, 128, 16, 1, [100, 33], "tokens", -0.2),
    (16, 4, 128, 528, 5, [1000, 4, 529, 531], "joint", None),
    (32, 2, 64, 64, 4, [700], "tokens", 0.0),
    (16, 4, 128, 16, 1, [5000, 17, 0, 1234], "tokens", None),
    (2, 2, 256, 16, 1, [3001], "tokens", None),
    (7, 1, 128, 16, 1, [3500], "tokens", None),
]


@pytest.mark.parametrize("case", ATTNS, ids=[f"{c[0]}-{c[1]}-{c[2]}-q{c[4]}-{c[5][0]}" for c in ATTNS])
def test_attention_over_codes(case):
    nq, nkv, hd, block, q, lens, layout, scale = case
    print(f"[gpu] attn fp8 {case}", flush=True)
    S = scs()
    g = torch.Generator().manual_seed(nq * 100 + q)
    c, table, k, v = paged_fp8(g, lens, nkv, hd, block, layout, np.random.default_rng(len(lens)))
    B, top = len(lens), max(max(lens), 1)
    query = randn(g, B * q, nq * hd + 8) * 2
    out = torch.full((B * q + 1, nq * hd), 7.5, dtype=BF16, device="cuda")
    wide = i32(np.pad(table, ((0, 0), (0, 3))))
    need = S.sc_paged_attn_fp8_workspace_bytes(B, q=q, max_seq_len=top, num_q_heads=nq,
                                               num_kv_heads=nkv, head_dim=hd)
    room = torch.full((need + 64,), 0xFF, dtype=U8, device="cuda")
    call = dict(q=q, max_seq_len=top, scale=scale)
    S.sc_paged_attn_decode_fp8(query.cuda()[:, :nq * hd], out, *c, wide[:, :table.shape[1]],
                               i32(lens), **call, workspace=room[:need])
    want, tol = ref(query[:, :nq * hd], k, v, lens, q, hd ** -0.5 if scale is None else scale)
    got = out.cpu()
    check_attn(got[:-1], want, tol)
    assert bool((got[-1] == 7.5).all()) and bool((room[need:] == 0xFF).all())
    for r, n in enumerate(lens):
        for j in range(q):
            if n - q + j < 0:
                assert bool((got[r * q + j] == 0).all()), "a row that sees nothing"
    again = torch.zeros_like(out)
    S.sc_paged_attn_decode_fp8(query.cuda()[:, :nq * hd], again, *c, i32(table), i32(lens), **call)
    assert torch.equal(again[:-1], out[:-1])


MANY = [  # nq, nkv, hd, q, requests, lengths, max_seq_len
    (8, 4, 64, 1, 400, "some", 700),
    (16, 4, 128, 2, 70, "long", 0),
    (4, 2, 256, 1, 300, "one", 512),
    (2, 1, 64, 2, 1030, "few", 0),      # one split, a wave's tiles past 64 and past 128
]


@pytest.mark.parametrize("case", MANY, ids=[f"{c[1]}x{c[2]}-{c[4]}-{c[5]}" for c in MANY])
def test_many_requests_over_codes(case):
    """Each request has its rows, whatever the order in which they are taken."""
    nq, nkv, hd, q, B, kind, top = case
    print(f"[gpu] attn fp8 many {case}", flush=True)
    g = torch.Generator().manual_seed(B)
    rng = np.random.default_rng(B)
    lens = {"some": rng.integers(0, 90, B),
            "long": np.where(np.arange(B) % 9 == 4, rng.integers(2000, 3300, B), rng.integers(0, 40, B)),
            "few": np.where(np.arange(B) == 77, 9001, np.where(np.arange(B) == 900, 4289, 3)),
            "one": np.where(np.arange(B) == 250, 129, 1)}[kind].tolist()
    c, table, k, v = paged_fp8(g, lens, nkv, hd, 16, "tokens", rng)
    top = top or max(lens)
    wide = np.full((B, -(-top // 16)), 10 ** 9)
    wide[:, :table.shape[1]] = table
    query = randn(g, B * q, nq * hd)
    out = torch.empty(B * q, nq * hd, dtype=BF16, device="cuda")
    scs().sc_paged_attn_decode_fp8(query.cuda(), out, *c, i32(wide), i32(lens), q=q, max_seq_len=top)
    want, tol = ref(query, k, v, lens, q, hd ** -0.5)
    check_attn(out.cpu(), want, tol)


def test_bad_pages_and_late_nans():
    """Pages outside the cache hold no token; a NaN code in a value that only later
    drafts see leaves the earlier rows as they were."""
    nq, nkv, hd, block, q = 4, 2, 64, 16, 3
    print("[gpu] attn fp8 bad pages, late NaN", flush=True)
    g = torch.Generator().manual_seed(3)
    lens = [70, 40, 50]
    c, table, k, v = paged_fp8(g, lens, nkv, hd, block, "tokens", np.random.default_rng(3))
    bad = table.copy()
    bad[0, 1], bad[0, 3], bad[1, :] = -1, c[0].shape[0], 2 ** 31 - 1
    c[2].view(U8)[table[2, 48 // block], 48 % block, 1, 7] = 0xFF     # token 48: rows 1 and 2
    query = randn(g, 3 * q, nq * hd)
    out = torch.full((3 * q, nq * hd), 7.5, dtype=BF16, device="cuda")
    scs().sc_paged_attn_decode_fp8(query.cuda(), out, *c, i32(bad), i32(lens), q=q, max_seq_len=80)
    got = out.cpu()
    keep = [t for t in range(70) if t // block not in (1, 3)]
    want, tol = ref(query[:q], [k[0][keep]], [v[0][keep]], [len(keep)], q, hd ** -0.5)
    check_attn(got[:q], want, tol)
    assert bool((got[q:2 * q] == 0).all())
    want, tol = ref(query[2 * q:], [k[2]], [v[2]], [50], q, hd ** -0.5)
    rows = got[2 * q:].view(q, nq, hd).clone()
    hit = torch.zeros(q, nq, hd, dtype=torch.bool)
    hit[1:, 2:, 7] = True
    assert bool(rows[hit].isnan().all())
    rows[hit] = want.view(q, nq, hd)[hit].to(BF16)
    check_attn(rows.flatten(1), want, tol)


def test_undefined_scale_of_a_later_draft():
    """A scale byte of 255 and NaN codes in a token that only the last draft sees, as
    in a place that is still to be written, leave the other rows as they were."""
    nq, nkv, hd, q = 4, 2, 128, 3
    print("[gpu] attn fp8 late scale", flush=True)
    g = torch.Generator().manual_seed(9)
    lens = [50, 33]
    c, table, k, v = paged_fp8(g, lens, nkv, hd, 16, "tokens", np.random.default_rng(9))
    for r, n in enumerate(lens):
        page, at = table[r, (n - 1) // 16], (n - 1) % 16
        for x in (0, 2):
            c[x].view(U8)[page, at] = 0x7F
            c[x + 1].view(U8)[page, :, at] = 255
    query = randn(g, 2 * q, nq * hd)
    out = torch.full((2 * q, nq * hd), 7.5, dtype=BF16, device="cuda")
    scs().sc_paged_attn_decode_fp8(query.cuda(), out, *c, i32(table), i32(lens), q=q, max_seq_len=64)
    want, tol = ref(query, k, v, lens, q, hd ** -0.5)
    for r in range(2):
        rows = slice(r * q, r * q + q - 1)
        check_attn(out.cpu()[rows], want[rows], tol[rows])


def test_scales_over_their_range():
    """Keys of size 2^-120 and values of 2^100: the scales leave the products as powers
    of two, so that neither is lost."""
    hd, n = 128, 40
    print("[gpu] attn fp8 scales", flush=True)
    g = torch.Generator().manual_seed(5)
    c = caches_fp8("tokens", 3, 16, 1, hd)
    k, v = [], []
    for b in range(3):
        x = (torch.randn(16, 1, hd, generator=g) * 2.0 ** -120).to(BF16)
        y = (torch.randn(16, 1, hd, generator=g) * 2.0 ** 100).to(BF16)
        k.append(put(c[0], c[1], b, 0, x))
        v.append(put(c[2], c[3], b, 0, y))
    k, v = torch.cat(k)[:n], torch.cat(v)[:n]
    query = (torch.randn(1, 2 * hd, generator=g) * 2.0 ** 119).to(BF16)
    out = torch.empty(1, 2 * hd, dtype=BF16, device="cuda")
    scs().sc_paged_attn_decode_fp8(query.cuda(), out, *c, i32([[0, 1, 2]]), i32([n]), max_seq_len=48)
    want, tol = ref(query, [k], [v], [n], 1, hd ** -0.5)
    check_attn(out.cpu(), want, tol)


def test_written_read_and_attended():
    """Prompts written quantised, then steps of drafts, each attended to: as a plain form
    over what the cache reads back as."""
    nq, nkv, hd, block, q = 8, 2, 128, 16, 2
    print("[gpu] fp8 write, read, attend", flush=True)
    S = scs()
    g = torch.Generator().manual_seed(9)
    lens = [37, 1, 64, 130]
    B = len(lens)
    c = caches_fp8("joint", 40, block, nkv, hd)
    table = np.random.default_rng(1).permutation(40).reshape(4, 10)
    ang = torch.arange(200, dtype=F64)[:, None] * torch.rand(hd // 2, generator=g, dtype=F64)
    turns = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    done = [0] * B
    for step in range(3):
        new = lens if step == 0 else [q] * B
        pos = np.concatenate([np.arange(n) + d for n, d in zip(new, done)])
        req = np.repeat(np.arange(B), new)
        slots = table[req, pos // block] * block + pos % block
        rows = randn(g, len(pos), (nq + 2 * nkv) * hd).cuda()
        qo = torch.empty(len(pos), nq * hd, dtype=BF16, device="cuda")
        S.sc_qk_norm_rope_fp8(rows[:, :nq * hd], rows[:, nq * hd:(nq + nkv) * hd],
                              rows[:, (nq + nkv) * hd:], qo, None, None, None, turns, i64(pos),
                              i64(slots), *c, head_dim=hd)
        done = [d + n for d, n in zip(done, new)]
        if step == 0:
            continue
        out = torch.empty_like(qo)
        S.sc_paged_attn_decode_fp8(qo, out, *c, i32(table), i32(done), q=q, max_seq_len=150)
        starts = np.concatenate([[0], np.cumsum(done)])
        ko, vo = (torch.empty(int(starts[-1]), nkv * hd, dtype=BF16, device="cuda") for _ in range(2))
        S.sc_paged_cache_read_fp8(*c, ko, vo, i32(table), i32(starts))
        k, v = ([x.cpu().view(-1, nkv, hd)[starts[r]:starts[r + 1]] for r in range(B)] for x in (ko, vo))
        want, tol = ref(qo.cpu(), k, v, done, q, hd ** -0.5)
        check_attn(out.cpu(), want, tol)


def test_captured_write_and_attention():
    """A step captured into a graph and replayed with other inputs, lengths and slots
    gives the eager step's results; two graphs with workspaces of their own."""
    nq, nkv, hd, block, B = 8, 2, 128, 16, 3
    print("[gpu] fp8 graph", flush=True)
    S = scs()
    g = torch.Generator().manual_seed(4)
    c, table, _, _ = paged_fp8(g, [2000, 700, 90], nkv, hd, block, "tokens", np.random.default_rng(2))
    table = i32(np.where(table > 10 ** 8, 0, table))
    rows = torch.empty(B, (nq + 2 * nkv) * hd, dtype=BF16, device="cuda")
    slots, lens = torch.empty(B, dtype=torch.int64, device="cuda"), torch.ones(B, dtype=torch.int32, device="cuda")
    qo, out = (torch.empty(B, nq * hd, dtype=BF16, device="cuda") for _ in range(2))
    need = S.sc_paged_attn_fp8_workspace_bytes(B, max_seq_len=2000, num_q_heads=nq, num_kv_heads=nkv,
                                               head_dim=hd)
    room = torch.empty(need, dtype=U8, device="cuda")
    back = [torch.empty(64, nkv * hd, dtype=BF16, device="cuda") for _ in range(2)]
    starts = i32([0, 32, 64])

    def step(out, workspace, back):
        S.sc_qk_norm_rope_fp8(rows[:, :nq * hd], rows[:, nq * hd:(nq + nkv) * hd],
                              rows[:, (nq + nkv) * hd:], qo, None, None, None, None, None, slots, *c,
                              head_dim=hd)
        S.sc_paged_attn_decode_fp8(qo, out, *c, table, lens, max_seq_len=2000, workspace=workspace)
        S.sc_paged_cache_read_fp8(*c, *back, table, starts)

    def fill(i):
        rows.copy_(randn(torch.Generator().manual_seed(i), *rows.shape))
        n = np.array([2000 - i, 5 + i, 90 - 7 * i])
        t = table.cpu().numpy()
        lens.copy_(i32(n))
        slots.copy_(i64(t[np.arange(B), (n - 1) // block] * block + (n - 1) % block))
    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(out, room, back)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out, room, back)
    for i in range(1, 5):
        fill(i)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), [x.clone() for x in back]
        eager, eb = torch.empty_like(out), [torch.empty_like(x) for x in back]
        step(eager, None, eb)
        assert torch.equal(got[0], eager) and all(torch.equal(x, y) for x, y in zip(got[1], eb))
