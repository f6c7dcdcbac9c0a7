"""Attention over shared prefixes in every way that its work is split and joined: many
pages to a split, many parts to a row, joins of one and of four waves a row, long
requests beside the groups. That each case goes its way is checked without a GPU."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import stateful_causal_short_amd as scs_lib  # noqa: E402
from tests._fp8 import BF16  # noqa: E402
from tests.test_attn_fp8_host import prefix  # noqa: E402
from tests.test_attn_host import BIG, INVALID, ODD, UNSUPPORTED, attn_desc  # noqa: E402
from tests.test_gpu_attn import attn_ref, i32, randn, scs  # noqa: E402
from tests.test_gpu_attn_prefix import CASES as SMALL, shared  # noqa: E402
from tests.test_gpu_attn_prefix_weights import check  # noqa: E402


def parts(fp8, nq, nkv, hd, B, q, top, longest, groups):
    """Parts of a row that a call makes, from the least workspace that it takes: with more
    it goes on to refuse its queries' address."""
    d = attn_desc(num_q_heads=nq, num_kv_heads=nkv, head_dim=hd, q_row_stride=nq * hd, out_row_stride=nq * hd,
                  block_table_row_stride=1 << 20)
    status = lambda n: prefix(d, fp8, q=ODD, blocks=1 << 20, groups=groups, batch=B, n=q, top=top,
                              longest=longest, ws_bytes=4 * (-(-2 * n * B * q * nq // 4) * 4 + n * B * q * nq * hd))
    n = next(n for n in range(1, 200) if status(n) != INVALID)
    assert status(n) == UNSUPPORTED
    return n


CASES = [  # nq, nkv, hd, block, q, group sizes, prefixes, own tokens, layout; what a row's parts are
    (64, 4, 64, 16, 1, [256], [4611], (1, 8), "tokens", "long splits"),
    (128, 2, 128, 16, 1, [128], [4611], (1, 8), "heads", "long splits"),
    (64, 4, 64, 16, 1, [32], [300], (1, 2100), "joint", "one wave"),
    (64, 1, 256, 32, 1, [32], [150], (1, 2100), "tokens", "one wave"),
    (64, 2, 128, 64, 1, [20, 14], [1000, 333], (1, 1500), "tokens", "one wave"),
    (4, 1, 64, 16, 1, [2], [20011], (1, 50), "tokens", "past 64"),
    (8, 2, 128, 16, 3, [3], [20011], (3, 50), "joint", "past 64"),
    (2, 1, 256, 64, 1, [2], [20011], (1, 50), "tokens", "past 64"),
    (4, 1, 256, 16, 1, [3], [1500], (1, 1500), "heads", "four waves"),
    (4, 2, 64, 16, 1, [2, 1], [700, 100], (1, 1500), "tokens", "four waves"),
]
IDS = [f"{c[0]}-{c[1]}-{c[2]}-q{c[4]}-{c[5][0]}on{c[6][0]}" for c in CASES]


def sizes_of(case):
    nq, nkv, hd, block, q, sizes, prefixes, own, layout, way = case
    rng = np.random.default_rng(hd)
    mine = rng.integers(own[0], own[1] + 1, sum(sizes))
    mine[0] = own[1]
    return rng, mine, max(p + mine[np.repeat(np.arange(len(sizes)), sizes) == i].max()
                          for i, p in enumerate(prefixes))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_cases_go_their_way(case, fp8):
    """256 CUs, as without a device. Own parts: one for each 1,024 tokens that max_seq_len
    leaves behind the longest prefix, or more."""
    nq, nkv, hd, block, q, sizes, prefixes, own, layout, way = case
    _, _, top = sizes_of(case)
    n = parts(fp8, nq, nkv, hd, sum(sizes), q, top, max(prefixes), len(sizes))
    rows = sum(sizes) * q * nq
    if way == "long splits":                    # one own part: n - 1 of the prefix
        assert top - max(prefixes) < 900 and max(prefixes) / (n - 1) > 1024
    elif way == "past 64":
        assert n > 64 + 16 and rows < 2048
    else:                                       # more own parts than one, so that a launch joins
        assert top - max(prefixes) > 1040 and n >= 3
        assert (rows >= 2048) == (way == "one wave")


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_long_own_parts_are_split(fp8):
    """Few requests on a prefix so long that it has as many parts as there may be, 96: a
    request of no group, which may be as long, has parts of its own."""
    assert parts(fp8, 4, 1, 128, 2, 1, 1_000_050, 1_000_000, 1) >= 96 + 16


def run(fp8, nq, nkv, hd, block, q, sizes, prefixes, mine, layout, scale, rng, seed):
    """One call, checked by check()."""
    g = torch.Generator().manual_seed(seed)
    B = sum(sizes)
    c, table, lens, k, v = shared(g, sizes, prefixes, mine, nkv, hd, block, layout, fp8, rng)
    query = randn(g, B * q, nq * hd)
    out = torch.full((B * q + 1, nq * hd), 7.5, dtype=BF16, device="cuda")
    fn = scs().sc_paged_attn_prefix_fp8 if fp8 else scs().sc_paged_attn_prefix
    fn(query.cuda(), out, *c, i32(table), i32(lens), i32(np.concatenate([[0], np.cumsum(sizes)])),
       i32(prefixes), q=q, max_seq_len=max(lens), max_prefix_len=max(prefixes), scale=scale)
    want, tol = attn_ref(query, k, v, lens, q, hd ** -0.5 if scale is None else scale)
    got = out.cpu()
    check(got[:-1], want, tol, max(float(x.abs().max()) for x in v))
    assert bool((got[-1] == 7.5).all())
    return max(lens)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_paths(case, fp8):
    nq, nkv, hd, block, q, sizes, prefixes, own, layout, way = case
    print(f"[gpu] prefix path {case} {fp8}", flush=True)
    rng, mine, top = sizes_of(case)
    assert run(fp8, nq, nkv, hd, block, q, sizes, prefixes, mine, layout, None, rng, nq + sum(sizes)) == top


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("case", SMALL, ids=[f"{c[0]}-{c[1]}-{c[2]}-q{c[4]}-{c[5][0]}on{c[6][0]}" for c in SMALL])
def test_small_cases_by_mean_square(case, fp8):
    nq, nkv, hd, block, q, sizes, prefixes, own, layout, scale = case
    print(f"[gpu] prefix mean square {case} {fp8}", flush=True)
    rng = np.random.default_rng(hd + 1)
    run(fp8, nq, nkv, hd, block, q, sizes, prefixes, rng.integers(own[0], own[1] + 1, sum(sizes)), layout,
        scale, rng, nq)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_long_requests_beside_a_group(fp8):
    """Requests of no group, and one token short of its prefix, as long as the others."""
    nq, nkv, hd, q, P = 8, 2, 128, 1, 12000
    print(f"[gpu] prefix beside long requests {fp8}", flush=True)
    g = torch.Generator().manual_seed(4)
    sizes = [4, 1, 2]
    own = np.array([30, 1, 7, -1, -200, 5, 300])
    c, table, lens, k, v = shared(g, sizes, [P, P, 900], own, nkv, hd, 16, "tokens", fp8,
                                  np.random.default_rng(4))
    query = randn(g, 7, nq * hd)
    want, tol = attn_ref(query, k, v, lens, q, hd ** -0.5)
    fn = scs().sc_paged_attn_prefix_fp8 if fp8 else scs().sc_paged_attn_prefix
    top = max(float(x.abs().max()) for x in v)
    for starts in ([0, 4], [0, 4, 5], [2, 4]):
        groups = len(starts) - 1
        assert parts(fp8, nq, nkv, hd, 7, 1, max(lens), P, groups) > 17
        out = torch.empty(7, nq * hd, dtype=BF16, device="cuda")
        fn(query.cuda(), out, *c, i32(table), i32(lens), i32(starts), i32([P] * groups), q=q,
           max_seq_len=max(lens), max_prefix_len=P)
        check(out.cpu(), want, tol, top)


def test_a_lost_part_is_seen():
    """The check refuses outputs without one part of 16 of the prefix, without the own
    tokens, or with weights rounded to bf16."""
    g = torch.Generator().manual_seed(1)
    B, P, own, hd = 12, 5001, 9, 128
    kp, vp = randn(g, P, 1, hd), randn(g, P, 1, hd)
    k, v = ([torch.cat([x, randn(g, own, 1, hd)]) for _ in range(B)] for x in (kp, vp))
    query = randn(g, B, 4 * hd)
    want, tol = attn_ref(query, k, v, [P + own] * B, 1, hd ** -0.5)
    top = max(float(x.abs().max()) for x in v)
    check(want.to(BF16), want, tol, top)
    for lost in (slice(1248, 1561), slice(P, P + own)):
        rest = [t for t in range(P + own) if not lost.start <= t < lost.stop]
        wrong, _ = attn_ref(query, [x[rest] for x in k], [x[rest] for x in v], [len(rest)] * B, 1, hd ** -0.5)
        with pytest.raises(AssertionError):
            check(wrong.to(BF16), want, tol, top)
    qq = query.double().view(B, 4, hd)
    rough = []
    for r in range(B):
        p = torch.exp(qq[r] @ k[r][:, 0].double().T * hd ** -0.5)
        p = (p / p.amax(-1, keepdim=True)).to(BF16).double()
        rough.append((p @ v[r][:, 0].double() / p.sum(-1, keepdim=True)).flatten())
    with pytest.raises(AssertionError):
        check(torch.stack(rough).to(BF16), want, tol, top)
