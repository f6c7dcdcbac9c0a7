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
from tests.test_gpu_attn_prefix import shared  # noqa: E402
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


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_long_own_parts_are_split(fp8):
    """Few requests on a prefix so long that it has as many parts as there may be, 96: a
    request of no group, which may be as long, has parts of its own."""
    assert parts(fp8, 4, 1, 128, 2, 1, 1_000_050, 1_000_000, 1) >= 96 + 16


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
