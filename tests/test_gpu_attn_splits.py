"""Attention on the GPU over a split cache, where rows and splits are odd in
number, in a workspace of exactly the bytes that are asked for; and of requests
that are taken by falling length."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_attn import BF16, attn_ref, check_attn, i32, paged, randn, scs  # noqa: E402

pytestmark = pytest.mark.gpu

CASES = [  # nq, nkv, hd, q, lens
    (7, 1, 128, 1, [3500]),
    (3, 3, 64, 1, [2300, 1, 0, 1100, 513]),
    (1, 1, 256, 1, [1400]),
    (5, 1, 64, 3, [4607]),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}-{c[1]}-{c[2]}-q{c[3]}" for c in CASES])
def test_odd_parts(case):
    nq, nkv, hd, q, lens = case
    print(f"[gpu] attn odd parts {case}", flush=True)
    S = scs()
    g = torch.Generator().manual_seed(sum(lens))
    kc, vc, table, k, v = paged(g, lens, nkv, hd, 16, "tokens", np.random.default_rng(hd))
    B = len(lens)
    query = randn(g, B * q, nq * hd)
    out = torch.full((B * q, nq * hd), 7.5, dtype=BF16, device="cuda")
    need = S.sc_paged_attn_workspace_bytes(B, q=q, max_seq_len=max(lens), num_q_heads=nq,
                                           num_kv_heads=nkv, head_dim=hd)
    room = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    S.sc_paged_attn_decode(query.cuda(), out, kc, vc, i32(table), i32(lens), q=q,
                           max_seq_len=max(lens), workspace=room[:need])
    want, tol = attn_ref(query, k, v, lens, q, hd ** -0.5)
    check_attn(out.cpu(), want, tol)
    assert bool((room[need:] == 0xFF).all())


ORDERED = [  # nq, nkv, hd, q, requests, lengths; max_seq_len of 512 and more
    (8, 4, 64, 1, 400, "some"),
    (4, 4, 64, 1, 512, "equal"),
    (8, 4, 64, 1, 513, "some"),        # one more than are put in order
    (4, 2, 256, 1, 300, "one"),
    (16, 4, 128, 2, 70, "none"),
]


@pytest.mark.parametrize("top", [512, 700])
@pytest.mark.parametrize("case", ORDERED, ids=[f"{c[1]}x{c[2]}-{c[4]}-{c[5]}" for c in ORDERED])
def test_requests_in_order(case, top):
    """Each request has its rows, whatever the order in which they are taken."""
    nq, nkv, hd, q, B, kind = case
    print(f"[gpu] attn ordered {case} {top}", flush=True)
    g = torch.Generator().manual_seed(B)
    rng = np.random.default_rng(B)
    lens = {"some": rng.integers(0, 90, B), "equal": np.full(B, 33),
            "one": np.where(np.arange(B) == 250, 129, 1), "none": np.zeros(B, int)}[kind].tolist()
    kc, vc, table, k, v = paged(g, lens, nkv, hd, 16, "tokens", rng)
    wide = np.full((B, 44), 10 ** 9)                       # 704 tokens; not read behind the end
    wide[:, :table.shape[1]] = table
    query = randn(g, B * q, nq * hd)
    out = torch.full((B * q + 1, nq * hd), 7.5, dtype=BF16, device="cuda")
    scs().sc_paged_attn_decode(query.cuda(), out[:-1], kc, vc, i32(wide), i32(lens), q=q,
                               max_seq_len=top)
    want, tol = attn_ref(query, k, v, lens, q, hd ** -0.5)
    got = out.cpu()
    check_attn(got[:-1].view(B * q, nq, hd), want.view(B * q, nq, hd), tol.view(B * q, nq, hd))
    assert bool((got[-1] == 7.5).all())
