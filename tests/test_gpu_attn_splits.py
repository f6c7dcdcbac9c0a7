"""Attention over a split cache on the GPU, where rows and splits are odd in
number, in a workspace of exactly the bytes that are asked for."""
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
