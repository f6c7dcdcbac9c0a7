"""Attention over shared prefixes: how far outputs are from 64-bit values, beyond their
own rounding to bf16, in every split and join of the parts."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests._fp8 import BF16, F64, U8, caches_fp8, put  # noqa: E402
from tests.test_gpu_attn import attn_ref, check_attn, i32, randn, scs  # noqa: E402
from tests.test_gpu_attn_prefix import shared  # noqa: E402


def check(got, want, tol, top):
    """Each value: attn_ref's tolerance, and for weights in two bf16 parts, off by 2^-15
    each, twice that (the mean is off by theirs and by their sum's) of the largest
    value. All of them: rounding (want + d) to bf16 leaves, in the mean square, what
    rounding `want` leaves, and d. The errors of the weights, and of fp32 scores, 2^-20 or
    less here, average as the values themselves do to outputs near zero: d is 2^-15 of
    the outputs at most, against 2^-9.2 for the rounding, under 2^-5 of it."""
    check_attn(got, want, tol + 2.0 ** -14 * top)
    best = float((want.to(BF16).to(F64) - want).norm())
    off = float((got.to(F64) - want).norm())
    assert off <= best * (1 + 2.0 ** -5), off / best


CASES = [  # nq, nkv, hd, block, q, requests, prefix, own tokens, layout
    (16, 4, 128, 16, 1, 70, 1500, 8, "tokens"),
    (8, 2, 64, 64, 3, 40, 900, 30, "joint"),
    (4, 1, 256, 16, 1, 33, 700, 50, "heads"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}-{c[1]}-{c[2]}-q{c[4]}-{c[5]}on{c[6]}" for c in CASES])
def test_weights(case, fp8):
    nq, nkv, hd, block, q, B, P, own, layout = case
    print(f"[gpu] prefix weights {case} {fp8}", flush=True)
    g = torch.Generator().manual_seed(B)
    rng = np.random.default_rng(B)
    c, table, lens, k, v = shared(g, [B], [P], rng.integers(q, own + 1, B), nkv, hd, block, layout, fp8, rng)
    query = randn(g, B * q, nq * hd)
    out = torch.empty(B * q, nq * hd, dtype=BF16, device="cuda")
    fn = scs().sc_paged_attn_prefix_fp8 if fp8 else scs().sc_paged_attn_prefix
    fn(query.cuda(), out, *c, i32(table), i32(lens), i32([0, B]), i32([P]), q=q, max_seq_len=max(lens),
       max_prefix_len=P)
    want, tol = attn_ref(query, k, v, lens, q, hd ** -0.5)
    check(out.cpu(), want, tol, max(float(x.abs().max()) for x in v))


@pytest.mark.gpu
def test_large_values_under_growing_scores():
    """A score that passes the first tile's by 2^7, over values near fp32's limit. Under
    weights of 2^-7 and one of 1 the values, 2^124 and every fourth 2^126, sum to less
    than 2^127; under weights that go on to 2^7 they would pass 2^128."""
    hd, P, B = 64, 320, 3
    print("[gpu] prefix large values", flush=True)
    k = torch.zeros(P + 16, 1, hd, dtype=BF16)
    k[P - 5, 0, 0] = 7.0
    v = torch.full((P + 16, 1, hd), 2.0 ** 124, dtype=BF16)
    v[::4] = 2.0 ** 126
    query = torch.zeros(B, hd, dtype=BF16)
    query[:, 0] = 1.0
    table = np.tile(np.arange(P // 16 + 1), (B, 1))
    out = torch.empty(B, hd, dtype=BF16, device="cuda")
    scs().sc_paged_attn_prefix(query.cuda(), out, k.cuda().view(-1, 16, 1, hd), v.cuda().view(-1, 16, 1, hd),
                               i32(table), i32([P + 1] * B), i32([0, B]), i32([P]), max_seq_len=P + 1,
                               max_prefix_len=P, scale=float(np.log(2.0)))
    s = query.to(F64) @ k[:P + 1, 0].to(F64).T * float(np.log(2.0))
    want = torch.softmax(s, -1) @ v[:P + 1, 0].to(F64)
    # the rounding, weights to 2^-15 twice, scores below 2^3 and sums to 2^-20
    tol = (2.0 ** -8 + 2.0 ** -13) * want.abs() + 2.0 ** -13 * 2.0 ** 126
    assert bool(((out.cpu().to(F64) - want).abs() <= tol).all())


@pytest.mark.gpu
def test_scales_over_their_range_in_a_prefix():
    """Keys of size 2^-120, some under the byte 0, and values of 2^122, one under the byte
    247. Codes enter the products as bf16, exactly but below 2^-126, where half a step is
    2^-134: a score is off by that times its query's sum."""
    hd, nq, P, B = 128, 2, 80, 3
    print("[gpu] prefix scales", flush=True)
    g = torch.Generator().manual_seed(5)
    blocks = P // 16 + 1
    c = caches_fp8("tokens", blocks, 16, 1, hd)
    k, v = [], []
    for b in range(blocks):
        x = (torch.randn(16, 1, hd, generator=g) * 2.0 ** -120).to(BF16)
        y = (torch.randn(16, 1, hd, generator=g) * 2.0 ** 122).to(BF16)
        if b == 2:
            y[7] = 1.875 * 2.0 ** 127
        k.append(put(c[0], c[1], b, 0, x))
        v.append(put(c[2], c[3], b, 0, y))
    assert int(c[3][2, 0, 7]) == 247 and int(c[1].view(U8).max()) == 1
    c[1].view(U8)[1, 0, :5] = 0
    k[1][:5] /= 2
    n = P + 1
    k, v = torch.cat(k)[:n], torch.cat(v)[:n]
    query = (torch.randn(B, nq * hd, generator=g) * 2.0 ** 119).to(BF16)
    out = torch.empty(B, nq * hd, dtype=BF16, device="cuda")
    table = np.tile(np.arange(blocks), (B, 1))
    scs().sc_paged_attn_prefix_fp8(query.cuda(), out, *c, i32(table), i32([n] * B), i32([0, B]), i32([P]),
                                   max_seq_len=n, max_prefix_len=P)
    want, tol = attn_ref(query, [k] * B, [v] * B, [n] * B, 1, hd ** -0.5)
    top = float(v.abs().max())
    off = 2.0 ** -134 * float(query.to(F64).abs().view(B, nq, hd).sum(-1).max()) * hd ** -0.5
    check_attn(out.cpu(), want, tol + (2.0 ** -14 + 2 * off) * top)
