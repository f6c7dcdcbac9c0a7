"""Attention over a quantised cache: the weights have all of fp32's bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests._fp8 import BF16, F64, caches_fp8, put  # noqa: E402
from tests.test_gpu_attn import i32, scs  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_weights_that_cancel(hd):
    """Three tokens: one of score 0 and value 0, and two of values 1 and -1 whose scores,
    in [-2, 0], differ by 2^-12 of themselves, so that their weights cancel to some 2^-13.

    Scores are sums of two exact products: no rounding but their factor's, the difference
    from the maximum's and exp2's, 2^-24 of 2 twice and 2^-23, times ln 2: below 2^-21.5
    of a weight; two weights of half at most, the sums and the quotient: 2^-20."""
    print(f"[gpu] attn fp8 cancelling weights {hd}", flush=True)
    B, nq = 80, 16
    c = caches_fp8("tokens", 1, 16, 1, hd)
    k = torch.zeros(3, 1, hd, dtype=BF16)
    k[1:, 0, 0] = 1.0
    k[2, 0, 1] = 2.0 ** -12
    v = torch.zeros(3, 1, hd, dtype=BF16)
    v[1], v[2] = 1.0, -1.0
    keys, values = put(c[0], c[1], 0, 0, k), put(c[2], c[3], 0, 0, v)
    g = torch.Generator().manual_seed(hd)
    query = torch.zeros(B, nq, hd, dtype=BF16)
    query[..., 0] = query[..., 1] = -2 * torch.rand(B, nq, generator=g)
    query = query.to(BF16)
    out = torch.empty(B, nq * hd, dtype=BF16, device="cuda")
    scs().sc_paged_attn_decode_fp8(query.flatten(1).cuda(), out, *c, i32(np.zeros((B, 1))), i32([3] * B),
                                   max_seq_len=3, scale=1.0)
    want = torch.softmax(query.to(F64) @ keys[:, 0].T, -1) @ values[:, 0]
    assert float(want.abs().max()) < 2.0 ** -11
    off = (out.cpu().view(B, nq, hd).to(F64) - want).abs()
    assert bool((off <= 2.0 ** -8 * want.abs() + 2.0 ** -20).all()), float(off.max())
