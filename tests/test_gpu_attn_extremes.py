"""Attention on the GPU at the ends of the scores' range."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_attn import BF16, F64, i32, randn, scs  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 20, 1100])
def test_lowest_scores_still_count(n):
    """Every score is -2.2e38 (-3.17e38 in base 2): the weights are equal and
    the row is the values' mean, not a row that sees nothing. One key of score
    0 more takes it all.

    Equal scores have weights of exactly 1, so before the bf16 rounding (half a
    step, 2^-8 of the value) there are n additions and a product by a rounded
    1/n: (n + 2) 2^-24 of the largest value."""
    print(f"[gpu] attn lowest scores {n}", flush=True)
    hd, pages = 64, -(-(n + 1) // 16)
    g = torch.Generator().manual_seed(n)
    k = torch.zeros(pages * 16, hd, dtype=BF16)
    k[:n, 0] = -2.0 ** 63
    v = randn(g, pages * 16, hd)
    query = torch.zeros(1, hd, dtype=BF16)
    query[0, 0] = 2.0 ** 64
    shape = (pages, 16, 1, hd)
    for length in (n, n + 1):
        out = torch.full((1, hd), 7.5, dtype=BF16, device="cuda")
        scs().sc_paged_attn_decode(query.cuda(), out, k.cuda().view(shape), v.cuda().view(shape),
                                   i32([list(range(pages))]), i32([length]), max_seq_len=length,
                                   scale=1.29)
        want = (v[:n].to(F64).mean(0) if length == n else v[n].to(F64))
        tol = 2.0 ** -8 * want.abs() + (n + 2) * 2.0 ** -24 * float(v.float().abs().max())
        assert bool(((out.cpu()[0].to(F64) - want).abs() <= tol).all())
