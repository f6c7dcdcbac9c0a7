"""The gated delta rule's varlen prefill on the GPU as a batch: what one request
holds stays out of the others', in the scan for few (request, head, 16 columns)
and in the scan for many."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import _gdn as G  # noqa: E402
from tests.test_gpu_gdn import call_args, gpu, i32, scs, sentinel  # noqa: E402

pytestmark = pytest.mark.gpu

# hk, hv, dk, dv: seven requests of them are 28 to 112 (request, head, 16 columns),
# at most one to a CU, or 896 and 1,792
SHAPES = [(1, 2, 128, 64), (2, 4, 64, 64), (1, 1, 128, 64), (16, 32, 128, 128), (8, 32, 64, 64)]


@pytest.mark.parametrize("hk,hv,dk,dv", SHAPES)
def test_rows_behind_a_request_are_not_read(hk, hv, dk, dv):
    """Requests that end 6, 40, 33 and 17 rows into a chunk, each with a request
    of NaN behind it, from its first row on; the last with rows of no request."""
    lens = [70, 30, 104, 5, 97, 50, 17]
    qsl = np.concatenate([[0], np.cumsum(lens)])
    T, pad = int(qsl[-1]), 70
    c = G.make(hk, hv, dk, dv, T + pad, 9, seed=hv + dk)
    d = gpu(c)
    print(f"[gpu] gdn rows behind a request, {hk}/{hv} x {dk}/{dv}", flush=True)
    has = torch.tensor([1, 0, 0, 1, 1, 0, 1], dtype=torch.uint8, device="cuda")
    runs = []
    for poison in (False, True):
        if poison:
            for r in (1, 3, 5):
                for name in ("mixed", "a", "b"):
                    d[name][qsl[r]:qsl[r + 1]] = float("nan")
            for name in ("mixed", "a", "b"):
                d[name][T:] = float("nan")
        out, pool = sentinel(T + pad, hv * dv), d["pool"].clone()
        scs().sc_gdn_prefill_varlen(*call_args(d, out, pool, slice(0, T)), i32(qsl),
                                    i32([4, 8, 0, 3, 7, 1, 5]), has)
        runs.append((out.cpu(), pool.cpu()))
    (clean, clean_pool), (got, got_pool) = runs
    for r, slot in ((0, 4), (2, 0), (4, 7), (6, 5)):
        rows = slice(qsl[r], qsl[r + 1])
        assert bool(clean[rows].isfinite().all())
        assert torch.equal(clean[rows], got[rows]), f"request {r}"
        assert torch.equal(clean_pool[slot], got_pool[slot]), f"state of request {r}"
    assert bool((got[T:] == 7.5).all())
    assert torch.equal(got_pool[[2, 6]], c["pool"][[2, 6]])
    assert bool(got[qsl[1]:qsl[2]].isnan().all())
