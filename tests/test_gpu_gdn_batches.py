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


# ---------------------------------------------------------------------------
# the scan for many (request, head, 16 columns): 3 x 32 x 8 of them and more
# ---------------------------------------------------------------------------
MANY = (16, 32, 128, 128)


def check_requests(c, got, got_pool, qsl, slots, has, l2norm=True):
    """Outputs and final states against the rule in 64 bits."""
    hv, dv, dk = c["pool"].shape[1:]
    for r, slot in enumerate(slots):
        rows = range(int(qsl[r]), int(qsl[r + 1]))
        S = c["pool"][slot].to(G.F64) if has[r] else torch.zeros(hv, dv, dk, dtype=G.F64)
        want, st, bd = G.reference(c, rows, S, dk ** -0.5, l2norm)
        bound = torch.stack(bd)
        bound = torch.maximum(bound, bound.amax(dim=(0, 2), keepdim=True))
        top = max(1.0, float(S.norm(dim=2).max()), max(float(s.norm(dim=2).max()) for s in st))
        n = len(rows)
        G.check_out(got[list(rows)].view(n, hv, dv), torch.stack(want), bound, n, dk, f"request {r}")
        G.check_state(got_pool[slot], st[-1], n, dk, top, f"request {r}")


def test_many_without_unit_lengths():
    hk, hv, dk, dv = MANY
    lens, slots, has = [70, 129, 33], [3, 0, 2], [1, 0, 1]
    qsl = np.concatenate([[0], np.cumsum(lens)])
    c = G.make(hk, hv, dk, dv, qsl[-1], 4, seed=31)
    c["mixed"] = (c["mixed"].float() / dk ** 0.5).bfloat16()      # keys about as long as unit keys
    d = gpu(c)
    print("[gpu] gdn many heads, raw lengths", flush=True)
    out, pool = sentinel(int(qsl[-1]), hv * dv), d["pool"].clone()
    scs().sc_gdn_prefill_varlen(*call_args(d, out, pool), i32(qsl), i32(slots),
                                torch.tensor(has, dtype=torch.uint8, device="cuda"),
                                qk_l2norm=False)
    check_requests(c, out.cpu(), pool.cpu(), qsl, slots, has, False)
    assert torch.equal(pool[1].cpu(), c["pool"][1])


def test_many_with_total_and_no_decay():
    """a = +inf forgets everything before the token, a = -inf nothing."""
    hk, hv, dk, dv, T = 2, 32, 64, 144, 90
    c = G.make(hk, hv, dk, dv, T, 2, gates="f32", seed=32)
    c["a"][:] = float("-inf")
    c["a"][10] = c["a"][69] = float("inf")
    d = gpu(c)
    print("[gpu] gdn many heads, limits of the decay", flush=True)
    out, pool = sentinel(T, hv * dv), d["pool"].clone()
    scs().sc_gdn_prefill_varlen(*call_args(d, out, pool), i32([0, T]), i32([1]),
                                torch.tensor([True], device="cuda"))
    c["a"] = c["a"].clamp(-1e4, 1e4)                              # e^-1e4 is zero in 64 bits too
    check_requests(c, out.cpu(), pool.cpu(), [0, T], [1], [1])


def test_many_again_and_in_a_used_workspace():
    """The same bits from a second call, and whatever the workspace held: bytes
    of 0xFF, or the matrices and the order of another batch."""
    hk, hv, dk, dv = MANY
    c = G.make(hk, hv, dk, dv, 400, 5, seed=33)
    d = gpu(c)
    print("[gpu] gdn many heads, used workspaces", flush=True)
    S = scs()
    need = S.sc_gdn_workspace_bytes(400, 4, num_k_heads=hk, num_v_heads=hv, head_k_dim=dk,
                                    head_v_dim=dv)
    used = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    idx = i32([4, 2, 0, 1])
    has = torch.tensor([1, 0, 1, 1], dtype=torch.uint8, device="cuda")
    batches = [i32([0, 20, 149, 333, 400]), i32([0, 201, 202, 202, 400])]
    want = {}
    for ws in (None, None, used, used, used):
        for i, qsl in enumerate(batches):
            out, pool = sentinel(400, hv * dv), d["pool"].clone()
            S.sc_gdn_prefill_varlen(*call_args(d, out, pool), qsl, idx, has, workspace=ws)
            if i not in want:
                want[i] = out, pool
                host = qsl.tolist()
                if i == 0:
                    check_requests(c, out.cpu(), pool.cpu(), host, idx.tolist(), has.tolist())
            assert torch.equal(out, want[i][0]) and torch.equal(pool, want[i][1])


def test_many_in_a_graph_with_other_lengths():
    """A captured call follows the lengths of the replay, and with them the
    order in which requests are taken; eager calls run in between."""
    hk, hv, dk, dv = MANY
    c = G.make(hk, hv, dk, dv, 300, 6, seed=34)
    d = gpu(c)
    print("[gpu] gdn many heads, graph", flush=True)
    S = scs()
    qsl, idx = i32([0, 100, 200, 290, 300]), i32([5, 3, 1, 0])
    has = torch.tensor([1, 0, 1, 0], dtype=torch.uint8, device="cuda")
    out, pool = sentinel(300, hv * dv), d["pool"].clone()

    def call(o, p):
        S.sc_gdn_prefill_varlen(*call_args(d, o, p), qsl, idx, has)

    call(out, pool)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out, pool)
    for lens in ([100, 100, 90, 10], [1, 0, 298, 1], [64, 128, 0, 108], [10, 20, 30, 240]):
        qsl.copy_(i32(np.concatenate([[0], np.cumsum(lens)])))
        eager, eager_pool = sentinel(300, hv * dv), d["pool"].clone()
        call(eager, eager_pool)
        out.fill_(7.5)
        pool.copy_(d["pool"])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(pool, eager_pool), lens


def test_many_on_a_side_stream():
    """The workspace of a call on another stream is that stream's, not a block
    that the current one still writes."""
    hk, hv, dk, dv, T = (*MANY, 200)
    c = G.make(hk, hv, dk, dv, T, 3, seed=35)
    d = gpu(c)
    print("[gpu] gdn many heads, side stream", flush=True)
    S = scs()
    need = S.sc_gdn_workspace_bytes(T, 3, num_k_heads=hk, num_v_heads=hv, head_k_dim=dk,
                                    head_v_dim=dv)
    has = torch.ones(3, dtype=torch.uint8, device="cuda")
    qsl, idx = i32([0, 30, 130, T]), i32([1, 0, 2])
    want, want_pool = sentinel(T, hv * dv), d["pool"].clone()
    S.sc_gdn_prefill_varlen(*call_args(d, want, want_pool), qsl, idx, has)
    side = torch.cuda.Stream()
    out, pool = sentinel(T, hv * dv), d["pool"].clone()
    torch.cuda.synchronize()
    for _ in range(3):
        pool.copy_(d["pool"])
        side.wait_stream(torch.cuda.current_stream())
        junk = torch.empty(need, dtype=torch.uint8, device="cuda")
        for _ in range(100):
            junk.fill_(0xFF)
        del junk                                          # freed, and still being written
        S.sc_gdn_prefill_varlen(*call_args(d, out, pool), qsl, idx, has, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(pool, want_pool)


def test_many_slots_past_four_gigabytes():
    """State offsets beyond 2^32 bytes and 2^31 elements."""
    hk, hv, dk, dv = MANY
    lens, far = [66, 5, 40], 4199                         # slot 4,199: 8.8 GB in
    qsl = np.concatenate([[0], np.cumsum(lens)])
    c = G.make(hk, hv, dk, dv, qsl[-1], 3, seed=36)
    d = gpu({k: v for k, v in c.items() if k != "pool"})
    print("[gpu] gdn many heads, far slots", flush=True)
    pool = torch.empty(far + 1, hv, dv, dk, device="cuda")
    slots = [far, 2, far - 50]
    pool[slots] = c["pool"].cuda()
    pool[far - 1] = 1.25
    out = sentinel(int(qsl[-1]), hv * dv)
    scs().sc_gdn_prefill_varlen(*call_args(d, out, pool), i32(qsl), i32(slots),
                                torch.ones(3, dtype=torch.uint8, device="cuda"))
    check_requests(c, out.cpu(), pool[slots].cpu(), qsl, [0, 1, 2], [1, 1, 1])
    assert bool((pool[far - 1] == 1.25).all())
