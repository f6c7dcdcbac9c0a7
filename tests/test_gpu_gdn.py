"""The gated delta rule on the GPU against the token-by-token rule in 64 bits:
updates, speculative updates and varlen prefill, at odd sizes, with padding
slots, strided rows, strong decays and non-finite neighbours."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import _gdn as G  # noqa: E402

pytestmark = pytest.mark.gpu


def scs():
    import stateful_causal_short_amd as m
    return m


def gpu(c):
    return {k: v.cuda() if torch.is_tensor(v) else v for k, v in c.items()}


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def call_args(d, out, pool, rows=slice(None)):
    q, k, v = G.parts(d["mixed"], d)
    return (q[rows], k[rows], v[rows], d["a"][rows], d["b"][rows], d["A_log"], d["dt_bias"],
            out[rows], pool)


def sentinel(rows, width):
    return torch.full((rows, width), 7.5, dtype=torch.bfloat16, device="cuda")


UPDATES = [  # hk, hv, dk, dv, batch, q, gates, pad
    (1, 1, 128, 128, 1, 1, "bf16", 0),
    (2, 4, 128, 128, 3, 1, "f32", 8),
    (1, 2, 64, 64, 5, 3, "bf16", 24),
    (2, 2, 128, 48, 7, 2, "bf16", 8),
    (4, 8, 64, 16, 9, 5, "f32", 0),
    (16, 32, 128, 128, 17, 2, "bf16", 0),
    (1, 3, 128, 144, 40, 1, "bf16", 0),
    (8, 32, 64, 256, 33, 1, "f32", 0),
]


@pytest.mark.parametrize("hk,hv,dk,dv,batch,q,gates,pad", UPDATES)
def test_update(hk, hv, dk, dv, batch, q, gates, pad):
    print(f"[gpu] gdn update {hk}/{hv} x {dk}/{dv}, {batch} x {q}", flush=True)
    slots = batch + 4
    c = G.make(hk, hv, dk, dv, batch * q + 2, slots, gates=gates, seed=batch * 7 + q, pad=pad)
    d = gpu(c)
    rng = np.random.default_rng(batch)
    idx = rng.permutation(slots)[:batch]
    has = rng.integers(0, 2, batch)
    if batch > 2:
        idx[1], idx[2] = -1, slots                       # padding rows
    out, pool = sentinel(batch * q + 2, hv * dv), d["pool"].clone()
    m = slice(0, batch * q)
    scs().sc_gdn_update(*call_args(d, out, pool, m), i32(idx),
                        torch.tensor(has, dtype=torch.bool, device="cuda"), q=q)
    want_pool = c["pool"].to(G.F64)
    got, got_pool = out.cpu(), pool.cpu()
    for r in range(batch):
        live = 0 <= idx[r] < slots
        S = want_pool[idx[r]] if live and has[r] else torch.zeros(hv, dv, dk, dtype=G.F64)
        top = max(1.0, float(S.norm(dim=2).max()))
        o, st, bd = G.reference(c, range(r * q, r * q + q), S, dk ** -0.5)
        G.check_out(got[r * q:r * q + q].view(q, hv, dv), torch.stack(o), torch.stack(bd), q, dk,
                    f"request {r}")
        if live:
            top = max([top] + [float(s.norm(dim=2).max()) for s in st])
            G.check_state(got_pool[idx[r]], st[-1], q, dk, top, f"request {r}")
    rest = [s for s in range(slots) if s not in set(idx.tolist())]
    assert torch.equal(got_pool[rest], c["pool"][rest]), "a slot of no request changed"
    assert bool((got[batch * q:] == 7.5).all()), "a row behind the batch changed"


@pytest.mark.parametrize("hk,hv,dk,dv,batch,q", [(1, 2, 128, 64, 3, 4), (2, 4, 64, 48, 5, 2),
                                                 (16, 32, 128, 128, 9, 3), (1, 1, 64, 16, 2, 1)])
def test_update_spec_rolls_back(hk, hv, dk, dv, batch, q):
    """Two steps: the second starts from each request's last accepted draft."""
    print(f"[gpu] gdn spec {hk}/{hv} x {dk}/{dv}, {batch} x {q}", flush=True)
    slots = batch * q + 3
    c = G.make(hk, hv, dk, dv, batch * q, slots, seed=q + batch)
    d = gpu(c)
    rng = np.random.default_rng(q)
    table = rng.permutation(slots)[:batch * q].reshape(batch, q)
    wide = np.full((batch, q + 2), -9)
    wide[:, :q] = table                                  # rows of slots q + 2 apart
    pool = d["pool"].clone()
    accepted = [rng.integers(1, q + 1, batch), rng.integers(1, q + 1, batch)]
    accepted[1][0] = q + 5                               # clamped to q
    ref = {int(s): c["pool"][s].to(G.F64) for s in range(slots)}
    n = 0
    for acc in accepted:
        out = sentinel(batch * q, hv * dv)
        scs().sc_gdn_update_spec(*call_args(d, out, pool), i32(wide)[:, :q], i32(acc), q=q)
        n += q
        got, got_pool = out.cpu(), pool.cpu()
        for r in range(batch):
            S = ref[int(table[r, min(acc[r], q) - 1])]
            top = max(1.0, float(S.norm(dim=2).max()))
            o, st, bd = G.reference(c, range(r * q, r * q + q), S, dk ** -0.5)
            G.check_out(got[r * q:r * q + q].view(q, hv, dv), torch.stack(o), torch.stack(bd),
                        n, dk, f"request {r}")
            for t in range(q):
                top = max(top, float(st[t].norm(dim=2).max()))
                ref[int(table[r, t])] = st[t]
                G.check_state(got_pool[table[r, t]], st[t], n, dk, top, f"request {r} draft {t}")
    rest = [s for s in range(slots) if s not in set(table.reshape(-1).tolist())]
    assert torch.equal(pool.cpu()[rest], c["pool"][rest])


PREFILLS = [  # hk, hv, dk, dv, lengths, gates, strong, pad
    (1, 1, 128, 128, [1], "bf16", False, 0),
    (1, 2, 128, 64, [63, 0, 64, 65], "f32", False, 8),
    (2, 2, 64, 48, [0, 5, 128, 0], "bf16", False, 0),
    (1, 3, 64, 16, [200, 1, 17], "f32", True, 16),
    (2, 4, 128, 144, [130, 70], "bf16", True, 0),
    (4, 8, 128, 128, [3] * 70, "bf16", False, 0),
    (1, 1, 128, 32, [1000], "bf16", False, 0),
    (16, 32, 128, 128, [129, 40], "bf16", False, 0),
    (8, 16, 64, 80, [65, 2, 0, 190] + [7] * 20, "f32", True, 8),
    (2, 4, 128, 16, [1, 70, 64] * 24, "bf16", False, 0),
    (4, 12, 64, 128, [100, 33, 1], "bf16", True, 16),
    # many requests, taken by falling length, equal and empty ones among them;
    # then more than are put in order
    (1, 1, 64, 16, [3, 1, 0, 7, 1, 1, 70] * 40 + [200, 0], "bf16", False, 0),
    (1, 2, 64, 32, [1] * 65 + [129] + [2] * 9, "f32", False, 0),
    (1, 1, 64, 16, [1] * 1000 + [0, 90] + [2] * 38, "bf16", False, 0),
]


@pytest.mark.parametrize("hk,hv,dk,dv,lens,gates,strong,pad", PREFILLS)
@pytest.mark.parametrize("l2norm", [True, False])
def test_prefill(hk, hv, dk, dv, lens, gates, strong, pad, l2norm):
    print(f"[gpu] gdn prefill {hk}/{hv} x {dk}/{dv}, {lens[:6]}", flush=True)
    if not l2norm and (hv > 8 or len(lens) > 8):
        pytest.skip("one of the two is enough at this size")
    B, T = len(lens), sum(lens)
    slots = B + 3
    c = G.make(hk, hv, dk, dv, T + 3, slots, gates=gates, seed=T, pad=pad, strong=strong)
    if not l2norm:    # keys of the length that unit keys would have
        c["mixed"] = (c["mixed"].float() / dk ** 0.5).bfloat16()
    d = gpu(c)
    rng = np.random.default_rng(T)
    idx = rng.permutation(slots)[:B]
    has = rng.integers(0, 2, B)
    if B > 2:
        idx[2] = -1
    qsl = np.concatenate([[0], np.cumsum(lens)])
    out, pool = sentinel(T + 3, hv * dv), d["pool"].clone()
    scs().sc_gdn_prefill_varlen(*call_args(d, out, pool), i32(qsl), i32(idx),
                                torch.tensor(has, dtype=torch.uint8, device="cuda"),
                                scale=0.25, qk_l2norm=l2norm)
    got, got_pool = out.cpu(), pool.cpu()
    for r in range(B):
        live = 0 <= idx[r] < slots
        S = c["pool"][idx[r]].to(G.F64) if live and has[r] else torch.zeros(hv, dv, dk, dtype=G.F64)
        if lens[r] == 0:
            if live:
                assert torch.equal(got_pool[idx[r]], c["pool"][idx[r]])
            continue
        o, st, bd = G.reference(c, range(qsl[r], qsl[r + 1]), S, 0.25, l2norm)
        top = max(1.0, float(S.norm(dim=2).max()), max(float(s.norm(dim=2).max()) for s in st))
        # a row's terms reach as far as the largest state of the request
        bound = torch.stack(bd).clamp_min(1e-30)
        bound = torch.maximum(bound, bound.amax(dim=(0, 2), keepdim=True))
        G.check_out(got[qsl[r]:qsl[r + 1]].view(lens[r], hv, dv), torch.stack(o), bound,
                    lens[r], dk, f"request {r}")
        if live:
            G.check_state(got_pool[idx[r]], st[-1], lens[r], dk, top, f"request {r}")
    rest = [s for s in range(slots) if s not in set(idx.tolist())]
    assert torch.equal(got_pool[rest], c["pool"][rest]), "a slot of no request changed"
    assert bool((got[T:] == 7.5).all()), "a row behind the last request changed"


def test_prefill_in_pieces_and_decode_agree():
    """One prompt at once, in two calls, and token by token end in states and
    outputs within one error bound of each other; the same call twice is equal."""
    hk, hv, dk, dv, T = 2, 4, 128, 128, 150
    c = G.make(hk, hv, dk, dv, T, 4, seed=5)
    d = gpu(c)
    print(f"[gpu] gdn pieces {T}", flush=True)
    S = scs()
    runs = []
    for cuts in ([0, T], [0, T], [0, 71, T], None):
        out, pool = sentinel(T, hv * dv), d["pool"].clone()
        if cuts is None:
            for t in range(T):
                S.sc_gdn_update(*call_args(d, out, pool, slice(t, t + 1)), i32([2]),
                                torch.tensor([t > 0], device="cuda"))
        else:
            for i, (s, e) in enumerate(zip(cuts, cuts[1:])):
                S.sc_gdn_prefill_varlen(*call_args(d, out, pool, slice(s, e)), i32([0, e - s]),
                                        i32([2]), torch.tensor([i > 0], device="cuda"))
        runs.append((out.cpu(), pool.cpu()))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
    want, st, bd = G.reference(c, range(T), torch.zeros(hv, dv, dk, dtype=G.F64), dk ** -0.5)
    bound = torch.stack(bd)
    bound = torch.maximum(bound, bound.amax(dim=(0, 2), keepdim=True))
    top = max(float(s.norm(dim=2).max()) for s in st)
    for out, pool in runs:
        G.check_out(out.view(T, hv, dv), torch.stack(want), bound, T, dk)
        G.check_state(pool[2], st[-1], T, dk, max(top, 1.0))


def test_non_finite_input_stays_in_its_request():
    hk, hv, dk, dv = 1, 2, 128, 64
    lens = [70, 30, 66]
    qsl = [0, 70, 100, 166]
    c = G.make(hk, hv, dk, dv, 166, 5, seed=9)
    d = gpu(c)
    print("[gpu] gdn non-finite neighbours", flush=True)
    outs = []
    for poison in (False, True):
        if poison:
            d["mixed"][75] = float("nan")
            d["a"][80] = float("inf")
            d["b"][81] = float("nan")
            d["pool"][3] = float("nan")                  # no request's slot, and a fresh one's
            d["pool"][1] = float("inf")
        out, pool = sentinel(166, hv * dv), d["pool"].clone()
        scs().sc_gdn_prefill_varlen(*call_args(d, out, pool), i32(qsl), i32([0, 1, 2]),
                                    torch.tensor([1, 0, 1], dtype=torch.uint8, device="cuda"))
        outs.append((out.cpu(), pool.cpu()))
    for r in (0, 2):
        assert torch.equal(outs[0][0][qsl[r]:qsl[r + 1]], outs[1][0][qsl[r]:qsl[r + 1]])
        assert torch.equal(outs[0][1][r], outs[1][1][r])
    assert bool(outs[1][0][75:100].isnan().any(1).all())


def test_total_and_no_decay():
    """a = +inf forgets everything before the token, a = -inf nothing; both are
    exact limits of the rule, in either form."""
    hk, hv, dk, dv, T = 1, 1, 64, 16, 90
    c = G.make(hk, hv, dk, dv, T, 2, gates="f32", seed=3)
    c["a"][:] = float("-inf")
    c["a"][10] = c["a"][69] = float("inf")
    d = gpu(c)
    print("[gpu] gdn limits of the decay", flush=True)
    x = c["a"].clone()
    x[x == float("inf")] = 1e4                           # e^-1e4 is zero in 64 bits too
    ref = dict(c, a=x.clamp(-1e4, 1e4))
    want, st, bd = G.reference(ref, range(T), c["pool"][1].to(G.F64), dk ** -0.5)
    bound = torch.stack(bd)
    bound = torch.maximum(bound, bound.amax(dim=(0, 2), keepdim=True))
    top = max(float(s.norm(dim=2).max()) for s in st)
    for prefill in (True, False):
        out, pool = sentinel(T, hv * dv), d["pool"].clone()
        if prefill:
            scs().sc_gdn_prefill_varlen(*call_args(d, out, pool), i32([0, T]), i32([1]),
                                        torch.tensor([True], device="cuda"))
        else:
            scs().sc_gdn_update(*call_args(d, out, pool), i32([1]), q=T)
        G.check_out(out.cpu().view(T, hv, dv), torch.stack(want), bound, T, dk)
        G.check_state(pool.cpu()[1], st[-1], T, dk, max(1.0, top))


def test_slots_past_four_gigabytes():
    """State offsets beyond 2^32 bytes and 2^31 elements."""
    hk, hv, dk, dv = 16, 32, 128, 128
    c = G.make(hk, hv, dk, dv, 70, 1, seed=2)
    slots = 4200                                         # 2.2e9 elements, 8.8 GB
    d = gpu({k: v for k, v in c.items() if k != "pool"})
    print("[gpu] gdn far slots", flush=True)
    pool = torch.empty(slots, hv, dv, dk, device="cuda")
    pool[slots - 1] = c["pool"][0].cuda()
    pool[0] = 1.25
    out = sentinel(70, hv * dv)
    has = torch.tensor([1], dtype=torch.uint8, device="cuda")
    scs().sc_gdn_prefill_varlen(*call_args(d, out, pool, slice(0, 67)), i32([0, 67]),
                                i32([slots - 1]), has)
    scs().sc_gdn_update(*call_args(d, out, pool, slice(67, 70)), i32([slots - 1]), q=3)
    want, st, bd = G.reference(c, range(70), c["pool"][0].to(G.F64), dk ** -0.5)
    bound = torch.stack(bd)
    bound = torch.maximum(bound, bound.amax(dim=(0, 2), keepdim=True))
    top = max(float(s.norm(dim=2).max()) for s in st)
    G.check_out(out.cpu().view(70, hv, dv), torch.stack(want), bound, 70, dk)
    G.check_state(pool[slots - 1].cpu(), st[-1], 70, dk, top)
    assert bool((pool[0] == 1.25).all())


def test_graph_replays_match_eager():
    """Prefill, update and speculative update captured, with the workspace of
    the capture; eager calls run between the replays."""
    hk, hv, dk, dv = 2, 4, 128, 64
    c = G.make(hk, hv, dk, dv, 300, 12, seed=11)
    d = gpu(c)
    print("[gpu] gdn graph", flush=True)
    S = scs()
    qsl, pslots = i32([0, 100, 100, 290]), i32([0, 1, 2])
    has = torch.tensor([1, 0, 0], dtype=torch.uint8, device="cuda")
    uslots, table, acc = i32([3, 4]), i32([[5, 6], [7, 8]]), i32([1, 2])
    out, pool = sentinel(300, hv * dv), d["pool"].clone()

    def step():
        S.sc_gdn_prefill_varlen(*call_args(d, out, pool, slice(0, 290)), qsl, pslots, has)
        S.sc_gdn_update(*call_args(d, out, pool, slice(290, 294)), uslots, q=2)
        S.sc_gdn_update_spec(*call_args(d, out, pool, slice(294, 298)), table, acc, q=2)

    step()
    want = out.clone(), pool.clone()
    g = torch.cuda.CUDAGraph()
    pool.copy_(d["pool"])
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        out.fill_(7.5)
        other = d["pool"].clone()
        S.sc_gdn_update(*call_args(d, sentinel(300, hv * dv), other, slice(0, 4)), uslots, q=2)
        pool.copy_(d["pool"])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(pool, want[1])


def test_other_stream_and_given_workspace():
    hk, hv, dk, dv, T = 1, 2, 64, 64, 100
    c = G.make(hk, hv, dk, dv, T, 3, seed=13)
    d = gpu(c)
    print("[gpu] gdn stream", flush=True)
    S = scs()
    need = S.sc_gdn_workspace_bytes(T, 1, num_k_heads=hk, num_v_heads=hv, head_k_dim=dk,
                                    head_v_dim=dv)
    has = torch.tensor([1], dtype=torch.uint8, device="cuda")
    qsl, idx = i32([0, T]), i32([1])
    results = []
    side = torch.cuda.Stream()
    for stream, ws in ((None, None), (side, None),
                       (side, torch.empty(need, dtype=torch.uint8, device="cuda"))):
        out, pool = sentinel(T, hv * dv), d["pool"].clone()
        torch.cuda.synchronize()
        S.sc_gdn_prefill_varlen(*call_args(d, out, pool), qsl, idx, has, stream=stream,
                                workspace=ws)
        torch.cuda.synchronize()
        results.append((out, pool))
    for out, pool in results[1:]:
        assert torch.equal(out, results[0][0]) and torch.equal(pool, results[0][1])
    with pytest.raises(S.ScError):
        S.sc_gdn_prefill_varlen(*call_args(d, out, pool), qsl, idx, has,
                                workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))


def test_workspace_belongs_to_the_stream_of_the_call():
    """A block that the current stream has freed but still writes to is not the
    workspace of a call on another stream."""
    hk, hv, dk, dv, T = 2, 4, 128, 128, 640
    c = G.make(hk, hv, dk, dv, T, 3, seed=14)
    d = gpu(c)
    print("[gpu] gdn workspace of a side stream", flush=True)
    S = scs()
    need = S.sc_gdn_workspace_bytes(T, 1, num_k_heads=hk, num_v_heads=hv, head_k_dim=dk,
                                    head_v_dim=dv)
    has = torch.tensor([1], dtype=torch.uint8, device="cuda")
    qsl, idx = i32([0, T]), i32([1])
    want, pool = sentinel(T, hv * dv), d["pool"].clone()
    S.sc_gdn_prefill_varlen(*call_args(d, want, pool), qsl, idx, has)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    out, pool2 = sentinel(T, hv * dv), d["pool"].clone()
    torch.cuda.synchronize()
    for _ in range(4):
        junk = torch.empty(need, dtype=torch.uint8, device="cuda")
        for _ in range(200):
            junk.fill_(0xFF)
        del junk                                         # freed, and still being written
        pool2.copy_(d["pool"])
        side.wait_stream(torch.cuda.current_stream())
        junk = torch.empty(need, dtype=torch.uint8, device="cuda")
        for _ in range(200):
            junk.fill_(0xFF)
        del junk
        S.sc_gdn_prefill_varlen(*call_args(d, out, pool2), qsl, idx, has, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(pool2, pool)


def test_zero_rows_and_no_pool():
    """Empty batches are no-ops; without slots every request starts from zeros."""
    hk, hv, dk, dv = 1, 2, 64, 32
    c = G.make(hk, hv, dk, dv, 70, 1, seed=15)
    d = gpu(c)
    print("[gpu] gdn empty calls", flush=True)
    S = scs()
    none = torch.empty(0, hv, dv, dk, device="cuda")
    out = sentinel(70, hv * dv)
    has = torch.ones(1, dtype=torch.uint8, device="cuda")
    S.sc_gdn_update(*call_args(d, out, none, slice(0, 0)), i32([]))
    S.sc_gdn_prefill_varlen(*call_args(d, out, none, slice(0, 0)), i32([0]), i32([]), has[:0])
    S.sc_gdn_prefill_varlen(*call_args(d, out, none, slice(0, 0)), i32([0, 0]), i32([0]), has)
    torch.cuda.synchronize()
    assert bool((out == 7.5).all())
    zero = torch.zeros(hv, dv, dk, dtype=G.F64)
    S.sc_gdn_prefill_varlen(*call_args(d, out, none, slice(0, 68)), i32([0, 68]), i32([0]), has)
    S.sc_gdn_update(*call_args(d, out, none, slice(68, 70)), i32([0]), q=2)
    for rows in (range(68), range(68, 70)):
        want, _, bd = G.reference(c, rows, zero, dk ** -0.5)
        bound = torch.stack(bd)
        bound = torch.maximum(bound, bound.amax(dim=(0, 2), keepdim=True))
        G.check_out(out.cpu()[list(rows)].view(len(rows), hv, dv), torch.stack(want), bound,
                    len(rows), dk)


def test_empty_speculative_batch_and_slots_of_2d_columns():
    """A speculative call of no requests is a no-op; prefill and updates take
    their slots from column 0 of a 2-D array."""
    hk, hv, dk, dv = 1, 2, 64, 32
    c = G.make(hk, hv, dk, dv, 9, 6, seed=16)
    d = gpu(c)
    print("[gpu] gdn 2-D slots", flush=True)
    S = scs()
    out, pool = sentinel(9, hv * dv), d["pool"].clone()
    S.sc_gdn_update_spec(*call_args(d, out, pool, slice(0, 0)), i32([]).view(0, 3), i32([]), q=3)
    torch.cuda.synchronize()
    assert bool((out == 7.5).all()) and torch.equal(pool, d["pool"])
    wide = i32([[4, 0, 0], [1, 0, 0], [2, 0, 0]])
    has = torch.ones(3, dtype=torch.uint8, device="cuda")
    for slots in (wide, wide[:, 0].contiguous()):
        got, p = sentinel(9, hv * dv), d["pool"].clone()
        S.sc_gdn_prefill_varlen(*call_args(d, got, p, slice(0, 9)), i32([0, 4, 5, 9]), slots, has)
        again, p2 = sentinel(9, hv * dv), d["pool"].clone()
        S.sc_gdn_update(*call_args(d, again, p2, slice(0, 9)), slots, q=3)
        if slots is wide:
            kept = (got, p, again, p2)
    for x, y in zip(kept, (got, p, again, p2)):
        assert torch.equal(x, y)
    assert not torch.equal(kept[1], d["pool"]) and torch.equal(kept[1][[0, 3, 5]], d["pool"][[0, 3, 5]])


def test_conv_then_delta_rule():
    """The two steps of such a layer together: the mixed-qkv conv, then the
    delta rule on column blocks of its output, for a prefill that continues one
    request and a decode step after it; each against 64 bits on the conv's
    outputs."""
    S = scs()
    hk, hv, dk, dv = 2, 4, 64, 64
    kw, vw = hk * dk, hv * dv
    C, K, lens = 2 * kw + vw, 4, [90, 33]
    T, B = sum(lens), 2
    c = G.make(hk, hv, dk, dv, T + B, 6, seed=21)
    d = gpu(c)
    print("[gpu] conv -> gdn", flush=True)
    g = torch.Generator().manual_seed(4)
    x = torch.randn(T + B, C, generator=g).bfloat16().cuda()
    w = (torch.randn(C, K, generator=g) * 0.4).bfloat16().cuda()
    conv_pool = torch.zeros(6, C, K - 1, dtype=torch.bfloat16, device="cuda")
    mixed, out, pool = torch.empty_like(x), sentinel(T + B, vw), d["pool"].clone()
    d["mixed"] = mixed
    qsl, idx = i32([0, lens[0], T]), i32([4, 1])
    has = torch.tensor([1, 0], dtype=torch.uint8, device="cuda")
    S.sc_conv_prefill_varlen(x[:T], mixed[:T], w, None, conv_pool, qsl, idx, has)
    S.sc_gdn_prefill_varlen(*call_args(d, out, pool, slice(0, T)), qsl, idx, has)
    S.sc_conv_update(x[T:], mixed[T:], w, None, conv_pool, idx)
    S.sc_gdn_update(*call_args(d, out, pool, slice(T, T + B)), idx)
    c["mixed"] = mixed.cpu()
    got, got_pool = out.cpu(), pool.cpu()
    starts = [0, lens[0]]
    for r, slot in enumerate((4, 1)):
        rows = list(range(starts[r], starts[r] + lens[r])) + [T + r]
        S0 = c["pool"][slot].to(G.F64) if r == 0 else torch.zeros(hv, dv, dk, dtype=G.F64)
        want, st, bd = G.reference(c, rows, S0, dk ** -0.5)
        bound = torch.stack(bd)
        bound = torch.maximum(bound, bound.amax(dim=(0, 2), keepdim=True))
        top = max(float(S0.norm(dim=2).max()), max(float(s.norm(dim=2).max()) for s in st))
        G.check_out(got[rows].view(len(rows), hv, dv), torch.stack(want), bound, len(rows), dk)
        G.check_state(got_pool[slot], st[-1], len(rows), dk, max(1.0, top))
