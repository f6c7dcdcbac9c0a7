"""Refusals of the gated delta rule calls, without a GPU: the C entries return
their status before any launch (the fake pointers are never read), and the
binding raises on tensors that do not fit each other."""
import ctypes

import pytest

import stateful_causal_short_amd as scs

OK, NULL, INVALID, DTYPE, UNSUPPORTED = 0, -1, -2, -3, -5
P, P2, ODD = (ctypes.c_void_p(x) for x in (0x10000, 0x20000, 0x10004))
BIG = 1 << 40


def desc(**kw):
    d = dict(num_k_heads=2, num_v_heads=4, head_k_dim=128, head_v_dim=64, dtype=1, gate_dtype=1,
             qk_l2norm=1, scale=1.0, q_row_stride=256, k_row_stride=256, v_row_stride=256,
             a_row_stride=4, b_row_stride=4, out_row_stride=256, state_indices_stride=1)
    d.update(kw)
    return scs.sc_gdn_desc(**d)


def prefill(d, *, q=P, k=P, v=P, a=P, A=P, out=P2, pool=P, slots=4, qsl=P, idx=P, has=P, batch=2,
            T=10, ws=P, ws_bytes=BIG):
    return scs.lib().sc_gdn_prefill_varlen(None if d is None else ctypes.byref(d), q, k, v, a, a,
                                           A, A, out, pool, slots, qsl, idx, has, batch, T, ws,
                                           ws_bytes, None)


def update(d, *, q=P, k=P, v=P, out=P2, pool=P, slots=4, idx=P, batch=2, n=1):
    return scs.lib().sc_gdn_update(None if d is None else ctypes.byref(d), q, k, v, P, P, P, P,
                                   out, pool, slots, idx, None, batch, n, None)


def spec(d, *, pool=P, slots=4, idx=P, acc=P, batch=2, n=1, out=P2):
    return scs.lib().sc_gdn_update_spec(None if d is None else ctypes.byref(d), P, P, P, P, P, P,
                                        P, out, pool, slots, idx, acc, batch, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=0), DTYPE), (dict(dtype=9), DTYPE), (dict(gate_dtype=5), DTYPE),
    (dict(num_k_heads=0), INVALID), (dict(num_v_heads=0), INVALID),
    (dict(num_v_heads=5), INVALID), (dict(head_k_dim=0), INVALID),
    (dict(head_v_dim=0), INVALID), (dict(qk_l2norm=2), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(q_row_stride=255), INVALID), (dict(k_row_stride=8), INVALID),
    (dict(v_row_stride=255), INVALID), (dict(out_row_stride=255), INVALID),
    (dict(a_row_stride=3), INVALID), (dict(b_row_stride=3), INVALID),
    (dict(state_indices_stride=0), INVALID),
    (dict(head_k_dim=96), UNSUPPORTED), (dict(head_v_dim=24), UNSUPPORTED),
    (dict(q_row_stride=260), UNSUPPORTED), (dict(k_row_stride=257), UNSUPPORTED),
])
def test_descriptor_refusals(kw, status):
    d = desc(**kw)
    assert prefill(d) == status
    assert update(d) == status
    assert spec(d) == status
    n = ctypes.c_int64(0)
    assert scs.lib().sc_gdn_workspace_bytes(ctypes.byref(d), 2, 10, ctypes.byref(n)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), INVALID), (dict(T=-1), INVALID), (dict(slots=-1), INVALID),
    (dict(ws_bytes=-1), INVALID), (dict(ws_bytes=100), INVALID), (dict(T=1 << 31), UNSUPPORTED),
    (dict(q=None), NULL), (dict(a=None), NULL), (dict(A=None), NULL), (dict(out=None), NULL),
    (dict(pool=None), NULL), (dict(qsl=None), NULL), (dict(idx=None), NULL),
    (dict(has=None), NULL), (dict(ws=None), NULL), (dict(out=P), INVALID),
    (dict(q=ODD), UNSUPPORTED), (dict(k=ODD), UNSUPPORTED), (dict(pool=ODD), UNSUPPORTED),
    (dict(ws=ODD), INVALID),
    (dict(batch=0, q=None, out=None, ws=None), OK), (dict(T=0, q=None, ws=None), OK),
])
def test_prefill_refusals(kw, status):
    assert prefill(desc(), **kw) == status


def test_update_refusals():
    assert update(None) == NULL and spec(None) == NULL and prefill(None) == NULL
    assert update(desc(), n=-1) == INVALID and update(desc(), batch=-1) == INVALID
    assert update(desc(), batch=1 << 20, n=1 << 20) == UNSUPPORTED
    assert update(desc(), n=0, q=None) == OK and update(desc(), batch=0, q=None) == OK
    assert update(desc(), q=None) == NULL and update(desc(), out=P) == INVALID
    assert spec(desc(), n=2) == INVALID                     # rows of one slot, two drafts
    assert spec(desc(state_indices_stride=2), n=2, acc=None) == NULL
    assert spec(desc(state_indices_stride=2), n=2, batch=0, acc=None) == OK


def test_workspace_bytes():
    need = lambda T, B: scs.sc_gdn_workspace_bytes(T, B, num_k_heads=2, num_v_heads=4,
                                                   head_k_dim=128, head_v_dim=64)
    assert need(0, 3) == 0 and need(10, 0) == 0
    assert need(64, 1) > need(63, 1) > 0
    assert need(1 << 20, 7) > need(1 << 19, 7)
    assert scs.lib().sc_gdn_workspace_bytes(None, 1, 1, None) == NULL
    d = desc()
    assert prefill(d, batch=2, T=10, ws_bytes=need(10, 2) - 1) == INVALID


def tensors():
    torch = pytest.importorskip("torch")
    bf = torch.bfloat16
    t = dict(query=torch.zeros(6, 256, dtype=bf), key=torch.zeros(6, 256, dtype=bf),
             value=torch.zeros(6, 256, dtype=bf), a=torch.zeros(6, 4, dtype=bf),
             b=torch.zeros(6, 4, dtype=bf), A_log=torch.zeros(4), dt_bias=torch.zeros(4),
             out=torch.zeros(6, 256, dtype=bf), state_pool=torch.zeros(5, 4, 64, 128),
             state_indices=torch.zeros(6, dtype=torch.int32))
    return torch, t


@pytest.mark.parametrize("change", [
    "pool_dtype", "pool_dims", "key_width", "value_width", "gate_width", "gate_types",
    "short_key", "short_out", "A_dtype", "A_len", "idx_dtype", "out_dtype", "few_slots", "q"])
def test_binding_refuses(change):
    torch, t = tensors()
    q = 1
    if change == "pool_dtype":
        t["state_pool"] = t["state_pool"].bfloat16()
    elif change == "pool_dims":
        t["state_pool"] = t["state_pool"][0]
    elif change == "key_width":
        t["key"] = t["key"][:, :128]
    elif change == "value_width":
        t["value"] = t["value"][:, :128]
    elif change == "gate_width":
        t["a"] = t["a"][:, :3]
    elif change == "gate_types":
        t["b"] = t["b"].float()
    elif change == "short_key":
        t["key"] = t["key"][:5]
    elif change == "short_out":
        t["out"] = t["out"][:5]
    elif change == "A_dtype":
        t["A_log"] = t["A_log"].bfloat16()
    elif change == "A_len":
        t["dt_bias"] = t["dt_bias"][:3]
    elif change == "idx_dtype":
        t["state_indices"] = t["state_indices"].long()
    elif change == "out_dtype":
        t["out"] = t["out"].float()
    elif change == "few_slots":
        t["state_indices"] = t["state_indices"][:5]
    else:
        q = 4
    with pytest.raises(ValueError):
        scs.sc_gdn_update(*t.values(), q=q)


def test_binding_refuses_host_tensors_and_short_slot_rows():
    torch, t = tensors()
    with pytest.raises(ValueError):
        scs.sc_gdn_update(*t.values())                      # all fits, but not on a GPU
    acc = torch.ones(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        scs.sc_gdn_update_spec(*t.values(), acc, q=2)       # 1-D slots
    t["state_indices"] = torch.zeros(3, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        scs.sc_gdn_update_spec(*t.values(), acc, q=2)       # one slot for two drafts
    t["state_indices"] = torch.zeros(3, 4, dtype=torch.int32)[:, ::2]
    with pytest.raises(ValueError):
        scs.sc_gdn_update_spec(*t.values(), acc, q=2)       # slots not adjacent


def test_binding_takes_empty_speculative_batches():
    """No requests: the slots are (0, q), whatever their strides; the only thing
    wrong with this call is where its tensors are."""
    torch, t = tensors()
    for name in ("query", "key", "value", "a", "b", "out"):
        t[name] = t[name][:0]
    t["state_indices"] = torch.zeros(0, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="on the GPU"):
        scs.sc_gdn_update_spec(*t.values(), torch.zeros(0, dtype=torch.int32), q=2)


def test_sizes_that_cannot_be_launched_are_refused_before_a_launch():
    """More workgroups than a grid holds, in the first launch or only in the
    second; the bytes of such a workspace may not fit 64 bits either."""
    n = ctypes.c_int64(-7)
    many = desc(num_k_heads=1, num_v_heads=1 << 19, head_v_dim=16, v_row_stride=1 << 23,
                out_row_stride=1 << 23, a_row_stride=1 << 19, b_row_stride=1 << 19)
    assert scs.lib().sc_gdn_workspace_bytes(ctypes.byref(many), (1 << 31) - 1, (1 << 31) - 1,
                                            ctypes.byref(n)) == UNSUPPORTED
    wide = desc(num_k_heads=1, num_v_heads=1, head_v_dim=1 << 22, v_row_stride=1 << 22,
                out_row_stride=1 << 22)
    assert scs.lib().sc_gdn_workspace_bytes(ctypes.byref(wide), 1 << 15, 1,
                                            ctypes.byref(n)) == UNSUPPORTED
    assert prefill(wide, batch=1 << 15, T=1) == UNSUPPORTED
    assert n.value == -7


def test_empty_calls_need_no_workspace_whatever_their_other_size():
    n = ctypes.c_int64(-7)
    for batch, tokens in ((1 << 30, 0), (0, 1 << 40)):
        assert scs.lib().sc_gdn_workspace_bytes(ctypes.byref(desc()), batch, tokens,
                                                ctypes.byref(n)) == OK
        assert n.value == 0
        assert prefill(desc(), batch=batch, T=tokens, q=None, ws=None) == OK
        n.value = -7
