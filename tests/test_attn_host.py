"""Refusals of the head norm and paged attention calls, without a GPU: the C
entries return their status before any launch (the fake pointers are never
read), and the binding raises on tensors that do not fit each other."""
import ctypes

import pytest

import stateful_causal_short_amd as scs

OK, NULL, INVALID, DTYPE, UNSUPPORTED = 0, -1, -2, -3, -5
P, P2, P3, P4, ODD = (ctypes.c_void_p(x) for x in (0x10000, 0x20000, 0x30000, 0x40000, 0x10004))
BIG = 1 << 40


def cache(data=0x50000, **kw):
    d = dict(block_stride=4096, token_stride=256, head_stride=128)
    d.update(kw)
    return scs.sc_paged_cache(data=data, **d)


def norm_desc(**kw):
    d = dict(num_q_heads=4, num_kv_heads=2, head_dim=128, rotary_dim=64, interleaved=0, dtype=1,
             table_dtype=0, eps=1e-6, block_size=16, num_blocks=8, q_row_stride=512,
             k_row_stride=256, v_row_stride=256, q_out_row_stride=512, k_out_row_stride=256,
             table_row_stride=64, max_position=100)
    d.update(kw)
    return scs.sc_qk_norm_desc(**d)


def norm(d, *, q=P, k=P2, v=P, q_out=P3, k_out=P4, table=P, pos=P, slots=P, kc=True, vc=True, T=5):
    ref = lambda c: None if c is None else ctypes.byref(cache() if c is True else c)
    return scs.lib().sc_qk_norm_rope(None if d is None else ctypes.byref(d), q, k, v, q_out, k_out,
                                     P, P, table, pos, slots, ref(kc), ref(vc), T, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=0), DTYPE), (dict(table_dtype=7), DTYPE), (dict(num_q_heads=0), INVALID),
    (dict(num_q_heads=3), INVALID), (dict(num_kv_heads=0), INVALID), (dict(head_dim=0), INVALID),
    (dict(head_dim=96), UNSUPPORTED), (dict(rotary_dim=-8), INVALID),
    (dict(rotary_dim=136), INVALID), (dict(rotary_dim=36), UNSUPPORTED),
    (dict(interleaved=2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(block_size=0), INVALID), (dict(num_blocks=-1), INVALID),
    (dict(q_row_stride=511), INVALID), (dict(k_row_stride=255), INVALID),
    (dict(v_row_stride=255), INVALID), (dict(q_out_row_stride=511), INVALID),
    (dict(k_out_row_stride=255), INVALID), (dict(table_row_stride=63), INVALID),
    (dict(max_position=0), INVALID), (dict(q_row_stride=514), UNSUPPORTED),
    (dict(v_row_stride=258), UNSUPPORTED), (dict(k_out_row_stride=257), UNSUPPORTED),
])
def test_norm_descriptor_refusals(kw, status):
    assert norm(norm_desc(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(T=0, q=None, q_out=None), OK), (dict(q=None), NULL),
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(q_out=None), NULL), (dict(table=None), NULL),
    (dict(pos=None), NULL), (dict(slots=None), NULL), (dict(kc=None), NULL), (dict(vc=None), NULL),
    (dict(kc=cache(data=None)), NULL), (dict(vc=cache(token_stride=-4)), INVALID),
    (dict(kc=cache(block_stride=4098)), UNSUPPORTED), (dict(vc=cache(data=0x50004)), UNSUPPORTED),
    (dict(q=ODD), UNSUPPORTED), (dict(k_out=ODD), UNSUPPORTED), (dict(v=ODD), UNSUPPORTED),
    (dict(q_out=P2), INVALID), (dict(k_out=P), INVALID), (dict(q_out=P4), INVALID),
])
def test_norm_refusals(kw, status):
    assert norm(norm_desc(), **kw) == status
    assert norm(None) == NULL


def test_norm_in_place_needs_one_stride():
    assert norm(norm_desc(q_out_row_stride=516), q_out=P) == INVALID
    assert norm(norm_desc(k_out_row_stride=260), k_out=P2) == INVALID


def attn_desc(**kw):
    d = dict(num_q_heads=4, num_kv_heads=2, head_dim=128, dtype=1, block_size=16, num_blocks=8,
             scale=0.1, q_row_stride=512, out_row_stride=512, block_table_row_stride=4)
    d.update(kw)
    return scs.sc_paged_attn_desc(**d)


def attn(d, *, q=P, out=P2, kc=True, vc=True, table=P, blocks=4, lens=P, batch=2, n=1, top=64,
         ws=P, ws_bytes=BIG):
    ref = lambda c: None if c is None else ctypes.byref(cache() if c is True else c)
    return scs.lib().sc_paged_attn_decode(None if d is None else ctypes.byref(d), q, out, ref(kc),
                                          ref(vc), table, blocks, lens, batch, n, top, ws, ws_bytes,
                                          None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=0), DTYPE), (dict(num_q_heads=0), INVALID), (dict(num_q_heads=5), INVALID),
    (dict(num_kv_heads=0), INVALID), (dict(head_dim=-1), INVALID), (dict(head_dim=80), UNSUPPORTED),
    (dict(block_size=0), INVALID), (dict(block_size=24), UNSUPPORTED), (dict(num_blocks=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(q_row_stride=511), INVALID),
    (dict(q_row_stride=516), UNSUPPORTED), (dict(out_row_stride=500), INVALID),
    (dict(out_row_stride=514), UNSUPPORTED), (dict(block_table_row_stride=0), INVALID),
])
def test_attn_descriptor_refusals(kw, status):
    d = attn_desc(**kw)
    assert attn(d) == status
    n = ctypes.c_int64(0)
    assert scs.lib().sc_paged_attn_workspace_bytes(ctypes.byref(d), 2, 1, 64, ctypes.byref(n)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), INVALID), (dict(n=-1), INVALID), (dict(top=-1), INVALID),
    (dict(top=65), INVALID), (dict(blocks=-1), INVALID), (dict(blocks=5), INVALID),
    (dict(ws_bytes=-1), INVALID), (dict(batch=1 << 29), UNSUPPORTED), (dict(q=None), NULL),
    (dict(out=None), NULL), (dict(out=P), INVALID), (dict(kc=None), NULL), (dict(vc=None), NULL),
    (dict(table=None), NULL), (dict(lens=None), NULL), (dict(kc=cache(data=None)), NULL),
    (dict(kc=cache(data=0x50008)), UNSUPPORTED), (dict(vc=cache(head_stride=12)), UNSUPPORTED),
    (dict(q=ODD), UNSUPPORTED), (dict(out=ODD), UNSUPPORTED),
    (dict(batch=0, q=None, kc=None), OK), (dict(n=0, q=None), OK),
    (dict(top=(1 << 30) + 1), UNSUPPORTED),
])
def test_attn_refusals(kw, status):
    assert attn(attn_desc(), **kw) == status
    assert attn(None) == NULL


def test_attn_workspace_is_checked():
    need = scs.sc_paged_attn_workspace_bytes(1, max_seq_len=1 << 16, num_q_heads=4, num_kv_heads=2,
                                             head_dim=128)
    assert need > 0
    d = attn_desc(block_table_row_stride=1 << 12, num_blocks=1 << 12)
    call = dict(batch=1, blocks=1 << 12, top=1 << 16)
    assert attn(d, **call, ws_bytes=need - 1) == INVALID
    assert attn(d, **call, ws=None) == NULL
    assert attn(d, **call, ws=ODD) == INVALID
    assert scs.lib().sc_paged_attn_workspace_bytes(None, 1, 1, 1, None) == NULL
    with pytest.raises(scs.ScError):
        scs.sc_paged_attn_workspace_bytes(-1, max_seq_len=1, num_q_heads=4, num_kv_heads=2,
                                          head_dim=128)


def attn_tensors():
    torch = pytest.importorskip("torch")
    bf = torch.bfloat16
    return torch, dict(query=torch.zeros(4, 512, dtype=bf), out=torch.zeros(4, 512, dtype=bf),
                       k_cache=torch.zeros(8, 16, 2, 128, dtype=bf),
                       v_cache=torch.zeros(8, 16, 2, 128, dtype=bf),
                       block_table=torch.zeros(4, 4, dtype=torch.int32),
                       seq_lens=torch.zeros(4, dtype=torch.int32))


@pytest.mark.parametrize("change", ["q", "width", "out", "out_dtype", "v_heads", "v_blocks",
                                    "cache_stride", "table_dtype", "table_stride", "few_lens",
                                    "few_rows", "lens_dtype", "host"])
def test_attn_binding_refuses(change):
    torch, t = attn_tensors()
    q = 1
    if change == "q":
        q = 3
    elif change == "width":
        t["query"] = t["query"][:, :500]
    elif change == "out":
        t["out"] = t["out"][:3]
    elif change == "out_dtype":
        t["out"] = t["out"].float()
    elif change == "v_heads":
        t["v_cache"] = t["v_cache"][:, :, :1]
    elif change == "v_blocks":
        t["v_cache"] = t["v_cache"][:7]
    elif change == "cache_stride":
        t["k_cache"] = torch.zeros(8, 16, 128, 2, dtype=torch.bfloat16).transpose(2, 3)
    elif change == "table_dtype":
        t["block_table"] = t["block_table"].long()
    elif change == "table_stride":
        t["block_table"] = torch.zeros(4, 8, dtype=torch.int32)[:, ::2]
    elif change == "few_lens":
        t["seq_lens"] = t["seq_lens"][:3]
    elif change == "few_rows":
        t["block_table"] = t["block_table"][:3]
    elif change == "lens_dtype":
        t["seq_lens"] = t["seq_lens"].long()
    with pytest.raises(ValueError):
        scs.sc_paged_attn_decode(*t.values(), max_seq_len=64, q=q)


@pytest.mark.parametrize("top", [-1, 1 << 31, (1 << 32) + 5])
def test_attn_binding_refuses_lengths_that_do_not_fit(top):
    _, t = attn_tensors()
    with pytest.raises(ValueError):
        scs.sc_paged_attn_decode(*t.values(), max_seq_len=top)


@pytest.mark.parametrize("change", ["head_dim", "one_cache", "value", "q_out", "k_out", "weight",
                                    "cache_heads", "cache_blocks", "host"])
def test_norm_binding_refuses(change):
    torch = pytest.importorskip("torch")
    bf = torch.bfloat16
    z = lambda *s: torch.zeros(*s, dtype=bf)
    t = dict(query=z(4, 512), key=z(4, 256), value=z(4, 256), q_out=z(4, 512), k_out=z(4, 256),
             q_weight=z(128), k_weight=z(128), cos_sin=torch.zeros(9, 64),
             positions=torch.zeros(4, dtype=torch.int64), slots=torch.zeros(4, dtype=torch.int64),
             k_cache=z(8, 16, 2, 128), v_cache=z(8, 16, 2, 128))
    hd = 128
    if change == "head_dim":
        hd = 100
    elif change == "one_cache":
        t["v_cache"] = None
    elif change == "value":
        t["value"] = t["value"][:3]
    elif change == "q_out":
        t["q_out"] = t["q_out"].float()
    elif change == "k_out":
        t["k_out"] = t["k_out"][:, :128]
    elif change == "weight":
        t["k_weight"] = t["k_weight"][:64]
    elif change == "cache_heads":
        t["k_cache"] = z(8, 16, 4, 128)
    elif change == "cache_blocks":
        t["v_cache"] = z(9, 16, 2, 128)
    with pytest.raises(ValueError):
        scs.sc_qk_norm_rope(*t.values(), head_dim=hd)


@pytest.mark.parametrize("nq,nkv,hd,batch,q,top", [(7, 1, 128, 1, 1, 3500), (3, 3, 64, 5, 1, 2300),
                                                   (1, 1, 256, 1, 1, 1400), (8, 2, 128, 2, 2, 4096)])
def test_attn_parts_are_whole_vectors(nq, nkv, hd, batch, q, top):
    """The parts of the splits are stored 16 bytes at a time, behind two floats
    for each: they begin at a multiple of 16 bytes, so that the workspace, parts
    of 4 hd bytes behind it, has whole vectors too."""
    need = scs.sc_paged_attn_workspace_bytes(batch, q=q, max_seq_len=top, num_q_heads=nq,
                                             num_kv_heads=nkv, head_dim=hd)
    assert need > 0 and need % 16 == 0


@pytest.mark.parametrize("missing", ["value", "slots", "positions"])
def test_norm_binding_names_what_is_missing(missing):
    """value and slots belong to the caches, positions to the table."""
    torch = pytest.importorskip("torch")
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    t = dict(query=z(4, 512), key=z(4, 256), value=z(4, 256), q_out=z(4, 512), k_out=None,
             q_weight=None, k_weight=None, cos_sin=torch.zeros(9, 64),
             positions=torch.zeros(4, dtype=torch.int64), slots=torch.zeros(4, dtype=torch.int64),
             k_cache=z(8, 16, 2, 128), v_cache=z(8, 16, 2, 128))
    t[missing] = None
    with pytest.raises(ValueError, match=missing):
        scs.sc_qk_norm_rope(*t.values(), head_dim=128)
