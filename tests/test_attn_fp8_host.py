"""Refusals of the calls on quantised caches and of attention over shared prefixes,
without a GPU: the C entries return their status before any launch (the fake
pointers are never read), and the binding raises on tensors that do not fit."""
import ctypes

import pytest

import stateful_causal_short_amd as scs

from tests.test_attn_host import (BIG, DTYPE, INVALID, NULL, ODD, OK, P, P2, P3, P4, UNSUPPORTED,
                                  attn_desc, cache, norm_desc)

OFF16 = ctypes.c_void_p(0x10008)


def q8(**kw):
    d = dict(data=0x50000, block_stride=4096, token_stride=256, head_stride=128, scale=0x60000,
             scale_block_stride=32, scale_head_stride=16)
    d.update(kw)
    return scs.sc_paged_cache_fp8(**d)


def ref(c, default=q8):
    return None if c is None else ctypes.byref(default() if c is True else c)


def norm(d, *, q=P, k=P2, v=P, q_out=P3, k_out=P4, slots=P, kc=True, vc=True, T=5):
    return scs.lib().sc_qk_norm_rope_fp8(None if d is None else ctypes.byref(d), q, k, v, q_out,
                                         k_out, P, P, P, P, slots, ref(kc), ref(vc), T, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(T=0, q=None), OK), (dict(q=None), NULL), (dict(v=None), NULL),
    (dict(slots=None), NULL), (dict(kc=None), NULL), (dict(vc=None), NULL),
    (dict(kc=None, vc=None), NULL), (dict(kc=q8(data=None)), NULL), (dict(vc=q8(scale=None)), NULL),
    (dict(vc=q8(token_stride=-4)), INVALID), (dict(kc=q8(scale_head_stride=-1)), INVALID),
    (dict(kc=q8(block_stride=4098)), UNSUPPORTED), (dict(vc=q8(data=0x50002)), UNSUPPORTED),
    (dict(vc=q8(scale=0x60003, scale_block_stride=33)), OK), (dict(q_out=P2), INVALID),
    (dict(q=ODD), UNSUPPORTED),
])
def test_quantising_norm_refusals(kw, status):
    if status == OK and "vc" in kw:
        kw = dict(kw, T=0)                       # accepted, without a launch
    assert norm(norm_desc(), **kw) == status
    assert norm(None) == NULL


@pytest.mark.parametrize("kw,status", [(dict(dtype=0), DTYPE), (dict(head_dim=96), UNSUPPORTED),
                                       (dict(v_row_stride=255), INVALID), (dict(block_size=0), INVALID)])
def test_quantising_norm_descriptor(kw, status):
    assert norm(norm_desc(**kw)) == status


def read(*, desc=None, kc=True, vc=True, k=P, v=P2, table=P, blocks=4, starts=P, first=None, batch=2,
         rows=9, **kw):
    d = dict(num_kv_heads=2, head_dim=128, block_size=16, num_blocks=8, k_row_stride=256,
             v_row_stride=256, block_table_row_stride=4)
    d.update(kw)
    d = ctypes.byref(scs.sc_cache_read_desc(**d)) if desc is None else None
    return scs.lib().sc_paged_cache_read_fp8(d, ref(kc), ref(vc), k, v, table, blocks, starts, first,
                                             batch, rows, None)


@pytest.mark.parametrize("kw,status", [
    (dict(desc=False), NULL), (dict(num_kv_heads=0), INVALID), (dict(head_dim=80), UNSUPPORTED),
    (dict(head_dim=0), INVALID), (dict(block_size=0), INVALID), (dict(num_blocks=-1), INVALID),
    (dict(k_row_stride=255), INVALID), (dict(v_row_stride=260), UNSUPPORTED),
    (dict(block_table_row_stride=3), INVALID), (dict(blocks=-1), INVALID), (dict(batch=-1), INVALID),
    (dict(rows=-1), INVALID), (dict(rows=1 << 31), UNSUPPORTED), (dict(rows=0, k=None), OK),
    (dict(batch=0, starts=None), OK), (dict(k=None), NULL), (dict(v=None), NULL), (dict(kc=None), NULL),
    (dict(vc=None), NULL), (dict(starts=None), NULL), (dict(table=None), NULL), (dict(v=P), INVALID),
    (dict(k=OFF16), UNSUPPORTED), (dict(kc=q8(data=0x50008)), UNSUPPORTED),
    (dict(vc=q8(token_stride=264)), UNSUPPORTED), (dict(kc=q8(scale=None)), NULL),
])
def test_read_refusals(kw, status):
    assert read(**kw) == status


def attn(d, *, q=P, out=P2, kc=True, vc=True, table=P, blocks=4, lens=P, batch=2, n=1, top=64, ws=P,
         ws_bytes=BIG):
    return scs.lib().sc_paged_attn_decode_fp8(None if d is None else ctypes.byref(d), q, out, ref(kc),
                                              ref(vc), table, blocks, lens, batch, n, top, ws, ws_bytes,
                                              None)


def prefix(d, fp8, *, q=P, out=P2, kc=True, vc=True, table=P, blocks=4, lens=P, starts=P, pre=P, groups=2,
           batch=2, n=1, top=64, longest=32, ws=P, ws_bytes=BIG):
    fn = scs.lib().sc_paged_attn_prefix_fp8 if fp8 else scs.lib().sc_paged_attn_prefix
    kind = q8 if fp8 else cache
    return fn(None if d is None else ctypes.byref(d), q, out, ref(kc, kind), ref(vc, kind), table, blocks,
              lens, starts, pre, groups, batch, n, top, longest, ws, ws_bytes, None)


CALLS = [(dict(batch=-1), INVALID), (dict(n=-1), INVALID), (dict(top=-1), INVALID),
         (dict(top=65), INVALID), (dict(blocks=5), INVALID), (dict(ws_bytes=-1), INVALID),
         (dict(batch=1 << 29), UNSUPPORTED), (dict(q=None), NULL), (dict(out=P), INVALID),
         (dict(kc=None), NULL), (dict(table=None), NULL), (dict(lens=None), NULL), (dict(q=ODD), UNSUPPORTED),
         (dict(out=ODD), UNSUPPORTED), (dict(batch=0, q=None), OK), (dict(n=0, q=None), OK)]


@pytest.mark.parametrize("kw,status", CALLS + [
    (dict(kc=q8(data=None)), NULL), (dict(vc=q8(scale=None)), NULL), (dict(kc=q8(data=0x50008)), UNSUPPORTED),
    (dict(vc=q8(head_stride=24)), UNSUPPORTED), (dict(vc=q8(scale=0x60002)), UNSUPPORTED),
    (dict(kc=q8(scale_block_stride=34)), UNSUPPORTED)])
def test_attention_over_codes_refusals(kw, status):
    assert attn(attn_desc(), **kw) == status
    assert attn(None) == NULL


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,status", CALLS + [
    (dict(groups=-1), INVALID), (dict(longest=-1), INVALID), (dict(longest=65), INVALID),
    (dict(starts=None), NULL), (dict(pre=None), NULL), (dict(groups=0, batch=0, starts=None, pre=None), OK),
    (dict(ws=None), NULL), (dict(ws=ODD), INVALID), (dict(ws_bytes=16), INVALID)])
def test_prefix_refusals(kw, status, fp8):
    assert prefix(attn_desc(), fp8, **kw) == status
    assert prefix(None, fp8) == NULL


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=0), DTYPE), (dict(num_q_heads=5), INVALID), (dict(head_dim=80), UNSUPPORTED),
    (dict(block_size=24), UNSUPPORTED), (dict(scale=float("inf")), INVALID), (dict(q_row_stride=516), UNSUPPORTED)])
def test_descriptor_refusals(kw, status):
    d = attn_desc(**kw)
    n = ctypes.c_int64(0)
    assert attn(d) == status and prefix(d, False) == status and prefix(d, True) == status
    L = scs.lib()
    assert L.sc_paged_attn_fp8_workspace_bytes(ctypes.byref(d), 2, 1, 64, ctypes.byref(n)) == status
    assert L.sc_paged_attn_prefix_workspace_bytes(ctypes.byref(d), 2, 1, 64, 1, 32, ctypes.byref(n)) == status


def test_workspaces():
    """Whole vectors, large enough to be used; a prefix call always needs one."""
    heads = dict(num_q_heads=7, num_kv_heads=1, head_dim=128)
    assert scs.sc_paged_attn_fp8_workspace_bytes(1, max_seq_len=3500, **heads) % 16 == 0
    for B, q, top, pre, groups in ((1, 1, 1, 0, 0), (3, 2, 5000, 4999, 3), (512, 1, 40000, 32768, 1)):
        need = scs.sc_paged_attn_prefix_workspace_bytes(B, q=q, max_seq_len=top, num_groups=groups,
                                                        max_prefix_len=pre, **heads)
        assert need >= B * q * 7 * (128 + 2) * 4 and need % 16 == 0
    for kw in (dict(batch=1 << 31), dict(num_groups=1 << 31), dict(max_prefix_len=1 << 32)):
        call = dict(batch=1, max_seq_len=64, num_groups=1, max_prefix_len=32, **heads)
        call.update(kw)
        with pytest.raises(ValueError):
            scs.sc_paged_attn_prefix_workspace_bytes(call.pop("batch"), **call)


@pytest.mark.parametrize("packer,structure", [("_CACHE_FP8_DESC", scs.sc_paged_cache_fp8),
                                              ("_CACHE_READ_DESC", scs.sc_cache_read_desc)])
def test_packed_descriptors(packer, structure):
    pack = getattr(scs, packer)
    assert pack.size == ctypes.sizeof(structure)
    values = range(3, 3 + len(structure._fields_))
    d = structure.from_buffer_copy(pack.pack(*values))
    assert [getattr(d, name) for name, _ in structure._fields_] == list(values)


def tensors():
    torch = pytest.importorskip("torch")
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)
    codes = lambda *s: z(*s, dtype=torch.uint8).view(torch.float8_e4m3fn)
    return torch, dict(query=z(4, 512), out=z(4, 512), k_cache=codes(8, 16, 2, 128),
                       k_scale=z(8, 2, 16, dtype=torch.uint8).view(torch.float8_e8m0fnu),
                       v_cache=codes(8, 16, 2, 128), v_scale=z(8, 2, 16, dtype=torch.uint8),
                       block_table=z(4, 4, dtype=torch.int32), seq_lens=z(4, dtype=torch.int32),
                       group_start_loc=z(3, dtype=torch.int32), prefix_lens=z(2, dtype=torch.int32))


CHANGES = {
    "bf16 codes": dict(k_cache=lambda t, x: x.to(t.bfloat16)),
    "value heads": dict(v_cache=lambda t, x: x[:, :, :1]),
    "no scale": dict(v_scale=lambda t, x: None),
    "scale order": dict(k_scale=lambda t, x: x.transpose(1, 2)),
    "scale stride": dict(v_scale=lambda t, x: t.zeros(8, 2, 32, dtype=t.uint8)[:, :, ::2]),
    "scale type": dict(v_scale=lambda t, x: x.int()),
    "scale blocks": dict(k_scale=lambda t, x: x[:7]),
    "table rows": dict(block_table=lambda t, x: x[:3]),
    "host": {},
}


@pytest.mark.parametrize("change", CHANGES)
def test_binding_refuses(change):
    torch, t = tensors()
    for name, f in CHANGES[change].items():
        t[name] = f(torch, t[name])
    a = [t[n] for n in ("query", "out", "k_cache", "k_scale", "v_cache", "v_scale", "block_table", "seq_lens")]
    with pytest.raises(ValueError):
        scs.sc_paged_attn_decode_fp8(*a, max_seq_len=64)
    with pytest.raises(ValueError):
        scs.sc_paged_attn_prefix_fp8(*a, t["group_start_loc"], t["prefix_lens"], max_seq_len=64, max_prefix_len=32)
    rows = torch.zeros(9, 256, dtype=torch.bfloat16)
    start = torch.zeros(5, dtype=torch.int32)
    with pytest.raises(ValueError):
        scs.sc_paged_cache_read_fp8(*a[2:6], rows, rows.clone(), t["block_table"], start)
    if change != "table rows":
        z = lambda n: torch.zeros(4, n, dtype=torch.bfloat16)
        with pytest.raises(ValueError):
            scs.sc_qk_norm_rope_fp8(z(512), z(256), z(256), z(512), None, None, None, None, None,
                                    torch.zeros(4, dtype=torch.int64), *a[2:6], head_dim=128)


@pytest.mark.parametrize("kw", [dict(group_start_loc=2), dict(prefix_lens="float"), dict(max_prefix_len=-1),
                                dict(max_prefix_len=1 << 31), dict(q=3)])
def test_prefix_binding_refuses(kw):
    torch, t = tensors()
    bf = torch.zeros(8, 16, 2, 128, dtype=torch.bfloat16)
    call = dict(max_seq_len=64, max_prefix_len=32)
    if "group_start_loc" in kw:
        t["group_start_loc"] = t["group_start_loc"][:2]
    elif "prefix_lens" in kw:
        t["prefix_lens"] = t["prefix_lens"].float()
    else:
        call.update(kw)
    with pytest.raises(ValueError):
        scs.sc_paged_attn_prefix(t["query"], t["out"], bf, bf, t["block_table"], t["seq_lens"],
                                 t["group_start_loc"], t["prefix_lens"], **call)


@pytest.mark.parametrize("change", ["starts", "starts type", "first", "width", "rows", "one row set"])
def test_read_binding_refuses(change):
    torch, t = tensors()
    k, v = (torch.zeros(9, 256, dtype=torch.bfloat16) for _ in range(2))
    starts, first = torch.zeros(5, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    if change == "starts":
        starts = starts[:0]
    elif change == "starts type":
        starts = starts.long()
    elif change == "first":
        first = first[:3]
    elif change == "width":
        k = k[:, :128]
    elif change == "rows":
        v = v[:8]
    else:
        v = v.float()
    with pytest.raises(ValueError):
        scs.sc_paged_cache_read_fp8(t["k_cache"], t["k_scale"], t["v_cache"], t["v_scale"], k, v,
                                    t["block_table"], starts, first)


def test_prefix_token_strides():
    """Sixteen tokens of a cache lie within 2^31 bytes."""
    for which in ("kc", "vc"):
        assert prefix(attn_desc(), False, **{which: cache(token_stride=1 << 26)}) == UNSUPPORTED
        assert prefix(attn_desc(), True, **{which: q8(token_stride=1 << 26)}) == UNSUPPORTED


def test_decode_token_strides():
    for which in ("kc", "vc"):
        assert attn(attn_desc(), **{which: q8(token_stride=1 << 26)}) == UNSUPPORTED
