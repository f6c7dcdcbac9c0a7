"""Tensors that the calls on quantised caches and shared prefixes cannot do without are
named if they are missing, without a GPU."""
import pytest

import stateful_causal_short_amd as scs
from tests.test_attn_fp8_host import tensors

CODES = ("k_cache", "k_scale", "v_cache", "v_scale")


@pytest.mark.parametrize("name", CODES + ("block_table", "start_loc", "k_out", "v_out"))
def test_read(name):
    torch, t = tensors()
    rows = torch.zeros(9, 256, dtype=torch.bfloat16)
    call = {n: t[n] for n in CODES + ("block_table",)}
    call.update(k_out=rows, v_out=rows.clone(), start_loc=torch.zeros(5, dtype=torch.int32))
    with pytest.raises(ValueError, match=name):
        scs.sc_paged_cache_read_fp8(**dict(call, **{name: None}))


@pytest.mark.parametrize("name", CODES)
def test_attention_over_codes(name):
    _, t = tensors()
    call = {n: x for n, x in t.items() if n not in ("group_start_loc", "prefix_lens")}
    with pytest.raises(ValueError, match=name):
        scs.sc_paged_attn_decode_fp8(**dict(call, **{name: None}), max_seq_len=64)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", ["k_cache", "v_cache", "group_start_loc", "prefix_lens"])
def test_attention_over_prefixes(name, fp8):
    torch, t = tensors()
    if not fp8:
        t = {n: x for n, x in t.items() if not n.endswith("_scale")}
        t["k_cache"] = t["v_cache"] = torch.zeros(8, 16, 2, 128, dtype=torch.bfloat16)
    fn = scs.sc_paged_attn_prefix_fp8 if fp8 else scs.sc_paged_attn_prefix
    with pytest.raises(ValueError, match=name):
        fn(**dict(t, **{name: None}), max_seq_len=64, max_prefix_len=32)
