"""What the binding offers and how it packs its arguments, without a GPU."""
import ctypes
from types import SimpleNamespace

import pytest

import stateful_causal_short_amd as scs


def test_star_import_gives_every_call():
    """All entry points of the library with a binding, and their descriptors."""
    names = {}
    exec("from stateful_causal_short_amd import *", names)
    plain = {"sc_status_string", "sc_abi_version"}      # reached through ScError and lib()
    for name in scs.EXPORTS:
        assert name in plain or callable(names.get(name)), name
    for name, x in vars(scs).items():
        if isinstance(x, type) and issubclass(x, ctypes.Structure):
            assert names.get(name) is x, name


@pytest.mark.parametrize("packer,structure", [
    ("_GDN_DESC", scs.sc_gdn_desc), ("_QK_NORM_DESC", scs.sc_qk_norm_desc),
    ("_ATTN_DESC", scs.sc_paged_attn_desc), ("_CACHE_DESC", scs.sc_paged_cache)])
def test_packed_descriptors_have_the_layout_of_the_structures(packer, structure):
    pack = getattr(scs, packer)
    assert pack.size == ctypes.sizeof(structure)
    values = range(3, 3 + len(structure._fields_))
    d = structure.from_buffer_copy(pack.pack(*values))
    assert [getattr(d, name) for name, _ in structure._fields_] == list(values)


@pytest.mark.parametrize("sizes", [dict(batch=(1 << 32) + 1), dict(q=(1 << 32) + 1),
                                   dict(max_seq_len=(1 << 32) + 64), dict(max_seq_len=1 << 31)])
def test_attention_workspace_sizes_are_not_cut(sizes):
    call = dict(batch=1, q=1, max_seq_len=64)
    call.update(sizes)
    with pytest.raises(ValueError):
        scs.sc_paged_attn_workspace_bytes(**call, num_q_heads=4, num_kv_heads=2, head_dim=128)


@pytest.mark.parametrize("tokens,batch", [(64, (1 << 32) + 1), (64, 1 << 31), ((1 << 64) + 64, 1)])
def test_delta_rule_workspace_sizes_are_not_cut(tokens, batch):
    with pytest.raises(ValueError):
        scs.sc_gdn_workspace_bytes(tokens, batch, num_k_heads=2, num_v_heads=4, head_k_dim=128,
                                   head_v_dim=64)


def test_streams_of_another_device_are_refused(monkeypatch):
    """The kernels run on the current device, and so must their stream."""
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    tensor = SimpleNamespace(is_cuda=True, get_device=lambda: 1)
    here, there = (SimpleNamespace(cuda_stream=77, device_index=i) for i in (1, 0))
    assert scs._stream(here, tensor) == 77
    with pytest.raises(ValueError, match="cuda:0"):
        scs._stream(there, tensor)
