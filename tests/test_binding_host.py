"""What the binding offers and how it packs its arguments, without a GPU."""
import ctypes

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
