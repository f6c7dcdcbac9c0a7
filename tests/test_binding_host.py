"""What the binding offers and how it packs its arguments, without a GPU."""
import ctypes

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
