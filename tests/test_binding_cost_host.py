"""How much the binding does for a call, without a GPU. A decode step is as long as
its marshalling, so the Python and C calls that each call makes are counted, on
host tensors, with the library, the stream and the addresses' checks stubbed."""
import sys

import pytest

import stateful_causal_short_amd as scs

torch = pytest.importorskip("torch")


class Library:
    def __getattr__(self, name):
        return lambda *args: scs.SC_OK


def calls(f):
    """Python and C calls that f() makes."""
    n = [0]

    def count(frame, event, arg):
        n[0] += event in ("call", "c_call")
    f()                                     # what is made once
    sys.setprofile(count)
    try:
        f()
    finally:
        sys.setprofile(None)
    return n[0] - 2                         # f itself and the last setprofile


@pytest.fixture
def stubs(monkeypatch):
    library = Library()
    monkeypatch.setattr(scs, "lib", lambda: library)
    monkeypatch.setattr(scs, "_stream", lambda stream, like=None: 0)
    monkeypatch.setattr(scs, "_device", lambda t: 0)
    monkeypatch.setattr(scs, "_addresses", lambda device, *tensors: [0] * len(tensors))


def test_attention_and_norms(stubs):
    """No more than when each had a body of its own."""
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)
    q, out, kc, vc = z(1, 2048), z(1, 2048), z(64, 16, 4, 128), z(64, 16, 4, 128)
    k, v, w = z(1, 512), z(1, 512), z(128)
    table, lens = z(1, 64, dtype=torch.int32), z(1, dtype=torch.int32)
    pos, angles, room = z(1, dtype=torch.int64), z(100, 128), z(4096, dtype=torch.uint8)
    attn = lambda **kw: scs.sc_paged_attn_decode(q, out, kc, vc, table, lens, max_seq_len=300, **kw)
    got = (calls(attn), calls(lambda: attn(workspace=room)),
           calls(lambda: scs.sc_qk_norm_rope(q, k, v, out, None, w, w, angles, pos, pos, kc, vc, head_dim=128)))
    assert all(a <= b for a, b in zip(got, (41, 40, 50))), got
