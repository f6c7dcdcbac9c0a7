"""Every code under every scale of the quantised cache, read back on the GPU."""
import pytest

torch = pytest.importorskip("torch")

from tests._fp8 import BF16, CODES, E4M3, F64, U8  # noqa: E402
from tests.test_gpu_attn import i32, scs  # noqa: E402

pytestmark = pytest.mark.gpu


def test_every_code_and_scale():
    """Exact in bf16's range: below 2^-126 in its steps of 2^-133, nearest even, and what
    reaches 2^128 is infinite. The byte 255 has no value."""
    print("[gpu] every code and scale", flush=True)
    hd, block = 256, 16
    codes = torch.arange(256, dtype=U8, device="cuda").expand(256, 1, hd).reshape(16, block, 1, hd).contiguous()
    scale = torch.arange(256, dtype=U8, device="cuda").view(16, 1, block)
    ko, vo = (torch.empty(256, hd, dtype=BF16, device="cuda") for _ in range(2))
    scs().sc_paged_cache_read_fp8(codes.view(E4M3), scale, codes.flip(0).contiguous().view(E4M3), scale, ko, vo,
                                  i32([list(range(16))]), i32([0, 256]))
    power = torch.pow(torch.tensor(2.0, dtype=F64), torch.arange(256, dtype=F64) - 127)[:, None]
    x = CODES * power
    # a double's rounding to bf16 in 64 bits: steps of 2^-7 of its power of two, 2^-133 at least
    step = torch.exp2(torch.clamp(torch.frexp(x)[1].to(F64) - 8, min=-133.0))
    want = torch.round(x / step) * step
    want = torch.where(want.abs() >= 2.0 ** 128, torch.copysign(torch.tensor(float("inf"), dtype=F64), want), want)
    for out in (ko, vo):
        assert torch.equal(out.cpu().to(F64)[:255].nan_to_num(nan=3.5), want[:255].nan_to_num(nan=3.5))


def test_keys_past_fp32():
    """A normalised key of sqrt(64) times a weight of 2^126 passes 2^128: a NaN code, and the
    others, 2^-20 of it, have the scale of the largest that is left."""
    print("[gpu] keys past fp32", flush=True)
    hd = 64
    k = torch.full((1, hd), 2.0 ** -20, dtype=BF16)
    k[0, 5] = 1.0
    w = torch.full((hd,), 2.0 ** 126, dtype=BF16)
    q = torch.zeros(1, hd, dtype=BF16, device="cuda")
    c = [torch.zeros(1, 1, 1, hd, dtype=U8, device="cuda").view(E4M3), torch.zeros(1, 1, 1, dtype=U8, device="cuda"),
         torch.zeros(1, 1, 1, hd, dtype=U8, device="cuda").view(E4M3), torch.zeros(1, 1, 1, dtype=U8, device="cuda")]
    scs().sc_qk_norm_rope_fp8(q, k.cuda(), q, torch.empty_like(q), None, None, w.cuda(), None, None,
                              torch.zeros(1, dtype=torch.int64, device="cuda"), *c, head_dim=hd, eps=0.0)
    x = k[0].to(F64)
    x = x / x.square().mean().sqrt() * 2.0 ** 126
    got = CODES[c[0].view(U8).cpu().view(-1).long()] * 2.0 ** (int(c[1]) - 127)
    rest = torch.arange(hd) != 5
    assert bool(got[5].isnan()) and bool(x[5] >= 2.0 ** 128)
    # one rounding to four significant bits, and the byte is of these alone: 2^109 = 256 2^101
    assert bool(((got[rest] - x[rest]).abs() <= 2.0 ** -4 * x[rest]).all()) and int(c[1]) == 101 + 127
