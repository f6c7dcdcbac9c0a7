"""The quantised cache's format in 64 bits, and caches of it for the tests."""
import numpy as np
import torch

F64, BF16, U8 = torch.float64, torch.bfloat16, torch.uint8
E4M3 = torch.float8_e4m3fn


def code_values():
    """The value of each of the 256 codes: sign, four bits of exponent, three of
    mantissa; no infinities, 0x7F and 0xFF NaN."""
    c = np.arange(256)
    e, m = c >> 3 & 15, c & 7
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = np.where(c & 127 == 127, np.nan, v)
    return torch.tensor(np.where(c & 128, -v, v))


CODES = code_values()


def scale_bytes(x):
    """The byte of the scale 2^(byte - 127) of heads x (..., hd) in 64 bits: the
    smallest, from 1 on, that brings the largest finite value to 448 or less."""
    top = torch.where(x.isfinite(), x, 0.0).abs().amax(-1)
    m, e = torch.frexp(top)                       # top = m 2^e, 1/2 <= m < 1; 448 = 7/8 2^9
    b = e - 9 + (m > 0.875).int() + 127
    return torch.where(top > 0, b, torch.ones_like(b)).clamp(min=1)


def dequantise(codes, scale):
    """Values in 64 bits of codes (blocks, block, nkv, hd) and the bytes (blocks, nkv,
    block) of their scales."""
    b = scale.view(U8).cpu().to(F64).transpose(1, 2)[..., None]
    return CODES[codes.view(U8).cpu().long()] * torch.pow(torch.tensor(2.0, dtype=F64), b - 127)


def quantise(x):
    """(codes, bytes) of bf16 heads x (..., hd), each value to the nearest code, ties to
    the even one; not a number where x is not finite."""
    x = x.to(F64)
    b = scale_bytes(x)
    y = x * torch.pow(torch.tensor(2.0, dtype=F64), 127 - b.to(F64))[..., None]
    size = CODES[:127]                             # rising with the code
    a = torch.nan_to_num(y.abs(), nan=0.0, posinf=0.0)
    hi = torch.searchsorted(size, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - size[lo], size[hi] - a
    c = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = torch.where(y.isfinite(), c, torch.full_like(c, 127))
    return (c + torch.where(torch.signbit(y) & y.isfinite(), 128, 0)).to(U8), b.to(U8)


def caches_fp8(layout, blocks, block, nkv, hd, code=0x7F, byte=255):
    """(k, k_scale, v, v_scale) filled with one code and one byte; "heads": heads before
    tokens, "joint": keys and values in one allocation, scales too."""
    full = lambda *s, v=code: torch.full(s, v, dtype=U8, device="cuda")
    if layout == "heads":
        t = [full(blocks, nkv, block, hd).transpose(1, 2) for _ in range(2)]
        s = [full(nkv, blocks, block, v=byte).transpose(0, 1) for _ in range(2)]
    elif layout == "joint":
        both, scales = full(blocks, 2, block, nkv, hd), full(blocks, 2, nkv, block, v=byte)
        t, s = [both[:, 0], both[:, 1]], [scales[:, 0], scales[:, 1]]
    else:
        t = [full(blocks, block, nkv, hd) for _ in range(2)]
        s = [full(blocks, nkv, block, v=byte) for _ in range(2)]
    return [t[0].view(E4M3), s[0].view(torch.float8_e8m0fnu), t[1].view(E4M3), s[1]]


def put(cache, scale, block, at, x):
    """Writes quantised heads x (n, nkv, hd) to tokens at.. of a block; their values."""
    codes, b = quantise(x)
    n = x.shape[0]
    cache.view(U8)[block, at:at + n] = codes.cuda()
    scale.view(U8)[block, :, at:at + n] = b.T.cuda()
    return CODES[codes.long()] * torch.pow(torch.tensor(2.0, dtype=F64), b.to(F64) - 127)[..., None]


def paged_fp8(g, lens, nkv, hd, block, layout, rng, spread=2.0):
    """Random keys and values of each request, of sizes that differ from token to
    token, in shuffled pages of quantised caches that hold NaN codes elsewhere.
    (caches, table, values of the keys, of the values)."""
    pages = [-(-n // block) for n in lens]
    blocks = sum(pages) + 2
    c = caches_fp8(layout, blocks, block, nkv, hd)
    order = rng.permutation(blocks)
    table = np.full((len(lens), max(max(pages), 1)), 10 ** 9)      # behind the end: not read
    made = [[], []]
    at = 0
    for r, p in enumerate(pages):
        table[r, :p] = order[at:at + p]
        for which in range(2):
            x = torch.randn(lens[r], nkv, hd, generator=g)
            if which:
                x = x * torch.exp2(spread * torch.randn(lens[r], nkv, 1, generator=g))
            x = x.to(BF16)
            vals = [put(c[2 * which], c[2 * which + 1], int(order[at + i]), 0,
                        x[i * block:(i + 1) * block]) for i in range(p)]
            made[which].append(torch.cat(vals) if vals else torch.zeros(0, nkv, hd, dtype=F64))
        at += p
    return c, table, made[0], made[1]
