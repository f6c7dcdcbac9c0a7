"""The quantising cache write and the read back, on the GPU against the format's
definition in 64 bits on the CPU."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests._fp8 import BF16, CODES, E4M3, F64, U8, caches_fp8, dequantise, quantise, scale_bytes  # noqa: E402
from tests.test_gpu_attn import check_norm, i32, i64, norm_ref, randn, scs  # noqa: E402

pytestmark = pytest.mark.gpu

WRITES = [  # nq, nkv, hd, rot, interleaved, weights, tokens, block, layout, k_out
    (1, 1, 64, 64, False, True, 1, 16, "tokens", False),
    (4, 2, 128, 128, False, True, 7, 48, "joint", True),
    (4, 1, 128, 64, True, False, 33, 1, "heads", True),
    (6, 3, 64, 16, False, True, 19, 5, "joint", False),
    (16, 2, 256, 256, True, True, 65, 16, "heads", True),
    (7, 7, 256, 8, False, True, 5, 16, "tokens", False),
    (3, 1, 128, 0, False, True, 21, 16, "tokens", False),
    (8, 8, 64, 48, False, False, 1300, 528, "joint", True),
]


def split(rows, T, nq, nkv, hd):
    w = nq * hd, (nq + nkv) * hd, (nq + 2 * nkv) * hd
    return rows[:T, :w[0]], rows[:T, w[0]:w[1]], rows[:T, w[1]:w[2]]


@pytest.mark.parametrize("case", WRITES, ids=[f"{c[0]}-{c[1]}-{c[2]}-rot{c[3]}-{c[8]}" for c in WRITES])
def test_quantising_write(case):
    """Values are exactly the format's. Keys: one rounding to a code, half a step (2^-4
    of the value, or 2^-10 of the scale below the smallest normal code), before it
    the fp32 arithmetic of the norm, under 16 roundings of 2^-24 of sqrt(2 hd)
    times the largest weight; the scale's byte is that of a largest value this near."""
    nq, nkv, hd, rot, inter, weights, T, block, layout, k_out = case
    print(f"[gpu] quantising write {case}", flush=True)
    g = torch.Generator().manual_seed(T)
    rng = np.random.default_rng(T)
    rows = randn(g, T + 2, (nq + 2 * nkv) * hd + 4)
    rows[:, (nq + nkv) * hd:] *= torch.exp2(8 * torch.randn(T + 2, 1, generator=g)).to(BF16)
    w = [randn(g, hd) for _ in range(2)] if weights else [None, None]
    wmax = max([1.0] + [float(x.abs().max()) for x in w if x is not None])
    table = None
    if rot:
        ang = torch.arange(50, dtype=F64)[:, None] * torch.rand(rot // 2, generator=g, dtype=F64)
        table = torch.cat([ang.cos(), ang.sin()], 1).float()
    pos = rng.integers(0, 50, T)
    blocks = -(-T // block) + 2
    slots = rng.permutation(blocks * block)[:T]
    if T > 4:
        slots[3], slots[4] = -1, blocks * block     # not written
    d = rows.cuda()
    q, k, v = split(d, T, nq, nkv, hd)
    c = caches_fp8(layout, blocks, block, nkv, hd, 0x55, 77)
    qo = torch.full((T + 1, nq * hd), 7.5, dtype=BF16, device="cuda")
    ko = torch.full((T + 1, nkv * hd), 7.5, dtype=BF16, device="cuda") if k_out else None
    scs().sc_qk_norm_rope_fp8(q, k, v, qo, ko, *[None if x is None else x.cuda() for x in w],
                              None if table is None else table.cuda(),
                              None if table is None else i64(pos), i64(slots), *c,
                              head_dim=hd, eps=1e-5, interleaved=inter)
    hq, hk, hv = split(rows, T, nq, nkv, hd)
    want_k = norm_ref(hk, w[1], table, pos, hd, 1e-5, inter)
    check_norm(qo[:T].cpu().unflatten(1, (-1, hd)), norm_ref(hq, w[0], table, pos, hd, 1e-5, inter),
               hd, wmax)
    if k_out:
        check_norm(ko[:T].cpu().unflatten(1, (-1, hd)), want_k, hd, wmax)
    assert torch.equal(d.cpu(), rows) and bool((qo[T:] == 7.5).all())
    codes, byte = quantise(hv.unflatten(1, (nkv, hd)))
    got_k, got_v = (dequantise(c[i], c[i + 1]) for i in (0, 2))
    kb, vb = (c[i].view(U8).cpu() for i in (1, 3))
    vc, kc = c[2].view(U8).cpu(), c[0].view(U8).cpu()
    written = torch.zeros(blocks, block, dtype=torch.bool)
    near = 16 * 2.0 ** -24 * math.sqrt(2 * hd) * wmax
    for t in range(T):
        if not 0 <= slots[t] < blocks * block:
            continue
        b, i = divmod(int(slots[t]), block)
        written[b, i] = True
        assert torch.equal(vc[b, i], codes[t]) and torch.equal(vb[b, :, i], byte[t])
        top = want_k[t].abs().amax(-1)
        lo, hi = (scale_bytes((top + s * near)[:, None]) for s in (-1, 1))
        bytes_t = kb[b, :, i].int()
        assert bool(((bytes_t >= lo) & (bytes_t <= hi)).all())
        step = torch.pow(torch.tensor(2.0, dtype=F64), bytes_t.to(F64) - 127 - 10)[:, None]
        tol = torch.maximum(2.0 ** -4 * want_k[t].abs(), step) + near * (1 + 2.0 ** -4)
        assert bool(((got_k[b, i] - want_k[t]).abs() <= tol).all())
    for x, s in ((kc, kb), (vc, vb)):
        assert bool((x[~written] == 0x55).all())
        assert bool((s.transpose(1, 2)[~written] == 77).all())


@pytest.mark.parametrize("hd, rot, inter", [(128, 128, False), (64, 32, True), (256, 0, False)])
def test_key_codes_are_the_nearest(hd, rot, inter):
    """Every key code and byte is that of the norm in 64 bits. Both sides are off by
    some 2^-50 of a value and eps by 2^-24 of its own 2^-17 part of the sum; of two
    million values spread over steps of 2^-4 one in some 10^4 runs could differ."""
    T, nkv, block = 1 << 20 >> (hd.bit_length() - 1), 2, 16
    print(f"[gpu] key codes {hd} {rot} {inter}", flush=True)
    g = torch.Generator().manual_seed(hd)
    k, w = randn(g, T, nkv * hd), randn(g, hd)
    ang = torch.arange(T, dtype=F64)[:, None] * torch.rand(max(rot // 2, 1), generator=g, dtype=F64)
    table = torch.cat([ang.cos(), ang.sin()], 1).float() if rot else None
    pos = np.arange(T)
    c = caches_fp8("heads", T // block, block, nkv, hd)
    d = k.cuda()
    scs().sc_qk_norm_rope_fp8(d, d, d, torch.empty_like(d), None, None, w.cuda(),
                              None if table is None else table.cuda(),
                              i64(pos) if rot else None, i64(pos), *c,
                              head_dim=hd, eps=1e-5, interleaved=inter)
    codes, byte = quantise(norm_ref(k, w, table, pos, hd, 1e-5, inter))
    assert torch.equal(c[0].view(U8).cpu().reshape(T, nkv, hd), codes)
    assert torch.equal(c[1].view(U8).cpu().transpose(1, 2).reshape(T, nkv), byte)


def test_values_at_the_ends_of_the_format():
    """Heads of zeros, of one size, at 448 and the next bf16 above it, ties, the
    smallest and largest bf16 values, infinities and NaN: each value the format's."""
    hd = 64
    print("[gpu] quantising ends", flush=True)
    g = torch.Generator().manual_seed(1)
    inf, nan = float("inf"), float("nan")
    heads = [torch.zeros(hd), torch.full((hd,), -3.0), torch.full((hd,), 448.0),
             torch.full((hd,), 450.0), torch.linspace(-448, 448, hd), torch.linspace(-2, 2, hd) * 2.0 ** -133,
             torch.full((hd,), 2.0 ** -133), torch.full((hd,), 3.3895e38),
             torch.arange(hd) * 2.0 ** -10, (torch.arange(hd) * 2 + 1) * 2.0 ** -10,
             2.0 ** torch.arange(-50.0, 14.0), -(2.0 ** torch.arange(-20.0, 44.0))]
    x = torch.stack(heads).to(BF16)
    more = torch.randn(9, hd, generator=g).to(BF16)
    more[0, 3], more[1, 0], more[2, 63], more[3, :] = inf, -inf, nan, nan
    more[4, :], more[5, ::2], more[6, 1::2], more[7, 5:7] = inf, nan, -inf, torch.tensor([inf, nan], dtype=BF16)
    x = torch.cat([x, more])
    T = len(x)
    c = caches_fp8("tokens", T, 1, 1, hd, 0x11, 3)
    row = x.cuda()
    scs().sc_qk_norm_rope_fp8(row, torch.ones_like(row), row, torch.empty_like(row), None, None, None,
                              None, None, i64(np.arange(T)), *c, head_dim=hd)
    codes, byte = quantise(x)
    got = c[2].view(U8).cpu().view(T, hd)
    want_nan = ~x.isfinite()
    assert bool(((got & 0x7F) == 0x7F)[want_nan].all())
    assert torch.equal(got[~want_nan], codes[~want_nan])
    assert torch.equal(c[3].view(U8).cpu().view(T), byte)
    # a head of ones has the norm 1: the same code throughout
    assert bool((dequantise(c[0], c[1]) == 1.0).all())


def test_keys_that_are_not_finite():
    """NaN in a key makes its norm NaN: all codes of that head, and of no other."""
    hd, T = 128, 5
    print("[gpu] quantising NaN keys", flush=True)
    g = torch.Generator().manual_seed(2)
    k = randn(g, T, 2 * hd)
    k[2, 3] = float("nan")
    q, v = randn(g, T, 2 * hd), randn(g, T, 2 * hd)
    c = caches_fp8("tokens", T, 1, 2, hd, 0x11, 3)
    scs().sc_qk_norm_rope_fp8(q.cuda(), k.cuda(), v.cuda(), torch.empty(T, 2 * hd, dtype=BF16, device="cuda"),
                              None, None, None, None, None, i64(np.arange(T)), *c, head_dim=hd)
    got = dequantise(c[0], c[1]).view(T, 2, hd)
    assert bool(got[2, 0].isnan().all())
    got[2, 0] = 0
    assert bool(got.isfinite().all())


READS = [  # nkv, hd, block, layout, lens, first tokens
    (1, 64, 16, "tokens", [1], None),
    (2, 128, 5, "joint", [3, 0, 17, 0, 1], None),
    (4, 128, 16, "heads", [300, 1, 16, 15], [0, 3, 16, 31]),
    (3, 256, 528, "tokens", [600, 5], [1, 527]),
    (8, 64, 1, "joint", [0, 40, 9], None),
    (4, 128, 64, "tokens", [5000, 0, 0, 3, 12000], None),
    (1, 256, 16, "heads", [1] * 300, None),
]


@pytest.mark.parametrize("case", READS, ids=[f"{c[0]}-{c[1]}-{c[3]}-{len(c[4])}x{c[4][0]}" for c in READS])
def test_read_back(case):
    """Exact; rows of no request stay as they were."""
    nkv, hd, block, layout, lens, first = case
    print(f"[gpu] read back {case}", flush=True)
    rng = np.random.default_rng(hd + block)
    begin = first or [0] * len(lens)
    pages = [-(-(n + f) // block) for n, f in zip(lens, begin)]
    blocks = sum(pages) + 2
    c = caches_fp8(layout, blocks, block, nkv, hd)
    for i in range(2):       # any finite codes, any scales that keep bf16's range
        codes = rng.integers(0, 256, c[2 * i].shape).astype(np.uint8)
        codes[codes & 127 == 127] = 0x38
        c[2 * i].view(U8).copy_(torch.tensor(codes))
        c[2 * i + 1].view(U8).copy_(torch.tensor(rng.integers(11, 240, c[2 * i + 1].shape), dtype=U8))
    order = rng.permutation(blocks)
    table = np.full((len(lens), max(max(pages), 1) + 1), 10 ** 9)
    at = 0
    for r, p in enumerate(pages):
        table[r, :p] = order[at:at + p]
        at += p
    skip = 2                                     # rows before the first request
    starts = np.concatenate([[0], np.cumsum(lens)]) + skip
    rows = int(starts[-1]) + 3                   # and behind the last
    wide = torch.full((rows, nkv * hd + 8), 7.5, dtype=BF16, device="cuda")
    ko, vo = wide[:, :nkv * hd], torch.full((rows, nkv * hd), 7.5, dtype=BF16, device="cuda")
    scs().sc_paged_cache_read_fp8(*c, ko, vo, i32(table)[:, :table.shape[1] - 1], i32(starts),
                                  None if first is None else i32(first))
    for i, out in ((0, ko), (2, vo)):
        vals = dequantise(c[i], c[i + 1]).flatten(2)
        got = out.cpu()
        for r, n in enumerate(lens):
            t = np.arange(n) + begin[r]
            want = vals[table[r, t // block], t % block] if n else torch.zeros(0, nkv * hd, dtype=F64)
            assert torch.equal(got[starts[r]:starts[r + 1]].to(F64), want)
        assert bool((got[:skip] == 7.5).all()) and bool((got[starts[-1]:] == 7.5).all())
    assert bool((wide[:, nkv * hd:] == 7.5).all())


def test_read_of_what_is_not_there():
    """Blocks outside the cache, tokens before the first and behind the table: zeros."""
    print("[gpu] read outside", flush=True)
    c = caches_fp8("tokens", 3, 16, 1, 64, 0x38, 127)          # all ones
    table = i32([[0, -1, 3], [2, 2 ** 31 - 1, 1]])
    ko, vo = (torch.full((120, 64), 7.5, dtype=BF16, device="cuda") for _ in range(2))
    scs().sc_paged_cache_read_fp8(*c, ko, vo, table, i32([0, 60, 110]), i32([0, -3]))
    want = torch.full((120,), 7.5)
    want[:60] = 0
    want[:16] = 1
    want[60:110] = 0
    want[63:79] = 1                                            # tokens 0..15 of the second
    want[95:110] = 1                                           # tokens 32..46
    for out in (ko, vo):
        assert bool((out.float().cpu() == want[:, None]).all())


def test_read_past_four_gigabytes():
    nkv, hd, block, blocks = 2, 128, 16, 1_100_000             # 4.5e9 codes
    print("[gpu] far quantised rows", flush=True)
    cache = torch.empty(blocks, block, nkv, hd, dtype=U8, device="cuda")
    scale = torch.empty(blocks, nkv, block, dtype=U8, device="cuda")
    T, first = 33, (blocks - 3) * block
    g = torch.Generator().manual_seed(3)
    v = randn(g, T, nkv * hd)
    q = randn(g, T, 4 * hd)
    S = scs()
    other = [torch.zeros(3, block, nkv, hd, dtype=U8, device="cuda").as_strided(
                 cache.shape, (0, nkv * hd, hd, 1)).view(E4M3),
             torch.zeros(nkv, block, dtype=U8, device="cuda").as_strided(scale.shape, (0, block, 1))]
    S.sc_qk_norm_rope_fp8(q.cuda(), v.cuda(), v.cuda(), torch.empty(T, 4 * hd, dtype=BF16, device="cuda"), None,
                          None, None, None, None, i64(first + np.arange(T)), *other,
                          cache.view(E4M3), scale, head_dim=hd)
    codes, byte = quantise(v.view(T, nkv, hd))
    assert torch.equal(cache.view(-1, nkv, hd)[first:first + T].cpu(), codes)
    ko, vo = (torch.empty(T, nkv * hd, dtype=BF16, device="cuda") for _ in range(2))
    table = i32([[blocks - 3, blocks - 2, blocks - 1]])
    S.sc_paged_cache_read_fp8(*other, cache.view(E4M3), scale, ko, vo, table, i32([0, T]))
    want = CODES[codes.long()] * torch.pow(torch.tensor(2.0, dtype=F64), byte.to(F64) - 127)[..., None]
    assert torch.equal(vo.cpu().to(F64), want.flatten(1))
