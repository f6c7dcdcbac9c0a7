"""The gated delta rule in 64 bits on the CPU, token by token, and the error
bounds of its tests."""
from __future__ import annotations

import math

import torch

F64 = torch.float64
EPS = 1e-6


def make(hk, hv, dk, dv, rows, slots, *, gates="bf16", seed=0, pad=0, strong=False):
    """Inputs on the CPU, with q, k and v as column blocks of one tensor of rows
    `pad` values wider than they are. strong: decays from none to total."""
    g = torch.Generator().manual_seed(seed)
    kw, vw = hk * dk, hv * dv
    mixed = torch.randn(rows, 2 * kw + vw + pad, generator=g)
    mixed = (mixed * torch.sigmoid(mixed)).bfloat16()
    gt = torch.float32 if gates == "f32" else torch.bfloat16
    a = torch.randn(rows, hv, generator=g)
    if strong:
        a = a * 8
    return {"mixed": mixed, "kw": kw, "vw": vw, "a": a.to(gt),
            "b": torch.randn(rows, hv, generator=g).to(gt),
            "A_log": torch.rand(hv, generator=g) * 2.7,
            "dt_bias": torch.rand(hv, generator=g) * 5 - 7,
            "pool": torch.randn(slots, hv, dv, dk, generator=g) * 0.3}


def parts(mixed, c):
    kw, vw = c["kw"], c["vw"]
    return mixed[:, :kw], mixed[:, kw:2 * kw], mixed[:, 2 * kw:2 * kw + vw]


def reference(c, rows, S, scale, l2norm=True):
    """Token rows `rows` from state S (HV, DV, DK; 64 bits). Returns (out, the
    states after each token, bound on |out| by Cauchy-Schwarz)."""
    hv, dv, dk = c["pool"].shape[1:]
    hk = c["kw"] // dk
    q, k, v = (x.to(F64) for x in parts(c["mixed"], c))
    outs, states, bounds = [], [], []
    for t in rows:
        qt, kt = (x[t].view(hk, dk).repeat_interleave(hv // hk, 0) for x in (q, k))
        if l2norm:
            qt = qt / torch.sqrt((qt * qt).sum(1, keepdim=True) + EPS)
            kt = kt / torch.sqrt((kt * kt).sum(1, keepdim=True) + EPS)
        x = c["a"][t].to(F64) + c["dt_bias"].to(F64)
        g = -torch.exp(c["A_log"].to(F64)) * torch.logaddexp(x, torch.zeros_like(x))
        beta = torch.sigmoid(c["b"][t].to(F64))
        S = S * torch.exp(g)[:, None, None]
        u = beta[:, None] * (v[t].view(hv, dv) - (S * kt[:, None]).sum(2))
        S = S + u[..., None] * kt[:, None]
        outs.append(scale * (S * qt[:, None]).sum(2))
        bounds.append(scale * S.norm(dim=2) * qt.norm(dim=1, keepdim=True))
        states.append(S)
    return outs, states, bounds


def check_out(got, want, bound, n, dk, what=""):
    """got (bf16 values) against want, both (tokens, heads, dv). One bf16
    rounding is half a step, 2^-8 of the value. Before it: a sum of dk products
    rounds by sqrt(dk) 2^-24 of its bound, once for each of the n tokens whose
    errors the state carries (the update never grows an error: decay and
    I - beta k k^T have norm at most 1), taken four times for the tail of the
    distribution, and the two-part products of a chunk leave 2^-16 of their
    terms' sum, which is at most 8 (the root of 64 terms) bounds."""
    tol = 2.0 ** -8 * want.abs() + (4 * math.sqrt(n * dk) * 2.0 ** -24 + 2.0 ** -13) * bound
    bad = (got.to(F64) - want).abs() > tol
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} values off, the " \
        f"worst by {float(((got.to(F64) - want).abs() / tol).max()):.2f} tolerances"


def check_state(got, want, n, dk, scale_of, what=""):
    """fp32 states: sqrt(n dk) 2^-24 as above, for the two sums of a token and
    four times for the tail, of the largest row norm that the state had."""
    tol = 8 * math.sqrt(max(n, 1) * dk) * 2.0 ** -24 * scale_of
    err = float((got.to(F64) - want).abs().max())
    assert err <= tol, f"{what}: state off by {err:.3g}, tolerance {tol:.3g}"
