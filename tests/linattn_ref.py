"""Plain 64-bit forms of the linear attention with decay and of the 8-bit
state cache, and the tolerances of the tests that use them (not collected by
pytest)."""

from __future__ import annotations

from typing import Optional, Sequence

import torch

STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative to the value


def scan(q, k, v, g, lens: Sequence[int], *, scale=1.0, init: Optional[torch.Tensor] = None, start: int = 0):
    """Token by token, S = exp(g) S + v k^T, o = scale S q, in float64 on the
    inputs' device, all sequences one token a step. Returns out [T, hv, dv]
    (zeros outside the sequences), the final states, and the same two sums
    with every factor replaced by its magnitude: what rounding errors are
    measured against."""
    T, hk, dk = q.shape
    hv, dv = v.shape[1], v.shape[2]
    dev, G, N = q.device, hv // hk, len(lens)
    q, k = (x.double().repeat_interleave(G, 1) for x in (q, k))
    v, a = v.double(), g.double().exp().expand(T, hv)
    L = torch.tensor(list(lens), device=dev)
    first = start + torch.cat([L.new_zeros(1), L.cumsum(0)[:-1]])
    S = torch.zeros(N, hv, dv, dk, dtype=torch.float64, device=dev)
    if init is not None:
        S += init.double()
    A = S.abs()
    out = torch.zeros(T + 1, hv, dv, dtype=torch.float64, device=dev)
    mag = torch.zeros_like(out)
    for t in range(max(lens, default=0)):
        on = t < L
        at = torch.where(on, first + t, 0)
        decay = torch.where(on[:, None], a[at], 1.0)[..., None, None]
        vt, kt, qt = torch.where(on[:, None, None], v[at], 0.0), k[at], q[at]
        # a token that is not there must not bring a NaN in
        kt = torch.where(on[:, None, None], kt, 0.0)
        S = decay * S + vt[..., None] * kt[..., None, :]
        A = decay * A + vt.abs()[..., None] * kt.abs()[..., None, :]
        to = torch.where(on, at, T)
        out[to] = scale * (S * qt[..., None, :]).sum(-1)
        mag[to] = abs(scale) * (A * qt.abs()[..., None, :]).sum(-1)
    out[T] = 0
    return out[:T], S, mag[:T], A


def prefill_bounds(out, S, mag, A, io, state, tokens: int, dk: int):
    """Per-element error bounds. fp32 sums: an addition or a product is off by
    at most 2^-24 of the magnitudes it combines; a term passes one addition
    per token of its sequence for the state, and for the output the state's
    dk products, or the key-query product's dk and the 64 of its block; the
    decays add their exponent's rounding, relative size x 2^-24 for exp(-x),
    x up to 104 before it underflows, and a few roundings of their own. With
    bf16 I/O every term of an output is rounded to bf16 once more inside, as
    part of the state or of a key-query score. At last the stored type."""
    ops = (tokens + 2 * dk + 64 + 104 + 32) * 2.0 ** -24
    tol_out = STEP[io] * out.abs() + (ops + (1.01 * STEP[io] if io == torch.bfloat16 else 0.0)) * mag + 1e-30
    tol_S = (STEP[state] * S.abs() if state == torch.bfloat16 else 0.0) + ops * A + 1e-30
    return tol_out, tol_S


def check(got, want, tol, what):
    """Every element within its bound; names the worst."""
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = ((got - want).abs() / tol).flatten()
    worst = int(over.argmax()) if over.numel() else 0
    assert not over.numel() or over[worst] <= 1.0, \
        f"{what}: element {worst} off by {float(over[worst]):.3g} times its bound " \
        f"({float(got.flatten()[worst])} for {float(want.flatten()[worst])})"


# ------------------------------------------------------------- 8-bit codes

def _nearest(y, values):
    """Index into the sorted `values` (their codes) of the nearest, ties to the even code."""
    hi = torch.searchsorted(values, y).clamp(1, len(values) - 1)
    lo = hi - 1
    d_lo, d_hi = y - values[lo], values[hi] - y
    pick_hi = (d_hi < d_lo) | ((d_hi == d_lo) & (hi % 2 == 0))
    return torch.where(pick_hi, hi, lo)


def quantise(x, code: torch.dtype):
    """(codes as values, scale) of states x [..., dk], from the exact quotients
    (64 bits separate a quotient of two fp32 numbers from a middle between
    codes: it differs by 2^-48 of it at least)."""
    x = x.double()
    top = 127.0 if code == torch.int8 else 448.0
    values = torch.arange(128.0, dtype=torch.float64) if code == torch.int8 else \
        torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    values = values.to(x.device)
    fine = torch.isfinite(x).all(-1)
    scale = (torch.where(fine[..., None], x, 0.0).abs().amax(-1) / top).float()
    scale = torch.where(torch.isinf(scale * top), torch.nextafter(scale, torch.zeros_like(scale)), scale)
    y = torch.where((scale > 0)[..., None] & fine[..., None], x.abs() / scale.double()[..., None], 0.0)
    codes = values[_nearest(y.clamp(max=top), values)] * torch.where(y > 0, x.sign(), 1.0)
    return codes, torch.where(fine, scale, float("nan"))
