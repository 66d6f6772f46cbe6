"""Inputs and error bounds of the served forms' tests (tests/test_gpu_served*.py).

Bounds count roundings: u = 2^-24 is half a float32 step.  Outputs written as bf16 add half a
bf16 step, 2^-8 of the value.
"""
import numpy as np
import torch

import ssd_inputs
from oracle import glue, served

U = 2.0 ** -24
BF16 = {"f32": 0.0, "bf16": 2.0 ** -8}


def store(a, io):
    """float64 values as the bits the kernel and the oracle both read."""
    return ssd_inputs.f32_to_bf16_bits(a) if io == "bf16" else a.astype(np.float32)


def up(a, io="f32"):
    t = torch.from_numpy(np.ascontiguousarray(a))
    if io == "bf16":
        t = t.view(torch.bfloat16)
    return t.cuda()


def up_rows(a, io="f32", pad=0, shift=0):
    """The tensor as columns of a wider one: rows `pad` elements apart, `shift` elements in."""
    rows = a.shape[0]
    width = int(np.prod(a.shape[1:]))
    big = torch.full((rows, width + pad + shift), 3.0, device="cuda",
                     dtype=torch.bfloat16 if io == "bf16" else torch.float32)
    view = big[:, shift:shift + width]
    view.copy_(up(a, io).reshape(rows, width))
    return view.unflatten(1, a.shape[1:]) if a.ndim > 2 else view


def down(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def excess(got, ref, bound):
    """How far the worst element lies past its bound (<= 0: all within), NaN never within."""
    d = np.abs(got - ref) - bound
    return float(np.max(np.where(np.isnan(d), np.inf, d))) if d.size else 0.0


def silu_bound(v, dv):
    """Error of silu(v) computed in float32 from v with error dv: |silu'| <= 1.1; e^-v carries
    (|v| + 4) steps of its own value, which silu passes on at most in full, and the sum, the
    division and the product 4 more."""
    return 1.1 * dv + (np.abs(v) + 8) * 2 * U * np.abs(glue.silu(v))


def conv_bound(u, w, bias, cu, state, slots, resume, io):
    """K products and K additions, each off by at most u of the running magnitude."""
    K = w.shape[1]
    mag, _ = _conv_linear(np.abs(glue._f64(u)), np.abs(w), None if bias is None else
                          np.abs(bias), cu, None if state is None else np.abs(glue._f64(state)),
                          slots, resume)
    lin, _ = _conv_linear(u, w, bias, cu, state, slots, resume)
    b = silu_bound(lin, (K + 1) * U * mag)
    return b + BF16[io] * (np.abs(glue.silu(lin)) + b)


def _conv_linear(u, w, bias, cu, state, slots, resume):
    """The convolution before its SiLU, through the oracle's walk."""
    keep = served.silu
    served.silu = lambda v: v
    try:
        return served.conv_silu(u, w, bias, cu, state, slots, resume)
    finally:
        served.silu = keep


def scan_bound(inp, ref, y_io):
    """A state is a sum of terms, each multiplied once per later token by a decay whose relative
    error is at most (2 |dt A| + 6) u (the rate's, the product's and the exponential's
    roundings), and rounded once more by the update: 8 u + 2 |dt A| u a step.  A term alive for m
    steps has the weight e^(-m s), s = dt |A|, so that sum m e^(-m s) / sum e^(-m s) <= 1 / s + 1
    steps count: (8 + 2 s) (1 / s + 1) + 24 (the term's own products, the softplus, the sum over
    the states, D x), relative to the sum of magnitudes."""
    args = dict(inp)
    dt = glue._f64(args["dt"])
    if args.get("dt_bias") is not None:
        dt = dt + args["dt_bias"]
    if args.get("use_softplus"):
        dt = glue.softplus(dt)
    s = max(float(np.min(np.abs(args["A"])) * np.min(dt)), 1e-3)
    s1 = float(np.max(np.abs(args["A"])) * np.max(dt))
    steps = (8 + 2 * min(s1, 20.0)) * (1 / s + 1) + 24 + args["A"].shape[1]
    z = args.pop("z", None)
    for k in ("x", "B", "C", "D", "state"):
        if args.get(k) is not None:
            args[k] = np.abs(glue._f64(args[k]))
    mag, hmag = served.selective_scan(**args)
    if z is not None:
        zv = glue._f64(z)
        mag = mag * np.abs(glue.silu(zv)) * (1 + (np.abs(zv) + 8) * 2 * U)
        steps = steps + 2 * float(np.max(np.abs(zv))) + 8
    by = steps * U * mag
    by = by + BF16[y_io] * (np.abs(ref[0]) + by)
    return by, None if hmag is None else steps * U * hmag
