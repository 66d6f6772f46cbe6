"""Float64 definitions of a Mamba block's served forms and its norm -- TEST INFRASTRUCTURE (only
``tests/``, ``__graft_entry__.smoke()`` and ``bench.py`` may use it).

The convolution and the selective scan over a packed batch of sequences with a cache ("State Space
Models (SSM)" (ultralytics.com glossary), sections "Come funzionano gli SSM" and "Da S4 a Mamba";
"Architektury Mamba-2, State Space Models i liniowa atencja" (tech.tersel.eu), "Od S4 do Mamba-1"),
sequence by sequence and token by token; the group norm with a SiLU gate and its gradients.
A single token of each sequence is a packed batch of sequences of length one that resume.
Pinned in ``tests/test_oracle_served.py``.
"""
import numpy as np

from .glue import _f64, silu, softplus


def _owned(slots, nslots):
    """The slot of each sequence, or None where it is left alone: negative, past the cache, or
    named by an earlier sequence."""
    seen, out = set(), []
    for s in slots:
        s = int(s)
        ok = 0 <= s < nslots and s not in seen
        if s >= 0:
            seen.add(s)
        out.append(s if ok else None)
    return out


def conv_silu(u, w, bias, cu, state=None, slots=None, resume=None, out=None):
    """u [T, C], w [C, K], bias [C] or None, cu [n + 1]; state [nslots, K-1, C] -> (out, state),
    float64.  Rows that no sequence covers keep the values of ``out`` (zeros by default)."""
    u, w = _f64(u), _f64(w)
    K, n = w.shape[1], len(cu) - 1
    b = np.zeros(u.shape[1]) if bias is None else _f64(bias)
    out = np.zeros_like(u) if out is None else _f64(out).copy()
    state = None if state is None else _f64(state).copy()
    slots = list(range(n)) if slots is None else list(slots)
    owned = _owned(slots, n if state is None else len(state))
    for i in range(n):
        if owned[i] is None:
            continue
        hist = np.zeros((K - 1, u.shape[1]))
        if state is not None and resume is not None and resume[i]:
            hist = state[owned[i]]
        v = np.concatenate([hist, u[cu[i]:cu[i + 1]]])
        for t in range(cu[i + 1] - cu[i]):
            out[cu[i] + t] = silu(b + np.sum(w.T * v[t:t + K], axis=0))
        if state is not None:
            state[owned[i]] = v[len(v) - (K - 1):]
    return out, state


def selective_scan(x, dt, A, B, C, cu, D=None, z=None, dt_bias=None, use_softplus=False,
                   state=None, slots=None, resume=None, out=None):
    """x, dt, z [T, dim]; A [dim, N]; B, C [T, G, N]; D, dt_bias [dim]; state [nslots, dim, N]
    -> (y, state), float64; rows that no sequence covers keep the values of ``out``."""
    x, dt, A, B, C = map(_f64, (x, dt, A, B, C))
    dim, N = A.shape
    per = dim // B.shape[1]
    n = len(cu) - 1
    if dt_bias is not None:
        dt = dt + _f64(dt_bias)
    if use_softplus:
        dt = softplus(dt)
    gate = 1.0 if z is None else silu(z)
    Dv = np.zeros(dim) if D is None else _f64(D)
    y = np.zeros_like(x) if out is None else _f64(out).copy()
    state = None if state is None else _f64(state).copy()
    slots = list(range(n)) if slots is None else list(slots)
    owned = _owned(slots, n if state is None else len(state))
    for i in range(n):
        if owned[i] is None:
            continue
        h = np.zeros((dim, N))
        if state is not None and resume is not None and resume[i]:
            h = state[owned[i]]
        for t in range(cu[i], cu[i + 1]):
            Bt, Ct = np.repeat(B[t], per, 0), np.repeat(C[t], per, 0)
            h = np.exp(dt[t][:, None] * A) * h + (dt[t] * x[t])[:, None] * Bt
            v = np.sum(Ct * h, axis=1) + Dv * x[t]
            y[t] = v if z is None else v * gate[t]
        if state is not None:
            state[owned[i]] = h
    return y, state


def group_norm(y, w, b=None, z=None, ngroups=1, eps=1e-5, center=False, gate_first=True):
    """y, z [rows, C]; w, b [C] -> dict(out, n, v, rstd, mean), float64 [rows, C] each."""
    y, w = _f64(y), _f64(w)
    rows, C = y.shape
    g = 1.0 if z is None else silu(z)
    v = (y * g if gate_first else y).reshape(rows, ngroups, C // ngroups)
    mean = np.mean(v, -1, keepdims=True) if center else np.zeros((rows, ngroups, 1))
    rstd = 1.0 / np.sqrt(np.mean((v - mean) ** 2, -1, keepdims=True) + eps)
    n = ((v - mean) * rstd).reshape(rows, C)
    out = n * w + (0.0 if b is None else _f64(b))
    if not gate_first:
        out = out * g
    full = lambda a: np.broadcast_to(a, v.shape).reshape(rows, C)  # noqa: E731
    return dict(out=out, n=n, v=v.reshape(rows, C), rstd=full(rstd), mean=full(mean))


def group_norm_backward(dout, y, w, b=None, z=None, ngroups=1, eps=1e-5, center=False,
                        gate_first=True):
    """Gradients of sum(dout * out): dict(y, z, weight, bias), and ``scale``: for y the sum of the
    magnitudes that cancel in it (what its rounding error is relative to)."""
    dout, w = _f64(dout), _f64(w)
    f = group_norm(y, w, b, z, ngroups, eps, center, gate_first)
    yv, n, rstd = _f64(y), f["n"], f["rstd"]
    rows, C = yv.shape
    grp = lambda a: a.reshape(rows, ngroups, C // ngroups)  # noqa: E731
    mean = lambda a: np.broadcast_to(np.mean(grp(a), -1, keepdims=True),  # noqa: E731
                                     (rows, ngroups, C // ngroups)).reshape(rows, C)
    gate = np.ones_like(yv) if z is None else silu(z)
    if z is not None:
        zv = _f64(z)
        sg = 1.0 / (1.0 + np.exp(-zv))
        slope = sg * (1.0 + zv * (1.0 - sg))
    do = dout if gate_first else dout * gate
    dn = do * w
    dv = rstd * (dn - (mean(dn) if center else 0.0) - n * mean(dn * n))
    mag = rstd * (np.abs(dn) + (mean(np.abs(dn)) if center else 0.0) +
                  (np.abs(n) + np.abs(f["mean"]) * rstd) * mean(np.abs(dn * n)))
    dz = None
    if z is not None:
        dz = dv * yv * slope if gate_first else \
            dout * (n * w + (0.0 if b is None else _f64(b))) * slope
    first = z is not None and gate_first
    return dict(y=dv * gate if first else dv, z=dz, weight=np.sum(do * n, 0),
                bias=None if b is None else np.sum(do, 0),
                scale=mag * (np.abs(gate) if first else 1.0), mag=mag,
                weight_scale=np.sum(np.abs(do) * (np.abs(n) + np.abs(f["mean"]) * rstd), 0),
                bias_scale=np.sum(np.abs(do), 0), slope=None if z is None else slope)
