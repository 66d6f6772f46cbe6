"""The serving and training operators of a Mamba block, as cases to measure: the short causal
convolution and the selective scan for packed prompts and for single tokens (with the caches they
keep), and the group norm with its SiLU gate, forward and backward.

``own`` chooses what ``run`` computes: False the operators in plain torch operations, True the
framework's calls.
"""
import math

import numpy as np
import torch

own = False

IO = {"bf16": torch.bfloat16, "f32": torch.float32}
SLOTS_PER_SEQ = 2   # a cache has room for more sequences than one call serves


def listed():
    return [
        # A batch of ragged prompts through the 2.7B layer's convolution (x, B and C channels);
        # some continue a prompt whose first part was served before.
        dict(name="conv prompts 16x, 5376 ch", op="conv_prompt", T=32768, S=16, C=5376, K=4,
             io="bf16", resume=True),
        # Short float32 prompts on an odd width, as small models and tests run them.
        dict(name="conv prompts 7x, 1537 ch f32", op="conv_prompt", T=1003, S=7, C=1537, K=3,
             io="f32", resume=True),
        # One token of one sequence: pure latency.
        dict(name="conv token 1x, 5376 ch", op="conv_token", S=1, C=5376, K=4, io="bf16"),
        # The decode batch of the layer: 256 sequences.
        dict(name="conv token 256x, 5376 ch", op="conv_token", S=256, C=5376, K=4, io="bf16"),
        # Four long ragged prompts at the 2.7B layer's width.
        dict(name="scan prompts 4x, 5120 ch", op="scan_prompt", T=16384, S=4, dim=5120, N=16, G=1,
             io="bf16", dt="f32", y="f32", gate=True, resume=False),
        # One long prompt at the 130M layer's width: few channels, many tokens.
        dict(name="scan prompt 1x, 1536 ch", op="scan_prompt", T=16384, S=1, dim=1536, N=16, G=1,
             io="bf16", dt="bf16", y="bf16", gate=True, resume=False),
        # Many short float32 continuations, B and C in two groups, no gate.
        dict(name="scan prompts 33x, 1536 ch f32", op="scan_prompt", T=2111, S=33, dim=1536, N=16,
             G=2, io="f32", dt="f32", y="f32", gate=False, resume=True),
        # One token of one sequence, then the decode batch.
        dict(name="scan token 1x, 5120 ch", op="scan_token", S=1, dim=5120, N=16, G=1, io="bf16",
             dt="bf16", y="bf16", gate=True),
        dict(name="scan token 256x, 5120 ch", op="scan_token", S=256, dim=5120, N=16, G=1,
             io="bf16", dt="f32", y="f32", gate=True),
        # The norm over a decode batch, eight groups.
        dict(name="norm 256 rows, 5120 ch", op="norm", T=256, C=5120, G=8, io="bf16", y="f32",
             out="bf16", center=False, gate="first", bias=False),
        # The norm over a training batch's tokens (float32 y as the scan writes it).
        dict(name="norm 16384 rows, 5120 ch", op="norm", T=16384, C=5120, G=1, io="bf16", y="f32",
             out="bf16", center=False, gate="first", bias=False),
        # Its gradients.
        dict(name="norm grad 16384 rows, 5120 ch", op="norm_grad", T=16384, C=5120, G=1,
             io="bf16", y="f32", out="bf16", center=False, gate="first", bias=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_prompt", "conv_token", "scan_prompt", "scan_token", "norm",
                     "norm_grad"])
    io = rng.choice(["bf16", "bf16", "f32"])
    other = lambda: rng.choice(["bf16", "f32"]) if io == "bf16" else "f32"  # noqa: E731
    if op == "conv_prompt":
        T = _log(rng, 64, 16384)
        return dict(op=op, T=T, S=min(T, _log(rng, 1, 64)), C=_log(rng, 64, 5376),
                    K=rng.choice([2, 3, 4, 4, 4, 8]), io=io, resume=rng.random() < 0.5)
    if op == "conv_token":
        return dict(op=op, S=_log(rng, 1, 512), C=_log(rng, 64, 5376),
                    K=rng.choice([2, 3, 4, 4, 4, 8]), io=io)
    if op == "scan_prompt":
        T = _log(rng, 64, 8192)
        G = rng.choice([1, 1, 2])
        return dict(op=op, T=T, S=min(T, _log(rng, 1, 64)), dim=G * _log(rng, 64, 5120 // G),
                    N=rng.choice([8, 16, 16, 16]), G=G, io=io, dt=other(), y=other(),
                    gate=rng.random() < 0.7, resume=rng.random() < 0.5)
    if op == "scan_token":
        G = rng.choice([1, 1, 2])
        return dict(op=op, S=_log(rng, 1, 512), dim=G * _log(rng, 64, 5120 // G),
                    N=rng.choice([8, 16, 16, 16]), G=G, io=io, dt=other(), y=other(),
                    gate=rng.random() < 0.7)
    G = rng.choice([1, 1, 2, 5, 8])
    return dict(op=op, T=_log(rng, 16, 8192), C=G * _log(rng, 16, 5120 // G), G=G, io=io,
                y=other(), out=other(), center=rng.random() < 0.3,
                gate=rng.choice(["first", "first", "last", "none"]), bias=rng.random() < 0.3)


# ---- inputs ----------------------------------------------------------------------------------

def _lengths(case, seed):
    """S lengths of at least one token that add up to T: ragged, as prompts are."""
    S, T = case["S"], case["T"]
    w = np.random.RandomState(seed % (1 << 31)).lognormal(0.0, 0.7, S)
    n = 1 + np.floor((T - S) * w / w.sum()).astype(np.int64)
    n[: T - int(n.sum())] += 1
    return [int(v) for v in n]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    op, io = case["op"], IO[case["io"]]

    def randn(*shape, dtype=torch.float32, scale=1.0, shift=0.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale + shift).to(dtype)

    s = {"case": dict(case)}
    if op in ("conv_prompt", "scan_prompt"):
        lens = _lengths(case, seed)
        s["max_seqlen"] = max(lens)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        s["resume"] = torch.tensor([case["resume"] and i % 2 == 0 for i in range(case["S"])],
                                   dtype=torch.bool, device=dev)
    if op in ("conv_prompt", "conv_token", "scan_prompt", "scan_token"):
        nslots = SLOTS_PER_SEQ * case["S"]
        s["slots"] = torch.randperm(nslots, generator=gen, device=dev)[: case["S"]].to(torch.int32)
    if op.startswith("conv"):
        C, K = case["C"], case["K"]
        rows = case["T"] if op == "conv_prompt" else case["S"]
        s["u"] = randn(rows, C, dtype=io)
        s["w"] = randn(C, K, scale=K ** -0.5)
        s["bias"] = randn(C, scale=0.1)
        s["history"] = randn(nslots, K - 1, C, dtype=io)
    elif op.startswith("scan"):
        dim, N, G = case["dim"], case["N"], case["G"]
        rows = case["T"] if op == "scan_prompt" else case["S"]
        s["x"] = randn(rows, dim, dtype=io)
        s["raw"] = randn(rows, dim, dtype=IO[case["dt"]], scale=0.5)
        s["dt_bias"] = torch.full((dim,), -2.0, device=dev) + randn(dim, scale=0.1)
        s["A"] = -torch.exp(torch.rand(dim, N, generator=gen, device=dev) * math.log(16.0))
        # B and C as they leave one projection, side by side
        bc = randn(rows, 2 * G * N, dtype=io, scale=N ** -0.5)
        s["B"] = bc[:, : G * N].unflatten(1, (G, N))
        s["C"] = bc[:, G * N:].unflatten(1, (G, N))
        s["D"] = randn(dim)
        s["z"] = randn(rows, dim, dtype=io) if case["gate"] else None
        s["state"] = randn(nslots, dim, N, scale=0.1)
    else:
        T, C = case["T"], case["C"]
        s["y"] = randn(T, C, dtype=IO[case["y"]])
        s["z"] = randn(T, C, dtype=io) if case["gate"] != "none" else None
        s["w"] = randn(C, scale=0.1, shift=1.0)
        s["b"] = randn(C, scale=0.1) if case["bias"] else None
        if op == "norm_grad":
            s["dout"] = randn(T, C, dtype=IO[case["out"]])
    return s


# ---- the operators, plain and the framework's ---------------------------------------------------

def run(s):
    return {"conv_prompt": _conv_prompt, "conv_token": _conv_token, "scan_prompt": _scan_prompt,
            "scan_token": _scan_token, "norm": _norm, "norm_grad": _norm_grad}[s["case"]["op"]](s)


def _silu(v):
    return v / (1 + torch.exp(-v))


def _softplus(v):
    return torch.clamp_min(v, 0) + torch.log1p(torch.exp(-torch.abs(v)))


def _seq_of(cu, T):
    """The sequence that each of T packed rows belongs to."""
    t = torch.arange(T, device=cu.device)
    return t, (t[:, None] >= cu[None, 1:]).sum(1)


def _conv_prompt(s):
    if own:
        import mamba_ssd_scan_03_b200 as ssd
        out = ssd.conv_silu_varlen(s["u"], s["w"], s["cu"], s["bias"], conv_state=s["history"],
                                   slots=s["slots"], resume=s["resume"])
        return {"out": out, "history": s["history"]}
    u, w, K = s["u"].float(), s["w"], s["case"]["K"]
    T, C = u.shape
    slots, cu = s["slots"].long(), s["cu"].long()
    hist = s["history"][slots].float() * s["resume"][:, None, None]  # [S, K-1, C]
    rows = torch.cat([hist.flatten(0, 1), u])                        # histories, then the tokens
    S = cu.numel() - 1
    t, seq = _seq_of(cu, T)
    k = torch.arange(K, device=u.device)
    # position within the sequence of each tap; negative positions are history rows
    pos = (t - cu[seq])[:, None] - (K - 1) + k
    at = torch.where(pos >= 0, S * (K - 1) + cu[seq][:, None] + pos,
                     seq[:, None] * (K - 1) + (K - 1) + pos)
    out = _silu((rows[at] * w.t()).sum(1) + s["bias"])
    # the last K - 1 rows of history and sequence together
    pos = (cu[1:] - cu[:-1])[:, None] - (K - 1) + torch.arange(K - 1, device=u.device)
    i = torch.arange(S, device=u.device)[:, None]
    at = torch.where(pos >= 0, S * (K - 1) + cu[:-1, None] + pos, i * (K - 1) + (K - 1) + pos)
    s["history"][slots] = rows[at].to(s["history"].dtype)
    return {"out": out.to(s["u"].dtype), "history": s["history"]}


def _conv_token(s):
    if own:
        import mamba_ssd_scan_03_b200 as ssd
        out = ssd.conv_silu_step(s["history"], s["u"], s["w"], s["bias"], slots=s["slots"])
        return {"out": out, "history": s["history"]}
    slots = s["slots"].long()
    win = torch.cat([s["history"][slots], s["u"][:, None]], 1)       # [S, K, C]
    out = _silu((win.float() * s["w"].t()).sum(1) + s["bias"])
    s["history"][slots] = win[:, 1:]
    return {"out": out.to(s["u"].dtype), "history": s["history"]}


def _scan_prompt(s):
    c = s["case"]
    if own:
        import mamba_ssd_scan_03_b200 as ssd
        y = ssd.selective_scan_varlen(
            s["x"], s["raw"], s["A"], s["B"], s["C"], s["cu"], D=s["D"], z=s["z"],
            dt_bias=s["dt_bias"], softplus=True, state=s["state"], slots=s["slots"],
            resume=s["resume"], y_dtype=IO[c["y"]], max_seqlen=s["max_seqlen"])
        return {"y": y, "state": s["state"]}
    G, N, dim = c["G"], c["N"], c["dim"]
    x, cu, slots = s["x"].float(), s["cu"].long(), s["slots"].long()
    T = x.shape[0]
    dt = _softplus(s["raw"].float() + s["dt_bias"])
    a = torch.exp(dt[:, :, None] * s["A"])                           # [T, dim, N]
    h = ((dt * x).view(T, G, dim // G, 1) * s["B"].float()[:, :, None, :]).view(T, dim, N)
    first = cu[:-1]
    h[first] += a[first] * s["state"][slots] * s["resume"][:, None, None]
    a[first] = 0                                                     # nothing crosses into a sequence
    # two neighbouring runs of steps (a1, h1), (a2, h2) are one step (a1 a2, a2 h1 + h2): runs of
    # doubling length cover the longest sequence in log2 of it many rounds
    n = 1
    while n < s["max_seqlen"]:
        h[n:] += a[n:] * h[:-n]
        a[n:] = a[n:] * a[:-n]
        n *= 2
    y = (h.view(T, G, dim // G, N) * s["C"].float()[:, :, None, :]).sum(-1).view(T, dim)
    y = y + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["state"][slots] = h[cu[1:] - 1]
    return {"y": y.to(IO[c["y"]]), "state": s["state"]}


def _scan_token(s):
    c = s["case"]
    if own:
        import mamba_ssd_scan_03_b200 as ssd
        y = ssd.selective_step(s["state"], s["x"], s["raw"], s["A"], s["B"], s["C"], s["D"],
                               z=s["z"], dt_bias=s["dt_bias"], softplus=True, slots=s["slots"],
                               y_dtype=IO[c["y"]])
        return {"y": y, "state": s["state"]}
    G, N, dim, S = c["G"], c["N"], c["dim"], c["S"]
    x, slots = s["x"].float(), s["slots"].long()
    dt = _softplus(s["raw"].float() + s["dt_bias"])
    h = torch.exp(dt[:, :, None] * s["A"]) * s["state"][slots]
    h = h + ((dt * x).view(S, G, dim // G, 1) * s["B"].float()[:, :, None, :]).view(S, dim, N)
    y = (h.view(S, G, dim // G, N) * s["C"].float()[:, :, None, :]).sum(-1).view(S, dim)
    y = y + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["state"][slots] = h
    return {"y": y.to(IO[c["y"]]), "state": s["state"]}


EPS = 1e-5


def _normalised(s):
    """silu(z) (or None), the gated y in groups, its normalised form and 1 / deviation."""
    c = s["case"]
    y = s["y"].float()
    g = None if s["z"] is None else _silu(s["z"].float())
    v = y * g if c["gate"] == "first" else y
    v = v.view(c["T"], c["G"], -1)
    if c["center"]:
        v = v - v.mean(-1, keepdim=True)
    r = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)
    return y, g, v * r, r


def _norm(s):
    c = s["case"]
    if own:
        import mamba_ssd_scan_03_b200 as ssd
        return ssd.group_norm_gate(s["y"], s["w"], s["b"], s["z"], ngroups=c["G"], eps=EPS,
                                   center=c["center"], gate_first=c["gate"] == "first",
                                   out_dtype=IO[c["out"]])
    _, g, n, _ = _normalised(s)
    out = n.view(c["T"], c["C"]) * s["w"]
    if s["b"] is not None:
        out = out + s["b"]
    if c["gate"] == "last":
        out = out * g
    return out.to(IO[c["out"]])


def _norm_grad(s):
    c = s["case"]
    if own:
        import mamba_ssd_scan_03_b200 as ssd
        return ssd.group_norm_gate_bwd(s["dout"], s["y"], s["w"], s["b"], s["z"], ngroups=c["G"],
                                       eps=EPS, center=c["center"],
                                       gate_first=c["gate"] == "first")
    T, C, G = c["T"], c["C"], c["G"]
    y, g, n, r = _normalised(s)
    do = s["dout"].float()
    flat = n.view(T, C)
    dz = None
    if s["z"] is not None:
        sig = 1 / (1 + torch.exp(-s["z"].float()))
        slope = sig * (1 + s["z"].float() * (1 - sig))               # of silu
    if c["gate"] == "last":
        dz = do * (flat * s["w"] + (0 if s["b"] is None else s["b"])) * slope
        do = do * g
    dn = (do * s["w"]).view(T, G, -1)
    dv = dn - n * (dn * n).mean(-1, keepdim=True)
    if c["center"]:
        dv = dv - dn.mean(-1, keepdim=True)
    dv = (dv * r).view(T, C)
    dy = dv
    if c["gate"] == "first":
        dy = dv * g
        dz = dv * y * slope
    return {"y": dy, "z": None if dz is None else dz.to(s["z"].dtype),
            "weight": (do * flat).sum(0), "bias": None if s["b"] is None else do.sum(0)}


# ---- what a pass cannot do without -------------------------------------------------------------

def work(case):
    op = case["op"]
    es = 2 if case["io"] == "bf16" else 4
    size = lambda k: 2 if case[k] == "bf16" else 4  # noqa: E731
    if op.startswith("conv"):
        C, K, S = case["C"], case["K"], case["S"]
        rows = case["T"] if op == "conv_prompt" else S
        back = (S + 1) // 2 if op == "conv_prompt" and case["resume"] else 0
        read = S if op == "conv_token" else back
        return {"bytes": 2 * rows * C * es + (S + read) * (K - 1) * C * es + 4 * C * (K + 1),
                "flops": rows * C * (2 * K + 5)}
    if op.startswith("scan"):
        dim, N, G, S = case["dim"], case["N"], case["G"], case["S"]
        rows = case["T"] if op == "scan_prompt" else S
        back = (S + 1) // 2 if op == "scan_prompt" and case["resume"] else 0
        read = S if op == "scan_token" else back
        per = es + size("dt") + size("y") + (es if case["gate"] else 0)
        return {"bytes": rows * (dim * per + 2 * G * N * es) + (S + read) * dim * N * 4
                + 4 * dim * (N + 2),
                # per state: dt A, exp, a h + u B (3), C h (2); per channel: softplus, u, D x, gate
                "flops": rows * dim * (7 * N + 15)}
    T, C = case["T"], case["C"]
    per = size("y") + (es if case["gate"] != "none" else 0) + size("out")
    if op == "norm":
        return {"bytes": T * C * per + 4 * C * (1 + case["bias"]), "flops": 12 * T * C}
    per += 4 + (es if case["gate"] != "none" else 0)
    return {"bytes": T * C * per + 8 * C * (1 + case["bias"]), "flops": 30 * T * C}


# ---- the same from the definitions, in 64 bits ---------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v
         for k, v in s.items()}
    op = case["op"]
    if op == "conv_prompt":
        u, cu = d["u"], s["cu"].tolist()
        out, hist = torch.zeros_like(u), d["history"].clone()
        K = case["K"]
        for i, slot in enumerate(s["slots"].tolist()):
            before = d["history"][slot] if bool(s["resume"][i]) else 0 * d["history"][slot]
            seq = torch.cat([before, u[cu[i]:cu[i + 1]]])
            v = (seq.unfold(0, K, 1) * d["w"]).sum(-1) + d["bias"]
            out[cu[i]:cu[i + 1]] = v * torch.sigmoid(v)
            hist[slot] = seq[seq.shape[0] - (K - 1):]
        return {"out": out, "history": hist}
    if op == "conv_token":
        out, hist = torch.zeros_like(d["u"]), d["history"].clone()
        for i, slot in enumerate(s["slots"].tolist()):
            win = torch.cat([d["history"][slot], d["u"][i:i + 1]])
            v = (win.t() * d["w"]).sum(1) + d["bias"]
            out[i] = v * torch.sigmoid(v)
            hist[slot] = win[1:]
        return {"out": out, "history": hist}
    if op in ("scan_prompt", "scan_token"):
        if op == "scan_prompt":
            first, last = s["cu"][:-1].long(), s["cu"][1:].long()
            keep, longest = s["resume"].double(), s["max_seqlen"]
        else:
            first = torch.arange(case["S"], device="cuda")
            last, keep, longest = first + 1, torch.ones(case["S"], device="cuda").double(), 1
        per = case["dim"] // case["G"]
        h = d["state"][s["slots"].long()] * keep[:, None, None]
        y = torch.zeros_like(d["x"])
        for t in range(longest):  # every sequence's t-th token; those past their end stand still
            at = torch.minimum(first + t, last - 1)
            on = (first + t < last).double()[:, None]
            dt = torch.logaddexp(d["raw"][at] + d["dt_bias"], torch.zeros((), device="cuda")) * on
            B = d["B"][at].repeat_interleave(per, 1)
            C = d["C"][at].repeat_interleave(per, 1)
            h = torch.exp(dt[:, :, None] * d["A"]) * h + (dt * d["x"][at])[:, :, None] * B
            v = (C * h).sum(-1) + d["D"] * d["x"][at]
            if d["z"] is not None:
                v = v * d["z"][at] * torch.sigmoid(d["z"][at])
            y[at] = torch.where(on > 0, v, y[at])
        state = d["state"].clone()
        state[s["slots"].long()] = h
        return {"y": y, "state": state}
    y, w, z, b = d["y"], d["w"], d["z"], d["b"]
    leaves = [v.requires_grad_(op == "norm_grad") if v is not None else None for v in (y, w, z, b)]
    v = y * z * torch.sigmoid(z) if case["gate"] == "first" else y
    v = v.unflatten(1, (case["G"], -1))
    mean = v.mean(-1, keepdim=True) if case["center"] else 0.0
    v = (v - mean) * (((v - mean) ** 2).mean(-1, keepdim=True) + EPS) ** -0.5
    out = v.flatten(1) * w + (0.0 if b is None else b)
    if case["gate"] == "last":
        out = out * z * torch.sigmoid(z)
    if op == "norm":
        return out
    have = [v for v in leaves if v is not None]
    got = dict(zip(map(id, have), torch.autograd.grad(out, have, d["dout"])))
    y, w, z, b = (None if v is None else got[id(v)] for v in leaves)
    return {"y": y, "z": z, "weight": w, "bias": b}
