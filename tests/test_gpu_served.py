"""GPU parity of the served forms -- convolution and selective scan over packed prompts and for
single tokens with their caches -- against the float64 oracle (oracle.served), within bounds that
count roundings (served_util)."""
import numpy as np
import pytest
import torch

import mamba_ssd_scan_03_b200 as ssd
from oracle import served
from served_util import (conv_bound, down, excess, scan_bound, silu_bound, store, up, up_rows)

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def flags(v):
    return torch.tensor([bool(b) for b in v], device="cuda")


def conv_inputs(T, C, K, nslots, io, seed=0):
    r = np.random.default_rng(seed)
    return dict(u=store(r.standard_normal((T, C)), io),
                w=(r.standard_normal((C, K)) / K ** 0.5).astype(np.float32),
                bias=(r.standard_normal(C) / 10).astype(np.float32),
                state=store(r.standard_normal((nslots, K - 1, C)), io))


def run_conv(g, cu, io, slots=None, resume=None, bias=True, keep=True, pad=0, shift=0):
    """Both sides; (got, got state, ref, ref state, bound) with unwritten rows marked 5."""
    T, C = g["u"].shape
    b = g["bias"] if bias else None
    st = up(g["state"], io) if keep else None
    out = up_rows(np.full((T, C), 5.0, np.float32) if io == "f32" else
                  store(np.full((T, C), 5.0), io), io, pad, shift)
    ssd.conv_silu_varlen(up_rows(g["u"], io, pad, shift), up(g["w"]), i32(cu),
                         None if b is None else up(b), st, None if slots is None else i32(slots),
                         None if resume is None else flags(resume), out=out)
    ref, rst = served.conv_silu(g["u"], g["w"], b, cu, g["state"] if keep else None, slots,
                                resume, out=np.full((T, C), 5.0))
    bound = conv_bound(g["u"], g["w"], b, cu, g["state"] if keep else None, slots, resume, io)
    return down(out), None if st is None else down(st), ref, rst, bound


CUTS = {
    "one": [0, 150],
    "ones": [0, 1, 2, 3, 4, 5, 6],
    "ragged": [0, 3, 70, 71, 73, 200, 333],
    "edges": [0, 64, 126, 128, 130, 191, 192, 194, 256],  # on and around the runs of 64 rows
    "empty": [0, 0, 5, 5, 64, 64, 64, 127, 127],
    "tail": [2, 60, 90],  # rows ahead of the first and behind the last sequence
}


@pytest.mark.parametrize("cut", sorted(CUTS))
@pytest.mark.parametrize("io,C,K,pad,shift", [
    ("bf16", 64, 4, 0, 0), ("bf16", 272, 4, 16, 8), ("bf16", 37, 4, 0, 0), ("f32", 40, 3, 4, 4),
    ("f32", 33, 2, 1, 3), ("bf16", 24, 8, 8, 1), ("f32", 8, 1, 0, 0), ("bf16", 1, 5, 0, 0),
    ("f32", 12, 7, 0, 0), ("bf16", 16, 6, 0, 0)])
def test_conv_prompts(cut, io, C, K, pad, shift):
    cu = CUTS[cut]
    n = len(cu) - 1
    T = cu[-1] + (7 if cut == "tail" else 0)
    g = conv_inputs(T, C, K, n + 2, io, seed=K)
    slots = list(np.random.default_rng(1).permutation(n + 2)[:n])
    for resume in ([i % 3 != 1 for i in range(n)], None):
        got, st, ref, rst, bound = run_conv(g, cu, io, slots, resume, keep=K > 1, pad=pad,
                                            shift=shift) if K > 1 else \
            run_conv(g, cu, io, keep=False, pad=pad, shift=shift)
        assert excess(got, ref, bound) <= 0
        if st is not None:
            assert np.array_equal(st, rst)  # the inputs' own bits
    assert ssd.device_status() == 0


def test_conv_prompts_without_cache_or_bias():
    g = conv_inputs(90, 48, 4, 3, "bf16")
    got, _, ref, _, bound = run_conv(g, [0, 30, 90], "bf16", keep=False, bias=False)
    assert excess(got, ref, bound) <= 0
    # the same rows through the dense call
    dense = ssd.conv_silu(up(g["u"], "bf16").view(3, 30, 48), up(g["w"]))
    packed = ssd.conv_silu_varlen(up(g["u"], "bf16"), up(g["w"]), i32([0, 30, 60, 90]))
    assert torch.equal(dense.view(90, 48), packed)


def test_conv_prompts_many_sequences():
    """More sequences than a warp has lanes, some of length zero, one or two."""
    r = np.random.default_rng(4)
    cu = [0] + [int(v) for v in np.cumsum(r.integers(0, 4, 150))]
    g = conv_inputs(cu[-1], 40, 4, 150, "f32")
    resume = [bool(v) for v in r.integers(0, 2, 150)]
    got, st, ref, rst, bound = run_conv(g, cu, "f32", None, resume)
    assert excess(got, ref, bound) <= 0 and np.array_equal(st, rst)


@pytest.mark.parametrize("io,batch,C,K,pad,shift", [
    ("bf16", 1, 64, 4, 0, 0), ("bf16", 37, 272, 4, 8, 8), ("f32", 5, 33, 2, 1, 0),
    ("bf16", 9, 1301, 3, 0, 0), ("f32", 300, 16, 8, 4, 4)])
def test_conv_token(io, batch, C, K, pad, shift):
    g = conv_inputs(batch, C, K, batch + 3, io)
    slots = [int(s) for s in np.random.default_rng(2).permutation(batch + 3)[:batch]]
    slots[batch // 2] = -1 if batch > 1 else slots[0]  # a padded row
    st = up(g["state"], io)
    out = up_rows(store(np.full((batch, C), 5.0), io), io, pad, shift)
    ssd.conv_silu_step(st, up_rows(g["u"], io, pad, shift), up(g["w"]), up(g["bias"]),
                       i32(slots), out=out)
    cu, one = list(range(batch + 1)), [True] * batch
    ref, rst = served.conv_silu(g["u"], g["w"], g["bias"], cu, g["state"], slots, one,
                                out=np.full((batch, C), 5.0))
    bound = conv_bound(g["u"], g["w"], g["bias"], cu, g["state"], slots, one, io)
    assert excess(down(out), ref, bound) <= 0
    assert np.array_equal(down(st), rst)
    assert ssd.device_status() == 0


def scan_inputs(T, dim, N, G, nslots, io="bf16", dt="f32", gate=True, seed=0):
    r = np.random.default_rng(seed)
    return dict(x=store(r.standard_normal((T, dim)), io),
                dt=store(0.5 * r.standard_normal((T, dim)), dt),
                A=-np.exp(r.uniform(0, np.log(16), (dim, N))).astype(np.float32),
                B=store(r.standard_normal((T, G, N)) / N ** 0.5, io),
                C=store(r.standard_normal((T, G, N)) / N ** 0.5, io),
                D=r.standard_normal(dim).astype(np.float32),
                dt_bias=(-2 + 0.1 * r.standard_normal(dim)).astype(np.float32),
                z=store(r.standard_normal((T, dim)), io) if gate else None,
                use_softplus=True,
                state=(0.3 * r.standard_normal((nslots, dim, N))).astype(np.float32))


def run_scan(g, cu, io, dt, y_io, slots=None, resume=None, pad=0, shift=0, hint=0, step=False):
    g = dict(g)
    T, dim = g["x"].shape
    st = None if g["state"] is None else up(g["state"])
    y = up_rows(store(np.full((T, dim), 5.0), y_io), y_io, pad, shift)
    rows = lambda k, f=io: up_rows(g[k], f, pad, shift)  # noqa: E731
    opt = lambda k: None if g[k] is None else up(g[k])  # noqa: E731
    z = None if g["z"] is None else rows("z")
    sl = None if slots is None else i32(slots)
    if step:
        ssd.selective_step(st, rows("x"), rows("dt", dt), up(g["A"]), rows("B"), rows("C"),
                           opt("D"), z, opt("dt_bias"), g["use_softplus"], sl, out=y)
    else:
        ssd.selective_scan_varlen(
            rows("x"), rows("dt", dt), up(g["A"]), rows("B"), rows("C"), i32(cu), opt("D"), z,
            opt("dt_bias"), g["use_softplus"], st, sl,
            None if resume is None else flags(resume), out=y, max_seqlen=hint)
    g["cu"], g["slots"], g["resume"] = cu, slots, resume
    ref = served.selective_scan(**g, out=np.full((T, dim), 5.0))
    by, bh = scan_bound(g, ref, y_io)
    assert excess(down(y), ref[0], by) <= 0
    if st is not None:
        assert excess(down(st), ref[1], bh) <= 0
        left = [s for s in range(len(g["state"])) if s not in
                (range(len(cu) - 1) if slots is None else slots)]
        assert np.array_equal(down(st)[left], g["state"][left].astype(np.float64))
    assert ssd.device_status() == 0


@pytest.mark.parametrize("cut", sorted(CUTS))
@pytest.mark.parametrize("io,dt,y_io,dim,N,G,pad,shift", [
    ("bf16", "f32", "f32", 64, 16, 1, 0, 0), ("bf16", "bf16", "bf16", 48, 16, 2, 8, 8),
    ("f32", "f32", "f32", 37, 16, 1, 1, 2), ("bf16", "f32", "bf16", 24, 8, 1, 0, 0),
    ("f32", "f32", "f32", 10, 5, 2, 0, 0), ("bf16", "bf16", "f32", 9, 32, 1, 0, 0),
    ("f32", "f32", "f32", 12, 50, 1, 0, 0), ("bf16", "f32", "f32", 20, 128, 2, 0, 4)])
def test_scan_prompts(cut, io, dt, y_io, dim, N, G, pad, shift):
    cu = CUTS[cut]
    n = len(cu) - 1
    g = scan_inputs(cu[-1] + (7 if cut == "tail" else 0), dim, N, G, n + 2, io, dt, seed=dim)
    slots = [int(s) for s in np.random.default_rng(1).permutation(n + 2)[:n]]
    run_scan(g, cu, io, dt, y_io, slots, [i % 3 != 1 for i in range(n)], pad, shift)


@pytest.mark.parametrize("T,hint", [(700, 0), (700, 500), (1000, 1000), (451, 401)])
@pytest.mark.parametrize("resume", [None, [1, 0, 1]])
def test_scan_prompts_in_chunks(T, hint, resume):
    """Few channels and long sequences: chunks with a summary pass, one sequence short."""
    assert ssd.selective_varlen_workspace_size(T, 3, 40, 16, 1, hint) > 0
    g = scan_inputs(T, 40, 16, 1, 3)
    run_scan(g, [0, T - 30, T - 20, T], "bf16", "f32", "f32", None, resume, hint=hint)


def test_scan_prompts_wide_batch():
    """Enough channels and sequences for two channels per lane; odd channel count."""
    g = scan_inputs(60, 6400 + 5, 16, 1, 8, "bf16", "f32")
    run_scan(g, [0, 10, 11, 13, 20, 33, 34, 50, 60], "bf16", "f32", "bf16", None,
             [1, 0, 1, 0, 1, 0, 1, 1])


def test_scan_prompts_plain():
    """No gate, skip, bias, softplus or cache; dt as given; equal to the dense call."""
    g = scan_inputs(64, 32, 16, 1, 2, gate=False)
    g.update(D=None, dt_bias=None, use_softplus=False, state=None,
             dt=np.abs(g["dt"]) + np.float32(0.05))
    run_scan(g, [0, 32, 64], "bf16", "f32", "f32")
    f = lambda k, io="f32": up(g[k], io).view((2, 32) + g[k].shape[1:])  # noqa: E731
    dense, _ = ssd.selective_scan_fwd(f("x", "bf16"), f("dt"), up(g["A"]), f("B", "bf16"),
                                      f("C", "bf16"))
    packed = ssd.selective_scan_varlen(up(g["x"], "bf16"), up(g["dt"]), up(g["A"]),
                                       up(g["B"], "bf16"), up(g["C"], "bf16"), i32([0, 32, 64]))
    assert torch.allclose(dense.view(64, 32), packed, rtol=0, atol=1e-5)


@pytest.mark.parametrize("N,G,io,dt,y_io", [
    (16, 1, "bf16", "f32", "f32"), (16, 2, "bf16", "bf16", "bf16"), (8, 1, "f32", "f32", "f32"),
    (5, 1, "bf16", "f32", "f32"), (33, 2, "f32", "f32", "f32"), (64, 1, "bf16", "bf16", "f32"),
    (128, 1, "bf16", "f32", "bf16"), (1, 1, "f32", "f32", "f32")])
@pytest.mark.parametrize("batch,dim", [(1, 70), (7, 34), (130, 640)])
def test_scan_token(N, G, io, dt, y_io, batch, dim):
    g = scan_inputs(batch, dim, N, G, batch + 2, io, dt)
    slots = [int(s) for s in np.random.default_rng(3).permutation(batch + 2)[:batch]]
    if batch > 1:
        slots[batch // 3] = -1
    run_scan(g, list(range(batch + 1)), io, dt, y_io, slots, [True] * batch, 3, 1, step=True)


def test_extreme_rates_and_steps():
    """Rates of -inf and 0, steps that underflow and saturate the softplus: finite, as the
    definition says."""
    g = scan_inputs(70, 16, 16, 1, 1, "f32", "f32")
    A = g["A"].copy()
    A[:, 0], A[:, 1], A[:, 2] = -np.inf, 0.0, -1e30
    dt = g["dt"].copy()
    dt[5], dt[6], dt[7] = 60.0, -60.0, 100.0
    y = ssd.selective_scan_varlen(up(g["x"]), up(dt), up(A), up(g["B"]), up(g["C"]),
                                  i32([0, 70]), softplus=True)
    with np.errstate(over="ignore"):
        ref, _ = served.selective_scan(g["x"], dt, A, g["B"], g["C"], [0, 70], use_softplus=True)
    assert np.all(np.isfinite(down(y)))
    assert excess(down(y), ref, 1e-5 * np.max(np.abs(ref))) <= 0


def test_bad_indices_are_left_out_and_reported():
    """A slot past the cache, one named twice and bounds that decrease: reported, nothing of theirs
    written, the other sequences as usual."""
    g = scan_inputs(12, 16, 16, 1, 4)
    c = conv_inputs(12, 16, 4, 4, "bf16")
    cu = [0, 3, 6, 9, 12]
    for slots in ([2, 4, 0, 1], [2, 0, 2, 1], [1, 2 ** 31 - 1, -5, 0]):
        st, cs = up(g["state"]), up(c["state"], "bf16")
        y = torch.full((12, 16), 5.0, device="cuda")
        ssd.selective_scan_varlen(up(g["x"], "bf16"), up(g["dt"]), up(g["A"]), up(g["B"], "bf16"),
                                  up(g["C"], "bf16"), i32(cu), softplus=True, state=st,
                                  slots=i32(slots), out=y)
        assert ssd.device_status() == 6
        ref, rst = served.selective_scan(g["x"], g["dt"], g["A"], g["B"], g["C"], cu,
                                         use_softplus=True, state=g["state"], slots=slots,
                                         out=np.full((12, 16), 5.0))
        assert np.max(np.abs(down(y) - ref)) < 1e-4 and np.max(np.abs(down(st) - rst)) < 1e-4
        out = torch.full((12, 16), 5.0, device="cuda", dtype=torch.bfloat16)
        ssd.conv_silu_varlen(up(c["u"], "bf16"), up(c["w"]), i32(cu), conv_state=cs,
                             slots=i32(slots), out=out)
        assert ssd.device_status() == 6
        ref, rst = served.conv_silu(c["u"], c["w"], None, cu, c["state"], slots,
                                    out=np.full((12, 16), 5.0))
        assert np.max(np.abs(down(out) - ref)) < 2e-2 and np.array_equal(down(cs), rst)
        # tokens
        st, cs = up(g["state"]), up(c["state"], "bf16")
        rows = slice(0, 4)
        y = torch.full((4, 16), 5.0, device="cuda")
        ssd.selective_step(st, up(g["x"], "bf16")[rows], up(g["dt"])[rows], up(g["A"]),
                           up(g["B"], "bf16")[rows], up(g["C"], "bf16")[rows], softplus=True,
                           slots=i32(slots), out=y)
        assert ssd.device_status() == 6
        one = [0, 1, 2, 3, 4]
        ref, rst = served.selective_scan(g["x"][rows], g["dt"][rows], g["A"], g["B"][rows],
                                         g["C"][rows], one, use_softplus=True, state=g["state"],
                                         slots=slots, resume=[1] * 4, out=np.full((4, 16), 5.0))
        assert np.max(np.abs(down(y) - ref)) < 1e-4 and np.max(np.abs(down(st) - rst)) < 1e-4
        out = torch.full((4, 16), 5.0, device="cuda", dtype=torch.bfloat16)
        ssd.conv_silu_step(cs, up(c["u"], "bf16")[rows], up(c["w"]), slots=i32(slots), out=out)
        assert ssd.device_status() == 6
        ref, rst = served.conv_silu(c["u"][rows], c["w"], None, one, c["state"], slots, [1] * 4,
                                    out=np.full((4, 16), 5.0))
        assert np.max(np.abs(down(out) - ref)) < 2e-2 and np.array_equal(down(cs), rst)
    for cu in ([0, 9, 6, 12, 12], [0, 3, 6, 9, 13], [-1, 3, 6, 9, 12], [5, 4, 3, 2, 1],
               [0, 12, 0, 12, 0]):
        ssd.selective_scan_varlen(up(g["x"], "bf16"), up(g["dt"]), up(g["A"]), up(g["B"], "bf16"),
                                  up(g["C"], "bf16"), i32(cu), softplus=True,
                                  state=up(g["state"]))
        assert ssd.device_status() == 6
        ssd.conv_silu_varlen(up(c["u"], "bf16"), up(c["w"]), i32(cu),
                             conv_state=up(c["state"], "bf16"))
        assert ssd.device_status() == 6


def test_empty_calls():
    """No rows, no sequences, only empty sequences: fresh slots become zero, the rest stays."""
    u = torch.zeros(0, 24, device="cuda")
    w = torch.ones(24, 4, device="cuda")
    cs = torch.ones(3, 3, 24, device="cuda")
    ssd.conv_silu_varlen(u, w, i32([0, 0, 0]), conv_state=cs, slots=i32([2, 0]),
                         resume=flags([0, 1]))
    assert torch.all(cs[2] == 0) and torch.all(cs[:2] == 1)
    ssd.conv_silu_varlen(u, w, i32([0]), conv_state=cs)
    ssd.conv_silu_step(cs, u, w)
    x, B = torch.zeros(0, 24, device="cuda"), torch.zeros(0, 1, 16, device="cuda")
    A, st = -torch.ones(24, 16, device="cuda"), torch.ones(3, 24, 16, device="cuda")
    ssd.selective_scan_varlen(x, x, A, B, B, i32([0, 0, 0]), state=st, slots=i32([2, 0]),
                              resume=flags([0, 1]))
    assert torch.all(st[2] == 0) and torch.all(st[:2] == 1)
    ssd.selective_scan_varlen(x, x, A, B, B, i32([0]), state=st)
    ssd.selective_step(st, x, x, A, B, B)
    assert torch.all(st[2] == 0) and torch.all(st[:2] == 1)
    assert ssd.device_status() == 0


def test_calls_on_another_stream_and_replayed():
    """Prompts then tokens, captured in one graph and replayed with new tokens, slots and bounds in
    the same buffers, equal to the same calls made eagerly."""
    r = np.random.default_rng(7)
    T, dim, K = 20, 32, 4
    g, c = scan_inputs(T, dim, 16, 1, 6), conv_inputs(T, dim, K, 6, "bf16")
    t = {k: up(g[k]) for k in ("dt", "A", "D", "dt_bias")}
    t |= {k: up(g[k], "bf16") for k in ("B", "C", "z")}
    u, w = up(c["u"], "bf16"), up(c["w"])
    cu, slots = i32([0, 5, 9, 20]), i32([4, 1, 2])
    cs, st = up(c["state"], "bf16"), up(g["state"])
    args = lambda s: dict(D=t["D"], dt_bias=t["dt_bias"], softplus=True, slots=slots)  # noqa

    def both(cs, st):
        x = ssd.conv_silu_varlen(u, w, cu, conv_state=cs, slots=slots)
        y = ssd.selective_scan_varlen(x, t["dt"], t["A"], t["B"], t["C"], cu, z=t["z"], state=st,
                                      **args(0))
        x1 = ssd.conv_silu_step(cs, u[:3], w, slots=slots)
        y1 = ssd.selective_step(st, x1, t["dt"][:3], t["A"], t["B"][:3], t["C"][:3], **args(0))
        return y, y1

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(cs.clone(), st.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, y1 = both(cs, st)
    for k in range(3):
        u.copy_(torch.from_numpy(r.standard_normal((T, dim))).to(u))
        cu.copy_(i32([[0, 5, 9, 20], [0, 0, 19, 20], [1, 2, 3, 18]][k]))
        slots.copy_(i32([[4, 1, 2], [0, -1, 3], [5, 4, 1]][k]))
        cs0, st0 = cs.clone(), st.clone()
        y.fill_(5.0), y1.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        e, e1 = both(cs0, st0)
        lo, hi = int(cu[0]), int(cu[-1])
        pad = [i for i in range(3) if int(slots[i]) < 0]
        on = [j for j in range(lo, hi) if not any(int(cu[i]) <= j < int(cu[i + 1]) for i in pad)]
        assert torch.equal(y[on], e[on])
        rows = [i for i in range(3) if i not in pad]
        assert torch.equal(y1[rows], e1[rows])
        assert torch.equal(cs, cs0) and torch.equal(st, st0)
    assert ssd.device_status() == 0


def test_prompt_then_tokens_is_the_whole_sequence():
    """A block as it is served -- convolution, scan with gate, norm -- over prompts in two pieces and
    then token by token, against the float64 block over the whole sequences."""
    r = np.random.default_rng(8)
    dim, N, K, n, L = 64, 16, 4, 3, 40
    pieces = [[17, 18, 20], [3, 15, 12]]  # lengths of the two prompt pieces
    g = scan_inputs(n * L, dim, N, 1, n, "f32")
    c = conv_inputs(n * L, dim, K, n, "f32")
    nw = (1 + 0.1 * r.standard_normal(dim)).astype(np.float32)
    seqs = lambda a: a.reshape((n, L) + a.shape[1:])  # noqa: E731
    # oracle: whole sequences from zeros
    cu = [0, L, 2 * L, 3 * L]
    xo, _ = served.conv_silu(c["u"], c["w"], c["bias"], cu)
    ref, _ = served.selective_scan(xo, g["dt"], g["A"], g["B"], g["C"], cu, g["D"], None,
                                   g["dt_bias"], True)
    ref = seqs(served.group_norm(ref, nw, None, g["z"], 4)["out"])
    st = torch.full((n, dim, N), 7.0, device="cuda")
    cs = torch.full((n, K - 1, dim), 7.0, device="cuda")
    slots, done, got = i32([2, 0, 1]), [0] * n, [[] for _ in range(n)]
    k = {a: up(g[a]) for a in ("A", "D", "dt_bias")}

    def rows(a, take):
        return up(np.concatenate([seqs(a)[i, done[i]:done[i] + take[i]] for i in range(n)]))

    def block(take, resume):
        lens = np.cumsum([0] + take).tolist()
        arg = (rows(g["dt"], take), k["A"], rows(g["B"], take), rows(g["C"], take))
        if max(take) == 1 == min(take) and resume:
            x = ssd.conv_silu_step(cs, rows(c["u"], take), up(c["w"]), up(c["bias"]), slots)
            y = ssd.selective_step(st, x, *arg, k["D"], None, k["dt_bias"], True, slots)
        else:
            x = ssd.conv_silu_varlen(rows(c["u"], take), up(c["w"]), i32(lens), up(c["bias"]), cs,
                                     slots, flags([resume] * n))
            y = ssd.selective_scan_varlen(x, *arg, i32(lens), k["D"], None, k["dt_bias"], True, st,
                                          slots, flags([resume] * n))
        y = down(ssd.group_norm_gate(y, up(nw), None, rows(g["z"], take), 4))
        for i in range(n):
            got[i].append(y[lens[i]:lens[i + 1]])
            done[i] += take[i]

    block(pieces[0], False)
    block(pieces[1], True)
    while min(done) < L:
        if max(done) < L:
            block([1] * n, True)
        else:  # finished sequences are padding
            live = [i for i in range(n) if done[i] < L]
            slots = i32([[2, 0, 1][i] if i in live else -1 for i in range(n)])
            take = [1 if i in live else 0 for i in range(n)]
            block(take, True)
    for i in range(n):
        # float32 through the convolution, 40 steps, the norm: (as scan_bound, on inputs with the
        # convolution's error) well below 1e-4 of the normalised output's unit scale
        assert np.max(np.abs(np.concatenate(got[i]) - ref[i])) <= 1e-4
    assert ssd.device_status() == 0
