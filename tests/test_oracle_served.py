"""Pins of the float64 oracle of the served forms (oracle.served): against the dense oracles of the
same operators, splitting a sequence, library routines and finite differences."""
import numpy as np
import pytest

from oracle import glue, selective, served


def _rng(seed=0):
    return np.random.default_rng(seed)


@pytest.mark.parametrize("K", [1, 2, 4, 8])
def test_conv_of_dense_sequences_is_the_dense_convolution(K):
    r = _rng(K)
    u, w, b = r.standard_normal((3, 11, 5)), r.standard_normal((5, K)), r.standard_normal(5)
    out, _ = served.conv_silu(u.reshape(33, 5), w, b, [0, 11, 22, 33])
    assert np.allclose(out.reshape(3, 11, 5), glue.conv_silu(u, w, b), atol=1e-14)


@pytest.mark.parametrize("cuts", [[0, 13], [0, 1, 2, 13], [0, 0, 2, 2, 5, 13, 13]])
def test_conv_in_pieces_is_the_whole(cuts):
    """One sequence served piece by piece through a slot, lengths 0 and 1 among the pieces."""
    r = _rng(1)
    K = 4
    u, w, b = r.standard_normal((13, 6)), r.standard_normal((6, K)), r.standard_normal(6)
    whole, end = served.conv_silu(u, w, b, [0, 13], state=np.zeros((1, K - 1, 6)))
    state, got = np.full((2, K - 1, 6), 7.0), []
    for i, (lo, hi) in enumerate(zip(cuts, cuts[1:])):
        o, state = served.conv_silu(u[lo:hi], w, b, [0, hi - lo], state=state, slots=[1],
                                    resume=[i > 0])
        got.append(o)
    assert np.allclose(np.concatenate(got), whole, atol=1e-14)
    assert np.array_equal(state[1], end[0]) and np.all(state[0] == 7.0)


def test_scan_of_dense_sequences_is_the_dense_scan():
    r = _rng(2)
    Bt, L, dim, N, G = 2, 9, 6, 5, 3
    x, raw = r.standard_normal((Bt, L, dim)), r.standard_normal((Bt, L, dim))
    A, D = -np.exp(r.standard_normal((dim, N))), r.standard_normal(dim)
    B, C = r.standard_normal((2, Bt, L, G, N))
    init, z = r.standard_normal((Bt, dim, N)), r.standard_normal((Bt, L, dim))
    dt = glue.softplus(raw + 0.25)
    y0, h0 = selective.selective_scan(x, dt, A, B, C, D, init)
    f = lambda a: a.reshape((Bt * L,) + a.shape[2:])  # noqa: E731
    y, h = served.selective_scan(f(x), f(raw), A, f(B), f(C), [0, L, 2 * L], D, f(z),
                                 np.full(dim, 0.25), True, state=init, resume=[1, 1])
    assert np.allclose(y, f(glue.gate_silu(y0, z)), atol=1e-13)
    assert np.allclose(h, h0, atol=1e-13)


def test_slots_padding_and_rows_outside():
    """Padding, a slot out of range and a slot named again are left alone; so are rows that no
    sequence covers."""
    r = _rng(3)
    x, A = r.standard_normal((8, 4)), -np.ones((4, 2))
    B = r.standard_normal((8, 1, 2))
    state = r.standard_normal((3, 4, 2))
    mark = np.full((8, 4), 9.0)
    y, h = served.selective_scan(x, np.abs(x), A, B, B, [1, 2, 4, 5, 6, 7], state=state,
                                 slots=[2, -1, 3, 2, 0], resume=[1, 1, 1, 1, 0], out=mark)
    assert np.all(y[[0, 2, 3, 4, 5, 7]] == 9.0) and not np.any(y[[1, 6]] == 9.0)
    assert np.array_equal(h[1], state[1]) and not np.any(h[2] == state[2])
    o, s = served.conv_silu(x, np.ones((4, 3)), None, [1, 2, 4, 5, 6, 7],
                            state=state.transpose(0, 2, 1), slots=[2, -1, 3, 2, 0], out=mark)
    assert np.all(o[[0, 2, 3, 4, 5, 7]] == 9.0)
    assert np.array_equal(s[2][1], x[1]) and np.all(s[2][0] == 0)
    assert np.array_equal(s[1], state.transpose(0, 2, 1)[1])


def test_group_norm_centred_is_the_library_group_norm():
    torch = pytest.importorskip("torch")
    r = _rng(4)
    y, w, b = r.standard_normal((7, 12)) + 3, r.standard_normal(12), r.standard_normal(12)
    got = served.group_norm(y, w, b, None, 3, 1e-3, center=True)["out"]
    ref = torch.nn.functional.group_norm(*map(torch.from_numpy, (y,)), 3, torch.from_numpy(w),
                                         torch.from_numpy(b), 1e-3)
    assert np.allclose(got, ref.numpy(), atol=1e-13)


def test_group_norm_gate_places():
    r = _rng(5)
    y, w, z = r.standard_normal((3, 8)), r.standard_normal(8), r.standard_normal((3, 8))
    first = served.group_norm(glue.gate_silu(y, z), w, None, None, 2)["out"]
    assert np.allclose(served.group_norm(y, w, None, z, 2)["out"], first, atol=1e-14)
    last = glue.gate_silu(served.group_norm(y, w, None, None, 2)["out"], z)
    assert np.allclose(served.group_norm(y, w, None, z, 2, gate_first=False)["out"], last,
                       atol=1e-14)


@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("gate", ["none", "first", "last"])
@pytest.mark.parametrize("ngroups", [1, 4])
def test_group_norm_gradients_against_differences(center, gate, ngroups):
    r = _rng(6)
    p = {"y": r.standard_normal((5, 8)), "z": r.standard_normal((5, 8)),
         "weight": r.standard_normal(8), "bias": r.standard_normal(8)}
    if gate == "none":
        p["z"] = None
    do = r.standard_normal((5, 8))

    def out(q):
        return served.group_norm(q["y"], q["weight"], q["bias"], q["z"], ngroups, 1e-2, center,
                                 gate != "last")["out"]

    g = served.group_norm_backward(do, p["y"], p["weight"], p["bias"], p["z"], ngroups, 1e-2,
                                   center, gate != "last")
    for k, v in p.items():
        if v is None:
            assert g[k] is None
            continue
        way = r.standard_normal(v.shape)
        e = 1e-5
        diff = (np.sum(do * out({**p, k: v + e * way})) -
                np.sum(do * out({**p, k: v - e * way}))) / (2 * e)
        assert abs(np.sum(g[k] * way) - diff) <= 1e-7 * (1 + abs(diff)), k
