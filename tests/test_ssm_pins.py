"""Pins of the fp64 oracle of the state space scan, its convolution and the
draft verification (oracle/ssm.py): closed forms, an independent formulation,
finite differences, and the distribution that verification has to leave."""
import numpy as np
import pytest

from oracle import ssm as O


def inputs(T, H=4, G=2, N=5, P=3, seed=0):
    r = np.random.default_rng(seed)
    return dict(x=r.standard_normal((T, H, P)), dt=r.standard_normal((T, H)), A=-r.uniform(0.1, 2, H),
                B=r.standard_normal((T, G, N)), C=r.standard_normal((T, G, N)), D=r.standard_normal(H),
                S0=r.standard_normal((H, N, P)), dt_bias=r.standard_normal(H))


def test_conv_is_a_correlation_with_the_reversed_filter():
    r = np.random.default_rng(1)
    x, w, cache = r.standard_normal((9, 3)), r.standard_normal((3, 4)), r.standard_normal((3, 3))
    y, after = O.conv(x, w, cache=cache, activation=False)
    line = np.concatenate([cache, x])
    for c in range(3):
        assert np.allclose(y[:, c], np.convolve(line[:, c], w[c, ::-1], "valid"))
    assert np.array_equal(after, line[-3:])
    # in two calls with the cache between them
    y1, mid = O.conv(x[:2], w, cache=cache)
    y2, end = O.conv(x[2:], w, cache=mid)
    assert np.allclose(np.concatenate([y1, y2]), O.conv(x, w, cache=cache)[0]) and np.array_equal(end, after)


def test_scan_without_decay_is_linear_attention():
    i = inputs(7)
    y, S = O.scan(i["x"], i["dt"], np.zeros(4), i["B"], i["C"], dt_bias=i["dt_bias"])
    d = O.softplus(i["dt"] + i["dt_bias"])
    Bh, Ch = np.repeat(i["B"], 2, 1), np.repeat(i["C"], 2, 1)
    score = np.einsum("thn,shn,sh->hts", Ch, Bh, d) * np.tril(np.ones((7, 7)))
    assert np.allclose(y, np.einsum("hts,shp->thp", score, i["x"]))
    assert np.allclose(S, np.einsum("sh,shn,shp->hnp", d, Bh, i["x"]))


def test_scan_quadratic_form():
    i = inputs(9)
    y, S = O.scan(i["x"], i["dt"], i["A"], i["B"], i["C"], i["D"], i["S0"], i["dt_bias"])
    d = O.softplus(i["dt"] + i["dt_bias"])
    g = np.cumsum(d * i["A"], 0)
    Bh, Ch = np.repeat(i["B"], 2, 1), np.repeat(i["C"], 2, 1)
    decay = np.exp(np.minimum(g[:, None] - g[None], 0)) * np.tril(np.ones((9, 9)))[:, :, None]
    ref = np.einsum("thn,shn,sh,tsh,shp->thp", Ch, Bh, d, decay, i["x"])
    ref += np.exp(g)[:, :, None] * np.einsum("hnp,thn->thp", i["S0"], Ch) + i["D"][:, None] * i["x"]
    assert np.allclose(y, ref)


def test_scan_total_forgetting_keeps_one_token():
    i = inputs(5)
    y, S = O.scan(i["x"], i["dt"], np.full(4, -1e6), i["B"], i["C"], S0=i["S0"])
    d = O.softplus(i["dt"])
    Bh, Ch = np.repeat(i["B"], 2, 1), np.repeat(i["C"], 2, 1)
    assert np.allclose(y, (d * (Bh * Ch).sum(-1))[:, :, None] * i["x"])


@pytest.mark.parametrize("soft", [True, False])
def test_scan_backward_against_differences(soft):
    i = inputs(6, seed=3)
    if not soft:
        i["dt"] = np.abs(i["dt"])
        i["dt_bias"] = None
    r = np.random.default_rng(4)
    gy, gS = r.standard_normal(i["x"].shape), r.standard_normal(i["S0"].shape)

    def loss(j):
        y, S = O.scan(j["x"], j["dt"], j["A"], j["B"], j["C"], j["D"], j["S0"], j["dt_bias"], soft)
        return (y * gy).sum() + (S * gS).sum()

    g = O.scan_backward(i["x"], i["dt"], i["A"], i["B"], i["C"], i["D"], i["S0"], gy, gS, i["dt_bias"], soft)
    h = 1e-6
    for name, key in (("x", "x"), ("dt", "dt"), ("A", "A"), ("B", "B"), ("C", "C"), ("D", "D"), ("S0", "S0"),
                      ("dt_bias", "bias")):
        if i[name] is None:
            continue
        for _ in range(4):
            at = tuple(r.integers(0, n) for n in i[name].shape)
            up, dn = ({k: None if v is None else v.copy() for k, v in i.items()} for _ in range(2))
            up[name][at] += h
            dn[name][at] -= h
            d = (loss(up) - loss(dn)) / (2 * h)
            # central differences: h^2 of a third derivative and eps / h of the loss
            assert abs(d - g[key][at]) < 1e-6 * (1 + abs(d)) * 10, name


def test_conv_backward_against_differences():
    r = np.random.default_rng(6)
    a = dict(x=r.standard_normal((5, 2)), w=r.standard_normal((2, 4)), bias=r.standard_normal(2),
             cache=r.standard_normal((3, 2)))
    gy = r.standard_normal((5, 2))
    g = dict(zip(("x", "w", "bias", "cache"), O.conv_backward(a["x"], a["w"], a["bias"], a["cache"], gy)))
    h = 1e-6
    for name in a:
        for at in np.ndindex(a[name].shape):
            up, dn = ({k: v.copy() for k, v in a.items()} for _ in range(2))
            up[name][at] += h
            dn[name][at] -= h
            d = ((O.conv(**up)[0] - O.conv(**dn)[0]) * gy).sum() / (2 * h)
            assert abs(d - g[name][at]) < 1e-6 * (1 + abs(d)) * 10, name


def test_verification_leaves_the_targets_distribution():
    """Drafts from q, then verification over a fine grid of u and u_next: the
    first token's distribution is p."""
    p = np.array([[0.5, 0.125, 0.25, 0.125], [0.25] * 4])
    q = np.array([[0.25, 0.5, 0.125, 0.125]])
    grid = (np.arange(64) + 0.5) / 64
    freq = np.zeros(4)
    for d in range(4):
        for u in grid:
            for v in grid:
                n, tok = O.verify(p, [d], [u], v, q)
                freq[tok[0]] += q[0, d] / 64 ** 2
    # the grid is exact to one cell in u and one in u_next
    assert np.max(np.abs(freq - p[0])) < 2 / 64


def test_verification_edges():
    p = np.array([[0.0, 1.0, 0.0], [0.5, 0.0, 0.5]])
    assert O.verify(p, [1], [0.99], 0.0)[0] == 1
    assert list(O.verify(p, [1], [0.99], 0.6)[1]) == [1, 2]
    assert list(O.verify(p, [0], [0.0], 0.5)[1]) == [1, -1]           # no mass: 0 < 0 fails
    assert list(O.verify(p, [7], [0.0], 0.5)[1]) == [1, -1]           # not a token
    assert list(O.verify(p, [1], [0.5], 0.5, n_draft=0)[1]) == [1, -1]
    assert list(O.verify(p, [1], [0.5], 0.0, q=p[:1])[1]) == [1, 0]
    assert list(O.verify(np.zeros((2, 3)), [1], [0.5], 0.5)[1]) == [0, -1]
    assert list(O.verify(np.full((2, 3), np.nan), [1], [0.5], 0.5)[1]) == [0, -1]
