"""GPU parity of the state space scan and its short convolution against the
fp64 oracle (oracle/ssm.py), forward, backward and recurrent, and a run of
them together with the draft verification.

Tolerances, elementwise.  One rounding is off by at most half a step: 2^-8 of
the value for bf16, 2^-24 for float32.  `mag` is the same oracle on the
absolute values of everything, so it bounds the sum of the absolute terms:

  - bf16 outputs: 2^-8 |ref| for the result and 2^-8 mag for the operands
    that are rounded once (the state in S^T C, the chunk matrix), plus the
    float32 part below;
  - float32 results: each term passes a few dozen float32 roundings (dt, its
    exponential, products, sums in the matrix cores), and a decay e^g with
    |g| up to about 50 before its terms vanish carries |g| 2^-24: 160 half
    steps, 1e-5 of mag.
"""
import numpy as np
import pytest

from kda_testlib import say
from oracle import ssm as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU-only container
    pytest.skip("no GPU", allow_module_level=True)

import gated_delta_rule_amd as kda  # noqa: E402

HALF = 2.0 ** -8
F32 = 1e-5


def dev(a, dtype=torch.float32):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dtype)


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def check(name, got, ref, mag, dtype, rounded=True):
    """got against ref within the tolerances above."""
    got, ref, mag = np.asarray(got, np.float64), np.asarray(ref), np.asarray(mag)
    tol = F32 * mag + 1e-30
    if dtype == torch.bfloat16:
        tol = tol + HALF * np.abs(ref) * 1.01 + (HALF * 1.01 * mag if rounded else 0.0)
    bad = np.abs(got - ref) / tol
    worst = float(bad.max()) if bad.size else 0.0
    assert np.isfinite(got).all() and worst <= 1.0, f"{name}: {worst:.3g} of the tolerance"
    return worst


def q(a, dtype):
    """Values that the input type holds exactly, as float64."""
    return torch.from_numpy(np.asarray(a, np.float32)).to(dtype).double().numpy()


# ------------------------------------------------------------ convolution

def conv_case(lens, c, W, dtype, cache, bias, seed=0):
    r = np.random.default_rng(seed)
    T = sum(lens)
    return dict(x=q(r.standard_normal((T, c)), dtype), w=np.float32(r.standard_normal((c, W))).astype(np.float64),
                bias=np.float32(r.standard_normal(c)).astype(np.float64) if bias else None,
                cache=np.float32(r.standard_normal((len(lens), W - 1, c))).astype(np.float64) if cache else None,
                gy=q(r.standard_normal((T, c)), dtype), cu=np.concatenate([[0], np.cumsum(lens)]))


CONV = [([1], 8, 2, True, True), ([0, 1, 2, 3, 0, 4, 5], 72, 4, True, True), ([257, 15, 16, 17], 264, 3, False, True),
        ([300], 40, 4, True, False), ([33, 1, 128], 2056, 4, False, False)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,c,W,cache,bias", CONV)
@pytest.mark.parametrize("activation", [True, False])
def test_conv_packed(lens, c, W, cache, bias, dtype, activation):
    a = conv_case(lens, c, W, dtype, cache, bias)
    cu, cd = dev(a["cu"], torch.int32), dev(a["cache"])
    # the rows lie inside wider ones
    wide = torch.full((sum(lens), c + 16), float("nan"), dtype=dtype, device="cuda")
    x = wide[:, 8:8 + c]
    x.copy_(dev(a["x"], dtype))
    gwide = torch.full_like(wide, float("nan"))
    gy = gwide[:, 16:16 + c]
    gy.copy_(dev(a["gy"], dtype))
    before = None if cd is None else cd.clone()
    y = kda.ssm_conv_fwd(x, dev(a["w"]), dev(a["bias"]), cd, cu, activation=activation)
    g = kda.ssm_conv_bwd(x, dev(a["w"]), dev(a["bias"]), gy, before, cu, activation=activation)
    torch.cuda.synchronize()
    ab = {k: None if v is None else np.abs(v) for k, v in a.items()}
    gw, gw_m, gb, gb_m = 0.0, 0.0, 0.0, 0.0
    for n, (s, e) in enumerate(zip(a["cu"], a["cu"][1:])):
        ca = None if a["cache"] is None else a["cache"][n]
        ref, after = O.conv(a["x"][s:e], a["w"], a["bias"], ca, activation)
        mag, _ = O.conv(ab["x"][s:e], ab["w"], ab["bias"], None if ca is None else np.abs(ca), False)
        check("y", host(y[s:e]), ref, mag, dtype, rounded=False)
        if ca is not None:
            assert np.array_equal(host(cd[n]), after)
        ref = O.conv_backward(a["x"][s:e], a["w"], a["bias"], ca, a["gy"][s:e], activation)
        # |silu'| <= 1.1 and its slope is at most 1/2: errors of z reach dz
        slope = 1.1 + mag
        mg = O.conv_backward(ab["x"][s:e], ab["w"], ab["bias"], None if ca is None else np.abs(ca),
                             ab["gy"][s:e] * slope, False)
        check("grad_x", host(g[0][s:e]), ref[0], mg[0], dtype, rounded=False)
        gw, gw_m, gb, gb_m = gw + ref[1], gw_m + mg[1], gb + ref[2], gb_m + mg[2]
        if ca is not None:
            check("grad_cache", host(g[3][n]), ref[3], mg[3], torch.float32)
    check("grad_w", host(g[1]), gw, gw_m, torch.float32)
    if bias:
        check("grad_bias", host(g[2]), gb, gb_m, torch.float32)
    else:
        assert g[2] is None


def test_conv_equal_lengths_match_packed_bitwise():
    a = conv_case([70, 70, 70], 136, 4, torch.bfloat16, True, True)
    x, w, b = dev(a["x"], torch.bfloat16), dev(a["w"]), dev(a["bias"])
    c1, c2 = dev(a["cache"]), dev(a["cache"])
    y1 = kda.ssm_conv_fwd(x, w, b, c1, dev(a["cu"], torch.int32))
    y2 = kda.ssm_conv_fwd(x.view(3, 70, 136), w, b, c2)
    torch.cuda.synchronize()
    assert torch.equal(y1, y2.view(210, 136)) and torch.equal(c1, c2)


def test_conv_rows_of_no_sequence_stay():
    """Rows before the first and behind the last sequence keep what they held,
    and NaN in them goes nowhere."""
    a = conv_case([20, 9], 64, 4, torch.float32, False, True)
    x = torch.full((50, 64), float("nan"), device="cuda")
    gy = x.clone()
    x[7:36], gy[7:36] = dev(a["x"]), dev(a["gy"])
    cu = dev(a["cu"] + 7, torch.int32)
    y = torch.full((50, 64), 5.0, device="cuda")
    kda.ssm_conv_fwd(x, dev(a["w"]), dev(a["bias"]), None, cu, y=y)
    g = kda.ssm_conv_bwd(x, dev(a["w"]), dev(a["bias"]), gy, None, cu)
    torch.cuda.synchronize()
    assert (y[:7] == 5).all() and (y[36:] == 5).all() and torch.isfinite(y).all()
    assert torch.isfinite(g[0][7:36]).all() and torch.isfinite(g[1]).all() and torch.isfinite(g[2]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,Tr,c,W,commit", [(1, 1, 0, 8, 4, True), (5, 3, 4, 72, 4, False), (3, 64, 64, 16, 2, True),
                                               (4, 2, 7, 40, 3, False), (2, 0, 5, 8, 4, True)])
def test_conv_step(B, T, Tr, c, W, commit, dtype):
    r = np.random.default_rng(B + T)
    x, rx = q(r.standard_normal((B, T, c)), dtype), q(r.standard_normal((B, Tr, c)), dtype)
    w, b = np.float32(r.standard_normal((c, W))), np.float32(r.standard_normal(c))
    cache = np.float32(r.standard_normal((B, W - 1, c)))
    nr = r.integers(-2, Tr + 3, B)      # clamped into [0, Tr]
    cd, rxd = dev(cache), dev(rx, dtype)
    for n in range(B):                  # tokens that were not accepted hold NaN
        rxd[n, max(0, min(Tr, nr[n])):] = float("nan")
    y = kda.ssm_conv_step(dev(x, dtype), dev(w), dev(b), cd, replay=rxd if Tr else None,
                          n_replay=dev(nr, torch.int32) if Tr else None, commit=commit)
    torch.cuda.synchronize()
    for n in range(B):
        k = max(0, min(Tr, int(nr[n])))
        _, mid = O.conv(rx[n, :k], w, b, cache[n])
        ref, end = O.conv(x[n], w, b, mid)
        mag, _ = O.conv(np.abs(x[n]), np.abs(w), np.abs(b), np.abs(mid), False)
        check("y", host(y[n]), ref, mag, dtype, rounded=False)
        assert np.array_equal(host(cd[n]), end if commit else mid)


# ------------------------------------------------------------------- scan

def scan_case(lens, H, G, N, P, dtype, seed=0, amin=1.0, amax=16.0):
    r = np.random.default_rng(seed)
    T = sum(lens)
    f = lambda a: np.float32(a).astype(np.float64)   # noqa: E731
    return dict(x=q(r.standard_normal((T, H, P)), dtype), dt=f(r.standard_normal((T, H))), A=f(-r.uniform(amin, amax, H)),
                B=q(r.standard_normal((T, G, N)), dtype), C=q(r.standard_normal((T, G, N)), dtype),
                D=f(r.standard_normal(H)), S0=f(r.standard_normal((len(lens), H, N, P))),
                dt_bias=f(r.uniform(-6, -2, H)), gy=q(r.standard_normal((T, H, P)), dtype),
                gS=f(r.standard_normal((len(lens), H, N, P))), cu=np.concatenate([[0], np.cumsum(lens)]))


def wide_parts(a, dtype, names=("x", "B", "C")):
    """x, B and C as parts of the same rows, with NaN around them."""
    T = a["x"].shape[0]
    parts = [dev(a[n], dtype).reshape(T, int(np.prod(a[n].shape[1:]))) for n in names]
    w = sum(p.shape[1] for p in parts)
    buf = torch.full((T, w + 24), float("nan"), dtype=dtype, device="cuda")
    out, at = [], 8
    for n, p in zip(names, parts):
        v = buf[:, at:at + p.shape[1]]
        v.copy_(p)
        out.append(v.view(a[n].shape) if v.is_contiguous() else v.unflatten(1, a[n].shape[1:]))
        at += p.shape[1]
    return out


def oracle_scan(a, use, back=False, soft=True):
    """Reference and magnitude, all sequences."""
    y, ym, S, Sm, g, gm = [], [], [], [], [], []
    ab = {k: None if v is None else np.abs(v) for k, v in a.items()}
    # magnitudes: absolute values of everything but the decay
    for n, (s, e) in enumerate(zip(a["cu"], a["cu"][1:])):
        D, S0, bias = (a["D"] if "D" in use else None), (a["S0"][n] if "S0" in use else None), \
            (a["dt_bias"] if "dt_bias" in use else None)
        aD, aS0 = None if D is None else np.abs(D), None if S0 is None else np.abs(S0)
        r = O.scan(a["x"][s:e], a["dt"][s:e], a["A"], a["B"][s:e], a["C"][s:e], D, S0, bias, soft)
        m = O.scan(ab["x"][s:e], a["dt"][s:e], a["A"], ab["B"][s:e], ab["C"][s:e], aD, aS0, bias, soft)
        y.append(r[0]), S.append(r[1]), ym.append(m[0]), Sm.append(m[1])
        if back:
            gS = a["gS"][n] if "gS" in use else None
            g.append(O.scan_backward(a["x"][s:e], a["dt"][s:e], a["A"], a["B"][s:e], a["C"][s:e], D, S0, a["gy"][s:e],
                                     gS, bias, soft))
            gm.append(grad_magnitude(a, ab, s, e, aD, aS0, ab["gy"][s:e], None if gS is None else np.abs(gS), bias, soft))
    return y, ym, S, Sm, g, gm


def grad_magnitude(a, ab, s, e, aD, aS0, agy, agS, bias, soft):
    """Bounds of the sums of absolute terms.  A is negative: with the sign of
    A turned in ddt = into . B + A da both parts add up."""
    p = O.scan_backward(ab["x"][s:e], a["dt"][s:e], a["A"], ab["B"][s:e], ab["C"][s:e], aD, aS0, agy, agS, bias, soft)
    # the part through the decay alone, from dA's terms: dt da summed; per
    # token it is (into . B - ddt) / |A|
    x, d = ab["x"][s:e], O._dt(a["dt"][s:e], bias, soft)[1]
    T, H, P = x.shape
    into = np.einsum("thp,thp->th", p["x"] - (0 if aD is None else aD[:, None] * agy), x) / np.maximum(d, 1e-300)
    raw = O._dt(a["dt"][s:e], bias, soft)[0]
    sg = O.sigmoid(raw) if soft else np.ones_like(raw)
    decay = into - p["dt"] / sg
    # sums over a chunk share their terms: bound a token by its chunk's largest
    p["dt"] = sg * (np.abs(into) + 4 * np.max(np.abs(decay), 0, keepdims=True, initial=0.0))
    p["A"] = (d * np.max(np.abs(decay) / np.abs(a["A"]), 0, keepdims=True, initial=0.0)).sum(0) * 4
    p["bias"] = p["dt"].sum(0)
    return p


SCAN = [([1], 1, 1, 64, 64), ([0, 1, 2, 63, 64, 65, 130, 0], 6, 2, 128, 64), ([200, 31, 33], 3, 1, 64, 128),
        ([129], 5, 5, 128, 128), ([97, 0, 64], 7, 1, 128, 64)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,H,G,N,P", SCAN)
def test_scan_packed(lens, H, G, N, P, dtype):
    a = scan_case(lens, H, G, N, P, dtype)
    x, B, C = wide_parts(a, dtype)
    say(f"[ssm] scan {lens} H={H} G={G} N={N} P={P} {dtype}")
    y, S = kda.ssm_chunk_fwd(x, dev(a["dt"]), dev(a["A"]), B, C, dev(a["D"]), dev(a["S0"]),
                             dev(a["cu"], torch.int32), dt_bias=dev(a["dt_bias"]))
    torch.cuda.synchronize()
    ry, my, rS, mS, _, _ = oracle_scan(a, ("D", "S0", "dt_bias"))
    w = check("y", host(y), np.concatenate(ry), np.concatenate(my), dtype)
    v = check("S_T", host(S), np.stack(rS), np.stack(mS), torch.float32)
    say(f"[ssm]   y {w:.2f}, S_T {v:.2f} of the tolerance")


@pytest.mark.parametrize("use", [(), ("D",), ("S0",), ("dt_bias",)])
def test_scan_optional_arguments(use):
    a = scan_case([70, 5], 4, 2, 64, 64, torch.bfloat16, seed=2)
    a["dt"] = np.abs(a["dt"]) * 0.1
    soft = "dt_bias" in use
    y, S = kda.ssm_chunk_fwd(dev(a["x"], torch.bfloat16), dev(a["dt"]), dev(a["A"]), dev(a["B"], torch.bfloat16),
                             dev(a["C"], torch.bfloat16), dev(a["D"]) if "D" in use else None,
                             dev(a["S0"]) if "S0" in use else None, dev(a["cu"], torch.int32),
                             dt_bias=dev(a["dt_bias"]) if soft else None, softplus=soft)
    torch.cuda.synchronize()
    ry, my, rS, mS, _, _ = oracle_scan(a, use, soft=soft)
    check("y", host(y), np.concatenate(ry), np.concatenate(my), torch.bfloat16)
    check("S_T", host(S), np.stack(rS), np.stack(mS), torch.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_scan_segments_and_one_chain(dtype):
    """A long sequence with few heads is cut into segments; both ways agree
    with the oracle, and S_T may be S0."""
    a = scan_case([2500], 2, 1, 64, 64, dtype, seed=5, amin=0.01, amax=0.1)
    assert kda.ssm_chunk_fwd_workspace_bytes(1, 2500, 2, 1, 64, 64, False) > 0
    ry, my, rS, mS, _, _ = oracle_scan(a, ("D", "S0"))
    t = {k: dev(a[k], dtype)[None] for k in ("x", "B", "C")}
    for cut in (True, False):
        for cu in (None, dev(a["cu"], torch.int32)):
            S = dev(a["S0"])
            y, S = kda.ssm_chunk_fwd(t["x"], dev(a["dt"])[None], dev(a["A"]), t["B"], t["C"], dev(a["D"]), S, cu, S_T=S,
                                     sequence_parallel=cut)
            torch.cuda.synchronize()
            check("y", host(y[0]), ry[0], my[0], dtype)
            check("S_T", host(S[0]), rS[0], mS[0], torch.float32)


def test_scan_ragged_segments():
    lens = [0, 700, 3, 1400, 0, 512, 0]
    a = scan_case(lens, 2, 2, 64, 64, torch.bfloat16, seed=6, amin=0.01, amax=0.3)
    assert kda.ssm_chunk_fwd_workspace_bytes(len(lens), sum(lens), 2, 2, 64, 64, True) > 0
    y, S = kda.ssm_chunk_fwd(dev(a["x"], torch.bfloat16), dev(a["dt"]), dev(a["A"]), dev(a["B"], torch.bfloat16),
                             dev(a["C"], torch.bfloat16), None, dev(a["S0"]), dev(a["cu"], torch.int32))
    torch.cuda.synchronize()
    ry, my, rS, mS, _, _ = oracle_scan(a, ("S0",))
    check("y", host(y), np.concatenate(ry), np.concatenate(my), torch.bfloat16)
    check("S_T", host(S), np.stack(rS), np.stack(mS), torch.float32)


@pytest.mark.parametrize("n", [64, 65, 200])
def test_scan_many_short_sequences(n):
    """Around the number of sequences up to which chains start with the
    longest, forward and backward."""
    lens = [int(v) for v in np.random.default_rng(n).integers(0, 70, n) // np.random.default_rng(n + 1).integers(1, 12, n)]
    lens[3] = lens[5] = 70
    a = scan_case(lens, 2, 1, 64, 64, torch.bfloat16, seed=33)
    use = ("S0", "gS")
    y, S = kda.ssm_chunk_fwd(dev(a["x"], torch.bfloat16), dev(a["dt"]), dev(a["A"]), dev(a["B"], torch.bfloat16),
                             dev(a["C"], torch.bfloat16), None, dev(a["S0"]), dev(a["cu"], torch.int32))
    r = run_bwd(a, torch.bfloat16, use)
    torch.cuda.synchronize()
    ry, my, rS, mS, _, _ = oracle_scan(a, ("S0",))
    check("y", host(y), np.concatenate(ry), np.concatenate(my), torch.bfloat16)
    check("S_T", host(S), np.stack(rS), np.stack(mS), torch.float32)
    check_bwd(r, a, use, torch.bfloat16)


@pytest.mark.parametrize("case", ["strong", "none", "mixed"])
def test_scan_extreme_decay(case):
    """Decays that wipe the state out within a token, none at all, and a huge
    one followed by tiny ones (the sums within a chunk must not lose them)."""
    a = scan_case([150], 2, 1, 64, 64, torch.float32, seed=7)
    a["A"] = np.array([-1.0, -1.0])
    a["dt"] = np.full((150, 2), 0.01)
    if case == "strong":
        a["dt"][:] = 300.0
        a["x"] /= 300.0
        a["x"] = q(a["x"], torch.float32)
    elif case == "none":
        a["A"][:] = 0.0
    else:
        a["dt"][3::64] = 20000.0
        a["x"][3::64] = 0.0
    a["dt"] = np.float32(a["dt"]).astype(np.float64)
    y, S = kda.ssm_chunk_fwd(dev(a["x"]), dev(a["dt"]), dev(a["A"]), dev(a["B"]), dev(a["C"]), None, dev(a["S0"]),
                             dev(a["cu"], torch.int32), softplus=False)
    torch.cuda.synchronize()
    ry, my, rS, mS, _, _ = oracle_scan(a, ("S0",), soft=False)
    check("y", host(y), ry[0], my[0], torch.float32)
    check("S_T", host(S[0]), rS[0], mS[0], torch.float32)


BWD = [([1], 1, 1, 64, 64), ([0, 1, 2, 63, 64, 65, 130, 0], 6, 2, 128, 64), ([100, 31, 33], 3, 1, 64, 128),
       ([129], 4, 4, 128, 128), ([97, 0, 64], 7, 1, 128, 64)]


def run_bwd(a, dtype, use, soft=True, cu=True, **kw):
    x, B, C = wide_parts(a, dtype)
    return kda.ssm_chunk_bwd(x, dev(a["dt"]), dev(a["A"]), B, C, dev(a["D"]) if "D" in use else None,
                             dev(a["S0"]) if "S0" in use else None, dev(a["gy"], dtype),
                             dev(a["gS"]) if "gS" in use else None, dev(a["cu"], torch.int32),
                             dt_bias=dev(a["dt_bias"]) if "dt_bias" in use else None, softplus=soft, **kw)


def check_bwd(r, a, use, dtype, soft=True):
    _, _, _, _, g, m = oracle_scan(a, use, back=True, soft=soft)
    cat = lambda k, which: np.concatenate([d[k] for d in which])   # noqa: E731
    tot = lambda k, which: sum(d[k] for d in which)                # noqa: E731
    gx, gdt, gA, gB, gC, gD, gb, gS0 = r
    w = {}
    for name, t, k in (("grad_x", gx, "x"), ("grad_B", gB, "B"), ("grad_C", gC, "C")):
        w[name] = check(name, host(t), cat(k, g), cat(k, m), dtype)
    w["grad_dt"] = check("grad_dt", host(gdt), cat("dt", g), cat("dt", m), torch.float32)
    w["grad_A"] = check("grad_A", host(gA), tot("A", g), tot("A", m), torch.float32)
    if "D" in use:
        w["grad_D"] = check("grad_D", host(gD), tot("D", g), tot("D", m), torch.float32)
    if "dt_bias" in use:
        w["grad_bias"] = check("grad_bias", host(gb), tot("bias", g), tot("bias", m), torch.float32)
    if gS0 is not None:
        w["grad_S0"] = check("grad_S0", host(gS0), np.stack([d["S0"] for d in g]), np.stack([d["S0"] for d in m]),
                             torch.float32)
    say("[ssm]   " + " ".join(f"{k} {v:.2f}" for k, v in w.items()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,H,G,N,P", BWD)
def test_scan_backward_packed(lens, H, G, N, P, dtype):
    a = scan_case(lens, H, G, N, P, dtype, seed=9, amin=0.1, amax=4.0)
    say(f"[ssm] scan backward {lens} H={H} G={G} N={N} P={P} {dtype}")
    use = ("D", "S0", "gS", "dt_bias")
    r = run_bwd(a, dtype, use)
    torch.cuda.synchronize()
    check_bwd(r, a, use, dtype)


@pytest.mark.parametrize("use,soft", [((), False), (("D", "dt_bias"), True), (("S0", "gS"), False)])
def test_scan_backward_optional_arguments(use, soft):
    a = scan_case([70, 5], 4, 2, 64, 64, torch.float32, seed=10)
    a["dt"] = np.abs(a["dt"]) * (0.1 if not soft else 1.0)
    a["dt"] = np.float32(a["dt"]).astype(np.float64)
    r = run_bwd(a, torch.float32, use, soft)
    torch.cuda.synchronize()
    check_bwd(r, a, use, torch.float32, soft)


def test_scan_backward_long_and_by_groups():
    """Segments in the walks; and with the smallest workspace, one group of
    heads at a time, the same gradients bitwise for the outputs whose sums do
    not depend on the split of heads."""
    a = scan_case([1300, 0, 900], 4, 2, 64, 64, torch.bfloat16, seed=11, amin=0.01, amax=0.2)
    use = ("D", "S0", "gS", "dt_bias")
    r = run_bwd(a, torch.bfloat16, use)
    torch.cuda.synchronize()
    check_bwd(r, a, use, torch.bfloat16)
    small = kda.ssm_chunk_bwd_workspace_bytes(torch.bfloat16, 3, 2200, 4, 2, 64, 64, True, groups=1)
    full = kda.ssm_chunk_bwd_workspace_bytes(torch.bfloat16, 3, 2200, 4, 2, 64, 64, True)
    assert small < full
    r2 = run_bwd(a, torch.bfloat16, use, workspace=torch.empty(small, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    check_bwd(r2, a, use, torch.bfloat16)


def reset_case(dtype, dt, A):
    """Every 21st token and the chunks' borders end all memory: a = dt A with
    e^a = 0 in float32, x there scaled so that its own term is of the others'
    size (dt x ~ 1)."""
    a = scan_case([200, 3, 64], 2, 1, 64, 64, dtype, seed=31, amin=0.5, amax=2.0)
    T = a["x"].shape[0]
    at = np.unique(np.concatenate([np.arange(5, T, 21), [0, 63, 64, 127, 199, 200, 202, 266]]))
    a["A"] = np.float32(a["A"] * A).astype(np.float64)
    a["dt"] = np.float32(np.abs(a["dt"]) * 0.1 / A).astype(np.float64)
    a["dt"][at] = np.float32(dt)
    a["x"][at] = q(a["x"][at] / dt, dtype) if dt < 1e30 else 0.0
    return a, at


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dt,A", [(1e4, 1.0), (2.0 ** 40, 1.0), (1e37, 100.0)])
def test_scan_resets(dt, A, dtype):
    """However large dt |A|, up to a product beyond float32, the tokens after
    a reset keep their own decays."""
    a, _ = reset_case(dtype, dt, A)
    y, S = kda.ssm_chunk_fwd(dev(a["x"], dtype), dev(a["dt"]), dev(a["A"]), dev(a["B"], dtype), dev(a["C"], dtype), None,
                             dev(a["S0"]), dev(a["cu"], torch.int32), softplus=False)
    torch.cuda.synchronize()
    ry, my, rS, mS, _, _ = oracle_scan(a, ("S0",), soft=False)
    check("y", host(y), np.concatenate(ry), np.concatenate(my), dtype)
    check("S_T", host(S), np.stack(rS), np.stack(mS), torch.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dt", [1e4, 2.0 ** 40])
def test_scan_backward_resets(dt, dtype):
    """A token that ends all memory has da = 0: grad_A = sum dt da is of the
    other tokens' size, however large dt there is."""
    a, at = reset_case(dtype, dt, 1.0)
    use = ("S0", "gS")
    r = run_bwd(a, dtype, use, soft=False)
    torch.cuda.synchronize()
    check_bwd(r, a, use, dtype, soft=False)
    _, _, _, _, g, _ = oracle_scan(a, use, back=True, soft=False)
    rest = dict(a, dt=a["dt"].copy())
    rest["dt"][at] = 1.0   # the tolerance of tokens with ordinary steps only
    _, _, _, _, _, m = oracle_scan(rest, use, back=True, soft=False)
    check("grad_A", host(r[2]), sum(d["A"] for d in g), sum(d["A"] for d in m), torch.float32)


def test_scan_backward_against_differences():
    """The directional derivative of the float32 forward pass.  A step h of
    2^-9 leaves h^2 of the third derivative and 2 y's rounding over h: a
    tolerance of 2e-3 of the sums of absolute terms covers both."""
    a = scan_case([90], 2, 1, 64, 64, torch.float32, seed=12, amin=0.5, amax=2.0)
    use = ("D", "S0", "gS", "dt_bias")
    gx, gdt, gA, gB, gC, gD, gb, gS0 = run_bwd(a, torch.float32, use)
    grads = dict(x=gx, dt=gdt, A=gA, B=gB, C=gC, D=gD, dt_bias=gb, S0=gS0)
    r = np.random.default_rng(13)
    cu = dev(a["cu"], torch.int32)

    def loss(b):
        y, S = kda.ssm_chunk_fwd(dev(b["x"]), dev(b["dt"]), dev(b["A"]), dev(b["B"]), dev(b["C"]), dev(b["D"]),
                                 dev(b["S0"]), cu, dt_bias=dev(b["dt_bias"]))
        return (host(y) * a["gy"]).sum() + (host(S) * a["gS"]).sum()

    h = 2.0 ** -9
    for name, g in grads.items():
        v = r.choice([-1.0, 1.0], a[name].shape)
        d = (loss({**a, name: a[name] + h * v}) - loss({**a, name: a[name] - h * v})) / (2 * h)
        want = (host(g) * v).sum()
        assert abs(d - want) <= 2e-3 * np.sqrt((host(g) ** 2).sum()) + 1e-3 * abs(want), name


def test_scan_rows_of_no_sequence_stay():
    a = scan_case([70, 9], 2, 1, 64, 64, torch.bfloat16, seed=14)
    T = 100

    def within(v, fill):
        t = torch.full((T,) + v.shape[1:], fill, dtype=torch.bfloat16 if v.ndim == 3 else torch.float32, device="cuda")
        t[5:84] = dev(v, t.dtype)
        return t

    x, B, C, dt, gy = (within(a[k], float("nan")) for k in ("x", "B", "C", "dt", "gy"))
    cu = dev(a["cu"] + 5, torch.int32)
    y = torch.full_like(x, 3.0)
    _, S = kda.ssm_chunk_fwd(x, dt, dev(a["A"]), B, C, dev(a["D"]), dev(a["S0"]), cu, y=y)
    gx, gB, gC = (torch.full_like(t, 3.0) for t in (x, B, C))
    r = kda.ssm_chunk_bwd(x, dt, dev(a["A"]), B, C, dev(a["D"]), dev(a["S0"]), gy, None, cu, grad_x=gx, grad_B=gB,
                          grad_C=gC)
    torch.cuda.synchronize()
    for t in (y, gx, gB, gC):
        assert torch.isfinite(t).all() and (t[:5] == 3).all() and (t[84:] == 3).all()
    assert torch.isfinite(r[1][5:84]).all() and torch.isfinite(r[2]).all() and torch.isfinite(S).all()
    ry, my, _, _, _, _ = oracle_scan(a, ("D", "S0"))
    check("y", host(y[5:84]), np.concatenate(ry), np.concatenate(my), torch.bfloat16)


@pytest.mark.parametrize("op", ["conv", "scan", "bwd"])
def test_captured_graph_replays(op):
    """A captured call replays with new inputs in the same buffers, with
    eager work between the replays."""
    a = scan_case([1200], 2, 1, 64, 64, torch.bfloat16, seed=15, amin=0.01, amax=0.2)
    t = {k: dev(a[k], torch.bfloat16)[None] for k in ("x", "B", "C", "gy")}
    dt, A, D, S0, gS = (dev(a[k]) for k in ("dt", "A", "D", "S0", "gS"))
    dt = dt[None]
    cx, w, cache = dev(a["x"], torch.bfloat16).view(1, 1200, 128), torch.randn(128, 4, device="cuda"), None

    def go():
        if op == "conv":
            return (kda.ssm_conv_fwd(cx, w, None, cache),) + kda.ssm_conv_bwd(cx, w, None, cx, None)[:2]
        if op == "scan":
            return kda.ssm_chunk_fwd(t["x"], dt, A, t["B"], t["C"], D, S0)
        return tuple(kda.ssm_chunk_bwd(t["x"], dt, A, t["B"], t["C"], D, S0, t["gy"], gS)[:6])

    go()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        go()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = go()
    for k in range(3):
        (cx if op == "conv" else t["x"]).normal_()
        g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        want = go()
        torch.cuda.synchronize()
        assert all(torch.equal(i, j) for i, j in zip(got, want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_padded_batch(dtype):
    """Sequences padded with tokens of dt = 0 give the packed batch's outputs,
    states and gradients."""
    lens, T, H, G, N, P = [150, 64, 3], 160, 4, 2, 64, 64
    a = scan_case(lens, H, G, N, P, dtype, seed=42)
    t = {k: dev(a[k], torch.float32 if k == "dt" else dtype) for k in ("x", "dt", "B", "C", "gy")}
    A, D, S0, gS, cu = dev(a["A"]), dev(a["D"]), dev(a["S0"]), dev(a["gS"]), dev(a["cu"], torch.int32)
    pad = {}
    for k, v in t.items():
        pad[k] = torch.full((len(lens), T) + v.shape[1:], {"dt": -1e4, "gy": 0.0}.get(k, 3.0), dtype=v.dtype, device="cuda")
        for i, (s, e) in enumerate(zip(a["cu"], a["cu"][1:])):
            pad[k][i, :e - s] = v[s:e]
    real = lambda v: torch.cat([v[i, :n] for i, n in enumerate(lens)])   # noqa: E731
    y, S = kda.ssm_chunk_fwd(t["x"], t["dt"], A, t["B"], t["C"], D, S0, cu, sequence_parallel=False)
    yp, Sp = kda.ssm_chunk_fwd(pad["x"], pad["dt"], A, pad["B"], pad["C"], D, S0, sequence_parallel=False)
    r = kda.ssm_chunk_bwd(t["x"], t["dt"], A, t["B"], t["C"], D, S0, t["gy"], gS, cu)
    rp = kda.ssm_chunk_bwd(pad["x"], pad["dt"], A, pad["B"], pad["C"], D, S0, pad["gy"], gS)
    torch.cuda.synchronize()
    assert torch.equal(real(yp), y) and torch.equal(Sp, S)
    # The packed rows and the padded ones are cut into other segments, up to
    # four, whose states pass through two more roundings each: 8 half steps,
    # 5e-7 of the largest state; and the input type's own rounding, once.
    torch.testing.assert_close(rp[7], r[7], rtol=0, atol=1e-5 * float(r[7].abs().max()))
    for i in (0, 1, 3, 4):
        got, want = real(rp[i]).float(), r[i].float()
        torch.testing.assert_close(got, want, rtol=2 ** -7 if dtype == torch.bfloat16 and i != 1 else 1e-5,
                                   atol=1e-5 * float(want.abs().max()))
    for i in (2, 5):
        torch.testing.assert_close(rp[i], r[i], rtol=1e-5, atol=1e-5 * float(r[1].abs().max()))


def test_sequences_without_tokens():
    """T = 0: states and caches stay, gradients of the parameters are zero and
    the state's passes through; no sequences at all: nothing."""
    H, N, P, c, n = 3, 64, 64, 24, 2
    f = lambda *s: torch.randn(*s, device="cuda")   # noqa: E731
    A, D, S0, gS = -torch.rand(H, device="cuda"), f(H), f(n, H, N, P), f(n, H, N, P)
    x, dt, B = f(n, 0, H, P), f(n, 0, H), f(n, 0, 1, N)
    cu = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    for a, packed in (((x, dt, A, B, B), None), ((x[0], dt[0], A, B[0], B[0]), cu)):
        y, S = kda.ssm_chunk_fwd(*a, D, S0, packed)
        assert y.shape == a[0].shape and torch.equal(S, S0)
        r = kda.ssm_chunk_bwd(*a, D, S0, a[0], gS, packed, dt_bias=D)
        assert torch.equal(r[7], gS) and all(not t.any() for t in (r[2], r[5], r[6]))
    w, bias, cache = f(c, 4), f(c), f(n, 3, c)
    old = cache.clone()
    for v, packed in ((f(n, 0, c), None), (f(0, c), cu)):
        assert kda.ssm_conv_fwd(v, w, bias, cache, packed).shape == v.shape and torch.equal(cache, old)
        g = kda.ssm_conv_bwd(v, w, bias, v, cache, packed)
        assert all(not t.any() for t in g[1:])
    assert kda.ssm_conv_step(f(n, 0, c), w, bias, cache).numel() == 0 and torch.equal(cache, old)
    none = kda.ssm_chunk_bwd(x[:0], dt[:0], A, B[:0], B[:0], D, S0[:0], x[:0])
    assert not none[2].any() and not none[5].any()
    na, tok = kda.verify_drafts(f(0, 3, 9), torch.zeros(0, 2, dtype=torch.int32, device="cuda"), f(0, 2), f(0))
    torch.cuda.synchronize()
    assert na.shape == (0,) and tok.shape == (0, 3)


@pytest.mark.parametrize("lens", [[130, 0, 65], [700]])
def test_given_outputs_and_state_gradient_in_place(lens):
    """Outputs and workspaces of the caller, too long a workspace among them,
    and grad_S0 written over grad_S_T through the C ABI (with and without
    segments)."""
    a = scan_case(lens, 2, 1, 64, 64, torch.bfloat16, seed=41)
    b = torch.bfloat16
    t = {k: dev(a[k], b) for k in ("x", "B", "C", "gy")}
    f = {k: dev(a[k]) for k in ("dt", "A", "D", "S0", "gS")}
    cu, n, T = dev(a["cu"], torch.int32), len(lens), sum(lens)
    args = (t["x"], f["dt"], f["A"], t["B"], t["C"], f["D"], f["S0"])
    y, S = kda.ssm_chunk_fwd(*args, cu)
    ws = torch.empty(kda.ssm_chunk_fwd_workspace_bytes(n, T, 2, 1, 64, 64, True) + 4096, dtype=torch.uint8, device="cuda")
    y2, S2 = torch.empty_like(y), torch.empty_like(S)
    out = kda.ssm_chunk_fwd(*args, cu, y=y2, S_T=S2, workspace=ws)
    torch.cuda.synchronize()
    assert out[0] is y2 and out[1] is S2 and torch.equal(y, y2) and torch.equal(S, S2)
    want = kda.ssm_chunk_bwd(*args, t["gy"], f["gS"], cu)
    lib = kda.load_library()
    need = kda.ssm_chunk_bwd_workspace_bytes(b, n, T, 2, 1, 64, 64, True)
    ws = torch.empty(need + 4096, dtype=torch.uint8, device="cuda")
    g = [torch.empty_like(v) for v in (t["x"], t["B"], t["C"], f["dt"], f["A"], f["D"])]
    state = f["gS"].clone()
    p = lambda v: v.data_ptr()   # noqa: E731
    rc = lib.kda_ssm_chunk_bwd(p(t["x"]), 128, p(t["B"]), 64, p(t["C"]), 64, kda.KDA_BF16, p(f["dt"]), None, 1, p(f["A"]),
                               p(f["D"]), p(f["S0"]), p(cu), n, T, 2, 1, 64, 64, p(t["gy"]), p(state), p(g[0]), 128, p(g[1]),
                               64, p(g[2]), 64, p(g[3]), p(g[4]), p(g[5]), None, p(state), p(ws), ws.numel(),
                               torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0
    for got, ref in zip(g + [state], (want[0], want[3], want[4], want[1], want[2], want[5], want[7])):
        assert torch.equal(got, ref)


def test_two_streams_at_once():
    """Two calls in flight on two streams give the bits of each alone."""
    runs = []
    for seed in (16, 17):
        a = scan_case([900, 400], 4, 1, 128, 64, torch.bfloat16, seed=seed)
        args = (dev(a["x"], torch.bfloat16), dev(a["dt"]), dev(a["A"]), dev(a["B"], torch.bfloat16),
                dev(a["C"], torch.bfloat16), dev(a["D"]), dev(a["S0"]))
        runs.append((args, dev(a["gy"], torch.bfloat16), dev(a["cu"], torch.int32)))

    def go(r):
        args, gy, cu = r
        return list(kda.ssm_chunk_fwd(*args, cu)) + list(kda.ssm_chunk_bwd(*args, gy, None, cu))[:6]

    alone = [go(r) for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    both = []
    for s, r in zip(streams, runs):
        with torch.cuda.stream(s):
            both.append(go(r))
    torch.cuda.synchronize()
    for i, j in zip(alone, both):
        assert all(torch.equal(x, y) for x, y in zip(i, j))


# -------------------------------------------------------------- recurrent

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,Tr,H,G,N,P,commit", [(1, 1, 0, 1, 1, 64, 64, True), (3, 5, 4, 6, 2, 128, 64, False),
                                                   (2, 64, 64, 2, 1, 64, 128, True), (4, 3, 9, 3, 3, 128, 128, False),
                                                   (2, 0, 5, 2, 1, 128, 64, True), (2, 9, 0, 2, 1, 64, 64, False)])
def test_recurrent(B, T, Tr, H, G, N, P, commit, dtype):
    new = scan_case([T] * B, H, G, N, P, dtype, seed=20)
    old = scan_case([Tr] * B, H, G, N, P, dtype, seed=21)
    r = np.random.default_rng(22)
    nr = r.integers(-1, Tr + 2, B)
    S = dev(new["S0"])
    x, Bm, C = (v.unflatten(0, (B, T)) for v in wide_parts(new, dtype))
    replay = None
    if Tr:
        rx, rB = (v.unflatten(0, (B, Tr)) for v in wide_parts(old, dtype, ("x", "B")))
        for n in range(B):
            rx[n, max(0, min(Tr, nr[n])):] = float("nan")    # drafts that fell
        replay = (rx, dev(old["dt"]).view(B, Tr, H), rB)
    y = kda.ssm_recurrent_fwd(x, dev(new["dt"]).view(B, T, H), dev(new["A"]), Bm, C, S, dev(new["D"]),
                              dt_bias=dev(new["dt_bias"]), replay=replay,
                              n_replay=dev(nr, torch.int32) if Tr else None, commit=commit)
    torch.cuda.synchronize()
    for n in range(B):
        k = max(0, min(Tr, int(nr[n])))
        sl, so = slice(n * T, (n + 1) * T), slice(n * Tr, n * Tr + k)
        ab = np.abs
        _, mid = O.scan(old["x"][so], old["dt"][so], new["A"], old["B"][so], old["C"][so], None, new["S0"][n],
                        new["dt_bias"])
        _, mid_m = O.scan(ab(old["x"][so]), old["dt"][so], new["A"], ab(old["B"][so]), ab(old["C"][so]), None,
                          ab(new["S0"][n]), new["dt_bias"])
        ry, end = O.scan(new["x"][sl], new["dt"][sl], new["A"], new["B"][sl], new["C"][sl], new["D"], mid, new["dt_bias"])
        my, end_m = O.scan(ab(new["x"][sl]), new["dt"][sl], new["A"], ab(new["B"][sl]), ab(new["C"][sl]), ab(new["D"]),
                           mid_m, new["dt_bias"])
        check("y", host(y[n]), ry, my, dtype, rounded=False)
        check("S", host(S[n]), end if commit else mid, end_m if commit else mid_m, torch.float32)


def test_recurrent_continues_the_scan():
    """Prompt, then tokens one by one: the outputs of the whole sequence."""
    a = scan_case([130], 4, 2, 128, 64, torch.float32, seed=23)
    t = {k: dev(a[k])[None] for k in ("x", "B", "C", "dt")}
    A, D, bias = dev(a["A"]), dev(a["D"]), dev(a["dt_bias"])
    ry, my, rS, mS, _, _ = oracle_scan(a, ("D", "S0", "dt_bias"))
    _, S = kda.ssm_chunk_fwd(t["x"][:, :100].contiguous(), t["dt"][:, :100].contiguous(), A, t["B"][:, :100].contiguous(),
                             t["C"][:, :100].contiguous(), D, dev(a["S0"]), dt_bias=bias)
    for i in range(100, 130):
        y = kda.ssm_recurrent_fwd(t["x"][:, i:i + 1], t["dt"][:, i:i + 1], A, t["B"][:, i:i + 1], t["C"][:, i:i + 1], S,
                                  D, dt_bias=bias)
        torch.cuda.synchronize()
        check("y", host(y[0]), ry[0][i:i + 1], my[0][i:i + 1], torch.float32)
    check("S", host(S[0]), rS[0], mS[0], torch.float32)


# ------------------------------------------------------------ all together

def test_layer_gradients_through_convolution_and_scan():
    """Training: convolution -> scan, and back through both, the scan's
    gradients written straight into the rows that the convolution's backward
    pass reads; against the oracle's chain in float32."""
    H, G, N, P, T = 4, 2, 64, 64, 150
    c = H * P + 2 * G * N
    r = np.random.default_rng(30)
    raw, w = q(r.standard_normal((T, c)), torch.float32), np.float32(r.standard_normal((c, 4)) / 4).astype(np.float64)
    a = scan_case([T], H, G, N, P, torch.float32, seed=31)
    cu = dev(a["cu"], torch.int32)

    def parts(t):
        x, B, C = t[:, :H * P], t[:, H * P:H * P + G * N], t[:, H * P + G * N:]
        f = (lambda v, n: v.unflatten(1, n)) if torch.is_tensor(t) else (lambda v, n: v.reshape((T,) + n))
        return f(x, (H, P)), f(B, (G, N)), f(C, (G, N))

    xr, wd = dev(raw), dev(w)
    xbc = kda.ssm_conv_fwd(xr, wd, None, None, cu)
    x, B, C = parts(xbc)
    y, _ = kda.ssm_chunk_fwd(x, dev(a["dt"]), dev(a["A"]), B, C, dev(a["D"]), None, cu)
    gxbc = torch.empty_like(xbc)
    gx, gB, gC = parts(gxbc)
    g = kda.ssm_chunk_bwd(x, dev(a["dt"]), dev(a["A"]), B, C, dev(a["D"]), None, dev(a["gy"]), None, cu, grad_x=gx,
                          grad_B=gB, grad_C=gC)
    gr = kda.ssm_conv_bwd(xr, wd, None, gxbc, None, cu)
    torch.cuda.synchronize()
    rx, _ = O.conv(raw, w)
    ox, oB, oC = parts(rx)
    ry, _ = O.scan(ox, a["dt"], a["A"], oB, oC, a["D"])
    og = O.scan_backward(ox, a["dt"], a["A"], oB, oC, a["D"], None, a["gy"])
    ogx = np.concatenate([og[k].reshape(T, -1) for k in ("x", "B", "C")], 1)
    oraw, ow, _, _ = O.conv_backward(raw, w, None, None, ogx)
    for name, t, ref in (("y", y, ry), ("grad_dt", g[1], og["dt"]), ("grad_A", g[2], og["A"]), ("grad_raw", gr[0], oraw),
                         ("grad_w", gr[1], ow)):
        err = np.abs(host(t) - ref).max() / np.abs(ref).max()
        say(f"[ssm]   {name} {err:.2e}")
        assert err < 1e-5, name


def test_speculative_decoding_loop():
    """Prompt, then steps of drafts -> convolution -> scan -> verification with
    the accepted counts replayed by the next step.  What stands in cache and
    state afterwards is that of the accepted tokens alone."""
    H, G, N, P, K, V, n = 2, 1, 64, 64, 3, 37, 4
    c = H * P + 2 * G * N
    r = np.random.default_rng(40)
    table = np.float32(r.standard_normal((V, c)))               # a token's row before the convolution
    tdt = np.float32(r.standard_normal((V, H)))
    head = dev(r.standard_normal((H * P, V)) / 8)
    w, bias = np.float32(r.standard_normal((c, 4)) / 2), np.float32(r.standard_normal(c))
    A, D = np.float32(-r.uniform(0.5, 2, H)), np.float32(r.standard_normal(H))
    td, dtd, wd, bd, Ad, Dd = dev(table), dev(tdt), dev(w), dev(bias), dev(A), dev(D)
    split = lambda t: (t[..., :H * P].unflatten(-1, (H, P)), t[..., H * P:H * P + N].unflatten(-1, (G, N)),   # noqa: E731
                       t[..., H * P + N:].unflatten(-1, (G, N)))
    cache, S = torch.zeros(n, 3, c, device="cuda"), torch.zeros(n, H, N, P, device="cuda")
    texts = [[] for _ in range(n)]
    last = torch.from_numpy(r.integers(0, V, n).astype(np.int32)).cuda()
    old, n_rep = None, None
    for step in range(5):
        drafts = torch.from_numpy(r.integers(0, V, (n, K)).astype(np.int32)).cuda()
        toks = torch.cat([last[:, None], drafts], 1).long()     # K + 1 tokens run
        raw, dt = td[toks], dtd[toks]
        xbc = kda.ssm_conv_step(raw, wd, bd, cache, replay=None if old is None else old[0], n_replay=n_rep, commit=False)
        x, B, C = split(xbc)
        rep = None
        if old is not None:
            ox, oB, _ = split(old[1])
            rep = (ox, old[2], oB)
        y = kda.ssm_recurrent_fwd(x, dt, Ad, B, C, S, Dd, replay=rep, n_replay=n_rep, commit=False)
        p = torch.softmax(y.reshape(n, K + 1, H * P) @ head, -1)
        u, un = (torch.from_numpy(np.float32(r.random(s))).cuda() for s in ((n, K), (n,)))
        uniform = torch.full((n, K, V), 1 / V, device="cuda")   # what the drafts are drawn from
        n_acc, out = kda.verify_drafts(p, drafts, u, un, uniform)
        for i in range(n):
            k = int(n_acc[i])
            texts[i] += [int(t) for t in toks[i, :k + 1]]
            assert [int(t) for t in out[i, :k]] == [int(t) for t in drafts[i, :k]] and (out[i, k + 1:] == -1).all()
        last = out[torch.arange(n, device="cuda"), n_acc.long()]
        old, n_rep = (raw, xbc, dt), n_acc + 1
    # bring cache and state up to the accepted tokens
    none = torch.empty(n, 0, c, device="cuda")
    kda.ssm_conv_step(none, wd, bd, cache, replay=old[0], n_replay=n_rep)
    x, B, C = split(torch.empty(n, 0, c, device="cuda"))
    ox, oB, _ = split(old[1])
    kda.ssm_recurrent_fwd(x, torch.empty(n, 0, H, device="cuda"), Ad, B, C, S, replay=(ox, old[2], oB), n_replay=n_rep)
    torch.cuda.synchronize()
    assert len({len(t) for t in texts}) > 1                     # requests went at their own pace
    for i, t in enumerate(texts):
        z, end = O.conv(table[t], w, bias)
        assert np.array_equal(host(cache[i]), end)
        x, B, C = z[:, :H * P].reshape(-1, H, P), z[:, H * P:H * P + N].reshape(-1, G, N), z[:, H * P + N:].reshape(-1, G, N)
        _, ref = O.scan(x, tdt[t], A, B, C, D)
        _, mag = O.scan(np.abs(x) + 1, tdt[t], A, np.abs(B) + 1, np.abs(C), D)
        check("S", host(S[i]), ref, mag, torch.float32)


def test_captured_decode_step():
    """Convolution, scan and verification captured as one graph: each replay
    reads the accepted counts that the replay before it left on the device
    and updates cache and state in place, as the eager calls do, bitwise."""
    H, G, N, P, K, V, n = 4, 2, 64, 64, 3, 1001, 3
    c, T = H * P + 2 * G * N, K + 1
    gen = torch.Generator(device="cuda").manual_seed(50)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)   # noqa: E731
    w, bias, A = rnd(c, 4) / 2, rnd(c), -torch.rand(H, device="cuda") - 0.1
    raw, dt = rnd(2, n, T, c).bfloat16(), rnd(2, n, T, H)
    p, un = torch.softmax(rnd(n, T, V), -1), torch.rand(n, device="cuda")
    u = torch.tensor([[0.0, 0, 0], [0, 1, 0], [1, 0, 0]], device="cuda")   # 0: the draft stands, 1: it does not
    drafts = torch.zeros(n, K, dtype=torch.int32, device="cuda")

    def split(t):
        return (t[..., :H * P].unflatten(-1, (H, P)), t[..., H * P:H * P + G * N].unflatten(-1, (G, N)),
                t[..., H * P + G * N:].unflatten(-1, (G, N)))

    def step(st):
        xbc = kda.ssm_conv_step(raw[0], w, bias, st["cache"], replay=raw[1], n_replay=st["acc"], commit=False)
        x, B, C = split(xbc)
        ox, oB, _ = split(st["old"])
        y = kda.ssm_recurrent_fwd(x, dt[0], A, B, C, st["S"], replay=(ox, dt[1], oB), n_replay=st["acc"], commit=False)
        acc, tok = kda.verify_drafts(p, drafts, u, un)
        st["acc"].copy_(acc)
        st["old"].copy_(xbc)
        return y, tok

    def fresh():
        return dict(cache=torch.ones(n, 3, c, device="cuda"), S=torch.ones(n, H, N, P, device="cuda"),
                    acc=torch.ones(n, dtype=torch.int32, device="cuda"),
                    old=torch.zeros(n, T, c, device="cuda", dtype=torch.bfloat16))

    warm = fresh()
    step(warm)
    torch.cuda.synchronize()
    a, b = fresh(), fresh()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(a)
    counts = set()
    for i in range(4):
        for t in (raw, dt, p):
            t.copy_(t.roll(1, -1))
        u.copy_(u.roll(1, 0))
        drafts.copy_(p[:, :K].argsort(-1, descending=True)[..., i].int())
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = step(b)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want))
        assert all(torch.equal(a[k], b[k]) for k in a)
        counts |= set(a["acc"].tolist())
    assert counts == {0, 1, 3}


def test_offsets_past_32_bits():
    """Tensors of more than 2^32 bytes (and elements past 2^31): what stands
    at their end is what the same call gives for it alone."""
    gen = torch.Generator(device="cuda").manual_seed(51)
    rnd = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)   # noqa: E731
    # convolution, packed: one long sequence and a last one of 70 tokens
    T, c, t = 270000, 8192, 70
    x, gy, w = rnd(T, c), rnd(T, c), torch.randn(c, 4, device="cuda", generator=gen)
    cu = torch.tensor([0, T - t, T], dtype=torch.int32, device="cuda")
    one = torch.tensor([0, t], dtype=torch.int32, device="cuda")
    tail = lambda v: v[T - t:].clone()   # noqa: E731
    assert torch.equal(kda.ssm_conv_fwd(x, w, cu_seqlens=cu)[T - t:], kda.ssm_conv_fwd(tail(x), w, cu_seqlens=one))
    gx = kda.ssm_conv_bwd(x, w, None, gy, cu_seqlens=cu)[0]
    assert torch.equal(gx[T - t:], kda.ssm_conv_bwd(tail(x), w, None, tail(gy), cu_seqlens=one)[0])
    del gx, gy
    # scan, the same rows as 128 heads of 64: chunks of one sequence are the
    # same products whatever stands before it
    H = 128
    x = x.view(T, H, 64)
    B, C = rnd(T, 1, 64), rnd(T, 1, 64)
    dt, A = torch.rand(T, H, device="cuda", generator=gen), -torch.rand(H, device="cuda", generator=gen) - 0.05
    y, S = kda.ssm_chunk_fwd(x, dt, A, B, C, cu_seqlens=cu, sequence_parallel=False)
    y1, S1 = kda.ssm_chunk_fwd(tail(x), tail(dt), A, tail(B), tail(C), cu_seqlens=one, sequence_parallel=False)
    assert torch.equal(y[T - t:], y1) and torch.equal(S[1], S1[0])
    r = kda.ssm_chunk_bwd(x, dt, A, B, C, None, None, y, cu_seqlens=cu)
    r1 = kda.ssm_chunk_bwd(tail(x), tail(dt), A, tail(B), tail(C), None, None, y1, cu_seqlens=one)
    assert torch.equal(r[0][T - t:], r1[0])
    torch.testing.assert_close(r[1][T - t:], r1[1], rtol=1e-5, atol=1e-5 * float(r1[1].abs().max()))
    for k in (3, 4):   # (the heads' partial sums meet in another order: two roundings to bf16)
        torch.testing.assert_close(r[k][T - t:].float(), r1[k].float(), rtol=2 ** -7, atol=1e-5 * float(r1[k].abs().max()))
    del x, y, r
    # states of 4.6 GB
    n, H = 1100, 128
    S = torch.empty(n, H, 128, 64, device="cuda").normal_(generator=gen)
    x, dt = rnd(n, 2, H, 64), torch.rand(n, 2, H, device="cuda", generator=gen)
    B, C = rnd(n, 2, 1, 128), rnd(n, 2, 1, 128)
    last = S[n - 1:].clone()
    y = kda.ssm_recurrent_fwd(x, dt, A, B, C, S)
    y1 = kda.ssm_recurrent_fwd(x[n - 1:], dt[n - 1:], A, B[n - 1:], C[n - 1:], last)
    assert torch.equal(y[n - 1:], y1) and torch.equal(S[n - 1:], last)
    del S
    # 160 requests of 17 rows of 10^6 probabilities
    n, K, V = 160, 16, 10 ** 6
    p = torch.empty(n, K + 1, V, dtype=torch.bfloat16, device="cuda").uniform_(generator=gen)
    d = torch.randint(0, V, (n, K), dtype=torch.int32, device="cuda", generator=gen)
    u, un = torch.rand(n, K, device="cuda", generator=gen) * 0.02, torch.rand(n, device="cuda", generator=gen)
    u[n - 1] = 0
    na, tok = kda.verify_drafts(p, d, u, un)
    na1, tok1 = kda.verify_drafts(p[n - 1:].clone(), d[n - 1:].clone(), u[n - 1:].clone(), un[n - 1:].clone())
    torch.cuda.synchronize()
    assert torch.equal(na[n - 1:], na1) and torch.equal(tok[n - 1:], tok1) and int(na1) == K


def test_python_refusals():
    x = torch.zeros(2, 8, 4, 64, device="cuda")
    dt, A, B = torch.zeros(2, 8, 4, device="cuda"), torch.zeros(4, device="cuda"), torch.zeros(2, 8, 1, 64, device="cuda")
    ok = dict(x=x, dt=dt, A=A, B=B, C=B)
    bad = [dict(x=x.transpose(1, 2)), dict(x=x[:, ::2]), dict(dt=dt.half()), dict(B=B[:, :7]), dict(C=B.bfloat16()),
           dict(A=A[:3]), dict(x=x.half()), dict(B=B[..., ::2], C=B[..., ::2]), dict(dt=dt.transpose(1, 2))]
    for b in bad:
        with pytest.raises(kda.KDAError):
            kda.ssm_chunk_fwd(**{**ok, **b})
    with pytest.raises(kda.KDAError):
        kda.ssm_chunk_fwd(**ok, cu_seqlens=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(kda.KDAError):
        kda.ssm_recurrent_fwd(x, dt, A, B, B, torch.zeros(2, 4, 64, 128, device="cuda"))
    with pytest.raises(kda.KDAError):
        kda.ssm_conv_fwd(torch.zeros(1, 4, 64, device="cuda"), torch.zeros(64, 5, device="cuda"))
    with pytest.raises(kda.KDAError):
        kda.ssm_conv_step(torch.zeros(1, 4, 64, device="cuda"), torch.zeros(64, 4, device="cuda"), None,
                          torch.zeros(2, 3, 64, device="cuda"))
