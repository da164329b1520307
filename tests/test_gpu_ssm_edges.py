"""GPU tests of the state space calls at the edges of what their headers allow.
Tolerances as in test_gpu_ssm.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU-only container
    pytest.skip("no GPU", allow_module_level=True)

import gated_delta_rule_amd as kda  # noqa: E402
from test_gpu_ssm import F32, HALF, check_bwd, dev, host, oracle_scan, run_bwd, scan_case  # noqa: E402

USE = ("D", "S0", "gS", "dt_bias")


def by_groups(a, dtype, n, H, G, N, P, groups):
    """The backward pass with a workspace for `groups` groups of heads, and behind it bytes that have to stay."""
    T = a["x"].shape[0]
    need = kda.ssm_chunk_bwd_workspace_bytes(dtype, n, T, H, G, N, P, True, groups=groups)
    buf = torch.full((need + (1 << 16),), 77, dtype=torch.uint8, device="cuda")
    r = run_bwd(a, dtype, USE, workspace=buf[:need])
    torch.cuda.synchronize()
    assert (buf[need:] == 77).all()
    return r


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,G,hpg,N,P,groups", [([70, 0, 130, 1], 3, 3, 64, 64, 2), ([150], 5, 2, 128, 64, 3),
                                                   ([65, 64], 4, 1, 64, 128, 3)])
def test_backward_by_groups_with_a_smaller_last_pass(lens, G, hpg, N, P, groups, dtype):
    H = G * hpg
    a = scan_case(lens, H, G, N, P, dtype, seed=60, amin=0.1, amax=2.0)
    check_bwd(by_groups(a, dtype, len(lens), H, G, N, P, groups), a, USE, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_backward_by_groups_where_fewer_heads_would_be_cut(dtype):
    """Seven groups, four at a time: a plan for the last three alone would cut
    the sequences into segments and need more than the four do."""
    lens, G, hpg, N, P = [17] * 8 + [3, 60, 0, 20, 11, 9, 20, 1], 7, 4, 64, 128
    if dtype == torch.bfloat16:
        lens = [2 * n for n in lens]
    H, T = G * hpg, sum(lens)
    need = [kda.ssm_chunk_bwd_workspace_bytes(dtype, len(lens), T, H, G, N, P, True, groups=g) for g in range(1, 8)]
    assert need[2] > need[3]
    a = scan_case(lens, H, G, N, P, dtype, seed=61, amin=0.1, amax=2.0)
    check_bwd(by_groups(a, dtype, len(lens), H, G, N, P, 4), a, USE, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_backward_by_groups_bitwise(dtype):
    """Chains without segments and one head per workgroup whatever the number
    of groups: all gradients have the same bits."""
    lens, H, G, N, P = [63, 5, 0, 64], 6, 3, 64, 64
    a = scan_case(lens, H, G, N, P, dtype, seed=62, amin=0.1, amax=2.0)
    want = run_bwd(a, dtype, USE)
    for groups in (1, 2):
        got = by_groups(a, dtype, len(lens), H, G, N, P, groups)
        for i, (g, w) in enumerate(zip(got, want)):
            assert torch.equal(g, w), i


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("P", [64, 128])
def test_skip_term_is_float32(P, dtype):
    """Where dt is zero and so is the state, y is D x, rounded once to its
    type, also where D itself is not of that type; a prompt and single tokens
    agree.  And beside other terms D's share of y keeps that accuracy."""
    H, N, T = 3, 64, 70
    gen = torch.Generator(device="cuda").manual_seed(63)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)   # noqa: E731
    x, B, C = rnd(1, T, H, P).to(dtype), rnd(1, T, 1, N).to(dtype), rnd(1, T, 1, N).to(dtype)
    D = torch.tensor([1 + 2 ** -8 + 2 ** -12, -0.37, 1e-3], device="cuda")
    A, dt = -torch.ones(H, device="cuda"), torch.full((1, T, H), -1e4, device="cuda")
    y, _ = kda.ssm_chunk_fwd(x, dt, A, B, C, D)
    S = torch.zeros(1, H, N, P, device="cuda")
    step = torch.cat([kda.ssm_recurrent_fwd(x[:, i:i + 64], dt[:, i:i + 64], A, B[:, i:i + 64], C[:, i:i + 64], S, D)
                      for i in (0, 64)], 1)
    torch.cuda.synchronize()
    want = (D[:, None] * x.float()).to(dtype)
    assert torch.equal(y, want) and torch.equal(step, want)
    a = scan_case([T], H, 1, N, P, dtype, seed=64)
    a["D"] = host(D)
    y, _ = kda.ssm_chunk_fwd(dev(a["x"], dtype), dev(a["dt"]), dev(a["A"]), dev(a["B"], dtype), dev(a["C"], dtype), D,
                             None, dev(a["cu"], torch.int32))
    torch.cuda.synchronize()
    ry, my, _, _, _, _ = oracle_scan(a, ("D",))
    _, rest, _, _, _, _ = oracle_scan(a, ())
    tol = F32 * my[0]
    if dtype == torch.bfloat16:
        tol = tol + 1.01 * HALF * (np.abs(ry[0]) + rest[0])
    assert (np.abs(host(y) - ry[0]) <= tol).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("P", [64, 128])
def test_skip_gradient_is_float32(P, dtype):
    """Where dt is zero and the state has no gradient, dx is D dy, rounded
    once; beside other terms D's share of dx keeps that accuracy."""
    H, N, T = 3, 64, 70
    gen = torch.Generator(device="cuda").manual_seed(65)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)   # noqa: E731
    x, B, C, gy = (rnd(1, T, *s).to(dtype) for s in ((H, P), (1, N), (1, N), (H, P)))
    D = torch.tensor([1 + 2 ** -8 + 2 ** -12, -0.37, 1e-3], device="cuda")
    A, dt = -torch.ones(H, device="cuda"), torch.full((1, T, H), -1e4, device="cuda")
    gx = kda.ssm_chunk_bwd(x, dt, A, B, C, D, None, gy)[0]
    torch.cuda.synchronize()
    assert torch.equal(gx, (D[:, None] * gy.float()).to(dtype))
    a = scan_case([T], H, 1, N, P, dtype, seed=66)
    a["D"] = host(D)
    gx = run_bwd(a, dtype, ("D",))[0]
    torch.cuda.synchronize()
    _, _, _, _, g, m = oracle_scan(a, ("D",), back=True)
    _, _, _, _, _, rest = oracle_scan(a, (), back=True)
    tol = F32 * m[0]["x"]
    if dtype == torch.bfloat16:
        tol = tol + 1.01 * HALF * (np.abs(g[0]["x"]) + rest[0]["x"])
    assert (np.abs(host(gx) - g[0]["x"]) <= tol).all()


@pytest.mark.parametrize("N,P", [(64, 64), (128, 64), (128, 128)])
def test_state_enters_outputs_beyond_bf16(N, P):
    """Tokens of dt = 0 read the initial state: y = S0^T C, rounded once.  The
    state's two bf16 parts leave 2^-16 of it, so a sum whose terms cancel keeps
    that accuracy (float32 sums as elsewhere)."""
    H, T = 3, 70
    a = scan_case([T], H, 1, N, P, torch.bfloat16, seed=67)
    a["dt"][:] = -1e4
    y, S = kda.ssm_chunk_fwd(dev(a["x"], torch.bfloat16), dev(a["dt"]), dev(a["A"]), dev(a["B"], torch.bfloat16),
                             dev(a["C"], torch.bfloat16), None, dev(a["S0"]), dev(a["cu"], torch.int32))
    torch.cuda.synchronize()
    ry, my, _, _, _, _ = oracle_scan(a, ("S0",))
    assert (np.abs(host(y) - ry[0]) <= 1.01 * HALF * np.abs(ry[0]) + (2.0 ** -16 + F32) * my[0]).all()
    assert torch.equal(S, dev(a["S0"]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_steps_continue_the_prompt_bitwise(W, dtype):
    """The convolution of 300 tokens at once, in steps of 64 and one by one:
    the same bits in outputs and cache."""
    n, T, c = 2, 300, 520
    gen = torch.Generator(device="cuda").manual_seed(68)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)   # noqa: E731
    x, w, bias, cache = (4 * rnd(n, T, c)).to(dtype), rnd(c, W), rnd(c), rnd(n, W - 1, c)
    whole = cache.clone()
    y = kda.ssm_conv_fwd(x, w, bias, whole)
    for step in (64, 1):
        c1 = cache.clone()
        parts = [kda.ssm_conv_step(x[:, i:i + step].contiguous(), w, bias, c1) for i in range(0, T, step)]
        torch.cuda.synchronize()
        assert torch.equal(torch.cat(parts, 1), y) and torch.equal(c1, whole)


@pytest.mark.parametrize("replay", [3, torch.zeros(1), (None, None, None), (None, None)])
def test_replay_is_no_triple_of_tensors(replay):
    x, dt, A, B = (torch.zeros(s, device="cuda") for s in ((1, 2, 2, 64), (1, 2, 2), (2,), (1, 2, 1, 64)))
    with pytest.raises(kda.KDAError):
        kda.ssm_recurrent_fwd(x, dt, A, B, B, torch.zeros(1, 2, 64, 64, device="cuda"), replay=replay)


def dirty(*likes):
    """Leaves NaN in the memory that the next tensors of these sizes get."""
    old = [torch.full_like(t, float("nan")) for t in likes for _ in range(3)]
    torch.cuda.synchronize()
    del old


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("before,lens,behind", [(5, [70, 9], 16), (0, [33, 0, 1], 300), (64, [40], 0), (3, [0], 4), (2, [], 30)])
def test_gradients_of_rows_of_no_sequence_are_zero(before, lens, behind, dtype):
    """What the call allocates is zero there, what is given stays, and the
    gradients of the sequences' rows are those of a batch without such rows."""
    H, G, N, P, c = 4, 2, 64, 64, 72
    n, real, T = len(lens), sum(lens), before + sum(lens) + behind
    gen = torch.Generator(device="cuda").manual_seed(69)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)   # noqa: E731
    at = slice(before, before + real)
    cu = torch.tensor([before + sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32, device="cuda")
    x, B, C, gy = (rnd(T, *s).to(dtype) for s in ((H, P), (G, N), (G, N), (H, P)))
    dt, A, D, S0 = rnd(T, H), -torch.rand(H, device="cuda", generator=gen), rnd(H), rnd(n, H, N, P)
    cx, cg, w, bias, cache = rnd(T, c).to(dtype), rnd(T, c).to(dtype), rnd(c, 4), rnd(c), rnd(n, 3, c)
    rest = [i for i in range(T) if not before <= i < before + real]
    for t in (x, B, C, gy, dt, cx, cg):
        t[rest] = float("nan")
    own = cu - before
    args = (x, dt, A, B, C, D, S0)
    part = tuple(t[at].contiguous() for t in (x, dt)) + (A,) + tuple(t[at].contiguous() for t in (B, C)) + (D, S0)
    dirty(x, B, C, dt, cx)
    for activation in (True, False):
        g = kda.ssm_conv_bwd(cx, w, bias, cg, cache, cu, activation=activation)
        ref = kda.ssm_conv_bwd(cx[at].contiguous(), w, bias, cg[at].contiguous(), cache, own, activation=activation)
        torch.cuda.synchronize()
        assert not g[0][rest].any() and torch.equal(g[0][at], ref[0]) and torch.equal(g[3], ref[3])
        assert torch.isfinite(g[1]).all() and torch.isfinite(g[2]).all()
    dirty(x, B, C, dt)
    r = kda.ssm_chunk_bwd(*args, gy, None, cu, dt_bias=D)
    given = [torch.full_like(t, 3.0) for t in (x, B, C)]
    r2 = kda.ssm_chunk_bwd(*args, gy, None, cu, dt_bias=D, grad_x=given[0], grad_B=given[1], grad_C=given[2])
    ref = kda.ssm_chunk_bwd(*part, gy[at].contiguous(), None, own, dt_bias=D)
    torch.cuda.synchronize()
    for i in (0, 1, 3, 4):
        assert not r[i][rest].any()
        if i != 1:
            assert (r2[i][rest] == 3).all()
        else:
            assert not r2[i][rest].any()
        assert torch.equal(r2[i][at], r[i][at])
        got, want = r[i][at].float(), ref[i].float()   # (segments may start elsewhere: rounding)
        torch.testing.assert_close(got, want, rtol=2 ** -7 if dtype == torch.bfloat16 and i != 1 else 1e-5,
                                   atol=1e-5 * float(want.abs().max()) if want.numel() else 0)
    assert all(torch.isfinite(t).all() for t in r)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_padded_batch_gradients(dtype):
    """Sequences padded with tokens of dt = 0, too short to be cut: the packed
    batch's gradients, bitwise where the padding only adds zeros to the same
    sums, and each sum over all tokens within its own tolerance."""
    lens, T, H, G, N, P = [150, 64, 3], 160, 4, 2, 64, 64
    a = scan_case(lens, H, G, N, P, dtype, seed=70)
    t = {k: dev(a[k], torch.float32 if k == "dt" else dtype) for k in ("x", "dt", "B", "C", "gy")}
    pad = {}
    for k, v in t.items():
        pad[k] = torch.full((len(lens), T) + v.shape[1:], {"dt": -1e4, "gy": 0.0}.get(k, 3.0), dtype=v.dtype, device="cuda")
        for i, (s, e) in enumerate(zip(a["cu"], a["cu"][1:])):
            pad[k][i, :e - s] = v[s:e]
    rest = [dev(a[k]) for k in ("D", "S0")]
    call = lambda v, cu: kda.ssm_chunk_bwd(v["x"], v["dt"], dev(a["A"]), v["B"], v["C"], *rest, v["gy"], dev(a["gS"]), cu,   # noqa: E731
                                           dt_bias=dev(a["dt_bias"]))
    r, rp = call(t, dev(a["cu"], torch.int32)), list(call(pad, None))
    torch.cuda.synchronize()
    for i in (0, 1, 3, 4):
        rp[i] = torch.cat([rp[i][j, :n] for j, n in enumerate(lens)])
        assert torch.equal(rp[i], r[i]), i
    assert torch.equal(rp[7], r[7])
    check_bwd(r, a, USE, dtype)
    check_bwd(rp, a, USE, dtype)


def test_calls_without_rows_need_no_stride():
    """No token rows: no pointer or row stride of theirs is looked at, by any
    of the calls, and states and caches stay."""
    lib, s = kda.load_library(), torch.cuda.current_stream().cuda_stream
    H, N, P, c, n = 2, 64, 64, 16, 3
    f = lambda *sh: torch.randn(*sh, device="cuda")   # noqa: E731
    cache, S, A, w, gA, gw = f(n, 3, c), f(n, H, N, P), -torch.rand(H, device="cuda"), f(c, 4), f(H), f(c, 4)
    old, S_old = cache.clone(), S.clone()
    p = lambda t: t.data_ptr()   # noqa: E731
    assert lib.kda_ssm_conv_fwd(None, 0, 0, p(w), None, p(cache), None, n, 0, c, 4, 1, None, s) == 0
    assert lib.kda_ssm_conv_step(None, 0, 0, p(w), None, p(cache), None, 0, None, n, 0, 0, c, 4, 1, 1, None, s) == 0
    assert lib.kda_ssm_conv_bwd(None, 0, 0, p(w), None, None, None, n, 0, c, 4, 1, None, 0, None, p(gw), None, None, None,
                                0, s) == 0
    assert lib.kda_ssm_chunk_fwd(None, 0, None, 0, None, 0, 0, None, None, 1, p(A), None, p(S), None, n, 0, H, 1, N, P, None,
                                 p(S), None, 0, s) == 0
    ws = torch.empty(kda.ssm_chunk_bwd_workspace_bytes(torch.bfloat16, n, 0, H, 1, N, P, False), dtype=torch.uint8, device="cuda")
    assert lib.kda_ssm_chunk_bwd(None, 0, None, 0, None, 0, 0, None, None, 1, p(A), None, None, None, n, 0, H, 1, N, P, None,
                                 p(S), None, 0, None, 0, None, 0, None, p(gA), None, None, p(S), p(ws), ws.numel(), s) == 0
    assert lib.kda_ssm_recurrent_fwd(None, 0, None, 0, None, 0, 0, None, None, 1, p(A), None, None, 0, None, 0, None, None,
                                     p(S), n, 0, 0, H, 1, N, P, 1, None, s) == 0
    torch.cuda.synchronize()
    assert torch.equal(cache, old) and torch.equal(S, S_old) and not gA.any() and not gw.any()
