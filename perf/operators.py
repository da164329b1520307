"""What is measured of the state-space operators and of the draft verification.

Operators (see include/kda_ssm.h and include/kda_spec.h):

  conv      y_t = silu(b + sum_j w_j x_{t-W+1+j}) per channel, with a cache of the last W - 1 inputs
  conv_bwd  its gradients
  scan      S_t = e^{dt_t A} S_{t-1} + dt_t B_t x_t^T,  y_t = S_t^T C_t + D x_t, dt = softplus(dt_raw + bias)
  scan_bwd  its gradients
  step      a decode step of the layer: the convolution and the recurrence for a few new tokens per request, after
            replaying the drafts that were accepted, cache and state in place
  verify    which of the drafted tokens stand, and the token that follows them

`own` picks the framework's kernels; otherwise the operators run in their plain form (32 bits, 64 for decay sums).
"""
import math
import random

import numpy as np
import torch

own = False

CHUNK = 64   # tokens per chunk of the plain scan


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the short convolution over one long prompt, all channels of a layer (64 heads of 64, one B / C group of 128)
        {"name": "conv prompt", "op": "conv", "dtype": "bf16", "n": 1, "T": 8192, "H": 64, "P": 64, "N": 128, "G": 1, "W": 4, "packed": False},
        # a few short ragged prompts of a small layer in 32 bits, where latency counts
        {"name": "conv ragged f32", "op": "conv", "dtype": "f32", "n": 5, "T": 333, "H": 6, "P": 64, "N": 64, "G": 2, "W": 4, "packed": True},
        # training of the same layer: two sequences of 4096
        {"name": "conv_bwd train", "op": "conv_bwd", "dtype": "bf16", "n": 2, "T": 4096, "H": 64, "P": 64, "N": 128, "G": 1, "W": 4, "packed": False},
        # a small ragged training batch with a three-tap filter
        {"name": "conv_bwd ragged f32", "op": "conv_bwd", "dtype": "f32", "n": 7, "T": 1001, "H": 6, "P": 64, "N": 64, "G": 2, "W": 3, "packed": True},
        # one long prompt
        {"name": "scan prompt", "op": "scan", "dtype": "bf16", "n": 1, "T": 8192, "H": 64, "P": 64, "N": 128, "G": 1, "packed": False},
        # prompts of many lengths packed on one axis, continued from their states: 96 heads of 128, eight groups
        {"name": "scan packed", "op": "scan", "dtype": "bf16", "n": 16, "T": 8192, "H": 96, "P": 128, "N": 128, "G": 8, "packed": True},
        # a training step's backward pass
        {"name": "scan_bwd train", "op": "scan_bwd", "dtype": "bf16", "n": 2, "T": 4096, "H": 64, "P": 64, "N": 128, "G": 1, "packed": False},
        # a small ragged one in 32 bits
        {"name": "scan_bwd ragged f32", "op": "scan_bwd", "dtype": "f32", "n": 3, "T": 517, "H": 6, "P": 64, "N": 64, "G": 2, "packed": True},
        # one request, one token: pure latency
        {"name": "step one", "op": "step", "dtype": "bf16", "n": 1, "T": 1, "Tr": 0, "H": 24, "P": 64, "N": 128, "G": 1, "W": 4},
        # a full serving batch with four drafts per request after a replay
        {"name": "step drafts", "op": "step", "dtype": "bf16", "n": 256, "T": 5, "Tr": 5, "H": 64, "P": 64, "N": 128, "G": 1, "W": 4},
        # one request with four drafts over a small vocabulary
        {"name": "verify one", "op": "verify", "dtype": "f32", "n": 1, "K": 4, "V": 32000, "drafts": "sampled"},
        # a full serving batch over a large vocabulary of odd size
        {"name": "verify batch", "op": "verify", "dtype": "f32", "n": 128, "K": 5, "V": 151001, "drafts": "sampled"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv_bwd", "scan", "scan_bwd", "step", "verify"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "verify":
        n = _log(rng, 1, 128)
        return {"op": op, "dtype": dtype, "n": n, "K": rng.randint(1, 8), "V": _log(rng, 1000, 160000 if n * 9 < 640 else 80000),
                "drafts": rng.choice(["sampled", "sampled", "fixed"])}
    P, N, W = rng.choice([64, 64, 128]), rng.choice([64, 128, 128]), rng.choice([2, 3, 4, 4])
    G = rng.choice([1, 1, 2, 4])
    if op == "step":
        T, Tr = rng.choice([1, 1, 2, 5, 8]), rng.choice([0, 0, 3, 5])
        return {"op": op, "dtype": dtype, "n": _log(rng, 1, 128), "T": T, "Tr": Tr, "H": G * rng.randint(3, 48 // G),
                "P": P, "N": N, "G": G, "W": W}
    packed = rng.random() < 0.5
    n = _log(rng, 1, 12)
    most = 3000 if op == "scan_bwd" else 7000      # tokens in all
    T = _log(rng, 64, most) if packed else max(1, _log(rng, 64, most) // n)
    case = {"op": op, "dtype": dtype, "n": n, "T": T, "H": G * rng.randint(2, 48 // G), "P": P, "N": N, "G": G, "packed": packed}
    return {**case, "W": W} if op.startswith("conv") else case


def _es(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    op, es = case["op"], _es(case)
    if op == "verify":   # the drafts' entries and one row of each distribution
        rows = 2 if case["drafts"] == "sampled" else 1
        return {"bytes": case["n"] * (case["V"] * es * rows + case["K"] * (2 * es + 12) + 16), "flops": case["n"] * case["V"] * 3}
    H, P, N, G = case["H"], case["P"], case["N"], case["G"]
    C = H * P + 2 * G * N
    if op == "step":
        rows = case["n"] * case["T"]
        rep = case["n"] * case["Tr"]
        return {"bytes": 8 * case["n"] * H * N * P + rows * (C + H * P) * es + rep * C * es + 8 * case["n"] * (case["W"] - 1) * C,
                "flops": 4 * (rows + rep / 2) * H * N * P}
    rows = case["T"] if case["packed"] else case["n"] * case["T"]
    state = 4 * case["n"] * H * N * P
    if op == "conv":
        return {"bytes": 2 * rows * C * es + 8 * case["n"] * (case["W"] - 1) * C + 4 * C * (case["W"] + 1), "flops": 2 * rows * C * case["W"]}
    if op == "conv_bwd":
        return {"bytes": 3 * rows * C * es + 8 * C * (case["W"] + 1), "flops": 6 * rows * C * case["W"]}
    if op == "scan":
        return {"bytes": rows * ((2 * H * P + 2 * G * N) * es + 4 * H) + 2 * state, "flops": 4 * rows * H * N * P}
    return {"bytes": rows * ((3 * H * P + 4 * G * N) * es + 8 * H) + 3 * state, "flops": 10 * rows * H * N * P}


# ----------------------------------------------------------------- inputs

def _lens(case, seed):
    """Sequence lengths of a packed batch: they add up to T, some far shorter than others."""
    r, n, T = random.Random(seed * 7919 + case["T"]), case["n"], case["T"]
    w = [r.uniform(0.1, 1.0) for _ in range(n)]
    lens = [int(T * x / sum(w)) for x in w]
    lens[-1] += T - sum(lens)
    return lens


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = {"op": case["op"]}
    n = case["n"]
    if case["op"] == "verify":
        K, V = case["K"], case["V"]
        base = 2.5 * normal(n, K + 1, V)
        s["p"] = torch.softmax(base, -1).to(dt)
        q = torch.softmax(base[:, :K] + 0.7 * normal(n, K, V), -1)
        if case["drafts"] == "sampled":
            s["q"] = q.to(dt)
            at = (torch.cumsum(q.double(), -1) < uniform(n, K, 1).double()).sum(-1)
        else:
            s["q"] = None
            at = q.argmax(-1)
        s["drafts"] = at.clamp(max=V - 1).to(torch.int32)
        s["u"], s["u_next"] = uniform(n, K), uniform(n)
        return s
    H, P, N, G = case["H"], case["P"], case["N"], case["G"]
    C = H * P + 2 * G * N
    s.update(H=H, P=P, N=N, G=G)
    if case["op"] == "step":
        T, Tr, W = case["T"], case["Tr"], case["W"]
        s["raw"], s["raw_old"] = normal(n, T, C).to(dt), normal(n, Tr, C).to(dt)
        s["xbc_old"] = torch.nn.functional.silu(normal(n, Tr, C)).to(dt)
        s["n_replay"] = torch.randint(0, Tr + 1, (n,), generator=g, device="cuda", dtype=torch.int32) if Tr else None
        s["dt"], s["dt_old"] = normal(n, T, H), normal(n, Tr, H)
        s["S"], s["cache"] = normal(n, H, N, P), normal(n, W - 1, C)
        s["commit"] = Tr == 0
    else:
        if case["packed"]:
            lens = _lens(case, seed)
            rows = (case["T"],)
            s["cu"] = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
            s["longest"] = max(lens)
        else:
            rows = (n, case["T"])
            s["cu"], s["longest"] = None, case["T"]
        s["n"] = n
        if case["op"].startswith("conv"):
            s["x"] = normal(*rows, C).to(dt)
            s["cache"] = normal(n, case["W"] - 1, C)
            if case["op"] == "conv_bwd":
                s["gy"] = normal(*rows, C).to(dt)
        else:
            s["xbc"] = torch.nn.functional.silu(normal(*rows, C)).to(dt)   # what the convolution puts out
            s["dt"] = normal(*rows, H)
            s["S0"] = normal(n, H, N, P)
            if case["op"] == "scan_bwd":
                s["gy"] = normal(*rows, H, P).to(dt)
                s["gS"] = 0.1 * normal(n, H, N, P)
    if "W" in case:
        s["w"], s["bias"] = normal(C, case["W"]) / case["W"], 0.1 * normal(C)
    if case["op"] in ("scan", "scan_bwd", "step"):
        s["A"] = -(1.0 + 15.0 * uniform(H))
        step = torch.exp(math.log(1e-3) + uniform(H) * math.log(100.0))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["D"] = 1.0 + 0.1 * normal(H)
    return s


def _split(s, xbc):
    """x, B and C as the parts of the convolution's channels."""
    HP, GN = s["H"] * s["P"], s["G"] * s["N"]
    x, B, C = xbc[..., :HP], xbc[..., HP:HP + GN], xbc[..., HP + GN:]
    return x.unflatten(-1, (s["H"], s["P"])), B.unflatten(-1, (s["G"], s["N"])), C.unflatten(-1, (s["G"], s["N"]))


# -------------------------------------------------------------------- run

def run(s):
    return (_run_own if own else _run_plain)[s["op"]](s)


# --- the framework's calls

def _own_conv(s):
    import gated_delta_rule_amd as kda
    y = kda.ssm_conv_fwd(s["x"], s["w"], s["bias"], s["cache"], s["cu"])
    return y, s["cache"]


def _own_conv_bwd(s):
    import gated_delta_rule_amd as kda
    return kda.ssm_conv_bwd(s["x"], s["w"], s["bias"], s["gy"], s["cache"], s["cu"])


def _own_scan(s):
    import gated_delta_rule_amd as kda
    x, B, C = _split(s, s["xbc"])
    return kda.ssm_chunk_fwd(x, s["dt"], s["A"], B, C, s["D"], s["S0"], s["cu"], dt_bias=s["dt_bias"])


def _own_scan_bwd(s):
    import gated_delta_rule_amd as kda
    x, B, C = _split(s, s["xbc"])
    g = torch.empty_like(s["xbc"])
    gx, gB, gC = _split(s, g)
    r = kda.ssm_chunk_bwd(x, s["dt"], s["A"], B, C, s["D"], s["S0"], s["gy"], s["gS"], s["cu"], dt_bias=s["dt_bias"],
                          grad_x=gx, grad_B=gB, grad_C=gC)
    return (g, r[1], r[2]) + tuple(r[5:])


def _own_step(s):
    import gated_delta_rule_amd as kda
    replay = s["n_replay"] is not None
    xbc = kda.ssm_conv_step(s["raw"], s["w"], s["bias"], s["cache"], replay=s["raw_old"] if replay else None,
                            n_replay=s["n_replay"], commit=s["commit"])
    x, B, C = _split(s, xbc)
    old = None
    if replay:
        rx, rB, _ = _split(s, s["xbc_old"])
        old = (rx, s["dt_old"], rB)
    y = kda.ssm_recurrent_fwd(x, s["dt"], s["A"], B, C, s["S"], s["D"], dt_bias=s["dt_bias"], replay=old,
                              n_replay=s["n_replay"], commit=s["commit"])
    return xbc, y, s["cache"], s["S"]


def _own_verify(s):
    import gated_delta_rule_amd as kda
    return kda.verify_drafts(s["p"], s["drafts"], s["u"], s["u_next"], s["q"])


_run_own = {"conv": _own_conv, "conv_bwd": _own_conv_bwd, "scan": _own_scan, "scan_bwd": _own_scan_bwd, "step": _own_step,
            "verify": _own_verify}


# --- the plain forms

def _rows(s, x):
    """Sequence, position and first row of every token row."""
    if s["cu"] is None:
        n, T = x.shape[:2]
        r = torch.arange(n * T, device=x.device)
        return r // T, r % T
    r = torch.arange(x.shape[0], device=x.device)
    n = torch.searchsorted(s["cu"].long(), r, right=True) - 1
    return n, r - s["cu"].long()[n]


def _input_at(x, cache, seq, row, pos):
    """x_pos of a sequence: a row of x, or before its start an entry of the cache.  `row`: the row of x_pos."""
    W1 = cache.shape[1]
    old = cache[seq, (W1 + pos).clamp(0, W1 - 1)]
    return torch.where((pos >= 0)[:, None], x[row.clamp(min=0)], old)


def _conv_plain(s, x, w, bias, cache):
    """Packed or not: silu of the convolution, rows [R, C], in 32 bits."""
    seq, pos = _rows(s, x)
    x = x.reshape(-1, x.shape[-1])
    row = torch.arange(x.shape[0], device=x.device)
    W = w.shape[1]
    z = bias + sum(w[:, W - 1 - d] * _input_at(x, cache, seq, row - d, pos - d) for d in range(W))
    return z / (1 + torch.exp(-z))


def _cache_after(s, x, cache):
    x = x.reshape(-1, x.shape[-1])
    n, W1 = cache.shape[:2]
    if s["cu"] is None:
        end = (torch.arange(n, device=x.device) + 1) * (x.shape[0] // n)
        length = torch.full_like(end, x.shape[0] // n)
    else:
        end = s["cu"].long()[1:]
        length = end - s["cu"].long()[:-1]
    return torch.stack([_input_at(x, cache, torch.arange(n, device=x.device), end - W1 + m, length - W1 + m) for m in range(W1)], 1)


def _plain_conv(s):
    x = s["x"].float()
    y = _conv_plain(s, x, s["w"], s["bias"], s["cache"]).to(s["x"].dtype).view(s["x"].shape)
    s["cache"].copy_(_cache_after(s, x, s["cache"]))
    return y, s["cache"]


def _plain_conv_bwd(s):
    with torch.enable_grad():
        leaves = [t.float().detach().requires_grad_() for t in (s["x"], s["w"], s["bias"], s["cache"])]
        y = _conv_plain(s, *leaves)
        g = torch.autograd.grad(y, leaves, s["gy"].float().view(y.shape))
    return (g[0].to(s["x"].dtype),) + g[1:]


def _softplus(t):
    return torch.clamp(t, min=0) + torch.log1p(torch.exp(-torch.abs(t)))


def _padded(s, t):
    """A packed batch as equal lengths, rows past a sequence's end zero."""
    if s["cu"] is None:
        return t
    start, end = s["cu"].long()[:-1, None], s["cu"].long()[1:, None]
    at = start + torch.arange(s["longest"], device=t.device)
    kept = (at < end).view(at.shape + (1,) * (t.dim() - 1))
    return t[at.clamp(max=t.shape[0] - 1)] * kept


def _scan_plain(x, dt, A, B, C, D, S0, L):
    """Equal lengths, in chunks of L tokens; dt is zero in rows that are to have no effect."""
    n, T, H, P = x.shape
    c = -(-T // L)

    def chunks(t):   # [n, c, heads, L, d]
        t = torch.nn.functional.pad(t, (0, 0, 0, 0, 0, c * L - T))
        return t.view(n, c, L, t.shape[2], t.shape[3]).transpose(2, 3)

    per = H // B.shape[2]
    xs, Bs, Cs = chunks(x), chunks(B), chunks(C)
    dts = chunks(dt[..., None])[..., 0]                            # [n, c, H, L]
    g = torch.cumsum((dts * A[:, None]).double(), -1)
    low = torch.tril(torch.ones(L, L, dtype=torch.bool, device=x.device))
    decay = torch.exp(torch.where(low, g[..., :, None] - g[..., None, :], -math.inf).float())
    M = (Cs @ Bs.transpose(-1, -2).contiguous()).repeat_interleave(per, 2) * decay * dts[..., None, :]
    Bh, Ch = Bs.repeat_interleave(per, 2), Cs.repeat_interleave(per, 2)
    put = Bh * (torch.exp((g[..., -1:] - g).float()) * dts)[..., None]
    E = put.transpose(-1, -2).contiguous() @ xs                    # what each chunk adds to the state
    total = torch.cumsum(g[..., -1], 1).transpose(1, 2)            # [n, H, c]
    upto = torch.cat([torch.zeros_like(total[..., :1]), total], -1)
    before = torch.tril(torch.ones(c + 1, c, dtype=torch.bool, device=x.device), -1)
    F = torch.exp(torch.where(before, upto[..., :, None] - total[..., None, :], -math.inf).float())
    S = F @ E.transpose(1, 2).reshape(n, H, c, -1) + torch.exp(upto.float())[..., None] * S0.reshape(n, H, 1, -1)
    S = S.view(n, H, c + 1, *S0.shape[2:])
    y = M @ xs + torch.exp(g.float())[..., None] * (Ch @ S[:, :, :-1].transpose(1, 2))
    y = y.transpose(2, 3).reshape(n, c * L, H, P)[:, :T] + D[:, None] * x
    return y, S[:, :, -1]


def _scan_of(s, xbc, dt, A, dt_bias, D, S0):
    x, B, C = _split(s, _padded(s, xbc))
    dt = _padded(s, _softplus(dt + dt_bias))
    y, S_T = _scan_plain(x, dt, A, B, C, D, S0, CHUNK)
    if s["cu"] is not None:
        seq, pos = _rows(s, xbc)
        y = y[seq, pos]
    return y, S_T


def _plain_scan(s):
    y, S_T = _scan_of(s, s["xbc"].float(), s["dt"], s["A"], s["dt_bias"], s["D"], s["S0"])
    return y.to(s["xbc"].dtype), S_T


def _plain_scan_bwd(s):
    with torch.enable_grad():
        leaves = [s[k].float().detach().requires_grad_() for k in ("xbc", "dt", "A", "dt_bias", "D", "S0")]
        y, S_T = _scan_of(s, *leaves)
        g = torch.autograd.grad([y, S_T], leaves, [s["gy"].float(), s["gS"]])
    gxbc, gdt, gA, gbias, gD, gS0 = g
    return gxbc.to(s["xbc"].dtype), gdt, gA, gD, gbias, gS0


def _plain_step(s):
    n, T, C = s["raw"].shape
    Tr = s["raw_old"].shape[1]
    raw = torch.cat([s["raw_old"], s["raw"]], 1).float()
    kept = s["n_replay"].long() if Tr else torch.zeros(n, dtype=torch.long, device=raw.device)
    W1 = s["cache"].shape[1]
    # the inputs in order: the cache, the replayed tokens that were accepted, the new tokens
    j = torch.arange(W1 + T, device=raw.device)
    at = kept[:, None] + j
    at = torch.where(at < W1 + kept[:, None], at, at - kept[:, None] + Tr)
    every = torch.cat([s["cache"], raw], 1)
    seen = torch.gather(every, 1, at[..., None].expand(-1, -1, C))
    z = s["bias"] + sum(s["w"][:, W1 - d] * seen[:, W1 - d:W1 - d + T] for d in range(W1 + 1))
    xbc = (z / (1 + torch.exp(-z))).to(s["raw"].dtype)
    s["cache"].copy_(seen[:, T:] if s["commit"] else seen[:, :W1])
    both = torch.cat([s["xbc_old"], xbc], 1).float()
    dt = _softplus(torch.cat([s["dt_old"], s["dt"]], 1) + s["dt_bias"])
    t = torch.arange(Tr + T, device=raw.device)
    x, B, Cm = _split(s, both)
    dt = dt * ((t < kept[:, None]) | (t >= Tr))[..., None]
    y, S_T = _scan_plain(x, dt, s["A"], B, Cm, s["D"], s["S"], Tr + T)
    if not s["commit"]:
        S_T = _scan_plain(x[:, :Tr], dt[:, :Tr], s["A"], B[:, :Tr], Cm[:, :Tr], s["D"], s["S"], Tr)[1]
    s["S"].copy_(S_T)
    return xbc, y[:, Tr:].to(s["raw"].dtype), s["cache"], s["S"]


def _plain_verify(s):
    p, q, d = s["p"], s["q"], s["drafts"].long()
    n, K = d.shape
    V = p.shape[-1]
    pd = torch.gather(p[:, :K], 2, d[..., None])[..., 0].double()
    qd = torch.ones_like(pd) if q is None else torch.gather(q, 2, d[..., None])[..., 0].double()
    stands = s["u"].double() * qd < pd
    n_acc = torch.cumprod(stands.long(), 1).sum(1)
    b = torch.arange(n, device=p.device)
    row = p[b, n_acc].double()
    cut = n_acc < K
    first = n_acc.clamp(max=K - 1)
    if q is None:
        less = torch.nn.functional.one_hot(d[b, first], V).double() * row
    else:
        less = q[b, first].double()
    rest = (row - less * cut[:, None]).clamp(min=0)
    rest = torch.where((rest.sum(-1, keepdim=True) > 0), rest, row)
    run_sum = torch.cumsum(rest, -1)
    token = (run_sum <= s["u_next"].double()[:, None] * run_sum[:, -1:]).sum(-1).clamp(max=V - 1)
    i = torch.arange(K + 1, device=p.device)
    out = torch.where(i < n_acc[:, None], torch.nn.functional.pad(d, (0, 1)), -1)
    out = torch.where(i == n_acc[:, None], token[:, None], out)
    return n_acc.to(torch.int32), out.to(torch.int32)


_run_plain = {"conv": _plain_conv, "conv_bwd": _plain_conv_bwd, "scan": _plain_scan, "scan_bwd": _plain_scan_bwd,
              "step": _plain_step, "verify": _plain_verify}


# ------------------------------------------------------------------ exact

def exact(case, seed):
    """The definitions, token by token in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "verify":
        return None
    d = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    if op == "step":
        return _exact_step(case, d)
    cu = s["cu"].tolist() if s["cu"] is not None else [i * case["T"] for i in range(case["n"] + 1)]
    if op.startswith("conv"):
        x = d["x"].reshape(cu[-1], -1)
        gy = d["gy"].reshape(cu[-1], -1) if op == "conv_bwd" else None
        parts = [_exact_conv(x[a:b], d["w"], d["bias"], d["cache"][i], None if gy is None else gy[a:b])
                 for i, (a, b) in enumerate(zip(cu, cu[1:]))]
        if gy is None:
            return torch.cat([p[0] for p in parts]).view(s["x"].shape), torch.stack([p[1] for p in parts])
        return (torch.cat([p[0] for p in parts]).view(s["x"].shape), sum(p[1] for p in parts), sum(p[2] for p in parts),
                torch.stack([p[3] for p in parts]))
    lens = [b - a for a, b in zip(cu, cu[1:])]
    if op == "scan_bwd" and max(lens) * case["n"] * case["H"] * case["N"] * case["P"] * 8 > 80e9:
        return None
    return _exact_scan(case, d, cu, op == "scan_bwd")


def _exact_conv(x, w, bias, cache, gy):
    W = w.shape[1]
    line = torch.cat([cache, x])
    T = x.shape[0]
    z = bias.expand(T, -1).clone()
    for j in range(W):
        z += w[:, j] * line[j:j + T]
    sig = torch.sigmoid(z)
    if gy is None:
        return z * sig, line[T:]
    gz = gy * sig * (1 + z * (1 - sig))
    gline = torch.zeros_like(line)
    gw = torch.zeros_like(w)
    for j in range(W):
        gline[j:j + T] += w[:, j] * gz
        gw[:, j] = (gz * line[j:j + T]).sum(0)
    return gline[W - 1:], gw, gz.sum(0), gline[:W - 1]


def _exact_scan(case, d, cu, grads):
    """All sequences side by side: at step t the ones that are that long."""
    H, P, N, G, n = case["H"], case["P"], case["N"], case["G"], case["n"]
    rows = cu[-1]
    xbc = d["xbc"].reshape(rows, -1)
    x = xbc[:, :H * P].reshape(rows, H, P)
    B = xbc[:, H * P:H * P + G * N].reshape(rows, G, N).repeat_interleave(H // G, 1)
    C = xbc[:, H * P + G * N:].reshape(rows, G, N).repeat_interleave(H // G, 1)
    raw = d["dt"].reshape(rows, H) + d["dt_bias"]
    dt = torch.where(raw > 30, raw, torch.log1p(torch.exp(raw.clamp(max=30))))
    A, D = d["A"], d["D"]
    lens = [b - a for a, b in zip(cu, cu[1:])]
    order = sorted(range(n), key=lambda i: -lens[i])
    start = torch.tensor([cu[i] for i in order], device=x.device)
    alive = [sum(lens[i] > t for i in order) for t in range(max(lens))]
    S = d["S0"][order].clone()
    y = torch.empty(rows, H, P, dtype=torch.float64, device=x.device)
    kept = []
    for t, m in enumerate(alive):
        r = start[:m] + t
        if grads:
            kept.append(S[:m].clone())
        S[:m] = torch.exp(dt[r] * A)[..., None, None] * S[:m] + (dt[r][..., None] * B[r])[..., :, None] * x[r][..., None, :]
        y[r] = (S[:m] * C[r][..., :, None]).sum(-2) + D[:, None] * x[r]
    back = torch.empty(n, dtype=torch.long)
    back[torch.tensor(order)] = torch.arange(n)
    if not grads:
        return y.view(d["xbc"].shape[:-1] + (H, P)), S[back.to(S.device)]
    gy = d["gy"].reshape(rows, H, P)
    gS = d["gS"][order].clone()
    gx, gB, gC = torch.empty_like(x), torch.empty_like(B), torch.empty_like(C)
    gdt, ga = torch.empty_like(dt), torch.empty_like(dt)
    for t in range(len(alive) - 1, -1, -1):
        m = alive[t]
        r = start[:m] + t
        old, e = kept.pop(), torch.exp(dt[r] * A)
        u = (dt[r][..., None] * B[r])[..., :, None]
        new = e[..., None, None] * old + u * x[r][..., None, :]
        gC[r] = (new * gy[r][..., None, :]).sum(-1)
        gS[:m] += C[r][..., :, None] * gy[r][..., None, :]
        gx[r] = (gS[:m] * u).sum(-2) + D[:, None] * gy[r]
        into = (gS[:m] * x[r][..., None, :]).sum(-1)
        gB[r] = dt[r][..., None] * into
        ga[r] = e * (gS[:m] * old).sum((-1, -2))
        gdt[r] = (into * B[r]).sum(-1) + A * ga[r]
        gS[:m] *= e[..., None, None]
    graw = gdt * torch.sigmoid(raw)
    fold = lambda t: t.view(rows, G, H // G, N).sum(2).reshape(rows, -1)   # noqa: E731
    gxbc = torch.cat([gx.reshape(rows, -1), fold(gB), fold(gC)], -1).view(d["xbc"].shape)
    return (gxbc, graw.view(d["dt"].shape), (ga * dt).sum(0), (gy * x).sum((0, 2)), graw.sum(0), gS[back.to(S.device)])


def _exact_step(case, d):
    H, P, N, G, n, T, Tr = (case[k] for k in ("H", "P", "N", "G", "n", "T", "Tr"))
    bf = case["dtype"] == "bf16"
    kept = d["n_replay"].tolist() if Tr else [0] * n
    W1 = d["cache"].shape[1]
    # the window of every request after its accepted tokens
    win = torch.stack([torch.cat([d["cache"][i], d["raw_old"][i, :k]])[-W1:] for i, k in enumerate(kept)])
    line = torch.cat([win, d["raw"]], 1)
    z = d["bias"].expand(n, T, -1).clone()
    for j in range(W1 + 1):
        z += d["w"][:, j] * line[:, j:j + T]
    xbc = z * torch.sigmoid(z)
    # the recurrence takes what the convolution hands it, in its type
    z32 = xbc.float()
    handed = z32.to(torch.bfloat16).double() if bf else z32.double()
    S = d["S"].clone()

    def put(S, xbc_t, raw_t, on):
        x = xbc_t[:, :H * P].reshape(n, H, P)
        B = xbc_t[:, H * P:H * P + G * N].reshape(n, G, N).repeat_interleave(H // G, 1)
        C = xbc_t[:, H * P + G * N:].reshape(n, G, N).repeat_interleave(H // G, 1)
        raw = raw_t + d["dt_bias"]
        dt = torch.log1p(torch.exp(raw)) * on[:, None]
        S = torch.exp(dt * d["A"])[..., None, None] * S + (dt[..., None] * B)[..., :, None] * x[..., None, :]
        return S, (S * C[..., :, None]).sum(-2) + d["D"][:, None] * x

    counts = torch.tensor(kept, device=S.device)
    for t in range(Tr):
        S, _ = put(S, d["xbc_old"][:, t], d["dt_old"][:, t], (counts > t).double())
    end, ys = S, []
    for t in range(T):
        end, y = put(end, handed[:, t], d["dt"][:, t], torch.ones_like(counts).double())
        ys.append(y)
    if d["commit"]:
        return xbc, torch.stack(ys, 1), line[:, T:], end
    return xbc, torch.stack(ys, 1), win, S
