"""GPU parity of softmax attention, its gradients and its paged cache against
the fp64 oracle (oracle/attn.py).

Tolerances, elementwise: the bounds of oracle/attn.py for float32 arithmetic
with each weight (and score gradient) rounded to bf16 once where the inputs
are bf16, plus the result's own rounding: 2^-8 |ref| for bf16, 2^-24 |ref| for
float32.  The bounds are worst cases of every rounding, not fits.
"""
import numpy as np
import pytest

from kda_testlib import say
from oracle import attn as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU-only container
    pytest.skip("no GPU", allow_module_level=True)

import gated_delta_rule_amd as kda  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


def half(dtype):
    return 2.0 ** -8 if dtype == BF16 else 0.0


def dev(a, dtype=F32):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dtype)


def host(t):
    return t.detach().double().cpu().numpy()


def check(name, got, ref, err, dtype):
    """got against ref within err and the result's own rounding."""
    got = np.asarray(got, np.float64)
    same = np.isneginf(ref) & np.isneginf(got)
    ref, err = np.where(same, 0.0, ref), np.where(same, 0.0, err)
    got = np.where(same, 0.0, got)
    tol = err * 1.01 + (2.0 ** -8 if dtype == BF16 else 2.0 ** -24) * np.abs(ref) * 1.01 + 1e-30
    assert np.isfinite(got).all(), f"{name}: not finite"
    worst = float((np.abs(got - ref) / tol).max()) if got.size else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3g} of the tolerance"
    return worst


def values(shape, dtype, r, scale=1.0):
    """Values that the type holds exactly, as float64."""
    return (torch.from_numpy(r.standard_normal(shape).astype(np.float32)) * scale).to(dtype).double().numpy()


def wide(a, dtype, left=16, right=8):
    """a [rows, heads, D] as columns of wider rows that hold NaN elsewhere."""
    rows, n, D = a.shape
    w = torch.full((rows, left + n * D + right), NAN, dtype=dtype, device="cuda")
    v = w[:, left:left + n * D].unflatten(-1, (n, D))
    v.copy_(dev(a, dtype))
    return v


# lengths, heads, groups, D
CASES = [([1], 1, 1, 64), ([0, 1, 2, 0, 3, 5], 3, 1, 128), ([63, 64, 65, 0, 1], 4, 2, 64), ([130, 17], 6, 2, 128),
         ([257], 5, 5, 64), ([128, 127, 129], 8, 1, 128), ([33, 300], 7, 1, 64)]


def batch(case, dtype, seed=0):
    lens, H, G, D = case
    r = np.random.default_rng(seed)
    T = sum(lens)
    return dict(q=values((T, H, D), dtype, r, 1.5), k=values((T, G, D), dtype, r), v=values((T, G, D), dtype, r),
                gy=values((T, H, D), dtype, r), cu=np.concatenate([[0], np.cumsum(lens)]), scale=D ** -0.5)


def reference(a, causal, dtype):
    """o, lse, their bounds, gradients and theirs, of all sequences in order."""
    parts = [[] for _ in range(10)]
    for s, e in zip(a["cu"], a["cu"][1:]):
        q, k, v, gy = (a[n][s:e] for n in ("q", "k", "v", "gy"))
        o, lse = O.attention(q, k, v, a["scale"], 0, causal)
        eo, el = O.bounds(q, k, v, a["scale"], half(dtype), 0, causal)
        g = O.attention_backward(q, k, v, gy, a["scale"], causal)
        eg = O.backward_bounds(q, k, v, gy, a["scale"], half(dtype), causal)
        for p, x in zip(parts, (o, lse, eo, el) + g + eg):
            p.append(x)
    return [np.concatenate(p) for p in parts]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", CASES)
def test_packed(case, causal, dtype):
    a = batch(case, dtype)
    lens, H, G, D = case
    T, pad = sum(lens), 3
    o_ref, lse_ref, eo, el, gq_r, gk_r, gv_r, eq, ek, ev = reference(a, causal, dtype)

    def padded(x):   # rows of no sequence around the batch
        n = np.full((T + 2 * pad,) + x.shape[1:], np.nan)
        n[pad:pad + T] = x
        return n

    q, k, v = (wide(padded(a[n]), dtype) for n in "qkv")
    gy = dev(padded(a["gy"]), dtype)
    cu = dev(a["cu"] + pad, torch.int32)
    o = torch.full((T + 2 * pad, H, D), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((T + 2 * pad, H), 7.0, device="cuda")
    kda.attn_fwd(q, k, v, cu, causal=causal, o=o, lse=lse)
    inside = slice(pad, pad + T)
    w = [check("o", host(o)[inside], o_ref, eo, dtype), check("lse", host(lse)[inside], lse_ref, el, F32)]
    for t in (o, lse):
        assert (t[:pad] == 7.0).all() and (t[pad + T:] == 7.0).all()
    g = kda.attn_bwd(q, k, v, o, lse, gy, cu, causal=causal)
    given = [torch.full_like(t.contiguous(), 3.0) for t in (q, k, v)]
    again = kda.attn_bwd(q, k, v, o, lse, gy, cu, causal=causal, grad_q=given[0], grad_k=given[1], grad_v=given[2])
    for name, x, y, ref, e in zip(("gq", "gk", "gv"), g, again, (gq_r, gk_r, gv_r), (eq, ek, ev)):
        w.append(check(name, host(x)[inside], ref, e, dtype))
        assert torch.equal(x[inside], y[inside])
        assert (x[:pad] == 0).all() and (x[pad + T:] == 0).all()      # made by the call
        assert (y[:pad] == 3.0).all() and (y[pad + T:] == 3.0).all()  # given
    say(f"[attn] {case} causal={causal} {dtype}: of the tolerance " + " ".join(f"{x:.2g}" for x in w))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,T,H,G,D", [(3, 70, 6, 2, 64), (2, 129, 4, 4, 128), (1, 513, 8, 1, 128)])
def test_equal_lengths_match_packed_bitwise(n, T, H, G, D, dtype):
    a = batch(([T] * n, H, G, D), dtype, 1)
    q, k, v, gy = (dev(a[x], dtype) for x in ("q", "k", "v", "gy"))
    cu = dev(a["cu"], torch.int32)
    o, lse = kda.attn_fwd(q, k, v, cu)
    g = kda.attn_bwd(q, k, v, o, lse, gy, cu)
    qb, kb, vb, gyb = (t.view(n, T, *t.shape[1:]) for t in (q, k, v, gy))
    ob, lseb = kda.attn_fwd(qb, kb, vb)
    gb = kda.attn_bwd(qb, kb, vb, ob, lseb, gyb)
    for x, y in zip((o, lse) + g, (ob, lseb) + gb):
        assert torch.equal(x, y.view(x.shape))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_scores_and_other_scale(dtype):
    # one key far ahead of the others, and scores that would overflow without the running maximum
    lens, H, G, D = [200], 2, 1, 64
    a = batch((lens, H, G, D), dtype, 2)
    a["k"][150] *= 64.0
    a["q"] *= 8.0
    a["scale"] = 0.5
    q, k, v, gy = (dev(a[x], dtype) for x in ("q", "k", "v", "gy"))
    cu = dev(a["cu"], torch.int32)
    ref = reference(a, True, dtype)
    o, lse = kda.attn_fwd(q, k, v, cu, scale=0.5)
    check("o", host(o), ref[0], ref[2], dtype)
    check("lse", host(lse), ref[1], ref[3], F32)
    for x, r, e in zip(kda.attn_bwd(q, k, v, o, lse, gy, cu, scale=0.5), ref[4:7], ref[7:10]):
        check("gradient", host(x), r, e, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_other_sequences_may_hold_anything(dtype):
    lens, H, G, D = [40, 30, 70], 4, 2, 128
    a = batch((lens, H, G, D), dtype, 3)
    q, k, v, gy = (dev(a[x], dtype) for x in ("q", "k", "v", "gy"))
    cu = dev(a["cu"], torch.int32)
    o, lse = kda.attn_fwd(q, k, v, cu)
    g = kda.attn_bwd(q, k, v, o, lse, gy, cu)
    for t in (q, k, v, gy):
        t[40:70] = NAN
    o2, lse2 = kda.attn_fwd(q, k, v, cu)
    g2 = kda.attn_bwd(q, k, v, o2, lse2, gy, cu)
    for x, y in zip((o, lse) + g, (o2, lse2) + g2):
        assert torch.equal(x[:40], y[:40]) and torch.equal(x[70:], y[70:])


def test_gradients_against_differences():
    lens, H, G, D = [50, 21], 4, 2, 64
    a = batch((lens, H, G, D), F32, 4)
    q, k, v, gy = (dev(a[x]) for x in ("q", "k", "v", "gy"))
    cu = dev(a["cu"], torch.int32)
    o, lse = kda.attn_fwd(q, k, v, cu)
    g = kda.attn_bwd(q, k, v, o, lse, gy, cu)
    r = torch.Generator(device="cuda").manual_seed(0)
    h = 2.0 ** -7
    for i in range(3):
        d = torch.randn((q, k, v)[i].shape, generator=r, device="cuda")
        plus, minus = [q, k, v], [q, k, v]
        plus[i], minus[i] = plus[i] + h * d, minus[i] - h * d
        slope = ((kda.attn_fwd(*plus, cu)[0] - kda.attn_fwd(*minus, cu)[0]).double() * gy.double()).sum() / (2 * h)
        want = (g[i].double() * d.double()).sum()
        # differences of float32 outputs (2^-24 of about 7000 of them of size 1, over 2 h) and their h^2 / 6 third derivatives
        assert abs(slope - want) <= 2e-2 + 1e-3 * abs(want), (i, float(slope), float(want))


# ------------------------------------------------------------ paged cache

class Paged:
    """Requests whose tokens lie in shuffled pages; unused places hold NaN."""

    def __init__(self, held, H, G, D, page, dtype, seed=0, layers=2, layer=1):
        r = np.random.default_rng(seed)
        self.held, self.page = held, page
        self.k = [values((n, G, D), dtype, r) for n in held]
        self.v = [values((n, G, D), dtype, r) for n in held]
        count = [-(-n // page) for n in held]
        n_pages, most = sum(count) + 3, max(count + [1]) + 2
        pool = torch.full((n_pages, layers, 2, G, page, D), NAN, dtype=dtype, device="cuda")
        self.pool, self.kp, self.vp = pool, pool[:, layer, 0], pool[:, layer, 1]
        order = list(r.permutation(n_pages))
        self.rows = [[int(order.pop()) for _ in range(c)] + [10 ** 6] * (most - c) for c in count]
        self.table = dev(np.array(self.rows), torch.int32)
        self.lengths = dev(np.array(held), torch.int32)
        for b in range(len(held)):
            self.fill(b, 0, held[b], dtype)

    def fill(self, b, s, e, dtype):
        for x in range(s, e):
            p, i = self.rows[b][x // self.page], x % self.page
            self.kp[p, :, i] = dev(self.k[b][x], dtype)
            self.vp[p, :, i] = dev(self.v[b][x], dtype)


def paged_reference(c, qs, dtype, scale, there=None):
    out = [[] for _ in range(4)]
    for b, q in enumerate(qs):
        first = c.held[b] - q.shape[0]
        ok = None if there is None else there[b]
        r = O.attention(q, c.k[b], c.v[b], scale, first, True, ok) + O.bounds(q, c.k[b], c.v[b], scale, half(dtype),
                                                                            first, True, ok)
        for p, x in zip(out, r):
            p.append(x)
    return [np.concatenate(p) for p in out]


# tokens held, new tokens, heads, groups, D, page
PAGED = [([5], [1], 1, 1, 64, 16), ([500], [1], 16, 2, 128, 16), ([1, 17, 0, 64, 300], [1] * 5, 8, 2, 64, 32),
         ([700, 90, 1], [5, 5, 5], 12, 4, 128, 64), ([33, 32, 31], [1, 8, 31], 6, 6, 64, 256),
         ([400, 129], [0, 100], 4, 1, 128, 128), ([1500, 20], [64, 3], 32, 8, 64, 16), ([2100], [3], 7, 1, 128, 16)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", PAGED)
def test_paged(case, dtype):
    held, new, H, G, D, page = case
    c = Paged(held, H, G, D, page, dtype)
    r = np.random.default_rng(5)
    qs = [values((t, H, D), dtype, r, 1.5) for t in new]
    T, pad = sum(new), 2
    flat = np.full((T + 2 * pad, H, D), np.nan)
    flat[pad:pad + T] = np.concatenate(qs)
    q = wide(flat, dtype)
    cu = dev(np.concatenate([[0], np.cumsum(new)]) + pad, torch.int32)
    o_ref, lse_ref, eo, el = paged_reference(c, qs, dtype, D ** -0.5)
    o = torch.full((T + 2 * pad, H, D), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((T + 2 * pad, H), 7.0, device="cuda")
    kda.attn_paged_fwd(q, c.kp, c.vp, c.table, c.lengths, cu, o=o, lse=lse)
    w = [check("o", host(o)[pad:pad + T], o_ref, eo, dtype), check("lse", host(lse)[pad:pad + T], lse_ref, el, F32)]
    for t in (o, lse):
        assert (t[:pad] == 7.0).all() and (t[pad + T:] == 7.0).all()
    if len(set(new)) == 1 and new[0]:
        qb = q[pad:pad + T].view(len(new), new[0], H, D) if len(new) == 1 else dev(np.stack(qs), dtype)
        ob, lseb = kda.attn_paged_fwd(qb, c.kp, c.vp, c.table, c.lengths)
        check("o", host(ob).reshape(o_ref.shape), o_ref, eo, dtype)
        check("lse", host(lseb).reshape(lse_ref.shape), lse_ref, el, F32)
    say(f"[paged] {case} {dtype}: of the tolerance " + " ".join(f"{x:.2g}" for x in w))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_paged_bad_pages_and_lengths(dtype):
    # pages that are none, requests shorter than their new tokens, lengths out of range
    H, G, D, page = 4, 2, 64, 16
    held = [100, 3, 64, 40]
    c = Paged(held, H, G, D, page, dtype, 6)
    r = np.random.default_rng(7)
    qs = [values((5, H, D), dtype, r) for _ in held]
    table = c.table.clone()
    there = [np.ones(n, bool) for n in held]
    for b, col, bad in ((0, 2, -1), (0, 6, 2 ** 31 - 1), (2, 0, c.kp.shape[0]), (3, 0, -2 ** 31), (3, 1, -5), (3, 2, -1)):
        table[b, col] = bad
        there[b][col * page:(col + 1) * page] = False
    o_ref, lse_ref, eo, el = paged_reference(c, qs, dtype, D ** -0.5, there)
    q = dev(np.stack(qs), dtype)
    o, lse = kda.attn_paged_fwd(q, c.kp, c.vp, table, c.lengths)
    check("o", host(o).reshape(o_ref.shape), o_ref, eo, dtype)
    check("lse", host(lse).reshape(lse_ref.shape), lse_ref, el, F32)
    assert (o[1, :2] == 0).all() and torch.isneginf(lse[1, :2]).all()     # no such token
    assert (o[3] == 0).all() and torch.isneginf(lse[3]).all()             # no page
    lengths = c.lengths.clone()
    lengths[1] = -7
    lengths[2] = 2 ** 31 - 1          # clamped to the row: its last entries are no pages
    o2, lse2 = kda.attn_paged_fwd(q, c.kp, c.vp, table, lengths)
    assert torch.equal(o2[0], o[0]) and (o2[1] == 0).all() and torch.isneginf(lse2[1]).all()
    assert torch.isfinite(o2[2]).all()
    before = c.pool.clone()
    bad = torch.full_like(table, -1)
    bad[1] = c.kp.shape[0]
    k = dev(values((4, 5, G, D), dtype, r), dtype)
    kda.kv_append(k, k, c.kp, c.vp, bad, c.lengths)
    assert torch.equal(before.nan_to_num(9.0), c.pool.nan_to_num(9.0))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("held,new,page", [([40, 16, 1, 2], [5, 16, 1, 3], 16), ([300, 129], [200, 1], 128), ([70, 9], [0, 9], 32)])
def test_append(held, new, page, dtype):
    G, D = 3, 64
    c = Paged(held, 3, G, D, page, dtype, 8)
    want = c.pool.clone()
    T = sum(new)
    r = np.random.default_rng(9)
    k, v = values((T, G, D), dtype, r), values((T, G, D), dtype, r)
    at = 0
    for b, t in enumerate(new):
        for i in range(t):
            x = held[b] - t + i
            if x >= 0:
                p = c.rows[b][x // page]
                want[p, 1, 0, :, x % page] = dev(k[at + i], dtype)
                want[p, 1, 1, :, x % page] = dev(v[at + i], dtype)
        at += t
    cu = dev(np.concatenate([[0], np.cumsum(new)]) + 1, torch.int32)
    edge = np.full((1, G, D), np.nan)
    kda.kv_append(wide(np.concatenate([edge, k, edge]), dtype), wide(np.concatenate([edge, v, edge]), dtype), c.kp, c.vp,
                  c.table, c.lengths, cu)
    assert torch.equal(want.nan_to_num(9.0), c.pool.nan_to_num(9.0))
